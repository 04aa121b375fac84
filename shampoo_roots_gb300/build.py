"""Build libprecond.so in-tree with nvcc for sm_103a (no cmake; the translation units compile in parallel)."""
import os
import shutil
import subprocess
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libprecond.so")
BINDING = os.path.join(HERE, "_binding.so")      # csrc/binding.c: the operators' argument marshalling
SOURCES = ["precond.cu", "operators.cu"]
FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC"]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources_newer_than(target):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    root = os.path.dirname(HERE)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(root, "include", "precond.h")]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force=False, verbose=False):
    if not force and not sources_newer_than(OUT) and not sources_newer_than(BINDING):
        return OUT
    tmp = OUT + ".tmp"
    with tempfile.TemporaryDirectory(prefix="precond_build_") as d:
        objs = [os.path.join(d, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[nvcc()] + FLAGS + ["-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objs)]
        link = [nvcc()] + FLAGS + ["-shared", "-o", tmp] + objs
        cmds.append(["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"], "-o", BINDING + ".tmp",
                     os.path.join(CSRC, "binding.c")])
        if verbose:
            for c in cmds + [link]:
                print(" ".join(c))
        procs = [subprocess.Popen(c, cwd=CSRC) for c in cmds]
        codes = [p.wait() for p in procs]
        for c, rc in zip(cmds, codes):
            if rc:
                raise subprocess.CalledProcessError(rc, c)
        subprocess.run(link, check=True, cwd=CSRC)
    os.replace(BINDING + ".tmp", BINDING)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose=True))
