"""Build libprecond.so in-tree with nvcc for sm_103a (no cmake; the translation units compile in parallel), and beside
it _binding.so, the operators' argument marshalling for Python, with the C compiler and CPython's headers."""
import os
import shutil
import subprocess
import sysconfig
import tempfile
import warnings

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


def sources_newer_than(target, names=None):
    """Whether one of the sources (all of csrc and the header, or `names` of csrc) is newer than the target."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    root = os.path.dirname(HERE)
    deps = [os.path.join(CSRC, f) for f in names or os.listdir(CSRC)]
    if names is None:
        deps.append(os.path.join(root, "include", "precond.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force=False, verbose=False):
    """Builds what is older than its sources.  The library needs nvcc alone: where only the binding cannot be built, that
    is a warning, and importing the operators says that it is missing."""
    library = force or sources_newer_than(OUT)
    binding = force or sources_newer_than(BINDING, ["binding.c"])
    with tempfile.TemporaryDirectory(prefix="precond_build_") as d:
        objs = [os.path.join(d, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[nvcc()] + FLAGS + ["-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objs)] if library else []
        procs = [_start(c, verbose) for c in cmds]
        why = _build_binding(verbose) if binding else None
        codes = [p.wait() for p in procs]
        for c, rc in zip(cmds, codes):
            if rc:
                raise subprocess.CalledProcessError(rc, c)
        if library:
            tmp = OUT + ".tmp"
            link = [nvcc()] + FLAGS + ["-shared", "-o", tmp] + objs
            rc = _start(link, verbose).wait()
            if rc:
                raise subprocess.CalledProcessError(rc, link)
            os.replace(tmp, OUT)
    if why:
        warnings.warn(f"the operators' Python binding was not built ({why}); the library was")
    return OUT


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, cwd=CSRC)


def _build_binding(verbose):
    """None, or why it could not be built; then one of older sources goes too."""
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"], "-o", BINDING + ".tmp",
           os.path.join(CSRC, "binding.c")]
    try:
        rc = _start(cmd, verbose).wait()
        why = f"gcc returned {rc}" if rc else None
    except OSError as e:
        why = str(e)
    if why is None:
        os.replace(BINDING + ".tmp", BINDING)
    elif os.path.exists(BINDING):
        os.remove(BINDING)
    return why


if __name__ == "__main__":
    print(build(force=True, verbose=True))
