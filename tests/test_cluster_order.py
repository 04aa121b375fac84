"""Distributed shared memory may be touched only when every block of the cluster has begun: each kernel that reaches
another block's shared memory has to pass a cluster barrier first.  Read off the kernels' source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "shampoo_roots_gb300", "csrc")
REMOTE = r"map_shared_rank|\bmapa\b|multicast::cluster|cta_group::2\.shared::cluster"
BARRIER = r"cluster\w*(?:\(\))?\.sync\(\)|barrier\.cluster\.wait"


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def functions(text):
    """(name, is a kernel, body) of every function that is marked for the device."""
    out = []
    for m in re.finditer(r"__(global|device)__\s[^;{}]*?\b(\w+)\s*\((?:[^(){};]|\([^(){};]*\))*\)\s*(?:const\s*)?\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out.append((m.group(2), m.group(1) == "global", text[m.end():i]))
    return out


def first(pattern, body):
    m = re.search(pattern, body)
    return m.start() if m else None


def spread(pattern, funcs):
    """The pattern, or a call of a device function that contains it, directly or through others."""
    names = set()
    while True:
        p = pattern + "".join(r"|\b%s\s*(?:<[^;(]*>)?\(" % n for n in sorted(names))
        more = {n for n, kernel, body in funcs if not kernel and first(p, body) is not None} - names
        if not more:
            return p
        names |= more


def late(sources):
    """Kernels that reach another block's shared memory, and those of them that do so before any cluster barrier."""
    funcs = [f for text in sources for f in functions(without_comments(text))]
    remote, barrier = spread(REMOTE, funcs), spread(BARRIER, funcs)
    reach, wrong = set(), set()
    for name, kernel, body in funcs:
        if not kernel or first(remote, body) is None:
            continue
        reach.add(name)
        at = first(barrier, body)
        if at is None or at > first(remote, body):
            wrong.add(name)
    return reach, wrong


def test_remote_shared_memory_comes_after_a_cluster_barrier():
    sources = [open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cuh")))]
    reach, wrong = late(sources)
    assert {"rms_norm_kernel", "rms_grad_kernel", "gemm8_kernel", "gemm8_pair_kernel", "distill_kernel"} <= reach
    assert not wrong, sorted(wrong)


@pytest.mark.parametrize("body,ok", [
    ("cluster.sync(); *cluster.map_shared_rank(p, 1) = 0;", True), ("*cluster.map_shared_rank(p, 1) = 0; cluster.sync();", False),
    ("put(p); cluster.sync();", False), ("meet(); put(p);", True), ("// cluster.sync();\n put(p);", False)])
def test_the_reading(body, ok):
    source = ("__device__ void put(int* p) { *cluster.map_shared_rank(p, 1) = 0; }\n"
              "__device__ void meet() { asm volatile(\"barrier.cluster.wait.acquire.aligned;\"); }\n"
              "__global__ void k(int* p) { %s }\n" % body)
    assert late([source]) == ({"k"}, set() if ok else {"k"})
