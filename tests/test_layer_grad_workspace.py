"""The workspace of the layer norm's gradients has room for the sums of dw and db of every block that a call may launch:
the rule of the launches (host.h, compiled for the host) over types, alignments, rows and columns, against what the
library asks for."""
import os
import shutil
import subprocess

import pytest

import shampoo_roots_gb300 as sr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COLS = [1, 15, 16, 17, 64, 100, 128, 129, 200, 256, 257, 272, 500, 512, 513, 1000, 2048, 4096, 6144, 6145, 8192, 8193, 12288, 12289,
        24576, 24577, 32768, 32769, 49152, 49153, 65536, 65537, 100000]
ROWS = [1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 152, 153, 304, 305, 400, 1000, 1216, 1217, 2432, 2433, 3000,
        4864, 4865, 7296, 9728, 10000, 20000, 32768, 1000000, 1 << 30]

PROGRAM = r'''
#include <cstdio>
#include "host.h"
using namespace precond;
// for every pair of rows and columns: the most blocks that leave sums, and whether every form of the rows needs none
int main() {
  long long rows, cols;
  while (scanf("%lld %lld", &rows, &cols) == 2) {
    int64_t most = 0;
    bool whole = true;
    for (int dtype : {PRECOND_F32, PRECOND_BF16})
      for (bool vec : {false, true}) {
        const RowShape s = layer_grad_shape(cols, dtype, vec);
        most = std::max(most, layer_grad_blocks(s, rows, dtype, PLAN_SMS, PLAN_CLUSTERS));
        whole = whole && layer_grad_whole(s, rows);
      }
    // rows that come through shared memory: a block an SM
    printf("%lld %d\n", (long long)std::max(most, std::min<int64_t>(rows, PLAN_SMS)), whole);
  }
}
'''


def test_room_for_every_block(tmp_path):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "blocks.cu", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                    os.path.join(ROOT, "shampoo_roots_gb300", "csrc"), "-o", str(exe), str(src)], check=True, capture_output=True)
    cases = [(r, c) for c in COLS for r in ROWS]
    out = subprocess.run([str(exe)], input="".join("%d %d\n" % x for x in cases), capture_output=True, text=True, check=True).stdout
    lines = out.split("\n")[:-1]
    assert len(lines) == len(cases)
    for (rows, cols), line in zip(cases, lines):
        most, whole = (int(v) for v in line.split())
        need = sr.precond_layer_norm_grad_workspace(rows, cols)
        room = need // 8 // (-(-cols // 16) * 16)
        assert room >= most if need else whole, (rows, cols, room, most)
