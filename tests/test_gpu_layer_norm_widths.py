"""The layer norm of many aligned rows at widths around those that fill a block with one vector a thread, with a residual
and without: every layout of a row on threads, and widths beside them whose last warp has fewer columns."""
import pytest

from test_gpu_layer_norm import check_norm, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1000, 2048), (900, 4080), (900, 4096), (900, 4112), (700, 5632), (700, 6128), (700, 6144), (700, 6160),
                                       (400, 8192), (400, 12272), (400, 12288), (400, 12304), (330, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(pc, rows, cols, dtype):  # noqa: F811
    check_norm(pc, rows, cols, dtype)
    check_norm(pc, rows, cols, dtype, wtype="bf16", residual=False, offset=-2.0)
