"""Layer norm over so many rows that a thread group walks many of them: the ring
is refilled, the 32 rows' statistics a lane holds are exchanged, rows that do
not start on a vector share it with their neighbours, and dw and db add up over
the group's rows.  Same checks as test_gpu_training's, element by element."""
import pytest

import test_gpu_training as base

pytestmark = pytest.mark.gpu

jg = base.jg
# odd widths of each class of threads a row (32 .. 512), and aligned ones; 90000 x 33 and 90000 x 40 give a group 37 rows
SHAPES = [(5000, 129, 0), (20000, 131, 0), (90000, 33, 0), (90000, 40, 0), (9000, 333, 0), (6000, 777, 0), (6000, 776, 0),
          (2500, 1537, 0), (700, 4093, 0), (700, 4096, 0), (400, 7001, 0), (400, 8185, 0), (400, 8192, 0), (700, 129, 1),
          (700, 8200, 0)]


@pytest.mark.parametrize("xt,yt", base.LN_TYPES)
@pytest.mark.parametrize("rows,dim,shift", SHAPES)
def test_forward(jg, rows, dim, shift, xt, yt):
    base.test_layernorm_fwd(jg, rows, dim, shift, xt, yt)


@pytest.mark.parametrize("xt,yt", base.LN_TYPES)
@pytest.mark.parametrize("rows,dim,shift", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_backward(jg, rows, dim, shift, xt, yt, res):
    base.test_layernorm_bwd(jg, rows, dim, shift, xt, yt, res)
