"""The RMS norm's backward where 1 / rms is very large or very small: its result is a float32 number although the
cube of 1 / rms is none."""
import pytest
import torch

import memory_bound_cnn_wtconv_b200 as wt
from test_maps import BF16, F32, check_backward, gen_of, make

pytestmark = pytest.mark.gpu

# All numbers of a case, its sums of up to 16401 squares among them, are normal in float32; so the tolerances are those of
# ordinary sizes.  Planes of whole chunks, of half chunks (in bf16, in fp32), ragged ones, buffers off their alignment, and
# many channels.
PLANES = [((2, 12, 4, 8), 0), ((2, 12, 3, 4), 0), ((2, 12, 3, 6), 0), ((2, 13, 3, 5), 0), ((2, 12, 4, 8), 1), ((1, 300, 3, 5), 0)]
# Chunks, single channels, rows of a CTA, and rows longer than its registers.
ROWS = [(9, 16, 1, 1), (9, 11, 1, 1), (3, 1200, 1, 1), (3, 1201, 1, 1), (2, 16400, 1, 1), (2, 16401, 1, 1)]


def check(shape, layout, dtype, size, dsize, eps, shift=0):
    gen = gen_of(shape, layout, size)
    h, dh = make(shape, layout, dtype, gen, size, shift), make(shape, layout, dtype, gen, dsize / size if size else 1.0, shift)
    dy = make(shape, layout, dtype, gen, dsize, shift)
    w = torch.randn(shape[1], generator=gen).cuda()
    _, _, rstd = wt.rms_norm_forward(h, w, eps=eps)
    for extra in (None, dh):
        dx, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, extra)
        assert torch.isfinite(dres).all()
        check_backward(h, dy, extra, w, None, dx, dres, dw, eps)
        drop = wt.Drop(0.3, "element", 5)
        check_backward(h, dy, extra, w, drop, *wt.rms_norm_backward(h, dy, w, rstd, extra, drop), eps)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,shift", PLANES, ids=str)
@pytest.mark.parametrize("size,dsize,eps", [(0.0, 1.0, 1e-28), (1e14, 1.0, 1e-6), (1e16, 1.0, 1e-6), (1e17, 1e-8, 1e-6),
                                            (1e-15, 1e10, 1e-36)], ids=str)
def test_planes(shape, shift, size, dsize, eps, dtype):
    check(shape, "nchw", dtype, size, dsize, eps, shift)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("size,dsize,eps", [(0.0, 1.0, 1e-28), (1e14, 1.0, 1e-6), (1e16, 1.0, 1e-6), (1e17, 1e-8, 1e-6),
                                            (1e-15, 1e10, 1e-36)], ids=str)
def test_rows(shape, size, dsize, eps, dtype):
    check(shape, "rows", dtype, size, dsize, eps)
