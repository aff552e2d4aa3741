"""What include/wtconv.h promises of the 8-bit norm's roundings, against the float32 values that it rounds."""
import numpy as np
import pytest
import torch

import memory_bound_cnn_wtconv_b200 as wt
import map_reference as ref
from test_maps import BF16, EPS, F32, U, check_forward, close, gen_of, make, wide

pytestmark = pytest.mark.gpu

# The roundings are counted in u = 2^-24, float32's half step.
TOPS = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def half_step(t, kind):
    """Half the distance between the 8-bit numbers around t."""
    if kind == torch.int8:
        return np.full_like(t, 0.5)
    return 0.5 * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(t), 1e-300))), -6.0) - 3.0)


@pytest.mark.parametrize("kind", list(TOPS), ids=["e4m3", "int8"])
@pytest.mark.parametrize("shape,layout", [((300, 768, 1, 1), "rows"), ((300, 101, 1, 1), "rows"), ((2, 96, 16, 16), "nhwc"),
                                          ((2, 96, 16, 16), "nchw"), ((2, 101, 9, 7), "nchw"), ((3, 40, 10, 3), "nchw")], ids=str)
def test_scales_and_values(shape, layout, kind):
    gen = gen_of("rounding", shape, layout)
    x = make(shape, layout, F32, gen)
    w = torch.randn(shape[1], generator=gen).cuda()
    # With one group a row the 8-bit norm sums as the float32 norm does, so y holds the very values that it rounds.
    v = wide(wt.rms_norm_forward(x, w, eps=EPS)[0])
    q, scale, _ = wt.rms_norm_q8(x, w, None, EPS, kind)
    s, top = wide(scale), TOPS[kind]
    want = np.maximum(np.abs(v).max(axis=1, keepdims=True) / top, 2.0 ** -126)
    close(s, want, 2.01 * U * want, "scale")  # two roundings
    t = v / s
    close(wide(q.float()), t, half_step(t, kind) + 3.01 * U * np.abs(t), "q")  # three units before the 8-bit rounding


def test_values_next_to_a_tie():
    # The largest value of a row is the type's largest number, so the quotients are the inputs, off by 8 * 2^-24 at most
    # (v and the largest v one rounding each, the scale two, the quotient three): 2^-18 from a tie decides its side.
    near = 2.0 ** -18
    for kind, top, mids in ((torch.int8, 127.0, [0.5, 1.5, 2.5, 63.5]), (torch.float8_e4m3fn, 448.0, [1.0625, 1.1875, 34.0, 248.0])):
        for side in (-1, 1):
            row = torch.tensor([[top] + [m * (1 + side * near) for m in mids] + [0.0] * 3], device="cuda")
            q = wt.rms_norm_q8(row, torch.ones(8, device="cuda"), dtype=kind)[0].float()[0, 1:5].tolist()
            for got, m in zip(q, mids):
                assert (got - m) * side > 0, (kind, m, side, got)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape", [(2, 96, 8, 8), (1, 40, 16, 4), (3, 130, 9, 7), (1, 1024, 4, 4)], ids=str)
def test_unaligned_buffers(shape, layout, dtype):
    # One element off, both 8-bit types, with and without a residual: every value of q, scale and h.
    gen = gen_of("unaligned q8", shape, layout)
    x, res = make(shape, layout, dtype, gen, shift=1), make(shape, layout, dtype, gen, shift=1)
    C = shape[1]
    w = torch.randn(C + 1, generator=gen).cuda()[1:]
    tol = ((C + 1) / 2 + 10) * U
    for residual in (None, res):
        for kind, top in TOPS.items():
            for group in (0, 32, 64, 128):
                q = torch.empty(x.numel() + 1, dtype=torch.int8, device="cuda")[1:].view(kind).as_strided(x.shape, x.stride())
                q, scale, h = wt.rms_norm_q8(x, w, residual, EPS, kind, group, q=q)
                if residual is None:
                    assert h is x
                else:
                    assert torch.equal(h, wt.rms_norm_forward(x, w, residual, eps=EPS)[1])
                    check_forward(x, residual, w, None, *wt.rms_norm_forward(x, w, residual, eps=EPS))
                v, _ = ref.norm(wide(h), w.double().cpu().numpy(), EPS)
                want = np.maximum(ref.group_max(v, group or C) / top, 2.0 ** -126)
                close(wide(scale), want, tol * want, "scale")
                s = np.repeat(wide(scale), group or C, axis=1)[:, :C]
                t = v / s
                close(wide(q.float()), t, half_step(t, kind) * (1 + 4 * tol) + 4 * tol * np.abs(t), "q")
