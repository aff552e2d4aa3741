"""Map operators (dropout, RMS norm over channels) on a B200, against plain float64 forms.

Tolerances, all derived: u = 2^-24 is float32's half step, `half(dtype)` the
stored type's (bf16 2^-8, fp32 2^-24, e4m3 2^-4).  A sum of C positive terms
is off by at most (C + 1) u relative to itself, whatever its order; the square
root halves that; each further operation adds u (rsqrtf two units in the last
place, 4 u).  A sum of terms of both signs is off by at most (C + 1) u times
the sum of their sizes.
"""
import zlib

import numpy as np
import pytest
import torch

import map_reference as ref
import memory_bound_cnn_wtconv_b200 as wt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
F32, BF16 = torch.float32, torch.bfloat16

# (B, C, H, W): one element; single rows and pixels; odd, ragged and vector-sized extents; planes that end inside a
# tile of pixels; channel counts around every way the kernels hold a row, and past them all.
MAPS = [(1, 1, 1, 1), (2, 37, 14, 14), (1, 96, 10, 9), (1, 3, 1, 1), (2, 1, 5, 7), (3, 5, 7, 7), (2, 8, 4, 4), (1, 17, 3, 11), (2, 96, 8, 8),
        (2, 101, 9, 5), (1, 130, 4, 12), (3, 64, 12, 11), (2, 192, 7, 7), (1, 320, 5, 8), (1, 768, 7, 7),
        (1, 1000, 2, 3), (1, 1030, 2, 8), (1, 2050, 1, 9), (1, 4100, 2, 4), (1, 9000, 1, 8), (1, 33000, 1, 2)]
ROWS = [(1, 1), (1, 7), (5, 8), (33, 96), (300, 100), (1, 768), (7, 1024), (3, 2048), (2, 4096), (2, 8200), (1, 33001)]


def half(dtype):
    return torch.finfo(dtype).eps / 2


def cases():
    out = []
    for s in MAPS:
        for layout in ("nchw", "nhwc"):
            out.append((s, layout))
    return out + [((n, c, 1, 1), "rows") for n, c in ROWS]


def make(shape, layout, dtype, gen, scale=1.0, shift=0):
    """A random activation; `shift` elements off its allocation's alignment."""
    B, C, H, W = shape
    size = (B, C) if layout == "rows" else shape
    t = (torch.randn(B * C * H * W + shift, generator=gen) * scale).to(dtype).cuda()[shift:]
    if layout == "nhwc":
        return t.view(B, H, W, C).permute(0, 3, 1, 2)
    return t.view(size)


def wide(t):
    """float64 [B, C, P] on the host."""
    return t.detach().double().cpu().reshape(t.shape[0], t.shape[1], -1).numpy()


def gen_of(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def close(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} times the tolerance"


def check_forward(x, residual, weight, drop, y, h, rstd, eps=EPS):
    C = x.shape[1]
    hw = wide(h)
    if residual is not None:
        keep = None
        if drop is not None:
            off = int(drop.offset) if not isinstance(drop.offset, torch.Tensor) else int(drop.offset.item())
            keep = ref.keep_mask(*wide(x).shape, drop.p, drop.mode, drop.seed & (2 ** 64 - 1), off)
        want = ref.join(wide(x), wide(residual), keep, drop.p if drop else 0.0)
        # one rounding to float32 and one to the stored type
        close(hw, want, (half(h.dtype) + 1.01 * U) * np.abs(want), "h")
    else:
        assert h is x
    want, r = ref.norm(hw, weight.double().cpu().numpy(), eps)
    tol = ((C + 1) / 2 + 8) * U
    close(wide(y), want, (tol + half(y.dtype) * (1 + tol)) * np.abs(want), "y")
    if rstd is not None:
        close(rstd.double().cpu().numpy().reshape(r.shape), r, tol * r, "rstd")


def check_backward(h, dy, dh, weight, drop, dx, dres, dw, eps=EPS):
    C, w = h.shape[1], weight.double().cpu().numpy()
    hw, dyw = wide(h), wide(dy)
    d, dweight = ref.norm_grad(hw, w, eps, dyw, None if dh is None else wide(dh))
    _, r = ref.norm(hw, w, eps)
    g = dyw * w[None, :, None]
    parts = np.abs(r * g) + (0.0 if dh is None else np.abs(wide(dh)))
    lin = np.abs(hw) * r ** 3 * np.abs(g * hw).mean(axis=1, keepdims=True)
    # r is off by ((C + 1) / 2 + 8) u and enters up to three times; the sum of g * h by (C + 2) u of its terms' sizes
    tol = ((C / 2 + 14) * parts + (2.5 * C + 40) * lin) * U
    if dres is not None:
        close(wide(dres), d, tol + half(dres.dtype) * (np.abs(d) + tol), "dres")
    if dx is not None and drop is not None:
        off = int(drop.offset) if not isinstance(drop.offset, torch.Tensor) else int(drop.offset.item())
        keep = ref.keep_mask(*hw.shape, drop.p, drop.mode, drop.seed, off)
        want = np.where(keep, d * ref.grown(drop.p), 0.0)
        close(wide(dx), want, (tol * ref.grown(drop.p) + (half(dx.dtype) + 2 * U) * (np.abs(want) + tol)) * keep, "dx")
    if dw is not None:
        N = hw.shape[0] * hw.shape[2]
        size = (np.abs(dyw * hw) * r).sum(axis=(0, 2))
        close(dw.double().cpu().numpy(), dweight, (N + C / 2 + 14) * U * size + 1e-300, "dweight")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,layout", cases(), ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_norm_forward_and_backward(shape, layout, dtype):
    gen = gen_of(shape, layout, str(dtype))
    x, res, dy, dh = (make(shape, layout, dtype, gen) for _ in range(4))
    w = torch.randn(shape[1], generator=gen).cuda()
    y, h, rstd = wt.rms_norm_forward(x, w, eps=EPS)
    check_forward(x, None, w, None, y, h, rstd)
    check_backward(h, dy, None, w, None, *wt.rms_norm_backward(h, dy, w, rstd))
    y, h, rstd = wt.rms_norm_forward(x, w, res, eps=EPS)
    check_forward(x, res, w, None, y, h, rstd)
    dx, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, dh)
    assert dx is dres
    check_backward(h, dy, dh, w, None, dx, dres, dw)
    for mode in ("element", "channel", "sample"):
        drop = wt.Drop(0.4, mode, 0x1234567890ABCDEF, 5)
        y, h, rstd = wt.rms_norm_forward(x, w, res, drop, EPS)
        check_forward(x, res, w, drop, y, h, rstd)
        check_backward(h, dy, dh, w, drop, *wt.rms_norm_backward(h, dy, w, rstd, dh, drop))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_norm_q8(dtype, kind, group, residual):
    for shape, layout in cases():
        gen = gen_of(shape, layout, group)
        x = make(shape, layout, dtype, gen)
        res = make(shape, layout, dtype, gen) if residual else None
        w = torch.randn(shape[1], generator=gen).cuda()
        q, scale, h = wt.rms_norm_q8(x, w, res, EPS, kind, group)
        assert q.dtype == kind and q.shape == x.shape and q.stride() == x.stride()
        if residual:
            check_forward(x, res, w, None, *wt.rms_norm_forward(x, w, res, eps=EPS))
            assert torch.equal(h, wt.rms_norm_forward(x, w, res, eps=EPS)[1])
        else:
            assert h is x
        C = shape[1]
        v, _ = ref.norm(wide(h), w.double().cpu().numpy(), EPS)
        G = group or C
        top = 448.0 if kind == torch.float8_e4m3fn else 127.0
        want = np.maximum(ref.group_max(v, G) / top, 2.0 ** -126)
        tol = ((C + 1) / 2 + 10) * U
        got = wide(scale)
        close(got, want, tol * want, f"scale {shape} {layout}")
        s = np.repeat(got, G, axis=1)[:, :C]
        qv = wide(q.float() if kind == torch.int8 else q.to(torch.float32))
        assert np.abs(qv).max() <= top
        # half a step of the 8-bit type (e4m3: 2^-4 of the value, 2^-10 below its smallest normal), and the arithmetic
        step = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) if top == 448.0 else 0.5 * s
        close(qv * s, v, step * (1 + 4 * tol) + 4 * tol * np.abs(v), f"q {shape} {layout}")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("mode", ["element", "channel", "sample"])
def test_dropout(dtype, mode):
    for shape, layout in cases():
        gen = gen_of(shape, layout, mode)
        x, res = make(shape, layout, dtype, gen), make(shape, layout, dtype, gen)
        for p in (0.0, 0.3, 0.9):
            drop = wt.Drop(p, mode, 99, (1 << 32) + 17)  # the offset counts modulo 2^32
            keep = ref.keep_mask(*wide(x).shape, p, mode, 99, 17)
            for r in (None, res):
                y = wt.dropout_forward(x, drop, r)
                want = ref.join(wide(x), None if r is None else wide(r), keep, p)
                close(wide(y), want, (half(dtype) + 1.01 * U) * np.abs(want), f"{shape} {layout} {p}")
            dx = wt.dropout_backward(x, drop)
            assert torch.equal(dx, wt.dropout_forward(x, drop))
            assert dx.stride() == x.stride()


def test_mask_is_the_same_in_both_layouts_types_and_operators():
    shape, gen = (3, 22, 9, 8), gen_of("layouts")
    x, res = make(shape, "nchw", F32, gen), make(shape, "nchw", F32, gen)
    cl = dict(memory_format=torch.channels_last)
    w = torch.randn(22, generator=gen).cuda()
    for mode in ("element", "channel", "sample"):
        drop = wt.Drop(0.5, mode, 3, 4)
        y = wt.dropout_forward(x, drop, res)
        assert torch.equal(y, wt.dropout_forward(x.contiguous(**cl), drop, res.contiguous(**cl)))
        ny, h, _ = wt.rms_norm_forward(x, w, res, drop)
        assert torch.equal(h, y)
        ones = torch.ones_like(x)
        assert torch.equal(wt.dropout_forward(ones, drop) != 0, wt.dropout_forward(ones.bfloat16(), drop) != 0)
    rows = wt.dropout_forward(torch.ones(5, 22, device="cuda"), wt.Drop(0.5, "element", 3, 4))
    assert torch.equal(rows, wt.dropout_forward(torch.ones(5, 22, 1, 1, device="cuda"), wt.Drop(0.5, "element", 3, 4))[:, :, 0, 0])


# Channel counts on both sides of every border at which the kernels hold a row in another way.
WIDTHS = [2, 4, 9, 16, 31, 32, 33, 40, 63, 64, 65, 96, 127, 128, 129, 192, 255, 256, 257, 320, 384, 511, 512, 513, 640,
          1000, 1024, 1025, 1536, 2048, 2049, 4096, 4097, 8191, 8192, 8193, 16384, 16385, 16392]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout,hw", [("rows", (1, 1)), ("nchw", (2, 8)), ("nchw", (1, 7)), ("nchw", (3, 43)), ("nchw", (2, 6)),
                                       ("nchw", (1, 10))])
def test_every_width(layout, hw, dtype):
    for C in WIDTHS:
        shape = (3 if layout == "rows" else 1, C, *hw)
        gen = gen_of("width", C, layout, hw)
        x, res, dy = (make(shape, layout, dtype, gen) for _ in range(3))
        w = torch.randn(C, generator=gen).cuda()
        drop = wt.Drop(0.3, "element", C, 1)
        y, h, rstd = wt.rms_norm_forward(x, w, res, drop, EPS)
        check_forward(x, res, w, drop, y, h, rstd)
        check_backward(h, dy, None, w, drop, *wt.rms_norm_backward(h, dy, w, rstd, None, drop))
        check_backward(h, dy, res, w, None, *wt.rms_norm_backward(h, dy, w, rstd, res))
        for group in (0, 32, 128):
            q, scale, _ = wt.rms_norm_q8(h, w, None, EPS, torch.int8, group)
            v, _ = ref.norm(wide(h), w.double().cpu().numpy(), EPS)
            tol, s = ((C + 1) / 2 + 10) * U, np.repeat(wide(scale), group or C, axis=1)[:, :C]
            close(wide(scale), np.maximum(ref.group_max(v, group or C) / 127.0, 2.0 ** -126), tol * wide(scale), "scale")
            close(wide(q) * s, v, 0.5 * s * (1 + 4 * tol) + 4 * tol * np.abs(v), "q")


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 147, 148, 149, 1183, 1185, 5000])
def test_few_and_many_rows(rows):
    # Row counts around those at which CTAs shrink or start to walk.
    for C in (6, 24, 96, 520):
        gen = gen_of("rows", rows, C)
        x, dy = make((rows, C, 1, 1), "rows", F32, gen), make((rows, C, 1, 1), "rows", F32, gen)
        w = torch.randn(C, generator=gen).cuda()
        y, h, rstd = wt.rms_norm_forward(x, w, eps=EPS)
        check_forward(x, None, w, None, y, h, rstd)
        check_backward(h, dy, None, w, None, *wt.rms_norm_backward(h, dy, w, rstd))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 4, 5, 8, 12, 16, 17])
def test_narrow_rows(C, dtype):
    # Rows of one or two chunks, or of few single channels: a thread or a few own one, and CTAs walk many of them.
    shape, layout = (2, C, 181, 211), "nhwc"
    gen = gen_of("narrow", C, dtype)
    x, res, dy = (make(shape, layout, dtype, gen) for _ in range(3))
    w = torch.randn(C, generator=gen).cuda()
    drop = wt.Drop(0.4, "element", C, 3)
    y, h, rstd = wt.rms_norm_forward(x, w, res, drop, EPS)
    check_forward(x, res, w, drop, y, h, rstd)
    check_backward(h, dy, res, w, drop, *wt.rms_norm_backward(h, dy, w, rstd, res, drop))
    v, _ = ref.norm(wide(h), w.double().cpu().numpy(), EPS)
    q, scale, _ = wt.rms_norm_q8(h, w, None, EPS, torch.int8)
    tol, s = ((C + 1) / 2 + 10) * U, np.repeat(wide(scale), C, axis=1)
    close(wide(scale), np.maximum(ref.group_max(v, C) / 127.0, 2.0 ** -126), tol * wide(scale), "scale")
    close(wide(q) * s, v, 0.5 * s * (1 + 4 * tol) + 4 * tol * np.abs(v), "q")


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 96, 8, 8), (1, 40, 16, 4), (1, 1024, 4, 4)], ids=str)
def test_unaligned_buffers(shape, dtype, layout):
    # One element off: every 16-byte path has to give way.
    gen = gen_of("unaligned", shape)
    x, res, dy, dh = (make(shape, layout, dtype, gen, shift=1) for _ in range(4))
    w = torch.randn(shape[1] + 1, generator=gen).cuda()[1:]
    drop = wt.Drop(0.25, "element", 1, 1)
    y, h, rstd = wt.rms_norm_forward(x, w, res, drop, EPS)
    check_forward(x, res, w, drop, y, h, rstd)
    out = [make(shape, layout, dtype, gen, shift=1) for _ in range(2)]
    dx, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, dh, drop, out[0], out[1])
    assert dx is out[0] and dres is out[1]
    check_backward(h, dy, dh, w, drop, dx, dres, dw)
    aligned = [t.clone() for t in (x, res)]
    assert torch.equal(wt.dropout_forward(x, drop, res), wt.dropout_forward(*aligned[:1], drop, aligned[1]))
    q, s, _ = wt.rms_norm_q8(x, w, res, EPS, group=32)
    q2, s2, _ = wt.rms_norm_q8(aligned[0], w, aligned[1], EPS, group=32)
    # another summing order: scales within its bound (half a step of the sum, twice)
    assert (s / s2 - 1).abs().max() <= (shape[1] + 20) * U and q.shape == q2.shape


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_unaligned_groups_of_larger_maps(group, dtype, layout):
    # Enough pixels that the kernels for unaligned buffers put all lanes of a warp along them.
    shape, gen = (8, 300, 32, 32), gen_of("groups", group, layout)
    x = make(shape, layout, dtype, gen, shift=1)
    w = torch.randn(300, generator=gen).cuda()
    q, scale, _ = wt.rms_norm_q8(x, w, None, EPS, torch.int8, group)
    v, _ = ref.norm(wide(x), w.double().cpu().numpy(), EPS)
    tol, s = (301 / 2 + 10) * U, np.repeat(wide(scale), group or 300, axis=1)[:, :300]
    close(wide(scale), ref.group_max(v, group or 300) / 127.0, tol * wide(scale), "scale")
    close(wide(q) * s, v, 0.5 * s * (1 + 4 * tol) + 4 * tol * np.abs(v), "q")
    # the largest value of each group is its top
    assert (np.concatenate([np.abs(wide(q))[:, k:k + (group or 300)].max(1) for k in range(0, 300, group or 300)]) == 127).all()


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_infinities_and_nan(layout):
    shape, gen = (2, 24, 4, 8), gen_of("nan", layout)
    x, res = make(shape, layout, F32, gen), make(shape, layout, F32, gen)
    w = torch.ones(24, device="cuda")
    drop = wt.Drop(0.5, "element", 7, 0)
    keep = torch.from_numpy(ref.keep_mask(2, 24, 32, 0.5, "element", 7, 0).copy()).view(shape).cuda()
    # Dropped places count as 0, whatever they hold.
    dirty = torch.where(keep, x, float("nan")).contiguous(memory_format=torch.channels_last if layout == "nhwc" else torch.contiguous_format)
    assert torch.equal(wt.dropout_forward(dirty, drop, res), wt.dropout_forward(x, drop, res))
    assert torch.equal(wt.rms_norm_forward(dirty, w, res, drop)[0], wt.rms_norm_forward(x, w, res, drop)[0])
    # A NaN stays in its pixel, and spoils all of it; an infinity leaves the others 0.
    x[0, 5, 1, 2], x[1, 3, 0, 0] = float("nan"), float("inf")
    y = wt.rms_norm_forward(x, w)[0]
    bad = torch.zeros(shape, dtype=torch.bool, device="cuda")
    bad[0, :, 1, 2], bad[1, 3, 0, 0] = True, True
    assert torch.equal(torch.isnan(y), bad)
    assert (y[1, torch.arange(24) != 3, 0, 0] == 0).all()
    for kind in (torch.float8_e4m3fn, torch.int8):
        q, s, _ = wt.rms_norm_q8(x, w, dtype=kind)
        lost = torch.zeros(2, 1, 4, 8, dtype=torch.bool, device="cuda")
        lost[0, 0, 1, 2], lost[1, 0, 0, 0] = True, True
        assert torch.equal(torch.isnan(s), lost)
        if kind == torch.int8:
            assert (q[0, :, 1, 2] == 0).all() and (q[1, :, 0, 0] == 0).all()
        else:
            assert torch.equal(torch.isnan(q.float()), lost.expand(shape))


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 10, 7, 7), (1, 70, 9, 9), (2, 16, 8, 8), (1, 300, 3, 5)], ids=str)
def test_infinite_values_stay_in_their_channel(shape, dtype, layout):
    # The first and last pixels of one channel's plane: what a kernel reads beyond a plane's or row's end must not
    # reach its neighbours' sums.
    gen = gen_of("inf", shape, layout)
    h, dy = make(shape, layout, dtype, gen), make(shape, layout, dtype, gen)
    w = torch.ones(shape[1], device="cuda")
    rstd = torch.ones(shape[0], shape[2], shape[3], device="cuda")
    c = 5
    for b in range(shape[0]):
        for y, x in ((0, 0), (0, 1), (shape[2] - 1, shape[3] - 1)):
            dy[b, c, y, x] = float("nan")
            h[b, c + 2, y, x] = float("inf")
    dx, _, dw = wt.rms_norm_backward(h, dy, w, rstd)
    bad = torch.zeros(shape[1], dtype=torch.bool, device="cuda")
    bad[[c, c + 2]] = True
    assert torch.equal(~torch.isfinite(dw), bad)
    pixels = torch.zeros_like(rstd, dtype=torch.bool)
    pixels[:, 0, :2] = pixels[:, -1, -1] = True
    assert torch.equal(torch.isfinite(dx).all(dim=1), ~pixels)


def test_zero_rows_and_the_largest_values():
    x = torch.zeros(3, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    y, _, rstd = wt.rms_norm_forward(x, w, eps=1e-6)
    assert not y.any() and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    q, s, _ = wt.rms_norm_q8(x, w)
    assert not q.float().any() and (s == 2.0 ** -126).all()
    # a row whose squares overflow float32: 1 / infinity, as the formula in float32 gives
    assert not wt.rms_norm_forward(torch.full((1, 40), 1e30, device="cuda"), w)[0].any()
    dx, _, dw = wt.rms_norm_backward(x, torch.ones_like(x), w, rstd)
    assert torch.allclose(dx, torch.full_like(dx, 1e3), rtol=1e-6) and not dw.any()


def test_empty_batch():
    w = torch.ones(6, device="cuda")
    for x in (torch.empty(0, 6, device="cuda"), torch.empty(0, 6, 3, 4, device="cuda"),
              torch.empty(0, 6, 3, 4, device="cuda").to(memory_format=torch.channels_last)):
        y, h, rstd = wt.rms_norm_forward(x, w, x.clone(), wt.Drop(0.1))
        dx, dres, dw = wt.rms_norm_backward(h, y, w, rstd, drop=wt.Drop(0.1), dweight=torch.full_like(w, 7.0))
        assert y.shape == dx.shape == dres.shape == x.shape and not dw.any()
        q, s, _ = wt.rms_norm_q8(x, w, group=32)
        assert q.shape == x.shape and s.shape[0] == 0
        assert wt.dropout_forward(x, wt.Drop(0.1)).shape == x.shape


def test_gradients_that_are_not_asked_for():
    gen = gen_of("asked")
    x, res, dy = (make((2, 20, 4, 4), "nchw", F32, gen) for _ in range(3))
    w, drop = torch.ones(20, device="cuda"), wt.Drop(0.3, "channel", 1)
    y, h, rstd = wt.rms_norm_forward(x, w, res, drop)
    full = wt.rms_norm_backward(h, dy, w, rstd, drop=drop)
    for k in range(3):
        ask = [None if i == k else False for i in range(3)]
        got = wt.rms_norm_backward(h, dy, w, rstd, None, drop, *ask)
        assert [g is None for g in got] == [i != k for i in range(3)] and torch.equal(got[k], full[k])
    assert wt.rms_norm_forward(x, w, rstd=False)[2] is None
    dx, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, dx=False)
    assert dx is None and dres is None and torch.equal(dw, full[2])


def test_binding_refusals():
    x, w = torch.randn(2, 8, 4, 4, device="cuda"), torch.ones(8, device="cuda")
    cl = x.contiguous(memory_format=torch.channels_last)
    drop = wt.Drop(0.1)
    y, h, rstd = wt.rms_norm_forward(x, w)
    for bad in (
        lambda: wt.rms_norm_forward(x[:, ::2], w[:4]), lambda: wt.rms_norm_forward(x[0], w),
        lambda: wt.rms_norm_forward(x, w[:4]), lambda: wt.rms_norm_forward(x, w.bfloat16()),
        lambda: wt.rms_norm_forward(x, w.cpu()), lambda: wt.rms_norm_forward(x, w, cl),
        lambda: wt.rms_norm_forward(x, w, x.bfloat16()), lambda: wt.rms_norm_forward(x, w, x[:1]),
        lambda: wt.rms_norm_forward(x, w, y=cl.clone()), lambda: wt.rms_norm_forward(x, w, h=torch.empty_like(x)),
        lambda: wt.rms_norm_forward(x, w, rstd=rstd[:1]), lambda: wt.rms_norm_backward(h, cl, w, rstd),
        lambda: wt.rms_norm_backward(h, y, w, rstd.double()), lambda: wt.rms_norm_q8(x, w, group=16),
        lambda: wt.rms_norm_q8(x, w, q=torch.empty_like(x)), lambda: wt.rms_norm_q8(x, w, scale=rstd),
        lambda: wt.rms_norm_backward(h, y, w, rstd, dx=torch.empty_like(x), dresidual=torch.empty_like(x)),
        lambda: wt.rms_norm_backward(h, y, w, rstd, workspace=torch.empty(64)),
        lambda: wt.dropout_forward(x, drop, cl), lambda: wt.rms_norm_forward(torch.empty(3, 0, device="cuda"), w[:0]),
    ):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wt.rms_norm_q8(x, w, dtype=torch.float16), lambda: wt.dropout_forward(x, 0.1),
                lambda: wt.rms_norm_forward(x, w, x.clone(), 0.1)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: wt.rms_norm_forward(x, w, drop=drop), lambda: wt.rms_norm_forward(x, w, eps=0.0),
                lambda: wt.rms_norm_forward(x, w, y=x), lambda: wt.dropout_forward(x, drop, y=x),
                lambda: wt.rms_norm_backward(h, y, w, rstd, workspace=torch.empty(1, device="cuda"))):
        with pytest.raises(wt.WTConvError):
            bad()


def test_repeats_are_bitwise_equal_and_the_workspace_can_be_given():
    gen = gen_of("repeat")
    for layout in ("nchw", "nhwc"):
        x, dy = make((8, 96, 28, 28), layout, BF16, gen), make((8, 96, 28, 28), layout, BF16, gen)
        w = torch.randn(96, generator=gen).cuda()
        y, h, rstd = wt.rms_norm_forward(x, w)
        ws = torch.full((wt.rms_norm_workspace_bytes(x),), 0xFF, dtype=torch.uint8, device="cuda")
        first = wt.rms_norm_backward(h, dy, w, rstd)
        for _ in range(3):
            again = wt.rms_norm_backward(h, dy, w, rstd, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams():
    gen = gen_of("streams")
    x, dy = make((4, 64, 14, 14), "nchw", F32, gen), make((4, 64, 14, 14), "nchw", F32, gen)
    w = torch.randn(64, generator=gen).cuda()
    drop = wt.Drop(0.2, "element", 5)
    y, h, rstd = wt.rms_norm_forward(x, w, dy, drop)
    want = (y, *wt.rms_norm_backward(h, dy, w, rstd, drop=drop))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for k in range(12):  # calls in flight on three streams at once, none ordered with another
        s = streams[k % 3]
        y, h, rstd = wt.rms_norm_forward(x, w, dy, drop, stream=s)
        got.append((y, *wt.rms_norm_backward(h, dy, w, rstd, drop=drop, stream=s)))
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_captured_step_draws_new_masks():
    gen = gen_of("graph")
    shape = (2, 48, 8, 8)
    x, res, dy = (make(shape, "nchw", F32, gen) for _ in range(3))
    w = torch.randn(48, generator=gen).cuda()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = wt.Drop(0.4, "element", 11, step)

    def call():
        y, h, rstd = wt.rms_norm_forward(x, w, res, drop, EPS)
        out = (y, h, rstd, *wt.rms_norm_backward(h, dy, w, rstd, None, drop))
        step.add_(1)
        return out

    call()
    torch.cuda.synchronize()
    step.zero_()
    graphs = []
    for _ in range(2):  # two graphs of the same call, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    step.zero_()
    for k in range(4):
        g, out = graphs[k % 2]
        g.replay()
        torch.cuda.synchronize()
        now = wt.Drop(0.4, "element", 11, k)
        check_forward(x, res, w, now, *out[:3])
        check_backward(out[1], dy, None, w, now, *out[3:])
    assert int(step) == 4


def test_autograd_through_the_layer_and_its_block():
    """WTConv2d, the branch joined to the residual stream, the norm: gradients against differences in float64."""
    torch.manual_seed(0)
    B, C, H, W, L, eps = 2, 4, 8, 8, 1, 1e-3
    import oracle as orc
    o = orc.default()
    conv, norm = wt.WTConv2d(C, 3, L, device="cuda"), wt.RMSNorm2d(C, eps, device="cuda")
    with torch.no_grad():
        norm.weight.copy_(torch.rand(C) + 0.5)
    x = torch.randn(B, C, H, W, device="cuda", requires_grad=True)
    dy, dh = torch.randn(B, C, H, W, device="cuda"), torch.randn(B, C, H, W, device="cuda")
    drop = wt.Drop(0.3, "element", 21, 2)
    y, h = norm(conv(x), x, drop)
    ((y * dy).sum() + (h * dh).sum()).backward()
    keep = ref.keep_mask(B, C, H * W, 0.3, "element", 21, 2)
    p = {k: getattr(conv, k).detach().double().cpu().numpy() for k in ("base_w", "base_b", "base_scale", "wt_w", "wt_scale")}
    wn = norm.weight.detach().double().cpu().numpy()
    xd = x.detach().double().cpu().numpy()

    def loss(xv, pv, wv):
        branch = o.forward(xv, pv["base_w"], pv["base_b"], pv["base_scale"], pv["wt_w"], pv["wt_scale"], L)
        hv = ref.join(branch.reshape(B, C, -1), xv.reshape(B, C, -1), keep, 0.3)
        return (ref.norm(hv, wv, eps)[0] * wide(dy)).sum() + (hv * wide(dh)).sum()

    rng, e = np.random.default_rng(1), 1e-6

    # The sums behind a gradient here have terms of up to about 30 and the longest path about 100 roundings:
    # 100 * 2^-24 * 30 < 2e-4.
    def slope(f):  # central difference; its own error is about 1e-9 here
        return (f(e) - f(-e)) / (2 * e)

    for _ in range(8):
        i = tuple(rng.integers(0, n) for n in xd.shape)
        d = np.zeros_like(xd)
        d[i] = 1.0
        assert abs(slope(lambda t: loss(xd + t * d, p, wn)) - float(x.grad[i])) <= 2e-4
        c = int(rng.integers(0, C))
        dwv = np.zeros_like(wn)
        dwv[c] = 1.0
        assert abs(slope(lambda t: loss(xd, p, wn + t * dwv)) - float(norm.weight.grad[c])) <= 2e-4
        name = ("base_w", "base_scale", "wt_w", "wt_scale")[int(rng.integers(0, 4))]
        j = tuple(rng.integers(0, n) for n in p[name].shape)
        dp = np.zeros_like(p[name])
        dp[j] = 1.0
        got = float(getattr(conv, name).grad[j])
        assert abs(slope(lambda t: loss(xd, {**p, name: p[name] + t * dp}, wn)) - got) <= 2e-4


def test_autograd_forms():
    gen = gen_of("autograd")
    for layout in ("nchw", "nhwc", "rows"):
        shape = (3, 20, 1, 1) if layout == "rows" else (3, 20, 5, 4)
        x, res, dy, dh = (make(shape, layout, BF16, gen) for _ in range(4))
        w = torch.randn(20, generator=gen).cuda().requires_grad_()
        xl, rl = x.clone().requires_grad_(), res.clone().requires_grad_()
        drop = wt.Drop(0.3, "channel", 8)
        y, h = wt.rms_norm(xl, w, rl, drop, EPS)
        torch.autograd.backward([y, h], [dy, dh])
        y2, h2, rstd = wt.rms_norm_forward(x, w.detach(), res, drop, EPS)
        want = wt.rms_norm_backward(h2, dy, w.detach(), rstd, dh, drop)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        for a, b in zip((xl.grad, rl.grad, w.grad), want):
            assert torch.equal(a, b)
        # only one of the two outputs used, only one leaf asked for
        xl.grad = rl.grad = w.grad = None
        wt.rms_norm(xl.detach(), w, rl, drop, EPS)[1].backward(dh)
        assert xl.grad is None and torch.equal(rl.grad, dh) and not w.grad.any()
        y = wt.rms_norm(xl, w.detach(), eps=EPS)
        y.backward(dy)
        y2, h2, rstd = wt.rms_norm_forward(x, w.detach(), eps=EPS)
        assert torch.equal(xl.grad, wt.rms_norm_backward(h2, dy, w.detach(), rstd)[0])
        xl.grad = rl.grad = None
        wt.dropout(xl, drop, rl).backward(dy)
        assert torch.equal(xl.grad, wt.dropout_backward(dy, drop)) and torch.equal(rl.grad, dy)
    # one tensor as both branch and residual; the two leaves' gradients are tensors of their own
    both = x.clone().requires_grad_()
    y, h = wt.rms_norm(both, w.detach(), both)
    torch.autograd.backward([y, h], [dy, dh])
    y2, h2, rstd = wt.rms_norm_forward(x, w.detach(), x)
    d = wt.rms_norm_backward(h2, dy, w.detach(), rstd, dh)[0]
    assert torch.equal(both.grad, d + d)
    xl, rl = x.clone().requires_grad_(), res.clone().requires_grad_()
    wt.rms_norm(xl, w.detach(), rl)[0].backward(dy)
    kept = rl.grad.clone()
    xl.grad.zero_()
    assert torch.equal(rl.grad, kept)
    # strided activations are laid out first; gradients arrive in any layout
    t = torch.randn(2, 6, 20, 5, device="cuda").transpose(1, 2).requires_grad_()
    g = torch.randn(2, 5, 6, 20, device="cuda").permute(0, 3, 2, 1)
    wt.rms_norm(t, w.detach()).backward(g)
    assert t.grad.shape == t.shape
    want = wt.rms_norm_forward(t.detach().contiguous(), w.detach())
    assert torch.equal(t.grad, wt.rms_norm_backward(want[1], g.contiguous(), w.detach(), want[2])[0])


def test_autograd_refusals():
    x = torch.randn(2, 8, device="cuda", requires_grad=True)
    w = torch.ones(8, device="cuda", requires_grad=True)
    y = wt.rms_norm(x, w)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        g.sum().backward()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    for f in (lambda: wt.dropout(x, wt.Drop(0.5, offset=step)),
              lambda: wt.rms_norm(x, w, x.detach().clone(), wt.Drop(0.5, offset=step))[0]):
        y = f()
        step.add_(1)  # the mask of the backward would be another one
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_serving_chain():
    """The layer, the branch joined to the residual stream, 8-bit activations: q * scale is the norm that training computes."""
    torch.manual_seed(5)
    conv, norm = wt.WTConv2d(32, 5, 2, device="cuda"), wt.RMSNorm2d(32, device="cuda")
    for fmt in (torch.contiguous_format, torch.channels_last):
        x = torch.randn(2, 32, 16, 16, device="cuda").to(BF16).contiguous(memory_format=fmt)
        with torch.no_grad():
            branch = conv(x)
            y, h = norm(branch, x)
            for kind, half_step in ((torch.float8_e4m3fn, 2.0 ** -4), (torch.int8, 0.5 / 127)):
                q, scale, h8 = wt.rms_norm_q8(branch, norm.weight, x, norm.eps, kind)
                assert torch.equal(h8, h) and h8.stride() == x.stride()
                got, want = wide(q.float()) * wide(scale), wide(y)
                # half a step of the 8-bit type (of the pixel's largest value for whole numbers), half a step of bf16
                size = np.abs(want) if kind != torch.int8 else np.abs(want).max(axis=1, keepdims=True)
                low = wide(scale) * 2.0 ** -10  # e4m3 below its smallest normal
                close(got, want, 1.01 * (half_step * size + low + half(BF16) * np.abs(want)), str(kind))


def test_captured_autograd_step_of_modules():
    torch.manual_seed(6)
    drop = wt.BranchDropout(0.4, "element", seed=9, capturable=True, device="cuda")
    norm = wt.RMSNorm2d(12, device="cuda")
    x = torch.randn(2, 12, 5, 6, device="cuda", requires_grad=True)
    res = torch.randn(2, 12, 5, 6, device="cuda", requires_grad=True)
    dy = torch.randn(2, 12, 5, 6, device="cuda")

    def call():
        y, h = norm(x, res, drop.next_drop())
        return (y, *torch.autograd.grad([y, drop(h)], [x, res, norm.weight], [dy, dy]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [t.detach() for t in call()]
    eager = wt.BranchDropout(0.4, "element", seed=9, device="cuda")
    for _ in range(3):
        eager.steps = int(drop.step)
        graph.replay()
        torch.cuda.synchronize()
        y, h = norm(x, res, eager.next_drop())
        want = (y, *torch.autograd.grad([y, eager(h)], [x, res, norm.weight], [dy, dy]))
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert int(drop.step) == 8  # two a call


def test_modules():
    torch.manual_seed(1)
    x, res = torch.randn(4, 16, 6, 6, device="cuda"), torch.randn(4, 16, 6, 6, device="cuda")
    for capturable in (False, True):
        m = wt.BranchDropout(0.5, "sample", capturable=capturable, device="cuda")
        outs = [m(x, res) for _ in range(3)]
        for k, y in enumerate(outs):
            assert torch.equal(y, wt.dropout_forward(x, wt.Drop(0.5, "sample", m.seed, k), res))
        m.eval()
        assert torch.equal(m(x, res), x + res) and m(x) is x
    # two forwards before the backward of the first (the step has moved on)
    m = wt.BranchDropout(0.5, "element", seed=4, capturable=True, device="cuda")
    leaf = x.clone().requires_grad_()
    a, b = m(leaf), m(leaf)
    (a.sum() + b.sum()).backward()
    ones = torch.ones_like(x)
    want = wt.dropout_backward(ones, wt.Drop(0.5, "element", 4, 0)) + wt.dropout_backward(ones, wt.Drop(0.5, "element", 4, 1))
    assert torch.equal(leaf.grad, want)
    norm = wt.RMSNorm2d(16, device="cuda")
    y, h = norm(x, res, wt.BranchDropout(0.1, "channel", seed=2).next_drop())
    assert torch.equal(y, wt.rms_norm_forward(h, norm.weight.detach())[0])


@pytest.mark.parametrize("B,side", [(1, 16400), (3, 10400)])
def test_offsets_past_31_bits(B, side):
    # The last pixels of maps of over 2^31 elements, in one sample or in several, in both layouts.
    C = 8
    H = W = side
    x = torch.zeros(B, C, H, W, dtype=BF16, device="cuda")
    tail = torch.randn(1, C, 1, 64, generator=gen_of("far")).to(BF16).cuda()
    w = torch.rand(C, generator=gen_of("far")).cuda() + 0.5
    drop = wt.Drop(0.5, "element", 13)
    for cl in (False, True):
        if cl:
            x = x.contiguous(memory_format=torch.channels_last)
        x[-1:, :, -1:, -64:] = tail
        y, _, rstd = wt.rms_norm_forward(x, w, eps=EPS)
        part = y[-1:, :, -1:, -64:].contiguous()
        check_forward(tail, None, w, None, part, tail, rstd[-1:, -1:, -64:].contiguous())
        assert not y[-1, :, -1, :-64].any() and not y[:, :, 0].any()
        dx, _, dw = wt.rms_norm_backward(x, y, w, rstd)
        last = dx[-1:, :, -1:, -64:].contiguous()
        check_backward(tail, part, None, w, None, last, last, None)
        assert not dx[:, :, 0].any()
        # the zeros add nothing: the sum of the last 64 rows, whatever shares of the rows the CTAs add up
        t = wide(tail)
        terms = wide(part) * t / np.sqrt((t ** 2).mean(1, keepdims=True) + EPS)
        close(dw.double().cpu().numpy(), terms.sum((0, 2)), (64 + C / 2 + 14) * U * np.abs(terms).sum((0, 2)), "dweight")
        del dx, y
        y = wt.dropout_forward(x, drop)
        row = np.arange(B * H * W - 64, B * H * W, dtype=np.uint64)
        words = [ref.philox4x32((np.full(64, q, np.uint64), row, row >> np.uint64(32), np.zeros(64, np.uint64)), (13, 0))
                 for q in range(2)]
        keep = np.stack([u for ws in words for u in ws]) >= np.uint64(1 << 31)
        assert np.array_equal(wide(y[-1:, :, -1:, -64:])[0], np.where(keep, wide(tail)[0] * 2.0, 0.0))
        q, scale, _ = wt.rms_norm_q8(x, w, group=32)
        v, _ = ref.norm(t, w.double().cpu().numpy(), 1e-6)
        s8 = wide(scale[-1:, :, -1:, -64:])
        close(wide(q[-1:, :, -1:, -64:].float()) * s8, v, np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s8) * 1.001 + 1e-5 * np.abs(v), "q")
        del y, q, scale


def test_rows_past_32_bits():
    # The counter's second word: mask rows over 2^32.
    B, side = 5, 1 << 15
    x = torch.ones(B, 1, side, side, dtype=BF16, device="cuda")
    y = wt.dropout_forward(x, wt.Drop(0.5, "element", 17, 3))
    for first in (0, (1 << 32) - 32, B * side * side - 64):
        row = np.arange(first, first + 64, dtype=np.uint64)
        word = ref.philox4x32((np.zeros(64, np.uint64), row & np.uint64(0xFFFFFFFF), row >> np.uint64(32),
                               np.full(64, 3, np.uint64)), (17, 0))[0]
        got = y.view(-1)[first:first + 64].double().cpu().numpy()
        assert np.array_equal(got, np.where(word >= np.uint64(1 << 31), 2.0, 0.0))
