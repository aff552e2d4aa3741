"""Random calls of the map operators, each buffer at an alignment of its own, against plain float64 forms; what lies
around the outputs stays as it was.  The tolerances are those of test_maps.py."""
import random

import numpy as np
import pytest
import torch

import map_reference as ref
import memory_bound_cnn_wtconv_b200 as wt
from test_maps import BF16, F32, U, check_backward, check_forward, close, gen_of, half, wide

pytestmark = pytest.mark.gpu

GUARD = 77  # every byte around an output


class Buffers:
    """Activations of one shape and layout, and a record of the outputs' surroundings."""

    def __init__(self, shape, layout, rng, gen):
        self.shape, self.layout, self.rng, self.gen, self.outputs = shape, layout, rng, gen, []

    def _view(self, flat):
        B, C, H, W = self.shape
        if self.layout == "nhwc":
            return flat.view(B, H, W, C).permute(0, 3, 1, 2)
        return flat.view((B, C) if self.layout == "rows" else self.shape)

    def _space(self, dtype):
        n, shift = int(np.prod(self.shape)), self.rng.choice([0, 0, 0, 0, 1, 2, 3, 4, 8])
        size = torch.empty((), dtype=dtype).element_size()
        space = torch.full(((n + shift + 32) * size,), GUARD, dtype=torch.uint8, device="cuda")
        return space, shift * size, n * size

    def input(self, dtype):
        space, first, size = self._space(dtype)
        flat = space[first:first + size].view(dtype)
        flat.copy_(torch.randn(flat.numel(), generator=self.gen))
        return self._view(flat)

    def output(self, dtype):
        space, first, size = self._space(dtype)
        self.outputs.append((space, first, size))
        return self._view(space[first:first + size].view(dtype))

    def check(self):
        for space, first, size in self.outputs:
            assert (space[:first] == GUARD).all() and (space[first + size:] == GUARD).all()


def draw(rng):
    def size(most):
        return int(round(2 ** rng.uniform(0, most)))

    layout = rng.choice(["nchw", "nchw", "nhwc", "rows"])
    C = size(rng.choice([5, 8, 11, 13]))
    H, W = (1, 1) if layout == "rows" else rng.choice([(size(6), size(6)), (7, 7), (14, 14), (28, 28), (4, 8)])
    B = max(1, min(size(8), (1 << 17) // (C * H * W)))
    return (B, C, H, W), layout


@pytest.mark.parametrize("seed", range(8))
def test_random_calls(seed):
    rng = random.Random(seed)
    for k in range(150):
        shape, layout = draw(rng)
        B, C, H, W = shape
        if B * C * H * W > 1 << 18:
            continue
        gen = gen_of("random", seed, k)
        at, dtype, eps = Buffers(shape, layout, rng, gen), rng.choice([F32, BF16]), rng.choice([1e-6, 1e-5, 1e-3])
        drop = wt.Drop(rng.choice([0.0, 0.1, 0.5, 0.9]), rng.choice(["element", "channel", "sample"]), rng.randrange(1 << 63), rng.randrange(1 << 33))
        x, res = at.input(dtype), at.input(dtype) if rng.random() < 0.7 else None
        w = torch.randn(C + 3, generator=gen).cuda()[rng.randrange(4):][:C]
        what = rng.choice(["dropout", "norm", "norm", "q8"])
        if what == "dropout":
            y = wt.dropout_forward(x, drop, res, at.output(dtype))
            keep = ref.keep_mask(*wide(x).shape, drop.p, drop.mode, drop.seed, drop.offset)
            want = ref.join(wide(x), None if res is None else wide(res), keep, drop.p)
            close(wide(y), want, (half(dtype) + 1.01 * U) * np.abs(want), "y")
        elif what == "q8":
            kind, group = rng.choice([torch.float8_e4m3fn, torch.int8]), rng.choice([0, 32, 64, 128])
            q, scale, h = wt.rms_norm_q8(x, w, res, eps, kind, group, at.output(kind), None,
                                         None if res is None else at.output(dtype))
            if res is not None:
                want = wide(x) + wide(res)
                close(wide(h), want, (half(dtype) + 1.01 * U) * np.abs(want), "h")
            v, _ = ref.norm(wide(h), w.double().cpu().numpy(), eps)
            G, top, tol = group or C, 448.0 if kind != torch.int8 else 127.0, ((C + 1) / 2 + 10) * U
            want = np.maximum(ref.group_max(v, G) / top, 2.0 ** -126)
            close(wide(scale), want, tol * want, "scale")
            s = np.repeat(wide(scale), G, axis=1)[:, :C]
            step = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) if top == 448.0 else 0.5 * s
            close(wide(q.float()) * s, v, step * (1 + 4 * tol) + 4 * tol * np.abs(v), "q")
        else:
            use = drop if res is not None and rng.random() < 0.6 else None
            y, h, rstd = wt.rms_norm_forward(x, w, res, use, eps, at.output(dtype), None if res is None else at.output(dtype))
            check_forward(x, res, w, use, y, h, rstd, eps)
            dy, dh = at.input(dtype), at.input(dtype) if rng.random() < 0.6 else None
            dres = at.output(dtype) if rng.random() < 0.8 else False
            dx = None if use is None else at.output(dtype) if rng.random() < 0.8 else False
            dx, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, dh, use, dx, dres, None if rng.random() < 0.8 else False)
            check_backward(h, dy, dh, w, use, dx, dres, dw, eps)
        at.check()
