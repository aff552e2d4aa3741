"""The tests' plain forms against what they stand for (CPU only)."""
import numpy as np
import pytest

import map_reference as ref


def test_philox_known_answers():
    # The known-answer vectors published with the generator (Philox4x32, 10 rounds).
    for counter, key, want in [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]:
        got = ref.philox4x32([np.array([c]) for c in counter], key)
        assert tuple(int(g[0]) for g in got) == want


@pytest.mark.parametrize("mode", ["element", "channel", "sample"])
def test_keep_mask_rate_and_cover(mode):
    B, C, P, p = 400, 30, 12, 0.3
    k = ref.keep_mask(B, C, P, p, mode, 7, 3)
    assert k.shape == (B, C, P)
    if mode != "element":
        assert (k == k[:, :, :1]).all()
    if mode == "sample":
        assert (k == k[:, :1]).all()
    n = {"element": B * C * P, "channel": B * C, "sample": B}[mode]
    assert abs(k.mean() - 0.7) < 5 * np.sqrt(0.21 / n)  # five standard deviations
    assert (k != ref.keep_mask(B, C, P, p, mode, 7, 4)).any() and (k != ref.keep_mask(B, C, P, p, mode, 8, 3)).any()


def test_norm_grad_against_differences():
    rng = np.random.default_rng(0)
    B, C, P, eps = 2, 5, 3, 1e-3
    h, dy, dh = (rng.normal(size=(B, C, P)) for _ in range(3))
    w = rng.normal(size=C)

    def loss(h, w):
        return (ref.norm(h, w, eps)[0] * dy).sum() + (h * dh).sum()

    d, dw = ref.norm_grad(h, w, eps, dy, dh)
    step = 1e-6
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = step
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - d[i]) < 1e-7
    for c in range(C):
        e = np.zeros_like(w)
        e[c] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[c]) < 1e-7
