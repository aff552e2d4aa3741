"""Map operators called from several host threads at once."""
import ctypes
import threading

import pytest
import torch

import memory_bound_cnn_wtconv_b200 as wt
from memory_bound_cnn_wtconv_b200 import maps
from test_maps import gen_of, make

pytestmark = pytest.mark.gpu


def test_host_threads_with_maps_of_different_sizes():
    # The channel counts share two kernels, forward and backward, whose dynamic shared memory is 50 to 198 KB by them.
    # Raw calls, which hold Python's lock for a moment only, so that the threads meet inside the library.
    widths, rounds = (96, 192, 320, 512), 4000
    lib = maps._lib()
    want, calls, keep = {}, {}, []

    def p(t):
        return ctypes.c_void_p(t.data_ptr())

    for C in widths:
        gen = gen_of("threads", C)
        x, res, dy = (make((1, C, 8, 8), "nchw", torch.float32, gen) for _ in range(3))
        w = torch.randn(C, generator=gen).cuda()
        y, h, rstd = wt.rms_norm_forward(x, w, res)
        _, dres, dw = wt.rms_norm_backward(h, dy, w, rstd, res)
        want[C] = (y, h, rstd, dres, dw)
        out = [torch.empty_like(t) for t in want[C]]
        ws = torch.empty(wt.rms_norm_workspace_bytes(x), dtype=torch.uint8, device="cuda")
        desc, stream = maps.MapDesc(1, C, 8, 8, wt.F32, wt.NCHW), torch.cuda.Stream()
        d, s = ctypes.byref(desc), ctypes.c_void_p(stream.cuda_stream)
        eps = ctypes.c_float(1e-6)
        calls[C] = out, (d, eps, p(x), p(res), None, p(w), p(out[0]), p(out[1]), p(out[2]), s), \
            (d, p(out[1]), p(dy), p(res), None, p(w), p(out[2]), p(out[3]), None, p(out[4]), p(ws), ws.numel(), s)
        keep.append((x, res, dy, w, ws, desc, stream))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(widths)), []

    def work(C):
        _, fwd, bwd = calls[C]
        forward, backward = lib.wtconv_rms_norm_forward, lib.wtconv_rms_norm_backward
        start.wait()
        for k in range(rounds):
            code = forward(*fwd) or backward(*bwd)
            if code:
                codes.append((C, k, code))
                return

    threads = [threading.Thread(target=work, args=(C,)) for C in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not codes, codes
    for C in widths:
        assert all(torch.equal(a, b) for a, b in zip(calls[C][0], want[C]))
