"""Map operators next to the layer: dropout and the RMS norm over channels.

``rms_norm`` and ``dropout`` are the autograd forms, ``RMSNorm2d`` and
``BranchDropout`` the modules; the ``*_forward`` / ``*_backward`` / ``*_q8``
calls marshal arguments for the C ABI in ``include/wtconv.h``, which has the
formulas.  Activations are [B, C, H, W] maps, contiguous (NCHW) or
channels-last contiguous (NHWC), or contiguous [N, C] rows, in float32 or
bfloat16 on one CUDA device; the activations of a call share shape, layout and
type.  Any size is taken, odd ones and B = 0 too, up to extents of 2^31 - 1,
2^30 pixels of a plane and 2^24 channels.

A call runs on ``stream`` if given (what it allocates then belongs to that
stream), else on the current stream of the activations' device.  Calls that may
run at the same time need workspaces of their own, as the allocated ones are.
In CUDA graphs: capture the ``*_forward`` / ``*_backward`` calls, or the
autograd forms with ``torch.autograd.grad``.  Everything
runs in the CUDA kernels of ``libwtconv_b200.so``; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F32, NCHW, NHWC, _check, load_library

__all__ = [
    "Drop", "dropout_forward", "dropout_backward", "rms_norm_forward", "rms_norm_backward", "rms_norm_q8",
    "rms_norm_workspace_bytes", "dropout", "rms_norm", "DropoutFunction", "RMSNormFunction", "RMSNorm2d",
    "BranchDropout",
]

_MODES = {"element": 0, "channel": 1, "sample": 2}
_Q8 = {torch.float8_e4m3fn: 0, torch.int8: 1}
_M64 = (1 << 64) - 1
_MOST = (1 << 31) - 1  # of the descriptor's C ints


class MapDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
                ("dtype", ctypes.c_int), ("layout", ctypes.c_int)]


class _DropArgs(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("mode", ctypes.c_int), ("seed", ctypes.c_ulonglong),
                ("offset", ctypes.c_ulonglong), ("offset_dev", ctypes.c_void_p)]


class Drop:
    """One call's dropout: probability ``p`` (0 <= p < 1), what a decision
    covers (``mode``: "element", "channel" of a sample, or "sample"), and the
    counter that names the mask: the same ``seed`` and ``offset`` give the same
    mask, in both layouts and types and in the backward.  Processes that share a
    batch out need a seed each: a call's rows and samples count from 0, so the
    same seed would drop the same places of different samples.

    ``offset`` is a number (of the step, say), or an int64 CUDA tensor of one
    element, which the kernels read when they run: a captured graph that moves
    it on between replays draws a new mask in each.  Do not change it between a
    forward and its backward (the autograd forms raise if it was).
    """

    __slots__ = ("p", "mode", "seed", "offset", "_args")

    def __init__(self, p: float, mode: str = "element", seed: int = 0, offset=0):
        p = float(p)
        if not 0.0 <= p < 1.0:
            raise ValueError(f"p must be at least 0 and below 1, got {p}")
        if mode not in _MODES:
            raise ValueError(f"mode must be one of {sorted(_MODES)}, got {mode!r}")
        self.p, self.mode, self.seed, self.offset = p, mode, int(seed), offset
        dev = None
        if isinstance(offset, torch.Tensor):
            if offset.dtype != torch.int64 or offset.numel() != 1 or not offset.is_cuda:
                raise ValueError("an offset tensor must be an int64 CUDA tensor of one element")
            dev, offset = offset.data_ptr(), 0
        self._args = _DropArgs(p, _MODES[mode], self.seed & _M64, int(offset) & _M64, dev)

    def __repr__(self) -> str:
        return f"Drop(p={self.p}, mode={self.mode!r}, seed={self.seed}, offset={self.offset})"


_fns = None


def _lib():
    """The library's map operators, with their argument types."""
    global _fns
    if _fns is None:
        lib = load_library()
        vp, dp, ap, f, i, sz = (ctypes.c_void_p, ctypes.POINTER(MapDesc), ctypes.POINTER(_DropArgs), ctypes.c_float,
                                ctypes.c_int, ctypes.c_size_t)
        lib.wtconv_dropout.argtypes = [dp, ap, vp, vp, vp, vp]
        lib.wtconv_rms_norm_forward.argtypes = [dp, f, vp, vp, ap, vp, vp, vp, vp, vp]
        lib.wtconv_rms_norm_q8.argtypes = [dp, f, vp, vp, vp, i, i, vp, vp, vp, vp]
        lib.wtconv_rms_norm_backward.argtypes = [dp, vp, vp, vp, ap, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.wtconv_rms_norm_workspace_bytes.argtypes = [dp]
        lib.wtconv_rms_norm_workspace_bytes.restype = sz
        for name in ("wtconv_dropout", "wtconv_rms_norm_forward", "wtconv_rms_norm_q8", "wtconv_rms_norm_backward"):
            getattr(lib, name).restype = i
        _fns = lib
    return _fns


class _Map:
    """What a call needs to know of the shape, type and layout of its activations."""

    __slots__ = ("desc", "ref", "C", "layout", "flat", "rows")

    def __init__(self, shape, dtype, layout: int):
        if max(shape) > _MOST:  # ctypes would pass it modulo 2^32
            raise ValueError(f"an extent is over {_MOST}: {tuple(shape)}")
        B, C, H, W = shape if len(shape) == 4 else (*shape, 1, 1)
        self.desc = MapDesc(B, C, H, W, F32 if dtype is torch.float32 else BF16, layout)
        self.ref = ctypes.byref(self.desc)
        self.C, self.layout = C, layout
        self.flat = layout == NCHW or len(shape) == 2  # contiguous, not channels-last
        self.rows = (B,) if len(shape) == 2 else (B, H, W)


_maps = {}  # by shape, type and layout


def _map_of(x: torch.Tensor, name: str) -> _Map:
    """The map that a tensor is; raises for what is none."""
    key = (x.shape, x.dtype, x.is_contiguous())
    if x.is_cuda and (m := _maps.get(key)) is not None and (key[2] or x.is_contiguous(memory_format=torch.channels_last)):
        return m
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"activations must be float32 or bfloat16, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() not in (2, 4):
        raise ValueError(f"{name} must be a [B, C, H, W] map or [N, C] rows, got {x.dim()} dimensions")
    if not key[2] and not (x.dim() == 4 and x.is_contiguous(memory_format=torch.channels_last)):
        raise ValueError(f"{name} must be contiguous (NCHW, rows) or channels-last contiguous (NHWC)")
    if 0 in x.shape[1:]:
        raise ValueError(f"{name} has no channels or no pixels: {tuple(x.shape)}")
    if len(_maps) >= 4096:
        _maps.clear()
    _maps[key] = m = _Map(tuple(x.shape), x.dtype, NCHW if key[2] and x.dim() == 4 else NHWC)
    return m


def _like(t: torch.Tensor, name: str, x: torch.Tensor, m: _Map, dtype=None) -> int:
    """The address of an activation that has to be as x is."""
    if t.dtype is not (dtype or x.dtype) or t.shape != x.shape or t.get_device() != x.get_device():
        raise ValueError(f"{name} must have the shape {tuple(x.shape)}, type {dtype or x.dtype} and device of the input")
    if not (t.is_contiguous() if m.flat else t.is_contiguous(memory_format=torch.channels_last)):
        raise ValueError(f"{name} must have the layout of the input ({'NHWC' if m.layout == NHWC else 'NCHW'})")
    return t.data_ptr()


def _vector(t: torch.Tensor, name: str, x: torch.Tensor, shape) -> int:
    if t.dtype is not torch.float32 or t.get_device() != x.get_device() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor on {x.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _drop_ref(drop, x):
    if not isinstance(drop, Drop):
        raise TypeError(f"drop must be a Drop, got {type(drop).__name__}")
    if drop._args.offset_dev is not None and drop.offset.device != x.device:
        raise ValueError(f"the offset tensor is on {drop.offset.device}, the activations on {x.device}")
    return ctypes.byref(drop._args)


def _elsewhere(x, stream) -> bool:
    """Whether a call is not for the current stream of the current device."""
    return stream is not None or x.get_device() != torch._C._cuda_getDevice()


def _there(x, stream):
    """The context in which that stream and the device of x are the current ones."""
    if stream is None:
        return torch.cuda.device(x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the activations on {x.device}")
    return torch.cuda.stream(stream)


def _stream_of(x) -> int:
    return torch._C._cuda_getCurrentRawStream(x.get_device())


def dropout_forward(x, drop: Drop, residual=None, y=None, stream=None):
    """y = residual + drop(x) via ``wtconv_dropout``; returns y (allocated if
    not given)."""
    m = _map_of(x, "x")
    if _elsewhere(x, stream):
        with _there(x, stream):
            return dropout_forward(x, drop, residual, y)
    ref = _drop_ref(drop, x)
    rp = None if residual is None else _like(residual, "residual", x, m)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _like(y, "y", x, m)
    _check(_lib().wtconv_dropout(m.ref, ref, x.data_ptr(), rp, yp, _stream_of(x)), "wtconv_dropout")
    return y


def dropout_backward(dy, drop: Drop, dx=None, stream=None):
    """The gradient of x, drop(dy) with the forward's mask (the residual's is
    dy); returns dx."""
    return dropout_forward(dy, drop, None, dx, stream)


def rms_norm_forward(x, weight, residual=None, drop: Drop = None, eps: float = 1e-6, y=None, h=None, rstd=None,
                     stream=None):
    """h = residual + drop(x), y = h / rms(h) * weight via
    ``wtconv_rms_norm_forward``; returns (y, h, rstd).  Without a residual h is
    x itself.  ``rstd=False`` leaves rstd out (inference): None is returned."""
    m = _map_of(x, "x")
    if _elsewhere(x, stream):
        with _there(x, stream):
            return rms_norm_forward(x, weight, residual, drop, eps, y, h, rstd)
    wp = _vector(weight, "weight", x, (m.C,))
    ref = None if drop is None else _drop_ref(drop, x)
    if residual is None:
        if h is not None:
            raise ValueError("without a residual, h is x: give none")
        h, rp, hp = x, None, None
    else:
        rp = _like(residual, "residual", x, m)
        if h is None:
            h = torch.empty_like(x)
            hp = h.data_ptr()
        else:
            hp = _like(h, "h", x, m)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _like(y, "y", x, m)
    if rstd is None:
        rstd = weight.new_empty(m.rows)
        sp = rstd.data_ptr()
    elif rstd is False:
        rstd = sp = None
    else:
        sp = _vector(rstd, "rstd", x, m.rows)
    _check(_lib().wtconv_rms_norm_forward(m.ref, eps, x.data_ptr(), rp, ref, wp, yp, hp, sp, _stream_of(x)),
           "wtconv_rms_norm_forward")
    return y, h, rstd


def rms_norm_workspace_bytes(x: torch.Tensor) -> int:
    """Workspace of ``rms_norm_backward`` for activations like x."""
    m = _map_of(x, "x")
    if _elsewhere(x, None):
        with _there(x, None):
            return rms_norm_workspace_bytes(x)
    return _lib().wtconv_rms_norm_workspace_bytes(m.ref)


def rms_norm_backward(h, dy, weight, rstd, dh=None, drop: Drop = None, dx=None, dresidual=None, dweight=None,
                      workspace=None, stream=None):
    """Gradients of ``rms_norm_forward`` from its h and rstd, via
    ``wtconv_rms_norm_backward``; ``dh`` is the gradient that reaches h itself.
    Returns (dx, dresidual, dweight).  Without ``drop`` (which has to be the
    forward's) the two activations' gradients are the same tensor.  A gradient
    given as False is left out (None is returned; without ``drop`` False for
    either of the two stands for both).  ``workspace`` is a CUDA tensor of at
    least ``rms_norm_workspace_bytes`` bytes; allocated here if not given."""
    m = _map_of(h, "h")
    if _elsewhere(h, stream):
        with _there(h, stream):
            return rms_norm_backward(h, dy, weight, rstd, dh, drop, dx, dresidual, dweight, workspace)
    dyp = _like(dy, "dy", h, m)
    wp = _vector(weight, "weight", h, (m.C,))
    rsp = _vector(rstd, "rstd", h, m.rows)
    dhp = None if dh is None else _like(dh, "dh", h, m)
    gp = ref = None
    if drop is None:
        if dx is False or dresidual is False:
            dresidual = False
        elif dx is not None:
            if dresidual is not None and dresidual is not dx:
                raise ValueError("without dropout dx and dresidual are the same: give one")
            dresidual = dx
    else:
        ref = _drop_ref(drop, h)
        if dx is None:
            dx = torch.empty_like(h)
            gp = dx.data_ptr()
        elif dx is False:
            dx = None
        else:
            gp = _like(dx, "dx", h, m)
    if dresidual is None:
        dresidual = torch.empty_like(h)
        rp = dresidual.data_ptr()
    elif dresidual is False:
        dresidual = rp = None
    else:
        rp = _like(dresidual, "dresidual", h, m)
    if drop is None:
        dx = dresidual
    lib = _lib()
    wsp = None
    nbytes = 0
    if dweight is False:
        dweight = dwp = None
        if rp is None and gp is None:
            return dx, dresidual, None
    else:
        if dweight is None:
            dweight = torch.empty_like(weight)
            dwp = dweight.data_ptr()
        else:
            dwp = _vector(dweight, "dweight", h, (m.C,))
        if workspace is None:
            nbytes = lib.wtconv_rms_norm_workspace_bytes(m.ref)
            workspace = weight.new_empty(((nbytes + 3) // 4,))
            wsp = workspace.data_ptr()
        else:
            if not workspace.is_cuda or workspace.device != h.device or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on {h.device}")
            wsp, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib.wtconv_rms_norm_backward(m.ref, h.data_ptr(), dyp, dhp, ref, wp, rsp, rp, gp, dwp, wsp, nbytes,
                                        _stream_of(h)), "wtconv_rms_norm_backward")
    return dx, dresidual, dweight


def rms_norm_q8(x, weight, residual=None, eps: float = 1e-6, dtype=torch.float8_e4m3fn, group: int = 0, q=None,
                scale=None, h=None, stream=None):
    """``rms_norm_forward`` with an 8-bit output (``torch.float8_e4m3fn`` or
    ``torch.int8``) and one float32 scale for each ``group`` adjacent channels
    of a pixel (32, 64, 128, or 0: all), via ``wtconv_rms_norm_q8``; q * scale
    stands for the norm.  Returns (q, scale, h): scale is [B, groups, H, W] (or
    [N, groups]) in the layout of x; h is x without a residual."""
    if dtype not in _Q8:
        raise TypeError(f"dtype must be torch.float8_e4m3fn or torch.int8, got {dtype}")
    if group not in (0, 32, 64, 128):
        raise ValueError(f"group must be 0, 32, 64 or 128, got {group}")
    m = _map_of(x, "x")
    if _elsewhere(x, stream):
        with _there(x, stream):
            return rms_norm_q8(x, weight, residual, eps, dtype, group, q, scale, h)
    wp = _vector(weight, "weight", x, (m.C,))
    if residual is None:
        if h is not None:
            raise ValueError("without a residual, h is x: give none")
        h, rp, hp = x, None, None
    else:
        rp = _like(residual, "residual", x, m)
        if h is None:
            h = torch.empty_like(x)
            hp = h.data_ptr()
        else:
            hp = _like(h, "h", x, m)
    if q is None:
        q = torch.empty_like(x, dtype=dtype)
        qp = q.data_ptr()
    else:
        qp = _like(q, "q", x, m, dtype)
    groups = -(-m.C // group) if group else 1
    shape = (x.shape[0], groups, *x.shape[2:])
    nhwc = not m.flat
    if scale is None:
        scale = weight.new_empty((shape[0], *shape[2:], groups) if nhwc else shape)
        if nhwc:
            scale = scale.permute(0, 3, 1, 2)
    elif scale.dtype is not torch.float32 or scale.shape != shape or scale.device != x.device \
            or not scale.is_contiguous(memory_format=torch.channels_last if nhwc else torch.contiguous_format):
        raise ValueError(f"scale must be a float32 tensor of shape {shape} in the layout of x on {x.device}")
    _check(_lib().wtconv_rms_norm_q8(m.ref, eps, x.data_ptr(), rp, wp, _Q8[dtype], group, qp,
                                     scale.data_ptr(), hp, _stream_of(x)), "wtconv_rms_norm_q8")
    return q, scale, h


def _laid_out(x):
    """x in one of the kernels' layouts (channels-last maps stay NHWC)."""
    return x if x.dim() == 4 and x.is_contiguous(memory_format=torch.channels_last) else x.contiguous()


def _as(t, x):
    """t in the layout of x."""
    if t is None:
        return None
    return t.contiguous(memory_format=torch.contiguous_format if x.is_contiguous() else torch.channels_last)


def _saved_offset(drop):
    """The offset tensor, for autograd's check that nothing changed it."""
    return drop.offset if drop is not None and isinstance(drop.offset, torch.Tensor) else None


class DropoutFunction(torch.autograd.Function):
    """y = residual + drop(x).  The backward computes the mask again; nothing of
    the size of x is saved."""

    @staticmethod
    def forward(ctx, x, residual, drop: Drop):
        x = _laid_out(x)
        ctx.drop = drop
        ctx.save_for_backward(_saved_offset(drop))
        ctx.like = x.is_contiguous(), x.dtype
        return dropout_forward(x, drop, _as(residual, x))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ctx.saved_tensors  # raises where the offset tensor has changed
        need = ctx.needs_input_grad
        dx = None
        if need[0]:
            fmt = torch.contiguous_format if ctx.like[0] else torch.channels_last
            dx = dropout_backward(dy.to(ctx.like[1]).contiguous(memory_format=fmt), ctx.drop)
        return dx, dy if need[1] else None, None


class RMSNormFunction(torch.autograd.Function):
    """(y, h) of ``rms_norm_forward``.  Saves h (x without a residual) and one
    float a pixel."""

    @staticmethod
    def forward(ctx, x, weight, residual, drop: Drop, eps: float):
        x = _laid_out(x)
        y, h, rstd = rms_norm_forward(x, weight, _as(residual, x), drop, eps)
        ctx.save_for_backward(h, weight, rstd, _saved_offset(drop))
        ctx.drop = drop
        ctx.set_materialize_grads(False)
        return (y, h) if residual is not None else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd, _ = ctx.saved_tensors
        need, drop = ctx.needs_input_grad, ctx.drop
        if dy is None and dh is None:
            return (None,) * 5
        dy = torch.zeros_like(h) if dy is None else _as(dy.to(h.dtype), h)
        if drop is None:
            dx = None if need[0] or need[2] else False
            dres = None
        else:
            dx, dres = (None if need[0] else False), (None if need[2] else False)
        dx, dres, dw = rms_norm_backward(h, dy, weight, rstd,
                                         None if dh is None else _as(dh.to(h.dtype), h), drop, dx, dres,
                                         None if need[1] else False)
        return dx if need[0] else None, dw, dres if need[2] else None, None, None


def dropout(x, drop: Drop, residual=None):
    """residual + drop(x) with autograd support."""
    return DropoutFunction.apply(x, residual, drop)


def rms_norm(x, weight, residual=None, drop: Drop = None, eps: float = 1e-6):
    """The norm of x over its channels, with autograd support; with a residual
    the pair (norm of residual + drop(x), that sum)."""
    return RMSNormFunction.apply(x, weight, residual, drop, eps)


class RMSNorm2d(torch.nn.Module):
    """RMS norm over the channels of a map (or of [N, C] rows), with a float32
    weight [C].  ``forward(x)`` is the norm; ``forward(x, residual, drop)`` is
    the pair (norm of residual + drop(x), that sum), in one pass."""

    def __init__(self, channels: int, eps: float = 1e-6, device=None):
        super().__init__()
        self.channels, self.eps = int(channels), float(eps)
        self.weight = torch.nn.Parameter(torch.ones((self.channels,), dtype=torch.float32, device=device))

    def forward(self, x, residual=None, drop: Drop = None):
        return RMSNormFunction.apply(x, self.weight, residual, drop, self.eps)

    def extra_repr(self) -> str:
        return f"channels={self.channels}, eps={self.eps}"


class BranchDropout(torch.nn.Module):
    """Dropout of a branch: ``forward(x, residual)`` is residual + drop(x) in
    training, and plainly residual + x in evaluation.

    ``seed`` names the module's masks (drawn from torch's CPU generator if not
    given).  Data-parallel processes that seed alike drop the same places of
    their shares: give each a seed of its own, such as one number plus the rank,
    and again after loading a state that they share.  Each training call takes
    the next step as its offset.  ``next_drop()`` is that call's ``Drop``, for a
    fused norm.  With ``capturable`` the step is a CUDA tensor which the calls
    move on, so every replay of a captured graph draws new masks.  Seed and
    step are part of the state dict.  Where a forward is run again for its
    backward (activation checkpointing), take ``next_drop()`` outside and pass it
    to ``dropout`` or ``rms_norm``: a second call of the module is a new step.
    """

    def __init__(self, p: float, mode: str = "element", seed: int = None, capturable: bool = False, device=None):
        super().__init__()
        Drop(p, mode)  # raises for what is out of range
        self.p, self.mode, self.capturable = float(p), mode, bool(capturable)
        self.seed = int(torch.randint(1 << 62, (1,), device="cpu")) if seed is None else int(seed)
        self.steps = 0
        if self.capturable:
            self.register_buffer("step", torch.zeros((1,), dtype=torch.int64, device=device))

    def get_extra_state(self):
        return {"seed": self.seed, "steps": self.steps}

    def set_extra_state(self, state):
        self.seed, self.steps = int(state["seed"]), int(state["steps"])

    def next_drop(self):
        """The ``Drop`` of one training call; None where nothing is dropped."""
        if not self.training or self.p == 0.0:
            return None
        if self.capturable:
            offset = self.step.clone()  # the call's own: the counter may move on before its backward
            self.step.add_(1)
        else:
            offset = self.steps
            self.steps += 1
        return Drop(self.p, self.mode, self.seed, offset)

    def forward(self, x, residual=None):
        drop = self.next_drop()
        if drop is None:
            if residual is None:
                return x
            drop = Drop(0.0, self.mode)
        return DropoutFunction.apply(x, residual, drop)

    def extra_repr(self) -> str:
        return f"p={self.p}, mode={self.mode!r}, capturable={self.capturable}"
