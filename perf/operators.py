"""Cases of the map operators that stand next to the wavelet convolution: the
RMS norm over channels with the residual's addition (training step and
inference), the same norm with an 8-bit output, and counter-based dropout.

Every operator works on [B, C, H, W] maps (NCHW or channels-last) or [N, C]
rows.  ``run`` computes one pass in plain torch operations, or with ``own``
through the framework's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
MASK32 = 0xFFFFFFFF


def listed():
    norm = dict(op="norm", train=True, residual=True, drop="none", p=0.0)
    q8 = dict(op="q8", group=0, kind="e4m3")
    drop = dict(op="drop", residual=True, train=True)
    return [
        # One image's 28x28 map of 192 channels at inference, no residual: launch latency.
        dict(norm, name="norm_infer_one", B=1, C=192, H=28, W=28, dtype="bf16", layout="nchw", train=False,
             residual=False),
        # The stage-1 training step: 32 maps of 96 channels at 56x56, fp32, branch joined to the residual stream.
        dict(norm, name="norm_train_stage1", B=32, C=96, H=56, W=56, dtype="f32", layout="nchw"),
        # The bf16 training shape in channels-last with stochastic depth on the branch.
        dict(norm, name="norm_train_bf16_path", B=64, C=96, H=56, W=56, dtype="bf16", layout="nhwc", drop="sample",
             p=0.1),
        # Odd channel count and plane, ragged rows: a pruned network with element dropout.
        dict(norm, name="norm_train_odd", B=13, C=101, H=23, W=19, dtype="f32", layout="nchw", drop="element", p=0.2),
        # The largest: a 256 MiB map of the shape sweep.
        dict(norm, name="norm_train_large", B=32, C=512, H=64, W=64, dtype="f32", layout="nhwc"),
        # Pooled features of a small serving batch, 8-bit rows for a classifier's product.
        dict(q8, name="q8_rows_small", B=8, C=768, H=1, W=1, dtype="bf16", layout="rows", residual=False),
        # A serving batch of stage-2 maps joined to the residual, block scales of 32 channels.
        dict(q8, name="q8_stage2_groups", B=128, C=192, H=28, W=28, dtype="bf16", layout="nhwc", residual=True,
             group=32),
        # int8 activations of an odd NCHW map, one scale a pixel.
        dict(q8, name="q8_int8_odd", B=9, C=130, H=31, W=27, dtype="f32", layout="nchw", residual=False, kind="int8"),
        # Element dropout joined to the residual at the bf16 training shape, forward and backward.
        dict(drop, name="drop_element_bf16", B=64, C=96, H=56, W=56, dtype="bf16", layout="nchw", mode="element",
             p=0.1),
        # Stochastic depth at stage 2, fp32.
        dict(drop, name="drop_path_stage2", B=32, C=192, H=28, W=28, dtype="f32", layout="nchw", mode="sample", p=0.3),
        # Whole channels of a few odd maps dropped, no residual.
        dict(drop, name="drop_channel_odd", B=3, C=67, H=15, W=17, dtype="f32", layout="nhwc", mode="channel", p=0.5,
             residual=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "q8", "drop"])
    layout = rng.choice(["nchw", "nhwc", "rows"])
    C = _spread(rng, 3, 1024)
    if rng.random() < 0.5:
        C = max(8, C // 8 * 8)
    if layout == "rows":
        B, H, W = _spread(rng, 1, min(1 << 17, (1 << 24) // C)), 1, 1
    else:
        H = _spread(rng, 3, 128)
        W = max(1, min(160, round(H * rng.uniform(0.7, 1.4))))
        if rng.random() < 0.5:
            W = max(8, W // 8 * 8)
        B = _spread(rng, 1, max(1, min(256, (1 << 24) // (C * H * W))))
    case = dict(op=op, B=B, C=C, H=H, W=W, dtype=rng.choice(["f32", "bf16"]), layout=layout,
                residual=rng.random() < 0.6)
    p = round(rng.uniform(0.02, 0.6), 3)
    if op == "norm":
        case["train"] = rng.random() < 0.8
        case["drop"] = rng.choice(["none", "element", "channel", "sample"]) if case["residual"] and case["train"] else "none"
        case["p"] = p if case["drop"] != "none" else 0.0
    elif op == "q8":
        case["group"] = rng.choice([0, 32, 64, 128])
        case["kind"] = rng.choice(["e4m3", "e4m3", "int8"])
    else:
        case["mode"], case["p"], case["train"] = rng.choice(["element", "channel", "sample"]), p, rng.random() < 0.8
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    B, C, H, W = (case[k] for k in "BCHW")
    rows = case["layout"] == "rows"

    def act(spread):
        # Activations of a network: each channel has a spread of its own, a few of them large.
        t = torch.randn((B, C) if rows else (B, C, H, W), generator=gen, device="cuda")
        t *= spread.view(1, C) if rows else spread.view(1, C, 1, 1)
        t = t.to(dt)
        return t.contiguous(memory_format=torch.channels_last) if case["layout"] == "nhwc" else t

    spread = torch.exp(0.6 * torch.randn(C, generator=gen, device="cuda"))
    s = {"case": case, "x": act(spread)}
    if case["residual"]:
        s["residual"] = act(2.0 * spread)
    s["weight"] = 1.0 + 0.2 * torch.randn(C, generator=gen, device="cuda")
    if case.get("train"):
        unit = torch.full((C,), 0.05, device="cuda")
        s["dy"] = act(unit)
        if case["op"] == "norm" and case["residual"]:
            s["dh"] = act(unit)
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63)
    s["offset"] = seed % 1000
    if own:
        import memory_bound_cnn_wtconv_b200 as wt
        mode = case["drop"] if case["op"] == "norm" else case.get("mode", "none")
        s["drop"] = wt.Drop(case["p"], mode, s["seed"], s["offset"]) if mode != "none" else None
    return s


# ---- plain forms ---------------------------------------------------------

def _channel(v, like):
    return v.view(1, -1) if like.dim() == 2 else v.view(1, -1, 1, 1)


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, 2011) on int64 tensors or numbers that hold 32-bit words."""
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # int64 products wrap to the unsigned product's 64 bits
        c0, c1, c2, c3 = ((b >> 32) & MASK32) ^ c1 ^ k0, b & MASK32, ((a >> 32) & MASK32) ^ c3 ^ k1, a & MASK32
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return c0, c1, c2, c3


def _keep(x, mode, p, seed, offset):
    """Truth values, broadcastable to x: the elements that stay."""
    B, C = x.shape[:2]
    pixels = x[0, 0].numel()
    rows = B * pixels if mode == "element" else B
    quads = 1 if mode == "sample" else (C + 3) // 4
    row = torch.arange(rows, device=x.device).view(rows, 1).expand(rows, quads)
    quad = torch.arange(quads, device=x.device).view(1, quads).expand(rows, quads)
    words = _philox(quad, row & MASK32, row >> 32, torch.full_like(row, offset & MASK32), seed & MASK32, seed >> 32)
    u = torch.stack(words, dim=-1).reshape(rows, 4 * quads)[:, :1 if mode == "sample" else C]
    keep = u >= math.floor(p * 2.0 ** 32)
    if mode == "element":
        keep = keep.reshape(B, pixels, C).transpose(1, 2)
        return keep.reshape(x.shape)
    return keep.reshape(B, -1) if x.dim() == 2 else keep.reshape(B, -1, 1, 1)


def _grown(p):
    """The factor of what stays, 1 / (1 - p), a float32 number by definition."""
    return float(np.float32(1.0 / (1.0 - p)))


def _join(s, mode, p):
    """The residual plus the dropped branch, and the mask.  In 64 bits with dropout: x / (1 - p) of 16-bit values
    often lies on the border between two of them."""
    h, keep = s["x"].float(), None
    if mode != "none":
        keep = _keep(s["x"], mode, p, s["seed"], s["offset"])
        h = torch.where(keep, h.double() * _grown(p), 0.0)
    if "residual" in s:
        h = s["residual"].to(h.dtype) + h
    return h, keep


def _plain_norm(s, case):
    dt = s["x"].dtype
    w = _channel(s["weight"], s["x"])
    h, keep = _join(s, case["drop"], case["p"])
    h = h.to(dt)
    hf = h.float()
    r = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS)
    y = (hf * r * w).to(dt)
    out = {"y": y}
    if case["residual"]:
        out["h"] = h
    if case["train"]:
        dy = s["dy"].float()
        g = dy * w
        d = r * (g - hf * ((g * hf).mean(dim=1, keepdim=True) * r * r))
        if "dh" in s:
            d = d + s["dh"].float()
        out["dweight"] = (dy * hf * r).sum(dim=[k for k in range(hf.dim()) if k != 1])
        if keep is not None:
            out["dresidual"] = d.to(dt)
            d = torch.where(keep, d * _grown(case["p"]), 0.0)
        out["dx"] = d.to(dt)
    return out


def _plain_q8(s, case):
    w = _channel(s["weight"], s["x"])
    h = _join(s, "none", 0.0)[0].to(s["x"].dtype)
    hf = h.float()
    y = hf * torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS) * w
    C = y.shape[1]
    G = case["group"] or C
    groups = -(-C // G)
    a = y.abs()
    if groups * G != C:
        a = torch.cat([a, a.new_zeros((a.shape[0], groups * G - C) + tuple(a.shape[2:]))], dim=1)
    top = 448.0 if case["kind"] == "e4m3" else 127.0
    scale = (a.reshape((a.shape[0], groups, G) + tuple(a.shape[2:])).amax(dim=2) / top).clamp_min(2.0 ** -126)
    v = y / scale.repeat_interleave(G, dim=1)[:, :C]
    if case["kind"] == "e4m3":
        q = v.clamp(-top, top).to(torch.float8_e4m3fn)
    else:
        q = v.round().clamp(-top, top).to(torch.bfloat16)
    out = {"q": q, "scale": scale}
    if case["residual"]:
        out["h"] = h
    return out


def _plain_drop(s, case):
    dt = s["x"].dtype
    y, keep = _join(s, case["mode"], case["p"])
    out = {"y": y.to(dt)}
    if case["train"]:
        out["dx"] = torch.where(keep, s["dy"].float() * _grown(case["p"]), 0.0).to(dt)
    return out


# ---- the framework's calls -----------------------------------------------

def _own_norm(s, case):
    import memory_bound_cnn_wtconv_b200 as wt
    if not case["train"]:
        y, h, _ = wt.rms_norm_forward(s["x"], s["weight"], s.get("residual"), eps=EPS, rstd=False)
        return {"y": y, "h": h} if case["residual"] else {"y": y}
    drop = s["drop"]
    y, h, rstd = wt.rms_norm_forward(s["x"], s["weight"], s.get("residual"), drop, eps=EPS)
    dx, dres, dw = wt.rms_norm_backward(h, s["dy"], s["weight"], rstd, s.get("dh"), drop)
    out = {"y": y, "dx": dx, "dweight": dw}
    if case["residual"]:
        out["h"] = h
    if drop is not None:
        out["dresidual"] = dres
    return out


def _own_q8(s, case):
    import memory_bound_cnn_wtconv_b200 as wt
    dtype = torch.float8_e4m3fn if case["kind"] == "e4m3" else torch.int8
    q, scale, h = wt.rms_norm_q8(s["x"], s["weight"], s.get("residual"), eps=EPS, dtype=dtype, group=case["group"])
    out = {"q": q if case["kind"] == "e4m3" else q.to(torch.bfloat16), "scale": scale}
    if case["residual"]:
        out["h"] = h
    return out


def _own_drop(s, case):
    import memory_bound_cnn_wtconv_b200 as wt
    out = {"y": wt.dropout_forward(s["x"], s["drop"], s.get("residual"))}
    if case["train"]:
        out["dx"] = wt.dropout_backward(s["dy"], s["drop"])
    return out


def run(state):
    case = state["case"]
    if own:
        return {"norm": _own_norm, "q8": _own_q8, "drop": _own_drop}[case["op"]](state, case)
    return {"norm": _plain_norm, "q8": _plain_q8, "drop": _plain_drop}[case["op"]](state, case)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    pixels = case["B"] * case["H"] * case["W"]
    n = pixels * case["C"]
    res = int(case["residual"])
    if case["op"] == "norm":
        moved, flops = n * e * (2 + 2 * res), 5 * n
        if case["train"]:
            # h, dy (and dh) read, dx (and the residual's own gradient) written
            moved += n * e * (3 + res + (case["drop"] != "none")) + 4 * pixels * 2
            flops += 10 * n
        drops = case["drop"] == "element"
    elif case["op"] == "q8":
        groups = -(-case["C"] // case["group"]) if case["group"] else 1
        moved, flops, drops = n * (e + 1 + 2 * res * e) + 4 * pixels * groups, 7 * n, False
    else:
        moved, flops = n * e * (2 + res + 2 * case["train"]), 2 * n
        drops = case["mode"] == "element"
    return {"bytes": moved, "flops": flops + (20 * n if drops else 0)}


# ---- the definition in 64 bits -------------------------------------------

def _words(c0, c1, c3, seed):
    """Philox4x32-10 in numpy's unsigned 64-bit words; the rows fit 32 bits here."""
    u = np.uint64
    m, k = u(MASK32), [seed & MASK32, seed >> 32]
    x = [c0.astype(u), c1.astype(u), np.zeros_like(c0, u), np.full_like(c0, c3, u)]
    for r in range(10):
        k0, k1 = u((k[0] + r * 0x9E3779B9) & MASK32), u((k[1] + r * 0xBB67AE85) & MASK32)
        lo, hi = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(hi >> u(32)) ^ x[1] ^ k0, hi & m, (lo >> u(32)) ^ x[3] ^ k1, lo & m]
    return x


def _factor(s, case, mode):
    """The factor of every element of x: 0 or the float32 number next to 1 / (1 - p), as [B, C, pixels] in float64."""
    B, C, P = case["B"], case["C"], case["H"] * case["W"]
    quads = np.arange(1 if mode == "sample" else -(-C // 4))
    rows = np.arange(B * P if mode == "element" else B)
    c1, c0 = np.meshgrid(rows, quads, indexing="ij")
    w = np.stack(_words(c0, c1, s["offset"], s["seed"]), axis=2).reshape(len(rows), -1)
    stay = torch.from_numpy(w >= np.uint64(math.floor(case["p"] * 2.0 ** 32))).cuda()
    if mode == "sample":
        stay = stay[:, :1].reshape(B, 1, 1).expand(B, C, P)
    elif mode == "channel":
        stay = stay[:, :C].reshape(B, C, 1).expand(B, C, P)
    else:
        stay = stay[:, :C].reshape(B, P, C).permute(0, 2, 1)
    return stay.double() * torch.tensor(1.0 / (1.0 - case["p"]), dtype=torch.float64).float().double().item()


def exact(case, seed):
    s = prepare(case, seed)
    B, C, P = case["B"], case["C"], case["H"] * case["W"]
    shape, dt = s["x"].shape, s["x"].dtype

    def wide(name):
        return s[name].double().reshape(B, C, P)

    def back(t):
        return t.reshape(shape)

    mode = case["drop"] if case["op"] == "norm" else case.get("mode", "none")
    f = _factor(s, case, mode) if mode != "none" else 1.0
    joined = wide("x") * f
    if case["residual"]:
        joined = joined + wide("residual")
    if case["op"] == "drop":
        out = {"y": back(joined)}
        if case["train"]:
            out["dx"] = back(wide("dy") * f)
        return out

    # The norm is of the sum as it is stored.
    h = joined.to(dt).double()
    w = s["weight"].double()[None, :, None]
    rms = (h.pow(2).sum(1, keepdim=True) / C + EPS).sqrt()
    y = h / rms * w
    if case["op"] == "q8":
        top = 448.0 if case["kind"] == "e4m3" else 127.0
        G = case["group"] or C
        parts = [y[:, k:k + G] for k in range(0, C, G)]
        scales = [q.abs().amax(1, keepdim=True).div(top).clamp_min(2.0 ** -126) for q in parts]
        scale = torch.cat(scales, 1)
        # The 8-bit value before its rounding; a rounded whole number has no nearer value in 64 bits.
        q = back(torch.cat([a / b for a, b in zip(parts, scales)], 1)) if case["kind"] == "e4m3" else None
        out = {"q": q, "scale": scale.reshape((B, -1) + tuple(shape[2:]))}
        if case["residual"]:
            out["h"] = back(joined)
        return out
    out = {"y": back(y)}
    if case["residual"]:
        out["h"] = back(joined)
    if case["train"]:
        dy = wide("dy")
        out["dweight"] = (dy * h / rms).sum((0, 2))
        d = dy * w / rms - h * (dy * w * h).sum(1, keepdim=True) / (C * rms.pow(3))
        if "dh" in s:
            d = d + wide("dh")
        if mode != "none":
            out["dresidual"] = back(d)
            d = d * f
        out["dx"] = back(d)
    return out
