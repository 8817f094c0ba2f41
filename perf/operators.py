"""The operators around an attention layer, as they are measured.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and through the package's entry points:

- the gated linear recurrence h_t = a_t h_{t-1} + u_t along the tokens of each
  head (forward, training step, single-token step);
- root-mean-square norm with the residual's addition (forward, forward with an
  8-bit output and a scale for each row, backward);
- rotary positions with several axes on queries and keys (and its inverse,
  which is its backward).

``own`` selects the side that ``run`` takes.
"""
import math

import torch

own = False

_PKG = None


def _hla2():
    global _PKG
    if _PKG is None:
        from higher_order_linear_gb300 import hla2
        _PKG = hla2
    return _PKG


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # ---- gated linear recurrence
        # decoding one sequence: 16 heads of 128, a call's latency
        {"name": "step, 16 heads of 128", "op": "step", "n": 16, "d": 128, "dtype": "bf16", "out": "bf16",
         "form": "sigmoid", "shared": False},
        # prefill of a long document, the sizes of the package's headline forward
        {"name": "scan, 65536 tokens, 16 x 128", "op": "scan", "B": 1, "H": 16, "T": 65536, "d": 128, "dtype": "bf16",
         "out": "f32", "form": "sigmoid", "shared": False, "reset": 0.0, "layout": "bhtd", "state": True},
        # training on packed documents (a reset where each begins), projections laid out [B, T, H, d]
        {"name": "scan train, 4 x 4096, 16 x 64", "op": "scan_train", "B": 4, "H": 16, "T": 4096, "d": 64,
         "dtype": "bf16", "out": "bf16", "form": "sigmoid", "shared": False, "reset": 0.002, "layout": "bthd",
         "state": True},
        # odd sizes in 32 bits, one decay for all channels of a head, trained
        {"name": "scan train, 1023 tokens, 3 x 80, f32", "op": "scan_train", "B": 2, "H": 3, "T": 1023, "d": 80,
         "dtype": "f32", "out": "f32", "form": "decay", "shared": True, "reset": 0.0, "layout": "bhtd", "state": False},
        # ---- root-mean-square norm
        # the norm before a layer in prefill: residual added, both kept
        {"name": "norm, 16384 rows of 2048", "op": "norm", "rows": 16384, "C": 2048, "dtype": "bf16", "out": "bf16",
         "residual": True},
        # the norm of each head's attention output (32 bits in, 16 bits out)
        {"name": "norm of heads, 2^20 rows of 128", "op": "norm", "rows": 1 << 20, "C": 128, "dtype": "f32",
         "out": "bf16", "residual": False},
        # decoding a batch: 8-bit input of the next projection
        {"name": "norm 8-bit, 16 rows of 2048", "op": "norm_q8", "rows": 16, "C": 2048, "dtype": "bf16",
         "residual": True},
        # prefill with 8-bit projections, wide rows
        {"name": "norm 8-bit, 8191 rows of 8192", "op": "norm_q8", "rows": 8191, "C": 8192, "dtype": "bf16",
         "residual": True},
        # training
        {"name": "norm backward, 16384 x 2048", "op": "norm_bwd", "rows": 16384, "C": 2048, "dtype": "bf16",
         "residual": True},
        # ---- rotary positions
        # a long video: queries and keys of 16 heads, positions of time, height and width
        {"name": "rotary, 65536 tokens, 16 x 128", "op": "rotary", "B": 1, "H": 16, "HK": 16, "T": 65536, "d": 128,
         "axes": 3, "rot": 128, "dtype": "bf16", "interleaved": False, "inverse": False, "layout": "bthd"},
        # decoding 256 sequences, one token each, shared key heads
        {"name": "rotary, 256 single tokens", "op": "rotary", "B": 256, "H": 16, "HK": 4, "T": 1, "d": 128, "axes": 3,
         "rot": 128, "dtype": "bf16", "interleaved": False, "inverse": False, "layout": "bthd"},
        # odd sizes in 32 bits, part of the channels rotated, gradients on their way back
        {"name": "rotary inverse, 777 tokens, f32", "op": "rotary", "B": 3, "H": 5, "HK": 0, "T": 777, "d": 80,
         "axes": 2, "rot": 72, "dtype": "f32", "interleaved": True, "inverse": True, "layout": "bhtd"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "step", "norm", "norm", "norm_q8", "norm_bwd",
                     "rotary", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        return {"op": op, "n": _log_int(rng, 1, 8192), "d": rng.choice([1, 16, 33, 64, 80, 96, 128]), "dtype": dtype,
                "out": rng.choice(["f32", dtype]), "form": rng.choice(["sigmoid", "decay"]),
                "shared": rng.random() < 0.3}
    if op in ("scan", "scan_train"):
        d = rng.choice([16, 33, 64, 64, 80, 96, 128, 128])
        B, H = rng.randint(1, 4), rng.choice([1, 3, 8, 16])
        # at most a fifth of the largest listed case's tokens: a training step moves more for each
        top = min(65536, (65536 * 16 * 128) // (5 * B * H * d))
        return {"op": op, "B": B, "H": H, "T": _log_int(rng, 1, top), "d": d, "dtype": dtype,
                "out": rng.choice(["f32", "bf16"]) if op == "scan" else dtype, "form": rng.choice(["sigmoid", "decay"]),
                "shared": rng.random() < 0.3, "reset": rng.choice([0.0, 0.002, 0.1]),
                "layout": rng.choice(["bhtd", "bthd"]), "state": rng.random() < 0.5}
    if op in ("norm", "norm_q8", "norm_bwd"):
        C = rng.choice([64, 128, 1000, 1024, 2048, 4096, 8192, _log_int(rng, 1, 16384)])
        rows = _log_int(rng, 1, max(2, min(1 << 20, (1 << 25) // C)))
        case = {"op": op, "rows": rows, "C": C, "dtype": dtype, "residual": rng.random() < 0.6}
        if op == "norm":
            case["out"] = rng.choice(["bf16", dtype])
        return case
    d = rng.choice([16, 64, 80, 128, 128])
    B, H = rng.randint(1, 4), rng.choice([1, 3, 8, 16])
    # 32-bit values only at the positions of an image or a video: at the end of one long axis the
    # plain form's own 32-bit angle (position times frequency) is off by more than such values are
    axes = rng.choice([2, 3] if dtype == "f32" else [1, 2, 3])
    top = min(4096 if dtype == "f32" else 65536, (1 << 25) // (B * H * d))
    return {"op": op, "B": B, "H": H, "HK": rng.choice([0, 1, H]), "T": _log_int(rng, 1, top),
            "d": d, "axes": axes, "rot": rng.choice([d, d, d - 8]), "dtype": dtype, "interleaved": rng.random() < 0.4,
            "inverse": rng.random() < 0.4, "layout": rng.choice(["bhtd", "bthd"])}


# ----------------------------------------------------------------- inputs ----
def _randn(gen, shape, dtype, scale=1.0, shift=0.0):
    x = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(shift, scale, generator=gen)
    return x.to(dtype)


def _heads(gen, B, H, T, d, dtype, layout, **kw):
    """[B, H, T, d] values, in that order in memory or in a projection's order [B, T, H, d]."""
    if layout == "bthd":
        return _randn(gen, (B, T, H, d), dtype, **kw).transpose(1, 2)
    return _randn(gen, (B, H, T, d), dtype, **kw)


def _gates(gen, case, shape):
    """Logits around 2 (a memory of ten to a few hundred tokens), or decays in (0.9, 1) with some zeros."""
    dt = _DT[case["dtype"]]
    if case["form"] == "sigmoid":
        return _randn(gen, shape, dt, scale=1.5, shift=2.0)
    a = 1.0 - 0.1 * torch.rand(shape, device="cuda", generator=gen)
    a[torch.rand(shape, device="cuda", generator=gen) < 0.001] = 0.0
    return a.to(dt)


def sections_of(case):
    """How many frequency pairs each axis has: the first axis takes what does not divide."""
    pairs, axes = case["rot"] // 2, case["axes"]
    each = pairs // axes
    return (pairs - each * (axes - 1),) + (each,) * (axes - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    dt = _DT[case["dtype"]]
    if op == "step":
        n, d = case["n"], case["d"]
        s["state0"] = _randn(gen, (n, d), torch.float32)
        s["x"] = _randn(gen, (n, d), dt)
        s["g"] = _gates(gen, case, (n,) if case["shared"] else (n, d))
    elif op in ("scan", "scan_train"):
        B, H, T, d = case["B"], case["H"], case["T"], case["d"]
        s["x"] = _heads(gen, B, H, T, d, dt, case["layout"])
        if case["shared"]:
            s["g"] = _gates(gen, case, (B, H, T))
        elif case["layout"] == "bthd":
            s["g"] = _gates(gen, case, (B, T, H, d)).transpose(1, 2)
        else:
            s["g"] = _gates(gen, case, (B, H, T, d))
        s["reset"] = (torch.rand((B, T), device="cuda", generator=gen) < case["reset"]) if case["reset"] > 0 else None
        s["h0"] = _randn(gen, (B, H, d), torch.float32) if case["state"] else None
        if op == "scan_train":
            s["do"] = _heads(gen, B, H, T, d, _DT[case["out"]], case["layout"])
            s["dlast"] = _randn(gen, (B, H, d), torch.float32) if case["state"] else None
    elif op in ("norm", "norm_q8", "norm_bwd"):
        rows, C = case["rows"], case["C"]
        level = torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=gen))
        s["x"] = (_randn(gen, (rows, C), torch.float32) * level).to(dt)
        s["w"] = _randn(gen, (C,), dt, scale=0.1, shift=1.0)
        s["r"] = _randn(gen, (rows, C), dt) if case["residual"] else None
        if op == "norm_bwd":
            s["dy"] = _randn(gen, (rows, C), dt)
    else:
        B, T, d = case["B"], case["T"], case["d"]
        s["q"] = _heads(gen, B, case["H"], T, d, dt, case["layout"])
        s["k"] = _heads(gen, B, case["HK"], T, d, dt, case["layout"]) if case["HK"] else None
        # tokens of a video in order: frames of 32 x 32, a start of its own for each sequence
        t = torch.arange(T, device="cuda") + torch.randint(0, 4096, (B, 1), device="cuda", generator=gen)
        grid = (t // 1024, t // 32 % 32, t % 32) if case["axes"] == 3 else (t // 32, t % 32) if case["axes"] == 2 else (t,)
        s["pos"] = torch.stack(grid).to(torch.int32)
        secs = sections_of(case)
        s["sections"] = secs
        s["axis"] = torch.cat([torch.full((m,), i, dtype=torch.int64) for i, m in enumerate(secs)]).cuda()
        s["freq"] = (10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) * 2 / case["rot"])).float().cuda()
    return s


# ------------------------------------------------------------ plain forms ----
def _scan_plain(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 2, by doubling: after the pass with distance k, (a, u) at t
    stand for the last 2k tokens."""
    T, k = u.shape[2], 1
    a = a.expand_as(u)
    while k < T:
        u = torch.cat([u[:, :, :k], u[:, :, k:] + a[:, :, k:] * u[:, :, :-k]], 2)
        a = torch.cat([a[:, :, :k], a[:, :, k:] * a[:, :, :-k]], 2)
        k *= 2
    return u


def _gate_plain(form, x, g):
    """(a, u) in 32 bits."""
    a = g.float()
    if a.dim() < x.dim():
        a = a[..., None]
    if form == "sigmoid":
        a = 1 / (1 + torch.exp(-a))
        return a, (1 - a) * x.float()
    return a, x.float()


def _with_start(a, u, reset, h0):
    """The decays with the resets in them, and the first token's input with the state before it."""
    if reset is not None:
        a = torch.where(reset[:, None, :, None], torch.zeros((), device=a.device), a)
    if h0 is not None:
        u = torch.cat([u[:, :, :1] + a[:, :, :1] * h0[:, :, None], u[:, :, 1:]], 2)
    return a, u


def _scan_forward_plain(s):
    c = s["case"]
    a, u = _gate_plain(c["form"], s["x"], s["g"])
    a, u = _with_start(a, u, s["reset"], s["h0"])
    return a, _scan_plain(a, u)


def _scan_train_plain(s):
    c = s["case"]
    x, g = s["x"].float(), s["g"]
    a, h = _scan_forward_plain(s)
    before = s["h0"][:, :, None] if s["h0"] is not None else torch.zeros_like(h[:, :, :1])
    before = torch.cat([before, h[:, :, :-1]], 2)
    if s["reset"] is not None:
        before = torch.where(s["reset"][:, None, :, None], torch.zeros((), device=x.device), before)
    dh = s["do"].float()
    if s["dlast"] is not None:
        dh = torch.cat([dh[:, :, :-1], dh[:, :, -1:] + s["dlast"][:, :, None]], 2)
    later = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], 2)  # a_{t+1}
    lam = _scan_plain(later.flip(2), dh.flip(2)).flip(2)
    if c["form"] == "sigmoid":
        gate, _ = _gate_plain("sigmoid", x, g)
        dx, dg = lam * (1 - gate), lam * (before - x) * gate * (1 - gate)
    else:
        dx, dg = lam, lam * before
    if c["shared"]:
        dg = dg.sum(-1)
    d0 = a[:, :, 0] * lam[:, :, 0]
    out = {"o": h.to(_DT[c["out"]]), "dx": dx.to(s["x"].dtype), "dg": dg.to(g.dtype)}
    if s["h0"] is not None:
        out["last"], out["d0"] = h[:, :, -1].contiguous(), d0
    return out


def _norm_plain(s, eps=1e-6):
    t = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    rstd = 1 / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    return t, t * rstd * s["w"].float()


def _norm_bwd_plain(s, eps=1e-6):
    t, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    rstd = 1 / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    n, gw = t * rstd, dy * w
    dx = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
    if s["r"] is not None:  # what reaches the residual stream from the layers above
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * n).sum(0)}


def _rotate_plain(x, ang, interleaved, inverse, rot):
    v = x.float()
    co, si = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if inverse:
        si = -si
    if interleaved:
        a, b = v[..., 0:rot:2], v[..., 1:rot:2]
        turned = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
    else:
        a, b = v[..., : rot // 2], v[..., rot // 2 : rot]
        turned = torch.cat([a * co - b * si, a * si + b * co], -1)
    return torch.cat([turned, v[..., rot:]], -1).to(x.dtype)


def _rotary_plain(s):
    c = s["case"]
    ang = s["pos"].float()[s["axis"]].permute(1, 2, 0) * s["freq"]  # [B, T, pairs]
    out = [_rotate_plain(s["q"], ang, c["interleaved"], c["inverse"], c["rot"])]
    if s["k"] is not None:
        out.append(_rotate_plain(s["k"], ang, c["interleaved"], c["inverse"], c["rot"]))
    return out


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "step":
        a, u = _gate_plain(c["form"], s["x"], s["g"])
        h = a * s["state0"] + u
        return {"o": h.to(_DT[c["out"]]), "state": h}
    if op == "scan":
        _, h = _scan_forward_plain(s)
        return {"o": h.to(_DT[c["out"]]), "last": h[:, :, -1].contiguous()}
    if op == "scan_train":
        return _scan_train_plain(s)
    if op == "norm":
        t, y = _norm_plain(s)
        out = {"y": y.to(_DT[c["out"]])}
        if s["r"] is not None:
            out["sum"] = t.to(s["x"].dtype)
        return out
    if op == "norm_q8":
        t, y = _norm_plain(s)
        top = y.abs().amax(-1, keepdim=True)
        scale = torch.where(top == 0, torch.ones_like(top), top / 448.0)
        out = {"q": (y / scale).to(torch.float8_e4m3fn), "scale": scale[:, 0]}
        if s["r"] is not None:
            out["sum"] = t.to(s["x"].dtype)
        return out
    if op == "norm_bwd":
        return _norm_bwd_plain(s)
    return _rotary_plain(s)


# ------------------------------------------------------- the package's own ----
def _run_own(s):
    c, L = s["case"], _hla2()
    op = c["op"]
    if op == "step":
        state = torch.empty_like(s["state0"])  # the state before the step is kept for the next pass
        o = L.hla2_gated_step(s["state0"], s["x"], s["g"], form=c["form"], out_dtype=_DT[c["out"]], state_out=state)
        return {"o": o, "state": state}
    if op == "scan":
        B, H, _, d = s["x"].shape
        last = torch.empty((B, H, d), device="cuda", dtype=torch.float32)
        o = L.hla2_gated_scan(s["x"], s["g"], form=c["form"], reset=s["reset"], state_in=s["h0"], state_out=last,
                              out_dtype=_DT[c["out"]])
        return {"o": o, "last": last}
    if op == "scan_train":
        B, H, T, d = s["x"].shape
        last = torch.empty((B, H, d), device="cuda", dtype=torch.float32)
        carry = torch.empty((B, H, L.hla2_gated_scan_carry_len(T, d)), device="cuda", dtype=torch.float32)
        o = L.hla2_gated_scan(s["x"], s["g"], form=c["form"], reset=s["reset"], state_in=s["h0"], state_out=last,
                              carry=carry, out_dtype=_DT[c["out"]])
        d0 = torch.empty_like(s["h0"]) if s["h0"] is not None else None
        dx, dg = L.hla2_gated_scan_backward(s["x"], s["g"], s["do"], carry, form=c["form"], reset=s["reset"],
                                            dstate_out=s["dlast"], dstate_in=d0)
        out = {"o": o, "dx": dx, "dg": dg}
        if s["h0"] is not None:
            out["last"], out["d0"] = last, d0
        return out
    if op == "norm":
        y, t = L.hla2_rmsnorm(s["x"], s["w"], residual=s["r"], out_dtype=_DT[c["out"]])
        return {"y": y} if s["r"] is None else {"y": y, "sum": t}
    if op == "norm_q8":
        q, scale, t = L.hla2_rmsnorm_q8(s["x"], s["w"], residual=s["r"])
        return {"q": q, "scale": scale} if s["r"] is None else {"q": q, "scale": scale, "sum": t}
    if op == "norm_bwd":
        dx, dw = L.hla2_rmsnorm_backward(s["x"], s["dy"], s["w"], dS=s["r"])
        return {"dx": dx, "dw": dw}
    q, k = L.hla2_rotary(s["q"], s["pos"], s["freq"], s["sections"], K=s["k"], interleaved=c["interleaved"],
                         inverse=c["inverse"])
    return [q] if s["k"] is None else [q, k]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work ----
def work(case):
    """What one pass cannot do without: inputs read once, outputs written once; the
    operations of the definitions, an exponential, sine or root counted as one."""
    op, e = case["op"], _SIZE[case["dtype"]]
    if op == "step":
        n = case["n"] * case["d"]
        g = case["n"] if case["shared"] else n
        return {"bytes": n * (4 + e + 4 + _SIZE[case["out"]]) + g * e, "flops": 6 * n}
    if op in ("scan", "scan_train"):
        n = case["B"] * case["H"] * case["T"] * case["d"]
        rows = case["B"] * case["H"]
        g = rows * case["T"] if case["shared"] else n
        reset = case["B"] * case["T"] if case["reset"] > 0 else 0
        state = rows * case["d"] * 4
        out = _SIZE[case["out"]]
        nb = n * (e + out) + g * e + reset + state * (2 if case["state"] else 1)
        if op == "scan":
            return {"bytes": nb, "flops": 6 * n}
        # a forward and a backward pass: the second reads x, g, the gradient and writes dx, dg
        nb += n * (e + out + e) + 2 * g * e + reset + state * (2 if case["state"] else 0)
        return {"bytes": nb, "flops": 20 * n}
    if op in ("norm", "norm_q8", "norm_bwd"):
        n, C = case["rows"] * case["C"], case["C"]
        if op == "norm_bwd":
            return {"bytes": n * e * (4 if case["residual"] else 3) + C * (e + 4), "flops": 12 * n}
        out = _SIZE[case["out"]] if op == "norm" else 1
        nb = n * (e * (3 if case["residual"] else 1) + out) + C * e + (4 * case["rows"] if op == "norm_q8" else 0)
        return {"bytes": nb, "flops": 6 * n}
    n = case["B"] * (case["H"] + case["HK"]) * case["T"] * case["d"]
    return {"bytes": 2 * n * e + case["axes"] * case["B"] * case["T"] * 4, "flops": 3 * n}


# ------------------------------------------------------------ 64-bit values ----
def _scan_exact(a, u, h0):
    """The recurrence token by token in 64 bits, all heads (and runs of about sqrt(T) tokens) at once:
    each run from zero with its decay, then the runs in order."""
    B, H, T, d = u.shape
    K = max(1, math.isqrt(T))
    N = -(-T // K)
    pad = N * K - T
    if pad:
        a = torch.cat([a, torch.ones((B, H, pad, d), device=a.device, dtype=a.dtype)], 2)
        u = torch.cat([u, torch.zeros((B, H, pad, d), device=a.device, dtype=a.dtype)], 2)
    a, u = a.reshape(B, H, N, K, d).clone(), u.reshape(B, H, N, K, d).clone()
    for k in range(1, K):
        u[:, :, :, k] += a[:, :, :, k] * u[:, :, :, k - 1]
        a[:, :, :, k] *= a[:, :, :, k - 1]
    h = torch.zeros((B, H, d), device=a.device, dtype=a.dtype) if h0 is None else h0.double()
    for n in range(N):
        u[:, :, n] += a[:, :, n] * h[:, :, None]
        h = u[:, :, n, K - 1]
    return u.reshape(B, H, N * K, d)[:, :, :T]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "step":
        g, x = s["g"].double(), s["x"].double()
        g = g[:, None] if case["shared"] else g
        a = torch.sigmoid(g) if case["form"] == "sigmoid" else g
        h = a * s["state0"].double() + (torch.sigmoid(-g) * x if case["form"] == "sigmoid" else x)
        return {"o": h, "state": h}
    if op in ("scan", "scan_train"):
        x, g = s["x"].double(), s["g"].double()
        if case["shared"]:
            g = g[..., None].expand_as(x)
        gate = torch.sigmoid(g) if case["form"] == "sigmoid" else g
        rest = torch.sigmoid(-g) if case["form"] == "sigmoid" else torch.ones_like(g)
        keep = torch.ones_like(x) if s["reset"] is None else (~s["reset"]).double()[:, None, :, None].expand_as(x)
        h = _scan_exact(gate * keep, rest * x, s["h0"])
        if op == "scan":
            return {"o": h, "last": h[:, :, -1]}
        dh = s["do"].double()
        if s["dlast"] is not None:
            dh[:, :, -1] += s["dlast"].double()
        # backwards in time: the gradient of h_t is its own and a_{t+1} times the next one's
        shifted = torch.roll((gate * keep).flip(2), 1, 2)
        shifted[:, :, 0] = 0
        lam = _scan_exact(shifted, dh.flip(2), None).flip(2)
        prev = torch.roll(h, 1, 2)
        prev[:, :, 0] = 0 if s["h0"] is None else s["h0"].double()
        prev *= keep
        dg = lam * (prev - x) * gate * rest if case["form"] == "sigmoid" else lam * prev
        out = {"o": h, "dx": lam * rest, "dg": dg.sum(-1) if case["shared"] else dg}
        if s["h0"] is not None:
            out["last"], out["d0"] = h[:, :, -1], (gate * keep * lam)[:, :, 0]
        return out
    if op in ("norm", "norm_q8"):
        t = s["x"].double() + (s["r"].double() if s["r"] is not None else 0)
        y = t / (t.square().sum(-1, keepdim=True) / case["C"] + 1e-6).sqrt() * s["w"].double()
        out = {"sum": t} if s["r"] is not None else {}
        if op == "norm":
            return {"y": y, **out}
        scale = y.abs().max(-1, keepdim=True).values / 448
        scale[scale == 0] = 1
        return {"q": y / scale, "scale": scale[:, 0], **out}  # q before its rounding to 8 bits
    if op == "norm_bwd":
        t, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        ms = t.square().sum(-1, keepdim=True) / case["C"] + 1e-6
        # y = w t ms^(-1/2)  =>  dt = ms^(-1/2) w dy - t ms^(-3/2) sum(w dy t) / C
        dx = w * dy / ms.sqrt() - t * (w * dy * t).sum(-1, keepdim=True) / case["C"] / ms ** 1.5
        return {"dx": dx + (s["r"].double() if s["r"] is not None else 0), "dw": (dy * t / ms.sqrt()).sum(0)}
    ang = torch.stack([s["pos"][i].double()[..., None] * f.double() for i, f in
                       zip(s["axis"].tolist(), s["freq"])], 2)[..., 0]  # [B, T, pairs]
    z = torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)[:, None]
    out = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        v, rot = x.double(), case["rot"]
        if case["interleaved"]:
            w = torch.view_as_complex(v[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
            turned = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(v[..., : rot // 2].contiguous(), v[..., rot // 2 : rot].contiguous()) * z
            turned = torch.cat([w.real, w.imag], -1)
        out.append(torch.cat([turned, v[..., rot:]], -1))
    return out
