"""First-order linear attention with a decay for each head, and the group norm
of its outputs, as they are measured.

Two operators, each in a plain form (elementary torch operations in 32 bits)
and through the package's entry points:

- linear attention S_t = g_h S_{t-1} + k_t v_t^T, o_t = S_t^T q_t (prompts,
  training step, single-token step);
- group norm, channels last, with an activation or a gate (forward, backward).

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
        # ---- linear attention
        # decoding one sequence: 16 heads of 128, a call's latency
        {"name": "linear step, 16 heads of 128", "op": "step", "n": 16, "H": 16, "d": 128, "dv": 128, "dtype": "bf16"},
        # decoding a large batch: as many heads as the package's own decode workload
        {"name": "linear step, 4096 heads of 128", "op": "step", "n": 4096, "H": 16, "d": 128, "dv": 128,
         "dtype": "f32"},
        # prefill of a long document, the sizes of the package's headline forward
        {"name": "linear prefill, 65536 tokens, 16 x 128", "op": "linear", "B": 1, "H": 16, "T": 65536, "d": 128,
         "dv": 128, "dtype": "bf16", "layout": "bhtd", "state": True, "ragged": False},
        # prefill of a padded batch of prompts, projections laid out [B, T, H, d]
        {"name": "linear prefill, 8 prompts, 16 x 64", "op": "linear", "B": 8, "H": 16, "T": 2048, "d": 64, "dv": 64,
         "dtype": "bf16", "layout": "bthd", "state": True, "ragged": True},
        # training at the sizes of the package's normalised forward
        {"name": "linear train, 4 x 4096, 16 x 64", "op": "linear_train", "B": 4, "H": 16, "T": 4096, "d": 64,
         "dv": 64, "dtype": "bf16", "layout": "bthd", "state": False, "ragged": False},
        # training on one long sequence in segments (a state comes in, its gradient goes back)
        {"name": "linear train, 16384 tokens, 16 x 128", "op": "linear_train", "B": 1, "H": 16, "T": 16384, "d": 128,
         "dv": 128, "dtype": "bf16", "layout": "bhtd", "state": True, "ragged": False},
        # odd sizes in 32 bits, trained
        {"name": "linear train, 1023 tokens, 3 x 80, f32", "op": "linear_train", "B": 2, "H": 3, "T": 1023, "d": 80,
         "dv": 48, "dtype": "f32", "layout": "bthd", "state": True, "ragged": False},
        # ---- group norm
        # the norm of each head's output and its gate in prefill (16 heads of 128)
        {"name": "group norm gated, 16384 x 2048", "op": "gnorm", "N": 16384, "L": 1, "C": 2048, "G": 16,
         "dtype": "bf16", "act": "silu", "gate": True},
        # the same when decoding a batch of 16
        {"name": "group norm gated, 16 x 2048", "op": "gnorm", "N": 16, "L": 1, "C": 2048, "G": 16, "dtype": "bf16",
         "act": "silu", "gate": True},
        # channels-last feature maps of 64 x 64 positions, norm and activation
        {"name": "group norm, 8 maps of 4096 x 512", "op": "gnorm", "N": 8, "L": 4096, "C": 512, "G": 32,
         "dtype": "bf16", "act": "silu", "gate": False},
        # training: gradients of input, gate, weight and bias (16 heads of 64)
        {"name": "group norm backward, 16384 x 1024", "op": "gnorm_bwd", "N": 16384, "L": 1, "C": 1024, "G": 16,
         "dtype": "bf16", "act": "silu", "gate": True},
        # odd sizes in 32 bits: small feature maps, trained
        {"name": "group norm backward, 5 x 777 x 240, f32", "op": "gnorm_bwd", "N": 5, "L": 777, "C": 240, "G": 8,
         "dtype": "f32", "act": "silu", "gate": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_train", "linear_train", "step", "gnorm", "gnorm", "gnorm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        H = rng.choice([1, 3, 8, 16])
        d = rng.choice([16, 33, 64, 80, 128])
        return {"op": op, "n": H * _log_int(rng, 1, 4096 // H), "H": H, "d": d,
                "dv": rng.choice([d, d, rng.randint(1, 128)]), "dtype": dtype}
    if op in ("linear", "linear_train"):
        d = rng.choice([16, 33, 64, 64, 64, 80, 128, 128])
        dv = rng.choice([d, d, d, rng.randint(1, 128)])
        B, H = rng.randint(1, 8), rng.choice([1, 3, 8, 16])
        # no more than the longest listed prompt's products; a training step costs several times as much, and
        # what misses the tensor cores (32 bits, odd widths) more again
        top = (65536 * 16) // (B * H * (4 if op == "linear_train" else 1))
        if dtype == "f32" or d % 8 or dv % 8:
            top //= 16
        return {"op": op, "B": B, "H": H, "T": _log_int(rng, 1, max(2, min(65536, top))), "d": d, "dv": dv,
                "dtype": dtype, "layout": rng.choice(["bhtd", "bthd"]), "state": rng.random() < 0.5,
                "ragged": rng.random() < 0.3}
    G = rng.choice([1, 3, 8, 16, 32])
    C = G * rng.choice([1, 8, 16, 30, 64, 64, 128])
    L = rng.choice([1, 1, 1, _log_int(rng, 2, 4096)])
    N = _log_int(rng, 1, max(2, (1 << 24) // (C * L)))
    return {"op": op, "N": N, "L": L, "C": C, "G": G, "dtype": dtype, "act": rng.choice(["silu", "silu", "none"]),
            "gate": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs ----
def _randn(gen, shape, dtype, scale=1.0, shift=0.0):
    x = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(shift, scale, generator=gen)
    return x.to(dtype)


def _heads(gen, B, H, T, d, dtype, layout, scale=1.0):
    """[B, H, T, d] values, in that order in memory or in a projection's order [B, T, H, d]."""
    if layout == "bthd":
        return _randn(gen, (B, T, H, d), dtype, scale).transpose(1, 2)
    return _randn(gen, (B, H, T, d), dtype, scale)


def _decays(H):
    """One decay for each head, exp(-2^(-8 h / H)) for h = 1..H: a memory of two tokens to a few hundred."""
    slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)
    return torch.exp(-slopes).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s, dt = case["op"], {"case": case}, _DT[case["dtype"]]
    if op == "step":
        n, d, dv = case["n"], case["d"], case["dv"]
        s["gamma"] = _decays(case["H"])
        s["state0"] = _randn(gen, (n, d, dv), torch.float32)
        s["q"], s["k"] = (_randn(gen, (n, d), dt, d ** -0.5) for _ in range(2))
        s["v"] = _randn(gen, (n, dv), dt)
    elif op in ("linear", "linear_train"):
        B, H, T, d, dv = (case[x] for x in ("B", "H", "T", "d", "dv"))
        s["gamma"] = _decays(H)
        s["q"], s["k"] = (_heads(gen, B, H, T, d, dt, case["layout"], d ** -0.5) for _ in range(2))
        s["v"] = _heads(gen, B, H, T, dv, dt, case["layout"])
        s["h0"] = _randn(gen, (B, H, d, dv), torch.float32) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), device="cuda", generator=gen).to(torch.int32)
            # tokens behind a prompt's end stay as they are: zeros here
            s["o"] = torch.zeros_like(s["v"])
        if op == "linear_train":
            s["do"] = _heads(gen, B, H, T, dv, dt, case["layout"])
            s["dlast"] = _randn(gen, (B, H, d, dv), torch.float32) if case["state"] else None
    else:
        N, L, C = case["N"], case["L"], case["C"]
        shape = (N, C) if L == 1 else (N, L, C)
        level = torch.exp(0.5 * torch.randn((N,) + (1,) * (len(shape) - 1), device="cuda", generator=gen))
        s["x"] = (_randn(gen, shape, torch.float32, 1.0, 0.5) * level).to(dt)
        s["w"], s["b"] = _randn(gen, (C,), torch.float32, 0.1, 1.0), _randn(gen, (C,), torch.float32, 0.1)
        s["z"] = _randn(gen, shape, dt) if case["gate"] else None
        if op == "gnorm_bwd":
            s["dy"] = _randn(gen, shape, dt)
            # mean and reciprocal deviation of each group, as the forward kept them
            t = s["x"].double().reshape(N, L, case["G"], C // case["G"])
            mean = t.mean((1, 3), keepdim=True)
            rstd = 1 / ((t - mean).square().mean((1, 3), keepdim=True) + 1e-5).sqrt()
            s["stats"] = torch.stack([mean.flatten(1), rstd.flatten(1)], -1).float()
    return s


# ------------------------------------------------------------ plain forms ----
_CHUNK = 256


def _in_chunks(x, pad):
    """[B, H, T, c] to 32-bit [B, H, N, _CHUNK, c], zeros behind the end."""
    x = x.float()
    x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad, x.shape[3]))], 2)
    return x.unflatten(2, (-1, min(_CHUNK, x.shape[2])))


def _linear_plain(gamma, q, k, v, h0):
    """o_t = sum_{j<=t} g^(t-j) (q_t . k_j) v_j + g^(t+1) h0^T q_t in chunks: products within a chunk, the
    states entering the chunks as one product with the decays between chunks."""
    B, H, T, _ = q.shape
    L = min(_CHUNK, T)
    pad = -T % L
    q, k, v = (_in_chunks(x, pad) for x in (q, k, v))
    N = q.shape[2]
    g = gamma.double()
    i = torch.arange(L, device=g.device)
    dist = i[:, None] - i
    within = torch.where(dist >= 0, g[:, None, None] ** dist.clamp(min=0), 0.0).float()
    o = (q @ k.transpose(-1, -2) * within[:, None]) @ v
    to_end = (g[:, None] ** (L - 1 - i)).float()
    u = (k * to_end[:, None, :, None]).transpose(-1, -2) @ v  # [B, H, N, d, dv]
    n = torch.arange(N, device=g.device)
    gap = n[:, None] - 1 - n
    between = torch.where(gap >= 0, g[:, None, None] ** (L * gap.clamp(min=0)), 0.0).float()
    s = (between @ u.flatten(3)).unflatten(3, u.shape[3:])
    if h0 is not None:
        s = s + (g[:, None] ** (L * n)).float()[:, :, None, None] * h0[:, :, None]
    o = o + (g[:, None] ** (i + 1)).float()[:, None, :, None] * (q @ s)
    return o.flatten(2, 3)[:, :, :T]


def _last_state_plain(gamma, k, v, h0, lengths):
    """The state after each sequence's last token: sum_j g^(len-1-j) k_j v_j^T + g^len h0."""
    B, H, T, _ = k.shape
    j = torch.arange(T, device=k.device)
    ends = torch.full((B,), T, device=k.device) if lengths is None else lengths
    back = ends.long()[:, None] - 1 - j
    f = torch.where(back[:, None] >= 0, gamma.double()[:, None] ** back[:, None].clamp(min=0), 0.0)
    s = (k.float() * f.float()[..., None]).transpose(-1, -2) @ v.float()
    if h0 is not None:
        s = s + (gamma.double() ** ends[:, None]).float()[..., None, None] * h0
    return s


def _valid(s):
    """[B, 1, T, 1]: the tokens before each sequence's end; None where all are."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["q"].shape[2], device="cuda") < s["lengths"][:, None])[:, None, :, None]


def _keep(x, valid):
    return x if valid is None else torch.where(valid, x, torch.zeros((), device=x.device, dtype=x.dtype))


def _linear_run_plain(s):
    c, gamma, dt = s["case"], s["gamma"], s["q"].dtype
    valid = _valid(s)
    q, k, v = (_keep(s[x], valid) for x in ("q", "k", "v"))
    o = _linear_plain(gamma, q, k, v, s["h0"])
    out = {"o": _keep(o, valid).to(dt)}
    if c["op"] == "linear" or s["h0"] is not None:
        out["last"] = _last_state_plain(gamma, k, v, s["h0"], s["lengths"])
    if c["op"] == "linear":
        return out
    # the gradients are the same sums: dQ over (dO, V, K); dK and dV backwards in time, the gradient of the
    # last state entering behind each sequence's last token
    do = _keep(s["do"], valid)
    h0t = None if s["h0"] is None else s["h0"].transpose(-1, -2)
    out["dq"] = _keep(_linear_plain(gamma, do, v, k, h0t), valid).to(dt)
    dk = _linear_plain(gamma, v.flip(2), do.flip(2), q.flip(2), None).flip(2)
    dv = _linear_plain(gamma, k.flip(2), q.flip(2), do.flip(2), None).flip(2)
    if s["dlast"] is not None:
        T = q.shape[2]
        ends = torch.full((q.shape[0],), T, device="cuda") if s["lengths"] is None else s["lengths"]
        back = (ends.long()[:, None] - 1 - torch.arange(T, device="cuda")).clamp(min=0)
        f = (gamma.double()[:, None] ** back[:, None]).float()[..., None]
        dk = dk + f * (v.float() @ s["dlast"].transpose(-1, -2))
        dv = dv + f * (k.float() @ s["dlast"])
        ahead = (gamma.double()[:, None] ** torch.arange(1, T + 1, device="cuda")).float()[..., None]
        out["d0"] = (q.float() * ahead).transpose(-1, -2) @ do.float() \
            + (gamma.double() ** ends[:, None]).float()[..., None, None] * s["dlast"]
    out["dk"], out["dv"] = _keep(dk, valid).to(dt), _keep(dv, valid).to(dt)
    return out


def _step_plain(s):
    n, H = s["case"]["n"], s["case"]["H"]
    g = s["gamma"].repeat(n // H)[:, None, None]
    state = g * s["state0"] + s["k"].float()[:, :, None] * s["v"].float()[:, None, :]
    o = (s["q"].float()[:, :, None] * state).sum(1)
    return {"o": o.to(s["q"].dtype), "state": state}


def _groups(case, x):
    return x.float().reshape(case["N"], case["L"], case["G"], case["C"] // case["G"])


def _silu_plain(x):
    return x / (1 + torch.exp(-x))


def _gnorm_plain(s, eps=1e-5):
    c = s["case"]
    t = _groups(c, s["x"])
    mean = t.mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt((t - mean).square().mean((1, 3), keepdim=True) + eps)
    z = ((t - mean) * rstd).reshape(s["x"].shape) * s["w"] + s["b"]
    act = _silu_plain if c["act"] == "silu" else (lambda x: x)
    y = act(z) if s["z"] is None else z * act(s["z"].float())
    return {"y": y.to(s["x"].dtype), "stats": torch.stack([mean.flatten(1), rstd.flatten(1)], -1)}


def _gnorm_bwd_plain(s):
    c = s["case"]
    shape, over = s["x"].shape, tuple(range(s["x"].dim() - 1))
    mean, rstd = (s["stats"][..., i].reshape(c["N"], 1, c["G"], 1) for i in (0, 1))
    n = ((_groups(c, s["x"]) - mean) * rstd).reshape(shape)
    z, dy, out = n * s["w"] + s["b"], s["dy"].float(), {}
    at = z if s["z"] is None else s["z"].float()
    sig = 1 / (1 + torch.exp(-at))
    value, slope = (at * sig, sig * (1 + at * (1 - sig))) if c["act"] == "silu" else (at, torch.ones_like(at))
    dz = dy * (slope if s["z"] is None else value)
    if s["z"] is not None:
        out["dgate"] = (dy * z * slope).to(s["x"].dtype)
    g = dz * s["w"]
    gg, nn = _groups(c, g), _groups(c, n)
    dx = rstd * (gg - gg.mean((1, 3), keepdim=True) - nn * (gg * nn).mean((1, 3), keepdim=True))
    out["dx"] = dx.reshape(shape).to(s["x"].dtype)
    out["dw"], out["db"] = (dz * n).sum(over), dz.sum(over)
    return out


def _run_plain(s):
    op = s["case"]["op"]
    if op == "step":
        return _step_plain(s)
    if op in ("linear", "linear_train"):
        return _linear_run_plain(s)
    return _gnorm_plain(s) if op == "gnorm" else _gnorm_bwd_plain(s)


# ------------------------------------------------------- the package's own ----
def _run_own(s):
    c, L = s["case"], _hla2()
    op = c["op"]
    if op == "step":
        state = torch.empty_like(s["state0"])  # the state before the step is kept for the next pass
        o = L.hla2_linear_step(s["state0"], s["q"], s["k"], s["v"], s["gamma"], state_out=state)
        return {"o": o, "state": state}
    if op in ("linear", "linear_train"):
        B, H, _, d = s["q"].shape
        last = None
        if op == "linear" or s["h0"] is not None:
            last = torch.empty((B, H, d, c["dv"]), device="cuda", dtype=torch.float32)
        o = L.hla2_linear_forward(s["q"], s["k"], s["v"], s["gamma"], O=s.get("o"), lengths=s["lengths"],
                                  state_in=s["h0"], state_out=last)
        out = {"o": o} if last is None else {"o": o, "last": last}
        if op == "linear":
            return out
        d0 = torch.empty_like(s["h0"]) if s["h0"] is not None else None
        dq, dk, dv = L.hla2_linear_backward(s["q"], s["k"], s["v"], s["gamma"], s["do"], lengths=s["lengths"],
                                            state_in=s["h0"], dstate_out=s["dlast"], dstate_in=d0)
        out["dq"] = dq
        if d0 is not None:
            out["d0"] = d0
        out["dk"], out["dv"] = dk, dv
        return out
    if op == "gnorm":
        stats = torch.empty((c["N"], c["G"], 2), device="cuda", dtype=torch.float32)
        y = L.hla2_groupnorm(s["x"], c["G"], s["w"], s["b"], gate=s["z"], activation=c["act"], stats=stats)
        return {"y": y, "stats": stats}
    dx, dw, db, dgate = L.hla2_groupnorm_backward(s["x"], s["dy"], s["stats"], s["w"], s["b"], gate=s["z"],
                                                  activation=c["act"])
    out = {} if s["z"] is None else {"dgate": dgate}
    return {**out, "dx": dx, "dw": dw, "db": db}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work ----
def work(case):
    """What one pass cannot do without: inputs read once, outputs written once; the operations of the
    definitions (the recurrence token by token), an exponential or root counted as one.  A ragged
    batch counts half of its tokens."""
    op, e = case["op"], _SIZE[case["dtype"]]
    if op == "step":
        n, d, dv = case["n"], case["d"], case["dv"]
        return {"bytes": n * (8 * d * dv + e * (2 * d + 2 * dv)) + 4 * case["H"], "flops": 5 * n * d * dv}
    if op in ("linear", "linear_train"):
        B, H, d, dv = (case[x] for x in ("B", "H", "d", "dv"))
        tokens = B * H * case["T"]
        if case["ragged"]:
            tokens = max(1, tokens // 2)
        state = 4 * B * H * d * dv
        nb = tokens * e * (2 * d + 2 * dv)
        if op == "linear":
            return {"bytes": nb + state * (2 if case["state"] else 1), "flops": 5 * tokens * d * dv}
        nb += tokens * e * (4 * d + 3 * dv)  # q, k, v, dO read, dq, dk, dv written
        return {"bytes": nb + state * (5 if case["state"] else 0), "flops": 17 * tokens * d * dv}
    n, C = case["N"] * case["L"] * case["C"], case["C"]
    stats = 8 * case["N"] * case["G"]
    if op == "gnorm":
        return {"bytes": n * e * (3 if case["gate"] else 2) + 8 * C + stats, "flops": 12 * n}
    return {"bytes": n * e * (5 if case["gate"] else 3) + 16 * C + stats, "flops": 24 * n}


# ------------------------------------------------------------ 64-bit values ----
def _linear_exact(g, q, k, v, state, len_b, reverse=False):
    """Runs of 64 tokens, one after another in 64 bits (backwards in time when `reverse`): the outputs and
    the state behind the last run.  A run's tokens beyond len_b are absent."""
    B, H, T, _ = q.shape
    o = torch.zeros(B, H, T, v.shape[3], dtype=torch.float64, device=q.device)
    lg = g.view(1, H, 1)
    for n in (range(-(-T // 64) - 1, -1, -1) if reverse else range(-(-T // 64))):
        a, z = 64 * n, min(T, 64 * n + 64)
        pos = torch.arange(a, z, device=q.device)
        here = (pos < len_b[:, None])[:, None, :, None]  # [B, 1, l, 1]
        qq, kk, vv = (torch.where(here, x[:, :, a:z].double(), 0.0) for x in (q, k, v))
        count = here.sum(2).view(B, 1, 1).double()
        r = (pos - a).view(1, 1, -1).double()
        if reverse:
            before, after = (count - 1 - r).clamp(min=0), r + 1
            near = (pos[None] - pos[:, None]).double()
        else:
            before, after = r + 1, (count - 1 - r).clamp(min=0)
            near = (pos[:, None] - pos[None]).double()
        w = torch.where(near >= 0, lg.unsqueeze(-1) ** near.clamp(min=0), 0.0)
        o[:, :, a:z] = torch.where(here, (torch.einsum("bhic,bhjc->bhij", qq, kk) * w) @ vv
                                   + (lg ** before)[..., None] * (qq @ state), 0.0)
        state = (lg ** count)[..., None] * state + torch.einsum("bhjc,bhjv->bhcv", kk * (lg ** after)[..., None], vv)
    return o, state


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "step":
        g = s["gamma"].double().repeat(case["n"] // case["H"]).view(-1, 1, 1)
        state = torch.baddbmm(g * s["state0"].double(), s["k"].double().unsqueeze(2), s["v"].double().unsqueeze(1))
        return {"o": torch.einsum("nc,ncv->nv", s["q"].double(), state), "state": state}
    if op in ("linear", "linear_train"):
        B, H, T, d, dv = (case[x] for x in ("B", "H", "T", "d", "dv"))
        g = s["gamma"].double()
        len_b = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
        zero = torch.zeros(B, H, d, dv, dtype=torch.float64, device="cuda")
        h0 = zero if s["h0"] is None else s["h0"].double()
        o, last = _linear_exact(g, s["q"], s["k"], s["v"], h0, len_b)
        out = {"o": o}
        if op == "linear" or s["h0"] is not None:
            out["last"] = last
        if op == "linear":
            return out
        dlast = zero if s["dlast"] is None else s["dlast"].double()
        out["dq"], _ = _linear_exact(g, s["do"], s["v"], s["k"], h0.mT, len_b)
        out["dv"], d0 = _linear_exact(g, s["k"], s["q"], s["do"], dlast, len_b, reverse=True)
        out["dk"], _ = _linear_exact(g, s["v"], s["do"], s["q"], dlast.mT, len_b, reverse=True)
        if s["h0"] is not None:
            out["d0"] = d0
        return out
    # every group a row of its own
    N, L, C, G = (case[x] for x in ("N", "L", "C", "G"))

    def rows(x):
        return x.double().view(N, L, G, C // G).transpose(1, 2).flatten(2)

    def back(r):
        return r.view(N, G, L, C // G).transpose(1, 2).reshape(s["x"].shape)

    x = rows(s["x"])
    w, b = (t.double().view(1, 1, C).expand(N, L, C) for t in (s["w"], s["b"]))
    w, b = rows(w.reshape(N, L, C)), rows(b.reshape(N, L, C))
    act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.Identity()
    if op == "gnorm":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        z = (x - mean) / (var + 1e-5).sqrt() * w + b
        y = act(z) if s["z"] is None else z * act(rows(s["z"]))
        return {"y": back(y), "stats": torch.cat([mean, (var + 1e-5).rsqrt()], -1)}
    mean, rstd = s["stats"].double().split(1, -1)
    n = (x - mean) * rstd
    dy = rows(s["dy"])
    with torch.enable_grad():
        z = (n * w + b).requires_grad_()
        gate = None if s["z"] is None else rows(s["z"]).requires_grad_()
        y = act(z) if gate is None else z * act(gate)
        grads = torch.autograd.grad(y, [z] if gate is None else [z, gate], dy)
    dz = grads[0]
    t = dz * w
    dx = rstd * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    out = {} if gate is None else {"dgate": back(grads[1])}
    return {**out, "dx": back(dx), "dw": back(dz * n).reshape(-1, C).sum(0), "db": back(dz).reshape(-1, C).sum(0)}
