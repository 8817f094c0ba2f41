"""Group norm, channels last (hla2_groupnorm, hla2_groupnorm_backward), against the formulas in 64 bits.

Tolerances, fixed before the first run, u = 2^-24:
- a mean or a mean square over a group is off by at most 30 u of the mean magnitude of its terms
  (eight values to a thread, the rest added in trees, runs of positions or 64 bits), which moves
  n = (x - mean) rstd by 30 u (A rstd + |n|), A the group's largest |x|, and a few roundings of |n|;
- the sigmoid is an exponential and a quotient of a few units in the last place, and an argument
  rounded to u |x|: (1.5 |x| + 10) u of itself; the slope of silu changes by at most 0.5 |dx|;
- what is formed from these adds up as the formulas say; 8 u for the products and sums on the way;
- dw and db are sums over rows: one rounding for each row at most;
- bf16 results: half a unit in the last place of each value on top.
"""
import pytest
import torch

from _rounding import excess
from higher_order_linear_gb300 import hla2

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(N, L, C, G, dtype, gate, wdtype, seed=0, shift=0.5):
    gen = torch.Generator().manual_seed(seed)
    shape = (N, C) if L == 0 else (N, L, C)
    x = {"x": (torch.randn(shape, generator=gen) * 1.5 + shift).to(dtype),
         "dy": torch.randn(shape, generator=gen).to(dtype),
         "z": (2 * torch.randn(shape, generator=gen)).to(dtype) if gate else None, "w": None, "b": None, "G": G}
    if wdtype is not None:
        x["w"] = (1 + 0.2 * torch.randn(C, generator=gen)).to(wdtype)
        x["b"] = (0.2 * torch.randn(C, generator=gen)).to(wdtype)
    return x


def formulas(x, act, eps=1e-5):
    """y, stats, dx, dw, db, dgate in 64 bits, each with what it may be off by."""
    shape, G = x["x"].shape, x["G"]
    N, C = shape[0], shape[-1]
    t = x["x"].double().reshape(N, -1, G, C // G)
    mean = t.mean((1, 3), keepdim=True)
    var = (t - mean).square().mean((1, 3), keepdim=True)
    rstd = (var + eps).rsqrt()
    top = t.abs().amax((1, 3), keepdim=True)

    def flat(v):
        return v.expand(t.shape).reshape(shape)

    def over(v):  # mean over a group
        return flat(v.reshape(t.shape).mean((1, 3), keepdim=True))

    n = flat((t - mean) * rstd)
    en = flat(30 * U * top * rstd) + 40 * U * n.abs()
    w = torch.ones(C, dtype=torch.float64) if x["w"] is None else x["w"].double()
    b = torch.zeros(C, dtype=torch.float64) if x["b"] is None else x["b"].double()
    z = n * w + b
    ez = w.abs() * en + 2 * U * ((n * w).abs() + b.abs())
    gate = None if x["z"] is None else x["z"].double()
    at = z if gate is None else gate
    eat = ez if gate is None else torch.zeros_like(z)
    if act == "silu":
        sig = torch.sigmoid(at)
        value, slope = at * sig, sig * (1 + at * (1 - sig))
        evalue = 1.1 * eat + value.abs() * (1.5 * at.abs() + 10) * U
        eslope = 0.5 * eat + (slope.abs() + sig * (1 + at.abs())) * (1.5 * at.abs() + 10) * U
    else:
        value, slope = at, torch.ones_like(at)
        evalue, eslope = eat, torch.zeros_like(at)
    dy = x["dy"].double()
    out = {}
    if gate is None:
        out["y"] = (value, evalue + 4 * U * value.abs())
        dz, edz = dy * slope, dy.abs() * eslope
    else:
        out["y"] = (z * value, ez * value.abs() + z.abs() * evalue + 4 * U * (z * value).abs())
        dz, edz = dy * value, dy.abs() * evalue
        out["dgate"] = (dy * z * slope, dy.abs() * (ez * slope.abs() + z.abs() * eslope) + 8 * U * (dy * z * slope).abs())
    edz = edz + 4 * U * dz.abs()
    g, eg = dz * w, edz * w.abs() + 2 * U * (dz * w).abs()
    m1, m2 = over(g), over(g * n)
    em1 = over(eg) + 30 * U * over(g.abs())
    em2 = over(eg * n.abs() + g.abs() * en) + 30 * U * over((g * n).abs())
    r = flat(rstd)
    out["dx"] = (r * (g - m1 - n * m2), r * (eg + em1 + n.abs() * em2 + m2.abs() * en)
                 + 40 * U * r * (g.abs() + m1.abs() + (n * m2).abs()))
    rows = x["x"].numel() // C

    def cols(v):
        return v.reshape(-1, C).sum(0)

    out["dw"] = (cols(dz * n), cols(edz * n.abs() + dz.abs() * en) + (rows + 70) * U * cols((dz * n).abs()))
    out["db"] = (cols(dz), cols(edz) + (rows + 70) * U * cols(dz.abs()))
    out["mean"] = (mean.flatten(1), (30 * U * top).flatten(1))
    out["rstd"] = (rstd.flatten(1), 60 * U * (rstd * (1 + top * rstd)).flatten(1))
    return out


def near(name, got, want):
    ref, slack = want
    slack = slack + 1e-30
    got = got.detach().cpu()
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    over = excess(got, ref, slack) - slack
    assert float(over.max()) <= 0, f"{name}: beyond the tolerance by {float(over.max())}"


def dev(t):
    return None if t is None else t.cuda()


def check(x, act, y=None, backward=True, eps=1e-5):
    want = formulas(x, act, eps)
    y = y or {k: (dev(v) if k != "G" else v) for k, v in x.items()}
    stats = torch.full((x["x"].shape[0], x["G"], 2), float("nan"), device="cuda")
    out = hla2.hla2_groupnorm(y["x"], x["G"], y["w"], y["b"], gate=y["z"], activation=act, stats=stats, eps=eps)
    near("y", out, want["y"])
    near("mean", stats[..., 0], want["mean"])
    near("rstd", stats[..., 1], want["rstd"])
    assert torch.equal(out, hla2.hla2_groupnorm(y["x"], x["G"], y["w"], y["b"], gate=y["z"], activation=act, eps=eps))
    if not backward:
        return
    dx, dw, db, dgate = hla2.hla2_groupnorm_backward(y["x"], y["dy"], stats, y["w"], y["b"], gate=y["z"], activation=act)
    for name, got in (("dx", dx), ("dw", dw), ("db", db), ("dgate", dgate)):
        if name in want:
            near(name, got, want[name])
        else:
            assert got is None


# ------------------------------------------------------------------- CPU ----
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("gate", [False, True])
def test_gradient_formulas_are_the_differences(gate, act):
    x = make(2, 3, 8, 2, torch.float64, gate, torch.float64, seed=3)
    want = formulas(x, act)
    gen = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("w", "dw"), ("b", "db"), ("z", "dgate")):
        if x[name] is None:
            continue
        step = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        hi, lo = (float((formulas({**x, name: x[name] + s * step}, act)["y"][0] * x["dy"]).sum()) for s in (1e-5, -1e-5))
        assert abs((hi - lo) / 2e-5 - float((want[grad][0] * step).sum())) < 1e-7


def test_entries_refuse():
    import ctypes
    L, a = hla2.lib(), ctypes.c_void_p
    r = [a(4096 * i) for i in range(1, 12)]

    def fwd(X=r[0], W=r[1], B=r[2], gate=None, Y=r[3], st=None, N=4, P=1, C=16, G=2, eps=1e-5, act=1, dt=0, wdt=0, ws=None, n=0):
        return L.hla2_groupnorm(X, W, B, gate, Y, st, N, P, C, G, None, eps, act, dt, wdt, ws, n, None)

    def bwd(X=r[0], dY=r[1], st=r[2], W=r[3], B=r[4], gate=None, dX=r[5], dg=None, dwb=r[6], N=4, P=1, C=16, G=2, act=1,
            dt=0, wdt=0, ws=r[7], n=1 << 20):
        return L.hla2_groupnorm_backward(X, dY, st, W, B, gate, dX, dg, dwb, N, P, C, G, None, act, dt, wdt, ws, n, None)

    inv, uns, wsp = hla2.HLA2_ERR_INVALID, hla2.HLA2_ERR_UNSUPPORTED, hla2.HLA2_ERR_WORKSPACE
    for kw in (dict(X=None), dict(Y=None), dict(N=0), dict(P=0), dict(C=0), dict(G=0), dict(G=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(X=a(4098)), dict(st=a(4100)), dict(W=a(4097))):
        assert fwd(**kw) == inv, kw
    for kw in (dict(C=16386), dict(dt=5), dict(wdt=5), dict(act=2), dict(N=1 << 31), dict(N=1 << 20, P=1 << 12)):
        assert fwd(**kw) == uns, kw
    need = hla2.hla2_groupnorm_workspace(2, 4096, 64, 4)
    assert need > 0 and need % 256 == 0
    big = dict(N=2, P=4096, C=64, G=4)
    assert fwd(**big) == wsp and fwd(**big, ws=r[8], n=need - 1) == wsp and fwd(**big, ws=a(4100), n=need) == inv
    for kw in (dict(X=None), dict(dY=None), dict(st=None), dict(dX=None), dict(gate=r[8]), dict(dg=r[8]),
               dict(gate=r[8], dg=r[5]), dict(G=5), dict(st=a(4100)), dict(dwb=a(4098)), dict(ws=a(4100))):
        assert bwd(**kw) == inv, kw
    assert bwd(act=7) == uns and bwd(C=20000) == uns and bwd(n=0) == wsp and bwd(ws=None) == wsp
    assert hla2.hla2_groupnorm_workspace(4, 1, 16, 3) == 0 and hla2.hla2_groupnorm_workspace(4, 1, 16, 2) == 0


def test_binding_refuses():
    f, b = hla2.hla2_groupnorm, hla2.hla2_groupnorm_backward
    x, w, st = torch.zeros(4, 16), torch.ones(16), torch.zeros(4, 2, 2)
    bad = [
        lambda: f(x, 3, w, w), lambda: f(x, 0, w, w), lambda: f(x[0], 2, w, w), lambda: f(x.half(), 2, w, w),
        lambda: f(x, 2, w[:8], w), lambda: f(x, 2, w, w.bfloat16()), lambda: f(x, 2, w, w, gate=x[:2]),
        lambda: f(x, 2, w, w, gate=x.bfloat16()), lambda: f(x, 2, w, w, activation="relu"),
        lambda: f(x, 2, w, w, Y=x[:2]), lambda: f(x, 2, w, w, Y=x.bfloat16()), lambda: f(x, 2, w, w, stats=st[:1]),
        lambda: f(x.t(), 2), lambda: f(x, 2, w, w), lambda: b(x, x, st[0], w, w), lambda: b(x, x[:2], st, w, w),
        lambda: b(x, x, st, w, w, dgate=x), lambda: b(x, x, st, w, w), lambda: b(x, x.bfloat16(), st, w, w),
        lambda: f(x[:, :1].expand(4, 16), 2, w, w, Y=x),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


@pytest.mark.parametrize("L", [2 ** 30, 2 ** 31 - 5 * 10 ** 6, 2 ** 31 - 10 ** 6, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1])
def test_workspace_up_to_the_largest_length(L):
    """A line of two sums for each run of one sample, as many runs as fill the SMs three times (of up to 200)."""
    for backward in (False, True):
        need = hla2.hla2_groupnorm_workspace(1, L, 1, 1, backward)
        assert 100 * 8 < need <= 601 * 8 + 256


@pytest.mark.parametrize("N,L,C,G", [(16384, 1, 8192, 1), (65536, 1, 16384, 1), (1 << 20, 1, 16384, 4), (1 << 20, 8, 512, 1),
                                     (1000, 2000, 240, 8)])
def test_workspace_of_many_samples(N, L, C, G):
    """The partial sums of large units do not grow with the batch beyond 256 MB (and two means for each group)."""
    for backward in (False, True):
        assert 0 < hla2.hla2_groupnorm_workspace(N, L, C, G, backward) <= (256 << 20) * (1 + 2 * G / (2 * C)) + 256


# ------------------------------------------------------------------- GPU ----
SHAPES = [  # N, L (0: two dimensions), C, G
    (1, 0, 1, 1), (3, 0, 8, 1), (2, 0, 30, 3), (5, 0, 240, 8), (7, 0, 2048, 16), (1000, 0, 64, 4), (4, 0, 2048, 1),
    (3, 0, 4096, 1), (2, 0, 6000, 3), (2, 0, 4500, 1), (2, 0, 16384, 2), (2, 5, 24, 3), (3, 100, 16, 2),
    (2, 4096, 64, 4), (5, 777, 240, 8), (2, 20, 2304, 2), (2, 9, 2060, 4), (300, 2, 8, 8), (2, 3000, 1, 1),
    (3, 513, 36, 4), (1, 1, 16, 2), (40, 64, 128, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act,gate", [("none", False), ("silu", False), ("none", True), ("silu", True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_and_gradient(shape, act, gate, dtype):
    check(make(*shape, dtype, gate, F32), act)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(6, 0, 256, 2), (4, 300, 64, 2)])
@pytest.mark.parametrize("wdtype", [None, BF])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_weights(shape, wdtype, dtype):
    check(make(*shape, dtype, True, wdtype), "silu")
    x = make(*shape, dtype, False, BF)
    x["b"] = None
    check(x, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(5, 0, 512, 4), (2, 2000, 32, 2)])
def test_mean_far_from_zero(shape):
    """The variance is that about the mean: a mean of a thousand deviations costs its own digits only."""
    check(make(*shape, F32, False, F32, shift=1000.0), "none")
    x = make(*shape, F32, False, F32)
    x["x"][..., 0] = 1e4  # the first of a group far out
    check(x, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4, 0, 64, 4), (2, 1000, 32, 4)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_equal_values(shape, dtype):
    """No variance at all: z is the bias, and no gradient comes back but rounding."""
    x = make(*shape, dtype, False, F32)
    x["x"][:] = 3.0
    y = hla2.hla2_groupnorm(x["x"].cuda(), 4, x["w"].cuda(), x["b"].cuda())
    assert torch.equal(y, x["b"].cuda().expand(x["x"].shape).to(dtype))
    check(x, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("L", [1, 700])
def test_strides(L, dtype, shift):
    """Slices of wider rows, at any offset."""
    N, C, G = 6, 64, 4
    gen = torch.Generator().manual_seed(1)
    wide = {k: torch.randn(N, L, 3 * C, generator=gen).to(dtype) for k in ("x", "dy", "z")}
    cuda = {k: v.cuda() for k, v in wide.items()}
    cut = slice(C + shift, 2 * C + shift)
    x = {**{k: v[:, :, cut] for k, v in wide.items()}, "w": torch.randn(C, generator=gen), "b": torch.randn(C, generator=gen), "G": G}
    y = {**{k: v[:, :, cut] for k, v in cuda.items()}, "w": x["w"].cuda(), "b": x["b"].cuda(), "G": G}
    if L == 1:
        x, y = ({k: (v[:, 0] if k in ("x", "dy", "z") else v) for k, v in t.items()} for t in (x, y))
    check(x, "silu", y)
    stats = torch.empty(N, G, 2, device="cuda")
    room = torch.full((N, L, 3 * C), 9.0, device="cuda", dtype=dtype)
    into = room[:, :, cut] if L > 1 else room[:, 0, cut]
    want = hla2.hla2_groupnorm(y["x"], G, y["w"], y["b"], gate=y["z"], activation="silu", stats=stats)
    hla2.hla2_groupnorm(y["x"], G, y["w"], y["b"], gate=y["z"], activation="silu", Y=into)
    assert torch.equal(into, want)
    assert bool((room[:, :, :C + shift] == 9).all()) and bool((room[:, :, 2 * C + shift:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(9, 0, 256, 2), (3, 1000, 48, 3)])
def test_in_place(shape):
    x = {k: (dev(v) if k != "G" else v) for k, v in make(*shape, BF, True, F32).items()}
    stats = torch.empty(shape[0], x["G"], 2, device="cuda")
    kw = dict(gate=x["z"], activation="silu")
    y = hla2.hla2_groupnorm(x["x"], x["G"], x["w"], x["b"], stats=stats, **kw)
    dx, dw, db, dgate = hla2.hla2_groupnorm_backward(x["x"], x["dy"], stats, x["w"], x["b"], **kw)
    for name in ("x", "z"):
        c = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
        hla2.hla2_groupnorm(c["x"], c["G"], c["w"], c["b"], gate=c["z"], activation="silu", Y=c[name])
        assert torch.equal(c[name], y)
    for name in ("x", "dy"):
        c = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
        got = hla2.hla2_groupnorm_backward(c["x"], c["dy"], stats, c["w"], c["b"], gate=c["z"], activation="silu",
                                           dX=c[name], dgate=c["z"])
        assert torch.equal(c[name], dx) and torch.equal(c["z"], dgate)
        assert torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(500, 0, 256, 4), (3, 1500, 96, 3)])
def test_stream_and_graph(shape):
    xs = [{k: (dev(v) if k != "G" else v) for k, v in make(*shape, BF, True, F32, seed=s).items()} for s in range(3)]

    def run(x, stream=None, ws=None):
        stats = torch.empty(shape[0], x["G"], 2, device="cuda")
        y = hla2.hla2_groupnorm(x["x"], x["G"], x["w"], x["b"], gate=x["z"], activation="silu", stats=stats,
                                stream=stream)
        return y, stats, *hla2.hla2_groupnorm_backward(x["x"], x["dy"], stats, x["w"], x["b"], gate=x["z"],
                                                       activation="silu", stream=stream)

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(xs[0], s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    bufs = [{k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in xs[0].items()} for _ in range(2)]
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(b))
        graphs.append(g)
    for i in (1, 2):
        for b, j in zip(bufs, (i, 3 - i)):
            for k in ("x", "z", "dy", "w", "b"):
                b[k].copy_(xs[j][k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, j in zip(outs, (i, 3 - i)):
            assert all(torch.equal(a, b) for a, b in zip(out, want[j]))


@pytest.mark.gpu
def test_behind_linear_attention():
    """A layer's gated branch: linear attention, the norm of each head's output, its gate, and all gradients, against
    the plain layer's in 64 bits through autograd.  Tolerance: the chain rounds to bf16 four times (o, its norm, the
    gradient of o, the results), each up to 2^-8 of the largest value that it feeds; products add their own three."""
    B, H, T, d = 2, 4, 200, 64
    gen = torch.Generator().manual_seed(0)
    q, k, v, gate, dy = (torch.randn(B, T, H * d, generator=gen).to(BF) for _ in range(5))
    q, k = q * d ** -0.5, k * d ** -0.5
    gamma = torch.exp(-(2.0 ** (-2.0 * torch.arange(1, H + 1))))
    w, b = 1 + 0.1 * torch.randn(H * d, generator=gen), 0.1 * torch.randn(H * d, generator=gen)
    leaves = [t.double().requires_grad_() for t in (q, k, v, gate, w, b)]
    Q, K, V = (t.unflatten(2, (H, d)).transpose(1, 2) for t in leaves[:3])
    i = torch.arange(T)
    decay = torch.where(i[:, None] >= i, gamma.double()[:, None, None] ** (i[:, None] - i).clamp(min=0), 0.0)
    o = ((Q @ K.mT) * decay) @ V
    o = o.transpose(1, 2).reshape(B * T, H, d)
    n = (o - o.mean(-1, keepdim=True)) / (o.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    y = (n.reshape(B, T, H * d) * leaves[4] + leaves[5]) * torch.nn.functional.silu(leaves[3])
    grads = torch.autograd.grad(y, leaves, dy.double())

    def heads(t):
        return t.cuda().unflatten(2, (H, d)).transpose(1, 2)

    og = hla2.hla2_linear_forward(heads(q), heads(k), heads(v), gamma.cuda())
    rows = og.transpose(1, 2).reshape(B * T, H * d)
    assert rows.data_ptr() == og.data_ptr()  # the output lies as the norm takes it
    stats = torch.empty(B * T, H, 2, device="cuda")
    gr, dyr = gate.cuda().view(B * T, -1), dy.cuda().view(B * T, -1)
    yg = hla2.hla2_groupnorm(rows, H, w.cuda(), b.cuda(), gate=gr, activation="silu", stats=stats)
    do, dw, db, dgate = hla2.hla2_groupnorm_backward(rows, dyr, stats, w.cuda(), b.cuda(), gate=gr, activation="silu")
    do = do.view(B, T, H, d).transpose(1, 2)
    dq, dk, dv = hla2.hla2_linear_backward(heads(q), heads(k), heads(v), gamma.cuda(), do)
    flat = [t.transpose(1, 2).reshape(B, T, H * d) for t in (dq, dk, dv)]
    for got, ref in zip([yg.view(B, T, -1), *flat, dgate.view(B, T, -1), dw, db], [y, *grads]):
        err, ref = (got.double().cpu() - ref).detach(), ref.detach()
        # early rows have few terms and a norm of tiny deviations: errors against the 2-norm of everything
        assert float(err.norm() / ref.norm()) < 7 * 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(1000, 0, 64, 4), (5, 777, 240, 8), (2, 4096, 64, 4), (2, 0, 4500, 1)])
def test_calls_in_a_row(shape, dtype, captured):
    """Each call's inputs are what the call before has just written, all in one workspace: the bits of the same calls
    with the device idle between them."""
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in make(*shape, dtype, True, F32).items()}
    N, L, C, G = shape
    need = max(hla2.hla2_groupnorm_workspace(N, max(L, 1), C, G, back) for back in (False, True))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    pause = lambda: None

    def run():
        a, dy, z, seen = x["x"], x["dy"], x["z"], []
        for _ in range(3):
            stats = torch.empty(N, G, 2, device="cuda")
            y = hla2.hla2_groupnorm(a, G, x["w"], x["b"], gate=z, activation="silu", stats=stats, workspace=ws)
            pause()
            gr = hla2.hla2_groupnorm_backward(a, dy, stats, x["w"], x["b"], gate=z, activation="silu", workspace=ws)
            pause()
            seen += [y, stats, *gr]
            a, dy = y, gr[0]
        return seen

    pause = torch.cuda.synchronize
    want = run()
    pause = lambda: None
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        for _ in range(3):
            g.replay()
    else:
        got = run()
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(512, 4096, 8, 8), (460, 4100, 12, 3), (3, 70001, 16, 2)])
def test_variance_behind_an_untypical_first_position(shape, dtype):
    """Padding in front of values far from zero: the variance of a long run does not depend on its first value."""
    x = make(*shape, dtype, False, F32, shift=1000.0)
    x["x"][:, 0] = 0.0
    check(x, "none", backward=False)


@pytest.mark.gpu
def test_gradient_of_equal_terms_over_long_runs():
    """dy and gate constant: t is its own mean, and n has none, so that dx is nothing but rounding however many
    positions a thread adds.  What dx may be is formulas()' tolerance at w = 1: the terms of t's mean (30 u beside the
    slope's own roundings, which are the same in all terms), n's mean times t's, and the products."""
    N, L, C, G = 456, 2048, 2048, 8
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.empty(N, L, C, device="cuda").normal_(generator=gen)
    dy, z = (torch.full((C,), v, device="cuda").expand(N, L, C) for v in (0.1, 0.3))
    stats = torch.empty(N, G, 2, device="cuda")
    hla2.hla2_groupnorm(x, G, gate=z, activation="silu", stats=stats, Y=torch.empty_like(x))
    dx, dw, db, dgate = hla2.hla2_groupnorm_backward(x, dy, stats, gate=z, activation="silu")
    t = float(torch.tensor(0.1).double() * torch.nn.functional.silu(torch.tensor(0.3).double()))
    for i in (0, 200, N - 1):
        mean, r = (s.repeat_interleave(C // G).double() for s in stats[i].unbind(-1))
        n = ((x[i].double() - mean) * r).abs()
        # n's own mean is 30 u of the largest |x|, which moves mean(t n) as much
        top = float(x[i].abs().max())
        slack = t * r * U * (30 + 80 + n * (30 * float(n.mean()) + 30 * top * float(r.max()) + 40))
        assert bool((dx[i].double().abs() <= slack).all()), float((dx[i].double().abs() / slack).max())
    # equal terms: a sum's error is that of its few levels
    assert float((db.double() / (t * N * L) - 1).abs().max()) <= 60 * U


@pytest.mark.gpu
def test_largest_length():
    """2^31 - 1 positions: the ends of the last runs."""
    L = 2 ** 31 - 1
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.empty(1, L, 1, device="cuda", dtype=BF).normal_(generator=gen)
    pieces = x.view(-1).split(2 ** 28)
    mean = sum(float(c.double().sum()) for c in pieces) / L
    rstd = (sum(float((c.double() - mean).square().sum()) for c in pieces) / L + 1e-5) ** -0.5
    stats = torch.empty(1, 1, 2, device="cuda")
    y = hla2.hla2_groupnorm(x, 1, stats=stats)
    top = float(x.abs().max())
    assert abs(float(stats[0, 0, 0]) - mean) <= 30 * U * top
    assert abs(float(stats[0, 0, 1]) - rstd) <= 60 * U * rstd * (1 + top * rstd)
    for c, got in zip(pieces, y.view(-1).split(2 ** 28)):
        n = (c.double() - mean) * rstd
        slack = 30 * U * top * rstd + 44 * U * n.abs()
        unit = torch.ldexp(torch.ones_like(n), torch.frexp((n.abs() + slack).clamp(min=2.0 ** -126)).exponent - 9)
        assert bool(((got.double() - n).abs() <= slack + unit).all())
        del n, slack, unit
    dx, dw, db, _ = hla2.hla2_groupnorm_backward(x, y, stats)
    # dy is y: the gradient is the rounding of y to bf16 alone, all along
    for c, g in zip(pieces, dx.view(-1).split(2 ** 28)):
        assert float(g.abs().max()) <= rstd * (2.0 ** -8 * (top - mean) * rstd * 2.5 + 1e-4)
    # dw of the statistics that it was given: two roundings of n, pieces of sixteen terms, a few levels on top
    mean, rstd = (float(v) for v in stats[0, 0])
    want = sum(float(((c.double() - mean) * rstd * g.double()).sum()) for c, g in zip(pieces, y.view(-1).split(2 ** 28)))
    assert abs(float(dw[0]) / want - 1) <= 40 * U


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(400, 0, 64, 4), (50, 0, 2048, 16), (30, 0, 90, 3), (20, 2, 2048, 2), (8, 1000, 32, 4), (3, 300, 45, 3)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_equal_values_of_all_bits(shape, dtype):
    """Equal values of 24 bits, another in each sample: n is zero but for what a first mean is off by (17 roundings: eight
    values to a thread, eight levels, the quotient), which the second pass takes away to 17 roundings of itself."""
    x = make(*shape, dtype, False, F32)
    gen = torch.Generator().manual_seed(7)
    v = (1000 + 1000 * torch.rand(shape[0], generator=gen)).to(dtype)
    x["x"][:] = v.view(-1, *[1] * (x["x"].dim() - 1))
    G = shape[3]
    stats = torch.empty(shape[0], G, 2, device="cuda")
    y = hla2.hla2_groupnorm(x["x"].cuda(), G, x["w"].cuda(), x["b"].cuda(), stats=stats).cpu().double()
    assert torch.equal(stats[..., 0].cpu(), v.float()[:, None].expand(-1, G))
    slack = (17 * U) ** 2 * 2000 * 1e-5 ** -0.5 * x["w"].double().abs() + U * x["b"].double().abs()
    assert bool((excess(y.to(dtype) if dtype == BF else y, x["b"].double().expand(y.shape), slack) <= slack).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gate", [(F32, False), (BF, True)])
@pytest.mark.parametrize("shape", [(8400, 0, 4096, 1), (8300, 0, 4102, 1), (2100, 0, 16384, 4)])
def test_more_samples_than_are_held_at_a_time(shape, dtype, gate):
    check(make(*shape, dtype, gate, F32), "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shift", [(BF, 0), (BF, 1), (F32, 0)])
@pytest.mark.parametrize("N,L,C,far", [(2, 1, 256, "sample"), (2, 300, 64, "sample"), (1, 3, 64, "position"), (1, 3, 4096, "position")])
def test_offsets_beyond_32_bits(N, L, C, far, dtype, shift):
    """Samples, or positions, more than 2^32 elements apart, in both forms."""
    G, step = 2, 2 ** 32 + 64
    x = make(N, L, C, G, dtype, True, F32)
    size = L * C if far == "sample" else C
    room = torch.empty(step * (N - 1 if far == "sample" else L - 1) + 5 * size + 64, device="cuda", dtype=dtype)

    def place(i):
        return room.as_strided((N, L, C), (step, C, 1) if far == "sample" else (64, step, 1), i * size + shift)

    y = {k: (dev(v) if k != "G" else v) for k, v in x.items()}
    for i, name in enumerate(("x", "dy", "z")):
        y[name] = place(i).copy_(y[name])
    check(x, "silu", y)
    want = formulas(x, "silu")
    stats = torch.empty(N, G, 2, device="cuda")
    kw = dict(gate=y["z"], activation="silu")
    near("y", hla2.hla2_groupnorm(y["x"], G, y["w"], y["b"], stats=stats, Y=place(3), **kw), want["y"])
    dx, _, _, dgate = hla2.hla2_groupnorm_backward(y["x"], y["dy"], stats, y["w"], y["b"], dX=place(3), dgate=place(4), **kw)
    near("dx", dx, want["dx"])
    near("dgate", dgate, want["dgate"])
    del room, y, dx, dgate
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("C,G,L", [(2048, 1, 0), (700, 2, 0), (96, 12, 20)])
def test_weight_gradients_of_equal_terms_over_many_rows(C, G, L):
    """dz constant: db is its multiple, off by the error of a sum of few levels, however many rows a thread adds."""
    N = 300000 * 2048 // (C * max(L, 1))
    gen = torch.Generator("cuda").manual_seed(0)
    shape = (N, L, C) if L else (N, C)
    x = torch.empty(shape, device="cuda").normal_(generator=gen)
    dy, z = (torch.full((C,), v, device="cuda").expand(shape) for v in (0.1, 0.3))
    stats = torch.empty(N, G, 2, device="cuda")
    hla2.hla2_groupnorm(x, G, gate=z, activation="silu", stats=stats, Y=torch.empty_like(x))
    _, dw, db, _ = hla2.hla2_groupnorm_backward(x, dy, stats, gate=z, activation="silu")
    t = float(torch.tensor(0.1).double() * torch.nn.functional.silu(torch.tensor(0.3).double()))
    assert float((db.double() / (t * N * max(L, 1)) - 1).abs().max()) <= 60 * U
    assert bool(torch.isfinite(dw).all())


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(5, 0, 512, 4), (2, 2000, 32, 2), (500, 2100, 2, 2)])
def test_mean_whose_square_overflows(shape):
    """Deviations of 1e16 about 3e19: no square of a value itself is formed."""
    x = make(*shape, F32, False, F32, shift=0.0)
    x["x"] = x["x"] * 1e16 + 3e19
    check(x, "none")
