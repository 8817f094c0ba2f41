"""First-order linear attention with a decay for each head (hla2_linear_forward,
hla2_linear_backward, hla2_linear_step) against the recurrence in 64 bits.

Tolerances, fixed before the first run.  u = 2^-24.  M1 is the same sum over the
magnitudes of all inputs, so that a result formed with n roundings of u on the way is
off by at most n u M1:
- scores are sums of d products, a block's outputs and states sums over its (at most
  128) tokens, and each block of the walk multiplies and adds the state once: n = d +
  128 + 4 blocks + 16 in fp32, and a whole unit (2 u) instead of half of one on the
  tensor cores, whose sums may be cut off, with three terms for each product of the state;
- on the tensor cores a block's scores and the state entering it are rounded to bf16
  (half a unit, 2^-8): 2^-8 M2 on top, M2 the sum over |score| |c| and |a| |state|;
- bf16 results: half a unit in the last place of each value on top.
"""
import pytest
import torch

from _rounding import excess
from higher_order_linear_gb300 import hla2

BLOCK = 128
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- 64 bits ----
def by_token(gamma, a, b, c, state, lens, reverse=False):
    """o and the last state by the recurrence itself, a token at a time."""
    B, H, T, _ = a.shape
    a, b, c = a.double(), b.double(), c.double()
    o = torch.zeros(B, H, T, c.shape[3], dtype=torch.float64)
    S = state.double().clone()
    g = gamma.double()[:, None, None]
    for i in range(B):
        n = lens[i]
        s = S[i]
        for t in (range(n - 1, -1, -1) if reverse else range(n)):
            if reverse:  # s: the gradient of the state behind token t, from the later ones
                s = s + b[i, :, t, :, None] * c[i, :, t, None]
                o[i, :, t] = (a[i, :, t, :, None] * s).sum(1)
                s = g * s
            else:
                s = g * s + b[i, :, t, :, None] * c[i, :, t, None]
                o[i, :, t] = (a[i, :, t, :, None] * s).sum(1)
        S[i] = s
    return o, S


def by_block(gamma, a, b, c, state, lens, reverse=False):
    """The same in blocks: (o, last state, M2 of o, M1 of o, M1 of the state)."""
    B, H, T, _ = a.shape
    a, b, c = a.double(), b.double(), c.double()
    zeros = torch.zeros(B, H, T, c.shape[3], dtype=torch.float64)
    o, m2, m1 = zeros.clone(), zeros.clone(), zeros.clone()
    S, A = state.double().clone(), state.double().abs()
    g = gamma.double()
    starts = list(range(0, T, BLOCK))
    for i in range(B):
        for t0 in (reversed(starts) if reverse else starts):
            n = min(BLOCK, lens[i] - t0)
            if n <= 0:
                continue
            x, y, z = (t[i, :, t0:t0 + n] for t in (a, b, c))
            r = torch.arange(n, dtype=torch.float64)
            far = r[None] - r[:, None] if reverse else r[:, None] - r[None]
            w = torch.where(far >= 0, g[:, None, None] ** far.clamp(min=0), 0.0)
            into = (n - 1 - r) if reverse else r + 1
            out = (r + 1) if reverse else n - 1 - r
            gi, go, gn = g[:, None, None] ** into[:, None], g[:, None, None] ** out[:, None], (g ** n)[:, None, None]
            p = (x @ y.mT) * w
            pa = (x.abs() @ y.abs().mT) * w
            o[i, :, t0:t0 + n] = p @ z + gi * (x @ S[i])
            m2[i, :, t0:t0 + n] = p.abs() @ z.abs() + gi * (x.abs() @ S[i].abs())
            m1[i, :, t0:t0 + n] = pa @ z.abs() + gi * (x.abs() @ A[i])
            S[i] = gn * S[i] + (y * go).mT @ z
            A[i] = gn * A[i] + (y.abs() * go).mT @ z.abs()
    return o, S, m2, m1, A


def on_tensor_cores(*tensors):
    return all(t.dtype == BF and t.shape[-1] % 8 == 0 and t.data_ptr() % 16 == 0 and
               all(s % 8 == 0 for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1) for t in tensors)


def near(got, ref, m1, m2, d, T, tc, what=""):
    n = (3 if tc else 1) * (d + BLOCK) + 4 * -(-T // (BLOCK if tc else 64)) + 16
    slack = n * U * (2 if tc else 1) * m1 + 1e-30
    if tc and m2 is not None:
        slack = slack + (2.0 ** -8) * m2 * 1.01
    got = got.detach().cpu()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    over = excess(got, ref, slack) - slack
    assert float(over.max()) <= 0, f"{what}: beyond the tolerance by {float(over.max())}, allowed up to {float(slack.max())}"


# ----------------------------------------------------------------- inputs ----
def heads(gen, B, H, T, d, dtype, layout, scale=1.0):
    if layout == "bthd":
        return (torch.randn(B, T, H, d, generator=gen) * scale).to(dtype).transpose(1, 2)
    return (torch.randn(B, H, T, d, generator=gen) * scale).to(dtype)


def decays(kind, H):
    if kind == "edge":  # none at all, nothing but the token itself, fast, nearly none
        return torch.tensor([1.0, 0.0, 0.01, 1 - 2.0 ** -13, 0.5, 0.9])[torch.arange(H) % 6]
    return torch.exp(-(2.0 ** (-8 * torch.arange(1, H + 1) / H)))


def make(B, H, T, d, dv, dtype, layout="bhtd", state=True, seed=0, kind="slopes"):
    gen = torch.Generator().manual_seed(seed)
    x = {"q": heads(gen, B, H, T, d, dtype, layout, d ** -0.5), "k": heads(gen, B, H, T, d, dtype, layout, d ** -0.5),
         "v": heads(gen, B, H, T, dv, dtype, layout), "do": heads(gen, B, H, T, dv, dtype, layout),
         "gamma": decays(kind, H)}
    x["h0"] = torch.randn(B, H, d, dv, generator=gen) if state else None
    x["dlast"] = torch.randn(B, H, d, dv, generator=gen) if state else None
    return x


def dev(x):
    return {k: None if t is None else (t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                                      if t.dim() == 4 and not t.is_contiguous() else t.cuda()) for k, t in x.items()}


def check_forward(x, lens=None, y=None):
    B, H, T, d = x["q"].shape
    dv = x["v"].shape[-1]
    y = y or dev(x)
    ls = [T] * B if lens is None else lens
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    last = torch.full((B, H, d, dv), float("nan"), device="cuda")
    o = torch.full((B, H, T, dv), 7.0, dtype=x["q"].dtype, device="cuda") if lens is not None else None
    got = hla2.hla2_linear_forward(y["q"], y["k"], y["v"], y["gamma"], O=o, lengths=lengths, state_in=y["h0"],
                                   state_out=last)
    zero = torch.zeros(B, H, d, dv)
    ref, S, m2, m1, A = by_block(x["gamma"], x["q"], x["k"], x["v"], zero if x["h0"] is None else x["h0"], ls)
    tc = on_tensor_cores(y["q"], y["k"], y["v"], got)
    for i in range(B):
        n = ls[i]
        near(got[i, :, :n], ref[i, :, :n], m1[i, :, :n], m2[i, :, :n], d, T, tc, "o") if n else None
        if n < T:
            assert bool((got[i, :, n:] == 7).all()), "rows behind the end were written"
    near(last, S, A, None, d, T, tc, "last state")
    return got, last


def check_backward(x, lens=None, y=None):
    B, H, T, d = x["q"].shape
    dv = x["v"].shape[-1]
    y = y or dev(x)
    ls = [T] * B if lens is None else lens
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    d0 = torch.full((B, H, d, dv), float("nan"), device="cuda")
    dq, dk, dvv = hla2.hla2_linear_backward(y["q"], y["k"], y["v"], y["gamma"], y["do"], lengths=lengths,
                                            state_in=y["h0"], dstate_out=y["dlast"], dstate_in=d0)
    zero = torch.zeros(B, H, d, dv)
    h0 = zero if x["h0"] is None else x["h0"]
    dl = zero if x["dlast"] is None else x["dlast"]
    g = x["gamma"]
    tc = on_tensor_cores(y["q"], y["k"], y["v"], y["do"], dq, dk, dvv)
    for name, got, args, width in (("dq", dq, (x["do"], x["v"], x["k"], h0.mT, ls), dv),
                                   ("dk", dk, (x["v"], x["do"], x["q"], dl.mT, ls, True), dv),
                                   ("dv", dvv, (x["k"], x["q"], x["do"], dl, ls, True), d)):
        ref, S, m2, m1, A = by_block(g, *args)
        near(got, ref, m1, m2, width, T, tc, name)
        if name == "dv":
            near(d0, S, A, None, d, T, tc, "dstate_in")
        for i in range(B):
            assert not bool(got[i, :, ls[i]:].any()), "gradients behind the end"


# ------------------------------------------------------------ CPU: oracle ----
@pytest.mark.parametrize("reverse", [False, True])
def test_blocks_are_the_recurrence(reverse):
    x = make(2, 3, 300, 5, 7, torch.float64, kind="edge")
    lens = [300, 129]
    o, S = by_token(x["gamma"], x["q"], x["k"], x["v"], x["h0"], lens, reverse)
    o2, S2, m2, m1, A = by_block(x["gamma"], x["q"], x["k"], x["v"], x["h0"], lens, reverse)
    assert torch.allclose(o, o2, rtol=0, atol=1e-12) and torch.allclose(S, S2, rtol=0, atol=1e-12)
    assert bool((m2 >= o2.abs() - 1e-12).all()) and bool((m1 >= m2 - 1e-12).all())


def test_gradient_formulas_are_the_differences():
    """dQ, dK, dV and the state's gradient, as the tests form them, against central differences."""
    x = make(1, 2, 9, 3, 4, torch.float64, seed=3)
    lens = [9]

    def loss(q, k, v, h0):
        o, S = by_token(x["gamma"], q, k, v, h0, lens)
        return float((o * x["do"]).sum() + (S * x["dlast"]).sum())

    dq, _ = by_token(x["gamma"], x["do"], x["v"], x["k"], x["h0"].mT, lens)
    dk, _ = by_token(x["gamma"], x["v"], x["do"], x["q"], x["dlast"].mT, lens, True)
    dv, d0 = by_token(x["gamma"], x["k"], x["q"], x["do"], x["dlast"], lens, True)
    gen = torch.Generator().manual_seed(1)
    base = [x["q"], x["k"], x["v"], x["h0"].double()]
    for i, grad in enumerate((dq, dk, dv, d0)):
        step = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        hi, lo = ([t + (s * step if j == i else 0) for j, t in enumerate(base)] for s in (1e-3, -1e-3))
        assert abs((loss(*hi) - loss(*lo)) / 2e-3 - float((grad * step).sum())) < 1e-9


# --------------------------------------------------------- CPU: refusals ----
def test_entries_refuse():
    import ctypes
    L = hla2.lib()
    a = ctypes.c_void_p
    r = [a(4096 * i) for i in range(1, 16)]

    def fwd(Q=r[0], K=r[1], V=r[2], g=r[3], ln=None, si=None, O=r[4], so=None, B=1, H=2, T=4, d=8, dv=8, dt=0, ws=None,
            n=0):
        return L.hla2_linear_forward(Q, K, V, g, ln, si, O, so, B, H, T, d, dv, None, dt, ws, n, None)

    for kw in (dict(Q=None), dict(K=None), dict(V=None), dict(g=None), dict(O=None), dict(T=0), dict(B=-1), dict(d=0),
               dict(Q=a(4098)), dict(O=a(16385)), dict(g=a(4097)), dict(ln=a(4098)),
               dict(O=r[0]), dict(O=r[2]), dict(si=a(65536), so=a(65536 + 64))):
        assert fwd(**kw) == hla2.HLA2_ERR_INVALID, kw
    for kw in (dict(d=129), dict(dv=129), dict(dt=7), dict(B=300, H=300)):
        assert fwd(**kw) == hla2.HLA2_ERR_UNSUPPORTED, kw
    need = hla2.hla2_linear_workspace(1, 2, 65536, 8, 8)
    assert need > 0 and need % 256 == 0
    assert fwd(T=65536) == hla2.HLA2_ERR_WORKSPACE
    assert fwd(T=65536, ws=r[9], n=need - 1) == hla2.HLA2_ERR_WORKSPACE
    assert fwd(T=65536, ws=a(4097), n=need) == hla2.HLA2_ERR_INVALID
    assert hla2.hla2_linear_workspace(1, 1, 64, 129, 8) == 0 and hla2.hla2_linear_workspace(1, 1, 0, 8, 8) == 0
    # up to the largest T: at most 1024 segments and one more slot, each a state
    top = hla2.hla2_linear_workspace(1, 1, 2 ** 31 - 1, 128, 128)
    assert 0 < top <= 1025 * 128 * 128 * 4 + 256

    def bwd(Q=r[0], K=r[1], V=r[2], g=r[3], ln=None, si=None, dO=r[4], dso=None, dQ=r[5], dK=r[6], dV=r[7], dsi=None,
            B=1, H=2, T=4, d=8, dv=8, dt=0):
        return L.hla2_linear_backward(Q, K, V, g, ln, si, dO, dso, dQ, dK, dV, dsi, B, H, T, d, dv, None, dt, None, 0,
                                      None)

    for kw in (dict(dO=None), dict(dQ=None), dict(dK=None), dict(dV=None), dict(dQ=r[0]), dict(dV=r[4]),
               dict(dK=r[5]), dict(dV=r[5]), dict(dso=a(65536), dsi=a(65540)), dict(si=a(65536), dsi=a(65540)),
               dict(T=0), dict(dQ=a(4098))):
        assert bwd(**kw) == hla2.HLA2_ERR_INVALID, kw
    for kw in (dict(d=200), dict(dt=2)):
        assert bwd(**kw) == hla2.HLA2_ERR_UNSUPPORTED, kw

    def step(s=r[0], q=r[1], k=r[2], v=r[3], g=r[4], o=r[5], so=None, n=4, H=2, d=8, dv=8, dt=0):
        return L.hla2_linear_step(s, q, k, v, g, o, so, n, H, d, dv, None, dt, None)

    for kw in (dict(s=None), dict(q=None), dict(g=None), dict(o=None), dict(n=3), dict(n=0), dict(H=0), dict(s=a(4098)),
               dict(so=a(4096 + 64)), dict(q=a(4097))):
        assert step(**kw) == hla2.HLA2_ERR_INVALID, kw
    for kw in (dict(d=129), dict(dv=200), dict(dt=9)):
        assert step(**kw) == hla2.HLA2_ERR_UNSUPPORTED, kw


def test_binding_refuses():
    f, b, s = hla2.hla2_linear_forward, hla2.hla2_linear_backward, hla2.hla2_linear_step
    q, v, g = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 4, 16), torch.zeros(3)
    bad = [
        lambda: f(q, q[:1], v, g), lambda: f(q, q, v[:, :, :3], g), lambda: f(q[0], q[0], v[0], g),
        lambda: f(q, q.bfloat16(), v, g), lambda: f(q.half(), q.half(), v.half(), g), lambda: f(q, q, v, g[:2]),
        lambda: f(q, q, v, g.double()), lambda: f(q, q, v, g, lengths=torch.zeros(2)),
        lambda: f(q, q, v, g, lengths=torch.zeros(3, dtype=torch.int32)),
        lambda: f(q, q, v, g, state_in=torch.zeros(2, 3, 16, 8)),
        lambda: f(q, q, v, g, state_out=torch.zeros(2, 3, 8, 16, dtype=BF)),
        lambda: f(q, q, v, g, O=torch.zeros(2, 3, 4, 16)),  # not on a GPU
        lambda: f(q.transpose(2, 3), q.transpose(2, 3), v, g),
        lambda: b(q, q, v, g, q), lambda: b(q, q, v, g, v, dQ=v), lambda: b(q, q, v, g, v.bfloat16()),
        lambda: b(q, q, v, g, v, dstate_in=torch.zeros(2, 3, 8, 8)),
        lambda: b(q, q, v, g, v),  # not on a GPU
        lambda: s(torch.zeros(6, 8, 16), q[0, 0], q[0, 0], v[0, 0], g), lambda: s(q[0], q[0, 0], q[0, 0], v[0, 0], g[:1]),
        lambda: s(torch.zeros(4, 8, 16), q[0, 0], q[0, 0], v[0, 0], g),  # 4 heads, 3 decays
        lambda: s(torch.zeros(4, 8, 16), q[0, 0], q[0, 0], v[0, 0], g[:2]),  # not on a GPU
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


def step_code(s, q, k, v, o, so=None, ld=None, n=4, d=8, dv=8, dt=0):
    import ctypes
    ld = None if ld is None else (ctypes.c_longlong * 4)(*ld)
    return hla2.lib().hla2_linear_step(*(None if t is None else ctypes.c_void_p(t) for t in (s, q, k, v, 1 << 16, o, so)), n, 1,
                                       d, dv, ld, dt, None)


def test_step_refuses_overlaps():
    """Few heads are cut into blocks that each read q and k: an output among them would be read half written."""
    s, q, k, v, o, so = (1 << 20) * 1, (1 << 20) * 2, (1 << 20) * 3, (1 << 20) * 4, (1 << 20) * 5, (1 << 20) * 6
    n, d = 4, 8
    state = n * d * d * 4
    for kw in (dict(o=q), dict(o=k), dict(o=q + 4), dict(o=k - 4), dict(o=v + 4), dict(o=q + n * d * 4 - 4),
               dict(o=s), dict(o=s + state - 4), dict(o=s - n * d * 4 + 4), dict(o=so), dict(so=q), dict(so=k - state + 4),
               dict(so=v), dict(s=v, o=o, so=None), dict(o=v, ld=[8, 8, 8, 16]), dict(o=q + 4 * 4, ld=[64, 64, 64, 64], q=q - 8),
               dict(o=q + 58 * 4, ld=[64, 8, 8, 57]), dict(o=q, ld=[0, 8, 8, 8])):
        args = dict(dict(s=s, q=q, k=k, v=v, o=o, so=so), **kw)
        assert step_code(**args) == hla2.HLA2_ERR_INVALID, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: what is not refused would be launched")
def test_step_refuses_overlaps_and_nothing_else():
    gen = torch.Generator().manual_seed(0)
    pick = lambda lo, hi: int(torch.randint(lo, hi, (), generator=gen))
    base = 1 << 20

    def touched(p, step, width, n):
        return {p + 4 * (i * step + c) for i in range(n) for c in range(width)}

    seen = [0, 0]
    for _ in range(3000):
        n, d, dv = pick(1, 6), pick(1, 7), pick(1, 7)
        lo, lq = pick(dv, 15), pick(0, 15)
        if pick(0, 2):
            lq = lo
        o = base + 4 * pick(-40, 40)
        meet = bool(touched(base, lq, d, n) & touched(o, lo, dv, n))
        code = step_code(1 << 24, base, 1 << 25, 1 << 26, o, ld=[lq, 8, 8, lo], n=n, d=d, dv=dv)
        assert code == (hla2.HLA2_ERR_INVALID if meet else hla2.HLA2_ERR_LAUNCH), (n, d, dv, lq, lo, o - base)
        seen[meet] += 1
    assert min(seen) > 300
    assert step_code(1 << 24, base, 1 << 25, 1 << 26, 1 << 26) == hla2.HLA2_ERR_LAUNCH  # o is v


# -------------------------------------------------------------- GPU tests ----
@pytest.mark.gpu
@pytest.mark.parametrize("n,d", [(1, 128), (3, 64), (1000, 32)])
def test_step_output_in_place_of_v(n, d):
    gen = torch.Generator().manual_seed(n)
    q, k, v = (torch.randn(n, d, generator=gen).cuda() for _ in range(3))
    S, g = torch.randn(n, d, d, generator=gen).cuda(), torch.tensor([0.9], device="cuda")
    want_state = torch.empty_like(S)
    want = hla2.hla2_linear_step(S, q, k, v, g, state_out=want_state)
    for o in (q, k, S[0, :n] if n <= d else q):
        with pytest.raises(hla2.HLA2Error):
            hla2.hla2_linear_step(S, q, k, v, g, o=o, state_out=torch.empty_like(S))
    assert hla2.hla2_linear_step(S, q, k, v, g, o=v) is v
    assert torch.equal(v, want) and torch.equal(S, want_state)
    # q, k, v and o as slices of one buffer
    room = torch.cat([q, k, want, torch.zeros_like(q)], 1)
    parts = [room[:, i * d:(i + 1) * d] for i in range(4)]
    S2 = S.clone()
    want = hla2.hla2_linear_step(S, q, k, want, g)
    hla2.hla2_linear_step(S2, *parts[:3], g, o=parts[3])
    assert torch.equal(parts[3], want) and torch.equal(S2, S)


SHAPES = [  # B, H, T, d, dv
    (1, 1, 1, 1, 1), (2, 3, 2, 16, 16), (1, 6, 63, 33, 20), (2, 2, 64, 64, 64), (1, 2, 65, 80, 48), (2, 2, 127, 64, 128),
    (1, 3, 128, 128, 128), (2, 1, 129, 128, 64), (3, 2, 300, 72, 72), (1, 2, 1000, 128, 128), (1, 3, 1025, 64, 64),
    (2, 6, 257, 8, 24),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, layout):
    check_forward(make(*shape, dtype, layout))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype, layout):
    check_backward(make(*shape, dtype, layout))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_edge_decays(d, dtype):
    x = make(1, 6, 400, d, d, dtype, kind="edge")
    check_forward(x)
    check_backward(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_states(dtype):
    x = make(2, 2, 200, 64, 64, dtype, state=False)
    check_forward(x)
    check_backward(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [24, 64, 128])
@pytest.mark.parametrize("lens", [[0, 1, 300], [299, 128, 127], [129, 256, 64], [300, 300, 2]])
def test_padded_batch(lens, d, dtype):
    """What stands behind a sequence's end is not used, whatever it is."""
    x = make(3, 2, 300, d, d, dtype, "bthd")
    y = dev(x)
    for i, n in enumerate(lens):
        for name, junk in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("-inf"))):
            y[name][i, :, n:] = junk
    check_forward(x, lens, y)
    check_backward(x, lens, y)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3000, 20000])
@pytest.mark.parametrize("d", [64, 128])
def test_long(T, d):
    """Many segments: few heads, long sequences, one of them ending early."""
    x = make(2, 1, T, d, d, BF, kind="slopes")
    x["gamma"][:] = 0.999
    check_forward(x)
    check_forward(x, [T, T // 3])
    check_backward(x, [T // 2 + 1, T])


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,d", [(1, 16, 8192, 128), (2, 40, 900, 64), (3, 8, 5000, 64)])
def test_again_and_again(B, H, T, d):
    """The same bits from call after call: no walk depends on how its warps happen to be timed."""
    x = dev(make(B, H, T, d, d, BF))
    args = (x["q"], x["k"], x["v"], x["gamma"])

    def run():
        last, d0 = torch.empty_like(x["h0"]), torch.empty_like(x["h0"])
        o = hla2.hla2_linear_forward(*args, state_in=x["h0"], state_out=last)
        return (o, last, *hla2.hla2_linear_backward(*args, x["do"], state_in=x["h0"], dstate_out=x["dlast"],
                                                    dstate_in=d0), d0)

    want = run()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        for a, b in zip(run(), want):
            differ += (a != b).any()
    assert int(differ) == 0
    assert hla2.hla2_device_status() == 0


@pytest.mark.gpu
def test_long_f32():
    x = make(1, 2, 9000, 40, 33, F32)
    check_forward(x)
    check_backward(x, [8999])


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T", [(40, 4, 200), (5, 16, 700)])
def test_many_heads(B, H, T):
    x = make(B, H, T, 64, 64, BF, "bthd")
    check_forward(x)
    check_backward(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_slices_of_one_projection(dtype, shift):
    """q, k and v as slices of one tensor, the second at any offset; v of one head for all (stride 0)."""
    B, H, T, d = 2, 2, 150, 64
    gen = torch.Generator().manual_seed(5)
    big = torch.randn(B, T, 3 * H * d + 16, generator=gen).to(dtype) * 0.3
    cuda = big.cuda()

    def cut(t, i):
        return t[:, :, shift + i * H * d:shift + (i + 1) * H * d].unflatten(2, (H, d)).transpose(1, 2)

    x = {"q": cut(big, 0), "k": cut(big, 1), "v": cut(big, 2), "do": cut(big, 2), "gamma": decays("slopes", H),
         "h0": None, "dlast": None}
    y = {**x, "q": cut(cuda, 0), "k": cut(cuda, 1), "v": cut(cuda, 2), "do": cut(cuda, 2), "gamma": x["gamma"].cuda()}
    check_forward(x, None, y)
    check_backward(x, None, y)
    x["v"], y["v"] = (t["v"][:, :1].expand(B, H, T, d) for t in (x, y))
    check_forward(x, None, y)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(100, 64), (5000, 128)])
def test_one_state_before_and_after(T, d):
    x = dev(make(1, 2, T, d, d, BF))
    want = torch.empty_like(x["h0"])
    o = hla2.hla2_linear_forward(x["q"], x["k"], x["v"], x["gamma"], state_in=x["h0"], state_out=want)
    both = x["h0"].clone()
    o2 = hla2.hla2_linear_forward(x["q"], x["k"], x["v"], x["gamma"], state_in=both, state_out=both)
    assert torch.equal(both, want) and torch.equal(o, o2)
    d0 = torch.empty_like(want)
    args = (x["q"], x["k"], x["v"], x["gamma"], x["do"])
    grads = hla2.hla2_linear_backward(*args, state_in=x["h0"], dstate_out=x["dlast"], dstate_in=d0)
    same = x["dlast"].clone()
    again = hla2.hla2_linear_backward(*args, state_in=x["h0"], dstate_out=same, dstate_in=same)
    assert torch.equal(same, d0) and all(torch.equal(s, t) for s, t in zip(grads, again))
    same = x["h0"].clone()
    again = hla2.hla2_linear_backward(*args, state_in=same, dstate_out=x["dlast"], dstate_in=same)
    assert torch.equal(same, d0) and all(torch.equal(s, t) for s, t in zip(grads, again))


@pytest.mark.gpu
def test_pieces_are_the_whole():
    """A prompt in two calls, the state handed over, is the prompt in one."""
    x = make(1, 2, 700, 64, 64, F32)
    y = dev(x)
    cut = 333
    mid = torch.empty(1, 2, 64, 64, device="cuda")
    a = hla2.hla2_linear_forward(*(y[n][:, :, :cut] for n in "qkv"), y["gamma"], state_in=y["h0"], state_out=mid)
    b = hla2.hla2_linear_forward(*(y[n][:, :, cut:] for n in "qkv"), y["gamma"], state_in=mid)
    ref, _, _, m1, _ = by_block(x["gamma"], x["q"], x["k"], x["v"], x["h0"], [700])
    near(torch.cat([a, b], 2), ref, m1, None, 64, 700, False)


@pytest.mark.gpu
def test_gradients_are_the_differences():
    """o is linear in each of q, k, v and the state: differences of the forward's fp32 outputs."""
    x = make(1, 2, 200, 16, 24, F32, seed=4)
    y = dev(x)

    def loss(**kw):
        z = {**y, **kw}
        last = torch.empty_like(y["h0"])
        o = hla2.hla2_linear_forward(z["q"], z["k"], z["v"], z["gamma"], state_in=z["h0"], state_out=last)
        return float((o.double() * y["do"].double()).sum() + (last.double() * y["dlast"].double()).sum())

    d0 = torch.empty_like(y["h0"])
    dq, dk, dv = hla2.hla2_linear_backward(y["q"], y["k"], y["v"], y["gamma"], y["do"], state_in=y["h0"],
                                           dstate_out=y["dlast"], dstate_in=d0)
    gen = torch.Generator().manual_seed(9)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("h0", d0)):
        step = torch.randn(grad.shape, generator=gen).cuda()
        diff = (loss(**{name: y[name] + step}) - loss(**{name: y[name] - step})) / 2
        size = float((grad.double() * step.double()).square().sum().sqrt())
        assert abs(diff - float((grad.double() * step.double()).sum())) < 1e-3 * size


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,H,d,dv", [(1, 1, 1, 1), (6, 3, 5, 7), (16, 16, 128, 128), (300, 4, 64, 64), (2, 2, 33, 20),
                                      (1000, 8, 16, 128), (4, 1, 128, 3), (700, 7, 128, 128), (70000, 7, 4, 8)])
def test_step(n, H, d, dv, dtype):
    gen = torch.Generator().manual_seed(n)
    g = decays("edge", H)
    q, k = ((torch.randn(n, d, generator=gen) * d ** -0.5).to(dtype) for _ in range(2))
    v, S = torch.randn(n, dv, generator=gen).to(dtype), torch.randn(n, d, dv, generator=gen)
    gg = g.double().repeat(n // H)[:, None, None]
    new = gg * S.double() + k.double()[:, :, None] * v.double()[:, None]
    o = (q.double()[:, :, None] * new).sum(1)
    mag = gg * S.double().abs() + (k.double().abs()[:, :, None] * v.double().abs()[:, None])
    st, out = S.cuda(), torch.empty(n, d, dv, device="cuda")
    got = hla2.hla2_linear_step(st, q.cuda(), k.cuda(), v.cuda(), g.cuda(), state_out=out)
    assert torch.equal(st.cpu(), S)
    # a state: a product, a sum; an output: d products and sums on top
    assert bool(((out.cpu().double() - new).abs() <= 2 * U * mag).all())
    slack = (d + 4) * U * (q.double().abs()[:, :, None] * mag).sum(1)
    assert bool((excess(got, o, slack) <= slack).all())
    got2 = hla2.hla2_linear_step(st, q.cuda(), k.cuda(), v.cuda(), g.cuda())
    assert torch.equal(st, out) and torch.equal(got, got2)


@pytest.mark.gpu
def test_step_strided_and_unaligned():
    n, d, dv = 8, 24, 40
    big = torch.randn(n, 3 * 64, device="cuda").bfloat16()
    q, k, v = big[:, 1:1 + d], big[:, 60:60 + d], big[:, 100:100 + dv]
    g = torch.tensor([0.5, 0.9], device="cuda")
    room = torch.randn(n * d * dv + 1, device="cuda")
    s1 = room[1:].view(n, d, dv)  # 4 bytes off a 16-byte step
    s2 = s1.clone()
    o2 = hla2.hla2_linear_step(s2, q.contiguous(), k.contiguous(), v.contiguous(), g)
    obig = torch.full((n, 64), 3.0, device="cuda", dtype=BF)
    o1 = hla2.hla2_linear_step(s1, q, k, v, g, o=obig[:, 5:5 + dv])
    tol = (d + 4) * 2 * U * 8
    assert float((s1 - s2).abs().max()) <= tol and float((o1.float() - o2.float()).abs().max()) <= 2.0 ** -7 * float(o2.float().abs().max())
    assert bool((obig[:, :5] == 3).all()) and bool((obig[:, 5 + dv:] == 3).all())


@pytest.mark.gpu
def test_prompt_then_steps():
    """The state of a prompt goes on token by token as the longer prompt would."""
    B, H, T, d, m = 2, 2, 130, 64, 5
    x = make(B, H, T + m, d, d, F32, "bthd")
    y = dev(x)
    state = torch.empty(B, H, d, d, device="cuda")
    hla2.hla2_linear_forward(*(y[n][:, :, :T] for n in "qkv"), y["gamma"], state_in=y["h0"], state_out=state)
    ref, S, _, m1, A = by_block(x["gamma"], x["q"], x["k"], x["v"], x["h0"], [T + m] * B)
    for t in range(T, T + m):
        q, k, v = (y[n][:, :, t].reshape(B * H, d) for n in "qkv")
        o = hla2.hla2_linear_step(state.view(B * H, d, d), q, k, v, y["gamma"])
        near(o.view(B, H, d), ref[:, :, t], m1[:, :, t], None, d, T + m, False)
    near(state, S, A, None, d, T + m, False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 40)])
def test_other_stream_and_same_bits(dtype, d):
    x = dev(make(1, 2, 2000, d, d, dtype))
    args = (x["q"], x["k"], x["v"], x["gamma"])
    o = hla2.hla2_linear_forward(*args, state_in=x["h0"])
    grads = hla2.hla2_linear_backward(*args, x["do"], state_in=x["h0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        o2 = hla2.hla2_linear_forward(*args, state_in=x["h0"], stream=s)
        g2 = hla2.hla2_linear_backward(*args, x["do"], state_in=x["h0"], stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(grads, g2))
    assert hla2.hla2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_captured(d):
    """Forward and backward in a graph, replayed on new values beside another graph with a workspace of its own."""
    T = 1500
    xs = [dev(make(1, 2, T, d, d, BF, seed=s)) for s in range(3)]
    bufs = [{k: (None if t is None else t.clone()) for k, t in xs[0].items()} for _ in range(2)]
    graphs, outs = [], []
    need = hla2.hla2_linear_workspace(1, 2, T, d, d)
    for b in bufs:
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
        b["ws"] = ws
        hla2.hla2_linear_forward(b["q"], b["k"], b["v"], b["gamma"], state_in=b["h0"], workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            last = torch.empty_like(b["h0"])
            o = hla2.hla2_linear_forward(b["q"], b["k"], b["v"], b["gamma"], state_in=b["h0"], state_out=last, workspace=ws)
            gr = hla2.hla2_linear_backward(b["q"], b["k"], b["v"], b["gamma"], b["do"], state_in=b["h0"],
                                           dstate_out=b["dlast"], workspace=ws)
        graphs.append(g)
        outs.append((o, last, *gr))
    for i in (1, 2):
        for b, x in zip(bufs, (xs[i], xs[3 - i])):
            for k in ("q", "k", "v", "do", "h0", "dlast"):
                b[k].copy_(x[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, x in zip(outs, (xs[i], xs[3 - i])):
            last = torch.empty_like(x["h0"])
            o = hla2.hla2_linear_forward(x["q"], x["k"], x["v"], x["gamma"], state_in=x["h0"], state_out=last)
            gr = hla2.hla2_linear_backward(x["q"], x["k"], x["v"], x["gamma"], x["do"], state_in=x["h0"], dstate_out=x["dlast"])
            assert all(torch.equal(a, b) for a, b in zip(out, (o, last, *gr)))


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,B,H,T,d", [(BF, 1, 4, 6000, 128), (BF, 2, 40, 900, 64), (BF, 3, 2, 130, 64), (F32, 1, 3, 700, 40)])
def test_calls_in_a_row(dtype, B, H, T, d, captured):
    """Each call's inputs are what the call before has just written, all in one workspace: the bits of the same calls
    with the device idle between them."""
    x = dev(make(B, H, T, d, d, dtype))
    ws = torch.full((max(hla2.hla2_linear_workspace(B, H, T, d, d), 16),), 255, dtype=torch.uint8, device="cuda")
    pause = lambda: None

    def run():
        q, k, v, do, h, dh = (x[n] for n in ("q", "k", "v", "do", "h0", "dlast"))
        seen = []
        for _ in range(3):
            last, first = torch.empty_like(h), torch.empty_like(h)
            o = hla2.hla2_linear_forward(q, k, v, x["gamma"], state_in=h, state_out=last, workspace=ws)
            pause()
            gr = hla2.hla2_linear_backward(q, k, o, x["gamma"], do, state_in=last, dstate_out=dh, dstate_in=first, workspace=ws)
            pause()
            v, do, h, dh = o.div_(8), gr[2].div_(8), last.div_(8), first.div_(8)
            pause()
            seen += [o, last, first, *gr]
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
    assert hla2.hla2_device_status() == 0


def backward_near(x, y, outs=None, lens=None):
    """check_backward with outputs of the caller's, on tensor cores or off them one by one: the wider tolerance."""
    B, H, T, d = x["q"].shape
    dv = x["v"].shape[-1]
    ls = [T] * B if lens is None else lens
    d0 = torch.full((B, H, d, dv), float("nan"), device="cuda")
    got = hla2.hla2_linear_backward(y["q"], y["k"], y["v"], y["gamma"], y["do"], *(outs or (None,) * 3), state_in=y["h0"],
                                    lengths=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(),
                                    dstate_out=y["dlast"], dstate_in=d0)
    for name, grad, args, width in (("dq", got[0], (x["do"], x["v"], x["k"], x["h0"].mT, ls), dv),
                                    ("dk", got[1], (x["v"], x["do"], x["q"], x["dlast"].mT, ls, True), dv),
                                    ("dv", got[2], (x["k"], x["q"], x["do"], x["dlast"], ls, True), d)):
        ref, S, m2, m1, A = by_block(x["gamma"], *args)
        near(grad, ref, m1, m2, width, T, True, name)
        if name == "dv":
            near(d0, S, A, None, d, T, True, "dstate_in")
    return got


def unaligned(t, off=1):
    """The same values `off` elements behind a 16-byte step, rows and heads as far apart as t's."""
    room = torch.empty(t.numel() + 8, device=t.device, dtype=t.dtype)
    out = room[off:off + t.numel()].view(t.shape)
    return out.copy_(t)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,d,dv", [(1, 2, 3000, 64, 64), (1, 1, 5000, 128, 96), (3, 40, 300, 64, 64)])
@pytest.mark.parametrize("off", ["k", "v", "dk", "dv", "dq", "do"])
def test_each_gradient_on_its_own_path(B, H, T, d, dv, off):
    """One tensor of the call alone keeps the walks that touch it from the tensor cores; the others go on there, and
    no walk takes the states of another's cut of the sequence."""
    x = make(B, H, T, d, dv, BF)
    y = dev(x)
    outs = [torch.empty_like(y[n]) for n in "qkv"]
    if off in y:
        y[off] = unaligned(y[off])
    else:
        outs["qkv".index(off[1])] = unaligned(outs["qkv".index(off[1])])
    backward_near(x, y, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(70, 64), (3000, 128)])
def test_states_off_their_step(T, d, dtype):
    """States 4 bytes off a 16-byte step, with one segment and with several."""
    x = make(1, 2, T, d, d, dtype)
    y = dev(x)
    want = torch.empty(1, 2, d, d, device="cuda")
    o = hla2.hla2_linear_forward(y["q"], y["k"], y["v"], y["gamma"], state_in=y["h0"], state_out=want)
    last = unaligned(want)
    last.fill_(float("nan"))
    o2 = hla2.hla2_linear_forward(y["q"], y["k"], y["v"], y["gamma"], state_in=unaligned(y["h0"]), state_out=last)
    assert torch.equal(o, o2) and torch.equal(want, last)
    args, d0 = (y["q"], y["k"], y["v"], y["gamma"], y["do"]), torch.empty_like(want)
    grads = hla2.hla2_linear_backward(*args, state_in=y["h0"], dstate_out=y["dlast"], dstate_in=d0)
    last.fill_(float("nan"))
    again = hla2.hla2_linear_backward(*args, state_in=unaligned(y["h0"]), dstate_out=unaligned(y["dlast"]), dstate_in=last)
    assert all(torch.equal(a, b) for a, b in zip((*grads, d0), (*again, last)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shift", [(BF, 0), (BF, 1), (F32, 0)])
@pytest.mark.parametrize("far", ["batch", "token"])
def test_offsets_beyond_32_bits(far, dtype, shift):
    """Sequences, or tokens, more than 2^32 elements apart."""
    B, H, T, d = (2, 2, 150, 16) if far == "batch" else (1, 2, 3, 16)
    step = 2 ** 32 + 64
    x = make(B, H, T, d, d, dtype)
    y = dev(x)
    size = H * T * d
    room = torch.empty(step * (B - 1 if far == "batch" else T - 1) + 8 * size + 64, device="cuda", dtype=dtype)

    def place(i):
        strides = (step, T * d, d, 1) if far == "batch" else (1 << 20, d, step, 1)
        return room.as_strided((B, H, T, d), strides, i * size + shift)

    for i, name in enumerate(("q", "k", "v", "do")):
        y[name] = place(i).copy_(y[name])
    ref, _, m2, m1, _ = by_block(x["gamma"], x["q"], x["k"], x["v"], x["h0"], [T] * B)
    o = hla2.hla2_linear_forward(y["q"], y["k"], y["v"], y["gamma"], O=place(4), state_in=y["h0"])
    near(o, ref, m1, m2, d, T, True, "o")
    backward_near(x, y, [place(i) for i in (5, 6, 7)])
    del room, o, y
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_lengths_outside_the_sequence(dtype):
    """Lengths are taken into 0..T."""
    x = make(4, 2, 200, 32, 32, dtype)
    y = dev(x)
    args, states = (y["q"], y["k"], y["v"], y["gamma"]), [torch.empty(4, 2, 32, 32, device="cuda") for _ in range(4)]
    outs = []
    for lens, last, d0 in (([-3, 205, 2 ** 31 - 1, 100], *states[:2]), ([0, 200, 200, 100], *states[2:])):
        ls = torch.tensor(lens, dtype=torch.int32).cuda()
        o = torch.zeros(4, 2, 200, 32, device="cuda", dtype=dtype)
        outs.append((hla2.hla2_linear_forward(*args, O=o, lengths=ls, state_in=y["h0"], state_out=last),
                     *hla2.hla2_linear_backward(*args, y["do"], lengths=ls, state_in=y["h0"], dstate_out=y["dlast"], dstate_in=d0)))
    assert all(torch.equal(a, b) for a, b in zip((*outs[0], *states[:2]), (*outs[1], *states[2:])))
    assert torch.equal(states[0][0], y["h0"][0]) and torch.equal(states[1][0], y["dlast"][0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_as_many_heads_as_there_may_be(dtype):
    x = make(257, 255, 3, 8, 8, dtype)
    check_forward(x)
    check_backward(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_new_output_of_a_padded_batch_is_zero_behind_the_ends(dtype):
    """Not what the memory held: a norm's weight gradient behind it sums over all rows."""
    x = dev(make(3, 2, 500, 64, 64, dtype, "bthd"))
    junk = torch.full_like(x["v"], float("nan"))
    del junk  # what the next output of this size is made of
    lens = torch.tensor([0, 130, 499], dtype=torch.int32).cuda()
    o = hla2.hla2_linear_forward(x["q"], x["k"], x["v"], x["gamma"], lengths=lens, state_in=x["h0"])
    assert bool(torch.isfinite(o).all()) and all(not bool(o[i, :, n:].any()) for i, n in enumerate((0, 130, 499)))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 1500])
def test_sliding_windows(T):
    """Inputs whose rows overlap in memory: token t's channels begin eight behind token t - 1's."""
    H, d = 2, 64
    gen = torch.Generator().manual_seed(3)
    flat = (torch.randn(4, H, 8 * T + d, generator=gen) * 0.3).to(BF)
    cuda = flat.cuda()
    wide = lambda t, i: t[i].as_strided((1, H, T, d), (t.stride(0), t.stride(1), 8, 1), t[i].storage_offset())
    x = {**make(1, H, T, d, d, BF), **{n: wide(flat, i) for i, n in enumerate(("q", "k", "v", "do"))}}
    y = {**dev(x), **{n: wide(cuda, i) for i, n in enumerate(("q", "k", "v", "do"))}}
    check_forward(x, None, y)
    backward_near(x, y)



@pytest.mark.gpu
def test_calls_at_once():
    """Calls of several widths, types and operators on three streams, each with memory of its own: the bits of each alone."""
    xs = [dev(make(B, H, T, d, d, dtype)) for B, H, T, d, dtype in
          ((2, 8, 2100, 64, BF), (1, 4, 3000, 128, BF), (1, 3, 500, 40, F32))]

    def run(x):
        last, d0 = torch.empty_like(x["h0"]), torch.empty_like(x["h0"])
        args = (x["q"], x["k"], x["v"], x["gamma"])
        o = hla2.hla2_linear_forward(*args, state_in=x["h0"], state_out=last)
        rows = o.transpose(1, 2).reshape(-1, o.shape[1] * o.shape[3])
        stats = torch.empty(rows.shape[0], o.shape[1], 2, device="cuda")
        n = hla2.hla2_groupnorm(rows, o.shape[1], gate=rows, activation="silu", stats=stats)
        dx, dw, _, _ = hla2.hla2_groupnorm_backward(rows, n, stats, gate=rows, activation="silu")
        return (o, last, n, dx, dw, *hla2.hla2_linear_backward(*args, x["do"], state_in=x["h0"], dstate_out=x["dlast"],
                                                               dstate_in=d0), d0)

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    seen = []
    for _ in range(20):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                seen.append(run(x))
    torch.cuda.synchronize()
    for i, got in enumerate(seen):
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 3]))
    assert hla2.hla2_device_status() == 0
