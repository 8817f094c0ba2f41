"""Gated linear recurrence (hla2_gated_scan, its backward, hla2_gated_step)
against the recurrence in 64 bits, token by token.

Tolerances, fixed before the first run:
- fp32 results: a token adds at most about 4 roundings of 2^-24 (gate, product,
  sum) to a value that the next tokens forget; with memories of up to a few
  hundred tokens they add up like a random walk to well below 2e-5 of the
  largest value.
- bf16 results: half a unit in the last place of each value on top.
- a shared gate's gradient is a sum over channels: its error is measured
  against the largest sum of the magnitudes of its terms.
"""
import numpy as np
import pytest
import torch

from _rounding import excess
from higher_order_linear_gb300 import hla2

F32 = 2e-5
FORMS = ["sigmoid", "decay"]


def make(B, H, T, d, dtype, form, shared, seed=0, layout="bhtd"):
    g = torch.Generator().manual_seed(seed)
    shape = (B, T, H, d) if layout == "bthd" else (B, H, T, d)
    x = torch.randn(shape, generator=g).to(dtype)
    gshape = (B, H, T) if shared else shape
    if form == "sigmoid":
        gate = (2 + 1.5 * torch.randn(gshape, generator=g)).to(dtype)
    else:
        gate = 1 - 0.1 * torch.rand(gshape, generator=g)
        gate[torch.rand(gshape, generator=g) < 0.01] = 0.0
        gate = gate.to(dtype)
    if layout == "bthd":
        x = x.transpose(1, 2)
        gate = gate if shared else gate.transpose(1, 2)
    return x, gate


def gates64(x, gate, form):
    a = gate.double()
    if a.dim() == 3:
        a = a[..., None].expand(x.shape)
    if form == "sigmoid":
        return torch.sigmoid(a), torch.sigmoid(-a) * x.double()
    return a.clone(), x.double()


def by_token(t, T):
    """[B,H,T,d] -> [T, B*H*d] numpy, in 64 bits."""
    B, H, _, d = t.shape
    return np.ascontiguousarray(t.double().permute(2, 0, 1, 3).reshape(T, B * H * d).numpy())


def from_tokens(a, B, H, T, d):
    return torch.from_numpy(a).reshape(T, B, H, d).permute(1, 2, 0, 3)


def kept(reset, B, H, T, d):
    """[T, B*H*d]: False where h_{t-1} counts as zero."""
    if reset is None:
        return None
    return np.ascontiguousarray((~reset).t()[:, :, None].expand(T, B, H * d).reshape(T, B * H * d).numpy())


def forward64(x, gate, form, reset=None, state=None):
    """h of every token, [B,H,T,d], in 64 bits."""
    B, H, T, d = x.shape
    a, u = (by_token(t, T) for t in gates64(x, gate, form))
    keep = kept(reset, B, H, T, d)
    h = np.zeros(B * H * d) if state is None else state.double().reshape(-1).numpy()
    out = np.empty((T, B * H * d))
    for t in range(T):
        if keep is not None:
            h = np.where(keep[t], h, 0.0)
        h = a[t] * h + u[t]
        out[t] = h
    return from_tokens(out, B, H, T, d)


def backward64(x, gate, do, form, reset=None, state=None, dlast=None):
    """dX, dG's terms before a shared gate's sum, dstate_in, by the formulas."""
    B, H, T, d = x.shape
    h = by_token(forward64(x, gate, form, reset, state), T)
    a, _ = (by_token(t, T) for t in gates64(x, gate, form))
    keep = kept(reset, B, H, T, d)
    first = np.zeros((1, B * H * d)) if state is None else state.double().reshape(1, -1).numpy()
    before = np.concatenate([first, h[:-1]])
    if keep is not None:
        before = np.where(keep, before, 0.0)
    mu = np.zeros(B * H * d) if dlast is None else dlast.double().reshape(-1).numpy()
    up = by_token(do, T)
    lam = np.empty_like(h)
    for t in range(T - 1, -1, -1):
        lam[t] = up[t] + mu
        mu = a[t] * lam[t]
        if keep is not None:
            mu = np.where(keep[t], mu, 0.0)
    if form == "sigmoid":
        g = gate.double() if gate.dim() == 4 else gate.double()[..., None].expand(x.shape)
        z = by_token(torch.sigmoid(-g), T)
        dx, dg = z * lam, lam * a * z * (before - by_token(x, T))
    else:
        dx, dg = lam, lam * before
    return from_tokens(dx, B, H, T, d), from_tokens(dg, B, H, T, d), torch.from_numpy(mu).reshape(B, H, d)


def rel(got, ref, den=None):
    """Largest error beyond the rounding to got's type, of the largest value (or of ``den``)."""
    ref = ref.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    den = float(ref.abs().max() if den is None else den) or 1.0
    return float(excess(got, ref, F32 * den).max()) / den


def resets(kind, B, T, seed=1):
    if kind == "none":
        return None
    r = torch.zeros(B, T, dtype=torch.bool)
    if kind == "first":
        r[:, 0] = True
    elif kind == "every":
        r[:] = True
    elif kind == "edges":  # around multiples of 64 and 128
        for t in (1, 63, 64, 65, 127, 128, 129, 255, 256, T - 1):
            if 0 <= t < T:
                r[t % B, t] = True
    else:
        r = torch.rand(B, T, generator=torch.Generator().manual_seed(seed)) < 0.02
    return r


def check(B, H, T, d, dtype, out_dtype, form, shared, reset="none", state=False, layout="bhtd", backward=True, seed=0):
    x, gate = make(B, H, T, d, dtype, form, shared, seed, layout)
    r = resets(reset, B, T)
    gen = torch.Generator().manual_seed(seed + 7)
    h0 = torch.randn(B, H, d, generator=gen) if state else None
    dlast = torch.randn(B, H, d, generator=gen) if state else None
    do = torch.randn(B, H, T, d, generator=gen).to(out_dtype)
    if layout == "bthd":
        do = do.transpose(1, 2).contiguous().transpose(1, 2)
    dev = lambda t: None if t is None else t.cuda()
    xc, gc, rc = x.cuda(), gate.cuda(), dev(r)
    last = torch.full((B, H, d), float("nan"), device="cuda")
    carry = torch.full((B, H, hla2.hla2_gated_scan_carry_len(T, d)), float("nan"), device="cuda")
    o = hla2.hla2_gated_scan(xc, gc, form=form, reset=rc, state_in=dev(h0), state_out=last, carry=carry,
                             out_dtype=out_dtype)
    ref = forward64(x, gate, form, r, h0)
    assert o.dtype == out_dtype and o.shape == x.shape
    assert rel(o, ref) < F32
    assert rel(last, ref[:, :, -1], ref.abs().max()) < F32
    assert torch.equal(o, hla2.hla2_gated_scan(xc, gc, form=form, reset=rc, state_in=dev(h0), out_dtype=out_dtype))
    if not backward:
        return
    d0 = torch.full((B, H, d), float("nan"), device="cuda")
    args = dict(form=form, reset=rc, dstate_out=dev(dlast), dstate_in=d0)
    dx, dg = hla2.hla2_gated_scan_backward(xc, gc, do.cuda(), carry, **args)
    rx, rg, r0 = backward64(x, gate, do, form, r, h0, dlast)
    assert dx.dtype == dtype and dg.dtype == dtype and dg.shape == gate.shape
    assert rel(dx, rx) < F32
    if shared:
        den = rg.abs().sum(-1).max()
        assert rel(dg, rg.sum(-1), den) < F32
    else:
        assert rel(dg, rg) < F32
    assert rel(d0, r0, max(r0.abs().max(), rx.abs().max())) < F32
    dx2, dg2 = hla2.hla2_gated_scan_backward(xc, gc, do.cuda(), carry, **args)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 2, 7, 63, 64, 65, 127, 128, 129, 257, 1000, 2049])
def test_lengths(T, form):
    check(2, 2, T, 64, torch.float32, torch.float32, form, False, "random", True)
    check(1, 3, T, 128, torch.bfloat16, torch.bfloat16, form, False, "random", True, "bthd")


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d", [1, 3, 4, 16, 33, 48, 64, 65, 80, 96, 100, 127, 128])
def test_channels(d, form):
    check(2, 3, 300, d, torch.float32, torch.float32, form, False, "edges", True)
    check(2, 3, 300, d, torch.bfloat16, torch.float32, form, True, "none", False)
    check(1, 2, 300, d, torch.bfloat16, torch.bfloat16, form, False, "none", True, "bthd")


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                       (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("reset", ["none", "first", "every", "edges", "random"])
def test_types_resets_and_shared_gates(form, shared, dtype, out, reset):
    check(2, 2, 517, 64, dtype, out, form, shared, reset, True)
    check(2, 2, 259, 128, dtype, out, form, shared, reset, False, "bthd")


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 70001, 16), (1, 2, 40000, 128), (2, 40, 5000, 64)])
def test_long(form, B, H, T, d):
    """Many tiles, groups of tiles and groups of groups; few rows and many."""
    check(B, H, T, d, torch.float32, torch.float32, form, False, "random" if B == 2 else "none", True)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_long_memory(form):
    """Gates that hardly forget: a = 1 - 1e-4 over 20000 tokens.  The state is a sum of about 1e4 terms:
    roundings of 2^-24 of it at every token, 1e4 of them remembered, at worst 1e4 * 2^-24 = 6e-4."""
    B, H, T, d = 1, 1, 20000, 32
    x = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(3))
    gate = torch.full((B, H, T, d), 9.2 if form == "sigmoid" else 0.9999)
    o = hla2.hla2_gated_scan(x.cuda(), gate.cuda(), form=form)
    assert rel(o, forward64(x, gate, form)) < 6e-4


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_extreme_gates(form):
    """Gates that forget all, nothing, or saturate."""
    B, H, T, d = 1, 1, 300, 16
    x = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(4))
    vals = torch.tensor([-1e4, -100.0, -30.0, 0.0, 30.0, 100.0, 1e4, float("inf"), -float("inf")]) if form == "sigmoid" \
        else torch.tensor([0.0, -0.0, 1.0, -1.0, 0.5, 1e-30, -1e-30, 1e-45])
    gate = vals[torch.randint(len(vals), (B, H, T, d), generator=torch.Generator().manual_seed(5))]
    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    o = hla2.hla2_gated_scan(x.cuda(), gate.cuda(), form=form, carry=carry)
    assert rel(o, forward64(x, gate, form)) < F32
    do = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(6))
    dx, dg = hla2.hla2_gated_scan_backward(x.cuda(), gate.cuda(), do.cuda(), carry, form=form)
    rx, rg, _ = backward64(x, gate, do, form)
    assert rel(dx, rx) < F32 and rel(dg, rg) < F32


def gate_slack(g):
    """How far a and z = 1 - a of a sigmoid gate may each be off, of themselves: the rounding of g log2(e) moves the
    exponent by |g| 2^-24 (and the constant's own by a quarter of that); the power of two has 2 ulp, the sum with 1
    a half, the reciprocal 1, their product a half: 4 ulp of 2^-23."""
    return g.double().abs() * 1.25 * 2.0 ** -24 + 4 * 2.0 ** -23


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.float32, 128), (torch.float32, 33),
                                     (torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 33)])
@pytest.mark.parametrize("shared", [False, True])
def test_both_ends_of_a_gate_keep_their_precision(dtype, d, shared):
    """One token, from h = 1 with x = 0 (h is a) and from 0 with x = 1 (h is z), and the gradients z, a z and a:
    each of its own size, however small."""
    n = 161
    g = torch.linspace(-80, 80, n, dtype=torch.float64).to(dtype)
    gate = g.view(1, n, 1) if shared else g.view(1, n, 1, 1).expand(1, n, 1, d).contiguous()
    a, z = torch.sigmoid(g.double()), torch.sigmoid(-g.double())
    slack = gate_slack(g)
    zero, one = torch.zeros(1, n, 1, d, dtype=dtype, device="cuda"), torch.ones(1, n, 1, d, dtype=dtype, device="cuda")
    h1 = torch.ones(1, n, d, device="cuda")
    gc = gate.cuda()

    def near(got, ref, times=1.0):
        ref, tol = ref.view(1, n, 1, 1), (times * slack * ref).view(1, n, 1, 1)
        assert (excess(got.view(1, n, 1, -1), ref, tol) <= tol).all()

    carry = torch.empty(1, n, hla2.hla2_gated_scan_carry_len(1, d), device="cuda")
    near(hla2.hla2_gated_scan(one, gc), z)
    near(hla2.hla2_gated_scan(zero, gc, state_in=h1, carry=carry), a)
    d0 = torch.empty(1, n, d, device="cuda")
    dx, dg = hla2.hla2_gated_scan_backward(zero, gc, one, carry, dstate_in=d0)
    near(dx, z, 2)  # z is 1 - a or a is 1 - z: a rounding more
    near(d0, a, 2)
    near(dg, d * a * z if shared else a * z, 4 + d / 16 if shared else 4)
    state = h1.view(n, d).clone()
    sg = gc.view(n) if shared else gc.view(n, d)
    near(hla2.hla2_gated_step(state, zero.view(n, d), sg), a)
    near(hla2.hla2_gated_step(torch.zeros_like(state), one.view(n, d), sg), z)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,T", [(torch.float32, 64, 700), (torch.float32, 33, 700), (torch.bfloat16, 64, 700),
                                       (torch.bfloat16, 128, 700), (torch.bfloat16, 128, 2100)])
def test_closing_gates_over_many_tokens(dtype, d, T):
    """Gates from closed to open, and positive values over several powers of ten: each token's result is good to its
    own size.  err, the relative error of h, goes by err' = w err + (gate's) + 2 roundings, w the part of h' that comes
    from h; twice that for the roundings of the maps of runs and tiles.  mu goes the same way, backwards; dG holds a
    difference h - x, whose error is that of both."""
    B, H = 1, 2
    gen = torch.Generator().manual_seed(95)
    gate = (-14 + 18 * torch.rand(B, H, T, d, generator=gen)).to(dtype)
    x = torch.exp(3 * torch.randn(B, H, T, d, generator=gen)).to(dtype)
    do = torch.exp(3 * torch.randn(B, H, T, d, generator=gen))
    h0 = torch.full((B, H, d), 1e6)
    g = gate.double()
    a, z, slack = torch.sigmoid(g), torch.sigmoid(-g), gate_slack(gate) + 2 * 2.0 ** -24
    h, err, hs, errs, before = h0.double(), torch.zeros(B, H, d, dtype=torch.float64), [], [], []
    befe = []
    for t in range(T):
        before.append(h)
        befe.append(err)
        new = a[:, :, t] * h + z[:, :, t] * x[:, :, t].double()
        err = a[:, :, t] * h / new * err + slack[:, :, t]
        h = new
        hs.append(h)
        errs.append(err)
    ref, err = torch.stack(hs, 2), torch.stack(errs, 2)
    before, befe = torch.stack(before, 2), torch.stack(befe, 2)
    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    o = hla2.hla2_gated_scan(x.cuda(), gate.cuda(), state_in=h0.cuda(), carry=carry)
    assert ((o.double().cpu() - ref).abs() <= 2 * err * ref).all()
    dx, dg = hla2.hla2_gated_scan_backward(x.cuda(), gate.cuda(), do.cuda(), carry)
    mu, me = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    lam, le = torch.empty_like(ref), torch.empty_like(ref)
    for t in range(T - 1, -1, -1):
        lam[:, :, t] = do[:, :, t].double() + mu
        le[:, :, t] = me * mu / lam[:, :, t] + 2.0 ** -24
        mu = a[:, :, t] * lam[:, :, t]
        me = le[:, :, t] + slack[:, :, t]
    tol = 2 * (le + slack) * z * lam
    assert (excess(dx, z * lam, tol) <= tol).all()
    size = a * z * lam
    tol = 2 * size * ((le + 2 * slack) * (before - x.double()).abs() + (befe + 2.0 ** -24) * before + 2.0 ** -24 * x.double())
    assert (excess(dg, size * (before - x.double()), tol) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("at", [5, 127, 128, 700])
def test_nothing_passes_a_reset(form, bad, at):
    """inf and NaN of one document reach its own later tokens and no other document's."""
    B, H, T, d = 1, 2, 2500, 64
    x, gate = make(B, H, T, d, torch.float32, form, False, 11)
    x[:, :, at] = bad
    for cut in (at + 1, at + 70, at + 900):
        r = torch.zeros(B, T, dtype=torch.bool)
        r[:, cut] = True
        o = hla2.hla2_gated_scan(x.cuda(), gate.cuda(), form=form, reset=r.cuda()).cpu()
        clean = x.clone()
        clean[:, :, at] = 0
        ref = forward64(clean, gate, form, r)
        assert torch.isfinite(o[:, :, :at]).all() and torch.isfinite(o[:, :, cut:]).all()
        assert not torch.isfinite(o[:, :, at]).any()
        assert rel(o[:, :, :at], ref[:, :, :at]) < F32
        assert rel(o[:, :, cut:], ref[:, :, cut:]) < F32


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.float32, 128), (torch.float32, 33),
                                     (torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 20)])
def test_nan_stays_without_a_reset(dtype, d, shared):
    """Decays of both signs whose products underflow: NaN in a state reaches every later token (0 * NaN is NaN),
    and in a gradient every earlier one, up to a reset and not beyond."""
    B, H, T, cut = 1, 3, 6000, 4500
    g = torch.Generator().manual_seed(91)
    shape = (B, H, T) if shared else (B, H, T, d)
    gate = ((0.2 + 0.3 * torch.rand(shape, generator=g)) * torch.where(torch.rand(shape, generator=g) < 0.5, -1.0, 1.0)).to(dtype)
    x = torch.randn(B, H, T, d, generator=g).to(dtype).cuda()
    h0 = torch.full((B, H, d), float("nan"), device="cuda")
    r = torch.zeros(B, T, dtype=torch.bool)
    r[:, cut] = True
    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    o = hla2.hla2_gated_scan(x, gate.cuda(), form="decay", state_in=h0, reset=r.cuda())
    assert torch.isnan(o[:, :, :cut]).all() and torch.isfinite(o[:, :, cut:]).all()
    hla2.hla2_gated_scan(x, gate.cuda(), form="decay", reset=r.cuda(), carry=carry)
    d0 = torch.empty(B, H, d, device="cuda")
    dx, dg = hla2.hla2_gated_scan_backward(x, gate.cuda(), x, carry, form="decay", reset=r.cuda(), dstate_out=h0, dstate_in=d0)
    assert torch.isfinite(dx[:, :, :cut]).all() and torch.isnan(dx[:, :, cut:]).all()
    assert torch.isfinite(d0).all()
    hla2.hla2_gated_scan(x, gate.cuda(), form="decay", carry=carry)
    dx, dg = hla2.hla2_gated_scan_backward(x, gate.cuda(), x, carry, form="decay", dstate_out=h0, dstate_in=d0)
    assert torch.isnan(dx).all() and torch.isnan(dg).all() and torch.isnan(d0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_gradient_against_differences(form):
    """Central differences of the 64-bit forward: their own error is about eps^2 = 1e-8."""
    B, H, T, d = 1, 2, 9, 4
    x, gate = make(B, H, T, d, torch.float32, form, False, 21)
    r = torch.zeros(B, T, dtype=torch.bool)
    r[0, 5] = True
    gen = torch.Generator().manual_seed(22)
    h0, do, dl = torch.randn(B, H, d, generator=gen), torch.randn(B, H, T, d, generator=gen), torch.randn(B, H, d, generator=gen)

    def loss(x, gate, h0):
        h = forward64(x, gate, form, r, h0)
        return float((h * do.double()).sum() + (h[:, :, -1] * dl.double()).sum())

    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    hla2.hla2_gated_scan(x.cuda(), gate.cuda(), form=form, reset=r.cuda(), state_in=h0.cuda(), carry=carry)
    d0 = torch.empty(B, H, d, device="cuda")
    dx, dg = hla2.hla2_gated_scan_backward(x.cuda(), gate.cuda(), do.cuda(), carry, form=form, reset=r.cuda(),
                                           dstate_out=dl.cuda(), dstate_in=d0)
    eps = 1e-4
    for got, at in ((dx, 0), (dg, 1), (d0, 2)):
        args = [x.double(), gate.double(), h0.double()]
        flat = got.double().cpu().reshape(-1)
        for i in range(0, flat.numel(), 3):
            vals = []
            for sgn in (1, -1):
                moved = [a.clone() for a in args]
                moved[at].view(-1)[i] += sgn * eps
                vals.append(loss(*moved))
            num = (vals[0] - vals[1]) / (2 * eps)
            assert abs(num - float(flat[i])) < 1e-5 * max(1.0, float(flat.abs().max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_operands(dtype):
    """Slices of a wider projection, odd offsets; the gaps of a strided output stay untouched."""
    B, H, T, d = 2, 3, 200, 24
    gen = torch.Generator().manual_seed(31)
    for off, width in ((0, 64), (1, 51), (8, 80)):
        wide = torch.randn(B, T, H, 2 * width, generator=gen).to(dtype).cuda()
        x = wide[..., off:off + d].transpose(1, 2)
        gate = wide[..., width + off:width + off + d].transpose(1, 2)
        full = torch.full((B, T, H, width), 7.0, device="cuda", dtype=dtype)
        o = full[..., off:off + d].transpose(1, 2)
        carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
        ret = hla2.hla2_gated_scan(x, gate, O=o, carry=carry)
        assert ret is o
        ref = forward64(x.cpu(), gate.cpu(), "sigmoid")
        assert rel(o, ref) < F32
        assert (full[..., :off] == 7).all() and (full[..., off + d:] == 7).all()
        do = torch.randn(B, H, T, d, generator=gen).to(dtype)
        gx, gg = torch.full_like(full, 7.0), torch.full_like(full, 7.0)
        dx, dg = (t[..., off:off + d].transpose(1, 2) for t in (gx, gg))
        hla2.hla2_gated_scan_backward(x, gate, do.cuda(), carry, dX=dx, dG=dg)
        rx, rg, _ = backward64(x.cpu(), gate.cpu(), do, "sigmoid")
        assert rel(dx, rx) < F32 and rel(dg, rg) < F32
        for t in (gx, gg):
            assert (t[..., :off] == 7).all() and (t[..., off + d:] == 7).all()


def check_large(B, H, T, d, dtype, out_dtype, form, shared, reset, seed, layout="bthd"):
    """check(), with the 64-bit recurrences on the GPU, all heads at once."""
    x, gate = make(B, H, T, d, dtype, form, shared, seed, layout)
    r = resets(reset, B, T)
    gen = torch.Generator().manual_seed(seed + 7)
    h0, dl = torch.randn(B, H, d, generator=gen), torch.randn(B, H, d, generator=gen)
    do = torch.randn(B, H, T, d, generator=gen).to(out_dtype)
    xc, gc, doc, h0c, dlc = x.cuda(), gate.cuda(), do.cuda(), h0.cuda(), dl.cuda()
    rc = None if r is None else r.cuda()
    a, u = gates64(xc, gc, form)
    z = torch.sigmoid(-(gc.double()[..., None] if shared else gc.double())) if form == "sigmoid" else None
    keep = torch.ones(B, T, dtype=torch.bool, device="cuda") if rc is None else ~rc
    h, hs, before = h0c.double(), torch.empty_like(u), torch.empty_like(u)
    for t in range(T):
        h = torch.where(keep[:, t, None, None], h, 0.0)
        before[:, :, t] = h
        h = a[:, :, t] * h + u[:, :, t]
        hs[:, :, t] = h
    mu, lam = dlc.double(), torch.empty_like(u)
    for t in range(T - 1, -1, -1):
        lam[:, :, t] = doc[:, :, t].double() + mu
        mu = torch.where(keep[:, t, None, None], a[:, :, t] * lam[:, :, t], 0.0)
    rx = z * lam if form == "sigmoid" else lam
    rg = lam * a * z * (before - xc.double()) if form == "sigmoid" else lam * before
    carry = torch.full((B, H, hla2.hla2_gated_scan_carry_len(T, d)), float("nan"), device="cuda")
    last, d0 = torch.empty_like(h0c), torch.empty_like(h0c)
    o = hla2.hla2_gated_scan(xc, gc, form=form, reset=rc, state_in=h0c, state_out=last, carry=carry, out_dtype=out_dtype)
    dx, dg = hla2.hla2_gated_scan_backward(xc, gc, doc, carry, form=form, reset=rc, dstate_out=dlc, dstate_in=d0)
    assert rel(o, hs.cpu()) < F32 and rel(last, h.cpu(), hs.abs().max()) < F32
    assert rel(dx, rx.cpu()) < F32 and rel(d0, mu.cpu(), max(mu.abs().max(), rx.abs().max())) < F32
    if shared:
        assert rel(dg, rg.sum(-1).cpu(), rg.abs().sum(-1).max()) < F32
    else:
        assert rel(dg, rg.cpu()) < F32


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float32)])
@pytest.mark.parametrize("B,H,T,d,reset", [(2, 40, 2500, 64, "random"), (1, 20, 3001, 128, "random"),
                                           (3, 25, 1200, 80, "edges"), (1, 64, 2000, 128, "none")])
def test_many_tiles_to_a_block(form, shared, dtype, out, B, H, T, d, reset):
    """940 to 2048 tiles, 6 to 14 for each SM of a GB300: every ring of stages is used again, with the resets, maps
    and flags that its stages hold, in each direction and with both layouts of gates."""
    check_large(B, H, T, d, dtype, out, form, shared, reset, 101)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_runs_beyond_the_range_of_products(dtype, d, shared):
    """Gates and inputs, here and there, whose products over a few tokens leave fp32's range, beside ordinary ones, in
    both directions."""
    B, H, T = 1, 40, 1500
    g = torch.Generator().manual_seed(103)
    shape = (B, H, T) if shared else (B, H, T, d)
    gate = 2 + 1.5 * torch.randn(shape, generator=g)
    odd = torch.rand(shape, generator=g)
    for i, v in enumerate((15.0, 40.0, 90.0, 1e4, -1e4, -90.0, float("inf"), -float("inf"))):
        gate[(odd >= 0.004 * i) & (odd < 0.004 * (i + 1))] = v
    gate[:, :, 700:800] += 12  # a stretch that hardly forgets
    gate = gate.to(dtype)
    x = torch.randn(B, H, T, d, generator=g).to(dtype)
    do = torch.randn(B, H, T, d, generator=g).to(dtype)
    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    ref = forward64(x, gate, "sigmoid")
    assert rel(hla2.hla2_gated_scan(x.cuda(), gate.cuda(), carry=carry), ref) < F32
    dx, dg = hla2.hla2_gated_scan_backward(x.cuda(), gate.cuda(), do.cuda(), carry)
    rx, rg, _ = backward64(x, gate, do, "sigmoid")
    assert rel(dx, rx) < F32
    assert (rel(dg, rg.sum(-1), rg.abs().sum(-1).max()) if shared else rel(dg, rg)) < F32
    by = 2.0 ** 100  # inputs that many times as large: so is every result
    assert rel(hla2.hla2_gated_scan(x.cuda() * by, gate.cuda()) / by, ref) < F32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.float32, 33), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("level", [-6.0, -2.0, 2.0, 9.0])
def test_inputs_of_any_size(dtype, d, shared, level):
    """The recurrence is linear in x, and its gradient in dO: inputs times a power of two give results times that, to
    the bounds of ordinary ones, beside runs of zeros and ordinary inputs too."""
    B, H, T = 1, 4, 600
    g = torch.Generator().manual_seed(107)
    gate = (level + 1.5 * torch.randn((B, H, T) if shared else (B, H, T, d), generator=g)).to(dtype)
    x = torch.randn(B, H, T, d, generator=g).to(dtype)
    do = torch.randn(B, H, T, d, generator=g).to(dtype)
    x[:, :, 200:290], do[:, :, 250:340] = 0, 0
    gc = gate.cuda()
    ref = forward64(x, gate, "sigmoid")
    rx, rg, _ = backward64(x, gate, do, "sigmoid")
    if shared:
        rg, den = rg.sum(-1), rg.abs().sum(-1).max()
    for by in (1.0, 2.0 ** -60, 2.0 ** -80, 2.0 ** -100, 2.0 ** 100):
        xs, ds = (x.float() * by).to(dtype).cuda(), (do.float() * by).to(dtype).cuda()
        carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
        assert rel(hla2.hla2_gated_scan(xs, gc, carry=carry).double() / by, ref) < F32
        hla2.hla2_gated_scan(x.cuda(), gc, carry=carry)
        dx, dg = hla2.hla2_gated_scan_backward(x.cuda(), gc, ds, carry)
        scale = lambda t: (t.double() / by).to(dtype)  # exact: a power of two
        assert rel(scale(dx), rx) < F32
        assert (rel(scale(dg), rg, den) if shared else rel(scale(dg), rg)) < F32


@pytest.mark.gpu
def test_graph_replays_on_new_values():
    """A graph of the scan, its gradient and the step, replayed on inputs changed in place, with the workspaces as the
    replay before left them (tickets and maps of other inputs)."""
    B, H, T, d = 2, 3, 3000, 64
    sets = [[t.cuda() for t in make(B, H, T, d, torch.bfloat16, "sigmoid", False, 111 + i)] for i in range(3)]
    x, gate = (t.clone() for t in sets[0])
    do = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(112)).cuda()
    o, dx, dg = torch.empty(x.shape, device="cuda"), torch.empty_like(x), torch.empty_like(gate)
    n = hla2.hla2_gated_scan_workspace(B, H, T, d)
    w1, w2 = (torch.empty(n, device="cuda", dtype=torch.uint8) for _ in range(2))
    carry = torch.zeros(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    state, so = torch.zeros(B * H, d, device="cuda"), torch.empty(B * H, d, device="cuda")
    xt, gt = (t[:, :, 5].reshape(B * H, d).clone() for t in (x, gate))

    def calls():
        hla2.hla2_gated_scan(x, gate, O=o, carry=carry, state_in=state.view(B, H, d), state_out=state.view(B, H, d),
                             workspace=w1)
        hla2.hla2_gated_scan_backward(x, gate, do, carry, dX=dx, dG=dg, workspace=w2)
        hla2.hla2_gated_step(state, xt, gt, o=so)

    calls()  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    state.zero_()
    follow = torch.zeros(B, H, d, device="cuda")
    for k in (0, 1, 2, 1):
        x.copy_(sets[k][0])
        gate.copy_(sets[k][1])
        xt.copy_(x[:, :, 5].reshape(B * H, d))
        gt.copy_(gate[:, :, 5].reshape(B * H, d))
        graph.replay()
        kept = torch.empty_like(carry)
        ref = hla2.hla2_gated_scan(x, gate, carry=kept, state_in=follow, state_out=follow)
        rx, rg = hla2.hla2_gated_scan_backward(x, gate, do, kept)
        rs = hla2.hla2_gated_step(follow.view(B * H, d), xt, gt)
        assert torch.equal(o, ref) and torch.equal(dx, rx) and torch.equal(dg, rg)
        assert torch.equal(so, rs) and torch.equal(state, follow.view(B * H, d))


def windows(T, d, seed, dtype=torch.float32, step=1):
    """[1, 2, T, d] whose rows are windows of d elements, `step` apart, of one sequence for each head."""
    base = torch.randn(2, (T - 1) * step + d, generator=torch.Generator().manual_seed(seed)).to(dtype)
    return base.as_strided((1, 2, T, d), (0, base.stride(0), step, 1))


def test_outputs_are_laid_out_for_the_kernels():
    """An output of the binding's own has a contiguous last dimension, whatever its input's strides."""
    for T, d, step in ((8, 16, 1), (16, 16, 1), (20, 16, 1), (3, 16, 5), (1, 16, 1), (5, 1, 1)):
        x = windows(T, d, 1, step=step)
        for o in (hla2._like(x), hla2._like(x, torch.bfloat16)):
            assert o.shape == x.shape and (d == 1 or o.stride(-1) == 1) \
                and o.untyped_storage().nbytes() == o.numel() * o.element_size()
    y = torch.zeros(2, 5, 3, 8).transpose(1, 2)
    assert hla2._like(y).stride() == y.stride()


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,step", [(8, 16, 1), (40, 64, 1), (300, 16, 4)])
def test_overlapping_inputs(T, d, step):
    """Sliding windows as inputs: elements that are in several places."""
    x, gate = windows(T, d, 43, step=step), windows(T, d, 44, step=step)
    dev = lambda t: t.as_strided((2, t.stride(1)), (t.stride(1), 1)).cuda().as_strided(t.shape, t.stride())
    xc, gc = dev(x), dev(gate)
    assert torch.equal(xc.cpu(), x)
    carry = torch.empty(1, 2, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    assert rel(hla2.hla2_gated_scan(xc, gc, carry=carry), forward64(x, gate, "sigmoid")) < F32
    do = windows(T, d, 45, step=step)
    dx, dg = hla2.hla2_gated_scan_backward(xc, gc, dev(do), carry)
    rx, rg, _ = backward64(x, gate, do, "sigmoid")
    assert rel(dx, rx) < F32 and rel(dg, rg) < F32


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Tokens whose element offset passes 2^31."""
    T, stride, d = 70000, 32768, 16
    base = torch.empty((T, stride), device="cuda", dtype=torch.bfloat16)
    x = torch.randn((T, d), generator=torch.Generator().manual_seed(41)).to(torch.bfloat16)
    base[:, :d] = x.cuda()
    view = base[None, None, :, :d]
    gate = torch.full((1, 1, T), 0.9, dtype=torch.bfloat16)
    o = hla2.hla2_gated_scan(view, gate.cuda(), form="decay", O=base[None, None, :, 64:64 + d])
    ref = forward64(x[None, None], gate, "decay")
    assert rel(o, ref) < F32


@pytest.mark.gpu
def test_other_stream():
    x, gate = make(2, 4, 3000, 128, torch.bfloat16, "sigmoid", False, 51)
    ref = hla2.hla2_gated_scan(x.cuda(), gate.cuda())
    s = torch.cuda.Stream()
    xc, gc = x.cuda(), gate.cuda()
    s.wait_stream(torch.cuda.current_stream())
    for how in (s, s.cuda_stream):
        o = hla2.hla2_gated_scan(xc, gc, stream=how)
        s.synchronize()
        assert torch.equal(o, ref)


@pytest.mark.gpu
def test_graph_capture():
    x, gate = make(1, 2, 2000, 64, torch.bfloat16, "sigmoid", False, 52)
    xc, gc = x.cuda(), gate.cuda()
    o = torch.empty(x.shape, device="cuda")
    ws = torch.empty(max(16, hla2.hla2_gated_scan_workspace(1, 2, 2000, 64)), device="cuda", dtype=torch.uint8)
    ref = hla2.hla2_gated_scan(xc, gc).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hla2.hla2_gated_scan(xc, gc, O=o, workspace=ws)
    for _ in range(3):
        o.zero_()
        ws.fill_(255)  # whatever the workspace held
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 128), (3, 33), (16, 128), (5, 80), (4096, 64), (1000, 6)])
def test_step(form, shared, n, d):
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)):
        x, gate = make(n, 1, 1, d, dtype, form, shared, 61)
        x, gate = x[:, 0, 0].contiguous(), (gate[:, 0, 0] if not shared else gate[:, 0, 0]).contiguous()
        h0 = torch.randn(n, d, generator=torch.Generator().manual_seed(62))
        ref = forward64(x[:, None, None], gate[:, None, None], form, None, h0[:, None])[:, 0, 0]
        state = h0.cuda()
        new = torch.full_like(state, float("nan"))
        o = hla2.hla2_gated_step(state, x.cuda(), gate.cuda(), form=form, out_dtype=out, state_out=new)
        assert torch.equal(state.cpu(), h0)
        assert rel(new, ref) < F32 and rel(o, ref) < F32
        hla2.hla2_gated_step(state, x.cuda(), gate.cuda(), form=form, o=torch.empty_like(o))
        assert torch.equal(state, new)


@pytest.mark.gpu
@pytest.mark.parametrize("off", [0, 1, 4])
def test_step_on_slices_of_a_projection(off):
    n, d = 9, 20
    wide = torch.randn(n, 70, generator=torch.Generator().manual_seed(63)).to(torch.bfloat16).cuda()
    x, g = wide[:, off:off + d], wide[:, 30 + off:30 + off + d]
    full = torch.full((n, 40), 9.0, device="cuda")
    state = torch.zeros(n, d, device="cuda")
    hla2.hla2_gated_step(state, x, g, o=full[:, off:off + d])
    ref = forward64(x.cpu()[:, None, None], g.cpu()[:, None, None], "sigmoid")[:, 0, 0]
    assert rel(full[:, off:off + d], ref) < F32 and rel(state, ref) < F32
    assert (full[:, :off] == 9).all() and (full[:, off + d:] == 9).all()


@pytest.mark.gpu
def test_steps_continue_a_scan():
    B, H, T, d, more = 2, 3, 200, 64, 5
    x, gate = make(B, H, T + more, d, torch.bfloat16, "sigmoid", False, 71)
    xc, gc = x.cuda(), gate.cuda()
    last = torch.empty(B, H, d, device="cuda")
    hla2.hla2_gated_scan(xc[:, :, :T].contiguous(), gc[:, :, :T].contiguous(), state_out=last)
    state = last.view(B * H, d)
    ref = forward64(x, gate, "sigmoid")
    for t in range(T, T + more):
        o = hla2.hla2_gated_step(state, xc[:, :, t].reshape(B * H, d), gc[:, :, t].reshape(B * H, d))
        assert rel(o.view(B, H, d), ref[:, :, t], ref.abs().max()) < F32


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,B,H,T,d", [(torch.bfloat16, 1, 16, 2000, 128), (torch.bfloat16, 2, 30, 700, 64),
                                           (torch.float32, 3, 50, 130, 80), (torch.float32, 1, 1, 9000, 33),
                                           (torch.bfloat16, 2, 2, 50, 16)])
def test_states_in_place(form, dtype, B, H, T, d):
    """One tensor as the state before and after, and one as the gradients of both: the same bits as with two."""
    x, gate = make(B, H, T, d, dtype, form, False, 81)
    g = torch.Generator().manual_seed(82)
    h0, dl = torch.randn(B, H, d, generator=g).cuda(), torch.randn(B, H, d, generator=g).cuda()
    do = torch.randn(B, H, T, d, generator=g).to(dtype).cuda()
    xc, gc = x.cuda(), gate.cuda()
    last, first = torch.empty_like(h0), torch.empty_like(h0)
    carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device="cuda")
    o = hla2.hla2_gated_scan(xc, gc, form=form, state_in=h0, state_out=last, carry=carry)
    dx, dg = hla2.hla2_gated_scan_backward(xc, gc, do, carry, form=form, dstate_out=dl, dstate_in=first)
    assert rel(o, forward64(x, gate, form, None, h0.cpu())) < F32
    for _ in range(20):
        state, grad = h0.clone(), dl.clone()
        o2 = hla2.hla2_gated_scan(xc, gc, form=form, state_in=state, state_out=state)
        assert torch.equal(o2, o) and torch.equal(state, last)
        dx2, dg2 = hla2.hla2_gated_scan_backward(xc, gc, do, carry, form=form, dstate_out=grad, dstate_in=grad)
        assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(grad, first)


@pytest.mark.gpu
def test_a_sequence_in_pieces():
    """Pieces of one sequence, the state handed on in place."""
    B, H, d, cuts = 2, 3, 64, [0, 1, 300, 301, 1500, 2000]
    x, gate = make(B, H, cuts[-1], d, torch.bfloat16, "sigmoid", False, 83)
    xc, gc = x.cuda(), gate.cuda()
    state = torch.zeros(B, H, d, device="cuda")
    o = [hla2.hla2_gated_scan(xc[:, :, a:b], gc[:, :, a:b], state_in=state, state_out=state) for a, b in zip(cuts, cuts[1:])]
    ref = forward64(x, gate, "sigmoid")
    assert rel(torch.cat(o, 2), ref) < F32 and rel(state, ref[:, :, -1], ref.abs().max()) < F32


# ---------------------------------------------------------------- refusals ----
def test_states_that_overlap_are_refused():
    import ctypes
    L = hla2.lib()
    p = lambda a: ctypes.c_void_p(a)
    B, H, T, d = 2, 3, 8, 16
    size = B * H * d * 4
    for off in (4, 16, size - 4, -4, 4 - size):
        assert L.hla2_gated_scan(p(4096), p(4096), None, p(65536), p(4096), p(65536 + off), None, B, H, T, d, None, 0, 0,
                                 0, 0, None, 0, None) == hla2.HLA2_ERR_INVALID
        assert "overlap" in hla2.hla2_last_error_detail()
        assert L.hla2_gated_scan_backward(p(4096), p(4096), None, p(4096), p(4096), p(65536), p(4096), p(4096),
                                          p(65536 + off), B, H, T, d, None, 0, 0, 0, 0, None, 0,
                                          None) == hla2.HLA2_ERR_INVALID
        assert "overlap" in hla2.hla2_last_error_detail()
        assert L.hla2_gated_step(p(65536), p(4096), p(4096), p(4096), p(65536 + off), B * H, d, None, 0, 0, 0, 0,
                                 None) == hla2.HLA2_ERR_INVALID
        assert "overlap" in hla2.hla2_last_error_detail()


def test_sizes_up_to_the_largest_int():
    for T in (1, 63, 64, 65, 128, 129, 1 << 30, 2 ** 31 - 129, 2 ** 31 - 64, 2 ** 31 - 1):
        for d, tile, channels in ((16, 128, 64), (64, 128, 64), (65, 64, 128), (128, 64, 128)):
            tiles = -(-T // tile)
            assert hla2.hla2_gated_scan_carry_len(T, d) == tiles * d
            assert hla2.hla2_gated_scan_workspace(1, 1, T, d) >= (tiles * channels * 8 if tiles > 1 else 0)


def test_no_launch_without_a_status_word():
    """Where the device's status word cannot be had (here: no device at all), the scan and its gradient say so
    before they launch anything that would report through it."""
    import os
    import subprocess
    import sys
    code = """
import ctypes
from higher_order_linear_gb300 import hla2
L = hla2.lib()
p = ctypes.c_void_p(4096)
for T in (8, 1000):
    n = hla2.hla2_gated_scan_workspace(1, 1, T, 16)
    for call in (lambda: L.hla2_gated_scan(p, p, None, None, p, None, None, 1, 1, T, 16, None, 0, 0, 0, 0, p, n, None),
                 lambda: L.hla2_gated_scan_backward(p, p, None, p, p, None, p, p, None, 1, 1, T, 16, None, 0, 0, 0, 0,
                                                    p, n, None)):
        assert call() == hla2.HLA2_ERR_LAUNCH
        assert "status word" in hla2.hla2_last_error_detail(), hla2.hla2_last_error_detail()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), check=True)


def test_binding_refuses():
    x, g = torch.zeros(2, 3, 8, 4), torch.zeros(2, 3, 8, 4)
    f, bw = hla2.hla2_gated_scan, hla2.hla2_gated_scan_backward
    with pytest.raises(ValueError, match="expected X"):
        f(x[0], g)
    with pytest.raises(ValueError, match="expected X"):
        f(x, g[..., :2])
    with pytest.raises(ValueError, match="share a dtype"):
        f(x, g.bfloat16())
    with pytest.raises(ValueError, match="unsupported input dtype"):
        f(x.double(), g.double())
    with pytest.raises(ValueError, match="unknown gate form"):
        f(x, g, form="tanh")
    with pytest.raises(ValueError, match="last dimension"):
        f(x.transpose(2, 3), g.transpose(2, 3))
    with pytest.raises(ValueError, match="reset has shape"):
        f(x, g, reset=torch.zeros(2, 7, dtype=torch.bool))
    with pytest.raises(ValueError, match="bool or uint8"):
        f(x, g, reset=torch.zeros(2, 8))
    with pytest.raises(ValueError, match="state_in has shape"):
        f(x, g, state_in=torch.zeros(2, 3, 5))
    with pytest.raises(ValueError, match="O has shape"):
        f(x, g, O=torch.zeros(2, 3, 8, 5))
    with pytest.raises(ValueError, match="expanded"):
        f(x, g, O=torch.zeros(2, 3, 1, 4).expand(2, 3, 8, 4))
    with pytest.raises(ValueError, match="unsupported output dtype"):
        f(x, g, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="is on meta"):
        f(x, g.to("meta"))
    with pytest.raises(ValueError, match="carry has shape"):
        bw(x, g, x, torch.zeros(2, 3, 1))
    with pytest.raises(ValueError, match="CUDA tensor"):
        f(x, g)
    s = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="state has shape"):
        hla2.hla2_gated_step(s[:2], s, s)
    with pytest.raises(ValueError, match="expected g"):
        hla2.hla2_gated_step(s, s, s[:, :3].contiguous())
    with pytest.raises(ValueError, match="CUDA tensor"):
        hla2.hla2_gated_step(s, s, s)


def test_entry_refuses():
    import ctypes
    L = hla2.lib()
    p = lambda a=4096: ctypes.c_void_p(a)
    INV, UNS, WS = hla2.HLA2_ERR_INVALID, hla2.HLA2_ERR_UNSUPPORTED, hla2.HLA2_ERR_WORKSPACE

    def fwd(x=p(), g=p(), o=p(), B=1, H=1, T=8, d=16, form=0, dtype=0, out=0, ws=None, nws=0):
        return L.hla2_gated_scan(x, g, None, None, o, None, None, B, H, T, d, None, form, 0, dtype, out, ws, nws, None)

    assert fwd(x=None) == INV and fwd(g=None) == INV and fwd(o=None) == INV
    assert fwd(x=p(4098)) == INV
    assert "aligned" in hla2.hla2_last_error_detail()
    for kw in (dict(B=0), dict(H=-1), dict(T=0), dict(d=0)):
        assert fwd(**kw) == INV
    assert fwd(d=129) == UNS and fwd(B=300, H=300) == UNS and fwd(form=2) == UNS and fwd(dtype=5) == UNS and fwd(out=2) == UNS
    need = hla2.hla2_gated_scan_workspace(1, 1, 100000, 128)
    if need:
        assert fwd(T=100000, d=128) == WS and fwd(T=100000, d=128, ws=p(), nws=need - 1) == WS
    assert hla2.hla2_gated_scan_workspace(1, 1, 1, 64) == 0
    assert hla2.hla2_gated_scan_workspace(0, 1, 100000, 64) == 0
    assert L.hla2_gated_scan_backward(p(), p(), None, None, p(), None, p(), p(), None, 1, 1, 8, 16, None, 0, 0, 0, 0,
                                      None, 0, None) == INV
    assert L.hla2_gated_step(None, p(), p(), p(), None, 4, 16, None, 0, 0, 0, 0, None) == INV
    assert L.hla2_gated_step(p(), p(), p(), p(), None, 0, 16, None, 0, 0, 0, 0, None) == INV
    assert L.hla2_gated_step(p(), p(), p(), p(), None, 4, 16, None, 7, 0, 0, 0, None) == UNS
