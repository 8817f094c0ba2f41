"""Root-mean-square norm with the residual's addition, its 8-bit output and its
gradient, against the formulas in 64 bits.

Tolerances, fixed before the first run: fp32 results carry the rounding of a
sum of up to 16384 squares in pieces (below 2e-6 relative) and a few roundings
more: 5e-6 of the row's largest value; bf16 results half a unit in the last
place of each value more; the 8-bit values stand within half a step of e4m3 (2^-4
of the value, or half its smallest subnormal, 2^-10, both times the scale).
dW sums rows of terms rounded to fp32: 1e-5 of the largest column sum of
magnitudes.
"""
import pytest
import torch

from _rounding import excess
from higher_order_linear_gb300 import hla2

F32 = 5e-6


def make(rows, C, dtype, residual, seed=0):
    g = torch.Generator().manual_seed(seed)
    level = torch.exp(torch.randn(rows, 1, generator=g))
    x = (torch.randn(rows, C, generator=g) * level).to(dtype)
    r = torch.randn(rows, C, generator=g).to(dtype) if residual else None
    w = (1 + 0.2 * torch.randn(C, generator=g))
    return x, r, w


def norm64(x, r, w, eps=1e-6):
    t = x.double() + (r.double() if r is not None else 0)
    y = t / (t.square().mean(-1, keepdim=True) + eps).sqrt()
    return t, y * w.double() if w is not None else y


def close(got, ref, rtol):
    """Each row against its largest value."""
    assert torch.isfinite(got).all()
    top = ref.abs().amax(-1, keepdim=True)
    assert (excess(got, ref, rtol * top) <= rtol * top + 1e-300).all()


SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (9, 63), (33, 64), (17, 65), (40, 128), (7, 200), (6, 256), (5, 511),
         (4, 512), (3, 1000), (5, 1024), (2, 1032), (3, 2048), (2, 2050), (2, 4096), (1, 5000), (2, 8192), (1, 9001),
         (2, 16384), (1, 16383)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward(rows, C, dtype):
    for residual in (False, True):
        x, r, w = make(rows, C, dtype, residual)
        t, ref = norm64(x, r, w.to(dtype))
        for out in (torch.float32, torch.bfloat16):
            y, s = hla2.hla2_rmsnorm(x.cuda(), w.to(dtype).cuda(), residual=None if r is None else r.cuda(), out_dtype=out)
            close(y, ref, F32)
            if residual:
                assert torch.equal(s.cpu(), (x.float() + r.float()).to(dtype))
            else:
                assert s is None
    x, r, w = make(rows, C, dtype, True, 5)
    y, _ = hla2.hla2_rmsnorm(x.cuda(), None, residual=r.cuda())
    close(y, norm64(x, r, None)[1], F32)
    y, _ = hla2.hla2_rmsnorm(x.cuda(), w.cuda())  # an fp32 weight with either input
    close(y, norm64(x, None, w)[1], F32)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_q8(rows, C, dtype):
    for residual in (False, True):
        x, r, w = make(rows, C, dtype, residual, 3)
        t, ref = norm64(x, r, w.to(dtype))
        q, scale, s = hla2.hla2_rmsnorm_q8(x.cuda(), w.to(dtype).cuda(), residual=None if r is None else r.cuda())
        assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and scale.shape == x.shape[:-1]
        top = ref.abs().amax(-1)
        assert ((scale.double().cpu() - top / 448).abs() <= 1e-5 * top / 448).all()
        back = q.float().double().cpu() * scale.double().cpu()[:, None]
        step = torch.maximum(ref.abs() * 2.0 ** -4, scale.double().cpu()[:, None] * 2.0 ** -10)
        assert ((back - ref).abs() <= step * (1 + 1e-4) + 1e-5 * top[:, None]).all()
        if residual:
            assert torch.equal(s.cpu(), (x.float() + r.float()).to(dtype))


@pytest.mark.gpu
def test_q8_special_rows():
    """Zero rows, tiny rows, rows with inf and NaN."""
    C = 256
    x = torch.randn(7, C, generator=torch.Generator().manual_seed(9))
    x[0] = 0
    x[1] = 0
    x[1, 5] = 1e-30
    x[2] *= 1e-20
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5] = 1e-42
    q, scale, _ = hla2.hla2_rmsnorm_q8(x.cuda())
    q, scale = q.float().cpu(), scale.cpu()
    assert (q[0] == 0).all() and scale[0] == 1
    assert q[1, 5] == 448 and (q[1].abs().sum() == 448)
    assert torch.isfinite(q[2]).all() and q[2].abs().max() == 448
    assert torch.isnan(q[3, 7]) and not torch.isfinite(scale[3])
    assert torch.isnan(q[4]).all() and torch.isnan(scale[4])
    assert torch.isfinite(q[5]).all()
    assert q[6].abs().max() == 448 and torch.isfinite(scale[6])
    y, _ = hla2.hla2_rmsnorm(x.cuda())
    y = y.cpu()
    assert (y[0] == 0).all() and torch.isfinite(y[[0, 1, 2, 5, 6]]).all() and torch.isnan(y[4]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", [(400, 64), (300, 100), (200, 127), (90, 1000), (60, 2048), (40, 8192), (15, 16384), (11, 9001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_q8_codes_are_those_of_the_exact_quotient(rows, C, dtype):
    """Q = e4m3(y / scale) = e4m3(448 t w / max|t w|), ties to even.  t and w of 8 bits make t w a number of 16
    bits and 448 t w one of 19: either the quotient stands between two codes exactly, or it is 2^-21 of itself
    and more from there, which fp32 tells.  So every code is the definition's."""
    g = torch.Generator().manual_seed(33)
    for by in (1.0, 2.0 ** -50, 2.0 ** 50, 2.0 ** -104, 2.0 ** 105):
        x = (torch.randn(rows, C, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(torch.bfloat16) * by
        w = (1 + 0.1 * torch.randn(C, generator=g)).to(torch.bfloat16)
        q, scale, _ = hla2.hla2_rmsnorm_q8(x.to(dtype).cuda(), w.to(dtype).cuda())
        tw = x.double() * w.double()
        top = tw.abs().amax(-1, keepdim=True)
        ref = (448 * tw / top).float().to(torch.float8_e4m3fn)
        assert torch.equal(q.cpu().float(), ref.float())


@pytest.mark.gpu
def test_q8_of_rows_whose_scale_leaves_the_range():
    """A scale that underflows, a row of zeros without eps: no NaN, and Q * scale is the row's (zero) value."""
    C = 96
    x = torch.zeros(3, C)
    x[0, ::2] = 1e-45
    x[1, ::3] = -3e-44
    q, scale, _ = hla2.hla2_rmsnorm_q8(x.cuda(), eps=1.0)
    q, scale = q.float().cpu(), scale.cpu()
    assert torch.isfinite(q).all() and (q[x == 0] == 0).all() and (scale >= 0).all() and (scale[:2] < 1e-45).all()
    assert scale[2] == 1
    q, scale, _ = hla2.hla2_rmsnorm_q8(x[2:].cuda(), eps=0.0)
    assert (q.float() == 0).all() and (scale == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SIZES + [(3000, 64), (2500, 128), (1500, 1024), (700, 2048), (400, 4096), (300, 8192)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(rows, C, dtype):
    g = torch.Generator().manual_seed(13)
    for residual in (False, True):
        t, ds, w = make(rows, C, dtype, residual, 13)
        wd = w.to(dtype)
        for ydt in {dtype, torch.float32}:
            dy = torch.randn(rows, C, generator=g).to(ydt)
            dx, dw = hla2.hla2_rmsnorm_backward(t.cuda(), dy.cuda(), wd.cuda(), dS=None if ds is None else ds.cuda())
            td, yd = t.double(), dy.double()
            rstd = 1 / (td.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            n, gw = td * rstd, yd * wd.double()
            ref = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
            size = rstd * (gw.abs().amax(-1, keepdim=True) + n.abs().amax(-1, keepdim=True) * (gw * n).abs().mean(-1, keepdim=True))
            if ds is not None:
                ref, size = ref + ds.double(), size + ds.double().abs().amax(-1, keepdim=True)
            assert (excess(dx, ref, F32 * size) <= F32 * size).all()
            terms = yd * n
            assert ((dw.double().cpu() - terms.sum(0)).abs() <= 1e-5 * terms.abs().sum(0).max()).all()
            dx2, dw2 = hla2.hla2_rmsnorm_backward(t.cuda(), dy.cuda(), wd.cuda(), dS=None if ds is None else ds.cuda())
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx, dw = hla2.hla2_rmsnorm_backward(t.cuda(), dy.cuda())
    assert dw is None


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 256, 1000, 2048, 12288])
@pytest.mark.parametrize("size,eps", [(1e14, 1e-6), (1e15, 1e-6), (1e16, 1e-6), (1e17, 1e-6), (1e-9, 0.0), (1e-13, 0.0),
                                      (1e-16, 0.0), (1e15, 0.0), (1e-3, 1e-6), (1e-13, 1e-12)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_large_and_small_rows(C, size, eps, dtype):
    """The bounds of test_backward, at sizes where a power of the rows' reciprocal root leaves fp32's range."""
    rows = 9
    g = torch.Generator().manual_seed(14)
    t = (torch.randn(rows, C, generator=g) * size).to(dtype)
    w = (1 + 0.2 * torch.randn(C, generator=g)).to(dtype)
    # a gradient along the row itself, where the projection takes most of it away, and one across it
    for dy in (torch.randn(rows, C, generator=g).to(dtype), (t.double() / size).to(dtype)):
        dx, dw = hla2.hla2_rmsnorm_backward(t.cuda(), dy.cuda(), w.cuda(), eps=eps)
        td, yd = t.double(), dy.double()
        rstd = 1 / (td.square().mean(-1, keepdim=True) + eps).sqrt()
        n, gw = td * rstd, yd * w.double()
        ref = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
        top = rstd * (gw.abs().amax(-1, keepdim=True) + n.abs().amax(-1, keepdim=True) * (gw * n).abs().mean(-1, keepdim=True))
        assert torch.isfinite(dx).all() and (excess(dx, ref, F32 * top) <= F32 * top).all()
        terms = yd * n
        assert ((dw.double().cpu() - terms.sum(0)).abs() <= 1e-5 * terms.abs().sum(0).max()).all()


@pytest.mark.gpu
def test_gradient_against_differences():
    """Central differences of the 64-bit norm (their own error is about 1e-8)."""
    rows, C, eps = 2, 6, 1e-4
    t, _, w = make(rows, C, torch.float32, False, 17)
    dy = torch.randn(rows, C, generator=torch.Generator().manual_seed(18))
    dx, dw = hla2.hla2_rmsnorm_backward(t.cuda(), dy.cuda(), w.cuda())
    loss = lambda t, w: float((norm64(t, None, w)[1] * dy.double()).sum())
    for got, at in ((dx, 0), (dw, 1)):
        flat = got.double().cpu().reshape(-1)
        for i in range(flat.numel()):
            vals = []
            for sgn in (1, -1):
                m = [t.double(), w.double()]
                m[at] = m[at].clone()
                m[at].view(-1)[i] += sgn * eps
                vals.append(loss(*m))
            assert abs((vals[0] - vals[1]) / (2 * eps) - float(flat[i])) < 1e-5 * max(1.0, float(flat.abs().max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_in_place(dtype):
    """Column slices with odd offsets; leading dimensions; the residual stream updated in place; gaps untouched."""
    rows, C = 37, 96
    gen = torch.Generator().manual_seed(23)
    for off, width in ((0, 128), (3, 101), (8, 104)):
        wide = torch.randn(rows, width, generator=gen).to(dtype).cuda()
        x = wide[:, off:off + C]
        r = torch.randn(rows, C, generator=gen).to(dtype).cuda()
        ref_t, ref = norm64(x.cpu(), r.cpu(), None)
        full = torch.full((rows, width), 3.0, device="cuda", dtype=dtype)
        y, s = hla2.hla2_rmsnorm(x, residual=r, Y=full[:, off:off + C], S=r)
        assert s is r
        close(y, ref, F32)
        assert torch.equal(r, ref_t.to(dtype).cuda()) or dtype == torch.float32
        assert (full[:, :off] == 3).all() and (full[:, off + C:] == 3).all()
        fq = torch.zeros((rows, width), device="cuda", dtype=torch.uint8).fill_(0x11).view(torch.float8_e4m3fn)
        q, scale, _ = hla2.hla2_rmsnorm_q8(x, Q=fq[:, off:off + C])
        assert (fq.view(torch.uint8)[:, :off] == 0x11).all() and (fq.view(torch.uint8)[:, off + C:] == 0x11).all()
        ref8 = norm64(x.cpu(), None, None)[1]
        back = q.float().double().cpu() * scale.double().cpu()[:, None]
        assert ((back - ref8).abs() <= ref8.abs() * 0.0626 + scale.double().cpu()[:, None] * 2.0 ** -9).all()
    x = torch.randn(2, 3, 5, 64, generator=gen).to(dtype).cuda()
    y, _ = hla2.hla2_rmsnorm(x)
    close(y, norm64(x.cpu(), None, None)[1], F32)


@pytest.mark.gpu
def test_offsets_beyond_32_bits_and_streams():
    rows, ld, C = 70000, 32768, 64
    base = torch.empty((rows, ld), device="cuda", dtype=torch.bfloat16)
    x = torch.randn(rows, C, generator=torch.Generator().manual_seed(29)).to(torch.bfloat16)
    base[:, :C] = x.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = hla2.hla2_rmsnorm(base[:, :C], Y=base[:, 64:64 + C], stream=s)
    s.synchronize()
    close(y, norm64(x, None, None)[1], F32)


@pytest.mark.gpu
def test_graph_replays_on_new_values():
    """A graph of the norms, as a decoding loop would keep it, on inputs changed in place."""
    rows, C = 16, 512
    g = torch.Generator().manual_seed(31)
    sets = [[torch.randn(rows, C, generator=g).to(torch.bfloat16).cuda() for _ in range(3)] for _ in range(3)]
    x, r, dy = (t.clone() for t in sets[0])
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(torch.bfloat16).cuda()
    calls = lambda: (*hla2.hla2_rmsnorm(x, w, residual=r), *hla2.hla2_rmsnorm_q8(x, w, residual=r),
                     *hla2.hla2_rmsnorm_backward(x, dy, w, dS=r))
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for s in sets:
        for to, value in zip((x, r, dy), s):
            to.copy_(value)
        graph.replay()
        for a, b in zip(held, calls()):
            assert torch.equal(a.float(), b.float())


# ---------------------------------------------------------------- refusals ----
def test_binding_refuses():
    x = torch.zeros(4, 8)
    f = hla2.hla2_rmsnorm
    with pytest.raises(ValueError, match="unsupported input dtype"):
        f(x.double())
    with pytest.raises(ValueError, match="weight has shape"):
        f(x, torch.zeros(7))
    with pytest.raises(ValueError, match="residual has shape"):
        f(x, residual=torch.zeros(4, 7))
    with pytest.raises(ValueError, match="residual must be"):
        f(x, residual=torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="one stride"):
        f(torch.zeros(4, 6, 8)[:, :3])
    with pytest.raises(ValueError, match="last dimension"):
        f(torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="overlap"):
        f(torch.zeros(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="unsupported output dtype"):
        f(x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="eps"):
        f(x, eps=-1.0)
    with pytest.raises(ValueError, match="is on meta"):
        f(x, torch.zeros(8, device="meta"))
    with pytest.raises(ValueError, match="Q must be"):
        hla2.hla2_rmsnorm_q8(x, Q=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="dY has shape"):
        hla2.hla2_rmsnorm_backward(x, torch.zeros(4, 9))
    for call in (lambda: f(x), lambda: hla2.hla2_rmsnorm_q8(x), lambda: hla2.hla2_rmsnorm_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_entry_refuses():
    import ctypes
    L = hla2.lib()
    p = lambda a=4096: ctypes.c_void_p(a)
    INV, UNS, WS = hla2.HLA2_ERR_INVALID, hla2.HLA2_ERR_UNSUPPORTED, hla2.HLA2_ERR_WORKSPACE

    def fwd(x=p(), y=p(), rows=4, C=8, ld=8, eps=1e-6, dtype=0, out=0, w=None, wdtype=0):
        return L.hla2_rmsnorm(x, None, w, None, y, rows, C, ld, 0, 0, ld, eps, dtype, wdtype, out, None)

    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(rows=0) == INV and fwd(C=0) == INV and fwd(ld=7) == INV
    assert fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV and fwd(x=p(4097)) == INV
    assert fwd(C=16385, ld=16385) == UNS and fwd(dtype=9) == UNS and fwd(out=2) == UNS and fwd(w=p(), wdtype=3) == UNS
    assert fwd(rows=1 << 31) == UNS
    assert L.hla2_rmsnorm_q8(p(), None, None, None, p(), None, 4, 8, 8, 0, 0, 8, 1e-6, 0, 0, None) == INV
    need = L.hla2_rmsnorm_backward_workspace(100, 64)
    assert need > 0 and L.hla2_rmsnorm_backward_workspace(0, 64) == 0

    def bwd(ws=p(), nws=need, t=p()):
        return L.hla2_rmsnorm_backward(t, p(), None, None, p(), p(), 100, 64, None, 1e-6, 0, 0, 0, ws, nws, None)

    assert bwd(ws=None) == WS and bwd(nws=16) == WS and bwd(t=None) == INV and bwd(ws=p(4100)) == INV
