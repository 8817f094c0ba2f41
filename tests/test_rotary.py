"""Rotary positions with several axes against the turn in 64 bits.

Tolerances, fixed before the first run: the angle is reduced exactly and the
sine and cosine are good to a few units of 2^-24, so fp32 results are within
1e-6 of the pair's length at every position; bf16 results half a unit in the
last place of each value more.
"""
import pytest
import torch

from _rounding import excess
from higher_order_linear_gb300 import hla2

F32 = 1e-6


def freqs(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def turn64(x, pos, freq, sections, interleaved, inverse):
    """x [B,H,T,d], pos [axes,B,T] -> turned, and each channel's pair length, in 64 bits."""
    v = x.double()
    pairs = freq.numel()
    axis = torch.cat([torch.full((n,), i, dtype=torch.int64) for i, n in enumerate(sections)])
    ang = pos.double()[axis].permute(1, 2, 0) * freq.double()  # [B,T,pairs]
    co, si = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if inverse:
        si = -si
    out, size = v.clone(), v.abs()
    ia = torch.arange(pairs) * 2 if interleaved else torch.arange(pairs)
    ib = ia + 1 if interleaved else ia + pairs
    a, b = v[..., ia], v[..., ib]
    out[..., ia] = a * co - b * si
    out[..., ib] = a * si + b * co
    size[..., ia] = size[..., ib] = (a * a + b * b).sqrt()
    return out, size


def check(B, H, HK, T, d, rot, sections, dtype, interleaved, inverse, layout="bhtd", start=0, seed=0, inplace=False):
    g = torch.Generator().manual_seed(seed)

    def heads(n):
        if layout == "bthd":
            return torch.randn(B, T, n, d, generator=g).to(dtype).transpose(1, 2)
        return torch.randn(B, n, T, d, generator=g).to(dtype)

    q, k = heads(H), heads(HK) if HK else None
    axes = len(sections)
    pos = torch.randint(0, 100, (axes, B, T), generator=g, dtype=torch.int32) + start
    freq = freqs(rot // 2)
    qc, kc = q.cuda(), None if k is None else k.cuda()
    kw = dict(OQ=qc, OK=kc) if inplace else {}
    oq, ok = hla2.hla2_rotary(qc, pos.cuda(), freq.cuda(), sections, K=kc, interleaved=interleaved, inverse=inverse, **kw)
    for got, x in ((oq, q), (ok, k)):
        if x is None:
            assert got is None
            continue
        ref, size = turn64(x, pos, freq, sections, interleaved, inverse)
        assert got.dtype == dtype and got.shape == x.shape
        assert (excess(got, ref, F32 * size) <= F32 * size + 1e-30).all()
        if rot < d:
            assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,sections", [(2, 2, (1,)), (16, 16, (3, 5)), (24, 8, (1, 1, 2)), (33, 32, (16,)),
                                            (64, 64, (16, 8, 8)), (80, 72, (18, 18)), (96, 96, (16, 16, 8, 8)),
                                            (127, 6, (2, 1)), (128, 120, (20, 20, 20)), (128, 128, (64,)),
                                            (128, 128, (22, 21, 21)), (128, 64, (32,))])
def test_sizes(dtype, interleaved, d, rot, sections):
    check(2, 3, 1, 37, d, rot, sections, dtype, interleaved, False)
    check(1, 5, 0, 130, d, rot, sections, dtype, interleaved, True, "bthd")
    check(1, 2, 7, 5, d, rot, sections, dtype, interleaved, False, "bthd", inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,HK,T", [(1, 1, 0, 1), (256, 16, 4, 1), (1, 33, 2, 1), (3, 16, 16, 700), (1, 1, 1, 5000)])
def test_shapes(B, H, HK, T):
    for dtype in (torch.float32, torch.bfloat16):
        check(B, H, HK, T, 128, 128, (24, 20, 20), dtype, False, False, "bthd")
        check(B, H, HK, T, 64, 64, (32,), dtype, True, True)


@pytest.mark.gpu
@pytest.mark.parametrize("start", [0, -100, 65536, (1 << 24) - 50, (1 << 24) + 3, (1 << 31) - 200, -(1 << 31)])
def test_far_positions(start):
    """The angle keeps its precision at every position an int32 can hold."""
    check(2, 2, 1, 50, 64, 64, (20, 12), torch.float32, False, False, start=start)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 7.0, 300.0, 1e4, 1e6, 1e9])
@pytest.mark.parametrize("start", [0, 5000, 1 << 20, (1 << 23) - 25, (1 << 24) - 25, (1 << 31) - 50, -(1 << 31)])
def test_large_frequencies(scale, start):
    """Frequencies above 1: angles of up to 3e18 radians, reduced in whole numbers (1 / 2 pi to 60
    digits); the bound of every other position."""
    from fractions import Fraction
    inv = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)
    T, pairs = 20, 8
    g = torch.Generator().manual_seed(9)
    x = torch.randn(1, 1, T, 2 * pairs, generator=g)
    f = (scale * (0.5 + torch.rand(pairs, generator=g))).float()
    pos = (torch.arange(T, dtype=torch.int64) + start).to(torch.int32)
    out, _ = hla2.hla2_rotary(x.cuda(), pos.view(1, 1, T).cuda(), f.cuda(), (pairs,))
    turns = [[float((Fraction(int(p)) * Fraction(float(v)) * inv) % 1) for v in f] for p in pos]
    ang = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64)
    a, b = x.double()[0, 0, :, :pairs], x.double()[0, 0, :, pairs:]
    ref = torch.cat([a * torch.cos(ang) - b * torch.sin(ang), a * torch.sin(ang) + b * torch.cos(ang)], -1)
    size = (a * a + b * b).sqrt().repeat(1, 2)
    assert ((out.double().cpu()[0, 0] - ref).abs() <= F32 * size).all()


@pytest.mark.gpu
def test_inverse_undoes_the_turn_and_shared_positions():
    g = torch.Generator().manual_seed(5)
    q = torch.randn(2, 4, 60, 128, generator=g).cuda()
    pos = torch.arange(60, dtype=torch.int32)[None].cuda()  # [axes, T]: the same for both sequences
    f = freqs(64).cuda()
    a, _ = hla2.hla2_rotary(q, pos, f, (64,))
    b, _ = hla2.hla2_rotary(a, pos, f, (64,), inverse=True)
    assert float((b - q).abs().max()) < 4e-6 * float(q.abs().max())
    two = pos[:, None].expand(1, 2, 60)
    c, _ = hla2.hla2_rotary(q, two, f, (64,))
    assert torch.equal(a, c)


@pytest.mark.gpu
def test_gradient_against_differences():
    """The turn is linear: <dO, turn(x)> changes by <inverse turn(dO), dx>."""
    g = torch.Generator().manual_seed(6)
    x, do, dx = (torch.randn(1, 2, 9, 16, generator=g) for _ in range(3))
    pos = torch.randint(0, 50, (2, 1, 9), generator=g, dtype=torch.int32)
    f = freqs(8)
    grad, _ = hla2.hla2_rotary(do.cuda(), pos.cuda(), f.cuda(), (5, 3), inverse=True)
    loss = lambda v: float((turn64(v, pos, f, (5, 3), False, False)[0] * do.double()).sum())
    num = (loss(x.double() + 1e-3 * dx.double()) - loss(x.double() - 1e-3 * dx.double())) / 2e-3
    assert abs(num - float((grad.double().cpu() * dx.double()).sum())) < 1e-5 * float((grad.cpu().abs() * dx.abs()).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_slices_and_gaps(dtype):
    """Queries and keys as slices of one projection, odd offsets; an output's gaps stay untouched."""
    B, T, H, d = 2, 33, 3, 32
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(0, 1000, (1, B, T), generator=g, dtype=torch.int32)
    f = freqs(16)
    for off, width in ((0, 64), (1, 67), (4, 72), (8, 80)):
        wide = torch.randn(B, T, H, width, generator=g).to(dtype)
        full = torch.full((B, T, H, width), 5.0, dtype=dtype, device="cuda")
        x = wide.cuda()[..., off:off + d].transpose(1, 2)
        o = full[..., off:off + d].transpose(1, 2)
        hla2.hla2_rotary(x, pos.cuda(), f.cuda(), (16,), OQ=o)
        ref, size = turn64(x.cpu(), pos, f, (16,), False, False)
        assert (excess(o, ref, F32 * size) <= F32 * size + 1e-30).all()
        assert (full[..., :off] == 5).all() and (full[..., off + d:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,step", [(8, 16, 1), (40, 64, 1), (300, 16, 4)])
def test_overlapping_inputs(T, d, step):
    """Sliding windows as inputs: elements that are in several places, strides that leave no order of their own."""
    base = torch.randn(3, (T - 1) * step + d, generator=torch.Generator().manual_seed(10))
    strides = (0, base.stride(0), step, 1)
    q, k = base.as_strided((1, 2, T, d), strides), base.as_strided((1, 2, T, d), strides, base.stride(0))
    dev = base.cuda()
    pos = torch.arange(T, dtype=torch.int32).view(1, 1, T)
    f = freqs(d // 2)
    oq, ok = hla2.hla2_rotary(dev.as_strided((1, 2, T, d), strides), pos.cuda(), f.cuda(), (d // 2,),
                              K=dev.as_strided((1, 2, T, d), strides, dev.stride(0)))
    for got, x in ((oq, q), (ok, k)):
        ref, size = turn64(x, pos, f, (d // 2,), False, False)
        assert (excess(got, ref, F32 * size) <= F32 * size + 1e-30).all()


@pytest.mark.gpu
def test_offsets_beyond_32_bits_and_streams():
    T, ld, d = 70000, 32768, 16
    base = torch.empty((T, ld), device="cuda", dtype=torch.bfloat16)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    base[:, :d] = x.cuda()
    pos = torch.arange(T, dtype=torch.int32)[None]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, _ = hla2.hla2_rotary(base[None, None, :, :d], pos.cuda(), freqs(8).cuda(), (8,), OQ=base[None, None, :, 64:64 + d],
                            stream=s)
    s.synchronize()
    ref, size = turn64(x[None, None], pos[:, None], freqs(8), (8,), False, False)
    assert (excess(o, ref, F32 * size) <= F32 * size + 1e-30).all()


@pytest.mark.gpu
def test_graph_replays_on_new_values():
    """A graph of single tokens, as a decoding loop would keep it, on positions and values changed in place."""
    g = torch.Generator().manual_seed(12)
    q, k = torch.randn(8, 1, 16, 64, generator=g).cuda().transpose(1, 2), torch.randn(8, 1, 4, 64, generator=g).cuda().transpose(1, 2)
    pos, f = torch.zeros(3, 8, 1, dtype=torch.int32, device="cuda"), freqs(32).cuda()
    call = lambda: hla2.hla2_rotary(q, pos, f, (12, 10, 10), K=k)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for step in range(3):
        pos.copy_(torch.randint(0, 5000, pos.shape, generator=g, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, generator=g))
        k.copy_(torch.randn(k.shape, generator=g))
        graph.replay()
        for a, b in zip(held, call()):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals ----
def test_binding_refuses():
    q, pos, f = torch.zeros(2, 3, 5, 8), torch.zeros(1, 2, 5, dtype=torch.int32), torch.zeros(4)
    r = hla2.hla2_rotary
    with pytest.raises(ValueError, match="expected Q"):
        r(q[0], pos, f, (4,))
    with pytest.raises(ValueError, match="pos must be"):
        r(q, pos.long(), f, (4,))
    with pytest.raises(ValueError, match="pos has shape"):
        r(q, pos, f, (2, 2))
    with pytest.raises(ValueError, match="one frequency"):
        r(q, pos, f, (3,))
    with pytest.raises(ValueError, match="expected K"):
        r(q, pos, f, (4,), K=torch.zeros(2, 3, 6, 8))
    with pytest.raises(ValueError, match="K must be"):
        r(q, pos, f, (4,), K=q.bfloat16())
    with pytest.raises(ValueError, match="OK without K"):
        r(q, pos, f, (4,), OK=q)
    with pytest.raises(ValueError, match="OQ has shape"):
        r(q, pos, f, (4,), OQ=q[..., :4])
    with pytest.raises(ValueError, match="last dimension"):
        r(q.transpose(2, 3), pos, f, (4,))
    with pytest.raises(ValueError, match="unsupported input dtype"):
        r(q.half(), pos, f, (4,))
    with pytest.raises(ValueError, match="CUDA tensor"):
        r(q, pos, f, (4,))


def test_entry_refuses():
    import ctypes
    L = hla2.lib()
    p = lambda a=4096: ctypes.c_void_p(a)
    INV, UNS = hla2.HLA2_ERR_INVALID, hla2.HLA2_ERR_UNSUPPORTED

    def call(q=p(), oq=p(), k=None, ok=None, pos=p(), f=p(), B=1, H=1, HK=0, T=4, d=8, rot=8, sec=(4,), dtype=0, naxes=None):
        return L.hla2_rotary(q, oq, k, ok, pos, f, B, H, HK, T, d, rot, len(sec) if naxes is None else naxes,
                             (ctypes.c_int * len(sec))(*sec), 0, 0, None, dtype, None)

    for kw in (dict(q=None), dict(oq=None), dict(pos=None), dict(f=None), dict(B=0), dict(T=0), dict(H=0), dict(d=0),
               dict(HK=2), dict(k=p(), ok=p()), dict(rot=7), dict(rot=10), dict(rot=0), dict(sec=(3,)), dict(sec=(5, -1)),
               dict(naxes=0), dict(sec=(1, 1, 1, 1, 0)), dict(q=p(4098))):
        assert call(**kw) == INV, kw
    assert call(d=130, rot=8) == UNS and call(dtype=4) == UNS and call(B=300, H=300) == UNS
