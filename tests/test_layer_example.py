"""The example layer (examples/layer.py): decoding continues a prefill, and the
gradients of its gated branch are those of the formulas.

Tolerances, fixed before the first run.  Decoding against prefill: the prefill's
HLA outputs and state carry 5e-3 of their largest value (its tensor-core bound);
the head norm divides by a head's root mean square, a few times smaller than its
largest value, and two 16-bit roundings (2^-8 each) follow: 3e-2 of the largest
output.  Gradients: three 16-bit roundings on the way (y, dy and the result),
each 2^-8 of its value: 2e-2 of the largest gradient.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,width,heads,d", [(2, 300, 256, 4, 64), (1, 129, 192, 2, 64), (3, 1, 64, 1, 64)])
def test_decoding_continues_a_prefill(B, T, width, heads, d):
    import layer
    assert layer.run(B, T, 4, width, heads, d) < 3e-2


@pytest.mark.gpu
def test_gradients_of_the_gated_branch():
    import layer
    B, H, T, d = 2, 4, 150, 64
    lay = layer.Layer()
    g = torch.Generator().manual_seed(3)
    o = torch.randn(B, H, T, d, generator=g)
    gate = (2 + torch.randn(B, H, T, d, generator=g)).to(torch.bfloat16)
    dh = torch.randn(B, H, T, d, generator=g).to(torch.bfloat16)
    reset = torch.rand(B, T, generator=g) < 0.03
    do, dgate, dnorm = lay.gated_branch_gradients(o.cuda(), gate.cuda(), dh.cuda(), reset.cuda())
    od, gd = o.double().requires_grad_(), gate.double().requires_grad_()
    wd = lay.head_norm.cpu().double().requires_grad_()
    y = od / (od.square().mean(-1, keepdim=True) + 1e-6).sqrt() * wd
    a = torch.sigmoid(gd)
    h, hs = torch.zeros(B, H, d, dtype=torch.float64), []
    for t in range(T):
        h = torch.where(reset[:, t, None, None], torch.zeros((), dtype=torch.float64), h)
        h = a[:, :, t] * h + (1 - a[:, :, t]) * y[:, :, t]
        hs.append(h)
    (torch.stack(hs, 2) * dh.double()).sum().backward()
    for got, ref in ((do, od.grad), (dgate, gd.grad), (dnorm, wd.grad)):
        assert float((got.double().cpu() - ref).abs().max()) < 2e-2 * float(ref.abs().max())
