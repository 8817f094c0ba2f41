"""A sequence-mixing layer made of this package's operators: prefill, decoding and
one training step of its gated branch.

    x, residual -> norm with the residual's addition, 8 bits and a scale per row
      -> projections to q, k, v and gate logits (plain torch products)
      -> rotary positions (time, height, width) on q and k
      -> masked second-order HLA
      -> norm of each head -> gated recurrence along the tokens -> projection out

Prefill keeps the HLA state and the recurrence's state of every head; decoding
continues from them one token at a time.  Run it on a GPU:

    python examples/layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from higher_order_linear_gb300 import hla2


class Layer:
    def __init__(self, width=256, heads=4, d=64, sections=(12, 10, 10), seed=0, device="cuda"):
        assert 2 * sum(sections) == d
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *shape, scale: (scale * torch.randn(shape, generator=g)).to(device, torch.bfloat16)
        self.H, self.d, self.sections = heads, d, sections
        self.norm = 1 + rnd(width, scale=0.1)
        self.head_norm = 1 + rnd(d, scale=0.1)
        self.w_in = rnd(width, 4 * heads * d, scale=width ** -0.5)
        self.w_out = rnd(heads * d, width, scale=(heads * d) ** -0.5)
        pairs = d // 2
        self.freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(device)

    def project(self, x, residual):
        """[B,T,width] twice -> q, k, v, gate as [B,H,T,d] views of one projection, and the residual stream."""
        B, T, _ = x.shape
        q8, scale, residual = hla2.hla2_rmsnorm_q8(x, self.norm, residual=residual)
        h = (q8.float() * scale[..., None]).to(torch.bfloat16) @ self.w_in
        q, k, v, gate = h.view(B, T, 4, self.H, self.d).permute(2, 0, 3, 1, 4)
        return q, k, v, gate, residual

    def out(self, h, residual):
        """[B,H,T,d] -> the layer's [B,T,width]."""
        B, H, T, d = h.shape
        return h.transpose(1, 2).reshape(B, T, H * d) @ self.w_out, residual

    def prefill(self, x, residual, pos):
        """pos int32 [3,B,T].  Returns the output, the residual stream and the state to decode from."""
        B, T, _ = x.shape
        q, k, v, gate, residual = self.project(x, residual)
        q, k = hla2.hla2_rotary(q, pos, self.freq, self.sections, K=k)
        scale = self.d ** -0.5
        hla = torch.empty(B * self.H, hla2.record_len(self.d, self.d), device=x.device)
        o = hla2.hla2_forward((q * scale).contiguous(), (k * scale).contiguous(), v.contiguous(), state_out=hla)
        y, _ = hla2.hla2_rmsnorm(o, self.head_norm, out_dtype=torch.bfloat16)
        rec = torch.empty(B, self.H, self.d, device=x.device)
        h = hla2.hla2_gated_scan(y, gate, state_out=rec, out_dtype=torch.bfloat16)
        return (*self.out(h, residual), (hla, rec.view(B * self.H, self.d)))

    def step(self, x, residual, pos, state):
        """One token of each sequence: x [B,1,width], pos [3,B,1]; the state is updated in place."""
        hla, rec = state
        n = x.shape[0] * self.H
        q, k, v, gate, residual = self.project(x, residual)
        q, k = hla2.hla2_rotary(q, pos, self.freq, self.sections, K=k)
        scale = self.d ** -0.5
        rows = lambda t: t.reshape(n, self.d)
        o = hla2.hla2_step(hla, rows(q * scale).float(), rows(k * scale).float(), rows(v).float())
        y, _ = hla2.hla2_rmsnorm(o, self.head_norm, out_dtype=torch.bfloat16)
        h = hla2.hla2_gated_step(rec, y, rows(gate), out_dtype=torch.bfloat16)
        return self.out(h.view(x.shape[0], self.H, 1, self.d), residual)

    def gated_branch_gradients(self, o, gate, dh, reset=None):
        """Gradients of head norm + gated recurrence, the layer's part after the attention:
        o [B,H,T,d] fp32, gate and dh [B,H,T,d] bf16 -> (d o, d gate, d head_norm)."""
        B, H, T, d = o.shape
        y, _ = hla2.hla2_rmsnorm(o, self.head_norm, out_dtype=torch.bfloat16)
        carry = torch.empty(B, H, hla2.hla2_gated_scan_carry_len(T, d), device=o.device)
        hla2.hla2_gated_scan(y, gate, reset=reset, carry=carry, out_dtype=torch.bfloat16)
        dy, dgate = hla2.hla2_gated_scan_backward(y, gate, dh, carry, reset=reset)
        do, dnorm = hla2.hla2_rmsnorm_backward(o, dy, self.head_norm)
        return do, dgate, dnorm


def video_positions(B, T, device="cuda"):
    t = torch.arange(T, device=device)
    return torch.stack((t // 64, t // 8 % 8, t % 8)).to(torch.int32)[:, None].expand(3, B, T).contiguous()


def run(B=2, T=300, more=4, width=256, heads=4, d=64, seed=1):
    """Prefill of T tokens and `more` steps against a prefill of all of them: the largest
    difference of the steps' outputs, relative to the largest output."""
    layer = Layer(width, heads, d)
    g = torch.Generator().manual_seed(seed)
    x, residual = (torch.randn((B, T + more, width), generator=g).to("cuda", torch.bfloat16) for _ in range(2))
    pos = video_positions(B, T + more)
    whole, _, _ = layer.prefill(x, residual, pos)
    part = lambda t, a, b: t[:, a:b].contiguous()
    _, _, state = layer.prefill(part(x, 0, T), part(residual, 0, T), pos[:, :, :T].contiguous())
    worst = 0.0
    for t in range(T, T + more):
        y, _ = layer.step(part(x, t, t + 1), part(residual, t, t + 1), pos[:, :, t:t + 1].contiguous(), state)
        worst = max(worst, float((y.float() - whole[:, t:t + 1].float()).abs().max() / whole.float().abs().max()))
    return worst


if __name__ == "__main__":
    print(f"decoding against prefill: {run():.2e} of the largest output")
