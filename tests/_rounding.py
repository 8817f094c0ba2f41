"""What rounding a result to 16 bits may add (tests only)."""
import torch


def half_unit(ref: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Half a unit in the last place of bf16 (8 significant bits) at each value; zero for fp32, whose own
    rounding is part of the tolerance."""
    if dtype != torch.bfloat16:
        return torch.zeros_like(ref)
    return torch.ldexp(torch.ones_like(ref), torch.frexp(ref.abs().clamp(min=2.0 ** -126)).exponent - 9)


def excess(got: torch.Tensor, ref: torch.Tensor, slack) -> torch.Tensor:
    """How far each value is from ``ref`` beyond its own rounding to got's type; ``slack`` is what the value
    may be off before that rounding (it may cross into the next power of two)."""
    g = got.detach().double().cpu()
    return ((g - ref).abs() - half_unit(ref.abs() + slack, got.dtype)).clamp(min=0)
