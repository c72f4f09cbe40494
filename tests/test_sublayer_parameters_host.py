"""What a sublayer hands to an optimizer: bf16 weights, and no code tensors."""
import pytest
import torch

from tests._harness import built_library

BF = torch.bfloat16


def _block(mx):
    from latent_mixture_experts_gb300 import GatedFFN
    block = GatedFFN.__new__(GatedFFN)
    block._h, block.mx, block.training = None, mx, not mx
    block._weights = {n: torch.zeros(64, 64, dtype=torch.uint8 if mx else BF) for n in ("gate", "up", "down")}
    return block


@pytest.mark.parametrize("gated", [False, True])
def test_codes_are_no_parameters(gated):
    built_library()
    from latent_mixture_experts_gb300 import FeedForwardSublayer, GatedSublayer
    w = torch.ones(64, dtype=BF)

    def make(mx):
        return GatedSublayer(_block(mx), w, w, res_gate=w) if gated else FeedForwardSublayer(w, _block(mx))
    with pytest.raises(ValueError, match="bf16"):
        make(True).parameters()
    sub = make(False)
    assert [p is w for p in sub.parameters()] == [True] * (3 if gated else 1) + [False] * 3
    assert all(p.dtype is BF for p in sub.parameters())
