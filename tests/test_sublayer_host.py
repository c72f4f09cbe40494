"""FeedForwardSublayer's refusals: before anything is launched."""
import pytest
import torch

from tests._harness import built_library


@pytest.fixture
def sub(monkeypatch):
    built_library()
    from latent_mixture_experts_gb300 import FeedForwardSublayer, GatedFFN, LatentMoE, sublayer

    def launched(*a, **kw):
        raise AssertionError("launched")
    for name in ("lmoe_add_rms_norm", "lmoe_add_rms_norm_backward"):
        monkeypatch.setattr(sublayer, name, launched)

    def make(kind):
        block = (LatentMoE if kind == "moe" else GatedFFN).__new__(LatentMoE if kind == "moe" else GatedFFN)
        block._h = None
        if kind != "moe":
            block.training, block.mx = False, kind == "mxfp8"
        return FeedForwardSublayer(torch.ones(64, dtype=torch.bfloat16), block)
    return make


@pytest.mark.parametrize("kind", ["moe", "bf16", "mxfp8"])
def test_blocks_that_do_not_train_are_refused(sub, kind):
    s = sub(kind)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="training=True"):
        s.forward_train(x, x)
    with pytest.raises(ValueError, match="training=True"):
        s.backward(x, None, None)
