"""The example's limits (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


def test_more_tokens_than_positions_are_refused():
    from serving_gdn_decode_gb300 import hybrid_step
    model = hybrid_step.Model(hybrid_step.Config(width=64, vocab=32, max_tokens=40), device="cpu")
    prompts = torch.zeros(2, 30, dtype=torch.int64)
    with pytest.raises(ValueError, match="41 tokens per request, but the model has 40 positions"):
        hybrid_step.generate(model, prompts, 11)
