"""The example's choice of caches (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


def test_unknown_caches_are_refused():
    from serving_gdn_decode_gb300 import hybrid_step
    model = hybrid_step.Model(hybrid_step.Config(width=64, vocab=32, cache="fp4"), device="cpu")
    with pytest.raises(ValueError, match="no cache of 'fp4'"):
        hybrid_step.Server(model, 1, 2, 3)
