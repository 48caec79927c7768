"""Refusals of the speculative step's wrappers that need no GPU, at the edges of what a caller may hand in."""
import pytest

from decode_attention_qjl_b200 import qjl as Q


@pytest.mark.parametrize("other", [{"m": 128}, {"m_out": 32}, {"value_bits": 2}])
def test_draft_cache_of_another_layout_is_refused(other):
    """Tiles of another size would be read past their end."""
    import torch

    make = lambda **k: Q.QJLCache.allocate(1, 2, 64, k.get("m", 256), k.get("m_out", 64), 8, device="cpu",  # noqa: E731
                                           value_bits=k.get("value_bits", 4))
    cache, draft = make(), make(**other)
    q = torch.zeros(1, 1, 2, Q.HEAD_DIM, dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="layout"):
        Q.qjl_tree_attention(None, cache, draft, q, 1, torch.zeros_like(q))
    with pytest.raises(ValueError, match="layout"):
        Q.qjl_cache_commit(None, cache, draft, one.view(1, 1), one, one)
