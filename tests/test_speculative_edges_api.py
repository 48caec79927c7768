"""Refusals of the speculative step's wrappers that need no GPU, at the edges of what a caller may hand in."""
import ctypes

import pytest

from decode_attention_qjl_b200 import build as build_mod
from decode_attention_qjl_b200 import qjl as Q


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return Q.load_library()


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


def test_commit_refuses_lengths_written_over_its_inputs(lib):
    """One block writes seqlens_out while others still read the inputs. (The check needs no context: with none, what
    does not overlap fails later, for the missing context.)"""
    B, A = 4, 3
    ints = (ctypes.c_int32 * 64)()
    at = lambda i: ctypes.addressof(ints) + 4 * i  # noqa: E731
    cache = Q.qjl_cache(None, None, B, 1, 64)
    path, acc, lens, apart = 0, 16, 24, 40

    def message(out, a=A):
        assert lib.qjl_cache_commit(None, ctypes.byref(cache), ctypes.byref(cache), a, at(path), at(acc), at(lens), at(out),
                                    None) == 1
        return lib.qjl_last_error().decode()

    for name, first, n in (("seqlens", lens, B), ("n_accepted", acc, B), ("path", path, A * B)):
        for out in {first, first + n - 1, max(first - B + 1, 0)}:
            assert f"seqlens_out overlaps {name}" in message(out)
    for out in (apart, lens + B, acc + B, path + A * B):
        assert "null context" in message(out)
    assert "null context" in message(path, a=0)  # no path is read
