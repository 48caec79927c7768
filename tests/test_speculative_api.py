"""The speculative step's entry points without a GPU: the rotation table, and every refusal before a launch."""
import ctypes
import math

import numpy as np
import pytest

from decode_attention_qjl_b200 import build as build_mod
from decode_attention_qjl_b200 import qjl as Q


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return Q.load_library()


def test_rope_table_plain_linear_and_by_parts(lib):
    i = np.arange(64)
    f = 10000.0 ** (-2.0 * i / 128)
    t = Q.qjl_rope_init()
    np.testing.assert_allclose(np.array(t.turns), f / (2 * math.pi), rtol=1e-15)
    assert (t.rot_dim, t.layout, t.amplitude) == (128, Q.QJL_ROPE_HALF, 1.0)
    t = Q.qjl_rope_init(rot_dim=64, base=500000.0, interleaved=True, factor=4.0, amplitude=1.5)
    f = 500000.0 ** (-2.0 * i[:32] / 64)
    np.testing.assert_allclose(np.array(t.turns)[:32], f / 4 / (2 * math.pi), rtol=1e-15)
    assert np.all(np.array(t.turns)[32:] == 0) and t.layout == Q.QJL_ROPE_INTERLEAVED and t.amplitude == 1.5
    t = Q.qjl_rope_init(factor=8.0, original_len=8192, low=1.0, high=4.0)
    f = 10000.0 ** (-2.0 * i / 128)
    turns = 8192 * f / (2 * math.pi)
    got = np.array(t.turns) * 2 * math.pi
    np.testing.assert_allclose(got[turns >= 4], f[turns >= 4], rtol=1e-14)      # short wavelengths stay
    np.testing.assert_allclose(got[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)  # long ones are stretched
    between = (turns > 1) & (turns < 4)
    assert between.any() and np.all(got[between] < f[between]) and np.all(got[between] > f[between] / 8)
    assert np.all(np.diff(got) < 0)


def test_rope_init_refusals(lib):
    t = Q.qjl_rope_table()
    ok = [128, 10000.0, 0, 1.0, 0.0, 1.0, 4.0, 1.0]
    assert lib.qjl_rope_init(*ok, ctypes.byref(t)) == 0
    assert lib.qjl_rope_init(*ok, None) == 1
    nan, inf = float("nan"), float("inf")
    for at, bad, want in [(0, 8, 3), (0, 24, 3), (0, 144, 3), (1, 0.0, 1), (1, nan, 1), (1, inf, 1), (2, 2, 1), (3, 0.0, 1),
                          (3, -1.0, 1), (4, -1.0, 1), (4, nan, 1), (7, inf, 1), (7, nan, 1)]:
        a = list(ok)
        a[at] = bad
        assert lib.qjl_rope_init(*a, ctypes.byref(t)) == want, (at, bad)
    assert lib.qjl_rope_init(128, 10000.0, 0, 2.0, 100.0, 4.0, 4.0, 1.0, ctypes.byref(t)) == 1  # low == high


def test_rope_refusals_before_a_launch(lib):
    t = Q.qjl_rope_init()
    buf = (ctypes.c_char * 4096)()
    base = (ctypes.addressof(buf) + 15) & ~15
    hd = lambda **k: (Q.qjl_rope_heads * 2)(*[Q.qjl_rope_heads(  # noqa: E731
        *[{**dict(x=base, y=base + 1024, H=1, x_sb=128, x_sh=128, x_st=128, y_sb=128, y_sh=128, y_st=128), **k}[n]
          for n, _ in Q.qjl_rope_heads._fields_])] * 2)
    call = lambda heads, n=1, dt=0, B=1, T=1, table=t: lib.qjl_rope(ctypes.byref(table), heads, n, dt, B, T, None, None, 0, None)  # noqa: E731,E501
    assert call(hd(), B=0) == 0 and call(hd(), T=0) == 0
    assert lib.qjl_rope(None, hd(), 1, 0, 1, 1, None, None, 0, None) == 1
    assert lib.qjl_rope(ctypes.byref(t), None, 1, 0, 1, 1, None, None, 0, None) == 1
    assert call(hd(), n=3) == 1 and call(hd(), n=0) == 1 and call(hd(), dt=2) == 1
    assert call(hd(), B=-1) == 1 and call(hd(), T=-1) == 1
    assert call(hd(H=0)) == 1 and call(hd(x=0)) == 1 and call(hd(y=base + 8)) == 1
    assert call(hd(x_st=129)) == 1 and call(hd(y_st=-128)) == 1
    assert call(hd(y_st=64), T=2) == 1 and call(hd(y_sh=0, H=2)) == 1 and call(hd(y_sb=0), B=2) == 1
    assert call(hd(y=base, y_st=256)) == 1                       # in place with other strides
    assert call(hd(), table=Q.qjl_rope_table()) == 1             # not filled


def test_refusals_without_a_context(lib):
    c = Q.qjl_cache()
    ref = ctypes.byref(c)
    assert lib.qjl_cache_read(None, ref, 1, None, None, None, 0, 0, 0, None, 0, 0, 0, 0, None) == 1
    assert lib.qjl_tree_attention(None, ref, ref, None, 0, 0, 0, 0, 1, 1, 1, None, None, None, 0.0, None, None, 0, None) == 1
    assert lib.qjl_cache_commit(None, ref, ref, 1, None, None, None, None, None) == 1
    assert lib.qjl_tree_attention_workspace_bytes(None, 1, 1, 1, 1) == 0


def test_draft_cache_shares_the_outlier_channels():
    import torch

    c = Q.QJLCache.allocate(2, 3, 200, 256, 64, 8, device="cpu", value_bits=2)
    d = c.draft()
    assert d.outlier_idx is c.outlier_idx and d.cap == 64 and d.tiles.shape == (2, 3, 1, c.tiles.shape[-1])
    assert (d.m, d.m_out, d.value_bits) == (256, 64, 2) and d.tiles.dtype == torch.uint8
    assert c.draft(65).cap == 128
