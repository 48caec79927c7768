"""Calls of the speculative step at the edges of its ranges, on the GPU. Bounds and helpers are those of
test_gpu_speculative.py; what a test adds to them is derived beside it."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
from decode_attention_qjl_b200 import qjl as Q  # noqa: E402
from tests import gpu_common as C  # noqa: E402
from tests.test_gpu_speculative import B16, D, H16, U, Case, check_tree, random_tree  # noqa: E402

pytestmark = pytest.mark.gpu


def section(case, cache, name):
    """Writable bytes [B, Hkv, tile, 64, bytes] of a section whose tokens lie in order."""
    off, nb, sec = next((o, n, s) for nm, o, n, s in Q.tile_sections(case.m, case.m_out, value_bits=case.vbits)
                        if nm == name)
    return cache.tiles[..., off:off + sec].unflatten(-1, (64, nb))


def set_value_group(case, cache, token, group, scale, zero):
    x = torch.tensor([scale, zero], dtype=torch.float16, device="cuda").view(torch.uint8)
    section(case, cache, "vsz")[:, :, token // 64, token % 64, 4 * group:4 * group + 4] = x


def check_rows(case, got, mask, seqlens=None, sm_scale=None):
    """check_tree for bf16 queries where channels of one row differ by many orders of magnitude: beside the relative
    bounds, a weight far below the row's largest is off by an absolute amount. fp16 rounds below 2^-14 by 2^-25 at
    most, and the largest weight is 2^4 at least (the reference lies 4 below a maximum that the row has seen), so
    each token's share of the sum moves by 2^-29 |v| at most."""
    sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    got = C.to64(got)
    num = den = 0.0
    for b in range(case.B):
        n = case.T if seqlens is None else seqlens[b]
        for hk in range(case.Hkv):
            pc, pd = case.host(case.cache, n, b, hk), case.host(case.draft, case.N, b, hk)
            val = np.concatenate([O.dequantize_values(x["codes"], x["scale"], x["zero"]) for x in (pc, pd)])
            norms = np.concatenate([pc["norms"], pd["norms"]]).astype(np.float64)
            for i in range(case.N):
                ok = np.array([True] * n + [bool(mask[b][i] >> j & 1) for j in range(case.N)])
                for h in range(hk * case.g, (hk + 1) * case.g):
                    sq = O.project_query(C.to64(case.Q[b, i, h]), case.S, case.So, pc["idx"])
                    x = sm * np.concatenate([O.estimate_scores(*sq, z["bits_in"], z["bits_out"], z["norms"], case.m,
                                                               case.m_out) for z in (pc, pd)])[ok]
                    v = val[ok]
                    delta = 4 * U * (np.abs(x).max() + 1.0)
                    for k, (s, n_proj) in enumerate(zip(sq, (case.m, case.m_out))):
                        if n_proj:
                            a = sm * math.sqrt(math.pi / 2) / n_proj * norms[ok, k].max()
                            delta += a * np.linalg.norm(s) * (6 / math.sqrt(3) * H16 + 8 * math.sqrt(n_proj + D) * U)
                    p = O.softmax(x)
                    want = p @ v
                    tol = 2 * delta * (1 + delta) * (p @ np.abs(v - want))
                    tol = tol + (2 * H16 + 8 * math.sqrt(len(x)) * U) * (p @ np.abs(v)) + 2.0 ** -29 * np.abs(v).sum(0)
                    tol = tol + B16 * (np.abs(want) + tol) + 1e-30
                    err = np.abs(got[b, i, h] - want)
                    assert np.all(err <= tol), (b, i, h, float((err / tol).max()), float(err.max()))
                    num, den = num + (err ** 2).sum(), den + (want ** 2).sum()
    assert math.sqrt(num) <= B16 * math.sqrt(den), math.sqrt(num / den)


# ------------------------------------------------------------------ values far below and far above one

@pytest.mark.parametrize("vbits", [4, 2])
@pytest.mark.parametrize("scale", [3e-4, 1e-4, 1e-5, 1e-6])
def test_tree_keeps_the_bits_of_small_values(scale, vbits):
    """Values whose steps are small or subnormal fp16 numbers: zero + code * scale is a multiple of 2^-24, so fp16
    holds it as well as any other (2^-11 relative, and exactly below 2^-13)."""
    case = Case(1, 2, 4, 333, 6, vbits=vbits, scale_v=scale)
    mask = random_tree(1, 6, 1)
    check_tree(case, case.tree(mask), mask)
    check_rows(case, case.tree(mask, sm_scale=0.4), mask, sm_scale=0.4)  # few tokens take all
    itself = [[1 << i for i in range(6)]]
    check_tree(case, case.tree(itself, [0]), itself, [0])                # one drafted token
    check_tree(case, case.tree([[0] * 6], [1]), [[0] * 6], [1])          # one committed token


WIDE = [(60000.0, -30000.0), (3000.0, 40000.0), (65504.0, 65504.0), (2048.0, 0.0), (1.0, 32768.0), (-9000.0, 0.0)]


@pytest.mark.parametrize("vbits", [4, 2])
def test_tree_values_past_the_fp16_range(vbits):
    """Groups whose zero + code * scale passes 65504 (an fp16 scale and zero reach 16 times as far)."""
    case = Case(2, 2, 4, 300, 6, vbits=vbits)
    for k, (s, z) in enumerate(WIDE):
        for g in range(4):
            set_value_group(case, case.cache, (5, 64, 130, 131, 255, 299)[k], g, s, z)
    for g in range(4):
        set_value_group(case, case.draft, 2, g, 60000.0, -30000.0)
    mask = random_tree(2, 6, 3)
    for sm in (None, 1e-3):  # a few tokens, and all of them
        check_rows(case, case.tree(mask, [300, 131], sm_scale=sm or 0.0), mask, [300, 131], sm_scale=sm)


def test_tree_values_past_the_fp16_range_where_logits_grow():
    """Growing norms lift tokens with such groups by up to 2^15 over the row's reference before it moves."""
    case = Case(1, 1, 4, 1500, 8, n_outlier=0, m_out=0)
    v = section(case, case.cache, "knorm")
    grow = (0.05 * torch.arange(v.shape[2] * 64, device="cuda").float()).half().view(1, 1, -1, 64)
    v.copy_(torch.stack([grow, torch.zeros_like(grow)], -1).contiguous().view(torch.uint8).reshape(1, 1, -1, 64, 4))
    for t in range(128, 1500, 2):
        for g in range(4):
            set_value_group(case, case.cache, t, g, 4000.0, -40000.0)
    mask = random_tree(1, 8, 5)
    check_rows(case, case.tree(mask), mask)
    case.Q.mul_(8)
    check_rows(case, case.tree(mask), mask)


@pytest.mark.parametrize("token", [0, 127, 128, 700, 1499, "draft"])
def test_tree_one_value_past_the_fp16_range(token):
    """One token of one kv head, in the first unit, a later one, the last or the drafts; the other heads' outputs stay
    bit for bit what they are without it."""
    case = Case(1, 3, 4, 1500, 8)
    mask = [[1 << i | 4 for i in range(8)]]  # every row sees drafted token 2
    plain = case.tree(mask)
    cache, t = (case.draft, 2) if token == "draft" else (case.cache, token)
    row = section(case, cache, "vsz")[0, 1, t // 64, t % 64]
    row.copy_(torch.tensor([60000.0, -30000.0] * 4, dtype=torch.float16, device="cuda").view(torch.uint8))
    got = case.tree(mask)
    check_rows(case, got, mask)
    assert torch.equal(got[:, :, :4], plain[:, :, :4]) and torch.equal(got[:, :, 8:], plain[:, :, 8:])
    assert torch.equal(case.tree(mask), got)


def test_tree_wait_limits_where_values_pass_the_fp16_range():
    case = Case(2, 4, 4, 6000, 8)
    for t in range(0, 6000, 333):
        set_value_group(case, case.cache, t, 2, 60000.0, -30000.0)
    mask = random_tree(2, 8, 7)
    want = case.tree(mask)
    try:
        Q.qjl_set_wait_limit(case.ctx.handle, 1)
        out = case.tree(mask)
        torch.cuda.synchronize()
        assert torch.isnan(out).any()
    finally:
        Q.qjl_set_wait_limit(case.ctx.handle, 2_000_000_000)
    assert torch.equal(case.tree(mask), want) and bool(torch.isfinite(want).all())


def test_tree_small_groups_beside_groups_past_the_fp16_range():
    """From the first unit with a scale of 2^11 or a zero of 2^15 and more on, a kv head's values are held divided by
    16: they are then off by the roundings of zero / 16 and of the sum, half an fp16 subnormal step each:
    2 * 2^-25 * 16 = 2^-20. The other kv head keeps all bits."""
    case = Case(1, 2, 2, 70, 9, scale_v=1e-4)
    vsz = section(case, case.draft, "vsz")
    for i in (1, 4, 8):
        vsz[:, 0, 0, i, 4:8] = torch.tensor([60000.0, -20000.0], dtype=torch.float16, device="cuda").view(torch.uint8)
    itself = [[1 << i for i in range(9)]]
    got = C.to64(case.tree(itself, [0]))
    for hk in range(2):
        x = case.host(case.draft, 9, 0, hk)
        v = O.dequantize_values(x["codes"], x["scale"], x["zero"])
        for i in range(9):
            tol = H16 * np.abs(v[i]) + (2.0 ** -20 if hk == 0 else 0.0)
            tol = tol + B16 * (np.abs(v[i]) + tol)
            for g in range(2):
                err = np.abs(got[0, i, 2 * hk + g] - v[i])
                assert np.all(err <= tol), (i, float((err - tol).max()))
            assert not np.any(np.isinf(got[0, i]))


# ------------------------------------------------------------------ draft caches

def test_draft_cache_with_other_outlier_channels_is_refused():
    case = Case(2, 2, 4, 100, 4)
    other = case.ctx.allocate_cache(2, 2, 64)  # channels of its own
    out, lens = torch.full_like(case.Q, 3.0), torch.tensor([100, 50], dtype=torch.int32, device="cuda")
    ws = case.ctx.tree_workspace(2, 4, 8, 2)
    with pytest.raises(Q.QJLError, match="outlier_idx"):
        Q.qjl_tree_attention(case.ctx.handle, case.cache, other, case.Q, 100, out, workspace=ws)
    before = case.cache.tiles.clone()
    with pytest.raises(Q.QJLError, match="outlier_idx"):
        Q.qjl_cache_commit(case.ctx.handle, case.cache, other, torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                           torch.ones_like(lens), lens)
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and torch.equal(case.cache.tiles, before)  # nothing was launched
    # without outliers the arrays hold nothing and may differ
    case = Case(1, 2, 4, 100, 4, m_out=0, n_outlier=0)
    other = case.ctx.allocate_cache(1, 2, 64)
    other.tiles.copy_(case.draft.tiles)
    want = case.tree()
    case.draft = other
    assert torch.equal(case.tree(), want)


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("shape", [(1, 32, 8), (1, 64, 8), (2, 8, 8), (16, 32, 8), (1, 8, 1), (3, 2, 1)])
@pytest.mark.parametrize("kw", [{}, {"m": 512, "m_out": 256, "value_bits": 2}, {"m": 96, "m_out": 0, "n_outlier": 0}])
def test_tree_workspace_never_falls_as_drafts_grow(shape, kw):
    B, Hq, Hkv = shape
    ctx = Q.QJLContext(0, D, **kw)
    sizes = [Q.qjl_tree_attention_workspace_bytes(ctx.handle, B, n, Hq, Hkv) for n in range(1, 65)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    ctx.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_smaller_steps_in_the_workspace_of_a_larger_one(dtype):
    """33 drafts of 4 query heads make two row blocks, 32 one larger one."""
    case = Case(1, 2, 4, 200, 33, dtype)
    ws = case.ctx.tree_workspace(1, 33, 8, 2)
    for n in (33, 32, 31, 16, 1):
        mask = random_tree(1, n, n)
        own = case.ctx.tree_workspace(1, n, 8, 2)
        q, case.N = case.Q[:, :n].contiguous(), n
        assert torch.equal(case.tree(mask, Q_=q, ws=ws), case.tree(mask, Q_=q, ws=own)), n


# ------------------------------------------------------------------ rotary positions

def check_rope_far(got, x, pos, inverse=False):
    """The plain rotation of all 128 dims against the formula with 64-bit mantissas, fp32 data. 12 u of the magnitudes
    as in test_gpu_speculative; the angle: the table's entry and its product with the position round by 2^-53 each and
    the table's own power and quotient by as much together, 2^-51 |P f| covers them."""
    x64, got = C.to64(x).astype(np.longdouble), C.to64(got)
    for i in range(D // 2):
        f = np.longdouble(10000.0) ** (-np.longdouble(2 * i) / D)
        a = pos.astype(np.longdouble) * f * (-1 if inverse else 1)
        c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
        u, v = x64[..., i], x64[..., i + D // 2]
        tol = (np.abs(u) + np.abs(v)) * (13 * U + 2.0 ** -51 * np.abs(a)[:, None, :])
        assert np.all(np.abs(got[..., i] - (u * c - v * s)) <= tol), i
        assert np.all(np.abs(got[..., i + D // 2] - (v * c + u * s)) <= tol), i


def test_rope_start_positions_run_past_31_bits():
    """P = t_start + t is not bound to int32."""
    start = np.array([2 ** 31 - 5, -2 ** 31, 2 ** 31 - 1], np.int64)
    x = torch.randn(3, 2, 9, D, generator=torch.Generator().manual_seed(3))
    got = Q.qjl_rope(Q.qjl_rope_init(), x.cuda(), t_start=torch.from_numpy(start.astype(np.int32)).cuda())
    check_rope_far(got, x, start[:, None] + np.arange(9))


@pytest.mark.parametrize("inverse", [False, True])
def test_rope_at_the_ends_of_the_position_range(inverse):
    g = torch.Generator().manual_seed(4)
    near = torch.randint(0, 2000, (4, 50), generator=g)
    ends = torch.tensor([2 ** 31 - 2001, -2 ** 31, 2 ** 27, -2 ** 24])[:, None] + near
    x = torch.randn(4, 2, 50, D, generator=g)
    got = Q.qjl_rope(Q.qjl_rope_init(), x.cuda(), positions=ends.to(torch.int32).cuda(), inverse=inverse)
    check_rope_far(got, x, ends.numpy(), inverse)


# ------------------------------------------------------------------ commit

def test_commit_between_overlapping_slabs_is_refused():
    """A draft slab that begins inside the cache's: source and target rows would be the same bytes."""
    case = Case(2, 2, 1, 128, 4)  # two tiles a slab
    flat = case.cache.tiles.flatten(0, 2)
    lens = torch.tensor([100, 50], dtype=torch.int32, device="cuda")
    path = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    before = case.cache.tiles.clone()
    for first in (0, 1, 4):
        part = Q.QJLCache(case.cache.outlier_idx, flat[first:first + 4].view(2, 2, 1, -1), 2, 2, 64, case.m, case.m_out)
        with pytest.raises(Q.QJLError, match="share"):
            Q.qjl_cache_commit(case.ctx.handle, case.cache, part, path, torch.ones_like(lens), lens)
    torch.cuda.synchronize()
    assert torch.equal(case.cache.tiles, before)
    # side by side in one buffer they may lie
    buf = torch.zeros(12, flat.shape[-1], dtype=torch.uint8, device="cuda")
    buf[:8].copy_(flat)
    buf[8:].copy_(case.draft.tiles.flatten(0, 2))
    make = lambda t, n: Q.QJLCache(case.cache.outlier_idx, t, 2, 2, 64 * n, case.m, case.m_out)  # noqa: E731
    Q.qjl_cache_commit(case.ctx.handle, make(buf[:8].view(2, 2, 2, -1), 2), make(buf[8:].view(2, 2, 1, -1), 1), path,
                       torch.ones_like(lens), lens)
    Q.qjl_cache_commit(case.ctx.handle, case.cache, case.draft, path, torch.ones_like(lens), lens)
    assert torch.equal(buf[:8], flat) and not torch.equal(case.cache.tiles, before)
