"""The speculative decode step on the GPU: rotary positions, tree attention, read-back and commit, each
against its formula in fp64 on the GPU-made cache, and a whole step of them together.

Tolerances (u = 2^-24, the half step of fp32; h = 2^-11 of fp16; b = 2^-8 of bf16), from the roundings that
the formulas admit:
  * a sum of n fp32 terms: each addition rounds a partial sum of about the terms' 2-norm, the n roundings
    add like a random walk: 8 sqrt(n) u times the 2-norm (8 standard deviations and more);
  * the projected query in fp16 (bf16 queries): n independent roundings of at most h, uniform, so a score moves
    by 6 h / sqrt(3) times A |sq|_2 at six standard deviations;
  * weights and dequantised values in fp16: h each, relative;
  * an output moves by at most 2 delta sum p |v - o| when every logit moves by at most delta;
  * the output's own rounding: b or u, relative.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
from decode_attention_qjl_b200 import inputs as I  # noqa: E402
from decode_attention_qjl_b200 import qjl as Q  # noqa: E402
from tests import gpu_common as C  # noqa: E402

pytestmark = pytest.mark.gpu
U, H16, B16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
D = 128


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ rotary positions

def rope_reference(x, pos, rot, base, interleaved, inverse, factor=1.0, original_len=0.0, low=1.0, high=4.0, amp=1.0):
    """x [B, H, T, d] fp64, pos [B, T]."""
    y = x.copy()
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if original_len > 0:
            s = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f = s * f + (1 - s) * f / factor
        else:
            f = f / factor
        a = pos.astype(np.float64) * f * (-1 if inverse else 1)
        c, s_ = np.cos(a)[:, None, :] * amp, np.sin(a)[:, None, :] * amp
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[..., u] = x[..., u] * c - x[..., v] * s_
        y[..., v] = x[..., v] * c + x[..., u] * s_
    return y


def rope_bound(x, y, rot, interleaved, amp, pos, dtype):
    """sincos: the reduced turn rounds to u relative (pi u of an angle), 2 ulp (4 u) of the function, u of the
    amplitude; two products and a sum: 2 u more; 12 u in all of amp (|x_u| + |x_v|). fp64 angles: the reference's own
    product, and the kernel's, round a position's angle to 2^-53 relative each."""
    e = np.zeros_like(x)
    half = rot // 2
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    mag = np.abs(x[..., u]) + np.abs(x[..., v])
    far = 8 * 2.0 ** -53 * np.abs(pos).max()
    e[..., u] = e[..., v] = mag * abs(amp) * (12 * U + far)
    return e + (half_step(dtype) * (np.abs(y) + e) if dtype != torch.float32 else U * np.abs(y))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, T, rot, interleaved, inverse, kwargs
    (1, 1, 1, 1, 128, False, False, {}),
    (2, 8, 2, 7, 128, False, False, {}),
    (3, 4, 4, 33, 64, True, False, {"factor": 8.0, "original_len": 512, "low": 1.0, "high": 4.0, "amplitude": 1.2}),
    (2, 5, 1, 65, 96, False, True, {"factor": 4.0}),
    (1, 3, 2, 257, 16, True, True, {"base": 500000.0}),
    (2, 32, 8, 130, 32, False, False, {"amplitude": 0.5}),
])
@pytest.mark.parametrize("layout", ["bhtd", "bthd", "in_place"])
def test_rope_matches_the_formula(dtype, case, layout):
    B, Hq, Hkv, T, rot, inter, inverse, kw = case
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(-70000, 1 << 21, (B, T), generator=g, dtype=torch.int32)
    table = Q.qjl_rope_init(rot_dim=rot, interleaved=inter, **kw)
    ref_kw = {"base": 10000.0, **{k: v for k, v in kw.items() if k != "amplitude"}}
    amp = kw.get("amplitude", 1.0)
    xs, dev = [], []
    for H in (Hq, Hkv):
        x = torch.randn(B, T, H, D, generator=g).to(dtype)
        x = x.transpose(1, 2) if layout == "bthd" else x.transpose(1, 2).contiguous()
        xs.append(x)
        dev.append(x.cuda())
    outs = {} if layout != "in_place" else {"Q_out": dev[0], "K_out": dev[1]}
    got = Q.qjl_rope(table, *dev, positions=pos.cuda(), inverse=inverse, **outs)
    if layout == "in_place":
        assert got[0].data_ptr() == dev[0].data_ptr()
    for x, y in zip(xs, got):
        x64 = C.to64(x)
        want = rope_reference(x64, pos.numpy(), rot, ref_kw["base"], inter, inverse, ref_kw.get("factor", 1.0),
                              ref_kw.get("original_len", 0.0), ref_kw.get("low", 1.0), ref_kw.get("high", 4.0), amp)
        err = np.abs(C.to64(y) - want)
        bound = rope_bound(x64, want, rot, inter, amp, pos.numpy(), dtype)
        assert np.all(err <= bound), float((err - bound).max())
        assert np.array_equal(C.to64(y)[..., rot:], x64[..., rot:])  # dims past rot_dim are copied


def test_rope_default_and_start_positions_and_single_tensor():
    g = torch.Generator().manual_seed(6)
    x = torch.randn(2, 3, 9, D, generator=g)
    table = Q.qjl_rope_init()
    start = torch.tensor([11, -4], dtype=torch.int32)
    for t_start in (None, start):
        pos = (torch.arange(9)[None] + (0 if t_start is None else t_start[:, None])).expand(2, 9).to(torch.int32).contiguous()
        a = Q.qjl_rope(table, x.cuda(), t_start=None if t_start is None else t_start.cuda())
        b = Q.qjl_rope(table, x.cuda(), positions=pos.cuda())
        assert torch.equal(a, b)


def test_rope_inverse_is_the_gradient_and_the_inverse():
    """<w, rope(x)> = <rope_inverse(w), x> for every x, and, amplitude 1, rope_inverse(rope(x)) = x."""
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(2, 4, 31, D, generator=g), torch.randn(2, 4, 31, D, generator=g)
    pos = torch.randint(0, 100000, (2, 31), generator=g, dtype=torch.int32).cuda()
    table = Q.qjl_rope_init(rot_dim=96, amplitude=1.3, interleaved=True)
    y, z = Q.qjl_rope(table, x.cuda(), positions=pos), Q.qjl_rope(table, w.cuda(), positions=pos, inverse=True)
    lhs, rhs = C.to64(w) * C.to64(y), C.to64(z) * C.to64(x)
    # each product is off by at most 13 u 1.3 (|.| + |.|)|.|: sum of the magnitudes bounds the difference
    mag = 1.3 * (np.abs(C.to64(w)).sum(-1) * np.abs(C.to64(x)).max(-1)).sum()
    assert abs(lhs.sum() - rhs.sum()) <= 4 * 13 * U * mag
    # against differences: d/dx_k of <w, rope(x)> along a direction
    e = torch.randn(2, 4, 31, D, generator=g)
    eps = 2.0 ** -3
    up = (C.to64(w) * C.to64(Q.qjl_rope(table, (x + eps * e).cuda(), positions=pos))).sum()
    dn = (C.to64(w) * C.to64(Q.qjl_rope(table, (x - eps * e).cuda(), positions=pos))).sum()
    slope = (C.to64(z) * C.to64(e)).sum()
    assert abs((up - dn) / (2 * eps) - slope) <= 4 * 16 * U * mag / eps
    plain = Q.qjl_rope_init()
    back = Q.qjl_rope(plain, Q.qjl_rope(plain, x.cuda(), positions=pos), positions=pos, inverse=True)
    assert float((back.cpu() - x).abs().max()) <= 4 * 13 * U * float(x.abs().max())


def test_rope_empty_calls_and_refusals():
    table = Q.qjl_rope_init()
    x = torch.randn(2, 3, 4, D, device="cuda")
    assert Q.qjl_rope(table, x[:0]).shape == (0, 3, 4, D)
    assert Q.qjl_rope(table, x[:, :, :0]).shape == (2, 3, 0, D)
    with pytest.raises(ValueError):
        Q.qjl_rope(table, x, K=x[:1])                        # another B
    with pytest.raises(ValueError):
        Q.qjl_rope(table, x, positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        Q.qjl_rope(table, x.cpu())
    with pytest.raises(TypeError):
        Q.qjl_rope(table, x.half())
    with pytest.raises(Q.QJLError, match="overlap"):
        Q.qjl_rope(table, x, Q_out=torch.empty_like(x)[:, :1].expand(2, 3, 4, D))
    with pytest.raises(Q.QJLError, match="strides"):
        y = torch.empty(2, 3, 4, D + 2, device="cuda")
        Q.qjl_rope(table, x, Q_out=y[..., :D])
    with pytest.raises(Q.QJLError, match="same strides"):
        Q.qjl_rope(table, x[:, :, :3], Q_out=x.as_strided((2, 3, 3, D), (12 * D, 3 * D, D, 1)))


# ------------------------------------------------------------------ caches

class Case:
    """A committed cache and a draft cache made by the library's quantisers, and their contents in fp64."""

    def __init__(self, B, Hkv, g, T, N, dtype=torch.bfloat16, m=256, m_out=64, n_outlier=8, vbits=4, cap=None, seed=3,
                 scale_v=1.0):
        w = I.Workload("t", B, Hkv * g, Hkv, max(T, 1), m, m_out, n_outlier,
                       "bf16" if dtype == torch.bfloat16 else "fp32", "x20")
        inp = I.make_inputs(w, seed=seed, device="cpu", B=B, T=max(T, 1) + N, Hkv=Hkv)
        self.B, self.Hkv, self.g, self.T, self.N, self.dtype = B, Hkv, g, T, N, dtype
        self.m, self.m_out, self.n_outlier, self.vbits = m, m_out, n_outlier, vbits
        self.K, self.V = inp["K"].cuda(), (inp["V"] * scale_v).to(dtype).cuda()
        T0 = max(T, 1)
        gen = torch.Generator().manual_seed(seed + 1)
        self.Q = torch.randn(B, N, Hkv * g, D, generator=gen).to(dtype).cuda()
        self.ctx = Q.QJLContext(0, D, m, m_out, n_outlier, vbits)
        self.cache = self.ctx.allocate_cache(B, Hkv, cap or T0)
        self.cache.tiles.fill_(0xFF)  # NaN norms, scales and zeros in every slot that is not written
        Q.qjl_quantize_keys(self.ctx.handle, self.cache, self.K[:, :, :T0], Q.QJL_PREFILL,
                            workspace=self.ctx.keys_workspace(B, Hkv))
        Q.qjl_quantize_values(self.ctx.handle, self.cache, self.V[:, :, :T0])
        self.draft = self.cache.draft()
        self.draft.tiles.fill_(0xFF)
        Q.qjl_quantize_keys(self.ctx.handle, self.draft, self.K[:, :, T0:], Q.QJL_APPEND)
        Q.qjl_quantize_values(self.ctx.handle, self.draft, self.V[:, :, T0:])
        torch.cuda.synchronize()
        self.S, self.So = O.sketch_pair(0, D, m, m_out)

    def host(self, cache, n, b, h):
        g = C.cache_to_numpy(cache, self.m_out, self.n_outlier, T=n, b=b, h=h)
        return {k: v[0, 0] for k, v in g.items()}

    def tree(self, mask=None, seqlens=None, n_draft=None, sm_scale=0.0, Q_=None, ws=None, out=None):
        q = self.Q if Q_ is None else Q_
        ws = self.ctx.tree_workspace(self.B, self.N, q.shape[2], self.Hkv) if ws is None else ws
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        mk = None if mask is None else torch.from_numpy(np.asarray(mask, dtype=np.uint64).view(np.int64)).cuda()
        Q.qjl_tree_attention(self.ctx.handle, self.cache, self.draft, q, self.T, out, seqlens=i32(seqlens),
                             n_draft=i32(n_draft), tree_mask=mk, sm_scale=sm_scale, workspace=ws)
        return out


def check_tree(case, got, mask, seqlens=None, n_draft=None, sm_scale=None, rows=None):
    """Every element of the output against the formula in fp64, with the bounds of the file's head."""
    sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    got = C.to64(got)
    bf = case.dtype == torch.bfloat16
    e16, eo = (H16, B16) if bf else (0.0, U)
    rng = np.random.default_rng(0)
    num = den = 0.0
    for b in range(case.B):
        n = min(max(case.T if seqlens is None else seqlens[b], 0), case.T)
        nd = min(max(case.N if n_draft is None else n_draft[b], 0), case.N)
        for hk in range(case.Hkv):
            pc, pd = case.host(case.cache, n, b, hk), case.host(case.draft, nd, b, hk)
            val = np.concatenate([O.dequantize_values(x["codes"], x["scale"], x["zero"]) for x in (pc, pd)])
            norms = np.concatenate([pc["norms"], pd["norms"]]).astype(np.float64)
            pick = list(range(case.N)) if rows is None else sorted(rng.choice(case.N, min(rows, case.N), replace=False))
            for i in pick:
                for gg in range(case.g):
                    h = hk * case.g + gg
                    o = got[b, i, h]
                    if i >= nd:
                        assert np.all(o == 0.0)
                        continue
                    sq = O.project_query(C.to64(case.Q[b, i, h]), case.S, case.So, pc["idx"])
                    row = int(mask[b][i]) if mask is not None else (2 << i) - 1
                    ok = np.array([True] * n + [bool(row >> j & 1) for j in range(nd)])
                    if not ok.any():
                        assert np.all(o == 0.0), (b, i, h)
                        continue
                    x = sm * np.concatenate([O.estimate_scores(*sq, z["bits_in"], z["bits_out"], z["norms"], case.m,
                                                               case.m_out) for z in (pc, pd)])[ok]
                    v = val[ok]
                    delta = 4 * U * (np.abs(x).max() + 1.0)
                    for k, (s, n_proj) in enumerate(zip(sq, (case.m, case.m_out))):
                        if n_proj:
                            a = sm * math.sqrt(math.pi / 2) / n_proj * norms[ok, k].max()
                            delta += a * np.linalg.norm(s) * (6 / math.sqrt(3) * e16 + 8 * math.sqrt(n_proj + D) * U)
                    p = O.softmax(x)
                    want = p @ v
                    mag = p @ np.abs(v)
                    tol = 2 * delta * (1 + delta) * (p @ np.abs(v - want)) + (2 * e16 + 8 * math.sqrt(len(x)) * U) * mag
                    tol = tol + eo * (np.abs(want) + tol) + 1e-30
                    err = np.abs(o - want)
                    assert np.all(err <= tol), (b, i, h, float((err / tol).max()), float(err.max()))
                    num, den = num + (err ** 2).sum(), den + (want ** 2).sum()
    # the roundings are independent: together they stay below the output's own half step (fp32: 64 of them)
    assert math.sqrt(num) <= (B16 if bf else 64 * U) * math.sqrt(den) + 1e-30, math.sqrt(num / max(den, 1e-300))


def random_tree(B, N, seed=0):
    rng = np.random.default_rng(seed)
    mask = [[0] * N for _ in range(B)]
    for b in range(B):
        for i in range(N):
            parent = int(rng.integers(-1, i)) if i else -1
            mask[b][i] = (mask[b][parent] if parent >= 0 else 0) | (1 << i)
    return mask


TREE_CASES = [
    # B, Hkv, g, T, N, kwargs, seqlens, n_draft
    (1, 1, 1, 1, 1, {}, None, None),
    (1, 2, 1, 63, 1, {}, None, None),
    (2, 2, 4, 64, 5, {}, None, None),
    (2, 1, 2, 65, 7, {"vbits": 2}, None, [7, 3]),
    (3, 2, 4, 300, 13, {}, [300, 0, 127], [13, 1, 0]),
    (1, 1, 8, 128, 16, {}, None, None),
    (1, 1, 8, 129, 64, {}, None, None),          # 512 rows of one kv head
    (2, 1, 1, 1000, 64, {"m": 512, "m_out": 256, "n_outlier": 32}, [1000, 999], None),
    (1, 2, 4, 700, 9, {"m": 96, "m_out": 0, "n_outlier": 0}, None, None),
    (1, 1, 4, 257, 33, {"m": 32, "m_out": 32, "n_outlier": 1, "vbits": 2}, None, None),
    (2, 3, 2, 2500, 11, {"m": 128, "m_out": 32, "n_outlier": 4}, [2500, 1234], [11, 11]),
    (5, 1, 1, 40, 3, {"m": 160, "m_out": 96, "n_outlier": 8}, [0, 1, 2, 39, 40], [3, 2, 1, 0, 3]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tc", TREE_CASES)
def test_tree_attention_matches_the_formula(dtype, tc):
    B, Hkv, g, T, N, kw, seqlens, n_draft = tc
    case = Case(B, Hkv, g, T, N, dtype, **kw)
    mask = random_tree(B, N)
    got = case.tree(mask, seqlens, n_draft)
    check_tree(case, got, mask, seqlens, n_draft, rows=12)
    chain = case.tree(None, seqlens, n_draft, sm_scale=0.2)
    check_tree(case, chain, None, seqlens, n_draft, sm_scale=0.2, rows=4)
    case.ctx.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_rows_with_nothing_left_and_masked_infinities(dtype):
    """Rows whose mask leaves nothing give 0; NaN norms and infinite values in masked drafts reach nobody else."""
    B, Hkv, g, N = 2, 2, 4, 9
    case = Case(B, Hkv, g, 70, N, dtype)
    bad = 4  # drafted token 4: NaN key norms, infinite value zeros
    for name, value in (("knorm", float("nan")), ("vsz", float("inf"))):
        off, nb, sec = next((o, n, s) for nm, o, n, s in Q.tile_sections(case.m, case.m_out) if nm == name)
        v = case.draft.tiles[..., off:off + sec].unflatten(-1, (64, nb))
        v[..., bad, :] = torch.full((nb // 2,), value, dtype=torch.float16, device="cuda").view(torch.uint8)
    mask = [[(1 << i) | 1 if i != bad else 1 << bad for i in range(N)] for _ in range(B)]
    mask[0][2] = 0
    mask[1][8] = (1 << 63) | (1 << 20)  # bits past the drafts only
    got = case.tree(mask, [0, 70])
    g64 = C.to64(got)
    assert np.all(g64[0, 2] == 0.0)
    assert np.all(np.isnan(g64[:, bad]))
    others = [i for i in range(N) if i != bad]
    assert np.all(np.isfinite(g64[:, others]))
    # with the value infinite but the key sound, the rows that attend to it are not finite and the others are
    off, nb, sec = next((o, n, s) for nm, o, n, s in Q.tile_sections(case.m, case.m_out) if nm == "knorm")
    v = case.draft.tiles[..., off:off + sec].unflatten(-1, (64, nb))
    v[..., bad, :] = torch.full((nb // 2,), 3.0, dtype=torch.float16, device="cuda").view(torch.uint8)
    g64 = C.to64(case.tree(mask, [0, 70]))
    assert not np.any(np.isfinite(g64[:, bad])) and np.all(np.isfinite(g64[:, others]))
    clean = Case(B, Hkv, g, 70, N, dtype)
    want = C.to64(clean.tree(mask, [0, 70]))
    assert np.array_equal(g64[:, others], want[:, others])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e4])
def test_tree_query_and_value_ranges(dtype, scale):
    """Queries and values far from one: scores near zero or one token taking all, values up to 4e4."""
    case = Case(1, 1, 4, 333, 6, dtype, scale_v=scale)
    case.Q.mul_(scale if scale < 1 else 20.0)
    mask = random_tree(1, 6, 1)
    check_tree(case, case.tree(mask), mask)


def test_tree_strided_queries_and_workspace_reuse():
    case = Case(2, 2, 4, 500, 8)
    mask = random_tree(2, 8, 2)
    want = case.tree(mask)
    ws = case.ctx.tree_workspace(2, 8, 8, 2)
    ws.fill_(0xFF)  # no initial contents needed
    big = torch.zeros(2, 8, 3, 8, D, dtype=torch.bfloat16, device="cuda")
    big[:, :, 1] = case.Q
    a = case.tree(mask, Q_=big[:, :, 1], ws=ws)
    head_major = case.Q.transpose(1, 2).contiguous().transpose(1, 2)  # [B, N, Hq, d] with heads outermost
    b = case.tree(mask, Q_=head_major, ws=ws, out=torch.empty(case.Q.shape, dtype=torch.bfloat16, device="cuda"))
    c = case.tree(mask, [250, 1], ws=ws)
    d = case.tree(mask, ws=ws)
    for x in (a, b, d):
        assert torch.equal(x, want)
    check_tree(case, c, mask, [250, 1])


def test_tree_repeats_and_long_context():
    """A long ragged batch (pairs shared by many blocks), the same bits at every call."""
    case = Case(3, 4, 4, 9000, 10, cap=9000 + 64)
    mask = random_tree(3, 10, 4)
    lens = [9000, 4097, 8191]
    a = case.tree(mask, lens)
    for _ in range(3):
        assert torch.equal(case.tree(mask, lens), a)
    check_tree(case, a, mask, lens, rows=3)


def test_chain_of_drafts_equals_decode_steps():
    """A chain of drafts gives what as many decode steps give (the same cache bytes, fp32 outputs)."""
    case = Case(2, 2, 4, 333, 5, cap=400)
    got = C.to64(case.tree(None))
    ws = case.ctx.decode_workspace(2, 8, 2, 400)
    o = torch.empty(2, 8, D, device="cuda")
    for i in range(5):
        Q.qjl_decode_step(case.ctx.handle, case.cache, case.Q[:, i].contiguous(), case.K[:, :, 333 + i].contiguous(),
                          case.V[:, :, 333 + i].contiguous(), 333 + i, o, workspace=ws)
        Q.qjl_decode_workspace_status(case.ctx.handle, ws, 2, 8, 2)
        want = C.to64(o)
        err = np.linalg.norm(got[:, i] - want) / np.linalg.norm(want)
        assert err <= B16, (i, err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_many_sequences_of_every_length(dtype):
    """More sequences than a warp has lanes, empty ones and ones without drafts among them, in every place."""
    B, N = 75, 3
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.choice([0, 0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 300], B)]
    nds = [int(x) for x in rng.integers(0, N + 1, B)]
    nds[0] = nds[-1] = 0
    lens[5], nds[5] = 0, 0
    case = Case(B, 1, 2, 300, N, dtype)
    mask = random_tree(B, N, 6)
    check_tree(case, case.tree(mask, lens, nds), mask, lens, nds)
    out = case.tree(mask, lens, [0] * B)
    assert int(out.count_nonzero()) == 0  # nobody drafts: all rows are zero


def test_tree_lengths_are_clamped_and_masks_of_64_drafts():
    case = Case(2, 1, 1, 150, 64)
    chain = [[(1 << (i + 1)) - 1 for i in range(64)] for _ in range(2)]
    want = case.tree(chain)
    assert torch.equal(case.tree(None), want)                                    # the default mask is the chain
    assert torch.equal(case.tree(chain, [10 ** 6, 150], [64, 99]), want)         # past T and N
    low = case.tree(chain, [-3, 0], [64, 64])
    check_tree(case, low, chain, [0, 0], rows=6)
    last = [[1 << 63] * 64 for _ in range(2)]                                    # only the last draft
    check_tree(case, case.tree(last), last, rows=6)
    none = case.tree(chain, [150, 150], [-1, 64])
    assert int(none[0].count_nonzero()) == 0 and torch.equal(none[1], want[1])


@pytest.mark.parametrize("g,N", [(1, 48), (2, 40), (4, 20), (4, 28), (8, 15), (8, 33)])
def test_tree_row_blocks(g, N):
    """48 to 264 rows of a kv head: every size of a row block, and several of them."""
    case = Case(1, 2, g, 700, N, m=128, m_out=64)
    mask = random_tree(1, N, N)
    check_tree(case, case.tree(mask), mask, rows=5)


def test_tree_logits_that_grow_along_the_context():
    """Keys whose norms grow with the position: every unit raises the maximum, and with it the references."""
    case = Case(1, 1, 4, 1500, 8, n_outlier=0, m_out=0)
    off, nb, sec = next((o, n, s) for nm, o, n, s in Q.tile_sections(256, 0) if nm == "knorm")
    v = case.cache.tiles[..., off:off + sec].unflatten(-1, (64, nb))
    grow = (0.05 * torch.arange(v.shape[2] * 64, device="cuda").float()).half().view(1, 1, -1, 64)
    pair = torch.stack([grow, torch.zeros_like(grow)], -1)
    v.copy_(pair.contiguous().view(torch.uint8).reshape(1, 1, -1, 64, 4))
    mask = random_tree(1, 8, 5)
    check_tree(case, case.tree(mask), mask)
    case.Q.mul_(8)
    check_tree(case, case.tree(mask), mask)


def test_tree_and_read_wait_limits():
    """Waits that run out end the call with NaN rows (no fault, no hang); the next call is whole again."""
    case = Case(2, 4, 4, 6000, 16)
    mask = random_tree(2, 16, 7)
    ws = case.ctx.tree_workspace(2, 16, 16, 4)
    want = case.tree(mask, ws=ws)
    K = torch.zeros(2, 4, 6000, D, dtype=torch.bfloat16, device="cuda")
    Q.qjl_cache_read(case.ctx.handle, case.cache, 6000, K)
    good = K.clone()
    try:
        Q.qjl_set_wait_limit(case.ctx.handle, 1)
        out = case.tree(mask, ws=ws)
        Q.qjl_cache_read(case.ctx.handle, case.cache, 6000, K)
        torch.cuda.synchronize()
        assert torch.isnan(out).any() and torch.isnan(K).any()
    finally:
        Q.qjl_set_wait_limit(case.ctx.handle, 2_000_000_000)
    assert torch.equal(case.tree(mask, ws=ws), want)
    Q.qjl_cache_read(case.ctx.handle, case.cache, 6000, K)
    assert torch.equal(K, good)


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rc", [
    # B, Hkv, tokens in the cache, T, start, seqlens, kwargs
    (1, 1, 1, 1, None, None, {}),
    (2, 3, 200, 130, [3, 65], [200, 140], {}),
    (1, 2, 700, 700, None, [700], {"vbits": 2}),
    (2, 2, 300, 129, [0, 171], None, {"m": 512, "m_out": 256, "n_outlier": 32}),
    (1, 1, 260, 255, [1], [260], {"m": 96, "m_out": 0, "n_outlier": 0}),
    (1, 2, 130, 140, [-5], [130], {"m": 160, "m_out": 32, "n_outlier": 3, "vbits": 2}),
    (3, 5, 64, 64, None, [0, 64, 31], {"m": 32, "m_out": 32, "n_outlier": 1}),
])
def test_cache_read_matches_the_formula(dtype, rc):
    B, Hkv, n, T, start, seqlens, kw = rc
    case = Case(B, Hkv, 1, n, 1, **kw)
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Ko = torch.full((B, T, Hkv, D), 7.0, dtype=dtype, device="cuda").transpose(1, 2)  # token-major
    Vo = torch.full((B, Hkv, T, D), 7.0, dtype=dtype, device="cuda")
    Q.qjl_cache_read(case.ctx.handle, case.cache, T, Ko, Vo, t_start=i32(start), seqlens=i32(seqlens or [n] * B))
    K64, V64 = C.to64(Ko), C.to64(Vo)
    for b in range(B):
        lim = n if seqlens is None else seqlens[b]
        pos = np.arange(T) + (start[b] if start else 0)
        live = (pos >= 0) & (pos < lim)
        assert np.all(K64[b][:, ~live] == 7.0) and np.all(V64[b][:, ~live] == 7.0)
        for h in range(Hkv):
            x = case.host(case.cache, lim, b, h)
            v = O.dequantize_values(x["codes"], x["scale"], x["zero"])[pos[live]]
            assert np.all(np.abs(V64[b, h, live] - v) <= (half_step(dtype) + U) * np.abs(v))
            nrm = x["norms"].astype(np.float64)[pos[live]]
            for part, S, mm, cols in ((0, case.S, case.m, np.setdiff1d(np.arange(D), x["idx"])),
                                      (1, case.So, case.m_out, x["idx"])):
                if mm == 0 or len(cols) == 0:
                    continue
                sg = O.unpack_signs(x["bits_out" if part else "bits_in"], mm)[pos[live]]
                f = math.sqrt(math.pi / 2) / mm * nrm[:, part][:, None]
                k = f * (sg @ S[:, cols])
                tol = f * 8 * math.sqrt(mm) * 2 * U * np.linalg.norm(S[:, cols], axis=0) + 4 * U * np.abs(k)
                tol = tol + half_step(dtype) * (np.abs(k) + tol)
                err = np.abs(K64[b, h, live][:, cols] - k)
                assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


def test_cache_read_one_output_only_and_scores():
    """K alone and V alone; and <q, K_hat> is the score that decode reports."""
    case = Case(1, 2, 2, 150, 1)
    K = torch.empty(1, 2, 150, D, device="cuda")
    V = torch.empty(1, 2, 150, D, device="cuda")
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    Q.qjl_cache_read(case.ctx.handle, case.cache, 150, K, V)
    Q.qjl_cache_read(case.ctx.handle, case.cache, 150, K_out=K2)
    Q.qjl_cache_read(case.ctx.handle, case.cache, 150, V_out=V2)
    assert torch.equal(K, K2) and torch.equal(V, V2)
    _, sc = C.run_decode(case.ctx, case.cache, case.Q[:, 0].contiguous(), 150)
    want = np.einsum("bhgd,bhtd->bhgt", C.to64(case.Q[:, 0]).reshape(1, 2, 2, D), C.to64(K)).reshape(1, 4, 150)
    floor = C.SCORE_FLOOR * np.sqrt((want ** 2).mean(-1, keepdims=True))
    assert np.all(np.abs(sc - want) <= C.SCORE_RTOL * np.maximum(np.abs(want), floor))


def test_cache_read_ranges():
    """Starts before, inside and far past the cache, more tokens than it holds, strides of a wider buffer."""
    case = Case(4, 2, 1, 300, 1, cap=320)
    lens = torch.tensor([300, 300, 300, 128], dtype=torch.int32, device="cuda")
    start = torch.tensor([-200, 299, 2 ** 31 - 10, 127], dtype=torch.int32, device="cuda")
    full = torch.zeros(4, 2, 320, D, device="cuda")
    Q.qjl_cache_read(case.ctx.handle, case.cache, 320, full, seqlens=torch.full_like(lens, 300))
    T = 777
    wide = torch.full((4, 2, T, 2, D), 5.0, device="cuda")
    Q.qjl_cache_read(case.ctx.handle, case.cache, T, K_out=wide[:, :, :, 1], t_start=start, seqlens=lens)
    want = torch.full_like(wide, 5.0)
    want[0, :, 200:500, 1] = full[0, :, :300]
    want[1, :, 0:1, 1] = full[1, :, 299:300]
    want[3, :, 0:1, 1] = full[3, :, 127:128]
    assert torch.equal(wide, want)
    Q.qjl_cache_read(case.ctx.handle, case.cache, 0, K_out=wide[:, :, :0, 1])  # nothing


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("kw", [{}, {"vbits": 2}, {"m": 512, "m_out": 256, "n_outlier": 32}, {"m": 96, "m_out": 0,
                                                                                              "n_outlier": 0}])
def test_commit_copies_every_section(kw):
    B, Hkv, N, cap = 4, 2, 20, 192
    case = Case(B, Hkv, 1, 100, N, cap=cap, **kw)
    path = torch.tensor([[0, 3, 4, 19, 7], [1, 2, 3, 4, 5], [5, 5, -1, 64, 2], [19, 18, 17, 16, 15]], dtype=torch.int32)
    acc = torch.tensor([4, 0, 9, 3], dtype=torch.int32)      # 9 is clamped to 5
    lens = torch.tensor([61, 100, 126, 190], dtype=torch.int32)
    out = torch.zeros(4, dtype=torch.int32, device="cuda")
    before = case.cache.tiles.clone()
    secs = ("kbits", "kbits_out", "knorm", "vcode", "vsz")
    want = {s: case.cache.section(s).clone() for s in secs}
    drafted = {s: case.draft.section(s) for s in secs}
    for b in range(B):
        for j in range(min(int(acc[b]), 5)):
            src, dst = int(path[b, j]), int(lens[b]) + j
            if 0 <= src < 64 and dst < cap:
                for s in secs:
                    want[s][b, :, dst] = drafted[s][b, :, src]
    Q.qjl_cache_commit(case.ctx.handle, case.cache, case.draft, path.cuda(), acc.cuda(), lens.cuda(), out)
    for s in secs:
        a, w = case.cache.section(s), want[s]
        assert torch.equal(a.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), s
    assert out.tolist() == [65, 100, 131, 192]
    assert torch.equal(case.cache.tiles[1], before[1])  # nothing accepted, nothing written
    Q.qjl_cache_commit(case.ctx.handle, case.cache, case.draft, path.cuda()[:, :0], acc.cuda(), lens.cuda(), out)
    assert out.tolist() == lens.tolist()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_speculative_step_equals_plain_decoding(dtype):
    """Rotate, sketch the drafts, attend over the tree, commit a path, and decode on: the same bytes and outputs as
    appending the accepted tokens one by one."""
    B, Hq, Hkv, T, N = 2, 8, 2, 190, 6
    w = I.Workload("t", B, Hq, Hkv, T, dtype="bf16" if dtype == torch.bfloat16 else "fp32")
    inp = I.make_inputs(w, seed=9, device="cpu", T=T + N)
    K, V = inp["K"].cuda(), inp["V"].cuda()
    g = torch.Generator().manual_seed(10)
    Qd = torch.randn(B, N, Hq, D, generator=g).to(dtype).cuda()
    parents = [-1, 0, 1, 1, 0, 4]
    mask, depth = [], []
    for i, p in enumerate(parents):
        mask.append((mask[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    table = Q.qjl_rope_init(base=500000.0)
    ctx = Q.QJLContext(0, D)
    caches = [ctx.allocate_cache(B, Hkv, T + N) for _ in range(2)]
    prefix = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    Kp = Q.qjl_rope(table, K[:, :, :T].contiguous(), positions=prefix)
    for c in caches:
        Q.qjl_quantize_keys(ctx.handle, c, Kp, Q.QJL_PREFILL, workspace=ctx.keys_workspace(B, Hkv))
        Q.qjl_quantize_values(ctx.handle, c, V[:, :, :T])
    spec, plain = caches
    pos = (T + torch.tensor(depth, dtype=torch.int32, device="cuda")).expand(B, N).contiguous()
    qr, kr = Q.qjl_rope(table, Qd.transpose(1, 2), K[:, :, T:], positions=pos)
    draft = spec.draft()
    Q.qjl_quantize_keys(ctx.handle, draft, kr, Q.QJL_APPEND)
    Q.qjl_quantize_values(ctx.handle, draft, V[:, :, T:])
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    out = torch.empty(B, N, Hq, D, dtype=dtype, device="cuda")
    mk = torch.tensor(mask, dtype=torch.int64, device="cuda").expand(B, N).contiguous()
    Q.qjl_tree_attention(ctx.handle, spec, draft, qr.transpose(1, 2), T, out, seqlens=lens, tree_mask=mk,
                         workspace=ctx.tree_workspace(B, N, Hq, Hkv))
    path = torch.tensor([[0, 1, 3], [0, 4, 5]], dtype=torch.int32, device="cuda")
    new = torch.empty_like(lens)
    Q.qjl_cache_commit(ctx.handle, spec, draft, path, torch.tensor([3, 3], dtype=torch.int32, device="cuda"), lens, new)
    assert new.tolist() == [T + 3, T + 3]
    # the same tokens one by one: rotated keys into the plain cache with decode steps
    ws = ctx.decode_workspace(B, Hq, Hkv, T + N)
    o = torch.empty(B, Hq, D, device="cuda")
    # bf16 outputs: within their own half step of the fp32 ones; fp32: what stands between the two is decode's
    # stated bound, C.OUT_ATOL absolute in every channel (its weights are split into two fp16 parts, its scores fixed
    # point), far above this operator's 64 u
    for j in range(3):
        pick = path[:, j].long()
        idx = torch.arange(B, device="cuda")
        kj, vj, qj = kr[idx, :, pick].contiguous(), V[:, :, T:][idx, :, pick].contiguous(), qr[idx, :, pick].contiguous()
        Q.qjl_decode_step(ctx.handle, plain, qj, kj, vj, T + j, o, workspace=ws)
        Q.qjl_decode_workspace_status(ctx.handle, ws, B, Hq, Hkv)
        got, want = C.to64(out[idx, pick]), C.to64(o)
        if dtype == torch.bfloat16:
            assert np.linalg.norm(got - want) <= B16 * np.linalg.norm(want), j
        else:
            assert np.abs(got - want).max() <= C.OUT_ATOL, j
    for s in ("kbits", "kbits_out", "knorm", "vcode", "vsz"):
        a, b = spec.section(s)[:, :, :T + 3], plain.section(s)[:, :, :T + 3]
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_steps_and_streams(dtype):
    """The whole step in a CUDA graph, replayed on changed inputs; two graphs with their own workspaces at once."""
    case = Case(2, 2, 4, 400, 6, dtype, cap=448)
    mask = torch.from_numpy(np.asarray(random_tree(2, 6, 3), dtype=np.uint64).view(np.int64)).cuda()
    table = Q.qjl_rope_init()
    h = case.ctx.handle
    lens = torch.tensor([400, 123], dtype=torch.int32, device="cuda")
    new = torch.zeros_like(lens)
    path = torch.tensor([[0, 2], [1, 3]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([2, 1], dtype=torch.int32, device="cuda")

    def step(q, out, ws, K, V):
        qr = Q.qjl_rope(table, q.transpose(1, 2), t_start=lens).transpose(1, 2)
        Q.qjl_tree_attention(h, case.cache, case.draft, qr, 400, out, seqlens=lens, tree_mask=mask, workspace=ws)
        Q.qjl_cache_read(h, case.draft, 6, K, V)
        Q.qjl_cache_commit(h, case.cache, case.draft, path, acc, lens, new)

    bufs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        q = torch.zeros_like(case.Q)
        bufs.append((q, torch.zeros_like(q), case.ctx.tree_workspace(2, 6, 8, 2),
                     torch.zeros(2, 2, 6, D, dtype=dtype, device="cuda"), torch.zeros(2, 2, 6, D, dtype=dtype, device="cuda")))
    step(*bufs[0])  # first launches outside capture
    torch.cuda.synchronize()
    for k in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=streams[k]):
            step(*bufs[k])
        graphs.append(gr)
    for r in range(3):
        qs = [(case.Q.float() * (1 + r) * (1 if k else -1)).to(dtype) for k in range(2)]
        want = []
        for k in range(2):
            ref = tuple(torch.zeros_like(x) for x in bufs[k])
            ref[0].copy_(qs[k])
            step(*ref)
            want.append(ref)
            bufs[k][0].copy_(qs[k])
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            for i in (1, 3, 4):
                assert torch.equal(bufs[k][i], want[k][i]), (r, k, i)
    assert new.tolist() == [402, 124]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("before", ["nothing", "copy", "memset", "kernel", "join", "decode", "tree"])
def test_tree_waits_for_what_came_before(before, captured):
    """The call's first kernel may start early: whatever precedes it on the stream is done before it reads or writes."""
    case = Case(2, 2, 4, 300, 4, cap=320)
    ws = case.ctx.tree_workspace(2, 4, 8, 2)
    q, out, alt = torch.empty_like(case.Q), torch.empty_like(case.Q), case.Q.float().mul(0.5).to(torch.bfloat16)
    lens, big = torch.empty(2, dtype=torch.int32, device="cuda"), torch.ones(1 << 26, device="cuda")
    dec_ws, o = case.ctx.decode_workspace(2, 8, 2, 320), torch.empty(2, 8, D, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    h = case.ctx.handle
    full = [300, 200]
    want = {"memset": case.tree(None, [0, 0]), "nothing": case.tree(None, full)}

    def call(src):
        if before == "copy":
            big.mul_(1.0)
            q.copy_(src)
        elif before == "memset":
            big.mul_(1.0)
            lens.zero_()
        elif before == "kernel":
            big.mul_(1.0)
            torch.mul(src, 1.0, out=q)
        elif before == "join":  # the last writer is on another stream
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.mul_(1.0)
                torch.mul(src, 1.0, out=q)
            torch.mul(alt, 1.0, out=out)
            torch.cuda.current_stream().wait_stream(side)
        elif before == "decode":  # of empty sequences: no block of it has work
            Q.qjl_decode_attention(h, case.cache, case.Q[:, 0].contiguous(), 300, o, seqlens=none, workspace=dec_ws)
        elif before == "tree":  # the same workspace and output, other queries
            Q.qjl_tree_attention(h, case.cache, case.draft, alt, 300, out, seqlens=lens, workspace=ws)
        Q.qjl_tree_attention(h, case.cache, case.draft, q, 300, out, seqlens=lens, workspace=ws)

    def reset():
        late = before in ("copy", "kernel", "join")
        q.zero_() if late else q.copy_(case.Q)
        lens.copy_(torch.tensor(full, dtype=torch.int32))
        out.fill_(float("nan"))

    reset()
    call(case.Q)
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(case.Q)
    for _ in range(4):
        reset()
        torch.cuda.synchronize()
        graph.replay() if captured else call(case.Q)
        torch.cuda.synchronize()
        assert torch.equal(out, want.get(before, want["nothing"]))


def test_refusals_on_the_gpu():
    case = Case(2, 2, 4, 100, 4)
    h, c, d, q = case.ctx.handle, case.cache, case.draft, case.Q
    ws, out = case.ctx.tree_workspace(2, 4, 8, 2), torch.zeros_like(case.Q)
    call = lambda **k: Q.qjl_tree_attention(h, k.get("c", c), k.get("d", d), k.get("q", q), k.get("T", 100),  # noqa: E731
                                            k.get("o", out), workspace=k.get("ws", ws), tree_mask=k.get("mask"))
    with pytest.raises(Q.QJLError, match="WORKSPACE"):
        call(ws=ws[:-256])
    with pytest.raises(Q.QJLError, match="WORKSPACE"):
        call(ws=None)
    with pytest.raises(Q.QJLError, match="T must be"):
        call(T=c.cap + 1)
    with pytest.raises(Q.QJLError, match="UNSUPPORTED"):
        call(q=q[:, :, :6], o=out[:, :, :6].contiguous())   # g = 3
    with pytest.raises(Q.QJLError, match="B and Hkv"):
        one = case.ctx.allocate_cache(2, 1, 64)
        call(d=one)
    with pytest.raises(Q.QJLError, match="N must be"):
        call(q=torch.zeros(2, 65, 8, D, dtype=torch.bfloat16, device="cuda"),
             o=torch.zeros(2, 65, 8, D, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(mask=torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        call(o=out.float())
    with pytest.raises(ValueError):
        call(o=out.transpose(1, 2).contiguous().transpose(1, 2))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    path = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(Q.QJLError, match="overlaps"):
        Q.qjl_cache_commit(h, c, d, path, lens, lens, lens)
    with pytest.raises(Q.QJLError, match="share"):
        Q.qjl_cache_commit(h, c, c, path, lens, lens)
    with pytest.raises(ValueError):
        Q.qjl_cache_read(h, c, 4)
    with pytest.raises(Q.QJLError, match="overlap"):
        Q.qjl_cache_read(h, c, 4, K_out=torch.zeros(1, 2, 4, D, device="cuda").expand(2, 2, 4, D))
    torch.cuda.synchronize()
    assert int(out.count_nonzero()) == 0  # nothing was launched
