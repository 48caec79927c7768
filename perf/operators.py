"""The operators of a speculative decode step over the QJL cache, in plain torch and through the library.

A step of speculative decoding with this library rotates the drafted tokens' queries and keys
(`rope`), sketches the drafts into a one-tile draft cache, attends from every drafted token to the
committed cache and to its ancestors among the drafts (`tree`), and copies the accepted drafts into the
cache (`commit`). `read` gives a stretch of the cache back as dense keys and values.

    y       = x rotated by position * f_i in plane i of the rotated dims               (rope)
    K^      = sqrt(pi/2)/m |k_in| S^T sign_in on the inlier channels,
              sqrt(pi/2)/m_out |k_out| S_out^T sign_out on the outlier ones,
    V^      = zero + code * scale                                                       (read)
    O_i     = softmax_t(sm_scale <q_i, K^_t>) V^_t over the committed tokens and the
              drafted tokens that bit t of mask_i allows                                (tree)
    slot (len_b + j) of the cache = slot path_bj of the draft cache, j < accepted_b     (commit)

With `own` false `run` computes these in elementary fp32 torch operations (fp64 for the angles); with
`own` true it calls the library. `exact` computes them in fp64 from the formulas above.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

D = 128           # head dimension
TILE = 64         # tokens of a cache tile
SKETCH_SEED = 0


# ------------------------------------------------------------------ cases

def _tree(name, B, N, Hq, Hkv, T, m=256, m_out=64, n_outlier=8, vbits=4, dtype="bf16", ragged=False):
    return {"name": name, "op": "tree", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "T": T, "m": m, "m_out": m_out,
            "n_outlier": n_outlier, "vbits": vbits, "dtype": dtype, "ragged": ragged}


def _read(name, B, Hkv, T, start, m=256, m_out=64, n_outlier=8, vbits=4, dtype="bf16", ragged=False):
    return {"name": name, "op": "read", "B": B, "Hkv": Hkv, "T": T, "start": start, "m": m, "m_out": m_out,
            "n_outlier": n_outlier, "vbits": vbits, "dtype": dtype, "ragged": ragged}


def _rope(name, B, Hq, Hkv, T, pos0, rot=D, interleaved=False, scaled=False, inverse=False, dtype="bf16"):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "pos0": pos0, "rot": rot,
            "interleaved": interleaved, "scaled": scaled, "inverse": inverse, "dtype": dtype}


def _commit(name, B, Hkv, T, A, m=256, m_out=64, n_outlier=8, vbits=4):
    return {"name": name, "op": "commit", "B": B, "Hkv": Hkv, "T": T, "A": A, "m": m, "m_out": m_out,
            "n_outlier": n_outlier, "vbits": vbits}


def listed():
    return [
        # a chat's first drafts: one short sequence, a small tree, every head its own kv head
        _tree("tree_short", 1, 5, 32, 32, 130),
        # a serving batch of grouped-query heads with ragged lengths and trees of up to 13 drafts
        _tree("tree_serving", 16, 13, 32, 8, 8192, ragged=True),
        # one long conversation, the widest tree
        _tree("tree_wide", 1, 64, 32, 32, 32768),
        # four contexts of 131072 tokens, 16 drafts each: the bandwidth-bound end, and the largest case
        _tree("tree_long", 4, 16, 32, 8, 131072),
        # an fp32 model, eight query heads on one kv head, 2-bit values
        _tree("tree_fp32", 2, 7, 8, 1, 1024, n_outlier=4, vbits=2, dtype="fp32", ragged=True),
        # a shared prefix handed to a dense consumer (a chunked prefill): the whole of four long caches
        _read("read_prefix", 4, 8, 32768, 0),
        # an odd window of a 2-bit cache with the widest sketch, in fp32, ragged
        _read("read_window", 3, 8, 2049, 777, m=512, vbits=2, dtype="fp32", ragged=True),
        # the new token of a decode batch
        _rope("rope_decode", 16, 32, 8, 1, 8192),
        # a prefill of one long context, wavelengths stretched by parts, interleaved pairs in part of the head
        _rope("rope_prefill", 1, 32, 32, 32768, 0, rot=64, interleaved=True, scaled=True),
        # the gradient of the rotation for an fp32 model, far positions
        _rope("rope_inverse", 2, 32, 8, 1021, 1000003, inverse=True, dtype="fp32"),
        # one sequence's accepted drafts, and a serving batch's
        _commit("commit_one", 1, 32, 4096, 4),
        _commit("commit_batch", 64, 8, 2048, 16),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "read", "rope", "commit"])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    g = rng.choice([1, 2, 4, 8]) if Hkv <= 8 else 1
    m, m_out, n_out = rng.choice([(256, 64, 8), (256, 64, 8), (128, 64, 8), (512, 64, 8), (256, 32, 4), (96, 0, 0)])
    vbits = rng.choice([4, 4, 2])
    if op == "tree":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        B = rng.choice([1, 2, 3, 7, 16])
        N = _log_between(rng, 1, 64)
        # the largest listed case has 4.2 million cached tokens times kv heads, with 64 rows each
        most = min(131072, (1 << 21) // (B * Hkv) if dtype == "bf16" else 4096, (1 << 26) // (B * Hkv * g * N))
        return _drop(_tree("", B, N, Hkv * g, Hkv, _log_between(rng, 1, most), m, m_out, n_out, vbits, dtype,
                           rng.random() < 0.5))
    if op == "read":
        B = rng.choice([1, 2, 3, 5])
        T = _log_between(rng, 1, min(65536, (1 << 20) // (B * Hkv)))
        return _drop(_read("", B, Hkv, T, rng.choice([0, 1, 63, 500]), m, m_out, n_out, vbits,
                           rng.choice(["bf16", "fp32"]), rng.random() < 0.5))
    if op == "rope":
        B = rng.choice([1, 2, 8, 16])
        T = _log_between(rng, 1, max(2, (1 << 21) // (B * Hkv * (g + 1))) if B * Hkv > 8 else 32768)
        return _drop(_rope("", B, Hkv * g, Hkv, T, rng.choice([0, 17, 100000, 1000000]),
                           rng.choice([128, 128, 64, 32, 96]), rng.random() < 0.5, rng.random() < 0.5,
                           rng.random() < 0.3, rng.choice(["bf16", "fp32"])))
    B = rng.choice([1, 3, 16, 64])
    return _drop(_commit("", B, Hkv, _log_between(rng, 130, max(131, min(8192, (1 << 20) // (B * Hkv)))),
                         rng.randint(1, 64), m, m_out, n_out, vbits))


def _drop(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ sizes

def _tile_sections(m, m_out, vbits):
    """name -> (offset, bytes) of a 64-token tile, and the tile's size."""
    sizes = [("kbits", TILE * m // 8), ("kbits_out", TILE * m_out // 8), ("knorm", TILE * 4),
             ("vcode", (D // 4) * (TILE + 4) if vbits == 2 else TILE * D // 2), ("vsz", TILE * D // 8)]
    out, off = {}, 0
    for name, n in sizes:
        out[name] = (off, n)
        off += n
    return out, off


def _lens(case):
    """Committed tokens of each sequence (for `read`: those from `start` on)."""
    T, B = case["T"], case["B"]
    return [T - (b * T) // (2 * B) if case.get("ragged") else T for b in range(B)]


def _drafts(case):
    """Drafted tokens of each sequence."""
    return [max(1, case["N"] - b % 4) if case["ragged"] else case["N"] for b in range(case["B"])]


def _token_bytes(case):
    return case["m"] // 8 + case["m_out"] // 8 + 4 + (D // 2 if case["vbits"] == 4 else D // 4) + D // 8


def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * (case["Hq"] + case["Hkv"]) * case["T"]
        return {"bytes": n * D * es * 2 + case["B"] * case["T"] * 4, "flops": n * case["rot"] * 3}
    if case["op"] == "commit":
        moved = sum(_accepted(case))
        return {"bytes": moved * case["Hkv"] * _token_bytes(case) * 2 + 12 * case["B"], "flops": 0}
    p = case["m"] + case["m_out"]
    if case["op"] == "read":
        # the outlier channels take the m_out part, the others the m part
        per = 2 * (case["m"] * (D - case["n_outlier"]) + case["m_out"] * case["n_outlier"]) + 2 * D
        n = sum(_lens(case)) * case["Hkv"]
        return {"bytes": n * (_token_bytes(case) + 2 * D * es), "flops": n * per}
    flops = nbytes = 0
    g = case["Hq"] // case["Hkv"]
    for n, nd in zip(_lens(case), _drafts(case)):
        rows = nd * g
        # scores from the projected queries, or from keys read back once for all rows: the cheaper
        per = min(rows * p, D * p + rows * D) + rows * D
        flops += case["Hkv"] * (n + nd) * 2 * per
        nbytes += case["Hkv"] * (n + nd) * _token_bytes(case) + nd * case["Hq"] * D * es * 2
    return {"bytes": nbytes, "flops": flops}


def _accepted(case):
    return [(case["A"] * (b + 1) + b) % (case["A"] + 1) if case["B"] > 1 else case["A"] for b in range(case["B"])]


# ------------------------------------------------------------------ inputs

def _splitmix_normal(rows, offset):
    """The library's sketch matrix of seed SKETCH_SEED: SplitMix64 counters, Box-Muller, rounded to bf16."""
    e = np.arange(rows * D, dtype=np.uint64)
    u = []
    with np.errstate(over="ignore"):
        for k in (1, 2):
            z = np.uint64(SKETCH_SEED) + (np.uint64(offset) + np.uint64(2) * e + np.uint64(k)) * np.uint64(0x9E3779B97F4A7C15)
            z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
            z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
            z = z ^ (z >> np.uint64(31))
            u.append(((z >> np.uint64(12)).astype(np.float64) + 0.5) * 2.0 ** -52)
    x = np.sqrt(-2.0 * np.log(u[0])) * np.cos(6.283185307179586 * u[1])
    return torch.from_numpy(x).to(torch.bfloat16).reshape(rows, D)


def _sketches(case):
    return (_splitmix_normal(case["m"], 0).cuda(), _splitmix_normal(case["m_out"], 1 << 62).cuda())


def _pack_bits(y):
    """Sign bits [..., n] as bytes [..., n / 8], bit i of byte k for row 8k + i."""
    b = (y >= 0).to(torch.uint8).unflatten(-1, (-1, 8))
    w = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.uint8, device=y.device)
    return (b * w).sum(-1, dtype=torch.uint8)


def _make_tiles(case, gen, B, T, S, So, idx):
    """Cache tiles [B, Hkv, ceil(T / 64), tile bytes] of random tokens; K ~ N(0,1) with x20 outlier channels."""
    Hkv, m_out, vbits = case["Hkv"], case["m_out"], case["vbits"]
    nt = -(-T // TILE)
    sec, size = _tile_sections(case["m"], m_out, vbits)
    tiles = torch.zeros(B, Hkv, nt, size, dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Hkv, 1, D, dtype=torch.bool, device="cuda").scatter_(3, idx[:, :, None, :], True)
    step = max(1, (1 << 19) // (TILE * nt))  # heads at a time
    for b in range(B):
        for h in range(0, Hkv, step):
            hs = slice(h, min(h + step, Hkv))
            n = hs.stop - hs.start
            K = torch.randn(n, nt * TILE, D, generator=gen, device="cuda")
            K = torch.where(out[b, hs], 20.0 * K, K).bfloat16().float()
            k_in, k_out = K.masked_fill(out[b, hs], 0.0), K.masked_fill(~out[b, hs], 0.0)
            V = torch.randn(n, nt * TILE, 4, 32, generator=gen, device="cuda").bfloat16().float()

            def put(name, x):
                o, nb = sec[name]
                tiles[b, hs, :, o:o + nb] = x.contiguous().view(torch.uint8).reshape(n, nt, -1)

            put("kbits", _pack_bits(k_in @ S.float().T))
            if m_out:
                put("kbits_out", _pack_bits(k_out @ So.float().T))
            put("knorm", torch.stack([k_in.norm(dim=-1), k_out.norm(dim=-1)], -1).half())
            lo, hi = V.amin(-1), V.amax(-1)
            zero, scale = lo.half(), ((hi - lo) / (2 ** vbits - 1)).half()
            code = ((V - zero.float()[..., None]) / scale.float()[..., None]).round().clamp(0, 2 ** vbits - 1)
            code = code.to(torch.uint8)
            put("vsz", torch.stack([scale, zero], -1))
            if vbits == 4:
                c = code.unflatten(-1, (16, 2))
                c = c[..., 0] | (c[..., 1] << 4)                       # [n, t, 4 groups, 16 bytes]
                j = torch.arange(nt * TILE, device="cuda") % TILE
                chunk = torch.arange(4, device="cuda")[None] ^ ((j[:, None] >> 1) & 3)
                put("vcode", torch.empty_like(c).scatter_(2, chunk[None, :, :, None].expand_as(c), c))
            else:
                c = code.unflatten(-1, (8, 4))
                c = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
                c = c.reshape(n, nt, TILE, D // 4).transpose(2, 3)      # [n, tile, line, token]
                put("vcode", torch.nn.functional.pad(c, (0, 4)))
    return tiles


def _channels(case, gen):
    """Outlier channels [B, Hkv, n_outlier], ascending."""
    r = torch.rand(case["B"], case["Hkv"], D, generator=gen, device="cuda")
    return r.argsort(-1)[..., :case["n_outlier"]].sort(-1).values


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        B, T = case["B"], case["T"]
        for name, H in (("Q", case["Hq"]), ("K", case["Hkv"])):
            x = torch.randn(B, T, H, D, generator=gen, device="cuda").to(_dtype(case))
            s[name] = x.transpose(1, 2)              # [B, H, T, d] as a model's projection leaves it
            s[name + "_out"] = torch.zeros_like(x).transpose(1, 2)
        jitter = torch.randint(0, 64, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = (case["pos0"] + jitter + torch.arange(T, device="cuda", dtype=torch.int32)[None]).contiguous()
        if own:
            from decode_attention_qjl_b200 import qjl as lib
            s["table"] = lib.qjl_rope_init(**_rope_args(case))
        return s
    B, Hkv, T = case["B"], case["Hkv"], case["T"]
    s["S"], s["So"] = _sketches(case)
    s["idx"] = _channels(case, gen)
    slots = T + (case.get("A") or 0) + case.get("start", 0)
    s["tiles"] = _make_tiles(case, gen, B, slots, s["S"], s["So"], s["idx"])
    s["lens"] = _i32([n + case.get("start", 0) for n in _lens(case)])
    if case["op"] in ("tree", "commit"):
        s["draft"] = _make_tiles(case, gen, B, TILE, s["S"], s["So"], s["idx"])
    if case["op"] == "tree":
        N = case["N"]
        s["Q"] = torch.randn(B, N, case["Hq"], D, generator=gen, device="cuda").to(_dtype(case))
        s["O"] = torch.zeros_like(s["Q"])
        s["n_draft"] = _i32(_drafts(case))
        # a random tree: draft i hangs below an earlier one or below the committed context
        r = torch.rand(B, N, generator=gen, device="cuda").cpu()
        mask = torch.zeros(B, N, dtype=torch.int64)
        for i in range(N):
            parent = (r[:, i] * (i + 1)).floor().long() - 1
            above = torch.where(parent >= 0, mask.gather(1, parent.clamp(min=0)[:, None])[:, 0], 0)
            mask[:, i] = above | (1 << i if i < 63 else -(1 << 63))
        s["mask"] = mask.cuda()
    elif case["op"] == "read":
        s["start"] = _i32([case["start"]] * B)
        for name in ("K_out", "V_out"):
            s[name] = torch.zeros(B, Hkv, T, D, dtype=_dtype(case), device="cuda")
    else:
        A = case["A"]
        s["path"] = torch.rand(B, TILE, generator=gen, device="cuda").argsort(-1)[:, :A].sort(-1).values.int().contiguous()
        s["accepted"] = _i32(_accepted(case))
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        from decode_attention_qjl_b200 import qjl as lib
        s["ctx"] = lib.QJLContext(SKETCH_SEED, D, case["m"], case["m_out"], case["n_outlier"], case["vbits"])
        idx = s["idx"].int().contiguous() if case["n_outlier"] else _i32([0] * (B * Hkv)).view(B, Hkv, 1)
        for name in ("tiles", "draft"):
            if name in s:
                s[name + "_cache"] = lib.QJLCache(idx, s[name], B, Hkv, s[name].shape[2] * TILE, case["m"],
                                                  case["m_out"], case["vbits"])
        if case["op"] == "tree":
            s["ws"] = s["ctx"].tree_workspace(B, case["N"], case["Hq"], Hkv)
    return s


def _rope_args(case):
    a = {"rot_dim": case["rot"], "base": 500000.0 if case["scaled"] else 10000.0, "interleaved": case["interleaved"]}
    if case["scaled"]:
        a.update(factor=8.0, original_len=8192, low=1.0, high=4.0, amplitude=1.0 + 0.1 * math.log(8.0))
    return a


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _run_own(case, s)
    return {"tree": _plain_tree, "read": _plain_read, "rope": _plain_rope, "commit": _plain_commit}[case["op"]](case, s)


def _run_own(case, s):
    from decode_attention_qjl_b200 import qjl as lib
    if case["op"] == "rope":
        return list(lib.qjl_rope(s["table"], s["Q"], s["K"], positions=s["pos"], Q_out=s["Q_out"], K_out=s["K_out"],
                                 inverse=case["inverse"]))
    h = s["ctx"].handle
    if case["op"] == "tree":
        return lib.qjl_tree_attention(h, s["tiles_cache"], s["draft_cache"], s["Q"], case["T"], s["O"],
                                      seqlens=s["lens"], n_draft=s["n_draft"], tree_mask=s["mask"], workspace=s["ws"])
    if case["op"] == "read":
        return list(lib.qjl_cache_read(h, s["tiles_cache"], case["T"], K_out=s["K_out"], V_out=s["V_out"],
                                       t_start=s["start"], seqlens=s["lens"]))
    lib.qjl_cache_commit(h, s["tiles_cache"], s["draft_cache"], s["path"], s["accepted"], s["lens"], s["new_lens"])
    return [s["tiles"], s["new_lens"]]


def _section(tiles, case, name, n):
    """Bytes of one section, tokens in order: [..., n, bytes] of tiles [..., tile, bytes] (n tokens)."""
    o, nb = _tile_sections(case["m"], case["m_out"], case["vbits"])[0][name]
    x = tiles[..., o:o + nb].unflatten(-1, (D // 4, TILE + 4))[..., :TILE].transpose(-1, -2) \
        if name == "vcode" and case["vbits"] == 2 else tiles[..., o:o + nb].unflatten(-1, (TILE, nb // TILE))
    return x.flatten(-3, -2)[..., :n, :]


def _bits_to_signs(b):
    """Bytes [..., n] -> fp32 +1 / -1 [..., 8 n]."""
    shift = torch.arange(8, dtype=torch.uint8, device=b.device)
    return (((b[..., None] >> shift) & 1).float() * 2.0 - 1.0).flatten(-2)


def _plain_values(tiles, case, n):
    c = _section(tiles, case, "vcode", n)
    if case["vbits"] == 4:
        j = torch.arange(n, device=c.device) % TILE
        chunk = torch.arange(4, device=c.device)[None] ^ ((j[:, None] >> 1) & 3)
        c = c.unflatten(-1, (4, 16))
        c = torch.gather(c, -2, chunk[..., None].expand(c.shape))
        code = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    else:
        code = torch.stack([(c >> (2 * k)) & 3 for k in range(4)], -1).flatten(-2).unflatten(-1, (4, 32))
    sz = _section(tiles, case, "vsz", n).contiguous().view(torch.float16).float().unflatten(-1, (4, 2))
    return (sz[..., 1:] + code.float() * sz[..., :1]).flatten(-2)


def _plain_signs(tiles, case, n):
    """Sign rows scaled by the estimator's factors: [..., n, m + m_out] in fp32."""
    norm = _section(tiles, case, "knorm", n).contiguous().view(torch.float16).float()
    c = math.sqrt(math.pi / 2)
    return torch.cat([_bits_to_signs(_section(tiles, case, "kbits", n)) * (norm[..., :1] * (c / case["m"])),
                      _bits_to_signs(_section(tiles, case, "kbits_out", n)) * (norm[..., 1:] * (c / max(case["m_out"], 1)))], -1)


def _outlier_mask(idx):
    return torch.zeros(*idx.shape[:-1], D, dtype=torch.bool, device=idx.device).scatter_(-1, idx, True)


def _plain_tree(case, s):
    B, N, Hq, Hkv, T = case["B"], case["N"], case["Hq"], case["Hkv"], case["T"]
    g = Hq // Hkv
    out = _outlier_mask(s["idx"])[:, :, None]                                            # [B, Hkv, 1, d]
    q = s["Q"].float().unflatten(2, (Hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)       # [B, Hkv, N g, d]
    sq = torch.cat([q.masked_fill(out, 0.0) @ s["S"].float().T, q.masked_fill(~out, 0.0) @ s["So"].float().T], -1)
    sq = sq * (1.0 / math.sqrt(D))
    bit = torch.arange(N, device="cuda")
    live = bit < s["n_draft"][:, None]                                                   # [B, N]
    allow = ((s["mask"][:, :, None] >> bit) & 1).bool() & live[:, None, :]               # [B, N, N]
    allow = allow[:, None].repeat_interleave(g, 2)
    there = (torch.arange(T, device="cuda") < s["lens"][:, None])[:, None, None]         # [B, 1, 1, T]
    x = torch.cat([(sq @ _plain_signs(s["tiles"], case, T).transpose(-1, -2)).masked_fill(~there, -math.inf),
                   (sq @ _plain_signs(s["draft"], case, N).transpose(-1, -2)).masked_fill(~allow, -math.inf)], -1)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = p @ torch.cat([_plain_values(s["tiles"], case, T), _plain_values(s["draft"], case, N)], -2)
    o = (o / p.sum(-1, keepdim=True)).unflatten(2, (N, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["O"].copy_(o.masked_fill(~live[:, :, None, None], 0.0))
    return s["O"]


def _plain_read(case, s):
    a, T = case["start"], case["T"]
    sg = _plain_signs(s["tiles"], case, a + T)[:, :, a:]
    k = torch.where(_outlier_mask(s["idx"])[:, :, None], sg[..., case["m"]:] @ s["So"].float(),
                    sg[..., :case["m"]] @ s["S"].float())
    v = _plain_values(s["tiles"], case, a + T)[:, :, a:]
    there = (a + torch.arange(T, device="cuda") < s["lens"][:, None])[:, None, :, None]
    for x, y in ((k, s["K_out"]), (v, s["V_out"])):
        y.copy_(torch.where(there, x.to(y.dtype), y))
    return [s["K_out"], s["V_out"]]


def _frequencies(case):
    """Angle per position (radians) of each rotated plane, and the amplitude."""
    a = _rope_args(case)
    f = a["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    if "factor" in a:
        r = a["original_len"] * f / (2 * math.pi)  # turns within the original length
        keep = ((r - a["low"]) / (a["high"] - a["low"])).clamp(0, 1)
        f = f * keep + f / a["factor"] * (1 - keep)
    return f.cuda(), a.get("amplitude", 1.0)


def _plain_rope(case, s):
    f, amp = _frequencies(case)
    ang = s["pos"].double()[:, None, :, None] * f
    sign = -1.0 if case["inverse"] else 1.0
    cos, sin = (torch.cos(ang) * amp).float(), (torch.sin(ang) * (amp * sign)).float()
    rot = case["rot"]
    for name in ("Q", "K"):
        x, y = s[name].float(), s[name + "_out"]
        head, rest = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            u, v = head[..., 0::2], head[..., 1::2]
            r = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        else:
            u, v = head[..., :rot // 2], head[..., rot // 2:]
            r = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        y.copy_(torch.cat([r, rest], -1))
    return [s["Q_out"], s["K_out"]]


def _plain_commit(case, s):
    A, B = case["A"], case["B"]
    j = torch.arange(A, device="cuda")
    pos = s["lens"].long()[:, None] + j                        # [B, A]
    keep = (j < s["accepted"][:, None])[:, :, None, None]
    bi = torch.arange(B, device="cuda")[:, None]
    src = s["path"].long()
    for name in _tile_sections(case["m"], case["m_out"], case["vbits"])[0]:
        o, nb = _tile_sections(case["m"], case["m_out"], case["vbits"])[0][name]
        if nb == 0:
            continue
        if name == "vcode" and case["vbits"] == 2:
            to = s["tiles"][..., o:o + nb].unflatten(-1, (D // 4, TILE + 4)).transpose(-1, -2)
            of = s["draft"][..., o:o + nb].unflatten(-1, (D // 4, TILE + 4)).transpose(-1, -2)
        else:
            to = s["tiles"][..., o:o + nb].unflatten(-1, (TILE, nb // TILE))
            of = s["draft"][..., o:o + nb].unflatten(-1, (TILE, nb // TILE))
        old = to[bi, :, pos // TILE, pos % TILE]               # [B, A, Hkv, bytes]
        row = of[bi, :, 0, src]
        if name == "vcode" and case["vbits"] == 4:             # each slot keeps its 16-byte chunks in its own order
            order = torch.arange(4, device="cuda") ^ (((pos % TILE // 2) ^ (src // 2)) & 3)[..., None]
            row = row.unflatten(-1, (4, 16))
            row = row.gather(3, order[:, :, None, :, None].expand(row.shape)).flatten(-2)
        to[bi, :, pos // TILE, pos % TILE] = torch.where(keep, row, old)
    torch.add(s["lens"], s["accepted"], out=s["new_lens"])
    return [s["tiles"], s["new_lens"]]


# ------------------------------------------------------------------ the definitions in fp64

def _exact_kv(tiles, case, idx, S, So, n):
    """Keys and values that a cache slab [tiles, bytes] of one (sequence, kv head) stands for, in fp64."""
    m, m_out, vb = case["m"], case["m_out"], case["vbits"]
    nt = -(-n // TILE)
    tiles = tiles[:nt]
    o = 0

    def take(width):
        nonlocal o
        x = tiles[:, o:o + TILE * width].reshape(nt * TILE, width)[:n]
        o += TILE * width
        return x

    def signs(x, rows):
        i = torch.arange(rows, device=x.device)
        return torch.where((x[:, i // 8].int() >> (i % 8).int()) % 2 == 1, 1.0, -1.0).double()

    s_in, s_out = signs(take(m // 8), m), signs(take(m_out // 8), m_out)
    norm = take(4).contiguous().view(torch.float16).double()
    i = torch.arange(D, device=tiles.device)
    if vb == 4:
        raw = take(D // 2)
        t = torch.arange(n, device=tiles.device)[:, None]
        byte = 16 * ((i // 32) ^ ((t % TILE) // 2 % 4)) + (i % 32) // 2
        code = torch.gather(raw, 1, byte).int() // torch.where(i % 2 == 1, 16, 1) % 16
    else:
        raw = tiles[:, o:o + D // 4 * (TILE + 4)].reshape(nt, D // 4, TILE + 4)
        o += D // 4 * (TILE + 4)
        t = torch.arange(n, device=tiles.device)
        code = raw[t // TILE][torch.arange(n, device=t.device), :, t % TILE][:, i // 4].int() // 4 ** (i % 4) % 4
    sz = take(D // 8).contiguous().view(torch.float16).double().reshape(n, 4, 2)
    V = sz[:, i // 32, 1] + code.double() * sz[:, i // 32, 0]
    K = math.sqrt(math.pi / 2) / m * norm[:, :1] * (s_in @ S.double())
    if m_out:
        K[:, idx] = math.sqrt(math.pi / 2) / m_out * norm[:, 1:] * (s_out @ So.double()[:, idx])
    return K, V


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "commit":
        return None
    if case["op"] == "rope":
        f, amp = _exact_frequencies(case)
        rot, outs = case["rot"], []
        z = torch.polar(torch.full_like(f, amp).expand(case["B"], case["T"], -1), s["pos"].double()[..., None] * f)
        z = (z.conj() if case["inverse"] else z)[:, None]
        for name in ("Q", "K"):
            y = s[name].double().clone()
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            w = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * z
            y[..., a], y[..., b] = w.real, w.imag
            outs.append(y)
        return outs
    B, Hkv, lens = case["B"], case["Hkv"], _lens(case)
    if case["op"] == "read":
        Ko = torch.zeros(B, Hkv, case["T"], D, dtype=torch.float64, device="cuda")
        Vo = torch.zeros_like(Ko)
        for b in range(B):
            for h in range(Hkv):
                K, V = _exact_kv(s["tiles"][b, h], case, s["idx"][b, h], s["S"], s["So"], case["start"] + lens[b])
                Ko[b, h, :lens[b]], Vo[b, h, :lens[b]] = K[case["start"]:], V[case["start"]:]
        return [Ko, Vo]
    O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    g = case["Hq"] // Hkv
    for b, nd in enumerate(_drafts(case)):
        ok = torch.tensor([[(int(w) >> t) & 1 for t in range(nd)] for w in s["mask"][b, :nd].tolist()], device="cuda") == 1
        for h in range(Hkv):
            K, V = _exact_kv(s["tiles"][b, h], case, s["idx"][b, h], s["S"], s["So"], lens[b])
            Kd, Vd = _exact_kv(s["draft"][b, h], case, s["idx"][b, h], s["S"], s["So"], nd)
            q = s["Q"][b, :nd, h * g:(h + 1) * g].double() / math.sqrt(D)                # [nd, g, d]
            x = torch.cat([q @ K.T, torch.where(ok[:, None, :], q @ Kd.T, -math.inf)], -1)
            O[b, :nd, h * g:(h + 1) * g] = torch.softmax(x, -1) @ torch.cat([V, Vd])
    return O


def _exact_frequencies(case):
    a = _rope_args(case)
    f = []
    for i in range(case["rot"] // 2):
        w = math.exp(-2 * i / case["rot"] * math.log(a["base"]))
        if "factor" in a:
            r = a["original_len"] * w / (2 * math.pi)
            t = min(1.0, max(0.0, (r - a["low"]) / (a["high"] - a["low"])))
            w = (1 - t) * w / a["factor"] + t * w
        f.append(w)
    return torch.tensor(f, dtype=torch.float64, device="cuda"), a.get("amplitude", 1.0)
