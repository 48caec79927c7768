// Dense keys and values of cached tokens.
//
// K_hat = sqrt(pi/2)/m |k_in| S^T sign_in on the inlier channels, the same of
// the outlier sketch on the outlier ones; V_hat = zero + code * scale. The key
// sums of 128 tokens are two products on the tensor cores,
//   D_in [token, channel] = signs_in [token, m] S [m, channel], D_out likewise,
// with +-1 in bf16, so every product is exact, the sums are fp32 and no pair
// needs an operand of its own: which of the two a channel takes, and the norm,
// are applied on the way out.
//
// Bound: HBM, 124 bytes read and 512 (bf16) written per token at m = 256; the
// products take 1300 of the 3500 SM cycles that this costs per 128 tokens. One
// block per SM, S and S_out in shared memory once (a K row per projection, 128
// channels, MN-major with 128-byte swizzle), and the roles
//   warps 0-7   sign words (global) -> tensor memory, lane = token, every other
//               pair of its words
//   warps 8-15  value codes (global) -> V_out, thread = half a token
//   warps 16-23 sums (tensor memory) -> K_out, lane = token, half of its channels
//   warp 24     issues the products
// Units of 128 token slots are dealt round robin. The output warps own a token
// per lane; 32 rows written by 32 lanes, a sector each, took 3.8 SM cycles per
// sector (208 us for 1 M token-heads, bf16), so they turn a piece of their rows
// through shared memory and write 128 bytes of a row with eight lanes.
// Measured, 1 M token-heads, m = 256, bf16: 186 us, 3.6 TB/s, on inputs that change
// from call to call, 167 us in a row on unchanged ones (HBM's rate would take 102);
// the roles' 13900 warp instructions per unit use two thirds of the issue slots.
// Values alone take 80 us.
#include "tc_common.cuh"

namespace qjl {
namespace {

using namespace tc;

constexpr int kReadUnit = 128;
constexpr int kReadThreads = 32 * 25;
constexpr int kReadWords = 4;                // sign words of a chunk: 64 tensor-memory columns
constexpr int kReadColOut = 256, kReadColA = 384;  // two D_in at 0 and 128, D_out, two sign chunks
constexpr int kReadMisc = 1024;

// The block's units: unit = pair * upb + k, dealt round robin.
struct ReadUnit {
  int unit, pair, k, step_pair, step_k;
  int64_t bh;
  int b, h, slot0;  // first token slot (a multiple of 128)
  int lo, hi;       // slots to give back
  int start;        // position of token 0
  // the first unit that has something to give back; false: none is left
  __device__ bool begin(const ReadParams& p, int upb, int n_units) {
    step_pair = static_cast<int>(gridDim.x) / upb;
    step_k = static_cast<int>(gridDim.x) - step_pair * upb;
    unit = blockIdx.x;
    pair = unit / upb;
    k = unit - pair * upb;
    load(p);
    return find(p, upb, n_units);
  }
  __device__ bool next(const ReadParams& p, int upb, int n_units) {
    advance(p, upb, n_units);
    return find(p, upb, n_units);
  }
  __device__ bool find(const ReadParams& p, int upb, int n_units) {
    while (unit < n_units) {
      slot0 = (lo / kReadUnit + k) * kReadUnit;
      if (lo < hi && slot0 >= 0 && slot0 < hi) return true;  // (not past the range, nor wrapped by a start near 2^31)
      advance(p, upb, n_units);
    }
    return false;
  }
  __device__ void advance(const ReadParams& p, int upb, int n_units) {
    unit += gridDim.x;
    const int before = pair;
    pair += step_pair;
    k += step_k;
    if (k >= upb) {
      k -= upb;
      ++pair;
    }
    if (pair != before && unit < n_units) load(p);
  }
  __device__ void load(const ReadParams& p) {
    bh = pair;
    b = pair / p.Hkv;
    h = pair - b * p.Hkv;
    start = p.t_start ? __ldg(p.t_start + b) : 0;
    const int lim = p.seqlens ? min(max(__ldg(p.seqlens + b), 0), p.cap) : p.cap;
    lo = max(start, 0);
    hi = static_cast<int>(min(static_cast<int64_t>(start) + p.T, static_cast<int64_t>(lim)));
  }
  __device__ bool live(int tt) const { return slot0 + tt >= lo && slot0 + tt < hi; }
  // the tile of slot slot0 + tt (its place in it is tt % 64: units are whole tile pairs)
  __device__ const unsigned char* tile(const ReadParams& p, int tt) const {
    return p.tiles + (bh * (p.cap / kDecodeTileTokens) + (slot0 + tt) / kDecodeTileTokens) * static_cast<int64_t>(p.tl.bytes);
  }
};

// 16 values zero + code * scale of consecutive codes in the low bits of c[]
// (BITS each). A code k places up in its word is 2^(BITS k) code, which the low
// 23 bits of a float with the exponent of 2^23 hold without a shift; the scale
// takes the 2^(-BITS k) (exact), so product and rounding are those of the code.
template <int BITS>
__device__ __forceinline__ void values16(const uint32_t* c, float scale, float zero, float (&x)[16]) {
  constexpr int kWord = 32 / BITS;                    // codes of a word
  constexpr int kIn = 23 / BITS;                      // of them in the low 23 bits
  constexpr uint32_t kMask = (1u << BITS) - 1u;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int k = i % kWord, at = k < kIn ? k : k - kIn;  // place within the (shifted) word
    const uint32_t w = k < kIn ? c[i / kWord] : c[i / kWord] >> (BITS * kIn);
    const float n = __uint_as_float((w & (kMask << (BITS * at))) | 0x4B000000u) - 8388608.0f;
    x[i] = fmaf(n, scale * __uint_as_float(static_cast<uint32_t>(127 - BITS * at) << 23), zero);
  }
}

// Rows of one warp's 32 tokens on their way out, a piece of SEG bytes of each
// at a time (128, or 64 where S leaves less room): every lane puts its row's
// values, then the warp writes the piece row by row.
template <typename T, int SEG>
struct RowStage {
  static constexpr int kChunks = SEG / 16;                           // 16-byte chunks of a row, and lanes that write it
  static constexpr int kValues = SEG / static_cast<int>(sizeof(T));  // values of a row
  unsigned char* buf;  // 32 rows of SEG bytes, 16-byte chunks swizzled
  uint32_t live;       // rows to write
  T* dst;              // the row of lane 0
  int64_t st;
  static __device__ int key(int r) { return SEG == 128 ? r & 7 : (r >> 1) & 3; }
  // 16 values of this lane's row, from chunk `c` of the piece on
  __device__ void put(const float (&x)[16], int c) {
    const int lane = threadIdx.x & 31;
    unsigned char* row = buf + lane * SEG;
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(T)); ++q) {
      uint32_t w[4];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(x[4 * q + k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * q + 2 * k], x[8 * q + 2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(row + (((c + q) ^ key(lane)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // value e of this lane's row of the piece
  __device__ void set(int e, T v) {
    const int lane = threadIdx.x & 31, bytes = e * static_cast<int>(sizeof(T));
    *reinterpret_cast<T*>(buf + lane * SEG + (((bytes >> 4) ^ key(lane)) << 4) + (bytes & 15)) = v;
  }
  // the piece, whose first value is value `at` of the rows
  __device__ void flush(int at) {
    constexpr int kPer = 32 / kChunks;  // rows of a step
    const int lane = threadIdx.x & 31, sub = lane % kChunks, r0 = lane / kChunks;
    __syncwarp();
    T* to = dst + at + sub * (16 / static_cast<int>(sizeof(T))) + r0 * st;
#pragma unroll
    for (int i = 0; i < kChunks; ++i, to += kPer * st) {
      const int r = r0 + kPer * i;
      const uint4 v = *reinterpret_cast<const uint4*>(buf + r * SEG + ((sub ^ key(r)) << 4));
      if ((live >> r) & 1u) *reinterpret_cast<uint4*>(to) = v;
    }
    __syncwarp();
  }
};

template <typename T, int SEG, int BITS>
__global__ void __launch_bounds__(kReadThreads, 1) cache_read_kernel(const __grid_constant__ ReadParams p, int upb,
                                                                     int n_units) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int wpt = p.m / 32, wpo = p.m_out / 32, words = wpt + wpo, rows = 32 * words;
  uint64_t* a_full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* a_empty = a_full + 2;
  uint64_t* d_full = a_empty + 2;
  uint64_t* d_empty = d_full + 2;    // D_in
  uint64_t* out_empty = d_empty + 2;  // D_out
  uint64_t* drain = out_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* err = reinterpret_cast<int*>(tmem_slot + 1);
  unsigned char* img = smem + kReadMisc;
  unsigned char* stage = img + (p.K ? rows * kHeadDim * 2 : 0);  // 16 warps' row pieces
  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      bar_init(&a_full[k], 8);
      bar_init(&a_empty[k], 1);
      bar_init(&d_full[k], 1);
      bar_init(&d_empty[k], 8);
    }
    bar_init(out_empty, 8);
    bar_init(drain, 1);
    *err = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (p.K) {
    if (warp == 0) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // S, S_out -> the B operand: row 32 w + expand_pos(i) holds projection 32 w + i, two planes of 64 channels
#pragma unroll 4
    for (int e = tid; e < rows * 16; e += kReadThreads) {
      const int i = e >> 4, ch = e & 15;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(i < p.m ? p.S + i * kHeadDim : p.S_out + (i - p.m) * kHeadDim) + ch);
      const int kk = (i & ~31) + expand_pos(i & 31);
      *reinterpret_cast<uint4*>(img + (ch >> 3) * rows * 128 + kk * 128 + (((ch ^ kk) & 7) << 4)) = v;
    }
    fence_async_smem();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = p.K ? __shfl_sync(0xffffffffu, *tmem_slot, 0) : 0u;
  const unsigned long long limit = p.wait_cycles;
  ReadUnit u;

  if (warp < 8) {
    // ============================================================ signs
    const int tt = 32 * (warp & 3) + lane, part = warp >> 2;  // words 2 part, 2 part + 1 of a chunk
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kReadColA + 32 * part;
    bool ok = p.K != nullptr;
    int ring = 0;
    uint32_t ph = 1;
    // the words of chunk w0 of unit u, fetched one chunk ahead of their use
    const uint32_t* kb = nullptr;  // this token's words (null: outside the range)
    const uint32_t* ko = nullptr;
    const bool pairs = ((wpt | wpo) & 1) == 0;  // word pairs are of one part and 8-byte aligned
    auto token = [&] {
      const unsigned char* tile = u.tile(p, tt);
      kb = u.live(tt) ? reinterpret_cast<const uint32_t*>(tile + p.tl.kbits) + (tt & 63) * wpt : nullptr;
      ko = reinterpret_cast<const uint32_t*>(tile + p.tl.kbits_out) + (tt & 63) * wpo - wpt;
    };
    auto fetch = [&](int w0, uint32_t(&x)[2]) {
      const int w = w0 + 2 * part;
      x[0] = x[1] = 0u;
      if (!kb || w >= words) return;
      if (pairs) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>((w < wpt ? kb : ko) + w));
        x[0] = v.x;
        x[1] = v.y;
      } else {
        x[0] = __ldg((w < wpt ? kb : ko) + w);
        if (w + 1 < words) x[1] = __ldg((w + 1 < wpt ? kb : ko) + w + 1);
      }
    };
    bool more = p.K && u.begin(p, upb, n_units);
    uint32_t x[2];
    if (more) {
      token();
      fetch(0, x);
    }
    for (int w0 = 0; more && ok;) {
      const int here = w0;
      w0 += kReadWords;
      if (w0 >= words) {
        w0 = 0;
        more = u.next(p, upb, n_units);
        if (more) token();
      }
      uint32_t y[2];
      if (more) fetch(w0, y);
      ok = __all_sync(0xffffffffu, bar_wait(&a_empty[ring], ph, limit, err));
      if (!ok) break;
      fence_after();
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (here + 2 * part + k < words) {
          uint32_t e[16];
          expand_word(x[k], 0x3F803F80u, e);
          st16(lane_addr + 64 * ring + 16 * k, e);
        }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&a_full[ring]);
      ring ^= 1;
      ph ^= ring == 0 ? 1u : 0u;
      x[0] = y[0];
      x[1] = y[1];
    }
  } else if (warp < 16) {
    // ============================================================ values
    const int tt = 32 * (warp & 3) + lane, part = (warp - 8) >> 2;  // dims 64 part ..
    RowStage<T, SEG> out{stage + 32 * SEG * (warp - 8), 0u, nullptr, p.v_st};
    struct Codes {  // of this thread's half token, fetched one unit ahead of their use
      uint2 sz;
      uint4 cw[2];
      T* dst;  // the warp's first row
      bool live;
    };
    auto fetch = [&](Codes& c) {
      c.dst = static_cast<T*>(p.V) + u.b * p.v_sb + u.h * p.v_sh + static_cast<int64_t>(u.slot0 + tt - lane - u.start) * p.v_st;
      c.live = u.live(tt);
      c.sz = make_uint2(0u, 0u);
      c.cw[0] = c.cw[1] = make_uint4(0u, 0u, 0u, 0u);
      if (!c.live) return;
      const int j = tt & 63;
      const unsigned char* tile = u.tile(p, tt);
      c.sz = __ldg(reinterpret_cast<const uint2*>(tile + p.tl.vsz + 16 * j) + part);
#pragma unroll
      for (int gg = 0; gg < 2; ++gg) {
        const int g = 2 * part + gg;
        if (BITS == 4) {
          c.cw[gg] = __ldg(reinterpret_cast<const uint4*>(tile + p.tl.vcode + j * (kHeadDim / 2) + 16 * vcode_chunk(j, g)));
        } else {  // eight bytes of four 2-bit codes
          uint32_t q[2] = {0u, 0u};
#pragma unroll
          for (int r = 0; r < 8; ++r)
            q[r >> 2] |= static_cast<uint32_t>(__ldg(tile + p.tl.vcode + v2_line(g, r) + j)) << (8 * (r & 3));
          c.cw[gg] = make_uint4(q[0], q[1], 0u, 0u);
        }
      }
    };
    bool more = p.V && u.begin(p, upb, n_units);
    Codes nxt;
    if (more) fetch(nxt);
    while (more) {
      const Codes cur = nxt;
      more = u.next(p, upb, n_units);
      if (more) fetch(nxt);
      out.dst = cur.dst;
      out.live = __ballot_sync(0xffffffffu, cur.live);
      const uint32_t sz[2] = {cur.sz.x, cur.sz.y};
      constexpr int kStep = static_cast<int>(sizeof(T));  // chunks of 16 values
      int fill = 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&sz[g]));  // (scale, zero)
        const uint32_t c[4] = {cur.cw[g].x, cur.cw[g].y, cur.cw[g].z, cur.cw[g].w};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float x[16];
          values16<BITS>(BITS == 4 ? c + 2 * hf : c + hf, f.x, f.y, x);
          out.put(x, fill);
          fill += kStep;
          if (fill == out.kChunks) {
            out.flush(64 * part + 32 * g + 16 * hf + 16 - out.kValues);
            fill = 0;
          }
        }
      }
    }
  } else if (warp < 24) {
    // ============================================================ keys
    const int quarter = warp & 3, tt = 32 * quarter + lane, part = (warp - 16) >> 2;  // channels 64 part ..
    const uint32_t laddr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    RowStage<T, SEG> out{stage + 32 * SEG * (warp - 8), 0u, nullptr, p.k_st};
    const float c_in = kSqrtHalfPi / static_cast<float>(p.m), c_out = p.m_out ? kSqrtHalfPi / static_cast<float>(p.m_out) : 0.0f;
    bool ok = true;
    int units = 0;
    struct Token {  // fetched one unit ahead of its use
      uint32_t norms;
      int oc;  // lane o: the pair's o-th outlier channel
      T* dst;  // the warp's first row
      bool live;
    };
    auto fetch = [&](Token& k) {
      k.dst = static_cast<T*>(p.K) + u.b * p.k_sb + u.h * p.k_sh + static_cast<int64_t>(u.slot0 + tt - lane - u.start) * p.k_st;
      k.live = u.live(tt);
      k.norms = 0u;
      k.oc = lane < p.n_out ? min(max(__ldg(p.idx + u.bh * p.n_out + lane), 0), kHeadDim - 1) : -1;
      if (!k.live) return;
      k.norms = __ldg(reinterpret_cast<const uint32_t*>(u.tile(p, tt) + p.tl.knorm) + (tt & 63));
    };
    bool more = p.K && u.begin(p, upb, n_units);
    Token nxt;
    if (more) fetch(nxt);
    while (more) {
      const Token cur = nxt;
      more = u.next(p, upb, n_units);
      if (more) fetch(nxt);
      const float2 norm = __half22float2(*reinterpret_cast<const __half2*>(&cur.norms));
      const int oc = cur.oc;
      out.dst = cur.dst;
      out.live = __ballot_sync(0xffffffffu, cur.live);
      const int buf = units & 1;
      if (ok) ok = bar_wait(&d_full[buf], (units >> 1) & 1, limit, err);
      ++units;
      ok = __all_sync(0xffffffffu, ok);
      fence_after();
      const float f_in = ok ? c_in * norm.x : __int_as_float(0x7fc00000), f_out = ok ? c_out * norm.y : __int_as_float(0x7fc00000);
      constexpr int kStep = static_cast<int>(sizeof(T));  // chunks of 16 values
      constexpr int span = RowStage<T, SEG>::kValues;      // channels of a piece
#pragma unroll 1
      for (int c0 = 64 * part; c0 < 64 * part + 64; c0 += span) {
#pragma unroll
        for (int q = 0; q < span / 16; ++q) {
          uint32_t v[16];
          ld16(v, laddr + 128 * buf + c0 + 16 * q);
          wait_ld();
          float x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(v[k]) * f_in;
          out.put(x, kStep * q);
        }
        // the outlier channels of the piece come from the other sums
        uint32_t some = __ballot_sync(0xffffffffu, oc >= c0 && oc < c0 + span);
        while (some != 0u) {
          int c[4];
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            c[k] = some != 0u ? __shfl_sync(0xffffffffu, oc, __ffs(some) - 1) : k ? c[0] : c0;
            some &= some - 1u;
            ld1(v[k], laddr + kReadColOut + c[k]);
          }
          wait_ld();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y = __uint_as_float(v[k]) * f_out;
            if constexpr (sizeof(T) == 4) out.set(c[k] - c0, y);
            else out.set(c[k] - c0, __float2bfloat16_rn(y));
          }
        }
        if (c0 + span == 64 * part + 64) {  // the sums are read
          fence_before();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(&d_empty[buf]);
            bar_arrive(out_empty);
          }
        }
        out.flush(c0);
      }
    }
  } else if (p.K) {
    // ============================================================ products (the whole warp, converged)
    bool ok = true;
    int ring = 0;
    int units = 0;
    uint32_t aph = 0;
    const uint32_t id = idesc_f16(kHeadDim, true, 0, 1);
    for (bool more = u.begin(p, upb, n_units); more && ok; more = u.next(p, upb, n_units)) {
      const int buf = units & 1;
      ok = __all_sync(0xffffffffu, units < 2 || bar_wait(&d_empty[buf], ((units >> 1) - 1) & 1, limit, err));
      uint64_t bd = desc_mn(smem_u32(img), rows * 128);
      for (int w0 = 0; w0 < words && ok; w0 += kReadWords) {
        ok = __all_sync(0xffffffffu, bar_wait(&a_full[ring], aph, limit, err));
        if (!ok) break;
        fence_after();
        uint32_t ad = tmem + kReadColA + 64 * ring;
        const int w1 = min(words, w0 + kReadWords);
#pragma unroll 1
        for (int w = w0; w < w1; ++w, ad += 16, bd += 256) {  // 32 rows of 128 bytes: 256 address units
          if (w == wpt && units > 0) {  // the one D_out
            ok = __all_sync(0xffffffffu, bar_wait(out_empty, (units - 1) & 1, limit, err));
            if (!ok) break;
            fence_after();
          }
          mma_ts_mn_32_warp(tmem + (w < wpt ? 128 * buf : kReadColOut), ad, bd, id, w != 0 && w != wpt);
        }
        if (!ok) break;
        commit_warp(&a_empty[ring]);
        ring ^= 1;
        aph ^= ring == 0 ? 1u : 0u;
      }
      if (ok) commit_warp(&d_full[buf]);
      ++units;
    }
    commit_warp(drain);  // every product ends before the block gives its memory back
    bar_wait(drain, 0, limit > 2000000000ull ? limit : 2000000000ull, nullptr);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (p.K && warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <typename T, int SEG, int BITS>
cudaError_t launch(const ReadParams& p, size_t smem, cudaStream_t s) {
  // 128-slot units that T tokens of any alignment can touch
  const int64_t upb = (static_cast<int64_t>(p.T < p.cap ? p.T : p.cap) + 2 * kReadUnit - 2) / kReadUnit;
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * upb;
  if (units > 0x3fffffff) return cudaErrorInvalidValue;  // (more slots than a device's memory holds)
  auto kernel = cache_read_kernel<T, SEG, BITS>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(units < p.num_sms ? units : p.num_sms), kReadThreads, smem, s>>>(
      p, static_cast<int>(upb), static_cast<int>(units));
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ReadParams& p, cudaStream_t s) {
  const size_t fixed = kReadMisc + 1024 + (p.K ? static_cast<size_t>(p.m + p.m_out) * kHeadDim * 2 : 0);
  const bool wide = fixed + 16 * 32 * 128 <= 227 * 1024;
  size_t smem = fixed + 16 * 32 * (wide ? 128 : 64);
  if (smem < 116 * 1024) smem = 116 * 1024;  // one block per SM: it takes all tensor-memory columns
  if (p.tl.vbits == 4) return wide ? launch<T, 128, 4>(p, smem, s) : launch<T, 64, 4>(p, smem, s);
  return wide ? launch<T, 128, 2>(p, smem, s) : launch<T, 64, 2>(p, smem, s);
}

}  // namespace

cudaError_t launch_cache_read(const ReadParams& p, qjl_dtype dt, cudaStream_t s) {
  return dt == QJL_BF16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace qjl
