// Attention of drafted tokens over the QJL cache on the tensor cores (bf16
// queries).
//
// Rows r = i G + g of a (sequence, kv head): drafted token i, query head g of
// the kv head. With sq the projected query of a row (the estimator's factors,
// sm_scale and log2(e) folded in) the logits of 128 tokens are one product,
//   X^T [token, row] = (signs * norm) [token, m + m_out] sq^T [m + m_out, row],
// because the norm of a key is stored as fp16: a sign bit times the norm is an
// fp16 number with that sign, exactly. Tokens are the M dimension of both
// products, rows the N dimension, so that a few rows cost a few columns:
//   O^T [dim, row] += V_hat^T [dim, token] P [token, row].
// The sign operand is written to tensor memory by the threads that own its
// tokens (lane = token), which keeps it out of shared memory.
//
// Roles of a persistent block (one per SM, all 512 tensor-memory columns):
//   warps 0-3    signs and norms of 128 tokens -> tensor memory (two buffers, of
//                all projections when they fit beside the accumulators)
//   warps 4-7    value codes -> fp16 values in shared memory, thread = token
//   warps 8-15   logits -> weights (fp16, shared memory), running maximum, sums
//   warp 16      issues every tcgen05.mma
//   warp 17      bulk copies of cache tiles (two 64-token tiles a stage)
// The work is the list of 128-token units of every (sequence, kv head, row
// block), cut into equal contiguous ranges; what two blocks share is joined by
// tree_join_kernel. The last unit of an item is the draft tile, the only one
// with a mask.
//
// Softmax: p = 2^(x - ref) with ref = (maximum seen) - 4, moved only when a
// logit passes ref + 15: weights stay below 2^15 in fp16, and those down to
// 2^-18 of the largest keep all their bits; smaller ones are rounded to
// multiples of 2^-28 of it at worst, so that n of them move an output by
// n 2^-29 max |V_hat| at most. V_hat is a multiple of 2^-24, as its scale and
// zero are: fp16 holds a value below 65504 to 2^-11 of itself, and exactly below
// 2^-13. From the first unit with a token that may pass 65504 on (wide_token),
// the values of an item are kept as V_hat / 16, which no fp16 scale and zero push
// past the range, to 2^-11 or 2^-20 absolute; that unit's product divides the
// outputs so far by 16. (Dividing from the start lost the bits of small values;
// looking for wide tokens costs 2 % of a long call with 64 rows, 8 % with 16.) All
// sums are fp32.
//
// Bound: HBM below about 35 rows of a kv head (124 bytes against 896 flops per
// row and token), the tensor rate above. Measured, 4 x 131072 tokens, 8 kv heads,
// 64 rows: 360 us in a row on unchanged inputs, 388 on inputs that change from call
// to call, where the tensor rate allows 146 and HBM 80; a unit costs
// about 2600 SM cycles, its products 1060 (an mma of 128 x 64 x 16 takes 33), and
// the roles issue 7500 warp instructions together, 59 % of the slots (320 of a sign
// warp's 430 per unit are the logic of the expansion, 240 of a value warp's 400
// the dequantisation); the rest are waits between roles. With 16 rows the call
// takes 305 us. A call's start, first unit, outputs and join cost about 35 us.
#include "tc_common.cuh"

namespace qjl {
namespace {

using namespace tc;

constexpr int kUnit = 128;              // tokens of a unit (MMA M)
constexpr int kKWarps = 4, kVWarps = 4, kSWarps = 8;
constexpr int kSWarp0 = kKWarps + kVWarps, kMmaWarp = kSWarp0 + kSWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kTreeTcThreads = 640;      // five warpgroups; two warps of the last are idle
// Registers per thread of the roles (setmaxnreg): 128 * (72 + 72 + 2 * 136 + 64) = 640 * 96, what the launch holds.
constexpr int kRegsExpand = 72, kRegsWeights = 136, kRegsIssue = 64;
constexpr int kMaxStages = 4;
constexpr int kVBytes = kUnit * kHeadDim * 2;       // values of a unit
constexpr int kPlane = kUnit * 128;                 // 64 rows' weights of a unit
constexpr float kRefBelow = 4.0f, kRefMove = 15.0f;
constexpr float kNothing = 3.0e38f;                 // -ref of a row that has seen nothing

struct TreeTcCfg {
  int rb;      // rows of a block (a multiple of 16, at most 128)
  int nrb;     // row blocks of N * G rows
  int nk;      // 64-projection steps
  int ck;      // steps of a sign operand chunk (two chunks in tensor memory)
  int np;      // weight buffers
  int ns;      // cache stages
  int stage;   // bytes of a stage
  int smem;
};
constexpr int kBadRing = 4;  // items that the value warps may have begun and the weight warps not ended (three), and one
constexpr int kMiscBytes = 3 * 128 * 4 + 4 * 128 * 4 + 2 * 128 * 8 + kBadRing * 64 * 4 + (kBadRing + 2) * 4 + 32 * 8 + 64;

// Row block, buffers and stages: the largest row block (fewest passes over the
// cache) that leaves two stages, then a second weight buffer, then stages. With at
// most 64, 96 and 128 rows a block: 1 x 32768 tokens, 8 kv heads, 128 rows 80, 80, 89
// us; 96 rows 79, 74, 74; 512 rows 207, 219, 217; 4 x 8192, 132 rows 110, 107, 107.
TreeTcCfg tree_tc_cfg(int N, int G, int m, int m_out, int tile_bytes) {
  TreeTcCfg c{};
  const int R = N * G, limit = 227 * 1024 - 1024;
  c.nk = (m + m_out + 63) / 64;
  c.stage = 2 * tile_bytes;
  for (int cap = 128;; cap -= 16) {
    c.nrb = (R + cap - 1) / cap;
    c.rb = ((R + c.nrb - 1) / c.nrb + 15) / 16 * 16;
    const int planes = c.rb > 64 ? 2 : 1;
    const int fixed = c.nk * c.rb * 128 + 2 * kVBytes + kMiscBytes;
    c.np = 1;
    c.ns = 2;
    auto total = [&] { return fixed + c.np * planes * kPlane + c.ns * c.stage; };
    if (total() > limit && cap > 16) continue;
    c.np = 2;
    if (total() > limit) c.np = 1;
    while (c.ns < kMaxStages) {
      ++c.ns;
      if (total() > limit) {
        --c.ns;
        break;
      }
    }
    c.smem = total() + 1024;
    // tensor memory: two logit buffers and the outputs, then the signs
    c.ck = (512 - 3 * c.rb) / 64;
    if (c.ck > c.nk) c.ck = c.nk;
    return c;
  }
}

struct TreeTcWs {
  size_t start, image, scale, part_o, part_ml, total;
};
TreeTcWs tree_tc_ws(const TreeTcCfg& c, int B, int Hkv, int num_sms) {
  auto a256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t items = static_cast<size_t>(B) * Hkv * c.nrb;
  TreeTcWs w{};
  w.start = 0;
  w.image = a256((static_cast<size_t>(B) + 1) * 8);
  w.scale = w.image + a256(items * c.nk * c.rb * 128);
  w.part_o = w.scale + a256(items * c.rb * 4);
  w.part_ml = w.part_o + a256(static_cast<size_t>(2) * num_sms * c.rb * kHeadDim * 4);
  w.total = w.part_ml + a256(static_cast<size_t>(2) * num_sms * c.rb * 8);
  return w;
}

struct TreeTcParams {
  TreeParams t;
  TreeTcCfg c;
  long long* start;      // [B + 1] first unit of each sequence
  unsigned char* image;  // [B * Hkv][nrb] projected queries as the B operand
  float* scale;          // [B * Hkv][nrb][rb] power-of-two scales of the rows
  float* part_o;         // [2 * grid][rb][d]
  float2* part_ml;       // [2 * grid][rb]
  int grid;
};

__device__ __forceinline__ int seq_len(const TreeParams& t, int b) {
  return t.seqlens ? min(max(t.seqlens[b], 0), t.T) : t.T;
}
__device__ __forceinline__ int seq_drafts(const TreeParams& t, int b) {
  return t.n_draft ? min(max(t.n_draft[b], 0), t.N) : t.N;
}
__device__ __forceinline__ int seq_units(const TreeParams& t, int b) {  // units of one item of sequence b
  return (seq_len(t, b) + kUnit - 1) / kUnit + 1;
}
__device__ __forceinline__ int seq_items(const TreeParams& t, const TreeTcCfg& c, int b) {
  return t.Hkv * ((seq_drafts(t, b) * t.G + c.rb - 1) / c.rb);
}

// ---------------------------------------------------------------- preparation

// Projected queries of 16 rows per block: sq = [S; S_out] q on bf16 MMAs (S in
// decode's A-fragment order, products exact, fp32 sums), scaled so that the
// row's largest entry lies in [2^14, 2^15), rounded to fp16 and written in the
// order and swizzle of the score product's B operand. Block (0, 0) also writes
// the first unit of every sequence. Launched before what precedes it ends, it
// waits for that before it touches anything but S: 1.4 us less at 130 tokens,
// 2 us less at 1024 (19.2 -> 17.8, 36.2 -> 34.0).
constexpr int kPrepWarps = 12;
constexpr int kPrepWords = (kMaxM + kMaxMOut) / 32 / kPrepWarps;  // sign words of a warp

__global__ void __launch_bounds__(32 * kPrepWarps) tree_prepare_kernel(TreeTcParams p) {
  const TreeParams& t = p.t;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / t.Hkv), hk = static_cast<int>(bh % t.Hkv);
  uint4 first_s[16];  // the warp's first word of [S; S_out], which no kernel writes, ahead of the wait
#pragma unroll
  for (int k = 0; k < 16; ++k)
    first_s[k] = warp < (t.m + t.m_out) / 32 ? __ldg(t.S_frag + (16 * warp + k) * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
  // whatever came before on the stream may write the inputs and read the
  // workspace; the next kernel is let in after it too, so that one which holds
  // all tensor memory never meets one still to allocate its own
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && bh == 0 && warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < t.B; b0 += 32) {
      const int bb = b0 + lane;
      long long n = bb < t.B ? static_cast<long long>(seq_units(t, bb)) * seq_items(t, p.c, bb) : 0;
      const long long own = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += o;
      }
      if (bb < t.B) p.start[bb] = base + n - own;
      base += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) p.start[t.B] = base;
  }
  const int nd = seq_drafts(t, b), live = nd * t.G;
  const int row0 = blockIdx.x * 16;                    // rows of nrb * rb
  if ((row0 / p.c.rb) * p.c.rb >= live) return;        // a row block nobody computes
  __shared__ float top_s[kPrepWarps][16];
  uint32_t om[4] = {0u, 0u, 0u, 0u};
  {
    const int c = lane < t.n_out ? min(max(t.idx[bh * t.n_out + lane], 0), kHeadDim - 1) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) om[k] = __reduce_or_sync(0xffffffffu, c >= 0 && (c >> 5) == k ? 1u << (c & 31) : 0u);
  }
  // B fragments of the 16 rows (two 8-column tiles), inlier and outlier channels
  const int q = lane & 3, r = lane >> 2;
  uint32_t bf[2][8][2], keep[8][2];
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 16 * ks + 8 * k + 2 * q;
      const uint32_t o = (om[ks >> 1] >> (c & 31)) & 3u;
      keep[ks][k] = (o & 1u ? 0u : 0x0000FFFFu) | (o & 2u ? 0u : 0xFFFF0000u);
    }
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int row = row0 + 8 * nt + r, i = row / t.G, g = row % t.G;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(t.Q) + b * t.q_sb + i * t.q_sn +
                               (static_cast<int64_t>(hk) * t.G + g) * t.q_sh;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        bf[nt][ks][k] = row < live ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 * k + 2 * q) : 0u;
  }
  const int wpt = t.m / 32, words = wpt + t.m_out / 32;
  float acc[kPrepWords][2][2][4];  // [word][16-row half][row tile]
  float top[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
  for (int s = 0; s < kPrepWords; ++s) {
    const int w = warp + kPrepWarps * s;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[s][hf][nt][k] = 0.0f;
    if (w < words) {
      const bool second = w >= wpt;
      const float f = kSqrtHalfPi / static_cast<float>(second ? t.m_out : t.m) * t.sm_scale_log2;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint4 a = s == 0 ? first_s[8 * hf + ks] : __ldg(t.S_frag + ((2 * w + hf) * 8 + ks) * 32 + lane);
          const uint32_t k0 = second ? ~keep[ks][0] : keep[ks][0], k1 = second ? ~keep[ks][1] : keep[ks][1];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            float* d = acc[s][hf][nt];
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                "{%0,%1,%2,%3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(bf[nt][ks][0] & k0), "r"(bf[nt][ks][1] & k1));
          }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[s][hf][nt][k] *= f;
            top[nt][k & 1] = fmaxf(top[nt][k & 1], fabsf(acc[s][hf][nt][k]));
          }
      }
    }
  }
  // the rows' largest entries: lanes 4r + q of a warp, then the warps
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v = top[nt][k];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
      if (lane < 4) top_s[warp][8 * nt + 2 * q + k] = v;
    }
  __syncthreads();
  unsigned char* img = p.image + (bh * p.c.nrb + row0 / p.c.rb) * static_cast<int64_t>(p.c.nk) * p.c.rb * 128;
  const int in_block = row0 % p.c.rb;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = 8 * nt + 2 * q + k;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kPrepWarps; ++w) v = fmaxf(v, top_s[w][col]);
      // 2^e <= v < 2^(e+1): scale by 2^(14 - e), at most 2^126 (a row that small has logits of zero)
      const int e = max(static_cast<int>(__float_as_uint(v) >> 23) - 127, -112);
      const float up = v > 0.0f ? __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23) : 1.0f;
      const float down = v > 0.0f ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) : 1.0f;
      const int row = in_block + col;
      if (warp == 0 && r == 0) p.scale[(bh * p.c.nrb + row0 / p.c.rb) * p.c.rb + row] = down;
#pragma unroll
      for (int s = 0; s < kPrepWords; ++s) {
        const int w = warp + kPrepWarps * s;
        if (w >= words) continue;
        // bits r, r + 8 (half 0) and r + 16, r + 24 (half 1) of word w: elements 2j, 2j + 1 of j = 15 - r and 7 - r
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const __half2 h = __floats2half2_rn(acc[s][0][nt][2 * z + k] * up, acc[s][1][nt][2 * z + k] * up);
          const int kk = 32 * (w & 1) + 2 * (15 - 8 * z - r);
          *reinterpret_cast<uint32_t*>(img + (w >> 1) * p.c.rb * 128 + row * 128 + ((((kk >> 3) ^ row) & 7) << 4) +
                                       (kk & 7) * 2) = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
}

// ---------------------------------------------------------------- main kernel

// The items (sequence, kv head, row block) of a block's range of units, in order.
struct Walk {
  int b, hk, rbk;            // current item
  int len, nd, units, nblk;  // of sequence b
  int u0, u1;                // this block's units of the item: [u0, u1) of `units`
  long long left;            // units of the range from the current item's u0 on
  __device__ bool begin(const TreeTcParams& p, long long first, long long end) {
    left = end - first;
    if (left <= 0) return false;
    int lo = 0, hi = p.t.B - 1;  // the last sequence whose first unit is <= first (empty sequences share it)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.start[mid] <= first) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    load(p);
    const long long off = first - p.start[b];
    const int item = static_cast<int>(off / units);
    hk = item / nblk;
    rbk = item % nblk;
    u0 = __shfl_sync(0xffffffffu, static_cast<int>(off % units), 0);
    u1 = __shfl_sync(0xffffffffu, static_cast<int>(min(static_cast<long long>(units), u0 + left)), 0);
    return true;
  }
  __device__ void load(const TreeTcParams& p) {
    len = seq_len(p.t, b);
    nd = seq_drafts(p.t, b);
    units = seq_units(p.t, b);
    nblk = (nd * p.t.G + p.c.rb - 1) / p.c.rb;
  }
  // WARP: called by a whole warp, which makes the bounds uniform values
  template <bool WARP>
  __device__ bool next(const TreeTcParams& p) {
    left -= u1 - u0;
    if (left <= 0) return false;
    if (++rbk >= nblk) {
      rbk = 0;
      if (++hk >= p.t.Hkv) {
        hk = 0;
        do ++b;
        while (seq_drafts(p.t, b) == 0);  // units are left, so a sequence with drafts follows
        load(p);
      }
    }
    u0 = 0;
    u1 = static_cast<int>(min(static_cast<long long>(units), left));
    if (WARP) u1 = __shfl_sync(0xffffffffu, u1, 0);
    return true;
  }
  __device__ bool draft(int u) const { return u == units - 1; }
  __device__ int tokens(int u) const { return draft(u) ? nd : min(kUnit, len - u * kUnit); }
  __device__ int64_t bh(const TreeTcParams& p) const { return static_cast<int64_t>(b) * p.t.Hkv + hk; }
};

struct TreeTcSmem {
  int sq, v, pw, raw, rowc, cmax, mask, bad, wide, bars, misc;
  __device__ explicit TreeTcSmem(const TreeTcCfg& c) {
    sq = 0;
    v = c.nk * c.rb * 128;
    pw = v + 2 * kVBytes;
    raw = pw + c.np * (c.rb > 64 ? 2 : 1) * kPlane;
    rowc = raw + c.ns * c.stage;  // float4 [64]: scales and -refs of two rows; float [128]: rescaling, then output factor
    cmax = rowc + 3 * 128 * 4;    // float [4][128]: column maxima, then sums, of the lane quarters
    mask = cmax + 4 * 128 * 4 + 128 * 8;  // (after int64 [128]: where a row's outputs go) uint64 [128]
    bad = mask + 128 * 8;         // uint32 [kBadRing][64]: value groups of a drafted token that are not finite
    wide = bad + kBadRing * 64 * 4;      // int [kBadRing]: the item's values are divided by 16; int [2]: since this unit
    bars = wide + (kBadRing + 2) * 4;
    misc = bars + 32 * 8;
  }
};

__device__ __forceinline__ uint64_t pack2(float a, float b) { return f32x2_pack(a, b); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The four weight warps that share their rows synchronise on their own barrier.
__device__ __forceinline__ bool s_any(int half, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(1 + half)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void s_sync(int half) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory"); }

__device__ __forceinline__ bool v_any(bool x) {  // the value warps
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, 3, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Reduces 16 values per lane over the 32 lanes, value k ending in lanes
// 2 rev(k), 2 rev(k) + 1; returns the column of this lane.
template <typename Op>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane, int* col, Op op) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int off = 16 >> s, n = 8 >> s;
    const bool up = lane & off;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
      v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  *col = (lane & 16 ? 8 : 0) + (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) + (lane & 2 ? 1 : 0);
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// zero + code * scale of one of a token's groups may pass 65504: a finite scale
// of 2^11 or a finite zero of 2^15 and more (below, 15 * 2^11 + 2^15 < 65504).
// Adding 2^10 to the bit patterns lets those that are not finite wrap to small ones.
__device__ __forceinline__ bool wide_token(const uint4& sz) {
  const uint32_t abs2 = 0x7FFF7FFFu, one = 0x04000400u;
  const uint32_t top = __vmaxu2(__vmaxu2((sz.x + one) & abs2, (sz.y + one) & abs2),
                                __vmaxu2((sz.z + one) & abs2, (sz.w + one) & abs2));
  return (top & 0xFFFFu) >= 0x6C00u || top >= 0x7C000000u;
}

// NBW: 16-row groups of a weight warp; BITS: of a value code.
template <int NBW, int BITS>
__global__ void __launch_bounds__(kTreeTcThreads, 1) tree_tc_kernel(const __grid_constant__ TreeTcParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const TreeParams& t = p.t;
  const TreeTcCfg& c = p.c;
  const TreeTcSmem L(c);
  // the warp index, and below what a role's warp walks over, as uniform values: addresses and operands then take the
  // uniform datapath
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* raw_empty = raw_full + kMaxStages;
  uint64_t* a_full = raw_empty + kMaxStages;
  uint64_t* a_empty = a_full + 2;
  uint64_t* s_full = a_empty + 2;
  uint64_t* pv_full = s_full + 2;    // weights and values of a unit
  uint64_t* pv_empty = pv_full + 2;  // their product is done
  uint64_t* sq_full = pv_empty + 2;
  uint64_t* o_full = sq_full + 1;
  uint64_t* o_empty = o_full + 1;
  uint64_t* drain = o_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L.misc);
  volatile int* err = reinterpret_cast<int*>(tmem_slot + 1);
  if (tid == 0) {
    for (int k = 0; k < kMaxStages; ++k) {
      bar_init(&raw_full[k], 1);
      bar_init(&raw_empty[k], kKWarps + kVWarps);
    }
    for (int k = 0; k < 2; ++k) {
      bar_init(&a_full[k], kKWarps);
      bar_init(&a_empty[k], 1);
      bar_init(&s_full[k], 1);
      bar_init(&pv_full[k], kSWarps + kVWarps);
      bar_init(&pv_empty[k], 1);
    }
    bar_init(sq_full, 1);
    bar_init(o_full, 1);
    bar_init(o_empty, kSWarps);
    bar_init(drain, 1);
    *err = 0;
    for (int k = 0; k < 2; ++k) reinterpret_cast<int*>(smem + L.wide)[kBadRing + k] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  griddep_wait();  // the projected queries and the unit table
  griddep_launch();
  const long long total = p.start[t.B];
  const long long first = total * blockIdx.x / p.grid, end = total * (blockIdx.x + 1) / p.grid;
  const int col_o = 2 * c.rb, col_a = 3 * c.rb;  // tensor-memory columns: logits at 0 and rb
  const unsigned long long limit = t.wait_cycles;
  const unsigned long long limit_drain = limit > 2000000000ull ? limit : 2000000000ull;
  Walk w;
  const bool any = w.begin(p, first, end);

  if (warp < kKWarps) {
    // ============================================================ signs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    const int tt = 32 * warp + lane, j = tt & 63;
    const int wpt = t.m / 32, wpo = t.m_out / 32, words = wpt + wpo;
    const bool even = ((wpt | wpo) & 1) == 0;  // word pairs are 8-byte aligned and of one part
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * warp) << 16) + col_a;
    bool ok = true;
    int st = 0, ring = 0;
    uint32_t sph = 0, rph = 1;  // phases: stage full, chunk empty (the first pass finds every chunk empty)
    for (bool more = any; more && ok; more = w.next<true>(p))
      for (int u = w.u0; u < w.u1 && ok; ++u) {
        ok = bar_wait(&raw_full[st], sph, limit, err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned char* tile = smem + L.raw + st * c.stage + (tt >> 6) * t.tl.bytes;
        const uint32_t norms = *reinterpret_cast<const uint32_t*>(tile + t.tl.knorm + 4 * j);
        const uint32_t n_in = __byte_perm(norms, 0, 0x1010), n_out = __byte_perm(norms, 0, 0x3232);
        const uint32_t* kb = reinterpret_cast<const uint32_t*>(tile + t.tl.kbits) + j * wpt;
        const uint32_t* ko = reinterpret_cast<const uint32_t*>(tile + t.tl.kbits_out) + j * wpo - wpt;
#pragma unroll 1
        for (int k0 = 0; k0 < c.nk; k0 += c.ck) {
          ok = bar_wait(&a_empty[ring], rph, limit, err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          fence_after();
          uint32_t dst = lane_addr + 32 * c.ck * ring;
          const int k1 = min(c.nk, k0 + c.ck);
          if (even) {  // word pairs of one part
            uint32_t e[16];
            const int ki = min(k1, wpt >> 1);
            int kc = k0;
#pragma unroll 1
            for (; kc < ki; ++kc, dst += 32) {
              const uint2 x = reinterpret_cast<const uint2*>(kb)[kc];
              expand_word(x.x, n_in, e);
              st16(dst, e);
              expand_word(x.y, n_in, e);
              st16(dst + 16, e);
            }
#pragma unroll 1
            for (; kc < k1; ++kc, dst += 32) {
              const uint2 x = *reinterpret_cast<const uint2*>(ko + 2 * kc);
              expand_word(x.x, n_out, e);
              st16(dst, e);
              expand_word(x.y, n_out, e);
              st16(dst + 16, e);
            }
          } else {
#pragma unroll 1
            for (int w = 2 * k0; w < 2 * k1; ++w, dst += 16) {
              uint32_t e[16];
              expand_word(w < wpt ? kb[w] : w < words ? ko[w] : 0u, w < wpt ? n_in : n_out, e);
              st16(dst, e);
            }
          }
          wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&a_full[ring]);
          ring ^= 1;
          rph ^= ring == 0 ? 1u : 0u;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&raw_empty[st]);
        if (++st == c.ns) {
          st = 0;
          sph ^= 1u;
        }
      }
  } else if (warp < kSWarp0) {
    // ============================================================ values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    const int tt = 32 * (warp - kKWarps) + lane, j = tt & 63;
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L.bad);
    bool ok = true;
    int st = 0, vb = 0, item = 0, n = 0;
    uint32_t sph = 0, vph = 1;
    int* wides = reinterpret_cast<int*>(smem + L.wide);
    const uint32_t key = (tt & 7) << 4;
    for (bool more = any; more && ok; more = w.next<true>(p), ++item) {  // (ok ends for all four warps at once)
      bool wide = false;  // the item's values are divided by 16 from here on
      if (tt == 0) wides[item % kBadRing] = 0;  // (read at the item's end)
      for (int u = w.u0; u < w.u1 && ok; ++u) {
        ok = bar_wait(&raw_full[st], sph, limit, err) && bar_wait(&pv_empty[vb], vph, limit, err);
        ok = __all_sync(0xffffffffu, ok);
        const unsigned char* tile = smem + L.raw + st * c.stage + (tt >> 6) * t.tl.bytes;
        const bool live = tt < w.tokens(u), draft = w.draft(u);
        const uint4 sz = *reinterpret_cast<const uint4*>(tile + t.tl.vsz + 16 * j);
        const uint32_t* szg = reinterpret_cast<const uint32_t*>(tile + t.tl.vsz + 16 * j);
        // The four warps must agree on the unit's factor, and leave together when a wait ran out in one: one barrier,
        // and seldom a second that tells which of the two it was.
        if (v_any(!ok | (live & wide_token(sz)))) {
          ok = !v_any(!ok);
          if (!ok) break;
          if (!wide && tt == 0) {
            wides[item % kBadRing] = 1;
            if (u > w.u0) wides[kBadRing + vb] = n;  // this unit's product divides what the item has so far
          }
          wide = true;
        }
        // from a code's bits to the code, or to the code / 16 (exact, as is its product with the scale inside the fma;
        // a zero / 16 below 2^-14 rounds by 2^-25 at most)
        const __half2 odd_mul = __float2half2_rn(wide ? 0.00390625f : 0.0625f), odd_add = __float2half2_rn(wide ? -4.0f : -64.0f);
        const __half2 even_mul = __float2half2_rn(wide ? 0.0625f : 1.0f), even_add = __float2half2_rn(wide ? -64.0f : -1024.0f);
        unsigned char* row = smem + L.v + vb * kVBytes + tt * 128;
        uint32_t bits = 0u;
        const bool special = draft || w.tokens(u) < kUnit;
#pragma unroll 2
        for (int g = 0; g < 4; ++g) {
          uint32_t use = szg[g];
          if (special) {
            // a masked drafted value that is not finite must not meet a weight of
            // zero in the product: it is left out here and added at the end
            const bool off = draft && ((use & 0x7C00u) == 0x7C00u || (use & 0x7C000000u) == 0x7C000000u);
            if (off) bits |= 1u << g;
            if (!live || off) use = 0u;
          }
          const __half2 s2 = __half2half2(__ushort_as_half(static_cast<unsigned short>(use)));
          const __half2 z2 = __hmul2(__half2half2(__ushort_as_half(static_cast<unsigned short>(use >> 16))), even_mul);
          uint32_t lo[4], hi[4];  // codes of dims (8c + k, 8c + k + 4), k = 0..3, of 8-dim chunk c: two fields 16 bits apart
          if (BITS == 4) {
            const uint4 cw = *reinterpret_cast<const uint4*>(tile + t.tl.vcode + j * (kHeadDim / 2) + 16 * vcode_chunk(j, g));
            const uint32_t cc[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              lo[k] = cc[k];
              hi[k] = cc[k] >> 8;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // two bits per code -> the nibble form: bits 0-1 and 2-3 of each byte to bits 0 and 4 of a half word
              const uint32_t x = static_cast<uint32_t>(tile[t.tl.vcode + v2_line(g, 2 * k) + j]) |
                                 (static_cast<uint32_t>(tile[t.tl.vcode + v2_line(g, 2 * k + 1) + j]) << 16);
              lo[k] = (x & 0x00030003u) | ((x & 0x000C000Cu) << 2);
              hi[k] = ((x >> 4) & 0x00030003u) | ((x & 0x00C000C0u) >> 2);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // 0x6400 | n is 1024 + n, and with the code four bits up 1024 + 16 n
            uint32_t y[4];
            const uint32_t f[4] = {(lo[k] & 0x000F000Fu) | 0x64006400u, (lo[k] & 0x00F000F0u) | 0x64006400u,
                                   (hi[k] & 0x000F000Fu) | 0x64006400u, (hi[k] & 0x00F000F0u) | 0x64006400u};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 h = *reinterpret_cast<const __half2*>(&f[e]);
              const __half2 n = e & 1 ? __hfma2(h, odd_mul, odd_add) : __hfma2(h, even_mul, even_add);
              const __half2 r = __hfma2(n, s2, z2);
              y[e] = *reinterpret_cast<const uint32_t*>(&r);
            }
            // 8-dim chunk 4 g + k of the row
            *reinterpret_cast<uint4*>(row + (g >> 1) * kPlane + (((4 * (g & 1) + k) << 4) ^ key)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        if (draft && tt < 64) bad[64 * (item % kBadRing) + tt] = live ? bits : 0u;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&pv_full[vb]);
          bar_arrive(&raw_empty[st]);
        }
        vb ^= 1;
        ++n;
        if (vb == 0) vph ^= 1u;
        if (++st == c.ns) {
          st = 0;
          sph ^= 1u;
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ============================================================ weights
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWeights));
    const int quarter = warp & 3, half = (warp - kSWarp0) >> 2, tt = 32 * quarter + lane, stid = tid & 127;
    const int col0 = 16 * NBW * half;                          // this warp's rows of the block
    const int nbw = min(NBW, c.rb / 16 - NBW * half);          // and their groups of 16
    float4* rowc = reinterpret_cast<float4*>(smem + L.rowc) + col0 / 2;
    float* fac = reinterpret_cast<float*>(smem + L.rowc) + 256 + col0;
    float* cmax = reinterpret_cast<float*>(smem + L.cmax) + col0;
    uint64_t* mrow = reinterpret_cast<uint64_t*>(smem + L.mask) + col0;
    const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + L.bad);
    const uint32_t laddr = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + static_cast<uint32_t>(col0);
    const int planes = c.rb > 64 ? 2 : 1;
    // logits are kept in registers between the two passes when they fit beside the sums
    constexpr bool kKeep = NBW <= 2;
    constexpr int kHeld = kKeep ? NBW : 1;
    bool ok = true;
    int n = 0;            // units so far
    uint32_t oph = 0;
    int it = 0;
    for (bool more = any; more; more = w.next<true>(p), ++it) {
      const int64_t item = w.bh(p) * c.nrb + w.rbk;
      uint64_t lsum[NBW][8];  // sums of this token's weights, pairs of rows
#pragma unroll
      for (int i = 0; i < NBW; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) lsum[i][k] = 0ull;
      if (stid < 16 * nbw) {
        const int col = col0 + stid, i = (w.rbk * c.rb + col) / t.G;
        float* rc = reinterpret_cast<float*>(rowc) + 4 * (stid >> 1) + (stid & 1);
        rc[0] = p.scale[item * c.rb + col];
        rc[2] = kNothing;
        mrow[stid] = i >= w.nd ? 0ull
                     : t.mask ? t.mask[static_cast<int64_t>(w.b) * t.N + i]
                     : i == 63 ? ~0ull : (2ull << i) - 1ull;
      }
      s_sync(half);
      for (int u = w.u0; u < w.u1; ++u, ++n) {
        const bool first_u = u == w.u0, draft = w.draft(u), live = tt < w.tokens(u);
        const bool special = draft || w.tokens(u) < kUnit;
        if (ok) ok = bar_wait(&s_full[n & 1], (n >> 1) & 1, limit, err);
        ok = __all_sync(0xffffffffu, ok);
        fence_after();
        const uint32_t saddr = laddr + c.rb * (n & 1);
        if (special) {  // logits that do not count become -inf
#pragma unroll 1
          for (int i = 0; i < nbw; ++i) {
            uint32_t z[16];
            ld16(z, saddr + 16 * i);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (!live || (draft && !((mrow[16 * i + k] >> (tt & 63)) & 1ull))) z[k] = 0xFF800000u;
            st16(saddr + 16 * i, z);
          }
          wait_st();
        }
        // x - ref of group i's rows, kept in registers for the weights when they fit beside the sums
        uint64_t y[kHeld][8];
        auto relative = [&](int i, uint64_t(&out)[8]) {
          uint32_t z[16];
          ld16(z, saddr + 16 * i);
          wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 rc = rowc[8 * i + k];
            asm("fma.rn.f32x2 %0, %1, %2, %3;"
                : "=l"(out[k])
                : "l"((static_cast<uint64_t>(z[2 * k + 1]) << 32) | z[2 * k]), "l"(pack2(rc.x, rc.y)), "l"(pack2(rc.z, rc.w)));
          }
        };
        bool move = first_u;
        if (!first_u) {  // does any logit pass its row's ref + 15?
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < NBW; ++i)
            if (i < nbw) {
              uint64_t(&x)[8] = y[kKeep ? i : 0];
              relative(i, x);
#pragma unroll
              for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaxf(f32x2_lo(x[k]), f32x2_hi(x[k])));
            }
          move = s_any(half, top > kRefMove);
        }
        if (move) {
          // column maxima of this unit
#pragma unroll 1
          for (int i = 0; i < nbw; ++i) {
            uint32_t z[16];
            ld16(z, saddr + 16 * i);
            wait_ld();
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              x[k] = __uint_as_float(z[k]) * reinterpret_cast<const float*>(rowc)[4 * (8 * i + (k >> 1)) + (k & 1)];
            int col;
            const float m = reduce16(x, lane, &col, [](float a, float b) { return fmaxf(a, b); });
            if (!(lane & 1)) cmax[128 * quarter + 16 * i + col] = m;
          }
          s_sync(half);
          if (stid < 16 * nbw) {
            const float m = fmaxf(fmaxf(cmax[stid], cmax[128 + stid]), fmaxf(cmax[256 + stid], cmax[384 + stid]));
            float* rc = reinterpret_cast<float*>(rowc) + 4 * (stid >> 1) + (stid & 1);
            const float old = rc[2];
            const float now = m == -INFINITY ? old : fminf(old, kRefBelow - m);
            rc[2] = now;
            fac[stid] = now == old ? 1.0f : ex2(now - old);  // 2^(old ref - new ref); nothing seen: 0
          }
          s_sync(half);
          if (!first_u) {
            // the sums and outputs so far, relative to the new references
#pragma unroll
            for (int i = 0; i < NBW; ++i)
              if (i < nbw)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float2 f = *reinterpret_cast<const float2*>(fac + 16 * i + 2 * k);
                  lsum[i][k] = pack2(f32x2_lo(lsum[i][k]) * f.x, f32x2_hi(lsum[i][k]) * f.y);
                }
            const int q = n - 1;  // the last product into the outputs
            if (ok) ok = bar_wait(&pv_empty[q & 1], (q >> 1) & 1, limit, err);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
#pragma unroll 1
            for (int i = 0; i < nbw; ++i) {
              uint32_t z[16];
              ld16(z, laddr + col_o + 16 * i);
              wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) z[k] = __float_as_uint(__uint_as_float(z[k]) * fac[16 * i + k]);
              st16(laddr + col_o + 16 * i, z);
            }
            wait_st();
          }
          if (kKeep)
#pragma unroll
            for (int i = 0; i < NBW; ++i)
              if (i < nbw) relative(i, y[kKeep ? i : 0]);
        }
        // weights
        const int pb = c.np == 2 ? n & 1 : 0, q = n - c.np;  // the buffer, and the unit whose product frees it
        if (q >= 0) {
          if (ok) ok = bar_wait(&pv_empty[q & 1], (q >> 1) & 1, limit, err);
          ok = __all_sync(0xffffffffu, ok);
        }
        unsigned char* prow = smem + L.pw + pb * planes * kPlane + tt * 128;
#pragma unroll
        for (int i = 0; i < NBW; ++i)
          if (i < nbw) {
            uint64_t(&x)[8] = y[kKeep ? i : 0];
            if (!kKeep) relative(i, x);
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float a = ex2(f32x2_lo(x[k])), b = ex2(f32x2_hi(x[k]));
              asm("add.rn.f32x2 %0, %1, %2;" : "=l"(lsum[i][k]) : "l"(lsum[i][k]), "l"(pack2(a, b)));
              const __half2 hh = __floats2half2_rn(a, b);
              h[k] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            const int blk = NBW * half + i;
            unsigned char* dst = prow + (blk >> 2) * kPlane;
            const int c0 = 2 * (blk & 3);
            *reinterpret_cast<uint4*>(dst + (((c0 ^ tt) & 7) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + ((((c0 + 1) ^ tt) & 7) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        fence_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&pv_full[n & 1]);  // (the logits are read, too)
      }
      // ---- the item's end: sums over the tokens, outputs
      s_sync(half);
#pragma unroll
      for (int i = 0; i < NBW; ++i)
        if (i < nbw) {
          float x[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[2 * k] = f32x2_lo(lsum[i][k]);
            x[2 * k + 1] = f32x2_hi(lsum[i][k]);
          }
          int col;
          const float s = reduce16(x, lane, &col, [](float a, float b) { return a + b; });
          if (!(lane & 1)) cmax[128 * quarter + 16 * i + col] = s;
        }
      if (ok) ok = bar_wait(o_full, oph, limit, err);
      oph ^= 1u;
      ok = __all_sync(0xffffffffu, ok);
      const bool fine = !s_any(half, !ok);
      fence_after();
      const bool whole = w.u0 == 0 && w.u1 == w.units;
      const bool has_draft = w.u1 == w.units;
      const long long item_start = first + ((end - first) - w.left) - w.u0;  // first unit of the item
      const int slot = 2 * blockIdx.x + (first < item_start ? 1 : 0);
      const float nan = __int_as_float(0x7fc00000);
      const float unit = reinterpret_cast<const int*>(smem + L.wide)[it % kBadRing] ? 16.0f : 1.0f;  // of the outputs
      // per row: where its dims go (-1: a row past the drafts) and the factor of its outputs
      long long* dest = reinterpret_cast<long long*>(cmax + 512 - col0) + col0;
      if (stid < 16 * nbw) {
        const int col = col0 + stid, row = w.rbk * c.rb + col, i = row / t.G, g = row - i * t.G;
        const float sum = (cmax[stid] + cmax[128 + stid]) + (cmax[256 + stid] + cmax[384 + stid]);
        if (whole) {
          dest[stid] = ((static_cast<long long>(w.b) * t.N + i) * t.Hq + w.hk * t.G + g) * kHeadDim;
          fac[stid] = !fine ? nan : sum == 0.0f ? 0.0f : unit / sum;
        } else {
          dest[stid] = (static_cast<long long>(slot) * c.rb + col) * kHeadDim;
          fac[stid] = fine ? unit : nan;
          p.part_ml[slot * c.rb + col] =
              make_float2(-reinterpret_cast<const float*>(rowc)[4 * (stid >> 1) + 2 + (stid & 1)], fine ? sum : nan);
        }
        if (i >= w.nd) dest[stid] = -1;
      }
      const uint32_t* badi = bad + 64 * (it % kBadRing);
      const bool some_bad = has_draft && __any_sync(0xffffffffu, (lane < w.nd && badi[lane] != 0u) ||
                                                                     (lane + 32 < w.nd && badi[lane + 32] != 0u));
      s_sync(half);
      // tensor-memory lane -> dim: values were paired four dims apart
      const int dim = (tt & ~7) + ((tt & 7) >> 1) + 4 * (tt & 1);
#pragma unroll 1
      for (int blk = 0; blk < nbw; ++blk) {
        uint32_t z[16];
        ld16(z, laddr + col_o + 16 * blk);
        wait_ld();
        if (some_bad) {  // drafted values that are not finite
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            bool hit = false;
            for (int d = 0; d < w.nd; ++d) hit |= ((badi[d] >> (dim >> 5)) & 1u) && ((mrow[16 * blk + k] >> d) & 1ull);
            if (hit) z[k] = 0x7fc00000u;
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const long long to = dest[16 * blk + k];
          const float f = fac[16 * blk + k], o = f == 0.0f ? 0.0f : __uint_as_float(z[k]) * f;
          if (to < 0) continue;
          if (whole) static_cast<__nv_bfloat16*>(t.O)[to + dim] = __float2bfloat16_rn(o);
          else p.part_o[to + dim] = o;
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(o_empty);
      s_sync(half);  // the row constants and sums may be overwritten
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kMmaWarp && elect_one()) {
      // ========================================================== products
      bool ok = true;
      int n = 0, ring = 0, item = 0;
      uint32_t aph = 0;
      const uint32_t sq_base = smem_u32(smem + L.sq), v_base = smem_u32(smem + L.v), p_base = smem_u32(smem + L.pw);
      const int p_bytes = (c.rb > 64 ? 2 : 1) * kPlane;
      const uint32_t id_s = idesc_f16(c.rb, false, 0, 0), id_o = idesc_f16(c.rb, false, 1, 1);
      const bool half_step = ((t.m + t.m_out) & 32) != 0;  // an odd number of sign words ends in half a step
      const uint32_t sq_bytes = static_cast<uint32_t>(c.nk) * c.rb * 128;
      bool sq_out = false;  // a copy of the projected queries is in flight
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = bar_wait(bar, parity, limit, err);
      };
      auto values = [&](int q, bool first_u, bool last_u) {  // O += V^T P of unit q
        const int pb = c.np == 2 ? q & 1 : 0, vb = q & 1;
        wait(&pv_full[vb], (q >> 1) & 1);
        if (first_u && item > 0) wait(o_empty, (item - 1) & 1);
        if (!ok) return;
        fence_after();
        const uint64_t vd = desc_mn(v_base + vb * kVBytes, kPlane), pd = desc_mn(p_base + pb * p_bytes, kPlane);
        const volatile int* turns = reinterpret_cast<const int*>(smem + L.wide) + kBadRing;
        if (turns[vb] == q) mma_ss_mn2<4>(tmem + col_o, vd, pd, id_o, true);  // the outputs so far divided by 16
        else mma_ss_mn2<0>(tmem + col_o, vd, pd, id_o, !first_u);
#pragma unroll
        for (int ks = 2; ks < kUnit / 16; ks += 2)
          mma_ss_mn2<0>(tmem + col_o, vd + ks * 128, pd + ks * 128, id_o, true);
        commit(&pv_empty[vb]);
        if (last_u) commit(o_full);
      };
      for (bool more = any; more && ok; more = w.next<false>(p), ++item) {
        // the last item's score products are done: its logits were read (s_full was waited for by the weights, and
        // `values` of its last unit waited for those)
        bar_expect(sq_full, sq_bytes);
        bulk_load(sq_base, p.image + (w.bh(p) * c.nrb + w.rbk) * static_cast<int64_t>(sq_bytes), sq_bytes, sq_full);
        sq_out = true;
        wait(sq_full, item & 1);
        if (!ok) break;
        sq_out = false;
        for (int u = w.u0; u < w.u1 && ok; ++u, ++n) {
          // (the logits of unit n - 2 in this buffer were read before its weights, which `values` waited for)
          uint64_t qd = desc_k(sq_base);
          const uint32_t sd = tmem + c.rb * (n & 1);
#pragma unroll 1
          for (int k0 = 0; k0 < c.nk; k0 += c.ck) {
            wait(&a_full[ring], aph);
            if (!ok) break;
            fence_after();
            uint32_t ad = tmem + col_a + 32 * c.ck * ring;
            const int k1 = min(c.nk, k0 + c.ck), full = k1 == c.nk && half_step ? k1 - 1 : k1;
#pragma unroll 1
            for (int kc = k0; kc < full; ++kc, ad += 32, qd += c.rb * 8) mma_ts_64<true>(sd, ad, qd, id_s, kc > 0);
            if (full < k1) mma_ts_64<false>(sd, ad, qd, id_s, full > 0);
            commit(&a_empty[ring]);
            ring ^= 1;
            aph ^= ring == 0 ? 1u : 0u;
          }
          if (!ok) break;
          commit(&s_full[n & 1]);
          if (u > w.u0) values(n - 1, u - 1 == w.u0, false);
        }
        if (ok) values(n - 1, w.u1 - 1 == w.u0, true);
      }
      // every product issued here ends before the block gives its memory back
      commit(drain);
      bar_wait(drain, 0, limit_drain, nullptr);
      if (sq_out) bar_wait(sq_full, item & 1, limit_drain, nullptr);
    }
    __syncwarp();
    if (warp == kLoadWarp) {
      // ========================================================== cache tiles (the whole warp, one lane copies)
      bool ok = true;
      int st = 0, issued = 0;
      uint32_t eph = 1;
      for (bool more = any; more && ok; more = w.next<true>(p)) {
        const int64_t bh = w.bh(p);
        for (int u = w.u0; u < w.u1; ++u) {
          ok = __all_sync(0xffffffffu, bar_wait(&raw_empty[st], eph, limit, err));
          if (!ok) break;
          const unsigned char* src;
          int tiles = 1;
          if (w.draft(u)) {
            src = t.draft + bh * (t.draft_cap / kDecodeTileTokens) * static_cast<int64_t>(t.tl.bytes);
          } else {
            src = t.tiles + (bh * (t.cap / kDecodeTileTokens) + 2 * u) * static_cast<int64_t>(t.tl.bytes);
            tiles = w.len - u * kUnit > kDecodeTileTokens ? 2 : 1;
          }
          const uint32_t bytes = static_cast<uint32_t>(tiles * t.tl.bytes);
          if (lane == 0) {
            bar_expect(&raw_full[st], bytes);
            bulk_load(smem_u32(smem + L.raw + st * c.stage), src, bytes, &raw_full[st]);
          }
          __syncwarp();
          ++issued;
          if (++st == c.ns) {
            st = 0;
            eph ^= 1u;
          }
        }
      }
      // every copy issued here lands before the block gives its memory back
      for (int q = issued > c.ns ? issued - c.ns : 0; q < issued; ++q)
        bar_wait(&raw_full[q % c.ns], (q / c.ns) & 1, limit_drain, nullptr);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---------------------------------------------------------------- join

// One warp per output row: rows past the drafts are zero, rows of an item that
// one block held whole are already written, the others are joined from the
// parts of the blocks that share the item, four parts in flight at a time. In
// 32 bits: the units of any cache that a device holds fit 31.
__global__ void __launch_bounds__(256) tree_join_kernel(TreeTcParams p) {
  griddep_wait();
  const TreeParams& t = p.t;
  const int row = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);  // (at most 65535 * 8 * 64)
  const int lane = threadIdx.x & 31;
  if (row >= t.B * t.N * t.Hq) return;
  const int bi = row / t.Hq, h = row - bi * t.Hq, b = bi / t.N, i = bi - b * t.N;
  const int total = static_cast<int>(p.start[t.B]), nd = seq_drafts(t, b), units = seq_units(t, b);
  int u0 = static_cast<int>(p.start[b]);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t.O) + static_cast<int64_t>(row) * kHeadDim + 4 * lane;
  if (i >= nd) {
    *reinterpret_cast<uint2*>(out) = make_uint2(0u, 0u);
    return;
  }
  const int hk = h / t.G, r = i * t.G + h - hk * t.G, rbk = r / p.c.rb, col = r - rbk * p.c.rb;
  u0 += (hk * ((nd * t.G + p.c.rb - 1) / p.c.rb) + rbk) * units;
  // the block of unit u: floor(((u + 1) grid - 1) / total); the quotient of these exact doubles is off by less than
  // its distance to an integer, 1 / total
  auto block_of = [&](int u) {
    return static_cast<int>((static_cast<double>(u + 1) * p.grid - 1.0) / static_cast<double>(total));
  };
  const int c0 = block_of(u0), c1 = block_of(u0 + units - 1);
  if (c0 == c1) return;
  const int q = total / p.grid, rest = total - q * p.grid;
  auto first = [&](int c) { return q * c + rest * c / p.grid; };  // first unit of block c
  float M = -kNothing, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int c = c0; c <= c1; c += 4) {
    float2 ml[4];
    float4 o[4];
    float top = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ml[k] = make_float2(-kNothing, 0.0f);
      o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int s0 = first(c + k);
      // (with more blocks than units some of them have none)
      if (c + k <= c1 && s0 != first(c + k + 1)) {
        const int s = (2 * (c + k) + (s0 < u0 ? 1 : 0)) * p.c.rb + col;
        ml[k] = p.part_ml[s];
        o[k] = reinterpret_cast<const float4*>(p.part_o)[static_cast<int64_t>(s) * (kHeadDim / 4) + lane];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
    const float f = M == top ? 1.0f : exp2f(M - top);
    M = top;
    L *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ml[k].y == 0.0f) continue;  // nothing seen (a NaN sum stays)
      const float g = ml[k].x == M ? 1.0f : exp2f(ml[k].x - M);
      L = fmaf(ml[k].y, g, L);
      acc.x = fmaf(o[k].x, g, acc.x);
      acc.y = fmaf(o[k].y, g, acc.y);
      acc.z = fmaf(o[k].z, g, acc.z);
      acc.w = fmaf(o[k].w, g, acc.w);
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

}  // namespace

size_t tree_tc_ws_bytes(int B, int N, int Hq, int Hkv, int m, int m_out, int vbits, int num_sms) {
  return tree_tc_ws(tree_tc_cfg(N, Hq / Hkv, m, m_out, tile_layout(m, m_out, vbits).bytes), B, Hkv, num_sms).total;
}

cudaError_t launch_tree_attention_tc(const TreeParams& t, cudaStream_t s) {
  TreeTcParams p{};
  p.t = t;
  p.c = tree_tc_cfg(t.N, t.G, t.m, t.m_out, t.tl.bytes);
  if (p.c.smem > 227 * 1024) return cudaErrorInvalidConfiguration;
  const TreeTcWs w = tree_tc_ws(p.c, t.B, t.Hkv, t.num_sms);
  p.start = reinterpret_cast<long long*>(t.ws + w.start);
  p.image = t.ws + w.image;
  p.scale = reinterpret_cast<float*>(t.ws + w.scale);
  p.part_o = reinterpret_cast<float*>(t.ws + w.part_o);
  p.part_ml = reinterpret_cast<float2*>(t.ws + w.part_ml);
  const int64_t units = (static_cast<int64_t>(t.T) + kUnit - 1) / kUnit + 1;
  const int64_t most = static_cast<int64_t>(t.B) * t.Hkv * p.c.nrb * units;
  p.grid = static_cast<int>(most < t.num_sms ? most : t.num_sms);
  // one block per SM: it takes all tensor-memory columns
  const size_t smem = p.c.smem < 116 * 1024 ? 116 * 1024 : static_cast<size_t>(p.c.smem);
  void (*const kernels[])(TreeTcParams) = {
      tree_tc_kernel<1, 4>, tree_tc_kernel<2, 4>, tree_tc_kernel<3, 4>, tree_tc_kernel<4, 4>,
      tree_tc_kernel<1, 2>, tree_tc_kernel<2, 2>, tree_tc_kernel<3, 2>, tree_tc_kernel<4, 2>};
  void (*const kernel)(TreeTcParams) = kernels[(t.tl.vbits == 4 ? 0 : 4) + (p.c.rb / 16 + 1) / 2 - 1];
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.c.nrb * p.c.rb / 16), static_cast<unsigned>(t.B * t.Hkv));
  cfg.blockDim = dim3(32 * kPrepWarps);
  e = cudaLaunchKernelEx(&cfg, tree_prepare_kernel, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(kTreeTcThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(t.B) * t.N * t.Hq;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel, p);
}

}  // namespace qjl
