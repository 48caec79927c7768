// Attention of drafted tokens over the QJL cache, in fp32 on the CUDA cores (fp32
// queries; bf16 ones take tree_attention_tc.cu).
//
// Rows: the N drafted tokens of a sequence times the G query heads of a kv
// head, row r = i G + g. With the projected query sq (m + m_out values, the
// estimator's factors, sm_scale and log2(e) folded in),
//   x_t = |k_in| sum_i sq_i sign_i + |k_out| sum_i sq_out_i sign_out_i,
// and the softmax runs online over units of 128 tokens with base 2. The last
// unit of a pair is its draft tile, where bit t of a row's mask decides.
//   1. tree_project_kernel: sq of every row, [pair][row block][projection][8],
//      a warp per projection (the row of S is one coalesced line)
//   2. tree_chunk_kernel: one block per (split of the units, row block of 8,
//      pair). A unit's two tiles are staged in shared memory; a thread sums one
//      token's scores for four rows (each sign word is read once for them), then
//      owns one channel of the four rows' outputs
//   3. tree_merge_kernel: the splits' (o, M, L) of a row, joined exactly
// Bound: the fp32 additions, 2 (m + m_out + 128) per row and token; few rows and
// tokens are bound by the three launches (33 us for 2 x 1024 tokens, 56 rows).
// A weight of zero takes no part in the draft tile, whatever the value holds
// (0 * inf must not reach the row); slots past the lengths are not used.
#include <algorithm>

#include "qjl_internal.cuh"

namespace qjl {
namespace {

constexpr int kTreeRows = 8;      // rows of a block
constexpr int kTreeUnit = 128;    // tokens of a unit, one per thread of a half
constexpr int kTreeThreads = 2 * kTreeUnit;  // half h of the block takes rows 4h .. 4h + 3
constexpr int kTreeHalf = kTreeRows / 2;
constexpr int kTreeProjSplit = 8; // blocks that share the projections of 8 rows

int tree_row_blocks(int N, int G) { return (N * G + kTreeRows - 1) / kTreeRows; }
// Splits of a pair's units: enough blocks for four per SM. With 1, 2, 4 and 8: 2 x
// 4096 tokens, 56 rows on one kv head 90, 90, 68, 68 us; 8 x 4096, 64 rows, 4 kv heads
// 855, 810, 781, 714; 2 x 1024 30 throughout. The workspace grows with them.
int tree_splits(int pairs, int row_blocks, int num_sms) {
  const int64_t b = static_cast<int64_t>(pairs) * row_blocks;
  const int64_t n = (4 * static_cast<int64_t>(num_sms) + b - 1) / b;
  return static_cast<int>(n < 1 ? 1 : n);
}

struct TreeWs {
  size_t sq, part_o, part_ml, total;
};
TreeWs tree_ws_fp32(int B, int N, int Hq, int Hkv, int m, int m_out, int num_sms) {
  auto a256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t pairs = static_cast<size_t>(B) * Hkv;
  const int rb = tree_row_blocks(N, Hq / Hkv);
  const size_t rows = pairs * rb * kTreeRows;
  const size_t splits = tree_splits(B * Hkv, rb, num_sms);
  TreeWs w{};
  w.sq = 0;
  w.part_o = a256(rows * (m + m_out) * sizeof(float));
  w.part_ml = w.part_o + a256(splits * rows * kHeadDim * sizeof(float));
  w.total = w.part_ml + a256(splits * rows * 2 * sizeof(float));
  return w;
}

__global__ void __launch_bounds__(kTreeThreads) tree_project_kernel(TreeParams p, float* sq) {
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / p.Hkv), hk = static_cast<int>(bh % p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rb = gridDim.x, proj = p.m + p.m_out;
  // lane l owns channels 4l .. 4l + 3 of the 8 rows
  uint32_t mine = 0u;  // its outlier channels
  for (int o = 0; o < p.n_out; ++o) {
    const int c = p.idx[bh * p.n_out + o];
    if ((c >> 2) == lane) mine |= 1u << (c & 3);
  }
  float4 q[kTreeRows];
#pragma unroll
  for (int k = 0; k < kTreeRows; ++k) {
    const int r = blockIdx.x * kTreeRows + k, i = r / p.G, g = r % p.G;
    q[k] = i < p.N ? reinterpret_cast<const float4*>(static_cast<const float*>(p.Q) + b * p.q_sb + i * p.q_sn +
                                                     (static_cast<int64_t>(hk) * p.G + g) * p.q_sh)[lane]
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  float* out = sq + (bh * rb + blockIdx.x) * static_cast<int64_t>(proj) * kTreeRows;
#pragma unroll 2
  for (int i = blockIdx.z * (kTreeThreads / 32) + warp; i < proj; i += kTreeProjSplit * (kTreeThreads / 32)) {
    const bool second = i >= p.m;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(second ? p.S_out + (i - p.m) * kHeadDim : p.S + i * kHeadDim) + lane);
    const uint32_t use = second ? mine : ~mine;
    const float s0 = use & 1u ? __uint_as_float(w.x << 16) : 0.0f, s1 = use & 2u ? __uint_as_float(w.x & 0xFFFF0000u) : 0.0f;
    const float s2 = use & 4u ? __uint_as_float(w.y << 16) : 0.0f, s3 = use & 8u ? __uint_as_float(w.y & 0xFFFF0000u) : 0.0f;
    // (a product with a masked zero would carry a non-finite query channel into the other part)
    float a[kTreeRows];
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) {
      float x = 0.0f;
      if (use & 1u) x = fmaf(q[k].x, s0, x);
      if (use & 2u) x = fmaf(q[k].y, s1, x);
      if (use & 4u) x = fmaf(q[k].z, s2, x);
      if (use & 8u) x = fmaf(q[k].w, s3, x);
      a[k] = x;
    }
    // over the lanes: after the halving steps lane l holds row (l >> 2) & 7, summed over 8 lanes
#pragma unroll
    for (int st = 0; st < 3; ++st) {
      const int off = 16 >> st, n = 4 >> st;
      const bool up = lane & off;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float send = up ? a[k] : a[k + n], keep = up ? a[k + n] : a[k];
        a[k] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
    }
    float v = a[0];
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    if ((lane & 3) == 0)
      out[i * kTreeRows + ((lane >> 2) & 7)] = v * (kSqrtHalfPi / static_cast<float>(second ? p.m_out : p.m) * p.sm_scale_log2);
  }
}

__global__ void __launch_bounds__(kTreeThreads) tree_chunk_kernel(TreeParams p, const float* __restrict__ sq,
                                                                  float* part_o, float* part_ml) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float4 ps[2][kTreeUnit];  // weights of a half's rows, by token
  __shared__ float ms[kTreeRows], ls[kTreeRows], fs[kTreeRows];
  float4* sqs = reinterpret_cast<float4*>(smem);  // [projection][2 halves]
  const int proj = p.m + p.m_out, wpt = p.m / 32, wpo = p.m_out / 32;
  unsigned char* raw = smem + proj * kTreeRows * 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = tid >> 7, tt = tid & 127;
  const int rb = gridDim.y, blk = blockIdx.y;
  const int64_t bh = blockIdx.z;
  const int b = static_cast<int>(bh / p.Hkv);
  const int len = p.seqlens ? min(max(p.seqlens[b], 0), p.T) : p.T;
  const int nd = p.n_draft ? min(max(p.n_draft[b], 0), p.N) : p.N;
  const int units = (len + kTreeUnit - 1) / kTreeUnit + 1;
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  const int64_t prow = (static_cast<int64_t>(blockIdx.x) * gridDim.z + bh) * rb * kTreeRows + blk * kTreeRows;
  if (tid < kTreeRows) {
    ms[tid] = -INFINITY;
    ls[tid] = 0.0f;
  }
  const bool any = blk * kTreeRows < nd * p.G && u0 < u1;
  if (any) {
    const float4* src = reinterpret_cast<const float4*>(sq + (bh * rb + blk) * static_cast<int64_t>(proj) * kTreeRows);
    for (int e = tid; e < 2 * proj; e += kTreeThreads) sqs[e] = src[e];
  }
  float o[kTreeHalf];  // channel tt of the half's rows
#pragma unroll
  for (int k = 0; k < kTreeHalf; ++k) o[k] = 0.0f;
  for (int u = u0; u < u1 && any; ++u) {
    const bool drafts = u == units - 1;
    const int t0 = drafts ? 0 : u * kTreeUnit;
    const int n = drafts ? nd : min(kTreeUnit, len - t0);
    if (n <= 0) continue;
    const unsigned char* from = drafts ? p.draft + bh * (p.draft_cap / kDecodeTileTokens) * static_cast<int64_t>(p.tl.bytes)
                                       : p.tiles + (bh * (p.cap / kDecodeTileTokens) + 2 * u) * static_cast<int64_t>(p.tl.bytes);
    __syncthreads();  // the last unit is done with
    const int chunks = (n > kDecodeTileTokens ? 2 : 1) * p.tl.bytes / 16;
    for (int e = tid; e < chunks; e += kTreeThreads) reinterpret_cast<uint4*>(raw)[e] = __ldg(reinterpret_cast<const uint4*>(from) + e);
    __syncthreads();
    const int j = tt & 63;
    // ---- scores of token tt
    float x[kTreeHalf] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (tt < n) {
      const unsigned char* tile = raw + (tt >> 6) * p.tl.bytes;
      const float2 norm = __half22float2(reinterpret_cast<const __half2*>(tile + p.tl.knorm)[j]);
      float part[2][kTreeHalf];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int k = 0; k < kTreeHalf; ++k) part[w][k] = 0.0f;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + (w ? p.tl.kbits_out : p.tl.kbits)) + j * (w ? wpo : wpt);
        const float4* sp = sqs + (w ? 2 * p.m : 0) + half;
        for (int i = 0; i < (w ? wpo : wpt); ++i) {
          const uint32_t neg = ~src[i];
#pragma unroll 8
          for (int bit = 0; bit < 32; ++bit) {
            const uint32_t s = (neg >> bit) << 31;
            const float4 v = sp[2 * (32 * i + bit)];
            part[w][0] += __uint_as_float(__float_as_uint(v.x) ^ s);
            part[w][1] += __uint_as_float(__float_as_uint(v.y) ^ s);
            part[w][2] += __uint_as_float(__float_as_uint(v.z) ^ s);
            part[w][3] += __uint_as_float(__float_as_uint(v.w) ^ s);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kTreeHalf; ++k) {
        const int i = (blk * kTreeRows + kTreeHalf * half + k) / p.G;
        bool ok = i < nd;
        if (drafts && ok) ok = p.mask ? (p.mask[static_cast<int64_t>(b) * p.N + i] >> tt) & 1ull : tt <= i;
        if (ok) x[k] = fmaf(norm.x, part[0][k], wpo ? norm.y * part[1][k] : 0.0f);
      }
    }
    ps[half][tt] = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    // ---- per row (warp r): maximum, weights, sum
    {
      float* row = reinterpret_cast<float*>(ps[warp / kTreeHalf]) + warp % kTreeHalf;
      float v[kTreeUnit / 32], top = -INFINITY;
#pragma unroll
      for (int e = 0; e < kTreeUnit / 32; ++e) {
        v[e] = row[4 * (lane + 32 * e)];
        top = fmaxf(top, v[e]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float old = ms[warp], now = fmaxf(old, top);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < kTreeUnit / 32; ++e) {
        // a row with nothing so far: every v is -inf and its weight 0
        const float w = v[e] == -INFINITY ? 0.0f : exp2f(v[e] - now);
        row[4 * (lane + 32 * e)] = w;
        sum += w;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      __syncwarp();
      if (lane == 0) {
        const float f = old == now ? 1.0f : exp2f(old - now);
        fs[warp] = f;
        ls[warp] = fmaf(ls[warp], f, sum);
        ms[warp] = now;
      }
    }
    __syncthreads();
    // ---- values: channel tt
#pragma unroll
    for (int k = 0; k < kTreeHalf; ++k) o[k] *= fs[kTreeHalf * half + k];
    const int g = tt / kValueGroup;
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      const int jt = t & 63;
      const unsigned char* tile = raw + (t >> 6) * p.tl.bytes;
      const float2 sz = __half22float2(reinterpret_cast<const __half2*>(tile + p.tl.vsz)[jt * (kHeadDim / kValueGroup) + g]);
      const int code = p.tl.vbits == 2
                           ? (tile[p.tl.vcode + v2_line(g, (tt % 32) / 4) + jt] >> (2 * (tt % 4))) & 3
                           : (tile[p.tl.vcode + jt * (kHeadDim / 2) + 16 * vcode_chunk(jt, g) + (tt % 32) / 2] >> (4 * (tt % 2))) & 15;
      const float v = fmaf(static_cast<float>(code), sz.x, sz.y);
      const float4 w = ps[half][t];
      // (in the draft tile a weight of zero takes no part)
      if (!drafts || w.x != 0.0f) o[0] = fmaf(w.x, v, o[0]);
      if (!drafts || w.y != 0.0f) o[1] = fmaf(w.y, v, o[1]);
      if (!drafts || w.z != 0.0f) o[2] = fmaf(w.z, v, o[2]);
      if (!drafts || w.w != 0.0f) o[3] = fmaf(w.w, v, o[3]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTreeHalf; ++k) part_o[(prow + kTreeHalf * half + k) * kHeadDim + tt] = o[k];
  if (tid < kTreeRows) {
    part_ml[2 * (prow + tid)] = ms[tid];
    part_ml[2 * (prow + tid) + 1] = ls[tid];
  }
}

// One warp per output row (b, i, query head); lane l owns channels 4l .. 4l + 3.
__global__ void __launch_bounds__(256) tree_merge_kernel(TreeParams p, const float* __restrict__ part_o,
                                                         const float* __restrict__ part_ml, int splits, int rb) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(p.B) * p.N * p.Hq) return;
  const int h = static_cast<int>(row % p.Hq), i = static_cast<int>(row / p.Hq % p.N);
  const int64_t b = row / p.Hq / p.N;
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
  const int64_t in_split = (b * p.Hkv + h / p.G) * rb * kTreeRows + i * p.G + h % p.G;
  const int64_t stride = pairs * rb * kTreeRows;
  float M = -INFINITY, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = lane; s < splits; s += 32) M = fmaxf(M, part_ml[2 * (s * stride + in_split)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const int64_t r = s * stride + in_split;
    const float2 ml = reinterpret_cast<const float2*>(part_ml)[r];
    if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // (a NaN sum stays)
    const float f = ml.x == M ? 1.0f : exp2f(ml.x - M);
    const float4 o = reinterpret_cast<const float4*>(part_o)[r * (kHeadDim / 4) + lane];
    L = fmaf(ml.y, f, L);
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  reinterpret_cast<float4*>(static_cast<float*>(p.O) + row * kHeadDim)[lane] =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

cudaError_t launch_tree_fp32(const TreeParams& p, cudaStream_t s) {
  const int rb = tree_row_blocks(p.N, p.G);
  const int pairs = p.B * p.Hkv;
  // (a split per unit at most)
  const int units = static_cast<int>((static_cast<int64_t>(p.T) + kTreeUnit - 1) / kTreeUnit) + 1;
  const int splits = std::min(tree_splits(pairs, rb, p.num_sms), units);
  const TreeWs w = tree_ws_fp32(p.B, p.N, p.Hq, p.Hkv, p.m, p.m_out, p.num_sms);
  float* sq = reinterpret_cast<float*>(p.ws + w.sq);
  float* part_o = reinterpret_cast<float*>(p.ws + w.part_o);
  float* part_ml = reinterpret_cast<float*>(p.ws + w.part_ml);
  const size_t smem = static_cast<size_t>(p.m + p.m_out) * kTreeRows * 4 + 2 * p.tl.bytes;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(tree_chunk_kernel), smem);
  if (e != cudaSuccess) return e;
  tree_project_kernel<<<dim3(rb, pairs, kTreeProjSplit), kTreeThreads, 0, s>>>(p, sq);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  tree_chunk_kernel<<<dim3(splits, rb, pairs), kTreeThreads, smem, s>>>(p, sq, part_o, part_ml);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.N * p.Hq;
  tree_merge_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(p, part_o, part_ml, splits, rb);
  return cudaGetLastError();
}

}  // namespace

// One size for both dtypes: what a call of N drafts uses.
size_t tree_ws_used(int B, int N, int Hq, int Hkv, int m, int m_out, int vbits, int num_sms) {
  const size_t a = tree_ws_fp32(B, N, Hq, Hkv, m, m_out, num_sms).total;
  const size_t b = tree_tc_ws_bytes(B, N, Hq, Hkv, m, m_out, vbits, num_sms);
  return a > b ? a : b;
}

// For up to N drafts. What a call uses does not grow with N throughout: its parts
// have a row block's rows, and one row more than fills a row block makes two
// smaller ones (32 and 33 drafts of 4 query heads: 20.4 and 13.1 MB).
size_t tree_ws_bytes(int B, int N, int Hq, int Hkv, int m, int m_out, int vbits, int num_sms) {
  size_t most = 0;
  for (int n = 1; n <= N; ++n) most = std::max(most, tree_ws_used(B, n, Hq, Hkv, m, m_out, vbits, num_sms));
  return most;
}

cudaError_t launch_tree_attention(const TreeParams& p, qjl_dtype dt, cudaStream_t s) {
  return dt == QJL_BF16 ? launch_tree_attention_tc(p, s) : launch_tree_fp32(p, s);
}

}  // namespace qjl
