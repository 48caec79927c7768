// Attention of drafted tokens over the QJL cache, in fp32 on the CUDA cores (fp32
// queries; bf16 ones take tree_attention_tc.cu).
//
// Rows: the N drafted tokens of a sequence times the G query heads of a kv
// head, row r = i G + g. With the projected query sq (m + m_out values, the
// estimator's factors, sm_scale and log2(e) folded in),
//   x_t = |k_in| sum_i sq_i sign_i + |k_out| sum_i sq_out_i sign_out_i,
// and the softmax runs online over units of 128 tokens with base 2. The last
// unit of a pair is its draft tile, where bit t of a row's mask decides.
//   1. tree_project_kernel: sq of every row, [pair][row block][projection][8]
//   2. tree_chunk_kernel: one block per (split of the units, row block of 8,
//      pair): a thread sums one token's scores for the 8 rows (each sign word is
//      read once for the 8 rows), then owns one channel of the outputs
//   3. tree_merge_kernel: the splits' (o, M, L) of a row, joined exactly
// A weight of zero takes no part in the draft tile, whatever the value holds
// (0 * inf must not reach the row); slots past the lengths are not read.
#include "qjl_internal.cuh"

namespace qjl {
namespace {

constexpr int kTreeRows = 8;      // rows of a block
constexpr int kTreeUnit = 128;    // tokens of a unit, one per thread
constexpr int kTreeThreads = 128;

int tree_row_blocks(int N, int G) { return (N * G + kTreeRows - 1) / kTreeRows; }
// Splits of a pair's units: enough blocks for four per SM.
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
  __shared__ float q[kHeadDim][kTreeRows];
  __shared__ bool outl[kHeadDim];
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / p.Hkv), hk = static_cast<int>(bh % p.Hkv), c = threadIdx.x;
  const int rb = gridDim.x, proj = p.m + p.m_out;
  bool outlier = false;
  for (int o = 0; o < p.n_out; ++o) outlier |= p.idx[bh * p.n_out + o] == c;
  outl[c] = outlier;
#pragma unroll
  for (int k = 0; k < kTreeRows; ++k) {
    const int r = blockIdx.x * kTreeRows + k, i = r / p.G, g = r % p.G;
    q[c][k] = i < p.N ? static_cast<const float*>(p.Q)[b * p.q_sb + i * p.q_sn + (hk * p.G + g) * p.q_sh + c] : 0.0f;
  }
  __syncthreads();
  float* out = sq + (bh * rb + blockIdx.x) * static_cast<int64_t>(proj) * kTreeRows;
  for (int i = threadIdx.x; i < proj; i += kTreeThreads) {
    const bool second = i >= p.m;
    float acc[kTreeRows];
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) acc[k] = 0.0f;
    for (int cc = 0; cc < kHeadDim; ++cc) {
      if (outl[cc] != second) continue;
      const float s = __bfloat162float(second ? p.S_out[(i - p.m) * kHeadDim + cc] : p.St[static_cast<int64_t>(cc) * p.m + i]);
#pragma unroll
      for (int k = 0; k < kTreeRows; ++k) acc[k] = fmaf(s, q[cc][k], acc[k]);
    }
    const float f = kSqrtHalfPi / static_cast<float>(second ? p.m_out : p.m) * p.sm_scale_log2;
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) out[i * kTreeRows + k] = acc[k] * f;
  }
}

__global__ void __launch_bounds__(kTreeThreads) tree_chunk_kernel(TreeParams p, const float* __restrict__ sq,
                                                                  float* part_o, float* part_ml) {
  __shared__ float ps[kTreeRows][kTreeUnit];
  __shared__ float ms[kTreeRows], ls[kTreeRows], fs[kTreeRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rb = gridDim.y, blk = blockIdx.y;
  const int64_t bh = blockIdx.z;
  const int b = static_cast<int>(bh / p.Hkv);
  const int len = p.seqlens ? min(max(p.seqlens[b], 0), p.T) : p.T;
  const int nd = p.n_draft ? min(max(p.n_draft[b], 0), p.N) : p.N;
  const int units = (len + kTreeUnit - 1) / kTreeUnit + 1;
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  const int proj = p.m + p.m_out, wpt = p.m / 32, wpo = p.m_out / 32;
  const float* sqr = sq + (bh * rb + blk) * static_cast<int64_t>(proj) * kTreeRows;
  const int64_t prow = (static_cast<int64_t>(blockIdx.x) * gridDim.z + bh) * rb * kTreeRows + blk * kTreeRows;
  if (tid < kTreeRows) {
    ms[tid] = -INFINITY;
    ls[tid] = 0.0f;
  }
  float o[kTreeRows];  // channel tid
#pragma unroll
  for (int k = 0; k < kTreeRows; ++k) o[k] = 0.0f;
  const bool any = blk * kTreeRows < nd * p.G;
  for (int u = u0; u < u1 && any; ++u) {
    const bool drafts = u == units - 1;
    const int t0 = drafts ? 0 : u * kTreeUnit;
    const int n = drafts ? nd : min(kTreeUnit, len - t0);
    if (n <= 0) continue;
    unsigned char* base = const_cast<unsigned char*>(drafts ? p.draft : p.tiles);
    const int cap = drafts ? p.draft_cap : p.cap;
    // ---- scores of token tid
    float x[kTreeRows];
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) x[k] = -INFINITY;
    if (tid < n) {
      int j;
      const unsigned char* tile = tile_of(base, p.tl, bh, cap, t0 + tid, &j);
      const float2 norm = __half22float2(reinterpret_cast<const __half2*>(tile + p.tl.knorm)[j]);
      float part[2][kTreeRows];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int k = 0; k < kTreeRows; ++k) part[w][k] = 0.0f;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + (w ? p.tl.kbits_out : p.tl.kbits)) + j * (w ? wpo : wpt);
        const float4* sp = reinterpret_cast<const float4*>(sqr + (w ? p.m : 0) * kTreeRows);
        for (int i = 0; i < (w ? wpo : wpt); ++i) {
          const uint32_t neg = ~src[i];
#pragma unroll 8
          for (int bit = 0; bit < 32; ++bit) {
            const uint32_t s = (neg >> bit) << 31;
            const float4 lo = __ldg(sp + 2 * (32 * i + bit)), hi = __ldg(sp + 2 * (32 * i + bit) + 1);
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int k = 0; k < kTreeRows; ++k) part[w][k] += __uint_as_float(__float_as_uint(v[k]) ^ s);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kTreeRows; ++k) {
        const int i = (blk * kTreeRows + k) / p.G;
        bool ok = i < nd;
        if (drafts && ok) ok = p.mask ? (p.mask[static_cast<int64_t>(b) * p.N + i] >> tid) & 1ull : tid <= i;
        if (ok) x[k] = fmaf(norm.x, part[0][k], wpo ? norm.y * part[1][k] : 0.0f);
      }
    }
    __syncthreads();  // the last unit's weights are read
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) ps[k][tid] = x[k];
    __syncthreads();
    // ---- per row: maximum, weights, sum; warp w takes rows w and w + 4
    for (int k = warp; k < kTreeRows; k += kTreeThreads / 32) {
      float v[kTreeUnit / 32], top = -INFINITY;
#pragma unroll
      for (int e = 0; e < kTreeUnit / 32; ++e) {
        v[e] = ps[k][lane + 32 * e];
        top = fmaxf(top, v[e]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float old = ms[k], now = fmaxf(old, top);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < kTreeUnit / 32; ++e) {
        // a row with nothing so far: every v is -inf and its weight 0
        const float w = v[e] == -INFINITY ? 0.0f : exp2f(v[e] - now);
        ps[k][lane + 32 * e] = w;
        sum += w;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) {
        const float f = old == now ? 1.0f : exp2f(old - now);
        fs[k] = f;
        ls[k] = fmaf(ls[k], f, sum);
        ms[k] = now;
      }
    }
    __syncthreads();
    // ---- values: channel tid
#pragma unroll
    for (int k = 0; k < kTreeRows; ++k) o[k] *= fs[k];
    const int g = tid / kValueGroup;
    for (int t = 0; t < n; ++t) {
      int j;
      const unsigned char* tile = tile_of(base, p.tl, bh, cap, t0 + t, &j);
      const float2 sz = __half22float2(reinterpret_cast<const __half2*>(tile + p.tl.vsz)[j * (kHeadDim / kValueGroup) + g]);
      int code;
      if (p.tl.vbits == 2)
        code = (tile[p.tl.vcode + v2_line(g, (tid % 32) / 4) + j] >> (2 * (tid % 4))) & 3;
      else
        code = (tile[p.tl.vcode + j * (kHeadDim / 2) + 16 * vcode_chunk(j, g) + (tid % 32) / 2] >> (4 * (tid % 2))) & 15;
      const float v = fmaf(static_cast<float>(code), sz.x, sz.y);
#pragma unroll
      for (int k = 0; k < kTreeRows; ++k) {
        const float w = ps[k][t];
        if (!drafts || w != 0.0f) o[k] = fmaf(w, v, o[k]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTreeRows; ++k) part_o[(prow + k) * kHeadDim + tid] = o[k];
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
  for (int s = 0; s < splits; ++s) M = fmaxf(M, part_ml[2 * (s * stride + in_split)]);
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
  const int splits = tree_splits(pairs, rb, p.num_sms);
  const TreeWs w = tree_ws_fp32(p.B, p.N, p.Hq, p.Hkv, p.m, p.m_out, p.num_sms);
  float* sq = reinterpret_cast<float*>(p.ws + w.sq);
  float* part_o = reinterpret_cast<float*>(p.ws + w.part_o);
  float* part_ml = reinterpret_cast<float*>(p.ws + w.part_ml);
  tree_project_kernel<<<dim3(rb, pairs), kTreeThreads, 0, s>>>(p, sq);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  tree_chunk_kernel<<<dim3(splits, rb, pairs), kTreeThreads, 0, s>>>(p, sq, part_o, part_ml);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.N * p.Hq;
  tree_merge_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(p, part_o, part_ml, splits, rb);
  return cudaGetLastError();
}

}  // namespace

// One size for both dtypes: a workspace serves any call of its shape.
size_t tree_ws_bytes(int B, int N, int Hq, int Hkv, int m, int m_out, int vbits, int num_sms) {
  const size_t a = tree_ws_fp32(B, N, Hq, Hkv, m, m_out, num_sms).total;
  const size_t b = tree_tc_ws_bytes(B, N, Hq, Hkv, m, m_out, vbits, num_sms);
  return a > b ? a : b;
}

cudaError_t launch_tree_attention(const TreeParams& p, qjl_dtype dt, cudaStream_t s) {
  return dt == QJL_BF16 ? launch_tree_attention_tc(p, s) : launch_tree_fp32(p, s);
}

}  // namespace qjl
