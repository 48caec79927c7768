// Dense keys and values of cached tokens.
//
// K_hat = sqrt(pi/2)/m |k_in| S^T sign_in on the inlier channels and the same of
// the outlier sketch on the outlier ones; V_hat = zero + code * scale.
#include "qjl_internal.cuh"

namespace qjl {
namespace {

template <typename T>
__device__ __forceinline__ T to_out(float x);
template <>
__device__ __forceinline__ float to_out<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int kReadTokens = 32;  // tokens of a block

// One block per 32 tokens of a (sequence, kv head); thread c owns channel c.
template <typename T>
__global__ void __launch_bounds__(kHeadDim) cache_read_kernel(ReadParams p) {
  __shared__ uint32_t words[kReadTokens][(kMaxM + kMaxMOut) / 32];
  const int c = threadIdx.x;
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / p.Hkv), h = static_cast<int>(bh % p.Hkv);
  const int start = p.t_start ? p.t_start[b] : 0;
  const int lim = p.seqlens ? min(p.seqlens[b], p.cap) : p.cap;
  const int t0 = blockIdx.x * kReadTokens;
  const int wpt = p.m / 32, wpo = p.m_out / 32;
  auto slot = [&](int t, int* j) -> const unsigned char* {
    const int64_t pos = static_cast<int64_t>(start) + t;
    if (t >= p.T || pos < 0 || pos >= lim) return nullptr;
    return tile_of(const_cast<unsigned char*>(p.tiles), p.tl, bh, p.cap, static_cast<int>(pos), j);
  };
  for (int e = c; e < kReadTokens * (wpt + wpo); e += kHeadDim) {
    const int i = e / (wpt + wpo), w = e % (wpt + wpo);
    int j;
    const unsigned char* tile = slot(t0 + i, &j);
    words[i][w] = !tile ? 0u
                  : w < wpt ? reinterpret_cast<const uint32_t*>(tile + p.tl.kbits)[j * wpt + w]
                            : reinterpret_cast<const uint32_t*>(tile + p.tl.kbits_out)[j * wpo + w - wpt];
  }
  __syncthreads();
  bool outlier = false;
  for (int o = 0; o < p.n_out; ++o) outlier |= p.idx[bh * p.n_out + o] == c;
  const int w0 = outlier ? wpt : 0, nw = outlier ? wpo : wpt;
  const __nv_bfloat16* S = outlier ? p.S_out : p.S;
  float acc[kReadTokens];
#pragma unroll
  for (int i = 0; i < kReadTokens; ++i) acc[i] = 0.0f;
  if (p.K)
    for (int w = 0; w < nw; ++w)
      for (int k = 0; k < 32; ++k) {
        const uint32_t s = __float_as_uint(__bfloat162float(S[(32 * w + k) * kHeadDim + c])) ^ 0x80000000u;
#pragma unroll
        for (int i = 0; i < kReadTokens; ++i)
          acc[i] += __uint_as_float(s ^ ((words[i][w0 + w] >> k) << 31));
      }
  const float f = kSqrtHalfPi / static_cast<float>(32 * nw);
#pragma unroll
  for (int i = 0; i < kReadTokens; ++i) {
    int j;
    const unsigned char* tile = slot(t0 + i, &j);
    if (!tile) continue;
    const int64_t t = t0 + i;
    if (p.K) {
      const float norm = __half2float(reinterpret_cast<const __half*>(tile + p.tl.knorm)[2 * j + (outlier ? 1 : 0)]);
      static_cast<T*>(p.K)[b * p.k_sb + h * p.k_sh + t * p.k_st + c] = to_out<T>(acc[i] * (f * norm));
    }
    if (p.V) {
      const int g = c / kValueGroup;
      const float2 sz = __half22float2(reinterpret_cast<const __half2*>(tile + p.tl.vsz)[j * (kHeadDim / kValueGroup) + g]);
      int code;
      if (p.tl.vbits == 2)
        code = (tile[p.tl.vcode + v2_line(g, (c % 32) / 4) + j] >> (2 * (c % 4))) & 3;
      else
        code = (tile[p.tl.vcode + j * (kHeadDim / 2) + 16 * vcode_chunk(j, g) + (c % 32) / 2] >> (4 * (c % 2))) & 15;
      static_cast<T*>(p.V)[b * p.v_sb + h * p.v_sh + t * p.v_st + c] = to_out<T>(fmaf(static_cast<float>(code), sz.x, sz.y));
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const ReadParams& p, qjl_dtype dt, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.T + kReadTokens - 1) / kReadTokens), static_cast<unsigned>(p.B * p.Hkv));
  if (dt == QJL_BF16)
    cache_read_kernel<__nv_bfloat16><<<grid, kHeadDim, 0, s>>>(p);
  else
    cache_read_kernel<float><<<grid, kHeadDim, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qjl
