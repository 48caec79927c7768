// Rotary positions of a step's queries and keys.
//
// Plane i of a head turns by a = P f_i: (u, v) -> (u cos a - v sin a,
// v cos a + u sin a). The angle is reduced in fp64, P f_i / (2 pi) minus its
// nearest integer: the table's entry and the product round by 2^-53 each, which
// leaves the angle within 2^-51 |P f_i| radians (the entry's own quotient and
// power included), below fp32's resolution of a radian up to |P| = 2^27 and 1e-6
// at 2^31, where an fp32 product would be off by whole radians near a million; sin
// and cos are then taken in fp32 of the reduced turn.
//
// Bound: HBM, every element is read and written once. A block takes TT tokens
// and all their heads: its threads compute the tokens' sines once into shared
// memory (the fp64 work is paid per token, not per head), then a thread keeps
// those of its two 16-byte chunks of a head row, which hold whole planes (chunks
// u and u + rot/(2 e) in the half layout, u and u + d/(2 e) in the interleaved
// one, e elements per chunk), and walks over the heads; eight (bf16) lanes cover
// 128 consecutive bytes with every load and store. Measured, 32768 tokens of 64
// heads, bf16, two sets of buffers in turn: 190 us, 5.7 TB/s (half layout, 128
// dims); 168 us, 6.4 TB/s (interleaved, 64 dims).
#include "qjl_internal.cuh"

namespace qjl {
namespace {

constexpr int kRopeThreads = 256;
// Blocks that an SM holds, which sets the registers of a thread: as many as leave
// at most 24 bytes of spills. bf16 in the half layout keeps the sines of 8 planes
// and two chunks of 8 values. Measured with 6, 5, 4 and 3 blocks, 32768 tokens of
// 64 heads: bf16 half 248, 207, 190, 210 us (half the dims 289, 208, 187, 206);
// bf16 interleaved, 64 dims 184, 168, 177 us; fp32 half, 16384 tokens 174, 168, 171.
template <typename T, int LAYOUT>
constexpr int kRopeBlocks = sizeof(T) == 2 && LAYOUT == QJL_ROPE_HALF ? 4 : 5;

template <typename T>
struct Chunk;  // 16 bytes as fp32 values
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void load(const void* base, int64_t i, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(u[k] << 16);
      v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  }
  __device__ static void store(void* base, int64_t i, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Chunk<float> {
  static constexpr int n = 4;
  __device__ static void load(const void* base, int64_t i, float (&v)[4]) {
    const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
  __device__ static void store(void* base, int64_t i, const float (&v)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

template <typename T, int LAYOUT, int TT>
__global__ void __launch_bounds__(kRopeThreads, (kRopeBlocks<T, LAYOUT>)) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int E = Chunk<T>::n;              // elements of a chunk
  constexpr int kPairs = kHeadDim / (2 * E);  // chunk pairs of a row
  __shared__ float2 turn[TT][kHeadDim / 2];   // (cos, sin) of plane i of token k, the amplitude in both
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T, tok0 = static_cast<int64_t>(blockIdx.x) * TT;
  const int rot = p.table.rot_dim, half = rot / 2;
  for (int e = threadIdx.x; e < TT * half; e += kRopeThreads) {
    const int k = e / half, i = e - k * half;
    const int64_t bt = tok0 + k;
    if (bt >= tokens) break;
    const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * p.T);
    const int64_t pos = p.positions ? p.positions[bt] : static_cast<int64_t>(p.t_start ? p.t_start[b] : 0) + t;
    const double x = static_cast<double>(pos) * p.table.turns[i];
    float sn, cs;
    sincospif(static_cast<float>(2.0 * (x - rint(x))), &sn, &cs);  // half turns in [-1, 1]
    turn[k][i] = make_float2(cs * p.table.amplitude, sn * (p.inverse ? -p.table.amplitude : p.table.amplitude));
  }
  __syncthreads();
  const int u = threadIdx.x % kPairs, k = threadIdx.x / kPairs % TT;
  const int64_t bt = tok0 + k;
  if (bt >= tokens) return;
  const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * p.T);
  // the thread's two chunks, and the first plane of each
  int c0, c1, plane0, plane1;
  if (LAYOUT == QJL_ROPE_HALF) {
    const int n = rot / (2 * E);  // rotated chunk pairs
    c0 = u < n ? u : 2 * n + (u - n);
    c1 = u < n ? u + n : c0 + (kPairs - n);
    plane0 = u < n ? u * E : -1;
    plane1 = plane0;
  } else {
    c0 = u;
    c1 = u + kPairs;
    plane0 = c0 * E < rot ? c0 * (E / 2) : -1;
    plane1 = c1 * E < rot ? c1 * (E / 2) : -1;
  }
  // half: cs/sn[k] of plane0 + k; interleaved: [0, E/2) of plane0 + k, [E/2, E) of plane1 + k
  float cs[E], sn[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int pl = LAYOUT == QJL_ROPE_HALF || i < E / 2 ? plane0 : plane1;
    const float2 v = pl >= 0 ? turn[k][pl + (LAYOUT == QJL_ROPE_HALF || i < E / 2 ? i : i - E / 2)] : make_float2(1.0f, 0.0f);
    cs[i] = v.x;
    sn[i] = v.y;
  }
  const int H = p.heads[0].H + (p.n_heads > 1 ? p.heads[1].H : 0);
  constexpr int kStep = kRopeThreads / (kPairs * TT);  // heads that the block takes at once
#pragma unroll 4
  for (int hh = threadIdx.x / (kPairs * TT); hh < H; hh += kStep) {
    const bool second = hh >= p.heads[0].H;
    const qjl_rope_heads& w = second ? p.heads[1] : p.heads[0];
    const int h = second ? hh - p.heads[0].H : hh;
    const int64_t xi = b * w.x_sb + h * w.x_sh + t * w.x_st;
    const int64_t yi = b * w.y_sb + h * w.y_sh + t * w.y_st;
    float a[E], c[E];
    Chunk<T>::load(w.x, xi + c0 * E, a);
    Chunk<T>::load(w.x, xi + c1 * E, c);
    if (LAYOUT == QJL_ROPE_HALF) {
      if (plane0 >= 0)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float x = a[k], y = c[k];
          a[k] = x * cs[k] - y * sn[k];
          c[k] = y * cs[k] + x * sn[k];
        }
    } else {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        if (plane0 >= 0) {
          const float x = a[2 * k], y = a[2 * k + 1];
          a[2 * k] = x * cs[k] - y * sn[k];
          a[2 * k + 1] = y * cs[k] + x * sn[k];
        }
        if (plane1 >= 0) {
          const float x = c[2 * k], y = c[2 * k + 1];
          c[2 * k] = x * cs[k + E / 2] - y * sn[k + E / 2];
          c[2 * k + 1] = y * cs[k + E / 2] + x * sn[k + E / 2];
        }
      }
    }
    Chunk<T>::store(w.y, yi + c0 * E, a);
    Chunk<T>::store(w.y, yi + c1 * E, c);
  }
}

template <typename T, int LAYOUT, int TT>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.B) * p.T + TT - 1) / TT;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  rope_kernel<T, LAYOUT, TT><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// A block per token while the device holds all of them at once, for the SMs'
// sake; past that four tokens a block, which fill it with whole planes of sines.
// Measured with 1 and 4 tokens a block (us), half layout, 40 heads: 592 tokens 5.5
// and 7.2, 740 7.9 and 8.4, 1184 9.6 and 9.5, 2368 16.2 and 13.1; 10 heads: 444
// 3.4 and 3.3, 1184 5.8 and 4.2.
template <typename T, int LAYOUT>
cudaError_t launch_l(const RopeParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return static_cast<int64_t>(p.B) * p.T <= static_cast<int64_t>(kRopeBlocks<T, LAYOUT>) * sms ? launch<T, LAYOUT, 1>(p, s)
                                                                                            : launch<T, LAYOUT, 4>(p, s);
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t s) {
  return p.table.layout == QJL_ROPE_HALF ? launch_l<T, QJL_ROPE_HALF>(p, s) : launch_l<T, QJL_ROPE_INTERLEAVED>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, qjl_dtype dt, cudaStream_t s) {
  return dt == QJL_BF16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace qjl
