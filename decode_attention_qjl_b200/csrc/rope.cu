// Rotary positions of a step's queries and keys.
//
// Plane i of a head turns by a = P f_i: (u, v) -> (u cos a - v sin a,
// v cos a + u sin a). The angle is reduced in fp64: P f_i / (2 pi) minus its
// nearest integer is exact to 2^-22 of a turn's fp32 resolution for every
// int32 position, where an fp32 product would be off by whole radians near a
// million; sin and cos are then taken in fp32 of the reduced turn.
//
// Bound: HBM, every element is read and written once. A thread owns two
// 16-byte chunks of a head row that hold whole planes (chunks u and u +
// rot/(2 e) in the half layout, u and u + d/(2 e) in the interleaved one, e
// elements per chunk), computes their sines once and walks over heads, so the
// fp64 work is paid once per token and not per head, and eight (bf16) lanes
// cover 128 consecutive bytes with every load and store.
#include "qjl_internal.cuh"

namespace qjl {
namespace {

constexpr int kRopeThreads = 256;

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

// Thread layout: consecutive threads take the pairs of one token's row, then
// tokens; blockIdx.y takes a range of the call's heads.
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int per) {
  constexpr int E = Chunk<T>::n;            // elements of a chunk
  constexpr int kPairs = kHeadDim / (2 * E);  // chunk pairs of a row
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int u = static_cast<int>(gid % kPairs);
  const int64_t bt = gid / kPairs;
  if (bt >= static_cast<int64_t>(p.B) * p.T) return;
  const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt % p.T);
  const int rot = p.table.rot_dim;
  const int pos = p.positions ? p.positions[bt] : (p.t_start ? p.t_start[b] : 0) + t;
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
  for (int k = 0; k < E; ++k) {
    const int i = LAYOUT == QJL_ROPE_HALF ? plane0 + k : k < E / 2 ? plane0 + k : plane1 + k - E / 2;
    const bool turn = LAYOUT == QJL_ROPE_HALF || k < E / 2 ? plane0 >= 0 : plane1 >= 0;
    cs[k] = 1.0f;
    sn[k] = 0.0f;
    if (turn) {
      const double x = static_cast<double>(pos) * p.table.turns[i];
      const float r = static_cast<float>(2.0 * (x - rint(x)));  // half turns in [-1, 1]
      sincospif(r, &sn[k], &cs[k]);
      cs[k] *= p.table.amplitude;
      sn[k] *= p.inverse ? -p.table.amplitude : p.table.amplitude;
    }
  }
  const int H = p.heads[0].H + (p.n_heads > 1 ? p.heads[1].H : 0);
  const int h0 = blockIdx.y * per, h1 = min(H, h0 + per);
#pragma unroll 4
  for (int hh = h0; hh < h1; ++hh) {
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

template <typename T>
cudaError_t launch(const RopeParams& p, dim3 grid, int per, cudaStream_t s) {
  if (p.table.layout == QJL_ROPE_HALF)
    rope_kernel<T, QJL_ROPE_HALF><<<grid, kRopeThreads, 0, s>>>(p, per);
  else
    rope_kernel<T, QJL_ROPE_INTERLEAVED><<<grid, kRopeThreads, 0, s>>>(p, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, qjl_dtype dt, cudaStream_t s) {
  const int H = p.heads[0].H + (p.n_heads > 1 ? p.heads[1].H : 0);
  const int pairs = kHeadDim / (2 * (dt == QJL_BF16 ? 8 : 4));
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  const int64_t blocks = (tokens * pairs + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // heads per thread: as many as still leave two thousand threads per SM
  constexpr int64_t kThreadsWanted = 148 * 2048;
  const int64_t most = tokens * pairs * H / kThreadsWanted;
  int per = static_cast<int>(most < 1 ? 1 : most < H ? most : H);
  const int groups = (H + per - 1) / per;
  per = (H + groups - 1) / groups;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((H + per - 1) / per));
  return dt == QJL_BF16 ? launch<__nv_bfloat16>(p, grid, per, s) : launch<float>(p, grid, per, s);
}

}  // namespace qjl
