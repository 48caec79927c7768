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
//   warps 0-3   sign words (global) -> tensor memory, lane = token
//   warps 4-7   value codes (global) -> V_out, thread = token
//   warps 8-11  sums (tensor memory) -> K_out, lane = token
//   warp 12     issues the products
// Units of 128 token slots are dealt round robin. A thread writes whole 32-byte
// sectors of its token's row, with 32-byte stores where the rows allow it.
#include "tc_common.cuh"

namespace qjl {
namespace {

using namespace tc;

constexpr int kReadUnit = 128;
constexpr int kReadThreads = 32 * 13;
constexpr int kReadWords = 8;                // sign words of a chunk: 128 tensor-memory columns
constexpr int kReadColA = 256;               // D_in at 0, D_out at 128, two sign chunks
constexpr int kReadMisc = 1024;

struct ReadUnit {
  int64_t bh;
  int b, h, slot0;  // first token slot (a multiple of 128)
  int lo, hi;       // slots to give back
  int start;        // position of token 0
  __device__ bool set(const ReadParams& p, int64_t unit, int upb) {
    bh = unit / upb;
    b = static_cast<int>(bh / p.Hkv);
    h = static_cast<int>(bh % p.Hkv);
    start = p.t_start ? p.t_start[b] : 0;
    const int lim = p.seqlens ? min(max(p.seqlens[b], 0), p.cap) : p.cap;
    lo = max(start, 0);
    hi = static_cast<int>(min(static_cast<int64_t>(start) + p.T, static_cast<int64_t>(lim)));
    slot0 = (lo / kReadUnit + static_cast<int>(unit % upb)) * kReadUnit;
    return slot0 < hi;  // (lo >= hi: nothing; slot0 is at most lo)
  }
  __device__ bool live(int tt) const { return slot0 + tt >= lo && slot0 + tt < hi; }
  __device__ const unsigned char* tile(const ReadParams& p, int tt, int* j) const {
    return tile_of(const_cast<unsigned char*>(p.tiles), p.tl, bh, p.cap, slot0 + tt, j);
  }
};

// 16 consecutive values of a row, as 32-byte (wide) or 16-byte stores.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(float* dst, const float (&x)[16], bool wide) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(x[8 * q + k]);
    store32(dst + 8 * q, w, wide);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  store32(dst, w, wide);
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads, 1) cache_read_kernel(const __grid_constant__ ReadParams p, int upb,
                                                                     int64_t n_units) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int wpt = p.m / 32, wpo = p.m_out / 32, words = wpt + wpo, rows = 32 * words;
  uint64_t* a_full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* a_empty = a_full + 2;
  uint64_t* d_full = a_empty + 2;
  uint64_t* d_empty = d_full + 1;
  uint64_t* drain = d_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* err = reinterpret_cast<int*>(tmem_slot + 1);
  unsigned char* img = smem + kReadMisc;
  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      bar_init(&a_full[k], 4);
      bar_init(&a_empty[k], 1);
    }
    bar_init(d_full, 1);
    bar_init(d_empty, 4);
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

  if (warp < 4) {
    // ============================================================ signs
    const int tt = 32 * warp + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * warp) << 16) + kReadColA;
    bool ok = p.K != nullptr;
    int ring = 0;
    uint32_t ph = 1;
    for (int64_t n = blockIdx.x; n < n_units && ok; n += gridDim.x) {
      if (!u.set(p, n, upb)) continue;
      int j = 0;
      const unsigned char* tile = u.live(tt) ? u.tile(p, tt, &j) : nullptr;
      const uint32_t* kb = tile ? reinterpret_cast<const uint32_t*>(tile + p.tl.kbits) + j * wpt : nullptr;
      const uint32_t* ko = tile ? reinterpret_cast<const uint32_t*>(tile + p.tl.kbits_out) + j * wpo - wpt : nullptr;
      for (int w0 = 0; w0 < words && ok; w0 += kReadWords) {
        uint32_t x[kReadWords];  // all loads before the first use
#pragma unroll
        for (int k = 0; k < kReadWords; ++k)
          x[k] = tile && w0 + k < words ? __ldg((w0 + k < wpt ? kb : ko) + w0 + k) : 0u;
        ok = __all_sync(0xffffffffu, bar_wait(&a_empty[ring], ph, limit, err));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int k = 0; k < kReadWords; ++k)
          if (w0 + k < words) {
            uint32_t e[16];
            expand_word(x[k], 0x3F803F80u, e);
            st16(lane_addr + 128 * ring + 16 * k, e);
          }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&a_full[ring]);
        ring ^= 1;
        ph ^= ring == 0 ? 1u : 0u;
      }
    }
  } else if (warp < 8) {
    // ============================================================ values
    const int tt = 32 * (warp - 4) + lane;
    const bool wide = p.V && ((reinterpret_cast<uintptr_t>(p.V) | static_cast<uintptr_t>((p.v_sb | p.v_sh | p.v_st) * sizeof(T))) & 31u) == 0;
    for (int64_t n = blockIdx.x; p.V && n < n_units; n += gridDim.x) {
      if (!u.set(p, n, upb) || !u.live(tt)) continue;
      int j;
      const unsigned char* tile = u.tile(p, tt, &j);
      const uint4 szv = __ldg(reinterpret_cast<const uint4*>(tile + p.tl.vsz + 16 * j));
      const uint32_t sz[4] = {szv.x, szv.y, szv.z, szv.w};
      uint4 cw[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (p.tl.vbits == 4) {
          cw[g] = __ldg(reinterpret_cast<const uint4*>(tile + p.tl.vcode + j * (kHeadDim / 2) + 16 * vcode_chunk(j, g)));
        } else {  // eight bytes of four 2-bit codes
          uint32_t q[2] = {0u, 0u};
#pragma unroll
          for (int r = 0; r < 8; ++r)
            q[r >> 2] |= static_cast<uint32_t>(__ldg(tile + p.tl.vcode + v2_line(g, r) + j)) << (8 * (r & 3));
          cw[g] = make_uint4(q[0], q[1], 0u, 0u);
        }
      }
      T* dst = static_cast<T*>(p.V) + u.b * p.v_sb + u.h * p.v_sh + (u.slot0 + tt - u.start) * p.v_st;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&sz[g]));  // (scale, zero)
        const uint32_t c[4] = {cw[g].x, cw[g].y, cw[g].z, cw[g].w};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int code = p.tl.vbits == 4 ? (c[2 * hf + (k >> 3)] >> (4 * (k & 7))) & 15 : (c[hf] >> (2 * k)) & 3;
            x[k] = fmaf(static_cast<float>(code), f.x, f.y);
          }
          store16(dst + 32 * g + 16 * hf, x, wide);
        }
      }
    }
  } else if (warp < 12) {
    // ============================================================ keys
    const int quarter = warp & 3, tt = 32 * quarter + lane;
    const uint32_t laddr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.K) | static_cast<uintptr_t>((p.k_sb | p.k_sh | p.k_st) * sizeof(T))) & 31u) == 0;
    const float c_in = kSqrtHalfPi / static_cast<float>(p.m), c_out = p.m_out ? kSqrtHalfPi / static_cast<float>(p.m_out) : 0.0f;
    bool ok = true;
    uint32_t ph = 0;
    for (int64_t n = blockIdx.x; p.K && n < n_units; n += gridDim.x) {
      if (!u.set(p, n, upb)) continue;
      const bool live = u.live(tt);
      float f_in = 0.0f, f_out = 0.0f;
      if (live) {
        int j;
        const unsigned char* tile = u.tile(p, tt, &j);
        const float2 norm = __half22float2(*reinterpret_cast<const __half2*>(tile + p.tl.knorm + 4 * j));
        f_in = c_in * norm.x;
        f_out = c_out * norm.y;
      }
      const int oc = lane < p.n_out ? min(max(p.idx[u.bh * p.n_out + lane], 0), kHeadDim - 1) : -1;
      T* dst = static_cast<T*>(p.K) + u.b * p.k_sb + u.h * p.k_sh + static_cast<int64_t>(u.slot0 + tt - u.start) * p.k_st;
      if (ok) ok = bar_wait(d_full, ph, limit, err);
      ph ^= 1u;
      ok = __all_sync(0xffffffffu, ok);
      fence_after();
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {  // 16 channels
        const uint32_t om = __reduce_or_sync(0xffffffffu, oc >= 0 && (oc >> 4) == q ? 1u << (oc & 15) : 0u);
        uint32_t v[16], o[16];
        ld16(v, laddr + 16 * q);
        if (om) ld16(o, laddr + 128 + 16 * q);
        wait_ld();
        float x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(v[k]) * f_in;
        if (om)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if ((om >> k) & 1u) x[k] = __uint_as_float(o[k]) * f_out;
        if (!ok)
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = __int_as_float(0x7fc00000);
        if (live) store16(dst + 16 * q, x, wide);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(d_empty);
    }
  } else if (p.K) {
    // ============================================================ products (the whole warp, converged)
    bool ok = true;
    int ring = 0;
    uint32_t aph = 0, dph = 1;
    const uint32_t id = idesc_f16(kHeadDim, true, 0, 1);
    for (int64_t n = blockIdx.x; n < n_units && ok; n += gridDim.x) {
      if (!u.set(p, n, upb)) continue;
      ok = __all_sync(0xffffffffu, bar_wait(d_empty, dph, limit, err));
      dph ^= 1u;
      uint64_t bd = desc_mn(smem_u32(img), rows * 128);
      for (int w0 = 0; w0 < words && ok; w0 += kReadWords) {
        ok = __all_sync(0xffffffffu, bar_wait(&a_full[ring], aph, limit, err));
        if (!ok) break;
        fence_after();
        uint32_t ad = tmem + kReadColA + 128 * ring;
        const int w1 = min(words, w0 + kReadWords);
#pragma unroll 1
        for (int w = w0; w < w1; ++w, ad += 16, bd += 256)  // 32 rows of 128 bytes: 256 address units
          mma_ts_mn_32(tmem + (w < wpt ? 0 : 128), ad, bd, id, w != 0 && w != wpt);
        commit(&a_empty[ring]);
        ring ^= 1;
        aph ^= ring == 0 ? 1u : 0u;
      }
      if (ok) commit(d_full);
    }
    commit(drain);  // every product ends before the block gives its memory back
    bar_wait(drain, 0, limit > 2000000000ull ? limit : 2000000000ull, nullptr);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (p.K && warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <typename T>
cudaError_t launch(const ReadParams& p, cudaStream_t s) {
  const int upb = static_cast<int>((static_cast<int64_t>(p.T) + 2 * kReadUnit - 2) / kReadUnit);  // of any alignment
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * upb;
  size_t smem = kReadMisc + 1024 + (p.K ? static_cast<size_t>(p.m + p.m_out) * kHeadDim * 2 : 0);
  if (smem < 116 * 1024) smem = 116 * 1024;  // one block per SM: it takes all tensor-memory columns
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(cache_read_kernel<T>), smem);
  if (e != cudaSuccess) return e;
  cache_read_kernel<T><<<static_cast<unsigned>(units < p.num_sms ? units : p.num_sms), kReadThreads, smem, s>>>(p, upb, units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_read(const ReadParams& p, qjl_dtype dt, cudaStream_t s) {
  return dt == QJL_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace qjl
