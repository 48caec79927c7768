// Copy of accepted drafted tokens from the draft cache into the cache.
//
// A token's bytes (124 per kv head at m = 256, m_out = 64, 4-bit codes) lie in
// the five sections of its tile; the copy keeps them bit for bit, but the
// chunks of the 4-bit value codes are swizzled by the slot, so a chunk moves to
// where its new slot keeps it. Bound: latency, a call moves kilobytes to a few
// megabytes: one warp per accepted token and kv head, a word per lane and
// step, every load issued before the first store. Measured: 2.4 us on the device
// for one sequence's four drafts.
#include "qjl_internal.cuh"

namespace qjl {
namespace {

constexpr int kCommitWarps = 8;

__global__ void __launch_bounds__(32 * kCommitWarps) cache_commit_kernel(CommitParams p) {
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31;
  const int j = blockIdx.z * kCommitWarps + (threadIdx.x >> 5);
  const int len = min(max(p.seqlens[b], 0), p.cap);
  const int n = min(max(p.n_accepted[b], 0), p.A);
  if (h == 0 && blockIdx.z == 0 && threadIdx.x == 0 && p.seqlens_out)
    p.seqlens_out[b] = static_cast<int>(min(static_cast<int64_t>(len) + n, static_cast<int64_t>(p.cap)));
  if (j >= n || static_cast<int64_t>(len) + j >= p.cap) return;
  const int src = p.path[static_cast<int64_t>(b) * p.A + j];
  if (src < 0 || src >= p.draft_cap) return;
  const int64_t bh = static_cast<int64_t>(b) * p.Hkv + h;
  int js, jd;
  const unsigned char* from = tile_of(const_cast<unsigned char*>(p.draft), p.tl, bh, p.draft_cap, src, &js);
  unsigned char* to = tile_of(p.tiles, p.tl, bh, p.cap, len + j, &jd);
  // word w of the token (4 bytes): [kbits | kbits_out | norm | scale, zero | codes]
  const int w1 = p.m / 32, w2 = w1 + p.m_out / 32, w3 = w2 + 1, w4 = w3 + kHeadDim / 32;
  const int words = p.tl.vbits == 4 ? w4 + kHeadDim / 8 : w4;
  constexpr int kSteps = (kMaxM / 32 + kMaxMOut / 32 + 1 + 4 + 16 + 31) / 32;
  uint32_t x[kSteps];
  int off[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int w = lane + 32 * i;
    int o = -1, d = -1;
    if (w < w1) {
      o = p.tl.kbits + 4 * (js * w1 + w);
      d = p.tl.kbits + 4 * (jd * w1 + w);
    } else if (w < w2) {
      o = p.tl.kbits_out + 4 * (js * (w2 - w1) + w - w1);
      d = p.tl.kbits_out + 4 * (jd * (w2 - w1) + w - w1);
    } else if (w < w3) {
      o = p.tl.knorm + 4 * js;
      d = p.tl.knorm + 4 * jd;
    } else if (w < w4) {
      o = p.tl.vsz + 4 * (4 * js + w - w3);
      d = p.tl.vsz + 4 * (4 * jd + w - w3);
    } else if (w < words) {
      const int g = (w - w4) >> 2, k = (w - w4) & 3;
      o = p.tl.vcode + js * (kHeadDim / 2) + 16 * vcode_chunk(js, g) + 4 * k;
      d = p.tl.vcode + jd * (kHeadDim / 2) + 16 * vcode_chunk(jd, g) + 4 * k;
    }
    off[i] = d;
    x[i] = o >= 0 ? *reinterpret_cast<const uint32_t*>(from + o) : 0u;
  }
  unsigned char code = 0;
  if (p.tl.vbits == 2) code = from[p.tl.vcode + lane * kV2LineBytes + js];  // line `lane` of 32
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    if (off[i] >= 0) *reinterpret_cast<uint32_t*>(to + off[i]) = x[i];
  if (p.tl.vbits == 2) to[p.tl.vcode + lane * kV2LineBytes + jd] = code;
}

}  // namespace

cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t s) {
  const unsigned z = static_cast<unsigned>(p.A > 0 ? (p.A + kCommitWarps - 1) / kCommitWarps : 1);
  cache_commit_kernel<<<dim3(static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B), z), 32 * kCommitWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qjl
