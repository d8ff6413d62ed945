// Attention of a chunk of new tokens over the paged cache: causal for dense heads, sink + local
// window for streaming heads.
//
// One warp per (token, query head): a lane holds 4 of the 128 dims, every key costs one 256-byte
// read and a five-step warp sum, and the running maximum and sum of the softmax stay in registers.
#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32) chunk_attn_kernel(const ChunkAttnArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / kv.Hq), hq = static_cast<int>(item % kv.Hq);
  if (t >= a.tokens) return;
  int lo = 0, hi = kv.B;  // first request whose tokens end behind t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.start[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= kv.B || t < a.start[lo] || t - a.start[lo] >= a.count[lo]) return;
  const int b = lo, h = hq / kv.G;
  const int L = request_len(kv, b);
  const int pos = L - a.count[b] + (t - a.start[b]);
  const bool win = kv.streaming != nullptr && kv.streaming[h] != 0;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  const size_t at = (static_cast<size_t>(t) * kv.Hq + hq) * kHeadDim + 4 * lane;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = __bfloat162float(a.q[at + e]);
  float m = -INFINITY, l = 0.f;
  const long long w0 = static_cast<long long>(pos) + 1 - a.local;  // first token of the window
  for (int s = 0; s <= pos; ++s) {
    if (win && s >= a.sink && s < w0) {
      s = static_cast<int>(w0) - 1;
      continue;
    }
    const int phys = kv.page_table[static_cast<size_t>(b) * kv.max_pages + s / kv.p];
    if (phys < 0 || phys >= kv.num_phys) {
      if (lane == 0) raise_status(kv.status, DSA_STATUS_BAD_PAGE);
      continue;
    }
    const size_t row = ((static_cast<size_t>(phys) * kv.Hkv + h) * kv.p + s % kv.p) * kHeadDim;
    const uint2 kr = *reinterpret_cast<const uint2*>(a.k_pages + row + 4 * lane);
    const uint2 vr = *reinterpret_cast<const uint2*>(a.v_pages + row + 4 * lane);
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(&kr);
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(&vr);
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) d += q[e] * __bfloat162float(k[e]);
    d = warp_sum(d) * a.scale_log2;
    const float mn = fmaxf(m, d);
    const float keep = m == mn ? 1.f : fast_exp2(m - mn), p = fast_exp2(d - mn);
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * keep + p * __bfloat162float(v[e]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint2 r;
  r.x = pack_bf16(o[0] * inv, o[1] * inv);
  r.y = pack_bf16(o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2*>(a.out + at) = r;
  if (lane == 0) {
    const size_t i = static_cast<size_t>(t) * kv.Hq + hq;
    if (a.m) a.m[i] = m * kLn2;
    if (a.l) a.l[i] = l;
  }
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.tokens) * a.kv.Hq;
  const long long blocks = (items + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(chunk_attn_kernel, static_cast<unsigned>(blocks), kWarps * 32, 0, s, a);
}

}  // namespace dsa
