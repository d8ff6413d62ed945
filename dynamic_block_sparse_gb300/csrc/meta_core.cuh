// Per-page key metadata of one page by one warp, shared by the metadata build (meta_score.cu) and
// the appends (meta_score.cu, chunk.cu).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace dsa {

// 16 bytes of a K row: through the read-only path, or through L2 when the row was written by the
// same kernel (the read-only path is not coherent with such writes).
template <bool COHERENT>
DSA_DEV uint4 ld16(const __nv_bfloat16* p) {
  return COHERENT ? __ldcg(reinterpret_cast<const uint4*>(p))
                  : __ldg(reinterpret_cast<const uint4*>(p));
}

// Metadata of the logical sub-pages [sub0, sub1) of page position j of a request of length L, KV head
// h, on physical page phys, computed by one warp.  Lane l reads 16-byte chunk (l & 15) of token rows of
// parity (l >> 4); the two half-warps are combined at the end of every logical page.  The build
// and the appends share it, so all write the same bits.
template <int KIND, bool COHERENT>
DSA_DEV void page_meta(const KvView& kv, const __nv_bfloat16* __restrict__ k_pages, int lp,
                       void* __restrict__ meta, int j, int h, int phys, int L, int lane, int sub0,
                       int sub1) {
  const int page = kv.p;
  const int valid = min(page, L - j * page);
  const int g = page / lp;
  const int half = lane >> 4, c = lane & 15;
  const __nv_bfloat16* base =
      k_pages + (static_cast<size_t>(phys) * kv.Hkv + h) * page * kHeadDim + c * 8;

  for (int sub = sub0; sub < sub1; ++sub) {
    const int t_lo = sub * lp, t_hi = min((sub + 1) * lp, valid);
    float a[8], bmin[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = (KIND == DSA_META_MINMAX) ? -INFINITY : 0.f;
      bmin[e] = INFINITY;
    }
    int t = t_lo + half;
#pragma unroll 1
    for (; t + 6 < t_hi; t += 8) {
      uint4 raw[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        raw[u] = ld16<COHERENT>(base + static_cast<size_t>(t + 2 * u) * kHeadDim);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(&raw[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __bfloat162float(v[e]);
          if (KIND == DSA_META_MINMAX) {
            a[e] = fmaxf(a[e], x);
            bmin[e] = fminf(bmin[e], x);
          } else {
            a[e] += x;
          }
        }
      }
    }
    for (; t < t_hi; t += 2) {
      const uint4 raw = ld16<COHERENT>(base + static_cast<size_t>(t) * kHeadDim);
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(&raw);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = __bfloat162float(v[e]);
        if (KIND == DSA_META_MINMAX) {
          a[e] = fmaxf(a[e], x);
          bmin[e] = fminf(bmin[e], x);
        } else {
          a[e] += x;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float oa = __shfl_xor_sync(0xffffffffu, a[e], 16);
      const float ob = __shfl_xor_sync(0xffffffffu, bmin[e], 16);
      if (KIND == DSA_META_MINMAX) {
        a[e] = fmaxf(a[e], oa);
        bmin[e] = fminf(bmin[e], ob);
      } else {
        a[e] += oa;
      }
    }
    const bool empty = t_hi <= t_lo;
    const size_t rec = (static_cast<size_t>(phys) * kv.Hkv + h) * g + sub;
    // lanes < 16 write dims 8c..8c+3, lanes >= 16 dims 8c+4..8c+7
    const int e0 = half * 4;
    if (KIND == DSA_META_MINMAX) {
      uint4 o;
      uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float hi = half ? a[4 + e] : a[e];
        const float lo = half ? bmin[4 + e] : bmin[e];
        __nv_bfloat162 pr = __floats2bfloat162_rn(empty ? 0.f : hi, empty ? 0.f : lo);
        w[e] = *reinterpret_cast<uint32_t*>(&pr);
      }
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(meta) + rec * (2 * kHeadDim) +
                           (c * 8 + e0) * 2;
      *reinterpret_cast<uint4*>(dst) = o;
    } else {
      const float cnt = static_cast<float>(max(t_hi - t_lo, 1));
      float4 o;
      o.x = empty ? 0.f : (half ? a[4] : a[0]) / cnt;
      o.y = empty ? 0.f : (half ? a[5] : a[1]) / cnt;
      o.z = empty ? 0.f : (half ? a[6] : a[2]) / cnt;
      o.w = empty ? 0.f : (half ? a[7] : a[3]) / cnt;
      float* dst = reinterpret_cast<float*>(meta) + rec * kHeadDim + c * 8 + e0;
      *reinterpret_cast<float4*>(dst) = o;
    }
  }
}

}  // namespace dsa
