// A chunk of new tokens enters the paged cache: the page plan (block tables, slot maps, the page
// stack) and the rotary append (q and k rotated, K and V into their pages, page metadata).
#include "common.cuh"
#include "internal.h"
#include "meta_core.cuh"

namespace dsa {
namespace {

// ---------------------------------------------------------------------------------------- plan
// Three prefix sums over the requests decide everything: start (new tokens), gone (pages given
// back) and need (pages taken).  Every CTA makes them for itself from the 8 bytes per request (B is
// small against what follows, and no CTA then waits for another): a thread sums a run of neighbouring
// requests, two block scans join the runs (need depends on start).  Kept in shared memory, they place
// the CTA's share of the tokens, of the taken pages and of the returned pages by binary search.
// Lengths and stack height may be updated in place, so they are written by the CTA that takes the last
// ticket, when every other CTA has read them.
// What bounds it is latency: a launch, one round of reads for the lengths, one for the table or the
// stack, one atomic.  Measured on a GB300, launches replayed in a graph: one token for each of 8 requests
// 3.7 us, 256 requests with 10183 tokens 6.8 us, 2048 requests with 88325 tokens 11.1 us.
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCtas = 152;
static_assert(2 * kPlanThreads * kPlanCtas <= 0x7fffffff - kPlanMaxAxis, "indexes count in 32 bits");

DSA_DEV int clamp_i32(long long v) {
  return static_cast<int>(v < 0x7fffffffLL ? v : 0x7fffffffLL);
}

// First index i with end[i] > v (end non-decreasing); n when there is none.
DSA_DEV int first_above(const int* end, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > v)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Exclusive prefix over the block of one value per thread; `part` holds kPlanWarps words.
template <typename T>
DSA_DEV T block_prefix(T v, T* part, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  T base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) base += part[w];
    sum += part[w];
  }
  *total = sum;
  return base + inc - v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_chunk_kernel(const PlanArgs a) {
  launch_dependents();
  extern __shared__ int sm[];
  int* s_end = sm;              // [B]: one past each request's last token
  int* s_gone = sm + a.B;       // [B]: pages given back by requests 0..b
  int* s_need = sm + 2 * a.B;   // [B]: pages needed by requests 0..b
  int* s_count = sm + 3 * a.B;  // [B]: new tokens that take part
  int* s_len = sm + 4 * a.B;    // [B]: length before
  int* s_keep = sm + 5 * a.B;   // [B]: length kept (below s_len where tokens are dropped)
  __shared__ long long s_part_ll[kPlanWarps];
  __shared__ int s_part[2][kPlanWarps];
  __shared__ int s_taken, s_last;
  const int tid = threadIdx.x;
  if (tid == 0) s_taken = 0;
  const int most = a.p * a.max_pages;
  auto pages = [&](int len) { return (len + a.p - 1) / a.p; };
  grid_dependency_wait();

  const int each = (a.B + kPlanThreads - 1) / kPlanThreads;  // neighbouring requests of a thread
  const int b0 = min(tid * each, a.B), b1 = min(b0 + each, a.B);
  const int held = min(max(a.free_in[0], 0), a.free_capacity);  // pages on the stack
  long long start = 0;
  int gone = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = min(max(a.lens_in[b], 0), most), delta = a.delta[b];
    const int keep =
        delta < 0 ? static_cast<int>(max(static_cast<long long>(len) + delta, 0LL)) : len;
    s_len[b] = len;
    s_keep[b] = keep;
    s_count[b] = max(delta, 0);
    start += max(delta, 0);
    gone += pages(len) - pages(keep);
  }
  long long start_total;
  int gone_total, need_total;
  start = block_prefix(start, s_part_ll, &start_total);
  gone = block_prefix(gone, s_part[0], &gone_total);
  int need = 0;
  for (int b = b0; b < b1; ++b) {
    const int want = s_count[b], len = s_len[b];
    start += want;
    gone += pages(len) - pages(s_keep[b]);
    // a request takes part when its tokens lie inside the chunk and its table row can hold them
    const bool fits = start <= a.tokens && static_cast<long long>(len) + want <= most;
    if (want > 0 && fits) need += pages(len + want) - pages(len);
    if (want > 0 && !fits) s_count[b] = -1;
    s_end[b] = clamp_i32(start);
    s_gone[b] = gone;
    s_need[b] = need;
  }
  need = block_prefix(need, s_part[1], &need_total);
  // Admission: a request that needs pages gets them when those of all requests up to it fit; one
  // that needs none is always admitted.  s_need never falls, so the pages taken are its last value
  // that fits.
  const int top = clamp_i32(static_cast<long long>(held) + gone_total);
  bool refused = false;
  int before = need, taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int end = s_need[b] + need;
    s_need[b] = end;
    if (end <= top) taken = end;
    const int want = s_count[b];
    if (want < 0 || (end > before && end > top)) {
      s_count[b] = 0;
      refused |= want != 0;
    }
    before = end;
  }
  if (taken > 0) atomicMax(&s_taken, taken);
  if (__syncthreads_or(refused) && tid == 0 && blockIdx.x == 0)
    raise_status(a.status, DSA_STATUS_NO_PAGES);
  taken = s_taken;
  int left = top - taken;
  if (left > a.free_capacity) {
    left = a.free_capacity;
    if (tid == 0 && blockIdx.x == 0) raise_status(a.status, DSA_STATUS_OVERFLOW);
  }

  // i-th page given back in this call, in request then position order
  auto returned = [&](int i) {
    const int b = first_above(s_gone, a.B, i);
    const int j = pages(s_keep[b]) + i - (b > 0 ? s_gone[b - 1] : 0);
    return a.page_table[static_cast<size_t>(b) * a.max_pages + j];
  };
  // k-th page taken in this call: from the top of the stack, returned pages included
  auto page_taken = [&](int k) {
    const int s = top - 1 - k;
    return s < held ? a.free_pages[s] : returned(s - held);
  };

  const int first = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
  for (int t = first; t < a.tokens; t += step) {
    const int b = first_above(s_end, a.B, t);
    int row = -1, pos = -1, slot = -1;
    if (b < a.B && s_count[b] > 0) {
      const int len = s_len[b], have = pages(len);
      row = b;
      pos = len + t - (b > 0 ? s_end[b - 1] : 0);
      if (a.slot) {
        const int j = pos / a.p;
        const int phys = j < have ? a.page_table[static_cast<size_t>(b) * a.max_pages + j]
                                  : page_taken((b > 0 ? s_need[b - 1] : 0) + j - have);
        if (phys >= 0 && phys < a.num_phys)
          slot = phys * a.p + pos - j * a.p;
        else
          raise_status(a.status, DSA_STATUS_BAD_PAGE);
      }
    }
    a.row[t] = row;
    a.pos[t] = pos;
    if (a.slot) a.slot[t] = slot;
  }
  for (int k = first; k < taken; k += step) {
    const int b = first_above(s_need, a.B, k);
    a.page_table[static_cast<size_t>(b) * a.max_pages + pages(s_len[b]) + k - (b > 0 ? s_need[b - 1] : 0)] =
        page_taken(k);
  }
  for (int s = held + first; s < left; s += step) a.free_pages[s] = returned(s - held);
  for (int b = first; b < a.B; b += step) {
    a.start[b + 1] = s_end[b];
    a.count[b] = s_count[b];
  }
  if (first == 0) a.start[0] = 0;

  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      s_last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) *a.ticket = 0;
  }
  for (int b = tid; b < a.B; b += kPlanThreads) a.lens_out[b] = s_keep[b] + s_count[b];
  if (tid == 0) a.free_out[0] = left;
}

// -------------------------------------------------------------------------------------- append
// Two kinds of CTA in one launch.  Query CTAs turn the queries, a warp a token (or some of its heads):
// nothing there depends on a page.  Key CTAs turn and write keys and values and renew the metadata.
// Their work is cut at logical-page boundaries so that one CTA writes every new key of the records it
// makes: a "run" is the new tokens of one request inside one unit of `unit` positions (a multiple of
// the logical page, at least 16 tokens where the page allows it), and CTA (x, y) takes the runs whose
// first token lies in [16 x, 16 x + 16) of the chunk, for its group of KV heads.  In both a warp's 32
// lanes hold 4 of the 128 dims each, with their cosines and sines in registers for all its rows of 256
// bytes, and the first rows are on their way while the sines are worked out.
// What bounds it is DRAM behind a chain (row, position, page, sines, rows, metadata) some 4 us long that
// the CTAs of an SM overlap.  Measured on a GB300, launches replayed in a graph: one token for each of 4
// requests, 32 + 8 heads, 4.3 us; 8398 tokens of 32 + 8 heads, three axes, min/max metadata, 39.5 us, 5.3
// TB/s, 0.79 of a measured copy; 3967 tokens of 32 + 32 heads, mean metadata, 40.5 us, 4.9 TB/s, 0.74.
constexpr int kAppThreads = 256;
constexpr int kAppTokens = 16;
constexpr int kAppRows = 4;
// Heads share a CTA (keys) or a warp (queries) and with it the sines, but a short chunk needs the CTAs:
// below kAppCtas of them heads are split (4 decode tokens 4.3 us, 7.5 with all heads together), and
// below kAppWarps query warps query heads (one token of 64 heads: 3.8 and 6.4 us).  Four CTAs run on an
// SM, at 64 registers with three words spilled; three, with none, take 43.9 and 41.6 us for the two long
// cases above.
constexpr int kAppCtas = 3 * 152, kAppWarps = 32 * 152;

// ---- cosine and sine of a fraction of a turn (64-bit fixed point), to the last bit of fp32 but for
// about one value in 10^5: keys that lie next to a rounding border of bf16 then fall on the same side
// as in an evaluation of wider precision, and with them the page metadata.  The nearest quadrant is
// taken off exactly; theta = 2 pi r in [-pi/4, pi/4] is a pair of floats (high, low), and the Taylor
// series of sin and cos are summed with their two largest coefficients and all products by them in
// such pairs (the terms behind weigh below 2^-11, so plain fp32 leaves 2^-35 there).
struct Pair {
  float h, l;
};
DSA_DEV Pair pair_sum(float a, float b) {  // |a| >= |b| or a == 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
DSA_DEV Pair pair_mul(const Pair& a, const Pair& b) {
  const float p = __fmul_rn(a.h, b.h);
  float e = __fmaf_rn(a.h, b.h, -p);
  e = __fmaf_rn(a.h, b.l, e);
  return {p, __fmaf_rn(a.l, b.h, e)};
}
DSA_DEV Pair pair_add(float ch, float cl, const Pair& p) {  // |ch| >= |p|
  const Pair s = pair_sum(ch, p.h);
  return {s.h, __fadd_rn(__fadd_rn(s.l, p.l), cl)};
}

DSA_DEV float2 cos_sin_turn(unsigned long long turn) {
  const unsigned q = static_cast<unsigned>((turn + (1ull << 61)) >> 62);  // nearest quarter
  const long long r = static_cast<long long>(turn - (static_cast<unsigned long long>(q) << 62));
  // r from its 24, 24 and 16 bits, each exact in a float; the second sum matters where the first one
  // cancels (a small negative r has -2^40 there), and its error is below 2^-47 of r
  const float rh = static_cast<float>(static_cast<int>(r >> 40)) * 1099511627776.f;
  const float rm = static_cast<float>(static_cast<unsigned>(r >> 16) & 0xffffffu) * 65536.f;
  Pair t = pair_sum(rh, rm);
  t = pair_sum(t.h, __fadd_rn(t.l, static_cast<float>(static_cast<unsigned>(r) & 0xffffu)));
  // theta = r * 2 pi / 2^64
  constexpr float kTurnH = 3.4061217e-19f, kTurnL = -9.4783964e-27f;
  float th = __fmul_rn(t.h, kTurnH);
  float tl = __fmaf_rn(t.h, kTurnH, -th);
  tl = __fmaf_rn(t.h, kTurnL, tl);
  tl = __fmaf_rn(t.l, kTurnH, tl);
  const Pair a = pair_sum(th, tl);
  const Pair z = pair_mul(a, a);
  // 1 / k!, alternating; the pairs are 1/6, 1/120 and 1/2, 1/24 to 48 bits
  float ps = __fmaf_rn(z.h, 1.6059044e-10f, -2.5052108e-08f);
  ps = __fmaf_rn(z.h, ps, 2.7557319e-06f);
  ps = __fmaf_rn(z.h, ps, -0.0001984127f);
  Pair s = pair_add(0.008333334f, -4.346172e-10f, pair_mul(z, {ps, 0.f}));
  s = pair_add(-0.16666667f, 4.967054e-09f, pair_mul(z, s));
  s = pair_add(a.h, a.l, pair_mul(a, pair_mul(z, s)));
  float pc = __fmaf_rn(z.h, -1.1470746e-11f, 2.0876756e-09f);
  pc = __fmaf_rn(z.h, pc, -2.755732e-07f);
  pc = __fmaf_rn(z.h, pc, 2.4801588e-05f);
  pc = __fmaf_rn(z.h, pc, -0.0013888889f);
  Pair c = pair_add(0.041666668f, -1.2417635e-09f, pair_mul(z, {pc, 0.f}));
  c = pair_add(-0.5f, 0.f, pair_mul(z, c));
  c = pair_add(1.f, 0.f, pair_mul(z, c));
  const float sn = __fadd_rn(s.h, s.l), cs = __fadd_rn(c.h, c.l);
  const float x = q & 1 ? sn : cs, y = q & 1 ? cs : sn;
  return make_float2(q == 1 || q == 2 ? -x : x, q & 2 ? -y : y);
}

// What a lane multiplies its four dims with: out = own * c + partner * s, each product rounded once, as
// the formulas x cos - y sin and y cos + x sin are written.
struct Turn {
  float c[4], s[4];
  int from;     // lane that holds the partner dims (half-split pairs)
  bool on;      // this lane's dims are turned
  bool inside;  // neighbouring pairs: the partner is the lane's own neighbour dim
};

DSA_DEV uint2 turn_row(const uint2& x, const Turn& r) {
  float own[4], other[4];
  own[0] = __uint_as_float(x.x << 16);
  own[1] = __uint_as_float(x.x & 0xffff0000u);
  own[2] = __uint_as_float(x.y << 16);
  own[3] = __uint_as_float(x.y & 0xffff0000u);
  if (r.inside) {
    other[0] = own[1];
    other[1] = own[0];
    other[2] = own[3];
    other[3] = own[2];
  } else {
    const uint32_t a = __shfl_sync(0xffffffffu, x.x, r.from), b = __shfl_sync(0xffffffffu, x.y, r.from);
    other[0] = __uint_as_float(a << 16);
    other[1] = __uint_as_float(a & 0xffff0000u);
    other[2] = __uint_as_float(b << 16);
    other[3] = __uint_as_float(b & 0xffff0000u);
  }
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __fadd_rn(__fmul_rn(own[i], r.c[i]), __fmul_rn(other[i], r.s[i]));
  uint2 y;
  y.x = pack_bf16(o[0], o[1]);
  y.y = pack_bf16(o[2], o[3]);
  return r.on ? y : x;
}

// The pairs lane and lane + 32 of a token, which this lane works out: their phases and axes.
struct Pairs {
  unsigned long long phase[2];
  int axis[2];
};
DSA_DEV Pairs lane_pairs(const AppendArgs& a, int lane) {
  Pairs p = {};
  if (a.phase == nullptr) return p;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int pr = lane + 32 * w;
    if (pr < a.rot_dim / 2) {
      p.phase[w] = a.phase[pr];
      p.axis[w] = a.axis ? min(static_cast<int>(a.axis[pr]), a.num_axes - 1) : 0;
    }
  }
  return p;
}

// Where those pairs of token t stand (pos: its chunk position).
DSA_DEV int2 pair_positions(const AppendArgs& a, const Pairs& p, int t, int pos) {
  if (a.positions == nullptr) return make_int2(pos, pos);
  return make_int2(a.positions[static_cast<size_t>(p.axis[0]) * a.tokens + t],
                   a.positions[static_cast<size_t>(p.axis[1]) * a.tokens + t]);
}

// The lane's Turn: every lane works out its two pairs and the warp shares them.
DSA_DEV Turn make_turn(const AppendArgs& a, const Pairs& p, int2 where, int lane) {
  const int half = a.rot_dim / 2;
  // position x phase modulo one turn, exact in 64-bit integers whatever the position
  const float2 v0 = cos_sin_turn(static_cast<unsigned long long>(static_cast<long long>(where.x)) * p.phase[0]);
  const float2 v1 = cos_sin_turn(static_cast<unsigned long long>(static_cast<long long>(where.y)) * p.phase[1]);
  Turn r;
  r.on = 4 * lane < a.rot_dim;
  r.inside = a.interleaved;
  const bool low = 4 * lane < half;
  r.from = !r.on ? lane : low ? lane + half / 4 : lane - half / 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = !r.on ? 0 : r.inside ? 2 * lane + i / 2 : low ? 4 * lane + i : 4 * lane - half + i;
    const float c0 = __shfl_sync(0xffffffffu, v0.x, pr & 31), c1 = __shfl_sync(0xffffffffu, v1.x, pr & 31);
    const float s0 = __shfl_sync(0xffffffffu, v0.y, pr & 31), s1 = __shfl_sync(0xffffffffu, v1.y, pr & 31);
    const bool minus = r.inside ? i % 2 == 0 : low;
    r.c[i] = pr < 32 ? c0 : c1;
    r.s[i] = pr < 32 ? s0 : s1;
    if (minus) r.s[i] = -r.s[i];
  }
  return r;
}

// N rows of 256 bytes, of which `rows` are there (strides in elements).
template <int N>
DSA_DEV void load_rows(uint2 (&x)[N], const __nv_bfloat16* src, int rows) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < rows) x[i] = *reinterpret_cast<const uint2*>(src + i * kHeadDim);
}
template <int N>
DSA_DEV void store_rows(const uint2 (&x)[N], __nv_bfloat16* dst, int step, int rows, bool turn,
                        const Turn& r) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < rows) *reinterpret_cast<uint2*>(dst + i * step) = turn ? turn_row(x[i], r) : x[i];
}

template <int KIND>
__global__ void __launch_bounds__(kAppThreads, 4) append_chunk_kernel(const AppendArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool turn = a.phase != nullptr;
  const Pairs pairs = lane_pairs(a, lane);

  if (static_cast<int>(blockIdx.x) >= a.key_ctas) {  // queries
    const long long x = static_cast<long long>(blockIdx.x - a.key_ctas) * (kAppThreads / 32) + warp;
    const int t = static_cast<int>(x / a.q_parts), part = static_cast<int>(x - static_cast<long long>(t) * a.q_parts);
    const int hq0 = part * a.q_heads, nq = min(a.q_heads, kv.Hq - hq0);
    if (t >= a.tokens || nq <= 0) return;
    const __nv_bfloat16* src = a.q + static_cast<size_t>(t) * a.q_stride + hq0 * kHeadDim + 4 * lane;
    __nv_bfloat16* dst = a.q_out + (static_cast<size_t>(t) * kv.Hq + hq0) * kHeadDim + 4 * lane;
    uint2 xq[kAppRows];
    load_rows(xq, src, nq);
    const int b = a.row[t], pos = a.pos[t];
    const int2 where = pair_positions(a, pairs, t, pos);
    if (b < 0) return;
    Turn r = {};
    if (turn) r = make_turn(a, pairs, where, lane);
    for (int h = 0; h < nq; h += kAppRows) {
      uint2 next[kAppRows];
      load_rows(next, src + (h + kAppRows) * kHeadDim, nq - h - kAppRows);
      store_rows(xq, dst + h * kHeadDim, kHeadDim, nq - h, turn, r);
#pragma unroll
      for (int i = 0; i < kAppRows; ++i) xq[i] = next[i];
    }
    return;
  }

  const int groups = (kv.Hkv + a.heads_per_cta - 1) / a.heads_per_cta;
  const int h0 = blockIdx.x % groups * a.heads_per_cta;
  const int nh = min(a.heads_per_cta, kv.Hkv - h0);
  const int g = kv.p / a.lp;
  const int t0 = blockIdx.x / groups * kAppTokens, t1 = min(t0 + kAppTokens, a.tokens);

  // The runs that begin here, found by one warp: a token each, their dependent reads side by side.
  // Token and metadata work of all runs are then one list each for the warps.
  struct Run {
    int lead, pos, len, phys;  // first token, its position, the request's length, the page (-1: bad)
    int sub0, subs;            // metadata records to renew: first, how many
    int token_end, meta_end;   // tokens and (head, record) pairs of the runs up to this one
  };
  __shared__ Run s_run[kAppTokens];
  if (warp == 0) {
    const int t = t0 + lane;
    Run r = {t, 0, 0, -1, 0, 0, 0, 0};
    int n = 0;
    if (lane < kAppTokens && t < t1) {
      const int b = a.row[t], pos = a.pos[t];
      if (b >= 0 && b < kv.B && pos >= 0) {
        const int first = a.start[b], n_new = a.count[b];
        if (t >= first && t - first < n_new && (t == first || pos % a.unit == 0)) {
          n = min(min(a.unit - pos % a.unit, first + n_new - t), a.tokens - t);
          r.pos = pos;
          r.len = request_len(kv, b);
          const int j = pos / kv.p;
          if (j < kv.max_pages) r.phys = kv.page_table[static_cast<size_t>(b) * kv.max_pages + j];
          if (r.phys < 0 || r.phys >= kv.num_phys) {
            r.phys = -1;
            raise_status(kv.status, DSA_STATUS_BAD_PAGE);
          } else if (a.meta != nullptr) {
            // records of the run's unit; the request's first run also renews those before it in its
            // page, its last run writes those behind it (no valid token: zeros), as the build does
            const int u0 = (pos - j * kv.p) / a.unit * a.unit;
            const bool last = t + n == first + n_new || (j + 1) * kv.p == pos + n;
            r.sub0 = t == first ? 0 : u0 / a.lp;
            r.subs = (last ? g : (u0 + a.unit) / a.lp) - r.sub0;
          }
        }
      }
    }
    int tokens = n, metas = r.subs * nh;
#pragma unroll
    for (int o = 1; o < kAppTokens; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, tokens, o), y = __shfl_up_sync(0xffffffffu, metas, o);
      if (lane >= o) {
        tokens += x;
        metas += y;
      }
    }
    r.token_end = tokens;
    r.meta_end = metas;
    if (lane < kAppTokens) s_run[lane] = r;
  }
  __syncthreads();

  const int token_total = s_run[kAppTokens - 1].token_end, meta_total = s_run[kAppTokens - 1].meta_end;
  const int my_token_end = s_run[lane & (kAppTokens - 1)].token_end;
  for (int x = warp; x < token_total; x += kAppThreads / 32) {
    const int at = __ffs(__ballot_sync(0xffffffffu, my_token_end > x)) - 1;
    const Run& run = s_run[at];
    const int i = x - (at > 0 ? s_run[at - 1].token_end : 0);  // token of the run
    const int t = run.lead + i, pos = run.pos + i, phys = run.phys;
    const __nv_bfloat16* ksrc = a.k + static_cast<size_t>(t) * a.k_stride + h0 * kHeadDim + 4 * lane;
    const __nv_bfloat16* vsrc = a.v + static_cast<size_t>(t) * a.v_stride + h0 * kHeadDim + 4 * lane;
    if (phys < 0) continue;
    uint2 xk[kAppRows], xv[kAppRows];
    load_rows(xk, ksrc, nh);
    load_rows(xv, vsrc, nh);
    Turn r = {};
    if (turn) r = make_turn(a, pairs, pair_positions(a, pairs, t, pos), lane);
    const size_t at_row =
        ((static_cast<size_t>(phys) * kv.Hkv + h0) * kv.p + pos % kv.p) * kHeadDim + 4 * lane;
    const int page_step = kv.p * kHeadDim;
    for (int h = 0; h < nh; h += kAppRows) {
      const size_t to = at_row + static_cast<size_t>(h) * page_step;
      store_rows(xv, a.v_pages + to, page_step, nh - h, false, r);
      store_rows(xk, a.k_pages + to, page_step, nh - h, turn, r);
      load_rows(xk, ksrc + (h + kAppRows) * kHeadDim, nh - h - kAppRows);
      load_rows(xv, vsrc + (h + kAppRows) * kHeadDim, nh - h - kAppRows);
    }
  }
  if (meta_total == 0) return;
  __threadfence_block();
  __syncthreads();  // the runs' keys are written
  const int my_meta_end = s_run[lane & (kAppTokens - 1)].meta_end;
  for (int x = warp; x < meta_total; x += kAppThreads / 32) {
    const int at = __ffs(__ballot_sync(0xffffffffu, my_meta_end > x)) - 1;
    const Run& run = s_run[at];
    const int i = x - (at > 0 ? s_run[at - 1].meta_end : 0);
    const int h = h0 + i / run.subs, sub = run.sub0 + i % run.subs;
    page_meta<KIND, true>(kv, a.k_pages, a.lp, a.meta, run.pos / kv.p, h, run.phys, run.len, lane, sub,
                          sub + 1);
  }
}

}  // namespace

size_t plan_smem_bytes(int B) { return static_cast<size_t>(B) * 6 * sizeof(int); }

cudaError_t launch_plan_chunk(const PlanArgs& a, cudaStream_t s) {
  const size_t bytes = plan_smem_bytes(a.B);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(plan_chunk_kernel), bytes);
  if (e != cudaSuccess) return e;
  int grid = (a.tokens + kPlanThreads - 1) / kPlanThreads;  // a token a thread, up to a CTA per SM
  grid = grid < 1 ? 1 : grid > kPlanCtas ? kPlanCtas : grid;
  return launch_pdl(plan_chunk_kernel, grid, kPlanThreads, bytes, s, a);
}

cudaError_t launch_append_chunk(const AppendArgs& in, int kind, cudaStream_t s) {
  AppendArgs a = in;
  if (a.tokens <= 0) return cudaSuccess;
  // the smallest multiple of the logical page that divides the page and holds 16 tokens
  a.unit = a.kv.p;
  for (int m = a.lp; m < a.kv.p; m += a.lp)
    if (m >= kAppTokens && a.kv.p % m == 0) {
      a.unit = m;
      break;
    }
  const int gx = (a.tokens + kAppTokens - 1) / kAppTokens;
  // KV heads of one CTA: all of them share the CTA's sines, but a short chunk needs the CTAs
  int hpc = a.kv.Hkv;
  while (hpc > 1 && static_cast<long long>(gx) * ((a.kv.Hkv + hpc - 1) / hpc) < kAppCtas)
    hpc = (hpc + 1) / 2;
  a.heads_per_cta = hpc;
  const long long key_ctas = static_cast<long long>(gx) * ((a.kv.Hkv + hpc - 1) / hpc);
  // query heads of one warp: all of a token's heads share its sines, but few tokens need the warps
  a.q_heads = a.kv.Hq;
  while (a.q_heads > kAppRows &&
         static_cast<long long>(a.tokens) * ((a.kv.Hq + a.q_heads - 1) / a.q_heads) < kAppWarps)
    a.q_heads = (a.q_heads + 1) / 2;
  a.q_parts = (a.kv.Hq + a.q_heads - 1) / a.q_heads;
  const long long q_warps = a.q ? static_cast<long long>(a.tokens) * a.q_parts : 0;
  const long long grid = key_ctas + (q_warps + kAppThreads / 32 - 1) / (kAppThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  a.key_ctas = static_cast<int>(key_ctas);
  const unsigned n = static_cast<unsigned>(grid);
  return kind == DSA_META_MINMAX
             ? launch_pdl(append_chunk_kernel<DSA_META_MINMAX>, n, kAppThreads, 0, s, a)
             : launch_pdl(append_chunk_kernel<DSA_META_MEAN>, n, kAppThreads, 0, s, a);
}

}  // namespace dsa
