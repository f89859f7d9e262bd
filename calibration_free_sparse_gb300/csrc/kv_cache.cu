// The paged key/value cache: its handle and argument checks, the page plan of
// a step, and the append of new rows with the summaries of their pages.
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "device_util.cuh"
#include "internal.cuh"
#include "kv.cuh"

namespace mr {
namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = kMaxRequests / kPlanThreads;   // requests per thread of the scan

__device__ __forceinline__ long long warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Largest r with at[r] <= i, at ascending with at[0] = 0 (entries may repeat:
// the last of equals holds i).
__device__ __forceinline__ int find_request(const int* at, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Every CTA scans the lengths itself (two prefix sums over at most 1024
// requests: new tokens and missing pages), then takes its share of the tokens
// and of the fresh table entries: one launch and no hand-off between CTAs.  A
// token whose page is fresh takes its id from free_pages, not from the table
// that another CTA is writing.  Bound by the launch and the scan: 3.1 us for a
// decode step of 16 requests, 4.7 us for 162 thousand tokens of 256 prompts
// (2 MB written).
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(moe_reader_kv_plan_args a, int shift, int num_pages, uint32_t* err) {
  __shared__ int s_start[kMaxRequests], s_page[kMaxRequests];
  __shared__ int s_prev[kMaxRequests], s_have[kMaxRequests];
  __shared__ long long w_tok[kPlanThreads / 32], w_page[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int ps = 1 << shift;
  const long long room = (long long)a.width << shift;     // tokens a table row can hold
  uint32_t bad = 0;

  int prev[kPlanPer], add[kPlanPer], have[kPlanPer], need[kPlanPer];
  long long tok = 0, pages = 0;
#pragma unroll
  for (int j = 0; j < kPlanPer; ++j) {
    const int r = tid * kPlanPer + j;
    prev[j] = add[j] = have[j] = need[j] = 0;
    if (r >= a.requests) continue;
    int p = __ldg(a.prev_lens + r), n = __ldg(a.new_lens + r);
    if (p < 0 || n < 0) bad |= kErrLength;
    p = max(p, 0);
    n = max(n, 0);
    if (p > room) p = (int)room, bad |= kErrLength;
    if ((long long)p + n > room) n = (int)(room - p), bad |= kErrLength;
    prev[j] = p;
    add[j] = n;
    have[j] = (int)(((long long)p + ps - 1) >> shift);
    need[j] = (int)(((long long)p + n + ps - 1) >> shift) - have[j];
    tok += n;
    pages += need[j];
  }
  const long long tok_in = warp_scan(tok), page_in = warp_scan(pages);
  if (lane == 31) {
    w_tok[wid] = tok_in;
    w_page[wid] = page_in;
  }
  __syncthreads();
  long long t0 = tok_in - tok, p0 = page_in - pages, t_all = 0, p_all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < wid) t0 += w_tok[w], p0 += w_page[w];
    t_all += w_tok[w];
    p_all += w_page[w];
  }
  if (t_all > a.max_tokens) bad |= kErrLength;
  if (p_all > a.num_free) bad |= kErrPool;
  const int total = (int)min(t_all, (long long)a.max_tokens);
  const bool first = blockIdx.x == 0;
#pragma unroll
  for (int j = 0; j < kPlanPer; ++j) {
    const int r = tid * kPlanPer + j;
    if (r < a.requests) {
      // sums are held to what an int can index: nothing is looked up beyond
      s_start[r] = (int)min(t0, (long long)a.max_tokens);
      s_page[r] = (int)min(p0, (long long)INT32_MAX);
      s_prev[r] = prev[j];
      s_have[r] = have[j];
      if (first) {
        a.lens[r] = prev[j] + add[j];
        a.starts[r] = s_start[r];
      }
    }
    t0 += add[j];
    p0 += need[j];
  }
  if (first && tid == 0) {
    a.starts[a.requests] = total;
    a.taken[0] = (int)min(p_all, (long long)max(a.num_free, 0));
    if (bad) atomicOr(err, bad);
  }
  __syncthreads();

  const long long stride = (long long)gridDim.x * kPlanThreads;
  const long long at = (long long)blockIdx.x * kPlanThreads + tid;
  for (long long i = at; i < min(p_all, (long long)INT32_MAX); i += stride) {
    const int r = find_request(s_page, a.requests, (int)i);
    const int id = i < a.num_free ? __ldg(a.free_pages + i) : -1;
    a.table[(size_t)r * a.width + s_have[r] + ((int)i - s_page[r])] = id;
  }
  bad = 0;
  for (long long i = at; i < a.max_tokens; i += stride) {
    int slot = -1, pos = -1, r = -1;
    if (i < total) {
      r = find_request(s_start, a.requests, (int)i);
      pos = s_prev[r] + ((int)i - s_start[r]);
      const int lp = pos >> shift, fresh = lp - s_have[r];
      int id = -1;
      if (fresh < 0) {
        id = __ldg(a.table + (size_t)r * a.width + lp);
      } else {
        const long long f = (long long)s_page[r] + fresh;
        if (f < a.num_free) id = __ldg(a.free_pages + f);
      }
      if (id >= 0 && id < num_pages) slot = (id << shift) + (pos & (ps - 1));
      else if (fresh < 0 || id != -1) bad |= kErrPage;
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
    a.token_requests[i] = r;
  }
  if (bad) atomicOr(err, bad);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;
constexpr int kKeyWindow = 64;       // tokens that a CTA's two ballots hold

template <int CT> struct Cell { using type = uint16_t; };
template <> struct Cell<MOE_READER_TYPE_E4M3> { using type = uint8_t; };

// x / scale for values that are then rounded to e4m3: Markstein's correction
// of x * (1 / scale) by one fused step gives the rounded quotient where
// nothing over- or underflows (IBM J. Res. Dev. 34, 1990).  Quotients above
// 1024 saturate as they are; ones so small that the step underflows round to
// zero either way.  Scales outside [2^-100, 2^100] take the plain division.
struct Divider {
  float scale, inv;
  bool plain;
  __device__ __forceinline__ explicit Divider(float s) {
    scale = s;
    inv = __frcp_rn(s);
    plain = !(s >= two_to(-100) && s <= two_to(100));
  }
  __device__ __forceinline__ float operator()(float x) const {
    if (plain) return __fdiv_rn(x, scale);
    const float q = x * inv;
    return fabsf(q) < 1024.f ? fmaf(fmaf(-q, scale, x), inv, q) : q;
  }
};

// Pairs of values of the cache's type.  The largest and smallest keys are
// taken in that type (e4m3 in fp16, which holds all its values); a NaN is
// passed over.
template <int CT> struct Pair { using type = __half2; };
template <> struct Pair<MOE_READER_TYPE_BF16> { using type = __nv_bfloat162; };

template <typename P> __device__ __forceinline__ P as_pair(uint32_t v) {
  return *reinterpret_cast<const P*>(&v);
}
template <typename P> __device__ __forceinline__ uint32_t bits_of(P v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 widen2(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ float2 widen2(__nv_bfloat162 v) { return __bfloat1622float2(v); }

// Loads go out for several rows before the first is used (volatile: between the
// branches that tell rows apart, the compiler would wait for each).
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Eight new values of a row as they come in.
__device__ __forceinline__ uint4 fetch_new(const uint16_t* p, bool wide) {
  if (wide) return load16(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The same as the cache stores them: 16 bytes, or 8 of e4m3 (in words 0 and 1).
template <int CT, int IT>
__device__ __forceinline__ uint4 stored(const uint4& in, const Divider& by) {
  if constexpr (CT == MOE_READER_TYPE_E4M3) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (IT == MOE_READER_TYPE_BF16)
        f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else
        f = __half22float2(as_pair<__half2>(w[i]));
      // the conversion saturates at +-448 and keeps NaN
      r[i] = __nv_cvt_float2_to_fp8x2(make_float2(by(f.x), by(f.y)), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint4(r[0] | r[1] << 16, r[2] | r[3] << 16, 0, 0);
  } else {
    return in;
  }
}
template <int CT> __device__ __forceinline__ void put8(void* p, uint4 v) {
  if constexpr (CT == MOE_READER_TYPE_E4M3) *static_cast<uint2*>(p) = make_uint2(v.x, v.y);
  else *static_cast<uint4*>(p) = v;
}
template <int CT> __device__ __forceinline__ uint4 fetch_old(const void* p) {
  if constexpr (CT == MOE_READER_TYPE_E4M3) {
    uint4 v = make_uint4(0, 0, 0, 0);
    asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
  } else {
    return load16(p);
  }
}
// The four pairs of a row's eight stored values.
template <int CT>
__device__ __forceinline__ void pairs_of(uint4 v, typename Pair<CT>::type (&p)[4]) {
  if constexpr (CT == MOE_READER_TYPE_E4M3) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
          (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      p[i] = __half2(r);
    }
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = as_pair<typename Pair<CT>::type>(w[i]);
  }
}

// A summary's step is 2^step_exponent(the largest magnitude).
__device__ __forceinline__ int step_exponent(float top) {
  top = fminf(fmaxf(top, two_to(-100)), two_to(100));
  const int e = floor_log2_held(top) - 6;
  return top > 127.f * two_to(e) ? e + 1 : e;
}
// Codes of the largest and the smallest key; inv: 1 / step.  A power-of-two
// step: the quotients are exact, but for those that underflow, which still round
// away from zero.
__device__ __forceinline__ int code_up(float v, float inv) {
  const float c = fminf(fmaxf(ceilf(v * inv), -127.f), 127.f);
  return (int)(v > 0.f ? fmaxf(c, 1.f) : c);
}
__device__ __forceinline__ int code_down(float v, float inv) {
  const float c = fminf(fmaxf(floorf(v * inv), -127.f), 127.f);
  return (int)(v < 0.f ? fminf(c, -1.f) : c);
}

// One new value as the cache stores it, and a stored value widened.
template <int CT, int IT>
__device__ __forceinline__ typename Cell<CT>::type stored1(uint16_t in, const Divider& by) {
  if constexpr (CT == MOE_READER_TYPE_E4M3) {
    const float f = IT == MOE_READER_TYPE_BF16 ? __uint_as_float((uint32_t)in << 16)
                                               : __half2float(__ushort_as_half(in));
    return __nv_cvt_float_to_fp8(by(f), __NV_SATFINITE, __NV_E4M3);
  } else {
    return in;
  }
}
template <int CT>
__device__ __forceinline__ float widen1(typename Cell<CT>::type v) {
  if constexpr (CT == MOE_READER_TYPE_E4M3)
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
  else if constexpr (CT == MOE_READER_TYPE_BF16)
    return __uint_as_float((uint32_t)v << 16);
  else
    return __half2float(__ushort_as_half(v));
}

// A window of keys.
struct Window {
  int slots[256 + kKeyWindow + 1];     // of its tokens, a page of them before and one behind
  unsigned long long ends;             // tokens that end a run
  unsigned long long followed, follows;   // those with another run of their page behind, before
  uint16_t back[256];                  // a row's token, counted back from the run's last; 0: none
  float top[kAppendThreads / 32];
};

// The keys of a window near which tokens are skipped: false, and nothing done,
// unless that cuts the new tokens of a page into several runs.  Then each run
// copies its rows, and the last one of a page sums the page up: other CTAs write
// the others' rows meanwhile, so it takes them from the input, too.  A thread per
// coordinate, and a function apart with its state in shared memory: this is
// rare, and registers of its own would cost the kernel occupancy.
template <int D, int CT, int IT>
__device__ __noinline__ bool append_cut_runs(Window& c, const moe_reader_kv_append_args& a,
                                             typename Cell<CT>::type* kc, int8_t* codes,
                                             float* steps, const float* k_scale, int heads, int shift,
                                             int pool, int first) {
  const int lane = threadIdx.x & 31, ps = 1 << shift;
  auto live = [&](int slot) { return (unsigned)slot < (unsigned)pool; };
  auto same_page = [&](int x, int y) { return (x ^ y) < ps; };
  __syncthreads();
  // runs with another of their page behind them, or before them
#pragma unroll 1
  for (int w = threadIdx.x >> 5; w < kKeyWindow; w += kAppendThreads / 32) {
    if (!(c.ends >> w & 1)) continue;
    const int slot = c.slots[ps + w];
#pragma unroll 1
    for (int b = 1; b <= ps; b += 32) {
      const int t = first + w + b + lane;
      const int at = b + lane <= ps && t < a.tokens ? __ldg(a.slots + t) : -1;
      const uint32_t any = __ballot_sync(0xffffffffu, live(at));
      if (!any) continue;
      if (lane == __ffs(any) - 1 && at > slot && same_page(at, slot))
        atomicOr(&c.followed, 1ull << w);
      break;
    }
    bool ended = false;
#pragma unroll 1
    for (int b = 1; b <= ps; b += 32) {
      const int back = min(b + lane, ps), at = c.slots[ps + w - back];
      const uint32_t out = __ballot_sync(0xffffffffu, ended || at != slot - back);
      const bool other = live(at) && !same_page(at, slot);
      if (out && live(at) && !other && at < slot && lane >= __ffs(out) - 1)
        atomicOr(&c.follows, 1ull << w);
      if (__any_sync(0xffffffffu, other)) break;
      ended |= out != 0;
    }
  }
  __syncthreads();
  if (!(c.followed | c.follows)) return false;

  const int head = blockIdx.y;
#pragma unroll 1
  for (int w = 0; w < kKeyWindow; ++w) {
    if (!(c.ends >> w & 1)) continue;
    const int slot = c.slots[ps + w], off = slot & (ps - 1);
    const size_t summary = (size_t)(slot >> shift) * heads + head;
    const bool sums = !(c.followed >> w & 1);
    __syncthreads();
    for (int o = threadIdx.x; o < ps; o += kAppendThreads) c.back[o] = 0;
    __syncthreads();
    for (int back = 1 + threadIdx.x; back <= ps; back += kAppendThreads) {
      const int at = c.slots[ps + w - back];
      if (live(at) && at < slot && same_page(at, slot)) c.back[at & (ps - 1)] = (uint16_t)back;
    }
    __syncthreads();
    constexpr int kPer = (D + kAppendThreads - 1) / kAppendThreads;
    float hi[kPer], lo[kPer], top = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = threadIdx.x + i * kAppendThreads;
      hi[i] = -INFINITY;
      lo[i] = INFINITY;
      bool run = true;                                 // the rows of this run
#pragma unroll 1
      for (int o = off; o >= 0 && d < D; --o) {
        const int back = o == off ? 0 : c.back[o];
        run &= back == off - o;
        if (!run && !sums) break;
        auto* at = kc + ((summary << shift) + o) * D + d;
        typename Cell<CT>::type v;
        if (o == off || back) {
          const Divider by(CT == MOE_READER_TYPE_E4M3 ? k_scale[head] : 1.f);
          v = stored1<CT, IT>(__ldg(static_cast<const uint16_t*>(a.k) + head * a.k_head_stride +
                                    (first + w - back) * a.k_token_stride + d), by);
          if (run) *at = v;
        } else {
          v = *at;
        }
        hi[i] = fmaxf(hi[i], widen1<CT>(v));
        lo[i] = fminf(lo[i], widen1<CT>(v));
      }
      if (hi[i] < lo[i]) hi[i] = lo[i] = 0.f;          // all NaN
      if (d < D) top = fmaxf(top, fmaxf(fabsf(hi[i]), fabsf(lo[i])));
    }
    if (!sums) continue;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) c.top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kAppendThreads / 32; ++v) top = fmaxf(top, c.top[v]);
    const int e = step_exponent(top);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = threadIdx.x + i * kAppendThreads;
      if (d >= D) continue;
      codes[summary * 2 * D + d] = (int8_t)code_up(hi[i], two_to(-e));
      codes[summary * 2 * D + D + d] = (int8_t)code_down(lo[i], two_to(-e));
    }
    if (threadIdx.x == 0) steps[summary] = two_to(e);
  }
  return true;
}

// The first `key_ctas` CTAs of a KV head look at `key_window` (at most 64)
// consecutive tokens each for their keys, the others at `value_window` each for
// their values: a prompt's pages are twice as many independent chains of loads.
// Values are copied row by row.  Keys are taken once per page: for the token
// that is the last new one of its page, with the run of new tokens that ends
// there (their slots are consecutive).  It copies the run's rows and, over the
// page's rows up to that token -- the older ones read from the cache, the new
// ones from the input -- forms the largest and smallest key per coordinate, so
// the summary needs no second pass and no other CTA's writes (append_cut_runs
// sees to pages whose new tokens have skipped ones between them).  D / 8 lanes
// share a row, 8 values each; a thread has kAhead rows in flight.
//
// Measured: 2.6 us for one token of 16 requests (4 KV heads of 128, pages of
// 16); 12.6 us for 10 thousand tokens into an e4m3 cache (31 MB, 2.4 TB/s: the
// quotients and conversions keep the issue slots 60 % busy, the rest is the
// latency of slot, row and summary); 17.6 us for 9 thousand tokens of 8 heads of
// 128 in bf16 (75 MB, 4.2 TB/s: one page in flight per CTA, whose next rows wait
// for the reduction).  On the way, for the e4m3 case: plain divisions
// and a scan per token 28.3 us, keys and values in one CTA 21.0, rows loaded one
// after the other 15.0, windows of 32 keys 12.9 and of 16 values 13.6.
template <int D, int CT, int IT>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const __grid_constant__ moe_reader_kv_append_args a, typename Cell<CT>::type* __restrict__ kc,
              typename Cell<CT>::type* __restrict__ vc, int8_t* __restrict__ codes,
              float* __restrict__ steps, const float* __restrict__ k_scale,
              const float* __restrict__ v_scale, int heads, int shift, int num_pages,
              int key_ctas, int key_window, int value_window, bool wide_k, bool wide_v,
              uint32_t* err) {
  using P2 = typename Pair<CT>::type;
  constexpr int kLanes = D / 8;                          // lanes of a row
  constexpr int kRows = kAppendThreads / kLanes;         // rows at a time
  constexpr int kWarps = kAppendThreads / 32;
  constexpr int kAhead = 4;
  __shared__ uint32_t s_hi[kWarps][D / 2], s_lo[kWarps][D / 2];
  __shared__ float s_max[kWarps];
  __shared__ Window s_window;
  __shared__ __align__(4) bool s_skips[kWarps];
  static_assert(kWarps == 4, "read as one word");
  int* s_slot = s_window.slots;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int head = blockIdx.y, ps = 1 << shift;
  const int col = (tid % kLanes) * 8, row0 = tid / kLanes;
  const long long slots_all = (long long)num_pages << shift;

  if ((int)blockIdx.x >= key_ctas) {
    const long long first = (long long)(blockIdx.x - key_ctas) * value_window;
    const Divider vd(CT == MOE_READER_TYPE_E4M3 ? v_scale[head] : 1.f);
    const uint16_t* vin = static_cast<const uint16_t*>(a.v) + head * a.v_head_stride + col;
    const int n = (int)min((long long)value_window, a.tokens - first);
    for (int i0 = row0; i0 < n; i0 += kRows * kAhead) {
      int slot[kAhead];
      uint4 vr[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kRows;
        slot[j] = -1;
        if (i < n) {
          slot[j] = __ldg(a.slots + first + i);
          vr[j] = fetch_new(vin + (first + i) * a.v_token_stride, wide_v);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (slot[j] < 0 || slot[j] >= slots_all) continue;
        const size_t row =
            (((size_t)(slot[j] >> shift) * heads + head) << shift) + (slot[j] & (ps - 1));
        put8<CT>(vc + row * D + col, stored<CT, IT>(vr[j], vd));
      }
    }
    return;
  }

  // the window's slots, a page before them and one behind, in one round of loads
  const long long first = (long long)blockIdx.x * key_window;
  int out = 0;
  for (int i = tid; i <= ps + key_window; i += kAppendThreads) {
    const long long t = first - ps + i;
    const bool in = t >= 0 && t < a.tokens;
    const int slot = in ? __ldg(a.slots + t) : -1;
    s_slot[i] = slot;
    out |= in ? slot | (int)(slots_all - 1 - slot) : 0;
  }
  // a sign: a skipped token among them (a barrier that reduces costs prompts 5 %)
  const bool some = __any_sync(0xffffffffu, out < 0);
  if (lane == 0) s_skips[wid] = some;
  __syncthreads();
  const bool skips = *reinterpret_cast<const uint32_t*>(s_skips) != 0;
  // the tokens of the window that close their page's run (the same in every warp)
  unsigned long long todo = 0;
#pragma unroll
  for (int half = 0; half < kKeyWindow; half += 32) {
    const int i = half + lane;
    bool closes = false;
    if (i < key_window && first + i < a.tokens) {
      const int slot = s_slot[ps + i];
      if (slot >= 0 && slot < slots_all)
        closes = (slot & (ps - 1)) == ps - 1 || s_slot[ps + i + 1] != slot + 1;
      else if (slot != -1 && wid == 0)
        atomicOr(err, kErrPage);
    }
    todo |= (unsigned long long)__ballot_sync(0xffffffffu, closes) << half;
  }
  if (!todo) return;
  if (skips && codes) {
    if (tid == 0) s_window.ends = todo, s_window.followed = s_window.follows = 0;
    if (append_cut_runs<D, CT, IT>(s_window, a, kc, codes, steps, k_scale, heads, shift,
                                   (int)slots_all, (int)first))
      return;
  }

  const Divider kd(CT == MOE_READER_TYPE_E4M3 ? k_scale[head] : 1.f);
  const uint16_t* kin = static_cast<const uint16_t*>(a.k) + head * a.k_head_stride + col;
  for (; todo; todo &= todo - 1) {
    const int w = __ffsll(todo) - 1;
    const long long t = first + w;
    const int slot = s_slot[ps + w], off = slot & (ps - 1);
    // the run of new tokens that ends here: its first offset in the page
    int run0 = 0;
    for (int b = 1; b <= off; b += 32) {
      const int back = b + lane;
      const bool in = back <= off && s_slot[ps + w - min(back, ps)] == slot - back;
      const uint32_t out = __ballot_sync(0xffffffffu, !in);
      if (out) {
        run0 = off - (b + __ffs(out) - 1) + 1;
        break;
      }
    }
    const size_t page = ((size_t)(slot >> shift) * heads + head) << shift;   // first row
    P2 hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) hi[i] = lo[i] = as_pair<P2>(0x7fff7fffu);    // NaN: nothing yet
    for (int o0 = (codes ? 0 : run0) + row0; o0 <= off; o0 += kRows * kAhead) {
      uint4 kr[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int o = o0 + j * kRows;
        if (o > off) continue;
        if (o >= run0) {
          const long long tt = t - (off - o);
          kr[j] = fetch_new(kin + tt * a.k_token_stride, wide_k);
        } else {
          kr[j] = fetch_old<CT>(kc + (page + o) * D + col);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int o = o0 + j * kRows;
        if (o > off) continue;
        if (o >= run0) {
          kr[j] = stored<CT, IT>(kr[j], kd);
          put8<CT>(kc + (page + o) * D + col, kr[j]);
        }
        if (codes) {
          P2 p[4];
          pairs_of<CT>(kr[j], p);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hi[i] = __hmax2(hi[i], p[i]);
            lo[i] = __hmin2(lo[i], p[i]);
          }
        }
      }
    }
    if (!codes) continue;
    // rows of a warp, then the warps
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = __hmax2(hi[i], as_pair<P2>(__shfl_xor_sync(0xffffffffu, bits_of(hi[i]), o)));
        lo[i] = __hmin2(lo[i], as_pair<P2>(__shfl_xor_sync(0xffffffffu, bits_of(lo[i]), o)));
      }
    if (lane < kLanes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s_hi[wid][lane * 4 + i] = bits_of(hi[i]);
        s_lo[wid][lane * 4 + i] = bits_of(lo[i]);
      }
    }
    __syncthreads();
    // thread d < D / 2 has two coordinates
    static_assert(D / 2 <= kAppendThreads, "a thread per pair");
    float2 h = make_float2(-INFINITY, -INFINITY), l = make_float2(INFINITY, INFINITY);
    float top = 0.f;
    if (tid < D / 2) {
      P2 hp = as_pair<P2>(s_hi[0][tid]), lp = as_pair<P2>(s_lo[0][tid]);
#pragma unroll
      for (int v = 1; v < kWarps; ++v) {
        hp = __hmax2(hp, as_pair<P2>(s_hi[v][tid]));
        lp = __hmin2(lp, as_pair<P2>(s_lo[v][tid]));
      }
      h = widen2(hp);
      l = widen2(lp);
      // a coordinate whose keys are all NaN says nothing, to the step neither
      if (h.x != h.x) h.x = l.x = 0.f;
      if (h.y != h.y) h.y = l.y = 0.f;
      top = fmaxf(fmaxf(fabsf(h.x), fabsf(l.x)), fmaxf(fabsf(h.y), fabsf(l.y)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_max[wid] = top;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kWarps; ++v) top = fmaxf(top, s_max[v]);
    const int e = step_exponent(top);
    const float inv = two_to(-e);
    const size_t at = (size_t)(slot >> shift) * heads + head;
    if (tid < D / 2) {
      char2* out = reinterpret_cast<char2*>(codes + at * 2 * D);
      out[tid] = make_char2((char)code_up(h.x, inv), (char)code_up(h.y, inv));
      out[D / 2 + tid] = make_char2((char)code_down(l.x, inv), (char)code_down(l.y, inv));
    }
    if (tid == 0) steps[at] = two_to(e);
    __syncthreads();   // s_hi, s_lo and s_max are free again
  }
}

template <int D, int CT, int IT>
void append_as(const moe_reader_kv& kv, const moe_reader_kv_append_args& a, cudaStream_t s) {
  using C = typename Cell<CT>::type;
  // Windows of one token while that is a few CTAs per SM: in a small decode step
  // every token closes its page's run.  A prompt closes a page only every
  // page_size tokens, so its windows are as long as its runs can be expected to
  // be, tokens / max_requests at least, up to a page and what the ballots hold:
  // few CTAs find nothing to close.  (A decode step of many requests must not
  // get long windows: a CTA closes one page after the other.  With windows of a
  // page 1024 requests of 8 heads of 128 in e4m3 took 125 us, with these 22: each
  // token reads the older keys of its page back, and a CTA does one page after
  // the other.)
  const int heads = kv.cfg.num_kv_heads, at_once = kAppendThreads * 8 / D;
  const long long rows = (long long)a.tokens * heads;
  const bool few = rows <= 16LL * kv.sms;
  const long long run = std::max(a.tokens / kv.cfg.max_requests, 1);
  const int key_window =
      few ? 1 : (int)std::min<long long>(std::min(kKeyWindow, kv.cfg.page_size),
                                         std::max(run, rows / (16 * kv.sms)));
  const int value_window =
      few ? 1 : at_once * (int)std::min<long long>(8, 1 + rows / (4 * kv.sms * at_once));
  const unsigned key_ctas = (unsigned)((a.tokens + key_window - 1) / key_window);
  const unsigned value_ctas = (unsigned)((a.tokens + value_window - 1) / value_window);
  auto wide = [](const void* p, int64_t ts, int64_t hs) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ts % 8 == 0 && hs % 8 == 0;
  };
  const dim3 grid(key_ctas + value_ctas, (unsigned)heads);
  append_kernel<D, CT, IT><<<grid, kAppendThreads, 0, s>>>(
      a, static_cast<C*>(kv.k), static_cast<C*>(kv.v), kv.codes, kv.steps, kv.k_scale, kv.v_scale,
      heads, kv.page_shift, kv.cfg.num_pages, (int)key_ctas, key_window, value_window,
      wide(a.k, a.k_token_stride, a.k_head_stride),
      wide(a.v, a.v_token_stride, a.v_head_stride), kv.err);
}

template <int D>
void append_dim(const moe_reader_kv& kv, const moe_reader_kv_append_args& a, cudaStream_t s) {
  switch (kv.cfg.cache_type) {
    case MOE_READER_TYPE_BF16: append_as<D, MOE_READER_TYPE_BF16, MOE_READER_TYPE_BF16>(kv, a, s); break;
    case MOE_READER_TYPE_F16: append_as<D, MOE_READER_TYPE_F16, MOE_READER_TYPE_F16>(kv, a, s); break;
    default:
      if (a.type == MOE_READER_TYPE_BF16)
        append_as<D, MOE_READER_TYPE_E4M3, MOE_READER_TYPE_BF16>(kv, a, s);
      else
        append_as<D, MOE_READER_TYPE_E4M3, MOE_READER_TYPE_F16>(kv, a, s);
  }
}

}  // namespace

cudaError_t launch_kv_plan(const moe_reader_kv& kv, const moe_reader_kv_plan_args& a,
                           cudaStream_t s) {
  // At least one CTA, and up to four per SM: each repeats the scan, but shortens
  // the others' token loops (640 thousand tokens: 15.5 us with one per SM, 10.3
  // with two, 9.0 with four, 11.7 with eight).
  const long long tokens = std::max(a.max_tokens, 1);
  const int grid =
      (int)std::min<long long>(4LL * kv.sms, (tokens + kPlanThreads - 1) / kPlanThreads);
  plan_kernel<<<grid, kPlanThreads, 0, s>>>(a, kv.page_shift, kv.cfg.num_pages, kv.err);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const moe_reader_kv& kv, const moe_reader_kv_append_args& a,
                             cudaStream_t s) {
  switch (kv.cfg.head_dim) {
    case 64: append_dim<64>(kv, a, s); break;
    case 128: append_dim<128>(kv, a, s); break;
    default: append_dim<256>(kv, a, s); break;
  }
  return cudaGetLastError();
}

}  // namespace mr

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
namespace {

bool at_multiple(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return MOE_READER_OK;
  return e == cudaErrorMemoryAllocation ? MOE_READER_ENOMEM : MOE_READER_ECUDA;
}

int check_kv_config(const moe_reader_kv_config* c) {
  if (!c || c->flags != 0) return MOE_READER_EINVAL;
  if (c->num_kv_heads < 1 || c->num_kv_heads > 1024 || c->num_q_heads < 1)
    return MOE_READER_EINVAL;
  if (c->num_q_heads % c->num_kv_heads || c->num_q_heads / c->num_kv_heads > mr::kMaxGroup)
    return MOE_READER_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_READER_EINVAL;
  const int ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1))) return MOE_READER_EINVAL;
  if (c->num_pages < 1 || (long long)c->num_pages * ps >= (1LL << 31)) return MOE_READER_EINVAL;
  if (c->max_requests < 1 || c->max_requests > mr::kMaxRequests) return MOE_READER_EINVAL;
  if (c->cache_type != MOE_READER_TYPE_BF16 && c->cache_type != MOE_READER_TYPE_F16 &&
      c->cache_type != MOE_READER_TYPE_E4M3)
    return MOE_READER_EINVAL;
  return MOE_READER_OK;
}

// Rows and queries have the cache's type; an 8-bit cache takes either 16-bit one.
bool type_fits(int cache, int type) {
  if (cache == MOE_READER_TYPE_E4M3)
    return type == MOE_READER_TYPE_BF16 || type == MOE_READER_TYPE_F16;
  return type == cache;
}

// An array of 32-bit words.
struct Words {
  const int32_t* at;
  long long count;
};
bool share_a_word(const Words& a, const Words& b) {
  if (a.count == 0 || b.count == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
  return a0 < b0 + 4 * b.count && b0 < a0 + 4 * a.count;
}

// Launches go to the calling thread's device: it has to be the handle's.
bool on_device(const moe_reader_kv* kv) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == kv->device;
}

}  // namespace

extern "C" {

int moe_reader_kv_create(const moe_reader_kv_config* cfg, void* k, void* v, int8_t* codes,
                         float* steps, const float* k_scale, const float* v_scale, void* stream,
                         moe_reader_kv_t** out) {
  if (!out) return MOE_READER_EINVAL;
  *out = nullptr;
  const int st = check_kv_config(cfg);
  if (st != MOE_READER_OK) return st;
  if (!k || !v || k == v || !at_multiple(k, 256) || !at_multiple(v, 256)) return MOE_READER_EINVAL;
  if (!codes != !steps || !at_multiple(codes, 16) || !at_multiple(steps, 4))
    return MOE_READER_EINVAL;
  const bool e4m3 = cfg->cache_type == MOE_READER_TYPE_E4M3;
  if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr)) return MOE_READER_EINVAL;
  if (!at_multiple(k_scale, 4) || !at_multiple(v_scale, 4)) return MOE_READER_EINVAL;
  moe_reader_kv* kv = static_cast<moe_reader_kv*>(calloc(1, sizeof(moe_reader_kv)));
  if (!kv) return MOE_READER_ENOMEM;
  kv->cfg = *cfg;
  kv->k = k;
  kv->v = v;
  kv->codes = codes;
  kv->steps = steps;
  kv->k_scale = k_scale;
  kv->v_scale = v_scale;
  kv->group = cfg->num_q_heads / cfg->num_kv_heads;
  while ((1 << kv->page_shift) < cfg->page_size) kv->page_shift++;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaGetDevice(&kv->device);
  const size_t o_bytes = (size_t)mr::kMaxSms * 2 * 16 * cfg->head_dim * sizeof(float);
  const size_t ml_bytes = (size_t)mr::kMaxSms * 2 * 2 * 16 * sizeof(float);
  const size_t items = (size_t)cfg->max_requests * cfg->num_kv_heads * mr::attend_row_tiles(*cfg);
  const size_t c_bytes = (items * 4 + 255) & ~(size_t)255;
  const size_t bytes = o_bytes + ml_bytes + c_bytes + 256;
  cudaError_t ce = mr::device_alloc(&kv->base, bytes);
  if (ce != cudaSuccess) {
    free(kv);
    return status_of(ce);
  }
  char* b = static_cast<char*>(kv->base);
  kv->part_o = reinterpret_cast<float*>(b);
  kv->part_ml = reinterpret_cast<float*>(b + o_bytes);
  kv->arrived = reinterpret_cast<uint32_t*>(b + o_bytes + ml_bytes);
  kv->arrived_bytes = c_bytes;
  kv->err = reinterpret_cast<uint32_t*>(b + o_bytes + ml_bytes + c_bytes);
  do {
    if ((ce = cudaDeviceGetAttribute(&kv->sms, cudaDevAttrMultiProcessorCount, kv->device)) !=
        cudaSuccess)
      break;
    kv->sms = std::min(kv->sms, mr::kMaxSms);
    if ((ce = mr::configure_kv_attend(*kv)) != cudaSuccess) break;
    if ((ce = mr::configure_kv_select(*kv)) != cudaSuccess) break;
    if ((ce = cudaMemsetAsync(kv->base, 0, bytes, s)) != cudaSuccess) break;
    ce = cudaStreamSynchronize(s);
  } while (0);
  if (ce != cudaSuccess) {
    cudaFree(kv->base);
    free(kv);
    return status_of(ce);
  }
  *out = kv;
  return MOE_READER_OK;
}

int moe_reader_kv_plan(moe_reader_kv_t* kv, const moe_reader_kv_plan_args* a, void* stream) {
  if (!kv || !a) return MOE_READER_EINVAL;
  if (a->requests < 0 || a->requests > kv->cfg.max_requests) return MOE_READER_EINVAL;
  if (a->width < 1 || a->num_free < 0 || a->max_tokens < 0) return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  if (!a->starts || !a->taken) return MOE_READER_EINVAL;
  if (a->requests && (!a->prev_lens || !a->new_lens || !a->table || !a->lens))
    return MOE_READER_EINVAL;
  if (a->num_free && !a->free_pages) return MOE_READER_EINVAL;
  if (a->max_tokens && (!a->slots || !a->positions || !a->token_requests))
    return MOE_READER_EINVAL;
  const void* words[] = {a->prev_lens, a->new_lens, a->table, a->free_pages, a->lens, a->starts,
                         a->slots, a->positions, a->token_requests, a->taken};
  for (const void* p : words)
    if (!at_multiple(p, 4)) return MOE_READER_EINVAL;
  // CTAs still read the inputs while others write the outputs
  const long long R = a->requests, T = a->max_tokens;
  const Words ins[] = {{a->prev_lens, R}, {a->new_lens, R}, {a->free_pages, a->num_free}};
  const Words outs[] = {{a->table, R * a->width}, {a->lens, R}, {a->starts, R + 1}, {a->slots, T},
                        {a->positions, T}, {a->token_requests, T}, {a->taken, 1}};
  for (const Words& o : outs) {
    for (const Words& i : ins)
      if (share_a_word(o, i)) return MOE_READER_EINVAL;
    for (const Words* p = outs; p != &o; ++p)
      if (share_a_word(o, *p)) return MOE_READER_EINVAL;
  }
  if (!on_device(kv)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(mr::launch_kv_plan(*kv, *a, s));
}

int moe_reader_kv_append(moe_reader_kv_t* kv, const moe_reader_kv_append_args* a, void* stream) {
  if (!kv || !a || a->tokens < 0) return MOE_READER_EINVAL;
  if (!type_fits(kv->cfg.cache_type, a->type)) return MOE_READER_EINVAL;
  if (a->tokens == 0) return MOE_READER_OK;
  if (!a->k || !a->v || !a->slots) return MOE_READER_EINVAL;
  if (!at_multiple(a->k, 2) || !at_multiple(a->v, 2) || !at_multiple(a->slots, 4))
    return MOE_READER_EINVAL;
  if (!on_device(kv)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(mr::launch_kv_append(*kv, *a, s));
}

int moe_reader_kv_attend(moe_reader_kv_t* kv, const moe_reader_kv_attend_args* a, void* stream) {
  if (!kv || !a) return MOE_READER_EINVAL;
  if (a->requests < 0 || a->requests > kv->cfg.max_requests) return MOE_READER_EINVAL;
  if (!type_fits(kv->cfg.cache_type, a->q_type)) return MOE_READER_EINVAL;
  if (a->width < 1 || a->window < 0 || (a->pages && a->keep < 1)) return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  // a row's keys and the work list are indexed with 32 bits
  const long long pages = a->pages ? a->keep : a->width;
  const long long items = (long long)a->requests * kv->cfg.num_kv_heads;
  if (pages << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  if (items * (pages << kv->page_shift) >= (1LL << 34)) return MOE_READER_EINVAL;
  if (a->requests == 0) return MOE_READER_OK;
  if (!a->q || !a->table || !a->lens || !a->out) return MOE_READER_EINVAL;
  if (!at_multiple(a->q, 2) || !at_multiple(a->out, 16)) return MOE_READER_EINVAL;
  {
    // a CTA writes its row's output while others read their rows' queries
    const long long heads = kv->cfg.num_q_heads, dim = kv->cfg.head_dim;
    const long long rs = (a->requests - 1) * a->q_request_stride, hs = (heads - 1) * a->q_head_stride;
    const uintptr_t q = reinterpret_cast<uintptr_t>(a->q), o = reinterpret_cast<uintptr_t>(a->out);
    const uintptr_t q0 = q + 2 * (std::min(rs, 0LL) + std::min(hs, 0LL));
    const uintptr_t q1 = q + 2 * (std::max(rs, 0LL) + std::max(hs, 0LL) + dim);
    if (q0 < o + 2 * a->requests * heads * dim && o < q1) return MOE_READER_EINVAL;
  }
  const void* words[] = {a->table, a->lens, a->pages, a->sinks, a->lse};
  for (const void* p : words)
    if (!at_multiple(p, 4)) return MOE_READER_EINVAL;
  if (!on_device(kv)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(mr::launch_kv_attend(*kv, *a, s));
}

int moe_reader_kv_select(moe_reader_kv_t* kv, const moe_reader_kv_select_args* a, void* stream) {
  if (!kv || !a || !kv->codes) return MOE_READER_EINVAL;
  if (a->requests < 0 || a->requests > kv->cfg.max_requests) return MOE_READER_EINVAL;
  if (!type_fits(kv->cfg.cache_type, a->q_type)) return MOE_READER_EINVAL;
  if (a->width < 1 || a->width > mr::kMaxSelectPages) return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  if (a->first < 0 || a->last < 0 || a->keep < 1 ||
      (long long)a->first + a->last > (long long)a->keep)
    return MOE_READER_EINVAL;
  if (a->requests == 0) return MOE_READER_OK;
  if (!a->q || !a->table || !a->lens || !a->pages) return MOE_READER_EINVAL;
  if (!at_multiple(a->q, 2) || !at_multiple(a->table, 4) || !at_multiple(a->lens, 4) ||
      !at_multiple(a->pages, 4))
    return MOE_READER_EINVAL;
  if (!on_device(kv)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(mr::launch_kv_select(*kv, *a, s));
}

int moe_reader_kv_status(moe_reader_kv_t* kv, uint32_t* bits_out) {
  if (!kv || !on_device(kv)) return MOE_READER_EINVAL;
  // the whole device: a captured call runs on whichever stream replays it
  cudaError_t ce = cudaDeviceSynchronize();
  if (ce != cudaSuccess) return status_of(ce);
  uint32_t bits = 0;
  if ((ce = cudaMemcpy(&bits, kv->err, 4, cudaMemcpyDeviceToHost)) != cudaSuccess)
    return status_of(ce);
  if (bits) {
    // cleared before this returns: streams need not wait for the default one.
    // What a launch that gave up has counted does not hold for the next one.
    ce = cudaMemsetAsync(kv->err, 0, 4, cudaStreamLegacy);
    if (ce == cudaSuccess && (bits & MOE_READER_ERR_TIMEOUT))
      ce = cudaMemsetAsync(kv->arrived, 0, kv->arrived_bytes, cudaStreamLegacy);
    if (ce == cudaSuccess) ce = cudaStreamSynchronize(cudaStreamLegacy);
    if (ce != cudaSuccess) return status_of(ce);
  }
  if (bits_out) *bits_out = bits;
  if (bits & MOE_READER_ERR_TIMEOUT) return MOE_READER_ETIMEOUT;
  return bits ? MOE_READER_EDEVICE : MOE_READER_OK;
}

void moe_reader_kv_destroy(moe_reader_kv_t* kv) {
  if (!kv) return;
  cudaDeviceSynchronize();
  cudaFree(kv->base);
  free(kv);
}

}  // extern "C"
