// Page selection: the reader's screen applied to attention.  Each page of a
// request is scored against the group's query heads from its int8 summary,
// and the best `keep` pages are listed for kv_attend.
//
// score(page) = step sum_d (hi_d P_d - lo_d N_d), P_d = sum_g max(q_gd, 0),
// N_d = sum_g max(-q_gd, 0): because max(q hi, q lo) = max(q,0) hi - max(-q,0) lo
// for hi >= lo, this is the sum over the group's heads of the largest q . k
// that a key inside the page's box could have, and costs one dot product of
// 2D bytes a page whatever the group's size.  P and N are rounded to 7 bits,
// so the sum is an integer dot product (dp4a) and, times a power of two, an
// exact fp32 number: no order of summation can change the choice.
//
// One cluster per (request, KV head).  All its CTAs score a share of the
// pages and store the order keys into the first CTA's shared memory; that CTA
// finds the threshold by a histogram over the keys' own range and writes the
// list.  One launch, no scratch in global memory, no atomics across CTAs.
//
// Bound by the chain of round trips, not by bytes.  8192 pages of 4 KV heads
// (8.4 MB of summaries) take 10.6 us: the page ids 1.5, the query's codes 1.6
// (summaries in flight meanwhile), the products 0.7, the hand-over to the first
// CTA 1.0, the threshold 3.2 (two histogram passes), the list 2.  With clusters
// of 8 CTAs instead of 16 the same selection took 5 us more.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv.cuh"

namespace cg = cooperative_groups;

namespace mr {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostCtas = 16;                  // CTAs of a cluster (above 8 on request)
constexpr uint32_t kForced = 0xffffffffu;      // above every score's key

struct Params {
  moe_reader_kv_select_args a;
  const int8_t* codes;
  const float* steps;
  int kv_heads, group, shift, num_pages;
  uint32_t* err;
};

__device__ __forceinline__ float load_q(const uint16_t* p, int type) {
  const uint16_t u = __ldg(p);
  const float f = type == MOE_READER_TYPE_BF16 ? __uint_as_float((uint32_t)u << 16)
                                               : __half2float(__ushort_as_half(u));
  return f == f ? f : 0.f;
}

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v = fmaxf(v, s[w]);
  return v;
}

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const Params P) {
  constexpr int kLanes = D / 8;                 // lanes of a page: 16 bytes each of 2D
  constexpr int kGroups = 32 / kLanes;          // pages a warp loads at a time
  constexpr int kHold = kLanes < 16 ? kLanes : 16;   // loads in flight per lane
  constexpr int kPages = kHold * kGroups;       // a warp's batch
  extern __shared__ uint32_t s_keys[];          // first CTA: a key per page
  __shared__ __align__(16) int8_t s_q[2 * D];
  __shared__ float s_red[kWarps];
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[2][kWarps];
  __shared__ uint32_t s_range[2];
  __shared__ int s_bin, s_need, s_in_bin;

  let_next_launch_start();
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int head = blockIdx.y, r = blockIdx.z;
  const moe_reader_kv_select_args& a = P.a;
  const int ps = 1 << P.shift, room = a.width << P.shift;
  int len = __ldg(a.lens + r);
  uint32_t bad = 0;
  if (len < 0) len = 0, bad = kErrLength;
  if (len > room) len = room, bad = kErrLength;
  if (bad && rank == 0 && head == 0 && tid == 0) atomicOr(P.err, bad);
  bad = 0;
  const int held = (len + ps - 1) >> P.shift;
  int32_t* out = a.pages + ((size_t)r * P.kv_heads + head) * a.keep;
  if (held <= a.keep) {                         // the same for the whole cluster
    if (rank == 0)
      for (int i = tid; i < a.keep; i += kThreads) out[i] = i < held ? i : -1;
    return;
  }
  cluster.barrier_arrive();                     // this CTA has started (waited for below)

  // ---- this CTA's pages; the first batch's summaries are on their way while
  // the query is coded ----
  const int32_t* table = a.table + (size_t)r * a.width;
  const int share = ((held + ctas - 1) / ctas + 31) & ~31;
  const int p_end = min(held, (rank + 1) * share);
  const int sub = lane / kLanes;
  // the lane's own page after the sums: load (lane % kHold), group sub
  const int own = (lane % kHold) * kGroups + sub;
  const bool owns = lane % kLanes < kHold;
  int4 c[kHold];
  int own_id = -1;
  float step = 0.f;
  auto fetch = [&](int base) {
    int id = -1;
    if (lane < kPages && base + lane < p_end) {
      id = __ldg(table + base + lane);
      if (id < 0 || id >= P.num_pages) bad |= kErrPage, id = -1;
    }
    own_id = __shfl_sync(0xffffffffu, id, own);
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int at = __shfl_sync(0xffffffffu, id, i * kGroups + sub);
      c[i] = make_int4(0, 0, 0, 0);
      if (at >= 0)
        c[i] = __ldg(reinterpret_cast<const int4*>(
            P.codes + ((size_t)at * P.kv_heads + head) * 2 * D + 16 * (lane % kLanes)));
    }
    step = own_id >= 0 ? __ldg(P.steps + (size_t)own_id * P.kv_heads + head) : 0.f;
  };
  int base = rank * share + wid * kPages;
  fetch(base);

  // ---- the group's query as 7-bit codes ----
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + r * a.q_request_stride +
                      (long long)head * P.group * a.q_head_stride;
  float top = 0.f;
  for (int i = tid; i < P.group * D; i += kThreads)
    top = fmaxf(top, fabsf(load_q(q + (i / D) * a.q_head_stride + i % D, a.q_type)));
  const float up = two_to(13 - floor_log2_held(block_max(top, s_red)));
  float pos = 0.f, neg = 0.f;                   // integers below 2^21: exact
  if (tid < D) {
#pragma unroll 4
    for (int g = 0; g < P.group; ++g) {
      // an infinite q is held to the range the codes can express
      const float f = rintf(fminf(fmaxf(load_q(q + g * a.q_head_stride + tid, a.q_type) * up,
                                        -16384.f), 16384.f));
      pos += fmaxf(f, 0.f);
      neg += fmaxf(-f, 0.f);
    }
  }
  const float most = block_max(fmaxf(fmaxf(pos, neg), 1.f), s_red);
  const float down = two_to(6 - floor_log2_held(most));
  if (tid < D) {
    s_q[tid] = (int8_t)fminf(rintf(pos * down), 127.f);
    s_q[D + tid] = (int8_t)-fminf(rintf(neg * down), 127.f);
  }
  __syncthreads();

  // ---- scores ----
  cluster.barrier_wait();                       // the first CTA's memory can be written
  uint32_t* keys = cluster.map_shared_rank(s_keys, 0);
  const int4 mine = *reinterpret_cast<const int4*>(s_q + 16 * (lane % kLanes));
  while (base < p_end) {
    int dot[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      int v = __dp4a(c[i].x, mine.x, 0);
      v = __dp4a(c[i].y, mine.y, v);
      v = __dp4a(c[i].z, mine.z, v);
      dot[i] = __dp4a(c[i].w, mine.w, v);
    }
    const int page = base + own, id = own_id;
    const float unit = step;
    base += kWarps * kPages;
    if (base < p_end) fetch(base);
    // sums over the lanes of a page, each lane ending with one page's
#pragma unroll
    for (int o = kLanes / 2; o >= kHold; o >>= 1)
#pragma unroll
      for (int i = 0; i < kHold; ++i) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
#pragma unroll
    for (int o = kHold / 2; o > 0; o >>= 1) {
      const bool high = lane & o;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const int send = high ? dot[i] : dot[i + o];
        const int keep = high ? dot[i + o] : dot[i];
        dot[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    if (owns && page < p_end) {
      // NaN (a step that nothing has written) ranks with the pages outside the
      // pool: its key would be the forced pages' and the list overrun
      const float score = (float)dot[0] * unit;
      uint32_t key = id < 0 || score != score ? 0u : order_key(score);
      if (page < a.first || page >= held - a.last) key = kForced;
      keys[page] = key;
    }
  }
  if (bad) atomicOr(P.err, bad);
  cluster.barrier_arrive();                     // the others only hand over their keys
  if (rank != 0) return;
  cluster.barrier_wait();

  // ---- threshold: the need-th largest key that is not forced ----
  int need = a.keep - (a.first + a.last);
  uint32_t T = kForced - 1;                     // nothing but the forced pages
  int need_eq = 0;
  if (need > 0) {
    uint32_t lo = kForced, hi = 0;
#pragma unroll 4
    for (int i = tid; i < held; i += kThreads) {
      const uint32_t k = s_keys[i];
      if (k == kForced) continue;
      lo = min(lo, k);
      hi = max(hi, k);
    }
    if (tid == 0) s_range[0] = kForced, s_range[1] = 0;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&s_range[0], lo);
      atomicMax(&s_range[1], hi);
    }
    __syncthreads();
    uint32_t from = s_range[0], span = s_range[1] - s_range[0];
    int shift = max(0, 32 - __clz(span) - 11);
    for (;;) {
      for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = tid; i < held; i += kThreads) {
        const uint32_t k = s_keys[i];
        if (k != kForced && k >= from && k - from <= span) atomicAdd(&s_hist[(k - from) >> shift], 1);
      }
      __syncthreads();
      // from the top: thread i has bins kBins - 1 - 4i and the three below
      constexpr int kPer = kBins / kThreads;
      int n[kPer], sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += n[j] = s_hist[kBins - 1 - tid * kPer - j];
      int in = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += u;
      }
      if (lane == 31) s_warp[0][wid] = in;
      __syncthreads();
      int above = in - sum;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) above += w < wid ? s_warp[0][w] : 0;
      if (above < need && need <= above + sum) {
        int j = 0;
#pragma unroll
        for (; j < kPer - 1; ++j) {
          if (above + n[j] >= need) break;
          above += n[j];
        }
        s_bin = kBins - 1 - tid * kPer - j;
        s_need = need - above;
        s_in_bin = s_hist[s_bin];
      }
      __syncthreads();
      const uint32_t at = from + ((uint32_t)s_bin << shift);
      need = s_need;
      if (s_in_bin == need) {                   // the whole bin is kept
        T = at - 1;
        break;
      }
      if (shift == 0) {
        T = at;
        need_eq = need;
        break;
      }
      from = at;
      span = (1u << shift) - 1;
      shift = max(0, shift - 11);
      __syncthreads();
    }
  }

  // ---- the list, ascending: keys above T, and the first need_eq at T ----
  const int seg = ((held + kWarps - 1) / kWarps + 31) & ~31;
  const int b0 = wid * seg, b1 = min(held, b0 + seg);
  int gt = 0, eq = 0;
#pragma unroll 8
  for (int i = b0 + lane; i < b1; i += 32) {
    gt += s_keys[i] > T;
    eq += s_keys[i] == T;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();
  if (lane == 0) {
    s_warp[0][wid] = gt;
    s_warp[1][wid] = eq;
  }
  __syncthreads();
  gt = eq = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    gt += w < wid ? s_warp[0][w] : 0;
    eq += w < wid ? s_warp[1][w] : 0;
  }
#pragma unroll 8
  for (int i = b0; i < b1; i += 32) {
    const uint32_t k = i + lane < b1 ? s_keys[i + lane] : 0;
    const bool in = i + lane < b1;
    const uint32_t m_gt = __ballot_sync(0xffffffffu, in && k > T);
    const uint32_t m_eq = __ballot_sync(0xffffffffu, in && k == T);
    const uint32_t below = (1u << lane) - 1;
    const int my_gt = gt + __popc(m_gt & below), my_eq = eq + __popc(m_eq & below);
    if (in && (k > T || (k == T && my_eq < need_eq))) out[my_gt + min(my_eq, need_eq)] = i + lane;
    gt += __popc(m_gt);
    eq += __popc(m_eq);
  }
}

template <int D>
cudaError_t launch(const Params& P, int sms, cudaStream_t s) {
  // CTAs per row: as many as the rows leave SMs for, each with a batch of 32
  // pages per warp at least
  const long long rows = (long long)P.a.requests * P.kv_heads;
  int ctas = 1;
  while (ctas < kMostCtas && rows * ctas <= sms && P.a.width > ctas * kThreads) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)P.kv_heads, (unsigned)P.a.requests);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)P.a.width * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<D>, P);
}

template <int D>
cudaError_t configure() {
  const cudaError_t e = cudaFuncSetAttribute(
      select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSelectPages * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

}  // namespace

cudaError_t configure_kv_select(const moe_reader_kv& kv) {
  switch (kv.cfg.head_dim) {
    case 64: return configure<64>();
    case 128: return configure<128>();
    default: return configure<256>();
  }
}

cudaError_t launch_kv_select(const moe_reader_kv& kv, const moe_reader_kv_select_args& a,
                             cudaStream_t s) {
  Params P;
  P.a = a;
  P.codes = kv.codes;
  P.steps = kv.steps;
  P.kv_heads = kv.cfg.num_kv_heads;
  P.group = kv.group;
  P.shift = kv.page_shift;
  P.num_pages = kv.cfg.num_pages;
  P.err = kv.err;
  switch (kv.cfg.head_dim) {
    case 64: return launch<64>(P, kv.sms, s);
    case 128: return launch<128>(P, kv.sms, s);
    default: return launch<256>(P, kv.sms, s);
  }
}

}  // namespace mr
