// A prompt's experts: pairs (token, slot) sorted by expert, and products grouped
// by expert over ragged numbers of rows.
#include <stdlib.h>

#include <algorithm>

#include "device_util.cuh"
#include "internal.cuh"
#include "moe_reader.h"

struct moe_reader_experts {
  moe_reader_experts_config cfg;
  int device;
  int sms;
  const void* gate;          // caller-owned [E][I][H]
  const void* up;
  const void* down;          // caller-owned [E][H][I]
  uint32_t* err;             // [1] device error word
};

namespace mr {
namespace {

constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

// CTA e lists the pairs of expert e, the last CTA those that belong to none.
// Each counts for itself the pairs of the experts before its own (one pass over
// the ids, from L2) and then writes its own in order: one launch, no hand-off
// between CTAs, and the order does not depend on their timing.
__global__ void __launch_bounds__(kPlanThreads)
experts_plan_kernel(moe_reader_experts_plan_args a) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_before, s_mine;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int e = blockIdx.x, E = a.num_experts;
  const long long pairs = (long long)a.tokens * a.experts_per_token;
  if (tid == 0) s_before = s_mine = 0;
  __syncthreads();
  int before = 0, mine = 0;
  for (long long i = tid; i < pairs; i += kPlanThreads) {
    const int id = __ldg(a.ids + i);
    const unsigned u = (unsigned)id < (unsigned)E ? id : E;
    before += u < e;
    mine += u == e;
  }
  before = warp_sum_i(before);
  mine = warp_sum_i(mine);
  if (lane == 0) {
    atomicAdd(&s_before, before);
    atomicAdd(&s_mine, mine);
  }
  __syncthreads();
  if (tid == 0) {
    a.offsets[e] = s_before;
    if (e == E) a.skipped[0] = s_mine;
  }
  int at = s_before;
  if (s_mine == 0) return;
  for (long long b = 0; b < pairs; b += kPlanThreads) {
    const long long i = b + tid;
    const int id = i < pairs ? __ldg(a.ids + i) : INT32_MIN;
    const bool is = i < pairs && (e < E ? id == e : (unsigned)id >= (unsigned)E);
    const uint32_t m = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_warp[wid] = __popc(m);
    __syncthreads();
    int off = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < wid) off += s_warp[w];
      all += s_warp[w];
    }
    if (is) {
      const int row = at + off + __popc(m & ((1u << lane) - 1));
      if (e < E) {
        a.order[row] = (int)i;
        a.places[i] = row;
      } else {
        a.order[row] = -1;
        a.places[i] = -1;
      }
    }
    at += all;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
template <int T> __device__ __forceinline__ float wide(const void* p, long long i) {
  if constexpr (T == MOE_READER_TYPE_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else if constexpr (T == MOE_READER_TYPE_F16)
    return __half2float(static_cast<const __half*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}
template <int T> __device__ __forceinline__ void put(void* p, long long i, float v) {
  if constexpr (T == MOE_READER_TYPE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else if constexpr (T == MOE_READER_TYPE_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ int expert_of(const int32_t* offsets, int E, int row) {
  int lo = 0, hi = E;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(offsets + mid) <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

constexpr int kChannels = 256;

template <int T>
__global__ void __launch_bounds__(kChannels)
activate_kernel(moe_reader_experts_activate_args a, const void* gate, const void* up, int H, int I,
                int E, int topk) {
  const int row = blockIdx.x, ch = blockIdx.y * kChannels + threadIdx.x;
  const int e = expert_of(a.offsets, E, row), pair = __ldg(a.order + row);
  if (e >= E || pair < 0 || pair >= (long long)a.tokens * topk || ch >= I) return;
  const long long x = (long long)(pair / topk) * a.x_stride, w = ((long long)e * I + ch) * H;
  float g = 0.f, v = 0.f;
  for (int i = 0; i < H; ++i) {
    const float xi = wide<T>(a.x, x + i);
    g += xi * wide<T>(gate, w + i);
    v += xi * wide<T>(up, w + i);
  }
  put<T>(a.act, (long long)row * I + ch, silu_f(g) * v);
}

template <int T>
__global__ void __launch_bounds__(kChannels)
down_kernel(moe_reader_experts_combine_args a, const void* down, int H, int I, int E) {
  const int row = blockIdx.x, ch = blockIdx.y * kChannels + threadIdx.x;
  const int e = expert_of(a.offsets, E, row);
  if (e >= E || ch >= H) return;
  const long long w = ((long long)e * H + ch) * I;
  float z = 0.f;
  for (int i = 0; i < I; ++i) z += wide<T>(a.act, (long long)row * I + i) * wide<T>(down, w + i);
  a.slots[(long long)row * H + ch] = z;
}

template <int T>
__global__ void __launch_bounds__(kChannels)
combine_kernel(moe_reader_experts_combine_args a, int H, int topk) {
  const int t = blockIdx.x, ch = blockIdx.y * kChannels + threadIdx.x;
  if (ch >= H) return;
  float y = 0.f;
  for (int s = 0; s < topk; ++s) {
    const int row = __ldg(a.places + (long long)t * topk + s);
    if (row >= 0 && row < (long long)a.tokens * topk)
      y += __ldg(a.weights + (long long)t * topk + s) * a.slots[(long long)row * H + ch];
  }
  put<T>(a.y, t * a.y_stride + ch, y);
}

template <int T>
cudaError_t activate_as(const moe_reader_experts& h, const moe_reader_experts_activate_args& a,
                        cudaStream_t s) {
  const dim3 grid((unsigned)(a.tokens * a.experts_per_token),
                  (unsigned)((h.cfg.inter + kChannels - 1) / kChannels));
  activate_kernel<T><<<grid, kChannels, 0, s>>>(a, h.gate, h.up, h.cfg.hidden, h.cfg.inter,
                                                h.cfg.num_experts, a.experts_per_token);
  return cudaGetLastError();
}

template <int T>
cudaError_t combine_as(const moe_reader_experts& h, const moe_reader_experts_combine_args& a,
                       cudaStream_t s) {
  const unsigned chunks = (unsigned)((h.cfg.hidden + kChannels - 1) / kChannels);
  const int topk = a.experts_per_token;
  down_kernel<T><<<dim3((unsigned)(a.tokens * topk), chunks), kChannels, 0, s>>>(
      a, h.down, h.cfg.hidden, h.cfg.inter, h.cfg.num_experts);
  const dim3 grid((unsigned)a.tokens, chunks);
  switch (a.y_type) {
    case MOE_READER_TYPE_BF16:
      combine_kernel<MOE_READER_TYPE_BF16><<<grid, kChannels, 0, s>>>(a, h.cfg.hidden, topk);
      break;
    case MOE_READER_TYPE_F16:
      combine_kernel<MOE_READER_TYPE_F16><<<grid, kChannels, 0, s>>>(a, h.cfg.hidden, topk);
      break;
    default:
      combine_kernel<MOE_READER_TYPE_F32><<<grid, kChannels, 0, s>>>(a, h.cfg.hidden, topk);
  }
  return cudaGetLastError();
}

}  // namespace
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

bool on_device(const moe_reader_experts* h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

// Bytes from `at` on.
struct Bytes {
  const void* at;
  long long count;
};
bool overlap(const Bytes& a, const Bytes& b) {
  if (a.count <= 0 || b.count <= 0 || !a.at || !b.at) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
  return a0 < b0 + b.count && b0 < a0 + a.count;
}
template <int I, int O>
bool apart(const Bytes (&ins)[I], const Bytes (&outs)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(outs[o], ins[i])) return false;
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return false;
  }
  return true;
}

// Pairs are counted with 32 bits, and so are rows of a token's pairs.
bool pairs_fit(int tokens, int topk) { return (long long)tokens * topk < (1LL << 30); }

}  // namespace

extern "C" {

int moe_reader_experts_create(const moe_reader_experts_config* c, const void* gate, const void* up,
                              const void* down, void* stream, moe_reader_experts_t** out) {
  if (!out) return MOE_READER_EINVAL;
  *out = nullptr;
  if (!c || c->flags != 0) return MOE_READER_EINVAL;
  if (c->hidden < 8 || c->hidden > 65536 || c->hidden % 8) return MOE_READER_EINVAL;
  if (c->inter < 8 || c->inter > 65536 || c->inter % 8) return MOE_READER_EINVAL;
  if (c->num_experts < 1 || c->num_experts > mr::kMaxExperts) return MOE_READER_EINVAL;
  if (c->type != MOE_READER_TYPE_BF16 && c->type != MOE_READER_TYPE_F16) return MOE_READER_EINVAL;
  if (!gate != !up || (!gate && !down)) return MOE_READER_EINVAL;
  if (!at_multiple(gate, 16) || !at_multiple(up, 16) || !at_multiple(down, 16))
    return MOE_READER_EINVAL;
  moe_reader_experts* h = static_cast<moe_reader_experts*>(calloc(1, sizeof(moe_reader_experts)));
  if (!h) return MOE_READER_ENOMEM;
  h->cfg = *c;
  h->gate = gate;
  h->up = up;
  h->down = down;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaGetDevice(&h->device);
  void* p = nullptr;
  cudaError_t ce = mr::device_alloc(&p, 256);
  if (ce != cudaSuccess) {
    free(h);
    return status_of(ce);
  }
  h->err = static_cast<uint32_t*>(p);
  do {
    if ((ce = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device)) !=
        cudaSuccess)
      break;
    if ((ce = cudaMemsetAsync(p, 0, 256, s)) != cudaSuccess) break;
    ce = cudaStreamSynchronize(s);
  } while (0);
  if (ce != cudaSuccess) {
    cudaFree(p);
    free(h);
    return status_of(ce);
  }
  *out = h;
  return MOE_READER_OK;
}

int moe_reader_experts_plan(const moe_reader_experts_plan_args* a, void* stream) {
  if (!a || a->tokens < 0) return MOE_READER_EINVAL;
  if (a->num_experts < 1 || a->num_experts > mr::kMaxExperts) return MOE_READER_EINVAL;
  if (a->experts_per_token < 1 || a->experts_per_token > mr::kMaxTopk) return MOE_READER_EINVAL;
  if (!pairs_fit(a->tokens, a->experts_per_token)) return MOE_READER_EINVAL;
  if (!a->offsets || !a->skipped) return MOE_READER_EINVAL;
  if (a->tokens && (!a->ids || !a->order || !a->places)) return MOE_READER_EINVAL;
  if (!at_multiple(a->ids, 4) || !at_multiple(a->order, 4) || !at_multiple(a->offsets, 4) ||
      !at_multiple(a->places, 4) || !at_multiple(a->skipped, 4))
    return MOE_READER_EINVAL;
  const long long n = 4LL * a->tokens * a->experts_per_token;
  const Bytes ins[] = {{a->ids, n}};
  const Bytes outs[] = {{a->order, n}, {a->offsets, 4LL * (a->num_experts + 1)}, {a->places, n},
                        {a->skipped, 4}};
  if (!apart(ins, outs)) return MOE_READER_EINVAL;
  mr::experts_plan_kernel<<<a->num_experts + 1, mr::kPlanThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(*a);
  return status_of(cudaGetLastError());
}

int moe_reader_experts_activate(moe_reader_experts_t* h, const moe_reader_experts_activate_args* a,
                                void* stream) {
  if (!h || !a || !h->gate || a->tokens < 0) return MOE_READER_EINVAL;
  const moe_reader_experts_config& c = h->cfg;
  if (a->experts_per_token < 1 || a->experts_per_token > mr::kMaxTopk) return MOE_READER_EINVAL;
  if (!pairs_fit(a->tokens, a->experts_per_token)) return MOE_READER_EINVAL;
  if (a->tokens == 0) return MOE_READER_OK;
  if (!a->x || !a->order || !a->offsets || !a->act) return MOE_READER_EINVAL;
  if (!at_multiple(a->x, 16) || !at_multiple(a->act, 16) || a->x_stride % 8)
    return MOE_READER_EINVAL;
  if (!at_multiple(a->order, 4) || !at_multiple(a->offsets, 4)) return MOE_READER_EINVAL;
  const long long pairs = (long long)a->tokens * a->experts_per_token;
  const long long reach = (a->tokens - 1) * a->x_stride;
  const Bytes ins[] = {
      {static_cast<const char*>(a->x) + 2 * std::min(reach, 0LL), 2 * (std::abs(reach) + c.hidden)},
      {a->order, 4 * pairs}, {a->offsets, 4LL * (c.num_experts + 1)},
      {h->gate, 2LL * c.num_experts * c.inter * c.hidden},
      {h->up, 2LL * c.num_experts * c.inter * c.hidden}};
  const Bytes outs[] = {{a->act, 2 * pairs * c.inter}};
  if (!apart(ins, outs) || !on_device(h)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(c.type == MOE_READER_TYPE_BF16
                       ? mr::activate_as<MOE_READER_TYPE_BF16>(*h, *a, s)
                       : mr::activate_as<MOE_READER_TYPE_F16>(*h, *a, s));
}

int moe_reader_experts_combine(moe_reader_experts_t* h, const moe_reader_experts_combine_args* a,
                               void* stream) {
  if (!h || !a || !h->down || a->tokens < 0) return MOE_READER_EINVAL;
  const moe_reader_experts_config& c = h->cfg;
  if (a->experts_per_token < 1 || a->experts_per_token > mr::kMaxTopk) return MOE_READER_EINVAL;
  if (!pairs_fit(a->tokens, a->experts_per_token)) return MOE_READER_EINVAL;
  if (a->y_type < MOE_READER_TYPE_F32 || a->y_type > MOE_READER_TYPE_F16) return MOE_READER_EINVAL;
  if (a->tokens == 0) return MOE_READER_OK;
  if (!a->act || !a->offsets || !a->places || !a->weights || !a->slots || !a->y)
    return MOE_READER_EINVAL;
  if (!at_multiple(a->act, 16) || !at_multiple(a->slots, 16) || !at_multiple(a->y, 16) ||
      a->y_stride % 8)
    return MOE_READER_EINVAL;
  if (!at_multiple(a->offsets, 4) || !at_multiple(a->places, 4) || !at_multiple(a->weights, 4))
    return MOE_READER_EINVAL;
  if (a->tokens > 1 && std::abs((long long)a->y_stride) < c.hidden) return MOE_READER_EINVAL;
  const long long pairs = (long long)a->tokens * a->experts_per_token;
  const long long size = a->y_type == MOE_READER_TYPE_F32 ? 4 : 2;
  const long long reach = (a->tokens - 1) * a->y_stride;
  const Bytes ins[] = {{a->act, 2 * pairs * c.inter}, {a->offsets, 4LL * (c.num_experts + 1)},
                       {a->places, 4 * pairs}, {a->weights, 4 * pairs},
                       {h->down, 2LL * c.num_experts * c.inter * c.hidden}};
  const Bytes outs[] = {{a->slots, 4 * pairs * c.hidden},
                        {static_cast<const char*>(a->y) + size * std::min(reach, 0LL),
                         size * (std::abs(reach) + c.hidden)}};
  if (!apart(ins, outs) || !on_device(h)) return MOE_READER_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(c.type == MOE_READER_TYPE_BF16
                       ? mr::combine_as<MOE_READER_TYPE_BF16>(*h, *a, s)
                       : mr::combine_as<MOE_READER_TYPE_F16>(*h, *a, s));
}

int moe_reader_experts_status(moe_reader_experts_t* h, uint32_t* bits_out) {
  if (!h || !on_device(h)) return MOE_READER_EINVAL;
  // the whole device: a captured call runs on whichever stream replays it
  cudaError_t ce = cudaDeviceSynchronize();
  if (ce != cudaSuccess) return status_of(ce);
  uint32_t bits = 0;
  if ((ce = cudaMemcpy(&bits, h->err, 4, cudaMemcpyDeviceToHost)) != cudaSuccess)
    return status_of(ce);
  if (bits) {
    // cleared before this returns: streams need not wait for the default one
    ce = cudaMemsetAsync(h->err, 0, 4, cudaStreamLegacy);
    if (ce == cudaSuccess) ce = cudaStreamSynchronize(cudaStreamLegacy);
    if (ce != cudaSuccess) return status_of(ce);
  }
  if (bits_out) *bits_out = bits;
  if (bits & MOE_READER_ERR_TIMEOUT) return MOE_READER_ETIMEOUT;
  return bits ? MOE_READER_EDEVICE : MOE_READER_OK;
}

void moe_reader_experts_destroy(moe_reader_experts_t* h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->err);
  free(h);
}

}  // extern "C"
