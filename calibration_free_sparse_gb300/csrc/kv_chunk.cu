// Attention of several new tokens per request over the paged cache.
#include <algorithm>

#include "device_util.cuh"
#include "internal.cuh"
#include "kv.cuh"

namespace mr {
namespace {

template <int CT>
__device__ __forceinline__ float cell(const void* base, long long at) {
  if constexpr (CT == MOE_READER_TYPE_E4M3)
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(
        static_cast<const __nv_fp8_storage_t*>(base)[at], __NV_E4M3)));
  else if constexpr (CT == MOE_READER_TYPE_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  else
    return __half2float(static_cast<const __half*>(base)[at]);
}

// A request's part of the call.
struct Span {
  int first;        // its first row of q
  int tokens;       // new tokens
  int len;          // tokens in the cache, the new ones among them
};
__device__ __forceinline__ Span span_of(const moe_reader_kv_chunk_args& a, int r, uint32_t& bad) {
  const int s = __ldg(a.starts + r), e = __ldg(a.starts + r + 1), len = __ldg(a.lens + r);
  Span x;
  x.first = min(max(s, 0), a.tokens);
  x.tokens = max(min(e, a.tokens) - x.first, 0);
  x.len = max(len, 0);
  if (s < 0 || e < s || e > a.tokens || len < 0 || x.tokens > x.len) bad |= kErrLength;
  return x;
}

constexpr int kRowWarps = 8;

// A warp per row (token, query head): online softmax, lanes over coordinates.
template <int D, int CT, int QT>
__global__ void __launch_bounds__(kRowWarps * 32)
chunk_row_kernel(moe_reader_kv_chunk_args a, const void* k, const void* v, const float* k_scale,
                 const float* v_scale, int heads, int kv_heads, int shift, int pool,
                 uint32_t* err) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int t = (int)(row / heads), head = (int)(row % heads);
  if (t >= a.tokens) return;
  const int kvh = head / (heads / kv_heads);
  uint32_t bad = 0;
  int r = 0;
  Span sp = {};
  for (; r < a.requests; ++r) {
    sp = span_of(a, r, bad);
    if (t >= sp.first && t < sp.first + sp.tokens) break;
  }
  if (r < a.requests) {
    const long long room = (long long)a.width << shift;
    if (sp.len > room) bad |= kErrLength;
    const int pos = sp.len - sp.tokens + t - sp.first;
    const int hi = (int)min((long long)pos + 1, room), lo = a.window ? max(0, pos + 1 - a.window) : 0;
    float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
    for (int i = 0; i < kPer; ++i) {
      q[i] = cell<QT>(a.q, t * a.q_token_stride + head * a.q_head_stride + lane + 32 * i);
      o[i] = 0.f;
    }
    const float scale = a.scale * (k_scale ? k_scale[kvh] : 1.f);
    for (int j = lo; j < hi; ++j) {
      const int page = __ldg(a.table + (size_t)r * a.width + (j >> shift));
      if ((unsigned)page >= (unsigned)pool) {
        bad |= kErrPage;
        continue;
      }
      const long long at =
          ((((long long)page * kv_heads + kvh) << shift) + (j & ((1 << shift) - 1))) * D + lane;
      float s = 0.f;
      for (int i = 0; i < kPer; ++i) s += q[i] * cell<CT>(k, at + 32 * i);
      s = warp_sum(s) * scale;
      const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
      const float f = expf(m - ref), p = expf(s - ref);
      m = top;
      l = l * f + p;
      for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + p * cell<CT>(v, at + 32 * i);
    }
    const float sink = a.sinks ? __ldg(a.sinks + head) : -INFINITY;
    const float top = fmaxf(m, sink), ref = top == -INFINITY ? 0.f : top;
    const float f = expf(m - ref);
    l = l * f + expf(sink - ref);
    const float inv = hi > lo && l != 0.f ? f / l * (v_scale ? v_scale[kvh] : 1.f) : 0.f;
    for (int i = 0; i < kPer; ++i) {
      const long long at = ((long long)t * heads + head) * D + lane + 32 * i;
      const float y = inv == 0.f ? 0.f : o[i] * inv;
      if constexpr (QT == MOE_READER_TYPE_BF16)
        static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
      else
        static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    }
    if (a.lse && lane == 0) a.lse[(long long)t * heads + head] = logf(l) + ref;
  }
  if (bad && lane == 0) atomicOr(err, bad);
}

template <int D, int CT, int QT>
cudaError_t chunk_as(const moe_reader_kv& kv, const moe_reader_kv_chunk_args& a, cudaStream_t s) {
  const long long rows = (long long)a.tokens * kv.cfg.num_q_heads;
  chunk_row_kernel<D, CT, QT><<<(unsigned)((rows + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0,
                                s>>>(a, kv.k, kv.v, kv.k_scale, kv.v_scale, kv.cfg.num_q_heads,
                                     kv.cfg.num_kv_heads, kv.page_shift, kv.cfg.num_pages, kv.err);
  return cudaGetLastError();
}

template <int D>
cudaError_t chunk_dim(const moe_reader_kv& kv, const moe_reader_kv_chunk_args& a, cudaStream_t s) {
  constexpr int B = MOE_READER_TYPE_BF16, H = MOE_READER_TYPE_F16, E = MOE_READER_TYPE_E4M3;
  if (kv.cfg.cache_type == B) return chunk_as<D, B, B>(kv, a, s);
  if (kv.cfg.cache_type == H) return chunk_as<D, H, H>(kv, a, s);
  return a.q_type == B ? chunk_as<D, E, B>(kv, a, s) : chunk_as<D, E, H>(kv, a, s);
}

}  // namespace

cudaError_t launch_kv_chunk(const moe_reader_kv& kv, const moe_reader_kv_chunk_args& a,
                            cudaStream_t s) {
  switch (kv.cfg.head_dim) {
    case 64: return chunk_dim<64>(kv, a, s);
    case 128: return chunk_dim<128>(kv, a, s);
    default: return chunk_dim<256>(kv, a, s);
  }
}

}  // namespace mr

extern "C" int moe_reader_kv_chunk(moe_reader_kv_t* kv, const moe_reader_kv_chunk_args* a,
                                   void* stream) {
  if (!kv || !a) return MOE_READER_EINVAL;
  if (a->requests < 0 || a->requests > kv->cfg.max_requests || a->tokens < 0)
    return MOE_READER_EINVAL;
  if (!mr::type_fits(kv->cfg.cache_type, a->q_type)) return MOE_READER_EINVAL;
  if (a->width < 1 || a->window < 0) return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  // rows of one request's head group, and of the call, are counted with 32 bits
  const long long heads = kv->cfg.num_q_heads, dim = kv->cfg.head_dim;
  if (a->tokens * heads >= (1LL << 31)) return MOE_READER_EINVAL;
  if (a->requests == 0 || a->tokens == 0) return MOE_READER_OK;
  if (!a->q || !a->table || !a->lens || !a->starts || !a->out) return MOE_READER_EINVAL;
  if (reinterpret_cast<uintptr_t>(a->q) % 2 || reinterpret_cast<uintptr_t>(a->out) % 16)
    return MOE_READER_EINVAL;
  const void* words[] = {a->table, a->lens, a->starts, a->sinks, a->lse};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_READER_EINVAL;
  {
    // a CTA writes its rows' output while others read their rows' queries
    const long long ts = (a->tokens - 1) * a->q_token_stride, hs = (heads - 1) * a->q_head_stride;
    const uintptr_t q = reinterpret_cast<uintptr_t>(a->q), o = reinterpret_cast<uintptr_t>(a->out);
    const uintptr_t q0 = q + 2 * (std::min(ts, 0LL) + std::min(hs, 0LL));
    const uintptr_t q1 = q + 2 * (std::max(ts, 0LL) + std::max(hs, 0LL) + dim);
    if (q0 < o + 2 * a->tokens * heads * dim && o < q1) return MOE_READER_EINVAL;
  }
  if (!mr::on_device(kv)) return MOE_READER_EINVAL;
  return mr::status_of(mr::launch_kv_chunk(*kv, *a, static_cast<cudaStream_t>(stream)));
}
