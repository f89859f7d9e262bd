// The norm after a block, its gate, the scaled residual and the norm before
// the next block in one pass over the rows:
//   z = y rsqrt(mean y^2 + eps) w_post,  h' = h + scale gate z,
//   x = h' rsqrt(mean h'^2 + eps) w_pre.
//
// Bound by HBM for many rows (8191 x 2880 bf16 with a gate: 41.8 us, 5.6 TB/s)
// and by latency for few (16 x 2048: 2.3 us, the launch included): a row is read
// once, held in registers through both sums, and written once.  A thread holds V
// vectors of eight neighbouring elements; a row's threads form one CTA.  Rows
// above 16384 elements (8192 with fp32 or mixed types) do not fit the registers
// that way: their kernel reads the row again (from L2) for each of its passes,
// every vector through a switch on its type (with 112 bytes of spills a thread).
// That bounds it: 4096 x 16384 fp32 in place with a bf16 y 254 us, 3.2 TB/s,
// against 82 us, 4.9 TB/s, at 8192 columns, which registers hold.
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "kv.cuh"

namespace mr {
namespace {

using Args = moe_reader_residual_norm_args;

// Eight neighbouring elements as they lie in memory: 16 bytes, or (kWide, a
// call that has an fp32 matrix) 16 or 32.  A row's loads all go out before the
// first one is converted (volatile: the compiler would move some behind the
// first sum).  Plain loads: h may be written in place.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <bool kWide>
struct Raw {
  uint4 a;
};
template <>
struct Raw<true> {
  uint4 a, b;
};

template <int V, bool kWide>
__device__ __forceinline__ void fetch(const void* p, long long row, int type, int first, int step,
                                      int end, Raw<kWide> (&f)[V]) {
  const int size = kWide && type == MOE_READER_TYPE_F32 ? 32 : 16;
  const char* at = static_cast<const char*>(p) + row * (size / 8);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = first + j * step;
    if (v < end) {
      f[j].a = load16(at + (size_t)v * size);
      if constexpr (kWide)
        if (size == 32) f[j].b = load16(at + (size_t)v * size + 16);
    }
  }
}

template <int V, bool kWide>
__device__ __forceinline__ void widen(const Raw<kWide> (&r)[V], int type, float (&f)[V][8]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t w[4] = {r[j].a.x, r[j].a.y, r[j].a.z, r[j].a.w};
    if constexpr (kWide) {
      if (type == MOE_READER_TYPE_F32) {
        const uint32_t u[4] = {r[j].b.x, r[j].b.y, r[j].b.z, r[j].b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[j][i] = __uint_as_float(w[i]);
          f[j][4 + i] = __uint_as_float(u[i]);
        }
        continue;
      }
    }
    if (type == MOE_READER_TYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[j][2 * i] = __uint_as_float(w[i] << 16);
        f[j][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[j][2 * i] = u.x;
        f[j][2 * i + 1] = u.y;
      }
    }
  }
}

// A weight vector's part, converted at once (all rows share it: it is in cache).
template <int V>
__device__ __forceinline__ void weights(const void* p, int type, int first, int step, int end,
                                        float (&f)[V][8]) {
  if (type == MOE_READER_TYPE_F32) {
    Raw<true> r[V];
    fetch<V, true>(p, 0, MOE_READER_TYPE_F32, first, step, end, r);
    widen<V, true>(r, MOE_READER_TYPE_F32, f);
  } else {
    Raw<false> r[V];
    fetch<V, false>(p, 0, type, first, step, end, r);
    widen<V, false>(r, type, f);
  }
}

__device__ __forceinline__ void load8(const void* p, long long at, int type, float (&f)[8]) {
  Raw<true> r[1];
  float g[1][8];
  fetch<1, true>(p, at, type, 0, 0, 1, r);
  widen<1, true>(r, type, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = g[0][i];
}

__device__ __forceinline__ float load1(const void* p, long long at, int type) {
  if (type == MOE_READER_TYPE_F32) return __ldg(static_cast<const float*>(p) + at);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + at);
  return type == MOE_READER_TYPE_BF16 ? __uint_as_float((uint32_t)u << 16)
                                      : __half2float(__ushort_as_half(u));
}

template <int T>
__device__ __forceinline__ void store8_as(void* p, long long at, const float (&f)[8]) {
  if constexpr (T == MOE_READER_TYPE_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == MOE_READER_TYPE_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int V>
__device__ __forceinline__ void store_row(void* p, long long row, int type, int first, int step,
                                          int end, const float (&f)[V][8]) {
  auto go = [&](auto t) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = first + j * step;
      if (v < end) store8_as<decltype(t)::value>(p, row + 8 * v, f[j]);
    }
  };
  if (type == MOE_READER_TYPE_BF16) go(std::integral_constant<int, MOE_READER_TYPE_BF16>{});
  else if (type == MOE_READER_TYPE_F32) go(std::integral_constant<int, MOE_READER_TYPE_F32>{});
  else go(std::integral_constant<int, MOE_READER_TYPE_F16>{});
}

__device__ __forceinline__ void store8(void* p, long long at, int type, const float (&f)[8]) {
  float g[1][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[0][i] = f[i];
  store_row<1>(p, at, type, 0, 0, 1, g);
}

// Sum over the CTA; `slot` alternates so that one barrier is enough.
__device__ __forceinline__ float block_sum(float v, float (*s)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) s[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < warps; ++w) v += s[slot][w];
  return v;
}

constexpr int kThreads = 512;        // at most, of the register kernel
constexpr int kLongThreads = 1024;

// kType: the one 16-bit type of all matrices, or kMixed.
constexpr int kMixed = -1;

template <int V, int kType>
__global__ void __launch_bounds__(kThreads)
residual_norm_kernel(const Args a, float inv_hidden) {
  constexpr bool kWide = kType == kMixed;
  const int h_type = kWide ? a.h_type : kType, y_type = kWide ? a.y_type : kType;
  const int x_type = kWide ? a.x_type : kType, g_type = kWide ? a.gate_type : kType;
  __shared__ float s_sum[2][32];
  const long long row = blockIdx.x;
  const int vecs = a.hidden / 8, first = threadIdx.x, step = blockDim.x;
  const bool gated = a.gate && a.gate_col_stride;
  Raw<kWide> rh[V], ry[V], rg[V];
  fetch<V, kWide>(a.h, row * a.h_stride, h_type, first, step, vecs, rh);
  if (a.y) fetch<V, kWide>(a.y, row * a.y_stride, y_type, first, step, vecs, ry);
  if (gated) fetch<V, kWide>(a.gate, row * a.gate_row_stride, g_type, first, step, vecs, rg);
  float one = a.scale;
  if (a.gate && !gated) one *= load1(a.gate, row * a.gate_row_stride, g_type);
  if (a.post_weight) {
    float z[V][8], ss = 0.f;
    widen<V, kWide>(ry, y_type, z);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (first + j * step < vecs)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += z[j][i] * z[j][i];
    one *= rsqrtf(block_sum(ss, s_sum, 0) * inv_hidden + a.eps);
  }
  // only the raw rows live across the barrier: widening y again is cheaper than
  // the registers that its floats would hold
  float h[V][8], w[V][8];
  widen<V, kWide>(rh, h_type, h);
  if (a.y) {
    float z[V][8];
    widen<V, kWide>(ry, y_type, z);
    if (a.post_weight) {
      weights<V>(a.post_weight, a.weight_type, first, step, vecs, w);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] *= w[j][i];
    }
    if (gated) {
      widen<V, kWide>(rg, g_type, w);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] *= w[j][i];
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] += one * z[j][i];
  }
  if (a.h_out) store_row<V>(a.h_out, row * a.h_out_stride, h_type, first, step, vecs, h);
  if (!a.x) return;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (first + j * step < vecs)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += h[j][i] * h[j][i];
  if (a.pre_weight) weights<V>(a.pre_weight, a.weight_type, first, step, vecs, w);
  const float inv = rsqrtf(block_sum(ss, s_sum, 1) * inv_hidden + a.eps);
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] *= a.pre_weight ? inv * w[j][i] : inv;
  store_row<V>(a.x, row * a.x_stride, x_type, first, step, vecs, h);
}

__global__ void __launch_bounds__(kLongThreads) residual_norm_long_kernel(const Args a) {
  __shared__ float s_sum[2][32];
  const long long row = blockIdx.x;
  const int vecs = a.hidden / 8;
  float inv_y = 1.f, one = a.scale;
  if (a.post_weight) {
    float ss = 0.f;
    for (int v = threadIdx.x; v < vecs; v += kLongThreads) {
      float z[8];
      load8(a.y, row * a.y_stride + 8 * v, a.y_type, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += z[i] * z[i];
    }
    inv_y = rsqrtf(block_sum(ss, s_sum, 0) / (float)a.hidden + a.eps);
  }
  if (a.gate && a.gate_col_stride == 0) one *= load1(a.gate, row * a.gate_row_stride, a.gate_type);
  auto joined = [&](int v, float (&h)[8]) {        // h' of one vector
    load8(a.h, row * a.h_stride + 8 * v, a.h_type, h);
    if (!a.y) return;
    float z[8], w[8];
    load8(a.y, row * a.y_stride + 8 * v, a.y_type, z);
    if (a.post_weight) {
      load8(a.post_weight, 8 * v, a.weight_type, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= inv_y * w[i];
    }
    if (a.gate && a.gate_col_stride) {
      load8(a.gate, row * a.gate_row_stride + 8 * v, a.gate_type, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += one * z[i];
  };
  float inv = 1.f;
  if (a.x) {
    float ss = 0.f;
    for (int v = threadIdx.x; v < vecs; v += kLongThreads) {
      float h[8];
      joined(v, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += h[i] * h[i];
    }
    inv = rsqrtf(block_sum(ss, s_sum, 1) / (float)a.hidden + a.eps);
  }
  for (int v = threadIdx.x; v < vecs; v += kLongThreads) {
    float h[8], w[8];
    joined(v, h);        // before h_out, which may be h, is written
    if (a.h_out) store8(a.h_out, row * a.h_out_stride + 8 * v, a.h_type, h);
    if (!a.x) continue;
    if (a.pre_weight) load8(a.pre_weight, 8 * v, a.weight_type, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] *= a.pre_weight ? inv * w[i] : inv;
    store8(a.x, row * a.x_stride + 8 * v, a.x_type, h);
  }
}

bool float_type(int t) {
  return t == MOE_READER_TYPE_F32 || t == MOE_READER_TYPE_BF16 || t == MOE_READER_TYPE_F16;
}
long long bytes_of(int t) { return t == MOE_READER_TYPE_F32 ? 4 : 2; }

// A matrix that the kernel reads or writes in vectors of eight elements.
bool rows_fit(const void* p, int type, int64_t stride) {
  return float_type(type) && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

// Rows of `width` bytes, `step` bytes apart.
struct Bytes {
  const void* at;
  long long step, width;
  int rows;
};
Bytes matrix(const void* p, int type, int64_t stride, int rows, int hidden) {
  return {p, stride * bytes_of(type), hidden * bytes_of(type), rows};
}

// Whether two of them share a byte: by their outer extents, but column slices of
// one buffer do not.
bool overlap(const Bytes& p, const Bytes& q) {
  if (!p.at || !q.at) return false;
  auto extent = [](const Bytes& m, long long& lo, long long& hi) {
    const long long last = (m.rows - 1) * m.step;
    lo = static_cast<long long>(reinterpret_cast<uintptr_t>(m.at)) + std::min(last, 0LL);
    hi = static_cast<long long>(reinterpret_cast<uintptr_t>(m.at)) + std::max(last, 0LL) + m.width;
  };
  long long a0, a1, b0, b1;
  extent(p, a0, a1);
  extent(q, b0, b1);
  if (a0 >= b1 || b0 >= a1) return false;
  if (p.step == q.step && p.step > 0) {
    const long long apart = ((b0 - a0) % p.step + p.step) % p.step;
    if (apart >= p.width && apart + q.width <= p.step) return false;
  }
  return true;
}

int check(const Args& a) {
  if (a.rows < 0 || a.hidden < 8 || a.hidden > 65536 || a.hidden % 8) return MOE_READER_EINVAL;
  if (a.rows == 0) return MOE_READER_OK;
  if (!a.h || (!a.h_out && !a.x)) return MOE_READER_EINVAL;
  if (!rows_fit(a.h, a.h_type, a.h_stride)) return MOE_READER_EINVAL;
  if (a.y && !rows_fit(a.y, a.y_type, a.y_stride)) return MOE_READER_EINVAL;
  if (a.h_out && !rows_fit(a.h_out, a.h_type, a.h_out_stride)) return MOE_READER_EINVAL;
  if (a.x && !rows_fit(a.x, a.x_type, a.x_stride)) return MOE_READER_EINVAL;
  if ((a.post_weight || a.pre_weight) && !float_type(a.weight_type)) return MOE_READER_EINVAL;
  if (reinterpret_cast<uintptr_t>(a.post_weight) % 16 ||
      reinterpret_cast<uintptr_t>(a.pre_weight) % 16)
    return MOE_READER_EINVAL;
  if (!a.y && (a.post_weight || a.gate)) return MOE_READER_EINVAL;
  if (a.gate) {
    if (!float_type(a.gate_type)) return MOE_READER_EINVAL;
    if (a.gate_col_stride == 1) {
      if (!rows_fit(a.gate, a.gate_type, a.gate_row_stride)) return MOE_READER_EINVAL;
    } else if (a.gate_col_stride != 0 ||
               reinterpret_cast<uintptr_t>(a.gate) % bytes_of(a.gate_type)) {
      return MOE_READER_EINVAL;
    }
  }
  const Bytes h = matrix(a.h, a.h_type, a.h_stride, a.rows, a.hidden);
  const Bytes y = matrix(a.y, a.y_type, a.y_stride, a.rows, a.hidden);
  const Bytes h_out = matrix(a.h_out, a.h_type, a.h_out_stride, a.rows, a.hidden);
  const Bytes x = matrix(a.x, a.x_type, a.x_stride, a.rows, a.hidden);
  const Bytes gate = matrix(a.gate, a.gate_type, a.gate_row_stride, a.rows,
                            a.gate_col_stride ? a.hidden : 1);
  const Bytes post = matrix(a.post_weight, a.weight_type, 0, 1, a.hidden);
  const Bytes pre = matrix(a.pre_weight, a.weight_type, 0, 1, a.hidden);
  // an output's rows are its own
  for (const Bytes* o : {&h_out, &x})
    if (o->at && a.rows > 1 && std::abs(o->step) < o->width) return MOE_READER_EINVAL;
  // h' may replace h in place; any other overlap would be read after a write
  const bool in_place = a.h_out == a.h && a.h_out_stride == a.h_stride;
  if (!in_place && overlap(h, h_out)) return MOE_READER_EINVAL;
  for (const Bytes* in : {&y, &gate, &post, &pre})
    if (overlap(*in, h_out) || overlap(*in, x)) return MOE_READER_EINVAL;
  if (overlap(h, x) || overlap(h_out, x)) return MOE_READER_EINVAL;
  return MOE_READER_OK;
}

// V vectors a thread; 0: the kernel for long rows.
template <int kType>
void launch(const Args& a, int V, cudaStream_t s) {
  const int threads = V ? ((a.hidden / 8 + V - 1) / V + 31) / 32 * 32 : kLongThreads;
  const unsigned rows = (unsigned)a.rows;
  const float inv = 1.f / (float)a.hidden;
  if (V == 1) return residual_norm_kernel<1, kType><<<rows, threads, 0, s>>>(a, inv);
  if (V == 2) return residual_norm_kernel<2, kType><<<rows, threads, 0, s>>>(a, inv);
  if constexpr (kType != kMixed) {
    if (V == 3) return residual_norm_kernel<3, kType><<<rows, threads, 0, s>>>(a, inv);
    if (V == 4) return residual_norm_kernel<4, kType><<<rows, threads, 0, s>>>(a, inv);
  }
  residual_norm_long_kernel<<<rows, threads, 0, s>>>(a);
}

}  // namespace
}  // namespace mr

extern "C" int moe_reader_residual_norm(const moe_reader_residual_norm_args* a, void* stream) {
  if (!a) return MOE_READER_EINVAL;
  const int st = mr::check(*a);
  if (st != MOE_READER_OK || a->rows == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Many rows: about four warps a row (eight with matrices of several types or
  // fp32), so that many rows share an SM and few warps meet at a row's barriers;
  // few rows: one vector a thread, for latency.  Measured, one vector / this
  // rule: 8191 x 2880 bf16 46.3 / 41.8 us (5.6 TB/s), 2048 x 8192 bf16 36.2 /
  // 25.8, 16384 x 2048 fp32 69.3 / 69.3 (6.8 TB/s; four warps: 72.8), 16 x 2048
  // fp32 2.3 (two vectors: 2.4).
  int type = a->h_type;
  if (type == MOE_READER_TYPE_F32 || (a->y && a->y_type != type) || (a->x && a->x_type != type) ||
      (a->gate && a->gate_type != type))
    type = mr::kMixed;
  constexpr int kFew = 2 * 152;        // two CTAs on each of the GB300's SMs
  const bool mixed = type == mr::kMixed, many = a->rows > kFew;
  const int vecs = a->hidden / 8, most = mixed ? 2 : 4, aim = mixed ? 256 : 128;
  const int least = (vecs + mr::kThreads - 1) / mr::kThreads;
  const int V = least > most ? 0 : std::max(least, std::min(many ? (vecs + aim - 1) / aim : 1, most));
  if (mixed) mr::launch<mr::kMixed>(*a, V, s);
  else if (type == MOE_READER_TYPE_BF16) mr::launch<MOE_READER_TYPE_BF16>(*a, V, s);
  else mr::launch<MOE_READER_TYPE_F16>(*a, V, s);
  return cudaGetLastError() == cudaSuccess ? MOE_READER_OK : MOE_READER_ECUDA;
}
