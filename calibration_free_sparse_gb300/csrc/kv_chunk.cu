// Attention of several new tokens per request over the paged cache.
#include <algorithm>
#include <type_traits>

#include "device_util.cuh"
#include "internal.cuh"
#include "kv.cuh"
#include "tc.cuh"

namespace mr {
namespace {

constexpr int kBf16 = MOE_READER_TYPE_BF16, kF16 = MOE_READER_TYPE_F16,
              kE4m3 = MOE_READER_TYPE_E4M3;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int CT>
__device__ __forceinline__ float cell(const void* base, long long at) {
  if constexpr (CT == kE4m3)
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(
        static_cast<const __nv_fp8_storage_t*>(base)[at], __NV_E4M3)));
  else if constexpr (CT == kBf16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  else
    return __half2float(static_cast<const __half*>(base)[at]);
}
template <int QT> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (QT == kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two weights' upper 16 bits, and what that cuts off: both parts above zero for
// a weight above zero, so that infinite values stay infinite.
__device__ __forceinline__ uint32_t cut2(float x, float y, uint32_t& rest) {
  const uint32_t a = max(__float_as_uint(x), 1u) - 1, b = max(__float_as_uint(y), 1u) - 1;
  rest = pack2<kBf16>(x - __uint_as_float(a & 0xffff0000u), y - __uint_as_float(b & 0xffff0000u));
  return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// n / d and the remainder for 0 <= n < 2^31 by a product: the estimate is at
// most one too small.
struct Divisor {
  uint32_t d, m;
};
__host__ __device__ __forceinline__ Divisor divisor(uint32_t d) { return {d, 0xffffffffu / d}; }
__device__ __forceinline__ int quotient(int n, Divisor by, int& rest) {
  uint32_t q = __umulhi((uint32_t)n, by.m), r = (uint32_t)n - q * by.d;
  if (r >= by.d) q++, r -= by.d;
  rest = (int)r;
  return (int)q;
}
__device__ __forceinline__ int quotient(int n, Divisor by) {
  int rest;
  return quotient(n, by, rest);
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

// ---------------------------------------------------------------------------
// Both products run on the tensor core: S = Q K^T with 128 rows (token, head
// of the group) a tile, and O += P V with P read from tensor memory, where it
// replaces S.  A CTA has two row tiles, so that one's softmax runs while the
// other's products do, and both share the keys (heads of 256: one tile, whose S
// has two buffers).  Four warps a row tile: a thread has a row, so maxima and
// sums need no exchange.  Three warps (e4m3: seven) bring pages, one issues
// products.
//
// Measured on a GB300 (the two products of a step of 128 keys and 256 rows are
// 2048 cycles):
//  - 8192 tokens at once, 32 query heads on 4 KV heads of 128, bf16: 350 us, 1.57
//    PFLOP/s (2700 cycles a step: from a tile's logits to its weights 1300, its
//    products, and a third of that under the other tile's).
//  - the same with pages by 16-byte copies of three warps 715, with products
//    issued by a lane of a divergent warp (operands moved to uniform registers
//    one by one) 490, without packed pairs and handing weights over in halves 420.
//  - 500 tokens over 32768 of an e4m3 cache, 32/8 heads: 291 us (widening).
//  - 5 tokens of 16 requests, 32/4 heads, up to 4096 tokens: 35 us, 73 MB; 4 of
//    them are found out by every CTA, 5 the first pages' way, 14 streaming, 6 the
//    joining of rows.
// ---------------------------------------------------------------------------
constexpr int kMaxItems = kChunkItems;   // that are dealt by steps
constexpr int kItemCost = 2;          // of an item beside its steps, in steps

template <int D, int CT = kBf16> struct ChunkShape {
  static constexpr int kTiles = D <= 128 ? 2 : 1;        // row tiles
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kKeys = D <= 128 ? 128 : 64;      // keys of a step
  static constexpr int kBlocks = D / 64;                 // 128-byte blocks of a row
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kSlotBytes = kKeys * D * 2;       // keys or values of a step
  // e4m3: two slots' worth of bytes as they come, so one slot of 16-bit values less
  static constexpr int kSlots = (D == 64 ? 8 : 4) - (CT == kE4m3);
  static constexpr int kRaw = CT == kE4m3 ? 2 : 0;
  // Warps: eight of softmax, the loaders, one that issues products.  Three
  // loaders leave 168 registers a thread, so that softmax holds a row's logits
  // of a step; seven (e4m3: one asks, six widen; with three, widening took twice
  // a step's products) leave 128, and it reads them twice.
  static constexpr int kLoaders = CT == kE4m3 ? 7 : 3;
  static constexpr int kThreads = 32 * (9 + kLoaders);
  static constexpr int kHeld = CT == kE4m3 && kKeys == 128 ? 64 : kKeys;   // logits held
  static constexpr size_t kSmem =
      kQBytes + (size_t)kSlots * kSlotBytes + kRaw * (kSlotBytes / 2) + 1024;
  // tensor memory: two S, then O
  static constexpr int kO = 2 * kKeys;
};

struct ChunkCall {
  moe_reader_kv_chunk_args a;
  const char* k;
  const char* v;
  const float* k_scale;
  const float* v_scale;
  float* part_o;             // [CTA][2][D / 4][kRows][4]
  float* part_ml;            // [CTA][2][2][kRows]
  uint32_t* arrived;         // [item]
  uint32_t* err;
  int heads, kv_heads, shift, pool;
  int rows;                  // of an item: whole groups of heads
  Divisor by_group, by_kv;   // query heads per KV head, KV heads
  int wide;                  // q can be read 16 bytes at a time
  int stall;                 // wait for a product that was never issued
  int mapped;                // q_map holds; else threads read q
  CUtensorMap q_map, k_map, v_map;      // k, v: of 16-bit caches
};

// Part of an item: the rows [row, row + rows) of a request's (token, head of
// the group) list, one KV head, the steps [step, last) of its keys.
struct alignas(16) Piece {
  Span sp;
  int request, head, row, rows;
  int p0, p1;                // positions of the first and the last row
  int lo, hi;                // keys that some row sees
  int base;                  // key of step 0
  int step, last;
  int item, index, count;    // index-th of the item's `count` pieces
  int owner;                 // the CTA of its first piece
  int turn;                  // of the CTA's pieces that have keys
};

template <int D>
__device__ __forceinline__ void item_range(const ChunkCall& c, Piece& x) {
  using S = ChunkShape<D>;
  const int before = x.sp.len - x.sp.tokens;
  x.p0 = before + quotient(x.row, c.by_group);
  x.p1 = before + quotient(x.row + x.rows - 1, c.by_group);
  x.lo = c.a.window ? max(0, x.p0 + 1 - c.a.window) : 0;
  x.hi = (int)min((long long)x.p1 + 1, (long long)c.a.width << c.shift);
  // steps begin at a page, or inside one at a multiple of theirs
  x.base = x.lo & -min(1 << c.shift, S::kKeys);
  x.step = 0;
  x.last = x.hi > x.lo ? (x.hi - x.base + S::kKeys - 1) / S::kKeys : 0;
}

// What every role looks its pieces up in.
struct Work {
  int blocks[kMaxRequests + 1];       // a request's first block of rows
  int first[kMaxRequests], tokens[kMaxRequests], len[kMaxRequests];
  long long at[kMaxItems + 1];        // steps and costs before an item, where they are dealt
};

// Item i: block of rows and KV head; the longest rows of a request first.
template <int D>
__device__ __forceinline__ Piece item_at(const ChunkCall& c, const Work& w, int i) {
  Piece x;
  const int b = quotient(i, c.by_kv, x.head);
  int lo = 0, hi = c.a.requests - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (w.blocks[mid] <= b) lo = mid; else hi = mid - 1;
  }
  x.sp = {w.first[lo], w.tokens[lo], w.len[lo]};
  x.request = lo;
  x.row = (w.blocks[lo + 1] - 1 - b) * c.rows;
  x.rows = min(c.rows, x.sp.tokens * (int)c.by_group.d - x.row);
  x.item = i;
  x.index = 0;
  x.count = 1;
  x.owner = 0;
  item_range<D>(c, x);
  return x;
}

// Whether some row of the piece does not see all of a step's keys.
template <int D>
__device__ __forceinline__ bool partial_step(const ChunkCall& c, const Piece& x, int k0) {
  const int lo = c.a.window ? max(0, x.p1 + 1 - c.a.window) : 0, hi = min(x.p0 + 1, x.hi);
  return k0 < lo || k0 + ChunkShape<D>::kKeys > hi;
}

__device__ __forceinline__ void put_smem(uint32_t at, uint32_t x, uint32_t y, uint32_t z,
                                         uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
               :: "r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 get_smem(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// One row without the tensor core, for pieces whose masked values are not
// finite (0 times those is not 0): a warp, lanes over coordinates.  Same
// reference and scaling as the tensor path's.
template <int D, int CT, int QT>
__device__ __noinline__ void plain_row(const ChunkCall& c, const Piece& x, int row, float factor,
                                       int klo, int khi, float lift, float* o, float& m, float& l) {
  int head;
  const int lane = threadIdx.x & 31, t = x.sp.first + quotient(row, c.by_group, head);
  head += x.head * c.by_group.d;
  const long long q = t * c.a.q_token_stride + head * c.a.q_head_stride + lane;
  const float sign = c.a.scale < 0.f ? -1.f : 1.f;
  m = -INFINITY;
  l = 0.f;
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j = klo; j < khi; ++j) {
    const int page = __ldg(c.a.table + (size_t)x.request * c.a.width + (j >> c.shift));
    if ((unsigned)page >= (unsigned)c.pool) continue;
    const long long at =
        ((((long long)page * c.kv_heads + x.head) << c.shift) + (j & ((1 << c.shift) - 1))) * D +
        lane;
    float s = 0.f;
    for (int i = 0; i < D / 32; ++i)
      s += sign * cell<QT>(c.a.q, q + 32 * i) * cell<CT>(c.k, at + 32 * i);
    s = warp_sum(s) * factor;
    const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
    const float f = exp2_fast(m - ref), p = exp2_fast(s - ref + lift);
    m = top;
    l = l * f + p;
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * f + p * cell<CT>(c.v, at + 32 * i);
  }
}

// Eight values of 16 bits, any of which is infinite or NaN.
template <int QT> __device__ __forceinline__ bool odd8(uint4 v) {
  constexpr uint32_t e = QT == kBf16 ? 0x7f80u : 0x7c00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    odd |= (w[i] & e) == e || (w[i] >> 16 & e) == e;
  return odd;
}

// Two e4m3 values in fp16, which holds them all.
__device__ __forceinline__ uint32_t widen2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffff), __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Of four lanes with a row each, four pieces long: lane i gets piece i of every
// row (in order), so that the four store a row's 64 bytes together.
__device__ __forceinline__ void exchange4(uint4 (&v)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & o) continue;
      // pieces i (kept by the lower lane) and i + o
      uint4 &a = v[i], &b = v[i + o];
      const uint4 give = up ? a : b;
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, o);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, o);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, o);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, o);
      if (up) a = got; else b = got;
    }
  }
}

// What a row adds up to with its sink: the factor of its sums, lse.
struct Close {
  float scale, lse;
};
__device__ __forceinline__ Close close_row(float m, float l, float sink, float lift) {
  sink *= kLog2e;
  const float top = fmaxf(m, sink);
  if (top == -INFINITY && !(l != l)) return {0.f, -INFINITY};
  if (sink == INFINITY) return {0.f, INFINITY};
  const float f = m == -INFINITY ? 0.f : exp2_fast(m - top);
  const float all = l * f + exp2_fast(sink - top + lift);
  return {f / all, (top - lift + log2f(all)) * kLn2};
}

template <int D, int CT, int QT>
__global__ void __launch_bounds__((ChunkShape<D, CT>::kThreads), 1)
chunk_kernel(const __grid_constant__ ChunkCall c) {
  using S = ChunkShape<D, CT>;
  // The products' type: the cache's, fp16 for e4m3 (the one conversion that
  // there is an instruction for; widening to bf16 took twice the issue slots and
  // left the weights three bits less).  Queries in bf16 are brought to fp16 by
  // a power of two per row that puts the largest near 2^15: exact down to 2^-30
  // of it.
  constexpr int MT = CT == kE4m3 ? kF16 : QT;
  constexpr bool kScaled = CT == kE4m3 && QT == kBf16;
  // bf16 weights of items of few rows, whose products wait for their keys anyway,
  // go in two parts: what the first cut off, in a second product of the same
  // type (16 bits of a weight instead of 8: the output's error is its own
  // rounding).  Where products bound the time they would take half as long again.
  constexpr bool kFine = CT == kBf16;
  constexpr int kFineRows = S::kTiles == 2 ? 128 : 64;
  constexpr float kLift = MT == kF16 ? 11.f : 0.f;     // fp16 weights reach down to 2^-35
  constexpr float kSlack = MT == kF16 ? 4.f : 8.f;     // how far a logit may pass the reference
  extern __shared__ char raw[];
  __shared__ Work work_list;
  __shared__ Piece s_piece[4];
  __shared__ uint64_t s_bar[4 * S::kSlots + 22];
  __shared__ float s_twin[2][128];
  __shared__ float s_q_scale[2][kScaled ? S::kRows : 1];    // by piece with keys, in turn
  // by piece with keys and by step, in turn: loaders are at most two pieces and
  // kSlots / 2 + 2 steps ahead of softmax
  __shared__ volatile uint32_t s_odd[4], s_bad[8];
  __shared__ uint32_t s_tmem, s_last;
  __shared__ volatile uint32_t s_quit;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int grid = gridDim.x;
  constexpr int kWideners = S::kLoaders - 1;
  const uint32_t q_at = (tc::smem_at(raw) + 1023) & ~1023u, kv_at = q_at + S::kQBytes;
  const uint32_t bars = tc::smem_at(s_bar);
  auto slot_full = [&](int s) { return bars + 8 * s; };
  auto slot_free = [&](int s) { return bars + 8 * (S::kSlots + s); };
  auto cleaned = [&](int s) { return bars + 8 * (2 * S::kSlots + s); };
  auto landed = [&](int s) { return bars + 8 * (3 * S::kSlots + s); };
  auto raw_full = [&](int i) { return bars + 8 * (2 * S::kSlots + i); };   // e4m3: in their place
  auto raw_free = [&](int i) { return bars + 8 * (2 * S::kSlots + 2 + i); };
  const uint32_t more = bars + 32 * S::kSlots;
  auto s_full = [&](int t) { return more + 8 * t; };          // logits of a tile are there
  auto p_full = [&](int t) { return more + 16 + 8 * t; };     // its weights are
  auto o_full = [&](int t) { return more + 32 + 8 * t; };     // they are added up
  const uint32_t q_full = more + 48, q_free = more + 56, join = more + 64, drained = more + 72;
  auto p_half = [&](int t) { return more + 80 + 8 * t; };     // the first half of its weights
  const uint32_t twin = more + 96, twin_done = more + 104;   // the second four's sums, taken
  auto piece_full = [&](int i) { return more + 112 + 8 * i; };
  auto piece_free = [&](int i) { return more + 144 + 8 * i; };

  if (tid == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      tc::bar_init(slot_full(s), CT == kE4m3 ? kWideners * 32 : 1);
      tc::bar_init(slot_free(s), 1);
      if (CT != kE4m3) {
        tc::bar_init(cleaned(s), 64);
        tc::bar_init(landed(s), 1);
      }
    }
    for (int i = 0; i < S::kRaw; ++i) {
      tc::bar_init(raw_full(i), 1);
      tc::bar_init(raw_free(i), kWideners * 32);
    }
    for (int t = 0; t < 2; ++t) {
      tc::bar_init(s_full(t), 1);
      tc::bar_init(p_full(t), 128);
      tc::bar_init(p_half(t), 128);
      tc::bar_init(o_full(t), 1);
    }
    tc::bar_init(q_full, c.mapped ? 1 : CT == kE4m3 ? 32 * S::kLoaders : 64);
    tc::bar_init(q_free, 1);
    tc::bar_init(join, 256);
    tc::bar_init(drained, 1);
    for (int i = 0; i < 4; ++i) {
      tc::bar_init(piece_full(i), 1);
      tc::bar_init(piece_free(i), 8 + S::kLoaders);      // all warps but the giver
    }
    tc::bar_init(twin, 128);
    tc::bar_init(twin_done, 128);
    for (int i = 0; i < 4; ++i) s_odd[i] = 0;
    s_quit = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  constexpr int kProducts = 8 + S::kLoaders;
  if (wid == kProducts) tc::tmem_alloc(tc::smem_at(&s_tmem), 512);
  if (tid == 32) {
    if (c.mapped) tc::prefetch_map(&c.q_map);
    if (CT != kE4m3) tc::prefetch_map(&c.k_map), tc::prefetch_map(&c.v_map);
  }
  wait_for_earlier_launch();
  let_next_launch_start();

  // ---- what there is to do: every CTA finds it out for itself ----
  uint32_t bad = 0;
  for (int r = tid; r < c.a.requests; r += S::kThreads) {
    const Span sp = span_of(c.a, r, bad);
    if (sp.len > ((long long)c.a.width << c.shift)) bad |= kErrLength;
    work_list.first[r] = sp.first;
    work_list.tokens[r] = sp.tokens;
    work_list.len[r] = sp.len;
    work_list.blocks[r] =
        (int)(((long long)sp.tokens * c.by_group.d + c.rows - 1) / c.rows);
  }
  if (bad && blockIdx.x == 0) atomicOr(c.err, bad);
  __syncthreads();
  if (wid == 0) {
    int sum = 0;
    for (int r0 = 0; r0 <= c.a.requests; r0 += 32) {
      const int r = r0 + lane, n = r < c.a.requests ? work_list.blocks[r] : 0;
      int at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += u;
      }
      if (r <= c.a.requests) work_list.blocks[r] = sum + at - n;
      sum += __shfl_sync(0xffffffffu, at, 31);
    }
  }
  __syncthreads();
  const long long items = (long long)work_list.blocks[c.a.requests] * c.kv_heads;
  // Few items: their steps, one item's after the other's, are dealt to the CTAs
  // in equal shares (whole items left a quarter of them idle towards the
  // end), and what a share cuts is added up.  Many: whole.
  const bool dealt = items <= min(3 * grid, kMaxItems);
  long long all = 0;
  if (dealt) {
    for (int i = tid; i < items; i += S::kThreads) {
      const Piece x = item_at<D>(c, work_list, i);
      work_list.at[i] = x.last - x.step + kItemCost;
    }
    __syncthreads();
    if (wid == 0) {
      long long sum = 0;
      for (int i0 = 0; i0 <= items; i0 += 32) {
        const int i = i0 + lane;
        const long long n = i < items ? work_list.at[i] : 0;
        long long at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += u;
        }
        __syncwarp();
        if (i <= items) work_list.at[i] = sum + at - n;
        sum += __shfl_sync(0xffffffffu, at, 31);
      }
    }
    __syncthreads();
    all = work_list.at[items];
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  // The first loader works a CTA's pieces out, one ahead, and hands them to the
  // other warps in a ring of four (each for itself took a quarter of a short
  // piece's time).
  const long long sharers = min((long long)grid, all / 4 + 1);     // four steps at least
  auto owner_of = [&](long long at) { return (int)(((at + 1) * sharers - 1) / all); };
  long long share_lo = 0, share_hi = 0;
  int next_item = 0;
  if (dealt && wid == 8 && blockIdx.x < sharers) {
    share_lo = blockIdx.x * all / sharers;
    share_hi = (blockIdx.x + 1) * all / sharers;
    int lo = 0, hi = (int)items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (work_list.at[mid] <= share_lo) lo = mid; else hi = mid - 1;
    }
    next_item = lo;
  }
  auto piece_at = [&](int round) {
    Piece x;
    x.rows = 0;
    if (!dealt) {
      // in turn, every other round backwards: a request's items get shorter, so
      // that a CTA's long ones meet its short ones
      const long long i =
          (long long)round * grid + (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
      return i < items ? item_at<D>(c, work_list, (int)i) : x;
    }
    while (next_item < items && work_list.at[next_item] < share_hi) {
      const int i = next_item++;
      const long long at = work_list.at[i];
      const int n = (int)(work_list.at[i + 1] - at) - kItemCost;
      const int from = (int)min(max(share_lo - at, 0LL), (long long)n);
      const int to = (int)min(share_hi - at, (long long)n);
      // (an item without keys is its first owner's)
      if (n > 0 ? from >= to : at < share_lo) continue;
      x = item_at<D>(c, work_list, i);
      if (n > 0) {
        x.owner = owner_of(at);
        x.index = (int)blockIdx.x - x.owner;
        x.count = owner_of(at + n - 1) - x.owner + 1;
        x.last = x.step + to;
        x.step += from;
      }
      break;
    }
    return x;
  };
  int turns = 0;                          // the giver's
  auto give = [&](int round) {
    if (!tc::bar_wait(piece_free(round & 3), (round >> 2 & 1) ^ 1, &s_quit)) return false;
    if (lane == 0) {
      Piece x = piece_at(round);
      x.turn = turns;
      turns += x.rows > 0 && x.step < x.last;
      s_piece[round & 3] = x;
      tc::bar_arrive(piece_full(round & 3));
    }
    __syncwarp();
    return true;
  };
  auto take = [&](int round) {
    return tc::bar_wait(piece_full(round & 3), round >> 2 & 1, &s_quit) &&
           s_piece[round & 3].rows > 0;
  };
  auto leave = [&](int round) {
    __syncwarp();
    if (lane == 0) tc::bar_arrive(piece_free(round & 3));
  };

  if (wid >= 8 && wid < kProducts) {
    // ------------------------------------------------------------------
    // loaders
    // ------------------------------------------------------------------
    // 16-bit caches: one warp brings pages by tensor copies, two the queries,
    // and these clear values that are in a page but not there (a page ends
    // inside the step, or is gone).  e4m3: one asks for bytes, six widen them.
    constexpr bool kCopies = CT != kE4m3;
    const int who = wid - (kCopies ? 9 : 8);
    constexpr int warps = S::kLoaders - kCopies;
    int s = 0;
    uint32_t phase = 1, q_phase = 1, work = 0, steps = 0, err = 0;
    uint32_t cleared = 0, clear_phase = 0;     // a bit per slot
    uint32_t raw_asked = 0;
    int issued = 0;
    // queries of a piece: blocks of 64 coordinates, each with all rows
    auto queries = [&](const Piece& x) {
      if (c.mapped) {
        if (who == 0) {
          if (!tc::bar_wait(q_free, q_phase, &s_quit)) return false;
          q_phase ^= 1;
          const int first = x.sp.first + quotient(x.row, c.by_group);
          if (tc::elected()) {
            tc::bar_expect(q_full, S::kBlocks * c.rows * 128);
            for (int b = 0; b < S::kBlocks; ++b)
              tc::load_box(q_at + b * S::kRows * 128, &c.q_map, b * 64, x.head * c.by_group.d,
                           first, q_full);
          }
          __syncwarp();
        }
        return true;
      }
      if (!tc::bar_wait(q_free, q_phase, &s_quit)) return false;
      q_phase ^= 1;
      const int piece = lane & 7;
      const uint16_t flip = c.a.scale < 0.f ? 0x8000 : 0;
      if constexpr (kScaled) {
        const int turn = x.turn & 1;
#pragma unroll 1
        for (int r = who * 4 + (lane >> 3); r < S::kRows; r += warps * 4) {
          const bool in = r < x.rows;
          int g;
          const int t = x.sp.first + quotient(x.row + r, c.by_group, g);
          const long long at = in ? t * c.a.q_token_stride +
                                        (int)(x.head * c.by_group.d + g) * c.a.q_head_stride +
                                        piece * 8
                                  : 0;
          const uint16_t* from = static_cast<const uint16_t*>(c.a.q) + at;
          uint4 v[S::kBlocks];
          float top = 0.f;
#pragma unroll
          for (int b = 0; b < S::kBlocks; ++b) {
            v[b] = make_uint4(0, 0, 0, 0);
            if (in && c.wide) {
              v[b] = __ldg(reinterpret_cast<const uint4*>(from + b * 64));
            } else if (in) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)__ldg(from + b * 64 + 2 * i) |
                       (uint32_t)__ldg(from + b * 64 + 2 * i + 1) << 16;
              v[b] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // (the powers and their inverses are normal numbers)
          const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127) - 14;
          const float by = two_to(-e) * (flip ? -1.f : 1.f);
          int cut = 0, large = 0;
          if (piece == 0) s_q_scale[turn][r] = two_to(e);
#pragma unroll
          for (int b = 0; b < S::kBlocks; ++b) {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float lo = bf16_lo(w[i]) * by, hi = bf16_hi(w[i]) * by;
              o[i] = pack2<kF16>(lo, hi);
              const float2 is = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
              cut |= (is.x != lo && lo == lo) | (is.y != hi && hi == hi);
              large += (fabsf(lo) >= 0.00390625f) + (fabsf(hi) >= 0.00390625f);
            }
            put_smem(q_at + b * S::kRows * 128 + tc::swizzled(r, piece), o[0], o[1], o[2], o[3]);
          }
          // bits lost far below the largest coordinate count where hardly any
          // other is near it: such pieces go row by row
          large += cut << 16;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) large += __shfl_xor_sync(0xffffffffu, large, o);
          if (large >> 16 && (large & 0xffff) < D / 8) s_odd[(x.turn + 1) & 3] = x.turn + 1;
        }
        tc::publish_smem();
        tc::bar_arrive(q_full);
        return true;
      }
      for (int r = who * 4 + (lane >> 3); r < S::kRows; r += warps * 4) {
        const bool in = r < x.rows;
        int g;
        const int t = x.sp.first + quotient(x.row + r, c.by_group, g);
        const long long at = in ? t * c.a.q_token_stride +
                                      (int)(x.head * c.by_group.d + g) * c.a.q_head_stride +
                                      piece * 8
                                : 0;
        const uint16_t* from = static_cast<const uint16_t*>(c.a.q) + at;
        const uint32_t to = q_at + tc::swizzled(r, piece);
        for (int b = 0; b < S::kBlocks; ++b) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint16_t e0 = in ? __ldg(from + b * 64 + 2 * i) ^ flip : 0;
            const uint16_t e1 = in ? __ldg(from + b * 64 + 2 * i + 1) ^ flip : 0;
            w[i] = (uint32_t)e0 | (uint32_t)e1 << 16;
          }
          put_smem(to + b * S::kRows * 128, w[0], w[1], w[2], w[3]);
        }
      }
      tc::publish_smem();
      tc::bar_arrive(q_full);
      return true;
    };
    // lane l has the page of keys 16 l.. of a step: -2 not in the pool, -1 out
    // of sight (it may be gone)
    auto page_of = [&](const Piece& x, int step) {
      const int key = x.base + step * S::kKeys + lane * 16;
      if (lane < S::kKeys / 16 && key < x.hi && ((key >> c.shift) + 1) << c.shift > x.lo) {
        const int p =
            __ldg(c.a.table + (size_t)x.request * c.a.width + (key >> c.shift));
        return (unsigned)p < (unsigned)c.pool ? p : -2;
      }
      return -1;
    };
    if constexpr (kCopies) {
      if (wid == 8) {
        const int rows = min(1 << c.shift, S::kKeys), boxes = S::kKeys / rows;
        if (!give(0)) goto loaders_end;
        for (int round = 0; s_piece[round & 3].rows > 0; ++round) {
          if (!give(round + 1)) goto loaders_end;
          const Piece& x = s_piece[round & 3];
          int next = page_of(x, x.step);
          for (int step = x.step; step < x.last; ++step) {
            const int page = next, k0 = x.base + step * S::kKeys;
            if (step + 1 < x.last) next = page_of(x, step + 1);
            const uint32_t lost = __ballot_sync(0xffffffffu, page == -2);
            if (lost) err |= kErrPage;
            if (lane == 0) s_bad[steps & 7] = lost;
            steps++;
            // lane l has box l; pages that are not there are read as zeros
            int from = __shfl_sync(0xffffffffu, page, (lane * rows >> 4) & 31);
            if (from < 0) from = c.pool;
            const bool partial = partial_step<D>(c, x, k0);
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
              if (!tc::bar_wait(slot_free(s), phase, &s_quit)) goto loaders_end;
              // values to be cleared first have a barrier of their own
              const bool clear = kind && partial;
              const uint32_t bar = clear ? landed(s) : slot_full(s);
              if (lane == 0) {
                tc::bar_expect(bar, S::kSlotBytes);
                if (clear) tc::bar_arrive(slot_full(s));
              }
              if (clear) cleared |= 1u << s, clear_phase ^= 1u << s;
              issued++;
              __syncwarp();
              if (lane < boxes) {
                const uint32_t to = kv_at + s * S::kSlotBytes + lane * rows * 128;
#pragma unroll
                for (int b = 0; b < S::kBlocks; ++b)
                  tc::load_box(to + b * S::kKeys * 128, kind ? &c.v_map : &c.k_map, b * 64,
                               k0 & ((1 << c.shift) - 1), x.head, from, bar);
              }
              if (++s == S::kSlots) s = 0, phase ^= 1;
            }
          }
        }
      } else {
        for (int round = 0; take(round); leave(round++)) {
          const Piece& x = s_piece[round & 3];
          if (x.step >= x.last) continue;
          work++;
          if (!queries(x)) goto loaders_end;
          for (int step = x.step; step < x.last; ++step) {
            const int k0 = x.base + step * S::kKeys;
            s = (s + 1) % S::kSlots;
            if (partial_step<D>(c, x, k0)) {
              const int page = page_of(x, step);
              if (!tc::bar_wait(landed(s), clear_phase >> s & 1, &s_quit)) goto loaders_end;
              clear_phase ^= 1u << s;
              bool odd = false;
              // (a short loop: it runs seldom, and code that is not in the
              // instruction cache costs more than its latency)
              const uint32_t at = kv_at + s * S::kSlotBytes;
#pragma unroll 1
              for (int r0 = who * 4; r0 < S::kKeys; r0 += 16) {
                uint4 v[2][S::kBlocks];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int b = 0; b < S::kBlocks; ++b)
                    v[h][b] = get_smem(at + b * S::kKeys * 128 +
                                       tc::swizzled(r0 + 8 * h + (lane >> 3), lane & 7));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int r = r0 + 8 * h + (lane >> 3), key = k0 + r;
                  const bool in = __shfl_sync(0xffffffffu, page, r >> 4) >= 0 && key >= x.lo &&
                                  key < x.hi;
#pragma unroll
                  for (int b = 0; b < S::kBlocks; ++b) {
                    if (in) odd |= odd8<MT>(v[h][b]);
                    else put_smem(at + b * S::kKeys * 128 + tc::swizzled(r, lane & 7), 0, 0, 0, 0);
                  }
                }
              }
              if (odd) s_odd[work & 3] = work;
              tc::publish_smem();
              tc::bar_arrive(cleaned(s));
            }
            s = (s + 1) % S::kSlots;
          }
        }
      }
    } else {
      // The bytes of a step's keys and values come by bulk copies (a page's
      // rows of a head lie on end), two slots' worth under way, and the step
      // after the next's are brought into L2.  Six warps widen them, 16
      // values a thread at a time, to fp16, which holds them exactly.
      constexpr int kRow = D / 16, kSub = 32 / kRow;
      constexpr int kN = (S::kKeys / kSub + kWideners - 1) / kWideners;
      const int piece = lane % kRow, sub = lane / kRow;
      const uint32_t raw_at = kv_at + S::kSlots * S::kSlotBytes;
      const int box = min(1 << c.shift, S::kKeys), boxes = S::kKeys / box;
      uint32_t& asked = raw_asked;
      uint32_t taken = 0;
      // a page's rows of a step: lane l has box l
      auto rows_at = [&](const Piece& x, const char* base, int k0, int p) {
        return base + ((((long long)p * c.kv_heads + x.head) << c.shift) +
                       (k0 & ((1 << c.shift) - 1))) * D;
      };
      auto box_page = [&](int page) {
        return __shfl_sync(0xffffffffu, page, (lane * box >> 4) & 31);
      };
      auto ask = [&](const Piece& x, int kind, int k0, int page) {
        const uint32_t at = asked & 1;
        if (!tc::bar_wait(raw_free(at), (asked >> 1 & 1) ^ 1, &s_quit)) return false;
        const int p = box_page(page);
        const bool mine = lane < boxes && p >= 0;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) tc::bar_expect(raw_full(at), n * box * D);
        __syncwarp();
        if (mine)
          tc::load_bytes(raw_at + at * (S::kSlotBytes / 2) + lane * box * D,
                         rows_at(x, kind ? c.v : c.k, k0, p), box * D, raw_full(at));
        asked++;
        return true;
      };
      auto widen = [&](const Piece& x, int k0, int page, bool hide, bool watch) {
        const uint32_t at = taken & 1;
        if (!tc::bar_wait(raw_full(at), taken >> 1 & 1, &s_quit)) return false;
        if (!tc::bar_wait(slot_free(s), phase, &s_quit)) return false;
        const uint32_t from = raw_at + at * (S::kSlotBytes / 2) + piece * 16;
        const uint32_t to = kv_at + s * S::kSlotBytes + (piece >> 2) * S::kKeys * 128;
        uint32_t odd = 0;
        uint4 v[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i)
          v[i] = get_smem(from + min((i * kWideners + who - 1) * kSub + sub, S::kKeys - 1) * D);
        tc::bar_arrive(raw_free(at));
        if (hide) {
          // rows out of sight, or of pages that are not there
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int r = (i * kWideners + who - 1) * kSub + sub, key = k0 + r;
            const bool in = __shfl_sync(0xffffffffu, page, r >> 4 & 31) >= 0 && key >= x.lo &&
                            key < x.hi;
            if (!in) v[i] = make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= (w[j] & 0x7f7f7f7fu) + 0x01010101u;
          }
        }
        // lanes of odd blocks store their second half first: those of a block lie
        // in the same banks as the other's
        const bool swap = piece >> 2 & 1;
        const int first = (piece & 3) * 2 + swap;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int r = (i * kWideners + who - 1) * kSub + sub;
          if (r >= S::kKeys) break;
          const uint32_t a0 = swap ? v[i].z : v[i].x, a1 = swap ? v[i].w : v[i].y;
          const uint32_t b0 = swap ? v[i].x : v[i].z, b1 = swap ? v[i].y : v[i].w;
          const uint32_t at0 = to + tc::swizzled(r, first), at1 = to + tc::swizzled(r, first ^ 1);
          put_smem(at0, widen2(a0), widen2(a0 >> 16), widen2(a1), widen2(a1 >> 16));
          put_smem(at1, widen2(b0), widen2(b0 >> 16), widen2(b1), widen2(b1 >> 16));
        }
        if (watch && odd & 0x80808080u) s_odd[work & 3] = work;
        taken++;
        tc::publish_smem();
        tc::bar_arrive(slot_full(s));
        if (++s == S::kSlots) s = 0, phase ^= 1;
        return true;
      };
      auto ahead = [&](const Piece& x, int step) {
        return step < x.last ? page_of(x, step) : -1;
      };
      if (wid == 8) {
        if (!give(0)) goto loaders_end;
        for (int round = 0; s_piece[round & 3].rows > 0; ++round) {
          if (!give(round + 1)) goto loaders_end;
          const Piece& x = s_piece[round & 3];
          int page = ahead(x, x.step), next = ahead(x, x.step + 1), far = ahead(x, x.step + 2);
          for (int step = x.step; step < x.last; ++step) {
            const int k0 = x.base + step * S::kKeys, farther = ahead(x, step + 3);
            if (!ask(x, 0, k0, page) || !ask(x, 1, k0, page)) goto loaders_end;
            if (step == x.step && !queries(x)) goto loaders_end;
            const int p = box_page(far);
            if (lane < boxes && p >= 0) {
              tc::prefetch_bytes(rows_at(x, c.k, k0 + 2 * S::kKeys, p), box * D);
              tc::prefetch_bytes(rows_at(x, c.v, k0 + 2 * S::kKeys, p), box * D);
            }
            page = next;
            next = far;
            far = farther;
          }
        }
      } else {
        for (int round = 0; take(round); leave(round++)) {
          const Piece& x = s_piece[round & 3];
          if (x.step >= x.last) continue;
          work++;
          if (!queries(x)) goto loaders_end;
          int page = ahead(x, x.step), next = ahead(x, x.step + 1);
          for (int step = x.step; step < x.last; ++step) {
            const int k0 = x.base + step * S::kKeys, far = ahead(x, step + 2);
            const uint32_t lost = __ballot_sync(0xffffffffu, page == -2);
            if (lost) err |= kErrPage;
            if (wid == 9 && lane == 0) s_bad[steps & 7] = lost;
            steps++;
            // (0 times NaN is not 0: keys' NaN reach the rows that see them)
            const bool hide = lost || partial_step<D>(c, x, k0);
            if (!widen(x, k0, page, hide, false) || !widen(x, k0, page, hide, true))
              goto loaders_end;
            page = next;
            next = far;
          }
        }
      }
    }
  loaders_end:
    // no copy is left under way
    if (c.mapped && who == 0) {
      volatile uint32_t ignore = 0;
      tc::bar_wait(q_full, q_phase, &ignore);
    }
    if (!kCopies && wid == 8) {
      volatile uint32_t ignore = 0;
      for (uint32_t i = raw_asked < 2 ? 0 : raw_asked - 2; i < raw_asked; ++i)
        tc::bar_wait(raw_full(i & 1), i >> 1 & 1, &ignore);
    }
    if (kCopies && wid == 8) {
      for (int i = 0; i < min(issued, S::kSlots); ++i) {
        if (--s < 0) s = S::kSlots - 1, phase ^= 1;
        volatile uint32_t ignore = 0;
        tc::bar_wait(slot_full(s), phase ^ 1, &ignore);
        if (cleared >> s & 1) tc::bar_wait(landed(s), ~clear_phase >> s & 1, &ignore);
      }
    }
    if (err && lane == 0) atomicOr(c.err, err);
  } else if (wid == kProducts) {
    // ------------------------------------------------------------------
    // products
    // ------------------------------------------------------------------
    constexpr uint32_t s_desc = tc::instr<MT == kBf16>(S::kKeys);
    constexpr uint32_t o_desc = tc::instr<MT == kBf16>(D, true);
    int s = 0;
    uint32_t phase = 0, q_phase = 0, p_phase[2] = {0, 0};
    uint32_t clean_phase = 0;                    // a bit per slot
    // a step's values: there, and cleared where they have to be
    auto values_in = [&](const Piece& x, int step) {
      if (CT == kE4m3 || !partial_step<D>(c, x, x.base + step * S::kKeys))
        return tc::bar_wait(slot_full(s), phase, &s_quit);
      const uint32_t want = clean_phase >> s & 1;
      clean_phase ^= 1u << s;
      return tc::bar_wait(cleaned(s), want, &s_quit);
    };
    auto next_slot = [&]() { if (++s == S::kSlots) s = 0, phase ^= 1; };
    // S of a row tile; afterwards up to two barriers more
    auto logits = [&](int tile, int at, int slot, uint32_t then, uint32_t then2) {
      const uint64_t q = tc::desc_k(q_at + (tile << 14));
      const uint64_t k = tc::desc_k(kv_at + slot * S::kSlotBytes);
      const uint32_t d = tmem + at * S::kKeys, bar = s_full(at);
      if (tc::elected()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          tc::mma(d, q + (i >> 2) * S::kRows * 8 + 2 * (i & 3), k + (i >> 2) * S::kKeys * 8 + 2 * (i & 3),
                  s_desc, i > 0);
        tc::commit(bar);
        if (then) tc::commit(then);
        if (then2) tc::commit(then2);
      }
      __syncwarp();
    };
    // O += P V, the first half of the keys as soon as its weights are there
    auto outputs = [&](int tile, int at, int slot, bool first, bool fine, uint32_t then) {
      const uint32_t want = p_phase[at];
      p_phase[at] ^= 1;
      if (!tc::bar_wait(p_half(at), want, &s_quit)) return false;
      tc::fence_after();
      const uint64_t v = tc::desc_mn(kv_at + slot * S::kSlotBytes, S::kKeys * 128);
      const uint32_t d = tmem + S::kO + tile * D, p = tmem + at * S::kKeys, bar = o_full(tile);
      if (tc::elected()) {
#pragma unroll
        for (int i = 0; i < S::kKeys / 32; ++i)
          tc::mma_ta(d, p + i * 8, v + i * 128, o_desc, !first || i > 0);
        if (kFine && fine) {
#pragma unroll
          for (int i = 0; i < S::kKeys / 32; ++i)
            tc::mma_ta(d, p + S::kKeys / 2 + i * 8, v + i * 128, o_desc, true);
        }
      }
      __syncwarp();
      if (!tc::bar_wait(p_full(at), want, &s_quit)) return false;
      tc::fence_after();
      if (tc::elected()) {
#pragma unroll
        for (int i = S::kKeys / 32; i < S::kKeys / 16; ++i)
          tc::mma_ta(d, p + i * 8, v + i * 128, o_desc, true);
        if (kFine && fine) {
#pragma unroll
          for (int i = S::kKeys / 32; i < S::kKeys / 16; ++i)
            tc::mma_ta(d, p + S::kKeys / 2 + i * 8, v + i * 128, o_desc, true);
        }
        tc::commit(bar);
        if (then) tc::commit(then);
      }
      __syncwarp();
      return true;
    };
    bool go = !c.stall || tc::bar_wait(drained, 0, &s_quit);
    for (int round = 0; go && take(round); leave(round++)) {
      const Piece& x = s_piece[round & 3];
      if (x.step >= x.last) continue;
      const int tiles = x.rows > 128 ? 2 : 1, n = x.last - x.step;
      if (!(go = tc::bar_wait(q_full, q_phase, &s_quit))) break;
      q_phase ^= 1;
      if (!(go = tc::bar_wait(slot_full(s), phase, &s_quit))) break;
      tc::fence_after();
      if (S::kTiles == 2 && tiles == 2) {
        for (int t = 0; t < 2; ++t)
          logits(t, t, s, t ? slot_free(s) : 0, t && n == 1 ? q_free : 0);
        next_slot();
        for (int j = 0; go && j < n; ++j) {
          const int v_slot = s;
          if (!(go = values_in(x, x.step + j))) break;
          next_slot();
          if (j + 1 < n && !(go = tc::bar_wait(slot_full(s), phase, &s_quit))) break;
          for (int t = 0; t < 2; ++t) {
            if (!(go = outputs(t, t, v_slot, j == 0, false, t ? slot_free(v_slot) : 0))) break;
            if (j + 1 < n) logits(t, t, s, t ? slot_free(s) : 0, t && j + 2 == n ? q_free : 0);
          }
          if (go && j + 1 < n) next_slot();
        }
      } else {
        // one tile of rows: its steps take the two S in turn, and, where they
        // fit, two O (whose sums softmax joins)
        const int ahead = S::kTiles;
        uint32_t k_phase = phase;
        int k_slot = s, asked = 0;
        auto ask = [&]() {
          logits(0, asked & 1, k_slot, slot_free(k_slot), asked == n - 1 ? q_free : 0);
          asked++;
          for (int i = 0; i < 2; ++i)
            if (++k_slot == S::kSlots) k_slot = 0, k_phase ^= 1;
        };
        ask();
        for (int j = 0; go && j < n; ++j) {
          next_slot();
          // S of the next step, unless its weights are still wanted
          if (asked < n && asked == j + 1) {
            if (!(go = tc::bar_wait(slot_full(k_slot), k_phase, &s_quit))) break;
            tc::fence_after();
            ask();
          }
          if (!(go = values_in(x, x.step + j))) break;
          if (!(go = outputs(ahead == 2 ? j & 1 : 0, j & 1, s, j < ahead, x.rows <= kFineRows,
                              slot_free(s)))) break;
          if (ahead == 2 && asked < n) {
            if (!(go = tc::bar_wait(slot_full(k_slot), k_phase, &s_quit))) break;
            tc::fence_after();
            ask();
          }
          next_slot();
        }
      }
    }
    // no product is left under way
    volatile uint32_t ignore = 0;
    if (tc::elected()) tc::commit(drained);
    __syncwarp();
    tc::bar_wait(drained, 0, &ignore);
  } else {
    // ------------------------------------------------------------------
    // softmax: a thread has a row
    // ------------------------------------------------------------------
    const int tile = wid >> 2, quarter = wid & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_at = tmem + S::kO + tile * D + lanes;
    uint32_t full_phase[2] = {0, 0}, added = 0, join_phase = 0, twin_phase = 0;
    uint32_t work = 0, steps = 0;
    for (int round = 0; take(round); leave(round++)) {
      const Piece& x = s_piece[round & 3];
      const int n = x.last - x.step;
      // One tile of rows: both fours have it, and every other step each.
      const bool twins = S::kTiles == 2 && x.rows <= 128;
      const int r = (twins ? 0 : tile * 128) + quarter * 32 + lane;
      const int first = twins ? tile : 0, stride = twins ? 2 : 1;
      const bool fine = kFine && x.rows <= kFineRows;
      const int own = twins ? (n - tile + 1) >> 1 : tile * 128 < x.rows ? n : 0;   // its steps
      int group_head;
      const int token = quotient(x.row + r, c.by_group, group_head);
      const int pos = x.sp.len - x.sp.tokens + token;
      const int khi = min(pos + 1, x.hi), klo = c.a.window ? max(0, pos + 1 - c.a.window) : 0;
      // logits in powers of two: |scale| (its sign went into q) times log2 e
      float factor = fabsf(c.a.scale) * kLog2e * (c.k_scale ? __ldg(c.k_scale + x.head) : 1.f);
      factor = fmaxf(factor, 1.1754943508222875e-38f);   // 0 times a masked -infinity is NaN
      float m = -INFINITY, l = 0.f;
      float by = factor;
      if (own > 0) {
        // keys that all of the tile's rows see
        const int r0 = twins ? 0 : tile * 128;
        const int t0 = x.sp.len - x.sp.tokens + quotient(x.row + r0, c.by_group);
        const int t1 =
            x.sp.len - x.sp.tokens + quotient(x.row + min(x.rows, r0 + 128) - 1, c.by_group);
        const int clear_lo = c.a.window ? max(0, t1 + 1 - c.a.window) : 0;
        const int clear_hi = min(t0 + 1, x.hi);
        for (int turn = 0; turn < own; ++turn) {
          const int j = first + turn * stride;
          const int at = S::kTiles == 2 ? tile : j & 1;
          const int k0 = x.base + (x.step + j) * S::kKeys;
          if (!tc::bar_wait(s_full(at), full_phase[at], &s_quit)) goto softmax_end;
          full_phase[at] ^= 1;
          tc::fence_after();
          if (kScaled && turn == 0)
            by = fmaxf(factor * s_q_scale[x.turn & 1][r], 1.1754943508222875e-38f);
          const uint32_t s_at = tmem + at * S::kKeys + lanes;
          constexpr int kHeld = S::kHeld;
          uint32_t v[kHeld];
          const uint32_t lost = s_bad[(steps + j) & 7];
          const bool hide = k0 < clear_lo || k0 + S::kKeys > clear_hi || lost;
          // logits i0.. of the step, those out of sight -infinity
          auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kHeld; i += 32) tc::ld32(s_at + i0 + i, v + i);
            tc::ld_wait();
            if (!hide) return;
            // a word of 32 keys' bits at a time
#pragma unroll
            for (int i = 0; i < kHeld; i += 32) {
              const int at0 = i0 + i;
              const int a0 = min(max(klo - k0 - at0, 0), 32), a1 = min(max(khi - k0 - at0, 0), 32);
              uint32_t see = a1 > a0 ? (0xffffffffu >> (32 - (a1 - a0))) << a0 : 0u;
              if (lost >> (at0 >> 4) & 1) see &= 0xffff0000u;
              if (lost >> (at0 >> 4) & 2) see &= 0x0000ffffu;
              if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(see >> e & 1)) v[i + e] = 0xff800000u;
              }
            }
          };
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i0 = 0; i0 < S::kKeys; i0 += kHeld) {
            fetch(i0);
#pragma unroll
            for (int i = 0; i < kHeld; i += 4) {
              top[0] = max3(top[0], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
              top[1] = max3(top[1], __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            }
          }
          const float high = fmaxf(top[0], top[1]) * by;
          const bool moves = high > m + kSlack;
          if (__any_sync(0xffffffffu, moves)) {
            // the reference follows the maximum (itself: the weight of a lone key
            // is a power of two, and its value comes out as it is); what is
            // added up so far follows it
            const float f = moves ? exp2_fast(m - high) : 1.f;
            if (moves) m = high;
            l *= f;
            if (turn > 0) {
              // (two tiles: S is made behind the products before it)
              if (S::kTiles == 1 && !tc::bar_wait(o_full(0), (added + turn - 1) & 1, &s_quit))
                goto softmax_end;
              tc::fence_after();
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                uint32_t o[16];
                tc::ld16(o_at + i, o);
                tc::ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc::st16(o_at + i, o);
              }
            }
          }
          const float bias = kLift - (m == -INFINITY ? 0.f : m);
          const uint64_t factors = pair(by, by), biases = pair(bias, bias);
          uint64_t add[2] = {0, 0};
          auto weigh = [&](auto parts) {
            constexpr bool kParts = decltype(parts)::value;
#pragma unroll
            for (int i = 0; i < S::kKeys; i += 32) {
              if (kHeld < S::kKeys && i % kHeld == 0) fetch(i);
              uint32_t w[16], rest[kParts ? 16 : 1];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const int at0 = i % kHeld + e;
                float x0, x1;
                unpair(fma_pair(pair(__uint_as_float(v[at0]), __uint_as_float(v[at0 + 1])), factors,
                                biases), x0, x1);
                x0 = exp2_fast(x0);
                x1 = exp2_fast(x1);
                add[e >> 1 & 1] = add_pair(add[e >> 1 & 1], pair(x0, x1));
                if constexpr (kParts) w[e / 2] = cut2(x0, x1, rest[e / 2]);
                else w[e / 2] = pack2<MT>(x0, x1);
              }
              tc::st16(s_at + i / 2, w);
              if constexpr (kParts) tc::st16(s_at + S::kKeys / 2 + i / 2, rest);
              if (i + 32 == S::kKeys / 2) {
                // the first half can be multiplied
                tc::st_wait();
                tc::fence_before();
                tc::bar_arrive(p_half(at));
              }
            }
          };
          if (kFine && fine) weigh(std::bool_constant<kFine>());
          else weigh(std::false_type());
          float l0, l1;
          unpair(add_pair(add[0], add[1]), l0, l1);
          l += l0 + l1;
          tc::st_wait();
          tc::fence_before();
          tc::bar_arrive(p_full(at));
        }
        added += own;
        if (S::kTiles == 1 && own > 1 && !tc::bar_wait(o_full(0), added & 1, &s_quit)) goto softmax_end;
        if (!tc::bar_wait(o_full(tile), (added - 1) & 1, &s_quit)) goto softmax_end;
        tc::fence_after();
      }
      steps += n;
      work += n > 0;
      // partial results: a share begins and ends inside an item at most
      const int part_slot = 2 * (int)blockIdx.x + (x.index == 0);
      const bool odd = n > 0 && s_odd[work & 3] == work;
      const bool whole = x.count == 1;
      const float v_scale = c.v_scale ? __ldg(c.v_scale + x.head) : 1.f;
      const bool joined = twins && n > 1;
      float f0 = 1.f, f1 = 0.f;
      if (joined) {
        // the second four's sums go to the first
        if (tile == 1) {
          s_twin[0][r] = m;
          s_twin[1][r] = l;
          tc::fence_before();
          tc::bar_arrive(twin);
          if (!tc::bar_wait(twin_done, twin_phase, &s_quit)) goto softmax_end;
        } else {
          if (!tc::bar_wait(twin, twin_phase, &s_quit)) goto softmax_end;
          tc::fence_after();
          const float m1 = s_twin[0][r], l1 = s_twin[1][r];
          const float both = fmaxf(m, m1), ref = both == -INFINITY ? 0.f : both;
          f0 = exp2_fast(m - ref);
          f1 = exp2_fast(m1 - ref);
          l = l * f0 + l1 * f1;
          m = both;
        }
        twin_phase ^= 1;
      }
      const bool mine = twins ? tile == 0 : tile * 128 < x.rows;
      if (mine && !odd) {
        const bool in = r < x.rows;
        const int head = x.head * c.by_group.d + group_head;
        const long long line = (long long)(x.sp.first + token) * c.heads + head;
        // 32 columns of the row's sums
        auto sums = [&](int i, float (&o)[32]) {
          uint32_t u[32];
          tc::ld32(o_at + i, u);
          tc::ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(u[e]);
          if (joined) {
            tc::ld32(o_at + D + i, u);
            tc::ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + __uint_as_float(u[e]) * f1;
          }
        };
        if (whole) {
          const float sink = in && c.a.sinks ? __ldg(c.a.sinks + head) : -INFINITY;
          const Close z = close_row(m, l, sink, kLift);
          const float f = z.scale * v_scale;
          if (in && c.a.lse) c.a.lse[line] = z.lse;
          // four lanes store four rows, one after the other, 64 bytes at a time
          // (a lane for itself would touch 32 lines a store)
          const long long mine_at = in ? line * D : -1;
          long long at[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            at[e] = __shfl_sync(0xffffffffu, mine_at, (lane & ~3) + e);
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            float o[32];
            sums(i, o);
            uint4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e].x = pack2<QT>(o[8 * e] * f, o[8 * e + 1] * f);
              w[e].y = pack2<QT>(o[8 * e + 2] * f, o[8 * e + 3] * f);
              w[e].z = pack2<QT>(o[8 * e + 4] * f, o[8 * e + 5] * f);
              w[e].w = pack2<QT>(o[8 * e + 6] * f, o[8 * e + 7] * f);
              if (z.scale == 0.f) w[e] = make_uint4(0, 0, 0, 0);
            }
            exchange4(w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at[e] >= 0)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.a.out) + at[e] + i +
                                          (lane & 3) * 8) = w[e];
          }
        } else {
          // four columns of all rows lie together
          float4* part = reinterpret_cast<float4*>(c.part_o) + (size_t)part_slot * S::kRows * D / 4 + r;
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            float o[32];
            sums(i, o);
            if (in) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                part[(i + e) / 4 * S::kRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (in) {
            float* ml = c.part_ml + (size_t)part_slot * 2 * S::kRows + r;
            ml[0] = m;
            ml[S::kRows] = l;
          }
        }
        tc::fence_before();
      } else if (mine) {
        // row by row: the warp's 32 rows
        for (int i = 0; i < 32; ++i) {
          const int rr = r - lane + i, one = x.row + rr;
          if (rr >= x.rows) break;
          int g;
          const int t = quotient(one, c.by_group, g);
          const int p = x.sp.len - x.sp.tokens + t;
          const int h1 = min(min(p + 1, x.hi), x.base + x.last * S::kKeys);
          const int h0 = max(c.a.window ? max(0, p + 1 - c.a.window) : 0,
                             x.base + x.step * S::kKeys);
          float o[D / 32], m1, l1;
          plain_row<D, CT, QT>(c, x, one, factor, h0, h1, kLift, o, m1, l1);
          const int head = x.head * c.by_group.d + g;
          const long long line = (long long)(x.sp.first + t) * c.heads + head;
          if (whole) {
            const float sink = c.a.sinks ? __ldg(c.a.sinks + head) : -INFINITY;
            const Close z = close_row(m1, l1, sink, kLift);
            if (lane == 0 && c.a.lse) c.a.lse[line] = z.lse;
            for (int e = 0; e < D / 32; ++e) {
              const float y = z.scale == 0.f ? 0.f : o[e] * z.scale * v_scale;
              static_cast<uint16_t*>(c.a.out)[line * D + lane + 32 * e] =
                  (uint16_t)pack2<QT>(y, 0.f);
            }
          } else {
            for (int e = 0; e < D / 32; ++e)
              c.part_o[(((size_t)part_slot * D / 4 + (lane + 32 * e) / 4) * S::kRows + rr) * 4 +
                       (lane & 3)] = o[e];
            if (lane == 0) {
              float* ml = c.part_ml + (size_t)part_slot * 2 * S::kRows + rr;
              ml[0] = m1;
              ml[S::kRows] = l1;
            }
          }
        }
      }
      if (joined && tile == 0) tc::bar_arrive(twin_done);
      if (!whole) {
        // the last piece of an item to arrive adds them up, in order
        __threadfence();
        tc::bar_arrive(join);
        if (!tc::bar_wait(join, join_phase, &s_quit)) goto softmax_end;
        join_phase ^= 1;
        if (tid == 0) {
          const uint32_t before = atomicAdd(c.arrived + x.item, 1);
          s_last = before == (uint32_t)x.count - 1;
          if (s_last) c.arrived[x.item] = 0;
          __threadfence();
        }
        tc::bar_arrive(join);
        if (!tc::bar_wait(join, join_phase, &s_quit)) goto softmax_end;
        join_phase ^= 1;
        if (s_last) {
          __threadfence();
          // a lane has a row, a warp some columns of 32 rows
          constexpr int kCols = D / 8;
          const int col = wid * kCols;
          for (int r0 = 0; r0 < x.rows; r0 += 32) {
            const bool in = r0 + lane < x.rows;
            const int rr = min(r0 + lane, x.rows - 1);
            float top = -INFINITY, all = 0.f, o[kCols];
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[e] = 0.f;
#pragma unroll 2
            for (int i = 0; i < x.count; ++i) {
              const size_t slot = 2 * (x.owner + i) + (i == 0);
              const float* ml = c.part_ml + slot * 2 * S::kRows + rr;
              const float mi = __ldcg(ml), li = __ldcg(ml + S::kRows);
              const float4* part = reinterpret_cast<const float4*>(c.part_o) +
                                   (slot * D + col) / 4 * S::kRows + rr;
              float4 p[kCols / 4];
#pragma unroll
              for (int e = 0; e < kCols / 4; ++e) p[e] = __ldcg(part + e * S::kRows);
              const float both = fmaxf(top, mi), ref = both == -INFINITY ? 0.f : both;
              const float was = exp2_fast(top - ref), is = exp2_fast(mi - ref);
              top = both;
              all = all * was + li * is;
#pragma unroll
              for (int e = 0; e < kCols / 4; ++e) {
                o[4 * e] = o[4 * e] * was + p[e].x * is;
                o[4 * e + 1] = o[4 * e + 1] * was + p[e].y * is;
                o[4 * e + 2] = o[4 * e + 2] * was + p[e].z * is;
                o[4 * e + 3] = o[4 * e + 3] * was + p[e].w * is;
              }
            }
            int head;
            const int t = x.sp.first + quotient(x.row + rr, c.by_group, head);
            head += x.head * c.by_group.d;
            const long long line = (long long)t * c.heads + head;
            const float sink = c.a.sinks ? __ldg(c.a.sinks + head) : -INFINITY;
            const Close z = close_row(top, all, sink, kLift);
            if (in && wid == 0 && c.a.lse) c.a.lse[line] = z.lse;
            uint4* out =
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.a.out) + line * D + col);
            const float f = z.scale * v_scale;
            if (in) {
#pragma unroll
              for (int e = 0; e < kCols; e += 8)
                out[e / 8] = z.scale == 0.f
                                 ? make_uint4(0, 0, 0, 0)
                                 : make_uint4(pack2<QT>(o[e] * f, o[e + 1] * f),
                                              pack2<QT>(o[e + 2] * f, o[e + 3] * f),
                                              pack2<QT>(o[e + 4] * f, o[e + 5] * f),
                                              pack2<QT>(o[e + 6] * f, o[e + 7] * f));
            }
          }
        }
      }
    }
  softmax_end:
    (void)0;
  }
  __syncthreads();
  if (wid == kProducts) tc::tmem_free(tmem, 512);
  if (tid == 0 && s_quit) atomicOr(c.err, kErrTimeout);
}

template <int D, int CT, int QT>
cudaError_t chunk_as(const moe_reader_kv& kv, const moe_reader_kv_chunk_args& a, cudaStream_t s) {
  ChunkCall c = {};
  c.a = a;
  c.k = static_cast<const char*>(kv.k);
  c.v = static_cast<const char*>(kv.v);
  c.k_scale = kv.k_scale;
  c.v_scale = kv.v_scale;
  c.part_o = kv.chunk_o;
  c.part_ml = kv.chunk_ml;
  c.arrived = kv.chunk_arrived;
  c.err = kv.err;
  c.heads = kv.cfg.num_q_heads;
  c.kv_heads = kv.cfg.num_kv_heads;
  c.by_group = divisor(kv.group);
  c.by_kv = divisor(kv.cfg.num_kv_heads);
  c.shift = kv.page_shift;
  c.pool = kv.cfg.num_pages;
  using S = ChunkShape<D>;
  c.rows = S::kRows / kv.group * kv.group;
  c.stall = take_prompt_stall();
  // a box: all of an item's tokens, one KV head's queries, 64 coordinates
  c.wide = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_token_stride % 8 == 0 &&
           a.q_head_stride % 8 == 0;
  c.mapped = c.wide && a.q_token_stride > 0 && a.q_head_stride > 0 && !(a.scale < 0.f) &&
             !(CT == kE4m3 && QT == kBf16);
  if (c.mapped) {
    const uint64_t sizes[3] = {(uint64_t)D, (uint64_t)c.heads, (uint64_t)a.tokens};
    const uint64_t strides[2] = {(uint64_t)a.q_head_stride, (uint64_t)a.q_token_stride};
    const uint32_t box[3] = {64, (uint32_t)kv.group, (uint32_t)(c.rows / kv.group)};
    c.mapped = tc::make_map(&c.q_map, a.q, QT == kBf16, 3, sizes, strides, box) == cudaSuccess;
  }
  c.k_map = kv.chunk_maps[0];
  c.v_map = kv.chunk_maps[1];
  using T = ChunkShape<D, CT>;
  return launch_early(chunk_kernel<D, CT, QT>, dim3(kv.sms), T::kThreads, T::kSmem, s, c);
}

template <int D>
cudaError_t chunk_dim(const moe_reader_kv& kv, const moe_reader_kv_chunk_args& a, cudaStream_t s) {
  if (kv.cfg.cache_type == kBf16) return chunk_as<D, kBf16, kBf16>(kv, a, s);
  if (kv.cfg.cache_type == kF16) return chunk_as<D, kF16, kF16>(kv, a, s);
  return a.q_type == kBf16 ? chunk_as<D, kE4m3, kBf16>(kv, a, s) : chunk_as<D, kE4m3, kF16>(kv, a, s);
}

template <int D, int CT, int QT> cudaError_t configure_as() {
  return cudaFuncSetAttribute(chunk_kernel<D, CT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)ChunkShape<D, CT>::kSmem);
}
template <int D> cudaError_t configure_dim(int type) {
  if (type == kBf16) return configure_as<D, kBf16, kBf16>();
  if (type == kF16) return configure_as<D, kF16, kF16>();
  const cudaError_t e = configure_as<D, kE4m3, kBf16>();
  return e != cudaSuccess ? e : configure_as<D, kE4m3, kF16>();
}

}  // namespace

int chunk_rows(const moe_reader_kv_config& c) {
  return c.head_dim <= 128 ? ChunkShape<128>::kRows : ChunkShape<256>::kRows;
}

cudaError_t configure_kv_chunk(moe_reader_kv& kv) {
  const moe_reader_kv_config& g = kv.cfg;
  // (an e4m3 cache's pages come by bulk copies: its maps are not used)
  for (int i = 0; i < 2; ++i) {
    const uint64_t D = g.head_dim, P = g.page_size, H = g.num_kv_heads;
    const uint64_t sizes[4] = {D, P, H, (uint64_t)g.num_pages}, strides[3] = {D, P * D, H * P * D};
    const uint32_t box[4] = {64, (uint32_t)std::min(g.page_size, D <= 128 ? 128 : 64), 1, 1};
    const cudaError_t e = tc::make_map(&kv.chunk_maps[i], i ? kv.v : kv.k, g.cache_type == kBf16, 4,
                                       sizes, strides, box);
    if (e != cudaSuccess) return e;
  }
  switch (kv.cfg.head_dim) {
    case 64: return configure_dim<64>(kv.cfg.cache_type);
    case 128: return configure_dim<128>(kv.cfg.cache_type);
    default: return configure_dim<256>(kv.cfg.cache_type);
  }
}

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
