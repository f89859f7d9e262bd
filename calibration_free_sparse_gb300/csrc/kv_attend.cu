// Attention of one new token per request over a paged cache, split over the
// cache's length and joined in the same launch.
//
// Per (request, KV head) the group's query heads share every key and value
// read, so the arithmetic intensity is about 2 * group operations per cached
// element: the kernel is bound by HBM, and the tensor cores only have to keep
// the group's products off the FP32 pipes.  The products are formed
// transposed, S^T = K Q^T (16 keys x 8 heads per instruction) and
// O^T = V^T P^T (16 coordinates x 8 heads): a group of up to 8 heads fills the
// short side of the instruction, K and V come from shared memory as the long
// side, and the accumulators cost D / 4 registers per 8 heads.
//
// Work is a list of (row, tile of keys), a row being a request, a KV head and
// up to 16 of its query heads.  The lengths are on the device, so every CTA
// counts the tiles itself and takes an equal contiguous share of the list (with
// few rows a whole number of CTAs per row, with many short ones whole rows per
// CTA or per warp; where lengths differ much, the short rows go to single warps,
// which take them before their CTA's share of the others).  Inside a CTA every
// warp takes every kWarps-th tile with a private cp.async pipeline, softmax state
// and output, and its copies run on across rows: no barrier until the share
// ends.  Where a row ends before the share does, the warps add their states to
// one in shared memory in turns, beginning with another warp each time, and go
// on; a barrier there left HBM idle for about 3 us a row.  A row that several
// CTAs hold is joined by the CTA that finishes it, in the order of the shares.
// All sums have a fixed order: the result does not depend on timing.
//
// Measured on a GB300 (read-only streams reach 7.3 TB/s there): 128 requests of
// up to 8192 tokens, 16 heads of 128 on each of 4 KV heads, bf16: 206 us for
// 1.28 GB, 6.2 TB/s, the tensor pipe 27 % busy (so a wider matrix instruction
// would not shorten it); 131071 tokens of e4m3 alone: 49 us for 268 MB; one
// request of 301 tokens: 7 us, of which 2 are the launch, 3 the lengths, shares,
// page ids and first keys (each a round trip), 1 the sum over the warps.
#include <algorithm>
#include <type_traits>

#include "kv.cuh"

namespace mr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kBf16 = MOE_READER_TYPE_BF16;
constexpr int kF16 = MOE_READER_TYPE_F16;
constexpr int kE4m3 = MOE_READER_TYPE_E4M3;

// Shapes of one instantiation: D coordinates, NT tiles of 8 query heads, cache type CT.
template <int D_, int NT_, int CT_>
struct Shape {
  static constexpr int D = D_, NT = NT_, CT = CT_;
  static constexpr int kBytes = CT == kE4m3 ? 1 : 2;
  static constexpr int kRow = D * kBytes;                    // bytes of a key
  static constexpr int kMt = kRow >= 256 ? 1 : kRow == 128 ? 2 : 4;   // 16-key subtiles per tile
  static constexpr int kKeys = 16 * kMt;                     // keys per tile
  static constexpr int kTile = 2 * kKeys * kRow;             // bytes of a tile, K then V
  // An e4m3 tile costs its conversions: a warp is busy with it for longer than
  // HBM takes to bring it, so such rows get more warps where the registers
  // allow (128 requests, 8 heads per KV head: D 64 151.5 -> 137.1 us, D 128 227.4
  // -> 221.7).
  static constexpr int kWarps = kRow >= 512 ? 4 : CT == kE4m3 && NT == 1 && D <= 128 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = 192 * 1024 / (kWarps * kTile);   // copies in flight: all but one
  static constexpr int kSplit = 64;                          // tiles that a join is worth
  // Weights are formed relative to a reference that lies 2^kLift below the
  // largest logit when it is set and follows that only when it has grown by
  // more than 2^kSlack: the sums stay exact to a common factor, and nearly
  // every tile saves the rescaling.  fp16 weights so reach 2^15, and what lies
  // 2^-35 below the largest is still a multiple of their least value (with the
  // reference at the largest, everything below 2^-25 of it was lost: 200 keys
  // beside a dominant one).  bf16 has fp32's range: there the weights stay below
  // one, so that no sum exceeds what the values allow.
  static constexpr float kLift = CT == kBf16 ? -8.f : 11.f;
  static constexpr float kSlack = CT == kBf16 ? 8.f : 4.f;
  static constexpr int kRows = 8 * NT;                       // query heads of a row
  // the sum over the warps at the end runs over slices of the coordinates
  static constexpr int kSlice = kWarps * kRows >= 96 ? 32 : 64;
  static constexpr int kPitch = kSlice + 4;
  // two rows' states in shared memory, for the rows that end inside a share
  static constexpr int kAccPitch = D + 4;
  static constexpr int kAcc = kRows * kAccPitch;
  static constexpr int kSumA = kWarps * kRows * kPitch * 4, kSumB = 2 * kAcc * 4;
  static constexpr int kPipe = kWarps * kStages * kTile;
  static constexpr int kSum = kSumA > kSumB ? kSumA : kSumB;
  static constexpr int kMl = kWarps * kRows * 2 * 4;
  static constexpr int kPos = kWarps * kStages * kMt * 4;
  static constexpr int kSmem = kPipe + kSum + kMl + kPos + (2 * kMaxRequests + 1) * 4 +
                               kMaxRequests * 2;
  static_assert(kRows * kMaxSms * 4 <= kSum, "join weights of a piece per CTA");
  static_assert(kSmem + 2048 <= 227 * 1024 && kStages >= 2, "shared memory");
};

struct Params {
  const void* q;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* pages;
  const float* sinks;
  void* out;
  float* lse;
  long long q_request, q_head;
  int q_type, q_pairs, requests, width, keep, window;
  float scale;
  const char* k;
  const char* v;
  const float* k_scale;
  const float* v_scale;
  int heads, kv_heads, group, row_tiles, shift, num_pages;
  float* part_o;
  float* part_ml;
  uint32_t* arrived;
  uint32_t* err;
  int polls;               // of a turn, at most
  uint32_t stall;          // added to the turn that is waited for: 0, or never reached
};

// ---- instructions ---------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
// zeros where `bytes` is 0
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// the same, rounded towards zero
template <bool BF>
__device__ __forceinline__ uint32_t truncate(float lo, float hi) {
  uint32_t r;
  if constexpr (BF) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF>
__device__ __forceinline__ float2 unpack(uint32_t v) {
  if constexpr (BF) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// The lower and the upper two of four e4m3 values.
__device__ __forceinline__ uint32_t e4m3_low(uint32_t four) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(four));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_high(uint32_t four) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(four));
  return r;
}
__device__ __forceinline__ float load_q(const uint16_t* p, int type) {
  const uint16_t u = __ldg(p);
  return type == kBf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// 16-byte chunk `c` of row `r`, placed so that the eight rows of a matrix load
// (and of its transpose) fall on different banks.
template <int kRow>
__device__ __forceinline__ uint32_t place(int r, int c) {
  constexpr int kChunks = kRow / 16;
  if constexpr (kChunks >= 8) return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4));
  else return (uint32_t)(r * kRow + ((c ^ ((r >> 1) & 3)) << 4));
}

// What is attended to of a request: keys [lo, len), as `span` virtual keys
// from `base` on (a multiple of 16).  With a page list the virtual keys are
// the listed pages' rows.
struct Row {
  int len, lo, base, span;
};

__device__ __forceinline__ Row row_of(const Params& P, int len) {
  Row w;
  w.len = len;
  w.lo = P.window ? max(0, w.len - P.window) : 0;
  if (P.pages) {
    w.base = 0;
    w.span = w.len > 0 ? P.keep << P.shift : 0;
  } else {
    w.base = w.lo & ~15;
    w.span = w.len - w.base;
  }
  return w;
}

template <class S>
__device__ __forceinline__ int tiles_of(const Row& w) {
  return (w.span + S::kKeys - 1) / S::kKeys;
}

// The item at an index of the list.
template <class S>
struct Item {
  int r, sub;            // request, KV head
  int begin, end, tiles; // the item's indices in the (padded) list, its real tiles
  Row row;
};

template <class S>
__device__ __forceinline__ Item<S> item_at(const Params& P, const int* prefix,
                                           const uint16_t* order, const int* lens, int per,
                                           int t) {
  int lo = 0, hi = P.requests - 1;
  while (lo < hi) {                      // the last request that begins at t or before
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * per <= t) lo = mid; else hi = mid - 1;
  }
  Item<S> o;
  o.r = order[lo];
  o.row = row_of(P, lens[o.r]);
  o.tiles = tiles_of<S>(o.row);
  const int first = prefix[lo] * per, padded = prefix[lo + 1] - prefix[lo];
  o.sub = (t - first) / padded;
  o.begin = first + o.sub * padded;
  o.end = o.begin + padded;
  return o;
}

// One 16-key subtile's source: its page and the first row in it, the position
// of that key (past the end where nothing is read) and the keys in use.
struct Source {
  int id, head, in, pos, lo, len;
};
constexpr int kNowhere = INT32_MAX - 64;

// Source of subtile s of the tile at index t.  The page id is used by the
// caller only later, so that its load is in flight meanwhile.
template <class S>
__device__ __forceinline__ Source source_at(const Params& P, const int* prefix,
                                            const uint16_t* order, const int* lens, int per,
                                            int t, int s, uint32_t& bad) {
  Source o;
  const Item<S> it = item_at<S>(P, prefix, order, lens, per, t);
  o.id = 0;
  o.pos = kNowhere;
  o.lo = it.row.lo;
  o.len = it.row.len;
  o.head = it.sub;
  const int v = (t - it.begin) * S::kKeys + s * 16;      // virtual key of the item
  const int j = it.row.base + v;
  o.in = j & ((1 << P.shift) - 1);
  if (t - it.begin >= it.tiles || v >= it.row.span) return o;
  int lp = j >> P.shift;
  if (P.pages) {
    const int listed = __ldg(P.pages + ((size_t)it.r * P.kv_heads + o.head) * P.keep + lp);
    if (listed < 0 || listed >= (it.row.len + (1 << P.shift) - 1) >> P.shift) {
      if (listed != -1) bad |= kErrPage;
      return o;
    }
    lp = listed;
  }
  o.id = __ldg(P.table + (size_t)it.r * P.width + lp);
  o.pos = (lp << P.shift) + o.in;
  return o;
}

// Copies one subtile's K and V rows; rows outside [lo, len) become zeros, so
// that whatever an unwritten row holds meets no weight.
template <class S>
__device__ __forceinline__ void copy_subtile(const Params& P, long long at, int pos, int lo,
                                             int len, uint32_t k_dst, uint32_t v_dst) {
  constexpr int kChunks = S::kRow / 16, kStep = 32 / kChunks;    // rows per 32 lanes
  const int lane = threadIdx.x & 31;
  const int r0 = lane / kChunks;
  const uint32_t d0 = place<S::kRow>(r0, lane % kChunks);
  const char* ks = P.k + at + lane * 16;
  const char* vs = P.v + at + lane * 16;
  const bool whole = pos >= lo && pos + 16 <= len;
#pragma unroll
  for (int i = 0; i < 16 / kStep; ++i) {
    // place(r0 + i kStep, c): r0 < kStep, so the row's swizzle bits split
    const uint32_t flip = kChunks >= 8 ? ((i * kStep) & 7) << 4 : 0;
    const uint32_t d = (d0 ^ flip) + i * 512;
    if (whole) {
      cp_async(k_dst + d, ks + i * 512);
      cp_async(v_dst + d, vs + i * 512);
    } else {
      const int p = pos + r0 + i * kStep;
      const bool in = p >= lo && p < len;
      cp_async_or_zero(k_dst + d, in ? ks + i * 512 : P.k, in ? 16 : 0);
      cp_async_or_zero(v_dst + d, in ? vs + i * 512 : P.v, in ? 16 : 0);
    }
  }
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_addr(p)) : "memory");
  return v;
}
// Waits until shared word `turn` reaches `want`; all lanes.  False where that
// took `most` polls (a fraction of a second; the warps that it waits for only
// compute, so only an injected stall gets there) or another wait of the CTA gave
// up: the turn is then not passed on, so that all later ones end soon, too, and
// the call ends with an error.
__device__ __forceinline__ bool wait_turn(const uint32_t* turn, uint32_t want, uint32_t* gave_up,
                                          int most) {
  bool mine = false;
  for (int n = 0; n < most; ++n) {
    mine = load_acquire(turn) == want;
    if (mine || ((n & 63) == 63 && load_acquire(gave_up))) break;
    __nanosleep(64);
  }
  mine = __all_sync(0xffffffffu, mine);
  if (!mine)
    asm volatile("st.release.cta.shared.u32 [%0], 1;" ::"r"(smem_addr(gave_up)) : "memory");
  return mine;
}
__device__ __forceinline__ void pass_turn(uint32_t* turn, uint32_t next) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_addr(turn)), "r"(next) : "memory");
}

// What scales a row's weighted sum to its output, and the log of its
// denominator: here the sink joins.  top and den: the row's reference (in
// units of log2; -infinity where nothing was seen) and the sum of its weights.
template <class S>
__device__ __forceinline__ void finish(const Params& P, int kvh, int head, float top, float den,
                                       float& mul, float& lse) {
  const float vs = S::CT == kE4m3 ? __ldg(P.v_scale + kvh) : 1.f;
  float ref = top;
  if (P.sinks) {
    const float sink = __ldg(P.sinks + head) * kLog2e;
    ref = fmaxf(top, sink);
    const float down = top == -INFINITY ? 0.f : exp2_fast(top - ref);
    // the larger of the two by its equality: both may be infinite
    den = den * down + (sink == -INFINITY ? 0.f : sink == ref ? 1.f : exp2_fast(sink - ref));
    mul = den == 0.f ? 0.f : vs * down / den;
  } else {
    mul = den == 0.f ? 0.f : vs / den;
  }
  lse = (ref + log2f(den)) * kLn2;          // of a sum of 0: -infinity
}

// Two neighbouring outputs of a query head.
__device__ __forceinline__ void store_out(const Params& P, int r, int head, int D, int d, float a,
                                          float b) {
  uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(P.out) +
                                             ((size_t)r * P.heads + head) * D + d);
  *at = P.q_type == kBf16 ? pack<true>(a, b) : pack<false>(a, b);
}

// Writes a row that one warp has computed.  The accumulators' 8 x 8 blocks
// (coordinate by head) are transposed, so that a lane has neighbouring
// coordinates of one head.
template <class S>
__device__ __forceinline__ void store_row(const Params& P, int r, int kvh, int head0, int rows,
                                          const float (&o)[S::D / 16][S::NT][4],
                                          const float (&m)[S::NT][2],
                                          const float (&l)[S::NT][2]) {
  constexpr int D = S::D;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int n = 0; n < S::NT; ++n) {
    float mul[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = n * 8 + 2 * t4 + i;
      float lse;
      finish<S>(P, kvh, head0 + (h < rows ? h : 0), m[n][i], l[n][i], mul[i], lse);
      if (g == 0 && h < rows && P.lse) P.lse[(size_t)r * P.heads + head0 + h] = lse;
    }
    const int h = n * 8 + g;
    uint16_t* out = static_cast<uint16_t*>(P.out) + ((size_t)r * P.heads + head0 + h) * D;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      uint32_t v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = o[x][n][2 * i] * mul[0], b = o[x][n][2 * i + 1] * mul[1];
        v[i] = transpose8(P.q_type == kBf16 ? pack<true>(a, b) : pack<false>(a, b));
      }
      if (h >= rows) continue;
      if constexpr (S::CT == kE4m3) {
        // rows g and g + 8 of the block are coordinates 2g and 2g + 1
        *reinterpret_cast<uint2*>(out + x * 16 + 4 * t4) =
            make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632));
      } else {
        *reinterpret_cast<uint32_t*>(out + x * 16 + 2 * t4) = v[0];
        *reinterpret_cast<uint32_t*>(out + x * 16 + 8 + 2 * t4) = v[1];
      }
    }
  }
}

// Sums the pieces of a row that several CTAs wrote, in order; all of the CTA.
template <class S>
__device__ __forceinline__ void join_row(const Params& P, const Item<S>& it, int rt, int U, int pieces,
                                         float* wgt, float* s_mul) {
  constexpr int D = S::D;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int kvh = it.sub, row0 = rt * S::kRows;
  const int rows = min(S::kRows, P.group - row0), head0 = kvh * P.group + row0;
  const int first = it.begin / U;
  // a CTA's first piece is in its slot 0, unless the row began inside its share
  auto slot = [&](int p) {
    return (size_t)((first + p) * P.row_tiles + rt) * 2 + ((first + p) * U >= it.begin ? 0 : 1);
  };
  for (int h = wid; h < rows; h += S::kWarps) {
    float top = -INFINITY;
    for (int p = lane; p < pieces; p += 32)
      top = fmaxf(top, __ldcg(P.part_ml + slot(p) * 32 + h));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    float den = 0.f;
    for (int p = lane; p < pieces; p += 32) {
      const float mp = __ldcg(P.part_ml + slot(p) * 32 + h);
      const float w = mp == -INFINITY ? 0.f : exp2_fast(mp - top);
      wgt[p * S::kRows + h] = w;
      den += w * __ldcg(P.part_ml + slot(p) * 32 + 16 + h);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(0xffffffffu, den, x);
    float mul, lse;
    finish<S>(P, kvh, head0 + h, top, den, mul, lse);
    if (lane == 0) {
      s_mul[h] = mul;
      if (P.lse) P.lse[(size_t)it.r * P.heads + head0 + h] = lse;
    }
  }
  __syncthreads();
  for (int e = tid; e < rows * D / 4; e += S::kThreads) {
    const int h = e / (D / 4), d = e % (D / 4) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < pieces; ++p) {
      const float4 v =
          __ldcg(reinterpret_cast<const float4*>(P.part_o + (slot(p) * 16 + h) * D + d));
      const float w = wgt[p * S::kRows + h];
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
    const float mul = s_mul[h];
    store_out(P, it.r, head0 + h, D, d, acc.x * mul, acc.y * mul);
    store_out(P, it.r, head0 + h, D, d + 2, acc.z * mul, acc.w * mul);
  }
  __syncthreads();
}

// ---- the kernel -----------------------------------------------------------
template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) attend_kernel(const Params P) {
  constexpr int D = S::D, NT = S::NT, kMt = S::kMt, kWarps = S::kWarps;
  constexpr bool kBf = S::CT == kBf16, k8 = S::CT == kE4m3;
  extern __shared__ __align__(1024) unsigned char smem[];
  float* s_sum = reinterpret_cast<float*>(smem + S::kPipe);
  float* s_ml = reinterpret_cast<float*>(smem + S::kPipe + S::kSum);
  int* s_pos = reinterpret_cast<int*>(smem + S::kPipe + S::kSum + S::kMl);
  int* s_prefix = s_pos + S::kPos / 4;
  int* s_len = s_prefix + kMaxRequests + 1;
  uint16_t* s_order = reinterpret_cast<uint16_t*>(s_len + kMaxRequests);   // requests of the list
  __shared__ int4 s_scan[kWarps];
  __shared__ int s_before[kWarps];
  __shared__ uint32_t s_turn[2], s_gave_up;
  __shared__ int s_last[2];
  __shared__ float s_mul[S::kRows];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  // Groups of more query heads than a row holds: their row tiles are dealt to
  // neighbouring CTAs with one share of keys, which then come from HBM once.
  const int per = P.kv_heads, rt = blockIdx.x % P.row_tiles, cta = blockIdx.x / P.row_tiles;
  uint32_t bad = 0;

  if (tid < 2) s_turn[tid] = 0, s_last[tid] = 0;
  if (tid == 0) s_gave_up = 0;
  wait_for_earlier_launch();
  // ---- shares of the rows that CTAs share: U tiles per CTA ----
  constexpr int kPer = (kMaxRequests + S::kThreads - 1) / S::kThreads;
  int mine[kPer], sum = 0, rows = 0, most = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int r = tid * kPer + j;
    mine[j] = 0;
    if (r < P.requests) {
      const int room = P.width << P.shift;
      int len = __ldg(P.lens + r);
      if (len < 0) len = 0, bad |= kErrLength;
      if (len > room) len = room, bad |= kErrLength;
      s_len[r] = len;
      mine[j] = tiles_of<S>(row_of(P, len));
    }
    sum += mine[j];
    rows += mine[j] > 0;
    most = max(most, mine[j]);
  }
  if (blockIdx.x == 0 && bad) atomicOr(P.err, bad);
  bad = 0;
  auto block_sums = [&](int& a, int& b, int& top) {    // two sums and a maximum
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_scan[wid] = make_int4(a, b, top, 0);
    __syncthreads();
    a = b = top = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int4 v = s_scan[w];
      a += v.x;
      b += v.y;
      top = max(top, v.z);
    }
  };
  block_sums(sum, rows, most);
  const int grid = (int)gridDim.x / P.row_tiles;
  int total = sum * per, items = rows * per;

  // Times below are in tiles of a warp's time (about 0.75 us).  A row that the
  // warps of a CTA share costs them about seven beside its tiles, a row that
  // CTAs share fifteen; a row that a single warp has to itself costs one and a
  // half, but all of its tiles are that warp's.  (Fitted to bf16 heads of 128,
  // eight warps; the other shapes use the same numbers.  128 requests lognormal
  // around 500 tokens, 8 KV heads: bf16 heads of 128 80 us of 55 at the measured
  // bandwidth, of 256 159 / 111; e4m3 heads of 128 79 / 28, of 64 52 / 14.)
  int short_most = 0;             // rows of at most so many tiles are single warps'
  const bool differ = items >= 16 && (long long)most * items >= 2LL * total;
  if (items > grid || differ) {
    const int each = total / (grid * kWarps);          // a warp's part
    if (items > grid) {
      const int meeting = each + 7 * (items / grid) +
                          (most < 20 * kWarps ? 7 + most / (2 * kWarps) : 15);
      if (max(most, each) + most / 4 + items * 3 / (2 * grid * kWarps) < meeting)
        short_most = most;
    }
    if (short_most == 0 && differ) {
      // The short rows go to single warps, where they are many, the others are
      // shared.  8 KV heads of 128, 128 requests: lengths lognormal around 500
      // (sigma 1) 109 -> 80 us, around 100 (1.2) 79 -> 40, one of 8192 tokens
      // and 127 of 5 96 -> 18.  Up to half a part instead: 89 us for the first.
      const int limit = max(each, 16);
      int b_sum = 0, b_rows = 0, none = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (mine[j] > 0 && mine[j] <= limit) b_sum += mine[j], ++b_rows;
      __syncthreads();                                 // s_scan is read above
      block_sums(b_sum, b_rows, none);
      if (b_rows * per * 2 >= grid && b_rows < rows) {
        short_most = limit;
        total -= b_sum * per;
        items -= b_rows * per;
      }
    }
  }
  // The other rows.  Equal shares: best where the cache is long.  A row of its
  // own per CTA (or a whole number of CTAs per row) where that costs no CTA more
  // than kSplit tiles extra.  More rows than CTAs, but short ones: whole rows, to
  // the CTAs in whose part of the list they begin, which costs half a row in
  // balance.  Measured, 8 KV heads of 128, 128 requests of up to 100 / 500 / 1000 /
  // 2000 tokens: equal shares 47 / 62 / 84 / 128 us, whole rows per CTA - / - / - /
  // 120, per warp 15 / 41 / 70 / 132; 40 requests of up to 600, 4 KV heads: 26 /
  // 18 / 27.
  constexpr int kSplit = S::kSplit;
  int U = max((total + grid - 1) / grid, kWarps);
  bool whole = false, aligned = false;
  if (items <= grid) {
    int W = most;                                      // no row split
    if (items < grid) {
      const int cut = max((total + (grid - items) - 1) / (grid - items), kWarps);
      if (cut + kSplit < W) W = cut;
    }
    if (W <= U + kSplit) whole = true, U = max(W, 1);
  } else if (most < 20 * kWarps) {
    aligned = true;
    U = 1 << 30;                                       // no row is cut
  }
  // The list: requests whose rows are shared, padded to whole shares, then those
  // whose rows are single warps'.
  int at_b = 0, at_n = 0, all_n = 0;                   // short requests: tiles and their number
  if (short_most > 0) {
    int b = 0, n = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (mine[j] > 0 && mine[j] <= short_most) b += mine[j], ++n;
    int ib = b, in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ub = __shfl_up_sync(0xffffffffu, ib, o), un = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) ib += ub, in += un;
    }
    __syncthreads();                                   // s_scan is read above
    if (lane == 31) s_scan[wid] = make_int4(ib, in, 0, 0);
    __syncthreads();
    at_b = ib - b;
    at_n = in - n;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int4 v = s_scan[w];
      if (w < wid) at_b += v.x, at_n += v.y;
      all_n += v.y;
    }
  }
  int a = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (whole && mine[j] > short_most) mine[j] = (mine[j] + U - 1) / U * U;
    if (mine[j] > short_most) a += mine[j];
  }
  int ia = a;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, ia, o);
    if (lane >= o) ia += up;
  }
  if (lane == 31) s_before[wid] = ia;
  __syncthreads();
  int at_a = ia - a, all_a = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int v = s_before[w];
    if (w < wid) at_a += v;
    all_a += v;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int r = tid * kPer + j;
    const bool brief = mine[j] > 0 && mine[j] <= short_most;
    if (r < P.requests) {
      const int i = brief ? P.requests - all_n + at_n : r - at_n;
      s_order[i] = (uint16_t)r;
      s_prefix[i] = brief ? all_a + at_b : at_a;
    }
    if (brief) at_b += mine[j], ++at_n;
    else at_a += mine[j];
  }
  if (tid == S::kThreads - 1) s_prefix[P.requests] = all_a + at_b;
  __syncthreads();
  const int shared_end = all_a * per, all = s_prefix[P.requests] * per;

  // rows with nothing to read
  for (int e = blockIdx.x; e < P.requests; e += gridDim.x) {
    if (s_prefix[e + 1] != s_prefix[e]) continue;
    const int r = s_order[e];
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + (size_t)r * P.heads * D);
    for (int i = tid; i < P.heads * D / 8; i += S::kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (P.lse)
      for (int i = tid; i < P.heads; i += S::kThreads)
        P.lse[(size_t)r * P.heads + i] = P.sinks ? P.sinks[i] : -INFINITY;
  }

  // [c0, c1): the CTA's share; [b0, b1): the rows that are this warp's own
  auto row_from = [&](long long t) {                   // the first row from t on
    if (t >= all) return all;
    const Item<S> it = item_at<S>(P, s_prefix, s_order, s_len, per, (int)t);
    return it.begin < t ? it.end : it.begin;
  };
  int c0 = 0, c1 = 0, b0 = 0, b1 = 0;
  if (aligned) {
    if (shared_end > 0) {
      c0 = min(row_from((long long)cta * shared_end / grid), shared_end);
      c1 = min(row_from((long long)(cta + 1) * shared_end / grid), shared_end);
    }
  } else if ((long long)cta * U < shared_end) {
    c0 = cta * U;
    c1 = min(shared_end - c0, U) + c0;
  }
  if (all > shared_end) {
    const long long part = cta * kWarps + wid, parts = grid * kWarps, own = all - shared_end;
    b0 = row_from(shared_end + part * own / parts);
    b1 = row_from(shared_end + (part + 1) * own / parts);
  }
  const int n_own = max(b1 - b0, 0);                   // the warp's tiles: its own rows first
  const int tiles = n_own + (c1 > c0 + wid ? (c1 - c0 - wid + kWarps - 1) / kWarps : 0);
  if (n_own == 0 && c0 >= c1) return;                  // all warps of a CTA share or none
  auto tile_at = [&](int n) { return n < n_own ? b0 + n : c0 + wid + (n - n_own) * kWarps; };

  // CTAs that hold a part of a row; one more part of it is written (the last
  // to say so gets true, and clears the counter for the next launch)
  auto pieces_of = [&](const Item<S>& it) {
    return (it.begin + it.tiles - 1) / U - it.begin / U + 1;
  };
  auto arrive = [&](const Item<S>& it) -> int {
    uint32_t* count = P.arrived + (it.r * per + it.sub) * P.row_tiles + rt;
    __threadfence();
    const bool last = atomicAdd(count, 1u) + 1 == (uint32_t)pieces_of(it);
    if (last) *count = 0;
    __threadfence();
    return last;
  };

  // ---- this warp's pipeline ----
  // Lane i looks up the source of subtile i of the warp's next 32 subtiles; a
  // batch is looked up while the one before it is copied.
  constexpr int kBatch = 32 / kMt;
  const uint32_t pipe = smem_addr(smem) + wid * S::kStages * S::kTile;
  int copied = 0;          // tiles copied by this warp
  Source now, next;
  long long now_at = 0;    // byte offset of the lane's subtile
  auto look = [&](int n) { // the batch that begins with the warp's tile n
    const int i = n + lane / kMt;
    next.pos = kNowhere;
    next.id = next.head = next.in = next.lo = next.len = 0;
    if (i < tiles)
      next = source_at<S>(P, s_prefix, s_order, s_len, per, tile_at(i), lane % kMt, bad);
  };
  int in_stage = 0, out_stage = 0;
  auto issue = [&]() {
    const int n = copied % kBatch;
    if (n == 0) {
      now = next;
      if (now.pos != kNowhere && (now.id < 0 || now.id >= P.num_pages)) {
        bad |= kErrPage;
        now.pos = kNowhere;
      }
      now_at = ((((long long)now.id * P.kv_heads + now.head) << P.shift) + now.in) * S::kRow;
      look(copied + kBatch);
    }
    if (copied < tiles) {
      const uint32_t base = pipe + in_stage * S::kTile;
#pragma unroll
      for (int s = 0; s < kMt; ++s) {
        const int from = n * kMt + s;
        copy_subtile<S>(P, __shfl_sync(0xffffffffu, now_at, from),
                        __shfl_sync(0xffffffffu, now.pos, from),
                        __shfl_sync(0xffffffffu, now.lo, from),
                        __shfl_sync(0xffffffffu, now.len, from), base + s * 16 * S::kRow,
                        base + (S::kKeys + s * 16) * S::kRow);
      }
      // the positions of the stage's keys, for the mask
      if (lane / kMt == n) s_pos[(wid * S::kStages + in_stage) * kMt + lane % kMt] = now.pos;
    }
    cp_commit();
    in_stage = in_stage + 1 == S::kStages ? 0 : in_stage + 1;
    ++copied;
  };
  look(0);
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) issue();

  // The lane's row and 16-byte chunk in the matrix loads; the loads of the next
  // 32 bytes of the rows flip bits above (place() is an exclusive or).
  const uint32_t k_lane = place<S::kRow>(lane & 15, lane >> 4);
  const uint32_t v_lane =
      k8 ? k_lane : place<S::kRow>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);

  // ---- pieces: the rows, or parts of rows, of this share ----
  float o[D / 16][NT][4], m[NT][2], l[NT][2];
  Item<S> cc;
  bool own = n_own > 0;
  int p0 = own ? b0 : c0, t = own ? b0 : c0 + wid;
  for (int k = 0;;) {                                  // k: shared pieces so far
    cc = item_at<S>(P, s_prefix, s_order, s_len, per, p0);
    const int p1 = own ? cc.end : min(c1, cc.end), step = own ? 1 : kWarps;
    const int real = min(p1, cc.begin + cc.tiles);     // tiles beyond are padding
    const int kvh = cc.sub, row0 = rt * S::kRows;
    const int rows_here = min(S::kRows, P.group - row0);
    const int head0 = kvh * P.group + row0;

    // the query's fragments: head g of each tile of eight, two coordinates a register
    uint32_t qf[NT][D / 16][2];
    float fac[NT][2];
    {
      const float ks = k8 ? __ldg(P.k_scale + kvh) : 1.f;
      const float base = P.scale * ks * kLog2e;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = n * 8 + g;
        const uint16_t* q = static_cast<const uint16_t*>(P.q) + cc.r * P.q_request +
                            (long long)(head0 + (h < rows_here ? h : 0)) * P.q_head;
        if constexpr (!k8) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint16_t* at = q + k * 16 + i * 8 + 2 * t4;
              qf[n][k][i] = P.q_pairs ? __ldg(reinterpret_cast<const uint32_t*>(at))
                                      : (uint32_t)__ldg(at) | (uint32_t)__ldg(at + 1) << 16;
            }
          fac[n][0] = fac[n][1] = base;
        } else {
          // q as fp16: a power of two brings the head's largest value to [2^14,
          // 2^15), and what lies 2^-28 (fp16) or 2^-31 (bf16) below it keeps every bit
          float top = 0.f;
          float f[D / 16][4];
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[k][i] = load_q(q + k * 16 + 4 * t4 + i, P.q_type);
              top = fmaxf(top, fabsf(f[k][i]));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = max((__float_as_int(top) >> 23) - 127 - 14, -126);
          const float down = two_to(-e);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            qf[n][k][0] = pack<false>(f[k][0] * down, f[k][1] * down);
            qf[n][k][1] = pack<false>(f[k][2] * down, f[k][3] * down);
          }
          const float up = two_to(e);
          fac[n][0] = base * __shfl_sync(0xffffffffu, up, 8 * t4);
          fac[n][1] = base * __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
        }
      }
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][n][i] = 0.f;
    }

#pragma unroll 1
    for (; t < p1; t += step) {
      cp_wait<S::kStages - 2>();
      __syncwarp();
      issue();          // into the stage that the previous tile left
      const uint32_t ks = pipe + out_stage * S::kTile, vs = ks + S::kKeys * S::kRow;
      const int* pos = s_pos + (wid * S::kStages + out_stage) * kMt;
      out_stage = out_stage + 1 == S::kStages ? 0 : out_stage + 1;
      if (t >= real) continue;
      bool any = false;
#pragma unroll
      for (int s = 0; s < kMt; ++s) any |= pos[s] < cc.row.len;
      if (!any) continue;                              // no page there

      // S^T = K Q^T, as kSplitK sums where the tile alone gives one chain of products
      constexpr int kSplitK = NT * kMt == 1 ? 2 : 1;
      float sc[kMt][NT][4], sx[NT][4];
#pragma unroll
      for (int n1 = 0; n1 < NT; ++n1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sx[n1][i] = 0.f;
#pragma unroll
          for (int s = 0; s < kMt; ++s) sc[s][n1][i] = 0.f;
        }
#pragma unroll
      for (int s = 0; s < kMt; ++s) {
        const uint32_t kb = ks + s * 16 * S::kRow + k_lane;   // ks: a multiple of the row
        if constexpr (!k8) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t a[4];
            ldsm(a, kb ^ (x << 5));
#pragma unroll
            for (int n1 = 0; n1 < NT; ++n1)
              mma<kBf>(kSplitK == 2 && (x & 1) ? sx[n1] : sc[s][n1], a, qf[n1][x][0], qf[n1][x][1]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t b[4];      // rows 0-7 and 8-15 of 16 coordinates, then of the next 16
            ldsm(b, kb ^ (x << 5));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a[4] = {e4m3_low(b[2 * j]), e4m3_low(b[2 * j + 1]),
                                     e4m3_high(b[2 * j]), e4m3_high(b[2 * j + 1])};
#pragma unroll
              for (int n1 = 0; n1 < NT; ++n1)
                mma<false>(kSplitK == 2 && j ? sx[n1] : sc[s][n1], a, qf[n1][2 * x + j][0],
                           qf[n1][2 * x + j][1]);
            }
          }
        }
      }

      // logits in units of log2, masked
#pragma unroll
      for (int s = 0; s < kMt; ++s) {
#pragma unroll
        for (int n1 = 0; n1 < NT; ++n1)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kSplitK == 2) sc[s][n1][i] += sx[n1][i];
            sc[s][n1][i] *= fac[n1][i & 1];
          }
        const int at = pos[s];
        if (at < cc.row.lo || at + 16 > cc.row.len) {
          const bool in0 = at + g >= cc.row.lo && at + g < cc.row.len;
          const bool in1 = at + g + 8 >= cc.row.lo && at + g + 8 < cc.row.len;
#pragma unroll
          for (int n1 = 0; n1 < NT; ++n1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(i < 2 ? in0 : in1)) sc[s][n1][i] = -INFINITY;
        }
      }
      // weights relative to the reference m, which follows the maximum lazily
      float top[NT][2];
      bool grown = false;
#pragma unroll
      for (int n1 = 0; n1 < NT; ++n1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = fmaxf(sc[0][n1][i], sc[0][n1][i + 2]);
#pragma unroll
          for (int s = 1; s < kMt; ++s) v = fmaxf(v, fmaxf(sc[s][n1][i], sc[s][n1][i + 2]));
          top[n1][i] = v;
          grown |= v > m[n1][i] + (S::kLift + S::kSlack);
        }
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int n1 = 0; n1 < NT; ++n1) {
          float a[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = fmaxf(top[n1][i] - S::kLift, m[n1][i]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            a[i] = exp2_fast(m[n1][i] - (v == -INFINITY ? 0.f : v));
            m[n1][i] = v;
            l[n1][i] *= a[i];
          }
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][n1][i] *= a[i & 1];
        }
      }
#pragma unroll
      for (int n1 = 0; n1 < NT; ++n1) {
        const float r0 = m[n1][0] == -INFINITY ? 0.f : m[n1][0];
        const float r1 = m[n1][1] == -INFINITY ? 0.f : m[n1][1];
#pragma unroll
        for (int s = 0; s < kMt; ++s) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[s][n1][i] = exp2_fast(sc[s][n1][i] - (i & 1 ? r1 : r0));
          l[n1][0] += sc[s][n1][0] + sc[s][n1][2];
          l[n1][1] += sc[s][n1][1] + sc[s][n1][3];
        }
      }

      // O^T += V^T P^T.  The products' type would round the weights as coarsely
      // as the output is rounded, which made the result's error 1.42 times that
      // of one rounding; so a weight is cut to that type and what was cut off
      // goes through a second product: 16 bits of it with bf16, 22 with fp16.
      // (A third bf16 part changed no output but by a rounding's side, and cost 1
      // to 5 %.)
      constexpr float kLeast = kBf ? 1.1754944e-38f : 5.9604645e-8f;   // 2^-126, 2^-24
#pragma unroll
      for (int s = 0; s < kMt; ++s) {
        uint32_t pf[NT][2], pr[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = sc[s][n][2 * i], b = sc[s][n][2 * i + 1];
            // above zero in both products wherever the weight is: an infinite
            // value stays infinite (an e4m3 cache has none)
            const float ta = k8 || a == 0.f ? 0.f : kLeast, tb = k8 || b == 0.f ? 0.f : kLeast;
            const uint32_t r = truncate<kBf>(fmaxf(a, ta), fmaxf(b, tb));
            const float2 f = unpack<kBf>(r);
            pf[n][i] = transpose8(r);
            pr[n][i] = transpose8(pack<kBf>(fmaxf(a - f.x, ta), fmaxf(b - f.y, tb)));
          }
        const uint32_t vb = vs + s * 16 * S::kRow + v_lane;
        if constexpr (!k8) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t a[4];
            ldsm_t(a, vb ^ (d << 5));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<kBf>(o[d][n], a, pf[n][0], pf[n][1]);
              mma<kBf>(o[d][n], a, pr[n][0], pr[n][1]);
            }
          }
        } else {
          // a transposed pair of bytes is coordinates 2g and 2g + 1 of two keys:
          // row g of the tile takes the even ones, row g + 8 the odd ones
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            uint32_t b[4];
            ldsm_t(b, vb ^ (d << 5));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t x = __byte_perm(b[2 * j], 0, 0x3120);
              const uint32_t y = __byte_perm(b[2 * j + 1], 0, 0x3120);
              const uint32_t a[4] = {e4m3_low(x), e4m3_high(x), e4m3_low(y), e4m3_high(y)};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma<false>(o[2 * d + j][n], a, pf[n][0], pf[n][1]);
                mma<false>(o[2 * d + j][n], a, pr[n][0], pr[n][1]);
              }
            }
          }
        }
      }
    }

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], x);
    // The maximum passes over NaN: where all logits are, the reference says
    // "nothing seen" while the sum is NaN.  Any finite reference carries the sum on.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (l[n][i] != l[n][i]) m[n][i] = fmaxf(m[n][i], 0.f);
    if (own) {
      store_row<S>(P, cc.r, kvh, head0, rows_here, o, m, l);
      p0 = p1;
      if (p1 < b1) continue;
      if (c0 >= c1) {
        if (bad) atomicOr(P.err, bad);
        return;
      }
      own = false;
      p0 = c0;
      t = c0 + wid;
      continue;
    }
    if (p1 == c1) break;

    // ---- the row ends here, the share does not: add to its state in turn ----
    const int b = k & 1, place_in_turn = (wid + kWarps - k % kWarps) % kWarps;
    float* acc = s_sum + b * S::kAcc;
    float* ref = s_ml + b * S::kRows;
    float* den = s_ml + (2 + b) * S::kRows;
    const uint32_t turn = (uint32_t)(k >> 1) * kWarps + place_in_turn;
    const bool my_turn = wait_turn(&s_turn[b], turn + P.stall, &s_gave_up, P.polls);
    if (!my_turn) bad |= MOE_READER_ERR_TIMEOUT;
    if (my_turn) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float keep[2] = {0.f, 0.f}, add[2];            // factors of the state and of this warp
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = n * 8 + 2 * t4 + i;
          const float before = place_in_turn ? ref[h] : -INFINITY;
          const float now_ref = fmaxf(before, m[n][i]);
          add[i] = m[n][i] == -INFINITY ? 0.f : exp2_fast(m[n][i] - now_ref);
          float d = l[n][i] * add[i];
          if (before != -INFINITY) {
            keep[i] = exp2_fast(before - now_ref);
            d += den[h] * keep[i];
          }
          __syncwarp();                                // all lanes of the column have read
          if (g == 0) ref[h] = now_ref, den[h] = d;
        }
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = n * 8 + 2 * t4 + (i & 1);
            float* at = acc + h * S::kAccPitch + x * 16 + (k8 ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
            const float v = o[x][n][i] * add[i & 1];
            *at = place_in_turn ? *at * keep[i & 1] + v : v;
          }
      }
    }
    __syncwarp();
    if (place_in_turn == kWarps - 1 && !my_turn) {     // the row's other CTAs still count this one
      if (cc.begin < c0 && lane == 0) s_last[0] = arrive(cc);
    } else if (place_in_turn == kWarps - 1) {
      if (cc.begin >= c0) {                            // the whole row
        if (lane < S::kRows) {
          float mul, lse;
          finish<S>(P, kvh, head0 + (lane < rows_here ? lane : 0), ref[lane], den[lane], mul, lse);
          if (lane < rows_here && P.lse) P.lse[(size_t)cc.r * P.heads + head0 + lane] = lse;
          den[lane] = mul;
        }
        __syncwarp();
        for (int e = lane; e < rows_here * D / 2; e += 32) {
          const int h = e / (D / 2), d = e % (D / 2) * 2;
          const float2 v = *reinterpret_cast<const float2*>(acc + h * S::kAccPitch + d);
          store_out(P, cc.r, head0 + h, D, d, v.x * den[h], v.y * den[h]);
        }
      } else {                                         // the end of a row: slot 0
        float* po = P.part_o + (size_t)blockIdx.x * 2 * 16 * D;
        float* pml = P.part_ml + (size_t)blockIdx.x * 2 * 32;
        for (int e = lane; e < S::kRows * D / 4; e += 32) {
          const int h = e / (D / 4), d = e % (D / 4) * 4;
          *reinterpret_cast<float4*>(po + h * D + d) =
              *reinterpret_cast<const float4*>(acc + h * S::kAccPitch + d);
        }
        if (lane < S::kRows) {
          pml[lane] = ref[lane];
          pml[16 + lane] = den[lane];
        }
        __syncwarp();
        if (lane == 0) s_last[0] = arrive(cc);
      }
      __syncwarp();
    }
    if (my_turn && lane == 0) pass_turn(&s_turn[b], turn + 1);
    p0 = p1;
    ++k;
  }

  // ---- the share's last piece: all warps at once ----
  const int kvh = cc.sub, row0 = rt * S::kRows;
  const int rows_here = min(S::kRows, P.group - row0);
  const int head0 = kvh * P.group + row0;
  __syncthreads();                                     // no turn uses the shared state any more
  if (g == 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = n * 8 + 2 * t4 + i;
        s_ml[wid * S::kRows + h] = m[n][i];
        s_ml[(kWarps + wid) * S::kRows + h] = l[n][i];
      }
  }
  __syncthreads();
  const bool alone = pieces_of(cc) == 1;
  const int which = p0 == c0 ? 0 : 1;
  const size_t slot = (size_t)blockIdx.x * 2 + which;
  float* po = P.part_o + slot * 16 * D;
  float* pml = P.part_ml + slot * 32;
  if (tid < S::kRows) {
    float top = -INFINITY, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * S::kRows + tid]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = s_ml[w * S::kRows + tid];
      if (mw != -INFINITY) den += s_ml[(kWarps + w) * S::kRows + tid] * exp2_fast(mw - top);
    }
    if (!alone) {
      pml[tid] = top;
      pml[16 + tid] = den;
    } else {
      float mul, lse;
      finish<S>(P, kvh, head0 + (tid < rows_here ? tid : 0), top, den, mul, lse);
      s_mul[tid] = mul;                                // read after the slices' barrier
      if (tid < rows_here && P.lse) P.lse[(size_t)cc.r * P.heads + head0 + tid] = lse;
    }
  }
  float mine_f[NT][2];      // this warp's factor per column
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = n * 8 + 2 * t4 + i;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * S::kRows + h]);
      mine_f[n][i] = m[n][i] == -INFINITY ? 0.f : exp2_fast(m[n][i] - top);
    }
#pragma unroll
  for (int sl = 0; sl < D / S::kSlice; ++sl) {
    constexpr int kDt = S::kSlice / 16;
#pragma unroll
    for (int dd = 0; dd < kDt; ++dd)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = n * 8 + 2 * t4 + (i & 1);
          const int d = dd * 16 + (k8 ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
          s_sum[(wid * S::kRows + h) * S::kPitch + d] =
              o[sl * kDt + dd][n][i] * mine_f[n][i & 1];
        }
    __syncthreads();
    for (int e = tid; e < S::kRows * S::kSlice / 2; e += S::kThreads) {
      const int h = e / (S::kSlice / 2), d = e % (S::kSlice / 2) * 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v =
            *reinterpret_cast<const float2*>(s_sum + (w * S::kRows + h) * S::kPitch + d);
        x += v.x;
        y += v.y;
      }
      if (!alone)
        *reinterpret_cast<float2*>(po + h * D + sl * S::kSlice + d) = make_float2(x, y);
      else if (h < rows_here)
        store_out(P, cc.r, head0 + h, D, sl * S::kSlice + d, x * s_mul[h], y * s_mul[h]);
    }
    __syncthreads();
  }
  if (!alone && tid == 0) s_last[which] = arrive(cc);
  __syncthreads();
  // ---- rows of several shares whose last piece was written here ----
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (!s_last[e]) continue;
    const Item<S> it = item_at<S>(P, s_prefix, s_order, s_len, per, e ? c1 - 1 : c0);
    join_row<S>(P, it, rt, U, pieces_of(it), s_sum, s_mul);
  }
  if (bad) atomicOr(P.err, bad);
}

template <class S>
cudaError_t configure() {
  return cudaFuncSetAttribute(attend_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              S::kSmem);
}
template <class S>
void launch(const Params& P, const moe_reader_kv& kv, const moe_reader_kv_attend_args& a,
            cudaStream_t s) {
  // one CTA per SM, fewer where even full tables cannot fill them
  const long long keys = (long long)(a.pages ? a.keep : a.width) << P.shift;
  const long long tiles = (keys + S::kKeys - 1) / S::kKeys * a.requests * P.kv_heads;
  const int grid = P.row_tiles * (int)std::min<long long>(std::max(1, kv.sms / P.row_tiles),
                                                         (tiles + S::kWarps - 1) / S::kWarps);
  launch_early(attend_kernel<S>, dim3(grid), S::kThreads, S::kSmem, s, P);
}

// Tiles of eight query heads per item: both where the group has more than eight
// heads and the accumulators of 16 fit the registers (D <= 128).
int head_tiles(const moe_reader_kv_config& c) {
  const int group = c.num_q_heads / c.num_kv_heads;
  return group > 8 && c.head_dim <= 128 ? 2 : 1;
}

// Calls f with the Shape of a handle.
template <class F>
auto with_shape(const moe_reader_kv_config& c, F f) {
  const int nt = head_tiles(c);
  auto typed = [&](auto d, auto n) {
    constexpr int D = decltype(d)::value, N = decltype(n)::value;
    switch (c.cache_type) {
      case kBf16: return f(Shape<D, N, kBf16>{});
      case kF16: return f(Shape<D, N, kF16>{});
      default: return f(Shape<D, N, kE4m3>{});
    }
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  using I256 = std::integral_constant<int, 256>;
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (c.head_dim == 64) return nt == 1 ? typed(I64{}, One{}) : typed(I64{}, Two{});
  if (c.head_dim == 128) return nt == 1 ? typed(I128{}, One{}) : typed(I128{}, Two{});
  return typed(I256{}, One{});
}

}  // namespace

int attend_row_tiles(const moe_reader_kv_config& c) {
  const int rows = 8 * head_tiles(c);
  return (c.num_q_heads / c.num_kv_heads + rows - 1) / rows;
}

cudaError_t configure_kv_attend(const moe_reader_kv& kv) {
  return with_shape(kv.cfg, [](auto s) { return configure<decltype(s)>(); });
}

cudaError_t launch_kv_attend(const moe_reader_kv& kv, const moe_reader_kv_attend_args& a,
                             cudaStream_t s) {
  Params P;
  P.q = a.q;
  P.table = a.table;
  P.lens = a.lens;
  P.pages = a.pages;
  P.sinks = a.sinks;
  P.out = a.out;
  P.lse = a.lse;
  P.q_request = a.q_request_stride;
  P.q_head = a.q_head_stride;
  P.q_type = a.q_type;
  P.q_pairs = reinterpret_cast<uintptr_t>(a.q) % 4 == 0 && a.q_request_stride % 2 == 0 &&
              a.q_head_stride % 2 == 0;
  P.requests = a.requests;
  P.width = a.width;
  P.keep = a.keep;
  P.window = a.window;
  P.scale = a.scale;
  P.k = static_cast<const char*>(kv.k);
  P.v = static_cast<const char*>(kv.v);
  P.k_scale = kv.k_scale;
  P.v_scale = kv.v_scale;
  P.heads = kv.cfg.num_q_heads;
  P.kv_heads = kv.cfg.num_kv_heads;
  P.group = kv.group;
  P.row_tiles = attend_row_tiles(kv.cfg);
  P.shift = kv.page_shift;
  P.num_pages = kv.cfg.num_pages;
  P.part_o = kv.part_o;
  P.part_ml = kv.part_ml;
  P.arrived = kv.arrived;
  P.err = kv.err;
  const bool stall = take_attend_stall();
  P.polls = stall ? 1 << 12 : 1 << 21;
  P.stall = stall ? 1u << 30 : 0u;
  with_shape(kv.cfg, [&](auto sh) { launch<decltype(sh)>(P, kv, a, s); return 0; });
  return cudaGetLastError();
}

}  // namespace mr
