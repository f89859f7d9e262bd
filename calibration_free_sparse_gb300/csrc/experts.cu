// A prompt's experts: pairs (token, slot) sorted by expert, and products grouped
// by expert over ragged numbers of rows.
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "device_util.cuh"
#include "internal.cuh"
#include "kv.cuh"
#include "moe_reader.h"
#include "tc.cuh"

struct moe_reader_experts {
  moe_reader_experts_config cfg;
  int device;
  int sms;
  const void* gate;          // caller-owned [E][I][H]
  const void* up;
  const void* down;          // caller-owned [E][H][I]
  CUtensorMap gate_map, up_map, down_map;
  uint32_t* err;             // [1] device error word
};

namespace mr {
namespace {

constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// CTA e lists the pairs of expert e, the last CTA those that belong to none.
// Each counts for itself the pairs of the experts before its own (one pass over
// the ids, from L2) and then writes its own in order: one launch, no hand-off
// between CTAs, and the order does not depend on their timing.  A warp has a run
// of the pairs, so that one barrier between counting and writing is enough (a
// barrier every 512 pairs took 29 us for 4096 tokens of 8), a lane four on end.
__global__ void __launch_bounds__(kPlanThreads)
experts_plan_kernel(moe_reader_experts_plan_args a) {
  __shared__ int s_before[kPlanThreads / 32], s_mine[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int e = blockIdx.x, E = a.num_experts;
  wait_for_earlier_launch();
  const long long pairs = (long long)a.tokens * a.experts_per_token;
  const long long run = (pairs + kPlanThreads / 32 * 128 - 1) / (kPlanThreads / 32 * 128) * 128;
  const long long lo = wid * run, hi = min(lo + run, pairs);
  const bool wide = reinterpret_cast<uintptr_t>(a.ids) % 16 == 0;
  // four ids from pair i on; those of no expert are E, those behind the last -1
  auto four = [&](long long i, int (&id)[4]) {
    if (wide && i + 4 <= hi) {
      const int4 v = __ldg(reinterpret_cast<const int4*>(a.ids + i));
      id[0] = v.x, id[1] = v.y, id[2] = v.z, id[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) id[j] = i + j < hi ? __ldg(a.ids + i + j) : 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if ((unsigned)id[j] >= (unsigned)E) id[j] = E;
      if (i + j >= hi) id[j] = -1;
    }
  };
  int before = 0, mine = 0;
#pragma unroll 4
  for (long long i = lo + 4 * lane; i < hi; i += 128) {
    int id[4];
    four(i, id);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      before += id[j] >= 0 && id[j] < e;
      mine += id[j] == e;
    }
  }
  before = warp_sum_i(before);
  mine = warp_sum_i(mine);
  if (lane == 0) s_before[wid] = before, s_mine[wid] = mine;
  __syncthreads();
  before = warp_sum_i(s_before[lane]);
  const int ahead = warp_sum_i(lane < wid ? s_mine[lane] : 0), all = warp_sum_i(s_mine[lane]);
  if (tid == 0) {
    a.offsets[e] = before;
    if (e == E) a.skipped[0] = all;
  }
  if (mine == 0) return;
  int at = before + ahead;
  for (long long b = lo; b < hi; b += 128) {
    int id[4], rank = at, n = 0;
    four(b + 4 * lane, id);
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool is = id[j] == e;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      rank += __popc(m & ((1u << lane) - 1));
      n += __popc(m);
      own |= (uint32_t)is << j;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!(own >> j & 1)) continue;
      const long long i = b + 4 * lane + j;
      a.order[rank] = e < E ? (int)i : -1;
      a.places[i] = e < E ? rank : -1;
      rank++;
    }
    at += n;
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// The weights' rows lie on the tensor core's 128 rows and the plan's rows on
// its columns, of which a product may have any multiple of 16: ragged numbers
// of rows cost few columns of nothing, and an expert with three tokens is read
// at the speed of its weights.  A tile is 2 x 128 weight rows (gate and up of
// 128 channels; 256 channels of down) by up to N plan rows; a persistent CTA per SM
// takes tiles in turn.  One warp brings weights by tensor copies, one the
// activations or eight the tokens, one issues the products, eight write a
// finished tile out while the next one is summed (two sets of accumulators where
// they fit).
//
// Measured on a GB300: activations of 57 tokens, 128 experts of 2048 x 768, 8 a
// token: 106 to 114 us with the plan, 7 TB/s: HBM.  4096 tokens: 205 us, 1.0
// PFLOP/s, and down products of 2000 tokens, 32 experts of 2880 x 2880: 140 us, 0.95:
// both at 13 to 14 TB/s from L2 to the SMs (tiles of 128 columns: 276 us and 173).
constexpr int kBoxBytes = 128 * 128;          // 128 weight rows of 64 values

template <int N> struct GroupShape {
  static constexpr int kStageBytes = 2 * kBoxBytes + N * 128;
  static constexpr int kStages = N >= 256 ? 3 : N >= 128 ? 4 : N >= 64 ? 5 : 6;
  static constexpr int kLag = kStages - 2;             // copies under way behind the newest
  static constexpr int kRowBox = N < 64 ? N : 64;      // plan rows of a tensor copy
  static constexpr int kSets = N <= 128 ? 2 : 1;       // sets of accumulators
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024;
};

struct GroupArgs {
  const void* in;            // rows of the right operand
  long long in_stride;       // elements
  const int32_t* order;      // the pair of each row (in = token rows), or null (in = plan rows)
  const int32_t* offsets;
  void* out;                 // act, or slots
  int experts, k, channels;  // channels: I, or H
  int pairs, topk;
  int stall;                 // wait for a product that was never issued
};

// Warps: weights, products, activations, none; eight write out; eight bring tokens.
template <bool kAct> constexpr int group_threads() { return kAct ? 640 : 384; }

template <int N, bool kBf16, bool kAct>
__global__ void __launch_bounds__(group_threads<kAct>(), 1)
group_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
             const __grid_constant__ CUtensorMap in_map, GroupArgs a, uint32_t* err) {
  using S = GroupShape<N>;
  extern __shared__ char raw[];
  __shared__ int s_first[kMaxExperts + 1], s_tiles[kMaxExperts + 1];
  __shared__ uint64_t s_bar[3 * S::kStages + 2 * S::kSets + 1];
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_quit;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t base = (tc::smem_at(raw) + 1023) & ~1023u, bars = tc::smem_at(s_bar);
  auto stage_at = [&](int s) { return base + s * S::kStageBytes; };
  auto weights_in = [&](int s) { return bars + 8 * s; };
  auto rows_in = [&](int s) { return bars + 8 * (S::kStages + s); };
  auto stage_free = [&](int s) { return bars + 8 * (2 * S::kStages + s); };
  auto sums_done = [&](int s) { return bars + 8 * (3 * S::kStages + s); };
  auto sums_free = [&](int s) { return bars + 8 * (3 * S::kStages + S::kSets + s); };
  const uint32_t drained = bars + 8 * (3 * S::kStages + 2 * S::kSets);

  if (wid == 0) tc::prefetch_map(&map0), tc::prefetch_map(&map1);
  wait_for_earlier_launch();
  let_next_launch_start();
  // the experts' first rows and tiles
  for (int e = tid; e <= a.experts; e += group_threads<kAct>())
    s_first[e] = min(max(__ldg(a.offsets + e), 0), a.pairs);
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      tc::bar_init(weights_in(s), 1);
      tc::bar_init(rows_in(s), kAct ? 256 : 1);
      tc::bar_init(stage_free(s), 1);
    }
    for (int s = 0; s < S::kSets; ++s) {
      tc::bar_init(sums_done(s), 1);
      tc::bar_init(sums_free(s), 256);
    }
    tc::bar_init(drained, 1);
    s_quit = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (wid == 1) tc::tmem_alloc(tc::smem_at(&s_tmem), 512);
  __syncthreads();
  const int per_tile = kAct ? 128 : 256;
  const int m_tiles = (a.channels + per_tile - 1) / per_tile;
  if (wid == 0) {
    int sum = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < a.experts) n = (max(s_first[e + 1] - s_first[e], 0) + N - 1) / N * m_tiles;
      int at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += u;
      }
      if (e <= a.experts) s_tiles[e] = sum + at - n;
      sum += __shfl_sync(0xffffffffu, at, 31);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  const int tiles = s_tiles[a.experts];
  const int k_steps = (a.k + 63) / 64;

  struct Tile {
    int expert, m, first, rows;      // weight tile, first plan row and number of them
  };
  auto tile_at = [&](int t) {
    int lo = 0, hi = a.experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tiles[mid] <= t) lo = mid; else hi = mid - 1;
    }
    // an expert's rows in tiles of about one size
    const int all = s_first[lo + 1] - s_first[lo], n_tiles = (all + N - 1) / N;
    const int at = t - s_tiles[lo], m = at / n_tiles, n = at - m * n_tiles;
    const int size = ((all + n_tiles - 1) / n_tiles + 15) & ~15, from = min(n * size, all);
    return Tile{lo, m, s_first[lo] + from, min(size, all - from)};
  };

  if (wid == 0) {
    // weights
    int s = 0, used = 0;
    uint32_t phase = 1;
    if (lane == 0) {
      for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const Tile x = tile_at(t);
        for (int k = 0; k < k_steps; ++k) {
          if (!tc::bar_wait(stage_free(s), phase, &s_quit)) goto weights_end;
          tc::bar_expect(weights_in(s), 2 * kBoxBytes);
          tc::load_box(stage_at(s), &map0, k * 64, x.m * per_tile, x.expert, weights_in(s));
          tc::load_box(stage_at(s) + kBoxBytes, &map1, k * 64,
                       x.m * per_tile + (kAct ? 0 : 128), x.expert, weights_in(s));
          used++;
          if (++s == S::kStages) s = 0, phase ^= 1;
        }
      }
    weights_end:
      // no copy is left under way
      for (int i = 0; i < min(used, S::kStages); ++i) {
        if (--s < 0) s = S::kStages - 1, phase ^= 1;
        volatile uint32_t ignore = 0;
        tc::bar_wait(weights_in(s), phase ^ 1, &ignore);
      }
    }
    __syncwarp();
  } else if (wid == 1) {
    // products
    int s = 0, set = 0;
    uint32_t phase = 0, set_phase = 1;
    bool go = !a.stall || tc::bar_wait(drained, 0, &s_quit);
    for (int t = blockIdx.x; go && t < tiles; t += gridDim.x) {
      const Tile x = tile_at(t);
      const uint32_t idesc = tc::instr<kBf16>((x.rows + 15) & ~15);
      const uint32_t d = tmem + set * 2 * N;
      if (!(go = tc::bar_wait(sums_free(set), set_phase, &s_quit))) break;
      tc::fence_after();
      for (int k = 0; k < k_steps; ++k) {
        if (!(go = tc::bar_wait(weights_in(s), phase, &s_quit) &&
                   tc::bar_wait(rows_in(s), phase, &s_quit)))
          break;
        tc::fence_after();
        const uint64_t a0 = tc::desc_k(stage_at(s)), a1 = tc::desc_k(stage_at(s) + kBoxBytes);
        const uint64_t b = tc::desc_k(stage_at(s) + 2 * kBoxBytes);
        const uint32_t bar = stage_free(s), last = k == k_steps - 1 ? sums_done(set) : 0;
        if (tc::elected()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tc::mma(d, a0 + 2 * i, b + 2 * i, idesc, k + i > 0);
            tc::mma(d + N, a1 + 2 * i, b + 2 * i, idesc, k + i > 0);
          }
          tc::commit(bar);
          if (last) tc::commit(last);
        }
        __syncwarp();
        if (++s == S::kStages) s = 0, phase ^= 1;
      }
      if (!go) break;
      if (++set == S::kSets) set = 0, set_phase ^= 1;
    }
    if (tc::elected()) tc::commit(drained);
    __syncwarp();
    volatile uint32_t ignore = 0;
    tc::bar_wait(drained, 0, &ignore);
  } else if (wid == 2 && !kAct) {
    // activations: the plan's rows on end, by tensor copies too (what they bring
    // of the next expert's is not multiplied)
    int s = 0, used = 0;
    uint32_t phase = 1;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile x = tile_at(t);
      const int boxes = (x.rows + S::kRowBox - 1) / S::kRowBox;
      for (int k = 0; k < k_steps; ++k) {
        if (!tc::bar_wait(stage_free(s), phase, &s_quit)) goto rows_end;
        if (tc::elected()) {
          tc::bar_expect(rows_in(s), boxes * S::kRowBox * 128);
          for (int i = 0; i < boxes; ++i)
            tc::load_box(stage_at(s) + 2 * kBoxBytes + i * S::kRowBox * 128, &in_map, k * 64,
                         x.first + i * S::kRowBox, 0, rows_in(s));
        }
        __syncwarp();
        used++;
        if (++s == S::kStages) s = 0, phase ^= 1;
      }
    }
  rows_end:
    // no copy is left under way
    for (int i = 0; i < min(used, S::kStages); ++i) {
      if (--s < 0) s = S::kStages - 1, phase ^= 1;
      volatile uint32_t ignore = 0;
      tc::bar_wait(rows_in(s), phase ^ 1, &ignore);
    }
  } else if (wid >= 12) {
    // Tokens, wherever they stand: eight lanes copy a row's 128 bytes, 32 rows at
    // once.  (Tensor copies of four rows take about 50 cycles each, one after the
    // other: 64 of them took three times a stage's products.)
    const int id = tid - 384, piece = id & 7, sub = id >> 3;
    int s = 0, late = 0, behind = 0;       // `late`: oldest stage not yet handed over
    uint32_t phase = 1;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile x = tile_at(t);
      const int n16 = (x.rows + 15) & ~15;
      constexpr int kTurns = (N + 31) / 32;
      const char* from[kTurns];
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int r = i * 32 + sub;
        long long at = 0;
        if (r < x.rows) {
          const int pair = __ldg(a.order + x.first + r);
          if ((unsigned)pair < (unsigned)a.pairs) in |= 1u << i, at = pair / a.topk;
        }
        from[i] = static_cast<const char*>(a.in) + at * a.in_stride * 2 + piece * 16;
      }
      for (int k = 0; k < k_steps; ++k) {
        if (!tc::bar_wait(stage_free(s), phase, &s_quit)) goto tokens_end;
        const uint32_t to = stage_at(s) + 2 * kBoxBytes + tc::swizzled(sub, piece);
        const bool k_in = k * 64 + piece * 8 < a.k;
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
          if (i * 32 + sub < n16) {
            const bool there = k_in && (in >> i & 1);
            tc::copy16(to + i * 4096, there ? from[i] + k * 128 : from[i] - piece * 16, there);
          }
        tc::copies_commit();
        if (behind == S::kLag) {
          tc::copies_wait<S::kLag>();
          tc::publish_smem();
          tc::bar_arrive(rows_in(late));
          if (++late == S::kStages) late = 0;
        } else {
          behind++;
        }
        if (++s == S::kStages) s = 0, phase ^= 1;
      }
    }
  tokens_end:
    tc::copies_wait<0>();
    tc::publish_smem();
    for (; behind > 0; --behind) {
      tc::bar_arrive(rows_in(late));
      if (++late == S::kStages) late = 0;
    }
  } else if (wid >= 4) {
    // a finished tile: a thread has one channel (row) and half of the columns
    const int quarter = wid & 3, half = (wid - 4) >> 2;
    int set = 0;
    uint32_t set_phase = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile x = tile_at(t);
      if (!tc::bar_wait(sums_done(set), set_phase, &s_quit)) break;
      tc::fence_after();
      const int n16 = (x.rows + 15) >> 4;
      const int ch = x.m * per_tile + quarter * 32 + lane;
      const uint32_t at = tmem + set * 2 * N + ((uint32_t)(quarter * 32) << 16);
      for (int c = half; c < n16; c += 2) {
        uint32_t u[16], v[16];
        tc::ld16(at + c * 16, u);
        tc::ld16(at + N + c * 16, v);
        tc::ld_wait();
        const int left = x.rows - c * 16;
        const long long row = x.first + c * 16;
        if constexpr (kAct) {
          // silu(gate) * up in fp32, rounded once
          uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.channels + ch;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = __uint_as_float(u[i]), g = __uint_as_float(v[i]);
            const float y = __fdividef(f, 1.f + __expf(-f)) * g;
            uint16_t bits;
            if constexpr (kBf16) bits = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            else bits = __half_as_ushort(__float2half_rn(y));
            if (i < left && ch < a.channels) *out = bits;
            out += a.channels;
          }
        } else {
          float* out = static_cast<float*>(a.out) + row * a.channels + ch;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (i < left && ch < a.channels) out[0] = __uint_as_float(u[i]);
            if (i < left && ch + 128 < a.channels) out[128] = __uint_as_float(v[i]);
            out += a.channels;
          }
        }
      }
      tc::fence_before();
      tc::bar_arrive(sums_free(set));
      if (++set == S::kSets) set = 0, set_phase ^= 1;
    }
  }
  __syncthreads();
  if (wid == 1) tc::tmem_free(tmem, 512);
  if (tid == 0 && s_quit) atomicOr(err, kErrTimeout);
}

// y_t: a thread has four columns of a token and adds its slots in order.  The
// products wait in fp32: 2000 tokens of 4 x 2880 take 19 us of 160 (92 MB), and
// adding them where they are made would leave their order to chance.
template <int T>
__global__ void __launch_bounds__(256)
combine_kernel(moe_reader_experts_combine_args a, int H, int topk) {
  const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  wait_for_earlier_launch();
  if (c >= H) return;
  const int pairs = a.tokens * topk;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < topk; ++s) {
    const int row = __ldg(a.places + (long long)t * topk + s);
    if ((unsigned)row >= (unsigned)pairs) continue;
    const float w = __ldg(a.weights + (long long)t * topk + s);
    const float4 z = *reinterpret_cast<const float4*>(a.slots + (long long)row * H + c);
    y.x += w * z.x;
    y.y += w * z.y;
    y.z += w * z.z;
    y.w += w * z.w;
  }
  const long long at = t * a.y_stride + c;
  if constexpr (T == MOE_READER_TYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = y;
  } else if constexpr (T == MOE_READER_TYPE_BF16) {
    __nv_bfloat162 v[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
        *reinterpret_cast<const uint2*>(v);
  } else {
    __half2 v[2] = {__floats2half2_rn(y.x, y.y), __floats2half2_rn(y.z, y.w)};
    *reinterpret_cast<uint2*>(static_cast<__half*>(a.y) + at) = *reinterpret_cast<const uint2*>(v);
  }
}

template <int N, bool kBf16, bool kAct>
cudaError_t group_as(const moe_reader_experts& h, const GroupArgs& a, cudaStream_t s) {
  const CUtensorMap& m0 = kAct ? h.gate_map : h.down_map;
  const CUtensorMap& m1 = kAct ? h.up_map : h.down_map;
  CUtensorMap in = {};
  if (!kAct) {
    const uint64_t sizes[3] = {(uint64_t)a.k, (uint64_t)a.pairs, 1};
    const uint64_t strides[2] = {(uint64_t)a.k, (uint64_t)a.k * a.pairs};
    const uint32_t box[3] = {64, (uint32_t)GroupShape<N>::kRowBox, 1};
    const cudaError_t e = tc::make_map(&in, a.in, kBf16, 3, sizes, strides, box);
    if (e != cudaSuccess) return e;
  }
  return launch_early(group_kernel<N, kBf16, kAct>, dim3(h.sms), group_threads<kAct>(),
                      GroupShape<N>::kSmem, s, m0, m1, in, a, h.err);
}

// Columns of a tile: about as many as an expert has rows on average.  A tile of
// more leaves less shared memory for the weights under way, one of fewer reads
// them again: 4096 tokens with 256 rows an expert take 276 us in tiles of 128
// columns and 241 in tiles of 256.
template <bool kBf16, bool kAct>
cudaError_t group(const moe_reader_experts& h, const GroupArgs& a, cudaStream_t s) {
  const int mean = a.pairs / a.experts;
  if (mean <= 32) return group_as<32, kBf16, kAct>(h, a, s);
  if (mean <= 64) return group_as<64, kBf16, kAct>(h, a, s);
  if (mean <= 112) return group_as<128, kBf16, kAct>(h, a, s);
  return group_as<256, kBf16, kAct>(h, a, s);
}

template <bool kBf16>
cudaError_t activate_as(const moe_reader_experts& h, const moe_reader_experts_activate_args& a,
                        cudaStream_t s) {
  const GroupArgs g = {a.x, a.x_stride, a.order, a.offsets, a.act,
                       h.cfg.num_experts, h.cfg.hidden, h.cfg.inter,
                       a.tokens * a.experts_per_token, a.experts_per_token, take_prompt_stall()};
  return group<kBf16, true>(h, g, s);
}

template <bool kBf16>
cudaError_t combine_as(const moe_reader_experts& h, const moe_reader_experts_combine_args& a,
                       cudaStream_t s) {
  const int H = h.cfg.hidden, topk = a.experts_per_token;
  const GroupArgs g = {a.act, h.cfg.inter, nullptr, a.offsets,
                       a.slots, h.cfg.num_experts, h.cfg.inter, H, a.tokens * topk, topk,
                       take_prompt_stall()};
  const cudaError_t e = group<kBf16, false>(h, g, s);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.tokens, (unsigned)((H + 1023) / 1024));
  switch (a.y_type) {
    case MOE_READER_TYPE_BF16:
      return launch_early(combine_kernel<MOE_READER_TYPE_BF16>, grid, 256, 0, s, a, H, topk);
    case MOE_READER_TYPE_F16:
      return launch_early(combine_kernel<MOE_READER_TYPE_F16>, grid, 256, 0, s, a, H, topk);
    default:
      return launch_early(combine_kernel<MOE_READER_TYPE_F32>, grid, 256, 0, s, a, H, topk);
  }
}

template <int N, bool kBf16, bool kAct>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(group_kernel<N, kBf16, kAct>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)GroupShape<N>::kSmem);
}
template <bool kBf16, bool kAct>
cudaError_t configure_group() {
  cudaError_t e = configure_one<32, kBf16, kAct>();
  if (e == cudaSuccess) e = configure_one<64, kBf16, kAct>();
  if (e == cudaSuccess) e = configure_one<128, kBf16, kAct>();
  if (e == cudaSuccess) e = configure_one<256, kBf16, kAct>();
  return e;
}
cudaError_t configure_experts(moe_reader_experts& h) {
  const bool bf16 = h.cfg.type == MOE_READER_TYPE_BF16;
  const uint64_t H = h.cfg.hidden, I = h.cfg.inter, E = h.cfg.num_experts;
  cudaError_t e = cudaSuccess;
  auto map = [&](CUtensorMap* m, const void* w, uint64_t rows, uint64_t cols) {
    const uint64_t sizes[3] = {cols, rows, E}, strides[2] = {cols, rows * cols};
    const uint32_t box[3] = {64, 128, 1};
    return tc::make_map(m, w, bf16, 3, sizes, strides, box);
  };
  if (h.gate) {
    e = map(&h.gate_map, h.gate, I, H);
    if (e == cudaSuccess) e = map(&h.up_map, h.up, I, H);
    if (e == cudaSuccess) e = bf16 ? configure_group<true, true>() : configure_group<false, true>();
  }
  if (e == cudaSuccess && h.down) {
    e = map(&h.down_map, h.down, H, I);
    if (e == cudaSuccess)
      e = bf16 ? configure_group<true, false>() : configure_group<false, false>();
  }
  return e;
}

}  // namespace
}  // namespace mr

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
namespace {

bool at_multiple(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

using mr::status_of;

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
  // (tensor maps want 64-byte alignment)
  moe_reader_experts* h = static_cast<moe_reader_experts*>(
      aligned_alloc(alignof(moe_reader_experts), sizeof(moe_reader_experts)));
  if (!h) return MOE_READER_ENOMEM;
  memset(h, 0, sizeof(moe_reader_experts));
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
    if ((ce = mr::configure_experts(*h)) != cudaSuccess) break;
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
  return status_of(mr::launch_early(mr::experts_plan_kernel, dim3(a->num_experts + 1),
                                    mr::kPlanThreads, 0, static_cast<cudaStream_t>(stream), *a));
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
                       ? mr::activate_as<true>(*h, *a, s)
                       : mr::activate_as<false>(*h, *a, s));
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
                       ? mr::combine_as<true>(*h, *a, s)
                       : mr::combine_as<false>(*h, *a, s));
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
