// Pages of the paged cache: which ones requests hold (collect), rows that share
// another row's pages (fork), the pages in use moved to the front of the pool
// (compact), and the copies that the last two ask for (copy).
#include <algorithm>

#include "device_util.cuh"
#include "internal.cuh"
#include "kv.cuh"

namespace mr {
namespace {

constexpr uint32_t kErrRow = MOE_READER_ERR_ROW;

// ---------------------------------------------------------------------------
// collect, compact
// ---------------------------------------------------------------------------
constexpr int kPoolCtas = 16;         // one cluster
constexpr int kPoolThreads = 1024;
// Pools and tables up to these sizes take one CTA, which counts in its shared
// memory.
constexpr int kSmallPool = 16384, kSmallTable = 8192;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; what they wrote to global and shared memory
// before can be seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
               : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)));
  return at;
}
__device__ __forceinline__ void put_cluster(uint32_t at, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ int get_cluster(uint32_t at) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Pages that a row holds.
__device__ __forceinline__ int held_pages(int len, int width, int shift, uint32_t& bad) {
  if (len < 0) bad |= kErrLength, len = 0;
  const int held = (int)(((long long)len + (1 << shift) - 1) >> shift);
  if (held > width) bad |= kErrLength;
  return min(held, width);
}

// Counts references, ranks the pages in use and the free ones by ballots, and
// (compact) pairs the k-th page in use behind the first `used` with the k-th
// free one among them.  Each phase needs all of the one before, so the grid is
// one cluster and its hardware barrier separates them, or one CTA where the pool
// is small (a barrier of the cluster and the trips to L2 between two took the
// most time: 2660 pages of 16 rows 10.8 us, 6.2 with one CTA; 10 thousand of 512
// rows 10.4 and 14.5): one launch, no counters
// that live between calls.  Warp w of the grid owns a run of the pool; ranks
// before a run are sums over the warps' totals, gathered in the first CTA.
// Between the phases free_pages holds the sources' ranks.
template <bool kCompact, int kCtas>
__global__ void __launch_bounds__(kPoolThreads)
pool_kernel(moe_reader_kv_pages_args a, int shift, int pool, uint32_t* err) {
  constexpr int kPoolWarps = kCtas * kPoolThreads / 32;
  extern __shared__ int s_refs[];       // one CTA: the references
  int* const refs = kCtas == 1 ? s_refs : a.refs;
  auto refs_of = [&](long long p) { return kCtas == 1 ? s_refs[p] : __ldcg(a.refs + p); };
  auto sync = [&]() {
    if (kCtas == 1) __syncthreads(); else cluster_sync();
  };
  __shared__ int s_total[kPoolWarps];   // the first CTA's: pages in use per warp's run
  __shared__ int s_front;               // the first CTA's: pages in use among the first `used`
  __shared__ int s_before[kPoolThreads / 32], s_used;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int cta = kCtas == 1 ? 0 : (int)cluster_rank(), warp = cta * (kPoolThreads / 32) + wid;
  const long long first = (long long)cta * kPoolThreads + threadIdx.x;
  constexpr long long kAll = (long long)kCtas * kPoolThreads;
  uint32_t bad = 0;
  wait_for_earlier_launch();

  for (long long p = first; p < pool; p += kAll) refs[p] = 0;
  sync();
  for (int r = warp; r < a.requests; r += kPoolWarps) {
    const int held = held_pages(__ldg(a.lens + r), a.width, shift, bad);
    for (int c = lane; c < held; c += 32) {
      const int p = a.table[(size_t)r * a.width + c];
      if ((unsigned)p < (unsigned)pool) atomicAdd(refs + p, 1);
      else bad |= kErrPage;
    }
  }
  sync();

  const int per = (int)(((long long)pool + kPoolWarps * 32 - 1) / (kPoolWarps * 32)) * 32;
  const long long lo = (long long)warp * per, hi = min(lo + per, (long long)pool);
  int mine = 0;
  for (long long p = lo; p < hi; p += 32)
    mine += __popc(__ballot_sync(0xffffffffu, p + lane < hi && refs_of(p + lane) > 0));
  if (lane == 0) put_cluster(in_first_cta(s_total + warp), mine);
  sync();
  // pages in use before this CTA's warps, and in all
  if (wid == 0) {
    int before = 0, all = 0;
    for (int w = lane; w < kPoolWarps; w += 32) {
      const int n = get_cluster(in_first_cta(s_total + w));
      all += n;
      if (w < cta * (kPoolThreads / 32)) before += n;
    }
    before = warp_sum_i(before);
    all = warp_sum_i(all);
    int at = get_cluster(in_first_cta(s_total + cta * (kPoolThreads / 32) + lane));
    const int own = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += u;
    }
    s_before[lane] = before + at - own;
    if (lane == 0) s_used = all;
  }
  __syncthreads();
  const int used = s_used, before = s_before[wid];

  if constexpr (kCompact) {
    // pages in use among the first `used`: counted by the warp that owns page `used`
    if (used >= lo && used < hi) {
      int n = before;
      for (long long p = lo; p < used; p += 32)
        n += __popc(__ballot_sync(0xffffffffu, p + lane < used && refs_of(p + lane) > 0));
      if (lane == 0) put_cluster(in_first_cta(&s_front), n);
    } else if (warp == 0 && used == pool && lane == 0) {
      put_cluster(in_first_cta(&s_front), used);
    }
    sync();
    const int front = get_cluster(in_first_cta(&s_front)), moves = used - front;
    int n = before;
    for (long long p = lo; p < hi; p += 32) {
      const bool in = p + lane < hi;
      const bool use = in && refs_of(p + lane) > 0;
      const uint32_t uses = __ballot_sync(0xffffffffu, use);
      const int id = (int)p + lane, rank = n + __popc(uses & ((1u << lane) - 1));
      if (in && use && id >= used) {
        a.src[rank - front] = id;
        a.free_pages[id] = rank - front;
      }
      if (in && !use && id < used) a.dst[id - rank] = id;
      n += __popc(uses);
    }
    for (long long k = moves + first; k < pool / 2; k += kAll) a.src[k] = a.dst[k] = -1;
    if (first == 0) {
      a.moves[0] = moves;
      a.count[0] = pool - used;
    }
    sync();
    for (int r = warp; r < a.requests; r += kPoolWarps) {
      uint32_t known = 0;
      const int held = held_pages(__ldg(a.lens + r), a.width, shift, known);
      for (int c = lane; c < held; c += 32) {
        int32_t* e = a.table + (size_t)r * a.width + c;
        const int p = *e;
        if (p >= used && p < pool) *e = __ldcg(a.dst + __ldcg(a.free_pages + p));
      }
    }
    for (long long k = first; k < moves; k += kAll) {
      const int s = __ldcg(a.src + k);
      refs[__ldcg(a.dst + k)] = refs_of(s);
      refs[s] = 0;
    }
    sync();
    for (long long i = first; i < pool; i += kAll)
      a.free_pages[i] = i < pool - used ? (int)(used + i) : -1;
  } else {
    int n = before;
    for (long long p = lo; p < hi; p += 32) {
      const bool in = p + lane < hi;
      const bool use = in && refs_of(p + lane) > 0;
      const uint32_t uses = __ballot_sync(0xffffffffu, use);
      const int id = (int)p + lane, rank = n + __popc(uses & ((1u << lane) - 1));
      if (in && !use) a.free_pages[id - rank] = id;
      n += __popc(uses);
    }
    for (long long i = pool - used + first; i < pool; i += kAll) a.free_pages[i] = -1;
    if (first == 0) a.count[0] = pool - used;
    sync();       // no CTA ends while others read the first one's memory
  }
  if (kCtas == 1) {
    __syncthreads();
    for (long long p = first; p < pool; p += kAll) a.refs[p] = s_refs[p];
  }
  if (bad) atomicOr(err, bad);
}

template <bool kCompact>
cudaError_t launch_pool(const moe_reader_kv& kv, const moe_reader_kv_pages_args& a,
                        cudaStream_t s) {
  const int pool = kv.cfg.num_pages;
  if (pool <= kSmallPool && (long long)a.requests * a.width <= kSmallTable)
    return launch_early(pool_kernel<kCompact, 1>, dim3(1), kPoolThreads, pool * sizeof(int), s, a,
                        kv.page_shift, pool, kv.err);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPoolCtas);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kPoolCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pool_kernel<kCompact, kPoolCtas>, a, kv.page_shift, pool, kv.err);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 256;

// A CTA per fork (512 rows 6.3 us, 4 rows 3.1).  Each finds out for itself which forks hold (at most 1024 of
// them) and how many fresh pages those before its own take: one launch and no
// hand-off between CTAs.
__global__ void __launch_bounds__(kForkThreads)
fork_kernel(moe_reader_kv_fork_args a, int shift, int pool, uint32_t* err) {
  __shared__ int s_first[kMaxRequests];       // a row's first fork as a child
  __shared__ uint8_t s_parent[kMaxRequests];  // a row is some fork's parent
  __shared__ int s_before, s_all;
  const int tid = threadIdx.x, mine = blockIdx.x, ps = 1 << shift;
  wait_for_earlier_launch();
  for (int r = tid; r < a.rows; r += kForkThreads) s_first[r] = a.forks, s_parent[r] = 0;
  if (tid == 0) s_before = s_all = 0;
  __syncthreads();
  auto in = [&](int r) { return (unsigned)r < (unsigned)a.rows; };
  for (int i = tid; i < a.forks; i += kForkThreads) {
    const int p = __ldg(a.parents + i), c = __ldg(a.children + i);
    if (in(p)) s_parent[p] = 1;
    if (in(c)) atomicMin(s_first + c, i);
  }
  __syncthreads();
  auto holds = [&](int i, int p, int c) {
    return in(p) && in(c) && !s_parent[c] && s_first[c] == i;
  };
  const long long room = (long long)a.width << shift;
  int before = 0, all = 0;
  for (int i = tid; i < a.forks; i += kForkThreads) {
    const int p = __ldg(a.parents + i), c = __ldg(a.children + i);
    if (!holds(i, p, c)) continue;
    const int n = (int)min((long long)max(a.lens[p], 0), room);
    if (n & (ps - 1)) all++, before += i < mine;
  }
  atomicAdd(&s_before, before);
  atomicAdd(&s_all, all);
  __syncthreads();
  uint32_t bad = 0;
  if (mine == 0 && tid == 0) {
    a.taken[0] = min(s_all, a.num_free);
    if (s_all > a.num_free) bad |= kErrPool;
  }
  if (mine < a.forks) {
    const int p = __ldg(a.parents + mine), c = __ldg(a.children + mine);
    int src = -1, dst = -1;
    if (holds(mine, p, c)) {
      const int len = a.lens[p];
      const int n = (int)min((long long)max(len, 0), room);
      if (len != n) bad |= kErrLength;
      const int full = n >> shift, cut = n & (ps - 1);
      const int32_t* from = a.table + (size_t)p * a.width;
      int32_t* to = a.table + (size_t)c * a.width;
      for (int i = tid; i < full; i += kForkThreads) to[i] = from[i];
      if (cut && tid == 0) {
        int fresh = s_before < a.num_free ? __ldg(a.free_pages + s_before) : -1;
        if ((unsigned)fresh >= (unsigned)pool) bad |= kErrPool, fresh = -1;
        to[full] = fresh;
        src = from[full];
        if ((unsigned)src >= (unsigned)pool) bad |= kErrPage, src = -1;
        dst = fresh;
        if (src < 0 || dst < 0) src = dst = -1;
      }
      if (tid == 0) a.lens[c] = n;
    } else {
      bad |= kErrRow;
    }
    if (tid == 0) {
      a.src[mine] = src;
      a.dst[mine] = dst;
    }
  }
  if (bad && tid == 0) atomicOr(err, bad);
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                    // in flight per thread
constexpr int kCopyUnit = kCopyThreads * kCopyVecs * 16;        // bytes of a unit

struct CopyShape {
  long long page_bytes;       // of one of the two arrays
  long long code_bytes;       // of a page's summary codes, 0 without
  int steps;                  // its steps
  int units;                  // units of an array's page
};

// Pages lie whole in memory, so a copy is 2 page_bytes and a summary; units of
// 16 KB are dealt to the CTAs in turn (2498 pages of 128 KB: 104 us, 6.2 TB/s read
// and written; 640 of 32 KB: 9.3, 4.5).
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(moe_reader_kv_copy_args a, CopyShape c, char* k, char* v, char* codes, float* steps,
            int pool, uint32_t* err) {
  wait_for_earlier_launch();
  long long n = a.count ? min(max(__ldg(a.count), 0), a.pages) : a.pages;
  const long long each = 2 * c.units + (codes != nullptr);
  for (long long u = blockIdx.x; u < n * each; u += gridDim.x) {
    const long long i = u / each;
    const int part = (int)(u - i * each);
    const int src = __ldg(a.src + i), dst = __ldg(a.dst + i);
    if (src == -1 || dst == -1 || src == dst) continue;
    if ((unsigned)src >= (unsigned)pool || (unsigned)dst >= (unsigned)pool) {
      if (part == 0 && threadIdx.x == 0) atomicOr(err, kErrPage);
      continue;
    }
    if (part == 2 * c.units) {
      const uint4* from = reinterpret_cast<const uint4*>(codes + src * c.code_bytes);
      uint4* to = reinterpret_cast<uint4*>(codes + dst * c.code_bytes);
      for (int j = threadIdx.x; j < c.code_bytes / 16; j += kCopyThreads) to[j] = from[j];
      for (int j = threadIdx.x; j < c.steps; j += kCopyThreads)
        steps[(size_t)dst * c.steps + j] = steps[(size_t)src * c.steps + j];
      continue;
    }
    char* base = part < c.units ? k : v;
    const long long at = (long long)(part < c.units ? part : part - c.units) * kCopyUnit;
    const long long left = c.page_bytes - at;
    const uint4* from = reinterpret_cast<const uint4*>(base + src * c.page_bytes + at);
    uint4* to = reinterpret_cast<uint4*>(base + dst * c.page_bytes + at);
    uint4 x[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
      const int e = threadIdx.x + j * kCopyThreads;
      if (e * 16LL < left) x[j] = ldg_stream(from + e);
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
      const int e = threadIdx.x + j * kCopyThreads;
      if (e * 16LL < left) to[e] = x[j];
    }
  }
}

}  // namespace

cudaError_t configure_kv_pages() {
  const int bytes = kSmallPool * (int)sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(pool_kernel<false, kPoolCtas>,
                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(pool_kernel<true, kPoolCtas>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(pool_kernel<false, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(pool_kernel<true, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
  return e;
}

cudaError_t launch_kv_collect(const moe_reader_kv& kv, const moe_reader_kv_pages_args& a,
                              cudaStream_t s) {
  return launch_pool<false>(kv, a, s);
}
cudaError_t launch_kv_compact(const moe_reader_kv& kv, const moe_reader_kv_pages_args& a,
                              cudaStream_t s) {
  return launch_pool<true>(kv, a, s);
}

cudaError_t launch_kv_fork(const moe_reader_kv& kv, const moe_reader_kv_fork_args& a,
                           cudaStream_t s) {
  return launch_early(fork_kernel, dim3(std::max(a.forks, 1)), kForkThreads, 0, s, a, kv.page_shift,
                      kv.cfg.num_pages, kv.err);
}

cudaError_t launch_kv_copy(const moe_reader_kv& kv, const moe_reader_kv_copy_args& a,
                           cudaStream_t s) {
  const moe_reader_kv_config& g = kv.cfg;
  CopyShape c;
  c.page_bytes = (long long)g.num_kv_heads * g.page_size * g.head_dim *
                 (g.cache_type == MOE_READER_TYPE_E4M3 ? 1 : 2);
  c.code_bytes = kv.codes ? 2LL * g.num_kv_heads * g.head_dim : 0;
  c.steps = kv.codes ? g.num_kv_heads : 0;
  c.units = (int)((c.page_bytes + kCopyUnit - 1) / kCopyUnit);
  const long long units = a.pages * (2LL * c.units + (kv.codes != nullptr));
  const int grid = (int)std::min<long long>(units, 8LL * kv.sms);
  return launch_early(copy_kernel, dim3(grid), kCopyThreads, 0, s, a, c, static_cast<char*>(kv.k),
                      static_cast<char*>(kv.v), reinterpret_cast<char*>(kv.codes), kv.steps,
                      g.num_pages, kv.err);
}

}  // namespace mr

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
namespace {

using mr::Words;

// No output may share a word with an input or another output.
template <int I, int O>
bool apart(const Words (&ins)[I], const Words (&outs)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (mr::share_a_word(outs[o], ins[i])) return false;
    for (int p = 0; p < o; ++p)
      if (mr::share_a_word(outs[o], outs[p])) return false;
  }
  return true;
}

int check_pages(const moe_reader_kv* kv, const moe_reader_kv_pages_args* a, bool compact) {
  if (!kv || !a) return MOE_READER_EINVAL;
  if (a->requests < 0 || a->requests > kv->cfg.max_requests || a->width < 1)
    return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  if (!a->refs || !a->free_pages || !a->count) return MOE_READER_EINVAL;
  if (a->requests && (!a->table || !a->lens)) return MOE_READER_EINVAL;
  const long long N = kv->cfg.num_pages, M = N / 2, R = a->requests;
  if (compact ? !a->moves || (M && (!a->src || !a->dst)) : a->moves || a->src || a->dst)
    return MOE_READER_EINVAL;
  const void* words[] = {a->table, a->lens, a->refs, a->free_pages, a->count, a->src, a->dst,
                         a->moves};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_READER_EINVAL;
  const Words table = {a->table, R * a->width}, lens = {a->lens, R}, none = {nullptr, 0};
  const Words ins[] = {lens, compact ? none : table};
  const Words outs[] = {compact ? table : none, {a->refs, N}, {a->free_pages, N}, {a->count, 1},
                        {a->src, compact ? M : 0}, {a->dst, compact ? M : 0},
                        {a->moves, compact ? 1 : 0}};
  if (!apart(ins, outs)) return MOE_READER_EINVAL;
  return mr::on_device(kv) ? MOE_READER_OK : MOE_READER_EINVAL;
}

}  // namespace

extern "C" {

int moe_reader_kv_collect(moe_reader_kv_t* kv, const moe_reader_kv_pages_args* a, void* stream) {
  const int st = check_pages(kv, a, false);
  if (st != MOE_READER_OK) return st;
  return mr::status_of(mr::launch_kv_collect(*kv, *a, static_cast<cudaStream_t>(stream)));
}

int moe_reader_kv_compact(moe_reader_kv_t* kv, const moe_reader_kv_pages_args* a, void* stream) {
  const int st = check_pages(kv, a, true);
  if (st != MOE_READER_OK) return st;
  return mr::status_of(mr::launch_kv_compact(*kv, *a, static_cast<cudaStream_t>(stream)));
}

int moe_reader_kv_fork(moe_reader_kv_t* kv, const moe_reader_kv_fork_args* a, void* stream) {
  if (!kv || !a) return MOE_READER_EINVAL;
  if (a->rows < 0 || a->rows > kv->cfg.max_requests || a->width < 1) return MOE_READER_EINVAL;
  if (a->forks < 0 || a->forks > kv->cfg.max_requests || a->num_free < 0) return MOE_READER_EINVAL;
  if ((long long)a->width << kv->page_shift >= (1LL << 30)) return MOE_READER_EINVAL;
  if (!a->taken || (a->num_free && !a->free_pages)) return MOE_READER_EINVAL;
  if (a->rows && (!a->table || !a->lens)) return MOE_READER_EINVAL;
  if (a->forks && (!a->parents || !a->children || !a->src || !a->dst)) return MOE_READER_EINVAL;
  const void* words[] = {a->parents, a->children, a->table, a->lens, a->free_pages, a->src, a->dst,
                         a->taken};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_READER_EINVAL;
  const long long F = a->forks, R = a->rows;
  const Words ins[] = {{a->parents, F}, {a->children, F}, {a->free_pages, a->num_free}};
  const Words outs[] = {{a->table, R * a->width}, {a->lens, R}, {a->src, F}, {a->dst, F},
                        {a->taken, 1}};
  if (!apart(ins, outs) || !mr::on_device(kv)) return MOE_READER_EINVAL;
  return mr::status_of(mr::launch_kv_fork(*kv, *a, static_cast<cudaStream_t>(stream)));
}

int moe_reader_kv_copy(moe_reader_kv_t* kv, const moe_reader_kv_copy_args* a, void* stream) {
  if (!kv || !a || a->pages < 0) return MOE_READER_EINVAL;
  if (a->pages == 0) return MOE_READER_OK;
  if (!a->src || !a->dst) return MOE_READER_EINVAL;
  const void* words[] = {a->src, a->dst, a->count};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_READER_EINVAL;
  if (!mr::on_device(kv)) return MOE_READER_EINVAL;
  return mr::status_of(mr::launch_kv_copy(*kv, *a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
