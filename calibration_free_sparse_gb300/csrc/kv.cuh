// Declarations shared by the paged cache's translation units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_reader.h"

struct moe_reader_kv {
  moe_reader_kv_config cfg;
  int device;
  int sms;                    // CTAs of attend: one per SM
  int page_shift;             // log2(page_size)
  int group;                  // query heads per KV head
  void* k;                    // caller-owned [num_pages][Hkv][page_size][D]
  void* v;
  int8_t* codes;              // caller-owned [num_pages][Hkv][2][D] or null
  float* steps;               // caller-owned [num_pages][Hkv] or null
  const float* k_scale;       // caller-owned [Hkv] or null
  const float* v_scale;
  // workspace
  void* base;
  float* part_o;              // [sms][2][16][D]  unnormalised outputs of split rows
  float* part_ml;             // [sms][2][2][16]  their references and sums of weights
  uint32_t* arrived;          // [rows]           pieces written; zero between launches
  size_t arrived_bytes;
  uint32_t* err;              // [1]              device error word
};

namespace mr {

constexpr int kMaxGroup = 64;
constexpr int kMaxRequests = 1024;
constexpr int kMaxSelectPages = 49152;
constexpr int kMaxSms = 256;          // CTAs of attend at most

constexpr uint32_t kErrLength = MOE_READER_ERR_LENGTH;
constexpr uint32_t kErrPage = MOE_READER_ERR_PAGE;
constexpr uint32_t kErrPool = MOE_READER_ERR_POOL;

cudaError_t launch_kv_plan(const moe_reader_kv& kv, const moe_reader_kv_plan_args& a,
                           cudaStream_t s);
cudaError_t launch_kv_append(const moe_reader_kv& kv, const moe_reader_kv_append_args& a,
                             cudaStream_t s);
cudaError_t launch_kv_attend(const moe_reader_kv& kv, const moe_reader_kv_attend_args& a,
                             cudaStream_t s);
cudaError_t configure_kv_attend(const moe_reader_kv& kv);
// One-shot injection of a turn that never comes in the next attend.
bool take_attend_stall();
// Items of attend: (request, KV head, tile of the group's query heads).
int attend_row_tiles(const moe_reader_kv_config& c);
cudaError_t launch_kv_select(const moe_reader_kv& kv, const moe_reader_kv_select_args& a,
                             cudaStream_t s);
cudaError_t configure_kv_select(const moe_reader_kv& kv);

// Launch that may start while the stream's previous kernel ends: it has to
// call wait_for_earlier_launch() before it touches global memory, which returns
// once that kernel is complete and its writes can be seen.
template <class... K, class... A>
inline cudaError_t launch_early(void (*kernel)(K...), dim3 grid, int threads, size_t smem,
                                cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...);
}
__device__ __forceinline__ void wait_for_earlier_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets such a launch behind this kernel take free SMs already.
__device__ __forceinline__ void let_next_launch_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2 a) of a finite a >= 0, held to -100 .. 100
__device__ __forceinline__ int floor_log2_held(float a) {
  a = fminf(fmaxf(a, 7.8886090522101181e-31f), 1.2676506002282294e30f);   // 2^-100, 2^100
  return (__float_as_int(a) >> 23) - 127;
}

}  // namespace mr
