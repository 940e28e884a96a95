// Shared device-side helpers of the GPTQ library (status block, loads, launch checks).
#pragma once

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/gptq.h"

namespace gptq {

// Index of the fields of the caller's device status block.
enum { ST_CODE = 0, ST_INFO = 1, ST_STAGE = 2, ST_LAUNCH = 3 };

// Stage ids recorded in d_status[ST_STAGE] next to an error.
enum {
  STAGE_HESSIAN = 1, STAGE_PREP_DIAG = 2, STAGE_POTRF = 3, STAGE_TRINV = 4,
  STAGE_INGEST = 5, STAGE_SWEEP = 6, STAGE_TRAILING = 7, STAGE_PACK = 8, STAGE_DEQUANT = 9,
  STAGE_LINEAR = 10, STAGE_ROPE = 11, STAGE_ATTENTION = 12, STAGE_KV4 = 13, STAGE_KV4_ATTENTION = 14
};

// First error wins; later kernels see a non-zero code and skip their work.
__device__ __forceinline__ void set_error(int32_t* st, int code, int info, int stage) {
  if (st == nullptr) return;
  if (atomicCAS(reinterpret_cast<int*>(st + ST_CODE), 0, code) == 0) {
    st[ST_INFO] = info;
    st[ST_STAGE] = stage;
    __threadfence();
  }
}

__device__ __forceinline__ bool has_error(const int32_t* st) {
  if (st == nullptr) return false;
  return *reinterpret_cast<const volatile int32_t*>(st + ST_CODE) != 0;
}

// For launches that go on past the errors they record (a bad token is left out, the others are
// not): has_error would stop the blocks, or the warps, that look after another one recorded
// something.  `launch` is the call's number (next_launch()), kept beside the error.
__device__ __forceinline__ void set_own_error(int32_t* st, int launch, int code, int info, int stage) {
  if (st == nullptr || has_error(st)) return;
  *reinterpret_cast<volatile int32_t*>(st + ST_LAUNCH) = launch;     // (the same value from every block)
  __threadfence();
  set_error(st, code, info, stage);
}

// An error that was there before the launch.  Where threads of a block depend on one another
// one thread asks for all.  From here on the error is nobody's own: a graph that holds the call
// which recorded it (under the same number in every replay) stops there too when it is replayed.
// (Replays of a graph of that call alone, which nobody else has seen the error of, go on.)
__device__ __forceinline__ bool stopped(int32_t* st, int launch) {
  if (!has_error(st)) return false;
  __threadfence();
  volatile int32_t* by = st + ST_LAUNCH;
  if (*by == launch) return false;
  *by = 0;
  return true;
}

template <typename T> __device__ __forceinline__ float load_as_float(const T* p);
template <> __device__ __forceinline__ float load_as_float<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float load_as_float<__half>(const __half* p) { return __half2float(*p); }
template <> __device__ __forceinline__ float load_as_float<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ constexpr size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace gptq

namespace gptq {
// Host-side count of enqueued kernels (see gptq_kernel_launches).
void count_launch();
int next_launch();                    // a call's number for set_own_error: never 0, another for every call
void count_launches(int64_t delta);   // a replayed graph's kernels (or, negative, a captured graph's)
}  // namespace gptq

// Host-side: turn a CUDA launch/runtime failure into GPTQ_ERR_CUDA.
#define GPTQ_CUDA_TRY(expr)                        \
  do {                                             \
    cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return GPTQ_ERR_CUDA;   \
  } while (0)

#define GPTQ_LAUNCH_CHECK()                                   \
  do {                                                        \
    ::gptq::count_launch();                                   \
    cudaError_t _e = cudaGetLastError();                      \
    if (_e != cudaSuccess) return GPTQ_ERR_CUDA;              \
  } while (0)
