// The norms around a block, fused with the block's gate, its residual scale and the
// residual addition (gptq_add_norm): per row x of the residual stream and row y of the
// block's output
//
//   xn = round(x + alpha . g . N(y; post))        h = round(N(xn; w))
//
// with N the RMS norm, v -> v / sqrt(mean(v^2) + eps) . w + b, or the layer norm
// (center), which subtracts mean(v) first.  xn is rounded to the stream's type before h
// is taken from it, so h is what a separate norm of the stored stream would give.
// Sums are fp32; the layer norm takes its squares from the centred values (a second
// pass over registers, not over memory), so a large mean costs no digits.
//
// Bound: HBM.  A row is read once into registers (16 values per thread up to d = 16384,
// 32 above) and every statistic is taken there; x, y and the gate are read and xn and h
// written once.  Rows of up to 1024 values take one warp each (no block barrier),
// longer rows one block.  Where a row does not start on a 16-byte boundary (an odd d or
// stride) the lanes read single values side by side instead of eight each.
#include "common.cuh"
#include "internal.h"
#include "vec_io.cuh"

namespace gptq {

namespace {

struct NormArgs {
  const void* X;
  const void* Y;
  const void* weight;
  const void* bias;
  const void* post_weight;
  const void* post_bias;
  const void* gate;
  void* Xn;
  void* h;
  int64_t ld_x, ld_y, ld_gate, ld_xn, ld_h;
  int p_dtype;
  int tokens, d;
  float alpha, eps;
  int center;
};

// Sum over the row's threads (blockDim.x; a warp, or the whole block through `part`).
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();                       // the previous sum's readers are done
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// V x 8 values per thread: VEC: 8 consecutive ones per vector; else single values, the
// row's threads side by side.
template <int V, bool VEC>
struct Place {
  __device__ static __forceinline__ int at(int v, int e) {
    return VEC ? (v * (int)blockDim.x + (int)threadIdx.x) * 8 + e
               : (v * 8 + e) * (int)blockDim.x + (int)threadIdx.x;
  }
};

template <typename T, int V, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int d, float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      const int i = Place<V, VEC>::at(v, 0);
      float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (i < d) load8(row + i, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v * 8 + e] = t[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = Place<V, VEC>::at(v, e);
        x[v * 8 + e] = i < d ? load_as_float(row + i) : 0.f;
      }
    }
  }
}

// A parameter row of run-time type p_dtype (the parameters stay in cache).
template <int V, bool VEC>
__device__ __forceinline__ void load_param(const void* row, int64_t off, int p_dtype, int d, float (&x)[V * 8]) {
  if (p_dtype == GPTQ_F32) load_row<float, V, VEC>(static_cast<const float*>(row) + off, d, x);
  else if (p_dtype == GPTQ_F16) load_row<__half, V, VEC>(static_cast<const __half*>(row) + off, d, x);
  else load_row<__nv_bfloat16, V, VEC>(static_cast<const __nv_bfloat16*>(row) + off, d, x);
}

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_row(T* row, int d, const float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      const int i = Place<V, VEC>::at(v, 0);
      if (i < d) store8(row + i, &x[v * 8]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = Place<V, VEC>::at(v, e);
        if (i < d) store_from_float(row + i, x[v * 8 + e]);
      }
    }
  }
}

// x <- N(x; w, b), the row's values in registers (values past d are 0 and stay unused).
template <int V, bool VEC>
__device__ __forceinline__ void norm_row(float (&x)[V * 8], const void* w, const void* b, const NormArgs& A,
                                         float* part) {
  const float inv_d = 1.f / (float)A.d;
  if (A.center) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V * 8; ++i) s += x[i];
    const float mean = row_sum(s, part) / (float)A.d;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[v * 8 + e] = Place<V, VEC>::at(v, e) < A.d ? x[v * 8 + e] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V * 8; ++i) q = fmaf(x[i], x[i], q);
  const float r = rsqrtf(row_sum(q, part) * inv_d + A.eps);
  float p[V * 8];
  load_param<V, VEC>(w, 0, A.p_dtype, A.d, p);
#pragma unroll
  for (int i = 0; i < V * 8; ++i) x[i] = x[i] * r * p[i];
  if (b != nullptr) {
    load_param<V, VEC>(b, 0, A.p_dtype, A.d, p);
#pragma unroll
    for (int i = 0; i < V * 8; ++i) x[i] += p[i];
  }
}

template <typename TX, typename TY, int V, bool VEC>
__global__ void __launch_bounds__(1024) add_norm_kernel(const NormArgs A, const int32_t* st) {
  __shared__ float part[32];
  if (has_error(st)) return;
  const int row = (int)blockIdx.x * (int)blockDim.y + (int)threadIdx.y;
  if (row >= A.tokens) return;           // blockDim.y > 1 only with one warp per row
  float x[V * 8];
  load_row<TX, V, VEC>(static_cast<const TX*>(A.X) + (int64_t)row * A.ld_x, A.d, x);
  if (A.Y != nullptr) {
    float y[V * 8];
    load_row<TY, V, VEC>(static_cast<const TY*>(A.Y) + (int64_t)row * A.ld_y, A.d, y);
    if (A.post_weight != nullptr) norm_row<V, VEC>(y, A.post_weight, A.post_bias, A, part);
    if (A.gate != nullptr) {
      float g[V * 8];
      load_param<V, VEC>(A.gate, (int64_t)row * A.ld_gate, A.p_dtype, A.d, g);
#pragma unroll
      for (int i = 0; i < V * 8; ++i) y[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < V * 8; ++i) x[i] = round_to<TX>(fmaf(A.alpha, y[i], x[i]));
    store_row<TX, V, VEC>(static_cast<TX*>(A.Xn) + (int64_t)row * A.ld_xn, A.d, x);
  }
  norm_row<V, VEC>(x, A.weight, A.bias, A, part);
  store_row<TX, V, VEC>(static_cast<TX*>(A.h) + (int64_t)row * A.ld_h, A.d, x);
}

template <typename TX, typename TY, bool VEC>
void launch(const NormArgs& A, const int32_t* st, cudaStream_t s) {
  if (A.d <= 1024) {
    const dim3 blk(32, 8);
    const unsigned grd = (unsigned)cdiv(A.tokens, 8);
    if (A.d <= 512) add_norm_kernel<TX, TY, 2, VEC><<<grd, blk, 0, s>>>(A, st);
    else add_norm_kernel<TX, TY, 4, VEC><<<grd, blk, 0, s>>>(A, st);
    return;
  }
  const int per = A.d <= 16384 ? 16 : 32;
  const unsigned thr = (unsigned)(cdiv(cdiv(A.d, per), 32) * 32);
  if (per == 16) add_norm_kernel<TX, TY, 2, VEC><<<(unsigned)A.tokens, thr, 0, s>>>(A, st);
  else add_norm_kernel<TX, TY, 4, VEC><<<(unsigned)A.tokens, thr, 0, s>>>(A, st);
}

template <typename TX, typename TY>
void launch_vec(const NormArgs& A, bool vec, const int32_t* st, cudaStream_t s) {
  if (vec) launch<TX, TY, true>(A, st, s);
  else launch<TX, TY, false>(A, st, s);
}

template <typename TX>
void launch_y(const NormArgs& A, int y_dtype, bool vec, const int32_t* st, cudaStream_t s) {
  if (A.Y == nullptr || y_dtype == GPTQ_F32) launch_vec<TX, float>(A, vec, st, s);
  else if (y_dtype == GPTQ_F16) launch_vec<TX, __half>(A, vec, st, s);
  else launch_vec<TX, __nv_bfloat16>(A, vec, st, s);
}

size_t width(int dtype) { return dtype == GPTQ_F32 ? 4 : 2; }

// Eight values of a row start on a 16-byte boundary in every row.
bool vec_ok(const void* p, int64_t ld, int dtype) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * (int64_t)width(dtype)) % 16 == 0);
}

}  // namespace

int launch_add_norm(const void* X, int x_dtype, int64_t ld_x, const void* Y, int y_dtype, int64_t ld_y,
                    const void* weight, const void* bias, const void* post_weight, const void* post_bias,
                    const void* gate, int64_t ld_gate, int p_dtype, int tokens, int d, float alpha, float eps,
                    int center, void* Xn, int64_t ld_xn, void* h, int64_t ld_h, const int32_t* st, cudaStream_t s) {
  NormArgs A{X, Y, weight, bias, post_weight, post_bias, gate, Xn, h, ld_x, ld_y, ld_gate, ld_xn, ld_h,
             p_dtype, tokens, d, alpha, eps, center};
  const bool vec = d % 8 == 0 && vec_ok(X, ld_x, x_dtype) && vec_ok(Y, ld_y, y_dtype) && vec_ok(h, ld_h, x_dtype) &&
                   (Y == nullptr || vec_ok(Xn, ld_xn, x_dtype)) && vec_ok(weight, 0, p_dtype) &&
                   vec_ok(bias, 0, p_dtype) && vec_ok(post_weight, 0, p_dtype) && vec_ok(post_bias, 0, p_dtype) &&
                   vec_ok(gate, ld_gate, p_dtype);
  const double n = (double)tokens * d, b = (double)width(x_dtype);
  TraceScope ts("add_norm", "byte", n * (Y != nullptr ? 3 * b + (double)width(y_dtype) : 2 * b) +
                                        (gate != nullptr && ld_gate != 0 ? n * (double)width(p_dtype) : 0.0), s);
  if (x_dtype == GPTQ_F32) launch_y<float>(A, y_dtype, vec, st, s);
  else if (x_dtype == GPTQ_F16) launch_y<__half>(A, y_dtype, vec, st, s);
  else launch_y<__nv_bfloat16>(A, y_dtype, vec, st, s);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
