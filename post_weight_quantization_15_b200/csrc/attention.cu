// Attention over the prompts of a packed batch (gptq_attention): per sequence and query
// head, o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j that query i sees (all,
// or with causal those up to i + Lk - Lq), hq / hk query heads per k/v head.  A query that
// sees no key gives 0; a key that a query does not see takes no part in it, whatever its
// row holds.
//
// One warp per query and head: 32 keys at a time, a lane per key for the scores, a running
// maximum and sum in fp32, then the lanes over the features for the values.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

template <typename T>
__global__ void __launch_bounds__(128) attention_rows_kernel(const AttentionArgs A, int32_t* st) {
  __shared__ float qs[4][128];
  if (has_error(st)) return;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int t = (int)blockIdx.x * 4 + warp, h = (int)blockIdx.y;
  if (t >= A.total_q) return;
  const int b = packed_sequence(A.cu_q, A.count, t);
  if (b < 0) return;
  const int q0 = A.cu_q[b], q1 = A.cu_q[b + 1], k0 = A.cu_k[b], k1 = A.cu_k[b + 1];
  if (q0 < 0 || q1 > A.total_q || k0 < 0 || k1 < k0 || k1 > A.total_k) {
    if (lane == 0) set_error(st, GPTQ_ERR_INVALID_ARG, b, STAGE_ATTENTION);
    return;
  }
  const T* q = static_cast<const T*>(A.q) + t * A.q_ts + h * A.q_hs;
  const int hk = h / (A.heads_q / A.heads_kv);
  for (int i = lane; i < A.head_dim; i += 32) qs[warp][i] = load_as_float(q + i) * A.scale;
  __syncwarp();
  int seen = k1 - k0;
  if (A.causal) seen = min(seen, t - q0 + 1 + (k1 - k0) - (q1 - q0));
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    float sc = -INFINITY;
    if (j < seen) {
      const T* k = static_cast<const T*>(A.k) + (k0 + j) * A.k_ts + hk * A.k_hs;
      sc = 0.f;
      for (int i = 0; i < A.head_dim; i += 8) {
        float x[8];
        load8(k + i, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sc = fmaf(qs[warp][i + e], x[e], sc);
      }
    }
    float mn = sc;
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float p = j < seen ? expf(sc - ref) : 0.f;
    const float f = expf(m - ref);
    m = mn;
    l *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
    for (int o = 0; o < 32 && j0 + o < seen; ++o) {
      const float w = __shfl_sync(0xffffffffu, p, o);
      l += w;
      const T* v = static_cast<const T*>(A.v) + (k0 + j0 + o) * A.v_ts + hk * A.v_hs;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e * 32 + lane < A.head_dim) acc[e] = fmaf(w, load_as_float(v + e * 32 + lane), acc[e]);
    }
  }
  T* o = static_cast<T*>(A.o) + t * A.o_ts + h * A.o_hs;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e * 32 + lane < A.head_dim) store_from_float(o + e * 32 + lane, seen > 0 ? acc[e] / l : 0.f);
}

}  // namespace

int launch_attention(const AttentionArgs& A, int dtype, int32_t* st, cudaStream_t s) {
  TraceScope ts("attention", "", 0.0, s);
  const dim3 grd((unsigned)cdiv(A.total_q, 4), (unsigned)A.heads_q);
  if (dtype == GPTQ_F16) attention_rows_kernel<__half><<<grd, 128, 0, s>>>(A, st);
  else attention_rows_kernel<__nv_bfloat16><<<grd, 128, 0, s>>>(A, st);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
