// Attention of one query token per sequence over its keys and values in the 4-bit cache
// (gptq_kv4_attention): o = sum_t softmax_t(scale q . k_t) v_t over the sequence's tokens,
// k_t and v_t = s (c - z) read from the cache's pages, hq / hk query heads per k/v head.
// A sequence without tokens gives 0.
//
// One block per query head and sequence: 128 tokens at a time, a thread per token for the
// scores, a running maximum and sum in fp32, then a thread per feature for the values.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

constexpr int TB = 128;

__device__ __forceinline__ float block_max(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

template <typename T>
__global__ void __launch_bounds__(TB) kv4_attention_kernel(const KV4Cache C, const T* q, int64_t q_ts, int64_t q_hs,
                                                           const int32_t* table, int width, const int32_t* lengths,
                                                           int heads_q, float scale, T* o, int64_t o_ts, int64_t o_hs,
                                                           int32_t* st) {
  __shared__ float qs[128], ps[TB], part[4];
  __shared__ int pages[TB];
  if (has_error(st)) return;
  const int hq = (int)blockIdx.x, b = (int)blockIdx.y, tid = (int)threadIdx.x;
  const int head = hq / (heads_q / C.heads);
  const int d = C.head_dim, words = d / 8, groups = d / C.group;
  const int len = lengths[b];
  if (len < 0 || len > (int64_t)width * C.page_size) {
    if (tid == 0) set_error(st, GPTQ_ERR_INVALID_ARG, b, STAGE_KV4_ATTENTION);
    return;
  }
  if (tid < d) qs[tid] = load_as_float(q + b * q_ts + hq * q_hs + tid) * scale;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < len; t0 += TB) {
    const int t = t0 + tid;
    int page = -1;
    if (t < len) {
      page = kv4_page(C, table, width, b, t);
      if (page < 0) set_error(st, GPTQ_ERR_INVALID_ARG, b, STAGE_KV4_ATTENTION);
    }
    __syncthreads();                      // qs is there; the last tile's readers are done
    pages[tid] = page;
    float sc = -INFINITY;
    if (page >= 0) {
      const int64_t row = kv4_row(C, page, head, t % C.page_size);
      sc = 0.f;
      for (int w = 0; w < words; ++w) {
        const uint32_t word = (uint32_t)C.codes[0][row * words + w];
        const __half2 par = reinterpret_cast<const __half2*>(C.params[0])[row * groups + w * 8 / C.group];
        float a = 0.f;
        for (int i = 0; i < 8; ++i) a = fmaf(qs[w * 8 + i], (float)((word >> (4 * i)) & 15u) - __high2float(par), a);
        sc = fmaf(__low2float(par), a, sc);
      }
    }
    const float mn = fmaxf(m, block_max(sc, part));
    const float p = page >= 0 ? expf(sc - mn) : 0.f;
    ps[tid] = p;
    __syncthreads();
    const float f = m == -INFINITY ? 0.f : expf(m - mn);
    m = mn;
    l *= f;
    acc *= f;
    for (int i = 0; i < TB && t0 + i < len; ++i) {
      if (pages[i] < 0) continue;
      l += ps[i];
      if (tid < d) {
        const int64_t row = kv4_row(C, pages[i], head, (t0 + i) % C.page_size);
        const uint32_t word = (uint32_t)C.codes[1][row * words + tid / 8];
        const __half2 par = reinterpret_cast<const __half2*>(C.params[1])[row * groups + tid / C.group];
        acc = fmaf(ps[i], __low2float(par) * ((float)((word >> (4 * (tid & 7))) & 15u) - __high2float(par)), acc);
      }
    }
  }
  if (tid < d) store_from_float(o + b * o_ts + hq * o_hs + tid, len > 0 ? acc / l : 0.f);
}

}  // namespace

size_t kv4_attention_ws_bytes(int, int, int, int, int64_t) { return 256; }

int launch_kv4_attention(const KV4Cache& C, const void* q, int64_t q_ts, int64_t q_hs, int dtype, int count,
                         int heads_q, const int32_t* table, int width, const int32_t* lengths, float scale, void* o,
                         int64_t o_ts, int64_t o_hs, void* ws, int32_t* st, cudaStream_t s) {
  TraceScope ts("kv4_attention", "", 0.0, s);
  const dim3 grd((unsigned)heads_q, (unsigned)count);
  if (dtype == GPTQ_F16)
    kv4_attention_kernel<__half><<<grd, TB, 0, s>>>(C, static_cast<const __half*>(q), q_ts, q_hs, table, width, lengths,
                                                    heads_q, scale, static_cast<__half*>(o), o_ts, o_hs, st);
  else
    kv4_attention_kernel<__nv_bfloat16><<<grd, TB, 0, s>>>(C, static_cast<const __nv_bfloat16*>(q), q_ts, q_hs, table,
                                                           width, lengths, heads_q, scale,
                                                           static_cast<__nv_bfloat16*>(o), o_ts, o_hs, st);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
