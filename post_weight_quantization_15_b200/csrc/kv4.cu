// The cache of keys and values held in 4 bits: tokens written into it (gptq_kv4_append)
// and read back (gptq_kv4_read).
//
// Each group of a head's features of one token has its own fp16 scale s and integer zero
// point z, chosen as the layer quantizer chooses an asymmetric group's: the range holds 0,
// lo = min(x, 0), hi = max(x, 0) (-1 and 1 when equal), s = fp16((hi - lo) / 15) within
// fp16's positive range, z = clamp(rint(-lo / s), 0, 15), code c = clamp(rint(x / s) + z,
// 0, 15), value s (c - z).  The quotients are IEEE divisions: for 16-bit x their rounding
// never crosses a half (x / s is at least 2^-17 relative away from a tie that is not one),
// so the codes are those of exact arithmetic.
//
// Bound: HBM.  A thread quantizes eight features (16 bytes in, one word of codes out); the
// group / 8 threads of a group find its range with shuffles.  A block takes one token,
// all heads, keys and values.
#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

struct KVInput {
  const void* p[2];                       // k, v
  int64_t token_stride[2], head_stride[2];
};

template <typename T>
__global__ void __launch_bounds__(256) kv4_append_kernel(const KV4Cache C, const KVInput in, const int32_t* table,
                                                         int width, const int32_t* cu, const int32_t* start,
                                                         int count, int32_t* st) {
  if (has_error(st)) return;
  const int t = (int)blockIdx.x;
  const int b = packed_sequence(cu, count, t);
  if (b < 0) return;
  const int64_t pos = (int64_t)start[b] + (t - cu[b]);
  const int page = kv4_page(C, table, width, b, pos);
  if (page < 0) {
    if (threadIdx.x == 0) set_error(st, GPTQ_ERR_INVALID_ARG, t, STAGE_KV4);
    return;
  }
  const int words = C.head_dim / 8, lanes = C.group / 8;
  const int per = C.heads * words;        // units of keys, then as many of values
  const int r = (int)(pos % C.page_size);
  for (int u0 = 0; u0 < 2 * per; u0 += 256) {
    const int u = u0 + (int)threadIdx.x;
    const bool on = u < 2 * per;          // groups are whole: 2 per is a multiple of lanes
    const int kv = on && u >= per ? 1 : 0;
    const int head = on ? (u - kv * per) / words : 0, w = on ? u % words : 0;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) load8(static_cast<const T*>(in.p[kv]) + t * in.token_stride[kv] + head * in.head_stride[kv] + w * 8, x);
    float lo = 0.f, hi = 0.f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      bad |= !(fabsf(x[i]) <= FLT_MAX);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (!on) continue;
    if (lo == hi) { lo = -1.f; hi = 1.f; }
    const __half s16 = __float2half_rn(fminf(fmaxf(__fdiv_rn(hi - lo, 15.f), 5.9604644775390625e-08f), 65504.f));
    const float s = __half2float(s16);
    const float z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)) + z, 0.f), 15.f);
      word |= (uint32_t)(int)c << (4 * i);
    }
    __half2 par = __halves2half2(s16, __float2half_rn(z));
    if (bad) {                            // the whole group reads back as NaN
      word = 0;
      par = __halves2half2(__ushort_as_half((unsigned short)0x7fffu), __ushort_as_half((unsigned short)0));
      if (w % lanes == 0) set_error(st, GPTQ_ERR_NONFINITE, t, STAGE_KV4);
    }
    const int64_t row = kv4_row(C, page, head, r);
    C.codes[kv][row * words + w] = (int32_t)word;
    if (w % lanes == 0)
      reinterpret_cast<__half2*>(C.params[kv])[row * (C.head_dim / C.group) + w / lanes] = par;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) kv4_read_kernel(const KV4Cache C, const int32_t* table, int width,
                                                       const int32_t* cu, const int32_t* start, int count, T* k,
                                                       T* v, int32_t* st) {
  if (has_error(st)) return;
  const int t = (int)blockIdx.x;
  const int b = packed_sequence(cu, count, t);
  if (b < 0) return;
  const int64_t pos = (start != nullptr ? (int64_t)start[b] : 0) + (t - cu[b]);
  const int page = kv4_page(C, table, width, b, pos);
  if (page < 0) {
    if (threadIdx.x == 0) set_error(st, GPTQ_ERR_INVALID_ARG, t, STAGE_KV4);
    return;
  }
  const int words = C.head_dim / 8, lanes = C.group / 8;
  const int per = C.heads * words;
  const int r = (int)(pos % C.page_size);
  for (int u = (int)threadIdx.x; u < 2 * per; u += 256) {
    const int kv = u >= per ? 1 : 0;
    const int head = (u - kv * per) / words, w = u % words;
    const int64_t row = kv4_row(C, page, head, r);
    const uint32_t word = (uint32_t)C.codes[kv][row * words + w];
    const __half2 par = reinterpret_cast<const __half2*>(C.params[kv])[row * (C.head_dim / C.group) + w / lanes];
    const float s = __low2float(par), z = __high2float(par);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s * ((float)((word >> (4 * i)) & 15u) - z);
    store8((kv ? v : k) + ((int64_t)t * C.heads + head) * C.head_dim + w * 8, x);
  }
}

double token_bytes(const KV4Cache& C) { return 2.0 * C.heads * (C.head_dim / 2 + 4.0 * (C.head_dim / C.group)); }

}  // namespace

int launch_kv4_append(const KV4Cache& C, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                      int64_t v_hs, int dtype, int tokens, const int32_t* table, int width, const int32_t* cu,
                      const int32_t* start, int count, int32_t* st, cudaStream_t s) {
  const KVInput in{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}};
  TraceScope ts("kv4_append", "byte", tokens * (token_bytes(C) + 4.0 * C.heads * C.head_dim), s);
  if (dtype == GPTQ_F16)
    kv4_append_kernel<__half><<<(unsigned)tokens, 256, 0, s>>>(C, in, table, width, cu, start, count, st);
  else
    kv4_append_kernel<__nv_bfloat16><<<(unsigned)tokens, 256, 0, s>>>(C, in, table, width, cu, start, count, st);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

int launch_kv4_read(const KV4Cache& C, const int32_t* table, int width, const int32_t* cu, const int32_t* start,
                    int count, int tokens, int dtype, void* k, void* v, int32_t* st, cudaStream_t s) {
  TraceScope ts("kv4_read", "byte", tokens * (token_bytes(C) + (dtype == GPTQ_F32 ? 8.0 : 4.0) * C.heads * C.head_dim), s);
  if (dtype == GPTQ_F32)
    kv4_read_kernel<float><<<(unsigned)tokens, 256, 0, s>>>(C, table, width, cu, start, count,
                                                            static_cast<float*>(k), static_cast<float*>(v), st);
  else if (dtype == GPTQ_F16)
    kv4_read_kernel<__half><<<(unsigned)tokens, 256, 0, s>>>(C, table, width, cu, start, count,
                                                             static_cast<__half*>(k), static_cast<__half*>(v), st);
  else
    kv4_read_kernel<__nv_bfloat16><<<(unsigned)tokens, 256, 0, s>>>(
        C, table, width, cu, start, count, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), st);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
