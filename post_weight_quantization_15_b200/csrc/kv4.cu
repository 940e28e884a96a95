// The cache of keys and values held in 4 bits: tokens written into it (gptq_kv4_append)
// and read back (gptq_kv4_read).
//
// Each group of a head's features of one token has its own fp16 scale s and integer zero
// point z, chosen as the layer quantizer chooses an asymmetric group's: the range holds 0,
// lo = min(x, 0), hi = max(x, 0) (-1 and 1 when equal), s = fp16((hi - lo) / 15) within
// fp16's positive range, z = clamp(rint(-lo / s), 0, 15), code c = clamp(rint(x / s) + z,
// 0, 15), value s (c - z).  x / s is a tie or at least 2^-17 relative away from one (x and s
// have few bits), so its integer needs no IEEE division: with r = 1 / s to 2^-23 the product
// q = x r is within 2^-22 of it, and q + r (x - q s), the residual exact but for its own
// rounding, lands on a tie's few bits exactly.  (hi - lo) / 15 is the rounded quotient by
// Markstein's theorem: a residual and the rounded reciprocal (checked for all fp32
// significands).  Adding 1.5 . 2^23 rounds to the nearest even integer and leaves it in the
// low bits, where the eight codes of a word are summed under their shifts (the constant's
// and the zero point's shares taken off once).
//
// Bound: HBM, with the issue slots close behind.  A thread quantizes 32 features of a group (16
// where the group has no more), eight at a time and side by side with the group's other
// threads, of keys and values; the group's range is found with shuffles on packed 16-bit
// values.  What a group costs (its range, scale, zero point, addresses) is as much as sixteen
// features do, hence so many per thread.  A block takes a few consecutive tokens, their places
// looked up once.  (15,625 tokens of 32 heads x 128 in bf16, groups of 128, written and read back:
// 369 us with one token per block, IEEE divisions and integer conversions; 203 with eight
// features per thread, 148 with sixteen, 135 with 32; 99 at the copy bandwidth.)
#include <type_traits>

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

constexpr int THREADS = 256;
constexpr int MOST = 64;                  // tokens of a block
constexpr int ENOUGH = 148 * 8;           // blocks that fill the SMs

// Tokens t0 .. t0 + n - 1 of the batch: the first head's row in the cache of each, or -1.  False,
// for the whole block, after an earlier launch's error; those of this launch (other blocks' tokens)
// stop nobody.
__device__ __forceinline__ bool find_rows(const KV4Cache& C, const int32_t* table, int width, const int32_t* cu,
                                          const int32_t* start, int count, int t0, int n, int64_t* rows, int32_t* st,
                                          int launch) {
  __shared__ int skip;
  if (threadIdx.x == THREADS - 1) skip = stopped(st, launch);
  if ((int)threadIdx.x < n) {
    const int t = t0 + (int)threadIdx.x, b = packed_sequence(cu, count, t);
    int64_t row = -1;
    if (b >= 0) {
      const int64_t pos = (start != nullptr ? (int64_t)start[b] : 0) + (t - cu[b]);
      const int page = kv4_page(C, table, width, b, pos);
      if (page < 0) set_own_error(st, launch, GPTQ_ERR_INVALID_ARG, t, STAGE_KV4);
      else row = kv4_row(C, page, 0, (int)(pos & (C.page_size - 1)));
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
  return !skip;
}

// A thread's place among a token's `per` units: unit u0 of every subs-th token, or units u0,
// u0 + 256, ... of every token.
struct Units {
  int per, sub, subs, u0;
  __device__ __forceinline__ explicit Units(int units) {
    per = units;
    subs = max(1, THREADS / per);
    sub = (int)threadIdx.x / per;                     // subs: no token
    u0 = per < THREADS ? (int)threadIdx.x % per : (int)threadIdx.x;
  }
};

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __half) {
  const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 wide2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ float2 wide2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ float reciprocal(float x) {     // to 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// N times eight values of a group that `lanes` threads share -> their N words, and the group's
// scale and zero point; `bad` if the group holds a NaN or an infinity.  Whole warp.
template <typename T, int N>
__device__ __forceinline__ void quantize(const uint4 (&raw)[N], int lanes, uint32_t (&word)[N], __half2& par,
                                         bool& bad) {
  uint32_t w[4 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[4 * i] = raw[i].x;
    w[4 * i + 1] = raw[i].y;
    w[4 * i + 2] = raw[i].z;
    w[4 * i + 3] = raw[i].w;
  }
  // (-smallest, largest) as one pair, 0 included
  uint32_t lo = w[0], hi = w[0];
#pragma unroll
  for (int i = 1; i < 4 * N; ++i) {
    lo = min2(lo, w[i], T());
    hi = max2(hi, w[i], T());
  }
  const uint32_t neg = lo ^ 0x80008000u;
  uint32_t ends = max2(__byte_perm(neg, hi, 0x5410), __byte_perm(neg, hi, 0x7632), T());
  ends = max2(ends, 0u, T());
  for (int o = 1; o < lanes; o <<= 1) ends = max2(ends, __shfl_xor_sync(0xffffffffu, ends, o), T());
  float2 e = wide2(ends, T());
  bad = !(e.x < INFINITY) || !(e.y < INFINITY);
  if (e.x == 0.f && e.y == 0.f) e = make_float2(1.f, 1.f);
  constexpr float FIFTEENTH = 1.f / 15.f;
  const float range = e.y + e.x;
  float scale = range * FIFTEENTH;
  scale = fmaf(fmaf(scale, -15.f, range), FIFTEENTH, scale);
  if (!(range < INFINITY)) scale = range;                 // (two bf16 ends beyond fp32 together)
  const __half s16 = __float2half_rn(fminf(fmaxf(scale, 5.9604644775390625e-08f), 65504.f));
  const float s = __half2float(s16), r = reciprocal(s);
  constexpr float ROUND = 12582912.f;     // 1.5 . 2^23
  float z = e.x * r;
  z = fminf(fmaf(r, fmaf(-z, s, e.x), z), 15.f) + ROUND;
  const uint32_t zi = __float_as_uint(z) - __float_as_uint(ROUND);
  z -= ROUND;
  const float most = 15.f - z;
  const uint32_t offset = (zi - __float_as_uint(ROUND)) * 0x11111111u;
#pragma unroll
  for (int h = 0; h < N; ++h) {
    uint32_t sum = offset;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = wide2(w[4 * h + i], T());
      const float v[2] = {x.x, x.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float q = v[k] * r;
        q = fmaf(r, fmaf(-q, s, v[k]), q);
        q = fminf(fmaxf(q, -z), most) + ROUND;
        sum += __float_as_uint(q) << (8 * i + 4 * k);
      }
    }
    word[h] = sum;
  }
  par = __halves2half2(s16, __float2half_rn(z));
}

// A thread takes N words of a group: w, w + lanes, ...
template <typename T, int N>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(const __grid_constant__ KV4Cache C,
                                                             const __grid_constant__ KVInput in, const int32_t* table,
                                                             int width, const int32_t* cu, const int32_t* start,
                                                             int count, int tokens, int per_block, int32_t* st, int launch) {
  __shared__ int64_t rows[MOST];
  const int t0 = (int)blockIdx.x * per_block, n = min(per_block, tokens - t0);
  if (!find_rows(C, table, width, cu, start, count, t0, n, rows, st, launch)) return;
  const Units U(C.heads * (C.head_dim / (8 * N)));
  const int words = C.head_dim / 8, lanes = C.group / (8 * N), groups = C.head_dim / C.group;
  const int lw = __ffs(words / N) - 1, ll = __ffs(lanes) - 1;
  // every thread goes through every step: the shuffles take whole warps
  for (int step = 0; step < U.per; step += THREADS) {
    const int u = U.u0 + step, head = u >> lw, in_head = u & (words / N - 1);
    const int group = in_head >> ll, lane = in_head & (lanes - 1), w = N * (group << ll) + lane;
    for (int i0 = 0; i0 < n; i0 += U.subs) {
      const int i = i0 + U.sub;
      const int64_t row = u < U.per && U.sub < U.subs && i < n ? rows[i] : -1;
      uint4 raw[2][N];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int c = 0; c < N; ++c) raw[kv][c] = make_uint4(0, 0, 0, 0);
        if (row >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(in.p[kv]) +
                                                            (int64_t)(t0 + i) * in.token_stride[kv] +
                                                            head * in.head_stride[kv]) + w;
#pragma unroll
          for (int c = 0; c < N; ++c) raw[kv][c] = __ldcs(src + c * lanes);
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        __half2 par;
        uint32_t word[N];
        bool bad;
        quantize<T, N>(raw[kv], lanes, word, par, bad);
        if (row < 0) continue;
        if (bad) {                        // the whole group reads back as NaN
#pragma unroll
          for (int c = 0; c < N; ++c) word[c] = 0;
          par = __halves2half2(__ushort_as_half((unsigned short)0x7fffu), __ushort_as_half((unsigned short)0));
          if (lane == 0) set_own_error(st, launch, GPTQ_ERR_NONFINITE, t0 + i, STAGE_KV4);
        }
        const int64_t at = row + (int64_t)head * C.page_size;
#pragma unroll
        for (int c = 0; c < N; ++c) C.codes[kv][at * words + w + c * lanes] = (int32_t)word[c];
        if (lane == 0) reinterpret_cast<__half2*>(C.params[kv])[at * groups + group] = par;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(const __grid_constant__ KV4Cache C, const int32_t* table,
                                                           int width, const int32_t* cu, const int32_t* start,
                                                           int count, int tokens, int per_block, T* k, T* v,
                                                           int32_t* st, int launch) {
  __shared__ int64_t rows[MOST];
  const int t0 = (int)blockIdx.x * per_block, n = min(per_block, tokens - t0);
  if (!find_rows(C, table, width, cu, start, count, t0, n, rows, st, launch)) return;
  const Units U(C.heads * (C.head_dim / 16));
  if (U.sub >= U.subs) return;
  const int words = C.head_dim / 8, lanes = C.group / 16, groups = C.head_dim / C.group;
  const int lw = __ffs(words / 2) - 1, ll = __ffs(lanes) - 1;
  for (int u = U.u0; u < U.per; u += THREADS) {
    const int head = u >> lw, in_head = u & (words / 2 - 1);
    const int group = in_head >> ll, w = 2 * (group << ll) + (in_head & (lanes - 1));      // words w, w + lanes
#pragma unroll 2
    for (int i = U.sub; i < n; i += U.subs) {
      const int64_t row = rows[i];
      if (row < 0) continue;
      const int64_t at = row + (int64_t)head * C.page_size;
      uint32_t word[2][2];
      __half2 par[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        word[kv][0] = (uint32_t)C.codes[kv][at * words + w];
        word[kv][1] = (uint32_t)C.codes[kv][at * words + w + lanes];
        par[kv] = reinterpret_cast<const __half2*>(C.params[kv])[at * groups + group];
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        // 2^23 + code is the code in the low bits of 2^23's pattern; less 2^23 + z it is code - z, exactly
        const float s = __low2float(par[kv]), z = 8388608.f + __high2float(par[kv]);
        T* dst = (kv ? v : k) + ((int64_t)(t0 + i) * C.heads + head) * C.head_dim + w * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = s * (__uint_as_float(0x4B000000u | ((word[kv][h] >> (4 * e)) & 15u)) - z);
          store8(dst + h * lanes * 8, x);
        }
      }
    }
  }
}

// Tokens of a block whose threads take `features` each: as many as keep its threads busy, more while there are blocks to spare.
int tokens_per_block(const KV4Cache& C, int tokens, int features) {
  const int per = C.heads * (C.head_dim / features);
  int n = per < THREADS ? THREADS / per : 1;
  if (n > MOST) n = MOST;
  while (n * 2 <= MOST && n * (int64_t)per < 8 * THREADS && cdiv(tokens, n * 2) >= ENOUGH) n *= 2;
  return n;
}

double token_bytes(const KV4Cache& C) { return 2.0 * C.heads * (C.head_dim / 2 + 4.0 * (C.head_dim / C.group)); }

}  // namespace

int launch_kv4_append(const KV4Cache& C, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                      int64_t v_hs, int dtype, int tokens, const int32_t* table, int width, const int32_t* cu,
                      const int32_t* start, int count, int32_t* st, cudaStream_t s) {
  const KVInput in{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}};
  const int features = C.group >= 64 ? 32 : 16;
  const int n = tokens_per_block(C, tokens, features);
  const unsigned grd = (unsigned)cdiv(tokens, n);
  TraceScope ts("kv4_append", "byte", tokens * (token_bytes(C) + 4.0 * C.heads * C.head_dim), s);
  const int launch = next_launch();
  auto go = [&](auto* kernel) { kernel<<<grd, THREADS, 0, s>>>(C, in, table, width, cu, start, count, tokens, n, st, launch); };
  if (dtype == GPTQ_F16) go(features == 32 ? kv4_append_kernel<__half, 4> : kv4_append_kernel<__half, 2>);
  else go(features == 32 ? kv4_append_kernel<__nv_bfloat16, 4> : kv4_append_kernel<__nv_bfloat16, 2>);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

int launch_kv4_read(const KV4Cache& C, const int32_t* table, int width, const int32_t* cu, const int32_t* start,
                    int count, int tokens, int dtype, void* k, void* v, int32_t* st, cudaStream_t s) {
  const int n = tokens_per_block(C, tokens, 16);
  const unsigned grd = (unsigned)cdiv(tokens, n);
  TraceScope ts("kv4_read", "byte", tokens * (token_bytes(C) + (dtype == GPTQ_F32 ? 8.0 : 4.0) * C.heads * C.head_dim), s);
  const int launch = next_launch();
  auto go = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    kv4_read_kernel<T><<<grd, THREADS, 0, s>>>(C, table, width, cu, start, count, tokens, n, p, static_cast<T*>(v), st,
                                               launch);
  };
  if (dtype == GPTQ_F32) go(static_cast<float*>(k));
  else if (dtype == GPTQ_F16) go(static_cast<__half*>(k));
  else go(static_cast<__nv_bfloat16*>(k));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
