// The cache of keys and values held in 4 bits: tokens written into it (gptq_kv4_append)
// and read back (gptq_kv4_read).
//
// Each group of a head's features of one token has its own fp16 scale s and integer zero
// point z, chosen as the layer quantizer chooses an asymmetric group's: the range holds 0,
// lo = min(x, 0), hi = max(x, 0) (-1 and 1 when equal), s = fp16((hi - lo) / 15) within
// fp16's positive range, z = clamp(rint(-lo / s), 0, 15), code c = clamp(rint(x / s) + z,
// 0, 15), value s (c - z).  x / s is a tie or at least 2^-17 relative away from one (x and s
// have few bits), so its integer needs no IEEE division: with r = 1 / s the product q = x r
// is within 2^-22 of it, and q + r (x - q s), the residual exact but for its own rounding,
// lands on a tie's few bits exactly.  Adding 1.5 . 2^23 rounds to the nearest even integer
// and leaves it in the low bits, where the eight codes of a word are summed under their
// shifts (the constant's and the zero point's shares taken off once).
//
// Bound: HBM, with the issue slots close behind (about twelve instructions per value).  A
// thread quantizes eight features (16 bytes in, one word of codes out); the group / 8
// threads of a group find its range with shuffles, on packed 16-bit values.  A block takes
// a few consecutive tokens, their places looked up once, and every thread reads its keys
// and values of two tokens before it uses the first.  (One token per block, IEEE divisions and
// integer conversions took 366 us for 15,625 tokens of 32 heads x 128 written and read back
// where these take 203.)
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

// Tokens t0 .. t0 + n - 1 of the batch: the first head's row in the cache of each, or -1.
__device__ __forceinline__ void find_rows(const KV4Cache& C, const int32_t* table, int width, const int32_t* cu,
                                          const int32_t* start, int count, int t0, int n, int64_t* rows, int32_t* st) {
  if ((int)threadIdx.x < n) {
    const int t = t0 + (int)threadIdx.x, b = packed_sequence(cu, count, t);
    int64_t row = -1;
    if (b >= 0) {
      const int64_t pos = (start != nullptr ? (int64_t)start[b] : 0) + (t - cu[b]);
      const int page = kv4_page(C, table, width, b, pos);
      if (page < 0) set_error(st, GPTQ_ERR_INVALID_ARG, t, STAGE_KV4);
      else row = kv4_row(C, page, 0, (int)(pos & (C.page_size - 1)));
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
}

// A thread's place: unit u (of heads . words) of every subs-th token, or units u, u + 256, ...
// of every token.
struct Units {
  int per, sub, subs, u0;
  __device__ __forceinline__ Units(const KV4Cache& C) {
    per = C.heads * (C.head_dim / 8);
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

// Eight values of a group (`lanes` threads share it) -> their word of codes, and the group's
// scale and zero point; `bad` if the group holds a NaN or an infinity.  Whole warp.
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const uint4& raw, int lanes, __half2& par, bool& bad) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // (-smallest, largest) as one pair, 0 included
  const uint32_t lo = min2(min2(w[0], w[1], T()), min2(w[2], w[3], T()), T());
  const uint32_t hi = max2(max2(w[0], w[1], T()), max2(w[2], w[3], T()), T());
  const uint32_t neg = lo ^ 0x80008000u;
  uint32_t ends = max2(__byte_perm(neg, hi, 0x5410), __byte_perm(neg, hi, 0x7632), T());
  ends = max2(ends, 0u, T());
  for (int o = 1; o < lanes; o <<= 1) ends = max2(ends, __shfl_xor_sync(0xffffffffu, ends, o), T());
  float2 e = wide2(ends, T());
  bad = !(fmaxf(e.x, e.y) < INFINITY) || e.x != e.x || e.y != e.y;
  if (e.x == 0.f && e.y == 0.f) e = make_float2(1.f, 1.f);
  const __half s16 = __float2half_rn(fminf(fmaxf(__fdiv_rn(e.y + e.x, 15.f), 5.9604644775390625e-08f), 65504.f));
  const float s = __half2float(s16), r = 1.f / s;
  const float z = fminf(rintf(__fdiv_rn(e.x, s)), 15.f);
  const float most = 15.f - z;
  constexpr float ROUND = 12582912.f;     // 1.5 . 2^23
  uint32_t word = ((uint32_t)(int)z - __float_as_uint(ROUND)) * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = wide2(w[i], T());
    const float v[2] = {x.x, x.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float q = v[k] * r;
      q = fmaf(r, fmaf(-q, s, v[k]), q);
      q = fminf(fmaxf(q, -z), most) + ROUND;
      word += __float_as_uint(q) << (8 * i + 4 * k);
    }
  }
  par = __halves2half2(s16, __float2half_rn(z));
  return word;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(const __grid_constant__ KV4Cache C,
                                                             const __grid_constant__ KVInput in, const int32_t* table,
                                                             int width, const int32_t* cu, const int32_t* start,
                                                             int count, int tokens, int per_block, int32_t* st) {
  __shared__ int64_t rows[MOST];
  if (has_error(st)) return;
  const int t0 = (int)blockIdx.x * per_block, n = min(per_block, tokens - t0);
  find_rows(C, table, width, cu, start, count, t0, n, rows, st);
  const Units U(C);
  const int words = C.head_dim / 8, lanes = C.group / 8, groups = C.head_dim / C.group;
  const int lw = __ffs(words) - 1, ll = __ffs(lanes) - 1;
  // every thread goes through every step: the shuffles take whole warps
  for (int step = 0; step < U.per; step += THREADS) {
    const int u = U.u0 + step, head = u >> lw, w = u & (words - 1);
    for (int i0 = 0; i0 < n; i0 += 2 * U.subs) {
      uint4 raw[2][2];
      int64_t row[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int i = i0 + a * U.subs + U.sub;
        row[a] = u < U.per && U.sub < U.subs && i < n ? rows[i] : -1;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          raw[a][kv] = make_uint4(0, 0, 0, 0);
          if (row[a] >= 0)
            raw[a][kv] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(in.p[kv]) +
                                                               (int64_t)(t0 + i) * in.token_stride[kv] +
                                                               head * in.head_stride[kv] + w * 8));
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          __half2 par;
          bool bad;
          uint32_t word = quantize8<T>(raw[a][kv], lanes, par, bad);
          if (row[a] < 0) continue;
          if (bad) {                      // the whole group reads back as NaN
            word = 0;
            par = __halves2half2(__ushort_as_half((unsigned short)0x7fffu), __ushort_as_half((unsigned short)0));
            if ((w & (lanes - 1)) == 0) set_error(st, GPTQ_ERR_NONFINITE, t0 + i0 + a * U.subs + U.sub, STAGE_KV4);
          }
          const int64_t at = row[a] + (int64_t)head * C.page_size;
          C.codes[kv][at * words + w] = (int32_t)word;
          if ((w & (lanes - 1)) == 0) reinterpret_cast<__half2*>(C.params[kv])[at * groups + (w >> ll)] = par;
        }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(const __grid_constant__ KV4Cache C, const int32_t* table,
                                                           int width, const int32_t* cu, const int32_t* start,
                                                           int count, int tokens, int per_block, T* k, T* v,
                                                           int32_t* st) {
  __shared__ int64_t rows[MOST];
  if (has_error(st)) return;
  const int t0 = (int)blockIdx.x * per_block, n = min(per_block, tokens - t0);
  find_rows(C, table, width, cu, start, count, t0, n, rows, st);
  const Units U(C);
  if (U.sub >= U.subs) return;
  const int words = C.head_dim / 8, lanes = C.group / 8, groups = C.head_dim / C.group;
  const int lw = __ffs(words) - 1, ll = __ffs(lanes) - 1;
  for (int u = U.u0; u < U.per; u += THREADS) {
    const int head = u >> lw, w = u & (words - 1);
#pragma unroll 2
    for (int i = U.sub; i < n; i += U.subs) {
      const int64_t row = rows[i];
      if (row < 0) continue;
      const int64_t at = row + (int64_t)head * C.page_size;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t word = (uint32_t)C.codes[kv][at * words + w];
        const __half2 par = reinterpret_cast<const __half2*>(C.params[kv])[at * groups + (w >> ll)];
        // 2^23 + code is the code in the low bits of 2^23's pattern; less 2^23 + z it is code - z, exactly
        const float s = __low2float(par), z = 8388608.f + __high2float(par);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s * (__uint_as_float(0x4B000000u | ((word >> (4 * e)) & 15u)) - z);
        store8((kv ? v : k) + ((int64_t)(t0 + i) * C.heads + head) * C.head_dim + w * 8, x);
      }
    }
  }
}

// Tokens of a block: as many as keep its threads busy, more while there are blocks to spare.
int tokens_per_block(const KV4Cache& C, int tokens) {
  const int per = C.heads * (C.head_dim / 8);
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
  const int n = tokens_per_block(C, tokens);
  const unsigned grd = (unsigned)cdiv(tokens, n);
  TraceScope ts("kv4_append", "byte", tokens * (token_bytes(C) + 4.0 * C.heads * C.head_dim), s);
  if (dtype == GPTQ_F16)
    kv4_append_kernel<__half><<<grd, THREADS, 0, s>>>(C, in, table, width, cu, start, count, tokens, n, st);
  else
    kv4_append_kernel<__nv_bfloat16><<<grd, THREADS, 0, s>>>(C, in, table, width, cu, start, count, tokens, n, st);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

int launch_kv4_read(const KV4Cache& C, const int32_t* table, int width, const int32_t* cu, const int32_t* start,
                    int count, int tokens, int dtype, void* k, void* v, int32_t* st, cudaStream_t s) {
  const int n = tokens_per_block(C, tokens);
  const unsigned grd = (unsigned)cdiv(tokens, n);
  TraceScope ts("kv4_read", "byte", tokens * (token_bytes(C) + (dtype == GPTQ_F32 ? 8.0 : 4.0) * C.heads * C.head_dim), s);
  auto go = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    kv4_read_kernel<T><<<grd, THREADS, 0, s>>>(C, table, width, cu, start, count, tokens, n, p, static_cast<T*>(v), st);
  };
  if (dtype == GPTQ_F32) go(static_cast<float*>(k));
  else if (dtype == GPTQ_F16) go(static_cast<__half*>(k));
  else go(static_cast<__nv_bfloat16*>(k));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
