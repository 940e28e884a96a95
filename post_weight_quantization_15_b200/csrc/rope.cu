// The rotary split of a q/k/v product (gptq_rope_qkv): the fp32 rows a product of the
// stacked q, k and v layers gives, plus their bias, become q, k and v in 16 bits; q and k
// features (a, b) of a pair turn by their token's angle,
//
//   a' = a cos - b sin        b' = a sin + b cos,
//
// pairs being (i, i + rot/2) of a head, or (2i, 2i + 1) when interleaved; features from
// rot on and all of v pass through.  The tables hold the cosines and sines per position.
//
// Bound: HBM (4 bytes in, 2 out per value).  One pass.  A thread keeps the same W pairs of
// every head it takes, so that their cosines and sines are read once into registers and a
// head costs two 16-byte loads (W = 4 of fp32, 8 of 16-bit types, side by side across a
// warp) and two stores; W = 1 for any even rot and any alignment.  Where there are tokens
// enough, a thread takes four heads or more and a block as many tokens as its threads hold.
// 8192 tokens of 96 heads x 128, fp32 in, bias: 190 us with 16 values per thread and the tables
// read again for every head, 117 so, 111 with two heads in flight instead of four and five
// blocks per SM (84% of the copy bandwidth); 89,731 tokens of 6 heads: 227 us with one token
// per block, 80 with eight.
#include "common.cuh"
#include "internal.h"
#include "vec_io.cuh"

namespace gptq {

namespace {

constexpr int THREADS = 256;
constexpr int ENOUGH = 148 * 4;           // blocks that fill the SMs

struct RopeArgs {
  const void* X;
  int64_t ld;
  const float* bias;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int max_pos, rot, interleaved;
  int tokens, hq, hk, d;
  void* q;
  void* k;
  void* v;
  int launch;                             // the call's number, for the errors it records
};

template <int W, typename T>
__device__ __forceinline__ void loadw(const T* p, float (&v)[W]) {
  if constexpr (W == 8) load8(p, v);
  else if constexpr (W == 4) load4(p, v);
  else v[0] = load_as_float(p);
}
template <int W, typename T>
__device__ __forceinline__ void storew(T* p, const float (&v)[W]) {
  if constexpr (W == 8) store8(p, v);
  else if constexpr (W == 4) store4(p, v);
  else store_from_float(p, v[0]);
}

// Thread: pairs j W .. j W + W - 1 of heads h0, h0 + subs, ... of one token; a head has `units` =
// d / (2 W) such pieces (W = 1: rot and d even), the first rot / (2 W) of them rotated in q and k
// heads.  A block has `per` tokens of subs . units threads, or (per 1) a part of one token's heads.
template <typename TX, typename TO, int W, bool BIAS>
__global__ void __launch_bounds__(THREADS, W == 8 ? 4 : 5)
rope_qkv_kernel(const __grid_constant__ RopeArgs A, int units, int subs, int per, int per_block, int32_t* st) {
  if (stopped(st, A.launch)) return;       // (threads work by themselves)
  const int turned = A.hq + A.hk, heads = turned + A.hk;
  const int sub = (int)threadIdx.x / units % subs, own = (int)threadIdx.x / (units * subs);
  const int t = (int)blockIdx.x * per + own;
  const int begin = (int)blockIdx.y * per_block, end = min(heads, begin + per_block);
  if (own >= per || t >= A.tokens) return;
  int pos = A.positions != nullptr ? A.positions[t] : t;
  if (A.rot > 0 && (pos < 0 || pos >= A.max_pos)) {
    if (threadIdx.x % (units * subs) == 0 && blockIdx.y == 0)
      set_own_error(st, A.launch, GPTQ_ERR_INVALID_ARG, t, STAGE_ROPE);
    pos = 0;
  }
  for (int j = (int)threadIdx.x % units; j < units; j += THREADS) {      // (a head may have more pieces than the block threads)
    const bool turn = j * 2 * W < A.rot;
    // the piece's two runs of W values inside a head
    const bool split = turn && !A.interleaved;
    const int i0 = split ? j * W : j * 2 * W;
    const int i1 = split ? j * W + A.rot / 2 : j * 2 * W + W;
    float c[W], s[W];
    if (turn) {
      loadw<W>(A.cos + (int64_t)pos * (A.rot / 2) + j * W, c);
      loadw<W>(A.sin + (int64_t)pos * (A.rot / 2) + j * W, s);
    }
    const TX* row = static_cast<const TX*>(A.X) + (int64_t)t * A.ld;
#pragma unroll 2
    for (int head = begin + sub; head < end; head += subs) {
      const int c0 = head * A.d + i0, c1 = head * A.d + i1;
      float a[W], b[W];
      loadw<W>(row + c0, a);
      loadw<W>(row + c1, b);
      if constexpr (BIAS) {
        float x[W], y[W];
        loadw<W>(A.bias + c0, x);
        loadw<W>(A.bias + c1, y);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          a[i] += x[i];
          b[i] += y[i];
        }
      }
      if (turn && head < turned) {
        if (A.interleaved) {
          // pair i of the piece: values 2i and 2i + 1 of the 2 W consecutive ones
          float x[2 * W];
#pragma unroll
          for (int i = 0; i < W; ++i) { x[i] = a[i]; x[W + i] = b[i]; }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float lo = x[2 * i], hi = x[2 * i + 1];
            x[2 * i] = lo * c[i] - hi * s[i];
            x[2 * i + 1] = lo * s[i] + hi * c[i];
          }
#pragma unroll
          for (int i = 0; i < W; ++i) { a[i] = x[i]; b[i] = x[W + i]; }
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float lo = a[i], hi = b[i];
            a[i] = lo * c[i] - hi * s[i];
            b[i] = lo * s[i] + hi * c[i];
          }
        }
      }
      TO* dst;
      if (head < A.hq) dst = static_cast<TO*>(A.q) + ((int64_t)t * A.hq + head) * A.d;
      else if (head < turned) dst = static_cast<TO*>(A.k) + ((int64_t)t * A.hk + head - A.hq) * A.d;
      else dst = static_cast<TO*>(A.v) + ((int64_t)t * A.hk + head - turned) * A.d;
      storew<W>(dst + i0, a);
      storew<W>(dst + i1, b);
    }
  }
}

template <typename TX, typename TO, int W>
void launch_w(const RopeArgs& A, int32_t* st, cudaStream_t s) {
  const int units = A.d / (2 * W), heads = A.hq + 2 * A.hk;
  const int most = THREADS / units > 0 ? THREADS / units : 1;
  // many tokens: four heads or more per thread, several tokens per block; few: a head per thread
  const bool many = (int64_t)A.tokens * units * heads >= (int64_t)ENOUGH * THREADS * 4;
  const int quarter = (heads + 3) / 4;
  int subs = many ? (quarter < most ? quarter : most) : (heads < most ? heads : most);
  const int per = many && units <= THREADS ? THREADS / (units * subs) : 1;
  const int64_t want = cdiv(heads, subs);
  const int64_t split = many ? 1 : (want < 64 ? want : 64);
  const int per_block = (int)cdiv(heads, split);
  const dim3 grd((unsigned)cdiv(A.tokens, per), (unsigned)cdiv(heads, per_block));
  if (A.bias != nullptr) rope_qkv_kernel<TX, TO, W, true><<<grd, THREADS, 0, s>>>(A, units, subs, per, per_block, st);
  else rope_qkv_kernel<TX, TO, W, false><<<grd, THREADS, 0, s>>>(A, units, subs, per, per_block, st);
}

template <typename TX, typename TO>
void launch(const RopeArgs& A, int w, int32_t* st, cudaStream_t s) {
  if constexpr (sizeof(TX) == 2)
    if (w == 8) { launch_w<TX, TO, 8>(A, st, s); return; }
  if (w >= 4) launch_w<TX, TO, 4>(A, st, s);
  else launch_w<TX, TO, 1>(A, st, s);
}

template <typename TX>
void launch_out(const RopeArgs& A, int w, int out_dtype, int32_t* st, cudaStream_t s) {
  if (out_dtype == GPTQ_F16) launch<TX, __half>(A, w, st, s);
  else launch<TX, __nv_bfloat16>(A, w, st, s);
}

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

int launch_rope_qkv(const void* X, int x_dtype, int64_t ld, const float* bias, const float* cos, const float* sin,
                    int max_pos, int rot, int interleaved, const int32_t* positions, int tokens, int hq, int hk,
                    int d, int out_dtype, void* q, void* k, void* v, int32_t* st, cudaStream_t s) {
  RopeArgs A{X, ld, bias, cos, sin, positions, max_pos, rot, interleaved, tokens, hq, hk, d, q, k, v, next_launch()};
  const int xb = x_dtype == GPTQ_F32 ? 4 : 2;
  const bool al = al16(X) && (ld * xb) % 16 == 0 && al16(q) && al16(k) && al16(v) && (rot == 0 || (al16(cos) && al16(sin))) &&
                  (bias == nullptr || al16(bias));
  int w = 1;
  if (al && rot % 16 == 0 && d % 16 == 0 && xb == 2) w = 8;
  else if (al && rot % 8 == 0 && d % 8 == 0) w = 4;
  const double cols = (double)(hq + 2 * hk) * d;
  TraceScope ts("rope_qkv", "byte", tokens * (cols * (xb + 2) + 4.0 * rot), s);
  if (x_dtype == GPTQ_F32) launch_out<float>(A, w, out_dtype, st, s);
  else if (x_dtype == GPTQ_F16) launch_out<__half>(A, w, out_dtype, st, s);
  else launch_out<__nv_bfloat16>(A, w, out_dtype, st, s);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
