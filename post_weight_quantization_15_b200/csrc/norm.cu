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
// Bound: HBM.  A row is read once into registers and every statistic is taken there; x, y and
// the gate are read and xn and h written once; the parameters come from L1 and are applied a
// row piece at a time, so that x and y are all that a thread holds (of 24 values or more y
// alone: x is read when it is added).  Rows of up to 1024 values take a warp each, 8 to 32
// values per thread, rows of up to 128 and 64 a half and a quarter of one (no block barrier;
// 200,000 rows of 64: 99 us with a warp each, 32 so; 40,906 rows of 576: 73 us with a block
// each, 50 so), longer rows a block of 32 values per thread (fewer threads meet at the
// barriers: 4000 rows of 8192 with norms on both sides 84 us with 16 values, 65 so; one row of
// 4096 though takes 8 us with 16 and 10 with 32, hence 16 where rows are few).  Where rows do
// not start on 16-byte boundaries (an
// odd d or stride) a thread of a 16-bit stream still takes eight consecutive values: it reads
// the aligned 16-byte pieces that hold them and shifts, and writes by way of shared memory,
// where each thread picks up what belongs to one aligned piece; single values only at a row's
// ends.  (fp32 streams read single values side by side.)  32768 rows of 4096, bf16 with fp32
// Y: 203 us, 1.01 of the measured copy bandwidth.  2039 rows of 5125, fp16, norms on both
// sides: 117 us with everything in registers that spilled, 65 with single values, 57 shifted, 51
// with three blocks per SM; about 1480 instructions per warp and row bound it.
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
  int y_dtype, p_dtype;
  int tokens, d;
  float alpha, eps;
  int center;
};

constexpr int ANY = -1;
constexpr int FEW = 148 * 2;              // rows below which their latency counts, not their number

// A row's threads and their places.  T = 0: any number of threads with eight consecutive
// values per piece, which lie on 16-byte boundaries; ANY: the same on any boundaries; else T
// threads with single values side by side.
template <int T>
struct Row {
  __device__ static __forceinline__ int threads() { return T > 0 ? T : (int)blockDim.x; }
  __device__ static __forceinline__ int at(int v, int e) {
    return T <= 0 ? (v * (int)blockDim.x + (int)threadIdx.x) * 8 + e : (v * 8 + e) * T + (int)threadIdx.x;
  }
};

// Sum over the row's threads (8, 16 or 32 of a warp, or the whole block through `part`, its own
// for each sum).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    if (o < Row<T>::threads()) v += w;
  }
  if (Row<T>::threads() <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = Row<T>::threads() >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// w[i] <- the word that starts `by` bytes (even, below 16) after w[i], i < N.
template <int N>
__device__ __forceinline__ void shift(uint32_t (&w)[N + 4], uint32_t by) {
  if (by & 8) {
#pragma unroll
    for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
  }
  if (by & 4) {
#pragma unroll
    for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
  }
  if (by & 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
}

// Eight values from e0 (a multiple of 8) of a row on any boundary.  Only aligned pieces that
// hold a value of the row are read.
template <typename S>
__device__ __forceinline__ void load8_any(const S* row, int d, int e0, float (&x)[8]) {
  constexpr int N = sizeof(S) * 2;        // words of eight values
  const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) - mis) + e0 / 8 * (N / 4);
  const int left = (d - e0) * (int)sizeof(S) + (int)mis;  // bytes of the row from p on
  uint32_t w[N + 4];
#pragma unroll
  for (int i = 0; i < N / 4 + 1; ++i) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (left > 16 * i && (i < N / 4 || mis != 0)) u = p[i];
    w[4 * i] = u.x;
    w[4 * i + 1] = u.y;
    w[4 * i + 2] = u.z;
    w[4 * i + 3] = u.w;
  }
  if (mis != 0) shift<N>(w, mis);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(S) == 4) {
      x[2 * i] = __uint_as_float(w[2 * i]);
      x[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
    } else {
      unpack2(w[i], x[2 * i], x[2 * i + 1], S());
    }
  }
  if (e0 + 8 > d) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e0 + e >= d) x[e] = 0.f;
  }
}

// Piece v (eight values) of a row; values past d read as 0.
template <int T, typename S>
__device__ __forceinline__ void load_piece(const S* row, int d, int v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
  if constexpr (T == 0) {
    if (Row<T>::at(v, 0) < d) load8(row + Row<T>::at(v, 0), x);
  } else if constexpr (T == ANY) {
    load8_any(row, d, Row<T>::at(v, 0), x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (Row<T>::at(v, e) < d) x[e] = load_as_float(row + Row<T>::at(v, e));
  }
}

template <int V, int T, typename S>
__device__ __forceinline__ void load_row(const S* row, int d, float (&x)[V * 8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float t[8];
    load_piece<T>(row, d, v, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[v * 8 + e] = t[e];
  }
}

// Runs f with a row pointer of the type that `dtype` names.
template <typename F>
__device__ __forceinline__ void typed(const void* p, int64_t off, int dtype, F f) {
  if (dtype == GPTQ_F32) f(static_cast<const float*>(p) + off);
  else if (dtype == GPTQ_F16) f(static_cast<const __half*>(p) + off);
  else f(static_cast<const __nv_bfloat16*>(p) + off);
}

// x <- op(x, parameter), piece by piece.
template <int V, int T, typename F>
__device__ __forceinline__ void apply(const void* p, int64_t off, int dtype, int d, float (&x)[V * 8], F op) {
  typed(p, off, dtype, [&](auto* row) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t[8];
      load_piece<T>(row, d, v, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v * 8 + e] = op(x[v * 8 + e], t[e]);
    }
  });
}

// A row of 16-bit values to any boundary, by way of `buf` (16 bytes for each eight values).
template <int V, typename S>
__device__ __forceinline__ void store_any(S* row, int d, const float (&x)[V * 8], uint4* buf, bool real) {
  const int n = (int)blockDim.x, pieces = (d + 7) / 8;
  if (n <= 32) __syncwarp();              // the last row's readers are done
  else __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float* y = &x[v * 8];
    const int i = v * n + (int)threadIdx.x;
    if (i < pieces) buf[i] = make_uint4(pack2(y[0], y[1], S()), pack2(y[2], y[3], S()), pack2(y[4], y[5], S()), pack2(y[6], y[7], S()));
  }
  if (n <= 32) __syncwarp();
  else __syncthreads();
  const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
  const int off = (int)mis / 2;           // piece c of memory: values 8 c - off .. 8 c - off + 7
  for (int c = (int)threadIdx.x; real && c * 8 - off < d; c += n) {
    const uint4 a = c > 0 ? buf[c - 1] : make_uint4(0, 0, 0, 0);
    const uint4 b = c < pieces ? buf[c] : make_uint4(0, 0, 0, 0);
    uint32_t w[8] = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    if (mis != 0) {
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      shift<4>(w, 16 - mis);
    }
    const int e0 = c * 8 - off;
    if (e0 >= 0 && e0 + 8 <= d) {
      *reinterpret_cast<uint4*>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e0 + e >= 0 && e0 + e < d)
          reinterpret_cast<uint16_t*>(row)[e0 + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
  }
}

template <int V, int T, typename S>
__device__ __forceinline__ void store_row(S* row, int d, const float (&x)[V * 8], uint4* buf, bool real) {
  if constexpr (T == ANY) {
    if constexpr (sizeof(S) == 2) store_any<V>(row, d, x, buf, real);
    return;
  }
  if (!real) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (T == 0) {
      if (Row<T>::at(v, 0) < d) store8(row + Row<T>::at(v, 0), &x[v * 8]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (Row<T>::at(v, e) < d) store_from_float(row + Row<T>::at(v, e), x[v * 8 + e]);
    }
  }
}

// x <- N(x; w, b), the row's values in registers (values past d are 0 and stay unused).
template <int V, int T>
__device__ __forceinline__ void norm_row(float (&x)[V * 8], const void* w, const void* b, const NormArgs& A,
                                         float (*part)[32]) {
  const float inv_d = 1.f / (float)A.d;
  if (A.center) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V * 8; ++i) s += x[i];
    const float mean = row_sum<T>(s, part[0]) / (float)A.d;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[v * 8 + e] = Row<T>::at(v, T == 0 ? 0 : e) < A.d ? x[v * 8 + e] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V * 8; ++i) q = fmaf(x[i], x[i], q);
  const float r = rsqrtf(row_sum<T>(q, part[1]) * inv_d + A.eps);
  apply<V, T>(w, 0, A.p_dtype, A.d, x, [r](float a, float p) { return a * r * p; });
  if (b != nullptr) apply<V, T>(b, 0, A.p_dtype, A.d, x, [](float a, float p) { return a + p; });
}

// Rows of blockDim.x threads: blockDim.y rows of part of a warp each (WARPS; T 0, ANY or 32), or
// one row per block of up to MAXT threads (384: three blocks to an SM, which hide each other's
// barriers; four would spill).
template <typename TX, int V, int T, bool WARPS, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 384 ? 3 : 1024 / MAXT)
add_norm_kernel(const NormArgs A, const int32_t* st) {
  __shared__ float part[4][32];
  extern __shared__ uint4 pieces[];       // ANY: 16 bytes for each eight values of the block's rows
  uint4* buf = pieces + (int)threadIdx.y * (V * (int)blockDim.x);
  if (has_error(st)) return;
  int row = WARPS ? (int)(blockIdx.x * blockDim.y + threadIdx.y) : (int)blockIdx.x;
  // a warp's last rows may be none: it goes through the last one again and writes nothing
  const bool real = !WARPS || row < A.tokens;
  if (WARPS) row = min(row, A.tokens - 1);
  const TX* X = static_cast<const TX*>(A.X) + (int64_t)row * A.ld_x;
  float y[V * 8];
  if (A.Y == nullptr) {
    load_row<V, T>(X, A.d, y);
  } else {
    float x[V * 8];
    typed(A.Y, (int64_t)row * A.ld_y, A.y_dtype, [&](auto* r) { load_row<V, T>(r, A.d, y); });
    if constexpr (V <= 2) load_row<V, T>(X, A.d, x);    // early; of 32 values only y is held through the norm
    if (A.post_weight != nullptr) norm_row<V, T>(y, A.post_weight, A.post_bias, A, part);
    if (A.gate != nullptr)
      apply<V, T>(A.gate, (int64_t)row * A.ld_gate, A.p_dtype, A.d, y, [](float a, float g) { return a * g; });
    if constexpr (V > 2) load_row<V, T>(X, A.d, x);
#pragma unroll
    for (int i = 0; i < V * 8; ++i) y[i] = round_to<TX>(fmaf(A.alpha, y[i], x[i]));
    store_row<V, T>(static_cast<TX*>(A.Xn) + (int64_t)row * A.ld_xn, A.d, y, buf, real);
  }
  norm_row<V, T>(y, A.weight, A.bias, A, part + 2);
  store_row<V, T>(static_cast<TX*>(A.h) + (int64_t)row * A.ld_h, A.d, y, buf, real);
}

template <typename TX>
void launch(const NormArgs& A, bool vec, const int32_t* st, cudaStream_t s) {
  const unsigned rows = (unsigned)A.tokens;
  // threads of a row that a warp holds; rows of a block of 256
  const unsigned lanes = A.d <= 64 ? 8 : (A.d <= 128 ? 16 : 32);
  const dim3 warps(lanes, 256 / lanes);
  const unsigned groups = (unsigned)cdiv(A.tokens, 256 / lanes);
  if (vec) {
    const bool few = A.tokens < FEW && A.d <= 16384;
    const unsigned thr = (unsigned)(cdiv(cdiv(A.d, few ? 16 : 32), 32) * 32);
    if (A.d <= 256) add_norm_kernel<TX, 1, 0, true, 256><<<groups, warps, 0, s>>>(A, st);
    else if (A.d <= 512) add_norm_kernel<TX, 2, 0, true, 256><<<groups, warps, 0, s>>>(A, st);
    else if (few) add_norm_kernel<TX, 2, 0, false, 1024><<<rows, thr, 0, s>>>(A, st);
    else if (A.d <= 768) add_norm_kernel<TX, 3, 0, true, 256><<<groups, warps, 0, s>>>(A, st);
    else if (A.d <= 1024) add_norm_kernel<TX, 4, 0, true, 256><<<groups, warps, 0, s>>>(A, st);
    else add_norm_kernel<TX, 4, 0, false, 1024><<<rows, thr, 0, s>>>(A, st);
    return;
  }
  if constexpr (sizeof(TX) == 2) {
    if (A.d <= 256) add_norm_kernel<TX, 1, ANY, true, 256><<<groups, warps, 256 * 16, s>>>(A, st);
    else if (A.d <= 512) add_norm_kernel<TX, 2, ANY, true, 256><<<groups, warps, 512 * 16, s>>>(A, st);
    else if (A.d <= 768) add_norm_kernel<TX, 3, ANY, true, 256><<<groups, warps, 768 * 16, s>>>(A, st);
    else if (A.d <= 16384) {
      const unsigned thr = (unsigned)(cdiv(cdiv(A.d, 16), 32) * 32);
      const size_t smem = (size_t)thr * 2 * 16;
      if (thr <= 384) add_norm_kernel<TX, 2, ANY, false, 384><<<rows, thr, smem, s>>>(A, st);
      else add_norm_kernel<TX, 2, ANY, false, 1024><<<rows, thr, smem, s>>>(A, st);
    } else {
      add_norm_kernel<TX, 4, 1024, false, 1024><<<rows, 1024, 0, s>>>(A, st);
    }
  } else {
    const dim3 warp32(32, 8);
    const unsigned groups32 = (unsigned)cdiv(A.tokens, 8);
    if (A.d <= 256) add_norm_kernel<TX, 1, 32, true, 256><<<groups32, warp32, 0, s>>>(A, st);
    else if (A.d <= 512) add_norm_kernel<TX, 2, 32, true, 256><<<groups32, warp32, 0, s>>>(A, st);
    else if (A.d <= 1024) add_norm_kernel<TX, 2, 64, false, 64><<<rows, 64, 0, s>>>(A, st);
    else if (A.d <= 2048) add_norm_kernel<TX, 2, 128, false, 128><<<rows, 128, 0, s>>>(A, st);
    else if (A.d <= 4096) add_norm_kernel<TX, 2, 256, false, 256><<<rows, 256, 0, s>>>(A, st);
    else if (A.d <= 8192) add_norm_kernel<TX, 2, 512, false, 512><<<rows, 512, 0, s>>>(A, st);
    else if (A.d <= 16384) add_norm_kernel<TX, 2, 1024, false, 1024><<<rows, 1024, 0, s>>>(A, st);
    else add_norm_kernel<TX, 4, 1024, false, 1024><<<rows, 1024, 0, s>>>(A, st);
  }
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
             y_dtype, p_dtype, tokens, d, alpha, eps, center};
  const bool vec = d % 8 == 0 && vec_ok(X, ld_x, x_dtype) && vec_ok(Y, ld_y, y_dtype) && vec_ok(h, ld_h, x_dtype) &&
                   (Y == nullptr || vec_ok(Xn, ld_xn, x_dtype)) && vec_ok(weight, 0, p_dtype) &&
                   vec_ok(bias, 0, p_dtype) && vec_ok(post_weight, 0, p_dtype) && vec_ok(post_bias, 0, p_dtype) &&
                   vec_ok(gate, ld_gate, p_dtype);
  const double n = (double)tokens * d, b = (double)width(x_dtype);
  TraceScope ts("add_norm", "byte", n * (Y != nullptr ? 3 * b + (double)width(y_dtype) : 2 * b) +
                                        (gate != nullptr && ld_gate != 0 ? n * (double)width(p_dtype) : 0.0), s);
  if (x_dtype == GPTQ_F32) launch<float>(A, vec, st, s);
  else if (x_dtype == GPTQ_F16) launch<__half>(A, vec, st, s);
  else launch<__nv_bfloat16>(A, vec, st, s);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace gptq
