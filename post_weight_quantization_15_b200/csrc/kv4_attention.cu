// Attention of one query token per sequence over its keys and values in the 4-bit cache
// (gptq_kv4_attention): o = sum_t softmax_t(scale q . k_t) v_t over the sequence's tokens,
// k_t and v_t = s (c - z) read from the cache's pages, hq / hk query heads per k/v head.
// A sequence without tokens gives 0.
//
// Bound: HBM, the codes and their scales read once (and close behind it the issue slots
// that unpack them).  Products are m16n8k16 (mma.sync, fp16 in, fp32 sums) with the query
// heads of a k/v head, eight at a time, as columns and the cache as rows (tokens for the
// scores, features for the values), so that no row is wasted on a group of eight or fewer:
//   scores   K [16 tokens, D] . q^T [D, 8]; the weights, transposed in registers
//            (movmatrix), are the B operand of  V^T [16 features, 16 tokens] . p^T.
// Two codes are masked into the mantissas of the fp16 pair 1024 + c (or 1024 + 16 c, from
// the next nibble) and one packed subtraction (or fma) leaves c - z, an exact fp16 integer;
// scales stay outside:
//   q . k_t = sum over groups of s sum q (c - z), q held in fp16 under a power of two per
//            row (its largest value in [2^11, 2^12): both 16-bit types fit, values below
//            2^-25 of the largest rounded);
//   sum_t p_t s_t (c_t - z_t) with p_t s_t rounded to fp16 under a power of two per group
//            (largest value below 2^15).
// (Without the subtraction, c as an fp16 subnormal and z taken off the sums, the sums
// cancel: the tensor cores align such products by their unnormalised exponents, and
// results near 0 were off by 2^-17 of a scale.)
// The running maximum is kept while no score passes it by more than 2^4 in the weights, so
// lanes exchange maxima only when it moves.
//
// Work: the sequences' tiles of 32 tokens, all heads, in one line, cut into equal runs, one
// per warp (a head set counts one tile more than it has, for its queries and its end).  A
// warp has a ring of its own that asynchronous 16-byte copies fill (the codes' pieces
// swizzled against bank conflicts) and waits for no other warp.  A head set whose tiles
// fall to one warp is finished there, from registers; of the others, what goes on past a
// warp's run is joined in the block first, and the blocks' and the last warp's (maximum,
// sum, weighted values) are left in the workspace, where kv4_join_kernel, a dependent
// launch, joins them in a fixed order.
//
// 131,071 tokens x 64/8 heads of 128, groups of 128: 51 us with cold caches, 21.8 at the copy
// bandwidth; 16 ragged sequences x 32 heads, groups of 32: 74 and 27.7.  (A block per query
// head and token after token: 68.8 and 2.41 ms; rows padded to 16 heads, TMA rings and joins
// per head set in the block: 100 and 620 us; cache as rows: 67 and 332; a run per warp: 65 and
// 104; one lop3 per masked pair: 57 and 82; zero points once per half tile: 51 and 74.)  What
// bounds it: instructions, 640 per tile of 32 tokens, 350 of them unpacking and products, at
// 59 to 63% of the issue slots with the 16 warps per SM that 128 registers allow (20 warps
// spill: 65 and 92 us; three stages per ring: 55 and 90).
#include <math.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

constexpr int PER_SM = 4;
constexpr int BLOCKS = 148 * PER_SM;      // resident blocks: the cut of the work, whatever the device
constexpr int WARPS = 4;
constexpr int RUNS = BLOCKS * WARPS;
constexpr int TT = 32;                    // tokens of a tile
constexpr int STAGES = 2;
constexpr int ROWS = 8;                   // query heads of a product
constexpr float LOG2E = 1.4426950408889634f;
constexpr float KEEP = 4.f;

struct KvaArgs {
  KV4Cache C;
  const void* q;
  void* o;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const int32_t* table;
  const int32_t* lengths;
  float* part_o;                          // [2 RUNS][rows][head_dim]
  float* part_ml;                         // [2 RUNS][rows][2]
  int width, count, per, sets, rows;      // per: query heads of a k/v head, in sets of up to 8 (rows)
  float scale;
  int half;                               // q and o are fp16 (else bf16)
  int launch;                             // the call's number, for the errors it records
};

// Sequence b's tiles (one head set); 0 for a length that the table does not hold.
__device__ __forceinline__ int tiles_of(const KvaArgs& A, int b) {
  const int len = A.lengths[b];
  return len < 0 || len > (int64_t)A.width * A.C.page_size ? 0 : (len + TT - 1) / TT;
}

struct Place {
  int b, hx, t, tiles;                    // sequence, head set, tile of it (tiles: none), tiles of the sequence
};

// A head set has tiles + 1 slots of the line, the last without a tile.
__device__ __forceinline__ int64_t slots_of(int tiles, int heads) { return tiles > 0 ? (int64_t)(tiles + 1) * heads : 0; }

// Walks the line of slots with a window of 32 sequences, one per lane.
struct Finder {
  int b0 = -32;
  int64_t base = 0, total = 0;            // slots before and in the window
  int64_t incl = 0;                       // this lane's sequence and those before it in the window
  int tiles = 0;

  __device__ __forceinline__ void advance(const KvaArgs& A, int heads) {
    const int lane = threadIdx.x & 31;
    base += total;
    b0 += 32;
    const int b = b0 + lane;
    tiles = b < A.count ? tiles_of(A, b) : 0;
    incl = slots_of(tiles, heads);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  // Each lane's slot (not before the window; lanes without one pass want = -1).
  __device__ __forceinline__ Place find(const KvaArgs& A, int heads, int64_t want) {
    Place p{0, 0, 0, 0};
    bool open = want >= 0;
    while (true) {
      const bool here = open && b0 >= 0 && want < base + total;
      const int64_t rel = want - base;
      int lo = 0;                         // the first lane whose incl exceeds rel
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const int64_t v = __shfl_sync(0xffffffffu, incl, lo + o - 1);
        if (here && v <= rel) lo += o;
      }
      const int64_t end = __shfl_sync(0xffffffffu, incl, lo);
      const int n = __shfl_sync(0xffffffffu, tiles, lo);
      if (here) {
        const int64_t r = rel - (end - slots_of(n, heads));
        p.b = b0 + lo;
        // (a quotient in 32 bits wherever it can be one)
        p.hx = r <= UINT32_MAX ? (int)((uint32_t)r / (uint32_t)(n + 1)) : (int)(r / (n + 1));
        p.t = (int)(r - (int64_t)p.hx * (n + 1));
        p.tiles = n;
        open = false;
      }
      if (!__any_sync(0xffffffffu, open) || b0 + 32 >= A.count) return p;
      advance(A, heads);
    }
  }
};

// Run c of the line.
__device__ __forceinline__ int64_t run_begin(int64_t all, int runs, int c) { return all * c / runs; }
__device__ __forceinline__ int run_of(int64_t all, int runs, int64_t slot) {
  int c = (int)(slot * runs / all);
  while (c + 1 < runs && run_begin(all, runs, c + 1) <= slot) ++c;
  return c;
}
// Down to one slot each: 300 tokens x 32/8 heads take 11 us, in runs of at least four 14.
__device__ __forceinline__ int runs_of(int64_t all) { return (int)(all < RUNS ? (all > 0 ? all : 1) : RUNS); }

template <int D, int GROUP>
struct KvaSmem {
  struct Stage {
    uint8_t codes[2][TT * D / 2];         // keys, values: token rows, 16-byte pieces swizzled (piece())
    __half2 params[2][TT * (D / GROUP)];
  };
  Stage ring[WARPS][STAGES];
  int4 desc[WARPS][STAGES];               // sequence, head set, first token (-1: no tile), pages that exist
  float ml[WARPS][ROWS][2];
  int late[WARPS];                        // the run's last head set goes on behind it (2: and is the only one)
  int skip;
  // the parts that go on, over the rings when these are done with
  __device__ __forceinline__ float* part(int w) { return reinterpret_cast<float*>(ring) + w * ROWS * D; }
  static_assert(sizeof(ring) >= WARPS * ROWS * D * sizeof(float), "parts fit");
};

// Where 16-byte piece `i` of token row `row` lies in a stage: a row has D / 32 pieces, and
// rows that would share banks hold them in another order.
template <int D>
__device__ __forceinline__ uint32_t piece(int row, int i) {
  return (uint32_t)(row * (D / 2) + ((i ^ (D == 128 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes -> c - z: the nibbles at bits 0 and 16, or at bits 4 and 20, of x; zero.lo holds
// -(1024 + z) per half, zero.hi -(64 + z).
struct Zero {
  __half2 lo, hi;
};
__device__ __forceinline__ Zero make_zero(__half2 z) {
  return Zero{__hneg2(__hadd2(z, __floats2half2_rn(1024.f, 1024.f))), __hneg2(__hadd2(z, __floats2half2_rn(64.f, 64.f)))};
}
// (x & mask) | 1024's pattern in both halves, in one instruction: with both constants visible
// it is split into two, and the ALU is what bounds this kernel.
__device__ __forceinline__ uint32_t mantissas(uint32_t x, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(0x64006400u));
  return r;
}
struct Masks {
  uint32_t lo, hi;
};
__device__ __forceinline__ Masks make_masks() {
  Masks m;
  asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(m.lo));
  asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(m.hi));
  return m;
}
__device__ __forceinline__ uint32_t code_lo(uint32_t x, const Masks& m, const Zero& z) {
  const uint32_t v = mantissas(x, m.lo);
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&v), z.lo);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t code_hi(uint32_t x, const Masks& m, const Zero& z) {
  const uint32_t v = mantissas(x, m.hi);
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(0.0625f, 0.0625f), z.hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight consecutive q values; o values likewise.
__device__ __forceinline__ void load_q(const KvaArgs& A, int64_t off, float (&x)[8]) {
  if (A.half) load8(static_cast<const __half*>(A.q) + off, x);
  else load8(static_cast<const __nv_bfloat16*>(A.q) + off, x);
}
__device__ __forceinline__ void store_o(const KvaArgs& A, int64_t off, const float* x) {
  if (A.half) store8(static_cast<__half*>(A.o) + off, x);
  else store8(static_cast<__nv_bfloat16*>(A.o) + off, x);
}

// Eight consecutive features of head 2 j + r from the accumulators (u of D / 64); returns
// the first feature.  Groups of 32 exchange with the lane four rows on.
template <int D, int GROUP>
__device__ __forceinline__ int eight(const float (&acc)[D / 16][4], int r, int u, float (&x)[8]) {
  const int g = (threadIdx.x & 31) >> 2;
  if constexpr (GROUP >= 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = acc[4 * u + i][r];
      x[i + 4] = acc[4 * u + i][2 + r];
    }
    return 8 * (8 * u + g);
  } else {
    const bool odd = g >> 2;              // this lane keeps tile pair 2 u, or 2 u + 1
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = acc[4 * u + (k & 1)][r + (k & 2)], hi = acc[4 * u + 2 + (k & 1)][r + (k & 2)];
      const float got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 16), own = odd ? hi : lo;
      x[2 * k] = odd ? got : own;
      x[2 * k + 1] = odd ? own : got;
    }
    return 8 * (4 * (2 * u + odd) + (g & 3));
  }
}

template <int D, int GROUP>
__global__ void __launch_bounds__(WARPS * 32, PER_SM)
kv4_attention_kernel(const __grid_constant__ KvaArgs A, int32_t* st) {
  using Smem = KvaSmem<D, GROUP>;
  constexpr int NG = D / GROUP;           // groups of a row
  constexpr int NW = D / 32;              // words of a key row per lane
  constexpr int MT = D / 16;              // feature tiles of the values
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) S.skip = stopped(st, A.launch);
  const int heads = A.C.heads * A.sets;
  int64_t all = 0;
  for (int b = lane; b < A.count; b += 32) all += slots_of(tiles_of(A, b), heads);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  __syncthreads();
  const int runs = runs_of(all), run = (int)blockIdx.x * WARPS + warp;
  if (S.skip || all == 0 || run - warp >= runs) return;
  // run_begin(all, runs, run), with one long division
  const int64_t each = all <= UINT32_MAX ? (int64_t)((uint32_t)all / (uint32_t)runs) : all / runs;
  const int over = (int)(all - each * runs), b0 = over * run / runs, b1 = over * (run + 1) / runs;   // RUNS^2 < 2^31
  const int64_t begin = each * run + b0;
  const int mine = run < runs ? (int)(each + b1 - b0) : 0;

  // lane i holds what slot (made & ~31) + i needs
  Finder finder;
  const int box = min(A.C.page_size, TT), parts = TT / box;      // tokens of a tile in one page; pages of a tile
  int made = 0;
  uint32_t row0 = 0, row1 = 0;            // (more than 2^32 rows do not fit the device)
  int4 d0 = make_int4(0, 0, 0, 0);
  auto produce = [&]() {
    if (made < mine) {
      if ((made & 31) == 0) {
        const int i = made + lane;
        const Place p = finder.find(A, heads, i < mine ? begin + i : -1);
        d0 = make_int4(0, 0, -1, 0);
        if (p.t < p.tiles) {
          const int head = p.hx / A.sets, t0 = p.t * TT;
          const int len = A.lengths[p.b];
          int ok = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // rows of a second page behind the sequence's end are those of page 0, not used
            const int pos = t0 + k * 16;
            int page = 0;
            if (pos < len) {
              page = kv4_page(A.C, A.table, A.width, p.b, pos);
              if (page < 0) {
                set_own_error(st, A.launch, GPTQ_ERR_INVALID_ARG, p.b, STAGE_KV4_ATTENTION);
                page = 0;
              } else {
                ok |= 1 << k;
              }
            } else if (parts == 1) {
              page = -1;                  // the same page as the first half
            }
            const uint32_t row = (uint32_t)kv4_row(A.C, page, head, pos & (A.C.page_size - 1));
            if (k == 0) row0 = row;
            else row1 = page < 0 ? row0 + 16 : row;
          }
          d0 = make_int4(p.b, p.hx, t0, ok);
        }
      }
      const int src = made & 31, s = made % STAGES;
      const uint32_t r[2] = {__shfl_sync(0xffffffffu, row0, src), __shfl_sync(0xffffffffu, row1, src)};
      if (lane == src) S.desc[warp][s] = d0;
      if (__shfl_sync(0xffffffffu, d0.z, src) >= 0) {
        auto& stage = S.ring[warp][s];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          constexpr int P16 = D / 2;        // pieces of 16 tokens
          const uint32_t dst = smem_addr(stage.codes[kv]) + piece<D>(lane / (D / 32), lane % (D / 32));
          const char* base = reinterpret_cast<const char*>(A.C.codes[kv]) + lane * 16;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < P16 / 32; ++i)    // 32 pieces on, the rows' swizzle repeats
              copy16(dst + (k * P16 + i * 32) * 16, base + (uint64_t)r[k] * (D / 2) + i * 512);
          constexpr int Q16 = 4 * NG;       // pieces of 16 tokens' scales and zero points
          if (lane < 2 * Q16) {
            const int k = lane / Q16;
            copy16(smem_addr(stage.params[kv]) + lane * 16,
                   reinterpret_cast<const char*>(A.C.params[kv]) + (uint64_t)(k ? r[1] : r[0]) * (NG * 4) + (lane % Q16) * 16);
          }
        }
      }
      ++made;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) produce();
  __syncwarp();

  const Masks masks = make_masks();
  // the state of the head set at hand: heads 2 j and 2 j + 1 of it
  float acc[MT][4], m[2], l[2];
  int ve[NG];                             // weights of group i carry 2^(10 - ve[i])
  uint32_t qb[D / 16][2];                 // head g's query as operand
  float rf[2] = {1.f, 1.f};               // log2 of a weight per unit of score
  int used = 0, sets = 0, late = 0;

  while (used < mine) {
    const int4 begins = S.desc[warp][used % STAGES];
    if (begins.z < 0) {                   // a slot without a tile
      __syncwarp();
      ++used;
      produce();
      __syncwarp();
      continue;
    }
    const int b = begins.x, hx = begins.y, len = A.lengths[b];
    const int first = hx / A.sets * A.per + (hx % A.sets) * ROWS, rows = min(ROWS, A.per - (hx % A.sets) * ROWS);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) ve[i] = -127;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    {                                     // its queries as operands
      float x[NW][8];
      float top = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int word = NG == 1 ? NW * j + w : j + 4 * w;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[w][e] = 0.f;
        if (g < rows) load_q(A, (int64_t)b * A.q_ts + (int64_t)(first + g) * A.q_hs + word * 8, x[w]);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[w][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e2 = top > 0.f && top <= 3.4028235e38f ? ilogbf(top) : 0;
      // a scale below 0 goes to the queries; one of 0 (or scores that vanish in fp32) makes them 0
      float f = ldexpf(fabsf(A.scale) * LOG2E, e2 - 11);
      const float sign = f == 0.f ? 0.f : (A.scale < 0.f ? -1.f : 1.f);
      f = f == 0.f ? 1.f : f;
      // 2^(11 - e2) in two factors: neither leaves fp32's range (e2 is at least -133)
      const int up = 11 - e2;
      const float up1 = __uint_as_float((uint32_t)(up / 2 + 127) << 23) * sign;
      const float up2 = __uint_as_float((uint32_t)(up - up / 2 + 127) << 23);
      rf[0] = __shfl_sync(0xffffffffu, f, 8 * j);
      rf[1] = __shfl_sync(0xffffffffu, f, 8 * j + 4);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[w][e] = x[w][e] * up1 * up2;
        // a word's codes come in the pairs (i, i + 4)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          qb[2 * w + k][0] = pack2(x[w][2 * k], x[w][2 * k + 4], __half());
          qb[2 * w + k][1] = pack2(x[w][2 * k + 1], x[w][2 * k + 5], __half());
        }
      }
    }
    int t0 = 0;
    while (used < mine) {
      const int s = used % STAGES;
      const int4 d = S.desc[warp][s];
      if (d.z < 0) break;                 // the head set's end
      t0 = d.z;
      const int ok = d.w, have = len - t0;
      const bool edge = have < TT || ok != 3;
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      auto& stage = S.ring[warp][s];
      const uint32_t kc = smem_addr(stage.codes[0]), vc = smem_addr(stage.codes[1]);
      const __half2* kp = stage.params[0];
      __half2* vp = stage.params[1];
      // token i of the tile counts
      auto seen = [&](int i) { return i < have && ((ok >> (i >> 4)) & 1); };

      if (edge) {                         // values that do not count: 0, whatever the page holds there
        if (!seen(lane)) {
#pragma unroll
          for (int i = 0; i < NG; ++i) vp[lane * NG + i] = __float2half2_rn(0.f);
        }
        __syncwarp();
      }
      // ---- scores: tokens 16 h + g (+ 8) against heads 2 j, 2 j + 1 ----
      float sc[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[2][NW];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = h * 16 + r * 8 + g;
          if constexpr (NG == 1 && D == 128) {
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[r][0]), "=r"(w[r][1]), "=r"(w[r][2]), "=r"(w[r][3]) : "r"(kc + piece<D>(row, j)));
          } else if constexpr (NG == 1) {
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                         : "=r"(w[r][0]), "=r"(w[r][1]) : "r"(kc + piece<D>(row, j >> 1) + (j & 1) * 8));
          } else {
#pragma unroll
            for (int i = 0; i < NW; ++i) w[r][i] = lds32(kc + piece<D>(row, i) + j * 4);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[h][e] = 0.f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const __half2 p0 = kp[(h * 16 + g) * NG + i], p1 = kp[(h * 16 + 8 + g) * NG + i];
          const Zero z0 = make_zero(__high2half2(p0)), z1 = make_zero(__high2half2(p1));
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = i * NW / NG; k < (i + 1) * NW / NG; ++k) {
            mma16816(c, code_lo(w[0][k], masks, z0), code_lo(w[1][k], masks, z1), code_hi(w[0][k], masks, z0), code_hi(w[1][k], masks, z1),
                     qb[2 * k][0], qb[2 * k][1]);
            const uint32_t x = w[0][k] >> 8, y = w[1][k] >> 8;
            mma16816(c, code_lo(x, masks, z0), code_lo(y, masks, z1), code_hi(x, masks, z0), code_hi(y, masks, z1), qb[2 * k + 1][0],
                     qb[2 * k + 1][1]);
          }
          const float s0 = __low2float(p0), s1 = __low2float(p1);
          sc[h][0] = fmaf(s0, c[0], sc[h][0]);
          sc[h][1] = fmaf(s0, c[1], sc[h][1]);
          sc[h][2] = fmaf(s1, c[2], sc[h][2]);
          sc[h][3] = fmaf(s1, c[3], sc[h][3]);
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!seen(h * 16 + (e >> 1) * 8 + g)) sc[h][e] = -INFINITY;
        }
      }

      // ---- the running maximum, weights and their sum ----
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        mx[r] = fmaxf(fmaxf(sc[0][r], sc[0][2 + r]), fmaxf(sc[1][r], sc[1][2 + r])) * rf[r];
      if (__any_sync(0xffffffffu, mx[0] - m[0] > KEEP || mx[1] - m[1] > KEEP)) {
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], o));
          mx[r] = fmaxf(mx[r], m[r]);
          f[r] = mx[r] == -INFINITY ? 1.f : ex2(m[r] - mx[r]);
          m[r] = mx[r];
          l[r] *= f[r];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] *= f[e & 1];
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = r; e < 4; e += 2) {
            sc[h][e] = ex2(fmaf(sc[h][e], rf[r], -ref));
            l[r] += sc[h][e];
          }
      }

      // ---- values ----
      uint32_t pb[NG][2][2];              // the weights of group i, tokens of half h, as B operand
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float sv[2][2];
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t = h * 16 + r * 8 + g;
            sv[h][r] = __low2float(vp[t * NG + i]);
            top = fmaxf(top, fabsf(sv[h][r]));
          }
        int e2 = min((int)(__float_as_uint(top) >> 23) - 127, 15);     // top < 2^(e2 + 1)
        if (__any_sync(0xffffffffu, e2 > ve[i])) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) e2 = max(e2, __shfl_xor_sync(0xffffffffu, e2, o));
          const float f = ex2((float)(ve[i] - e2));
          ve[i] = e2;
#pragma unroll
          for (int a = i * MT / NG; a < (i + 1) * MT / NG; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[a][e] *= f;
        }
        const float mul = __uint_as_float((uint32_t)(10 - ve[i] + 127) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float k = sv[h][r] * mul;
            pb[i][h][r] = transpose8x8(pack2(sc[h][2 * r] * k, sc[h][2 * r + 1] * k, __half()));
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ta = h * 16 + 2 * j;    // this lane's tokens: ta, ta + 1, ta + 8, ta + 9
        auto zeros = [&](int i, int t) {
          return make_zero(__highs2half2(vp[t * NG + i], vp[(t + 1) * NG + i]));
        };
        auto word = [&](int t, int w) { return lds32(vc + piece<D>(t, w >> 2) + (w & 3) * 4); };
        if constexpr (GROUP >= 64) {
          // rows g and g + 8 of feature tile (f, i): nibbles i and i + 4 of word 8 f + g
          Zero z0[NG], z1[NG];
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            z0[i] = zeros(i, ta);
            z1[i] = zeros(i, ta + 8);
          }
#pragma unroll
          for (int f = 0; f < D / 64; ++f) {
            const int w = 8 * f + g, grp = f * 64 / GROUP;
            const Zero za = z0[grp], zb = z1[grp];
            const uint32_t wa = word(ta, w), wb = word(ta + 1, w), wc = word(ta + 8, w), wd = word(ta + 9, w);
            uint32_t x0 = __byte_perm(wa, wb, 0x5410), x1 = __byte_perm(wa, wb, 0x7632);
            uint32_t y0 = __byte_perm(wc, wd, 0x5410), y1 = __byte_perm(wc, wd, 0x7632);
            const uint32_t p0 = pb[grp][h][0], p1 = pb[grp][h][1];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              mma16816(acc[4 * f + i], code_lo(x0, masks, za), code_lo(x1, masks, za), code_lo(y0, masks, zb), code_lo(y1, masks, zb), p0, p1);
              mma16816(acc[4 * f + i + 1], code_hi(x0, masks, za), code_hi(x1, masks, za), code_hi(y0, masks, zb), code_hi(y1, masks, zb), p0, p1);
              x0 >>= 8; x1 >>= 8; y0 >>= 8; y1 >>= 8;
            }
          }
        } else {
          // a tile's rows stay in one group of 32: nibbles 2 i + g / 4 (and 4 on) of word g mod 4 of it
          const int sh = (g >> 2) * 4;
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const int w = 4 * q + (g & 3);
            const Zero za = zeros(q, ta), zb = zeros(q, ta + 8);
            const uint32_t wa = word(ta, w), wb = word(ta + 1, w), wc = word(ta + 8, w), wd = word(ta + 9, w);
            uint32_t x0 = __byte_perm(wa, wb, 0x5410) >> sh, x1 = __byte_perm(wa, wb, 0x7632) >> sh;
            uint32_t y0 = __byte_perm(wc, wd, 0x5410) >> sh, y1 = __byte_perm(wc, wd, 0x7632) >> sh;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma16816(acc[2 * q + i], code_lo(x0, masks, za), code_lo(x1, masks, za), code_lo(y0, masks, zb), code_lo(y1, masks, zb),
                       pb[q][h][0], pb[q][h][1]);
              x0 >>= 8; x1 >>= 8; y0 >>= 8; y1 >>= 8;
            }
          }
        }
      }
      __syncwarp();                       // every lane has read the stage
      ++used;
      produce();
      __syncwarp();                       // the next tiles' descriptors are there
    }

    // ---- its end ----
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (l[r] != l[r]) m[r] = 0.f;       // a NaN score: a part without a maximum would not count
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      const int i = a * NG / MT;
      const float mul = ve[i] < -116 ? 0.f : __uint_as_float((uint32_t)(ve[i] - 10 + 127) << 23);   // unset: acc is 0
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[a][e] *= mul;
    }
    ++sets;
    const bool early = begins.z > 0;
    if (used == mine && len - t0 > TT) {
      late = early && sets == 1 ? 2 : 1;
      break;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 2 * j + r;
      const float inv = m[r] == -INFINITY ? 0.f : 1.f / l[r];
      const int64_t at = (int64_t)(2 * run) * A.rows + row;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        float x[8];
        const int dim = eight<D, GROUP>(acc, r, u, x);
        if (row < rows) {
          if (early) {
            store8(A.part_o + at * D + dim, x);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            store_o(A, (int64_t)b * A.o_ts + (int64_t)(first + row) * A.o_hs + dim, x);
          }
        }
      }
      if (early && row < rows && g == 0) {
        A.part_ml[at * 2] = m[r];
        A.part_ml[at * 2 + 1] = l[r];
      }
    }
  }

  // ---- what goes on behind the warps' runs, joined where it is one head set ----
  if (lane == 0) S.late[warp] = late;
  __syncthreads();                        // every warp is done with its ring
  if (late) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 2 * j + r;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        float x[8];
        const int dim = eight<D, GROUP>(acc, r, u, x);
        if (row < A.rows) store8(S.part(warp) + row * D + dim, x);
      }
      if (g == 0) {
        S.ml[warp][row][0] = m[r];
        S.ml[warp][row][1] = l[r];
      }
    }
  }
  __syncthreads();
  for (int w0 = 0, w1; w0 < WARPS; w0 = w1) {
    w1 = w0 + 1;
    if (!S.late[w0]) continue;
    while (w1 < WARPS && S.late[w1] == 2) ++w1;
    for (int u = (int)threadIdx.x; u < A.rows * (D / 8); u += WARPS * 32) {
      const int row = u / (D / 8), c8 = u % (D / 8);
      float top = -INFINITY, sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int w = w0; w < w1; ++w) top = fmaxf(top, S.ml[w][row][0]);
      for (int w = w0; w < w1; ++w) {
        if (S.ml[w][row][0] == -INFINITY) continue;
        const float f = ex2(S.ml[w][row][0] - top);
        sum = fmaf(S.ml[w][row][1], f, sum);
        const float* o = S.part(w) + row * D + c8 * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(o[e], f, x[e]);
      }
      const int64_t at = (int64_t)(2 * (run - warp + w0) + 1) * A.rows + row;
      store8(A.part_o + at * D + c8 * 8, x);
      if (c8 == 0) {
        A.part_ml[at * 2] = top;
        A.part_ml[at * 2 + 1] = sum;
      }
    }
  }
}

// Joins the parts of one query row whose tiles fell to several blocks; writes the rows of
// sequences without tokens.  One block per row: every part's maximum and sum at once, then a
// warp w the values of parts w, w + 8, ..., several in flight.
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ KvaArgs A, int32_t* st) {
  constexpr int V = D / 32;               // values per lane
  constexpr int MOST = RUNS / WARPS + 2;  // parts of a row
  __shared__ float o[8][D];
  __shared__ float weight[MOST];
  __shared__ float ml[8][2];
  __shared__ long long sums[8][2];
  __shared__ int skip;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hx = (int)blockIdx.x / A.rows, row = (int)blockIdx.x % A.rows, b = (int)blockIdx.y;
  const int heads = A.C.heads * A.sets;
  // what the attention launch records is this call's own and stops no row: the answer is the same
  // before and after it
  if (threadIdx.x == 255) skip = stopped(st, A.launch);
  long long before = 0, all = 0;
  for (int i = (int)threadIdx.x; i < A.count; i += 256) {
    const int64_t n = slots_of(tiles_of(A, i), heads);
    all += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, k);
    before += __shfl_xor_sync(0xffffffffu, before, k);
  }
  if (lane == 0) { sums[warp][0] = all; sums[warp][1] = before; }
  __syncthreads();
  all = before = 0;
  for (int w = 0; w < 8; ++w) { all += sums[w][0]; before += sums[w][1]; }
  // every block waits for the attention launch: this launch's end stands for both
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int in_set = min(ROWS, A.per - (hx % A.sets) * ROWS);
  if (skip || row >= in_set) return;
  const int q = hx / A.sets * A.per + (hx % A.sets) * ROWS + row;
  const int n = tiles_of(A, b), len = A.lengths[b];
  if (n == 0 && len != 0) {
    if (threadIdx.x == 0) set_own_error(st, A.launch, GPTQ_ERR_INVALID_ARG, b, STAGE_KV4_ATTENTION);
    return;
  }
  const int64_t at = (int64_t)b * A.o_ts + (int64_t)q * A.o_hs;
  if (n == 0) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (threadIdx.x < D / 8) store_o(A, at + threadIdx.x * 8, zero);
    return;
  }
  const int runs = runs_of(all);
  const int64_t t0 = before + (int64_t)hx * (n + 1), t1 = t0 + n - 1;
  const int c0 = run_of(all, runs, t0), c1 = run_of(all, runs, t1);
  if (c0 == c1) return;                   // finished by its warp
  // the parts: run c0's, those of the blocks after it (their first run's), and the last run's
  const int parts = 2 + (c1 - 1) / WARPS - c0 / WARPS;
  auto slot_of = [&](int i) {
    return (int64_t)(i == parts - 1 ? 2 * c1 : 2 * (i == 0 ? c0 : (c0 / WARPS + i) * WARPS) + 1) * A.rows + row;
  };
  float top = -INFINITY;
  for (int i = (int)threadIdx.x; i < parts; i += 256) {
    weight[i] = A.part_ml[slot_of(i) * 2];
    top = fmaxf(top, weight[i]);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  if (lane == 0) ml[warp][0] = top;
  __syncthreads();
  for (int w = 0; w < 8; ++w) top = fmaxf(top, ml[w][0]);
  float sum = 0.f;
  for (int i = (int)threadIdx.x; i < parts; i += 256) {
    const float f = weight[i] == -INFINITY ? 0.f : ex2(weight[i] - top);
    weight[i] = f;
    sum = fmaf(A.part_ml[slot_of(i) * 2 + 1], f, sum);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if (lane == 0) ml[warp][1] = sum;
  __syncthreads();
  float x[V];
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < parts; i += 8) {
    const float* part = A.part_o + slot_of(i) * D + lane * V;
    const float f = weight[i];
    float y[V];
    if constexpr (V == 4) {
      const float4 v4 = *reinterpret_cast<const float4*>(part);
      y[0] = v4.x; y[1] = v4.y; y[2] = v4.z; y[3] = v4.w;
    } else {
      const float2 v2 = *reinterpret_cast<const float2*>(part);
      y[0] = v2.x; y[1] = v2.y;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = fmaf(y[e], f, x[e]);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) o[warp][lane * V + e] = x[e];
  __syncthreads();
  if ((int)threadIdx.x >= D / 8) return;
  float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  sum = 0.f;
  for (int w = 0; w < 8; ++w) {
    sum += ml[w][1];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += o[w][threadIdx.x * 8 + e];
  }
  const float inv = top == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= inv;
  store_o(A, at + threadIdx.x * 8, y);
}

int head_sets(int per) { return (per + ROWS - 1) / ROWS; }
int set_rows(int per) { return per < ROWS ? per : ROWS; }

template <int D, int GROUP>
int launch(const KvaArgs& A, int32_t* st, cudaStream_t s) {
  const size_t smem = sizeof(KvaSmem<D, GROUP>);
  auto* kernel = kv4_attention_kernel<D, GROUP>;
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  kernel<<<BLOCKS, WARPS * 32, smem, s>>>(A, st);
  GPTQ_LAUNCH_CHECK();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(A.C.heads * A.sets * A.rows), (unsigned)A.count);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  GPTQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv4_join_kernel<D>, A, st));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

size_t kv4_attention_ws_bytes(int, int heads_q, int heads_kv, int head_dim, int64_t) {
  return (size_t)2 * RUNS * set_rows(heads_q / heads_kv) * (head_dim + 2) * sizeof(float);
}

int launch_kv4_attention(const KV4Cache& C, const void* q, int64_t q_ts, int64_t q_hs, int dtype, int count,
                         int heads_q, const int32_t* table, int width, const int32_t* lengths, float scale, void* o,
                         int64_t o_ts, int64_t o_hs, void* ws, int32_t* st, cudaStream_t s) {
  const int per = heads_q / C.heads, rows = set_rows(per);
  KvaArgs A{C, q, o, q_ts, q_hs, o_ts, o_hs, table, lengths, static_cast<float*>(ws),
            static_cast<float*>(ws) + (size_t)2 * RUNS * rows * C.head_dim, width, count, per, head_sets(per), rows,
            scale, dtype == GPTQ_F16, next_launch()};
  TraceScope ts("kv4_attention", "", 0.0, s);
  if (C.head_dim == 64) return C.group == 32 ? launch<64, 32>(A, st, s) : launch<64, 64>(A, st, s);
  if (C.group == 32) return launch<128, 32>(A, st, s);
  return C.group == 64 ? launch<128, 64>(A, st, s) : launch<128, 128>(A, st, s);
}

}  // namespace gptq
