// Attention of one query token per sequence over its keys and values in the 4-bit cache
// (gptq_kv4_attention): o = sum_t softmax_t(scale q . k_t) v_t over the sequence's tokens,
// k_t and v_t = s (c - z) read from the cache's pages, hq / hk query heads per k/v head.
// A sequence without tokens gives 0.
//
// Bound: HBM, the codes and their scales read once (and close behind it the issue slots
// that unpack them).  The query heads of a k/v head are the rows of m16n8k16 products
// (mma.sync, fp16 in, fp32 sums), up to 16 at a time.  Two codes are masked into the
// mantissas of the fp16 pair 1024 + c (or 1024 + 16 c, from the next nibble) and one
// packed subtraction (or fma) leaves c - z, an exact fp16 integer; scales stay outside:
//   scores   q . k_t = sum over groups of s sum q (c - z), q held in fp16 under a power of
//            two per row (its largest value in [2^11, 2^12): both 16-bit types fit, values
//            below 2^-25 of the largest rounded);
//   values   sum_t p_t s_t (c_t - z_t) with p_t s_t rounded to fp16 under a power of two
//            per group (largest value below 2^15).
// (Without the subtraction, c as an fp16 subnormal and z taken off the sums, the sums
// cancel: the tensor cores align such products by their unnormalised exponents, and
// results near 0 were off by 2^-17 of a scale.)
// The running maximum is kept while it grows by less than 2^4 in the weights.
//
// Work: the sequences' tiles of 32 tokens, all heads, in one line, cut into equal runs, one
// per block of four warps (three blocks per SM); a block's warps take its tiles in turn,
// each with a ring of its own that TMA fills (codes swizzled, scales as they lie).  A head
// whose tiles fall to one block is finished there; otherwise the blocks leave their
// (maximum, sum, weighted values) in the workspace and kv4_join_kernel, a dependent launch,
// joins them in a fixed order.  Every wait is bounded (GPTQ_ERR_TIMEOUT).
#include <math.h>

#include <climits>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "tc_common.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

constexpr int BLOCKS = 148 * 3;           // resident blocks: the cut of the work, whatever the device
constexpr int WARPS = 4;
constexpr int TT = 32;                    // tokens of a tile
constexpr int STAGES = 3;
constexpr int ROWS = 16;                  // query heads of a product
constexpr float LOG2E = 1.4426950408889634f;
constexpr float KEEP = 4.f;

struct KvaArgs {
  KV4Cache C;
  const void* q;
  void* o;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const int32_t* table;
  const int32_t* lengths;
  float* part_o;                          // [2 BLOCKS][rows][head_dim]
  float* part_ml;                         // [2 BLOCKS][rows][2]
  int width, count, per, sets, rows;      // per: query heads of a k/v head, in sets of up to 16 (rows)
  float scale;
  int half;                               // q and o are fp16 (else bf16)
};

// Sequence b's tiles (one head set); 0 for a length that the table does not hold.
__device__ __forceinline__ int tiles_of(const KvaArgs& A, int b) {
  const int len = A.lengths[b];
  return len < 0 || len > (int64_t)A.width * A.C.page_size ? 0 : (len + TT - 1) / TT;
}

struct Place {
  int b, hx, t, tiles;                    // sequence, head set, tile of it, tiles of the sequence
  uint32_t ord;                           // head sets with tiles before this one
};

// Walks the line of tiles with a window of 32 sequences, one per lane.
struct Finder {
  int b0 = -32;
  int64_t base = 0, total = 0;            // tiles before and in the window
  int64_t incl = 0;                       // this lane's sequence and those before it in the window
  int tiles = 0, full_before = 0, ones = 0;   // sequences with tiles before the window; up to this lane

  __device__ __forceinline__ void advance(const KvaArgs& A, int heads) {
    const int lane = threadIdx.x & 31;
    if (b0 >= 0) full_before += __shfl_sync(0xffffffffu, ones, 31);
    base += total;
    b0 += 32;
    const int b = b0 + lane;
    tiles = b < A.count ? tiles_of(A, b) : 0;
    incl = (int64_t)tiles * heads;
    ones = tiles > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      const int n = __shfl_up_sync(0xffffffffu, ones, o);
      if (lane >= o) { incl += up; ones += n; }
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  // Each lane's tile (not before the window; lanes without one pass want = -1).
  __device__ __forceinline__ Place find(const KvaArgs& A, int heads, int64_t want) {
    Place p{0, 0, 0, 0, 0};
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
      const int k = __shfl_sync(0xffffffffu, ones, lo);
      if (here) {
        const int64_t r = rel - (end - (int64_t)n * heads);
        p.b = b0 + lo;
        p.hx = (int)(r / n);
        p.t = (int)(r % n);
        p.tiles = n;
        p.ord = (uint32_t)(full_before + k - 1) * (uint32_t)heads + (uint32_t)p.hx;
        open = false;
      }
      if (!__any_sync(0xffffffffu, open) || b0 + 32 >= A.count) return p;
      advance(A, heads);
    }
  }
};

// Block c's run of the line.
__device__ __forceinline__ int64_t run_begin(int64_t all, int blocks, int c) { return all * c / blocks; }
__device__ __forceinline__ int run_of(int64_t all, int blocks, int64_t tile) {
  int c = (int)(tile * blocks / all);
  while (c + 1 < blocks && run_begin(all, blocks, c + 1) <= tile) ++c;
  return c;
}
__device__ __forceinline__ int runs_of(int64_t all) {
  const int64_t n = (all + WARPS - 1) / WARPS;
  return (int)(n < BLOCKS ? n : BLOCKS);
}

template <int D, int GROUP>
struct KvaSmem {
  static constexpr int kCodes = TT * D / 2;
  static constexpr int kParams = TT * (D / GROUP) * 4;
  struct Stage {
    alignas(512) uint8_t codes[2][kCodes];
    uint8_t params[2][kParams];
  };
  Stage ring[WARPS][STAGES];
  float out[ROWS][D];
  float ml[2][WARPS][ROWS][2];
  int4 desc[WARPS][STAGES];
  int2 seg[2];
  uint64_t full[WARPS][STAGES];
  int abort, skip;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes -> c - z: the nibbles at bits 0 and 16, or at bits 4 and 20, of x; zero.lo holds
// -(1024 + z) per half, zero.hi -(64 + z).
struct Zero {
  __half2 lo, hi;
};
__device__ __forceinline__ Zero make_zero(__half2 z) {
  return Zero{__hneg2(__hadd2(z, __floats2half2_rn(1024.f, 1024.f))), __hneg2(__hadd2(z, __floats2half2_rn(64.f, 64.f)))};
}
__device__ __forceinline__ uint32_t code_lo(uint32_t x, const Zero& z) {
  const uint32_t v = (x & 0x000F000Fu) | 0x64006400u;
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&v), z.lo);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t code_hi(uint32_t x, const Zero& z) {
  const uint32_t v = (x & 0x00F000F0u) | 0x64006400u;
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(0.0625f, 0.0625f), z.hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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

template <int D, int GROUP>
__global__ void __launch_bounds__(WARPS * 32, 3)
kv4_attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ KvaArgs A, int32_t* st) {
  using Smem = KvaSmem<D, GROUP>;
  constexpr int NG = D / GROUP;           // groups of a row
  constexpr int NW = D / 32;              // words of a key row per lane
  constexpr int NT = TT / 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    S.skip = has_error(st);
    S.abort = 0;
    for (int w = 0; w < WARPS; ++w)
      for (int s = 0; s < STAGES; ++s) tc::mbar_init(&S.full[w][s], 1);
    tc::fence_barrier_init();
  }
  const int heads = A.C.heads * A.sets;
  int64_t all = 0;
  {
    int64_t mine = 0;
    for (int b = lane; b < A.count; b += 32) mine += tiles_of(A, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    all = mine * heads;
  }
  __syncthreads();
  const int runs = runs_of(all);
  if (S.skip || (int)blockIdx.x >= runs) return;
  const int64_t begin = run_begin(all, runs, (int)blockIdx.x), end = run_begin(all, runs, (int)blockIdx.x + 1);
  Finder finder;
  const Place ends = finder.find(A, heads, lane == 0 ? begin : (lane == 1 ? end - 1 : -1));
  const uint32_t ord0 = __shfl_sync(0xffffffffu, ends.ord, 0);
  const int ord1 = (int)(__shfl_sync(0xffffffffu, ends.ord, 1) - ord0);   // the last head set, from the first
  const bool from_before = __shfl_sync(0xffffffffu, ends.t, 0) > 0;
  const bool goes_on = __shfl_sync(0xffffffffu, ends.t + 1 < ends.tiles, 1) != 0;
  finder = Finder();

  volatile int* abort_flag = &S.abort;
  // this warp's tiles: begin + warp + 4 i
  const int mine = (int)((end - begin - warp + WARPS - 1) / WARPS);
  const int box = min(A.C.page_size, TT), parts = TT / box;      // page rows of one copy; copies of a tile
  const int page_shift = 31 - __clz(A.C.page_size);
  int made = 0;
  // the batch of 32 tiles that lane i describes tile (made & ~31) + i of
  int row0 = 0, row1 = 0;
  int4 d0 = make_int4(0, 0, 0, 0);
  auto produce = [&]() {
    if (made >= mine) return;
    if ((made & 31) == 0) {
      const int i = made + lane;
      const int64_t want = i < mine ? begin + warp + (int64_t)WARPS * i : -1;
      const Place p = finder.find(A, heads, want);
      if (want >= 0) {
        const int head = p.hx / A.sets, t0 = p.t * TT;
        int ok = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // a tile's second page may lie behind the sequence's end: its table entry is not read
          const int pos = t0 + k * box;
          int page = 0;
          if (k < parts && pos < A.lengths[p.b]) {
            page = kv4_page(A.C, A.table, A.width, p.b, pos);
            if (page < 0) {
              set_error(st, GPTQ_ERR_INVALID_ARG, p.b, STAGE_KV4_ATTENTION);
              page = 0;
            } else {
              ok |= parts == 1 ? 3 : 1 << k;
            }
          }
          const int row = (int)kv4_row(A.C, page, head, pos & (A.C.page_size - 1));
          if (k == 0) row0 = row;
          else row1 = row;
        }
        d0 = make_int4(p.b, p.hx | (ok << 28), t0, (int)(p.ord - ord0));
      }
    }
    const int src = made & 31, s = made % STAGES;
    const int r0 = __shfl_sync(0xffffffffu, row0, src), r1 = __shfl_sync(0xffffffffu, row1, src);
    const int4 d = make_int4(__shfl_sync(0xffffffffu, d0.x, src), __shfl_sync(0xffffffffu, d0.y, src),
                             __shfl_sync(0xffffffffu, d0.z, src), __shfl_sync(0xffffffffu, d0.w, src));
    if (lane == 0) {
      S.desc[warp][s] = d;
      auto& stage = S.ring[warp][s];
      uint64_t* bar = &S.full[warp][s];
      tc::mbar_arrive_expect_tx(bar, 2 * (Smem::kCodes + Smem::kParams));
      const uint32_t pb = (uint32_t)(box * NG * 4);
      for (int k = 0; k < parts; ++k) {
        const int r = k == 0 ? r0 : r1;
        tc::tma_load_2d(stage.codes[0] + k * box * (D / 2), &tk, bar, 0, r);
        tc::tma_load_2d(stage.codes[1] + k * box * (D / 2), &tv, bar, 0, r);
#pragma unroll
        for (int n = 0; n < 2; ++n)
          bulk_load(tc::smem_u32(stage.params[n]) + k * pb, A.C.params[n] + (int64_t)r * NG * 2, pb,
                    tc::smem_u32(bar));
      }
    }
    __syncwarp();
    ++made;
  };
  for (int i = 0; i < STAGES; ++i) produce();

  // the state of the head set at hand: rows g and g + 8
  float acc[D / 8][4], m[2], l[2];
  int ve[NG];                             // weights of group i carry 2^(10 - ve[i])
  uint32_t qa[D / 16][4];
  float rf[2];
  int used = 0, cur = -1, at_b = 0, at_hx = 0;

  for (int ord = 0; ord <= ord1; ++ord) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) ve[i] = -127;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;

    while (used < mine) {
      const int s = used % STAGES;
      const int4 d = S.desc[warp][s];
      if (d.w != ord) break;
      const int b = d.x, hx = d.y & 0x0fffffff, ok = (int)((uint32_t)d.y >> 28), t0 = d.z;
      if (cur != ord) {
        // this warp's first tile of the head set: its queries as operands
        cur = ord;
        at_b = b;
        at_hx = hx;
        const int head = hx / A.sets, first = head * A.per + (hx % A.sets) * ROWS;
        const int rows = min(ROWS, A.per - (hx % A.sets) * ROWS);
        float x[2][NW][8];
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const int word = NG == 1 ? NW * j + w : j + 4 * w;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[r][w][e] = 0.f;
            if (g + 8 * r < rows)
              load_q(A, (int64_t)b * A.q_ts + (int64_t)(first + g + 8 * r) * A.q_hs + word * 8, x[r][w]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top[r] = fmaxf(top[r], fabsf(x[r][w][e]));
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          const int e2 = top[r] > 0.f && top[r] <= 3.4028235e38f ? ilogbf(top[r]) : 0;
          rf[r] = ldexpf(A.scale * LOG2E, e2 - 11);
#pragma unroll
          for (int w = 0; w < NW; ++w) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[r][w][e] = ldexpf(x[r][w][e], 11 - e2);
            // a word's codes come in the pairs (i, i + 4)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              qa[2 * w + k][r] = pack2(x[r][w][2 * k], x[r][w][2 * k + 4], __half());
              qa[2 * w + k][2 + r] = pack2(x[r][w][2 * k + 1], x[r][w][2 * k + 5], __half());
            }
          }
        }
      }
      const int have = A.lengths[b] - t0;
      const bool edge = have < TT || ok != 3;
      int fine = 0;
      if (lane == 0) fine = tc::mbar_wait(&S.full[warp][s], (uint32_t)(used / STAGES) & 1u, abort_flag);
      fine = __shfl_sync(0xffffffffu, fine, 0);
      if (fine) {
        auto& stage = S.ring[warp][s];
        const uint32_t kc = tc::smem_u32(stage.codes[0]), vc = tc::smem_u32(stage.codes[1]);
        const __half2* kp = reinterpret_cast<const __half2*>(stage.params[0]);
        const __half2* vp = reinterpret_cast<const __half2*>(stage.params[1]);
        // token i of the tile counts
        auto seen = [&](int i) { return i < have && ((ok >> (i >> 4)) & 1); };

        // ---- scores ----
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = n * 8 + g;
          uint32_t w[NW];
          if constexpr (NG == 1 && D == 128) {
            const uint32_t a = kc + row * 64 + ((j ^ ((row >> 1) & 3)) << 4);
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
          } else if constexpr (NG == 1) {
            const uint32_t a = kc + row * 32 + (((j >> 1) ^ ((row >> 2) & 1)) << 4) + (j & 1) * 8;
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
          } else {
            const uint32_t sw = D == 128 ? (row >> 1) & 3 : (row >> 2) & 1;
#pragma unroll
            for (int i = 0; i < NW; ++i) w[i] = lds32(kc + row * (D / 2) + ((i ^ sw) << 4) + j * 4);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            const Zero z = make_zero(__high2half2(kp[row * NG + i]));
#pragma unroll
            for (int k = i * NW / NG; k < (i + 1) * NW / NG; ++k) {
              const uint32_t hi = w[k] >> 8;
              mma16816(c, qa[2 * k], code_lo(w[k], z), code_hi(w[k], z));
              mma16816(c, qa[2 * k + 1], code_lo(hi, z), code_hi(hi, z));
            }
            const float s0 = __low2float(kp[(n * 8 + 2 * j) * NG + i]);
            const float s1 = __low2float(kp[(n * 8 + 2 * j + 1) * NG + i]);
            sc[n][0] = fmaf(s0, c[0], sc[n][0]);
            sc[n][1] = fmaf(s1, c[1], sc[n][1]);
            sc[n][2] = fmaf(s0, c[2], sc[n][2]);
            sc[n][3] = fmaf(s1, c[3], sc[n][3]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] *= rf[e >> 1];
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!seen(n * 8 + 2 * j + (e & 1))) sc[n][e] = -INFINITY;
          }
        }

        // ---- running maximum, weights and their sum ----
        float mx[2];
        bool up = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = m[r];
#pragma unroll
          for (int n = 0; n < NT; ++n) mx[r] = fmaxf(mx[r], fmaxf(sc[n][2 * r], sc[n][2 * r + 1]));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          up |= mx[r] - m[r] > KEEP;
        }
        if (__any_sync(0xffffffffu, up)) {
          float f[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const bool mine_up = mx[r] - m[r] > KEEP;
            f[r] = mine_up ? ex2(m[r] - mx[r]) : 1.f;
            if (mine_up) m[r] = mx[r];
            l[r] *= f[r];
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] *= f[e >> 1];
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][e] = ex2(sc[n][e] - ref[e >> 1]);
            l[e >> 1] += sc[n][e];
          }

        // ---- values ----
        uint32_t pa[NG][TT / 16][4];
        __half2 zv[NG][NT];               // zero points of tokens 2 j, 2 j + 1
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          float sv[NT][2];
          float top = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            {
              __half2 p0 = vp[(n * 8 + 2 * j) * NG + i], p1 = vp[(n * 8 + 2 * j + 1) * NG + i];
              if (edge) {
                if (!seen(n * 8 + 2 * j)) p0 = __half2half2(__ushort_as_half((unsigned short)0));
                if (!seen(n * 8 + 2 * j + 1)) p1 = __half2half2(__ushort_as_half((unsigned short)0));
              }
              sv[n][0] = __low2float(p0);
              sv[n][1] = __low2float(p1);
              zv[i][n] = __highs2half2(p0, p1);
              top = fmaxf(top, fmaxf(fabsf(sv[n][0]), fabsf(sv[n][1])));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e2 = min((int)(__float_as_uint(top) >> 23) - 127, 15);   // top < 2^(e2 + 1)
          if (e2 > ve[i]) {               // the same in every lane
            const float f = ex2((float)(ve[i] - e2));
            ve[i] = e2;
            constexpr int PER = D / 8 / NG;
#pragma unroll
            for (int a = 0; a < PER; ++a)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i * PER + a][e] *= f;
          }
          const float mul = __uint_as_float((uint32_t)(10 - ve[i] + 127) << 23);
#pragma unroll
          for (int k = 0; k < TT / 16; ++k) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float s0 = sv[2 * k + n][0] * mul, s1 = sv[2 * k + n][1] * mul;
              pa[i][k][2 * n] = pack2(sc[2 * k + n][0] * s0, sc[2 * k + n][1] * s1, __half());
              pa[i][k][2 * n + 1] = pack2(sc[2 * k + n][2] * s0, sc[2 * k + n][3] * s1, __half());
            }
          }
        }
        auto vword = [&](int row, int word) {
          const uint32_t sw = D == 128 ? (row >> 1) & 3 : (row >> 2) & 1;
          return lds32(vc + row * (D / 2) + (((word >> 2) ^ sw) << 4) + (word & 3) * 4);
        };
#pragma unroll
        for (int k = 0; k < TT / 16; ++k) {
          const int ra = k * 16 + 2 * j;
          if constexpr (GROUP >= 64) {
            // column n of a product: word n (+ 8), nibble i of it per product
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf) {
              const int word = g + 8 * hf;
              const uint32_t wa = vword(ra, word), wb = vword(ra + 1, word);
              const uint32_t wc = vword(ra + 8, word), wd = vword(ra + 9, word);
              const uint32_t x[2] = {__byte_perm(wa, wb, 0x5410), __byte_perm(wa, wb, 0x7632)};
              const uint32_t y[2] = {__byte_perm(wc, wd, 0x5410), __byte_perm(wc, wd, 0x7632)};
              const Zero za = make_zero(zv[hf * 64 / GROUP][2 * k]), zb = make_zero(zv[hf * 64 / GROUP][2 * k + 1]);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint32_t x8 = x[u] >> 8, y8 = y[u] >> 8;
                const int a = hf * 8 + u * 4;
                const uint32_t(&p)[4] = pa[hf * 64 / GROUP][k];
                mma16816(acc[a], p, code_lo(x[u], za), code_lo(y[u], zb));
                mma16816(acc[a + 1], p, code_hi(x[u], za), code_hi(y[u], zb));
                mma16816(acc[a + 2], p, code_lo(x8, za), code_lo(y8, zb));
                mma16816(acc[a + 3], p, code_hi(x8, za), code_hi(y8, zb));
              }
            }
          } else {
            // a product's columns stay in one group of 32: word n mod 4 of it, nibble 2 i + n / 4
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              const int word = 4 * i + (g & 3), sh = (g >> 2) * 4;
              const uint32_t wa = vword(ra, word), wb = vword(ra + 1, word);
              const uint32_t wc = vword(ra + 8, word), wd = vword(ra + 9, word);
              const uint32_t x[2] = {__byte_perm(wa, wb, 0x5410) >> sh, __byte_perm(wa, wb, 0x7632) >> sh};
              const uint32_t y[2] = {__byte_perm(wc, wd, 0x5410) >> sh, __byte_perm(wc, wd, 0x7632) >> sh};
              const Zero za = make_zero(zv[i][2 * k]), zb = make_zero(zv[i][2 * k + 1]);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                mma16816(acc[4 * i + 2 * u], pa[i][k], code_lo(x[u], za), code_lo(y[u], zb));
                mma16816(acc[4 * i + 2 * u + 1], pa[i][k], code_lo(x[u] >> 8, za), code_lo(y[u] >> 8, zb));
              }
            }
          }
        }
      }
      __syncwarp();
      ++used;
      produce();
    }

    // ---- the four warps' parts of this head set joined, in order ----
    float (*ml)[ROWS][2] = S.ml[ord & 1];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (j == 0) {
        ml[warp][g + 8 * r][0] = m[r];
        ml[warp][g + 8 * r][1] = l[r];
      }
    }
    if (cur == ord && lane == 0) S.seg[ord & 1] = make_int2(at_b, at_hx);
    __syncthreads();
    const int b = S.seg[ord & 1].x, hx = S.seg[ord & 1].y;
    const int first = hx / A.sets * A.per + (hx % A.sets) * ROWS, rows = min(ROWS, A.per - (hx % A.sets) * ROWS);
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w][g + 8 * r][0]);
      f[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
    }
    for (int w = 0; w < WARPS; ++w) {
      if (warp == w) {
#pragma unroll
        for (int a = 0; a < D / 8; ++a) {
          const int i = a * NG / (D / 8);
          const float mul = ve[i] < -116 ? 0.f : __uint_as_float((uint32_t)(ve[i] - 10 + 127) << 23);   // unset: acc is 0
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = 2 * j + (e & 1), row = g + 8 * (e >> 1);
            const int dim = GROUP >= 64 ? 8 * (col + 8 * (a / 8)) + a % 8
                                        : 8 * (4 * (a / 4) + (col & 3)) + 2 * (a % 4) + (col >> 2);
            const float v = acc[a][e] * mul * f[e >> 1];
            S.out[row][dim] = w == 0 ? v : S.out[row][dim] + v;
          }
        }
      }
      __syncthreads();
    }
    const bool early = ord == 0 && from_before, late = ord == ord1 && goes_on;
    const int slot = 2 * (int)blockIdx.x + (early ? 0 : 1);
    for (int u = (int)threadIdx.x; u < rows * (D / 8); u += WARPS * 32) {
      const int row = u / (D / 8), c8 = u % (D / 8);
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w][row][0]);
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        if (ml[w][row][0] != -INFINITY) sum += ml[w][row][1] * ex2(ml[w][row][0] - top);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = S.out[row][c8 * 8 + e];
      if (!early && !late) {
        const float inv = top == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        store_o(A, (int64_t)b * A.o_ts + (int64_t)(first + row) * A.o_hs + c8 * 8, x);
      } else {
        const int64_t at = (int64_t)slot * A.rows + row;
        store8(A.part_o + at * D + c8 * 8, x);
        if (c8 == 0) {
          A.part_ml[at * 2] = top;
          A.part_ml[at * 2 + 1] = sum;
        }
      }
    }
  }
  if (*abort_flag) {
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) {
        const int n = (made - s + STAGES - 1) / STAGES;
        const uint64_t t0 = tc::globaltimer();
        while (n > 0 && !tc::mbar_try_wait(&S.full[warp][s], (uint32_t)(n - 1) & 1u))
          if (tc::globaltimer() - t0 > 1000000000ull) break;
      }
    }
    if (threadIdx.x == 0) set_error(st, GPTQ_ERR_TIMEOUT, (int)blockIdx.x, STAGE_KV4_ATTENTION);
  }
}

// Joins the parts of one query row whose tiles fell to several blocks; writes the rows of
// sequences without tokens.  One block per row: warp w takes the parts w, w + 8, ...
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ KvaArgs A, int32_t* st) {
  constexpr int V = D / 32;               // values per lane
  __shared__ float o[8][D];
  __shared__ float ml[8][2];
  __shared__ long long sums[8][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hx = (int)blockIdx.x / A.rows, row = (int)blockIdx.x % A.rows, b = (int)blockIdx.y;
  const int heads = A.C.heads * A.sets;
  long long before = 0, all = 0;
  for (int i = (int)threadIdx.x; i < A.count; i += 256) {
    const int n = tiles_of(A, i);
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
  if (row >= in_set) return;
  const int q = hx / A.sets * A.per + (hx % A.sets) * ROWS + row;
  const int n = tiles_of(A, b), len = A.lengths[b];
  if (n == 0 && len != 0) {
    if (threadIdx.x == 0) set_error(st, GPTQ_ERR_INVALID_ARG, b, STAGE_KV4_ATTENTION);
    return;
  }
  if (has_error(st)) return;
  const int64_t at = (int64_t)b * A.o_ts + (int64_t)q * A.o_hs;
  if (n == 0) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (threadIdx.x < D / 8) store_o(A, at + threadIdx.x * 8, zero);
    return;
  }
  all *= heads;
  const int runs = runs_of(all);
  const int64_t t0 = before * heads + (int64_t)hx * n, t1 = t0 + n - 1;
  const int c0 = run_of(all, runs, t0), c1 = run_of(all, runs, t1);
  if (c0 == c1) return;                   // finished by its block
  float m = -INFINITY, l = 0.f, x[V];
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += 8) {
    const int64_t p = (int64_t)(2 * c + (c == c0 ? 1 : 0)) * A.rows + row;
    const float pm = A.part_ml[p * 2], pl = A.part_ml[p * 2 + 1];
    const float mn = fmaxf(m, pm), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref), w = ex2(pm - ref);
    m = mn;
    l = l * f + pl * w;
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = x[e] * f + A.part_o[p * D + e * 32 + lane] * w;
  }
  if (lane == 0) { ml[warp][0] = m; ml[warp][1] = l; }
#pragma unroll
  for (int e = 0; e < V; ++e) o[warp][e * 32 + lane] = x[e];
  __syncthreads();
  if ((int)threadIdx.x >= D / 8) return;
  float top = -INFINITY, sum = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < 8; ++w) top = fmaxf(top, ml[w][0]);
  for (int w = 0; w < 8; ++w) {
    if (ml[w][0] == -INFINITY) continue;
    const float f = ex2(ml[w][0] - top);
    sum += ml[w][1] * f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += o[w][threadIdx.x * 8 + e] * f;
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
  // a cache row per line, in boxes of as many rows as a page or a tile holds
  const uint64_t rows = (uint64_t)A.C.pages * A.C.heads * A.C.page_size;
  const uint32_t box = (uint32_t)(A.C.page_size < TT ? A.C.page_size : TT);
  const CUtensorMapSwizzle swz = D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  CUtensorMap map[2];
  for (int i = 0; i < 2; ++i) {
    const int rc = make_tmap_2d(&map[i], CU_TENSOR_MAP_DATA_TYPE_INT32, A.C.codes[i], D / 8, rows, D / 2, D / 8, box, swz);
    if (rc != GPTQ_OK) return rc;
  }
  const size_t smem = sizeof(KvaSmem<D, GROUP>) + 1024;
  auto* kernel = kv4_attention_kernel<D, GROUP>;
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  kernel<<<BLOCKS, WARPS * 32, smem, s>>>(map[0], map[1], A, st);
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
  return (size_t)2 * BLOCKS * set_rows(heads_q / heads_kv) * (head_dim + 2) * sizeof(float);
}

int launch_kv4_attention(const KV4Cache& C, const void* q, int64_t q_ts, int64_t q_hs, int dtype, int count,
                         int heads_q, const int32_t* table, int width, const int32_t* lengths, float scale, void* o,
                         int64_t o_ts, int64_t o_hs, void* ws, int32_t* st, cudaStream_t s) {
  const int per = heads_q / C.heads, rows = set_rows(per);
  KvaArgs A{C, q, o, q_ts, q_hs, o_ts, o_hs, table, lengths, static_cast<float*>(ws),
            static_cast<float*>(ws) + (size_t)2 * BLOCKS * rows * C.head_dim, width, count, per, head_sets(per), rows,
            scale, dtype == GPTQ_F16};
  TraceScope ts("kv4_attention", "", 0.0, s);
  if (C.head_dim == 64) return C.group == 32 ? launch<64, 32>(A, st, s) : launch<64, 64>(A, st, s);
  if (C.group == 32) return launch<128, 32>(A, st, s);
  return C.group == 64 ? launch<128, 64>(A, st, s) : launch<128, 128>(A, st, s);
}

}  // namespace gptq
