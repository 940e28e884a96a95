// Attention over the prompts of a packed batch (gptq_attention): per sequence and query
// head, o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j that query i sees (all,
// or with causal those up to i + Lk - Lq), hq / hk query heads per k/v head.  A query that
// sees no key gives 0; a key that a query does not see takes no part in it, whatever its
// row holds.
//
// One pass over the keys with a running maximum m and sum l per query (scores s):
//   m' = max(m, max_j s_j),  p_j = 2^(c (s_j - m')),  l' = l f + sum_j p_j,
//   o' = o f + sum_j p_j v_j,  f = 2^(c (m - m')),  c = scale log2(e),  and o / l at the end.
// While m' exceeds m by less than 2^8 in the weights, m is kept (f = 1): the weights stay
// below 256 and the accumulated o needs no rescaling, which then is rare.
//
// A block takes 256 queries of one head as two tiles of 128, and the keys and values in
// tiles of 128, on the tcgen05 tensor cores with the accumulators in TMEM; then the next 256,
// one block per SM going through all of them (in strides: neighbours share keys in L2):
//   warps 0-3, 4-7   one tile each, a thread per query: S from TMEM, the softmax in
//                    registers, P back over S as 16-bit values, and at the end O / l;
//   warp 8           looks the pairs of tiles up and hands them out; TMA loads of Q and a ring
//                    of K and V tiles, on into the next pair;
//   warp 9           issues the products: S = Q K^T (both from shared memory), O += P V (P
//                    from TMEM, V from shared memory with its features contiguous; the first
//                    64 keys' part as soon as their weights are there).  While one tile is in
//                    its softmax, the other's products run; while a pair is finished, the next
//                    pair's first products.
// Every wait is bounded (GPTQ_ERR_TIMEOUT).
//
// 16 x 2048 causal tokens x 32 heads of 128: 795 us with waits polled by one lane of a warp and
// passed on, 730 polled by all lanes, 700 with the products issued by one elected thread, 680
// with the weights handed over in two parts, 627 with blocks that stay (877 TFLOP/s); packed
// sequences up to 6007, 64/8 heads: 1245, 1126, 1074, 1040, 1005 us, and 942 with eight heads to a
// tile (1059 TFLOP/s).  What bounds it: the chain of one tile, about 2300 cycles of softmax (1024
// of them exponentials) and 1500 for 16 products of 64 cycles and their latencies, of which the
// other tile hides half.  Tried and not kept: a quarter of the exponentials as polynomials on
// the fma units (slower or even), two threads per query (6% slower: the exchange of maxima),
// turns to and fro.
//
// Query heads of a k/v head may share tiles, whose rows then are the heads of one query, then those
// of the next (packed_heads).
//
// Few queries over many keys leave SMs idle: then a cluster of 2, 4 or 8 blocks shares a pair
// of tiles, each block taking a run of the key tiles; their (m, l, o) stay in shared memory,
// and every block joins its share of the rows from all of them.  37 queries after 2011 keys,
// 16/4 heads of 64: 39 us on one block per head, 16 on four, 12 with four heads to a tile; one
// query after 8000 keys, 8 heads of 128: 148 us on one, 23 on eight.
//
// Rows that no query may see: scores of keys past a row's limit are replaced before they are
// used; values past the sequence's end are zeroed in shared memory.  Inside a sequence a
// causal tile still multiplies weights of 0 with values behind the diagonal, which is
// exact unless one of them is not finite: a query whose result holds a NaN is therefore
// computed again one key at a time (seen_row), reading only what it sees.  Not where its sum of
// weights is a NaN: that comes from scores it sees, which make its whole row NaN (60,000 queries
// after a NaN key would each go through all keys by themselves).
#include <math.h>

#include <climits>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "vec_io.cuh"

namespace gptq {

namespace {

constexpr int TQ = 128;                   // queries of a tile, keys of a tile
constexpr int ATHREADS = 320;
constexpr int SMS = 148;                  // blocks, one to an SM, that go through the pairs of tiles
constexpr float LOG2E = 1.4426950408889634f;
constexpr int MOST = 64;                  // keys whose weights are handed over first
constexpr float KEEP = 8.f;               // log2 of the largest weight under a kept maximum

// A pair of tiles of one pack of heads: its sequence's first rows and lengths (pair -1: no more).
struct Work {
  int pair, h, q0, k0, lq, lk;
};

template <int KD>
struct AttnSmem {
  static constexpr int kTile = TQ * KD * 2;
  static constexpr int kStages = KD == 128 ? 5 : 10;
  uint8_t q[2][kTile];
  uint8_t kv[kStages][kTile];
  uint64_t q_full[2];
  uint64_t kv_full[kStages];
  uint64_t kv_empty[kStages];
  uint64_t s_full[2];
  uint64_t p_most[2];                     // the weights of the first MOST keys are in TMEM
  uint64_t p_full[2];
  uint64_t o_full[2];
  uint64_t q_empty[2];
  uint64_t work_full[2];
  uint64_t work_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int skip;
  int q_armed[2], kv_armed, committed;    // loads issued, products committed: what an abort waits for
  int valid;                              // this block's part of a shared pair of tiles is there
  Work work[2];                           // what the loader has handed out
  Work mine;                              // a shared pair of tiles (SPLIT)
};

// One tile's place: its queries, what they see, and how many key tiles that takes.
struct Tile {
  int row0, rows;                         // first query (of the sequence) and how many are real
  int shift;                              // query i sees keys below min(lk, i + shift)
  int blocks;
};

__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 32 columns of this thread's TMEM lane; the values are there after tmem_wait(v).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
        "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
        "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
        "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
      :: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      :: "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
         "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
         "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
         "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      :: "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
         "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] . B[smem], kind::f16: A as 16-bit pairs per column, a row per lane.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// B operand with its N dimension contiguous (values: a token's features), 128-byte
// swizzle: rows of 64 features, 8-token atoms of 1024 bytes, the next 64 features
// `lead` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;  // leading byte offset: the next 64 features
  d |= (uint64_t)(1024u >> 4) << 32;             // stride byte offset: 8 tokens
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ bool drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = tc::globaltimer();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (tc::globaltimer() - t0 > 1000000000ull) return false;
  }
  return true;
}

// A whole warp waits for a barrier's phase.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag));
}

// One thread of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Slot `slot` (the sequences in order, a sequence's pairs from the last, which sees the most
// keys, to the first) of head h; whole warp.  The slots of one warp's calls ascend: b0 and base
// (0 at first) say where the last one was found.  Sequences with bad bounds have no pairs and
// are recorded.
__device__ __forceinline__ Work find_work(const AttentionArgs& A, int slot, int h, int& b0, int& base, int32_t* st) {
  const int lane = threadIdx.x & 31;
  Work w{-1, h, 0, 0, 0, 0};
  for (; b0 < A.count; b0 += 32) {
    const int b = b0 + lane;
    int pairs = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    if (b < A.count) {
      q0 = A.cu_q[b];
      q1 = A.cu_q[b + 1];
      k0 = A.cu_k[b];
      k1 = A.cu_k[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > A.total_q || k0 < 0 || k1 < k0 || k1 > A.total_k)
        set_own_error(st, A.launch, GPTQ_ERR_INVALID_ARG, b, STAGE_ATTENTION);
      else
        pairs = (int)((((int64_t)(q1 - q0) << A.packed) + 2 * TQ - 1) / (2 * TQ));
    }
    int incl = pairs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > slot);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.pair = __shfl_sync(0xffffffffu, base + incl - 1 - slot, src);
      w.q0 = __shfl_sync(0xffffffffu, q0, src);
      w.k0 = __shfl_sync(0xffffffffu, k0, src);
      w.lq = __shfl_sync(0xffffffffu, q1, src) - w.q0;
      w.lk = __shfl_sync(0xffffffffu, k1, src) - w.k0;
      return w;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

__device__ __forceinline__ Tile make_tile(const AttentionArgs& A, int first, int lq, int lk) {
  Tile t;
  t.row0 = first;
  t.rows = max(0, min(TQ, (lq << A.packed) - first));
  t.shift = A.causal ? 1 + lk - lq : lk;
  const int last = t.rows > 0 ? (A.causal ? min(lk, ((first + t.rows - 1) >> A.packed) + t.shift) : lk) : 0;
  t.blocks = last > 0 ? (last + TQ - 1) / TQ : 0;
  return t;
}

// Row `row` of a pair: its query, head, and how many keys it sees (0 behind the sequence's end).
struct Row {
  int query, head, seen;
  __device__ __forceinline__ Row(const AttentionArgs& A, const Work& w, int row) {
    const int i = w.pair * 2 * TQ + row;
    query = i >> A.packed;
    head = (w.h << A.packed) + (i & ((1 << A.packed) - 1));
    seen = query < w.lq ? max(0, min(w.lk, A.causal ? query + 1 + w.lk - w.lq : w.lk)) : 0;
  }
};

// The two tiles of a pair, as one block of `size` that share it takes them.
struct Tiles {
  Tile t[2];
  int first;                              // this block's first key
  int blocks;                             // key tiles
  int tail;                               // the last tile of values reaches past the sequence's end: rows it has
  __device__ __forceinline__ Tiles(const AttentionArgs& A, const Work& w, int size, int rank) {
    t[0] = make_tile(A, w.pair * 2 * TQ, w.lq, w.lk);
    t[1] = make_tile(A, w.pair * 2 * TQ + TQ, w.lq, w.lk);
    first = 0;
    if (size > 1) {
      const int share = (max(t[0].blocks, t[1].blocks) + size - 1) / size;
      first = rank * share * TQ;
#pragma unroll
      for (int i = 0; i < 2; ++i) t[i].blocks = max(0, min(share, t[i].blocks - rank * share));
    }
    blocks = max(t[0].blocks, t[1].blocks);
    tail = blocks > 0 && first + blocks * TQ > w.lk ? w.lk - first - (blocks - 1) * TQ : 0;
  }
};

// One query against the keys it sees, one after another, by a whole warp (see above).
template <typename T>
__device__ __forceinline__ void seen_row(const AttentionArgs& A, int t, int h, int hk, int k0, int seen) {
  const int lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(A.q) + t * A.q_ts + h * A.q_hs;
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    float sc = -INFINITY;
    if (j < seen) {
      const T* k = static_cast<const T*>(A.k) + (int64_t)(k0 + j) * A.k_ts + hk * A.k_hs;
      sc = 0.f;
      for (int i = 0; i < A.head_dim; i += 8) {
        float x[8], y[8];
        load8(k + i, x);
        load8(q + i, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) sc = fmaf(y[e], x[e], sc);
      }
      sc *= A.scale;
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
      const T* v = static_cast<const T*>(A.v) + (int64_t)(k0 + j0 + o) * A.v_ts + hk * A.v_hs;
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

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
template <int N>
__device__ __forceinline__ void load_cluster(uint32_t addr, float (&v)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr) : "memory");
}

// Where a part's values lie in shared memory: row r's pieces of 4, in another order per row
// (rows would share banks).
template <int KD>
__device__ __forceinline__ int part_at(int r, int piece) { return r * KD + ((piece ^ (r & (KD / 4 - 1))) << 2); }

// Joins a share of the rows of a pair of tiles from the parts of the cluster's blocks: a warp
// per row.
template <int KD, typename T>
__device__ __forceinline__ void join_parts(const AttentionArgs& A, AttnSmem<KD>& S) {
  constexpr int V = KD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t size = cluster_size(), rank = tc::cluster_rank();
  int ok = 1;                                             // lane c: block c's word, its (m, l)
  if (lane < (int)size)
    asm volatile("ld.shared::cluster.b32 %0, [%1];"
                 : "=r"(ok) : "r"(tc::map_to_cta(tc::smem_u32(&S.valid), lane)) : "memory");
  if (!__all_sync(0xffffffffu, ok)) return;
  const Work w = S.mine;
  const int hk = (w.h << A.packed) / (A.heads_q / A.heads_kv);
  const int rows = min(2 * TQ, (w.lq << A.packed) - w.pair * 2 * TQ);
  for (int r = (int)rank + warp * (int)size; r < rows; r += (int)size * (ATHREADS / 32)) {
    const Row me(A, w, r);
    const uint32_t ml_at = tc::smem_u32(S.q[0]) + r * 8;
    // feature piece: V consecutive values per lane
    const uint32_t o_at = tc::smem_u32(S.kv[0]) + (part_at<KD>(r, lane * V / 4) + lane * V % 4) * 4;
    float ml[2] = {-INFINITY, 0.f};
    if (lane < (int)size) load_cluster(tc::map_to_cta(ml_at, lane), ml);
    // a block that saw no key of this row has no values either
    const unsigned live = __ballot_sync(0xffffffffu, !(ml[0] == -INFINITY && ml[1] == 0.f));
    float o[8][V];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
      for (int e = 0; e < V; ++e) o[c][e] = 0.f;
      if (live >> c & 1) load_cluster(tc::map_to_cta(o_at, c), o[c]);
    }
    float top = ml[0];
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i, 8));
    const float f = exp2_approx(ml[0] - (top == -INFINITY ? 0.f : top));
    float l = ml[1] * f, acc[V];
#pragma unroll
    for (int i = 4; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i, 8);
    l = __shfl_sync(0xffffffffu, l, 0);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float x = __shfl_sync(0xffffffffu, f, c);
      if (live >> c & 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(o[c][e], x, acc[e]);
      }
    }
    const float inv = 1.f / l;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      acc[e] = me.seen == 0 ? 0.f : acc[e] * inv;
      nan |= acc[e] != acc[e];
    }
    T* dst = static_cast<T*>(A.o) + (int64_t)(w.q0 + me.query) * A.o_ts + me.head * A.o_hs;
    if (lane * V < A.head_dim) {
      uint32_t u[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) u[e] = pack2(acc[2 * e], acc[2 * e + 1], T());
      if constexpr (V == 4) *reinterpret_cast<uint2*>(dst + lane * V) = make_uint2(u[0], u[1]);
      else *reinterpret_cast<uint32_t*>(dst + lane * V) = u[0];
    }
    if (__any_sync(0xffffffffu, nan) && l == l) {
      __syncwarp();                                       // the row's first values before its second
      seen_row<T>(A, w.q0 + me.query, me.head, hk, w.k0, me.seen);
    }
  }
}

template <int KD, typename T, bool SPLIT>
__global__ void __launch_bounds__(ATHREADS, 1)
attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ AttentionArgs A, int pairs, int32_t* st) {
  using Smem = AttnSmem<KD>;
  constexpr int NST = Smem::kStages, TILE = Smem::kTile;
  constexpr uint32_t FMT = std::is_same<T, __half>::value ? 0 : 1;
  constexpr uint32_t IDESC_S = tc::idesc_f32acc(FMT, TQ, TQ);
  constexpr uint32_t IDESC_O = tc::idesc_f32acc(FMT, TQ, KD) | (1u << 16);    // B with N contiguous
  constexpr uint32_t O_COL = 2 * TQ;                                          // TMEM: S0, S1, O0, O1
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int size = SPLIT ? (int)cluster_size() : 1, rank = SPLIT ? (int)tc::cluster_rank() : 0;
  const int step = (int)gridDim.x / size;                 // pairs of tiles taken at once
  const int packs = A.heads_q >> A.packed;
  int at = (int)blockIdx.x / size;                        // the loader's pair (of every head), then at + step, ...
  Work w{-1, 0, 0, 0, 0, 0};

  if (warp == 9) tc::tmem_alloc<512>(&S.tmem_base);
  int b0 = 0, base = 0;
  if (warp == 8) w = find_work(A, at / packs, at % packs, b0, base, st);
  if (warp == 0 && lane == 0) {
    S.skip = stopped(st, A.launch);
    S.abort = 0;
    S.q_armed[0] = S.q_armed[1] = S.kv_armed = S.committed = 0;
    S.mine.pair = -1;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&S.q_full[i], 1);
      tc::mbar_init(&S.q_empty[i], 1);
      tc::mbar_init(&S.s_full[i], 1);
      tc::mbar_init(&S.p_most[i], 4);
      tc::mbar_init(&S.p_full[i], 4);
      tc::mbar_init(&S.o_full[i], 1);
      tc::mbar_init(&S.work_full[i], 1);
      tc::mbar_init(&S.work_empty[i], 9);
    }
    for (int i = 0; i < NST; ++i) { tc::mbar_init(&S.kv_full[i], 1); tc::mbar_init(&S.kv_empty[i], 1); }
    tc::mbar_init(&S.drain, 1);
    tc::fence_barrier_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = S.tmem_base;
  volatile int* abort_flag = &S.abort;
  // the n-th pair that the loader hands out (whole warp; given back with done(n)); false after the
  // last, or on an abort
  auto handed = [&](int n) {
    const volatile Work& v = S.work[n & 1];
    return Work{v.pair, v.h, v.q0, v.k0, v.lq, v.lk};
  };
  auto take = [&](int n) {
    if (!warp_wait(&S.work_full[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag)) return false;
    w = handed(n);
    return w.pair >= 0;
  };
  auto done = [&](int n) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&S.work_empty[n & 1]);
  };

  if (!S.skip) {
    if (warp == 8) {
      int it = 0, q_uses[2] = {0, 0};                     // loads into the ring, into Q
      for (int n = 0;; ++n) {
        if (!warp_wait(&S.work_empty[n & 1], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag)) break;
        if (lane == 0) {
          S.work[n & 1] = w;
          if (SPLIT && w.pair >= 0) S.mine = w;
          tc::mbar_arrive(&S.work_full[n & 1]);
        }
        if (w.pair < 0) break;
        const Tiles tl(A, w, size, rank);
        const int hk = (w.h << A.packed) / (A.heads_q / A.heads_kv);
        int ok = 1;
        if (lane == 0) {
          for (int i = 0; i < 2 * tl.blocks && ok; ++i, ++it) {
            if (i < 2 && tl.t[i].blocks > 0) {
              ok = tc::mbar_wait(&S.q_empty[i], ((uint32_t)q_uses[i] & 1u) ^ 1u, abort_flag);
              if (!ok) break;
              tc::mbar_arrive_expect_tx(&S.q_full[i], TILE);
#pragma unroll
              for (int c = 0; c < KD / 64; ++c)
                tma_load_3d(S.q[i] + c * (TQ * 128), &tq, &S.q_full[i], c * 64, w.h << A.packed,
                            w.q0 + (tl.t[i].row0 >> A.packed));
              S.q_armed[i] = ++q_uses[i];
            }
            const int s = it % NST;
            ok = tc::mbar_wait(&S.kv_empty[s], ((uint32_t)(it / NST) & 1u) ^ 1u, abort_flag);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(&S.kv_full[s], TILE);
            const CUtensorMap* map = (i & 1) ? &tv : &tk;
#pragma unroll
            for (int c = 0; c < KD / 64; ++c)
              tma_load_3d(S.kv[s] + c * (TQ * 128), map, &S.kv_full[s], c * 64, hk, w.k0 + tl.first + (i >> 1) * TQ);
            S.kv_armed = it + 1;
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        at += step;
        w.pair = -1;
        if (!SPLIT && at < pairs)
          w = find_work(A, at / packs, at % packs, b0, base, st);
      }
    } else if (warp == 9) {
      // The whole warp walks the loop, so that the products' descriptors stay in uniform
      // registers, and one elected thread issues (under a branch on the lane every product cost
      // about 90 cycles to issue, 64 to run).
      const bool one = elect_one();
      // S of tile t from the key tile in stage s; `last`: Q is not needed any more
      auto product_s = [&](int t, int s, bool last) {
        const uint64_t a0 = tc::sdesc_k_sw128(tc::smem_u32(S.q[t])), b0 = tc::sdesc_k_sw128(tc::smem_u32(S.kv[s]));
        if (one) {
#pragma unroll
          for (int k = 0; k < KD / 16; ++k) {
            const uint32_t off = ((k / 4) * (TQ * 128) + (k % 4) * 32) >> 4;   // in the descriptor's units
            tc::mma_f16(taddr + t * TQ, a0 + off, b0 + off, IDESC_S, k > 0);
          }
          tc::mma_commit(&S.s_full[t]);
          if (last) tc::mma_commit(&S.q_empty[t]);
        }
      };
      bool ok = true;
      int it = 0;                                         // the pair's first load in the ring
      uint32_t q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
      for (int n = 0; ok && take(n); ++n) {
        const Tiles tl(A, w, size, rank);
        done(n);
        const int blocks = tl.blocks;
        if (blocks == 0) continue;
        ok = tc::mbar_wait(&S.kv_full[it % NST], (uint32_t)(it / NST) & 1u, abort_flag);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || tl.t[t].blocks == 0) continue;
          ok = tc::mbar_wait(&S.q_full[t], q_uses[t] & 1u, abort_flag);
          if (!ok) break;
          ++q_uses[t];
          tc::tc_fence_after();
          product_s(t, it % NST, tl.t[t].blocks == 1);
        }
        if (ok && one) tc::mma_commit(&S.kv_empty[it % NST]);
        for (int j = 0; j < blocks && ok; ++j) {
          const int iv = it + 2 * j + 1, ik = it + 2 * j + 2;
          const int sv = iv % NST, sk = ik % NST;
          ok = tc::mbar_wait(&S.kv_full[sv], (uint32_t)(iv / NST) & 1u, abort_flag);
          if (ok && tl.tail > 0 && j == blocks - 1) {     // rows behind the sequence's end, zeroed
            for (int i = tl.tail * 8 + lane; i < TQ * 8; i += 32)
#pragma unroll
              for (int c = 0; c < KD / 64; ++c)
                *reinterpret_cast<uint4*>(S.kv[sv] + c * (TQ * 128) + i * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          if (ok && j + 1 < blocks) ok = tc::mbar_wait(&S.kv_full[sk], (uint32_t)(ik / NST) & 1u, abort_flag);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) break;
            if (j < tl.t[t].blocks) {
              const uint64_t b0 = sdesc_mn_sw128(tc::smem_u32(S.kv[sv]), TQ * 128);
              ok = tc::mbar_wait(&S.p_most[t], p_uses[t] & 1u, abort_flag);
              if (!ok) break;
              tc::tc_fence_after();
              if (one) {
#pragma unroll
                for (int k = 0; k < MOST / 16; ++k)
                  mma_f16_ts(taddr + O_COL + t * KD, taddr + t * TQ + k * 8, b0 + (k * 2048 >> 4), IDESC_O, j > 0 || k > 0);
              }
              ok = tc::mbar_wait(&S.p_full[t], p_uses[t] & 1u, abort_flag);
              if (!ok) break;
              ++p_uses[t];
              tc::tc_fence_after();
              if (one) {
#pragma unroll
                for (int k = MOST / 16; k < TQ / 16; ++k)
                  mma_f16_ts(taddr + O_COL + t * KD, taddr + t * TQ + k * 8, b0 + (k * 2048 >> 4), IDESC_O, true);
                if (j + 1 == tl.t[t].blocks) tc::mma_commit(&S.o_full[t]);
              }
            }
            if (t == 1 && one) tc::mma_commit(&S.kv_empty[sv]);
            if (j + 1 < tl.t[t].blocks) product_s(t, sk, j + 2 == tl.t[t].blocks);
            if (t == 1 && j + 1 < blocks && one) tc::mma_commit(&S.kv_empty[sk]);
          }
        }
        it += 2 * blocks;
      }
      // every commit has arrived before the block's shared memory is given up
      __syncwarp();
      if (one) {
        tc::mma_commit(&S.drain);
        S.committed = 1;
        if (!*abort_flag) drain_wait(&S.drain, 0);
      }
    } else {
      const int t = warp >> 2;                            // warps 0-3: tile 0, 4-7: tile 1
      const int r = (warp & 3) * 32 + lane;               // this thread's query in the tile
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = taddr + lanes + t * TQ, to = taddr + lanes + O_COL + t * KD;
      uint32_t s_uses = 0, o_uses = 0;
      bool ok = true;
      for (int n = 0; ok && take(n); ++n) {
        int blocks, see0;                                 // key tiles; keys that this thread's query sees, from `first`
        {
          const Tiles tl(A, w, size, rank);
          blocks = tl.t[t].blocks;
          see0 = Row(A, w, t * TQ + r).seen - tl.first;
        }
        const float c0 = A.scale * LOG2E;
        const float c = c0 > 0.f ? c0 : 1.f;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < blocks; ++j) {
          ok = warp_wait(&S.s_full[t], s_uses & 1u, abort_flag);
          if (!ok) break;
          ++s_uses;
          tc::tc_fence_after();
          float s[TQ];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(ts + i * 32, s + i * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_wait(s + i * 32);
          if (!(c0 > 0.f)) {                                // a scale of 0 or below: the product first
#pragma unroll
            for (int i = 0; i < TQ; ++i) s[i] *= c0;
          }
          const int see = see0 - j * TQ;
          if (__any_sync(0xffffffffu, see < TQ)) {
#pragma unroll
            for (int i = 0; i < TQ; ++i) s[i] = i < see ? s[i] : -INFINITY;
          }
          float mx[4] = {m, m, m, m};
#pragma unroll
          for (int i = 0; i < TQ; i += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[e]) : "f"(s[i + 2 * e]), "f"(s[i + 2 * e + 1]));
          }
          const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          if (j == 0) {
            m = mn;
          } else {
            const bool up = (mn - m) * c > KEEP;            // -inf to finite included
            if (__any_sync(0xffffffffu, up)) {
              // S's arrival also says that the products into O issued before it are done
              const float f = up ? exp2_approx((m - mn) * c) : 1.f;
              if (up) m = mn;
              l *= f;
#pragma unroll 1
              for (int i = 0; i < KD; i += 32) {
                float o[32];
                tmem_ld32(to + i, o);
                tmem_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(to + i, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m * c;
          const uint64_t c2 = pack_f32x2(c, c), r2 = pack_f32x2(-ref, -ref);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < TQ; i += 32) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              unpack_f32x2(fma2(pack_f32x2(s[i + 2 * e], s[i + 2 * e + 1]), c2, r2), a, b);
              a = exp2_approx(a);
              b = exp2_approx(b);
              sum[e & 3] = add2(sum[e & 3], pack_f32x2(a, b));
              p[e] = pack2(a, b, T());
            }
            tmem_st16(ts + i / 2, p);
            if (i + 32 == MOST) {                           // their product may begin
              tmem_st_wait();
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&S.p_most[t]);
            }
          }
          float a, b;
          unpack_f32x2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
          l += a + b;
          tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&S.p_full[t]);
        }
        if constexpr (SPLIT) {
          // both tiles' products are done with the shared memory that the parts go to
          const Tiles tl(A, w, size, rank);
          for (int u = 0; u < 2; ++u)
            if (ok && tl.t[u].blocks > 0) ok = warp_wait(&S.o_full[u], 0, abort_flag);
          if (ok) {
            tc::tc_fence_after();
            const int row = t * TQ + r;
            reinterpret_cast<float2*>(S.q[0])[row] = make_float2(m * c, l);
            float* part = reinterpret_cast<float*>(S.kv[0]);
            if (blocks > 0) {
#pragma unroll 1
              for (int i = 0; i < KD; i += 32) {
                float o[32];
                tmem_ld32(to + i, o);
                tmem_wait(o);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<float4*>(part + part_at<KD>(row, (i + e) / 4)) =
                      make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
              }
            }
          }
        } else if (ok) {
          if (blocks > 0) ok = warp_wait(&S.o_full[t], o_uses++ & 1u, abort_flag);
          if (ok) {
            tc::tc_fence_after();
            const Work v = handed(n);
            const Row me(A, v, t * TQ + r);
            const int limit = me.seen;
            const bool mine = me.query < v.lq;
            T* dst = static_cast<T*>(A.o) + (int64_t)(v.q0 + me.query) * A.o_ts + me.head * A.o_hs;
            const float inv = limit > 0 ? 1.f / l : 0.f;
            bool nan = false;
#pragma unroll 1
            for (int i = 0; i < KD; i += 16) {
              float o[16];
              tmem_ld16_wait(to + i, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                o[e] = limit > 0 ? o[e] * inv : 0.f;
                nan |= o[e] != o[e];
              }
              if (mine) {
                if (i < A.head_dim) store8(dst + i, o);
                if (i + 8 < A.head_dim) store8(dst + i + 8, o + 8);
              }
            }
            unsigned again = __ballot_sync(0xffffffffu, nan && mine);
            __syncwarp();                                 // a row's first values before its second
            while (again != 0) {
              const int src = __ffs(again) - 1;
              again &= again - 1;
              const float sum = __shfl_sync(0xffffffffu, l, src);
              if (sum != sum) continue;                   // (asked here: with the ballot all rows took 0.7% longer)
              const Row row(A, v, t * TQ + r - lane + src);
              seen_row<T>(A, v.q0 + row.query, row.head, row.head / (A.heads_q / A.heads_kv), v.k0, row.seen);
            }
          }
        }
        done(n);
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 8 && lane == 0) {
      for (int it = max(0, S.kv_armed - NST); it < S.kv_armed; ++it)
        drain_wait(&S.kv_full[it % NST], (uint32_t)(it / NST) & 1u);
      for (int i = 0; i < 2; ++i)
        if (S.q_armed[i] > 0) drain_wait(&S.q_full[i], (uint32_t)(S.q_armed[i] - 1) & 1u);
    }
    if (warp == 9 && lane == 0 && S.committed) drain_wait(&S.drain, 0);
    if (threadIdx.x == 0) set_error(st, GPTQ_ERR_TIMEOUT, blockIdx.x, STAGE_ATTENTION);
    __syncthreads();
  }
  if (warp == 9) {
    __syncwarp();
    tc::tmem_dealloc<512>(taddr);
  }
  if constexpr (SPLIT) {
    if (threadIdx.x == 0) S.valid = !S.skip && !*abort_flag && S.mine.pair >= 0;
    __syncwarp();
    tc::cluster_sync();                                   // every block's part is there, or said not to be
    join_parts<KD, T>(A, S);
    __syncwarp();
    tc::cluster_sync();                                   // and has been read
  }
}

// Pairs of tiles, of every pack of heads, at most.
int64_t most_pairs(const AttentionArgs& A) {
  return ((((int64_t)A.total_q << A.packed) / (2 * TQ)) + A.count) * (A.heads_q >> A.packed);
}

// Query heads of one k/v head share tiles (2^packed of them, their rows the queries' heads in
// turn): until an average sequence fills a tile, and on while there is work for every SM four
// times over (a pair of tiles then spans fewer queries, whose causal limits are closer: packed
// sequences, 64/8 heads: 1005 us with none, 942 with eight; 64 queries, 32/8 heads: 8 us with
// none or two, 11 with four, whose blocks are too few).
int packed_heads(AttentionArgs A) {
  const int per = A.heads_q / A.heads_kv;
  A.packed = 0;
  while (A.packed < 4 && per % (2 << A.packed) == 0 && ((int64_t)A.total_q << (A.packed + 1)) <= INT32_MAX - 2 * TQ &&
         ((((int64_t)A.total_q / A.count) << A.packed) < TQ || most_pairs(A) >= 4 * SMS))
    ++A.packed;
  return A.packed;
}

// Blocks that share a pair of tiles: as many as run at once (74 clusters of two, 33 of four,
// 15 of eight at this shared memory: a cluster stays in one part of the chip) and have two
// key tiles or more of an average sequence.
int cluster_of(const AttentionArgs& A) {
  const int64_t work = most_pairs(A), tiles = A.total_k / A.count / TQ;
  if (work <= 15 && tiles >= 16) return 8;
  if (work <= 33 && tiles >= 8) return 4;
  return work <= 74 && tiles >= 4 ? 2 : 1;
}

template <int KD, typename T, bool SPLIT>
int launch(const AttentionArgs& A, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int size,
           int32_t* st, cudaStream_t s) {
  const size_t smem = sizeof(AttnSmem<KD>) + 1024;
  auto* kernel = attention_kernel<KD, T, SPLIT>;
  GPTQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  const int64_t pairs = most_pairs(A) + 1;                // and one block that reads every bound
  if (pairs * size > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? pairs * size : (pairs < SMS ? pairs : SMS)));
  cfg.blockDim = dim3(ATHREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)size;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = SPLIT ? 1 : 0;
  GPTQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, A, (int)pairs, st));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int KD, typename T>
int launch_any(const AttentionArgs& A, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int32_t* st,
               cudaStream_t s) {
  const int size = cluster_of(A);
  return size > 1 ? launch<KD, T, true>(A, tq, tk, tv, size, st, s) : launch<KD, T, false>(A, tq, tk, tv, 1, st, s);
}

// [tokens, heads, head_dim] in boxes of 128 rows (tokens, each of 2^packed heads) by 64
// features; features past head_dim and tokens past the end read as 0.
int head_map(CUtensorMap* map, CUtensorMapDataType dt, const void* p, int tokens, int heads, int head_dim, int64_t ts,
             int64_t hs, int packed) {
  return make_tmap_3d(map, dt, p, (uint64_t)head_dim, (uint64_t)heads, (uint64_t)tokens, (uint64_t)hs * 2,
                      (uint64_t)ts * 2, 64, 1u << packed, (uint32_t)(TQ >> packed), CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

int launch_attention(const AttentionArgs& args, int dtype, int32_t* st, cudaStream_t s) {
  AttentionArgs A = args;
  A.packed = packed_heads(A);
  A.launch = next_launch();
  CUtensorMap tq, tk, tv;
  const CUtensorMapDataType dt = dtype == GPTQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int rc = head_map(&tq, dt, A.q, A.total_q, A.heads_q, A.head_dim, A.q_ts, A.q_hs, A.packed);
  if (rc != GPTQ_OK) return rc;
  tk = tv = tq;                           // without any key nothing is loaded through them
  if (A.total_k > 0) {
    rc = head_map(&tk, dt, A.k, A.total_k, A.heads_kv, A.head_dim, A.k_ts, A.k_hs, 0);
    if (rc == GPTQ_OK) rc = head_map(&tv, dt, A.v, A.total_k, A.heads_kv, A.head_dim, A.v_ts, A.v_hs, 0);
    if (rc != GPTQ_OK) return rc;
  }
  TraceScope ts("attention", "", 0.0, s);
  if (A.head_dim <= 64)
    return dtype == GPTQ_F16 ? launch_any<64, __half>(A, tq, tk, tv, st, s)
                             : launch_any<64, __nv_bfloat16>(A, tq, tk, tv, st, s);
  return dtype == GPTQ_F16 ? launch_any<128, __half>(A, tq, tk, tv, st, s)
                           : launch_any<128, __nv_bfloat16>(A, tq, tk, tv, st, s);
}

}  // namespace gptq
