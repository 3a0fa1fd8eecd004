// Attention of many new tokens per request over its paged cache (hs_paged_attend):
//
//   s_n = scale q_h . K_n;  s_n <- cap tanh(s_n / cap);  s_n <- s_n - slope_h |p - n|
//   o_h = sum_n softmax_n(s_n) V_n,  lse_h = ln sum_n exp(s_n)
//
// over the positions n that the token at p sees, in one pass with a running maximum m and sum l.
//
// Bound: the tensor cores for prompts (4 d flops for a query, a head and a position it sees), HBM for
// a few tokens over long contexts.  Rows of a block are (token, query head) pairs of one kv head, token
// by token, whatever the group's size, so that every head of the group shares the rows of keys and
// values that are read and short prompts fill blocks.
//
// Measured (GB300; bf16 products at 1940 TFLOP/s, copies at 6.8 TB/s).  32/8 heads of 128, bf16: 8192
// tokens on 24576 positions 2.48 ms, 1550 TFLOP/s (80 % of measured); a prompt of 8192 453 us, 1215
// TFLOP/s, with capped scores 705 us, with a distance bias 610 us, over 8-bit pages 645 us, 4-bit ones 675;
// 512 tokens on 30 K positions of 4-bit pages 500 us, 1015 TFLOP/s; 64 requests of 5 tokens on 4 K
// positions 205 us, 5.3 TB/s; one of them 22 us.  (The first kernel, a warp per token and head, took 489 ms for the capped prompt.)
//
// A CTA per SM, its warps in roles.  Scores: tcgen05 S = Q K^T, 128 x 128 x d, queries and keys in shared
// memory, sums in TMEM; weights go back to TMEM as 16-bit numbers and are the first operand of O += P V.
// Two tiles of 128 rows take turns, so that one's softmax runs while the other's products do; at d = 256,
// where TMEM holds one tile's sums only, tiles of 64 positions and two buffers of scores do the same.
//   softmax   a warp per 32 rows, a thread per row: no exchange between threads; the sums are rescaled
//             only where a score is far above the reference (pa::SLACK), which is rare
//   products  one warp issues everything, as one, so that descriptors stay in uniform registers: issued
//             by a lone thread they took longer than the products (8192 tokens: 852 -> 703 us)
//   copies    a warp: pages by TMA into a ring of stages (keys, values, keys ...), 128-byte swizzled
//   a look    a warp: values that no row of the block sees become 0 (a weight of 0 would leave a NaN)
//   queries   a warp: rows of any strides by 16-byte copies into the swizzled tile, for the next piece
//             while this one ends
//   8/4 bits  four warps turn rows of those pages into fp16 between two rings (exactly: their scales are
//             folded into the scores and the output, or, of 4-bit rows, have 4 bits); bf16 queries come
//             as fp16 under a power of two per row
// Code size is what the inner loops were made short for: unrolled over a tile's 128 columns, the softmax's
// and the turning's code (13 KB each) left warps waiting for instructions (4-bit chunks 774 -> 484 us when
// the turning became a loop, 8192 tokens 703 -> 582 us with the softmax's).
//
// Weights are rounded to 16 bits once (bf16 2^-8, fp16 and 8- and 4-bit pages 2^-11 of themselves): the
// relative error of bf16 outputs is 0.0022 where 32-bit weights give 0.0017; a second part, as one-token
// attention has, would cost half as much again of the tensor time.  Sums and the softmax are in 32 bits.
//
// Work.  Segments (block of rows, kv head) have as many tiles as their last row sees; all tiles of the
// call, and for each segment the cost of its start, form one sequence, and every CTA takes an equal share
// of it.  What lies wholly in a share is written out; a segment cut by shares goes to the workspace in
// pieces (at most two per CTA) that a second kernel joins.  So one request of 5 tokens on 4 K positions
// and a batch of ragged prompts are spread the same way.  Nothing is kept between calls.
#ifndef HS_PAGED_ATTEND_CUH_
#define HS_PAGED_ATTEND_CUH_

#include "hs_paged_attention.cuh"

namespace hs {
namespace pt {

using pa::FP16_SHIFT;
using pa::LOG2_E;
using pa::pow2;
using pa::SLACK;

template <int D_, int QTYPE_, int PAGES_>
struct Cfg {
  static constexpr int D = D_, QTYPE = QTYPE_, PAGES = PAGES_;
  static constexpr bool CONV = PAGES != PAGES_SAME;            // pages are turned into fp16 on the way
  static constexpr bool BF16 = QTYPE == HS_BF16 && !CONV;      // type of the products
  static constexpr int NQ = D == 256 ? 1 : 2;                  // tiles of 128 rows of a block
  static constexpr int KT = D == 256 ? 64 : 128;               // positions of a tile
  static constexpr int ROWS = 128 * NQ;
  static constexpr int BLK = D / 64;                           // 128-byte blocks of a row
  static constexpr int QB = 128 * D * 2;                       // bytes of a tile's queries
  static constexpr int STAGE = KT * D * 2;
  static constexpr int STAGES = D == 64 ? 8 : CONV ? 4 : 5;
  // 8- and 4-bit pages: what a tile's keys or values (8 bits: half of them) take there, and places for that
  static constexpr bool INT4 = PAGES == PAGES_INT4;
  static constexpr int UNIT_BYTES = INT4 ? 9 * D : 16 * D;
  static constexpr int PARTS = CONV && !INT4 ? 2 : 1, RAW_ROWS = KT / PARTS;
  static constexpr int RAW = CONV ? RAW_ROWS / PG_UNIT * UNIT_BYTES : 0;
  static constexpr int RAWS = CONV ? (INT4 ? 3 : 4) : 0;
  static constexpr int SOFT = 4 * NQ;                          // softmax warps
  static constexpr int W_MMA = SOFT, W_LOAD = SOFT + 1, W_FIX = SOFT + 2, W_Q = SOFT + 3, W_CONV = SOFT + 4;
  static constexpr int Q0 = CONV ? W_FIX : W_Q, Q_WARPS = W_Q - Q0 + 1;   // warps that bring queries
  static constexpr int WARPS = SOFT + 4 + (CONV ? 4 : 0);
  static constexpr int THREADS = 32 * WARPS;
  // columns of TMEM
  // two buffers of scores, two of weights, the sums.  Products of one shape run in the order of their
  // issue, so that at d = 128, where both products are 128 x 128, weights may lie over the scores they came
  // from (the next scores follow the product that reads them); elsewhere they need columns of their own.
  static constexpr int T_S = 0;
  static constexpr int T_P = D == 128 ? 0 : 2 * KT;
  static constexpr int P_STEP = D == 128 ? KT : KT / 2;
  static constexpr int T_O = D == 128 ? 2 * KT : 3 * KT;
  static constexpr int TCOLS = 512;
  static constexpr int SM_RING = NQ * QB;
  static constexpr int SM_RAW = SM_RING + STAGES * STAGE;
  static constexpr int SM_META = (SM_RAW + RAWS * RAW + 1023) / 1024 * 1024;
  static constexpr size_t SMEM = 1024 + SM_META + sizeof(int) * 256;
  static constexpr int PIECE = ROWS * D + 2 * ROWS;            // floats of a piece: o [d / 4][row][4], m, l
  // of a segment on top of its tiles, in tiles: queries, the first scores, output: some 6 us (where rows are
  // turned, 10), of tiles of 1.6 us at d = 128 and 1 us, of 64 positions, at 256; with 4 and 7 a prompt of
  // 8192 over 4-bit pages takes 815 and 675 us, with 3 and 5 one over 16-bit pages 494 and 456
  static constexpr int SEGMENT_COST = D == 64 ? 4 : D == 128 && !CONV ? 5 : 7;
};

struct Meta {
  uint64_t full[8], empty[8], ready[8], raw_full[6], raw_empty[6];
  uint64_t q_full, q_empty, s_full[2], p_ready[2][2], o_done[2], drain;
  uint32_t tmem;
  int abort;
  int begin[7];                  // of the share: request, block, head, first tile; 1: there is one; what lies of the
                                 // segment before it; cost of a segment on top of its tiles
  unsigned char bad[8];          // of a tile: its units of 16 positions on pages out of range
  signed char q_exp[2][256];     // power of two that a row of queries was divided by
};
static_assert(sizeof(Meta) <= 1024, "meta");

// ---- tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The products' warp runs as one, so that operands are uniform registers, and `one` (of its lanes) issues.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t one) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
               "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)), "r"(one)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
               "r"((uint32_t)add), "r"(one)
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
               "r"((uint32_t)add), "r"(one)
               : "memory");
}
#define HS_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define HS_S8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of the thread's lane
__device__ __forceinline__ void tmem_load32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : HS_R8(r, 0), HS_R8(r, 8), HS_R8(r, 16), HS_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::HS_S8(r, 0), HS_S8(r, 8), HS_S8(r, 16), HS_S8(r, 24), "r"(addr)
      : "memory");
}
#undef HS_R8
#undef HS_S8
// (and no use of what was loaded moves before it)
template <int N>
__device__ __forceinline__ void tmem_wait_load(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_load8(uint32_t* r, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
               : "memory");
}

// ---- two 32-bit numbers at a time
using F2 = unsigned long long;
__device__ __forceinline__ F2 two(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 apart(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// tanh(x) / x as a polynomial of x^2, the one with the least relative error on its range (found by
// exchange): 5.5e-7 for |x| <= 1/2, 6.2e-7 for |x| <= 1, and 7.6e-7 with the roundings of 32 bits.  Six or eight products a score, where e^2x and its
// reciprocal would cost two special functions and as many (a tile of 128 scores a thread: 8000 cycles).
template <int N>
__device__ __forceinline__ F2 capped2(F2 s, F2 mul, float cap) {
  constexpr float K4[4] = {0.99999946f, -0.33326318f, 0.13190297f, -0.044402229f};
  constexpr float K6[6] = {0.99999941f, -0.33329042f, 0.13281434f, -0.051605674f, 0.016743115f, -0.0030670604f};
  auto k = [&](int i) {
    const float c = (N == 4 ? K4[i] : K6[i]) * cap;
    return two(c, c);
  };
  const F2 x = mul2(s, mul), y = mul2(x, x);
  F2 r = fma2(y, k(N - 1), k(N - 2));
#pragma unroll
  for (int i = N - 3; i >= 0; --i) r = fma2(r, y, k(i));
  return mul2(r, x);
}

// Shared-memory operand of 128-byte rows under the 128-byte swizzle, eight rows 1024 bytes apart.
// `lead`: bytes between blocks of 64 elements along a row where rows are not the contraction's
// (values: [position][d], the contraction over positions); else unused.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Products of 128 x n with 32-bit sums; values: the second operand's rows are the contraction's.
__device__ __forceinline__ constexpr uint32_t product(bool bf16, int n, bool values) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((values ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(0), "r"(row), "r"(block)
      : "memory");
}

// Waits for a phase; false once a wait of the CTA has run out (every role then leaves).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > WAIT_LIMIT_NS) {
        *abort = 1;
        set_error(err, HS_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

// ---- the work
struct Request {      // of the call
  int req;            // -1: a bad one
  int first, n;       // its rows of the call
  int len, all;       // positions held before, positions that every token sees at least (the prefix's)
};
__device__ __forceinline__ Request request_of(const PagedAttendParams& p, int i, unsigned* err) {
  Request r = {-1, 0, 0, 0, 0};
  if (!p.tok_offsets) {
    r.first = i * p.tok_per_req;
    r.n = p.tok_per_req;
  } else {
    const int a = p.tok_offsets[i], b = p.tok_offsets[i + 1];
    if (a >= 0 && b >= a && b <= p.n_tok) {
      r.first = a;
      r.n = b - a;
    } else {
      *err |= HS_DEVERR_OFFSETS;
    }
  }
  const int req = p.req_ids ? p.req_ids[i] : i;
  if (req < 0 || req >= p.max_requests) {
    *err |= HS_DEVERR_REQ_RANGE;
    return r;
  }
  r.len = p.lengths[req];
  if (r.len < 0 || (long long)r.len + r.n > (long long)p.max_pages << p.page_shift) {
    *err |= HS_DEVERR_CAPACITY;
    return r;
  }
  r.req = req;
  if (p.prefix) r.all = max(0, min(p.prefix[req], r.len + r.n));
  return r;
}
template <typename C>
__device__ __forceinline__ int blocks_of(const PagedAttendParams& p, const Request& r) {
  return r.req < 0 ? 0 : (int)(((long long)r.n * p.group + C::ROWS - 1) / C::ROWS);
}
struct Block {
  int rows;           // of the block
  int lo, hi;         // positions that its rows see between them
  int start;          // the first tile's first position: on a page's (or a tile's) border
  int tiles;
};
template <typename C>
__device__ __forceinline__ Block block_of(const PagedAttendParams& p, const Request& r, int blk) {
  Block b;
  const int row0 = blk * C::ROWS;
  b.rows = min(C::ROWS, r.n * p.group - row0);
  b.hi = max(r.len + (row0 + b.rows - 1) / p.group + 1, r.all);
  b.lo = p.window > 0 ? max(0, r.len + row0 / p.group - p.window + 1) : 0;
  b.start = b.lo & ~(min(p.page_size, C::KT) - 1);
  b.tiles = (b.hi - b.start + C::KT - 1) / C::KT;
  return b;
}
// tiles that a tile of 128 rows takes part in: those from its last row's end on it leaves out
template <typename C>
__device__ __forceinline__ int tiles_of(const PagedAttendParams& p, const Request& r, const Block& b, int blk, int slot) {
  if (slot * 128 >= b.rows) return 0;
  const int last = blk * C::ROWS + min(b.rows, (slot + 1) * 128) - 1;
  const int hi = max(r.len + last / p.group + 1, r.all);
  return (hi - b.start + C::KT - 1) / C::KT;
}

// A CTA's share of the sequence of tiles, piece by piece.  Every role walks it by itself.
template <typename C>
struct Walk {
  const PagedAttendParams& p;
  int i, blk, head;
  long long left;               // cost that the share has left, from the segment's begin on
  int seg;                      // cost of a segment on top of its tiles
  int from, to;                 // tiles of the piece
  Request r;
  Block b;
  unsigned err = 0;
  __device__ Walk(const PagedAttendParams& p_, const int* begin, long long left_) : p(p_), left(left_), seg(begin[6]) {
    i = begin[0];
    blk = begin[1];
    head = begin[2];
    from = begin[3];
    to = 0;
    if (!begin[4]) {
      left = 0;
      return;
    }
    left += begin[5];
    r = request_of(p, i, &err);
    b = block_of<C>(p, r, blk);
    to = (int)min((long long)b.tiles, left - seg);
  }
  // whether there is a piece (empty ones are passed over)
  __device__ bool piece() {
    while (left > 0) {
      if (to > from) return true;
      next();
    }
    return false;
  }
  __device__ void next() {
    left -= b.tiles + seg;
    from = 0;
    if (left <= 0) return;
    if (++head == p.h_kv) {
      head = 0;
      ++blk;
      if (blk >= blocks_of<C>(p, r)) {
        blk = 0;
        do {
          if (++i >= p.n_req) {
            left = 0;
            return;
          }
          r = request_of(p, i, &err);
        } while (blocks_of<C>(p, r) == 0);
      }
      b = block_of<C>(p, r, blk);
    }
    to = (int)min((long long)b.tiles, left - seg);
  }
};

struct Chain {        // a segment that goes on in other CTAs
  int i, blk, head, last;     // last: -1: none
};

// where a CTA's pieces and its chain are in the workspace
template <typename C>
__host__ __device__ inline size_t ws_piece(int cta, int goes_on) { return (size_t)(cta * 2 + goes_on) * C::PIECE; }
template <typename C>
__host__ __device__ inline size_t ws_chain(int grid) { return (size_t)grid * 2 * C::PIECE; }

template <typename C>
__global__ void __launch_bounds__(C::THREADS, 1)
    paged_attend_kernel(const __grid_constant__ PagedAttendParams p, const __grid_constant__ CUtensorMap map) {
  constexpr int D = C::D, KT = C::KT, NQ = C::NQ;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  Meta& M = *reinterpret_cast<Meta*>(smem + C::SM_META);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&M.full[s], C::CONV ? 4 : 1);
      mbar_init(&M.empty[s], C::CONV ? 1 : 2);
      mbar_init(&M.ready[s], 1);
    }
    for (int s = 0; s < C::RAWS; ++s) {
      mbar_init(&M.raw_full[s], 1);
      mbar_init(&M.raw_empty[s], 4);
    }
    mbar_init(&M.q_full, C::Q_WARPS);
    mbar_init(&M.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&M.s_full[s], 1);
      mbar_init(&M.p_ready[0][s], 4);
      mbar_init(&M.p_ready[1][s], 4);
      mbar_init(&M.o_done[s], 1);
    }
    mbar_init(&M.drain, 1);
    fence_mbar_init();
    M.abort = 0;
    M.begin[4] = 0;
  }
  griddep_wait();
  griddep_launch_dependents();
  // (behind the wait: a kernel before this one may still want its columns)
  if (warp == 0) tmem_alloc(&M.tmem, C::TCOLS);

  // ---- the share: blocks before each request, then the cost of a thread's blocks, then the place of its begin
  long long share, mine;
  int seg, unsound;
  {
    int* pre = reinterpret_cast<int*>(smem + C::SM_RING);               // n_req + 1
    long long* part = reinterpret_cast<long long*>(smem);               // a sum per warp
    int* scan = reinterpret_cast<int*>(smem + 8 * C::WARPS);
    unsigned err = 0;
    const int per = (p.n_req + C::THREADS - 1) / C::THREADS;
    const int i0 = min(p.n_req, tid * per), i1 = min(p.n_req, i0 + per);
    int sum = 0, all;
    for (int i = i0; i < i1; ++i) sum += blocks_of<C>(p, request_of(p, i, &err));
    int at = block_exclusive_scan<C::THREADS>(sum, scan, &all);
    for (int i = i0; i < i1; ++i) {
      pre[i] = at;
      at += blocks_of<C>(p, request_of(p, i, &err));
    }
    if (tid == 0) pre[p.n_req] = all;
    if (err && blockIdx.x == 0) set_error(p.dev_error, err);
    unsound = __syncthreads_or(err != 0);
    if (unsound) {                               // offsets that decrease may let requests claim rows twice, without a bound
      long long rows = 0;
      for (int i = i0; i < i1; ++i) rows += request_of(p, i, &err).n;
#pragma unroll
      for (int o = 16; o; o >>= 1) rows += __shfl_xor_sync(FULL_MASK, rows, o);
      if (lane == 0) part[warp] = rows;
      __syncthreads();
      rows = 0;
      for (int t = 0; t < C::WARPS; ++t) rows += part[t];
      if (rows > p.n_tok) all = unsound = 0;     // nobody gets any (blocks may have left 32 bits)
      __syncthreads();
    }
    const int chunk = (all + C::THREADS - 1) / C::THREADS;
    const int b0 = min(all, tid * chunk), b1 = min(all, b0 + chunk);
    auto request_at = [&](int b) {               // the last request with pre <= b that has blocks
      int lo = 0, hi = p.n_req;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= b) lo = mid; else hi = mid;
      }
      return lo;
    };
    // f(request, its place, block) for the thread's blocks, until it returns false
    auto each = [&](auto f) {
      if (b0 >= b1) return;
      int i = request_at(b0);
      Request r = request_of(p, i, &err);
      for (int b = b0; b < b1; ++b) {
        if (b >= pre[i + 1]) {
          do ++i; while (pre[i + 1] <= b);
          r = request_of(p, i, &err);
        }
        if (!f(i, r, b - pre[i])) return;
      }
    };
    long long cost = 0;                          // tiles of the thread's blocks, for one head
    each([&](int, const Request& r, int blk) {
      cost += block_of<C>(p, r, blk).tiles;
      return true;
    });
    long long before = cost, total = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(FULL_MASK, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) part[warp] = before;
    __syncthreads();
    before -= cost;
#pragma unroll
    for (int t = 0; t < C::WARPS; ++t) {
      const long long x = part[t];
      if (t < warp) before += x;
      total += x;
    }
    // where a share is a few tiles, every CTA starts a segment anyway
    seg = (int)min((long long)C::SEGMENT_COST, total * p.h_kv / gridDim.x);
    total = (total + (long long)all * seg) * p.h_kv;
    before = (before + (long long)b0 * seg) * p.h_kv;
    cost = (cost + (long long)(b1 - b0) * seg) * p.h_kv;
    share = max((total + gridDim.x - 1) / gridDim.x, (long long)seg + 1);
    const long long x0 = min(total, blockIdx.x * share), x1 = min(total, x0 + share);
    mine = x1 - x0;
    if (tid == 0) M.begin[6] = seg;
    if (mine > 0 && x0 >= before && x0 < before + cost) {
      long long x = x0 - before;
      each([&](int i, const Request& r, int blk) {
        const int one = block_of<C>(p, r, blk).tiles + seg;
        if (x >= (long long)one * p.h_kv) {
          x -= (long long)one * p.h_kv;
          return true;
        }
        const int head = (int)(x / one), rest = (int)(x - (long long)head * one);
        M.begin[0] = i;
        M.begin[1] = blk;
        M.begin[2] = head;
        M.begin[3] = max(0, rest - seg);
        M.begin[5] = rest;
        M.begin[4] = 1;
        return false;
      });
    }
    fence_proxy_async_smem();                    // copies go where the tables were
    fence_before();
    __syncthreads();
    fence_after();
  }
  const uint32_t tmem = M.tmem;
  volatile int* abort = &M.abort;
  unsigned* err = p.dev_error;
  const uint32_t smem_s = smem_addr(smem), ring_s = smem_s + C::SM_RING;

  if (warp < C::SOFT) {
    // ================= softmax: a thread per row =================
    const int slot = NQ == 2 ? warp >> 2 : 0, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_o = lanes + C::T_O + slot * D;
    uint32_t used[2] = {0, 0}, tile_no = 0, piece_no = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL_MASK, wait_for(bar, parity, abort, err)); };
    Walk<C> w(p, M.begin, mine);
    Chain chain = {0, 0, 0, -1};
    auto run = [&] {
      for (; w.piece(); w.next(), ++piece_no) {
        const int tiles = w.to - w.from;
        const int count = max(0, min(w.to, tiles_of<C>(p, w.r, w.b, w.blk, slot)) - w.from);
        const bool whole = w.from == 0 && w.to == w.b.tiles;
        const bool mine_row = slot * 128 + row < w.b.rows;
        const int rr = w.blk * C::ROWS + min(slot * 128 + row, w.b.rows - 1);    // (rows behind the last: as the last)
        const int tok = rr / p.group, g = rr - tok * p.group, h = w.head * p.group + g;
        const int pos = w.r.len + tok;
        const int ahead = __reduce_min_sync(FULL_MASK, pos);       // the first position of the warp's rows
        const int hi = max(pos + 1, w.r.all), lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        const bool shaped = p.cap_in != 0.f || p.slopes;
        const float slope = p.slopes ? p.slopes[h] * LOG2_E : 0.f;   // to powers of two
        float mul = p.cap_in != 0.f ? p.cap_in : p.scale_log2;
        if (C::CONV) mul *= p.kv_scale[w.head] * (C::PAGES == PAGES_INT4 ? pa::INT4_SHIFT : 1.f);
        float m = -INFINITY, l = 0.f;
        // The product of tile j with the values is through.  (Where scores are made two tiles ahead, the one
        // before it may not be yet: tiles of odd and even number have a barrier each, whose phase before the
        // awaited one is over, as the scores of this tile were made behind that product.)
        auto sums = [&](int j, uint32_t tiles_since) {
          const int buf = NQ == 2 ? slot : j & 1;
          const bool ok = wait(&M.o_done[buf], (used[buf] - 1 - (NQ == 2 ? tiles_since : 0)) & 1);
          fence_after();
          return ok;
        };
        for (int j = 0; j < count; ++j) {
          const int buf = NQ == 2 ? slot : j & 1;
          if (!wait(&M.s_full[buf], used[buf] & 1)) return;
          ++used[buf];
          fence_after();
          if (C::CONV && j == 0) {
            const int e = M.q_exp[piece_no & 1][slot * 128 + row];
            mul *= exp2f((float)(e / 2)) * exp2f((float)(e - e / 2));
          }
          const uint32_t t_s = lanes + C::T_S + buf * KT;
          const int n0 = w.b.start + (w.from + j) * KT;
          const float to2 = shaped ? 1.f : mul;    // what makes powers of two of S
          const unsigned bad = M.bad[(tile_no + j) & 7];
          const bool part = __any_sync(FULL_MASK, lo > n0 || hi < n0 + KT) || bad;
          float top[2] = {-INFINITY, -INFINITY};
          // 64 scores from column c0 on: cap, bias, masks (what they become goes back to its place), the largest.
          auto shape = [&](auto capped, auto biased, auto masked, uint32_t (&s)[64], int c0) {
            auto S = [&](int c) -> float { return __uint_as_float(s[c]); };
            const int from = lo - n0 - c0, to = hi - n0 - c0;
            const unsigned off = bad >> (c0 / 16);
            auto unseen = [&](int c) { return c < from || c >= to || (off >> (c / 16) & 1); };
            if constexpr (decltype(capped)::value) {
              float most[2] = {0.f, 0.f};
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                if constexpr (decltype(masked)::value)     // (what hidden columns hold decides nothing)
                  most[c >> 1 & 1] = max3(most[c >> 1 & 1], unseen(c) ? 0.f : fabsf(S(c)), unseen(c + 1) ? 0.f : fabsf(S(c + 1)));
                else
                  most[c >> 1 & 1] = max3(most[c >> 1 & 1], fabsf(S(c)), fabsf(S(c + 1)));
              }
              // (votes of their own: a lane must not pass one over)
              const float far = fmaxf(most[0], most[1]) * fabsf(mul);
              const bool over_half = __any_sync(FULL_MASK, mine_row && !(far <= 0.5f));
              const bool over_one = __any_sync(FULL_MASK, mine_row && !(far <= 1.f));
              auto all = [&](auto n) {
                const F2 by = two(mul, mul);
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                  const float2 z = apart(capped2<decltype(n)::value>(two(S(c), S(c + 1)), by, p.cap_log2));
                  s[c] = __float_as_uint(z.x);
                  s[c + 1] = __float_as_uint(z.y);
                }
              };
              if (!over_half) {
                all(std::integral_constant<int, 4>{});
              } else if (!over_one) {
                all(std::integral_constant<int, 6>{});
              } else {
#pragma unroll 1
                for (int c = 0; c < 64; c += 8) {          // (few instructions: columns by way of their place)
                  uint32_t z[8];
                  tmem_load8(z, t_s + c0 + c);
                  tmem_wait_load<8>(z);
#pragma unroll
                  for (int e = 0; e < 8; ++e) z[e] = __float_as_uint(p.cap_log2 * pa::tanh32(__uint_as_float(z[e]) * mul));
                  tmem_store8(t_s + c0 + c, z);
                }
                tmem_wait_store();
                tmem_load32(s, t_s + c0);
                tmem_load32(s + 32, t_s + c0 + 32);
                tmem_wait_load<64>(s);
              }
            }
            if constexpr (decltype(biased)::value) {
              const float far = (float)(n0 + c0 - pos), by = decltype(capped)::value ? 1.f : mul;
              const F2 by2 = two(by, by);
              if (n0 + c0 + 63 <= ahead) {                 // nobody's position lies within: the distance has one sign
                const float from = slope * far;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                  const F2 b = two(fmaf(slope, (float)c, from), fmaf(slope, (float)(c + 1), from)), x = two(S(c), S(c + 1));
                  const float2 z = apart(decltype(capped)::value ? add2(x, b) : fma2(x, by2, b));
                  s[c] = __float_as_uint(z.x);
                  s[c + 1] = __float_as_uint(z.y);
                }
              } else
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                const float2 z = decltype(capped)::value ? make_float2(S(c), S(c + 1)) : apart(mul2(two(S(c), S(c + 1)), by2));
                s[c] = __float_as_uint(fmaf(-slope, fabsf(far + (float)c), z.x));
                s[c + 1] = __float_as_uint(fmaf(-slope, fabsf(far + (float)(c + 1)), z.y));
              }
            }
            if constexpr (decltype(masked)::value) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (unseen(c)) s[c] = 0xff800000u;
            }
            tmem_store32(t_s + c0, s);
            tmem_store32(t_s + c0 + 32, s + 32);
#pragma unroll
            for (int c = 0; c < 64; c += 2) top[c >> 1 & 1] = max3(top[c >> 1 & 1], S(c), S(c + 1));
          };
          // Twice over the scores, by loops: held in registers between, they would take code of thousands of
          // instructions, which warps of different phases then wait for
          uint32_t x[32], y[32];
          auto each = [&](auto capped, auto biased, auto masked) {
#pragma unroll 1
            for (int c = 0; c < KT; c += 64) {
              uint32_t s[64];
              tmem_load32(s, t_s + c);
              tmem_load32(s + 32, t_s + c + 32);
              tmem_wait_load<64>(s);
              shape(capped, biased, masked, s, c);
            }
            tmem_wait_store();
          };
          constexpr std::true_type yes{};
          constexpr std::false_type no{};
          if (shaped) {
            if (p.cap_in == 0.f) {
              if (part) each(no, yes, yes); else each(no, yes, no);
            } else if (p.slopes) {
              if (part) each(yes, yes, yes); else each(yes, yes, no);
            } else {
              if (part) each(yes, no, yes); else each(yes, no, no);
            }
          } else if (part) {
            each(no, no, yes);
          } else {
            constexpr int HELD = C::CONV ? 64 : KT;
#pragma unroll
            for (int c0 = 0; c0 < KT; c0 += HELD) {
              uint32_t s[HELD];
              float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < HELD; c += 32) tmem_load32(s + c, t_s + c0 + c);
              tmem_wait_load<HELD>(s);
#pragma unroll
              for (int c = 0; c < HELD; c += 2) t[c >> 1 & 3] = max3(t[c >> 1 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
              top[0] = max3(top[0], t[0], t[1]);
              top[1] = max3(top[1], t[2], t[3]);
            }
          }
          tmem_load32(x, t_s);
          const float mx = fmaxf(top[0], top[1]) * to2;
          if (__any_sync(FULL_MASK, mine_row && mx > m + SLACK)) {    // (a row behind the last may hold anything)
            const float n = fmaxf(m, mx);
            const float keep = pow2(m - (n == -INFINITY ? 0.f : n));
            m = n;
            l *= keep;
            if (j > 0) {                           // the sums so far, once the product before is through
              if (!sums(j - 1, 1)) return;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_load32(o, t_o + c);
                tmem_wait_load<32>(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_store32(t_o + c, o);
              }
            }
          }
          const float base = (m == -INFINITY ? 0.f : m) - (C::BF16 ? 0.f : FP16_SHIFT);
          F2 sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
          const F2 to2s = two(to2, to2), less = two(-base, -base);
          const uint32_t t_p = lanes + C::T_P + buf * C::P_STEP;
          auto weights = [&](uint32_t (&s)[32], int c0) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 z = apart(fma2(two(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), to2s, less));
              const float a = pow2(z.x), b = pow2(z.y);
              sum[c >> 1 & 1] = add2(sum[c >> 1 & 1], two(a, b));
              s[c / 2] = pa::pack2<C::BF16 ? HS_BF16 : HS_FP16>(a, b);
            }
            tmem_store16(t_p + c0 / 2, s);
            if (KT == 64 || c0 & 32) {             // a half of the tile: the product with the values starts on the first
              tmem_wait_store();
              fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&M.p_ready[KT == 64 ? c0 / 32 : c0 / 64][buf]);
            }
          };
#pragma unroll 1
          for (int c = 0; c < KT; c += 64) {
            tmem_wait_load<32>(x);
            tmem_load32(y, t_s + c + 32);
            weights(x, c);
            tmem_wait_load<32>(y);
            if (c + 64 < KT) tmem_load32(x, t_s + c + 64);
            weights(y, c + 32);
          }
          const float2 both = apart(add2(sum[0], sum[1]));
          l += both.x + both.y;
        }
        tile_no += tiles;
        // ---- the piece's rows
        if (count > 0 && !sums(count - 1, 0)) return;
        const float vs = C::CONV ? p.kv_scale[p.h_kv + w.head] * (C::PAGES == PAGES_INT4 ? pa::INT4_SHIFT : 1.f) : 1.f;
        const float inv = pa::inverse(l) * vs;
        const long long orow = (long long)(w.r.first + tok) * p.h_q + h;
        float* ws = p.ws + ws_piece<C>(blockIdx.x, w.from == 0);
        if (slot * 128 < w.b.rows) {
          // where an element of 32 is (4-bit pages: eight are in the order of their codes)
          auto column = [](int e) { return C::INT4 ? (e & ~7) + (e & 3) * 2 + (e >> 2 & 1) : e; };
          long long row4[4];                       // of the lane's four
#pragma unroll
          for (int k = 0; k < 4; ++k) row4[k] = __shfl_sync(FULL_MASK, mine_row ? orow : -1, (lane & ~3) + k);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (count > 0) {
              tmem_load32(o, t_o + c);
              tmem_wait_load<32>(o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (whole) {
              // four lanes hand each other 16-byte parts, so that together they store 64 bytes of a row (a lane
              // storing its own row touches 32 lines at a time)
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                y[e] = pa::pack2<C::QTYPE>(__uint_as_float(o[column(2 * e)]), __uint_as_float(o[column(2 * e + 1)]));
#pragma unroll
              for (int x = 1; x < 4; x <<= 1) {
                const bool up = lane & x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (k & x) continue;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    uint32_t& a = y[k * 4 + e];
                    uint32_t& b = y[(k | x) * 4 + e];
                    const uint32_t got = __shfl_xor_sync(FULL_MASK, up ? a : b, x);
                    if (up) a = got; else b = got;
                  }
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (row4[k] >= 0)
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row4[k] * D + c + (lane & 3) * 8) =
                      make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            } else {
              if (mine_row) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<uint4*>(ws + ((size_t)((c + e) / 4) * C::ROWS + slot * 128 + row) * 4) =
                      make_uint4(o[column(e)], o[column(e + 1)], o[column(e + 2)], o[column(e + 3)]);
              }
            }
          }
          if (mine_row) {
            if (whole) {
              if (p.lse) p.lse[orow] = pa::log_sum<C::BF16>(m, l);
            } else {
              ws[C::ROWS * D + slot * 128 + row] = m;
              ws[C::ROWS * D + C::ROWS + slot * 128 + row] = l;
            }
          }
        }
        if (w.from == 0 && !whole) {               // goes on in other CTAs: to the one with the segment's end
          const long long end = blockIdx.x * share + mine - w.left + w.b.tiles + seg - 1;
          chain = Chain{w.i, w.blk, w.head, (int)(end / share)};
        }
        fence_before();                            // (these reads before what the next piece's products write)
      }
    };
    run();
    if (tid == 0) reinterpret_cast<Chain*>(p.ws + ws_chain<C>(gridDim.x))[blockIdx.x] = chain;
  } else {
    if (warp == C::W_MMA) {
      // ================= products =================
      auto run = [&] {
        constexpr uint32_t qk = product(C::BF16, KT, false), pv = product(C::BF16, D, true);
        const uint32_t one = elect();
        uint32_t stage = 0, phase = 0, p_used[2] = {0, 0}, q_no = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          const bool ok = __all_sync(FULL_MASK, wait_for(bar, parity, abort, err));
          fence_after();
          return ok;
        };
        // stages come keys, values, keys, values ...: the k-th ahead of the current one
        auto at = [&](uint32_t ahead, uint32_t* ph) {
          uint32_t s = stage + ahead;
          *ph = phase;
          if (s >= C::STAGES) {
            s -= C::STAGES;
            *ph ^= 1;
          }
          return s;
        };
        auto keys = [&](int s, int tile_slot, int buf) {     // S = Q K^T
          const uint64_t q = operand(smem_s + tile_slot * C::QB, 16), k = operand(ring_s + s * C::STAGE, 16);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            mma_ss(tmem + C::T_S + buf * KT, q + (((c / 4) * (128 * 128) + (c % 4) * 32) >> 4),
                   k + (((c / 4) * (KT * 128) + (c % 4) * 32) >> 4), qk, c > 0, one);
          mma_commit(&M.s_full[buf], one);
        };
        auto values = [&](int s, int tile_slot, int buf, bool add) {   // O += P V
          const uint64_t v = operand(ring_s + s * C::STAGE, KT * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(&M.p_ready[h][buf], p_used[buf] & 1)) return false;
#pragma unroll
            for (int c = h * (KT / 32); c < (h + 1) * (KT / 32); ++c)
              mma_ts(tmem + C::T_O + tile_slot * D, tmem + C::T_P + buf * C::P_STEP + c * 8, v + (c * 2048 >> 4), pv, add || c > 0, one);
          }
          ++p_used[buf];
          mma_commit(&M.o_done[buf], one);
          return true;
        };
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next(), ++q_no) {
          const int tiles = w.to - w.from;
          int count[NQ];
#pragma unroll
          for (int s = 0; s < NQ; ++s) count[s] = max(0, min(w.to, tiles_of<C>(p, w.r, w.b, w.blk, s)) - w.from);
          if (!wait(&M.q_full, q_no & 1)) return;
          uint32_t ph;
          constexpr int AHEAD = NQ == 2 ? 1 : 2;              // tiles whose scores are made before their turn
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) {
            if (j >= tiles) break;
            const uint32_t s = at(2 * j, &ph);
            if (!wait(&M.full[s], ph)) return;
#pragma unroll
            for (int x = 0; x < NQ; ++x)
              if (j < count[x]) keys(s, x, NQ == 2 ? x : j);
            mma_commit(&M.empty[s], one);
            if (j == tiles - 1) mma_commit(&M.q_empty, one);
          }
          for (int j = 0; j < tiles; ++j) {
            const uint32_t v = at(1, &ph);
            if (!wait(C::CONV ? &M.full[v] : &M.ready[v], ph)) return;
            const bool more = j + AHEAD < tiles;
            bool have = false;
            uint32_t kph;
            const uint32_t k = at(2 * AHEAD, &kph);
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
              if (j >= count[x]) continue;
              const int buf = NQ == 2 ? x : j & 1;
              if (!values(v, x, buf, j > 0)) return;
              if (more && j + AHEAD < count[x]) {
                if (!have && !wait(&M.full[k], kph)) return;
                have = true;
                keys(k, x, buf);
              }
            }
            mma_commit(&M.empty[v], one);
            if (more) {
              if (!have && !wait(&M.full[k], kph)) return;
              mma_commit(&M.empty[k], one);
              if (j + AHEAD == tiles - 1) mma_commit(&M.q_empty, one);
            }
            stage += 2;
            if (stage >= C::STAGES) {
              stage -= C::STAGES;
              phase ^= 1;
            }
          }
        }
      };
      run();
      mma_commit(&M.drain, elect());                 // every product is through before TMEM is freed
      mbar_wait_bounded(&M.drain, 0);
    } else if (warp == C::W_LOAD) {
      // ================= pages, by TMA: into the ring, or to be turned into fp16 on the way there =================
      constexpr int PLACES = C::CONV ? C::RAWS : C::STAGES;
      uint64_t* full = C::CONV ? M.raw_full : M.full;
      uint64_t* empty = C::CONV ? M.raw_empty : M.empty;
      uint32_t stage = 0, phase = 0, tile_no = 0, copied = 0;
      auto run = [&] {
        Walk<C> w(p, M.begin, mine);
        // a lane's copy: rows of one page (and block of 64 elements), or a unit of 16
        const int rows = C::CONV ? PG_UNIT : min(p.page_size, KT), boxes = KT / rows * (C::CONV ? 1 : C::BLK);
        for (; w.piece(); w.next()) {
          const int32_t* table = p.page_table + (long long)w.r.req * p.max_pages;
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            const int n0 = w.b.start + j * KT;
            const int u = C::CONV ? lane : lane / C::BLK, n = n0 + u * rows;
            const bool want = lane < boxes && n < w.b.hi;
            const int page = want ? table[n >> p.page_shift] : 0;
            const bool off = want && (page < 0 || page >= p.n_pages);
            // the bad units, of 16 positions
            const unsigned bits = __reduce_or_sync(FULL_MASK, off ? ((1u << (rows / 16)) - 1) << (u * (rows / 16)) : 0u);
            if (lane == 0) {
              if (bits) set_error(err, HS_DEVERR_PAGE);
              M.bad[tile_no & 7] = (unsigned char)bits;
            }
            const bool copy = want && !off;
            const int in_page = n & (p.page_size - 1);
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll
              for (int part = 0; part < C::PARTS; ++part) {
                const bool now = copy && (C::PARTS == 1 || u / (C::RAW_ROWS / 16) == part);
                const int copies = __popc(__ballot_sync(FULL_MASK, now));
                if (!__all_sync(FULL_MASK, wait_for(&empty[stage], phase ^ 1, abort, err))) return;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], copies * (C::CONV ? C::UNIT_BYTES : rows * 128));
                __syncwarp();
                if (now) {
                  const int row = ((page * 2 + which) * p.h_kv + w.head) * p.page_size + in_page;
                  if constexpr (C::CONV)
                    bulk_g2s(smem + C::SM_RAW + stage * C::RAW + u % (C::RAW_ROWS / 16) * C::UNIT_BYTES,
                             p.pages + (long long)(row >> 4) * C::UNIT_BYTES, C::UNIT_BYTES, &full[stage]);
                  else
                    tma_rows(ring_s + stage * C::STAGE + (lane % C::BLK) * (KT * 128) + u * rows * 128, &map, row, lane % C::BLK,
                             &full[stage]);
                }
                ++copied;
                if (++stage == PLACES) {
                  stage = 0;
                  phase ^= 1;
                }
              }
          }
        }
      };
      run();
      if (*abort)                                  // copies in flight land before the shared memory goes
        for (uint32_t k = copied < PLACES ? 0 : copied - PLACES; k < copied; ++k)
          mbar_wait_bounded(&full[k % PLACES], (k / PLACES) & 1);
    } else if (warp == C::W_FIX && !C::CONV) {
      // ================= values of positions that no row sees become 0 =================
      auto run = [&] {
        uint32_t stage = 0, phase = 0, tile_no = 0;
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next())
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            // Every stage is waited for here, in order, and refilled once this warp has passed it too, so that no
            // wait is for a phase behind the next (copies land in any order) or before the last
            if (!__all_sync(FULL_MASK, wait_for(&M.full[stage], phase, abort, err))) return;
            if (lane == 0) {
              mbar_arrive(&M.ready[stage]);
              mbar_arrive(&M.empty[stage]);
            }
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
            if (!__all_sync(FULL_MASK, wait_for(&M.full[stage], phase, abort, err))) return;
            const int n0 = w.b.start + j * KT;
            const unsigned bad = M.bad[tile_no & 7];
            if (n0 < w.b.lo || n0 + KT > w.b.hi || bad) {
              unsigned char* v = smem + C::SM_RING + stage * C::STAGE;
              for (int e = lane; e < KT * C::BLK * 8; e += 32) {
                const int r = (e >> 3) % KT, n = n0 + r;
                if (n < w.b.lo || n >= w.b.hi || (bad >> (r / 16) & 1)) *reinterpret_cast<int4*>(v + e * 16) = make_int4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) {
              mbar_arrive(&M.ready[stage]);
              mbar_arrive(&M.empty[stage]);
            }
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
      };
      run();
    } else if (warp >= C::Q0 && warp <= C::W_Q) {
      // ================= queries =================
      auto run = [&] {
        uint32_t no = 0;
        constexpr int PER = D / 8, TOGETHER = 32 / PER;       // 16-byte parts of a row, rows at a time
        constexpr int STEP = TOGETHER * C::Q_WARPS;
        const int c = lane % PER, r0 = (warp - C::Q0) * TOGETHER + lane / PER;
        unsigned char* to = smem + (c / 8) * (128 * 128);
        auto dst_of = [&](int r) { return to + (r / 128) * C::QB + (r % 128) * 128 + (((c % 8) ^ (r & 7)) << 4); };
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next(), ++no) {
          if (!__all_sync(FULL_MASK, wait_for(&M.q_empty, (no & 1) ^ 1, abort, err))) return;
          const int row0 = w.blk * C::ROWS;
          const uint16_t* q = static_cast<const uint16_t*>(p.q) + (long long)w.r.first * p.q_ts + (long long)w.head * p.group * p.q_hs + c * 8;
          // rows of a block from its first token on: below 2^13, so a product in 32 bits divides them
          const int tok0 = row0 / p.group, g0 = row0 - tok0 * p.group;
          const float one = 1.0f / p.group;
          q += tok0 * p.q_ts;
#pragma unroll 8
          for (int r = r0; r < w.b.rows; r += STEP) {
            const int tok = (int)(((float)(g0 + r) + 0.5f) * one), g = g0 + r - tok * p.group;
            cp_async_16(dst_of(r), q + tok * p.q_ts + g * p.q_hs);
          }
          cp_async_wait_all();
          if constexpr (C::CONV) {
            // 16 bits of another range become fp16: a row under a power of two that brings its largest into [1, 2)
#pragma unroll 4
            for (int rb = (warp - C::Q0) * TOGETHER; rb < w.b.rows; rb += STEP) {
              const int r = rb + lane / PER;
              const bool in = r < w.b.rows;
              if constexpr (C::QTYPE == HS_BF16) {
                uint4* at = reinterpret_cast<uint4*>(dst_of(in ? r : 0));
                const uint4 u = in ? *at : make_uint4(0, 0, 0, 0);
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
                // the largest of a row as whole numbers: bits without a sign order as values do (a NaN above all)
                uint32_t mx = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, uw[e] & 0x7fff7fffu);
#pragma unroll
                for (int o = PER / 2; o; o >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(FULL_MASK, mx, o));
                const int bits = max(mx & 0xffff, mx >> 16), field = bits >> 7;     // exponent of bf16
                const int e2 = field == 0 || field == 255 ? 0 : max(-126, min(126, field - 127));
                const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[2 * e] = bf16lo(uw[e]);
                  x[2 * e + 1] = bf16hi(uw[e]);
                }
                if (in) {
                  // (4-bit pages: elements of eight in the order in which their codes are turned)
                  auto pair = [&](int i) {
                    const int e = C::INT4 ? i : 2 * i, f = C::INT4 ? i + 4 : 2 * i + 1;
                    return pa::pack2<HS_FP16>(x[e] * down, x[f] * down);
                  };
                  *at = make_uint4(pair(0), pair(1), pair(2), pair(3));
                  if (c == 0) M.q_exp[no & 1][r] = (signed char)e2;
                }
              } else if (in) {
                if constexpr (C::INT4) {
                  uint4* at = reinterpret_cast<uint4*>(dst_of(r));
                  const uint4 u = *at;
                  *at = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                                   __byte_perm(u.y, u.w, 0x7632));
                }
                if (c == 0) M.q_exp[no & 1][r] = 0;
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.q_full);
        }
      };
      run();
    } else if (C::CONV && warp >= C::W_CONV) {
      // ================= 8-bit and 4-bit pages, turned into fp16 =================
      auto run = [&] {
        uint32_t stage = 0, phase = 0, place = 0, place_phase = 0, tile_no = 0;
        const int ct = tid - 32 * C::W_CONV;
        constexpr int EL = C::INT4 ? 32 : 16;                      // elements of 16 bytes of codes
        constexpr int PER = D / EL, STEP = 128 / PER, N = C::RAW_ROWS / STEP;   // parts of a row, rows at a time, parts of a thread
        const int part = ct % PER, r0 = ct / PER;
        // where the thread's rows go: the swizzle of their 16-byte pieces is the same for all of them
        static_assert(STEP % 8 == 0, "");
        unsigned char* const to0 = smem + C::SM_RING + part * EL / 64 * (KT * 128) + r0 * 128;
        const int piece0 = part * EL / 8 % 8, sw = r0 & 7;
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next())
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            const int n0 = w.b.start + j * KT;
#pragma unroll 1
            for (int step = 0; step < 2 * C::PARTS; ++step) {
              const int which = step / C::PARTS, half = step % C::PARTS;
              if (half == 0 && !__all_sync(FULL_MASK, wait_for(&M.empty[stage], phase ^ 1, abort, err))) return;
              if (!__all_sync(FULL_MASK, wait_for(&M.raw_full[place], place_phase, abort, err))) return;
              const unsigned bad = M.bad[tile_no & 7];
              const bool all = n0 >= w.b.lo && n0 + KT <= w.b.hi && !bad;
              const unsigned char* from = smem + C::SM_RAW + place * C::RAW;
              unsigned char* to = to0 + stage * C::STAGE + half * (C::RAW_ROWS * 128);
              // of 4-bit rows: where the thread's codes and scales are in a unit
              const int code_row = which ? 16 : D / 2, code0 = which ? part * 256 : part * 16;
              const int scale_row = which ? 1 : D / 16, scale0 = 8 * D + (which ? part * 32 : part * 2), scale_step = which ? 16 : 1;
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const int q = r0 + i * STEP, n = n0 + half * C::RAW_ROWS + q;
                // (rows that no token sees hold anything: they become 0)
                const bool seen = all || (n >= w.b.lo && n < w.b.hi && !(bad >> ((n - n0) / 16) & 1));
                auto put = [&](int k, uint4 v) {    // the k-th eight elements
                  *reinterpret_cast<uint4*>(to + i * (STEP * 128) + (((piece0 + k) ^ sw) << 4)) = v;
                };
                if constexpr (!C::INT4) {
                  const uint4 u = seen ? *reinterpret_cast<const uint4*>(from + q * D + part * 16) : make_uint4(0, 0, 0, 0);
                  uint4 v;
                  pa::e4m3x4_to_half2(u.x, v.x, v.y);
                  pa::e4m3x4_to_half2(u.y, v.z, v.w);
                  put(0, v);
                  pa::e4m3x4_to_half2(u.z, v.x, v.y);
                  pa::e4m3x4_to_half2(u.w, v.z, v.w);
                  put(1, v);
                } else {
                  const unsigned char* unit = from + (q / 16) * (9 * D);
                  const uint4 u = *reinterpret_cast<const uint4*>(unit + code0 + q % 16 * code_row);
                  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
                  const unsigned char* at = unit + scale0 + q % 16 * scale_row;
                  const uint32_t two = pa::e4m3x2_to_half2((uint16_t)(seen ? at[0] | (unsigned)at[scale_step] << 8 : 0));
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const pa::Int4Scale s4 = pa::int4_scale(__byte_perm(two, 0, h ? 0x3232 : 0x1010));
#pragma unroll
                    for (int k = 2 * h; k < 2 * h + 2; ++k) {
                      uint32_t a[4];                // elements (0, 4), (1, 5), (2, 6), (3, 7) of eight: they stay so, as
                      pa::int4x8_to_half2(x[k], s4, a);   // queries come, and outputs leave, in that order
                      put(k, make_uint4(a[0], a[1], a[2], a[3]));
                    }
                  }
                }
              }
              if (half == C::PARTS - 1) fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&M.raw_empty[place]);
                if (half == C::PARTS - 1) mbar_arrive(&M.full[stage]);
              }
              if (++place == C::RAWS) {
                place = 0;
                place_phase ^= 1;
              }
              if (half == C::PARTS - 1 && ++stage == C::STAGES) {
                stage = 0;
                phase ^= 1;
              }
            }
          }
      };
      run();
    }
  }

  // ---- rows of bad requests
  for (int i = unsound ? blockIdx.x : p.n_req; i < p.n_req; i += gridDim.x) {
    unsigned e = 0;
    const Request r = request_of(p, i, &e);
    if (r.req >= 0 || r.n == 0) continue;
    const long long n = (long long)r.n * p.h_q;
    for (long long x = tid; x < n * (D / 8); x += C::THREADS)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (long long)r.first * p.h_q * D + x * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (long long x = tid; x < n; x += C::THREADS) p.lse[(long long)r.first * p.h_q + x] = -INFINITY;
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_free(tmem, C::TCOLS);
}

// Joins the pieces of the segment that starts in CTA blockIdx.x and goes on behind it: 32 rows
// and 32 elements a block, a lane per row; a warp takes every eighth piece, and the warps' sums
// are added in a fixed order.
constexpr int JOIN_WARPS = 8;
template <typename C>
__global__ void __launch_bounds__(32 * JOIN_WARPS) paged_attend_join_kernel(const __grid_constant__ PagedAttendParams p) {
  __shared__ float4 s_o[JOIN_WARPS][8][32];
  __shared__ float s_m[JOIN_WARPS][32], s_l[JOIN_WARPS][32];
  griddep_wait();
  griddep_launch_dependents();
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Chain ch = reinterpret_cast<const Chain*>(p.ws + ws_chain<C>(p.grid))[cta];
  if (ch.last < 0) return;
  unsigned err = 0;
  const Request r = request_of(p, ch.i, &err);
  const Block b = block_of<C>(p, r, ch.blk);
  const int row = blockIdx.y * 32 + lane;
  if ((int)blockIdx.y * 32 >= b.rows) return;
  const bool in = row < b.rows;
  const int n = ch.last - cta + 1, c0 = blockIdx.z * 8;
  // all pieces' references first, so that the sums behind them wait for nothing but their own reads
  auto piece = [&](int j) { return p.ws + ws_piece<C>(cta + j, j == 0); };
  float m = -INFINITY;
#pragma unroll 4
  for (int j = warp; j < n; j += JOIN_WARPS) m = fmaxf(m, in ? piece(j)[C::ROWS * C::D + row] : -INFINITY);
  s_m[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < JOIN_WARPS; ++k) m = fmaxf(m, s_m[k][lane]);
  const float mm = m, base = mm == -INFINITY ? 0.f : mm;
  float l = 0.f;
  float4 acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int j = warp; j < n; j += JOIN_WARPS) {
    const float* at = piece(j);
    float4 x[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      x[c] = in ? *reinterpret_cast<const float4*>(at + ((size_t)(c0 + c) * C::ROWS + row) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float w = in ? exp2f(at[C::ROWS * C::D + row] - base) : 0.f;
    l += in ? w * at[C::ROWS * C::D + C::ROWS + row] : 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      acc[c].x += x[c].x * w;
      acc[c].y += x[c].y * w;
      acc[c].z += x[c].z * w;
      acc[c].w += x[c].w * w;
    }
  }
  s_l[warp][lane] = l;
#pragma unroll
  for (int c = 0; c < 8; ++c) s_o[warp][c][lane] = acc[c];
  __syncthreads();
  float ll = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < JOIN_WARPS; ++k) {
    const float4 x = s_o[k][warp][lane];
    ll += s_l[k][lane];
    o.x += x.x;
    o.y += x.y;
    o.z += x.z;
    o.w += x.w;
  }
  if (!in) return;
  const int rr = ch.blk * C::ROWS + row, tok = rr / p.group, h = ch.head * p.group + rr - tok * p.group;
  const float vs = C::CONV ? p.kv_scale[p.h_kv + ch.head] * (C::PAGES == PAGES_INT4 ? pa::INT4_SHIFT : 1.f) : 1.f;
  const float inv = pa::inverse(ll) * vs;
  const long long orow = (long long)(r.first + tok) * p.h_q + h;
  pa::store_out4<C::QTYPE>(p.out, orow * C::D + (c0 + warp) * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (p.lse && warp == 0 && c0 == 0) p.lse[orow] = pa::log_sum<C::BF16>(mm, ll);
}

template <typename C>
struct Kernels {
  static cudaError_t prepare() {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, paged_attend_join_kernel<C>);
    if (e != cudaSuccess) return e;
    return allow_smem(paged_attend_kernel<C>, C::SMEM);
  }
  static cudaError_t launch(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st) {
    const cudaError_t e = launch_pdl(paged_attend_kernel<C>, dim3(p.grid), dim3(C::THREADS), C::SMEM, st, p, map);
    if (e != cudaSuccess) return e;
    const int rows = (int)std::min<long long>(C::ROWS, (long long)p.n_tok * p.group);    // of a block, at most
    return launch_pdl(paged_attend_join_kernel<C>, dim3(p.grid, (rows + 31) / 32, C::D / 32), dim3(32 * JOIN_WARPS), 0, st, p);
  }
};

// The kernels of one head width are compiled together (hs_paged_attend_*.cu).
template <int D>
cudaError_t paged_attend_of(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st);
template <int D>
cudaError_t prepare_attend_of(int type, int page_type);
template <int D, typename F>
cudaError_t by_kind(int type, int page_type, F f) {
  const Pages k = pages_kind(page_type);
  if (type == HS_BF16)
    return k == PAGES_INT4   ? f(Kernels<Cfg<D, HS_BF16, PAGES_INT4>>{})
           : k == PAGES_E4M3 ? f(Kernels<Cfg<D, HS_BF16, PAGES_E4M3>>{})
                             : f(Kernels<Cfg<D, HS_BF16, PAGES_SAME>>{});
  return k == PAGES_INT4   ? f(Kernels<Cfg<D, HS_FP16, PAGES_INT4>>{})
         : k == PAGES_E4M3 ? f(Kernels<Cfg<D, HS_FP16, PAGES_E4M3>>{})
                           : f(Kernels<Cfg<D, HS_FP16, PAGES_SAME>>{});
}
#define HS_PAGED_ATTEND_OF(D)                                                                               \
  template <>                                                                                               \
  cudaError_t paged_attend_of<D>(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st) {     \
    return by_kind<D>(p.type, p.page_type, [&](auto k) { return k.launch(p, map, st); });                   \
  }                                                                                                         \
  template <>                                                                                               \
  cudaError_t prepare_attend_of<D>(int type, int page_type) {                                               \
    return by_kind<D>(type, page_type, [](auto k) { return k.prepare(); });                                 \
  }

}  // namespace pt
}  // namespace hs

#endif  // HS_PAGED_ATTEND_CUH_
