// Attention of many new tokens per request over its paged cache (hs_paged_attend).
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
  static constexpr int STAGES = D == 64 ? 8 : 5;
  static constexpr int SOFT = 4 * NQ;                          // softmax warps
  static constexpr int W_MMA = SOFT, W_LOAD = SOFT + 1, W_FIX = SOFT + 2, W_Q = SOFT + 3, W_CONV = SOFT + 4;
  static constexpr int WARPS = SOFT + 4 + (CONV ? 4 : 0);
  static constexpr int THREADS = 32 * WARPS;
  // registers of a thread at launch, of the softmax warps, of the others: the shares add up to the launch's
  static constexpr int REGS_SOFT = NQ == 1 ? 0 : CONV ? 168 : 208;
  static constexpr int REGS_REST = NQ == 1 ? 0 : 88;
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
  static constexpr int SM_META = SM_RING + STAGES * STAGE;
  static constexpr size_t SMEM = 1024 + SM_META + sizeof(int) * 256;
  static constexpr int PIECE = ROWS * D + 2 * ROWS;            // floats of a piece: o [d / 4][row][4], m, l
  static constexpr int SEGMENT_COST = 2;                       // of a segment on top of its tiles, in tiles
};

struct Meta {
  uint64_t full[8], empty[8], vok[8];
  uint64_t q_full, q_empty, s_full[2], p_ready[2], o_done[2], drain;
  uint32_t tmem;
  int abort;
  int begin[6];                  // place of the share's first tile: request, block, head, tile; 1: there is one
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
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

template <int A>
__device__ __forceinline__ void setmaxnreg() {   // (to A registers: whether that is more or fewer, the caller knows)
  if constexpr (A >= 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(A));
  else if constexpr (A > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(A));
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
  int from, to;                 // tiles of the piece
  Request r;
  Block b;
  unsigned err = 0;
  __device__ Walk(const PagedAttendParams& p_, const int* begin, long long left_) : p(p_), left(left_) {
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
    to = (int)min((long long)b.tiles, left - C::SEGMENT_COST);
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
    left -= b.tiles + C::SEGMENT_COST;
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
    to = (int)min((long long)b.tiles, left - C::SEGMENT_COST);
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
      mbar_init(&M.empty[s], 1);
      mbar_init(&M.vok[s], 1);
    }
    mbar_init(&M.q_full, 1);
    mbar_init(&M.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&M.s_full[s], 1);
      mbar_init(&M.p_ready[s], 4);
      mbar_init(&M.o_done[s], 1);
    }
    mbar_init(&M.drain, 1);
    fence_mbar_init();
    M.abort = 0;
    M.begin[4] = 0;
  }
  if (warp == 0) tmem_alloc(&M.tmem, C::TCOLS);
  griddep_wait();
  griddep_launch_dependents();

  // ---- the share: blocks before each request, then the cost of a thread's blocks, then the place of its begin
  long long share, mine;
  {
    int* pre = reinterpret_cast<int*>(smem + C::SM_RING);               // n_req + 1
    long long* part = reinterpret_cast<long long*>(smem);               // a sum per thread
    int* scan = reinterpret_cast<int*>(smem + 8 * C::THREADS);
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
    __syncthreads();
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
    long long cost = 0;
    each([&](int, const Request& r, int blk) {
      cost += (long long)(block_of<C>(p, r, blk).tiles + C::SEGMENT_COST) * p.h_kv;
      return true;
    });
    part[tid] = cost;
    __syncthreads();
    long long before = 0, total = 0;
    for (int t = 0; t < C::THREADS; ++t) {
      const long long x = part[t];
      if (t < tid) before += x;
      total += x;
    }
    share = (total + gridDim.x - 1) / gridDim.x;
    if (share < C::SEGMENT_COST + 1) share = C::SEGMENT_COST + 1;
    const long long x0 = min(total, blockIdx.x * share), x1 = min(total, x0 + share);
    mine = x1 - x0;
    if (mine > 0 && x0 >= before && x0 < before + cost) {
      long long x = x0 - before;
      each([&](int i, const Request& r, int blk) {
        const int one = block_of<C>(p, r, blk).tiles + C::SEGMENT_COST;
        if (x >= (long long)one * p.h_kv) {
          x -= (long long)one * p.h_kv;
          return true;
        }
        const int head = (int)(x / one), rest = (int)(x - (long long)head * one);
        M.begin[0] = i;
        M.begin[1] = blk;
        M.begin[2] = head;
        M.begin[3] = max(0, rest - C::SEGMENT_COST);
        M.begin[5] = rest;                       // cost of the segment before the share
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
    setmaxnreg<C::REGS_SOFT>();
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
        const int hi = max(pos + 1, w.r.all), lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        const bool shaped = p.cap_in != 0.f || p.slopes;
        const float slope = p.slopes ? p.slopes[h] * LOG2_E : 0.f;
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
          uint32_t s[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 32) tmem_load32(s + c, t_s + c);
          tmem_wait_load(s);
          auto S = [&](int c) { return __uint_as_float(s[c]); };
          const int n0 = w.b.start + (w.from + j) * KT;
          float to2 = mul;                        // what makes powers of two of S
          if (shaped) {
            to2 = 1.f;
            if (p.cap_in != 0.f) {
#pragma unroll
              for (int c = 0; c < KT; ++c) s[c] = __float_as_uint(p.cap_log2 * pa::tanh32(S(c) * mul));
            } else {
#pragma unroll
              for (int c = 0; c < KT; ++c) s[c] = __float_as_uint(S(c) * mul);
            }
            if (p.slopes) {
              const float far = (float)(n0 - pos);
#pragma unroll
              for (int c = 0; c < KT; ++c) s[c] = __float_as_uint(fmaf(-slope, fabsf(far + (float)c), S(c)));
            }
          }
          const unsigned bad = M.bad[(tile_no + j) & 7];
          if (__any_sync(FULL_MASK, lo > n0 || hi < n0 + KT) || bad) {
            const int c0 = lo - n0, c1 = hi - n0;
#pragma unroll
            for (int c = 0; c < KT; ++c)
              if (c < c0 || c >= c1 || (bad >> (c / 16) & 1)) s[c] = 0xff800000u;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < KT; ++c) top[c & 3] = fmaxf(top[c & 3], S(c));
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * to2;
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
                tmem_wait_load(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_store32(t_o + c, o);
              }
            }
          }
          const float base = (m == -INFINITY ? 0.f : m) - (C::BF16 ? 0.f : FP16_SHIFT);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < KT; c += 2) {
            const float a = pow2(fmaf(S(c), to2, -base)), b = pow2(fmaf(S(c + 1), to2, -base));
            sum[c & 2] += a;
            sum[(c & 2) + 1] += b;
            s[c / 2] = pa::pack2<C::BF16 ? HS_BF16 : HS_FP16>(a, b);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
          for (int c = 0; c < KT / 2; c += 32) tmem_store32(lanes + C::T_P + buf * C::P_STEP + c, s + c);
          tmem_wait_store();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.p_ready[buf]);
        }
        tile_no += tiles;
        // ---- the piece's rows
        if (count > 0 && !sums(count - 1, 0)) return;
        const float vs = C::CONV ? p.kv_scale[p.h_kv + w.head] * (C::PAGES == PAGES_INT4 ? pa::INT4_SHIFT : 1.f) : 1.f;
        const float inv = pa::inverse(l) * vs;
        const long long orow = (long long)(w.r.first + tok) * p.h_q + h;
        float* ws = p.ws + ws_piece<C>(blockIdx.x, w.from == 0);
        if (slot * 128 < w.b.rows) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (count > 0) {
              tmem_load32(o, t_o + c);
              tmem_wait_load(o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (mine_row) {
              if (whole) {
                uint16_t* dst = static_cast<uint16_t*>(p.out) + orow * D + c;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  uint4 v;
                  v.x = pa::pack2<C::QTYPE>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                  v.y = pa::pack2<C::QTYPE>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                  v.z = pa::pack2<C::QTYPE>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                  v.w = pa::pack2<C::QTYPE>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                  *reinterpret_cast<uint4*>(dst + e) = v;
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<uint4*>(ws + ((size_t)((c + e) / 4) * C::ROWS + slot * 128 + row) * 4) =
                      make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
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
          const long long end = blockIdx.x * share + mine - w.left + w.b.tiles + C::SEGMENT_COST - 1;
          chain = Chain{w.i, w.blk, w.head, (int)(end / share)};
        }
        fence_before();                            // (these reads before what the next piece's products write)
      }
    };
    run();
    if (tid == 0) reinterpret_cast<Chain*>(p.ws + ws_chain<C>(gridDim.x))[blockIdx.x] = chain;
  } else {
    setmaxnreg<C::REGS_REST>();
    if (warp == C::W_MMA) {
      // ================= products: one thread =================
      auto run = [&] {
        const uint32_t qk = product(C::BF16, KT, false), pv = product(C::BF16, D, true);
        uint32_t stage = 0, phase = 0, p_used[2] = {0, 0}, q_no = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          const bool ok = wait_for(bar, parity, abort, err);
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
          const uint32_t q = smem_s + tile_slot * C::QB, k = ring_s + s * C::STAGE;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            mma_ss(tmem + C::T_S + buf * KT, operand(q + (c / 4) * (128 * 128) + (c % 4) * 32, 16),
                   operand(k + (c / 4) * (KT * 128) + (c % 4) * 32, 16), qk, c > 0);
          mma_commit(&M.s_full[buf]);
        };
        auto values = [&](int s, int tile_slot, int buf, bool add) {   // O += P V
          const uint32_t v = ring_s + s * C::STAGE;
#pragma unroll
          for (int c = 0; c < KT / 16; ++c)
            mma_ts(tmem + C::T_O + tile_slot * D, tmem + C::T_P + buf * C::P_STEP + c * 8, operand(v + c * 2048, KT * 128), pv, add || c > 0);
          mma_commit(&M.o_done[buf]);
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
            mma_commit(&M.empty[s]);
            if (j == tiles - 1) mma_commit(&M.q_empty);
          }
          for (int j = 0; j < tiles; ++j) {
            const uint32_t v = at(1, &ph);
            if (!wait(C::CONV ? &M.full[v] : &M.vok[v], ph)) return;
            const bool more = j + AHEAD < tiles;
            bool have = false;
            uint32_t kph;
            const uint32_t k = at(2 * AHEAD, &kph);
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
              if (j >= count[x]) continue;
              const int buf = NQ == 2 ? x : j & 1;
              if (!wait(&M.p_ready[buf], p_used[buf] & 1)) return;
              ++p_used[buf];
              values(v, x, buf, j > 0);
              if (more && j + AHEAD < count[x]) {
                if (!have && !wait(&M.full[k], kph)) return;
                have = true;
                keys(k, x, buf);
              }
            }
            mma_commit(&M.empty[v]);
            if (more) {
              if (!have && !wait(&M.full[k], kph)) return;
              mma_commit(&M.empty[k]);
              if (j + AHEAD == tiles - 1) mma_commit(&M.q_empty);
            }
            stage += 2;
            if (stage >= C::STAGES) {
              stage -= C::STAGES;
              phase ^= 1;
            }
          }
        }
      };
      if (lane == 0) {
        run();
        mma_commit(&M.drain);                     // every product is through before TMEM is freed
        mbar_wait_bounded(&M.drain, 0);
      }
    } else if (warp == C::W_LOAD && !C::CONV) {
      // ================= pages by TMA =================
      uint32_t stage = 0, phase = 0, tile_no = 0;
      uint32_t flying[2] = {0, 0};                // stages with copies that nobody may have waited for, by phase
      auto run = [&] {
        Walk<C> w(p, M.begin, mine);
        const int rows = min(p.page_size, KT), boxes = KT / rows * C::BLK;
        for (; w.piece(); w.next()) {
          const int32_t* table = p.page_table + (long long)w.r.req * p.max_pages;
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            const int n0 = w.b.start + j * KT;
            const int u = lane / C::BLK, n = n0 + u * rows;
            const bool want = lane < boxes && n < w.b.hi;
            int page = want ? table[n >> p.page_shift] : 0;
            const bool off = want && (page < 0 || page >= p.n_pages);
            if (__any_sync(FULL_MASK, off)) {
              // the bad units, of 16 positions
              unsigned bits = off ? ((1u << (rows / 16)) - 1) << (u * (rows / 16)) : 0u;
              bits = __reduce_or_sync(FULL_MASK, bits);
              if (lane == 0) {
                set_error(err, HS_DEVERR_PAGE);
                M.bad[tile_no & 7] = (unsigned char)bits;
              }
            } else if (lane == 0) {
              M.bad[tile_no & 7] = 0;
            }
            const bool copy = want && !off;
            const int copies = __popc(__ballot_sync(FULL_MASK, copy));
            const int in_page = n & (p.page_size - 1);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              if (!__all_sync(FULL_MASK, wait_for(&M.empty[stage], phase ^ 1, abort, err))) return;
              if (lane == 0) mbar_arrive_expect_tx(&M.full[stage], copies * rows * 128);
              __syncwarp();
              if (copy)
                tma_rows(ring_s + stage * C::STAGE + (lane % C::BLK) * (KT * 128) + u * rows * 128, &map,
                         ((page * 2 + which) * p.h_kv + w.head) * p.page_size + in_page, lane % C::BLK, &M.full[stage]);
              flying[phase] |= 1u << stage;
              flying[phase ^ 1] &= ~(1u << stage);
              if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1;
              }
            }
          }
        }
      };
      run();
      if (*abort)                                  // copies in flight land before the shared memory goes
        for (int s = 0; s < C::STAGES; ++s)
          for (int ph = 0; ph < 2; ++ph)
            if (flying[ph] >> s & 1) mbar_wait_bounded(&M.full[s], ph);
    } else if (warp == C::W_FIX && !C::CONV) {
      // ================= values of positions that no row sees become 0 =================
      auto run = [&] {
        uint32_t stage = 0, phase = 0, tile_no = 0;
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next())
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            // keys are passed on as they are (a stage holds keys in one round and values in the next)
            if (!__all_sync(FULL_MASK, wait_for(&M.full[stage], phase, abort, err))) return;
            if (lane == 0) mbar_arrive(&M.vok[stage]);
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
            if (lane == 0) mbar_arrive(&M.vok[stage]);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
      };
      run();
    } else if (warp == C::W_Q) {
      // ================= queries =================
      auto run = [&] {
        uint32_t no = 0;
        constexpr int PER = D / 8, TOGETHER = 32 / PER ? 32 / PER : 1;    // 16-byte parts of a row, rows at a time
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next(), ++no) {
          if (!__all_sync(FULL_MASK, wait_for(&M.q_empty, (no & 1) ^ 1, abort, err))) return;
          const int row0 = w.blk * C::ROWS, c = lane % PER;
          const uint16_t* q = static_cast<const uint16_t*>(p.q) + (long long)w.r.first * p.q_ts + (long long)w.head * p.group * p.q_hs;
          auto dst_of = [&](int r) {
            return smem + (r / 128) * C::QB + (c / 8) * (128 * 128) + (r % 128) * 128 + (((c % 8) ^ (r & 7)) << 4);
          };
          if constexpr (!C::CONV) {
            for (int r = lane / PER; r < w.b.rows; r += TOGETHER) {
              const int tok = (row0 + r) / p.group, g = row0 + r - tok * p.group;
              cp_async_16(dst_of(r), q + tok * p.q_ts + g * p.q_hs + c * 8);
            }
            cp_async_wait_all();
          } else {
            // as fp16, a row under a power of two that brings its largest into [1, 2)
            for (int rb = 0; rb < w.b.rows; rb += TOGETHER) {
              const int r = rb + lane / PER;
              const bool in = r < w.b.rows;
              const int tok = (row0 + (in ? r : 0)) / p.group, g = row0 + (in ? r : 0) - tok * p.group;
              const uint4 u = in ? *reinterpret_cast<const uint4*>(q + tok * p.q_ts + g * p.q_hs + c * 8) : make_uint4(0, 0, 0, 0);
              const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
              float x[8], mx = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 v = pa::unpack2<C::QTYPE>(uw[e]);
                x[2 * e] = v.x;
                x[2 * e + 1] = v.y;
                mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
              }
#pragma unroll
              for (int o = PER / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, o));
              const int e2 = mx > 0.f && mx < INFINITY ? max(-126, min(126, ilogbf(mx))) : 0;
              const float down = exp2f((float)(-e2 / 2)), down2 = exp2f((float)(-e2 - (-e2 / 2)));
              uint4 y;
              y.x = pa::pack2<HS_FP16>(x[0] * down * down2, x[1] * down * down2);
              y.y = pa::pack2<HS_FP16>(x[2] * down * down2, x[3] * down * down2);
              y.z = pa::pack2<HS_FP16>(x[4] * down * down2, x[5] * down * down2);
              y.w = pa::pack2<HS_FP16>(x[6] * down * down2, x[7] * down * down2);
              if (in) {
                *reinterpret_cast<uint4*>(dst_of(r)) = y;
                if (c == 0) M.q_exp[no & 1][r] = (signed char)e2;
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
        uint32_t stage = 0, phase = 0, tile_no = 0;
        const int ct = tid - 32 * C::W_CONV;
        constexpr int EL = C::PAGES == PAGES_INT4 ? 32 : 16;       // elements of 16 bytes of codes
        constexpr int PER = D / EL, STEP = 128 / PER, N = KT / STEP;   // parts of a row, rows at a time, parts of a thread
        const int part = ct % PER, r0 = ct / PER;
        Walk<C> w(p, M.begin, mine);
        for (; w.piece(); w.next()) {
          const int32_t* table = p.page_table + (long long)w.r.req * p.max_pages;
          for (int j = w.from; j < w.to; ++j, ++tile_no) {
            const int n0 = w.b.start + j * KT;
            if (warp == C::W_CONV) {
              const int n = n0 + lane * 16;
              const bool want = lane < KT / 16 && n < w.b.hi;
              const int page = want ? table[n >> p.page_shift] : 0;
              const unsigned bits = __ballot_sync(FULL_MASK, page < 0 || page >= p.n_pages);
              if (lane == 0) {
                M.bad[tile_no & 7] = (unsigned char)bits;
                if (bits) set_error(err, HS_DEVERR_PAGE);
              }
            }
            int pages[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int n = n0 + r0 + i * STEP;
              pages[i] = n >= w.b.lo && n < w.b.hi ? table[n >> p.page_shift] : -1;
              if (pages[i] >= p.n_pages) pages[i] = -1;
            }
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              uint4 raw[N];
              uint32_t sc[N];
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const int n = n0 + r0 + i * STEP;
                raw[i] = make_uint4(0, 0, 0, 0);
                sc[i] = 0;
                if (pages[i] >= 0) {
                  const long long at = ((((long long)pages[i] * 2 + which) * p.h_kv + w.head) << p.page_shift) + (n & (p.page_size - 1));
                  if constexpr (C::PAGES == PAGES_E4M3) {
                    raw[i] = *reinterpret_cast<const uint4*>(p.pages + at * D + part * 16);
                  } else {
                    const unsigned char* u = p.pages + (at >> 4) * (9 * D);
                    const int k = n & 15;
                    raw[i] = *reinterpret_cast<const uint4*>(u + (which ? part * 256 + k * 16 : k * (D / 2) + part * 16));
                    const unsigned char* b = u + 8 * D + (which ? part * 32 + k : k * (D / 16) + part * 2);
                    sc[i] = b[0] | (uint32_t)b[which ? 16 : 1] << 8;
                  }
                }
              }
              if (!__all_sync(FULL_MASK, wait_for(&M.empty[stage], phase ^ 1, abort, err))) return;
              unsigned char* to = smem + C::SM_RING + stage * C::STAGE;
#pragma unroll
              for (int i = 0; i < N; ++i) {
                const int r = r0 + i * STEP;
                auto put = [&](int e, uint4 v) {    // elements e .. e + 7
                  *reinterpret_cast<uint4*>(to + (e / 64) * (KT * 128) + r * 128 + (((e / 8 % 8) ^ (r & 7)) << 4)) = v;
                };
                const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                if constexpr (C::PAGES == PAGES_E4M3) {
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    uint4 v;
                    pa::e4m3x4_to_half2(x[2 * k], v.x, v.y);
                    pa::e4m3x4_to_half2(x[2 * k + 1], v.z, v.w);
                    put(part * 16 + k * 8, v);
                  }
                } else {
                  const uint32_t two = pa::e4m3x2_to_half2((uint16_t)sc[i]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const pa::Int4Scale s4 = pa::int4_scale(__byte_perm(two, 0, k < 2 ? 0x1010 : 0x3232));
                    uint32_t a[4];                  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
                    pa::int4x8_to_half2(x[k], s4, a);
                    put(part * 32 + k * 8, make_uint4(__byte_perm(a[0], a[1], 0x5410), __byte_perm(a[2], a[3], 0x5410),
                                                      __byte_perm(a[0], a[1], 0x7632), __byte_perm(a[2], a[3], 0x7632)));
                  }
                }
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&M.full[stage]);
              if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1;
              }
            }
          }
        }
      };
      run();
    }
  }

  // ---- rows of bad requests
  for (int i = blockIdx.x; i < p.n_req; i += gridDim.x) {
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
  auto piece = [&](int j) { return p.ws + ws_piece<C>(cta + j, j == 0); };
  float mm = -INFINITY;
  for (int j = 0; j < n; ++j) mm = fmaxf(mm, in ? piece(j)[C::ROWS * C::D + row] : -INFINITY);
  const float base = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  for (int j = 0; j < n; ++j)
    if (in) ll += exp2f(piece(j)[C::ROWS * C::D + row] - base) * piece(j)[C::ROWS * C::D + C::ROWS + row];
  float4 acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = warp; j < n; j += JOIN_WARPS) {
    if (!in) break;
    const float* at = piece(j);
    const float w = exp2f(at[C::ROWS * C::D + row] - base);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(at + ((size_t)(c0 + c) * C::ROWS + row) * 4);
      acc[c].x += w * x.x;
      acc[c].y += w * x.y;
      acc[c].z += w * x.z;
      acc[c].w += w * x.w;
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) s_o[warp][c][lane] = acc[c];
  __syncthreads();
  float4 o = s_o[0][warp][lane];
#pragma unroll
  for (int k = 1; k < JOIN_WARPS; ++k) {
    const float4 x = s_o[k][warp][lane];
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
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, paged_attend_kernel<C>);
    if (e != cudaSuccess) return e;
    // the softmax warps would wait for ever for registers that the launch did not bring
    if (C::REGS_SOFT && fa.numRegs * C::WARPS < C::REGS_SOFT * C::SOFT + C::REGS_REST * (C::WARPS - C::SOFT))
      return cudaErrorInvalidConfiguration;
    return allow_smem(paged_attend_kernel<C>, C::SMEM);
  }
  static cudaError_t launch(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st) {
    const cudaError_t e = launch_pdl(paged_attend_kernel<C>, dim3(p.grid), dim3(C::THREADS), C::SMEM, st, p, map);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attend_join_kernel<C>, dim3(p.grid, C::ROWS / 32, C::D / 32), dim3(32 * JOIN_WARPS), 0, st, p);
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
