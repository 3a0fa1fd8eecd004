// Attention of one new token per request over its paged cache:
//
//   o_h = sum_n softmax_n(scale * q_h . K_n) V_n,  lse_h = ln sum_n exp(scale * q_h . K_n)
//
// over n in [max(0, N - window), N), in one pass with a running maximum m and sum l
// (of two pieces: m = max, l and o weighted by 2^(m_i - m)).
//
// Bound: HBM.  A row of keys and values serves the h_q / h_kv query heads of its
// kv head, a few flops per byte, so the time is the cache's bytes; what the design
// is after is an even share of them for every SM and enough of them in flight.
// Measured (GB300; a kernel that only reads as many bytes reaches 7.1 to 7.5 TB/s, a copy
// 6.7): 16 requests x 32 K positions, 32/8 heads of 128, bf16: 318 to 321 us, 6.7 TB/s
// (the plain read 288 us; tensor pipe 14 % busy); one request of 200 K: 130 us, 6.4 TB/s
// (114 us); 64 of 17 .. 20 K positions, 8-bit pages: 75 us, 5.5 TB/s (57 us).  Around the
// stream of rows stand about 10 us: lengths, page ids and the first rows (4 us), the
// joining of pieces (1 to 3 us) and the second kernel (3 us): all of the 9 us that one
// request of 4 K positions takes.
//
// Work.  The positions of every (request, kv head) are cut into units of 16; all
// units of the call, request by request and head by head, form one sequence, and
// every CTA (one per SM) takes an equal contiguous share of it, every warp an equal
// share of its CTA's.  So one request of 200 K positions and a batch of short ones
// are spread the same way, with no table of splits: a CTA finds its place by a
// prefix sum over the lengths.  (A CTA per request and head, tile by tile, took 12.8
// ms for the 16 x 32 K above and 54 ms for the 200 K.)
//
// A warp runs alone: it has its own ring of stages in shared memory, starts the
// TMA copies of its next units itself (one copy of 16 rows of keys and of values: a
// unit never crosses a page), waits for its own mbarriers, and keeps its own m, l
// and output.  No barrier joins warps before the end of the share.  192 KB are in
// flight per SM; what slows the stream then is instructions: separate copies for keys
// and values, which refill half a stage earlier, cost 1 to 3 %, and taking the running
// maximum's shuffles and the masks out of most units gained 4 %.
//
// Products on mma.sync m16n8k16 with 32-bit sums, transposed so that the wide side
// is the cache's: S^T = K Q^T (16 rows x 8 heads per tile), O^T += V^T P^T (16
// output elements x 8 heads); the tensor pipe is far from the bound.  P^T becomes
// the second product's operand by movmatrix.  Bytes of 8-bit pages are turned into
// fp16 (exactly) between ldmatrix and the product, in an order of the elements that
// needs no shuffling: queries are loaded in the order in which key bytes come, and
// output rows leave in that of the value bytes.
//
// 4-bit pages come by two plain copies a unit (its keys lie together, and its values).  A lane's keys are 16
// consecutive bytes of a row; values come by ldmatrix, four elements of two positions in a word, which
// is the operand's order already.  A code becomes fp16 by one mask and one fused multiply-add, exactly.  16 x 32 K
// positions over 4-bit pages: 178 us (bf16: 320), 3.4 TB/s; the ALU pipe is 64 % busy, 65 % of the issue slots
// are used: 500 instructions a unit of 16 positions, half of them for turning codes.
//
// Scores with a cap or a bias are kernels of their own (SCORES): the cap by tanh32, the bias from the
// positions; 16 x 32 K with a cap or a bias takes as long as without over 16- and 8-bit pages (320 to 325 us, 171
// to 175), over 4-bit pages, where instructions count, 199 us with a cap and 189 with a bias (181 without).
//
// Short contexts.  Where no request of the call can have more than a few dozen units (by
// the table's width or the window), CTAs take whole segments: nothing crosses CTAs, and
// the second kernel, 3 us on the GPU and 4 of a call through the API, is not launched.
//
// Pieces.  A (request, head) wholly inside a warp's share is written out by the
// warp.  What crosses warps is joined by the CTA at its end, what crosses CTAs goes
// to the workspace and is joined by the second kernel (a programmatic dependent):
// at most one such chain starts in a CTA, so that kernel has one small block per
// CTA and head.  Nothing is kept between calls, so calls that overlap need only a
// workspace each.
#ifndef HS_PAGED_ATTENTION_CUH_
#define HS_PAGED_ATTENTION_CUH_

#include "hs_paged.cuh"

namespace hs {
namespace pa {

constexpr int UNIT = PG_UNIT;            // positions
// what a segment costs on top of its units, in units: about two of them by the warps' ends (64 ragged
// requests over 8-bit pages: 83, 78 and 76 us with 1, 2 and 4; no change from there up to 12)
constexpr int SEGMENT_COST = 4;
constexpr int RING_BYTES = 192 * 1024;
// Units of a segment up to which CTAs take whole ones (see above).  Of 32/8 heads of 128, bf16: one
// request of 512 positions 7.9 us either way, of 1024 11.0 instead of 8.0, but 16 of 1024 15.2 instead of
// 18.6 and 128 of them 89 instead of 93; through the API every such call takes 12.4 us instead of 16.3.
// The gain is the call's, not always the GPU's: 33 requests with a window of 1000 (24/8 heads of 64, fp16)
// take 12.6 us in a graph, shared they took 11.6.  The rule counts units whatever their bytes, asks for
// MANY_SEGMENTS, which is fewer than the SMs (64 to 127 segments of 33 to 64 units were not measured), and
// goes by the table's width or the window, as the host does not know the lengths: a window of 1000 passes
// (64 units with the one it lies across), one of 1024 does not (66).
constexpr int WHOLE_UNITS = 32, WHOLE_UNITS_MANY = 64, MANY_SEGMENTS = 64;

template <int D, int NT, int QTYPE, int PAGES>
struct Cfg {
  static constexpr bool E4M3 = PAGES == PAGES_E4M3, INT4 = PAGES == PAGES_INT4;
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int HEADS = 8 * NT;                       // query heads of a pass
  static constexpr int ROW = D * ES < 128 ? D * ES : 128;    // bytes of a row in one swizzled block
  static constexpr int BLOCKS = D * ES / ROW;                // blocks side by side in a row
  static constexpr int HALF = INT4 ? 9 * D : UNIT * D * ES;  // bytes of a unit's keys (or values)
  static constexpr int STAGE = 2 * HALF;
  // Eight warps with three stages or six; four where a unit is 16 KB; sixteen where units are
  // small or turning bytes into fp16 takes a warp long (8-bit, d = 128: 128 -> 90 us with the
  // segments' cost), if the registers allow it.
  static constexpr int WARPS = STAGE >= 16384 ? 4 : STAGE <= 2048 || ((E4M3 || INT4) && D == 128 && NT == 1) ? 16 : 8;
  static constexpr int STAGES = RING_BYTES / (WARPS * STAGE) < 12 ? RING_BYTES / (WARPS * STAGE) : 12;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int PROW = D + 4;                         // floats of a piece's head row (bank spread)
  static constexpr int PIECE = HEADS * PROW + 2 * HEADS;     // o rows, then m, then l
  static_assert(PIECE * 4 <= STAGES * STAGE, "a piece fits a warp's ring");
  static constexpr int SM_RING = 0;
  static constexpr int SM_BARS = WARPS * STAGES * STAGE;
  static constexpr int SM_META = SM_BARS + WARPS * STAGES * 8;
  static constexpr int SM_SCAN = SM_META + 2 * WARPS * 32;
  static constexpr int SM_PRE = SM_SCAN + (WARPS + 2) * 4 * 2;
  static size_t smem(int n_req) { return 1024 + SM_PRE + (size_t)(n_req + 1) * 4; }
};

// where the second kernel finds a chain of pieces that starts in a CTA
struct Chain {
  int32_t ri, hc;      // request of the call, kv head and chunk of its query heads
  int32_t last;        // the chain's last CTA; -1: none starts here
  int32_t _pad;
};

// workspace: two pieces per CTA (0: of the segment that came in, 1: of the one that
// goes on), one per warp, then a Chain per CTA
__host__ __device__ inline size_t ws_cta(int piece, int cta, int slot) { return (size_t)(cta * 2 + slot) * piece; }
__host__ __device__ inline size_t ws_warp(int piece, int grid, int warps, int cta, int warp) {
  return ((size_t)grid * 2 + (size_t)cta * warps + warp) * piece;
}
__host__ __device__ inline size_t ws_chain(int piece, int grid, int warps) { return (size_t)grid * (2 + warps) * piece; }

struct Meta {          // a piece that does not cover its segment
  float* at;           // null: none
  int32_t ri, hc, from, to, n, _pad;
};

template <int QTYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (QTYPE == HS_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <int QTYPE>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (QTYPE == HS_BF16) return make_float2(bf16lo(u), bf16hi(u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 values (low byte first) as two and two fp16: exact
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// two e4m3 values (low byte first) as fp16: exact
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
  return r;
}

// Rows of 4 bits, as fp16: eight codes c of a word become (c - 8) s, exactly.  c | 0x6400 is the fp16
// 1024 + c, and 0x6400 | 16 c (a nibble higher) is 1024 + 16 c: one fused multiply-add takes the offset
// and brings the scale in, with both products' operands in 11 bits (129 s, 9 s: s has 4).  Pairs of the
// result are codes (0, 4), (1, 5), (2, 6), (3, 7) of the word.  Scales are taken 2^-6 as large
// (1032 * 448 is beyond fp16); whoever uses the values puts INT4_SHIFT back.
constexpr float INT4_SHIFT = 64.f;
struct Int4Scale {
  uint32_t s, off, s16, off16;        // s, -1032 s, s / 16, -72 s
};
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ Int4Scale int4_scale(uint32_t two) {
  Int4Scale x;
  x.s = hmul2(two, 0x24002400u);      // 2^-6
  x.off = hmul2(x.s, 0xe408e408u);    // -1032
  x.s16 = hmul2(x.s, 0x2c002c00u);    // 1 / 16
  x.off16 = hmul2(x.s, 0xd480d480u);  // -72
  return x;
}
__device__ __forceinline__ void int4x8_to_half2(uint32_t w, const Int4Scale& x, uint32_t (&r)[4]) {
  const uint32_t v = w >> 8;
  r[0] = hfma2((w & 0x000f000fu) | 0x64006400u, x.s, x.off);
  r[1] = hfma2((w & 0x00f000f0u) | 0x64006400u, x.s16, x.off16);
  r[2] = hfma2((v & 0x000f000fu) | 0x64006400u, x.s, x.off);
  r[3] = hfma2((v & 0x00f000f0u) | 0x64006400u, x.s16, x.off16);
}
// the w-th word (of eight codes) that lane t of a row's four holds: 16 bytes at a time, side by side
template <int D>
__device__ __forceinline__ int int4_word(int t, int w) {
  return D == 64 ? 2 * t + w : (w / 4) * 16 + 4 * t + w % 4;
}

// what a value's sum is multiplied with at the end
template <int PAGES>
__device__ __forceinline__ float value_scale(const PagedDecodeParams& p, int kvh) {
  return PAGES == PAGES_SAME ? 1.f : p.kv_scale[p.h_kv + kvh] * (PAGES == PAGES_INT4 ? INT4_SHIFT : 1.f);
}

// L2 policy of the pool's rows: read once by a call, they leave first (the whole of L2
// then serves queries, pieces and the next kernels: 43.3 -> 40.8 us for a step of 64
// requests of heads of 256); where several passes read them, as any other data.
__device__ __forceinline__ uint64_t pool_policy(bool once) {
  uint64_t pol;
  if (once)
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ void tma_unit(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst), "l"(map), "r"(bar), "r"(0), "r"(row), "r"(0), "r"(0), "l"(policy)
      : "memory");
}

// 2^x (to 2^-22 of it; below 2^-126: 0)
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float LOG2_E = 1.4426950408889634f;

// tanh to about 2^-20 of itself: near zero by its series (five terms: 2^-22 of itself at 0.3),
// elsewhere 1 - 2 / (e^2|x| + 1)
__device__ __forceinline__ float tanh32(float x) {
  const float a = fabsf(x), y = x * x;
  float near = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f) * x;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(pow2(a * (2.f * LOG2_E)) + 1.f));
  return a < 0.3f ? near : copysignf(fmaf(-2.f, r, 1.f), x);
}

// The softmax's reference m.  Weights are 2^(s - m) with m near the running maximum, not
// at it: m is raised (to the maximum, by shuffles, with o and l rescaled) only once a score
// is more than SLACK above it, so most units need no exchange between lanes.  Weights are
// then at most 2^SLACK.  Those that go to fp16 are taken 2^FP16_SHIFT times as large (and
// so is their sum): at most 2^15, and with fp16's full precision down to 2^-21 of the
// reference, where unscaled ones would lose it below 2^-14.
constexpr float SLACK = 8.f;
constexpr float FP16_SHIFT = 7.f;

// Units of request i of the call (0 with an error bit for a bad one).
__device__ __forceinline__ int request_units(const PagedDecodeParams& p, int i, int* first_unit, int* first, int* len,
                                             int* req, unsigned* err) {
  *req = p.req_ids ? p.req_ids[i] : i;
  *len = *first = *first_unit = 0;
  if (*req < 0 || *req >= p.max_requests) {
    *err |= HS_DEVERR_REQ_RANGE;
    return 0;
  }
  const int n = p.lengths[*req];
  if (n < 0 || n > p.max_pages << p.page_shift) {
    *err |= HS_DEVERR_CAPACITY;
    return 0;
  }
  *len = n;
  *first = p.window > 0 ? max(0, n - p.window) : 0;
  *first_unit = *first / UNIT;
  return (n + UNIT - 1) / UNIT - *first_unit;
}

template <int QTYPE>
__device__ __forceinline__ void store_out4(void* out, long long at, float4 v) {
  uint2 w;
  w.x = pack2<QTYPE>(v.x, v.y);
  w.y = pack2<QTYPE>(v.z, v.w);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
}

// a lane's VW elements of a row of 32 VW
template <int VW>
__device__ __forceinline__ void load_lane(const float* p, float (&x)[VW]) {
  if constexpr (VW == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + e);
      x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
    }
  }
}
template <int VW>
__device__ __forceinline__ void save_lane(float* p, const float (&x)[VW]) {
  if constexpr (VW == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int e = 0; e < VW; e += 4) *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  }
}
template <int QTYPE, int VW>
__device__ __forceinline__ void store_lane(void* out, long long at, const float (&x)[VW]) {
  uint32_t w[VW / 2];
#pragma unroll
  for (int e = 0; e < VW / 2; ++e) w[e] = pack2<QTYPE>(x[2 * e], x[2 * e + 1]);
  uint16_t* dst = static_cast<uint16_t*>(out) + at;
  if constexpr (VW == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
  if constexpr (VW == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  if constexpr (VW == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / l of a finished row: 0 where nothing was attended
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

template <bool BF16>
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l) - (BF16 ? 0.f : FP16_SHIFT)) * 0.693147180559945f;
}

struct Place {   // a unit of the sequence
  int ri, hc, u, n;
};

template <int D, int NT, int QTYPE, int PAGES, bool SCORES>
__global__ void __launch_bounds__(Cfg<D, NT, QTYPE, PAGES>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ CUtensorMap map) {
  using C = Cfg<D, NT, QTYPE, PAGES>;
  constexpr bool E4M3 = C::E4M3, INT4 = C::INT4, SCALED = E4M3 || INT4;
  constexpr bool BF16 = QTYPE == HS_BF16 && !SCALED;   // type of the products
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::SM_BARS);
  Meta* meta = reinterpret_cast<Meta*>(smem + C::SM_META);
  int* scan = reinterpret_cast<int*>(smem + C::SM_SCAN);
  int* pre = reinterpret_cast<int*>(smem + C::SM_PRE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  uint64_t* bar = bars + warp * C::STAGES;
  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
  }
  if (lane < 2) meta[warp * 2 + lane].at = nullptr;
  griddep_wait();
  griddep_launch_dependents();

  // ---- the sequence: units before each request, for one head.  Few requests: every
  // warp by itself (they all write the same values), no barrier; many: the CTA together
  {
    const bool few = p.n_req <= 4 * 32;
    int a, b, c, r;
    unsigned err = 0;
    if (few) {
      const int per = (p.n_req + 31) / 32;
      int n[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = lane * per + k;
        n[k] = k < per && i < p.n_req ? request_units(p, i, &a, &b, &c, &r, &err) : 0;
        sum += n[k];
      }
      int at = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(FULL_MASK, at, o);
        if (lane >= o) at += x;
      }
      if (lane == 31) pre[p.n_req] = at;
      at -= sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = lane * per + k;
        if (k < per && i < p.n_req) pre[i] = at;
        at += n[k];
      }
      if (err && blockIdx.x == 0 && warp == 0) set_error(p.dev_error, err);
      __syncwarp();
    } else {
      const int per = (p.n_req + C::THREADS - 1) / C::THREADS;
      const int i0 = min(p.n_req, tid * per), i1 = min(p.n_req, i0 + per);
      int sum = 0;
      for (int i = i0; i < i1; ++i) sum += request_units(p, i, &a, &b, &c, &r, &err);
      int all;
      int at = block_exclusive_scan<C::THREADS>(sum, scan, &all);
      for (int i = i0; i < i1; ++i) {
        pre[i] = at;
        at += request_units(p, i, &a, &b, &c, &r, &err);
      }
      if (tid == 0) pre[p.n_req] = all;
      if (err && blockIdx.x == 0) set_error(p.dev_error, err);
      __syncthreads();
    }
  }
  const int chunks = (p.group + C::HEADS - 1) / C::HEADS;
  const int hcn = p.h_kv * chunks;
  // Shares are of cost: a segment's units and SEGMENT_COST more before them (its queries,
  // its first page ids, its output), so that many short segments weigh what they take.
  auto cost_before = [&](int r) { return ((long long)pre[r] + (long long)SEGMENT_COST * r) * hcn; };
  const long long total = cost_before(p.n_req);
  // (64-bit divisions take a while: only for sequences that need them)
  long long share = total < (1 << 30) ? ((int)total + (int)gridDim.x - 1) / (int)gridDim.x
                                      : (total + gridDim.x - 1) / gridDim.x;
  if (share < C::WARPS && !p.whole) share = C::WARPS;
  // the request in which a cost position x < total lies
  auto request_at = [&](long long x) {
    int lo = 0, hi = p.n_req;       // cost_before(lo) <= x < cost_before(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cost_before(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  // Each of these is worked out for the share's begin by the even lanes, for its end by the odd ones.
  long long edge = min(total, (blockIdx.x + (lane & 1)) * share);
  if (p.whole && edge < total) {    // whole segments: up to where one begins
    const int r = request_at(edge), n = pre[r + 1] - pre[r] + SEGMENT_COST;
    const int off = (int)(edge - cost_before(r)) % n;
    edge += off ? n - off : 0;
  }
  const long long cta0 = __shfl_sync(FULL_MASK, edge, 0), cta1 = __shfl_sync(FULL_MASK, edge, 1);
  const long long wshare = (cta1 - cta0 + C::WARPS - 1) / C::WARPS;
  // units before a cost position, and the place of the next one
  const long long x0 = min(cta1, cta0 + warp * wshare);
  const long long x1 = min(cta1, x0 + wshare);
  Place at = {0, 0, 0, 1};          // the unit to be consumed next
  long long w0, w1;
  {
    const long long x = lane & 1 ? x1 : x0;
    long long units = (long long)pre[p.n_req] * hcn;
    if (x < total) {
      const int lo = request_at(x);
      const int n = pre[lo + 1] - pre[lo], rem = (int)(x - cost_before(lo));
      const int hc = rem / (n + SEGMENT_COST);
      const int u = max(0, rem - hc * (n + SEGMENT_COST) - SEGMENT_COST);
      at = Place{lo, hc, u, n};
      units = (long long)pre[lo] * hcn + (long long)hc * n + u;
    }
    __syncwarp();
    w0 = __shfl_sync(FULL_MASK, units, 0);
    w1 = __shfl_sync(FULL_MASK, units, 1);
    at.ri = __shfl_sync(FULL_MASK, at.ri, 0);
    at.hc = __shfl_sync(FULL_MASK, at.hc, 0);
    at.u = __shfl_sync(FULL_MASK, at.u, 0);
    at.n = __shfl_sync(FULL_MASK, at.n, 0);
  }

  const unsigned char* ring = smem + C::SM_RING + (size_t)warp * C::STAGES * C::STAGE;
  const uint32_t ring_s = smem_addr(ring);

  if (w0 < w1) {
    while (at.n == 0) {             // requests without positions have no units
      ++at.ri;
      at.hc = at.u = 0;
      at.n = pre[at.ri + 1] - pre[at.ri];
    }
    Place is = at;                  // the unit whose copy starts next
    int to_issue = (int)(w1 - w0), to_do = to_issue;   // (2^40 units at the most, over 608 warps or more: 2^30.8)
    auto step = [&](Place& x) {
      if (++x.u == x.n) {
        x.u = 0;
        if (++x.hc == hcn) {
          x.hc = 0;
          do ++x.ri; while (x.ri < p.n_req && pre[x.ri + 1] == pre[x.ri]);
          x.n = x.ri < p.n_req ? pre[x.ri + 1] - pre[x.ri] : 1;
        }
      }
    };

    // ---- copies
    int i_ri = -1, i_unit0 = 0, i_pages = 0;        // the request whose copies are being started
    const int32_t* i_table = nullptr;
    int win = 0, win_page = -1;                     // its page ids win .. win + 31, one per lane
    int i_row = 0, i_left = 0;                      // pool row of the next unit, units left on its page
    bool i_bad = false;                             // its page id was out of range
    unsigned bad = 0;                               // the same of each stage
    const int upp = p.page_shift - 4;               // units of a page: 2^upp
    const uint64_t policy = pool_policy(chunks == 1);
    auto issue = [&](int stage) {
      if (i_left == 0) {                            // a page begins, or a segment
        if (is.ri != i_ri) {
          int first, len, req;
          unsigned err = 0;
          request_units(p, is.ri, &i_unit0, &first, &len, &req, &err);
          i_ri = is.ri;
          i_pages = (len + p.page_size - 1) >> p.page_shift;
          i_table = p.page_table + (long long)req * p.max_pages;
          win = -64;
        }
        const int ua = i_unit0 + is.u;
        const int pg = ua >> upp;
        if (pg < win || pg >= win + 32) {
          win = pg;
          win_page = win + lane < i_pages ? i_table[win + lane] : -1;
        }
        int page = __shfl_sync(FULL_MASK, win_page, pg - win);
        i_bad = page < 0 || page >= p.n_pages;
        if (i_bad) {
          page = 0;                 // some page: its rows are not used
          if (lane == 0) set_error(p.dev_error, HS_DEVERR_PAGE);
        }
        const int in_page = ua & ((1 << upp) - 1);
        i_row = ((page * 2 * p.h_kv + is.hc / chunks) << p.page_shift) + in_page * UNIT;
        i_left = min((1 << upp) - in_page, is.n - is.u);
      }
      bad = (bad & ~(1u << stage)) | ((unsigned)i_bad << stage);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar[stage], C::STAGE);
        if constexpr (INT4) {                       // a unit's keys lie together, and its values
          const unsigned char* k = p.pages + (long long)(i_row >> 4) * C::HALF;
          unsigned char* to = smem + C::SM_RING + ((size_t)warp * C::STAGES + stage) * C::STAGE;
          bulk_g2s_hint(to, k, C::HALF, &bar[stage], policy);
          bulk_g2s_hint(to + C::HALF, k + ((long long)p.h_kv << (p.page_shift - 4)) * C::HALF, C::HALF, &bar[stage], policy);
        } else {
          tma_unit(ring_s + stage * C::STAGE, &map, i_row, smem_addr(&bar[stage]), policy);
        }
      }
      i_row += UNIT;
      --i_left;
      step(is);
    };
    for (int s = 0; s < C::STAGES && to_issue > 0; ++s, --to_issue) issue(s);

    // ---- lane's places in a stage: ldmatrix rows and the swizzle of their 16-byte pieces
    auto place = [&](int row, int piece) {
      const int sw = C::ROW == 128 ? (row & 7) : ((row >> 1) & 3);
      return (uint32_t)(row * C::ROW + ((piece ^ sw) << 4));
    };
    const uint32_t k_at = place(lane & 15, lane >> 4);
    const uint32_t v_at = C::HALF + (INT4 ? (lane >> 4) * 256 + (lane & 15) * 16
                                     : E4M3 ? k_at : place((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
    // piece 2 i + b of a row: b is in the lane's place, 2 i changes bits that the place's xor keeps apart
    auto piece2 = [&](uint32_t base, int i) {
      constexpr int PER = C::ROW / 32;              // pairs of pieces in a block
      return (base ^ ((i % PER) << 5)) + (i / PER) * (UNIT * C::ROW);
    };

    uint32_t qf[NT][D / 16][2];
    float fac[NT][2];                               // scores to powers of two (or shares of the cap), by head
    [[maybe_unused]] float slope[NT][2];            // of the distance, to powers of two
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    int first = 0, len = 0, unit0 = 0, from = 0;
    bool fresh = true, alive = true;
    int stage = 0;
    uint32_t phase = 0;

    for (; to_do > 0; --to_do) {
      if (fresh) {                                  // a segment begins (or the share does)
        int req;
        unsigned err = 0;
        request_units(p, at.ri, &unit0, &first, &len, &req, &err);
        from = at.u;
        const int kvh = at.hc / chunks, chunk = at.hc - kvh * chunks;
        const float ks = E4M3 ? p.kv_scale[kvh] : INT4 ? p.kv_scale[kvh] * INT4_SHIFT : 1.f;
        const float to_score = SCORES && p.cap_in != 0.f ? p.cap_in : p.scale_log2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hg = chunk * C::HEADS + nt * 8 + g;        // head within the group
          const bool have = hg < p.group;
          const uint16_t* qrow = static_cast<const uint16_t*>(p.q) + at.ri * p.q_ts + (kvh * p.group + (have ? hg : 0)) * p.q_hs;
          if constexpr (SCALED) {
            // columns 4t .. 4t+3 of each 16, or pairs of the lane's eights: the order in which the keys come
            float x[D / 16][4], mx = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; c += INT4 ? 2 : 1) {
              if constexpr (INT4) {
                const uint4 w = *reinterpret_cast<const uint4*>(qrow + int4_word<D>(t, c / 2) * 8);
                const float2 a = unpack2<QTYPE>(w.x), b = unpack2<QTYPE>(w.y), d = unpack2<QTYPE>(w.z), f = unpack2<QTYPE>(w.w);
                x[c][0] = a.x; x[c][1] = d.x; x[c][2] = a.y; x[c][3] = d.y;
                x[c + 1][0] = b.x; x[c + 1][1] = f.x; x[c + 1][2] = b.y; x[c + 1][3] = f.y;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(qrow + c * 16 + t * 4);
                const float2 a = unpack2<QTYPE>(w.x), b = unpack2<QTYPE>(w.y);
                x[c][0] = a.x; x[c][1] = a.y; x[c][2] = b.x; x[c][3] = b.y;
              }
#pragma unroll
              for (int e = 0; e < (INT4 ? 8 : 4); ++e) mx = fmaxf(mx, fabsf(x[c + (e >> 2)][e & 3]));
            }
            mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 2));
            // the row under a power of two, its largest in [1, 2): fp16 holds it as well as its own type
            const int e2 = mx > 0.f && mx < INFINITY ? ilogbf(mx) : 0;
            const float down = exp2f((float)(-e2 / 2)), down2 = exp2f((float)(-e2 - (-e2 / 2)));
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              qf[nt][c][0] = have ? pack2<HS_FP16>(x[c][0] * down * down2, x[c][1] * down * down2) : 0u;
              qf[nt][c][1] = have ? pack2<HS_FP16>(x[c][2] * down * down2, x[c][3] * down * down2) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ee = __shfl_sync(FULL_MASK, e2, (2 * t + e) << 2);
              fac[nt][e] = to_score * ks * exp2f((float)(ee / 2)) * exp2f((float)(ee - ee / 2));
            }
          } else {
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(qrow + c * 16 + e * 8 + t * 2);
                qf[nt][c][e] = have ? w : 0u;
              }
            fac[nt][0] = fac[nt][1] = to_score;
          }
          if constexpr (SCORES) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int hs = chunk * C::HEADS + nt * 8 + 2 * t + e;
              slope[nt][e] = p.slopes && hs < p.group ? p.slopes[kvh * p.group + hs] * LOG2_E : 0.f;
            }
          }
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) o[nt][c][0] = o[nt][c][1] = o[nt][c][2] = o[nt][c][3] = 0.f;
        }
        fresh = false;
      }

      if (alive) {
        alive = __all_sync(FULL_MASK, mbar_wait_bounded(&bar[stage], phase));
        if (!alive) {                               // a copy did not come: none is started any more
          if (lane == 0) set_error(p.dev_error, HS_DEVERR_TIMEOUT);
          // those in flight get their time before the shared memory goes on to something else
          const int flying = min(to_do, C::STAGES);
          for (int j = 0; j < flying; ++j) {
            const int s = stage + j;
            mbar_wait_bounded(&bar[s < C::STAGES ? s : s - C::STAGES], s < C::STAGES ? phase : phase ^ 1u);
          }
        }
      }
      if (alive) {
        const uint32_t st = ring_s + stage * C::STAGE;
        // ---- S^T = K Q^T
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
        if constexpr (INT4) {
          const unsigned char* unit = smem + C::SM_RING + ((size_t)warp * C::STAGES + stage) * C::STAGE;
          constexpr int WORDS = D / 32;             // of eight codes, of a lane and row
          uint32_t w[2][WORDS];
          uint16_t sb[2][WORDS > 4 ? 2 : 1];        // the scales of the lane's blocks
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const unsigned char* row = unit + (g + 8 * r) * (D / 2);
            const unsigned char* srow = unit + 8 * D + (g + 8 * r) * (D / 16);
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(row + t * 8);
              w[r][0] = v.x; w[r][1] = v.y;
              sb[r][0] = srow[t];
            } else {
#pragma unroll
              for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + i * 64 + t * 16);
                w[r][4 * i] = v.x; w[r][4 * i + 1] = v.y; w[r][4 * i + 2] = v.z; w[r][4 * i + 3] = v.w;
                sb[r][i] = *reinterpret_cast<const uint16_t*>(srow + i * 8 + 2 * t);
              }
            }
          }
          Int4Scale sc[2];
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            uint32_t a[2][4];                       // by row: pairs of the word's eight
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (D == 64 ? i == 0 : i % 2 == 0) {
                const uint32_t two = e4m3x2_to_half2(sb[r][i / 4]);
                sc[r] = int4_scale(__byte_perm(two, 0, D == 64 || i % 4 == 0 ? 0x1010 : 0x3232));
              }
              int4x8_to_half2(w[r][i], sc[r], a[r]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t f[4] = {a[0][2 * c], a[1][2 * c], a[0][2 * c + 1], a[1][2 * c + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<false>(c ? s2[nt] : s[nt], f, qf[nt][2 * i + c][0], qf[nt][2 * i + c][1]);
            }
          }
        } else if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t r[4];
            ldsm4(r, st + piece2(k_at, i));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t a[4];
              e4m3x4_to_half2(r[2 * c], a[0], a[2]);
              e4m3x4_to_half2(r[2 * c + 1], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<false>(c ? s2[nt] : s[nt], a, qf[nt][2 * i + c][0], qf[nt][2 * i + c][1]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t a[4];
            ldsm4(a, st + piece2(k_at, c));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(c & 1 ? s2[nt] : s[nt], a, qf[nt][c][0], qf[nt][c][1]);
          }
        }
        // ---- rows of the unit that are attended: [lo, hi)
        const int pos = (unit0 + at.u) * UNIT;
        const int lo = max(0, first - pos), hi = (bad >> stage) & 1 ? 0 : min(UNIT, len - pos);
        const bool part = lo > 0 || hi < UNIT;
        const bool in0 = !part || (g >= lo && g < hi), in1 = !part || (g + 8 >= lo && g + 8 < hi);
        if (part) {
          // the others may hold anything: their values become 0 (a weight of 0 would leave a NaN one)
          if constexpr (INT4) {                     // (with a scale of 0, whatever their codes)
            unsigned char* sv = smem + C::SM_RING + ((size_t)warp * C::STAGES + stage) * C::STAGE + C::HALF + 8 * D;
            for (int e = lane; e < D; e += 32)
              if ((e & 15) < lo || (e & 15) >= hi) sv[e] = 0;
          } else
          for (int e = lane; e < UNIT * C::BLOCKS * (C::ROW / 16); e += 32) {
            const int row = (e / (C::ROW / 16)) % UNIT;
            if (row < lo || row >= hi)
              *reinterpret_cast<int4*>(smem + C::SM_RING + ((size_t)warp * C::STAGES + stage) * C::STAGE + C::HALF + e * 16) =
                  make_int4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();                 // before the next copy to this place
          __syncwarp();
        }
        bool grows = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[nt][e] = (s[nt][e] + s2[nt][e]) * fac[nt][e];
            s[nt][e + 2] = (s[nt][e + 2] + s2[nt][e + 2]) * fac[nt][e];
            if constexpr (SCORES) {
              if (p.cap_in != 0.f) {
                s[nt][e] = p.cap_log2 * tanh32(s[nt][e]);
                s[nt][e + 2] = p.cap_log2 * tanh32(s[nt][e + 2]);
              }
              s[nt][e] += slope[nt][e] * (float)(pos + g - (len - 1));
              s[nt][e + 2] += slope[nt][e] * (float)(pos + g + 8 - (len - 1));
            }
            s[nt][e] = in0 ? s[nt][e] : -INFINITY;
            s[nt][e + 2] = in1 ? s[nt][e + 2] : -INFINITY;
            grows = grows || fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + SLACK;
          }
        if (__any_sync(FULL_MASK, grows)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float n = fmaxf(s[nt][e], s[nt][e + 2]);
              n = fmaxf(n, __shfl_xor_sync(FULL_MASK, n, 4));
              n = fmaxf(n, __shfl_xor_sync(FULL_MASK, n, 8));
              n = fmaxf(n, __shfl_xor_sync(FULL_MASK, n, 16));
              n = fmaxf(n, m[nt][e]);
              const float keep = pow2(m[nt][e] - (n == -INFINITY ? 0.f : n));
              m[nt][e] = n;
              l[nt][e] *= keep;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                o[nt][c][e] *= keep;
                o[nt][c][e + 2] *= keep;
              }
            }
        }
        // Weights for values of 16 bits go as two numbers of their type, a rounded one and what it
        // leaves: one alone would put half a step on every weight, as much again as the output's own
        // rounding (relative error of a step over wide heads 0.0021 with one, 0.0017 with two and with
        // 32-bit weights; the second takes 1.3 % of the time).  8-bit values, themselves 2^-4 off, get
        // one fp16, and the tensor pipe's time back.
        constexpr int PARTS = SCALED ? 1 : 2;
        constexpr int WTYPE = BF16 ? HS_BF16 : HS_FP16;
        uint32_t pf[NT][PARTS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float base = (m[nt][e] == -INFINITY ? 0.f : m[nt][e]) - (BF16 ? 0.f : FP16_SHIFT);
            w[e] = pow2(s[nt][e] - base);
            w[e + 2] = pow2(s[nt][e + 2] - base);
            l[nt][e] += w[e] + w[e + 2];
          }
          const uint32_t x = pack2<WTYPE>(w[0], w[1]), y = pack2<WTYPE>(w[2], w[3]);
          pf[nt][0][0] = transpose8(x);
          pf[nt][0][1] = transpose8(y);
          if constexpr (PARTS == 2) {
            const float2 xr = unpack2<WTYPE>(x), yr = unpack2<WTYPE>(y);
            pf[nt][1][0] = transpose8(pack2<WTYPE>(w[0] - xr.x, w[1] - xr.y));
            pf[nt][1][1] = transpose8(pack2<WTYPE>(w[2] - yr.x, w[3] - yr.y));
          }
        }
        // ---- O^T += V^T P^T
        if constexpr (INT4) {
          const unsigned char* sv = smem + C::SM_RING + ((size_t)warp * C::STAGES + stage) * C::STAGE + C::HALF + 8 * D;
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t r[4];                          // [32 elements of the 64][positions 0-7, 8-15]
            ldsm4_trans(r, st + v_at + i * 512);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t a[2][4];                     // by positions: the four elements of a lane
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint16_t two = *reinterpret_cast<const uint16_t*>(sv + ((2 * i + q) * 2 + (g >> 2)) * 16 + h * 8 + 2 * t);
                int4x8_to_half2(r[2 * q + h], int4_scale(e4m3x2_to_half2(two)), a[h]);
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t f[4] = {a[0][2 * c], a[0][2 * c + 1], a[1][2 * c], a[1][2 * c + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][4 * i + 2 * q + c], f, pf[nt][0][0], pf[nt][0][1]);
              }
            }
          }
        } else if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t r[4];
            ldsm4_trans(r, st + piece2(v_at, i));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t x = r[2 * c], y = r[2 * c + 1];
              // a row pair of the tile is elements 2g and 2g+1 of the 16
              uint32_t a[4];
              e4m3x4_to_half2(__byte_perm(x, 0, 0x3120), a[0], a[1]);
              e4m3x4_to_half2(__byte_perm(y, 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][2 * i + c], a, pf[nt][0][0], pf[nt][0][1]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t a[4];
            ldsm4_trans(a, st + piece2(v_at, c));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int part = 0; part < PARTS; ++part) mma16816<BF16>(o[nt][c], a, pf[nt][part][0], pf[nt][part][1]);
          }
        }
        __syncwarp();                               // every lane has read the stage
        if (to_issue > 0) {
          issue(stage);
          --to_issue;
        }
      }
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }

      const bool ends = at.u + 1 == at.n;
      if (ends || to_do == 1) {
        // ---- a piece is done: [from, to) of its segment
        const int to = at.u + 1;
        const int kvh = at.hc / chunks, chunk = at.hc - kvh * chunks;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = l[nt][e];
            x += __shfl_xor_sync(FULL_MASK, x, 4);
            x += __shfl_xor_sync(FULL_MASK, x, 8);
            x += __shfl_xor_sync(FULL_MASK, x, 16);
            l[nt][e] = x;
          }
        // an accumulator's row 0 / 1 of the pair: elements of the 16 (4-bit pages: of the 32)
        const int d0 = INT4 ? 4 * g : E4M3 ? 2 * g : g, d1 = INT4 ? 4 * g + 1 : E4M3 ? 2 * g + 1 : g + 8;
        auto first_of = [](int c) { return INT4 ? (c >> 1) * 32 + (c & 1) * 2 : c * 16; };
        if (from == 0 && ends) {
          const float vs = value_scale<PAGES>(p, kvh);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int hg = chunk * C::HEADS + nt * 8 + 2 * t + e;
              if (hg < p.group) {
                const long long h = (long long)at.ri * p.h_q + kvh * p.group + hg;
                const float inv = inverse(l[nt][e]) * vs;
                uint16_t* row = static_cast<uint16_t*>(p.out) + h * D;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  const uint32_t two = pack2<QTYPE>(o[nt][c][e] * inv, o[nt][c][e + 2] * inv);
                  row[first_of(c) + d0] = (uint16_t)two;
                  row[first_of(c) + d1] = (uint16_t)(two >> 16);
                }
                if (p.lse && g == 0) p.lse[h] = log_sum<BF16>(m[nt][e], l[nt][e]);
              }
            }
        } else {
          // the share's last piece goes to the warp's own ring (no copy is in flight), one before it to the workspace
          float* dst = to_do == 1 ? reinterpret_cast<float*>(smem + C::SM_RING + (size_t)warp * C::STAGES * C::STAGE)
                                  : p.ws + ws_warp(C::PIECE, gridDim.x, C::WARPS, blockIdx.x, warp);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int h = nt * 8 + 2 * t + e;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                dst[h * C::PROW + first_of(c) + d0] = o[nt][c][e];
                dst[h * C::PROW + first_of(c) + d1] = o[nt][c][e + 2];
              }
              if (g == 0) {
                dst[C::HEADS * C::PROW + h] = m[nt][e];
                dst[C::HEADS * C::PROW + C::HEADS + h] = l[nt][e];
              }
            }
          if (lane == 0) meta[warp * 2 + (to_do == 1)] = Meta{dst, at.ri, at.hc, from, to, at.n, 0};
        }
        fresh = true;
      }
      step(at);
    }
  }
  __syncthreads();

  // ---- pieces of the CTA, in sequence order: neighbours of one segment are joined, a
  // warp per group of them and head.  Lane i knows piece i.
  {
    static_assert(2 * C::WARPS <= 32, "a piece per lane");
    constexpr int VW = D / 32;                      // elements of a lane
    const Meta a = lane < 2 * C::WARPS ? meta[lane] : Meta{};
    const unsigned valid = __ballot_sync(FULL_MASK, a.at != nullptr);
    const unsigned before = valid & ((1u << lane) - 1);
    const int prev = before ? 31 - __clz(before) : 0;
    const int prev_ri = __shfl_sync(FULL_MASK, a.ri, prev), prev_hc = __shfl_sync(FULL_MASK, a.hc, prev);
    const bool lead = a.at && (!before || prev_ri != a.ri || prev_hc != a.hc);
    unsigned leads = __ballot_sync(FULL_MASK, lead);
    Chain chain = {0, 0, -1, 0};
    for (int grp = 0; leads; ++grp) {
      const int first_piece = __ffs(leads) - 1;
      leads &= leads - 1;
      const unsigned members = valid & ~((1u << first_piece) - 1) & (leads ? (1u << (__ffs(leads) - 1)) - 1 : ~0u);
      const int last_piece = 31 - __clz(members);
      const int from = __shfl_sync(FULL_MASK, a.from, first_piece), to = __shfl_sync(FULL_MASK, a.to, last_piece);
      const int n = __shfl_sync(FULL_MASK, a.n, first_piece);
      const int ri = __shfl_sync(FULL_MASK, a.ri, first_piece), hc = __shfl_sync(FULL_MASK, a.hc, first_piece);
      const int kvh = hc / chunks, chunk = hc - kvh * chunks;
      if (from == 0 && to < n) {                    // goes on in other CTAs: to the one with the segment's end
        const long long end = cost_before(ri) + (long long)(hc + 1) * (n + SEGMENT_COST) - 1;
        chain = Chain{ri, hc, total < (1 << 30) ? (int)end / (int)share : (int)(end / share), 0};
      }
      // the next group's heads go to the warps behind this one's
      for (int h = (unsigned)(warp - grp * min(C::HEADS, p.group)) % C::WARPS; h < C::HEADS; h += C::WARPS) {
        const int hg = chunk * C::HEADS + h;
        if (hg >= p.group) continue;
        // the first four pieces' rows are on their way before the weights are known
        float x[4][VW];
        int j[4];
        unsigned rest = members;
        auto fetch = [&] {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            j[k] = rest ? __ffs(rest) - 1 : -1;
            const float* at_j = reinterpret_cast<const float*>(
                __shfl_sync(FULL_MASK, reinterpret_cast<unsigned long long>(a.at), j[k] & 31));
            rest &= rest - 1;
#pragma unroll
            for (int e = 0; e < VW; ++e) x[k][e] = 0.f;
            if (j[k] >= 0) load_lane<VW>(at_j + h * C::PROW + lane * VW, x[k]);
          }
        };
        fetch();
        const bool in = (members >> lane) & 1;
        const float pm = in ? a.at[C::HEADS * C::PROW + h] : -INFINITY;
        const float pl = in ? a.at[C::HEADS * C::PROW + C::HEADS + h] : 0.f;
        float mm = pm;
#pragma unroll
        for (int o = C::WARPS; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(FULL_MASK, mm, o));
        mm = __shfl_sync(FULL_MASK, mm, 0);
        const float w = exp2f(pm - (mm == -INFINITY ? 0.f : mm));
        float ll = 0.f, acc[VW] = {};
        while (true) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float wj = __shfl_sync(FULL_MASK, w, j[k] & 31), lj = __shfl_sync(FULL_MASK, pl, j[k] & 31);
            if (j[k] >= 0) {
              ll += wj * lj;
#pragma unroll
              for (int e = 0; e < VW; ++e) acc[e] += wj * x[k][e];
            }
          }
          if (!rest) break;
          fetch();
        }
        if (from == 0 && to == n) {
          const long long row = (long long)ri * p.h_q + kvh * p.group + hg;
          const float inv = inverse(ll) * value_scale<PAGES>(p, kvh);
#pragma unroll
          for (int e = 0; e < VW; ++e) acc[e] *= inv;
          store_lane<QTYPE, VW>(p.out, row * D + lane * VW, acc);
          if (p.lse && lane == 0) p.lse[row] = log_sum<BF16>(mm, ll);
        } else {
          float* dst = p.ws + ws_cta(C::PIECE, blockIdx.x, from == 0);
          save_lane<VW>(dst + h * C::PROW + lane * VW, acc);
          if (lane == 0) {
            dst[C::HEADS * C::PROW + h] = mm;
            dst[C::HEADS * C::PROW + C::HEADS + h] = ll;
          }
        }
      }
    }
    if (tid == 0 && !p.whole) reinterpret_cast<Chain*>(p.ws + ws_chain(C::PIECE, gridDim.x, C::WARPS))[blockIdx.x] = chain;
  }

  // ---- requests without a position
  for (int i = blockIdx.x; i < p.n_req; i += gridDim.x) {
    if (pre[i + 1] != pre[i]) continue;
    for (int e = tid; e < p.h_q * (D / 4); e += C::THREADS)
      store_out4<QTYPE>(p.out, (long long)i * p.h_q * D + e * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse)
      for (int h = tid; h < p.h_q; h += C::THREADS) p.lse[(long long)i * p.h_q + h] = -INFINITY;
  }
}

// The chains: block (cta, head) joins the pieces of the segment that starts in `cta`
// and goes on in cta + 1 .. last, for one head of the pass.  Every warp works out all
// pieces' weights (a lane per piece, five times over), then takes every eighth piece's
// row; the warps' sums are added in a fixed order.
constexpr int JOIN_WARPS = 8;

template <int D, int NT, int QTYPE, int PAGES>
__global__ void __launch_bounds__(32 * JOIN_WARPS) paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  using C = Cfg<D, NT, QTYPE, PAGES>;
  constexpr bool BF16 = QTYPE == HS_BF16 && PAGES == PAGES_SAME;
  constexpr int VW = D / 32, PER = PG_MAX_CTAS / 32;
  __shared__ float s_o[JOIN_WARPS][D];
  griddep_wait();
  griddep_launch_dependents();
  const int cta = blockIdx.x, h = blockIdx.y;
  const Chain ch = reinterpret_cast<const Chain*>(p.ws + ws_chain(C::PIECE, p.grid, C::WARPS))[cta];
  if (ch.last < 0) return;
  const int chunks = (p.group + C::HEADS - 1) / C::HEADS;
  const int kvh = ch.hc / chunks, hg = (ch.hc - kvh * chunks) * C::HEADS + h;
  if (hg >= p.group) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = ch.last - cta + 1;
  auto piece = [&](int j) { return p.ws + ws_cta(C::PIECE, cta + j, j == 0); };
  float m[PER], l[PER], mm = -INFINITY, ll = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = i * 32 + lane;
    m[i] = j < n ? piece(j)[C::HEADS * C::PROW + h] : -INFINITY;
    l[i] = j < n ? piece(j)[C::HEADS * C::PROW + C::HEADS + h] : 0.f;
  }
  float acc[VW] = {};
  float x[4][VW];
  auto fetch = [&](int i) {                // pieces warp + 8 (4 i + k) = 32 i + (warp + 8 k)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int e = 0; e < VW; ++e) x[k][e] = 0.f;
      const int j = 32 * i + warp + 8 * k;
      if (j < n) load_lane<VW>(piece(j) + h * C::PROW + lane * VW, x[k]);
    }
  };
  fetch(0);
#pragma unroll
  for (int i = 0; i < PER; ++i) mm = fmaxf(mm, m[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(FULL_MASK, mm, o));
  const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    m[i] = exp2f(m[i] - base);
    ll += m[i] * l[i];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ll += __shfl_xor_sync(FULL_MASK, ll, o);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (32 * i < n) {
      if (i) fetch(i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = __shfl_sync(FULL_MASK, m[i], warp + 8 * k);
#pragma unroll
        for (int e = 0; e < VW; ++e) acc[e] += w * x[k][e];
      }
    }
  }
  save_lane<VW>(&s_o[warp][lane * VW], acc);
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int g = 1; g < JOIN_WARPS; ++g) {
    float y[VW];
    load_lane<VW>(&s_o[g][lane * VW], y);
#pragma unroll
    for (int e = 0; e < VW; ++e) acc[e] += y[e];
  }
  const long long row = (long long)ch.ri * p.h_q + kvh * p.group + hg;
  const float inv = inverse(ll) * value_scale<PAGES>(p, kvh);
#pragma unroll
  for (int e = 0; e < VW; ++e) acc[e] *= inv;
  store_lane<QTYPE, VW>(p.out, row * D + lane * VW, acc);
  if (p.lse && lane == 0) p.lse[row] = log_sum<BF16>(mm, ll);
}

template <int D, int NT, int QTYPE, int PAGES, bool SCORES>
struct Kernels {
  using C = Cfg<D, NT, QTYPE, PAGES>;
  static cudaError_t prepare() {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, paged_join_kernel<D, NT, QTYPE, PAGES>);
    return e != cudaSuccess ? e : allow_smem(paged_decode_kernel<D, NT, QTYPE, PAGES, SCORES>, C::smem(PG_MAX_REQUESTS));
  }
  static cudaError_t launch(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) {
    const cudaError_t e = launch_pdl(paged_decode_kernel<D, NT, QTYPE, PAGES, SCORES>, dim3(p.grid), dim3(C::THREADS),
                                     C::smem(p.n_req), st, p, map);
    if (e != cudaSuccess || p.whole) return e;
    return launch_pdl(paged_join_kernel<D, NT, QTYPE, PAGES>, dim3(p.grid, C::HEADS), dim3(32 * JOIN_WARPS), 0, st, p);
  }
};

// f(kernels) for a configuration.  Query heads of a pass: up to 8 or 16 of a kv head's; more
// are taken in several passes over its rows.
template <int D, int PAGES, bool SCORES, typename F>
cudaError_t by_group(int group, int type, F f) {
  if (type == HS_BF16)
    return group <= 8 ? f(Kernels<D, 1, HS_BF16, PAGES, SCORES>{}) : f(Kernels<D, 2, HS_BF16, PAGES, SCORES>{});
  return group <= 8 ? f(Kernels<D, 1, HS_FP16, PAGES, SCORES>{}) : f(Kernels<D, 2, HS_FP16, PAGES, SCORES>{});
}

// The kernels of one head width and kind of page are compiled together (hs_paged_attention_*.cu).
template <int D, int PAGES, bool SCORES>
cudaError_t paged_decode_of(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st);
template <int D, int PAGES, bool SCORES>
cudaError_t prepare_paged_of(int group, int type);
#define HS_PAGED_DECODE_OF(D, PAGES, SCORES)                                                                  \
  template <>                                                                                                 \
  cudaError_t paged_decode_of<D, PAGES, SCORES>(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) { \
    return by_group<D, PAGES, SCORES>(p.group, p.type, [&](auto k) { return k.launch(p, map, st); });         \
  }                                                                                                           \
  template <>                                                                                                 \
  cudaError_t prepare_paged_of<D, PAGES, SCORES>(int group, int type) {                                       \
    return by_group<D, PAGES, SCORES>(group, type, [](auto k) { return k.prepare(); });                       \
  }

template <int D, int NT, int PAGES>
size_t ws_bytes(int grid) {
  using C = Cfg<D, NT, HS_BF16, PAGES>;
  return ws_chain(C::PIECE, grid, C::WARPS) * 4 + (size_t)grid * sizeof(Chain);
}

}  // namespace pa
}  // namespace hs

#endif  // HS_PAGED_ATTENTION_CUH_
