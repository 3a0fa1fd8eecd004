// Rows into 4-bit pages (hs_paged_append) and rows of any pages back as values
// (hs_paged_read): a lane has eight elements of a row, a warp 256 / d rows of one token side by side.
//
// 4-bit rows.  x' = x / kv_scale (as a product with 1 / kv_scale, in 32 bits); 16 elements share
// s = e4m3(max |x'| / 7); code = clamp(round(x' / s), -7, 7) + 8, so a row stands for
// (code - 8) s kv_scale.  Both quotients are rounded as divisions are, so that the codes are
// those of the formula: q = a y with y the rounded reciprocal, then q + (a - q b) y, the
// remainder exact in a fused multiply-add.  (No quotient that is not a half itself is within
// 2^-24 of one: halves times s have 8 bits.)  A normal scale is rounded down by 2^-4 of itself at most,
// which leaves |x' / s| below 7.5 and every element within half a step; one below 2^-6 is a multiple
// k 2^-9, rounded by up to half of 2^-9, which leaves up to 7 (1 + 1 / 2k), 10.5 at k = 1: clamped to 7,
// up to 3.5 steps off.  7 / amax would waste the code 0 (-8), which rows may hold but none is given:
// levels that are symmetric about zero keep signs fair.
//
// Bound: instructions (70 to 77 % of the issue slots).  Measured (GB300): 24.1 K ragged tokens of 8 + 8
// heads of 128, fp16, stored in 60 us (a copy of the bytes: 19 us; 86 us with four elements a lane and
// divisions; 63 us where blocks are quiet enough to be clamped) and read back in 32 us (19 us), from 8-bit
// pages in 31 us (22 us), from 16-bit ones in 33 us (29 us).  With a rotation and 32 heads of queries: 243 us
// (77 us; into 8-bit pages, by their own kernel, 85 us); the sines of a lane's eight elements are worked out
// anew for every four of its rows.  16 tokens 2.8 us each way.
#include "hs_paged_attention.cuh"
#include "hs_paged_place.cuh"

namespace hs {
namespace {

constexpr int ROWS_THREADS = 256;
constexpr int ROWS_WARPS = ROWS_THREADS / 32;
constexpr int VW = 8;              // elements of a lane
constexpr int AHEAD = 4;           // rows of a lane on their way at once
template <int D>
constexpr int SIDE = 32 * VW / D;  // rows side by side in a warp

template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t u) { return make_float2(bf16lo(u), bf16hi(u)); }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct Two<__half> {
  static __device__ __forceinline__ float2 up(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// eight 16-bit elements as words
__device__ __forceinline__ uint4 load8(const uint16_t* p, bool wide) {
  if (wide) return *reinterpret_cast<const uint4*>(p);
  auto w = [&](int i) { return (uint32_t)p[i] | ((uint32_t)p[i + 1] << 16); };
  return make_uint4(w(0), w(2), w(4), w(6));
}
__device__ __forceinline__ void store8(uint16_t* p, uint4 x, bool wide) {
  if (wide) {
    *reinterpret_cast<uint4*>(p) = x;
  } else {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[2 * e] = (uint16_t)w[e];
      p[2 * e + 1] = (uint16_t)(w[e] >> 16);
    }
  }
}
template <typename T>
__device__ __forceinline__ void up8(uint4 x, float (&y)[VW]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = Two<T>::up(w[e]);
    y[2 * e] = v.x;
    y[2 * e + 1] = v.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 down8(const float (&x)[VW]) {
  return make_uint4(Two<T>::down(x[0], x[1]), Two<T>::down(x[2], x[3]), Two<T>::down(x[4], x[5]), Two<T>::down(x[6], x[7]));
}

__device__ __forceinline__ float e4m3_up(unsigned char b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// bytes of a lane's codes and of a block's scale within a unit, for row `slot` (0 .. 15) of it
__device__ __forceinline__ int code_at(int d, bool values, int slot, int e) {
  return values ? (e >> 5) * 256 + slot * 16 + ((e & 31) >> 1) : slot * (d >> 1) + (e >> 1);
}
__device__ __forceinline__ int scale_at(int d, bool values, int slot, int block) {
  return 8 * d + (values ? block * 16 + slot : slot * (d >> 4) + block);
}

// a lane's elements -> 4-bit codes, and its block's scale (of two lanes), in the unit at `unit`
template <int D>
__device__ __forceinline__ void store4(unsigned char* unit, bool values, int slot, int e0, const float (&x)[VW], float inv_scale, bool on) {
  float y[VW];
  unsigned top = 0;                                      // as whole numbers, so that a NaN is the largest
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    y[e] = x[e] * inv_scale;
    top = max(top, __float_as_uint(fabsf(y[e])));
  }
  top = max(top, __shfl_xor_sync(FULL_MASK, top, 1));
  constexpr float SEVENTH = 1.f / 7.f;
  const float a = fminf(__uint_as_float(top), 3e38f), q7 = a * SEVENTH;
  const unsigned char sb = top > 0x7f800000u
                               ? (unsigned char)0x7f
                               : __nv_cvt_float_to_fp8(fmaf(fmaf(-q7, 7.f, a), SEVENTH, q7), __NV_SATFINITE, __NV_E4M3);
  const float s = e4m3_up(sb), r = s == 0.f ? 0.f : __frcp_rn(s);
  // a normal scale keeps quotients below 7.5 up to 464 * 7; beyond, it stays at 448, and below 2^-6 (bytes 1 to
  // 7) it may be a third too small: there values are clamped (code 16 would be stored as 0, the other sign)
  if (__any_sync(FULL_MASK, __uint_as_float(top) > 3248.f || (unsigned)(sb - 1) < 7u)) {
    const float most = 7.f * s;
#pragma unroll
    for (int e = 0; e < VW; ++e) y[e] = fminf(fmaxf(y[e], -most), most);
  }
  unsigned codes = 0;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const float z = y[e], q = z * r;
    // the whole number in the low bits of a sum with 1.5 * 2^23 (rounded to nearest, ties to even), and 8
    const float n = fmaf(fmaf(-q, s, z), r, q) + 12582920.f;
    codes |= (__float_as_uint(n) & 15u) << (4 * e);
  }
  if (top > 0x7f800000u) codes = 0x11111111u;            // (any: the scale makes them NaN)
  if (!on) return;
  *reinterpret_cast<uint32_t*>(unit + code_at(D, values, slot, e0)) = codes;
  if ((e0 & 8) == 0) unit[scale_at(D, values, slot, e0 >> 4)] = sb;
}

template <typename T, int D>
__global__ void __launch_bounds__(ROWS_THREADS) append4_kernel(const __grid_constant__ RotateParams p, bool interleaved, bool wide) {
  __shared__ float s_row[ROWS_WARPS][32 * VW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = lane / (D / VW), e0 = lane % (D / VW) * VW;
  const int vi = blockIdx.x >= p.first_cta[2] ? 2 : blockIdx.x >= p.first_cta[1] ? 1 : 0;
  const RowView& view = p.v[vi];
  const unsigned unit = (blockIdx.x - p.first_cta[vi]) * ROWS_WARPS + warp;
  const unsigned tu = unit / view.chunks;                // the token
  const bool mine = tu < (unsigned)p.n_tok;
  const int t = mine ? (int)tu : 0;
  const int h0 = (unit - tu * view.chunks) * view.chunk_heads + side;
  const int h1 = mine ? min(view.heads, h0 - side + view.chunk_heads) : 0;
  const int steps = mine ? (h1 - (h0 - side) + SIDE<D> - 1) / SIDE<D> : 0;    // of the warp
  griddep_wait();
  griddep_launch_dependents();
  const uint16_t* in = static_cast<const uint16_t*>(view.in) + t * view.in_ts + h0 * view.in_hs + e0;
  uint4 raw[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (h0 + i * SIDE<D> < h1) raw[i] = load8(in + i * SIDE<D> * view.in_hs, wide);
  }

  write_next_lengths(p);
  if (p.n_tok == 0) return;
  __syncwarp();
  const Token tok = locate(p, t, mine);
  if (!mine || !tok.ok || (view.kind != VIEW_ROTATE && tok.page < 0)) return;

  // the pair of each of the lane's elements: its angle, its partner, its place in the pair
  const int half = p.rot_dim / 2;
  const bool turn = view.kind != VIEW_VALUES && p.rot_dim > 0;
  float cs[VW], sn[VW];
  if (turn) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int at = e0 + e;
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (at < p.rot_dim) {
        const int pair = interleaved ? at >> 1 : at < half ? at : at - half;
        const uint64_t angle = (uint64_t)(int64_t)tok.pos * p.turns[pair];
        const float x = (float)(int32_t)(angle >> 32) * (1.0f / 2147483648.0f);
        sincospif(x, &sn[e], &cs[e]);
        cs[e] *= p.magnitude;
        sn[e] *= p.magnitude;
      }
    }
  }
  float* row = s_row[warp] + side * D;
  const int slot = tok.slot & (PG_UNIT - 1);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    if (i >= steps) break;
    const int h = h0 + i * SIDE<D>;
    const bool on = h < h1;
    float x[VW];
    up8<T>(raw[i], x);
    if (turn) {
      float z[VW];                                       // the partners
      if (interleaved) {
#pragma unroll
        for (int e = 0; e < VW; e += 2) {
          z[e] = x[e + 1];
          z[e + 1] = x[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < VW; e += 4) *reinterpret_cast<float4*>(row + e0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const int at = e0 + e;
          z[e] = row[at < half ? at + half : at < p.rot_dim ? at - half : at];
        }
        __syncwarp();
      }
      // the roundings of each product and sum are those of the other pages' kernel
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const int at = e0 + e;
        const bool first = interleaved ? !(at & 1) : at < half;
        const float o = __fmul_rn(z[e], sn[e]);
        if (at < p.rot_dim) x[e] = __fmaf_rn(x[e], cs[e], first ? -o : o);
      }
    }
    if (view.kind == VIEW_ROTATE) {
      if (on) store8(static_cast<uint16_t*>(view.out) + t * view.out_ts + h * view.out_hs + e0, down8<T>(x), wide);
    } else {
      const bool values = view.kind == VIEW_VALUES;
      const long long u = ((((long long)tok.page * 2 + values) * p.h_kv + h) << (p.page_shift - 4)) + (tok.slot >> 4);
      store4<D>(p.pages + u * (9 * D), values, slot, e0, x, on ? 1.0f / p.kv_scale[values * p.h_kv + h] : 0.f, on);
    }
  }
}

// A token's keys and values, [2][h_kv][d] of its output row.
template <typename T, int D, int PAGES>
__global__ void __launch_bounds__(ROWS_THREADS) read_kernel(const __grid_constant__ RotateParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = lane / (D / VW), e0 = lane % (D / VW) * VW;
  const RowView& view = p.v[0];
  const unsigned unit = blockIdx.x * ROWS_WARPS + warp;
  const unsigned tu = unit / view.chunks;
  const bool mine = tu < (unsigned)p.n_tok;
  const int t = mine ? (int)tu : 0;
  const int r0 = (unit - tu * view.chunks) * view.chunk_heads + side;     // of 2 h_kv rows
  const int r1 = mine ? min(view.heads, r0 - side + view.chunk_heads) : 0;
  griddep_wait();
  griddep_launch_dependents();
  const Token tok = locate(p, t, mine);
  if (!mine || !tok.row) return;
  uint16_t* out = static_cast<uint16_t*>(view.out) + (long long)t * view.out_ts + e0;
  const bool held = tok.ok && tok.page >= 0;
  // every row's bytes on their way before the first is turned
  uint4 raw[AHEAD];
  uint32_t s[AHEAD];               // of a 4-bit row: the block's scale, twice
  float scale[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int r = r0 + i * SIDE<D>;
    raw[i] = make_uint4(0, 0, 0, 0);
    s[i] = 0;
    scale[i] = 0.f;
    if (!held || r >= r1) continue;
    const int which = r >= p.h_kv, h = r - which * p.h_kv;
    const long long row = ((((long long)tok.page * 2 + which) * p.h_kv + h) << p.page_shift) + tok.slot;
    if constexpr (PAGES != PAGES_SAME) scale[i] = p.kv_scale[r];
    if constexpr (PAGES == PAGES_SAME) raw[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.pages) + row * D + e0);
    if constexpr (PAGES == PAGES_E4M3) {
      const uint2 v = *reinterpret_cast<const uint2*>(p.pages + row * D + e0);
      raw[i].x = v.x;
      raw[i].y = v.y;
    }
    if constexpr (PAGES == PAGES_INT4) {
      const unsigned char* u = p.pages + (row >> 4) * (9 * D);
      raw[i].x = *reinterpret_cast<const uint32_t*>(u + code_at(D, which, tok.slot & 15, e0));
      s[i] = 0x101u * u[scale_at(D, which, tok.slot & 15, e0 >> 4)];
    }
  }
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int r = r0 + i * SIDE<D>;
    if (r >= r1) break;
    uint4 y = raw[i];
    if constexpr (PAGES != PAGES_SAME) {
      float x[VW];
      if constexpr (PAGES == PAGES_E4M3) {
#pragma unroll
        for (int e = 0; e < VW; e += 2) {
          const uint32_t w = e < 4 ? raw[i].x : raw[i].y;
          const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (e & 2 ? 16 : 0)), __NV_E4M3)));
          x[e] = v.x * scale[i];
          x[e + 1] = v.y * scale[i];
        }
      } else {
        // code times the block's scale as fp16, 2^-6 as large: exact; then one product in 32 bits
        uint32_t a[4];               // elements (0, 4), (1, 5), (2, 6), (3, 7)
        pa::int4x8_to_half2(raw[i].x, pa::int4_scale(pa::e4m3x2_to_half2((uint16_t)s[i])), a);
        const float by = scale[i] * pa::INT4_SHIFT;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&a[e]));
          x[e] = v.x * by;
          x[e + 4] = v.y * by;
        }
      }
      y = held ? down8<T>(x) : make_uint4(0, 0, 0, 0);
    }
    *reinterpret_cast<uint4*>(out + (long long)r * D) = y;
  }
}

// f(kernel of the element type and row width)
template <template <typename, int> class F, typename... A>
cudaError_t by_row(int type, int d, A... a) {
  if (type == HS_BF16)
    return d == 64 ? F<__nv_bfloat16, 64>::go(a...) : d == 128 ? F<__nv_bfloat16, 128>::go(a...) : F<__nv_bfloat16, 256>::go(a...);
  return d == 64 ? F<__half, 64>::go(a...) : d == 128 ? F<__half, 128>::go(a...) : F<__half, 256>::go(a...);
}

// Rows of a warp: as many as it has places for, fewer while the call has not 32 warps for each of 152 SMs.
bool split(RotateParams& p, int v, int side, long long* cta) {
  const long long rows = (long long)p.n_tok * p.v[v].heads;
  const long long each = std::max<long long>(1, rows / (152 * 32 * side));
  p.v[v].chunk_heads = (int)std::min<long long>(p.v[v].heads, std::min<long long>(AHEAD, each) * side);
  p.v[v].chunks = (p.v[v].heads + p.v[v].chunk_heads - 1) / p.v[v].chunk_heads;
  const long long units = (long long)p.n_tok * p.v[v].chunks;
  p.first_cta[v] = (unsigned)*cta;
  *cta += (units + ROWS_WARPS - 1) / ROWS_WARPS;
  return units <= 0xf0000000LL && *cta <= 0x7fffffffLL;    // counted with 32 bits
}

template <typename T, int D>
struct Append4 {
  static cudaError_t go(RotateParams p, bool interleaved, bool wide, cudaStream_t st) {
    long long cta = 0;
    if (p.n_views == 0) p.v[0].heads = p.v[0].chunks = p.v[0].chunk_heads = 1;   // no tokens: next_lengths only
    for (int v = 0; v < 3; ++v) {
      p.first_cta[v] = v ? 0xffffffffu : 0u;
      if (v < p.n_views && !split(p, v, SIDE<D>, &cta)) return cudaErrorInvalidConfiguration;
    }
    return launch_pdl(append4_kernel<T, D>, dim3((unsigned)std::max(1LL, cta)), dim3(ROWS_THREADS), 0, st, p, interleaved, wide);
  }
};
template <typename T, int D>
struct Read {
  template <typename K>
  static cudaError_t pick(int page_type, K f) {
    const Pages k = pages_kind(page_type);
    return k == PAGES_INT4 ? f(read_kernel<T, D, PAGES_INT4>) : k == PAGES_E4M3 ? f(read_kernel<T, D, PAGES_E4M3>) : f(read_kernel<T, D, PAGES_SAME>);
  }
  static cudaError_t go(RotateParams p, int page_type, cudaStream_t st) {
    long long cta = 0;
    if (!split(p, 0, SIDE<D>, &cta)) return cudaErrorInvalidConfiguration;
    return pick(page_type, [&](auto kern) { return launch_pdl(kern, dim3((unsigned)cta), dim3(ROWS_THREADS), 0, st, p); });
  }
};
template <typename T, int D>
struct Prepare {
  static cudaError_t go(int page_type) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaSuccess;
    if (page_type == HS_INT4) e = cudaFuncGetAttributes(&fa, append4_kernel<T, D>);
    if (e != cudaSuccess) return e;
    return Read<T, D>::pick(page_type, [&](auto kern) { return cudaFuncGetAttributes(&fa, kern); });
  }
};

}  // namespace

cudaError_t launch_append4(const RotateParams& p, int type, bool interleaved, bool wide, cudaStream_t st) {
  return by_row<Append4>(type, p.d, p, interleaved, wide, st);
}
cudaError_t launch_read(const RotateParams& p, int type, int page_type, cudaStream_t st) {
  return by_row<Read>(type, p.d, p, page_type, st);
}
cudaError_t prepare_rows(int d, int type, int page_type) { return by_row<Prepare>(type, d, page_type); }

}  // namespace hs
