// Rows into 4-bit pages (hs_paged_append) and rows of any pages back as values
// (hs_paged_read): a warp moves the rows of one token, head by head, 1/32 of a row a lane.
//
// 4-bit rows.  x' = x / kv_scale (as a product with 1 / kv_scale, in 32 bits); 16 elements share
// s = e4m3(max |x'| / 7); code = clamp(round(x' / s), -7, 7) + 8, so a row stands for
// (code - 8) s kv_scale.  Both quotients are divisions rounded to nearest, so that the codes
// are those of the formula.  A scale rounded down by up to 2^-4 leaves |x' / s| up to
// 7.47: clamped, still within half a step.  7 / amax would waste the code 0 (-8), which rows
// may hold but none is given: levels that are symmetric about zero keep signs fair.
#include "hs_paged_place.cuh"

namespace hs {
namespace {

constexpr int ROWS_THREADS = 256;
constexpr int ROWS_WARPS = ROWS_THREADS / 32;
constexpr int ROWS_AHEAD = 8;      // rows of a warp on their way at once

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

// VW 16-bit elements as words
template <int VW>
struct Words {
  uint32_t w[VW / 2];
};
template <int VW>
__device__ __forceinline__ Words<VW> load_words(const uint16_t* p, bool wide) {
  Words<VW> x;
  if (wide) {
    if constexpr (VW == 2) x.w[0] = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (VW == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x.w[0] = v.x; x.w[1] = v.y;
    }
    if constexpr (VW == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      x.w[0] = v.x; x.w[1] = v.y; x.w[2] = v.z; x.w[3] = v.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VW / 2; ++e) x.w[e] = (uint32_t)p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
  }
  return x;
}
template <int VW>
__device__ __forceinline__ void store_words(uint16_t* p, const Words<VW>& x, bool wide) {
  if (wide) {
    if constexpr (VW == 2) *reinterpret_cast<uint32_t*>(p) = x.w[0];
    if constexpr (VW == 4) *reinterpret_cast<uint2*>(p) = make_uint2(x.w[0], x.w[1]);
    if constexpr (VW == 8) *reinterpret_cast<uint4*>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < VW / 2; ++e) {
      p[2 * e] = (uint16_t)x.w[e];
      p[2 * e + 1] = (uint16_t)(x.w[e] >> 16);
    }
  }
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

// VW elements of a lane -> 4-bit codes and its block's scale in the unit at `unit`
template <int VW>
__device__ __forceinline__ void store4(unsigned char* unit, bool values, int slot, const float (&x)[VW], float inv_scale) {
  constexpr int D = 32 * VW, PER = 16 / VW;              // lanes of a block
  const int lane = threadIdx.x & 31, e0 = lane * VW;
  float y[VW];
  unsigned top = 0;                                      // as whole numbers, so that a NaN is the largest
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    y[e] = x[e] * inv_scale;
    top = max(top, __float_as_uint(fabsf(y[e])));
  }
#pragma unroll
  for (int o = 1; o < PER; o <<= 1) top = max(top, __shfl_xor_sync(FULL_MASK, top, o));
  const unsigned char sb = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(top), 7.f), __NV_SATFINITE, __NV_E4M3);
  const float s = e4m3_up(sb);
  unsigned codes = 0;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const float q = s == 0.f ? 0.f : fminf(fmaxf(rintf(__fdiv_rn(y[e], s)), -7.f), 7.f);
    codes |= (unsigned)((int)q + 8) << (4 * e);
  }
  unsigned char* at = unit + code_at(D, values, slot, e0);
  if constexpr (VW == 2) *at = (unsigned char)codes;
  if constexpr (VW == 4) *reinterpret_cast<uint16_t*>(at) = (uint16_t)codes;
  if constexpr (VW == 8) *reinterpret_cast<uint32_t*>(at) = codes;
  if (lane % PER == 0) unit[scale_at(D, values, slot, e0 >> 4)] = sb;
}

template <typename T, int VW>
__global__ void __launch_bounds__(ROWS_THREADS) append4_kernel(const __grid_constant__ RotateParams p, bool interleaved, bool wide) {
  constexpr int D = 32 * VW;
  __shared__ float s_row[ROWS_WARPS][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vi = blockIdx.x >= p.first_cta[2] ? 2 : blockIdx.x >= p.first_cta[1] ? 1 : 0;
  const RowView& view = p.v[vi];
  const unsigned unit = (blockIdx.x - p.first_cta[vi]) * ROWS_WARPS + warp;
  const unsigned tu = unit / view.chunks;                // the token
  const bool mine = tu < (unsigned)p.n_tok;
  const int t = mine ? (int)tu : 0;
  const int h0 = (unit - tu * view.chunks) * view.chunk_heads;
  const int n = mine ? min(view.heads - h0, view.chunk_heads) : 0;
  const int e0 = lane * VW;
  griddep_wait();
  griddep_launch_dependents();
  const uint16_t* in = static_cast<const uint16_t*>(view.in) + t * view.in_ts + h0 * view.in_hs + e0;
  Words<VW> raw[ROWS_AHEAD];
#pragma unroll
  for (int i = 0; i < ROWS_AHEAD; ++i)
    if (i < n) raw[i] = load_words<VW>(in + i * view.in_hs, wide);

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
  float* row = s_row[warp];
  const int slot = tok.slot & (PG_UNIT - 1);
#pragma unroll
  for (int i = 0; i < ROWS_AHEAD; ++i) {
    if (i >= n) break;
    const int h = h0 + i;
    float x[VW];
#pragma unroll
    for (int e = 0; e < VW; e += 2) {
      const float2 v = Two<T>::up(raw[i].w[e / 2]);
      x[e] = v.x;
      x[e + 1] = v.y;
    }
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
        for (int e = 0; e < VW; ++e) row[e0 + e] = x[e];
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
      Words<VW> y;
#pragma unroll
      for (int e = 0; e < VW; e += 2) y.w[e / 2] = Two<T>::down(x[e], x[e + 1]);
      store_words<VW>(static_cast<uint16_t*>(view.out) + t * view.out_ts + h * view.out_hs + e0, y, wide);
    } else {
      const bool values = view.kind == VIEW_VALUES;
      const long long u = ((((long long)tok.page * 2 + values) * p.h_kv + h) << (p.page_shift - 4)) + (tok.slot >> 4);
      store4<VW>(p.pages + u * (9 * D), values, slot, x, 1.0f / p.kv_scale[values * p.h_kv + h]);
    }
  }
}

// A token's keys and values, [2][h_kv][d] of its output row.
template <typename T, int VW, int PAGES>
__global__ void __launch_bounds__(ROWS_THREADS) read_kernel(const __grid_constant__ RotateParams p) {
  constexpr int D = 32 * VW;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * VW;
  const RowView& view = p.v[0];
  const unsigned unit = blockIdx.x * ROWS_WARPS + warp;
  const unsigned tu = unit / view.chunks;
  const bool mine = tu < (unsigned)p.n_tok;
  const int t = mine ? (int)tu : 0;
  const int r0 = (unit - tu * view.chunks) * view.chunk_heads;
  const int n = mine ? min(view.heads - r0, view.chunk_heads) : 0;   // of 2 h_kv rows
  griddep_wait();
  griddep_launch_dependents();
  const Token tok = locate(p, t, mine);
  if (!mine || !tok.row) return;
  uint16_t* out = static_cast<uint16_t*>(view.out) + (long long)t * view.out_ts + (long long)r0 * D + e0;
  const bool held = tok.ok && tok.page >= 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    Words<VW> y = {};
    if (held) {
      const int which = r0 + i >= p.h_kv, h = r0 + i - which * p.h_kv;
      const long long row = ((((long long)tok.page * 2 + which) * p.h_kv + h) << p.page_shift) + tok.slot;
      if constexpr (PAGES == PAGES_SAME) {
        y = load_words<VW>(reinterpret_cast<const uint16_t*>(p.pages) + row * D + e0, true);
      } else {
        float x[VW];
        const float scale = p.kv_scale[which * p.h_kv + h];
        if constexpr (PAGES == PAGES_E4M3) {
          const unsigned char* b = p.pages + row * D + e0;
#pragma unroll
          for (int e = 0; e < VW; e += 2) {
            const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const uint16_t*>(b + e), __NV_E4M3);
            const float2 v = __half22float2(__half2(two));
            x[e] = v.x * scale;
            x[e + 1] = v.y * scale;
          }
        } else {
          const unsigned char* u = p.pages + (row >> 4) * (9 * D);
          const int slot = tok.slot & 15;
          const unsigned char* c = u + code_at(D, which, slot, e0);
          unsigned codes;
          if constexpr (VW == 2) codes = *c;
          if constexpr (VW == 4) codes = *reinterpret_cast<const uint16_t*>(c);
          if constexpr (VW == 8) codes = *reinterpret_cast<const uint32_t*>(c);
          const float s = e4m3_up(u[scale_at(D, which, slot, e0 >> 4)]);
#pragma unroll
          for (int e = 0; e < VW; ++e) x[e] = (float)((int)((codes >> (4 * e)) & 15) - 8) * s * scale;
        }
#pragma unroll
        for (int e = 0; e < VW; e += 2) y.w[e / 2] = Two<T>::down(x[e], x[e + 1]);
      }
    }
    store_words<VW>(out + (long long)i * D, y, true);
  }
}

// f(kernel of the element type and row width)
template <template <typename, int> class F, typename... A>
cudaError_t by_row(int type, int d, A... a) {
  if (type == HS_BF16)
    return d == 64 ? F<__nv_bfloat16, 2>::go(a...) : d == 128 ? F<__nv_bfloat16, 4>::go(a...) : F<__nv_bfloat16, 8>::go(a...);
  return d == 64 ? F<__half, 2>::go(a...) : d == 128 ? F<__half, 4>::go(a...) : F<__half, 8>::go(a...);
}

// Rows of a warp: as many as it has places for, fewer while the call has not 32 warps for each of 152 SMs.
bool split(RotateParams& p, int v, long long* cta) {
  const long long rows = (long long)p.n_tok * p.v[v].heads;
  p.v[v].chunk_heads = (int)std::min<long long>(std::min<int>(ROWS_AHEAD, p.v[v].heads), std::max<long long>(1, rows / (152 * 32)));
  p.v[v].chunks = (p.v[v].heads + p.v[v].chunk_heads - 1) / p.v[v].chunk_heads;
  const long long units = (long long)p.n_tok * p.v[v].chunks;
  p.first_cta[v] = (unsigned)*cta;
  *cta += (units + ROWS_WARPS - 1) / ROWS_WARPS;
  return units <= 0xf0000000LL && *cta <= 0x7fffffffLL;    // counted with 32 bits
}

template <typename T, int VW>
struct Append4 {
  static cudaError_t go(RotateParams p, bool interleaved, bool wide, cudaStream_t st) {
    long long cta = 0;
    if (p.n_views == 0) p.v[0].heads = p.v[0].chunks = p.v[0].chunk_heads = 1;   // no tokens: next_lengths only
    for (int v = 0; v < 3; ++v) {
      p.first_cta[v] = v ? 0xffffffffu : 0u;
      if (v < p.n_views && !split(p, v, &cta)) return cudaErrorInvalidConfiguration;
    }
    return launch_pdl(append4_kernel<T, VW>, dim3((unsigned)std::max(1LL, cta)), dim3(ROWS_THREADS), 0, st, p, interleaved, wide);
  }
};
template <typename T, int VW>
struct Read {
  template <typename K>
  static cudaError_t pick(int page_type, K f) {
    const Pages k = pages_kind(page_type);
    return k == PAGES_INT4 ? f(read_kernel<T, VW, PAGES_INT4>) : k == PAGES_E4M3 ? f(read_kernel<T, VW, PAGES_E4M3>) : f(read_kernel<T, VW, PAGES_SAME>);
  }
  static cudaError_t go(RotateParams p, int page_type, cudaStream_t st) {
    long long cta = 0;
    if (!split(p, 0, &cta)) return cudaErrorInvalidConfiguration;
    return pick(page_type, [&](auto kern) { return launch_pdl(kern, dim3((unsigned)cta), dim3(ROWS_THREADS), 0, st, p); });
  }
};
template <typename T, int VW>
struct Prepare {
  static cudaError_t go(int page_type) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaSuccess;
    if (page_type == HS_INT4) e = cudaFuncGetAttributes(&fa, append4_kernel<T, VW>);
    if (e != cudaSuccess) return e;
    return Read<T, VW>::pick(page_type, [&](auto kern) { return cudaFuncGetAttributes(&fa, kern); });
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
