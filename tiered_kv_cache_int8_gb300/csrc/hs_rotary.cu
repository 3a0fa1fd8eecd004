// Rotary positions, alone (hs_rotary_apply) and on the way into a paged cache
// (hs_paged_append): one kernel template moves head rows and turns the pairs of
// their first rot_dim elements.
//
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t),  t = position * f
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: position times
// the table entry wraps modulo one turn exactly, so a position of a million loses
// nothing (in 32-bit floats its angle would be off by 0.06 rad); the top 32 bits
// then go through sincospi.  The cosines and sines of a CTA's tokens are computed
// once per pair, into shared memory, and serve every head.
//
// Memory-bound: each element is read and written once, 16 bytes at a time where
// the views allow it.
#include "hs_paged.cuh"

namespace hs {
namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_MAX_TOK = 4;   // tokens of a CTA

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};

// VEC consecutive elements: one 16-byte access, or one element (VEC = 1).
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T* p, T (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = p[0];
  } else {
    static_assert(sizeof(T) * VEC == 16, "16-byte accesses");
    *reinterpret_cast<int4*>(x) = *reinterpret_cast<const int4*>(p);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const float (&x)[VEC]) {
  alignas(16) T y[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) y[i] = Elem<T>::down(x[i]);
  if constexpr (VEC == 1) {
    p[0] = y[0];
  } else {
    *reinterpret_cast<int4*>(p) = *reinterpret_cast<const int4*>(y);
  }
}
// the same into 8-bit pages: value / scale, saturated (a NaN stays one)
template <int VEC>
__device__ __forceinline__ void store_e4m3(unsigned char* p, const float (&x)[VEC], float scale) {
  alignas(8) unsigned char y[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) y[i] = __nv_cvt_float_to_fp8(__fdiv_rn(x[i], scale), __NV_SATFINITE, __NV_E4M3);
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(y);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = y[i];
  }
}

// Where a token goes: its position, and its page row (pages of the layer are
// [n_pages][2][h_kv][page_size] rows), -1 where it is not stored.
struct Token {
  int pos;        // its position
  int ok;         // 0: the token belongs to no request of the call (nothing is read or written)
  int page, slot; // page < 0: not stored
};

// The request of token row t: the last i with tok_offsets[i] <= t, found by one
// warp, 32 probes at a time.
__device__ __forceinline__ int request_of(const int32_t* offs, int n_req, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_req;                       // offs[lo] <= t < offs[hi] if the offsets are sound
  while (hi - lo > 1) {
    const int n = hi - lo - 1;                  // interior entries lo + 1 .. hi - 1
    const int step = (n + 31) / 32;
    const int at = lo + 1 + lane * step;
    const bool below = at < hi && offs[at] <= t;
    const unsigned m = __ballot_sync(FULL_MASK, below);
    const int c = __popc(m);                    // probes at or below t (sound offsets: a prefix of the lanes)
    const int nlo = c ? lo + 1 + (c - 1) * step : lo;
    const int nhi = min(hi, lo + 1 + c * step);
    lo = min(nlo, hi - 1);
    hi = max(nhi, lo + 1);
  }
  return lo;
}

// new tokens of request i of the call; 0 with an error bit for unsound offsets
__device__ __forceinline__ int new_tokens(const RotateParams& p, int i, int* first, unsigned* err) {
  if (!p.tok_offsets) {
    *first = i * p.tok_per_req;
    return p.tok_per_req;
  }
  const int a = p.tok_offsets[i], b = p.tok_offsets[i + 1];
  *first = a;
  if (a < 0 || b < a || b > p.n_tok) {
    *err |= HS_DEVERR_OFFSETS;
    return 0;
  }
  return b - a;
}

// whether request `req` takes `n` tokens on its `len` positions
__device__ __forceinline__ bool takes(const RotateParams& p, int req, int len, int n, unsigned* err) {
  if (len < 0 || (long long)len + n > (long long)p.max_pages << p.page_shift) {
    *err |= HS_DEVERR_CAPACITY;
    return false;
  }
  return true;
}

__device__ Token locate(const RotateParams& p, int t) {   // one warp
  Token k = {0, 0, -1, 0};
  unsigned err = 0;
  const int i = p.tok_offsets ? request_of(p.tok_offsets, p.n_req, t) : t / p.tok_per_req;
  int first;
  const int n = new_tokens(p, i, &first, &err);
  const int j = t - first;
  if (j >= 0 && j < n) {
    const int req = p.req_ids ? p.req_ids[i] : i;
    if (req < 0 || req >= p.max_requests) {
      err |= HS_DEVERR_REQ_RANGE;
    } else {
      const int len = p.lengths[req];
      if (takes(p, req, len, n, &err)) {
        k.ok = 1;
        k.pos = len + j;
        const int page = p.page_table[(long long)req * p.max_pages + (k.pos >> p.page_shift)];
        k.slot = k.pos & (p.page_size - 1);
        if (page >= 0 && page < p.n_pages)
          k.page = page;
        else
          err |= HS_DEVERR_PAGE;
      }
    }
  }
  if (err && (threadIdx.x & 31) == 0) set_error(p.dev_error, err);
  return k;
}

// T: the views' type; VEC: elements per access; INTER: pairs (2i, 2i+1) instead of
// (i, i + rot/2); APPEND: positions from lengths, views of kind KEYS and VALUES go
// to the pages (E4M3: 8-bit pages).
//
// Work items of a row, in order: half layout: rot / (2 VEC) items of two accesses
// (i and i + rot/2), then (d - rot) / VEC copies; interleaved: d / VEC accesses.
template <typename T, int VEC, bool INTER, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(ROT_THREADS) rotate_kernel(const __grid_constant__ RotateParams p) {
  extern __shared__ float2 s_cs[];              // [tok_per_cta][rot / 2]: (cos, sin) times magnitude
  __shared__ Token s_tok[ROT_MAX_TOK];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * p.tok_per_cta;
  const int nt = min(p.tok_per_cta, p.n_tok - t0);
  if constexpr (APPEND) {
    for (int w = tid >> 5; w < nt; w += ROT_THREADS / 32) {
      const Token k = locate(p, t0 + w);
      if ((tid & 31) == 0) s_tok[w] = k;
    }
    if (p.next_lengths) {
      for (int i = blockIdx.x * ROT_THREADS + tid; i < p.n_req; i += gridDim.x * ROT_THREADS) {
        const int req = p.req_ids ? p.req_ids[i] : i;
        unsigned err = 0;
        int first;
        const int n = new_tokens(p, i, &first, &err);
        if (req < 0 || req >= p.max_requests) {
          err |= HS_DEVERR_REQ_RANGE;
        } else {
          const int len = p.lengths[req];
          p.next_lengths[req] = takes(p, req, len, n, &err) ? len + n : len;
        }
        if (err) set_error(p.dev_error, err);
      }
    }
    if (nt <= 0) return;
    __syncthreads();
  }
  const int half = p.rot_dim / 2;
  for (int e = tid; e < nt * half; e += ROT_THREADS) {
    const int t = e / half, i = e - t * half;
    int pos;
    if constexpr (APPEND) pos = s_tok[t].pos; else pos = p.positions[t0 + t];
    const uint64_t turn = (uint64_t)(int64_t)pos * p.turns[i];
    // the top 32 bits, signed: a fraction of a turn in [-1/2, 1/2)
    const float x = (float)(int32_t)(turn >> 32) * (1.0f / 2147483648.0f);
    float s, c;
    sincospif(x, &s, &c);
    s_cs[e] = make_float2(c * p.magnitude, s * p.magnitude * p.sign);
  }
  __syncthreads();

  const int n_turn = INTER ? p.rot_dim / VEC : half / VEC;   // items that turn pairs (VEC = 1, INTER: see below)
  const int per = p.items;
  for (int it = tid; it < nt * p.rows * per; it += ROT_THREADS) {
    const int j = it % per;
    const int r = it / per;
    const int t = r / p.rows;
    int h = r - t * p.rows;
    int v = 0;
    while (h >= p.v[v].heads) h -= p.v[v++].heads;
    const RowView& view = p.v[v];
    Token tok = {0, 1, 0, 0};
    if constexpr (APPEND) {
      tok = s_tok[t];
      if (!tok.ok || (view.kind != VIEW_ROTATE && tok.page < 0)) continue;
    }
    const T* in = static_cast<const T*>(view.in) + (t0 + t) * view.in_ts + h * view.in_hs;
    T* out = nullptr;
    unsigned char* out8 = nullptr;
    float scale = 1.0f;
    if (!APPEND || view.kind == VIEW_ROTATE) {
      out = static_cast<T*>(view.out) + (t0 + t) * view.out_ts + h * view.out_hs;
    } else {
      const int which = view.kind == VIEW_VALUES;
      const long long row = ((((long long)tok.page * 2 + which) * p.h_kv + h) << p.page_shift) + tok.slot;
      if constexpr (E4M3) {
        out8 = p.pages + row * p.d;
        scale = p.kv_scale[which * p.h_kv + h];
      } else {
        out = reinterpret_cast<T*>(p.pages) + row * p.d;
      }
    }
    auto put = [&](int at, const float (&y)[VEC]) {
      if (E4M3 && out8)
        store_e4m3<VEC>(out8 + at, y, scale);
      else
        store_row<T, VEC>(out + at, y);
    };
    const bool turn = view.kind != VIEW_VALUES;
    const float2* cs = s_cs + t * half;
    if (INTER && VEC > 1) {
      alignas(16) T x[VEC];
      float y[VEC];
      load_row<T, VEC>(in + j * VEC, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = Elem<T>::up(x[e]);
      if (turn && j < n_turn) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 w = cs[(j * VEC + e) / 2];
          const float a = y[e], b = y[e + 1];
          y[e] = a * w.x - b * w.y;
          y[e + 1] = b * w.x + a * w.y;
        }
      }
      put(j * VEC, y);
    } else {
      // pairs at (ia, ib): VEC of them per item; VEC = 1 takes either layout
      const int pairs = half / VEC;
      if (j < pairs) {
        const int ia = INTER ? 2 * j : j * VEC, ib = INTER ? 2 * j + 1 : half + j * VEC;
        alignas(16) T xa[VEC];
        alignas(16) T xb[VEC];
        float ya[VEC], yb[VEC];
        load_row<T, VEC>(in + ia, xa);
        load_row<T, VEC>(in + ib, xb);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float a = Elem<T>::up(xa[e]), b = Elem<T>::up(xb[e]);
          const float2 w = turn ? cs[j * VEC + e] : make_float2(1.f, 0.f);
          ya[e] = turn ? a * w.x - b * w.y : a;
          yb[e] = turn ? b * w.x + a * w.y : b;
        }
        put(ia, ya);
        put(ib, yb);
      } else {
        const int at = p.rot_dim + (j - pairs) * VEC;
        alignas(16) T x[VEC];
        float y[VEC];
        load_row<T, VEC>(in + at, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = Elem<T>::up(x[e]);
        put(at, y);
      }
    }
  }
}

template <typename T, int VEC, bool INTER, bool APPEND, bool E4M3>
cudaError_t go(RotateParams p, cudaStream_t st) {
  const int half = p.rot_dim / 2;
  p.items = INTER && VEC > 1 ? p.d / VEC : half / VEC + (p.d - p.rot_dim) / VEC;
  p.tok_per_cta = p.n_tok >= 4 * 152 * ROT_MAX_TOK ? ROT_MAX_TOK : 1;
  const int grid = std::max(1, (p.n_tok + p.tok_per_cta - 1) / p.tok_per_cta);
  const size_t smem = (size_t)p.tok_per_cta * half * sizeof(float2);
  return launch_pdl(rotate_kernel<T, VEC, INTER, APPEND, E4M3>, dim3(grid), dim3(ROT_THREADS), smem, st, p);
}

template <typename T, int W, bool APPEND, bool E4M3>
cudaError_t pick(const RotateParams& p, bool interleaved, bool wide, cudaStream_t st) {
  if (wide) return interleaved ? go<T, W, true, APPEND, E4M3>(p, st) : go<T, W, false, APPEND, E4M3>(p, st);
  return interleaved ? go<T, 1, true, APPEND, E4M3>(p, st) : go<T, 1, false, APPEND, E4M3>(p, st);
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int type, int page_type, bool append, bool interleaved,
                          bool wide, cudaStream_t st) {
  const bool e = page_type == HS_E4M3;
  if (append) {
    if (type == HS_BF16)
      return e ? pick<__nv_bfloat16, 8, true, true>(p, interleaved, wide, st)
               : pick<__nv_bfloat16, 8, true, false>(p, interleaved, wide, st);
    return e ? pick<__half, 8, true, true>(p, interleaved, wide, st)
             : pick<__half, 8, true, false>(p, interleaved, wide, st);
  }
  if (type == HS_BF16) return pick<__nv_bfloat16, 8, false, false>(p, interleaved, wide, st);
  if (type == HS_FP16) return pick<__half, 8, false, false>(p, interleaved, wide, st);
  return pick<float, 4, false, false>(p, interleaved, wide, st);
}

}  // namespace hs
