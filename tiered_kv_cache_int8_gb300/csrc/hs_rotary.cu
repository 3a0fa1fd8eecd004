// Rotary positions, alone (hs_rotary_apply) and on the way into a paged cache
// (hs_paged_append): one kernel template moves head rows and turns the pairs of
// their first rot_dim elements.
//
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t),  t = position * f
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: position times
// the table entry wraps modulo one turn exactly, so a position of a million loses
// nothing (in 32-bit floats its angle would be off by 0.06 rad); the top 32 bits
// then go through sincospi, as a float of half turns: rounded to 24 bits, the angle is
// off by up to 2^-25 of half a turn, 9e-8 rad.  That is most of a step of an fp32 output (relative
// error of a rotation in fp32 5.5e-8, with angles in 64 bits 4.2e-8) and nothing in 16 bits.
//
// Memory-bound: each element is read and written once, 16 bytes at a time where
// the views allow it.  Measured (GB300, copy rate 6.7 TB/s): 32768 tokens of 40 heads
// of 128, bf16: 98 us, 6.9 TB/s; 20 K tokens of 32 + 8 + 8 heads into 8-bit pages: 73
// us, 6.3 TB/s (issue slots 70 % busy); 16 tokens: 1.9 us, and 2.8 us into pages.
#include "hs_paged.cuh"

namespace hs {
namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_AHEAD = 128;    // most bytes of a thread in flight (256: no faster, fewer CTAs an SM)
constexpr int LENGTH_CTAS = PG_MAX_REQUESTS / ROT_THREADS;   // CTAs that write next_lengths

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  using Two = __nv_bfloat162;
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ Two down2(float x, float y) { return __floats2bfloat162_rn(x, y); }
};
template <>
struct Elem<__half> {
  using Two = __half2;
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ Two down2(float x, float y) { return __floats2half2_rn(x, y); }
};
template <>
struct Elem<float> {
  using Two = float2;
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
  static __device__ __forceinline__ Two down2(float x, float y) { return make_float2(x, y); }
};

// VEC consecutive elements: one 16-byte store, or one element (VEC = 1).
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = Elem<T>::down(x[0]);
  } else {
    alignas(16) typename Elem<T>::Two y[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC; i += 2) y[i / 2] = Elem<T>::down2(x[i], x[i + 1]);
    *reinterpret_cast<int4*>(p) = *reinterpret_cast<const int4*>(y);
  }
}
// the same into 8-bit pages: times 1 / scale, saturated (a NaN stays one)
template <int VEC>
__device__ __forceinline__ void store_e4m3(unsigned char* p, const float (&x)[VEC], float inv_scale) {
  if constexpr (VEC == 1) {
    p[0] = __nv_cvt_float_to_fp8(x[0] * inv_scale, __NV_SATFINITE, __NV_E4M3);
  } else {
    static_assert(VEC == 8, "8-byte stores");
    alignas(8) __nv_fp8x2_storage_t y[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
      y[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(x[i] * inv_scale, x[i + 1] * inv_scale), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(y);
  }
}

// One rounding of each product and sum is fixed here, so that every variant of the
// kernel (access widths, layouts, alone or on the way into the pages) gives the same bits.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = x;
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

// rows from offset a to b; none, with an error bit, for unsound ones
__device__ __forceinline__ int count_rows(const RotateParams& p, int a, int b, unsigned* err) {
  if (a >= 0 && b >= a && b <= p.n_tok) return b - a;
  *err |= HS_DEVERR_OFFSETS;
  return 0;
}

// new tokens of request i of the call
__device__ __forceinline__ int new_tokens(const RotateParams& p, int i, int* first, unsigned* err) {
  if (!p.tok_offsets) {
    *first = i * p.tok_per_req;
    return p.tok_per_req;
  }
  *first = p.tok_offsets[i];
  return count_rows(p, *first, p.tok_offsets[i + 1], err);
}

// whether request `req` takes `n` tokens on its `len` positions
__device__ __forceinline__ bool takes(const RotateParams& p, int req, int len, int n, unsigned* err) {
  if (len < 0 || (long long)len + n > (long long)p.max_pages << p.page_shift) {
    *err |= HS_DEVERR_CAPACITY;
    return false;
  }
  return true;
}

// The place of token row t of request i of the call, whose rows are first .. first + n - 1.
// `len`: the request's length where it is known already, else null.
__device__ __forceinline__ Token place_of(const RotateParams& p, int t, int i, int first, int n, int req,
                                          const int* len, unsigned err) {
  Token k = {0, 0, -1, 0};
  const int j = t - first;
  if (j >= 0 && j < n) {
    if (req < 0 || req >= p.max_requests) {
      err |= HS_DEVERR_REQ_RANGE;
    } else {
      const int held = len ? *len : p.lengths[req];
      if (takes(p, req, held, n, &err)) {
        k.ok = 1;
        k.pos = held + j;
        const int page = p.page_table[(long long)req * p.max_pages + (k.pos >> p.page_shift)];
        k.slot = k.pos & (p.page_size - 1);
        if (page >= 0 && page < p.n_pages)
          k.page = page;
        else
          err |= HS_DEVERR_PAGE;
      }
    }
  }
  if (err) set_error(p.dev_error, err);
  return k;
}

// The place of each lane's token row t (one warp; lanes without a token give any).
__device__ Token locate(const RotateParams& p, int t, bool mine) {
  const int lane = threadIdx.x & 31;
  unsigned err = 0;
  int i, first, n;
  if (!p.tok_offsets) {
    i = t / p.tok_per_req;
    first = i * p.tok_per_req;
    n = p.tok_per_req;
  } else if (p.n_req <= 32) {
    // lane i reads request i's offset, id and length, all at once; then nothing is left to read
    // but the page id (the search below takes three dependent reads more: 3.1 instead of 2.8 us
    // for 16 requests of one token)
    const int off = p.tok_offsets[min(lane, p.n_req)], end = p.tok_offsets[p.n_req];
    const int id = lane < p.n_req ? (p.req_ids ? p.req_ids[lane] : lane) : -1;
    int len = id >= 0 && id < p.max_requests ? p.lengths[id] : -1;
    i = 0;
#pragma unroll
    for (int s = 16; s; s >>= 1) {
      const int at = __shfl_sync(FULL_MASK, off, (i + s) & 31);
      if (i + s < p.n_req && at <= t) i += s;
    }
    first = __shfl_sync(FULL_MASK, off, i);
    const int next = __shfl_sync(FULL_MASK, off, (i + 1) & 31);
    n = count_rows(p, first, i + 1 < p.n_req ? next : end, &err);
    const int req = __shfl_sync(FULL_MASK, id, i);
    len = __shfl_sync(FULL_MASK, len, i);
    return mine ? place_of(p, t, i, first, n, req, &len, err) : Token{0, 0, -1, 0};
  } else {
    // the request of the warp's first token, then each lane's from there (tokens do not descend
    // along a warp): strides that double, then halve
    i = request_of(p.tok_offsets, p.n_req, __reduce_min_sync(FULL_MASK, mine ? t : p.n_tok - 1));
    int hi = i + 1, step = 1;
    while (hi < p.n_req && p.tok_offsets[hi] <= t) {
      i = hi;
      step <<= 1;
      hi = min(p.n_req, hi + step);
    }
    while (hi - i > 1) {
      const int mid = (i + hi) >> 1;
      if (p.tok_offsets[mid] <= t) i = mid; else hi = mid;
    }
    n = new_tokens(p, i, &first, &err);
  }
  if (!mine) return Token{0, 0, -1, 0};
  return place_of(p, t, i, first, n, p.req_ids ? p.req_ids[i] : i, nullptr, err);
}

// T: the views' type; VEC: elements per access; INTER: pairs (2i, 2i+1) instead of
// (i, i + rot/2); APPEND: positions from lengths, views of kind KEYS and VALUES go
// to the pages (E4M3: 8-bit pages).
//
// Work items of a row, in order: half layout (and VEC = 1): rot / (2 VEC) items of two
// accesses (i and i + rot/2), then the rest of the row by two accesses (single ones kept
// half the bytes in flight: 132 instead of 96 us for 32768 tokens of 40 heads of 128 with
// a quarter rotated); interleaved: d / VEC accesses.
// A thread has one item of one token and goes down the token's heads with it, so the
// cosines and sines of its pairs are computed once, by it, and stay in registers: no
// table, no barrier, and the next head is a stride further.  All its heads start on
// their way into shared memory (each thread's own 16-byte places: nothing to wait for but
// its own copies) before the token's position and pages are looked up, which takes five
// dependent reads: with the next heads in registers instead, those reads and the latency
// of each pair of heads were exposed (20 K tokens of 48 heads into 8-bit pages: 103 us;
// now 75 us, 6.2 TB/s).  A view's heads are split over several threads, fewer each
// where there are few tokens.
template <typename T, int VEC_, bool INTER>
struct Shape {
  static constexpr int VEC = VEC_;
  static constexpr bool PAIRS = INTER && VEC > 1;              // both elements of a pair in one access
  static constexpr int PER_ITEM = PAIRS ? VEC / 2 : VEC;       // pairs of an item
  static constexpr int ACCESSES = PAIRS ? 1 : 2;
  static constexpr int GROUPS = 4;                             // copies are waited for in this many steps
  static constexpr int STEP = VEC > 1 ? ROT_AHEAD / (16 * ACCESSES * GROUPS) : 1;   // heads of a step
  static constexpr int HEADS = STEP * GROUPS;                  // most heads of a thread
  // rows taken by single elements may need 512 threads
  static constexpr int MAX_THREADS = VEC > 1 ? ROT_THREADS : 512;
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_left(int n) {   // n: a constant once unrolled
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

template <typename T, int VEC, bool INTER, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(Shape<T, VEC, INTER>::MAX_THREADS, VEC > 1 ? 4 : 1)
    rotate_kernel(const __grid_constant__ RotateParams p) {
  using S = Shape<T, VEC, INTER>;
  const int tid = threadIdx.x;
  const int vi = blockIdx.x >= p.first_cta[2] ? 2 : blockIdx.x >= p.first_cta[1] ? 1 : 0;
  const RowView& view = p.v[vi];
  const int per = p.items, half = p.rot_dim / 2;
  const int pairs = half / S::PER_ITEM;         // items that turn pairs
  const int grp = tid / per, j = tid - grp * per;
  const unsigned unit = (blockIdx.x - p.first_cta[vi]) * p.groups + grp;
  const unsigned tu = unit / view.chunks;       // the token
  const int chunk = unit - tu * view.chunks;
  const bool mine = grp < p.groups && tu < (unsigned)p.n_tok;
  const int t = mine ? (int)tu : 0;
  int h = chunk * view.chunk_heads;
  const int h1 = mine ? min(view.heads, h + view.chunk_heads) : h;
  griddep_wait();
  griddep_launch_dependents();

  const T* in = static_cast<const T*>(view.in) + t * view.in_ts + h * view.in_hs;
  // the item's places in a row
  const int rest = p.rot_dim + (j - pairs) * VEC;   // of an item behind the pairs: neighbours side by side, twice
  const int ia = S::PAIRS ? j * VEC : j >= pairs ? rest : INTER ? 2 * j : j * VEC;
  const int ib = j >= pairs ? rest + (per - pairs) * VEC : INTER ? 2 * j + 1 : half + j * VEC;
  const bool two = !S::PAIRS && ib < p.d;
  const long long in_hs = view.in_hs;
  extern __shared__ int4 s_in[];                // [head][access][thread]
  if constexpr (VEC > 1) {
#pragma unroll
    for (int g = 0; g < S::GROUPS; ++g) {
#pragma unroll
      for (int i = 0; i < S::STEP; ++i) {
        const int u = g * S::STEP + i;
        if (h + u < h1) {
          cp_async_16(&s_in[(u * S::ACCESSES) * ROT_THREADS + tid], in + u * in_hs + ia);
          if (two) cp_async_16(&s_in[(u * S::ACCESSES + 1) * ROT_THREADS + tid], in + u * in_hs + ib);
        }
      }
      cp_async_commit();
    }
  }

  const int kind = APPEND ? view.kind : VIEW_ROTATE;
  const bool turn = kind != VIEW_VALUES && j < pairs;
  int pos = 0;
  Token tok = {0, 1, -1, 0};
  if constexpr (APPEND) {
    // the first CTAs only: blockIdx.x * blockDim.x of all of them may pass 32 bits
    if (p.next_lengths && blockIdx.x < LENGTH_CTAS) {
      const int ctas = min(gridDim.x, (unsigned)LENGTH_CTAS);
      for (int i = blockIdx.x * blockDim.x + tid; i < p.n_req; i += ctas * blockDim.x) {
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
    if (p.n_tok == 0) return;
    __syncwarp();
    tok = locate(p, t, mine);
    pos = tok.pos;
  } else {
    if (mine) pos = p.positions[t];
  }
  if (!mine) return;

  float cs[S::PER_ITEM], sn[S::PER_ITEM];
  if (turn) {
#pragma unroll
    for (int e = 0; e < S::PER_ITEM; ++e) {
      const uint64_t angle = (uint64_t)(int64_t)pos * p.turns[j * S::PER_ITEM + e];
      // the top 32 bits, signed: a fraction of a turn in [-1/2, 1/2)
      const float x = (float)(int32_t)(angle >> 32) * (1.0f / 2147483648.0f);
      sincospif(x, &sn[e], &cs[e]);
      cs[e] *= p.magnitude;
      sn[e] *= p.magnitude * p.sign;
    }
  }

  T* out = nullptr;
  unsigned char* out8 = nullptr;
  long long out_hs = view.out_hs;
  const float* scale = nullptr;
  if (APPEND && (kind == VIEW_ROTATE ? !tok.ok : tok.page < 0)) {   // nothing to store
    cp_async_wait_all();
    return;
  }
  if (kind == VIEW_ROTATE) {
    out = static_cast<T*>(view.out) + t * view.out_ts + h * out_hs;
  } else {
    const int which = kind == VIEW_VALUES;
    const long long row = ((((long long)tok.page * 2 + which) * p.h_kv + h) << p.page_shift) + tok.slot;
    out_hs = (long long)p.d << p.page_shift;
    if constexpr (E4M3) {
      out8 = p.pages + row * p.d;
      scale = p.kv_scale + which * p.h_kv;
    } else {
      out = reinterpret_cast<T*>(p.pages) + row * p.d;
    }
  }
#pragma unroll
  for (int g = 0; g < S::GROUPS; ++g) {
    if (h + g * S::STEP >= h1) break;
    if constexpr (VEC > 1) cp_async_left(S::GROUPS - 1 - g);
#pragma unroll
    for (int i = 0; i < S::STEP; ++i) {
      const int u = g * S::STEP + i;
      if (h + u < h1) {
        alignas(16) T xa[VEC];
        alignas(16) T xb[VEC];
        if constexpr (VEC > 1) {
          *reinterpret_cast<int4*>(xa) = s_in[(u * S::ACCESSES) * ROT_THREADS + tid];
          if (two) *reinterpret_cast<int4*>(xb) = s_in[(u * S::ACCESSES + 1) * ROT_THREADS + tid];
        } else {
          xa[0] = in[u * in_hs + ia];
          if (two) xb[0] = in[u * in_hs + ib];
        }
        float ya[VEC], yb[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) ya[e] = Elem<T>::up(xa[e]);
        if constexpr (S::PAIRS) {
          if (turn) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) turn_pair(ya[e], ya[e + 1], cs[e / 2], sn[e / 2]);
          }
        } else if (two) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            yb[e] = Elem<T>::up(xb[e]);
            if (turn) turn_pair(ya[e], yb[e], cs[e], sn[e]);
          }
        }
        bool to8 = false;
        if constexpr (E4M3) {
          if (out8) {
            const float inv = 1.0f / scale[h + u];
            store_e4m3<VEC>(out8 + u * out_hs + ia, ya, inv);
            if (two) store_e4m3<VEC>(out8 + u * out_hs + ib, yb, inv);
            to8 = true;
          }
        }
        if (!to8) {
          store_row<T, VEC>(out + u * out_hs + ia, ya);
          if (two) store_row<T, VEC>(out + u * out_hs + ib, yb);
        }
      }
    }
  }
}

template <typename S, typename K>
cudaError_t go(K kern, RotateParams p, cudaStream_t st) {
  constexpr int VEC = S::VEC;
  const int half = p.rot_dim / 2;
  p.items = S::PAIRS ? p.d / VEC : half / VEC + ((p.d - p.rot_dim) / VEC + 1) / 2;
  const int threads = p.items <= ROT_THREADS ? ROT_THREADS : (p.items + 31) / 32 * 32;
  p.groups = threads / p.items;
  if (p.n_views == 0) p.v[0].heads = p.v[0].chunks = p.v[0].chunk_heads = 1;   // no tokens: next_lengths only
  long long cta = 0;
  int heads = 1;
  for (int v = 0; v < 3; ++v) {
    p.first_cta[v] = v < p.n_views ? (unsigned)cta : v ? 0xffffffffu : 0u;
    if (v >= p.n_views) continue;
    // a thread's heads: as many as it has places for, fewer while the call has not four CTAs for each of 152 SMs
    const long long rows = (long long)p.n_tok * p.v[v].heads;
    const long long wide = (rows * p.items + 4 * 152 * ROT_THREADS - 1) / (4 * 152 * ROT_THREADS);
    p.v[v].chunk_heads = (int)std::min<long long>(std::min(S::HEADS, p.v[v].heads), std::max<long long>(1, wide));
    heads = std::max(heads, p.v[v].chunk_heads);
    p.v[v].chunks = (p.v[v].heads + p.v[v].chunk_heads - 1) / p.v[v].chunk_heads;
    const long long units = (long long)p.n_tok * p.v[v].chunks;
    if (units > 0xf0000000LL) return cudaErrorInvalidConfiguration;   // counted with 32 bits
    cta += (units + p.groups - 1) / p.groups;
  }
  if (cta > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const size_t smem = VEC > 1 ? (size_t)heads * S::ACCESSES * ROT_THREADS * 16 : 0;
  static_assert(ROT_AHEAD * ROT_THREADS <= 48 * 1024, "within what needs no allowance");
  return launch_pdl(kern, dim3((unsigned)std::max(1LL, cta)), dim3(threads), smem, st, p);
}

// f(kernel shape) for the variant that takes a call
template <typename T, int W, bool APPEND, bool E4M3, typename F>
cudaError_t pick(bool interleaved, bool wide, F f) {
  if (wide)
    return interleaved ? f(rotate_kernel<T, W, true, APPEND, E4M3>, Shape<T, W, true>{})
                       : f(rotate_kernel<T, W, false, APPEND, E4M3>, Shape<T, W, false>{});
  return interleaved ? f(rotate_kernel<T, 1, true, APPEND, E4M3>, Shape<T, 1, true>{})
                     : f(rotate_kernel<T, 1, false, APPEND, E4M3>, Shape<T, 1, false>{});
}

template <typename F>
cudaError_t by_type(int type, int page_type, bool append, bool interleaved, bool wide, F f) {
  const bool e = page_type == HS_E4M3;
  if (append) {
    if (type == HS_BF16)
      return e ? pick<__nv_bfloat16, 8, true, true>(interleaved, wide, f)
               : pick<__nv_bfloat16, 8, true, false>(interleaved, wide, f);
    return e ? pick<__half, 8, true, true>(interleaved, wide, f) : pick<__half, 8, true, false>(interleaved, wide, f);
  }
  if (type == HS_BF16) return pick<__nv_bfloat16, 8, false, false>(interleaved, wide, f);
  if (type == HS_FP16) return pick<__half, 8, false, false>(interleaved, wide, f);
  return pick<float, 4, false, false>(interleaved, wide, f);
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int type, int page_type, bool append, bool interleaved,
                          bool wide, cudaStream_t st) {
  return by_type(type, page_type, append, interleaved, wide,
                 [&](auto kern, auto shape) { return go<decltype(shape)>(kern, p, st); });
}

cudaError_t prepare_rotate(int type, int page_type, bool append) {
  for (int variant = 0; variant < 4; ++variant) {
    const cudaError_t e = by_type(type, page_type, append, variant & 1, variant & 2, [](auto kern, auto) {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, kern);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hs
