// Where the tokens of a call go in a paged cache: shared by the kernels that append
// rows (hs_rotary.cu, hs_paged_rows.cu) and that read them (hs_paged_rows.cu).
#ifndef HS_PAGED_PLACE_CUH_
#define HS_PAGED_PLACE_CUH_

#include "hs_paged.cuh"

namespace hs {

// Where a token goes: its position, and its page row (pages of the layer are
// [n_pages][2][h_kv][page_size] rows), -1 where it is not stored.
struct Token {
  int pos;        // its position
  int ok;         // 0: the token belongs to no request of the call, or to a bad one (nothing is read or written)
  int page, slot; // page < 0: not stored
  int row;        // 1: a row of a request, a bad one's among them
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
  Token k = {0, 0, -1, 0, 0};
  const int j = t - first;
  if (j >= 0 && j < n) {
    k.row = 1;
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
__device__ __forceinline__ Token locate(const RotateParams& p, int t, bool mine) {
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
    return mine ? place_of(p, t, i, first, n, req, &len, err) : Token{0, 0, -1, 0, 0};
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
  if (!mine) return Token{0, 0, -1, 0, 0};
  return place_of(p, t, i, first, n, p.req_ids ? p.req_ids[i] : i, nullptr, err);
}

// next_lengths of an append's requests, written by the first CTAs (blockIdx.x * blockDim.x of
// all of them may pass 32 bits).
constexpr int LENGTH_CTAS = PG_MAX_REQUESTS / 256;
__device__ __forceinline__ void write_next_lengths(const RotateParams& p) {
  if (!p.next_lengths || blockIdx.x >= LENGTH_CTAS) return;
  const int ctas = min(gridDim.x, (unsigned)LENGTH_CTAS);
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.n_req; i += ctas * blockDim.x) {
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

}  // namespace hs

#endif  // HS_PAGED_PLACE_CUH_
