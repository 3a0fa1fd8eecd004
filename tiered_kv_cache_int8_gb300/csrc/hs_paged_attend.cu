// Attention of many new tokens per request over its paged cache (hs_paged_attend).
//
//   s_n = scale q_h . K_n;  s_n <- cap tanh(s_n / cap);  s_n <- s_n - slope_h |p - n|
//   o_h = sum_n softmax_n(s_n) V_n over the positions that the token at p sees
//
// One warp per token and query head, 32 positions at a time with a running maximum and sum.
#include "hs_paged_attention.cuh"

namespace hs {
namespace {

constexpr int AT_WARPS = 8;

template <int VW, int PAGES, bool BF16>
__device__ __forceinline__ void load_part(const PagedAttendParams& p, int page, int which, int kvh, int slot, int e0, float (&x)[VW]) {
  const int d = p.d;
  const long long row = ((((long long)page * 2 + which) * p.h_kv + kvh) << p.page_shift) + slot;
  if constexpr (PAGES == PAGES_SAME) {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(p.pages) + row * d + e0;
#pragma unroll
    for (int e = 0; e < VW; ++e)
      x[e] = BF16 ? __uint_as_float((uint32_t)r[e] << 16) : __half2float(*reinterpret_cast<const __half*>(r + e));
  } else if constexpr (PAGES == PAGES_E4M3) {
    const unsigned char* r = p.pages + row * d + e0;
    const float sc = p.kv_scale[which * p.h_kv + kvh];
#pragma unroll
    for (int e = 0; e < VW; ++e) x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(r[e], __NV_E4M3))) * sc;
  } else {
    const unsigned char* u = p.pages + (row >> 4) * (9 * d);
    const int i = slot & 15;
    const float sc = p.kv_scale[which * p.h_kv + kvh];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int at = e0 + e;
      const unsigned char c = u[which ? (at >> 5) * 256 + i * 16 + ((at & 31) >> 1) : i * (d >> 1) + (at >> 1)];
      const unsigned char s = u[8 * d + (which ? (at >> 4) * 16 + i : i * (d >> 4) + (at >> 4))];
      x[e] = (float)((at & 1 ? c >> 4 : c & 15) - 8) * __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3))) * sc;
    }
  }
}

template <int VW, int PAGES, bool BF16>
__global__ void __launch_bounds__(32 * AT_WARPS) attend_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int D = 32 * VW;
  __shared__ float s_q[AT_WARPS][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const long long unit = (long long)blockIdx.x * AT_WARPS + warp;
  if (unit >= (long long)p.n_tok * p.h_q) return;
  const int t = (int)(unit / p.h_q), h = (int)(unit - (long long)t * p.h_q), kvh = h / p.group;
  int first = 0, n_new = p.tok_per_req, i = 0;
  if (!p.tok_offsets) {
    i = t / p.tok_per_req;
    first = i * p.tok_per_req;
  } else {
    for (i = 0; i < p.n_req; ++i) {
      first = p.tok_offsets[i];
      const int end = p.tok_offsets[i + 1];
      n_new = end - first;
      if (first < 0 || end < first || end > p.n_tok) {
        if (lane == 0) set_error(p.dev_error, HS_DEVERR_OFFSETS);
        continue;
      }
      if (t >= first && t < end) break;
    }
    if (i == p.n_req) return;
  }
  const int req = p.req_ids ? p.req_ids[i] : i;
  int len = -1, total = 0;
  if (req < 0 || req >= p.max_requests) {
    if (lane == 0) set_error(p.dev_error, HS_DEVERR_REQ_RANGE);
  } else {
    len = p.lengths[req];
    if (len < 0 || (long long)len + n_new > (long long)p.max_pages << p.page_shift) {
      if (lane == 0) set_error(p.dev_error, HS_DEVERR_CAPACITY);
      len = -1;
    }
  }
  const long long orow = (long long)t * p.h_q + h;
  float m = -INFINITY, l = 0.f, o[VW] = {};
  if (len >= 0) {
    total = len + n_new;
    const int pos = len + t - first;
    int hi = pos + 1;
    if (p.prefix) hi = max(hi, min(p.prefix[req], total));
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_ts + h * p.q_hs;
    for (int e = lane; e < D; e += 32)
      s_q[warp][e] = BF16 ? __uint_as_float((uint32_t)q[e] << 16) : __half2float(*reinterpret_cast<const __half*>(q + e));
    __syncwarp();
    const float slope = p.slopes ? p.slopes[h] * pa::LOG2_E : 0.f;
    for (int n0 = lo; n0 < hi; n0 += 32) {
      const int n = n0 + lane;
      int page = -1;
      if (n < hi) {
        page = p.page_table[(long long)req * p.max_pages + (n >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) {
          set_error(p.dev_error, HS_DEVERR_PAGE);
          page = -1;
        }
      }
      float s = -INFINITY;
      if (page >= 0) {
        s = 0.f;
        for (int e = 0; e < D; e += 8) {
          float x[8];
          load_part<8, PAGES, BF16>(p, page, 0, kvh, n & (p.page_size - 1), e, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) s = fmaf(s_q[warp][e + j], x[j], s);
        }
        if (p.cap_in != 0.f) s = p.cap_log2 * pa::tanh32(s * p.cap_in); else s *= p.scale_log2;
        s -= slope * fabsf((float)(pos - n));
      }
      float mx = s;
#pragma unroll
      for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, d));
      mx = fmaxf(mx, m);
      const float base = mx == -INFINITY ? 0.f : mx, keep = exp2f(m - base);
      const float w = exp2f(s - base);
      m = mx;
      float sum = w;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
      l = l * keep + sum;
#pragma unroll
      for (int e = 0; e < VW; ++e) o[e] *= keep;
      for (int j = 0; j < min(32, hi - n0); ++j) {
        const int pj = __shfl_sync(FULL_MASK, page, j);
        const float wj = __shfl_sync(FULL_MASK, w, j);
        if (pj < 0) continue;
        float x[VW];
        load_part<VW, PAGES, BF16>(p, pj, 1, kvh, (n0 + j) & (p.page_size - 1), lane * VW, x);
#pragma unroll
        for (int e = 0; e < VW; ++e) o[e] = fmaf(wj, x[e], o[e]);
      }
    }
  }
  const float inv = pa::inverse(l);
#pragma unroll
  for (int e = 0; e < VW; ++e) o[e] *= inv;
  pa::store_lane<BF16 ? HS_BF16 : HS_FP16, VW>(p.out, orow * D + lane * VW, o);
  if (p.lse && lane == 0) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
}

template <typename F>
cudaError_t pick(int d, int type, int page_type, F f) {
  auto with = [&](auto vw, auto bf) {
    const Pages k = pages_kind(page_type);
    return k == PAGES_INT4 ? f(attend_kernel<vw(), PAGES_INT4, bf()>)
                           : k == PAGES_E4M3 ? f(attend_kernel<vw(), PAGES_E4M3, bf()>) : f(attend_kernel<vw(), PAGES_SAME, bf()>);
  };
  auto width = [&](auto bf) {
    return d == 64 ? with(std::integral_constant<int, 2>{}, bf) : d == 128 ? with(std::integral_constant<int, 4>{}, bf)
                                                                           : with(std::integral_constant<int, 8>{}, bf);
  };
  return type == HS_BF16 ? width(std::true_type{}) : width(std::false_type{});
}

}  // namespace

int64_t attend_workspace_bytes(int d, int ctas) { return 256; }

cudaError_t prepare_attend(int d, int type, int page_type) {
  return pick(d, type, page_type, [](auto kern) {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern);
  });
}

cudaError_t launch_paged_attend(const PagedAttendParams& p, cudaStream_t st) {
  const long long ctas = ((long long)p.n_tok * p.h_q + AT_WARPS - 1) / AT_WARPS;
  return pick(p.d, p.type, p.page_type, [&](auto kern) { return launch_pdl(kern, dim3((unsigned)ctas), dim3(32 * AT_WARPS), 0, st, p); });
}

}  // namespace hs
