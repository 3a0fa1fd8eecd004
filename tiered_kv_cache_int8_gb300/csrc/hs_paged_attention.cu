// Attention of one new token per request over its paged cache:
//   o_h = sum_n softmax_n(scale * q_h . K_n) V_n,  lse_h = ln sum_n exp(scale * q_h . K_n)
// over n in [max(0, N - window), N).
//
// One CTA per (request, query head): tiles of 128 positions, one score per
// thread, a running maximum and sum, one output element per thread and round.
#include "hs_paged.cuh"

namespace hs {
namespace {

constexpr int PA_THREADS = 128;

__device__ __forceinline__ float as_float(const unsigned char* p, long long i, int type) {
  if (type == HS_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  if (type == HS_FP16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
}

__global__ void __launch_bounds__(PA_THREADS) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  __shared__ float s_q[256], s_p[PA_THREADS], s_red[PA_THREADS / 32];
  __shared__ long long s_row[PA_THREADS];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x, ri = blockIdx.y, tid = threadIdx.x;
  const int hk = h / p.group;
  const int req = p.req_ids ? p.req_ids[ri] : ri;
  int len = 0;
  unsigned err = 0;
  if (req < 0 || req >= p.max_requests) {
    err = HS_DEVERR_REQ_RANGE;
  } else {
    len = p.lengths[req];
    if (len < 0 || len > p.max_pages << p.page_shift) {
      err = HS_DEVERR_CAPACITY;
      len = 0;
    }
  }
  const int first = p.window > 0 ? max(0, len - p.window) : 0;
  const float ks = p.kv_scale ? p.kv_scale[hk] : 1.0f, vs = p.kv_scale ? p.kv_scale[p.h_kv + hk] : 1.0f;
  for (int e = tid; e < p.d; e += PA_THREADS)
    s_q[e] = as_float(static_cast<const unsigned char*>(p.q), ri * p.q_ts + h * p.q_hs + e, p.type) *
             (p.scale_log2 * ks);
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  __syncthreads();
  for (int n0 = first; n0 < len; n0 += PA_THREADS) {
    const int n = n0 + tid;
    float s = -INFINITY;
    long long row = -1;
    if (n < len) {
      const int page = p.page_table[(long long)req * p.max_pages + (n >> p.page_shift)];
      if (page < 0 || page >= p.n_pages) {
        err |= HS_DEVERR_PAGE;
      } else {
        row = ((((long long)page * 2) * p.h_kv + hk) << p.page_shift) + (n & (p.page_size - 1));
        s = 0.f;
        for (int e = 0; e < p.d; ++e) s += s_q[e] * as_float(p.pages, row * p.d + e, p.page_type);
      }
    }
    float mx = s;
    for (int o2 = 16; o2; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, o2));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    float mn = m;
    for (int w = 0; w < PA_THREADS / 32; ++w) mn = fmaxf(mn, s_red[w]);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float keep = exp2f(m - base);
    s_p[tid] = exp2f(s - base);
    s_row[tid] = row;
    m = mn;
    __syncthreads();
    l *= keep;
    for (int i = 0; i < PA_THREADS; ++i) l += s_p[i];
    for (int r = 0, e = tid; e < p.d; ++r, e += PA_THREADS) {
      float a = o[r] * keep;
      for (int i = 0; i < PA_THREADS; ++i)
        if (s_row[i] >= 0)
          a += s_p[i] * as_float(p.pages, (s_row[i] + ((long long)p.h_kv << p.page_shift)) * p.d + e, p.page_type);
      o[r] = a;
    }
    __syncthreads();
  }
  const float inv = l > 0.f ? vs / l : (l == 0.f ? 0.f : l);
  for (int r = 0, e = tid; e < p.d; ++r, e += PA_THREADS) {
    const long long at = ((long long)ri * p.h_q + h) * p.d + e;
    if (p.type == HS_BF16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o[r] * inv);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(o[r] * inv);
  }
  if (p.lse && tid == 0) p.lse[(long long)ri * p.h_q + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  if (err) set_error(p.dev_error, err);
}

}  // namespace

int64_t paged_workspace_bytes(int, int, int, int) { return 256; }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t st) {
  return launch_pdl(paged_decode_kernel, dim3(p.h_q, p.n_req), dim3(PA_THREADS), 0, st, p);
}

}  // namespace hs
