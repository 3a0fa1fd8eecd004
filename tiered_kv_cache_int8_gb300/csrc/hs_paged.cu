// Host side of the rotary and paged-cache entry points declared in include/hs.h:
// frequency tables, argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>
#include <numeric>
#include <string>

#include "hs_paged.cuh"

namespace {

int fail(int code, const char* msg) { return hs::set_static_error(code, msg); }

int fail_cuda(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  char msg[256];
  std::snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return fail(HS_ERR_CUDA, msg);
}

// Makes `device` current for a call and puts the caller's device back.
struct DeviceScope {
  int prev = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceScope(int device) {
    int cur = -1;
    err = cudaGetDevice(&cur);
    if (err == cudaSuccess && cur != device) {
      err = cudaSetDevice(device);
      if (err == cudaSuccess) prev = cur;
    }
  }
  ~DeviceScope() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Elements from the view's first to one past its last.
long long extent(const hs_heads_t& v, int n_tok, int d) {
  return (long long)(n_tok - 1) * v.token_stride + (long long)(v.heads - 1) * v.head_stride + d;
}

// "" or why the view cannot be used
const char* check_view(const hs_heads_t& v, int n_tok, int d, size_t es, bool written) {
  if (!v.data) return "a view's data is null";
  if (v.heads < 1 || v.heads > 4096) return "a view's heads must be in [1, 4096]";
  const int64_t lim = (int64_t)1 << 40;
  if (v.token_stride < 0 || v.head_stride < 0 || v.token_stride > lim || v.head_stride > lim)
    return "a view's strides must be in [0, 2^40]";
  if (reinterpret_cast<uintptr_t>(v.data) % es) return "a view's data is not aligned to its element type";
  // (so that extents, and bytes behind an address, stay far inside 64 bits)
  const int64_t reach = (int64_t)1 << 46;
  if ((v.token_stride && n_tok - 1 > reach / v.token_stride) || (v.head_stride && v.heads - 1 > reach / v.head_stride))
    return "a view's last token and head must be within 2^46 elements of its first";
  if (written) {
    const bool one_t = n_tok == 1, one_h = v.heads == 1;
    const bool th = (one_h || v.head_stride >= d) &&
                    (one_t || v.token_stride >= (int64_t)(v.heads - 1) * (one_h ? 0 : v.head_stride) + d);
    const bool ht = (one_t || v.token_stride >= d) &&
                    (one_h || v.head_stride >= (int64_t)(n_tok - 1) * (one_t ? 0 : v.token_stride) + d);
    if (!th && !ht) return "an output view's elements overlap";
  }
  return "";
}

bool same_view(const hs_heads_t& a, const hs_heads_t& b, int n_tok) {
  return a.data == b.data && (n_tok == 1 || a.token_stride == b.token_stride) &&
         (a.heads == 1 || a.head_stride == b.head_stride);
}

// Whether no element of `a` (n_tok tokens, aligned to its type) is one of `b`: their ranges
// of bytes do not meet, or neither do the places that they take modulo a stride which both
// keep to: one token's heads modulo the tokens' stride (slices of one projection), a head of
// every token modulo the heads' stride, single rows modulo what divides all strides
// ([tokens][heads][q, k, v][d]).  Views that none of these parts pass as meeting.
bool apart(const hs_heads_t& a, const hs_heads_t& b, int n_tok, int d, size_t es) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.data), b0 = reinterpret_cast<uintptr_t>(b.data);
  if (a0 + (size_t)extent(a, n_tok, d) * es <= b0 || b0 + (size_t)extent(b, n_tok, d) * es <= a0) return true;
  const int64_t delta = (int64_t)(b0 - a0) / (int64_t)es;
  const int64_t at = n_tok > 1 ? a.token_stride : 0, bt = n_tok > 1 ? b.token_stride : 0;
  const int64_t ah = a.heads > 1 ? a.head_stride : 0, bh = b.heads > 1 ? b.head_stride : 0;
  auto distinct = [&](int64_t stride, int64_t a_span, int64_t b_span) {   // of [0, a_span) and [delta, delta + b_span)
    if (stride == 0) return false;
    const int64_t r = (delta % stride + stride) % stride;
    return a_span <= r && r + b_span <= stride;
  };
  const int64_t t = std::gcd(at, bt), h = std::gcd(ah, bh);
  return distinct(t, (a.heads - 1) * ah + d, (b.heads - 1) * bh + d) ||
         distinct(h, (n_tok - 1) * at + d, (n_tok - 1) * bt + d) || distinct(std::gcd(t, h), d, d);
}

// whether every row of a view is 16-byte aligned (the stride of a single token or head says nothing)
bool wide_view(const hs_heads_t& v, int n_tok, size_t es) {
  return reinterpret_cast<uintptr_t>(v.data) % 16 == 0 && (n_tok == 1 || (v.token_stride * es) % 16 == 0) &&
         (v.heads == 1 || (v.head_stride * es) % 16 == 0);
}

// in -> out of a rotation: "" or why not
const char* check_pair(const hs_heads_t& in, const hs_heads_t& out, int n_tok, int d, size_t es) {
  const char* why = check_view(in, n_tok, d, es, false);
  if (*why) return why;
  why = check_view(out, n_tok, d, es, true);
  if (*why) return why;
  if (in.heads != out.heads) return "an output view has another number of heads than its input";
  if (!same_view(in, out, n_tok) && !apart(in, out, n_tok, d, es))
    return "an output view overlaps its input without being the same view";
  return "";
}

const char* check_rotary(const hs_rotary_t& r, int d) {
  if (!r.turns) return "the rotation's table is null";
  if (reinterpret_cast<uintptr_t>(r.turns) % 8) return "the rotation's table is not 8-byte aligned";
  if (r.rot_dim < 2 || r.rot_dim > d || r.rot_dim % 2) return "rot_dim must be even and in [2, d]";
  if ((r.interleaved & ~1) || (r.transpose & ~1)) return "interleaved and transpose must be 0 or 1";
  if (!std::isfinite(r.magnitude)) return "the rotation's magnitude must be finite";
  return "";
}

// whether the 16-byte kernels can take a rotation of these sizes
bool wide_rotary(const hs_rotary_t* r, int d, size_t es) {
  const size_t vec = 16 / es;
  if (d % vec) return false;
  if (!r) return true;
  return r->interleaved ? r->rot_dim % vec == 0 : (r->rot_dim / 2) % vec == 0;
}

int named(int code, const char* call, const char* why) {
  char msg[320];
  std::snprintf(msg, sizeof msg, "%s: %s", call, why);
  return fail(code, msg);
}

hs::RowView row_view(const hs_heads_t& in, const hs_heads_t* out, int kind) {
  hs::RowView v = {};
  v.in = in.data;
  v.in_ts = in.token_stride;
  v.in_hs = in.head_stride;
  v.heads = in.heads;
  v.kind = kind;
  if (out) {
    v.out = out->data;
    v.out_ts = out->token_stride;
    v.out_hs = out->head_stride;
  }
  return v;
}

bool is_pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

const char* check_paged(const hs_paged_config_t& c) {
  if (c.n_layers < 1) return "n_layers must be >= 1";
  if (c.n_pages < 1) return "n_pages must be >= 1";
  if (!is_pow2(c.page_size) || c.page_size < 16 || c.page_size > 256) return "page_size must be 16, 32, 64, 128 or 256";
  if (c.max_requests < 1 || c.max_requests > hs::PG_MAX_REQUESTS) return "max_requests must be in [1, 4096]";
  if (c.max_pages < 1 || (long long)c.max_pages * c.page_size > hs::PG_MAX_POSITIONS)
    return "max_pages must be >= 1 and max_pages * page_size at most 2^22";
  if (c.d != 64 && c.d != 128 && c.d != 256) return "d must be 64, 128 or 256";
  if (c.h_kv < 1 || c.h_kv > 1024) return "h_kv must be in [1, 1024]";
  if (c.h_q < c.h_kv || c.h_q > 4096 || c.h_q % c.h_kv) return "h_q must be a multiple of h_kv, at most 4096";
  if (c.type != HS_BF16 && c.type != HS_FP16) return "type must be HS_BF16 or HS_FP16";
  if (c.page_type != c.type && c.page_type != HS_E4M3) return "page_type must be type or HS_E4M3";
  if (c.window < 0) return "window must be >= 0";
  if (!(c.softmax_scale >= 0.f) || !std::isfinite(c.softmax_scale)) return "softmax_scale must be finite and >= 0";
  // rows of a layer are addressed with 31 bits
  if ((long long)c.n_pages * 2 * c.h_kv * c.page_size > 0x7fffffffLL)
    return "n_pages * 2 * h_kv * page_size must be below 2^31";
  return "";
}

size_t layer_bytes(const hs_paged_config_t& c) {
  return (size_t)c.n_pages * 2 * c.h_kv * c.page_size * c.d * hs::type_bytes(c.page_type);
}

}  // namespace

extern "C" {

int hs_rotary_table(const hs_rotary_config_t* cfg, const double* inv_freq, uint64_t* turns, float* magnitude) {
  if (!cfg || !turns || !magnitude) return fail(HS_ERR_INVALID, "hs_rotary_table: null argument");
  const hs_rotary_config_t& c = *cfg;
  if (c.rot_dim < 2 || c.rot_dim > 1024 || c.rot_dim % 2)
    return fail(HS_ERR_CONFIG, "hs_rotary_table: rot_dim must be even and in [2, 1024]");
  if (!(c.magnitude >= 0.0) || !std::isfinite(c.magnitude))
    return fail(HS_ERR_CONFIG, "hs_rotary_table: magnitude must be finite and >= 0");
  const double two_pi = 6.283185307179586476925286766559;
  const int n = c.rot_dim / 2;
  if (!inv_freq) {
    if (!(c.base > 1.0) || !std::isfinite(c.base))
      return fail(HS_ERR_CONFIG, "hs_rotary_table: base must be finite and > 1");
    if (c.scaling < HS_ROTARY_PLAIN || c.scaling > HS_ROTARY_BY_PARTS)
      return fail(HS_ERR_CONFIG, "hs_rotary_table: scaling must be one of HS_ROTARY_*");
    if (c.scaling != HS_ROTARY_PLAIN && (!(c.factor >= 1.0) || !std::isfinite(c.factor)))
      return fail(HS_ERR_CONFIG, "hs_rotary_table: factor must be finite and >= 1");
    if (c.scaling == HS_ROTARY_NTK && c.rot_dim == 2)
      return fail(HS_ERR_CONFIG, "hs_rotary_table: HS_ROTARY_NTK needs rot_dim > 2");
    if (c.scaling == HS_ROTARY_BY_PARTS &&
        (!(c.original_context > 0.0) || !std::isfinite(c.original_context) || !(c.high > c.low) ||
         !std::isfinite(c.low) || !std::isfinite(c.high)))
      return fail(HS_ERR_CONFIG, "hs_rotary_table: HS_ROTARY_BY_PARTS needs original_context > 0 and high > low");
  } else {
    for (int i = 0; i < n; ++i)
      if (!(inv_freq[i] >= 0.0) || !std::isfinite(inv_freq[i]))
        return fail(HS_ERR_CONFIG, "hs_rotary_table: inv_freq must be finite and >= 0");
  }
  double base = c.base;
  if (!inv_freq && c.scaling == HS_ROTARY_NTK) base *= std::pow(c.factor, (double)c.rot_dim / (c.rot_dim - 2));
  for (int i = 0; i < n; ++i) {
    double f;
    if (inv_freq) {
      f = inv_freq[i];
    } else {
      f = std::pow(base, -2.0 * i / c.rot_dim);
      if (c.scaling == HS_ROTARY_LINEAR) {
        f /= c.factor;
      } else if (c.scaling == HS_ROTARY_BY_PARTS) {
        double w = (c.original_context * f / two_pi - c.low) / (c.high - c.low);
        w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
        f = w * f + (1.0 - w) * f / c.factor;
      }
    }
    const double t = f / two_pi;
    turns[i] = (uint64_t)std::ldexp(t - std::floor(t), 64);   // t - floor(t) <= 1 - 2^-53
  }
  *magnitude = c.magnitude > 0.0 ? (float)c.magnitude
               : !inv_freq && c.scaling == HS_ROTARY_BY_PARTS && c.factor > 1.0
                   ? (float)(0.1 * std::log(c.factor) + 1.0)
                   : 1.0f;
  return HS_OK;
}

int hs_rotary_apply(const hs_rotary_t* rot, int32_t type, int32_t d, int32_t n_tok, const int32_t* positions,
                    int32_t n_views, const hs_heads_t* in, const hs_heads_t* out, int32_t device, void* stream) {
  static const char* me = "hs_rotary_apply";
  if (type != HS_BF16 && type != HS_FP16 && type != HS_FP32)
    return named(HS_ERR_INVALID, me, "type must be HS_BF16, HS_FP16 or HS_FP32");
  if (d < 2 || d > 1024) return named(HS_ERR_INVALID, me, "d must be in [2, 1024]");
  if (n_tok < 0) return named(HS_ERR_INVALID, me, "n_tok < 0");
  if (n_views < 1 || n_views > 2) return named(HS_ERR_INVALID, me, "n_views must be 1 or 2");
  if (!rot || !in || !out) return named(HS_ERR_INVALID, me, "null argument");
  if (const char* why = check_rotary(*rot, d); *why) return named(HS_ERR_INVALID, me, why);
  if (n_tok == 0) return HS_OK;
  if (!positions) return named(HS_ERR_INVALID, me, "null positions");
  if (reinterpret_cast<uintptr_t>(positions) % 4) return named(HS_ERR_INVALID, me, "positions must be 4-byte aligned");
  const size_t es = hs::type_bytes(type);
  hs::RotateParams p = {};
  bool wide = wide_rotary(rot, d, es);
  for (int i = 0; i < n_views; ++i) {
    if (const char* why = check_pair(in[i], out[i], n_tok, d, es); *why) return named(HS_ERR_INVALID, me, why);
    wide = wide && wide_view(in[i], n_tok, es) && wide_view(out[i], n_tok, es);
    p.v[i] = row_view(in[i], &out[i], hs::VIEW_ROTATE);
  }
  // threads of different views run in no order
  if (n_views == 2 && !(apart(out[0], out[1], n_tok, d, es) && apart(out[0], in[1], n_tok, d, es) &&
                        apart(out[1], in[0], n_tok, d, es)))
    return named(HS_ERR_INVALID, me, "an output view overlaps the other output or the other input");
  p.n_views = n_views;
  p.d = d;
  p.n_tok = n_tok;
  p.rot_dim = rot->rot_dim;
  p.magnitude = rot->magnitude;
  p.sign = rot->transpose ? -1.f : 1.f;
  p.turns = rot->turns;
  p.positions = positions;
  DeviceScope dev(device);
  if (dev.err != cudaSuccess) return fail_cuda(dev.err, "hs_rotary_apply: device");
  const cudaError_t e =
      hs::launch_rotate(p, type, type, false, rot->interleaved != 0, wide, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS_OK : fail_cuda(e, "hs_rotary_apply: launch");
}

int hs_paged_create(const hs_paged_config_t* cfg, void* pages, const float* kv_scale, uint32_t* error_word,
                    hs_paged_t** out) {
  static const char* me = "hs_paged_create";
  if (!cfg || !out) return named(HS_ERR_INVALID, me, "null argument");
  *out = nullptr;
  if (const char* why = check_paged(*cfg); *why) return named(HS_ERR_CONFIG, me, why);
  if (!pages || reinterpret_cast<uintptr_t>(pages) % 16)
    return named(HS_ERR_INVALID, me, "pages must be 16-byte aligned and not null");
  if ((cfg->page_type == HS_E4M3) != (kv_scale != nullptr))
    return named(HS_ERR_INVALID, me, "kv_scale goes with HS_E4M3 pages, and with them only");
  if (reinterpret_cast<uintptr_t>(kv_scale) % 4) return named(HS_ERR_INVALID, me, "kv_scale must be 4-byte aligned");
  if (!error_word || reinterpret_cast<uintptr_t>(error_word) % 4)
    return named(HS_ERR_INVALID, me, "error_word must be 4-byte aligned and not null");
  hs_paged* h = new (std::nothrow) hs_paged();
  if (!h) return named(HS_ERR_OOM, me, "out of host memory");
  h->cfg = *cfg;
  h->pages = pages;
  h->kv_scale = kv_scale;
  while ((1 << h->page_shift) < cfg->page_size) ++h->page_shift;
  const float scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / std::sqrt((float)cfg->d);
  h->scale_log2 = scale * 1.4426950408889634f;
  h->dev_error = error_word;
  // a handle is host memory only: without a device the calls' checks still run
  if (cudaDeviceGetAttribute(&h->ctas, cudaDevAttrMultiProcessorCount, cfg->device) != cudaSuccess) {
    (void)cudaGetLastError();
    h->ctas = 0;
  } else {
    h->ctas = std::min(h->ctas, hs::PG_MAX_CTAS);
    h->maps.reset(new (std::nothrow) CUtensorMap[cfg->n_layers]);
    if (!h->maps) {
      delete h;
      return named(HS_ERR_OOM, me, "out of host memory");
    }
    if (!hs::paged_maps(h, layer_bytes(*cfg))) {
      delete h;
      return named(HS_ERR_CUDA, me, "the driver made no tensor map of the pool");
    }
    // the kernels are loaded here, so that a first call may be a captured one
    DeviceScope dev(cfg->device);
    cudaError_t e = dev.err;
    if (e == cudaSuccess) e = hs::prepare_paged(cfg->d, cfg->h_q / cfg->h_kv, cfg->type, cfg->page_type);
    if (e == cudaSuccess) e = hs::prepare_rotate(cfg->type, cfg->page_type, true);
    if (e != cudaSuccess) {
      delete h;
      return fail_cuda(e, "hs_paged_create: kernel set-up");
    }
  }
  *out = h;
  return HS_OK;
}

void hs_paged_destroy(hs_paged_t* h) { delete h; }

int hs_paged_append(hs_paged_t* h, int32_t layer, int32_t n_req, const int32_t* req_ids, int32_t n_tok,
                    const int32_t* tok_offsets, const int32_t* page_table, const int32_t* lengths,
                    int32_t* next_lengths, const hs_rotary_t* rot, const hs_heads_t* q, const hs_heads_t* q_out,
                    const hs_heads_t* k, const hs_heads_t* v, void* stream) {
  static const char* me = "hs_paged_append";
  if (!h) return named(HS_ERR_INVALID, me, "null handle");
  const hs_paged_config_t& c = h->cfg;
  if (layer < 0 || layer >= c.n_layers) return named(HS_ERR_INVALID, me, "layer out of range");
  if (n_req < 0 || n_req > c.max_requests) return named(HS_ERR_INVALID, me, "n_req out of range");
  if (n_tok < 0) return named(HS_ERR_INVALID, me, "n_tok < 0");
  if (n_req == 0) return HS_OK;
  if (!tok_offsets && n_tok % n_req)
    return named(HS_ERR_INVALID, me, "without tok_offsets, n_tok must be a multiple of n_req");
  if (!page_table || !lengths) return named(HS_ERR_INVALID, me, "null page_table or lengths");
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lengths) |
        reinterpret_cast<uintptr_t>(next_lengths) | reinterpret_cast<uintptr_t>(req_ids) |
        reinterpret_cast<uintptr_t>(tok_offsets)) % 4) != 0)
    return named(HS_ERR_INVALID, me, "an int32 array is not 4-byte aligned");
  if (next_lengths && next_lengths < lengths + c.max_requests && lengths < next_lengths + c.max_requests)
    return named(HS_ERR_INVALID, me, "next_lengths overlaps lengths");
  if ((q == nullptr) != (q_out == nullptr)) return named(HS_ERR_INVALID, me, "q and q_out go together");
  if (q && !rot) return named(HS_ERR_INVALID, me, "q and q_out need a rotation");
  if (rot) {
    if (const char* why = check_rotary(*rot, c.d); *why) return named(HS_ERR_INVALID, me, why);
    if (rot->transpose) return named(HS_ERR_INVALID, me, "keys are not stored by the transposed rotation");
  }
  const size_t es = hs::type_bytes(c.type);
  hs::RotateParams p = {};
  bool wide = wide_rotary(rot, c.d, es);
  if (n_tok > 0) {
    if (!k || !v) return named(HS_ERR_INVALID, me, "null k or v");
    const char* why = check_view(*k, n_tok, c.d, es, false);
    if (!*why) why = check_view(*v, n_tok, c.d, es, false);
    if (!*why && q) why = check_pair(*q, *q_out, n_tok, c.d, es);
    if (*why) return named(HS_ERR_INVALID, me, why);
    if (k->heads != c.h_kv || v->heads != c.h_kv) return named(HS_ERR_INVALID, me, "k and v must have h_kv heads");
    if (q && q->heads != c.h_q) return named(HS_ERR_INVALID, me, "q must have h_q heads");
    if (q && !(apart(*q_out, *k, n_tok, c.d, es) && apart(*q_out, *v, n_tok, c.d, es)))
      return named(HS_ERR_INVALID, me, "q_out overlaps k or v");
    int n = 0;
    if (q) {
      wide = wide && wide_view(*q, n_tok, es) && wide_view(*q_out, n_tok, es);
      p.v[n++] = row_view(*q, q_out, hs::VIEW_ROTATE);
    }
    wide = wide && wide_view(*k, n_tok, es) && wide_view(*v, n_tok, es);
    p.v[n++] = row_view(*k, nullptr, hs::VIEW_KEYS);
    p.v[n++] = row_view(*v, nullptr, hs::VIEW_VALUES);
    p.n_views = n;
  }
  p.d = c.d;
  p.n_tok = n_tok;
  if (rot) {
    p.rot_dim = rot->rot_dim;
    p.magnitude = rot->magnitude;
    p.sign = 1.f;
    p.turns = rot->turns;
  }
  p.req_ids = req_ids;
  p.tok_offsets = tok_offsets;
  p.page_table = page_table;
  p.lengths = lengths;
  p.next_lengths = next_lengths;
  p.n_req = n_req;
  p.tok_per_req = tok_offsets ? 0 : n_tok / n_req;
  p.max_requests = c.max_requests;
  p.max_pages = c.max_pages;
  p.n_pages = c.n_pages;
  p.page_size = c.page_size;
  p.page_shift = h->page_shift;
  p.h_kv = c.h_kv;
  p.pages = static_cast<unsigned char*>(h->pages) + layer_bytes(c) * layer;
  p.kv_scale = h->kv_scale ? h->kv_scale + (size_t)layer * 2 * c.h_kv : nullptr;
  p.dev_error = h->dev_error;
  DeviceScope dev(c.device);
  if (dev.err != cudaSuccess) return fail_cuda(dev.err, "hs_paged_append: device");
  const cudaError_t e = hs::launch_rotate(p, c.type, c.page_type, true, rot && rot->interleaved, wide,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS_OK : fail_cuda(e, "hs_paged_append: launch");
}

int64_t hs_paged_workspace_bytes(const hs_paged_t* h) {
  return h ? hs::paged_workspace_bytes(h->cfg.d, h->cfg.h_q / h->cfg.h_kv, h->cfg.page_type, h->ctas) : 0;
}

int hs_paged_decode(hs_paged_t* h, int32_t layer, int32_t n_req, const int32_t* req_ids, const int32_t* page_table,
                    const int32_t* lengths, const hs_heads_t* q, void* out, float* lse, void* workspace,
                    void* stream) {
  static const char* me = "hs_paged_decode";
  if (!h) return named(HS_ERR_INVALID, me, "null handle");
  const hs_paged_config_t& c = h->cfg;
  if (layer < 0 || layer >= c.n_layers) return named(HS_ERR_INVALID, me, "layer out of range");
  if (n_req < 0 || n_req > c.max_requests) return named(HS_ERR_INVALID, me, "n_req out of range");
  if (n_req == 0) return HS_OK;
  if (!page_table || !lengths || !q || !out || !workspace) return named(HS_ERR_INVALID, me, "null argument");
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lengths) |
        reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(req_ids)) % 4) != 0)
    return named(HS_ERR_INVALID, me, "an int32 or float array is not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(out) % 16) return named(HS_ERR_INVALID, me, "out must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return named(HS_ERR_INVALID, me, "workspace must be 256-byte aligned");
  const size_t es = hs::type_bytes(c.type);
  if (const char* why = check_view(*q, n_req, c.d, es, false); *why) return named(HS_ERR_INVALID, me, why);
  if (q->heads != c.h_q) return named(HS_ERR_INVALID, me, "q must have h_q heads");
  if (!wide_view(*q, n_req, es)) return named(HS_ERR_INVALID, me, "q's rows must be 16-byte aligned");
  hs_heads_t o = {out, (int64_t)c.h_q * c.d, c.d, c.h_q, 0};
  if (!same_view(*q, o, n_req) && !apart(*q, o, n_req, c.d, es))
    return named(HS_ERR_INVALID, me, "out overlaps q without being the same memory in the same order");
  hs::PagedDecodeParams p = {};
  p.req_ids = req_ids;
  p.page_table = page_table;
  p.lengths = lengths;
  p.q = q->data;
  p.q_ts = q->token_stride;
  p.q_hs = q->head_stride;
  p.out = out;
  p.lse = lse;
  p.ws = static_cast<float*>(workspace);
  p.pages = static_cast<const unsigned char*>(h->pages) + layer_bytes(c) * layer;
  p.kv_scale = h->kv_scale ? h->kv_scale + (size_t)layer * 2 * c.h_kv : nullptr;
  p.dev_error = h->dev_error;
  p.n_req = n_req;
  p.max_requests = c.max_requests;
  p.max_pages = c.max_pages;
  p.n_pages = c.n_pages;
  p.page_size = c.page_size;
  p.page_shift = h->page_shift;
  p.h_q = c.h_q;
  p.h_kv = c.h_kv;
  p.group = c.h_q / c.h_kv;
  p.d = c.d;
  p.window = c.window;
  p.type = c.type;
  p.page_type = c.page_type;
  p.grid = h->ctas;
  p.scale_log2 = h->scale_log2;
  DeviceScope dev(c.device);
  if (dev.err != cudaSuccess) return fail_cuda(dev.err, "hs_paged_decode: device");
  if (h->ctas < 1) return named(HS_ERR_CUDA, me, "the handle was created without its device");
  const cudaError_t e = hs::launch_paged_decode(p, h->maps[layer], static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS_OK : fail_cuda(e, "hs_paged_decode: launch");
}

int hs_paged_error(hs_paged_t* h, uint32_t* out) {
  if (!h || !out) return fail(HS_ERR_INVALID, "hs_paged_error: null argument");
  *out = 0;
  DeviceScope dev(h->cfg.device);
  cudaError_t e = dev.err;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  unsigned int word = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&word, h->dev_error, sizeof word, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda(e, "hs_paged_error");
  *out = word;
  if (word) return fail(HS_ERR_DEVICE, "hs_paged_error: the device error word is non-zero");
  return HS_OK;
}

}  // extern "C"
