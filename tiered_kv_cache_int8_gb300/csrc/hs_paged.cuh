// Shared between the rotary / append kernels (hs_rotary.cu), the paged
// attention kernels (hs_paged_attention.cu) and their host side (hs_paged.cu).
#ifndef HS_PAGED_CUH_
#define HS_PAGED_CUH_

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <memory>

#include "hs_internal.cuh"

struct hs_paged {
  hs_paged_config_t cfg;
  void* pages = nullptr;
  const float* kv_scale = nullptr;
  unsigned int* dev_error = nullptr;
  std::unique_ptr<CUtensorMap[]> maps;   // of each layer's pool, for one-token attention and, behind
                                         // those, for prompts; null without a device
  int ctas = 0;                          // of the attention kernel; 0 without a device
  int page_shift = 0;
  float scale = 0.f, scale_log2 = 0.f;
  float softcap = 0.f;                   // 0: none
  const float* slopes = nullptr;         // null: none
};

namespace hs {

constexpr int PG_MAX_REQUESTS = 4096;
constexpr int PG_MAX_POSITIONS = 1 << 22;
constexpr int PG_MAX_CTAS = 160;   // of the attention kernel: one per SM; its join holds five pieces a lane

constexpr int PG_UNIT = 16;        // positions of one head that lie together in every kind of page

inline size_t type_bytes(int t) { return t == HS_FP32 ? 4 : t == HS_E4M3 ? 1 : 2; }
// bytes of PG_UNIT rows of one head's keys or values
__host__ __device__ inline size_t unit_bytes(int d, int page_type) {
  return page_type == HS_INT4 ? 9 * d : page_type == HS_E4M3 ? 16 * d : 32 * d;
}
// The pages' kinds that kernels are made for.
enum Pages { PAGES_SAME = 0, PAGES_E4M3 = 1, PAGES_INT4 = 2 };
inline Pages pages_kind(int page_type) {
  return page_type == HS_INT4 ? PAGES_INT4 : page_type == HS_E4M3 ? PAGES_E4M3 : PAGES_SAME;
}

// One tensor of a rotation or append: rows of `heads` heads per token.
enum ViewKind { VIEW_ROTATE = 0, VIEW_KEYS = 1, VIEW_VALUES = 2 };
struct RowView {
  const void* in;
  void* out;          // VIEW_ROTATE only
  int64_t in_ts, in_hs, out_ts, out_hs;
  int32_t heads;
  int32_t kind;
  int32_t chunk_heads, chunks;   // heads of a thread, threads for a row's heads
};

struct RotateParams {
  RowView v[3];
  int32_t n_views;
  int32_t d;
  int32_t n_tok;
  uint32_t first_cta[3]; // of each view
  int32_t groups;        // (token, chunk of heads) pairs of a CTA
  int32_t rot_dim;       // 0: no rotation
  int32_t items;         // work items of a row
  float magnitude;
  float sign;            // -1: the transposed rotation
  const uint64_t* turns;
  const int32_t* positions;   // hs_rotary_apply
  // append
  const int32_t* req_ids;
  const int32_t* tok_offsets;
  const int32_t* page_table;
  const int32_t* lengths;
  int32_t* next_lengths;
  int32_t n_req, tok_per_req, max_requests, max_pages, n_pages, page_size, page_shift, h_kv;
  unsigned char* pages;       // of the layer
  const float* kv_scale;      // of the layer
  unsigned int* dev_error;
};

struct PagedDecodeParams {
  const int32_t* req_ids;
  const int32_t* page_table;
  const int32_t* lengths;
  const void* q;
  int64_t q_ts, q_hs;
  void* out;
  float* lse;
  float* ws;
  const unsigned char* pages;  // of the layer
  const float* kv_scale;       // of the layer, or null
  unsigned int* dev_error;
  int32_t n_req, max_requests, max_pages, n_pages, page_size, page_shift;
  int32_t h_q, h_kv, group, d, window, type, page_type;
  int32_t grid;
  int32_t whole;         // every CTA takes whole segments
  float scale_log2;
  // scores with a cap or a bias (prepared by scores_of)
  float cap_in;          // scale / cap (the scale's factor in place of scale_log2); 0: no cap
  float cap_log2;        // cap * log2(e)
  const float* slopes;   // [h_q], or null
};

struct PagedAttendParams {
  const int32_t* req_ids;
  const int32_t* tok_offsets;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* prefix;       // or null
  const void* q;
  int64_t q_ts, q_hs;
  void* out;
  float* lse;
  float* ws;
  const unsigned char* pages;  // of the layer
  const float* kv_scale;       // of the layer, or null
  unsigned int* dev_error;
  int32_t n_req, n_tok, tok_per_req, max_requests, max_pages, n_pages, page_size, page_shift;
  int32_t h_q, h_kv, group, d, window, type, page_type;
  int32_t grid;
  float scale_log2, cap_in, cap_log2;
  const float* slopes;
};

cudaError_t launch_append4(const RotateParams& p, int type, bool interleaved, bool wide, cudaStream_t st);
cudaError_t launch_read(const RotateParams& p, int type, int page_type, cudaStream_t st);
cudaError_t prepare_rows(int d, int type, int page_type);
cudaError_t launch_paged_attend(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st);
int attend_box_rows(int d, int page_size);   // of a copy of 16-bit pages
cudaError_t prepare_attend(int d, int type, int page_type);
int64_t attend_workspace_bytes(int d, int ctas);
cudaError_t launch_rotate(const RotateParams& p, int type, int page_type, bool append, bool interleaved,
                          bool wide, cudaStream_t st);
cudaError_t launch_paged_decode(PagedDecodeParams p, const CUtensorMap& map, cudaStream_t st);
// load the kernels of a configuration on the current device and set what they need
cudaError_t prepare_paged(int d, int group, int type, int page_type, bool scores);
cudaError_t prepare_rotate(int type, int page_type, bool append);
bool paged_maps(::hs_paged* h, size_t layer_bytes);   // false: no tensor maps could be made
int64_t paged_workspace_bytes(int d, int group, int page_type, int ctas);

}  // namespace hs

#endif  // HS_PAGED_CUH_
