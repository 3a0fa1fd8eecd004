// Host side of the paged attention: the tensor map of a layer's pool, the choice of
// the kernel, and the workspace.
#include "hs_paged_attention.cuh"

namespace hs {

namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

// The layer's pool as [keys or values][block of a row][row][bytes of the block]: one
// copy brings 16 rows of keys and of values, each block's rows together and swizzled.
bool pool_map(const hs_paged_config_t& p, void* pages, CUtensorMap* map) {
  const Encode encode = encoder();
  if (!encode) return false;
  const int es = p.page_type == HS_E4M3 ? 1 : 2;
  const int row = std::min(p.d * es, 128);            // bytes of a row in one block
  const cuuint64_t dims[4] = {(cuuint64_t)(row / es), (cuuint64_t)p.n_pages * 2 * p.h_kv * p.page_size,
                              (cuuint64_t)(p.d * es / row), 2};
  const cuuint64_t strides[3] = {(cuuint64_t)p.d * es, (cuuint64_t)row, (cuuint64_t)p.h_kv * p.page_size * p.d * es};
  const cuuint32_t box[4] = {(cuuint32_t)(row / es), pa::UNIT, (cuuint32_t)(p.d * es / row), 2};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                            pages, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The pool as rows of 64-element blocks: a copy brings some rows of one block.
bool rows_map(const hs_paged_config_t& p, void* pages, CUtensorMap* map) {
  const Encode encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)p.n_pages * 2 * p.h_kv * p.page_size, (cuuint64_t)(p.d / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)attend_box_rows(p.d, p.page_size), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, pages, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// f(head width, kind of page) as constants
template <typename F>
auto by_pages(int d, int page_type, F f) {
  auto with = [&](auto dd) {
    const Pages k = pages_kind(page_type);
    return k == PAGES_INT4   ? f(dd, std::integral_constant<int, PAGES_INT4>{})
           : k == PAGES_E4M3 ? f(dd, std::integral_constant<int, PAGES_E4M3>{})
                             : f(dd, std::integral_constant<int, PAGES_SAME>{});
  };
  return d == 64    ? with(std::integral_constant<int, 64>{})
         : d == 128 ? with(std::integral_constant<int, 128>{})
                    : with(std::integral_constant<int, 256>{});
}

int64_t paged_workspace_bytes(int d, int group, int page_type, int ctas) {
  const size_t n = by_pages(d, page_type, [&](auto dd, auto pages) {
    return group > 8 ? pa::ws_bytes<dd(), 2, pages()>(ctas) : pa::ws_bytes<dd(), 1, pages()>(ctas);
  });
  return (int64_t)((n + 255) / 256 * 256);
}

bool paged_maps(hs_paged* h, size_t layer_bytes) {
  if (h->cfg.page_type == HS_INT4) return true;       // plain copies: units lie together
  const bool rows = h->cfg.page_type == h->cfg.type;  // (8-bit rows are turned into fp16 on the way to prompts)
  for (int l = 0; l < h->cfg.n_layers; ++l) {
    unsigned char* pages = static_cast<unsigned char*>(h->pages) + layer_bytes * l;
    if (!pool_map(h->cfg, pages, &h->maps[l])) return false;
    if (rows && !rows_map(h->cfg, pages, &h->maps[(size_t)h->cfg.n_layers + l])) return false;
  }
  return true;
}

cudaError_t prepare_paged(int d, int group, int type, int page_type, bool scores) {
  return by_pages(d, page_type, [&](auto dd, auto pages) {
    return scores ? pa::prepare_paged_of<dd(), pages(), true>(group, type) : pa::prepare_paged_of<dd(), pages(), false>(group, type);
  });
}

cudaError_t launch_paged_decode(PagedDecodeParams p, const CUtensorMap& map, cudaStream_t st) {
  // the most units a request can have: a window may lie across one more than it fills
  const int units = p.max_pages << (p.page_shift - 4);
  const int most = p.window > 0 ? std::min(units, p.window / pa::UNIT + 2) : units;
  p.whole = most <= (p.n_req * p.h_kv >= pa::MANY_SEGMENTS ? pa::WHOLE_UNITS_MANY : pa::WHOLE_UNITS);
  const bool scores = p.cap_in != 0.f || p.slopes;
  return by_pages(p.d, p.page_type, [&](auto dd, auto pages) {
    return scores ? pa::paged_decode_of<dd(), pages(), true>(p, map, st) : pa::paged_decode_of<dd(), pages(), false>(p, map, st);
  });
}

}  // namespace hs
