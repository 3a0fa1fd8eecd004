// Host side of the paged attention: the tensor map of a layer's pool, the choice of
// the kernel, and the workspace.
#include "hs_paged_attention.cuh"

namespace hs {

cudaError_t paged_decode_d64(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st);
cudaError_t paged_decode_d128(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st);
cudaError_t paged_decode_d256(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st);
cudaError_t prepare_paged_d64(int group, int type, int page_type);
cudaError_t prepare_paged_d128(int group, int type, int page_type);
cudaError_t prepare_paged_d256(int group, int type, int page_type);

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

}  // namespace

int64_t paged_workspace_bytes(int d, int group, int page_type, int ctas) {
  const bool e = page_type == HS_E4M3, two = group > 8;
  size_t n;
  if (d == 64)
    n = e ? (two ? pa::ws_bytes<64, 2, true>(ctas) : pa::ws_bytes<64, 1, true>(ctas))
          : (two ? pa::ws_bytes<64, 2, false>(ctas) : pa::ws_bytes<64, 1, false>(ctas));
  else if (d == 128)
    n = e ? (two ? pa::ws_bytes<128, 2, true>(ctas) : pa::ws_bytes<128, 1, true>(ctas))
          : (two ? pa::ws_bytes<128, 2, false>(ctas) : pa::ws_bytes<128, 1, false>(ctas));
  else
    n = e ? (two ? pa::ws_bytes<256, 2, true>(ctas) : pa::ws_bytes<256, 1, true>(ctas))
          : (two ? pa::ws_bytes<256, 2, false>(ctas) : pa::ws_bytes<256, 1, false>(ctas));
  return (int64_t)((n + 255) / 256 * 256);
}

bool paged_maps(hs_paged* h, size_t layer_bytes) {
  for (int l = 0; l < h->cfg.n_layers; ++l)
    if (!pool_map(h->cfg, static_cast<unsigned char*>(h->pages) + layer_bytes * l, &h->maps[l])) return false;
  return true;
}

cudaError_t prepare_paged(int d, int group, int type, int page_type) {
  return d == 64    ? prepare_paged_d64(group, type, page_type)
         : d == 128 ? prepare_paged_d128(group, type, page_type)
                    : prepare_paged_d256(group, type, page_type);
}

cudaError_t launch_paged_decode(PagedDecodeParams p, const CUtensorMap& map, cudaStream_t st) {
  // the most units a request can have: a window may lie across one more than it fills
  const int units = p.max_pages << (p.page_shift - 4);
  const int most = p.window > 0 ? std::min(units, p.window / pa::UNIT + 2) : units;
  p.whole = most <= (p.n_req * p.h_kv >= pa::MANY_SEGMENTS ? pa::WHOLE_UNITS_MANY : pa::WHOLE_UNITS);
  return p.d == 64 ? paged_decode_d64(p, map, st) : p.d == 128 ? paged_decode_d128(p, map, st) : paged_decode_d256(p, map, st);
}

}  // namespace hs
