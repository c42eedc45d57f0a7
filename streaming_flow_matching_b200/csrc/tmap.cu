// Host-side creation of TMA tensor maps (cuTensorMapEncodeTiled, fetched from
// the driver through the runtime so that the library itself does not link
// against libcuda and still loads on a machine without a GPU driver).
#include <mutex>

#include "sm100.cuh"

namespace sfm {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
std::once_flag g_once;

void load_encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = (EncodeTiledFn)fn;
  else
    cudaGetLastError();
}

}  // namespace

int make_tmap_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                   const uint64_t* strides_bytes, const uint32_t* box) {
  std::call_once(g_once, load_encoder);
  if (!g_encode) return SFM_ECUDA;
  if (rank < 2 || rank > 5 || ((uintptr_t)base & 15u)) return SFM_EINVAL;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], e[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    e[i] = 1;
  }
  for (int i = 0; i + 1 < rank; ++i) {
    if (strides_bytes[i] % 16) return SFM_EINVAL;
    s[i] = strides_bytes[i];
  }
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                              const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SFM_OK : SFM_EINVAL;
}

int make_rows_map(CUtensorMap* m, const void* p, long long rows, int heads, int box_rows) {
  const uint64_t dims[3] = {128, (uint64_t)heads, (uint64_t)rows};
  const uint64_t strides[2] = {256, (uint64_t)heads * 256};
  const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
  return make_tmap_bf16(m, p, 3, dims, strides, box);
}

}  // namespace sfm
