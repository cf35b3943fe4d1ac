// sa_tma_host.cu -- host-side construction of TMA tensor maps (2D bf16, 3D bytes)
// through the driver entry point exposed by the runtime.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <mutex>

#include "sa_launch.h"

namespace sa {

static PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
static std::once_flag g_encode_once;

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// A [rows][cols] bf16 matrix whose rows are row_stride_bytes apart; boxes of
// box_rows x 64 columns land in shared memory in the 128-byte swizzled layout.
// Out-of-range box elements are filled with zeros.
bool make_tmap_bf16(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t row_stride_bytes,
                    uint32_t box_rows) {
  auto enc = encoder();
  if (!enc || !base || rows == 0 || cols == 0 || box_rows == 0 || box_rows > 256) return false;
  if (((uintptr_t)base & 15u) || (row_stride_bytes & 15u)) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// [rows][heads][d] codes of one byte: boxes of box_rows rows x box_d columns (64 or 128,
// the swizzle as wide) of one head, coordinates (column, head, row).
bool make_tmap_codes(CUtensorMap* map, const void* base, uint64_t rows, uint64_t heads, uint64_t d, uint32_t box_d,
                     uint32_t box_rows) {
  auto enc = encoder();
  if (!enc || !base || rows == 0 || heads == 0 || ((uintptr_t)base & 15u) || (d & 15u)) return false;
  if ((box_d != 64 && box_d != 128) || box_rows == 0 || box_rows > 256) return false;
  cuuint64_t dims[3] = {d, heads, rows};
  cuuint64_t strides[2] = {d, d * heads};
  cuuint32_t box[3] = {box_d, 1, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, box_d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace sa
