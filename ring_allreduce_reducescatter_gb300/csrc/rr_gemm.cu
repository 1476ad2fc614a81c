// rr_gemm.cu -- the tensor maps of the 16-bit products' operands.
#include "rr_gemm.cuh"

namespace rr {

namespace gemm {

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

}  // namespace

bool make_operand_map(CUtensorMap *map, const Operand &o, int box) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  // (the elements' format does not matter to a copy; outside the matrix it reads zeros)
  const cuuint64_t inner = (cuuint64_t)(o.mn ? o.rows : o.k), outer = (cuuint64_t)(o.mn ? o.k : o.rows);
  const cuuint64_t dims[3] = {inner, outer, (cuuint64_t)o.batch};
  const cuuint64_t pitch = (cuuint64_t)o.ld * 2;
  const cuuint64_t strides[2] = {pitch, o.batch > 1 ? (cuuint64_t)o.batch_stride * 2 : pitch * outer};
  const cuuint32_t boxes[3] = {kStep, o.mn ? kStep : (cuuint32_t)box, 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(o.at), dims, strides, boxes, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemm

}  // namespace rr
