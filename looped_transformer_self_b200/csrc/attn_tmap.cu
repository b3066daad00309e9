// TMA descriptors of the attention operators.
#include "attn_tc.cuh"

namespace lt {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

int attn_tmap(CUtensorMap* map, const void* base, int hd, int heads, long long tokens, long long stride,
              int box_heads, int box_tokens, int box_chunks) {
  static EncodeTiledFn enc = nullptr;
  if (!enc) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return -1;
    enc = (EncodeTiledFn)p;
  }
  const int chunks = hd == 128 ? 2 : 1;
  cuuint64_t dims[4] = {(cuuint64_t)(hd / chunks), (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)chunks};
  cuuint64_t strides[3] = {(cuuint64_t)hd * 2, (cuuint64_t)stride * 2, 128};
  cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, (cuuint32_t)(box_chunks < chunks ? box_chunks : chunks)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : -3;
}

}  // namespace lt
