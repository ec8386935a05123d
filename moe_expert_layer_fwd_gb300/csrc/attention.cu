// Softmax attention of new queries over the paged 8-bit cache.
#include "attention_internal.h"

#include <cudaTypedefs.h>

#include <mutex>

namespace moe {
bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const KvBatch& c, int box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  if (!encode) return false;
  const cuuint64_t rows = (cuuint64_t)(c.n_pages > 0 ? c.n_pages : 1) * c.Hkv * c.page;
  const cuuint64_t dims[2] = {kHeadDim, rows}, strides[1] = {kHeadDim};
  const cuuint32_t box[2] = {kHeadDim, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Up to 32 rows per key/value head the products are memory bound on either kernel and the one that keeps the keys as
// the large operand reads the cache at its rate; above, a 128-row product is no longer mostly padding.
size_t attention_scratch_bytes(int Hq, int Hkv, int max_q, int n_sms) {
  const int G = Hq / Hkv;
  return attention_decode_fits(G, max_q) ? attention_decode_scratch(G, max_q, n_sms) : attention_prefill_scratch(n_sms);
}

cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream) {
  return attention_decode_fits(c.Hq / c.Hkv, a.max_q) ? launch_attention_decode(c, a, n_sms, stream)
                                                      : launch_attention_prefill(c, a, n_sms, stream);
}

}  // namespace moe
