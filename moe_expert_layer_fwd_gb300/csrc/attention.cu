// Softmax attention of new queries over the paged 8-bit cache.
#include "attention_tiles.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

// out = sum_k 2^(r_k - r) o_k / sum_k 2^(r_k - r) l_k over an item's parts, in their order.  kWarps warps share a row and
// split its parts (few rows, many parts: decoding), or each has a row (kWarps = 1); a lane has four dims.  Blocks whose run
// (blockIdx.x) does not hold an item's second part have nothing to do.
template <int kWarps>
__global__ void __launch_bounds__(kJoinThreads)
    attention_join_kernel(const KvBatch c, const AttentionArgs a, int rows, const float* part_o, const float2* part_rl,
                          const JoinInfo* info) {
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_sum[kJoinThreads / 32];
  pdl_wait();
  const JoinInfo j = info[blockIdx.x];
  if (!j.split || j.c0 != (int)blockIdx.x - 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = c.Hq / c.Hkv;
  const int row = (int)blockIdx.y * (kJoinThreads / 32 / kWarps) + warp / kWarps, sub = warp % kWarps;
  const int t0 = __ldg(c.q_start + j.b), t1 = __ldg(c.q_start + j.b + 1);
  const bool live = row < rows && j.row0 + row < (t1 - t0) * G;
  auto part = [&](int k) { return (size_t)(2 * k + (k == j.c0 ? j.slot0 : 0)) * rows + row; };
  float top = -CUDART_INF_F, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int k = j.c0 + lane; k <= j.c1; k += 32) top = fmaxf(top, part_rl[part(k)].x);
    top = warp_max(top);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll 4
    for (int k = j.c0 + sub; k <= j.c1; k += kWarps) {
      const float2 rl = part_rl[part(k)];
      const float4 o = reinterpret_cast<const float4*>(part_o + part(k) * kHeadDim)[lane];
      const float f = ex2(rl.x - ref);
      sum = fmaf(rl.y, f, sum);
      acc.x = fmaf(o.x, f, acc.x);
      acc.y = fmaf(o.y, f, acc.y);
      acc.z = fmaf(o.z, f, acc.z);
      acc.w = fmaf(o.w, f, acc.w);
    }
  }
  if (kWarps > 1) {
    s_acc[threadIdx.x] = acc;
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 o = s_acc[threadIdx.x + 32 * w];
      sum += s_sum[warp + w];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
  }
  if (!live) return;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int rho = j.row0 + row, i = rho / G;
  uint16_t* out = a.out + ((size_t)(t0 + i) * c.Hq + j.h * G + rho - i * G) * kHeadDim;
  reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace

cudaError_t launch_attention_join(const KvBatch& c, const AttentionArgs& a, int blocks, int rows, const float* part_o,
                                  const float2* part_rl, const JoinInfo* info, cudaStream_t stream) {
  constexpr int kAll = kJoinThreads / 32;
  if (rows <= 32) return launch_kernel(attention_join_kernel<kAll>, dim3(blocks, rows), dim3(kJoinThreads), 0, stream, true, c, a, rows, part_o, part_rl, info);
  return launch_kernel(attention_join_kernel<1>, dim3(blocks, (rows + kAll - 1) / kAll), dim3(kJoinThreads), 0, stream, true, c, a, rows, part_o, part_rl, info);
}

bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const KvBatch& c) {
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
  const cuuint32_t box[2] = {kHeadDim, (cuuint32_t)c.page}, step[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// By the rows of one key/value head that a sequence brings (32 sequences of 4000-8000 tokens, 4 key/value heads): at 16 rows
// the kernel with the keys as the large operand takes 69 us and the one with the rows 87 us (whose tile has 128 of them,
// whatever is used), at 24 rows it is 96 against 87 us, at 32 rows 103 against 87 us.
size_t attention_scratch_bytes(int Hq, int Hkv, int max_q, int n_sms) {
  const int G = Hq / Hkv;
  return attention_decode_fits(G, max_q) ? attention_decode_scratch(G, max_q, n_sms) : attention_prefill_scratch(G, max_q, n_sms);
}

static unsigned g_limit_us = 2000000;
static int g_withhold = 0;

int attention_debug_set(int what, unsigned long long value) {
  if (what == 1) g_limit_us = value == 0 ? 2000000u : value < 2000000000ull ? (unsigned)(value / 1000 + 1) : 2000000u;
  else if (what == 4) g_withhold = value != 0;
  else return -1;
  return 0;
}

cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& args, int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  a.limit_us = g_limit_us;
  a.withhold = g_withhold;
  return attention_decode_fits(c.Hq / c.Hkv, a.max_q) ? launch_attention_decode(c, a, n_sms, stream)
                                                      : launch_attention_prefill(c, a, n_sms, stream);
}

}  // namespace moe
