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
template <int kWarps, int kPass>
__global__ void __launch_bounds__(kJoinThreads)
    attention_join_kernel(const KvBatch c, const AttentionArgs a, int rows, float base, const float* part_o,
                          const float2* part_rl, const JoinInfo* info) {
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_sum[kJoinThreads / 32];
  if (kPass == 1) pdl_launch_dependents();
  pdl_wait();
  const JoinInfo j = info[blockIdx.x];
  if (!j.split || j.c0 != (int)blockIdx.x - 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = c.Hq / c.Hkv;
  const int row = (int)blockIdx.y * (kJoinThreads / 32 / kWarps) + warp / kWarps, sub = warp % kWarps;
  const int t0 = __ldg(c.q_start + j.b), t1 = __ldg(c.q_start + j.b + 1);
  const bool live = row < rows && j.row0 + row < (t1 - t0) * G;
  auto part = [&](int k) { return (size_t)(2 * k + (k == j.c0 ? j.slot0 : 0)) * rows + row; };
  const int rho = j.row0 + row, i = rho / G;
  const size_t at = (size_t)(t0 + i) * c.Hq + j.h * G + rho - i * G;
  float before = -CUDART_INF_F;  // of the pass before, on its way while the parts are read
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  if (kPass == 2 && live && a.prior) {
    before = prior_lse(a, at);
    p = reinterpret_cast<const float4*>(a.prior + at * kHeadDim)[lane];
  }
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
  if (kPass > 0) {
    const RowEnd e = end_row<kPass>(a, at, inv, top - base, sum, before, lane == 0);
    acc = make_float4(acc.x * e.f, acc.y * e.f, acc.z * e.f, acc.w * e.f);
    if (kPass == 2 && a.prior) {
      acc = make_float4(fmaf(p.x, e.f1, acc.x), fmaf(p.y, e.f1, acc.y), fmaf(p.z, e.f1, acc.z), fmaf(p.w, e.f1, acc.w));
    }
    if (kPass == 1) reinterpret_cast<float4*>(a.out32 + at * kHeadDim)[lane] = acc;
    else reinterpret_cast<uint2*>(a.out + at * kHeadDim)[lane] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    return;
  }
  uint16_t* out = a.out + at * kHeadDim;
  reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace

cudaError_t launch_attention_join(const KvBatch& c, const AttentionArgs& args, int blocks, int rows, float base, const float* part_o,
                                  const float2* part_rl, const JoinInfo* info, cudaStream_t stream) {
  AttentionArgs a = args;
  if (a.pass == 3) a.prior = nullptr;  // the prefixes' tables lie there; their keys are in the sums
  constexpr int kAll = kJoinThreads / 32;
  auto kern = rows <= 32 ? (a.pass == 0 ? attention_join_kernel<kAll, 0> : a.pass == 1 ? attention_join_kernel<kAll, 1> : attention_join_kernel<kAll, 2>)
                         : (a.pass == 0 ? attention_join_kernel<1, 0> : a.pass == 1 ? attention_join_kernel<1, 1> : attention_join_kernel<1, 2>);
  const dim3 grid(blocks, rows <= 32 ? rows : (rows + kAll - 1) / kAll);
  return launch_kernel(kern, grid, dim3(kJoinThreads), 0, stream, true, c, a, rows, base, part_o, part_rl, info);
}

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return encode;
}

bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const KvBatch& c) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t rows = (cuuint64_t)(c.n_pages > 0 ? c.n_pages : 1) * c.Hkv * c.page;
  const cuuint64_t dims[2] = {kHeadDim, rows}, strides[1] = {kHeadDim};
  const cuuint32_t box[2] = {kHeadDim, (cuuint32_t)c.page}, step[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_query_map(CUtensorMap* m, const AttentionArgs& a, const KvBatch& c, int heads, int tokens) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)c.Hq, (cuuint64_t)c.T};
  const cuuint64_t strides[2] = {kHeadDim * sizeof(uint16_t), (cuuint64_t)a.q_stride * sizeof(uint16_t)};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens}, step[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), dims, strides, box, step,
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

// Above 128 rows per key/value head and sequence, on average, an item of 256 rows is a sequence's own anyhow, and the prefix's tiles come
// from L2 whoever asks: one pass saves the second one's items and the rows in between (16 sequences of 20-250 tokens, 8 heads a
// key/value head, behind 4001: 254 us as two passes, 191 as one).  Below, rows of several sequences share the tiles.
bool shared_attention_joins(const KvBatch& prefixes, const KvBatch& c) {
  return (long long)c.T * (c.Hq / c.Hkv) > 128LL * c.B &&
         ((long long)prefixes.max_pages + c.max_pages) * c.page < (1LL << 31) - 2048;
}

// Two passes, each with the kernel that its rows per key/value head call for: over the prefixes, whose readers' tokens are one
// sequence that sees all of it (so a prefix is read once for all of them, and its rows fill the tiles), then over the
// sequences' own tokens, whose ends add the first pass's rows.  The rows in between are fp32.  The second pass starts while the
// first one ends (scratch of its own, and it waits for the first one's rows where it needs them): a block's way to its first
// scores takes 6 us.
cudaError_t launch_shared_attention(const KvBatch& prefixes, int max_prefix_q, void* prefix_scratch, const KvBatch& c,
                                    const AttentionArgs& args, float* rows, float* rows_lse, int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  a.pass = 2;
  if (prefixes.B && !rows) {
    a.pass = 3;
    a.n_prefixes = prefixes.B;
    a.prefix_max_pages = prefixes.max_pages;
    a.prefix_start = prefixes.q_start;
    a.prefix_len = prefixes.kv_len;
    a.prefix_table = prefixes.page_table;
  }
  if (rows) {
    AttentionArgs p = a;
    p.pass = 1;
    p.causal = p.window = 0;
    p.max_q = max_prefix_q;
    p.scratch = prefix_scratch;
    p.out32 = rows;
    p.lse = rows_lse;
    p.lse_unit = 1.f;
    const cudaError_t e = launch_paged_attention(prefixes, p, n_sms, stream);
    if (e != cudaSuccess) return e;
    a.prior = rows;
    a.prior_lse = rows_lse;
  }
  return launch_paged_attention(c, a, n_sms, stream);
}

cudaError_t launch_kv_weights(const KvBatch& c, const AttentionArgs& args, const float* lse, const float* weight_in, float* weight_out,
                              int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  a.limit_us = g_limit_us;
  a.withhold = g_withhold;
  return launch_kv_weights_rows(c, a, lse, weight_in, weight_out, n_sms, stream);
}

cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& args, int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  a.limit_us = g_limit_us;
  a.withhold = g_withhold;
  const bool few = attention_decode_fits(c.Hq / c.Hkv, a.max_q) ||
                   ((a.pass == 1 || a.pass == 2) && attention_decode_chunks_fit(c, a.max_q, n_sms));
  return few ? launch_attention_decode(c, a, n_sms, stream) : launch_attention_prefill(c, a, n_sms, stream);
}

}  // namespace moe
