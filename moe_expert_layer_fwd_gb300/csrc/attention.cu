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
    attention_join_kernel(const KvBatch c, const AttentionArgs a, const AttentionParts p) {
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_sum[kJoinThreads / 32];
  pdl_wait();
  const JoinInfo j = p.info[blockIdx.x];
  if (!j.split || j.c0 != (int)blockIdx.x - 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = c.Hq / c.Hkv;
  const int row = (int)blockIdx.y * (kJoinThreads / 32 / kWarps) + warp / kWarps, sub = warp % kWarps;
  const int t0 = __ldg(c.q_start + j.b), t1 = __ldg(c.q_start + j.b + 1);
  const bool live = row < p.rows && j.row0 + row < (t1 - t0) * G;
  auto part = [&](int k) { return (size_t)(2 * k + (k == j.c0 ? j.slot0 : 0)) * p.rows + row; };
  float top = -CUDART_INF_F, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int k = j.c0 + lane; k <= j.c1; k += 32) top = fmaxf(top, p.rl[part(k)].x);
    top = warp_max(top);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll 4
    for (int k = j.c0 + sub; k <= j.c1; k += kWarps) {
      const float2 rl = p.rl[part(k)];
      const float4 o = reinterpret_cast<const float4*>(p.o + part(k) * kHeadDim)[lane];
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
  const size_t at = (size_t)(t0 + i) * c.Hq + j.h * G + rho - i * G;
  uint16_t* out = a.out + at * kHeadDim;
  reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) write_lse(a, at, top - p.base, sum);
}

// Ends two passes: out = sum_k 2^(x_k) o_k / sum_k 2^(x_k) l_k over what either left of a row, its parts where it was split (x = r - base)
// or else the row itself (x the logarithm of its denominator, l = 1), and lse = log2 of that denominator.  kWarps warps a row, as above.
struct PassRows {
  const int32_t* q_start;
  int B;
  const float* rows;
  const float* lse;
  AttentionParts parts;
};
// The parts of one row, as a pass left it.
struct RowParts {
  int n, c0, slot0;  // n parts, of the blocks from c0 on; c0 < 0: the row itself
  size_t row;        // of a part
  float whole;       // the row's denominator
};
__device__ __forceinline__ RowParts row_parts(const PassRows& s, int Hq, int G, int t, int head) {
  const size_t at = (size_t)t * Hq + head;
  RowParts r = {1, -1, 0, at, s.lse[at]};
  const unsigned mark = __float_as_uint(r.whole);
  if ((mark & 0xFFC00000u) != kSplitMark) return r;
  // (a row that no block wrote may hold anything: what it says is checked before it is used)
  const int k = (int)(mark & 0x3FFFFFu) + 1;
  r.n = 0;
  if (k >= s.parts.blocks) return r;
  const JoinInfo j = s.parts.info[k];
  if (!j.split || j.c0 != k - 1 || j.c1 < k || j.c1 >= s.parts.blocks || j.b < 0 || j.b >= s.B || (j.slot0 & ~1)) return r;
  const int rho = (t - __ldg(s.q_start + j.b)) * G + head - j.h * G - j.row0;
  if (rho < 0 || rho >= s.parts.rows) return r;
  r.n = j.c1 - j.c0 + 1;
  r.c0 = j.c0;
  r.slot0 = j.slot0;
  r.row = (size_t)rho;
  return r;
}
__device__ __forceinline__ size_t part_at(const PassRows& s, const RowParts& r, int k) {
  return (size_t)(2 * (r.c0 + k) + (k == 0 ? r.slot0 : 0)) * s.parts.rows + r.row;
}

template <int kWarps>
__global__ void __launch_bounds__(kJoinThreads)
    attention_end_kernel(const PassRows s0, const PassRows s1, int Hq, int G, long long rows, const AttentionArgs a) {
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_sum[kJoinThreads / 32];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kWarps;
  const long long row = (long long)blockIdx.x * (kJoinThreads / 32 / kWarps) + warp / kWarps;
  const bool live = row < rows;
  float top = -CUDART_INF_F, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    const int t = (int)(row / Hq), head = (int)(row - (long long)t * Hq);
    const RowParts r0 = row_parts(s0, Hq, G, t, head), r1 = row_parts(s1, Hq, G, t, head);
    auto highest = [&](const PassRows& s, const RowParts& r) {
      if (r.c0 < 0) {
        if (r.n) top = fmaxf(top, r.whole);
      } else {
        for (int k = lane; k < r.n; k += 32) top = fmaxf(top, s.parts.rl[part_at(s, r, k)].x - s.parts.base);
      }
    };
    highest(s0, r0);
    highest(s1, r1);
    top = warp_max(top);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    auto add = [&](float x, float l, const float4& o) {
      const float f = ex2(x - ref);
      sum = fmaf(l, f, sum);
      acc.x = fmaf(o.x, f, acc.x);
      acc.y = fmaf(o.y, f, acc.y);
      acc.z = fmaf(o.z, f, acc.z);
      acc.w = fmaf(o.w, f, acc.w);
    };
    auto add_all = [&](const PassRows& s, const RowParts& r, int from) {
      if (r.c0 < 0) {
        if (r.n && sub == from) add(r.whole, 1.f, reinterpret_cast<const float4*>(s.rows + r.row * kHeadDim)[lane]);
      } else {
#pragma unroll 4
        for (int k = sub; k < r.n; k += kWarps) {
          const size_t at = part_at(s, r, k);
          const float2 rl = s.parts.rl[at];
          add(rl.x - s.parts.base, rl.y, reinterpret_cast<const float4*>(s.parts.o + at * kHeadDim)[lane]);
        }
      }
    };
    add_all(s0, r0, 0);
    add_all(s1, r1, kWarps - 1);
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
  reinterpret_cast<uint2*>(a.out + (size_t)row * kHeadDim)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) write_lse(a, (size_t)row, top, sum);
}

}  // namespace

cudaError_t launch_attention_join(const KvBatch& c, const AttentionArgs& a, const AttentionParts& p, cudaStream_t stream) {
  constexpr int kAll = kJoinThreads / 32;
  if (p.rows <= 32) return launch_kernel(attention_join_kernel<kAll>, dim3(p.blocks, p.rows), dim3(kJoinThreads), 0, stream, true, c, a, p);
  return launch_kernel(attention_join_kernel<1>, dim3(p.blocks, (p.rows + kAll - 1) / kAll), dim3(kJoinThreads), 0, stream, true, c, a, p);
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
// from L2 whoever asks: one pass saves the second one's items and the rows in between (16 sequences of 20-240 tokens, 8 heads a
// key/value head, behind 4001: 241 us as two passes, 176 as one; 16 of 17 tokens 87 and 68; 64 of 33 tokens 255 and 268).  Below, rows of several
// sequences share the tiles.  But a mean says nothing of a batch of long and short ones: at least T / max_q of them are long, and each of
// the others may be an item of its own that goes over the whole prefix with a few rows.  So one pass is for batches where those are at
// most 0.4 of the items' number.  Decoding sequences and one chunk of tokens, 8 heads, behind 8200, as two passes and as one: 63 and 1100 tokens (1.7)
// 462 and 741 us, 63 and 4000 (0.5) 1373 and 1520, 15 and 1100 (0.43) 390 and 404, 63 and 8000 (0.25) 3081 and 3036, 15 and 4000 (0.12) 1304
// and 1174; 16 beside 8 of 200 tokens (0.32), behind 4001, 196 and 174.
bool shared_attention_joins(const KvBatch& prefixes, const KvBatch& c, int max_q) {
  const long long rows = (long long)c.T * (c.Hq / c.Hkv);
  const double items = (double)rows / 256.0, others = c.B - (double)c.T / (max_q > 0 ? max_q : 1);
  return rows > 128LL * c.B && others <= 0.4 * items && ((long long)prefixes.max_pages + c.max_pages) * c.page < (1LL << 31) - 2048;
}

// Two passes, each with the kernel that its rows per key/value head call for: over the prefixes, whose readers' tokens are one
// sequence that sees all of it (so a prefix is read once for all of them, and its rows fill the tiles), and over the sequences' own
// tokens; then one kernel that ends both, parts of split rows among them.  What is between them is fp32.  The second pass starts
// where the first one's blocks have ended: a block's way to its first scores takes 6 us.  (With each pass's parts joined by itself, and
// the second one adding the first one's rows: 64 sequences behind 8200 tokens 93 us instead of 84, 12 behind 224-943 64 instead of 33.)
cudaError_t launch_shared_attention(const KvBatch& prefixes, int max_prefix_q, const KvBatch& c, const AttentionArgs& args,
                                    const SharedBuffers& s, int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  if (!prefixes.B) {
    a.pass = 2;
    return launch_paged_attention(c, a, n_sms, stream);
  }
  if (shared_attention_joins(prefixes, c, a.max_q)) {
    a.pass = 3;
    a.n_prefixes = prefixes.B;
    a.prefix_max_pages = prefixes.max_pages;
    a.prefix_start = prefixes.q_start;
    a.prefix_len = prefixes.kv_len;
    a.prefix_table = prefixes.page_table;
    return launch_paged_attention(c, a, n_sms, stream);
  }
  PassRows left[2] = {{prefixes.q_start, prefixes.B, s.rows[0], s.lse[0], {}}, {c.q_start, c.B, s.rows[1], s.lse[1], {}}};
  for (int i = 0; i < 2; ++i) {
    AttentionArgs p = a;
    p.pass = 1;
    p.follows = i;
    p.out32 = s.rows[i];
    p.lse = s.lse[i];
    p.lse_unit = 1.f;
    if (i == 0) {
      p.causal = 0;
      p.max_q = max_prefix_q;
      p.scratch = s.prefix_scratch;
    }
    const cudaError_t e = launch_paged_attention(i == 0 ? prefixes : c, p, n_sms, stream, &left[i].parts);
    if (e != cudaSuccess) return e;
  }
  // Eight warps a row where rows are few and may have many parts: with 128-608 rows the two are within 2 us of one another (4-19 sequences
  // of 32 heads behind 500 and 8200), but 54 and 48 us for 128 rows behind 30000; with 4096 rows a warp each takes 71 us and eight 79.
  constexpr int kAll = kJoinThreads / 32;
  const long long rows = (long long)c.T * c.Hq;
  const int G = c.Hq / c.Hkv;
  if (rows <= 4LL * n_sms)
    return launch_kernel(attention_end_kernel<kAll>, dim3((unsigned)rows), dim3(kJoinThreads), 0, stream, true, left[0], left[1], c.Hq, G, rows, a);
  return launch_kernel(attention_end_kernel<1>, dim3((unsigned)((rows + kAll - 1) / kAll)), dim3(kJoinThreads), 0, stream, true, left[0], left[1],
                       c.Hq, G, rows, a);
}

cudaError_t launch_kv_weights(const KvBatch& c, const AttentionArgs& args, const float* lse, const float* weight_in, float* weight_out,
                              int n_sms, cudaStream_t stream) {
  AttentionArgs a = args;
  a.limit_us = g_limit_us;
  a.withhold = g_withhold;
  return launch_kv_weights_rows(c, a, lse, weight_in, weight_out, n_sms, stream);
}

cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& args, int n_sms, cudaStream_t stream, AttentionParts* parts) {
  AttentionArgs a = args;
  a.limit_us = g_limit_us;
  a.withhold = g_withhold;
  const bool few = attention_decode_fits(c.Hq / c.Hkv, a.max_q) ||
                   (a.pass == 1 && attention_decode_chunks_fit(c, a.max_q, n_sms));
  return few ? launch_attention_decode(c, a, n_sms, stream, parts) : launch_attention_prefill(c, a, n_sms, stream, parts);
}

}  // namespace moe
