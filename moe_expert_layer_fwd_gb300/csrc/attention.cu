// Softmax attention of new queries over the paged 8-bit cache.
#include "attention_common.cuh"

#include <cudaTypedefs.h>
#include <math_constants.h>

#include <mutex>

namespace moe {
namespace {

// One block per (new token, query head): 128 threads take one key each, then one output element each.
__global__ void __launch_bounds__(128) attention_simple_kernel(const KvBatch c, const AttentionArgs a) {
  __shared__ float s_q[kHeadDim], s_p[128], s_red[4], s_vs[128];
  __shared__ size_t s_row[128];
  const int t = blockIdx.x / c.Hq, hq = blockIdx.x - t * c.Hq, h = hq / (c.Hq / c.Hkv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = warp_search(c.B, t, [&](int i) { return __ldg(c.q_start + i); });
  SeqRange s;
  if (!load_seq(c, b, s) || t < s.t0 || t >= s.t1) return;
  const int pos = s.first() + t - s.t0;
  const int end = a.causal ? min(s.len, pos + 1) : s.len;
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  s_q[tid] = __uint_as_float((uint32_t)a.q[(size_t)t * a.q_stride + hq * kHeadDim + tid] << 16);
  __syncthreads();
  float m = -CUDART_INF_F, sum = 0.f, acc = 0.f;
  for (int j0 = begin; j0 < end; j0 += 128) {
    const int j = j0 + tid;
    float z = -CUDART_INF_F;
    int pg = -1;
    if (j < end) pg = load_page(c, b, j >> c.page_log2);
    s_row[tid] = 0;
    s_vs[tid] = 0.f;
    if (pg >= 0) {
      const size_t unit = (size_t)pg * c.Hkv + h;
      const size_t row = ((unit << c.page_log2) + (j & (c.page - 1))) * kHeadDim;
      const uint32_t* k = reinterpret_cast<const uint32_t*>(c.k_codes + row);
      float dot = 0.f;
      for (int i = 0; i < kHeadDim / 4; ++i) {
        const uint32_t w = __ldg(k + i);
        const float2 x = e4m3x2_f32(w & 0xFFFFu), y = e4m3x2_f32(w >> 16);
        dot += s_q[4 * i] * x.x + s_q[4 * i + 1] * x.y + s_q[4 * i + 2] * y.x + s_q[4 * i + 3] * y.y;
      }
      z = dot * exp2f((float)((int)__ldg(c.k_scale + unit) - 127)) * a.scale_log2;
      s_row[tid] = row;
      s_vs[tid] = exp2f((float)((int)__ldg(c.v_scale + unit) - 127));
    }
    float top = z;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
    const float m2 = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float ref = m2 == -CUDART_INF_F ? 0.f : m2;
    const float p = pg >= 0 ? exp2f(z - ref) : 0.f;
    s_p[tid] = p;
    const float fix = exp2f(m - ref);
    m = m2;
    __syncthreads();
    float add = 0.f;
    acc *= fix;
    for (int i = 0; i < 128; ++i) {
      const float w = s_p[i];
      add += w;
      if (w != 0.f) {
        __half_raw hr = __nv_cvt_fp8_to_halfraw(c.v_codes[s_row[i] + tid], __NV_E4M3);
        acc += w * (s_vs[i] * __half2float(__half(hr)));
      }
    }
    sum = sum * fix + add;
    __syncthreads();
  }
  a.out[((size_t)t * c.Hq + hq) * kHeadDim + tid] = f32_to_bf16_rne(sum != 0.f ? acc / sum : 0.f);
}

}  // namespace

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

size_t attention_scratch_bytes(int, int, int Hq, int Hkv, int max_q, int n_sms) {
  const int G = Hq / Hkv;
  return attention_decode_fits(G, max_q) ? attention_decode_scratch(G, max_q, n_sms) : 0;
}

cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream) {
  if (attention_decode_fits(c.Hq / c.Hkv, a.max_q)) return launch_attention_decode(c, a, n_sms, stream);
  attention_simple_kernel<<<(unsigned)((size_t)c.T * c.Hq), 128, 0, stream>>>(c, a);
  return cudaGetLastError();
}

}  // namespace moe
