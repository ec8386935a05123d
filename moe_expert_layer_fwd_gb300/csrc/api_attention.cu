// C-ABI entry points of the attention operators: host-side validation and launches.
// Declarations and full argument documentation are in include/moe.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe.h"
#include "attention_internal.h"

namespace {

constexpr size_t kHeader = 256;  // status word + padding, as in every workspace
constexpr long long kMaxRows = 1LL << 31;
constexpr long long kMaxLen = kMaxRows - 1024;  // tokens of a sequence: the ends of its tiles and rows are ints, too

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ok_ptr(const void* p) { return p && aligned16(p); }

// SMs of the current device, asked once per device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

int check_desc(const moe_kv_desc* d) {
  if (!d || d->B < 0 || d->T < 0 || d->Hq < 1 || d->Hkv < 1 || d->D < 1 || d->page < 1 || d->n_pages < 0 ||
      d->max_pages < 0)
    return MOE_ERR_INVALID_ARG;
  if (d->Hq % d->Hkv != 0) return MOE_ERR_INVALID_ARG;
  if (d->B == 0 && d->T > 0) return MOE_ERR_INVALID_ARG;
  if (d->D != moe::kHeadDim || d->Hq > 1024) return MOE_ERR_UNSUPPORTED;
  if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128) return MOE_ERR_UNSUPPORTED;
  if (d->B > 65536) return MOE_ERR_UNSUPPORTED;
  if ((long long)d->max_pages * d->page >= kMaxLen || (long long)d->n_pages * d->Hkv * d->page >= kMaxRows ||
      (long long)d->T * d->Hq >= kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::KvBatch make_batch(const moe_kv_desc* d, const moe_kv_cache* kv, const int32_t* page_table, unsigned* status) {
  moe::KvBatch c = {};
  c.B = d->B;
  c.T = d->T;
  c.Hq = d->Hq;
  c.Hkv = d->Hkv;
  c.page = d->page;
  while ((1 << c.page_log2) < d->page) ++c.page_log2;
  c.n_pages = d->n_pages;
  c.max_pages = d->max_pages;
  c.page_table = page_table;
  c.k_codes = kv->k_codes;
  c.v_codes = kv->v_codes;
  c.k_scale = kv->k_scale;
  c.v_scale = kv->v_scale;
  c.status = status;
  return c;
}

int check_cache(const moe_kv_cache* kv) {
  if (!kv || !ok_ptr(kv->k_codes) || !ok_ptr(kv->v_codes) || !kv->k_scale || !kv->v_scale)
    return MOE_ERR_INVALID_ARG;
  if (kv->k_codes == kv->v_codes || kv->k_scale == kv->v_scale) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ok_ptr(ws)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

bool ok_stride(long long stride, int heads) { return stride >= (long long)heads * moe::kHeadDim && stride % 8 == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

int moe_rope_table(int max_pos, int rot_dim, double base, float* cos_sin, void* stream) {
  if (max_pos < 0 || rot_dim < 1 || !(base > 0) || !isfinite(base)) return MOE_ERR_INVALID_ARG;
  if (rot_dim > moe::kHeadDim || rot_dim % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (max_pos == 0) return MOE_OK;
  if (!ok_ptr(cos_sin)) return MOE_ERR_INVALID_ARG;
  return cuda_status(moe::launch_rope_table(max_pos, rot_dim, base, cos_sin, (cudaStream_t)stream));
}

int moe_kv_append(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                  const uint16_t* v, long long v_stride, const int32_t* q_start, const int32_t* kv_len,
                  const int32_t* page_table, const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                  const uint16_t* q_norm_weight, const uint16_t* k_norm_weight, float eps, uint16_t* q_out,
                  const moe_kv_cache* kv, void* ws, size_t ws_bytes, void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (max_pos < 0 || rot_dim < 0 || !(eps >= 0)) return MOE_ERR_INVALID_ARG;
  if (rot_dim > d->D || rot_dim % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (d->T == 0) return MOE_OK;
  if (!ok_ptr(k) || !ok_ptr(v) || !ok_ptr(q_start) || !ok_ptr(kv_len) || !ok_ptr(page_table)) return MOE_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || !aligned16(q) || !aligned16(q_out)) return MOE_ERR_INVALID_ARG;
  if (rot_dim > 0 && !ok_ptr(cos_sin)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q_norm_weight) || !aligned16(k_norm_weight) || (!q && q_norm_weight)) return MOE_ERR_INVALID_ARG;
  if ((q && !ok_stride(q_stride, d->Hq)) || !ok_stride(k_stride, d->Hkv) || !ok_stride(v_stride, d->Hkv))
    return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, kHeader))) return s;
  moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws);
  c.q_start = q_start;
  c.kv_len = kv_len;
  moe::KvAppendArgs a = {q, k, v, q_stride, k_stride, v_stride, cos_sin, rot_dim > 0 ? max_pos : INT32_MAX, rot_dim,
                         interleaved != 0, q_norm_weight, k_norm_weight, eps, q_out};
  return cuda_status(moe::launch_kv_append(c, a, sm_count(), (cudaStream_t)stream));
}

int moe_kv_gather(const moe_kv_desc* d, const int32_t* start, const int32_t* out_start, const int32_t* page_table,
                  const moe_kv_cache* kv, int n_rows, uint16_t* k, uint16_t* v, void* ws, size_t ws_bytes,
                  void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (n_rows < 0 || (d->B == 0 && n_rows > 0)) return MOE_ERR_INVALID_ARG;
  if ((long long)n_rows * d->Hkv * d->D >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (n_rows == 0) return MOE_OK;
  if (!ok_ptr(start) || !ok_ptr(out_start) || !ok_ptr(page_table) || !ok_ptr(k) || !ok_ptr(v)) return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, kHeader))) return s;
  const moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws);
  return cuda_status(moe::launch_kv_gather(c, start, out_start, n_rows, k, v, (cudaStream_t)stream));
}

size_t moe_paged_attention_workspace_size(const moe_kv_desc* d, int max_q) {
  if (check_desc(d) || max_q < 0) return 0;
  return kHeader + moe::attention_scratch_bytes(d->Hq, d->Hkv, max_q, sm_count());
}

int moe_paged_attention(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* page_table, const moe_kv_cache* kv, int max_q,
                        float scale, int causal, int window, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (max_q < 0 || window < 0 || !(scale > 0) || !isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (window > 0 && !causal) return MOE_ERR_INVALID_ARG;
  if (d->T == 0) return MOE_OK;
  if (max_q < 1 || max_q > d->T || (long long)max_q * d->B < d->T) return MOE_ERR_INVALID_ARG;
  if (!ok_ptr(q) || !ok_ptr(q_start) || !ok_ptr(kv_len) || !ok_ptr(page_table) || !ok_ptr(out)) return MOE_ERR_INVALID_ARG;
  if (!ok_stride(q_stride, d->Hq)) return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, moe_paged_attention_workspace_size(d, max_q)))) return s;
  moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws);
  c.q_start = q_start;
  c.kv_len = kv_len;
  moe::AttentionArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.causal = causal != 0;
  a.window = window;
  a.max_q = max_q;
  a.scratch = (char*)ws + kHeader;
  return cuda_status(moe::launch_paged_attention(c, a, sm_count(), (cudaStream_t)stream));
}

}  // extern "C"
