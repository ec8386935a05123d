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

int moe_rope_rows(int n_axes, int T, const int32_t* positions, long long positions_stride, const uint8_t* axes, const float* cos_sin,
                  int max_pos, int rot_dim, float* rows, void* ws, size_t ws_bytes, void* stream) {
  if (n_axes < 1 || T < 0 || max_pos < 0 || rot_dim < 1 || positions_stride < 0) return MOE_ERR_INVALID_ARG;
  if (n_axes > moe::kMaxAxes || rot_dim > moe::kHeadDim || rot_dim % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (!axes) return MOE_ERR_INVALID_ARG;
  moe::RopeAxes x = {};
  for (int f = 0; f < rot_dim / 2; ++f) {
    if (axes[f] >= n_axes) return MOE_ERR_INVALID_ARG;
    x.axis[f] = axes[f];
  }
  if (T == 0) return MOE_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u) || !ok_ptr(cos_sin) || !ok_ptr(rows)) return MOE_ERR_INVALID_ARG;
  const int s = check_ws(ws, ws_bytes, kHeader);
  if (s) return s;
  return cuda_status(moe::launch_rope_rows(x, T, positions, positions_stride, cos_sin, max_pos, rot_dim, rows, (unsigned*)ws,
                                           (cudaStream_t)stream));
}

static int kv_append(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                     const uint16_t* v, long long v_stride, const int32_t* q_start, const int32_t* kv_len,
                     const int32_t* page_table, const float* cos_sin, int max_pos, bool by_token, int rot_dim, int interleaved,
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
  moe::KvAppendArgs a = {q, k, v, q_stride, k_stride, v_stride, cos_sin, rot_dim > 0 && !by_token ? max_pos : INT32_MAX, rot_dim,
                         interleaved != 0, by_token, q_norm_weight, k_norm_weight, eps, q_out};
  return cuda_status(moe::launch_kv_append(c, a, sm_count(), (cudaStream_t)stream));
}

int moe_kv_append(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                  const uint16_t* v, long long v_stride, const int32_t* q_start, const int32_t* kv_len,
                  const int32_t* page_table, const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                  const uint16_t* q_norm_weight, const uint16_t* k_norm_weight, float eps, uint16_t* q_out,
                  const moe_kv_cache* kv, void* ws, size_t ws_bytes, void* stream) {
  return kv_append(d, q, q_stride, k, k_stride, v, v_stride, q_start, kv_len, page_table, cos_sin, max_pos, false, rot_dim, interleaved,
                   q_norm_weight, k_norm_weight, eps, q_out, kv, ws, ws_bytes, stream);
}

int moe_kv_append_at(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                     const uint16_t* v, long long v_stride, const int32_t* q_start, const int32_t* kv_len,
                     const int32_t* page_table, const float* rows, int rot_dim, int interleaved, const uint16_t* q_norm_weight,
                     const uint16_t* k_norm_weight, float eps, uint16_t* q_out, const moe_kv_cache* kv, void* ws, size_t ws_bytes,
                     void* stream) {
  return kv_append(d, q, q_stride, k, k_stride, v, v_stride, q_start, kv_len, page_table, rows, 0, true, rot_dim, interleaved,
                   q_norm_weight, k_norm_weight, eps, q_out, kv, ws, ws_bytes, stream);
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

static int check_attention(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const int32_t* q_start, const int32_t* kv_len,
                           const int32_t* page_table, int max_q, bool table_needed = true) {
  if (max_q < 1 || max_q > d->T || (long long)max_q * d->B < d->T) return MOE_ERR_INVALID_ARG;
  if (!ok_ptr(q) || !ok_ptr(q_start) || !ok_ptr(kv_len) || !aligned16(page_table)) return MOE_ERR_INVALID_ARG;
  if (!page_table && table_needed) return MOE_ERR_INVALID_ARG;
  return ok_stride(q_stride, d->Hq) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// The prefixes of a shared attention as a batch of their own: its sequences are the prefixes, its tokens their readers'.
static int prefix_desc(const moe_kv_desc* d, const moe_kv_prefix* p, moe_kv_desc* out) {
  if (p->n < 1 || p->max_pages < 0 || p->max_q < 0) return MOE_ERR_INVALID_ARG;
  *out = *d;
  out->B = p->n;
  out->max_pages = p->max_pages;
  return check_desc(out);
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// (no more than the sizes: neither pointers nor lengths)
static bool shared_joins(const moe_kv_desc* d, const moe_kv_desc* pd, int max_q) {
  const moe_kv_cache none = {};
  return moe::shared_attention_joins(make_batch(pd, &none, nullptr, nullptr), make_batch(d, &none, nullptr, nullptr), max_q);
}

size_t moe_paged_attention_shared_workspace_size(const moe_kv_desc* d, int max_q, const moe_kv_prefix* prefix) {
  if (check_desc(d) || max_q < 0) return 0;
  const size_t scratch = moe::attention_scratch_bytes(d->Hq, d->Hkv, max_q, sm_count());
  if (!prefix) return kHeader + scratch;
  moe_kv_desc pd;
  if (prefix_desc(d, prefix, &pd)) return 0;
  if (shared_joins(d, &pd, max_q)) return kHeader + scratch;
  const size_t rows = (size_t)d->T * d->Hq;
  return kHeader + 2 * (up256(rows * moe::kHeadDim * sizeof(float)) + up256(rows * sizeof(float))) +
         up256(moe::attention_scratch_bytes(d->Hq, d->Hkv, prefix->max_q, sm_count())) + scratch;
}

int moe_paged_attention_shared(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const int32_t* q_start,
                               const int32_t* kv_len, const int32_t* page_table, const moe_kv_cache* kv, int max_q, float scale,
                               int causal, int window, const moe_kv_prefix* prefix, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (max_q < 0 || window < 0 || !(scale > 0) || !isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (window > 0 && (!causal || prefix)) return MOE_ERR_INVALID_ARG;
  moe_kv_desc pd = {};
  if (prefix && (s = prefix_desc(d, prefix, &pd))) return s;
  if (d->T == 0) return MOE_OK;
  if ((s = check_attention(d, q, q_stride, q_start, kv_len, page_table, max_q))) return s;
  // (a table without columns is not read: its prefixes have no tokens)
  if (prefix && (s = check_attention(&pd, q, q_stride, prefix->q_start, prefix->len, prefix->page_table, prefix->max_q, prefix->max_pages > 0)))
    return s;
  if (!ok_ptr(out) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, moe_paged_attention_shared_workspace_size(d, max_q, prefix)))) return s;
  moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws), pc = {};
  c.q_start = q_start;
  c.kv_len = kv_len;
  char* at = (char*)ws + kHeader;
  moe::SharedBuffers buffers = {};
  if (prefix) {
    pc = make_batch(&pd, kv, prefix->page_table, (unsigned*)ws);
    pc.q_start = prefix->q_start;
    pc.kv_len = prefix->len;
  }
  if (prefix && !shared_joins(d, &pd, max_q)) {
    for (int i = 0; i < 2; ++i) {
      buffers.rows[i] = (float*)at;
      at += up256((size_t)d->T * d->Hq * moe::kHeadDim * sizeof(float));
      buffers.lse[i] = (float*)at;
      at += up256((size_t)d->T * d->Hq * sizeof(float));
    }
    buffers.prefix_scratch = at;
    at += up256(moe::attention_scratch_bytes(d->Hq, d->Hkv, prefix->max_q, sm_count()));
  }
  moe::AttentionArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.causal = causal != 0;
  a.window = window;
  a.max_q = max_q;
  a.scratch = at;
  a.lse = lse;
  a.lse_unit = 0.693147180559945309f;
  return cuda_status(moe::launch_shared_attention(pc, prefix ? prefix->max_q : 0, c, a, buffers, sm_count(), (cudaStream_t)stream));
}

int moe_kv_weights(const moe_kv_desc* d, const uint16_t* q, long long q_stride, const float* lse, const int32_t* q_start,
                   const int32_t* kv_len, const int32_t* page_table, const moe_kv_cache* kv, int max_q, float scale, int causal,
                   int window, const float* weight_in, float* weight_out, void* ws, size_t ws_bytes, void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (max_q < 0 || window < 0 || !(scale > 0) || !isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (window > 0 && !causal) return MOE_ERR_INVALID_ARG;
  if (d->T == 0) return MOE_OK;
  if ((s = check_attention(d, q, q_stride, q_start, kv_len, page_table, max_q))) return s;
  if (!ok_ptr(lse) || !aligned16(weight_in) || !ok_ptr(weight_out)) return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, kHeader))) return s;
  moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws);
  c.q_start = q_start;
  c.kv_len = kv_len;
  moe::AttentionArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.causal = causal != 0;
  a.window = window;
  a.max_q = max_q;
  return cuda_status(moe::launch_kv_weights(c, a, lse, weight_in, weight_out, sm_count(), (cudaStream_t)stream));
}

int moe_kv_evict(const moe_kv_desc* d, float* weight, const int32_t* kv_len, const int32_t* page_table, const int32_t* keep, int sink,
                 int recent, const int32_t* new_table, int new_max_pages, const moe_kv_cache* kv, int32_t* new_len, int32_t* kept,
                 void* ws, size_t ws_bytes, void* stream) {
  int s = check_desc(d);
  if (s) return s;
  if (sink < 0 || recent < 0 || new_max_pages < 1) return MOE_ERR_INVALID_ARG;
  if ((long long)new_max_pages * d->page > (1LL << 30) || (long long)d->B * d->Hkv * new_max_pages >= kMaxRows ||
      (long long)d->B * d->Hkv * 8 >= kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  if (d->B == 0) return MOE_OK;
  if (!ok_ptr(weight) || !ok_ptr(kv_len) || !ok_ptr(page_table) || !ok_ptr(keep) || !ok_ptr(new_table) || !ok_ptr(new_len) || !ok_ptr(kept))
    return MOE_ERR_INVALID_ARG;
  if ((s = check_cache(kv))) return s;
  if ((s = check_ws(ws, ws_bytes, kHeader))) return s;
  moe::KvBatch c = make_batch(d, kv, page_table, (unsigned*)ws);
  c.kv_len = kv_len;
  const moe::KvEvictArgs e = {weight, keep, sink, recent, new_table, new_max_pages, new_len, kept};
  return cuda_status(moe::launch_kv_evict(c, e, sm_count(), (cudaStream_t)stream));
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
