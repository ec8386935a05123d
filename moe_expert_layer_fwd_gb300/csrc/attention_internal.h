// Launchers and shared arguments of the attention operators (paged 8-bit key/value cache).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kHeadDim = 128;      // elements per head: one code row is 128 bytes
constexpr int kMinScaleExp = -64;  // smallest exponent of a page's scale

// The batch and its cache, as the entry points give them.
struct KvBatch {
  int B, T, Hq, Hkv, page, page_log2, n_pages, max_pages;
  const int32_t* q_start;     // [B+1] first new token of each sequence
  const int32_t* kv_len;      // [B] tokens of each sequence, the new ones included
  const int32_t* page_table;  // [B, max_pages]
  uint8_t* k_codes;           // [n_pages, Hkv, page, 128] E4M3
  uint8_t* v_codes;
  uint8_t* k_scale;           // [n_pages, Hkv] E8M0
  uint8_t* v_scale;
  unsigned* status;
};

struct KvAppendArgs {
  const uint16_t* q;          // [T, Hq, 128] bf16, token stride q_stride (elements); NULL: keys and values only
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  const float* cos_sin;       // [max_pos, rot]: cosines, then sines; or [T, rot], a row for each new token
  int max_pos, rot, interleaved, by_token;
  const uint16_t* q_norm;     // [128] bf16 or NULL
  const uint16_t* k_norm;
  float eps;
  uint16_t* q_out;            // [T, Hq, 128]
};
cudaError_t launch_kv_append(const KvBatch& c, const KvAppendArgs& a, int n_sms, cudaStream_t stream);

// Rows [0, n_rows): row r of sequence b (out_start[b] <= r < out_start[b+1]) is token start[b] + r - out_start[b].
cudaError_t launch_kv_gather(const KvBatch& c, const int32_t* start, const int32_t* out_start, int n_rows, uint16_t* k,
                             uint16_t* v, cudaStream_t stream);

// rows [T, rot]: of token t and frequency f the cosine and sine at position positions[axis[f] * stride + t].
constexpr int kMaxAxes = 8;
struct RopeAxes {
  uint8_t axis[kHeadDim / 2];
};
cudaError_t launch_rope_rows(const RopeAxes& axes, int T, const int32_t* positions, long long stride, const float* cos_sin,
                             int max_pos, int rot, float* rows, unsigned* status, cudaStream_t stream);

cudaError_t launch_rope_table(int max_pos, int rot, double base, float* cos_sin, cudaStream_t stream);

struct AttentionArgs {
  const uint16_t* q;          // [T, Hq, 128] bf16, token stride q_stride
  long long q_stride;
  uint16_t* out;              // [T, Hq, 128]
  float scale_log2;           // softmax scale * log2(e)
  int causal, window, max_q;
  unsigned limit_us;          // of every wait inside the kernels
  int withhold;               // failure injection (tests only): the values' copies are not issued, so that waits run out
  void* scratch;              // after the status word of the workspace
  // What a call is.  0: one of its own, with rows only.  1: one of two passes over different keys, whose rows (out32) and denominators (lse)
  // another kernel puts together; rows that are split over blocks are marked in lse and stay parts.  2: one of its own, with lse.
  // 3: both passes in one, each row over its prefix's keys and then its own; with lse.
  int pass;
  int follows;                // pass 1: may start while the kernel before it ends
  union {
    float* out32;             // pass 1: [T, Hq, 128] fp32, instead of out
    struct {                  // pass 3: as KvBatch's q_start, kv_len and page_table
      const int32_t* prefix_start;
      const int32_t* prefix_len;
      const int32_t* prefix_table;
    };
  };
  float* lse;                 // [T, Hq] or NULL: lse_unit times the logarithm (base 2) of the rows' denominators (-inf: nothing seen)
  float lse_unit;
  int n_prefixes, prefix_max_pages;  // pass 3
};
size_t attention_scratch_bytes(int Hq, int Hkv, int max_q, int n_sms);
// parts (pass 1): where the rows are that were split.
struct AttentionParts;
cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream, AttentionParts* parts = nullptr);

// Whether sequences (of at most max_q new tokens) bring so many rows that each goes over its prefix by itself, in one pass.
bool shared_attention_joins(const KvBatch& prefixes, const KvBatch& c, int max_q);
// What the two passes leave for the kernel that ends them: rows [T, Hq, 128], denominators [T, Hq], and the scratch of either (the
// second's is the call's).
struct SharedBuffers {
  float* rows[2];
  float* lse[2];
  void* prefix_scratch;
};
// Sequences b of `prefixes` are the prefixes, its q_start cuts the T tokens into their readers (B = 0: no prefixes).
cudaError_t launch_shared_attention(const KvBatch& prefixes, int max_prefix_q, const KvBatch& c, const AttentionArgs& a,
                                    const SharedBuffers& s, int n_sms, cudaStream_t stream);


// Failure injection (tests only): what 1 = wait limit in ns (0: the default 2 s), what 4 = nonzero: withhold the values'
// copies.  Returns 0, or -1 for another `what`.
int attention_debug_set(int what, unsigned long long value);

// weight_out [n_pages, Hkv, page]: for each cached token that a query of a sees, and each new one, weight_in (0 for new ones; NULL: 0)
// plus the weights that the queries give it; lse [T, Hq] their denominators' natural logarithms.
cudaError_t launch_kv_weights(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                              int n_sms, cudaStream_t stream);
cudaError_t launch_kv_weights_rows(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                                   int n_sms, cudaStream_t stream);

struct KvEvictArgs {
  float* weight;             // [n_pages, Hkv, page]
  const int32_t* keep;       // [B] tokens that stay
  int sink, recent;          // first and last tokens that stay before all others
  const int32_t* new_table;  // [B, new_max_pages]
  int new_max_pages;
  int32_t* new_len;          // [B]
  int32_t* kept;             // [B, Hkv, new_max_pages * page]
};
cudaError_t launch_kv_evict(const KvBatch& c, const KvEvictArgs& e, int n_sms, cudaStream_t stream);

// Few query rows per key/value head: G grouped heads times max_q new tokens at most 16.
bool attention_decode_fits(int G, int max_q);
bool attention_decode_chunks_fit(const KvBatch& c, int max_q, int n_sms);  // or 16 of them at a time (calls of two passes)
size_t attention_decode_scratch(int G, int max_q, int n_sms);
cudaError_t launch_attention_decode(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream, AttentionParts* parts);

// Any number of rows.
size_t attention_prefill_scratch(int G, int max_q, int n_sms);
cudaError_t launch_attention_prefill(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream, AttentionParts* parts);

// ---------------------------------------------------------------- rows that were split
// What block k of a kernel that cuts its work into runs tells the joining kernel: whether its run begins with a part of
// an item (some rows of one sequence and head) that is not the item's first.  Blocks c0 .. c1 have the item's parts, block
// k's part is number 2k, but c0's is 2 c0 + slot0 (a run's second kind of part: an item that it does not begin with).
struct JoinInfo {
  int split;
  int b, h, row0;     // rows row0 .. of the sequence's new tokens x grouped heads
  int c0, c1, slot0;
  int pad;
};
// The parts of a launch of `blocks` blocks: o [2 blocks][rows][128], rl [2 blocks][rows]: unscaled sums, their reference exponent r and
// denominator l; the sums are of 2^(u - r + base).
struct AttentionParts {
  int blocks, rows;
  float base;
  const float* o;
  const float2* rl;
  const JoinInfo* info;  // [blocks]
};
cudaError_t launch_attention_join(const KvBatch& c, const AttentionArgs& a, const AttentionParts& parts, cudaStream_t stream);

// What a pass 1 puts in place of the denominator of a row that is split: a NaN that no arithmetic makes, with the number of the block that
// has the row's first part.
constexpr unsigned kSplitMark = 0xFFC00000u;

// The codes as a matrix of 128-byte rows (one token of one head each), boxes of one page with the 128-byte swizzle.
bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const KvBatch& c);

// The queries [T][Hq][128], boxes of `tokens` times `heads` rows of 64 dims with the 128-byte swizzle.
bool make_query_map(CUtensorMap* m, const AttentionArgs& a, const KvBatch& c, int heads, int tokens);

}  // namespace moe
