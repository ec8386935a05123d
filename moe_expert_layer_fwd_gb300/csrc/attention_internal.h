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
  const float* cos_sin;       // [max_pos, rot]: cosines, then sines
  int max_pos, rot, interleaved;
  const uint16_t* q_norm;     // [128] bf16 or NULL
  const uint16_t* k_norm;
  float eps;
  uint16_t* q_out;            // [T, Hq, 128]
};
cudaError_t launch_kv_append(const KvBatch& c, const KvAppendArgs& a, int n_sms, cudaStream_t stream);

// Rows [0, n_rows): row r of sequence b (out_start[b] <= r < out_start[b+1]) is token start[b] + r - out_start[b].
cudaError_t launch_kv_gather(const KvBatch& c, const int32_t* start, const int32_t* out_start, int n_rows, uint16_t* k,
                             uint16_t* v, cudaStream_t stream);

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
};
size_t attention_scratch_bytes(int Hq, int Hkv, int max_q, int n_sms);
cudaError_t launch_paged_attention(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream);


// Failure injection (tests only): what 1 = wait limit in ns (0: the default 2 s), what 4 = nonzero: withhold the values'
// copies.  Returns 0, or -1 for another `what`.
int attention_debug_set(int what, unsigned long long value);

// Few query rows per key/value head: G grouped heads times max_q new tokens at most 16.
bool attention_decode_fits(int G, int max_q);
size_t attention_decode_scratch(int G, int max_q, int n_sms);
cudaError_t launch_attention_decode(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream);

// Any number of rows.
size_t attention_prefill_scratch(int G, int max_q, int n_sms);
cudaError_t launch_attention_prefill(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream);

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
// part_o [parts][rows][128], part_rl [parts][rows]: unscaled sums, their reference exponent r and denominator l.
cudaError_t launch_attention_join(const KvBatch& c, const AttentionArgs& a, int blocks, int rows, const float* part_o,
                                  const float2* part_rl, const JoinInfo* info, cudaStream_t stream);

// The codes as a matrix of 128-byte rows (one token of one head each), boxes of one page with the 128-byte swizzle.
bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const KvBatch& c);

}  // namespace moe
