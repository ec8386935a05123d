// The paged 8-bit key/value cache: appending with normalisation and rotation, reading back, the rotation table.
//
// Sources: Hy3 295B MoE practice, section 1.1 (per-head RMS norm of queries and keys before the rotation, grouped query
// heads) and 4 (new keys and values scattered into the cache by slot); the inference note's KV paging section (pages
// of a fixed number of tokens, a page table per sequence).  The 8-bit format is this library's own choice: E4M3 codes
// and one E8M0 scale per (page, head), the element and scale types of its MXFP8 token rows.
//
// Append, for a new token at position p of its sequence (both halves of a pair (a, b) come from one head):
//   x^   = x * rsqrt(mean(x^2) + eps) * w              (queries and keys, when norm weights are given)
//   a'   = a cos(p f_i) - b sin(p f_i),  b' = a sin(p f_i) + b cos(p f_i)        (the first `rot` elements)
//   e    = max(-64, ceil(log2(amax / 448)), the page's exponent if it holds earlier tokens of the sequence)
//   code = e4m3(x' * 2^-e)
// with amax over the page's new tokens of one head.  A power of two costs an E4M3 value nothing but range: relative
// precision is the same at every scale, and when e grows the earlier codes are rescaled exactly unless they become
// subnormal.  Everything between the bf16 input and the one rounding of the output is fp32.
#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kWarps = kAppendThreads / 32;
constexpr int kSteps = 4;          // rows of keys (and of values) that a half-warp has in flight: 16 lanes x 8 elements each
constexpr int kQBlocksPerSm = 5;   // blocks that rotate queries
constexpr int kQHeads = 16;        // query heads of one token that a warp rotates, two at a time

// A row in registers: lane l of a half-warp holds elements 8l .. 8l+7.
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

// What a lane needs of the rotation, the same for every row of a token.
struct Rotary {
  float cs[8], sn[8];  // half-split: of elements 8 (l mod rot/16) + i, the sine negated in the lower half;
                       // interleaved: of pairs 4l + (i / 2)
  int partner;         // lane holding the other halves of the pairs (half-split)
  bool on, upper;
};

__device__ __forceinline__ void rotary_lane(Rotary& r, const KvAppendArgs& a, int l) {
  const int half = a.rot >> 4;  // lanes of one half of the rotated part
  r.on = l < 2 * half;
  r.upper = !a.interleaved && l >= half;
  r.partner = !r.on || a.interleaved ? l : (r.upper ? l - half : l + half);
}

__device__ __forceinline__ void rotary_load(Rotary& r, const KvAppendArgs& a, int l, int pos) {
  if (!r.on) return;
  const float* row = a.cos_sin + (size_t)pos * a.rot;
  if (a.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + (a.rot >> 1) + 4 * l));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.cs[i] = cc[i >> 1];
      r.sn[i] = ss[i >> 1];
    }
  } else {
    const float* p = row + 8 * (r.upper ? l - (a.rot >> 4) : l);
    const float* q = p + (a.rot >> 1);
    const float sign = r.upper ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(p + i));
      const float4 s = __ldg(reinterpret_cast<const float4*>(q + i));
      r.cs[i] = c.x; r.cs[i + 1] = c.y; r.cs[i + 2] = c.z; r.cs[i + 3] = c.w;
      r.sn[i] = sign * s.x; r.sn[i + 1] = sign * s.y; r.sn[i + 2] = sign * s.z; r.sn[i + 3] = sign * s.w;
    }
  }
}

// Pairs of floats in one 64-bit register: one instruction for two products or sums, each rounded by itself.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}

// Normalises (w: the norm weights of this lane's elements) and rotates one row.  Products and sums are rounded one by one
// (no fused multiply-add), so that the result does not depend on which of a pair's two products is fused.  The
// queries' part is bound by these instructions (scalar, with both halves of a pair normalised by either lane, 173 of them for two
// rows: 152 us for 16384 tokens where 127 us are needed so).
__device__ __forceinline__ void norm_rotate(const uint4& raw, const Rotary& r, const KvAppendArgs& a, bool norm,
                                            const float (&w)[8], float (&x)[8]) {
  unpack8(raw, x);
  if (norm) {
    uint64_t sq = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) sq = fma2(pair(x[i], x[i + 1]), pair(x[i], x[i + 1]), sq);
    float ss, s1;
    unpair(sq, ss, s1);
    ss += s1;
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, 16);
    const float rs = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; i += 2) unpair(mul2(mul2(pair(x[i], x[i + 1]), pair(rs, rs)), pair(w[i], w[i + 1])), x[i], x[i + 1]);
  }
  if (a.interleaved) {
    if (!r.on) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float p = x[i], q = x[i + 1];
      x[i] = __fsub_rn(__fmul_rn(p, r.cs[i]), __fmul_rn(q, r.sn[i]));
      x[i + 1] = __fadd_rn(__fmul_rn(p, r.sn[i]), __fmul_rn(q, r.cs[i]));
    }
  } else if (a.rot > 0) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], r.partner, 16);
    if (!r.on) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      unpair(add2(mul2(pair(x[i], x[i + 1]), pair(r.cs[i], r.cs[i + 1])), mul2(pair(y[i], y[i + 1]), pair(r.sn[i], r.sn[i + 1]))),
             x[i], x[i + 1]);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// This lane's norm weights (ones when there are none).
__device__ __forceinline__ void load_weights(const uint16_t* weight, int l, float (&w)[8]) {
  uint4 v = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  if (weight) v = __ldg(reinterpret_cast<const uint4*>(weight) + l);
  unpack8(v, w);
}

// The smallest exponent >= -64 with amax * 2^-e <= 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExp);
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
  uint2 o;
  o.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
  o.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return o;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // infinities and NaN do not set the scale
}

// Queries: a warp takes (token, 16 heads) items in turn, the next one's rows on their way to shared memory while it works on
// the present one's (a lane reads back only what it fetched itself).
constexpr int kQPieces = kQHeads / 2;                                   // of 16 bytes a lane, per item
constexpr int kQShared = 2 * kWarps * kQPieces * 32 * (int)sizeof(uint4);  // 32 KB
__device__ __forceinline__ void rope_queries(const KvBatch& c, const KvAppendArgs& a, int block, int blocks, uint4* shared) {
  uint4(*s_rows)[kWarps][kQPieces][32] = reinterpret_cast<uint4(*)[kWarps][kQPieces][32]>(shared);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
  Rotary rt;
  rotary_lane(rt, a, l);
  float weight[8];
  load_weights(a.q_norm, l, weight);
  const int chunks = (c.Hq + kQHeads - 1) / kQHeads;
  const long long items = (long long)c.T * chunks, stride = (long long)blocks * kWarps;
  auto fetch = [&](long long w, int stage) {
    if (w < items) {
      const int t = (int)(w / chunks), h = (int)(w - (long long)t * chunks) * kQHeads + half;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)t * a.q_stride + (size_t)h * kHeadDim) + l;
#pragma unroll
      for (int i = 0; i < kQPieces; ++i)
        if (h + 2 * i < c.Hq) cp_async16(smem_u32(&s_rows[stage][warp][i][lane]), src + 2 * i * (kHeadDim / 8), 16);
    }
    cp_async_commit();
  };
  long long w = (long long)block * kWarps + warp;
  fetch(w, 0);
  int stage = 0;
#pragma unroll 1
  for (; w < items; w += stride, stage ^= 1) {
    fetch(w + stride, stage ^ 1);
    const int t = (int)(w / chunks), h0 = (int)(w - (long long)t * chunks) * kQHeads + half;
    const int b = warp_search(c.B, t, [&](int i) { return __ldg(c.q_start + i); });
    SeqRange s;
    const bool ok = load_seq(c, b, s) && t >= s.t0 && t < s.t1;
    const int pos = ok ? s.first() + t - s.t0 : -1;
    const bool there = pos >= 0 && pos < a.max_pos;
    if (!there && lane == 0) set_status(c.status, DEV_ERR_BOUNDS);
    if (there) rotary_load(rt, a, l, a.by_token ? t : pos);
    cp_async_wait<1>();
    if (!there) continue;
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) {
      float x[8];
      norm_rotate(s_rows[stage][warp][i][lane], rt, a, a.q_norm != nullptr, weight, x);
      const int h = h0 + 2 * i;
      if (h < c.Hq) {
        const uint4 o = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        reinterpret_cast<uint4*>(a.q_out + ((size_t)t * c.Hq + h) * kHeadDim)[l] = o;
      }
    }
  }
  cp_async_wait<0>();
}

// Keys and values: a block per unit, one touched page of one sequence and one head.  Sequence b's touched pages take the
// slots from q_start[b] / page + 2b on: n new tokens touch at most (n - 1) / page + 2 pages, so the slots of different
// sequences never meet and T / page + 2B of them are enough.  Every unit is found from the lengths on the device: the host
// never needs them.  The rotated keys wait in shared memory for their scale; the values are read a second time (from L1 or L2).
__device__ __forceinline__ void append_unit(const KvBatch& c, const KvAppendArgs& a, int unit_block, float (*s_amax)[kWarps],
                                            float4* s_k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
  Rotary rt;
  rotary_lane(rt, a, l);
  const int slot = unit_block / c.Hkv, h = unit_block - slot * c.Hkv;
  const int b = warp_search(c.B, slot, [&](int i) { return (__ldg(c.q_start + i) >> c.page_log2) + 2 * i; });
  SeqRange s;
  if (!load_seq(c, b, s) || s.t1 == s.t0) return;
  const int first = s.first(), j = (first >> c.page_log2) + slot - ((s.t0 >> c.page_log2) + 2 * b);
  const int end = min(s.len, a.max_pos);  // tokens at positions that the table does not have are left out, as their queries are
  if ((first < 0 || s.len > end) && threadIdx.x == 0) set_status(c.status, first < 0 ? DEV_ERR_CONFIG : DEV_ERR_BOUNDS);
  if (first < 0 || first >= end || j < (first >> c.page_log2) || j > ((end - 1) >> c.page_log2)) return;
  const int pg = load_page(c, b, j);
  if (pg < 0) return;
  const size_t unit = (size_t)pg * c.Hkv + h;
  const int p0 = j << c.page_log2;                                 // position of the page's first token
  const int r0 = max(0, first - p0), r1 = min(c.page, end - p0);    // its new rows
  int old_k = kMinScaleExp, old_v = kMinScaleExp;
  if (r0 > 0) {
    old_k = min((int)c.k_scale[unit] - 127, 126);
    old_v = min((int)c.v_scale[unit] - 127, 126);
  }
  const uint16_t* k_rows = a.k + (size_t)h * kHeadDim + 8 * l;
  const uint16_t* v_rows = a.v + (size_t)h * kHeadDim + 8 * l;
  float weight[8];
  load_weights(a.k_norm, l, weight);
  const bool norm = a.k_norm != nullptr;

  // the first step that has new rows; whole warps, as the shuffles below need both halves
  const int base0 = r0 / (2 * kWarps) * 2 * kWarps + warp * 2;
  float amax_k = 0.f, amax_v = 0.f;
#pragma unroll 1
  for (int base = base0; base < r1; base += kSteps * 2 * kWarps) {
    uint4 kr[kSteps], vr[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = base + half + i * 2 * kWarps;
      kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
      if (r >= r0 && r < r1) {
        const size_t t = (size_t)(s.t0 + p0 + r - first);
        kr[i] = __ldg(reinterpret_cast<const uint4*>(k_rows + t * a.k_stride));
        vr[i] = __ldg(reinterpret_cast<const uint4*>(v_rows + t * a.v_stride));
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (base + i * 2 * kWarps >= r1) break;
      const int r = base + half + i * 2 * kWarps;
      const bool here = r >= r0 && r < r1;
      if (here) rotary_load(rt, a, l, a.by_token ? s.t0 + p0 + r - first : p0 + r);
      float x[8], v[8];
      norm_rotate(kr[i], rt, a, norm, weight, x);
      unpack8(vr[i], v);
      // A NaN in a token's value is kept in its key instead, as a NaN key row: the queries that see the token become
      // NaN through their score, and those that do not are untouched (0 * NaN in the product with V would reach them).
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bad |= v[e] != v[e] || x[e] != x[e];
        amax_k = fmaxf(amax_k, finite_abs(x[e]));
        amax_v = fmaxf(amax_v, finite_abs(v[e]));
      }
      if (__ballot_sync(0xffffffffu, bad) >> (16 * half) & 0xFFFFu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __int_as_float(0x7FFFFFFF);
      }
      if (here) {
        s_k[(r * 2) * 16 + l] = make_float4(x[0], x[1], x[2], x[3]);
        s_k[(r * 2 + 1) * 16 + l] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    amax_k = fmaxf(amax_k, __shfl_xor_sync(0xffffffffu, amax_k, o));
    amax_v = fmaxf(amax_v, __shfl_xor_sync(0xffffffffu, amax_v, o));
  }
  if (lane == 0) {
    s_amax[0][warp] = amax_k;
    s_amax[1][warp] = amax_v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    amax_k = fmaxf(amax_k, s_amax[0][i]);
    amax_v = fmaxf(amax_v, s_amax[1][i]);
  }
  const int ek = max(scale_exponent(amax_k), old_k), ev = max(scale_exponent(amax_v), old_v);
  if (threadIdx.x == 0) {
    c.k_scale[unit] = (uint8_t)(ek + 127);
    c.v_scale[unit] = (uint8_t)(ev + 127);
  }
  const float inv_k = exp2_int(-ek), inv_v = exp2_int(-ev);
  // new tokens: each half-warp its own rows again
#pragma unroll 4
  for (int r = base0 + half; r < r1; r += 2 * kWarps) {
    if (r < r0) continue;
    const uint4 vr = __ldg(reinterpret_cast<const uint4*>(v_rows + (size_t)(s.t0 + p0 + r - first) * a.v_stride));
    const float4 x0 = s_k[(r * 2) * 16 + l], x1 = s_k[(r * 2 + 1) * 16 + l];
    const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float v[8];
    unpack8(vr, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] != v[e] ? 0.f : v[e];
    const size_t row = ((unit << c.page_log2) + r) * kHeadDim;
    reinterpret_cast<uint2*>(c.k_codes + row)[l] = quantise8(x, inv_k);
    reinterpret_cast<uint2*>(c.v_codes + row)[l] = quantise8(v, inv_v);
  }
  // earlier tokens of the page, when the scale grew
  if (ek > old_k || ev > old_v) {
    const float fk = exp2_int(max(old_k - ek, -126)), fv = exp2_int(max(old_v - ev, -126));
    for (int r = warp * 2 + half; r < r0; r += 2 * kWarps) {
      const size_t row = ((unit << c.page_log2) + r) * kHeadDim;
      if (ek > old_k) {
        uint2* kc = reinterpret_cast<uint2*>(c.k_codes + row) + l;
        const uint2 o = *kc;
        *kc = make_uint2(rescale4(o.x, fk), rescale4(o.y, fk));
      }
      if (ev > old_v) {
        uint2* vc = reinterpret_cast<uint2*>(c.v_codes + row) + l;
        const uint2 o = *vc;
        *vc = make_uint2(rescale4(o.x, fv), rescale4(o.y, fv));
      }
    }
  }
}

// Blocks [0, q_blocks): queries; the others: a cache unit each.  One launch, which a decode step notices (64 sequences: 5.4 us,
// 8.3 us as two).  Of a long prompt the queries come first and the units fill their places as they end: 132 us for 16384
// tokens (64 + 8 + 8 heads, 638 MB, 71 % of the memory's copy rate); 127 us as two kernels with registers of their own, and
// 141-160 us with the two kinds of blocks mixed or fewer of the first.  The queries are bound by their instructions (issue
// slots 69 % busy before they went to pairs), the units by a chain of reads: lengths, page, rows, table, scale.
__global__ void __launch_bounds__(kAppendThreads, 5) kv_append_kernel(const KvBatch c, const KvAppendArgs a, int q_blocks) {
  extern __shared__ uint4 shared[];  // queries on their way, or the page's new keys, rotated: [row][2][16 lanes] of float4
  __shared__ float s_amax[2][kWarps];
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) check_starts(c);
  if ((int)blockIdx.x < q_blocks) rope_queries(c, a, (int)blockIdx.x, q_blocks, shared);
  else append_unit(c, a, (int)blockIdx.x - q_blocks, s_amax, reinterpret_cast<float4*>(shared));
}

constexpr int kGatherRowsPerBlock = 32;
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads)
    kv_gather_kernel(const KvBatch c, const int32_t* start, const int32_t* out_start, int n_rows, uint16_t* k_out,
                     uint16_t* v_out) {
  __shared__ int s_page[kGatherRowsPerBlock], s_slot[kGatherRowsPerBlock];
  const int r0 = (int)blockIdx.x * kGatherRowsPerBlock;
  const int rows = min(kGatherRowsPerBlock, n_rows - r0);
  if ((int)threadIdx.x < rows) {
    const int r = r0 + (int)threadIdx.x;
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(out_start + mid) <= r) lo = mid; else hi = mid;
    }
    const long long pos = (long long)__ldg(start + lo) + r - __ldg(out_start + lo);
    const bool ok = r >= __ldg(out_start + lo) && r < __ldg(out_start + lo + 1) && pos >= 0 &&
                    pos < (long long)c.max_pages * c.page;
    if (!ok) set_status(c.status, DEV_ERR_BOUNDS);
    s_page[threadIdx.x] = ok ? load_page(c, lo, (int)(pos >> c.page_log2)) : -1;
    s_slot[threadIdx.x] = (int)(pos & (c.page - 1));
  }
  __syncthreads();
  const int per_row = c.Hkv * (kHeadDim / 16);  // 16 codes a thread
  const bool is_v = blockIdx.y;
  const uint8_t* codes = is_v ? c.v_codes : c.k_codes;
  const uint8_t* scale = is_v ? c.v_scale : c.k_scale;
  uint16_t* out = is_v ? v_out : k_out;
  for (int i = threadIdx.x; i < rows * per_row; i += kGatherThreads) {
    const int r = i / per_row, q = i - r * per_row, h = q >> 3, d = (q & 7) * 16;
    const int pg = s_page[r];
    uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};  // a row that is not there reads as zeros
    if (pg >= 0) {
      const size_t unit = (size_t)pg * c.Hkv + h;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(codes + ((unit << c.page_log2) + s_slot[r]) * kHeadDim + d));
      // 2^e as a product of two halves, each a normal number
      const int e = (int)__ldg(scale + unit) - 127;
      const float f0 = exp2_int(e >> 1), f1 = exp2_int(e - (e >> 1));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t u[8];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 a = e4m3x2_f32(w[m] & 0xFFFFu), b = e4m3x2_f32(w[m] >> 16);
        u[2 * m] = bf16_pair(a.x * f0 * f1, a.y * f0 * f1);
        u[2 * m + 1] = bf16_pair(b.x * f0 * f1, b.y * f0 * f1);
      }
      o[0] = make_uint4(u[0], u[1], u[2], u[3]);
      o[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
    uint4* to = reinterpret_cast<uint4*>(out + ((size_t)(r0 + r) * c.Hkv + h) * kHeadDim + d);
    to[0] = o[0];
    to[1] = o[1];
  }
}

// cos and sin of p * base^(-2i / rot), the angle and both functions in double: at position 10^6 the largest angle has
// lost 20 of fp32's 24 bits.
__global__ void rope_table_kernel(int max_pos, int rot, double base, float* cos_sin) {
  const int half = rot >> 1;
  const long long n = (long long)max_pos * half;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long p = i / half;
    const int f = (int)(i - p * half);
    double s, co;
    sincos((double)p * pow(base, -2.0 * f / rot), &s, &co);
    cos_sin[p * rot + f] = (float)co;
    cos_sin[p * rot + half + f] = (float)s;
  }
}

// The rotation of each new token, positions on one axis per frequency: read from the table once a step, for every layer's append
// (which then reads whole rows as it does from the table).  Four frequencies a thread; a position that the table does not have
// makes the row's part of it NaN, so that the token does not pass for one at another place.
__global__ void __launch_bounds__(256) rope_rows_kernel(const __grid_constant__ RopeAxes axes, int T, const int32_t* positions, long long stride,
                                                        const float* cos_sin, int max_pos, int rot, float* rows, unsigned* status) {
  const int half = rot >> 1, quads = half >> 2;
  const long long n = (long long)T * quads;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long t = i / quads;
    const int f = (int)(i - t * quads) * 4;
    float c[4], s[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int pos = __ldg(positions + axes.axis[f + x] * stride + t);
      const bool ok = pos >= 0 && pos < max_pos;
      if (!ok) set_status(status, DEV_ERR_BOUNDS);
      const float* row = cos_sin + (size_t)(ok ? pos : 0) * rot + f + x;
      c[x] = ok ? __ldg(row) : __int_as_float(0x7FFFFFFF);
      s[x] = ok ? __ldg(row + half) : __int_as_float(0x7FFFFFFF);
    }
    float* out = rows + t * rot + f;
    *reinterpret_cast<float4*>(out) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(out + half) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

}  // namespace

cudaError_t launch_rope_rows(const RopeAxes& axes, int T, const int32_t* positions, long long stride, const float* cos_sin,
                             int max_pos, int rot, float* rows, unsigned* status, cudaStream_t stream) {
  const long long blocks = ((long long)T * (rot >> 3) + 255) / 256;
  rope_rows_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(axes, T, positions, stride, cos_sin, max_pos, rot,
                                                                                rows, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvBatch& c, const KvAppendArgs& a, int n_sms, cudaStream_t stream) {
  const long long slots = (long long)c.T / c.page + 2LL * c.B;
  const long long chunks = (c.Hq + kQHeads - 1) / kQHeads, need = a.q ? ((long long)c.T * chunks + kWarps - 1) / kWarps : 0;
  const long long most = (long long)kQBlocksPerSm * n_sms, q_blocks = need < most ? need : most;
  const int keys = c.page * kHeadDim * (int)sizeof(float), bytes = q_blocks && keys < kQShared ? kQShared : keys;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kv_append_kernel), 128 * kHeadDim * (int)sizeof(float), allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_append_kernel, dim3((unsigned)(q_blocks + slots * c.Hkv)), dim3(kAppendThreads), bytes, stream, false, c,
                       a, (int)q_blocks);
}

cudaError_t launch_kv_gather(const KvBatch& c, const int32_t* start, const int32_t* out_start, int n_rows, uint16_t* k,
                             uint16_t* v, cudaStream_t stream) {
  const dim3 grid((n_rows + kGatherRowsPerBlock - 1) / kGatherRowsPerBlock, 2);
  kv_gather_kernel<<<grid, kGatherThreads, 0, stream>>>(c, start, out_start, n_rows, k, v);
  return cudaGetLastError();
}

cudaError_t launch_rope_table(int max_pos, int rot, double base, float* cos_sin, cudaStream_t stream) {
  const long long n = (long long)max_pos * (rot >> 1);
  const long long blocks = (n + 255) / 256;
  rope_table_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(max_pos, rot, base, cos_sin);
  return cudaGetLastError();
}

}  // namespace moe
