// What the attention kernels share: key tiles of 128 tokens, their distribution over blocks, tensor-core
// descriptors for E4M3 operands and the joining of split rows.
#pragma once

#include "attention_common.cuh"

#include <math_constants.h>

namespace moe {

constexpr int kTile = 128;                        // keys per tile
constexpr int kTileBytes = kTile * kHeadDim;      // E4M3 codes of one head's keys (or values) of a tile: 16 KB

// Now and then while a wait lasts: has it lasted longer than the limit (abort_flag[1], in us; then the abort flag and
// DEV_ERR_TIMEOUT are set), or has another role given up?  Not inline: these kernels have some thirty waits in their loops, and with a timer's code in each
// of them instruction fetch became what the loops waited for.
static __device__ __noinline__ bool wait_is_over(unsigned long long* since, volatile int* abort_flag, unsigned* status) {
  const unsigned long long now = globaltimer_ns();
  if (*since == 0) *since = now;
  if (*abort_flag == 1) return true;
  if (now - *since < 1000ull * (unsigned)abort_flag[1]) return false;
  *abort_flag = 1;
  set_status(status, DEV_ERR_TIMEOUT);
  return true;
}
// Waits for the phase with the given parity to complete; false when it gave up.
__device__ __forceinline__ bool mbar_wait_tries(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  bool ok = mbar_try_wait(bar, parity);
  unsigned long long since = 0;
#pragma unroll 1
  for (uint32_t i = 1; !ok; ++i) {
    ok = mbar_try_wait(bar, parity);
    if ((i & 127u) == 0 && !ok && wait_is_over(&since, abort_flag, status)) return false;
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  return __all_sync(0xffffffffu, mbar_wait_tries(bar, parity, abort_flag, status));
}
// Two or three barriers at a time, the lanes sharing them out: a try takes 100 cycles and more while the tensor core's
// operands keep shared memory busy, and tries one after another add up.
__device__ __forceinline__ bool warp_wait2(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, volatile int* abort_flag,
                                           unsigned* status) {
  const bool second = threadIdx.x & 1;
  return warp_wait(second ? b1 : b0, second ? p1 : p0, abort_flag, status);
}
__device__ __forceinline__ bool warp_wait3(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2,
                                           volatile int* abort_flag, unsigned* status) {
  const int which = (threadIdx.x & 31) < 11 ? 0 : (threadIdx.x & 1) + 1;
  return warp_wait(which == 0 ? b0 : which == 1 ? b1 : b2, which == 0 ? p0 : which == 1 ? p1 : p2, abort_flag, status);
}

// The first key that a query at this position sees.  Positions may be negative (a sequence may bring more new tokens than it
// has) and a window as large as an int: no step of this leaves an int's range, as pos - window + 1 would there -- and then
// the first key, with the page of it, could be anything.
__device__ __forceinline__ int window_lo(int pos, int window) { return window > 0 ? max(0, max(pos, -1) - (window - 1)) : 0; }

// The keys that any new token of a sequence sees: [lo, hi), in tiles [tile0, tile0 + nt).  A sequence with new
// tokens has at least one tile, so that its rows are written even when they see nothing.
struct KeyRange {
  int lo, hi, tile0, nt;
};
__device__ __forceinline__ KeyRange key_range(const SeqRange& s, const AttentionArgs& a) {
  KeyRange r;
  r.hi = s.len;
  r.lo = window_lo(s.first(), a.window);
  r.tile0 = r.lo / kTile;
  r.nt = s.t1 > s.t0 ? max(1, (r.hi + kTile - 1) / kTile - r.tile0) : 0;
  return r;
}

// What all sequences before this thread's share of them cost, and all together: `threads` threads each take a run of sequences.
template <typename Cost>
__device__ __forceinline__ long long scan_batch(const KvBatch& c, int threads, long long* s_warp, long long& mine, long long& total,
                                                Cost cost) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (c.B + threads - 1) / threads;
  mine = 0;
#pragma unroll 1
  for (int b = tid * per; b < min(c.B, (tid + 1) * per); ++b) mine += cost(b);
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll 1
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  __syncthreads();
  return before + x - mine;
}

// 3-D tiled bulk tensor load global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------- tcgen05 with E4M3 operands
// Instruction descriptor of kind::f8f6f4, E4M3 A and B, fp32 accumulator; a_mn, b_mn: A, B stored with M, N
// contiguous (else K).
__device__ __forceinline__ uint32_t umma_idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  uint32_t d = 0;
  d |= 1u << 4;                    // D format: f32 (A and B format 0: E4M3)
  d |= (a_mn ? 1u : 0u) << 15;
  d |= (b_mn ? 1u : 0u) << 16;
  d |= (uint32_t)(N >> 3) << 17;
  d |= (uint32_t)(M >> 4) << 24;
  return d;
}

// Descriptor of an 8-bit operand stored without swizzle, M or N contiguous: 16 bytes (16 rows of the operand) per K index,
// eight K indexes to 128 contiguous bytes, the next eight 128 bytes on, the next 16 rows `block` bytes on.
__device__ __forceinline__ uint64_t umma_desc_mn16(uint32_t smem_addr, uint32_t block) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;   // leading byte offset: along K
  d |= (uint64_t)(block >> 4) << 32;  // stride byte offset: along M or N
  d |= (uint64_t)1u << 46;            // descriptor version
  return d;
}

__device__ __forceinline__ void umma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 2^x (ex2.approx: 2 ulp; subnormal results are zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(s - 127) of a scale byte (255 reads as 254; 0, which no append writes, as 0).
__device__ __forceinline__ float exp2_byte(uint32_t s) { return __int_as_float((int)min(s, 254u) << 23); }

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The denominator of a row, l = sum of 2^(u - r), as such calls leave it.
__device__ __forceinline__ void write_lse(const AttentionArgs& a, size_t row, float r, float l) {
  if (a.lse) a.lse[row] = (r + log2f(l)) * a.lse_unit;
}
__device__ __forceinline__ void mark_split(const AttentionArgs& a, size_t row) { a.lse[row] = __uint_as_float(kSplitMark | blockIdx.x); }

// Pairs of floats in one 64-bit register: one instruction for two products or sums.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
// A query row in E4M3 twice over: q * 2^-e = hi + lo with hi the nearest E4M3 value and lo the rest's, e chosen so that
// the row's largest element lies in [128, 256).  bf16 has 8 significant bits and an E4M3 value 4: the rest of a
// rounding to 4 bits fits 4 bits again, so the sum is exact for every element above 2^-9 of the row's largest and
// within 2^-17 of that one below.  hi . k + lo . k then takes E4M3 keys as they lie in the cache.
__device__ __forceinline__ int query_exponent(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127 - 7;
  return amax > 0.f ? max(e, -100) : 0;
}
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = e4m3x2(a, b);
  const float2 h = e4m3x2_f32(hi);
  lo = e4m3x2(a - h.x, b - h.y);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two bf16 numbers times inv as split_e4m3x2 does it, by way of f16: 8 bits below 2^9 are exact there down to 2^-16, and
// what is smaller has two halves of zero.
__device__ __forceinline__ void split_bf16x2(uint32_t w, float inv, uint32_t& hi, uint32_t& lo) {
  __half2_raw v, h;
  *reinterpret_cast<uint32_t*>(&v) = pack_f16x2(bf16_lo(w) * inv, bf16_hi(w) * inv);
  hi = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3);
  h = __hsub2(__half2(v), __half2(h));
  lo = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace moe
