// Device helpers of the attention operators: batch lookups, E4M3 and E8M0 conversions.
#pragma once

#include "attention_internal.h"
#include "moe_common.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

namespace moe {

// The largest i in [0, n) with key(i) <= u, for keys that do not decrease (0 when key(0) > u): a warp
// probes 32 places at a time, so 1024 sequences take two dependent loads.  The whole warp gives the same u.
template <typename Key>
__device__ __forceinline__ int warp_search(int n, int u, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const bool at = lane * step < n && key(lo + lane * step) <= u;
    const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, at)));
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  return lo;
}

// New tokens [t0, t1) of sequence b and its length; false (and DEV_ERR_CONFIG) when they contradict each other.
struct SeqRange {
  int t0, t1, len;
  __device__ __forceinline__ int first() const { return len - (t1 - t0); }  // position of the first new token
};
__device__ __forceinline__ bool load_seq(const KvBatch& c, int b, SeqRange& s) {
  s.t0 = __ldg(c.q_start + b);
  s.t1 = __ldg(c.q_start + b + 1);
  s.len = __ldg(c.kv_len + b);
  const bool ok = s.t0 >= 0 && s.t1 >= s.t0 && s.t1 <= c.T && s.len >= 0 && s.len <= (long long)c.max_pages * c.page;
  if (!ok) set_status(c.status, DEV_ERR_CONFIG);
  return ok;
}

// Every token has a sequence: one thread of a launch looks.
__device__ __forceinline__ void check_starts(const KvBatch& c) {
  if (__ldg(c.q_start) != 0 || __ldg(c.q_start + c.B) != c.T) set_status(c.status, DEV_ERR_CONFIG);
}

// Page of a sequence's tokens [j * page, (j+1) * page), or -1 (and DEV_ERR_BOUNDS) when it is not in the pool.
__device__ __forceinline__ int load_page(const KvBatch& c, int b, int j) {
  if (j < 0 || j >= c.max_pages) {
    set_status(c.status, DEV_ERR_BOUNDS);
    return -1;
  }
  const int p = __ldg(c.page_table + (size_t)b * c.max_pages + j);
  if (p < 0 || p >= c.n_pages) {
    set_status(c.status, DEV_ERR_BOUNDS);
    return -1;
  }
  return p;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Two floats -> two E4M3 codes (nearest, ties to even; beyond +-448 saturates; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Two E4M3 codes (low 16 bits) -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(h));
}

// 16 bytes from global to shared memory, in the background: the first `bytes` of them (0 or 16), then zeros.  A later
// cp_async_wait<n> waits for all but the last n groups.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// An arrival of this thread at an mbarrier once all its copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Host: gives a kernel its dynamic shared memory, once per device (`done`: one bit each, a static of the caller's).
inline cudaError_t allow_shared_memory(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace moe
