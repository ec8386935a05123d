// Eviction from the paged cache: each key/value head of a sequence keeps its tokens of the largest accumulated weights.
//
// Choosing.  The weights are ordered by their bits (a float above 0 orders as an unsigned integer; anything else counts as 0, a
// token that stays in any case as the largest), and the m-th largest is found digit by digit from the top: 11, 10 and 10 bits
// below the sign, a histogram of the tokens that agree so far at each.  Tokens above it stay, and of its equals the first ones that there is
// room for.  A cluster of blocks shares one (sequence, head): each holds a piece of the tokens in shared memory, reads the others'
// histograms there, and knows from the others' counts where its own tokens go.  So the weights are read once, and the choice
// and its order depend on nothing but them.
//
// Packing.  A block per (new page, head): its tokens' rows come from wherever they were, 128 bytes each, which memory reads
// whole.  The page's scale is the largest of their pages' scales, known before the codes come: rows of pages of that scale are copied, the
// others' codes are rounded again (exact unless they become subnormal).  The bytes of the kept rows bound it.
//
// Measured (32 sequences of 3000-9000 tokens, 8 heads, cut to 1500-2200): choosing 15-18 us (5,500 cycles until the weights are there, 4,000 a
// digit, 7,000 for the tokens' places), packing 36-42 (250 MB, 6-7 TB/s).
#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPerThread = kBins / kThreads;
constexpr int kMaxRanks = 8;
constexpr int kMostKeys = 49152;  // keys that a block keeps in shared memory; of a longer piece the rest is read for every digit

constexpr uint32_t kStays = 0xFFFFFFFFu;  // the key of a token that stays in any case
static_assert(kWarps == 32 && kPerThread == 2, "scans");

// The sum of the values of this warp's lanes below this one.
__device__ __forceinline__ uint32_t warp_before(uint32_t v, uint32_t& all) {
  const int lane = threadIdx.x & 31;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  all = __shfl_sync(0xffffffffu, x, 31);
  return x - v;
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld_shared_cluster_u32x2(uint32_t cluster_addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_addr) : "memory");
  return v;
}

// Tokens of sequence b and how many stay; false (and DEV_ERR_CONFIG) when they do not fit the tables.
__device__ __forceinline__ bool load_evict(const KvBatch& c, const KvEvictArgs& e, int b, int& len, int& m) {
  len = __ldg(c.kv_len + b);
  const int keep = __ldg(e.keep + b);
  m = min(len, keep);
  const bool ok = len >= 0 && keep >= 0 && len <= (long long)c.max_pages * c.page && m <= (long long)e.new_max_pages * c.page;
  if (!ok && threadIdx.x == 0) set_status(c.status, DEV_ERR_CONFIG);
  return ok;
}

__global__ void __launch_bounds__(kThreads) kv_select_kernel(const KvBatch c, const KvEvictArgs e, int ranks, int cap) {
  extern __shared__ __align__(16) uint32_t s_keys[];  // [cap]
  __shared__ __align__(8) uint32_t s_hist[2][kBins];
  __shared__ uint32_t s_warp[kWarps], s_above[kWarps], s_equal[kWarps];
  __shared__ uint32_t s_digit, s_need;
  __shared__ uint32_t s_count[2];       // this block's tokens above the m-th weight, and equal to it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x % ranks, unit = (int)blockIdx.x / ranks, b = unit / c.Hkv, h = unit - b * c.Hkv;
  const int width = e.new_max_pages << c.page_log2;
  int32_t* kept = e.kept + (size_t)unit * width;
  pdl_launch_dependents();
  int len, m;
  const bool ok = load_evict(c, e, b, len, m);
  if (h == 0 && rank == 0 && tid == 0) e.new_len[b] = ok ? m : -1;
  if (!ok) m = 0;
  for (int i = m + rank * kThreads + tid; i < width; i += ranks * kThreads) kept[i] = -1;
  if (m == 0) return;  // the whole cluster

  // this block's piece [lo, lo + n)
  const int share = ((len + ranks - 1) / ranks + kThreads - 1) / kThreads * kThreads;
  const int lo = (int)min((long long)len, (long long)rank * share), n = min(share, len - lo);
  const int32_t* table = c.page_table + (size_t)b * c.max_pages;
  const int stay0 = min(e.sink, len), stay1 = max(stay0, len - min(e.recent, len));  // tokens before the one and from the other on
  auto to_key = [&](float w, int j) { return j < stay0 || j >= stay1 ? kStays : w > 0.f ? __float_as_uint(w) : 0u; };  // (behind the end: stays)
  // the weights of the tokens from lo + i on, as far as their page goes (nullptr: on no page)
  auto weights_at = [&](int i) -> const float* {
    const int j = lo + i, p = __ldg(table + (j >> c.page_log2));
    if (p < 0 || p >= c.n_pages) {
      set_status(c.status, DEV_ERR_BOUNDS);
      return nullptr;
    }
    return e.weight + (((size_t)p * c.Hkv + h) << c.page_log2) + (j & (c.page - 1));
  };
  const int cached = min(n, cap);
#pragma unroll 4
  for (int i = 4 * tid; i < cached; i += 4 * kThreads) {  // four at a time: pages hold multiples of 16
    const float* w = weights_at(i);
    const float4 v = w ? *reinterpret_cast<const float4*>(w) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int j = lo + i;
    *reinterpret_cast<uint4*>(s_keys + i) = make_uint4(to_key(v.x, j), to_key(v.y, j + 1), to_key(v.z, j + 2), to_key(v.w, j + 3));
  }
  auto key = [&](int i) {
    if (i < cached) return s_keys[i];
    const float* w = weights_at(i);
    return to_key(w ? *w : 0.f, lo + i);
  };

  __syncthreads();
  const int stay = len - (stay1 - stay0);
  uint32_t prefix = m <= stay ? kStays : 0u, need = (uint32_t)(m <= stay ? m : m - stay);
#pragma unroll 1
  for (int pass = 0; pass < (m <= stay ? 0 : 3); ++pass) {
    const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0;
    const uint32_t seen = pass == 0 ? 0x80000000u : 0xFFFFFFFFu << (shift + 10), mask = pass == 0 ? 0x7FFu : 0x3FFu;
    uint32_t* hist = s_hist[pass & 1];
#pragma unroll
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    auto count = [&](uint32_t k) {
      if ((k & seen) == prefix) atomicAdd(&hist[k >> shift & mask], 1u);
    };
#pragma unroll 2
    for (int i = 4 * tid; i < cached; i += 4 * kThreads) {
      const uint4 k = *reinterpret_cast<const uint4*>(s_keys + i);
      count(k.x);
      count(k.y);
      count(k.z);
      count(k.w);
    }
    for (int i = cached + tid; i < n; i += kThreads) count(key(i));
    if (ranks > 1) cluster_sync(); else __syncthreads();
    // the digit, from the top: thread t has the bins kBins - 1 - 2t and the one below it
    const int top = kBins - 1 - 2 * tid;
    uint32_t v0 = 0, v1 = 0, all;
    if (ranks > 1) {
      for (int r = 0; r < ranks; ++r) {
        const uint2 v = ld_shared_cluster_u32x2(mapa_shared(smem_u32(hist + top - 1), (uint32_t)r));
        v0 += v.y;
        v1 += v.x;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(hist + top - 1);
      v0 = v.y;
      v1 = v.x;
    }
    uint32_t before = warp_before(v0 + v1, all);
    if (lane == 0) s_warp[warp] = all;
    __syncthreads();
    before += __shfl_sync(0xffffffffu, warp_before(s_warp[lane], all), warp);
    if (before < need && need <= before + v0 + v1) {  // one thread
      const bool first = need <= before + v0;
      s_digit = (uint32_t)(first ? top : top - 1);
      s_need = need - before - (first ? 0u : v0);
    }
    __syncthreads();
    prefix |= s_digit << shift;
    need = s_need;
  }

  // Tokens above the m-th weight stay, and `need` of its equals.  Each warp has a piece of its own, in order.
  const int per_warp = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
  uint32_t above = 0, equal = 0;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const uint32_t k = i < w1 ? key(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < w1 && k > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, i < w1 && k == prefix));
  }
  if (lane == 0) {
    s_above[warp] = above;
    s_equal[warp] = equal;
  }
  __syncthreads();
  uint32_t all_above, all_equal;
  above = __shfl_sync(0xffffffffu, warp_before(s_above[lane], all_above), warp);
  equal = __shfl_sync(0xffffffffu, warp_before(s_equal[lane], all_equal), warp);
  if (ranks > 1) {
    if (tid == 0) {
      s_count[0] = all_above;
      s_count[1] = all_equal;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const uint32_t at = mapa_shared(smem_u32(s_count), (uint32_t)r);
      above += ld_shared_cluster_u32(at);
      equal += ld_shared_cluster_u32(at + 4);
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const uint32_t k = i < w1 ? key(i) : 0u;
    const bool is_above = i < w1 && k > prefix, is_equal = i < w1 && k == prefix;
    const uint32_t m_above = __ballot_sync(0xffffffffu, is_above), m_equal = __ballot_sync(0xffffffffu, is_equal);
    const uint32_t eq = equal + __popc(m_equal & below);
    if (is_above || (is_equal && eq < need)) kept[above + __popc(m_above & below) + min(eq, need)] = lo + i;
    above += __popc(m_above);
    equal += __popc(m_equal);
  }
  if (ranks > 1) cluster_sync();  // the others may still read this block's counts
}

constexpr int kCopyThreads = 128;

__global__ void __launch_bounds__(kCopyThreads) kv_pack_kernel(const KvBatch c, const KvEvictArgs e) {
  __shared__ long long s_row[128];  // the tokens' rows in the pool, -1: none
  __shared__ uint32_t s_scale[128];  // their scales: key | value << 8
  __shared__ uint32_t s_top[2][kCopyThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int i = (int)(blockIdx.x % (unsigned)e.new_max_pages), unit = (int)(blockIdx.x / (unsigned)e.new_max_pages);
  const int b = unit / c.Hkv, h = unit - b * c.Hkv;
  pdl_wait();
  int len, m;
  if (!load_evict(c, e, b, len, m)) return;
  const int n = min(c.page, m - (i << c.page_log2));
  if (n <= 0) return;
  const int pg = __ldg(e.new_table + (size_t)b * e.new_max_pages + i);
  if (pg < 0 || pg >= c.n_pages) {
    if (tid == 0) set_status(c.status, DEV_ERR_BOUNDS);
    return;
  }
  const size_t to = (size_t)pg * c.Hkv + h;
  uint32_t sk = 0, sv = 0;
  if (tid < n) {
    const int j = e.kept[((size_t)unit * e.new_max_pages + i << c.page_log2) + tid];
    const int p = j >= 0 && j < len ? __ldg(c.page_table + (size_t)b * c.max_pages + (j >> c.page_log2)) : -1;
    const bool there = p >= 0 && p < c.n_pages;
    const size_t from = there ? (size_t)p * c.Hkv + h : 0;
    const long long row = there ? (long long)(from << c.page_log2) + (j & (c.page - 1)) : -1;
    if (there) {
      sk = c.k_scale[from];
      sv = c.v_scale[from];
    } else {
      set_status(c.status, DEV_ERR_BOUNDS);
    }
    s_row[tid] = row;
    s_scale[tid] = sk | sv << 8;
    e.weight[(to << c.page_log2) + tid] = there ? e.weight[row] : 0.f;
  }
  sk = __reduce_max_sync(0xffffffffu, sk);
  sv = __reduce_max_sync(0xffffffffu, sv);
  if (lane == 0) {
    s_top[0][tid >> 5] = sk;
    s_top[1][tid >> 5] = sv;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCopyThreads / 32; ++w) {
    sk = max(sk, s_top[0][w]);
    sv = max(sv, s_top[1][w]);
  }
  if (tid == 0) {
    c.k_scale[to] = (uint8_t)sk;
    c.v_scale[to] = (uint8_t)sv;
  }
  // 16 codes of a key and of a value a thread and step
  constexpr int kPieces = kHeadDim / 16;
#pragma unroll 4
  for (int x = tid; x < n * kPieces; x += kCopyThreads) {
    const int r = x / kPieces;
    const long long row = s_row[r];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;  // a token that is on no page becomes zeros
    if (row >= 0) {
      k = *reinterpret_cast<const uint4*>(c.k_codes + row * kHeadDim + (x % kPieces) * 16);
      v = *reinterpret_cast<const uint4*>(c.v_codes + row * kHeadDim + (x % kPieces) * 16);
      const int dk = (int)(s_scale[r] & 255u) - (int)sk, dv = (int)(s_scale[r] >> 8) - (int)sv;
      if (dk) {
        const float f = exp2_int(max(dk, -126));
        k = make_uint4(rescale4(k.x, f), rescale4(k.y, f), rescale4(k.z, f), rescale4(k.w, f));
      }
      if (dv) {
        const float f = exp2_int(max(dv, -126));
        v = make_uint4(rescale4(v.x, f), rescale4(v.y, f), rescale4(v.z, f), rescale4(v.w, f));
      }
    }
    const size_t at = ((to << c.page_log2) + r) * kHeadDim + (x % kPieces) * 16;
    *reinterpret_cast<uint4*>(c.k_codes + at) = k;
    *reinterpret_cast<uint4*>(c.v_codes + at) = v;
  }
}

}  // namespace

// A cluster where a block's piece would not fit its shared memory, or where it is long and blocks are few.  Lengths are the device's: the
// table's width stands for them, so a wide table costs time whatever is in it (8 sequences of 2000 tokens, 8 heads: 18 us in a tight table, 64
// in one of 131072 tokens; 32 of 3000-9000: 68 and 141; one of 700, 4 heads: 14 and 16).
cudaError_t launch_kv_evict(const KvBatch& c, const KvEvictArgs& e, int n_sms, cudaStream_t stream) {
  const long long units = (long long)c.B * c.Hkv, most = (long long)c.max_pages * c.page;
  int ranks = 1;
  while (ranks < kMaxRanks && (most / ranks > kMostKeys || (most / ranks > 16384 && units * ranks < 2 * n_sms))) ranks *= 2;
  const long long share = ((most + ranks - 1) / ranks + kThreads - 1) / kThreads * kThreads;
  const int cap = (int)(share < kMostKeys ? share : kMostKeys);
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t r = allow_shared_memory(reinterpret_cast<const void*>(kv_select_kernel), kMostKeys * 4, allowed);
  if (r != cudaSuccess) return r;
  r = launch_kernel_cluster(kv_select_kernel, dim3((unsigned)(units * ranks)), dim3(kThreads), (size_t)cap * 4, stream, false, ranks, c,
                            e, ranks, cap);
  if (r != cudaSuccess) return r;
  return launch_kernel(kv_pack_kernel, dim3((unsigned)(units * e.new_max_pages)), dim3(kCopyThreads), 0, stream, true, c, e);
}

}  // namespace moe
