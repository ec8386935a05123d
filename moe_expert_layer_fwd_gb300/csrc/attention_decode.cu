// Attention of few query rows per key/value head (decoding, and the check of a few speculated tokens): the cache is
// read once and everything else is small, so the bytes of the cache bound it.
//
// The keys are the M operand: for one key/value head a tile of 128 keys, E4M3 as cached, times the query rows that read
// this head (columns: new tokens x grouped heads, NC of them),
//   S^T[128 keys, 2 NC] = K . [q_hi | q_lo]^T           tcgen05 kind::f8f6f4, M = 128, N = 2 NC
//   u = (S_hi + S_lo) * scale * 2^(e_k + e_q) + e_v     log2 of the weight times the size of the page's values
//   r = max(r, max_j u),  p'_j = 2^(u_j - r + 6),  l = l f + sum_j p'_j 2^-e_v
//   p'_j = hi + lo / 32 if p'_j >= 2^-7, else 2^-15 (hi + lo / 32); hi, lo in E4M3
//   O^T[128 dims, 4 NC] = V^T . [hi | lo | hi of small weights | lo of them]   the same instruction, V read with its dims contiguous
// so that neither keys nor values pass through a register: TMA writes the pages' codes to shared memory with the
// 128-byte swizzle and the tensor core reads them there, once each.  Scales never touch the codes: those of the keys
// are multiplied onto S, those of the values are added to the exponent.  The reference r follows the running maximum of u:
// the largest p' lies within 2^6 .. 2^8 whatever the pages' scales are, errors are relative to the largest
// term of the sum that is being computed, and the denominator takes the scale out again.
//
// Range of the weights: the four kinds of parts have accumulators of their own, so each has a scale of its own.  A weight keeps
// 8 bits down to 2^-28 of the largest and is rounded to multiples of 2^-35 of it below.  That is needed: a key that takes
// most of the softmax leaves thousands of others with 2^-16 .. 2^-24 of its weight and, together, a share that counts.  (Two parts
// of one scale keep multiples of 2^-15: 8000 equal keys 12 nats below one lose their whole share, 5 % of the output.)  The parts of
// the small weights cost a decode batch of 64 sequences 2 us (117 -> 119).
//
// A softmax thread owns one key and half of the columns (S, p'), and one output dim of them (O, accumulated in tensor memory
// and rescaled only when r moves).
//
// Work: all (sequence, head, tile) in one order, cut into equal runs, one per block (two blocks per SM): a long sequence is
// split over as many blocks as it takes, a short one shares a block.  A row whose tiles lie in one block
// is finished there; otherwise the parts (sum, maximum, denominator) go to the workspace and a second kernel joins them in a
// fixed order.  The host knows none of the lengths.
//
// Measured (64 sequences of 1500-8190 tokens, 64 query heads on 8, 685 MB of cache): 119 us a call; from the first copy to the last
// product 94 us = 7.3 TB/s, the memory's rate; the rest is 6 us until the first scores (lengths, page table, first copies, one
// after another), 10 us in which the slowest blocks finish, and the join.  Small sequences are bound by that chain of waits.
//
// Warps: 8 softmax (four for each half of the columns), then TMA, MMA, queries.  Every wait is bounded (2 s).
#include "attention_tiles.cuh"

namespace moe {
namespace {

constexpr int kWholeTiles = 4;    // rows of at most so many tiles are not split
constexpr int kMinRun = 4;        // tiles in a block's run, at least (4 sequences of 2000, 8 key/value heads: 21.6 us at 2,
                                  // 19.6 at 4, 23.7 at 6; one of 1000: 17.5, 17.5, 21.6)
// p' = 2^(u - r + kBase) with u <= r + kSlack is at most 2^8; r moves so seldom that the sums in tensor memory are hardly ever
// rescaled.
constexpr float kBase = 6.f, kSlack = 2.f;
// What hi leaves of a number up to 2^8 is at most 8, so lo can be stored 32 times larger; weights below 2^kSmall are stored 2^15
// times larger, at most 2^8 then.  Rounded to multiples of E4M3's smallest number, 2^-9 / 32, a number has 8 bits from 2^-7 on.
constexpr float kSmall = -7.f, kSmallDown = 1.f / 32768.f;
constexpr float kLoUp = 32.f, kLoDown = 1.f / 32.f;

struct TileInfo {    // per 16 keys of a tile
  float kf[8];       // 2^e_k
  float lv[8];       // e_v
  float un[8];       // 2^-e_v
  uint32_t have;     // bit i: the page of keys 16 i .. 16 i + 15 is there
  uint32_t pad[3];
};

template <int NC>
struct Cfg {
  static constexpr int kPerSm = 2;
  static constexpr int kStages = NC == 8 ? 3 : 2;
  static constexpr int kQBufs = 2;                          // the next segment's scores start before this one has ended
  static constexpr int kGroups = 2;                         // groups of four softmax warps, each with half of the columns
  static constexpr int kCols = NC / kGroups;
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kQWarp = kSoftWarps + 2;
  static constexpr int kThreads = 32 * (kSoftWarps + 3);
  static constexpr int kRows = 2 * NC;                      // hi and lo rows of the queries
  static constexpr int kPRows = 4 * NC;                     // columns of the weights' product: hi, lo; hi, lo of small ones
  static constexpr int kQBytes = kRows * 128;
  static constexpr int kPBlock = kTile * 16;                // the weights of 16 columns: 16 bytes a key
  static constexpr int kPOff = kStages * 2 * kTileBytes;
  static constexpr int kPBytes = kPRows / 16 * kPBlock;
  static constexpr int kQOff = kPOff + 2 * kPBytes;         // the weights of even and odd tiles
  static constexpr int kBarOff = kQOff + kQBufs * kQBytes;
  static constexpr int kNumBars = 4 * kStages + 2 * kQBufs + 9;
  static constexpr int kInfoOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // TileInfo [kStages]
  static constexpr int kQfOff = kInfoOff + kStages * (int)sizeof(TileInfo);  // float qf[kQBufs][NC], int token[kQBufs][NC]
  static constexpr int kMaxOff = kQfOff + kQBufs * NC * 8;  // float [3][NC][4]: maxima of even, odd tiles; denominators
  static constexpr int kMiscOff = kMaxOff + 3 * NC * 16;
  static constexpr int kBytes = 1024 + kMiscOff + 64;
  static constexpr int kTmemCols = 2 * kRows + kPRows;      // S twice, O (a power of two)
  static constexpr int kOCol = 2 * kRows;
  static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

// A run of tiles of one (sequence, head): the tiles [i0, i1) of its nt.
struct Segment {
  int b, h, i0, i1;
  SeqRange s;
  KeyRange r;
};

// Walks the segments of a block's run of tiles.
struct Walk {
  const KvBatch& c;
  const AttentionArgs& a;
  long long left;
  int b, h, i;
  __device__ Walk(const KvBatch& c_, const AttentionArgs& a_, long long n, int b_, int h_, int i_)
      : c(c_), a(a_), left(n), b(b_), h(h_), i(i_) {}
  __device__ bool next(Segment& g) {
    while (left > 0 && b < c.B) {
      const bool ok = load_seq(c, b, g.s);
      g.r = key_range(g.s, a);
      if (!ok || g.r.nt == 0) {
        ++b;
        h = i = 0;
        continue;
      }
      g.b = b;
      g.h = h;
      g.i0 = i;
      g.i1 = (int)min((long long)g.r.nt, i + left);
      left -= g.i1 - i;
      i = g.i1;
      if (i == g.r.nt) {
        i = 0;
        if (++h == c.Hkv) {
          h = 0;
          ++b;
        }
      }
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ int seq_tiles(const KvBatch& c, const AttentionArgs& a, int b) {
  SeqRange s;
  return load_seq(c, b, s) ? key_range(s, a).nt : 0;
}

// Tiles of all sequences before this thread's share of them, and of all: `threads` threads each take a run of sequences.
__device__ __forceinline__ long long scan_tiles(const KvBatch& c, const AttentionArgs& a, int threads, long long* s_warp,
                                                long long& mine, long long& total) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (c.B + threads - 1) / threads;
  mine = 0;
#pragma unroll 1
  for (int b = tid * per; b < min(c.B, (tid + 1) * per); ++b) mine += seq_tiles(c, a, b);
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

// Tiles per block: equal runs over the grid.
__device__ __forceinline__ long long tiles_per_block(long long n, int blocks) {
  return max((long long)kMinRun, (n + blocks - 1) / blocks);
}

// acc[x] += column x + column `lo` + x of this thread's tensor-memory lane.
template <int N>
__device__ __forceinline__ void add_product(uint32_t taddr, int lo, float (&acc)[N]) {
  uint32_t s[N], t[N];
  tmem_ld_async(taddr, s);
  tmem_ld_async(taddr + lo, t);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < N; ++x) acc[x] += __uint_as_float(s[x]) + __uint_as_float(t[x]);
}

// The sums of the weights' parts: columns x, `lo` + x, 2 `lo` + x and 3 `lo` + x of this thread's tensor-memory lane.
template <int N>
__device__ __forceinline__ void add_parts(uint32_t taddr, int lo, float (&acc)[N]) {
  uint32_t s[N], t[N];
  tmem_ld_async(taddr + 2 * lo, s);
  tmem_ld_async(taddr + 3 * lo, t);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < N; ++x) acc[x] = fmaf(__uint_as_float(t[x]), kLoDown, __uint_as_float(s[x])) * kSmallDown;
  tmem_ld_async(taddr, s);
  tmem_ld_async(taddr + lo, t);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < N; ++x) acc[x] += fmaf(__uint_as_float(t[x]), kLoDown, __uint_as_float(s[x]));
}

// Columns x and `lo` + x of this thread's tensor-memory lane, times f[x].
template <int N>
__device__ __forceinline__ void scale_columns(uint32_t taddr, int lo, const float (&f)[N]) {
  uint32_t s[N], t[N];
  tmem_ld_async(taddr, s);
  tmem_ld_async(taddr + lo, t);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < N; ++x) {
    s[x] = __float_as_uint(__uint_as_float(s[x]) * f[x]);
    t[x] = __float_as_uint(__uint_as_float(t[x]) * f[x]);
  }
  tmem_st(taddr, s);
  tmem_st(taddr + lo, t);
  tmem_wait_st();
}

// The warp's maxima of N columns, each lane bringing one value of each: v[0] is that of the returned column.  Lanes halve
// the columns they keep while they exchange the others, so N columns take N + 2 or so shuffles instead of 5 N.
template <int N>
__device__ __forceinline__ int columns_max(float (&v)[N], int lane) {
  int off = 16, col = 0;
#pragma unroll
  for (int half = N / 2; half >= 1; half /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int x = 0; x < half; ++x) {
      const float send = up ? v[x] : v[half + x], keep = up ? v[half + x] : v[x];
      v[x] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
    col += up ? half : 0;
  }
#pragma unroll
  for (; off >= 1; off /= 2) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return col;
}

// Two weights as hi + lo / kLoUp.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = e4m3x2(a, b);
  const float2 h = e4m3x2_f32(hi);
  lo = e4m3x2((a - h.x) * kLoUp, (b - h.y) * kLoUp);
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, Cfg<NC>::kPerSm)
    attention_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const KvBatch c, const AttentionArgs a, int split, float* part_o, float2* part_rl,
                            JoinInfo* info) {
  using C = Cfg<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* k_empty = k_full + C::kStages;
  uint64_t* v_full = k_empty + C::kStages;
  uint64_t* v_empty = v_full + C::kStages;
  uint64_t* q_full = v_empty + C::kStages;
  uint64_t* q_empty = q_full + C::kQBufs;
  uint64_t* s_full = q_empty + C::kQBufs;   // [2]
  uint64_t* s_empty = s_full + 2;           // [2]
  uint64_t* p_full = s_empty + 2;           // [2]
  uint64_t* o_full = p_full + 2;            // [2]
  uint64_t* done = o_full + 2;
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  float* s_qf = reinterpret_cast<float*>(smem + C::kQfOff);
  int* s_tok = reinterpret_cast<int*>(s_qf + C::kQBufs * NC);
  float* s_max = reinterpret_cast<float*>(smem + C::kMaxOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_begin = reinterpret_cast<int*>(smem + C::kMiscOff + 12);  // b, h, tile
  // [group][3]: a softmax warp of the group gave up (as s_max).  A group's own: its warps read it between two of the group's
  // barriers, where no other warp writes it, so all of them leave or all stay; a flag of both groups' could be set by the
  // other one while they read it, and those that stayed would wait at the barrier for those that left, with no limit.
  volatile int* s_bad_all = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 24);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv;
  pdl_launch_dependents();
  if (blockIdx.x == 0 && tid == C::kThreads - 1) check_starts(c);

  // ---- this block's run of tiles
  long long run = 0;
  int slot0 = 2 * (int)blockIdx.x;
  if (split) {
    long long mine, total;
    // the scan's scratch is the weights' operand, free until the roles start
    long long* s_warp = reinterpret_cast<long long*>(smem + C::kPOff);
    const long long before = scan_tiles(c, a, C::kThreads, s_warp, mine, total);
    const long long all = total * c.Hkv, per = tiles_per_block(all, gridDim.x);
    const long long begin = (long long)blockIdx.x * per;
    run = min(per, all - begin);
    if (run <= 0) {
      if (tid == 0) info[blockIdx.x].split = 0;
      return;
    }
    if (before * c.Hkv <= begin && begin < (before + mine) * c.Hkv) {
      long long at = before;
      int b = tid * ((c.B + C::kThreads - 1) / C::kThreads), nt;
      while ((at + (nt = seq_tiles(c, a, b))) * c.Hkv <= begin) {
        at += nt;
        ++b;
      }
      const long long rel = begin - at * c.Hkv;
      s_begin[0] = b;
      s_begin[1] = (int)(rel / nt);
      s_begin[2] = (int)(rel % nt);
      JoinInfo j = {};
      j.split = s_begin[2] != 0;
      if (j.split) {
        const long long i0 = begin - s_begin[2];
        j.b = b;
        j.h = s_begin[1];
        j.c0 = (int)(i0 / per);
        j.c1 = (int)((i0 + nt - 1) / per);
        j.slot0 = i0 > j.c0 * per ? 1 : 0;
      }
      info[blockIdx.x] = j;
    }
  } else {
    const int b = (int)blockIdx.x / c.Hkv;
    run = seq_tiles(c, a, b);
    if (run <= 0) return;
    if (tid == 0) {
      s_begin[0] = b;
      s_begin[1] = (int)blockIdx.x - b * c.Hkv;
      s_begin[2] = 0;
    }
  }

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_full[i], 2);  // the copies, and the scales
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1 + C::kSoftWarps);  // the last QK product of a segment, and the softmax warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], C::kSoftWarps);
      mbar_init(&p_full[i], C::kSoftWarps);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(done, 1);
    abort_flag[0] = 0;
    abort_flag[1] = (int)a.limit_us;
    for (int i = 0; i < 3 * C::kGroups; ++i) s_bad_all[i] = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  if (tid == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk(c, a, run, s_begin[0], s_begin[1], s_begin[2]);
  Segment g;

  if (warp == C::kTmaWarp) {
    // ------------------------------------------------------------ TMA: lane = 16 keys of the tile.  It also brings the scales.
    const uint64_t pol = policy_evict_first();
    const int per_log2 = c.page_log2 - 4;  // lanes of one page
    const uint32_t box = (uint32_t)c.page * kHeadDim;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const int32_t* row = c.page_table + (size_t)g.b * c.max_pages;
      // page of this lane's keys in tile i (-1: none), two tiles ahead; its scales, one ahead
      auto page_at = [&](int i) {
        const int j = (g.r.tile0 + i) * kTile + (lane & 7) * 16;
        const bool in = i < g.i1 && j + 15 >= g.r.lo && j < g.r.hi;
        const int p = in ? __ldg(row + (j >> c.page_log2)) : -1;
        if (in && (p < 0 || p >= c.n_pages)) set_status(c.status, DEV_ERR_BOUNDS);
        return p < c.n_pages ? p : -1;
      };
      auto scales_at = [&](int p) {  // key scale | value scale << 8
        if (p < 0) return 127u | 127u << 8;
        const size_t u = (size_t)p * c.Hkv + g.h;
        return (uint32_t)__ldg(c.k_scale + u) | (uint32_t)__ldg(c.v_scale + u) << 8;
      };
      int pg = page_at(g.i0), pg1 = page_at(g.i0 + 1);
      uint32_t sc = scales_at(pg);
#pragma unroll 1
      for (int i = g.i0; i < g.i1; ++i) {
        const int pg2 = page_at(i + 2);
        const uint32_t sc1 = scales_at(pg1);
        const int st = (int)(n % C::kStages);
        const uint32_t ph = (n / C::kStages) & 1u;
        // pages are loaded whole: by the first of a page's lanes that has it (a tile's first page may begin before the keys
        // that are seen, and its first lanes then have none)
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0) & 0xFFu;
        const uint32_t group = ((1u << (1 << per_log2)) - 1u) << ((lane & 7) >> per_log2 << per_log2);
        const bool load = lane < 8 && pg >= 0 && __ffs(have & group) - 1 == lane;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * box;
        uint8_t* dst = smem + st * 2 * kTileBytes + ((lane & 7) >> per_log2) * box;
        const int y = load ? (int)(((long long)pg * c.Hkv + g.h) << c.page_log2) : 0;
        ok = warp_wait(&k_empty[st], ph ^ 1u, abort_flag, c.status) && warp_wait(&v_empty[st], ph ^ 1u, abort_flag, c.status);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&k_full[st], bytes);
          mbar_arrive_expect_tx(&v_full[st], bytes);
        }
        __syncwarp();
        if (load) {
          tma_load_2d(dst, &tm_k, 0, y, &k_full[st], pol);
          if (!a.withhold) tma_load_2d(dst + kTileBytes, &tm_v, 0, y, &v_full[st], pol);
        }
        // the scales, which take longer to come than the copies to be issued: the keys' barrier wants them too
        if (lane < 8) {
          infos[st].kf[lane] = exp2_byte(sc & 255u);
          infos[st].lv[lane] = (float)((int)(sc >> 8) - 127);
          infos[st].un[lane] = ex2((float)(127 - (int)(sc >> 8)));
          if (lane == 0) infos[st].have = have;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[st]);
        ++n;
        pg = pg1;
        pg1 = pg2;
        sc = sc1;
      }
    }
    // Every copy lands before the block ends.
    if (lane == 0) {
      for (int st = 0; st < C::kStages; ++st) {
        const uint32_t fills = n / C::kStages + ((uint32_t)st < n % C::kStages ? 1u : 0u);
        if (!fills) continue;
        mbar_wait_bounded(&k_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
        mbar_wait_bounded(&v_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
      }
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA: scores run one tile ahead of the weighted sums.  The
    // whole warp walks along and one lane issues: descriptors stay in uniform registers.
    const uint32_t id_s = umma_idesc_e4m3(kTile, C::kRows, false, false), id_o = umma_idesc_e4m3(kHeadDim, C::kPRows, true, true);
    const uint64_t desc = umma_desc_sw128(smem_u32(smem));
    const uint64_t pdesc = umma_desc_mn16(smem_u32(smem) + C::kPOff, C::kPBlock);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t n = 0, segs = 0;  // n: tiles whose scores were issued
    uint32_t begins = 0;       // bit m & 1: tile m is its segment's first
    bool ok = true, more = walk.next(g);
    int i = more ? g.i0 : 0;
#pragma unroll 1
    for (long long x = -1; ok && x < run; ++x) {
      if (more) {
        const int st = (int)(n % C::kStages), qb = (int)(segs % C::kQBufs), sb = (int)(n & 1u);
        if (i == g.i0) ok = warp_wait(&q_full[qb], (segs / C::kQBufs) & 1u, abort_flag, c.status);
        ok = ok && warp_wait(&k_full[st], (n / C::kStages) & 1u, abort_flag, c.status) &&
             warp_wait(&s_empty[sb], ((n >> 1) & 1u) ^ 1u, abort_flag, c.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = desc + (uint64_t)((st * 2 * kTileBytes) >> 4);
        const uint64_t bd = desc + (uint64_t)((C::kQOff + qb * C::kQBytes) >> 4);
        begins = (begins & ~(1u << sb)) | (i == g.i0 ? 1u : 0u) << sb;
        const bool ends = ++i == g.i1;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kHeadDim / 32; ++k) umma_e4m3(tm + sb * C::kRows, ad + 2 * k, bd + 2 * k, id_s, k != 0);
          umma_commit(&k_empty[st]);
          umma_commit(&s_full[sb]);
          if (ends) umma_commit(&q_empty[qb]);
        }
        __syncwarp();
        ++n;
        if (ends) {
          ++segs;
          more = walk.next(g);
          i = more ? g.i0 : 0;
        }
      }
      if (x >= 0) {
        const uint32_t m = (uint32_t)x, pb = m & 1u;
        const int st = (int)(m % C::kStages);
        ok = warp_wait(&v_full[st], (m / C::kStages) & 1u, abort_flag, c.status) &&
             warp_wait(&p_full[pb], (m >> 1) & 1u, abort_flag, c.status);
        if (!ok) break;
        tc_fence_after();
        // V[token][dim]: the 128-byte rows are the K index, eight rows (1 KB) to a swizzle atom, 32 tokens an MMA
        const uint64_t ad = desc + (uint64_t)((st * 2 * kTileBytes + kTileBytes) >> 4);
        const uint64_t bd = pdesc + (uint64_t)((pb * C::kPBytes) >> 4);
        const bool adds = !(begins >> pb & 1u);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            umma_e4m3(tm + C::kOCol, ad + (uint64_t)((k * 32 * 128) >> 4), bd + (uint64_t)((k * 32 * 16) >> 4), id_o,
                      k != 0 || adds);
          umma_commit(&v_empty[st]);
          umma_commit(&o_full[pb]);
        }
        __syncwarp();
      }
    }
    // whatever was issued has finished before tensor memory is given back (after an abort too)
    if (elect_one()) umma_commit(done);
    __syncwarp();
    mbar_wait_bounded(done, 0, abort_flag, 1000ull * a.limit_us, c.status, false);
  } else if (warp == C::kQWarp) {
    // ------------------------------------------------------------ queries
    uint32_t n = 0;
    while (walk.next(g)) {
      const int qb = (int)(n % C::kQBufs), rows = g.s.t1 - g.s.t0, cols = min(NC, rows * G);
      constexpr int kAtOnce = 8;  // rows
      uint2 raw[kAtOnce];
      auto load = [&](int x0) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          raw[x] = make_uint2(0, 0);
          if (x0 + x < cols) {
            const int i = (x0 + x) / G;
            raw[x] = __ldg(reinterpret_cast<const uint2*>(a.q + (size_t)(g.s.t0 + i) * a.q_stride +
                                                         (size_t)(g.h * G + x0 + x - i * G) * kHeadDim) + lane);
          }
        }
      };
      load(0);
      if (!warp_wait(&q_empty[qb], ((n / C::kQBufs) & 1u) ^ 1u, abort_flag, c.status)) break;
      uint8_t* op = smem + C::kQOff + qb * C::kQBytes;
#pragma unroll 1
      for (int x0 = 0; x0 < NC; x0 += kAtOnce) {
        if (x0 > 0) load(x0);
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const float v[4] = {bf16_lo(raw[x].x), bf16_hi(raw[x].x), bf16_lo(raw[x].y), bf16_hi(raw[x].y)};
          float top = 0.f;
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = fabsf(v[e]);
            bad |= !(m <= 3.402823466e38f);
            top = fmaxf(top, m);
          }
          top = warp_max(top);
          bad = __any_sync(0xffffffffu, bad);
          const int e = bad ? 0 : query_exponent(top);
          const float inv = exp2_int(-e);
          uint32_t h0, l0, h1, l1;
          split_e4m3x2(v[0] * inv, v[1] * inv, h0, l0);
          split_e4m3x2(v[2] * inv, v[3] * inv, h1, l1);
          uint32_t hi = h0 | (h1 << 16), lo = l0 | (l1 << 16);
          if (bad) hi = lo = 0x7F7F7F7Fu;  // a row with an infinity or NaN has NaN scores
          const uint32_t sw = ((((uint32_t)lane >> 2) ^ (x & 7)) << 4) + (lane & 3) * 4;
          *reinterpret_cast<uint32_t*>(op + (x0 + x) * 128 + sw) = hi;
          *reinterpret_cast<uint32_t*>(op + (NC + x0 + x) * 128 + sw) = lo;
          if (lane == 0) {
            s_qf[qb * NC + x0 + x] = a.scale_log2 * exp2_int(e);
            s_tok[qb * NC + x0 + x] = x0 + x < cols ? (x0 + x) / G : 0;
          }
        }
      }
      if (rows * G > NC && lane == 0) set_status(c.status, DEV_ERR_CONFIG);  // more new tokens than max_q
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
      ++n;
    }
  } else {
    // ------------------------------------------------------------ softmax: thread = key of the tile and output dim
    constexpr int N = C::kCols;
    const int group = warp >> 2, w4 = warp & 3, key = tid & 127, col0 = group * N;
    uint32_t n = 0, segs = 0;
    bool ok = true;
    const uint32_t mine = tmem + ((uint32_t)(w4 * 32) << 16) + col0;  // this thread's lane and columns
    volatile int* s_bad = s_bad_all + 3 * group;
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
    float r[N], l[N];
    while (walk.next(g)) {
      const int qb = (int)(segs % C::kQBufs);
      const float* qf = s_qf + qb * NC + col0;
      const int* tok = s_tok + qb * NC + col0;
      const int first = g.s.first(), rows = g.s.t1 - g.s.t0;
      const int last = a.causal ? first + rows : g.r.hi;         // one past the last visible key of any row
      const int all_lo = window_lo(first + rows - 1, a.window);  // keys [all_lo, all_hi) are seen by
      const int all_hi = a.causal ? first + 1 : g.r.hi;          // every row
#pragma unroll
      for (int x = 0; x < N; ++x) {
        r[x] = -CUDART_INF_F;
        l[x] = 0.f;
      }
      ok = ok && warp_wait(&q_full[qb], (segs / C::kQBufs) & 1u, abort_flag, c.status);
#pragma unroll 1
      for (int i = g.i0; i < g.i1; ++i, ++n) {
        const int j0 = (g.r.tile0 + i) * kTile, j = j0 + key, st = (int)(n % C::kStages);
        // (the keys' barrier is behind the scales; the scores come later)
        ok = ok && warp_wait(&k_full[st], (n / C::kStages) & 1u, abort_flag, c.status);
        const float ks = infos[st].kf[key >> 4], lv = infos[st].lv[key >> 4], un = infos[st].un[key >> 4];
        const bool there = (infos[st].have >> (key >> 4) & 1u) && j < last;
        ok = ok && warp_wait(&s_full[n & 1u], (n >> 1) & 1u, abort_flag, c.status);
        float u[N];
#pragma unroll
        for (int x = 0; x < N; ++x) u[x] = 0.f;
        if (ok) {
          tc_fence_after();
          add_product<N>(mine + (n & 1u) * C::kRows, NC, u);
          tc_fence_before();
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&s_empty[n & 1u]);
        const bool whole = j0 >= all_lo && j0 + kTile <= all_hi;
#pragma unroll
        for (int x = 0; x < N; ++x) u[x] = there ? fmaf(u[x] * ks, qf[x], lv) : -CUDART_INF_F;
        if (!whole) {
#pragma unroll
          for (int x = 0; x < N; ++x) {
            const int pos = first + tok[x];
            if ((a.causal && j > pos) || j < window_lo(pos, a.window)) u[x] = -CUDART_INF_F;
          }
        }
        float* tops = s_max + (n & 1u) * NC * 4 + col0 * 4;
        {
          float v[N];
#pragma unroll
          for (int x = 0; x < N; ++x) v[x] = u[x];
          const int col = columns_max<N>(v, lane);
          if ((lane & (32 / N - 1)) == 0) tops[col * 4 + w4] = v[0];
        }
        if (lane == 0 && !ok) s_bad[n & 1u] = 1;
        group_sync();
        // the warps of a group leave together, so that none waits at the barrier for one that gave up
        if (s_bad[n & 1u]) {
          ok = false;
          break;
        }
        // The references follow the maxima when one of them has grown by more than kSlack (the same for the whole group)
        // (without a branch per column, which would have each of these loads wait for the one before)
        float top[N], f[N];
        bool moved = false;
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const float4 m = *reinterpret_cast<const float4*>(tops + x * 4);
          top[x] = fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w));
          moved |= top[x] > r[x] + kSlack;  // r = -infinity: any finite maximum
        }
        if (moved) {
#pragma unroll
          for (int x = 0; x < N; ++x) {
            top[x] = fmaxf(top[x], r[x]);
            f[x] = top[x] == r[x] ? 1.f : ex2(r[x] - top[x]);
            l[x] *= f[x];
            r[x] = top[x];
          }
        }
        if (moved && i > g.i0) {
          // the sums so far, of which the tile before is the last, to the new reference: this thread's dim of its columns
          ok = ok && warp_wait(&o_full[(n - 1u) & 1u], ((n - 1u) >> 1) & 1u, abort_flag, c.status);
          if (ok) {
            tc_fence_after();
            scale_columns<N>(mine + C::kOCol, NC, f);
            scale_columns<N>(mine + C::kOCol + 2 * NC, NC, f);
            tc_fence_before();
          }
        }
        // 16 columns to a block of 16 bytes a key: the hi parts of all columns, then the lo parts, then both of small weights.  (The
        // product that read these bytes two tiles ago was issued before this tile's scores, so it has finished.)
        uint8_t* pw = smem + C::kPOff + (n & 1u) * C::kPBytes + key * 16;
        auto put = [&](int col, uint32_t v) { *reinterpret_cast<uint32_t*>(pw + col / 16 * C::kPBlock + col % 16) = v; };
#pragma unroll
        for (int x = 0; x < N; x += 4) {
          float p[4];
          uint32_t small = 0;  // a byte of ones where the weight is
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float z = u[x + y] - (r[x + y] == -CUDART_INF_F ? 0.f : r[x + y]) + kBase;
            p[y] = ex2(z);
            l[x + y] = fmaf(p[y], un, l[x + y]);
            const bool is_small = z < kSmall;  // not a NaN
            p[y] *= is_small ? 1.f / kSmallDown : 1.f;
            small |= is_small ? 0xFFu << (8 * y) : 0u;
          }
          uint32_t h0, l0, h1, l1;
          split_weights(p[0], p[1], h0, l0);
          split_weights(p[2], p[3], h1, l1);
          const uint32_t hi = h0 | h1 << 16, lo = l0 | l1 << 16;
          const int at = col0 + x;
          put(at, hi & ~small);
          put(NC + at, lo & ~small);
          put(2 * NC + at, hi & small);
          put(3 * NC + at, lo & small);
        }
        // A key that no row sees has weight 0, but its value bytes may be anything: 0 * NaN.  They become zeros.
        const bool gone = !there || j < g.r.lo;
        if (group == 0 && ok && __any_sync(0xffffffffu, gone)) {
          ok = warp_wait(&v_full[st], (n / C::kStages) & 1u, abort_flag, c.status);
          if (ok && gone) {
            uint4* vr = reinterpret_cast<uint4*>(smem + st * 2 * kTileBytes + kTileBytes + key * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) vr[x] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&p_full[n & 1u]);
      }
      if (ok) ok = warp_wait(&o_full[(n - 1u) & 1u], ((n - 1u) >> 1) & 1u, abort_flag, c.status);
      float acc[N];
#pragma unroll
      for (int x = 0; x < N; ++x) acc[x] = 0.f;
      if (ok) {
        tc_fence_after();
        add_parts<N>(mine + C::kOCol, NC, acc);
        tc_fence_before();
      }
      // the denominators: over the warp, then over the group
      float* sums = s_max + 2 * NC * 4 + col0 * 4;
#pragma unroll
      for (int x = 0; x < N; ++x) {
        float t = l[x];
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) sums[x * 4 + w4] = t;
      }
      if (lane == 0) {
        if (!ok) s_bad[2] = 1;
        else mbar_arrive(&q_empty[qb]);
      }
      group_sync();
      if (s_bad[2]) break;
      const bool complete = g.i0 == 0 && g.i1 == g.r.nt;
      const int slot = slot0 + (g.i0 == 0 && segs > 0 ? 1 : 0);
      const int cols = min(NC, rows * G);
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const float4 m = *reinterpret_cast<const float4*>(sums + x * 4);
        const float sum = (m.x + m.y) + (m.z + m.w);
        const int col = col0 + x;
        if (col < cols) {
          if (complete) {
            const int i = col / G;
            a.out[((size_t)(g.s.t0 + i) * c.Hq + g.h * G + col - i * G) * kHeadDim + key] =
                f32_to_bf16_rne(sum != 0.f ? acc[x] / sum : 0.f);
          } else {
            part_o[((size_t)slot * NC + col) * kHeadDim + key] = acc[x];
            if (key == 0) part_rl[(size_t)slot * NC + col] = make_float2(r[x], sum);
          }
        }
      }
      ++segs;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

int width_of(int cols) { return cols <= 8 ? 8 : 16; }

int blocks_of(int n_sms) { return 2 * n_sms; }

template <int NC>
cudaError_t launch(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream) {
  using C = Cfg<NC>;
  CUtensorMap tk, tv;
  if (!make_cache_map(&tk, c.k_codes, c) || !make_cache_map(&tv, c.v_codes, c)) return cudaErrorInvalidValue;
  auto kern = attention_decode_kernel<NC>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kBytes, allowed);
  if (e != cudaSuccess) return e;
  // Rows of a few tiles at most (the table's width bounds them) are one block's each: nothing to join.
  const bool split = (long long)c.max_pages * c.page > kWholeTiles * kTile;
  const int blocks = split ? blocks_of(n_sms) : c.B * c.Hkv;
  float* part_o = reinterpret_cast<float*>(a.scratch);
  float2* part_rl = reinterpret_cast<float2*>(part_o + (size_t)2 * blocks_of(n_sms) * NC * kHeadDim);
  JoinInfo* info = reinterpret_cast<JoinInfo*>(part_rl + (size_t)2 * blocks_of(n_sms) * NC);
  e = launch_kernel(kern, dim3(blocks), dim3(C::kThreads), C::kBytes, stream, false, tk, tv, c, a, (int)split, part_o, part_rl,
                    info);
  if (e != cudaSuccess || !split) return e;
  return launch_attention_join(c, a, blocks, NC, part_o, part_rl, info, stream);
}

}  // namespace

bool attention_decode_fits(int G, int max_q) { return (long long)G * max_q <= 16; }

size_t attention_decode_scratch(int G, int max_q, int n_sms) {
  const int nc = width_of(G * max_q);
  return blocks_of(n_sms) * ((size_t)2 * nc * (kHeadDim * sizeof(float) + sizeof(float2)) + sizeof(JoinInfo));
}

cudaError_t launch_attention_decode(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream) {
  return width_of(c.Hq / c.Hkv * a.max_q) == 8 ? launch<8>(c, a, n_sms, stream) : launch<16>(c, a, n_sms, stream);
}

}  // namespace moe
