// Accumulated attention weights: what the new queries of a sequence give to each of its cached keys.
//
// For one key/value head and key j, over the rows (new tokens x grouped heads) that see it,
//   w[j] = w_before[j] + sum_rows 2^(scale * log2(e) * q . k_j - lse2),     lse2 = lse * log2(e)
// with the logarithm lse of a row's denominator as the attention left it: no maximum, no second pass, and a key's sum is its own.
// So the keys are the M operand, as in the decode kernel: a tile of 128 of them, E4M3 as cached, times NC rows,
//   S^T[128 keys, NC] = K . q_hi^T + K . q_lo^T       tcgen05 kind::f8f6f4, queries in two E4M3 halves
// and a softmax thread owns a key: it adds up its lane of S^T, and nothing crosses threads.  Neither values nor joins are needed.
//
// Rows beyond NC are taken in chunks: a block keeps kStages tiles of keys in shared memory and walks the chunks over them, so that a
// chunk's conversion to E4M3 serves that many tiles.
//
// Work: all (sequence, head, tile) in one order, a tile costing its sequence's chunks, cut into equal runs, one per block (two blocks
// per SM).  The sums of a key are one thread's in a fixed order: the same inputs give the same bits.
//
// What bounds it: few rows, the bytes of the keys; many, exponentials (32 a cycle and SM) and the products, which take the same
// 256 cycles for a tile and 64 rows.
//
// Warps: 8 softmax (four for the even tiles of a group, four for the odd), TMA, MMA, then queries.  Every wait is bounded (2 s).
#include "attention_tiles.cuh"

namespace moe {
namespace {

struct TileInfo {    // per 16 keys of a tile
  float kf[8];       // 2^e_k
  int page[8];       // -1: none
};

struct RowInfo {     // a query row: its score is S * qf, its weight 2^(S qf kf - lse2)
  float qf, lse2;
};

template <int NC>
struct Cfg {
  static constexpr bool kWide = NC > 16;                    // hi and lo products in the same columns (else side by side: half
                                                            // the instructions, which small ones are bound by)
  static constexpr int kStages = kWide ? 4 : 6;             // tiles of keys
  static constexpr int kQBufs = 2;
  static constexpr int kQWarps = kWide ? 4 : 1;
  static constexpr int kSoftWarps = 8;
  static constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kQWarp = kSoftWarps + 2;
  static constexpr int kThreads = 32 * (kQWarp + kQWarps);
  static constexpr int kQBytes = 2 * NC * 128;
  static constexpr int kQOff = kStages * kTileBytes;
  static constexpr int kBarOff = kQOff + kQBufs * kQBytes;
  static constexpr int kNumBars = 3 * kStages + 2 * kQBufs + 5;
  static constexpr int kInfoOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;           // TileInfo [kStages]
  static constexpr int kRowOff = kInfoOff + kStages * (int)sizeof(TileInfo);         // RowInfo [kQBufs][NC]
  static constexpr int kPosOff = kRowOff + kQBufs * NC * (int)sizeof(RowInfo);       // int [kQBufs][NC]
  static constexpr int kAccOff = kPosOff + kQBufs * NC * 4;                          // float [kStages][128]
  static constexpr int kMiscOff = kAccOff + (kWide ? kStages * kTile * 4 : 0);
  static constexpr int kBytes = 1024 + kMiscOff + 32;
  static constexpr int kSCols = kWide ? NC : 2 * NC;
  static constexpr int kTmemCols = 2 * kSCols;              // a power of two, at least 32
  static_assert(2 * (kBytes + 1024) <= 228 * 1024, "shared memory");
  static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
};

// Tiles [i0, i1) of one (sequence, head), and the chunks of its rows.
struct Segment {
  int b, h, i0, i1, chunks;
  SeqRange s;
  KeyRange r;
};

__device__ __forceinline__ int row_chunks(const SeqRange& s, int G, int nc) {
  return (int)(((long long)(s.t1 - s.t0) * G + nc - 1) / nc);
}

template <int NC>
__device__ __forceinline__ long long seq_cost(const KvBatch& c, const AttentionArgs& a, int G, int b) {
  SeqRange s;
  if (!load_seq(c, b, s)) return 0;
  return (long long)key_range(s, a).nt * row_chunks(s, G, NC);
}

// Walks the segments of a block's run: the tiles whose cost begins within it.
template <int NC>
struct Walk {
  const KvBatch& c;
  const AttentionArgs& a;
  int G;
  long long at, left;  // where the run begins in the present (sequence, head); how much of it is left
  int b, h;
  __device__ Walk(const KvBatch& c_, const AttentionArgs& a_, int G_, long long n, int b_, int h_, long long at_)
      : c(c_), a(a_), G(G_), at(at_), left(n), b(b_), h(h_) {}
  __device__ bool next(Segment& g) {
    while (left > 0 && b < c.B) {
      const bool ok = load_seq(c, b, g.s);
      g.r = key_range(g.s, a);
      if (!ok || g.r.nt == 0) {
        ++b;
        h = 0;
        at = 0;
        continue;
      }
      g.b = b;
      g.h = h;
      g.chunks = row_chunks(g.s, G, NC);
      const long long cost = (long long)g.r.nt * g.chunks;
      g.i0 = (int)((at + g.chunks - 1) / g.chunks);
      g.i1 = (int)min((long long)g.r.nt, (at + left + g.chunks - 1) / g.chunks);
      left -= cost - at;
      at = 0;
      if (++h == c.Hkv) {
        h = 0;
        ++b;
      }
      if (g.i0 < g.i1) return true;
    }
    return false;
  }
};

// The chunks with a row that sees a key of [j0, j1): c0 .. c1, one at least (the keys' sums are written all the same).
__device__ __forceinline__ void chunks_of(const Segment& g, const AttentionArgs& a, int G, int nc, int j0, int j1, int& c0, int& c1) {
  c0 = 0;
  c1 = g.chunks - 1;
  if (g.chunks == 1) return;
  const int first = g.s.first(), last = g.s.t1 - g.s.t0 - 1;  // rows i of positions first + i
  if (a.causal) c0 = (int)((long long)min(max(0, j0 - first), last) * G / nc);
  if (a.window > 0) {
    // row i sees keys from first + i - window + 1 on: the last row that sees j1 - 1
    const long long i = (long long)j1 - 1 - first + a.window - 1;
    c1 = (int)(((i < 0 ? 0 : i > last ? last : i) * G + G - 1) / nc);
    c1 = max(c0, min(c1, g.chunks - 1));
  }
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, 2)
    kv_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const KvBatch c, const AttentionArgs a, const float* lse,
                      const float* weight_in, float* weight_out) {
  using C = Cfg<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* k_empty = k_full + C::kStages;
  uint64_t* i_full = k_empty + C::kStages;
  uint64_t* q_full = i_full + C::kStages;
  uint64_t* q_empty = q_full + C::kQBufs;
  uint64_t* s_full = q_empty + C::kQBufs;   // [2]
  uint64_t* s_empty = s_full + 2;           // [2]
  uint64_t* done = s_empty + 2;
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  RowInfo* s_row = reinterpret_cast<RowInfo*>(smem + C::kRowOff);
  int* s_pos = reinterpret_cast<int*>(smem + C::kPosOff);
  float* s_acc = reinterpret_cast<float*>(smem + C::kAccOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_begin = reinterpret_cast<int*>(smem + C::kMiscOff + 12);  // b, h
  long long* s_at = reinterpret_cast<long long*>(smem + C::kMiscOff + 24);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv;
  if (blockIdx.x == 0 && tid == C::kThreads - 1) check_starts(c);

  // ---- this block's run
  long long run;
  {
    auto cost = [&](int b) { return seq_cost<NC>(c, a, G, b); };
    long long mine, total;
    long long* s_warp = reinterpret_cast<long long*>(s_row);  // free until the roles start
    const long long before = scan_batch(c, C::kThreads, s_warp, mine, total, cost);
    const long long all = total * c.Hkv, per = max(1LL, (all + gridDim.x - 1) / (long long)gridDim.x);
    const long long begin = (long long)blockIdx.x * per;
    run = min(per, all - begin);
    if (run <= 0) return;
    if (before * c.Hkv <= begin && begin < (before + mine) * c.Hkv) {
      long long at = before, u;
      int b = tid * ((c.B + C::kThreads - 1) / C::kThreads);
      while ((at + (u = cost(b))) * c.Hkv <= begin) {
        at += u;
        ++b;
      }
      const long long rel = begin - at * c.Hkv;
      s_begin[0] = b;
      s_begin[1] = (int)(rel / u);
      *s_at = rel % u;
    }
  }

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1 + 4);  // the tile's last product, and the softmax warps that have its scales
      mbar_init(&i_full[i], 1);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&q_full[i], C::kQWarps);
      mbar_init(&q_empty[i], 1 + C::kSoftWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(done, 1);
    abort_flag[0] = 0;
    abort_flag[1] = (int)a.limit_us;
    tma_prefetch_desc(&tm_k);
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk<NC> walk(c, a, G, run, s_begin[0], s_begin[1], *s_at);
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
      // page of this lane's keys in tile i (-1: none), two tiles ahead; its scale, one ahead
      auto page_at = [&](int i) {
        const int j = (g.r.tile0 + i) * kTile + (lane & 7) * 16;
        const bool in = i < g.i1 && j + 15 >= g.r.lo && j < g.r.hi;
        const int p = in ? __ldg(row + (j >> c.page_log2)) : -1;
        if (in && (p < 0 || p >= c.n_pages)) set_status(c.status, DEV_ERR_BOUNDS);
        return p < c.n_pages ? p : -1;
      };
      auto scale_at = [&](int p) { return p < 0 ? 127u : (uint32_t)__ldg(c.k_scale + (size_t)p * c.Hkv + g.h); };
      int pg = page_at(g.i0), pg1 = page_at(g.i0 + 1);
      uint32_t sc = scale_at(pg);
#pragma unroll 1
      for (int i = g.i0; i < g.i1; ++i) {
        const int pg2 = page_at(i + 2);
        const uint32_t sc1 = scale_at(pg1);
        const int st = (int)(n % C::kStages);
        // pages are loaded whole, by the first of a page's lanes that has it
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0) & 0xFFu;
        const uint32_t group = ((1u << (1 << per_log2)) - 1u) << ((lane & 7) >> per_log2 << per_log2);
        const bool load = lane < 8 && pg >= 0 && __ffs(have & group) - 1 == lane;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * box;
        uint8_t* dst = smem + st * kTileBytes + ((lane & 7) >> per_log2) * box;
        const int y = load ? (int)(((long long)pg * c.Hkv + g.h) << c.page_log2) : 0;
        ok = warp_wait(&k_empty[st], ((n / C::kStages) & 1u) ^ 1u, abort_flag, c.status);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], bytes);
        __syncwarp();
        if (load && !a.withhold) tma_load_2d(dst, &tm_k, 0, y, &k_full[st], pol);
        if (lane < 8) {
          infos[st].kf[lane] = exp2_byte(sc);
          infos[st].page[lane] = pg;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_full[st]);
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
        if (fills) mbar_wait_bounded(&k_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
      }
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA: the whole warp walks along and one lane issues
    const uint32_t idesc = umma_idesc_e4m3(kTile, C::kSCols, false, false);
    const uint64_t desc = umma_desc_sw128(smem_u32(smem));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t n = 0, fills = 0, used[2] = {0, 0};  // tiles of earlier groups; query buffers; uses of the score buffers
    bool ok = true;
    while (ok && walk.next(g)) {
      if (g.chunks == 1) {
        ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
        ++fills;
      }
#pragma unroll 1
      for (int i = g.i0; ok && i < g.i1; i += C::kStages) {
        const int nt = min(C::kStages, g.i1 - i), j0 = (g.r.tile0 + i) * kTile;
        int c0, c1;
        chunks_of(g, a, G, NC, j0, j0 + nt * kTile, c0, c1);
#pragma unroll 1
        for (int ch = c0; ok && ch <= c1; ++ch) {
          if (g.chunks > 1) {
            ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
            ++fills;
          }
          const int qb = (int)((fills - 1u) % C::kQBufs);
          const uint64_t bd = desc + (uint64_t)((C::kQOff + qb * C::kQBytes) >> 4);
          const bool q_ends = g.chunks > 1 || i + nt == g.i1;
#pragma unroll 1
          for (int t = 0; ok && t < nt; ++t) {
            const uint32_t m = n + t;
            const int st = (int)(m % C::kStages), sb = t & 1;
            ok = warp_wait2(&k_full[st], (m / C::kStages) & 1u, &s_empty[sb], (used[sb] & 1u) ^ 1u, abort_flag, c.status);
            if (!ok) break;
            ++used[sb];
            tc_fence_after();
            const uint64_t ad = desc + (uint64_t)((st * kTileBytes) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kHeadDim / 32; ++k) umma_e4m3(tm + sb * C::kSCols, ad + 2 * k, bd + 2 * k, idesc, k != 0);
              if (C::kWide) {
#pragma unroll
                for (int k = 0; k < kHeadDim / 32; ++k)
                  umma_e4m3(tm + sb * C::kSCols, ad + 2 * k, bd + (uint64_t)((NC * 128) >> 4) + 2 * k, idesc, 1);
              }
              umma_commit(&s_full[sb]);
              if (ch == c1) umma_commit(&k_empty[st]);
              if (q_ends && t == nt - 1) umma_commit(&q_empty[qb]);
            }
            __syncwarp();
          }
        }
        n += nt;
      }
    }
    // whatever was issued has finished before tensor memory is given back (after an abort too)
    if (elect_one()) umma_commit(done);
    __syncwarp();
    mbar_wait_bounded(done, 0, abort_flag, 1000ull * a.limit_us, c.status, false);
  } else if (warp >= C::kQWarp) {
    // ------------------------------------------------------------ queries: each warp a part of the chunk's rows
    constexpr int kMine = NC / C::kQWarps, kAtOnce = 8;
    const int x_first = (warp - C::kQWarp) * kMine;
    uint32_t fills = 0;
    bool ok = true;
    auto fill = [&](int ch) {
      const int qb = (int)(fills % C::kQBufs), first = g.s.first();
      const long long rows = (long long)(g.s.t1 - g.s.t0) * G;
      uint8_t* op = smem + C::kQOff + qb * C::kQBytes;
#pragma unroll 1
      for (int x0 = x_first; x0 < x_first + kMine; x0 += kAtOnce) {
        uint2 raw[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const long long rho = (long long)ch * NC + x0 + x;
          raw[x] = make_uint2(0, 0);
          if (rho < rows) {
            const int i = (int)(rho / G), head = g.h * G + (int)(rho - (long long)i * G);
            raw[x] = __ldg(reinterpret_cast<const uint2*>(a.q + (size_t)(g.s.t0 + i) * a.q_stride + (size_t)head * kHeadDim) + lane);
          }
        }
        // lane x has the row x's denominator
        float row_lse = CUDART_INF_F;
        int pos = 0;
        if (lane < kAtOnce) {
          const long long rho = (long long)ch * NC + x0 + lane;
          if (rho < rows) {
            const int i = (int)(rho / G), head = g.h * G + (int)(rho - (long long)i * G);
            const float v = __ldg(lse + (size_t)(g.s.t0 + i) * c.Hq + head) * 1.44269504088896341f;
            if (fabsf(v) <= 3.402823466e38f) row_lse = v;  // a row that saw nothing, or whose denominator is no number, gives nothing
            pos = first + i;
          }
        }
        if (x0 == x_first) {
          ok = warp_wait(&q_empty[qb], ((fills / C::kQBufs) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) return;
        }
        float qf = 0.f;
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
          const uint32_t hi = bad ? 0u : h0 | (h1 << 16), lo = bad ? 0u : l0 | (l1 << 16);
          const uint32_t sw = ((((uint32_t)lane >> 2) ^ (x & 7)) << 4) + (lane & 3) * 4;
          *reinterpret_cast<uint32_t*>(op + (x0 + x) * 128 + sw) = hi;
          *reinterpret_cast<uint32_t*>(op + (NC + x0 + x) * 128 + sw) = lo;
          if (lane == x) {
            qf = a.scale_log2 * exp2_int(e);
            if (bad) row_lse = CUDART_INF_F;  // a row with an infinity or NaN has no weights
          }
        }
        if (lane < kAtOnce) {
          s_row[qb * NC + x0 + lane] = {qf, row_lse};
          s_pos[qb * NC + x0 + lane] = pos;
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
      ++fills;
    };
    while (ok && walk.next(g)) {
      if (g.chunks == 1) {
        fill(0);
        continue;
      }
#pragma unroll 1
      for (int i = g.i0; ok && i < g.i1; i += C::kStages) {
        const int nt = min(C::kStages, g.i1 - i), j0 = (g.r.tile0 + i) * kTile;
        int c0, c1;
        chunks_of(g, a, G, NC, j0, j0 + nt * kTile, c0, c1);
#pragma unroll 1
        for (int ch = c0; ok && ch <= c1; ++ch) fill(ch);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax: thread = key; a group of four warps has every other tile
    const int group = warp >> 2, w4 = warp & 3, key = tid & 127;
    const uint32_t mine = tmem + ((uint32_t)(w4 * 32) << 16) + group * C::kSCols;
    uint32_t n = 0, fills = 0, used = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const int first = g.s.first();
      const long long rows = (long long)(g.s.t1 - g.s.t0) * G;
      if (g.chunks == 1) {
        ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
        ++fills;
      }
#pragma unroll 1
      for (int i = g.i0; ok && i < g.i1; i += C::kStages) {
        const int nt = min(C::kStages, g.i1 - i), jg = (g.r.tile0 + i) * kTile;
        int c0, c1;
        chunks_of(g, a, G, NC, jg, jg + nt * kTile, c0, c1);
#pragma unroll 1
        for (int ch = c0; ok && ch <= c1; ++ch) {
          if (g.chunks > 1) {
            ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
            if (!ok) break;
            ++fills;
          }
          const int qb = (int)((fills - 1u) % C::kQBufs);
          const RowInfo* row = s_row + qb * NC;
          const int* pos = s_pos + qb * NC;
          const int pos_lo = first + (int)((long long)ch * NC / G);  // positions of the chunk's rows
          const int pos_hi = first + (int)(min(rows, (long long)(ch + 1) * NC) - 1) / G;
#pragma unroll 1
          for (int t = group; t < nt; t += 2) {
            const uint32_t m = n + t;
            const int st = (int)(m % C::kStages), j0 = jg + t * kTile, j = j0 + key;
            ok = warp_wait(&i_full[st], (m / C::kStages) & 1u, abort_flag, c.status);
            if (!ok) break;
            const float ks = infos[st].kf[key >> 4];
            const int pg = infos[st].page[key >> 4];
            float acc = C::kWide && ch > c0 ? s_acc[st * kTile + key] : 0.f;
            // the key's weight so far, on its way while the scores are waited for
            const bool ends = ch == c1, writes = ends && pg >= 0 && j >= g.r.lo && j < g.r.hi;
            const size_t at = writes ? ((((size_t)pg * c.Hkv + g.h) << c.page_log2) + (j & (c.page - 1))) : 0;
            float before = 0.f;
            if (writes && weight_in && j < first) before = weight_in[at];
            if (ends) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&k_empty[st]);
            }
            ok = warp_wait(&s_full[group], used & 1u, abort_flag, c.status);
            if (!ok) break;
            ++used;
            tc_fence_after();
            const bool whole = (!a.causal || j0 + kTile - 1 <= pos_lo) && j0 >= window_lo(pos_hi, a.window);
            constexpr int P = C::kWide ? 32 : 8;  // columns at a time
#pragma unroll
            for (int x0 = 0; x0 < NC; x0 += P) {
              float s[P];
              if constexpr (C::kWide) {
                uint32_t v[32];
                tmem_ld32_async(mine + x0, v);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < P; ++x) s[x] = __uint_as_float(v[x]);
              } else {
                uint32_t v[8], w[8];
                tmem_ld_async(mine + x0, v);
                tmem_ld_async(mine + NC + x0, w);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < P; ++x) s[x] = __uint_as_float(v[x]) + __uint_as_float(w[x]);
              }
              if (x0 + P == NC) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[group]);
              }
              const uint64_t ks2 = f32x2(ks, ks);
              uint64_t sum = 0;
#pragma unroll
              for (int x = 0; x < P; x += 2) {
                const float4 r = *reinterpret_cast<const float4*>(row + x0 + x);  // qf, lse2 of two rows
                float z0, z1;
                uint64_t u;
                asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(u) : "l"(f32x2(s[x], s[x + 1])), "l"(ks2));
                f32x2_split(fma_f32x2(u, f32x2(r.x, r.z), f32x2(-r.y, -r.w)), z0, z1);
                if (!whole) {
                  const int2 ps = *reinterpret_cast<const int2*>(pos + x0 + x);
                  if ((a.causal && j > ps.x) || j < window_lo(ps.x, a.window)) z0 = -CUDART_INF_F;
                  if ((a.causal && j > ps.y) || j < window_lo(ps.y, a.window)) z1 = -CUDART_INF_F;
                }
                sum = add_f32x2(sum, f32x2(ex2(z0), ex2(z1)));
              }
              float s0, s1;
              f32x2_split(sum, s0, s1);
              acc += s0 + s1;
            }
            if (!ends) {
              if (C::kWide) s_acc[st * kTile + key] = acc;
            } else if (writes) {
              weight_out[at] = before + (acc == acc ? acc : 0.f);  // a key that is no number has no weight
            }
          }
          if (ok && (g.chunks > 1 || i + nt == g.i1)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_empty[qb]);
          }
        }
        n += nt;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int NC>
cudaError_t launch(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out, int n_sms,
                   cudaStream_t stream) {
  using C = Cfg<NC>;
  CUtensorMap tk;
  if (!make_cache_map(&tk, c.k_codes, c)) return cudaErrorInvalidValue;
  auto kern = kv_weights_kernel<NC>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(2 * n_sms), dim3(C::kThreads), C::kBytes, stream, false, tk, c, a, lse, weight_in, weight_out);
}

}  // namespace

cudaError_t launch_kv_weights_rows(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                                   int n_sms, cudaStream_t stream) {
  const long long rows = (long long)(c.Hq / c.Hkv) * a.max_q;
  if (rows <= 8) return launch<8>(c, a, lse, weight_in, weight_out, n_sms, stream);
  if (rows <= 16) return launch<16>(c, a, lse, weight_in, weight_out, n_sms, stream);
  return launch<64>(c, a, lse, weight_in, weight_out, n_sms, stream);
}

}  // namespace moe
