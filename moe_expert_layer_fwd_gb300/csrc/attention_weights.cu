// Accumulated attention weights: what the new queries of a sequence give to each of its cached keys.
//
// For one key/value head and key j, over the rows (new tokens x grouped heads) that see it,
//   w[j] = w_before[j] + sum_rows 2^(scale * log2(e) * q . k_j - lse2),     lse2 = lse * log2(e)
// with the logarithm lse of a row's denominator as the attention left it: no maximum, no second pass, and a key's sum is its own.
// So the keys are the M operand, as in the decode kernel: a tile of 128 of them, E4M3 as cached, times NC rows,
//   S^T[128 keys, NC] = K . q_hi^T + K . q_lo^T       tcgen05 kind::f8f6f4, queries in two E4M3 halves
// and a softmax thread owns a key: it adds up its lane of S^T, and nothing crosses threads.  Neither values nor joins are needed.
//
// Rows beyond NC (a sequence with more than the most that was said) are taken in chunks: a block keeps kStages tiles of keys in shared
// memory and walks the chunks over them.  More than 16 rows as a rule: the kernel for many rows.
//
// Work: all (sequence, head, tile) in one order, a tile costing its sequence's chunks, cut into equal runs, one per block (two blocks per
// SM).  The sums of a key are one thread's in a fixed order: the same inputs give the same bits.
//
// The bytes of the keys bound it: 64 sequences of 1500-8190 tokens, 8 key/value heads, 317 MB of keys, take 61 us (54 at the memory's copy
// rate), of which 6 are the way to the first scores (lengths, page table, scales, copies, one after another).
//
// Warps: 8 softmax (two groups of four, which take the tiles in turn), TMA, MMA, queries.  Every wait is bounded (2 s).
#include "attention_weights.cuh"

namespace moe {
namespace {

struct TileInfo {    // per 16 keys of a tile
  float kf[8];       // 2^e_k
  int page[8];       // -1: none
};

struct RowPair {     // two query rows: a weight is 2^(S kf qf + minus)
  float qf[2], minus[2];  // minus = -lse2
};

template <int NC>
struct Cfg {
  static constexpr int kPerSm = 2;                          // blocks
  static constexpr int kStages = 6;                         // tiles of keys
  static constexpr int kGroups = 2, kSBufs = 2 * kGroups;   // groups of four softmax warps, and buffers of scores
  static constexpr int kQBufs = 2;
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kQWarp = kSoftWarps + 2;
  static constexpr int kThreads = 32 * (kQWarp + 1);
  static constexpr int kQBytes = 2 * NC * 128;
  static constexpr int kQOff = kStages * kTileBytes;
  static constexpr int kBarOff = kQOff + kQBufs * kQBytes;
  static constexpr int kNumBars = 3 * kStages + 2 * kQBufs + 2 * kSBufs + 1;
  static constexpr int kInfoOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;           // TileInfo [kStages]
  static constexpr int kRowOff = kInfoOff + kStages * (int)sizeof(TileInfo);         // RowPair [kQBufs][NC / 2]
  static constexpr int kSeenOff = kRowOff + kQBufs * NC / 2 * (int)sizeof(RowPair);  // RowSeen [kQBufs][NC]
  static constexpr int kAllOff = kSeenOff + kQBufs * NC * (int)sizeof(RowSeen);      // int2 [kQBufs]
  static constexpr int kAccOff = kAllOff + kQBufs * (int)sizeof(int2);               // float [kStages][128]
  static constexpr int kMiscOff = kAccOff + kStages * kTile * 4;
  static constexpr int kBytes = 1024 + kMiscOff + 32;
  static constexpr int kSCols = 2 * NC;                     // hi and lo products side by side: half the instructions of sums in
                                                            // one column
  static constexpr int kTmemCols = kSBufs * kSCols;         // a power of two, at least 32
  static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory");
  static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
};

// A key's weights of a chunk's rows, from its lane of tensor memory, those left out that are not finite (a key with a NaN, a denominator
// far below its scores: as in the kernel for many rows); frees the scores once they are in registers.
template <int NC, bool kMasked>
__device__ __forceinline__ float add_weights(uint32_t taddr, const RowPair* row, const RowSeen* seen, float ks, int j, uint64_t* s_empty,
                                             int lane) {
  constexpr int P = 8, kSteps = NC / P;  // columns at a time: the next ones come while these are added up
  const uint64_t ks2 = f32x2(ks, ks);
  uint64_t sum = 0;
  uint32_t v[2][P], w[2][P];
  tmem_ld_async(taddr, v[0]);
  tmem_ld_async(taddr + NC, w[0]);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    tmem_wait_ld();
    if (k + 1 < kSteps) {
      tmem_ld_async(taddr + (k + 1) * P, v[(k + 1) & 1]);
      tmem_ld_async(taddr + NC + (k + 1) * P, w[(k + 1) & 1]);
    } else {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_empty);
    }
    float s[P];
#pragma unroll
    for (int x = 0; x < P; ++x) s[x] = __uint_as_float(v[k & 1][x]) + __uint_as_float(w[k & 1][x]);
#pragma unroll
    for (int x = 0; x < P; x += 2) {
      const float4 r = *reinterpret_cast<const float4*>(row + (k * P + x) / 2);
      float z0, z1;
      f32x2_split(fma_f32x2(mul_f32x2(f32x2(s[x], s[x + 1]), ks2), f32x2(r.x, r.y), f32x2(r.z, r.w)), z0, z1);
      if (kMasked) {
        const int4 see = *reinterpret_cast<const int4*>(seen + k * P + x);
        if ((unsigned)(j - see.x) > (unsigned)see.y) z0 = -CUDART_INF_F;
        if ((unsigned)(j - see.z) > (unsigned)see.w) z1 = -CUDART_INF_F;
      }
      const float p0 = ex2(z0), p1 = ex2(z1);
      sum = add_f32x2(sum, f32x2(p0 < CUDART_INF_F ? p0 : 0.f, p1 < CUDART_INF_F ? p1 : 0.f));
    }
  }
  float s0, s1;
  f32x2_split(sum, s0, s1);
  return s0 + s1;
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, Cfg<NC>::kPerSm)
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
  uint64_t* s_full = q_empty + C::kQBufs;   // [kSBufs]: a group's in turn
  uint64_t* s_empty = s_full + C::kSBufs;   // [kSBufs]
  uint64_t* done = s_empty + C::kSBufs;
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  RowPair* s_row = reinterpret_cast<RowPair*>(smem + C::kRowOff);
  int2* s_all = reinterpret_cast<int2*>(smem + C::kAllOff);  // keys [x, y) are seen by every row of the chunk
  RowSeen* s_seen = reinterpret_cast<RowSeen*>(smem + C::kSeenOff);
  float* s_acc = reinterpret_cast<float*>(smem + C::kAccOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_begin = reinterpret_cast<int*>(smem + C::kMiscOff + 12);  // b, h
  long long* s_at = reinterpret_cast<long long*>(smem + C::kMiscOff + 24);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv;
  if (blockIdx.x == 0 && tid == C::kThreads - 1) check_starts(c);

  long long run;
  if (!weight_run<NC>(c, a, G, C::kThreads, reinterpret_cast<long long*>(s_row), run, s_begin, s_at)) return;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1 + 4);  // the tile's last product, and the softmax warps that have its scales
      mbar_init(&i_full[i], 1);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1 + C::kSoftWarps);
    }
    for (int i = 0; i < C::kSBufs; ++i) {
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
  WeightWalk<NC> walk(c, a, G, run, s_begin[0], s_begin[1], *s_at);
  WeightSegment g;

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
    // ------------------------------------------------------------ MMA: the whole warp walks along and one lane issues;
    // bounds by shuffle, so that loops and descriptors are the warp's and not a lane's
    const uint32_t idesc = umma_idesc_e4m3(kTile, C::kSCols, false, false);
    const uint64_t desc = umma_desc_sw128(smem_u32(smem));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t n = 0, fills = 0, used[2] = {0, 0};  // tiles of earlier groups; query buffers; tiles given to a group of warps
    bool ok = true;
    while (ok && walk.next(g)) {
      const int i0 = __shfl_sync(0xffffffffu, g.i0, 0), i1 = __shfl_sync(0xffffffffu, g.i1, 0), chunks = __shfl_sync(0xffffffffu, g.chunks, 0);
      if (chunks == 1) {
        ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
        ++fills;
      }
#pragma unroll 1
      for (int i = i0; ok && i < i1; i += C::kStages) {
        const int nt = min(C::kStages, i1 - i), j0 = (g.r.tile0 + i) * kTile;
        int c0, c1;
        chunks_of(g, a, G, NC, j0, j0 + nt * kTile, c0, c1);
        c0 = __shfl_sync(0xffffffffu, c0, 0);
        c1 = __shfl_sync(0xffffffffu, c1, 0);
#pragma unroll 1
        for (int ch = c0; ok && ch <= c1; ++ch) {
          if (chunks > 1) {
            ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
            ++fills;
          }
          const int qb = (int)((fills - 1u) % C::kQBufs);
          const uint64_t bd = desc + (uint64_t)((C::kQOff + qb * C::kQBytes) >> 4);
          const bool q_ends = chunks > 1 || i + nt == i1;
#pragma unroll 1
          for (int t = 0; ok && t < nt; ++t) {
            const uint32_t m = n + t;
            const uint32_t u = t & 1 ? used[1]++ : used[0]++;
            const int st = (int)(m % C::kStages), sb = (t & 1) * 2 + (int)(u & 1u);
            ok = warp_wait2(&k_full[st], (m / C::kStages) & 1u, &s_empty[sb], ((u >> 1) & 1u) ^ 1u, abort_flag, c.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = desc + (uint64_t)((st * kTileBytes) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kHeadDim / 32; ++k) umma_e4m3(tm + sb * C::kSCols, ad + 2 * k, bd + 2 * k, idesc, k != 0);
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
  } else if (warp == C::kQWarp) {
    // ------------------------------------------------------------ queries
    constexpr int kAtOnce = 8;
    uint32_t fills = 0;
    bool ok = true;
    auto fill = [&](int ch) {
      const int qb = (int)(fills % C::kQBufs), first = g.s.first(), rows = (g.s.t1 - g.s.t0) * G;
      uint8_t* op = smem + C::kQOff + qb * C::kQBytes;
#pragma unroll 1
      for (int x0 = 0; x0 < NC; x0 += kAtOnce) {
        const int rho0 = ch * NC + x0;
        int i = rho0 / G, head = rho0 - i * G;
        const uint16_t* src = a.q + (size_t)(g.s.t0 + i) * a.q_stride + (size_t)(g.h * G + head) * kHeadDim + lane * 4;
        uint2 raw[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          raw[x] = make_uint2(0, 0);
          if (rho0 + x < rows) raw[x] = __ldg(reinterpret_cast<const uint2*>(src));
          src += kHeadDim;
          if (++head == G) {
            head = 0;
            src += a.q_stride - (long long)G * kHeadDim;
          }
        }
        // lane x has row x's denominator
        float minus = -CUDART_INF_F, qf = 0.f;
        RowSeen seen = {INT_MAX, 0u};
        if (lane < kAtOnce && rho0 + lane < rows) {
          const int il = (rho0 + lane) / G;
          const float v = __ldg(lse + (size_t)(g.s.t0 + il) * c.Hq + g.h * G + rho0 + lane - il * G) * 1.44269504088896341f;
          if (fabsf(v) <= 3.402823466e38f) minus = -v;  // a row that saw nothing, or whose denominator is no number, gives nothing
          const int pos = first + il;
          if (!a.causal) seen = {0, INT_MAX};
          else if (pos >= 0) seen = {window_lo(pos, a.window), (unsigned)(pos - window_lo(pos, a.window))};
        }
        if (x0 == 0) {
          ok = warp_wait(&q_empty[qb], ((fills / C::kQBufs) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) return;
        }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          uint32_t top = __vmaxu2(raw[x].x & 0x7FFF7FFFu, raw[x].y & 0x7FFF7FFFu);  // bf16 magnitudes order as integers
          top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
          const bool bad = top >= 0x7F80u;
          const int e = bad ? 0 : query_exponent(__uint_as_float(top << 16));
          const float inv = exp2_int(-e);
          uint32_t h0, l0, h1, l1;
          split_bf16x2(bad ? 0u : raw[x].x, inv, h0, l0);
          split_bf16x2(bad ? 0u : raw[x].y, inv, h1, l1);
          const uint32_t sw = ((((uint32_t)lane >> 2) ^ (x & 7)) << 4) + (lane & 3) * 4;
          *reinterpret_cast<uint32_t*>(op + (x0 + x) * 128 + sw) = h0 | (h1 << 16);
          *reinterpret_cast<uint32_t*>(op + (NC + x0 + x) * 128 + sw) = l0 | (l1 << 16);
          if (lane == x) {
            qf = a.scale_log2 * exp2_int(e);
            if (bad) minus = -CUDART_INF_F;  // a row with an infinity or NaN has no weights
          }
        }
        if (lane < kAtOnce) {
          RowPair& r = s_row[(qb * NC + x0 + lane) / 2];
          r.qf[lane & 1] = qf;
          r.minus[lane & 1] = minus;
          s_seen[qb * NC + x0 + lane] = seen;
        }
      }
      if (lane == 0) {
        const int pos_lo = first + ch * NC / G, pos_hi = first + min(rows - 1, ch * NC + NC - 1) / G;
        s_all[qb] = make_int2(window_lo(pos_hi, a.window), a.causal ? pos_lo + 1 : INT_MAX);
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
    // ------------------------------------------------------------ softmax: thread = key; a group of four warps has every kGroups-th tile
    const int group = warp >> 2, w4 = warp & 3, key = tid & 127;
    const uint32_t mine = tmem + ((uint32_t)(w4 * 32) << 16);
    uint32_t n = 0, fills = 0, used = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
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
          const int2 all = s_all[qb];
#pragma unroll 1
          for (int t = group; t < nt; t += C::kGroups) {
            const uint32_t m = n + t;
            const int st = (int)(m % C::kStages), j0 = jg + t * kTile, j = j0 + key;
            if (ch == c0) ok = warp_wait(&i_full[st], (m / C::kStages) & 1u, abort_flag, c.status);
            if (!ok) break;
            const float ks = infos[st].kf[key >> 4];
            float acc = ch > c0 ? s_acc[st * kTile + key] : 0.f;
            // the key's weight so far, on its way while the scores are waited for
            const bool ends = ch == c1;
            float before = 0.f;
            float* to = nullptr;
            if (ends) {
              const int pg = infos[st].page[key >> 4];
              if (pg >= 0 && j >= g.r.lo && j < g.r.hi) {
                const size_t at = (((size_t)pg * c.Hkv + g.h) << c.page_log2) + (j & (c.page - 1));
                to = weight_out + at;
                if (weight_in && j < g.s.first()) before = weight_in[at];
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&k_empty[st]);
            }
            const int sb = group * 2 + (int)(used & 1u);
            ok = warp_wait(&s_full[sb], (used >> 1) & 1u, abort_flag, c.status);
            if (!ok) break;
            ++used;
            tc_fence_after();
            // (two copies of the loop: masks written out under a condition are issued whether it holds or not, twice the rest)
            acc += j0 >= all.x && j0 + kTile <= all.y
                       ? add_weights<NC, false>(mine + sb * C::kSCols, s_row + qb * NC / 2, s_seen + qb * NC, ks, j, &s_empty[sb], lane)
                       : add_weights<NC, true>(mine + sb * C::kSCols, s_row + qb * NC / 2, s_seen + qb * NC, ks, j, &s_empty[sb], lane);
            if (!ends) {
              s_acc[st * kTile + key] = acc;
            } else if (to) {
              *to = before + acc;
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
  return launch_kernel(kern, dim3(C::kPerSm * n_sms), dim3(C::kThreads), C::kBytes, stream, false, tk, c, a, lse, weight_in, weight_out);
}

}  // namespace

cudaError_t launch_kv_weights_rows(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                                   int n_sms, cudaStream_t stream) {
  const long long rows = (long long)(c.Hq / c.Hkv) * a.max_q;
  if (rows <= 8) return launch<8>(c, a, lse, weight_in, weight_out, n_sms, stream);
  // Up to 16 rows a tile of keys is a product and little else; above, their conversion to bf16 pays.  64 sequences of 1500-8190 tokens, 8
  // key/value heads, this kernel and the other: 16 rows 76 and 137 us, 24 rows 113 and 129, 32 rows 121 and 129, 48 rows 162 and 131; 4 of
  // 5000-16000: 16 rows 23 and 29, 24 rows 31 and 31, 48 rows 43 and 29; one of 130 tokens: 16 rows 12 and 14, 24 rows 14 and 12.  Eight columns
  // against 16 for up to 8 rows: 62 and 64 us, 21 and 23, 10 and 12.
  // (the other kernel takes the rows' denominators through its product, divided by the scale)
  if (rows <= 16 || a.scale_log2 < 1e-9f) return launch<16>(c, a, lse, weight_in, weight_out, n_sms, stream);
  return launch_kv_weights_many(c, a, lse, weight_in, weight_out, n_sms, stream);
}

}  // namespace moe
