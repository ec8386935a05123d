// Accumulated attention weights of many query rows per key/value head (the last tokens of a prompt, chunks): products and
// exponentials bound it, 576 and 512 cycles for a tile and 128 rows.
//
// As in the kernel for few rows the keys are the M operand and a softmax thread owns a key, but with a hundred rows to a tile what the
// thread does for each row is all that counts, so everything that belongs to a row goes through the product:
//   S^T[128 keys, NC] = K . q^T + (1 / kf) m^T            tcgen05 kind::f16, bf16: keys converted once (exactly), queries as given
//   weight = 2^(c S),   c = kf * scale * log2(e),   m = -lse / scale
// kf = 2^e_k is the key's page's scale; m is three bf16 parts (24 bits) against three times 1 / kf (a power of two), one more K = 16 step of
// the product.  A row that gives nothing has m = -2^100.  What is left is a product, an exponential and a sum, two and a half
// instructions for a row; with the row's factor and denominator read from shared memory (and E4M3 halves of the queries made anew for
// every few tiles) a step took 2,900 cycles in the softmax warps where it takes 1,200.
//
// A block keeps kTiles tiles of keys in shared memory, converted, and walks the chunks of NC rows over them.
//
// Measured: the last 40-64 tokens of 4 prompts of 5000-16000, 8 query heads a key/value head, 64 us (35.6 GFLOP of scores, 18 us at the
// bf16 rate).  Of a block's 111,000 cycles (the slowest of 150 has 125,000) 4,700 pass before its roles begin, 10,700 more before its first
// product and 2,900 after its last.  The 61 steps between take 1,520 each: the MMA warp waits 300 for keys, 180 for room for scores and
// 80 for queries, and is 960 at issuing a step's nine products (576 at the tensor core's rate).
//
// Warps: 8 softmax (two groups of four, which take the tiles in turn, two buffers of scores each), 4 that convert keys, TMA, MMA, 4 for
// the queries (two for either buffer).  Every wait is bounded (2 s).
#include "attention_weights.cuh"

namespace moe {
namespace {

struct TileInfo {     // per 16 keys of a tile
  float kf[8];        // 2^e_k
  int page[8];        // -1: none
  uint32_t inv[8];    // 1 / kf as bf16, 0: codes that count as zeros (kf = 1)
};

constexpr float kNothing = -1.2676506e30f;  // -2^100: exact in bf16, and below any sum

template <int NC>
struct Cfg {
  static constexpr int kTiles = NC > 64 ? 3 : 4, kCodes = 2, kInfos = 8, kQBufs = 2;
  static constexpr int kGroups = 2, kSBufs = 2 * kGroups;
  static constexpr int kConvWarp = 4 * kGroups, kTmaWarp = kConvWarp + 4, kMmaWarp = kTmaWarp + 1, kQWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kQWarp + 2 * kQBufs);
  static constexpr int kKBytes = 2 * kTileBytes;            // bf16 [2 halves of the dims][128 keys of 128 bytes]
  static constexpr int kQBytes = 2 * NC * 128;              // the same of the rows
  static constexpr int kQOff = kTiles * kKBytes;
  static constexpr int kCodeOff = kQOff + kQBufs * kQBytes; // E4M3 as cached
  static constexpr int kKxOff = kCodeOff + kCodes * kTileBytes;  // the extra K = 16 step: 32 bytes a key, 8 keys by 16 bytes at a time
  static constexpr int kQxOff = kKxOff + kTiles * kTile * 32;
  static constexpr int kBarOff = kQxOff + kQBufs * NC * 32;
  static constexpr int kNumBars = 2 * kCodes + 2 * kTiles + 2 * kQBufs + 2 * kSBufs + 1;
  static constexpr int kInfoOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSeenOff = kInfoOff + kInfos * (int)sizeof(TileInfo);     // RowSeen [kQBufs][NC]
  static constexpr int kAllOff = kSeenOff + kQBufs * NC * (int)sizeof(RowSeen);  // int2 [kQBufs]
  static constexpr int kAccOff = kAllOff + kQBufs * (int)sizeof(int2);           // float [kTiles][128]
  static constexpr int kMiscOff = kAccOff + kTiles * kTile * 4;
  static constexpr int kBytes = 1024 + kMiscOff + 32;
  static constexpr int kTmemCols = kSBufs * NC;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kTmemCols <= 512, "tensor memory");
};

// The K = 16 step: rows of 32 bytes without swizzle, K contiguous: 8 rows of 16 bytes, then those rows' other 16 bytes, then the next 8 rows.
__device__ __forceinline__ uint64_t desc_extra(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;   // leading byte offset: along K
  d |= (uint64_t)(256u >> 4) << 32;   // stride byte offset: along M or N
  d |= (uint64_t)1u << 46;            // descriptor version
  return d;
}
__device__ __forceinline__ uint32_t extra_at(int row) { return (uint32_t)(row >> 3) * 256u + (uint32_t)(row & 7) * 16u; }

// Two E4M3 codes as bf16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint32_t codes) {
  const float2 f = e4m3x2_f32(codes);
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A key's weights of a chunk's rows, from its lane of tensor memory.  kFinite: leaves out those that are not finite.
template <int NC, bool kMasked, bool kFinite>
__device__ __forceinline__ float add_weights(uint32_t taddr, const RowSeen* seen, float factor, int j) {
  constexpr int P = 32, kSteps = NC / P;  // columns at a time: the next ones come while these are added up
  const uint64_t f2 = f32x2(factor, factor);
  uint64_t sum = 0, sum1 = 0;
  uint32_t v[2][P];
  tmem_ld32_async(taddr, v[0]);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    tmem_wait_ld();
    if (k + 1 < kSteps) tmem_ld32_async(taddr + (k + 1) * P, v[(k + 1) & 1]);
    const uint32_t* s = v[k & 1];
#pragma unroll
    for (int x = 0; x < P; x += 2) {
      float z0, z1;
      f32x2_split(mul_f32x2(f32x2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), f2), z0, z1);
      if (kMasked) {
        const int4 see = *reinterpret_cast<const int4*>(seen + k * P + x);
        if ((unsigned)(j - see.x) > (unsigned)see.y) z0 = -CUDART_INF_F;
        if ((unsigned)(j - see.z) > (unsigned)see.w) z1 = -CUDART_INF_F;
      }
      float p0 = ex2(z0), p1 = ex2(z1);
      if (kFinite) {
        p0 = p0 < CUDART_INF_F ? p0 : 0.f;
        p1 = p1 < CUDART_INF_F ? p1 : 0.f;
      }
      uint64_t& to = x & 2 ? sum1 : sum;
      to = add_f32x2(to, f32x2(p0, p1));
    }
  }
  float s0, s1;
  f32x2_split(add_f32x2(sum, sum1), s0, s1);
  return s0 + s1;
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, 1)
    kv_weights_many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, int q_boxes, const KvBatch c,
                           const AttentionArgs a, const float* lse, const float* weight_in, float* weight_out) {
  using C = Cfg<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* c_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // codes
  uint64_t* c_empty = c_full + C::kCodes;
  uint64_t* k_full = c_empty + C::kCodes;   // converted keys
  uint64_t* k_empty = k_full + C::kTiles;
  uint64_t* q_full = k_empty + C::kTiles;
  uint64_t* q_empty = q_full + C::kQBufs;
  uint64_t* s_full = q_empty + C::kQBufs;   // [kSBufs]: a group's in turn
  uint64_t* s_empty = s_full + C::kSBufs;
  uint64_t* done = s_empty + C::kSBufs;
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  RowSeen* s_seen = reinterpret_cast<RowSeen*>(smem + C::kSeenOff);
  int2* s_all = reinterpret_cast<int2*>(smem + C::kAllOff);  // keys [x, y) are seen by every row of the chunk
  float* s_acc = reinterpret_cast<float*>(smem + C::kAccOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_begin = reinterpret_cast<int*>(smem + C::kMiscOff + 12);  // b, h
  long long* s_at = reinterpret_cast<long long*>(smem + C::kMiscOff + 24);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv;
  if (blockIdx.x == 0 && tid == C::kThreads - 1) check_starts(c);

  long long run;
  if (!weight_run<NC>(c, a, G, C::kThreads, reinterpret_cast<long long*>(s_acc), run, s_begin, s_at)) return;

  if (tid == 0) {
    for (int i = 0; i < C::kCodes; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], 4);
    }
    for (int i = 0; i < C::kTiles; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1 + 4);  // the tile's last product, and the softmax warps that have its scales
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 1 + 4 * C::kGroups);
    }
    for (int i = 0; i < C::kSBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(done, 1);
    abort_flag[0] = 0;
    abort_flag[1] = (int)a.limit_us;
    tma_prefetch_desc(&tm_k);
    if (q_boxes) tma_prefetch_desc(&tm_q);
    fence_mbar_init();
  }
  // of the extra step only the first 16 bytes of a row are ever written again
  for (int i = tid; i < (C::kTiles * kTile + C::kQBufs * NC) * 2; i += C::kThreads)
    reinterpret_cast<uint4*>(smem + C::kKxOff)[i] = make_uint4(0, 0, 0, 0);
  fence_async_shared();
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
        const int st = (int)(n % C::kCodes);
        // pages are loaded whole, by the first of a page's lanes that has it
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0) & 0xFFu;
        const uint32_t group = ((1u << (1 << per_log2)) - 1u) << ((lane & 7) >> per_log2 << per_log2);
        const bool load = lane < 8 && pg >= 0 && __ffs(have & group) - 1 == lane;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * box;
        uint8_t* dst = smem + C::kCodeOff + st * kTileBytes + ((lane & 7) >> per_log2) * box;
        const int y = load ? (int)(((long long)pg * c.Hkv + g.h) << c.page_log2) : 0;
        ok = warp_wait(&c_empty[st], ((n / C::kCodes) & 1u) ^ 1u, abort_flag, c.status);
        if (!ok) break;
        // (kInfos is beyond what can be between this tile and the oldest in use: kCodes and kTiles.  Scales below 2^-95 are none
        // that an append writes; their keys count as zeros)
        if (lane < 8) {
          TileInfo& ti = infos[n % C::kInfos];
          const uint32_t s = min(sc, 254u);
          const bool none = s < 32u;
          ti.kf[lane] = none ? 1.f : exp2_byte(s);
          ti.inv[lane] = none ? 0u : s == 254u ? 0x40u : (254u - s) << 7;
          ti.page[lane] = pg;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&c_full[st], bytes);
        __syncwarp();
        if (load && !a.withhold) tma_load_2d(dst, &tm_k, 0, y, &c_full[st], pol);
        ++n;
        pg = pg1;
        pg1 = pg2;
        sc = sc1;
      }
    }
    // Every copy lands before the block ends.
    if (lane == 0) {
      for (int st = 0; st < C::kCodes; ++st) {
        const uint32_t fills = n / C::kCodes + ((uint32_t)st < n % C::kCodes ? 1u : 0u);
        if (fills) mbar_wait_bounded(&c_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
      }
    }
    __syncwarp();
  } else if (warp >= C::kConvWarp && warp < C::kTmaWarp) {
    // ------------------------------------------------------------ keys: E4M3 -> bf16, 32 keys a warp.  A lane has 16 dims of a key; four
    // lanes are one key's, the next four that key's whose place in the eight differs by 5, so that eight lanes meet eight
    // different banks in the reads (16-byte pieces quad ^ place of a row) as in the writes (pieces 2 quad ^ place, and its neighbour).
    const int w = warp - C::kConvWarp, place = (lane >> 3) ^ ((lane & 4) ? 5 : 0), quad = lane & 3, key0 = w * 32 + place;
    const uint32_t from = key0 * 128 + ((quad ^ place) << 4), to = key0 * 128 + (((2 * quad) ^ place) << 4);
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
#pragma unroll 1
      for (int i = g.i0; i < g.i1; ++i, ++n) {
        const int st = (int)(n % C::kCodes), slot = (int)(n % C::kTiles);
        ok = warp_wait2(&c_full[st], (n / C::kCodes) & 1u, &k_empty[slot], ((n / C::kTiles) & 1u) ^ 1u, abort_flag, c.status);
        if (!ok) break;
        const uint32_t* inv = infos[n % C::kInfos].inv + w * 2;  // of the warp's keys, 16 each
        const uint8_t* src = smem + C::kCodeOff + st * kTileBytes;
        uint8_t* dst = smem + slot * C::kKBytes;
#pragma unroll
        for (int x = 0; x < 8; x += 4) {
          uint4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const uint4*>(src + (from ^ ((y & 1) << 6)) + ((x + y) >> 1) * 1024);
          if (inv[x >> 2] == 0u) {
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint8_t* at = dst + (y & 1) * kTileBytes + ((x + y) >> 1) * 1024;
            *reinterpret_cast<uint4*>(at + to) = make_uint4(e4m3x2_bf16x2(v[y].x & 0xFFFFu), e4m3x2_bf16x2(v[y].x >> 16),
                                                            e4m3x2_bf16x2(v[y].y & 0xFFFFu), e4m3x2_bf16x2(v[y].y >> 16));
            *reinterpret_cast<uint4*>(at + (to ^ 16)) = make_uint4(e4m3x2_bf16x2(v[y].z & 0xFFFFu), e4m3x2_bf16x2(v[y].z >> 16),
                                                                   e4m3x2_bf16x2(v[y].w & 0xFFFFu), e4m3x2_bf16x2(v[y].w >> 16));
          }
        }
        {
          const uint32_t u = inv[lane >> 4] ? inv[lane >> 4] : 0x3F80u;
          *reinterpret_cast<uint4*>(smem + C::kKxOff + slot * kTile * 32 + extra_at(w * 32 + lane)) = make_uint4(u | u << 16, u, 0, 0);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&k_full[slot]);
          mbar_arrive(&c_empty[st]);
        }
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA: the whole warp walks along and one lane issues; bounds by shuffle,
    // so that loops and descriptors are the warp's and not a lane's
    const uint32_t idesc = umma_idesc_bf16(kTile, NC);
    const uint64_t desc = umma_desc_sw128(smem_u32(smem)), xdesc = desc_extra(smem_u32(smem));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t n = 0, fills = 0, used[2] = {0, 0}, odd = 0;  // tiles of earlier groups; query buffers; tiles given to a group of warps
    bool ok = true;
    while (ok && walk.next(g)) {
      const int i0 = __shfl_sync(0xffffffffu, g.i0, 0), i1 = __shfl_sync(0xffffffffu, g.i1, 0), chunks = __shfl_sync(0xffffffffu, g.chunks, 0);
      if (chunks == 1) {
        ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
        ++fills;
      }
#pragma unroll 1
      for (int i = i0; ok && i < i1; i += C::kTiles) {
        const int nt = min(C::kTiles, i1 - i), j0 = (g.r.tile0 + i) * kTile;
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
          const uint64_t bx = xdesc + (uint64_t)((C::kQxOff + qb * NC * 32) >> 4);
          const bool q_ends = chunks > 1 || i + nt == i1;
#pragma unroll 1
          for (int t = 0; ok && t < nt; ++t) {
            const uint32_t m = n + t;
            const uint32_t who = (t ^ odd) & 1u, u = who ? used[1]++ : used[0]++;
            const int slot = (int)(m % C::kTiles), sb = (int)(who * 2 + (u & 1u));
            ok = warp_wait2(&k_full[slot], (m / C::kTiles) & 1u, &s_empty[sb], ((u >> 1) & 1u) ^ 1u, abort_flag, c.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = desc + (uint64_t)((slot * C::kKBytes) >> 4);
            const uint64_t ax = xdesc + (uint64_t)((C::kKxOff + slot * kTile * 32) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kHeadDim / 16; ++k)
                umma_bf16(tm + sb * NC, ad + (k >> 2) * (kTileBytes >> 4) + 2 * (k & 3), bd + (k >> 2) * ((NC * 128) >> 4) + 2 * (k & 3), idesc,
                          k != 0);
              umma_bf16(tm + sb * NC, ax, bx, idesc, 1);
              umma_commit(&s_full[sb]);
              if (ch == c1) umma_commit(&k_empty[slot]);
              if (q_ends && t == nt - 1) umma_commit(&q_empty[qb]);
            }
            __syncwarp();
          }
        }
        n += nt;
        odd ^= nt;
      }
    }
    // whatever was issued has finished before tensor memory is given back (after an abort too)
    if (elect_one()) umma_commit(done);
    __syncwarp();
    mbar_wait_bounded(done, 0, abort_flag, 1000ull * a.limit_us, c.status, false);
  } else if (warp >= C::kQWarp) {
    // ------------------------------------------------------------ queries: two warps for either buffer, half of the chunk's rows each
    constexpr int kMine = NC / 2;  // rows, two at a time: 16 lanes x 16 bytes a row
    const int mine_qb = (warp - C::kQWarp) >> 1, r_first = ((warp - C::kQWarp) & 1) * kMine, piece = lane & 15;
    const uint64_t pol = policy_evict_last();
    uint32_t fills = 0;
    bool ok = true;
    // Where G does not divide NC: 16 bytes a lane, where the copies of whole boxes would put them.
    auto copy_rows = [&](int ch, int rows, int qb) {
      int r = r_first + (lane >> 4), i = (ch * NC + r) / G, head = ch * NC + r - i * G, left = rows - (ch * NC + r);
      const uint16_t* src = a.q + (size_t)(g.s.t0 + i) * a.q_stride + (size_t)(g.h * G + head) * kHeadDim + piece * 8;
      const long long wrap = a.q_stride - (long long)G * kHeadDim;
      const uint32_t op = smem_u32(smem) + C::kQOff + qb * C::kQBytes + (piece >> 3) * NC * 128;
#pragma unroll 4
      for (int k = 0; k < kMine / 2; ++k, r += 2, left -= 2) {
        cp_async16(op + r * 128 + (((piece & 7) ^ (r & 7)) << 4), left > 0 ? src : a.q, left > 0 ? 16 : 0);
        src += 2 * kHeadDim;
        head += 2;
#pragma unroll
        for (int x = 0; x < 2; ++x)  // G may be 1
          if (head >= G) {
            head -= G;
            src += wrap;
          }
      }
      cp_async_commit();
    };
    auto fill = [&](int ch) {
      const int qb = (int)(fills % C::kQBufs);
      if (qb != mine_qb) {
        ++fills;
        return;
      }
      const int rows = (g.s.t1 - g.s.t0) * G, first = g.s.first();
      // of this lane's rows: minus their denominator over the scale, in three parts, and the keys that they see
      uint4 part[kMine / 32];
      RowSeen seen[kMine / 32];
#pragma unroll
      for (int k = 0; k < kMine / 32; ++k) {
        const int rho = ch * NC + r_first + k * 32 + lane;
        float m = kNothing;
        seen[k] = {INT_MAX, 0u};
        if (rho < rows) {
          const int i = rho / G, pos = first + i;
          const float v = __ldg(lse + (size_t)(g.s.t0 + i) * c.Hq + g.h * G + rho - i * G) * (-1.44269504088896341f / a.scale_log2);
          if (fabsf(v) < 1e29f) m = v;  // a row that saw nothing, or whose denominator is no number, gives nothing
          if (!a.causal) seen[k] = {0, INT_MAX};
          else if (pos >= 0) seen[k] = {window_lo(pos, a.window), (unsigned)(pos - window_lo(pos, a.window))};
        }
        const uint32_t m0 = f32_to_bf16_rne(m);
        m -= bf16_lo(m0);
        const uint32_t m1 = f32_to_bf16_rne(m);
        m -= bf16_lo(m1);
        part[k] = make_uint4(m0 | m1 << 16, f32_to_bf16_rne(m), 0, 0);
      }
      ok = warp_wait(&q_empty[qb], ((fills / C::kQBufs) & 1u) ^ 1u, abort_flag, c.status);
      if (!ok) return;
      if (!q_boxes) copy_rows(ch, rows, qb);
#pragma unroll
      for (int k = 0; k < kMine / 32; ++k) {
        const int x = r_first + k * 32 + lane;
        *reinterpret_cast<uint4*>(smem + C::kQxOff + qb * NC * 32 + extra_at(x)) = part[k];
        s_seen[qb * NC + x] = seen[k];
      }
      if (r_first == 0 && lane == 0) {
        const int pos_lo = first + ch * NC / G, pos_hi = first + min(rows - 1, ch * NC + NC - 1) / G;
        s_all[qb] = make_int2(window_lo(pos_hi, a.window), a.causal ? pos_lo + 1 : INT_MAX);
      }
      if (!q_boxes) cp_async_wait<0>();
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (q_boxes && r_first == 0) {
          mbar_arrive_expect_tx(&q_full[qb], C::kQBytes);
          for (int half = 0; half < 2; ++half)
            tma_load_3d(smem + C::kQOff + qb * C::kQBytes + half * NC * 128, &tm_q, half * 64, g.h * G, g.s.t0 + ch * NC / G, &q_full[qb], pol);
        } else {
          mbar_arrive(&q_full[qb]);
        }
      }
      ++fills;
    };
    while (ok && walk.next(g)) {
      if (g.chunks == 1) {
        fill(0);
        continue;
      }
#pragma unroll 1
      for (int i = g.i0; ok && i < g.i1; i += C::kTiles) {
        const int nt = min(C::kTiles, g.i1 - i), j0 = (g.r.tile0 + i) * kTile;
        int c0, c1;
        chunks_of(g, a, G, NC, j0, j0 + nt * kTile, c0, c1);
#pragma unroll 1
        for (int ch = c0; ok && ch <= c1; ++ch) fill(ch);
      }
    }
    // every copy lands before the block ends
    if (q_boxes && r_first == 0 && lane == 0) {
      const uint32_t mine = fills / C::kQBufs + ((uint32_t)mine_qb < fills % C::kQBufs ? 1u : 0u);  // fills of this buffer
      if (mine) mbar_wait_bounded(&q_full[mine_qb], (mine - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax: thread = key
    const int group = warp >> 2, w4 = warp & 3, key = tid & 127;
    const uint32_t mine = tmem + ((uint32_t)(w4 * 32) << 16);
    uint32_t n = 0, fills = 0, used = 0, odd = 0;  // odd: which group of warps begins
    bool ok = true;
    while (ok && walk.next(g)) {
      if (g.chunks == 1) {
        ok = warp_wait(&q_full[fills % C::kQBufs], (fills / C::kQBufs) & 1u, abort_flag, c.status);
        ++fills;
      }
#pragma unroll 1
      for (int i = g.i0; ok && i < g.i1; i += C::kTiles) {
        const int nt = min(C::kTiles, g.i1 - i), jg = (g.r.tile0 + i) * kTile;
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
          for (int t = (int)((group ^ odd) & 1u); t < nt; t += C::kGroups) {
            const uint32_t m = n + t;
            const int slot = (int)(m % C::kTiles), j0 = jg + t * kTile, j = j0 + key;
            if (ch == c0) ok = warp_wait(&k_full[slot], (m / C::kTiles) & 1u, abort_flag, c.status);
            if (!ok) break;
            const TileInfo& ti = infos[m % C::kInfos];
            const float factor = ti.kf[key >> 4] * a.scale_log2;
            float acc = ch > c0 ? s_acc[slot * kTile + key] : 0.f;
            // the key's weight so far, on its way while the scores are waited for
            const bool ends = ch == c1;
            float before = 0.f;
            float* to = nullptr;
            if (ends) {
              const int pg = ti.page[key >> 4];
              if (pg >= 0 && j >= g.r.lo && j < g.r.hi) {
                const size_t at = (((size_t)pg * c.Hkv + g.h) << c.page_log2) + (j & (c.page - 1));
                to = weight_out + at;
                if (weight_in && j < g.s.first()) before = weight_in[at];
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&k_empty[slot]);
            }
            const int sb = group * 2 + (int)(used & 1u);
            ok = warp_wait(&s_full[sb], (used >> 1) & 1u, abort_flag, c.status);
            if (!ok) break;
            ++used;
            tc_fence_after();
            // (two copies of the loop: masks written out under a condition are issued whether it holds or not, twice the rest)
            const RowSeen* seen = s_seen + qb * NC;
            float sum = j0 >= all.x && j0 + kTile <= all.y ? add_weights<NC, false, false>(mine + sb * NC, seen, factor, j)
                                                           : add_weights<NC, true, false>(mine + sb * NC, seen, factor, j);
            // A row with an infinity or NaN has none but such scores, and so has a key with a NaN: once more without them.
            if (__any_sync(0xffffffffu, !(sum < CUDART_INF_F))) sum = add_weights<NC, true, true>(mine + sb * NC, seen, factor, j);
            acc += sum;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sb]);
            if (!ends) {
              s_acc[slot * kTile + key] = acc;
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
        odd ^= nt;
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
  const int G = c.Hq / c.Hkv, q_boxes = NC % G == 0;
  CUtensorMap tq = {};
  if (q_boxes && !make_query_map(&tq, a, c, G, NC / G)) return cudaErrorInvalidValue;
  auto kern = kv_weights_many_kernel<NC>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(n_sms), dim3(C::kThreads), C::kBytes, stream, false, tk, tq, q_boxes, c, a, lse, weight_in, weight_out);
}

}  // namespace

cudaError_t launch_kv_weights_many(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                                   int n_sms, cudaStream_t stream) {
  // By the most rows of a sequence.  32 sequences of 1000-4000 tokens and 4 of 5000-16000, 8 key/value heads, chunks of 64 and of 128: 32 rows
  // 49 and 64 us, 29 and 31; 64 rows 47 and 59, 29 and 33; 72 rows (two chunks of 64) 86 and 62, 45 and 37; 128 rows 76 and 59, 39 and 31.
  const long long rows = (long long)(c.Hq / c.Hkv) * a.max_q;
  return rows <= 64 ? launch<64>(c, a, lse, weight_in, weight_out, n_sms, stream) : launch<128>(c, a, lse, weight_in, weight_out, n_sms, stream);
}

}  // namespace moe
