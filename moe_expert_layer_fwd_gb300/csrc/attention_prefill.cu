// Attention of many query rows per key/value head (prompts and chunks): matrix products bound it.
//
// The rows of one key/value head, new tokens x grouped heads, are the M operand: an item is 256 of them, two M = 128 tiles
// that take turns on the tensor core -- while one's softmax runs, the other's products do -- against key tiles of 128:
//   S[128, 128 keys] = Q_hi . K^T + Q_lo . K^T     kind::f8f6f4: queries split in two E4M3 halves, keys as cached
//   u = S * scale * 2^(e_k + e_q) + e_v            per page of the tile: a factor and a summand for its columns
//   p' = 2^(u - r + 9) in f16,  l += 2^-e_v sum p'
//   O[128, 128 dims] += p' . V                     kind::f16, p' in tensor memory over S, V as exact f16 numbers
// Two products of E4M3 cost what one of bf16 does, and the keys need no conversion; the values are converted once per tile
// for both M tiles by four warps of their own (an E4M3 code is an f16 number; their scales stay out of them).  r follows the
// running maximum of u, and with it O is rescaled, only when that of one of a warp's rows has grown by more than 2^6.9 since (then
// all of them follow): p' stays below 2^15.9 of f16's 65504 and keeps 11 bits down to 2^-23 of the largest, 8 down to 2^-26; below, it
// is rounded to multiples of 2^-33 of that one.  (One key may take most of a row, whose thousands of others then count together.
// Each factor of two more costs rescaling: a ragged batch of chunks takes 487 us at 2^8 and a smallest step of 2^-31, 490 so,
// 499 at 2^5.9 and 521 at 2^3.9.)
//
// Work: the items' tiles in one order, cut into equal runs, one per block and SM, as in the decode kernel: causal items of
// any length fill all SMs evenly, and a chunk of few rows over a long cache is split along its keys.  The rows of a split item
// (one at each end of a run, at most) are joined by a second kernel.
//
// Items of at most 128 rows (kSplit): both M tiles hold the same rows and take its key tiles in turn, and the second one's
// sums are added to the first one's at the end (32 rows a head over long caches: 87 us, and 103 as a half-empty item).
//
// Measured (8 query heads per key/value head, causal): a prompt of 16,384 tokens 1.74 ms a call, 1,270 TFLOP/s; a ragged batch of
// chunks 0.49 ms, 1,050 TFLOP/s.  What bounds it is the chain of one M tile: scores read, weights made and written
// (1,900 cycles), then the products of these weights and of the next scores (1,400 with their latency), where the products
// of both M tiles would take 2,050; and an item's own 11,000 cycles or so between its neighbours' tiles.
//
// Warps (16): 0-3 and 4-7 softmax of the M tiles (thread = row; they also fetch the queries, rescale and write the output),
// 8-11 values, 12 TMA, 13 MMA, 14 scales of the tiles' pages, and it walks the run; 15 has nothing to do.  Registers: 192 a
// thread for the softmax, 64 for the rest.  Every wait is bounded (2 s).
#include "attention_tiles.cuh"

namespace moe {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kValWarp = 8, kTmaWarp = 12, kMmaWarp = 13, kScaleWarp = 14;
constexpr int kThreads = 512;
constexpr int kReaders = kSoftWarps + 4 + 1 + 1;  // warps that read the run's parts
constexpr int kM = 128;
constexpr int kKeys = kTile;                 // keys of a tile
constexpr int kInfos = 4, kParts = 2;
constexpr int kPieces = kKeys / 16;
constexpr int kMinRun = 6;                   // cost of a block's run, at least
constexpr int kItemCost = 5;                 // an item's own cost (loading its queries, writing its rows), in tiles:
                                             // a prompt of 16,384 takes 1,808 us at 3, 1,700 at 5, 1,711 at 6

// A run that begins within an item has a tile of it, then: the joins count on that.
static_assert(kMinRun > kItemCost, "runs");

constexpr float kBase = 9.f, kSlack = 6.9f;  // p' = 2^(u - r + kBase), u <= r + kSlack: below 65504, the largest f16 number

struct TileInfo {    // per 16 keys of a tile
  float kf[8];       // 2^e_k
  float lv[8];       // e_v
  float un[8];       // 2^-e_v
  uint32_t have;     // bit i: the page of keys 16 i .. 16 i + 15 is there
  uint32_t pad[3];
};
struct Part {  // an item (rows [qt * kRows, (qt + 1) * kRows) of a sequence's n * G for head h) and its tiles [i0, i1) in this run
  int b, h, qt, i0, i1, nt, tile0, lo, hi;  // keys [lo, hi) are seen by some row; nt == 0: the run is over
  int later;                                // not the item that the run begins in
  int t0, n, first;                         // first new token, new tokens, position of the first
  int own0, plen, prefix;                   // pass 3: the sequence's own keys begin here, behind the plen keys of this prefix
};

// kSplit: both M tiles hold the same 128 rows and take an item's key tiles in turn (else 256 rows, the same tiles).
template <bool kSplit>
struct Cfg {
  static constexpr int kRows = kSplit ? kM : 2 * kM;   // rows of an item
  static constexpr int kStep = kSplit ? 2 : 1;         // tiles that the two M tiles take at a time
  static constexpr int kKStages = kSplit ? 4 : 3, kVStages = 2, kV16s = kSplit ? 3 : 2;
  static constexpr int kQOff = 0;                      // [hi, lo][128 rows of 128 bytes], one for each M tile unless kSplit
  static constexpr int kKOff = kQOff + (kSplit ? 2 : 4) * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;     // E4M3 as cached
  static constexpr int kV16Off = kVOff + kVStages * kTileBytes;   // f16 [2 halves of the dims][128 tokens of 128 bytes]
  static constexpr int kV16Bytes = 2 * kTileBytes;
  static constexpr int kInfoOff = kV16Off + kV16s * kV16Bytes;
  static constexpr int kPartOff = kInfoOff + kInfos * (int)sizeof(TileInfo);
  static constexpr int kRlOff = kPartOff + kParts * (int)sizeof(Part);  // kSplit: float2 [128], the queries' factors (x), then M tile 1's r and l
  static constexpr int kBarOff = kRlOff + (kSplit ? kM * 8 : 0);
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 2 * kV16s + 2 * kInfos + 2 * kParts + 2 + 2 + 2 + 2 + 2 + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kBytes = 1024 + kMiscOff + 32;
  static_assert(kBytes <= 232448, "shared memory");
  // Tiles of a part, made whole steps: one past its end is there, and empty.
  static __device__ __forceinline__ int tiles(const Part& g) { return (g.i1 - g.i0 + kStep - 1) / kStep * kStep; }
};

// Pass 3: the keys of a sequence are its prefix's, in whole tiles (the last one's rest is nobody's), and then its own: a row that has
// begun its queries and sums goes on with them.  Lengths and positions count the prefix's tiles.
template <int kPass>
struct ItemSeq : SeqRange {};
template <>
struct ItemSeq<3> : SeqRange {
  int own0, plen, prefix;
};
template <int kPass>
__device__ __forceinline__ bool load_item_seq(const KvBatch& c, const AttentionArgs& a, int b, ItemSeq<kPass>& s) {
  bool ok = load_seq(c, b, s);
  if constexpr (kPass == 3) {
    s.own0 = s.plen = s.prefix = 0;
    if (ok && s.t1 > s.t0) {
      int lo = 0, hi = a.n_prefixes;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.prefix_start + mid) <= s.t0) lo = mid; else hi = mid;
      }
      s.prefix = lo;
      s.plen = __ldg(a.prefix_len + lo);
      ok = __ldg(a.prefix_start + lo) <= s.t0 && __ldg(a.prefix_start + lo + 1) >= s.t1 && s.plen >= 0 &&
           s.plen <= (long long)a.prefix_max_pages * c.page;
      if (!ok) set_status(c.status, DEV_ERR_CONFIG);
      s.own0 = ok ? (s.plen + kKeys - 1) / kKeys * kKeys : 0;
      s.len += s.own0;
    }
  }
  return ok;
}

template <int kRows, int kPass>
__device__ __forceinline__ void item_range(const ItemSeq<kPass>& s, const AttentionArgs& a, int G, int qt, int& lo, int& hi) {
  const int i_min = qt * kRows / G, i_max = min(s.t1 - s.t0 - 1, (qt * kRows + kRows - 1) / G);
  hi = a.causal ? max(0, min(s.len, s.first() + i_max + 1)) : s.len;
  if constexpr (kPass == 3) hi = max(hi, s.own0);  // every row sees all of the prefix
  lo = window_lo(s.first() + i_min, a.window);
}
__device__ __forceinline__ int item_tiles(int lo, int hi) { return max(1, (hi + kKeys - 1) / kKeys - lo / kKeys); }

__device__ __forceinline__ int item_cost(int nt) { return nt > 0 ? nt + kItemCost : 0; }

// Sequence b's items take the places from q_start[b] * G / kRows + b on (some stay empty), so that a place's item is
// found without a table of all of them.
template <int kRows>
__device__ __forceinline__ int place_of(const KvBatch& c, int G, int b) {
  return (int)((long long)__ldg(c.q_start + b) * G / kRows) + b;
}
template <int kRows>
__device__ __forceinline__ int places(const KvBatch& c, int G) { return (int)((long long)c.T * G / kRows) + c.B; }

// Walks places in order.
template <int kRows, int kPass>
struct Places {
  const KvBatch& c;
  const AttentionArgs& a;
  int G, place, b;
  bool ok;
  ItemSeq<kPass> s;
  __device__ Places(const KvBatch& c_, const AttentionArgs& a_, int G_, int place_) : c(c_), a(a_), G(G_), place(place_) {
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (place_of<kRows>(c, G, mid) <= place) lo = mid; else hi = mid;
    }
    b = lo;
    ok = load_item_seq<kPass>(c, a, b, s);
  }
  // tiles of the item at this place (0: empty), for one head
  __device__ int tiles(int& qt, int& lo, int& hi) const {
    qt = place - place_of<kRows>(c, G, b);
    if (!ok || qt < 0 || (long long)qt * kRows >= (long long)(s.t1 - s.t0) * G) return 0;
    item_range<kRows, kPass>(s, a, G, qt, lo, hi);
    return item_tiles(lo, hi);
  }
  __device__ void next() {
    ++place;
    if (b + 1 < c.B && place_of<kRows>(c, G, b + 1) <= place) {
      ++b;
      ok = load_item_seq<kPass>(c, a, b, s);
    }
  }
};

// An item costs its tiles and kItemCost more, all of it at its first tile: tile i lies at the place pos(i) of the item's
// cost, and a run has the tiles whose places it covers.
__device__ __forceinline__ int first_tile_from(long long rel, int nt) {
  return rel <= 0 ? 0 : (int)min((long long)nt, max(1LL, rel - kItemCost));
}

template <int kRows, int kPass>
struct Walk {
  Places<kRows, kPass> p;
  long long left, rel;  // cost left in the run; where it starts in the present item
  int h, end, later = 0;
  __device__ Walk(const KvBatch& c, const AttentionArgs& a, int G, long long n, int place, int h_, int rel_)
      : p(c, a, G, place), left(n), rel(rel_), h(h_), end(places<kRows>(c, G)) {}
  __device__ bool next(Part& g) {
    while (left > 0 && p.place < end) {
      g.nt = p.tiles(g.qt, g.lo, g.hi);
      if (g.nt == 0) {
        p.next();
        continue;
      }
      g.b = p.b;
      g.t0 = p.s.t0;
      g.n = p.s.t1 - p.s.t0;
      g.first = p.s.first();
      if constexpr (kPass == 3) {
        g.own0 = p.s.own0;
        g.plen = p.s.plen;
        g.prefix = p.s.prefix;
      }
      g.h = h;
      g.tile0 = g.lo / kKeys;
      g.i0 = first_tile_from(rel, g.nt);
      g.i1 = first_tile_from(rel + left, g.nt);
      g.later = later;
      left -= g.nt + kItemCost - rel;
      rel = 0;
      later = 1;
      if (++h == p.c.Hkv) {
        h = 0;
        p.next();
      }
      if (g.i0 < g.i1) return true;
    }
    g.nt = 0;
    return false;
  }
};

// A role's place in the run's parts, which the walking warp keeps a few ahead in shared memory.
struct Reader {
  const Part* parts;
  uint64_t *full, *empty;
  uint32_t n;
  // The next part (whole warp); false at the end of the run, or after a timeout.
  __device__ bool next(Part& g, volatile int* abort_flag, unsigned* status) {
    const int slot = (int)(n % kParts);
    if (!warp_wait(&full[slot], (n / kParts) & 1u, abort_flag, status)) return false;
    g = parts[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[slot]);
    ++n;
    return g.nt != 0;
  }
  // The part that next() will give, as it stands in shared memory until then (whole warp); nullptr after a timeout.
  __device__ const Part* peek(volatile int* abort_flag, unsigned* status) const {
    return warp_wait(&full[n % kParts], (n / kParts) & 1u, abort_flag, status) ? &parts[n % kParts] : nullptr;
  }
};

__device__ __forceinline__ uint32_t idesc_pv() {
  uint32_t d = 0;
  d |= 1u << 4;                          // D f32, A and B f16
  d |= 1u << 16;                         // B with N (the dims) contiguous
  d |= (uint32_t)(kHeadDim >> 3) << 17;
  d |= (uint32_t)(kM >> 4) << 24;
  return d;
}
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}
// The lowest n bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}

__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t see) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(see & (1u << x))) s[x] = 0xFF800000u;  // -infinity
}

__device__ __forceinline__ float max16(const uint32_t* v) {
  float t0 = __uint_as_float(v[0]), t1 = __uint_as_float(v[1]);
#pragma unroll
  for (int x = 2; x < 14; x += 4) {
    t0 = max3(t0, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
    t1 = max3(t1, __uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
  }
  return fmaxf(max3(t0, __uint_as_float(v[14]), __uint_as_float(v[15])), t1);
}

// The larger bf16 magnitudes of pairs.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t top, const uint4& v) {
  top = __vmaxu2(top, v.x & 0x7FFF7FFFu);
  top = __vmaxu2(top, v.y & 0x7FFF7FFFu);
  top = __vmaxu2(top, v.z & 0x7FFF7FFFu);
  return __vmaxu2(top, v.w & 0x7FFF7FFFu);
}

// 64 columns of this thread's tensor-memory lane times f.
__device__ __forceinline__ void rescale_lane64(uint32_t taddr, float f) {
#pragma unroll
  for (int x = 0; x < 64; x += 8) {
    uint32_t o[8];
    tmem_ld_async(taddr + x, o);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    tmem_st(taddr + x, o);
  }
}

template <bool kSplit, int kPass>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prefill_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                             const KvBatch c, const AttentionArgs a, float* part_o, float2* part_rl, JoinInfo* info) {
  using C = Cfg<kSplit>;
  constexpr int kRows = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* k_empty = k_full + C::kKStages;
  uint64_t* v_full = k_empty + C::kKStages;
  uint64_t* v_empty = v_full + C::kVStages;
  uint64_t* v16_full = v_empty + C::kVStages;
  uint64_t* v16_empty = v16_full + C::kV16s;
  uint64_t* i_full = v16_empty + C::kV16s;
  uint64_t* i_empty = i_full + kInfos;
  uint64_t* r_full = i_empty + kInfos;
  uint64_t* r_empty = r_full + kParts;
  uint64_t* q_full = r_empty + kParts;       // [2], by M tile, as the next three
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* x_full = o_full + 2;             // kSplit: M tile 1's sums are in the queries' place
  uint64_t* x_empty = x_full + 1;            // that place is free
  uint64_t* done = x_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_begin = reinterpret_cast<int*>(smem + C::kMiscOff + 12);  // place, head, cost into the item
  Part* parts = reinterpret_cast<Part*>(smem + C::kPartOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = c.Hq / c.Hkv;
  pdl_launch_dependents();
  if (blockIdx.x == 0 && tid == kThreads - 1) check_starts(c);

  // ---- this block's run: each thread sums a run of places
  long long run;
  {
    long long* s_warp = reinterpret_cast<long long*>(smem);
    const int n = places<kRows>(c, G), per = (n + kThreads - 1) / kThreads;
    const int p0 = min(n, tid * per), p1 = min(n, p0 + per);
    long long mine = 0;
    int qt, lo, hi;
    if (p0 < p1) {
      Places<kRows, kPass> p(c, a, G, p0);
#pragma unroll 1
      for (; p.place < p1; p.next()) mine += item_cost(p.tiles(qt, lo, hi));
    }
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    const long long all = total * c.Hkv, share = max((long long)kMinRun, (all + gridDim.x - 1) / (long long)gridDim.x);
    const long long begin = (long long)blockIdx.x * share;
    run = min(share, all - begin);
    if (run <= 0) {
      if (tid == 0) info[blockIdx.x].split = 0;
      if (kPass == 1) pdl_wait();  // this pass does not end before the one that it may overlap
      return;
    }
    if (before * c.Hkv <= begin && begin < (before + mine) * c.Hkv) {
      Places<kRows, kPass> p(c, a, G, p0);
      long long at = before;
      int nt;
      for (;; p.next()) {
        nt = p.tiles(qt, lo, hi);
        if ((at + item_cost(nt)) * c.Hkv > begin) break;
        at += item_cost(nt);
      }
      const int cost = item_cost(nt);
      const long long rel = (begin - at * c.Hkv) % cost;
      s_begin[0] = p.place;
      s_begin[1] = (int)((begin - at * c.Hkv) / cost);
      s_begin[2] = (int)rel;
      // does this run begin inside an item, with a part of it that is not its first?
      JoinInfo j = {};
      const int i0 = first_tile_from(rel, nt);
      j.split = i0 > 0 && i0 < nt;
      if (j.split) {
        const long long start = begin - rel, last = start + (nt == 1 ? 0 : kItemCost + nt - 1);
        j.b = p.b;
        j.h = s_begin[1];
        j.row0 = qt * kRows;
        j.c0 = (int)(start / share);
        j.c1 = (int)(last / share);
        j.slot0 = start > (long long)j.c0 * share ? 1 : 0;
      }
      info[blockIdx.x] = j;
    }
  }

  if (tid == 0) {
    // who reads a stage: both M tiles' products (the second one's commit tells), or one's
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 4);
    }
    for (int i = 0; i < C::kV16s; ++i) {
      mbar_init(&v16_full[i], 4);
      mbar_init(&v16_empty[i], 1);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], (kSplit ? 4 : 8) + 4);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(x_full, 4);
    mbar_init(x_empty, 4);
    mbar_init(done, 1);
    abort_flag[0] = 0;
    abort_flag[1] = (int)a.limit_us;
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Reader reader{parts, r_full, r_empty, 0};
  Part g;

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ------------------------------------------------------------ softmax: thread = row of M tile mt
    const int mt = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = lanes + mt * 128, t_o = lanes + 256 + mt * kHeadDim;
    uint32_t n0 = 0, steps = 0, xs = 0;  // tiles of earlier parts; steps of this M tile; halves of sums handed over
    uint32_t segs = 0;                   // parts
    bool ok = true;
    float2* other_rl = reinterpret_cast<float2*>(smem + C::kRlOff) + row;  // kSplit only
    uint8_t* hi_row = smem + C::kQOff + (kSplit ? 0 : mt * 2 * kTileBytes) + row * 128;
    // Copies this warp's 32 query rows of a part to where their E4M3 halves will be, two whole rows at a time: a row's 16-byte
    // pieces in turn where its hi half and where its lo half goes, so that a row can be split in place piece by piece.
    // Threads that loaded their own rows touched 32 lines with each instruction, and that, with the loops below written
    // out, made a ragged batch take 515 us for 490.
    auto fetch_queries = [&](const Part& p) {
      const int piece = lane & 15, rows = p.n * G;
      int r = quarter * 32 + (lane >> 4), at = p.qt * kRows + (kSplit ? 0 : mt * kM) + r;
      int i = at / G, head = at - i * G;
      uint8_t* dst = smem + C::kQOff + (kSplit ? 0 : mt * 2 * kTileBytes) + (piece & 1) * kTileBytes;
      const uint16_t* src = a.q + (size_t)p.t0 * a.q_stride + (size_t)p.h * G * kHeadDim + piece * 8;
#pragma unroll 2
      for (int k = 0; k < 16; ++k, r += 2, at += 2) {
        const bool live = at < rows;
        cp_async16(smem_u32(dst + r * 128 + (((piece >> 1) ^ (r & 7)) << 4)),
                   live ? src + (size_t)i * a.q_stride + (size_t)head * kHeadDim : a.q, live ? 16 : 0);
        head += 2;
#pragma unroll
        for (int x = 0; x < 2; ++x)  // G may be 1
          if (head >= G) {
            head -= G;
            ++i;
          }
      }
      cp_async_commit();
    };
    if (!kSplit) {
      const Part* next = reader.peek(abort_flag, c.status);
      if (next && next->nt) fetch_queries(*next);
    }
    while (ok && reader.next(g, abort_flag, c.status)) {
      const int row0 = g.qt * kRows + (kSplit ? 0 : mt * kM);  // this M tile's first
      const int rho = row0 + row;
      const bool live = rho < g.n * G;
      const int i_row = rho / G, head = g.h * G + rho - i_row * G;
      const int pos = g.first + i_row;
      // ---- this row's query, split into two E4M3 halves
      float qf;
      if (!kSplit || mt == 0) {
        if (kSplit) {
          if (segs > 0) {  // the other warps of M tile 0 have read the sums of the part before, which lie here too
            ok = warp_wait(x_empty, (segs & 1u) ^ 1u, abort_flag, c.status);
            if (!ok) break;
          }
          fetch_queries(g);
        }
        cp_async_wait<0>();
        __syncwarp();
        uint32_t top = 0;  // bf16 magnitudes order as integers
#pragma unroll 4
        for (int x = 0; x < 8; ++x) {
          const uint8_t* at = hi_row + ((x ^ (row & 7)) << 4);
          top = max_magnitude(top, *reinterpret_cast<const uint4*>(at));
          top = max_magnitude(top, *reinterpret_cast<const uint4*>(at + kTileBytes));
        }
        top = max(top & 0xFFFFu, top >> 16);
        const bool bad = top >= 0x7F80u;
        const int e = bad ? 0 : query_exponent(__uint_as_float(top << 16));
        const float inv = bad ? CUDART_NAN_F : exp2_int(-e);  // a row with an infinity or NaN has NaN scores
        qf = a.scale_log2 * exp2_int(e);
#pragma unroll 2
        for (int x = 0; x < 8; ++x) {  // 16 dims: two pieces of bf16, then one of either half in their places
          uint8_t* at = hi_row + ((x ^ (row & 7)) << 4);
          const uint4 v0 = *reinterpret_cast<const uint4*>(at), v1 = *reinterpret_cast<const uint4*>(at + kTileBytes);
          const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t h0, l0, h1, l1;
            split_bf16x2(w[2 * y], inv, h0, l0);
            split_bf16x2(w[2 * y + 1], inv, h1, l1);
            hi[y] = h0 | h1 << 16;
            lo[y] = l0 | l1 << 16;
          }
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + kTileBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (kSplit) other_rl->x = qf;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[mt]);
      } else {  // M tile 0's rows are this one's
        ok = warp_wait(&q_full[0], segs & 1u, abort_flag, c.status);
        if (!ok) break;
        qf = other_rl->x;
      }
      ++segs;
      // keys [w_lo, w_hi) are seen by every row of this warp
      const int warp_rho = row0 + quarter * 32, tiles = C::tiles(g);
      // one past the last key that a row at this position sees; pass 3: every row sees the keys before own0, up to plen
      auto seen_end = [&](int pos) {
        if constexpr (kPass == 3) return a.causal ? min(g.hi, max(pos + 1, g.own0)) : g.hi;
        return a.causal ? min(g.hi, pos + 1) : g.hi;
      };
      const int w_hi = kPass == 3 ? seen_end(g.first + warp_rho / G) : a.causal ? min(g.hi, g.first + warp_rho / G + 1) : g.hi;
      const int w_lo = window_lo(g.first + (warp_rho + 31) / G, a.window);
      float r = -CUDART_INF_F, l = 0.f;
#pragma unroll 1
      for (int x = kSplit ? mt : 0; x < tiles; x += C::kStep, ++steps) {
        const int i = g.i0 + x;
        const uint32_t n = n0 + x;
        const int slot = (int)(n % kInfos);
        ok = warp_wait2(&i_full[slot], (n / kInfos) & 1u, &s_full[mt], steps & 1u, abort_flag, c.status);
        if (!ok) break;
        const TileInfo& ti = infos[slot];
        const uint32_t have = ti.have;
        tc_fence_after();
        uint32_t s[kKeys / 32][32];
#pragma unroll
        for (int w = 0; w < kKeys / 32; ++w) tmem_ld32_async(t_s + 32 * w, s[w]);
        tmem_wait_ld();
        const int j0 = (g.tile0 + i) * kKeys;
        const bool rest = kPass == 3 && j0 < g.own0 && j0 + kKeys > g.plen;  // the prefix ends within this tile
        if (j0 < w_lo || j0 + kKeys > w_hi || have != (1u << kPieces) - 1u || rest) {
          // bit x of word w: this row sees key 32 w + x of the tile
          const int hi_col = (kPass == 3 ? (rest ? g.plen : seen_end(pos)) : (a.causal ? min(g.hi, pos + 1) : g.hi)) - j0, lo_col = window_lo(pos, a.window) - j0;
#pragma unroll
          for (int w = 0; w < kKeys / 32; ++w) {
            const uint32_t pages = have >> (2 * w);
            mask32(s[w], (((pages & 1u) ? 0xFFFFu : 0u) | ((pages & 2u) ? 0xFFFF0000u : 0u)) & low_bits(hi_col - 32 * w) &
                             ~low_bits(lo_col - 32 * w));
          }
        }
        float m = -CUDART_INF_F;
#pragma unroll
        for (int b = 0; b < kPieces; ++b) m = fmaxf(m, fmaf(max16(&s[b >> 1][(b & 1) * 16]), qf * ti.kf[b], ti.lv[b]));
        const bool grows = __any_sync(0xffffffffu, m > r + kSlack), grow = grows && m > r;  // r = -infinity: any finite m
        if (x >= C::kStep && grows) {
          // the sums so far are of the tile before: wait for its product, then bring them to the new reference
          ok = warp_wait(&o_full[mt], (steps - 1u) & 1u, abort_flag, c.status);
          if (!ok) break;
          tc_fence_after();
          const float f = grow ? ex2(r - m) : 1.f;
          l *= f;
          rescale_lane64(t_o, f);
          rescale_lane64(t_o + 64, f);
          tmem_wait_st();
        }
        if (grow) r = m;
        const float base = kBase - (r == -CUDART_INF_F ? 0.f : r);
#pragma unroll
        for (int b = 0; b < kPieces; ++b) {
          const float kf = qf * ti.kf[b], add = base + ti.lv[b];
          const uint64_t kf2 = f32x2(kf, kf), add2 = f32x2(add, add);
          uint64_t sum = 0;
          const uint32_t* v = &s[b >> 1][(b & 1) * 16];
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            float z0, z1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), kf2, add2), z0, z1);
            const float p0 = ex2(z0), p1 = ex2(z1);
            sum = add_f32x2(sum, f32x2(p0, p1));
            // packed in place: weights of keys 2c and 2c + 1 in column c
            s[b >> 2][(b & 3) * 8 + (x >> 1)] = pack_f16x2(p0, p1);
          }
          float s0, s1;
          f32x2_split(sum, s0, s1);
          l = fmaf(s0 + s1, ti.un[b], l);
        }
#pragma unroll
        for (int w = 0; w < kKeys / 64; ++w) tmem_st32(t_s + 32 * w, s[w]);  // over the scores
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&p_full[mt]);
          mbar_arrive(&i_empty[slot]);
        }
      }
      n0 += tiles;
      // all of this M tile's scores are done: the next part's queries may come over these
      if (!kSplit && ok) {
        const Part* next = reader.peek(abort_flag, c.status);
        ok = next != nullptr;
        if (ok && next->nt) fetch_queries(*next);
      }
      // ---- the rows' outputs
      ok = ok && warp_wait(&o_full[mt], (steps - 1u) & 1u, abort_flag, c.status);
      if (!ok) break;
      tc_fence_after();
      const bool complete = g.i0 == 0 && g.i1 == g.nt;
      const size_t part = (size_t)(2 * (int)blockIdx.x + g.later) * kRows + (kSplit ? 0 : mt * kM) + row;
      uint16_t* out = a.out + ((size_t)(g.t0 + i_row) * c.Hq + head) * kHeadDim;
      // kSplit: M tile 1 puts its r and l, and its sums in two halves of the dims, where the queries were once both tiles'
      // scores are done with them; M tile 0 adds them to its own.  A row's 16-byte pieces are rotated by the row.
      // x_empty completes three times a part: for the first half, for the second, and for the next part's queries.
      float4* sums = reinterpret_cast<float4*>(smem + C::kQOff) + row * 16;
      float f = 1.f, f1 = 0.f;
      if (kSplit && mt == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(x_empty);
      }
      if (kSplit && mt == 1) *other_rl = make_float2(r, l);
      auto write = [&](int d, const float (&o)[32], float inv) {  // dims d .. d + 31 of this row
        if (complete) {
          if (kPass == 1 && live) {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<float4*>(a.out32 + ((size_t)(g.t0 + i_row) * c.Hq + head) * kHeadDim + d + y) =
                  make_float4(o[y] * inv, o[y + 1] * inv, o[y + 2] * inv, o[y + 3] * inv);
          } else if (live) {
#pragma unroll
            for (int y = 0; y < 32; y += 8)
              *reinterpret_cast<uint4*>(out + d + y) =
                  make_uint4(pack_bf16x2(o[y] * inv, o[y + 1] * inv), pack_bf16x2(o[y + 2] * inv, o[y + 3] * inv),
                             pack_bf16x2(o[y + 4] * inv, o[y + 5] * inv), pack_bf16x2(o[y + 6] * inv, o[y + 7] * inv));
          }
        } else {
#pragma unroll
          for (int y = 0; y < 32; y += 4)
            *reinterpret_cast<float4*>(part_o + part * kHeadDim + d + y) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
        }
      };
      float inv = l != 0.f ? 1.f / l : 0.f;
      if (!complete && !kSplit) part_rl[part] = make_float2(r, l);
#pragma unroll 1
      for (int d = 0; d < kHeadDim; d += 32) {
        uint32_t v[32];
        tmem_ld32_async(t_o + d, v);
        tmem_wait_ld();
        float o[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = __uint_as_float(v[y]);
        if (!kSplit) {
          write(d, o, inv);
          continue;
        }
        const int piece0 = (d & 32) / 4;
        if (mt == 1) {
          if ((d & 32) == 0) {
            ok = warp_wait(x_empty, (segs - 1u + (uint32_t)(d >> 6)) & 1u, abort_flag, c.status);
            if (!ok) break;
          }
#pragma unroll
          for (int y = 0; y < 8; ++y)
            sums[(piece0 + y) ^ (row & 15)] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          __syncwarp();
          if ((d & 32) && lane == 0) mbar_arrive(x_full);
        } else {
          if ((d & 32) == 0) {
            ok = warp_wait(x_full, xs & 1u, abort_flag, c.status);
            if (!ok) break;
          }
          if (d == 0) {
            const float2 rl = *other_rl;
            const float top = fmaxf(r, rl.x), ref = top == -CUDART_INF_F ? 0.f : top;
            f = ex2(r - ref);
            f1 = ex2(rl.x - ref);
            l = l * f + rl.y * f1;
            r = top;
            inv = l != 0.f ? 1.f / l : 0.f;
            if (!complete) part_rl[part] = make_float2(r, l);
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float4 w = sums[(piece0 + y) ^ (row & 15)];
            o[4 * y] = o[4 * y] * f + w.x * f1;
            o[4 * y + 1] = o[4 * y + 1] * f + w.y * f1;
            o[4 * y + 2] = o[4 * y + 2] * f + w.z * f1;
            o[4 * y + 3] = o[4 * y + 3] * f + w.w * f1;
          }
          write(d, o, inv);
          __syncwarp();
          if ((d & 32) && lane == 0) mbar_arrive(x_empty);
        }
        if (d & 32) ++xs;
      }
      if (!ok) break;
      if (kPass > 0 && live && (!kSplit || mt == 0)) {
        const size_t at = (size_t)(g.t0 + i_row) * c.Hq + head;
        if (complete) write_lse(a, at, r - kBase, l);
        else if (kPass == 1 && g.i0 == 0) mark_split(a, at);
      }
      tc_fence_before();
    }
    cp_async_wait<0>();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp < kTmaWarp) {
      // ---------------------------------------------------------- values: E4M3 -> f16, keys nobody sees -> zeros
      uint32_t n = 0;
      bool ok = true;
      // A warp has 32 tokens, eight (1 KB of codes) at a time, first the lower half of their dims, then the upper.  A lane has 16
      // dims of a token: four lanes are one token's, the next four that token's whose place in the eight differs by 5
      // (0 and 5, 1 and 4, ..): then eight lanes meet eight different banks in the reads (16-byte pieces c ^ place of a row)
      // as in the writes (pieces 2c ^ place and, after it, (2c + 1) ^ place).
      const int place = (lane >> 3) ^ ((lane & 4) ? 5 : 0), quad = lane & 3, tok0 = (warp - kValWarp) * 32 + place;
      const uint32_t from = tok0 * 128 + ((quad ^ place) << 4), to = tok0 * 128 + (((2 * quad) ^ place) << 4);
      while (ok && reader.next(g, abort_flag, c.status)) {
        for (int i = g.i0; i < g.i0 + C::tiles(g); ++i, ++n) {
          const int st = (int)(n % C::kVStages), slot = (int)(n % kInfos);
          ok = warp_wait3(&i_full[slot], (n / kInfos) & 1u, &v_full[st], (n / C::kVStages) & 1u, &v16_empty[n % C::kV16s],
                          ((n / C::kV16s) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) break;
          const uint32_t have = infos[slot].have;
          const int j0 = (g.tile0 + i) * kKeys;
          const uint8_t* src = smem + C::kVOff + st * kTileBytes;
          uint8_t* dst = smem + C::kV16Off + (n % C::kV16s) * C::kV16Bytes;
          const int end = kPass == 3 && j0 < g.own0 ? g.plen : g.hi;
          const bool whole = j0 >= g.lo && j0 + kKeys <= end && have == (1u << kPieces) - 1u;
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            uint4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const uint4*>(src + (from ^ ((y & 1) << 6)) + ((x + y) >> 1) * 1024);
            if (!whole) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int tok = tok0 + ((x + y) >> 1) * 8;
                if (j0 + tok < g.lo || j0 + tok >= end || !(have >> (tok >> 4) & 1u)) v[y] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint8_t* at = dst + (y & 1) * kTileBytes + ((x + y) >> 1) * 1024;
              *reinterpret_cast<uint4*>(at + to) = make_uint4(e4m3x2_f16x2(v[y].x & 0xFFFFu), e4m3x2_f16x2(v[y].x >> 16),
                                                              e4m3x2_f16x2(v[y].y & 0xFFFFu), e4m3x2_f16x2(v[y].y >> 16));
              *reinterpret_cast<uint4*>(at + (to ^ 16)) = make_uint4(e4m3x2_f16x2(v[y].z & 0xFFFFu), e4m3x2_f16x2(v[y].z >> 16),
                                                                     e4m3x2_f16x2(v[y].w & 0xFFFFu), e4m3x2_f16x2(v[y].w >> 16));
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v16_full[n % C::kV16s]);
            mbar_arrive(&v_empty[st]);
            mbar_arrive(&i_empty[slot]);
          }
        }
      }
    } else if (warp == kTmaWarp) {
      // ---------------------------------------------------------- TMA: lane = page of the tile
      const uint64_t pol = policy_evict_last();
      const int boxes = kKeys >> c.page_log2;
      const uint32_t box = kHeadDim << c.page_log2;
      uint32_t n = 0, nv = 0;
      bool ok = true;
      while (ok && reader.next(g, abort_flag, c.status)) {
        const int32_t* row = c.page_table + (size_t)g.b * c.max_pages;
        const int32_t* prefix = kPass == 3 ? a.prefix_table + (size_t)g.prefix * a.prefix_max_pages : nullptr;
        // page of this lane's box of tile i, read one tile ahead; -1: nothing to load
        auto page_at = [&](int i) {
          const int j = (g.tile0 + i) * kKeys + (lane << c.page_log2);
          if (kPass == 3) {
            if (lane >= boxes || i >= g.i1) return -1;
            if (j < g.own0) return j < g.plen ? __ldg(prefix + (j >> c.page_log2)) : -1;
            return j < g.hi ? __ldg(row + ((j - g.own0) >> c.page_log2)) : -1;
          }
          return lane < boxes && i < g.i1 && j + c.page > g.lo && j < g.hi ? __ldg(row + (j >> c.page_log2)) : -1;
        };
        int pg = page_at(g.i0);
        for (int i = g.i0; i < g.i0 + C::tiles(g); ++i) {
          const int next = page_at(i + 1);
          const bool have = pg >= 0 && pg < c.n_pages;
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, have)) * box;
          const int y = have ? (int)(((long long)pg * c.Hkv + g.h) << c.page_log2) : 0;
          const int ks = (int)(n % C::kKStages), vs = (int)(nv % C::kVStages);
          ok = warp_wait(&k_empty[ks], ((n / C::kKStages) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], bytes);
          __syncwarp();
          if (have) tma_load_2d(smem + C::kKOff + ks * kTileBytes + lane * box, &tm_k, 0, y, &k_full[ks], pol);
          ++n;
          ok = warp_wait(&v_empty[vs], ((nv / C::kVStages) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], bytes);
          __syncwarp();
          if (have && !a.withhold) tma_load_2d(smem + C::kVOff + vs * kTileBytes + lane * box, &tm_v, 0, y, &v_full[vs], pol);
          ++nv;
          pg = next;
        }
      }
      // every copy lands before the block ends
      if (lane == 0) {
        for (int st = 0; st < C::kKStages; ++st) {
          const uint32_t fills = n / C::kKStages + ((uint32_t)st < n % C::kKStages ? 1u : 0u);
          if (fills) mbar_wait_bounded(&k_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
        }
        for (int st = 0; st < C::kVStages; ++st) {
          const uint32_t fills = nv / C::kVStages + ((uint32_t)st < nv % C::kVStages ? 1u : 0u);
          if (fills) mbar_wait_bounded(&v_full[st], (fills - 1u) & 1u, abort_flag, 1000ull * a.limit_us, c.status, false);
        }
      }
      __syncwarp();
    } else if (warp == kScaleWarp) {
      // ---------------------------------------------------------- scales: lane = 16 keys of the tile
      // It also walks the run, and gives the others its parts.
      Walk<kRows, kPass> walk(c, a, G, run, s_begin[0], s_begin[1], s_begin[2]);
      uint32_t n = 0;
      bool ok = true;
      for (uint32_t np = 0; ok; ++np) {
        const int at = (int)(np % kParts);
        const bool more = walk.next(g);
        if (!warp_wait(&r_empty[at], ((np / kParts) & 1u) ^ 1u, abort_flag, c.status)) break;
        if (lane == 0) {
          parts[at] = g;
          mbar_arrive(&r_full[at]);
        }
        __syncwarp();
        if (!more) break;
        const int32_t* row = c.page_table + (size_t)g.b * c.max_pages;
        const int32_t* prefix = kPass == 3 ? a.prefix_table + (size_t)g.prefix * a.prefix_max_pages : nullptr;
        auto page_at = [&](int i) {
          const int j = (g.tile0 + i) * kKeys + (lane & (kPieces - 1)) * 16;
          const bool in_prefix = kPass == 3 && j < g.own0;
          const bool in = i < g.i1 && j + 15 >= g.lo && j < (in_prefix ? g.plen : g.hi);
          const int p = !in ? -1 : in_prefix ? __ldg(prefix + (j >> c.page_log2)) : __ldg(row + ((kPass == 3 ? j - g.own0 : j) >> c.page_log2));
          if (in && (p < 0 || p >= c.n_pages)) set_status(c.status, DEV_ERR_BOUNDS);
          return p < c.n_pages ? p : -1;
        };
        int pg = page_at(g.i0);
        for (int i = g.i0; i < g.i0 + C::tiles(g); ++i, ++n) {
          const int slot = (int)(n % kInfos);
          uint32_t sk = 127, sv = 127;
          if (pg >= 0) {
            const size_t u = (size_t)pg * c.Hkv + g.h;
            sk = __ldg(c.k_scale + u);
            sv = __ldg(c.v_scale + u);
          }
          const int next = page_at(i + 1);
          const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0) & ((1u << kPieces) - 1u);
          ok = warp_wait(&i_empty[slot], ((n / kInfos) & 1u) ^ 1u, abort_flag, c.status);
          if (!ok) break;
          if (lane < kPieces) {
            infos[slot].kf[lane] = exp2_byte(sk);
            infos[slot].lv[lane] = (float)((int)sv - 127);
            infos[slot].un[lane] = ex2((float)(127 - (int)sv));
            if (lane == 0) infos[slot].have = have;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&i_full[slot]);
          pg = next;
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA.  The whole warp walks along and one lane issues, so that
      // descriptors stay in uniform registers: with one diverged thread an instruction took ~110 cycles to issue, and one
      // of this size runs for 64.  The order PV0 QK0 PV1 QK1 keeps the M tiles half a turn apart.  A product that
      // overwrites S starts after the one before it in the stream that reads p' there.
      const uint32_t id_s = umma_idesc_e4m3(kM, kKeys, false, false), id_o = idesc_pv();
      const uint64_t desc = umma_desc_sw128(smem_u32(smem));
      // V16: 64-dim halves kTileBytes apart (leading), groups of 8 tokens 1 KB apart (stride)
      const uint64_t vdesc = (desc & ~((uint64_t)0x3FFFu << 16)) | (uint64_t)(kTileBytes >> 4) << 16;
      uint32_t n0 = 0, steps0 = 0, segs = 0;
      bool ok = true;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      while (ok && reader.next(g, abort_flag, c.status)) {
        const int tiles = __shfl_sync(0xffffffffu, C::tiles(g), 0), steps = tiles / C::kStep;
        // Step i: the weights of an M tile's i-th tile against V (from i = 0 on), then the scores of its next one.  One copy
        // of either's instructions for all steps and M tiles.
#pragma unroll 1
        for (int i = -1; ok && i < steps; ++i) {
          const bool more = i + 1 < steps;
#pragma unroll 1
          for (int mt = 0; ok && mt < 2; ++mt) {
            // number of the tile whose weights, whose scores are next
            const uint32_t tp = n0 + i * C::kStep + (kSplit ? mt : 0), tn = tp + C::kStep;
            if (kSplit || mt == 0) {
              uint64_t *v = &v16_full[tp % C::kV16s], *k = &k_full[tn % C::kKStages];
              const uint32_t vp = (tp / C::kV16s) & 1u, kp = (tn / C::kKStages) & 1u;
              ok = i < 0 ? warp_wait(k, kp, abort_flag, c.status) : warp_wait2(v, vp, more ? k : v, more ? kp : vp, abort_flag, c.status);
            }
            const uint32_t s_at = tm + mt * kTile;
            if (i >= 0) {
              ok = ok && warp_wait(&p_full[mt], (steps0 + i) & 1u, abort_flag, c.status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t o = tm + 256 + mt * kHeadDim;
              const uint64_t bd = vdesc + (uint64_t)((C::kV16Off + (tp % C::kV16s) * C::kV16Bytes) >> 4);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  umma_f16_ts(o, s_at + 8 * k, bd + (uint64_t)((k * 16 * 128) >> 4), id_o, k > 0 || i > 0);
                umma_commit(&o_full[mt]);
                if (kSplit || mt == 1) umma_commit(&v16_empty[tp % C::kV16s]);
              }
              __syncwarp();
            } else {
              ok = ok && warp_wait(&q_full[kSplit ? 0 : mt], segs & 1u, abort_flag, c.status);
              if (!ok) break;
              tc_fence_after();
            }
            if (more) {
              const uint64_t bd = desc + (uint64_t)((C::kKOff + (tn % C::kKStages) * kTileBytes) >> 4);
              const uint64_t ad = desc + (uint64_t)((C::kQOff + (kSplit ? 0 : mt * 2 * kTileBytes)) >> 4);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 2 * kHeadDim / 32; ++k)  // the hi half of the queries, then the lo half
                  umma_e4m3(s_at, ad + (k >> 2) * (kTileBytes >> 4) + 2 * (k & 3), bd + 2 * (k & 3), id_s, k != 0);
                umma_commit(&s_full[mt]);
                if (kSplit || mt == 1) umma_commit(&k_empty[tn % C::kKStages]);
              }
              __syncwarp();
            }
          }
        }
        n0 += tiles;
        steps0 += steps;
        ++segs;
      }
      // whatever was issued has finished before tensor memory is given back (after an abort too)
      if (elect_one()) umma_commit(done);
      __syncwarp();
      mbar_wait_bounded(done, 0, abort_flag, 1000ull * a.limit_us, c.status, false);
    }
  }
  if (kPass == 1) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kSplit, int kPass>
cudaError_t launch(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream, AttentionParts* parts) {
  using C = Cfg<kSplit>;
  CUtensorMap tk, tv;
  if (!make_cache_map(&tk, c.k_codes, c) || !make_cache_map(&tv, c.v_codes, c)) return cudaErrorInvalidValue;
  auto kern = attention_prefill_kernel<kSplit, kPass>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kBytes, allowed);
  if (e != cudaSuccess) return e;
  float* part_o = reinterpret_cast<float*>(a.scratch);
  float2* part_rl = reinterpret_cast<float2*>(part_o + (size_t)n_sms * 2 * C::kRows * kHeadDim);
  JoinInfo* info = reinterpret_cast<JoinInfo*>(part_rl + (size_t)n_sms * 2 * C::kRows);
  e = launch_kernel(kern, dim3(n_sms), dim3(kThreads), C::kBytes, stream, kPass == 1 && a.follows, tk, tv, c, a, part_o, part_rl, info);
  const AttentionParts p = {n_sms, C::kRows, kBase, part_o, part_rl, info};
  if (kPass == 1) *parts = p;
  if (kPass == 1 || e != cudaSuccess) return e;
  return launch_attention_join(c, a, p, stream);
}

// Whether a sequence's rows of one head fit an M tile: it is then the keys that the two tiles share out.
bool splits_keys(int G, int max_q) { return (long long)G * max_q <= kM; }

}  // namespace

size_t attention_prefill_scratch(int G, int max_q, int n_sms) {
  const int rows = splits_keys(G, max_q) ? Cfg<true>::kRows : Cfg<false>::kRows;
  return (size_t)n_sms * (2 * rows * (kHeadDim * sizeof(float) + sizeof(float2)) + sizeof(JoinInfo));
}

cudaError_t launch_attention_prefill(const KvBatch& c, const AttentionArgs& a, int n_sms, cudaStream_t stream, AttentionParts* parts) {
  const bool split = splits_keys(c.Hq / c.Hkv, a.max_q);
  if (a.pass == 0) return split ? launch<true, 0>(c, a, n_sms, stream, parts) : launch<false, 0>(c, a, n_sms, stream, parts);
  if (a.pass == 1) return split ? launch<true, 1>(c, a, n_sms, stream, parts) : launch<false, 1>(c, a, n_sms, stream, parts);
  if (a.pass == 3) return launch<false, 3>(c, a, n_sms, stream, parts);
  return split ? launch<true, 2>(c, a, n_sms, stream, parts) : launch<false, 2>(c, a, n_sms, stream, parts);
}

}  // namespace moe
