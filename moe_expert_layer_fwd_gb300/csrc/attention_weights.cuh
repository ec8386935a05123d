// What the two kernels that add up attention weights share: the distribution of (sequence, head, tile) over blocks, and the chunks of
// query rows that a tile of keys is multiplied with.
#pragma once

#include "attention_tiles.cuh"

#include <limits.h>

namespace moe {

struct RowSeen {     // the keys lo .. lo + span that a row sees
  int lo;
  unsigned span;
};

// Tiles [i0, i1) of one (sequence, head), and the chunks of its rows.
struct WeightSegment {
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
struct WeightWalk {
  const KvBatch& c;
  const AttentionArgs& a;
  int G;
  long long at, left;  // where the run begins in the present (sequence, head); how much of it is left
  int b, h;
  __device__ WeightWalk(const KvBatch& c_, const AttentionArgs& a_, int G_, long long n, int b_, int h_, long long at_)
      : c(c_), a(a_), G(G_), at(at_), left(n), b(b_), h(h_) {}
  __device__ bool next(WeightSegment& g) {
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
__device__ __forceinline__ void chunks_of(const WeightSegment& g, const AttentionArgs& a, int G, int nc, int j0, int j1, int& c0, int& c1) {
  c0 = 0;
  c1 = g.chunks - 1;
  if (g.chunks == 1) return;
  const int first = g.s.first(), last = g.s.t1 - g.s.t0 - 1;  // new token i has position first + i; rows are below 2^31
  if (a.causal) c0 = (int)((unsigned)(min(max(0, j0 - first), last) * G) / (unsigned)nc);
  if (a.window > 0) {
    // token i sees keys from first + i - window + 1 on: the last one that sees j1 - 1
    const long long i = (long long)j1 - 1 - first + a.window - 1;
    c1 = (int)((unsigned)((i < 0 ? 0 : i > last ? last : (int)i) * G + G - 1) / (unsigned)nc);
    c1 = max(c0, min(c1, g.chunks - 1));
  }
}

// This block's run of tiles: `run` of cost from *s_at on in (sequence s_begin[0], head s_begin[1]); false when there is none.  s_warp: scratch
// of a long long a warp.
template <int NC>
__device__ __forceinline__ bool weight_run(const KvBatch& c, const AttentionArgs& a, int G, int threads, long long* s_warp, long long& run,
                                           int* s_begin, long long* s_at) {
  auto cost = [&](int b) { return seq_cost<NC>(c, a, G, b); };
  long long mine, total;
  const long long before = scan_batch(c, threads, s_warp, mine, total, cost);
  const long long all = total * c.Hkv, per = max(1LL, (all + gridDim.x - 1) / (long long)gridDim.x);
  const long long begin = (long long)blockIdx.x * per;
  run = min(per, all - begin);
  if (run <= 0) return false;
  if (before * c.Hkv <= begin && begin < (before + mine) * c.Hkv) {
    long long at = before, u;
    int b = (int)threadIdx.x * ((c.B + threads - 1) / threads);
    while ((at + (u = cost(b))) * c.Hkv <= begin) {
      at += u;
      ++b;
    }
    const long long rel = begin - at * c.Hkv;
    s_begin[0] = b;
    s_begin[1] = (int)(rel / u);
    *s_at = rel % u;
  }
  return true;
}

// More than 16 query rows per key/value head.
cudaError_t launch_kv_weights_many(const KvBatch& c, const AttentionArgs& a, const float* lse, const float* weight_in, float* weight_out,
                                   int n_sms, cudaStream_t stream);

}  // namespace moe
