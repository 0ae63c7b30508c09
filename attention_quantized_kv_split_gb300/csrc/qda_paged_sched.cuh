// How a paged attention call is shared among its CTAs (sm_103a), from lengths that only the device knows.
//
// The rows of a sequence under one KV head, r = i * nrep + j for new token i and the head's query head j, are cut into
// tiles of MT rows; a tile walks the keys that its last row sees. All (sequence, unit, tile) triples in that order (a unit is a KV head, or
// for a kernel that cannot hold a head's values at once, a KV head and a part of its values)
// form one line, each with a length in keys: exact for cross attention, linear in the tile's index for causal attention (plus a constant for a
// tile's fixed work). CTA c takes the c-th of `ctas` equal pieces of the line, so ragged lengths, chunks and single
// tokens are balanced alike, whatever they are. A piece border inside a tile falls on the border of a key block in proportion; the tile's partial
// results are merged in CTA order, so results do not depend on timing. Every CTA (and the merge) finds its piece by itself: a scan
// over the B lengths, then closed forms.
#pragma once

#include "qda_paged.h"
#include "qda_ptx.cuh"

namespace qda {

// Keys of a tile's fixed work (its query rows, its epilogue) on the line.
constexpr int kTileCost = 64;

struct PagedSeq {
  int rows, tiles, n_all, first;   // query rows and tiles, keys, first token's row in q
  int base;                        // causal: keys before the first new token (may be negative); cross: keys
  long long step2;                 // causal: MT (keys grow by step2 / nrep a tile); cross: 0
};

__device__ __forceinline__ PagedSeq paged_seq(const QdaPagedParams& p, int b, int MT) {
  PagedSeq s;
  const int q0 = min(max(p.q_start[b], 0), p.total_q), q1 = min(max(p.q_start[b + 1], q0), p.total_q);
  const long long cap = (long long)p.max_pages << p.page_shift;
  const int n = max(p.kv_len[b], 0);
  s.first = q0;
  s.rows = (q1 - q0) * p.nrep;
  s.tiles = (s.rows + MT - 1) / MT;
  s.n_all = (int)min((long long)n, cap);
  s.base = p.causal ? n - (q1 - q0) : s.n_all;
  s.step2 = p.causal ? MT : 0;
  return s;
}

// Keys that row r of the sequence sees.
__device__ __forceinline__ int paged_seen(const QdaPagedParams& p, const PagedSeq& s, int r) {
  return p.causal ? max(0, min(s.n_all, s.base + r / p.nrep + 1)) : s.n_all;
}

// Length of the sequence's first i tiles (of one unit) on the line.
__device__ __forceinline__ long long paged_prefix(const QdaPagedParams& p, const PagedSeq& s, long long i) {
  return i * (kTileCost + max(s.base, 0)) + s.step2 * (i * (i + 1) / 2) / p.nrep;
}

// The line's per-sequence starts, in shared memory: line[b] for b <= B.
struct PagedLine {
  long long at[QDA_MAX_B + 1];
  long long warp_tot[32];
};

// Scan of the sequences' lengths on the line; every thread of the CTA calls it (ends with a barrier).
__device__ __forceinline__ void paged_line(const QdaPagedParams& p, int MT, PagedLine& line) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  long long carry = 0;
  if (tid == 0) line.at[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += nt) {
    const int b = b0 + tid;
    long long v = 0;
    if (b < p.B) {
      const PagedSeq s = paged_seq(p, b, MT);
      v = p.units * paged_prefix(p, s, s.tiles);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) line.warp_tot[warp] = v;
    __syncthreads();
    long long before = carry, all = carry;
    for (int w = 0; w < (nt + 31) / 32; ++w) {
      if (w < warp) before += line.warp_tot[w];
      all += line.warp_tot[w];
    }
    if (b < p.B) line.at[b + 1] = before + v;
    carry = all;
    __syncthreads();
  }
}

// CTAs that share the line: as many as there are, but no piece shorter than min_keys.
__device__ __forceinline__ int paged_ctas(long long total, int ctas, int min_keys) {
  return (int)max(1LL, min((long long)ctas, total / min_keys));
}

__device__ __forceinline__ long long paged_border(long long total, int ctas, int c) { return total / ctas * c + total % ctas * c / ctas; }

// A tile on the line.
struct PagedTile {
  int b, unit, i;       // sequence, unit (KV head, or a part of its values), tile of the sequence
  long long lo, hi;     // its place on the line
  PagedSeq s;
};

// The tile that holds place x of the line (0 <= x < line.at[B]).
__device__ __forceinline__ PagedTile paged_tile_at(const QdaPagedParams& p, const PagedLine& line, int MT, long long x) {
  PagedTile t;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {   // sequences without rows have no length: the last start at or below x holds x
    const int mid = (lo + hi) >> 1;
    if (line.at[mid] <= x) lo = mid; else hi = mid;
  }
  t.b = lo;
  t.s = paged_seq(p, lo, MT);
  const long long head = paged_prefix(p, t.s, t.s.tiles);
  const long long y = x - line.at[lo];
  t.unit = (int)(y / head);
  const long long z = y - t.unit * head;
  int a = 0, e = t.s.tiles;
  while (e - a > 1) {
    const int mid = (a + e) >> 1;
    if (paged_prefix(p, t.s, mid) <= z) a = mid; else e = mid;
  }
  t.i = a;
  const long long at = line.at[lo] + t.unit * head;
  t.lo = at + paged_prefix(p, t.s, t.i);
  t.hi = at + paged_prefix(p, t.s, t.i + 1);
  return t;
}

// The next tile on the line; false behind the last. Tiles are contiguous on the line, so it starts where this one ends.
__device__ __forceinline__ bool paged_tile_next(const QdaPagedParams& p, int MT, PagedTile& t) {
  if (++t.i >= t.s.tiles) {
    t.i = 0;
    if (++t.unit >= p.units) {
      t.unit = 0;
      do {
        if (++t.b >= p.B) return false;
        t.s = paged_seq(p, t.b, MT);
      } while (t.s.tiles == 0);
    }
  }
  t.lo = t.hi;
  t.hi = t.lo + paged_prefix(p, t.s, t.i + 1) - paged_prefix(p, t.s, t.i);
  return true;
}

// Keys that a tile walks: what its last row sees.
__device__ __forceinline__ int paged_tile_keys(const QdaPagedParams& p, const PagedTile& t, int MT) {
  return paged_seen(p, t.s, min((t.i + 1) * MT, t.s.rows) - 1);
}

// Key block at place x of a tile of nblk blocks.
__device__ __forceinline__ int paged_block_at(const PagedTile& t, int nblk, long long x) {
  if (x <= t.lo) return 0;
  if (x >= t.hi) return nblk;
  return (int)((x - t.lo) * nblk / (t.hi - t.lo));
}

}  // namespace qda
