// How a paged attention call is shared among its CTAs (sm_103a), from lengths that only the device knows.
//
// The rows of a sequence under one KV head, r = i * nrep + j for new token i and the head's query head j, are cut into
// tiles of MT rows; a tile walks the keys that its last row sees. All (sequence, unit, tile) triples in that order (a unit
// is a KV head, or for a kernel that cannot hold a head's values at once, a KV head and a part of its values) form one
// line, each with a length in keys: exact for cross attention, linear in the tile's index for causal attention (plus a
// constant for a tile's fixed work). CTA c takes the c-th of `ctas` equal pieces of the line, so ragged lengths, chunks and
// single tokens are balanced alike, whatever they are. A piece border inside a tile falls on the border of a key block in
// proportion; the tile's partial results are merged in CTA order, so results do not depend on timing. Every CTA finds its
// piece by itself: a scan over the B lengths, then closed forms.
#pragma once

#include "qda_paged.h"
#include "qda_ptx.cuh"

namespace qda {

// A tile's fixed work (its query rows, its results), in keys. Chunk kernel (tiles of 128 rows or more): ragged chunks of 1
// to 1023 tokens at D = 256 take 470 us with 300, 451 with 448, 427 with 700, 432 with 900, 437 with 1600, cross attention
// at D = 64 65.6, 65.5, 64.1, 66.1 and 65.8 us: anything from 700 to 1200 will do. Split kernel: over fourteen sets of
// lengths each (medians, us, with 100, 160, 250, 400, 700) one token of each of 64 sequences at D = 128 takes 99.4, 98.2,
// 96.9, 96.9 and 98.6, one to four tokens of 24 short sequences 37.4, 35.6, 33.6, 33.4 and 33.3, one sequence of about 130000
// keys at D = 256 60.0 with all, other shapes within 1 %: anything from 250 to 400 will do. Single lengths differ by luck
// (131072 keys: 55 with 250 or 350, 58 with 240, 256, 300 or 400): the cost is spread over a tile's blocks, so a border just
// behind a tile's start hands one or two blocks to a CTA that pays the whole cost for them.
__device__ __forceinline__ constexpr int paged_tile_cost(int MT) { return MT >= 128 ? 700 : 250; }

struct PagedSeq {
  int rows, tiles, n_all, first;   // query rows and tiles, keys, first token's row in q
  int base;                        // causal: keys before the first new token (may be negative); cross: keys
};

// Sequence b from its first token's row, the next sequence's and its number of keys.
__device__ __forceinline__ PagedSeq paged_seq(const QdaPagedParams& p, int start, int end, int n, int MT) {
  PagedSeq s;
  const int q0 = min(max(start, 0), p.total_q), q1 = min(max(end, q0), p.total_q);
  n = max(n, 0);
  s.first = q0;
  s.rows = (q1 - q0) * p.nrep;
  s.tiles = (s.rows + MT - 1) / MT;
  // (sums with a block's keys stay in range)
  s.n_all = (int)min(min((long long)n, (long long)p.max_pages << p.page_shift), 0x7ffffe00LL);
  s.base = p.causal ? n - (q1 - q0) : s.n_all;
  return s;
}
__device__ __forceinline__ PagedSeq paged_seq(const QdaPagedParams& p, int b, int MT) {
  return paged_seq(p, p.q_start[b], p.q_start[b + 1], p.kv_len[b], MT);
}

// Keys that row r of the sequence sees.
__device__ __forceinline__ int paged_seen(const QdaPagedParams& p, const PagedSeq& s, int r) {
  return p.causal ? max(0, min(s.n_all, s.base + r / p.nrep + 1)) : s.n_all;
}

// Length of the sequence's first i tiles (of one unit) on the line, in keys times nrep: no division. Keys and a tile's
// fixed work are added without a sign: lengths up to INT_MAX (which may lie) keep the line ascending.
__device__ __forceinline__ long long paged_prefix(const QdaPagedParams& p, const PagedSeq& s, int MT, int i) {
  const long long flat = (long long)i * (((uint32_t)paged_tile_cost(MT) + (uint32_t)max(s.base, 0)) * (long long)p.nrep);
  return p.causal ? flat + (long long)MT * ((long long)i * (i + 1) / 2) : flat;
}

// a / b for b > 0; 64-bit division only where it is needed.
__device__ __forceinline__ long long paged_div(unsigned long long a, unsigned long long b) {
  if ((a | b) >> 32) return (long long)(a / b);
  return (uint32_t)a / (uint32_t)b;
}

// The line's per-sequence starts and the sequences' lengths, in shared memory.
struct PagedLine {
  long long at[QDA_MAX_B + 1];
  int start[QDA_MAX_B + 1], n[QDA_MAX_B];
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
      const int q0 = p.q_start[b], q1 = p.q_start[b + 1], n = p.kv_len[b];
      line.start[b] = q0;
      if (b + 1 == p.B) line.start[p.B] = q1;
      line.n[b] = n;
      const PagedSeq s = paged_seq(p, q0, q1, n, MT);
      v = p.units * paged_prefix(p, s, MT, s.tiles);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    const bool one = p.B - b0 <= 32;   // the first warp holds all there is
    if (!one && lane == 31) line.warp_tot[warp] = v;
    if (!one) __syncthreads();
    long long before = carry, all = carry;
    if (!one) {
      for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += line.warp_tot[w];
        all += line.warp_tot[w];
      }
    }
    if (b < p.B) line.at[b + 1] = before + v;
    carry = all;
    __syncthreads();
  }
}

// The pieces of the line: equal, but none shorter than min_keys.
struct PagedPieces {
  long long total, piece;
  int ctas;   // pieces that there are
};
__device__ __forceinline__ PagedPieces paged_pieces(const QdaPagedParams& p, long long total) {
  PagedPieces c;
  c.total = total;
  c.piece = max(paged_div(total + p.ctas - 1, p.ctas), (long long)p.min_keys * p.nrep);
  c.ctas = (int)paged_div(total + c.piece - 1, c.piece);
  return c;
}
__device__ __forceinline__ long long paged_border(const PagedPieces& c, int k) { return min(c.total, k * c.piece); }

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
  t.s = paged_seq(p, line.start[lo], line.start[lo + 1], line.n[lo], MT);
  const long long head = paged_prefix(p, t.s, MT, t.s.tiles);
  const long long y = x - line.at[lo];
  t.unit = (int)paged_div(y, head);
  const long long z = y - t.unit * head;
  int a = 0, e = t.s.tiles;
  while (e - a > 1) {
    const int mid = (a + e) >> 1;
    if (paged_prefix(p, t.s, MT, mid) <= z) a = mid; else e = mid;
  }
  t.i = a;
  const long long at = line.at[lo] + t.unit * head;
  t.lo = at + paged_prefix(p, t.s, MT, t.i);
  t.hi = at + paged_prefix(p, t.s, MT, t.i + 1);
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
  t.hi = t.lo + paged_prefix(p, t.s, MT, t.i + 1) - paged_prefix(p, t.s, MT, t.i);
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
  return (int)paged_div((unsigned long long)(x - t.lo) * nblk, t.hi - t.lo);   // below 2^31 * 2^6 * 2^27
}

// Behind CTA k's part [j0, j1) of tile t (one thread): what the merge has to know of the tile, if it starts in piece k and
// goes on behind it, and which of the CTA's two slots it has filled.
__device__ __forceinline__ void paged_record(const QdaPagedParams& p, const PagedPieces& c, const PagedTile& t, int MT,
                                             int nblk, int j0, int j1, int k) {
  QdaPagedSplitTile& r = p.split[k];
  const bool mine = paged_border(c, k) <= t.lo;
  const bool filled = j0 < j1 && !(j0 == 0 && j1 == nblk);
  if (!mine) {
    r.first_filled = filled;
    return;
  }
  bool go = t.hi > paged_border(c, k + 1) && nblk > 0 && j1 < nblk;
  // a CTA behind this one may have had every block (and written the tile itself)
  for (int x = k + 1; go && x < c.ctas && paged_border(c, x) < t.hi; ++x) {
    const int e = paged_block_at(t, nblk, paged_border(c, x + 1));
    if (j1 == 0 && e == nblk) go = false;
    if (e > 0) break;
  }
  r.last_filled = filled;
  if (!go) return;
  r.go = 1;
  r.last = min((int)paged_div(t.hi - 1, c.piece), c.ctas - 1);
  r.row0 = t.i * MT;
  r.rows = min(MT, t.s.rows - t.i * MT);
  r.token0 = t.s.first;
  r.unit = t.unit;
}

}  // namespace qda
