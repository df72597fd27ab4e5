// mx_chunk_plan.cuh -- how the chunk attention's work is cut and shared out.
// The lengths are device data, so every block derives the same plan from them.
//
// A sequence's new tokens times the G query heads of a KV head are its rows
// (row r: token r / G, head r % G); tile_rows consecutive ones make a query
// tile, which sees the key tiles of kKeys tokens that its mask reaches.  All
// query tiles in a row (sequence, KV head, query tile), each worth
//   tile + its key tiles * (kPairCost above 128 rows, else kHalfCost)
// units (tile: what it costs besides its keys, queries in and outputs out), are
// cut into `blocks` equal ranges of units, one a block.  A block so does the end
// of one query tile, some whole ones and the beginning of another: the work is
// even whatever the lengths are, a long cache with few rows spreads over the
// whole GPU, and a block leaves at most two partial results, however many rows
// there are.  (Where the query tiles are not more
// than the blocks, and the longest is not much longer than an equal share, each
// is one block's instead, and worth one unit: nothing has to be merged then.)
#pragma once
#include "mx_chunk.h"
#include "mx_device.cuh"

namespace fsops {
namespace chunk {

constexpr int kKeys = 112;     // tokens of a key tile
constexpr int kPairCost = 8;   // a key tile against two halves of 128 rows
constexpr int kHalfCost = 5;   // a key tile against one

struct Seq {
  int n, len;  // new tokens, length with them (n = 0: nothing to do or not valid)
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const ChunkArgs& a, int b) {
  Seq s;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  s.len = __ldg(a.lens + b);
  s.n = c1 - c0;
  s.bad = c0 < 0 || c1 < c0 || c1 > a.T ||
          (s.n > 0 && (s.len < s.n || static_cast<long long>(s.len) > (static_cast<long long>(a.max_pages) << a.log2P)));
  if (s.bad) s.n = 0;
  return s;
}

// A sequence's query tiles one after another, without divisions.
struct Tiles {
  int j, R;            // tile, rows of the sequence
  int f, fr;           // first row = f * G + fr
  int qs, rs;          // tile_rows / G and the rest
  int base;            // len - n: token of row 0
  int n;
  __device__ __forceinline__ void start(const ChunkArgs& a, const Seq& s, int qs_, int rs_) {
    j = f = fr = 0;
    qs = qs_, rs = rs_;
    R = s.n * a.G;
    n = s.n;
    base = s.len - s.n;
  }
  __device__ __forceinline__ bool more(const ChunkArgs& a) const { return j * a.tile_rows < R; }
  // tokens [lo, hi) seen, key tiles from tb, nt of them, rows of the tile
  __device__ __forceinline__ void get(const ChunkArgs& a, int& lo, int& hi, int& tb, int& nt, int& rows) const {
    int nf = f + qs, nr = fr + rs;
    if (nr >= a.G) nr -= a.G, ++nf;
    const int last = min(n - 1, nr == 0 ? nf - 1 : nf);
    rows = min(a.tile_rows, R - j * a.tile_rows);
    hi = base + last + 1;
    lo = a.window > 0 ? max(0, base + f - a.window + 1) : 0;
    tb = lo / kKeys;
    nt = (hi + kKeys - 1) / kKeys - tb;
  }
  __device__ __forceinline__ void next(const ChunkArgs& a) {
    f += qs, fr += rs;
    if (fr >= a.G) fr -= a.G, ++f;
    ++j;
  }
};
__device__ __forceinline__ int key_cost(int rows) { return rows > 128 ? kPairCost : kHalfCost; }
struct Units {
  int tile;  // of a query tile besides its keys
  int one;   // a query tile is one unit, whatever its keys
};
__device__ __forceinline__ long long tile_units(int nt, int rows, const Units& v) {
  return v.one ? 1 : v.tile + static_cast<long long>(nt) * key_cost(rows);
}
// Units of one KV head of a sequence; the most that a query tile has joins `most`.
__device__ __forceinline__ long long seq_units(const ChunkArgs& a, const Seq& s, int qs, int rs, const Units& v,
                                               long long& most) {
  long long u = 0;
  Tiles t;
  for (t.start(a, s, qs, rs); t.more(a); t.next(a)) {
    int lo, hi, tb, nt, rows;
    t.get(a, lo, hi, tb, nt, rows);
    const long long x = tile_units(nt, rows, v);
    u += x;
    most = max(most, x);
  }
  return u;
}
// Key tiles of a query tile (nt of them, cost w each) that lie before unit y of it.
__device__ __forceinline__ int tiles_before(long long y, int nt, int w, const Units& v) {
  if (v.one) return y > 0 ? nt : 0;
  if (y <= v.tile) return 0;
  y += w - 1 - v.tile;
  const long long t = w == kPairCost ? y / kPairCost : y / kHalfCost;
  return t < nt ? static_cast<int>(t) : nt;
}

// The ranges of the blocks: block c has units [start(c), start(c + 1)).
struct Ranges {
  long long each;
  int more, blocks;  // the first `more` blocks have one unit more
  Units v;
  // for `tiles` query tiles of `most` units at most, whose parts cost `part_cost`
  // to write and merge; a block has at least `least`
  __device__ __forceinline__ void make(long long units, long long tiles, long long most, int grid, int part_cost, int least) {
    long long b = units / least;
    v.one = tiles <= grid && tiles > 0 && most <= units / max(min(b, static_cast<long long>(grid)), 1LL) + 2 * part_cost;
    if (v.one) b = units = tiles;
    blocks = b < 1 ? 1 : b < grid ? static_cast<int>(b) : grid;
    each = units / blocks;
    more = static_cast<int>(units - each * blocks);
  }
  __device__ __forceinline__ long long start(int c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int block_of(long long x) const {
    const long long cut = (each + 1) * more;
    return x < cut ? static_cast<int>(x / (each + 1)) : more + static_cast<int>((x - cut) / each);
  }
};

// One block's part of a query tile.
struct Item {
  int b, hk, n, len, c0;  // sequence, KV head, new tokens, length, first row of the sequence in q and out
  int r0, rows;           // first row of the tile, its rows
  int lo, hi;             // tokens some row of the tile sees
  int t0, t1;             // key tiles of this part (t0 == t1: no more work)
  int whole;              // the part is the whole tile
  int tb, nt;             // key tiles of the tile
  int first, last;        // blocks that have a share of the tile
  int parts;              // how many of them have a key tile
  int slot;               // where the part's results go (unless it is the whole tile)
  long long x;            // unit at which the tile begins
};
// Block c's part of the tile: its slot, or -1 when it has no key tile.
__device__ __forceinline__ int part_slot(const Item& w, const Ranges& r, int c) {
  const long long s = r.start(c), e = r.start(c + 1);
  const int kc = key_cost(w.rows);
  if (tiles_before(e - w.x, w.nt, kc, r.v) <= tiles_before(s - w.x, w.nt, kc, r.v)) return -1;
  return 2 * c + (s >= w.x ? 0 : 1);  // the tile that a block begins with, else the one it ends with
}

// Block-wide: the ranges; reports sequences that are not valid.  red: three values a warp.
__device__ inline void make_ranges(const ChunkArgs& a, int qs, int rs, int tile_cost, int part_cost, int least,
                                   long long (*red)[3], Ranges& ranges) {
  const int t = threadIdx.x;
  long long u = 0, n = 0, most = 0;
  const Units v{tile_cost, 0};
  for (int b = t; b < a.B; b += blockDim.x) {
    const Seq s = load_seq(a, b);
    u += seq_units(a, s, qs, rs, v, most);
    n += (static_cast<long long>(s.n) * a.G + a.tile_rows - 1) / a.tile_rows;
    if (s.bad) atomicCAS(a.status, 0u, (1u << 24) | (1u << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  }
  if ((t & 31) == 0) red[t >> 5][0] = u, red[t >> 5][1] = n, red[t >> 5][2] = most;
  __syncthreads();
  if (t == 0) {
    for (int w = 1; w < static_cast<int>(blockDim.x) / 32; ++w)
      u += red[w][0], n += red[w][1], most = max(most, red[w][2]);
    ranges.v = v;
    ranges.make(u * a.Hkv, n * a.Hkv, most, a.grid, part_cost, least);
  }
}

// A warp's way through its block's range.
struct Walk {
  Ranges r;
  int qs, rs, block;
  long long x, end;      // where it is, where the range ends
  long long head;        // unit at which the current KV head began (the tile's units follow)
  long long at;          // unit at which the current query tile begins
  int b, hk, c0;
  Seq s;
  Tiles t;

  __device__ inline void init(const ChunkArgs& a, const Ranges& rr, int block_, int qs_, int rs_, int lane) {
    r = rr, qs = qs_, rs = rs_, block = block_;
    b = a.B;
    x = end = 0;
    if (block >= r.blocks) return;
    x = r.start(block), end = r.start(block + 1);
    if (x >= end) return;
    // the sequence that holds x: 32 at a time
    long long before = 0;
    for (int base = 0; base < a.B; base += 32) {
      Seq ls;
      ls.n = ls.len = 0;
      if (base + lane < a.B) ls = load_seq(a, base + lane);
      long long most = 0;
      const long long mine = seq_units(a, ls, qs, rs, r.v, most);
      long long incl = mine * a.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, before + incl > x);
      if (past != 0) {
        const int k = __ffs(static_cast<int>(past)) - 1;
        b = base + k;
        s.n = __shfl_sync(0xFFFFFFFFu, ls.n, k);
        s.len = __shfl_sync(0xFFFFFFFFu, ls.len, k);
        const long long u = __shfl_sync(0xFFFFFFFFu, mine, k);
        head = before + __shfl_sync(0xFFFFFFFFu, incl, k) - u * a.Hkv;
        hk = static_cast<int>((x - head) / u);
        head += hk * u;
        c0 = __ldg(a.cu + b);
        t.start(a, s, qs, rs);
        at = head;
        return;
      }
      before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
  }
  // The next part with key tiles; false: the range is done.
  __device__ inline bool next(const ChunkArgs& a, int lane, Item& w) {
    while (x < end && b < a.B) {
      if (!t.more(a)) {  // the next KV head or sequence
        if (++hk == a.Hkv || s.n == 0) {
          hk = 0;
          if (++b >= a.B) return false;
          s = load_seq(a, b);
          c0 = __ldg(a.cu + b);
        }
        t.start(a, s, qs, rs);
        continue;
      }
      t.get(a, w.lo, w.hi, w.tb, w.nt, w.rows);
      const int kc = key_cost(w.rows), j = t.j;
      const long long stop = at + tile_units(w.nt, w.rows, r.v);
      t.next(a);
      w.x = at;
      at = stop;
      if (stop <= x) continue;  // before the range
      const long long to = min(stop, end);
      const int p0 = tiles_before(x - w.x, w.nt, kc, r.v), p1 = tiles_before(to - w.x, w.nt, kc, r.v);
      x = to;
      if (p0 == p1) continue;
      w.b = b, w.hk = hk, w.n = s.n, w.len = s.len, w.c0 = c0;
      w.r0 = j * a.tile_rows;
      w.t0 = w.tb + p0, w.t1 = w.tb + p1;
      w.whole = p0 == 0 && p1 == w.nt;
      w.parts = 1;
      w.slot = -1;
      if (!w.whole) {
        w.first = r.block_of(w.x), w.last = r.block_of(stop - 1);
        w.slot = part_slot(w, r, block);
        w.parts = 0;
        for (int c = w.first; c <= w.last; c += 32)
          w.parts += __popc(__ballot_sync(0xFFFFFFFFu, c + lane <= w.last && part_slot(w, r, c + lane) >= 0));
      }
      return true;
    }
    return false;
  }
};

}  // namespace chunk
}  // namespace fsops
