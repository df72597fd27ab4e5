// mx_chunk_plan.cuh -- how the chunk attention's work is cut and handed out.
// The lengths are device data, so every block derives the same plan from them.
//
// A sequence's new tokens times the G query heads of a KV head are its rows
// (row r: token r / G, head r % G); `rows` consecutive ones make a query
// tile, which sees the key tiles [lo, hi) of `kt` tokens that its mask
// reaches.  An item is (sequence, query tile, split, KV head), a split being S
// key tiles of the query tile.  S is one for the whole call: about half of a
// block's even share of the work, so that few rows over a long cache spread
// over the GPU and many rows are not split at all, doubled until the partial
// results fit the workspace.  Items are handed out by a counter, the query
// tiles of a sequence from its end, where a causal mask leaves most keys.
#pragma once
#include "mx_chunk.h"
#include "mx_device.cuh"

namespace fsops {
namespace chunk {

struct Seq {
  int n, len;   // new tokens, length with them (n = 0: nothing to do or not valid)
  int nq;       // query tiles
  int tiles;    // key tiles of a query tile at most
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const ChunkArgs& a, int b, int rows, int kt) {
  Seq s;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  s.len = __ldg(a.lens + b);
  s.n = c1 - c0;
  s.bad = c0 < 0 || c1 < c0 || c1 > a.T ||
          (s.n > 0 && (s.len < s.n || static_cast<long long>(s.len) > (static_cast<long long>(a.max_pages) << a.log2P)));
  if (s.bad || s.n <= 0) {
    s.n = s.nq = s.tiles = 0;
    return s;
  }
  s.nq = (s.n * a.G + rows - 1) / rows;
  s.tiles = (s.len + kt - 1) / kt;
  if (a.window > 0) {
    const int span = min(a.window, s.len) + min(s.n, rows / a.G + 2);  // tokens a query tile can reach
    s.tiles = min(s.tiles, (span + kt - 1) / kt + 1);
  }
  return s;
}

// One item.
struct Item {
  int b, j, split, hk;   // sequence, query tile, split, KV head
  int n, len, c0;        // new tokens, length, first row of the sequence
  int t0, t1;            // key tiles [t0, t1) of this split
  int ns;                // splits of the query tile that have keys
  int lo, hi;            // tokens some row of the tile sees
  uint32_t rec, group;   // first partial-result row and counter of the tile (ns > 1)
};

// Block-wide: the tiles of a split.  `red` holds one value a warp.
__device__ inline int split_tiles(const ChunkArgs& a, int rows, int kt, int smin, unsigned long long* red) {
  const int nt = blockDim.x, t = threadIdx.x;
  auto total = [&](unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((t & 31) == 0) red[t >> 5] = v;
    __syncthreads();
    unsigned long long s = 0;
    for (int w = 0; w < nt / 32; ++w) s += red[w];
    return s;
  };
  unsigned long long cost = 0;
  for (int b = t; b < a.B; b += nt) {
    const Seq s = load_seq(a, b, rows, kt);
    // a causal chunk's query tiles see half of the chunk's own keys on average
    const int avg = a.window > 0 ? s.tiles : max(1, s.tiles - s.n / (2 * kt));
    cost += static_cast<unsigned long long>(s.nq) * avg;
    if (s.bad) atomicCAS(a.status, 0u, (1u << 24) | (1u << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
  }
  cost = total(cost) * a.Hkv;
  long long S = static_cast<long long>((cost + 2ull * a.grid - 1) / (2ull * a.grid));
  if (S < smin) S = smin;
  for (;;) {
    // rows of partial results in the low 40 bits' place, counters above
    unsigned long long need = 0, groups = 0;
    for (int b = t; b < a.B; b += nt) {
      const Seq s = load_seq(a, b, rows, kt);
      const long long ns = (s.tiles + S - 1) / S;
      if (ns > 1) {
        need += static_cast<unsigned long long>(ns) * s.n * a.Hq;
        groups += static_cast<unsigned long long>(s.nq) * a.Hkv;
      }
    }
    need = total(need);
    groups = total(groups);
    if (need <= a.rec_rows && groups <= kChunkMaxGroups) break;
    S *= 2;
  }
  return static_cast<int>(S > (1 << 28) ? (1 << 28) : S);
}

// A warp's way through the items, which it meets in increasing order: the
// sequences [base, base + 32), one a lane, with the sums of what lies before.
struct Cursor {
  int S, rows, kt;
  int base;
  long long items0;           // items of the sequences before `base`
  uint32_t rec0, group0;
  Seq s;                      // the lane's sequence
  long long incl;             // items up to and with the lane's sequence, from base
  uint32_t rincl, gincl;

  __device__ __forceinline__ void load(const ChunkArgs& a, int lane) {
    const int b = base + lane;
    s.n = s.nq = s.tiles = s.len = 0;
    if (b < a.B) s = load_seq(a, b, rows, kt);
    const int ns = (s.tiles + S - 1) / S;
    incl = static_cast<long long>(s.nq) * ns * a.Hkv;
    rincl = ns > 1 ? static_cast<uint32_t>(ns) * s.n * a.Hq : 0u;
    gincl = ns > 1 ? static_cast<uint32_t>(s.nq) * a.Hkv : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      const uint32_t r = __shfl_up_sync(0xFFFFFFFFu, rincl, o), g = __shfl_up_sync(0xFFFFFFFFu, gincl, o);
      if (lane >= o) incl += v, rincl += r, gincl += g;
    }
  }
  __device__ __forceinline__ void init(const ChunkArgs& a, int S_, int rows_, int kt_, int lane) {
    S = S_, rows = rows_, kt = kt_;
    base = 0, items0 = 0, rec0 = 0, group0 = 0;
    load(a, lane);
  }
  // Item number `it` (not below an earlier one); false: none left.  Empty
  // splits give t0 == t1.
  __device__ __forceinline__ bool find(const ChunkArgs& a, long long it, int lane, Item& w) {
    for (;;) {
      const long long all = __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (it < items0 + all) break;
      if (base + 32 >= a.B) return false;
      items0 += all;
      rec0 += __shfl_sync(0xFFFFFFFFu, rincl, 31);
      group0 += __shfl_sync(0xFFFFFFFFu, gincl, 31);
      base += 32;
      load(a, lane);
    }
    const unsigned after = __ballot_sync(0xFFFFFFFFu, it < items0 + incl);
    const int k = __ffs(static_cast<int>(after)) - 1;
    const int before = max(k - 1, 0);
    const long long ib = __shfl_sync(0xFFFFFFFFu, incl, before);
    const uint32_t rb = __shfl_sync(0xFFFFFFFFu, rincl, before), gb = __shfl_sync(0xFFFFFFFFu, gincl, before);
    w.b = base + k;
    w.n = __shfl_sync(0xFFFFFFFFu, s.n, k);
    w.len = __shfl_sync(0xFFFFFFFFu, s.len, k);
    const int nq = __shfl_sync(0xFFFFFFFFu, s.nq, k), tiles = __shfl_sync(0xFFFFFFFFu, s.tiles, k);
    const int nsb = (tiles + S - 1) / S;
    int i = static_cast<int>(it - items0 - (k ? ib : 0));
    w.hk = i % a.Hkv;
    i /= a.Hkv;
    w.split = i % nsb;
    w.j = nq - 1 - i / nsb;
    w.c0 = __ldg(a.cu + w.b);
    // the tokens that the tile's rows see
    const int R = w.n * a.G, first = w.j * rows / a.G, last = (min(R, (w.j + 1) * rows) - 1) / a.G;
    const int p0 = w.len - w.n + first;
    w.hi = w.len - w.n + last + 1;
    w.lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    const int tb = w.lo / kt, te = (w.hi + kt - 1) / kt;
    w.ns = (te - tb + S - 1) / S;
    w.t0 = min(te, tb + w.split * S);
    w.t1 = min(te, w.t0 + S);
    // a sequence's partial results: [query tile][KV head][split][rows of the tile]
    const int tr = min(rows, R - w.j * rows);
    w.rec = rec0 + (k ? rb : 0u) +
            (static_cast<uint32_t>(w.j) * rows * a.Hkv + static_cast<uint32_t>(w.hk) * tr) * static_cast<uint32_t>(nsb);
    w.group = group0 + (k ? gb : 0u) + static_cast<uint32_t>(w.j) * a.Hkv + w.hk;
    return true;
  }
};

// A block leaves: the last one hands the counters back at zero.
__device__ __forceinline__ void leave(const ChunkArgs& a) {
  if (atomicAdd(a.done, 1u) == static_cast<uint32_t>(a.grid) - 1u) {
    *a.work = 0u;
    *a.done = 0u;
  }
}

}  // namespace chunk
}  // namespace fsops
