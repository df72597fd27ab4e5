// mx_pages.cu -- what is done with the paged cache's pages between two steps:
//
//   pages_update_kernel  page tables brought to new lengths: forks, releases,
//                        growth, a shared last page split off before it is
//                        written to.
//   copy_pages_kernel    pages copied, in all layers.
//   compact_kernel       the accepted tokens of a drafted tree moved together,
//                        in all layers.
#include <cooperative_groups.h>

#include <algorithm>

#include "mx_pages.h"

namespace fsops {

namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ void report(uint32_t* status, uint32_t site, int b) {
  atomicCAS(status, 0u, (1u << 24) | (site << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
}

// ---------------------------------------------------------------- page tables
// The steps need all tables, then all counts, then all free pages, with a meeting
// of the blocks between them, and are short: one cluster.  A page is counted by the
// entries of the new table that hold it (and by what else holds it); a page that
// nothing holds is free.  Free pages are handed out in increasing order to the
// sequences in order, so nothing depends on the order of atomics.  What bounds it is
// latency: five meetings and some ten loads one after another.  So a warp has 128
// entries of a table at a time, four loads of a lane together, and counts its pages
// by ballots, with one sum over the block.  64 sequences of 63-375 pages take
// 10.6 us, 512 of up to 250 16.0 (a warp a row, an entry a load: 16.2 and 24.6;
// clusters of 8 blocks 11.2 and 20.8).
// Small tables are one block's, with the counts in its shared memory.  Measured
// against 16 blocks (us): 28 entries in 33 pages 5.0 to 8.8, 2704 in 1700 6.2 to 9.4,
// in 16700 8.9 to 10.0, in 32000 11.8 to 10.3; 8064 in 5200 10.0 to 10.0, 11600 in
// 7500 10.1 to 9.9, 23300 in 16000 14.7 to 10.8.
constexpr int kMostBlocks = 16, kUpdateThreads = 1024, kUpdateWarps = kUpdateThreads / 32;
constexpr int kEntries = 128;  // of a table row at a time
constexpr int kMostHeld = 1 << 30;  // of what else holds a page: entries of the tables on top still fit an int
constexpr int kOnePages = 16384, kOneEntries = 8192;  // pages and entries of the tables up to which one block does it all

struct Row {
  int from;        // sequence whose pages it takes (-1: none)
  int keep, want;  // tokens
};
__device__ __forceinline__ Row row_of(const PagesArgs& a, int b, bool tell) {
  Row r;
  const int keep = __ldg(a.keep + b), want = __ldg(a.want + b);
  r.from = a.parent != nullptr ? __ldg(a.parent + b) : b;
  const int most = a.max_pages << a.log2P;
  int len = 0;
  bool bad = r.from >= a.B;
  if (bad || r.from < 0) r.from = -1;
  if (r.from >= 0) {
    len = a.lens[r.from];
    if (len < 0 || len > most) bad = true, len = 0;
  }
  r.keep = min(max(keep, 0), len);
  r.want = max(want, r.keep);
  if (r.want > most) bad = true, r.want = r.keep;
  if (bad && tell) report(a.status, 1u, b);
  return r;
}
__device__ __forceinline__ int pages_of(const PagesArgs& a, int tokens) { return (tokens + (1 << a.log2P) - 1) >> a.log2P; }

template <class T>
__device__ __forceinline__ T warp_sum_upto(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// Inclusive sum over the block; `all` gets the block's total.
template <class T>
__device__ __forceinline__ T block_sum(T v, T* red, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum_upto(v, lane);
  __syncthreads();  // the last sum's have been read
  if (lane == 31) red[warp] = v;
  __syncthreads();
  const T sums = warp_sum_upto(red[lane], lane);
  all = __shfl_sync(0xFFFFFFFFu, sums, 31);
  const T before = __shfl_sync(0xFFFFFFFFu, sums, (warp + 31) & 31);
  return warp > 0 ? v + before : v;
}

template <int kUpdateBlocks>
__global__ void __launch_bounds__(kUpdateThreads, 1) pages_update_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ int counts[];  // (one block) of each page
  cg::cluster_group cluster = cg::this_cluster();
  int* const refs = kUpdateBlocks == 1 ? counts : a.refs;
  auto held_by = [&](int p) { return kUpdateBlocks == 1 ? refs[p] : __ldcg(refs + p); };
  auto meet = [&]() {
    if constexpr (kUpdateBlocks == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  __shared__ long long red[kUpdateWarps];
  __shared__ int from_row[kUpdateThreads], have_pages[kUpdateThreads];  // of a thread's sequence
  __shared__ long long needed[kUpdateBlocks], freed[kUpdateBlocks];  // of each block: pages that its sequences need, free ones
  static_assert(kUpdateWarps == 32, "a warp has all warps' sums");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, rank = static_cast<int>(blockIdx.x);
  // the block's sequences and pages
  const int b0 = static_cast<int>(static_cast<long long>(a.B) * rank / kUpdateBlocks),
            b1 = static_cast<int>(static_cast<long long>(a.B) * (rank + 1) / kUpdateBlocks);
  const int p0 = static_cast<int>(static_cast<long long>(a.num_pages) * rank / kUpdateBlocks),
            p1 = static_cast<int>(static_cast<long long>(a.num_pages) * (rank + 1) / kUpdateBlocks);
#pragma unroll 4
  for (int p = p0 + t; p < p1; p += kUpdateThreads) refs[p] = a.held != nullptr ? min(max(__ldg(a.held + p), 0), kMostHeld) : 0;
  meet();
  // what stays of the tables, and how many entries hold a page
  const bool in_place = a.table == a.new_table;
  const int pieces = (a.max_pages + kEntries - 1) / kEntries;
  for (int base = b0; base < b1; base += kUpdateThreads) {
    const int rows = min(kUpdateThreads, b1 - base);
    __syncthreads();  // (the last ones are done)
    if (t < rows) {
      const Row r = row_of(a, base + t, true);
      from_row[t] = max(r.from, 0);
      have_pages[t] = pages_of(a, r.keep);
      a.rows[base + t] = make_int4(r.keep, r.want, -1, 0);
    }
    __syncthreads();
    const long long items = static_cast<long long>(rows) * pieces;
    for (long long u = warp; u < items; u += kUpdateWarps) {
      const int i = static_cast<int>(u / pieces), b = base + i, j0 = static_cast<int>(u - static_cast<long long>(i) * pieces) * kEntries + lane;
      const int have = have_pages[i];
      const int32_t* from = a.table + static_cast<long long>(from_row[i]) * a.max_pages;
      int32_t* to = a.new_table + static_cast<long long>(b) * a.max_pages;
      int page[kEntries / 32];
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) page[k] = j0 + 32 * k < have ? from[j0 + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) {
        const int j = j0 + 32 * k;
        bool bad = false;
        if (j < have) {
          bad = page[k] < 0 || page[k] >= a.num_pages;
          if (bad) {
            report(a.status, 2u, b);
            page[k] = -1;
          } else {
            atomicAdd(refs + page[k], 1);
          }
          if (j == have - 1) a.rows[b].z = page[k];
        }
        if (j < a.max_pages && (!in_place || bad || j >= have)) to[j] = page[k];
      }
    }
  }
  meet();
  // pages that each sequence needs, and pages that are free
  long long total = 0;
  for (int base = b0; base < b1; base += kUpdateThreads) {
    const int b = base + t;
    int need = 0, split = 0;
    int4 r = make_int4(0, 0, -1, 0);
    if (b < b1) {
      r = __ldcg(a.rows + b);
      if (r.y > r.x) {
        split = (r.x & ((1 << a.log2P) - 1)) != 0 && r.z >= 0 && held_by(r.z) > 1 ? 1 : 0;
        need = pages_of(a, r.y) - pages_of(a, r.x) + split;
      }
    }
    long long all;
    const long long upto = block_sum(static_cast<long long>(need), red, all);
    if (b < b1) {
      a.upto[b] = total + upto;
      r.w = 2 * need + split;
      a.rows[b] = r;
    }
    total += all;
  }
  // (a warp has consecutive pages, 32 at a time)
  const int per = ((p1 - p0 + kUpdateThreads - 1) / kUpdateThreads) * 32, w0 = min(p0 + warp * per, p1), w1 = min(w0 + per, p1);
  int mine = 0;
#pragma unroll 4
  for (int p = w0 + lane; p < w1; p += 32) mine += held_by(p) == 0 ? 1 : 0;
  long long free_here;
  const long long free_upto = block_sum(static_cast<long long>(mine), red, free_here);
  if constexpr (kUpdateBlocks == 1) {
    if (t == 0) needed[0] = total, freed[0] = free_here;
  } else if (t < kUpdateBlocks) {
    *cluster.map_shared_rank(needed + rank, t) = total;
    *cluster.map_shared_rank(freed + rank, t) = free_here;
  }
  meet();
  long long needed_before = 0, freed_before = 0, needed_all = 0, freed_all = 0;
#pragma unroll
  for (int r = 0; r < kUpdateBlocks; ++r) {
    if (r < rank) needed_before += needed[r], freed_before += freed[r];
    needed_all += needed[r], freed_all += freed[r];
  }
  // the free pages in order, as many as are needed
  long long at = freed_before + __shfl_sync(0xFFFFFFFFu, free_upto - mine, 0);  // of the warp's first one
  for (int base = w0; base < w1 && at < needed_all; base += 32) {
    const int p = base + lane;
    const bool is_free = p < w1 && held_by(p) == 0;
    const unsigned some = __ballot_sync(0xFFFFFFFFu, is_free);
    const long long place = at + __popc(some & ((1u << lane) - 1u));
    if (is_free && place < needed_all) a.fresh[place] = p;
    at += __popc(some);
  }
  meet();  // (the last one: nothing of another block's shared memory is read after it)
  // handed out: few pages by the sequence's thread, more by its warp
  for (int base = b0 + 32 * warp; base < b1; base += kUpdateThreads) {
    const int b = base + lane;
    int4 r = make_int4(0, 0, -1, 0);
    long long upto = 0;
    if (b < b1) r = __ldcg(a.rows + b), upto = needed_before + __ldcg(a.upto + b);
    const int need = r.w >> 1, split = r.w & 1;
    const bool fits = need == 0 || upto <= freed_all;
    auto hand = [&](int b, const int4& r, long long first, int need, int j0, int step) {
      const int split = r.w & 1, have = pages_of(a, r.x);
      int32_t* to = a.new_table + static_cast<long long>(b) * a.max_pages;
      for (int j = j0; j < need; j += step) {
        const int page = __ldcg(a.fresh + first + j);
        refs[page] = 1;
        to[have + j - split] = page;
        if (j == 0 && split) {
          atomicSub(refs + r.z, 1);
          a.copy_src[b] = r.z;
          a.copy_dst[b] = page;
        }
      }
    };
    const bool many = need > 4 && fits;
    if (b < b1) {
      if (need > 0 && !fits) report(a.status, 3u, b);
      if (!many && fits) hand(b, r, upto - need, need, 0, 1);
      a.new_lens[b] = fits ? r.y : r.x;
      if (!(split && fits)) a.copy_src[b] = a.copy_dst[b] = -1;
    }
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, many); left != 0u; left &= left - 1u) {
      const int l = __ffs(static_cast<int>(left)) - 1;
      const int4 q = make_int4(__shfl_sync(0xFFFFFFFFu, r.x, l), __shfl_sync(0xFFFFFFFFu, r.y, l), __shfl_sync(0xFFFFFFFFu, r.z, l),
                               __shfl_sync(0xFFFFFFFFu, r.w, l));
      hand(base + l, q, __shfl_sync(0xFFFFFFFFu, upto - need, l), q.w >> 1, lane, 32);
    }
  }
  if constexpr (kUpdateBlocks == 1) {
    __syncthreads();
#pragma unroll 4
    for (int p = t; p < a.num_pages; p += kUpdateThreads) a.refs[p] = refs[p];
  }
}

// ---------------------------------------------------------------- copies
// 16 bytes a lane, eight loads on their way together; a warp copies a piece of
// 4 KB.  Pages and their scales are whole numbers of 64 bytes.  Bound by HBM: 769 MB
// read and written in 121 us, 6.3 TB/s, 0.93 of the copy rate; 34 MB (mostly in L2)
// in 6 us.
constexpr int kCopyThreads = 256, kPieceBytes = 4096;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a, int code_pieces,
                                                                  int scale_pieces, long long units) {
  const PagedCache& c = a.cache;
  const int lane = threadIdx.x & 31, pieces = 2 * (code_pieces + scale_pieces);
  const int code_bytes = c.Hkv * 128 << c.log2P, scale_bytes = code_bytes / 32;
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  for (long long u = static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const long long pl = u / pieces;
    int piece = static_cast<int>(u - pl * pieces);
    const int layer = static_cast<int>(pl / a.n), i = static_cast<int>(pl - static_cast<long long>(layer) * a.n);
    const int src = __ldg(a.src + i), dst = __ldg(a.dst + i);
    if (src < 0 || dst < 0 || src >= c.num_pages || dst >= c.num_pages || src == dst) {
      if (src >= 0 && dst >= 0 && src != dst && layer == 0 && piece == 0 && lane == 0) report(a.status, 2u, i);
      continue;
    }
    const int v = piece & 1;
    piece >>= 1;
    const bool is_scale = piece >= code_pieces;
    if (is_scale) piece -= code_pieces;
    uint8_t* base = is_scale ? c.scales[v] : c.codes[v];
    const int bytes = is_scale ? scale_bytes : code_bytes;
    const long long first = static_cast<long long>(layer) * c.num_pages;
    const uint8_t* from = base + (first + src) * bytes;
    uint8_t* to = base + (first + dst) * bytes;
    const int at = piece * kPieceBytes + 16 * lane;
    uint4 x[kPieceBytes / 512];
#pragma unroll
    for (int k = 0; k < kPieceBytes / 512; ++k)
      if (at + 512 * k < bytes) x[k] = *reinterpret_cast<const uint4*>(from + at + 512 * k);
#pragma unroll
    for (int k = 0; k < kPieceBytes / 512; ++k)
      if (at + 512 * k < bytes) *reinterpret_cast<uint4*>(to + at + 512 * k) = x[k];
  }
}

// ---------------------------------------------------------------- accepted tokens
// A warp has one head of one layer of a sequence, K and V, and moves its tokens 16
// at a time: all of them are read before any is written.  As a path goes up
// (path[j] >= j), what a later group of 16 reads lies behind everything that an
// earlier one writes.  Bound by latency (the path, the pages, the tokens), so many
// warps with few registers: 64 sequences' paths of up to 16 tokens, 28 layers of 4
// heads, 45 MB, take 12.7 us, 15 with 32 tokens of K or of V a warp.
constexpr int kCompactThreads = 128, kMove = 16;

__global__ void __launch_bounds__(kCompactThreads, 8) compact_kernel(const __grid_constant__ CompactArgs a, long long units) {
  const PagedCache& c = a.cache;
  const int lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (kCompactThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  const int per = c.Hkv * c.layers, b = static_cast<int>(u / per), rest = static_cast<int>(u - static_cast<long long>(b) * per);
  const int layer = rest / c.Hkv, h = rest - layer * c.Hkv;
  const bool tell = rest == 0;
  const int n = __ldg(a.count + b), start = __ldg(a.start + b);
  const int32_t* path = a.path + static_cast<long long>(b) * a.max_path;
  const int32_t* table = a.table + static_cast<long long>(b) * a.max_pages;
  const long long tokens = static_cast<long long>(a.max_pages) << c.log2P;
  // the path goes up and stays within the table (its first 32 places are read with the count)
  const int p0 = lane < a.max_path ? __ldg(path + lane) : 0, left = __shfl_up_sync(0xFFFFFFFFu, p0, 1);
  auto good = [&](int p, int before) { return p > before && p >= 0 && static_cast<long long>(start) + p < tokens; };
  bool ok = n >= 0 && n <= a.max_path && (start >= 0 || n == 0);  // (no early end: all three loads are on their way together)
  if (ok && lane < n) ok = good(p0, lane > 0 ? left : -1);
  for (int j = lane + 32; ok && j < n; j += 32) ok = good(__ldg(path + j), __ldg(path + j - 1));
  if (!__all_sync(0xFFFFFFFFu, ok)) {
    if (tell && lane == 0) report(a.status, 1u, b);
    return;
  }
  const long long first = static_cast<long long>(layer) * c.num_pages;
  const int mask = (1 << c.log2P) - 1;
  for (int base = 0; base < n; base += kMove) {
    // where token base + lane % 16 comes from and goes to (-1: it stays)
    long long from = -1, to = -1;
    const int j = base + (lane & (kMove - 1)), early = __shfl_sync(0xFFFFFFFFu, p0, j & 31);
    if (j < n) {
      const int s = start + (base < 32 ? early : __ldg(path + j)), d = start + j;
      if (s != d) {
        const int sp = __ldg(table + (s >> c.log2P)), dp = __ldg(table + (d >> c.log2P));
        if (sp < 0 || sp >= c.num_pages || dp < 0 || dp >= c.num_pages) {
          if (tell) report(a.status, 2u, b);
        } else {
          from = (((first + sp) * c.Hkv + h) << c.log2P) + (s & mask);
          to = (((first + dp) * c.Hkv + h) << c.log2P) + (d & mask);
        }
      }
    }
    if (!__any_sync(0xFFFFFFFFu, to >= 0)) continue;
    uint4 x[2][kMove / 4];
    uint32_t sc = 0;
    // (scales: K's by the first half of the warp, V's by the second)
    if (to >= 0) sc = *reinterpret_cast<const uint32_t*>(c.scales[lane / kMove] + from * 4);
#pragma unroll
    for (int k = 0; k < kMove / 4; ++k) {  // four tokens, eight lanes each
      const long long row = __shfl_sync(0xFFFFFFFFu, from, 4 * k + (lane >> 3));
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (row >= 0) x[v][k] = *reinterpret_cast<const uint4*>(c.codes[v] + row * 128 + 16 * (lane & 7));
    }
    __syncwarp();
    if (to >= 0) *reinterpret_cast<uint32_t*>(c.scales[lane / kMove] + to * 4) = sc;
#pragma unroll
    for (int k = 0; k < kMove / 4; ++k) {
      const long long row = __shfl_sync(0xFFFFFFFFu, to, 4 * k + (lane >> 3));
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (row >= 0) *reinterpret_cast<uint4*>(c.codes[v] + row * 128 + 16 * (lane & 7)) = x[v][k];
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t stream) {
  cudaError_t e;
  if (a.num_pages <= kOnePages && static_cast<long long>(a.B) * a.max_pages <= kOneEntries) {
    const int bytes = a.num_pages * static_cast<int>(sizeof(int));
    // (the same limit in every call: another host thread's may come between this one and the launch)
    e = cudaFuncSetAttribute(pages_update_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOnePages * sizeof(int));
    if (e != cudaSuccess) return e;
    pages_update_kernel<1><<<1, kUpdateThreads, bytes, stream>>>(a);
    return cudaGetLastError();
  }
  e = cudaFuncSetAttribute(pages_update_kernel<kMostBlocks>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMostBlocks);
  cfg.blockDim = dim3(kUpdateThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kMostBlocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, pages_update_kernel<kMostBlocks>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyPagesArgs& a, int sms, cudaStream_t stream) {
  const long long code_bytes = static_cast<long long>(a.cache.Hkv) * 128 << a.cache.log2P;
  const int code_pieces = static_cast<int>((code_bytes + kPieceBytes - 1) / kPieceBytes),
            scale_pieces = static_cast<int>((code_bytes / 32 + kPieceBytes - 1) / kPieceBytes);
  const long long units = static_cast<long long>(a.n) * a.cache.layers * 2 * (code_pieces + scale_pieces);
  const long long blocks = std::min<long long>((units + kCopyThreads / 32 - 1) / (kCopyThreads / 32), 6LL * sms);
  copy_pages_kernel<<<static_cast<unsigned>(blocks), kCopyThreads, 0, stream>>>(a, code_pieces, scale_pieces, units);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.B) * a.cache.layers * a.cache.Hkv;
  const long long blocks = (units + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  compact_kernel<<<static_cast<unsigned>(blocks), kCompactThreads, 0, stream>>>(a, units);
  return cudaGetLastError();
}

}  // namespace fsops
