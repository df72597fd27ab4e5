// mx_chunk_few.cu -- the chunk attention of mx_chunk.cu for few rows: query
// tiles of up to 32 rows (single tokens, drafted tokens), whose time is the
// cache's bytes.
//
// With queries as the 128 rows of a product, a few of them would leave most of
// it empty, and all exponentials to one warp.  So here the products are turned
// round: keys are the rows of the scores, S^T = K Q^T, and dimensions the rows
// of the outputs, O^T = V^T P^T, and the query rows their columns.
//   S^T  [112 keys][2 x rows]  block-scaled E4M3 MMA on K's own codes; the two
//        E4M3 terms of the queries are two groups of columns, added afterwards;
//   P^T  [112 keys][32 rows] bf16 in shared memory, N-major;
//   O^T  [128 dimensions][32 rows] with V widened to bf16 as the M-major operand.
// A key tile costs 4 + 7 MMAs this way (about 500 cycles of the tensor pipe),
// less than its 30 KB take to arrive (1250 cycles at the card's copy rate), and
// a thread has one key and 16 rows of a tile: four warps for each 16 rows.
//
// A row's scale (its running maximum) is the same for all keys, so the four
// warps of a row vote, once for two tiles: while no score passes the scale by
// more than 2^8, and nearly always none does, nothing but the vote is exchanged.
// Else they find the maximum together, rescale, and compute the probabilities
// again.  A row's sum stays apart in its 112 threads until the item's end.
//
// Products of two key tiles run under the exponentials of the next two (scores
// and probabilities are double buffered); loads run ahead over the items' ends,
// and the next item's first scores are computed under this one's end.
//
// The code that runs once an item (queries, first maximum, end) is rolled up on
// purpose: it is fetched anew each time, and straight-line code there cost
// 10000 cycles an item, mostly of instruction fetches.
//
// Measured: 64 sequences of 2k-6k tokens with 5 drafted tokens each (32 query, 8
// KV heads, pages of 16), 558 MB, in 136 us: 4.1 TB/s, 0.61 of the copy rate.
// Loads without widening and exponentials take 110 us, with one of them 125 and
// 128.  Four tiles of K, three of V and three widened ones in flight: 140 us
// against 142 for 5, 4, 2, 143 for 5, 3, 2 and 157 for 4, 2, 3.
#include "mx_chunk_parts.cuh"

namespace fsops {

namespace {

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kConvWarps, kLoadWarp = kMmaWarp + 2;  // two warps each
constexpr int kBlock = 32 * (kLoadWarp + 2);
constexpr int NK = 4, NV = 3, kSlots = 3;       // tiles of K and of V's codes in flight, of V as bf16
constexpr int kRows = kChunkFewRows;
// The plan's costs, in fifths of a key tile.  Measured, a query tile a block
// against equal shares: 12 to 15 us for 8 query tiles of 5 key tiles, 16 to 23
// for 64 of 9, 24 to 17 for 8 of 19, 31 to 26 for 64 of 27.
constexpr int kTileCost = 10;
constexpr int kPartCost = 25;    // units that a part costs to write and merge
constexpr int kLeastUnits = 10;  // of a block
constexpr uint32_t kProbs = kKeys * kRows * 2;  // a tile's probabilities
static_assert(kRows == 32, "64 bytes of probabilities a key, one swizzle atom wide");
constexpr uint32_t kSwizzle64B = 4;
// Columns of tensor memory: the scores of two times two tiles, the outputs, scale
// factors of the queries and of K (four tiles).
constexpr uint32_t kColS = 64, kColO = 256, kColSfq = 288, kColSfk = 292;
constexpr float kNone = -3e38f;  // the scale of a row that has seen nothing

struct Ctl {
  uint64_t k_full[NK], k_empty[NK], r_full[NV], r_empty[NV];  // rings of K and V codes
  uint64_t v_full[kSlots], v_empty[kSlots];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];  // two tiles each, by turns
  uint64_t q_full, vote[2], fin[2], it_full[2], it_empty[2];
  Item item[2];
  HiddenNan hidden[2];
  alignas(16) float scale[2][kRows];     // the rows' scales (base 2), the one in use by turns
  alignas(16) float fall[kRows];         // what the last change of scale makes of a row
  float peak[2][4][16];      // a group's maxima, of each warp
  float sums[4][kRows];
  uint32_t grown[2];         // the last vote that found a larger score
  long long red[kBlock / 32][3];
  chunk::Ranges ranges;
  uint32_t tmem, stop;
};
struct L {
  static constexpr uint32_t q = 0, v = 2 * kRows * kD, p = v + kSlots * kOperand, k = p + 4 * kProbs, raw = k + NK * kCodes,
                            sfk = raw + NV * kCodes, sv = sfk + NK * kScales, sfq = sv + NV * kScales,
                            ctl = sfq + kScales, bytes = ctl + sizeof(Ctl);
};
static_assert(L::bytes <= 232448 && NK <= 5 && NV <= 4, "shared memory");
static_assert(L::ctl % 16 == 0 && alignof(Ctl) == 16 && L::p % 1024 == 0 && L::v % 1024 == 0 && L::k % 1024 == 0, "alignment");
static_assert(NV * kCodes >= 16 * kD, "the 128-row product reads 16 rows behind the last K tile");

// kind::f16, fp32 sums, bf16 operands, M = 128 (M-major, bit 15), N = 32 (N-major, bit 16).
constexpr uint32_t kIdescPv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                              ((static_cast<uint32_t>(kRows) >> 3) << 17) | ((128u >> 4) << 24);
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Sixteen values of every lane combined over the lanes: lane i ends with value i / 2's.
template <bool sum>
__device__ __forceinline__ float across(float (&v)[16], int lane) {
  auto both = [](float x, float y) { return sum ? x + y : fmaxf(x, y); };
#pragma unroll
  for (int n = 8; n; n >>= 1) {
    const bool up = (lane & (2 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = both(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2 * n));
    }
  }
  return both(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// A warp's share (16 rows from row0 on, the 32 stored dimensions from dim0 on) of
// a query tile added up over the tile's parts, in the blocks' order.  A lane has
// four dimensions of every fourth row.
__device__ __forceinline__ void merge_share(const ChunkArgs& a, const Item& w, const chunk::Ranges& rg, int row0, int dim0,
                                            int lane) {
  const int blocks = w.last - w.first + 1, dim = dim0 + 4 * (lane & 7);
  // the first row of each part's results, 32 parts at a time, a lane each (parts
  // without a key tile read the first slot, with no weight; no branches, so that
  // several parts' loads are on their way together)
  auto rows_of = [&](int base) {
    const int sl = base + lane < blocks ? chunk::part_slot(w, rg, w.first + base + lane) : -1;
    return sl < 0 ? -1 : sl * a.slot_rows;
  };
  float M = -INFINITY;  // of row lane % 16
#pragma unroll 1
  for (int base = 0; base < blocks; base += 32) {
    const int mine = rows_of(base), n = min(32, blocks - base);
#pragma unroll 1
    for (int p = 0; p < n; p += 8) {  // (lanes past the last part have none)
      int at[8];
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) at[i] = __shfl_sync(0xFFFFFFFFu, mine, p + i);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = __ldcg(&a.rec_ml[max(at[i], 0) + min(row0 + (lane & 15), w.rows - 1)].x);
#pragma unroll
      for (int i = 0; i < 8; ++i) M = fmaxf(M, at[i] < 0 ? -INFINITY : m[i]);
    }
  }
  float den[4];
  float4 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) den[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int base = 0; base < blocks; base += 32) {
    const int mine = rows_of(base), n = min(32, blocks - base);
#pragma unroll 1
    for (int p = 0; p < n; p += 2) {
      int at[2];
      float2 ml[2][4];
      float4 x[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) at[q] = __shfl_sync(0xFFFFFFFFu, mine, p + q);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = max(at[q], 0) + min(row0 + 4 * i + (lane >> 3), w.rows - 1);
          ml[q][i] = __ldcg(&a.rec_ml[row]);
          x[q][i] = __ldcg(reinterpret_cast<const float4*>(a.rec + static_cast<size_t>(row) * kD + dim));
        }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = __shfl_sync(0xFFFFFFFFu, M, 4 * i + (lane >> 3));
          const bool none = at[q] < 0 || ml[q][i].x == -INFINITY;
          const float f = none ? 0.f : exp2_fast(ml[q][i].x - m);
          const float4 v = none ? make_float4(0.f, 0.f, 0.f, 0.f) : x[q][i];
          den[i] = fmaf(f, at[q] < 0 ? 0.f : ml[q][i].y, den[i]);
          o[i].x = fmaf(f, v.x, o[i].x), o[i].y = fmaf(f, v.y, o[i].y);
          o[i].z = fmaf(f, v.z, o[i].z), o[i].w = fmaf(f, v.w, o[i].w);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 4 * i + (lane >> 3), rr = w.r0 + row, tok = rr / a.G;
    const float inv = divisor(__shfl_sync(0xFFFFFFFFu, M, 4 * i + (lane >> 3)), den[i]);
    if (row < w.rows)  // (stored order 0, 2, 1, 3)
      *reinterpret_cast<uint2*>(a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + rr - tok * a.G) * kD + dim) =
          make_uint2(bf16x2_rn(o[i].x * inv, o[i].z * inv), bf16x2_rn(o[i].y * inv, o[i].w * inv));
  }
}

__global__ void __launch_bounds__(kBlock, 1) chunk_few_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + L::ctl);
  const Ctx c{a, &ctl->stop, a.tries};
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int qs = a.tile_rows / a.G, rs = a.tile_rows % a.G;
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      mbar_init(&ctl->k_full[i], 32);
      mbar_init(&ctl->k_empty[i], 1);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      mbar_init(&ctl->r_full[i], 32);
      mbar_init(&ctl->r_empty[i], kConvWarps);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl->v_full[i], kConvWarps);
      mbar_init(&ctl->v_empty[i], 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_free[i], kSoftWarps);
      mbar_init(&ctl->p_full[i], kSoftWarps);
      mbar_init(&ctl->p_free[i], 1 + a.extra_arrivals);
      mbar_init(&ctl->vote[i], 4);
      mbar_init(&ctl->fin[i], 1);
      mbar_init(&ctl->it_full[i], 32);
      mbar_init(&ctl->it_empty[i], kSoftWarps + kConvWarps + 3);
      ctl->grown[i] = 0u;
    }
    mbar_init(&ctl->q_full, kSoftWarps);
    ctl->stop = 0u;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  chunk::make_ranges(a, qs, rs, kTileCost, kPartCost, kLeastUnits, ctl->red, ctl->ranges);  // a block-wide barrier inside
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // the shared memory starts on a swizzle atom (checked, as all offsets rely on it)
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (t == 0) {
      atomicCAS(a.status, 0u, (3u << 24) | (9u << 16));
      ctl->stop = 9u;
    }
    __syncthreads();
  } else if (warp >= kLoadWarp) {
    load_items<NK, NV>(c, ctl, smem + L::k, smem + L::raw, smem + L::sfk, smem + L::sv, qs, rs, warp > kLoadWarp, lane);
  } else if (warp >= kMmaWarp) {
    // ---- products, one warp the scores, one the outputs; one lane issues
    const bool pv = warp > kMmaWarp;
    const uint64_t dk = smem_desc(smem_u32(smem + L::k), 16, 1024, kSwizzle128B);
    const uint64_t dq = smem_desc(smem_u32(smem + L::q), 16, 1024, kSwizzle128B);
    const uint64_t dsk = smem_desc(smem_u32(smem + L::sfk), 0, 128, kSwizzleNone);
    const uint64_t dsq = smem_desc(smem_u32(smem + L::sfq), 0, 128, kSwizzleNone);
    const uint64_t dv = smem_desc(smem_u32(smem + L::v), kHalf, 1024, kSwizzle128B);
    const uint64_t dp = smem_desc(smem_u32(smem + L::p), kProbs, 512, kSwizzle64B);
    Ring<2> it, buf;
    Ring<NK> kr;
    Ring<kSlots> vr;
    uint32_t q_phase = 0;
    for (bool ok = true; ok; it.step()) {
      if (!wait(c, &ctl->it_full[it.slot], it.phase, 4u)) break;
      const int tiles = __shfl_sync(0xFFFFFFFFu, ctl->item[it.slot].t1 - ctl->item[it.slot].t0, 0);
      const uint32_t groups = __shfl_sync(0xFFFFFFFFu, (ctl->item[it.slot].rows + 15) >> 4, 0);
      warp_arrive(&ctl->it_empty[it.slot], lane);
      if (tiles == 0) break;
      if (!pv) {
        if (!wait(c, &ctl->q_full, q_phase, 5u)) break;
        q_phase ^= 1u;
        tc_fence_after();
        if (elect_one()) tc_cp_32x128b_warpx4(tmem + kColSfq, dsq);
        __syncwarp();
        const uint32_t idesc = idesc_mxf8_e4m3(32 * groups, 0, 0);
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          const uint32_t u = j & 1;
          ok = (u || wait(c, &ctl->s_free[buf.slot], buf.phase ^ 1u, 7u)) && wait(c, &ctl->k_full[kr.slot], kr.phase, 6u);
          if (!ok) break;
          const bool last = u || j + 1 == tiles;  // of the two
          fence_proxy_async_shared();             // the codes came by generic copies
          tc_fence_after();
          if (elect_one()) {
            const uint32_t at = 2 * buf.slot + u, sfk = tmem + kColSfk + 4 * at;
            tc_cp_32x128b_warpx4(sfk, dsk + kr.slot * (kScales >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 dimensions
              tc_mma_mxf8(tmem + kColS * at, dk + kr.slot * (kCodes >> 4) + ((32 * k) >> 4), dq + ((32 * k) >> 4),
                          idesc | (k << 4) | (k << 29), sfk, tmem + kColSfq, k > 0);
            tc_commit(&ctl->k_empty[kr.slot]);
            if (last) tc_commit(&ctl->s_full[buf.slot]);
          }
          __syncwarp();
          kr.step();
          if (last) buf.step();
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          const uint32_t u = j & 1;
          ok = (u || wait(c, &ctl->p_full[buf.slot], buf.phase, 8u)) && wait(c, &ctl->v_full[vr.slot], vr.phase, 8u);
          if (!ok) break;
          const bool last = u || j + 1 == tiles;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)  // 16 tokens
              mma_ss(tmem + kColO, dv + vr.slot * (kOperand >> 4) + k * (2048 >> 4),
                     dp + (2 * buf.slot + u) * (kProbs >> 4) + k * (1024 >> 4), kIdescPv, (j > 0 || k > 0) ? 1u : 0u);
            tc_commit(&ctl->v_empty[vr.slot]);
            if (last) tc_commit(&ctl->p_free[buf.slot]);
          }
          __syncwarp();
          vr.step();
          if (last) buf.step();
        }
      }
    }
  } else if (warp >= kSoftWarps) {
    convert_items<NV, kSlots>(c, ctl, smem + L::raw, smem + L::sv, smem + L::v, t - 32 * kSoftWarps, lane);
  } else {
    // ---- softmax: rows 16 h .. 16 h + 15, a thread a key
    const int h = warp >> 2, wl = warp & 3, key = 32 * wl + lane;
    const bool live = key < kKeys;
    const uint32_t lanes = static_cast<uint32_t>(32 * wl) << 16;
    const float scale = a.scale_log2;
    // the key's probabilities in a tile's buffer: 16-byte pieces 2 h and 2 h + 1
    const uint32_t prow = L::p + key * 64 + ((2 * h ^ ((key >> 1) & 3)) << 4);
    uint32_t n = 0, votes = 0;  // pairs of key tiles, votes so far
    auto queries = [&](int slot) {
      const Item& w = ctl->item[slot];
      if (w.t0 == w.t1) return;
      const int rows = (w.rows + 15) & ~15, R = w.n * a.G;
      const uint32_t flip = a.negate ? 0x80008000u : 0u;
      uint4 x = make_uint4(0u, 0u, 0u, 0u), x1 = x;
#pragma unroll 1
      for (int i = rows / 16 - 1; i >= 0; --i) {
        x1 = x;
        const int rr = min(w.r0 + 16 * i + 2 * warp + (lane >> 4), R - 1), tok = rr / a.G;
        x = __ldg(reinterpret_cast<const uint4*>(a.q + static_cast<long long>(w.c0 + tok) * a.ldq +
                                                 (w.hk * a.G + rr - tok * a.G) * kD) + (lane & 15));
      }
#pragma unroll 1
      for (int i = 0; 16 * i < rows; ++i, x = x1)
        store_query(x, flip, smem + L::q, smem + L::sfq, 16 * i + 2 * warp + (lane >> 4), rows, lane & 15);
      fence_proxy_async_shared();
      warp_arrive(&ctl->q_full, lane);
    };
    auto meet = [&]() -> bool {  // the warps of a row
      warp_arrive(&ctl->vote[h], lane);
      return wait(c, &ctl->vote[h], votes++ & 1u, 11u);
    };
    Ring<2> it;
    int turn = 0;  // which of the scales is in use
    bool ok = wait(c, &ctl->it_full[0], 0, 4u);
    if (ok) queries(0);
#pragma unroll 1
    while (ok) {
      float2 l[8];  // the thread's sums
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] = make_float2(0.f, 0.f);
      const int groups = (ctl->item[it.slot].rows + 15) >> 4;
      {
        const Item& w = ctl->item[it.slot];  // given back at the item's end
        if (w.t0 == w.t1) break;
        const int t1 = w.t1, hi = w.len - w.n + 1 + w.r0 / a.G,  // all rows see the tokens lo .. hi - 1
                  lo = a.window > 0 ? w.len - w.n + 1 + (w.r0 + w.rows - 1) / a.G - a.window : 0;
        turn ^= 1;
        if (lane < 16) ctl->scale[turn][16 * h + lane] = kNone;  // (every warp of the row writes the same)
        __syncwarp();
#pragma unroll 1
        for (int k0 = w.t0; k0 < t1; k0 += 2, ++n) {
          const uint32_t buf = n & 1u, phase = (n >> 1) & 1u;
          const int k1 = min(k0 + 2, t1);
          ok = wait(c, &ctl->s_full[buf], phase, 10u) && wait(c, &ctl->p_free[buf], phase ^ 1u, 12u);
          if (!ok) break;
          tc_fence_after();
          if (h < groups) {
            // the scores of tile k (not yet scaled)
            auto scores = [&](int k, float2(&s)[8]) {
              const uint32_t S = tmem + lanes + kColS * (2 * buf + (k - k0)) + 16 * h;
              float x[16], y[16];
              tmem_ld16f(S, x);
              tmem_ld16f(S + 16 * groups, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                s[i] = __fadd2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(y[2 * i], y[2 * i + 1]));
              if (k * kKeys < lo || (k + 1) * kKeys > hi) {
                const int r = w.r0 + 16 * h, tok = k * kKeys + key;
                int upto = w.len - w.n + 1 + r / a.G, in = r % a.G;
                uint32_t hide = 0;
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                  const int u = min(upto, w.len);
                  if (tok >= u || (a.window > 0 && tok < u - a.window)) hide |= 1u << i;
                  if (++in == a.G) in = 0, ++upto;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  if (hide & (1u << (2 * i))) s[i].x = -INFINITY;
                  if (hide & (2u << (2 * i))) s[i].y = -INFINITY;
                }
              }
            };
            float2 add[8];
#pragma unroll 1
            for (bool again = false;; again = true) {
              if (again || k0 > w.t0) {  // (there is no scale before the first tiles)
                const float4* ms = reinterpret_cast<const float4*>(ctl->scale[turn] + 16 * h);
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) add[i] = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                  float2 s[8];
                  uint32_t p[8];
                  scores(k, s);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float4 m = ms[i];
                    s[2 * i] = __ffma2_rn(s[2 * i], make_float2(scale, scale), make_float2(-m.x, -m.y));
                    s[2 * i + 1] = __ffma2_rn(s[2 * i + 1], make_float2(scale, scale), make_float2(-m.z, -m.w));
                  }
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    top = max3(top, s[i].x, s[i].y);
                    s[i].x = exp2_fast(s[i].x), s[i].y = exp2_fast(s[i].y);
                    add[i] = __fadd2_rn(add[i], s[i]);
                    p[i] = bf16x2_rn(s[i].x, s[i].y);
                  }
                  if (live) {
                    uint8_t* d = smem + (prow + (2 * buf + (k - k0)) * kProbs);
                    *reinterpret_cast<uint4*>(d) = make_uint4(p[0], p[1], p[2], p[3]);
                    *reinterpret_cast<uint4*>(smem + ((prow ^ 16u) + (2 * buf + (k - k0)) * kProbs)) =
                        make_uint4(p[4], p[5], p[6], p[7]);
                  }
                }
                if (again) break;
                volatile uint32_t* grown = &ctl->grown[h];
                if (__any_sync(0xFFFFFFFFu, live && top > kGrow) && lane == 0) *grown = votes + 1u;
                ok = meet();
                if (!ok || *grown != votes) break;
              }
              // the rows' maxima, and what has been added up so far in the new unit
              float x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = -INFINITY;
#pragma unroll 1
              for (int k = k0; k < k1; ++k) {
                float2 s[8];
                scores(k, s);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = fmaxf(x[i], live ? (i & 1 ? s[i >> 1].y : s[i >> 1].x) : -INFINITY);
              }
              const float mx = across<false>(x, lane) * scale;
              if ((lane & 1) == 0) ctl->peak[h][wl][lane >> 1] = mx;
              ok = meet();
              if (!ok) break;
              if (lane < 16) {  // (every warp of the row writes the same)
                const float(*pk)[16] = ctl->peak[h];
                const float m = fmaxf(max3(pk[0][lane], pk[1][lane], pk[2][lane]), pk[3][lane]),
                            mo = ctl->scale[turn][16 * h + lane], mn = m > mo + kGrow ? m : mo;
                ctl->scale[turn ^ 1][16 * h + lane] = mn;
                ctl->fall[16 * h + lane] = exp2_fast(mo - mn);
              }
              turn ^= 1;
              __syncwarp();
              if (k0 > w.t0) {
                ok = wait(c, &ctl->p_free[buf ^ 1u], ((n - 1u) >> 1) & 1u, 11u);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float4 f = *reinterpret_cast<const float4*>(ctl->fall + 16 * h + 4 * i);
                  const uint32_t O = tmem + lanes + kColO + 16 * h + 4 * i;
                  float o[4];
                  tmem_ld4(O, o);
                  tmem_ld_wait();
                  tmem_st4(O, __float_as_uint(o[0] * f.x), __float_as_uint(o[1] * f.y), __float_as_uint(o[2] * f.z),
                           __float_as_uint(o[3] * f.w));
                  l[2 * i].x *= f.x, l[2 * i].y *= f.y, l[2 * i + 1].x *= f.z, l[2 * i + 1].y *= f.w;
                }
                tmem_st_wait();
              }
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = __fadd2_rn(l[i], add[i]);
          }
          tc_fence_before();
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ctl->s_free[buf]);
            mbar_arrive(&ctl->p_full[buf]);
          }
        }
      }
      if (!ok) break;
      // the next item's queries go in under this one's end: all its scores have been read
      const int slot = it.slot;
      it.step();
      ok = wait(c, &ctl->it_full[it.slot], it.phase, 4u);
      if (!ok) break;
      queries(it.slot);
      const Item& w = ctl->item[slot];
      const bool whole = w.whole;
      if (h < groups) {
        // the rows' sums
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = live ? (i & 1 ? l[i >> 1].y : l[i >> 1].x) : 0.f;
        const float part = across<true>(x, lane);
        if ((lane & 1) == 0) ctl->sums[wl][16 * h + (lane >> 1)] = part;
        ok = meet() && wait(c, &ctl->p_free[(n - 1u) & 1u], ((n - 1u) >> 1) & 1u, 11u);
        if (!ok) break;
        tc_fence_after();
        const int r = 16 * h + (lane & 15);
        float sum = (ctl->sums[0][r] + ctl->sums[1][r]) + (ctl->sums[2][r] + ctl->sums[3][r]);
        if (ctl->hidden[slot].any != 0u) sum = sum_or_nan(a, w, ctl->hidden[slot], r, sum);
        const float m = ctl->scale[turn][r];
        const float f = whole ? divisor(m, sum) : m == kNone ? 0.f : 1.f;
        const size_t rec = whole ? 0 : static_cast<size_t>(w.slot) * a.slot_rows;
        if (!whole && lane < 16 && r < w.rows)  // (all four warps write the same)
          a.rec_ml[rec + r] = make_float2(m == kNone ? -INFINITY : m, sum);
        const int dim = (key & ~3) | ((key & 1) << 1) | ((key >> 1) & 1);  // stored order 0, 2, 1, 3
        const int rr = w.r0 + 16 * h, left = w.rows - 16 * h;
        int tok = rr / a.G, in = rr - tok * a.G;
        uint16_t* y = a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + in) * kD + dim;
        float* z = a.rec + (rec + 16 * h) * kD + key;
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 4) {
          float o[4];
          tmem_ld4(tmem + lanes + kColO + 16 * h + i0, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = __shfl_sync(0xFFFFFFFFu, f, i0 + i) * o[i];
            if (i0 + i < left) {
              if (whole)
                *y = static_cast<uint16_t>(bf16x2_rn(v, 0.f));
              else
                *z = v;
            }
            z += kD, y += kD;
            if (++in == a.G) in = 0, y += a.ldo - static_cast<long long>(a.G) * kD;
          }
        }
        tc_fence_before();
      }
      if (!whole && h < groups) {
        // Of each warp, the last part's to arrive adds the parts up: it needs
        // what the same warps of the other blocks wrote, no more.
        __threadfence();
        __syncwarp();
        uint32_t* count = a.count + kChunkCounters * w.first + warp;
        const uint32_t before = __shfl_sync(0xFFFFFFFFu, lane == 0 ? atomicAdd(count, 1u) : 0u, 0);
        if (before == static_cast<uint32_t>(w.parts) - 1u) {
          if (lane == 0) *count = 0u;
          __threadfence();
          merge_share(a, w, ctl->ranges, 16 * h, 32 * wl, lane);
        }
      }
      warp_arrive(&ctl->it_empty[slot], lane);
    }
  }
  finish(a, ctl, kMmaWarp, t);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_chunk_few(const ChunkArgs& a, cudaStream_t stream) {
  const int bytes = static_cast<int>(L::bytes);
  const cudaError_t e = cudaFuncSetAttribute(chunk_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  chunk_few_kernel<<<a.grid, kBlock, bytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fsops
