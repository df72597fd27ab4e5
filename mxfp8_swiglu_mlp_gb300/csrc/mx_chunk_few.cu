// mx_chunk_few.cu -- the chunk attention of mx_chunk.cu for few rows: query
// tiles of up to 64 rows (single tokens, drafted tokens), whose time is the
// cache's bytes.
//
// With queries as the 128 rows of a product, a few of them would leave most of
// it empty, and all exponentials to one warp.  So here the products are turned
// round: keys are the rows of the scores, S^T = K Q^T, and dimensions the rows
// of the outputs, O^T = V^T P^T, and the query rows their columns.
//   S^T  [112 keys][2 x rows]  block-scaled E4M3 MMA on K's own codes; the two
//        E4M3 terms of the queries are two groups of columns, added afterwards;
//   P^T  [112 keys][64 rows] bf16 in shared memory, N-major;
//   O^T  [128 dimensions][64 rows] with V widened to bf16 as the M-major operand.
// A key tile costs 4 + 7 MMAs this way (with 32 rows about 200 + 330 cycles of
// the tensor pipe), less than its 30 KB take to arrive (1250 cycles at the
// card's copy rate), and a thread has one key and 16 rows of a tile: 8 warps,
// four a group of 16 rows (two groups for more than 32 rows).
//
// A row's scale (its running maximum) is the same for all keys of a tile, so
// the four warps of a row vote: while no score passes the scale by more than
// 2^8, and nearly always none does, nothing is exchanged but the vote, and the
// exponentials are computed under it.  Else they find the maximum together and
// rescale.  A row's sum stays apart in the 112 threads until the item's end.
//
// Products of one key tile run under the exponentials of another (scores and
// probabilities are double buffered); loads run ahead over the items' ends, and
// the next item's first scores are computed under this one's end.
#include "mx_chunk_parts.cuh"

namespace fsops {

namespace {

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kConvWarps, kLoadWarp = kMmaWarp + 2;  // two warps each
constexpr int kBlock = 32 * (kLoadWarp + 2);
constexpr int NK = 5, NV = 3;                 // tiles of K and of V's codes in flight
constexpr int kRows = kChunkFewRows;
constexpr uint32_t kProbs = kKeys * kRows * 2;  // a tile's probabilities
static_assert(kRows == 64, "128 bytes of probabilities a key, one swizzle atom wide");
// Columns of tensor memory: two tiles of scores, the outputs, scale factors of
// the queries and of K (two tiles).
constexpr uint32_t kColS = 128, kColO = 256, kColSfq = 320, kColSfk = 324;
constexpr float kNone = -3e38f;  // the scale of a row that has seen nothing

struct Ctl {
  uint64_t k_full[NK], k_empty[NK], r_full[NV], r_empty[NV];  // rings of K and V codes
  uint64_t v_full[kSlots], v_empty[kSlots];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];  // by tile parity
  uint64_t q_full, vote[2], group, fin[2], it_full[2], it_empty[2];
  Item item[2];
  float scale[2][kRows];     // the rows' scales (base 2), the one in use by turns
  float peak[2][4][16];      // a group's maxima, of each warp
  float sums[4][kRows];
  uint32_t grown[2];         // the last vote that found a larger score
  long long red[kBlock / 32];
  chunk::Ranges ranges;
  uint32_t tmem, stop, last;
};
struct L {
  static constexpr uint32_t q = 0, v = 128 * kD, p = v + kSlots * kOperand, k = p + 2 * kProbs, raw = k + NK * kCodes,
                            sfk = raw + NV * kCodes, sv = sfk + NK * kScales, sfq = sv + NV * kScales,
                            ctl = sfq + kScales, bytes = ctl + sizeof(Ctl);
};
static_assert(L::bytes <= 232448 && NK <= 5 && NV <= 4, "shared memory");
static_assert(NV * kCodes >= 16 * kD, "the 128-row product reads 16 rows behind the last K tile");

// kind::f16, fp32 sums, bf16 operands, M = 128 (M-major, bit 15), N = 64 (N-major, bit 16).
constexpr uint32_t kIdescPv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                              ((static_cast<uint32_t>(kRows) >> 3) << 17) | ((128u >> 4) << 24);
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

// One row of a query tile added up over the tile's parts, in the blocks' order,
// by a warp: four (stored) dimensions a lane.
__device__ __forceinline__ void merge_row(const ChunkArgs& a, const Item& w, const chunk::Ranges& rg, int row, int lane) {
  const int blocks = w.last - w.first + 1;
  auto part = [&](int p, float2& ml) {  // the lane's part: its slot, maximum and sum
    const int sl = p < blocks ? chunk::part_slot(w, rg, w.first + p) : -1;
    ml = sl >= 0 ? __ldcg(&a.rec_ml[static_cast<size_t>(sl) * a.slot_rows + row]) : make_float2(-INFINITY, 0.f);
    return sl;
  };
  float2 ml;
  float M = -INFINITY;
  for (int base = 0; base < blocks; base += 32) {
    part(base + lane, ml);
    M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float den = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < blocks; base += 32) {
    const int sl = part(base + lane, ml);
    const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - M);
    den = fmaf(f, ml.y, den);
    const int n = min(32, blocks - base);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const int slp = __shfl_sync(0xFFFFFFFFu, sl, p);
      const float fp = __shfl_sync(0xFFFFFFFFu, f, p);
      if (fp == 0.f) continue;
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.rec + (static_cast<size_t>(slp) * a.slot_rows + row) * kD) + lane);
      o.x = fmaf(fp, x.x, o.x), o.y = fmaf(fp, x.y, o.y), o.z = fmaf(fp, x.z, o.z), o.w = fmaf(fp, x.w, o.w);
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, s);
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const int rr = w.r0 + row, tok = rr / a.G;
  uint16_t* y = a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + rr - tok * a.G) * kD;
  // (stored order 0, 2, 1, 3)
  *reinterpret_cast<uint2*>(y + 4 * lane) = make_uint2(bf16x2_rn(o.x * inv, o.z * inv), bf16x2_rn(o.y * inv, o.w * inv));
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->v_full[i], kConvWarps);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_free[i], kSoftWarps);
      mbar_init(&ctl->p_full[i], kSoftWarps);
      mbar_init(&ctl->p_free[i], 1);
      mbar_init(&ctl->vote[i], 4);
      mbar_init(&ctl->fin[i], 1);
      mbar_init(&ctl->it_full[i], 32);
      mbar_init(&ctl->it_empty[i], kSoftWarps + kConvWarps + 3);
      ctl->grown[i] = 0u;
    }
    mbar_init(&ctl->q_full, kSoftWarps);
    mbar_init(&ctl->group, kSoftWarps);
    ctl->stop = 0u;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  const long long units = chunk::all_units(a, qs, rs, ctl->red);  // a block-wide barrier inside
  if (t == 0) ctl->ranges.make(units, a.grid);
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
    const uint64_t dp = smem_desc(smem_u32(smem + L::p), kProbs, 1024, kSwizzle128B);
    Ring<2> it, buf;
    Ring<NK> kr;
    Ring<kSlots> vr;
    uint32_t q_phase = 0;
    bool issued = false;
    for (bool ok = true; ok; it.step()) {
      if (!wait(c, &ctl->it_full[it.slot], it.phase, 4u)) break;
      const int tiles = __shfl_sync(0xFFFFFFFFu, ctl->item[it.slot].t1 - ctl->item[it.slot].t0, 0);
      const uint32_t groups = __shfl_sync(0xFFFFFFFFu, (ctl->item[it.slot].rows + 15) >> 4, 0);
      warp_arrive(&ctl->it_empty[it.slot], lane);
      if (tiles == 0) break;
      issued = true;
      if (!pv) {
        if (!wait(c, &ctl->q_full, q_phase, 5u)) break;
        q_phase ^= 1u;
        tc_fence_after();
        if (elect_one()) tc_cp_32x128b_warpx4(tmem + kColSfq, dsq);
        __syncwarp();
        const uint32_t idesc = idesc_mxf8_e4m3(32 * groups, 0, 0);
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          ok = wait(c, &ctl->k_full[kr.slot], kr.phase, 6u) && wait(c, &ctl->s_free[buf.slot], buf.phase ^ 1u, 7u);
          if (!ok) break;
          fence_proxy_async_shared();  // the scales came by generic copies
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sfk = tmem + kColSfk + 4 * buf.slot;
            tc_cp_32x128b_warpx4(sfk, dsk + kr.slot * (kScales >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 dimensions
              tc_mma_mxf8(tmem + kColS * buf.slot, dk + kr.slot * (kCodes >> 4) + ((32 * k) >> 4), dq + ((32 * k) >> 4),
                          idesc | (k << 4) | (k << 29), sfk, tmem + kColSfq, k > 0);
            tc_commit(&ctl->s_full[buf.slot]);
            tc_commit(&ctl->k_empty[kr.slot]);
          }
          __syncwarp();
          kr.step();
          buf.step();
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          ok = wait(c, &ctl->v_full[vr.slot], vr.phase, 8u) && wait(c, &ctl->p_full[buf.slot], buf.phase, 8u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)  // 16 tokens
              mma_ss(tmem + kColO, dv + vr.slot * (kOperand >> 4) + k * (2048 >> 4),
                     dp + buf.slot * (kProbs >> 4) + k * (2048 >> 4), kIdescPv, (j > 0 || k > 0) ? 1u : 0u);
            tc_commit(&ctl->p_free[buf.slot]);
            tc_commit(&ctl->v_empty[vr.slot]);
          }
          __syncwarp();
          vr.step();
          buf.step();
        }
      }
    }
    if (issued && *c.stop != 0u) {  // products in flight end before tensor memory is given back
      if (elect_one()) tc_commit(&ctl->fin[pv]);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&ctl->fin[pv], 0) && globaltimer_ns() - t0 < 20000000ull) {
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarps) {
    convert_items<NV>(c, ctl, smem + L::raw, smem + L::sv, smem + L::v, t - 32 * kSoftWarps, lane);
  } else {
    // ---- softmax: group of rows h (and h + 2), a thread a key
    const int h = warp >> 2, wl = warp & 3, key = 32 * wl + lane;
    const bool live = key < kKeys;
    const uint32_t lanes = static_cast<uint32_t>(32 * wl) << 16;
    const float scale = a.scale_log2;
    uint8_t* const prow = smem + L::p + key * 128;  // the key's probabilities (of the first buffer)
    uint32_t n = 0, votes = 0;                      // key tiles, votes so far
    auto queries = [&](int slot) {
      const Item& w = ctl->item[slot];
      if (w.t0 == w.t1) return;
      const int rows = (w.rows + 15) & ~15;
      load_queries<kSoftWarps, true>(a, w, w.r0, smem + L::q, smem + L::sfq, 0, rows, rows, warp, lane);
      fence_proxy_async_shared();
      warp_arrive(&ctl->q_full, lane);
    };
    auto meet = [&]() -> bool {  // the warps of a row
      warp_arrive(&ctl->vote[h], lane);
      return wait(c, &ctl->vote[h], votes++ & 1u, 11u);
    };
    uint32_t g_phase = 0;
    auto meet_all = [&]() -> bool {
      warp_arrive(&ctl->group, lane);
      const bool r = wait(c, &ctl->group, g_phase, 13u);
      g_phase ^= 1u;
      return r;
    };
    Ring<2> it;
    bool ok = wait(c, &ctl->it_full[0], 0, 4u);
    if (ok) queries(0);
#pragma unroll 1
    while (ok) {
      float2 l[8], l1[8];  // the thread's sums, of a second group of rows too
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] = l1[i] = make_float2(0.f, 0.f);
      int turn = 0, turn1 = 0;  // which of the scales is in use
      const int groups = (ctl->item[it.slot].rows + 15) >> 4;
      {
        const Item& w = ctl->item[it.slot];  // given back at the item's end
        if (w.t0 == w.t1) break;
        const int t0 = w.t0, t1 = w.t1;
        // all rows see the tokens lo .. hi - 1
        const int base = w.len - w.n + 1, hi = base + w.r0 / a.G,
                  lo = a.window > 0 ? base + (w.r0 + w.rows - 1) / a.G - a.window : 0;
#pragma unroll 1
        for (int k = t0; k < t1; ++k, ++n) {
          const uint32_t buf = n & 1u, phase = (n >> 1) & 1u;
          const bool fresh = k == t0, masked = k * kKeys < lo || (k + 1) * kKeys > hi;
          ok = wait(c, &ctl->s_full[buf], phase, 10u);
          if (!ok) break;
          tc_fence_after();
          if (h >= groups) warp_arrive(&ctl->s_free[buf], lane);
#pragma unroll 1
          for (int g = h; g < groups; g += 2) {
            float2 s[8];
            {
              float x[16], y[16];
              const uint32_t S = tmem + lanes + kColS * buf + 16 * g;
              tmem_ld16f(S, x);
              tmem_ld16f(S + 16 * groups, y);
              tmem_ld_wait();
              if (g + 2 >= groups) {
                tc_fence_before();
                warp_arrive(&ctl->s_free[buf], lane);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                s[i] = __fadd2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(y[2 * i], y[2 * i + 1]));
            }
            if (masked) {
              const int r = w.r0 + 16 * g, tok = k * kKeys + key;
              int upto = base + r / a.G, in = r % a.G;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int u = min(upto, w.len);
                if (tok >= u || (a.window > 0 && tok < u - a.window)) (i & 1 ? s[i >> 1].y : s[i >> 1].x) = -INFINITY;
                if (++in == a.G) in = 0, ++upto;
              }
            }
            float* ms = ctl->scale[turn] + 16 * g;
            uint32_t p[8];
            float2 e[8];
            float top = -INFINITY;
            auto probs = [&]() {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 m4 = *reinterpret_cast<const float4*>(ms + 4 * i);
                e[2 * i] = __ffma2_rn(s[2 * i], make_float2(scale, scale), make_float2(-m4.x, -m4.y));
                e[2 * i + 1] = __ffma2_rn(s[2 * i + 1], make_float2(scale, scale), make_float2(-m4.z, -m4.w));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                top = max3(top, e[i].x, e[i].y);
                e[i].x = exp2_fast(e[i].x), e[i].y = exp2_fast(e[i].y);
                p[i] = bf16x2_rn(e[i].x, e[i].y);
              }
            };
            if (!fresh) {
              probs();
              if (__any_sync(0xFFFFFFFFu, live && top > kGrow) && lane == 0)
                *reinterpret_cast<volatile uint32_t*>(&ctl->grown[h]) = votes + 1u;
            }
            ok = meet();
            if (!ok) break;
            if (fresh || *reinterpret_cast<volatile uint32_t*>(&ctl->grown[h]) == votes) {
              // the rows' maxima, and what has been added up so far in the new unit
              float x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = live ? (i & 1 ? s[i >> 1].y : s[i >> 1].x) * scale : -INFINITY;
              const float mx = across<false>(x, lane);
              if ((lane & 1) == 0) ctl->peak[h][wl][lane >> 1] = mx;
              ok = meet();
              if (!ok) break;
              float* mn = ctl->scale[turn ^ 1] + 16 * g;
              if (lane < 16) {  // (every warp of the row writes the same)
                const float(*pk)[16] = ctl->peak[h];
                const float m = fmaxf(max3(pk[0][lane], pk[1][lane], pk[2][lane]), pk[3][lane]), mo = fresh ? kNone : ms[lane];
                mn[lane] = m > mo + kGrow ? m : mo;
              }
              __syncwarp();
              if (!fresh) {
                ok = wait(c, &ctl->p_free[buf ^ 1u], ((n - 1u) >> 1) & 1u, 11u);
                if (!ok) break;
                tc_fence_after();
                float o[16];
                uint32_t v[16];
                tmem_ld16f(tmem + lanes + kColO + 16 * g, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float al = exp2_fast(ms[i] - mn[i]);
                  (i & 1 ? l[i >> 1].y : l[i >> 1].x) *= al;
                  v[i] = __float_as_uint(o[i] * al);
                }
                tmem_st16(tmem + lanes + kColO + 16 * g, v);
                tmem_st_wait();
                tc_fence_before();
              }
              turn ^= 1;
              ms = mn;
              probs();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = __fadd2_rn(l[i], e[i]);
            ok = wait(c, &ctl->p_free[buf], phase ^ 1u, 12u);
            if (!ok) break;
            if (live) {
              uint4* d = reinterpret_cast<uint4*>(prow + buf * kProbs);
              d[(2 * g) ^ (key & 7)] = make_uint4(p[0], p[1], p[2], p[3]);
              d[(2 * g + 1) ^ (key & 7)] = make_uint4(p[4], p[5], p[6], p[7]);
            }
            if (h + 2 < groups) {  // the other group of the warp comes next
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 x = l[i];
                l[i] = l1[i], l1[i] = x;
              }
              const int x = turn;
              turn = turn1, turn1 = x;
            }
          }
          if (!ok) break;
          fence_proxy_async_shared();
          warp_arrive(&ctl->p_full[buf], lane);
        }
      }
      if (!ok) break;
      // the next item's queries go in under this one's end: all its scores have been read
      const int slot = it.slot;
      it.step();
      ok = wait(c, &ctl->it_full[it.slot], it.phase, 4u);
      if (!ok) break;
      queries(it.slot);
      // the rows' sums
#pragma unroll 1
      for (int g = h; g < groups; g += 2) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 s = g == h ? l[i >> 1] : l1[i >> 1];
          x[i] = live ? (i & 1 ? s.y : s.x) : 0.f;
        }
        const float sum = across<true>(x, lane);
        if ((lane & 1) == 0) ctl->sums[wl][16 * g + (lane >> 1)] = sum;
      }
      ok = meet() && wait(c, &ctl->p_free[(n - 1u) & 1u], ((n - 1u) >> 1) & 1u, 11u);
      if (!ok) break;
      tc_fence_after();
      const Item& w = ctl->item[slot];
      const bool whole = w.whole;
      const size_t rec = whole ? 0 : static_cast<size_t>(chunk::part_slot(w, ctl->ranges, blockIdx.x)) * a.slot_rows;
#pragma unroll 1
      for (int g = h; g < groups; g += 2) {
        const int r = 16 * g + (lane & 15);
        const float sum = (ctl->sums[0][r] + ctl->sums[1][r]) + (ctl->sums[2][r] + ctl->sums[3][r]);
        const float m = ctl->scale[g == h ? turn : turn1][r];
        const float f = whole ? (sum > 0.f ? 1.f / sum : 0.f) : m == kNone ? 0.f : 1.f;
        if (!whole && wl == 0 && lane < 16 && r < w.rows)
          a.rec_ml[rec + r] = make_float2(m == kNone ? -INFINITY : m, sum);
        float o[16];
        tmem_ld16f(tmem + lanes + kColO + 16 * g, o);
        tmem_ld_wait();
        const int rr = w.r0 + 16 * g, left = w.rows - 16 * g;
        int tok = rr / a.G, in = rr - tok * a.G;
        const int dim = (key & ~3) | ((key & 1) << 1) | ((key >> 1) & 1);  // stored order 0, 2, 1, 3
        uint16_t* y = a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + in) * kD + dim;
        float* z = a.rec + (rec + 16 * g) * kD + key;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float fi = __shfl_sync(0xFFFFFFFFu, f, i), v = fi != 0.f ? fi * o[i] : 0.f;
          if (i < left) {
            if (whole)
              *y = static_cast<uint16_t>(bf16x2_rn(v, 0.f));
            else
              z[i * kD] = v;
          }
          y += kD;
          if (++in == a.G) in = 0, y += a.ldo - static_cast<long long>(a.G) * kD;
        }
      }
      tc_fence_before();
      if (!whole) {
        // the last part to arrive adds them up, in the blocks' order
        __threadfence();
        ok = meet_all();
        if (!ok) break;
        if (t == 0) {
          uint32_t* count = a.count + 2 * w.first;
          const bool last = atomicAdd(count, 1u) == static_cast<uint32_t>(w.parts) - 1u;
          if (last) *count = 0u;
          ctl->last = last;
          __threadfence();
        }
        ok = meet_all();
        if (!ok) break;
        if (ctl->last)
          for (int row = warp; row < w.rows; row += kSoftWarps) merge_row(a, w, ctl->ranges, row, lane);
      }
      warp_arrive(&ctl->it_empty[slot], lane);
    }
  }
  // ---- the end: every role is here, and nothing is in flight
  __syncthreads();
  if (t == 0 && ctl->stop != 0u)  // FSOPS_ERR_TIMEOUT
    atomicCAS(a.status, 0u, (5u << 24) | (ctl->stop << 16) | (blockIdx.x & 0xFFFFu));
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
