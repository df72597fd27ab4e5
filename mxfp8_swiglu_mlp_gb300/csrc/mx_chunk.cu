// mx_chunk.cu -- attention of a chunk of new tokens of each sequence over the
// paged MXFP8 cache.
//
//   out[i, h] = sum_t p[t] V^[t] / sum_t p[t],  p[t] = exp(sm_scale q[i, h] . K^[t] - m)
//   over the tokens t <= pos(i) (and t > pos(i) - window),
// with K^, V^ the dequantised cache: one pass over the keys in tiles of 112,
// with a running maximum m and sum a row.  This kernel takes query tiles of 256
// rows; batches of up to kChunkFewRows rows a sequence go to mx_chunk_few.cu.
//
// One persistent block an SM; its share of the work is a range of key tiles of
// consecutive query tiles (mx_chunk_plan.cuh).  Its warps:
//   softmax   two groups of four warps, a thread a row: scores from tensor
//             memory, exponentials, probabilities back as bf16;
//   convert   V's codes times their block's power of two to bf16 operand tiles
//             in shared memory;
//   mma       two warps, one a stream, issue the products (tcgen05);
//   load      two warps copy pages of codes into a ring for K and one for V,
//             and their scales; one of them walks the plan.
// The two softmax groups ("streams") have score and output tiles of their own
// in tensor memory, so that the products of one run under the exponentials of
// the other.  With more than 128 rows a stream is a half of the query tile and
// both see every key tile; with fewer, the streams share the rows and take the
// key tiles in turn, and their results are added at the end.
//
// Scores.  K stays as it is in the cache: its codes and scales (one per 32
// dimensions, the depth of one block-scaled MMA step) are an operand of
// tcgen05.mma kind::mxf8f6f4.  A query (bf16, 8 significant bits) is the sum of
// two E4M3 numbers (4 bits each), its rounding and the rest, each with its own
// block scales, so two such products give q . K^: exact for elements down to
// 2^-14 of their block's largest, to 2^-22 of it below.  At twice the bf16 rate
// they cost what one bf16 product would, and K needs no conversion.
// Outputs.  V's scales vary along the summed dimension, so V is widened to
// bf16 (exact: four significant bits) by the convert warps, once a key tile,
// and multiplied by the probabilities from tensor memory.
// A key tile is 112 tokens: two score tiles, two outputs of 128 columns and the
// scale factors then share the 512 columns of tensor memory.  A stream's scores
// are two sections of 64 and 48 keys, each computed, turned into probabilities
// (in its place) and used by itself: while one is under the exponentials, the
// other's products and the next tile's scores are.
//
// The probabilities are rounded to bf16 (2^-8 at most, the size of the output's
// own rounding, independent from token to token); maxima, sums and outputs are
// fp32.  The maximum that scales a row is raised only when it would grow by
// more than 2^8 (bf16 keeps its relative precision up there), which spares
// nearly every rescaling of the outputs.
//
// What bounds it: the products read their operands from shared memory at 128
// bytes a cycle (48 cycles for 128 rows, 64 keys and 32 dimensions, 42 for 48
// keys; 64 for 16 tokens of V), 2340 cycles for a key tile and 256 rows; the
// streams' exponentials and hand-offs bring that to 3100.  Measured: 2048 tokens
// of 32 query heads against 16 k tokens (515 GFLOP) in 397 us, 1.30 PFLOP/s, 0.69
// of cuBLAS's bf16 rate.
// The roles' code is at the limit of what is fetched in time: the same roles in
// other orders of their branches take 399 to 485 us (this order is among the
// best), and code at an item's ends that is a little longer up to 8 % more.
// (V is widened by a loop of 45 instructions for the same reason: 7 copies of them
// took 118 us instead of 97 for trees of 15 nodes.)
// A 112-token tile kept whole instead of two sections took 515 us (its scores
// and probabilities at once are more registers than a thread has), 16 softmax
// warps and eight converting ones more as well.
//
// Drafted trees (TreeArgs) are the same but for what a row sees: all held tokens that
// its window leaves, and of its own sequence's new ones those whose bits its mask has.
// A row's bits of a key tile are four words, looked up ahead of the tile's scores, at
// the few tiles in which rows differ; they cost nothing to speak of (32 sequences of
// 4096 tokens, 4 heads a KV head, tree against causal chunk: 8 nodes 78.0 us to 77.5,
// 15 nodes 97.5 to 93.9, 64 nodes 143.8 to 142.3).  A row that sees nothing has no
// maximum: its outputs are zeros.
// With up to 64 rows of a tile the time goes to the products' chain (a key tile every
// 1800 cycles, 1170 of them products) and to the items' ends (10000 cycles each, a
// third of them the next queries, a fifth the outputs): 283 MB of cache, 32 sequences
// of 2 k to 6 k tokens with 6 to 24 nodes, take 97 us, 2.9 TB/s.
#include "mx_chunk_parts.cuh"

namespace fsops {

namespace {

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kConvWarps, kLoadWarp = kMmaWarp + 2;  // two warps each
constexpr int kBlock = 32 * (kLoadWarp + 2);
constexpr int NK = 4, NV = 3;                         // tiles of K and of V's codes in flight
constexpr int kSlots = 2;                             // bf16 V tiles
// The plan's costs, in eighths of a key tile against 256 rows.  Measured: tile
// 50 against 10: 77 to 96 us for three prompt chunks of 512 tokens among 21
// decoding sequences; least 80 against 10: 55 to 115 us for 64 rows of one
// sequence against 8000 tokens; a query tile a block against equal shares: 78
// to 90 us for 128 query tiles of 39 key tiles, 142 to 137 for tiles of 77.
constexpr int kTileCost = 50;
constexpr int kPartCost = 55;                         // units that a part costs to write and merge
constexpr int kLeastUnits = 80;                      // of a block
constexpr uint32_t kQCodes = 128 * kD;                // bytes of one term of a query tile's half
constexpr int kFirst = 64;                            // keys of a tile's first section
// Columns of tensor memory: scores and (in their place) probabilities of the
// streams, outputs, scale factors of the queries (stream, term) and of K
// (stream, tile parity).
constexpr uint32_t kColS = 128, kColO = 256, kColSfq = 112, kColSfk = 240;
static_assert(kColS == 128, "a stream's scores and outputs are equally far apart");

struct Ctl {
  uint64_t k_full[NK], k_empty[NK], r_full[NV], r_empty[NV];  // rings of K and V codes
  uint64_t v_full[kSlots], v_empty[kSlots];
  uint64_t s_full[2][2], p_full[2][2];  // stream, section
  uint64_t o_first[2], o_done[2], q_full, q_free, fin[2];
  uint64_t second, taken;  // the second stream's sums ready, and read
  uint64_t it_full[2], it_empty[2];
  Item item[2];
  HiddenNan hidden[2];
  float2 ml[128];                    // maxima and sums of the second stream's rows
  long long red[kBlock / 32][3];
  chunk::Ranges ranges;
  uint32_t tmem, stop;
};
struct L {
  static constexpr uint32_t q = 0, v = 2 * 2 * kQCodes, k = v + kSlots * kOperand, raw = k + NK * kCodes,
                            sfk = raw + NV * kCodes, sv = sfk + NK * kScales, sfq = sv + NV * kScales,
                            ctl = sfq + 2 * 2 * kScales, bytes = ctl + sizeof(Ctl);
};
static_assert(L::bytes <= 232448, "shared memory");

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// kind::f16, fp32 sums, bf16 operands, M = N = 128, B N-major (bit 16).
constexpr uint32_t kIdescPv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// ---------------------------------------------------------------- softmax warps
// Rows first .. first + rows - 1 of a query tile's half (row i is row r0 + i of
// the sequence; the last one stands in for rows past the end), by four warps
// (rows a multiple of 16), the next rows on their way meanwhile.
__device__ __forceinline__ void load_queries(const ChunkArgs& a, const Item& w, int r0, uint8_t* codes, uint8_t* sf, int first,
                                             int rows, int warp, int lane) {
  const int R = w.n * a.G;
  const uint32_t flip = a.negate ? 0x80008000u : 0u;
  const int c = lane & 15, i0 = first + warp * 2 + (lane >> 4);
  auto load = [&](int i) {
    const int rr = min(r0 + i, R - 1), tok = rr / a.G;
    return __ldg(reinterpret_cast<const uint4*>(a.q + static_cast<long long>(w.c0 + tok) * a.ldq +
                                                (w.hk * a.G + rr - tok * a.G) * kD) + c);
  };
  uint4 x0 = load(i0), x1 = load(i0 + 8);
#pragma unroll 1
  for (int i = 0; i < rows; i += 16) {
    const uint4 y0 = x0, y1 = x1;
    if (i + 16 < rows) x0 = load(i0 + i + 16), x1 = load(i0 + i + 24);
    store_query(y0, flip, codes, sf, i0 + i, 128, c);
    store_query(y1, flip, codes, sf, i0 + i + 8, 128, c);
  }
}

struct RowState {
  float m, l;  // running maximum (base 2, scaled) and sum
};
// Scores of one key tile of the thread's row to probabilities.  from / upto:
// the columns that the row sees are from <= column < upto.
template <int n>
__device__ __forceinline__ void mask_cols(float (&s)[n], int col0, int from, int upto) {
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (col0 + i < from || col0 + i >= upto) s[i] = -INFINITY;
}
// Of a tree: the section's columns col0 .. col0 + 31 that drafted token i sees,
// held ones by from <= column < upto, drafted ones (from upto on) by its mask.
__device__ __forceinline__ uint32_t tree_cols(const TreeArgs& a, const Item& w, int i, int from, int upto, int col0) {
  auto below = [](int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
  return tree_bits(a, w, i, col0 - upto) | (below(upto - col0) & ~below(from - col0));
}
template <int n>
__device__ __forceinline__ void hide_cols(float (&s)[n], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (!(seen >> i & 1u)) s[i] = -INFINITY;
}
template <int n>
__device__ __forceinline__ float max_cols(const float (&s)[n]) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i + 7 < n; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max3(m[j], s[i + 2 * j], s[i + 2 * j + 1]);
#pragma unroll
  for (int i = n - 4; i < n; ++i) m[i & 3] = fmaxf(m[i & 3], s[i]);
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
// p = 2^(s * scale - ms) as bf16 pairs; the sum of p joins `sum`.
template <int n>
__device__ __forceinline__ void exp_cols(const float (&s)[n], float scale, float ms, float2& sum, uint32_t (&p)[n / 2]) {
  const float2 sc = make_float2(scale, scale), mm = make_float2(-ms, -ms);
#pragma unroll
  for (int i = 0; i < n / 2; ++i) {
    float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), sc, mm);
    x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
    sum = __fadd2_rn(sum, x);
    p[i] = bf16x2_rn(x.x, x.y);
  }
}
// Section u of a key tile (64 or 48 columns at S) of the thread's row; from /
// upto: the section's columns that it sees.  `before`: the barrier that says
// that the products before are done with the outputs.  (Few branches: each one
// that the compiler takes for divergent costs as much as ten columns.)
template <int u, class Args>
__device__ __forceinline__ bool softmax_section(const Ctx<Args>& c, uint32_t S, uint32_t O, bool masked, int from, int upto,
                                                bool first, RowState& st, uint64_t* before, uint32_t phase,
                                                uint32_t seen0, uint32_t seen1) {
  constexpr int n1 = u == 0 ? 32 : 16;
  const float scale = c.a.scale_log2;
  float x0[32], x1[n1];
  tmem_ld32(S, x0);
  if constexpr (u == 0)
    tmem_ld32(S + 32, x1);
  else
    tmem_ld16f(S + 32, x1);
  tmem_ld_wait();
  if constexpr (Args::kTree) {
    if (__any_sync(0xFFFFFFFFu, masked)) {
      hide_cols(x0, seen0);
      hide_cols(x1, seen1);
    }
  } else {
    if (__any_sync(0xFFFFFFFFu, masked)) mask_cols(x0, 0, from, upto), mask_cols(x1, 32, from, upto);
  }
  const float mx = fmaxf(max_cols(x0), max_cols(x1)) * scale;
  const float mo = st.m, mn = mx > mo + kGrow || mo == -INFINITY ? fmaxf(mo, mx) : mo;
  const float ms = mn == -INFINITY ? 0.f : mn;
  const float al = mn == mo ? 1.f : exp2_fast(mo - ms);
  st.m = mn;
  if (__any_sync(0xFFFFFFFFu, al != 1.f) && !first) {  // the outputs so far in the new unit
    if (!wait(c, before, phase, 11u)) return false;
    tc_fence_after();
    float o[16];
#pragma unroll 1
    for (int col = 0; col < kD; col += 16) {
      tmem_ld16f(O + col, o);
      tmem_ld_wait();
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(o[i] * al);
      tmem_st16(O + col, v);
    }
  }
  float2 sum = make_float2(0.f, 0.f), sum1 = sum;
  // the probabilities take the scores' place (all of them are in registers)
  uint32_t p0[16], p1[n1 / 2];
  exp_cols(x0, scale, ms, sum, p0);
  tmem_st16(S, p0);
  exp_cols(x1, scale, ms, sum1, p1);
  if constexpr (u == 0)
    tmem_st16(S + 16, p1);
  else
    tmem_st8(S + 16, p1);
  st.l = fmaf(st.l, al, (sum.x + sum.y) + (sum1.x + sum1.y));
  tmem_st_wait();
  return true;
}

// 32 outputs (in the order of V's stored columns) times f to a row.
__device__ __forceinline__ void put32(uint16_t* y, const float (&o)[32], float f) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    *reinterpret_cast<uint4*>(y + i) =
        make_uint4(bf16x2_rn(o[i] * f, o[i + 2] * f), bf16x2_rn(o[i + 1] * f, o[i + 3] * f),
                   bf16x2_rn(o[i + 4] * f, o[i + 6] * f), bf16x2_rn(o[i + 5] * f, o[i + 7] * f));
}
// Up to 32 rows of the tile (from row0 on, a lane a row) added up over the tile's
// parts, always in the blocks' order.  The parts lie column by column, so that a
// warp reads whole lines.
template <class Args>
__device__ __forceinline__ void merge_rows(const Args& a, const Item& w, const chunk::Ranges& rg, int row0, int rows,
                                           int lane) {
  const int own = row0 + min(lane, rows - 1);
  const int blocks = w.last - w.first + 1;
  int slots = -1, from = -32;  // slots of the parts from .. from + 31, one a lane
  auto slot_of = [&](int p) {
    if (p >= from + 32 || p < from) {
      from = p & ~31;
      slots = from + lane < blocks ? chunk::part_slot(w, rg, w.first + from + lane) : -1;
    }
    return __shfl_sync(0xFFFFFFFFu, slots, p & 31);
  };
  float M = -INFINITY;
#pragma unroll 1
  for (int p = 0; p < blocks; p += 4) {  // four loads on their way together
    int sl[4];
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sl[i] = p + i < blocks ? slot_of(p + i) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __ldcg(&a.rec_ml[static_cast<size_t>(max(sl[i], 0)) * a.slot_rows + own].x);
#pragma unroll
    for (int i = 0; i < 4; ++i) M = fmaxf(M, sl[i] < 0 ? -INFINITY : m[i]);
  }
  const int rr = w.r0 + own, tok = rr / a.G;
  uint16_t* y = a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + rr - tok * a.G) * kD;
#pragma unroll 1
  for (int chunk = 0; chunk < kD / 32; ++chunk) {
    float o[32], den = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 1
    for (int p = 0; p < blocks; ++p) {
      const int sl = slot_of(p);
      if (sl < 0) continue;
      const float* src = a.rec + (static_cast<size_t>(sl) * kD + 32 * chunk) * a.slot_rows + own;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __ldcg(src + static_cast<size_t>(i) * a.slot_rows);
      const float2 ml = __ldcg(&a.rec_ml[static_cast<size_t>(sl) * a.slot_rows + own]);
      const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - M);
      den = fmaf(f, ml.y, den);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = fmaf(f, v[i], o[i]);
    }
    float inv = divisor(M, den);
    if constexpr (Args::kTree)
      if (M == -INFINITY) inv = divisor_of_none(a, w, own);
    if (lane < rows) put32(y + 32 * chunk, o, inv);
  }
}

template <class Args>
__global__ void __launch_bounds__(kBlock, 1) chunk_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + L::ctl);
  const Ctx<Args> c{a, &ctl->stop, a.tries};
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int qs = a.tile_rows / a.G, rs = a.tile_rows % a.G;
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      mbar_init(&ctl->k_full[i], 32);
      mbar_init(&ctl->k_empty[i], 2);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      mbar_init(&ctl->r_full[i], 32);
      mbar_init(&ctl->r_empty[i], kConvWarps);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl->v_full[i], kConvWarps);
      mbar_init(&ctl->v_empty[i], 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mbar_init(&ctl->s_full[i][u], 1);
        mbar_init(&ctl->p_full[i][u], 128);
      }
      mbar_init(&ctl->o_first[i], 1);
      mbar_init(&ctl->o_done[i], 1 + a.extra_arrivals);
      mbar_init(&ctl->fin[i], 1);
      mbar_init(&ctl->it_full[i], 32);
      mbar_init(&ctl->it_empty[i], kSoftWarps + kConvWarps + 3);
    }
    mbar_init(&ctl->q_full, kSoftWarps);
    mbar_init(&ctl->q_free, 2);
    mbar_init(&ctl->second, 4);
    mbar_init(&ctl->taken, 4);
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
    // ---- products of stream m: the warp walks together, one lane issues
    const int m = warp - kMmaWarp;
    const uint64_t dk = smem_desc(smem_u32(smem + L::k), 16, 1024, kSwizzle128B);
    const uint64_t dv = smem_desc(smem_u32(smem + L::v), kHalf, 1024, kSwizzle128B);
    const uint64_t dsk = smem_desc(smem_u32(smem + L::sfk), 0, 128, kSwizzleNone);
    const uint32_t S = tmem + m * kColS, O = tmem + kColO + m * 128, sfq = tmem + kColSfq + 8 * m;
    Ring<2> it;
    Ring<NK> kr;
    Ring<kSlots> vr;
    uint32_t q_phase = 0, p_phase = 0, odd = 0;
    for (;; it.step()) {
      if (!wait(c, &ctl->it_full[it.slot], it.phase, 4u)) break;
      const int tiles = __shfl_sync(0xFFFFFFFFu, ctl->item[it.slot].t1 - ctl->item[it.slot].t0, 0);
      const bool pair = __shfl_sync(0xFFFFFFFFu, ctl->item[it.slot].rows, 0) > 128;
      warp_arrive(&ctl->it_empty[it.slot], lane);
      if (tiles == 0) break;
      if (!wait(c, &ctl->q_full, q_phase, 5u)) break;
      q_phase ^= 1u;
      tc_fence_after();
      // the stream's queries (one half of the tile, or all of it) and their scales
      const int qt = pair ? 2 * m : 0;
      const uint64_t dq = smem_desc(smem_u32(smem + L::q + qt * kQCodes), 16, 1024, kSwizzle128B);
      const uint64_t dsq = smem_desc(smem_u32(smem + L::sfq + qt * kScales), 0, 128, kSwizzleNone);
      if (elect_one()) {
        tc_cp_32x128b_warpx4(sfq, dsq);
        tc_cp_32x128b_warpx4(sfq + 4, dsq + (kScales >> 4));
      }
      __syncwarp();
      const int step = pair ? 1 : 2, begin = pair ? 0 : m;
      const int last = tiles - 1 - (pair ? 0 : ((tiles - 1 - begin) & 1));  // the stream's last tile (below begin: none)
      int kt = 0, vt = 0;  // the next tile of the ring, of the bf16 slots
      // tiles of the other stream are let go unused
      auto skip_k = [&](int to) -> bool {
        for (; kt < to; ++kt) {
          if (!wait(c, &ctl->k_full[kr.slot], kr.phase, 6u)) return false;
          if (lane == 0) mbar_arrive(&ctl->k_empty[kr.slot]);
          kr.step();
        }
        return true;
      };
      auto skip_v = [&](int to) -> bool {
        for (; vt < to; ++vt) {
          if (!wait(c, &ctl->v_full[vr.slot], vr.phase, 7u)) return false;
          if (lane == 0) mbar_arrive(&ctl->v_empty[vr.slot]);
          vr.step();
        }
        return true;
      };
      // a tile's K and its scales are there
      auto keys = [&](int j) -> bool {
        if (!skip_k(j) || !wait(c, &ctl->k_full[kr.slot], kr.phase, 6u)) return false;
        fence_proxy_async_shared();  // the scales came by generic copies
        odd ^= 1u;
        return true;
      };
      // (by one lane) section u of a tile's scores; the first one brings K's scales
      auto scores = [&](int u, bool end) {
        const uint64_t k0 = dk + kr.slot * (kCodes >> 4) + u * (kFirst * kD >> 4);
        const uint32_t sfk = tmem + kColSfk + 8 * m + 4 * odd, d = S + kFirst * u;
        const uint32_t idesc = idesc_mxf8_e4m3(0, 0, 0) | (((u ? kKeys - kFirst : kFirst) >> 3) << 17);
        if (u == 0) tc_cp_32x128b_warpx4(sfk, dsk + kr.slot * (kScales >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // step k / 2 of 32 dimensions, term k % 2
          const uint32_t o = (32 * (k >> 1)) >> 4;
          tc_mma_mxf8(d, dq + (k & 1) * (kQCodes >> 4) + o, k0 + o, idesc | ((k >> 1) << 4) | ((k >> 1) << 29),
                      sfq + 4 * (k & 1), sfk + 2 * u, k > 0);
        }
        tc_commit(&ctl->s_full[m][u]);
        if (u) {
          tc_commit(&ctl->k_empty[kr.slot]);
          if (end) tc_commit(&ctl->q_free);
        }
      };
      auto keys_done = [&]() {
        kr.step();
        ++kt;
      };
      // Tile j: what does not depend on the probabilities is waited for first;
      // once they are there, their products and the next tile's scores go out
      // in one piece.  (Tile begin - step has no probabilities.)
      bool ok = true;
      if (begin > last && lane == 0) mbar_arrive(&ctl->q_free);
#pragma unroll 1
      for (int j = begin - step; ok && j <= last && begin <= last; j += step) {
        const bool head = j < begin, more = j < last;
        if (!head) ok = skip_v(j) && wait(c, &ctl->v_full[vr.slot], vr.phase, 7u);
        if (ok && more) ok = keys(j + step);
        const uint64_t v0 = dv + vr.slot * (kOperand >> 4);
#pragma unroll 1
        for (int u = 0; ok && u < 2; ++u) {
          if (!head) ok = wait(c, &ctl->p_full[m][u], p_phase, 8u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vu = v0 + u * (kFirst * 128 >> 4);
          const uint32_t p = S + kFirst * u;
          if (elect_one()) {
            if (!head) {
#pragma unroll
              for (int k = 0; k < 3; ++k)
                mma_ts(O, p + 8 * k, vu + k * (2048 >> 4), kIdescPv, (j > begin || u > 0 || k > 0) ? 1u : 0u);
              if (u == 0) {
                mma_ts(O, p + 24, vu + 3 * (2048 >> 4), kIdescPv, 1u);
                if (!more) tc_commit(&ctl->o_first[m]);
              } else {
                tc_commit(&ctl->v_empty[vr.slot]);
                if (!more) tc_commit(&ctl->o_done[m]);
              }
            }
            if (more) scores(u, j + step == last);
          }
          __syncwarp();
        }
        if (!head) {
          p_phase ^= 1u;
          vr.step();
          ++vt;
        }
        if (more) keys_done();
      }
      ok = ok && skip_k(tiles) && skip_v(tiles);
      if (!ok) break;
    }
  } else if (warp >= kSoftWarps) {
    convert_items<NV, kSlots, 1>(c, ctl, smem + L::raw, smem + L::sv, smem + L::v, t - 32 * kSoftWarps, lane);
  } else {
    // ---- softmax: stream m, a thread a row
    const int m = warp >> 2, wl = warp & 3, row = 32 * wl + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * wl) << 16;
    const uint32_t S = tmem + lanes + m * kColS;  // (the outputs are kColO further)
    // the queries of the item in a slot, when the products are done with the last ones
    auto queries = [&](int slot) {
      const Item& w = ctl->item[slot];
      if (w.t0 == w.t1) return;
      // (each of a pair its half; else half of the rows of warps that have any: 16 to 64)
      const bool pair = w.rows > 128;
      const int rows = pair ? 128 : 16 * ((w.rows + 31) >> 5);
      load_queries(a, w, w.r0 + (pair ? 128 * m : 0), smem + L::q + (pair ? m * 2 * kQCodes : 0),
                   smem + L::sfq + (pair ? m * 2 * kScales : 0), pair ? 0 : rows * m, rows, wl, lane);
      fence_proxy_async_shared();
      warp_arrive(&ctl->q_full, lane);
    };
    Ring<2> it;
    uint32_t s_phase = 0, o_phase = 0, x_phase = 0, f_phase = 0;
    bool ok = wait(c, &ctl->it_full[0], 0, 4u);
    if (ok) queries(0);
    // (what an item's end needs is read again there, to keep the loop's registers few)
#pragma unroll 1
    while (ok) {
      RowState st{-INFINITY, 0.f};
      bool any;
      {
        const Item& w = ctl->item[it.slot];  // given back at the item's end
        if (w.t0 == w.t1) break;
        const bool pair = w.rows > 128;
        const int rr = w.r0 + min((pair ? 128 * m : 0) + row, w.rows - 1);
        // the row sees the tokens from .. upto - 1, the warp's rows all of those lo .. hi - 1
        // (of a tree: the held tokens from .. upto - 1, all rows all of those lo .. hi - 1)
        const int tok = rr / a.G, upto = w.len - w.n + (Args::kTree ? 0 : tok + 1);
        int from = a.window > 0 ? upto - a.window : 0;
        if constexpr (Args::kTree) from = tree_from(a, w, tok);
        const int lo = __reduce_max_sync(0xFFFFFFFFu, from), hi = __reduce_min_sync(0xFFFFFFFFu, upto);
        const bool busy = (pair ? 128 * m : 0) + 32 * wl < w.rows;  // the warp has a row
        const int step = pair ? 1 : 2, t1 = w.t1;
        int k = w.t0 + (pair ? 0 : m);
        any = k < t1;
#pragma unroll 1
        for (bool first = true; k < t1; k += step, first = false) {
          const int tok0 = k * kKeys, tok1 = tok0 + kFirst;
          // (of a tree: the tile's columns that the row sees, looked up while the scores are computed)
          uint32_t seen[4] = {0u, 0u, 0u, 0u};
          if constexpr (Args::kTree) {
            if (tok0 < lo || tok0 + kKeys > hi) {
#pragma unroll
              for (int i = 0; i < 4; ++i) seen[i] = tree_cols(a, w, tok, from - tok0, upto - tok0, 32 * i);
            }
          }
          // the products before a section are done when the scores issued after
          // them are there: this tile's second ones, the next tile's first
          ok = wait(c, &ctl->s_full[m][0], s_phase, 10u);
          if (!ok) break;
          tc_fence_after();
          if (busy)
            ok = softmax_section<0>(c, S, S + kColO, tok0 < lo || tok1 > hi, from - tok0, upto - tok0, first, st,
                                    &ctl->s_full[m][1], s_phase, seen[0], seen[1]);
          tc_fence_before();
          mbar_arrive(&ctl->p_full[m][0]);
          ok = ok && wait(c, &ctl->s_full[m][1], s_phase, 10u);
          if (!ok) break;
          tc_fence_after();
          const bool more = k + step < t1;
          if (busy)
            ok = softmax_section<1>(c, S + kFirst, S + kColO, tok1 < lo || tok0 + kKeys > hi, from - tok1, upto - tok1, false,
                                    st, more ? &ctl->s_full[m][0] : &ctl->o_first[m], more ? s_phase ^ 1u : o_phase, seen[2], seen[3]);
          tc_fence_before();
          mbar_arrive(&ctl->p_full[m][1]);
          if (!ok) break;
          s_phase ^= 1u;
        }
      }
      // the next item's queries go in under this one's end
      ok = ok && wait(c, &ctl->q_free, f_phase, 5u);
      if (!ok) break;
      f_phase ^= 1u;
      const int slot = it.slot;
      it.step();
      ok = wait(c, &ctl->it_full[it.slot], it.phase, 4u);
      if (!ok) break;
      queries(it.slot);
      if (any) {
        ok = wait(c, &ctl->o_done[m], o_phase, 11u);
        if (!ok) break;
        o_phase ^= 1u;
        tc_fence_after();
      }
      const Item& w = ctl->item[slot];
      const bool pair = w.rows > 128;
      const int tr = (pair ? 128 * m : 0) + row;                  // row in the tile
      const bool busy = tr - lane < w.rows, write = tr < w.rows;  // of the warp, of the thread
      float f0 = 1.f, f1 = 0.f;  // the streams' shares of the row's output
      if (!pair) {
        // the second stream's maximum and sum to the first, which adds both up
        if (m == 1) {
          ctl->ml[row] = make_float2(st.m, st.l);
          warp_arrive(&ctl->second, lane);
        } else {
          ok = wait(c, &ctl->second, x_phase, 12u);
          if (!ok) break;
          const float m1 = ctl->ml[row].x, l1 = ctl->ml[row].y, M = fmaxf(st.m, m1);
          f0 = st.m == -INFINITY ? 0.f : exp2_fast(st.m - M);
          f1 = m1 == -INFINITY ? 0.f : exp2_fast(m1 - M);
          st.l = f0 * st.l + f1 * l1;
          st.m = M;
          tc_fence_after();
        }
      }
      if (pair || m == 0) {
        if (ctl->hidden[slot].any != 0u) st.l = sum_or_nan(a, w, ctl->hidden[slot], tr, st.l);
        const bool two = !pair && w.t1 - w.t0 > 1, whole = w.whole;
        float* rec = nullptr;
        uint16_t* y = nullptr;
        if (whole) {
          float inv = divisor(st.m, st.l);
          if constexpr (Args::kTree)
            if (st.m == -INFINITY) inv = divisor_of_none(a, w, tr);
          f0 *= inv, f1 *= inv;
          const int rr = w.r0 + min(tr, w.rows - 1), tok = rr / a.G;
          y = a.out + static_cast<long long>(w.c0 + tok) * a.ldo + (w.hk * a.G + rr - tok * a.G) * kD;
        } else {
          const size_t slot = w.slot;
          rec = a.rec + slot * kD * a.slot_rows + min(tr, w.rows - 1);
          if (write) a.rec_ml[slot * a.slot_rows + tr] = make_float2(st.m, st.l);
        }
        if (busy) {
#pragma unroll 1
          for (int col = 0; col < kD; col += 32) {
            float o[32];
            tmem_ld32(S + kColO + col, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f0;
            if (two) {
              float o1[32];
              tmem_ld32(S + kColO + 128 + col, o1);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(f1, o1[i], o[i]);
            }
            if (write) {
              if (whole) {
                put32(y + col, o, 1.f);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) rec[static_cast<size_t>(col + i) * a.slot_rows] = o[i];
              }
            }
          }
        }
        tc_fence_before();
        if (!whole && busy) {
          // Of each warp, the last part's to arrive adds the parts up: it needs
          // what the same warps of the other blocks wrote, no more.
          __threadfence();
          __syncwarp();
          uint32_t* count = a.count + kChunkCounters * w.first + warp;
          const uint32_t before = __shfl_sync(0xFFFFFFFFu, lane == 0 ? atomicAdd(count, 1u) : 0u, 0);
          if (before == static_cast<uint32_t>(w.parts) - 1u) {
            if (lane == 0) *count = 0u;
            __threadfence();
            merge_rows(a, w, ctl->ranges, tr - lane, min(32, w.rows - (tr - lane)), lane);
          }
        }
      }
      if (!pair) {  // the second stream goes on when its tiles have been read
        if (m == 0) {
          warp_arrive(&ctl->taken, lane);
        } else {
          ok = wait(c, &ctl->taken, x_phase, 14u);
          if (!ok) break;
          tc_fence_after();
        }
        x_phase ^= 1u;
      }
      warp_arrive(&ctl->it_empty[slot], lane);
    }
  }
  finish(a, ctl, kMmaWarp, t);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

// Which kernel: by the average rows of a sequence.  Measured, this one against the
// one for few rows (us): 16 sequences of 3000 tokens with 8 rows 37 to 35, with 32
// rows 37 to 35, with 40 rows 39 to 61; 64 of 2 k to 6 k tokens with 4 rows 163 to
// 127, with 32 161 to 137, with 40 164 to 246.
int chunk_tile_rows(int T, int B, int G) {
  return static_cast<long long>(T) * G > static_cast<long long>(kChunkFewRows) * B ? 256 : kChunkFewRows;
}

// Trees: the kernel for few rows too where its query tiles are no more than the blocks
// and no block has more than some 24 key tiles, by the lengths that the tables have room
// for or, where it is less, a window with a mask's nodes (lengths themselves are on the
// device).  There a call's time is its longest chain, and shorter items make that shorter.
// Measured, trees of 16 nodes, 4 heads a KV head of 8, this kernel against that one (us):
// one tree and 500 tokens 16.4 to 14.5, 4 k 37 to 25, 16 k (15 key tiles a block) 50 to
// 35, 64 k (62) 81 to 78; one of 64 nodes and 4 k (16) 47 to 35, 16 k (62) 66 to 76; one
// of 128 and 4 k (31) 49 to 48; 8 trees and 2 k (15) 28.9 to 26.9, 8 k (62) 60 to 78; 16
// trees and 500 tokens (256 query tiles) 16.7 to 33.  With a window, 8 k tokens in tables
// for 128 k: one tree of 16 nodes and 512 tokens 16.1 to 14.5, 2 k 28.3 to 19.9, 4 k 33.8
// to 29.9; of 64 nodes and 512 24.7 to 16.2, 2 k 41.7 to 26.8; 8 trees and 512 16.9 to 14.8.
int tree_tile_rows(int T, int B, int G, int Hkv, long long tokens, int blocks) {
  const long long rows = (static_cast<long long>(T) * G + B - 1) / B;  // of a sequence, on average
  const long long tiles = (rows + kChunkFewRows - 1) / kChunkFewRows * B * Hkv, keys = (tokens + kKeys - 1) / kKeys;
  return tiles <= blocks && tiles * keys <= 24LL * blocks ? kChunkFewRows : chunk_tile_rows(T, B, G);
}

template <class Args>
static cudaError_t launch_many(const Args& a, cudaStream_t stream) {
  const int bytes = static_cast<int>(L::bytes);
  const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  chunk_kernel<Args><<<a.grid, kBlock, bytes, stream>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t stream) {
  return a.tile_rows == 256 ? launch_many(a, stream) : launch_chunk_few(a, stream);
}
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  return a.tile_rows == 256 ? launch_many(a, stream) : launch_tree_few(a, stream);
}

}  // namespace fsops
