// mx_chunk_parts.cuh -- what the two kernels of the chunk attention (mx_chunk.cu
// for many rows, mx_chunk_few.cu for few) share: bounded waits, the warps that
// load the cache and widen V, and the queries' operand.
#pragma once
#include <cuda_bf16.h>

#include "mx_chunk.h"
#include "mx_chunk_plan.cuh"

namespace fsops {

namespace {

using chunk::Item;
using chunk::kKeys;

constexpr int kD = kChunkD;
constexpr int kConvWarps = 4;
constexpr uint32_t kCodes = kKeys * kD;        // bytes of a K or V tile of codes
constexpr uint32_t kScales = 512;              // bytes kept for a tile's scales
constexpr uint32_t kOperand = kKeys * kD * 2;  // V as bf16: two halves of 64 dimensions,
constexpr uint32_t kHalf = kOperand / 2;       // [tokens][128 bytes], 128-byte swizzle
constexpr float kGrow = 8.f;                   // in powers of two
// A row's maximum in fp32 is off by half its last bit, which all its probabilities
// and their sum have as a common factor: 2^64 at most below this maximum, but
// beyond fp32 above it.
constexpr float kTopScore = 2147483648.f;
__device__ __forceinline__ float divisor(float m, float l) {
  return fabsf(m) < kTopScore ? 1.f / l : __int_as_float(0x7FC00000);
}
static_assert(kKeys % 16 == 0 && kCodes % 1024 == 0, "16-token groups, whole swizzle atoms");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// One lane of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct Ctx {
  const ChunkArgs& a;
  volatile uint32_t* stop;  // the site of a wait that ran out
  uint32_t tries;
};
// Bounded wait by a whole warp, whose lanes go on or give up together.  Every
// wait is for another warp of the block, so thousandths of a second at most;
// a failed try sleeps for microseconds, so the limit is a number of tries.
// Where one runs out the block stops, and says so at its end.  (The code is
// kept this short on purpose: the roles' loops together have to stay in the
// instruction cache, and there are some thirty waits.)
__device__ __forceinline__ bool wait(const Ctx& c, uint64_t* bar, uint32_t parity, uint32_t site) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xFFFFFFFFu, ok)) {
#pragma unroll 1
    for (uint32_t n = c.tries; !(ok = mbar_try_wait(bar, parity)); --n) {
      if (n == 0) *c.stop = site;
      if (*c.stop != 0u) break;
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
  }
  return ok;
}
// A warp's arrival, after all its lanes' writes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// A position in a ring of n stages.
template <int n>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == n) slot = 0, phase ^= 1u;
  }
};

// Tokens of an item whose values are not finite and which only some rows see
// (noted by the convert warps).
constexpr uint32_t kPlainScale = 134u;  // the largest scale byte s with 2^(s - 7) a bf16
struct HiddenNan {
  uint32_t any;
  uint32_t bits[2][8];  // tokens from the tile's first on; from the first behind those that all rows see
};

// Four codes times m (a bf16 power of two, twice).  A code s eeee mmm moved to
// s 0000eeee mmm0000 is the bf16 2^-120 times its value (subnormal codes
// included), which m takes back.  Within four codes the order is 0, 2, 1, 3: the
// outputs' columns are put back at the end.
__device__ __forceinline__ uint2 widen4(uint32_t w, uint32_t m) {
  const uint32_t even = ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u);
  const uint32_t odd = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
  return make_uint2(mul_bf16x2(even, m), mul_bf16x2(odd, m));
}
// Of four codes, bits 7, 15, 23, 31 say whether one is NaN (all bits but the sign
// set): adding one changes the bit above.  A negative NaN carries into the next
// code, which may be taken for NaN then (448 is); nan_bits_exact leaves the signs
// out.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w + 0x01010101u) ^ w; }
__device__ __forceinline__ uint32_t nan_bits_exact(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }
constexpr uint32_t kNanBits = 0x80808080u;

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---------------------------------------------------------------- load warps
// One of them copies K's key tiles into its ring, with the 128-byte swizzle that
// the products read, the other V's (with the halves of odd rows exchanged, for
// the warps that widen it), and their scales: K's in the order that tcgen05.cp
// wants, V's token by token.  A page holds whole groups
// of 16 tokens, 2 KB of codes: with 16-byte asynchronous copies (four
// instructions of a warp a group) a tile takes its warp a third of the cycles
// that a bulk or tensor copy a group takes, whose issue is about 100 cycles each.
// Four tiles' groups are looked up at a time, one a lane, and the next four's
// pages fetched meanwhile.
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The thread's arrival on `bar` when its copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
struct Loader {
  bool v;
  int stages;
  uint8_t *codes, *sf;
  const uint8_t* scales;
  uint64_t *full, *empty;
  int slot = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ bool item(const Ctx& c, const Item& w, int lane) {
    constexpr int kGroups = kKeys / 16, kBatch = 4;  // groups of a tile, tiles of a batch
    const ChunkArgs& a = c.a;
    const int t0 = w.t0, t1 = w.t1, lo = w.lo, hi = w.hi, hk = w.hk, mask = (1 << a.log2P) - 1;
    const int32_t* table = a.table + static_cast<long long>(w.b) * a.max_pages;
    auto page = [&](int tok) { return __ldg(table + (min(max(tok, lo), hi - 1) >> a.log2P)); };
    int tok = 16 * (t0 * kGroups + lane);  // the lane's group
    int pid = page(tok);
    const int part = lane >> 2, in = 4 * (lane & 3);  // the lane's four tokens among a tile's scales
    // a lane's 16 bytes of four rows: where they go in the first four, in the second
    // (V: the halves of odd rows exchanged)
    const int r4 = lane >> 3;
    const uint32_t at0 = r4 * kD + (((lane & 7) ^ (v ? 4 * (r4 & 1) : r4)) << 4), at1 = v ? at0 : at0 ^ 64u;
    const uint8_t* src = v ? a.vc : a.kc;
    const uint32_t sdst = v ? 16u * lane : ((4u * lane) & 31u) * 16u + ((4u * lane) >> 5) * 4u;
#pragma unroll 1
    for (int k = t0; k < t1; k += kBatch) {
      if (pid < 0 || pid >= a.num_pages) {  // reported, and page 0 read instead
        atomicCAS(a.status, 0u, (1u << 24) | (2u << 16) | (static_cast<uint32_t>(w.b) & 0xFFFFu));
        pid = 0;
      }
      // first row of the group (below 2^31), -1 when no row of the queries sees it
      const bool seen = lane < kGroups * kBatch && tok < hi && tok + 16 > lo;
      const int row = seen ? ((pid * a.Hkv + hk) << a.log2P) + (tok & mask) : -1;
      tok += 16 * kGroups * kBatch;
      pid = page(tok);
#pragma unroll 1
      for (int i = 0; i < kBatch && k + i < t1; ++i) {
        const int srow = __shfl_sync(0xFFFFFFFFu, row, min(kGroups * i + part, 31));
        uint64_t* bar = full + slot;
        if (!wait(c, empty + slot, phase ^ 1u, 3u)) return false;
        fence_proxy_async_shared();
        const uint32_t to = smem_u32(codes) + slot * kCodes;
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          const int grow = __shfl_sync(0xFFFFFFFFu, row, kGroups * i + g);
          if (grow >= 0) {
            const uint8_t* s = src + static_cast<size_t>(grow) * kD + 16 * lane;
            const uint32_t d = to + g * 16 * kD;
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_async16(d + 4 * kD * j + (j & 1 ? at1 : at0), s + 4 * kD * j);
          }
        }
        if (part < kGroups && srow >= 0) {
          const uint8_t* s = scales + static_cast<size_t>(srow + in) * (kD / 32);
          const uint32_t d = smem_u32(sf + slot * kScales) + sdst;
          if (v) {
            copy_async16(d, s);
          } else {  // token 4 lane + i at row % 32 times 16 bytes, row / 32 times 4
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_async4(d + 16 * j, s + 4 * j);
          }
        }
        copy_async_arrive(bar);
        if (++slot == stages) slot = 0, phase ^= 1u;
      }
    }
    return true;
  }
};

// The role of a load warp (v: the one for V); the other one walks the plan.
template <int NK, int NV, class Ctl>
__device__ __forceinline__ void load_items(const Ctx& c, Ctl* ctl, uint8_t* k, uint8_t* raw, uint8_t* sfk, uint8_t* sv,
                                           int qs, int rs, bool v, int lane) {
  const ChunkArgs& a = c.a;
  Loader ld;
  ld.v = v;
  ld.stages = ld.v ? NV : NK;
  ld.codes = v ? raw : k, ld.sf = v ? sv : sfk;
  ld.scales = ld.v ? a.vs : a.ks;
  ld.full = ld.v ? ctl->r_full : ctl->k_full, ld.empty = ld.v ? ctl->r_empty : ctl->k_empty;
  chunk::Walk walk;
  if (!ld.v) walk.init(a, ctl->ranges, blockIdx.x, qs, rs, lane);
  Ring<2> it;
#pragma unroll 1
  for (;; it.step()) {
    Item& w = ctl->item[it.slot];
    if (!ld.v) {
      Item next;
      if (!walk.next(a, lane, next)) {
        next.t0 = next.t1 = 0;
      } else {  // its queries on their way to L2
        for (int r = lane; r < next.rows; r += 32) {
          const int rr = next.r0 + r, tok = rr / a.G;
          const uint16_t* q = a.q + static_cast<long long>(next.c0 + tok) * a.ldq + (next.hk * a.G + rr - tok * a.G) * kD;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
        }
      }
      if (!wait(c, &ctl->it_empty[it.slot], it.phase ^ 1u, 2u)) break;
      if (lane == 0) w = next;
      if (lane < static_cast<int>(sizeof(HiddenNan) / 4)) reinterpret_cast<uint32_t*>(&ctl->hidden[it.slot])[lane] = 0u;
      __syncwarp();
      mbar_arrive(&ctl->it_full[it.slot]);
    } else if (!wait(c, &ctl->it_full[it.slot], it.phase, 4u)) {
      break;
    }
    if (w.t0 == w.t1 || !ld.item(c, w, lane)) break;
    if (ld.v) warp_arrive(&ctl->it_empty[it.slot], lane);
  }
  // the thread's copies have landed when the block ends, whatever the reason
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- the end
// All threads, after their roles.  Where a wait ran out, the products that the two
// product warps have issued (one lane of each, always the same) end before tensor
// memory is given back; a role may give up long after the product warps have
// left, so this is decided here and not by them.
template <class Ctl>
__device__ __forceinline__ void finish(const ChunkArgs& a, Ctl* ctl, int product_warp, int t) {
  __syncthreads();
  if (ctl->stop == 0u) return;
  const int m = (t >> 5) - product_warp;
  if (m == 0 || m == 1) {
    if (elect_one()) tc_commit(&ctl->fin[m]);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(&ctl->fin[m], 0) && globaltimer_ns() - t0 < 20000000ull) {
    }
    __syncwarp();
  }
  if (t == 0)  // FSOPS_ERR_TIMEOUT
    atomicCAS(a.status, 0u, (5u << 24) | (ctl->stop << 16) | (blockIdx.x & 0xFFFFu));
  __syncthreads();
}

// ---------------------------------------------------------------- values that are not finite
// The second product multiplies hidden places too, by a probability of zero,
// and zero times NaN is NaN.  So what is not finite stands in V's operand only
// at tokens that every row of the query tile sees; at the others the operand
// gets zeros, the token is noted, and at the item's end the rows that see
// it become NaN.  All of it is off the path of finite values.
// The tokens from .. upto - 1 that row r of the tile sees.
__device__ __forceinline__ void row_sees(const ChunkArgs& a, const Item& w, int r, int& from, int& upto) {
  upto = w.len - w.n + 1 + (w.r0 + r) / a.G;
  from = a.window > 0 ? max(0, upto - a.window) : 0;
}
// A row's sum, NaN where the row sees a noted token.
__device__ __noinline__ float sum_or_nan(const ChunkArgs& a, const Item& w, const HiddenNan& hn, int row, float sum) {
  int from, upto, all_from, all_upto, none;
  row_sees(a, w, min(row, w.rows - 1), from, upto);
  row_sees(a, w, w.rows - 1, all_from, none);
  row_sees(a, w, 0, none, all_upto);
#pragma unroll 1
  for (int i = 0; i < 512; ++i) {
    const int tok = (i < 256 ? w.lo : all_upto) + (i & 255);
    const bool noted = (hn.bits[i >> 8][(i & 255) >> 5] >> (i & 31) & 1u) != 0u;
    if (noted && tok >= from && tok < upto) sum = __int_as_float(0x7FC00000);
  }
  return sum;
}
// A thread's share of a V tile (16 codes of every 16th token from tok on, see
// convert_tile) once more, with what convert16 leaves out: scales from 2^8 on and
// what is not finite.
template <int kPasses>
__device__ __noinline__ void convert_rest(const ChunkArgs& a, const Item& w, HiddenNan& hn, const uint8_t* raw,
                                          const uint8_t* sc, uint8_t* row, int first, int tok) {
  int all_from, all_upto, none;
  row_sees(a, w, w.rows - 1, all_from, none);
  row_sees(a, w, 0, none, all_upto);
#pragma unroll 1
  for (int i = 0; i < kPasses; ++i, tok += 16, raw += 16 * kD, sc += 64, row += 16 * 128) {
    const uint32_t s = *sc;
    if (tok < w.lo || tok >= w.hi) continue;
    bool bad = false;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = reinterpret_cast<const uint32_t*>(raw)[k];
      uint2 p = widen4(x, (min(s, kPlainScale) + 120u) * 0x00800080u);  // 2^(s - 127 + 120)
      if (s > kPlainScale) {  // the rest of it
        const uint32_t m = ((s - kPlainScale + 127u) << 7) * 0x10001u;
        p = make_uint2(mul_bf16x2(p.x, m), mul_bf16x2(p.y, m));
      }
      const uint32_t n = s == 255u ? kNanBits : nan_bits_exact(x);
      p.x |= (n & 0x80u ? 0x7FFFu : 0u) | (n & 0x800000u ? 0x7FFF0000u : 0u);
      p.y |= (n & 0x8000u ? 0x7FFFu : 0u) | (n & 0x80000000u ? 0x7FFF0000u : 0u);
#pragma unroll
      for (int h = 0; h < 32; h += 16) bad |= (p.x >> h & 0x7F80u) == 0x7F80u || (p.y >> h & 0x7F80u) == 0x7F80u;
      *reinterpret_cast<uint2*>(row + (k < 2 ? first : first ^ 16) + 8 * (k & 1)) = p;
    }
    if (!bad || (tok >= all_from && tok < all_upto)) continue;
    *reinterpret_cast<uint4*>(row + first) = *reinterpret_cast<uint4*>(row + (first ^ 16)) = make_uint4(0u, 0u, 0u, 0u);
    const int at = tok < all_from ? tok - w.lo : tok - all_upto;  // below 256: a tile's rows are as many tokens at most
    atomicOr(&hn.bits[tok < all_from ? 0 : 1][at >> 5], 1u << (at & 31));
    hn.any = 1u;
  }
}

// ---------------------------------------------------------------- convert warps
// V's codes of tokens from tok0 to a bf16 tile; tokens outside [lo, hi) become
// zeros whatever the ring holds there.  A thread has 16 codes of every 16th
// token: eight lanes four pieces of two tokens each, which keeps their 16-byte
// stores (and, with the ring's halves exchanged in every other row, their
// loads) apart in the banks.  nan: nan_bits of all codes, top: the largest scale.
// (Measured, the chunk of 2048 tokens against 16 k / five drafted tokens for each
// of 64 sequences: 410 / 137 us; with NaN found by maxima of magnitudes and the
// scales' second product here 442 / 144.)
__device__ __forceinline__ void convert16(const uint8_t* raw, uint32_t s, uint8_t* row, int first, bool on, uint32_t& nan,
                                          uint32_t& top) {
  const uint4 x = *reinterpret_cast<const uint4*>(raw);
  const uint32_t m = on ? s * 0x00800080u + 120u * 0x00800080u : 0u;  // 2^(s - 127 + 120), twice
  const uint2 p0 = widen4(x.x, m), p1 = widen4(x.y, m), p2 = widen4(x.z, m), p3 = widen4(x.w, m);
  *reinterpret_cast<uint4*>(row + first) = make_uint4(p0.x, p0.y, p1.x, p1.y);
  *reinterpret_cast<uint4*>(row + (first ^ 16)) = make_uint4(p2.x, p2.y, p3.x, p3.y);
  nan |= nan_bits(x.x), nan |= nan_bits(x.y), nan |= nan_bits(x.z), nan |= nan_bits(x.w);
  top = max(top, s);
}
__device__ __forceinline__ void convert_tile(const ChunkArgs& a, const Item& w, HiddenNan& hn, const uint8_t* raw,
                                             const uint8_t* sc, uint8_t* out, int tok0, int lo, int hi, int t) {
  static_assert(kConvWarps == 4, "16 tokens a pass");
  constexpr int kPasses = kKeys / 16;
  const int half = (t >> 3) & 1, piece = 4 * half + (t & 3), r0 = 2 * (t >> 4) + ((t >> 2) & 1);
  const int first = ((2 * (t & 3)) ^ (r0 & 7)) << 4;
  out += half * kHalf + r0 * 128;
  raw += r0 * kD + 16 * (piece ^ (4 * (r0 & 1))), sc += 4 * r0 + (piece >> 1);
  uint32_t nan = 0u, top = 0u;
  if (tok0 >= lo && tok0 + kKeys <= hi) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) convert16(raw + i * 16 * kD, sc[i * 64], out + i * 16 * 128, first, true, nan, top);
  } else {
#pragma unroll 1
    for (int i = 0; i < kPasses; ++i) {
      const int tok = tok0 + r0 + i * 16;
      const bool on = tok >= lo && tok < hi;
      uint32_t n = 0u, s = 0u;
      convert16(raw + i * 16 * kD, sc[i * 64], out + i * 16 * 128, first, on, n, s);
      if (on) nan |= n, top = max(top, s);
    }
  }
  if ((nan & kNanBits) != 0u || top > kPlainScale)
    convert_rest<kPasses>(a, w, hn, raw, sc, out, first, tok0 + r0);
}

// The role of the convert warps, thread ct of them.
template <int NV, int kSlots, class Ctl>
__device__ __forceinline__ void convert_items(const Ctx& c, Ctl* ctl, const uint8_t* raw, const uint8_t* sv, uint8_t* v,
                                              int ct, int lane) {
  Ring<2> it;
  Ring<NV> ring;
  Ring<kSlots> vr;
  for (bool ok = true; ok; it.step()) {
    if (!wait(c, &ctl->it_full[it.slot], it.phase, 4u)) break;
    const int t0 = ctl->item[it.slot].t0, t1 = ctl->item[it.slot].t1, lo = ctl->item[it.slot].lo,
              hi = ctl->item[it.slot].hi;
    warp_arrive(&ctl->it_empty[it.slot], lane);
    if (t0 == t1) break;
    for (int k = t0; k < t1; ++k) {
      ok = wait(c, &ctl->r_full[ring.slot], ring.phase, 3u) && wait(c, &ctl->v_empty[vr.slot], vr.phase ^ 1u, 6u);
      if (!ok) break;
      // (the item stays until the softmax warps give it back, after its last product)
      convert_tile(c.a, ctl->item[it.slot], ctl->hidden[it.slot], raw + ring.slot * kCodes, sv + ring.slot * kScales,
                   v + vr.slot * kOperand, k * kKeys, lo, hi, ct);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->v_full[vr.slot]);
        mbar_arrive(&ctl->r_empty[ring.slot]);
      }
      ring.step();
      vr.step();
    }
  }
}

// ---------------------------------------------------------------- queries
// Where an operand keeps row r's scales: tiles of 128 rows, as tcgen05.cp wants them.
__device__ __forceinline__ int scale_at(int r) { return (r >> 7) * static_cast<int>(kScales) + (r & 31) * 16 + ((r >> 5) & 3) * 4; }
// 8 dimensions (piece c of 16) of row r of a query operand as two E4M3 terms
// with their scales, the second `lo` rows further on.  Four lanes hold a block
// of 32 dimensions.
__device__ __forceinline__ void store_query(uint4 x, uint32_t flip, uint8_t* codes, uint8_t* sf, int r, int lo, int c) {
  const uint32_t u[4] = {x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip};
  uint32_t am = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) am = __vmaxu2(am, u[k] & 0x7FFF7FFFu);
  am = max(am & 0xFFFFu, am >> 16);
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  // the largest below 2^8 in units of the first scale: nothing saturates, and
  // the rest is at most 2^3 of them, four bits again
  const int e = static_cast<int>(am >> 7);
  const uint32_t s0 = static_cast<uint32_t>(max(e - 7, 0)), s1 = static_cast<uint32_t>(max(e - 11, 0));
  const float i0 = inv_scale_from_ue8m0(s0), i1 = inv_scale_from_ue8m0(s1);
  const float back = s0 != 0 ? __uint_as_float(s0 << 23) : __uint_as_float(0x00400000u);
  uint32_t h[2], l[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float v0 = bf16_lo(u[2 * k]), v1 = bf16_hi(u[2 * k]), v2 = bf16_lo(u[2 * k + 1]), v3 = bf16_hi(u[2 * k + 1]);
    h[k] = e4m3x4_code(v0 * i0, v1 * i0, v2 * i0, v3 * i0);
    const __nv_fp8x4_e4m3* hc = reinterpret_cast<const __nv_fp8x4_e4m3*>(&h[k]);
    const float4 hv = static_cast<float4>(*hc);
    if (e == 255) h[k] = 0x7F7F7F7Fu;  // not finite: NaN scores, not saturated ones
    l[k] = e4m3x4_code(fmaf(-hv.x, back, v0) * i1, fmaf(-hv.y, back, v1) * i1, fmaf(-hv.z, back, v2) * i1,
                       fmaf(-hv.w, back, v3) * i1);
  }
  uint8_t* d = codes + r * 128 + ((((c >> 1) ^ (r & 7)) << 4) | ((c & 1) << 3));
  *reinterpret_cast<uint2*>(d) = make_uint2(h[0], h[1]);
  *reinterpret_cast<uint2*>(d + lo * 128) = make_uint2(l[0], l[1]);
  if ((c & 3) == 0) {
    sf[scale_at(r) + (c >> 2)] = static_cast<uint8_t>(s0);
    sf[scale_at(r + lo) + (c >> 2)] = static_cast<uint8_t>(s1);
  }
}

}  // namespace

}  // namespace fsops
