// mx_sample.cu -- tokens from logits: temperature, top-k, top-p, min-p, and a
// given random number a row.
//
//   w[i] = exp((x[i] - max x) / T).  In the order of falling x, ties by rising
//   index: the first k tokens; of those the ones with less than p of the k's mass
//   ahead of them; of those the ones with w[i] >= min_p.  The token is the first
//   one, by index, where the mass of the kept tokens up to it is above u times
//   all of it.
//
// A token is a whole number: it is the same whatever the order of sums only if
// the sums are.  So weights are whole numbers, units of 2^-45 of the largest, and
// added as such, and each is good to a unit and 2^-37 of itself (the median is off by
// one unit, the worst of the largest by some 160): u falls between a border here and
// the same border in 64-bit floating point about once in 10^10 / V rows.  (Weights that
// are alike are rounded alike, so V of a few units each can move a border by V units.)
// (With weights good to 2^-22, as of a hardware exponential, every other row of a
// flat distribution over 150000 tokens would be in doubt.)
//
// The weight.  With c = log2(e) / T as two fp32 numbers, x c = i / 64 + r, |r| <
// 2^-6.9: the product's rounding is what an fma gives back, the difference to the
// nearest 64th is exact, and r is kept in two parts.  2^(x c) is a table entry for
// i mod 64 (61 bits after the point), times 1 + f with f = 2^r - 1 from the series
// in units of 2^-38, shifted by i / 64.  The common factor 2^(max c) is taken out
// to the nearest 64th, which is all it needs: the same factor in every weight
// changes nothing.
// Sums over many tokens are taken in fp32 first, with a bound of their error (2^-20
// of the mass): where u, or top-p's cut, lies further from the borders than that,
// the answer is the exact one's; else the sum is taken again in exact weights, at
// five times the instructions.
//
// A cluster of up to 8 blocks has a row, each block a part of it in shared memory,
// read from HBM once; a thread has a run of consecutive vectors.  Then, over those:
//   1 the largest logit;
//   2 top-k of up to 100: each block names a logit that a C-th of k of its elements
//     are not below, and what lies below the lowest of these cannot be kept.  What is
//     left, some hundred tokens, goes to the first block, which does the rest alone;
//   3 (top-k, top-p) counts by distance from the largest, 512 bins of 1 / 16 of a
//     power of two each; they give top-k's bin and, by the weights at their edges,
//     the bins between which top-p's cut lies;
//   4 (top-p) the mass of all, of what is above those bins, and of a 512th each of
//     the logits between;
//   5 the cut inside its bin: of up to 256 tokens by adding up what is ahead of each
//     (by the first block), of more by counts (and masses) of a 512th each of the
//     float codes that occur there, again until they are few, or a single value
//     (equals are kept by index);
//   6 the kept tokens' mass, thread by thread in the order of the indices, and the
//     place where u falls.
// What blocks tell each other they write into each other's shared memory before they
// meet, so that nobody waits for a remote load.
//
// What bounds it: phases.  A row alone is 4 (top-k of few) to 25 of them, each with
// a barrier of the block or the cluster and some hundred instructions that are
// fetched once; many rows run two blocks an SM, which issue half of the time.  (Two
// blocks leave a thread 64 registers; the clusters' kernel spills 52 to 76 bytes, the
// rows' none.)
// Measured (us): one row of 150001 bf16 logits, top-k 50 and top-p 10.6, unfiltered
// 16, top-p alone 32 (a peaked row) to 42 (a flat one); 1024 x 32003 bf16 unfiltered
// 48 (1.4 TB/s); 256 x 128000 fp32 with a mixture of all filters 148, with top-k 50
// throughout 54, unfiltered 62, top-p alone 260 to 310.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "mx_sample.h"

namespace fsops {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 512;
constexpr uint32_t kFinish = kThreads / 2;  // tokens around a cut that are put in order by themselves
// top-k up to which lists are made, their length (of a block).  Measured, lists
// against bins (us): 32 x 128000 logits with top-k 50 16 to 32, with 100 24 to 35.
constexpr int kListK = 100, kList = 192;
constexpr int kMaxCluster = 8;
constexpr float kInf = __builtin_huge_valf();

// 2^(j / 64) in units of 2^-61
__device__ const u64 kPowers[64] = {
    0x2000000000000000ULL, 0x2059347CEF00C1DDULL, 0x20B361A62B0AE876ULL, 0x210E8A30EB379012ULL,
    0x216AB0D9F3121EC5ULL, 0x21C7D865A7A34404ULL, 0x222603A024B6A14AULL, 0x2285355D525BBF67ULL,
    0x22E57078FAA2F5BAULL, 0x2346B7D6DF96EA79ULL, 0x23A90E62D17354F0ULL, 0x240C7710C519AC77ULL,
    0x2470F4DCEAC470CEULL, 0x24D68ACBC4F9BA4BULL, 0x253D3BEA3FBDC258ULL, 0x25A50B4DC8061680ULL,
    0x260DFC14636E2A5CULL, 0x26781164C82DFE99ULL, 0x26E34E6E7553954EULL, 0x274FB669CB3FEDD4ULL,
    0x27BD4C982468446BULL, 0x282C1443EE5C53F1ULL, 0x289C10C0C3125A06ULL, 0x290D456B8279A028ULL,
    0x297FB5AA6C544E3BULL, 0x29F364ED3A594D5AULL, 0x2A6856AD3A9F03BEULL, 0x2ADE8E6D6A4FB4CEULL,
    0x2B560FBA90A852B2ULL, 0x2BCEDE2B5A4290DDULL, 0x2C48FD6074AB0964ULL, 0x2CC47104AA444922ULL,
    0x2D413CCCFE779921ULL, 0x2DBF6478CA345DE4ULL, 0x2E3EEBD1D8BEE7BAULL, 0x2EBFD6AC84CF917FULL,
    0x2F4228E7D6030DB0ULL, 0x2FC5E66D9E9CC421ULL, 0x304B1332999C2516ULL, 0x30D1B3368925D902ULL,
    0x3159CA845541B6B7ULL, 0x31E35D322AEE6C57ULL, 0x326E6F619B8BC9E9ULL, 0x32FB053FBC9C9F17ULL,
    0x3389230547E12039ULL, 0x3418CCF6BBCAC965ULL, 0x34AA07647C4AB917ULL, 0x353CD6AAF3FB7E88ULL,
    0x35D13F32B5A75ABDULL, 0x366745709E2BF5EDULL, 0x36FEEDE5F6BC8DD5ULL, 0x37983D209783A449ULL,
    0x383337BB0AA53844ULL, 0x38CFE25CAFA29694ULL, 0x396E41B9DF20D22AULL, 0x3A0E5A940F12F71AULL,
    0x3AB031B9F7490E4CULL, 0x3B53CC07B6650AE1ULL, 0x3BF92E66F736BD73ULL, 0x3CA05DCF167FEC4EULL,
    0x3D495F454921B30BULL, 0x3DF437DCC2B44EEEULL, 0x3EA0ECB6DC8A80CFULL, 0x3F4F83033D21B05DULL,
};

// ---------------------------------------------------------------- weights
// (All of it in fp32 and whole numbers: an fp64 instruction takes an SM some 30
// cycles a warp.)
struct Scale {
  float ch, cl;  // log2(e) / T
  int top;       // 64 times the largest logit's power of two
  float low;     // logits below it weigh nothing
  int wide;      // powers that the table's way does not take (is_wide)
  float max;
  double c;      // log2(e) / T, where wide
};
// Powers too large for fp32 to tell 2^-38 of one; and from temperatures of 2^99 on, where the
// parts of log2(e) / T come near fp32's last bit, 2^-149, logits beyond kFar (up to there x c is
// good to 2^-40; below that temperature it is whatever they are, as those that weigh anything
// are at most 2^11 / c).  With logits as models give them such a temperature, infinity for
// instance, is not wide: 256 x 128000 of them take 1510 us in fp64, 150 as fp32 and the table.
constexpr float kHot = 0x1p99f, kFar = 0x1p109f;
__device__ __forceinline__ bool is_wide(float max_power, float ch, bool far) { return !(fabsf(max_power) < 2000.f && ch < 1e30f) || far; }
__device__ __noinline__ double powers_per(float T) { return 0x1.71547652b82fep+0 / static_cast<double>(T); }
constexpr float kMagic = 12582912.f;  // 3 * 2^22: a float near it has its last bit at one
constexpr int kUnit = 45;

// The last bit is always set: what is cut off is half a unit, as often above as
// below, so that sums of many small weights are not too small.
__device__ __noinline__ u64 weight_wide(float x, const Scale& s) {
  return static_cast<u64>(__double2ll_rd(exp2((static_cast<double>(x) - static_cast<double>(s.max)) * s.c + kUnit))) | 1ull;
}
__device__ __forceinline__ u64 weight_near(float x, float ch, float cl, int top, const u64* powers) {
  const float p = x * ch;
  const float t = fmaf(p, 64.f, kMagic);
  const int g = __float_as_int(t) - (__float_as_int(kMagic) + top);
  const float r0 = fmaf(t - kMagic, -0.015625f, p);                // exact
  const float rl = fmaf(x, cl, fmaf(x, ch, -p));
  const float r = r0 + rl, re = rl - (r - r0);
  // 2^r - 1 in units of 2^-38: q + tail
  constexpr float kL = 0x1.62e43p+37f, kLlo = -0x1.05c61p+9f;      // ln 2
  const float q = r * kL;
  float tail = fmaf(re, kL, fmaf(r, kLlo, fmaf(r, kL, -q)));
  const float series = fmaf(r, fmaf(r, fmaf(r, 0x1.5d87fep+28f, 0x1.3b2ab6p+31f), 0x1.c6b08ep+33f), 0x1.ebfbep+35f);
  tail = fmaf(r * r, series, tail);                                // below 2^22
  const int f = __float2int_rn(q) + (__float_as_int(tail + kMagic) - __float_as_int(kMagic));
  const u64 e = powers[g & 63];
  const long long more = static_cast<long long>(static_cast<int>(e >> 31)) * f;  // units of 2^-68
  const u64 w = e + static_cast<u64>(more >> 7);
  return (w >> (min(61 - kUnit - (g >> 6), 63) & 63)) | 1ull;
}
// The same of two logits, step by step.
__device__ __forceinline__ void weight_near2(float2 x, float2 ch, float2 cl, int top, const u64* powers, u64& w0, u64& w1) {
  auto both = [](float v) { return make_float2(v, v); };
  auto less = [](float2 v) { return make_float2(-v.x, -v.y); };
  constexpr float kL = 0x1.62e43p+37f, kLlo = -0x1.05c61p+9f;
  const float2 p = __fmul2_rn(x, ch), t = __ffma2_rn(p, both(64.f), both(kMagic));
  const float2 r0 = __ffma2_rn(__fadd2_rn(t, both(-kMagic)), both(-0.015625f), p);
  const float2 rl = __ffma2_rn(x, cl, __ffma2_rn(x, ch, less(p)));
  const float2 r = __fadd2_rn(r0, rl), re = __fadd2_rn(rl, less(__fadd2_rn(r, less(r0))));
  const float2 q = __fmul2_rn(r, both(kL));
  float2 tail = __ffma2_rn(re, both(kL), __ffma2_rn(r, both(kLlo), __ffma2_rn(r, both(kL), less(q))));
  float2 series = __ffma2_rn(r, both(0x1.5d87fep+28f), both(0x1.3b2ab6p+31f));
  series = __ffma2_rn(r, __ffma2_rn(r, series, both(0x1.c6b08ep+33f)), both(0x1.ebfbep+35f));
  tail = __ffma2_rn(__fmul2_rn(r, r), series, tail);
  const float2 m = __fadd2_rn(tail, both(kMagic));
  auto one = [&](float tt, float qq, float mm) {
    const int g = __float_as_int(tt) - (__float_as_int(kMagic) + top);
    const int f = __float2int_rn(qq) + (__float_as_int(mm) - __float_as_int(kMagic));
    const u64 e = powers[g & 63];
    const long long more = static_cast<long long>(static_cast<int>(e >> 31)) * f;
    return ((e + static_cast<u64>(more >> 7)) >> (min(61 - kUnit - (g >> 6), 63) & 63)) | 1ull;
  };
  w0 = one(t.x, q.x, m.x), w1 = one(t.y, q.y, m.y);
}
// Of any logit; the few that a search or a cut looks at.
__device__ __noinline__ u64 weight(float x, const Scale& s, const u64* powers) {
  if (x < s.low) return 0ull;
  return s.wide ? weight_wide(x, s) : weight_near(x, s.ch, s.cl, s.top, powers);
}

// The same in fp32, for logits of `low` and more of rows that are not wide: all of
// them together off by 2^-21 of the row's mass at most.  (The fraction f of the
// power, which the fma finds from the whole product, and the other part of c are
// each rounded by 2^-26 at most, the exponential is good to 2^-22, and a vector is
// added up by pairs, 3 * 2^-24.  What moves all weights alike moves nothing, so the
// unit is the whole power of two above the largest one.)
__device__ __forceinline__ float rough(float x, float ch, float cl, float unit) {
  const float t = fmaf(x, ch, unit);  // kMagic less that power: whole numbers
  const float f = fmaf(x, cl, fmaf(x, ch, unit - t));
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(f));
  return __uint_as_float(__float_as_uint(w) + (__float_as_uint(t) << 23));
}
// The same of two logits; one below `low` counts as `low`, whose 2^-46 of the
// largest weight nothing feels that a sum of fp32 weights decides (NaN too).
__device__ __forceinline__ float2 rough2(float2 x, float2 ch, float2 cl, float2 unit, float low) {
  x.x = fmaxf(x.x, low), x.y = fmaxf(x.y, low);
  const float2 t = __ffma2_rn(x, ch, unit);
  const float2 f = __ffma2_rn(x, cl, __ffma2_rn(x, ch, __fadd2_rn(unit, make_float2(-t.x, -t.y))));
  float2 w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.x) : "f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.y) : "f"(f.y));
  w.x = __uint_as_float(__float_as_uint(w.x) + (__float_as_uint(t.x) << 23));
  w.y = __uint_as_float(__float_as_uint(w.y) + (__float_as_uint(t.y) << 23));
  return w;
}
constexpr int kRough = 21;
constexpr float kOne = static_cast<float>(1ull << kUnit);
// 2^d for a whole d, 0 for ones below fp32's, 1 above 0.
__device__ __forceinline__ float power_of_two(float d) {
  return d < -126.f ? 0.f : __int_as_float((127 + static_cast<int>(fminf(d, 0.f))) << 23);
}
// A sum of them: vectors by pairs, the vectors' sums with what their additions lose.
struct RoughSum {
  float s = 0.f, lost = 0.f;
  template <int n>
  __device__ __forceinline__ void add(const float (&w)[n]) {
    float v[n];
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = w[i];
#pragma unroll
    for (int d = n / 2; d; d >>= 1)
#pragma unroll
      for (int i = 0; i < d; ++i) v[i] += v[i + d];
    add(v[0]);
  }
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    lost += (s - (t - b)) + (v - b);
    s = t;
  }
  __device__ __forceinline__ u64 units() const {
    return __float2ull_rn(s * kOne) + static_cast<u64>(__float2ll_rn(lost * kOne));
  }
};

// ---------------------------------------------------------------- order
// Whole numbers in the order of the floats (-0 as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// Bin of a logit, the nearest to its distance: grows as x falls.
__device__ __forceinline__ int bin_of(float x, float max, float per) {
  constexpr float kWhole = 8388608.f;  // 2^23
  return min(kBins - 1, __float_as_int(fmaf(max - x, per, kWhole)) - __float_as_int(kWhole));
}
constexpr float kMost = 3.402823466e38f;
// The smallest distance (of keys, from `top`) whose logit has a bin of b or more below `max`, one behind the lowest
// logit's if none has; every lane of a warp calls it.  Nearly always it is among the 32 next to where it would be
// without roundings.
__device__ __noinline__ uint32_t bin_start(int b, uint32_t top, float max, float per, int lane) {
  const uint32_t end = top - key_of(-kMost) + 1;
  auto there = [&](uint32_t at) { return at >= end || bin_of(fminf(of_key(top - min(at, end)), max), max, per) >= b; };
  const uint32_t near = min(top - min(key_of(fmaxf(max - (static_cast<float>(b) - 0.5f) / per, -kMost)), top), end), low = near > 15u ? near - 15u : 0u;
  unsigned yes = __ballot_sync(0xFFFFFFFFu, there(low + lane));
  if ((yes != 0u && !(yes & 1u)) || (yes & 1u && low == 0u)) return min(low + __ffs(static_cast<int>(yes)) - 1, end);
  uint32_t lo = 0, hi = end;
  while (lo < hi) {
    const uint32_t step = (hi - lo + 31) / 32, at = lo + static_cast<uint32_t>(lane) * step;
    yes = __ballot_sync(0xFFFFFFFFu, at >= hi || there(at));
    if (yes == 0u) {
      lo = lo + 31 * step + 1;
      continue;
    }
    const uint32_t first = __ffs(static_cast<int>(yes)) - 1;
    hi = min(hi, lo + first * step);
    if (first > 0) lo += (first - 1) * step + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- shared memory
struct Found {
  int bin;          // -1: none
  uint32_t before;  // count, mass before it
  uint32_t count;
  u64 mass_before, mass;
  int b1, b2;       // of the first counts: the bins between which top-p's cut lies
  int flat;         // fp32 sums would leave that cut in doubt
  uint32_t lo[2], hi[2];  // distances of the bin, and of b1 .. b2
};
// What is kept: logits of `least` and more, and the first `ties` (by index) of those that are `tie`.
struct Cut {
  float least, tie;
  uint32_t ties;
};

constexpr int kParts = 4;  // of a mass, 12 bits each and the rest, so that a row's sums stay in 32 bits
struct Ctl {
  u64 powers[64];
  uint32_t hist[2][1 + kParts][kBins];  // counts and masses: the block's, and (of the first block) the cluster's
  alignas(16) float list[kMaxCluster * kList];  // of the first block: what may be among the k largest, or at a cut
  uint32_t list_index[kMaxCluster * kList];
  u64 span[kWarps], red64[kWarps];
  uint32_t red32[kWarps];
  float redf[2][kWarps];
  Scale scale;
  int first[2];
  uint32_t nearest, farthest;
  // Written by the other blocks (as the first one's list, list_index and hist[1] are), each
  // before one meeting and read behind it; what is written again is not before another.
  float max[kMaxCluster], edge[kMaxCluster];  // once
  uint32_t index[kMaxCluster], ties[kMaxCluster], far[kMaxCluster];  // once
  uint32_t listed[kMaxCluster], from[kMaxCluster], to[kMaxCluster];  // each step of a search
  u64 mass[2][kMaxCluster];  // each pass for top-p's mass
  u64 all[kMaxCluster];      // the counts' (read before they are shared), each pass of the draw
  Found found;               // by the first block, when it has looked through the counts
  Cut cut;                   // by the first block, at the end of a search over a few
  uint32_t redo;             // set by the block itself before a meeting, cleared by the one that drew behind it, read behind the next
};

template <bool half>
struct Vec {
  static constexpr int n = half ? 8 : 4;
};
template <bool half>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[Vec<half>::n]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (half) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}
// Element i of a block's part.
template <bool half>
__device__ __forceinline__ float element(const uint4* data, int i) {
  if constexpr (half)
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(data)[i]) << 16);
  else
    return reinterpret_cast<const float*>(data)[i];
}
template <bool half>
__device__ __forceinline__ void set_element(void* data, int i, float x) {
  if constexpr (half)
    static_cast<uint16_t*>(data)[i] = static_cast<uint16_t>(__float_as_uint(x) >> 16);
  else
    static_cast<float*>(data)[i] = x;
}

template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Inclusive sum over the block.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* red, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  static_assert(kWarps == 16, "half a warp of sums");
  T sums = red[lane & 15];
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, sums, o, 16);
    if ((lane & 15) >= o) sums += x;
  }
  all = __shfl_sync(0xFFFFFFFFu, sums, 15);
  const T before = __shfl_sync(0xFFFFFFFFu, sums, (warp + 15) & 15);
  return warp > 0 ? v + before : v;
}

// p as a fraction of 2^64, rounded down; below 0 (and NaN) as 0, 1 and above as just below 1
__device__ __forceinline__ u64 fraction(float p) {
  if (!(p > 0.f)) return 0ull;
  if (p >= 1.f) return ~0ull;
  const uint32_t b = __float_as_uint(p);
  const int shift = static_cast<int>(b >> 23) - 86;  // of 24 bits, to 2^-64
  const u64 m = (b & 0x7FFFFFu) | 0x800000u;
  return shift >= 0 ? m << shift : shift > -24 ? m >> -shift : 0ull;
}

// A row's part, or its list.
template <bool half>
struct Row {
  Ctl* ctl;
  const uint4* data;
  cg::cluster_group cluster;
  int C, rank;  // blocks of the row, and which one this is
  int per;      // vectors of a thread: an odd number, so that the threads' loads lie in different banks
  int v0, v1;   // its vectors
  static constexpr int E = Vec<half>::n;

  __device__ __forceinline__ void spread(const uint4* from, int nvec) {
    data = from;
    per = ((nvec + kThreads - 1) / kThreads) | 1;
    v0 = min(static_cast<int>(threadIdx.x) * per, nvec);
    v1 = min(v0 + per, nvec);
  }
  __device__ __forceinline__ void meet() {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  }
  template <class T>
  __device__ __forceinline__ T* of(T* p, int r) {
    return C > 1 ? cluster.map_shared_rank(p, r) : p;
  }
  // (by threads below C) this block's value to block threadIdx.x
  template <class T>
  __device__ __forceinline__ void tell(T* slots, T value) {
    *of(slots + rank, static_cast<int>(threadIdx.x)) = value;
  }
  __device__ __forceinline__ float largest() {
    if constexpr (half) {
      __nv_bfloat162 m = __float2bfloat162_rn(-kInf);
      for (int v = v0; v < v1; ++v) {
        const uint4 w = data[v];
        const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(&w);
        m = __hmax2(m, __hmax2(__hmax2(q[0], q[1]), __hmax2(q[2], q[3])));
      }
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      float m = -kInf;
      for (int v = v0; v < v1; ++v) {
        float x[E];
        unpack<half>(data[v], x);
        m = fmaxf(fmaxf(m, fmaxf(x[0], x[1])), fmaxf(x[2], x[3]));
      }
      return m;
    }
  }
  // f of the elements from lo to hi
  template <class F>
  __device__ __forceinline__ void between(float lo, float hi, F f) {
#pragma unroll 1
    for (int v = v0; v < v1; ++v) {
      float x[E];
      unpack<half>(data[v], x);
      uint32_t in = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) in |= x[e] >= lo && x[e] <= hi ? 1u << e : 0u;
#pragma unroll 1
      for (; in != 0u; in &= in - 1u) {
        const int i = v * E + __ffs(static_cast<int>(in)) - 1;
        f(element<half>(data, i), i);
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void each(F f) {
    for (int v = v0; v < v1; ++v) {
      float x[E];
      unpack<half>(data[v], x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e]);
    }
  }
  template <class F>
  __device__ __forceinline__ void pairs(F f) {
    for (int v = v0; v < v1; ++v) {
      float x[E];
      unpack<half>(data[v], x);
#pragma unroll
      for (int e = 0; e < E; e += 2) f(x[e], x[e + 1]);
    }
  }
  __device__ __forceinline__ void clear(bool masses) {
    __syncthreads();  // (the last counts have been read)
    ctl->hist[0][0][threadIdx.x] = 0u;
    if (masses) {
#pragma unroll
      for (int p = 1; p <= kParts; ++p) ctl->hist[0][p][threadIdx.x] = 0u;
    }
    __syncthreads();
  }
  __device__ __forceinline__ void count(int b, u64 w, bool masses) {
    atomicAdd(&ctl->hist[0][0][b], 1u);
    if (masses) {
#pragma unroll
      for (int p = 0; p < kParts; ++p)
        atomicAdd(&ctl->hist[0][1 + p][b], p + 1 < kParts ? static_cast<uint32_t>(w >> (12 * p)) & 0xFFFu : static_cast<uint32_t>(w >> (12 * p)));
    }
  }
  // The blocks' counts (and masses) to the first one.
  __device__ __forceinline__ void combine(bool masses) {
    __syncthreads();
    if (C > 1) {
      const uint32_t n = ctl->hist[0][0][threadIdx.x];
      if (n != 0u) {
        Ctl* first = of(ctl, 0);
        atomicAdd(&first->hist[1][0][threadIdx.x], n);
        if (masses) {
#pragma unroll
          for (int p = 1; p <= kParts; ++p) {
            const uint32_t m = ctl->hist[0][p][threadIdx.x];
            if (m != 0u) atomicAdd(&first->hist[1][p][threadIdx.x], m);
          }
        }
      }
      meet();
    }
  }
  // (by the first block) the first bin up to which the count is `count` or the mass is `mass`; its counts back to zero
  __device__ __forceinline__ uint32_t find(bool masses, uint32_t count, u64 mass) {
    static_assert(kBins == kThreads, "a bin a thread");
    const int i = static_cast<int>(threadIdx.x);
    uint32_t(*h)[kBins] = ctl->hist[C > 1 ? 1 : 0];
    if (i == 0) ctl->found.bin = -1;
    const uint32_t n0 = h[0][i];
    uint32_t all;
    const uint32_t n = block_scan(n0, ctl->red32, all) - n0;
    u64 m0 = 0, m = 0;
    if (masses) {
#pragma unroll
      for (int p = 0; p < kParts; ++p) m0 += static_cast<u64>(h[1 + p][i]) << (12 * p);
      u64 sum;
      m = block_scan(m0, ctl->red64, sum) - m0;
    }
    if (masses ? m < mass && m + m0 >= mass : n < count && n + n0 >= count) {
      Found& f = ctl->found;
      f.bin = i;
      f.before = n, f.count = n0;
      f.mass_before = m, f.mass = m0;
    }
    h[0][i] = 0u;
    if (masses) {
#pragma unroll
      for (int p = 1; p <= kParts; ++p) h[p][i] = 0u;
    }
    __syncthreads();
    return n0;
  }
  // What the first block found, to all.
  __device__ __forceinline__ Found share() {
    if (C > 1) {
      if (rank == 0 && threadIdx.x > 0 && static_cast<int>(threadIdx.x) < C) *of(&ctl->found, static_cast<int>(threadIdx.x)) = ctl->found;
      meet();
    } else {
      __syncthreads();
    }
    return ctl->found;
  }
};

// A logit that k of the block's elements are not below (-kMost where there are too
// few): the k-th largest of the warps' largest where k is no more than the warps,
// else the lowest of the first `warps` warps' k / warps-th largest threads.
__device__ __forceinline__ float edge_of(Ctl* ctl, float own, int k, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = k <= kWarps ? 1 : warps > 0 ? (k + warps - 1) / warps : 33;
  uint32_t left = key_of(own), bound = 0u;
  if (each <= 32) {
#pragma unroll 1
    for (int i = 0; i < each; ++i) {
      bound = __reduce_max_sync(0xFFFFFFFFu, left);
      if (lane == __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, left == bound))) - 1) left = 0u;
    }
    if (k > kWarps && warp >= warps) bound = 0xFFFFFFFFu;
  }
  __syncthreads();
  if (lane == 0) ctl->red32[warp] = bound;
  if (threadIdx.x == 0) ctl->first[0] = 0;
  __syncthreads();
  bound = ctl->red32[lane & (kWarps - 1)];
  if (k <= kWarps) {
    int ahead = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t x = __shfl_sync(0xFFFFFFFFu, bound, w);
      ahead += x > bound || (x == bound && w < (lane & (kWarps - 1))) ? 1 : 0;
    }
    bound = __shfl_sync(0xFFFFFFFFu, bound, __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, ahead == k - 1))) - 1);
  } else {
    bound = __reduce_min_sync(0xFFFFFFFFu, bound);
  }
  return bound > key_of(-kMost) ? of_key(bound) : -kMost;
}

// ln of a token's share of the mass `whole`, of which the largest weight is `most`.
// (Half of each logit: a row may reach from the lowest fp32 to the largest.)
__device__ __forceinline__ float log_share(float x, float max, float T, float whole, float most) {
  return (0.5f * x - 0.5f * max) / T * 2.f - logf(whole / most);
}

// How many of the warps with `per` of `vecs` vectors each have all of theirs.
__device__ __forceinline__ int w_full(int vecs, int per) { return per >= 32 ? vecs / per : 0; }

// Whether a logit of the row (each thread's vectors v0 .. v1 - 1) lies beyond kFar; -inf does not.
template <bool half>
__device__ __noinline__ bool any_far(const uint4* data, int v0, int v1, Ctl* ctl, int C, int rank) {
  float m = 0.f;
  for (int v = v0; v < v1; ++v) {
    float x[Vec<half>::n];
    unpack<half>(data[v], x);
#pragma unroll
    for (int e = 0; e < Vec<half>::n; ++e) m = fmaxf(m, x[e] == -kInf ? 0.f : fabsf(x[e]));
  }
  uint32_t far = __syncthreads_or(m > kFar) != 0 ? 1u : 0u;
  if (C > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (static_cast<int>(threadIdx.x) < C) cluster.map_shared_rank(ctl->far, static_cast<int>(threadIdx.x))[rank] = far;
    cluster.sync();
    for (int r = 0; r < C; ++r) far |= ctl->far[r];
  }
  return far != 0u;
}

// The smallest logit that min-p leaves; by one thread.
__device__ __noinline__ float least_of(float max, float min_p, float T) {
  const double at = static_cast<double>(max) + log(static_cast<double>(fminf(min_p, 1.f))) * static_cast<double>(T);
  const float least = static_cast<float>(at);
  return static_cast<double>(least) < at ? nextafterf(least, kInf) : least;
}

// The rest of a row whose k largest are among the list's, by the first block alone:
// what may be among them again, put in order by counting the larger ones, weighed,
// cut, and drawn from in the order of the indices.
__device__ __noinline__ void sample_list(const SampleArgs& a, Ctl* ctl, int row, int k, float p, float min_p, float T, float max) {
  const int t = threadIdx.x;
  constexpr int kSlots = kMaxCluster * kList, kOwn = kSlots / kThreads;
  static_assert(kSlots % kThreads == 0 && kListK <= kThreads, "slots of a thread");
  u64* some = reinterpret_cast<u64*>(&ctl->hist[0][0][0]);       // (value, index), the larger the earlier
  static_assert(sizeof(ctl->hist) >= 8 * kSlots, "room for the list");
  u64* sorted = reinterpret_cast<u64*>(ctl->list_index);
  u64* weights = sorted + kListK;
  float x[kOwn], own = -kInf;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) x[i] = ctl->list[t + i * kThreads], own = fmaxf(own, x[i]);
  const float edge = edge_of(ctl, own, k, kWarps);
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (x[i] >= edge) some[atomicAdd(&ctl->first[0], 1)] = static_cast<u64>(key_of(x[i])) << 32 | static_cast<uint32_t>(~ctl->list_index[t + i * kThreads]);
  if (t == 0 && min_p > 0.f) ctl->redf[0][0] = least_of(max, min_p, T);
  __syncthreads();
  const int n = ctl->first[0], kk = min(k, n);
  for (int i = t; i < n; i += kThreads) {
    const u64 mine = some[i];
    int at = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) at += some[j] > mine ? 1 : 0;
    if (at < kk) sorted[at] = mine;
  }
  __syncthreads();
  const u64 mine = t < kk ? sorted[t] : 0ull;
  const float v = of_key(static_cast<uint32_t>(mine >> 32));
  const u64 w = t < kk ? weight(v, ctl->scale, ctl->powers) : 0ull;
  u64 all;
  const u64 ahead = block_scan(w, ctl->red64, all) - w;
  bool kept = t < kk;
  if (p < 1.f) {
    const u64 frac = fraction(p);
    u64 target = __umul64hi(frac, all);
    if (frac * all != 0ull) ++target;  // rounded up
    kept = kept && (t == 0 || ahead < target);
  }
  if (min_p > 0.f) kept = kept && v >= ctl->redf[0][0];
  const int n_kept = __syncthreads_count(kept);  // the first ones
  if (kept) weights[t] = w;
  if (t == n_kept - 1) ctl->span[0] = ahead + w;
  __syncthreads();
  if (!kept) return;
  const u64 whole = ctl->span[0], at = __umul64hi(fraction(__ldg(a.u + row)), whole);
  const uint32_t place = ~static_cast<uint32_t>(mine);
  u64 before = 0;
#pragma unroll 4
  for (int j = 0; j < n_kept; ++j) before += ~static_cast<uint32_t>(sorted[j]) < place ? weights[j] : 0ull;
  if (before <= at && at < before + w) {
    a.tokens[row] = static_cast<int32_t>(place);
    if (a.logprobs != nullptr)
      a.logprobs[row] = log_share(v, max, T, static_cast<float>(whole), static_cast<float>(weight(max, ctl->scale, ctl->powers)));
  }
}

// ---------------------------------------------------------------- one block a row
// Many rows: a block reads a row once, from end to end, and is done with it if all
// that is asked for is the largest logit, the top-k of few (whose list a second look
// at some threads' elements gives), or a draw from everything (whose mass is added
// up on the way, in fp32, in the unit of the largest so far; powers of two apart,
// so that nothing is lost when it changes).  Other rows, and those where fp32 leaves
// doubt, it leaves to the clusters, whose launch is made ready while this one runs and
// waits for its end (256 rows with top-k 50: 59 us to 54).  Measured against clusters for
// all (us): 64 rows of 128000 with top-k 50 27 to 27, unfiltered 41 to 27; 96 33 to 37
// and 45 to 38; 128 35 to 46 and 47 to 49; 256 54 to 82 and 63 to 83.  (Rows that fit one
// block's shared memory are read once either way: 1024 x 32003 75 to 48.)
// The loads go to shared memory by themselves: four vectors a thread on their way that
// way instead of in registers took 150 rows' largest from 28 us to 23; eight 21, but
// 256 rows with top-k 50, whose second look then finds no room in L1, 70.
constexpr int32_t kLeft = -0x7FFFFFFF - 1;
constexpr int kRowsFrom = 128;  // rows of a call from which on it is used
constexpr int kAhead = 4;       // vectors of a thread on their way (a power of two)

template <bool half>
__global__ void __launch_bounds__(kThreads, 2) sample_rows_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint4 ring[];  // a thread's next vectors, every kThreads-th
  __shared__ Ctl shared;
  constexpr int E = Vec<half>::n, kBytes = 16 / E;
  Ctl* ctl = &shared;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, row = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;");  // (which wait for this launch's end)
  float T = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
  const int k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
  const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;
  const bool greedy = !(T >= 1.17549435e-38f) || k == 1, list = k > 0 && k <= kListK, plain = !greedy && k <= 0 && !(p < 1.f) && !(min_p > 0.f);
  if (!greedy && !list && !plain) {
    if (t == 0) a.tokens[row] = kLeft;
    return;
  }
  T = fminf(T, kMost);
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
  const float ch = kLog2e / T, cl = (fmaf(-ch, T, kLog2e) + kLog2eLo) / T, span = (kUnit + 1.5f) * 0.6931472f * T;
  if (t < 64) ctl->powers[t] = kPowers[t];

  const uint8_t* start = static_cast<const uint8_t*>(a.logits) + static_cast<long long>(row) * a.ld * kBytes;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(start) & 15u) / kBytes);
  const int vecs = (off + a.V + E - 1) / E, per = (vecs + kWarps - 1) / kWarps;
  const int w0 = min(warp * per, vecs), w1 = min(w0 + per, vecs);  // the warp's vectors, lane after lane
  const uint4* from = reinterpret_cast<const uint4*>(start - off * kBytes);
  const bool last_whole = off + a.V == vecs * E;
  const int whole0 = off != 0 ? 1 : 0, whole1 = last_whole ? vecs : vecs - 1;  // vectors that are the row's alone
  // vector v; elements that are not the row's (the first and the last vector only) are -inf
  auto load = [&](int v) -> uint4 {
    if (v >= whole0 && v < whole1) return __ldg(from + v);
    uint4 w = half ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                   : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    for (int e = 0; e < E; ++e) {
      const int i = v * E + e - off;
      if (i < 0 || i >= a.V) continue;
      if constexpr (half)
        reinterpret_cast<uint16_t*>(&w)[e] = reinterpret_cast<const uint16_t*>(start)[i];
      else
        reinterpret_cast<uint32_t*>(&w)[e] = reinterpret_cast<const uint32_t*>(start)[i];
    }
    return w;
  };

  // of the warp's those are f0 .. f1 - 1, lane after lane; the others are lane 0's
  const int f0 = max(w0, whole0), f1 = min(w1, whole1);
  const bool edge0 = w0 < w1 && f0 > w0, edge1 = w0 < w1 && f1 < w1 && f1 >= f0;

  // ---- the one pass: the thread's largest, and the mass
  const float2 ch2 = make_float2(ch, ch), cl2 = make_float2(cl, cl);
  float own = -kInf, unit = kMagic, low = -kMost;
  const float nothing = -2100.f / ch;  // logits of no weight in rows that are not left below (-inf is one)
  RoughSum sum;
  auto take = [&](const uint4& w) {
    float x[E];
    unpack<half>(w, x);
    float m = x[0];  // (NaN is passed over)
#pragma unroll
    for (int e = 1; e < E; ++e) m = fmaxf(m, x[e]);
    if (!plain || !(m > nothing)) {
      own = fmaxf(own, m);
      return;
    }
    if (m > own) {
      own = m;
      const float u = kMagic - fminf(fmaxf(ceilf(m * ch), -4000.f), 4000.f);
      if (u != unit) {
        const float f = power_of_two(u - unit);
        sum.s *= f, sum.lost *= f;
        unit = u;
      }
      low = fmaxf(m - span, -kMost);
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < E; e += 4) {  // by pairs, two and two
      const float2 a2 = rough2(make_float2(x[e], x[e + 1]), ch2, cl2, make_float2(unit, unit), low);
      const float2 b2 = rough2(make_float2(x[e + 2], x[e + 3]), ch2, cl2, make_float2(unit, unit), low);
      s2 = e == 0 ? __fadd2_rn(a2, b2) : __fadd2_rn(s2, __fadd2_rn(a2, b2));
    }
    sum.add(s2.x + s2.y);
  };
  {
    if (lane == 0 && edge0) take(load(w0));
    if (lane == 0 && edge1) take(load(w1 - 1));
    const int n = max(f1 - f0 - lane + 31, 0) >> 5;
    const uint4* at = from + f0 + lane;
    uint4* const slots = ring + t;
    auto fetch = [&](int i) {
      if (i < n)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(slots + (i & (kAhead - 1)) * kThreads))),
                     "l"(at + 32 * i) : "memory");
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      take(slots[(i & (kAhead - 1)) * kThreads]);
      fetch(i + kAhead);
    }
  }
  float mx = own;
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) ctl->redf[0][warp] = mx;
  __syncthreads();
  mx = ctl->redf[0][lane & (kWarps - 1)];
#pragma unroll
  for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  // f of the elements (and their indices) of the warp's threads that `some` names, the warp together over each
  auto again = [&](unsigned some, auto f) {
    auto look = [&](int v) {
      float x[E];
      unpack<half>(load(v), x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e], v * E + e - off);
    };
    if ((some & 1u) && lane == 0 && edge0) look(w0);
    if ((some & 1u) && lane == 0 && edge1) look(w1 - 1);
    const int chunks = (f1 - f0 + 1023) >> 10;  // of 32 vectors of a thread
    int c = 0;
#pragma unroll 1
    while (some != 0u && chunks > 0) {  // four loads on their way together
      uint4 w[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int v = f0 + __ffs(static_cast<int>(some)) - 1 + 32 * lane + 1024 * c;
        at[u] = some != 0u && v < f1 ? v : -1;
        if (at[u] >= 0) w[u] = __ldg(from + v);
        if (++c == chunks) c = 0, some &= some - 1u;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (at[u] < 0) continue;
        float x[E];
        unpack<half>(w[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) f(x[e], at[u] * E + e - off);
      }
    }
  };
  if (mx == -kInf) {
    if (t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs != nullptr) a.logprobs[row] = -kInf;
    }
    return;
  }
  if (greedy) {
    uint32_t best = 0xFFFFFFFFu;
    again(__ballot_sync(0xFFFFFFFFu, own == mx), [&](float x, int i) {
      if (x == mx) best = min(best, static_cast<uint32_t>(i));
    });
    best = __reduce_min_sync(0xFFFFFFFFu, best);
    if (lane == 0) ctl->red32[warp] = best;
    __syncthreads();
    if (t == 0) {
      for (int w = 0; w < kWarps; ++w) best = min(best, ctl->red32[w]);
      a.tokens[row] = static_cast<int32_t>(best);
      if (a.logprobs != nullptr) a.logprobs[row] = 0.f;
    }
    return;
  }
  const float max_power = mx * ch, row_low = fmaxf(mx - span, -kMost);
  const bool wide = is_wide(max_power, ch, T >= kHot);  // (no look at all logits: a list's few weights are fast either way)
  if (mx == kInf || (plain && (wide || row_low <= -kMost))) {  // (the last: forbidden logits counted as the lowest ones, which weigh something)
    if (t == 0) a.tokens[row] = kLeft;
    return;
  }
  if (list) {
    if (t == 0) ctl->scale = Scale{ch, cl, wide ? 0 : __float2int_rn(64.f * max_power), row_low, wide ? 1 : 0, mx, wide ? powers_per(T) : 0.0};
    for (int i = t; i < kMaxCluster * kList; i += kThreads) ctl->list[i] = -kInf;
    const float edge = edge_of(ctl, own, k, w_full(vecs, per));
    again(__ballot_sync(0xFFFFFFFFu, own >= edge), [&](float x, int i) {
      if (x >= edge) {
        const int at = atomicAdd(&ctl->first[0], 1);
        if (at < kMaxCluster * kList) ctl->list[at] = x, ctl->list_index[at] = static_cast<uint32_t>(i);
      }
    });
    __syncthreads();
    const int n = ctl->first[0];
    __syncthreads();
    if (n > kMaxCluster * kList) {
      if (t == 0) a.tokens[row] = kLeft;
      return;
    }
    sample_list(a, ctl, row, k, p, min_p, T, mx);
    return;
  }
  // ---- a draw from everything: the warp, a sixteenth of it, and the place there
  const float row_unit = kMagic - ceilf(max_power);
  const float f = power_of_two(row_unit - unit);
  sum.s *= f, sum.lost *= f;
  const u64 upto = warp_sum(sum.units());
  if (lane == 0) ctl->span[warp] = upto;
  __syncthreads();
  u64 before = 0, whole = 0;
  int at_warp = 0;
  for (int w = 0; w < kWarps; ++w) whole += ctl->span[w];
  const u64 at = __umul64hi(fraction(__ldg(a.u + row)), whole), doubt = (whole >> (kRough - 1)) + (1ull << 17);
  for (; at_warp < kWarps - 1 && at >= before + ctl->span[at_warp]; ++at_warp) before += ctl->span[at_warp];
  const int s0 = min(at_warp * per, vecs), s1 = min(s0 + per, vecs), part = ((s1 - s0 + kWarps - 1) / kWarps + 31) & ~31;
  const int q0 = min(s0 + warp * part, s1), q1 = min(q0 + part, s1);
  RoughSum mine;
  for (int v = q0 + lane; v < q1; v += 32) {
    float x[E];
    unpack<half>(load(v), x);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] >= row_low ? rough(x[e], ch, cl, row_unit) : 0.f;
    mine.add(x);
  }
  const u64 here = warp_sum(mine.units());
  if (lane == 0) ctl->red64[warp] = here;
  if (t == 0) a.tokens[row] = kLeft;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += ctl->red64[w];
  if (before <= at && at < before + here) {
    for (int v = q0; v < q1; v += 32) {
      float x[E], w[E];
      if (v + lane < q1) {
        unpack<half>(load(v + lane), x);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = -kInf;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = x[e] >= row_low ? rough(x[e], ch, cl, row_unit) : 0.f;
      RoughSum r;
      r.add(w);
      const u64 units = r.units(), sums = warp_scan(units, lane), all = __shfl_sync(0xFFFFFFFFu, sums, 31);
      if (at >= before + all) {
        before += all;
        continue;
      }
      u64 m = before + sums - units;
      if (m <= at && at < m + units) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const u64 one = __float2ull_rn(w[e] * kOne);
          if (at >= m + doubt && at + doubt < m + one) {
            a.tokens[row] = (v + lane) * E + e - off;
            if (a.logprobs != nullptr)
              a.logprobs[row] = log_share(x[e], mx, T, static_cast<float>(whole), rough(mx, ch, cl, row_unit) * kOne);
          }
          m += one;
        }
      }
      break;
    }
  }
}

template <bool half>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int C, int left_only) {
  extern __shared__ __align__(16) uint4 part[];
  __shared__ Ctl shared;
  constexpr int E = Vec<half>::n, kBytes = 16 / E;
  Ctl* ctl = &shared;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = static_cast<int>(blockIdx.x) / C, rank = static_cast<int>(blockIdx.x) % C;
  Row<half> R{ctl, part, cg::this_cluster(), C, rank, 1, 0, 0};
  // (what the launch before left; read before the blocks meet, and written behind that)
  if (left_only) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (left_only && __ldcg(a.tokens + row) != kLeft) return;

  if (C > 1) R.cluster.barrier_arrive();  // (waited for before the first write to another block)

  // ---- what the row asks for
  float T = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
  const int k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
  const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;

  // ---- the block's part of the row, in vectors of 16 bytes; the elements of the
  // first and the last vector that are not the row's count as -inf
  const uint8_t* start = static_cast<const uint8_t*>(a.logits) + static_cast<long long>(row) * a.ld * kBytes;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(start) & 15u) / kBytes);
  const int vecs = (off + a.V + E - 1) / E, slice = (vecs + C - 1) / C;
  const int f0 = min(rank * slice, vecs);
  const int nvec = min(slice, vecs - f0);
  int base = f0 * E - off;  // index of the part's first element
  const uint4* from = reinterpret_cast<const uint4*>(start - off * kBytes) + f0;
  float most = -kInf;  // of what the thread has loaded
  __nv_bfloat162 most2 = __float2bfloat162_rn(-kInf);
  {
    auto put = [&](int v, uint4 w) {
      if constexpr (half) {  // (NaN counts as -inf)
        uint32_t* q = &w.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(q + i), __float2bfloat162_rn(-kInf));
          q[i] = *reinterpret_cast<const uint32_t*>(&m);
          most2 = __hmax2(most2, m);
        }
      } else {
        float* q = reinterpret_cast<float*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = fmaxf(q[i], -kInf), most = fmaxf(most, q[i]);
      }
      part[v] = w;
    };
    const int whole0 = base < 0 ? 1 : 0;  // vectors whole0 .. whole1 - 1 are the row's alone
    const int whole1 = (f0 + nvec) * E - off > a.V ? nvec - 1 : nvec;
    constexpr int kAhead = 8;
    int v = whole0 + t;
    for (; v + (kAhead - 1) * kThreads < whole1; v += kAhead * kThreads) {
      uint4 w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) w[i] = __ldcs(from + v + i * kThreads);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) put(v + i * kThreads, w[i]);
    }
    if (v < whole1) {
      uint4 w[kAhead - 1];
#pragma unroll
      for (int i = 0; i < kAhead - 1; ++i)
        if (v + i * kThreads < whole1) w[i] = __ldcs(from + v + i * kThreads);
#pragma unroll
      for (int i = 0; i < kAhead - 1; ++i)
        if (v + i * kThreads < whole1) put(v + i * kThreads, w[i]);
    }
    if (t < 2) {
      const int v = t == 0 ? 0 : nvec - 1;
      if (nvec > 0 && (t == 0 ? whole0 == 1 : whole1 < nvec && (nvec > 1 || whole0 == 0))) {
        uint4 w = half ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                       : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        for (int e = 0; e < E; ++e) {
          const int i = base + v * E + e;
          if (i < 0 || i >= a.V) continue;
          if constexpr (half)
            reinterpret_cast<uint16_t*>(&w)[e] = reinterpret_cast<const uint16_t*>(from + v)[e];
          else
            reinterpret_cast<uint32_t*>(&w)[e] = reinterpret_cast<const uint32_t*>(from + v)[e];
        }
        put(v, w);
      }
    }
  }
  if (t < 64) ctl->powers[t] = kPowers[t];
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i <= kParts; ++i) ctl->hist[1][i][t] = 0u;
    for (int i = t; i < kMaxCluster * kList; i += kThreads) ctl->list[i] = -kInf;
  }
  __syncthreads();

  // ---- the largest
  R.spread(part, nvec);
  if constexpr (half) most = fmaxf(__low2float(most2), __high2float(most2));
  const bool plain = k <= 0 && !(p < 1.f);
  float own = plain ? kInf : R.largest();  // no element of the thread's run is larger
  const bool greedy = !(T >= 1.17549435e-38f) || k == 1, listing = !greedy && k > 0 && k <= kListK;
  float mx = most;
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) ctl->redf[0][warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ctl->redf[0][w]);
  // (top-k of few: what k elements are not below, a C-th of them in each block)
  float edge = listing ? edge_of(ctl, own, (k + C - 1) / C, nvec / (32 * R.per)) : 0.f;
  if (C > 1) {
    R.cluster.barrier_wait();
    if (t < C) R.tell(ctl->max, mx), R.tell(ctl->edge, edge);
    R.meet();
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < C) mx = fmaxf(mx, ctl->max[r]), edge = fminf(edge, ctl->edge[r]);
  }
  if (mx == -kInf) {  // no token
    if (rank == 0 && t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs != nullptr) a.logprobs[row] = -kInf;
    }
    return;
  }
  if (greedy) {  // the largest one, the first of its equals
    uint32_t best = 0xFFFFFFFFu;
    if (own >= mx) {
      for (int v = R.v1 - 1; v >= R.v0; --v) {
        float x[E];
        unpack<half>(part[v], x);
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
          if (x[e] == mx) best = static_cast<uint32_t>(base + v * E + e);
      }
    }
    best = __reduce_min_sync(0xFFFFFFFFu, best);
    if (lane == 0) ctl->red32[warp] = best;
    __syncthreads();
    if (t == 0) {
      for (int w = 0; w < kWarps; ++w) best = min(best, ctl->red32[w]);
      *R.of(ctl->index + rank, 0) = best;
    }
    R.meet();
    if (rank == 0 && t == 0) {
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < C) best = min(best, ctl->index[r]);
      a.tokens[row] = static_cast<int32_t>(best);
      if (a.logprobs != nullptr) a.logprobs[row] = 0.f;
    }
    return;
  }
  T = fminf(T, kMost);
  if (mx == kInf) {  // only the infinite ones count, all alike
    for (int v = R.v0; v < R.v1; ++v)
      for (int e = 0; e < E; ++e) set_element<half>(part, v * E + e, element<half>(part, v * E + e) == kInf ? 0.f : -kInf);
    own = plain || own == kInf ? 0.f : -kInf;
    edge = edge == kInf ? 0.f : -kMost;
    mx = 0.f;
  }
  const bool far = T >= kHot && any_far<half>(part, R.v0, R.v1, ctl, C, rank);
  // log2(e) / T as two numbers
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
  const float ch = kLog2e / T, cl = (fmaf(-ch, T, kLog2e) + kLog2eLo) / T;
  const float max_power = mx * ch, low = fmaxf(fmaf(-(kUnit + 1.5f) * 0.6931472f, T, mx), -kMost);
  const bool wide = is_wide(max_power, ch, far);
  const int powers_top = wide ? 0 : __float2int_rn(64.f * max_power);
  const float unit = kMagic - ceilf(wide ? 0.f : max_power);  // for rough weights
  if (t == 0) ctl->scale = Scale{ch, cl, powers_top, low, wide ? 1 : 0, mx, wide ? powers_per(T) : 0.0};
  __syncthreads();
  const Scale& s = ctl->scale;  // (for calls)
  const bool by_mass = p < 1.f;
  const uint32_t top = key_of(mx);
  const float per = 16.f * ch;

  const int room = kMaxCluster / C * kList;  // of each block's part of the list

  // ---- top-k of few: a list of what may be among them
  if (listing) {
    if (own >= edge) {
      float* list = R.of(ctl->list, 0);
      uint32_t* to = R.of(ctl->list_index, 0);
      R.between(edge, kInf, [&](float x, int i) {
        const int at = atomicAdd(&ctl->first[0], 1);
        if (at < room) {
          list[rank * room + at] = x;
          to[rank * room + at] = static_cast<uint32_t>(base + i);
        }
      });
    }
    __syncthreads();
    if (t < C) R.tell(ctl->listed, static_cast<uint32_t>(ctl->first[0]));
    R.meet();
    bool fits = true;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) fits = fits && (r >= C || ctl->listed[r] <= static_cast<uint32_t>(room));
    if (fits) {
      if (rank == 0) sample_list(a, ctl, row, k, p, min_p, T, mx);
      return;
    }
  }
  // by how much two sums of rough weights may be off against each other
  auto doubt_of = [](u64 whole) { return (whole >> (kRough - 1)) + (1ull << 17); };

  // ---- the cut
  Cut cut{-kInf, 0.f, 0u};
  if (k > 0 || by_mass) {
    // all of it added up on the way, in fp32 (behind a top-k it would say little of what is left: 17000 of 128000
    // logits 96 us for 65)
    const bool whole_mass = by_mass && !wide && k <= 0;
    R.clear(false);
    if (whole_mass) {
      RoughSum sum;
      const float2 ch2 = make_float2(ch, ch), cl2 = make_float2(cl, cl), unit2 = make_float2(unit, unit);
      for (int v = R.v0; v < R.v1; ++v) {
        float x[E];
        unpack<half>(R.data[v], x);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (x[e] != -kInf) R.count(bin_of(x[e], mx, per), 0ull, false);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float2 w = __fadd2_rn(rough2(make_float2(x[e], x[e + 1]), ch2, cl2, unit2, low),
                                      rough2(make_float2(x[e + 2], x[e + 3]), ch2, cl2, unit2, low));
          sum.add(w.x + w.y);
        }
      }
      const u64 all = warp_sum(sum.units());
      if (lane == 0) ctl->red64[warp] = all;
      __syncthreads();
      if (t == 0) {
        u64 sums = 0;
        for (int w = 0; w < kWarps; ++w) sums += ctl->red64[w];
        *R.of(ctl->all + R.rank, 0) = sums;
      }
    } else {
      R.each([&](float x) {
        if (x != -kInf) R.count(bin_of(x, mx, per), 0ull, false);
      });
    }
    R.combine(false);
    if (R.rank == 0) {
      const uint32_t most = k > 0 ? static_cast<uint32_t>(k) : 0xFFFFFFFFu;
      const uint32_t n0 = R.find(false, most, 0ull);
      if (by_mass) {  // by the weights at the bins' edges
        uint32_t all;
        const uint32_t n = block_scan(n0, ctl->red32, all) - n0;
        const float kept = n < most ? static_cast<float>(min(n0, most - n)) : 0.f;
        const float hi0 = kept * exp2f(fminf(-0.0625f * (t - 0.5f), 0.f)), lo0 = t + 1 < kBins ? kept * exp2f(-0.0625f * (t + 0.5f)) : 0.f;
        float hi_all, lo_all;
        const float hi = block_scan(hi0, ctl->redf[0], hi_all), lo = block_scan(lo0, ctl->redf[1], lo_all);
        if (t == 0) ctl->first[0] = ctl->first[1] = kBins - 1;
        __syncthreads();
        float mass = hi_all;
        if (whole_mass) {
          // the mass is known: what lies behind the cut is nearer to its edges' weights than what lies ahead
          u64 sums = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            if (r < R.C) sums += ctl->all[r];
          mass = static_cast<float>(sums) / kOne * exp2f(ceilf(max_power) - max_power);  // (of the largest)
          if (lo_all - lo <= 1.0001f * (1.f - p) * mass + 2e-6f * mass) atomicMin(&ctl->first[0], t);
          if (hi_all - hi <= 0.9999f * (1.f - p) * mass - 2e-6f * mass) atomicMin(&ctl->first[1], t);
        } else {
          if (hi >= 0.999f * p * lo_all) atomicMin(&ctl->first[0], t);
          if (lo >= 1.001f * p * hi_all) atomicMin(&ctl->first[1], t);
        }
        __syncthreads();
        const int b1 = ctl->first[0], b2 = max(ctl->first[1], b1);
        __syncthreads();
        if (t == 0) {
          Found& f = ctl->found;
          f.b1 = b1, f.b2 = b2;
          // a token there weighs so little that fp32 sums would leave it in doubt four times in ten or more
          f.flat = exp2f(-0.0625f * b1) < 10.f * mass * (1.f / (1 << kRough)) ? 1 : 0;
        }
        __syncthreads();
      }
      if (warp < 4) {  // where those bins begin and end
        Found& f = ctl->found;
        const int b = warp == 0 ? f.bin : warp == 1 ? f.bin + 1 : warp == 2 ? f.b1 : f.b2 + 1;
        const uint32_t d = warp < 2 ? (f.bin >= 0 ? bin_start(b, top, mx, per, lane) : 0u) : by_mass ? bin_start(b, top, mx, per, lane) : 0u;
        if (lane == 0) (warp & 1 ? f.hi : f.lo)[warp >> 1] = warp & 1 ? d - 1u : d;
      }
      __syncthreads();
    }
    const Found f0 = R.share();
    const uint32_t lowest = top - key_of(-kMost);

    // The cut within the distances lo .. hi: the first `need` tokens there, or as
    // many as bring the mass from `base` to `target`, which may be off by `doubt`.
    // false: not there, or in doubt.  A few tokens go to the first block, which
    // adds up what is ahead of each; of more, the 512th that the cut is in.
    auto search = [&](bool masses, uint32_t lo, uint32_t hi, uint32_t need, u64 base, u64 target, u64 doubt) -> bool {
      // whether the mass without the last token is below the target, and with it is not
      auto sure = [&](u64 without, u64 with) { return doubt == 0 || (without + doubt < target && with >= target + doubt); };
#pragma unroll 1
      for (;;) {
        float xhi = of_key(top - lo), xlo = of_key(top - hi);
        __syncthreads();
        if (t == 0) ctl->first[0] = 0, ctl->nearest = 0xFFFFFFFFu, ctl->farthest = 0u;
        __syncthreads();
        if (own >= xlo) {
          float* list = R.of(ctl->list, 0);
          uint32_t near = 0xFFFFFFFFu, far = 0u;
          R.between(xlo, xhi, [&](float x, int) {
            const int at = atomicAdd(&ctl->first[0], 1);
            if (at < room) list[R.rank * room + at] = x;
            near = min(near, top - key_of(x)), far = max(far, top - key_of(x));
          });
          if (near <= far) atomicMin(&ctl->nearest, near), atomicMax(&ctl->farthest, far);
        }
        __syncthreads();
        if (t < R.C) {
          R.tell(ctl->listed, static_cast<uint32_t>(ctl->first[0]));
          R.tell(ctl->from, ctl->nearest);
          R.tell(ctl->to, ctl->farthest);
        }
        R.meet();
        uint32_t n = 0, most = 0, near = 0xFFFFFFFFu, far = 0u;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < R.C) n += ctl->listed[r], most = max(most, ctl->listed[r]), near = min(near, ctl->from[r]), far = max(far, ctl->to[r]);
        if (n <= kFinish && most <= static_cast<uint32_t>(room)) {
          if (R.rank == 0) {
            u64* w = reinterpret_cast<u64*>(ctl->list_index);
            float* v = reinterpret_cast<float*>(w + kFinish);
            static_assert(sizeof(ctl->list_index) >= kFinish * 12, "room for the few");
            if (t < static_cast<int>(n)) {
              uint32_t at = t, r = 0;
              for (; at >= ctl->listed[r]; ++r) at -= ctl->listed[r];
              v[t] = ctl->list[r * room + at];
              w[t] = masses ? weight(v[t], s, ctl->powers) : 1ull;
            }
            if (t == 0) ctl->cut = Cut{0.f, 0.f, 0xFFFFFFFFu};
            __syncthreads();
            // each by 2 to 8 lanes
            const int lanes = n > kThreads / 4 ? 2 : n > kThreads / 8 ? 4 : 8, mine = t / lanes;
            if (mine - lane / lanes < static_cast<int>(n)) {
              const float x = v[min(mine, static_cast<int>(n) - 1)];
              u64 ahead = 0;
              uint32_t equals = 0, earlier = 0;
#pragma unroll 4
              for (int j = t & (lanes - 1); j < static_cast<int>(n); j += lanes) {
                const float y = v[j];
                ahead += y > x ? w[j] : 0ull;
                equals += y == x ? 1u : 0u;
                earlier += y == x && j < mine ? 1u : 0u;
              }
              for (int o = 1; o < lanes; o <<= 1) {
                ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, o);
                equals += __shfl_xor_sync(0xFFFFFFFFu, equals, o);
                earlier += __shfl_xor_sync(0xFFFFFFFFu, earlier, o);
              }
              ahead += base;
              const u64 one = w[min(mine, static_cast<int>(n) - 1)], to = masses ? target : base + need;
              if (mine < static_cast<int>(n) && (t & (lanes - 1)) == 0 && earlier == 0u && ahead < to && to <= ahead + equals * one) {
                const uint32_t last = masses ? static_cast<uint32_t>((to - ahead + one - 1) / one) : static_cast<uint32_t>(to - ahead);
                if (!masses || sure(ahead + (last - 1) * one, ahead + last * one))
                  ctl->cut = last >= equals ? Cut{x, 0.f, 0u} : Cut{of_key(key_of(x) + 1u), x, last};
              }
            }
            __syncthreads();
            if (t > 0 && t < R.C) *R.of(&ctl->cut, t) = ctl->cut;
          }
          R.meet();
          const Cut c = ctl->cut;
          if (c.ties == 0xFFFFFFFFu) return false;
          cut = c;
          return true;
        }
        if (n == 0u) return false;
        // (what is there reaches from `near` to `far`)
        lo = near, hi = far;
        const uint32_t range = hi - lo;
        uint32_t count = n;
        u64 one = 0;
        if (range > 0u) {
          const int shift = range < kBins ? 0 : 23 - __clz(static_cast<int>(range));
          xhi = of_key(top - lo), xlo = of_key(top - hi);
          R.clear(masses);
          if (own >= xlo) {
            R.between(xlo, xhi, [&](float x, int) {
              const uint32_t d = top - key_of(x) - lo;
              if (d > range) return;  // (a zero beside -0)
              R.count(static_cast<int>(d >> shift), masses ? weight(x, s, ctl->powers) : 0ull, masses);
            });
          }
          R.combine(masses);
          if (R.rank == 0) R.find(masses, need, target - base);
          const Found f = R.share();
          if (f.bin < 0) return false;
          need -= f.before;
          base += f.mass_before;
          lo += static_cast<uint32_t>(f.bin) << shift;
          hi = min(hi, lo + ((1u << shift) - 1u));
          if (masses ? f.count == 1u : need == f.count) {  // all of it
            cut.least = of_key(top - hi);
            cut.ties = 0u;
            return !masses || sure(base, base + f.mass);
          }
          if (shift != 0) continue;
          count = f.count;
          if (masses) one = f.mass / f.count;
        } else if (masses) {
          one = weight(of_key(top - lo), s, ctl->powers);
        }
        // one value: so many of its equals
        if (masses) {
          if (target <= base || one == 0ull) return false;
          const u64 last = (target - base + one - 1) / one;
          if (last > count || !sure(base + (last - 1) * one, base + last * one)) return false;
          need = static_cast<uint32_t>(last);
        } else if (need > count) {
          return false;
        }
        cut.tie = of_key(top - lo);
        cut.ties = need;
        if (need >= count) {
          cut.least = cut.tie;
          cut.ties = 0u;
        } else {
          cut.least = lo > 0 ? of_key(top - (lo - 1)) : kInf;
        }
        return true;
      }
    };
    uint32_t last = lowest;  // distance of the last token that top-k leaves (but for ties)
    if (k > 0 && f0.bin >= 0) {
      search(false, f0.lo[0], f0.hi[0], static_cast<uint32_t>(k) - f0.before, 0ull, 0ull, 0ull);
      last = cut.least == kInf ? 0u : top - key_of(cut.least);
    }
    if (by_mass) {
      const uint32_t hi = min(f0.hi[1], last), lo = min(f0.lo[1], hi);
      const Cut by_k = cut;
      const u64 frac = fraction(p);
      const float xhi = of_key(top - lo), xlo = of_key(top - hi), part_per = (kBins - 2) / fmaxf(xhi - xlo, 1e-30f);
      // from rough units to exact ones
      const u64 scale = __float2ull_rn(exp2f(ceilf(max_power) - powers_top * 0.015625f) * 4611686018427387904.f);  // 1 .. 2, in 2^-62
      auto exact_units = [&](u64 x) { return __umul64hi(x, scale) << 2; };
#pragma unroll 1
      for (bool exact = wide || f0.flat != 0;; exact = true) {
        cut = by_k;
        // the mass of all, of what lies above the bins, and (many tokens) of a 512th each of the logits between
        u64 all = 0, ahead = 0;
        const float least = fmaxf(by_k.least, low);
        const bool fine = !wide;
        if (fine) R.clear(true);
        if (wide) {
          if (own >= least) {
            R.between(least, kInf, [&](float x, int) {
              const u64 w = weight(x, s, ctl->powers);
              all += w;
              if (x > xhi) ahead += w;
            });
          }
        } else {
          const float2 ch2 = make_float2(ch, ch), cl2 = make_float2(cl, cl), unit2 = make_float2(unit, unit);
          const float inside = fmaxf(xlo, least);
          RoughSum sum, sum_ahead;
#pragma unroll 1
          for (int v = R.v0; v < R.v1; ++v) {
            float x[E];
            unpack<half>(R.data[v], x);
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) in |= x[e] >= inside && x[e] <= xhi ? 1u << e : 0u;
            if (exact) {
#pragma unroll
              for (int e = 0; e < E; e += 2) {
                u64 w0, w1;
                weight_near2(make_float2(x[e], x[e + 1]), ch2, cl2, powers_top, ctl->powers, w0, w1);
                all += (x[e] >= least ? w0 : 0ull) + (x[e + 1] >= least ? w1 : 0ull);
                ahead += (x[e] > xhi ? w0 : 0ull) + (x[e + 1] > xhi ? w1 : 0ull);
              }
            } else {
#pragma unroll
              for (int e = 0; e < E; e += 2) {
                const float2 w = rough2(make_float2(x[e], x[e + 1]), ch2, cl2, unit2, low);
                const float w0 = x[e] >= least ? w.x : 0.f, w1 = x[e + 1] >= least ? w.y : 0.f;
                sum.add(w0 + w1);
                sum_ahead.add((x[e] > xhi ? w0 : 0.f) + (x[e + 1] > xhi ? w1 : 0.f));
              }
            }
#pragma unroll 1
            for (; in != 0u; in &= in - 1u) {  // few
              const float z = element<half>(R.data, v * E + __ffs(static_cast<int>(in)) - 1);
              R.count(bin_of(z, xhi, part_per),
                      exact ? weight_near(z, ch, cl, powers_top, ctl->powers) : __float2ull_rn(rough(z, ch, cl, unit) * kOne), true);
            }
          }
          if (!exact) all = sum.units(), ahead = sum_ahead.units();
        }
        all = warp_sum(all), ahead = warp_sum(ahead);
        __syncthreads();
        if (lane == 0) ctl->red64[warp] = all, ctl->span[warp] = ahead;
        __syncthreads();
        if (t < R.C) {
          all = ahead = 0;
          for (int w = 0; w < kWarps; ++w) all += ctl->red64[w], ahead += ctl->span[w];
          R.tell(ctl->mass[0], all);
          R.tell(ctl->mass[1], ahead);
        }
        if (fine)
          R.combine(true);
        else
          R.meet();
        all = ahead = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < R.C) all += ctl->mass[0][r], ahead += ctl->mass[1][r];
        const u64 one = by_k.ties == 0u ? 0ull : exact ? weight(by_k.tie, s, ctl->powers)
                        : by_k.tie < low ? 0ull : __float2ull_rn(rough(by_k.tie, ch, cl, unit) * kOne);
        const u64 whole = all + by_k.ties * one;
        u64 target = __umul64hi(frac, whole);
        if (frac * whole != 0ull) ++target;  // rounded up
        target = target > 0ull ? target : 1ull;
        if (by_k.ties > 0u && target + (exact ? 0ull : doubt_of(whole)) > all) {  // among top-k's last equals, or next to them
          if (exact) {
            cut.ties = static_cast<uint32_t>(min((target - all + one - 1) / max(one, 1ull), static_cast<u64>(cut.ties)));
            break;
          }
          if (R.rank == 0) {
#pragma unroll
            for (int i = 0; i <= kParts; ++i) ctl->hist[1][i][t] = 0u;
          }
          R.meet();
          continue;
        }
        uint32_t first = lo, end = hi;
        bool there = ahead < target;
        if (fine) {
          if (R.rank == 0) {
            R.find(true, 0u, there ? target - ahead : 1ull);
            Found& f = ctl->found;
            if (warp < 2 && f.bin >= 0) {
              const uint32_t d = bin_start(f.bin + warp, top, xhi, part_per, lane);
              if (lane == 0) (warp ? f.hi : f.lo)[1] = warp ? min(hi, d - 1u) : max(lo, d);
            }
            __syncthreads();
          }
          const Found f = R.share();
          there = there && f.bin >= 0;
          if (there) first = f.lo[1], end = f.hi[1], ahead += f.mass_before;
        }
        if (!exact) ahead = exact_units(ahead), target = exact_units(target), all = exact_units(all);
        const bool found = there && search(true, first, end, 0u, ahead, target, exact ? 0ull : doubt_of(all));
        if (!found && exact) {
          R.meet();  // (a search may end right behind its reading of what others write again)
          cut = by_k;
          search(true, 0u, last, 0u, 0ull, target, 0ull);  // (it lies elsewhere: the edges' weights were too rough)
        }
        if (found || exact) break;
        R.meet();
      }
    }
  }
  if (min_p > 0.f) {
    __syncthreads();
    if (t == 0) ctl->redf[0][0] = least_of(mx, min_p, T);
    __syncthreads();
    const float least = ctl->redf[0][0];
    cut.least = fmaxf(cut.least, least);
    if (cut.tie < least) cut.ties = 0u;
  }

  // ---- how many equals at the cut lie before the thread's own
  uint32_t ties_before = 0, own_ties = 0;
  if (cut.ties > 0u) {
    uint32_t all;
    R.each([&](float x) { own_ties += x == cut.tie ? 1u : 0u; });
    ties_before = block_scan(own_ties, ctl->red32, all) - own_ties;
    if (t < R.C) R.tell(ctl->ties, all);
    R.meet();
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < R.rank) ties_before += ctl->ties[r];
    own_ties = min(own_ties, cut.ties - min(cut.ties, ties_before));  // that are kept
  }
  // ---- the kept tokens' mass, thread by thread, and the token: the first one up to
  // which there is more than u of it.  In fp32 first; where u then lies next to a
  // border, exactly.
#pragma unroll 1
  for (bool exact = wide;; exact = true) {
    u64 sum = 0;
    const float least = fmaxf(cut.least, low);
    if (wide) {
      if (own >= least) R.between(least, kInf, [&](float x, int) { sum += weight(x, s, ctl->powers); });
    } else if (exact) {
      R.pairs([&](float x, float y) {
        u64 w[2];
        weight_near2(make_float2(x, y), make_float2(ch, ch), make_float2(cl, cl), powers_top, ctl->powers, w[0], w[1]);
        if (x >= least) sum += w[0];
        if (y >= least) sum += w[1];
      });
    } else {
      RoughSum r;
      const float2 ch2 = make_float2(ch, ch), cl2 = make_float2(cl, cl), unit2 = make_float2(unit, unit);
      if (least == low && low > -kMost) {  // (what weighs nothing counts as `low`)
        for (int v = R.v0; v < R.v1; ++v) {
          float x[E];
          unpack<half>(R.data[v], x);
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float2 w = __fadd2_rn(rough2(make_float2(x[e], x[e + 1]), ch2, cl2, unit2, low),
                                        rough2(make_float2(x[e + 2], x[e + 3]), ch2, cl2, unit2, low));
            r.add(w.x + w.y);
          }
        }
      } else {
        for (int v = R.v0; v < R.v1; ++v) {
          float x[E];
          unpack<half>(R.data[v], x);
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float2 w0 = rough2(make_float2(x[e], x[e + 1]), ch2, cl2, unit2, low),
                         w1 = rough2(make_float2(x[e + 2], x[e + 3]), ch2, cl2, unit2, low);
            r.add(((x[e] >= least ? w0.x : 0.f) + (x[e + 1] >= least ? w0.y : 0.f)) +
                  ((x[e + 2] >= least ? w1.x : 0.f) + (x[e + 3] >= least ? w1.y : 0.f)));
          }
        }
      }
      sum = r.units();
    }
    if (own_ties > 0u) sum += own_ties * (exact ? weight(cut.tie, s, ctl->powers) : cut.tie < low ? 0ull : __float2ull_rn(rough(cut.tie, ch, cl, unit) * kOne));
    const u64 upto = warp_scan(sum, lane);
    if (lane == 31) ctl->span[warp] = upto;
    if (t == 0) ctl->redo = exact ? 0u : 1u;
    __syncthreads();
    if (t < R.C) {
      u64 all = 0;
      for (int w = 0; w < kWarps; ++w) all += ctl->span[w];
      R.tell(ctl->all, all);
    }
    R.meet();
    u64 before = 0, whole = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r < R.C) {
        const u64 m = ctl->all[r];
        if (r < R.rank) before += m;
        whole += m;
      }
    }
    const u64 at = __umul64hi(fraction(__ldg(a.u + row)), whole);
    const u64 doubt = exact ? 0ull : doubt_of(whole);
    for (int w = 0; w < warp; ++w) before += ctl->span[w];
    if (before <= at && at < before + ctl->span[warp]) {
      // the thread, and all lanes over its elements
      const int from_lane = __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, at < before + upto))) - 1;
      before += __shfl_sync(0xFFFFFFFFu, upto - sum, from_lane);
      uint32_t ties = __shfl_sync(0xFFFFFFFFu, ties_before, from_lane);
      const int e0 = __shfl_sync(0xFFFFFFFFu, R.v0, from_lane) * E, e1 = __shfl_sync(0xFFFFFFFFu, R.v1, from_lane) * E;
      for (int i = e0; i < e1; i += 32) {
        const float x = i + lane < e1 ? element<half>(R.data, i + lane) : -kInf;
        bool kept = x >= cut.least && x != -kInf;
        if (cut.ties > 0u) {
          const unsigned tied = __ballot_sync(0xFFFFFFFFu, x == cut.tie && x != -kInf);
          if (x == cut.tie) kept = kept || ties + __popc(tied & ((1u << lane) - 1u)) < cut.ties;
          ties += __popc(tied);
        }
        const u64 w = !kept ? 0ull : exact ? weight(x, s, ctl->powers) : x < low ? 0ull : __float2ull_rn(rough(x, ch, cl, unit) * kOne);
        const u64 sums = warp_scan(w, lane);
        const unsigned past = __ballot_sync(0xFFFFFFFFu, at < before + sums);
        if (past == 0u) {
          before += __shfl_sync(0xFFFFFFFFu, sums, 31);
          continue;
        }
        if (lane == __ffs(static_cast<int>(past)) - 1) {
          const u64 mine = before + sums - w;
          if (exact || (at >= mine + doubt && at + doubt < mine + w)) {
            a.tokens[row] = base + i + lane;
            if (a.logprobs != nullptr) {
              const u64 most = exact ? weight(mx, s, ctl->powers) : __float2ull_rn(rough(mx, ch, cl, unit) * kOne);
              a.logprobs[row] = log_share(x, mx, T, static_cast<float>(whole), static_cast<float>(most));
            }
            if (!exact) {
#pragma unroll
              for (int r = 0; r < kMaxCluster; ++r)
                if (r < R.C) *R.of(&ctl->redo, r) = 0u;
            }
          }
        }
        break;
      }
    }
    if (exact) break;  // (no block writes into another's any more)
    R.meet();
    const uint32_t redo = ctl->redo;
    if (redo == 0u) break;
    __syncthreads();  // (all of the block have read it)
  }
}

template <bool half>
cudaError_t launch(const SampleArgs& a, int sms, cudaStream_t stream) {
  constexpr int E = Vec<half>::n;
  // Blocks a row: as few as hold it with two blocks an SM (1024 x 32003 bf16 logits:
  // one block 52 us, two 69; 256 x 128000 fp32 with top-p: eight 335, four with an SM
  // each 351), more while SMs are free (16 rows with top-p: eight 66, four 89).
  constexpr long long kSlice = (115 << 10) - static_cast<long long>(sizeof(Ctl)) - 2048;
  const long long bytes = static_cast<long long>(a.V + E - 1 + E - 1) / E * 16;  // wherever a row begins
  int C = 1;
  while (C < kMaxCluster && ((bytes + C - 1) / C > kSlice || (static_cast<long long>(a.N) * C * 2 <= sms && bytes / C > 8192))) C *= 2;
  const int smem = static_cast<int>((bytes / 16 + C - 1) / C * 16);
  // (the same limit in every call: another host thread's may come between this one and the launch)
  constexpr int kMostBytes = ((kSampleMaxVocab + 2 * E - 2) / E + kMaxCluster - 1) / kMaxCluster * 16;
  static_assert(kMostBytes + sizeof(Ctl) <= 232448, "the largest vocabulary in shared memory");
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<half>, cudaFuncAttributeMaxDynamicSharedMemorySize, std::max(kMostBytes, static_cast<int>(kSlice) + 16));
  if (e != cudaSuccess) return e;
  const int by_row = a.N >= kRowsFrom && C > 1 ? 1 : 0;
  if (by_row) {
    constexpr int kRing = kAhead * kThreads * 16;
    e = cudaFuncSetAttribute(sample_rows_kernel<half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (e != cudaSuccess) return e;
    sample_rows_kernel<half><<<static_cast<unsigned>(a.N), kThreads, kRing, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.N) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (behind the rows' launch: blocks ready when it ends)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = by_row ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<half>, a, C, by_row);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int sms, cudaStream_t stream) {
  return a.half ? launch<true>(a, sms, stream) : launch<false>(a, sms, stream);
}

}  // namespace fsops
