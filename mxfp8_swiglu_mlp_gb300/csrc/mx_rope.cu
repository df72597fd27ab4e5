// mx_rope.cu -- what stands between the projections and the attention over the
// paged MXFP8 cache:
//
//   norm_rope_kernel  per-head RMSNorm and position rotation of q and k, bf16
//                     to bf16.
//   kv_append_kernel  the new tokens' keys (norm, rotation) and values,
//                     quantised to MXFP8 straight from fp32 into their pages.
//
// Mathematics.  For a head x of D elements at position p:
//   x' = x * rsqrt(mean(x^2) + eps) * gamma        (without gamma: x' = x)
//   (u, w) -> (u cos a - w sin a, w cos a + u sin a),  a = p * inv_freq[i],
// on the R / 2 pairs of its first R dimensions.  The angle is taken modulo a
// turn in integers: inv_freq / 2 pi as a 64-bit fraction of a turn (good to
// 2^-64, from a sum of two fp64 numbers) times p, the overflow of the product
// being whole turns.  Its top 32 bits, good to 2^-32, become an fp32 number of
// half turns, which costs 2^-26 of a turn at most.  So a position of any size
// keeps an angle good to 2^-25 turns, where the fp32 product p * inv_freq is off
// by p * 2^-24 radians, and an fp64 one by p * 2^-54.
//
// Both kernels move each byte once and are bound by HBM (long inputs) or by
// launch latency (a decode step).  A lane holds two chunks of 8 consecutive
// elements (16-byte loads) of a head, in the half-split order one from each
// half: so a rotation's pairs are in one lane, D / 16 lanes hold a head, and
// its sum of squares takes log2(lanes) shuffles.  A warp computes a token's
// R / 2 sines and cosines once, one frequency a lane, hands them round through
// shared memory and keeps its lanes' eight in registers over the token's
// heads.  The turn fractions (fp64, whose rate is a small part of fp32's here)
// are computed once a block, whose warps go on to further tokens.
//
// Measured: 16384 tokens of 32 + 8 heads of 128 (336 MB) in 60 us, 5.6 TB/s; the
// append of 14 k tokens of 8 heads (87 MB) in 22 us; one token 2.6 and 3.2 us.
// With fractions, sines and pair partners computed lane by lane the two took 166
// and 104 us.
#include <cuda_bf16.h>

#include <algorithm>

#include "mx_device.cuh"
#include "mx_rope.h"

namespace fsops {

namespace {

constexpr int kRopeThreads = 128;
// Blocks an SM, at 80 and 96 registers a thread.  Measured: norm_rope with 16384
// tokens of 32 + 8 heads of 128 takes 60 us with 6, 65 with 5, 81 with 8 (spills);
// the append of 14 k tokens of 8 heads 22 us with 5, 25 with 6 (spills).
constexpr int kRopeBlocks = 6, kAppendBlocks = 5;
constexpr int kMaxRotary = 256;

// Fraction of a turn per position, in units of 2^-64 turns (|inv_freq| up to 2^40).
// (An fp64 instruction takes an SM some 30 cycles a warp, so what integers can do
// for them is left to integers: widening, and the product with 2^64.)
__device__ __forceinline__ long long turn_fraction(float inv_freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi) = kHi + kLo
  const uint32_t b = __float_as_uint(inv_freq);  // (zero and subnormal ones become 2^-127 or so)
  const double f = __longlong_as_double((static_cast<long long>(b & 0x7FFFFFFFu) << 29) + (896LL << 52) |
                                        static_cast<long long>(static_cast<unsigned long long>(b >> 31) << 63));
  const double r = f * kHi;
  // what the roundings of the product and of the constant left, below 2^-15: added to a
  // number whose last bit is 2^-64, so that it stands in the last bits
  constexpr double kLast = 0x1.8p-12;
  const double rest = fma(f, kLo, fma(f, kHi, -r)) + kLast;
  // without the whole turns per position, times 2^64; a sum that overflows is one more turn
  const double turn = __longlong_as_double(__double_as_longlong(r - rint(r)) + (64LL << 52));
  return static_cast<long long>(static_cast<unsigned long long>(__double2ll_rn(turn)) +
                                static_cast<unsigned long long>(__double_as_longlong(rest) - __double_as_longlong(kLast)));
}
// sine and cosine of position p's angle.
__device__ __forceinline__ void turn_sincos(long long f, int p, float* sn, float* cs) {
  const unsigned long long turns = static_cast<unsigned long long>(f) * static_cast<unsigned long long>(static_cast<long long>(p));
  // the top 32 bits, signed: [-1/2, 1/2) turns = [-1, 1) half turns
  const float half = static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half, sn, cs);
}

// The block's turn fractions, a thread each.
__device__ __forceinline__ void load_turns(long long* turns, const RopeArgs& a) {
  for (int i = threadIdx.x; i < a.R / 2; i += kRopeThreads)
    turns[i] = turn_fraction(__ldg(a.inv_freq + i));
  __syncthreads();
}

// A lane's place in a head of D / 16 lanes: its chunks of 8 elements, and
// whether they are rotated, by the frequencies 8 l .. 8 l + 7 either way.
struct Place {
  int c0, c1;  // first elements of the chunks
  bool on, rot, split;
};
__device__ __forceinline__ Place lane_place(int l, int D, const RopeArgs& a) {
  Place p;
  p.split = !a.interleaved;
  const int half = p.split ? a.R / 16 : 0;  // lanes with a chunk of each half
  p.c0 = 8 * (l < half ? l : 2 * l);
  p.c1 = 8 * (l < half ? l + half : 2 * l + 1);
  p.on = 16 * l < D;
  p.rot = 16 * l < a.R;
  return p;
}

struct Angles {
  float cs[8], sn[8];
};
// The token's angles, by the whole warp through its `tab`.
__device__ __forceinline__ void token_angles(Angles& g, const long long* turns, const RopeArgs& a, const Place& p, int l,
                                             int lane, int pos, float2* tab) {
  if (a.R == 0) return;
  __syncwarp();  // the last token's have been read
#pragma unroll 1
  for (int i = lane; i < a.R / 2; i += 32) {
    float sn, cs;
    turn_sincos(turns[i], pos, &sn, &cs);
    tab[i] = make_float2(cs, sn);
  }
  __syncwarp();
  if (p.rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(tab + 8 * l)[i];
      g.cs[2 * i] = x.x, g.sn[2 * i] = x.y, g.cs[2 * i + 1] = x.z, g.sn[2 * i + 1] = x.w;
    }
  }
}

struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_chunks(const uint16_t* head, const Place& p, bool on) {
  Raw w;
  w.a = w.b = make_uint4(0u, 0u, 0u, 0u);
  if (on) {
    w.a = *reinterpret_cast<const uint4*>(head + p.c0);
    w.b = *reinterpret_cast<const uint4*>(head + p.c1);
  }
  return w;
}
__device__ __forceinline__ uint32_t word(const Raw& w, int i) {
  const uint4& v = i < 4 ? w.a : w.b;
  return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
}

// The lane's 16 elements in fp32, normed with the gains gw and rotated.  Every
// lane of the warp calls it; LPH lanes hold a head.
template <int LPH>
__device__ __forceinline__ void norm_rotate(const Raw& w, bool norm, const Raw& gw, float inv_d, float eps,
                                            const Place& p, bool rot, const Angles& g, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[2 * i] = bf16_lo(word(w, i)), v[2 * i + 1] = bf16_hi(word(w, i));
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  if (norm) {
    const float rn = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] *= rn * bf16_lo(word(gw, i));
      v[2 * i + 1] *= rn * bf16_hi(word(gw, i));
    }
  }
  if (!rot) return;
  if (p.split) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = v[i], x = v[8 + i];
      v[i] = fmaf(u, g.cs[i], -x * g.sn[i]);
      v[8 + i] = fmaf(x, g.cs[i], u * g.sn[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = v[2 * i], x = v[2 * i + 1];
      v[2 * i] = fmaf(u, g.cs[i], -x * g.sn[i]);
      v[2 * i + 1] = fmaf(x, g.cs[i], u * g.sn[i]);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Unit (token, part): heads 0 .. of q then k, 32 / LPH a step; `parts` units
// share a token's steps.  Each step's loads are issued a step ahead.
template <int LPH>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int parts, unsigned units) {
  constexpr int HW = 32 / LPH;  // heads of a step
  __shared__ __align__(16) float2 tab[kRopeThreads / 32][kMaxRotary / 2];
  __shared__ long long turns[kMaxRotary / 2];
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH, warp = threadIdx.x >> 5;
  const unsigned warps = gridDim.x * (kRopeThreads / 32);
  load_turns(turns, a.rope);
  unsigned u = blockIdx.x * (kRopeThreads / 32) + warp;
  if (u >= units) return;
  int pos = a.rope.R > 0 ? __ldg(a.positions + u / parts) : 0;
  const Place p = lane_place(l, a.D, a.rope);
  const int heads = a.H[0] + a.H[1], steps = (heads + HW - 1) / HW;
  const float inv_d = 1.f / static_cast<float>(a.D);
  const Raw gq = load_chunks(a.gamma[0], p, p.on && a.gamma[0] != nullptr);
  const Raw gk = load_chunks(a.gamma[1], p, p.on && a.gamma[1] != nullptr);
  for (; u < units; u += warps) {
    const int t = static_cast<int>(u / parts), part = static_cast<int>(u % parts);
    const uint16_t* q = a.x[0] + t * a.ldx[0];
    const uint16_t* k = a.x[1] + t * a.ldx[1] - static_cast<long long>(a.H[0]) * a.D;
    uint16_t* yq = a.y[0] + t * a.ldy[0];
    uint16_t* yk = a.y[1] + t * a.ldy[1] - static_cast<long long>(a.H[0]) * a.D;
    int h = part * HW + sub;
    Raw w = load_chunks((h < a.H[0] ? q : k) + h * a.D, p, p.on && h < heads);
    const int at = pos;
    if (a.rope.R > 0 && u + warps < units) pos = __ldg(a.positions + (u + warps) / parts);
    Angles g;
    token_angles(g, turns, a.rope, p, l, lane, at, tab[warp]);
    for (int s = part; s < steps; s += parts) {
      const int hn = h + parts * HW;
      const Raw next = load_chunks((hn < a.H[0] ? q : k) + hn * a.D, p, p.on && hn < heads);
      const bool is_k = h >= a.H[0];
      float v[16];
      norm_rotate<LPH>(w, (is_k ? a.gamma[1] : a.gamma[0]) != nullptr, is_k ? gk : gq, inv_d, a.eps, p, p.rot, g, v);
      if (p.on && h < heads) {
        uint16_t* y = (is_k ? yk : yq) + h * a.D;
        *reinterpret_cast<uint4*>(y + p.c0) =
            make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
        *reinterpret_cast<uint4*>(y + p.c1) = make_uint4(bf16x2_rn(v[8], v[9]), bf16x2_rn(v[10], v[11]),
                                                         bf16x2_rn(v[12], v[13]), bf16x2_rn(v[14], v[15]));
      }
      w = next;
      h = hn;
    }
  }
}

// The sequence that holds row t, cu[0] <= t < cu[B]: the largest b < B with
// cu[b] <= t.  A warp narrows the range 32-fold a step.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, at < hi && __ldg(cu + min(at, B)) <= t);
    const int top = 31 - __clz(static_cast<int>(le | 1u));
    hi = min(hi, lo + (top + 1) * step);
    lo += top * step;
  }
  return lo;
}

__device__ __forceinline__ void report(uint32_t* status, uint32_t code, uint32_t site, int b) {
  atomicCAS(status, 0u, (code << 24) | (site << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
}

// Whether a sequence's offsets and length are within the limits (the length
// only where there are new tokens).
__device__ __forceinline__ bool sequence_ok(const KvAppendArgs& a, int c0, int c1, int len) {
  const bool offsets = (c0 >= 0) & (c0 <= c1) & (c1 <= a.T), length = (len >= c1 - c0) & (len <= (a.max_pages << a.log2P));
  return offsets & (length | (c0 == c1));
}
// The sequences looked at by one of `blocks` blocks.  (Not by the rows: none
// finds a sequence whose offsets decrease or lie outside the rows.)
__device__ __forceinline__ void check_sequences(const KvAppendArgs& a, int block, int blocks) {
#pragma unroll 1
  for (int b = block * kRopeThreads + threadIdx.x; b < a.B; b += blocks * kRopeThreads)
    if (!sequence_ok(a, __ldg(a.cu + b), __ldg(a.cu + b + 1), __ldg(a.lens + b))) report(a.status, 1u, 1u, b);
}

// Where a token goes: its row of head 0 in the cache (-1: nowhere).
struct Slot {
  long long row;
  int pos;
};
__device__ __forceinline__ Slot find_slot(const KvAppendArgs& a, int t, int lane) {
  Slot r;
  r.row = -1;
  r.pos = 0;
  const int b = find_sequence(a.cu, a.B, t, lane);
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.lens + b);
  // (no short circuits: the three loads go out together)
  if (!((t >= c0) & (t < c1) & sequence_ok(a, c0, c1, len))) return r;  // reported by check_sequences
  const int place = len - (c1 - t);
  const int page = __ldg(a.table + static_cast<long long>(b) * a.max_pages + (place >> a.log2P));
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) report(a.status, 1u, 2u, b);
    return r;
  }
  r.row = ((static_cast<long long>(page) * a.Hkv) << a.log2P) + (place & ((1 << a.log2P) - 1));
  r.pos = a.positions != nullptr ? __ldg(a.positions + t) : place;
  return r;
}

// Unit (token, part): the KV heads of k, then of v, four a step.  The last
// `checks` blocks look at the sequences instead, beside the others.
__global__ void __launch_bounds__(kRopeThreads, kAppendBlocks)
    kv_append_kernel(const __grid_constant__ KvAppendArgs a, int parts, unsigned units, int checks) {
  constexpr int D = 128, LPH = 8, HW = 4;
  __shared__ __align__(16) float2 tab[kRopeThreads / 32][D / 2];
  __shared__ long long turns[D / 2];
  __shared__ __align__(16) float peak[kRopeThreads / 32][HW][D / 8];  // largest magnitude of each chunk
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH, warp = threadIdx.x >> 5;
  const int blocks = static_cast<int>(gridDim.x) - checks;
  const unsigned warps = blocks * (kRopeThreads / 32);
  if (static_cast<int>(blockIdx.x) >= blocks) {
    check_sequences(a, blockIdx.x - blocks, checks);
    return;
  }
  load_turns(turns, a.rope);
  unsigned u = blockIdx.x * (kRopeThreads / 32) + warp;
  if (u >= units) return;
  const Place p = lane_place(l, D, a.rope);
  const int heads = 2 * a.Hkv, steps = (heads + HW - 1) / HW;
  const int row0 = __ldg(a.cu), row1 = __ldg(a.cu + a.B);
  const Raw gk = load_chunks(a.gamma, p, a.gamma != nullptr);
  for (; u < units; u += warps) {
    const int t = static_cast<int>(u / parts), part = static_cast<int>(u % parts);
    const uint16_t* k = a.x[0] + t * a.ldx[0];
    const uint16_t* v0 = a.x[1] + t * a.ldx[1] - static_cast<long long>(a.Hkv) * D;
    int h = part * HW + sub;
    if (t < row0 || t >= row1) continue;  // a padding row
    Raw w = load_chunks((h < a.Hkv ? k : v0) + h * D, p, h < heads);
    const Slot to = find_slot(a, t, lane);
    if (to.row < 0) continue;
    Angles g;
    if (part * HW < a.Hkv) token_angles(g, turns, a.rope, p, l, lane, to.pos, tab[warp]);
    for (int s = part; s < steps; s += parts) {
      const int hn = h + parts * HW;
      const Raw next = load_chunks((hn < a.Hkv ? k : v0) + hn * D, p, hn < heads);
      const bool is_k = h < a.Hkv;
      float v[16];
      norm_rotate<LPH>(w, is_k && a.gamma != nullptr, gk, 1.f / D, a.eps, p, is_k && p.rot, g, v);
      // a block of 32 is four chunks, of two or four lanes: their peaks by way
      // of shared memory; fp32 straight to E4M3, one rounding
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m0 = fmaxf(m0, fabsf(v[i])), m1 = fmaxf(m1, fabsf(v[8 + i]));
      float* pk = peak[warp][sub];
      __syncwarp();  // the last step's have been read
      pk[p.c0 / 8] = m0;
      pk[p.c1 / 8] = m1;
      __syncwarp();
      const float4 q0 = *reinterpret_cast<const float4*>(pk + p.c0 / 32 * 4);
      const float4 q1 = *reinterpret_cast<const float4*>(pk + p.c1 / 32 * 4);
      const uint32_t s0 = ue8m0_from_amax(fmaxf(fmaxf(q0.x, q0.y), fmaxf(q0.z, q0.w)));
      const uint32_t s1 = ue8m0_from_amax(fmaxf(fmaxf(q1.x, q1.y), fmaxf(q1.z, q1.w)));
      const float i0 = inv_scale_from_ue8m0(s0), i1 = inv_scale_from_ue8m0(s1);
      if (h < heads) {
        const long long row = to.row + (static_cast<long long>(is_k ? h : h - a.Hkv) << a.log2P);
        uint8_t* c = (is_k ? a.codes[0] : a.codes[1]) + row * D;
        uint8_t* sc = (is_k ? a.scales[0] : a.scales[1]) + row * (D / 32);
        *reinterpret_cast<uint2*>(c + p.c0) = make_uint2(e4m3x4_code(v[0] * i0, v[1] * i0, v[2] * i0, v[3] * i0),
                                                         e4m3x4_code(v[4] * i0, v[5] * i0, v[6] * i0, v[7] * i0));
        *reinterpret_cast<uint2*>(c + p.c1) =
            make_uint2(e4m3x4_code(v[8] * i1, v[9] * i1, v[10] * i1, v[11] * i1),
                       e4m3x4_code(v[12] * i1, v[13] * i1, v[14] * i1, v[15] * i1));
        if (p.c0 % 32 == 0) sc[p.c0 / 32] = static_cast<uint8_t>(s0);
        if (p.c1 % 32 == 0) sc[p.c1 / 32] = static_cast<uint8_t>(s1);
      }
      w = next;
      h = hn;
    }
  }
}

// Units that share a token's steps: one step each while all of them fit the
// GPU at once (latency), else fewer (a token's sines and cosines are computed
// once a unit).
int token_parts(long long tokens, int steps, int blocks) {
  const long long resident = static_cast<long long>(blocks) * (kRopeThreads / 32);
  int parts = steps;
  while (parts > 1 && tokens * parts > resident) parts = (parts + 1) / 2;
  return parts;
}
unsigned unit_blocks(int units, int blocks) {
  return static_cast<unsigned>(std::min((units - 1) / (kRopeThreads / 32) + 1, blocks));
}

template <int LPH>
cudaError_t norm_rope_lph(const NormRopeArgs& a, int sms, cudaStream_t stream) {
  const int hw = 32 / LPH, steps = (a.H[0] + a.H[1] + hw - 1) / hw;
  const int parts = token_parts(a.T, steps, sms * kRopeBlocks), units = a.T * parts;
  norm_rope_kernel<LPH><<<unit_blocks(units, sms * kRopeBlocks), kRopeThreads, 0, stream>>>(a, parts, units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int sms, cudaStream_t stream) {
  const int lanes = a.D / 16;
  if (lanes <= 2) return norm_rope_lph<2>(a, sms, stream);
  if (lanes <= 4) return norm_rope_lph<4>(a, sms, stream);
  if (lanes <= 8) return norm_rope_lph<8>(a, sms, stream);
  return norm_rope_lph<16>(a, sms, stream);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int sms, cudaStream_t stream) {
  const int steps = (2 * a.Hkv + 3) / 4;
  const int parts = token_parts(a.T, steps, sms * kAppendBlocks), units = a.T * parts;
  const int checks = std::min((a.B - 1) / kRopeThreads + 1, 32);
  const unsigned blocks = unit_blocks(units, sms * kAppendBlocks - checks);  // (all of them resident at once)
  kv_append_kernel<<<blocks + checks, kRopeThreads, 0, stream>>>(a, parts, units, checks);
  return cudaGetLastError();
}

}  // namespace fsops
