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
// turn in integers: inv_freq / 2 pi as a 64-bit fraction of a turn (from fp64,
// relative error 2^-53) times p, the overflow of the product being whole
// turns.  So a position of any size keeps an angle good to 2^-31 turns, where
// the fp32 product p * inv_freq is off by p * 2^-24 radians.
//
// Both kernels move each byte once and are bound by HBM (long inputs) or by
// launch latency (a decode step).  A lane holds 16 consecutive elements of a
// head (two 16-byte loads), so a group of D / 16 lanes holds the head: its
// sum of squares takes log2(lanes) shuffles, the pair partner of a lane in
// the half-split order is the lane R / 32 further, and a 32-element MXFP8
// block is two lanes.  A warp keeps one token's sines and cosines in registers
// over the heads it does.
#include <cuda_bf16.h>

#include "mx_device.cuh"
#include "mx_rope.h"

namespace fsops {

namespace {

constexpr int kRopeThreads = 128;

// Fraction of a turn per position, in units of 2^-64 turns.
__device__ __forceinline__ long long turn_fraction(float inv_freq) {
  double r = static_cast<double>(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
  r -= rint(r);                                                       // whole turns per position
  return __double2ll_rn(r * 18446744073709551616.0);                  // 2^64
}
// sine and cosine of position p's angle.
__device__ __forceinline__ void turn_sincos(long long f, int p, float* sn, float* cs) {
  const unsigned long long turns = static_cast<unsigned long long>(f) * static_cast<unsigned long long>(static_cast<long long>(p));
  // the top 32 bits, signed: [-1/2, 1/2) turns = [-1, 1) half turns
  const float half = static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half, sn, cs);
}

// A lane's place and tables: lane `l` of the head's D / 16.  nf frequencies
// (16 in the half-split order, 8 for adjacent pairs) as sn / cs; `rot` when
// the lane's elements are rotated.
struct LaneRope {
  float sn[16], cs[16];  // adjacent pairs use the first 8
  bool rot;
  int partner;           // lane offset of the pair partner (half-split)
};
__device__ __forceinline__ void load_rope(LaneRope& r, const RopeArgs& a, int l, int pos) {
  r.rot = 16 * l < a.R;
  r.partner = 0;
  if (!r.rot) return;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_sincos(turn_fraction(__ldg(a.inv_freq + 8 * l + i)), pos, &r.sn[i], &r.cs[i]);
  } else {
    const int h = a.R / 32;  // lanes of a half
    const bool second = l >= h;
    r.partner = second ? -h : h;
    const int f0 = 16 * (second ? l - h : l);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      turn_sincos(turn_fraction(__ldg(a.inv_freq + f0 + i)), pos, &r.sn[i], &r.cs[i]);
      if (!second) r.sn[i] = -r.sn[i];  // u' = u cos - w sin, w' = w cos + u sin
    }
  }
}

// The lane's 16 elements (raw bf16) normed and rotated, in fp32.  gw / gp are
// the gains of the lane's and of its partner's elements (bf16 pairs).  Every
// lane of the warp calls it; LPH lanes hold a head.
template <int LPH>
__device__ __forceinline__ void norm_rotate(const uint32_t (&w)[8], bool norm, const uint32_t (&gw)[8],
                                            const uint32_t (&gp)[8], float inv_d, float eps, const LaneRope& r,
                                            bool split, float (&v)[16]) {
  float rn = 1.f;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), fmaf(bf16_hi(w[i]), bf16_hi(w[i]), ss));
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    rn = rsqrtf(fmaf(ss, inv_d, eps));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
    if (norm) {
      v[2 * i] *= rn * bf16_lo(gw[i]);
      v[2 * i + 1] *= rn * bf16_hi(gw[i]);
    }
  }
  if (split) {
    const int src = (threadIdx.x & 31) + r.partner;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t pw = __shfl_sync(0xFFFFFFFFu, w[i], src);
      if (r.rot) {
        float p0 = bf16_lo(pw), p1 = bf16_hi(pw);
        if (norm) {
          p0 *= rn * bf16_lo(gp[i]);
          p1 *= rn * bf16_hi(gp[i]);
        }
        v[2 * i] = fmaf(v[2 * i], r.cs[2 * i], p0 * r.sn[2 * i]);
        v[2 * i + 1] = fmaf(v[2 * i + 1], r.cs[2 * i + 1], p1 * r.sn[2 * i + 1]);
      }
    }
  } else if (r.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = v[2 * i], x = v[2 * i + 1];
      v[2 * i] = fmaf(u, r.cs[i], -x * r.sn[i]);
      v[2 * i + 1] = fmaf(x, r.cs[i], u * r.sn[i]);
    }
  }
}

__device__ __forceinline__ void load16(const uint16_t* p, bool on, uint32_t (&w)[8]) {
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  if (on) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 8);
  }
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Warp (token, part): heads of q (which = 0), then of k (which = 1), 32 / LPH
// at a time; `parts` warps share a token's heads.
template <int LPH>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int parts) {
  constexpr int HW = 32 / LPH;  // heads of a warp step
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const long long wid = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(wid / parts), part = static_cast<int>(wid % parts);
  if (t >= a.T) return;
  const bool on = 16 * l < a.D;
  LaneRope r;
  load_rope(r, a.rope, on ? l : LPH * 1024, __ldg(a.positions + t));
  const bool split = a.rope.R > 0 && !a.rope.interleaved;
  const float inv_d = 1.f / static_cast<float>(a.D);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int steps = (a.H[which] + HW - 1) / HW;
    if (steps == 0) continue;
    const bool norm = a.gamma[which] != nullptr;
    uint32_t gw[8], gp[8];
    load16(a.gamma[which] + 16 * l, norm && on, gw);
    load16(a.gamma[which] + 16 * (l + r.partner), norm && on, gp);
    const uint16_t* x = a.x[which] + static_cast<long long>(t) * a.ldx[which] + 16 * l;
    uint16_t* y = a.y[which] + static_cast<long long>(t) * a.ldy[which] + 16 * l;
    for (int s = part; s < steps; s += parts) {
      const int h = s * HW + sub;
      const bool mine = on && h < a.H[which];
      uint32_t w[8];
      load16(x + h * a.D, mine, w);
      float v[16];
      norm_rotate<LPH>(w, norm, gw, gp, inv_d, a.eps, r, split, v);
      if (mine) {
        uint4* d = reinterpret_cast<uint4*>(y + h * a.D);
        d[0] = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
        d[1] = make_uint4(bf16x2_rn(v[8], v[9]), bf16x2_rn(v[10], v[11]), bf16x2_rn(v[12], v[13]),
                          bf16x2_rn(v[14], v[15]));
      }
    }
  }
}

// The sequence that holds row t: the largest b < B with cu[b] <= t, or -1
// when t lies before the first or behind the last sequence.  A warp narrows
// the range 32-fold a step.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
  if (t >= __ldg(cu + B) || t < __ldg(cu)) return -1;
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

// Warp (token, part): the KV heads of k (which = 0), then of v.
__global__ void __launch_bounds__(kRopeThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int parts) {
  constexpr int D = 128, LPH = 8, HW = 4;
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const long long wid = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(wid / parts), part = static_cast<int>(wid % parts);
  if (t >= a.T) return;
  const int b = find_sequence(a.cu, a.B, t, lane);
  if (b < 0) return;  // a padding row
  const int place = __ldg(a.lens + b) - (__ldg(a.cu + b + 1) - t);  // lens[b] - n + (t - cu[b])
  if (place < 0 || (place >> a.log2P) >= a.max_pages) {
    if (lane == 0) report(a.status, 1u, 1u, b);
    return;
  }
  const int page = __ldg(a.table + static_cast<long long>(b) * a.max_pages + (place >> a.log2P));
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) report(a.status, 1u, 2u, b);
    return;
  }
  const int P = 1 << a.log2P, slot = place & (P - 1);
  LaneRope r;
  const int steps = (a.Hkv + HW - 1) / HW;
  const bool split = a.rope.R > 0 && !a.rope.interleaved;
  if (part < steps)
    load_rope(r, a.rope, l, a.positions != nullptr ? __ldg(a.positions + t) : place);
  else
    r.rot = false, r.partner = 0;
  const bool norm = a.gamma != nullptr;
  uint32_t gw[8], gp[8];
  load16(a.gamma + 16 * l, norm, gw);
  load16(a.gamma + 16 * (l + r.partner), norm, gp);
  for (int s = part; s < 2 * steps; s += parts) {
    const int which = s >= steps, h = (which ? s - steps : s) * HW + sub;
    const bool mine = h < a.Hkv;
    uint32_t w[8];
    load16(a.x[which] + static_cast<long long>(t) * a.ldx[which] + h * D + 16 * l, mine, w);
    float v[16];
    if (which == 0) {
      norm_rotate<LPH>(w, norm, gw, gp, 1.f / D, a.eps, r, split, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    }
    // the MXFP8 block of lanes l and l ^ 1; fp32 straight to E4M3, one rounding
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    const uint32_t sc = ue8m0_from_amax(amax);
    const float inv = inv_scale_from_ue8m0(sc);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x4_code(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    // the head's four scale bytes in one word
    uint32_t sw = sc << (8 * (l >> 1));
    sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 2);
    sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 4);
    if (mine) {
      const long long row = (static_cast<long long>(page) * a.Hkv + h) * P + slot;
      *reinterpret_cast<uint4*>(a.codes[which] + row * D + 16 * l) = make_uint4(c[0], c[1], c[2], c[3]);
      if (l == 0) *reinterpret_cast<uint32_t*>(a.scales[which] + row * (D / 32)) = sw;
    }
  }
}

// Warps that share a token's `steps` warp steps: one step a warp while all of
// them fit the GPU at once (latency), the whole token in one warp when there
// are tokens enough (its sines and cosines are computed once).
int token_parts(long long tokens, int steps, int sms) {
  const long long resident = static_cast<long long>(sms) * 16;
  int parts = steps;
  while (parts > 1 && tokens * parts > resident) parts = (parts + 1) / 2;
  return parts;
}

template <int LPH>
cudaError_t norm_rope_lph(const NormRopeArgs& a, int sms, cudaStream_t stream) {
  const int hw = 32 / LPH;
  const int steps = (a.H[0] + hw - 1) / hw > (a.H[1] + hw - 1) / hw ? (a.H[0] + hw - 1) / hw : (a.H[1] + hw - 1) / hw;
  const int parts = token_parts(a.T, steps, sms);
  const long long warps = static_cast<long long>(a.T) * parts;
  norm_rope_kernel<LPH><<<static_cast<unsigned>((warps + 3) / 4), kRopeThreads, 0, stream>>>(a, parts);
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
  const int steps = 2 * ((a.Hkv + 3) / 4);
  const int parts = token_parts(a.T, steps, sms);
  const long long warps = static_cast<long long>(a.T) * parts;
  kv_append_kernel<<<static_cast<unsigned>((warps + 3) / 4), kRopeThreads, 0, stream>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace fsops
