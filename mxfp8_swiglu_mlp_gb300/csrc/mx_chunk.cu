// mx_chunk.cu -- attention of a chunk of new tokens of each sequence over the
// paged MXFP8 cache.
//
//   out[i, h] = sum_t p[t] V^[t] / sum_t p[t],  p[t] = exp(sm_scale q[i, h] . K^[t] - m)
//   over the tokens t <= pos(i) (and t > pos(i) - window),
// with K^, V^ the dequantised cache and m the running maximum of the row: one
// pass over the keys, the sums rescaled when m grows.
//
//   chunk_kernel  items of 64 rows (tokens x query heads of a KV head) against
//                 64 keys at a time: the block's threads turn the codes into
//                 bf16 in shared memory (exact: an E4M3 value times a power of
//                 two has four significant bits), each warp multiplies 16 rows
//                 with mma.sync, softmax in registers.
//
// p is rounded to bf16 for the second product (relative 2^-8 at most, the
// size of the output's own rounding, and independent from token to token); the
// sum of p that divides the result adds the same rounded values, so a row
// that sees one token returns it exactly.  Scores, maxima and sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "mx_chunk.h"
#include "mx_chunk_plan.cuh"

namespace fsops {

namespace {

constexpr int kTileRows = 64, kTileKeys = 64, kChunkThreads = 128;
constexpr int kD = kChunkD;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ float scale_value(uint32_t s) {  // 2^(s - 127)
  return s != 0 ? __uint_as_float(s << 23) : __uint_as_float(0x00400000u);
}
// Four E4M3 codes times f as two words of bf16 pairs.
__device__ __forceinline__ uint2 dequant4(uint32_t w, float f) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(lo)), y = __half22float2(__half2(hi));
  return make_uint2(bf16x2_rn(x.x * f, x.y * f), bf16x2_rn(y.x * f, y.y * f));
}
// Byte offset of 16-byte piece c of row r in a [rows][128] bf16 tile.
__device__ __forceinline__ int tile_ofs(int r, int c) { return r * 256 + ((c ^ (r & 7)) << 4); }

// 64 tokens from `tok` of KV head hk into a bf16 tile; tokens outside
// [lo, hi) become zeros (what the cache holds there is not read).
__device__ __forceinline__ void load_tile(const ChunkArgs& a, const chunk::Item& w, const uint8_t* codes,
                                          const uint8_t* scales, int tok, uint8_t* tile) {
#pragma unroll
  for (int i = 0; i < kTileKeys * 8 / kChunkThreads; ++i) {
    const int r = (i * kChunkThreads + threadIdx.x) >> 3, c = threadIdx.x & 7;  // 16 codes: pieces 2 c, 2 c + 1
    const int t = tok + r;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    float f = 0.f;
    if (t >= w.lo && t < w.hi) {
      const int page = __ldg(a.table + static_cast<long long>(w.b) * a.max_pages + (t >> a.log2P));
      if (page >= 0 && page < a.num_pages) {
        const long long row = ((static_cast<long long>(page) * a.Hkv + w.hk) << a.log2P) + (t & ((1 << a.log2P) - 1));
        x = __ldg(reinterpret_cast<const uint4*>(codes + row * kD) + c);
        f = scale_value(__ldg(scales + row * (kD / 32) + (c >> 1)));
      } else {
        atomicCAS(a.status, 0u, (1u << 24) | (2u << 16) | (static_cast<uint32_t>(w.b) & 0xFFFFu));
      }
    }
    const uint2 p0 = dequant4(x.x, f), p1 = dequant4(x.y, f), p2 = dequant4(x.z, f), p3 = dequant4(x.w, f);
    *reinterpret_cast<uint4*>(tile + tile_ofs(r, 2 * c)) = make_uint4(p0.x, p0.y, p1.x, p1.y);
    *reinterpret_cast<uint4*>(tile + tile_ofs(r, 2 * c + 1)) = make_uint4(p2.x, p2.y, p3.x, p3.y);
  }
}

__global__ void __launch_bounds__(kChunkThreads) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ __align__(128) uint8_t kt[kTileKeys * 256];
  __shared__ __align__(128) uint8_t vt[kTileKeys * 256];
  __shared__ unsigned long long red[kChunkThreads / 32];
  __shared__ chunk::Item item;
  __shared__ int flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int S = chunk::split_tiles(a, kTileRows, kTileKeys, 4, red);
  chunk::Cursor cur;
  if (warp == 0) cur.init(a, S, kTileRows, kTileKeys, lane);

  for (;;) {
    __syncthreads();  // the previous item and its flag have been read
    if (warp == 0) {
      uint32_t it = 0;
      if (lane == 0) it = atomicAdd(a.work, 1u);
      it = __shfl_sync(0xFFFFFFFFu, it, 0);
      chunk::Item w;
      const bool some = cur.find(a, it, lane, w);
      if (lane == 0) {
        item = w;
        flag = some;
      }
    }
    __syncthreads();
    if (!flag) break;
    const chunk::Item w = item;
    if (w.t0 >= w.t1) continue;
    const int R = w.n * a.G, r0 = w.j * kTileRows, nrows = min(kTileRows, R - r0);
    // the lane's two rows and their last visible token
    int tok[2], pos[2];
    const uint16_t* qp[2];
    bool mine[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * warp + g + 8 * i;
      mine[i] = r < nrows;
      const int rr = r0 + min(r, nrows - 1);
      tok[i] = rr / a.G;
      pos[i] = w.len - w.n + tok[i];
      qp[i] = a.q + static_cast<long long>(w.c0 + tok[i]) * a.ldq + (w.hk * a.G + rr % a.G) * kD;
    }
    uint32_t qf[8][4];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qf[kk][i] = __ldg(reinterpret_cast<const uint32_t*>(qp[i & 1] + 16 * kk + 8 * (i >> 1) + 2 * tq));
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int kti = w.t0; kti < w.t1; ++kti) {
      const int tok0 = kti * kTileKeys;
      __syncthreads();
      load_tile(a, w, a.kc, a.ks, tok0, kt);
      load_tile(a, w, a.vc, a.vs, tok0, vt);
      __syncthreads();
      if (16 * warp >= nrows) continue;
      float s[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          uint32_t b[4];
          ldmatrix_x4(b, kt + tile_ofs(nt * 16 + (lane >> 4) * 8 + (lane & 7), 2 * kk + ((lane >> 3) & 1)));
          mma_bf16(s[2 * nt], qf[kk], b[0], b[1]);
          mma_bf16(s[2 * nt + 1], qf[kk], b[2], b[3]);
        }
      // mask and online softmax; column of s[nt][e]: 8 nt + 2 tq + (e & 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tok0 + 8 * nt + 2 * tq + e;
            float& x = s[nt][2 * i + e];
            const bool seen = t <= pos[i] && (a.window == 0 || t > pos[i] - a.window);
            x = seen ? x * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float mn = fmaxf(m[i], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        const float al = exp2_fast(m[i] - ms);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[nt][2 * i + e];
            x = __bfloat162float(__float2bfloat16_rn(exp2_fast(x - ms)));
            sum += x;
          }
        l[i] = fmaf(l[i], al, sum);
#pragma unroll
        for (int nd = 0; nd < 16; ++nd) {
          o[nd][2 * i] *= al;
          o[nd][2 * i + 1] *= al;
        }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t p[4] = {bf16x2_rn(s[2 * kk][0], s[2 * kk][1]), bf16x2_rn(s[2 * kk][2], s[2 * kk][3]),
                               bf16x2_rn(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                               bf16x2_rn(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
        for (int nd = 0; nd < 8; ++nd) {
          uint32_t b[4];
          ldmatrix_x4_trans(b, vt + tile_ofs(kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * nd + (lane >> 4)));
          mma_bf16(o[2 * nd], p, b[0], b[1]);
          mma_bf16(o[2 * nd + 1], p, b[2], b[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
    }
    if (w.ns == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!mine[i]) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const int rr = r0 + 16 * warp + g + 8 * i;
        uint16_t* y = a.out + static_cast<long long>(w.c0 + tok[i]) * a.ldo + (w.hk * a.G + rr % a.G) * kD + 2 * tq;
#pragma unroll
        for (int nd = 0; nd < 16; ++nd)
          *reinterpret_cast<uint32_t*>(y + 8 * nd) = bf16x2_rn(o[nd][2 * i] * inv, o[nd][2 * i + 1] * inv);
      }
      continue;
    }
    // ---- one of several splits: leave the partial result; the last split to
    // arrive adds them up, always in the splits' order
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!mine[i]) continue;
      const uint32_t rec = w.rec + static_cast<uint32_t>(w.split * nrows + 16 * warp + g + 8 * i);
      float* y = a.rec + static_cast<size_t>(rec) * kD + 2 * tq;
#pragma unroll
      for (int nd = 0; nd < 16; ++nd) *reinterpret_cast<float2*>(y + 8 * nd) = make_float2(o[nd][2 * i], o[nd][2 * i + 1]);
      if (tq == 0) a.rec_ml[rec] = make_float2(m[i], l[i]);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const bool last = atomicAdd(a.groups + w.group, 1u) == static_cast<uint32_t>(w.ns) - 1u;
      if (last) a.groups[w.group] = 0u;
      flag = last;
      __threadfence();
    }
    __syncthreads();
    if (flag) {
      for (int r = 0; r < nrows; ++r) {
        float M = -INFINITY;
        for (int sp = 0; sp < w.ns; ++sp) M = fmaxf(M, __ldcg(&a.rec_ml[w.rec + sp * nrows + r]).x);
        float num = 0.f, den = 0.f;
        for (int sp = 0; sp < w.ns; ++sp) {
          const float2 ml = __ldcg(&a.rec_ml[w.rec + sp * nrows + r]);
          if (ml.x == -INFINITY) continue;
          const float f = exp2_fast(ml.x - M);
          num = fmaf(f, __ldcg(a.rec + static_cast<size_t>(w.rec + sp * nrows + r) * kD + tid), num);
          den = fmaf(f, ml.y, den);
        }
        const int rr = r0 + r;
        const __nv_bfloat16 y = __float2bfloat16_rn(den > 0.f ? num / den : 0.f);
        a.out[static_cast<long long>(w.c0 + rr / a.G) * a.ldo + (w.hk * a.G + rr % a.G) * kD + tid] =
            *reinterpret_cast<const uint16_t*>(&y);
      }
    }
  }
  if (tid == 0) chunk::leave(a);
}

}  // namespace

uint32_t chunk_rec_rows(int T, int Hq, int sms) {
  // few rows: every row in up to two splits for each block of the GPU; many
  // rows: as many splits as 64 K rows of partial results hold (34 MB)
  const long long most = static_cast<long long>(T) * Hq * 2 * sms;
  return static_cast<uint32_t>(most < 65536 ? most : 65536);
}

cudaError_t launch_chunk(const ChunkArgs& args, int sms, cudaStream_t stream) {
  ChunkArgs a = args;
  a.grid = 2 * sms;
  chunk_kernel<<<a.grid, kChunkThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fsops
