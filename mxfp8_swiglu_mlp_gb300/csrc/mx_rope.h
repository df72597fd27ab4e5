// mx_rope.h -- per-head norm with position rotation of queries and keys, and
// the append of new keys and values to the paged MXFP8 cache (mx_rope.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fsops {

// Rotation of the first R dimensions of a head (R a multiple of 32; 0: none).
struct RopeArgs {
  const float* inv_freq;  // [R / 2] radians per position
  int R;
  int interleaved;        // pairs (2 i, 2 i + 1) instead of (i, i + R / 2)
};

struct NormRopeArgs {
  const uint16_t* x[2];      // q, k: row t, head h at t * ld + h * D
  uint16_t* y[2];
  long long ldx[2], ldy[2];
  const uint16_t* gamma[2];  // [D] bf16, null: no norm
  const int32_t* positions;  // [T]
  RopeArgs rope;
  float eps;
  int T, H[2], D;
};

struct KvAppendArgs {
  const uint16_t* x[2];      // k, v
  long long ldx[2];
  const uint16_t* gamma;     // of k, null: no norm
  const int32_t* positions;  // [T] or null: the place in the sequence
  RopeArgs rope;
  float eps;
  uint8_t* codes[2];         // [num_pages, Hkv, P, 128]
  uint8_t* scales[2];        // [num_pages, Hkv, P, 4]
  const int32_t* table;      // [B, max_pages]
  const int32_t* cu;         // [B + 1]
  const int32_t* lens;       // [B]
  uint32_t* status;
  int T, B, Hkv, log2P, num_pages, max_pages;
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendArgs& a, int sms, cudaStream_t stream);

}  // namespace fsops
