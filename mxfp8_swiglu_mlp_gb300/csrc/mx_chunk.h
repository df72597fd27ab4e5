// mx_chunk.h -- attention of a chunk of new tokens of each sequence over the
// paged MXFP8 cache (mx_chunk.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fsops {

constexpr int kChunkD = 128;            // head dimension
constexpr int kChunkMaxGroup = 64;      // query heads per KV head
constexpr int kChunkFewRows = 32;       // rows of a query tile of the kernel for few rows
constexpr size_t kChunkHeaderBytes = 256;
constexpr int kChunkCounters = 8;       // of a block: parts of a query tile that have arrived, by warp or stream
constexpr size_t kChunkCounterBytes = 256 * kChunkCounters * sizeof(uint32_t);  // blocks <= 256

struct ChunkArgs {
  const uint16_t* q;          // row t, head h at t * ldq + h * 128
  uint16_t* out;
  long long ldq, ldo;
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* table;       // [B, max_pages]
  const int32_t* cu;          // [B + 1]
  const int32_t* lens;        // [B]
  uint32_t* status;           // first error (status << 24 | site << 16 | sequence)
  uint32_t* count;            // [grid][kChunkCounters] (zero between calls)
  float* rec;                 // [2 * grid] unnormalised outputs of parts: [128][slot_rows], for few rows [slot_rows][128]
  float2* rec_ml;             // [2 * grid][slot_rows] running maximum (base 2) and sum
  int slot_rows;
  int T, B, Hq, Hkv, G, log2P, num_pages, max_pages, window;
  float scale_log2;           // |sm_scale| * log2(e)
  int negate;                 // sm_scale < 0: q enters with its sign turned
  int tile_rows;              // rows of a query tile: 256, or kChunkFewRows for the kernel for few rows
  int grid;
  uint32_t tries;             // of a wait before it gives up
  uint32_t extra_arrivals;    // test hook: arrivals more than any product makes when a tile's outputs are done
};

// Rows of a query tile for T rows of B sequences in groups of G heads.
int chunk_tile_rows(int T, int B, int G);
// Partial-result slots of a call and their rows.
inline int chunk_slots(int sms) { return 2 * sms; }
inline int chunk_slot_rows(int T, int G, int tile_rows) {
  const long long r = static_cast<long long>(T) * G;
  return r < tile_rows ? static_cast<int>(r) : tile_rows;
}
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_few(const ChunkArgs& a, cudaStream_t stream);

}  // namespace fsops
