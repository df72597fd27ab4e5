// mx_chunk.h -- attention of a chunk of new tokens of each sequence over the
// paged MXFP8 cache (mx_chunk.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fsops {

constexpr int kChunkD = 128;            // head dimension
constexpr int kChunkMaxGroup = 64;      // query heads per KV head
constexpr size_t kChunkHeaderBytes = 256;
constexpr uint32_t kChunkMaxGroups = 16384;  // (sequence, query tile, KV head) triples that may be split

struct ChunkArgs {
  const uint16_t* q;          // row t, head h at t * ldq + h * 128
  uint16_t* out;
  long long ldq, ldo;
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* table;       // [B, max_pages]
  const int32_t* cu;          // [B + 1]
  const int32_t* lens;        // [B]
  uint32_t* status;           // first error (status << 24 | site << 16 | sequence)
  uint32_t* work;             // items handed out (zero between calls)
  uint32_t* done;             // blocks that have left (zero between calls)
  uint32_t* groups;           // [kChunkMaxGroups] splits finished (zero between calls)
  float* rec;                 // [rec_rows][128] unnormalised outputs of split rows
  float2* rec_ml;             // [rec_rows] running maximum (base 2) and sum
  uint32_t rec_rows;
  int T, B, Hq, Hkv, G, log2P, num_pages, max_pages, window;
  float scale_log2;           // sm_scale * log2(e)
  int grid;
  uint64_t timeout_ns;
};

// Rows of partial results a call may need (a row is one query token and head).
uint32_t chunk_rec_rows(int T, int Hq, int sms);
cudaError_t launch_chunk(const ChunkArgs& a, int sms, cudaStream_t stream);

}  // namespace fsops
