// Arguments of the tensor-core kernel over a shared prefix (kvarn_shared_tc.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kvarn {

struct SharedTcArgs {
  const void* q;  // [token rows][Hq][128]
  float qscale;   // sm_scale log2(e) / sqrt(128)
  int32_t bf16;
  const uint8_t* cache;
  int64_t num_pages;
  const int32_t* table;   // the prefix's pages
  int32_t Hq, Hkv, G;
  int32_t rows_per_head;  // token rows x G
  int32_t N, tiles, tps;  // tile tokens, prefix tiles, tiles per split
  int32_t k_bits, v_bits, scale_bytes;
  int32_t page_bytes, k_part, tile_bytes;
  int32_t ring;           // tiles of pages in shared memory (set by the launch)
  float* ws;              // partials [row][slots]
  int32_t slots;          // splits
  long long wait_limit;   // clock cycles a wait lasts before the kernel gives up
  int32_t withhold;       // diagnostic: every copy is announced this many bytes larger (its phase never completes)
  uint32_t* err;
};

// Splits (and tiles per split) of `units` (KV head, 128 rows) pairs over the
// prefix's tiles; the launch with grid (A.slots, units).
int shared_tc_splits(int units, int tiles, int stages_per_tile, int* tps);
cudaError_t launch_shared_tc(const SharedTcArgs& A, int units, cudaStream_t st);

}  // namespace kvarn
