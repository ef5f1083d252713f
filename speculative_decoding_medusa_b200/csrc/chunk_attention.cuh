// What the two chunk attention kernels (CUDA cores in fp32, tensor cores in
// bf16) are launched with.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

struct ChunkParams {
  const void* q;
  long long q_stride;
  const void *K, *V;
  const int32_t *table, *cu_q, *kv_len;
  int n_pages, page_size, max_pages;
  int B, T, Hq, Hkv, G;
  float scale;
  void* out;
  int32_t* status;
};

size_t chunk_attention_tc_workspace(int dh);
medusa_status_t chunk_attention_tc(const ChunkParams& p, int dh, void* ws, cudaStream_t stream);

}  // namespace medusa
