// Launch descriptor of the cache append kernel (append.cu).
#pragma once

#include "common.cuh"

namespace da {

struct AppendLaunch {
  const void* k_new;
  const void* v_new;  // null: shared latent
  const void* q_new;  // null: no queries
  long long k_stride, v_stride, q_stride;  // elements between tokens
  const int32_t* positions;
  const int32_t* rows;  // null: token i is row i
  const int32_t* table;
  void* k;
  void* v;
  __nv_bfloat16* q_out;
  int32_t* err;
  const float* inv_freq;
  long long num_blocks;
  long long kv_rows;  // entries in a cache (NVFP4: its block scales follow its codes)
  int n_tokens, x_bf16, B, H_q, H_kv, D;
  int layout, page_size, width, kv_type;
  long long capacity;
  int rope_dim, rope_offset, interleaved;
  float gain, k_scale, v_scale;
};

cudaError_t launch_append(const AppendLaunch& p, int sms, cudaStream_t stream);

}  // namespace da
