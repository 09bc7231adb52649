// Host side of the 4-bit cache's operators, for their entry points and for the
// step program's per-op graph.
#pragma once
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "wpk_internal.h"

namespace wpk {

struct Kv4Tensor {  // [token][head][head_dim], strides in elements
  const void* p;
  int64_t token, head;
};

int kv4_view(const wpk_kv4_cache* cache, const int32_t* pos, const int32_t* indptr, int total, int dtype,
             const float* rope, int rope_positions, Kv4Dev* d);
int kv4_append_launch(const Kv4Dev& d, int head_dim, const Kv4Tensor& k, const Kv4Tensor& v, int dtype,
                      const float* rope, cudaStream_t s);
int kv4_attention_launch(const Kv4Dev& d, int head_dim, int max_new, const Kv4Tensor& q, int n_heads, int dtype,
                         const float* rope, float scale, const Kv4Tensor& out, cudaStream_t s);

// Many query rows a kv head (kv4_prefill.cu), kPrefillRows a CTA; the checks are done.
constexpr int kPrefillRows = 128;
cudaError_t kv4_prefill_launch(const Kv4Dev& d, int head_dim, int max_new, const Kv4Tensor& q, int group, int dtype,
                               const float* rope, float scale_log2, const Kv4Tensor& out, cudaStream_t s);

}  // namespace wpk
