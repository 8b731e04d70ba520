// rotary_host.h -- launchers of the rotary kernels, called by the C ABI after its
// checks of the arguments.
#pragma once

#include "host.h"
#include "wq.h"

namespace wqh {

cudaError_t run_rotary(const void* X, int64_t x_stride, int rows, int heads, int head_dim,
                       const int* positions, const wq_rotary_spec& spec, bool transpose, void* Y,
                       int64_t y_stride, cudaStream_t s, int sms);
cudaError_t run_kv4_write_rotary(const void* Q, int64_t q_stride, int q_heads, void* Q_out,
                                 int64_t qo_stride, const void* K, int64_t k_stride,
                                 const void* V, int64_t v_stride, const wq_rotary_spec& spec,
                                 const int* positions, const wq_kv4_cache& cache,
                                 const wq_kv4_batch& batch, cudaStream_t s, int sms);

}  // namespace wqh
