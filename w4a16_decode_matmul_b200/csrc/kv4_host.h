// kv4_host.h -- launchers of the 4-bit key/value cache's kernels, called by
// the C ABI after its checks of the arguments.
#pragma once

#include "host.h"
#include "wq.h"

namespace wqh {

cudaError_t run_kv4_write(const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                          const wq_kv4_cache& cache, const wq_kv4_batch& batch, cudaStream_t s);
cudaError_t run_kv4_read(const wq_kv4_cache& cache, const wq_kv4_batch& batch, void* K, void* V,
                         cudaStream_t s);
cudaError_t run_kv4_attention(const void* Q, int64_t q_stride, int q_heads,
                              const wq_kv4_cache& cache, const wq_kv4_batch& batch, float scale,
                              void* O, int64_t o_stride, void* workspace, cudaStream_t s,
                              const DeviceInfo& dev);
size_t kv4_workspace_bytes();

// The same over a list of pages for every row and kv head (wq_kv4_select's).  `after`, here
// and below: launched as a programmatic dependent of the kernel before, whose results it
// waits for.
cudaError_t run_kv4_attention_pages(const void* Q, int64_t q_stride, int q_heads,
                                    const wq_kv4_cache& cache, int rows,
                                    const wq_kv4_selection& sel, float scale, void* O,
                                    int64_t o_stride, void* workspace, bool after,
                                    cudaStream_t s, const DeviceInfo& dev);
cudaError_t run_kv4_update_bounds(const wq_kv4_cache& cache, const wq_kv4_bounds& bounds,
                                  const wq_kv4_batch& batch, cudaStream_t s);
cudaError_t run_kv4_select(const void* Q, int64_t q_stride, int q_heads,
                           const wq_kv4_cache& cache, const wq_kv4_bounds& bounds,
                           const wq_kv4_batch& batch, const wq_kv4_selection& sel, bool after,
                           cudaStream_t s, int sms);
// Pages of a sequence and heads of a group that a selection can take.
int64_t kv4_select_max_pages();
int kv4_select_max_group();

// Address of the device status word on the current device (looked up once per
// device); null on failure.
unsigned int* status_address();

}  // namespace wqh
