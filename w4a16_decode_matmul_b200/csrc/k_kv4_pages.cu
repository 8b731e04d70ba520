// k_kv4_pages.cu -- launcher of the attention over lists of pages: the kernel of few rows
// per sequence, compiled with a page table for every row and kv head.
#include <algorithm>

#include "kv4_attn_launch.cuh"

namespace wqh {

cudaError_t run_kv4_attention_pages(const void* Q, int64_t q_stride, int q_heads,
                                    const wq_kv4_cache& cache, int rows,
                                    const wq_kv4_selection& sel, float scale, void* O,
                                    int64_t o_stride, void* workspace, bool after,
                                    cudaStream_t s, const DeviceInfo& dev) {
  kv4::AttnParams p = attn_params(Q, q_stride, q_heads, cache, scale, O, o_stride, workspace);
  const wq_kv4_batch each_row = {rows,       rows,      nullptr,
                                 sel.lens,   sel.lists, sel.max_pages,
                                 int64_t(sel.max_pages) * cache.kv_heads, 1};
  p.batch = device_batch(each_row, cache.page_size);
  if (p.batch.status == nullptr) return cudaErrorInitializationError;
  p.head_stride = sel.max_pages;
  return dispatch_kv4<Attn<true>::Op>(cache.head_dim, cache.group, p,
                                      std::min(p.gqa, kv4::kMaxRows), after, s, dev.sms);
}

}  // namespace wqh
