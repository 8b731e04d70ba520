// kv4_launch.cuh -- what the launchers of the 4-bit cache's kernels share: the
// kernels' view of a cache and a batch, and the choice of a format.
#pragma once

#include <algorithm>

#include "kv4_host.h"
#include "kv4_attn.cuh"

namespace wqh {

namespace kv4 = wq::kv4;

inline kv4::Cache device_cache(const wq_kv4_cache& c) {
  kv4::Cache d = {};
  d.k_codes = static_cast<uint8_t*>(c.k_codes);
  d.k_meta = static_cast<__half2*>(c.k_meta);
  d.v_codes = static_cast<uint8_t*>(c.v_codes);
  d.v_meta = static_cast<__half2*>(c.v_meta);
  d.pages = c.pages;
  while ((1 << d.page_shift) < c.page_size) ++d.page_shift;
  d.kv_heads = c.kv_heads;
  return d;
}

inline kv4::Batch device_batch(const wq_kv4_batch& b, int page_size) {
  kv4::Batch d = {};
  d.row_starts = b.row_starts;
  d.seq_lens = b.seq_lens;
  d.page_table = b.page_table;
  d.table_stride = b.table_stride;
  d.seqs = b.seqs;
  d.rows = b.rows;
  d.rows_per_seq = b.row_starts ? 0 : b.rows / b.seqs;
  d.max_len = int(std::min<int64_t>(int64_t(b.table_width) * page_size, 0x7fffff00));
  d.status = status_address();
  return d;
}

// Calls every (head dim, group) the cache supports through F<D, G>::run.
template <template <int, int> class F, typename... Args>
cudaError_t dispatch_kv4(int head_dim, int group, const Args&... args) {
#define WQ_CASE(D, G) \
  if (head_dim == D && group == G) return F<D, G>::run(args...);
  WQ_CASE(64, 32) WQ_CASE(64, 64)
  WQ_CASE(128, 32) WQ_CASE(128, 64) WQ_CASE(128, 128)
#undef WQ_CASE
  return cudaErrorInvalidValue;
}

inline kv4::FastDiv fast_div(uint32_t d) {
  uint32_t shift = 0;
  while ((uint64_t(1) << shift) < d) ++shift;
  const uint64_t one = uint64_t(1) << 32;
  return {uint32_t(one * ((uint64_t(1) << shift) - d) / d + 1), shift};
}

// Warps per row (each takes up to kRowIterations * 32 pieces of 16 elements),
// and the CTAs that all rows make.
inline int row_chunks(const wq_kv4_cache& c) {
  const int64_t pieces = int64_t(c.kv_heads) * (c.head_dim / 16);
  const int per_warp = kv4::kRowIterations * 32;
  return int((pieces + per_warp - 1) / per_warp);
}

}  // namespace wqh
