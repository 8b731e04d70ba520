// k_kv4_select.cu -- launchers of the kernels that keep bounds of the 4-bit
// cache's pages and choose pages by them.
#include <algorithm>

#include "kv4_launch.cuh"
#include "kv4_select.cuh"

namespace wqh {
namespace {

template <int D, int G>
struct BoundsOp {
  static cudaError_t run(const kv4::BoundsParams& p, cudaStream_t s) {
    const int64_t check = std::min<int64_t>(
        (int64_t(p.batch.seqs) + kv4::kBoundThreads - 1) / kv4::kBoundThreads, 1024);
    const int64_t ctas = int64_t(p.items) * p.cache.kv_heads + check;
    if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    kv4::bounds_kernel<D, G><<<unsigned(ctas), kv4::kBoundThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
};

// CTAs of a cluster: one for each 256 pages that a sequence can have, as long as there is an
// SM for each (128 lists of about 650 pages: 1 CTA each 11.6 us, 2 each 13.3).  The keys'
// shared memory goes by the page table's width, since the lengths are in device memory: 64
// sequences of 250 pages and 8 kv heads take 20.7 us with a table of 250 and 28.9 with one of
// 40,000, which leaves one CTA an SM; up to 16 such sequences there is no difference.
int select_ctas(int64_t width, int64_t units, int sms) {
  int ctas = 1;
  while (ctas < kv4::kMaxCluster && ctas * 256 < width && units * ctas * 2 <= sms) ctas *= 2;
  return ctas;
}

template <int D>
cudaError_t launch_select(kv4::SelectParams p, int64_t width, bool after, cudaStream_t s,
                          int sms) {
  const int64_t units = int64_t(p.rows) * p.kv_heads;
  p.ctas = select_ctas(width, units, sms);
  const size_t smem = round_up(size_t(width) * 4, 16);
  static int configured[kMaxDevices] = {};
  auto kernel = kv4::select_kernel<D>;
  const cudaError_t e = configure_smem(kernel, configured, size_t(kv4::kMaxSelectPages) * 4);
  if (e != cudaSuccess) return e;
  if ((units + 1) * p.ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  // one cluster behind those of the rows checks the sequences
  cfg.gridDim = dim3(unsigned((units + 1) * p.ctas));
  cfg.blockDim = dim3(kv4::kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (p.ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {unsigned(p.ctas), 1, 1};
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

int64_t kv4_select_max_pages() { return kv4::kMaxSelectPages; }

int kv4_select_max_group() { return kv4::kMaxGroupHeads; }

cudaError_t run_kv4_update_bounds(const wq_kv4_cache& cache, const wq_kv4_bounds& bounds,
                                  const wq_kv4_batch& batch, cudaStream_t s) {
  kv4::BoundsParams p = {};
  p.cache = device_cache(cache);
  p.batch = device_batch(batch, cache.page_size);
  if (p.batch.status == nullptr) return cudaErrorInitializationError;
  p.codes = static_cast<int8_t*>(bounds.codes);
  p.grid = static_cast<float*>(bounds.grid);
  const int64_t items = batch.row_starts
                            ? int64_t(batch.rows) / cache.page_size + 2 * int64_t(batch.seqs)
                            : (int64_t(batch.rows) / batch.seqs / cache.page_size + 2) * batch.seqs;
  if (items >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  p.items = int(items);
  return dispatch_kv4<BoundsOp>(cache.head_dim, cache.group, p, s);
}

cudaError_t run_kv4_select(const void* Q, int64_t q_stride, int q_heads,
                           const wq_kv4_cache& cache, const wq_kv4_bounds& bounds,
                           const wq_kv4_batch& batch, const wq_kv4_selection& sel, bool after,
                           cudaStream_t s, int sms) {
  kv4::SelectParams p = {};
  p.batch = device_batch(batch, cache.page_size);
  if (p.batch.status == nullptr) return cudaErrorInitializationError;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.q_stride = q_stride;
  p.codes = static_cast<const int8_t*>(bounds.codes);
  p.grid = static_cast<const float*>(bounds.grid);
  p.pages = cache.pages;
  p.page_shift = device_cache(cache).page_shift;
  p.kv_heads = cache.kv_heads;
  p.gqa = q_heads / cache.kv_heads;
  p.max_pages = sel.max_pages;
  p.first = sel.first;
  p.last = sel.last;
  p.rows = batch.rows;
  p.lists = sel.lists;
  p.lens = sel.lens;
  // what the longest sequence can have
  const int64_t width =
      std::min<int64_t>(batch.table_width, (int64_t(p.batch.max_len) >> p.page_shift) + 1);
  return cache.head_dim == 64 ? launch_select<64>(p, width, after, s, sms)
                              : launch_select<128>(p, width, after, s, sms);
}

}  // namespace wqh
