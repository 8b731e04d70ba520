// k_kv4_prefill.cu -- launcher of the attention kernel for many rows.
//
// Compiled as a whole program: the kernel moves registers between its
// warpgroups, which is ignored in relocatable device code.  So the unit cannot name
// the library's device status word (common.cuh's declaration would define another):
// the kernel gets its address with the batch.
#define g_status g_unused_status
#include "kv4_host.h"
#include "kv4_prefill.cuh"

namespace wqh {
namespace {

namespace kv4 = wq::kv4;

template <int D, int G>
cudaError_t launch(const kv4::PrefillParams& p, cudaStream_t s) {
  using C = kv4::PrefillConfig<D>;
  static int configured[kMaxDevices] = {};
  auto kernel = kv4::prefill_kernel<D, G>;
  const cudaError_t e = configure_smem(kernel, configured, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks =
      (int64_t(p.a.batch.rows) * p.a.gqa / kv4::kBlockRows + p.a.batch.seqs) *
      p.a.cache.kv_heads * p.splits;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  kernel<<<unsigned(blocks), kv4::kPrefillThreads, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t run_kv4_prefill(int head_dim, int group, const kv4::PrefillParams& p,
                            cudaStream_t s) {
  if (head_dim == 64) return group == 32 ? launch<64, 32>(p, s) : launch<64, 64>(p, s);
  return group == 32   ? launch<128, 32>(p, s)
         : group == 64 ? launch<128, 64>(p, s)
                       : launch<128, 128>(p, s);
}

}  // namespace wqh
