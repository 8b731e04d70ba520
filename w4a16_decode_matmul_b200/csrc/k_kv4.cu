// k_kv4.cu -- launchers of the 4-bit key/value cache's kernels: rows in,
// rows out, and attention of a few rows per sequence.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv4_host.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "kv4_prefill.cuh"

namespace wqh {

// k_kv4_prefill.cu
cudaError_t run_kv4_prefill(int head_dim, int group, const wq::kv4::PrefillParams& p,
                            cudaStream_t s);

namespace {

namespace kv4 = wq::kv4;

// Test hooks of the timeout path (wq_internal_kv4_timeout_test).
int g_kv4_stuck_cta = -1;
unsigned int g_kv4_wait_ns = unsigned(wq::kWaitLimitNs);

kv4::Cache device_cache(const wq_kv4_cache& c) {
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

kv4::Batch device_batch(const wq_kv4_batch& b, int page_size) {
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

// Warps per row (each takes up to kRowIterations * 32 pieces of 16 elements),
// and the CTAs that all rows make.
int row_chunks(const wq_kv4_cache& c) {
  const int64_t pieces = int64_t(c.kv_heads) * (c.head_dim / 16);
  const int per_warp = kv4::kRowIterations * 32;
  return int((pieces + per_warp - 1) / per_warp);
}

int64_t row_warps(const wq_kv4_cache& c, int rows) { return int64_t(rows) * row_chunks(c); }

// And some that check the sequences, 32 a warp and at once.
constexpr int kCheckWarps = 1024;

unsigned row_ctas(const wq_kv4_cache& c, const wq_kv4_batch& b) {
  const int64_t warps =
      row_warps(c, b.rows) + std::min<int64_t>((int64_t(b.seqs) + 31) / 32, kCheckWarps);
  return unsigned((warps + kv4::kRowWarps - 1) / kv4::kRowWarps);
}

template <int D, int G>
struct WriteOp {
  static cudaError_t run(const void* K, int64_t ks, const void* V, int64_t vs,
                         const wq_kv4_cache& c, const wq_kv4_batch& b, cudaStream_t s) {
    if (row_warps(c, b.rows) + kCheckWarps >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const kv4::Batch batch = device_batch(b, c.page_size);
    if (batch.status == nullptr) return cudaErrorInitializationError;
    kv4::write_kernel<D, G><<<row_ctas(c, b), kv4::kRowWarps * 32, 0, s>>>(
        static_cast<const __nv_bfloat16*>(K), ks, static_cast<const __nv_bfloat16*>(V), vs,
        device_cache(c), batch, row_chunks(c));
    return cudaGetLastError();
  }
};

template <int D, int G>
struct ReadOp {
  static cudaError_t run(const wq_kv4_cache& c, const wq_kv4_batch& b, void* K, void* V,
                         cudaStream_t s) {
    if (row_warps(c, b.rows) + kCheckWarps >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const kv4::Batch batch = device_batch(b, c.page_size);
    if (batch.status == nullptr) return cudaErrorInitializationError;
    kv4::read_kernel<D, G><<<row_ctas(c, b), kv4::kRowWarps * 32, 0, s>>>(
        device_cache(c), batch, static_cast<__nv_bfloat16*>(K),
        static_cast<__nv_bfloat16*>(V), row_chunks(c));
    return cudaGetLastError();
  }
};

template <int D, int G, int NT, int WARPS, int TILES>
cudaError_t launch_attn(const kv4::AttnParams& p, cudaStream_t s, int sms) {
  using C = kv4::AttnConfig<D, G, NT, WARPS>;
  constexpr size_t smem = C::kOffCtl + C::kCtlBytes;
  static_assert(smem <= 232448, "shared memory of one CTA");
  static int configured[kMaxDevices] = {};
  auto kernel = kv4::attn_kernel<D, G, NT, WARPS, TILES>;
  const cudaError_t e = configure_smem(kernel, configured, smem);
  if (e != cudaSuccess) return e;
  kernel<<<unsigned(std::min(sms, kv4::kMaxCtas)), C::kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

// Warps of a CTA and 16-token tiles per softmax step, by the registers that the
// format needs (12 warps leave 168 a thread, 8 warps 255).  Measured on B200:
//   one block of 8 columns, four groups: one tile 67 us, two (spilling) 118;
//     one or two groups: 58 either way;
//   two blocks of columns, groups of 64, head dim 128: 8 warps 46 us, 12
//     (spilling) 72; head dim 64: 12 warps 34 us, 8 37.  Groups of 32 spill in
//     both of the forms chosen (about 210 and 60 bytes).
// A batch of up to four units of 32 tokens per warp takes 8 warps (one sequence
// of 1,000 tokens, 8 kv heads: 10.1 us, with 12 warps 12.2; of 16,000: 16.7 and
// 16.5); a larger one is limited by how many instructions are in flight (8
// warps 63 us, 12 warps 55).
template <int D, int G>
struct AttnOp {
  static cudaError_t run(const kv4::AttnParams& p, int max_columns, cudaStream_t s, int sms) {
    constexpr int kTiles = D / G == 4 ? 1 : 2;
    if (max_columns > 8) return launch_attn<D, G, 2, D == 64 ? 12 : 8, 1>(p, s, sms);
    const int64_t units =
        int64_t(p.batch.seqs) * p.cache.kv_heads * (p.batch.max_len / kv4::kUnit + 1);
    if (units <= int64_t(4) * 8 * sms) return launch_attn<D, G, 1, 8, kTiles>(p, s, sms);
    return launch_attn<D, G, 1, 12, kTiles>(p, s, sms);
  }
};

kv4::FastDiv fast_div(uint32_t d) {
  uint32_t shift = 0;
  while ((uint64_t(1) << shift) < d) ++shift;
  const uint64_t one = uint64_t(1) << 32;
  return {uint32_t(one * ((uint64_t(1) << shift) - d) / d + 1), shift};
}

// CTAs of the tensor-memory kernel that share a block's tokens: as many as fit
// on the SMs together (each has a slot of the workspace), where that is two or
// more.
int prefill_splits(const wq_kv4_batch& b, int kv_heads, int gqa, int sms) {
  const int64_t blocks = (int64_t(b.rows) * gqa / kv4::kBlockRows + b.seqs) * kv_heads;
  return int(std::max<int64_t>(1, std::min(sms, kv4::kMaxCtas) / blocks));
}

// Measured on B200 (head dim 128), time per cached token: 0.054 ns for each
// block of 16 rows and head in the warp-level kernel (all SMs share them), 17.7
// ns for each wave of CTAs of 256 rows in the tensor-memory kernel, divided by
// its splits.  The constants are used for head dim 64 too.  Where row_starts is
// given the host does not know how the rows are spread, and every sequence counts
// as a block of its own, also those of one row: a chunk of 512 rows beside 127
// single tokens counts as eight waves, though it is one, and goes to the
// warp-level kernel.
bool prefer_prefill(const wq_kv4_batch& b, int kv_heads, int gqa, int sms) {
  const int64_t columns = int64_t(b.rows) * gqa;  // rows times heads of a group
  const int64_t each = b.row_starts ? 0 : columns / b.seqs;
  const auto blocks = [&](int64_t n) {
    return (b.row_starts ? columns / n + b.seqs : (each + n - 1) / n * b.seqs) * kv_heads;
  };
  const int64_t waves = (blocks(kv4::kBlockRows) + sms - 1) / sms;
  return 0.054 * double(blocks(kv4::kMaxRows)) * prefill_splits(b, kv_heads, gqa, sms) >
         17.7 * double(waves);
}

constexpr size_t kCounterBytes = kv4::kMaxCtas * kv4::kMaxRows * 4;

}  // namespace

size_t kv4_workspace_bytes() {
  constexpr size_t few = kv4::AttnConfig<128, 32, 2, 8>::kPartialBytes;
  constexpr size_t many = size_t(kv4::kMaxCtas) * kv4::kBlockRows * (128 + 2) * 4;
  return round_up(kCounterBytes, 256) + std::max(few, many);
}

cudaError_t run_kv4_write(const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                          const wq_kv4_cache& cache, const wq_kv4_batch& batch, cudaStream_t s) {
  return dispatch_kv4<WriteOp>(cache.head_dim, cache.group, K, k_stride, V, v_stride, cache,
                               batch, s);
}

cudaError_t run_kv4_read(const wq_kv4_cache& cache, const wq_kv4_batch& batch, void* K, void* V,
                         cudaStream_t s) {
  return dispatch_kv4<ReadOp>(cache.head_dim, cache.group, cache, batch, K, V, s);
}

cudaError_t run_kv4_attention(const void* Q, int64_t q_stride, int q_heads,
                              const wq_kv4_cache& cache, const wq_kv4_batch& batch, float scale,
                              void* O, int64_t o_stride, void* workspace, cudaStream_t s,
                              const DeviceInfo& dev) {
  kv4::AttnParams p = {};
  p.cache = device_cache(cache);
  p.batch = device_batch(batch, cache.page_size);
  if (p.batch.status == nullptr) return cudaErrorInitializationError;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.q_stride = q_stride;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.o_stride = o_stride;
  p.gqa = q_heads / cache.kv_heads;
  p.by_gqa = fast_div(uint32_t(p.gqa));
  // finite for every finite scale: an infinite one would make NaN of scores of zero
  p.scale_log2 = float(std::clamp(double(scale) * 1.4426950408889634, -double(FLT_MAX),
                                  double(FLT_MAX)));
  p.arrived = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       round_up(kCounterBytes, 256));
  p.test_stuck_cta = g_kv4_stuck_cta;
  p.wait_ns = g_kv4_wait_ns;
  const int64_t max_rows = batch.row_starts ? batch.max_rows : batch.rows / batch.seqs;
  // Sequences with up to 16 rows (times the heads of a group) stream the cache
  // through the warp-level kernel.  With more there is the choice between that
  // kernel, once per 16 rows but spread over every SM, and the tensor-memory
  // kernel, once per 256 rows with a CTA for each.
  constexpr int kFew = kv4::kMaxRows;
  const int64_t bound = max_rows > 0 ? max_rows : batch.rows;
  p.max_columns = 1 << 30;
  if (bound * p.gqa > kFew && prefer_prefill(batch, cache.kv_heads, p.gqa, dev.sms)) {
    kv4::PrefillParams pp = {p, kFew + 1,
                             prefill_splits(batch, cache.kv_heads, p.gqa, dev.sms), p.partial};
    const cudaError_t e = run_kv4_prefill(cache.head_dim, cache.group, pp, s);
    if (e != cudaSuccess || !batch.row_starts) return e;
    p.max_columns = kFew;  // a ragged batch may hold both kinds
  }
  const int max_columns = int(std::min<int64_t>(bound * p.gqa, kFew));
  return dispatch_kv4<AttnOp>(cache.head_dim, cache.group, p, max_columns, s, dev.sms);
}

}  // namespace wqh

extern "C" {

// Test hook, not part of the public ABI: make the timeout path of the attention
// kernels run.  In CTA `stuck_cta` (-1: none) the first warp's copies, or the
// keys of the kernel for many rows, never count as complete; the waits of every
// CTA give up after `wait_ns` nanoseconds (0 restores the default limit).  Every
// copy and product that the CTA starts ends by itself long before.
void wq_internal_kv4_timeout_test(int stuck_cta, unsigned int wait_ns) {
  wqh::g_kv4_stuck_cta = stuck_cta;
  wqh::g_kv4_wait_ns = wait_ns > 0 ? wait_ns : unsigned(wq::kWaitLimitNs);
}

}  // extern "C"
