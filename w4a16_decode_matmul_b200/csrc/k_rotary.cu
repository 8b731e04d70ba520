// k_rotary.cu -- launchers of the rotary kernels: rows turned where they are or
// into other memory, and on their way into the 4-bit cache.
#include <algorithm>

#include "kv4_launch.cuh"
#include "rotary.cuh"
#include "rotary_host.h"

namespace wqh {
namespace {

namespace rotary = wq::rotary;

rotary::Spec device_spec(const wq_rotary_spec& s) { return {s.freqs, s.dim, s.amplitude}; }

// Rows of a CTA: several as soon as the GPU is full with that many.
int rows_each(int rows, int sms) {
  int each = 1;
  while (each < rotary::kRowsEach && rows >= int64_t(each) * 8 * sms) each *= 2;
  return each;
}

rotary::Units units_of_head(const rotary::Spec& spec, bool interleaved, int head_dim, bool copy) {
  rotary::Units u = {};
  u.turned = interleaved ? (spec.dim + 7) / 8 : spec.dim / 16;
  u.copied = !copy ? 0 : interleaved ? head_dim / 8 - u.turned : (head_dim - spec.dim) / 8;
  u.by_turned = fast_div(uint32_t(std::max(u.turned, 1)));
  u.by_copied = fast_div(uint32_t(std::max(u.copied, 1)));
  return u;
}

cudaError_t launch_rotary(rotary::RotaryParams p, bool interleaved, cudaStream_t s, int sms) {
  // Several rows a CTA as long as their angles fit; where there are fewer rows than SMs a
  // row is spread over several CTAs.
  p.rows_each = std::min(rows_each(p.rows, sms), std::max(1, rotary::kTurns / p.spec.dim));
  const unsigned row_ctas = unsigned((int64_t(p.rows) + p.rows_each - 1) / p.rows_each);
  const int few = std::max(1, 2 * sms / p.rows);
  // (rows of angles lie on 16-byte boundaries where dim is a multiple of 4)
  if (p.spec.dim % (interleaved ? 4 : 16) != 0) {
    const dim3 grid{row_ctas, unsigned(std::min(few, p.heads))};
    rotary::rotary_staged_kernel<<<grid, rotary::kStagedThreads, 0, s>>>(
        p, interleaved, fast_div(uint32_t(p.head_dim / 8)), fast_div(uint32_t(p.heads)));
    return cudaGetLastError();
  }
  p.units = units_of_head(p.spec, interleaved, p.head_dim, p.copy);
  const int per_head = p.units.turned + p.units.copied;
  const int64_t units = int64_t(p.heads) * per_head;
  const int64_t split = std::min<int64_t>(few, (units + 127) / 128);
  const int64_t mine = (units * p.rows_each + split - 1) / split;
  const int64_t rounds = (mine + 511) / 512;
  const int threads = int(((mine + rounds - 1) / rounds + 31) / 32 * 32);
  p.by_row = fast_div(uint32_t(units));
  const dim3 grid{row_ctas, unsigned(split)};
  if (interleaved)
    rotary::rotary_kernel<true><<<grid, threads, 0, s>>>(p);
  else
    rotary::rotary_kernel<false><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D, int G>
struct WriteRotaryOp {
  static cudaError_t run(rotary::WriteParams p, const wq_kv4_cache& c, int interleaved,
                         cudaStream_t s, int sms) {
    p.rows_each = rows_each(p.batch.rows, sms);
    p.chunks = (c.kv_heads * (D / 16) + 31) / 32;
    p.units = units_of_head(p.spec, interleaved, D, p.copy_q);
    const int64_t units = int64_t(p.q_heads) * (p.units.turned + p.units.copied);
    const int64_t share = 32 * rotary::kQueryUnits;
    const int shares = p.chunks + int((units + share - 1) / share);
    const int warps = std::min(shares * p.rows_each, rotary::kWriteWarps);
    // CTAs behind the rows' check the sequences, 32 a warp
    const int64_t check =
        std::min<int64_t>((int64_t(p.batch.seqs) + 32 * warps - 1) / (32 * warps), 1024);
    const unsigned ctas = unsigned((p.batch.rows + p.rows_each - 1) / p.rows_each + check);
    if (interleaved)
      rotary::write_rotary_kernel<D, G, true><<<ctas, warps * 32, 0, s>>>(p, shares);
    else
      rotary::write_rotary_kernel<D, G, false><<<ctas, warps * 32, 0, s>>>(p, shares);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t run_rotary(const void* X, int64_t x_stride, int rows, int heads, int head_dim,
                       const int* positions, const wq_rotary_spec& spec, bool transpose, void* Y,
                       int64_t y_stride, cudaStream_t s, int sms) {
  rotary::RotaryParams p = {};
  p.X = static_cast<const __nv_bfloat16*>(X);
  p.x_stride = x_stride;
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.y_stride = y_stride;
  p.positions = positions;
  p.spec = device_spec(spec);
  p.rows = rows;
  p.heads = heads;
  p.head_dim = head_dim;
  p.copy = X != Y;
  p.sign = transpose ? -1.f : 1.f;
  return launch_rotary(p, spec.interleaved != 0, s, sms);
}

cudaError_t run_kv4_write_rotary(const void* Q, int64_t q_stride, int q_heads, void* Q_out,
                                 int64_t qo_stride, const void* K, int64_t k_stride,
                                 const void* V, int64_t v_stride, const wq_rotary_spec& spec,
                                 const int* positions, const wq_kv4_cache& cache,
                                 const wq_kv4_batch& batch, cudaStream_t s, int sms) {
  rotary::WriteParams p = {};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.q_stride = q_stride;
  p.Q_out = static_cast<__nv_bfloat16*>(Q_out);
  p.qo_stride = qo_stride;
  p.q_heads = q_heads;
  p.copy_q = Q != Q_out;
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.k_stride = k_stride;
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.v_stride = v_stride;
  p.positions = positions;
  p.spec = device_spec(spec);
  p.cache = device_cache(cache);
  p.batch = device_batch(batch, cache.page_size);
  if (p.batch.status == nullptr) return cudaErrorInitializationError;
  return dispatch_kv4<WriteRotaryOp>(cache.head_dim, cache.group, p, cache, spec.interleaved, s,
                                     sms);
}

}  // namespace wqh
