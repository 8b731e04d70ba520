// kv4_attn_launch.cuh -- launching the attention of few rows per sequence, shared by the
// units that compile it for page tables of sequences and for lists of every kv head.
#pragma once

#include "kv4_launch.cuh"

namespace wqh {

// The parameters that both forms share (k_kv4.cu).
kv4::AttnParams attn_params(const void* Q, int64_t q_stride, int q_heads,
                            const wq_kv4_cache& cache, float scale, void* O, int64_t o_stride,
                            void* workspace);

template <int D, int G, int NT, int WARPS, int TILES, bool LISTS>
cudaError_t launch_attn(const kv4::AttnParams& p, bool after, cudaStream_t s, int sms) {
  using C = kv4::AttnConfig<D, G, NT, WARPS>;
  constexpr size_t smem = C::kOffCtl + C::kCtlBytes;
  static_assert(smem <= 232448, "shared memory of one CTA");
  static int configured[kMaxDevices] = {};
  auto kernel = kv4::attn_kernel<D, G, NT, WARPS, TILES, LISTS>;
  const cudaError_t e = configure_smem(kernel, configured, smem);
  if (e != cudaSuccess) return e;
  const unsigned ctas = unsigned(std::min(sms, kv4::kMaxCtas));
  if (!LISTS || !after) {
    kernel<<<ctas, C::kThreads, smem, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
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
template <bool LISTS>
struct Attn {
  template <int D, int G>
  struct Op {
    static cudaError_t run(const kv4::AttnParams& p, int max_columns, bool after, cudaStream_t s,
                           int sms) {
      constexpr int kTiles = D / G == 4 ? 1 : 2;
      if (max_columns > 8)
        return launch_attn<D, G, 2, D == 64 ? 12 : 8, 1, LISTS>(p, after, s, sms);
      const int64_t units =
          int64_t(p.batch.seqs) * p.cache.kv_heads * (p.batch.max_len / kv4::kUnit + 1);
      if (units <= int64_t(4) * 8 * sms)
        return launch_attn<D, G, 1, 8, kTiles, LISTS>(p, after, s, sms);
      return launch_attn<D, G, 1, 12, kTiles, LISTS>(p, after, s, sms);
    }
  };
};

}  // namespace wqh
