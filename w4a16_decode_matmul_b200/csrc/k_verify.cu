// k_verify.cu -- launcher of the verification of drafted tokens.
#include <algorithm>

#include "kv4_host.h"
#include "verify.cuh"
#include "verify_host.h"

namespace wqh {
namespace {

namespace verify = wq::verify;

template <typename T>
cudaError_t launch(verify::Params p, bool logits, cudaStream_t s, int sms) {
  constexpr int N = 16 / int(sizeof(T));
  // CTAs of a sequence: one for 4,096 tokens, as long as all are on the GPU at once
  p.ctas = 1;
  while (p.ctas < verify::kMaxCluster && p.ctas * 4096 < p.vocab &&
         int64_t(p.seqs) * p.ctas < 2 * sms)
    p.ctas *= 2;
  const int64_t clusters = int64_t(p.seqs) * p.ctas;
  if (clusters >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  if (logits) {
    // rows that do not begin on a 16-byte boundary have up to N - 1 elements in front
    const int64_t tiles = (int64_t(p.vocab) + N - 1 + verify::kTile - 1) / verify::kTile;
    const int64_t each = (tiles + verify::kPieces - 1) / verify::kPieces;
    p.piece = int(each * verify::kTile);
    const bool aligned = p.target_stride % N == 0 && (p.draft == nullptr || p.draft_stride % N == 0);
    p.n_pieces = int((int64_t(p.vocab) + (aligned ? 0 : N - 1) + p.piece - 1) / p.piece);
    const int64_t ctas = int64_t(p.n_pieces) * p.rows * (p.draft != nullptr ? 2 : 1);
    if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    verify::stats_kernel<T><<<unsigned(ctas), verify::kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters));
  cfg.blockDim = dim3(verify::kSampleThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (p.ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {unsigned(p.ctas), 1, 1};
  }
  if (logits) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  return logits ? cudaLaunchKernelEx(&cfg, verify::verify_kernel<T, true>, p)
                : cudaLaunchKernelEx(&cfg, verify::verify_kernel<T, false>, p);
}

}  // namespace

size_t verify_workspace_bytes(int64_t rows) {
  return size_t(rows) * 2 * verify::kPieces * sizeof(verify::Piece);
}

cudaError_t run_verify_drafts(const wq_verification& v, void* workspace, cudaStream_t s,
                              int sms) {
  verify::Params p = {};
  p.target = v.target;
  p.draft = v.draft;
  p.target_stride = v.target_stride;
  p.draft_stride = v.draft_stride;
  p.tokens = v.tokens;
  p.uniform = v.uniform;
  p.temperature = v.temperature;
  p.row_starts = v.row_starts;
  p.seq_lens = v.out_lens != nullptr ? v.seq_lens : nullptr;
  p.out_tokens = v.out_tokens;
  p.accepted = v.accepted;
  p.out_lens = v.out_lens;
  p.pieces = static_cast<verify::Piece*>(workspace);
  p.rows = v.rows;
  p.seqs = v.seqs;
  p.rows_per_seq = v.row_starts ? 0 : v.rows / v.seqs;
  p.vocab = v.vocab;
  p.status = status_address();
  if (p.status == nullptr) return cudaErrorInitializationError;
  const bool logits = (v.flags & WQ_VERIFY_LOGITS) != 0;
  return v.dtype == WQ_OUT_BF16 ? launch<__nv_bfloat16>(p, logits, s, sms)
                                : launch<float>(p, logits, s, sms);
}

}  // namespace wqh
