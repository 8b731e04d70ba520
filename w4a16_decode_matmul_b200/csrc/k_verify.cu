// k_verify.cu -- launcher of the verification of drafted tokens.
#include <algorithm>

#include "kv4_host.h"
#include "verify.cuh"
#include "verify_host.h"

namespace wqh {
namespace {

namespace verify = wq::verify;

// One launch, as a programmatic dependent of the one before where `after` is true, in
// clusters of `cluster` CTAs.
template <class Kernel>
cudaError_t launch_one(Kernel kernel, const verify::Params& p, int64_t ctas, int threads,
                       int cluster, bool after, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {unsigned(cluster), 1, 1};
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, bool LOGITS>
cudaError_t launch(verify::Params p, cudaStream_t s, int sms) {
  constexpr int N = 16 / int(sizeof(T)), kStep = 32 * N;
  // rows that do not begin on a 16-byte boundary have up to N - 1 elements in front
  const int64_t most = int64_t(p.vocab) + N - 1;
  if (LOGITS) {
    const int64_t each = ((most + verify::kTile - 1) / verify::kTile + verify::kPieces - 1) /
                         verify::kPieces;
    p.piece = int(each * verify::kTile);
    const bool aligned =
        p.target_stride % N == 0 && (p.draft == nullptr || p.draft_stride % N == 0);
    p.n_pieces = int(((aligned ? p.vocab : most) + p.piece - 1) / p.piece);
    const int64_t ctas = int64_t(p.n_pieces) * p.rows * (p.draft != nullptr ? 2 : 1);
    if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    verify::stats_kernel<T><<<unsigned(ctas), verify::kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // A cluster a sequence while all are on the GPU at once (two CTAs an SM) and a warp's share
  // of the row is a step or two of its loop; else three kernels.  Measured on B200, rows of 6,
  // cluster and three kernels, us of a captured call: 32,000 binary32 logits, 1 sequence
  // 13.3 and 14.0, 18: 19.9 and 20.7, 32: 26.6 and 29.0, 48: 38.8 and 34.6; 50,021: 17.5 and
  // 15.1, 32.0 and 28.0, 38.7 and 37.2; 131,072: 25.3 and 16.5, 51.1 and 43.1, 68.8 and 63.1,
  // 64: 116 and 103.  (The cluster is two launches less on the host.)
  // bfloat16 logits, 4, 18, 32, 37, 48 sequences: 32,000: 16.6 and 18.7, 22.8 and 24.8, 24.8 and
  // 28.9, 32.0 and 31.0, 38.1 and 34.7; 50,021: 20.5 and 19.3, 29.6 and 26.9, 35.1 and 35.2,
  // 42.1 and 39.2, 51.5 and 42.9.  Probabilities, one launch or three: binary32, 32,000: 8.8 and
  // 10.4, 10.5 and 10.5, 10.4 and 12.5, 14.6 and 12.5, 15.0 and 12.5; 50,021: 14.5 and 10.5, 14.5
  // and 12.5, 14.5 and 12.5, 18.7 and 14.6, 21.0 and 14.6; bfloat16, 32,000: 10.4 and 14.5, 10.5
  // and 14.5, 10.4 and 14.7, 14.6 and 14.6, 15.6 and 14.7; 50,021: within 2 either way up to 37.
  constexpr int kClusterVocab = 40960;
  if (p.vocab <= kClusterVocab && int64_t(p.seqs) * verify::kMaxCluster <= 2 * sms) {
    p.ctas = 1;
    while (p.ctas < verify::kMaxCluster && p.ctas * 4096 < p.vocab) p.ctas *= 2;
    return launch_one(verify::verify_kernel<T, LOGITS, 16>, p, int64_t(p.seqs) * p.ctas, 512,
                      p.ctas, LOGITS, s);
  }
  // Elements of a share: so many that there are 24 warps an SM, since a warp alone is bound by
  // the latency of its exponentials, but not more than 1,024, for the balance of the last
  // ones, nor so few that a sequence has more than its slots of the workspace.
  const auto steps = [](int64_t n) { return (n + kStep - 1) / kStep * kStep; };
  const int64_t even = steps(most * p.seqs / (24 * int64_t(sms)) + 1);
  p.share = int(std::max(std::min<int64_t>(verify::kShareMost, even),
                         steps((most + p.slots - 1) / p.slots)));
  p.n_shares = int((most + p.share - 1) / p.share);
  const int64_t ctas =
      int64_t(p.seqs) * ((p.n_shares + verify::kShareWarps - 1) / verify::kShareWarps);
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  cudaError_t e = launch_one(verify::decide_kernel<T, LOGITS>, p, p.seqs,
                             verify::kDecideWarps * 32, 1, LOGITS, s);
  if (e == cudaSuccess)
    e = launch_one(verify::share_kernel<T, LOGITS>, p, ctas, verify::kShareWarps * 32, 1, true, s);
  if (e == cudaSuccess)
    e = launch_one(verify::find_kernel<T, LOGITS>, p, p.seqs, verify::kFindWarps * 32, 1, true, s);
  return e;
}

// Where the parts of the workspace begin, and how many shares it holds: as many as a row can
// have for the first 1,024 rows, then so many that 16 a row are left -- many sequences fill
// the GPU with few shares each (with 256 for every row it was 12 KB a row, 103 GB at most).
struct Workspace {
  size_t decisions, shares, bytes;
  int64_t slots;
};

Workspace layout(int64_t rows) {
  Workspace w;
  w.slots = std::max(std::min<int64_t>(rows, 1024) * verify::kShares, rows * 16);
  w.decisions = size_t(rows) * 2 * verify::kPieces * sizeof(verify::Piece);
  w.shares = w.decisions + round_up(size_t(rows) * sizeof(verify::Decision), 16);
  w.bytes = w.shares + size_t(w.slots) * sizeof(verify::Share);
  return w;
}

}  // namespace

size_t verify_workspace_bytes(int64_t rows) { return layout(rows).bytes; }

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
  const Workspace w = layout(v.rows);
  unsigned char* const base = static_cast<unsigned char*>(workspace);
  p.pieces = reinterpret_cast<verify::Piece*>(base);
  p.decisions = reinterpret_cast<verify::Decision*>(base + w.decisions);
  p.shares = reinterpret_cast<verify::Share*>(base + w.shares);
  p.slots = int(std::min<int64_t>(verify::kShares, w.slots / std::min(v.rows, v.seqs)));
  p.rows = v.rows;
  p.seqs = v.seqs;
  p.rows_per_seq = v.row_starts ? 0 : v.rows / v.seqs;
  p.vocab = v.vocab;
  p.status = status_address();
  if (p.status == nullptr) return cudaErrorInitializationError;
  const bool logits = (v.flags & WQ_VERIFY_LOGITS) != 0;
  if (v.dtype == WQ_OUT_BF16)
    return logits ? launch<__nv_bfloat16, true>(p, s, sms)
                  : launch<__nv_bfloat16, false>(p, s, sms);
  return logits ? launch<float, true>(p, s, sms) : launch<float, false>(p, s, sms);
}

}  // namespace wqh
