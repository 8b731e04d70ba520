// verify.cuh -- verification of drafted tokens against the target's distribution.
//
// Mathematics ("vLLM 量化与推测解码", speculative decoding: a = min(1, p/q), residual
// max(p - q, 0)).  A sequence's rows hold the tokens fed to the target: row 0 a token
// that stands, rows 1 .. T - 1 drafts.  Draft row i is accepted while
//   u_i q_i(x_i) < p_{i-1}(x_i),
// p_{i-1} the target's distribution behind row i - 1, q_i the one x_i was drawn from.
// Behind a accepted drafts one token is sampled: from max(p_a - q_{a+1}, 0) where a
// draft was rejected, from p_a where none was, by u_0: the first token whose running
// sum passes u_0 times the whole.
//
// Precision.  That token is an integer, decided by a running sum over the vocabulary.
// An error of e in every mass, of either sign, puts a boundary off by e times the root
// of the masses' squares' sum, about e / 20, so that about vocabulary e / 20 of all
// numbers u_0 lead to a neighbour: one in a hundred with binary32's exponentials,
// one in 10^9 with those below.  An error of the sums that p and q are divided by
// moves all boundaries of max(p - q, 0) at once and costs twenty times as much.  So the
// sampled row's (and its draft row's) masses and sums are in binary64, exponentials
// within 2^-43.  A draft's acceptance has one border: there the sums of exponentials
// are binary32's, added in binary64 from 32 terms on, off by some 10^-7.
//
// Two kernels.  Logits first go through stats_kernel: largest logit and sum of
// exponentials of every piece of every row, which reads each row once.  verify_kernel,
// a cluster per sequence, joins the pieces, accepts, and samples: where max(p - q, 0)
// is needed it forms the two rows' sums again in binary64, then each warp sums its share
// of the masses, and the warp in whose share the number falls looks for the token.
// Probabilities need no statistics and no first kernel.
#pragma once

#include "common.cuh"

namespace wq {
namespace verify {

constexpr int kPieces = 64;      // of a row, at most: slots of the workspace
constexpr int kThreads = 256;    // of stats_kernel
constexpr int kPerThread = 32;   // elements of a thread in registers
constexpr int kTile = kThreads * kPerThread;
constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 8;

struct Piece {
  double sum;  // of exp((x - top) / temperature)
  float top;   // largest logit; -inf: no mass
  int first;   // where it is first
};

struct Params {
  const void *target, *draft;        // [rows][vocab]; draft null: the drafted token has all of it
  int64_t target_stride, draft_stride;
  const int* tokens;                 // [rows]
  const float* uniform;              // [rows]
  const float* temperature;          // [seqs] or null (1)
  const int* row_starts;             // [seqs + 1] or null: rows_per_seq each
  const int* seq_lens;               // [seqs] or null
  int *out_tokens, *accepted, *out_lens;
  Piece* pieces;                     // [2][rows][kPieces]: target, draft
  int rows, seqs, rows_per_seq, vocab;
  int piece;                         // elements of a piece
  int n_pieces, ctas;
  unsigned int* status;
};

// Rows of sequence b, inside the batch whatever row_starts holds.
struct Rows {
  int first, count;
};

__device__ __forceinline__ Rows load_rows(const Params& p, int b) {
  if (p.row_starts == nullptr) return {b * p.rows_per_seq, p.rows_per_seq};
  const int r0 = p.row_starts[b], r1 = p.row_starts[b + 1];
  const int first = min(max(r0, 0), p.rows), end = min(max(r1, first), p.rows);
  if (first != r0 || end != r1) record_status(1u, p.status);
  return {first, end - first};
}

// ---- exponentials.  exp(d / temperature) = 2^(k/64) 2^(r/64), |r| <= 1/2: the table's
// 2^((k mod 64)/64), shared memory, times the exponent k div 64 and the series of 2^(r/64)
// to r^4: the next term is (r ln 2 / 64)^5 / 120 < 2^-44.  Table-driven exponentials:
// P. T. P. Tang, ACM TOMS 15 (1989).
struct Exp {
  const double* table;  // 2^(j/64)
  double scale;         // 64 log2(e) / temperature
  double top;           // the largest logit
  float cut;            // logits below it (or NaN) have no mass: less than 2^-995 of the largest's
  __device__ __forceinline__ double operator()(float x) const {
    const double d = double(fmaxf(x, cut)) - top;
    const double magic = 6755399441055744.0;  // 1.5 * 2^52: rounds to an integer, the low word
    const double shifted = fma(d, scale, magic);
    const int k = __double2loint(shifted);
    const double r = fma(d, scale, magic - shifted);
    constexpr double c = 0.6931471805599453 / 64;  // ln 2 / 64
    double e = fma(r, c * c * c * c / 24, c * c * c / 6);
    e = fma(e, r, c * c / 2);
    e = fma(e, r, c);
    const double base = table[k & 63];
    e = fma(e * r, base, base);
    const double y =
        __hiloint2double(__double2hiint(e) + (k & ~63) * (1 << 14), __double2loint(e));
    return x >= cut ? y : 0.0;
  }
};

__device__ __forceinline__ Exp make_exp(const double* table, float top, float hot) {
  const float cut = fmaxf(top - 690.f * hot, -3.4028234e38f);
  return {table, 64 * 1.4426950408889634 / double(hot), double(top), cut};
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < 64) table[threadIdx.x] = exp2(double(threadIdx.x) * (1.0 / 64));
}

// A distribution over one row.  kShared: all logits of +infinity have the same mass.
struct Mass {
  enum Kind { kNone, kProbabilities, kLogits, kShared, kOne };
  Kind kind;
  int one;         // kOne: the token that has all
  double inverse;  // of the sum
  Exp exp;
  __device__ __forceinline__ double operator()(float x, int i) const {
    if (kind == kProbabilities) return x > 0.f ? double(x) : 0.0;
    if (kind == kLogits) return exp(x) * inverse;
    if (kind == kShared) return x == INFINITY ? inverse : 0.0;
    return kind == kOne && i == one ? 1.0 : 0.0;
  }
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// Sixteen bytes of elements `at` .. of a row, as floats; where they are not aligned or reach
// out of [0, end), element by element, `none` outside.
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* row, int64_t at, int64_t end, float none,
                                         float (&x)[N]) {
  static_assert(N * sizeof(T) == 16, "");
  const T* from = row + at;
  if (at >= 0 && at + N <= end && (reinterpret_cast<uintptr_t>(from) & 15u) == 0) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = at + i >= 0 && at + i < end ? to_float(from[i]) : none;
  }
}

// Elements from the last 16-byte boundary to a row's first element.
template <typename T>
__device__ __forceinline__ int row_lead(const T* row) {
  return int(uint32_t(reinterpret_cast<uintptr_t>(row)) & 15u) / int(sizeof(T));
}

// Largest logit of a piece of a row, and the sum of exponentials relative to it.
// Pieces begin on 16-byte boundaries: the first at the last boundary before the row,
// with nothing in front of it.  All of a thread's loads are in flight at once, and its
// elements stay in registers from the maximum to the sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) stats_kernel(const Params p) {
  constexpr int N = 16 / int(sizeof(T)), kRuns = kPerThread / N;
  __shared__ double sums[kThreads / 32];
  __shared__ float tops[kThreads / 32];
  __shared__ int firsts[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int index = int(blockIdx.x) / p.n_pieces, piece = int(blockIdx.x) - index * p.n_pieces;
  const bool is_draft = index >= p.rows;
  const int r = is_draft ? index - p.rows : index;
  // ---- the row's sequence: its temperature, and whether the row is needed
  int b = 0;
  if (p.row_starts == nullptr) {
    b = r / p.rows_per_seq;
  } else {
    int lo = 0, n = p.seqs + 1;
    if (p.row_starts[0] > r) return;
    while (n > 1) {
      const int step = (n + 32) / 33;
      const int at = lo + (lane + 1) * step;
      const bool below = at < lo + n && p.row_starts[at] <= r;
      // (the first that is not, so that a bad range does not move the rows before it)
      const unsigned beyond = ~__ballot_sync(0xffffffffu, below);
      const int skip = beyond ? __ffs(beyond) - 1 : 32;
      lo += skip * step;
      n = min(step, n - skip * step);
    }
    if (lo >= p.seqs) return;
    b = lo;
  }
  const float hot = p.temperature != nullptr ? p.temperature[b] : 1.f;
  const bool greedy = !(hot > 0.f);
  if (is_draft) {
    const int first = p.row_starts != nullptr ? p.row_starts[b] : b * p.rows_per_seq;
    if (greedy || r <= first) return;  // not a draft, or its distribution is not looked at
  }
  const T* const row = is_draft ? static_cast<const T*>(p.draft) + int64_t(r) * p.draft_stride
                                : static_cast<const T*>(p.target) + int64_t(r) * p.target_stride;
  const int64_t begin = int64_t(piece) * p.piece - row_lead(row);
  const int64_t end = min(begin + p.piece, int64_t(p.vocab));
  // log2(e) / temperature in two parts: a binary32 product would be off by 2^-24 of the
  // exponent, for all terms in the same direction
  const double log2_unit = fmin(fmax(1.4426950408889634 / double(hot), 1e-30), 1e30);
  const float unit = float(log2_unit), unit_low = float(log2_unit - double(unit));
  const float lowest = -200.f / unit;  // 2^-200: nothing in binary32
  double sum = 0.0;
  float top = -INFINITY;
  int first = 0x7fffffff;
  for (int64_t tile = begin; tile < end; tile += kTile) {
    float x[kRuns][N];
#pragma unroll
    for (int k = 0; k < kRuns; ++k)
      load_run<T, N>(row, tile + (k * kThreads + tid) * N, end, -INFINITY, x[k]);
    float high = -INFINITY;
#pragma unroll
    for (int k = 0; k < kRuns; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) high = fmaxf(high, x[k][i]);
    if (greedy) {
      if (high > top) {
        top = high;
#pragma unroll
        for (int k = kRuns - 1; k >= 0; --k)
#pragma unroll
          for (int i = N - 1; i >= 0; --i)
            if (x[k][i] == high) first = int(tile + (k * kThreads + tid) * N + i);
      }
      continue;
    }
    // each thread relative to its own largest
    if (fmaxf(top, high) == -INFINITY) continue;
    if (high > top) {
      sum *= double(exp2_approx(fmaxf(top - high, lowest) * unit));
      top = high;
    }
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    if (top == INFINITY) {
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i & 3] += x[k][i] == INFINITY ? 1.f : 0.f;
    } else {
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float d = fmaxf(x[k][i] - top, lowest);
          const float e = exp2_approx(fmaf(d, unit, d * unit_low));
          part[i & 3] += x[k][i] >= -3.4028234e38f ? e : 0.f;
        }
    }
    sum += double((part[0] + part[1]) + (part[2] + part[3]));
  }
  // ---- the CTA's
  float high = top;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, m));
  if (lane == 0) tops[warp] = high;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) high = fmaxf(high, tops[w]);
  int at = top == high ? first : 0x7fffffff;
  if (top != high) sum *= double(exp2_approx(fmaxf(top - high, lowest) * unit));
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    at = min(at, __shfl_xor_sync(0xffffffffu, at, m));
  }
  if (lane == 0) sums[warp] = sum, firsts[warp] = at;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) {
      sum += sums[w];
      at = min(at, firsts[w]);
    }
    p.pieces[int64_t(index) * kPieces + piece] = {sum, high, at};
  }
}

// The distribution of a row from its pieces, by all lanes of a warp.
__device__ __forceinline__ Mass join_pieces(const Params& p, bool is_draft, int r, float hot,
                                            const double* table, int lane) {
  const Piece* from = p.pieces + (int64_t(is_draft ? p.rows : 0) + r) * kPieces;
  Piece mine[kPieces / 32];
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kPieces / 32; ++k) {
    const int i = lane + 32 * k;
    mine[k] = {0.0, -INFINITY, 0x7fffffff};
    if (i < p.n_pieces) {
      mine[k].sum = __ldcg(&from[i].sum);
      mine[k].top = __ldcg(&from[i].top);
      mine[k].first = __ldcg(&from[i].first);
    }
    top = fmaxf(top, mine[k].top);
  }
#pragma unroll
  for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  const Exp exp = make_exp(table, top, hot);
  double sum = 0.0;
  int first = 0x7fffffff;
#pragma unroll
  for (int k = 0; k < kPieces / 32; ++k) {
    if (mine[k].top == top) {
      first = min(first, mine[k].first);
      sum += mine[k].sum;
    } else if (hot > 0.f) {
      sum += mine[k].sum * exp(mine[k].top);
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    first = min(first, __shfl_xor_sync(0xffffffffu, first, m));
  }
  if (top == -INFINITY) return {Mass::kNone, -1, 0.0, exp};
  if (!(hot > 0.f)) return {Mass::kOne, first, 1.0, exp};
  return {top == INFINITY ? Mass::kShared : Mass::kLogits, -1, 1.0 / sum, exp};
}

// A uniform number as it is used: inside [0, 1), a NaN as 0.
__device__ __forceinline__ double uniform_of(float u) {
  return double(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
}

// The first of N shares, which begin at `from`, whose end is beyond `wanted`; the last
// with any mass if none is.
template <int N, typename Sum>
__device__ __forceinline__ int owner_of(double wanted, double from, Sum sum) {
  int owner = -1, last = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double s = sum(i);
    if (s > 0.0) last = i;
    from += s;
    if (owner < 0 && s > 0.0 && from > wanted) owner = i;
  }
  return owner < 0 ? last : owner;
}

__device__ __forceinline__ double ld_dsmem_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// One sequence a cluster.  Every CTA decides the drafts for itself (a warp a draft,
// a few numbers each), then sums its share of the vocabulary.
template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kSampleThreads) verify_kernel(const Params p) {
  constexpr int N = 16 / int(sizeof(T));
  __shared__ double table[64];
  // sums of the warps' shares, and of the CTA's: of both rows, of the masses that are
  // left, of the target's
  __shared__ double sums[4][kSampleWarps], cta_sum[4];
  __shared__ int rejected;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  const int b = int(blockIdx.x) / p.ctas;
  const Rows rows = load_rows(p, b);
  if (rows.count == 0) {
    if (rank == 0 && tid == 0) {
      p.accepted[b] = 0;
      if (p.out_lens != nullptr) p.out_lens[b] = p.seq_lens[b];
    }
    return;
  }
  if (LOGITS) fill_table(table);
  if (tid == 0) rejected = rows.count - 1;
  const float hot = LOGITS && p.temperature != nullptr ? p.temperature[b] : 1.f;
  const bool greedy = !(hot > 0.f);
  const Exp no_exp = {};
  __syncthreads();
  if (LOGITS) grid_dependency_wait();

  auto target_row = [&](int r) { return static_cast<const T*>(p.target) + r * p.target_stride; };
  auto draft_row = [&](int r) { return static_cast<const T*>(p.draft) + r * p.draft_stride; };
  auto target_mass = [&](int r) -> Mass {
    if (!LOGITS) return {Mass::kProbabilities, -1, 1.0, no_exp};
    return join_pieces(p, false, r, hot, table, lane);
  };
  auto draft_mass = [&](int r, int token) -> Mass {
    if (p.draft == nullptr) return {Mass::kOne, token, 1.0, no_exp};
    if (!LOGITS) return {Mass::kProbabilities, -1, 1.0, no_exp};
    // greedy: whatever the draft's distribution, the token is accepted if it is the
    // target's, and what is left is the target's
    if (greedy) return {Mass::kOne, token, 1.0, no_exp};
    return join_pieces(p, true, r, hot, table, lane);
  };

  // ---- drafts
  for (int i = 1 + warp; i < rows.count; i += kSampleWarps) {
    const int r = rows.first + i, token = p.tokens[r];
    bool accept = false;
    if (token >= 0 && token < p.vocab) {
      const Mass target = target_mass(r - 1), draft = draft_mass(r, token);
      const double judged = target(to_float(target_row(r - 1)[token]), token);
      const double drawn =
          draft(draft.kind == Mass::kOne ? 0.f : to_float(draft_row(r)[token]), token);
      accept = uniform_of(p.uniform[r]) * drawn < judged;
    }
    if (!accept && lane == 0) atomicMin(&rejected, i - 1);
  }
  __syncthreads();
  const int a = rejected, at = rows.first + a;
  const bool refused = a < rows.count - 1;
  if (rank == 0) {
    for (int i = tid; i < rows.count; i += kSampleThreads)
      if (i != a) p.out_tokens[rows.first + i] = i < a ? p.tokens[rows.first + i + 1] : -1;
    if (tid == 0) {
      p.accepted[b] = a;
      if (p.out_lens != nullptr) p.out_lens[b] = p.seq_lens[b] - (rows.count - 1 - a);
    }
  }

  // ---- the token behind them
  Mass target = target_mass(at);
  if (target.kind == Mass::kNone || target.kind == Mass::kOne) {
    if (rank == 0 && tid == 0) p.out_tokens[at] = target.one;
    return;
  }
  const T* const row = target_row(at);
  const T* other = nullptr;
  Mass draft = {Mass::kNone, -1, 0.0, no_exp};
  if (refused) {
    draft = draft_mass(at + 1, p.tokens[at + 1]);
    if (draft.kind != Mass::kOne) other = draft_row(at + 1);
  }
  // shares are runs of whole 16 bytes of the target's row where it is aligned
  const int lead = row_lead(row);
  const int64_t shares = int64_t(p.ctas) * kSampleWarps;
  const int64_t share =
      ((p.vocab + lead + shares - 1) / shares + 32 * N - 1) / (32 * N) * (32 * N);
  const int64_t begin = (int64_t(rank) * kSampleWarps + warp) * share - lead;
  const int64_t end = min(begin + share, int64_t(p.vocab));
  // the masses of the run at `i` of the row
  auto masses = [&](int64_t i, bool less, double (&m)[N]) {
    float x[N], y[N];
    constexpr float kNone = LOGITS ? -INFINITY : 0.f;
    load_run<T, N>(row, i, end, kNone, x);
    if (less && other != nullptr) load_run<T, N>(other, i, end, kNone, y);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      m[k] = target(x[k], int(i) + k);
      if (less)
        m[k] = fmax(m[k] - draft(other != nullptr ? y[k] : 0.f, int(i) + k), 0.0);
    }
  };
  // What the CTA's warps and the cluster's CTAs hold of one sum: this CTA's warps' in
  // sums[which], all CTAs' in cta_sums, and their total.
  auto exchange = [&](double sum, int which, double (&all)[kMaxCluster]) -> double {
#pragma unroll
    for (int m = 1; m < 32; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == 0) sums[which][warp] = sum;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kSampleWarps; ++w) s += sums[which][w];
      cta_sum[which] = s;
    }
    double total = 0.0;
    if (p.ctas > 1) {
      cluster_sync();
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        all[c] = c < p.ctas
                     ? ld_dsmem_f64(map_to_rank(smem_addr(&cta_sum[which]), uint32_t(c)))
                     : 0.0;
        total += all[c];
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) all[c] = c == 0 ? cta_sum[which] : 0.0;
      total = all[0];
    }
    return total;
  };
  auto leave = [&] {  // no CTA ends while its sums are read
    if (p.ctas > 1) cluster_sync();
  };
  double cta_sums[kMaxCluster];
  // ---- both rows' sums, where one is taken from the other; alone a row's masses may
  // keep any common factor
  if (LOGITS && other != nullptr) {
    target.inverse = draft.inverse = 1.0;
    double sum_p = 0.0, sum_q = 0.0;
    for (int64_t i = begin + lane * N; i < end; i += 32 * N) {
      float x[N];
      load_run<T, N>(row, i, end, -INFINITY, x);
#pragma unroll
      for (int k = 0; k < N; ++k) sum_p += target(x[k], int(i) + k);
      load_run<T, N>(other, i, end, -INFINITY, x);
#pragma unroll
      for (int k = 0; k < N; ++k) sum_q += draft(x[k], int(i) + k);
    }
    target.inverse = 1.0 / exchange(sum_p, 0, cta_sums);
    sum_q = exchange(sum_q, 1, cta_sums);
    draft.inverse = sum_q > 0.0 ? 1.0 / sum_q : 0.0;
  } else if (target.kind == Mass::kLogits) {
    target.inverse = 1.0;
  }
  bool less = refused;
  for (int round = 2;; ++round) {
    double sum = 0.0;
    for (int64_t i = begin + lane * N; i < end; i += 32 * N) {
      double m[N];
      masses(i, less, m);
#pragma unroll
      for (int k = 0; k < N; ++k) sum += m[k];
    }
    const double total = exchange(sum, round, cta_sums);
    if (!(total > 0.0)) {
      if (less) {  // nothing is left: the target's own distribution
        less = false;
        continue;
      }
      if (rank == 0 && tid == 0) p.out_tokens[at] = -1;
      leave();
      return;
    }
    leave();
    // ---- the share in which u_0 of the whole falls: the first whose end passes it (the
    // last with any mass, should a rounding leave none), CTAs first, then their warps.
    // All compute the same ends in the same order, so exactly one share is chosen.
    const double wanted = uniform_of(p.uniform[rows.first]) * total;
    double before = 0.0;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < rank) before += cta_sums[c];
    if (owner_of<kMaxCluster>(wanted, 0.0, [&](int c) { return cta_sums[c]; }) != rank) return;
    if (owner_of<kSampleWarps>(wanted, before, [&](int w) { return sums[round][w]; }) != warp) return;
    for (int w = 0; w < warp; ++w) before += sums[round][w];
    double upto = before;
    int found = -1, latest = -1;
    for (int64_t base = begin; base < end && found < 0; base += 32 * N) {
      double m[N], own = 0.0;
      masses(base + lane * N, less, m);
#pragma unroll
      for (int k = 0; k < N; ++k) own += m[k];
      double incl = own;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const double v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      double run = upto + (incl - own);
      int hit = -1, any = -1;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        run += m[k];
        if (m[k] > 0.0) {
          any = int(base) + lane * N + k;
          if (hit < 0 && run > wanted) hit = any;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
      if (hits) found = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
      const unsigned some = __ballot_sync(0xffffffffu, any >= 0);
      if (some) latest = __shfl_sync(0xffffffffu, any, 31 - __clz(some));
      upto += __shfl_sync(0xffffffffu, incl, 31);
    }
    // (the sums of a share in another order can end a rounding short)
    if (lane == 0) p.out_tokens[at] = found >= 0 ? found : latest;
    return;
  }
}

}  // namespace verify
}  // namespace wq
