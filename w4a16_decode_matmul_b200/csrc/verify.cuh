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
// are binary32's, added in binary64 from 32 terms on.  For random logits they are off by 5 to 8
// 10^-8 (ex2 is low on average), where all errors have one sign by up to 21.7 2^-24 = 1.3 10^-6:
// 4 for ex2's two units in the last place, 2 ln 2 t for the rounding of x - top and of the
// exponent -t, of which the weighted mean is at most 2.7 among a thread's 32 elements, 9 for the
// additions, 5 from a thread's largest logit to the CTA's.  From 2^18 tokens on a thread has
// more than 32 elements, and each further tile costs 6.7 (4 10^-7) at most: 5 where it raises
// the largest logit, and what t grows.
//
// max(p - q, 0) with one pass over the two rows.  One pass forms the rows' sums Zp and Zq in
// binary64, and of the elements with p > q the sum D of the differences and the sum P of
// the p, all by stats_kernel's approximate sums: factors 1/Zp' and 1/Zq' for 1/Zp =
// (1 + a)/Zp' and 1/Zq = (1 + b)/Zq' (P binary64 too, though 10^-7 of it counts); what is
// left is then D (1 + b) + (a - b) P.  An element's p - q is (1 + a)(p' - q') + (a - b) q', of
// the sign of p' - q' where that is more than 2^-20 of q' and |a - b| is less; so a share with
// an element that is nearer goes over its rows a second time, and where the exact sums say that
// a and b are 2^-21 or more apart, all shares do (rounding errors of one sign throughout a row
// only: for random logits both are 5 to 8 10^-8, in the same direction).
//
// Kernels.  Logits first go through stats_kernel: largest logit and sum of exponentials
// of every piece of every row, which reads each row once.  Then, for few sequences of few
// tokens, verify_kernel, a cluster per sequence: it accepts, each warp sums its share of
// the masses, and the warp in whose share the number falls looks for the token.  Else the
// same in three kernels (decide, share, find): what is to be summed differs by a factor of
// five from one sequence to the next, and clusters left the SMs idle for a third of their
// time.  Probabilities need no statistics.
//
// Measured on B200, 64 sequences of 6 rows of 131,072 binary32 logits, drafts too (369 MB):
// statistics 62 us (5.9 TB/s, HBM bound), decisions 4, shares 28 (binary64 exponentials of
// 35 instructions each), tokens 4 to 8: 103 us in all.  With binary64 exponentials in the
// statistics 288; clusters for all 126.  32 ragged sequences of 50,021 bfloat16 logits 27 us;
// one by one, with cold caches, its kernels take 11, 7, 12 and 16: statistics wait for
// loads (half of the issue slots used), decisions and tokens are a CTA for each of 32 SMs
// that waits for loads and barriers, and find_kernel spills 228 bytes at the 64 registers
// that two CTAs an SM leave.  One sequence of 5 rows of 32,000 probabilities 8 us; 64 x 6
// rows of 131,072 binary32 probabilities 25 (10.2 at the copy rate; three kernels).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "verify_jobs.h"

namespace wq {
namespace verify {

constexpr int kPieces = 64;      // of a row, at most: slots of the workspace
constexpr int kThreads = 128;    // of stats_kernel
constexpr int kPerThread = 32;   // elements of a thread in registers
constexpr int kTile = kThreads * kPerThread;
constexpr int kMaxWarps = 16;    // of verify_kernel
constexpr int kMaxCluster = 8;
constexpr int kShares = 256;     // of a row, at most, in share_kernel
constexpr int kShareWarps = 4;   // of its CTAs, a warp a share
constexpr int kShareMost = 1024; // elements of a share, where a row's do not make more than kShares
constexpr int kDecideWarps = 16;
constexpr int kFindWarps = 16;

struct Piece {
  double sum;  // of exp((x - top) / temperature)
  float top;   // largest logit; -inf: no mass
  int first;   // where it is first
};

// What is sampled from: a row's masses, those without one token's, or what they are above
// another row's.
enum Mode { kWhole, kWithoutOne, kDifference, kDone };

// What a row is: nothing, probabilities, logits, logits of which some are +infinity (they
// share the mass), all mass on one token.
enum Kind { kNone, kProbabilities, kLogits, kShared, kOne };

// What is left to do of a sequence when its drafts are judged.
struct Decision {
  double inverse_p, inverse_q;  // what the rows' masses are multiplied by, about
  float top_p, top_q;           // largest logits
  int row, one;                 // row a of the target; the token that kWithoutOne leaves out
  int mode, kind_p, kind_q;
};

// What a share of a row holds, in units of e^top: see the head of this file.
struct Share {
  double zp, zq, d, p;
  int near;
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
  // The workspace: [2][rows][kPieces] (target, draft); [rows], at a sequence's first row; a
  // sequence's shares slots apart, by its number, or by its first row where there are
  // fewer rows than sequences
  Piece* pieces;
  Decision* decisions;
  Share* shares;
  int slots;
  int rows, seqs, rows_per_seq, vocab;
  int piece, n_pieces;               // elements of a piece, pieces of a row
  int share, n_shares;               // of share_kernel
  int ctas;                          // of verify_kernel's clusters
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
// 2^((k mod 64)/64), shared memory, times the exponent k div 64 and the series of
// 2^(r/64) to r^4: the next term is (r ln 2 / 64)^5 / 120 < 2^-44.  Table-driven
// exponentials: P. T. P. Tang, ACM TOMS 15 (1989).  Each lane of a half warp has a copy
// of the table in its own pair of banks: with one copy of 256 powers (and the series to
// r^3) a warp's look-up took six or seven cycles and was what bounded the sums.
constexpr int kTable = 64, kCopies = 16;

// What is no mass, and adds nothing to a sum that has any: of 2^30 logits below the cut,
// which come out as less than 2^-1022 each, the sum is still less.  Every other mass, every
// difference of two (of 53 bits, the whole row's mass at most 2^30 of the largest's) and
// every sum of them is more: e^-600 2^-30 2^-53 = 3e-286.
constexpr double kNoMass = 1e-290;
constexpr float kCut = 600.f;  // of the largest logit's mass, in e^-1

struct Exp {
  const double* table;  // 2^(j/64), this lane's copy: kCopies apart
  double scale;         // 64 log2(e) / temperature
  double top;           // the largest logit
  float cut;            // logits below it (e^-kCut of the largest's mass) and NaN have no mass
  __device__ __forceinline__ double operator()(float x) const {
    const double d = double(x) - top;
    const double magic = 6755399441055744.0;  // 1.5 * 2^52: rounds to an integer, the low word
    const double shifted = fma(d, scale, magic);
    const int k = __double2loint(shifted);
    const double r = fma(d, scale, magic - shifted);
    constexpr double c = 0.6931471805599453 / kTable;
    double e = fma(r, c * c * c * c / 24, c * c * c / 6);
    e = fma(e, r, c * c / 2);
    e = fma(e, r, c);
    const double base = table[(k & (kTable - 1)) * kCopies];
    e = fma(e * r, base, base);
    // (without its high word whatever came out is below 2^-1022)
    const int high = __double2hiint(e) + (k & ~(kTable - 1)) * (1 << 14);
    return __hiloint2double(x >= cut ? high : 0, __double2loint(e));
  }
};

__device__ __forceinline__ double exp_scale(float hot) {
  return kTable * 1.4426950408889634 / double(hot);
}

__device__ __forceinline__ Exp make_exp(const double* table, double scale, float top, float hot) {
  return {table, scale, double(top), fmaxf(__fsub_ru(top, kCut * hot), -3.4028234e38f)};
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^((from - to) (unit + unit_low)), to >= from: what a sum of exponentials relative to one
// logit is multiplied by to be relative to another.  All of a thread's elements share its
// error, so the exponent is held in two parts (Knuth's two-sum, the product's own error): what
// is left is ex2's 2^-22 and a rounding.  Where the exponent was one product, sums of two
// levels 8.3 apart were off by 6 10^-7.  (32 ragged sequences, a pass alone: 29.2 us so, 29.6
// now, 30.2 in binary64.)
__device__ __forceinline__ double rescale(float from, float to, float unit, float unit_low) {
  const float d = from - to, back = d - from;
  const float error = (from - (d - back)) - (to + back);
  const float t = d * unit;
  const float low = fmaf(d, unit, -t) + fmaf(d, unit_low, error * unit);
  const float y = exp2_approx(t);
  return t >= -120.f ? double(fmaf(y, low * 0.69314718f, y)) : 0.0;
}

// 2^(j/64) by the series of e^x, in the order of growing terms from the smallest.
constexpr double power_of_two(int j) {
  const double x = 0.6931471805599453 * j / kTable;
  double y = 1.0;
  for (int n = 22; n > 0; --n) y = 1.0 + y * x / n;
  return y;
}

struct Powers {
  double of[kTable];
  constexpr Powers() : of() {
    for (int j = 0; j < kTable; ++j) of[j] = power_of_two(j);
  }
};
static __device__ const Powers kPowers;

__device__ __forceinline__ void fill_table(double* table) {
  for (int i = threadIdx.x; i < kTable * 2; i += blockDim.x) {
    const double v = kPowers.of[i / 2];
#pragma unroll
    for (int c = 0; c < kCopies / 2; ++c) table[i * (kCopies / 2) + c] = v;
  }
}

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

// The mass of an element of a row of any kind but kOne, in units of e^top.
struct Mass {
  Kind kind;
  Exp exp;
  __device__ __forceinline__ double operator()(float x) const {
    if (kind == kProbabilities) return x > 0.f ? double(x) : 0.0;
    if (kind == kLogits) return exp(x);
    return kind == kShared && x == INFINITY ? 1.0 : 0.0;
  }
};

// The floats of 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void floats_of(const uint32_t (&w)[4], float (&x)[N]) {
  static_assert(N * sizeof(T) == 16, "");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void load_16(const T* from, float (&x)[N]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  floats_of<T, N>(w, x);
}

// 16 bytes that begin `lead` elements behind a 16-byte boundary, out of the two aligned
// 16 bytes that hold them.
template <typename T, int N>
__device__ __forceinline__ void load_across(const T* from, int lead, float (&x)[N]) {
  const uint4* const at = reinterpret_cast<const uint4*>(from - lead);
  const uint4 a = __ldg(at), b = __ldg(at + 1);
  const int bytes = lead * int(sizeof(T));
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(w[i], w[i + 1], (bytes & 2) * 8);
  floats_of<T, N>(v, x);
}

// Elements at .. at + N - 1 of a row as floats, `none` outside [0, end): 16 bytes at once
// where they are inside; `lead`: elements between a 16-byte boundary and element `at`.
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* row, int at, int end, int lead, float none,
                                         float (&x)[N]) {
  if (lead == 0 && at >= 0 && at <= end - N) {
    load_16<T, N>(row + at, x);
  } else if (lead != 0 && at >= N && at <= end - 2 * N) {
    load_across<T, N>(row + at, lead, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = at + i >= 0 && at + i < end ? to_float(row[at + i]) : none;
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
  int b = 0, stands = 0;  // the sequence's row whose token is no draft
  float hot = 1.f;
  if (p.row_starts == nullptr) {
    b = r / p.rows_per_seq;
    stands = b * p.rows_per_seq;
    if (p.temperature != nullptr) hot = p.temperature[b];
  } else if (p.seqs < 32) {
    // all of them at once
    const int start = p.row_starts[min(lane, p.seqs)];
    if (p.temperature != nullptr) hot = p.temperature[min(lane, p.seqs - 1)];
    // (the first that is not, so that a bad range does not move the rows before it)
    const unsigned beyond = __ballot_sync(0xffffffffu, lane > p.seqs || start > r);
    b = beyond ? __ffs(beyond) - 2 : 31;
    if (b < 0 || b >= p.seqs) return;
    stands = __shfl_sync(0xffffffffu, start, b);
    hot = __shfl_sync(0xffffffffu, hot, b);
  } else {
    int lo = 0, n = p.seqs + 1;
    if (p.row_starts[0] > r) return;
    while (n > 1) {
      const int step = (n + 32) / 33;
      const int at = lo + (lane + 1) * step;
      const bool below = at < lo + n && p.row_starts[at] <= r;
      const unsigned beyond = ~__ballot_sync(0xffffffffu, below);
      const int skip = beyond ? __ffs(beyond) - 1 : 32;
      lo += skip * step;
      n = min(step, n - skip * step);
    }
    if (lo >= p.seqs) return;
    b = lo;
    stands = p.row_starts[b];
    if (p.temperature != nullptr) hot = p.temperature[b];
  }
  const bool greedy = !(hot > 0.f);
  if (is_draft && (greedy || r <= stands)) return;  // its distribution is not looked at
  const T* const row = is_draft ? static_cast<const T*>(p.draft) + int64_t(r) * p.draft_stride
                                : static_cast<const T*>(p.target) + int64_t(r) * p.target_stride;
  const int begin = piece * p.piece - row_lead(row);
  const int end = min(begin + p.piece, p.vocab);
  // the elements stay in the registers as they are stored: half as many for bfloat16
  constexpr uint32_t kNothing = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
  auto load = [&](int tile, uint32_t (&w)[kRuns][4]) {
    if (tile >= 0 && tile <= end - kTile) {
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        const uint4 v =
            __ldg(reinterpret_cast<const uint4*>(row + tile + (k * kThreads + tid) * N));
        w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        const int at = tile + (k * kThreads + tid) * N;
        if (at >= 0 && at <= end - N) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + at));
          w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4) {
            w[k][i] = at + i >= 0 && at + i < end ? __float_as_uint(row[at + i]) : kNothing;
          } else {
            const int e = at + 2 * i;
            const uint32_t one =
                e >= 0 && e < end ? __bfloat16_as_ushort(row[e]) : kNothing & 0xffffu;
            const uint32_t two =
                e + 1 >= 0 && e + 1 < end ? __bfloat16_as_ushort(row[e + 1]) : kNothing >> 16;
            w[k][i] = one | (two << 16);
          }
        }
      }
    }
  };
  // element pair j of a run: (2j, 2j + 1)
  auto pair_of = [](const uint32_t (&w)[4], int j) -> float2 {
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else
      return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  };
  // log2(e) / temperature in two parts: a binary32 product would be off by 2^-24 of the
  // exponent, for all terms in the same direction
  const double log2_unit = fmin(fmax(1.4426950408889634 / double(hot), 1e-30), 1e30);
  const float unit = float(log2_unit), unit_low = float(log2_unit - double(unit));
  const float lowest = -200.f / unit;  // 2^-200: nothing in binary32
  double sum = 0.0;
  float top = -INFINITY;
  int first = 0x7fffffff;
  for (int tile = begin; tile < end; tile += kTile) {
    uint32_t w[kRuns][4];
    load(tile, w);
    grid_dependents_launch();
    float high = -INFINITY;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) high = fmaxf(high, __uint_as_float(w[k][i]));
    } else {
      uint32_t most = kNothing;
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) most = bmax2(most, w[k][i]);
      high = fmaxf(__uint_as_float(most << 16), __uint_as_float(most & 0xffff0000u));
    }
    if (greedy) {
      if (high > top) {
        top = high;
#pragma unroll
        for (int k = kRuns - 1; k >= 0; --k)
#pragma unroll
          for (int j = N / 2 - 1; j >= 0; --j) {
            const float2 x = pair_of(w[k], j);
            const int at = tile + (k * kThreads + tid) * N + 2 * j;
            if (x.y == high) first = at + 1;
            if (x.x == high) first = at;
          }
      }
      continue;
    }
    // each thread relative to its own largest
    if (fmaxf(top, high) == -INFINITY) continue;
    if (high > top) {
      if (sum > 0.0) sum *= rescale(top, high, unit, unit_low);
      top = high;
    }
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (top == INFINITY) {
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 x = pair_of(w[k], j);
          part[0].x += (x.x == INFINITY ? 1.f : 0.f) + (x.y == INFINITY ? 1.f : 0.f);
        }
    } else {
      const float2 below = make_float2(-top, -top), u = make_float2(unit, unit);
      const float2 u_low = make_float2(unit_low, unit_low);
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          // -inf and NaN end up at the lowest, whose exponential is 0
          float2 d = add2(pair_of(w[k], j), below);
          d = make_float2(fmaxf(d.x, lowest), fmaxf(d.y, lowest));
          const float2 t = fma2(d, u, mul2(d, u_low));
          part[j & 1] = add2(part[j & 1], make_float2(exp2_approx(t.x), exp2_approx(t.y)));
        }
    }
    part[0] = add2(part[0], part[1]);
    sum += double(part[0].x + part[0].y);
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
  if (top != high) sum *= rescale(top, high, unit, unit_low);
#pragma unroll
  for (int m = 1; m < 32; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  at = __reduce_min_sync(0xffffffffu, at);
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

// What is known of a row: its kind, the token that has all, the largest logit, what its
// masses are multiplied by, and the mass of the token in question.
struct RowStat {
  double inverse, of_token;
  float top;
  int one;
  Kind kind;
};

// A row's statistics from its pieces, by all lanes of a warp; x is the logit of token
// `token` of it.
__device__ __forceinline__ RowStat join_pieces(const Params& p, int index, float hot, double scale,
                                               const double* table, float x, int token, int lane) {
  const Piece* from = p.pieces + int64_t(index) * kPieces;
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
  if (top == -INFINITY) return {0.0, 0.0, top, -1, kNone};
  if (!(hot > 0.f)) {
    int first = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kPieces / 32; ++k)
      if (mine[k].top == top) first = min(first, mine[k].first);
    first = __reduce_min_sync(0xffffffffu, first);
    return {1.0, first == token ? 1.0 : 0.0, top, first, kOne};
  }
  const bool shared = top == INFINITY;
  const Exp exp = make_exp(table, scale, top, hot);
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kPieces / 32; ++k)
    sum += mine[k].top == top ? mine[k].sum : shared ? 0.0 : mine[k].sum * exp(mine[k].top);
#pragma unroll
  for (int m = 1; m < 32; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const double inverse = 1.0 / sum;
  const Mass mass = {shared ? kShared : kLogits, exp};
  const double of_token = mass(x) * inverse;
  return {inverse, of_token < kNoMass ? 0.0 : of_token, top, -1, mass.kind};
}

// A uniform number as it is used: inside [0, 1), a NaN as 0.
__device__ __forceinline__ double uniform_of(float u) {
  return double(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
}

// The first of n shares, which begin at `from`, whose end is beyond `wanted` (the last
// with any mass if none is); `from` becomes where it begins.
__device__ __forceinline__ int owner_of(const double* sums, int n, double wanted, double& from) {
  int owner = -1;
  double at = from;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const double s = sums[i], end = at + s;
    if (s > kNoMass) {
      owner = i;
      from = at;
      if (end > wanted) break;
    }
    at = end;
  }
  return owner;
}

__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// Two rows (or one) as a warp reads them, 32 runs of 16 bytes at a time, on the first row's
// boundaries.
template <typename T, bool LOGITS, int MODE>
struct Reader {
  static constexpr int N = 16 / int(sizeof(T)), kStep = 32 * N;
  static constexpr float kNothing = LOGITS ? -INFINITY : 0.f;
  const T *row, *other;
  int lead, other_lead;  // elements between boundaries and the runs
  int lane;
  __device__ __forceinline__ Reader(const T* row, const T* other, int lane)
      : row(row), other(other), lead(row_lead(row)), lane(lane) {
    other_lead = MODE == kDifference ? (row_lead(other) - lead + N) % N : 0;
  }
  // Runs from i0 on that need no checks: whole, and inside the rows where they lie across
  // the other row's boundaries.
  __device__ __forceinline__ bool safe(int i0, int end) const {
    const int margin = MODE == kDifference && other_lead != 0 ? N : 0;
    return i0 >= margin && i0 <= end - kStep - margin;
  }
  __device__ __forceinline__ void load(int i0, int end, float (&x)[N]) const {
    if (safe(i0, end))
      load_16<T, N>(row + i0 + lane * N, x);
    else
      load_run<T, N>(row, i0 + lane * N, end, 0, kNothing, x);
  }
  __device__ __forceinline__ void load_other(int i0, int end, float (&y)[N]) const {
    if (!safe(i0, end))
      load_run<T, N>(other, i0 + lane * N, end, other_lead, kNothing, y);
    else if (other_lead == 0)
      load_16<T, N>(other + i0 + lane * N, y);
    else
      load_across<T, N>(other + i0 + lane * N, other_lead, y);
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int m = 1; m < 32; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// What is sampled from, over elements [begin, end) of the rows, by all lanes of a warp.
// P and Q: masses of an element of either row.
template <typename T, bool LOGITS, int MODE, class P, class Q>
struct Masses {
  using R = Reader<T, LOGITS, MODE>;
  static constexpr int N = R::N;
  // logits' sums are known about, and exactly only when a pass is over; alone a row's
  // masses may keep any factor
  static constexpr bool kTwoSums = LOGITS && MODE == kDifference;
  R rows;
  P p;
  Q q;
  double inverse_p, inverse_q;  // about
  int one;

  __device__ __forceinline__ Share share(int begin, int end) const {
    Share s = {0.0, 0.0, 0.0, 0.0, 0};
    bool near = false;
    float next_x[N], next_y[N];
    if (begin < end) {
      rows.load(begin, end, next_x);
      if (MODE == kDifference) rows.load_other(begin, end, next_y);
    }
    for (int i0 = begin; i0 < end; i0 += R::kStep) {
      float x[N], y[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        x[k] = next_x[k];
        if (MODE == kDifference) y[k] = next_y[k];
      }
      if (i0 + R::kStep < end) {  // loads a step ahead
        rows.load(i0 + R::kStep, end, next_x);
        if (MODE == kDifference) rows.load_other(i0 + R::kStep, end, next_y);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const double e = p(x[k]);
        s.zp += e;
        if (MODE == kWithoutOne && i0 + rows.lane * N + k != one) s.d += e;
        if (MODE == kDifference) {
          const double f = q(y[k]), taken = f * inverse_q;
          const double left = fma(e, inverse_p, -taken);
          const int high = __double2hiint(left);
          if (kTwoSums) {
            s.zq += f;
            near |= __double2hiint(taken) - (high & 0x7fffffff) > (20 << 20);
            s.p += __hiloint2double(high >= 0 ? __double2hiint(e) : 0, __double2loint(e));
          }
          // (without its high word a number is below 2^-1022)
          s.d += __hiloint2double(high >= 0 ? high : 0, __double2loint(left));
        }
      }
    }
    s.zp = warp_sum(s.zp);
    if (MODE != kWhole) s.d = warp_sum(s.d);
    if (kTwoSums) {
      s.zq = warp_sum(s.zq);
      s.p = warp_sum(s.p);
      s.near = __any_sync(0xffffffffu, near);
    }
    if (MODE == kWhole) s.d = s.zp;
    return s;
  }

  // The rows' factors from their whole sums.
  __device__ __forceinline__ void factors(double zp, double zq, double& of_p,
                                          double& of_q) const {
    of_p = kTwoSums ? 1.0 / zp : MODE == kDifference ? inverse_p : 1.0;
    of_q = kTwoSums ? (zq > kNoMass ? 1.0 / zq : 0.0) : inverse_q;
  }

  // The masses of a lane's run.
  __device__ __forceinline__ void run(int i0, int end, bool whole, double of_p, double of_q,
                                      double (&m)[N]) const {
    float x[N], y[N];
    rows.load(i0, end, x);
    if (MODE == kDifference && !whole) rows.load_other(i0, end, y);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      m[k] = p(x[k]);
      if (whole) continue;
      if (MODE == kWithoutOne && i0 + rows.lane * N + k == one) m[k] = 0.0;
      // (products rounded alike: of equal rows nothing is left)
      if (MODE == kDifference)
        m[k] = fmax(__dsub_rn(__dmul_rn(m[k], of_p), __dmul_rn(of_q, q(y[k]))), 0.0);
    }
  }

  __device__ __forceinline__ double sum(int begin, int end, bool whole, double of_p,
                                        double of_q) const {
    double s = 0.0;
    for (int i0 = begin; i0 < end; i0 += R::kStep) {
      double m[N];
      run(i0, end, whole, of_p, of_q, m);
#pragma unroll
      for (int k = 0; k < N; ++k) s += m[k];
    }
    return warp_sum(s);
  }

  // What the factors are above those by which the shares were formed, of themselves.
  __device__ __forceinline__ double above_p(double of_p) const {
    return (of_p - inverse_p) / inverse_p;
  }
  __device__ __forceinline__ double above_q(double of_q) const {
    return inverse_q > 0.0 ? (of_q - inverse_q) / inverse_q : 0.0;
  }

  // Whether a share was formed by factors too far from the rows' to tell where p > q.
  __device__ __forceinline__ bool unsure(const Share& s, double of_p, double of_q) const {
    return kTwoSums && (s.near || fabs(above_p(of_p) - above_q(of_q)) >= 0x1p-21);
  }

  // The mass of any other share.
  __device__ __forceinline__ double finish(const Share& s, double of_p, double of_q) const {
    if (!kTwoSums) return s.d;
    const double a = above_p(of_p), b = above_q(of_q);
    return fmax(fma(s.d, b, s.d) + (a - b) * (inverse_p * s.p), 0.0);
  }

  // A lane's sum of its run; incl: of the lanes up to it.
  __device__ __forceinline__ static double scan(const double (&m)[N], double& incl) {
    double own = 0.0;
#pragma unroll
    for (int k = 0; k < N; ++k) own += m[k];
    incl = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const double v = __shfl_up_sync(0xffffffffu, incl, d);
      if (int(threadIdx.x & 31) >= d) incl += v;
    }
    return own;
  }

  // The first element of the warp's runs from i0 on at whose end the running sum, which is
  // `at` ahead of this lane's, is beyond `wanted`, or -1; latest: the last with any mass.
  __device__ __forceinline__ int pick(int i0, const double (&m)[N], double at, double wanted,
                                      int& latest) const {
    int hit = -1, any = -1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      at += m[k];
      if (m[k] > kNoMass) {
        any = i0 + rows.lane * N + k;
        if (hit < 0 && at > wanted) hit = any;
      }
    }
    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
    const unsigned held = __ballot_sync(0xffffffffu, any >= 0);
    if (held) latest = __shfl_sync(0xffffffffu, any, 31 - __clz(held));
    return hits ? __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1) : -1;
  }

  // The first element of [begin, end) at whose end the running sum, which is `before` ahead
  // of them, is beyond `wanted`; the last with any mass where a rounding leaves none.
  __device__ __forceinline__ int find(int begin, int end, bool whole, double of_p, double of_q,
                                      double before, double wanted) const {
    int found = -1, latest = -1;
    for (int i0 = begin; i0 < end && found < 0; i0 += R::kStep) {
      double m[N], incl;
      run(i0, end, whole, of_p, of_q, m);
      const double own = scan(m, incl);
      found = pick(i0, m, before + (incl - own), wanted, latest);
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return found >= 0 ? found : latest;
  }
};

// Calls use(masses) with what is sampled from by a decision.
template <typename T, bool LOGITS, class Use>
__device__ __forceinline__ void with_masses(const Params& p, const Decision& d, float hot,
                                            double scale, const double* table, int lane,
                                            Use use) {
  const T* const row = static_cast<const T*>(p.target) + int64_t(d.row) * p.target_stride;
  const T* const other = static_cast<const T*>(p.draft) + int64_t(d.row + 1) * p.draft_stride;
  const Mass mp = {Kind(d.kind_p), make_exp(table, scale, d.top_p, hot)};
  const Mass mq = {Kind(d.kind_q), make_exp(table, scale, d.top_q, hot)};
  if (d.mode == kWhole) {
    Reader<T, LOGITS, kWhole> r(row, nullptr, lane);
    if (LOGITS && d.kind_p == kLogits)
      use(Masses<T, LOGITS, kWhole, Exp, Exp>{r, mp.exp, mp.exp, 1.0, 1.0, -1});
    else
      use(Masses<T, LOGITS, kWhole, Mass, Mass>{r, mp, mp, 1.0, 1.0, -1});
  } else if (d.mode == kWithoutOne) {
    Reader<T, LOGITS, kWithoutOne> r(row, nullptr, lane);
    if (LOGITS && d.kind_p == kLogits)
      use(Masses<T, LOGITS, kWithoutOne, Exp, Exp>{r, mp.exp, mp.exp, 1.0, 1.0, d.one});
    else
      use(Masses<T, LOGITS, kWithoutOne, Mass, Mass>{r, mp, mp, 1.0, 1.0, d.one});
  } else {
    Reader<T, LOGITS, kDifference> r(row, other, lane);
    if (LOGITS && d.kind_p == kLogits && d.kind_q == kLogits)
      use(Masses<T, LOGITS, kDifference, Exp, Exp>{r, mp.exp, mq.exp, d.inverse_p, d.inverse_q,
                                                   -1});
    else
      use(Masses<T, LOGITS, kDifference, Mass, Mass>{r, mp, mq, d.inverse_p, d.inverse_q, -1});
  }
}

// Judges a sequence's drafts, by all warps of a CTA, up to kBlock at a time, and writes the
// outputs where `writes` is true -- all but the sampled token, for which the decision
// says what is left to do.  A warp a row: target row i judges the token of row i + 1,
// which draft row i + 1 drew.  `wait` is called before the pieces are read.
constexpr int kBlock = 32;

struct DecideShared {
  RowStat stats[2][kBlock + 1];  // target rows base .., draft rows base ..
  int rejected;
};

template <typename T, bool LOGITS, int WARPS, class Wait>
__device__ __forceinline__ Decision decide(const Params& p, DecideShared& s, int b,
                                           const Rows& rows, float hot, double scale,
                                           const double* table, bool writes, Wait wait) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int drafts = rows.count - 1;
  if (tid == 0) s.rejected = drafts;
  int base = 0;
  while (true) {
    const int n = min(drafts - base, kBlock);
    const double mine = tid < n ? uniform_of(p.uniform[rows.first + base + tid + 1]) : 0.0;
    // a job: its row, the token in question and that token's element
    const int jobs = jobs_of(n);
    Job at;
    int token;
    bool known, one;
    float x;
    auto fetch = [&](int job) {
      at = job_of(job, n, base);
      const int r = rows.first + at.row;
      token = at.token_row <= drafts ? p.tokens[rows.first + at.token_row] : -1;
      known = token >= 0 && token < p.vocab;
      one = at.is_draft && (p.draft == nullptr || !(hot > 0.f));
      x = 0.f;
      if (known && !one)
        x = to_float(at.is_draft
                         ? static_cast<const T*>(p.draft)[int64_t(r) * p.draft_stride + token]
                         : static_cast<const T*>(p.target)[int64_t(r) * p.target_stride + token]);
    };
    if (warp < jobs) fetch(warp);
    if (base == 0) wait();
    for (int job = warp; job < jobs; job += WARPS) {
      if (job != warp) fetch(job);
      RowStat stat;
      if (one) {
        // a draft without a distribution; greedy: whatever it is, the token is accepted if
        // it is the target's, and what is left is the target's
        stat = {1.0, 1.0, 0.f, token, kOne};
      } else if (!LOGITS) {
        stat = {1.0, known && x > 0.f ? double(x) : 0.0, 0.f, -1, kProbabilities};
      } else {
        const int r = rows.first + at.row;
        stat = join_pieces(p, (at.is_draft ? p.rows : 0) + r, hot, scale, table, x, token, lane);
        if (!known) stat.of_token = 0.0;
      }
      if (lane == 0) s.stats[at.is_draft][at.row - base] = stat;
    }
    __syncthreads();
    if (tid < n) {
      const int token = p.tokens[rows.first + base + tid + 1];
      if (token < 0 || token >= p.vocab ||
          !(mine * s.stats[1][tid + 1].of_token < s.stats[0][tid].of_token))
        atomicMin(&s.rejected, base + tid);
    }
    __syncthreads();
    if (s.rejected < base + n || base + n == drafts) break;
    base += kBlock;
  }
  const int a = s.rejected, at = rows.first + a;
  const bool refused = a < drafts;
  if (writes) {
    for (int i = tid; i < rows.count; i += WARPS * 32)
      if (i != a) p.out_tokens[rows.first + i] = i < a ? p.tokens[rows.first + i + 1] : -1;
    if (tid == 0) {
      p.accepted[b] = a;
      if (p.out_lens != nullptr) p.out_lens[b] = p.seq_lens[b] - (drafts - a);
    }
  }
  const RowStat target = s.stats[0][a - base];
  Decision d = {target.inverse, 0.0, target.top, 0.f, at, -1, kWhole, target.kind, kNone};
  if (target.kind == kNone || target.kind == kOne) {
    if (writes && tid == 0) p.out_tokens[at] = target.one;
    d.mode = kDone;
  } else if (refused) {
    const RowStat draft = s.stats[1][a - base + 1];
    d.mode = draft.kind == kOne ? kWithoutOne : kDifference;
    d.one = draft.one;
    d.inverse_q = draft.inverse;
    d.top_q = draft.top;
    d.kind_q = draft.kind;
  }
  return d;
}

__device__ __forceinline__ Share* shares_of(const Params& p, int b, const Rows& rows) {
  return p.shares + int64_t(p.seqs <= p.rows ? b : rows.first) * p.slots;
}

__device__ __forceinline__ void no_rows(const Params& p, int b) {
  p.accepted[b] = 0;
  if (p.out_lens != nullptr) p.out_lens[b] = p.seq_lens[b];
}

__device__ __forceinline__ float heat(const Params& p, bool logits, int b) {
  return logits && p.temperature != nullptr ? p.temperature[b] : 1.f;
}

// ---- few sequences of few tokens: one a cluster -----------------------------------------------

// What an exchange leaves: the sums of this CTA's warps, and of the cluster's CTAs.
struct Sums {
  double warp[kMaxWarps], cta[kMaxCluster];
};

// Joins what the cluster's threads hold of n sums, in a fixed order: every CTA's share
// is in every CTA's sums[i] then, as those of its own warps; total[i] the whole.
template <int WARPS, int COUNT>
__device__ __forceinline__ void exchange(Sums* sums, const double (&mine)[COUNT],
                                         double (&total)[COUNT], int ctas, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < COUNT; ++i)
    if (lane == 0) sums[i].warp[warp] = mine[i];
  __syncthreads();
  if (warp < COUNT) {
    double s = lane < WARPS ? sums[warp].warp[lane] : 0.0;
#pragma unroll
    for (int m = 1; m < WARPS; m *= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (ctas == 1) {
      if (lane == 0) sums[warp].cta[0] = s;
    } else if (lane < ctas) {
      st_dsmem_f64(map_to_rank(smem_addr(&sums[warp].cta[rank]), uint32_t(lane)), s);
    }
    __syncwarp();
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    total[i] = 0.0;
    for (int c = 0; c < ctas; ++c) total[i] += sums[i].cta[c];
  }
}

template <typename T, bool LOGITS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 32 / WARPS) verify_kernel(const Params p) {
  __shared__ double table_s[LOGITS ? kTable * kCopies : 1];
  __shared__ Sums sums[4];  // of both rows' masses, of what is sampled from
  __shared__ DecideShared ds;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const double* const table = table_s + (lane & (kCopies - 1));
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  const int b = int(blockIdx.x) / p.ctas;
  if (p.ctas > 1) cluster_arrive();  // all CTAs run when the first sums are exchanged
  const Rows rows = load_rows(p, b);
  if (rows.count == 0) {
    if (rank == 0 && tid == 0) no_rows(p, b);
    if (p.ctas > 1) cluster_wait();
    if (LOGITS) grid_dependency_wait();  // no grid is over before the one it depends on
    return;
  }
  const float hot = heat(p, LOGITS, b);
  const double scale = exp_scale(hot), number = uniform_of(p.uniform[rows.first]);
  if (LOGITS) fill_table(table_s);
  __syncthreads();
  const Decision d = decide<T, LOGITS, WARPS>(p, ds, b, rows, hot, scale, table, rank == 0, [] {
    if (LOGITS) grid_dependency_wait();
  });
  if (p.ctas > 1) cluster_wait();
  if (d.mode == kDone) return;
  with_masses<T, LOGITS>(p, d, hot, scale, table, lane, [&](const auto& m) {
    using M = std::decay_t<decltype(m)>;
    constexpr int kStep = M::R::kStep;
    const int lead = m.rows.lead, shares = p.ctas * WARPS;
    const int size = ((p.vocab + lead + shares - 1) / shares + kStep - 1) / kStep * kStep;
    const int64_t first = int64_t(rank * WARPS + warp) * size - lead;
    const int begin = int(min(first, int64_t(p.vocab)));
    const int end = int(min(first + size, int64_t(p.vocab)));
    const Share share = m.share(begin, end);
    double of_p, of_q, z[2] = {share.zp, share.zq};
    if (M::kTwoSums) exchange<WARPS, 2>(sums, {share.zp, share.zq}, z, p.ctas, rank);
    m.factors(z[0], z[1], of_p, of_q);
    double total[1];
    const double mass = m.unsure(share, of_p, of_q) ? m.sum(begin, end, false, of_p, of_q)
                                                    : m.finish(share, of_p, of_q);
    exchange<WARPS, 1>(sums + 2, {mass}, total, p.ctas, rank);
    bool whole = false;
    Sums* of = sums + 2;
    if (!(total[0] > kNoMass)) {  // nothing is left: the target's own distribution
      whole = true;
      of = sums + 3;
      exchange<WARPS, 1>(sums + 3, {share.zp}, total, p.ctas, rank);
      if (!(total[0] > kNoMass)) {
        if (rank == 0 && tid == 0) p.out_tokens[d.row] = -1;
        return;
      }
    }
    // The share in which the number falls: CTAs first, then their warps.  All compute the
    // same ends in the same order, so exactly one share is chosen.
    const double wanted = number * total[0];
    double before = 0.0;
    if (owner_of(of->cta, p.ctas, wanted, before) != rank) return;
    if (owner_of(of->warp, WARPS, wanted, before) != warp) return;
    const int token = m.find(begin, end, whole, of_p, of_q, before, wanted);
    if (lane == 0) p.out_tokens[d.row] = token;
  });
}

// ---- the others: three kernels ------------------------------------------------

template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kDecideWarps * 32) decide_kernel(const Params p) {
  __shared__ double table_s[LOGITS ? kTable * kCopies : 1];
  __shared__ DecideShared ds;
  const int tid = threadIdx.x, lane = tid & 31, b = int(blockIdx.x);
  grid_dependents_launch();
  const Rows rows = load_rows(p, b);
  if (rows.count == 0) {
    if (tid == 0) no_rows(p, b);
    if (LOGITS) grid_dependency_wait();  // no grid is over before the one it depends on
    return;
  }
  const float hot = heat(p, LOGITS, b);
  if (LOGITS) fill_table(table_s);
  __syncthreads();
  const Decision d =
      decide<T, LOGITS, kDecideWarps>(p, ds, b, rows, hot, exp_scale(hot),
                                      table_s + (lane & (kCopies - 1)), true, [] {
                                        if (LOGITS) grid_dependency_wait();
                                      });
  if (tid == 0) p.decisions[rows.first] = d;
}

// A warp a share; CTAs of four shares of one sequence.
template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kShareWarps * 32, 6) share_kernel(const Params p) {
  __shared__ double table_s[LOGITS ? kTable * kCopies : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = (p.n_shares + kShareWarps - 1) / kShareWarps;
  const int b = int(blockIdx.x) / ctas;
  const int i = (int(blockIdx.x) - b * ctas) * kShareWarps + warp;
  grid_dependents_launch();
  const Rows rows = load_rows(p, b);
  const float hot = heat(p, LOGITS, b);
  if (LOGITS) fill_table(table_s);
  __syncthreads();
  grid_dependency_wait();
  if (rows.count == 0) return;
  const Decision d = p.decisions[rows.first];
  if (d.mode == kDone || i >= p.n_shares) return;
  with_masses<T, LOGITS>(p, d, hot, exp_scale(hot), table_s + (lane & (kCopies - 1)), lane,
                         [&](const auto& m) {
                           const int64_t first = int64_t(i) * p.share - m.rows.lead;
                           const Share s = m.share(int(min(first, int64_t(p.vocab))),
                                                   int(min(first + p.share, int64_t(p.vocab))));
                           if (lane == 0) shares_of(p, b, rows)[i] = s;
                         });
}

// The sum of one number of each thread, the same in all.
template <int WARPS>
__device__ __forceinline__ double block_sum(double v, double* scratch) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) s += scratch[w];
  return s;
}

// The token of each sequence, from its shares.  A CTA a sequence: the chosen share is cut
// once more among its warps.
template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kFindWarps * 32, 2) find_kernel(const Params p) {
  __shared__ double table_s[LOGITS ? kTable * kCopies : 1];
  __shared__ double masses[kShares], scratch[kFindWarps], scratch_q[kFindWarps], ends[1];
  __shared__ int chosen, near[kShares], near_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = int(blockIdx.x);
  const Rows rows = load_rows(p, b);
  const float hot = heat(p, LOGITS, b);
  if (rows.count == 0) {
    grid_dependency_wait();
    return;
  }
  const double number = uniform_of(p.uniform[rows.first]);
  if (LOGITS) fill_table(table_s);
  if (tid == 0) near_count = 0;
  __syncthreads();
  grid_dependency_wait();
  const Decision d = p.decisions[rows.first];
  if (d.mode == kDone) return;
  const Share* const shares = shares_of(p, b, rows);
  with_masses<T, LOGITS>(
      p, d, hot, exp_scale(hot), table_s + (lane & (kCopies - 1)), lane, [&](const auto& m) {
        using M = std::decay_t<decltype(m)>;
        auto part = [&](int i, int& begin, int& end) {
          const int64_t first = int64_t(i) * p.share - m.rows.lead;
          begin = int(min(first, int64_t(p.vocab)));
          end = int(min(first + p.share, int64_t(p.vocab)));
        };
        static_assert(kShares <= kFindWarps * 32, "a thread a share");
        Share s = {0.0, 0.0, 0.0, 0.0, 0};
        if (tid < p.n_shares) s = shares[tid];
        double of_p, of_q, zp = s.zp, zq = s.zq;
        if (M::kTwoSums) {
          zp = warp_sum(s.zp);
          zq = warp_sum(s.zq);
          if (lane == 0) scratch[warp] = zp, scratch_q[warp] = zq;
          __syncthreads();
          zp = zq = 0.0;
#pragma unroll
          for (int w = 0; w < kFindWarps; ++w) zp += scratch[w], zq += scratch_q[w];
        }
        m.factors(zp, zq, of_p, of_q);
        if (tid < kShares) {
          if (tid < p.n_shares && m.unsure(s, of_p, of_q)) near[atomicAdd(&near_count, 1)] = tid;
          masses[tid] = m.finish(s, of_p, of_q);
        }
        __syncthreads();
        // shares that have to be gone over again: a few, each by all warps, or a warp a share
        const bool many = near_count >= kFindWarps;
        for (int k0 = 0; k0 < near_count; k0 += many ? kFindWarps : 1) {
          const int k = many ? k0 + warp : k0;
          int begin = 0, end = 0;
          if (k < near_count) part(near[k], begin, end);
          const int steps = (end - begin + M::R::kStep - 1) / M::R::kStep;
          const int each = (many ? steps : (steps + kFindWarps - 1) / kFindWarps) * M::R::kStep;
          const int from = min(begin + (many ? 0 : warp * each), end), to = min(from + each, end);
          const double own = m.sum(from, to, false, of_p, of_q);
          if (many) {
            if (lane == 0 && k < near_count) masses[near[k]] = own;
          } else {
            const double mass = block_sum<kFindWarps>(lane == 0 ? own : 0.0, scratch);
            if (tid == 0) masses[near[k]] = mass;
          }
        }
        __syncthreads();
        double total = block_sum<kFindWarps>(tid < p.n_shares ? masses[tid] : 0.0, scratch);
        bool whole = false;
        if (!(total > kNoMass)) {  // nothing is left: the target's own distribution
          whole = true;
          __syncthreads();
          if (tid < kShares) masses[tid] = s.zp;
          total = block_sum<kFindWarps>(s.zp, scratch);
          if (!(total > kNoMass)) {
            if (tid == 0) p.out_tokens[d.row] = -1;
            return;
          }
        }
        const double wanted = number * total;
        if (warp == 0) {
          // a lane's eight shares in order, then the lanes'
          constexpr int kEach = kShares / 32;
          double own = 0.0;
          for (int k = 0; k < kEach; ++k)
            own += lane * kEach + k < p.n_shares ? masses[lane * kEach + k] : 0.0;
          double incl = own;
#pragma unroll
          for (int k = 1; k < 32; k *= 2) {
            const double v = __shfl_up_sync(0xffffffffu, incl, k);
            if (lane >= k) incl += v;
          }
          const unsigned past = __ballot_sync(0xffffffffu, incl > wanted && own > kNoMass);
          const unsigned held = __ballot_sync(0xffffffffu, own > kNoMass);
          if (lane == (past ? __ffs(past) - 1 : held ? 31 - __clz(held) : 0)) {
            double before = incl - own;
            const int n = min(kEach, p.n_shares - lane * kEach);
            chosen = max(0, lane * kEach + owner_of(masses + lane * kEach, n, wanted, before));
            ends[0] = before;
          }
        }
        __syncthreads();
        // ---- the chosen share, a contiguous part of it a warp
        int begin, end;
        part(chosen, begin, end);
        constexpr int kStep = M::R::kStep;
        const int steps = (end - begin + kStep - 1) / kStep;
        const int each = (steps + kFindWarps - 1) / kFindWarps * kStep;
        const int from = min(begin + warp * each, end), to = min(from + each, end);
        if (each == kStep) {  // a step a warp: its masses stay where they are
          double run[M::N], incl;
          m.run(from, to, whole, of_p, of_q, run);
          const double own = M::scan(run, incl);
          if (lane == 31) scratch[warp] = incl;
          __syncthreads();
          double before = ends[0];
          if (owner_of(scratch, kFindWarps, wanted, before) != warp) return;
          int latest = -1;
          int token = m.pick(from, run, before + (incl - own), wanted, latest);
          if (token < 0) token = latest;
          if (lane == 0) p.out_tokens[d.row] = token;
          return;
        }
        const double mine = m.sum(from, to, whole, of_p, of_q);
        if (lane == 0) scratch[warp] = mine;
        __syncthreads();
        double before = ends[0];
        if (owner_of(scratch, kFindWarps, wanted, before) != warp) return;
        const int token = m.find(from, to, whole, of_p, of_q, before, wanted);
        if (lane == 0) p.out_tokens[d.row] = token;
      });
}

}  // namespace verify
}  // namespace wq
