// kv4_attn.cuh -- attention of a few query rows per sequence over the 4-bit
// cache (decode, speculative verification): every key and value code is read
// from HBM once and goes to the tensor cores as an exact integer.
//
// Mathematics, for one kv head and one query row q (base 2 logarithms):
//   S_t = c sum_g s_{t,g} sum_{d in g} q_d (u_{t,d} - z_{t,g}),  c = scale log2 e
//   O_d = sum_t 2^(S_t) s'_{t,g} (u'_{t,d} - z'_{t,g}) / sum_t 2^(S_t)
// with a running maximum over the tokens.  Both products run with the codes
// as the 16-row operand of mma.sync (16 tokens x 16 dims, then 16 dims x 16
// tokens) and the query rows as its 8 columns, so one instruction takes 256
// codes.  The codes enter as u - 8 (exact in binary16; one shift, four LOP3
// and four packed FMA-pipe instructions per eight codes) and the rest is
// exact algebra in binary32: sum q (u - z) = sum q (u - 8) + (8 - z) sum q,
// and likewise for the values with the weights in q's place.
//
// Roundings.  A query row is scaled by a power of two that puts its largest
// magnitude in [2^14, 2^15) and rounded to binary16: exact for every bfloat16
// within 2^-21 of that magnitude.  The weights W_t = 2^(S_t - m) s'_{t,g} are
// rounded to binary16 (half a step is 2^-11, an eighth of the output's bfloat16
// half step).  m is the running maximum not of S_t but of S_t + log2 max_g
// s'_{t,g}, so that W_t fits binary16 whatever the values' scale, and
// it is raised only when a W_t would pass 2^15 (a warp vote), then so that the
// largest becomes 2^7: weights down to 2^-21 of the largest keep all their bits.
// The exponent is the exact product less m, as long as m is small: from 2^12 on a
// warp rounds every product first, as its steps with masked tokens always do, so
// that equal scores have equal weights in all steps; and from 2^24 on, where the
// rounding of m could take a weight out of binary16's range, m is the largest
// rounded score itself, and the largest W_t the value scale.
// Scores, sums, statistics and outputs are held in binary32.
//
// Work split.  A unit is 32 tokens of one (sequence, block of rows, head); the
// units of the whole batch, in that order, are cut into equal ranges for the
// CTAs (one per SM) and each CTA's range into equal ranges for its warps, so
// ragged batches and single long sequences load every SM alike.  A warp
// streams its range through its own ring in shared memory (bulk copies, one
// mbarrier per stage; nothing in the loop synchronizes warps) and keeps the
// softmax state of its present segment in registers.  A segment that lies in
// one warp's range is written at once; pieces of the others meet in shared
// memory at the CTA's end, and where a segment spans CTAs, as partial results
// in the workspace, which the last CTA to arrive adds in CTA order.  No CTA
// waits for another, and every sum has a fixed order, so results are
// deterministic.
//
// Measured on B200 (8 kv heads, 4 query heads each, D = 128, G = 64): 128
// sequences of 2,048 to 8,192 tokens (763 MB) 206 us, 3.7 TB/s; the copies alone
// with the same plan take 134 us.  What bounds it: about 440 warp instructions
// per 16 tokens and head, half of them unpack and products, the rest scores,
// weights, copies and plan, at 2.2 a cycle (issue 56 %, ALU 44 % of active cycles);
// short batches by the chain of dependent steps (sequence length, page number,
// copy, one unit, two merges: 10.1 us for one sequence of 1,000 tokens).  Tried
// and slower: one warp that issues all copies (58 -> 69 us for a quarter of the
// batch: its lanes serve few warps at a time), 16 warps (spills) and 8 warps
// (latency shows) where there is work for 12; without effect: accumulators
// that start at the zero correction, one more pass that takes the scale out of
// every score.
#pragma once

#include "kv4.cuh"
#include "unpack.cuh"

namespace wq {
namespace kv4 {

constexpr int kUnit = 32;      // tokens of a unit
constexpr int kMaxCtas = 160;  // CTAs the workspace has room for
constexpr int kMaxRows = 16;   // rows of a block

// Quotient by a divisor known at launch, for 0 <= n < 2^31.
struct FastDiv {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return int((__umulhi(uint32_t(n), mul) + uint32_t(n)) >> shift);
  }
};

struct AttnParams {
  Cache cache;
  Batch batch;
  const __nv_bfloat16* Q;  // [rows][q_heads][D], rows q_stride elements apart
  int64_t q_stride;
  __nv_bfloat16* O;  // [rows][q_heads][D], rows o_stride elements apart
  int64_t o_stride;
  int gqa;            // query heads per kv head
  int max_columns;    // sequences with more rows times gqa are another kernel's
  FastDiv by_gqa;
  float scale_log2;   // softmax scale times log2 e
  // Test hooks of the timeout path (set only through an internal export): the
  // CTA whose copies never count as complete (-1: none; they are made all the
  // same), and the limit of the kernels' waits, in nanoseconds.
  int test_stuck_cta;
  unsigned int wait_ns;
  unsigned* arrived;  // [kMaxCtas][kMaxRows] zero counters
  float* partial;     // [2 kMaxCtas][piece]
};

template <int D, int G, int NT, int WARPS>
struct AttnConfig {
  static constexpr int kChunks = D / 32;
  static constexpr int kGroups = D / G;
  static constexpr int kRows = 8 * NT;
  static constexpr int kThreads = WARPS * 32;
  static constexpr int kCodeBytes = kUnit * D / 2;
  static constexpr int kMetaBytes = kUnit * kGroups * 4;
  static constexpr int kStageBytes = 2 * (kCodeBytes + kMetaBytes);
  // a piece: O [rows][D], m [rows], l [rows]
  static constexpr int kPieceFloats = kRows * (D + 2);
  static constexpr int kPieceBytes = kPieceFloats * 4;
  static constexpr int kCtlBytes = 8192;
  // as many stages of each warp's ring as fit, four at most; the last piece
  // of a warp reuses its drained ring
  static constexpr int kFit = (232448 - kCtlBytes) / WARPS - kPieceBytes;
  static constexpr int kStages = kFit / kStageBytes < 4 ? kFit / kStageBytes : 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static_assert(kStages >= 2 && kRingBytes >= kPieceBytes && kRingBytes % 16 == 0 &&
                    kPieceBytes % 16 == 0,
                "");
  static constexpr int kOffHead = WARPS * kRingBytes;
  static constexpr int kOffCtl = kOffHead + WARPS * kPieceBytes;
  static constexpr int kPartialBytes = 2 * kMaxCtas * kPieceBytes;
};

// One (sequence, block of rows, head): its units are [u0, u0 + units) of the
// batch's.
struct Segment {
  int b, rb, h;
  int row0, rows, len;  // of the sequence
  int limit;            // tokens that some row of the block sees
  int units;            // of one head of this block of rows
  int64_t u0;
};

struct PieceInfo {
  int rb, h, row0, rows;
  int64_t u0, u1;
};

template <int WARPS>
struct AttnControl {
  uint64_t full[WARPS][4];
  int64_t warp_sum[WARPS];
  int64_t upto[WARPS * 32];     // inclusive prefix of a thread inside its warp
  unsigned pieces[WARPS];       // 1: head, 2: tail of a warp
  PieceInfo head[WARPS], tail[WARPS];
};

// Sequence b with its rows, none if it is another kernel's.
__device__ __forceinline__ Sequence attn_sequence(const AttnParams& p, int b) {
  Sequence s = load_sequence(p.batch, b);
  if (s.rows * p.gqa > p.max_columns) s.rows = 0;
  return s;
}

// Tokens that some row of block rb sees.
template <int ROWS>
__device__ __forceinline__ int block_limit(const Sequence& s, int rb, const AttnParams& p) {
  const int last = min(s.rows * p.gqa, (rb + 1) * ROWS) - 1;
  return max(0, s.len - s.rows + p.by_gqa(last) + 1);
}

// The units they make: one at least, so that rows that see nothing are
// written too.
__device__ __forceinline__ int limit_units(int limit) {
  return max(1, (limit + kUnit - 1) / kUnit);
}

template <int ROWS>
__device__ __forceinline__ int row_blocks(const Sequence& s, int gqa) {
  return (s.rows * gqa + ROWS - 1) / ROWS;
}

template <int ROWS>
__device__ __forceinline__ int64_t sequence_units(const AttnParams& p, const Sequence& s) {
  int64_t n = 0;
  const int blocks = row_blocks<ROWS>(s, p.gqa);
  for (int rb = 0; rb < blocks; ++rb) n += limit_units(block_limit<ROWS>(s, rb, p));
  return n * p.cache.kv_heads;
}

// The segment after s (its u0 follows); the caller knows that there is one.
template <int ROWS>
__device__ __forceinline__ void next_segment(const AttnParams& p, Segment& s) {
  s.u0 += s.units;
  if (++s.h < p.cache.kv_heads) return;
  s.h = 0;
  Sequence q = {s.row0, s.rows, s.len};
  if (++s.rb >= row_blocks<ROWS>(q, p.gqa)) {
    s.rb = 0;
    do {
      q = attn_sequence(p, ++s.b);
    } while (q.rows == 0);
    s.row0 = q.row0;
    s.rows = q.rows;
    s.len = q.len;
  }
  s.limit = block_limit<ROWS>(q, s.rb, p);
  s.units = limit_units(s.limit);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Transpose of an 8x8 matrix of binary16 held as pairs (lane (g, t): row g,
// columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// N 32-bit words of shared memory in one load.
template <int N>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x, r[1] = v.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

__device__ __forceinline__ float2 meta_pair(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Offset of row r of the segment that begins at row0, of kv head h.
__device__ __forceinline__ int64_t row_offset(const AttnParams& p, int row0, int r, int h,
                                              int64_t stride, int D) {
  const int i = p.by_gqa(r);
  return int64_t(row0 + i) * stride + int64_t(h * p.gqa + (r - i * p.gqa)) * D;
}

// The reference of a row that has seen no token yet: finite, so that no
// difference of two is NaN, and no larger than any finite score.
constexpr float kNoReference = -0x1.fffffep127f;

// Scores (base 2) from which a binary32 reference cannot be trusted to be
// within a few units of the exact one: half a step is 1 here, 16 at 2^28.
constexpr float kFarScore = 0x1p24f;

// References (base 2) from which the warp-level kernel rounds its products: a
// product of this size rounds by 2^-12.
constexpr float kLargeScore = 0x1p12f;

// The segment of unit q, which is `rem` units behind the first of sequence b,
// and q's place in it.
template <int ROWS>
__device__ __forceinline__ int segment_at(const AttnParams& p, int b, const Sequence& seq,
                                          int64_t rem, int64_t q, Segment* out) {
  Segment s;
  s.b = b;
  s.row0 = seq.row0;
  s.rows = seq.rows;
  s.len = seq.len;
  for (s.rb = 0;; ++s.rb) {
    s.limit = block_limit<ROWS>(seq, s.rb, p);
    s.units = limit_units(s.limit);
    const int64_t n = int64_t(s.units) * p.cache.kv_heads;
    if (rem < n) break;
    rem -= n;
  }
  s.h = rem < (int64_t(1) << 31) ? int(uint32_t(rem) / uint32_t(s.units)) : int(rem / s.units);
  const int unit = int(rem - int64_t(s.h) * s.units);
  s.u0 = q - unit;
  *out = s;
  return unit;
}

// The same for a warp that asks with all its lanes: the block's threads have
// left the prefix sums of their sequences' units in shared memory.
template <int ROWS, int WARPS>
__device__ __forceinline__ int find_segment(const AttnParams& p, const AttnControl<WARPS>& ctl,
                                            int per_thread, int64_t q, int lane, Segment* out) {
  int64_t sum = lane < WARPS ? ctl.warp_sum[lane] : 0;
  const int64_t own = sum;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, sum, m);
    if (lane >= m) sum += v;
  }
  const int w = __ffs(__ballot_sync(0xffffffffu, sum > q)) - 1;
  int64_t rem = q - __shfl_sync(0xffffffffu, sum - own, w);
  const int64_t upto = ctl.upto[w * 32 + lane];
  const int i = __ffs(__ballot_sync(0xffffffffu, upto > rem)) - 1;
  const int64_t before = __shfl_up_sync(0xffffffffu, upto, 1);
  if (i > 0) rem -= __shfl_sync(0xffffffffu, before, i);
  int b = (w * 32 + i) * per_thread;
  Sequence seq = attn_sequence(p, b);
  while (per_thread > 1) {
    const int64_t n = sequence_units<ROWS>(p, seq);
    if (rem < n) break;
    rem -= n;
    seq = attn_sequence(p, ++b);
  }
  return segment_at<ROWS>(p, b, seq, rem, q, out);
}

// Waits, for a limited time each, for the `copies` stages of a ring from `st` on.
static __device__ __noinline__ void wait_for_copies(uint64_t* full, int stages, int st,
                                                    uint32_t parity, int copies,
                                                    unsigned int* status,
                                                    unsigned long long limit_ns) {
  for (; copies > 0; --copies) {
    mbar_wait(&full[st], parity, status, limit_ns);
    if (++st == stages) st = 0, parity ^= 1u;
  }
}

template <int D, int G, int NT, int WARPS, int TILES>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_kernel(const AttnParams p) {
  using C = AttnConfig<D, G, NT, WARPS>;
  constexpr int NC = C::kChunks, NG = C::kGroups, ROWS = C::kRows, NS = C::kStages;
  constexpr int kChunksPerGroup = G / 32;
  static_assert(sizeof(AttnControl<WARPS>) <= C::kCtlBytes, "");
  extern __shared__ __align__(128) unsigned char smem[];
  auto* ctl = reinterpret_cast<AttnControl<WARPS>*>(smem + C::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;

  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&ctl->full[warp][i], 1);
    fence_mbar_init();
    ctl->pieces[warp] = 0u;
  }
  __syncwarp();

  // ---- the units of the batch.  Up to 32 sequences: every warp counts them
  // by itself, lane b sequence b.  More: thread i counts those of a contiguous
  // range of sequences, and the prefix sums meet in shared memory.
  const bool few = p.batch.seqs <= 32;
  const int per_thread = (p.batch.seqs + C::kThreads - 1) / C::kThreads;
  Sequence mine = {0, 0, 0};
  int64_t upto = 0, total = 0;
  if (few) {
    if (lane < p.batch.seqs) {
      mine = attn_sequence(p, lane);
      upto = sequence_units<ROWS>(p, mine);
    }
  } else {
    const int b_begin = min(p.batch.seqs, tid * per_thread);
    const int b_end = min(p.batch.seqs, b_begin + per_thread);
    for (int b = b_begin; b < b_end; ++b) upto += sequence_units<ROWS>(p, attn_sequence(p, b));
  }
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += v;
  }
  if (few) {
    total = __shfl_sync(0xffffffffu, upto, 31);
  } else {
    ctl->upto[tid] = upto;
    if (lane == 31) ctl->warp_sum[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) total += ctl->warp_sum[w];
  }

  // ---- this CTA's range (one unit per warp at least, where the batch has
  // fewer units than warps; the first `extra` CTAs have one more than the
  // others), and its warps'
  const int ctas = int(min(int64_t(gridDim.x), (total + WARPS - 1) / WARPS));
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  const bool narrow = total < (int64_t(1) << 31);
  const int64_t per_cta = narrow ? int64_t(uint32_t(total) / uint32_t(ctas)) : total / ctas;
  const int extra = int(total - per_cta * ctas);
  const int64_t r0 = cta * per_cta + min(cta, extra);
  const int n_cta = int(per_cta) + (cta < extra ? 1 : 0);
  const int64_t r1 = r0 + n_cta;
  const int per_warp = n_cta / WARPS, extra_warps = n_cta - per_warp * WARPS;
  auto warp_begin = [&](int w) { return r0 + w * per_warp + min(w, extra_warps); };

  const int64_t q0 = warp_begin(warp);
  const int n_units = per_warp + (warp < extra_warps ? 1 : 0);
  if (n_units > 0) {
    const int64_t q1 = q0 + n_units;
    unsigned char* const ring = smem + warp * C::kRingBytes;
    Segment cs;  // of the unit being computed
    int unit;
    if (few) {
      const int i = __ffs(__ballot_sync(0xffffffffu, upto > q0)) - 1;
      const int64_t before = __shfl_up_sync(0xffffffffu, upto, 1);
      const int64_t skipped = __shfl_sync(0xffffffffu, before, i);
      const Sequence seq = {__shfl_sync(0xffffffffu, mine.row0, i),
                            __shfl_sync(0xffffffffu, mine.rows, i),
                            __shfl_sync(0xffffffffu, mine.len, i)};
      unit = segment_at<ROWS>(p, i, seq, i > 0 ? q0 - skipped : q0, q0, &cs);
    } else {
      unit = find_segment<ROWS>(p, *ctl, per_thread, q0, lane, &cs);
    }

    // ---- copies.  Lane 4 sub + kind copies the codes or metadata of one run
    // of tokens inside a page; page numbers are read one unit ahead.
    Segment pf = cs;  // of the next unit to copy
    int pf_unit = unit, to_copy = n_units, pf_page = 0;
    const int sub_shift = min(p.cache.page_shift, 5);
    const int kind = lane & 3, sub = lane >> 2;
    const uint32_t row_bytes = kind & 1 ? NG * 4 : D / 2;
    const unsigned char* const copy_src =
        kind == 0   ? p.cache.k_codes
        : kind == 1 ? reinterpret_cast<const unsigned char*>(p.cache.k_meta)
        : kind == 2 ? p.cache.v_codes
                    : reinterpret_cast<const unsigned char*>(p.cache.v_meta);
    unsigned char* const copy_dst = ring + (kind >> 1) * (C::kCodeBytes + C::kMetaBytes) +
                                    (kind & 1) * C::kCodeBytes +
                                    (sub << sub_shift) * int(row_bytes);
    const uint64_t policy = l2_policy_evict_first();
    auto read_page = [&] {
      const int pos = pf_unit * kUnit + (sub << sub_shift);
      if (sub < (kUnit >> sub_shift) && pos < pf.limit)
        pf_page = p.batch.page_table[int64_t(pf.b) * p.batch.table_stride +
                                     (pos >> p.cache.page_shift)];
    };
    auto copy_unit = [&](int s) {
      const int tok0 = pf_unit * kUnit;
      const int subs = max(0, min(kUnit >> sub_shift,
                                  (pf.limit - tok0 + (1 << sub_shift) - 1) >> sub_shift));
      if (lane == 0)
        mbar_arrive_expect_tx(&ctl->full[warp][s],
                              uint32_t(subs) * uint32_t((2 * (NG * 4 + D / 2)) << sub_shift));
      __syncwarp();
      if (sub < subs) {
        if (uint32_t(pf_page) >= uint32_t(p.cache.pages)) {
          record_status(kStatusInvalid, p.batch.status);
          pf_page = 0;  // any page of the cache can be read
        }
        const int64_t token =
            ((int64_t(pf_page) * p.cache.kv_heads + pf.h) << p.cache.page_shift) +
            ((tok0 + (sub << sub_shift)) & ((1 << p.cache.page_shift) - 1));
        bulk_load(copy_dst + s * C::kStageBytes, copy_src + token * row_bytes,
                  row_bytes << sub_shift, &ctl->full[warp][s], policy);
      }
      if (--to_copy > 0) {
        if (++pf_unit == pf.units) {
          next_segment<ROWS>(p, pf);
          pf_unit = 0;
        }
        read_page();
      }
    };
    // Queries of column g of a segment.  Where registers allow it they are
    // loaded before the copies wait for their page numbers.
    constexpr bool kAhead = NT == 1 && WARPS == 8;
    uint4 raw[NC];
    auto load_queries = [&](int nt) {
      const int r = cs.rb * ROWS + nt * 8 + g;
      const __nv_bfloat16* row = p.Q + row_offset(p, cs.row0, r, cs.h, p.q_stride, D) + 8 * t;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (r < cs.rows * p.gqa) raw[j] = *reinterpret_cast<const uint4*>(row + 32 * j);
      }
    };
    read_page();
    if (kAhead) load_queries(0);
    // (at the kernel's start, where the parameters are not in the constant cache
    // yet, this comparison cost 0.4 us)
    if (int(blockIdx.x) == p.test_stuck_cta && tid == 0) mbar_expect_tx(&ctl->full[0][0], 16u);
    for (int s = 0; s < NS - 1; ++s)
      if (to_copy > 0) copy_unit(s);

    // ---- state of the present segment
    float O[2 * NC][NT][4];  // m-tile i: dims 32(i/2) + 4g + 2(i%2) + {0, 1}; columns 2t, 2t + 1
    uint32_t q[NT][2 * NC][2];
    float sum_q[NT][NG][2], q_scale[NT][2], m[NT][2], l[NT][2], zc[NT][NG][2];
    int limit[NT][2], seen_by_all = 0;
    bool fresh = true, large = false;

    // lane group g holds tokens pi(g) and pi(g) + 8 of each 16: with this
    // order of the tokens the value loads below touch every bank group
    const int tok_a = 2 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));
    // columns 2t, 2t + 1 (and + 8) of the value operand: tokens pi(2t), pi(2t + 1)
    const int tok_v0 = 2 * t + (t & 1), tok_v1 = 2 * t + 1 - (t & 1);

    int st = 0;
    uint32_t parity = 0;
    for (int left = n_units; left > 0; --left) {
      // the stage freed by the previous unit
      if (to_copy > 0) copy_unit(st == 0 ? NS - 1 : st - 1);
      bool raise = fresh;
      if (fresh) {
        fresh = large = false;
        seen_by_all = cs.len - cs.rows + p.by_gqa(cs.rb * ROWS) + 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // ---- queries of column g, scaled to binary16
          if (!kAhead) load_queries(nt);
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = bf16x2_to_float2(w[k]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int exponent = int(__float_as_uint(top) >> 23);  // biased
          const int up = top > 0.f ? min(141 - exponent, 126) : 0;
          // the sign of the softmax scale goes to the queries
          const float mult =
              copysignf(__uint_as_float(uint32_t(up + 127) << 23), p.scale_log2);
          float sums[NG];
#pragma unroll
          for (int k = 0; k < NG; ++k) sums[k] = 0.f;
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = bf16x2_to_float2(w[k]);
              f[2 * k] = __half2float(__float2half_rn(v.x * mult));
              f[2 * k + 1] = __half2float(__float2half_rn(v.y * mult));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sums[j / kChunksPerGroup] += f[k];
            // operand pairs in the order of the codes' unpack: (0, 4), (1, 5), ...
            q[nt][2 * j][0] = pack_half2(f[0], f[4]);
            q[nt][2 * j][1] = pack_half2(f[1], f[5]);
            q[nt][2 * j + 1][0] = pack_half2(f[2], f[6]);
            q[nt][2 * j + 1][1] = pack_half2(f[3], f[7]);
          }
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], 1);
            sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], 2);
#pragma unroll
            for (int c = 0; c < 2; ++c)
              sum_q[nt][k][c] = __shfl_sync(0xffffffffu, sums[k], (2 * t + c) * 4);
          }
          const float qs = fabsf(p.scale_log2) * __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            q_scale[nt][c] = __shfl_sync(0xffffffffu, qs, (2 * t + c) * 4);
            const int rc = cs.rb * ROWS + nt * 8 + 2 * t + c;
            limit[nt][c] = rc < cs.rows * p.gqa ? cs.len - cs.rows + p.by_gqa(rc) + 1 : 0;
            m[nt][c] = kNoReference;
            l[nt][c] = 0.f;
#pragma unroll
            for (int k = 0; k < NG; ++k) zc[nt][k][c] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) O[k][nt][c] = 0.f;
        }
      }

      if (!__all_sync(0xffffffffu, mbar_wait(&ctl->full[warp][st], parity, p.batch.status,
                                             p.wait_ns))) {
        // given up: no more copies, and none in flight when the warp's ring is used
        // for a piece or the CTA ends
        wait_for_copies(ctl->full[warp], NS, st, parity, left - to_copy, p.batch.status, p.wait_ns);
        break;
      }
      const unsigned char* const stage = ring + st * C::kStageBytes;
      const int tok0 = unit * kUnit;
      // tokens that every row of the block sees need no mask
      bool masked = large || tok0 + kUnit > seen_by_all;

#pragma unroll
      for (int h0 = 0; h0 < 2; h0 += TILES) {
      // ---- scores (base 2) of TILES times 16 tokens
      float x[TILES][NT][4];  // tokens a, a, b, b; columns 2t, 2t + 1
      uint32_t vm[TILES][2][NG];
      // the tiles' chains of products interleave; a single group's is cut in two
      constexpr int ACC = NG == 1 ? 2 : NG;
      float acc[TILES][NT][ACC][4];
      uint32_t wa[TILES][NC], wb[TILES][NC], km[TILES][2][NG];
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        const int ta = 16 * (h0 + h) + tok_a;
        load_words<NC>(stage + ta * (D / 2) + t * NC * 4, wa[h]);
        load_words<NC>(stage + (ta + 8) * (D / 2) + t * NC * 4, wb[h]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_words<NG>(stage + C::kCodeBytes + (ta + 8 * i) * NG * 4, km[h][i]);
          load_words<NG>(stage + 2 * C::kCodeBytes + C::kMetaBytes + (ta + 8 * i) * NG * 4,
                         vm[h][i]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < ACC; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[h][nt][k][c] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        constexpr bool kCut = NG == 1;
        const int k0 = kCut ? 0 : j / kChunksPerGroup, k1 = kCut ? 1 : k0;
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
          uint32_t ua[4], ub[4];
          unpack_u4_h<8>(wa[h][j], ua);
          unpack_u4_h<8>(wb[h][j], ub);
          const uint32_t a0[4] = {ua[0], ub[0], ua[1], ub[1]};
          const uint32_t a1[4] = {ua[2], ub[2], ua[3], ub[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(acc[h][nt][k0], a0, q[nt][2 * j]);
            mma_f16_16816(acc[h][nt][k1], a1, q[nt][2 * j + 1]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        const int ta = 16 * (h0 + h) + tok_a;
        if (NG == 1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[h][nt][0][c] += acc[h][nt][ACC - 1][c];
        }
        if (masked) {
          // tokens that no row of the block sees may not have been copied, and what
          // lies behind the end of a sequence can be anything, NaN included
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (tok0 + ta + 8 * i >= cs.limit)
#pragma unroll
              for (int k = 0; k < NG; ++k) km[h][i][k] = vm[h][i][k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = meta_pair(km[h][i][k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float y = fmaf(8.f - f.y, sum_q[nt][k][c], acc[h][nt][k][2 * i + c]);
                x[h][nt][2 * i + c] = k == 0 ? f.x * y : fmaf(f.x, y, x[h][nt][2 * i + c]);
              }
          }
        if (masked) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[h][nt][c] = tok0 + ta + 8 * (c >> 1) >= limit[nt][c & 1]
                                ? -INFINITY
                                : x[h][nt][c] * q_scale[nt][c & 1];
        }
      }

      // ---- weights.  The reference m is raised where a segment begins and
      // when a weight passes 2^15, so that the largest becomes 2^7, and the
      // unit's weights are formed again.
      float scale[NT][2];  // of the scores (masked ones have it already)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) scale[nt][c] = masked ? 1.f : q_scale[nt][c];
      uint32_t w16[TILES][2][NG][NT];  // pairs (columns 2t, 2t + 1) of tokens a and b
      while (true) {
        if (raise) {
          float lw[TILES][2];  // log2 of the largest value scale of a token
#pragma unroll
          for (int h = 0; h < TILES; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = meta_pair(vm[h][i][0]).x;
#pragma unroll
              for (int k = 1; k < NG; ++k) top = fmaxf(top, meta_pair(vm[h][i][k]).x);
              lw[h][i] = log2_approx(top);
            }
          float next[NT][2], most_next = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = -INFINITY;
#pragma unroll
              for (int h = 0; h < TILES; ++h)
                top = fmaxf(top, fmaxf(fmaf(x[h][nt][c], scale[nt][c], lw[h][0]),
                                       fmaf(x[h][nt][c + 2], scale[nt][c], lw[h][1])));
#pragma unroll
              for (int d = 4; d < 32; d *= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              next[nt][c] = fmaxf(m[nt][c], top - 7.f);
              if (next[nt][c] != kNoReference) most_next = fmaxf(most_next, fabsf(next[nt][c]));
            }
          if (__any_sync(0xffffffffu, most_next >= kLargeScore)) {
            // rounded products from here to the segment's end
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float high = -INFINITY;
#pragma unroll
                for (int h = 0; h < TILES; ++h)
#pragma unroll
                  for (int i = 0; i < 4; i += 2) {
                    x[h][nt][c + i] = __fmul_rn(x[h][nt][c + i], scale[nt][c]);
                    high = fmaxf(high, x[h][nt][c + i]);
                  }
#pragma unroll
                for (int d = 4; d < 32; d *= 2)
                  high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
                scale[nt][c] = 1.f;
                if (fabsf(next[nt][c]) >= kFarScore) next[nt][c] = fmaxf(m[nt][c], high);
              }
            masked = large = true;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float f = exp2_approx(m[nt][c] - next[nt][c]);
              m[nt][c] = next[nt][c];
              l[nt][c] *= f;
#pragma unroll
              for (int k = 0; k < NG; ++k) zc[nt][k][c] *= f;
#pragma unroll
              for (int k = 0; k < 2 * NC; ++k) {
                O[k][nt][c] *= f;
                O[k][nt][c + 2] *= f;
              }
            }
        }
        float l_next[NT][2], zc_next[NT][NG][2];
        uint32_t most[NT];  // the largest weights (none is negative) of two columns
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            most[nt] = 0u;
            l_next[nt][c] = l[nt][c];
#pragma unroll
            for (int k = 0; k < NG; ++k) zc_next[nt][k][c] = zc[nt][k][c];
          }
#pragma unroll
        for (int h = 0; h < TILES; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float e[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                e[c] = exp2_approx(fmaf(x[h][nt][2 * i + c], scale[nt][c], -m[nt][c]));
                l_next[nt][c] += e[c];
              }
#pragma unroll
              for (int k = 0; k < NG; ++k) {
                const float2 f = meta_pair(vm[h][i][k]);
                const float w0 = e[0] * f.x, w1 = e[1] * f.x;
                zc_next[nt][k][0] = fmaf(w0, f.y - 8.f, zc_next[nt][k][0]);
                zc_next[nt][k][1] = fmaf(w1, f.y - 8.f, zc_next[nt][k][1]);
                w16[h][i][k][nt] = pack_half2(w0, w1);
                most[nt] = hmax2(most[nt], w16[h][i][k][nt]);
              }
            }
        // 0x7800 is 2^15; a NaN (above infinity, 0x7c00) raises nothing
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t hi = most[nt] >> 16, lo = most[nt] & 0xffffu;
          over |= (hi > 0x7800u && hi <= 0x7c00u) || (lo > 0x7800u && lo <= 0x7c00u);
        }
        raise = !raise && over;
        if (!__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              l[nt][c] = l_next[nt][c];
#pragma unroll
              for (int k = 0; k < NG; ++k) zc[nt][k][c] = zc_next[nt][k][c];
            }
          break;
        }
        raise = true;
      }

      // ---- values
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        uint32_t b[NG][NT][2];
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) b[k][nt][i] = transpose8x8(w16[h][i][k][nt]);
        constexpr int VW = NC / 2;  // words of a lane and token
        const unsigned char* const vbase = stage + C::kCodeBytes + C::kMetaBytes +
                                           16 * (h0 + h) * (D / 2) + g * NC * 2;
        uint32_t x0[VW], x1[VW], x2[VW], x3[VW];
        load_words<VW>(vbase + tok_v0 * (D / 2), x0);
        load_words<VW>(vbase + tok_v1 * (D / 2), x1);
        load_words<VW>(vbase + (tok_v0 + 8) * (D / 2), x2);
        load_words<VW>(vbase + (tok_v1 + 8) * (D / 2), x3);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          uint32_t ua[4], ub[4];
          unpack_u4_h<8>(__byte_perm(x0[j / 2], x1[j / 2], sel), ua);
          unpack_u4_h<8>(__byte_perm(x2[j / 2], x3[j / 2], sel), ub);
          const uint32_t a0[4] = {ua[0], ua[1], ub[0], ub[1]};
          const uint32_t a1[4] = {ua[2], ua[3], ub[2], ub[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(O[2 * j][nt], a0, b[j / kChunksPerGroup][nt]);
            mma_f16_16816(O[2 * j + 1][nt], a1, b[j / kChunksPerGroup][nt]);
          }
        }
      }
        raise = false;
      }
      __syncwarp();  // the stage may be refilled
      if (++st == NS) {
        st = 0;
        parity ^= 1u;
      }

      // ---- end of the segment, or of this warp's part of it
      if (unit + 1 == cs.units || left == 1) {
        const int64_t u1 = cs.u0 + cs.units;
        const bool from_before = cs.u0 < q0;
        const bool whole = !from_before && u1 <= q1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
              l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], d);
#pragma unroll
              for (int k = 0; k < NG; ++k)
                zc[nt][k][c] += __shfl_xor_sync(0xffffffffu, zc[nt][k][c], d);
            }
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) {
              O[k][nt][c] -= zc[nt][k / 2 / kChunksPerGroup][c];
              O[k][nt][c + 2] -= zc[nt][k / 2 / kChunksPerGroup][c];
            }
          }
        if (whole) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int r = cs.rb * ROWS + nt * 8 + 2 * t + c;
              if (r >= cs.rows * p.gqa) continue;
              const float inv = l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];
              __nv_bfloat16* row = p.O + row_offset(p, cs.row0, r, cs.h, p.o_stride, D) + 4 * g;
#pragma unroll
              for (int j = 0; j < NC; ++j)
                *reinterpret_cast<uint2*>(row + 32 * j) = make_uint2(
                    pack_bf162(O[2 * j][nt][c] * inv, O[2 * j][nt][c + 2] * inv),
                    pack_bf162(O[2 * j + 1][nt][c] * inv, O[2 * j + 1][nt][c + 2] * inv));
            }
        } else {
          float* piece = reinterpret_cast<float*>(
              from_before ? smem + C::kOffHead + warp * C::kPieceBytes : ring);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int rl = nt * 8 + 2 * t + c;
#pragma unroll
              for (int j = 0; j < NC; ++j)
                *reinterpret_cast<float4*>(piece + rl * D + 32 * j + 4 * g) =
                    make_float4(O[2 * j][nt][c], O[2 * j][nt][c + 2], O[2 * j + 1][nt][c],
                                O[2 * j + 1][nt][c + 2]);
              if (g == 0) {
                piece[ROWS * D + rl] = m[nt][c];
                piece[ROWS * D + ROWS + rl] = l[nt][c];
              }
            }
          if (lane == 0) {
            (from_before ? ctl->head : ctl->tail)[warp] = {cs.rb,   cs.h,  cs.row0,
                                                           cs.rows, cs.u0, u1};
            ctl->pieces[warp] |= from_before ? 1u : 2u;
          }
        }
        if (left > 1) {
          next_segment<ROWS>(p, cs);
          unit = 0;
          fresh = true;
          if (kAhead) load_queries(0);
        }
      } else {
        ++unit;
      }
    }
  }

  // ---- pieces of segments that span warps.  Chain 0 is the segment that
  // began before this CTA; chain w + 1 the one that begins in warp w and goes
  // on.  A warp adds one row of one chain at a time, in warp order; where the
  // segment spans CTAs the row's sums go to the workspace, and the warp that
  // is the last of all CTAs' to bring that row adds them, in CTA order.
  __syncthreads();
  constexpr int VF = D / 32;  // floats of a lane
  const unsigned kinds = lane < WARPS ? ctl->pieces[lane] : 0u;
  const unsigned has_head = __ballot_sync(0xffffffffu, kinds & 1u);
  const unsigned has_tail = __ballot_sync(0xffffffffu, kinds & 2u);
  const int first = has_head ? __ffs(has_head) - 1 : 0;
  // the segment that began before this CTA is the first warp's with units
  const bool from_before = has_head != 0u && ctl->head[first].u0 < r0;
  int task = 0;
  for (unsigned todo = (has_tail << 1) | (from_before ? 1u : 0u); todo != 0u; todo &= todo - 1u) {
    const int chain = __ffs(todo) - 1;
    const PieceInfo s = chain == 0 ? ctl->head[first] : ctl->tail[chain - 1];
    const int rows = min(ROWS, s.rows * p.gqa - s.rb * ROWS);
    // lane w holds the statistics of warp w's piece
    const bool is_tail = lane == chain - 1;
    const bool mine = is_tail || (lane < WARPS && lane >= max(chain, first) &&
                                  ((has_head >> lane) & 1u) != 0u && ctl->head[lane].u0 == s.u0);
    const unsigned char* piece = is_tail ? smem + lane * C::kRingBytes
                                         : smem + C::kOffHead + lane * C::kPieceBytes;
    const unsigned pieces = __ballot_sync(0xffffffffu, mine);
    for (int rl = 0; rl < rows; ++rl, ++task) {
      if (task % WARPS != warp) continue;
      const float* stats = reinterpret_cast<const float*>(piece) + ROWS * D + rl;
      const float own_m = mine ? stats[0] : kNoReference;
      float top = own_m;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float weight = mine ? exp2_approx(own_m - top) : 0.f;
      float l = mine ? weight * stats[ROWS] : 0.f;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
      float o[VF];
#pragma unroll
      for (int k = 0; k < VF; ++k) o[k] = 0.f;
#pragma unroll 4
      for (int w = 0; w < WARPS; ++w) {
        const float f = __shfl_sync(0xffffffffu, weight, w);
        if (!((pieces >> w) & 1u)) continue;
        uint32_t v[VF];
        load_words<VF>((w == chain - 1 ? smem + w * C::kRingBytes
                                       : smem + C::kOffHead + w * C::kPieceBytes) +
                           (rl * D + lane * VF) * 4,
                       v);
#pragma unroll
        for (int k = 0; k < VF; ++k) o[k] = fmaf(f, __uint_as_float(v[k]), o[k]);
      }
      if (s.u0 < r0 || s.u1 > r1) {
        auto slot = [&](int c, bool begins) {
          return p.partial + (2 * int64_t(c) + (begins ? 1 : 0)) * C::kPieceFloats;
        };
        float* to = slot(cta, s.u0 >= r0);
#pragma unroll
        for (int k = 0; k < VF; ++k) __stcg(to + rl * D + lane * VF + k, o[k]);
        if (lane == 0) {
          __stcg(to + ROWS * D + rl, top);
          __stcg(to + ROWS * D + ROWS + rl, l);
        }
        // the CTAs of the segment's first and last unit
        const int64_t wide = extra * (per_cta + 1);  // units of the CTAs with one more
        auto cta_of = [&](int64_t u) {
          const int64_t a = u < wide ? u : u - wide, n = u < wide ? per_cta + 1 : per_cta;
          return (u < wide ? 0 : extra) + (narrow ? int(uint32_t(a) / uint32_t(n)) : int(a / n));
        };
        const int c0 = s.u0 >= r0 ? cta : cta_of(s.u0);
        const int c1 = s.u1 <= r1 ? cta : cta_of(s.u1 - 1);
        __syncwarp();
        unsigned before = 0u;
        if (lane == 0) {
          __threadfence();
          before = atomicAdd(&p.arrived[c0 * kMaxRows + rl], 1u);
          __threadfence();
        }
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before != unsigned(c1 - c0)) continue;
        __syncwarp();  // lane 0's fence holds for the other lanes' loads
        // every CTA of the segment has brought its row
        if (lane == 0) p.arrived[c0 * kMaxRows + rl] = 0u;
        constexpr int kAtOnce = 8;
        top = kNoReference;
        l = 0.f;
#pragma unroll
        for (int k = 0; k < VF; ++k) o[k] = 0.f;
        for (int base = c0; base <= c1; base += kAtOnce) {
          float v[kAtOnce][VF];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const float* from = slot(min(base + i, c1), base + i == c0) + rl * D + lane * VF;
#pragma unroll
            for (int k = 0; k < VF / 2; ++k) {
              const float2 f = __ldcg(reinterpret_cast<const float2*>(from) + k);
              v[i][2 * k] = f.x, v[i][2 * k + 1] = f.y;
            }
          }
          const int c = base + lane;
          const bool there = lane < kAtOnce && c <= c1;
          const float* from = slot(min(c, c1), c == c0) + ROWS * D + rl;
          const float m_c = there ? __ldcg(from) : kNoReference;
          const float l_c = there ? __ldcg(from + ROWS) : 0.f;
          float next = fmaxf(top, m_c);
#pragma unroll
          for (int d = 1; d < 32; d *= 2)
            next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, d));
          const float keep = exp2_approx(top - next);
          const float w_c = there ? exp2_approx(m_c - next) : 0.f;
          float add = w_c * l_c;
#pragma unroll
          for (int d = 1; d < kAtOnce; d *= 2) add += __shfl_xor_sync(0xffffffffu, add, d);
          l = fmaf(l, keep, __shfl_sync(0xffffffffu, add, 0));
#pragma unroll
          for (int k = 0; k < VF; ++k) o[k] *= keep;
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const float f = __shfl_sync(0xffffffffu, w_c, i);
#pragma unroll
            for (int k = 0; k < VF; ++k) o[k] = fmaf(f, v[i][k], o[k]);
          }
          top = next;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t* to = reinterpret_cast<uint32_t*>(
          p.O + row_offset(p, s.row0, s.rb * ROWS + rl, s.h, p.o_stride, D) + lane * VF);
#pragma unroll
      for (int k = 0; k < VF / 2; ++k) to[k] = pack_bf162(o[2 * k] * inv, o[2 * k + 1] * inv);
    }
  }
}

}  // namespace kv4
}  // namespace wq
