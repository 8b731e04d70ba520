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
// s'_{t,g}, so that the largest W_t is near 1 whatever the values' scale, and
// it is raised only when a W_t would pass 2^8 (a warp vote; binary16 holds
// 2^15).  Scores, sums, statistics and outputs are held in binary32.
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
#pragma once

#include "kv4.cuh"
#include "unpack.cuh"

namespace wq {
namespace kv4 {

constexpr int kUnit = 32;      // tokens of a unit
constexpr int kMaxCtas = 160;  // CTAs the workspace has room for

struct AttnParams {
  Cache cache;
  Batch batch;
  const __nv_bfloat16* Q;  // [rows][q_heads][D], rows q_stride elements apart
  int64_t q_stride;
  __nv_bfloat16* O;  // [rows][q_heads][D], rows o_stride elements apart
  int64_t o_stride;
  int gqa;            // query heads per kv head
  float scale_log2;   // softmax scale times log2 e
  unsigned* arrived;  // [kMaxCtas] zero counters
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
  // the last piece of a warp reuses its drained ring
  static constexpr int kStages = D == 64 ? 4 : (WARPS == 8 ? 4 : 2);
  static constexpr int kRingBytes = kStages * kStageBytes;
  static_assert(kRingBytes >= kPieceBytes && kRingBytes % 16 == 0 && kPieceBytes % 16 == 0, "");
  static constexpr int kOffHead = WARPS * kRingBytes;
  static constexpr int kOffBars = kOffHead + WARPS * kPieceBytes;
  static constexpr int kOffCtl = kOffBars + WARPS * kStages * 8;
  static constexpr int kPartialBytes = 2 * kMaxCtas * kPieceBytes;
};

// One (sequence, block of rows, head): its units are [u0, u0 + units) of the
// batch's.
struct Segment {
  int b, rb, h;
  int row0, rows, len;  // of the sequence
  int units;            // of one head of this block of rows
  int64_t u0;
};

struct PieceInfo {
  int valid;
  int b, rb, h;
  int row0, rows;
  int64_t u0, u1;
};

template <int WARPS>
struct AttnControl {
  int64_t warp_sum[WARPS];
  int64_t start_rem[WARPS];  // units from the start of sequence start_b
  int start_b[WARPS];
  int last[2];
  PieceInfo head[WARPS], tail[WARPS];
};

// Tokens that some row of block rb sees, and the units they make (one at
// least, so that rows that see nothing are written too).
template <int ROWS>
__device__ __forceinline__ int block_limit(const Sequence& s, int rb, int gqa) {
  const int last = min(s.rows * gqa, (rb + 1) * ROWS) - 1;
  return max(0, s.len - s.rows + last / gqa + 1);
}

template <int ROWS>
__device__ __forceinline__ int block_units(const Sequence& s, int rb, int gqa) {
  return max(1, (block_limit<ROWS>(s, rb, gqa) + kUnit - 1) / kUnit);
}

template <int ROWS>
__device__ __forceinline__ int row_blocks(const Sequence& s, int gqa) {
  return (s.rows * gqa + ROWS - 1) / ROWS;
}

template <int ROWS>
__device__ __forceinline__ int64_t sequence_units(const AttnParams& p, int b) {
  const Sequence s = load_sequence(p.batch, b);
  int64_t n = 0;
  const int blocks = row_blocks<ROWS>(s, p.gqa);
  for (int rb = 0; rb < blocks; ++rb) n += block_units<ROWS>(s, rb, p.gqa);
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
      q = load_sequence(p.batch, ++s.b);
    } while (q.rows == 0);
    s.row0 = q.row0;
    s.rows = q.rows;
    s.len = q.len;
  }
  s.units = block_units<ROWS>(q, s.rb, p.gqa);
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

// Transpose of an 8x8 matrix of binary16 held as pairs (lane (g, t): row g,
// columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// N 32-bit words of shared memory in one load.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    const uint4 v = lds128(addr);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    r[0] = v.x, r[1] = v.y;
  } else {
    r[0] = lds32(addr);
  }
}

__device__ __forceinline__ float2 meta_pair(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The (row, query head) of a row r of a segment.
__device__ __forceinline__ int64_t row_offset(int row0, int r, int h, int gqa, int64_t stride,
                                              int D) {
  return int64_t(row0 + r / gqa) * stride + int64_t(h * gqa + r % gqa) * D;
}

template <int D, int G, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_kernel(const AttnParams p) {
  using C = AttnConfig<D, G, NT, WARPS>;
  constexpr int NC = C::kChunks, NG = C::kGroups, ROWS = C::kRows, NS = C::kStages;
  constexpr int kChunksPerGroup = G / 32;
  extern __shared__ __align__(128) unsigned char smem[];
  auto* ctl = reinterpret_cast<AttnControl<WARPS>*>(smem + C::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int gqa = p.gqa;
  unsigned char* ring = smem + warp * C::kRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBars) + warp * NS;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    ctl->head[warp].valid = 0;
    ctl->tail[warp].valid = 0;
  }

  // ---- this CTA's and its warps' ranges of units.  Thread i counts the units
  // of a contiguous range of sequences; the thread whose range holds a warp's
  // first unit finds its sequence.
  const int per_thread = (p.batch.seqs + C::kThreads - 1) / C::kThreads;
  const int b_begin = min(p.batch.seqs, tid * per_thread);
  const int b_end = min(p.batch.seqs, b_begin + per_thread);
  int64_t own = 0;
  for (int b = b_begin; b < b_end; ++b) own += sequence_units<ROWS>(p, b);
  int64_t upto = own;  // inclusive prefix
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += v;
  }
  if (lane == 31) ctl->warp_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) upto += ctl->warp_sum[w];
    total += ctl->warp_sum[w];
  }
  // one unit per warp at least, where the batch has fewer units than warps
  const int64_t ctas = min(int64_t(gridDim.x), (total + WARPS - 1) / WARPS);
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  const int64_t r0 = cta * total / ctas, r1 = (cta + 1) * total / ctas;
  auto warp_begin = [&](int w) { return r0 + w * (r1 - r0) / WARPS; };
  if (own > 0) {
    for (int w = 0; w < WARPS; ++w) {
      const int64_t q = warp_begin(w);
      if (q < upto - own || q >= upto) continue;
      int64_t rem = q - (upto - own);
      int b = b_begin;
      for (;; ++b) {
        const int64_t n = sequence_units<ROWS>(p, b);
        if (rem < n) break;
        rem -= n;
      }
      ctl->start_b[w] = b;
      ctl->start_rem[w] = rem;
    }
  }
  __syncthreads();
  const int64_t q0 = warp_begin(warp), q1 = warp_begin(warp + 1);

  if (q0 < q1) {
    // ---- the first segment
    Segment pf;  // of the next unit to copy
    int pf_unit;
    {
      pf.b = ctl->start_b[warp];
      int64_t rem = ctl->start_rem[warp];
      const Sequence s = load_sequence(p.batch, pf.b);
      pf.row0 = s.row0;
      pf.rows = s.rows;
      pf.len = s.len;
      pf.rb = 0;
      for (;; ++pf.rb) {
        pf.units = block_units<ROWS>(s, pf.rb, gqa);
        const int64_t n = int64_t(pf.units) * p.cache.kv_heads;
        if (rem < n) break;
        rem -= n;
      }
      pf.h = int(rem / pf.units);
      pf_unit = int(rem % pf.units);
      pf.u0 = q0 - pf_unit;
    }
    Segment cs = pf;  // of the unit being computed
    int cs_unit = pf_unit;

    const int sub_shift = min(p.cache.page_shift, 5);  // a copy stays inside one page
    const int sub_tokens = 1 << sub_shift;
    const uint32_t smem_ring = smem_addr(ring);
    const uint64_t policy = l2_policy_evict_first();
    int64_t to_copy = q1 - q0;

    // Starts the copies of the next unit into stage `s`: lane 4 sub + kind
    // copies the codes or metadata of one run of tokens inside a page.
    auto copy_unit = [&](int s) {
      const Sequence seq = {pf.row0, pf.rows, pf.len};
      const int limit = block_limit<ROWS>(seq, pf.rb, gqa);
      const int tok0 = pf_unit * kUnit;
      const int subs = min(kUnit >> sub_shift, (limit - tok0 + sub_tokens - 1) >> sub_shift);
      const int kind = lane & 3, sub = lane >> 2;
      const uint32_t row_bytes = kind & 1 ? NG * 4 : D / 2;
      if (lane == 0) {
        const uint32_t bytes =
            uint32_t(max(subs, 0)) * uint32_t(sub_tokens) * uint32_t(2 * (NG * 4 + D / 2));
        mbar_arrive_expect_tx(&bars[s], bytes);
      }
      __syncwarp();
      if (sub < subs) {
        const int pos = tok0 + sub * sub_tokens;
        int64_t page = load_page(p.batch, p.cache, pf.b, pos);
        if (page < 0) page = 0;  // recorded; any page of the cache can be read
        const int64_t token = ((page * p.cache.kv_heads + pf.h) << p.cache.page_shift) +
                              (pos & ((1 << p.cache.page_shift) - 1));
        const unsigned char* base =
            kind == 0   ? p.cache.k_codes
            : kind == 1 ? reinterpret_cast<const unsigned char*>(p.cache.k_meta)
            : kind == 2 ? p.cache.v_codes
                        : reinterpret_cast<const unsigned char*>(p.cache.v_meta);
        const int off = (kind >> 1) * (C::kCodeBytes + C::kMetaBytes) +
                        (kind & 1) * C::kCodeBytes + sub * sub_tokens * int(row_bytes);
        bulk_load(ring + s * C::kStageBytes + off, base + token * row_bytes,
                  uint32_t(sub_tokens) * row_bytes, &bars[s], policy);
      }
      --to_copy;
      if (++pf_unit == pf.units && to_copy > 0) {
        next_segment<ROWS>(p, pf);
        pf_unit = 0;
      }
    };

    // ---- state of the present segment
    float O[2 * NC][NT][4];   // m-tile i: dims 32(i/2) + 4g + 2(i%2) + {0, 1}; columns 2t, 2t + 1
    uint32_t q[NT][2 * NC][2];
    float sum_q[NT][NG][2], q_scale[NT][2], m[NT][2], l[NT][2], zc[NT][NG][2];
    int limit[NT][2];
    bool fresh = true, alive = true;

    for (int s = 0; s < NS - 1; ++s)
      if (to_copy > 0) copy_unit(s);

    const int64_t n = q1 - q0;
    for (int64_t i = 0; i < n; ++i) {
      const int st = int(i % NS);
      // the stage freed by the previous unit
      if (to_copy > 0) copy_unit(int((i + NS - 1) % NS));

      if (fresh) {
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // ---- queries of column g, scaled to binary16
          const int r = cs.rb * ROWS + nt * 8 + g;
          const bool have = r < cs.rows * gqa;
          uint4 raw[NC];
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            raw[j] = make_uint4(0, 0, 0, 0);
            if (have)
              raw[j] = *reinterpret_cast<const uint4*>(
                  p.Q + row_offset(cs.row0, r, cs.h, gqa, p.q_stride, D) + 32 * j + 8 * t);
          }
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
          const float mult = __uint_as_float(uint32_t(up + 127) << 23);
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
          const float qs = p.scale_log2 * __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            q_scale[nt][c] = __shfl_sync(0xffffffffu, qs, (2 * t + c) * 4);
            const int rc = cs.rb * ROWS + nt * 8 + 2 * t + c;
            limit[nt][c] = rc < cs.rows * gqa ? cs.len - cs.rows + rc / gqa + 1 : 0;
            m[nt][c] = -INFINITY;
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

      if (alive) alive = mbar_wait(&bars[st], uint32_t(i / NS) & 1u);
      const uint32_t stage = smem_ring + st * C::kStageBytes;
      const int tok0 = cs_unit * kUnit;
      // tokens that every row of the block sees need no mask
      const int seen_by_all = cs.len - cs.rows + (cs.rb * ROWS) / gqa + 1;
      const bool masked = tok0 + kUnit > seen_by_all;

      // lane group g holds tokens pi(g) and pi(g) + 8 of each 16: with this
      // order of the tokens the value loads below touch every bank group
      const int tok_a = 2 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[NT][4];  // scores, then weights; tokens a, a, b, b
        float vs[2][NG], vz[2][NG];
        const int ta = 16 * h + tok_a;
        uint32_t wa[NC], wb[NC], ma[NG], mb[NG];
        lds_words<NC>(stage + ta * (D / 2) + t * NC * 4, wa);
        lds_words<NC>(stage + (ta + 8) * (D / 2) + t * NC * 4, wb);
        lds_words<NG>(stage + C::kCodeBytes + ta * NG * 4, ma);
        lds_words<NG>(stage + C::kCodeBytes + (ta + 8) * NG * 4, mb);
        float acc[NT][NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < NG; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[nt][k][c] = 8.f * sum_q[nt][k][c & 1];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          uint32_t ua[4], ub[4];
          unpack_u4_h<8>(wa[j], ua);
          unpack_u4_h<8>(wb[j], ub);
          const uint32_t a0[4] = {ua[0], ub[0], ua[1], ub[1]};
          const uint32_t a1[4] = {ua[2], ub[2], ua[3], ub[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(acc[nt][j / kChunksPerGroup], a0, q[nt][2 * j]);
            mma_f16_16816(acc[nt][j / kChunksPerGroup], a1, q[nt][2 * j + 1]);
          }
        }
        uint32_t va[NG], vb[NG];
        lds_words<NG>(stage + 2 * C::kCodeBytes + C::kMetaBytes + ta * NG * 4, va);
        lds_words<NG>(stage + 2 * C::kCodeBytes + C::kMetaBytes + (ta + 8) * NG * 4, vb);
        if (masked) {
          // what lies behind the sequence's end can be anything, NaN included
          if (tok0 + ta >= cs.len)
#pragma unroll
            for (int k = 0; k < NG; ++k) ma[k] = va[k] = 0u;
          if (tok0 + ta + 8 >= cs.len)
#pragma unroll
            for (int k = 0; k < NG; ++k) mb[k] = vb[k] = 0u;
        }
        float lw[2] = {0.f, 0.f};  // the largest value scale of tokens a and b
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const float2 fa = meta_pair(va[k]), fb = meta_pair(vb[k]);
          vs[0][k] = fa.x, vz[0][k] = fa.y - 8.f;
          vs[1][k] = fb.x, vz[1][k] = fb.y - 8.f;
          lw[0] = fmaxf(lw[0], fa.x);
          lw[1] = fmaxf(lw[1], fb.x);
        }
        lw[0] = log2_approx(lw[0]);
        lw[1] = log2_approx(lw[1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[nt][c] = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const float2 fa = meta_pair(ma[k]), fb = meta_pair(mb[k]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 f = c < 2 ? fa : fb;
              x[nt][c] = fmaf(f.x, fmaf(-f.y, sum_q[nt][k][c & 1], acc[nt][k][c]), x[nt][c]);
            }
        }
        // scores in base 2, masked; the reference m rises only when a weight
        // would pass 2^8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[nt][c] *= q_scale[nt][c & 1];
            if (masked && tok0 + ta + 8 * (c >> 1) >= limit[nt][c & 1]) x[nt][c] = -INFINITY;
          }
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) rise |= x[nt][c] + lw[c >> 1] > m[nt][c & 1] + 8.f;
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(x[nt][c] + lw[0], x[nt][c + 2] + lw[1]);
#pragma unroll
              for (int d = 4; d < 32; d *= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              const float next = fmaxf(m[nt][c], top);
              const float f = next == -INFINITY ? 1.f : exp2_approx(m[nt][c] - next);
              m[nt][c] = next;
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
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float ref = m[nt][c & 1] == -INFINITY ? 0.f : m[nt][c & 1];
            x[nt][c] = exp2_approx(x[nt][c] - ref);
            l[nt][c & 1] += x[nt][c];
          }
        // ---- values of these 16 tokens
        uint32_t b[NG][NT][2];
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              w[c] = x[nt][c] * vs[c >> 1][k];
              zc[nt][k][c & 1] = fmaf(w[c], vz[c >> 1][k], zc[nt][k][c & 1]);
            }
            b[k][nt][0] = transpose8x8(pack_half2(w[0], w[1]));
            b[k][nt][1] = transpose8x8(pack_half2(w[2], w[3]));
          }
        // columns k = 2t, 2t + 1, 2t + 8, 2t + 9 of the operand are tokens
        // pi(2t), pi(2t + 1) and those + 8
        const int t0 = 16 * h + 2 * t + (t & 1), t1 = 16 * h + 2 * t + 1 - (t & 1);
        constexpr int VW = NC / 2;  // words of a lane and token
        const uint32_t vbase = stage + C::kCodeBytes + C::kMetaBytes + g * NC * 2;
        uint32_t x0[VW], x1[VW], x2[VW], x3[VW];
        lds_words<VW>(vbase + t0 * (D / 2), x0);
        lds_words<VW>(vbase + t1 * (D / 2), x1);
        lds_words<VW>(vbase + (t0 + 8) * (D / 2), x2);
        lds_words<VW>(vbase + (t1 + 8) * (D / 2), x3);
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
      __syncwarp();  // the stage may be refilled

      // ---- end of the segment, or of this warp's part of it
      const bool last = i + 1 == n;
      if (cs_unit + 1 == cs.units || last) {
        const int64_t u1 = cs.u0 + cs.units;
        const bool from_before = cs.u0 < q0, goes_on = u1 > q1;
        const bool whole = !from_before && !goes_on;
        float* piece = from_before ? reinterpret_cast<float*>(smem + C::kOffHead) +
                                         warp * C::kPieceFloats
                                   : reinterpret_cast<float*>(ring);
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
            const int rl = nt * 8 + 2 * t + c, r = cs.rb * ROWS + rl;
            const float inv = l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];
#pragma unroll
            for (int j = 0; j < NC; ++j) {
              const float z = zc[nt][j / kChunksPerGroup][c];
              const float4 o = make_float4(O[2 * j][nt][c] - z, O[2 * j][nt][c + 2] - z,
                                           O[2 * j + 1][nt][c] - z, O[2 * j + 1][nt][c + 2] - z);
              if (!whole) {
                *reinterpret_cast<float4*>(piece + rl * D + 32 * j + 4 * g) = o;
              } else if (r < cs.rows * gqa) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
                *reinterpret_cast<uint2*>(
                    p.O + row_offset(cs.row0, r, cs.h, gqa, p.o_stride, D) + 32 * j + 4 * g) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                               *reinterpret_cast<const uint32_t*>(&hi));
              }
            }
            if (!whole && g == 0) {
              piece[ROWS * D + rl] = m[nt][c];
              piece[ROWS * D + ROWS + rl] = l[nt][c];
            }
          }
        if (!whole && lane == 0) {
          PieceInfo& info = from_before ? ctl->head[warp] : ctl->tail[warp];
          info = {1, cs.b, cs.rb, cs.h, cs.row0, cs.rows, cs.u0, u1};
        }
        if (!last) {
          next_segment<ROWS>(p, cs);
          cs_unit = 0;
          fresh = true;
        }
      } else {
        ++cs_unit;
      }
    }
  }

  // ---- pieces of segments that span warps.  Chain 0 is the segment that
  // began before this CTA; chain w + 1 the one that begins in warp w and goes
  // on.  A warp adds one row of one chain at a time, in warp order.
  __syncthreads();
  constexpr int VF = D / 32;  // floats of a lane
  auto head_piece = [&](int w) {
    return reinterpret_cast<const float*>(smem + C::kOffHead) + w * C::kPieceFloats;
  };
  auto tail_piece = [&](int w) {
    return reinterpret_cast<const float*>(smem + w * C::kRingBytes);
  };
  auto slot = [&](int64_t i) { return p.partial + i * C::kPieceFloats; };
  auto store_row = [&](const PieceInfo& s, int rl, const float (&o)[VF], float l) {
    const int r = s.rb * ROWS + rl;
    if (r >= s.rows * gqa) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[VF / 2];
#pragma unroll
    for (int k = 0; k < VF / 2; ++k) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(
        p.O + row_offset(s.row0, r, s.h, gqa, p.o_stride, D) + lane * VF);
#pragma unroll
    for (int k = 0; k < VF / 2; ++k) to[k] = w[k];
  };
  int first = 0;  // the first warp with units
  while (first < WARPS - 1 && warp_begin(first + 1) == r0) ++first;
  for (int task = warp; task < (WARPS + 1) * ROWS; task += WARPS) {
    const int chain = task / ROWS, rl = task % ROWS;
    const PieceInfo& s = chain == 0 ? ctl->head[first] : ctl->tail[chain - 1];
    if (!s.valid || s.rb * ROWS + rl >= s.rows * gqa) continue;
    float top = -INFINITY;
    auto each = [&](auto&& f) {
      if (chain != 0) f(tail_piece(chain - 1));
      for (int w = chain == 0 ? first : chain; w < WARPS; ++w) {
        const int64_t at = warp_begin(w);
        if (at >= s.u1) break;
        if (at < warp_begin(w + 1)) f(head_piece(w));
      }
    };
    each([&](const float* f) { top = fmaxf(top, f[ROWS * D + rl]); });
    float o[VF], l = 0.f;
#pragma unroll
    for (int k = 0; k < VF; ++k) o[k] = 0.f;
    each([&](const float* f) {
      const float m = f[ROWS * D + rl];
      const float weight = m == -INFINITY ? 0.f : exp2_approx(m - top);
      l = fmaf(weight, f[ROWS * D + ROWS + rl], l);
#pragma unroll
      for (int k = 0; k < VF; ++k) o[k] = fmaf(weight, f[rl * D + lane * VF + k], o[k]);
    });
    if (s.u0 >= r0 && s.u1 <= r1) {
      store_row(s, rl, o, l);
    } else {
      float* to = slot(2 * cta + (s.u0 < r0 ? 0 : 1));
#pragma unroll
      for (int k = 0; k < VF; ++k) to[rl * D + lane * VF + k] = o[k];
      if (lane == 0) {
        to[ROWS * D + rl] = top;
        to[ROWS * D + ROWS + rl] = l;
      }
    }
  }

  // ---- segments that span CTAs: the last to arrive adds their partial sums
  auto cta_of = [&](int64_t u) { return int(((u + 1) * ctas - 1) / total); };
  int open = -1;  // the warp whose tail goes on into the next CTA
  for (int w = 0; w < WARPS; ++w)
    if (ctl->tail[w].valid && ctl->tail[w].u1 > r1) open = w;
  const bool spans[2] = {ctl->head[first].valid != 0 && ctl->head[first].u0 < r0, open >= 0};
  if (!spans[0] && !spans[1]) return;
  __syncthreads();
  if (tid == 0) {
    __threadfence();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ctl->last[k] = 0;
      if (!spans[k]) continue;
      const PieceInfo& s = k == 0 ? ctl->head[first] : ctl->tail[open];
      const int c0 = cta_of(s.u0), c1 = cta_of(s.u1 - 1);
      const unsigned before = atomicAdd(&p.arrived[c0], 1u);
      if (before == unsigned(c1 - c0)) {
        p.arrived[c0] = 0u;  // every CTA of the segment has arrived
        ctl->last[k] = 1;
      }
    }
    __threadfence();
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!spans[k] || !ctl->last[k]) continue;
    const PieceInfo& s = k == 0 ? ctl->head[first] : ctl->tail[open];
    const int c0 = cta_of(s.u0), c1 = cta_of(s.u1 - 1);
    for (int rl = warp; rl < ROWS; rl += WARPS) {
      if (s.rb * ROWS + rl >= s.rows * gqa) break;
      float top = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32)
        top = fmaxf(top, __ldcg(slot(2 * c + (c == c0 ? 1 : 0)) + ROWS * D + rl));
#pragma unroll
      for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float o[VF], l = 0.f;
#pragma unroll
      for (int j = 0; j < VF; ++j) o[j] = 0.f;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const float* f = slot(2 * c + (c == c0 ? 1 : 0));
        const float m = __ldcg(f + ROWS * D + rl);
        const float weight = m == -INFINITY ? 0.f : exp2_approx(m - top);
        l = fmaf(weight, __ldcg(f + ROWS * D + ROWS + rl), l);
#pragma unroll
        for (int j = 0; j < VF; ++j)
          o[j] = fmaf(weight, __ldcg(f + rl * D + lane * VF + j), o[j]);
      }
      store_row(s, rl, o, l);
    }
  }
}

}  // namespace kv4
}  // namespace wq
