// kv4_prefill.cuh -- attention of many query rows per sequence over the 4-bit
// cache (chunks, whole prompts) on the fifth generation tensor cores.
//
// One CTA computes up to 256 rows (query tokens times the heads that share a
// kv head) of one sequence and kv head, as two tiles of 128 rows that take
// turns on the tensor cores, over all the tokens they see, 128 at a time:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread owns a row (a lane of
//                   tensor memory), so row maxima and sums need no exchange;
//   warps 8-11      dequantize: a token's codes from global memory (one tile
//                   ahead in registers) to binary16 values s (u - z) in shared
//                   memory, 128-byte swizzled, two stages each of keys and
//                   values;
//   warp 12         one thread issues tcgen05.mma: S_i = Q_i K^T (both operands
//                   in shared memory) and O_i += P_i V (P_i in tensor memory,
//                   written over S_i by the softmax), 512 columns in all:
//                   S_0, S_1, O_0, O_1.
// Keys and values share one image in shared memory, [token][64 dims] rows of
// 128 bytes: it is the K-major operand of the first product (k = dims) and the
// MN-major operand of the second (n = dims).  The eight dims of a 16-byte
// chunk keep the order of the codes' unpack (0, 4, 1, 5, 2, 6, 3, 7): the
// query tile is stored in the same order and the output put back at the end.
//
// Roundings.  Queries: scaled by a power of two per row to [2^14, 2^15) and
// rounded to binary16 (exact for every bfloat16 within 2^-21 of the row's
// largest).  Keys and values: s (u - z) rounded once to binary16 (2^-11 half
// step; exact where it is subnormal, since s is a multiple of 2^-24).  A token's
// key or value with a scale of 4368 or more, the only ones that can pass 65504, is
// halved, and the softmax doubles its score or its weight; what other groups of
// that key or value hold near binary16's smallest rounds by 2^-24 then.  Nothing
// that is not halved is touched by it, in the same tile or otherwise.  Weights:
// 2^(S - m) rounded to
// binary16; the reference m is raised only when the weights of a step would add
// up to more than 2^15, then so that the largest becomes 2^7 (and the row's
// output is rescaled), or 1 where scores reach 2^24.
// Products, sums and statistics in binary32.
//
// Work split.  Where the blocks of 256 rows do not fill half of the SMs, each
// block's tokens are divided among `splits` CTAs.  A softmax warp then leaves
// its rows' sums in the workspace, and the warp that is the last of all splits'
// to bring its 32 rows adds them in split order (no CTA waits for another).
//
// What bounds it.  Per 256 rows x 128 tokens (D = 128) the tensor cores need
// 2,048 cycles and the exponentials (16 a cycle) as many; a step takes about
// 4,200.  Each tile is a chain of softmax (2,000 cycles), two products (1,700
// while the other roles load shared and tensor memory; 1,024 alone) and
// hand-overs, and the two tiles' softmax warps share their schedulers with the
// dequantize warps.  Measured on B200: a prompt of 8,192 tokens, 32 query heads
// on 8 kv heads (550 GFLOP) 573 us alone, ten in a row (960 TFLOP/s), 615 to 630
// in a longer run, whose clocks are lower (875-895).  (A form of 580 us alone:
// without dequantizing 515, without softmax 430, without both 410.)  Tried and
// slower: polling instead of suspended waits
// (620-670), handing over half of the weights early (730), scores of half
// steps ahead of the products (750: both softmax groups then run at once),
// dequantizing on three schedulers only (630), a quarter of the exponentials
// as a polynomial (580).
#pragma once

#include <type_traits>

#include "gemm2.cuh"
#include "kv4_attn.cuh"

namespace wq {
namespace kv4 {

using gemm::fence_async_shared;
using gemm::tc_commit;
using gemm::tc_fence_after;
using gemm::tc_fence_before;
using gemm::tmem_ld32;
using gemm::tmem_wait_ld;
using gemm::tmem_wait_st;
using gemm2::tc_mma_ts;
using gemm2::tmem_st16;

constexpr int kTile = 128;       // rows of a tile, tokens of a step
constexpr int kBlockRows = 256;  // rows of a CTA
constexpr int kPrefillThreads = 16 * 32;  // four warpgroups; the last has one busy warp
// Scales from 4368 on (the binary16 after 4364) can stand for values past
// 65504: 15 * 4364 = 65460.
constexpr uint32_t kWideScaleBits = 0x6C44u;

// Whether a token's key or value is halved (scale bits in the low halves).
template <int NG>
__device__ __forceinline__ bool is_wide(const uint32_t (&meta)[NG]) {
  uint32_t most = meta[0];
#pragma unroll
  for (int k = 1; k < NG; ++k) most = hmax2(most, meta[k]);
  return (most & 0xffffu) >= kWideScaleBits;
}
constexpr int kMmaWarp = 12;

struct PrefillParams {
  AttnParams a;
  int min_columns;  // sequences with fewer rows times heads are left alone
  int splits;        // CTAs that share the tokens of a block (see below)
  float* partial;    // with splits > 1: one slot for each CTA of the grid
};

template <int D>
struct PrefillConfig {
  static constexpr int kHalves = D / 64;                    // 64-dim blocks of a row
  static constexpr int kBlockBytes = kTile * 128;           // one block of a tile
  static constexpr int kTileBytes = kHalves * kBlockBytes;
  static constexpr int kOffQ = 1024;
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;      // 2 stages
  static constexpr int kOffV = kOffK + 2 * kTileBytes;      // 2 stages
  // with the alignment's slack; more than half an SM's, since a second CTA
  // would wait for tensor memory
  static constexpr int kUsed = kOffV + 2 * kTileBytes + 1024;
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

struct PrefillControl {
  uint64_t q_full[2];
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];  // stages
  uint64_t s_full[2], p_full[2], o_done[2];              // tiles
  uint64_t mma_done;
  int wide[4];             // of the last steps: a key or a value is halved
  uint8_t halved[4][2][16];  // which: a bit a token, of keys and of values
  uint32_t tmem;
  int abort;
};

// Shared-memory operand in the 128-byte swizzled layout: lbo is the distance
// of 64-element blocks of a MN-major operand (unused when K-major), 1024 the
// distance of 8-row groups.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t lbo) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// binary16 operands, binary32 accumulator, M = 128; B K-major or MN-major.
__host__ __device__ constexpr uint32_t instr_desc_f16(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
         (uint32_t(kTile >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :
      : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// One thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Whether the predicate holds for any of the `threads` threads of a barrier.
__device__ __forceinline__ bool named_barrier_or(uint32_t id, uint32_t threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(p)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Codes of four tokens, 32 apart, to a tile's values s (u - z), in the unpack's
// order; `put` are the places of the first token's chunks.  WIDE: the tile has
// tokens to halve; the exact u - z is halved, so that the product is rounded once.
template <int NC, int NG, bool VALUES, bool WIDE>
__device__ __forceinline__ void expand_tile(const uint32_t (&code)[4][NC],
                                            const uint32_t (&meta)[4][NG],
                                            const uint32_t (&put)[NC], uint32_t tile) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t f = WIDE && is_wide(meta[u]) ? 0x38003800u : 0x3C003C00u;  // 1/2 or 1
    uint32_t s2 = 0, lo = 0, hi = 0;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (k % (NC / NG) == 0) {
        const uint32_t m = meta[u][k / (NC / NG)], z2 = __byte_perm(m, m, 0x3232);
        s2 = __byte_perm(m, m, 0x1010);
        lo = hadd2(z2, 0x64006400u);  // 1024 + z
        hi = hsub2(0xD400D400u, z2);  // -(64 + z)
        if (WIDE) lo = hmul2(lo, f), hi = hmul2(hi, f);
      }
      // a value word is made of the halfwords of two g (see kv4.cuh)
      const uint32_t word = VALUES ? __byte_perm(code[u][k / 2], code[u][NC / 2 + k / 2],
                                                 (k & 1) ? 0x7632 : 0x5410)
                                   : code[u][k];
      // u - z, times f, of the codes in the low and in the high nibbles of bytes
      auto low = [&](uint32_t w) {
        const uint32_t x = lop3_and_or(w, 0x000F000Fu, 0x64006400u);
        return WIDE ? hfma2(x, f, lo ^ 0x80008000u) : hsub2(x, lo);
      };
      auto high = [&](uint32_t w) {
        const uint32_t x = lop3_and_or(w, 0x00F000F0u, 0x64006400u);
        return hfma2(x, WIDE ? hmul2(f, 0x2C002C00u) : 0x2C002C00u, hi);
      };
      const uint32_t w8 = word >> 8;
      sts128(tile + put[k] + 4096u * u, hmul2(low(word), s2), hmul2(high(word), s2),
             hmul2(low(w8), s2), hmul2(high(w8), s2));
    }
  }
}

// The rows of a block of 256: the blocks of sequence b begin at index
// row_starts[b] gqa / 256 + b, which leaves each sequence at least as many
// indices as it has blocks.
struct Block {
  int b;
  Sequence s;
  int row;       // first row (query token times heads) of the block
  int columns;   // rows of the sequence
};

__device__ __forceinline__ bool find_block(const PrefillParams& p, int index, int lane,
                                           Block* out) {
  const Batch& batch = p.a.batch;
  auto first_block = [&](int b) {
    const int start = batch.row_starts != nullptr
                          ? min(max(batch.row_starts[b], 0), batch.rows)
                          : b * batch.rows_per_seq;
    return start * p.a.gqa / kBlockRows + b;
  };
  int lo = 0, n = batch.seqs;  // the largest b with first_block(b) <= index
  while (n > 1) {
    const int step = (n + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool below = at < lo + n && first_block(at) <= index;
    const int skip = __popc(__ballot_sync(0xffffffffu, below));
    lo += skip * step;
    n = min(step, n - skip * step);
  }
  out->b = lo;
  out->s = load_sequence(batch, lo);
  out->columns = out->s.rows * p.a.gqa;
  const int rb = index - first_block(lo);
  out->row = rb * kBlockRows;
  return rb >= 0 && out->row < out->columns && out->columns >= p.min_columns;
}

// Waits for a phase; false once any role's wait has run out of time.
__device__ __forceinline__ bool prefill_wait(PrefillControl* ctl, uint64_t* bar, uint32_t parity,
                                             unsigned int* status, unsigned long long limit_ns) {
  volatile int* const abort_flag = &ctl->abort;
  if (mbar_test_wait(bar, parity)) return true;
  if (*abort_flag) return false;
  if (!mbar_wait(bar, parity, status, limit_ns)) {
    *abort_flag = 1;
    return false;
  }
  return true;
}

// The softmax's state of a row, and of its warp: whether a row's reference is
// kFarScore or more, and whether no wait has given up.
struct RowState {
  float m, l;
  bool far, ok;
};

// A step that `weights` did not do: the first, one whose sums passed 2^15, one
// with halved keys or values, and all of a warp with far scores.  Rows with
// `over` get a higher reference, so that the largest weight becomes 2^7, and
// the output so far is put on it; then the weights are formed, once, whatever
// they add up to: nothing here repeats.  `compared` (the same for the warp, whose
// lanes load tensor memory together): whether `over` is known.
//
// weights() subtracts the reference from the exact product.  From kFarScore on
// a rounded reference can be many units off the largest exact product, so there
// it is the largest rounded product itself, and the warp's products are rounded
// before the subtraction, as in a softmax of binary32 scores: the largest weight
// is 1.
//
// A function of its own, so that the usual path has the registers and the
// instruction cache to itself (inlined, a prompt took 4 % longer).
template <int D>
__device__ __noinline__ RowState rare_step(RowState row, PrefillControl* ctl, uint32_t s_tmem,
                                           uint32_t o_tmem, uint64_t* o_done, float c, int j,
                                           int seen, bool wide, bool compared, bool over,
                                           unsigned int* status,
                                           unsigned long long limit_ns) {
  // which of 32 tokens have halved keys (0) or values (1)
  auto halved = [&](int kind, int ch) {
    return *reinterpret_cast<volatile uint32_t*>(&ctl->halved[j & 3][kind][4 * ch]);
  };
  if (wide) {
    // scores of halved keys, doubled where they are
#pragma unroll 1
    for (int k = 0; k < kTile / 16; ++k) {
      const uint32_t bits = halved(0, k >> 1) >> (16 * (k & 1));
      float x[16];
      gemm2::tmem_ld16(s_tmem + 16 * k, x);
      tmem_wait_ld();
      uint32_t r[16];
#pragma unroll
      for (int n = 0; n < 16; ++n)
        r[n] = __float_as_uint((bits >> n) & 1u ? 2.f * x[n] : x[n]);
      tmem_st16(s_tmem + 16 * k, r);
    }
    tmem_wait_st();
  }
  // exponents of 32 tokens' weights; -inf where masked
  auto exponents = [&](int ch, float (&x)[32]) {
    tmem_ld32(s_tmem + 32 * ch, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float e = fmaf(row.far ? __fmul_rn(x[k], c) : x[k], row.far ? 1.f : c, -row.m);
      x[k] = 32 * ch + k < seen ? e : -INFINITY;
    }
  };
  if (!compared) {
    // as in weights(); halved values will double their weights
    float sum = 0.f;
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
      float x[32];
      exponents(ch, x);
#pragma unroll
      for (int k = 0; k < 32; ++k) sum += exp2_approx(x[k]);
    }
    over = sum > 16384.f;
  }
  if (__any_sync(0xffffffffu, over)) {
    float top = -INFINITY;
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
      float x[32];
      tmem_ld32(s_tmem + 32 * ch, x);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (32 * ch + k < seen) top = fmaxf(top, x[k]);
    }
    const float product = __fmul_rn(top, c);
    float next = fabsf(product) >= kFarScore ? product : fmaf(top, c, -7.f);
    if (!over || top == -INFINITY) next = row.m;  // a row that sees nothing has no reference
    row.far = row.far || __any_sync(0xffffffffu, next != row.m && fabsf(next) >= kFarScore);
    const float f = exp2_approx(row.m - next);
    row.m = next;
    row.l *= f;
    if (j > 0) {
      row.ok = __all_sync(0xffffffffu,
                          prefill_wait(ctl, o_done, uint32_t(j - 1) & 1u, status, limit_ns));
      if (!row.ok) return row;
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < D / 16; ++k) {
        float o[16];
        gemm2::tmem_ld16(o_tmem + 16 * k, o);
        tmem_wait_ld();
        uint32_t r[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) r[n] = __float_as_uint(o[n] * f);
        tmem_st16(o_tmem + 16 * k, r);
      }
    }
  }
  float2 sum = make_float2(0.f, 0.f);
  // 32 scores make 16 words: those of chunk ch lie before the scores of ch + 1
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    float x[32];
    exponents(ch, x);
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 e = make_float2(exp2_approx(x[2 * k]), exp2_approx(x[2 * k + 1]));
      sum = add2(sum, e);
      w[k] = pack_half2(e.x, e.y);
    }
    tmem_st16(s_tmem + 16 * ch, w);
  }
  row.l += sum.x + sum.y;
  if (wide) {
    // weights of halved values, doubled
    tmem_wait_st();
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
      const uint32_t bits = halved(1, ch);
      float x[16];
      gemm2::tmem_ld16(s_tmem + 16 * ch, x);
      tmem_wait_ld();
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        w[k] = hmul2(__float_as_uint(x[k]), ((bits >> (2 * k)) & 1u ? 0x4000u : 0x3C00u) |
                                                ((bits >> (2 * k + 1)) & 1u ? 0x40000000u
                                                                            : 0x3C000000u));
      tmem_st16(s_tmem + 16 * ch, w);
    }
  }
  return row;
}

template <int D, int G>
__global__ void __launch_bounds__(kPrefillThreads, 1) prefill_kernel(const PrefillParams p) {
  using C = PrefillConfig<D>;
  constexpr int NC = D / 32, NG = D / G;
  extern __shared__ unsigned char raw_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // the later rows of a sequence see more tokens: they come first
  Block block;
  const int heads = p.a.cache.kv_heads;
  const int cta = int(gridDim.x) - 1 - int(blockIdx.x);
  const int split = cta % p.splits, group = cta / p.splits;
  const int head = group % heads;
  if (!find_block(p, group / heads, lane, &block)) return;
  const Sequence& seq = block.s;
  const int rows = min(kBlockRows, block.columns - block.row);
  const int tiles = rows > kTile ? 2 : 1;
  // tokens the block's last row sees
  const int limit = seq.len - seq.rows + p.a.by_gqa(block.row + rows - 1) + 1;
  const int all_steps = (max(limit, 0) + kTile - 1) / kTile;
  const int splits = max(1, min(p.splits, all_steps));
  if (split >= splits) return;
  // this CTA's steps, and its first token
  const int step0 = int(int64_t(split) * all_steps / splits);
  const int steps = int(int64_t(split + 1) * all_steps / splits) - step0;
  const int token0 = step0 * kTile;

  unsigned char* const smem =
      raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);  // swizzle atoms
  auto* ctl = reinterpret_cast<PrefillControl*>(smem);
  static_assert(sizeof(PrefillControl) <= C::kOffQ, "");
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 4);
      mbar_init(&ctl->k_full[i], cta == p.a.test_stuck_cta ? 5 : 4);
      mbar_init(&ctl->v_full[i], 4);
      mbar_init(&ctl->k_free[i], 1);
      mbar_init(&ctl->v_free[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->o_done[i], 1);
    }
    mbar_init(&ctl->mma_done, 1);
    *reinterpret_cast<volatile int*>(&ctl->abort) = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&ctl->tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&ctl->tmem);

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return prefill_wait(ctl, bar, parity, p.a.batch.status, p.a.wait_ns);
  };

  // Registers: 512 threads at 128; the softmax holds a step's scores and
  // weights.  2 * 128 * 176 + 128 * 104 + 128 * 56 = 65,536 = 512 * 128.
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ---- matrix products.  The whole warp runs the loop, so that descriptors
    // stay in uniform registers; one elected thread issues.
    if (warp == kMmaWarp) {
      constexpr uint32_t kDescQK = instr_desc_f16(kTile, false);
      constexpr uint32_t kDescPV = instr_desc_f16(D, true);
      const uint64_t q_desc = swizzled_desc(smem_addr(smem + C::kOffQ), 16),
                     k_desc = swizzled_desc(smem_addr(smem + C::kOffK), 16),
                     v_desc = swizzled_desc(smem_addr(smem + C::kOffV), C::kBlockBytes);
      const bool leader = elect_one();
      bool ok = true;
      for (int i = 0; i < tiles && ok; ++i) ok = wait(&ctl->q_full[i], 0);
      auto scores = [&](int i, int stage) {
        const uint64_t a = q_desc + uint32_t(i * (C::kTileBytes >> 4)),
                       b = k_desc + uint32_t(stage * (C::kTileBytes >> 4));
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * C::kBlockBytes + (ks & 3) * 32) >> 4;
            tc_mma_ss(tmem + i * kTile, a + off, b + off, kDescQK, ks > 0);
          }
          tc_commit(&ctl->s_full[i]);
        }
        __syncwarp();
      };
      // S_i of step j + 1 follows O_i of step j: it writes over P_i
      if (ok && steps > 0 && (ok = wait(&ctl->k_full[0], 0))) {
        for (int i = 0; i < tiles; ++i) scores(i, 0);
        if (leader) tc_commit(&ctl->k_free[0]);
      }
      for (int j = 0; j < steps && ok; ++j) {
        const int stage = j & 1, next = stage ^ 1;
        const bool more = j + 1 < steps;
        for (int i = 0; i < tiles && ok; ++i) {
          ok = wait(&ctl->p_full[i], uint32_t(j) & 1u) &&
               (i > 0 || wait(&ctl->v_full[stage], uint32_t(j >> 1) & 1u));
          if (!ok) break;
          const uint64_t b = v_desc + uint32_t(stage * (C::kTileBytes >> 4));
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_ts(tmem + 2 * kTile + i * kTile, tmem + i * kTile + ks * 8, b + ks * 128,
                        kDescPV, j > 0 || ks > 0);
            tc_commit(&ctl->o_done[i]);
            if (i == tiles - 1) tc_commit(&ctl->v_free[stage]);
          }
          __syncwarp();
          if (more) {
            if (i == 0) ok = wait(&ctl->k_full[next], uint32_t((j + 1) >> 1) & 1u);
            if (!ok) break;
            scores(i, next);
            if (i == tiles - 1 && leader) tc_commit(&ctl->k_free[next]);
          }
        }
      }
      // all of this CTA's products are done before tensor memory is freed
      if (leader) tc_commit(&ctl->mma_done);
      __syncwarp();
      mbar_wait(&ctl->mma_done, 0, p.a.batch.status, p.a.wait_ns);
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    // ---- keys and values.  Thread (token, t): words t of every chunk of the
    // rows of four tokens of each tile; neighbouring lanes take tokens 4 apart,
    // so that 8 lanes write 8 different bank groups.
    const int t = lane & 3, o = lane >> 2;
    const int perm = 4 * (o & 1) + (o >> 1);
    const int tok = 8 * (warp - 8) + perm;  // and + 32, 64, 96
    const int* const table =
        p.a.batch.page_table + int64_t(block.b) * p.a.batch.table_stride;
    const Cache& cache = p.a.cache;
    const int page_mask = (1 << cache.page_shift) - 1;
    // byte offset of chunk k of token `tok` in a tile; token tok + 32 u follows
    // 4096 u bytes behind
    uint32_t put[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int chunk = 4 * k + t;
      put[k] =
          uint32_t((chunk >> 3) * C::kBlockBytes + tok * 128 + (((chunk & 7) ^ perm) << 4));
    }
    uint32_t kc[4][NC], vc[4][NC], km[4][NG], vm[4][NG];
    int page[4];
    int64_t at[4];  // row of the cache, or -1 behind the last token
    auto read_pages = [&](int j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pos = token0 + j * kTile + 32 * u + tok;
        page[u] = pos < limit ? table[pos >> cache.page_shift] : -1;
      }
    };
    auto read_keys = [&](int j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pos = token0 + j * kTile + 32 * u + tok;
        at[u] = -1;
#pragma unroll
        for (int k = 0; k < NC; ++k) kc[u][k] = 0u;
#pragma unroll
        for (int k = 0; k < NG; ++k) km[u][k] = 0u;
        if (pos >= limit) continue;
        if (uint32_t(page[u]) >= uint32_t(cache.pages)) {
          record_status(kStatusInvalid, p.a.batch.status);
          page[u] = 0;  // any page of the cache can be read
        }
        at[u] = ((int64_t(page[u]) * heads + head) << cache.page_shift) + (pos & page_mask);
        load_words<NC>(cache.k_codes + at[u] * (D / 2) + t * NC * 4, kc[u]);
        load_words<NG>(reinterpret_cast<const unsigned char*>(cache.k_meta + at[u] * NG), km[u]);
      }
    };
    auto read_values = [&] {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int k = 0; k < NC; ++k) vc[u][k] = 0u;
#pragma unroll
        for (int k = 0; k < NG; ++k) vm[u][k] = 0u;
        if (at[u] < 0) continue;
        load_words<NC>(cache.v_codes + at[u] * (D / 2) + t * NC * 4, vc[u]);
        load_words<NG>(reinterpret_cast<const unsigned char*>(cache.v_meta + at[u] * NG), vm[u]);
      }
    };
    if (steps > 0) {
      read_pages(0);
      read_keys(0);
      read_values();
      if (steps > 1) read_pages(1);
    }
    const uint32_t k_tiles = smem_addr(smem + C::kOffK), v_tiles = smem_addr(smem + C::kOffV);
    bool ok = true;
    for (int j = 0; j < steps; ++j) {
      const int stage = j & 1;
      const uint32_t parity = (uint32_t(j >> 1) & 1u) ^ 1u;
      uint32_t most = 0u;  // low half: the scales (positive); high: the zeros
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < NG; ++k) most = hmax2(most, hmax2(km[u][k], vm[u][k]));
      const bool wide = named_barrier_or(1, 128, (most & 0xffffu) >= kWideScaleBits);
      // after a wait that gave up, the loop only keeps the barrier's count
      ok = ok && __all_sync(0xffffffffu, wait(&ctl->k_free[stage], parity));
      if (!ok) continue;
      if (wide) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t keys = __reduce_or_sync(0xffffffffu, is_wide(km[u]) ? 1u << perm : 0u),
                         values = __reduce_or_sync(0xffffffffu, is_wide(vm[u]) ? 1u << perm : 0u);
          if (lane == 0) {
            auto* const to = reinterpret_cast<volatile uint8_t*>(&ctl->halved[j & 3][0][0]);
            to[4 * u + warp - 8] = uint8_t(keys);
            to[16 + 4 * u + warp - 8] = uint8_t(values);
          }
        }
        expand_tile<NC, NG, false, true>(kc, km, put, k_tiles + stage * C::kTileBytes);
      } else {
        expand_tile<NC, NG, false, false>(kc, km, put, k_tiles + stage * C::kTileBytes);
      }
      if (tid == 256) *reinterpret_cast<volatile int*>(&ctl->wide[j & 3]) = wide ? 1 : 0;
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->k_full[stage]);
      if (j + 1 < steps) read_keys(j + 1);

      ok = __all_sync(0xffffffffu, wait(&ctl->v_free[stage], parity));
      if (!ok) continue;
      if (wide)
        expand_tile<NC, NG, true, true>(vc, vm, put, v_tiles + stage * C::kTileBytes);
      else
        expand_tile<NC, NG, true, false>(vc, vm, put, v_tiles + stage * C::kTileBytes);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->v_full[stage]);
      if (j + 1 < steps) {
        read_values();
        if (j + 2 < steps) read_pages(j + 2);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // ---- softmax: this thread's row
    if ((warp >> 2) < tiles) {
    const int i = warp >> 2, local = (warp & 3) * 32 + lane;
    const int r = block.row + i * kTile + local;
    const bool have = i * kTile + local < rows;
    const uint32_t s_tmem = tmem + i * kTile + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t o_tmem = s_tmem + 2 * kTile;
    float c;  // base 2 scale of the row's scores, not negative
    {
      uint4 raw[D / 8];
      const __nv_bfloat16* row = p.a.Q + row_offset(p.a, seq.row0, r, head, p.a.q_stride, D);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        raw[e] = make_uint4(0, 0, 0, 0);
        if (have) raw[e] = *reinterpret_cast<const uint4*>(row + 8 * e);
      }
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const uint32_t w[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = bf16x2_to_float2(w[k]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      const int exponent = int(__float_as_uint(top) >> 23);  // biased
      const int up = top > 0.f ? min(141 - exponent, 126) : 0;
      // the sign of the softmax scale goes to the queries
      const float mult = copysignf(__uint_as_float(uint32_t(up + 127) << 23), p.a.scale_log2);
      c = fabsf(p.a.scale_log2) * __uint_as_float(uint32_t(127 - up) << 23);
      unsigned char* const tile = smem + C::kOffQ + i * C::kTileBytes + local * 128;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const float2 a = bf16x2_to_float2(raw[e].x), b = bf16x2_to_float2(raw[e].y),
                     d = bf16x2_to_float2(raw[e].z), f = bf16x2_to_float2(raw[e].w);
        *reinterpret_cast<uint4*>(tile + (e >> 3) * C::kBlockBytes +
                                  (((e & 7) ^ (local & 7)) << 4)) =
            make_uint4(pack_half2(a.x * mult, d.x * mult), pack_half2(a.y * mult, d.y * mult),
                       pack_half2(b.x * mult, f.x * mult), pack_half2(b.y * mult, f.y * mult));
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[i]);
    }
    const int my_limit = have ? seq.len - seq.rows + p.a.by_gqa(r) + 1 : 0;
    const int least = __reduce_min_sync(0xffffffffu, my_limit);
    float m = kNoReference, l = 0.f;
    bool ok = true;
    bool far = false;  // of the warp: a row's reference is kFarScore or more
    // One step's weights, formed with the row's present reference; they go over
    // the scores in tensor memory.  They do not, and the function returns true,
    // where some row's sum passes 2^15 (*over for this thread's row) or the step is
    // a halved one.  (Following the largest packed weight instead of the sum cost
    // 5 % of the kernel's time; asking for `wide` before the scores are loaded 1 %.)
    auto weights = [&](auto masked_tag, int seen, bool wide, bool* over) {
      constexpr bool kMasked = decltype(masked_tag)::value;
      uint32_t w[4][16];
      float v[2][32];  // each chunk is loaded while the one before it is computed
      tmem_ld32(s_tmem, v[0]);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        float(&x)[32] = v[ch & 1];
        tmem_wait_ld();
        if (ch < 3) tmem_ld32(s_tmem + 32 * (ch + 1), v[(ch + 1) & 1]);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(c, c),
                          make_float2(-m, -m));
          e.x = exp2_approx(e.x);
          e.y = exp2_approx(e.y);
          if (kMasked) {
            if (32 * ch + 2 * k >= seen) e.x = 0.f;
            if (32 * ch + 2 * k + 1 >= seen) e.y = 0.f;
          }
          sum = add2(sum, e);
          w[ch][k] = pack_half2(e.x, e.y);
        }
      }
      // no weight is larger than the sum (a NaN raises nothing)
      *over = sum.x + sum.y > 32768.f;
      if (__builtin_expect(__any_sync(0xffffffffu, *over || wide), 0)) return true;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) tmem_st16(s_tmem + 16 * ch, w[ch]);
      l += sum.x + sum.y;
      return false;
    };
    bool usual = false;  // neither the first step nor far scores
    for (int j = 0; j < steps; ++j) {
      ok = __all_sync(0xffffffffu, wait(&ctl->s_full[i], uint32_t(j) & 1u));
      if (!ok) break;
      tc_fence_after();
      const bool wide = *reinterpret_cast<volatile int*>(&ctl->wide[j & 3]) != 0;
      const int seen = my_limit - token0 - j * kTile;  // columns below `seen` count
      bool over = true, rare = true;
      if (usual)
        rare = token0 + (j + 1) * kTile > least ? weights(std::true_type{}, seen, wide, &over)
                                                : weights(std::false_type{}, seen, wide, &over);
      if (__builtin_expect(rare, 0)) {
        const RowState row =
            rare_step<D>({m, l, far, ok}, ctl, s_tmem, o_tmem, &ctl->o_done[i], c, j, seen, wide,
                         j == 0 || (usual && !wide), over, p.a.batch.status, p.a.wait_ns);
        m = row.m, l = row.l, far = row.far, ok = row.ok;
        usual = !far;
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[i]);
    }
    if (ok && steps > 0)
      ok = __all_sync(0xffffffffu, wait(&ctl->o_done[i], uint32_t(steps - 1) & 1u));
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* row = p.a.O + row_offset(p.a, seq.row0, r, head, p.a.o_stride, D);
      // 32 dims of the row, in the tile's order 0, 4, 1, 5, 2, 6, 3, 7
      auto store = [&](int ch, const float (&v)[32], float inv) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            x[(k >> 1) + 4 * (k & 1)] = inv == 0.f ? 0.f : v[8 * e + k] * inv;
          if (have)
            *reinterpret_cast<uint4*>(row + 32 * ch + 8 * e) =
                make_uint4(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]),
                           pack_bf162(x[4], x[5]), pack_bf162(x[6], x[7]));
        }
      };
      if (splits == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          float v[32];
          if (steps > 0) {
            tmem_ld32(o_tmem + 32 * ch, v);
            tmem_wait_ld();
          }
          store(ch, v, inv);
        }
      } else {
        // a slot: [D / 4][256 rows] of four sums, then m [256], l [256]
        constexpr int kSlot = kBlockRows * (D + 2);
        const int my_row = i * kTile + local;
        auto sums = [&](int c) {
          return reinterpret_cast<float4*>(p.partial + int64_t(group * p.splits + c) * kSlot) +
                 my_row;
        };
        auto stats = [&](int c) {
          return p.partial + int64_t(group * p.splits + c) * kSlot + kBlockRows * D + my_row;
        };
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          float v[32];
          tmem_ld32(o_tmem + 32 * ch, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(sums(split) + (8 * ch + k) * kBlockRows,
                   make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
        }
        __stcg(stats(split), m);
        __stcg(stats(split) + kBlockRows, l);
        __syncwarp();
        unsigned* const arrived = p.a.arrived + group * kMaxRows + warp;
        unsigned before = 0u;
        if (lane == 0) {
          __threadfence();
          before = atomicAdd(arrived, 1u);
          __threadfence();
        }
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == unsigned(splits - 1)) {
          __syncwarp();  // lane 0's fence holds for the other lanes' loads
          if (lane == 0) *arrived = 0u;
          float top = kNoReference;
          for (int c = 0; c < splits; ++c) top = fmaxf(top, __ldcg(stats(c)));
          float all = 0.f;
#pragma unroll 4
          for (int c = 0; c < splits; ++c)
            all = fmaf(exp2_approx(__ldcg(stats(c)) - top), __ldcg(stats(c) + kBlockRows), all);
          const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll 2
            for (int c = 0; c < splits; ++c) {
              const float f = exp2_approx(__ldcg(stats(c)) - top);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 x = __ldcg(sums(c) + (8 * ch + k) * kBlockRows);
                v[4 * k] = fmaf(f, x.x, v[4 * k]);
                v[4 * k + 1] = fmaf(f, x.y, v[4 * k + 1]);
                v[4 * k + 2] = fmaf(f, x.z, v[4 * k + 2]);
                v[4 * k + 3] = fmaf(f, x.w, v[4 * k + 3]);
              }
            }
            store(ch, v, inv);
          }
        }
      }
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

}  // namespace kv4
}  // namespace wq
