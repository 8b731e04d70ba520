// kv4_select.cuh -- which pages of the 4-bit cache a query attends to: bounds of
// the keys of every page, and the choice of the pages whose bounds allow the
// largest scores.
//
// Mathematics.  lo_d and hi_d, the smallest and largest value of dimension d among a
// page's keys of one kv head, bound every score of the page: q . k <= sum_d
// max(q_d lo_d, q_d hi_d).  They are held in 8 bits on the page's grid 2^e, lo rounded
// down and hi up, 2^e the smallest power of two with 127 2^e >= all of them: the
// rounded bounds still hold.  The queries of a kv head's group are rounded to 8 bits
// likewise, q8 = rint(q / 2^e'), with one e' for the group, and a page's score is the
// sum of the heads' bounds,
//   2^e sum_d (Q+_d hi_d + Q-_d lo_d),  Q+ = sum_heads max(q8, 0), Q- = sum_heads min(q8, 0),
// an integer of up to 31 bits (256 heads a group) rounded once to binary32, times
// a power of two.  So the order of pages, ties to the lowest included, is exact and
// independent of how the sum is cut.
#pragma once

#include "kv4.cuh"

namespace wq {
namespace kv4 {

// 2^e of the format for the largest magnitude `top` (normal, or zero: then 1), as the
// biased exponent of a binary32: top = m 2^x, m in [1/2, 1), e = x - 7 where
// m <= 127/128, else x - 6.
__device__ __forceinline__ uint32_t grid_exponent(float top) {
  const uint32_t bits = __float_as_uint(top);
  if (bits == 0u) return 127u;
  const int x = int(bits >> 23) - 126;
  const int e = (bits & 0x7fffffu) <= 0x7e0000u ? x - 7 : x - 6;
  return uint32_t(max(e + 127, 1));
}

constexpr int kBoundThreads = 128;
constexpr int kBoundLoads = 8;  // words of a thread in flight

struct BoundsParams {
  Cache cache;
  Batch batch;
  int8_t* codes;  // [pages][kv_heads][2][D]: lo, hi
  float* grid;    // [pages][kv_heads]: 2^e
  int items;      // rows / page + 2 seqs; the CTAs behind items x kv_heads check the sequences
};

// Bounds of the pages that the batch's rows are in, from the pages' codes: tokens up
// to the sequence's length.  One CTA a page and head.  Sequence b has the items from
// row_starts[b] / page + 2 b on: rows that begin inside a page touch at most
// rows / page + 2 pages.
//
// Bound by the chain length -> page -> codes, 2 us for one page or 128; 4.6 KB read a page
// of 64 and head of 128, all of a thread's loads in flight at once.  A prompt's pages, 100,000
// tokens of 8 heads of 128 (61 MB): 43 us, the same chain once for each of 12,504 CTAs.
template <int D, int G>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const BoundsParams p) {
  constexpr int NC = D / 32, NG = D / G, kWords = D / 8;  // words of a row
  constexpr int kTokens = kBoundThreads / kWords;         // tokens of a pass
  constexpr int kWarps = kBoundThreads / 32;
  __shared__ float lo_s[kWarps][D], hi_s[kWarps][D];
  __shared__ float top_s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = p.cache.page_shift, page_tokens = 1 << shift;
  grid_dependents_launch();
  const int item = int(blockIdx.x) / p.cache.kv_heads;
  const int head = int(blockIdx.x) - item * p.cache.kv_heads;
  if (item >= p.items) {
    const int first = p.items * p.cache.kv_heads;
    check_sequences(p.batch, (int(blockIdx.x) - first) * kWarps + warp,
                    (int(gridDim.x) - first) * kWarps, lane);
    return;
  }
  // ---- the page: the largest b whose items begin at or before this one
  int b;
  int first_item;
  if (p.batch.row_starts == nullptr) {
    const int each = (p.batch.rows_per_seq >> shift) + 2;
    b = item / each;
    first_item = b * each;
    if (b >= p.batch.seqs) return;
  } else {
    auto begin = [&](int s) {
      return (min(max(p.batch.row_starts[s], 0), p.batch.rows) >> shift) + 2 * s;
    };
    int lo = 0, n = p.batch.seqs;
    while (n > 1) {
      const int step = (n + 32) / 33;
      const int at = lo + (lane + 1) * step;
      const bool below = at < lo + n && begin(at) <= item;
      const int skip = __popc(__ballot_sync(0xffffffffu, below));
      lo += skip * step;
      n = min(step, n - skip * step);
    }
    b = lo;
    first_item = begin(b);
  }
  const Sequence seq = load_sequence(p.batch, b);
  if (seq.rows == 0 || item < first_item) return;
  const int64_t pos0 = (int64_t(max(0, seq.len - seq.rows) >> shift) + (item - first_item))
                       << shift;
  if (pos0 >= seq.len) return;
  const int64_t page = load_page(p.batch, p.cache, b, int(pos0));
  if (page < 0) return;
  const int tokens = int(min(int64_t(page_tokens), seq.len - pos0));
  const int64_t row0 = (page * p.cache.kv_heads + head) << shift;

  // ---- this thread's word of every kTokens-th token
  const int word = threadIdx.x % kWords, sub = threadIdx.x / kWords;
  const int chunk = word % NC, dim0 = chunk * 32 + 8 * (word / NC), group = chunk * 32 / G;
  const uint32_t* const codes = reinterpret_cast<const uint32_t*>(p.cache.k_codes) + word;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  for (int t0 = sub; t0 < tokens; t0 += kTokens * kBoundLoads) {
    uint32_t w[kBoundLoads];
    __half2 m[kBoundLoads];
#pragma unroll
    for (int i = 0; i < kBoundLoads; ++i) {
      // behind the last token: the pass's first once more
      const int64_t row = row0 + (t0 + i * kTokens < tokens ? t0 + i * kTokens : t0);
      w[i] = codes[row * kWords];
      m[i] = p.cache.k_meta[row * NG + group];
    }
#pragma unroll
    for (int i = 0; i < kBoundLoads; ++i) {
      const float s = __low2float(m[i]);
      const __half2 zero = __high2half2(m[i]);
      uint32_t u[4];  // elements (0, 4), (1, 5), (2, 6), (3, 7)
      unpack_u4_h<0>(w[i], u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = half2_to_float2(hsub2(u[j], *reinterpret_cast<const uint32_t*>(&zero)));
        const float x = s * f.x, y = s * f.y;
        lo[j] = fminf(lo[j], x), hi[j] = fmaxf(hi[j], x);
        lo[j + 4] = fminf(lo[j + 4], y), hi[j + 4] = fmaxf(hi[j + 4], y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int d = kWords; d < 32; d *= 2) {
      lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], d));
      hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], d));
    }
    if (lane < kWords) lo_s[warp][dim0 + i] = lo[i], hi_s[warp][dim0 + i] = hi[i];
  }
  __syncthreads();
  const int d = threadIdx.x;
  float l = 0.f, h = 0.f, top = 0.f;
  if (d < D) {
    l = lo_s[0][d], h = hi_s[0][d];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) l = fminf(l, lo_s[w][d]), h = fmaxf(h, hi_s[w][d]);
    top = fmaxf(fabsf(l), fabsf(h));
  }
#pragma unroll
  for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  if (lane == 0) top_s[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, top_s[w]);
  const uint32_t e = grid_exponent(top);
  const float inv = __uint_as_float((254u - e) << 23);  // 2^-e: e lies in 2^-31 .. 2^13
  if (d < D) {
    int8_t* const to = p.codes + (page * p.cache.kv_heads + head) * (2 * D) + d;
    to[0] = int8_t(max(-127, min(127, __float2int_rd(l * inv))));
    to[D] = int8_t(max(-127, min(127, __float2int_ru(h * inv))));
  }
  if (threadIdx.x == 0) p.grid[page * p.cache.kv_heads + head] = __uint_as_float(e << 23);
}

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxGroupHeads = 256;    // 127 * 256 fits 16 bits
constexpr int kMaxSelectPages = 53248; // whose keys fit the shared memory of one CTA
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
constexpr int kHeldHeads = 4;          // queries that a thread keeps from one pass to the next

struct SelectParams {
  Batch batch;
  const __nv_bfloat16* Q;
  int64_t q_stride;
  const int8_t* codes;
  const float* grid;
  int64_t pages;
  int page_shift, kv_heads, gqa;
  int max_pages, first, last;
  int rows, ctas;  // ctas: of a cluster
  int* lists;      // [rows][kv_heads][max_pages]
  int* lens;       // [rows]
};

// Order-preserving unsigned of a binary32.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

struct SelectControl {
  uint32_t hist[kBins];
  uint32_t warp_sum[kSelectWarps], low[kSelectWarps], high[kSelectWarps];
  uint32_t bin, above, inside;  // found by one thread
  float top[kSelectWarps];
  int plus[128], minus[128];
  alignas(16) int16_t plus16[128], minus16[128];
};

// The pages of one row and kv head: a cluster of CTAs, each of which scores a slice of the
// sequence's pages (integer dot products of 256 bytes a page, eight lanes a page of 128-wide
// heads) and leaves the keys in the first CTA's shared memory.  That CTA finds the
// smallest key that is chosen, 11 bits of the range of keys a pass -- two passes as a rule,
// since it stops when the pages of a bin are all chosen -- and writes the chosen pages in
// the order of their tokens.
//
// Bound by latency: 2,048 pages of one sequence and head (532 KB) in 8 us on 8 CTAs, of
// which look-ups of the sequence 1.2, queries 0.5, scores 2.1, the keys' range 0.5, two
// passes 1.2, pages 1.5; 128 lists of about 650 pages (21 MB) 11.6 us; 16,384 lists, of a
// prompt's 2,048 rows on up to 512 pages, 513 us.  With histograms of all
// CTAs added through distributed shared memory in four passes of 8 bits it was 20,800
// cycles for the one sequence, half of them the cluster's barriers.
template <int D>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const SelectParams p) {
  constexpr int LPP = D / 16, PPW = 32 / LPP, kUnroll = 2;
  constexpr int kHeadStep = kSelectThreads / D;  // heads that are looked at at once
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelectControl ctl;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  const int unit = int(blockIdx.x) / p.ctas;
  const int r = unit / p.kv_heads, head = unit - r * p.kv_heads;
  if (r >= p.rows) {  // a cluster behind the rows
    check_sequences(p.batch, rank * kSelectWarps + warp, p.ctas * kSelectWarps, lane);
    grid_dependency_wait();
    return;
  }
  grid_dependents_launch();
  if (p.ctas > 1) cluster_arrive();  // the first CTA runs before its shared memory is written
  // ---- queries, on their way while the sequence is looked up
  const __nv_bfloat16* const q =
      p.Q + int64_t(r) * p.q_stride + int64_t(head) * p.gqa * D + tid % D;
  __nv_bfloat16 raw[kHeldHeads];
#pragma unroll
  for (int i = 0; i < kHeldHeads; ++i) {
    const int h = tid / D + i * kHeadStep;
    raw[i] = h < p.gqa ? q[h * D] : __ushort_as_bfloat16(0);
  }
  int* const list = p.lists + int64_t(unit) * p.max_pages;
  const int b = find_sequence(p.batch, r, lane);
  Sequence seq = {0, 0, 0};
  if (b >= 0) seq = load_sequence(p.batch, b);
  const bool mine = b >= 0 && r >= seq.row0 && r < seq.row0 + seq.rows;
  const int limit = mine ? max(0, seq.len - seq.rows + (r - seq.row0) + 1) : 0;
  const int n = int((int64_t(limit) + (1 << p.page_shift) - 1) >> p.page_shift);
  const int count = min(n, p.max_pages);
  if (rank == 0 && head == 0 && tid == 0)
    p.lens[r] = !mine ? -1 : n == 0 ? 0 : limit - ((n - count) << p.page_shift);
  const int* const table = p.batch.page_table + int64_t(max(b, 0)) * p.batch.table_stride;
  if (rank == 0)
    for (int i = count + tid; i < p.max_pages; i += kSelectThreads) list[i] = -1;
  if (n <= p.max_pages) {
    for (int i = tid; rank == 0 && i < n; i += kSelectThreads) {
      const int page = table[i];
      if (page < 0 || page >= p.pages) record_status(kStatusInvalid, p.batch.status);
      list[i] = page;
    }
    if (p.ctas > 1) cluster_wait();
    grid_dependency_wait();  // the grid may not be over before the one that it depends on
    return;
  }
  // ---- pages j0 .. j0 + m - 1 are this CTA's, of those that are not chosen in any case
  const int middle = n - p.first - p.last, wanted = count - p.first - p.last;
  const int per = (middle + p.ctas - 1) / p.ctas;
  const int s0 = min(middle, rank * per), m = min(middle, s0 + per) - s0, j0 = p.first + s0;
  const int part = lane % LPP, own = lane / LPP;
  int next[kUnroll];
  auto read_table = [&](int base) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int j = base + i * PPW + own;
      next[i] = j < m ? table[j0 + j] : 0;
    }
  };
  constexpr int kWarpPages = PPW * kUnroll;
  read_table(warp * kWarpPages);

  // ---- the group's queries: largest magnitude, then the sums of their 8-bit values
  float top = 0.f, held[kHeldHeads];
#pragma unroll
  for (int i = 0; i < kHeldHeads; ++i) {
    held[i] = __bfloat162float(raw[i]);
    top = fmaxf(top, fabsf(held[i]));
  }
  for (int h = tid / D + kHeldHeads * kHeadStep; h < p.gqa; h += kHeadStep)
    top = fmaxf(top, fabsf(__bfloat162float(q[h * D])));
#pragma unroll
  for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  if (lane == 0) ctl.top[warp] = top;
  if (tid < D) ctl.plus[tid] = ctl.minus[tid] = 0;
  for (int i = tid; i < kBins; i += kSelectThreads) ctl.hist[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) top = fmaxf(top, ctl.top[w]);
  {
    // magnitudes whose grid would leave the normal binary32 are raised first, exactly
    const float raise = top < 0x1p-60f ? 0x1p66f : 1.f;
    const float inv = __uint_as_float((254u - grid_exponent(top * raise)) << 23);
    int plus = 0, minus = 0;
    auto add = [&](float x) {
      const int v = max(-127, min(127, __float2int_rn(x * raise * inv)));
      plus += max(v, 0);
      minus += min(v, 0);
    };
#pragma unroll
    for (int i = 0; i < kHeldHeads; ++i) add(held[i]);
    for (int h = tid / D + kHeldHeads * kHeadStep; h < p.gqa; h += kHeadStep)
      add(__bfloat162float(q[h * D]));
    atomicAdd(&ctl.plus[tid % D], plus);
    atomicAdd(&ctl.minus[tid % D], minus);
  }
  __syncthreads();
  if (tid < D) {
    ctl.plus16[tid] = int16_t(ctl.plus[tid]);
    ctl.minus16[tid] = int16_t(ctl.minus[tid]);
  }
  __syncthreads();

  // ---- scores
  int qp[8], qm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qp[i] = reinterpret_cast<const int*>(ctl.plus16)[part * 8 + i];
    qm[i] = reinterpret_cast<const int*>(ctl.minus16)[part * 8 + i];
  }
  if (p.ctas > 1) cluster_wait();
  grid_dependency_wait();  // the bounds (launched as a dependent of their update)
  const uint32_t to =
      p.ctas > 1 ? map_to_rank(smem_addr(keys + s0), 0u) : smem_addr(keys + s0);
  for (int base = warp * kWarpPages; base < m; base += kSelectWarps * kWarpPages) {
    int64_t at[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int page = next[i];
      if (page < 0 || page >= p.pages) {
        record_status(kStatusInvalid, p.batch.status);
        page = 0;  // any page can be read
      }
      at[i] = int64_t(page) * p.kv_heads + head;
    }
    int4 lo[kUnroll], hi[kUnroll];
    float grid[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int4* const box = reinterpret_cast<const int4*>(p.codes + at[i] * (2 * D)) + part;
      lo[i] = __ldg(box);
      hi[i] = __ldg(box + D / 16);
      grid[i] = __ldg(p.grid + at[i]);
    }
    read_table(base + kSelectWarps * kWarpPages);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int l[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
      const int h[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
      int sum = 0, sum_low = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum = __dp2a_lo(qp[2 * k], h[k], sum);
        sum_low = __dp2a_lo(qm[2 * k], l[k], sum_low);
        sum = __dp2a_hi(qp[2 * k + 1], h[k], sum);
        sum_low = __dp2a_hi(qm[2 * k + 1], l[k], sum_low);
      }
      sum += sum_low;
#pragma unroll
      for (int d = 1; d < LPP; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int j = base + i * PPW + own;
      if (part == 0 && j < m) {
        const uint32_t key = order_key(float(sum) * grid[i]);
        if (p.ctas > 1)
          st_dsmem_u32(to + 4u * uint32_t(j), key);
        else
          keys[j] = key;
      }
    }
  }
  if (p.ctas > 1) {
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the range of the keys
  uint32_t low = 0xffffffffu, high = 0u;
  for (int j = tid; j < middle; j += kSelectThreads) {
    low = min(low, keys[j]);
    high = max(high, keys[j]);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) ctl.low[warp] = low, ctl.high[warp] = high;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    low = min(low, ctl.low[w]);
    high = max(high, ctl.high[w]);
  }

  // ---- the smallest chosen key, and how many pages of that key are chosen: in each pass
  // the keys from low on in bins of 2^shift, `above` chosen pages behind the last bin
  int shift = max(0, 32 - __clz(int(high - low)) - kBinBits);
  uint32_t above = 0u, ties = 0u;
  uint32_t span = 0u;  // of the keys looked at: low .. low + span
  for (span = high - low; wanted > 0;) {
    for (int j = tid; j < middle; j += kSelectThreads) {
      const uint32_t off = keys[j] - low;
      if (keys[j] >= low && off <= span) atomicAdd(&ctl.hist[off >> shift], 1u);
    }
    __syncthreads();
    // thread t has bins kBins - 1 - 4 t downwards
    constexpr int kEach = kBins / kSelectThreads;
    uint32_t bins[kEach], sum = 0u;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      bins[i] = ctl.hist[kBins - 1 - (tid * kEach + i)];
      sum += bins[i];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) ctl.warp_sum[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w)
      if (w < warp) upto += ctl.warp_sum[w];
    // the bin in which the last chosen page lies
    uint32_t before = above + upto - sum;
    if (before < uint32_t(wanted) && above + upto >= uint32_t(wanted)) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (before < uint32_t(wanted) && before + bins[i] >= uint32_t(wanted)) {
          ctl.bin = uint32_t(kBins - 1 - (tid * kEach + i));
          ctl.above = before;
          ctl.inside = bins[i];
        }
        before += bins[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) ctl.hist[kBins - 1 - (tid * kEach + i)] = 0u;
    __syncthreads();
    low += ctl.bin << shift;
    above = ctl.above;
    ties = uint32_t(wanted) - above;
    if (shift == 0 || ctl.inside == ties) break;  // one key, or all of the bin
    span = (1u << shift) - 1u;
    shift = max(0, shift - kBinBits);
    __syncthreads();  // the bin has been read
  }
  // chosen: keys above `limit_key`, and the first `ties` of those equal to it
  const bool all = wanted == 0 || shift > 0 || ctl.inside == ties;
  const uint32_t limit_key = wanted == 0 ? 0xffffffffu : all ? low - 1u : low;
  if (all) ties = 0u;

  // ---- the pages.  Warp w has a contiguous part of the middle ones; their places are
  // gathered first, in the histogram's memory, as many as it holds at a time, so that the
  // look-ups in the page table are on their way together.
  const int chunk = ((middle + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int c0 = min(middle, warp * chunk), c1 = min(middle, c0 + chunk);
  uint32_t over = 0u, equal = 0u;
  for (int j = c0 + lane; j - lane < c1; j += 32) {
    const uint32_t key = j < c1 ? keys[j] : 0u;
    over += __popc(__ballot_sync(0xffffffffu, j < c1 && key > limit_key));
    equal += __popc(__ballot_sync(0xffffffffu, j < c1 && key == limit_key));
  }
  __syncthreads();
  if (lane == 0) ctl.warp_sum[warp] = over, ctl.low[warp] = equal;
  __syncthreads();
  over = equal = 0u;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w)
    if (w < warp) over += ctl.warp_sum[w], equal += ctl.low[w];
  for (int g0 = 0; g0 == 0 || g0 < wanted; g0 += kBins) {
    uint32_t passed = over, level = equal;
    for (int j = c0 + lane; j - lane < c1; j += 32) {
      const uint32_t key = j < c1 ? keys[j] : 0u;
      const bool is_over = j < c1 && key > limit_key, is_equal = j < c1 && key == limit_key;
      const uint32_t over_mask = __ballot_sync(0xffffffffu, is_over);
      const uint32_t equal_mask = __ballot_sync(0xffffffffu, is_equal);
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t my_equal = level + __popc(equal_mask & below);
      if (is_over || (is_equal && my_equal < ties)) {
        const int to = int(passed + __popc(over_mask & below) + min(my_equal, ties)) - g0;
        if (to >= 0 && to < kBins) ctl.hist[to] = uint32_t(p.first + j);
      }
      passed += __popc(over_mask);
      level += __popc(equal_mask);
    }
    __syncthreads();
    // the first and the last pages with the first group
    const int from = g0 == 0 ? 0 : p.first + g0;
    const int upto = g0 == 0 ? count : min(p.first + g0 + kBins, count - p.last);
    for (int i = from + tid; i < upto; i += kSelectThreads) {
      const int mid = i - p.first - g0;  // of this group
      int j;
      if (i < p.first)
        j = i;
      else if (i >= count - p.last)
        j = n - (count - i);
      else if (mid < kBins)
        j = int(min(ctl.hist[mid], uint32_t(n - 1)));
      else
        continue;
      const int page = table[j];
      if (page < 0 || page >= p.pages) record_status(kStatusInvalid, p.batch.status);
      list[i] = page;
    }
    __syncthreads();
  }
}

}  // namespace kv4
}  // namespace wq
