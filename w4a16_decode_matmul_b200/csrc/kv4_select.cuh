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
// Bound by the chain length -> page -> codes; 4.6 KB read a page of 64 and head of
// 128, all of a thread's loads in flight at once.
template <int D, int G>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const BoundsParams p) {
  constexpr int NC = D / 32, NG = D / G, kWords = D / 8;  // words of a row
  constexpr int kTokens = kBoundThreads / kWords;         // tokens of a pass
  constexpr int kWarps = kBoundThreads / 32;
  __shared__ float lo_s[kWarps][D], hi_s[kWarps][D];
  __shared__ float top_s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = p.cache.page_shift, page_tokens = 1 << shift;
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

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxGroupHeads = 256;  // 127 * 256 fits 16 bits
constexpr int kDigits = 4;           // radix passes of 8 bits

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
  int* lists;  // [rows][kv_heads][max_pages]
  int* lens;   // [rows]
};

// Order-preserving unsigned of a binary32.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

struct SelectControl {
  uint32_t hist[kDigits][256];
  uint32_t warp_sum[kSelectWarps];
  uint32_t found[2];      // digit, pages above it
  uint32_t counts[2];     // pages of this CTA above the threshold, and at it
  float top[kSelectWarps];
  alignas(16) int16_t plus[128], minus[128];
};

// The pages of one row and kv head: a cluster of CTAs, each with a slice of the
// sequence's pages, whose keys stay in shared memory.  Scores are integer dot products
// of 256 bytes a page (eight lanes a page of 128-wide heads); the smallest key that is
// chosen is found digit by digit, the cluster's histograms added through distributed
// shared memory; then each CTA writes its chosen pages behind those of the CTAs
// before it, in the order of their tokens.
template <int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  constexpr int LPP = D / 16, PPW = 32 / LPP, kUnroll = 4;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelectControl ctl;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  const int unit = int(blockIdx.x) / p.ctas;
  const int r = unit / p.kv_heads, head = unit - r * p.kv_heads;
  if (r >= p.rows) {  // a cluster behind the rows
    check_sequences(p.batch, rank * kSelectWarps + warp, p.ctas * kSelectWarps, lane);
    return;
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
    for (int i = rank * kSelectThreads + tid; i < n; i += p.ctas * kSelectThreads) {
      const int page = table[i];
      if (page < 0 || page >= p.pages) record_status(kStatusInvalid, p.batch.status);
      list[i] = page;
    }
    return;
  }

  // ---- the group's queries: largest magnitude, then the sums of their 8-bit values
  const __nv_bfloat16* const q =
      p.Q + int64_t(r) * p.q_stride + int64_t(head) * p.gqa * D;
  for (int i = tid; i < kDigits * 256; i += kSelectThreads) (&ctl.hist[0][0])[i] = 0u;
  float top = 0.f;
  for (int i = tid; i < p.gqa * D; i += kSelectThreads)
    top = fmaxf(top, fabsf(__bfloat162float(q[i])));
#pragma unroll
  for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  if (lane == 0) ctl.top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) top = fmaxf(top, ctl.top[w]);
  if (tid < D) {
    // magnitudes whose grid would leave the normal binary32 are raised first, exactly
    const float raise = top < 0x1p-60f ? 0x1p66f : 1.f;
    const float inv = __uint_as_float((254u - grid_exponent(top * raise)) << 23);
    int plus = 0, minus = 0;
    for (int h = 0; h < p.gqa; ++h) {
      const float x = __bfloat162float(q[h * D + tid]) * raise * inv;
      const int v = max(-127, min(127, __float2int_rn(x)));
      plus += max(v, 0);
      minus += min(v, 0);
    }
    ctl.plus[tid] = int16_t(plus);
    ctl.minus[tid] = int16_t(minus);
  }
  __syncthreads();

  // ---- scores of this CTA's pages
  const int per = (n + p.ctas - 1) / p.ctas;
  const int j0 = min(n, rank * per), m = min(n, j0 + per) - j0;
  const int part = lane % LPP, own = lane / LPP;
  int qp[8], qm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qp[i] = reinterpret_cast<const int*>(ctl.plus)[part * 8 + i];
    qm[i] = reinterpret_cast<const int*>(ctl.minus)[part * 8 + i];
  }
  for (int base = warp * (PPW * kUnroll); base < m; base += kSelectWarps * PPW * kUnroll) {
    int64_t at[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int j = base + i * PPW + own;
      int page = j < m ? table[j0 + j] : 0;
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
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int l[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
      const int h[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
      int sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum = __dp2a_lo(qp[2 * k], h[k], sum);
        sum = __dp2a_hi(qp[2 * k + 1], h[k], sum);
        sum = __dp2a_lo(qm[2 * k], l[k], sum);
        sum = __dp2a_hi(qm[2 * k + 1], l[k], sum);
      }
#pragma unroll
      for (int d = 1; d < LPP; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int j = base + i * PPW + own;
      if (part == 0 && j < m) {
        const int page = j0 + j;
        const bool always = page < p.first || page >= n - p.last;
        keys[j] = always ? 0xffffffffu : order_key(float(sum) * grid[i]);
      }
    }
  }
  __syncthreads();

  // ---- the smallest chosen key, eight bits a pass: `above` pages have a larger one
  uint32_t prefix = 0u, above = 0u;
  for (int pass = 0; pass < kDigits; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int j = tid; j < m; j += kSelectThreads) {
      const uint32_t key = keys[j];
      if (pass == 0 || (key >> (shift + 8)) == prefix)
        atomicAdd(&ctl.hist[pass][(key >> shift) & 255u], 1u);
    }
    uint32_t sum;  // of the bin 255 - tid
    if (p.ctas > 1) {
      cluster_sync();
      sum = 0u;
      const uint32_t here = smem_addr(&ctl.hist[pass][255 - tid]);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < p.ctas) sum += ld_dsmem_u32(map_to_rank(here, uint32_t(c)));
    } else {
      __syncthreads();
      sum = ctl.hist[pass][255 - tid];
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
    // the bin in which the max_pages-th largest key lies
    if (above + upto >= uint32_t(count) && above + upto - sum < uint32_t(count)) {
      ctl.found[0] = uint32_t(255 - tid);
      ctl.found[1] = above + upto - sum;
    }
    __syncthreads();
    prefix = (prefix << 8) | ctl.found[0];
    above = ctl.found[1];
  }

  // ---- pages of this CTA above the threshold and at it, and of those before it
  uint32_t mine_above = 0u, mine_at = 0u;
  for (int j0w = warp * 32; j0w < m; j0w += kSelectThreads) {
    const uint32_t key = j0w + lane < m ? keys[j0w + lane] : 0u;
    mine_above += __popc(__ballot_sync(0xffffffffu, j0w + lane < m && key > prefix));
    mine_at += __popc(__ballot_sync(0xffffffffu, j0w + lane < m && key == prefix));
  }
  if (tid < 2) ctl.counts[tid] = 0u;
  __syncthreads();
  if (lane == 0) {
    atomicAdd(&ctl.counts[0], mine_above);
    atomicAdd(&ctl.counts[1], mine_at);
  }
  uint32_t before_above = 0u, before_at = 0u;
  if (p.ctas > 1) {
    cluster_sync();
    const uint32_t here = smem_addr(&ctl.counts[0]);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < rank) {
        before_above += ld_dsmem_u32(map_to_rank(here, uint32_t(c)));
        before_at += ld_dsmem_u32(map_to_rank(here + 4, uint32_t(c)));
      }
  }
  const uint32_t ties = uint32_t(count) - above;  // of the pages at it: the first ones
  for (int base = 0; base < m; base += kSelectThreads) {
    const int j = base + tid;
    const uint32_t key = j < m ? keys[j] : 0u;
    const bool over = j < m && key > prefix, at = j < m && key == prefix;
    const uint32_t over_mask = __ballot_sync(0xffffffffu, over);
    const uint32_t at_mask = __ballot_sync(0xffffffffu, at);
    __syncthreads();  // the sums of the round before have been read
    if (lane == 0) ctl.warp_sum[warp] = uint32_t(__popc(over_mask)) | uint32_t(__popc(at_mask)) << 16;
    __syncthreads();
    uint32_t my_above = before_above + __popc(over_mask & ((1u << lane) - 1u));
    uint32_t my_at = before_at + __popc(at_mask & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
      const uint32_t s = ctl.warp_sum[w];
      if (w < warp) my_above += s & 0xffffu, my_at += s >> 16;
      before_above += s & 0xffffu, before_at += s >> 16;
    }
    if (over || (at && my_at < ties)) {
      const uint32_t to = my_above + min(my_at, ties);
      if (to < uint32_t(count)) list[to] = table[j0 + j];
    }
  }
  if (p.ctas > 1) cluster_sync();  // no CTA ends while its counts are read
}

}  // namespace kv4
}  // namespace wq
