// kv4.cuh -- the 4-bit key/value cache: its format, the description of a
// batch, and the kernels that write rows into it and read them back.
//
// Format (per page, head and token, for keys and for values alike): D codes
// of 4 bits and, for every group of G of them, one (scale, zero) pair of
// binary16.  A value x is taken to binary16 (nearest, saturating at the
// largest finite value: exact for every bfloat16 of magnitude 2^-17 ..
// 65504) and quantized as the asymmetric weights are ("vLLM 量化与推测解码"
// section 1): lo = min(0, min x), hi = max(0, max x), s the smallest binary16
// >= (hi - lo)/15 (1 when hi = lo), z = clamp(round(-lo/s), 0, 15),
// u = clamp(round(x/s) + z, 0, 15); it stands for s (u - z).
//
// Order of a row's codes.  The attention kernels feed the tensor cores from
// the packed words, so a row is stored in the order in which a lane needs
// it: seen as [D/32 chunks][4 words of 8 codes], a key row is stored with
// the words of one word index together ([4][D/32]: lane t of a quad reads
// word t of every chunk in one load), and a value row, seen as [D/32][8
// halfwords of 4 codes], as [8][D/32] (lane group g reads halfword g of
// every chunk).  Any group of 32, 64 or 128 is a whole number of chunks, so
// each tensor-core step stays inside one group.
#pragma once

#include "common.cuh"
#include "quantize.cuh"

namespace wq {
namespace kv4 {

// Codes and metadata of one kind (keys or values):
// codes [pages][kv_heads][page][D/2], meta [pages][kv_heads][page][D/G].
struct Cache {
  uint8_t* k_codes;
  __half2* k_meta;
  uint8_t* v_codes;
  __half2* v_meta;
  int64_t pages;
  int page_shift;  // log2 of the tokens of a page
  int kv_heads;
};

// Rows (new tokens) of a batch of sequences; see wq_kv4_batch in wq.h.
struct Batch {
  const int* row_starts;  // [seqs + 1] or null: rows_per_seq rows each
  const int* seq_lens;    // [seqs]
  const int* page_table;  // [seqs][table_stride]
  int64_t table_stride;
  int seqs;
  int rows;
  int rows_per_seq;
  int max_len;  // tokens that a row of the page table can hold
};

constexpr unsigned int kStatusInvalid = 1;  // WQ_ERR_INVALID_ARG

// First row, number of rows and length of sequence b, inside the batch's
// bounds whatever the device arrays hold.
struct Sequence {
  int row0, rows, len;
};

__device__ __forceinline__ Sequence load_sequence(const Batch& p, int b) {
  Sequence s;
  s.len = p.seq_lens[b];
  if (p.row_starts != nullptr) {
    const int r0 = p.row_starts[b], r1 = p.row_starts[b + 1];
    s.row0 = min(max(r0, 0), p.rows);
    const int end = min(max(r1, s.row0), p.rows);
    if (s.row0 != r0 || end != r1) record_status(kStatusInvalid);
    s.rows = end - s.row0;
  } else {
    s.row0 = b * p.rows_per_seq;
    s.rows = p.rows_per_seq;
  }
  if (s.len > p.max_len) {
    record_status(kStatusInvalid);
    s.len = p.max_len;
  }
  s.len = max(s.len, 0);
  return s;
}

// The page behind position pos of sequence b, or -1 (recorded) if the table
// holds no page of the cache there.
__device__ __forceinline__ int64_t load_page(const Batch& p, const Cache& c, int b, int pos) {
  const int64_t page = p.page_table[int64_t(b) * p.table_stride + (pos >> c.page_shift)];
  if (page < 0 || page >= c.pages) {
    record_status(kStatusInvalid);
    return -1;
  }
  return page;
}

// The sequence that row r belongs to, found by all lanes of a warp together
// (33-ary search: one load a lane and round); -1 for a row behind the last
// sequence or before the first.
__device__ __forceinline__ int find_sequence(const Batch& p, int r, int lane) {
  if (p.row_starts == nullptr) return r / p.rows_per_seq;
  // the largest b in [lo, hi) with row_starts[b] <= r; rows of b end at
  // row_starts[b + 1]
  int lo = 0, n = p.seqs + 1;
  if (p.row_starts[0] > r) return -1;
  while (n > 1) {
    const int step = (n + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool below = at < lo + n && p.row_starts[at] <= r;
    const int skip = __popc(__ballot_sync(0xffffffffu, below));
    lo += skip * step;
    n = min(step, n - skip * step);
  }
  return lo < p.seqs ? lo : -1;
}

// Where row r's token lives: page (-1: nothing to do), slot, and whether the
// row belongs to a sequence but holds no token.
struct Place {
  int64_t page;
  int slot;
  bool empty;
};

__device__ __forceinline__ Place find_place(const Batch& p, const Cache& c, int r, int lane) {
  Place at = {-1, 0, false};
  const int b = find_sequence(p, r, lane);
  if (b < 0) return at;
  const Sequence s = load_sequence(p, b);
  const int pos = s.len - s.rows + (r - s.row0);
  if (r < s.row0 || r >= s.row0 + s.rows) return at;
  if (pos < 0) {
    at.empty = true;
    return at;
  }
  at.page = load_page(p, c, b, pos);
  at.slot = pos & ((1 << c.page_shift) - 1);
  return at;
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// A bfloat16 as the binary16 value the format quantizes.
__device__ __forceinline__ float to_format(float x) {
  return __half2float(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
}

// Eight values of a group that LANES adjacent lanes share -> the word of
// their codes, scale and zero.  The scale is exact: __fadd_ru and __fdiv_ru
// round up in binary32 and __float2half_ru to binary16; 15 c has 15
// significant bits for a binary16 c, so no c lies between (hi - lo)/15 and
// its binary32 round-ups, and the result is the smallest binary16 that is not
// below the exact quotient.
template <int LANES>
__device__ __forceinline__ uint32_t quantize8(const uint4& raw, float* scale, float* zero) {
  float x[8];
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    x[2 * i] = to_format(f.x);
    x[2 * i + 1] = to_format(f.y);
    lo = fminf(lo, fminf(x[2 * i], x[2 * i + 1]));
    hi = fmaxf(hi, fmaxf(x[2 * i], x[2 * i + 1]));
  }
#pragma unroll
  for (int m = 1; m < LANES; m *= 2) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const float s =
      hi > lo ? __half2float(__float2half_ru(__fdiv_ru(__fadd_ru(hi, -lo), 15.f))) : 1.f;
  const float z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) + 0.f;  // never -0
  const float inv = __frcp_rn(s);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rint_quotient(x[i], s, inv) + z, 0.f), 15.f);
    word |= uint32_t(int(q)) << (4 * i);
  }
  *scale = s;
  *zero = z;
  return word;
}

constexpr int kRowWarps = 8;       // warps of a CTA of the two row kernels
constexpr int kRowIterations = 4;  // 16-byte pieces of keys and values per lane

// Rows into the cache, values as kv4.cuh's header defines them.  A warp takes
// up to 128 pieces of 8 elements of one row (four heads of 64 ... ), all of
// its loads first.  HBM bound: 4 D bytes read and D + 8 D/G written per row
// and head.
template <int D, int G>
__global__ void __launch_bounds__(kRowWarps * 32)
    write_kernel(const __nv_bfloat16* __restrict__ K, int64_t k_stride,
                 const __nv_bfloat16* __restrict__ V, int64_t v_stride, Cache cache, Batch batch,
                 int chunks) {
  constexpr int NC = D / 32, NG = D / G, kPieces = D / 8;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item >= int64_t(batch.rows) * chunks) return;
  const int r = int(item / chunks), chunk = int(item % chunks);
  const int pieces = cache.kv_heads * kPieces;
  uint4 k[kRowIterations], v[kRowIterations];
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    const int e = (chunk * kRowIterations + it) * 32 + lane;
    if (e < pieces) {
      k[it] = ldg_stream128(K + int64_t(r) * k_stride + int64_t(e) * 8);
      v[it] = ldg_stream128(V + int64_t(r) * v_stride + int64_t(e) * 8);
    } else {
      k[it] = v[it] = make_uint4(0, 0, 0, 0);
    }
  }
  const Place at = find_place(batch, cache, r, lane);
  if (at.page < 0) return;  // the whole warp: one row
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    const int e = (chunk * kRowIterations + it) * 32 + lane;
    if (e - lane >= pieces) break;
    float ks, kz, vs, vz;
    const uint32_t kw = quantize8<G / 8>(k[it], &ks, &kz);
    const uint32_t vw = quantize8<G / 8>(v[it], &vs, &vz);
    // value halfwords of chunks j (even) and j + 1 are neighbours in memory:
    // lanes of the two chunks swap one halfword each and store one word each
    const int l = e % kPieces, j = l / 4, t = l % 4;
    const uint32_t give = (j & 1) ? (vw & 0xffffu) : (vw >> 16);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
    if (e >= pieces) continue;
    const int64_t token =
        ((at.page * cache.kv_heads + e / kPieces) << cache.page_shift) + at.slot;
    reinterpret_cast<uint32_t*>(cache.k_codes + token * (D / 2))[t * NC + j] = kw;
    const uint32_t pair = (j & 1) ? (got | (vw & 0xffff0000u)) : ((vw & 0xffffu) | (got << 16));
    reinterpret_cast<uint32_t*>(cache.v_codes + token * (D / 2))[((2 * t + (j & 1)) * NC + j) / 2] =
        pair;
    if (l % (G / 8) == 0) {
      cache.k_meta[token * NG + l / (G / 8)] = __floats2half2_rn(ks, kz);
      cache.v_meta[token * NG + l / (G / 8)] = __floats2half2_rn(vs, vz);
    }
  }
}

// Eight codes -> eight bfloat16 values s (u - z): the product is exact in
// binary32 (11 + 4 bits) and rounded once.
__device__ __forceinline__ uint4 values8(uint32_t word, __half2 meta) {
  const float2 m = __half22float2(meta);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = m.x * (float((word >> (8 * i)) & 15u) - m.y);
    const float b = m.x * (float((word >> (8 * i + 4)) & 15u) - m.y);
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    out[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The values of cached rows, bfloat16 [rows][kv_heads][D].  Rows of a
// sequence that hold no token get zeros; rows of no sequence are left alone.
template <int D, int G>
__global__ void __launch_bounds__(kRowWarps * 32)
    read_kernel(Cache cache, Batch batch, __nv_bfloat16* __restrict__ K,
                __nv_bfloat16* __restrict__ V, int chunks) {
  constexpr int NC = D / 32, NG = D / G, kPieces = D / 8;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (item >= int64_t(batch.rows) * chunks) return;
  const int r = int(item / chunks), chunk = int(item % chunks);
  const int pieces = cache.kv_heads * kPieces;
  const Place at = find_place(batch, cache, r, lane);
  if (at.page < 0 && !at.empty) return;
  uint32_t kw[kRowIterations], vw[kRowIterations];
  __half2 km[kRowIterations], vm[kRowIterations];
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    const int e = (chunk * kRowIterations + it) * 32 + lane;
    kw[it] = vw[it] = 0;
    km[it] = vm[it] = __half2half2(__ushort_as_half(0));
    if (e < pieces && !at.empty) {
      const int l = e % kPieces, j = l / 4, t = l % 4;
      const int64_t token =
          ((at.page * cache.kv_heads + e / kPieces) << cache.page_shift) + at.slot;
      kw[it] = reinterpret_cast<const uint32_t*>(cache.k_codes + token * (D / 2))[t * NC + j];
      const uint16_t* vrow = reinterpret_cast<const uint16_t*>(cache.v_codes + token * (D / 2));
      vw[it] = uint32_t(vrow[2 * t * NC + j]) | (uint32_t(vrow[(2 * t + 1) * NC + j]) << 16);
      km[it] = cache.k_meta[token * NG + l / (G / 8)];
      vm[it] = cache.v_meta[token * NG + l / (G / 8)];
    }
  }
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    const int e = (chunk * kRowIterations + it) * 32 + lane;
    if (e < pieces) {
      const int64_t to = (int64_t(r) * pieces + e) * 8;
      *reinterpret_cast<uint4*>(K + to) = values8(kw[it], km[it]);
      *reinterpret_cast<uint4*>(V + to) = values8(vw[it], vm[it]);
    }
  }
}

}  // namespace kv4
}  // namespace wq
