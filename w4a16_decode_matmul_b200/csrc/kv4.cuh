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
#include "unpack.cuh"

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
  unsigned int* status;  // the library's device status word
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
    if (s.row0 != r0 || end != r1) record_status(kStatusInvalid, p.status);
    s.rows = end - s.row0;
  } else {
    s.row0 = b * p.rows_per_seq;
    s.rows = p.rows_per_seq;
  }
  if (s.len > p.max_len) {
    record_status(kStatusInvalid, p.status);
    s.len = p.max_len;
  }
  s.len = max(s.len, 0);
  return s;
}

// Records what is out of bounds in any sequence, also in those that no row of the
// call is found in.  The row kernels have warps of their own for it, behind those
// of the rows, and it is a function of its own: a write of 32,768 rows and their
// read take 89.4 us so, 90.8 with it inlined, 91.5 as a part of each row's warp.
static __device__ __noinline__ void check_sequences(const Batch p, int warp, int warps,
                                                    int lane) {
  for (int64_t b = int64_t(warp) * 32 + lane; b < p.seqs; b += int64_t(warps) * 32)
    load_sequence(p, int(b));
}

// The page behind position pos of sequence b, or -1 (recorded) if the table
// holds no page of the cache there.
__device__ __forceinline__ int64_t load_page(const Batch& p, const Cache& c, int b, int pos) {
  const int64_t page = p.page_table[int64_t(b) * p.table_stride + (pos >> c.page_shift)];
  if (page < 0 || page >= c.pages) {
    record_status(kStatusInvalid, p.status);
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

// Two bfloat16 as the binary16 values the format quantizes (saturating).
__device__ __forceinline__ uint32_t to_format(uint32_t v) {
  const float2 f = bf16x2_to_float2(v);
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
  return r;
}

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Smallest binary16 that is not below r / 15, for the range r >= 0 of a group
// rounded up to binary32: 15 c has 15 significant bits for a binary16 c, so
// rounding r up crosses no 15 c, and the comparisons below are exact.  The
// first guess is within one step.
__device__ __forceinline__ float range_scale(float r) {
  const unsigned short guess = __half_as_ushort(__float2half_ru(r * (1.f / 15.f)));
  const float here = __half2float(__ushort_as_half(guess));
  const float below = __half2float(__ushort_as_half((unsigned short)(guess - 1)));
  const float above = __half2float(__ushort_as_half((unsigned short)(guess + 1)));
  return 15.f * below >= r ? below : 15.f * here >= r ? here : above;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Sixteen values of a group that LANES adjacent lanes share -> the two words
// of their codes, scale and zero.
//
// The codes are round-half-even of the exact quotients x / s of the binary16
// values x; the range is found on the bfloat16, whose order rounding keeps.
// With inv within 2^-23 of 1/s (relative), x inv is within 15 * 2^-22 < 2^-18
// of x / s, so rounding it decides every code whose x inv is farther than 2^-16
// from a half-integer; a lane with a nearer one, or a NaN, decides its codes by
// the exact rule.  Outside that window no code needs a clamp: (hi - lo) / s <=
// 15, and rint(hi/s) + rint(-lo/s) can be 16 only when both quotients are
// half-integers.
template <int LANES>
__device__ __forceinline__ uint2 quantize16(const uint4 (&raw)[2], float* scale, float* zero) {
  const uint32_t b[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                         raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t hi = 0u, lo = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = bmax2(hi, b[i]);
    lo = bmin2(lo, b[i]);
  }
  // (hi, -lo) in one word
  hi = bmax2(hi, __byte_perm(hi, hi, 0x1032));
  lo = bmin2(lo, __byte_perm(lo, lo, 0x1032));
  uint32_t ends = __byte_perm(hi, lo ^ 0x80008000u, 0x5410);
#pragma unroll
  for (int m = 1; m < LANES; m *= 2) ends = bmax2(ends, __shfl_xor_sync(0xffffffffu, ends, m));
  const float2 end = half2_to_float2(to_format(ends));
  const float range = __fadd_ru(end.x, end.y);
  const float s = range > 0.f ? range_scale(range) : 1.f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float z = fminf(rint_quotient(end.y, s, inv), 15.f);
  // 1.5 * 2^23 + z: the sum below lands on the integers, its low byte the code
  const float shift = 12582912.f + z;
  uint32_t u[8];    // low byte: the codes of a pair
  float off = 0.f;  // the largest distance from the rounded value, or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = half2_to_float2(to_format(b[i]));
    const float2 a = fma2(x, make_float2(inv, inv), make_float2(shift, shift));
    // shift - a is minus the rounded quotient, exactly
    const float2 r = fma2(a, make_float2(-1.f, -1.f), make_float2(shift, shift));
    const float2 e = fma2(x, make_float2(inv, inv), r);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(off) : "f"(e.x), "f"(e.y), "f"(off));
    u[i] = __float_as_uint(a.y) * 16u + __float_as_uint(a.x);
  }
  uint32_t word[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    word[i] = __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0040),
                          __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0040), 0x5410);
  if (!(off <= 0.5f - 0x1p-16f)) {
    word[0] = word[1] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = half2_to_float2(to_format(b[i]));
      const float even = fminf(fmaxf(rint_quotient(f.x, s, inv) + z, 0.f), 15.f);
      const float odd = fminf(fmaxf(rint_quotient(f.y, s, inv) + z, 0.f), 15.f);
      word[i >> 2] |= (uint32_t(int(even)) | (uint32_t(int(odd)) << 4)) << (8 * (i & 3));
    }
  }
  *scale = s;
  *zero = z + 0.f;  // never -0
  return make_uint2(word[0], word[1]);
}

// Halfwords of value codes: a lane holds those of g0 .. g0 + 3 of one chunk
// (two words); the lane two further or back holds the neighbouring chunk's.
// What is adjacent in memory is the pair of chunks of one g: after the swap
// the lane of the even chunk has the pairs of g0 and g0 + 1, the other those of
// g0 + 2 and g0 + 3.  The same swap undoes itself.
__device__ __forceinline__ uint2 swap_chunks(uint2 w, bool odd) {
  // words as pairs (g, g + 1) of one chunk <-> pairs (even, odd chunk) of one g
  const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w.x : w.y, 2);
  const uint32_t even = odd ? got : w.x, other = odd ? w.y : got;
  return make_uint2(__byte_perm(even, other, 0x5410), __byte_perm(even, other, 0x7632));
}

__device__ __forceinline__ uint2 unswap_chunks(uint2 w, bool odd) {
  // w.x = (even, odd) of g, w.y of g + 1
  const uint32_t even = __byte_perm(w.x, w.y, 0x5410), other = __byte_perm(w.x, w.y, 0x7632);
  const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? even : other, 2);
  return odd ? make_uint2(got, other) : make_uint2(even, got);
}

// Eight codes -> eight bfloat16 values s (u - z): u - z is exact in binary16,
// the product in binary32 (11 + 4 bits), and it is rounded once.
__device__ __forceinline__ uint4 values8(uint32_t word, __half2 meta) {
  const float s = __low2float(meta);
  const __half2 zero = __high2half2(meta);
  uint32_t u[4];  // (0, 4), (1, 5), (2, 6), (3, 7)
  unpack_u4_h<0>(word, u);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_to_float2(hsub2(u[i], *reinterpret_cast<const uint32_t*>(&zero)));
    x[i] = s * f.x;
    x[i + 4] = s * f.y;
  }
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    out[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Warps of a CTA of the two row kernels: one, so that a row's place on the SM is
// free as soon as the row is done (against 8, 4 and 2 a CTA at the same
// registers, kernels alone, back to back: read 85,514 rows 80 us, 92, 86, 82; write
// 32,768 and read them back 85, 88, 88, 88).
constexpr int kRowWarps = 1;
constexpr int kRowIterations = 2;  // pieces of 16 keys and 16 values per lane

// The place of a lane in the rows: it takes elements 16 lambda .. of every
// (32 / lanes of a head)-th head.
template <int D, int G>
struct RowLane {
  static constexpr int kLanes = D / 16;          // of a head
  static constexpr int kHeads = 32 / kLanes;     // of an iteration
  static constexpr int NC = D / 32, NG = D / G;
  int head, elem, chunk, t, group;
  bool odd, owns_meta;
  __device__ RowLane(int lane, int chunk_of_row) {
    const int lambda = lane % kLanes;
    head = chunk_of_row * kRowIterations * kHeads + lane / kLanes;
    elem = 16 * lambda;
    chunk = lambda >> 1;
    t = 2 * (lambda & 1);
    group = elem / G;
    odd = chunk & 1;
    owns_meta = elem % G == 0;
  }
  // word of key word t of this chunk; words of the value pairs after the swap
  __device__ int key_word(int i) const { return (t + i) * NC + chunk; }
  __device__ int value_word(int i) const {
    return ((2 * t + (odd ? 2 : 0) + i) * NC + (chunk & ~1)) / 2;
  }
};

// Rows into the cache, values as kv4.cuh's header defines them.  A warp takes
// up to 1,024 keys and values of one row, all of its loads first.  HBM bytes:
// 4 D read and D + 8 D/G written per row and head.
//
// Measured on B200: 32,768 rows of 8 heads of 128 (134 MB in, 36 MB out, groups
// of 128) 52 us, 3.2 TB/s.  Instructions (17 per value and lane, issue 60 %) and
// the wait of each row for its page and its values share the time: quotients
// formed from the bfloat16, several instructions a pair fewer, measured no
// faster (written and read back 87.4 and 88.2 us).  With
// one value per instruction throughout and 8 values a lane (twice the work per
// group) it was 115 us; with packed ranges but 8 values a lane 83.  64 registers
// (32 warps an SM) against 80: 57 and 62.
template <int D, int G>
__global__ void __launch_bounds__(kRowWarps * 32, 32)
    write_kernel(const __nv_bfloat16* __restrict__ K, int64_t k_stride,
                 const __nv_bfloat16* __restrict__ V, int64_t v_stride, Cache cache, Batch batch,
                 int chunks) {
  using L = RowLane<D, G>;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int row_warps = batch.rows * chunks;
  if (item >= row_warps) {
    check_sequences(batch, item - row_warps, int(gridDim.x) * kRowWarps - row_warps, lane);
    return;
  }
  const int r = item / chunks;
  const L my(lane, item - r * chunks);
  uint4 k[kRowIterations][2], v[kRowIterations][2];
  const uint4* from_k =
      reinterpret_cast<const uint4*>(K + int64_t(r) * k_stride + my.head * D + my.elem);
  const uint4* from_v =
      reinterpret_cast<const uint4*>(V + int64_t(r) * v_stride + my.head * D + my.elem);
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[it][i] = v[it][i] = make_uint4(0, 0, 0, 0);
      if (my.head + it * L::kHeads < cache.kv_heads) {
        k[it][i] = __ldg(from_k + it * (L::kHeads * D / 8) + i);
        v[it][i] = __ldg(from_v + it * (L::kHeads * D / 8) + i);
      }
    }
  const Place at = find_place(batch, cache, r, lane);
  if (at.page < 0) return;  // the whole warp: one row
  int64_t token = ((at.page * cache.kv_heads + my.head) << cache.page_shift) + at.slot;
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    float ks, kz, vs, vz;
    const uint2 kw = quantize16<G / 16>(k[it], &ks, &kz);
    const uint2 vw = swap_chunks(quantize16<G / 16>(v[it], &vs, &vz), my.odd);
    if (my.head + it * L::kHeads < cache.kv_heads) {
      uint32_t* const to_k = reinterpret_cast<uint32_t*>(cache.k_codes + token * (D / 2));
      uint32_t* const to_v = reinterpret_cast<uint32_t*>(cache.v_codes + token * (D / 2));
      to_k[my.key_word(0)] = kw.x;
      to_k[my.key_word(1)] = kw.y;
      to_v[my.value_word(0)] = vw.x;
      to_v[my.value_word(1)] = vw.y;
      if (my.owns_meta) {
        cache.k_meta[token * L::NG + my.group] = __floats2half2_rn(ks, kz);
        cache.v_meta[token * L::NG + my.group] = __floats2half2_rn(vs, vz);
      }
    }
    token += int64_t(L::kHeads) << cache.page_shift;
  }
}

// The values of cached rows, bfloat16 [rows][kv_heads][D].  Rows of a
// sequence that hold no token get zeros; rows of no sequence are left alone.
// HBM bound, six bytes written for each read: 85,514 rows of 8 heads of 128 in
// groups of 32 (460 MB) in 80 us alone (5.7 TB/s), 88 us a call through the binding.
template <int D, int G>
__global__ void __launch_bounds__(kRowWarps * 32, 32)
    read_kernel(Cache cache, Batch batch, __nv_bfloat16* __restrict__ K,
                __nv_bfloat16* __restrict__ V, int chunks) {
  using L = RowLane<D, G>;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int row_warps = batch.rows * chunks;
  if (item >= row_warps) {
    check_sequences(batch, item - row_warps, int(gridDim.x) * kRowWarps - row_warps, lane);
    return;
  }
  const int r = item / chunks;
  const L my(lane, item - r * chunks);
  const Place at = find_place(batch, cache, r, lane);
  if (at.page < 0 && !at.empty) return;
  uint2 kw[kRowIterations], vw[kRowIterations];
  __half2 km[kRowIterations], vm[kRowIterations];
  int64_t token = ((at.page * cache.kv_heads + my.head) << cache.page_shift) + at.slot;
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    kw[it] = vw[it] = make_uint2(0, 0);
    km[it] = vm[it] = __half2half2(__ushort_as_half(0));
    if (my.head + it * L::kHeads < cache.kv_heads && !at.empty) {
      const uint32_t* const k = reinterpret_cast<const uint32_t*>(cache.k_codes + token * (D / 2));
      const uint32_t* const v = reinterpret_cast<const uint32_t*>(cache.v_codes + token * (D / 2));
      kw[it] = make_uint2(k[my.key_word(0)], k[my.key_word(1)]);
      vw[it] = make_uint2(v[my.value_word(0)], v[my.value_word(1)]);
      km[it] = cache.k_meta[token * L::NG + my.group];
      vm[it] = cache.v_meta[token * L::NG + my.group];
    }
    token += int64_t(L::kHeads) << cache.page_shift;
  }
  const int64_t first = (int64_t(r) * cache.kv_heads + my.head) * D + my.elem;
#pragma unroll
  for (int it = 0; it < kRowIterations; ++it) {
    const uint2 w = unswap_chunks(vw[it], my.odd);
    if (my.head + it * L::kHeads < cache.kv_heads) {
      uint4* const to_k = reinterpret_cast<uint4*>(K + first + it * (L::kHeads * D));
      uint4* const to_v = reinterpret_cast<uint4*>(V + first + it * (L::kHeads * D));
      to_k[0] = values8(kw[it].x, km[it]);
      to_k[1] = values8(kw[it].y, km[it]);
      to_v[0] = values8(w.x, vm[it]);
      to_v[1] = values8(w.y, vm[it]);
    }
  }
}

}  // namespace kv4
}  // namespace wq
