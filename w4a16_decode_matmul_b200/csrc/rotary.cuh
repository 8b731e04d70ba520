// rotary.cuh -- rotary positions: rows turned by the angles of their
// positions, alone and on the way into the 4-bit key/value cache.
//
// Mathematics.  Element pairs (x1, x2) of a head, n = dim / 2 of them -- (i, i +
// n), or (2i, 2i + 1) where the layout is interleaved -- turn by the angle p f_i
// of the row's position p; the elements from dim on stay:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,  c = a cos(p f_i),  s = a sin(p f_i)
// with a the amplitude.  The transpose (the gradient) is the same with -s.
//
// Roundings.  The angle is a product in binary64 (exact below 2^29 positions)
// and so are sine and cosine: a binary32 product is off by up to 2^-24 of
// itself, 0.03 radians at position 10^6.  c and s are rounded to binary32, the
// result to bfloat16.  Between the two, queries take a multiply-add in binary32;
// keys that go into the cache are the result to within 3 2^-39 of |x1 c| + |x2 s|,
// rounded to binary32 (one in some 10^7 other than the exact result's), because a bit of
// a key next to a border between two codes is a whole step of the value that the cache
// holds.
#pragma once

#include "kv4_attn.cuh"

namespace wq {
namespace rotary {

struct Spec {
  const float* freqs;  // [dim / 2], radians a position
  int dim;
  float amplitude;
};

// (c, s) of one position and frequency, in binary64 arithmetic that all heads share.
// The angle less a multiple of pi/2 that is held in two parts (W. J. Cody and W. Waite,
// 1980; what the two leave of pi/2, 1.5 10^-33, counts from 2^60 on, and the multiple is the
// nearest or next to it below 2^50), then the series of sine and cosine to the 15th and 16th
// power: for |r| <= pi/4 the next terms are below 2^-54.  (A function of its own: its
// registers are not the kernels', which keep their loads in flight meanwhile.)
static __device__ __noinline__ float2 turn_of(int position, float freq, float amplitude) {
  const double a = double(position) * double(freq);
  const double k = rint(a * 0.6366197723675814);         // 2/pi
  double r = fma(-k, 1.5707963267948966, a);             // pi/2 ...
  r = fma(-k, 6.123233995736766e-17, r);                 // ... and the rest of it
  const double z = r * r;
  double s = fma(z, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  double c = fma(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  s = fma(s, z, -1.0 / 39916800.0);
  c = fma(c, z, 1.0 / 479001600.0);
  s = fma(s, z, 1.0 / 362880.0);
  c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, -1.0 / 5040.0);
  c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 120.0);
  c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, -1.0 / 6.0);
  c = fma(c, z, 1.0 / 24.0);
  s = fma(s * z, r, r);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int quarter = int(__double2ll_rn(k)) & 3;
  const double x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  const double m = double(amplitude);
  return make_float2(float(((quarter + 1) & 2) ? -(m * x) : m * x),
                     float((quarter & 2) ? -(m * y) : m * y));
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The angles of a row as the kernels read them, an entry for each turned element e of a
// head: y_e = x_e c_e + z_e n_e, z_e the other element of its pair, n_e = -s for the
// first element of the pair and s for the second.
__device__ __forceinline__ void put_turn(float2 t, int j, int half, bool interleaved, float* c,
                                         float* n) {
  const int one = interleaved ? 2 * j : j, two = interleaved ? 2 * j + 1 : j + half;
  c[one] = c[two] = t.x;
  n[one] = -t.y;
  n[two] = t.y;
}

__device__ __forceinline__ float2 negative(float2 x) { return mul2(x, make_float2(-1.f, -1.f)); }

// Eight entries.
struct Eight {
  float2 of[4];
  __device__ __forceinline__ explicit Eight(const float* from) {
    const float4 a = reinterpret_cast<const float4*>(from)[0];
    const float4 b = reinterpret_cast<const float4*>(from)[1];
    of[0] = make_float2(a.x, a.y), of[1] = make_float2(a.z, a.w);
    of[2] = make_float2(b.x, b.y), of[3] = make_float2(b.z, b.w);
  }
};

// What one thread turns at a time: eight pairs (two runs of eight elements, or one
// of eight for interleaved pairs, which are four), or eight elements that stay.  A row's
// units that turn come first, those of all heads, then those that are copied: a warp does one
// or the other.
struct Units {
  int turned, copied;        // of a head
  kv4::FastDiv by_turned, by_copied;
};

// Unit i of a row with `first` units that turn: its head and first element.
struct UnitAt {
  int head, k;
  bool turned;
};

__device__ __forceinline__ UnitAt unit_at(const Units& u, int i, int first) {
  UnitAt at;
  at.turned = i < first;
  const int j = at.turned ? i : i - first, each = at.turned ? u.turned : u.copied;
  at.head = (at.turned ? u.by_turned : u.by_copied)(j);
  at.k = j - at.head * each;
  return at;
}

// Offset of its first element in its head.
template <bool INTERLEAVED>
__device__ __forceinline__ int unit_offset(const Units& u, const UnitAt& at, int dim) {
  return 8 * at.k + (at.turned ? 0 : INTERLEAVED ? 8 * u.turned : dim);
}

// The sequence of row r, its place there and its token's position, by all lanes of a warp;
// seq -1: the row is in no sequence.
struct RowAt {
  int seq, token;
};

__device__ __forceinline__ RowAt find_row(const kv4::Batch& p, int r, int lane) {
  if (p.row_starts != nullptr && p.seqs < 32) {  // few sequences: all of them at once
    const int start = p.row_starts[min(lane, p.seqs)];
    int len = p.seq_lens[min(lane, p.seqs - 1)];
    const int next = __shfl_down_sync(0xffffffffu, start, 1);
    const bool mine = lane < p.seqs && start >= 0 && start <= r && r < next && next <= p.rows;
    const unsigned found = __ballot_sync(0xffffffffu, mine);
    if (found) {  // (what is out of bounds is recorded where the sequences are checked)
      const int b = __ffs(found) - 1;
      len = max(0, min(__shfl_sync(0xffffffffu, len, b), p.max_len));
      return {b, len - __shfl_sync(0xffffffffu, next, b) + r};
    }
  }
  const int b = kv4::find_sequence(p, r, lane);
  if (b < 0) return {-1, 0};
  const kv4::Sequence seq = kv4::load_sequence(p, b);
  if (r < seq.row0 || r >= seq.row0 + seq.rows) return {-1, 0};
  return {b, seq.len - seq.rows + (r - seq.row0)};
}

// Two runs of eight elements that are each other's pairs; c and n at the first's.
__device__ __forceinline__ void turn_runs(uint4& a, uint4& b, const float* c, const float* n) {
  const Eight cs(c), ns(n);
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = kv4::bf16x2_to_float2(x[i]), q = kv4::bf16x2_to_float2(y[i]);
    const float2 one = fma2(q, ns.of[i], mul2(p, cs.of[i]));
    const float2 two = fma2(p, negative(ns.of[i]), mul2(q, cs.of[i]));
    x[i] = pack_bf162(one.x, one.y);
    y[i] = pack_bf162(two.x, two.y);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

// Pairs side by side; the first `pairs` of the run's four turn.
__device__ __forceinline__ void turn_interleaved(uint4& a, const float* c, const float* n,
                                                 int pairs) {
  const Eight cs(c), ns(n);
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < pairs) {
      const float2 p = kv4::bf16x2_to_float2(x[i]);
      const float2 y = fma2(make_float2(p.y, p.x), ns.of[i], mul2(p, cs.of[i]));
      x[i] = pack_bf162(y.x, y.y);
    }
  a = make_uint4(x[0], x[1], x[2], x[3]);
}

constexpr int kMaxHead = 512;
constexpr int kTurns = 1024;  // entries of turned elements that a CTA holds: of several rows

struct RotaryParams {
  const __nv_bfloat16* X;  // [rows][heads][head_dim], rows x_stride elements apart
  int64_t x_stride;
  __nv_bfloat16* Y;  // X itself, or other memory
  int64_t y_stride;
  const int* positions;  // [rows]
  Spec spec;
  int rows, heads, head_dim;
  int rows_each;  // rows of a CTA
  Units units;
  kv4::FastDiv by_row;  // by the units of a row
  bool copy;      // Y is other memory: the elements that stay are copied
  float sign;     // -1: the transpose
};

struct RotaryTurns {
  // (a head whose turned part ends inside a run of eight is read to the run's end)
  alignas(16) float c[kTurns + 8], n[kTurns + 8];
};

constexpr int kRowsEach = 4;  // rows of a CTA, at most

// The angles of a CTA's rows r0 .. r0 + count - 1, all threads together.
__device__ __forceinline__ void make_turns(const RotaryParams& p, bool interleaved, int64_t r0,
                                           int count, RotaryTurns& t) {
  const int half = p.spec.dim / 2;
  for (int j = threadIdx.x; j < count * half; j += blockDim.x) {
    const int row = j / half, f = j - row * half;
    float2 cs = turn_of(p.positions[r0 + row], p.spec.freqs[f], p.spec.amplitude);
    cs.y *= p.sign;
    put_turn(cs, f, half, interleaved, t.c + row * p.spec.dim, t.n + row * p.spec.dim);
  }
  __syncthreads();
}

// A CTA takes a few rows (blockIdx.x) -- the angles' arithmetic, a chain of some 60 dependent
// operations in binary64, is then paid once for all of them -- or, where there are few
// rows, a part of one row's units (blockIdx.y).  The loads of each thread's first unit are
// on their way meanwhile.  HBM bound, two bytes in and two out an element.
//
// Measured on B200: 8,192 rows of 40 heads of 128 (168 MB) 33 us, 5.1 TB/s.  A row a CTA
// 50; angles as (c, s) pairs and an element an instruction 41.  3,001 rows of 24 heads of 64,
// half of each side by side (18 MB): 5 us; 751 CTAs of 384 threads are 1.27 waves, and its
// warps wait for the angles (two of five at the barrier) and for loads.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(512, 3) rotary_kernel(const RotaryParams p) {
  __shared__ RotaryTurns turns;
  const int64_t r0 = int64_t(blockIdx.x) * p.rows_each;
  const int n = int(min(int64_t(p.rows_each), p.rows - r0));
  const int half = p.spec.dim / 2, first = p.heads * p.units.turned;
  const int each = first + p.heads * p.units.copied, units = each * n;
  const int step = int(gridDim.y * blockDim.x);
  bool ready = false;
  for (int i = int(blockIdx.y * blockDim.x + threadIdx.x);; i += step) {
    const bool there = i < units;
    const int row = p.by_row(i);
    const UnitAt u = unit_at(p.units, i - row * each, first);
    const int at = u.head * p.head_dim + unit_offset<INTERLEAVED>(p.units, u, p.spec.dim);
    const __nv_bfloat16* const from = p.X + (r0 + row) * p.x_stride + at;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (there) {
      a = *reinterpret_cast<const uint4*>(from);
      if (!INTERLEAVED && u.turned) b = *reinterpret_cast<const uint4*>(from + half);
    }
    if (!ready) {
      ready = true;
      make_turns(p, INTERLEAVED, r0, n, turns);
    }
    if (!there) return;
    __nv_bfloat16* const to = p.Y + (r0 + row) * p.y_stride + at;
    if (u.turned) {
      const int e = row * p.spec.dim + 8 * u.k;
      if (INTERLEAVED) {
        turn_interleaved(a, turns.c + e, turns.n + e, half - 4 * u.k);
      } else {
        turn_runs(a, b, turns.c + e, turns.n + e);
        *reinterpret_cast<uint4*>(to + half) = b;
      }
    }
    *reinterpret_cast<uint4*>(to) = a;
  }
}

// The same where the other elements of a run's pairs, or its angles, do not lie on 16-byte
// boundaries (dim not a multiple of 16 in halves, of 4 side by side).  Heads go through
// shared memory, 16 KB of whole heads at a time, so that memory is read and written in
// runs all the same, and each run is read by all before it is written where Y is X: 8,192
// rows of 40 heads, 126 of 128 elements turned, 62 us (a pair a thread, two bytes at a
// time, 84; 128 turned, rotary_kernel, 33).  Shared memory bounds it (92 % of its rate): the
// other element of each pair comes two bytes at a time, its angles eight.
constexpr int kStaged = 8192;  // elements
constexpr int kStagedThreads = 256;

static __global__ void __launch_bounds__(kStagedThreads, 4)
    rotary_staged_kernel(const RotaryParams p, bool interleaved, kv4::FastDiv by_runs,
                         kv4::FastDiv by_heads) {
  __shared__ RotaryTurns turns;
  __shared__ __align__(16) __nv_bfloat16 staged[kStaged];
  const int64_t r0 = int64_t(blockIdx.x) * p.rows_each;
  const int n = int(min(int64_t(p.rows_each), p.rows - r0));
  const int dim = p.spec.dim, half = dim / 2, runs = p.head_dim / 8;
  // heads of all rows of the CTA, a contiguous part of them for each blockIdx.y
  const int all = n * p.heads, part = (all + int(gridDim.y) - 1) / int(gridDim.y);
  const int begin = min(all, int(blockIdx.y) * part), end = min(all, begin + part);
  const int tile = kStaged / p.head_dim;
  for (int g0 = begin; g0 < end; g0 += tile) {
    const int count = min(tile, end - g0) * runs;
    for (int i = threadIdx.x; i < count; i += kStagedThreads) {
      const int h = by_runs(i), g = g0 + h, row = by_heads(g);
      reinterpret_cast<uint4*>(staged)[i] = *reinterpret_cast<const uint4*>(
          p.X + (r0 + row) * p.x_stride + int64_t(g - row * p.heads) * p.head_dim +
          8 * (i - h * runs));
    }
    if (g0 == begin) make_turns(p, interleaved, r0, n, turns);  // synchronizes
    else __syncthreads();
    for (int i = threadIdx.x; i < count; i += kStagedThreads) {
      const int h = by_runs(i), g = g0 + h, row = by_heads(g), e0 = 8 * (i - h * runs);
      if (e0 >= dim && !p.copy) continue;
      const __nv_bfloat16* const head = staged + h * p.head_dim;
      const uint4 raw = reinterpret_cast<const uint4*>(staged)[i];
      uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + 2 * k;  // dim is even: a word turns or stays as a whole
        if (e >= dim) break;
        const float2 x = kv4::bf16x2_to_float2(w[k]);
        const float2 c = *reinterpret_cast<const float2*>(turns.c + row * dim + e);
        const float2 s = *reinterpret_cast<const float2*>(turns.n + row * dim + e);
        float2 z = make_float2(x.y, x.x);
        if (!interleaved)
          z = make_float2(__bfloat162float(head[e < half ? e + half : e - half]),
                          __bfloat162float(head[e + 1 < half ? e + 1 + half : e + 1 - half]));
        const float2 y = fma2(z, s, mul2(x, c));
        w[k] = pack_bf162(y.x, y.y);
      }
      *reinterpret_cast<uint4*>(p.Y + (r0 + row) * p.y_stride +
                                int64_t(g - row * p.heads) * p.head_dim + e0) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();  // read before the next heads come
  }
}

// ------------------------------------------- on the way into the 4-bit cache

// A binary32 c as the sum of its leading 16 bits and the rest: products with a
// bfloat16 (8 bits) are exact with each part.
__device__ __forceinline__ float2 split16(float c) {
  const float hi = __uint_as_float(__float_as_uint(c) & 0xffffff00u);
  return make_float2(hi, c - hi);
}

// The entries of a row's angles with both factors split.
template <int D>
struct SplitTurns {
  alignas(16) float c[D], n[D], c_high[D], c_low[D], n_high[D], n_low[D];
};

// Eight keys, two at a time: x c + z n rounded once to binary32.  The leading products are
// exact, the error of their sum is found exactly (Knuth's two-sum), and what the low parts
// add is at most 2^-15 of the products, with two roundings of 2^-24 of that.  z: the
// other elements of the pairs; e: the first key's entry.
template <int D>
__device__ __forceinline__ uint4 turn_keys(const uint4& xs, const uint4& zs,
                                           const SplitTurns<D>& t, int e) {
  const uint32_t xw[4] = {xs.x, xs.y, xs.z, xs.w}, zw[4] = {zs.x, zs.y, zs.z, zs.w};
  const Eight ch(t.c_high + e), cl(t.c_low + e), nh(t.n_high + e), nl(t.n_low + e);
  float2 y[4], lead[4];
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = kv4::bf16x2_to_float2(xw[i]), z = kv4::bf16x2_to_float2(zw[i]);
    const float2 minus = make_float2(-1.f, -1.f);
    const float2 a = mul2(x, ch.of[i]), b = mul2(z, nh.of[i]);
    const float2 d = add2(a, b);
    const float2 back = fma2(a, minus, d);
    const float2 err = add2(fma2(fma2(back, minus, d), minus, a), fma2(back, minus, b));
    const float2 low = fma2(x, cl.of[i], mul2(z, nl.of[i]));
    y[i] = add2(d, add2(err, low));
    lead[i] = d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(most) : "f"(d.x), "f"(d.y), "f"(most));
  }
  if (!(most <= 3.4028234e38f)) {  // infinite or NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(fabsf(lead[i].x) <= 3.4028234e38f)) y[i].x = lead[i].x;
      if (!(fabsf(lead[i].y) <= 3.4028234e38f)) y[i].y = lead[i].y;
    }
  }
  return make_uint4(pack_bf162(y[0].x, y[0].y), pack_bf162(y[1].x, y[1].y),
                    pack_bf162(y[2].x, y[2].y), pack_bf162(y[3].x, y[3].y));
}

// The place of a lane in a row's keys and values: 16 elements of one head, the row's
// share of a warp being 512 elements (half of kv4.cuh's write kernel's, for its
// registers: with 1,024 two CTAs fit an SM).
template <int D, int G>
struct KeyLane : kv4::RowLane<D, G> {
  __device__ KeyLane(int lane, int share) : kv4::RowLane<D, G>(lane, 0) {
    this->head += share * kv4::RowLane<D, G>::kHeads;
  }
};

struct WriteParams {
  const __nv_bfloat16 *Q, *K, *V;
  int64_t q_stride, k_stride, v_stride;
  __nv_bfloat16* Q_out;
  int64_t qo_stride;
  const int* positions;  // [rows], or null: the tokens' own
  Spec spec;
  kv4::Cache cache;
  kv4::Batch batch;
  int q_heads, chunks;  // chunks: warps' shares of a row's keys and values
  bool copy_q;          // Q_out is other memory than Q
  int rows_each;        // rows of a CTA
  Units units;          // of queries
};

constexpr int kWriteWarps = 8;
constexpr int kQueryUnits = 2;  // units of queries a lane has in flight

// What a CTA knows of one of its rows: page -1 where nothing is written, seq -1 where the row
// is left alone.
struct RowPlace {
  int64_t page;
  int seq, slot, position;
};

// Queries turned, keys turned and quantized, values quantized.  A CTA takes p.rows_each
// rows: a warp finds each row's place, all threads make the rows' angles, then the warps
// take the rows' shares in turn: the first `chunks` shares of a row are 512 keys and
// values each, the others 64 units of queries.  A warp's first share is on its way
// meanwhile.  CTAs behind the rows check the sequences.
//
// Measured on B200 (15,609 rows, 32 + 2 * 8 heads of 128, half of each turned, 330 MB): 86
// us, 3.8 TB/s, 3,400 warp instructions a row, of which the quantizer has a third.  Nothing
// is full (issue 58 %, ALU 46 %, shared memory 60 %): of the 6.9 warps that a scheduler has
// under 64 registers, 1.7 wait for loads, 0.9 for shared memory and 0.8 at barriers.  With
// the queries in a launch of their own 54 + 51 us; a row a CTA 102; keys and values last,
// or always in the same warps, 92 to 99; three CTAs an SM, which spill nothing, 94.
template <int D, int G, bool INTERLEAVED>
__global__ void __launch_bounds__(kWriteWarps * 32, 4)
    write_rotary_kernel(const WriteParams p, int shares) {
  using L = KeyLane<D, G>;
  __shared__ SplitTurns<D> turns[kRowsEach];
  __shared__ RowPlace places[kRowsEach];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int ctas = (p.batch.rows + p.rows_each - 1) / p.rows_each;
  if (int(blockIdx.x) >= ctas) {
    kv4::check_sequences(p.batch, (int(blockIdx.x) - ctas) * warps + warp,
                         (int(gridDim.x) - ctas) * warps, lane);
    return;
  }
  const int r0 = int(blockIdx.x) * p.rows_each, n = min(p.rows_each, p.batch.rows - r0);
  const int half = p.spec.dim / 2, first = p.q_heads * p.units.turned;
  const int units = first + p.q_heads * p.units.copied;
  bool ready = false;
  auto prepare = [&] {
    if (ready) return;
    ready = true;
    for (int i = warp; i < n; i += warps) {
      const int r = r0 + i;
      const RowAt row = find_row(p.batch, r, lane);
      RowPlace at = {-1, row.seq, 0, 0};
      if (row.seq >= 0) {
        at.position = p.positions != nullptr ? p.positions[r] : row.token;
        if (row.token >= 0) at.page = kv4::load_page(p.batch, p.cache, row.seq, row.token);
        at.slot = row.token & ((1 << p.cache.page_shift) - 1);
      }
      if (lane == 0) places[i] = at;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n * half; j += blockDim.x) {
      const int i = j / half, f = j - i * half;
      if (places[i].seq < 0) continue;
      const float2 t = turn_of(places[i].position, p.spec.freqs[f], p.spec.amplitude);
      const float2 c = split16(t.x), s = split16(t.y);
      put_turn(t, f, half, INTERLEAVED, turns[i].c, turns[i].n);
      put_turn(make_float2(c.x, s.x), f, half, INTERLEAVED, turns[i].c_high, turns[i].n_high);
      put_turn(make_float2(c.y, s.y), f, half, INTERLEAVED, turns[i].c_low, turns[i].n_low);
    }
    __syncthreads();
  };
  // keys and values of all rows first: they are several times the work of queries
  const int kv_work = n * p.chunks, query_shares = shares - p.chunks;
  for (int work = warp; work < n * shares; work += warps) {
    const bool is_kv = work < kv_work;
    const int row = is_kv ? work / p.chunks : (work - kv_work) / query_shares;
    const int item = is_kv ? work - row * p.chunks : work - kv_work - row * query_shares;
    const int r = r0 + row;
    const SplitTurns<D>& t = turns[row];
    if (!is_kv) {
    // ---- queries
      const int i0 = item * (32 * kQueryUnits) + lane;
      const __nv_bfloat16* const from = p.Q + int64_t(r) * p.q_stride;
      uint4 a[kQueryUnits], c[kQueryUnits];
      UnitAt u[kQueryUnits];
      int at[kQueryUnits];
#pragma unroll
      for (int k = 0; k < kQueryUnits; ++k) {
        const int i = i0 + 32 * k;
        u[k] = unit_at(p.units, i, first);
        at[k] = u[k].head * D + unit_offset<INTERLEAVED>(p.units, u[k], p.spec.dim);
        a[k] = c[k] = make_uint4(0, 0, 0, 0);
        if (i < units) {
          a[k] = *reinterpret_cast<const uint4*>(from + at[k]);
          if (!INTERLEAVED && u[k].turned)
            c[k] = *reinterpret_cast<const uint4*>(from + at[k] + half);
        }
      }
      prepare();
      if (places[row].seq < 0) continue;
      __nv_bfloat16* const to = p.Q_out + int64_t(r) * p.qo_stride;
#pragma unroll
      for (int k = 0; k < kQueryUnits; ++k) {
        if (i0 + 32 * k >= units) continue;
        if (u[k].turned) {
          const int e = 8 * u[k].k;
          if (INTERLEAVED) {
            turn_interleaved(a[k], t.c + e, t.n + e, 4);
          } else {
            turn_runs(a[k], c[k], t.c + e, t.n + e);
            *reinterpret_cast<uint4*>(to + at[k] + half) = c[k];
          }
        }
        *reinterpret_cast<uint4*>(to + at[k]) = a[k];
      }
      continue;
    }
    // ---- keys and values
    const L my(lane, item);
    const bool there = my.head < p.cache.kv_heads;
    uint4 k[2], v[2], z[2];
    const __nv_bfloat16* from_k = p.K + int64_t(r) * p.k_stride + my.head * D + my.elem;
    const __nv_bfloat16* from_v = p.V + int64_t(r) * p.v_stride + my.head * D + my.elem;
    // a run of eight keys lies in the first half of the turned elements, in the
    // second, or behind them (dim is a multiple of 16)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = my.elem + 8 * i;
      k[i] = v[i] = z[i] = make_uint4(0, 0, 0, 0);
      if (there) {
        k[i] = *reinterpret_cast<const uint4*>(from_k + 8 * i);
        v[i] = *reinterpret_cast<const uint4*>(from_v + 8 * i);
        if (!INTERLEAVED && e < p.spec.dim)
          z[i] = *reinterpret_cast<const uint4*>(from_k + 8 * i + (e < half ? half : -half));
      }
    }
    prepare();
    const int64_t page = places[row].page;
    if (page < 0) continue;  // no token, no sequence, or a bad page
    const int slot = places[row].slot;
    const int64_t at = ((page * p.cache.kv_heads + my.head) << p.cache.page_shift) + slot;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (INTERLEAVED)
        z[i] = make_uint4(__byte_perm(k[i].x, 0u, 0x1032), __byte_perm(k[i].y, 0u, 0x1032),
                          __byte_perm(k[i].z, 0u, 0x1032), __byte_perm(k[i].w, 0u, 0x1032));
      if (my.elem + 8 * i < p.spec.dim) k[i] = turn_keys<D>(k[i], z[i], t, my.elem + 8 * i);
    }
    float ks, kz, vs, vz;
    const uint2 kw = kv4::quantize16<G / 16>(k, &ks, &kz);
    const uint2 vw = kv4::swap_chunks(kv4::quantize16<G / 16>(v, &vs, &vz), my.odd);
    if (there) {
      uint32_t* const to_k = reinterpret_cast<uint32_t*>(p.cache.k_codes + at * (D / 2));
      uint32_t* const to_v = reinterpret_cast<uint32_t*>(p.cache.v_codes + at * (D / 2));
      to_k[my.key_word(0)] = kw.x;
      to_k[my.key_word(1)] = kw.y;
      to_v[my.value_word(0)] = vw.x;
      to_v[my.value_word(1)] = vw.y;
      if (my.owns_meta) {
        p.cache.k_meta[at * L::NG + my.group] = __floats2half2_rn(ks, kz);
        p.cache.v_meta[at * L::NG + my.group] = __floats2half2_rn(vs, vz);
      }
    }
  }
  prepare();  // (the last CTA can have fewer shares than warps, all of which make the angles)
}

}  // namespace rotary
}  // namespace wq
