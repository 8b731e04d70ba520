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
// keys that go into the cache are the exact result rounded to binary32 (but for
// one in 2^20 or so), because a bit of a key next to a border between two codes is
// a whole step of the value that the cache holds.
#pragma once

#include "kv4.cuh"

namespace wq {
namespace rotary {

struct Spec {
  const float* freqs;  // [dim / 2], radians a position
  int dim;
  float amplitude;
};

// (c, s) of one position and frequency, in binary64 arithmetic that all heads share.
// The angle less a multiple of pi/2 that is held in two parts (W. J. Cody and W. Waite,
// 1980), then the series of sine and cosine to the 15th and 16th power: for |r| <= pi/4
// the next terms are below 2^-54.
__device__ __forceinline__ float2 turn_of(int position, float freq, float amplitude) {
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

// One pair in binary32.
__device__ __forceinline__ float2 turn_pair(float x1, float x2, float2 t) {
  return make_float2(fmaf(x1, t.x, -(x2 * t.y)), fmaf(x2, t.x, x1 * t.y));
}

// What one thread turns at a time: eight pairs (two runs of eight elements, or one
// of eight for interleaved pairs, which are four), or eight elements that stay.
// Units of a head: the turned ones first.
template <bool INTERLEAVED>
struct Units {
  int turned, all, half;
  __device__ __forceinline__ Units(int dim, int head_dim, bool copy) {
    half = dim / 2;
    turned = INTERLEAVED ? (dim + 7) / 8 : dim / 16;
    all = turned + (copy ? INTERLEAVED ? head_dim / 8 - turned : (head_dim - dim) / 8 : 0);
  }
  // offset of unit k's first element in its head
  __device__ __forceinline__ int offset(int k) const {
    return !INTERLEAVED && k >= turned ? 2 * half + 8 * (k - turned) : 8 * k;
  }
};

__device__ __forceinline__ void turn_runs(uint4& a, uint4& b, const float2* turn) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = kv4::bf16x2_to_float2(x[i]), q = kv4::bf16x2_to_float2(y[i]);
    const float4 t = *reinterpret_cast<const float4*>(turn + 2 * i);
    const float2 lo = turn_pair(p.x, q.x, make_float2(t.x, t.y));
    const float2 hi = turn_pair(p.y, q.y, make_float2(t.z, t.w));
    x[i] = pack_bf162(lo.x, hi.x);
    y[i] = pack_bf162(lo.y, hi.y);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

// Pairs side by side; the first `pairs` of the run's four turn.
__device__ __forceinline__ void turn_interleaved(uint4& a, const float2* turn, int pairs) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < pairs) {
      const float2 p = kv4::bf16x2_to_float2(x[i]);
      const float2 y = turn_pair(p.x, p.y, turn[i]);
      x[i] = pack_bf162(y.x, y.y);
    }
  a = make_uint4(x[0], x[1], x[2], x[3]);
}

constexpr int kMaxHead = 512;

struct RotaryParams {
  const __nv_bfloat16* X;  // [rows][heads][head_dim], rows x_stride elements apart
  int64_t x_stride;
  __nv_bfloat16* Y;  // X itself, or other memory
  int64_t y_stride;
  const int* positions;  // [rows]
  Spec spec;
  int heads, head_dim;
  bool copy;      // Y is other memory: the elements that stay are copied
  float sign;     // -1: the transpose
};

// A CTA takes one row (blockIdx.x) and, where there are few rows, a part of its
// units (blockIdx.y): the loads of each thread's first unit, the row's angles, then
// all heads.  HBM bound, two bytes in and two out an element.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(512, 2) rotary_kernel(const RotaryParams p) {
  __shared__ __align__(16) float2 turn[kMaxHead / 2];
  const int64_t r = blockIdx.x;
  const Units<INTERLEAVED> u(p.spec.dim, p.head_dim, p.copy);
  const unsigned units = unsigned(p.heads) * unsigned(u.all);
  const unsigned step = gridDim.y * blockDim.x;
  const __nv_bfloat16* const from = p.X + r * p.x_stride;
  __nv_bfloat16* const to = p.Y + r * p.y_stride;
  bool ready = false;
  for (unsigned i = blockIdx.y * blockDim.x + threadIdx.x;; i += step) {
    const bool there = i < units;
    const unsigned head = i / unsigned(u.all);
    const int k = int(i - head * unsigned(u.all));
    const int64_t at = int64_t(head) * p.head_dim + u.offset(k);
    const bool turned = k < u.turned;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (there) {
      a = *reinterpret_cast<const uint4*>(from + at);
      if (!INTERLEAVED && turned) b = *reinterpret_cast<const uint4*>(from + at + u.half);
    }
    if (!ready) {
      ready = true;
      const int position = p.positions[r];
      for (int j = threadIdx.x; j < u.half; j += blockDim.x) {
        const float2 t = turn_of(position, p.spec.freqs[j], p.spec.amplitude);
        turn[j] = make_float2(t.x, p.sign * t.y);
      }
      __syncthreads();
    }
    if (!there) return;
    if (turned) {
      if (INTERLEAVED) {
        turn_interleaved(a, turn + 4 * k, u.half - 4 * k);
      } else {
        turn_runs(a, b, turn + 8 * k);
        *reinterpret_cast<uint4*>(to + at + u.half) = b;
      }
    }
    *reinterpret_cast<uint4*>(to + at) = a;
  }
}

// The same for half layouts whose halves are not whole runs of eight elements
// (dim not a multiple of 16): a pair, or an element that stays, at a time.
static __global__ void __launch_bounds__(512, 2) rotary_pair_kernel(const RotaryParams p) {
  __shared__ __align__(16) float2 turn[kMaxHead / 2];
  const int64_t r = blockIdx.x;
  const int half = p.spec.dim / 2;
  const unsigned all = unsigned(half + (p.copy ? p.head_dim - 2 * half : 0));
  const unsigned units = unsigned(p.heads) * all;
  const int position = p.positions[r];
  for (int j = threadIdx.x; j < half; j += blockDim.x) {
    const float2 t = turn_of(position, p.spec.freqs[j], p.spec.amplitude);
    turn[j] = make_float2(t.x, p.sign * t.y);
  }
  __syncthreads();
  for (unsigned i = blockIdx.y * blockDim.x + threadIdx.x; i < units;
       i += gridDim.y * blockDim.x) {
    const unsigned head = i / all;
    const int k = int(i - head * all);
    const __nv_bfloat16* const from = p.X + r * p.x_stride + int64_t(head) * p.head_dim;
    __nv_bfloat16* const to = p.Y + r * p.y_stride + int64_t(head) * p.head_dim;
    if (k < half) {
      const float2 y = turn_pair(__bfloat162float(from[k]), __bfloat162float(from[k + half]),
                                 turn[k]);
      to[k] = __float2bfloat16_rn(y.x);
      to[k + half] = __float2bfloat16_rn(y.y);
    } else {
      to[k + half] = from[k + half];
    }
  }
}

// ------------------------------------------- on the way into the 4-bit cache

// A binary32 c as the sum of its leading 16 bits and the rest: products with a
// bfloat16 (8 bits) are exact with each part.
__device__ __forceinline__ float2 split16(float c) {
  const float hi = __uint_as_float(__float_as_uint(c) & 0xffffff00u);
  return make_float2(hi, c - hi);
}

// x c - z s rounded once to binary32: the leading products are exact, the error of
// their difference is found exactly (Knuth's two-sum), and what the low parts add is
// 2^-16 of the products with an error of 2^-24 of that.
__device__ __forceinline__ float turned_exactly(float x, float z, const float4& t) {
  const float a = x * t.x, b = z * t.z;
  const float d = a - b;
  const float back = d - a;
  const float err = (a - (d - back)) - (b + back);
  const float low = fmaf(x, t.y, -(z * t.w));
  const float y = d + (err + low);
  return fabsf(d) <= 3.4028234e38f ? y : d;  // infinite or NaN
}

// Eight keys (two words each of x and, for runs, of the partners z), turned.
template <bool INTERLEAVED>
__device__ __forceinline__ uint4 turn_keys(const uint4& x, const uint4& z, float sign,
                                           const float4* split) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z.x, z.y, z.z, z.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = kv4::bf16x2_to_float2(xs[i]), q = kv4::bf16x2_to_float2(zs[i]);
    if (INTERLEAVED) {
      const float4 t = split[i];
      y[i] = pack_bf162(turned_exactly(p.x, p.y, t), turned_exactly(p.y, -p.x, t));
    } else {
      y[i] = pack_bf162(turned_exactly(p.x, sign * q.x, split[2 * i]),
                        turned_exactly(p.y, sign * q.y, split[2 * i + 1]));
    }
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
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
};

constexpr int kMaxWarps = 8;
constexpr int kQueryUnits = 2;  // units of queries a lane has in flight

// Queries turned, keys turned and quantized, values quantized: one CTA a row, whose
// angles its warps share; the first `chunks` shares are 512 keys and values each, the
// others 64 units of queries.  CTAs behind the
// rows check the sequences.
template <int D, int G, bool INTERLEAVED>
__global__ void __launch_bounds__(kMaxWarps * 32, 4)
    write_rotary_kernel(const WriteParams p, int warps_of_rows) {
  using L = KeyLane<D, G>;
  __shared__ __align__(16) float2 turn[D / 2];
  __shared__ float4 split[D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (int(blockIdx.x) >= p.batch.rows) {
    kv4::check_sequences(p.batch, (int(blockIdx.x) - p.batch.rows) * warps + warp,
                         (int(gridDim.x) - p.batch.rows) * warps, lane);
    return;
  }
  const int r = blockIdx.x;
  const Units<INTERLEAVED> u(p.spec.dim, D, p.copy_q);
  const unsigned units = unsigned(p.q_heads) * unsigned(u.all);
  const int b = kv4::find_sequence(p.batch, r, lane);
  if (b < 0) return;
  const kv4::Sequence seq = kv4::load_sequence(p.batch, b);
  if (r < seq.row0 || r >= seq.row0 + seq.rows) return;
  const int token = seq.len - seq.rows + (r - seq.row0);
  bool ready = false;
  auto make_turns = [&] {
    if (ready) return;
    ready = true;
    const int position = p.positions != nullptr ? p.positions[r] : token;
    for (int j = threadIdx.x; j < u.half; j += blockDim.x) {
      const float2 t = turn_of(position, p.spec.freqs[j], p.spec.amplitude);
      const float2 c = split16(t.x), s = split16(t.y);
      turn[j] = t;
      split[j] = make_float4(c.x, c.y, s.x, s.y);
    }
    __syncthreads();
  };
  for (int item = warp; item < warps_of_rows; item += warps) {
    if (item >= p.chunks) {
      // ---- queries
      const unsigned i0 = unsigned(item - p.chunks) * (32 * kQueryUnits) + lane;
      uint4 a[kQueryUnits], c[kQueryUnits];
#pragma unroll
      for (int k = 0; k < kQueryUnits; ++k) {
        const unsigned i = i0 + 32 * k, head = i / unsigned(u.all);
        const int unit = int(i - head * unsigned(u.all));
        const __nv_bfloat16* from =
            p.Q + int64_t(r) * p.q_stride + int64_t(head) * D + u.offset(unit);
        a[k] = c[k] = make_uint4(0, 0, 0, 0);
        if (i < units) {
          a[k] = *reinterpret_cast<const uint4*>(from);
          if (!INTERLEAVED && unit < u.turned)
            c[k] = *reinterpret_cast<const uint4*>(from + u.half);
        }
      }
      make_turns();
#pragma unroll
      for (int k = 0; k < kQueryUnits; ++k) {
        const unsigned i = i0 + 32 * k, head = i / unsigned(u.all);
        const int unit = int(i - head * unsigned(u.all));
        if (i >= units) continue;
        __nv_bfloat16* to = p.Q_out + int64_t(r) * p.qo_stride + int64_t(head) * D + u.offset(unit);
        if (unit < u.turned) {
          if (INTERLEAVED) {
            turn_interleaved(a[k], turn + 4 * unit, 4);
          } else {
            turn_runs(a[k], c[k], turn + 8 * unit);
            *reinterpret_cast<uint4*>(to + u.half) = c[k];
          }
        }
        *reinterpret_cast<uint4*>(to) = a[k];
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
    int run_at[2];
    float sign[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = my.elem + 8 * i;
      run_at[i] = e >= p.spec.dim ? -1 : INTERLEAVED ? e / 2 : e >= u.half ? e - u.half : e;
      sign[i] = e < u.half ? 1.f : -1.f;
      k[i] = v[i] = z[i] = make_uint4(0, 0, 0, 0);
      if (there) {
        k[i] = *reinterpret_cast<const uint4*>(from_k + 8 * i);
        v[i] = *reinterpret_cast<const uint4*>(from_v + 8 * i);
        if (!INTERLEAVED && run_at[i] >= 0)
          z[i] = *reinterpret_cast<const uint4*>(from_k + 8 * i +
                                                 (sign[i] > 0.f ? u.half : -u.half));
      }
    }
    make_turns();
    if (token < 0) continue;  // the row holds no token
    const int64_t page = kv4::load_page(p.batch, p.cache, b, token);
    if (page < 0) continue;
    const int slot = token & ((1 << p.cache.page_shift) - 1);
    const int64_t at = ((page * p.cache.kv_heads + my.head) << p.cache.page_shift) + slot;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (run_at[i] >= 0)
        k[i] = turn_keys<INTERLEAVED>(k[i], z[i], sign[i], split + run_at[i]);
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
}

}  // namespace rotary
}  // namespace wq
