// rope.cu - rotary positions: pairs of each head's values turned by position * frequency.
//
//   (a, b) -> s (a cos t - b sin t, b cos t + a sin t),  t = position * freqs[j]
// half layout: pair j is (j, j + rot/2); interleaved: (2j, 2j + 1).  What lies behind rot is copied.
//
// Angles: a far position loses the angle in FP32 (2^20 * 2^-24 is 1/16 rad) and FP64 is slow here,
// so angles are integers: a frequency becomes the 64-bit fraction of a turn per position, the product
// with the position wraps as turns do, and the angle is off by at most 2^31 * 2^-64 turns before sine
// and cosine are taken in FP32 of what is left of the nearest quarter turn.
//
// Bound: the bytes (16384 tokens x 40 heads of 128 BF16, in one tensor: 52.9 us, 6.3 TB/s); small calls by
// latency (one token 2.0 us: positions, frequencies, table, a barrier, the heads).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

// Turns per position of a frequency in radians (|f| <= 2^32), as a 64-bit fraction (whole turns dropped): the
// 53 bits of f times 1 / (2 pi) in 128 bits, cut off where the fraction ends.  (FP64 arithmetic for this took
// 0.6 us more of a small call: an SM has little of it.)
__device__ __forceinline__ uint64_t turns(uint64_t f) {  // f: the FP64 number's bits
  const uint64_t c_hi = 0x28BE60DB9391054AULL, c_lo = 0x7F09D5F47D4D3770ULL;
  const uint32_t exponent = (uint32_t)(f >> 52) & 0x7FFu;
  const uint64_t m = (f & 0xFFFFFFFFFFFFFull) | (exponent ? 1ull << 52 : 0ull);  // f = m 2^(exponent - 1075)
  const uint64_t mid = m * c_hi, carry = __umul64hi(m, c_lo);
  const uint64_t p1 = mid + carry, p2 = __umul64hi(m, c_hi) + (p1 < mid ? 1u : 0u);  // above the low 64 bits
  const uint32_t shift = 64u + 1075u - max(exponent, 1u);  // at least 84
  const uint64_t r = shift < 128 ? p1 >> (shift - 64) | p2 << (128 - shift)
                                 : shift < 192 ? p2 >> (shift - 128) : 0ull;
  return f >> 63 ? 0ull - r : r;
}

// cosine and sine of a 64-bit fraction of a turn
__device__ __forceinline__ float2 cos_sin(uint64_t a) {
  const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(a - ((uint64_t)quarter << 62));  // within an eighth of a turn
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

template <int TYPE>
struct Elem;
template <>
struct Elem<QW_T_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ T put(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};
template <>
struct Elem<QW_T_F16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ T put(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
template <>
struct Elem<QW_T_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_ITEMS = 5 * ROPE_THREADS;    // that a CTA takes tokens for
constexpr int ROPE_TABLE = 2048;                // cosines and sines of a CTA, unless one token has more

struct Shape {
  RopeArgs a;
  int32_t tokens;    // of a CTA
  int32_t turn;      // items of a head that are turned
  int32_t per_head;  // ... and copied
  // a step of all threads, in heads and items of a head
  int32_t step_heads, step_items;
  int32_t groups;    // threads that share a frequency
  uint32_t by_half, by_head, by_heads;  // ceil(2^32 / d) for rot / 2, per_head and heads (0: d is 1)
};
// n / d; where n d passes 2^32 it may be one more
__device__ __forceinline__ int divide(int n, uint32_t by) { return by ? (int)__umulhi((uint32_t)n, by) : n; }
inline uint32_t divisor(int64_t d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + (uint64_t)d - 1) / (uint64_t)d); }

// A CTA makes its tokens' cosines and sines once for all heads, then each thread takes an item of V values of
// a head at a time (half layout: two vectors of V, rot / 2 apart; interleaved: one): 16 bytes where pitch,
// alignment and sizes allow, else 8, 4 or a value.  Items are counted on without divisions, which took most of
// the narrow forms' time (16384 tokens, 20 heads of 256, 126 turned: interleaved FP16 202 -> 109 us, half BF16
// 208 -> 148).
template <int TYPE, int LAYOUT, int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ Shape s) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  struct alignas(V * sizeof(T)) Vec {
    T v[V];
  };
  const RopeArgs& a = s.a;
  extern __shared__ float2 table[];  // [tokens][rot / 2]
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = (int64_t)blockIdx.x * s.tokens;
  const int tokens = (int)min64(s.tokens, a.T - t0), half = a.rot / 2;
  {
    const int groups = s.groups, group = groups > 1 ? divide((int)threadIdx.x, s.by_half) : 0;
    for (int j = (int)threadIdx.x - group * half; j < half && group < groups; j += ROPE_THREADS) {
      const uint64_t f = reinterpret_cast<const uint64_t*>(a.freqs)[j];
      const bool ok = (f & ~(1ull << 63)) <= 0x41F0000000000000ull;  // |f| <= 2^32 (NaN and infinity are above)
      if (!ok) set_error(a.err, QW_ERR_VALUE);
      const uint64_t per = ok ? turns(f) : 0;
      for (int t = group; t < tokens; t += groups) {
        float2 cs = cos_sin(per * (uint64_t)(int64_t)a.positions[t0 + t]);
        cs.x *= a.scale, cs.y *= a.scale;
        table[t * half + j] = ok ? cs : make_float2(NAN, NAN);
      }
      if (groups > 1) break;
    }
  }
  __syncthreads();
  constexpr int PAIRS = LAYOUT == QW_ROPE_HALF ? V : (V == 1 ? 1 : V / 2);  // of an item
  const int first = (int)(threadIdx.x + blockIdx.y * ROPE_THREADS);
  int head = divide(first, s.by_head), k = first - head * s.per_head, t = divide(head, s.by_heads);
  head -= t * a.heads;
  if (head < 0) head += a.heads, --t;  // (over 2^15 heads: one too many)
  auto advance = [&] {
    k += s.step_items;
    head += s.step_heads;
    if (k >= s.per_head) k -= s.per_head, ++head;
    while (head >= a.heads) head -= a.heads, ++t;
  };
  constexpr bool TWO = LAYOUT == QW_ROPE_HALF || V == 1;  // a pair's values lie in two vectors
  const int apart = LAYOUT == QW_ROPE_HALF ? half : 1;
  // (p, q) or p turned by the V / 2 or V angles from cs on
  auto turn = [](Vec& p, Vec& q, const float2* cs) {
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const float2 r = cs[j];
      T& lo = TWO ? p.v[j % V] : p.v[2 * j % V];
      T& hi = TWO ? q.v[j % V] : p.v[(2 * j + 1) % V];
      const float u = E::get(lo), w = E::get(hi);
      lo = E::put(u * r.x - w * r.y);
      hi = E::put(w * r.x + u * r.y);
    }
  };
  // Narrow items go several at a time, so that enough is on its way.
  constexpr int BYTES = V * (int)sizeof(T), U = BYTES >= 8 ? 1 : BYTES == 4 && LAYOUT == QW_ROPE_HALF ? 2 : 4;
  while (t < tokens) {
    if constexpr (U == 1) {
      const T* x = static_cast<const T*>(a.X) + (t0 + t) * a.ldx + (int64_t)head * a.head_dim;
      T* y = static_cast<T*>(a.Y) + (t0 + t) * a.ldy + (int64_t)head * a.head_dim;
      if (k >= s.turn) {
        const int c = a.rot + (k - s.turn) * V;
        *reinterpret_cast<Vec*>(y + c) = *reinterpret_cast<const Vec*>(x + c);
      } else {
        const int c = LAYOUT == QW_ROPE_HALF ? k * V : 2 * k * PAIRS;
        Vec p = *reinterpret_cast<const Vec*>(x + c), q{};
        if constexpr (TWO) q = *reinterpret_cast<const Vec*>(x + apart + c);
        turn(p, q, table + t * half + k * PAIRS);
        *reinterpret_cast<Vec*>(y + c) = p;
        if constexpr (TWO) *reinterpret_cast<Vec*>(y + apart + c) = q;
      }
      advance();
    } else {
      Vec p[U], q[U];
      T* y[U];
      const float2* cs[U];
      bool turned[U];
      int there = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (t >= tokens) continue;
        there = i + 1;
        turned[i] = k < s.turn;
        const int c = !turned[i] ? a.rot + (k - s.turn) * V : LAYOUT == QW_ROPE_HALF ? k * V : 2 * k * PAIRS;
        const T* x = static_cast<const T*>(a.X) + (t0 + t) * a.ldx + (int64_t)head * a.head_dim + c;
        y[i] = static_cast<T*>(a.Y) + (t0 + t) * a.ldy + (int64_t)head * a.head_dim + c;
        cs[i] = table + t * half + k * PAIRS;
        p[i] = *reinterpret_cast<const Vec*>(x);
        if (TWO && turned[i]) q[i] = *reinterpret_cast<const Vec*>(x + apart);
        advance();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (i >= there) continue;
        if (turned[i]) {
          turn(p[i], q[i], cs[i]);
          if (TWO) *reinterpret_cast<Vec*>(y[i] + apart) = q[i];
        }
        *reinterpret_cast<Vec*>(y[i]) = p[i];
      }
    }
  }
}

template <int TYPE, int LAYOUT, int V>
qw_status launch(const RopeArgs& a, cudaStream_t st) {
  Shape s{a};
  const int half = a.rot / 2, pairs = LAYOUT == QW_ROPE_HALF ? V : std::max(1, V / 2);
  s.turn = half / pairs;
  s.per_head = s.turn + (a.X == a.Y ? 0 : (a.head_dim - a.rot) / V);
  const int64_t per_token = (int64_t)s.per_head * a.heads;
  const int64_t sms = device_sm_count();
  int64_t tokens = std::min<int64_t>(ROPE_ITEMS / per_token, ROPE_TABLE / half);
  tokens = std::max<int64_t>(1, std::min(tokens, (a.T + 4 * sms - 1) / (4 * sms)));
  s.tokens = (int32_t)tokens;
  const int64_t blocks = (a.T + tokens - 1) / tokens;
  // few tokens: a token's heads are shared out among CTAs
  const int64_t need = (per_token * tokens + ROPE_THREADS - 1) / ROPE_THREADS;
  const int64_t split = std::max<int64_t>(1, std::min(need, 2 * sms / blocks));
  const int64_t step = split * ROPE_THREADS;
  s.step_heads = (int32_t)(step / s.per_head);
  s.step_items = (int32_t)(step % s.per_head);
  s.groups = std::max(1, ROPE_THREADS / half);
  s.by_half = divisor(half);
  s.by_head = divisor(s.per_head);
  s.by_heads = divisor(a.heads);
  const dim3 grid((unsigned)blocks, (unsigned)split);
  return launch_pdl(rope_kernel<TYPE, LAYOUT, V>, grid, dim3(ROPE_THREADS),
                    (size_t)tokens * half * sizeof(float2), st, s);
}

// the widest access that everything is a multiple of
template <int TYPE, int LAYOUT, int V>
qw_status launch_wide(const RopeArgs& a, cudaStream_t st) {
  constexpr int SIZE = TYPE == QW_T_F32 ? 4 : 2;
  const int part = LAYOUT == QW_ROPE_HALF ? a.rot / 2 : a.rot;
  const bool fits = ((uintptr_t)a.X | (uintptr_t)a.Y) % (V * SIZE) == 0 && a.ldx % V == 0 &&
                    a.ldy % V == 0 && a.head_dim % V == 0 && part % V == 0;
  if constexpr (V > 1) {
    if (!fits) return launch_wide<TYPE, LAYOUT, V / 2>(a, st);
  }
  return launch<TYPE, LAYOUT, V>(a, st);
}

template <int TYPE>
qw_status launch_layout(const RopeArgs& a, int32_t layout, cudaStream_t st) {
  constexpr int V = TYPE == QW_T_F32 ? 4 : 8;
  return layout == QW_ROPE_HALF ? launch_wide<TYPE, QW_ROPE_HALF, V>(a, st)
                                : launch_wide<TYPE, QW_ROPE_INTERLEAVED, V>(a, st);
}

}  // namespace

qw_status launch_rope(const RopeArgs& a, int32_t type, int32_t layout, cudaStream_t st) {
  if (type == QW_T_BF16) return launch_layout<QW_T_BF16>(a, layout, st);
  if (type == QW_T_F16) return launch_layout<QW_T_F16>(a, layout, st);
  return launch_layout<QW_T_F32>(a, layout, st);
}

// Frequencies in radians per position (host arithmetic in FP64).
qw_status rope_frequencies(int32_t method, double base, int32_t rot, double factor, double original,
                           double low, double high, double* freqs, float* attention) {
  const double two_pi = 6.283185307179586;
  if (method == QW_ROPE_NTK && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
  // mixed by index: the last pair that is kept, the first that is stretched as a whole
  auto pair_of = [&](double turns) { return rot * std::log(original / (two_pi * turns)) / (2.0 * std::log(base)); };
  double first = 0.0, last = 0.0;
  if (method == QW_ROPE_YARN_INDEX) {
    first = std::fmax(std::floor(pair_of(high)), 0.0);
    last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);  // (low 0: no pair is that slow)
  }
  for (int j = 0; j < rot / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot);
    if (method == QW_ROPE_LINEAR) f /= factor;
    double keep = 1.0;
    if (method == QW_ROPE_YARN || method == QW_ROPE_BANDS) {
      // turns within the original length: over `high` kept, under `low` stretched, between them mixed
      const double turns = original * f / two_pi;
      keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
    } else if (method == QW_ROPE_YARN_INDEX) {
      keep = j <= first ? 1.0 : j >= last ? 0.0 : 1.0 - (j - first) / (last - first);
    }
    if (keep < 1.0) f = f * (keep + (1.0 - keep) / factor);
    freqs[j] = f;
  }
  *attention = method == QW_ROPE_YARN || method == QW_ROPE_YARN_INDEX ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return QW_OK;
}

}  // namespace qw
