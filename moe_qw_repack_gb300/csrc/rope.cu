// rope.cu - rotary positions: pairs of each head's values turned by position * frequency.
//
//   (a, b) -> s (a cos t - b sin t, b cos t + a sin t),  t = position * freqs[j]
// half layout: pair j is (j, j + rot/2); interleaved: (2j, 2j + 1).  What lies behind rot is copied.
//
// Angles: a far position loses the angle in FP32 (2^20 * 2^-24 is 1/16 rad) and FP64 is slow here,
// so angles are integers: a frequency becomes the 64-bit fraction of a turn per position, the product
// with the position wraps as turns do, and the angle is off by at most 2^31 * 2^-64 turns before sine
// and cosine are taken in FP32 of what is left of the nearest quarter turn.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

// Turns per position of a frequency in radians, as a 64-bit fraction (whole turns dropped).
// 1/(2 pi) in two FP64 parts: 0.15915494309189535 - 9.8393383375... e-18.
__device__ __forceinline__ uint64_t turns(double f) {
  const double c_hi = 0.15915494309189535, c_lo = -9.839338337591243e-18;
  const double hi = f * c_hi, lo = fma(f, c_hi, -hi) + f * c_lo;
  return __double2ull_rn((hi - floor(hi)) * 0x1p64) + (uint64_t)__double2ll_rn(lo * 0x1p64);
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
constexpr int ROPE_TOKENS = 4;

// V: elements of a thread's vector (16 bytes), or 1 where pitch, alignment or sizes do not allow it.
template <int TYPE, int LAYOUT, int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeArgs a) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  struct alignas(V * sizeof(T)) Vec {
    T v[V];
  };
  extern __shared__ float2 table[];  // [tokens][rot / 2]
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = (int64_t)blockIdx.x * ROPE_TOKENS;
  const int tokens = (int)min64(ROPE_TOKENS, a.T - t0), half = a.rot / 2;
  for (int j = threadIdx.x; j < half; j += ROPE_THREADS) {
    const double f = a.freqs[j];
    const bool ok = fabs(f) <= 0x1p32;
    if (!ok) set_error(a.err, QW_ERR_VALUE);
    const uint64_t per = ok ? turns(f) : 0;
    for (int t = 0; t < tokens; ++t) {
      float2 cs = cos_sin(per * (uint64_t)(int64_t)a.positions[t0 + t]);
      cs.x *= a.scale, cs.y *= a.scale;
      table[t * half + j] = ok ? cs : make_float2(NAN, NAN);
    }
  }
  __syncthreads();
  const T* X = static_cast<const T*>(a.X);
  T* Y = static_cast<T*>(a.Y);
  // A head's items: vectors of pairs (half layout: two vectors, rot / 2 apart), then (unless in place)
  // vectors to copy.
  constexpr int PAIRS = LAYOUT == QW_ROPE_HALF ? V : (V == 1 ? 1 : V / 2);  // of an item
  const int turn = half / PAIRS, keep = a.X == a.Y ? 0 : (a.head_dim - a.rot) / V;
  const int per_head = turn + keep, per_token = per_head * a.heads;
  for (int i = threadIdx.x + blockIdx.y * ROPE_THREADS; i < per_token * tokens;
       i += ROPE_THREADS * gridDim.y) {
    const int t = i / per_token, rest = i - t * per_token, head = rest / per_head;
    const int k = rest - head * per_head;
    const T* x = X + (t0 + t) * a.ldx + (int64_t)head * a.head_dim;
    T* y = Y + (t0 + t) * a.ldy + (int64_t)head * a.head_dim;
    if (k >= turn) {
      const int c = a.rot + (k - turn) * V;
      *reinterpret_cast<Vec*>(y + c) = *reinterpret_cast<const Vec*>(x + c);
    } else if constexpr (LAYOUT == QW_ROPE_HALF) {
      const int c = k * V;
      Vec p = *reinterpret_cast<const Vec*>(x + c), q = *reinterpret_cast<const Vec*>(x + half + c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 cs = table[t * half + c + j];
        const float u = E::get(p.v[j]), w = E::get(q.v[j]);
        p.v[j] = E::put(u * cs.x - w * cs.y);
        q.v[j] = E::put(w * cs.x + u * cs.y);
      }
      *reinterpret_cast<Vec*>(y + c) = p;
      *reinterpret_cast<Vec*>(y + half + c) = q;
    } else if constexpr (V == 1) {
      const float2 cs = table[t * half + k];
      const float u = E::get(x[2 * k]), w = E::get(x[2 * k + 1]);
      y[2 * k] = E::put(u * cs.x - w * cs.y);
      y[2 * k + 1] = E::put(w * cs.x + u * cs.y);
    } else {
      Vec p = *reinterpret_cast<const Vec*>(x + k * V);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 cs = table[t * half + k * PAIRS + j];
        const float u = E::get(p.v[2 * j]), w = E::get(p.v[2 * j + 1]);
        p.v[2 * j] = E::put(u * cs.x - w * cs.y);
        p.v[2 * j + 1] = E::put(w * cs.x + u * cs.y);
      }
      *reinterpret_cast<Vec*>(y + k * V) = p;
    }
  }
}

template <int TYPE, int LAYOUT>
qw_status launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int SIZE = TYPE == QW_T_F32 ? 4 : 2, V = 16 / SIZE;
  const int part = LAYOUT == QW_ROPE_HALF ? a.rot / 2 : a.rot;
  const bool wide = ((uintptr_t)a.X | (uintptr_t)a.Y) % 16 == 0 && a.ldx % V == 0 &&
                    a.ldy % V == 0 && a.head_dim % V == 0 && part % V == 0;
  const int64_t blocks = (a.T + ROPE_TOKENS - 1) / ROPE_TOKENS;
  const int64_t items = (int64_t)a.heads * a.head_dim * ROPE_TOKENS / (wide ? V : 1);
  int64_t split = (items + 2 * ROPE_THREADS - 1) / (2 * ROPE_THREADS);
  const int64_t most = std::max<int64_t>(1, 2 * device_sm_count() / blocks);
  split = std::max<int64_t>(1, std::min(split, most));
  const dim3 grid((unsigned)blocks, (unsigned)split);
  const size_t smem = (size_t)ROPE_TOKENS * (a.rot / 2) * sizeof(float2);
  return wide ? launch_pdl(rope_kernel<TYPE, LAYOUT, V>, grid, dim3(ROPE_THREADS), smem, st, a)
              : launch_pdl(rope_kernel<TYPE, LAYOUT, 1>, grid, dim3(ROPE_THREADS), smem, st, a);
}

template <int TYPE>
qw_status launch_layout(const RopeArgs& a, int32_t layout, cudaStream_t st) {
  return layout == QW_ROPE_HALF ? launch<TYPE, QW_ROPE_HALF>(a, st)
                                : launch<TYPE, QW_ROPE_INTERLEAVED>(a, st);
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
  for (int j = 0; j < rot / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot);
    if (method == QW_ROPE_LINEAR) f /= factor;
    if (method == QW_ROPE_YARN || method == QW_ROPE_BANDS) {
      // turns within the original length: over `high` kept, under `low` stretched, between them mixed
      const double turns = original * f / two_pi;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f = f * (keep + (1.0 - keep) / factor);
    }
    freqs[j] = f;
  }
  *attention = method == QW_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return QW_OK;
}

}  // namespace qw
