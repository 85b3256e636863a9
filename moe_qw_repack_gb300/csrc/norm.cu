// norm.cu - residual addition, root-mean-square norm and the operand of the product behind it, in one
// pass over the row.
//
//   h = x + r (as stored: rounded to r's type; without r: x)
//   y[k] = h[k] w[k] / sqrt(mean h^2 + eps)
// y leaves as BF16, as MXFP8 (qw_quantize_mxfp8's conversion) or as INT8 codes with a scale per row
// (qw_quantize_int8's), both from the FP32 y: rounded to BF16 on the way, a code would be off by up to
// 1/4 of a step more.
//
// Arithmetic: sums of squares in FP32.  h w is formed first: of BF16 values it is exact, and an FP32
// h costs one rounding; 1 / rms is held as a sum of two FP32 numbers, so y has one more rounding.
// Squares that pass FP32 (|h| above 2^63 or so) take a second reduction on h scaled by a power of two.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Eight values of a row from element 8 i, as they lie in memory.  Plain loads: the previous kernel may have
// written them, and this one may write h or y to the same place.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void fetch8(const void* row, int i, Raw<F32>& x) {
  const uint4* p = static_cast<const uint4*>(row);
  if constexpr (F32)
    x.v[0] = p[2 * i], x.v[1] = p[2 * i + 1];
  else
    x.v[0] = p[i];
}
template <bool F32>
__device__ __forceinline__ void widen8(const Raw<F32>& x, float (&f)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[4 * j] = __uint_as_float(x.v[j].x), f[4 * j + 1] = __uint_as_float(x.v[j].y);
      f[4 * j + 2] = __uint_as_float(x.v[j].z), f[4 * j + 3] = __uint_as_float(x.v[j].w);
    }
  } else {
    unpack8(x.v[0], f);
  }
}
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int i, float (&f)[8]) {
  Raw<F32> x;
  fetch8<F32>(row, i, x);
  widen8<F32>(x, f);
}
template <bool F32>
__device__ __forceinline__ const void* row_of(const void* p, int64_t r, int64_t ld) {
  return static_cast<const uint8_t*>(p) + r * ld * (F32 ? 4 : 2);
}

// What a row is held as: nothing beside x, or a residual in BF16 or FP32.
enum { R_NONE = 0, R_BF16 = 1, R_F32 = 2 };
enum { Q_NONE = 0, Q_INT8 = 1, Q_MXFP8 = 2 };

constexpr int NORM_WARPS = 4;  // rows of a CTA where a warp takes a row

__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
template <bool ONE_WARP>
struct Reduce {
  float* part;  // [32]
  // Sums or maxima over the row's threads; every thread gets the result.
  template <class F>
  __device__ __forceinline__ float operator()(float v, F&& join) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if constexpr (!ONE_WARP) {
      const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
      __syncthreads();  // (the last result has been read)
      if (lane == 0) part[threadIdx.x >> 5] = v;
      __syncthreads();
      v = part[lane < warps ? lane : 0];
      if (lane >= warps) v = 0.f;  // (sums, and maxima of magnitudes)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v) const {
    return (*this)(v, [](float a, float b) { return a + b; });
  }
  // of magnitudes, NaN above all
  __device__ __forceinline__ float top(float v) const {
    return (*this)(v, [](float a, float b) { return max_nan(a, b); });
  }
};

// two FP32 values -> two E4M3 codes, x0 in the low byte (round to nearest even, saturate)
__device__ __forceinline__ uint32_t e4m3x2(float x0, float x1) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(x1), "f"(x0));
  return d;
}

// How rows are shared out; a thread has VEC vectors of eight values.
//   ROWS_WARP   a warp takes a row (K <= 1024): no barrier
//   ROWS_ONE    a CTA takes one row: few rows, or long ones
//   ROWS_MANY   CTAs take rows in turn, the next row's values on their way while one is worked on, and keep
//               the weights
// Bound: the bytes, and close under them the instructions (29 an element to BF16 and MXFP8), whose reductions
// and addresses are per row: more vectors a thread are fewer of them.  8192 x 4096, residual, to BF16 and MXFP8:
// 55.2 us with a CTA a row, 54.0 in turn with two vectors a thread, 50.9 with four (5.95 TB/s).
enum { ROWS_WARP = 0, ROWS_ONE = 1, ROWS_MANY = 2 };
constexpr int threads_of(int form) { return form == ROWS_WARP ? NORM_WARPS * 32 : form == ROWS_ONE ? 1024 : 512; }

template <bool X32, int RK, int QF, int VEC, int FORM>
__global__ void __launch_bounds__(threads_of(FORM), FORM == ROWS_WARP ? 6 : 1)
    rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool ONE_WARP = FORM == ROWS_WARP, MANY = FORM == ROWS_MANY;
  constexpr bool R32 = RK == R_F32;
  __shared__ float part[32];
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = ONE_WARP ? 32 : blockDim.x;
  const int me = ONE_WARP ? threadIdx.x & 31 : threadIdx.x;
  int64_t row = ONE_WARP ? (int64_t)blockIdx.x * NORM_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (ONE_WARP && row >= a.rows) return;
  const Reduce<ONE_WARP> reduce{part};
  const int n8 = a.K / 8;
  const uint4* w = static_cast<const uint4*>(a.W);
  Raw<X32> raw_x[VEC];
  Raw<R32> raw_r[VEC];
  uint4 weights[MANY ? VEC : 1];
  auto fetch = [&](int64_t row) {
    const void* xr = row_of<X32>(a.X, row, a.ldx);
    const void* rr = row_of<R32>(a.R, row, a.ldr);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int i = me + v * lanes;
      if (i >= n8) continue;
      fetch8<X32>(xr, i, raw_x[v]);
      if constexpr (RK != R_NONE) fetch8<R32>(rr, i, raw_r[v]);
    }
  };
  fetch(row);
  if constexpr (MANY) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (me + v * lanes < n8) weights[v] = w[me + v * lanes];
  }
  do {
    const void* xr = row_of<X32>(a.X, row, a.ldx);
    const void* rr = row_of<R32>(a.R, row, a.ldr);
    void* ro = RK == R_NONE ? nullptr : const_cast<void*>(row_of<R32>(a.R_out, row, a.ldro));
    const bool keep_h = RK != R_NONE && a.R_out != nullptr;
    // h, from x and r, rounded as r is
    auto join8 = [&](int i, const Raw<X32>& x, const Raw<R32>& rv, float (&h)[8]) {
      widen8<X32>(x, h);
      if constexpr (RK != R_NONE) {
        float r[8];
        widen8<R32>(rv, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
        if constexpr (RK == R_BF16) {
          const uint4 v = pack8(h);
          unpack8(v, h);
          if (keep_h) static_cast<uint4*>(ro)[i] = v;
        } else if (keep_h) {
          float4* o = static_cast<float4*>(ro) + 2 * i;
          o[0] = make_float4(h[0], h[1], h[2], h[3]);
          o[1] = make_float4(h[4], h[5], h[6], h[7]);
        }
      }
    };
    auto sum8 = [&](int i, float (&h)[8]) {
      Raw<X32> x;
      Raw<R32> r;
      fetch8<X32>(xr, i, x);
      if constexpr (RK != R_NONE) fetch8<R32>(rr, i, r);
      join8(i, x, r, h);
    };
    // ... again, for what the registers do not hold: h as it was stored (r may be gone by now)
    auto again8 = [&](int i, float (&h)[8]) {
      if (keep_h)
        load8<R32>(ro, i, h);
      else
        sum8(i, h);
    };
    float h[VEC][8], ss = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int i = me + v * lanes;
      if (i < n8) {
        join8(i, raw_x[v], raw_r[v], h[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] = 0.f;
      }
    }
    if (MANY && row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[v][j], h[v][j], ss);
    for (int i = me + VEC * lanes; i < n8; i += lanes) {
      float t[8];
      sum8(i, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(t[j], t[j], ss);
    }
    ss = reduce.sum(ss);
    float pre = 1.f;  // h is taken times this power of two
    if (!(ss < 0x1p126f)) {  // (the same in all of the row's threads)
      float top = 0.f;
      auto more = [&](const float (&t)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          top = max_nan(top, fabsf(t[j]));
      };
#pragma unroll
      for (int v = 0; v < VEC; ++v) more(h[v]);
      for (int i = me + VEC * lanes; i < n8; i += lanes) {
        float t[8];
        again8(i, t);
        more(t);
      }
      top = reduce.top(top);
      pre = top < INFINITY ? 0x1p-96f : __uint_as_float(0x7FC00000u);
      ss = 0.f;
      auto squares = [&](const float (&t)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(t[j] * pre, t[j] * pre, ss);
      };
#pragma unroll
      for (int v = 0; v < VEC; ++v) squares(h[v]);
      for (int i = me + VEC * lanes; i < n8; i += lanes) {
        float t[8];
        again8(i, t);
        squares(t);
      }
      ss = reduce.sum(ss);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] *= pre;
    }
    // 1 / sqrt(m) and what its rounding left: one Newton step from the exact residual 1 - m r^2
    const float m = ss / (float)a.K + a.eps * pre * pre;
    const float r_hi = rsqrtf(m), mr = m * r_hi;
    const float r_lo = 0.5f * r_hi * fmaf(-fmaf(m, r_hi, -mr), r_hi, fmaf(-mr, r_hi, 1.f));
    auto out8 = [&](const uint4& wv, const float (&h8)[8], float (&y)[8]) {
      float w8[8];
      unpack8(wv, w8);
      if (a.offset != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w8[j] += a.offset;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = h8[j] * w8[j];
        y[j] = fmaf(p, r_hi, p * r_lo);
      }
    };
    auto tail8 = [&](int i, float (&y)[8]) {
      again8(i, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= pre;
      out8(w[i], y, y);
    };
    auto weight = [&](int v, int i) { return MANY ? weights[MANY ? v : 0] : w[i]; };
    uint16_t* yr = a.Y ? static_cast<uint16_t*>(a.Y) + row * a.ldy : nullptr;
    float inv = 0.f, scale = 0.f, down = 1.f;
    bool bad = pre != pre;
    if constexpr (QF == Q_INT8) {
      float top = 0.f;
      auto more = [&](const float (&y)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          top = max_nan(top, fabsf(y[j]));
      };
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int i = me + v * lanes;
        if (i < n8) {
          out8(weight(v, i), h[v], h[v]);
          more(h[v]);
        }
      }
      for (int i = me + VEC * lanes; i < n8; i += lanes) {
        float t[8];
        tail8(i, t);
        more(t);
      }
      top = reduce.top(top);
      bad = bad || !(top < INFINITY);
      scale = bad ? __uint_as_float(0x7FC00000u) : top / 127.f;
      inv = bad || top < FLT_MIN ? 0.f : 127.f / top;
      // Below 2^-121 the quotient passes FP32: such a row is taken times 2^64, which is exact.  (A factor in all
      // rows: 8192 x 4096 38.4 us instead of 37.6.)  A row without a normal number has codes 0.
      if (top < 0x1p-119f) {
        down = 0x1p-64f;
        if (top >= FLT_MIN) inv = 127.f / (top * 0x1p64f);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) h[v][j] *= 0x1p64f;
      }
    }
    auto put8 = [&](int i, const float (&y)[8]) {
      if (yr) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = QF == Q_INT8 ? y[j] * down : y[j];
        reinterpret_cast<uint4*>(yr)[i] = pack8(z);
      }
      if constexpr (QF == Q_INT8) {
        // adding 1.5 * 2^23 rounds to an integer, ties to even, in the sum's low bits
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          q[j] = __float_as_uint(__fadd_rn(__fmul_rn(y[j], inv), 12582912.f));
        uint2 o;
        o.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
        o.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
        if (bad) o = make_uint2(0, 0);
        reinterpret_cast<uint2*>(a.Q)[row * n8 + i] = o;
      }
    };
    // (MXFP8: all lanes of a warp together; K % 32 == 0, so that a group's four threads are there or not)
    auto put8_mx = [&](int i, const float (&y)[8], bool live) {
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(y[j]));
      most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      const uint32_t top = __float_as_uint(most);
      const bool sick = !(most < INFINITY);
      bad = bad || sick;
      int X = -127;
      if (top != 0) {
        const int ef = (int)(top >> 23);
        const int fl = ef > 0 ? ef - 127 : -149 + (31 - __clz(top));  // floor(log2 max |y|)
        X = max(-127, min(127, fl - 8));
      }
      const float to = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X, X in [-127, 119]
      uint2 q;
      q.x = e4m3x2(y[0] * to, y[1] * to) | (e4m3x2(y[2] * to, y[3] * to) << 16);
      q.y = e4m3x2(y[4] * to, y[5] * to) | (e4m3x2(y[6] * to, y[7] * to) << 16);
      if (live) {
        if (yr) reinterpret_cast<uint4*>(yr)[i] = pack8(y);
        reinterpret_cast<uint2*>(a.Q)[row * n8 + i] = sick ? make_uint2(0, 0) : q;
        if ((i & 3) == 0)
          static_cast<uint8_t*>(a.Q_sf)[row * (n8 / 4) + (i >> 2)] = sick ? 0xFF : (uint8_t)(X + 127);
      }
    };
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int i = me + v * lanes;
      if constexpr (QF == Q_MXFP8) {
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < n8) out8(weight(v, i), h[v], y);
        put8_mx(i, y, i < n8);
      } else if (i < n8) {
        if constexpr (QF == Q_NONE) out8(weight(v, i), h[v], h[v]);  // (INT8: already y)
        put8(i, h[v]);
      }
    }
    for (int i0 = VEC * lanes; i0 < n8; i0 += lanes) {
      const int i = i0 + me;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (i < n8) tail8(i, y);
      if (QF == Q_INT8 && down != 1.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= 0x1p64f;
      }
      if constexpr (QF == Q_MXFP8)
        put8_mx(i, y, i < n8);
      else if (i < n8)
        put8(i, y);
    }
    if constexpr (QF == Q_INT8) {
      if (me == 0) static_cast<float*>(a.Q_sf)[row] = scale;
    }
    if (bad) set_error(a.err, QW_ERR_VALUE);
    row += gridDim.x;
  } while (MANY && row < a.rows);
}

template <bool X32, int RK, int QF>
qw_status launch(const NormArgs& a, cudaStream_t st) {
  const int n8 = a.K / 8, sms = device_sm_count();
  auto go = [&](auto kernel, int64_t grid, int threads) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3((unsigned)threads), 0, st, a);
  };
  auto threads = [&](int vec) { return ((n8 + vec - 1) / vec + 31) / 32 * 32; };
  if (n8 <= 128)
    return go(rmsnorm_kernel<X32, RK, QF, 4, ROWS_WARP>, (a.rows + NORM_WARPS - 1) / NORM_WARPS, NORM_WARPS * 32);
  // One vector a thread while each row has an SM (us at 1 x 4096: 2.1, with two vectors 2.6, with four 3.5),
  // two while they are no more than what runs at once, or where a row is too long to be kept.
  constexpr bool heavy = X32 || RK == R_F32;  // twice the registers for what is on its way
  constexpr int VEC = heavy ? 2 : 4;
  const int64_t at_once = (int64_t)sms * std::max(1, 512 / threads(VEC));
  if (n8 > 512 * VEC || a.rows <= at_once) {
    if (n8 <= 1024 && a.rows <= sms) return go(rmsnorm_kernel<X32, RK, QF, 1, ROWS_ONE>, a.rows, threads(1));
    return go(rmsnorm_kernel<X32, RK, QF, 2, ROWS_ONE>, a.rows, std::min(1024, threads(2)));
  }
  return go(rmsnorm_kernel<X32, RK, QF, VEC, ROWS_MANY>, at_once, threads(VEC));
}

template <bool X32, int RK>
qw_status launch_q(const NormArgs& a, int q_fmt, cudaStream_t st) {
  if (q_fmt == QW_A_INT8_TOKEN) return launch<X32, RK, Q_INT8>(a, st);
  if (q_fmt == QW_A_MXFP8_G32) return launch<X32, RK, Q_MXFP8>(a, st);
  return launch<X32, RK, Q_NONE>(a, st);
}
template <bool X32>
qw_status launch_r(const NormArgs& a, int r_type, int q_fmt, cudaStream_t st) {
  if (!a.R) return launch_q<X32, R_NONE>(a, q_fmt, st);
  return r_type == QW_T_F32 ? launch_q<X32, R_F32>(a, q_fmt, st) : launch_q<X32, R_BF16>(a, q_fmt, st);
}

}  // namespace

qw_status launch_rmsnorm(const NormArgs& a, int32_t x_type, int32_t r_type, int32_t q_fmt,
                         cudaStream_t st) {
  return x_type == QW_T_F32 ? launch_r<true>(a, r_type, q_fmt, st)
                            : launch_r<false>(a, r_type, q_fmt, st);
}

}  // namespace qw
