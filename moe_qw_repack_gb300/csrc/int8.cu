// int8.cu - the INT8 product with a scale per token and per output channel, its gated form,
// and the per-token quantiser in front of them.
//
//   q[m][k] = rint(a[m][k] * min(127 / amax_m, FLT_MAX)),  sa_m = amax_m / 127
//   C[m][n] = sa_m * sw_n * sum_k q[m][k] w[n][k] + bias[n]
//   Y[m][i] = silu(C[m][i]) * C[m][I + i]                               (gated)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A signed 8-bit integer as its FP16 number's bits (exact).
__device__ __forceinline__ uint32_t f16_of(float q) {
  return (uint32_t)__half_as_ushort(__float2half_rn(q));
}

// Row r of A -> codes (INT8, or the same integers as FP16 for the tensor cores) and the row's
// scale.  One CTA per row.  A thread keeps its part of rows of up to 256 x 8 vectors of 16 bytes
// (K <= 16384) in registers, so the row is read once; what lies beyond is read a second time.
constexpr int QTHREADS = 256, QVEC = 8;
template <bool F16>
__global__ void __launch_bounds__(QTHREADS)
    quantize_int8_kernel(const uint16_t* __restrict__ A, int64_t lda, int32_t K,
                         void* __restrict__ Q, float* __restrict__ S, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(A + r * lda);
  const int n8 = K / 8;
  uint4 keep[QVEC];
  uint32_t amax = 0;  // largest |v| as BF16 bits (finite values order like their bit patterns)
  auto fold = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  };
#pragma unroll
  for (int j = 0; j < QVEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    keep[j] = i < n8 ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < QVEC; ++j) fold(keep[j]);
  for (int i = threadIdx.x + QVEC * QTHREADS; i < n8; i += QTHREADS) fold(__ldg(src + i));
  __shared__ uint32_t part[QTHREADS / 32];
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = part[0];
#pragma unroll
  for (int i = 1; i < QTHREADS / 32; ++i) amax = max(amax, part[i]);
  const float top = __uint_as_float(amax << 16);
  const bool finite = amax < 0x7F80u;
  const float inv = finite ? fminf(127.0f / top, 3.4028234663852886e38f) : 0.f;
  if (threadIdx.x == 0) {
    S[r] = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
    if (!finite) set_error(err, QW_ERR_VALUE);
  }
  auto put = [&](int i, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (F16) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = finite ? f16_of(rintf(bf16_lo(w[j]) * inv)) | (f16_of(rintf(bf16_hi(w[j]) * inv)) << 16)
                      : 0u;
      reinterpret_cast<uint4*>(Q)[r * (K / 8) + i] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = finite ? __float2int_rn(((j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1])) * inv) : 0;
        o[j >> 2] |= ((uint32_t)q & 0xFFu) << (8 * (j & 3));
      }
      reinterpret_cast<uint2*>(Q)[r * (K / 8) + i] = make_uint2(o[0], o[1]);
    }
  };
#pragma unroll
  for (int j = 0; j < QVEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    if (i < n8) put(i, keep[j]);
  }
  for (int i = threadIdx.x + QVEC * QTHREADS; i < n8; i += QTHREADS) put(i, __ldg(src + i));
}

// INT8 codes [M][lda] -> the same integers as FP16 [M][K]; a thread takes 16 codes at a time.
__global__ void __launch_bounds__(256)
    widen_int8_kernel(const int8_t* __restrict__ A, int64_t lda, int64_t M, int32_t K,
                      uint4* __restrict__ Q) {
  pdl_wait();
  pdl_launch_dependents();
  const int32_t per_row = K / 16;
  const int64_t total = M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row;
    const int32_t c = (int32_t)(i - r * per_row);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(A + r * lda) + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) int8x4_to_f16x2(w[j], o[2 * j], o[2 * j + 1]);
    Q[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    Q[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// 64 x 64 output tile, dp4a over 64-byte K steps.
constexpr int TILE = 64, KSTEP = 64;
template <bool GATED>
__global__ void __launch_bounds__(256) int8_tile_kernel(const Int8Problem p) {
  __shared__ uint32_t sa[TILE][KSTEP / 4 + 1];
  __shared__ uint32_t sw[GATED ? 2 : 1][TILE][KSTEP / 4 + 1];
  const int64_t m0 = (int64_t)blockIdx.y * TILE;
  const int64_t n0 = (int64_t)blockIdx.x * TILE;
  const int64_t cols = GATED ? p.N / 2 : p.N;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[GATED ? 2 : 1][4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += KSTEP) {
    for (int i = threadIdx.x; i < TILE * (KSTEP / 4); i += 256) {
      const int r = i / (KSTEP / 4), c = i % (KSTEP / 4);
      const bool kin = k0 + 4 * c < p.K;
      sa[r][c] = kin && m0 + r < p.M
                     ? *reinterpret_cast<const uint32_t*>(p.A + (m0 + r) * p.lda + k0 + 4 * c)
                     : 0u;
      for (int h = 0; h < (GATED ? 2 : 1); ++h)
        sw[h][r][c] = kin && n0 + r < cols ? *reinterpret_cast<const uint32_t*>(
                                                 p.W + (h * cols + n0 + r) * p.K + k0 + 4 * c)
                                           : 0u;
    }
    __syncthreads();
    for (int c = 0; c < KSTEP / 4; ++c)
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[h][i][j] = __dp4a((int)sa[ty + 16 * i][c], (int)sw[h][tx + 16 * j][c], acc[h][i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= cols) continue;
      float v[2];
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const int64_t c = h * cols + n;
        v[h] = (float)acc[h][i][j] * (p.a_scale[m] * p.w_scale[c]);
        if (p.bias) v[h] += __uint_as_float((uint32_t)p.bias[c] << 16);
      }
      const float y = GATED ? v[0] / (1.f + expf(-v[0])) * v[1] : v[0];
      if (p.c_f32) {
        static_cast<float*>(p.C)[m * p.ldc + n] = y;
      } else {
        static_cast<__nv_bfloat16*>(p.C)[m * p.ldc + n] = __float2bfloat16_rn(y);
      }
    }
}

}  // namespace

qw_status launch_quantize_int8(const void* A, int64_t lda, int64_t rows, int32_t K, void* Q,
                               float* scale, bool f16, int32_t* err, cudaStream_t st) {
  const uint16_t* a = static_cast<const uint16_t*>(A);
  if (f16)
    return launch_pdl(quantize_int8_kernel<true>, dim3((unsigned)rows), dim3(QTHREADS), 0, st, a,
                      lda, K, Q, scale, err);
  return launch_pdl(quantize_int8_kernel<false>, dim3((unsigned)rows), dim3(QTHREADS), 0, st, a,
                    lda, K, Q, scale, err);
}

qw_status launch_widen_int8(const void* A, int64_t lda, int64_t M, int32_t K, void* Q,
                            cudaStream_t st) {
  const int64_t want = (M * (K / 16) + 255) / 256, cap = (int64_t)device_sm_count() * 8;
  return launch_pdl(widen_int8_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st,
                    static_cast<const int8_t*>(A), lda, M, K, static_cast<uint4*>(Q));
}

qw_status launch_gemv_int8(const Int8Problem& p, bool gated, int32_t* err, cudaStream_t st) {
  const int64_t cols = gated ? p.N / 2 : p.N;
  const dim3 grid((unsigned)((cols + TILE - 1) / TILE), (unsigned)((p.M + TILE - 1) / TILE));
  if (gated)
    int8_tile_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    int8_tile_kernel<false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace qw
