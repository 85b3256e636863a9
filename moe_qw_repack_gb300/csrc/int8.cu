// int8.cu - the INT8 product with a scale per token and per output channel, its gated form,
// and the per-token quantiser in front of them.
//
//   q[m][k] = rint(a[m][k] * min(127 / amax_m, FLT_MAX)),  sa_m = amax_m / 127
//   C[m][n] = sa_m * sw_n * sum_k q[m][k] w[n][k] + bias[n]
//   Y[m][i] = silu(C[m][i]) * C[m][I + i]                               (gated)
#include <cuda_bf16.h>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Row r of A -> INT8 codes and the row's scale; one CTA per row, the row read twice.
__global__ void __launch_bounds__(256)
    quantize_int8_kernel(const uint16_t* __restrict__ A, int64_t lda, int32_t K,
                         int8_t* __restrict__ Q, float* __restrict__ S, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(A + r * lda);
  const int n8 = K / 8;
  uint32_t amax = 0;
  for (int i = threadIdx.x; i < n8; i += blockDim.x) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  }
  __shared__ uint32_t part[8];
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0;
  for (int i = 0; i < 8; ++i) amax = max(amax, part[i]);
  const float top = __uint_as_float(amax << 16);
  const bool finite = amax < 0x7F80u;
  const float inv = fminf(127.0f / top, 3.4028234663852886e38f);
  if (threadIdx.x == 0) {
    S[r] = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
    if (!finite) set_error(err, QW_ERR_VALUE);
  }
  for (int i = threadIdx.x; i < n8; i += blockDim.x) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
      const int q = finite ? __float2int_rn(x * inv) : 0;
      o[j >> 2] |= ((uint32_t)q & 0xFFu) << (8 * (j & 3));
    }
    reinterpret_cast<uint2*>(Q + r * K)[i] = make_uint2(o[0], o[1]);
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
                               float* scale, int32_t* err, cudaStream_t st) {
  return launch_pdl(quantize_int8_kernel, dim3((unsigned)rows), dim3(256), 0, st,
                    static_cast<const uint16_t*>(A), lda, K, static_cast<int8_t*>(Q), scale, err);
}

qw_status launch_gemm_int8(const Int8Problem& p, bool gated, int32_t* err, cudaStream_t st) {
  const int64_t cols = gated ? p.N / 2 : p.N;
  const dim3 grid((unsigned)((cols + TILE - 1) / TILE), (unsigned)((p.M + TILE - 1) / TILE));
  if (gated)
    int8_tile_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    int8_tile_kernel<false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace qw
