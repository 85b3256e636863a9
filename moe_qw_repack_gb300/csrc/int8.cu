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

// x rounded to an integer (ties to even), |x| < 2^22: adding 1.5 * 2^23 rounds at the units.
// The sum's low bits are the integer in two's complement.
constexpr float kRound = 12582912.f;

// Row r of A -> codes (INT8, or the same integers as FP16 for the tensor cores) and the row's
// scale.  One CTA per row.  A thread keeps VEC 16-byte vectors of the row (K <= 2048 VEC) in
// registers, so the row is read once; what lies beyond is read a second time.
constexpr int QTHREADS = 256;
template <bool F16, int VEC>
__global__ void __launch_bounds__(QTHREADS)
    quantize_int8_kernel(const uint16_t* __restrict__ A, int64_t lda, int32_t K,
                         void* __restrict__ Q, float* __restrict__ S, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(A + r * lda);
  const int n8 = K / 8;
  uint4 keep[VEC];
  uint32_t amax = 0;  // largest |v| as BF16 bits (finite values order like their bit patterns)
  auto fold = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  };
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    keep[j] = i < n8 ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) fold(keep[j]);
  for (int i = threadIdx.x + VEC * QTHREADS; i < n8; i += QTHREADS) fold(__ldg(src + i));
  __shared__ uint32_t part[QTHREADS / 32];
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = part[0];
#pragma unroll
  for (int i = 1; i < QTHREADS / 32; ++i) amax = max(amax, part[i]);
  const float top = __uint_as_float(amax << 16);
  const bool finite = amax < 0x7F80u;
  const float inv = fminf(127.0f / top, 3.4028234663852886e38f);
  if (threadIdx.x == 0) {
    S[r] = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
    if (!finite) set_error(err, QW_ERR_VALUE);
  }
  auto put = [&](int i, uint4 v) {
    if (!finite) v = make_uint4(0, 0, 0, 0);  // codes 0 (0 * inv is 0: inv is finite there too)
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // the product is rounded to FP32 before the code is (no fused multiply-add)
      q[2 * j] = __fadd_rn(__fmul_rn(bf16_lo(w[j]), inv), kRound);
      q[2 * j + 1] = __fadd_rn(__fmul_rn(bf16_hi(w[j]), inv), kRound);
    }
    if constexpr (F16) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(q[2 * j] - kRound, q[2 * j + 1] - kRound);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      reinterpret_cast<uint4*>(Q)[r * (K / 8) + i] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      uint32_t o[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t lo = __byte_perm(__float_as_uint(q[4 * j]), __float_as_uint(q[4 * j + 1]), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(q[4 * j + 2]), __float_as_uint(q[4 * j + 3]), 0x0040);
        o[j] = __byte_perm(lo, hi, 0x5410);
      }
      reinterpret_cast<uint2*>(Q)[r * (K / 8) + i] = make_uint2(o[0], o[1]);
    }
  };
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    if (i < n8) put(i, keep[j]);
  }
  for (int i = threadIdx.x + VEC * QTHREADS; i < n8; i += QTHREADS) put(i, __ldg(src + i));
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

// ------------------------------------------------------------------ up to 16 tokens
// The weights are streamed once; integer sums are exact, so any order gives the same result.
// A CTA of four warps takes RB blocks of 16 weight rows (gated: 16 gate rows and the 16 up rows
// of the same outputs) and a slice of K; its warps take 64 x U bytes of every row in turn.  A lane
// of mma.m16n8k32 (s8) owns rows g and g + 8 and, as k may be permuted if both operands agree,
// 16 consecutive bytes of each per two MMAs: weights and tokens come in 16-byte loads in
// fragment order, with nothing staged.  Partial sums meet in shared memory, those of a K split
// over a cluster's CTAs in rank 0's.
constexpr int GW = 4, GTHREADS = GW * 32;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldg_stream(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NT, int RB, bool GATED>
__global__ void __launch_bounds__(GTHREADS, 8)
    gemv_int8_kernel(const Int8Problem p, const int csize, const bool early) {
  static_assert(!GATED || RB == 2, "a gate block and its up block");
  constexpr int U = 4 / RB / NT;              // steps of 64 k loaded at a time
  constexpr int ROWS = GATED ? 16 : 16 * RB;  // outputs of a CTA
  __shared__ int part[GW][RB][NT][128];
  __shared__ int total[RB][NT][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = csize > 1 ? (int)(blockIdx.x % csize) : 0;
  const int32_t cols = GATED ? p.N / 2 : p.N;
  const int32_t n0 = (int32_t)(blockIdx.x / csize) * ROWS;

  // this CTA's 64-k steps, and this lane's first byte of each of its rows
  const int steps = (p.K + 63) / 64, per = (steps + csize - 1) / csize;
  const int sbeg = min(steps, rank * per), send = min(steps, sbeg + per);
  const int8_t* wp[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // rows past the last are read as the last and not stored
      const int32_t n = min(n0 + (GATED ? 0 : 16 * b) + g + 8 * h, cols - 1);
      wp[b][h] = p.W + ((int64_t)(GATED && b ? cols : 0) + n) * p.K + 16 * t;
    }
  const int8_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xp[i] = p.A + (int64_t)min((int64_t)(8 * i + g), p.M - 1) * p.lda + 16 * t;

  int acc[RB][NT][4] = {};
  uint4 w[U][RB][2], x[U][NT];
  auto load_w = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = (s0 + u) * 64;
          w[u][b][h] = s0 + u < send && k + 16 * t < p.K ? ldg_stream(wp[b][h] + k)
                                                         : make_uint4(0, 0, 0, 0);
        }
  };
  // `early`: the previous kernel on the stream is this call's own quantiser, which waited for
  // everything before it; the weights may be read while it runs
  if (early) load_w(sbeg + warp * U);
  pdl_wait();
  pdl_launch_dependents();
  if (!early) load_w(sbeg + warp * U);
  for (int s0 = sbeg + warp * U; s0 < send; s0 += GW * U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int k = (s0 + u) * 64;
        x[u][i] = s0 + u < send && k + 16 * t < p.K && 8 * i + g < p.M
                      ? __ldg(reinterpret_cast<const uint4*>(xp[i] + k))
                      : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma_s8(acc[b][i], w[u][b][0].x, w[u][b][1].x, w[u][b][0].y, w[u][b][1].y, x[u][i].x,
                 x[u][i].y);
          mma_s8(acc[b][i], w[u][b][0].z, w[u][b][1].z, w[u][b][0].w, w[u][b][1].w, x[u][i].z,
                 x[u][i].w);
        }
    load_w(s0 + GW * U);
  }

  // element (row r, token c) of an accumulator at 16 c + r
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[warp][b][i][16 * (2 * t + (e & 1)) + g + 8 * (e >> 1)] = acc[b][i][e];
  __syncthreads();
  int sum[RB][NT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      sum[b][i] = 0;
#pragma unroll
      for (int v = 0; v < GW; ++v) sum[b][i] += part[v][b][i][threadIdx.x];
    }
  if (csize > 1) {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int i = 0; i < NT; ++i) total[b][i][threadIdx.x] = sum[b][i];
    cluster_sync();
    if (rank == 0)
      for (int c = 1; c < csize; ++c)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            sum[b][i] += __float_as_int(ld_shared_cluster_f32(
                mapa_shared(smem_u32(&total[b][i][threadIdx.x]), (uint32_t)c)));
    cluster_sync();
    if (rank != 0) return;
  }
  const int r = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t m = 8 * i + (threadIdx.x >> 4);
    if (m >= p.M) continue;
    const float sa = p.a_scale[m];
    float v[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int32_t n = n0 + (GATED ? 0 : 16 * b) + r;
      if (n >= cols) continue;
      const int64_t wr = (GATED && b ? cols : 0) + (int64_t)n;
      v[b] = (float)sum[b][i] * (sa * __ldg(p.w_scale + wr));
      if (p.bias) v[b] += __uint_as_float((uint32_t)__ldg(p.bias + wr) << 16);
      if constexpr (!GATED) {
        if (p.c_f32)
          static_cast<float*>(p.C)[m * p.ldc + n] = v[b];
        else
          static_cast<__nv_bfloat16*>(p.C)[m * p.ldc + n] = __float2bfloat16_rn(v[b]);
      }
    }
    if constexpr (GATED)
      if (n0 + r < cols)
        static_cast<__nv_bfloat16*>(p.C)[m * p.ldc + n0 + r] =
            __float2bfloat16_rn(v[0] / (1.f + expf(-v[0])) * v[1]);
  }
}

template <int NT, int RB, bool GATED>
qw_status launch_gemv(const Int8Problem& p, bool early, cudaStream_t st) {
  const int32_t cols = GATED ? p.N / 2 : p.N, rows = GATED ? 16 : 16 * RB;
  const int64_t blocks = ((int64_t)cols + rows - 1) / rows;
  int csize = 1;
  while (csize < 8 && blocks * csize < 4 * device_sm_count() && p.K / csize >= 2048) csize *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * csize));
  cfg.blockDim = dim3(GTHREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemv_int8_kernel<NT, RB, GATED>, p, csize, early) == cudaSuccess
             ? QW_OK
             : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_quantize_int8(const void* A, int64_t lda, int64_t rows, int32_t K, void* Q,
                               float* scale, bool f16, int32_t* err, cudaStream_t st) {
  const uint16_t* a = static_cast<const uint16_t*>(A);
  const bool wide = K > 2 * 8 * QTHREADS;
  auto* kern = f16 ? (wide ? quantize_int8_kernel<true, 8> : quantize_int8_kernel<true, 2>)
                   : (wide ? quantize_int8_kernel<false, 8> : quantize_int8_kernel<false, 2>);
  return launch_pdl(kern, dim3((unsigned)rows), dim3(QTHREADS), 0, st, a, lda, K, Q, scale, err);
}

qw_status launch_widen_int8(const void* A, int64_t lda, int64_t M, int32_t K, void* Q,
                            cudaStream_t st) {
  const int64_t want = (M * (K / 16) + 255) / 256, cap = (int64_t)device_sm_count() * 8;
  return launch_pdl(widen_int8_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st,
                    static_cast<const int8_t*>(A), lda, M, K, static_cast<uint4*>(Q));
}

qw_status launch_gemv_int8(const Int8Problem& p, bool gated, bool early, cudaStream_t st) {
  if (gated)
    return p.M <= 8 ? launch_gemv<1, 2, true>(p, early, st) : launch_gemv<2, 2, true>(p, early, st);
  return p.M <= 8 ? launch_gemv<1, 1, false>(p, early, st) : launch_gemv<2, 2, false>(p, early, st);
}

}  // namespace qw
