// int8.cu - the INT8 product with a scale per token and per output channel, its gated form,
// and the per-token quantiser in front of them.
//
//   q[m][k] = rint(a[m][k] * (127 / amax_m)),  sa_m = amax_m / 127
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

// largest |v| of eight BF16 values as BF16 bits (finite values order like their bit patterns)
__device__ __forceinline__ uint32_t bf16x8_absmax(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  return m;
}

// A row's scale and codes from its largest magnitude (BF16 bits).  A row with a non-finite value has
// the scale NaN and codes 0.  Below 2^-121 the quotient 127 / amax may pass FP32's range: such a row is
// multiplied by 2^64 first, which is exact.  A row without a normal number has codes 0: its scale would
// keep too few bits.
struct RowScale {
  // adding 1.5 * 2^23 rounds |x| < 2^22 to an integer (ties to even), which the sum's low bits hold
  // in two's complement
  static constexpr float kRound = 12582912.f;
  bool finite;
  float scale, up, inv;
  __device__ __forceinline__ explicit RowScale(uint32_t amax) {
    const float top = __uint_as_float(amax << 16);
    finite = amax < 0x7F80u;
    scale = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
    up = amax < 0x0300u ? 0x1p64f : 1.f;  // (0x0300: 2^-121)
    inv = amax < 0x0080u ? 0.f : 127.0f / (top * up);
  }
  // eight values' codes plus kRound; the product is rounded to FP32 before the code is (no fused
  // multiply-add)
  __device__ __forceinline__ void rounded(const uint4& v, float (&q)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[2 * j] = finite ? __fadd_rn(__fmul_rn(bf16_lo(w[j]) * up, inv), kRound) : kRound;
      q[2 * j + 1] = finite ? __fadd_rn(__fmul_rn(bf16_hi(w[j]) * up, inv), kRound) : kRound;
    }
  }
  __device__ __forceinline__ uint2 codes(const uint4& v) const {
    float q[8];
    rounded(v, q);
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = __byte_perm(__float_as_uint(q[4 * j]), __float_as_uint(q[4 * j + 1]), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(q[4 * j + 2]), __float_as_uint(q[4 * j + 3]), 0x0040);
      o[j] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(o[0], o[1]);
  }
  __device__ __forceinline__ uint4 codes16(const uint4& v) const {  // as FP16 numbers
    float q[8];
    rounded(v, q);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(q[2 * j] - kRound, q[2 * j + 1] - kRound);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// Row r of A -> codes (INT8, or the same integers as FP16 for the tensor cores) and the row's
// scale.  One CTA per row.  A thread keeps VEC 16-byte vectors of the row (K <= 2048 VEC) in
// registers, so the row is read once; what lies beyond is read a second time.
constexpr int QTHREADS = 256;
template <bool F16, int VEC>
__global__ void __launch_bounds__(QTHREADS)
    quantize_int8_kernel(const uint16_t* A, int64_t lda, int32_t K,
                         void* __restrict__ Q, float* __restrict__ S, int32_t* err) {
  // FP16 codes are only written in front of the tensor-core kernel, which reads nothing before its own
  // wait and lets the next kernel start only after it: it may be set up while this one still waits
  // (333 x 1000 x 1040 9.2 -> 8.7 us).  The other kernels' CTAs would only take the place of the
  // previous call's.
  if (F16) pdl_launch_dependents();
  pdl_wait();
  if (!F16) pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(A + r * lda);
  const int n8 = K / 8;
  uint4 keep[VEC];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    keep[j] = i < n8 ? src[i] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) amax = max(amax, bf16x8_absmax(keep[j]));
  for (int i = threadIdx.x + VEC * QTHREADS; i < n8; i += QTHREADS)
    amax = max(amax, bf16x8_absmax(src[i]));
  __shared__ uint32_t part[QTHREADS / 32];
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = part[0];
#pragma unroll
  for (int i = 1; i < QTHREADS / 32; ++i) amax = max(amax, part[i]);
  const RowScale rs(amax);
  if (threadIdx.x == 0) {
    S[r] = rs.scale;
    if (!rs.finite) set_error(err, QW_ERR_VALUE);
  }
  auto put = [&](int i, const uint4& v) {
    if constexpr (F16)
      reinterpret_cast<uint4*>(Q)[r * (K / 8) + i] = rs.codes16(v);
    else
      reinterpret_cast<uint2*>(Q)[r * (K / 8) + i] = rs.codes(v);
  };
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = threadIdx.x + j * QTHREADS;
    if (i < n8) put(i, keep[j]);
  }
  for (int i = threadIdx.x + VEC * QTHREADS; i < n8; i += QTHREADS) put(i, src[i]);
}

// INT8 codes [M][lda] -> the same integers as FP16 [M][K]; a thread takes eight times eight codes at a
// time, so that what a warp stores is contiguous.  I: 32 bits wherever they reach (16 codes a thread
// and a 64-bit division for them took 12.6 us for 4096 x 4096, 8.5 now).
template <typename I>
__global__ void __launch_bounds__(256)
    widen_int8_kernel(const int8_t* A, int64_t lda, I total, I per_row,
                      uint4* __restrict__ Q) {
  pdl_launch_dependents();  // (as the quantiser above)
  pdl_wait();
  constexpr int U = 8;
  const I step = (I)gridDim.x * 256;
  for (I i = (I)blockIdx.x * 256 + threadIdx.x; i < total; i += U * step) {
    uint2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const I at = i + u * step, r = at / per_row;
      v[u] = at < total ? reinterpret_cast<const uint2*>(A + (int64_t)r * lda)[at - r * per_row]
                        : make_uint2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const I at = i + u * step;
      if (at >= total) break;
      uint4 o;
      int8x4_to_f16x2(v[u].x, o.x, o.y);
      int8x4_to_f16x2(v[u].y, o.z, o.w);
      Q[at] = o;
    }
  }
}

// ------------------------------------------------------------------ one or two tokens
// The weights are streamed once; integer sums are exact, so any order gives the same result.
// A CTA of two warps takes R = 2 RW weight rows (gated: gate rows and the up rows of the same
// outputs) and slices of at most SLICE of their k, the next on its way while one is multiplied.  Its
// rows arrive in shared memory by bulk copies that one warp issues before anything else, so that all
// of a CTA's bytes are in flight at once, however few its threads; a lane then multiplies 16
// consecutive k of RW rows with the same k of every token (dp4a), and one warp reduction per row and
// token ends the work.  Where there are few rows, the CTAs of a cluster share a block's slices and
// their sums meet in its rank 0.
// (Quantising BF16 tokens in here instead of a kernel in front of it loses the weights' head start
// under that kernel: 1 x 14336 x 4096 12.3 for 12.8 us, but gated 22.9 for 21.9, two tokens 14.6 for
// 13.6 and 1 x 4096 x 4096 4.5 for 3.9.)
constexpr int GW = 2, GTHREADS = GW * 32, SLICE = 4096;

struct GemvShape {
  int32_t len;     // k of a slice (a multiple of 16)
  int32_t slices;
  int32_t csize;   // CTAs that share a block of rows
};

template <int MT, int RW, bool GATED>
__global__ void __launch_bounds__(GTHREADS)
    gemv_int8_kernel(const Int8Problem p, const GemvShape g, const bool early, int32_t* err) {
  constexpr int R = GW * RW;                     // weight rows of a CTA
  constexpr int OUTS = GATED ? R / 2 : R;        // outputs of a CTA
  static_assert(!GATED || RW % 2 == 0, "a warp has its gate rows' up rows");
  extern __shared__ __align__(128) uint8_t smem[];  // [2 or 1][R][pitch] weights
  __shared__ uint64_t full[2];
  __shared__ int abort_flag;
  __shared__ int part[R * MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = g.csize > 1 ? (int)(blockIdx.x % (unsigned)g.csize) : 0;
  const int32_t cols = GATED ? p.N / 2 : p.N;
  const int32_t n0 = (int32_t)(blockIdx.x / (unsigned)g.csize) * OUTS;
  const int pitch = (g.len + 511) / 512 * 512;

  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  // Row i of the CTA: warp i / RW's row i % RW; gated: outputs n0 + (i / RW) RW / 2 + .., the gate
  // rows in the first half of a warp's rows.  -1: no such row.
  auto row_of = [&](int i) -> int64_t {
    const int w = i / RW, r = i % RW;
    const int32_t n = GATED ? n0 + w * (RW / 2) + r % (RW / 2) : n0 + i;
    if (n >= cols) return -1;
    return (GATED && r >= RW / 2) ? (int64_t)cols + n : n;
  };
  auto fetch = [&](int s, int buffer) {  // warp 0
    if (s >= g.slices) return;
    const int k0 = s * g.len, len = min(g.len, p.K - k0);
    const int64_t row = lane < R ? row_of(lane) : -1;
    const int rows = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0));
    if (lane == 0) mbar_arrive_expect_tx(&full[buffer], (uint32_t)(rows * len));
    __syncwarp();
    if (row >= 0)
      bulk_load(smem + (buffer * R + lane) * pitch, p.W + row * p.K + k0, (uint32_t)len,
                &full[buffer]);
  };
  // `early`: the previous kernel on the stream is this call's own quantiser, which waited for
  // everything before it; the weights may be read while it runs
  if (early && warp == 0) fetch(rank, 0);
  pdl_wait();
  pdl_launch_dependents();
  if (!early && warp == 0) fetch(rank, 0);

  int acc[RW][MT] = {};
  int buffer = 0;
  uint32_t phase = 0;
  for (int s = rank; s < g.slices; s += g.csize) {
    const int k0 = s * g.len, len = min(g.len, p.K - k0);
    if (s != rank) __syncthreads();  // the slice before, whose buffer the next one takes, is done
    if (warp == 0) fetch(s + g.csize, buffer ^ 1);
    // a lane's k of every token, for all of its warp's rows; zeros past the slice and the tokens
    constexpr int XREG = SLICE / 512;
    uint4 x[XREG][MT];
#pragma unroll
    for (int j = 0; j < XREG; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int k = j * 512 + lane * 16;
        x[j][m] = k < len && m < p.M
                      ? *reinterpret_cast<const uint4*>(p.A + m * p.lda + k0 + k)
                      : make_uint4(0, 0, 0, 0);
      }
    if (!warp_wait(&full[buffer], phase, &abort_flag, err)) wait_landed(&full[buffer], phase);
    const uint8_t* wrow = smem + (buffer * R + warp * RW) * pitch + lane * 16;
#pragma unroll
    for (int j = 0; j < XREG; ++j) {
      if (j * 512 >= len) break;
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        // (rows that do not exist, and k past the slice, hold anything: their products are
        // not stored, or are with zeros)
        const uint4 w = *reinterpret_cast<const uint4*>(wrow + r * pitch + j * 512);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[r][m] = __dp4a((int)w.x, (int)x[j][m].x, acc[r][m]);
          acc[r][m] = __dp4a((int)w.y, (int)x[j][m].y, acc[r][m]);
          acc[r][m] = __dp4a((int)w.z, (int)x[j][m].z, acc[r][m]);
          acc[r][m] = __dp4a((int)w.w, (int)x[j][m].w, acc[r][m]);
        }
      }
    }
    phase ^= (uint32_t)buffer;  // a buffer's phase turns every second slice
    buffer ^= 1;
  }

  // sum (row i, token m) of the slices this CTA had at i MT + m
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int v = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
      if (lane == 0) part[(warp * RW + r) * MT + m] = v;
    }
  if (g.csize > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank == 0) {
    for (int i = threadIdx.x; i < OUTS * MT; i += GTHREADS) {
      const int o = i / MT, m = i % MT;  // output n0 + o
      const int32_t n = n0 + o;
      if (n >= cols || m >= p.M) continue;
      float v[GATED ? 2 : 1];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const int row = GATED ? o / (RW / 2) * RW + o % (RW / 2) + h * (RW / 2) : o;
        int sum = part[row * MT + m];
        for (int c = 1; c < g.csize; ++c)
          sum += __float_as_int(
              ld_shared_cluster_f32(mapa_shared(smem_u32(&part[row * MT + m]), (uint32_t)c)));
        const int64_t wr = (int64_t)(h ? cols : 0) + n;
        v[h] = (float)sum * (p.a_scale[m] * p.w_scale[wr]);
        if (p.bias) v[h] += __uint_as_float((uint32_t)p.bias[wr] << 16);
      }
      const float y = GATED ? gate_up(v[0], v[GATED ? 1 : 0]) : v[0];
      if (p.c_f32)
        static_cast<float*>(p.C)[m * p.ldc + n] = y;
      else
        static_cast<__nv_bfloat16*>(p.C)[m * p.ldc + n] = __float2bfloat16_rn(y);
    }
  }
  if (g.csize > 1) cluster_sync();  // nobody leaves while its sums are read
}

template <int MT, int RW, bool GATED>
qw_status launch_gemv(const Int8Problem& p, bool early, int32_t* err, cudaStream_t st) {
  constexpr int R = GW * RW, OUTS = GATED ? R / 2 : R;
  const int32_t cols = GATED ? p.N / 2 : p.N;
  const int64_t blocks = ((int64_t)cols + OUTS - 1) / OUTS;
  // Slices of at most SLICE.  Few blocks share them out over clusters, shorter ones if need be, while
  // each keeps 1024.  (A cluster costs more than it gives where there are blocks enough:
  // 1 x 4096 x 14336 15.8 us with clusters of four, 12.0 without.)
  const int sms = device_sm_count();
  int slices = (p.K + SLICE - 1) / SLICE, csize = 1;
  while (csize < 8 && blocks * csize < 4 * sms && p.K / (2 * csize) >= 1024) csize *= 2;
  if (slices < csize) slices = csize;
  GemvShape g;
  g.len = ((p.K + slices - 1) / slices + 15) / 16 * 16;
  g.slices = (p.K + g.len - 1) / g.len;
  g.csize = g.slices < csize ? g.slices : csize;
  const int buffers = g.slices > g.csize ? 2 : 1;
  const int pitch = (g.len + 511) / 512 * 512;
  constexpr int kMaxSmem = 2 * R * SLICE;
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [] {
        return cudaFuncSetAttribute(gemv_int8_kernel<MT, RW, GATED>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMaxSmem) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * g.csize));
  cfg.blockDim = dim3(GTHREADS);
  cfg.dynamicSmemBytes = (size_t)buffers * R * pitch;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)g.csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = g.csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemv_int8_kernel<MT, RW, GATED>, p, g, early, err) == cudaSuccess
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
  const int64_t total = M * (K / 8), want = (total + 255) / 256, cap = (int64_t)device_sm_count() * 8;
  const dim3 grid((unsigned)(want < cap ? want : cap));
  const int8_t* a = static_cast<const int8_t*>(A);
  uint4* q = static_cast<uint4*>(Q);
  if (total < (int64_t)1 << 31)  // (what is added to it below is less than 2^31)
    return launch_pdl(widen_int8_kernel<uint32_t>, grid, dim3(256), 0, st, a, lda, (uint32_t)total,
                      (uint32_t)(K / 8), q);
  return launch_pdl(widen_int8_kernel<int64_t>, grid, dim3(256), 0, st, a, lda, total,
                    (int64_t)(K / 8), q);
}

qw_status launch_gemv_int8(const Int8Problem& p, bool gated, bool early, int32_t* err,
                           cudaStream_t st) {
  if (gated)
    return p.M == 1 ? launch_gemv<1, 2, true>(p, early, err, st)
                    : launch_gemv<2, 2, true>(p, early, err, st);
  return p.M == 1 ? launch_gemv<1, 2, false>(p, early, err, st)
                  : launch_gemv<2, 2, false>(p, early, err, st);
}

}  // namespace qw
