// gemm_int8_mma.cu - the INT8 product (and its gated form) for a few tokens, on mma.sync.
//
// Mathematics: C[m][n] = a_scale[m] w_scale[n] sum_k q[m][k] w[n][k] + bias[n].  Both sides' codes
// are exact in FP16; m16n8k16 MMAs add their products in FP32.  (With integer MMAs, which need no
// conversion, eight tokens more cost 8.5 us where these cost 2 at 14336 x 4096.)
//
// Bound: the weights' bytes, as long as the MMAs (weights as the 16-row operand, eight tokens a
// column group) hide under them.  Small blocks of rows keep every SM reading, where tcgen05's tiles
// of 128 rows leave a part of the SMs idle and each CTA a longer pipeline to fill: 14336 x 4096 with 16
// tokens 20.2 us there, 15.2 here; with 32 tokens 19.6 there, 38 here.
//
// A CTA of eight computing warps and one that copies has BR weight rows (gated: BR / 2 gate rows,
// then the up rows of the same outputs) and all of K, or a cluster's share of it.  Weights and tokens
// come in chunks of CK k into a ring, in TMA boxes of KB k.  (One bulk copy per row of a chunk
// instead: 28 us for 21.)  Of each chunk a warp multiplies 64 k of every row: a lane reads 16
// consecutive codes of a row at once, and as the order of k is free as long as both operands have the
// same, its j-th four codes are its operand of the j-th MMA.  The warps' sums meet in shared memory at
// the end, those of a cluster's CTAs in a second step; both are added in rank order.
// BR and the ring are such that three CTAs fit an SM: many small blocks even the SMs' loads out, and
// one's start and end hide under another's middle (64 rows and two CTAs 17.9 us, 32 rows and two CTAs
// 19.6, four CTAs with two stages 18.8, 16 rows 18.6).
#include <cuda_fp16.h>

#include "int8_map.cuh"
#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

constexpr int BR = 32, CK = 512, KB = 128, STAGES = 3, CTAS_PER_SM = 3;
constexpr int NUM_MMA_WARPS = CK / 64, NUM_THREADS = (NUM_MMA_WARPS + 1) * 32;
// words between two tokens' sums: the four tokens that a warp writes at a time fall into different
// banks
constexpr int SUM_PITCH = BR + 8;

template <int NT>
struct Geo {
  static constexpr int TOKENS = 8 * NT;
  static constexpr int STAGE_BYTES = (BR + TOKENS) * CK;
  static constexpr int SMEM = STAGES * STAGE_BYTES + 1024;
  static_assert(NUM_MMA_WARPS * TOKENS * SUM_PITCH * 4 <= SMEM - 1024, "the sums take the ring's place");
  static_assert(CTAS_PER_SM * (SMEM + 1024 + 128) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The row of a tile of eight that lane / 4 stands for: in this order the eight lanes that read at a
// time (two rows of the swizzled box) fall into different banks.  Column 2 j of a sum is then token
// j, column 2 j + 1 token j + 4.
__device__ __forceinline__ int mma_row(int lane) { return (lane >> 3) | (lane & 4); }

template <int NT, bool GATED>
__global__ void __launch_bounds__(NUM_THREADS, CTAS_PER_SM)
    gemm_int8_mma_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmW, const Int8Problem p,
                         const int32_t k_len, const int32_t csize, int32_t* err) {
  using GE = Geo<NT>;
  constexpr int OUTS = GATED ? BR / 2 : BR;  // outputs of a CTA
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[STAGES], empty[STAGES];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)csize);
  const int32_t cols = GATED ? p.N / 2 : p.N;
  const int32_t n0 = (int32_t)(blockIdx.x / (unsigned)csize) * OUTS;
  const int32_t k_beg = rank * k_len, k_end = min(p.K, k_beg + k_len);
  const int chunks = (k_end - k_beg + CK - 1) / CK;  // (k_len is a multiple of CK)
  const int M = (int)p.M;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NUM_MMA_WARPS);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();

  float acc[BR / 16][NT][4] = {};
  if (warp == NUM_MMA_WARPS) {
    // ------------------------------------------------------------ copies
    pdl_wait();
    int c = 0;
    for (; c < chunks; ++c) {
      const int s = c % STAGES, k0 = k_beg + c * CK;
      if (!warp_wait(&empty[s], (uint32_t)(c / STAGES + 1) & 1u, &abort_flag, err)) break;
      const int boxes = min(CK, k_end - k0 + KB - 1) / KB;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(boxes * KB * (BR + GE::TOKENS)));
      __syncwarp();
      uint8_t* dst = smem + s * GE::STAGE_BYTES;
      if (lane < boxes) {
        tma_load_2d(dst + lane * BR * KB, &tmW, &full[s], k0 + lane * KB, n0);
        if constexpr (GATED)
          tma_load_2d(dst + (lane * BR + OUTS) * KB, &tmW, &full[s], k0 + lane * KB, cols + n0);
        tma_load_2d(dst + BR * CK + lane * GE::TOKENS * KB, &tmA, &full[s], k0 + lane * KB, 0);
      }
    }
    if (c < chunks)
      for (int i = max(0, c - STAGES); i < c; ++i)
        wait_landed(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
  } else {
    // ------------------------------------------------------------ products
    // A ring's worth of the rows on its way to L2 while the previous kernel, most often this call's
    // own quantiser, still runs: 2 to 4 %.  (All of K: 18.2 us for 15.2.  The tensor maps are not used
    // before the wait: they lie in the launch's parameters, whose addresses later launches use again.)
    const int lines = min(k_end - k_beg, STAGES * CK) / KB;
    for (int i = threadIdx.x; i < BR * lines; i += NUM_MMA_WARPS * 32) {
      const int r = i / lines;
      const int32_t n = n0 + r % OUTS;
      if (n < cols)
        prefetch_l2(p.W + ((int64_t)(r / OUTS ? cols : 0) + n) * p.K + k_beg + (i - r * lines) * KB);
    }
    // The copies begin when the previous kernel has ended, and waits for them are limited: they must
    // not count that kernel's time.
    pdl_wait();
    const uint32_t row = mma_row(lane), chunk = (uint32_t)(warp & 1) * 4 + (lane & 3);
    const uint32_t off = row * KB + ((chunk ^ row) << 4);
    for (int c = 0; c < chunks; ++c) {
      const int s = c % STAGES;
      if (!warp_wait(&full[s], (uint32_t)(c / STAGES) & 1u, &abort_flag, err)) {
        wait_landed(&full[s], (uint32_t)(c / STAGES) & 1u);
        break;
      }
      // (boxes past the end of K are not copied)
      if (k_beg + c * CK + warp * 64 < k_end) {
        const uint8_t* w = smem + s * GE::STAGE_BYTES + (warp >> 1) * BR * KB + off;
        const uint8_t* x = smem + s * GE::STAGE_BYTES + BR * CK + (warp >> 1) * GE::TOKENS * KB + off;
        uint32_t b[NT][8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = *reinterpret_cast<const uint4*>(x + 8 * n * KB);
          int8x4_to_f16x2(v.x, b[n][0], b[n][1]);
          int8x4_to_f16x2(v.y, b[n][2], b[n][3]);
          int8x4_to_f16x2(v.z, b[n][4], b[n][5]);
          int8x4_to_f16x2(v.w, b[n][6], b[n][7]);
        }
#pragma unroll
        for (int i = 0; i < BR / 16; ++i) {
          const uint4 lo = *reinterpret_cast<const uint4*>(w + 16 * i * KB);
          const uint4 hi = *reinterpret_cast<const uint4*>(w + (16 * i + 8) * KB);
          const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            int8x4_to_f16x2(l[j], a0, a2);
            int8x4_to_f16x2(h[j], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16(acc[i][n], a0, a1, a2, a3, b[n][2 * j], b[n][2 * j + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
  }
  pdl_launch_dependents();
  __syncthreads();  // the ring has been read

  // sums of [warp][token][row], then of [token][row] where warp 0's were
  float* sums = reinterpret_cast<float*>(smem);
  if (warp < NUM_MMA_WARPS) {
    float* o = sums + (warp * GE::TOKENS + (lane & 3)) * SUM_PITCH + mma_row(lane);
#pragma unroll
    for (int i = 0; i < BR / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[(8 * n + (e & 1) * 4) * SUM_PITCH + 16 * i + (e >> 1) * 8] = acc[i][n][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < M * BR; i += NUM_THREADS) {
    float* o = sums + i / BR * SUM_PITCH + i % BR;
    float v = o[0];
#pragma unroll
    for (int w = 1; w < NUM_MMA_WARPS; ++w) v += o[w * GE::TOKENS * SUM_PITCH];
    o[0] = v;
  }
  if (csize > 1)
    cluster_sync();
  else
    __syncthreads();
  if (abort_flag == 0) {
    for (int i = rank * NUM_THREADS + threadIdx.x; i < M * OUTS; i += csize * NUM_THREADS) {
      const int m = i / OUTS;
      const int32_t n = n0 + i % OUTS;
      if (n >= cols) continue;
      const float sa = p.a_scale[m];
      float v[GATED ? 2 : 1];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const float* o = sums + m * SUM_PITCH + h * OUTS + i % OUTS;
        float sum = 0.f;
        if (csize > 1)
          for (int r = 0; r < csize; ++r)
            sum += ld_shared_cluster_f32(mapa_shared(smem_u32(o), (uint32_t)r));
        else
          sum = *o;
        const int64_t wr = (int64_t)(h ? cols : 0) + n;
        v[h] = sum * (sa * p.w_scale[wr]);
        if (p.bias) v[h] += __uint_as_float((uint32_t)p.bias[wr] << 16);
      }
      const float y = GATED ? gate_up(v[0], v[GATED ? 1 : 0]) : v[0];
      if (p.c_f32)
        static_cast<float*>(p.C)[m * p.ldc + n] = y;
      else
        static_cast<__nv_bfloat16*>(p.C)[m * p.ldc + n] = __float2bfloat16_rn(y);
    }
  }
  if (csize > 1) cluster_sync();  // nobody leaves while its sums are read
}

template <int NT, bool GATED>
qw_status launch(const Int8Problem& p, int32_t* err, cudaStream_t st) {
  using GE = Geo<NT>;
  constexpr int OUTS = GATED ? BR / 2 : BR;
  const int32_t cols = GATED ? p.N / 2 : p.N;
  const int64_t blocks = ((int64_t)cols + OUTS - 1) / OUTS;
  // Few blocks share K out over clusters while each CTA keeps a chunk of it; with a little more than one
  // block per SM that evens the SMs' loads out, and pays where much K is left (us without and with:
  // 16 x 5120 x 8192 17.0, 15.6; 16 x 6144 x 16384 28.9, 24.1; but 16 x 6144 x 2048 7.1, 7.6 and
  // 16 x 7168 x 8192 17.5, 17.7).
  const int sms = device_sm_count();
  auto split = [&](int c) {
    return p.K / (2 * c) >= CK &&
           (blocks * c <= sms || (10 * blocks * c <= 13 * sms && p.K / (2 * c) >= 5 * CK));
  };
  int csize = 1;
  while (csize < 8 && split(csize)) csize *= 2;
  const int32_t k_len = ((p.K + csize - 1) / csize + CK - 1) / CK * CK;
  csize = (p.K + k_len - 1) / k_len;
  CUtensorMap tmA, tmW;
  if (!encode_int8_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.A, p.K, p.M, p.lda, KB, GE::TOKENS) ||
      !encode_int8_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.W, p.K, p.N, p.K, KB, OUTS))
    return QW_ERR_CUDA;
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [] {
        return cudaFuncSetAttribute(gemm_int8_mma_kernel<NT, GATED>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    GE::SMEM) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * csize));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = GE::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_int8_mma_kernel<NT, GATED>, tmA, tmW, p, k_len, csize, err) ==
                 cudaSuccess
             ? QW_OK
             : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_gemm_int8_mma(const Int8Problem& p, bool gated, int32_t* err,
                               cudaStream_t st) {
  if (p.M <= 8)
    return gated ? launch<1, true>(p, err, st) : launch<1, false>(p, err, st);
  return gated ? launch<2, true>(p, err, st) : launch<2, false>(p, err, st);
}

}  // namespace qw
