// gemm_int8_tc.cu - the INT8 product (and its gated form) for more than a few tokens, on the
// tcgen05 tensor cores.
//
// Mathematics: C[m][n] = a_scale[m] w_scale[n] sum_k q[m][k] w[n][k] + bias[n].  Every INT8 code
// is an FP16 number and every product of two an FP32 integer, so kind::f16 MMAs with FP32
// accumulation give the integer sum exactly while partial sums stay below 2^24 (sm_103a's own
// integer tensor rate is far below its 16-bit one).
//
// Structure (persistent, one CTA per SM; a tile is 128 weight rows x BT tokens):
//   warp 0      TMA producer of the tokens' tile: FP16 codes [M][K] of the workspace, 64 k
//               (128-byte swizzle) a stage;
//   warp 2      TMA producer of the weights: INT8, 128 rows x 128 k a stage;
//   warp 1      TMEM owner and MMA issuer: weights are the A operand, read from tensor memory,
//               tokens the B operand, read from shared memory;
//   warps 4-11  converters: warp w covers TMEM lanes 32 (w % 4) .. + 31 and one 64-k half of a
//               weight stage; a lane takes 64 codes of its own row, makes them FP16 (byte b ->
//               the FP16 number 1024 + (b + 128), minus 1152: exact) and stores them as the
//               MMA's A operand with one tcgen05.st;
//   warps 12-19 epilogue: tcgen05.ld the accumulator (a lane holds one weight row, a register
//               one token), scale, add bias, (gated) exchange gate and up, round and store.
// The gated form gives each 32 TMEM lanes 16 gate rows and the 16 up rows of the same outputs,
// so that a gate and its up value meet through one shuffle.
// Every wait is bounded; on expiry the kernel reports QW_ERR_TIMEOUT and shuts down.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

constexpr int BW = 128;              // weight rows per tile (MMA M)
constexpr int KA = 64;               // k of a token stage and of a TMEM operand slot
constexpr int KW = 128;              // k of a weight stage
constexpr int W_BYTES = BW * KW;
constexpr int CVT_WARP0 = 4, NUM_CVT_WARPS = 8;
constexpr int EPI_WARP0 = CVT_WARP0 + NUM_CVT_WARPS, NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = (EPI_WARP0 + NUM_EPI_WARPS) * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr int A_SLOT_COLS = KA / 2;  // 32-bit columns of one operand slot

template <int BT>
struct Geo {
  static constexpr int B_BYTES = BT * KA * 2;
  static constexpr int B_STAGES = BT == 256 ? 5 : 8;
  static constexpr int W_STAGES = BT == 256 ? 3 : 5;
  static constexpr int A_SLOTS = 8;
  static constexpr int A_COL0 = 256;
  static constexpr size_t SMEM = (size_t)B_STAGES * B_BYTES + W_STAGES * W_BYTES +
                                 NUM_EPI_WARPS * (BT / 2) * 4 + 512 + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  // kind::f16: FP32 accumulator (bit 4), A = B = FP16 (0), both K-major, N >> 3 at bit 17,
  // M >> 4 at bit 24
  static constexpr uint32_t IDESC =
      (1u << 4) | ((uint32_t)(BT >> 3) << 17) | ((uint32_t)(BW >> 4) << 24);
};

struct Params {
  int64_t M;
  int32_t cols;       // output columns: N, or I of the gated form
  int32_t K;
  int32_t num_n_tiles, num_m_tiles;
  const float* a_scale;
  const float* w_scale;
  const uint16_t* bias;
  void* C;
  int64_t ldc;
  int32_t c_f32;
  int32_t* err;
};

__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
}

template <int BT, bool GATED>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_int8_tc_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmW, const Params p) {
  using GE = Geo<BT>;
  constexpr int B_STAGES = GE::B_STAGES, W_STAGES = GE::W_STAGES, A_SLOTS = GE::A_SLOTS;
  constexpr int TILE_COLS = GATED ? BW / 2 : BW;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sB = smem;
  uint8_t* sW = sB + B_STAGES * GE::B_BYTES;
  float* sScale = reinterpret_cast<float*>(sW + W_STAGES * W_BYTES);  // [8 warps][BT/2]
  uint64_t* b_full = reinterpret_cast<uint64_t*>(sScale + NUM_EPI_WARPS * (BT / 2));
  uint64_t* b_empty = b_full + B_STAGES;
  uint64_t* w_full = b_empty + B_STAGES;
  uint64_t* w_empty = w_full + W_STAGES;
  uint64_t* a_full = w_empty + W_STAGES;
  uint64_t* a_empty = a_full + A_SLOTS;
  uint64_t* acc_full = a_empty + A_SLOTS;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* final_bar = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(final_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < B_STAGES; ++s) {
      mbar_init(&b_full[s], 1);
      mbar_init(&b_empty[s], 1);
    }
    for (int s = 0; s < W_STAGES; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], NUM_CVT_WARPS);
    }
    for (int s = 0; s < A_SLOTS; ++s) {
      mbar_init(&a_full[s], NUM_CVT_WARPS / 2);
      mbar_init(&a_empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, NUM_EPI_WARPS);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // set-up above overlaps the previous kernel's tail; every global access comes after this
  pdl_wait();

  const int64_t num_tiles = (int64_t)p.num_m_tiles * p.num_n_tiles;
  const int KB = (p.K + KA - 1) / KA;  // token stages and operand slots per tile
  const int KWB = (p.K + KW - 1) / KW;

  if (warp == 0) {
    // ------------------------------------------------------------ tokens
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const int32_t m0 = (int32_t)(t / p.num_n_tiles) * BT;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&b_empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&b_full[stage], GE::B_BYTES);
          tma_load_2d(sB + stage * GE::B_BYTES, &tmA, &b_full[stage], kb * KA, m0);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == B_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int s = 0; s < B_STAGES; ++s)
        if (issued & (1u << s)) drain_wait(&b_full[s], (issued_phase >> s) & 1u);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const int32_t n0 = (int32_t)(t % p.num_n_tiles) * TILE_COLS;
        for (int kb = 0; kb < KWB; ++kb) {
          if (!mbar_wait(&w_empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&w_full[stage], W_BYTES);
          if constexpr (GATED) {
            tma_load_2d(sW + stage * W_BYTES, &tmW, &w_full[stage], kb * KW, n0);
            tma_load_2d(sW + stage * W_BYTES + W_BYTES / 2, &tmW, &w_full[stage], kb * KW,
                        p.cols + n0);
          } else {
            tma_load_2d(sW + stage * W_BYTES, &tmW, &w_full[stage], kb * KW, n0);
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == W_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int s = 0; s < W_STAGES; ++s)
        if (issued & (1u << s)) drain_wait(&w_full[s], (issued_phase >> s) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, slot = 0;
      uint32_t phase = 0, sphase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        if (!mbar_wait(acc_empty, acc_phase ^ 1u, abort_flag, p.err)) break;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&b_full[stage], phase, abort_flag, p.err) ||
              !mbar_wait(&a_full[slot], sphase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b0 = smem_u32(sB + stage * GE::B_BYTES);
#pragma unroll
          for (int s = 0; s < KA / 16; ++s)
            tc_mma_f16_tmem_a(tbase, tbase + GE::A_COL0 + slot * A_SLOT_COLS + 8 * s,
                              smem_desc(b0 + s * 32, 16, 1024, 2), GE::IDESC,
                              (kb | s) != 0 ? 1u : 0u);
          tc_commit(&b_empty[stage]);
          tc_commit(&a_empty[slot]);
          if (++stage == B_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (++slot == A_SLOTS) {
            slot = 0;
            sphase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(acc_full);
        acc_phase ^= 1u;
      }
      tc_commit(final_bar);
      drain_wait(final_bar, 0);
    }
  } else if (warp >= CVT_WARP0 && warp < EPI_WARP0) {
    // ------------------------------------------------------------ converters
    const int q = warp & 3, half = (warp - CVT_WARP0) >> 2;
    const int row = GATED ? (lane < 16 ? 16 * q + lane : 64 + 16 * q + lane - 16) : 32 * q + lane;
    const uint32_t roff = (uint32_t)row * KW, rx = row & 7;
    int stage = 0, slot = half;  // this half's next operand slot: slots advance in k order
    uint32_t phase = 0, sphase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
      for (int kb = 0; kb < KB; kb += 2) {
        if (!mbar_wait(&w_full[stage], phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const bool live = kb + half < KB;
        uint32_t v[32];
        if (live) {
          const uint32_t src = smem_u32(sW + stage * W_BYTES) + roff;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 x = lds128(src + (((uint32_t)(4 * half + c) ^ rx) << 4));
            int8x4_to_f16x2(x.x, v[8 * c + 0], v[8 * c + 1]);
            int8x4_to_f16x2(x.y, v[8 * c + 2], v[8 * c + 3]);
            int8x4_to_f16x2(x.z, v[8 * c + 4], v[8 * c + 5]);
            int8x4_to_f16x2(x.w, v[8 * c + 6], v[8 * c + 7]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[stage]);
        if (live) {
          if (!mbar_wait(&a_empty[slot], sphase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          tc_st_32x32b_x32(tbase + ((uint32_t)(32 * q) << 16) + GE::A_COL0 + slot * A_SLOT_COLS, v);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_full[slot]);
        }
        if (++stage == W_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        // the pair of slots moves on by the number of halves this stage had
        const int step = kb + 1 < KB ? 2 : 1;
        slot += step;
        if (slot >= A_SLOTS) {
          slot -= A_SLOTS;
          sphase ^= 1u;
        }
      }
    }
  } else if (warp >= EPI_WARP0) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                    // TMEM lane quadrant: 32 weight rows
    const int part = (warp - EPI_WARP0) >> 2;  // tokens [part BT/2, + BT/2) of the tile
    // the scales of this warp's tokens: kept per warp, so that no barrier among the epilogue
    // warps is needed (one that gave up would leave the others waiting in it)
    float* sc = sScale + (warp - EPI_WARP0) * (BT / 2);
    uint32_t acc_phase = 0;
    for (int64_t t = blockIdx.x; t < num_tiles; t += gridDim.x) {
      const int64_t m0 = (t / p.num_n_tiles) * BT;
      const int32_t n0 = (int32_t)(t % p.num_n_tiles) * TILE_COLS;
      // output column of this lane, and the weight row its accumulator belongs to
      const int32_t n = n0 + (GATED ? 16 * q + (lane & 15) : 32 * q + lane);
      const bool nvalid = n < p.cols;
      const int64_t wrow = (GATED && lane >= 16) ? (int64_t)p.cols + n : n;
      const float sw = nvalid ? __ldg(p.w_scale + wrow) : 0.f;
      const float bias =
          p.bias && nvalid ? __uint_as_float((uint32_t)__ldg(p.bias + wrow) << 16) : 0.f;
      __syncwarp();  // the previous tile's scales have been read
#pragma unroll
      for (int i = lane; i < BT / 2; i += 32) {
        const int64_t m = m0 + part * (BT / 2) + i;
        sc[i] = m < p.M ? __ldg(p.a_scale + m) : 0.f;
      }
      __syncwarp();
      if (!mbar_wait(acc_full, acc_phase, abort_flag, p.err)) break;
      tc_fence_after();
      acc_phase ^= 1u;
      constexpr int CHUNKS = BT / 64;
#pragma unroll 1
      for (int c = 0; c < CHUNKS; ++c) {
        const int col0 = part * (BT / 2) + 32 * c;
        uint32_t r[32];
        tc_ld_32x32b_x32(tbase + ((uint32_t)(32 * q) << 16) + col0, r);
        tc_wait_ld();
        if (c == CHUNKS - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty);
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = fmaf(__uint_as_float(r[i]), sc[32 * c + i] * sw, bias);
        const int64_t left = p.M - (m0 + col0);  // tokens of this chunk
        if constexpr (GATED) {
          const int odd = lane >> 4;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i] : v[i + 1], 16);
            const float g = odd ? other : v[i], u = odd ? v[i + 1] : other;
            const float y = g / (1.f + expf(-g)) * u;
            if (nvalid && i + odd < left)
              static_cast<__nv_bfloat16*>(p.C)[(m0 + col0 + i + odd) * p.ldc + n] =
                  __float2bfloat16_rn(y);
          }
        } else if (p.c_f32) {
          float* out = static_cast<float*>(p.C) + (m0 + col0) * p.ldc + n;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (nvalid && i < left) out[i * p.ldc] = v[i];
        } else {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.C) + (m0 + col0) * p.ldc + n;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (nvalid && i < left) out[i * p.ldc] = __float2bfloat16_rn(v[i]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner,
               uint64_t rows, uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dim[2] = {inner, rows};
  cuuint64_t str[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(base), dim, str, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT, bool GATED>
qw_status launch(const Int8Problem& pr, const void* codes16, int32_t* err, cudaStream_t st) {
  using GE = Geo<BT>;
  CUtensorMap tmA, tmW;
  if (!encode_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, codes16, pr.K, pr.M, (uint64_t)pr.K * 2, KA,
                 BT) ||
      !encode_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, pr.W, pr.K, pr.N, pr.K, KW,
                 GATED ? BW / 2 : BW))
    return QW_ERR_CUDA;
  Params p{};
  p.M = pr.M;
  p.cols = GATED ? pr.N / 2 : pr.N;
  p.K = pr.K;
  constexpr int TILE_COLS = GATED ? BW / 2 : BW;
  p.num_n_tiles = (p.cols + TILE_COLS - 1) / TILE_COLS;
  p.num_m_tiles = (int32_t)((pr.M + BT - 1) / BT);
  p.a_scale = pr.a_scale;
  p.w_scale = pr.w_scale;
  p.bias = pr.bias;
  p.C = pr.C;
  p.ldc = pr.ldc;
  p.c_f32 = pr.c_f32;
  p.err = err;
  static const cudaError_t attr = cudaFuncSetAttribute(
      gemm_int8_tc_kernel<BT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GE::SMEM);
  if (attr != cudaSuccess) return QW_ERR_CUDA;
  const int64_t tiles = (int64_t)p.num_n_tiles * p.num_m_tiles;
  const int sms = device_sm_count();
  return launch_pdl(gemm_int8_tc_kernel<BT, GATED>, dim3((unsigned)(tiles < sms ? tiles : sms)),
                    dim3(NUM_THREADS), GE::SMEM, st, tmA, tmW, p);
}

}  // namespace

qw_status launch_gemm_int8_tc(const Int8Problem& p, const void* codes16, bool gated, int32_t* err,
                              cudaStream_t st) {
  if (p.M <= 64) return gated ? launch<64, true>(p, codes16, err, st) : launch<64, false>(p, codes16, err, st);
  if (p.M <= 128) return gated ? launch<128, true>(p, codes16, err, st) : launch<128, false>(p, codes16, err, st);
  return gated ? launch<256, true>(p, codes16, err, st) : launch<256, false>(p, codes16, err, st);
}

}  // namespace qw
