// gemm_int8_tc.cu - the INT8 product (and its gated form) for more than a few tokens, on the
// tcgen05 tensor cores.
//
// Mathematics: C[m][n] = a_scale[m] w_scale[n] sum_k q[m][k] w[n][k] + bias[n].  Every INT8 code
// is an FP16 number and every product of two an FP32 integer, so kind::f16 MMAs with FP32
// accumulation give the integer sum exactly while partial sums stay below 2^24, and lose up to 2^-23
// of one a step above (sm_103a's own integer tensor rate is far below its 16-bit one).
//
// Structure (persistent, one CTA per SM; a tile is 128 weight rows x BT tokens):
//   warp 0      TMA producer of the tokens' tile: FP16 codes [M][K] of the workspace, 64 k
//               (128-byte swizzle) a stage;
//   warp 2      TMA producer of the weights: INT8, 128 rows x 128 k a stage of their own ring;
//   warp 1      TMEM owner and MMA issuer: weights are the A operand, read from tensor memory,
//               tokens the B operand, read from shared memory;
//   warps 4-11  converters in two groups that take weight stages in turn: warp w covers TMEM lanes
//               32 (w % 4) .. + 31; a lane takes the 128 codes of its own row, makes them FP16
//               (byte b -> the FP16 number 1024 + (b + 128), minus 1152: exact) and stores them as
//               the MMA's A operand with one tcgen05.st for each of two operand slots.  (All eight
//               warps on every slot pay a slot's waits twice as often: 318 us for 261.)
//   warps 12-19 epilogue: tcgen05.ld the accumulator (a lane holds one weight row, a register
//               one token), release it, scale, add bias, (gated) exchange gate and up, round and
//               store while the next tile's MMAs run.  They take registers from the other warps
//               (setmaxnreg), so that half a tile's share and the packed other half fit.
// Who waits on a barrier has to see every phase of it (a wait by parity cannot tell a phase from
// the one two before).  So each weight buffer and each operand slot belongs to one converter group
// for good: the rings are even in weight stages, and a weight stage always fills two slots (past K
// both operands are zeros).
// A token stage and an operand slot of tensor memory belong together: one barrier says that both
// are full and one commit that both are free (a second commit per stage cost 8 % of the MMA rate).
// The gated form gives each 32 TMEM lanes 16 gate rows and the 16 up rows of the same outputs,
// so that a gate and its up value meet through one shuffle.
// Few tiles of long K are split: the CTAs of a cluster take slices of K, leave their FP32 sums in
// shared memory, and each finishes a share of the tile's tokens, adding the slices in rank order.
// Every wait is bounded; on expiry the kernel reports QW_ERR_TIMEOUT and shuts down.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "int8_map.cuh"
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
constexpr int A_COL0 = 256;          // the accumulator uses columns [0, BT)

// Registers: launched with 96 a thread, then shared out by warpgroup (the sum below is not above what
// the launch holds; launch() checks that the kernel was compiled to LAUNCH_REGS), and given back when a
// role ends: what comes after all roles is compiled once for every warp, to the launch's share.  The
// others' increase waits until the epilogue, which ends whatever happens, has decreased.  No role calls a
// subroutine, whose registers would not follow the share: a 64-bit division is one, so tiles are
// counted in 32 bits and stepped by additions.
constexpr int LAUNCH_REGS = 96, MISC_REGS = 56, CVT_REGS = 72, EPI_REGS = 136;
static_assert(128 * MISC_REGS + NUM_CVT_WARPS * 32 * CVT_REGS + NUM_EPI_WARPS * 32 * EPI_REGS <=
                  NUM_THREADS * LAUNCH_REGS,
              "a split above the launch's registers would wait forever");
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// the end of a role: its warps together (between two setmaxnreg a warpgroup has to be)
template <int ROLE, int WARPS>
__device__ __forceinline__ void role_end() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(ROLE), "n"(WARPS * 32) : "memory");
}

template <int BT>
struct Geo {
  static constexpr int B_BYTES = BT * KA * 2;
  static constexpr int STAGES = BT == 256 ? 4 : 8;  // token stages and operand slots
  static constexpr int W_STAGES = BT == 64 ? 6 : 4;
  static_assert(STAGES % 4 == 0 && W_STAGES % 2 == 0, "one converter group to a slot and a buffer");
  static constexpr int PARTIAL_BYTES = BT == 256 ? 0 : BW * BT * 4;  // over the ring, at the end
  static constexpr size_t SMEM = (size_t)STAGES * B_BYTES + W_STAGES * W_BYTES +
                                 NUM_EPI_WARPS * (BT / 2) * 4 + 512 + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(PARTIAL_BYTES <= STAGES * B_BYTES, "partial sums fit the token ring");
  static_assert(A_COL0 + STAGES * A_SLOT_COLS <= 512, "tensor memory");
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
  int32_t group;         // token tiles of a group
  uint32_t group_tiles;  // group x num_n_tiles
  const float* a_scale;
  const int8_t* W;
  const float* w_scale;
  const uint16_t* bias;
  void* C;
  int64_t ldc;
  int32_t c_f32;
  int32_t csize;      // CTAs that share a tile's K (1 where tiles fill the GPU)
  uint32_t b_bytes;   // of a token stage's copy (fewer rows than BT where M has fewer)
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
// one lane of the warp (converged), the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// What a thread does with the finished sums of its weight row: scale, bias, gate, round, store.
template <bool GATED>
struct Out {
  void* C;
  int64_t ldc;
  int32_t n;       // output column of this lane
  bool nvalid, c_f32;
  float sw, bias;  // of the lane's weight row
  int lane;

  __device__ __forceinline__ float value(float sum, float sa) const {
    return fmaf(sum, sa * sw, bias);
  }
  // (gated) lanes 0-15 hold the gate rows and finish the first of two tokens, lanes 16-31 the up
  // rows and finish the second
  __device__ __forceinline__ float gate(float a, float b) const {
    const bool odd = lane >= 16;
    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 16);
    const float g = odd ? other : a, u = odd ? b : other;
    return gate_up(g, u);
  }
  // FP32 results (BT <= 128: for 256 tokens a tile the registers do not reach): 128 contiguous
  // bytes a token as they are.
  __device__ __forceinline__ void store_f32(const uint32_t (&r)[2][32], const float* sc, int step,
                                            int64_t m, int64_t left) const {
    float* o = static_cast<float*>(C) + m * ldc + n;
    const int count = nvalid ? (int)min64(left, step) : 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      if (i < count) *o = value(__uint_as_float(r[i / 32][i % 32]), sc[i]);
      o += ldc;
    }
  }
  // Sums of STEP tokens -> BF16, two to a register: tokens 2j and 2j + 1, or (gated) what the lane
  // has of the token pairs 2j and 2j + 1.
  template <int STEP>
  __device__ __forceinline__ void pack(const uint32_t (&r)[2][32], const float* sc,
                                       uint32_t (&packed)[STEP / (GATED ? 4 : 2)]) const {
#pragma unroll
    for (int i = 0; i < STEP; i += 4) {
      const float4 s = *reinterpret_cast<const float4*>(sc + i);
      const float a = value(__uint_as_float(r[i / 32][i % 32]), s.x);
      const float b = value(__uint_as_float(r[i / 32][i % 32 + 1]), s.y);
      const float c = value(__uint_as_float(r[i / 32][i % 32 + 2]), s.z);
      const float d = value(__uint_as_float(r[i / 32][i % 32 + 3]), s.w);
      if constexpr (GATED) {
        packed[i / 4] = pack_bf16x2(gate(a, b), gate(c, d));
      } else {
        packed[i / 2] = pack_bf16x2(a, b);
        packed[i / 2 + 1] = pack_bf16x2(c, d);
      }
    }
  }
  // ... to memory: a warp's 32 columns of a token are 64 contiguous bytes (gated: 16 of each of
  // two tokens).  Through shared memory into 16-byte stores the same took five times as long: the
  // detour costs more shared-memory passes than the narrow stores do.
  template <int STEP>
  __device__ __forceinline__ void store(const uint32_t (&packed)[STEP / (GATED ? 4 : 2)], int64_t m,
                                        int64_t left) const {
    constexpr int APART = GATED ? 2 : 1;  // tokens between a register's two values
    uint16_t* o = static_cast<uint16_t*>(C) + (m + (GATED ? lane >> 4 : 0)) * ldc + n;
    const int count = nvalid ? (int)min64(left, STEP) - (GATED ? lane >> 4 : 0) : 0;
    const int64_t apart = APART * ldc;
#pragma unroll
    for (int i = 0; i < STEP / (GATED ? 4 : 2); ++i) {
      if (2 * i * APART < count) *o = (uint16_t)packed[i];
      o += apart;
      if ((2 * i + 1) * APART < count) *o = (uint16_t)(packed[i] >> 16);
      o += apart;
    }
  }
};

template <int BT, bool GATED>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_int8_tc_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmW, const Params p) {
  using GE = Geo<BT>;
  constexpr int STAGES = GE::STAGES, W_STAGES = GE::W_STAGES;
  constexpr int TILE_COLS = GATED ? BW / 2 : BW;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sB = smem;
  uint8_t* sW = sB + STAGES * GE::B_BYTES;
  float* sScale = reinterpret_cast<float*>(sW + W_STAGES * W_BYTES);  // [8 warps][BT/2]
  uint64_t* full = reinterpret_cast<uint64_t*>(sScale + NUM_EPI_WARPS * (BT / 2));
  uint64_t* empty = full + STAGES;
  uint64_t* w_full = empty + STAGES;
  uint64_t* w_empty = w_full + W_STAGES;
  uint64_t* acc_full = w_empty + W_STAGES;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* final_bar = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(final_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1 + NUM_CVT_WARPS / 2);  // the tokens' copy and a converter group
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < W_STAGES; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], NUM_CVT_WARPS / 2);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, NUM_EPI_WARPS);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int csize = p.csize;
  const int rank = (int)(blockIdx.x % (unsigned)csize);
  const uint32_t cluster = blockIdx.x / (unsigned)csize, clusters = gridDim.x / (unsigned)csize;
  const uint32_t num_n = (uint32_t)p.num_n_tiles, num_tiles = (uint32_t)p.num_m_tiles * num_n;
  // Tile t: groups of `group` token tiles, in each the weight tiles in turn, for each the group's token
  // tiles.
  struct Tile {
    uint32_t t, mt, nt;
  };
  auto locate = [&](Tile& x) {
    const uint32_t m0 = x.t / p.group_tiles * (uint32_t)p.group;
    const uint32_t r = x.t % p.group_tiles, gm = min((uint32_t)p.group, (uint32_t)p.num_m_tiles - m0);
    x.nt = r / gm;
    x.mt = m0 + r % gm;
  };
  auto next = [&](Tile& x) {
    x.t += clusters;
    if (x.t < num_tiles) locate(x);
  };
  Tile first{cluster, 0, 0};
  locate(first);
  // this CTA's k stages of every tile, in weight stages of two
  const int KWB = (p.K + KW - 1) / KW, kw_per = (KWB + csize - 1) / csize;
  const int kw_beg = min(KWB, rank * kw_per), kw_end = min(KWB, kw_beg + kw_per);
  const int kb_beg = 2 * kw_beg, kb_end = 2 * kw_end;

  if constexpr (BT == 64) {
    // the first weight stages on their way to L2 while the call's quantiser runs (32 and 64 tokens:
    // 20.3 -> 19.5 us at 14336 x 4096)
    const int r = threadIdx.x % BW, kw = kw_beg + threadIdx.x / BW;
    const int32_t n = (int32_t)(first.nt * TILE_COLS) + r % TILE_COLS;
    if (kw < kw_end && n < p.cols)
      prefetch_l2(p.W + ((int64_t)(r / TILE_COLS ? p.cols : 0) + n) * p.K + kw * KW);
  }
  // What is above overlaps the previous kernel's tail; everything else comes after this, the
  // first use of the tensor maps included: they lie in the launch's parameters, whose addresses
  // are used again by later launches, and an SM may hold a map of an earlier one until here.  The next
  // kernel may start now: whatever came before this call is complete.
  pdl_wait();
  pdl_launch_dependents();

  if (warp < CVT_WARP0) {
    regs_dec<MISC_REGS>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- tokens
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (Tile x = first; ok && x.t < num_tiles; next(x)) {
        const int32_t m0 = (int32_t)(x.mt * BT);
        for (int kb = kb_beg; kb < kb_end; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], p.b_bytes);
          tma_load_2d(sB + stage * GE::B_BYTES, &tmA, &full[stage], kb * KA, m0);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // (after a wait that gave up, a stage may also lack its converters: bounded either way)
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) wait_landed(&full[s], (issued_phase >> s) & 1u);
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------- weights
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (Tile x = first; ok && x.t < num_tiles; next(x)) {
        const int32_t n0 = (int32_t)(x.nt * TILE_COLS);
        for (int kb = kw_beg; kb < kw_end; ++kb) {
          if (!mbar_wait(&w_empty[stage], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&w_full[stage], W_BYTES);
          tma_load_2d(sW + stage * W_BYTES, &tmW, &w_full[stage], kb * KW, n0);
          if constexpr (GATED)
            tma_load_2d(sW + stage * W_BYTES + W_BYTES / 2, &tmW, &w_full[stage], kb * KW,
                        p.cols + n0);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == W_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int s = 0; s < W_STAGES; ++s)
        if (issued & (1u << s)) wait_landed(&w_full[s], (issued_phase >> s) & 1u);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one elected lane issues: descriptors, addresses and
      // loop state then stay in uniform registers.  (With a single-lane loop a stage's issue took
      // 600 cycles, more than its MMAs.)
      const bool leader = elect_one();
      const uint64_t desc0 = smem_desc(smem_u32(sB), 16, 1024, 2);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (Tile x = first; ok && x.t < num_tiles; next(x)) {
        if (!warp_wait(acc_empty, acc_phase ^ 1u, abort_flag, p.err)) break;
        for (int kb = kb_beg; kb < kb_end; ++kb) {
          if (!warp_wait(&full[stage], phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t desc = desc0 + (uint32_t)(stage * (GE::B_BYTES >> 4));
          const uint32_t a = tbase + A_COL0 + stage * A_SLOT_COLS;
          if (leader) {
#pragma unroll
            for (int s = 0; s < KA / 16; ++s)  // 32 bytes of k: 2 in the descriptor's units
              tc_mma_f16_tmem_a(tbase, a + 8 * s, desc + 2 * s, GE::IDESC,
                                kb != kb_beg || s != 0 ? 1u : 0u);
            tc_commit(&empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (leader) tc_commit(acc_full);
        __syncwarp();
        acc_phase ^= 1u;
      }
      if (leader) {
        tc_commit(final_bar);
        wait_landed(final_bar, 0);
      }
    }
    role_end<1, CVT_WARP0>();
    regs_inc<LAUNCH_REGS>();
  } else if (warp < EPI_WARP0) {
    // ------------------------------------------------------------ converters
    regs_dec<CVT_REGS>();
    const int q = warp & 3, group = (warp - CVT_WARP0) >> 2;
    const int row = GATED ? (lane < 16 ? 16 * q + lane : 64 + 16 * q + lane - 16) : 32 * q + lane;
    const uint32_t roff = (uint32_t)row * KW, rx = row & 7;
    const uint32_t dst = tbase + ((uint32_t)(32 * q) << 16) + A_COL0;
    // this group's next weight buffer and first operand slot, and their phases
    int wstage = group, slot = 2 * group;
    uint32_t wphase = 0, phase = 0;
    bool ok = true;
    int mine = group;  // weight stages until this group's next
    for (Tile x = first; ok && x.t < num_tiles; next(x)) {
      for (int kw = kw_beg; kw < kw_end; ++kw, mine ^= 1) {
        if (mine) continue;
        if (!warp_wait(&w_full[wstage], wphase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        uint4 w[8];
        const uint32_t src = smem_u32(sW + wstage * W_BYTES) + roff;
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = lds128(src + (((uint32_t)c ^ rx) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[wstage]);
        wstage += 2;
        if (wstage >= W_STAGES) {
          wstage = group;
          wphase ^= 1u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            int8x4_to_f16x2(w[4 * h + c].x, v[8 * c + 0], v[8 * c + 1]);
            int8x4_to_f16x2(w[4 * h + c].y, v[8 * c + 2], v[8 * c + 3]);
            int8x4_to_f16x2(w[4 * h + c].z, v[8 * c + 4], v[8 * c + 5]);
            int8x4_to_f16x2(w[4 * h + c].w, v[8 * c + 6], v[8 * c + 7]);
          }
          if (!warp_wait(&empty[slot + h], phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          tc_st_32x32b_x32(dst + (slot + h) * A_SLOT_COLS, v);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot + h]);
        }
        if (!ok) break;
        slot += 4;
        if (slot >= STAGES) {
          slot = 2 * group;
          phase ^= 1u;
        }
      }
    }
    role_end<2, NUM_CVT_WARPS>();
    regs_inc<LAUNCH_REGS>();
  } else {
    // ------------------------------------------------------------ epilogue
    regs_inc<EPI_REGS>();
    const int q = warp & 3;                    // TMEM lane quadrant: 32 weight rows
    const int part = (warp - EPI_WARP0) >> 2;  // tokens [part BT/2, + BT/2) of the tile
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    // the scales of this warp's tokens: kept per warp, so that no barrier among the epilogue
    // warps is needed (one that gave up would leave the others waiting in it)
    float* sc = sScale + (warp - EPI_WARP0) * (BT / 2);
    Out<GATED> out{};
    out.C = p.C;
    out.ldc = p.ldc;
    out.c_f32 = p.c_f32;
    out.lane = lane;
    uint32_t acc_phase = 0;
    for (Tile x = first; x.t < num_tiles; next(x)) {
      const int64_t m0 = (int64_t)x.mt * BT;
      out.n = (int32_t)(x.nt * TILE_COLS) + (GATED ? 16 * q + (lane & 15) : 32 * q + lane);
      out.nvalid = out.n < p.cols;
      const int64_t wrow = (GATED && lane >= 16) ? (int64_t)p.cols + out.n : out.n;
      out.sw = out.nvalid ? p.w_scale[wrow] : 0.f;
      out.bias = p.bias && out.nvalid ? __uint_as_float((uint32_t)p.bias[wrow] << 16) : 0.f;
      __syncwarp();  // the previous tile's scales have been read
      const int64_t mw = m0 + part * (BT / 2);  // first token of this warp
#pragma unroll
      for (int i = lane; i < BT / 2; i += 32) sc[i] = mw + i < p.M ? p.a_scale[mw + i] : 0.f;
      __syncwarp();
      if (!warp_wait(acc_full, acc_phase, abort_flag, p.err)) break;
      tc_fence_after();
      acc_phase ^= 1u;
      const uint32_t acc = tbase + lane_base + part * (BT / 2);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      };
      // 64 tokens at a time, in a loop that is kept short (fully unrolled for 128 tokens, the
      // epilogue spent most of its time fetching instructions).  The first 64 are rounded and
      // packed, which frees their registers for the others; then the accumulator is released,
      // and only then does anything go to memory.
      constexpr int COLS = BT / 2, STEP = COLS < 64 ? COLS : 64;
      uint32_t r[2][32];
      auto load = [&](int c0) {
        __syncwarp();  // .sync.aligned wants the whole warp
        tc_ld_32x32b_x32(acc + c0, r[0]);
        if constexpr (STEP > 32) tc_ld_32x32b_x32(acc + c0 + 32, r[1]);
        tc_wait_ld();
        if (c0 + STEP == COLS) release();
      };
      load(0);
      if constexpr (BT < 256) {
        if (csize > 1) {
          // K split over the cluster: sums of [token][row] over the token ring, which every MMA
          // has read; finished below, with every warp of the CTAs
          float* sum = reinterpret_cast<float*>(sB) + (int64_t)(part * COLS) * BW + 32 * q + lane;
#pragma unroll
          for (int i = 0; i < STEP; ++i) sum[i * BW] = __uint_as_float(r[i / 32][i % 32]);
          break;  // one tile per cluster
        }
      }
#pragma unroll 1
      for (int c0 = 0; c0 < COLS; c0 += STEP) {
        const int64_t m = mw + c0, left = p.M - m;  // tokens of this step
        if constexpr (!GATED && BT < 256) {
          if (p.c_f32) {
            out.store_f32(r, sc, STEP, m, left);
            break;  // one step: COLS <= 64
          }
        }
        uint32_t packed[STEP / (GATED ? 4 : 2)];
        out.template pack<STEP>(r, sc + c0, packed);
        if (c0 + STEP < COLS) load(c0 + STEP);
        out.template store<STEP>(packed, m, left);
      }
    }
    role_end<3, NUM_EPI_WARPS>();
    regs_dec<LAUNCH_REGS>();
  }

  if constexpr (BT < 256) {
    if (csize > 1) {
      // Every CTA's sums are in its shared memory; this one finishes tokens rank, rank + csize, .. of
      // the tile, adding the slices in rank order.  A lane has four weight rows of a token.
      const int64_t m0 = (int64_t)first.mt * BT;
      const bool up = GATED && (lane & 4);
      const int32_t n = (int32_t)(first.nt * TILE_COLS) +
                        (GATED ? 16 * (lane >> 3) + 4 * (lane & 3) : 4 * lane);
      float sw[4] = {}, bias[4] = {};
      if (warp >= EPI_WARP0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < p.cols) {
            const int64_t wrow = (int64_t)(up ? p.cols : 0) + n + j;
            sw[j] = p.w_scale[wrow];
            if (p.bias) bias[j] = __uint_as_float((uint32_t)p.bias[wrow] << 16);
          }
      }
      cluster_sync();
      if (warp >= EPI_WARP0 && *abort_flag == 0) {
        const int tokens = (int)min64(BT, p.M - m0), step = csize * NUM_EPI_WARPS;
        // Two tokens at a time: one waits for more latencies, four are more instructions, which a CTA
        // has to fetch for the few times that it runs them (us with 1, 2 and 4 tokens:
        // 256 x 4096 x 4096 17.4, 16.6, 17.9; 128 x 1024 x 4096 10.0, 11.1, 12.7).
        constexpr int U = 2;
        for (int i0 = rank + csize * (warp - EPI_WARP0); i0 < tokens; i0 += step * U) {
          float sum[U][4] = {}, sa[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            sa[u] = i0 + step * u < tokens ? p.a_scale[m0 + i0 + step * u] : 0.f;
          for (int c = 0; c < csize; ++c) {
            const uint32_t from = mapa_shared(smem_u32(sB) + lane * 16, (uint32_t)c);
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (i0 + step * u < tokens) {
                const float4 v = ld_cluster_f32x4(from + (uint32_t)(i0 + step * u) * (BW * 4));
                sum[u][0] += v.x;
                sum[u][1] += v.y;
                sum[u][2] += v.z;
                sum[u][3] += v.w;
              }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (i0 + step * u >= tokens) break;
            const int64_t at = (m0 + i0 + step * u) * p.ldc + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float y = fmaf(sum[u][j], sa[u] * sw[j], bias[j]);
              if constexpr (GATED) y = gate_up(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
              if (up || n + j >= p.cols) continue;
              if (p.c_f32)
                static_cast<float*>(p.C)[at + j] = y;
              else
                static_cast<__nv_bfloat16*>(p.C)[at + j] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      cluster_sync();  // nobody leaves while its sums are read
    }
  }
  __syncwarp();  // single-lane roles have left their warps apart
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

// Clusters of csize CTAs that run at once (fewer than SMs / csize: a cluster lies within one GPC)
template <int BT>
int max_clusters(int csize) {
  static std::atomic<int> cache[4][64];
  const int found = once_per_device(cache[csize == 8 ? 3 : csize >> 1], [=] {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)csize);
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = Geo<BT>::SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)csize;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(gemm_int8_tc_kernel<BT, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Geo<BT>::SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, gemm_int8_tc_kernel<BT, false>, &cfg) != cudaSuccess)
      return 0;
    return n + 1;  // (none is an answer too)
  });
  // without an answer (or an SM free of others) tiles are counted in rounds over all SMs, none split
  return found > 1 ? found - 1 : csize > 1 ? 0 : device_sm_count();
}

struct Plan {
  int64_t cost;
  int csize;  // CTAs that share a tile's K
};
// The cheapest split of K with tiles of BT tokens, and what the product then takes in quarters of the
// time of one k at BT <= 128 (the MMAs are bound by the weight operand there, whose 128 rows x 16 k
// take as long for 64 tokens as for 128; 256 take 5/4 of it): each round of tiles over the SMs pays its
// k and its epilogue, a split also the joining.
template <int BT>
Plan plan(const Int8Problem& p, bool gated) {
  const int64_t n_tiles = gated ? (p.N / 2 + BW / 2 - 1) / (BW / 2) : (p.N + BW - 1) / BW;
  const int64_t tiles = n_tiles * ((p.M + BT - 1) / BT);
  const int64_t rounds = (tiles + max_clusters<BT>(1) - 1) / max_clusters<BT>(1);
  Plan best{rounds * ((int64_t)p.K * (BT == 256 ? 5 : 4) + 8 * BT), 1};
  for (int c = 2; BT < 256 && c <= 8; c *= 2) {
    const int stages = (p.K + KW - 1) / KW, per = (stages + c - 1) / c;
    if (tiles > max_clusters<BT>(c) || p.K / c < 512) break;
    if ((c - 1) * per >= stages) continue;  // every CTA has a share (its accumulator holds sums)
    const int64_t cost = (int64_t)per * KW * 4 + 8 * BT + 2048;
    if (cost < best.cost) best = Plan{cost, c};
  }
  return best;
}

template <int BT, bool GATED>
qw_status launch(const Int8Problem& pr, const void* codes16, int csize, int32_t* err,
                 cudaStream_t st) {
  using GE = Geo<BT>;
  CUtensorMap tmA, tmW;
  // A tile's rows past M: none are copied where M is below BT (whatever the stage holds there
  // ends in accumulator columns that nobody reads), zeros in the last of several token tiles.
  // (Copies of 64 rows, most of them outside the tensor, cost 5 us of 20 at M = 4 to 8.)
  const uint32_t box_rows = (uint32_t)min64(BT, (pr.M + 7) / 8 * 8);
  if (!encode_int8_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, codes16, pr.K, pr.M, (uint64_t)pr.K * 2, KA,
                 box_rows) ||
      !encode_int8_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, pr.W, pr.K, pr.N, pr.K, KW,
                 GATED ? BW / 2 : BW))
    return QW_ERR_CUDA;
  Params p{};
  p.M = pr.M;
  p.cols = GATED ? pr.N / 2 : pr.N;
  p.K = pr.K;
  constexpr int TILE_COLS = GATED ? BW / 2 : BW;
  p.num_n_tiles = (p.cols + TILE_COLS - 1) / TILE_COLS;
  p.num_m_tiles = (int32_t)((pr.M + BT - 1) / BT);
  // What the CTAs work on at a time is then a few weight tiles for a group's token tiles, and all
  // weights pass by once per group.  (us with groups of one tile, 8, 16, 32 and 64 MB: gated
  // 4096 x 2x14336 x 4096 587, 553, 530, 536, 543; 16384 x 4096 x 4096 347, 330, 331, 344, 394.)
  constexpr int64_t kGroupBytes = 16 << 20;
  p.group = (int32_t)std::max<int64_t>(1, min64(p.num_m_tiles, kGroupBytes / ((int64_t)BT * pr.K * 2)));
  p.group_tiles = (uint32_t)min64((int64_t)p.group * p.num_n_tiles, 0x7FFFFFFF);
  p.a_scale = pr.a_scale;
  p.W = pr.W;
  p.w_scale = pr.w_scale;
  p.bias = pr.bias;
  p.C = pr.C;
  p.ldc = pr.ldc;
  p.c_f32 = pr.c_f32;
  p.b_bytes = box_rows * KA * 2;
  p.err = err;
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [] {
        cudaFuncAttributes fa{};
        return cudaFuncSetAttribute(gemm_int8_tc_kernel<BT, GATED>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)GE::SMEM) == cudaSuccess &&
               cudaFuncGetAttributes(&fa, gemm_int8_tc_kernel<BT, GATED>) == cudaSuccess &&
               fa.numRegs == LAUNCH_REGS;  // the register split depends on it
      }) <= 0)
    return QW_ERR_CUDA;
  const int64_t tiles = (int64_t)p.num_n_tiles * p.num_m_tiles;
  const int sms = device_sm_count();
  if (tiles > 0x7FFFFFFF - sms) return QW_ERR_UNSUPPORTED;  // counted in 32 bits
  p.csize = csize;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(csize > 1 || tiles < sms ? tiles * csize : sms));
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
  return cudaLaunchKernelEx(&cfg, gemm_int8_tc_kernel<BT, GATED>, tmA, tmW, p) == cudaSuccess
             ? QW_OK
             : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_gemm_int8_tc(const Int8Problem& p, const void* codes16, bool gated, int32_t* err,
                              cudaStream_t st) {
  // The cheapest tile (us with 64, 128 and 256 tokens a tile, those of the rule in brackets:
  // 333 x 1000 x 1040 [9.0] 9.5 13.4, 512 x 4096 x 4096 26.9 [21.4] 26.8, 256 x 4096 x 14336 55 [36] 71,
  // 4096 x 14336 x 4096 [258] with 256.)  FP32 results do not leave 256 tokens' sums the registers.
  const Plan p64 = plan<64>(p, gated), p128 = plan<128>(p, gated), p256 = plan<256>(p, gated);
  const bool use256 = !p.c_f32 && p256.cost < std::min(p64.cost, p128.cost);
  auto go = [&](auto bt, const Plan& l) {
    constexpr int BT = decltype(bt)::value;
    return gated ? launch<BT, true>(p, codes16, l.csize, err, st)
                 : launch<BT, false>(p, codes16, l.csize, err, st);
  };
  if (use256) return go(std::integral_constant<int, 256>{}, p256);
  if (p128.cost < p64.cost) return go(std::integral_constant<int, 128>{}, p128);
  return go(std::integral_constant<int, 64>{}, p64);
}

}  // namespace qw
