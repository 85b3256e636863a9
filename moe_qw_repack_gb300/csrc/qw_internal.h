// qw_internal.h - host-side launchers shared between the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "../../include/qw.h"

namespace qw {

// Number of SMs of the current device (cached per device).
int device_sm_count();
// What `find` says (a positive number; anything else is a failure, which is not kept) of the current
// device, found once for each.
template <class F>
int once_per_device(std::atomic<int> (&cache)[64], F&& find) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  int v = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (v > 0) return v;
  v = find();
  if (v > 0 && dev < 64) cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Packed-layout geometry shared by repack and the GEMM kernels.
constexpr int kIntGroup = 128;       // K elements per BF16 scale (INT formats)
constexpr int kMxGroup = 32;         // K elements per E8M0 scale (MX formats)
constexpr int kInt4BlockBytes = 1024;  // 16 rows x 128 k of INT4, fragment order
constexpr int kInt2BlockBytes = 512;   // 16 rows x 128 k of INT2, fragment order
constexpr int kInt3BlockBytes = 768;   // 16 rows x 128 k of INT3 (two bit planes)
constexpr int kFp8BlockBytes = 2048;   // 16 rows x 128 k of E4M3 codes, fragment order
constexpr int kInt1BlockBytes = 256;   // 16 rows x 128 k of INT1 sign bits, fragment order
constexpr int kFp4BlockBytes = 1024;   // 16 rows x 128 k of E2M1 codes, fragment order
// Format codes of the WnA16 kernels' templates: the integer bit width (4, 3, 2, 1), 8 for
// E4M3 weights and kBitsFp4 for E2M1 weights (FP4 codes in the INT4 block geometry).
constexpr int kBitsFp4 = 5;
// Bytes of one packed 16 x 128 block of a WnA16 format code.
__host__ __device__ constexpr int wna16_block_bytes(int bits) {
  return bits == kBitsFp4 ? kFp4BlockBytes : bits * 256;
}
constexpr int kSfChunkBytes = 512;     // 128 rows x 4 groups of E8M0 scales
constexpr int kNvGroup = 16;           // K elements per E4M3 scale (NVFP4)
constexpr int kNvChunkBytes = 2048;    // 128 rows x 16 groups of E4M3 scales (NVFP4)

qw_status launch_repack(const qw_packed_desc& d, const void* w_canon, const void* s_canon,
                        void* w_packed, void* s_packed, int32_t* err, cudaStream_t st);
qw_status launch_unpack(const qw_packed_desc& d, const void* w_packed, const void* s_packed,
                        void* w_canon, void* s_canon, int32_t* err, cudaStream_t st);
// second-level scales: fill the packed plane with 1.0, copy [E][N] <-> [E][N_pad]
qw_status launch_scale2_fill(float* t_packed, int64_t n, cudaStream_t st);
qw_status launch_scale2_repack(const float* t_canon, float* t_packed, int32_t E, int32_t N,
                               int32_t N_pad, int32_t* err, cudaStream_t st);
qw_status launch_scale2_unpack(const float* t_packed, float* t_canon, int32_t E, int32_t N,
                               int32_t N_pad, cudaStream_t st);

// Rows of a GEMM call: dense (offsets == nullptr, rows [0, M)) or grouped by expert
// (device offsets [E+1]; the work list of (expert, row tile) is built on the device).
struct RowSet {
  int64_t rows;                // M (dense) or total rows (grouped)
  const int32_t* offsets;      // device [E+1] or nullptr
  int32_t E;
  // Indexed grouped calls: row r of the problem is activation row gather[r] / topk of an
  // unpermuted [a_rows][K] input (gather = the router's sorted pair ids); else nullptr.
  const int32_t* gather = nullptr;
  int32_t topk = 1;
  int64_t a_rows = 0;
  // second-level scales: device FP32 [E][N_pad] multiplying each output channel's sum
  // before the bias, or nullptr
  const float* scale2 = nullptr;
};

// Small-M W4A16: tensor-core GEMV over the fragment-ordered packed weights.
qw_status launch_gemv_w4a16(const qw_packed_desc& d, const void* w_packed, const void* s_packed,
                            const void* A, const void* bias, void* C, const RowSet& rs,
                            void* ws, uint64_t ws_bytes, int32_t* err, cudaStream_t st);
uint64_t gemv_w4a16_workspace(const qw_packed_desc& d, int64_t max_rows);

// Large-M W4A16: in-SM dequantization into tensor memory + tcgen05 BF16 GEMM.
qw_status launch_gemm_w4a16_tc(const qw_packed_desc& d, const void* w_packed,
                               const void* s_packed, const void* A, const void* bias, void* C,
                               const RowSet& rs, void* ws, uint64_t ws_bytes, int32_t* err,
                               cudaStream_t st);
uint64_t gemm_w4a16_tc_workspace(const qw_packed_desc& d, int64_t max_rows);

// Rows from which W4A16 runs on the tensor-core path (dense M above it, or a grouped call
// averaging at least this many rows per expert); below it the GEMV streams the weights.
// Measured on GB300 (14336 x 4096 INT4): the GEMV is faster at M <= 16, the tcgen05 path
// from M = 32 (23.8 vs 36.3 us); MoE up projection E=128: GEMV 214 us vs tcgen05 114 us
// at 16 rows per expert.
constexpr int64_t kW4A16TensorCoreRows = 16;

// Activation-side MoE steps (act.cu).
qw_status launch_quantize_mxfp8(const void* A, int64_t rows, int32_t K, void* Q, void* SF,
                                int32_t* err, cudaStream_t st);
qw_status launch_silu_mul(const void* GU, int64_t rows, int32_t I, void* Y, cudaStream_t st);
qw_status launch_moe_combine(const void* Y, const int32_t* sorted_pairs, const int32_t* topk_ids,
                             const float* logits, int32_t T, int32_t E, int32_t topk, int32_t N,
                             void* out, int32_t* inv, int32_t* err, cudaStream_t st);

// Large-M W4A8: TMA + tcgen05 block-scaled GEMM.
qw_status launch_gemm_w4a8(const qw_packed_desc& d, const void* w_packed, const void* s_packed,
                           const void* A, const void* A_sf, const void* bias, void* C,
                           const RowSet& rs, void* ws, uint64_t ws_bytes, int32_t* err,
                           cudaStream_t st);
uint64_t gemm_w4a8_workspace(const qw_packed_desc& d, int64_t max_rows);

// Dense W4A8 (MXFP4 weights) calls of at most this many rows whose staged activations
// (FP16 B fragments and FP32 scales of every group) fit kW4A8GemvMaxSmem run the
// streaming GEMV.
constexpr int kW4A8GemvRows = 8;
constexpr size_t kW4A8GemvMaxSmem = 96 * 1024;
constexpr size_t w4a8_gemv_smem_bytes(int K, int M) {
  return (size_t)(K / 32) * ((size_t)M * 64 + 32);
}
qw_status launch_gemv_w4a8(const qw_packed_desc& d, const void* w_packed, const void* s_packed,
                           const void* A, const void* A_sf, const void* bias, const float* scale2,
                           void* C, int M, int32_t* err, cudaStream_t st);

// INT8 product and its gated form (int8.cu): INT8 codes and FP32 scales on both sides.
struct Int8Problem {
  const int8_t* A;       // [M][lda] codes
  int64_t lda;
  const float* a_scale;  // [M]
  const int8_t* W;       // [N][K] codes (gated: N = 2 I, gate rows first)
  const float* w_scale;  // [N]
  const uint16_t* bias;  // BF16 [N] or null
  void* C;               // BF16 or FP32 [M][ldc]
  int64_t ldc;
  int64_t M;
  int32_t N, K;
  bool c_f32;
};
// largest K whose 32-bit integer sums cannot overflow (128 * 128 * K < 2^31), K % 16 == 0
constexpr int32_t kInt8MaxK = 131056;
// largest N: columns are counted in 32 bits, rounded up to whole tiles (of at most 128)
constexpr int32_t kInt8MaxN = 0x7FFFFFFF - 255;
// One or two tokens: dp4a.  Up to kInt8MmaRows: mma.sync.  More: tcgen05.  At N = 14336, K = 4096
// (us): 2 tokens 13.4 with dp4a, 14.1 with mma.sync; 4 tokens 17.4 and 14.1; 16 tokens 15.2 with
// mma.sync, 20.2 with tcgen05; 32 tokens 38 and 19.6.
constexpr int64_t kInt8GemvRows = 2, kInt8MmaRows = 16;
// f16: write the codes as FP16 integers (the tensor-core kernel's operand) instead of INT8
qw_status launch_quantize_int8(const void* A, int64_t lda, int64_t rows, int32_t K, void* Q,
                               float* scale, bool f16, int32_t* err, cudaStream_t st);
qw_status launch_widen_int8(const void* A, int64_t lda, int64_t M, int32_t K, void* Q,
                            cudaStream_t st);
// early: the call's own quantiser was enqueued directly before
qw_status launch_gemv_int8(const Int8Problem& p, bool gated, bool early, int32_t* err,
                           cudaStream_t st);
// M <= kInt8MmaRows
qw_status launch_gemm_int8_mma(const Int8Problem& p, bool gated, int32_t* err, cudaStream_t st);
// codes16: the activations' codes as FP16 [M][K] (p.A is not read)
qw_status launch_gemm_int8_tc(const Int8Problem& p, const void* codes16, bool gated, int32_t* err,
                              cudaStream_t st);

// Log probabilities (logprobs.cu); null outputs are not computed.
struct LogprobsArgs {
  const void* logits;
  int64_t ld;
  int32_t V;
  const int32_t* tokens;
  float* token_logprob;
  int32_t* token_rank;
  float* entropy;
  int32_t topk;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* err;
};
constexpr int32_t kLogprobsMaxTop = 32;
constexpr int64_t kLogprobsMaxRows = (int64_t)1 << 26;  // rows of one call (grid size)
qw_status launch_logprobs(const LogprobsArgs& a, int32_t type, int64_t T, cudaStream_t st);

// Residual addition, norm and 8-bit operand (norm.cu); R, R_out, Y and Q may be null.
struct NormArgs {
  const void* X;   // BF16 or FP32
  int64_t ldx;
  const void* R;   // BF16 or FP32
  int64_t ldr;
  void* R_out;     // R's type
  int64_t ldro;
  const void* W;   // BF16 [K]
  float offset, eps;
  int64_t rows;
  int32_t K;
  void* Y;         // BF16
  int64_t ldy;
  void* Q;         // codes [rows][K]
  void* Q_sf;
  int32_t* err;
};
qw_status launch_rmsnorm(const NormArgs& a, int32_t x_type, int32_t r_type, int32_t q_fmt,
                         cudaStream_t st);

// Low-rank adapters (lora.cu); scales, ranks and base may be null.
struct LoraArgs {
  const uint16_t* X;      // BF16 [M][ldx]
  int64_t ldx;
  const uint16_t* A;      // BF16 [L][R][K]
  const uint16_t* B;      // BF16 [L][N][R]
  const float* scales;    // [L]
  const int32_t* ranks;   // [L]
  int32_t L, R;
  const int32_t* ids;     // [M]
  const void* base;       // C's type
  int64_t ld_base;
  void* C;
  int64_t ldc;
  int64_t M;
  int32_t N, K;
  int32_t* err;
};
constexpr int32_t kLoraMaxRank = 256;
constexpr int32_t kLoraMaxDim = 1 << 30;  // N and K: counted in 32 bits, rounded up to whole blocks
constexpr int64_t kLoraMaxRows = (int64_t)1 << 26;  // tokens of one call (grid size)
qw_status launch_lora(const LoraArgs& a, bool c_f32, cudaStream_t st);
// on tcgen05, for more tokens
bool lora_tc_takes(const LoraArgs& a, bool c_f32);
qw_status launch_lora_tc(const LoraArgs& a, bool c_f32, cudaStream_t st);

// Rotary positions (rope.cu).
struct RopeArgs {
  const void* X;
  int64_t ldx;
  void* Y;
  int64_t ldy;
  int64_t T;
  int32_t heads, head_dim, rot;
  const int32_t* positions;  // [T]
  const double* freqs;       // [rot / 2]
  float scale;
  int32_t* err;
};
constexpr int32_t kRopeMaxDim = 1024;       // of a head
constexpr int32_t kRopeMaxWidth = 1 << 24;  // of a token's heads together
qw_status launch_rope(const RopeArgs& a, int32_t type, int32_t layout, cudaStream_t st);
qw_status rope_frequencies(int32_t method, double base, int32_t rot, double factor, double original,
                           double low, double high, double* freqs, float* attention);

// MoE scheduling.
qw_status launch_moe_route(const float* logits, int32_t T, int32_t E, int32_t topk,
                           int32_t* topk_ids, int32_t* sorted_pairs, int32_t* offsets, void* ws,
                           uint64_t ws_bytes, int32_t* err, cudaStream_t st);
uint64_t moe_route_workspace(int32_t T, int32_t E, int32_t topk);
qw_status launch_moe_permute(int32_t afmt, const void* A, const void* A_sf, int32_t K,
                             const int32_t* sorted_pairs, int64_t P, int32_t topk,
                             void* A_sorted, void* A_sf_sorted, cudaStream_t st);

// Device tile queue for grouped GEMMs: entry = (expert, row_begin, row_end) for each
// tile of `tile_rows` rows of every expert; count at queue[0].
uint64_t tile_queue_bytes(int32_t E, int64_t rows, int32_t tile_rows);
// Offsets outside [0, total_rows] or decreasing are reported (QW_ERR_INVALID_ARG) and
// produce no tiles.
qw_status launch_build_tile_queue(const int32_t* offsets, int32_t E, int32_t tile_rows,
                                  int64_t total_rows, int32_t* queue, int64_t max_entries,
                                  int32_t* err, cudaStream_t st);

qw_status launch_wait_timeout_probe(int32_t* err, int64_t limit_ns, cudaStream_t st);
// Diagnostics: a plain streaming read of `bytes` at `src` (one fold word per CTA to `sink`).
qw_status launch_stream_read(const void* src, uint64_t bytes, uint32_t* sink, bool chained,
                             cudaStream_t st);
// Diagnostics: the tcgen05 MMA issue rate (qw_mma_rate_probe; arguments checked there).
qw_status launch_mma_probe(int mode, int n, int iters, uint64_t* out, int32_t* err,
                           cudaStream_t st);

}  // namespace qw
