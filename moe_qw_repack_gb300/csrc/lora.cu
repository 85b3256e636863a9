// lora.cu - low-rank adapters of many requests beside a shared projection.
//
//   C[m][n] = base[m][n] + s_a sum_{r < rank_a} B_a[n][r] (sum_k A_a[r][k] X[m][k]),  a = ids[m]
#include <cuda_bf16.h>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

constexpr int THREADS = 256;

// One CTA per token: a warp a row of A at a time, then a thread a row of B at a time.
template <bool C32>
__global__ void __launch_bounds__(THREADS) lora_kernel(const LoraArgs p) {
  __shared__ float low[kLoraMaxRank];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t m = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int id = p.ids[m];
  int rank = 0;
  if (id >= 0 && id < p.L) {
    rank = p.ranks ? p.ranks[id] : p.R;
    if (rank < 0 || rank > p.R) rank = 0, set_error(p.err, QW_ERR_INVALID_ARG);
  } else if (id != -1) {
    set_error(p.err, QW_ERR_INVALID_ARG);
  }
  const float scale = rank > 0 && p.scales ? p.scales[id] : 1.f;
  for (int r = warp; r < rank; r += THREADS / 32) {
    const uint4* a = reinterpret_cast<const uint4*>(p.A + ((int64_t)id * p.R + r) * p.K);
    const uint4* x = reinterpret_cast<const uint4*>(p.X + m * p.ldx);
    float s = 0.f;
    for (int k = lane; k < p.K / 8; k += 32) {
      const uint4 u = a[k], v = x[k];
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s = fmaf(bf16_lo(uw[j]), bf16_lo(vw[j]), s);
        s = fmaf(bf16_hi(uw[j]), bf16_hi(vw[j]), s);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) low[r] = s * scale;
  }
  __syncthreads();
  for (int n = threadIdx.x; n < p.N; n += THREADS) {
    float s = 0.f;
    if (rank > 0) {
      const uint16_t* b = p.B + ((int64_t)id * p.N + n) * p.R;
      for (int r = 0; r < rank; ++r) s = fmaf(__uint_as_float((uint32_t)b[r] << 16), low[r], s);
    }
    if constexpr (C32) {
      float* c = static_cast<float*>(p.C) + m * p.ldc + n;
      const float* o = static_cast<const float*>(p.base);
      const float v = o ? o[m * p.ld_base + n] : 0.f;
      *c = rank > 0 ? v + s : v;
    } else {
      uint16_t* c = static_cast<uint16_t*>(p.C) + m * p.ldc + n;
      const uint16_t* o = static_cast<const uint16_t*>(p.base);
      const uint16_t v = o ? o[m * p.ld_base + n] : (uint16_t)0;
      *c = rank > 0 ? __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float((uint32_t)v << 16) + s)) : v;
    }
  }
}

}  // namespace

qw_status launch_lora(const LoraArgs& a, bool c_f32, cudaStream_t st) {
  return c_f32 ? launch_pdl(lora_kernel<true>, dim3((unsigned)a.M), dim3(THREADS), 0, st, a)
               : launch_pdl(lora_kernel<false>, dim3((unsigned)a.M), dim3(THREADS), 0, st, a);
}

}  // namespace qw
