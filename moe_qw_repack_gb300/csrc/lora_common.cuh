// lora_common.cuh - what the adapters' two kernels share.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ float bf16_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// the first `n` of eight BF16 values, zeros behind them (what lies there may be anything)
__device__ __forceinline__ uint4 first_of(uint4 v, int n) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = n >= 2 * j + 2 ? w[j] : n == 2 * j + 1 ? w[j] & 0xFFFFu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The next of the BF16 numbers that t is held as: t rounded, but none above BF16's largest number for a finite
// t (the numbers after it have the rest; the last one gets what is infinite or NaN).
__device__ __forceinline__ __nv_bfloat16 next_part(float t, bool last) {
  constexpr float TOP = 0x1.FEp127f;
  return __float2bfloat16_rn(last ? t : fminf(fmaxf(t, -TOP), TOP));
}

// A token's adapter and rank: -1 where it has none, or none that works (which sets the error).
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int64_t m, int& rank) {
  const int id = p.ids[m];
  rank = id >= 0 && id < p.L ? (p.ranks ? p.ranks[id] : p.R) : 0;
  if (id < -1 || id >= p.L || rank < 0 || rank > p.R) {
    set_error(p.err, QW_ERR_INVALID_ARG);
    rank = 0;
  }
  return rank > 0 ? id : -1;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Rows without adapter: base's bits.
template <bool C32>
__device__ __forceinline__ void copy_row(const LoraArgs& p, bool wide, int64_t m, int32_t n0, int32_t n1) {
  using T = std::conditional_t<C32, uint32_t, uint16_t>;
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const T* b = p.base ? static_cast<const T*>(p.base) + m * p.ld_base : nullptr;
  T* c = static_cast<T*>(p.C) + m * p.ldc;
  int32_t n = n0;
  if (wide) {  // (eight pieces under way: with one, 512 such rows took 75 us)
    const int32_t end = n0 + (n1 - n0) / V * V;
    for (n += lane * V; n < end; n += 8 * 32 * V) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = b && n + i * 32 * V < end ? *reinterpret_cast<const uint4*>(b + n + i * 32 * V) : zero4();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i * 32 * V < end) *reinterpret_cast<uint4*>(c + n + i * 32 * V) = x[i];
    }
    n = end;
  }
  for (n += lane; n < n1; n += 8 * 32) {
    T x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = b && n + i * 32 < n1 ? b[n + i * 32] : (T)0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i * 32 < n1) c[n + i * 32] = x[i];
  }
}

// Whether base and C take 16-byte accesses.
inline bool lora_wide(const LoraArgs& a, bool c_f32) {
  const int vec = c_f32 ? 4 : 8;
  return ((uintptr_t)a.C | (uintptr_t)a.base) % 16 == 0 && a.ldc % vec == 0 && (!a.base || a.ld_base % vec == 0);
}

}  // namespace qw
