// logprobs.cu - what a server answers with once it has logits: the log probability and rank of
// a given token, the entropy and the top alternatives of each row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (TYPE == QW_T_F32) return static_cast<const float*>(p)[i];
  if constexpr (TYPE == QW_T_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Order of the alternatives as one integer: larger value first, equal values by the lower id.
__device__ __forceinline__ uint64_t order_key(float x, int32_t id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)o << 32) | (0xFFFFFFFFu - (uint32_t)id);
}

template <class T, class F>
__device__ T block_reduce(T v, F f, T* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (unsigned i = 1; i < blockDim.x / 32; ++i) v = f(v, sh[i]);
  return v;
}

template <int TYPE>
__global__ void __launch_bounds__(512) logprobs_kernel(const LogprobsArgs a) {
  __shared__ float shf[32];
  __shared__ unsigned long long shk[32];
  const int64_t row = blockIdx.x;
  const int64_t off = row * a.ld;
  auto maxf = [](float x, float y) { return fmaxf(x, y); };
  auto addf = [](float x, float y) { return x + y; };
  float m = -INFINITY;
  bool bad = false;
  for (int32_t i = threadIdx.x; i < a.V; i += blockDim.x) {
    const float x = load_logit<TYPE>(a.logits, off + i);
    bad = bad || !(x < INFINITY);
    m = fmaxf(m, x);
  }
  bad = __syncthreads_or(bad);
  m = block_reduce(m, maxf, shf);
  const bool none = m == -INFINITY;
  const int32_t tok = a.tokens ? a.tokens[row] : -1;
  const bool tok_ok = tok >= 0 && tok < a.V;
  const float xt = tok_ok ? load_logit<TYPE>(a.logits, off + tok) : 0.f;
  float s = 0.f, t = 0.f, above = 0.f;
  for (int32_t i = threadIdx.x; i < a.V; i += blockDim.x) {
    const float x = load_logit<TYPE>(a.logits, off + i);
    const float d = fmaxf(x - m, -1e4f);
    const float e = expf(d);
    s += e;
    t += e * d;
    above += (x > xt || (x == xt && i < tok)) ? 1.f : 0.f;
  }
  s = block_reduce(s, addf, shf);
  t = block_reduce(t, addf, shf);
  above = block_reduce(above, addf, shf);
  const float ls = logf(s);
  const float nan = __uint_as_float(0x7FC00000u);
  auto logp = [&](float x) { return bad ? nan : none ? -INFINITY : (x - m) - ls; };
  if (threadIdx.x == 0) {
    if (bad) set_error(a.err, QW_ERR_VALUE);
    if (a.tokens && !tok_ok) set_error(a.err, QW_ERR_INVALID_ARG);
    if (a.token_logprob) a.token_logprob[row] = tok_ok ? logp(xt) : nan;
    if (a.token_rank) a.token_rank[row] = tok_ok ? 1 + (int32_t)above : 0;
    if (a.entropy) a.entropy[row] = bad ? nan : none ? 0.f : ls - t / s;
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.topk; ++j) {
    unsigned long long best = 0;
    for (int32_t i = threadIdx.x; i < a.V; i += blockDim.x) {
      const unsigned long long k = order_key(load_logit<TYPE>(a.logits, off + i), i);
      if (k < last && k > best) best = k;
    }
    best = block_reduce(best, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; }, shk);
    last = best;
    if (threadIdx.x == 0) {
      const int32_t id = (int32_t)(0xFFFFFFFFu - (uint32_t)best);
      a.top_ids[row * a.topk + j] = id;
      a.top_logprobs[row * a.topk + j] = logp(load_logit<TYPE>(a.logits, off + id));
    }
  }
}

}  // namespace

qw_status launch_logprobs(const LogprobsArgs& a, int32_t type, int64_t T, cudaStream_t st) {
  const dim3 grid((unsigned)T);
  if (type == QW_T_F32)
    logprobs_kernel<QW_T_F32><<<grid, 512, 0, st>>>(a);
  else if (type == QW_T_F16)
    logprobs_kernel<QW_T_F16><<<grid, 512, 0, st>>>(a);
  else
    logprobs_kernel<QW_T_BF16><<<grid, 512, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace qw
