// logprobs.cu - what a server answers with once it has logits: the log probability and rank of
// a given token, the entropy and the top alternatives of each row, in one pass over the row.
//
// Mathematics.  In base 2, with y = x log2(e) - r for a running reference r (the largest x so far
// times log2(e), rounded): s = sum 2^y and t = sum 2^y y.  A new reference r' rescales
// t <- 2^(r-r') (t + s (r - r')), s <- 2^(r-r') s, which also merges the partial sums of threads,
// warps and CTAs.  Then log p(x) = ln2 (x log2(e) - r - log2 s) and the entropy is
// ln2 (log2 s - t / s).  r's own rounding cancels there, but it is part of every y: half a unit of r,
// which is 2 at |x| = 2^25 and would leave 2^y nothing (or infinity) from about 2^31 on.  So sums leave
// out what is below LOW, and a row whose largest logit is far from 0 (2^24 and more) is summed once
// more, against that logit itself.
//
// Alternatives: ids are ordered by a 64-bit key (the value's bits as an ordered integer above the
// complement of the id), so ties need no second pass.  While the row streams by, a thread only notes
// the largest logit of its vectors of each block (rounded up to 16 bits).  At the end the topk-th
// largest of 64 sets of threads' maxima bounds the topk-th key from below (topk different logits are
// at least that); what reaches it, about topk threads' vectors of some block, is listed and read
// once more, from L2, a vector to a thread, and the logits at or above the bound are ranked.  Where
// very many reach it (rows of ties), the bound rises to the topk-th key of a full buffer until what
// is left fits.
// (Offering while streaming - a bound that rises, a buffer, cuts of it - left 4096 x 131072 BF16 with
// 20 alternatives at 264 us: the candidates' latency stood in the stream's way.  Reading again whole
// quarters of a thread's blocks: 304 us.)
//
// Bound: the row is read once (HBM); the work per logit is one exponential and about nine
// instructions.  A CTA of 256 threads takes a row through a ring of bulk-copied blocks in shared
// memory.  Few long rows are split over the CTAs of a cluster, whose rank 0 merges the partial
// results through distributed shared memory in a fixed order; many short ones go to CTAs of 128 or
// 64 threads.  (4096 x 131072 BF16 with 20 alternatives: 190 us = 0.83 of the copy rate; without
// alternatives 161 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qw_common.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

constexpr int RV = 4;               // vectors of a thread per block
constexpr int CAP = 512;            // candidate buffer
constexpr int SETS = 64;            // sets of threads whose largest logits bound the k-th
constexpr int HITS = 512;           // of them that the bound lets through to the list
constexpr int VHITS = 256;          // ... and of their vectors
constexpr int MAX_CLUSTER = 8;
constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

// Per element type: VE, values per 16-byte vector; LOW: sums skip vectors whose maximum is not above it,
// and unpack_floored raises smaller values to it (FP16: to the lowest finite one), so that 0 * y never is
// 0 * inf; ROW_LOW, ROW_HIGH: the sums stand if the row's maximum is above the one and not above the other
// (next to such a maximum everything at or below LOW is zero), else the row is summed against its maximum.
template <int TYPE>
struct El;
template <>
struct El<QW_T_F32> {
  static constexpr int VE = 4;
  static constexpr float LOW = -0x1p25f, ROW_LOW = -0x1p24f, ROW_HIGH = 0x1p24f;
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return static_cast<const float*>(p)[i];
  }
  static __device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float vmax(const uint4& v, const uint4& w) {
    return max_nan(vmax(v), vmax(w));
  }
  static __device__ __forceinline__ uint4 masked() {  // a vector of -inf
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void unpack_floored(const uint4& v, float (&x)[4]) {
    unpack(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaxf(x[i], LOW);
  }
  // counters of values at or above t, kept per thread and read out once per block
  using Count = int;
  static __device__ __forceinline__ void count(const uint4& v, float t, Count& c) {
    float x[4];
    unpack(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) c += x[i] >= t;
  }
  static __device__ __forceinline__ int total(Count c) { return c; }
  // the next value of the type above x
  static __device__ __forceinline__ float next_up(float x) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float(x == 0.f ? 1u : (b & 0x80000000u) ? b - 1 : b + 1);
  }
};

__device__ __forceinline__ uint32_t as_u32(const __nv_bfloat162& h) {
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t as_u32(const __half2& h) {
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the two 16-bit types: H2 their packed pair
template <class H2>
struct Pair;
template <>
struct Pair<__nv_bfloat162> {
  static __device__ __forceinline__ __nv_bfloat162 splat(float x) { return __float2bfloat162_rn(x); }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
};
template <>
struct Pair<__half2> {
  static __device__ __forceinline__ __half2 splat(float x) { return __float2half2_rn(x); }
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
};

template <class H2>
struct El16 {
  static constexpr int VE = 8;
  static __device__ __forceinline__ H2 pair(uint32_t w) { return *reinterpret_cast<const H2*>(&w); }
  static __device__ __forceinline__ H2 pmax(const uint4& v) {
    return __hmax2_nan(__hmax2_nan(pair(v.x), pair(v.y)), __hmax2_nan(pair(v.z), pair(v.w)));
  }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    const uint32_t m = as_u32(pmax(v));
    return El<QW_T_F32>::max_nan(Pair<H2>::lo(m), Pair<H2>::hi(m));
  }
  static __device__ __forceinline__ float vmax(const uint4& v, const uint4& w) {
    const uint32_t m = as_u32(__hmax2_nan(pmax(v), pmax(w)));
    return El<QW_T_F32>::max_nan(Pair<H2>::lo(m), Pair<H2>::hi(m));
  }
  static __device__ __forceinline__ uint4 masked() {  // a vector of -inf
    const uint32_t m = as_u32(Pair<H2>::splat(-INFINITY));
    return make_uint4(m, m, m, m);
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = Pair<H2>::lo(w[i]);
      x[2 * i + 1] = Pair<H2>::hi(w[i]);
    }
  }
  static __device__ __forceinline__ void unpack_floored(const uint4& v, float floor, float (&x)[8]) {
    const H2 f = Pair<H2>::splat(floor);
    unpack(make_uint4(as_u32(__hmax2(pair(v.x), f)), as_u32(__hmax2(pair(v.y), f)),
                      as_u32(__hmax2(pair(v.z), f)), as_u32(__hmax2(pair(v.w), f))),
           x);
  }
  // 1.0 or 0.0 added in each half: exact, as at most 4 RV are added between two read-outs
  using Count = H2;
  static __device__ __forceinline__ void count(const uint4& v, float t, Count& c) {
    const H2 tt = Pair<H2>::splat(t);  // t is a value of the type: exact
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __hadd2(c, __hge2(pair(w[i]), tt));
  }
  static __device__ __forceinline__ int total(const Count& c) {
    return (int)(Pair<H2>::lo(as_u32(c)) + Pair<H2>::hi(as_u32(c)));
  }
  static __device__ __forceinline__ float next_up(float x) {
    uint32_t b = as_u32(Pair<H2>::splat(x)) & 0xFFFFu;
    b = x == 0.f ? 1u : (b & 0x8000u) ? b - 1 : b + 1;
    return Pair<H2>::lo(b);
  }
};
template <>
struct El<QW_T_BF16> : El16<__nv_bfloat162> {
  static constexpr float LOW = -0x1p25f, ROW_LOW = -0x1p24f, ROW_HIGH = 0x1p24f;
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static __device__ __forceinline__ void unpack_floored(const uint4& v, float (&x)[8]) {
    El16<__nv_bfloat162>::unpack_floored(v, LOW, x);
  }
};
template <>
struct El<QW_T_F16> : El16<__half2> {
  // FP16 values next to it are 32 apart
  static constexpr float LOW = -60000.f, ROW_LOW = LOW, ROW_HIGH = 65504.f;
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
  static __device__ __forceinline__ void unpack_floored(const uint4& v, float (&x)[8]) {
    El16<__half2>::unpack_floored(v, -65504.f, x);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Order of the alternatives as one integer: larger value first, equal values by the lower id.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(float x, int32_t id) {
  return ((uint64_t)order_of(x) << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

// Partial result of some of a row's logits.
struct Part {
  float rmax;  // largest logit
  float r, s, t;
  int32_t above;
  int32_t bad;
  int32_t n;  // entries of the sorted list
};
__device__ __forceinline__ void merge(float& r, float& s, float& t, float r2, float s2, float t2) {
  const float m = fmaxf(r, r2);
  const float f = ex2(r - m), f2 = ex2(r2 - m);
  t = f * (t + s * (r - m)) + f2 * (t2 + s2 * (r2 - m));
  s = f * s + f2 * s2;
  r = m;
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int STAGES = 2;  // blocks of vectors in shared memory
template <int THREADS>
constexpr size_t ring_bytes() {
  return (size_t)STAGES * THREADS * RV * 16;
}
// a reference is kept until a logit passes it by more than this (2^12 x 2^31 terms stay finite, 2^14 x 2^31
// with the rounding of a reference of 2^25; and the entropy, a difference of two numbers of that many
// bits, loses four of its own)
constexpr float HEADROOM = 8.f;

// BF16 bits of a number that is x or above it
__device__ __forceinline__ uint16_t bf16_above(float x) {
  const uint32_t b = __float_as_uint(x);
  return (uint16_t)(((b & 0x80000000u) ? b : b + 0xFFFFu) >> 16);
}

template <int TYPE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    logprobs_kernel(const LogprobsArgs a, const int csize) {
  using E = El<TYPE>;
  constexpr int WARPS = THREADS / 32;
  constexpr int BLOCK = THREADS * RV;               // vectors of a block
  constexpr int NOTES = THREADS == 256 ? 32 : THREADS == 128 ? 16 : 4;  // blocks (or runs) noted
  constexpr int VE = E::VE;
  constexpr int ES = 16 / VE;
  extern __shared__ __align__(128) uint4 ring[];  // [STAGES][BLOCK]
  __shared__ __align__(16) uint64_t buf[CAP];
  __shared__ uint64_t sorted[kLogprobsMaxTop];
  __shared__ int cnt, merged;
  __shared__ uint32_t largest[THREADS];  // of each thread's logits, by their order
  __shared__ uint32_t kth;
  __shared__ uint16_t note[NOTES][THREADS];  // upper bounds (BF16 bits) of a thread's maxima
  __shared__ uint16_t list[HITS];            // note x THREADS + thread
  __shared__ int32_t vlist[VHITS];           // vectors of the row
  __shared__ int hits, vhits;
  __shared__ Part wpart[WARPS];
  __shared__ Part part;  // this CTA's result; on rank 0, at the end, the row's
  __shared__ uint64_t full[STAGES];
  __shared__ int abort_flag, failed;  // failed: the block whose wait gave up

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    cnt = merged = hits = vhits = 0;
    abort_flag = 0;
    failed = 0x7FFFFFFF;
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t row = blockIdx.x / (unsigned)csize;
  const int rank = (int)(blockIdx.x % (unsigned)csize);
  const int64_t off = row * a.ld;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + off * ES;
  const int k = a.topk;

  // 16-byte vectors of the row, and the logits before and after them
  const int head = min((int)(((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / ES), a.V);
  const int nv = (a.V - head) / VE;
  const int tail = a.V - head - nv * VE;
  const uint4* vec = reinterpret_cast<const uint4*>(base + (int64_t)head * ES);
  // this CTA's: whole blocks, but for the row's end
  const int per = ((nv + BLOCK - 1) / BLOCK + csize - 1) / csize * BLOCK;
  const int vbeg = (int)min64(nv, (int64_t)rank * per), vend = min(nv, vbeg + per);
  const int nblk = (vend - vbeg + BLOCK - 1) / BLOCK;
  const int run = max(1, (nblk + NOTES - 1) / NOTES);  // blocks to a note

  auto fetch = [&](int b) {  // thread 0
    const int v = vbeg + b * BLOCK;
    const uint32_t bytes = (uint32_t)min(BLOCK, vend - v) * 16;
    mbar_arrive_expect_tx(&full[b % STAGES], bytes);
    bulk_load(ring + (b % STAGES) * BLOCK, vec + v, bytes, &full[b % STAGES]);
  };
  if (tid == 0)
    for (int b = 0; b < min(STAGES, nblk); ++b) fetch(b);

  const int32_t tok = a.tokens ? a.tokens[row] : -1;
  const bool tok_ok = tok >= 0 && tok < a.V;
  // a value above every logit counts nothing
  const bool want_rank = tok_ok && a.token_rank;
  const float xtok = tok_ok && (a.token_rank || a.token_logprob) ? E::load(base, tok) : INFINITY;
  const float xt = want_rank ? xtok : INFINITY;
  const float xt_up = want_rank ? E::next_up(xt) : INFINITY;
  // vectors with a logit before the token: equal logits count in them
  const int vlim = tok > head ? min(nv, (tok - head + VE - 1) / VE) : 0;

  // M: the logit the reference r was made from (LOW: none yet)
  float rmax = -INFINITY, M = E::LOW, r = E::LOW * LOG2E;
  uint64_t s2 = 0, t2 = 0;
  int above = 0;
  bool bad = false;
  // ... and those of the token's own vector, if it begins before the token, from the token on are
  // taken back
  if (want_rank && tid < VE && vlim > vbeg && vlim <= vend) {
    const int i = head + (vlim - 1) * VE + tid;
    above = i >= tok && E::load(base, i) == xt ? -1 : 0;
  }
  auto rise = [&](float m) {  // a new reference
    const float rn = m * LOG2E, d = r - rn, f = ex2(d);
    const uint64_t f2 = pack2(f, f);
    t2 = fma2(f2, fma2(s2, pack2(d, d), t2), 0);
    s2 = fma2(f2, s2, 0);
    M = m;
    r = rn;
  };

  // the logits beside the vectors: one a thread of rank 0
  float side = -INFINITY;
  const int32_t side_id = tid < head ? tid : a.V - tail + (tid - head);
  if (rank == 0 && tid < head + tail) {
    side = E::load(base, side_id);
    bad = !(side < INFINITY);
    rmax = side;
    if (side > E::LOW) {
      rise(side);
      const float y = fmaf(side, LOG2E, -r), e = ex2(y);  // (y: what r lost in rounding)
      s2 = pack2(e, 0.f);
      t2 = pack2(e * y, 0.f);
    }
    above += side > xt || (side == xt && side_id < tok);
  }

  float pmax = -INFINITY;  // of this thread's vectors since the last note
  int notes = 0, in_run = 0;
#pragma unroll 1
  for (int b = 0; b < nblk; ++b) {
    uint4* blk = ring + (b % STAGES) * BLOCK + tid;
    const int v0 = vbeg + b * BLOCK + tid;
    if (v0 - tid + BLOCK > vend) {  // the row's last block: masked vectors behind it
#pragma unroll
      for (int j = 0; j < RV; ++j)
        if (v0 + j * THREADS >= vend) blk[j * THREADS] = E::masked();
    }
    // (a thread reads only vectors that it filled itself or that the copy brings)
    if (!warp_wait(&full[b % STAGES], (uint32_t)(b / STAGES) & 1u, &abort_flag, a.err)) failed = b;
    typename E::Count count{};
    // all at once, so that one look at their maximum decides for all (two at a time: 4096 x 131072
    // BF16 200 us for 191)
    uint4 x4[RV];
#pragma unroll
    for (int j = 0; j < RV; ++j) x4[j] = blk[j * THREADS];
    static_assert(RV == 4);
    const float vm = El<QW_T_F32>::max_nan(E::vmax(x4[0], x4[1]), E::vmax(x4[2], x4[3]));
    pmax = fmaxf(pmax, vm);
    if (vm >= xt) {  // (masked vectors behind the row are not above anything)
#pragma unroll
      for (int j = 0; j < RV; ++j) E::count(x4[j], v0 + j * THREADS < vlim ? xt : xt_up, count);
    }
    if (!(vm < (M == E::LOW ? E::LOW : M + HEADROOM))) {
      bad = bad || !(vm < INFINITY);
      if (vm > E::LOW) rise(vm);
    }
    if (vm > E::LOW) {
      const uint64_t l2 = pack2(LOG2E, LOG2E), nr = pack2(-r, -r);
#pragma unroll
      for (int j = 0; j < RV; ++j) {
        float x[VE];
        E::unpack_floored(x4[j], x);
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          const uint64_t y = fma2(pack2(x[i], x[i + 1]), l2, nr);
          const float2 yy = unpack2(y);
          const uint64_t e = pack2(ex2(yy.x), ex2(yy.y));
          s2 = add2(s2, e);
          t2 = fma2(e, y, t2);
        }
      }
    }
    if (want_rank) above += E::total(count);
    if (k > 0 && (++in_run == run || b + 1 == nblk)) {
      note[notes++][tid] = bf16_above(pmax);
      rmax = fmaxf(rmax, pmax);
      pmax = -INFINITY;
      in_run = 0;
    }
    __syncthreads();  // every thread is done with the block
    // (not abort_flag: a warp ahead may raise it for the next block before all have looked here, and
    // the barriers that follow want all threads)
    if (failed <= b) {
      // a wait gave up: let the copies in flight land before shared memory goes away
      for (int i = b; tid == 0 && i < min(nblk, b + STAGES); ++i)
        wait_landed(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
      break;
    }
    if (tid == 0 && b + STAGES < nblk) fetch(b + STAGES);
  }

  rmax = fmaxf(rmax, pmax);

  // the k largest of the buffer's n keys to `sorted`, in order
  auto rank_keys = [&](int n) {
    const ulonglong2* two = reinterpret_cast<const ulonglong2*>(buf);
    for (int i = tid; i < n; i += THREADS) {
      const uint64_t key = buf[i];
      int before = (n & 1) && buf[n - 1] > key;
#pragma unroll 8
      for (int j = 0; j < n / 2; ++j) {
        const ulonglong2 q = two[j];
        before += (q.x > key) + (q.y > key);
      }
      if (before < k) sorted[before] = key;
    }
  };

  int settled = 0;  // keys in `sorted`
  if (k > 0) {
    // lower bound of the k-th key, and its value; -inf is never offered (the masked ids that
    // follow are added at the end)
    constexpr float kLowest = -3.4028234663852886e38f;
    uint64_t thr = (uint64_t)order_of(kLowest) << 32;
    float thr_x = kLowest;
    {
      // The k-th largest of the maxima of 64 sets of threads (the logits beside the vectors may be
      // among them: they are offered too).  A warp has all of them, two a lane, and looks at eight.
      // (32 sets leave k / 32 of them below the bound's set: with k = 32 the bound was the least of
      // all and let 200 logits and more through.  Sets of threads that lie 64 apart have logits of
      // their own even where a row has few vectors.)
      largest[tid] = order_of(rmax);
      __syncthreads();
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < THREADS; i += SETS) {
        lo = max(lo, largest[i + lane]);
        hi = max(hi, largest[i + 32 + lane]);
      }
      static_assert(SETS == 64 && SETS / WARPS * WARPS == SETS && kLogprobsMaxTop <= SETS);
#pragma unroll
      for (int i = 0; i < SETS / WARPS; ++i) {
        const int at = warp * (SETS / WARPS) + i;  // a set; equal ones in this order
        const uint32_t v = __shfl_sync(0xFFFFFFFFu, at < 32 ? lo : hi, at & 31);
        const int before = __popc(__ballot_sync(0xFFFFFFFFu, lo > v || (lo == v && lane < at))) +
                           __popc(__ballot_sync(0xFFFFFFFFu, hi > v || (hi == v && lane + 32 < at)));
        if (before == k - 1 && lane == 0) kth = v;
      }
      __syncthreads();
      const uint64_t key = (uint64_t)kth << 32;
      if (key > thr) {
        thr = key;
        thr_x = value_of(key);
      }
    }
    bool lost = false;
    auto offer = [&](float x, int32_t id) {
      if (!(x >= thr_x)) return;
      const uint64_t key = order_key(x, id);
      if (key < thr) return;
      int pos = *(volatile int*)&cnt;  // (a full buffer costs a read, not an atomic)
      if (pos < CAP) pos = atomicAdd(&cnt, 1);
      if (pos < CAP)
        buf[pos] = key;
      else
        lost = true;
    };
#pragma unroll 4
    for (int i = 0; i < notes; ++i)
      if (__uint_as_float((uint32_t)note[i][tid] << 16) >= thr_x) {
        const int pos = atomicAdd(&hits, 1);
        if (pos < HITS) list[pos] = (uint16_t)(i * THREADS + tid);
      }
    __syncthreads();
    // the last blocks are still in the ring
    auto place = [&](int gb, int v) {
      return gb + STAGES >= nblk ? ring + gb % STAGES * BLOCK + (v - vbeg - gb * BLOCK) : vec + v;
    };
    const int listed = hits;
    if (listed <= HITS) {
      for (int b = 0; b < run; ++b)
        for (int i = tid; i < listed * RV; i += THREADS) {
          const int e = list[i / RV], gb = e / THREADS * run + b;
          const int v = vbeg + gb * BLOCK + i % RV * THREADS + e % THREADS;
          if (gb >= nblk || v >= vend || !(E::vmax(*place(gb, v)) >= thr_x)) continue;
          const int pos = atomicAdd(&vhits, 1);
          if (pos < VHITS) vlist[pos] = v;
        }
    }
    __syncthreads();
    const bool few = listed <= HITS && vhits <= VHITS;
    const int found = vhits;
    for (;;) {
      if (side > -INFINITY) offer(side, side_id);
      if (few) {
        // a logit to a thread (a vector to a thread: few of them work, and long)
        for (int i = tid; i < found * VE; i += THREADS) {
          const int v = vlist[i / VE];
          offer(E::load(place((v - vbeg) / BLOCK, v), i % VE), head + v * VE + i % VE);
        }
      } else {
        for (int64_t i = head + vbeg * VE + tid; i < head + vend * VE; i += THREADS)
          offer(E::load(base, i), (int32_t)i);
      }
      const bool again = __syncthreads_or(lost);
      const int n = min(cnt, CAP);
      rank_keys(n);
      __syncthreads();
      settled = min(n, k);
      if (!again) break;
      // overflow: the k-th of CAP keys is a bound above the last one
      thr = sorted[k - 1];
      thr_x = value_of(thr);
      lost = false;
      if (tid == 0) cnt = 0;
      __syncthreads();
    }
  }

  // threads -> warps -> the CTA
  const float2 ss = unpack2(s2), tt = unpack2(t2);
  float s = ss.x + ss.y, t = tt.x + tt.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float r_o = __shfl_xor_sync(0xFFFFFFFFu, r, o), s_o = __shfl_xor_sync(0xFFFFFFFFu, s, o),
                t_o = __shfl_xor_sync(0xFFFFFFFFu, t, o);
    merge(r, s, t, r_o, s_o, t_o);
    rmax = fmaxf(rmax, __shfl_xor_sync(0xFFFFFFFFu, rmax, o));
    above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane == 0) wpart[warp] = Part{rmax, r, s, t, above, bad ? 1 : 0, 0};
  __syncthreads();
  // lane w of a warp has part w (and every WARPS-th lane the same again)
  auto merge_parts = [&](Part p, int n) {
    for (int o = 1; o < n; o <<= 1) {
      merge(p.r, p.s, p.t, __shfl_xor_sync(0xFFFFFFFFu, p.r, o),
            __shfl_xor_sync(0xFFFFFFFFu, p.s, o), __shfl_xor_sync(0xFFFFFFFFu, p.t, o));
      p.rmax = fmaxf(p.rmax, __shfl_xor_sync(0xFFFFFFFFu, p.rmax, o));
      p.above += __shfl_xor_sync(0xFFFFFFFFu, p.above, o);
      p.bad |= __shfl_xor_sync(0xFFFFFFFFu, p.bad, o);
    }
    return p;
  };
  if (warp == 0) {
    Part p = merge_parts(wpart[lane % WARPS], WARPS);
    p.n = settled;
    if (lane == 0) part = p;
  }
  if (THREADS == 256 && csize > 1) {
    cluster_sync();  // every CTA's part and list are written
    if (rank != 0) {
      cluster_sync();  // rank 0 has read
      return;
    }
    // Everything of the others is asked for at once: lane c has CTA c's part, and (sorted lists) warp
    // c CTA c's keys.  Two bounds leave few of them: a CTA's k-th key, and the least of the CTAs'
    // m-th, m x csize >= k.
    static_assert(kLogprobsMaxTop <= 32 && (MAX_CLUSTER <= WARPS || THREADS < 256),
                  "a warp per list");
    const int c = lane & (csize - 1), m = (k + csize - 1) / csize;
    const uint32_t q = mapa_shared(smem_u32(&part), (uint32_t)c);
    const int n_c = (int)ld_cluster_u32(q + offsetof(Part, n));
    Part p{ld_shared_cluster_f32(q + offsetof(Part, rmax)),
           ld_shared_cluster_f32(q + offsetof(Part, r)),
           ld_shared_cluster_f32(q + offsetof(Part, s)),
           ld_shared_cluster_f32(q + offsetof(Part, t)),
           (int32_t)ld_cluster_u32(q + offsetof(Part, above)),
           (int32_t)ld_cluster_u32(q + offsetof(Part, bad)),
           0};
    if (k > 0) {
      const uint32_t list = mapa_shared(smem_u32(sorted), (uint32_t)c);
      uint64_t kth = ld_cluster_u64(list + 8 * (k - 1)), mth = ld_cluster_u64(list + 8 * (m - 1));
      const uint64_t key = ld_cluster_u64(
          mapa_shared(smem_u32(sorted), (uint32_t)min(warp, csize - 1)) + 8 * min(lane, k - 1));
      kth = n_c >= k ? kth : 0;  // (what lies past a list's end is anything)
      mth = n_c >= m ? mth : 0;
      for (int o = 1; o < csize; o <<= 1) {
        kth = max(kth, __shfl_xor_sync(0xFFFFFFFFu, kth, o));
        mth = min(mth, __shfl_xor_sync(0xFFFFFFFFu, mth, o));
      }
      if (lane < __shfl_sync(0xFFFFFFFFu, n_c, warp) && warp < csize && key >= max(kth, mth))
        buf[atomicAdd(&merged, 1)] = key;
    }
    if (warp == 0) p = merge_parts(p, csize);
    cluster_arrive();  // this thread has read (the wait is at the end)
    __syncthreads();
    if (tid == 0) part = p;
    const int n = merged;
    rank_keys(n);
    settled = min(n, k);
  }
  __syncthreads();

  const Part p = part;
  const bool none = p.rmax == -INFINITY;
  const bool far = !none && !p.bad && (p.rmax <= E::ROW_LOW || p.rmax > E::ROW_HIGH);
  const float ref = p.r;
  float l2s = log2f(p.s), ent = (l2s - p.t / p.s) * LN2;
  if (far) {
    // (in slow motion: rows like this are masked ones, or broken)
    float sl = 0.f, tl = 0.f;
    for (int64_t i = tid; i < a.V; i += THREADS) {
      const float y = fmaxf((E::load(base, i) - p.rmax) * LOG2E, -1e4f), e = ex2(y);
      sl += e;
      tl += e * y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sl += __shfl_xor_sync(0xFFFFFFFFu, sl, o);
      tl += __shfl_xor_sync(0xFFFFFFFFu, tl, o);
    }
    if (lane == 0) {
      wpart[warp].s = sl;
      wpart[warp].t = tl;
    }
    __syncthreads();
    sl = tl = 0.f;
    for (int w = 0; w < WARPS; ++w) {
      sl += wpart[w].s;
      tl += wpart[w].t;
    }
    l2s = log2f(sl);
    ent = (l2s - tl / sl) * LN2;
  }
  const float nan = __uint_as_float(0x7FC00000u);
  auto logp = [&](float x) {
    if (p.bad) return nan;
    if (none) return -INFINITY;
    if (far) return (x - p.rmax) - l2s * LN2;
    if (x < -1e30f) return x - p.rmax;  // x log2(e) may overflow; log s is lost beside it
    return (fmaf(x, LOG2E, -ref) - l2s) * LN2;
  };
  if (tid == 0) {
    if (p.bad) set_error(a.err, QW_ERR_VALUE);
    if (a.tokens && !tok_ok) set_error(a.err, QW_ERR_INVALID_ARG);
    if (a.token_logprob) a.token_logprob[row] = tok_ok ? logp(xtok) : nan;
    if (a.token_rank) a.token_rank[row] = tok_ok ? 1 + p.above : 0;
    if (a.entropy) a.entropy[row] = p.bad ? nan : none ? 0.f : ent;
  }
  if (tid == 0) cnt = settled;
  if (k > settled && warp == 0) {
    // fewer ids than asked for are left by the mask: the masked ones follow in id order
    int n = settled;
    for (int64_t i0 = 0; i0 < a.V && n < k; i0 += 32) {
      const bool gone = i0 + lane < a.V && E::load(base, i0 + lane) == -INFINITY;
      const uint32_t set = __ballot_sync(0xFFFFFFFFu, gone);
      const int at = n + __popc(set & ((1u << lane) - 1u));
      if (gone && at < k) sorted[at] = order_key(-INFINITY, (int32_t)i0 + lane);
      n += __popc(set);
      if (lane == 0) cnt = min(n, k);
    }
  }
  if (k > settled) __syncthreads();
  if (tid < k) {
    // (a row with NaN may not have that many: what is missing names id 0)
    const uint64_t key = tid < (k > settled ? cnt : settled) ? sorted[tid] : 0xFFFFFFFFull;
    a.top_ids[row * k + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
    a.top_logprobs[row * k + tid] = logp(value_of(key));
  }
  if (THREADS == 256 && csize > 1) {
    __syncwarp();
    cluster_wait();
  }
}

template <int TYPE, int THREADS>
qw_status launch_type(const LogprobsArgs& a, int64_t T, int csize, cudaStream_t st) {
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [] {
        return cudaFuncSetAttribute(logprobs_kernel<TYPE, THREADS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)ring_bytes<THREADS>()) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.dynamicSmemBytes = ring_bytes<THREADS>();
  cfg.gridDim = dim3((unsigned)(T * csize));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE, THREADS>, a, csize) == cudaSuccess ? QW_OK
                                                                                   : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_logprobs(const LogprobsArgs& a, int32_t type, int64_t T, cudaStream_t st) {
  // CTAs to a row: while there are fewer than SMs and each keeps 8192 logits.  (What a CTA does besides
  // reading costs more than splitting further gives: 64 x 32003 FP32 8.6 us, 11.3 with 4096 logits each;
  // 64 x 131072 BF16 11.1 us, 13.7 with two CTAs per SM; 777 x 50021 FP16 28.6 us with one CTA a row,
  // 40.9 with two towards even rounds of the four CTAs that fit an SM.)
  int csize = 1;
  while (csize < MAX_CLUSTER && T * csize < device_sm_count() && a.V / csize > 8192) csize *= 2;
  // Many rows: smaller CTAs, so that more rows are under way and one's ends hide under others' middles
  // (us with 256, 128 and 64 threads: 4000 x 2000 BF16 42, 28, 24; 4000 x 8000 BF16 43, 35, 35;
  // 4000 x 50021 FP16 98, 85; but 777 x 50021 27.0, 28.6; 1000 x 131072 BF16 54, 58; 2048 x 131072 FP32
  // 174, 178).
  const int64_t vectors = (int64_t)a.V * (type == QW_T_F32 ? 4 : 2) / 16, sms = device_sm_count();
  const int threads = T <= 4 * sms                                             ? 256
                      : vectors <= 256                                         ? 64
                      : vectors <= 1024 || (vectors <= 6400 && T > 8 * sms) ? 128
                                                                               : 256;
  auto go = [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    return threads == 256   ? launch_type<TYPE, 256>(a, T, csize, st)
           : threads == 128 ? launch_type<TYPE, 128>(a, T, 1, st)
                            : launch_type<TYPE, 64>(a, T, 1, st);
  };
  if (type == QW_T_F32) return go(std::integral_constant<int, QW_T_F32>{});
  if (type == QW_T_F16) return go(std::integral_constant<int, QW_T_F16>{});
  return go(std::integral_constant<int, QW_T_BF16>{});
}

}  // namespace qw
