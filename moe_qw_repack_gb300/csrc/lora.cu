// lora.cu - low-rank adapters of many requests beside a shared projection, on mma.sync.
//
//   C[m][n] = base[m][n] + s_a sum_{r < rank_a} B_a[n][r] t[m][r],  t[m][r] = sum_k A_a[r][k] X[m][k],
//   a = ids[m]
//
// One launch.  A tile is 64 tokens; the tokens of one adapter in it (a group, wherever they stand) go
// through the adapter's weights together, 8 NT at a time, as the 8-column operand of m16n8k16 MMAs with
// the weights' rows as the other: a lone token costs its adapter's bytes and little else.  A group is
// worked on by a cluster: its CTAs take slices of K for t, leave them in shared memory, add them up in
// rank order, and take slices of N for the second product.  So t never leaves the SMs.
// t is held as a sum of BF16 numbers for the second product: two for BF16 results (2^-17 t is lost
// of what the result rounds to 2^-9), three for FP32 ones (all 24 bits).
// The order of k and r within an MMA is free as long as both operands have the same: a lane reads 16
// bytes of a row at once, two MMAs' share.  In the second product row 8 g + i of 64 belongs to the lanes
// of group g, so that a lane ends with eight neighbouring columns of a token, one 16-byte access of C.
#include <algorithm>

#include "lora_common.cuh"

namespace qw {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int TM = 64;  // tokens of a tile
constexpr int BN = 64;  // columns of a warp's block in the second product

// How a call is cut up: a cluster of csize CTAs takes K in slices of k_len and, of the columns of its
// part (nsplit of them), slices of n_len.
struct Cut {
  int32_t csize, nsplit, k_len, n_len;
  bool wide;  // base and C take 16-byte accesses
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// t of one 16-row block of A for 8 NT tokens over 32-k chunks [c0, c1) from k0, below k1.
template <int NT>
__device__ __forceinline__ void shrink_block(const uint16_t* a_lo, const uint16_t* a_hi, bool lo, bool hi,
                                             const uint16_t* const (&x)[NT], const bool (&live)[NT],
                                             int32_t k0, int32_t k1, int c0, int c1,
                                             float (&acc)[NT][4]) {
  constexpr int U = NT == 1 ? 4 : 2;
  const int t = threadIdx.x & 3;
  for (int c = c0; c < c1; c += U) {
    uint4 u[U], v[U], w[U][NT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int32_t k = k0 + 32 * (c + i) + 8 * t;
      const bool in = c + i < c1 && k < k1;
      u[i] = in && lo ? *reinterpret_cast<const uint4*>(a_lo + k) : zero4();
      v[i] = in && hi ? *reinterpret_cast<const uint4*>(a_hi + k) : zero4();
#pragma unroll
      for (int j = 0; j < NT; ++j)
        w[i][j] = in && live[j] ? *reinterpret_cast<const uint4*>(x[j] + k) : zero4();
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16(acc[j], u[i].x, v[i].x, u[i].y, v[i].y, w[i][j].x, w[i][j].y);
        mma_bf16(acc[j], u[i].z, v[i].z, u[i].w, v[i].w, w[i][j].z, w[i][j].w);
      }
  }
}

// Eight neighbouring results of a token: base + sums.
template <bool C32>
__device__ __forceinline__ void put8(const LoraArgs& p, bool wide, int64_t m, int32_t n,
                                     const float (&s)[8]) {
  if constexpr (C32) {
    const float* b = p.base ? static_cast<const float*>(p.base) + m * p.ld_base + n : nullptr;
    float* c = static_cast<float*>(p.C) + m * p.ldc + n;
    if (wide && n + 8 <= p.N) {
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
      if (b) u = reinterpret_cast<const float4*>(b)[0], v = reinterpret_cast<const float4*>(b)[1];
      reinterpret_cast<float4*>(c)[0] = make_float4(u.x + s[0], u.y + s[1], u.z + s[2], u.w + s[3]);
      reinterpret_cast<float4*>(c)[1] = make_float4(v.x + s[4], v.y + s[5], v.z + s[6], v.w + s[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < p.N) c[i] = (b ? b[i] : 0.f) + s[i];
    }
  } else {
    const uint16_t* b = p.base ? static_cast<const uint16_t*>(p.base) + m * p.ld_base + n : nullptr;
    uint16_t* c = static_cast<uint16_t*>(p.C) + m * p.ldc + n;
    if (wide && n + 8 <= p.N) {
      const uint4 u = b ? *reinterpret_cast<const uint4*>(b) : zero4();
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(__uint_as_float(w[j] << 16) + s[2 * j],
                           __uint_as_float(w[j] & 0xFFFF0000u) + s[2 * j + 1]);
      *reinterpret_cast<uint4*>(c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < p.N)
          c[i] = __bfloat16_as_ushort(__float2bfloat16_rn((b ? bf16_of(b[i]) : 0.f) + s[i]));
    }
  }
}

struct Smem {
  int rows;  // ranks, rounded up to 32
  int tokens;
  int splits;
  __host__ __device__ int pitch() const { return rows + 8; }  // BF16 numbers of a token's t
  __host__ __device__ int part_pitch() const { return tokens + 2; }
  __host__ __device__ int sum_bytes() const { return rows * tokens * 4; }
  __host__ __device__ int part_bytes() const {
    return (rows > 16 * WARPS ? rows : 16 * WARPS) * part_pitch() * 4;
  }
  __host__ __device__ int t_bytes() const { return splits * tokens * pitch() * 2; }
  __host__ __device__ int bytes() const {
    return sum_bytes() + (part_bytes() > t_bytes() ? part_bytes() : t_bytes());
  }
};

template <bool C32, int NTM>
struct Pass {
  static constexpr int NS = C32 ? 3 : 2;

  // t of this CTA's slice of K for the listed tokens, into sums[r][8 NT]
  template <int NT>
  static __device__ __forceinline__ void shrink(const LoraArgs& p, const Cut& cut, int crank, int64_t m0,
                                                int id, int rank, const uint8_t* list, int cnt,
                                                float* sums, float* part, int part_pitch) {
    constexpr int T = 8 * NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int blocks = (rank + 15) / 16;
    const int ks = blocks > 4 ? 1 : WARPS / blocks;  // warps that share a block's k
    const int32_t k0 = crank * cut.k_len, k1 = min(p.K, k0 + cut.k_len);
    const int chunks = k1 > k0 ? (k1 - k0 + 31) / 32 : 0, per = (chunks + ks - 1) / ks;
    const uint16_t* x[NT];
    bool live[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      live[j] = 8 * j + g < cnt;
      x[j] = p.X + (m0 + (live[j] ? list[8 * j + g] : 0)) * p.ldx;
    }
    const int part_of = warp / blocks;
    for (int b = ks > 1 ? warp % blocks : warp; b < blocks && part_of < ks; b += ks > 1 ? blocks : WARPS) {
      const int s = ks > 1 ? part_of : 0;
      const uint16_t* a = p.A + ((int64_t)id * p.R + 16 * b + g) * p.K;
      float acc[NT][4] = {};
      shrink_block<NT>(a, a + 8 * (int64_t)p.K, 16 * b + g < rank, 16 * b + g + 8 < rank, x, live, k0, k1,
                       s * per, min(chunks, (s + 1) * per), acc);
      float* o = part + (16 * (s * blocks + b) + g) * part_pitch + 2 * t;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        *reinterpret_cast<float2*>(o + 8 * j) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(o + 8 * part_pitch + 8 * j) = make_float2(acc[j][2], acc[j][3]);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * blocks * T; i += THREADS) {
      const int r = i / T, c = i % T;
      float v = 0.f;
      for (int s = 0; s < ks; ++s) v += part[(16 * s * blocks + r) * part_pitch + c];
      sums[i] = v;
    }
  }

  // the cluster's sums, scaled, as BF16 numbers ts[split][token][r], zeros up to a multiple of 32
  template <int NT>
  static __device__ __forceinline__ void gather(const Cut& cut, int rank, float scale, const float* sums,
                                                uint16_t* ts, int pitch) {
    constexpr int T = 8 * NT;
    const int have = (rank + 15) / 16 * 16, rows = (rank + 31) / 32 * 32;
    const uint32_t at = smem_u32(sums);
    for (int i = threadIdx.x; i < rows * T; i += THREADS) {
      const int r = i / T, c = i % T;
      float v = 0.f;
      if (r < have)
        for (int q = 0; q < cut.csize; ++q) v += ld_shared_cluster_f32(mapa_shared(at + 4 * i, q));
      v *= scale;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        ts[(s * T + c) * pitch + r] = __bfloat16_as_ushort(h);
        v -= __bfloat162float(h);
      }
    }
  }

  // base + B t for this CTA's columns
  template <int NT>
  static __device__ __forceinline__ void expand(const LoraArgs& p, const Cut& cut, int64_t m0, int id,
                                                int rank, const uint8_t* list, int cnt, int32_t n0,
                                                int32_t n1, const uint16_t* ts, int pitch) {
    constexpr int T = 8 * NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int32_t nb = n0 + warp * BN; nb < n1; nb += WARPS * BN) {
      const int32_t n = nb + 8 * g;
      const uint16_t* b = p.B + ((int64_t)id * p.N + n) * p.R + 8 * t;
      float acc[4][NT][4] = {};
      for (int r0 = 0; r0 < rank; r0 += 32) {
        const int left = rank - r0 - 8 * t;  // of this lane's eight, how many count
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = left > 0 && n + i < n1 ? *reinterpret_cast<const uint4*>(b + (int64_t)i * p.R + r0)
                                        : zero4();
        if (left < 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = first_of(w[i], left);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 v = *reinterpret_cast<const uint4*>(ts + (s * T + 8 * j + g) * pitch + r0 + 8 * t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              mma_bf16(acc[i][j], w[2 * i].x, w[2 * i + 1].x, w[2 * i].y, w[2 * i + 1].y, v.x, v.y);
              mma_bf16(acc[i][j], w[2 * i].z, w[2 * i + 1].z, w[2 * i].w, w[2 * i + 1].w, v.z, v.w);
            }
          }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int slot = 8 * j + 2 * t + e;
          if (slot >= cnt || n >= n1) continue;
          float s[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[2 * i] = acc[i][j][e];
            s[2 * i + 1] = acc[i][j][2 + e];
          }
          put8<C32>(p, cut.wide, m0 + list[slot], n, s);
        }
    }
  }
};

template <bool C32, int NTM>
__global__ void __launch_bounds__(THREADS, NTM == 1 ? 3 : 2) lora_mma_kernel(const LoraArgs p, const Cut cut) {
  using P = Pass<C32, NTM>;
  constexpr int T = 8 * NTM;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int32_t ids[TM];
  __shared__ uint8_t first[TM], list[TM];
  const Smem lay{(p.R + 31) / 32 * 32, T, P::NS};
  float* sums = reinterpret_cast<float*>(smem);
  float* part = reinterpret_cast<float*>(smem + lay.sum_bytes());
  uint16_t* ts = reinterpret_cast<uint16_t*>(part);
  const int crank = (int)(blockIdx.x % (unsigned)cut.csize);
  const unsigned cluster = blockIdx.x / (unsigned)cut.csize;
  const int64_t m0 = (int64_t)(cluster / (unsigned)cut.nsplit) * TM;
  const int64_t at = (int64_t)(cluster % (unsigned)cut.nsplit * cut.csize + crank) * cut.n_len;
  const int32_t n0 = (int32_t)min64(p.N, at), n1 = (int32_t)min64(p.N, at + cut.n_len);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();

  // The tokens' adapters: -1 none (or none that works), -2 behind the last token.
  if (threadIdx.x < TM) {
    const int64_t m = m0 + threadIdx.x;
    int id = -2;
    if (m < p.M) {
      int rank;
      id = adapter_of(p, m, rank);
    }
    ids[threadIdx.x] = id;
  }
  __syncthreads();
  {  // which tokens are their adapter's first: four threads a token, 16 comparisons each
    const int i = threadIdx.x / 4, j0 = (threadIdx.x & 3) * (TM / 4);
    const int id = ids[i];
    bool before = false;
    for (int j = j0; j < j0 + TM / 4; ++j) before = before || (j < i && ids[j] == id);
    before = __any_sync(0xFu << (lane & 28), before);
    if ((threadIdx.x & 3) == 0) first[i] = id >= 0 && !before;
  }
  __syncthreads();
  uint64_t leaders = __ballot_sync(0xFFFFFFFFu, first[lane]) |
                     (uint64_t)__ballot_sync(0xFFFFFFFFu, first[lane + 32]) << 32;
  if (blockIdx.y == 0 && p.C != p.base)
    for (int i = warp; i < TM; i += WARPS)
      if (ids[i] == -1) copy_row<C32>(p, cut.wide, m0 + i, n0, n1);

  bool reading = false;  // others may still read this CTA's sums
  for (int group = 0; leaders; ++group) {
    const int leader = __ffsll((long long)leaders) - 1;
    leaders &= leaders - 1;
    if (group % (int)gridDim.y != (int)blockIdx.y) continue;
    const int id = ids[leader];
    const int rank = p.ranks ? p.ranks[id] : p.R;
    const float scale = p.scales ? p.scales[id] : 1.f;
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, ids[lane] == id);
    const uint32_t hi = __ballot_sync(0xFFFFFFFFu, ids[lane + 32] == id);
    const int cnt_lo = __popc(lo), cnt = cnt_lo + __popc(hi);
    {  // the second product's weights on their way to L2
      const int lines = (rank * 2 + 127) / 128;
      const uint16_t* b = p.B + ((int64_t)id * p.N + n0) * p.R;
      for (int i = threadIdx.x; i < (n1 - n0) * lines; i += THREADS)
        prefetch_l2(b + (int64_t)(i / lines) * p.R + i % lines * 64);
    }
    __syncthreads();  // (the last group's list has been read)
    if (warp == 0) {
      const uint32_t below = (1u << lane) - 1u;
      if (lo >> lane & 1) list[__popc(lo & below)] = (uint8_t)lane;
      if (hi >> lane & 1) list[cnt_lo + __popc(hi & below)] = (uint8_t)(lane + 32);
    }
    __syncthreads();
    for (int done = 0; done < cnt; done += T) {
      const int now = min(T, cnt - done);
      auto run = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (reading) cluster_wait();
        P::template shrink<NT>(p, cut, crank, m0, id, rank, list + done, now, sums, part, lay.part_pitch());
        cluster_sync();
        P::template gather<NT>(cut, rank, scale, sums, ts, lay.pitch());
        cluster_arrive();
        reading = true;
        __syncthreads();
        P::template expand<NT>(p, cut, m0, id, rank, list + done, now, n0, n1, ts, lay.pitch());
        __syncthreads();  // (ts and part share their place)
      };
      if (NTM > 1 && now <= 8)
        run(std::integral_constant<int, 1>{});
      else
        run(std::integral_constant<int, NTM>{});
    }
  }
  if (reading) cluster_wait();
}

template <bool C32, int NTM>
qw_status launch(const LoraArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  const int64_t tiles = (a.M + TM - 1) / TM;
  const int64_t groups = std::min<int64_t>(std::min<int64_t>(TM, a.M), a.L);  // of a tile, at most
  Cut cut{};
  cut.csize = 1;
  while (cut.csize < 8 && (a.K >= 256 * cut.csize || a.N >= 2 * BN * cut.csize)) cut.csize *= 2;
  cut.nsplit = 1;
  while (tiles * groups * cut.csize * cut.nsplit * 2 <= 2 * sms &&
         (int64_t)a.N * a.R * 2 / (cut.csize * cut.nsplit) > 32768)
    cut.nsplit *= 2;
  const int parts = cut.csize * cut.nsplit;
  cut.k_len = ((a.K + cut.csize - 1) / cut.csize + 63) / 64 * 64;
  cut.n_len = (int32_t)(((int64_t)a.N + parts - 1) / parts + BN - 1) / BN * BN;
  const int vec = C32 ? 4 : 8;
  cut.wide = ((uintptr_t)a.C | (uintptr_t)a.base) % 16 == 0 && a.ldc % vec == 0 &&
             (!a.base || a.ld_base % vec == 0);
  const int64_t x = tiles * parts;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(groups, (4 * sms + x - 1) / x));
  if (x > 0x7FFFFFFF) return QW_ERR_UNSUPPORTED;
  const Smem lay{(a.R + 31) / 32 * 32, 8 * NTM, Pass<C32, NTM>::NS};
  constexpr Smem most{kLoraMaxRank, 8 * NTM, Pass<C32, NTM>::NS};
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [&] {
        return cudaFuncSetAttribute(lora_mma_kernel<C32, NTM>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    most.bytes()) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)x, (unsigned)y);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)lay.bytes();
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cut.csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cut.csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lora_mma_kernel<C32, NTM>, a, cut) == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_lora(const LoraArgs& a, bool c_f32, cudaStream_t st) {
  if (a.M > 16 && lora_tc_takes(a, c_f32)) return launch_lora_tc(a, c_f32, st);
  if (a.M <= 8) return c_f32 ? launch<true, 1>(a, st) : launch<false, 1>(a, st);
  return c_f32 ? launch<true, 4>(a, st) : launch<false, 4>(a, st);
}

}  // namespace qw
