// lora.cu - low-rank adapters of many requests beside a shared projection, on mma.sync: calls in which an
// adapter meets a few tokens.
//
//   C[m][n] = base[m][n] + s_a sum_{r < rank_a} B_a[n][r] t[m][r],  t[m][r] = sum_k A_a[r][k] X[m][k],
//   a = ids[m]
//
// One launch.  A tile is 64 tokens; the tokens of one adapter in it (a group, wherever they stand) go
// through the adapter's weights together, eight at a time, as the 8-column operand of m16n8k16 MMAs with
// the weights' rows as the other: a lone token costs its adapter's bytes and little else.  A group is
// worked on by a cluster: its CTAs take slices of K for t, leave them in shared memory, add them up in
// rank order, and take slices of N for the second product.  So t never leaves the SMs.
// t is held as a sum of BF16 numbers for the second product: two for BF16 results (2^-17 t is lost
// of what the result rounds to 2^-9), three for FP32 ones (all 24 bits).
// The order of k and r within an MMA is free as long as both operands have the same: a lane reads 16
// bytes of a row at once, two MMAs' share.  In the second product row 8 g + i of 64 belongs to the lanes
// of group g, so that a lane ends with eight neighbouring columns of a token, one 16-byte access of C.
// Bound: latencies, one after the other (ids, ranks, A and X, the cluster's sums, B and base).  B's lines
// are fetched to L2 from the start, and a block's weights and base before the sums are there.
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
  int32_t csize, csize_log, nsplit, k_len, n_len;
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
// t of one 16-row block of A for eight tokens over 32-k chunks [c0, c1) from k0, below k1.
__device__ __forceinline__ void shrink_block(const uint16_t* a_lo, const uint16_t* a_hi, bool lo, bool hi,
                                             const uint16_t* x, bool live, int32_t k0, int32_t k1, int c0,
                                             int c1, float (&acc)[4]) {
  constexpr int U = 8;
  const int t = threadIdx.x & 3;
  for (int c = c0; c < c1; c += U) {
    uint4 u[U], v[U], w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int32_t k = k0 + 32 * (c + i) + 8 * t;
      const bool in = c + i < c1 && k < k1;
      u[i] = in && lo ? *reinterpret_cast<const uint4*>(a_lo + k) : zero4();
      v[i] = in && hi ? *reinterpret_cast<const uint4*>(a_hi + k) : zero4();
      w[i] = in && live ? *reinterpret_cast<const uint4*>(x + k) : zero4();
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      mma_bf16(acc, u[i].x, v[i].x, u[i].y, v[i].y, w[i].x, w[i].y);
      mma_bf16(acc, u[i].z, v[i].z, u[i].w, v[i].w, w[i].z, w[i].w);
    }
  }
}

// base of a lane's eight columns of a token, as it lies in memory
template <bool C32>
struct Piece {
  uint4 v[C32 ? 2 : 1];
};
template <bool C32>
__device__ __forceinline__ Piece<C32> get8(const LoraArgs& p, bool wide, int64_t m, int32_t n) {
  Piece<C32> x;
  constexpr int SIZE = C32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < (C32 ? 2 : 1); ++i) x.v[i] = zero4();
  if (!p.base) return x;
  const uint8_t* b = static_cast<const uint8_t*>(p.base) + (m * p.ld_base + n) * SIZE;
  if (wide && n + 8 <= p.N) {
#pragma unroll
    for (int i = 0; i < (C32 ? 2 : 1); ++i) x.v[i] = reinterpret_cast<const uint4*>(b)[i];
  } else {
    uint32_t w[C32 ? 8 : 4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + i >= p.N) continue;
      if constexpr (C32)
        w[i] = reinterpret_cast<const uint32_t*>(b)[i];
      else
        w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(b)[i] << (16 * (i % 2));
    }
#pragma unroll
    for (int i = 0; i < (C32 ? 2 : 1); ++i)
      x.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return x;
}
// ... plus sums, to C
template <bool C32>
__device__ __forceinline__ void put8(const LoraArgs& p, bool wide, int64_t m, int32_t n,
                                     const Piece<C32>& x, const float (&s)[8]) {
  constexpr int SIZE = C32 ? 4 : 2;
  uint8_t* c = static_cast<uint8_t*>(p.C) + (m * p.ldc + n) * SIZE;
  uint32_t o[C32 ? 8 : 4];
  if constexpr (C32) {
    const uint32_t w[8] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w, x.v[1].x, x.v[1].y, x.v[1].z, x.v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(w[j]) + s[j]);
  } else {
    const uint32_t w[4] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack_bf16x2(__uint_as_float(w[j] << 16) + s[2 * j],
                         __uint_as_float(w[j] & 0xFFFF0000u) + s[2 * j + 1]);
  }
  if (wide && n + 8 <= p.N) {
#pragma unroll
    for (int i = 0; i < (C32 ? 2 : 1); ++i)
      reinterpret_cast<uint4*>(c)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n + i >= p.N) continue;
      if constexpr (C32)
        reinterpret_cast<uint32_t*>(c)[i] = o[i];
      else
        reinterpret_cast<uint16_t*>(c)[i] = (uint16_t)(o[i / 2] >> (16 * (i % 2)));
    }
  }
}

constexpr int T = 8;  // tokens of a pass
struct Smem {
  int rows;  // ranks, rounded up to 32
  int splits;
  static constexpr int kPartPitch = T + 2;
  __host__ __device__ int pitch() const { return rows + 8; }  // BF16 numbers of a token's t
  __host__ __device__ int sum_bytes() const { return rows * T * 4; }
  __host__ __device__ int part_bytes() const { return (rows > 16 * WARPS ? rows : 16 * WARPS) * kPartPitch * 4; }
  __host__ __device__ int t_bytes() const { return splits * T * pitch() * 2; }
  __host__ __device__ int bytes() const {
    return sum_bytes() + (part_bytes() > t_bytes() ? part_bytes() : t_bytes());
  }
};

// Up to eight of a group's tokens (their places in the tile in `list`) through its weights.
template <bool C32>
struct Pass {
  static constexpr int NS = C32 ? 3 : 2;
  const LoraArgs& p;
  const Cut& cut;
  int64_t m0;
  int id, rank, cnt;
  const uint8_t* list;
  int lane, warp, g, t;

  // t of this CTA's slice of K, into sums[r][T]
  __device__ __forceinline__ void shrink(int crank, float* sums, float* part) const {
    const int blocks = (rank + 15) / 16;
    // warps that share a block's k: 8, 4, 2 or 1
    const int ks_log = blocks == 1 ? 3 : blocks == 2 ? 2 : blocks <= 4 ? 1 : 0, ks = 1 << ks_log;
    int b0 = warp, s = 0;
    if (ks > 1)
      while (b0 >= blocks) b0 -= blocks, ++s;
    const int32_t k0 = (int32_t)min64(p.K, (int64_t)crank * cut.k_len);
    const int32_t k1 = (int32_t)min64(p.K, (int64_t)k0 + cut.k_len);
    const int chunks = (k1 - k0 + 31) / 32, per = (chunks + ks - 1) >> ks_log;
    const bool live = g < cnt;
    const uint16_t* x = p.X + (m0 + (live ? list[g] : 0)) * p.ldx;
    if (s < ks)
      for (int b = b0; b < blocks; b += ks > 1 ? blocks : WARPS) {
        const uint16_t* a = p.A + ((int64_t)id * p.R + 16 * b + g) * p.K;
        float acc[4] = {};
        shrink_block(a, a + 8 * (int64_t)p.K, 16 * b + g < rank, 16 * b + g + 8 < rank, x, live, k0, k1,
                     s * per, min(chunks, (s + 1) * per), acc);
        float* o = part + (16 * (s * blocks + b) + g) * Smem::kPartPitch + 2 * t;
        *reinterpret_cast<float2*>(o) = make_float2(acc[0], acc[1]);
        *reinterpret_cast<float2*>(o + 8 * Smem::kPartPitch) = make_float2(acc[2], acc[3]);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * blocks * T; i += THREADS) {
      const int r = i / T, c = i % T;
      float v = 0.f;
      for (int q = 0; q < ks; ++q) v += part[(16 * q * blocks + r) * Smem::kPartPitch + c];
      sums[i] = v;
    }
  }

  // the cluster's sums, scaled, as BF16 numbers ts[split][token][r], zeros up to a multiple of 32
  __device__ __forceinline__ void gather(float scale, const float* sums, uint16_t* ts, int pitch) const {
    const int have = (rank + 15) / 16 * 16, rows = (rank + 31) / 32 * 32;
    const uint32_t at = smem_u32(sums);
    for (int i = threadIdx.x; i < rows * T; i += THREADS) {
      const int r = i / T, c = i % T;
      float x[8], v = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        x[q] = r < have && q < cut.csize ? ld_shared_cluster_f32(mapa_shared(at + 4 * i, q)) : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += x[q];
      v *= scale;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        ts[(s * T + c) * pitch + r] = __bfloat16_as_ushort(h);
        v -= __bfloat162float(h);
      }
    }
  }

  // of a block of 64 columns: the weights of 32 r of a lane's eight rows
  struct Weights {
    uint4 w[8];
  };
  __device__ __forceinline__ void load(int32_t nb, int32_t n1, int r0, Weights& x) const {
    const int32_t n = nb + 8 * g;
    const int left = rank - r0 - 8 * t;  // of this lane's eight r, how many count
    const uint16_t* b = p.B + ((int64_t)id * p.N + n) * p.R + r0 + 8 * t;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x.w[i] = left > 0 && n + i < n1 ? *reinterpret_cast<const uint4*>(b + (int64_t)i * p.R) : zero4();
  }
  // base + B t for this CTA's columns; `next`: the first block's weights
  __device__ __forceinline__ void expand(int32_t n0, int32_t n1, const uint16_t* ts, int pitch,
                                         Weights& next) const {
    for (int32_t nb = n0 + warp * BN; nb < n1; nb += WARPS * BN) {
      const int32_t n = nb + 8 * g;
      Piece<C32> was[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < cnt && n < n1) was[e] = get8<C32>(p, cut.wide, m0 + list[2 * t + e], n);
      float acc[4][4] = {};
      for (int r0 = 0; r0 < rank; r0 += 32) {
        Weights x = next;
        const bool more = r0 + 32 < rank;
        load(more ? nb : nb + WARPS * BN, n1, more ? r0 + 32 : 0, next);
        const int left = rank - r0 - 8 * t;
        if (left < 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x.w[i] = first_of(x.w[i], left);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const uint4 v = *reinterpret_cast<const uint4*>(ts + (s * T + g) * pitch + r0 + 8 * t);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_bf16(acc[i], x.w[2 * i].x, x.w[2 * i + 1].x, x.w[2 * i].y, x.w[2 * i + 1].y, v.x, v.y);
            mma_bf16(acc[i], x.w[2 * i].z, x.w[2 * i + 1].z, x.w[2 * i].w, x.w[2 * i + 1].w, v.z, v.w);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (2 * t + e >= cnt || n >= n1) continue;
        float s[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[2 * i] = acc[i][e];
          s[2 * i + 1] = acc[i][2 + e];
        }
        put8<C32>(p, cut.wide, m0 + list[2 * t + e], n, was[e], s);
      }
    }
  }
};

template <bool C32>
__global__ void __launch_bounds__(THREADS, 2) lora_mma_kernel(const __grid_constant__ LoraArgs p,
                                                              const __grid_constant__ Cut cut) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint8_t lists[WARPS][TM];
  const Smem lay{(p.R + 31) / 32 * 32, C32 ? 3 : 2};
  float* sums = reinterpret_cast<float*>(smem);
  float* part = reinterpret_cast<float*>(smem + lay.sum_bytes());
  uint16_t* ts = reinterpret_cast<uint16_t*>(part);
  const int crank = (int)(blockIdx.x & (unsigned)(cut.csize - 1));
  const unsigned cluster = blockIdx.x >> cut.csize_log;
  const unsigned tile = cluster / (unsigned)cut.nsplit;
  const int64_t m0 = (int64_t)tile * TM;
  const int64_t at = (int64_t)((cluster - tile * (unsigned)cut.nsplit) * cut.csize + crank) * cut.n_len;
  const int32_t n0 = (int32_t)min64(p.N, at), n1 = (int32_t)min64(p.N, at + cut.n_len);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();

  // The tokens' adapters, two a lane, each warp for itself: -1 none (or none that works), -2 behind the
  // last token.  A group's first token stands for it.
  int rank_lo = 0, rank_hi = 0;
  const int id_lo = m0 + lane < p.M ? adapter_of(p, m0 + lane, rank_lo) : -2;
  const int id_hi = m0 + 32 + lane < p.M ? adapter_of(p, m0 + 32 + lane, rank_hi) : -2;
  const uint32_t same_lo = __match_any_sync(0xFFFFFFFFu, id_lo);
  const bool first_lo = id_lo >= 0 && __ffs((int)same_lo) - 1 == lane;
  bool first_hi = false;
  if (m0 + 32 < p.M) {
    const uint32_t same_hi = __match_any_sync(0xFFFFFFFFu, id_hi);
    first_hi = id_hi >= 0 && __ffs((int)same_hi) - 1 == lane;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const int other = __shfl_sync(0xFFFFFFFFu, id_lo, j);
      first_hi = first_hi && other != id_hi;
    }
  }
  uint64_t leaders = __ballot_sync(0xFFFFFFFFu, first_lo) |
                     (uint64_t)__ballot_sync(0xFFFFFFFFu, first_hi) << 32;

  bool reading = false;  // others may still read this CTA's sums
  for (int group = 0, mine = (int)blockIdx.y; leaders; ++group) {
    const int leader = __ffsll((long long)leaders) - 1;
    leaders &= leaders - 1;
    if (group != mine) continue;
    mine += (int)gridDim.y;
    const int id = __shfl_sync(0xFFFFFFFFu, leader < 32 ? id_lo : id_hi, leader & 31);
    const int rank = __shfl_sync(0xFFFFFFFFu, leader < 32 ? rank_lo : rank_hi, leader & 31);
    const float scale = p.scales ? p.scales[id] : 1.f;
    {  // the second product's weights on their way to L2
      const uint16_t* b = p.B + (int64_t)id * p.N * p.R;
      for (int32_t n = n0 + (int32_t)threadIdx.x; n < n1; n += THREADS)
        for (int r = 0; r < rank; r += 64) prefetch_l2(b + (int64_t)n * p.R + r);
    }
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, id_lo == id), hi = __ballot_sync(0xFFFFFFFFu, id_hi == id);
    const int cnt_lo = __popc(lo), cnt = cnt_lo + __popc(hi);
    const uint32_t below = (1u << lane) - 1u;
    __syncwarp();  // (the last group's list has been read)
    if (lo >> lane & 1) lists[warp][__popc(lo & below)] = (uint8_t)lane;
    if (hi >> lane & 1) lists[warp][cnt_lo + __popc(hi & below)] = (uint8_t)(lane + 32);
    __syncwarp();
    for (int done = 0; done < cnt; done += T) {
      const int now = min(T, cnt - done);
      const Pass<C32> pass{p, cut, m0, id, rank, now, lists[warp] + done, lane, warp, lane >> 2, lane & 3};
      // base, too
      for (int i = warp; i < now && p.base; i += WARPS) {
        const uint8_t* b = static_cast<const uint8_t*>(p.base) + (m0 + pass.list[i]) * p.ld_base * (C32 ? 4 : 2);
        for (int32_t n = n0 + lane * 64; n < n1; n += 32 * 64)
          for (int h = 0; h < (C32 ? 2 : 1); ++h) prefetch_l2(b + (int64_t)n * (C32 ? 4 : 2) + 128 * h);
      }
      typename Pass<C32>::Weights w;
      if (reading) cluster_wait();
      pass.shrink(crank, sums, part);
      pass.load(n0 + warp * BN, n1, 0, w);
      cluster_sync();
      pass.gather(scale, sums, ts, lay.pitch());
      cluster_arrive();
      reading = true;
      __syncthreads();
      pass.expand(n0, n1, ts, lay.pitch(), w);
      __syncthreads();  // (ts and part share their place)
    }
  }
  if (p.C != p.base)
    for (int i = warp + WARPS * (int)blockIdx.y; i < TM; i += WARPS * (int)gridDim.y) {
      const int id = __shfl_sync(0xFFFFFFFFu, i < 32 ? id_lo : id_hi, i & 31);
      if (id == -1) copy_row<C32>(p, cut.wide, m0 + i, n0, n1);
    }
  if (reading) cluster_wait();
}

template <bool C32>
qw_status launch(const LoraArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  const int64_t tiles = (a.M + TM - 1) / TM;
  const int64_t groups = std::min<int64_t>(std::min<int64_t>(TM, a.M), a.L);  // of a tile, at most
  Cut cut{};
  cut.csize = 1;
  while (cut.csize < 8 && (a.K >= 256 * cut.csize || a.N >= 2 * BN * cut.csize)) cut.csize *= 2, ++cut.csize_log;
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
  const Smem lay{(a.R + 31) / 32 * 32, C32 ? 3 : 2};
  constexpr Smem most{kLoraMaxRank, C32 ? 3 : 2};
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [&] {
        return cudaFuncSetAttribute(lora_mma_kernel<C32>,
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
  return cudaLaunchKernelEx(&cfg, lora_mma_kernel<C32>, a, cut) == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_lora(const LoraArgs& a, bool c_f32, cudaStream_t st) {
  // Tokens of an adapter that are more than a few go through the tensor cores together.
  if (a.M > 16 && a.M > 8 * (int64_t)a.L && lora_tc_takes(a, c_f32)) return launch_lora_tc(a, c_f32, st);
  return c_f32 ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace qw
