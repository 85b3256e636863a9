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
// t is held as a sum of BF16 numbers for the second product: two for BF16 results (up to 2^-17 t is lost, where
// the result is rounded by up to 2^-8 of itself), three for FP32 ones (all 24 bits).
// The order of k and r within an MMA is free as long as both operands have the same: a lane reads 16
// bytes of a row at once, two MMAs' share.  In the second product row 4 g + i of 32 belongs to the lanes
// of group g, so that a lane ends with four neighbouring columns of a token.
// Bound: latencies, one after the other (ids, ranks, A and X, the cluster's sums, B).  So B comes through a
// ring of TMA boxes of each warp's own (32 rows x 64 r, or 32 r where the rank is no more), filled from the
// moment the adapter is known, and base two blocks ahead.  (Through registers alone 25.3 us for 64 tokens of
// 32 adapters, 14336 x 4096; 16 warps a CTA 26.5; the rest of B prefetched to L2 26.3; now 23.3.)
#include <algorithm>

#include "int8_map.cuh"
#include "lora_common.cuh"

namespace qw {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int TM = 64;  // tokens of a tile
constexpr int BN = 32;  // columns of a warp's block in the second product
constexpr int BR = 64;  // r of a box
constexpr int SLOT = BN * BR * 2, SLOTS = 3;

// How a call is cut up: a cluster of csize CTAs takes K in slices of k_len and, of the columns of its
// part (nsplit of them), slices of n_len.
struct Cut {
  int32_t csize, csize_log, nsplit, k_len, n_len;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// `bytes` (a multiple of 16) from a 16-byte boundary on their way to L2
__device__ __forceinline__ void bulk_prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
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

// Four columns of a token.
template <bool C32>
using Piece = std::conditional_t<C32, uint4, uint2>;
// base of them as it lies in memory: BF16 rows that begin anywhere in the words that they touch
template <bool C32, bool WIDE>
struct Raw {
  uint32_t w[C32 ? 4 : WIDE ? 2 : 3];
};
// (`left`: columns from there to the end)
template <bool C32, bool WIDE>
__device__ __forceinline__ Raw<C32, WIDE> get4(const uint8_t* b, int32_t left) {
  Raw<C32, WIDE> x{};
  if constexpr (WIDE) {
    if (left >= 4) {
      const Piece<C32> v = *reinterpret_cast<const Piece<C32>*>(b);
      x.w[0] = v.x, x.w[1] = v.y;
      if constexpr (C32) x.w[2] = v.z, x.w[3] = v.w;
      return x;
    }
  }
  if constexpr (C32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) x.w[i] = reinterpret_cast<const uint32_t*>(b)[i];
  } else if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) x.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(b)[i] << (16 * (i % 2));
  } else {  // (whole words, whosever the other half of the first and the last is; put together when they are used)
    const int shift = (int)((uintptr_t)b & 2);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (4 * i < 2 * min(left, 4) + shift) x.w[i] = *reinterpret_cast<const uint32_t*>(b - shift + 4 * i);
  }
  return x;
}
template <bool C32, bool WIDE>
__device__ __forceinline__ Piece<C32> four(const Raw<C32, WIDE>& x, const uint8_t* b) {
  if constexpr (C32)
    return make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  else if constexpr (WIDE)
    return make_uint2(x.w[0], x.w[1]);
  else {
    const uint32_t shift = 8 * (uint32_t)((uintptr_t)b & 2);
    return make_uint2(__funnelshift_r(x.w[0], x.w[1], shift), __funnelshift_r(x.w[1], x.w[2], shift));
  }
}
// ... plus sums, to C
template <bool C32, bool WIDE>
__device__ __forceinline__ void put4(uint8_t* c, int32_t left, const Piece<C32>& x, float s0, float s1, float s2,
                                     float s3) {
  Piece<C32> o;
  uint32_t w[4];
  if constexpr (C32) {
    w[0] = __float_as_uint(__uint_as_float(x.x) + s0), w[1] = __float_as_uint(__uint_as_float(x.y) + s1);
    w[2] = __float_as_uint(__uint_as_float(x.z) + s2), w[3] = __float_as_uint(__uint_as_float(x.w) + s3);
    o = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    w[0] = pack_bf16x2(__uint_as_float(x.x << 16) + s0, __uint_as_float(x.x & 0xFFFF0000u) + s1);
    w[1] = pack_bf16x2(__uint_as_float(x.y << 16) + s2, __uint_as_float(x.y & 0xFFFF0000u) + s3);
    o = make_uint2(w[0], w[1]);
  }
  if (WIDE && left >= 4) {
    *reinterpret_cast<Piece<C32>*>(c) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) continue;
      if constexpr (C32)
        reinterpret_cast<uint32_t*>(c)[i] = w[i];
      else
        reinterpret_cast<uint16_t*>(c)[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
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
        const __nv_bfloat16 h = next_part(v, s == NS - 1);
        ts[(s * T + c) * pitch + r] = __bfloat16_as_ushort(h);
        v -= __bfloat162float(h);
      }
    }
  }

};

// A warp's ring of B's boxes: those of its blocks (every eighth of the CTA's), r after r.
struct Ring {
  uint8_t* slots;
  uint64_t* full;
  int32_t n0, end;        // the warp's first column, where the CTA's end
  int id, rank;
  // what is asked for next (one lane), and the next slots to fill and to read
  int32_t n, r;
  uint32_t ask, take, phase;

  __device__ __forceinline__ void start() { n = n0, r = 0; }
  __device__ __forceinline__ void request(const CUtensorMap& wide, const CUtensorMap& narrow) {
    if (n >= end) return;
    const bool half = rank <= 32;
    mbar_arrive_expect_tx(&full[ask], half ? SLOT / 2 : SLOT);
    tma_load_3d(slots + ask * SLOT, half ? &narrow : &wide, &full[ask], r, n, id);
    r += BR;
    if (r >= rank) r = 0, n += WARPS * BN;
    ask = ask + 1 == SLOTS ? 0 : ask + 1;
  }
  __device__ __forceinline__ void next() {
    if (++take == SLOTS) take = 0, phase ^= 1u;
  }
};

template <bool C32, bool WIDE>
__global__ void __launch_bounds__(THREADS, 2)
    lora_mma_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB32,
                    const __grid_constant__ LoraArgs p, const __grid_constant__ Cut cut) {
  constexpr int NS = C32 ? 3 : 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (0u - smem_u32(smem_raw) & 1023u);  // (stays a shared address)
  __shared__ uint8_t lists[WARPS][TM];
  __shared__ uint64_t full[WARPS][SLOTS];
  __shared__ int abort_shared;
  volatile int* abort_flag = &abort_shared;
  const Smem lay{(p.R + 31) / 32 * 32, NS};
  float* sums = reinterpret_cast<float*>(smem + WARPS * SLOTS * SLOT);
  float* part = reinterpret_cast<float*>(smem + WARPS * SLOTS * SLOT + lay.sum_bytes());
  uint16_t* ts = reinterpret_cast<uint16_t*>(part);
  const int crank = (int)(blockIdx.x & (unsigned)(cut.csize - 1));
  const unsigned cluster = blockIdx.x >> cut.csize_log;
  const unsigned tile = cluster / (unsigned)cut.nsplit;
  const int64_t m0 = (int64_t)tile * TM;
  const int64_t at = (int64_t)((cluster - tile * (unsigned)cut.nsplit) * cut.csize + crank) * cut.n_len;
  const int32_t n0 = (int32_t)min64(p.N, at), n1 = (int32_t)min64(p.N, at + cut.n_len);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < WARPS * SLOTS) mbar_init(&full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) abort_shared = 0;
  fence_barrier_init();
  __syncthreads();
  pdl_wait();  // (before the first use of the tensor maps too: their addresses are used again by later launches)
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
  const uint32_t below = (1u << lane) - 1u;
  const uint32_t firsts_lo = __ballot_sync(0xFFFFFFFFu, first_lo), firsts_hi = __ballot_sync(0xFFFFFFFFu, first_hi);
  const int groups = __popc(firsts_lo) + __popc(firsts_hi);
  const int my_lo = __popc(firsts_lo & below), my_hi = __popc(firsts_lo) + __popc(firsts_hi & below);

  bool reading = false;  // others may still read this CTA's sums
  bool ok = true;
  Ring ring{smem + warp * (SLOTS * SLOT), full[warp], n0 + warp * BN, n1};
  const int g = lane >> 2, t = lane & 3;
  for (int group = (int)blockIdx.y; group < groups; group += (int)gridDim.y) {
    const uint32_t in_lo = __ballot_sync(0xFFFFFFFFu, first_lo && my_lo == group);
    const uint32_t in_hi = __ballot_sync(0xFFFFFFFFu, first_hi && my_hi == group);
    const int leader = __ffs((int)(in_lo | in_hi)) - 1;
    const int id = __shfl_sync(0xFFFFFFFFu, in_lo ? id_lo : id_hi, leader);
    const int rank = __shfl_sync(0xFFFFFFFFu, in_lo ? rank_lo : rank_hi, leader);
    const float scale = p.scales ? p.scales[id] : 1.f;
    ring.id = id, ring.rank = rank;
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, id_lo == id), hi = __ballot_sync(0xFFFFFFFFu, id_hi == id);
    const int cnt_lo = __popc(lo), cnt = cnt_lo + __popc(hi);
    __syncwarp();  // (the last group's list has been read)
    if (lo >> lane & 1) lists[warp][__popc(lo & below)] = (uint8_t)lane;
    if (hi >> lane & 1) lists[warp][cnt_lo + __popc(hi & below)] = (uint8_t)(lane + 32);
    __syncwarp();
    for (int done = 0; done < cnt; done += T) {
      const int now = min(T, cnt - done);
      const uint8_t* list = lists[warp] + done;
      ring.start();
      if (lane == 0 && ok)
        for (int i = 0; i < SLOTS; ++i) ring.request(tmB, tmB32);
      if (lane == 0 && warp < now && p.base) {  // base on its way to L2, as far as it is whole 16 bytes
        constexpr int SIZE = C32 ? 4 : 2;
        const uint8_t* x = static_cast<const uint8_t*>(p.base) + ((m0 + list[warp]) * p.ld_base + n0) * SIZE;
        const int skip = (int)(0u - (uint32_t)(uintptr_t)x & 15u);
        const int64_t bytes = (int64_t)(n1 - n0) * SIZE - skip;
        if (bytes >= 16) bulk_prefetch_l2(x + skip, (uint32_t)(bytes & ~15ll));
      }
      __syncwarp();
      const Pass<C32> pass{p, cut, m0, id, rank, now, list, lane, warp, g, t};
      if (reading) cluster_wait();
      pass.shrink(crank, sums, part);
      cluster_sync();
      pass.gather(scale, sums, ts, lay.pitch());
      cluster_arrive();
      reading = true;
      __syncthreads();
      // base + B t for this warp's blocks: a lane's rows of a box, its tokens' rows of base and C
      constexpr int SIZE = C32 ? 4 : 2;
      const int shift = rank <= 32 ? 6 : 7;
      int at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * g + i;
        at[i] = (row << shift) + ((t ^ (shift == 7 ? row & 7 : row >> 1 & 3)) << 4);
      }
      const uint16_t* my_t = ts + g * lay.pitch() + 8 * t;
      const uint8_t* b[2] = {};
      uint8_t* c[2];
      int32_t n = ring.n0 + 4 * g;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t m = m0 + (2 * t + e < now ? list[2 * t + e] : 0);
        if (p.base) b[e] = static_cast<const uint8_t*>(p.base) + (m * p.ld_base + n) * SIZE;
        c[e] = static_cast<uint8_t*>(p.C) + (m * p.ldc + n) * SIZE;
      }
      const bool mine0 = 2 * t < now, mine1 = 2 * t + 1 < now;
      Raw<C32, WIDE> one[2] = {}, two[2] = {};  // base of the next two blocks
      auto ahead = [&](int32_t to, Raw<C32, WIDE>(&x)[2]) {
        const int32_t left = n1 - n - to;
        if (left <= 0 || !p.base) return;
        if (mine0) x[0] = get4<C32, WIDE>(b[0] + (int64_t)to * SIZE, left);
        if (mine1) x[1] = get4<C32, WIDE>(b[1] + (int64_t)to * SIZE, left);
      };
      ahead(0, one);
      ahead(WARPS * BN, two);
      for (int32_t nb = ring.n0; nb < n1; nb += WARPS * BN) {
        const Raw<C32, WIDE> was[2] = {one[0], one[1]};
        one[0] = two[0], one[1] = two[1];
        ahead(2 * WARPS * BN, two);
        float acc[2][4] = {};
#pragma unroll 1
        for (int r = 0; r < rank; r += BR) {
          if (ok) ok = warp_wait(&full[warp][ring.take], ring.phase, abort_flag, p.err);
          const uint8_t* box = ring.slots + ring.take * SLOT;
#pragma unroll
          for (int r0 = 0; r0 < BR; r0 += 32) {
            const int left = rank - r - r0;
            if (left <= 0) break;
            uint4 w[4];
            const bool some = left > 8 * t;  // (what lies past the rank may be anything)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = some ? *reinterpret_cast<const uint4*>(box + (at[i] ^ 2 * r0)) : zero4();
            if (rank & 7 && left < 32) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = first_of(w[i], left - 8 * t);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const uint4 v = *reinterpret_cast<const uint4*>(my_t + s * T * lay.pitch() + r + r0);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                mma_bf16(acc[i], w[2 * i].x, w[2 * i + 1].x, w[2 * i].y, w[2 * i + 1].y, v.x, v.y);
                mma_bf16(acc[i], w[2 * i].z, w[2 * i + 1].z, w[2 * i].w, w[2 * i + 1].w, v.z, v.w);
              }
            }
          }
          __syncwarp();  // the box has been read
          ring.next();
          if (lane == 0 && ok) ring.request(tmB, tmB32);
        }
        const int32_t left = n1 - n;
        if (left > 0) {
          if (mine0)
            put4<C32, WIDE>(c[0], left, four<C32, WIDE>(was[0], b[0]), acc[0][0], acc[0][2], acc[1][0], acc[1][2]);
          if (mine1)
            put4<C32, WIDE>(c[1], left, four<C32, WIDE>(was[1], b[1]), acc[0][1], acc[0][3], acc[1][1], acc[1][3]);
        }
        n += WARPS * BN;
#pragma unroll
        for (int e = 0; e < 2; ++e) b[e] += WARPS * BN * SIZE, c[e] += WARPS * BN * SIZE;
      }
      __syncthreads();  // (ts and part share their place)
    }
  }
  if (!ok && lane == 0)  // after a wait that gave up: let the copies land
    for (int i = 0; i < SLOTS; ++i) wait_landed(&full[warp][i], i < (int)ring.take ? ring.phase ^ 1u : ring.phase);
  if (p.C != p.base)
    for (int i = warp + WARPS * (int)blockIdx.y; i < TM; i += WARPS * (int)gridDim.y) {
      const int id = __shfl_sync(0xFFFFFFFFu, i < 32 ? id_lo : id_hi, i & 31);
      if (id == -1) copy_row<C32>(p, WIDE, m0 + i, n0, n1);
    }
  if (reading) cluster_wait();
}

template <bool C32, bool WIDE>
qw_status launch(const LoraArgs& a, cudaStream_t st) {
  const int sms = device_sm_count();
  const int64_t tiles = (a.M + TM - 1) / TM;
  const int64_t groups = std::min<int64_t>(std::min<int64_t>(TM, a.M), a.L);  // of a tile, at most
  Cut cut{};
  cut.csize = 1;
  while (cut.csize < 8 && (a.K >= 256 * cut.csize || a.N >= 128 * cut.csize)) cut.csize *= 2, ++cut.csize_log;
  cut.nsplit = 1;
  while (tiles * groups * cut.csize * cut.nsplit * 2 <= 2 * sms &&
         (int64_t)a.N * a.R * 2 / (cut.csize * cut.nsplit) > 32768)
    cut.nsplit *= 2;
  const int parts = cut.csize * cut.nsplit;
  cut.k_len = ((a.K + cut.csize - 1) / cut.csize + 63) / 64 * 64;
  cut.n_len = (int32_t)((((int64_t)a.N + parts - 1) / parts + 63) / 64 * 64);
  const int64_t x = tiles * parts;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(groups, (4 * sms + x - 1) / x));
  if (x > 0x7FFFFFFF) return QW_ERR_UNSUPPORTED;
  const Smem lay{(a.R + 31) / 32 * 32, C32 ? 3 : 2};
  constexpr Smem most{kLoraMaxRank, C32 ? 3 : 2};
  constexpr int RING = 1024 + WARPS * SLOTS * SLOT;
  CUtensorMap tmB, tmB32;
  if (!encode_bf16_3d(&tmB, a.B, a.R, a.N, a.L, BR, BN) ||
      !encode_bf16_3d(&tmB32, a.B, a.R, a.N, a.L, 32, BN, CU_TENSOR_MAP_SWIZZLE_64B))
    return QW_ERR_CUDA;
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [&] {
        return cudaFuncSetAttribute(lora_mma_kernel<C32, WIDE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    RING + most.bytes()) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)x, (unsigned)y);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)(RING + lay.bytes());
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cut.csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cut.csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lora_mma_kernel<C32, WIDE>, tmB, tmB32, a, cut) == cudaSuccess ? QW_OK : QW_ERR_CUDA;
}

}  // namespace

qw_status launch_lora(const LoraArgs& a, bool c_f32, cudaStream_t st) {
  // Many tokens of an adapter go through the tensor cores together, and so do large calls, whose tokens may all
  // be one adapter's (us here and there, K = 4096: 32 tokens of one adapter, N = 4096, rank 64 22, 13; of two,
  // N = 14336, rank 16 17, 15; 96 of 8, N = 4096, rank 16 12, 13; 128 of 8, N = 14336, rank 64 27, 24; 192 of 32,
  // N = 4096, rank 32 27, 20; 192 of 64, rank 64 46, 34; 256 of 300, rank 16 52, 90 and 512 98, 93; 4096 of 8 in
  // runs, N = 14336, rank 64 277, 61).  L is what is loaded, the ids are on the device: in all of these a call meets
  // about as many.  Of one adapter out of 300, N = 4096, rank 64, 128 tokens take 47 here, out of one 14 there.
  const bool many = a.M > 512 || (a.M > 128 && a.M > 2 * (int64_t)a.L) || (a.M > 16 && a.M > 12 * (int64_t)a.L);
  if (many && lora_tc_takes(a, c_f32)) return launch_lora_tc(a, c_f32, st);
  if (lora_wide(a, c_f32)) return c_f32 ? launch<true, true>(a, st) : launch<false, true>(a, st);
  return c_f32 ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace qw
