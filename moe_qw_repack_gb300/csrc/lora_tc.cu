// lora_tc.cu - low-rank adapters of many requests beside a shared projection, on the tcgen05 tensor
// cores: calls of more than a few tokens.
//
//   C[m][n] = base[m][n] + s_a sum_{r < rank_a} B_a[n][r] t[m][r],  t[m][r] = sum_k A_a[r][k] X[m][k],
//   a = ids[m]
//
// One launch.  An item is up to 128 tokens of one adapter out of a window of 512 (wherever they stand
// in it); a cluster of CTAs works on an item:
//   1  D1[token][r] = X A^T over a CTA's slice of K, in stages of 64 k.  A comes by TMA, and so do tokens
//      that stand together; other rows by cp.async of the epilogue's warps, which have nothing else to do
//      yet.  Four threads ask for the copies by turns.  (TMA gather4 copies, four rows each, took 75 cycles
//      apiece, 2400 a stage.)  A warp that copies nothing puts the fence between those rows and the MMAs: a
//      fence waits for all of its thread's copies, also those of later stages (0.65 us a stage).
//   2  t = s_a (sum of the CTAs' D1, in rank order): each CTA fetches its tokens' shares, adds them up
//      and leaves its tokens' t, which the others fetch; all reads of 256 bytes in a row.  t is held as
//      BF16 numbers that add up to it, two where results are BF16 (up to 2^-17 t is lost, where the result
//      is rounded by up to 2^-8 of itself), three for FP32 ones (24 bits), and lands as the second product's
//      operand: it never leaves the SMs.
//   3  D2[token][n] = t B^T for 128 columns at a time of the CTA's slice of N.  An epilogue warp takes
//      32 tokens (a lane holds a token, a register a column) and a share of the columns: base into
//      shared memory, D2 added to it there, and out to C.  32 tokens that stand together in the call
//      go by TMA boxes, others in pieces of rows (cp.async).
//      Items of up to 64 or 32 tokens have t's rows twice or four times, so that all warps share the
//      columns.  (With a column a lane every element costs accesses of its own: 20 instructions an
//      element, 106 us for 4096 x 14336 x 4096.)
// B's stages have a place of their own and the first are on their way from the start.  Several clusters may
// share an item's columns, each with a t of its own, where that fills the SMs.  Every wait on a barrier is
// bounded; on expiry the kernel reports QW_ERR_TIMEOUT and shuts down.
// Bound by: an item's chain (list 2, X A^T and t 6 to 10, 2 us a tile and group) in small calls; in large ones
// by L2 while all SMs read X and A, where DRAM has little to do (17 us of 4096 x 14336 x 4096, rank 64, with a CTA
// on all of K, 6 with three and 5 to join), then by base and C through shared memory, on 123 of 152 SMs there:
// 61 us, 288 MB at 4.7 TB/s in all (mean of 40 inputs, 56 to 70 by where runs begin and meet).
#include <algorithm>

#include "int8_map.cuh"
#include "lora_common.cuh"

namespace qw {
namespace {

constexpr int TT = 128;      // tokens of an item
constexpr int WINDOW = 512;  // tokens that an item is taken from
constexpr int BN = 128;      // columns of a tile
constexpr int BK = 64;       // k (and r) of a stage: 128 bytes, a swizzle row
constexpr int SLOT = TT * BK * 2;
// warp 0: TMA; warp 1: MMAs and tensor memory; warps 2-17: the epilogue, in two groups of eight that take tiles by
// turns (warp w may read tensor memory's lanes 32 (w % 4) on).  The first group also brings X's rows and
// makes t.
constexpr int EPI_WARP0 = 2, GROUP_WARPS = 8, EPI_WARPS = 2 * GROUP_WARPS, WARPS = EPI_WARP0 + EPI_WARPS;
constexpr int THREADS = 32 * WARPS, GROUP_THREADS = 32 * GROUP_WARPS;
constexpr uint32_t TMEM_COLS = 512;  // D1 (up to 256), and in its place the buffers of D2
constexpr int ACCS = 4;
constexpr int MAX_STAGES = 8;
constexpr int BOX_ROW = 128;              // bytes of a row of a TMA box of base and C: 64 columns of BF16, 32 of FP32
constexpr int UNIT_BYTES = 32 * BOX_ROW;  // a box, a warp's unit of base in shared memory
constexpr int MAX_UNITS = 2;              // of a warp
constexpr int HASH = 2 * WINDOW;
constexpr int SEGS = WINDOW / 32;

struct Params {
  LoraArgs a;
  int32_t csize;
  int32_t parts;      // clusters that share an item's columns (each makes t for itself)
  int32_t k_stages;   // of a CTA's slice of K
  int32_t n_tiles;    // of a CTA's slice of N
  int32_t r16;        // R, rounded up to 16
  int32_t r_slots;    // ... to 64, in stages
  int32_t s2;         // stages of B
  int32_t t_bytes;
  int32_t first_bytes;  // t and the units; before them the first product's stages
  int32_t units;      // of a warp
};

// X in boxes of 64 k and 8, 32 or 128 rows
struct Rows {
  CUtensorMap map[3];
};

// kind::f16: FP32 accumulator (bit 4), A = B = BF16 (bits 7, 10), N >> 3 at bit 17, M >> 4 at bit 24
__device__ __forceinline__ uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// 32 lanes x 8, 16 or 32 columns; complete after tc_landed()
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t taddr, float (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
                   "=f"(r[7])
                 : "r"(taddr));
  else if constexpr (N == 32)
    tc_ld_32x32b_x32(taddr, reinterpret_cast<uint32_t(&)[32]>(r));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]),
          "=f"(r[15])
        : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tc_landed(float (&r)[N]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));  // (no use of them above the wait)
}
__device__ __forceinline__ uint4 ld_cluster_u32x4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 16 bytes to shared memory, of which the first `bytes` are read and the others zero
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
               : "memory");
}
// shared memory to global memory, a box
__device__ __forceinline__ void tma_store_2d(const void* map, const void* smem_src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(smem_src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// ... until the stores' sources have been read / until they are done
__device__ __forceinline__ void tma_store_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// an arrival of this thread on `bar` when its copies so far are there (counted in the barrier's number)
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// ... until at most n (0 to 3, 7; else 7) of this thread's groups are under way
__device__ __forceinline__ void cp_async_wait_upto(int n) {
  if (n == 0)
    cp_async_wait<0>();
  else if (n == 1)
    cp_async_wait<1>();
  else if (n == 2)
    cp_async_wait<2>();
  else if (n == 3)
    cp_async_wait<3>();
  else
    cp_async_wait<7>();
}
// Four neighbouring r of a token's t into the second product's operand, split NS ways.
template <int NS>
__device__ __forceinline__ void put_t(uint8_t* at, int r_slots, int token, int r, const float (&v)[4]) {
  float w[4] = {v[0], v[1], v[2], v[3]};
  const int chunk = ((r & 63) >> 3) ^ (token & 7);
  uint8_t* to = at + (r >> 6) * SLOT + token * 128 + chunk * 16 + (r & 7) * 2;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    __nv_bfloat16 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = next_part(w[i], s == NS - 1);
      w[i] -= __bfloat162float(h[i]);
    }
    *reinterpret_cast<uint2*>(to + s * r_slots * SLOT) =
        make_uint2(__bfloat16_as_ushort(h[0]) | (uint32_t)__bfloat16_as_ushort(h[1]) << 16,
                   __bfloat16_as_ushort(h[2]) | (uint32_t)__bfloat16_as_ushort(h[3]) << 16);
  }
}

// 16 bytes of base plus D2, rounded
template <bool C32>
__device__ __forceinline__ uint4 add_piece(const uint4& was, const float* d) {
  const uint32_t w[4] = {was.x, was.y, was.z, was.w};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (C32)
      o[q] = __float_as_uint(__uint_as_float(w[q]) + d[q]);
    else
      o[q] = pack_bf16x2(__uint_as_float(w[q] << 16) + d[2 * q],
                         __uint_as_float(w[q] & 0xFFFF0000u) + d[2 * q + 1]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 bytes to C, of which `left` elements are there
template <bool C32>
__device__ __forceinline__ void put_piece(uint8_t* to, const uint4& x, int left) {
  if (left >= (C32 ? 4 : 8)) {
    *reinterpret_cast<uint4*>(to) = x;
  } else {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < (C32 ? 4 : 8); ++j)
      if (j < left) {
        if constexpr (C32)
          reinterpret_cast<uint32_t*>(to)[j] = w[j];
        else
          reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
      }
  }
}

// the sum of v over the lanes up to this one
__device__ __forceinline__ int scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int before = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += before;
  }
  return v;
}

// What the CTA knows of its window and of the item at hand.
struct Plan {
  int32_t ids[WINDOW];       // adapters: -1 none, -2 behind the last token
  uint16_t start[WINDOW];    // an adapter's first token: its first item, counted from its 32 tokens' first
  uint8_t items[WINDOW];     // ... and how many it has (0: not a first token)
  int32_t seg[SEGS];         // items of 32 tokens
  int16_t row[TT];           // the item's tokens: where in the window
  int64_t off_c[TT], off_b[TT];  // bytes to the tokens' rows of C and base
};

template <bool C32, bool WIDE>  // (WIDE: base and C take 16-byte accesses)
__global__ void __launch_bounds__(640, 1)  // (registers as for 20 warps: they are shared out by four)
    lora_tc_kernel(const __grid_constant__ Rows tmX, const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmBase, const __grid_constant__ CUtensorMap tmC,
                   const __grid_constant__ CUtensorMap tmC8,
                   const __grid_constant__ Params p) {
  constexpr int NS = C32 ? 3 : 2, SIZE = C32 ? 4 : 2;
  using T = std::conditional_t<C32, float, uint16_t>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (0u - smem_u32(smem_raw) & 1023u);  // (stays a shared address)
  uint8_t* const s_t = smem;
  uint8_t* const ring1 = smem;  // the first product's stages reach over t's place and the units'
  uint8_t* const s_unit = smem + p.t_bytes;
  uint8_t* const ring2 = smem + p.first_bytes;
  __shared__ Plan plan;
  __shared__ uint64_t full1[MAX_STAGES], empty1[MAX_STAGES], landed[MAX_STAGES], full2[MAX_STAGES], empty2[MAX_STAGES];
  __shared__ uint64_t d1_full, acc_full[ACCS], acc_empty[ACCS], base_full[EPI_WARPS][MAX_UNITS], final_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_shared;
  volatile int* abort_flag = &abort_shared;
  const LoraArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int csize = p.csize;
  const unsigned cluster = blockIdx.x / (unsigned)csize;
  const int crank = (int)(blockIdx.x - cluster * (unsigned)csize);
  const unsigned window = cluster / (unsigned)p.parts;
  const int64_t m0 = (int64_t)window * WINDOW;
  const int share = (int)(cluster - window * (unsigned)p.parts) * csize + crank;  // of the columns
  const int win = (int)min64(WINDOW, a.M - m0);

  if (warp == 0) {  // (a lane a few barriers each: one after the other they take 0.4 us)
    if (lane < MAX_STAGES) {
      mbar_init(&full1[lane], 2);  // A and X
      mbar_init(&landed[lane], GROUP_THREADS);
      mbar_init(&empty1[lane], 1);
      mbar_init(&full2[lane], 1);
      mbar_init(&empty2[lane], 1);
    } else if (lane < MAX_STAGES + ACCS) {
      mbar_init(&acc_full[lane - MAX_STAGES], 1);
      mbar_init(&acc_empty[lane - MAX_STAGES], GROUP_WARPS);
    } else if (lane == 31) {
      mbar_init(&d1_full, 1);
      mbar_init(&final_bar, 1);
      abort_shared = 0;
    }
    for (int w = lane; w < EPI_WARPS * MAX_UNITS; w += 32) mbar_init(&base_full[0][0] + w, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
  pdl_wait();  // (before the first use of the tensor maps too: their addresses are used again by later launches)
  pdl_launch_dependents();

  // ---------------------------------------------------------------- the window's items
  // Each adapter's first token and count, by hashing (in the ring's place, which holds nothing yet).
  // Items are numbered by their adapters' first tokens, so that all CTAs number them alike.
  {
    int32_t* key = reinterpret_cast<int32_t*>(ring2);
    int32_t* at = key + HASH;
    int32_t* count = at + HASH;
    for (int i = threadIdx.x; i < HASH; i += THREADS) key[i] = -1, at[i] = WINDOW, count[i] = 0;
    for (int i = threadIdx.x; i < WINDOW; i += THREADS) {
      int rank;
      plan.ids[i] = i < win ? adapter_of(a, m0 + i, rank) : -2;
    }
    __syncthreads();
    for (int s = warp; 32 * s < win; s += WARPS) {
      const int i = 32 * s + lane, id = plan.ids[i];
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
      if (id < 0 || __ffs((int)same) - 1 != lane) continue;  // (one atomic for a warp's tokens of an adapter)
      uint32_t h = (uint32_t)id * 2654435761u >> 16 & (HASH - 1);
      for (;; h = (h + 1) & (HASH - 1)) {  // (ends: half of the places stay free)
        const int was = atomicCAS(&key[h], -1, id);
        if (was == -1 || was == id) break;
      }
      atomicMin(&at[h], i);
      atomicAdd(&count[h], __popc(same));
    }
    __syncthreads();
    for (int s = warp; s < SEGS; s += WARPS) {
      const int i = 32 * s + lane, id = plan.ids[i];
      int n = 0;
      if (id >= 0) {
        uint32_t h = (uint32_t)id * 2654435761u >> 16 & (HASH - 1);
        while (key[h] != id) h = (h + 1) & (HASH - 1);
        if (at[h] == i) n = (count[h] + TT - 1) / TT;
      }
      const int sum = scan(n);
      plan.items[i] = (uint8_t)n;
      plan.start[i] = (uint16_t)(sum - n);
      if (lane == 31) plan.seg[s] = sum;
    }
    fence_proxy_async_smem();  // (the hash's place is written by copies from here on)
    __syncthreads();
  }
  // every warp: items of segment `lane`, of those before it and of the window
  const int seg_items = lane < SEGS ? plan.seg[lane] : 0, seg_sum = scan(seg_items), seg_before = seg_sum - seg_items;
  const int total = __shfl_sync(0xFFFFFFFFu, seg_sum, 31);

  const int64_t all_tiles = ((int64_t)a.N + BN - 1) / BN;
  const int tile0 = (int)min64(all_tiles, (int64_t)share * p.n_tiles);
  const int tiles = (int)min64(p.n_tiles, all_tiles - tile0);
  const int all_k = (a.K + BK - 1) / BK;
  const int kb0 = min(all_k, crank * p.k_stages), nk = min(p.k_stages, all_k - kb0);
  const int ew = warp - EPI_WARP0, group = ew >> 3;                      // of the epilogue (its first group: `worker`)
  const int e = ((int)threadIdx.x - 32 * EPI_WARP0) & (GROUP_THREADS - 1);  // of its group
  const bool worker = warp >= EPI_WARP0 && group == 0;
  const int quad = warp & 3, half = (ew & 7) >> 2;
  // uses so far of the first product's barriers, of D1 and of the D2 buffers (all roles count alike), and
  // the next slot of B's ring and its phase (its two roles count alike)
  uint32_t u1 = 0, ux = 0, ud = 0, ua = 0, slot2 = 0, phase2 = 0;  // (ux: of `landed`)
  uint32_t base_phase = 0;  // of this warp's units of base, a bit each

  for (int item = (int)blockIdx.y; item < total; item += (int)gridDim.y) {
    // -------------------------------------------------------------- the item's tokens (every warp: one barrier)
    const int in_seg = item - seg_before;
    const int seg = __ffs((int)__ballot_sync(0xFFFFFFFFu, in_seg >= 0 && in_seg < seg_items)) - 1;
    const int in_adapter = __shfl_sync(0xFFFFFFFFu, in_seg, seg) - plan.start[32 * seg + lane];
    const int first = __ffs((int)__ballot_sync(0xFFFFFFFFu, in_adapter >= 0 &&
                                                            in_adapter < plan.items[32 * seg + lane])) - 1;
    const int id = plan.ids[32 * seg + first], chunk = __shfl_sync(0xFFFFFFFFu, in_adapter, first);
    int members = 0;  // of segment `lane`
#pragma unroll
    for (int s = 0; s < SEGS; ++s) {
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, plan.ids[32 * s + lane] == id);
      if (lane == s) members = __popc(b);
    }
    const int member_sum = scan(members);
    const int now = min(TT, __shfl_sync(0xFFFFFFFFu, member_sum, 31) - chunk * TT);
    for (int s = warp; s < SEGS; s += WARPS) {
      const int before = __shfl_sync(0xFFFFFFFFu, member_sum - members, s);
      const bool mine = plan.ids[32 * s + lane] == id;
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, mine);
      const int at = before + __popc(b & ((1u << lane) - 1u)) - chunk * TT;
      if (mine && at >= 0 && at < TT) {
        plan.row[at] = (int16_t)(32 * s + lane);
        plan.off_c[at] = (m0 + 32 * s + lane) * a.ldc * SIZE;
        plan.off_b[at] = (m0 + 32 * s + lane) * a.ld_base * SIZE;
      }
    }
    __syncthreads();
    const int rank = a.ranks ? a.ranks[id] : a.R;
    const int slots = (rank + BK - 1) / BK;
    const int uses2 = tiles * slots;
    // The first product's stages hold the item's tokens and A; the MMA's other rows are whatever lies behind
    // (at the end some of B's ring, or what is on its way there).  Their barriers are used in turn, eight of
    // them, whatever the number of stages.
    const bool together = plan.row[now - 1] - plan.row[0] == now - 1;
    const int x_map = now <= 8 ? 0 : now <= 32 ? 1 : 2;
    const int x_bytes = together ? 1024 << (2 * x_map) : (now + 7) / 8 * 1024, stage1 = x_bytes + p.r16 * BK * 2;
    const int s1 = min(MAX_STAGES, p.first_bytes / stage1);
    // t has the tokens' rows 128 / span times
    const int span_log = now <= 32 ? 5 : now <= 64 ? 6 : 7, span = 1 << span_log;
    int issued2 = 0;
    bool ok = true;
    auto stage1_free = [&](int kb) {  // wait until stage kb's place has been read
      const uint32_t u = u1 + (uint32_t)(kb - s1);
      return kb < s1 || mbar_wait(&empty1[u % MAX_STAGES], u / MAX_STAGES & 1u, abort_flag, a.err);
    };

    auto next2 = [&]() {
      if (++slot2 == (uint32_t)p.s2) slot2 = 0, phase2 ^= 1u;
    };
    int b_tile = 0, b_slot = 0;
    auto load_b = [&](int upto) {  // (one lane)
      for (; ok && issued2 < upto; ++issued2) {
        if (!mbar_wait(&empty2[slot2], phase2 ^ 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full2[slot2], SLOT);
        tma_load_2d(ring2 + slot2 * SLOT, &tmB, &full2[slot2], b_slot * BK,
                    (int32_t)((int64_t)id * a.N + (int64_t)(tile0 + b_tile) * BN));
        next2();
        if (++b_slot == slots) b_slot = 0, ++b_tile;
      }
    };
    auto prefetch_base = [&](int tile) {  // a line of the tile's base per thread of a group
      const int token = e >> 1;
      if (tile >= tiles || token >= now || !a.base) return;
      const int32_t n = (tile0 + tile) * BN + (e & 1) * (BN / 2);
      const uint8_t* b = static_cast<const uint8_t*>(a.base) + plan.off_b[token];
      if (n < a.N) prefetch_l2(b + (int64_t)n * SIZE);
      if (C32 && n + 32 < a.N) prefetch_l2(b + (int64_t)(n + 32) * SIZE);
    };

    // -------------------------------------------------------------- 1: X A^T
    auto bring_a = [&](int first) {  // every other stage (one lane; false: a wait gave up)
      for (int kb = first; kb < nk; kb += 2) {
        if (!stage1_free(kb)) return false;
        uint64_t* bar = &full1[(u1 + (uint32_t)kb) % MAX_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)(p.r16 * BK * 2));
        tma_load_2d(ring1 + kb % s1 * stage1 + x_bytes, &tmA, bar, (kb0 + kb) * BK, (int32_t)((int64_t)id * a.R));
      }
      return true;
    };
    auto bring_x = [&](int first) {
      const int32_t y = (int32_t)m0 + plan.row[0];
      for (int kb = first; kb < nk && stage1_free(kb); kb += 2) {
        uint64_t* bar = &full1[(u1 + (uint32_t)kb) % MAX_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)x_bytes);
        tma_load_2d(ring1 + kb % s1 * stage1, &tmX.map[x_map], bar, (kb0 + kb) * BK, y);
      }
    };
    if (warp >= EPI_WARP0 && !worker) {
      const int job = ew - GROUP_WARPS;
      if (lane == 0) {
        if (together && job < 2) bring_x(job);
        if (job == 2) bring_a(1);
      }
      __syncwarp();
      for (int kb = 0; job == 0 && !together && kb < nk; ++kb) {
        const uint32_t u = ux + (uint32_t)kb;
        if (!warp_wait(&landed[u % MAX_STAGES], u / MAX_STAGES & 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full1[(u1 + (uint32_t)kb) % MAX_STAGES]);
      }
      for (int i = 0; i < min(tiles, 2); ++i) prefetch_base(i);
    } else if (worker) {
      if (!together) {  // the listed rows, eight threads a row of a stage
        const uint16_t* x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = (e >> 3) + 32 * q;
          x[q] = a.X + (m0 + (row < now ? plan.row[row] : 0)) * a.ldx + (e & 7) * 8;
        }
        for (int kb = 0, slot = 0; kb < nk; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, stage1_free(kb))) {
            ok = false;
            break;
          }
          const int32_t k = (kb0 + kb) * BK;
          const bool in = k + (e & 7) * 8 < a.K;
          uint8_t* to = ring1 + slot * stage1 + (e >> 3) * 128 + (((e & 7) ^ (e >> 3 & 7)) << 4);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((e >> 3) + 32 * q < now) cp_async16(to + q * 32 * 128, in ? x[q] + k : a.X, in ? 16 : 0);
          if (++slot == s1) slot = 0;
          cp_async_arrive(&landed[(ux + (uint32_t)kb) % MAX_STAGES]);
        }
      }
      if (nk > 0 && ok) ok = warp_wait(&d1_full, ud & 1u, abort_flag, a.err);
      tc_fence_after();
    } else if (warp == 0) {
      if (lane == 0) {
        ok = bring_a(0);
        load_b(min(uses2, p.s2));
      }
      __syncwarp();
    } else if (warp == 1) {
      const bool leader = elect_one();
      const uint32_t id1 = idesc(p.r16);
      for (int kb = 0, slot = 0; ok && kb < nk; ++kb) {
        const uint32_t u = u1 + (uint32_t)kb, s = u % MAX_STAGES;
        if (!warp_wait(&full1[s], u / MAX_STAGES & 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = smem_u32(ring1 + slot * stage1);
        if (++slot == s1) slot = 0;
        const uint64_t dx = smem_desc(at, 16, 1024, 2), da = smem_desc(at + x_bytes, 16, 1024, 2);
        if (leader) {
#pragma unroll
          for (int i = 0; i < BK / 16; ++i)
            tc_mma_f16(tbase, dx + 2 * i, da + 2 * i, id1, kb != 0 || i != 0 ? 1u : 0u);
          tc_commit(&empty1[s]);
        }
        __syncwarp();
      }
      if (nk > 0 && ok && leader) tc_commit(&d1_full);
      __syncwarp();
    }
    // -------------------------------------------------------------- 2: t
    const float scale = a.scales ? a.scales[id] : 1.f;
    const int token = 32 * quad + lane;
    if (worker) {
      for (int r = half * (p.r16 / 2); r < (half + 1) * (p.r16 / 2); r += 8) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (nk > 0) {
          tc_ld<8>(tbase + ((uint32_t)(32 * quad) << 16) + r, v);
          tc_landed(v);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (csize > 1) {  // [r / 4][token] of four r
            reinterpret_cast<float4*>(s_t)[(r / 4 + i) * TT + token] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = r + 4 * i + j < rank ? v[4 * i + j] * scale : 0.f;
            if (token < now)
              for (int row = token; row < TT; row += span) put_t<NS>(s_t, p.r_slots, row, r + 4 * i, w);
          }
        }
      }
      tc_fence_before();
    }
    if (csize > 1) {
      // tokens that a CTA adds up, and the power of two they fit
      const int each = (TT + csize - 1) / csize, each_log = 32 - __clz(each - 1);
      const int n4 = p.r16 / 4 << each_log;
      const int own = (65536 + each - 1) / each;  // row * own >> 16: the CTA that adds up the row
      cluster_sync();
      auto join = [&](auto most) {
        constexpr int MOST = decltype(most)::value;  // of a thread
        float v[MOST][4];
#pragma unroll
        for (int q = 0; q < MOST; ++q) {
          const int i = e + q * GROUP_THREADS, r = (i >> each_log) * 4, of = i & ((1 << each_log) - 1);
          const int mine = crank * each + of;
          const uint32_t at = smem_u32(s_t) + (uint32_t)((i >> each_log) * TT + mine) * 16;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          if (worker && i < n4 && of < each && mine < now) {
            uint4 x[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = c < csize ? ld_cluster_u32x4(mapa_shared(at, c)) : zero4();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              sum.x += __uint_as_float(x[c].x), sum.y += __uint_as_float(x[c].y);
              sum.z += __uint_as_float(x[c].z), sum.w += __uint_as_float(x[c].w);
            }
          }
          v[q][0] = r < rank ? sum.x * scale : 0.f;
          v[q][1] = r + 1 < rank ? sum.y * scale : 0.f;
          v[q][2] = r + 2 < rank ? sum.z * scale : 0.f;
          v[q][3] = r + 3 < rank ? sum.w * scale : 0.f;
        }
        cluster_sync();  // all sums have been read
#pragma unroll
        for (int q = 0; q < MOST; ++q) {
          const int i = e + q * GROUP_THREADS, of = i & ((1 << each_log) - 1), mine = crank * each + of;
          if (worker && i < n4 && of < each && mine < now) put_t<NS>(s_t, p.r_slots, mine, (i >> each_log) * 4, v[q]);
        }
      };
      if (n4 <= GROUP_THREADS)
        join(std::integral_constant<int, 1>{});
      else
        // (two or three CTAs with 128 r, or more)
        join(std::integral_constant<int, TT * 256 / 4 / 4 / GROUP_THREADS>{});
      cluster_sync();
      if (worker) {  // the tokens' rows to all their places, eight threads a row
        const int chunk = (e & 7) ^ (e >> 3 & 7);  // (rows 32 apart are swizzled alike)
        for (int s = 0, in_r = 0; s < NS * p.r_slots; ++s, in_r = in_r + 1 == p.r_slots ? 0 : in_r + 1) {
          if (in_r * BK + chunk * 8 >= p.r16) continue;
          uint4 x[4];
          uint8_t* to = s_t + s * SLOT + (e >> 3) * 128 + (e & 7) * 16;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = (e >> 3) + 32 * q;
            if (row < now) x[q] = ld_cluster_u32x4(mapa_shared(smem_u32(to + q * 32 * 128), row * own >> 16));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = (e >> 3) + 32 * q;
            if (row < now)
              for (int r = row * own >> 16 == crank ? row + span : row; r < TT; r += span)
                *reinterpret_cast<uint4*>(to + (r - (e >> 3)) * 128) = x[q];
          }
        }
      }
    }
    if (worker) fence_proxy_async_smem();
    __syncthreads();
    // -------------------------------------------------------------- 3: base + B t^T
    if (warp == 0) {
      if (lane == 0) load_b(uses2);
      __syncwarp();
    } else if (warp == 1) {
      const bool leader = elect_one();
      tc_fence_after();
      const uint32_t id2 = idesc(BN);
      const uint64_t dt = smem_desc(smem_u32(s_t), 16, 1024, 2);
      const int odd = rank % 16;
      for (int i = 0; ok && i < tiles; ++i) {
        const uint32_t v = ua + (uint32_t)i, buf = v % ACCS;
        if (!warp_wait(&acc_empty[buf], (v / ACCS & 1u) ^ 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int q = 0; q < slots; ++q) {
          if (!warp_wait(&full2[slot2], phase2, abort_flag, a.err)) {
            ok = false;
            break;
          }
          uint8_t* const at = ring2 + slot2 * SLOT;
          if (odd && q == slots - 1) {
            // B's columns past the rank, up to the MMA's 16, may hold anything: zeros
            const int e0 = rank % BK, c1 = (e0 + 15) / 16 * 2;
            for (int r = lane; r < BN; r += 32)
              for (int c = e0 / 8; c < c1; ++c) {
                uint4* x = reinterpret_cast<uint4*>(at + r * 128 + ((c ^ (r & 7)) << 4));
                const int keep = e0 - 8 * c;
                *x = keep > 0 ? first_of(*x, keep) : zero4();
              }
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          const uint64_t db = smem_desc(smem_u32(at), 16, 1024, 2);
          const int steps = min(BK / 16, (rank - q * BK + 15) / 16);
          if (leader) {
#pragma unroll
            for (int w = 0; w < NS; ++w) {
              const uint64_t d = dt + (uint32_t)((w * p.r_slots + q) * (SLOT >> 4));
#pragma unroll
              for (int j = 0; j < BK / 16; ++j)
                if (j < steps)
                  tc_mma_f16(tbase + buf * BN, d + 2 * j, db + 2 * j, id2, q != 0 || w != 0 || j != 0 ? 1u : 0u);
            }
            tc_commit(&empty2[slot2]);
          }
          __syncwarp();
          next2();
        }
        if (!ok) break;
        if (leader) tc_commit(&acc_full[buf]);
        __syncwarp();
      }
    } else if (warp >= EPI_WARP0) {
      // This warp's tokens, and its share of a tile's columns in units of 32 (FP32: 16), or of 16 where the
      // share is no more.  Up to `depth` units' base is under way.
      const int t0 = 32 * quad & (span - 1), count = min(32, now - t0);
      const int width = 64 >> (7 - span_log), col0 = ((32 * quad >> span_log) * 2 + half) * width;
      const int cols = min(width, C32 ? 16 : 32), cols_log = cols == 32 ? 5 : 4;
      const int per_log = (span_log - 1) - cols_log;  // units of a tile
      // (Both groups on every tile, half its columns each: 4096 x 14336 x 4096 73 us instead of 70.)
      const int my_tiles = (tiles + 1 - group) >> 1;  // tiles group, group + 2, ...
      const int units = count > 0 ? my_tiles << per_log : 0, last = (1 << per_log) - 1;
      int rows_log = 3;
      while (rows_log < 5 && 1 << rows_log < count) ++rows_log;
      const int row_log = cols_log + (C32 ? 2 : 1);        // bytes of a unit's row: 64 or 32
      const int pieces_log = row_log - 4;                   // in pieces of 16 bytes
      // Rows that 16-byte accesses do not fit: base comes in the 16-byte pieces that it lies in (one more than
      // its length, an odd number: lanes that hold a row each meet different banks), C goes in words.
      const int words_log = row_log - 2, pitch = (1 << row_log) + 16;
      const int place_bytes = WIDE ? 1 << (rows_log + row_log) : pitch << rows_log;
      int depth = 1;
      while (depth < 8 && 2 * depth * place_bytes <= p.units * UNIT_BYTES) depth *= 2;
      if (depth == 2 && 3 * place_bytes <= p.units * UNIT_BYTES) depth = 3;
      constexpr int EACH = 16 / SIZE;                       // elements of a piece
      uint8_t* const mine = s_unit + ew * p.units * UNIT_BYTES;
      // where piece j of row r lies: eight neighbouring rows' pieces j are in different banks
      auto piece = [&](int r, int j) {
        return (r << row_log) + ((j ^ (pieces_log == 2 ? r >> 1 : r >> 2)) & ((1 << pieces_log) - 1)) * 16;
      };
      auto column = [&](int unit) {
        return (tile0 + 2 * (unit >> per_log) + group) * BN + col0 + ((unit & last) << cols_log);
      };
      const int row1 = lane >> pieces_log, piece1 = lane & ((1 << pieces_log) - 1), rows1 = 32 >> pieces_log;
      const int word1 = lane & ((1 << words_log) - 1), rows2 = 32 >> words_log;
      auto load = [&](int unit, int slot) {
        if (unit < units && a.base) {
          uint8_t* to = mine + slot * place_bytes;
          const int32_t n0 = column(unit);
          const uint8_t* from = static_cast<const uint8_t*>(a.base) + (int64_t)n0 * SIZE;
          const int left = min(cols, a.N - n0) * SIZE;  // bytes of a row
          if constexpr (WIDE) {
            int64_t off[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = plan.off_b[t0 + min(row1 + i * rows1, count - 1)];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (row1 + i * rows1 < count && left > piece1 * 16)
                cp_async16(to + piece(row1 + i * rows1, piece1), from + off[i] + piece1 * 16,
                           min(16, left - piece1 * 16));
          } else if (left > 0) {  // (whole pieces, whosever the ends of the first and the last are)
            // (all offsets before the first copy: nothing is read across one)
            const uint8_t* x[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int r = i < 4 ? row1 + i * rows1 : lane;
              x[i] = from + plan.off_b[t0 + min(r, count - 1)];
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int r = i < 4 ? row1 + i * rows1 : lane, at = 16 * (i < 4 ? piece1 : 1 << pieces_log);
              const int shift = (int)((uintptr_t)x[i] & 15);
              if (r < count && at < left + shift) cp_async16(to + r * pitch + at, x[i] - shift + at);
            }
          }
        }
        cp_async_commit();
      };
      auto store = [&](int unit, int slot) {
        const uint8_t* from = mine + slot * place_bytes;
        const int32_t n0 = column(unit);
        uint8_t* to = static_cast<uint8_t*>(a.C) + (int64_t)n0 * SIZE;
        if constexpr (WIDE) {
          const int left = a.N - n0 - piece1 * EACH;
          int64_t off[4];
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = min(row1 + i * rows1, count - 1);
            off[i] = plan.off_c[t0 + r];
            x[i] = *reinterpret_cast<const uint4*>(from + piece(r, piece1));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (row1 + i * rows1 >= count) continue;
            put_piece<C32>(to + off[i] + piece1 * 16, x[i], left);
          }
        } else {
          const int left = min(cols, a.N - n0) * SIZE;
          for (int r0 = lane >> words_log; r0 < count; r0 += 8 * rows2) {
            uint8_t* row[8];
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = min(r0 + i * rows2, count - 1);
              row[i] = to + plan.off_c[t0 + r];
              x[i] = *reinterpret_cast<const uint32_t*>(from + r * pitch + 4 * word1);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int at = 4 * word1 - (int)((uintptr_t)row[i] & 3);  // in the unit's row
              if (r0 + i * rows2 < count && at >= 0 && at + 4 <= left) *reinterpret_cast<uint32_t*>(row[i] + at) = x[i];
            }
          }
          if (!C32 && lane < count && left > 0) {  // halves of words at the ends
            uint8_t* row = to + plan.off_c[t0 + lane];
            const int shift = (int)((uintptr_t)row & 3), end = left + shift;
            const uint8_t* x = from + lane * pitch;
            if (shift) *reinterpret_cast<uint16_t*>(row) = *reinterpret_cast<const uint16_t*>(x + 2);
            if (end & 2)
              *reinterpret_cast<uint16_t*>(row + left - 2) = *reinterpret_cast<const uint16_t*>(x + end - 2);
          }
        }
      };
      const uint32_t lanes = (uint32_t)(32 * quad) << 16;
      const int my_row = lane & ((1 << rows_log) - 1);
      if (WIDE && span == TT && count > 0) {
        // A whole share of rows that 16-byte accesses fit, 128 bytes of each at a time.  Where the tokens stand
        // together by TMA: a box of base may reach past them; C takes a box of 32 rows, or boxes of 8 and what
        // is left in pieces.  Others in pieces (in units of 64 bytes, four under way: 84 us instead of 74 where
        // some 128 tokens of 4096 x 14336 x 4096 do not stand together).
        const bool tma = plan.row[t0 + count - 1] - plan.row[t0] == count - 1;
        constexpr int COLS = BOX_ROW / SIZE, PER = 64 / COLS;  // columns of a box, boxes of a tile
        const int32_t y = (int32_t)m0 + plan.row[t0];
        const bool leader = elect_one();
        constexpr int PIECES = BOX_ROW / 16;
        auto fetch = [&](int unit, int slot) {  // (the warp; by TMA its leader asks)
          const int32_t n = (tile0 + 2 * (unit / PER) + group) * BN + col0 + unit % PER * COLS;
          const bool in = unit < my_tiles * PER && n < a.N && a.base;
          if (tma) {
            if (in && leader) {
              mbar_arrive_expect_tx(&base_full[ew][slot], UNIT_BYTES);
              tma_load_2d(mine + slot * UNIT_BYTES, &tmBase, &base_full[ew][slot], n, y);
            }
            __syncwarp();
          } else {
            const int j = lane % PIECES, left = min(COLS, a.N - n) * SIZE - 16 * j;  // bytes of the row from here
            const uint8_t* from = static_cast<const uint8_t*>(a.base) + (int64_t)n * SIZE + 16 * j;
            if (in && left > 0) {
#pragma unroll
              for (int i = 0; i < PIECES; ++i) {
                const int r = lane / PIECES + 32 / PIECES * i;
                if (r < count)
                  cp_async16(mine + slot * UNIT_BYTES + r * BOX_ROW + ((j ^ (r & 7)) << 4), from + plan.off_b[t0 + r],
                             min(16, left));
              }
            }
            cp_async_commit();
          }
        };
        fence_proxy_async_smem();  // (an item before may have written the place in pieces)
        __syncwarp();
        int slot = 0;
        for (int unit = 0; unit < my_tiles * PER; ++unit) {
          const int k = unit / PER, u = unit % PER;
          const uint32_t v = ua + (uint32_t)(2 * k + group), buf = v % ACCS;
          // With two places the next unit is asked for before this one is waited for, as soon as the store of the
          // one before has read its place.  (After this one: 77 us instead of 73 for 4096 x 14336 x 4096.)
          if (unit > 0) {
            tma_store_read();
            __syncwarp();
          }
          for (int d = unit == 0 ? 0 : p.units - 1; d < p.units; ++d)  // (one copy of the code: it is long as it is)
            fetch(unit + d, slot + d < p.units ? slot + d : slot + d - p.units);
          if (u == 0) {
            if (ok) ok = warp_wait(&acc_full[buf], v / ACCS & 1u, abort_flag, a.err);
            tc_fence_after();
          }
          const int32_t n = (tile0 + 2 * k + group) * BN + col0 + u * COLS;
          if (n >= a.N) {
            if (u == PER - 1) {
              tc_fence_before();
              __syncwarp();
              if (leader) mbar_arrive(&acc_empty[buf]);
            }
            continue;
          }
          if (a.base) {
            if (tma) {
              if (ok) ok = warp_wait(&base_full[ew][slot], base_phase >> slot & 1u, abort_flag, a.err);
              base_phase ^= 1u << slot;
            } else {
              if (p.units == MAX_UNITS)
                cp_async_wait<MAX_UNITS - 1>();
              else
                cp_async_wait<0>();
              __syncwarp();
            }
          }
          uint8_t* const box = mine + slot * UNIT_BYTES;
          uint8_t* const at = box + lane * BOX_ROW;
          const int sw = lane & 7;  // the box's swizzle
          constexpr int STEP = COLS < 32 ? COLS : 32;
#pragma unroll 1
          for (int c = 0; c < COLS; c += STEP) {
            float d[STEP];
            uint4 was[STEP / EACH];
            tc_ld<STEP>(tbase + ((uint32_t)(32 * quad) << 16) + buf * BN + col0 + u * COLS + c, d);
#pragma unroll
            for (int j = 0; j < STEP / EACH; ++j)
              was[j] = a.base ? *reinterpret_cast<const uint4*>(at + (((c / EACH + j) ^ sw) << 4)) : zero4();
            tc_landed(d);
            if (u == PER - 1 && c + STEP == COLS) {  // D2 has been read
              tc_fence_before();
              __syncwarp();
              if (leader) mbar_arrive(&acc_empty[buf]);
            }
#pragma unroll
            for (int j = 0; j < STEP / EACH; ++j)
              *reinterpret_cast<uint4*>(at + (((c / EACH + j) ^ sw) << 4)) = add_piece<C32>(was[j], d + j * EACH);
          }
          // (a box's last columns are stored in whole 16 bytes: not where the row ends within them)
          const bool boxed = tma && (n + COLS <= a.N || a.N % EACH == 0);
          const int eights = boxed ? count / 8 : 0;
          if (8 * eights < count) {
            __syncwarp();
            for (int q = 8 * eights * PIECES + lane; q < count * PIECES; q += 32) {
              const int r = q / PIECES, j = q % PIECES, left = a.N - n - j * EACH;
              const uint4 x = *reinterpret_cast<const uint4*>(
                  box + r * BOX_ROW + ((j ^ (r & 7)) << 4));
              put_piece<C32>(static_cast<uint8_t*>(a.C) + plan.off_c[t0 + r] + (int64_t)(n + j * EACH) * SIZE, x,
                             left);
            }
          }
          if (tma) fence_proxy_async_smem();
          __syncwarp();
          if (boxed && count == 32) {
            if (leader && ok) tma_store_2d(&tmC, box, n, y);
          } else if (lane < eights && ok) {
            tma_store_2d(&tmC8, box + lane * 8 * BOX_ROW, n, y + 8 * lane);
          }
          tma_store_commit();
          if (++slot == p.units) slot = 0;
        }
        tma_store_done();
        cp_async_wait<0>();
        __syncwarp();
      } else {
        for (int d = 0; d < depth; ++d) load(d, d);
        int slot = 0;
        for (int k = 0; k < my_tiles; ++k) {
          const uint32_t v = ua + (uint32_t)(2 * k + group), buf = v % ACCS;
          prefetch_base(2 * k + group + 4);
          if (ok) ok = warp_wait(&acc_full[buf], v / ACCS & 1u, abort_flag, a.err);
          tc_fence_after();
          for (int unit = k << per_log; unit < min(units, (k + 1) << per_log); ++unit) {
            cp_async_wait_upto(depth - 1);
            __syncwarp();  // the unit's base is there
            uint8_t* at = mine + slot * place_bytes;
            const uint32_t d2 = tbase + lanes + buf * BN + col0 + ((unit & last) << cols_log);
            if constexpr (WIDE) {
              for (int c = 0; c < cols; c += 16) {
                float d[16];
                uint4 was[16 / EACH];
                tc_ld<16>(d2 + c, d);
#pragma unroll
                for (int j = 0; j < 16 / EACH; ++j)
                  was[j] = a.base ? *reinterpret_cast<const uint4*>(at + piece(my_row, c / EACH + j)) : zero4();
                tc_landed(d);
#pragma unroll
                for (int j = 0; j < 16 / EACH; ++j) {
                  const uint4 o = add_piece<C32>(was[j], d + j * EACH);
                  if (lane < count) *reinterpret_cast<uint4*>(at + piece(my_row, c / EACH + j)) = o;
                }
              }
            } else {
              // this lane's row: from where it lies in base to where its words lie in C
              uint4* w = reinterpret_cast<uint4*>(at + my_row * pitch);
              const int64_t n0 = column(unit);
              const int mine_row = t0 + min(lane, count - 1);
              const uint32_t from = (uint32_t)((uintptr_t)a.base + plan.off_b[mine_row] + n0 * SIZE) & 15u;
              const uint32_t to = (uint32_t)((uintptr_t)a.C + plan.off_c[mine_row] + n0 * SIZE) & 3u;
              constexpr int WORDS = 16 * SIZE / 4;  // of 16 columns
              uint32_t carry = 0;
              for (int c = 0; c < cols / 16; ++c) {
                float d[16];
                uint32_t x[WORDS + 4];
                tc_ld<16>(d2 + 16 * c, d);
#pragma unroll
                for (int j = 0; j <= WORDS / 4; ++j)
                  *reinterpret_cast<uint4*>(&x[4 * j]) = a.base ? w[c * WORDS / 4 + j] : zero4();
#pragma unroll
                for (int j = 0; j < WORDS + 2; ++j) x[j] = from & 8 ? x[j + 2] : x[j];
#pragma unroll
                for (int j = 0; j < WORDS + 1; ++j) x[j] = from & 4 ? x[j + 1] : x[j];
                tc_landed(d);
#pragma unroll
                for (int j = 0; j < WORDS; ++j) {
                  if constexpr (C32) {
                    x[j] = __float_as_uint(__uint_as_float(x[j]) + d[j]);
                  } else {
                    const uint32_t b = __funnelshift_r(x[j], x[j + 1], 8 * (from & 2));
                    const uint32_t sum = pack_bf16x2(__uint_as_float(b << 16) + d[2 * j],
                                                     __uint_as_float(b & 0xFFFF0000u) + d[2 * j + 1]);
                    x[j] = __funnelshift_l(carry, sum, 8 * to);
                    carry = sum;
                  }
                }
                if (lane < count) {
#pragma unroll
                  for (int j = 0; j < WORDS / 4; ++j)
                    w[c * WORDS / 4 + j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                }
              }
              if (!C32 && lane < count) w[cols * SIZE / 16].x = carry >> 16;
            }
            __syncwarp();  // its results are
            store(unit, slot);
            __syncwarp();
            load(unit + depth, slot);
            if (++slot == depth) slot = 0;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        cp_async_wait<0>();
      }
    }
    u1 += (uint32_t)nk;
    if (!together) ux += (uint32_t)nk;
    ud += nk > 0 ? 1u : 0u;
    ua += (uint32_t)tiles;
    if (warp >= EPI_WARP0) fence_proxy_async_smem();  // (the units' place is the next item's first stages')
    cluster_sync();  // t, the lists and the rings are free
    tc_fence_after();
  }
  // The rows without adapter: by the clusters that have no item, if there are two at least (and not by the
  // others behind their items: 67 us instead of 56 for 4096 tokens of which 1300 have none).
  const int idle = (int)gridDim.y - total, copiers = idle >= 2 ? idle : (int)gridDim.y;
  const int copier = (int)blockIdx.y - ((int)gridDim.y - copiers);
  if (a.C != a.base && copier >= 0) {
    const int32_t n0 = tile0 * BN, n1 = min(a.N, (tile0 + tiles) * BN);
    for (int i = copier + copiers * warp; i < win; i += copiers * WARPS)
      if (plan.ids[i] == -1) copy_row<C32>(a, WIDE, m0 + i, n0, n1);
  }
  // After a wait that gave up, copies may still be under way to the rings, some on barriers that will never have all
  // their arrivals: they have as long as any wait.
  if (*abort_flag && threadIdx.x == 0)
    for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kWaitLimitNs;) {
    }
  __syncwarp();
  if (warp == 1) {  // (after a wait that gave up, MMAs may still run)
    if (elect_one()) {
      tc_commit(&final_bar);
      wait_landed(&final_bar, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

constexpr int kSmemCta = 232448;  // of one CTA

template <bool C32, bool WIDE>
qw_status launch(const LoraArgs& a, cudaStream_t st) {
  constexpr int NS = C32 ? 3 : 2;
  static std::atomic<int> fixed_smem[64];
  const int fixed = once_per_device(fixed_smem, [] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, lora_tc_kernel<C32, WIDE>) == cudaSuccess ? (int)fa.sharedSizeBytes + 1 : 0;
  }) - 1;
  if (fixed < 0) return QW_ERR_CUDA;
  const int sms = device_sm_count();
  Params p{};
  p.a = a;
  const int64_t windows = (a.M + WINDOW - 1) / WINDOW;
  const int64_t per = std::min<int64_t>(WINDOW, a.M);  // tokens of a window
  const int64_t most = std::min<int64_t>(per, a.L + per / TT);  // items of one
  const int64_t all_tiles = ((int64_t)a.N + BN - 1) / BN, all_k = ((int64_t)a.K + BK - 1) / BK;
  p.r16 = (a.R + 15) / 16 * 16;
  p.r_slots = (a.R + BK - 1) / BK;
  p.t_bytes = NS * p.r_slots * SLOT;
  const int stage1 = SLOT + p.r16 * BK * 2;
  constexpr int UNITS = EPI_WARPS * UNIT_BYTES;
  const int all = kSmemCta - fixed - 1024 - p.t_bytes;
  p.units = std::max(1, std::min(MAX_UNITS, (all - 2 * SLOT) / UNITS));
  p.s2 = std::min(MAX_STAGES, (all - p.units * UNITS) / SLOT);
  p.first_bytes = p.t_bytes + p.units * UNITS;
  if (p.first_bytes / stage1 < 2 || p.s2 < 1) return QW_ERR_UNSUPPORTED;
  // The cheapest cluster and number of clusters on an item's columns, in rounds of what runs at once (a cluster
  // lies within one GPC: 152, 76, 46, 36 and 15 of them) of what an item takes, in us: to find, to join, each
  // CTA's stages and tiles.  What is past one round starts late.  The items: 128 tokens each, and a part of that
  // for each adapter.  (us measured, cluster x clusters: 4096 x 14336 x 4096 rank 64 in runs of 8 adapters 1x3
  // 69, 2x2 72, [3x1] 64, 4x1 76, 8x1 87; 2048 mixed tokens of 8, 4096 x 4096 rank 16 2x1 39, 3x1 31, [4x1] 26,
  // 8x1 49; 256 tokens of 64, rank 32 1x1 48, [2x1] 31, 3x1 48; 128 of one, rank 64 4x1 25, 8x1 18, 8x2 16, [8x4]
  // 15.)
  const double items = (double)((a.M + TT - 1) / TT) + 1 + std::min<int64_t>(a.L, a.M);
  constexpr struct {
    int csize;
    double sms;  // of all
  } sizes[] = {{1, 1.0}, {2, 1.0}, {3, 0.9}, {4, 0.94}, {8, 0.79}};
  double least = 1e30;
  for (const auto& size : sizes)
    for (int parts = 1; parts <= 8; ++parts) {
      const int c = size.csize;
      const int64_t shares = (int64_t)c * parts;
      if ((c > 1 && c > all_k && c > all_tiles) || ((c == 2 || c == 3) && a.R > 128) ||
          (parts > 1 && shares > all_tiles))
        continue;
      const double rounds = items * shares / (sms * size.sms);
      const double cost = (rounds <= 1 ? 1 : rounds + 0.25) * (6 + (c > 1 ? 5 : 0) + (all_k + c - 1) / c * 0.3 +
                                                               (all_tiles + shares - 1) / shares * 1.7);
      if (cost < least) least = cost, p.csize = c, p.parts = parts;
    }
  const int csize = p.csize;
  p.k_stages = (int32_t)((all_k + csize - 1) / csize);
  const int shares = csize * p.parts;
  p.n_tiles = (int32_t)((all_tiles + shares - 1) / shares);
  CUtensorMap tmA, tmB;
  Rows tmX;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_int8_2d(&tmA, bf16, a.A, a.K, (uint64_t)a.L * a.R, (uint64_t)a.K * 2, BK, p.r16) ||
      !encode_int8_2d(&tmB, bf16, a.B, a.R, (uint64_t)a.L * a.N, (uint64_t)a.R * 2, BK, BN))
    return QW_ERR_CUDA;
  for (int i = 0; i < 3; ++i)
    if (!encode_int8_2d(&tmX.map[i], bf16, a.X, a.K, a.M, (uint64_t)a.ldx * 2, BK, 8u << (2 * i))) return QW_ERR_CUDA;
  CUtensorMap tmBase{}, tmC[2]{};
  if constexpr (WIDE) {
    const auto type = C32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : bf16;
    constexpr int SIZE = C32 ? 4 : 2;
    constexpr uint32_t cols = BOX_ROW / SIZE, rows[2] = {32, 8};
    for (int i = 0; i < 2; ++i)
      if (!encode_int8_2d(&tmC[i], type, a.C, a.N, a.M, (uint64_t)a.ldc * SIZE, cols, rows[i]))
        return QW_ERR_CUDA;
    if (a.base &&
        !encode_int8_2d(&tmBase, type, a.base, a.N, a.M, (uint64_t)a.ld_base * SIZE, cols, 32))
      return QW_ERR_CUDA;
  }
  static std::atomic<int> ready[64];
  if (once_per_device(ready, [=] {
        return cudaFuncSetAttribute(lora_tc_kernel<C32, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemCta - fixed) == cudaSuccess;
      }) <= 0)
    return QW_ERR_CUDA;
  const int64_t x = windows * shares;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(most, (4 * sms + x - 1) / x));
  if (x > 0x7FFFFFFF) return QW_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)x, (unsigned)y);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)(1024 + p.first_bytes + p.s2 * SLOT);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lora_tc_kernel<C32, WIDE>, tmX, tmA, tmB, tmBase, tmC[0], tmC[1], p) == cudaSuccess
             ? QW_OK
             : QW_ERR_CUDA;
}

}  // namespace

// Whether this kernel takes a call: tensor coordinates are 32-bit, and t in three parts with more than
// 128 ranks leaves the rings no room.
bool lora_tc_takes(const LoraArgs& a, bool c_f32) {
  return (int64_t)a.L * a.R <= kInt8MaxN && (int64_t)a.L * a.N <= kInt8MaxN &&
         a.ldx < ((int64_t)1 << 38) && a.ldc < ((int64_t)1 << 37) && a.ld_base < ((int64_t)1 << 37) &&
         !(c_f32 && a.R > 128);
}

qw_status launch_lora_tc(const LoraArgs& a, bool c_f32, cudaStream_t st) {
  if (lora_wide(a, c_f32)) return c_f32 ? launch<true, true>(a, st) : launch<false, true>(a, st);
  return c_f32 ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace qw
