// linear.cu — matrix products with a fused epilogue, bf16 in and out, fp32 accumulation
// on the tensor cores: out = act(A B + bias) + residual, optionally with the
// pre-activation A B + bias beside it. Either operand may be stored along or across the
// reduction (the tensor cores read both from shared memory, K-major or MN-major), so one
// set of kernels serves the forward product x W and the gradients dpre W^T and x^T dpre
// without a transposed copy of anything.
//
//   linear_tile_kernel   one 128 x BN output tile per thread block (or per cluster of up
//                        to 8 blocks that share the tile's reduction and add their
//                        partial tiles through distributed shared memory in a fixed
//                        order). With few rows the roles are exchanged: the 128 side runs
//                        along the weight's columns and BN (16 to 128) along the rows.
//   linear_pair_kernel   for large products: 256 x 256 tiles on pairs of SMs
//                        (cta_group::2), persistent, two accumulators, so that the
//                        epilogue of one tile runs beside the products of the next; with
//                        few tiles the reduction is split over pairs as well, the partial
//                        sums going through fp32 scratch to split_reduce_kernel.
//
// The sums, the bias, the activation and the residual are fp32; the one rounding is the
// store to bf16.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "block_ops.h"
#include "linear_epi.cuh"
#include "sm100.cuh"
#include "tma_map.h"

namespace infini {
namespace {

constexpr int kKStep = 64;  // reduction elements per ring stage: one 128-byte swizzle row

__device__ __forceinline__ void tma_load_tile(void* smem_dst, const CUtensorMap* m, uint64_t* bar,
                                              int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// A wait without the error report, for work that is in flight when a block leaves.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > 200000000ull) break;  // 200 ms
  }
}

// Operand tile of `mn` rows or columns x 64 reduction elements in shared memory: K-major,
// mn rows of 128 bytes; MN-major, blocks of 64 columns, each 64 rows of 128 bytes (8 KB).
// Descriptor of its kk-th 16 reduction elements. The storage order is a template parameter
// of the kernels: the issuing thread's work per product has to stay below the product's
// 128 tensor cycles.
template <bool MN_MAJOR>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int kk) {
  return MN_MAJOR ? sdesc(base + (uint32_t)kk * 2048, 8192, 1024)
                  : sdesc(base + (uint32_t)kk * 32, 16, 1024);
}

struct Epilogue {
  const float* bias;
  const __nv_bfloat16* res;
  __nv_bfloat16* out;
  __nv_bfloat16* pre;
  long long ldr, ldo, ldp;
  int act;
};

// Stores into the shared memory of a block of this cluster (address in its window).
__device__ __forceinline__ void st_cluster_f4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void st_cluster_f1(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_shared_f1(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The address in the cluster's window of this block's shared address, in block `rank`.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// The two halves of a barrier over all threads of the cluster.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Eight neighbouring outputs of one row (the row length is a multiple of 8, so that a
// group of 8 is inside or outside as a whole).
__device__ __forceinline__ void finish8(float (&v)[8], const Epilogue& e, long long row,
                                        long long col) {
  if (e.bias) {
    const float4 b0 = __ldg(reinterpret_cast<const float4*>(e.bias + col));
    const float4 b1 = __ldg(reinterpret_cast<const float4*>(e.bias + col + 4));
    v[0] += b0.x; v[1] += b0.y; v[2] += b0.z; v[3] += b0.w;
    v[4] += b1.x; v[5] += b1.y; v[6] += b1.z; v[7] += b1.w;
  }
  if (e.pre) *reinterpret_cast<uint4*>(e.pre + row * e.ldp + col) = pack8(v);
  with_act(e.act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) act_pair<decltype(a)::value>(v[i], v[i + 1]);
  });
  if (e.res) {
    const uint4 r = *reinterpret_cast<const uint4*>(e.res + row * e.ldr + col);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += bf16_lo(w[i]);
      v[2 * i + 1] += bf16_hi(w[i]);
    }
  }
  *reinterpret_cast<uint4*>(e.out + row * e.ldo + col) = pack8(v);
}

// ---- one tile per block or cluster ------------------------------------------------------

struct TileParams {
  unsigned tiles_b;  // BN-wide tiles along the B side
  int ksteps;        // of the whole reduction
  int split;         // blocks (cluster size: 1, 2, 4 or 8) sharing the reduction
  long long rows, cols;  // of the output
  Epilogue epi;
};

// Counts this warp in at a barrier without waiting.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// What the 16-byte unit of a row of `units` (2, 4, 8, 16 or 32) units is xored with: below
// units, and different for the rows that share 128 bytes of shared memory with eight
// neighbours' accesses.
__device__ __forceinline__ uint32_t recv_swizzle(uint32_t row, uint32_t units) {
  return units >= 8 ? row & 7u : units == 4 ? (row >> 1) & 3u : (row >> 2) & 1u;
}

constexpr int kTileThreads = 256;
constexpr int tile_stages(int bn) { return bn <= 16 ? 10 : bn <= 32 ? 9 : bn <= 64 ? 7 : 5; }
constexpr int tile_stage_bytes(int bn) { return (128 + bn) * 128; }
constexpr int tile_ring(int bn) { return tile_stages(bn) * tile_stage_bytes(bn); }
// ring, partial sums of the block's share of the tile, barriers, alignment
constexpr int tile_smem(int bn) { return tile_ring(bn) + 128 * bn * 4 + 256 + 1024; }
static_assert(tile_smem(128) <= 232448 && tile_smem(64) <= 232448, "shared memory of a block");

// Warp 4 brings the operands (TMA), warp 5 issues the products; then all eight warps share
// the epilogue (warp w drains accumulator lanes 32 (w % 4)..; warps 4-7 the upper half of
// its columns). The blocks of a cluster split the reduction; each owns an equal share of
// the tile's columns (rows with SWAP) and gets the others' partial sums of it stored into
// its shared memory, so that one cluster barrier is all that the exchange takes, and adds
// them in rank order, the same sums every time. A block alone takes the same way inside its
// own shared memory: the accumulator's lanes are rows (columns with SWAP) of the output, and
// writing them out from registers, 16 bytes to each of 32 rows at a time, took 1700 cycles
// per 128 x 128 tile.
// Bound by latency when small (the operands' first bytes, one pass through the tensor
// cores, the exchange: one row x 1024 x 4096 4.6 us) and by the stream of the weights with few
// rows (1 x 4096 x 4096 8.8 us), for which every block keeps its whole ring (160 to 180 KB)
// in flight; in between by an SM's share of L2 (32 KB per k-step of 128 x 128: 0.29 us).
template <int BN, bool SWAP, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kTileThreads, 1)
linear_tile_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, const TileParams p) {
  constexpr int ST = tile_stages(BN);
  constexpr int kABytes = 128 * 128, kStage = tile_stage_bytes(BN);
  constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* recv = smem + tile_ring(BN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(recv + 128 * BN * 4);
  uint64_t *full = bars, *empty = bars + ST, *acc = bars + 2 * ST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rank = cluster_ctarank();
  const unsigned t = blockIdx.x / (unsigned)p.split;
  const int a0 = 128 * (int)(t / p.tiles_b), b0 = BN * (int)(t % p.tiles_b);
  const int ks0 = (int)((long long)p.ksteps * rank / p.split);
  const int ks1 = (int)((long long)p.ksteps * (rank + 1) / p.split);
  int issued = 0;

  auto load = [&](int st) {
    uint8_t* sa = smem + st * kStage;
    uint8_t* sb = sa + kABytes;
    const int k = kKStep * (ks0 + issued);
    mbar_arrive_expect_tx(&full[st], (uint32_t)kStage);
    if (A_MN) {
      tma_load_tile(sa, &tm_a, &full[st], a0, k);
      tma_load_tile(sa + 8192, &tm_a, &full[st], a0 + 64, k);
    } else {
      tma_load_tile(sa, &tm_a, &full[st], k, a0);
    }
    if (B_MN) {
#pragma unroll
      for (int i = 0; i < (BN + 63) / 64; ++i)
        tma_load_tile(sb + 8192 * i, &tm_b, &full[st], b0 + 64 * i, k);
    } else {
      tma_load_tile(sb, &tm_b, &full[st], k, b0);
    }
    ++issued;
  };

  cluster_arrive();  // waited for before the exchange: every block has started by then
  uint32_t tmem = 0;
  if (warp == 4) {
    // the first copies are on their way while the block sets up the rest
    if (lane < 2 * ST + 1) mbar_init(&bars[lane], 1);
    fence_barrier_init();
    __syncwarp();
    named_bar_arrive(1, kTileThreads);
  } else {
    if (warp == 5) {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(1, kTileThreads);
    tc_fence_after();
  }

  if (warp == 4) {
    if (lane == 0) {
      while (issued < ST && ks0 + issued < ks1) load(issued);
      while (ks0 + issued < ks1) {
        const int st = issued % ST;
        if (!mbar_wait(&empty[st], (uint32_t)((issued / ST - 1) & 1))) break;
        load(st);
      }
      // every copy into this block's ring has landed before the block leaves
      for (int st = 0; st < ST && st < issued; ++st)
        drain_wait(&full[st], (uint32_t)(((issued - 1 - st) / ST) & 1));
    }
    __syncwarp();
  } else if (warp == 5) {
    constexpr uint32_t idesc = idesc_f32acc(1, A_MN, B_MN, 128, BN);
    tmem = *tmem_slot;
    uint32_t st = 0, phase = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
      if (!mbar_wait_warp(&full[st], phase)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = smem_u32(smem + st * kStage), sb = sa + kABytes;
#pragma unroll
        for (int kk = 0; kk < kKStep / 16; ++kk)
          mma_bf16_ss(tmem, operand_desc<A_MN>(sa, kk), operand_desc<B_MN>(sb, kk), idesc,
                      (ks > ks0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[st]);
      }
      __syncwarp();
      if (++st == ST) st = 0, phase ^= 1;
    }
    if (elect_one()) mma_commit(acc);
    __syncwarp();
  }
  mbar_wait_warp(acc, 0);  // the sums are complete (and tmem_slot long written)
  tc_fence_after();
  tmem = *tmem_slot;

  const int m = 32 * (warp & 3) + lane;  // index along the 128 side
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  constexpr int kCols = BN >= 64 ? BN / 2 : BN;  // accumulator columns of a warp
  const int c0 = BN >= 64 ? kCols * (warp >> 2) : 0;
  const bool drains = BN >= 64 || warp < 4;
  cluster_wait();
  const uint32_t log_s = 31u - (uint32_t)__clz(p.split);
  const uint32_t dst = smem_u32(recv);
  if (drains) {
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
      uint32_t a[32];
      tmem_ld32(tmem + lanes + (uint32_t)(c0 + c), a);
      tmem_wait_ld();
      if (SWAP) {
        // share of rank q: rows [q BN / S, ..) of BN; from rank r: [r][row][128]
        const uint32_t per = BN >> log_s;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t r = (uint32_t)(c0 + c + i);
          if (r >= BN || (long long)b0 + r >= p.rows) continue;
          const uint32_t at = dst + ((rank * per + r % per) * 128 + (uint32_t)m) * 4;
          if (p.split == 1)
            st_shared_f1(at, a[i]);
          else
            st_cluster_f1(mapa(at, r / per), a[i]);
        }
      } else {
        // share of rank q: columns [q BN / S, ..); from rank r: [r][128 rows][BN / S],
        // 16-byte units of a row swizzled
        const uint32_t per = (uint32_t)BN >> log_s, units = per / 4;
        const uint32_t x = recv_swizzle((uint32_t)m, units);
        if ((long long)a0 + m < p.rows) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const uint32_t col = (uint32_t)(c0 + c + i), u = (col % per) / 4;
            const uint32_t at = dst + ((rank * 128 + (uint32_t)m) * units + (u ^ x)) * 16;
            if (p.split == 1)
              st_shared_v4(at, a[i], a[i + 1], a[i + 2], a[i + 3]);
            else
              st_cluster_f4(mapa(at, col / per), a + i);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  auto finish = [&](auto split) {
    constexpr uint32_t S = decltype(split)::value;
    constexpr uint32_t per = BN / S;
    const float4* src = reinterpret_cast<const float4*>(recv);
    constexpr uint32_t total = 128 * per / 8;  // pieces of 8 columns
#pragma unroll 2
    for (uint32_t u = threadIdx.x; u < total; u += kTileThreads) {
      const uint32_t row = SWAP ? u / 16 : u / (per / 8), c8 = SWAP ? u % 16 : u % (per / 8);
      const long long orow = SWAP ? (long long)b0 + rank * per + row : (long long)a0 + row;
      const long long ocol = SWAP ? (long long)a0 + 8 * c8 : (long long)b0 + rank * per + 8 * c8;
      if (orow >= p.rows || ocol >= p.cols) continue;
      float4 x[S], y[S];
#pragma unroll
      for (uint32_t q = 0; q < S; ++q) {
        if (SWAP) {
          x[q] = src[(q * per + row) * 32 + 2 * c8];
          y[q] = src[(q * per + row) * 32 + 2 * c8 + 1];
        } else {
          constexpr uint32_t units = per / 4;
          const uint32_t z = recv_swizzle(row, units);
          x[q] = src[(q * 128 + row) * units + ((2 * c8) ^ z)];
          y[q] = src[(q * 128 + row) * units + ((2 * c8 + 1) ^ z)];
        }
      }
      float v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, y[0].x, y[0].y, y[0].z, y[0].w};
#pragma unroll
      for (uint32_t q = 1; q < S; ++q) {
        v[0] += x[q].x; v[1] += x[q].y; v[2] += x[q].z; v[3] += x[q].w;
        v[4] += y[q].x; v[5] += y[q].y; v[6] += y[q].z; v[7] += y[q].w;
      }
      finish8(v, p.epi, orow, ocol);
    }
  };
  switch (p.split) {
    case 1: finish(std::integral_constant<uint32_t, 1>{}); break;
    case 2: finish(std::integral_constant<uint32_t, 2>{}); break;
    case 4: finish(std::integral_constant<uint32_t, 4>{}); break;
    default: finish(std::integral_constant<uint32_t, 8>{}); break;
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- 256 x 256 tiles on pairs of SMs -----------------------------------------------------

struct PairParams {
  unsigned tiles_n, tiles;  // of 256 columns; in all
  unsigned units;           // tiles * split
  int ksteps, split;
  long long rows, cols;
  Epilogue epi;    // out, res and pre go through tensor maps
  float* partial;  // split > 1 (plain products): [split][rows][cols]
};

struct PairMaps {
  CUtensorMap out, res, pre;  // boxes of 64 columns x 32 rows, 128-byte swizzle
};

// Epilogue warps of a CTA: four lane quarters x four parts of the columns. Half as many had
// longer latencies to hide each: 131072 x 1024 x 4096 with tanh gelu 998 us against 932 (at
// the power limit; without an activation 890 and 893).
constexpr int kEpiWarps = 16;
constexpr int kEpiCols = 1024 / kEpiWarps;  // columns of a warp
constexpr int kPairThreads = 32 * (kEpiWarps + 2);
constexpr int kPairStages = 5;
constexpr int kPairA = 16384, kPairStage = 2 * kPairA;  // this CTA's half of A and of B
constexpr int kSlot = 32 * 128;                         // staging of a warp: 32 rows, 64 columns
constexpr int kPairStaging = kEpiWarps * kSlot;
static_assert(kEpiCols == 64, "one box of columns per warp");
enum {
  Q_FULL = 0,
  Q_EMPTY = Q_FULL + kPairStages,
  Q_AFULL = Q_EMPTY + kPairStages,
  Q_AEMPTY = Q_AFULL + 2,
  Q_DRAIN = Q_AEMPTY + 2,
  Q_RES = Q_DRAIN + 1,  // one per epilogue warp
  Q_COUNT = Q_RES + kEpiWarps
};
constexpr int kPairBars = 512;
static_assert(Q_COUNT * 8 + 4 <= kPairBars, "barrier area");
constexpr int kPairSmem = kPairStages * kPairStage + kPairStaging + kPairBars + 1024;
static_assert(kPairSmem <= 232448, "shared memory of a block");

// A copy into this CTA's shared memory that completes on a barrier of the pair (address in
// the cluster's window).
__device__ __forceinline__ void tma_load_half(void* smem_dst, const CUtensorMap* m,
                                              uint32_t bar_cluster, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_store_box(const CUtensorMap* m, const void* smem_src, int c0,
                                              int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(smem_u32(smem_src)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Warps 0-15 of each CTA: epilogue (warp w drains accumulator lanes 32 (w % 4).. and columns
// 64 (w / 4)..); warp 16: copies; warp 17 of the even CTA: the pair's products (M = 256,
// N = 256, K = 16 each). Each k-step of 64 brings 128 rows (columns) of A and of B into
// each CTA, both CTAs' copies completing on the even CTA's barrier. An epilogue warp's 32
// rows x 64 columns go from the accumulator through registers into its swizzled staging slot
// and out by one TMA store of whole 128-byte lines, clipped at the edges; a residual comes
// into the slot by a TMA load while the products still run and is replaced by the output in
// place; a pre-activation goes out through the slot first. The accumulator is read 32 columns
// at a time (twice with a pre-activation).
// Bound by the tensor cores, and over seconds by the power limit: 131072 x 1024 x 4096 in
// 788 us (1395 TFLOP/s, 82% of the measured burst peak; cuBLAS 756), at the limit 912 (905),
// with bias and tanh gelu 932, with the pre-activation stored too 1082. Two boxes of 32
// columns per warp with a slot each were 1 to 2.5% faster there but 5 to 14% slower where a
// launch has few tiles per pair (8192 x 1024 x 1024: 18.1 us, now 16.9; cuBLAS 15.0).
template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ PairMaps io, const PairParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + kPairStages * kPairStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kPairStaging);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Q_COUNT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const unsigned pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const bool has_res = p.epi.res != nullptr, has_pre = p.epi.pre != nullptr;
  if (threadIdx.x < Q_COUNT) {
    const int x = (int)threadIdx.x;
    mbar_init(&bars[x], (x == Q_AEMPTY || x == Q_AEMPTY + 1) ? 2u * kEpiWarps : 1u);
    fence_barrier_init();
  }
  if (warp == kEpiWarps && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&io.out);
  }
  __syncwarp();
  cluster_arrive();  // barriers initialised in both CTAs before any remote use
  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  cluster_wait();
  uint32_t tmem = 0;
  if (warp != kEpiWarps) {  // the copies start without tensor memory
    tc_fence_before();
    named_bar_sync(1, kPairThreads - 32);
    tc_fence_after();
    tmem = *tmem_slot;
  }
  bool ok = true;

  if (warp == kEpiWarps) {
    // The whole warp runs the loop and one elected lane issues: the values stay uniform, and
    // the way to the copies short enough for a k-step's 512 cycles.
    const uint32_t full0 = smem_cluster_addr(&bars[Q_FULL], 0);
    int it = 0;
    uint32_t st = 0, phase = 1;  // the first use of every stage waits for nothing
    for (unsigned u = pair; ok && u < p.units; u += npairs) {
      const unsigned t = u % p.tiles, part = u / p.tiles;
      const int row = 256 * (int)(t / p.tiles_n) + 128 * (int)rank;
      const int col = 256 * (int)(t % p.tiles_n) + 128 * (int)rank;
      const int ks1 = (int)((long long)p.ksteps * (part + 1) / p.split);
      for (int ks = (int)((long long)p.ksteps * part / p.split); ks < ks1; ++ks, ++it) {
        if (!mbar_wait_warp(&bars[Q_EMPTY + st], phase)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* sa = smem + st * kPairStage;
          uint8_t* sb = sa + kPairA;
          if (rank == 0) mbar_arrive_expect_tx(&bars[Q_FULL + st], 2 * kPairStage);
          const uint32_t full = full0 + 8 * st;
          const int k = kKStep * ks;
          if (A_MN) {
            tma_load_half(sa, &tm_a, full, row, k);
            tma_load_half(sa + 8192, &tm_a, full, row + 64, k);
          } else {
            tma_load_half(sa, &tm_a, full, k, row);
          }
          if (B_MN) {
            tma_load_half(sb, &tm_b, full, col, k);
            tma_load_half(sb + 8192, &tm_b, full, col + 64, k);
          } else {
            tma_load_half(sb, &tm_b, full, k, col);
          }
        }
        __syncwarp();
        if (++st == kPairStages) st = 0, phase ^= 1;
      }
    }
    // every copy into this CTA's ring has landed once its stage has been released
    if (lane < kPairStages && lane < it)
      drain_wait(&bars[Q_EMPTY + lane], (uint32_t)(((it - 1 - lane) / kPairStages) & 1));
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_f32acc(1, A_MN, B_MN, 256, 256);
      uint32_t st = 0, phase = 0;
      int lt = 0;
      for (unsigned u = pair; ok && u < p.units; u += npairs, ++lt) {
        const int acc = lt & 1, use = lt >> 1;
        if (use > 0 && !mbar_wait_warp(&bars[Q_AEMPTY + acc], (uint32_t)((use - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const unsigned part = u / p.tiles;
        const int ks0 = (int)((long long)p.ksteps * part / p.split);
        const int ks1 = (int)((long long)p.ksteps * (part + 1) / p.split);
        const uint32_t td = tmem + (uint32_t)acc * 256;
        for (int ks = ks0; ks < ks1; ++ks) {
          if (!mbar_wait_warp(&bars[Q_FULL + st], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = smem_u32(smem + st * kPairStage), sb = sa + kPairA;
#pragma unroll
            for (int kk = 0; kk < kKStep / 16; ++kk)
              mma_bf16_ss_pair(td, operand_desc<A_MN>(sa, kk), operand_desc<B_MN>(sb, kk), idesc,
                               (ks > ks0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(&bars[Q_EMPTY + st], 3);
            if (ks == ks1 - 1) mma_commit_pair(&bars[Q_AFULL + acc], 3);
          }
          __syncwarp();
          if (++st == kPairStages) st = 0, phase ^= 1;
        }
      }
      if (elect_one()) mma_commit_pair(&bars[Q_DRAIN], 3);
      __syncwarp();
      // both CTAs' epilogues have released every accumulator (their arrivals have landed)
      if (lane == 0)
        for (int acc = 0; acc < 2; ++acc) {
          const int uses = (lt + 1 - acc) / 2;
          if (uses > 0) drain_wait(&bars[Q_AEMPTY + acc], (uint32_t)((uses - 1) & 1));
        }
      __syncwarp();
    }
    // no product into either CTA's tensor memory is in flight past this point
    if (lane == 0) drain_wait(&bars[Q_DRAIN], 0);
    __syncwarp();
  } else {
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    uint8_t* slot = staging + warp * kSlot;
    const uint32_t so = smem_u32(slot);
    uint64_t* rbar = &bars[Q_RES + warp];
    const bool res = has_res, bias = p.epi.bias != nullptr;
    int lt = 0, loads = 0;  // residual copies asked for; every one but the last waited for
    auto pack32 = [&](int half, const float (&v)[32]) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        st_shared_v4(so + sw128(lane, 4 * half + q), pack_bf16x2(v[8 * q], v[8 * q + 1]),
                     pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                     pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                     pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    };
    for (unsigned u = pair; ok && u < p.units; u += npairs, ++lt) {
      const unsigned t = u % p.tiles, part = u / p.tiles;
      const int acc = lt & 1;
      const long long row0 = 256ll * (t / p.tiles_n) + 128 * (int)rank + 32 * (warp & 3);
      const long long col0 = 256ll * (t % p.tiles_n) + kEpiCols * (warp >> 2);
      const bool in = row0 < p.rows && col0 < p.cols;
      const uint32_t ta = tmem + (uint32_t)acc * 256 + lanes + (uint32_t)(kEpiCols * (warp >> 2));
      auto load_res = [&]() {
        bulk_wait_group_read0();  // the slot's last store has been read
        mbar_arrive_expect_tx(rbar, kSlot);
        tma_load_tile(slot, &io.res, rbar, (int)col0, (int)row0);
      };
      // acc + bias of 32 columns
      auto sums = [&](int half, float (&v)[32]) {
        uint32_t a[32];
        tmem_ld32(ta + 32 * half, a);
        if (bias) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
            const long long col = col0 + 32 * half + i;
            if (col < p.cols) b = __ldg(reinterpret_cast<const float4*>(p.epi.bias + col));
            v[i] = b.x; v[i + 1] = b.y; v[i + 2] = b.z; v[i + 3] = b.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(a[i]);
      };
      auto release = [&]() {  // the accumulator may take the next tile
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(smem_cluster_addr(&bars[Q_AEMPTY + acc], 0));
      };
      if (res && !has_pre && in) {
        if (lane == 0) load_res();
        ++loads;
      }
      // this tile's bias into L1 while its products run
      if (bias && lane < kEpiCols / 32 && col0 + 32 * lane < p.cols)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.epi.bias + col0 + 32 * lane));
      if (!mbar_wait_warp(&bars[Q_AFULL + acc], (uint32_t)((lt >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (!in) {
        release();
        continue;
      }
      float v[32];
      if (p.split > 1) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          sums(half, v);
          if (row0 + lane < p.rows) {
            float* dst = p.partial + ((long long)part * p.rows + row0 + lane) * p.cols + col0;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (col0 + 32 * half + i < p.cols)
                st_global_v8(dst + 32 * half + i, reinterpret_cast<const uint32_t*>(v + i));
          }
        }
        release();
        continue;
      }
      if (has_pre) {
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          sums(half, v);
          pack32(half, v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_box(&io.pre, slot, (int)col0, (int)row0);
          tma_store_commit();
          if (res) load_res();
        }
        if (res) ++loads;
      }
      if (res) {
        if (!mbar_wait_warp(rbar, (uint32_t)((loads - 1) & 1))) {
          ok = false;
          break;
        }
      } else {
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
      }
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        sums(half, v);
        if (half == 1) release();
        with_act(p.epi.act, [&](auto k) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) act_pair<decltype(k)::value>(v[i], v[i + 1]);
        });
        if (res) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 r = ld_shared_v4(so + sw128(lane, 4 * half + q));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[8 * q + 2 * i] += bf16_lo(w[i]);
              v[8 * q + 2 * i + 1] += bf16_hi(w[i]);
            }
          }
        }
        pack32(half, v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_box(&io.out, slot, (int)col0, (int)row0);
        tma_store_commit();
      }
    }
    if (lane == 0) {
      // a residual copy that a given-up wait left behind has landed, and every store has
      // been read from shared memory
      if (!ok && loads > 0) drain_wait(rbar, (uint32_t)((loads - 1) & 1));
      bulk_wait_group_read0();
    }
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();  // both CTAs done with tensor memory and with each other's barriers
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// out from the partial sums of a split reduction, added in order. HBM- or L2-bound; a thread
// has 8 neighbouring columns.
__global__ void __launch_bounds__(256)
split_reduce_kernel(const float* __restrict__ partial, int split, long long rows, long long cols,
                    __nv_bfloat16* __restrict__ out, long long ldo) {
  const long long units = rows * (cols / 8), per = cols / 8;
  for (long long u = blockIdx.x * 256ll + threadIdx.x; u < units; u += gridDim.x * 256ll) {
    const long long row = u / per, col = 8 * (u % per);
    float v[8] = {};
    for (int q = 0; q < split; ++q) {
      const float4* src =
          reinterpret_cast<const float4*>(partial + ((long long)q * rows + row) * cols + col);
      const float4 x = __ldcs(src), y = __ldcs(src + 1);
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    *reinterpret_cast<uint4*>(out + row * ldo + col) = pack8(v);
  }
}

// ---- host side --------------------------------------------------------------------------

// Map over a stored matrix [outer][inner], rows ld elements apart; boxes of 64 inner x
// box_outer outer elements, 128-byte swizzle. Reads outside the matrix give zeros, stores
// outside it are dropped.
bool make_map(CUtensorMap* m, const void* base, long long inner, long long outer, long long ld,
              uint32_t box_outer) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of an operand whose tile is `mn` rows or columns wide.
bool operand_map(CUtensorMap* m, const __nv_bfloat16* p, long long ld, bool mn_major,
                 long long extent, long long R, int mn) {
  return mn_major ? make_map(m, p, extent, R, ld, 64)
                  : make_map(m, p, R, extent, ld, (uint32_t)mn);
}

// Map of an output (or residual) in boxes of 64 columns x 32 rows, 128-byte swizzle.
bool box_map(CUtensorMap* m, const __nv_bfloat16* p, long long rows, long long cols,
             long long ld) {
  return make_map(m, p, cols, rows, ld, 32);
}

// CTA pairs that can be resident at once, looked up once per device.
int pair_count(int sms) {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(sms & ~1));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel<false, true>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 0;
  }
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t pair_launch(const GemmArgs& g, int split, float* partial, int sms,
                        cudaStream_t stream) {
  const int pairs = pair_count(sms);
  if (pairs < 1) return cudaErrorLaunchOutOfResources;
  CUtensorMap ma, mb;
  PairMaps io;
  if (!operand_map(&ma, g.a, g.lda, g.a_mn, g.P, g.R, 128) ||
      !operand_map(&mb, g.b, g.ldb, g.b_mn, g.Q, g.R, 128) ||
      !box_map(&io.out, g.out, g.P, g.Q, g.ldo))
    return cudaErrorInvalidValue;
  io.res = io.pre = io.out;
  if (g.res && !box_map(&io.res, g.res, g.P, g.Q, g.ldr)) return cudaErrorInvalidValue;
  if (g.pre && !box_map(&io.pre, g.pre, g.P, g.Q, g.ldp)) return cudaErrorInvalidValue;
  PairParams p;
  const long long tiles_n = (g.Q + 255) / 256, units = (g.P + 255) / 256 * tiles_n * split;
  if (units >= (1ll << 31)) return cudaErrorInvalidValue;
  p.tiles_n = (unsigned)tiles_n;
  p.units = (unsigned)units;
  p.tiles = p.units / (unsigned)split;
  p.ksteps = (int)((g.R + kKStep - 1) / kKStep);
  p.split = split;
  p.rows = g.P;
  p.cols = g.Q;
  p.epi = Epilogue{g.bias, g.res, g.out, g.pre, g.ldr, g.ldo, g.ldp, g.act};
  p.partial = partial;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(2 * (p.units < (unsigned)pairs ? p.units : (unsigned)pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = g.a_mn   ? cudaLaunchKernelEx(&cfg, linear_pair_kernel<true, true>, ma, mb, io, p)
                  : g.b_mn ? cudaLaunchKernelEx(&cfg, linear_pair_kernel<false, true>, ma, mb, io, p)
                           : cudaLaunchKernelEx(&cfg, linear_pair_kernel<false, false>, ma, mb, io, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || split == 1) return e;
  const long long blocks = (g.P * (g.Q / 8) + 255) / 256;
  split_reduce_kernel<<<(unsigned)(blocks < 16ll * sms ? blocks : 16ll * sms), 256, 0, stream>>>(
      partial, split, g.P, g.Q, g.out, g.ldo);
  return cudaGetLastError();
}

template <int BN, bool SWAP, bool A_MN, bool B_MN>
cudaError_t tile_launch(const GemmArgs& g, int split, cudaStream_t stream) {
  const long long a_extent = SWAP ? g.Q : g.P, b_extent = SWAP ? g.P : g.Q;
  CUtensorMap ma, mb;
  const bool ok = SWAP ? operand_map(&ma, g.b, g.ldb, g.b_mn, g.Q, g.R, 128) &&
                             operand_map(&mb, g.a, g.lda, g.a_mn, g.P, g.R, BN)
                       : operand_map(&ma, g.a, g.lda, g.a_mn, g.P, g.R, 128) &&
                             operand_map(&mb, g.b, g.ldb, g.b_mn, g.Q, g.R, BN);
  if (!ok) return cudaErrorInvalidValue;
  TileParams p;
  const long long tiles_b = (b_extent + BN - 1) / BN;
  const long long blocks = (a_extent + 127) / 128 * tiles_b * split;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  p.tiles_b = (unsigned)tiles_b;
  p.ksteps = (int)((g.R + kKStep - 1) / kKStep);
  p.split = split;
  p.rows = g.P;
  p.cols = g.Q;
  p.epi = Epilogue{g.bias, g.res, g.out, g.pre, g.ldr, g.ldo, g.ldp, g.act};
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = tile_smem(BN);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_tile_kernel<BN, SWAP, A_MN, B_MN>, ma, mb, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename K>
cudaError_t set_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

cudaError_t linear_set_attributes() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* kernel, int bytes) {
    if (e == cudaSuccess) e = set_smem(kernel, bytes);
  };
  set(linear_tile_kernel<16, true, true, false>, tile_smem(16));
  set(linear_tile_kernel<16, true, false, false>, tile_smem(16));
  set(linear_tile_kernel<32, true, true, false>, tile_smem(32));
  set(linear_tile_kernel<32, true, false, false>, tile_smem(32));
  set(linear_tile_kernel<64, true, true, false>, tile_smem(64));
  set(linear_tile_kernel<64, true, false, false>, tile_smem(64));
  set(linear_tile_kernel<64, false, false, true>, tile_smem(64));
  set(linear_tile_kernel<64, false, false, false>, tile_smem(64));
  set(linear_tile_kernel<64, false, true, true>, tile_smem(64));
  set(linear_tile_kernel<128, false, false, true>, tile_smem(128));
  set(linear_tile_kernel<128, false, false, false>, tile_smem(128));
  set(linear_tile_kernel<128, false, true, true>, tile_smem(128));
  set(linear_pair_kernel<false, true>, kPairSmem);
  set(linear_pair_kernel<false, false>, kPairSmem);
  set(linear_pair_kernel<true, true>, kPairSmem);
  return e;
}

namespace {

// How a product is run.
struct GemmPlan {
  bool pair;
  int bn;     // tile width without a pair
  int split;  // blocks of a cluster, or parts of a pair launch
};

// Estimated time (us) of the tile kernel: a launch, and for every wave of blocks the time to
// the first operands, the k-steps, which bring (128 + bn) x 128 bytes into an SM at its
// share of L2 bandwidth, and the exchange of a split. Against measured times of 34 products
// that take this kernel, from 100 x 512 x 1024 to 16384 x 256 x 512 in all three storage orders,
// the estimates lie between 12% below and 16% above, but for one of 5.8 us (7.5 estimated).
double tile_time(int bn, int split, long long blocks, long long ksteps, int sms) {
  static const double step128 = 0.29, step64 = 0.20, step32 = 0.165, step16 = 0.15;
  static const double swap128[4] = {0.0, 2.3, 3.2, 4.4};  // for 1, 2, 4, 8 blocks
  const double step = bn >= 128 ? step128 : bn >= 64 ? step64 : bn >= 32 ? step32 : step16;
  const int i = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
  // clusters of eight find room on fewer SMs
  const long long room = split == 8 ? sms * 3 / 4 : sms;
  const double waves = (double)((blocks + room - 1) / room);
  const double part = (double)((ksteps + split - 1) / split);
  return 1.8 + waves * (2.8 + part * step + swap128[i] * (0.3 + 0.7 * bn / 128));
}

// The same for the pair kernel: persistent, a k-step of 256 x 256 in 0.31 us, the last
// tile's epilogue exposed; a split adds a launch and the partial sums' way through L2. Up to
// 8192 x 1024 x 1024 within 12% of measured times; 13 to 33% too low for ragged products (rows
// off 128-byte lines and edge tiles cost more: 5003 x 1160 x 2056 24 us estimated, 32 taken)
// and for long ones, whose clock is lower (32768 x 4096 x 1024 146 and 180).
double pair_time(long long P, long long Q, int split, long long units, long long ksteps,
                 int sms) {
  const long long pairs = sms / 2, part = (ksteps + split - 1) / split;
  const double waves = (double)((units + pairs - 1) / pairs);
  double t = 6.6 + waves * (part * 0.31 > 1.9 ? part * 0.31 : 1.9);
  if (split > 1) t += 3.0 + (double)split * P * Q * 8 / 8e6;
  return t;
}

int tile_split(int bn, long long tiles, long long ksteps, int sms) {
  int best = 1;
  double t = tile_time(bn, 1, tiles, ksteps, sms);
  for (int s = 2; s <= 8 && ksteps >= 2 * s; s *= 2) {
    const double u = tile_time(bn, s, tiles * s, ksteps, sms);
    if (u < t) t = u, best = s;
  }
  return best;
}

// The fastest by the estimates. A split over pairs needs scratch and is for plain products: the
// gradients', whose reductions are long and whose tiles are few.
GemmPlan gemm_plan(long long P, long long Q, long long R, bool scratch, int sms) {
  const long long ksteps = (R + kKStep - 1) / kKStep;
  const long long big = (P + 255) / 256 * ((Q + 255) / 256);
  GemmPlan best{true, 256, 1};
  double t = pair_time(P, Q, 1, big, ksteps, sms);
  for (int s = 2; scratch && s <= 8 && ksteps >= 8 * s && big * s <= sms / 2; ++s) {
    const double u = pair_time(P, Q, s, big * s, ksteps, sms);
    if (u < t) t = u, best = GemmPlan{true, 256, s};
  }
  for (int bn = 64; bn <= 128; bn *= 2) {
    const long long tiles = (P + 127) / 128 * ((Q + bn - 1) / bn);
    const int s = tile_split(bn, tiles, ksteps, sms);
    const double u = tile_time(bn, s, tiles * s, ksteps, sms);
    if (u < t) t = u, best = GemmPlan{false, bn, s};
  }
  return best;
}

}  // namespace

size_t linear_gemm_scratch(long long P, long long Q, long long R, int sms) {
  const GemmPlan g = gemm_plan(P, Q, R, true, sms);
  return g.pair && g.split > 1 ? (size_t)g.split * P * Q * 4 : 0;
}

// The products there are: x W (A along the reduction, B across it), d W^T (both along),
// x^T d (both across).
cudaError_t linear_gemm_launch(const GemmArgs& g, void* scratch, int sms, cudaStream_t stream) {
  if (g.a_mn && !g.b_mn) return cudaErrorInvalidValue;
  // Few rows, stored along the reduction: the rows take the narrow side of the tile.
  if (g.P <= 64 && !g.a_mn) {
    const int bn = g.P <= 16 ? 16 : g.P <= 32 ? 32 : 64;
    const int s = tile_split(bn, (g.Q + 127) / 128, (g.R + kKStep - 1) / kKStep, sms);
    if (bn == 16)
      return g.b_mn ? tile_launch<16, true, true, false>(g, s, stream)
                    : tile_launch<16, true, false, false>(g, s, stream);
    if (bn == 32)
      return g.b_mn ? tile_launch<32, true, true, false>(g, s, stream)
                    : tile_launch<32, true, false, false>(g, s, stream);
    return g.b_mn ? tile_launch<64, true, true, false>(g, s, stream)
                  : tile_launch<64, true, false, false>(g, s, stream);
  }
  const bool plain = !g.bias && !g.res && !g.pre && g.act == kActNone;
  const GemmPlan f = gemm_plan(g.P, g.Q, g.R, plain && scratch, sms);
  if (f.pair) return pair_launch(g, f.split, static_cast<float*>(scratch), sms, stream);
  if (f.bn == 64)
    return g.a_mn   ? tile_launch<64, false, true, true>(g, f.split, stream)
           : g.b_mn ? tile_launch<64, false, false, true>(g, f.split, stream)
                    : tile_launch<64, false, false, false>(g, f.split, stream);
  return g.a_mn   ? tile_launch<128, false, true, true>(g, f.split, stream)
         : g.b_mn ? tile_launch<128, false, false, true>(g, f.split, stream)
                  : tile_launch<128, false, false, false>(g, f.split, stream);
}

// ---- the activation's gradient and the bias gradient --------------------------------------

namespace {

constexpr int kActThreads = 256;
constexpr int kBatch = 3;
constexpr int kActBlocks = 3;      // resident per SM
constexpr int kActNarrowRows = 1024;

// Columns of a block: 256 (a warp per row), or 32 for few rows (64 rows at a time), where
// one block then takes all of them and the column sums need no second launch. Narrow and wide
// with tanh gelu, us: 64 rows 2.4 and 4.2 (512 columns), 5.4 and 6.7 (16384); 512 rows 5.0 and
// 4.8, 12.7 and 13.7; 1024 rows 8.0 and 5.4 (512), 8.2 and 6.3 (1408), 8.6 and 8.4 (4096), 23.1
// and 22.5 (16384); 2048 rows 13.7 and 6.5, 47.7 and 41.8. Between 512 and 1024 rows the wide
// form would save up to 2.6 us where columns are few.
constexpr int act_cols(long long M) { return M <= kActNarrowRows ? 32 : 256; }

// dpre = dy act'(pre), one 16-byte piece of a row per thread and step, and the column
// sums of dpre before its rounding (fp32, one row of `part` per row chunk). HBM-bound:
// dy and pre read once, dpre written once (16384 x 4096: 75 us = 5.4 TB/s with silu, 79 with
// tanh gelu, 82 with gelu, 29 us = 4.6 TB/s for the sums alone).
template <int ACT, int COLS>
__global__ void __launch_bounds__(kActThreads, kActBlocks)
act_grad_kernel(const __nv_bfloat16* __restrict__ dy, long long lddy,
                const __nv_bfloat16* __restrict__ pre, long long ldp,
                __nv_bfloat16* __restrict__ dpre, float* __restrict__ part, long long M, int N) {
  constexpr int kLanes = COLS / 8, kRows = kActThreads / kLanes;  // rows at a time
  __shared__ float sums[kRows][COLS];
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int col = blockIdx.x * COLS + 8 * lane;
  const bool in = col < N;
  const long long r0 = M * blockIdx.y / gridDim.y, r1 = M * (blockIdx.y + 1) / gridDim.y;
  float s[8] = {};
  if (in) {
    // kBatch rows' loads in flight before the first is used
    for (long long r = r0 + row; r < r1; r += kBatch * kRows) {
      uint4 g[kBatch], z[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const long long rk = r + k * kRows;
        if (rk < r1) {
          g[k] = __ldcs(reinterpret_cast<const uint4*>(dy + rk * lddy + col));
          if (ACT != kActNone) z[k] = __ldcs(reinterpret_cast<const uint4*>(pre + rk * ldp + col));
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const long long rk = r + k * kRows;
        if (rk >= r1) break;
        const uint32_t gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        const uint32_t zw[4] = {z[k].x, z[k].y, z[k].z, z[k].w};
        float d[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[2 * i] = bf16_lo(gw[i]);
          d[2 * i + 1] = bf16_hi(gw[i]);
          if (ACT != kActNone) {
            float a = bf16_lo(zw[i]), b = bf16_hi(zw[i]);
            act_deriv_pair<ACT>(a, b);
            d[2 * i] *= a;
            d[2 * i + 1] *= b;
          }
          s[2 * i] += d[2 * i];
          s[2 * i + 1] += d[2 * i + 1];
        }
        // bf16 because the tensor cores read it: 2^-8 relative at most, as every operand
        if (ACT != kActNone)
          *reinterpret_cast<uint4*>(dpre + rk * (long long)N + col) = pack8(d);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[row][8 * lane + i] = s[i];
  __syncthreads();
  const int c = blockIdx.x * COLS + threadIdx.x;
  if (threadIdx.x < COLS && c < N) {
    float v = 0.f;
#pragma unroll 8
    for (int w = 0; w < kRows; ++w) v += sums[w][threadIdx.x];
    part[(long long)blockIdx.y * N + c] = v;
  }
}

// Fixed-order sums: 32 columns x 8 partial sums of every eighth row. The grid's rows are
// the sets, then the groups (in layers of gy, a grid axis holding 65535).
__global__ void __launch_bounds__(256) colsum_kernel(const ColsumArgs a, const unsigned gy) {
  __shared__ float sums[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float* src;
  float* dst;
  long long count, step;
  if (blockIdx.z == 0 && blockIdx.y < (unsigned)a.sets) {
    dst = a.out[blockIdx.y];
    src = a.part + (long long)blockIdx.y * a.D;
    count = a.count;
    step = (long long)a.sets * a.D;
  } else {
    if (blockIdx.y < (unsigned)a.sets) return;
    const long long g = (blockIdx.y - (unsigned)a.sets) + (long long)blockIdx.z * gy;
    if (g >= a.groups) return;
    dst = a.dgate + g * a.D;
    src = a.gpart + g * a.cpg * a.D;
    count = a.cpg;
    step = a.D;
  }
  if (!dst) return;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < a.D)
#pragma unroll 4
    for (long long k = w; k < count; k += 8) v += src[k * step + c];
  sums[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < a.D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += sums[i][lane];
    dst[c] = v;
  }
}

}  // namespace

int act_grad_chunks(long long M, int N, int sms) {
  if (M <= kActNarrowRows) return 1;
  // one wave of resident blocks, one batch of rows per warp at least
  const long long across = (N + act_cols(M) - 1) / act_cols(M);
  long long c = (long long)kActBlocks * sms / across;
  const long long most = (M + 8 * kBatch - 1) / (8 * kBatch);
  c = c < most ? c : most;
  return (int)(c < 1 ? 1 : (c > 65535 ? 65535 : c));
}

namespace {
template <int ACT>
void act_grad(const dim3& grid, const __nv_bfloat16* dy, long long lddy, const __nv_bfloat16* pre,
              long long ldp, __nv_bfloat16* dpre, float* part, long long M, int N,
              cudaStream_t stream) {
  if (act_cols(M) == 32)
    act_grad_kernel<ACT, 32><<<grid, kActThreads, 0, stream>>>(dy, lddy, pre, ldp, dpre, part, M,
                                                              N);
  else
    act_grad_kernel<ACT, 256><<<grid, kActThreads, 0, stream>>>(dy, lddy, pre, ldp, dpre, part, M,
                                                               N);
}
}  // namespace

cudaError_t act_grad_launch(const __nv_bfloat16* dy, long long lddy, const __nv_bfloat16* pre,
                            long long ldp, int act, __nv_bfloat16* dpre, float* part, int chunks,
                            long long M, int N, cudaStream_t stream) {
  const dim3 grid((unsigned)((N + act_cols(M) - 1) / act_cols(M)), (unsigned)chunks);
  switch (act) {
    case kActNone: act_grad<kActNone>(grid, dy, lddy, pre, ldp, dpre, part, M, N, stream); break;
    case kActRelu: act_grad<kActRelu>(grid, dy, lddy, pre, ldp, dpre, part, M, N, stream); break;
    case kActSilu: act_grad<kActSilu>(grid, dy, lddy, pre, ldp, dpre, part, M, N, stream); break;
    case kActGelu: act_grad<kActGelu>(grid, dy, lddy, pre, ldp, dpre, part, M, N, stream); break;
    case kActGeluTanh:
      act_grad<kActGeluTanh>(grid, dy, lddy, pre, ldp, dpre, part, M, N, stream);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t colsum_launch(const ColsumArgs& a, cudaStream_t stream) {
  const long long groups = a.gpart ? a.groups : 0;
  const unsigned gy = (unsigned)(groups < 32768 ? groups : 32768);
  const long long gz = gy ? (groups + gy - 1) / gy : 1;
  if (gz > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((a.D + 31) / 32), (unsigned)a.sets + gy, (unsigned)gz);
  colsum_kernel<<<grid, 256, 0, stream>>>(a, gy);
  return cudaGetLastError();
}

}  // namespace infini
