// norm_common.cuh — what the norm kernels share: the layout of a row over its threads,
// loads and stores, and sums over a row's threads.
//
// A row of D elements belongs to TPR threads of a block (a "worker"); each thread holds E
// (16 or 32) elements as fp32 pairs, on which the arithmetic is packed (f32x2). Elements come
// in pieces of PIECE neighbours, one load each, 16 bytes where every row starts on 16 bytes
// and is a whole number of them, fewer where widths or addresses are odd: piece j of thread t is
// the (t + j TPR)-th of the row, so that neighbouring threads read neighbouring pieces.
// Elements outside the row are held as 0.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "block_ops.h"
#include "sm100.cuh"

namespace infini {

__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// A thread's elements of one row.
template <int E>
struct Row {
  uint64_t p[E / 2];
};
#define INFINI_EACH_PAIR _Pragma("unroll") for (int i = 0; i < kE / 2; ++i)

template <typename T, int TPR, int PIECE, int E>
struct RowLayout {
  static constexpr int kE = E;
  static constexpr int kPiece = PIECE;  // elements of a piece
  static constexpr int kPieces = kE / kPiece;
  // Column of element e of thread t.
  __device__ static __forceinline__ int col(int t, int e) {
    return kPiece * (t + TPR * (e / kPiece)) + e % kPiece;
  }
};

// One row's elements of one thread as loaded.
template <typename T, int TPR, int PIECE, int kE>
struct RowRaw {
  using L = RowLayout<T, TPR, PIECE, kE>;
  uint32_t w[kE * sizeof(T) / 4];

  __device__ __forceinline__ void load(const void* base, long long row, int D, int t) {
    const T* p = static_cast<const T*>(base) + row * D;
    constexpr int kBytes = PIECE * (int)sizeof(T);
    if constexpr (kBytes == 16) {
#pragma unroll
      for (int j = 0; j < L::kPieces; ++j) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const int c = L::col(t, j * PIECE);
        if (c < D) v = __ldcs(reinterpret_cast<const uint4*>(p + c));
        w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
#pragma unroll
      for (int j = 0; j < L::kPieces; ++j) {
        uint2 v = make_uint2(0, 0);
        const int c = L::col(t, j * PIECE);
        if (c < D) v = __ldcs(reinterpret_cast<const uint2*>(p + c));
        w[2 * j] = v.x; w[2 * j + 1] = v.y;
      }
    } else if constexpr (kBytes == 4) {
#pragma unroll
      for (int j = 0; j < L::kPieces; ++j) {
        const int c = L::col(t, j * PIECE);
        w[j] = c < D ? __ldcs(reinterpret_cast<const unsigned*>(p + c)) : 0u;
      }
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const uint32_t lo = L::col(t, i) < D ? q[L::col(t, i)] : 0u;
        const uint32_t hi = L::col(t, i + 1) < D ? q[L::col(t, i + 1)] : 0u;
        w[i / 2] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ Row<kE> get() const {
    Row<kE> r;
    INFINI_EACH_PAIR {
      if constexpr (sizeof(T) == 4)
        r.p[i] = (uint64_t)w[2 * i] | ((uint64_t)w[2 * i + 1] << 32);
      else
        r.p[i] = f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    return r;
  }
};

template <typename T, int TPR, int PIECE, int kE>
__device__ __forceinline__ void store_row(void* base, long long row, int D, int t,
                                          const Row<kE>& v) {
  using L = RowLayout<T, TPR, PIECE, kE>;
  T* p = static_cast<T*>(base) + row * D;
  constexpr int kBytes = PIECE * (int)sizeof(T);
  if constexpr (kBytes == 16) {
#pragma unroll
    for (int j = 0; j < L::kPieces; ++j) {
      const int c = L::col(t, j * PIECE);
      if (c >= D) continue;
      uint4 o;
      if constexpr (sizeof(T) == 2)
        o = make_uint4(pack_bf16x2(lo_of(v.p[4 * j]), hi_of(v.p[4 * j])),
                       pack_bf16x2(lo_of(v.p[4 * j + 1]), hi_of(v.p[4 * j + 1])),
                       pack_bf16x2(lo_of(v.p[4 * j + 2]), hi_of(v.p[4 * j + 2])),
                       pack_bf16x2(lo_of(v.p[4 * j + 3]), hi_of(v.p[4 * j + 3])));
      else
        o = make_uint4((uint32_t)v.p[2 * j], (uint32_t)(v.p[2 * j] >> 32),
                       (uint32_t)v.p[2 * j + 1], (uint32_t)(v.p[2 * j + 1] >> 32));
      *reinterpret_cast<uint4*>(p + c) = o;
    }
  } else if constexpr (kBytes >= 4) {
    constexpr int kWords = kBytes / 4;
#pragma unroll
    for (int j = 0; j < L::kPieces; ++j) {
      const int c = L::col(t, j * PIECE);
      if (c >= D) continue;
      uint32_t o[kWords];
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        if constexpr (sizeof(T) == 2) {
          const uint64_t f = v.p[(PIECE * j) / 2 + k];
          o[k] = pack_bf16x2(lo_of(f), hi_of(f));
        } else {
          const uint64_t f = v.p[(PIECE * j + k) / 2];
          o[k] = (PIECE * j + k) % 2 ? (uint32_t)(f >> 32) : (uint32_t)f;
        }
      }
      if constexpr (kBytes == 8)
        *reinterpret_cast<uint2*>(p + c) = make_uint2(o[0], o[1]);
      else
        *reinterpret_cast<uint32_t*>(p + c) = o[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (L::col(t, e) < D)
        p[L::col(t, e)] = __float2bfloat16(e % 2 ? hi_of(v.p[e / 2]) : lo_of(v.p[e / 2]));
  }
}

// A vector of fp32 parameters in the row's layout.
template <typename L>
__device__ __forceinline__ Row<L::kE> load_param(const float* p, int D, int t) {
  constexpr int kE = L::kE;
  Row<kE> r;
  if constexpr (L::kPiece == 8) {
    // 32 bytes per load: a warp reads whole lines (two 16-byte loads per thread read every
    // line twice, and the L1 pipe was the busiest unit of the kernels). volatile keeps the
    // load under its condition and its caller's: the compiler may execute other asm early,
    // which for a load from an absent vector or past its end is an illegal access
#pragma unroll
    for (int e = 0; e < kE; e += 8) {
      const int c = L::col(t, e);
      float f[8] = {};
      if (c < D)
        asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]),
                       "=f"(f[6]), "=f"(f[7])
                     : "l"(p + c));
#pragma unroll
      for (int i = 0; i < 4; ++i) r.p[e / 2 + i] = f2pack(f[2 * i], f[2 * i + 1]);
    }
  } else if constexpr (L::kPiece == 2) {
    INFINI_EACH_PAIR {
      const int c = L::col(t, 2 * i);
      float2 f = make_float2(0.f, 0.f);
      if (c < D) f = __ldg(reinterpret_cast<const float2*>(p + c));
      r.p[i] = f2pack(f.x, f.y);
    }
  } else if constexpr (L::kPiece > 1) {
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const int c = L::col(t, e);
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < D) f = __ldg(reinterpret_cast<const float4*>(p + c));
      r.p[e / 2] = f2pack(f.x, f.y);
      r.p[e / 2 + 1] = f2pack(f.z, f.w);
    }
  } else {
    INFINI_EACH_PAIR r.p[i] = f2pack(L::col(t, 2 * i) < D ? __ldg(p + L::col(t, 2 * i)) : 0.f,
                                     L::col(t, 2 * i + 1) < D ? __ldg(p + L::col(t, 2 * i + 1)) : 0.f);
  }
  return r;
}

// Sums over the TPR threads of a row, the same in every thread and in a fixed order
// (butterfly inside a warp, then the warps in order). Workers of several warps exchange
// through two alternating shared-memory buffers, one barrier per sum: a warp can reach a
// buffer's next use only past the barrier of the sum in between, which every warp passes
// after it has read the buffer.
template <int TPR>
struct RowSum {
  static constexpr int kWarps = TPR / 32;
  float2 (*buf)[2][kWarps];  // this worker's
  int bar;
  int flip = 0;
  __device__ __forceinline__ float2 sum2(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (kWarps > 1) {
      const int w = (threadIdx.x % TPR) >> 5;
      if ((threadIdx.x & 31) == 0) (*buf)[flip][w] = make_float2(a, b);
      named_bar_sync((uint32_t)bar, TPR);
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float2 v = (*buf)[flip][i];
        a += v.x;
        b += v.y;
      }
      flip ^= 1;
    }
    return make_float2(a, b);
  }
  __device__ __forceinline__ float sum(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (kWarps > 1) {
      const int w = (threadIdx.x % TPR) >> 5;
      if ((threadIdx.x & 31) == 0) (*buf)[flip][w].x = a;
      named_bar_sync((uint32_t)bar, TPR);
      a = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) a += (*buf)[flip][i].x;
      flip ^= 1;
    }
    return a;
  }
};

// The sum of the two halves of a pair.
__device__ __forceinline__ float halves(uint64_t v) { return lo_of(v) + hi_of(v); }

// v -> (v - mean) / sd or v / rms; elements outside the row stay 0. The variance is the
// mean of the squared distances from the mean (a second sum), never E v^2 - mean^2.
template <typename L, bool LAYER, typename R>
__device__ __forceinline__ float normalise(Row<L::kE>& v, int t, int D, float inv_d, float eps,
                                           R& red) {
  constexpr int kE = L::kE;
  if constexpr (LAYER) {
    uint64_t s = v.p[0];
#pragma unroll
    for (int i = 1; i < kE / 2; ++i) s = add2(s, v.p[i]);
    const float mean = red.sum(halves(s)) * inv_d;
    INFINI_EACH_PAIR {
      const uint64_t c = add2(v.p[i], both(-mean));
      v.p[i] = f2pack(L::col(t, 2 * i) < D ? lo_of(c) : 0.f,
                      L::col(t, 2 * i + 1) < D ? hi_of(c) : 0.f);
    }
  }
  uint64_t s = 0;
  INFINI_EACH_PAIR s = fma2(v.p[i], v.p[i], s);
  const float inv = rsqrtf(fmaf(red.sum(halves(s)), inv_d, eps));
  INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], both(inv));
  return inv;
}

// Asks for a row's bytes in L2 ahead of their loads (rows on 16 bytes only).
template <typename T>
__device__ __forceinline__ void prefetch_row(const void* base, long long row, int D) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const T*>(base) +
                                                                  row * D),
               "r"((uint32_t)(D * sizeof(T)))
               : "memory");
}

// Threads per row for a width and a number of elements per thread, and threads per block.
constexpr int norm_tpr(int D, int E) {
  int t = 32;
  while (t * E < D) t *= 2;
  return t;
}
constexpr int norm_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

}  // namespace infini
