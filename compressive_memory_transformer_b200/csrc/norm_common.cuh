// norm_common.cuh — what the norm kernels share: the layout of a row over its threads,
// loads and stores, and sums over a row's threads.
//
// A row of D elements belongs to TPR threads of a block (a "worker"); each thread holds 8
// elements in fp32 registers. Vector layout (16-byte pieces): bf16, thread t has elements
// [8t, 8t + 8); fp32, [4t, 4t + 4) and [4 TPR + 4t, + 4), so that neighbouring threads
// read neighbouring 16-byte pieces. Scalar layout, for odd widths and rows that do not
// start on 16 bytes: element t + i TPR for i = 0..7.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "block_ops.h"
#include "sm100.cuh"

namespace infini {

constexpr int kE = 8;  // elements of a row per thread

template <typename T, int TPR, bool VEC>
struct RowLayout {
  static constexpr bool kF32 = sizeof(T) == 4;
  // First element of piece j of thread t (VEC) and the pieces' length.
  static constexpr int kPieces = VEC ? (kF32 ? 2 : 1) : kE;
  static constexpr int kPiece = kE / kPieces;
  __device__ static __forceinline__ int col(int t, int j) {
    if constexpr (VEC) return kF32 ? 4 * t + 4 * TPR * j : 8 * t;
    return t + TPR * j;
  }
};

// One row's elements of one thread as loaded (16 bytes of bf16, 32 of fp32).
template <typename T, int TPR, bool VEC>
struct RowRaw {
  using L = RowLayout<T, TPR, VEC>;
  uint32_t w[sizeof(T) == 2 ? 4 : 8];

  __device__ __forceinline__ void load(const void* base, long long row, int D, int t) {
    const T* p = static_cast<const T*>(base) + row * D;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < L::kPieces; ++j) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (L::col(t, j) < D) v = __ldcs(reinterpret_cast<const uint4*>(p + L::col(t, j)));
        w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        w[i] = L::col(t, i) < D ? reinterpret_cast<const uint32_t*>(p)[L::col(t, i)] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        const uint32_t lo = L::col(t, i) < D ? q[L::col(t, i)] : 0u;
        const uint32_t hi = L::col(t, i + 1) < D ? q[L::col(t, i + 1)] : 0u;
        w[i / 2] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[kE]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// Whether element i of thread t lies inside a row.
template <typename L>
__device__ __forceinline__ bool inside(int t, int i, int D) {
  return L::col(t, i / L::kPiece) < D;
}

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_row(void* base, long long row, int D, int t,
                                          const float (&v)[kE]) {
  using L = RowLayout<T, TPR, VEC>;
  T* p = static_cast<T*>(base) + row * D;
  if constexpr (VEC && sizeof(T) == 2) {
    if (L::col(t, 0) < D)
      *reinterpret_cast<uint4*>(p + L::col(t, 0)) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
  } else if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (L::col(t, j) < D)
        *reinterpret_cast<float4*>(p + L::col(t, j)) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (L::col(t, i) < D) {
        if constexpr (sizeof(T) == 2)
          p[L::col(t, i)] = __float2bfloat16(v[i]);
        else
          p[L::col(t, i)] = v[i];
      }
  }
}

// A vector of fp32 parameters in the row's layout (`fill` outside the row).
template <typename L, bool VEC>
__device__ __forceinline__ void load_param(const float* p, int D, int t, float (&v)[kE]) {
#pragma unroll
  for (int i = 0; i < kE; ++i) v[i] = 0.f;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kE; i += 4) {
      const int c = L::col(t, i / L::kPiece) + i % L::kPiece;
      if (c < D) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p + c));
        v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (L::col(t, i) < D) v[i] = __ldg(p + L::col(t, i));
  }
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
  __device__ __forceinline__ float sum(float a) { return sum2(a, 0.f).x; }
};

// v -> (v - mean) / sd or v / rms; elements outside the row become 0. The variance is the
// mean of the squared distances from the mean (a second sum), never E v^2 - mean^2.
template <typename L, bool LAYER, typename R>
__device__ __forceinline__ float normalise(float (&v)[kE], int t, int D, float inv_d, float eps,
                                           R& red) {
  float s = 0.f;
  if constexpr (LAYER) {
#pragma unroll
    for (int i = 0; i < kE; ++i) s += v[i];
    const float mean = red.sum(s) * inv_d;
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = inside<L>(t, i, D) ? v[i] - mean : 0.f;
    s = 0.f;
  }
#pragma unroll
  for (int i = 0; i < kE; ++i) s = fmaf(v[i], v[i], s);
  const float inv = 1.f / sqrtf(fmaf(red.sum(s), inv_d, eps));
#pragma unroll
  for (int i = 0; i < kE; ++i) v[i] *= inv;
  return inv;
}

// Threads per row for a width, and threads per block.
constexpr int norm_tpr(int D) {
  return D <= 256 ? 32 : D <= 1024 ? 128 : D <= 2048 ? 256 : D <= 4096 ? 512 : 1024;
}
constexpr int norm_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

}  // namespace infini
