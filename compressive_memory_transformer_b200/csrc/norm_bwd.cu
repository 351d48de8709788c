// norm_bwd.cu — the gradients of norm_fwd.cu's pass, from its inputs x and b and the
// gradients dr and dh of its outputs. With bn = n(b), rn = n(r), and inv the factor that
// n divides by:
//
//   g = dh w_pre
//   d = dr + inv_r (g - [mean g] - rn mean(g rn))       gradient of r ([..]: layer norm)
//   dx = alpha d;  dgate = sum over the gate's rows of d u;  e = gate d
//   dw_post = sum e bn, dc_post = sum e;  g' = e w_post
//   db = inv_b (g' - [mean g'] - bn mean(g' bn))
//   dw_pre = sum dh rn, dc_pre = sum dh
//
// The statistics are formed again from x and b, which have to be read for dw_post and dgate
// anyway. HBM-bound: x, b, dr, dh read once, dx, db written once. A row's thread keeps the
// sums over rows of its columns: of d bn and of d in registers, for as long as the gate row
// stays the same (dgate = w sum d bn + c sum d; dw_post and dc_post get gate times the
// sums), the others in shared memory: with them in registers the kernel spilled 0.5 to 1 KB
// per thread. Each block leaves one row of partial sums per vector, each chunk of a gate
// group one row of dgate, and one launch adds them in a fixed order. The next row is
// asked for in L2 while the present one is worked on. 131072 x 1024 bf16: 290 us = 5.5 TB/s;
// 32768 x 4096: 370 us = 4.4 TB/s, where two rows per SM are in work and the four sums of a
// row, one after another, show.
#include "norm_common.cuh"

namespace infini {
namespace {

constexpr int kResident = 512;  // threads per SM: 128 registers each
constexpr int kE = 16;          // elements per thread

// Shared memory of a block: its sums over rows, and gate times w (layer norms: and c, and the
// unit's sum of d).
constexpr int slots_bytes(bool layer, int threads) {
  return (layer ? norm_sets(kNormLayer) + 3 : norm_sets(kNormRms) + 1) * (kE / 2) * threads * 8;
}
static_assert(slots_bytes(true, 512) <= 227 * 1024, "shared memory of a block");

// The part of a norm's gradient that both norms share: with t the gradient of n(v) and vn =
// n(v), t - [mean t] - vn mean(t vn), in place of t (to be multiplied by n's factor).
template <bool LAYER, typename R>
__device__ __forceinline__ void centre(Row<kE>& t, const Row<kE>& vn, float inv_d, R& red) {
  uint64_t s1 = 0, s2 = 0;
  INFINI_EACH_PAIR {
    s1 = fma2(t.p[i], vn.p[i], s1);
    if constexpr (LAYER) s2 = add2(s2, t.p[i]);
  }
  if constexpr (LAYER) {
    const float2 m = red.sum2(halves(s1), halves(s2));
    const uint64_t m1 = both(-m.x * inv_d), m2 = both(-m.y * inv_d);
    INFINI_EACH_PAIR t.p[i] = add2(fma2(vn.p[i], m1, t.p[i]), m2);
  } else {
    const uint64_t m1 = both(-red.sum(halves(s1)) * inv_d);
    INFINI_EACH_PAIR t.p[i] = fma2(vn.p[i], m1, t.p[i]);
  }
}

template <typename T, int TPR, int PIECE, bool LAYER>
__global__ void __launch_bounds__(norm_threads(TPR), kResident / norm_threads(TPR))
norm_backward_kernel(const NormArgs a) {
  using L = RowLayout<T, TPR, PIECE, kE>;
  constexpr int kThreads = norm_threads(TPR), kWorkers = kThreads / TPR;
  constexpr int kSets = norm_sets(LAYER ? kNormLayer : kNormRms);
  __shared__ float2 sbuf[kWorkers][2][TPR / 32];
  extern __shared__ uint64_t slots[];  // [set][pair][thread]
  const int w = threadIdx.x / TPR, t = threadIdx.x % TPR;
  RowSum<TPR> red{&sbuf[w], 1 + w};
  const int D = a.D;
  const float inv_d = 1.f / (float)D;
  // sets: 0 dw_pre, 1 dw_post, (2 dc_pre, 3 dc_post,) gate w (, gate c)
  auto slot = [&](int set, int i) -> uint64_t& {
    return slots[(set * (kE / 2) + i) * kThreads + threadIdx.x];
  };
#pragma unroll
  for (int s = 0; s < kSets; ++s)
    INFINI_EACH_PAIR slot(s, i) = 0;
  const long long units = a.groups * a.cpg;
  for (long long u0 = (long long)blockIdx.x * kWorkers + w; u0 < units;
       u0 += (long long)gridDim.x * kWorkers) {
    const long long g = u0 / a.cpg, c = u0 % a.cpg;
    const long long r0 = g * a.group_rows + a.group_rows * c / a.cpg;
    const long long r1 = g * a.group_rows + a.group_rows * (c + 1) / a.cpg;
    // gate w and gate c of this unit's rows (w, the gate, or 1 alone where the others are
    // absent): r = alpha x + (gate w) bn + gate c
    const bool shift = LAYER && a.post_b != nullptr;
    if (a.b) {
      Row<kE> q, k;
      INFINI_EACH_PAIR q.p[i] = both(1.f);
      if (a.post_w) q = load_param<L>(a.post_w, D, t);
      if (shift) k = load_param<L>(a.post_b, D, t);
      if (a.gate) {
        const Row<kE> f = load_param<L>(a.gate + g * D, D, t);
        INFINI_EACH_PAIR {
          q.p[i] = mul2(q.p[i], f.p[i]);
          if (shift) k.p[i] = mul2(k.p[i], f.p[i]);
        }
      }
      INFINI_EACH_PAIR {
        slot(kSets, i) = q.p[i];
        if (shift) slot(kSets + 1, i) = k.p[i];
      }
    }
    Row<kE> pn;  // sum over the unit's rows of d bn; of d: slot(kSets + 2)
    INFINI_EACH_PAIR {
      pn.p[i] = 0;
      if constexpr (LAYER) slot(kSets + 2, i) = 0;
    }
    for (long long row = r0; row < r1; ++row) {
      RowRaw<T, TPR, PIECE, kE> rx, rb, rr, rh;
      rx.load(a.x, row, D, t);
      if (a.b) rb.load(a.b, row, D, t);
      // dh, and dr later, when registers are free again (fp32: both later)
      if (sizeof(T) == 2 && a.dh) rh.load(a.dh, row, D, t);
      if (PIECE * sizeof(T) == 16 && t == 0 && row + 1 < r1) {
        prefetch_row<T>(a.x, row + 1, D);
        if (a.b) prefetch_row<T>(a.b, row + 1, D);
        if (a.dh) prefetch_row<T>(a.dh, row + 1, D);
        if (a.dr) prefetch_row<T>(a.dr, row + 1, D);
      }
      Row<kE> v = rx.get(), bn;
      float inv_b = 1.f;
      INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], both(a.alpha));
      if (a.b) {
        bn = rb.get();
        if (a.post_w) inv_b = normalise<L, LAYER>(bn, t, D, inv_d, a.eps, red);
        INFINI_EACH_PAIR {
          v.p[i] = fma2(slot(kSets, i), bn.p[i], v.p[i]);
          if (shift) v.p[i] = add2(v.p[i], slot(kSets + 1, i));
        }
      }
      if (a.dr) rr.load(a.dr, row, D, t);
      Row<kE> d;
      INFINI_EACH_PAIR d.p[i] = 0;
      if (a.dh) {
        if (sizeof(T) == 4) rh.load(a.dh, row, D, t);
        const uint64_t inv_r = both(normalise<L, LAYER>(v, t, D, inv_d, a.eps, red));
        Row<kE> h = rh.get();
        const Row<kE> q = load_param<L>(a.pre_w, D, t);
        INFINI_EACH_PAIR {
          slot(0, i) = fma2(h.p[i], v.p[i], slot(0, i));
          if constexpr (LAYER) slot(2, i) = add2(slot(2, i), h.p[i]);
          h.p[i] = mul2(h.p[i], q.p[i]);
        }
        centre<LAYER>(h, v, inv_d, red);
        INFINI_EACH_PAIR d.p[i] = mul2(h.p[i], inv_r);
      }
      if (a.dr) {
        const Row<kE> k = rr.get();
        INFINI_EACH_PAIR d.p[i] = add2(d.p[i], k.p[i]);
      }
      if (a.dx) {
        INFINI_EACH_PAIR v.p[i] = mul2(d.p[i], both(a.alpha));
        store_row<T, TPR, PIECE>(a.dx, row, D, t, v);
      }
      if (!a.b) continue;
      INFINI_EACH_PAIR {
        pn.p[i] = fma2(d.p[i], bn.p[i], pn.p[i]);
        if constexpr (LAYER) slot(kSets + 2, i) = add2(slot(kSets + 2, i), d.p[i]);
        d.p[i] = mul2(d.p[i], slot(kSets, i));
      }
      if (a.post_w) {
        centre<LAYER>(d, bn, inv_d, red);
        INFINI_EACH_PAIR d.p[i] = mul2(d.p[i], both(inv_b));
      }
      if (a.db) store_row<T, TPR, PIECE>(a.db, row, D, t, d);
    }
    // the unit's rows share a gate row
    if (a.post_w) {
      Row<kE> e = pn, f;
      if constexpr (LAYER) INFINI_EACH_PAIR f.p[i] = slot(kSets + 2, i);
      if (a.gate) {
        const Row<kE> q = load_param<L>(a.gate + g * D, D, t);
        INFINI_EACH_PAIR {
          e.p[i] = mul2(e.p[i], q.p[i]);
          if constexpr (LAYER) f.p[i] = mul2(f.p[i], q.p[i]);
        }
      }
      INFINI_EACH_PAIR {
        slot(1, i) = add2(slot(1, i), e.p[i]);
        if constexpr (LAYER) slot(3, i) = add2(slot(3, i), f.p[i]);
      }
    }
    if (a.gpart) {
      if (a.post_w) {
        const Row<kE> q = load_param<L>(a.post_w, D, t);
        INFINI_EACH_PAIR pn.p[i] = mul2(pn.p[i], q.p[i]);
        if (LAYER && a.post_b) {
          const Row<kE> k = load_param<L>(a.post_b, D, t);
          INFINI_EACH_PAIR pn.p[i] = fma2(slot(kSets + 2, i), k.p[i], pn.p[i]);
        }
      }
      float* dst = a.gpart + u0 * D;
      INFINI_EACH_PAIR {
        if (L::col(t, 2 * i) < D) dst[L::col(t, 2 * i)] = lo_of(pn.p[i]);
        if (L::col(t, 2 * i + 1) < D) dst[L::col(t, 2 * i + 1)] = hi_of(pn.p[i]);
      }
    }
  }
  if (!a.part) return;
  __syncthreads();
  if (w != 0) return;
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    float* dst = a.part + ((long long)blockIdx.x * kSets + s) * D;
    INFINI_EACH_PAIR {
      uint64_t v = slot(s, i);
#pragma unroll
      for (int k = 1; k < kWorkers; ++k)
        v = add2(v, slots[(s * (kE / 2) + i) * kThreads + k * TPR + t]);
      if (L::col(t, 2 * i) < D) dst[L::col(t, 2 * i)] = lo_of(v);
      if (L::col(t, 2 * i + 1) < D) dst[L::col(t, 2 * i + 1)] = hi_of(v);
    }
  }
}

// f(threads per row) for a width.
template <typename F>
cudaError_t with_tpr(int D, F&& f) {
  switch (norm_tpr(D, kE)) {
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 256: return f(std::integral_constant<int, 256>{});
    default: return f(std::integral_constant<int, 512>{});
  }
}

template <typename T, int PIECE, bool LAYER>
cudaError_t launch(const NormArgs& a, int blocks, cudaStream_t stream) {
  return with_tpr(a.D, [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value, kThreads = norm_threads(TPR);
    norm_backward_kernel<T, TPR, PIECE, LAYER>
        <<<blocks, kThreads, slots_bytes(LAYER, kThreads), stream>>>(a);
    return cudaGetLastError();
  });
}

template <typename T, int PIECE, bool LAYER>
cudaError_t allow() {
  cudaError_t e = cudaSuccess;
  for (int d : {512, 1024, 2048, 4096, 8192}) {  // one width of each number of threads
    const cudaError_t f = with_tpr(d, [](auto tpr) {
      constexpr int TPR = decltype(tpr)::value;
      return cudaFuncSetAttribute(norm_backward_kernel<T, TPR, PIECE, LAYER>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  slots_bytes(LAYER, norm_threads(TPR)));
    });
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace

void norm_backward_plan(long long rows, int D, long long groups, int sms, int* blocks,
                        long long* cpg) {
  const int threads = norm_threads(norm_tpr(D, kE)), workers = threads / norm_tpr(D, kE);
  const long long per_sm = kResident / threads;
  long long nb = (rows + workers - 1) / workers;
  if (nb > per_sm * sms) nb = per_sm * sms;
  *blocks = (int)(nb < 1 ? 1 : nb);
  const long long group_rows = rows / (groups < 1 ? 1 : groups);
  long long c = ((long long)*blocks * workers + groups - 1) / (groups < 1 ? 1 : groups);
  if (c > group_rows) c = group_rows;
  *cpg = c < 1 ? 1 : c;
}

cudaError_t norm_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (auto f : {allow<__nv_bfloat16, 8, false>, allow<__nv_bfloat16, 8, true>,
                 allow<__nv_bfloat16, 2, false>, allow<__nv_bfloat16, 2, true>,
                 allow<__nv_bfloat16, 1, false>, allow<__nv_bfloat16, 1, true>,
                 allow<float, 4, false>, allow<float, 4, true>, allow<float, 2, false>,
                 allow<float, 2, true>, allow<float, 1, false>, allow<float, 1, true>})
    if (e == cudaSuccess) e = f();
  return e;
}

namespace {
template <typename T, int MOST>
cudaError_t by_piece(const NormArgs& a, int kind, int piece, int blocks, cudaStream_t stream) {
  const bool layer = kind == kNormLayer;
  if (piece == MOST)
    return layer ? launch<T, MOST, true>(a, blocks, stream) : launch<T, MOST, false>(a, blocks, stream);
  if (piece == 2)
    return layer ? launch<T, 2, true>(a, blocks, stream) : launch<T, 2, false>(a, blocks, stream);
  return layer ? launch<T, 1, true>(a, blocks, stream) : launch<T, 1, false>(a, blocks, stream);
}
}  // namespace

cudaError_t norm_backward_launch(const NormArgs& a, int kind, bool f32, int blocks,
                                 cudaStream_t stream) {
  const int piece = norm_piece(a, f32);
  return f32 ? by_piece<float, 4>(a, kind, piece, blocks, stream)
             : by_piece<__nv_bfloat16, 8>(a, kind, piece, blocks, stream);
}

}  // namespace infini
