// norm_fwd.cu — the norms around a block, with the block's gate and the scaled residual
// stream, in one pass over the rows:
//
//   u = post(b)            (or b)             post, pre: n(v) w + c with
//   r = alpha x + gate u   (or alpha x + u)   n(v) = v / sqrt(mean v^2 + eps), or
//   h = pre(r)                                n(v) = (v - mean v) / sqrt(var v + eps)
//
// b absent: r = alpha x, so that h is the plain norm of x. Everything between the loads
// and the two stores is fp32 in registers; h is formed from the unrounded r.
// HBM-bound: x and b read once, r and h written once. A worker (threads of one row) asks
// for its next row before it works on the present one.
#include "norm_common.cuh"

namespace infini {
namespace {

#ifndef NF_RES
#define NF_RES 512
#endif
constexpr int kResident = NF_RES;  // threads per SM

template <typename T, int TPR, bool VEC, bool LAYER>
__global__ void __launch_bounds__(norm_threads(TPR), kResident / norm_threads(TPR))
norm_forward_kernel(const NormArgs a) {
  using L = RowLayout<T, TPR, VEC>;
  constexpr int kWorkers = norm_threads(TPR) / TPR;
  __shared__ float2 sbuf[kWorkers][2][TPR / 32];
  const int w = threadIdx.x / TPR, t = threadIdx.x % TPR;
  RowSum<TPR> red{&sbuf[w], 1 + w};
  const float inv_d = 1.f / (float)a.D;
  const int D = a.D;
  const long long step = (long long)gridDim.x * kWorkers;
  long long row = (long long)blockIdx.x * kWorkers + w;
  RowRaw<T, TPR, VEC> nx, nb;
  if (row < a.rows) {
    nx.load(a.x, row, D, t);
    if (a.b) nb.load(a.b, row, D, t);
  }
  for (; row < a.rows; row += step) {
    Row16 v = nx.get();
    INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], both(a.alpha));
    if (a.b) {
      Row16 u = nb.get();
      if (row + step < a.rows) {
        nx.load(a.x, row + step, D, t);
        nb.load(a.b, row + step, D, t);
      }
      if (a.post_w) {
        normalise<L, LAYER>(u, t, D, inv_d, a.eps, red);
        const Row16 q = load_param<L>(a.post_w, D, t);
        if (a.post_b) {
          const Row16 c = load_param<L>(a.post_b, D, t);
          INFINI_EACH_PAIR u.p[i] = fma2(u.p[i], q.p[i], c.p[i]);
        } else {
          INFINI_EACH_PAIR u.p[i] = mul2(u.p[i], q.p[i]);
        }
      }
      if (a.gate) {
        const Row16 q = load_param<L>(a.gate + (row / a.group_rows) * D, D, t);
        INFINI_EACH_PAIR v.p[i] = fma2(u.p[i], q.p[i], v.p[i]);
      } else {
        INFINI_EACH_PAIR v.p[i] = add2(u.p[i], v.p[i]);
      }
    } else if (row + step < a.rows) {
      nx.load(a.x, row + step, D, t);
    }
    if (a.r) store_row<T, TPR, VEC>(a.r, row, D, t, v);
    if (a.h) {
      normalise<L, LAYER>(v, t, D, inv_d, a.eps, red);
      const Row16 q = load_param<L>(a.pre_w, D, t);
      if (a.pre_b) {
        const Row16 c = load_param<L>(a.pre_b, D, t);
        INFINI_EACH_PAIR v.p[i] = fma2(v.p[i], q.p[i], c.p[i]);
      } else {
        INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], q.p[i]);
      }
      store_row<T, TPR, VEC>(a.h, row, D, t, v);
    }
  }
}

template <typename T, bool VEC>
cudaError_t launch(const NormArgs& a, int kind, int sms, cudaStream_t stream) {
  return with_tpr(a.D, [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    constexpr int kThreads = norm_threads(TPR), kWorkers = kThreads / TPR;
    const long long need = (a.rows + kWorkers - 1) / kWorkers;
    const long long most = (long long)sms * (kResident / kThreads);
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (kind == kNormLayer)
      norm_forward_kernel<T, TPR, VEC, true><<<grid, kThreads, 0, stream>>>(a);
    else
      norm_forward_kernel<T, TPR, VEC, false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

// Every row of every array starts on 16 bytes (and the vectors beside bf16 rows on 32).
bool norm_vectorised(const NormArgs& a, bool f32) {
  bool ok = a.D % (f32 ? 4 : 8) == 0;
  for (const void* p : {a.x, a.b, a.dr, a.dh, static_cast<const void*>(a.r),
                        static_cast<const void*>(a.h), static_cast<const void*>(a.dx),
                        static_cast<const void*>(a.db)})
    ok = ok && on(p, 16);
  for (const float* p : {a.gate, a.post_w, a.post_b, a.pre_w, a.pre_b})
    ok = ok && on(p, f32 ? 16 : 32);
  return ok;
}

cudaError_t norm_forward_launch(const NormArgs& a, int kind, bool f32, int sms,
                                cudaStream_t stream) {
  if (norm_vectorised(a, f32))
    return f32 ? launch<float, true>(a, kind, sms, stream)
               : launch<__nv_bfloat16, true>(a, kind, sms, stream);
  return f32 ? launch<float, false>(a, kind, sms, stream)
             : launch<__nv_bfloat16, false>(a, kind, sms, stream);
}

}  // namespace infini
