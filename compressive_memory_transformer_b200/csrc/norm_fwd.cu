// norm_fwd.cu — the norms around a block, with the block's gate and the scaled residual
// stream, in one pass over the rows:
//
//   u = post(b)            (or b)             post, pre: n(v) w + c with
//   r = alpha x + gate u   (or alpha x + u)   n(v) = v / sqrt(mean v^2 + eps), or
//   h = pre(r)                                n(v) = (v - mean v) / sqrt(var v + eps)
//
// b absent: r = alpha x, so that h is the plain norm of x. Everything between the loads
// and the two stores is fp32 in registers; h is formed from the unrounded r.
// HBM-bound: x and b read once, r and h written once (131072 x 1024 bf16: 167 us = 6.4 TB/s,
// a plain copy's rate, launched back to back; 188 us = 5.7 TB/s as a pass of a program, with new
// outputs and inputs each time). A worker (threads of one row) asks for its next row before
// it works on the present one.
#include "norm_common.cuh"

namespace infini {
namespace {

constexpr int kResident = 512;  // threads per SM: 128 registers each

template <typename T, int TPR, int PIECE, int kE, bool LAYER>
__global__ void __launch_bounds__(norm_threads(TPR), kResident / norm_threads(TPR))
norm_forward_kernel(const NormArgs a) {
  using L = RowLayout<T, TPR, PIECE, kE>;
  constexpr int kWorkers = norm_threads(TPR) / TPR;
  // the row after next in L2 early: 8 rows of 1024 bf16 in flight are too few for an SM's
  // share of the bandwidth (205 -> 172 us for 131072 of them); fp32 rows have twice the
  // bytes and lose by it (170 -> 186 us for 65536)
  constexpr bool kAhead = PIECE * sizeof(T) == 16 && sizeof(T) == 2;
  // the next row in registers (32 elements per thread leave no room: from L2 then)
  constexpr bool kHold = kE == 16;
  __shared__ float2 sbuf[kWorkers][2][TPR / 32];
  const int w = threadIdx.x / TPR, t = threadIdx.x % TPR;
  RowSum<TPR> red{&sbuf[w], 1 + w};
  const float inv_d = 1.f / (float)a.D;
  const int D = a.D;
  const long long step = (long long)gridDim.x * kWorkers;
  long long row = (long long)blockIdx.x * kWorkers + w;
  RowRaw<T, TPR, PIECE, kE> nx, nb;
  if (kHold && row < a.rows) {
    nx.load(a.x, row, D, t);
    if (a.b) nb.load(a.b, row, D, t);
  }
  for (; row < a.rows; row += step) {
    if (!kHold) {
      nx.load(a.x, row, D, t);
      if (a.b) nb.load(a.b, row, D, t);
    }
    const long long ahead = row + (kHold ? 2 : 1) * step;
    if (kAhead && t == 0 && ahead < a.rows) {
      prefetch_row<T>(a.x, ahead, D);
      if (a.b) prefetch_row<T>(a.b, ahead, D);
    }
    Row<kE> v = nx.get();
    INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], both(a.alpha));
    if (a.b) {
      Row<kE> u = nb.get();
      if (kHold && row + step < a.rows) {
        nx.load(a.x, row + step, D, t);
        nb.load(a.b, row + step, D, t);
      }
      if (a.post_w) {
        normalise<L, LAYER>(u, t, D, inv_d, a.eps, red);
        const Row<kE> q = load_param<L>(a.post_w, D, t);
        if (a.post_b) {
          const Row<kE> c = load_param<L>(a.post_b, D, t);
          INFINI_EACH_PAIR u.p[i] = fma2(u.p[i], q.p[i], c.p[i]);
        } else {
          INFINI_EACH_PAIR u.p[i] = mul2(u.p[i], q.p[i]);
        }
      }
      if (a.gate) {
        const Row<kE> q = load_param<L>(a.gate + (row / a.group_rows) * D, D, t);
        INFINI_EACH_PAIR v.p[i] = fma2(u.p[i], q.p[i], v.p[i]);
      } else {
        INFINI_EACH_PAIR v.p[i] = add2(u.p[i], v.p[i]);
      }
    } else if (kHold && row + step < a.rows) {
      nx.load(a.x, row + step, D, t);
    }
    if (a.r) store_row<T, TPR, PIECE>(a.r, row, D, t, v);
    if (a.h) {
      normalise<L, LAYER>(v, t, D, inv_d, a.eps, red);
      const Row<kE> q = load_param<L>(a.pre_w, D, t);
      if (a.pre_b) {
        const Row<kE> c = load_param<L>(a.pre_b, D, t);
        INFINI_EACH_PAIR v.p[i] = fma2(v.p[i], q.p[i], c.p[i]);
      } else {
        INFINI_EACH_PAIR v.p[i] = mul2(v.p[i], q.p[i]);
      }
      store_row<T, TPR, PIECE>(a.h, row, D, t, v);
    }
  }
}

template <typename T, int TPR, int PIECE, int E>
cudaError_t launch(const NormArgs& a, int kind, int sms, cudaStream_t stream) {
  constexpr int kThreads = norm_threads(TPR), kWorkers = kThreads / TPR;
  const long long need = (a.rows + kWorkers - 1) / kWorkers;
  const long long most = (long long)sms * (kResident / kThreads);
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (kind == kNormLayer)
    norm_forward_kernel<T, TPR, PIECE, E, true><<<grid, kThreads, 0, stream>>>(a);
  else
    norm_forward_kernel<T, TPR, PIECE, E, false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Elements per thread: 16; for wide bf16 rows 32, which keeps twice the rows in work at a
// time and halves the warps of a row's sums (32768 x 4096: 213 -> 196 us, 16384 x 8192: 255
// -> 210; 65536 x 2048 would lose, 173 -> 187).
template <typename T, int PIECE>
cudaError_t by_width(const NormArgs& a, int kind, int sms, cudaStream_t stream) {
  if constexpr (PIECE * sizeof(T) == 16 && sizeof(T) == 2) {
    if (a.D > 2048) {
      return norm_tpr(a.D, 32) == 128 ? launch<T, 128, PIECE, 32>(a, kind, sms, stream)
                                      : launch<T, 256, PIECE, 32>(a, kind, sms, stream);
    }
  }
  switch (norm_tpr(a.D, 16)) {
    case 32: return launch<T, 32, PIECE, 16>(a, kind, sms, stream);
    case 64: return launch<T, 64, PIECE, 16>(a, kind, sms, stream);
    case 128: return launch<T, 128, PIECE, 16>(a, kind, sms, stream);
    case 256: return launch<T, 256, PIECE, 16>(a, kind, sms, stream);
    default: return launch<T, 512, PIECE, 16>(a, kind, sms, stream);
  }
}

bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Every row and vector starts on its pieces' size.
bool pieces_fit(const NormArgs& a, int piece, bool f32) {
  bool ok = a.D % piece == 0;
  for (const void* p : {a.x, a.b, a.dr, a.dh, static_cast<const void*>(a.r),
                        static_cast<const void*>(a.h), static_cast<const void*>(a.dx),
                        static_cast<const void*>(a.db)})
    ok = ok && on(p, (uintptr_t)piece * (f32 ? 4 : 2));
  for (const float* p : {a.gate, a.post_w, a.post_b, a.pre_w, a.pre_b})
    ok = ok && on(p, (uintptr_t)piece * 4);
  return ok;
}

}  // namespace

int norm_piece(const NormArgs& a, bool f32) {
  const int most = f32 ? 4 : 8;
  return pieces_fit(a, most, f32) ? most : pieces_fit(a, 2, f32) ? 2 : 1;
}

cudaError_t norm_forward_launch(const NormArgs& a, int kind, bool f32, int sms,
                                cudaStream_t stream) {
  const int piece = norm_piece(a, f32);
  if (f32)
    return piece == 4   ? by_width<float, 4>(a, kind, sms, stream)
           : piece == 2 ? by_width<float, 2>(a, kind, sms, stream)
                        : by_width<float, 1>(a, kind, sms, stream);
  return piece == 8   ? by_width<__nv_bfloat16, 8>(a, kind, sms, stream)
         : piece == 2 ? by_width<__nv_bfloat16, 2>(a, kind, sms, stream)
                      : by_width<__nv_bfloat16, 1>(a, kind, sms, stream);
}

}  // namespace infini
