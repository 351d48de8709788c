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
// The statistics are formed again from x and b, which have to be read for dw_post and
// dgate anyway. HBM-bound: x, b, dr, dh read once, dx, db written once. The sums over rows
// stay in fp32 registers of the thread that holds the column, over all rows that its
// worker takes; each block leaves one row of partial sums per vector, each chunk of a
// gate group one row of dgate partials, and colsum / gate_sum add them in a fixed order.
#include "norm_common.cuh"

namespace infini {
namespace {

template <typename T, int TPR, bool VEC, bool LAYER>
__global__ void __launch_bounds__(norm_threads(TPR))
norm_backward_kernel(const NormArgs a) {
  using L = RowLayout<T, TPR, VEC>;
  constexpr int kThreads = norm_threads(TPR), kWorkers = kThreads / TPR;
  constexpr int kSets = norm_sets(LAYER ? kNormLayer : kNormRms);
  __shared__ float2 sbuf[kWorkers][2][TPR / 32];
  __shared__ float comb[kWorkers > 1 ? kThreads * kE : 1];
  const int w = threadIdx.x / TPR, t = threadIdx.x % TPR;
  RowSum<TPR> red{&sbuf[w], 1 + w};
  const int D = a.D;
  const float inv_d = 1.f / (float)D;
  // 0: pre weight, 1: post weight, 2: pre bias, 3: post bias
  float acc[kSets][kE] = {};
  const long long units = a.groups * a.cpg;
  for (long long u0 = (long long)blockIdx.x * kWorkers + w; u0 < units;
       u0 += (long long)gridDim.x * kWorkers) {
    const long long g = u0 / a.cpg, c = u0 % a.cpg;
    const long long r0 = g * a.group_rows + a.group_rows * c / a.cpg;
    const long long r1 = g * a.group_rows + a.group_rows * (c + 1) / a.cpg;
    float ag[kE] = {};
    for (long long row = r0; row < r1; ++row) {
      RowRaw<T, TPR, VEC> raw;
      float q[kE], u[kE], bn[kE], v[kE], d[kE];
      float inv_b = 1.f;
      raw.load(a.x, row, D, t);
      raw.get(v);
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        v[i] *= a.alpha;
        d[i] = u[i] = bn[i] = 0.f;
      }
      if (a.b) {
        raw.load(a.b, row, D, t);
        raw.get(bn);
        if (a.post_w) {
          inv_b = normalise<L, LAYER>(bn, t, D, inv_d, a.eps, red);
          load_param<L, VEC>(a.post_w, D, t, q);
#pragma unroll
          for (int i = 0; i < kE; ++i) u[i] = bn[i] * q[i];
          if (a.post_b) {
            load_param<L, VEC>(a.post_b, D, t, q);
#pragma unroll
            for (int i = 0; i < kE; ++i) u[i] += q[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < kE; ++i) u[i] = bn[i];
        }
        if (a.gate) {
          load_param<L, VEC>(a.gate + g * D, D, t, q);
#pragma unroll
          for (int i = 0; i < kE; ++i) v[i] = fmaf(q[i], u[i], v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kE; ++i) v[i] += u[i];
        }
      }
      if (a.dr) {
        raw.load(a.dr, row, D, t);
        raw.get(d);
      }
      if (a.dh) {
        float p[kE];
        const float inv_r = normalise<L, LAYER>(v, t, D, inv_d, a.eps, red);
        raw.load(a.dh, row, D, t);
        raw.get(p);
        load_param<L, VEC>(a.pre_w, D, t, q);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          acc[0][i] = fmaf(p[i], v[i], acc[0][i]);
          if constexpr (LAYER) acc[2][i] += p[i];
          p[i] *= q[i];
          s1 = fmaf(p[i], v[i], s1);
          s2 += p[i];
        }
        const float2 m = red.sum2(s1, s2);
        const float m1 = m.x * inv_d, m2 = LAYER ? m.y * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (inside<L>(t, i, D)) d[i] = fmaf(inv_r, p[i] - m2 - v[i] * m1, d[i]);
      }
      if (a.dx) {
#pragma unroll
        for (int i = 0; i < kE; ++i) v[i] = a.alpha * d[i];
        store_row<T, TPR, VEC>(a.dx, row, D, t, v);
      }
      if (!a.b) continue;
      if (a.gate) {
        load_param<L, VEC>(a.gate + g * D, D, t, q);
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          ag[i] = fmaf(d[i], u[i], ag[i]);
          d[i] *= q[i];
        }
      }
      if (a.post_w) {
        load_param<L, VEC>(a.post_w, D, t, q);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          acc[1][i] = fmaf(d[i], bn[i], acc[1][i]);
          if constexpr (LAYER) acc[3][i] += d[i];
          d[i] *= q[i];
          s1 = fmaf(d[i], bn[i], s1);
          s2 += d[i];
        }
        const float2 m = red.sum2(s1, s2);
        const float m1 = m.x * inv_d, m2 = LAYER ? m.y * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) d[i] = inv_b * (d[i] - m2 - bn[i] * m1);
      }
      if (a.db) store_row<T, TPR, VEC>(a.db, row, D, t, d);
    }
    if (a.gpart) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (inside<L>(t, i, D))
          a.gpart[u0 * D + L::col(t, i / L::kPiece) + i % L::kPiece] = ag[i];
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    float* dst = a.part + ((long long)blockIdx.x * kSets + s) * D;
    if constexpr (kWorkers > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kE; ++i) comb[i * kThreads + threadIdx.x] = acc[s][i];
      __syncthreads();
      if (w == 0) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          float v = acc[s][i];
#pragma unroll
          for (int k = 1; k < kWorkers; ++k) v += comb[i * kThreads + k * TPR + t];
          if (inside<L>(t, i, D)) dst[L::col(t, i / L::kPiece) + i % L::kPiece] = v;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (inside<L>(t, i, D)) dst[L::col(t, i / L::kPiece) + i % L::kPiece] = acc[s][i];
    }
  }
}

template <typename T, int TPR, bool VEC>
cudaError_t launch(const NormArgs& a, int kind, int blocks, cudaStream_t stream) {
  constexpr int kThreads = norm_threads(TPR);
  if (kind == kNormLayer)
    norm_backward_kernel<T, TPR, VEC, true><<<blocks, kThreads, 0, stream>>>(a);
  else
    norm_backward_kernel<T, TPR, VEC, false><<<blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t by_width(const NormArgs& a, int kind, int blocks, cudaStream_t stream) {
  switch (norm_tpr(a.D)) {
    case 32: return launch<T, 32, VEC>(a, kind, blocks, stream);
    case 128: return launch<T, 128, VEC>(a, kind, blocks, stream);
    case 256: return launch<T, 256, VEC>(a, kind, blocks, stream);
    case 512: return launch<T, 512, VEC>(a, kind, blocks, stream);
    default: return launch<T, 1024, VEC>(a, kind, blocks, stream);
  }
}

__global__ void __launch_bounds__(256)
gate_sum_kernel(const float* __restrict__ gpart, float* __restrict__ dgate, long long cpg, int D) {
  __shared__ float sums[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const long long g = blockIdx.y + (long long)blockIdx.z * gridDim.y;
  float v = 0.f;
  if (c < D)
#pragma unroll 4
    for (long long k = w; k < cpg; k += 8) v += gpart[(g * cpg + k) * D + c];
  sums[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += sums[i][lane];
    dgate[g * D + c] = v;
  }
}

}  // namespace

void norm_backward_plan(long long rows, int D, long long groups, int sms, int* blocks,
                        long long* cpg) {
  const int threads = norm_threads(norm_tpr(D)), workers = threads / norm_tpr(D);
  const long long per_sm = 1024 / threads;
  long long nb = (rows + workers - 1) / workers;
  if (nb > per_sm * sms) nb = per_sm * sms;
  *blocks = (int)(nb < 1 ? 1 : nb);
  const long long group_rows = rows / (groups < 1 ? 1 : groups);
  long long c = ((long long)*blocks * workers + groups - 1) / (groups < 1 ? 1 : groups);
  if (c > group_rows) c = group_rows;
  *cpg = c < 1 ? 1 : c;
}

cudaError_t norm_backward_launch(const NormArgs& a, int kind, bool f32, int blocks,
                                 cudaStream_t stream) {
  if (norm_vectorised(a, f32))
    return f32 ? by_width<float, true>(a, kind, blocks, stream)
               : by_width<__nv_bfloat16, true>(a, kind, blocks, stream);
  return f32 ? by_width<float, false>(a, kind, blocks, stream)
             : by_width<__nv_bfloat16, false>(a, kind, blocks, stream);
}

cudaError_t gate_sum_launch(const float* gpart, float* dgate, long long groups, long long cpg,
                            int D, cudaStream_t stream) {
  // the groups over the grid's second and third axes (65535 rows each)
  const unsigned gy = (unsigned)(groups < 32768 ? groups : 32768);
  if (groups % gy) {  // whole layers of gy groups, then the rest
    const long long head = groups / gy * gy;
    const cudaError_t e = gate_sum_launch(gpart, dgate, head, cpg, D, stream);
    if (e != cudaSuccess) return e;
    return gate_sum_launch(gpart + head * cpg * D, dgate + head * D, groups - head, cpg, D, stream);
  }
  const long long gz = groups / gy;
  if (gz > 65535) return cudaErrorInvalidValue;
  gate_sum_kernel<<<dim3((unsigned)((D + 31) / 32), gy, (unsigned)gz), 256, 0, stream>>>(
      gpart, dgate, cpg, D);
  return cudaGetLastError();
}

}  // namespace infini
