// block_ops.h — the operators around the attention layer (linear.cu, norm_fwd.cu,
// norm_bwd.cu) as seen by their C ABI (block_api.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace infini {

// Values of infini_act_t / infini_norm_t (include/infini_attn.h).
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
enum : int { kNormRms = 0, kNormLayer = 1 };

// ---- matrix products (linear.cu) ------------------------------------------------------
// out [P][Q] = A B over a reduction of length R, both operands bf16 in global memory:
//   a_mn = false: A is stored [P][R]; true: [R][P] (rows lda apart either way)
//   b_mn = false: B is stored [Q][R]; true: [R][Q]
// then out = act(A B + bias) + residual, pre = A B + bias (each part optional).
struct GemmArgs {
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  long long lda, ldb;
  bool a_mn, b_mn;
  long long P, Q, R;
  const float* bias;  // [Q] or NULL
  int act;
  const __nv_bfloat16* res;  // NULL or [P][Q], rows ldr apart
  __nv_bfloat16* out;
  __nv_bfloat16* pre;  // NULL or [P][Q], rows ldp apart
  long long ldr, ldo, ldp;
};

cudaError_t linear_set_attributes();
// Scratch of one plain product, without bias, activation, residual or pre-activation (0 for
// most shapes). With it a launch may split the reduction over pairs of SMs.
size_t linear_gemm_scratch(long long P, long long Q, long long R, int sms);
cudaError_t linear_gemm_launch(const GemmArgs& g, void* scratch, int sms, cudaStream_t stream);

// dpre = dy * act'(pre) (bf16, only with act != none) and the column sums of the
// unrounded dpre as one row of fp32 partials per row chunk (part, only when wanted).
int act_grad_chunks(long long M, int N, int sms);
cudaError_t act_grad_launch(const __nv_bfloat16* dy, long long lddy, const __nv_bfloat16* pre,
                            long long ldp, int act, __nv_bfloat16* dpre, float* part, int chunks,
                            long long M, int N, cudaStream_t stream);

// Sums of partial vectors of D columns in a fixed order, in one launch:
//   out[s][c] = sum over k < count of part[k][s][c] (a NULL out[s] is skipped),
//   dgate[g][c] = sum over k < cpg of gpart[g][k][c] (with gpart).
// count = 0 writes zeros.
constexpr int kMaxSets = 4;
struct ColsumArgs {
  const float* part;
  float* out[kMaxSets];
  int sets, D;
  long long count;
  const float* gpart;
  float* dgate;
  long long groups, cpg;
};
cudaError_t colsum_launch(const ColsumArgs& a, cudaStream_t stream);

// ---- norms (norm_fwd.cu, norm_bwd.cu) ---------------------------------------------------
struct NormArgs {
  const void *x, *b;  // [rows][D]; b may be NULL
  const float* gate;  // [groups][D] or NULL
  const float *post_w, *post_b, *pre_w, *pre_b;  // [D] or NULL
  void *r, *h;        // forward outputs, each may be NULL
  const void *dr, *dh;   // backward inputs, each may be NULL (zero)
  void *dx, *db;         // backward outputs, each may be NULL
  float *part;           // backward: [blocks][sets][D] column partials
  float *gpart;          // backward: [groups * cpg][D] gate partials
  long long rows, group_rows;
  long long groups, cpg;  // backward: groups of rows, chunks per group
  int D;
  float alpha, eps;
};

constexpr int kMaxNormDim = 8192;
cudaError_t norm_set_attributes();
int norm_piece(const NormArgs& a, bool f32);  // elements of a row per load
cudaError_t norm_forward_launch(const NormArgs& a, int kind, bool f32, int sms,
                                cudaStream_t stream);
// Thread blocks of the backward, and chunks per gate group, for these sizes.
void norm_backward_plan(long long rows, int D, long long groups, int sms, int* blocks,
                        long long* cpg);
constexpr int norm_sets(int kind) { return kind == kNormLayer ? 4 : 2; }
cudaError_t norm_backward_launch(const NormArgs& a, int kind, bool f32, int blocks,
                                 cudaStream_t stream);
}  // namespace infini
