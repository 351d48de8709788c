// block_api.cu — the C ABI of the operators around the attention layer
// (include/infini_attn.h): the linear layer with its epilogue, the norms with gate and
// residual, their gradients, and the block that runs them around the attention layer.
// Argument checks, scratch memory and launch sequences; the kernels are in linear.cu,
// norm_fwd.cu and norm_bwd.cu.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "infini_attn.h"
#include "block_ops.h"

namespace infini {
namespace {

typedef __nv_bfloat16 bf16;

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What a call reads or writes: n bytes from p, or (pitch > 0) rows of `width` bytes, `pitch`
// bytes apart, that end within n bytes.
struct Range {
  const void* p;
  size_t n;
  size_t width = 0, pitch = 0;
};

// Two ranges with a byte in common. Rows of one pitch are apart where their columns are, as
// slices of one wide array beside each other; other pitches are judged by the whole span.
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.n || y >= x + a.n) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  // where b's rows start between the starts of a's
  const size_t at = x <= y ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
  return at < a.width || at + b.width > a.pitch;
}

// Every output apart from the inputs and the other outputs.
bool aliased(const Range* in, int ni, const Range* out, int no) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

struct Scratch {
  void* ptr = nullptr;
  bool owned = false;
  cudaStream_t stream = nullptr;
  ~Scratch() {
    if (owned && ptr) cudaFreeAsync(ptr, stream);
  }
};

int get_scratch(Scratch& s, size_t bytes, const infini_attn_opts_t* opts, cudaStream_t stream) {
  if (bytes == 0) return INFINI_OK;
  if (opts && opts->workspace) {
    if (opts->workspace_bytes < bytes) return INFINI_ERR_NOMEM;
    if (!aligned(opts->workspace, 256)) return INFINI_ERR_ALIGN;
    s.ptr = opts->workspace;
    return INFINI_OK;
  }
  if (cudaMallocAsync(&s.ptr, bytes, stream) != cudaSuccess) {
    cudaGetLastError();
    s.ptr = nullptr;
    return INFINI_ERR_NOMEM;
  }
  s.owned = true;
  s.stream = stream;
  return INFINI_OK;
}

void record(const infini_attn_opts_t* opts, int i, cudaStream_t stream) {
  if (opts && opts->stage_events[i])
    cudaEventRecord(static_cast<cudaEvent_t>(opts->stage_events[i]), stream);
}

int status(cudaError_t e) { return e == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA; }

// The current device's SM count, after the kernels' attributes have been set on it once.
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

int prepare(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return INFINI_ERR_CUDA;
  *sms = g_sms[dev].load(std::memory_order_acquire);
  if (*sms > 0) return INFINI_OK;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1 ||
      linear_set_attributes() != cudaSuccess || norm_set_attributes() != cudaSuccess)
    return INFINI_ERR_CUDA;
  *sms = n;
  g_sms[dev].store(n, std::memory_order_release);  // the same value from every thread
  return INFINI_OK;
}

// SM count for the scratch-size queries, which need no device: the current device's, or a
// B200's without one.
int query_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices &&
      (n = g_sms[dev].load(std::memory_order_acquire)) > 0)
    return n;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// ---- linear ---------------------------------------------------------------------------

constexpr long long kMaxLd = 1ll << 36;  // a tensor map's stride is below 2^40 bytes

// Row stride of a matrix with `cols` columns: 0 means contiguous; -1 on a bad value.
long long row_stride(long long ld, long long cols) {
  if (ld == 0) return cols;
  return ld < cols || ld % 8 != 0 || ld > kMaxLd ? -1 : ld;
}

// A bf16 matrix of `rows` rows, ld elements apart.
Range matrix(const void* p, long long rows, long long cols, long long ld) {
  const size_t width = (size_t)cols * 2, pitch = (size_t)ld * 2;
  return {p, rows > 0 ? (size_t)(rows - 1) * pitch + width : 0, width, pitch};
}

int linear_sizes(long long M, int K, int N, int act) {
  if (M < 0 || K < 1 || N < 1 || M >= (1ll << 31)) return INFINI_ERR_SHAPE;
  if (K % 8 != 0 || N % 8 != 0) return INFINI_ERR_UNSUPPORTED;
  if (act < INFINI_ACT_NONE || act > INFINI_ACT_GELU_TANH) return INFINI_ERR_UNSUPPORTED;
  return INFINI_OK;
}

int linear_impl(const infini_attn_linear_t* p, cudaStream_t stream) {
  if (!p || !p->W || (p->M > 0 && (!p->x || !p->y))) return INFINI_ERR_NULL;
  int st = linear_sizes(p->M, p->K, p->N, p->act);
  if (st != INFINI_OK) return st;
  const long long ldx = row_stride(p->ldx, p->K), ldw = row_stride(p->ldw, p->N);
  const long long ldr = row_stride(p->ldr, p->N), ldy = row_stride(p->ldy, p->N);
  const long long ldp = row_stride(p->ldp, p->N);
  if (ldx < 0 || ldw < 0 || ldr < 0 || ldy < 0 || ldp < 0) return INFINI_ERR_SHAPE;
  for (const void* q : {p->x, p->W, static_cast<const void*>(p->bias), p->residual,
                        static_cast<const void*>(p->y), static_cast<const void*>(p->preact)})
    if (!aligned(q, 16)) return INFINI_ERR_ALIGN;
  // the residual may be y itself: every element is read by the thread that then writes it
  const bool in_place = p->residual == p->y && ldr == ldy;
  const Range in[4] = {matrix(p->x, p->M, p->K, ldx), matrix(p->W, p->K, p->N, ldw),
                       {p->bias, (size_t)p->N * 4},
                       matrix(in_place ? nullptr : p->residual, p->M, p->N, ldr)};
  const Range out[2] = {matrix(p->y, p->M, p->N, ldy), matrix(p->preact, p->M, p->N, ldp)};
  if (aliased(in, 4, out, 2)) return INFINI_ERR_ALIAS;
  if (p->M == 0) return INFINI_OK;
  int sms = 0;
  if ((st = prepare(&sms)) != INFINI_OK) return st;
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  g.a = static_cast<const bf16*>(p->x);
  g.b = static_cast<const bf16*>(p->W);
  g.lda = ldx;
  g.ldb = ldw;
  g.b_mn = true;
  g.P = p->M;
  g.Q = p->N;
  g.R = p->K;
  g.bias = p->bias;
  g.act = p->act;
  g.res = static_cast<const bf16*>(p->residual);
  g.ldr = ldr;
  g.out = static_cast<bf16*>(p->y);
  g.ldo = ldy;
  g.pre = static_cast<bf16*>(p->preact);
  g.ldp = ldp;
  return status(linear_gemm_launch(g, nullptr, sms, stream));
}

// Scratch of the gradient: dpre, the bias partials, the products' own.
struct GradPlan {
  size_t dpre, part, gemm;
  int chunks;
  size_t bytes() const { return dpre + part + gemm; }
};

GradPlan grad_plan(long long M, int K, int N, int act, bool dbias, bool dx, bool dW, int sms) {
  GradPlan f;
  memset(&f, 0, sizeof(f));
  f.chunks = act_grad_chunks(M, N, sms);
  if (act != INFINI_ACT_NONE) f.dpre = up256((size_t)M * N * 2);
  if (dbias && f.chunks > 1) f.part = up256((size_t)f.chunks * N * 4);
  const size_t a = dx ? linear_gemm_scratch(M, K, N, sms) : 0;
  const size_t b = dW ? linear_gemm_scratch(K, N, M, sms) : 0;
  f.gemm = up256(a > b ? a : b);
  return f;
}

int linear_backward_impl(const infini_attn_linear_grad_t* p, const infini_attn_opts_t* opts,
                         cudaStream_t stream) {
  if (!p || (!p->dx && !p->dW && !p->dbias)) return INFINI_ERR_NULL;
  int st = linear_sizes(p->M, p->K, p->N, p->act);
  if (st != INFINI_OK) return st;
  const bool act = p->act != INFINI_ACT_NONE;
  if (p->M > 0 && (!p->dy || (act && !p->preact) || (p->dx && !p->W) || (p->dW && !p->x)))
    return INFINI_ERR_NULL;
  const long long ldx = row_stride(p->ldx, p->K), ldw = row_stride(p->ldw, p->N);
  const long long ldp = row_stride(p->ldp, p->N), lddy = row_stride(p->lddy, p->N);
  const long long lddx = row_stride(p->lddx, p->K), lddw = row_stride(p->lddw, p->N);
  if (ldx < 0 || ldw < 0 || ldp < 0 || lddy < 0 || lddx < 0 || lddw < 0) return INFINI_ERR_SHAPE;
  for (const void* q : {p->x, p->W, p->preact, p->dy, static_cast<const void*>(p->dx),
                        static_cast<const void*>(p->dW), static_cast<const void*>(p->dbias)})
    if (!aligned(q, 16)) return INFINI_ERR_ALIGN;
  const Range in[4] = {matrix(p->x, p->M, p->K, ldx), matrix(p->W, p->K, p->N, ldw),
                       matrix(act ? p->preact : nullptr, p->M, p->N, ldp),
                       matrix(p->dy, p->M, p->N, lddy)};
  const Range out[3] = {matrix(p->dx, p->M, p->K, lddx), matrix(p->dW, p->K, p->N, lddw),
                        {p->dbias, (size_t)p->N * 4}};
  if (aliased(in, 4, out, 3)) return INFINI_ERR_ALIAS;
  int sms = 0;
  if ((st = prepare(&sms)) != INFINI_OK) return st;
  if (p->M == 0) {  // sums over no rows
    record(opts, 0, stream);
    if (p->dbias && cudaMemsetAsync(p->dbias, 0, (size_t)p->N * 4, stream) != cudaSuccess)
      return INFINI_ERR_CUDA;
    record(opts, 1, stream);
    if (p->dW && cudaMemset2DAsync(p->dW, (size_t)lddw * 2, 0, (size_t)p->N * 2, (size_t)p->K,
                                   stream) != cudaSuccess)
      return INFINI_ERR_CUDA;
    record(opts, 2, stream);
    return INFINI_OK;
  }
  const GradPlan f = grad_plan(p->M, p->K, p->N, p->act, p->dbias != nullptr, p->dx != nullptr,
                               p->dW != nullptr, sms);
  Scratch sc;
  if ((st = get_scratch(sc, f.bytes(), opts, stream)) != INFINI_OK) return st;
  char* base = static_cast<char*>(sc.ptr);
  const bf16* dy = static_cast<const bf16*>(p->dy);
  bf16* dpre = act ? reinterpret_cast<bf16*>(base) : nullptr;
  // one chunk's sums are dbias itself
  float* part = f.part ? reinterpret_cast<float*>(base + f.dpre) : p->dbias;
  void* gemm = f.gemm ? base + f.dpre + f.part : nullptr;
  record(opts, 0, stream);
  if (dpre || part) {
    if (act_grad_launch(dy, lddy, static_cast<const bf16*>(p->preact), ldp, p->act, dpre, part,
                        f.chunks, p->M, p->N, stream) != cudaSuccess)
      return INFINI_ERR_CUDA;
    if (f.part) {
      ColsumArgs c;
      memset(&c, 0, sizeof(c));
      c.part = part;
      c.out[0] = p->dbias;
      c.sets = 1;
      c.count = f.chunks;
      c.D = p->N;
      if (colsum_launch(c, stream) != cudaSuccess) return INFINI_ERR_CUDA;
    }
  }
  record(opts, 1, stream);
  const bf16* d = act ? dpre : dy;
  const long long ldd = act ? p->N : lddy;
  GemmArgs g;
  if (p->dx) {  // dx [M][K] = d [M][N] W^T: both stored along the reduction
    memset(&g, 0, sizeof(g));
    g.a = d;
    g.lda = ldd;
    g.b = static_cast<const bf16*>(p->W);
    g.ldb = ldw;
    g.P = p->M;
    g.Q = p->K;
    g.R = p->N;
    g.out = static_cast<bf16*>(p->dx);
    g.ldo = lddx;
    if (linear_gemm_launch(g, gemm, sms, stream) != cudaSuccess) return INFINI_ERR_CUDA;
  }
  if (p->dW) {  // dW [K][N] = x^T d: both stored across it
    memset(&g, 0, sizeof(g));
    g.a = static_cast<const bf16*>(p->x);
    g.lda = ldx;
    g.a_mn = true;
    g.b = d;
    g.ldb = ldd;
    g.b_mn = true;
    g.P = p->K;
    g.Q = p->N;
    g.R = p->M;
    g.out = static_cast<bf16*>(p->dW);
    g.ldo = lddw;
    if (linear_gemm_launch(g, gemm, sms, stream) != cudaSuccess) return INFINI_ERR_CUDA;
  }
  record(opts, 2, stream);
  return INFINI_OK;
}

// ---- norms ------------------------------------------------------------------------------

int norm_sizes(long long rows, int dim, int kind, int dtype, float eps) {
  if (rows < 0 || rows >= (1ll << 40) || dim < 1) return INFINI_ERR_SHAPE;
  if (dim > kMaxNormDim) return INFINI_ERR_UNSUPPORTED;
  if (kind != INFINI_NORM_RMS && kind != INFINI_NORM_LAYER) return INFINI_ERR_UNSUPPORTED;
  if (dtype != INFINI_DTYPE_BF16 && dtype != INFINI_DTYPE_F32) return INFINI_ERR_UNSUPPORTED;
  if (!(eps >= 0.f)) return INFINI_ERR_SHAPE;
  return INFINI_OK;
}

// What the forward and its gradient have in common: which parts there are.
int norm_parts(const infini_attn_residual_norm_t* p) {
  const int st = norm_sizes(p->rows, p->dim, p->kind, p->dtype, p->eps);
  if (st != INFINI_OK) return st;
  if (p->rows > 0 && !p->x) return INFINI_ERR_NULL;
  // without the block's output there is nothing to gate or to normalise after it; an empty
  // call has no pointers to go by
  if (p->rows > 0 && !p->b && (p->gate || p->post_weight)) return INFINI_ERR_NULL;
  if ((p->pre_bias && !p->pre_weight) || (p->post_bias && !p->post_weight)) return INFINI_ERR_NULL;
  if (p->kind == INFINI_NORM_RMS && (p->pre_bias || p->post_bias)) return INFINI_ERR_UNSUPPORTED;
  // a gate row per token of no tokens is no gate row
  const bool no_gate_rows = p->rows == 0 && p->gate_groups == 0;
  if (p->gate && !no_gate_rows && (p->gate_groups < 1 || p->gate_groups > (1ll << 31) ||
                                   p->rows % p->gate_groups != 0))
    return INFINI_ERR_SHAPE;
  const size_t e = p->dtype == INFINI_DTYPE_BF16 ? 2 : 4;
  for (const void* q : {p->x, p->b})
    if (!aligned(q, e)) return INFINI_ERR_ALIGN;
  for (const float* q : {p->gate, p->post_weight, p->post_bias, p->pre_weight, p->pre_bias})
    if (!aligned(q, 4)) return INFINI_ERR_ALIGN;
  return INFINI_OK;
}

NormArgs norm_args(const infini_attn_residual_norm_t* p) {
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = p->x;
  a.b = p->b;
  a.gate = p->gate;
  a.post_w = p->post_weight;
  a.post_b = p->post_bias;
  a.pre_w = p->pre_weight;
  a.pre_b = p->pre_bias;
  a.rows = p->rows;
  a.groups = p->gate && p->gate_groups > 0 ? p->gate_groups : 1;
  a.group_rows = p->rows / a.groups;
  a.D = p->dim;
  a.alpha = p->alpha;
  a.eps = p->eps;
  return a;
}

// The vectors a call reads, as ranges; returns how many.
int norm_vectors(const infini_attn_residual_norm_t* p, Range* r) {
  const size_t n = (size_t)p->dim * 4;
  int k = 0;
  r[k++] = {p->gate, p->gate ? n * (size_t)p->gate_groups : 0};
  for (const float* q : {p->post_weight, p->post_bias, p->pre_weight, p->pre_bias})
    r[k++] = {q, n};
  return k;
}

int residual_norm_impl(const infini_attn_residual_norm_t* p, cudaStream_t stream) {
  if (!p) return INFINI_ERR_NULL;
  int st = norm_parts(p);
  if (st != INFINI_OK) return st;
  if (p->rows > 0 && ((!p->r && !p->h) || (p->h && !p->pre_weight))) return INFINI_ERR_NULL;
  const size_t e = p->dtype == INFINI_DTYPE_BF16 ? 2 : 4;
  if (!aligned(p->r, e) || !aligned(p->h, e)) return INFINI_ERR_ALIGN;
  const size_t n = (size_t)p->rows * p->dim * e;
  Range in[7];
  int k = norm_vectors(p, in);
  // an output may be x or b itself (every element is read by the thread that then writes it)
  const void* io[2] = {p->r, p->h};
  const Range out[2] = {{p->r, n}, {p->h, n}};
  for (int i = 0; i < 2; ++i)
    for (const void* q : {p->x, p->b})
      if (io[i] != q && overlap(out[i], {q, n})) return INFINI_ERR_ALIAS;
  if (aliased(in, k, out, 2)) return INFINI_ERR_ALIAS;
  if (p->rows == 0) return INFINI_OK;
  int sms = 0;
  if ((st = prepare(&sms)) != INFINI_OK) return st;
  NormArgs a = norm_args(p);
  a.r = p->r;
  a.h = p->h;
  return status(norm_forward_launch(a, p->kind, p->dtype == INFINI_DTYPE_F32, sms, stream));
}

struct NormGradPlan {
  int blocks;
  long long cpg;
  size_t part, gpart;
};

NormGradPlan norm_grad_plan(long long rows, int dim, long long groups, int kind, bool gate,
                            int sms) {
  NormGradPlan f;
  norm_backward_plan(rows, dim, groups, sms, &f.blocks, &f.cpg);
  f.part = up256((size_t)f.blocks * norm_sets(kind) * dim * 4);
  f.gpart = gate && f.cpg > 1 ? up256((size_t)groups * f.cpg * dim * 4) : 0;
  return f;
}

int residual_norm_backward_impl(const infini_attn_residual_norm_t* p,
                                const infini_attn_residual_norm_grad_t* g,
                                const infini_attn_opts_t* opts, cudaStream_t stream) {
  if (!p || !g) return INFINI_ERR_NULL;
  int st = norm_parts(p);
  if (st != INFINI_OK) return st;
  if (p->rows > 0 && ((!g->dr && !g->dh) || (g->dh && !p->pre_weight))) return INFINI_ERR_NULL;
  if (p->rows > 0 && g->db && !p->b) return INFINI_ERR_NULL;
  if ((g->dgate && !p->gate) || (g->dpost_weight && !p->post_weight) ||
      (g->dpost_bias && !p->post_bias) || (g->dpre_weight && !p->pre_weight) ||
      (g->dpre_bias && !p->pre_bias))
    return INFINI_ERR_NULL;
  const size_t e = p->dtype == INFINI_DTYPE_BF16 ? 2 : 4;
  for (const void* q : {g->dr, g->dh, static_cast<const void*>(g->dx),
                        static_cast<const void*>(g->db)})
    if (!aligned(q, e)) return INFINI_ERR_ALIGN;
  for (const float* q : {g->dgate, g->dpost_weight, g->dpost_bias, g->dpre_weight, g->dpre_bias})
    if (!aligned(q, 4)) return INFINI_ERR_ALIGN;
  const size_t n = (size_t)p->rows * p->dim * e, nv = (size_t)p->dim * 4;
  Range in[9];
  int k = norm_vectors(p, in);
  const Range out[7] = {{g->dx, n}, {g->db, n}, {g->dgate, p->gate ? nv * (size_t)p->gate_groups : 0},
                        {g->dpost_weight, nv}, {g->dpost_bias, nv}, {g->dpre_weight, nv},
                        {g->dpre_bias, nv}};
  // dx and db may each be one of x, b, dr, dh (a row is read before it is written)
  for (int i = 0; i < 7; ++i)
    for (const void* q : {p->x, p->b, g->dr, g->dh})
      if ((i >= 2 || out[i].p != q) && overlap(out[i], {q, n})) return INFINI_ERR_ALIAS;
  if (aliased(in, k, out, 7)) return INFINI_ERR_ALIAS;
  int sms = 0;
  if ((st = prepare(&sms)) != INFINI_OK) return st;
  NormArgs a = norm_args(p);
  const bool sums = g->dpost_weight || g->dpost_bias || g->dpre_weight || g->dpre_bias;
  const NormGradPlan f =
      norm_grad_plan(p->rows, p->dim, a.groups, p->kind, g->dgate != nullptr, sms);
  Scratch sc;
  if (p->rows > 0 &&
      (st = get_scratch(sc, (sums ? f.part : 0) + f.gpart, opts, stream)) != INFINI_OK)
    return st;
  char* base = static_cast<char*>(sc.ptr);
  if (p->rows > 0) {
    a.dr = g->dr;
    a.dh = g->dh;
    a.dx = g->dx;
    a.db = g->db;
    a.cpg = f.cpg;
    a.part = sums ? reinterpret_cast<float*>(base) : nullptr;
    if (g->dgate)
      a.gpart = f.gpart ? reinterpret_cast<float*>(base + (sums ? f.part : 0)) : g->dgate;
    if (norm_backward_launch(a, p->kind, p->dtype == INFINI_DTYPE_F32, f.blocks, stream) !=
        cudaSuccess)
      return INFINI_ERR_CUDA;
  } else if (g->dgate && p->gate_groups > 0 &&
             cudaMemsetAsync(g->dgate, 0, nv * (size_t)p->gate_groups, stream) != cudaSuccess) {
    return INFINI_ERR_CUDA;
  }
  const bool gates = p->rows > 0 && f.gpart;
  if (sums || gates) {
    ColsumArgs c;
    memset(&c, 0, sizeof(c));
    if (sums) {
      c.part = a.part;
      c.sets = norm_sets(p->kind);
      c.out[0] = g->dpre_weight;
      c.out[1] = g->dpost_weight;
      if (p->kind == INFINI_NORM_LAYER) {
        c.out[2] = g->dpre_bias;
        c.out[3] = g->dpost_bias;
      }
      c.count = p->rows > 0 ? f.blocks : 0;
    }
    if (gates) {
      c.gpart = a.gpart;
      c.dgate = g->dgate;
      c.groups = a.groups;
      c.cpg = f.cpg;
    }
    c.D = p->dim;
    if (colsum_launch(c, stream) != cudaSuccess) return INFINI_ERR_CUDA;
  }
  return INFINI_OK;
}

// ---- the block ----------------------------------------------------------------------------

struct BlockPlan {
  size_t act, ff, layer;  // one [tokens][D_model] array, the MLP's middle, the layer's scratch
  size_t bytes() const { return 3 * act + ff + layer; }
};

BlockPlan block_plan(int B, long long L, int D_model, int D_ff, int H, int H_kv, int N, int d,
                     int mode) {
  const size_t tokens = (size_t)B * (size_t)L;
  return {up256(tokens * D_model * 2), up256(tokens * D_ff * 2),
          up256(infini_attn_layer_workspace_size(B, L, D_model, H, H_kv, N, d, mode))};
}

// The sizes that the block takes, for the call and for its scratch query.
int block_sizes(int B, long long L, int D_model, int D_ff, int H, int H_kv, int N, int d,
                int mode) {
  if (B < 1 || L < 1 || D_model < 1 || D_ff < 1 || H < 1 || H_kv < 1 || N < 1 || H % H_kv != 0 ||
      L >= (1ll << 31) / B)
    return INFINI_ERR_SHAPE;
  const long long tokens = B * L;
  int st = linear_sizes(tokens, D_model, D_ff, INFINI_ACT_NONE);
  if (st != INFINI_OK) return st;
  if ((st = norm_sizes(tokens, D_model, INFINI_NORM_RMS, INFINI_DTYPE_BF16, 0.f)) != INFINI_OK)
    return st;
  if ((mode != INFINI_LINEAR && mode != INFINI_DELTA) || d != 128 || D_model % 128 != 0 ||
      tokens % 128 != 0)
    return INFINI_ERR_UNSUPPORTED;
  return infini_attn_layer_workspace_size(B, L, D_model, H, H_kv, N, d, mode) == 0
             ? INFINI_ERR_SHAPE
             : INFINI_OK;
}

// Everything that the block's steps would refuse, before the first launch.
int block_checks(const infini_attn_block_t* p) {
  if (!p || !p->x || !p->y || !p->Wq || !p->Wk || !p->Wv || !p->Wo || !p->beta ||
      !p->attn_norm || !p->mlp_norm || !p->W_up || !p->W_down)
    return INFINI_ERR_NULL;
  if ((p->M_in == nullptr) != (p->z_in == nullptr) ||
      (p->M_out == nullptr) != (p->z_out == nullptr) ||
      (p->attn_post_norm_bias && !p->attn_post_norm) || (p->mlp_post_norm_bias && !p->mlp_post_norm))
    return INFINI_ERR_NULL;
  int st = block_sizes(p->B, p->L, p->D_model, p->D_ff, p->H, p->H_kv, p->N, p->d, p->mode);
  if (st != INFINI_OK) return st;
  const long long tokens = p->B * p->L;
  if ((st = linear_sizes(tokens, p->D_model, p->D_ff, p->act)) != INFINI_OK) return st;
  if ((st = norm_sizes(tokens, p->D_model, p->kind, INFINI_DTYPE_BF16, p->eps)) != INFINI_OK)
    return st;
  if (p->kind == INFINI_NORM_RMS && (p->attn_norm_bias || p->attn_post_norm_bias ||
                                     p->mlp_norm_bias || p->mlp_post_norm_bias))
    return INFINI_ERR_UNSUPPORTED;
  if ((p->attn_gate || p->mlp_gate) &&
      (p->gate_groups < 1 || p->gate_groups > tokens || tokens % p->gate_groups != 0))
    return INFINI_ERR_SHAPE;
  for (const void* q : {p->x, p->Wq, p->Wk, p->Wv, p->Wo, p->W_up, p->W_down,
                        static_cast<const void*>(p->y), static_cast<const void*>(p->b_up),
                        static_cast<const void*>(p->b_down), static_cast<const void*>(p->M_in),
                        static_cast<const void*>(p->M_out)})
    if (!aligned(q, 16)) return INFINI_ERR_ALIGN;
  const float* vectors[] = {p->attn_norm, p->attn_norm_bias, p->attn_post_norm,
                            p->attn_post_norm_bias, p->attn_gate, p->mlp_norm, p->mlp_norm_bias,
                            p->mlp_post_norm, p->mlp_post_norm_bias, p->mlp_gate};
  for (const float* q : vectors)
    if (!aligned(q, 4)) return INFINI_ERR_ALIGN;
  // y apart from everything that is read, the state apart from x and the weights
  const size_t nx = (size_t)tokens * p->D_model * 2, nf = (size_t)p->D_model * p->D_ff * 2;
  const size_t nq = (size_t)p->D_model * p->H * p->d * 2;
  const size_t nkv = (size_t)p->D_model * p->H_kv * p->d * 2;
  const size_t nv = (size_t)p->D_model * 4;
  const size_t nM = (size_t)p->B * p->H_kv * p->d * p->d * 4, nz = nM / p->d;
  Range in[20] = {{p->x, nx},       {p->Wq, nq},   {p->Wk, nkv},  {p->Wv, nkv},
                  {p->Wo, nq},      {p->W_up, nf}, {p->W_down, nf},
                  {p->b_up, (size_t)p->D_ff * 4},  {p->b_down, nv},
                  {p->beta, (size_t)p->H * 4}};
  int k = 10;
  for (const float* q : vectors)
    in[k++] = {q, q == p->attn_gate || q == p->mlp_gate ? nv * (size_t)p->gate_groups : nv};
  const Range out[3] = {{p->y, nx}, {p->M_out, nM}, {p->z_out, nz}};
  if (aliased(in, k, out, 3)) return INFINI_ERR_ALIAS;
  const Range state[2] = {{p->M_in, nM}, {p->z_in, nz}};
  return aliased(state, 2, out, 1) ? INFINI_ERR_ALIAS : INFINI_OK;
}

int block_forward_impl(const infini_attn_block_t* p, const infini_attn_opts_t* opts,
                       cudaStream_t stream) {
  int st = block_checks(p);
  if (st != INFINI_OK) return st;
  const BlockPlan f = block_plan(p->B, p->L, p->D_model, p->D_ff, p->H, p->H_kv, p->N, p->d,
                                 p->mode);
  Scratch sc;
  if ((st = get_scratch(sc, f.bytes(), opts, stream)) != INFINI_OK) return st;
  char* base = static_cast<char*>(sc.ptr);
  char *h = base, *a = base + f.act, *r = base + 2 * f.act, *m = base + 3 * f.act;
  infini_attn_residual_norm_t n;
  memset(&n, 0, sizeof(n));
  n.rows = p->B * p->L;
  n.dim = p->D_model;
  n.kind = p->kind;
  n.dtype = INFINI_DTYPE_BF16;
  n.eps = p->eps;
  // h = norm(x)
  n.x = p->x;
  n.alpha = 1.f;
  n.pre_weight = p->attn_norm;
  n.pre_bias = p->attn_norm_bias;
  n.h = h;
  if ((st = residual_norm_impl(&n, stream)) != INFINI_OK) return st;
  // a = layer(h)
  infini_attn_opts_t lo;
  memset(&lo, 0, sizeof(lo));
  lo.workspace = m + f.ff;
  lo.workspace_bytes = f.layer;
  st = infini_attn_layer_forward_ex(h, p->Wq, p->Wk, p->Wv, p->Wo, p->beta, p->M_in, p->z_in, a,
                                    p->M_out, p->z_out, p->B, p->L, p->D_model, p->H, p->H_kv,
                                    p->N, p->d, p->mode, &lo, stream);
  if (st != INFINI_OK) return st;
  record(opts, 0, stream);
  // r = alpha x + gate post(a); h = norm(r)
  n.b = a;
  n.alpha = p->alpha;
  n.gate = p->attn_gate;
  n.gate_groups = p->gate_groups;
  n.post_weight = p->attn_post_norm;
  n.post_bias = p->attn_post_norm_bias;
  n.pre_weight = p->mlp_norm;
  n.pre_bias = p->mlp_norm_bias;
  n.r = r;
  if ((st = residual_norm_impl(&n, stream)) != INFINI_OK) return st;
  record(opts, 1, stream);
  // m = act(h W_up + b_up)
  infini_attn_linear_t l;
  memset(&l, 0, sizeof(l));
  l.x = h;
  l.W = p->W_up;
  l.bias = p->b_up;
  l.y = m;
  l.M = p->B * p->L;
  l.K = p->D_model;
  l.N = p->D_ff;
  l.act = p->act;
  if ((st = linear_impl(&l, stream)) != INFINI_OK) return st;
  // y = alpha r + gate post(m W_down + b_down); a plain residual goes into the epilogue
  const bool plain = !p->mlp_gate && !p->mlp_post_norm && p->alpha == 1.f;
  l.x = m;
  l.W = p->W_down;
  l.bias = p->b_down;
  l.residual = plain ? r : nullptr;
  l.y = plain ? p->y : a;
  l.K = p->D_ff;
  l.N = p->D_model;
  l.act = INFINI_ACT_NONE;
  if ((st = linear_impl(&l, stream)) != INFINI_OK) return st;
  if (!plain) {
    n.x = r;
    n.gate = p->mlp_gate;
    n.post_weight = p->mlp_post_norm;
    n.post_bias = p->mlp_post_norm_bias;
    n.pre_weight = n.pre_bias = nullptr;
    n.r = p->y;
    n.h = nullptr;
    if ((st = residual_norm_impl(&n, stream)) != INFINI_OK) return st;
  }
  record(opts, 2, stream);
  return INFINI_OK;
}

}  // namespace
}  // namespace infini

using namespace infini;

extern "C" {

int infini_attn_linear(const infini_attn_linear_t* p, void* stream) {
  return linear_impl(p, static_cast<cudaStream_t>(stream));
}

int infini_attn_linear_backward(const infini_attn_linear_grad_t* p,
                                const infini_attn_opts_t* opts, void* stream) {
  return linear_backward_impl(p, opts, static_cast<cudaStream_t>(stream));
}

size_t infini_attn_linear_backward_workspace_size(long long M, int K, int N, int act) {
  if (linear_sizes(M, K, N, act) != INFINI_OK || M == 0) return 0;
  return grad_plan(M, K, N, act, true, true, true, query_sms()).bytes();
}

int infini_attn_residual_norm(const infini_attn_residual_norm_t* p, void* stream) {
  return residual_norm_impl(p, static_cast<cudaStream_t>(stream));
}

int infini_attn_residual_norm_backward(const infini_attn_residual_norm_t* p,
                                       const infini_attn_residual_norm_grad_t* g,
                                       const infini_attn_opts_t* opts, void* stream) {
  return residual_norm_backward_impl(p, g, opts, static_cast<cudaStream_t>(stream));
}

size_t infini_attn_residual_norm_backward_workspace_size(long long rows, int dim,
                                                         long long gate_groups, int kind) {
  if (norm_sizes(rows, dim, kind, INFINI_DTYPE_BF16, 0.f) != INFINI_OK || rows == 0) return 0;
  if (gate_groups < 0 || (gate_groups > 0 && rows % gate_groups != 0)) return 0;
  const NormGradPlan f = norm_grad_plan(rows, dim, gate_groups > 0 ? gate_groups : 1, kind,
                                        gate_groups > 0, query_sms());
  return f.part + f.gpart;
}

int infini_attn_norm(const void* x, const float* weight, const float* bias, void* h,
                     long long rows, int dim, int kind, int dtype, float eps, void* stream) {
  infini_attn_residual_norm_t n;
  memset(&n, 0, sizeof(n));
  if (!weight || (rows > 0 && !h)) return INFINI_ERR_NULL;
  n.x = x;
  n.alpha = 1.f;
  n.pre_weight = weight;
  n.pre_bias = bias;
  n.h = h;
  n.rows = rows;
  n.dim = dim;
  n.kind = kind;
  n.dtype = dtype;
  n.eps = eps;
  return residual_norm_impl(&n, static_cast<cudaStream_t>(stream));
}

int infini_attn_norm_backward(const void* x, const float* weight, const void* dh, void* dx,
                              float* dweight, float* dbias, long long rows, int dim, int kind,
                              int dtype, float eps, const infini_attn_opts_t* opts,
                              void* stream) {
  infini_attn_residual_norm_t n;
  infini_attn_residual_norm_grad_t g;
  memset(&n, 0, sizeof(n));
  memset(&g, 0, sizeof(g));
  if (!weight || (rows > 0 && !dh)) return INFINI_ERR_NULL;
  n.x = x;
  n.alpha = 1.f;
  n.pre_weight = weight;
  n.pre_bias = dbias ? weight : nullptr;  // its value does not enter the gradients
  n.rows = rows;
  n.dim = dim;
  n.kind = kind;
  n.dtype = dtype;
  n.eps = eps;
  g.dh = dh;
  g.dx = dx;
  g.dpre_weight = dweight;
  g.dpre_bias = dbias;
  return residual_norm_backward_impl(&n, &g, opts, static_cast<cudaStream_t>(stream));
}

int infini_attn_block_forward(const infini_attn_block_t* p, const infini_attn_opts_t* opts,
                              void* stream) {
  return block_forward_impl(p, opts, static_cast<cudaStream_t>(stream));
}

size_t infini_attn_block_workspace_size(int B, long long L, int D_model, int D_ff, int H,
                                        int H_kv, int N, int d, int mode) {
  if (block_sizes(B, L, D_model, D_ff, H, H_kv, N, d, mode) != INFINI_OK) return 0;
  return block_plan(B, L, D_model, D_ff, H, H_kv, N, d, mode).bytes();
}

}  // extern "C"
