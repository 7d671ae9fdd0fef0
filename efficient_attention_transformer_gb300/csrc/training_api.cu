// C ABI of the operators around the layer in a training step: argument
// checks, then the launches on the caller's stream (kernels in
// residual_norm.cu, adamw.cu and xent.cu).
#include <float.h>
#include <math.h>

#include "api_checks.h"
#include "flash_gau_internal.h"

using namespace flashgau;

namespace {

constexpr size_t kAlign = 256;

// ---- residual stream -------------------------------------------------------
int check_norm(int kind, const float *g, const float *b) {
  if (kind < FLASH_GAU_NORM_NONE || kind > FLASH_GAU_NORM_SCALE) return FLASH_GAU_EINVAL;
  if ((kind != FLASH_GAU_NORM_NONE && !g) || !aligned(g, 4) || !aligned(b, 4))
    return FLASH_GAU_EINVAL;
  return FLASH_GAU_OK;
}

int check_residual(const flash_gau_residual *o, long long M, int d, int dtype) {
  if (!o || M <= 0 || d <= 0 || !io_type(dtype)) return FLASH_GAU_EINVAL;
  // a normal number: its inverse is one too
  if (!(o->eps >= FLT_MIN) || !isfinite(o->eps) || !aligned(o->scale, 4)) return FLASH_GAU_EINVAL;
  int st = check_norm(o->post, o->post_g, o->post_b);
  if (st == FLASH_GAU_OK) st = check_norm(o->norm, o->norm_g, o->norm_b);
  if (st != FLASH_GAU_OK) return st;
  if (d > kResidualMaxD || M > (1LL << 32)) return FLASH_GAU_ENOTSUP;
  return FLASH_GAU_OK;
}

ResidualProblem residual_problem(const flash_gau_residual *o, const void *y, long long M, int d,
                                 int dtype, void *stream) {
  ResidualProblem q;
  q.o = *o;
  q.y = y;
  q.M = M;
  q.d = d;
  q.dtype = dtype;
  q.num_sms = 0;
  q.stream = static_cast<cudaStream_t>(stream);
  return q;
}

// ---- cross entropy ---------------------------------------------------------
constexpr size_t kPieceBytes = (size_t)2 << 30;  // of a piece's [tokens, V]

int check_xent(long long N, int d, int V, int dtype) {
  if (N <= 0 || d <= 0 || V <= 0 || !io_type(dtype)) return FLASH_GAU_EINVAL;
  if (N > (1LL << 30) || V > (1 << 22) || d > 65536) return FLASH_GAU_ENOTSUP;
  if (dtype == FLASH_GAU_BF16 && d % 8 != 0) return FLASH_GAU_ENOTSUP;
  return FLASH_GAU_OK;
}

size_t xent_layout(long long N, int d, int V, int dtype, bool grad, char *base, XentLayout *L) {
  const bool bf16 = dtype == FLASH_GAU_BF16;
  const size_t terms = bf16 ? 1 : 3;
  XentLayout l = {};
  size_t off = 0;
  auto take = [&](size_t bytes) -> char * {
    char *p = base ? base + off : nullptr;
    off = (off + bytes + kAlign - 1) / kAlign * kAlign;
    return p;
  };
  l.status = reinterpret_cast<int *>(take(kAlign));
  l.live = l.status + 16;
  l.done = l.status + 17;
  l.factor = reinterpret_cast<float *>(l.status + 18);
  const size_t parts = ((size_t)V + 127) / 128;
  if (xent_few(N, d, dtype, grad)) {
    l.ref = reinterpret_cast<float *>(take(8 * sizeof(float)));
    l.part = reinterpret_cast<float2 *>(take(kXentFewBlocks * 8 * sizeof(float2)));
    if (L) *L = l;
    return off;
  }
  l.ldE = ((long long)V + 63) / 64 * 64;
  l.term = bf16 ? d : (d + 63) / 64 * 64;
  // whole tiles of rows, pieces of about the same size: [rows, V] of E, or
  // without gradients an eighth of that of the sums of 128 words
  const size_t row = grad ? terms * l.ldE * 2 : 8 * parts * sizeof(float2);
  long long most = (long long)(kPieceBytes / row) / 256 * 256;
  if (most < 256) most = 256;
  const long long about = (N + most - 1) / most;
  l.piece = ((N + about - 1) / about + 255) / 256 * 256;
  const long long pieces = (N + l.piece - 1) / l.piece;
  const size_t rows = ((size_t)N + 255) / 256 * 256, n = (size_t)l.piece;
  l.index = reinterpret_cast<int *>(take(rows * 4));
  l.labels = reinterpret_cast<int *>(take(rows * 4));
  l.ref = reinterpret_cast<float *>(take(rows * 4));
  l.Xc = take(n * terms * l.term * 2);
  if (!bf16) l.Ws = take((size_t)V * terms * l.term * 2);
  l.part = reinterpret_cast<float2 *>(take(parts * n * sizeof(float2)));
  if (grad) {
    l.row_scale = reinterpret_cast<float *>(take(n * 4));
    if (bf16) l.left = reinterpret_cast<float *>(take(n * 4));
    l.E = take(n * terms * l.ldE * 2);
    l.ld_part = (d + 63) / 64 * 64;
    l.dx_part = reinterpret_cast<float *>(take(xent_dx_part_rows(l.piece, d) * l.ld_part * 4));
    l.ld_dw = (d + 3) / 4 * 4;
    if (pieces > 1 || (!bf16 && d % 4 != 0))
      l.dw_sum = reinterpret_cast<float *>(take((size_t)V * l.ld_dw * 4));
  }
  if (L) *L = l;
  return off;
}

// ---- AdamW -----------------------------------------------------------------
int check_tensor(const flash_gau_adamw_tensor &t, int state_bits, bool step) {
  if (t.n < 0) return FLASH_GAU_EINVAL;
  if (t.n == 0) return FLASH_GAU_OK;
  const size_t state = state_bits == 8 ? 1 : 4;
  if (t.n > (1LL << 40) || !t.m || !t.v || !aligned(t.m, state) || !aligned(t.v, state))
    return FLASH_GAU_EINVAL;
  if (state_bits == 8 &&
      (!t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
    return FLASH_GAU_EINVAL;
  const size_t n = (size_t)t.n, ns = state_bits == 8 ? (n + 255) / 256 * 4 : 0;
  const Span states[4] = {{t.m, n * state}, {t.v, n * state}, {ns ? t.m_scale : nullptr, ns},
                          {ns ? t.v_scale : nullptr, ns}};
  if (!step) return separate(states, {{nullptr, 0}}, false) ? FLASH_GAU_OK : FLASH_GAU_EINVAL;
  if (!t.p || !t.g || !io_type(t.g_dtype) || !isfinite(t.weight_decay) || t.weight_decay < 0.f)
    return FLASH_GAU_EINVAL;
  const size_t gs = t.g_dtype == FLASH_GAU_BF16 ? 2 : 4;
  if (!aligned(t.p, 4) || !aligned(t.copy, 2) || !aligned(t.g, gs)) return FLASH_GAU_EINVAL;
  const Span out[6] = {states[0], states[1], states[2], states[3], {t.p, n * 4}, {t.copy, n * 2}};
  const Span in[1] = {{t.g, n * gs}};
  return separate(out, in, false) ? FLASH_GAU_OK : FLASH_GAU_EINVAL;
}

}  // namespace

extern "C" {

int flash_gau_residual_norm(const void *h, const void *y, const flash_gau_residual *o, long long M,
                            int d, int dtype, void *r, void *n, void *stream) {
  int st = check_residual(o, M, d, dtype);
  if (st != FLASH_GAU_OK) return st;
  const bool norm = o->norm != FLASH_GAU_NORM_NONE;
  if (!h || norm != (n != nullptr) || (!r && !n)) return FLASH_GAU_EINVAL;
  if (!y && (o->post != FLASH_GAU_NORM_NONE || o->gate || o->scale)) return FLASH_GAU_EINVAL;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4, bytes = (size_t)M * d * io;
  for (const void *p : {h, y, (const void *)r, (const void *)n, o->gate})
    if (!aligned(p, io)) return FLASH_GAU_EINVAL;
  const Span out[2] = {{r, bytes}, {n, bytes}};
  const size_t pg = (size_t)(o->post == FLASH_GAU_NORM_LAYER ? d : 1) * 4;
  const size_t ng = (size_t)(o->norm == FLASH_GAU_NORM_LAYER ? d : 1) * 4;
  const Span in[8] = {{h, bytes},       {y, bytes},       {o->gate, bytes}, {o->scale, (size_t)d * 4},
                      {o->post_g, pg},  {o->post_b, pg},  {o->norm_g, ng},  {o->norm_b, ng}};
  // rows may take their inputs' place; parameters are read for every row
  const Span params[5] = {in[3], in[4], in[5], in[6], in[7]};
  if (!separate(out, in, true) || !separate(out, params, false)) return FLASH_GAU_EINVAL;
  ResidualProblem q = residual_problem(o, y, M, d, dtype, stream);
  if ((st = current_sms(&q.num_sms)) != FLASH_GAU_OK) return st;
  return status_of(residual_norm(q, h, r, n));
}

size_t flash_gau_residual_norm_backward_workspace_bytes(long long M, int d) {
  if (M <= 0 || d <= 0 || d > kResidualMaxD || M > (1LL << 32)) return 0;
  const size_t n = residual_norm_part_bytes(M, d);
  return (n + kAlign - 1) / kAlign * kAlign;
}

int flash_gau_residual_norm_backward(const void *dr, const void *dn, const void *r, const void *y,
                                     const flash_gau_residual *o, long long M, int d, int dtype,
                                     const flash_gau_residual_grads *g, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  int st = check_residual(o, M, d, dtype);
  if (st != FLASH_GAU_OK) return st;
  if (!g || !g->dh || !workspace) return FLASH_GAU_EINVAL;
  const bool norm = o->norm != FLASH_GAU_NORM_NONE, post = o->post != FLASH_GAU_NORM_NONE;
  if (norm != (dn != nullptr) || (norm && !r) || (!norm && !dr)) return FLASH_GAU_EINVAL;
  if ((post || o->gate || o->scale) && (!y || !g->dy)) return FLASH_GAU_EINVAL;
  // no gradients of what is not there
  if ((g->dgate && !o->gate) || (g->dscale && !o->scale) || (g->dpost_g && !post) ||
      (g->dnorm_g && !norm) || (g->dpost_b && o->post != FLASH_GAU_NORM_LAYER) ||
      (g->dnorm_b && o->norm != FLASH_GAU_NORM_LAYER))
    return FLASH_GAU_EINVAL;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4, bytes = (size_t)M * d * io;
  for (const void *p : {dr, dn, r, y, o->gate, (const void *)g->dh, (const void *)g->dy,
                        (const void *)g->dgate})
    if (!aligned(p, io)) return FLASH_GAU_EINVAL;
  for (const void *p : {g->dscale, g->dpost_g, g->dpost_b, g->dnorm_g, g->dnorm_b})
    if (!aligned(p, 4)) return FLASH_GAU_EINVAL;
  if (!aligned(workspace, kAlign) ||
      workspace_bytes < flash_gau_residual_norm_backward_workspace_bytes(M, d))
    return FLASH_GAU_EWORKSPACE;
  const size_t pg = (size_t)(o->post == FLASH_GAU_NORM_LAYER ? d : 1) * 4;
  const size_t ng = (size_t)(o->norm == FLASH_GAU_NORM_LAYER ? d : 1) * 4;
  const size_t col = (size_t)d * 4;
  const Span out[9] = {{g->dh, bytes},   {g->dy, bytes},   {g->dgate, bytes},
                       {g->dscale, col}, {g->dpost_g, pg}, {g->dpost_b, pg},
                       {g->dnorm_g, ng}, {g->dnorm_b, ng},
                       {workspace, flash_gau_residual_norm_backward_workspace_bytes(M, d)}};
  const Span in[10] = {{dr, bytes},      {dn, bytes},     {r, bytes},      {y, bytes},
                       {o->gate, bytes}, {o->scale, col}, {o->post_g, pg}, {o->post_b, pg},
                       {o->norm_g, ng},  {o->norm_b, ng}};
  // the rows of the gradients may take their inputs' place; parameters are
  // read for every row, and their gradients and the workspace written while
  // other rows are still read
  const Span sums[6] = {out[3], out[4], out[5], out[6], out[7], out[8]};
  const Span params[5] = {in[5], in[6], in[7], in[8], in[9]};
  if (!separate(out, in, true) || !separate(out, params, false) || !separate(sums, in, false))
    return FLASH_GAU_EINVAL;
  ResidualProblem q = residual_problem(o, y, M, d, dtype, stream);
  if ((st = current_sms(&q.num_sms)) != FLASH_GAU_OK) return st;
  return status_of(residual_norm_grad(q, dr, dn, r, *g, workspace));
}

size_t flash_gau_xent_workspace_bytes(long long N, int d, int V, int dtype, int grad) {
  if (check_xent(N, d, V, dtype) != FLASH_GAU_OK) return 0;
  return xent_layout(N, d, V, dtype, grad != 0, nullptr, nullptr);
}

int flash_gau_xent(const void *X, const void *W, const int *labels, long long N, int d, int V,
                   int dtype, int reduction, float scale, const flash_gau_xent_out *out,
                   void *workspace, size_t workspace_bytes, void *stream) {
  if (!X || !W || !labels || !out || !out->total || !out->loss || !workspace)
    return FLASH_GAU_EINVAL;
  if ((reduction != FLASH_GAU_MEAN && reduction != FLASH_GAU_SUM) || !isfinite(scale))
    return FLASH_GAU_EINVAL;
  int st = check_xent(N, d, V, dtype);
  if (st != FLASH_GAU_OK) return st;
  const bool bf16 = dtype == FLASH_GAU_BF16, grad = out->dX || out->dW;
  const size_t io = bf16 ? 2 : 4;
  for (const void *p : {X, W, (const void *)out->dX, (const void *)out->dW})
    if (!aligned(p, 16)) return FLASH_GAU_EINVAL;
  for (const void *p : {(const void *)labels, (const void *)out->total, (const void *)out->loss,
                        (const void *)out->lse})
    if (!aligned(p, 4)) return FLASH_GAU_EINVAL;
  XentProblem q;
  const size_t bytes = xent_layout(N, d, V, dtype, grad, static_cast<char *>(workspace), &q.L);
  if (!aligned(workspace, kAlign) || workspace_bytes < bytes) return FLASH_GAU_EWORKSPACE;
  const size_t n = (size_t)N;
  const Span outs[6] = {{out->total, 4}, {out->loss, n * 4}, {out->lse, n * 4},
                        {out->dX, n * d * io}, {out->dW, (size_t)V * d * io}, {workspace, bytes}};
  const Span in[3] = {{X, n * d * io}, {W, (size_t)V * d * io}, {labels, n * 4}};
  if (!separate(outs, in, false)) return FLASH_GAU_EINVAL;
  if ((st = current_sms(&q.num_sms)) != FLASH_GAU_OK) return st;
  q.X = X;
  q.W = W;
  q.labels = labels;
  q.N = N;
  q.d = d;
  q.V = V;
  q.mean = reduction == FLASH_GAU_MEAN;
  q.scale = scale;
  q.loss = out->loss;
  q.lse = out->lse;
  q.total = out->total;
  q.dX = out->dX;
  q.dW = out->dW;
  q.stream = static_cast<cudaStream_t>(stream);
  return status_of(xent(q, dtype));
}

int flash_gau_adamw_step(const flash_gau_adamw_tensor *tensors, int n_tensors,
                         const flash_gau_adamw_hyper *h, void *stream) {
  if (!h || n_tensors < 0 || (n_tensors && !tensors)) return FLASH_GAU_EINVAL;
  // the step's size and eps are fp32 on the device, and a subnormal eps zero
  if (!(h->lr >= 0.0) || !(h->beta1 >= 0.0 && h->beta1 < 1.0) ||
      !(h->lr / (1.0 - h->beta1) <= FLT_MAX) || !(h->beta2 >= 0.0 && h->beta2 < 1.0) ||
      !(h->eps >= FLT_MIN && h->eps <= FLT_MAX) || h->step < 1 || (h->state_bits != 8 && h->state_bits != 32) || !aligned(h->grad_scale, 4))
    return FLASH_GAU_EINVAL;
  for (int k = 0; k < n_tensors; ++k)
    if (check_tensor(tensors[k], h->state_bits, true) != FLASH_GAU_OK) return FLASH_GAU_EINVAL;
  AdamwProblem q;
  int num_sms = 0;  // the device check
  const int st = current_sms(&num_sms);
  if (st != FLASH_GAU_OK) return st;
  q.tensors = tensors;
  q.n_tensors = n_tensors;
  q.state_bits = h->state_bits;
  q.lr = h->lr;
  q.beta1 = h->beta1;
  q.beta2 = h->beta2;
  q.eps = h->eps;
  q.step = h->step;
  q.grad_scale = h->grad_scale;
  q.stream = static_cast<cudaStream_t>(stream);
  return status_of(adamw_step(q));
}

int flash_gau_adamw_moments(const flash_gau_adamw_tensor *tensors, int n_tensors,
                            float *const *m_out, float *const *v_out, void *stream) {
  if (n_tensors < 0 || (n_tensors && (!tensors || !m_out || !v_out))) return FLASH_GAU_EINVAL;
  for (int k = 0; k < n_tensors; ++k) {
    if (check_tensor(tensors[k], 8, false) != FLASH_GAU_OK) return FLASH_GAU_EINVAL;
    const flash_gau_adamw_tensor &t = tensors[k];
    if (!t.n) continue;
    if (!m_out[k] || !v_out[k] || !aligned(m_out[k], 4) || !aligned(v_out[k], 4))
      return FLASH_GAU_EINVAL;
    const size_t n = (size_t)t.n, ns = (n + 255) / 256 * 4;
    const Span out[2] = {{m_out[k], n * 4}, {v_out[k], n * 4}};
    const Span in[4] = {{t.m, n}, {t.v, n}, {t.m_scale, ns}, {t.v_scale, ns}};
    if (!separate(out, in, false)) return FLASH_GAU_EINVAL;
  }
  AdamwProblem q = {};
  int num_sms = 0;
  const int st = current_sms(&num_sms);
  if (st != FLASH_GAU_OK) return st;
  q.tensors = tensors;
  q.n_tensors = n_tensors;
  q.state_bits = 8;
  q.step = 1;
  q.stream = static_cast<cudaStream_t>(stream);
  return status_of(adamw_moments(q, m_out, v_out));
}

}  // extern "C"
