// C ABI of the operators of a language model on the layer: argument checks,
// then the launches on the caller's stream (kernels in bucket_bias.cu,
// checkpoint.cu and sample.cu).
#include <float.h>
#include <math.h>

#include "api_checks.h"
#include "flash_gau_internal.h"

using namespace flashgau;

namespace {

constexpr size_t kAlign = 256;

// ---- relative position bias --------------------------------------------------
int check_buckets(int H, int buckets, int max_distance, int C, int causal) {
  if (H < 1 || H > 65535 || C < 1 || C > 4096) return FLASH_GAU_EINVAL;
  if (buckets < 2 || buckets > kBucketMax || (!causal && (buckets < 4 || buckets % 2 != 0)))
    return FLASH_GAU_EINVAL;
  const int near = (causal ? buckets : buckets / 2) / 2;
  return max_distance > near && max_distance <= (1 << 20) ? FLASH_GAU_OK : FLASH_GAU_EINVAL;
}

BucketProblem bucket_problem(int H, int buckets, int max_distance, int C, int causal,
                             void *stream) {
  BucketProblem q;
  q.H = H;
  q.buckets = buckets;
  q.far = max_distance;
  q.C = C;
  q.causal = causal != 0;
  q.stream = static_cast<cudaStream_t>(stream);
  return q;
}

// ---- checkpoints ---------------------------------------------------------------
int check_checkpoint(const flash_gau_residual *o, long long M, int d, int dtype) {
  if (!o || M <= 0 || d <= 0 || !io_type(dtype)) return FLASH_GAU_EINVAL;
  if (o->post != FLASH_GAU_NORM_NONE || o->gate || o->scale || o->post_g || o->post_b)
    return FLASH_GAU_EINVAL;
  if (o->norm < FLASH_GAU_NORM_NONE || o->norm > FLASH_GAU_NORM_SCALE) return FLASH_GAU_EINVAL;
  if (o->norm != FLASH_GAU_NORM_NONE && !o->norm_g) return FLASH_GAU_EINVAL;
  if (!aligned(o->norm_g, 4) || !aligned(o->norm_b, 4)) return FLASH_GAU_EINVAL;
  if (!(o->eps >= FLT_MIN) || !isfinite(o->eps)) return FLASH_GAU_EINVAL;
  if (d > kCheckpointMaxD || M > (1LL << 32)) return FLASH_GAU_ENOTSUP;
  return FLASH_GAU_OK;
}

// The spans of a checkpoint's arrays.
struct Sizes {
  size_t rows, codes, scales, g, b;
  Sizes(const flash_gau_residual *o, long long M, int d, int dtype)
      : rows((size_t)M * d * (dtype == FLASH_GAU_BF16 ? 2 : 4)),
        codes((size_t)M * d),
        scales((size_t)M * ((d + kCheckpointGroup - 1) / kCheckpointGroup) * 4),
        g((size_t)(o->norm == FLASH_GAU_NORM_LAYER ? d : 1) * 4),
        b((size_t)d * 4) {}
};

CheckpointArgs checkpoint_args(const flash_gau_residual *o, const signed char *codes,
                               const float *scales, long long M, int d) {
  CheckpointArgs a = {};
  a.codes = const_cast<signed char *>(codes);
  a.scales = const_cast<float *>(scales);
  a.norm = o->norm;
  a.norm_g = o->norm_g;
  a.norm_b = o->norm == FLASH_GAU_NORM_LAYER ? o->norm_b : nullptr;
  a.eps = o->eps;
  a.M = M;
  a.d = d;
  return a;
}

int supported() {
  int num_sms = 0;  // the device check
  return current_sms(&num_sms);
}

}  // namespace

extern "C" {

int flash_gau_bucket_bias(const float *table, int H, int buckets, int max_distance, int C,
                          int causal, float *relpos, void *stream) {
  if (!table || !relpos || !aligned(table, 4) || !aligned(relpos, 4)) return FLASH_GAU_EINVAL;
  int st = check_buckets(H, buckets, max_distance, C, causal);
  if (st != FLASH_GAU_OK) return st;
  const Span out[1] = {{relpos, (size_t)H * (2 * C - 1) * 4}};
  const Span in[1] = {{table, (size_t)H * buckets * 4}};
  if (!separate(out, in, false)) return FLASH_GAU_EINVAL;
  if ((st = supported()) != FLASH_GAU_OK) return st;
  return status_of(
      bucket_bias(bucket_problem(H, buckets, max_distance, C, causal, stream), table, relpos));
}

int flash_gau_bucket_bias_backward(const float *drelpos, int R, int H, int buckets,
                                   int max_distance, int C, int causal, float *dtable,
                                   void *stream) {
  if (!drelpos || !dtable || !aligned(drelpos, 4) || !aligned(dtable, 4)) return FLASH_GAU_EINVAL;
  if (R < 1 || R > kBucketMostShared) return FLASH_GAU_EINVAL;
  int st = check_buckets(H, buckets, max_distance, C, causal);
  if (st != FLASH_GAU_OK) return st;
  const Span out[1] = {{dtable, (size_t)H * buckets * 4}};
  const Span in[1] = {{drelpos, (size_t)R * H * (2 * C - 1) * 4}};
  if (!separate(out, in, false)) return FLASH_GAU_EINVAL;
  if ((st = supported()) != FLASH_GAU_OK) return st;
  return status_of(bucket_bias_grad(bucket_problem(H, buckets, max_distance, C, causal, stream),
                                    drelpos, R, dtable));
}

int flash_gau_checkpoint_pack(const void *h, const void *y, const flash_gau_residual *o,
                              long long M, int d, int dtype, void *r, void *n,
                              signed char *codes, float *scales, void *stream) {
  int st = check_checkpoint(o, M, d, dtype);
  if (st != FLASH_GAU_OK) return st;
  if (!h || !codes || !scales || (o->norm != FLASH_GAU_NORM_NONE) != (n != nullptr))
    return FLASH_GAU_EINVAL;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4;
  for (const void *p : {h, y, (const void *)r, (const void *)n})
    if (!aligned(p, io)) return FLASH_GAU_EINVAL;
  if (!aligned(scales, 4)) return FLASH_GAU_EINVAL;
  const Sizes z(o, M, d, dtype);
  const Span out[4] = {{r, z.rows}, {n, z.rows}, {codes, z.codes}, {scales, z.scales}};
  const Span in[4] = {{h, z.rows}, {y, z.rows}, {o->norm_g, z.g}, {o->norm_b, z.b}};
  // rows may take their inputs' place; parameters are read for every row
  const Span rows[2] = {out[0], out[1]}, packed[2] = {out[2], out[3]};
  const Span params[2] = {in[2], in[3]};
  if (!separate(out, params, false) || !separate(rows, in, true) || !separate(packed, in, false) ||
      !separate(packed, rows, false))
    return FLASH_GAU_EINVAL;
  if ((st = supported()) != FLASH_GAU_OK) return st;
  CheckpointArgs a = checkpoint_args(o, codes, scales, M, d);
  a.h = h;
  a.y = y;
  a.r = r;
  a.n = n;
  return status_of(checkpoint_pack(a, dtype, static_cast<cudaStream_t>(stream)));
}

int flash_gau_checkpoint_restore(const signed char *codes, const float *scales,
                                 const flash_gau_residual *o, long long M, int d, int dtype,
                                 void *x, void *n, void *stream) {
  int st = check_checkpoint(o, M, d, dtype);
  if (st != FLASH_GAU_OK) return st;
  if (!codes || !scales || (!x && !n) || (o->norm != FLASH_GAU_NORM_NONE) != (n != nullptr))
    return FLASH_GAU_EINVAL;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4;
  if (!aligned(x, io) || !aligned(n, io) || !aligned(scales, 4)) return FLASH_GAU_EINVAL;
  const Sizes z(o, M, d, dtype);
  const Span out[2] = {{x, z.rows}, {n, z.rows}};
  const Span in[4] = {{codes, z.codes}, {scales, z.scales}, {o->norm_g, z.g}, {o->norm_b, z.b}};
  if (!separate(out, in, false)) return FLASH_GAU_EINVAL;
  if ((st = supported()) != FLASH_GAU_OK) return st;
  CheckpointArgs a = checkpoint_args(o, codes, scales, M, d);
  a.r = x;
  a.n = n;
  return status_of(checkpoint_restore(a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t flash_gau_checkpoint_backward_workspace_bytes(long long M, int d) {
  if (M <= 0 || d <= 0 || d > kCheckpointMaxD || M > (1LL << 32)) return 0;
  return (checkpoint_part_bytes(d) + kAlign - 1) / kAlign * kAlign;
}

int flash_gau_checkpoint_backward(const void *dr, const void *dn, const signed char *codes,
                                  const float *scales, const flash_gau_residual *o, long long M,
                                  int d, int dtype, const flash_gau_residual_grads *g,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_checkpoint(o, M, d, dtype);
  if (st != FLASH_GAU_OK) return st;
  if (o->norm == FLASH_GAU_NORM_NONE || !dn || !codes || !scales || !g || !g->dh || !workspace)
    return FLASH_GAU_EINVAL;
  if (g->dy || g->dgate || g->dscale || g->dpost_g || g->dpost_b ||
      (g->dnorm_b && o->norm != FLASH_GAU_NORM_LAYER))
    return FLASH_GAU_EINVAL;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4;
  for (const void *p : {dr, dn, (const void *)g->dh})
    if (!aligned(p, io)) return FLASH_GAU_EINVAL;
  if (!aligned(scales, 4) || !aligned(g->dnorm_g, 4) || !aligned(g->dnorm_b, 4))
    return FLASH_GAU_EINVAL;
  const size_t need = flash_gau_checkpoint_backward_workspace_bytes(M, d);
  if (!aligned(workspace, kAlign) || workspace_bytes < need) return FLASH_GAU_EWORKSPACE;
  const Sizes z(o, M, d, dtype);
  const Span rows[1] = {{g->dh, z.rows}};
  const Span sums[3] = {{g->dnorm_g, z.g}, {g->dnorm_b, z.b}, {workspace, need}};
  const Span in[6] = {{dr, z.rows},         {dn, z.rows},      {codes, z.codes},
                      {scales, z.scales},   {o->norm_g, z.g},  {o->norm_b, z.b}};
  const Span grads[2] = {in[0], in[1]}, rest[4] = {in[2], in[3], in[4], in[5]};
  if (!separate(rows, grads, true) || !separate(rows, rest, false) || !separate(sums, in, false) ||
      !separate(sums, rows, false))
    return FLASH_GAU_EINVAL;
  int num_sms = 0;
  if ((st = current_sms(&num_sms)) != FLASH_GAU_OK) return st;
  CheckpointArgs a = checkpoint_args(o, codes, scales, M, d);
  a.dr = dr;
  a.dn = dn;
  a.dh = g->dh;
  a.part = static_cast<float *>(workspace);
  return status_of(checkpoint_backward(a, g->dnorm_g, g->dnorm_b, dtype, num_sms,
                                       static_cast<cudaStream_t>(stream)));
}

int flash_gau_sample(const void *logits, long long ld, long long N, int V, int dtype,
                     const float *u, const flash_gau_sampling *s, int *token, float *logp,
                     int *kept, void *stream) {
  if (!logits || !u || !s || !token || N <= 0 || V <= 0 || ld < V || !io_type(dtype))
    return FLASH_GAU_EINVAL;
  if (V > (1 << 22) || N > (1LL << 30) || ld > (1LL << 32)) return FLASH_GAU_ENOTSUP;
  const size_t io = dtype == FLASH_GAU_BF16 ? 2 : 4, n = (size_t)N;
  if (!aligned(logits, io)) return FLASH_GAU_EINVAL;
  for (const void *p : {(const void *)u, (const void *)s->temperature, (const void *)s->top_k,
                        (const void *)s->top_p, (const void *)s->min_p, (const void *)token,
                        (const void *)logp, (const void *)kept})
    if (!aligned(p, 4)) return FLASH_GAU_EINVAL;
  const Span out[3] = {{token, n * 4}, {logp, n * 4}, {kept, n * 4}};
  const Span in[6] = {{logits, ((n - 1) * (size_t)ld + V) * io}, {u, n * 4},
                      {s->temperature, n * 4}, {s->top_k, n * 4},
                      {s->top_p, n * 4}, {s->min_p, n * 4}};
  if (!separate(out, in, false)) return FLASH_GAU_EINVAL;
  int num_sms = 0;
  const int st = current_sms(&num_sms);
  if (st != FLASH_GAU_OK) return st;
  SampleArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.V = V;
  a.temperature = s->temperature;
  a.top_k = s->top_k;
  a.top_p = s->top_p;
  a.min_p = s->min_p;
  a.u = u;
  a.token = token;
  a.logp = logp;
  a.kept = kept;
  return status_of(sample(a, (int)N, dtype, num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
