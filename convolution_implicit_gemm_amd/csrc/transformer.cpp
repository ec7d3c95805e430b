// Entry points of include/fusedconv_transformer.h: checks, handles, dispatch.
#include <math.h>
#include <stdint.h>

#include <new>

#include "checks.h"

struct fusedconv_layer_norm {
  fc::NormProblem p;
  int32_t has_weight, has_bias;
  size_t workspace;
};
struct fusedconv_rotary {
  fc::RotaryProblem p;
};
struct fusedconv_attention {
  fc::AttnParams p;
  fc::AttnPlan plan;
};

using namespace fc;

extern "C" {

// ------------------------------------------------------------------ layer norm

int fusedconv_layer_norm_create(const fusedconv_layer_norm_desc* d, fusedconv_layer_norm** out) {
  if (out) *out = nullptr;
  if (!d || !out) return fail(FUSEDCONV_ERR_NULL_ARG, "desc and out must not be NULL");
  if (!known(d->dtype)) return fail(FUSEDCONV_ERR_DTYPE, "dtype is not float32, float16 or bfloat16");
  if (d->n < 0 || d->c < 1 || d->inner < 1)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "n must be >= 0, c and inner >= 1");
  if (!(d->eps > 0.0f) || !isfinite(d->eps))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "eps must be positive and finite");
  if (d->c > (1 << 24) || d->inner > INT32_MAX / 2 || product(1, d->c, d->inner, INT32_MAX / 4) < 0 ||
      product(d->n, d->c, d->inner, kMaxElements) < 0 || d->n > INT32_MAX / 2 ||
      (d->inner > 1 && product(d->n, d->inner / 32 + 1, 1, INT32_MAX / 2) < 0))
    return fail(FUSEDCONV_ERR_TOO_LARGE, "X exceeds the index limits");
  const int64_t row = d->c * d->inner;
  if (d->n > 1 && (d->x_stride < row || d->dy_stride < row))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "x_stride and dy_stride must be at least c * inner");
  if (d->n > 1 && (d->x_stride > kMaxElements / d->n || d->dy_stride > kMaxElements / d->n))
    return fail(FUSEDCONV_ERR_TOO_LARGE, "X exceeds the index limits");
  fusedconv_layer_norm* h = new (std::nothrow) fusedconv_layer_norm();
  if (!h) return fail(FUSEDCONV_ERR_ALLOC, "out of host memory");
  h->p = {d->dtype, d->n, d->c, d->inner, d->n > 1 ? d->x_stride : row,
          d->n > 1 ? d->dy_stride : row, d->eps};
  h->has_weight = d->has_weight != 0;
  h->has_bias = d->has_bias != 0;
  h->workspace = fc::norm_workspace(h->p);
  *out = h;
  fc::clear_last_error();
  return FUSEDCONV_OK;
}

int fusedconv_layer_norm_workspace_size(const fusedconv_layer_norm* h, size_t* bytes) {
  if (!h || !bytes) return fail(FUSEDCONV_ERR_NULL_ARG, "NULL argument");
  *bytes = h->workspace;
  return FUSEDCONV_OK;
}

int fusedconv_layer_norm_forward(const fusedconv_layer_norm* h, const void* x, const void* weight,
                                 const void* bias, void* y, float* mean, float* rstd,
                                 void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  if (!weight != !h->has_weight || !bias != !h->has_bias)
    return fail(FUSEDCONV_ERR_NULL_ARG, "weight and bias are given iff they were declared");
  if (!mean != !rstd) return fail(FUSEDCONV_ERR_NULL_ARG, "give both mean and rstd or neither");
  if (h->p.n == 0) return FUSEDCONV_OK;
  if (!x || !y) return fail(FUSEDCONV_ERR_NULL_ARG, "x and y are required");
  if (!aligned16(x) || !aligned16(y) || !aligned16(weight) || !aligned16(bias) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  const int64_t es = elem_size(h->p.dtype), row = h->p.c * h->p.inner * es;
  const bool in_place = x == y && h->p.x_stride * es == row;
  if (!in_place && rows_meet(x, h->p.n, row, h->p.x_stride * es, y, h->p.n * row))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "y is x, both contiguous, or overlaps it nowhere");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  fc::NormArgs a{};
  a.x = x; a.w = weight; a.b = bias; a.out = y; a.mean = mean; a.rstd = rstd; a.stream = stream;
  a.in_place = in_place;
  return launched([&] { return fc::launch_norm_forward(h->p, a); });
}

int fusedconv_layer_norm_backward(const fusedconv_layer_norm* h, const void* dy, const void* x,
                                  const void* weight, const float* mean, const float* rstd,
                                  void* dx, float* dweight, float* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  if (!weight != !h->has_weight)
    return fail(FUSEDCONV_ERR_NULL_ARG, "weight is given iff it was declared");
  if (h->p.n > 0 && (!dy || !x || !mean || !rstd || !dx))
    return fail(FUSEDCONV_ERR_NULL_ARG, "dy, x, mean, rstd and dx are required");
  if (!aligned16(dy) || !aligned16(x) || !aligned16(weight) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !aligned16(dx) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4) ||
      !aligned16(workspace))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (h->workspace > 0 && (dweight || dbias) && (!workspace || workspace_bytes < h->workspace))
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_layer_norm_workspace_size() reports");
  const int64_t es = elem_size(h->p.dtype), row = h->p.c * h->p.inner * es;
  if (h->p.n > 0 && (rows_meet(x, h->p.n, row, h->p.x_stride * es, dx, h->p.n * row) ||
                     rows_meet(dy, h->p.n, row, h->p.dy_stride * es, dx, h->p.n * row)))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "dx must not overlap x or dy");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  fc::NormArgs a{};
  a.x = x; a.dy = dy; a.w = weight; a.out = dx;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dw = dweight; a.db = dbias; a.part = (float*)workspace; a.stream = stream;
  return launched([&] { return fc::launch_norm_backward(h->p, a); });
}

void fusedconv_layer_norm_destroy(fusedconv_layer_norm* h) { delete h; }

// ---------------------------------------------------------------------- rotary

int fusedconv_rotary_create(const fusedconv_rotary_desc* d, fusedconv_rotary** out) {
  if (out) *out = nullptr;
  if (!d || !out) return fail(FUSEDCONV_ERR_NULL_ARG, "desc and out must not be NULL");
  if (!known(d->dtype)) return fail(FUSEDCONV_ERR_DTYPE, "dtype is not float32, float16 or bfloat16");
  if (d->position_dtype < FUSEDCONV_POS_I32 || d->position_dtype > FUSEDCONV_POS_F32)
    return fail(FUSEDCONV_ERR_DTYPE, "positions are not int32, int64 or float32");
  if (d->batch < 0 || d->len < 0 || d->heads < 1 || d->kv_heads < 0)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "batch, len, kv_heads must be >= 0, heads >= 1");
  const int64_t es = elem_size(d->dtype);
  if (d->head_dim < 1 || d->head_dim % (16 / es) != 0)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "a head must be whole 16-byte pieces");
  if (d->pairs < 1 || d->pairs > d->head_dim / 2)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "pairs must be in [1, head_dim / 2]");
  if (d->num_axes < 1 || d->num_axes > 8)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "num_axes must be in [1, 8]");
  if (d->head_dim > 4096 || d->heads > (1 << 16) || d->kv_heads > (1 << 16) ||
      d->len > INT32_MAX / 16 || product(d->batch, d->len, 1, INT32_MAX) < 0 ||
      product(d->batch, d->len, (d->heads + d->kv_heads) * d->head_dim, kMaxElements) < 0)
    return fail(FUSEDCONV_ERR_TOO_LARGE, "Q or K exceeds the index limits");
  if (d->position_batch_stride != 0 && d->position_batch_stride != d->len * d->num_axes &&
      d->batch > 1)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "position_batch_stride is len * num_axes, or 0");
  if (!strides_ok(d->q_strides, d->batch, d->len, d->heads, es) ||
      !strides_ok(d->q_out_strides, d->batch, d->len, d->heads, es) ||
      (d->kv_heads && (!strides_ok(d->k_strides, d->batch, d->len, d->kv_heads, es) ||
                       !strides_ok(d->k_out_strides, d->batch, d->len, d->kv_heads, es))))
    return fail(FUSEDCONV_ERR_ALIGNMENT, "strides must be non-negative, whole 16-byte pieces and within the index limits");
  if (!apart(d->q_out_strides, d->batch, d->len, d->heads, d->head_dim) ||
      (d->kv_heads && !apart(d->k_out_strides, d->batch, d->len, d->kv_heads, d->head_dim)))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "an output's strides make its elements overlap");
  fusedconv_rotary* h = new (std::nothrow) fusedconv_rotary();
  if (!h) return fail(FUSEDCONV_ERR_ALLOC, "out of host memory");
  h->p.d = *d;
  *out = h;
  fc::clear_last_error();
  return FUSEDCONV_OK;
}

int fusedconv_rotary_run(const fusedconv_rotary* h, const void* q, const void* k,
                         const void* positions, const float* inv_freq, const int32_t* axes,
                         void* q_out, void* k_out, void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  const fusedconv_rotary_desc& d = h->p.d;
  if (d.batch == 0 || d.len == 0) return FUSEDCONV_OK;
  if (!q || !q_out || !positions || !inv_freq || !axes || (d.kv_heads && (!k || !k_out)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned_to(positions, d.position_dtype == FUSEDCONV_POS_I64 ? 8 : 4) ||
      !aligned_to(inv_freq, 4) || !aligned_to(axes, 4))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  fc::RotaryArgs a{q, k, positions, inv_freq, axes, q_out, k_out, stream};
  return launched([&] { return fc::launch_rotary(h->p, a); });
}

void fusedconv_rotary_destroy(fusedconv_rotary* h) { delete h; }

// ------------------------------------------------------------------- attention

int fusedconv_attention_create(const fusedconv_attention_desc* d, fusedconv_attention** out) {
  if (out) *out = nullptr;
  if (!d || !out) return fail(FUSEDCONV_ERR_NULL_ARG, "desc and out must not be NULL");
  if (!known(d->dtype)) return fail(FUSEDCONV_ERR_DTYPE, "dtype is not float32, float16 or bfloat16");
  if (d->batch < 0 || d->q_len < 0 || d->k_len < 0 || d->heads < 1 || d->kv_heads < 1)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "lengths must be >= 0, heads >= 1");
  if (d->heads % d->kv_heads != 0)
    return fail(FUSEDCONV_ERR_GROUP, "heads must be a multiple of kv_heads");
  if (d->head_dim < 8 || d->head_dim > 128 || d->head_dim % 8 != 0)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "head_dim must be a multiple of 8, at most 128");
  if (!isfinite(d->scale)) return fail(FUSEDCONV_ERR_ATTR_VALUE, "scale must be finite");
  if (d->window_left < -1 || d->window_right < -1)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "window limits must be >= -1");
  constexpr int64_t kMaxLen = 1 << 28;
  if (d->q_len > kMaxLen || d->k_len > kMaxLen || d->heads > (1 << 16) ||
      product(d->batch, d->heads, 1, 1 << 24) < 0 ||
      product(d->batch, d->q_len, d->heads * d->head_dim, kMaxElements) < 0 ||
      product(d->batch, d->k_len, d->kv_heads * d->head_dim, kMaxElements) < 0 ||
      product(d->batch, d->heads, d->q_len / 32 + d->k_len / 32 + 4, INT32_MAX / 2) < 0)
    return fail(FUSEDCONV_ERR_TOO_LARGE, "a tensor exceeds the index limits");
  const int64_t es = elem_size(d->dtype);
  const int64_t* qs[] = {d->q_strides, d->o_strides, d->do_strides, d->dq_strides};
  const int64_t* ks[] = {d->k_strides, d->v_strides, d->dk_strides, d->dv_strides};
  for (const int64_t* s : qs)
    if (!strides_ok(s, d->batch, d->q_len, d->heads, es))
      return fail(FUSEDCONV_ERR_ALIGNMENT, "strides must be non-negative, whole 16-byte pieces and within the index limits");
  for (const int64_t* s : ks)
    if (!strides_ok(s, d->batch, d->k_len, d->kv_heads, es))
      return fail(FUSEDCONV_ERR_ALIGNMENT, "strides must be non-negative, whole 16-byte pieces and within the index limits");
  if (!apart(d->o_strides, d->batch, d->q_len, d->heads, d->head_dim) ||
      !apart(d->dq_strides, d->batch, d->q_len, d->heads, d->head_dim) ||
      !apart(d->dk_strides, d->batch, d->k_len, d->kv_heads, d->head_dim) ||
      !apart(d->dv_strides, d->batch, d->k_len, d->kv_heads, d->head_dim))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "an output's strides make its elements overlap");
  fusedconv_attention* h = new (std::nothrow) fusedconv_attention();
  if (!h) return fail(FUSEDCONV_ERR_ALLOC, "out of host memory");
  const auto limit = [](int64_t w) { return (int32_t)(w > kMaxLen ? -1 : w); };
  fc::AttnParams& p = h->p;
  p.batch = (int32_t)d->batch;
  p.sq = (int32_t)d->q_len;
  p.sk = (int32_t)d->k_len;
  p.heads = (int32_t)d->heads;
  p.kv_heads = (int32_t)d->kv_heads;
  p.group = (int32_t)(d->heads / d->kv_heads);
  p.d = (int32_t)d->head_dim;
  p.scale = d->scale;
  p.left = limit(d->window_left);
  p.right = limit(d->window_right);
  const auto qof = [&](const int64_t* s) { return strides_of(s, d->batch, d->q_len, d->heads); };
  const auto kof = [&](const int64_t* s) { return strides_of(s, d->batch, d->k_len, d->kv_heads); };
  p.q = qof(d->q_strides); p.o = qof(d->o_strides); p.dout = qof(d->do_strides); p.dq = qof(d->dq_strides);
  p.k = kof(d->k_strides); p.v = kof(d->v_strides); p.dk = kof(d->dk_strides); p.dv = kof(d->dv_strides);
  h->plan.dtype = d->dtype;
  fc::plan_attention(p, h->plan);
  *out = h;
  fc::clear_last_error();
  return FUSEDCONV_OK;
}

int fusedconv_attention_workspace_size(const fusedconv_attention* h, size_t* forward_bytes,
                                       size_t* backward_bytes) {
  if (!h || !forward_bytes || !backward_bytes) return fail(FUSEDCONV_ERR_NULL_ARG, "NULL argument");
  *forward_bytes = h->plan.forward_bytes;
  *backward_bytes = h->plan.backward_bytes;
  return FUSEDCONV_OK;
}

int fusedconv_attention_forward(const fusedconv_attention* h, const void* q, const void* k,
                                const void* v, const int32_t* q_lengths,
                                const int32_t* k_lengths, void* o, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  if (h->p.batch == 0 || h->p.sq == 0) return FUSEDCONV_OK;
  if (!q || !o || (h->p.sk > 0 && (!k || !v)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "q, k, v and o are required");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned_to(lse, 4) ||
      !aligned_to(q_lengths, 4) || !aligned_to(k_lengths, 4) || !aligned16(workspace))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (h->plan.forward_bytes > 0 && (!workspace || workspace_bytes < h->plan.forward_bytes))
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_attention_workspace_size() reports");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  fc::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_lengths = q_lengths; a.k_lengths = k_lengths;
  a.o = o; a.lse = lse; a.ws = workspace; a.stream = stream;
  return launched([&] { return fc::launch_attention_forward(h->p, h->plan, a); });
}

int fusedconv_attention_backward(const fusedconv_attention* h, const void* dout, const void* q,
                                 const void* k, const void* v, const void* o, const float* lse,
                                 const int32_t* q_lengths, const int32_t* k_lengths, void* dq,
                                 void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  const fc::AttnParams& p = h->p;
  if (p.batch == 0 || (p.sq == 0 && p.sk == 0)) return FUSEDCONV_OK;
  if ((p.sq > 0 && (!dout || !q || !o || !lse || !dq)) || (p.sk > 0 && (!k || !v || !dk || !dv)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "a required pointer is NULL");
  if (!aligned16(dout) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      !aligned_to(lse, 4) || !aligned_to(q_lengths, 4) || !aligned_to(k_lengths, 4) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(workspace))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (h->plan.backward_bytes > 0 && (!workspace || workspace_bytes < h->plan.backward_bytes))
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_attention_workspace_size() reports");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  fc::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.o_in = o; a.dout = dout; a.lse_in = lse;
  a.q_lengths = q_lengths; a.k_lengths = k_lengths;
  a.dq = dq; a.dk = dk; a.dv = dv; a.ws = workspace; a.stream = stream;
  return launched([&] { return fc::launch_attention_backward(p, h->plan, a); });
}

void fusedconv_attention_destroy(fusedconv_attention* h) { delete h; }

}  // extern "C"
