// Entry points of include/fusedconv_block.h: checks, handles, dispatch.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "block.h"
#include "checks.h"

using namespace fc;

struct fusedconv_qk_norm_rotary {
  fusedconv_qk_norm_rotary_desc d;
  size_t workspace;
};

struct fusedconv_gated_ffn {
  GatedProblem p;
  GatedPlan plan;
};

namespace {
constexpr char kStrides[] =
    "strides must be non-negative, whole 16-byte pieces and within the index limits";
}  // namespace

extern "C" {

// ------------------------------------------ norms of queries and keys, and rotary

int fusedconv_qk_norm_rotary_create(const fusedconv_qk_norm_rotary_desc* d,
                                    fusedconv_qk_norm_rotary** out) {
  if (out) *out = nullptr;
  if (!d || !out) return fail(FUSEDCONV_ERR_NULL_ARG, "desc and out must not be NULL");
  if (!known(d->dtype)) return fail(FUSEDCONV_ERR_DTYPE, "dtype is not float32, float16 or bfloat16");
  if (d->position_dtype < FUSEDCONV_POS_I32 || d->position_dtype > FUSEDCONV_POS_F32)
    return fail(FUSEDCONV_ERR_DTYPE, "positions are not int32, int64 or float32");
  if (d->batch < 0 || d->len < 0 || d->heads < 1 || d->kv_heads < 0)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "batch, len, kv_heads must be >= 0, heads >= 1");
  const int64_t es = elem_size(d->dtype);
  if (d->head_dim < 1 || d->head_dim > 256 || d->head_dim % (16 / es) != 0)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE, "a head must be whole 16-byte pieces, at most 256 values");
  if (d->pairs < 1 || d->pairs > d->head_dim / 2)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "pairs must be in [1, head_dim / 2]");
  if (d->num_axes < 1 || d->num_axes > 8)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "num_axes must be in [1, 8]");
  if (!(d->eps > 0.0f) || !isfinite(d->eps))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "eps must be positive and finite");
  if (d->heads > (1 << 16) || d->kv_heads > (1 << 16) || d->len > INT32_MAX / 16 ||
      product(d->batch, d->len, 1, INT32_MAX) < 0 ||
      product(d->batch, d->len, (d->heads + d->kv_heads) * d->head_dim, kMaxElements) < 0)
    return fail(FUSEDCONV_ERR_TOO_LARGE, "Q or K exceeds the index limits");
  if (d->position_batch_stride != 0 && d->position_batch_stride != d->len * d->num_axes &&
      d->batch > 1)
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "position_batch_stride is len * num_axes, or 0");
  for (const int64_t* s : {d->q_strides, d->q_out_strides, d->dq_strides})
    if (!strides_ok(s, d->batch, d->len, d->heads, es)) return fail(FUSEDCONV_ERR_ALIGNMENT, kStrides);
  if (d->kv_heads)
    for (const int64_t* s : {d->k_strides, d->k_out_strides, d->dk_strides})
      if (!strides_ok(s, d->batch, d->len, d->kv_heads, es))
        return fail(FUSEDCONV_ERR_ALIGNMENT, kStrides);
  fusedconv_qk_norm_rotary* h = new (std::nothrow) fusedconv_qk_norm_rotary();
  if (!h) return fail(FUSEDCONV_ERR_ALLOC, "out of host memory");
  h->d = *d;
  const int64_t tokens = d->batch * d->len;
  h->workspace = (size_t)(tokens < kQkBlocks ? tokens : kQkBlocks) * 2 * d->head_dim * sizeof(float);
  *out = h;
  clear_last_error();
  return FUSEDCONV_OK;
}

int fusedconv_qk_norm_rotary_workspace_size(const fusedconv_qk_norm_rotary* h, size_t* bytes) {
  if (!h || !bytes) return fail(FUSEDCONV_ERR_NULL_ARG, "NULL argument");
  *bytes = h->workspace;
  return FUSEDCONV_OK;
}

namespace {

// What both directions check of the pointers they share; y: the outputs, with
// their strides.
int check_qk(const fusedconv_qk_norm_rotary_desc& d, const void* q, const void* k,
             const void* q_weight, const void* k_weight, const void* positions,
             const float* inv_freq, const int32_t* axes, const void* yq, const void* yk,
             const int64_t* yq_strides, const int64_t* yk_strides) {
  if (!q_weight != !d.has_q_weight || !k_weight != !d.has_k_weight)
    return fail(FUSEDCONV_ERR_NULL_ARG, "weights are given iff they were declared");
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned_to(inv_freq, 4) || !aligned_to(axes, 4))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (d.batch == 0 || d.len == 0) return FUSEDCONV_OK;
  if (!q || !yq || !positions || !inv_freq || !axes || (d.kv_heads && (!k || !yk)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(yq) || !aligned16(yk) ||
      !aligned_to(positions, d.position_dtype == FUSEDCONV_POS_I64 ? 8 : 4))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (!apart(yq_strides, d.batch, d.len, d.heads, d.head_dim) ||
      (d.kv_heads && !apart(yk_strides, d.batch, d.len, d.kv_heads, d.head_dim)))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "an output's strides make its elements overlap");
  return FUSEDCONV_OK;
}

}  // namespace

int fusedconv_qk_norm_rotary_forward(const fusedconv_qk_norm_rotary* h, const void* q,
                                     const void* k, const void* q_weight, const void* k_weight,
                                     const void* positions, const float* inv_freq,
                                     const int32_t* axes, void* q_out, void* k_out, void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  const fusedconv_qk_norm_rotary_desc& d = h->d;
  int rc = check_qk(d, q, k, q_weight, k_weight, positions, inv_freq, axes, q_out, k_out,
                    d.q_out_strides, d.k_out_strides);
  if (rc != FUSEDCONV_OK || d.batch == 0 || d.len == 0) return rc;
  rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  QkArgs a{};
  a.q = q; a.k = k; a.q_weight = q_weight; a.k_weight = k_weight;
  a.positions = positions; a.inv_freq = inv_freq; a.axes = axes;
  a.qo = q_out; a.ko = k_out; a.stream = stream;
  return launched([&] { return launch_qk_norm_forward(d, a); });
}

int fusedconv_qk_norm_rotary_backward(const fusedconv_qk_norm_rotary* h, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const void* q_weight, const void* k_weight,
                                      const void* positions, const float* inv_freq,
                                      const int32_t* axes, void* dq, void* dk, float* dq_weight,
                                      float* dk_weight, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  const fusedconv_qk_norm_rotary_desc& d = h->d;
  int rc = check_qk(d, q, k, q_weight, k_weight, positions, inv_freq, axes, dq, dk, d.dq_strides,
                    d.dk_strides);
  if (rc != FUSEDCONV_OK) return rc;
  if (d.batch > 0 && d.len > 0 && (!dq_out || (d.kv_heads && !dk_out)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "a required pointer is NULL");
  if (dk_weight && !d.kv_heads)
    return fail(FUSEDCONV_ERR_NULL_ARG, "dk_weight is given without K");
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned_to(dq_weight, 4) ||
      !aligned_to(dk_weight, 4) || !aligned16(workspace))
    return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (h->workspace > 0 && (dq_weight || dk_weight) && (!workspace || workspace_bytes < h->workspace))
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_qk_norm_rotary_workspace_size() reports");
  rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  QkArgs a{};
  a.q = q; a.k = k; a.q_weight = q_weight; a.k_weight = k_weight;
  a.positions = positions; a.inv_freq = inv_freq; a.axes = axes;
  a.dq = dq_out; a.dk = dk_out; a.qo = dq; a.ko = dk;
  a.dqw = dq_weight; a.dkw = dk_weight; a.part = (float*)workspace; a.stream = stream;
  return launched([&] { return launch_qk_norm_backward(d, a); });
}

void fusedconv_qk_norm_rotary_destroy(fusedconv_qk_norm_rotary* h) { delete h; }

// ---------------------------------------------------- gated feed-forward block

int fusedconv_gated_ffn_create(const fusedconv_gated_ffn_desc* d, fusedconv_gated_ffn** out) {
  if (out) *out = nullptr;
  if (!d || !out || !d->activation)
    return fail(FUSEDCONV_ERR_NULL_ARG, "desc, its activation and out must not be NULL");
  if (!known(d->dtype)) return fail(FUSEDCONV_ERR_DTYPE, "dtype is not float32, float16 or bfloat16");
  if (d->rows < 0 || d->in < 8 || d->hidden < 8 || d->out < 8 || d->in % 8 || d->hidden % 8 || d->out % 8)
    return fail(FUSEDCONV_ERR_OUTPUT_SHAPE,
                "rows must be >= 0; in, hidden and out positive multiples of 8");
  static const char* const names[] = {"Sigmoid", "Relu", "QuickGelu", "Gelu", "FastGelu"};  // GateAct
  const bool silu = strcmp(d->activation, "Silu") == 0;  // QuickGelu with alpha 1
  const char* name = silu ? "QuickGelu" : d->activation;
  int act = 0;
  while (act < 5 && strcmp(name, names[act]) != 0) ++act;
  if (act == 5)
    return fail(FUSEDCONV_ERR_ACTIVATION, "activation is not Silu, QuickGelu, Gelu, FastGelu, Sigmoid or Relu");
  if (!isfinite(d->alpha)) return fail(FUSEDCONV_ERR_ATTR_VALUE, "alpha must be finite");
  const int64_t es = elem_size(d->dtype);
  // a tile's 256 rows have to fit 31-bit byte offsets
  const int64_t most = ((int64_t(1) << 31) / 256 - 1) / es;
  if (d->in > most || d->hidden > most || d->out > most || d->rows > INT32_MAX / 2 ||
      product(d->rows, d->hidden, 1, kMaxElements / 4) < 0 || product(d->rows, d->in, 1, kMaxElements / 4) < 0 ||
      product(d->rows, d->out, 1, kMaxElements / 4) < 0 || product(d->hidden, d->in, 1, kMaxElements / 8) < 0 ||
      product(d->out, d->hidden, 1, kMaxElements / 8) < 0)  // tiles and blocks stay below 2^31
    return fail(FUSEDCONV_ERR_TOO_LARGE, "a tensor exceeds the index limits");
  if (d->rows > 1 && (d->x_stride < 0 || d->dy_stride < 0 || d->x_stride % (16 / es) || d->dy_stride % (16 / es) ||
                      d->x_stride > most || d->dy_stride > most))
    return fail(FUSEDCONV_ERR_ALIGNMENT,
                "strides must be non-negative, whole 16-byte pieces and within the index limits");
  fusedconv_gated_ffn* h = new (std::nothrow) fusedconv_gated_ffn();
  if (!h) return fail(FUSEDCONV_ERR_ALLOC, "out of host memory");
  h->p = {d->dtype, (int32_t)d->rows, (int32_t)d->in, (int32_t)d->hidden, (int32_t)d->out, act,
          silu ? 1.0f : d->alpha,
          d->rows > 1 ? d->x_stride : d->in, d->rows > 1 ? d->dy_stride : d->out};
  plan_gated(h->p, h->plan);
  *out = h;
  clear_last_error();
  return FUSEDCONV_OK;
}

int fusedconv_gated_ffn_workspace_size(const fusedconv_gated_ffn* h, size_t* forward_bytes,
                                       size_t* backward_bytes) {
  if (!h || !forward_bytes || !backward_bytes) return fail(FUSEDCONV_ERR_NULL_ARG, "NULL argument");
  *forward_bytes = h->plan.forward_bytes;
  *backward_bytes = h->plan.backward_bytes;
  return FUSEDCONV_OK;
}

int fusedconv_gated_ffn_forward(const fusedconv_gated_ffn* h, const void* x, const void* gate,
                                const void* up, const void* down, void* y, void* g, void* u,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  if (!g != !u) return fail(FUSEDCONV_ERR_NULL_ARG, "give both g and u or neither");
  if (h->p.m == 0) return FUSEDCONV_OK;
  if (!x || !gate || !up || !down || !y)
    return fail(FUSEDCONV_ERR_NULL_ARG, "x, gate, up, down and y are required");
  for (const void* p : {x, gate, up, down, (const void*)y, (const void*)g, (const void*)u, (const void*)workspace})
    if (!aligned16(p)) return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (!workspace || workspace_bytes < h->plan.forward_bytes)
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_gated_ffn_workspace_size() reports");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  GatedArgs a{};
  a.x = x; a.gate = gate; a.up = up; a.down = down;
  a.y = y; a.g = g; a.u = u; a.ws = workspace; a.stream = stream;
  return launched([&] {
    return h->p.dtype == FUSEDCONV_F32   ? gated_forward_f32(h->p, h->plan, a)
           : h->p.dtype == FUSEDCONV_F16 ? gated_forward_f16(h->p, h->plan, a)
                                         : gated_forward_bf16(h->p, h->plan, a);
  });
}

int fusedconv_gated_ffn_backward(const fusedconv_gated_ffn* h, const void* dy, const void* x,
                                 const void* gate, const void* up, const void* down,
                                 const void* g, const void* u, void* dx, void* dgate, void* dup,
                                 void* ddown, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!h) return fail(FUSEDCONV_ERR_NULL_ARG, "h is required");
  if (!dgate != !dup || !dgate != !ddown)
    return fail(FUSEDCONV_ERR_NULL_ARG, "give all three of dgate, dup and ddown or none");
  if (!gate || !up || !down || (h->p.m > 0 && (!dy || !x || !g || !u || !dx)))
    return fail(FUSEDCONV_ERR_NULL_ARG, "a required pointer is NULL");
  for (const void* p : {dy, x, gate, up, down, g, u, (const void*)dx, (const void*)dgate, (const void*)dup,
                        (const void*)ddown, (const void*)workspace})
    if (!aligned16(p)) return fail(FUSEDCONV_ERR_ALIGNMENT, kAlignment);
  if (!workspace || workspace_bytes < h->plan.backward_bytes)
    return fail(FUSEDCONV_ERR_WORKSPACE,
                "workspace smaller than fusedconv_gated_ffn_workspace_size() reports");
  const int rc = ready(stream);
  if (rc != FUSEDCONV_OK) return rc;
  GatedArgs a{};
  a.dy = dy; a.x = x; a.gate = gate; a.up = up; a.down = down;
  a.g = const_cast<void*>(g); a.u = const_cast<void*>(u);
  a.dx = dx; a.dgate = dgate; a.dup = dup; a.ddown = ddown; a.ws = workspace; a.stream = stream;
  return launched([&] {
    return h->p.dtype == FUSEDCONV_F32   ? gated_backward_f32(h->p, h->plan, a)
           : h->p.dtype == FUSEDCONV_F16 ? gated_backward_f16(h->p, h->plan, a)
                                         : gated_backward_bf16(h->p, h->plan, a);
  });
}

void fusedconv_gated_ffn_destroy(fusedconv_gated_ffn* h) { delete h; }

}  // extern "C"
