// Host-side sweep of the handles of include/fusedconv_block.h, run under
// AddressSanitizer and UndefinedBehaviorSanitizer (built by
// tests/test_block_sanitizers_cpu.py): seeded descriptions, most of them valid, some
// with one field set to a value from the ends of its range, through create, workspace
// size, the checks in front of a launch and destroy.  No kernel is launched: what the
// entry points need of the rest of the library stands below, and a launcher throws
// now and then, which must not leave a C function.  Prints one line and exits 0; a
// sanitizer finding aborts.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <new>
#include <string>

#include "block.h"
#include "internal.h"

namespace {
uint64_t g_state = 0x9e3779b97f4a7c15ull;
uint64_t rnd() {  // xorshift64*
  g_state ^= g_state >> 12;
  g_state ^= g_state << 25;
  g_state ^= g_state >> 27;
  return g_state * 0x2545f4914f6cdd1dull;
}
int g_created, g_rejected, g_launched;
int launch() {
  ++g_launched;
  if (rnd() % 16 == 0) throw std::bad_alloc();
  return rnd() % 2 ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}
}  // namespace

namespace fc {
int set_last_error(int code, const std::string&) {
  if (rnd() % 64 == 0) throw std::bad_alloc();
  return code;
}
int check_device(void*) { return FUSEDCONV_OK; }
void clear_last_error() {}
int launch_qk_norm_forward(const fusedconv_qk_norm_rotary_desc&, const QkArgs&) { return launch(); }
int launch_qk_norm_backward(const fusedconv_qk_norm_rotary_desc&, const QkArgs&) { return launch(); }
int gated_forward_f32(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
int gated_forward_f16(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
int gated_forward_bf16(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
int gated_backward_f32(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
int gated_backward_f16(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
int gated_backward_bf16(const GatedProblem&, const GatedPlan&, const GatedArgs&) { return launch(); }
}  // namespace fc

namespace {

int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)((rnd() >> 20) % (uint64_t)(hi - lo + 1)); }

// A value from the ends of the range: near a power of two, near the limits, or negative.
int64_t wild() {
  const int64_t near = pick(-9, 9);
  switch (pick(0, 3)) {
    case 0: return (int64_t)((uint64_t(1) << pick(0, 62)) + (uint64_t)near);
    case 1: return near < 0 ? INT64_MAX + near : INT64_MAX - near;
    case 2: return near < 0 ? INT64_MIN - near : INT64_MIN + near;
    default: return near;
  }
}

void set(int64_t (&s)[3], int64_t len, int64_t h, int64_t d) {
  const int64_t gap = pick(0, 2) * 8;
  s[0] = len * (h * d + gap);
  s[1] = h * d + gap;
  s[2] = d;
}

void qk(bool spoil) {
  fusedconv_qk_norm_rotary_desc d{};
  d.dtype = (int32_t)pick(0, 2);
  d.position_dtype = (int32_t)pick(0, 2);
  d.batch = pick(0, 5);
  d.len = pick(0, 3000);
  d.kv_heads = pick(0, 8);
  d.heads = (d.kv_heads ? d.kv_heads : 1) * pick(1, 8);
  d.head_dim = 8 * pick(1, 32);
  d.pairs = pick(1, d.head_dim / 2);
  d.num_axes = (int32_t)pick(1, 8);
  d.position_batch_stride = pick(0, 1) * d.len * d.num_axes;
  d.interleaved = (int32_t)pick(0, 1);
  d.has_q_weight = (int32_t)pick(0, 1);
  d.has_k_weight = (int32_t)pick(0, 1);
  d.eps = 1e-6f;
  set(d.q_strides, d.len, d.heads, d.head_dim);
  set(d.q_out_strides, d.len, d.heads, d.head_dim);
  set(d.dq_strides, d.len, d.heads, d.head_dim);
  set(d.k_strides, d.len, d.kv_heads, d.head_dim);
  set(d.k_out_strides, d.len, d.kv_heads, d.head_dim);
  set(d.dk_strides, d.len, d.kv_heads, d.head_dim);
  if (spoil) {
    int64_t* fields[] = {&d.batch, &d.len, &d.heads, &d.kv_heads, &d.head_dim, &d.pairs, &d.position_batch_stride,
                         &d.q_strides[pick(0, 2)], &d.k_strides[pick(0, 2)], &d.q_out_strides[pick(0, 2)],
                         &d.k_out_strides[pick(0, 2)], &d.dq_strides[pick(0, 2)], &d.dk_strides[pick(0, 2)]};
    const int n = (int)pick(0, 14);
    if (n < 13) *fields[n] = wild();
    else if (n == 13) d.dtype = (int32_t)wild();
    else d.num_axes = (int32_t)wild();
  }
  fusedconv_qk_norm_rotary* h = nullptr;
  if (fusedconv_qk_norm_rotary_create(&d, &h) != FUSEDCONV_OK) {
    ++g_rejected;
    return;
  }
  ++g_created;
  size_t bytes = 0;
  if (fusedconv_qk_norm_rotary_workspace_size(h, &bytes) != FUSEDCONV_OK) abort();
  float* p = (float*)4096;  // never read
  const void *qw = d.has_q_weight ? p : nullptr, *kw = d.has_k_weight ? p : nullptr;
  (void)fusedconv_qk_norm_rotary_forward(h, p, p, qw, kw, p, p, (int32_t*)p, p, p, nullptr);
  (void)fusedconv_qk_norm_rotary_backward(h, p, p, p, p, qw, kw, p, p, (int32_t*)p, p, p, p, d.kv_heads ? p : nullptr, p,
                                          bytes, nullptr);
  fusedconv_qk_norm_rotary_destroy(h);
}

void ffn(bool spoil) {
  const char* names[] = {"Silu", "QuickGelu", "Gelu", "FastGelu", "Sigmoid", "Relu", "None", ""};
  fusedconv_gated_ffn_desc d{};
  d.dtype = (int32_t)pick(0, 2);
  const int top = (int)pick(0, 16);
  d.rows = pick(0, (int64_t)1 << top);
  d.in = 8 * pick(1, 1024);
  d.hidden = 8 * pick(1, 2048);
  d.out = 8 * pick(1, 1024);
  d.x_stride = d.in + 8 * pick(0, 3);
  d.dy_stride = d.out + 8 * pick(0, 3);
  d.activation = names[pick(0, 5)];
  d.alpha = 1.f;
  if (spoil) {
    int64_t* fields[] = {&d.rows, &d.in, &d.hidden, &d.out, &d.x_stride, &d.dy_stride};
    const int n = (int)pick(0, 8);
    if (n < 6) *fields[n] = pick(0, 2) ? wild() : wild() & ~7;
    else if (n == 6) d.dtype = (int32_t)wild();
    else if (n == 7) d.activation = names[pick(6, 7)];
    else d.activation = nullptr;
  }
  fusedconv_gated_ffn* h = nullptr;
  if (fusedconv_gated_ffn_create(&d, &h) != FUSEDCONV_OK) {
    ++g_rejected;
    return;
  }
  ++g_created;
  size_t f = 0, b = 0;
  if (fusedconv_gated_ffn_workspace_size(h, &f, &b) != FUSEDCONV_OK) abort();
  if (f < (size_t)d.rows * d.hidden * 2 || b < 3 * (size_t)d.rows * d.hidden * 2) abort();
  void* p = (void*)4096;  // never read
  (void)fusedconv_gated_ffn_forward(h, p, p, p, p, p, p, p, p, f, nullptr);
  (void)fusedconv_gated_ffn_backward(h, p, p, p, p, p, p, p, p, p, p, p, p, b, nullptr);
  fusedconv_gated_ffn_destroy(h);
}

}  // namespace

int main(int argc, char** argv) {
  const int n = argc > 1 ? atoi(argv[1]) : 1000;
  for (int i = 0; i < n; ++i) {
    qk(i % 3 == 0);
    ffn(i % 3 == 0);
  }
  printf("created %d rejected %d launched %d\n", g_created, g_rejected, g_launched);
  return 0;
}
