// Host-side sweep of layer norm, rotary and attention handles, run under
// AddressSanitizer and UndefinedBehaviorSanitizer (built by
// tests/test_transformer_sanitizers_cpu.py): seeded descriptions, most of them
// valid, some with one field set to a value from the ends of its range, through
// create, workspace size and destroy.  Attention's forward pass is also run up to the
// point where it asks for a kernel's LDS, which has to be one size a kernel: the limit
// is a kernel's, whatever its calls need.  No kernel is launched; what the entry points
// need of the rest of the library stands below.  Prints one line and exits 0; a
// sanitizer finding aborts.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <new>
#include <string>

#include "fusedconv_transformer.h"
#include "internal.h"

namespace {
uint64_t g_state = 0x9e3779b97f4a7c15ull;
uint64_t rnd() {  // xorshift64*
  g_state ^= g_state >> 12;
  g_state ^= g_state << 25;
  g_state ^= g_state >> 27;
  return g_state * 0x2545f4914f6cdd1dull;
}
}  // namespace

namespace fc {
int set_last_error(int code, const std::string&) { return code; }
int check_device(void*) { return FUSEDCONV_OK; }
void clear_last_error() {}
std::map<const void*, int> g_lds;
int set_max_dynamic_lds(const void* kernel, int bytes) {
  const int before = g_lds.emplace(kernel, bytes).first->second;
  if (bytes != before) {
    printf("a kernel's LDS limit is set to %d and to %d bytes\n", before, bytes);
    fflush(stdout);
    abort();
  }
  // nothing is launched after either; what is thrown must not leave a C function
  if (rnd() % 16 == 0) throw std::bad_alloc();
  return FUSEDCONV_ERR_LAUNCH;
}
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

struct Head {
  int64_t s[3];
};
// Strides of a [batch][len][heads][d] tensor in one of three orders, some with gaps.
Head strides(int64_t b, int64_t len, int64_t h, int64_t d) {
  const int64_t gap = pick(0, 2) * 8;
  switch (pick(0, 2)) {
    case 0: return {{len * (h * d + gap), h * d + gap, d}};
    case 1: return {{len * h * (d + gap), d + gap, len * (d + gap)}};
    default: return {{h * d, b * h * d, d}};
  }
}
void set(int64_t (&to)[3], const Head& from) {
  for (int i = 0; i < 3; ++i) to[i] = from.s[i];
}

int g_created, g_rejected;

void norm(bool mess) {
  fusedconv_layer_norm_desc d{};
  d.dtype = (int32_t)pick(0, 2);
  d.n = pick(0, 3000);
  d.c = pick(1, 20000);
  d.inner = pick(0, 1) ? 1 : pick(1, 4000);
  d.x_stride = d.dy_stride = d.c * d.inner + pick(0, 1) * 8;
  d.has_weight = (int32_t)pick(0, 1);
  d.has_bias = (int32_t)pick(0, 1);
  d.eps = 1e-5f;
  if (mess) {
    int64_t* fields[] = {&d.n, &d.c, &d.inner, &d.x_stride, &d.dy_stride};
    *fields[pick(0, 4)] = wild();
    if (pick(0, 9) == 0) d.dtype = (int32_t)wild();
  }
  fusedconv_layer_norm* h = nullptr;
  if (fusedconv_layer_norm_create(&d, &h) != FUSEDCONV_OK) {
    ++g_rejected;
    return;
  }
  ++g_created;
  size_t bytes = 0;
  if (fusedconv_layer_norm_workspace_size(h, &bytes) != FUSEDCONV_OK) abort();
  fusedconv_layer_norm_destroy(h);
}

void rotary(bool mess) {
  fusedconv_rotary_desc d{};
  d.dtype = (int32_t)pick(0, 2);
  d.position_dtype = (int32_t)pick(0, 2);
  d.batch = pick(0, 5);
  d.len = pick(0, 500);
  d.heads = pick(1, 40);
  d.kv_heads = pick(0, 8);
  d.head_dim = 8 * pick(1, 32);
  d.pairs = pick(1, d.head_dim / 2);
  d.num_axes = (int32_t)pick(1, 8);
  d.position_batch_stride = pick(0, 1) ? d.len * d.num_axes : 0;
  set(d.q_strides, strides(d.batch, d.len, d.heads, d.head_dim));
  set(d.q_out_strides, strides(d.batch, d.len, d.heads, d.head_dim));
  set(d.k_strides, strides(d.batch, d.len, d.kv_heads, d.head_dim));
  set(d.k_out_strides, strides(d.batch, d.len, d.kv_heads, d.head_dim));
  if (mess) {
    int64_t* fields[] = {&d.batch, &d.len, &d.heads, &d.kv_heads, &d.head_dim, &d.pairs,
                         &d.position_batch_stride,
                         &d.q_strides[pick(0, 2)], &d.k_strides[pick(0, 2)],
                         &d.q_out_strides[pick(0, 2)], &d.k_out_strides[pick(0, 2)]};
    *fields[pick(0, 10)] = wild();
    if (pick(0, 9) == 0) d.num_axes = (int32_t)wild();
  }
  fusedconv_rotary* h = nullptr;
  if (fusedconv_rotary_create(&d, &h) != FUSEDCONV_OK) {
    ++g_rejected;
    return;
  }
  ++g_created;
  if (d.pairs > d.head_dim / 2) abort();
  fusedconv_rotary_destroy(h);
}

void attention(bool mess) {
  fusedconv_attention_desc d{};
  d.dtype = (int32_t)pick(0, 2);
  d.batch = pick(0, 5);
  d.q_len = pick(0, 1) ? pick(0, 40) : pick(0, 9000);
  d.k_len = pick(0, 1) ? pick(0, 40) : pick(0, 60000);
  d.kv_heads = pick(1, 6);
  d.heads = d.kv_heads * pick(1, 8);
  d.head_dim = 8 * pick(1, 16);
  d.scale = 0.1f;
  d.window_left = pick(-1, 3000);
  d.window_right = pick(-1, 300);
  int64_t(*qs[])[3] = {&d.q_strides, &d.o_strides, &d.do_strides, &d.dq_strides};
  int64_t(*ks[])[3] = {&d.k_strides, &d.v_strides, &d.dk_strides, &d.dv_strides};
  for (auto* s : qs) set(*s, strides(d.batch, d.q_len, d.heads, d.head_dim));
  for (auto* s : ks) set(*s, strides(d.batch, d.k_len, d.kv_heads, d.head_dim));
  if (mess) {
    int64_t* fields[] = {&d.batch, &d.q_len, &d.k_len, &d.heads, &d.kv_heads, &d.head_dim,
                         &d.window_left, &d.window_right,
                         &(*qs[pick(0, 3)])[pick(0, 2)], &(*ks[pick(0, 3)])[pick(0, 2)]};
    *fields[pick(0, 9)] = wild();
  }
  fusedconv_attention* h = nullptr;
  if (fusedconv_attention_create(&d, &h) != FUSEDCONV_OK) {
    ++g_rejected;
    return;
  }
  ++g_created;
  size_t forward = 0, backward = 0;
  if (fusedconv_attention_workspace_size(h, &forward, &backward) != FUSEDCONV_OK) abort();
  void* const p = (void*)4096;  // never read
  const int rc =
      fusedconv_attention_forward(h, p, p, p, nullptr, nullptr, p, nullptr, p, forward, nullptr);
  if (rc != FUSEDCONV_OK && rc != FUSEDCONV_ERR_LAUNCH && rc != FUSEDCONV_ERR_ALLOC) abort();
  fusedconv_attention_destroy(h);
}

}  // namespace

int main(int argc, char** argv) {
  const int n = argc > 1 ? atoi(argv[1]) : 1000;
  for (int i = 0; i < n; ++i) {
    norm(i & 1);
    rotary(i & 1);
    attention(i & 1);
  }
  printf("handles: %d created, %d rejected, %d kernels\n", g_created, g_rejected, (int)fc::g_lds.size());
  return 0;
}
