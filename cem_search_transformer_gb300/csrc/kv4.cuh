// Declarations of the 4-bit paged key/value cache: filling and reading it, attention over it, and
// eviction from it.
//
// Cache of one layer: e2m1 codes k, v [num_pages][kv_heads][page_size][head_dim / 2], the even element
// in the low half of a byte, and e4m3 scales [num_pages][kv_heads][page_size][head_dim / 16], one
// for 16 elements of a token. An element stands for code * scale * unit with the power of two
// unit[kv_head]. Every (token, head, 16 elements) stands for itself: no append changes earlier
// tokens, and a token can be moved as it is.
#pragma once

#include "kv8.cuh"

namespace jepa {

constexpr int KV4_BLOCK = 16;                 // elements of a scale
constexpr float KV4_SCALE_MIN = 0x1p-9f;      // the least scale written: e4m3's least value above zero

struct Kv4View : PageView {
  uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_unit, *v_unit;               // [heads] or null: 1
};

// A head's unit as the cache's contract has it: a power of two within [2^-40, 2^40], the one at or below
// what is given.
__device__ __forceinline__ float kv4_unit(const float* units, int head) {
  if (!units) return 1.f;
  const float u = load_late(units + head);
  const float sane = u >= KV8_SCALE_MIN ? fminf(u, KV8_SCALE_MAX) : KV8_SCALE_MIN;
  return __uint_as_float(__float_as_uint(sane) & 0x7f800000u);
}
__device__ __forceinline__ float kv4_inverse(float unit) {   // of a power of two
  return __uint_as_float(0x7f000000u - __float_as_uint(unit));
}

// Byte `i` of w, two e2m1 codes, as f16 (exact).
template <int I>
__device__ __forceinline__ uint32_t f16x2_of_e2m1x2(uint32_t w) {
  uint32_t h;
  if (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
  else if (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
  else if (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
// Two e4m3 codes in the low 16 bits of w as f16 (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t f16x2_of_e4m3_pair(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
  return h;
}

// ---- launchers (each returns the launch's error) ----

cudaError_t rope_append_kv4(const Kv4View& c, const AppendArgs& a, int* err_flag, cudaStream_t s);

cudaError_t kv4_read(const Kv4View& c, const int* cu, const int* first, int tokens, bf16* k_out,
                     bf16* v_out, int* err_flag, cudaStream_t s);

// What the tokens of a cache received: mass_out = decay * mass + the weights of this call, for the
// cached tokens. [batch][heads][max_pages * page] each.
struct MassArgs {
  const float* mass;   // or null: zeros
  float* out;
  float decay;
};

// Workspace of attention_kv4 (partial results of sequences split over CTAs).
size_t attention_kv4_workspace(int dim, int num_sms);
cudaError_t attention_kv4(const Kv4View& c, const bf16* q, int q_tokens, int q_heads,
                          const int* kv_len, float scale, int causal, bf16* out, float* lse,
                          const MassArgs* mass, void* workspace, int* err_flag, int num_sms,
                          cudaStream_t s);

// Workspace of kv4_evict: the kept tokens' places.
size_t kv4_evict_workspace(const PageView& c, int keep);
cudaError_t kv4_evict(const Kv4View& c, const int* kv_len, const float* mass, int keep, int recent,
                      const Kv4View& to, int* len_out, float* mass_out, void* workspace,
                      int* err_flag, int num_sms, cudaStream_t s);

}  // namespace jepa
