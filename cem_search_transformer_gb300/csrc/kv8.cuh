// Declarations of the 8-bit paged key/value cache and of the attention kernels beside it.
//
// Cache of one layer: e4m3 codes k, v [num_pages][kv_heads][page_size][head_dim] and one fp32
// scale per (page, head) each; a page table [batch][max_pages] names the pages of a sequence.
// The value a code stands for is code * scale. Scales are powers of two, 2^-40 .. 2^40, so
// that moving a page to a larger scale only rounds codes that become subnormal.
#pragma once

#include "common.cuh"
#include "kv8_index.h"

namespace jepa {

// Bits of the context's error word.
constexpr int DEV_ERR_TIMEOUT = 1;   // a bounded wait gave up
constexpr int DEV_ERR_INDEX = 2;     // a page, position or offset outside its buffer (skipped)

constexpr float KV8_SCALE_MIN = 0x1p-40f;
constexpr float KV8_SCALE_MAX = 0x1p+40f;

// The pages of a cache of either width: table [batch][max_pages] into num_pages blocks of `page`
// tokens a head.
struct PageView {
  const int* table;
  int num_pages, page, page_log2, heads, dim, batch, max_pages;
};

struct Kv8View : PageView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
};

// Loads that stay behind a griddepcontrol.wait, being volatile like it: __ldg is for what no one writes while the kernel
// lives, and may be moved ahead of the wait. Stores to elsewhere hold them back as little as __ldg (plain loads of an
// eviction's weights took a microsecond more, 20 and 103).
__device__ __forceinline__ float load_late(const float* p) {
  float x;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ float4 load_late(const float4* p) {
  float4 x;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
  return x;
}

// ---- launchers (each returns the launch's error) ----

cudaError_t rope_table(int positions, int rot, double base, double factor, float* table,
                       cudaStream_t s);

struct AppendArgs {
  const bf16 *q, *k, *v;                     // token rows; q may be null
  long long q_stride, k_stride, v_stride;    // elements between tokens
  int tokens, q_heads;
  const float *q_norm, *k_norm;              // [dim] or null
  float eps;
  const float* rope;                         // [positions][rot]
  int positions, rot, interleaved;
  const int *cu, *start;                     // [batch + 1], [batch]
  const int* rope_start = nullptr;           // [batch]: positions for the rotation where they are not the places
  bf16 *q_out, *k_out;                       // dense; k_out may be null
};
cudaError_t rope_append_kv8(const Kv8View& c, const AppendArgs& a, int* err_flag,
                            cudaStream_t s);

cudaError_t kv8_read(const Kv8View& c, const int* cu, const int* first, int tokens, bf16* k_out,
                     bf16* v_out, int* err_flag, cudaStream_t s);

// Workspace of attention_kv8 (partial results of sequences split over CTAs).
size_t attention_kv8_workspace(int dim, int num_sms);
cudaError_t attention_kv8(const Kv8View& c, const bf16* q, int q_tokens, int q_heads,
                          const int* kv_len, float scale, int causal, bf16* out, float* lse,
                          void* workspace, int* err_flag, int num_sms, cudaStream_t s);

cudaError_t attention_packed(const bf16* q, long long q_stride, const bf16* k, long long k_stride,
                             const bf16* v, long long v_stride, int tokens_q, int tokens_k,
                             int batch, int q_heads, int kv_heads, int dim, const int* cu_q,
                             const int* cu_k, float scale, int frame, bf16* out, float* lse,
                             int* err_flag, int num_sms, cudaStream_t s);

}  // namespace jepa
