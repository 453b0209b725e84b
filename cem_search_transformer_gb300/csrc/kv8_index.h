// Index arithmetic of the 8-bit paged cache's kernels, in plain C++ so that a host build can
// check it over all its range.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KV8_HD __host__ __device__
#else
#define KV8_HD
#endif

namespace jepa {

// Whether a packed sequence's tokens [begin, end) are rows of a buffer of `tokens` (none is fine).
KV8_HD inline bool kv8_span_ok(int begin, int end, int tokens) {
  // as unsigned a negative offset lies behind every other
  return ((uint32_t)begin <= (uint32_t)end) & ((uint32_t)end <= (uint32_t)tokens);
}

// Page holding position `pos` of sequence s, or -1 where the position, the table's entry or the
// page is out of range.
KV8_HD inline int kv8_page_at(const int* table, int max_pages, int num_pages,
                                           int page_log2, long long s, int pos) {
  const int slot = pos >> page_log2;
  if (pos < 0 || slot >= max_pages) return -1;
  const int pg = table[s * max_pages + slot];
  return pg >= 0 && pg < num_pages ? pg : -1;
}

// Exponent e of a block's scale 2^e: the least with amax <= 448 * 2^e (448 = 1.75 * 2^8), within
// [-40, 40]. amax >= 0, not NaN (infinity takes the largest scale and saturates).
KV8_HD inline int kv8_exponent(uint32_t amax_bits) {
  int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < -40) e = -40;
  if (e > 40) e = 40;
  return e;
}

// Worker w of `workers` takes units [kv8_share(w), kv8_share(w + 1)) of a total.
KV8_HD inline long long kv8_share(long long total, int workers, int w) {
  return total / workers * w + (total % workers < w ? total % workers : w);
}
// The worker whose share holds unit u (inverse of kv8_share).
KV8_HD inline int kv8_worker_of(long long total, int workers, long long u) {
  const long long each = total / workers, more = total % workers;
  if (u < more * (each + 1)) return (int)(u / (each + 1));
  return (int)(more + (u - more * (each + 1)) / each);
}

}  // namespace jepa
