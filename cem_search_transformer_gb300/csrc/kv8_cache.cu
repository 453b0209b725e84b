// Filling and reading the 8-bit paged key/value cache: per-head RMS norm and rotary position of
// queries and keys, quantisation of keys and values to e4m3 with one power-of-two scale per
// (page, head), and the read-back to bf16.
//
// Bound by bytes on long appends (2 (q_heads + 2 kv_heads) dim read, 2 q_heads dim + 2 kv_heads dim
// written a token) and by latency on short ones. Nine prompts of 100 to 4500 tokens, 32 query heads
// over 8 of 128: queries 57 us (5.6 TB/s), keys 30 us (2 TB/s: a page's chain of search, table,
// loads, angles and maximum with 16 warps a SM), read-back 26 us (4.6 TB/s). A page and head is quantised by exactly one team
// of warps: that of its "owner", the first new token that lies in the page. No atomics: the result
// depends neither on the launch shape nor on the order of blocks.
#include "rope_rows.cuh"

#include <cuda_fp16.h>

#include <cmath>

namespace jepa {

namespace {

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(hi), "f"(lo));
  return p;
}
__device__ __forceinline__ float2 e4m3x2_values(uint16_t p) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8], float inv) {
  uint2 u;
  u.x = (uint32_t)e4m3x2(y[0] * inv, y[1] * inv) | ((uint32_t)e4m3x2(y[2] * inv, y[3] * inv) << 16);
  u.y = (uint32_t)e4m3x2(y[4] * inv, y[5] * inv) | ((uint32_t)e4m3x2(y[6] * inv, y[7] * inv) << 16);
  return u;
}
// A scale as the cache's contract has it: positive and within [2^-40, 2^40].
__device__ __forceinline__ float sane_scale(float s) {
  return s >= KV8_SCALE_MIN ? fminf(s, KV8_SCALE_MAX) : KV8_SCALE_MIN;
}

template <class LaneT>
__device__ __forceinline__ void store_codes(uint8_t* row, const LaneT& ln, const float (&y)[16], float inv) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = y[i];
    b[i] = y[8 + i];
  }
  *reinterpret_cast<uint2*>(row + 8 * ln.c0) = e4m3x8(a, inv);
  *reinterpret_cast<uint2*>(row + 8 * ln.c1) = e4m3x8(b, inv);
}
__device__ __forceinline__ float abs_max(const float (&y)[16], float m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(y[i]));   // fmaxf drops NaN
  return m;
}

__device__ __forceinline__ float abs_max(const uint4 (&u)[2], float m) {
  __nv_bfloat162 x = __float2bfloat162_rn(m);   // exact: m is a bf16 value here
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = w[i] & 0x7fff7fffu;
      x = __hmax2(x, *reinterpret_cast<const __nv_bfloat162*>(&b));   // drops NaN
    }
  }
  return fmaxf(__low2float(x), __high2float(x));
}

// Codes of a page's `off` earlier tokens moved to a scale 1 / factor times theirs (exact but for
// codes that become subnormal), `members` threads together.
template <int D>
__device__ __forceinline__ void rescale_codes(uint8_t* base, int off, float factor, int member,
                                              int members) {
  for (int i = member; i < off * (D / 8); i += members) {
    uint2* at = reinterpret_cast<uint2*>(base) + i;
    const uint2 u = *at;
    float z[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = e4m3x2_values((uint16_t)((k < 2 ? u.x : u.y) >> (16 * (k & 1))));
      z[2 * k] = f.x;
      z[2 * k + 1] = f.y;
    }
    *at = e4m3x8(z, factor);
  }
}

// The part of a sequence's new tokens that lies in one page.
struct Piece {
  int t, n, off, pos, page;   // first packed token, tokens, slot in the page, position, page (-1: bad)
};
// What begins at packed token t of the sequence `at`; false where t's page belongs to an earlier
// owner. Advances t behind it.
__device__ __forceinline__ bool next_piece(const Kv8View& c, const AppendArgs& a, const Place& at,
                                           int& t, Piece& p) {
  p.t = t;
  p.pos = (int)((unsigned)at.first + (unsigned)(t - at.begin));
  p.off = p.pos & (c.page - 1);
  p.n = min(c.page - p.off, at.end - t);
  t += p.n;
  if (p.t != at.begin && p.off != 0) return false;
  p.page = at.first >= 0 && p.pos >= 0 && (long long)p.pos + p.n <= positions_of(c, a)
               ? kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, at.s, p.pos)
               : -1;
  return true;
}

// Short appends (a few tokens a sequence): a warp takes one owner token and, of k or v, as many
// heads as it has groups of D / 16 lanes. Segments of more than one token are read twice.
template <int D, bool INTER>
__device__ __forceinline__ void append_short(const Kv8View& c, const AppendArgs& a, long long unit,
                                             int* err_flag) {
  constexpr int L = D / 16, HEADS = 32 / L;
  const int blocks = (c.heads + HEADS - 1) / HEADS;
  const bool is_v = unit & 1;
  const int t0 = (int)((unit >> 1) / blocks), h0 = (int)((unit >> 1) - (long long)t0 * blocks) * HEADS;
  if (t0 >= a.tokens) return;
  const int lane = threadIdx.x & 31, head = h0 + lane / L;
  const bool on = head < c.heads;
  const Lane<D, INTER> ln(a.rot);
  const bf16* src = (is_v ? a.v : a.k) + (long long)(on ? head : 0) * D;
  const long long stride = is_v ? a.v_stride : a.k_stride;
  uint4 raw[2];
  load16(src + t0 * stride, ln, raw);
  const Place at = locate(a.cu, a.start, c.batch, t0);
  if (!holds(at, t0, a.tokens)) return;
  int t = t0;
  Piece p;
  if (!next_piece(c, a, at, t, p)) return;
  if (p.page < 0) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  const long long block = (long long)p.page * c.heads + (on ? head : 0);
  float* const scale_at = (is_v ? c.v_scale : c.k_scale) + block;
  const float was = p.off != 0 ? sane_scale(*scale_at) : 0.f;
  // row r of the segment, normed and rotated (keys); all lanes call it
  auto row_values = [&](int r, float (&y)[16]) {
    if (r > 0) load16(src + (p.t + r) * stride, ln, raw);
    widen(raw, y);
    if (!is_v) {
      float an[16];
      if (ln.rotates) load_angles(an, a.rope + (long long)(p.pos + r) * a.rot, a.rot, ln.p);
      norm_rotate<D, INTER>(y, ln, a.k_norm, a.eps, an);
    }
  };
  float y[16], m = 0.f;
  for (int r = p.n - 1; r >= 0; --r) {   // the first row last: it then is at hand
    if (r == 0 && p.n > 1) load16(src + p.t * stride, ln, raw);
    row_values(r, y);
    m = abs_max(y, m);
  }
#pragma unroll
  for (int o = L / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!on) m = 0.f;
  float scale = pow2(kv8_exponent(__float_as_uint(m)));
  uint8_t* const base = (is_v ? c.v : c.k) + block * ((long long)c.page * D);
  __syncwarp();                          // all lanes have read the scale
  if (p.off != 0 && on) {
    if (scale > was) rescale_codes<D>(base, p.off, was / scale, lane % L, L);
    scale = fmaxf(scale, was);           // a page that holds tokens never shrinks its scale
  }
  if (on && lane % L == 0) *scale_at = scale;
  const float inv = 1.0f / scale;
  for (int r = 0; r < p.n; ++r) {
    if (r > 0) row_values(r, y);
    if (on) {
      store_codes(base + (long long)(p.off + r) * D, ln, y, inv);
      if (!is_v && a.k_out) store16(a.k_out + ((long long)(p.t + r) * c.heads + head) * D, ln, y);
    }
  }
}

// Short appends: key / value warps, then query warps, in one grid. Three CTAs a SM: two, with a few
// registers more, take a fifth longer where there are waves of them (4000 single tokens 35 us, 28).
template <int D, bool INTER>
__global__ void __launch_bounds__(THREADS, 3) k_append_short(Kv8View c, AppendArgs a, long long kv_units,
                                                          int* err_flag) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long unit = (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  if (unit < kv_units)
    append_short<D, INTER>(c, a, unit, err_flag);
  else if (a.q)
    rotate_queries<D, INTER>(c, a, unit - kv_units, err_flag);
  report_offsets(a.cu, c.batch, a.tokens, err_flag);
}

// Long appends: a team of T warps takes a chunk of `page` packed tokens of one head and
// quantises the pages that have their owner in it (two at most for a long sequence). Each lane
// holds IT rows' 16 elements between the maximum and the codes, so that the rows are read once.
template <int D, bool INTER, int T, int IT, bool V>
__device__ __forceinline__ void append_pages(const Kv8View& c, const AppendArgs& a, long long units,
                                             int* err_flag) {
  constexpr int L = D / 16, WARPS = THREADS / 32, ROWS = T * (32 / L);   // tokens a pass
  __shared__ float red[2][WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / T;
  const long long unit = (long long)blockIdx.x * (WARPS / T) + team;
  if (unit >= units) return;
  const int head = (int)(unit % c.heads);
  const int t0 = (int)(unit / c.heads) << c.page_log2;
  const int member = (warp % T) * 32 + lane, row = member / L;
  const Lane<D, INTER> ln(a.rot);
  const bf16* src = (V ? a.v : a.k) + (long long)head * D;
  const long long stride = V ? a.v_stride : a.k_stride;
  Place at = locate(a.cu, a.start, c.batch, t0);
  if (at.s < 0) {                          // the chunk begins ahead of the first sequence
    at.s = 0;
    at.begin = __ldg(a.cu);
    at.end = __ldg(a.cu + 1);
    at.first = __ldg(a.start);
  }
  const int t1 = min(t0 + c.page, a.tokens);
  int parity = 0;
  for (int t = max(t0, at.begin); t < t1;) {
    while (t >= at.end) {                  // the next sequence that has tokens
      if (++at.s >= c.batch) return;
      at.begin = at.end;
      at.end = __ldg(a.cu + at.s + 1);
      at.first = __ldg(a.start + at.s);
    }
    if (!kv8_span_ok(at.begin, at.end, a.tokens)) {
      t = at.end;
      continue;
    }
    Piece p;
    if (!next_piece(c, a, at, t, p)) continue;
    if (p.page < 0) {
      if (member == 0) atomicOr(err_flag, DEV_ERR_INDEX);
      continue;
    }
    const long long block = (long long)p.page * c.heads + head;
    float* const scale_at = (V ? c.v_scale : c.k_scale) + block;
    const float was = p.off != 0 ? sane_scale(*scale_at) : 0.f;
    uint4 raw[IT][2];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * ROWS + row;
      raw[it][0] = raw[it][1] = make_uint4(0, 0, 0, 0);
      if (r < p.n) load16(src + (long long)(p.t + r) * stride, ln, raw[it]);
    }
    float y[V ? 1 : IT][16], m = 0.f;   // keys between the maximum and the codes; values stay raw
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * ROWS + row;
      if (V) {
        m = abs_max(raw[it], m);         // rows past the end are zeros
      } else {
        widen(raw[it], y[it]);
        float an[16];
        if (ln.rotates && r < p.n) load_angles(an, a.rope + (long long)(p.pos + r) * a.rot, a.rot, ln.p);
        norm_rotate<D, INTER>(y[it], ln, a.k_norm, a.eps, an);
        if (r < p.n) m = abs_max(y[it], m);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (T > 1) {
      if (lane == 0) red[parity][warp] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(T * 32) : "memory");
#pragma unroll
      for (int i = 0; i < T; ++i) m = fmaxf(m, red[parity][team * T + i]);
      parity ^= 1;
    } else {
      __syncwarp();                        // all lanes have read the scale
    }
    float scale = pow2(kv8_exponent(__float_as_uint(m)));
    uint8_t* const base = (V ? c.v : c.k) + block * ((long long)c.page * D);
    if (p.off != 0) {
      if (scale > was) rescale_codes<D>(base, p.off, was / scale, member, T * 32);
      scale = fmaxf(scale, was);           // a page that holds tokens never shrinks its scale
    }
    if (member == 0) *scale_at = scale;
    const float inv = 1.0f / scale;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * ROWS + row;
      if (r >= p.n) continue;
      if (V) widen(raw[it], y[0]);
      store_codes(base + (long long)(p.off + r) * D, ln, y[V ? 0 : it], inv);
      if (!V && a.k_out) store16(a.k_out + ((long long)(p.t + r) * c.heads + head) * D, ln, y[V ? 0 : it]);
    }
  }
}

// Values and keys in a kernel each: values need half the registers and no arithmetic but the scale,
// so twice the warps (nine prompts of 100 to 4500 tokens, 8 heads of 128: 123 us with the queries and
// the read-back, 127 with both in one kernel; queries in the same grid too: 150). They share no
// data with the kernel ahead of them in the call and run beside its last blocks (24 frames of 258
// tokens: 35 us, 42 one after the other); the wait at the end keeps the order for what comes next.
template <int D, bool INTER, int T, int IT, bool V>
__global__ void __launch_bounds__(THREADS, V ? 4 : 2)
    k_append_pages(Kv8View c, AppendArgs a, long long units, int* err_flag) {
  asm volatile("griddepcontrol.launch_dependents;");
  append_pages<D, INTER, T, IT, V>(c, a, units, err_flag);
  if (V) report_offsets(a.cu, c.batch, a.tokens, err_flag);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Cached tokens back as bf16 (code * power of two has at most four significant bits: exact).
// A warp per packed token; a lane moves 16 codes at a time.
template <int D>
__device__ __forceinline__ void read_token(const Kv8View& c, const int* __restrict__ cu,
                                           const int* __restrict__ first, int tokens,
                                           bf16* __restrict__ k_out, bf16* __restrict__ v_out,
                                           int* err_flag) {
  const int t = (int)(((long long)blockIdx.x * THREADS + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const Place p = locate(cu, first, c.batch, t);
  if (!holds(p, t, tokens)) return;
  const int pos = (int)((unsigned)p.first + (unsigned)(t - p.begin));
  const int pg =
      p.first < 0 ? -1 : kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, p.s, pos);
  if (pg < 0) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  const int off = pos & (c.page - 1), vecs = c.heads * (D / 16);
  constexpr int AHEAD = 4;                 // loads a lane has in flight
  for (int i0 = lane; i0 < 2 * vecs; i0 += 32 * AHEAD) {
    uint4 u[AHEAD];
    float scale[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + 32 * k;
      if (i >= 2 * vecs) break;
      const bool is_v = i >= vecs;
      const int j = is_v ? i - vecs : i, head = j / (D / 16), e0 = 16 * (j % (D / 16));
      const long long block = (long long)pg * c.heads + head;
      u[k] = *reinterpret_cast<const uint4*>((is_v ? c.v : c.k) + (block * c.page + off) * D + e0);
      scale[k] = (is_v ? c.v_scale : c.k_scale)[block];
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + 32 * k;
      if (i >= 2 * vecs) break;
      const bool is_v = i >= vecs;
      const int j = is_v ? i - vecs : i;
      const float f = sane_scale(scale[k]);
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      float z[2][8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 x = e4m3x2_values((uint16_t)(w[q >> 1] >> (16 * (q & 1))));
        z[q >> 2][2 * (q & 3)] = x.x * f;
        z[q >> 2][2 * (q & 3) + 1] = x.y * f;
      }
      bf16* to = (is_v ? v_out : k_out) + (long long)t * c.heads * D + 16 * j;
      store8(to, z[0]);
      store8(to + 8, z[1]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 5) k_kv8_read(Kv8View c, const int* __restrict__ cu,
                                                      const int* __restrict__ first, int tokens,
                                                      bf16* __restrict__ k_out,
                                                      bf16* __restrict__ v_out, int* err_flag) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  read_token<D>(c, cu, first, tokens, k_out, v_out, err_flag);
  report_offsets(cu, c.batch, tokens, err_flag);
}

// cos and sin of position / factor * base^(-2 i / rot), in 64 bits: fp32 angles of far positions
// would be off by whole degrees' worth of rounding (position 10^6: 2^-4 rad).
__global__ void k_rope_table(int positions, int rot, double log2_base, double inv_factor,
                             float* __restrict__ table) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int half = rot >> 1;
  if (i >= (long long)positions * half) return;
  const int p = (int)(i / half), j = (int)(i % half);
  double sn, cs;
  sincos((double)p * inv_factor * exp2(-log2_base * (2.0 * j / rot)), &sn, &cs);
  table[(long long)p * rot + j] = (float)cs;
  table[(long long)p * rot + half + j] = (float)sn;
}

template <int D, bool INTER, int PAGE, int T, int IT>
cudaError_t launch_pages(const Kv8View& c, const AppendArgs& a, int* err_flag, cudaStream_t s) {
  static_assert(T * (512 / D) * IT == PAGE, "a team's lanes hold a page's rows, no less and no more");
  const long long units = (((long long)a.tokens + c.page - 1) >> c.page_log2) * c.heads;
  const long long blocks = blocks_for(units * T * 32, c.batch);   // a team has T warps
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = launch_early(k_append_pages<D, INTER, T, IT, true>, (unsigned)blocks, a.q != nullptr, s,
                                     c, a, units, err_flag);
  if (e != cudaSuccess) return e;
  return launch_early(k_append_pages<D, INTER, T, IT, false>, (unsigned)blocks, true, s, c, a, units, err_flag);
}

template <int D, bool INTER>
cudaError_t launch_append(const Kv8View& c, const AppendArgs& a, int* err_flag, cudaStream_t s) {
  constexpr int WARPS = THREADS / 32, HEADS = 32 / (D / 16);
  const long long q_units = a.q ? (long long)a.tokens * ((a.q_heads + Q_HEADS - 1) / Q_HEADS) : 0;
  // Up to four new tokens a sequence on average: latency, one launch. The lengths are on the device, so
  // the average is all there is to go by, and either side of it has its batches. Uniform ones of 64
  // sequences, 8 heads of 128, pages of 64, here / the page kernels: 5 tokens 12 / 33 us, 8 14 / 23,
  // 16 21 / 16; pages of 128: 5 12 / 54, 16 21 / 23 (a team's sequences come one after the other).
  // A higher limit would send pieces of a page among single tokens here, a row at a time: 12 of 64
  // tokens beside 200 single ones 76 us, the page kernels 15.
  if (a.tokens <= 4LL * c.batch) {
    const long long kv_units = 2LL * a.tokens * ((c.heads + HEADS - 1) / HEADS);
    const long long blocks = blocks_for(32 * (kv_units + q_units), c.batch);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(k_append_short<D, INTER>, (unsigned)blocks, true, s, c, a, kv_units, err_flag);
  }
  if (q_units) {
    const long long blocks = (q_units + WARPS - 1) / WARPS;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    k_rope_queries<D, INTER><<<(unsigned)blocks, THREADS, 0, s>>>(c, a, err_flag);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // 64 elements a lane (32 where a page of 16 rows gives one warp no more)
  if constexpr (D == 128) {
    switch (c.page) {
      case 16: return launch_pages<D, INTER, 16, 1, 4>(c, a, err_flag, s);
      case 32: return launch_pages<D, INTER, 32, 2, 4>(c, a, err_flag, s);
      case 64: return launch_pages<D, INTER, 64, 4, 4>(c, a, err_flag, s);
      default: return launch_pages<D, INTER, 128, 8, 4>(c, a, err_flag, s);
    }
  } else {
    switch (c.page) {
      case 16: return launch_pages<D, INTER, 16, 1, 2>(c, a, err_flag, s);
      case 32: return launch_pages<D, INTER, 32, 1, 4>(c, a, err_flag, s);
      case 64: return launch_pages<D, INTER, 64, 2, 4>(c, a, err_flag, s);
      default: return launch_pages<D, INTER, 128, 4, 4>(c, a, err_flag, s);
    }
  }
}

}  // namespace

cudaError_t rope_append_kv8(const Kv8View& c, const AppendArgs& a, int* err_flag,
                            cudaStream_t s) {
  if (a.tokens <= 0) return cudaSuccess;
  if (c.dim == 64)
    return a.interleaved ? launch_append<64, true>(c, a, err_flag, s)
                         : launch_append<64, false>(c, a, err_flag, s);
  if (c.dim == 128)
    return a.interleaved ? launch_append<128, true>(c, a, err_flag, s)
                         : launch_append<128, false>(c, a, err_flag, s);
  return cudaErrorInvalidValue;
}

cudaError_t kv8_read(const Kv8View& c, const int* cu, const int* first, int tokens, bf16* k_out,
                     bf16* v_out, int* err_flag, cudaStream_t s) {
  if (tokens <= 0) return cudaSuccess;
  const unsigned grid = (unsigned)blocks_for(32LL * tokens, c.batch);
  if (c.dim == 64)
    return launch_early(k_kv8_read<64>, grid, true, s, c, cu, first, tokens, k_out, v_out, err_flag);
  if (c.dim == 128)
    return launch_early(k_kv8_read<128>, grid, true, s, c, cu, first, tokens, k_out, v_out, err_flag);
  return cudaErrorInvalidValue;
}

cudaError_t rope_table(int positions, int rot, double base, double factor, float* table,
                       cudaStream_t s) {
  const long long n = (long long)positions * (rot >> 1);
  if (n <= 0) return cudaSuccess;
  const long long blocks = (n + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_rope_table<<<(unsigned)blocks, THREADS, 0, s>>>(positions, rot, log2(base), 1.0 / factor, table);
  return cudaGetLastError();
}

}  // namespace jepa
