// Filling and reading the 4-bit paged key/value cache: per-head RMS norm and rotary position of
// queries and keys, keys and values to e2m1 codes with an e4m3 scale for every 16 elements, and
// the read-back to bf16.
//
// Bound by bytes on long appends (2 (q_heads + 2 kv_heads) dim read, 2 q_heads dim + 9/8 kv_heads dim
// written a token) and by latency on short ones. No token's codes depend on another token: a warp
// takes a token and up to eight heads of its queries, keys or values, which share the angles.
//
// Measured: nine prompts of 100 to 4500 tokens, 32 query heads over 8 of 128: append 97 us (4.5 TB/s; issue 65% of the
// slots), read-back 20 (4.5 TB/s), both 115; one token for each of 64 sequences 4 us each (latency).
//
// A code is the nearest e2m1 value to x / (scale * unit), and neighbours are a third apart, so what
// decides between them is computed as the definition has it: the norm's factor is correctly rounded (sum of
// squares in two floats), the products of the rotation are rounded one by one, and quotients are correctly rounded.
#include "rope_rows.cuh"

#include "kv4.cuh"

namespace jepa {

namespace {

constexpr int HEADS = 8;   // heads of a token that a warp takes

typedef unsigned long long pair;   // two fp32 numbers (the packed operations of common.cuh)

__device__ __forceinline__ pair f2_sub(pair a, pair b) { return f2_fma(b, f2_pack(-1.f, -1.f), a); }
__device__ __forceinline__ pair f2_both(float x) { return f2_pack(x, x); }

__device__ __forceinline__ void two_sum(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

// Whether a mean of squares (with its epsilon) was taken within fp32: neither past its end (NaN and infinities count as
// that) nor where squares vanish.
__device__ __forceinline__ bool mean_in_range(float m) {
  return __float_as_uint(m) - 0x0a800000u < 0x7b800000u - 0x0a800000u;   // 2^-106 <= m < 2^120
}
// A mean of squares from 64 bits, brought into fp32 with its head: x * f has the mean m + rest.
struct NearMean {
  float f, m, rest;
  __device__ __forceinline__ explicit NearMean(double mean) {
    const int e = (__double2hiint(mean) >> 20 & 0x7ff) - 1023, k = max(-120, min(120, e >> 1));
    f = pow2(-k);
    const double near = mean * f * f;
    m = (float)near;
    rest = (float)(near - m);
  }
};

// 1 / sqrt(sum / D + eps), correctly rounded but for ties of 2^-40: the sum of squares, which are
// exact in fp32, over the lanes of a head in two floats, and one Newton step whose remainder is exact.
// y: a lane's elements in pairs. Heads whose squares leave fp32, at either end, have their sum in 64 bits and are brought
// near 1 by a power of two: the factor is that of the y that is left (nine prompts: 0.6 us of 114 for the look).
template <int D>
__device__ __forceinline__ float norm_factor(pair (&y)[8], float eps) {
  constexpr int L = D / 16;
  pair hi2 = f2_mul(y[0], y[0]), lo2 = f2_both(0.f);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const pair x = f2_mul(y[i], y[i]), s = f2_add(hi2, x), b = f2_sub(s, hi2);
    lo2 = f2_add(lo2, f2_add(f2_sub(hi2, f2_sub(s, b)), f2_sub(x, b)));
    hi2 = s;
  }
  const float2 h2 = f2_unpack(hi2), l2 = f2_unpack(lo2);
  float hi = h2.x, lo = __fadd_rn(l2.x, l2.y);
  two_sum(hi, lo, h2.y);
#pragma unroll
  for (int o = L / 2; o; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
    // both lanes add the larger to the smaller in the same order
    float a = fmaxf(hi, h), b = __fadd_rn(lo, l);
    two_sum(a, b, fminf(hi, h));
    hi = a;
    lo = b;
  }
  hi *= 1.0f / D;
  lo *= 1.0f / D;
  two_sum(hi, lo, eps);
  float m = __fadd_rn(hi, lo), rest = __fsub_rn(lo, __fsub_rn(m, hi));
  const bool far = !mean_in_range(m);
  if (__any_sync(0xffffffffu, far)) {
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = f2_unpack(y[i]);
      sum += (double)x.x * x.x + (double)x.y * x.y;
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (far) {
      const NearMean near(sum / D + eps);
      m = near.m;
      rest = near.rest;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = f2_mul(y[i], f2_both(near.f));
    }
  }
  const float r = __frsqrt_rn(m);
  if (!(m > 0.f && m < INFINITY)) return r;
  const float t = __fmul_rn(m, r), tl = __fmaf_rn(m, r, -t);    // m r = t + tl
  float e = __fmaf_rn(-t, r, 1.f);                              // 1 - (m + rest) r^2
  e = __fmaf_rn(-tl, r, e);
  e = __fmaf_rn(-rest, __fmul_rn(r, r), e);
  return __fmaf_rn(0.5f * r, e, r);
}

// y = x * (r * w), then (a, b) -> (a cos - b sin, b cos + a sin), each product and sum rounded. A lane's
// elements in pairs (2 i, 2 i + 1) of its two chunks.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate_exact(pair (&y)[8], const Lane<D, INTER>& ln,
                                                  const float* __restrict__ w, float eps,
                                                  const float (&an)[16]) {
  if (w) {
    const pair r = f2_both(norm_factor<D>(y, eps));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 g = load_late(reinterpret_cast<const float4*>(w + 8 * (i < 4 ? ln.c0 : ln.c1) + 2 * (i & 3)));
      y[i] = f2_mul(y[i], f2_mul(r, f2_pack(g.x, g.y)));
      y[i + 1] = f2_mul(y[i + 1], f2_mul(r, f2_pack(g.z, g.w)));
    }
  }
  if (ln.rotates) {
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = f2_unpack(y[i]);
        y[i] = f2_pack(__fsub_rn(__fmul_rn(p.x, an[i]), __fmul_rn(p.y, an[8 + i])),
                       __fadd_rn(__fmul_rn(p.y, an[i]), __fmul_rn(p.x, an[8 + i])));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const pair c = f2_pack(an[2 * i], an[2 * i + 1]), sn = f2_pack(an[8 + 2 * i], an[9 + 2 * i]);
        const pair p = y[i], q = y[4 + i];
        y[i] = f2_sub(f2_mul(p, c), f2_mul(q, sn));
        y[4 + i] = f2_add(f2_mul(q, c), f2_mul(p, sn));
      }
    }
  }
}

// Largest of three, NaN where there is one.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Largest magnitude of 8 elements; NaN where there is one.
__device__ __forceinline__ float top_of(const pair (&y)[8], int from) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = f2_unpack(y[from + i]);
    m = max3(m, fabsf(x.x), fabsf(x.y));
  }
  return m;
}

// The largest magnitudes of the two blocks of 16 that a lane's chunks of 8 lie in. All lanes of the
// warp call it.
template <int D, bool INTER>
__device__ __forceinline__ void block_tops(const pair (&y)[8], const Lane<D, INTER>& ln, int rot,
                                           float (&top)[2]) {
  const float a = top_of(y, 0), b = top_of(y, 4);
  top[0] = top[1] = max3(a, b, 0.f);        // neighbours: one block
  if (INTER) return;
  constexpr int L = D / 16;
  const int first = (threadIdx.x & 31) / L * L, lanes = rot >> 4;   // lanes of a head that rotate
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int other = (h ? ln.c1 : ln.c0) ^ 1;                      // the block's other chunk
    const int src = first + (ln.rotates ? (other < lanes ? other : other - lanes) : ln.p);
    const float x = __shfl_sync(0xffffffffu, a, src), z = __shfl_sync(0xffffffffu, b, src);
    if (ln.rotates) top[h] = max3(h ? b : a, other < lanes ? x : z, 0.f);
  }
}

// x / d, correctly rounded: `inv` is 1 / d to a step or two, and the remainder of its quotient is exact.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
  const float z = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-z, d, x), inv, z);
}

// Code of a block's scale for its largest magnitude: e4m3(top / 6 / unit), nearest even, at least
// 2^-9; NaN where the block is not finite.
__device__ __forceinline__ uint32_t scale_code(float top, float inv_unit) {
  if (!(top < INFINITY)) return 0x7f;
  const float s = fmaxf(__fmul_rn(quotient(top, 6.f, 1.f / 6.f), inv_unit), KV4_SCALE_MIN);
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(0.f), "f"(s));
  return p & 0xffu;
}

// Codes of 8 elements, the first in the lowest bits. `most`: the scale is e4m3's largest, so that quotients may
// lie far beyond 6.
__device__ __forceinline__ uint32_t e2m1x8(const pair (&y)[8], int from, float scale, bool most) {
  float inv1;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv1) : "f"(scale));
  const pair inv = f2_both(inv1), neg = f2_both(-scale);
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const pair x = y[from + i], z = f2_mul(x, inv);
    const float2 f = f2_unpack(f2_fma(f2_fma(z, neg, x), inv, z));   // the quotients, correctly rounded
    q[2 * i] = f.x;
    q[2 * i + 1] = f.y;
  }
  if (most) {
    // a quotient past fp32 has no remainder: infinity less infinity. Its code is that of 8, as of all beyond 6
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = f2_unpack(y[from + i / 2]);
      const float one = i & 1 ? x.y : x.x;
      if (fabsf(one) > 8.f * scale) q[i] = copysignf(8.f, one);
    }
  }
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

// A lane's 16 elements into the cache: `at` counts tokens of all (page, head) blocks.
template <int D, bool INTER>
__device__ __forceinline__ void quantise_store(uint8_t* codes, uint8_t* scales, long long at, bool on,
                                               const pair (&y)[8], const Lane<D, INTER>& ln,
                                               int rot, float unit) {
  float top[2];
  block_tops<D, INTER>(y, ln, rot, top);
  if (!on) return;
  const float inv_unit = kv4_inverse(unit);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int chunk = h ? ln.c1 : ln.c0;
    const uint32_t sc = scale_code(top[h], inv_unit);
    const uint32_t f = f16x2_of_e4m3_pair(sc);
    const float scale = __half2float(__ushort_as_half((unsigned short)(f & 0xffffu))) * unit;
    *reinterpret_cast<uint32_t*>(codes + at * (D / 2) + 4 * chunk) =
        sc == 0x7f ? 0u : e2m1x8(y, 4 * h, scale, sc == 0x7e);
    if (!(chunk & 1)) scales[at * (D / 16) + (chunk >> 1)] = (uint8_t)sc;
  }
}

// A warp takes one token and up to HEADS heads of its keys or of its values. Values are not rotated,
// so that a lane's elements are neighbours.
template <int D, bool INTER, bool V>
__device__ __forceinline__ void append_heads(const Kv4View& c, const AppendArgs& a, int t, int h0, int* err_flag) {
  constexpr int L = D / 16, ROWS = 32 / L, PASSES = HEADS / ROWS;
  const int lane = threadIdx.x & 31, sub = lane / L;
  const Lane<D, INTER> ln(a.rot);
  const bf16* src = V ? a.v + t * a.v_stride : a.k + t * a.k_stride;
  uint4 raw[PASSES][2];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int h = h0 + p * ROWS + sub;
    raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    if (h < c.heads) load16(src + (long long)h * D, ln, raw[p]);
  }
  const Place at = locate(a.cu, a.start, c.batch, t);
  if (!holds(at, t, a.tokens)) return;            // left as it is
  int pos, rope_row;
  const int page = place_of<true>(c, a, at, t, pos, rope_row)
                       ? kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, at.s, pos)
                       : -1;
  if (page < 0) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  float an[16];
  if (!V && ln.rotates) load_angles(an, a.rope + (long long)rope_row * a.rot, a.rot, ln.p);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int h = h0 + p * ROWS + sub;
    const bool on = h < c.heads;
    pair y[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t w[4] = {raw[p][q].x, raw[p][q].y, raw[p][q].z, raw[p][q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) y[4 * q + i] = (pair)(w[i] << 16) | ((pair)(w[i] & 0xffff0000u) << 32);
    }
    if (!V) norm_rotate_exact<D, INTER>(y, ln, a.k_norm, a.eps, an);
    const long long row = (((long long)page * c.heads + (on ? h : 0)) << c.page_log2) + (pos & (c.page - 1));
    const float unit = kv4_unit(V ? c.v_unit : c.k_unit, on ? h : 0);
    quantise_store<D, INTER>(V ? c.v : c.k, V ? c.v_scale : c.k_scale, row, on, y, ln, a.rot, unit);
    if (!V && a.k_out && on) {
      float z[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = f2_unpack(y[i]);
        z[2 * i] = f.x;
        z[2 * i + 1] = f.y;
      }
      store16(a.k_out + ((long long)t * c.heads + h) * D, ln, z);
    }
  }
}

// Unit of keys and values: a token's blocks of heads, keys first.
template <int D, bool INTER>
__device__ __forceinline__ void append_unit(const Kv4View& c, const AppendArgs& a, long long unit, int* err_flag) {
  const int blocks = (c.heads + HEADS - 1) / HEADS;
  const long long token = unit / (2 * blocks);
  if (token >= a.tokens) return;
  const int block = (int)(unit - token * (2 * blocks));
  if (block < blocks)
    append_heads<D, INTER, false>(c, a, (int)token, block * HEADS, err_flag);
  else
    append_heads<D, true, true>(c, a, (int)token, (block - blocks) * HEADS, err_flag);
}

// Key / value warps, then query warps, in one grid. Four CTAs a SM in 64 registers: nine prompts of 100 to
// 4500 tokens 93 us, three in 80 registers 103, queries and the rest in a kernel each 99 (all of them without the
// looks for heads whose squares leave fp32, 2 us).
template <int D, bool INTER>
__global__ void __launch_bounds__(THREADS, 4) k_append_kv4(Kv4View c, AppendArgs a, long long kv_units, int* err_flag) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long unit = (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  if (unit < kv_units)
    append_unit<D, INTER>(c, a, unit, err_flag);
  else if (a.q)
    rotate_queries<D, INTER, true>(c, a, unit - kv_units, err_flag);
  report_offsets(a.cu, c.batch, a.tokens, err_flag);
}

// Cached tokens back as bf16 (code * scale has at most six significant bits: exact). A warp per
// packed token; a lane moves 8 elements at a time, so that a warp's stores are whole lines.
template <int D>
__device__ __forceinline__ void read_token(const Kv4View& c, const int* cu, const int* first, int tokens,
                                           bf16* __restrict__ k_out, bf16* __restrict__ v_out,
                                           int* err_flag) {
  const long long t = ((long long)blockIdx.x * THREADS + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const Place p = locate(cu, first, c.batch, (int)t);
  if (!holds(p, (int)t, tokens)) return;
  const int pos = (int)((unsigned)p.first + (unsigned)((int)t - p.begin));
  const int pg =
      p.first < 0 ? -1 : kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, p.s, pos);
  if (pg < 0) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  // A lane's place in a head stays the same from turn to turn: its addresses move on by constants.
  constexpr int CH = D / 8, TURN = 32 / CH, AHEAD = 4;   // chunks a head, heads of a turn, turns in flight
  const int chunk = lane % CH, h0 = lane / CH;
  const long long row = (((long long)pg * c.heads + h0) << c.page_log2) + (pos & (c.page - 1));
  const long long codes = row * (D / 2) + 4 * chunk, scales = row * (D / 16) + (chunk >> 1);
  const long long out = (t * c.heads + h0) * D + 8 * chunk;
  const int step = TURN << c.page_log2;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const uint8_t *from = (kind ? c.v : c.k) + codes, *sc_from = (kind ? c.v_scale : c.k_scale) + scales;
    const float* units = kind ? c.v_unit : c.k_unit;
    bf16* to = (kind ? v_out : k_out) + out;
    for (int h = h0; h < c.heads; h += TURN * AHEAD) {
      uint32_t u[AHEAD], sc[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (h + TURN * k < c.heads) {
          u[k] = *reinterpret_cast<const uint32_t*>(from + (long long)(step * k) * (D / 2));
          sc[k] = sc_from[(long long)(step * k) * (D / 16)];
        }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (h + TURN * k < c.heads) {
          const uint32_t f2 = f16x2_of_e4m3_pair(sc[k]);
          const float f = __half2float(__ushort_as_half((unsigned short)(f2 & 0xffffu))) * kv4_unit(units, h + TURN * k);
          const uint32_t x[4] = {f16x2_of_e2m1x2<0>(u[k]), f16x2_of_e2m1x2<1>(u[k]), f16x2_of_e2m1x2<2>(u[k]),
                                 f16x2_of_e2m1x2<3>(u[k])};
          float z[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[q]));
            z[2 * q] = y.x * f;
            z[2 * q + 1] = y.y * f;
          }
          store8(to + TURN * k * D, z);
        }
      from += (long long)(step * AHEAD) * (D / 2);
      sc_from += (long long)(step * AHEAD) * (D / 16);
      to += TURN * AHEAD * D;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 5)
    k_kv4_read(Kv4View c, const int* cu, const int* first, int tokens,
               bf16* __restrict__ k_out, bf16* __restrict__ v_out, int* err_flag) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  read_token<D>(c, cu, first, tokens, k_out, v_out, err_flag);
  report_offsets(cu, c.batch, tokens, err_flag);
}

template <int D, bool INTER>
cudaError_t launch_append(const Kv4View& c, const AppendArgs& a, int* err_flag, cudaStream_t s) {
  const long long q_units = a.q ? (long long)a.tokens * ((a.q_heads + Q_HEADS - 1) / Q_HEADS) : 0;
  const long long kv_units = 2LL * a.tokens * ((c.heads + HEADS - 1) / HEADS);
  const long long blocks = blocks_for(32 * (kv_units + q_units), c.batch);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_early(k_append_kv4<D, INTER>, (unsigned)blocks, true, s, c, a, kv_units, err_flag);
}

}  // namespace

cudaError_t rope_append_kv4(const Kv4View& c, const AppendArgs& a, int* err_flag, cudaStream_t s) {
  if (a.tokens <= 0) return cudaSuccess;
  if (c.dim == 64)
    return a.interleaved ? launch_append<64, true>(c, a, err_flag, s)
                         : launch_append<64, false>(c, a, err_flag, s);
  if (c.dim == 128)
    return a.interleaved ? launch_append<128, true>(c, a, err_flag, s)
                         : launch_append<128, false>(c, a, err_flag, s);
  return cudaErrorInvalidValue;
}

cudaError_t kv4_read(const Kv4View& c, const int* cu, const int* first, int tokens, bf16* k_out,
                     bf16* v_out, int* err_flag, cudaStream_t s) {
  if (tokens <= 0) return cudaSuccess;
  const long long blocks = blocks_for(32LL * tokens, c.batch);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (c.dim == 64)
    return launch_early(k_kv4_read<64>, (unsigned)blocks, true, s, c, cu, first, tokens, k_out, v_out, err_flag);
  if (c.dim == 128)
    return launch_early(k_kv4_read<128>, (unsigned)blocks, true, s, c, cu, first, tokens, k_out, v_out, err_flag);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
