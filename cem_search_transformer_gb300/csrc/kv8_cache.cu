// Filling and reading the 8-bit paged key/value cache: per-head RMS norm and rotary position of
// queries and keys, quantisation of keys and values to e4m3 with one power-of-two scale per
// (page, head), and the read-back to bf16.
//
// A page and head is quantised by exactly one team (a warp or a CTA): the team of its "owner",
// the first new token that lies in the page. No atomics: the result depends neither on the
// launch shape nor on the order of blocks.
#include "kv8.cuh"

#include <cuda_fp16.h>

#include <cmath>

namespace jepa {

namespace {

constexpr int THREADS = 256;

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
__device__ __forceinline__ void load8(const bf16* p, float (&y)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(bf16* p, const float (&y)[8]) {
  uint4 u;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  u.x = w[0]; u.y = w[1]; u.z = w[2]; u.w = w[3];
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A scale as the cache's contract has it: positive and within [2^-40, 2^40].
__device__ __forceinline__ float sane_scale(float s) {
  return s >= KV8_SCALE_MIN ? fminf(s, KV8_SCALE_MAX) : KV8_SCALE_MIN;
}

// Sequence of packed token t: the largest s with cu[s] <= t (cu ascending), found by the whole
// warp with one 32-way probe per level; -1 before the first sequence.
__device__ __forceinline__ int find_sequence(const int* cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  if (__ldg(cu) > t) return -1;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && __ldg(cu + lo + at) <= t;
    const int last = 31 - __clz((int)(__ballot_sync(0xffffffffu, le) | 1u));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// cos / sin of the pairs that a lane's 8 elements (8 c .. 8 c + 7) belong to.
struct Angles {
  float c[8], s[8];
};

template <bool INTER>
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int rot, int e0) {
  if (e0 >= rot) return;
  const int half = rot >> 1;
  if (INTER) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
    a.c[0] = c.x; a.c[1] = c.y; a.c[2] = c.z; a.c[3] = c.w;
    a.s[0] = s.x; a.s[1] = s.y; a.s[2] = s.z; a.s[3] = s.w;
  } else {
    const int at = e0 < half ? e0 : e0 - half;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + at + i));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + at + i));
      a.c[i] = c.x; a.c[i + 1] = c.y; a.c[i + 2] = c.z; a.c[i + 3] = c.w;
      a.s[i] = s.x; a.s[i + 1] = s.y; a.s[i + 2] = s.z; a.s[i + 3] = s.w;
    }
  }
}

// Norm and rotation of one head row held by the D / 8 lanes of a group, 8 elements a lane:
// y = x * w / sqrt(mean(x^2) + eps), then (a, b) -> (a cos - b sin, b cos + a sin) for the pairs
// (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1), i < rot / 2. All lanes of the warp call it.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(float (&y)[8], const float* __restrict__ w, float eps,
                                            const Angles& a, int rot) {
  constexpr int L = D / 8;
  const int lane = threadIdx.x & 31, c = lane % L, e0 = 8 * c;
  if (w) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = __frsqrt_rn(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 g = __ldg(reinterpret_cast<const float4*>(w + e0 + i));
      y[i] *= r * g.x; y[i + 1] *= r * g.y; y[i + 2] *= r * g.z; y[i + 3] *= r * g.w;
    }
  }
  if (INTER) {
    if (e0 < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = y[2 * i], q = y[2 * i + 1];
        y[2 * i] = p * a.c[i] - q * a.s[i];
        y[2 * i + 1] = q * a.c[i] + p * a.s[i];
      }
    }
  } else {
    // the partner elements sit rot / 16 lanes away (rot is a multiple of 16)
    const int away = rot >> 4;
    const bool first = e0 < (rot >> 1), on = e0 < rot;
    const int src = on ? (lane + (first ? away : -away)) : lane;
    float other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, y[i], src);
    if (on) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = first ? y[i] * a.c[i] - other[i] * a.s[i] : y[i] * a.c[i] + other[i] * a.s[i];
    }
  }
}

__device__ __forceinline__ float abs_max(const float (&y)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));   // fmaxf drops NaN
  return m;
}

// Queries: a warp takes one token and up to Q_HEADS_PER_WARP of its heads, so that the angles
// are read once for them.
constexpr int Q_HEADS_PER_WARP = 8;

template <int D, bool INTER>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int batch, int positions_max,
                                               long long unit, int* err_flag) {
  constexpr int L = D / 8, ROWS = 32 / L, PASSES = Q_HEADS_PER_WARP / ROWS;
  const int blocks = (a.q_heads + Q_HEADS_PER_WARP - 1) / Q_HEADS_PER_WARP;
  if (unit >= (long long)a.tokens * blocks) return;
  const int t = (int)(unit / blocks), h0 = (int)(unit % blocks) * Q_HEADS_PER_WARP;
  const int lane = threadIdx.x & 31, sub = lane / L, e0 = 8 * (lane % L);
  float y[PASSES][8];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int h = h0 + p * ROWS + sub;
    if (h < a.q_heads) {
      load8(a.q + t * a.q_stride + (long long)h * D + e0, y[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[p][i] = 0.f;
    }
  }
  const int s = find_sequence(a.cu, batch, t);
  if (s < 0 || t >= __ldg(a.cu + batch)) return;   // behind the last sequence: left as it is
  const int first = __ldg(a.start + s);
  const int pos = (int)((unsigned)first + (unsigned)(t - __ldg(a.cu + s)));
  if (first < 0 || pos < 0 || pos >= positions_max) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  Angles an;
  load_angles<INTER>(an, a.rope + (long long)pos * a.rot, a.rot, e0);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    norm_rotate<D, INTER>(y[p], a.q_norm, a.eps, an, a.rot);
    const int h = h0 + p * ROWS + sub;
    if (h < a.q_heads) store8(a.q_out + ((long long)t * a.q_heads + h) * D + e0, y[p]);
  }
}

// Keys or values of one head for the owners among packed tokens [t0, t1): each owner's segment
// (its page's new tokens) is read once into registers, its maximum taken, and quantised.
// TEAM threads (a warp or the CTA) work together, IT rows of 8 elements a thread.
template <int D, bool INTER, int TEAM, int IT>
__device__ __forceinline__ void append_owned(const Kv8View& c, const AppendArgs& a, int t0, int t1,
                                             int head, bool is_v, float* red, int* err_flag) {
  constexpr int L = D / 8, ROWS = TEAM / L;    // tokens a pass
  const int lane = threadIdx.x & 31, member = TEAM == 32 ? lane : threadIdx.x;
  const int row = member / L, e0 = 8 * (member % L);
  const int limit = min(a.positions, c.max_pages << c.page_log2);
  const int last = min(__ldg(a.cu + c.batch), a.tokens);
  const bf16* src = is_v ? a.v : a.k;
  const long long stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* codes = is_v ? c.v : c.k;
  float* scales = is_v ? c.v_scale : c.k_scale;
  t1 = min(t1, last);
  if (t0 >= t1) return;
  int s = find_sequence(a.cu, c.batch, t0);
  if (s < 0) return;
  for (int t = t0; t < t1;) {
    while (s + 1 < c.batch && __ldg(a.cu + s + 1) <= t) ++s;
    const int begin = __ldg(a.cu + s), end = min(__ldg(a.cu + s + 1), last);
    const int first = __ldg(a.start + s), pos = (int)((unsigned)first + (unsigned)(t - begin));
    if (end <= t) return;                      // offsets that do not ascend
    const int off = pos & (c.page - 1), n = min(c.page - off, end - t);
    if (t != begin && off != 0) {              // this page belongs to an earlier owner
      t += n;
      continue;
    }
    const int pg = first >= 0 && pos + n <= limit
                       ? kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, s, pos)
                       : -1;
    if (pg < 0) {
      if (member == 0) atomicOr(err_flag, DEV_ERR_INDEX);
      t += n;
      continue;
    }
    // row r of the segment, normed and rotated (keys); all threads of the team call it
    auto row_values = [&](int r, float (&z)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = 0.f;
      if (r < n) load8(src + (long long)(t + r) * stride + (long long)head * D + e0, z);
      if (!is_v) {
        Angles an;
        if (r < n) load_angles<INTER>(an, a.rope + (long long)(pos + r) * a.rot, a.rot, e0);
        norm_rotate<D, INTER>(z, a.k_norm, a.eps, an, a.rot);
      }
    };
    float y[IT][8];
    float m = 0.f;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (it * ROWS >= n) break;               // the same for the whole team
      const int r = it * ROWS + row;
      row_values(r, y[it]);
      if (r < n) m = abs_max(y[it], m);
    }
    for (int r0 = IT * ROWS; r0 < n; r0 += ROWS) {   // warps with a long segment: read twice
      float z[8];
      row_values(r0 + row, z);
      if (r0 + row < n) m = abs_max(z, m);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (TEAM > 32) {
      __syncthreads();
      if (lane == 0) red[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TEAM / 32; ++i) m = fmaxf(m, red[i]);
    }
    const long long block = (long long)pg * c.heads + head;
    uint8_t* base = codes + block * ((long long)c.page * D);
    float scale = pow2(kv8_exponent(__float_as_uint(m)));
    if (off != 0) {
      // the page holds `off` earlier tokens: its scale never shrinks, and where it grows their
      // codes move to it (exact but for codes that become subnormal)
      const float was = sane_scale(scales[block]);
      if (TEAM > 32) __syncthreads(); else __syncwarp();   // read by all before it is written
      if (scale > was) {
        const float factor = was / scale;
        for (int i = member; i < off * (D / 8); i += TEAM) {
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
      } else {
        scale = was;
      }
    }
    if (member == 0) scales[block] = scale;
    const float inv = 1.0f / scale;
    auto put = [&](int r, const float (&z)[8]) {
      if (r >= n) return;
      *reinterpret_cast<uint2*>(base + (long long)(off + r) * D + e0) = e4m3x8(z, inv);
      if (!is_v && a.k_out)
        store8(a.k_out + ((long long)(t + r) * c.heads + head) * D + e0, z);
    };
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (it * ROWS >= n) break;
      put(it * ROWS + row, y[it]);
    }
    for (int r0 = IT * ROWS; r0 < n; r0 += ROWS) {
      float z[8];
      row_values(r0 + row, z);
      put(r0 + row, z);
    }
    t += n;
  }
}

// Grid: first the key / value teams, then the query warps.
//   BY_CTA  a CTA per (chunk of `page` packed tokens, head, k | v), for long appends;
//   else    a warp per (token, head, k | v), for short ones: most warps of a long append would
//           find that their token owns nothing.
template <int D, bool INTER, bool BY_CTA, int IT>
__global__ void __launch_bounds__(THREADS) k_rope_append(Kv8View c, AppendArgs a, int kv_blocks,
                                                         int* err_flag) {
  __shared__ float red[THREADS / 32];
  if ((int)blockIdx.x < kv_blocks) {
    if (BY_CTA) {
      const int unit = blockIdx.x, head = (unit >> 1) % c.heads, chunk = (unit >> 1) / c.heads;
      const int t0 = chunk << c.page_log2;
      append_owned<D, INTER, THREADS, IT>(c, a, t0, t0 + c.page, head, unit & 1, red, err_flag);
    } else {
      const long long unit = (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
      const long long th = unit >> 1;
      const int head = (int)(th % c.heads);
      const long long t = th / c.heads;
      if (t < a.tokens)
        append_owned<D, INTER, 32, IT>(c, a, (int)t, (int)t + 1, head, unit & 1, red, err_flag);
    }
  } else {
    const long long unit =
        (long long)(blockIdx.x - kv_blocks) * (THREADS / 32) + (threadIdx.x >> 5);
    rotate_queries<D, INTER>(a, c.batch, min(a.positions, c.max_pages << c.page_log2), unit,
                             err_flag);
  }
}

// Cached tokens back as bf16 (code * power of two has at most four significant bits: exact).
// A warp per packed token; a lane moves 16 codes at a time.
template <int D>
__global__ void __launch_bounds__(THREADS) k_kv8_read(Kv8View c, const int* __restrict__ cu,
                                                      const int* __restrict__ first, int tokens,
                                                      bf16* __restrict__ k_out,
                                                      bf16* __restrict__ v_out, int* err_flag) {
  const int t = (int)(((long long)blockIdx.x * THREADS + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const int s = find_sequence(cu, c.batch, t);
  if (s < 0 || t >= __ldg(cu + c.batch)) return;
  const int f = __ldg(first + s), pos = (int)((unsigned)f + (unsigned)(t - __ldg(cu + s)));
  const int pg =
      f < 0 ? -1 : kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, s, pos);
  if (pg < 0) {
    if (lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  const int off = pos & (c.page - 1), vecs = c.heads * (D / 16);
  for (int i = lane; i < 2 * vecs; i += 32) {
    const bool is_v = i >= vecs;
    const int j = is_v ? i - vecs : i, head = j / (D / 16), e0 = 16 * (j % (D / 16));
    const long long block = (long long)pg * c.heads + head;
    const uint4 u = *reinterpret_cast<const uint4*>((is_v ? c.v : c.k) +
                                                    (block * c.page + off) * D + e0);
    const float scale = sane_scale((is_v ? c.v_scale : c.k_scale)[block]);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float z[2][8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 x = e4m3x2_values((uint16_t)(w[q >> 1] >> (16 * (q & 1))));
      z[q >> 2][2 * (q & 3)] = x.x * scale;
      z[q >> 2][2 * (q & 3) + 1] = x.y * scale;
    }
    bf16* to = (is_v ? v_out : k_out) + ((long long)t * c.heads + head) * D + e0;
    store8(to, z[0]);
    store8(to + 8, z[1]);
  }
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

template <int D, bool INTER>
cudaError_t launch_append(const Kv8View& c, const AppendArgs& a, int* err_flag, cudaStream_t s) {
  constexpr int WARPS = THREADS / 32;
  const long long q_units =
      a.q ? (long long)a.tokens * ((a.q_heads + Q_HEADS_PER_WARP - 1) / Q_HEADS_PER_WARP) : 0;
  const long long q_blocks = (q_units + WARPS - 1) / WARPS;
  // up to four new tokens a sequence on average: one warp holds a segment in registers
  const bool by_warp = a.tokens <= 4LL * c.batch;
  const long long kv_blocks =
      by_warp ? ((long long)a.tokens * c.heads * 2 + WARPS - 1) / WARPS
              : (((long long)a.tokens + c.page - 1) >> c.page_log2) * c.heads * 2;
  if (kv_blocks + q_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(kv_blocks + q_blocks);
  const int per_pass = THREADS / (D / 8);   // tokens a CTA holds in one pass
  if (by_warp)
    k_rope_append<D, INTER, false, 1><<<grid, THREADS, 0, s>>>(c, a, (int)kv_blocks, err_flag);
  else if (c.page <= per_pass)
    k_rope_append<D, INTER, true, 1><<<grid, THREADS, 0, s>>>(c, a, (int)kv_blocks, err_flag);
  else if (c.page <= 2 * per_pass)
    k_rope_append<D, INTER, true, 2><<<grid, THREADS, 0, s>>>(c, a, (int)kv_blocks, err_flag);
  else if (c.page <= 4 * per_pass)
    k_rope_append<D, INTER, true, 4><<<grid, THREADS, 0, s>>>(c, a, (int)kv_blocks, err_flag);
  else
    k_rope_append<D, INTER, true, 8><<<grid, THREADS, 0, s>>>(c, a, (int)kv_blocks, err_flag);
  return cudaGetLastError();
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
  const unsigned grid = (unsigned)(((long long)tokens * 32 + THREADS - 1) / THREADS);
  if (c.dim == 64)
    k_kv8_read<64><<<grid, THREADS, 0, s>>>(c, cu, first, tokens, k_out, v_out, err_flag);
  else if (c.dim == 128)
    k_kv8_read<128><<<grid, THREADS, 0, s>>>(c, cu, first, tokens, k_out, v_out, err_flag);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
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
