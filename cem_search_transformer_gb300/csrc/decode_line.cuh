// What the attention kernels over paged caches share: the line of work that is shared out over the
// CTAs, the rows of a call, and the instructions of the transposed products. attention_kv8.cu says
// why the work is cut like this.
#pragma once

#include "kv8.cuh"

#include <cuda_fp16.h>

namespace jepa {

namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int MAX_CTAS_PER_SM = 4;  // of any shape: sizes the workspace
constexpr int MAX_SMS = 160;        // of the whole chip; this part has 152 in use
constexpr int MIN_UNITS = 4;        // units a CTA takes at least where items are split
constexpr int WHOLE_UNITS = 8;      // items up to this many units are not split
constexpr int ITEM_UNITS = 2;       // what an item costs besides its units: start and joining

// Probabilities are 2^(s - m + P_SHIFT) for the running reference m, which trails the maximum by
// P_SLACK at most: up to 2^15 as f16, so that the many small weights of a long context keep
// their bits (f16 ends at 2^-24, here 2^-31 of the largest).
constexpr float P_SHIFT = 7.f, P_SLACK = 8.f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 8 x 8 f16 matrix (lane (g, t) holds row g, columns 2t, 2t + 1) transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct Args {
  const bf16* q;
  const int* kv_len;
  bf16* out;
  float* lse;
  int4* split;       // workspace: [CTA] (sequence, item, last CTA, 1) of an item begun and split
  float* part;       // workspace: [CTA][2][ROWS * (D + 2)]
  float scale_log2;
  int q_tokens, q_heads, group, tiles, causal;
};

// Cached length of sequence s, clamped to what the table can name.
__device__ __forceinline__ int length_of(const PageView& c, const Args& a, int s, int* err_flag) {
  const int n = a.kv_len[s], most = c.max_pages << c.page_log2;
  if (n < 0 || n > most) {
    if (err_flag) atomicOr(err_flag, DEV_ERR_INDEX);
    return n < 0 ? 0 : most;
  }
  return n;
}

__device__ __forceinline__ int units_of(int len, int unit) {
  return len > 0 ? (len + unit - 1) / unit : 1;   // an empty sequence has its (zero) rows written
}
// Places of an item in the line: ITEM_UNITS for its start and end, then its units; none where there
// is nothing to read.
__device__ __forceinline__ int places_of(int len, int unit) {
  return len > 0 ? units_of(len, unit) + ITEM_UNITS : 0;
}

// The line: sequence by sequence, each with heads * tiles items of places_of(len) places.
// Totals by one warp (every warp of the CTA computes the same).
__device__ __forceinline__ long long total_places(const PageView& c, const Args& a, int unit,
                                                 int* err_flag) {
  const int lane = threadIdx.x & 31;
  long long n = 0;
  for (int s = lane; s < c.batch; s += 32) n += places_of(length_of(c, a, s, err_flag), unit);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * c.heads * a.tiles;
}

// Position in the line: sequence s whose items begin at place `base`, of `n` places each.
struct Cursor {
  int s, n, len;
  long long base;
};
__device__ __forceinline__ void seek(const PageView& c, const Args& a, int unit, long long u,
                                     Cursor& at) {
  const int lane = threadIdx.x & 31;
  const long long per = (long long)c.heads * a.tiles;
  if (u < at.base + at.n * per) return;          // another item of the same sequence
  long long base = at.base;
  for (int s0 = at.s; s0 < c.batch; s0 += 32) {
    const int s = s0 + lane;
    const int len = s < c.batch ? length_of(c, a, s, nullptr) : 0;
    const int n = s < c.batch ? places_of(len, unit) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, base + incl * per > u);
    if (beyond) {
      const int src = __ffs((int)beyond) - 1;
      at.s = s0 + src;
      at.n = __shfl_sync(0xffffffffu, n, src);
      at.len = __shfl_sync(0xffffffffu, len, src);
      at.base = base + (__shfl_sync(0xffffffffu, incl, src) - at.n) * per;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31) * per;
  }
  at.s = c.batch;
}

// CTAs that take part in a split line: each has MIN_UNITS places at least.
__device__ __forceinline__ int workers_of(long long total, int grid) {
  const long long w = (total + MIN_UNITS - 1) / MIN_UNITS;
  return w < grid ? (int)w : grid;
}

// Zeros for the sequences that are not in the line, those with nothing cached.
template <int D>
__device__ __forceinline__ void write_empty(const PageView& c, const Args& a) {
  const int rows = a.q_tokens * a.q_heads;
  for (int s = blockIdx.x; s < c.batch; s += gridDim.x) {
    if (length_of(c, a, s, nullptr) != 0) continue;
    for (int i = threadIdx.x; i < rows * (D / 8); i += THREADS)
      reinterpret_cast<uint4*>(a.out + (long long)s * rows * D)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = threadIdx.x; i < rows; i += THREADS) a.lse[(long long)s * rows + i] = -INFINITY;
  }
}

// Row r of an item's tile as an index into [batch][q_tokens][q_heads].
__device__ __forceinline__ long long row_at(const Args& a, int s, int head, int r) {
  const int tok = r / a.group;
  return ((long long)s * a.q_tokens + tok) * a.q_heads + head * a.group + (r - tok * a.group);
}

// Units [k0, k1) of n of one item: what a CTA does before it goes on to the next.
struct Segment {
  int s, item, len, n, k0, k1;
  int head, r0;        // of the item: key / value head, first row
  long long next;      // place in the line where the CTA's next segment begins
  long long last;      // the item's last place
};

// a / b for a, b >= 0: a 64-bit division (some hundred instructions) only where it has to be one.
__device__ __forceinline__ long long divided(long long a, int b) {
  return a <= 0xffffffffLL ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int UNIT, int ROWS>
__device__ __forceinline__ bool plan(const PageView& c, const Args& a, int whole, long long u,
                                     long long u_end, Cursor& cur, Segment& g) {
  if (whole) {
    if (u >= u_end) return false;
    const int per = c.heads * a.tiles;
    g.s = (int)divided(u, per);
    g.item = (int)(u - (long long)g.s * per);
    g.len = length_of(c, a, g.s, nullptr);
    g.n = units_of(g.len, UNIT);
    g.k0 = 0;
    g.k1 = g.n;
    g.next = u + 1;
    g.head = a.tiles == 1 ? g.item : g.item / a.tiles;
    g.r0 = (g.item - g.head * a.tiles) * ROWS;
    return true;
  }
  while (u < u_end) {
    seek(c, a, UNIT, u, cur);
    const long long in = u - cur.base;
    const int item = (int)divided(in, cur.n);
    const int at = (int)(in - (long long)item * cur.n);
    const int to = (int)min((long long)cur.n, at + (u_end - u));
    u += to - at;
    if (to <= ITEM_UNITS) continue;              // nothing but the item's start
    g.s = cur.s;
    g.item = item;
    g.len = cur.len;
    g.n = cur.n - ITEM_UNITS;
    g.k0 = max(at - ITEM_UNITS, 0);
    g.k1 = to - ITEM_UNITS;
    g.next = u;
    g.last = cur.base + (item + 1LL) * cur.n - 1;
    g.head = a.tiles == 1 ? item : item / a.tiles;
    g.r0 = (item - g.head * a.tiles) * ROWS;
    return true;
  }
  return false;
}

// Query rows of an item's tile as B fragments: row g of each 8-row tile as f16, times 2^-e so that
// |q| < 2^15. A lane (g = lane / 4, t = lane % 4) holds elements [t D/4, (t+1) D/4) of row g.
template <int D, int NR>
struct Queries {
  uint32_t qf[NR][D / 16][2];
  float qs[NR][2];       // of rows 2t, 2t + 1: 2^e * softmax scale * log2(e)
  int lim[NR][2];        // keys that they see
  int lim_g[NR];         // keys that row g sees
  int lim_min;           // the fewest that any row sees
  __device__ __forceinline__ void load(const Args& a, int s, int head, int r0, int rows, int len) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    lim_min = len;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = r0 + 8 * nr + g;
      const bool valid = r < rows;
      const bf16* src = a.q + row_at(a, s, head, valid ? r : 0) * D + t * (D / 4);
      uint32_t w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = valid ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
      uint32_t top = 0;   // largest |q| as bits (bf16 magnitudes compare as integers)
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent e with |q| 2^-e < 2^15; a row of zeros, infinities or NaN keeps a harmless one
      int e = (int)(top >> 7) - 127 - 14;
      e = max(-126, min(e, 113));
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[nr][i >> 1][i & 1] = pack_f16(__uint_as_float(w[i] << 16) * down,
                                         __uint_as_float(w[i] & 0xffff0000u) * down);
      lim_g[nr] = len;
      if (a.causal && valid) lim_g[nr] = max(0, len - a.q_tokens + r / a.group + 1);
      lim_min = min(lim_min, lim_g[nr]);
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        qs[nr][e2] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + e2));
        lim[nr][e2] = __shfl_sync(0xffffffffu, lim_g[nr], 4 * (2 * t + e2));
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
  }
};

template <int D, int NR>
__device__ __forceinline__ float* part_of(const Args& a, int cta, int which) {
  return a.part + ((long long)cta * 2 + which) * (8 * NR * (D + 2));
}

// fp32 row of a warp's output for the joining
template <int D>
constexpr int OUT_ROW = D + 4;

// Joins the four warps' maxima, sums and outputs of an item's segment, which lie in shared memory
// behind a barrier: whole items to out and lse, others to the workspace.
template <int D, int NR>
__device__ __forceinline__ void join_warps(const Args& a, const Segment& sg, int rows, long long total,
                                           int workers, const float* sm_o,
                                           const float (&sm_m)[WARPS][8 * NR],
                                           const float (&sm_l)[WARPS][8 * NR], int4& begun) {
  constexpr int ROWS = 8 * NR, OUT_LD = OUT_ROW<D>;
  constexpr int TPR = THREADS / ROWS;    // threads a row
  constexpr int CPT = D / TPR;           // columns a thread (4 or more)
  const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * CPT;
  float mx = -INFINITY, sum = 0.f, f[WARPS];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sm_m[w][row]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    f[w] = sm_m[w][row] == -INFINITY ? 0.f : ex2f(sm_m[w][row] - mx);   // its outputs are zeros
    sum = fmaf(sm_l[w][row], f[w], sum);
  }
  float acc[CPT];
#pragma unroll
  for (int i = 0; i < CPT; i += 4) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float4 y =
          *reinterpret_cast<const float4*>(sm_o + (w * ROWS + row) * OUT_LD + c0 + i);
      x.x = fmaf(y.x, f[w], x.x); x.y = fmaf(y.y, f[w], x.y);
      x.z = fmaf(y.z, f[w], x.z); x.w = fmaf(y.w, f[w], x.w);
    }
    acc[i] = x.x; acc[i + 1] = x.y; acc[i + 2] = x.z; acc[i + 3] = x.w;
  }
  const int r = sg.r0 + row;
  if (sg.k0 == 0 && sg.k1 == sg.n) {
    if (r < rows) {
      const long long at = row_at(a, sg.s, sg.head, r);
      const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < CPT; i += 4) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[i + 2] * inv, acc[i + 3] * inv);
        uint2 x;
        x.x = *reinterpret_cast<const uint32_t*>(&lo);
        x.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(a.out + at * D + c0 + i) = x;
      }
      if (a.lse && c0 == 0)
        a.lse[at] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
  } else {
    // part 1 begins in this CTA and goes on in the next; part 0 began in an earlier one
    float* to = part_of<D, NR>(a, blockIdx.x, sg.k0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < CPT; i += 4)
      *reinterpret_cast<float4*>(to + row * D + c0 + i) =
          make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    if (c0 == 0) {
      to[ROWS * D + row] = mx;
      to[ROWS * D + ROWS + row] = sum;
    }
    if (sg.k0 == 0) begun = make_int4(sg.s, sg.item, kv8_worker_of(total, workers, sg.last), 1);
  }
}

// Joins the items that were split: the parts of an item lie with consecutive CTAs, the first of
// which notes them. D / 4 lanes a row; they read all maxima side by side and then the outputs,
// 16 parts in flight: one after the other, 28 parts took 20 us.
template <int D, int NR>
__global__ void __launch_bounds__(128) k_combine(Args a, int max_parts) {
  constexpr int ROWS = 8 * NR, LPR = D / 4, RPB = 128 / LPR, AHEAD = 16;
  extern __shared__ float factors[];                   // [2][RPB][max_parts]: maxima, sums
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts are there
  const int w0 = blockIdx.x;
  const int4 split = a.split[w0];
  if (!split.w) return;
  const int sub = threadIdx.x / LPR, li = threadIdx.x % LPR, row = blockIdx.y * RPB + sub, c0 = li * 4;
  const int s = split.x, head = split.y / a.tiles, r = (split.y % a.tiles) * ROWS + row;
  const int n = split.z - w0 + 1;                      // at most max_parts = CTAs of the call
  float* const f = factors + sub * max_parts;
  // part k: the second of CTA w0, the first of each further one
  auto part = [&](int k) { return part_of<D, NR>(a, w0 + k, k == 0); };
  float mx = -INFINITY, sum = 0.f;
  for (int k = li; k < n; k += LPR) {
    const float* p = part(k) + ROWS * D + row;
    f[k] = p[0];
    f[max_parts * RPB + k] = p[ROWS];
    mx = fmaxf(mx, f[k]);
  }
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  for (int k = li; k < n; k += LPR) {
    const float x = f[k] == -INFINITY ? 0.f : ex2f(f[k] - mx);   // a part that saw no key holds zeros
    f[k] = x;
    sum = fmaf(f[max_parts * RPB + k], x, sum);
  }
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += AHEAD) {
    float4 x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k0 + k < n) x[k] = *reinterpret_cast<const float4*>(part(k0 + k) + row * D + c0);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k0 + k < n) {
        const float y = f[k0 + k];
        acc.x = fmaf(x[k].x, y, acc.x); acc.y = fmaf(x[k].y, y, acc.y);
        acc.z = fmaf(x[k].z, y, acc.z); acc.w = fmaf(x[k].w, y, acc.w);
      }
  }
  if (r >= a.q_tokens * a.group) return;
  const long long at = row_at(a, s, head, r);
  const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 x;
  x.x = *reinterpret_cast<const uint32_t*>(&lo);
  x.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(a.out + at * D + c0) = x;
  if (a.lse && c0 == 0)
    a.lse[at] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
}

// k_combine: a maximum and a sum of each part for its 512 / D rows (heads of 64: 38 KB on 152 SMs),
// bytes a CTA of the call
template <int D>
constexpr int COMBINE_SMEM = 2 * (512 / D) * (int)sizeof(float);

// Set up while the first kernel runs; it waits for that kernel's end before it reads.
template <int D, int NR>
cudaError_t launch_combine(const Args& a, int grid, cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 8 * NR * D / 512);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = COMBINE_SMEM<D> * grid;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_combine<D, NR>, a, grid);
}

// Bytes of the split notes at the head of the workspace.
size_t notes_bytes(int num_sms) { return (size_t)num_sms * MAX_CTAS_PER_SM * sizeof(int4); }

}  // namespace

}  // namespace jepa
