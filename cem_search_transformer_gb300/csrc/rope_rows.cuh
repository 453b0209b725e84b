// Rows of packed tokens: which sequence a token belongs to, and how the lanes of a warp hold a head row
// between norm, rotation and quantisation. Shared by the appends of the 8-bit and the 4-bit cache.
//
// A head row is held by D / 16 lanes, 16 elements each: both elements of every rotated pair lie in
// one lane (no exchange), and its 8 angles serve 16 elements.
#pragma once

#include "kv8.cuh"

namespace jepa {

namespace {

constexpr int THREADS = 256;

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

// Sequence of a packed token and where it lies.
struct Place {
  int s, begin, end, first;   // sequence (-1: none), its packed tokens [begin, end), start[s]
};
// The largest s with cu[s] <= t (cu ascending), by the whole warp: 32-way probes, the last of
// which brings the bounds and the start along.
// Offsets and starts are read by plain loads: the kernel stands by while the one before it may still write them.
__device__ __forceinline__ Place locate(const int* cu, const int* start, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 32) {
    const int step = (n + 31) >> 5, at = lane * step;
    const bool le = at < n && cu[lo + at] <= t;
    const int last = 31 - __clz((int)(__ballot_sync(0xffffffffu, le) | 1u));
    lo += last * step;
    n = min(step, n - last * step);
  }
  int b = 0x7fffffff, e = 0, f = 0;
  if (lane < n) {
    b = cu[lo + lane];
    e = cu[lo + lane + 1];
    f = start[lo + lane];
  }
  const uint32_t le = __ballot_sync(0xffffffffu, b <= t);
  const int last = le ? 31 - __clz((int)le) : 0;
  Place p;
  p.s = le ? lo + last : -1;
  p.begin = __shfl_sync(0xffffffffu, b, last);
  p.end = __shfl_sync(0xffffffffu, e, last);
  p.first = __shfl_sync(0xffffffffu, f, last);
  return p;
}

// Whether packed token t belongs to the sequence that locate found. Not where it lies ahead of the
// first sequence or behind the last, nor in one whose offsets leave the rows: that one is skipped.
__device__ __forceinline__ bool holds(const Place& p, int t, int tokens) {
  return p.s >= 0 && t < p.end && kv8_span_ok(p.begin, p.end, tokens);
}

// Reports the sequences that are skipped, empty ones too, each by one thread of the grid (which has a
// thread for each). Stands at a kernel's end, where the offsets are in the cache.
__device__ __forceinline__ void report_offsets(const int* cu, int batch, int tokens,
                                               int* err_flag) {
  const long long s = (long long)blockIdx.x * THREADS + threadIdx.x;
  if (s < batch && !kv8_span_ok(cu[s], cu[s + 1], tokens)) atomicOr(err_flag, DEV_ERR_INDEX);
}
// Blocks for `threads` of work and at least one thread a sequence.
long long blocks_for(long long threads, int batch) {
  return ((threads > batch ? threads : batch) + THREADS - 1) / THREADS;
}

// The 16 elements of a head row that a lane holds: chunks of 8 at c0 and c1.
template <int D, bool INTER>
struct Lane {
  int c0, c1, p;
  bool rotates;
  __device__ __forceinline__ explicit Lane(int rot) {
    constexpr int L = D / 16;
    p = (threadIdx.x & 31) % L;
    rotates = 16 * p < rot;
    if (INTER || !rotates) {
      // neighbours; past rot these are the chunks rot / 8 + 2 (p - rot / 16) and the next
      c0 = 2 * p;
      c1 = 2 * p + 1;
    } else {
      c0 = p;
      c1 = p + (rot >> 4);
    }
  }
};

// cos (first 8) and sin of a lane's pairs 8 p .. 8 p + 7 from a row of the table.
__device__ __forceinline__ void load_angles(float (&an)[16], const float* row, int rot, int p) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 x = load_late(reinterpret_cast<const float4*>(row + h * (rot >> 1) + 8 * p + i));
      an[8 * h + i] = x.x; an[8 * h + i + 1] = x.y; an[8 * h + i + 2] = x.z; an[8 * h + i + 3] = x.w;
    }
}

template <class LaneT>
__device__ __forceinline__ void load16(const bf16* row, const LaneT& ln, uint4 (&u)[2]) {
  u[0] = *reinterpret_cast<const uint4*>(row + 8 * ln.c0);
  u[1] = *reinterpret_cast<const uint4*>(row + 8 * ln.c1);
}
__device__ __forceinline__ void widen(const uint4 (&u)[2], float (&y)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
      y[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <class LaneT>
__device__ __forceinline__ void store16(bf16* row, const LaneT& ln, const float (&y)[16]) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = y[i];
    b[i] = y[8 + i];
  }
  store8(row + 8 * ln.c0, a);
  store8(row + 8 * ln.c1, b);
}
__device__ __forceinline__ int positions_of(const PageView& c, const AppendArgs& a) {
  return min(a.positions, c.max_pages << c.page_log2);
}

// Place of packed token t of the sequence `at` in the cache, and its row of the rotary table (the same number
// but where APART). False where either is out of range.
template <bool APART>
__device__ __forceinline__ bool place_of(const PageView& c, const AppendArgs& a, const Place& at, int t, int& pos,
                                         int& row) {
  pos = (int)((unsigned)at.first + (unsigned)(t - at.begin));
  row = pos;
  if (!APART || !a.rope_start) return at.first >= 0 && pos >= 0 && pos < positions_of(c, a);
  const int from = a.rope_start[at.s];
  row = (int)((unsigned)from + (unsigned)(t - at.begin));
  return at.first >= 0 && pos >= 0 && pos < (c.max_pages << c.page_log2) && from >= 0 && row >= 0 && row < a.positions;
}

// Launch that, with `early`, begins while the kernel before it in the stream still runs: what may
// not overlap stands behind a griddepcontrol.wait, which lasts until that kernel's end.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned blocks, bool early, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = early;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// y = x * w / sqrt(mean(x^2) + eps), then (a, b) -> (a cos - b sin, b cos + a sin) for the pairs
// (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1), i < rot / 2. All lanes of the warp call it. Products are
// fused and sums plain fp32: what goes to bf16 or to 8 bits behind it can differ by a step from another order's where
// a rotation nearly cancels or a value lies next to a border (4-bit keys, whose steps are wide, are taken exactly).
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(float (&y)[16], const Lane<D, INTER>& ln,
                                            const float* __restrict__ w, float eps,
                                            const float (&an)[16]) {
  constexpr int L = D / 16;
  if (w) {
    float part[4] = {0.f, 0.f, 0.f, 0.f};   // short chains: fewer roundings on the way
#pragma unroll
    for (int i = 0; i < 16; ++i) part[i & 3] = fmaf(y[i], y[i], part[i & 3]);
    float ss = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // Heads whose squares leave fp32, or vanish where no epsilon holds their mean up, come to where they do not by a power of
    // two, and the epsilon by its square. Nine prompts: 1 us of 114 for the look.
    const bool far = !(ss < 0x1p120f && ss >= (eps < 0x1p-106f ? 0x1p-96f : 0.f));
    if (__any_sync(0xffffffffu, far)) {
      float top = 0.f;                    // drops NaN, which reach the sum all the same
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
#pragma unroll
      for (int o = L / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float f = 1.f;
      if (far && top >= 0x1p50f && top < INFINITY) f = pow2(50 - (int)(__float_as_uint(top) >> 23) + 127);
      if (far && top < 0x1p-40f) f = 0x1p75f;
      eps = eps * f * f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        y[i] *= f;
        sum = fmaf(y[i], y[i], sum);
      }
#pragma unroll
      for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (far) ss = sum;
    }
    const float r = __frsqrt_rn(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 g =
          load_late(reinterpret_cast<const float4*>(w + 8 * (i < 8 ? ln.c0 : ln.c1) + (i & 7)));
      y[i] *= r * g.x; y[i + 1] *= r * g.y; y[i + 2] *= r * g.z; y[i + 3] *= r * g.w;
    }
  }
  if (ln.rotates) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 8 + i;
      const float p = y[ia], q = y[ib];
      y[ia] = p * an[i] - q * an[8 + i];
      y[ib] = q * an[i] + p * an[8 + i];
    }
  }
}

// Queries: a warp takes one token and up to Q_HEADS of its heads, which share the angles. The
// loads of the rows and of the token's sequence go out together.
constexpr int Q_HEADS = 8;

template <int D, bool INTER, bool APART = false>
__device__ __forceinline__ void rotate_queries(const PageView& c, const AppendArgs& a,
                                               long long unit, int* err_flag) {
  constexpr int L = D / 16, ROWS = 32 / L, PASSES = Q_HEADS / ROWS;
  const int blocks = (a.q_heads + Q_HEADS - 1) / Q_HEADS;
  if (unit >= (long long)a.tokens * blocks) return;
  const int t = (int)(unit / blocks), h0 = (int)(unit - (long long)t * blocks) * Q_HEADS;
  const int sub = (threadIdx.x & 31) / L;
  const Lane<D, INTER> ln(a.rot);
  uint4 raw[PASSES][2];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int h = h0 + p * ROWS + sub;
    raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    if (h < a.q_heads) load16(a.q + t * a.q_stride + (long long)h * D, ln, raw[p]);
  }
  const Place at = locate(a.cu, a.start, c.batch, t);
  if (!holds(at, t, a.tokens)) return;            // left as it is
  int pos, row;
  if (!place_of<APART>(c, a, at, t, pos, row)) {
    if ((threadIdx.x & 31) == 0) atomicOr(err_flag, DEV_ERR_INDEX);
    return;
  }
  float an[16];
  if (ln.rotates) load_angles(an, a.rope + (long long)row * a.rot, a.rot, ln.p);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    float y[16];
    widen(raw[p], y);
    norm_rotate<D, INTER>(y, ln, a.q_norm, a.eps, an);
    const int h = h0 + p * ROWS + sub;
    if (h < a.q_heads) store16(a.q_out + ((long long)t * a.q_heads + h) * D, ln, y);
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(THREADS, 4) k_rope_queries(PageView c, AppendArgs a, int* err_flag) {
  asm volatile("griddepcontrol.launch_dependents;");
  rotate_queries<D, INTER>(c, a, (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5), err_flag);
}

}  // namespace

}  // namespace jepa
