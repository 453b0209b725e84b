// Residual addition, RMS norm and 8-bit codes in one pass over a row:
//
//   s = x + delta,  y = s w / sqrt(mean(s^2) + eps),  scale = max|y| / 448,  code = e4m3(y 448 / max|y|)
//
// with s to x_out, codes and scales as the fp8 linear layers take them and, where asked for, y as
// bf16. Bound by the bytes of x, delta and the outputs, each touched once: a row stays in registers
// between its sum of squares, its maximum and its codes. Measured: 6192 rows of 1024 in fp32 14.0 us (5.9 TB/s,
// 0.88 of the copy rate), 4099 of 8192 in bf16 with a bf16 output 55 us (5.5 TB/s), one row 2 us (4 by itself).
#include "add_rmsnorm.cuh"

namespace jepa {

namespace {

struct Args {
  const void *x, *delta;
  long long x_stride, delta_stride, out_stride;
  const float* w;
  float eps;
  int rows, cols;
  void* x_out;
  uint8_t* codes;
  float* scales;
  bf16* y;
};

// Weights, whose lines the CTAs of an SM share: as read-only data they stay in its L1 (6192 rows of 1024 14.1 us, by
// ordinary loads 15.5). Volatile, as the griddepcontrol.wait is, so that they stay behind it: the kernel before may be
// the one that wrote them.
__device__ __forceinline__ float4 load_weights(const float4* p) {
  float4 x;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
  return x;
}
// Rows by plain loads: x is written where the sum goes back in place, and __ldg is for what no one writes.
template <bool HALF>
__device__ __forceinline__ void load8(const void* base, long long at, float (&v)[8]) {
  if (HALF) {
    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool HALF>
__device__ __forceinline__ void store8(void* base, long long at, const float (&v)[8]) {
  if (HALF) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float f) {
  uint16_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p[i]) : "f"(v[2 * i + 1] * f), "f"(v[2 * i] * f));
  return make_uint2((uint32_t)p[0] | ((uint32_t)p[1] << 16), (uint32_t)p[2] | ((uint32_t)p[3] << 16));
}

// Elements whose squares leave fp32: a warp that holds some has its elements times 2^-75, its sum of squares by the
// square of that. `far`: this warp's are so. Rows of which one warp is far become so as a whole.
constexpr float DOWN = 0x1p-75f;

// Sum of `v` and maximum of `m` over the T threads of a row. `sm`: two floats a warp of the row, and one more.
// Returns whether the row is far: sum and maximum are then those of elements times 2^-75.
template <int T>
__device__ __forceinline__ bool over_row(float& v, float& m, bool far, float2* sm, float* sm_far) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (T == 32) return far;
  if ((threadIdx.x & 31) == 0) {
    sm[threadIdx.x % T >> 5] = make_float2(far ? INFINITY : v, m);
    if (far) sm_far[threadIdx.x % T >> 5] = v;
  }
  __syncthreads();
  v = m = 0.f;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    const float2 x = sm[i];
    v += x.x;
    m = fmaxf(m, x.y);
  }
  if (v < INFINITY) return false;
  v = m = 0.f;
#pragma unroll 1
  for (int i = 0; i < T / 32; ++i) {
    const float2 x = sm[i];
    const bool near = x.x < INFINITY;
    v += near ? x.x * DOWN * DOWN : sm_far[i];
    m = fmaxf(m, near ? x.y * DOWN : x.y);
  }
  return true;
}

// Largest of `top` over the T threads of a row. `sm`: a float a warp of the row.
template <int T>
__device__ __forceinline__ float top_of_row(float top, float* sm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (T == 32) return top;
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x % T >> 5] = top;
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < T / 32; ++i) top = fmaxf(top, sm[i]);
  return top;
}

constexpr float MOST = 0x1p126f;         // the largest factor of the codes

// T threads a row, V vectors of 8 elements a thread, R rows a CTA. BARE: an epsilon that does not hold up the mean of
// squares that vanish (one kernel with a branch for both: 6192 rows of 1024 15.4 us instead of 14.0).
template <int T, int V, int R, bool XH, bool DH, bool BARE>
__global__ void __launch_bounds__(T * R) k_add_rmsnorm(Args a) {
  __shared__ float2 sm[T * R / 32];
  __shared__ float sm_far[T * R / 32], sm_top[T * R / 32];
  static_assert(T == 32 || T * R <= 1024, "rows of several warps meet at the CTA's barrier");
  const long long row = (long long)blockIdx.x * R + threadIdx.x / T;
  const int tid = threadIdx.x % T, vecs = a.cols >> 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernel before writes is there
  if (T == 32 && row >= a.rows) return;
  const bool on = row < a.rows;            // rows of several warps meet at the barrier all the same
  float s[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[k][j] = 0.f;
    if (on && i < vecs) load8<XH>(a.x, row * a.x_stride + 8 * i, s[k]);
  }
  if (a.delta) {
    float d[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = tid + k * T;
      if (on && i < vecs) load8<DH>(a.delta, row * a.delta_stride + 8 * i, d[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (on && tid + k * T < vecs)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[k][j] += d[k][j];
  }
  float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (on && a.x_out && i < vecs) store8<XH>(a.x_out, row * a.out_stride + 8 * i, s[k]);
    if (!BARE)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[j & 3] = fmaf(s[k][j], s[k][j], part[j & 3]);
  }
  float eps = a.eps;
  const int warp0 = threadIdx.x / T * (T / 32);        // of the row
  if (BARE) {
    // rows of small elements come near 1, by a power of two
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(s[k][j]));
    top = top_of_row<T>(top, sm_top + warp0);
    if (top < 0x1p-40f) {
      // the larger of the row and the epsilon's root
      const int e = max((int)(__float_as_uint(top) >> 23), (int)(__float_as_uint(eps) >> 24) + 64) - 127;
      const float f = __uint_as_float((uint32_t)(127 - max(e, -120)) << 23);
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[k][j] *= f;
      eps = eps * f * f;
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[j & 3] = fmaf(s[k][j], s[k][j], part[j & 3]);
  }
  float sum = (part[0] + part[1]) + (part[2] + part[3]);
  // 1024 threads' sums below 2^110 stay in fp32; NaN and infinities count as far
  const bool far = __any_sync(0xffffffffu, !(sum < 0x1p110f));
  if (far) {
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[k][j] *= DOWN;
        sum = fmaf(s[k][j], s[k][j], sum);
      }
  }
  // z = s w takes s's place; its maximum goes through the CTA together with the sum
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (i >= vecs) continue;
    const float4* wp = reinterpret_cast<const float4*>(a.w + 8 * i);
    const float4 w0 = load_weights(wp), w1 = load_weights(wp + 1);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[k][j] *= w[j];
      m = fmaxf(m, fabsf(s[k][j]));      // drops NaN
    }
  }
  const bool far_row = over_row<T>(sum, m, far, sm + warp0, sm_far + warp0);
  if (!on) return;
  if (far_row) eps = eps * DOWN * DOWN;
  // brings this warp's elements to where the row's are; taken into the factors (the elements themselves: 4 us of 55 for
  // 4099 rows of 8192)
  const float g = far_row && !far ? DOWN : 1.f;
  const float r = 1.f / sqrtf(sum / (float)a.cols + eps);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (a.y && i < vecs) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = s[k][j] * (r * g);
      store8<true>(a.y, row * a.cols + 8 * i, y);
    }
  }
  if (!a.codes) return;
  // y 448 / max|y| = z 448 / max|z|: the codes carry three roundings, and none of r's. Where the row
  // has no maximum to go by (zeros, infinities, NaN) the codes are those of y itself, zero or NaN.
  const bool some = r * m > 0.f && m < INFINITY;
  const float f = some ? fminf(448.f / m, MOST) : r * 0.f;
  if (tid == 0) a.scales[row] = !some ? 1.f : f < MOST ? r * m / 448.f : r / f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (i < vecs) *reinterpret_cast<uint2*>(a.codes + row * a.cols + 8 * i) = e4m3x8(s[k], f * g);
  }
}

template <int T, int V, int R, bool BARE>
cudaError_t start(const Args& a, int x_bf16, int delta_bf16, cudaStream_t s) {
  auto* kernel = x_bf16 ? (delta_bf16 ? k_add_rmsnorm<T, V, R, true, true, BARE> : k_add_rmsnorm<T, V, R, true, false, BARE>)
                        : (delta_bf16 ? k_add_rmsnorm<T, V, R, false, true, BARE> : k_add_rmsnorm<T, V, R, false, false, BARE>);
  cudaLaunchAttribute attr;                // begins while the kernel before it ends
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.rows + R - 1) / R));
  cfg.blockDim = dim3(T * R);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <int T, int V, int R>
cudaError_t launch(const Args& a, int x_bf16, int delta_bf16, cudaStream_t s) {
  return a.eps < 0x1p-106f ? start<T, V, R, true>(a, x_bf16, delta_bf16, s)
                           : start<T, V, R, false>(a, x_bf16, delta_bf16, s);
}

}  // namespace

cudaError_t add_rmsnorm(const void* x, int x_bf16, long long x_stride, const void* delta,
                        int delta_bf16, long long delta_stride, const float* w, float eps, int rows,
                        int cols, void* x_out, long long out_stride, uint8_t* codes, float* scales,
                        bf16* y, cudaStream_t s) {
  const Args a{x, delta, x_stride, delta_stride, out_stride, w, eps, rows, cols, x_out, codes, scales, y};
  // One vector a thread while that leaves few warps a row: more of a SM's rows in flight, and a short
  // chain for a single one. Wider rows take more, as their barriers cost more than the registers. Measured in this
  // form, us: 6192 x 1024 fp32: 128 threads 14.0, 64 with two vectors 16.0, a warp with four 16.3; 1000 x 4096
  // bf16: 256 with two 8.6, 128 with four 9.6; 4099 x 8192 bf16 and bf16 rows: 256 with four 55, 512 with two 57,
  // 1024 69; 1000 x 16384 bf16: 1024 with two 32.0, 512 with four 32.8.
  if (cols <= 256) return launch<32, 1, 8>(a, x_bf16, delta_bf16, s);
  if (cols <= 512) return launch<64, 1, 2>(a, x_bf16, delta_bf16, s);
  if (cols <= 1024) return launch<128, 1, 1>(a, x_bf16, delta_bf16, s);
  if (cols <= 4096) return launch<256, 2, 1>(a, x_bf16, delta_bf16, s);
  if (cols <= 8192) return launch<256, 4, 1>(a, x_bf16, delta_bf16, s);
  if (cols <= 16384) return launch<1024, 2, 1>(a, x_bf16, delta_bf16, s);
  if (cols <= ADD_RMSNORM_MAX_COLS) return launch<1024, 4, 1>(a, x_bf16, delta_bf16, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
