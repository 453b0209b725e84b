// Residual addition, RMS norm and 8-bit codes in one pass over a row:
//
//   s = x + delta,  y = s w / sqrt(mean(s^2) + eps),  scale = max|y| / 448,  code = e4m3(y 448 / max|y|)
//
// with s to x_out, codes and scales as the fp8 linear layers take them and, where asked for, y as
// bf16. Bound by the bytes of x, delta and the outputs, each touched once: a row stays in registers
// between its sum of squares, its maximum and its codes. Measured: 6192 rows of 1024 in fp32 13.7 us (6 TB/s,
// 0.90 of the copy rate), 4099 of 8192 in bf16 with a bf16 output 57 us (5.3 TB/s), one row 4 us.
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

template <bool HALF>
__device__ __forceinline__ void load8(const void* base, long long at, float (&v)[8]) {
  if (HALF) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(base) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
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

// Sum of `v` and maximum of `m` over the T threads of a row. `sm`: two floats a warp of the row.
template <int T>
__device__ __forceinline__ void over_row(float& v, float& m, float2* sm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (T == 32) return;
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x % T >> 5] = make_float2(v, m);
  __syncthreads();
  v = m = 0.f;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    const float2 x = sm[i];
    v += x.x;
    m = fmaxf(m, x.y);
  }
}

constexpr float MOST = 0x1p126f;         // the largest factor of the codes

// T threads a row, V vectors of 8 elements a thread, R rows a CTA.
template <int T, int V, int R, bool XH, bool DH>
__global__ void __launch_bounds__(T * R) k_add_rmsnorm(Args a) {
  __shared__ float2 sm[T * R / 32];
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
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j & 3] = fmaf(s[k][j], s[k][j], part[j & 3]);
  }
  // z = s w takes s's place; its maximum goes through the CTA together with the sum
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (i >= vecs) continue;
    float w[8];
    load8<false>(a.w, 8 * i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[k][j] *= w[j];
      m = fmaxf(m, fabsf(s[k][j]));      // drops NaN
    }
  }
  float sum = (part[0] + part[1]) + (part[2] + part[3]);
  over_row<T>(sum, m, sm + threadIdx.x / T * (T / 32));
  if (!on) return;
  const float r = 1.f / sqrtf(sum / (float)a.cols + a.eps);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = tid + k * T;
    if (a.y && i < vecs) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = s[k][j] * r;
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
    if (i < vecs) *reinterpret_cast<uint2*>(a.codes + row * a.cols + 8 * i) = e4m3x8(s[k], f);
  }
}

template <int T, int V, int R>
cudaError_t launch(const Args& a, int x_bf16, int delta_bf16, cudaStream_t s) {
  auto* kernel = x_bf16 ? (delta_bf16 ? k_add_rmsnorm<T, V, R, true, true> : k_add_rmsnorm<T, V, R, true, false>)
                        : (delta_bf16 ? k_add_rmsnorm<T, V, R, false, true> : k_add_rmsnorm<T, V, R, false, false>);
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

}  // namespace

cudaError_t add_rmsnorm(const void* x, int x_bf16, long long x_stride, const void* delta,
                        int delta_bf16, long long delta_stride, const float* w, float eps, int rows,
                        int cols, void* x_out, long long out_stride, uint8_t* codes, float* scales,
                        bf16* y, cudaStream_t s) {
  const Args a{x, delta, x_stride, delta_stride, out_stride, w, eps, rows, cols, x_out, codes, scales, y};
  // One vector a thread while that leaves few warps a row: more of a SM's rows in flight, and a short
  // chain for a single one. Wider rows take more, as their barriers cost more than the registers. Measured, us:
  // 6192 x 1024 fp32: 128 threads 16.4, 64 with two vectors 18.1, a warp with four 18.5; 1000 x 4096
  // bf16: 256 with two 10.2, 128 with four 11.0; 4099 x 8192 bf16: 256 with four 55, 512 with two 58, 1024 68;
  // 1000 x 16384: 1024 with two 37, 512 with four 41.
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
