// Residual addition, RMS norm and 8-bit codes (add_rmsnorm.cu).
#pragma once

#include "common.cuh"

namespace jepa {

constexpr int ADD_RMSNORM_MAX_COLS = 32768;   // a row stays in the registers of one CTA

cudaError_t add_rmsnorm(const void* x, int x_bf16, long long x_stride, const void* delta,
                        int delta_bf16, long long delta_stride, const float* w, float eps, int rows,
                        int cols, void* x_out, long long out_stride, uint8_t* codes, float* scales,
                        bf16* y, cudaStream_t s);

}  // namespace jepa
