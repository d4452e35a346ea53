// A matrix in 4 bits with a power-of-two scale for each 32 columns: its
// layout from fp32 or bf16 weights, and its product with a few vectors.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "head.h"
#include "head_device.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

constexpr int kThreads = 256;

// 2^(e-127) for a scale byte; 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t e) {
    return e == 255 ? __uint_as_float(0x7FC00000u)
                    : e == 0 ? 0x1p-127f : __uint_as_float(e << 23);
}

// A code's value: sign bit 3, two exponent bits, one mantissa bit.
__device__ __forceinline__ float e2m1(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u;
    const float m = e == 0 ? 0.5f * static_cast<float>(c & 1u)
                           : __uint_as_float(((126u + e) << 23) | ((c & 1u) << 22));
    return (c & 8u) != 0 ? -m : m;
}

// One thread a block of 32.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_w4_quantize(const T* w, int64_t ldw, int64_t rows,
                                                          int64_t cols, uint8_t* packed,
                                                          uint8_t* scales, T* values,
                                                          int64_t ldv) {
    const int64_t kb = (cols + 31) / 32;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= rows * kb) return;
    const int64_t row = i / kb, c0 = (i % kb) * 32;
    const int n = static_cast<int>(cols - c0 < 32 ? cols - c0 : 32);
    uint32_t b = 0;
    for (int j = 0; j < n; ++j) {
        const uint32_t u = abs_bits(to_f32(w[row * ldw + c0 + j]));
        b = u > b ? u : b;
    }
    int e = static_cast<int>((b + 0x3FFFFFu) >> 23) - 2;
    e = e < 0 ? 0 : e;
    if (b >= 0x7F800000u) e = 255;
    scales[i] = static_cast<uint8_t>(e);
    const float back = e == 255 ? 0.0f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    uint32_t byte = 0;
    for (int j = 0; j < 32; ++j) {
        uint32_t code = 0;
        if (j < n && e != 255) {
            const float v = to_f32(w[row * ldw + c0 + j]) * back, m = __builtin_fabsf(v);
            code = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) +
                   (m >= 3.5f) + (m > 5.0f);
            code |= (__float_as_uint(v) >> 31) << 3;
        }
        if (j < n && values != nullptr)
            values[row * ldv + c0 + j] = from_f32<T>(e2m1(code) * scale_of(e));
        byte |= code << (4 * (j & 1));
        if (j & 1) {
            packed[i * 16 + j / 2] = static_cast<uint8_t>(byte);
            byte = 0;
        }
    }
}

__device__ __forceinline__ float e4m3(uint32_t c) {
    const uint32_t e = (c >> 3) & 15u, m = c & 7u;
    float v = e == 0 ? static_cast<float>(m) * 0x1p-9f
                     : __uint_as_float(((e + 120u) << 23) | (m << 20));
    if ((c & 127u) == 127u) v = __uint_as_float(0x7FC00000u);
    return (c & 128u) != 0 ? -v : v;
}

// One wave an element of y.
template <typename Y>
__global__ __launch_bounds__(kThreads) void k_w4_matvec(MatvecArgs a, int x_scale_kind) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / kWave) +
                        threadIdx.x / kWave;
    if (row >= a.rows) return;
    const int v = blockIdx.y;
    const int64_t kb = (a.cols + 31) / 32;
    float t = 0;
    for (int64_t k = threadIdx.x % kWave; k < a.cols; k += kWave) {
        const uint32_t byte = a.packed[row * kb * 16 + k / 2];
        const float w = e2m1((byte >> (4 * (k & 1))) & 15u) * scale_of(a.scales[row * kb + k / 32]);
        float x;
        if (x_scale_kind == DL_SCALE_NONE) {
            x = to_f32(static_cast<const bf16*>(a.x)[v * a.ldx + k]);
        } else {
            x = e4m3(static_cast<const uint8_t*>(a.x)[v * a.ldx + k]);
            if (x_scale_kind == DL_SCALE_BLOCK32)
                x *= scale_of(static_cast<const uint8_t*>(a.x_scales)[v * kb + k / 32]);
        }
        t += w * x;
    }
    t = wave_sum(t);
    if (x_scale_kind == DL_SCALE_ROW) t *= static_cast<const float*>(a.x_scales)[v];
    if (threadIdx.x % kWave == 0) static_cast<Y*>(a.y)[v * a.ldy + row] = from_f32<Y>(t);
}

}  // namespace

hipError_t w4_quantize(const void* w, int64_t ldw, int dtype, int64_t rows, int64_t cols,
                       uint8_t* packed, uint8_t* scales, void* values, int64_t ldvalues,
                       hipStream_t s) {
    const int64_t blocks = rows * ((cols + 31) / 32);
    const dim3 grid(static_cast<unsigned>((blocks + kThreads - 1) / kThreads)), block(kThreads);
    if (dtype == DL_F32)
        k_w4_quantize<<<grid, block, 0, s>>>(static_cast<const float*>(w), ldw, rows, cols, packed,
                                             scales, static_cast<float*>(values), ldvalues);
    else
        k_w4_quantize<<<grid, block, 0, s>>>(static_cast<const bf16*>(w), ldw, rows, cols, packed,
                                             scales, static_cast<bf16*>(values), ldvalues);
    return hipGetLastError();
}

hipError_t w4_matvec(const MatvecArgs& a, int, int x_scale_kind, int y_dtype, hipStream_t s) {
    const int per = kThreads / kWave;
    const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per),
                    static_cast<unsigned>(a.count)),
        block(kThreads);
    if (y_dtype == DL_F32) k_w4_matvec<float><<<grid, block, 0, s>>>(a, x_scale_kind);
    else k_w4_matvec<bf16><<<grid, block, 0, s>>>(a, x_scale_kind);
    return hipGetLastError();
}

}  // namespace dlk
