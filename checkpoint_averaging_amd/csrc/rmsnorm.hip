// Root-mean-square norm with the residual's addition, and its gradients.
//
//   s = x + residual ; inv = 1/sqrt(mean s^2 + eps) ; y = (s inv) w
//   g = dy w ; h = s inv ; dx = inv (g - h mean(g h)) + dsum ; dw = sum dy h
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "head.h"
#include "head_device.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int64_t kMaxGrid = 1 << 20;

template <typename T> __device__ __forceinline__ T block_sum(T v, T* lds) {
    v = wave_sum(v);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    T t = lds[0];
    for (int i = 1; i < kWaves; ++i) t += lds[i];
    __syncthreads();
    return t;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* lds) {
    v = wave_max(v);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    uint32_t t = lds[0];
    for (int i = 1; i < kWaves; ++i) t = lds[i] > t ? lds[i] : t;
    __syncthreads();
    return t;
}

__device__ __forceinline__ uint8_t e4m3_of(float v) {
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false) & 0xFF);
}

template <typename T>
__device__ __forceinline__ float stream_value(const NormArgs& a, int64_t row, int c) {
    const float x = to_f32(static_cast<const T*>(a.x)[row * a.ldx + c]);
    if (a.residual == nullptr) return x;
    return to_f32(from_f32<T>(x + to_f32(static_cast<const T*>(a.residual)[row * a.ldres + c])));
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_rmsnorm(NormArgs a, int y_dtype, int scale_kind) {
    __shared__ double lds_d[kWaves];
    __shared__ uint32_t lds_u[kWaves];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    double ss = 0;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const double s = stream_value<T>(a, row, c);
        ss += s * s;
    }
    ss = block_sum(ss, lds_d);
    const float inv =
        static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
    if (threadIdx.x == 0 && a.inv_rms != nullptr) a.inv_rms[row] = inv;

    uint32_t amax = 0;
    float back = 0.0f;
    if (scale_kind == DL_SCALE_ROW) {
        for (int c = threadIdx.x; c < a.cols; c += kThreads) {
            const uint32_t b = abs_bits((stream_value<T>(a, row, c) * inv) * a.weight[c]);
            amax = b > amax ? b : amax;
        }
        amax = block_max(amax, lds_u);
        const float m = __uint_as_float(amax);
        float scale = 0.0f;
        if (amax >= 0x7F800000u) {
            scale = __uint_as_float(0x7FC00000u);
        } else if (m >= 0x1p-100f) {
            scale = m / 448.0f;
            back = 448.0f / m;
        }
        if (threadIdx.x == 0) static_cast<float*>(a.scales)[row] = scale;
    }
    const int padded = (a.cols + 31) / 32 * 32;
    for (int c = threadIdx.x; c < padded; c += kThreads) {
        const bool in = c < a.cols;
        const float s = in ? stream_value<T>(a, row, c) : 0.0f;
        const float y = in ? (s * inv) * a.weight[c] : 0.0f;
        if (scale_kind == DL_SCALE_BLOCK32) {
            uint32_t b = abs_bits(y);
            for (int o = 16; o > 0; o >>= 1) {
                const uint32_t u = __shfl_xor(b, o, 32);
                b = u > b ? u : b;
            }
            int e = static_cast<int>((b + 0x1FFFFFu) >> 23) - 8;
            e = e < 0 ? 0 : e;
            if (b >= 0x7F800000u) e = 255;
            back = e == 255 ? 0.0f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
            if (c % 32 == 0)
                static_cast<uint8_t*>(a.scales)[row * (padded / 32) + c / 32] =
                    static_cast<uint8_t>(e);
        }
        if (!in) continue;
        if (a.sum != nullptr) static_cast<T*>(a.sum)[row * a.ldsum + c] = from_f32<T>(s);
        const int64_t at = row * a.ldy + c;
        if (y_dtype == DL_F32) static_cast<float*>(a.y)[at] = y;
        else if (y_dtype == DL_BF16) static_cast<bf16*>(a.y)[at] = from_f32<bf16>(y);
        else static_cast<uint8_t*>(a.y)[at] = back == 0.0f ? 0 : e4m3_of(y * back);
    }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_rmsnorm_dx(NormBackwardArgs a) {
    __shared__ float lds[kWaves];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float inv = a.inv_rms[row];
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* sum = static_cast<const T*>(a.sum) + row * a.ldsum;
    float c0 = 0;
    for (int c = threadIdx.x; c < a.cols; c += kThreads)
        c0 += to_f32(dy[c]) * a.weight[c] * (to_f32(sum[c]) * inv);
    c0 = block_sum(c0, lds) / static_cast<float>(a.cols);
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const float g = to_f32(dy[c]) * a.weight[c], h = to_f32(sum[c]) * inv;
        float d = inv * (g - h * c0);
        if (a.dsum != nullptr) d += to_f32(static_cast<const T*>(a.dsum)[row * a.lddsum + c]);
        static_cast<T*>(a.dx)[row * a.lddx + c] = from_f32<T>(d);
    }
    }
}

// One column a thread, rows in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_rmsnorm_dw(NormBackwardArgs a) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.cols) return;
    float t = 0;
    for (int64_t row = 0; row < a.rows; ++row)
        t += to_f32(static_cast<const T*>(a.dy)[row * a.lddy + c]) *
             (to_f32(static_cast<const T*>(a.sum)[row * a.ldsum + c]) * a.inv_rms[row]);
    a.dweight[c] = t;
}

}  // namespace

hipError_t rmsnorm(const NormArgs& a, int dtype, int y_dtype, int scale_kind, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid)), block(kThreads);
    if (dtype == DL_F32) k_rmsnorm<float><<<grid, block, 0, s>>>(a, y_dtype, scale_kind);
    else k_rmsnorm<bf16><<<grid, block, 0, s>>>(a, y_dtype, scale_kind);
    return hipGetLastError();
}

int64_t rmsnorm_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t rmsnorm_backward(const NormBackwardArgs& a, int dtype, hipStream_t s) {
    const dim3 block(kThreads);
    if (a.dweight != nullptr) {     // before dx, which may be dy itself
        const dim3 grid((a.cols + kThreads - 1) / kThreads);
        if (dtype == DL_F32) k_rmsnorm_dw<float><<<grid, block, 0, s>>>(a);
        else k_rmsnorm_dw<bf16><<<grid, block, 0, s>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.rows == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid));
    if (dtype == DL_F32) k_rmsnorm_dx<float><<<grid, block, 0, s>>>(a);
    else k_rmsnorm_dx<bf16><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dlk
