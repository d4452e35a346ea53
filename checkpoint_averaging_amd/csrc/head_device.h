// Device helpers shared by the output head's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dlk {

constexpr int kWave = 64;

// bfloat16 storage: the high half of a binary32 word.
struct bf16 {
    uint16_t bits;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) {
    return __uint_as_float(static_cast<uint32_t>(v.bits) << 16);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) {
    return bf16{__builtin_bit_cast(uint16_t, static_cast<__bf16>(v))};   // nearest, ties to even
}

// Reductions over a wavefront: every lane gets the result (the same pairing,
// so the same bits, in every lane).
template <typename T> __device__ __forceinline__ T wave_sum(T v) {
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    for (int o = kWave / 2; o > 0; o >>= 1) {
        const uint32_t u = __shfl_xor(v, o);
        v = u > v ? u : v;
    }
    return v;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace dlk
