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

// kVec elements of one row in one 128-bit access.  Rows start at any element
// (odd leading dimensions), so the access is declared aligned to an element
// only: the hardware takes global accesses at any such address.
template <typename T> struct Vec;

template <> struct Vec<float> {
    static constexpr int n = 4;
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    static __device__ __forceinline__ void unpack(const raw& r, float* v) {
        for (int i = 0; i < n; ++i) v[i] = r[i];
    }
    static __device__ __forceinline__ raw pack(const float* v) {
        raw r;
        for (int i = 0; i < n; ++i) r[i] = v[i];
        return r;
    }
};

template <> struct Vec<bf16> {
    static constexpr int n = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    static __device__ __forceinline__ void unpack(const raw& r, float* v) {
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ raw pack(const float* v) {
        raw r;
        for (int i = 0; i < 4; ++i)
            r[i] = from_f32<bf16>(v[2 * i]).bits |
                   (static_cast<uint32_t>(from_f32<bf16>(v[2 * i + 1]).bits) << 16);
        return r;
    }
};

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
