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
// only: the hardware takes global accesses at any such address.  NT: without
// a stay in the caches.
template <typename T> struct Vec;

template <> struct Vec<float> {
    static constexpr int n = 4;
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    template <bool NT = false> static __device__ __forceinline__ raw load(const float* p) {
        const raw* q = reinterpret_cast<const raw*>(p);
        if constexpr (NT) return __builtin_nontemporal_load(q);
        else return *q;
    }
    template <bool NT = false> static __device__ __forceinline__ void store(float* p, raw v) {
        raw* q = reinterpret_cast<raw*>(p);
        if constexpr (NT) __builtin_nontemporal_store(v, q);
        else *q = v;
    }
    static __device__ __forceinline__ void unpack(const raw& r, float* v) {
        for (int i = 0; i < n; ++i) v[i] = r[i];
    }
    static __device__ __forceinline__ void unpack4(const raw& r, int, float* v) { unpack(r, v); }
    static __device__ __forceinline__ raw pack(const float* v) {
        raw r;
        for (int i = 0; i < n; ++i) r[i] = v[i];
        return r;
    }
};

template <> struct Vec<bf16> {
    static constexpr int n = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    template <bool NT = false> static __device__ __forceinline__ raw load(const bf16* p) {
        const raw* q = reinterpret_cast<const raw*>(p);
        if constexpr (NT) return __builtin_nontemporal_load(q);
        else return *q;
    }
    template <bool NT = false> static __device__ __forceinline__ void store(bf16* p, raw v) {
        raw* q = reinterpret_cast<raw*>(p);
        if constexpr (NT) __builtin_nontemporal_store(v, q);
        else *q = v;
    }
    static __device__ __forceinline__ void unpack(const raw& r, float* v) {
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
    // the four from 4h on
    static __device__ __forceinline__ void unpack4(const raw& r, int h, float* v) {
        const uint32_t a = h == 0 ? r[0] : r[2], b = h == 0 ? r[1] : r[3];
        v[0] = __uint_as_float(a << 16);
        v[1] = __uint_as_float(a & 0xFFFF0000u);
        v[2] = __uint_as_float(b << 16);
        v[3] = __uint_as_float(b & 0xFFFF0000u);
    }
    static __device__ __forceinline__ raw pack(const float* v) {
        raw r;
        for (int i = 0; i < 4; ++i)
            r[i] = from_f32<bf16>(v[2 * i]).bits |
                   (static_cast<uint32_t>(from_f32<bf16>(v[2 * i + 1]).bits) << 16);
        return r;
    }
};

// Eight elements from column c on of a row of n, 0 past the end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t n, float* v) {
    constexpr int NV = Vec<T>::n;
    if (c + 8 <= n) {
        for (int i = 0; i < 8; i += NV) Vec<T>::unpack(Vec<T>::load(row + c + i), v + i);
    } else {
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? to_f32(row[c + i]) : 0.0f;
    }
}
// N elements (1, 2, 4) of a row in one access, at any element.
template <int N, typename T> __device__ __forceinline__ void store_few(T* p, const float* v) {
    T t[N];
    for (int i = 0; i < N; ++i) t[i] = from_f32<T>(v[i]);
    __builtin_memcpy(p, t, sizeof t);
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t n, const float* v) {
    constexpr int NV = Vec<T>::n;
    if (c + 8 <= n) {
        for (int i = 0; i < 8; i += NV) Vec<T>::store(row + c + i, Vec<T>::pack(v + i));
    } else if (c < n) {
        const int left = static_cast<int>(n - c);
        float u[4] = {v[0], v[1], v[2], v[3]};
        T* p = row + c;
        if (left & 4) {
            store_few<4>(p, v);
            p += 4;
            for (int i = 0; i < 4; ++i) u[i] = v[4 + i];
        }
        if (left & 2) {
            store_few<2>(p, u);
            p += 2;
            u[0] = u[2];
        }
        if (left & 1) store_few<1>(p, u);
    }
}

// Eight e4m3 codes, nearest, ties to even.
__device__ __forceinline__ uint2 e4m3_of(const float* v) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
    return uint2{static_cast<uint32_t>(a), static_cast<uint32_t>(b)};
}

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// Eight codes from column c on of a row of n.
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c, int64_t n, uint2 q) {
    if (c + 8 <= n) {
        *reinterpret_cast<u32x2_any*>(row + c) = u32x2_any{q.x, q.y};
    } else if (c < n) {
        const int left = static_cast<int>(n - c);
        uint8_t* p = row + c;
        uint32_t u = q.x;
        if (left & 4) {
            __builtin_memcpy(p, &u, 4);
            p += 4;
            u = q.y;
        }
        if (left & 2) {
            const uint16_t h = static_cast<uint16_t>(u);
            __builtin_memcpy(p, &h, 2);
            p += 2;
            u >>= 16;
        }
        if (left & 1) *p = static_cast<uint8_t>(u);
    }
}

// Reductions over a wavefront; every lane gets the result.  Within rows of 16
// lanes values move by DPP (no LDS), in a fixed pairing that gives every lane
// of a row the same bits; the four rows' are read as scalars.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL> __device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<CTRL>(static_cast<uint32_t>(u));
    const uint64_t hi = dpp<CTRL>(static_cast<uint32_t>(u >> 32));
    return __builtin_bit_cast(double, lo | (hi << 32));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(lane_value(__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = lane_value(static_cast<uint32_t>(u), lane);
    const uint64_t hi = lane_value(static_cast<uint32_t>(u >> 32), lane);
    return __builtin_bit_cast(double, lo | (hi << 32));
}

struct Sum {
    template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return a > b ? a : b;
    }
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// over 2, 4, 8 or 16 neighbouring lanes
template <int N, typename T, typename Op> __device__ __forceinline__ T lanes_reduce(T v, Op op) {
    if constexpr (N >= 2) v = op(v, dpp<0xB1>(v));     // lanes 1 0 3 2
    if constexpr (N >= 4) v = op(v, dpp<0x4E>(v));     // lanes 2 3 0 1
    if constexpr (N >= 8) v = op(v, dpp<0x141>(v));    // halves of a row mirrored
    if constexpr (N >= 16) v = op(v, dpp<0x140>(v));   // rows mirrored
    return v;
}
template <typename T, typename Op> __device__ __forceinline__ T wave_reduce(T v, Op op) {
    v = lanes_reduce<16>(v, op);
    return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}
template <typename T> __device__ __forceinline__ T wave_sum(T v) { return wave_reduce(v, Sum{}); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace dlk
