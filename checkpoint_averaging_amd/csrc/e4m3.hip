// Matrices in 8 bits (e4m3) with a power-of-two scale for each 128 x 128
// elements or each 128 of a row: their layout, and the product of the two.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "head.h"
#include "head_device.h"
#include "tiles.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

// ---- the layout --------------------------------------------------------------

constexpr int kBlock = 128;
constexpr int kThreads = 256;

// The exponent byte of the smallest power of two b with amax <= 448 b = 1.75 * 2^8 b; 255
// for a NaN or infinity.
__device__ __forceinline__ uint32_t byte_of(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255;
    const int e = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
    return static_cast<uint32_t>(e < 0 ? 0 : e);
}

// Eight codes of v / 2^(e-127), and v replaced by what they stand for.
__device__ __forceinline__ uint2 encode(float* v, uint32_t e) {
    const float back = __uint_as_float((254 - e) << 23);
    uint2 q{0, 0};
    if (e != 255) {
        for (int k = 0; k < 8; ++k) v[k] *= back;
        q = e4m3_of(v);
    }
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    // (the conversion takes the scale's exponent bits: all zeros is 2^-127, all ones NaN)
    const float s = __uint_as_float(e << 23);
    const f32x2 o[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, s, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, s, true),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, s, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, s, true)};
    for (int k = 0; k < 8; ++k) v[k] = o[k / 2][k % 2];
    return q;
}

struct QuantizeArgs {
    const void* x;
    int64_t ldx, rows, cols;
    uint8_t* codes;
    int64_t ldc;
    uint8_t* scales;
    void* values;                         // or nullptr
    int64_t ldv;
};

template <typename T>
__device__ __forceinline__ void emit(const QuantizeArgs& a, int64_t row, int64_t c, float* v,
                                     uint32_t e) {
    const uint2 q = encode(v, e);
    store_codes(a.codes + row * a.ldc, c, a.cols, q);
    if (a.values != nullptr) store8(static_cast<T*>(a.values) + row * a.ldv, c, a.cols, v);
}

// One scale for 128 columns of a row: eight columns a lane, 16 lanes a block.
template <typename T> __global__ __launch_bounds__(kThreads) void k_e4m3_blocks(QuantizeArgs a) {
    const int64_t kb = (a.cols + kBlock - 1) / kBlock, all = a.rows * kb;
    const int lane = threadIdx.x % 16;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + threadIdx.x / 16; i < all;
         i += static_cast<int64_t>(gridDim.x) * (kThreads / 16)) {
        const int64_t row = i / kb, c = i % kb * kBlock + lane * 8;
        float v[8];
        load8(static_cast<const T*>(a.x) + row * a.ldx, c, a.cols, v);
        uint32_t b = 0;
        for (int k = 0; k < 8; ++k) b = Max{}(b, abs_bits(v[k]));
        const uint32_t e = byte_of(lanes_reduce<16>(b, Max{}));
        if (lane == 0) a.scales[i] = static_cast<uint8_t>(e);
        emit<T>(a, row, c, v, e);
    }
}

// One scale for 128 x 128: a tile a workgroup, kept in registers between its largest
// magnitude and its codes.
template <typename T> __global__ __launch_bounds__(kThreads) void k_e4m3_tiles(QuantizeArgs a) {
    constexpr int kRows = kThreads / 16, kTurns = kBlock / kRows;
    __shared__ uint32_t lds[kThreads / kWave];
    const int64_t kb = (a.cols + kBlock - 1) / kBlock;
    const int64_t all = (a.rows + kBlock - 1) / kBlock * kb;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int64_t row0 = i / kb * kBlock + threadIdx.x / 16;
        const int64_t c = i % kb * kBlock + threadIdx.x % 16 * 8;
        float v[kTurns][8] = {};
        uint32_t b = 0;
        for (int t = 0; t < kTurns; ++t) {
            const int64_t row = row0 + t * kRows;
            if (row < a.rows) load8(static_cast<const T*>(a.x) + row * a.ldx, c, a.cols, v[t]);
        }
        for (int t = 0; t < kTurns; ++t)
            for (int k = 0; k < 8; ++k) b = Max{}(b, abs_bits(v[t][k]));
        b = wave_reduce(b, Max{});
        __syncthreads();                  // the last tile's have been read
        if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = b;
        __syncthreads();
        for (int w = 0; w < kThreads / kWave; ++w) b = Max{}(b, lds[w]);
        const uint32_t e = byte_of(b);
        if (threadIdx.x == 0) a.scales[i] = static_cast<uint8_t>(e);
        for (int t = 0; t < kTurns; ++t)
            if (row0 + t * kRows < a.rows) emit<T>(a, row0 + t * kRows, c, v[t], e);
    }
}

// ---- the product -------------------------------------------------------------
//
// y = x W^T.  The matrix cores' 8-bit instruction takes a step's 128 columns, all with one
// scale, at once, scales included.  It drops low bits of the smaller of its products, 1.4e-5
// to 2.5e-5 of the result in the 2-norm whatever its width: little beside bf16's own rounding
// (1.7e-3), too much for a binary32 result.  That one takes codes as bf16 numbers, which
// they are exactly with their scales, at half the rate.

template <bool EXACT, typename Y> struct ProductTile {
    StoreTile<Y> store;
    const uint8_t* w_scales;
    const uint8_t* x_scales;
    int64_t kb;

    template <int NT> struct Steps {
        const uint8_t* ws;
        const uint8_t* xs[NT];
        uint32_t w, x[NT];
        int64_t at, end;
        __device__ __forceinline__ void read() {
            if (at >= end) return;
            w = ws[at];
#pragma unroll
            for (int u = 0; u < NT; ++u) x[u] = xs[u][at];
            ++at;
        }
        __device__ __forceinline__ void enter(const ProductTile& e, const Place& p, int64_t) {
            const int64_t m = p.m0 < p.m ? p.m0 : p.m - 1;
            ws = e.w_scales + m / kBlock * e.kb;
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const int64_t n = p.n0 + u * 16 + threadIdx.x % 16;
                xs[u] = e.x_scales + (n < p.n ? n : p.n - 1) * e.kb;
            }
            at = 0;
            end = e.kb;
            read();
        }

        template <class SideA, class SideB, int MT, class Middle>
        __device__ __forceinline__ void product(const uint8_t* la, const uint8_t* lb, int wm, int wn,
                                                f32x4 (&acc)[MT][NT], Middle middle) {
            const uint32_t ew = w;
            uint32_t ex[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) ex[u] = x[u];
            read();                       // the next step's
            if constexpr (EXACT) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1) middle();
                    bf16x8 vb[NT][2];
#pragma unroll
                    for (int u = 0; u < NT; ++u) decode(SideB::codes(lb, wn, u, h), ex[u], vb[u]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        bf16x8 va[2];
                        decode(SideA::codes(la, wm, t, h), ew, va);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            for (int u = 0; u < NT; ++u)
                                acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    va[q], vb[u][q], acc[t][u], 0, 0, 0);
                    }
                }
            } else {
                auto whole = [](u32x4 a, u32x4 b) {
                    return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]),
                                 static_cast<int>(a[2]), static_cast<int>(a[3]),
                                 static_cast<int>(b[0]), static_cast<int>(b[1]),
                                 static_cast<int>(b[2]), static_cast<int>(b[3])};
                };
                i32x8 vb[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u)
                    vb[u] = whole(SideB::codes(lb, wn, u, 0), SideB::codes(lb, wn, u, 1));
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (t == MT / 2) middle();
                    const i32x8 va = whole(SideA::codes(la, wm, t, 0), SideA::codes(la, wm, t, 1));
#pragma unroll
                    for (int u = 0; u < NT; ++u)
                        acc[t][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            va, vb[u], acc[t][u], 0, 0, 0, static_cast<int>(ew), 0,
                            static_cast<int>(ex[u]));
                }
            }
        }

        // 16 codes as 2 x 8 bf16 values, the scale applied.
        static __device__ __forceinline__ void decode(u32x4 c, uint32_t byte, bf16x8* out) {
            const float b = __uint_as_float(byte << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4 v = {
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     c[2 * i], b, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     c[2 * i], b, true)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     c[2 * i + 1], b, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     c[2 * i + 1], b, true))};
                out[i] = __builtin_bit_cast(bf16x8, v);
            }
        }
    };

    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x4 (&acc)[MT][NT], const Place& at) const {
        store.finish(acc, at);
    }
};

template <bool EXACT, typename Y> hipError_t matmul_of(const E4m3ProductArgs& a, hipStream_t s) {
    const ProductArgs p{a.w, a.ldw, a.x, a.ldx, a.rows, a.count, a.cols, 1, nullptr, false};
    const ProductTile<EXACT, Y> e{StoreTile<Y>(a.y, a.ldy), a.w_scales, a.x_scales,
                                  (a.cols + kBlock - 1) / kBlock};
    const dim3 block(kTileThreads);
    // Few tiles: smaller ones, so that more CUs have some.
    const int64_t big = (a.rows + 255) / 256 * ((a.count + 255) / 256);
    if (big >= 128) {
        k_product<ViaCodes, false, false, 256, 256, 2, 4, ProductTile<EXACT, Y>>
            <<<dim3(product_grid(a.rows, a.count, 256, 256, 1, kTileGroups)), block, 0, s>>>(p, e);
    } else {
        k_product<ViaCodes, false, false, 128, 64, 4, 2, ProductTile<EXACT, Y>>
            <<<dim3(product_grid(a.rows, a.count, 128, 64, 1, 2 * kTileGroups)), block, 0, s>>>(p, e);
    }
    return hipGetLastError();
}

template <typename T> hipError_t quantize(const QuantizeArgs& a, int kind, hipStream_t s) {
    const int64_t kb = (a.cols + kBlock - 1) / kBlock;
    const dim3 block(kThreads);
    if (kind == DL_SCALE_BLOCK128) {
        const int64_t n = (a.rows * kb + kThreads / 16 - 1) / (kThreads / 16);
        k_e4m3_blocks<T><<<dim3(static_cast<unsigned>(n < 16384 ? n : 16384)), block, 0, s>>>(a);
    } else {
        const int64_t n = (a.rows + kBlock - 1) / kBlock * kb;
        k_e4m3_tiles<T><<<dim3(static_cast<unsigned>(n < 16384 ? n : 16384)), block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t e4m3_quantize(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* codes, int64_t ldc, uint8_t* scales, int scale_kind,
                         void* values, int64_t ldvalues, hipStream_t s) {
    const QuantizeArgs a{x, ldx, rows, cols, codes, ldc, scales, values, ldvalues};
    return dtype == DL_F32 ? quantize<float>(a, scale_kind, s) : quantize<bf16>(a, scale_kind, s);
}

hipError_t e4m3_matmul(const E4m3ProductArgs& a, int y_dtype, hipStream_t s) {
    return y_dtype == DL_F32 ? matmul_of<true, float>(a, s) : matmul_of<false, bf16>(a, s);
}

}  // namespace dlk
