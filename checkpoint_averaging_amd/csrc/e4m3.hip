// Matrices in 8 bits (e4m3) with a power-of-two scale for each 128 x 128
// elements or each 128 of a row: their layout, and the product of the two.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "few.h"
#include "head.h"
#include "head_device.h"
#include "tiles.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

// ---- the layout --------------------------------------------------------------
//
// Bound by memory: an element is read once, its block's largest magnitude is found by a
// reduction over lanes (and LDS, where a block has 128 rows), and its code and value are
// written from the registers that held it.  73,760 x 2048 fp32 with values: 258 us (1.36 GB, 5.3
// TB/s); 16,383 x 2048 bf16 in blocks of a row, with values: 32 us (5.3 TB/s).

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
//
// 73,760 x 2048 with 2048 tokens: 0.58 ms in fp32 (1.06 PFLOP/s, as a bf16 product reaches), 0.35
// in bf16 (1.76); 5632 x 2048 with 8191 tokens in bf16: 94 us, 2.0 PFLOP/s.  The power that the
// matrix cores may take bounds the large ones: clocks fall from 2.4 GHz to 1.9.  Up to 32
// tokens (few.h) read W once: one token 29 us, 5.2 TB/s; 32 tokens 37 against the tiles' 33 to
// 40, and with 2048 rows, whose tiles are few, 19 against 33.

template <typename Y> struct ProductTile : StoreTile<Y> {
    const uint8_t* w_scales;
    const uint8_t* x_scales;
    int64_t kb;
};

// The scales of a wave's rows of W (in one block of 128) and of its lanes' tokens, read one
// step ahead.
template <class Epilogue, int NT> struct Scales {
    const uint8_t* ws;
    const uint8_t* xs[NT];
    uint32_t w, x[NT], w_next, x_next[NT];
    int64_t at, end;

    __device__ __forceinline__ void read() {
        const int64_t i = at < end ? at : end - 1;
        w_next = ws[i];
        for (int u = 0; u < NT; ++u) x_next[u] = xs[u][i];
        ++at;
    }
    __device__ __forceinline__ void enter(const Epilogue& e, const Place& p) {
        const int64_t m = p.m0 < p.m ? p.m0 : p.m - 1;
        ws = e.w_scales + m / kBlock * e.kb;
        for (int u = 0; u < NT; ++u) {
            const int64_t n = p.n0 + u * kSquare + threadIdx.x % kSquare;
            xs[u] = e.x_scales + (n < p.n ? n : p.n - 1) * e.kb;
        }
        at = 0;
        end = e.kb;
        read();
    }
    __device__ __forceinline__ void step() {
        w = w_next;
        for (int u = 0; u < NT; ++u) x[u] = x_next[u];
        read();
    }
};

// The matrix cores' 8-bit products: 64 codes of a row at once, 32 of them in each half of the
// lanes.
template <class Epilogue, int MT, int NT, int SUBS> struct CodeMath : Scales<Epilogue, NT> {
    static constexpr int kSubs = SUBS / 2, kAhead = 1, kSlots = 2;
    struct A {
        u32x4 h[2];
    };
    struct B {
        A v[NT];
    };
    __device__ __forceinline__ void take(const B&) {}
    template <class S> __device__ __forceinline__ A read_a(const uint8_t* l, int w, int t, int sub) {
        const int c = 4 * sub + threadIdx.x % kWave / 32 * 2;
        return A{{S::codes(l, w, t, c), S::codes(l, w, t, c + 1)}};
    }
    template <class S> __device__ __forceinline__ B read_b(const uint8_t* l, int w, int sub) {
        B b;
        for (int u = 0; u < NT; ++u) b.v[u] = read_a<S>(l, w, u, sub);
        return b;
    }
    __device__ __forceinline__ void multiply(const A& a, const B& b, f32x16 (&acc)[NT]) {
        const i32x8 va = __builtin_bit_cast(i32x8, a);
        for (int u = 0; u < NT; ++u)
            acc[u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                va, __builtin_bit_cast(i32x8, b.v[u]), acc[u], 0, 0, 0, static_cast<int>(this->w),
                0, static_cast<int>(this->x[u]));
    }
};

// Codes as bf16 numbers, which they are exactly with their scales: 16 of each lane's row at
// once, for two bf16 instructions.
template <class Epilogue, int MT, int NT, int SUBS> struct ExactCodeMath : Scales<Epilogue, NT> {
    static constexpr int kSubs = SUBS, kAhead = 1, kSlots = 1;
    typedef u32x4 A;
    struct B {
        u32x4 v[NT];
    };
    bf16x8 held[NT][2];

    // 16 codes as 2 x 8 bf16 values, the scale applied.
    static __device__ __forceinline__ void decode(u32x4 c, uint32_t byte, bf16x8* out) {
        const float b = __uint_as_float(byte << 23);
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
    __device__ __forceinline__ void take(const B& b) {
        for (int u = 0; u < NT; ++u) decode(b.v[u], this->x[u], held[u]);
    }
    template <class S> __device__ __forceinline__ A read_a(const uint8_t* l, int w, int t, int sub) {
        return S::codes(l, w, t, sub * 2 + threadIdx.x % kWave / 32);
    }
    template <class S> __device__ __forceinline__ B read_b(const uint8_t* l, int w, int sub) {
        B b;
        for (int u = 0; u < NT; ++u) b.v[u] = read_a<S>(l, w, u, sub);
        return b;
    }
    __device__ __forceinline__ void multiply(const A& a, const B&, f32x16 (&acc)[NT]) {
        bf16x8 va[2];
        decode(a, this->w, va);
        for (int q = 0; q < 2; ++q)
            for (int u = 0; u < NT; ++u)
                acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[q], held[u][q], acc[u], 0, 0, 0);
    }
};

// A few tokens: each result written as it is.
template <typename Y> struct StoreFew {
    static constexpr bool kRowsFirst = true;
    Y* y;
    int64_t ld;
    __device__ __forceinline__ void begin() {}
    __device__ __forceinline__ void value(float c, int64_t row, int v) {
        y[v * ld + row] = from_f32<Y>(c);
    }
    __device__ __forceinline__ void end(float*, int) {}
};

constexpr int kFewTokens = 32;

template <typename Y> hipError_t few_tokens(const E4m3ProductArgs& a, hipStream_t s) {
    const FewArgs f{a.w, a.ldw, a.rows, a.cols, a.x, a.ldx, static_cast<int>(a.count), a.w_scales,
                    a.x_scales};
    const StoreFew<Y> e{static_cast<Y*>(a.y), a.ldy};
    // Two row tiles a wave keep more bytes under way; with few rows there are more workgroups
    // with one.
    const bool many = a.rows >= 8 * 1024;
    if (a.count <= 16)
        return many ? few<FewCodes<8>, 1, 2>(f, e, 512, s) : few<FewCodes<8>, 1, 1>(f, e, 512, s);
    return many ? few<FewCodes<8>, 2, 2>(f, e, 256, s) : few<FewCodes<8>, 2, 1>(f, e, 256, s);
}

template <template <class, int, int, int> class Math, typename Y>
hipError_t matmul_of(const E4m3ProductArgs& a, hipStream_t s) {
    typedef ProductTile<Y> E;
    const ProductArgs p{a.w, a.ldw, a.x, a.ldx, a.rows, a.count, a.cols, 1, nullptr, false, 0, 0};
    const E e{StoreTile<Y>(a.y, a.ldy), a.w_scales, a.x_scales, (a.cols + kBlock - 1) / kBlock};
    if (a.count <= kFewTokens) return few_tokens<Y>(a, s);
    const dim3 block(kTileThreads);
    // Few tiles: smaller ones, so that more CUs have some (5632 rows x 2048, bf16 out: 512
    // tokens 19.6 us against 28.4, 1024 31.8 against 30.3, 1600 47.8 against 32.5).  And while
    // half of a large tile's tokens or more would be none (73,760 rows x 2048: 64 tokens 38 us
    // against 98 in fp32; 128 tokens 52 against 57 and 160 63 against 58 in bf16, 192 89 against
    // 106 and 256 126 against 111 in fp32, whose products take longer).
    const int64_t big = (a.rows + 255) / 256 * ((a.count + 255) / 256);
    if (big >= 128 && a.count > (sizeof(Y) == 4 ? 192 : 128)) {
        const dim3 grid(product_grid(a.rows, a.count, 256, 256, 1, kTileGroups));
        if (direct(a.w, a.ldw, 1, a.cols) && direct(a.x, a.ldx, 1, a.cols))
            k_product_direct<ViaCodes, false, false, 256, 256, 2, 4, E, Math>
                <<<grid, block, 0, s>>>(p, e);
        else
            k_product<ViaCodes, false, false, 256, 256, 2, 4, E, Math><<<grid, block, 0, s>>>(p, e);
    } else {
        k_product<ViaCodes, false, false, 128, 64, 4, 2, E, Math>
            <<<dim3(product_grid(a.rows, a.count, 128, 64, 1, 2 * kTileGroups)), block, 0, s>>>(p,
                                                                                               e);
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
    return y_dtype == DL_F32 ? matmul_of<ExactCodeMath, float>(a, s) : matmul_of<CodeMath, bf16>(a, s);
}

}  // namespace dlk
