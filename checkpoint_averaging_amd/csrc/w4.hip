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

// ---- the layout --------------------------------------------------------------
//
// Elementwise but for a block's largest magnitude, so bound by the bytes in and
// out.  A lane takes eight neighbouring columns and four lanes a block: the
// largest magnitude goes round them by DPP, and the hardware's conversion
// rounds to the eight magnitudes (nearest, ties to even) with the scale a power
// of two, so that nothing but this rounding is inexact.  73760 x 2048 fp32 with
// the values written too: 227 us, 5.7 TB/s.

template <typename F> __device__ __forceinline__ uint32_t bits_of(F v) {
    static_assert(sizeof(F) == 4, "");
    return __builtin_bit_cast(uint32_t, v);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_w4_quantize(const T* w, int64_t ldw, int64_t rows,
                                                          int64_t cols, uint8_t* packed,
                                                          uint8_t* scales, T* values,
                                                          int64_t ldv, int64_t slab) {
    // All rows' groups of eight columns in a line, `slab` rows for each y of
    // the grid so that 32 bits count them.
    const uint32_t lanes = static_cast<uint32_t>((cols + 31) / 32 * 4);
    const int64_t kb = lanes / 4;
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * slab;
    const uint32_t n = static_cast<uint32_t>(rows - row0 < slab ? rows - row0 : slab) * lanes;
    const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
    if (at < n) {                             // (four lanes of a block together)
        const int64_t row = row0 + at / lanes, i = at % lanes;
        float v[8];
        load8(w + row * ldw, i * 8, cols, v);
        uint32_t b = 0;
        for (int k = 0; k < 8; ++k) b = Max{}(b, abs_bits(v[k]));
        b = lanes_reduce<4>(b, Max{});
        // the smallest power of two s with amax <= 6 s = 1.5 * 2^2 s
        int e = static_cast<int>((b + 0x3FFFFFu) >> 23) - 2;
        e = e < 0 ? 0 : e;
        const bool bad = b >= 0x7F800000u;
        const float back = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        uint32_t q = 0;
        if (bad) {
            e = 255;
        } else {
            for (int k = 0; k < 8; ++k) v[k] *= back;
            q = static_cast<uint32_t>(
                __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.0f, 0));
            q = static_cast<uint32_t>(
                __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1));
            q = static_cast<uint32_t>(
                __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.0f, 2));
            q = static_cast<uint32_t>(
                __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.0f, 3));
        }
        reinterpret_cast<uint32_t*>(packed)[row * kb * 4 + i] = q;
        if (threadIdx.x % 4 == 0) scales[row * kb + i / 4] = static_cast<uint8_t>(e);
        if (values != nullptr) {
            // (the conversion takes the scale's exponent bits: all zeros is 2^-127, all ones NaN)
            const float s = __uint_as_float(static_cast<uint32_t>(e) << 23);
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 o[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2),
                                __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3)};
            for (int k = 0; k < 8; ++k) v[k] = o[k / 2][k % 2];
            store8(values + row * ldv, i * 8, cols, v);
        }
    }
}

// ---- the product -------------------------------------------------------------
//
// y[v][r] = sum_k x[v][k] W[r][k] as 16 x 16 tiles of v_mfma_f32_16x16x32_bf16:
// rows of W against (up to 16) vectors.  A code times its block's power of two
// is a bfloat16 number, and so is an e4m3 value times its own: products are
// exact and sums binary32.
//
// Bound by the weights' bytes (17 for 32 weights) once there are enough of
// them.  A lane's 16 bytes are the 32 codes of one row's block, all with one
// scale, and the four lanes of a row take four neighbouring blocks (a span of
// 128 columns): the four products of a span take eight codes each of every
// lane, whatever columns these are, as x is laid out the same.  The vectors
// stay in registers: a wave has kSpans spans of them and passes rows by, so
// x is read once a workgroup, not once a tile (past 2048 columns, again for
// every 2048; spans enough for 8192 in registers, or the next ones under way,
// leave too few waves and were slower).  The waves of a workgroup take
// different spans of the same rows, and their sums meet in LDS.
//
// The matrix cores also have a product of 4-bit and 8-bit values with block
// scales (v_mfma_scale_f32_16x16x128_f8f6f4).  It drops low bits of the smaller
// of its 128 products: up to 5e-4 of the sum of magnitudes on random codes (6e-5
// with all scales equal), too many for a binary32 result.

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

constexpr int kMatThreads = 512;
constexpr int kMatWaves = kMatThreads / kWave;
constexpr int kSpans = 2;

// 32 codes (four words) as 4 x 8 bf16 values, the block's scale applied.
__device__ __forceinline__ void decode(u32x4 w, uint32_t byte, bf16x8* out) {
    // The conversion takes a scale's exponent from a binary32 number's: all
    // ones is NaN there, all zeros 2^-127.
    const float b = __uint_as_float(byte << 23);
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = w[i];
        const u32x4 v = {bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, b, 0)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, b, 1)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, b, 2)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, b, 3))};
        out[i] = __builtin_bit_cast(bf16x8, v);
    }
}

// 32 elements of one vector from column k0 on, 0 past the end, in the order in
// which decode() has the weights.
template <int KIND>
__device__ __forceinline__ void load_vector(const MatvecArgs& a, int v, int64_t k0, bf16x8* out) {
    const int64_t kb = (a.cols + 31) / 32;
    u32x4 q[4] = {};
    if (KIND == DL_SCALE_NONE) {
        if (v < a.count && k0 < a.cols) {
            const uint16_t* p = static_cast<const uint16_t*>(a.x) + v * a.ldx + k0;
            if (k0 + 32 <= a.cols) {
                for (int i = 0; i < 4; ++i) q[i] = reinterpret_cast<const u32x4_any*>(p)[i];
            } else {
                const int n = static_cast<int>(a.cols - k0);
                for (int i = 0; i < 16; ++i) {
                    const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
                    q[i / 4][i % 4] = lo | (hi << 16);
                }
            }
        }
        for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(bf16x8, q[i]);
        return;
    }
    uint32_t byte = 127;
    if (v < a.count && k0 < a.cols) {
        const uint8_t* p = static_cast<const uint8_t*>(a.x) + v * a.ldx + k0;
        if (KIND == DL_SCALE_BLOCK32) byte = static_cast<const uint8_t*>(a.x_scales)[v * kb + k0 / 32];
        if (k0 + 32 <= a.cols) {
            for (int i = 0; i < 2; ++i) q[i] = reinterpret_cast<const u32x4_any*>(p)[i];
        } else {
            const int n = static_cast<int>(a.cols - k0);
            for (int i = 0; i < 32; ++i)
                q[i / 16][i / 4 % 4] |= (i < n ? static_cast<uint32_t>(p[i]) : 0) << (8 * (i % 4));
        }
    }
    const float b = __uint_as_float(byte << 23);
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = q[i / 2][i % 2 * 2], d = q[i / 2][i % 2 * 2 + 1];
        const u32x4 r = {bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, b, false)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, b, true)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, b, false)),
                         bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, b, true))};
        out[i] = __builtin_bit_cast(bf16x8, r);
    }
}

// MT tiles of 16 vectors, RT tiles of 16 rows a wave; kw of the workgroup's
// waves (2, 4 or 8) share rows and split the columns, the others take other
// rows.
template <int KIND, int MT, int RT, typename Y>
__global__ __launch_bounds__(kMatThreads) void k_w4_matvec(MatvecArgs a, int kw) {
    __shared__ f32x4 part[kMatWaves][RT][MT][16][4];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int l16 = lane % 16, j = lane / 16;
    const int k_of = wave % kw, tw = kMatWaves / kw, t_of = wave / kw;
    const int64_t kb = (a.cols + 31) / 32;
    const int64_t chunk = static_cast<int64_t>(kw) * kSpans * 4;          // blocks of all waves
    const int64_t groups = (a.rows + 16 * RT - 1) / (16 * RT);
    bf16x8 x[MT][kSpans][4];
    // The weights of one chunk of columns of one group of rows, a step.  Four
    // neighbouring lanes load 64 bytes of a row; the lane that the product
    // wants them in gets them at use.  A row's eight scale bytes come in one
    // load where it has as many.
    auto load = [&](int64_t g, int64_t c, u32x4 (&w)[RT][kSpans], uint32_t (&e)[RT][kSpans]) {
        const int64_t b0 = c + static_cast<int64_t>(k_of) * (kSpans * 4);
        const int64_t r0 = (g + t_of) * (16 * RT);
        for (int t = 0; t < RT; ++t) {
            int64_t row = r0 + t * 16 + lane / 4;
            row = row < a.rows ? row : a.rows - 1;
            for (int s = 0; s < kSpans; ++s) {
                const int64_t b = b0 + s * 4 + lane % 4;
                w[t][s] = u32x4{};
                if (b < kb) w[t][s] = *reinterpret_cast<const u32x4*>(a.packed + (row * kb + b) * 16);
            }
            row = r0 + t * 16 + l16;
            row = row < a.rows ? row : a.rows - 1;
            if (b0 + kSpans * 4 <= kb) {
                const u32x2_any q = *reinterpret_cast<const u32x2_any*>(a.scales + row * kb + b0);
                for (int s = 0; s < kSpans; ++s) e[t][s] = q[s];
            } else {
                for (int s = 0; s < kSpans; ++s) {
                    const int64_t b = b0 + s * 4 + j;
                    e[t][s] = b < kb ? static_cast<uint32_t>(a.scales[row * kb + b]) << (8 * j) : 0;
                }
            }
        }
    };
    int64_t g0 = static_cast<int64_t>(blockIdx.x) * tw, c0 = 0;
    u32x4 w[RT][kSpans];
    uint32_t e[RT][kSpans];
    f32x4 acc[RT][MT] = {};
    if (g0 < groups) load(g0, c0, w, e);
    bool first = true;
    while (g0 < groups) {
        // the next step's weights are under way during this step's products
        int64_t g1 = g0, c1 = c0 + chunk;
        if (c1 >= kb) {
            c1 = 0;
            g1 = g0 + static_cast<int64_t>(gridDim.x) * tw;
        }
        if (first || chunk < kb) {
            const int64_t b0 = c0 + (static_cast<int64_t>(k_of) * kSpans) * 4 + j;
            for (int m = 0; m < MT; ++m)
                for (int s = 0; s < kSpans; ++s)
                    load_vector<KIND>(a, m * 16 + l16, (b0 + s * 4) * 32, x[m][s]);
            first = false;
        }
        u32x4 wn[RT][kSpans];
        uint32_t en[RT][kSpans];
        if (g1 < groups) load(g1, c1, wn, en);
        for (int s = 0; s < kSpans; ++s)
            for (int t = 0; t < RT; ++t) {
                bf16x8 v[4];
                u32x4 q;
                for (int i = 0; i < 4; ++i)
                    q[i] = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(
                        (l16 * 4 + j) * 4, static_cast<int>(w[t][s][i])));
                decode(q, (e[t][s] >> (8 * j)) & 0xFFu, v);
                for (int m = 0; m < MT; ++m)
                    for (int i = 0; i < 4; ++i)
                        acc[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[i], x[m][s][i],
                                                                            acc[t][m], 0, 0, 0);
            }
        const int64_t row0 = (g0 + t_of) * (16 * RT);
        const bool done = c1 == 0;
        g0 = g1;
        c0 = c1;
        for (int t = 0; t < RT; ++t)
            for (int s = 0; s < kSpans; ++s) {
                w[t][s] = wn[t][s];
                e[t][s] = en[t][s];
            }
        if (!done) continue;
        // Lane (j, l16) has rows 4j .. 4j+3 of vector l16 of each tile.
        __syncthreads();                      // the last rows' sums have been read
        for (int t = 0; t < RT; ++t)
            for (int m = 0; m < MT; ++m) part[wave][t][m][l16][j] = acc[t][m];
        __syncthreads();
        constexpr int kOut = RT * MT * 64;    // four rows of a vector each
        for (int o = k_of * kWave + lane; o < kOut; o += kw * kWave) {
            const int jj = o % 4, t = o / 4 % RT, v = o / (4 * RT);
            f32x4 r = part[wave - k_of][t][v / 16][v % 16][jj];
            for (int q = 1; q < kw; ++q) r += part[wave - k_of + q][t][v / 16][v % 16][jj];
            const int64_t row = row0 + t * 16 + jj * 4;
            if (v < a.count) {
                if (KIND == DL_SCALE_ROW) r *= static_cast<const float*>(a.x_scales)[v];
                Y* y = static_cast<Y*>(a.y) + v * a.ldy + row;
                for (int i = 0; i < 4; ++i)
                    if (row + i < a.rows) y[i] = from_f32<Y>(r[i]);
            }
        }
        for (int t = 0; t < RT; ++t)
            for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{};
    }
}

template <int KIND, int MT, int RT>
hipError_t matvec(const MatvecArgs& a, int y_dtype, hipStream_t s) {
    const int64_t spans = ((a.cols + 31) / 32 + 3) / 4;
    int kw = 2;
    while (kw < kMatWaves && kw * kSpans < spans) kw *= 2;
    const int64_t groups = (a.rows + 16 * RT - 1) / (16 * RT);
    const int64_t tw = kMatWaves / kw;
    int64_t blocks = (groups + tw - 1) / tw;
    // what is resident at once: two workgroups a CU, one with two tiles of vectors
    constexpr int64_t kMost = MT == 1 ? 512 : 256;
    blocks = blocks < kMost ? blocks : kMost;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kMatThreads);
    if (y_dtype == DL_F32) k_w4_matvec<KIND, MT, RT, float><<<grid, block, 0, s>>>(a, kw);
    else k_w4_matvec<KIND, MT, RT, bf16><<<grid, block, 0, s>>>(a, kw);
    return hipGetLastError();
}

template <int KIND> hipError_t matvec_of(const MatvecArgs& a, int y_dtype, hipStream_t s) {
    // Two row tiles a wave keep more bytes under way (73760 x 2048: 19 us, 25 us
    // with one, 22 us with four, which leave room for half the waves); few rows
    // are spread over more workgroups instead (5632 x 2048: 4.3 us, 5.0 us).
    const bool many = a.rows >= 8 * 1024;
    if (a.count <= 16)
        return many ? matvec<KIND, 1, 2>(a, y_dtype, s) : matvec<KIND, 1, 1>(a, y_dtype, s);
    return many ? matvec<KIND, 2, 2>(a, y_dtype, s) : matvec<KIND, 2, 1>(a, y_dtype, s);
}

}  // namespace

hipError_t w4_quantize(const void* w, int64_t ldw, int dtype, int64_t rows, int64_t cols,
                       uint8_t* packed, uint8_t* scales, void* values, int64_t ldvalues,
                       hipStream_t s) {
    const int64_t lanes = (cols + 31) / 32 * 4;
    int64_t slab = (int64_t(1) << 30) / lanes;
    slab = slab < rows ? slab : rows;
    const dim3 grid(static_cast<unsigned>((slab * lanes + kThreads - 1) / kThreads),
                    static_cast<unsigned>((rows + slab - 1) / slab)),
        block(kThreads);
    if (dtype == DL_F32)
        k_w4_quantize<<<grid, block, 0, s>>>(static_cast<const float*>(w), ldw, rows, cols, packed,
                                             scales, static_cast<float*>(values), ldvalues, slab);
    else
        k_w4_quantize<<<grid, block, 0, s>>>(static_cast<const bf16*>(w), ldw, rows, cols, packed,
                                             scales, static_cast<bf16*>(values), ldvalues, slab);
    return hipGetLastError();
}

hipError_t w4_matvec(const MatvecArgs& a, int x_scale_kind, int y_dtype, hipStream_t s) {
    if (x_scale_kind == DL_SCALE_NONE) return matvec_of<DL_SCALE_NONE>(a, y_dtype, s);
    if (x_scale_kind == DL_SCALE_ROW) return matvec_of<DL_SCALE_ROW>(a, y_dtype, s);
    return matvec_of<DL_SCALE_BLOCK32>(a, y_dtype, s);
}

}  // namespace dlk
