// The product of a long matrix with a few vectors, shared by the output head's
// kernels (headloss.hip, e4m3.hip):
//
//   C[v][r] = sum over k < cols of X[v][k] M[r][k],    v < count <= 16 NT
//
// Bound by the matrix's bytes, each read once.  A workgroup's eight waves take
// different columns of the same rows (kw of them; with fewer columns the others
// take other rows) and keep the vectors' parts in registers, as the matrix
// instruction (16 rows x 16 vectors x 32 columns) wants them; past kw * STEPS * 32
// columns they are loaded again for every chunk of them.  The next rows are under way
// while these are multiplied.  One load has 64 bytes of each of 16 rows, by four lanes
// 16 apart (of binary32 every other 16 of 128).  The waves' sums meet in LDS, where one
// thread a result adds them and hands it to the epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.h"
#include "tiles.h"

namespace dlk {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct FewArgs {
    const void* matrix;
    int64_t ld;
    int64_t rows;
    int64_t cols;
    const void* x;
    int64_t ldx;
    int count;
    const uint8_t* scales;                // of codes, for 128 x 128
    const uint8_t* x_scales;              // for 128 of a vector
};

// 16 bytes of a row from element c on, 0 past its end.
template <typename T>
__device__ __forceinline__ u32x4 piece_of(const T* row, int64_t c, int64_t cols) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    u32x4 v = {};
    if (c + kPer <= cols) {
        v = *reinterpret_cast<const typename Raw<T>::any*>(row + c);
    } else if (c < cols) {
        const int n = static_cast<int>(cols - c);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            constexpr int kIn = 4 / static_cast<int>(sizeof(T));
            uint32_t e = 0;
            __builtin_memcpy(&e, row + c + i, sizeof(T));
            e <<= i % kIn * 8 * static_cast<int>(sizeof(T)) % 32;
            for (int k = 0; k < 4; ++k) v[k] |= i / kIn == k ? e : 0;
        }
    }
    return v;
}

// What STEPS steps of 32 columns of a row are in memory (raw, a lane's share of them), and as
// operands.  Lane group g = lane / 16 has of each 64 bytes (bf16, codes) or 128 (binary32) the
// g-th quarter.
template <int STEPS> struct FewBf16 {
    typedef bf16 elem;
    static constexpr int kSteps = STEPS, kPieces = STEPS, kPlanes = 1;
    static __device__ __forceinline__ int64_t column(int i, int g) { return i * 32 + g * 8; }
    static __device__ __forceinline__ void operand(const u32x4* raw, int step, uint32_t,
                                                   bf16x8* out) {
        out[0] = __builtin_bit_cast(bf16x8, raw[step]);
    }
};
template <int STEPS> struct FewSplit {
    typedef float elem;
    static constexpr int kSteps = STEPS, kPieces = 2 * STEPS, kPlanes = 3;
    static __device__ __forceinline__ int64_t column(int i, int g) {
        return i / 2 * 32 + g * 8 + i % 2 * 4;
    }
    static __device__ __forceinline__ void operand(const u32x4* raw, int step, uint32_t,
                                                   bf16x8* out) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        u32x4 q[3];
        for (int i = 0; i < 4; ++i) {
            const u32x4 r = raw[2 * step + i / 2];
            float x = __uint_as_float(r[i % 2 * 2]), y = __uint_as_float(r[i % 2 * 2 + 1]);
            for (int p = 0; p < 3; ++p) {
                q[p][i] = __builtin_bit_cast(uint32_t,
                                             __builtin_convertvector((f32x2{x, y}), bf16x2));
                x -= __uint_as_float(q[p][i] << 16);
                y -= __uint_as_float(q[p][i] & 0xFFFF0000u);
            }
        }
        for (int p = 0; p < 3; ++p) out[p] = __builtin_bit_cast(bf16x8, q[p]);
    }
};
template <int STEPS> struct FewCodes {
    typedef uint8_t elem;
    static constexpr int kSteps = STEPS, kPieces = STEPS / 2, kPlanes = 1;
    static __device__ __forceinline__ int64_t column(int i, int g) { return i * 64 + g * 16; }
    // (step i of a lane: half of the 16 codes of piece i/2, whatever columns these are)
    static __device__ __forceinline__ void operand(const u32x4* raw, int step, uint32_t scale,
                                                   bf16x8* out) {
        const float b = __uint_as_float(scale << 23);
        u32x4 v;
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = raw[step / 2][step % 2 * 2 + i / 2];
            v[i] = i % 2 == 0
                       ? __builtin_bit_cast(uint32_t,
                                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, b, false))
                       : __builtin_bit_cast(uint32_t,
                                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, b, true));
        }
        out[0] = __builtin_bit_cast(bf16x8, v);
    }
};

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;

// Src: one of the above; NT: tiles of 16 vectors; RT: tiles of 16 rows a wave.
template <class Src, int NT, int RT, class Epilogue>
__global__ __launch_bounds__(kFewThreads, 2) void k_few(FewArgs a, Epilogue e, int kw) {
    typedef typename Src::elem T;
    constexpr bool kScaled = sizeof(T) == 1;
    constexpr int kSteps = Src::kSteps, kPieces = Src::kPieces, kPlanes = Src::kPlanes;
    // (a wave's columns begin at a block of 128)
    constexpr int kScales = kScaled ? kSteps / 4 : 1;
    static_assert(!kScaled || kSteps % 4 == 0, "");
    __shared__ f32x4 part[2][kFewWaves][RT][NT][16][4];
    const int wave = scalar(static_cast<int>(threadIdx.x / kWave)), lane = threadIdx.x % kWave;
    const int l16 = lane % 16, g = lane / 16;
    const int k_of = wave % kw, t_of = wave / kw, tw = kFewWaves / kw;
    const int64_t chunk = static_cast<int64_t>(kw) * kSteps * 32;
    const int64_t groups = (a.rows + 16 * RT - 1) / (16 * RT);
    const int64_t kb = (a.cols + 127) / 128;
    const T* const matrix = static_cast<const T*>(a.matrix);
    auto scale_at = [&](const uint8_t* scales, int64_t line, int64_t c) -> uint32_t {
        return c < a.cols ? scales[line * kb + c / 128] : 127;
    };
    // The matrix's share of this wave: rows of group q, columns of the chunk from c on.
    auto load = [&](int64_t q, int64_t c, u32x4 (&raw)[RT][kPieces], uint32_t (&s)[RT][kScales]) {
        const int64_t c0 = c + static_cast<int64_t>(k_of) * kSteps * 32;
        for (int t = 0; t < RT; ++t) {
            int64_t row = (q + t_of) * (16 * RT) + t * 16;
            const int64_t first = row < a.rows ? row : a.rows - 1;
            row = row + l16 < a.rows ? row + l16 : a.rows - 1;
            for (int i = 0; i < kPieces; ++i)
                raw[t][i] = piece_of(matrix + row * a.ld, c0 + Src::column(i, g), a.cols);
            for (int i = 0; i < kScales; ++i)
                s[t][i] = kScaled ? scale_at(a.scales, first / 128, c0 + i * 128) : 0;
        }
    };
    bf16x8 x[NT][kSteps][kPlanes];
    auto load_x = [&](int64_t c) {
        const int64_t c0 = c + static_cast<int64_t>(k_of) * kSteps * 32;
        for (int u = 0; u < NT; ++u) {
            const int v = u * 16 + l16;
            u32x4 raw[kPieces];
            for (int i = 0; i < kPieces; ++i)
                raw[i] = v < a.count ? piece_of(static_cast<const T*>(a.x) + v * a.ldx,
                                                c0 + Src::column(i, g), a.cols)
                                     : u32x4{};
            for (int i = 0; i < kSteps; ++i) {
                const uint32_t s = kScaled && v < a.count
                                       ? scale_at(a.x_scales, v, c0 + i / 4 * 128) : 127;
                Src::operand(raw, i, s, x[u][i]);
            }
        }
    };
    int64_t q0 = static_cast<int64_t>(blockIdx.x) * tw, c0 = 0;
    u32x4 raw[RT][kPieces];
    uint32_t s[RT][kScales];
    f32x4 acc[RT][NT] = {};
    load(q0, c0, raw, s);
    load_x(0);
    e.begin();
    int buf = 0;
    while (q0 < groups) {
        int64_t q1 = q0, c1 = c0 + chunk;
        if (c1 >= a.cols) {
            c1 = 0;
            q1 = q0 + static_cast<int64_t>(gridDim.x) * tw;
        }
        u32x4 raw_next[RT][kPieces];
        uint32_t s_next[RT][kScales];
        if (q1 < groups) load(q1, c1, raw_next, s_next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            for (int t = 0; t < RT; ++t) {
                bf16x8 m[kPlanes];
                Src::operand(raw[t], i, s[t][kScaled ? i / 4 : 0], m);
                for (int u = 0; u < NT; ++u) {
                    if constexpr (kPlanes == 3) {
                        constexpr int pa[6] = {0, 2, 1, 0, 1, 0}, pb[6] = {2, 0, 1, 1, 0, 0};
                        for (int p = 0; p < 6; ++p)
                            acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                m[pa[p]], x[u][i][pb[p]], acc[t][u], 0, 0, 0);
                    } else {
                        acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(m[0], x[u][i][0],
                                                                            acc[t][u], 0, 0, 0);
                    }
                }
            }
        const int64_t row0 = q0 * (16 * RT);
        q0 = q1;
        c0 = c1;
        for (int t = 0; t < RT; ++t) {
            for (int i = 0; i < kPieces; ++i) raw[t][i] = raw_next[t][i];
            for (int i = 0; i < kScales; ++i) s[t][i] = s_next[t][i];
        }
        if (chunk < a.cols) load_x(c0);
        if (c0 != 0) continue;
        // Lane (g, l16) has rows 4g .. 4g+3 of vector l16 of each tile.
        for (int t = 0; t < RT; ++t)
            for (int u = 0; u < NT; ++u) {
                part[buf][wave][t][u][l16][g] = acc[t][u];
                acc[t][u] = f32x4{};
            }
        __syncthreads();
        const float* sums = reinterpret_cast<const float*>(part[buf]);
        const int results = tw * RT * NT * 256;
        for (int o = threadIdx.x; o < results; o += kFewThreads) {
            // a vector's rows side by side, or a row's vectors
            const int v = Epilogue::kRowsFirst ? o / (16 * RT) % (16 * NT) : o % (16 * NT);
            const int r = Epilogue::kRowsFirst ? o % (16 * RT) + o / (256 * RT * NT) * (16 * RT)
                                               : o / (16 * NT);
            const int t = r / 16 % RT, of = r / (16 * RT) * kw;
            float c = 0;
            for (int k = 0; k < kw; ++k)
                c += sums[((((of + k) * RT + t) * NT + v / 16) * 16 + v % 16) * 16 + r % 16];
            if (v < a.count && row0 + r < a.rows) e.value(c, row0 + r, v);
        }
        buf ^= 1;                         // (the next turn's sums go where nobody reads)
    }
    e.end(reinterpret_cast<float*>(part), a.count);
}

template <class Src, int NT, int RT, class Epilogue>
hipError_t few(const FewArgs& a, const Epilogue& e, int most, hipStream_t s,
               int* workgroups = nullptr) {
    int kw = 1;
    while (kw < kFewWaves && kw * Src::kSteps * 32 < a.cols) kw *= 2;
    const int64_t groups = (a.rows + 16 * RT - 1) / (16 * RT);
    const int64_t tw = kFewWaves / kw;
    int64_t blocks = (groups + tw - 1) / tw;
    blocks = blocks < most ? blocks : most;
    if (workgroups != nullptr) *workgroups = static_cast<int>(blocks);
    k_few<Src, NT, RT, Epilogue><<<dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), 0, s>>>(
        a, e, kw);
    return hipGetLastError();
}

}  // namespace dlk
