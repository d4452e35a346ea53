// Root-mean-square norm with the residual's addition, and its gradients.
//
//   s = x + residual ; inv = 1/sqrt(mean s^2 + eps) ; y = (s inv) w
//   g = dy w ; h = s inv ; dx = inv (g - h mean(g h)) + dsum ; dw = sum dy h
//
// Forward, and backward for rows of up to 8192 columns, each element is read
// once and the row kept in registers, so these are bound by the bytes in and
// out.  A row is shared by 16, 64, 256 or 1024 lanes, each with up to four
// groups of eight neighbouring columns.  The workgroups walk over the rows, so
// that the weight is loaded, and dweight's part written, once for many of them.
//
// Measured (out of the caches; a large copy reaches 4.9 TB/s): 16384 x 2048 bf16
// with the residual's addition to e4m3 with row scales 50 us (4.7 TB/s), block
// scales 52 us; the same rows 2047 long, whose ends are single elements, to bf16
// 67 us (2048: 53 us); 8191 x 2048 bf16 forward 28 us, backward 34 us and
// dweight's sum 5 us; one row 2.5 us.  fp32 in and out 5.3 to 5.7 TB/s from 2048
// to 32768 columns, to e4m3 with block scales 4.2 to 5.1.
//
// Four groups a lane take all 128 registers: most e4m3 forms then, and some of
// 256 lanes to the other types, put up to 32 of them (12 to 72 bytes a lane) into
// scratch memory.  It shows most where the bytes are fewest: 47662 x 5632 bf16 to
// e4m3 with block scales 312 us (2.6 TB/s; to bf16 215 us, 5.0).
//
// What is rounded to 8 bits must not depend on an order of additions, so the
// mean of squares is summed in binary64 (at most 2^-40 off for any order) and
// everything after it is single binary32 operations.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "head.h"
#include "head_device.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

constexpr int kCols = 8;             // neighbouring columns a lane takes at once
constexpr int kMaxPartials = 1024;   // workgroups of the backward pass

// Lanes a row, and threads a workgroup.
template <int LANES> constexpr int threads_of() { return LANES > 256 ? LANES : 256; }

// A reduction over the LANES threads of a row; every one gets the result.
template <int LANES, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, Op op, T* lds) {
    if constexpr (LANES == 16) {
        return lanes_reduce<16>(v, op);
    } else {
        v = wave_reduce(v, op);
        if constexpr (LANES > kWave) {       // the row is the workgroup's
            constexpr int kWaves = LANES / kWave;
            __syncthreads();                 // an earlier result has been read
            if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
            __syncthreads();
            v = lds[0];
            for (int i = 1; i < kWaves; ++i) v = op(v, lds[i]);
        }
        return v;
    }
}

// Eight e4m3 codes.
__device__ __forceinline__ uint2 e4m3_of(const float* v) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
    return uint2{static_cast<uint32_t>(a), static_cast<uint32_t>(b)};
}

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ void store_codes(uint8_t* row, int c, int n, uint2 q) {
    if (c + kCols <= n) {
        *reinterpret_cast<u32x2_any*>(row + c) = u32x2_any{q.x, q.y};
    } else if (c < n) {
        const int left = n - c;
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

// OUT: element type of y; KIND: its scales.
template <typename T, int OUT, int KIND, int LANES, int NV>
__global__ __launch_bounds__(threads_of<LANES>(), 4) void k_rmsnorm(NormArgs a) {
    constexpr int kThreads = threads_of<LANES>();
    constexpr int kRows = kThreads / LANES;              // rows at a time
    __shared__ double lds_d[LANES > kWave ? LANES / kWave : 1];
    __shared__ uint32_t lds_u[LANES > kWave ? LANES / kWave : 1];
    const int lane = threadIdx.x % LANES;
    float w[NV][kCols];
    for (int i = 0; i < NV; ++i) load8(a.weight, (i * LANES + lane) * kCols, a.cols, w[i]);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / LANES; row < a.rows;
         row += step) {
        float s[NV][kCols];
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        for (int i = 0; i < NV; ++i) load8(x, (i * LANES + lane) * kCols, a.cols, s[i]);
        if (a.residual != nullptr) {
            const T* r = static_cast<const T*>(a.residual) + row * a.ldres;
            float t[NV][kCols];
            for (int i = 0; i < NV; ++i) load8(r, (i * LANES + lane) * kCols, a.cols, t[i]);
            for (int i = 0; i < NV; ++i)
                for (int k = 0; k < kCols; ++k) s[i][k] = to_f32(from_f32<T>(s[i][k] + t[i][k]));
            if (a.sum != nullptr)
                for (int i = 0; i < NV; ++i)
                    store8(static_cast<T*>(a.sum) + row * a.ldsum, (i * LANES + lane) * kCols, a.cols,
                           s[i]);
        }
        double ss = 0;
        for (int i = 0; i < NV; ++i)
            for (int k = 0; k < kCols; ++k) {
                const double d = s[i][k];
                ss = __builtin_fma(d, d, ss);
            }
        ss = row_reduce<LANES>(ss, Sum{}, lds_d);
        const float inv = static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
        if (a.inv_rms != nullptr && lane == 0) a.inv_rms[row] = inv;
        // y in place of s; columns past the end stay 0 unless inv is infinite
        uint32_t amax = 0;
        for (int i = 0; i < NV; ++i)
            for (int k = 0; k < kCols; ++k) {
                s[i][k] = (s[i][k] * inv) * w[i][k];
                if constexpr (KIND != DL_SCALE_NONE)
                    if ((i * LANES + lane) * kCols + k >= a.cols) s[i][k] = 0.0f;
                if constexpr (KIND == DL_SCALE_ROW) amax = Max{}(amax, abs_bits(s[i][k]));
            }
        if constexpr (KIND == DL_SCALE_ROW) {
            amax = row_reduce<LANES>(amax, Max{}, lds_u);
            const float m = __uint_as_float(amax);
            float scale = 0.0f, back = 0.0f;             // below 2^-100: zeros
            if (amax >= 0x7F800000u) {
                scale = __uint_as_float(0x7FC00000u);
            } else if (m >= 0x1p-100f) {
                scale = m / 448.0f;
                back = 448.0f / m;
            }
            if (lane == 0) static_cast<float*>(a.scales)[row] = scale;
            for (int i = 0; i < NV; ++i) {
                for (int k = 0; k < kCols; ++k) s[i][k] = back == 0.0f ? 0.0f : s[i][k] * back;
                store_codes(static_cast<uint8_t*>(a.y) + row * a.ldy, (i * LANES + lane) * kCols,
                            a.cols, e4m3_of(s[i]));
            }
        } else if constexpr (KIND == DL_SCALE_BLOCK32) {
            const int64_t kb = (a.cols + 31) / 32;
            for (int i = 0; i < NV; ++i) {
                const int c = (i * LANES + lane) * kCols;
                uint32_t b = 0;
                for (int k = 0; k < kCols; ++k) b = Max{}(b, abs_bits(s[i][k]));
                b = lanes_reduce<4>(b, Max{});           // the 32 columns' four lanes
                // the smallest power of two p with amax <= 448 p = 1.75 * 2^8 p
                int e = static_cast<int>((b + 0x1FFFFFu) >> 23) - 8;
                e = e < 0 ? 0 : e;
                const bool bad = b >= 0x7F800000u;
                const float back = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                for (int k = 0; k < kCols; ++k) s[i][k] = bad ? 0.0f : s[i][k] * back;
                if (lane % 4 == 0 && c < a.cols)
                    static_cast<uint8_t*>(a.scales)[row * kb + c / 32] =
                        static_cast<uint8_t>(bad ? 255 : e);
                store_codes(static_cast<uint8_t*>(a.y) + row * a.ldy, c, a.cols, e4m3_of(s[i]));
            }
        } else if constexpr (OUT == DL_F32) {
            for (int i = 0; i < NV; ++i)
                store8(static_cast<float*>(a.y) + row * a.ldy, (i * LANES + lane) * kCols, a.cols,
                       s[i]);
        } else {
            for (int i = 0; i < NV; ++i)
                store8(static_cast<bf16*>(a.y) + row * a.ldy, (i * LANES + lane) * kCols, a.cols,
                       s[i]);
        }
    }
}

// dx of the rows, and this workgroup's part of dweight.  With HOLD the row
// stays in registers between the sum and its use; rows past 8192 columns (1024
// lanes of 128 registers each) are read again instead: 8192 x 16384 fp32 391 us
// (4.1 TB/s of the bytes that one read and one write take), and past 16384
// columns, where dweight's sums spill too (some 450 bytes a lane), 4096 x 32768
// 553 us (2.9 TB/s; 16384 x 8192, held: 300 us, 5.4).
template <typename T, int LANES, int NV, bool HOLD>
__global__ __launch_bounds__(threads_of<LANES>()) void k_rmsnorm_backward(NormBackwardArgs a) {
    constexpr int kThreads = threads_of<LANES>();
    constexpr int kRows = kThreads / LANES;
    __shared__ float lds[LANES > kWave ? LANES / kWave : 1];
    __shared__ float parts[kRows > 1 ? kThreads : 1][kCols];
    const int lane = threadIdx.x % LANES;
    float dw[NV][kCols] = {};
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    // Every lane takes part in every turn: a row past the end is all zeros.
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + threadIdx.x / LANES;
        const bool here = row < a.rows;
        const int n = here ? a.cols : 0;
        const int64_t at = here ? row : 0;
        const T* dy = static_cast<const T*>(a.dy) + at * a.lddy;
        const T* sum = static_cast<const T*>(a.sum) + at * a.ldsum;
        const float inv = a.inv_rms[at];
        float y[HOLD ? NV : 1][kCols], s[HOLD ? NV : 1][kCols];
        float c = 0;
        if constexpr (HOLD)
            for (int i = 0; i < NV; ++i) {
                const int col = (i * LANES + lane) * kCols;
                load8(dy, col, n, y[i]);
                load8(sum, col, n, s[i]);
            }
        for (int i = 0; i < NV; ++i) {
            const int q = HOLD ? i : 0, col = (i * LANES + lane) * kCols;
            if constexpr (!HOLD) {
                load8(dy, col, n, y[q]);
                load8(sum, col, n, s[q]);
            }
            float w[kCols];
            load8(a.weight, col, a.cols, w);
            for (int k = 0; k < kCols; ++k) c += (y[q][k] * w[k]) * (s[q][k] * inv);
        }
        c = row_reduce<LANES>(c, Sum{}, lds) / static_cast<float>(a.cols);
        for (int i = 0; i < NV; ++i) {
            const int q = HOLD ? i : 0, col = (i * LANES + lane) * kCols;
            if constexpr (!HOLD) {
                load8(dy, col, n, y[q]);
                load8(sum, col, n, s[q]);
            }
            float w[kCols], d[kCols] = {};
            load8(a.weight, col, a.cols, w);
            if (a.dsum != nullptr)
                load8(static_cast<const T*>(a.dsum) + at * a.lddsum, col, n, d);
            for (int k = 0; k < kCols; ++k) {
                const float h = s[q][k] * inv;
                // (a term of nothing would be NaN where inv is infinite)
                if (col + k < n) dw[i][k] += y[q][k] * h;
                const float g = inv * (y[q][k] * w[k] - h * c);
                d[k] = a.dsum != nullptr ? g + d[k] : g;
            }
            store8(static_cast<T*>(a.dx) + at * a.lddx, col, n, d);
        }
    }
    if (a.dweight == nullptr) return;
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    for (int i = 0; i < NV; ++i) {
        const int col = (i * LANES + lane) * kCols;
        if constexpr (kRows > 1) {                       // the rows of one turn, in order
            __syncthreads();
            for (int k = 0; k < kCols; ++k) parts[threadIdx.x][k] = dw[i][k];
            __syncthreads();
            if (threadIdx.x < LANES)
                for (int r = 1; r < kRows; ++r)
                    for (int k = 0; k < kCols; ++k) dw[i][k] += parts[threadIdx.x + r * LANES][k];
        }
        if (threadIdx.x < LANES) store8(out, col, a.cols, dw[i]);
    }
}

// dweight from the workgroups' parts: 16 columns a workgroup, whose 64 groups
// of 16 threads take every 64th part.  A chain of loads and little else, so many
// threads share it (1024 parts of 128 columns: 3.6 us, 4.4 us with 64 columns and
// 16 groups a workgroup; of 2048 columns 5 us either way).
constexpr int kSumCols = 16, kSumGroups = 64;

__global__ __launch_bounds__(kSumCols * kSumGroups) void k_rmsnorm_dw(const float* partial,
                                                                      int parts, int cols,
                                                                      float* dweight) {
    __shared__ float lds[kSumGroups][kSumCols];
    const int g = threadIdx.x / kSumCols, k = threadIdx.x % kSumCols;
    const int c = blockIdx.x * kSumCols + k;
    float t = 0;
    if (c < cols) {
#pragma unroll 8
        for (int p = g; p < parts; p += kSumGroups) t += partial[static_cast<int64_t>(p) * cols + c];
    }
    for (int n = kSumGroups; n > 1; n /= 8) {             // eight groups' sums into one, in order
        lds[g][k] = t;
        __syncthreads();
        if (g < n / 8) {
            t = lds[8 * g][k];
            for (int i = 1; i < 8; ++i) t += lds[8 * g + i][k];
        }
        __syncthreads();
    }
    if (g == 0 && c < cols) dweight[c] = t;
}

// Lanes a row and groups of eight columns a lane.
struct Shape {
    int lanes, groups;
};

// Forward: the fewest lanes that hold the row in four groups, as a wave needs
// no barrier (16384 x 2048 bf16 to e4m3 with row scales: 50 us, 59 us with 256
// lanes a row).  Few rows take more lanes, as one row's time is then all there
// is.
Shape forward_shape(int64_t rows, int cols) {
    int lanes = cols <= 512 ? 16 : cols <= 2048 ? 64 : cols <= 8192 ? 256 : 1024;
    if (rows <= 256 && lanes < 256 && cols > 512) lanes = 256;
    const int groups = (cols + lanes * kCols - 1) / (lanes * kCols);
    return Shape{lanes, groups <= 1 ? 1 : groups <= 2 ? 2 : 4};
}

// Backward: one group a lane, which leaves registers for more waves (8191 x
// 2048 bf16: 34 us, 45 us with 64 lanes of four groups).
Shape backward_shape(int cols) {
    const int lanes = cols <= 128 ? 16 : cols <= 512 ? 64 : cols <= 2048 ? 256 : 1024;
    const int groups = (cols + lanes * kCols - 1) / (lanes * kCols);
    return Shape{lanes, groups <= 1 ? 1 : groups <= 2 ? 2 : 4};
}

template <int N> struct Int {
    static constexpr int value = N;
};

// Workgroups of the forward pass: enough to fill the GPU, and several rows each.
constexpr int64_t kMaxBlocks = 2048;

template <typename T, int OUT, int KIND> hipError_t forward(const NormArgs& a, hipStream_t s) {
    const Shape shape = forward_shape(a.rows, a.cols);
    auto launch = [&](auto lanes, auto groups) {
        constexpr int kLanes = decltype(lanes)::value;
        constexpr int kRows = threads_of<kLanes>() / kLanes;
        int64_t blocks = (a.rows + kRows - 1) / kRows;
        blocks = blocks < kMaxBlocks ? blocks : kMaxBlocks;
        k_rmsnorm<T, OUT, KIND, kLanes, decltype(groups)::value>
            <<<dim3(static_cast<unsigned>(blocks)), dim3(threads_of<kLanes>()), 0, s>>>(a);
        return hipGetLastError();
    };
    // (64 lanes come with 513 columns or more, 1024 with 8193, so with two groups at least)
    auto of_groups = [&](auto lanes) {
        if constexpr (decltype(lanes)::value == 16 || decltype(lanes)::value == 256)
            if (shape.groups == 1) return launch(lanes, Int<1>{});
        return shape.groups <= 2 ? launch(lanes, Int<2>{}) : launch(lanes, Int<4>{});
    };
    return shape.lanes == 16 ? of_groups(Int<16>{})
           : shape.lanes == 64 ? of_groups(Int<64>{})
           : shape.lanes == 256 ? of_groups(Int<256>{}) : of_groups(Int<1024>{});
}

template <typename T>
hipError_t forward_to(const NormArgs& a, int y_dtype, int kind, hipStream_t s) {
    if (kind == DL_SCALE_ROW) return forward<T, DL_E4M3, DL_SCALE_ROW>(a, s);
    if (kind == DL_SCALE_BLOCK32) return forward<T, DL_E4M3, DL_SCALE_BLOCK32>(a, s);
    return y_dtype == DL_F32 ? forward<T, DL_F32, DL_SCALE_NONE>(a, s)
                             : forward<T, DL_BF16, DL_SCALE_NONE>(a, s);
}

int64_t backward_blocks(int64_t rows, int cols) {
    const int lanes = backward_shape(cols).lanes;
    const int at_a_time = lanes < 256 ? 256 / lanes : 1;
    const int64_t blocks = (rows + at_a_time - 1) / at_a_time;
    const int64_t most = lanes > 256 ? kMaxPartials / 2 : kMaxPartials;
    return blocks < most ? blocks : most;
}

template <typename T> hipError_t backward(const NormBackwardArgs& a, hipStream_t s) {
    const Shape shape = backward_shape(a.cols);
    auto launch = [&](auto lanes, auto groups) {
        constexpr int kLanes = decltype(lanes)::value, kGroups = decltype(groups)::value;
        const int64_t blocks = backward_blocks(a.rows, a.cols);
        k_rmsnorm_backward<T, kLanes, kGroups, kGroups == 1>
            <<<dim3(static_cast<unsigned>(blocks)), dim3(threads_of<kLanes>()), 0, s>>>(a);
        return hipGetLastError();
    };
    return shape.lanes == 16 ? launch(Int<16>{}, Int<1>{})
           : shape.lanes == 64 ? launch(Int<64>{}, Int<1>{})
           : shape.lanes == 256 ? launch(Int<256>{}, Int<1>{})
           : shape.groups == 1 ? launch(Int<1024>{}, Int<1>{})
           : shape.groups == 2 ? launch(Int<1024>{}, Int<2>{}) : launch(Int<1024>{}, Int<4>{});
}

}  // namespace

hipError_t rmsnorm(const NormArgs& a, int dtype, int y_dtype, int scale_kind, hipStream_t s) {
    return dtype == DL_F32 ? forward_to<float>(a, y_dtype, scale_kind, s)
                           : forward_to<bf16>(a, y_dtype, scale_kind, s);
}

int64_t rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
    return rows == 0 ? 0 : backward_blocks(rows, static_cast<int>(cols)) * cols * 4;
}

hipError_t rmsnorm_backward(const NormBackwardArgs& a, int dtype, hipStream_t s) {
    int64_t parts = 0;
    if (a.rows > 0) {
        const hipError_t e = dtype == DL_F32 ? backward<float>(a, s) : backward<bf16>(a, s);
        if (e != hipSuccess) return e;
        parts = backward_blocks(a.rows, a.cols);
    }
    if (a.dweight == nullptr) return hipSuccess;
    k_rmsnorm_dw<<<dim3(static_cast<unsigned>((a.cols + kSumCols - 1) / kSumCols)),
                   dim3(kSumCols * kSumGroups), 0, s>>>(a.partial, static_cast<int>(parts), a.cols,
                                                        a.dweight);
    return hipGetLastError();
}

}  // namespace dlk
