// A tiled matrix product on the matrix cores, shared by the output head's
// kernels over many tokens (headloss.hip, e4m3.hip):
//
//   C[n][m] = sum over k of A(m, k) B(n, k),    m < M, n < N, k < K
//
// with the tile of sums handed to an epilogue while it is in registers.
//
// A workgroup of eight waves keeps TM x TN sums in registers and steps along k
// by 128 bytes of an operand's row: the next step's 16-byte pieces are under
// way from memory to registers while this step's products run, and are put
// into the other one of two LDS buffers halfway through them, so that a step
// costs one barrier and no wait for memory that its products do not cover.  The
// pipeline runs on across tiles: a tile's epilogue has the next tile's first
// step in LDS and its second under way.
//
// An operand's rows are along k in memory (ACROSS false) or across it (true: k
// is the slow index, and the LDS reads transpose).  Elements go through as they
// are (bf16, e4m3 codes), or, from binary32, as three bf16 numbers whose sum
// they are (each the rest rounded: 2^-9 and 2^-18 of the whole are left): of the
// nine products of two such triples the three of at most 2^-27 of the whole are
// left out, which all together is less than a rounding of it, and the other six
// take six times bf16's time (a binary32 matrix instruction: sixteen times).
//
// LDS holds 16-byte pieces at places permuted by exclusive or, so that eight
// lanes' reads (and sixteen lanes' transposing ones) meet all banks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.h"

namespace dlk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;
constexpr int kStepBytes = 128;          // of an operand's row, a step

struct ProductArgs {
    const void* a;
    int64_t lda;
    const void* b;
    int64_t ldb;
    int64_t m, n, k;
    int slices;                          // parts of k, each with sums of its own
    const int* count;                    // or nullptr: the number of rows that n (or k) stands for
    bool count_is_k;
};

// ---- from memory to registers to LDS -----------------------------------------

// 16 bytes of a row, at any element.
template <typename T> struct Raw;
template <> struct Raw<float> {
    typedef uint32_t any __attribute__((ext_vector_type(4), aligned(4)));
};
template <> struct Raw<bf16> {
    typedef uint32_t any __attribute__((ext_vector_type(4), aligned(2)));
};
template <> struct Raw<uint8_t> {
    typedef uint32_t any __attribute__((ext_vector_type(4), aligned(1)));
};

// What the matrix instructions are fed with.
struct ViaBf16 {                         // bf16 as they are
    typedef bf16 elem;
    static constexpr int kPlanes = 1;
};
struct ViaSplit {                        // binary32 as three bf16 numbers
    typedef float elem;
    static constexpr int kPlanes = 3;
};
struct ViaCodes {                        // e4m3 codes
    typedef uint8_t elem;
    static constexpr int kPlanes = 1;
};

// One operand's side of a step: ROWS rows (m or n) by kStep elements of k.
// FIRST: operand A, whose rows a lane's sums run along (see a_row below).
template <class Via, bool ACROSS, int ROWS, bool FIRST> struct Side {
    typedef typename Via::elem T;
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    static constexpr int kStep = kStepBytes / static_cast<int>(sizeof(T));
    static constexpr int kLine = (ACROSS ? ROWS : kStep) / kPer;     // pieces in a line of memory
    static constexpr int kLines = ACROSS ? kStep : ROWS;
    static constexpr int kMine = kLine * kLines / kTileThreads;
    static constexpr int kApart = kTileThreads / kLine;              // lines between a thread's
    static constexpr int kHeld = Via::kPlanes == 3 ? 2 : static_cast<int>(sizeof(T));
    static constexpr int kRowBytes = (ACROSS ? ROWS : kStep) * kHeld;
    static constexpr int kPlaneBytes = kRowBytes * kLines;
    static constexpr int kBytes = kPlaneBytes * Via::kPlanes;
    static_assert(kMine >= 1 && kMine * kTileThreads == kLine * kLines, "");

    u32x4 v[kMine];

    // Rows row0 .. row0 + ROWS - 1 and k from k0 on; 0 outside rows < rows, k < k1.
    __device__ __forceinline__ void load(const void* p, int64_t ld, int64_t row0, int64_t rows,
                                         int64_t k0, int64_t k1) {
        const int c = threadIdx.x % kLine * kPer, l = threadIdx.x / kLine;
        const int64_t lines = ACROSS ? k1 - k0 : rows - row0;
        const int64_t wide = ACROSS ? rows - row0 : k1 - k0;
        const T* at = static_cast<const T*>(p) + (ACROSS ? k0 * ld + row0 : row0 * ld + k0) +
                      l * ld + c;
        if (lines >= kLines && wide >= kLine * kPer) {
            for (int j = 0; j < kMine; ++j)
                v[j] = *reinterpret_cast<const typename Raw<T>::any*>(at + j * (kApart * ld));
        } else {
            for (int j = 0; j < kMine; ++j) {
                const T* q = at + j * (kApart * ld);
                v[j] = u32x4{};
                if (l + j * kApart >= lines) continue;
                if (c + kPer <= wide) {
                    v[j] = *reinterpret_cast<const typename Raw<T>::any*>(q);
                } else if (c < wide) {
                    T t[kPer] = {};
                    for (int i = 0; i < kPer; ++i)
                        if (c + i < wide) t[i] = q[i];
                    __builtin_memcpy(&v[j], t, 16);
                }
            }
        }
    }

    // The 16-byte piece of row `row` that holds its piece c is at piece c ^ key(row).
    // Eight lanes read the same piece of eight rows: neighbouring ones, or for A rows
    // 0 1 2 3 8 9 10 11 of each 16.
    static __device__ __forceinline__ int key(int row) {
        if constexpr (kRowBytes == 128)
            return FIRST ? (row & 3) | ((row >> 1) & 4) : row & 7;
        else
            return FIRST ? ((row >> 1) & 1) | ((row >> 2) & 2) : (row >> 1) & 3;
    }
    // Across k, four lines of 64 (A) or 32 (B) bytes are read together.
    static __device__ __forceinline__ int key_across(int k) { return (k & 3) << (FIRST ? 6 : 5); }

    __device__ __forceinline__ void put(uint8_t* lds) const {
        const int c = threadIdx.x % kLine, l = threadIdx.x / kLine;
        for (int j = 0; j < kMine; ++j) {
            const int line = l + j * kApart;
            if constexpr (Via::kPlanes == 1) {
                const int at = line * kRowBytes +
                               (ACROSS ? (c * 16) ^ key_across(line) : (c ^ key(line)) * 16);
                *reinterpret_cast<u32x4*>(lds + at) = v[j];
            } else {
                const int at = line * kRowBytes +
                               (ACROSS ? (c * 8) ^ key_across(line)
                                       : ((c >> 1) ^ key(line)) * 16 + (c & 1) * 8);
                uint32_t q[3][2];
                for (int i = 0; i < 2; ++i) {
                    float x = __uint_as_float(v[j][2 * i]), y = __uint_as_float(v[j][2 * i + 1]);
                    for (int p = 0; p < 3; ++p) {
                        typedef float f32x2 __attribute__((ext_vector_type(2)));
                        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                        q[p][i] = __builtin_bit_cast(
                            uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
                        x -= __uint_as_float(q[p][i] << 16);
                        y -= __uint_as_float(q[p][i] & 0xFFFF0000u);
                    }
                }
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<u32x2*>(lds + p * kPlaneBytes + at) = u32x2{q[p][0], q[p][1]};
            }
        }
    }

    // The first operand's rows in the order that leaves a lane eight neighbouring sums of a
    // pair of tiles: row r of tile t is row 32 (t/2) + 8 (r/4) + 4 (t%2) + r%4 of the wave's.
    static __device__ __forceinline__ int a_row(int t, int r) {
        return 32 * (t / 2) + 8 * (r / 4) + 4 * (t % 2) + r % 4;
    }

    // 8 elements of k for each lane: row `lane % 16` of 16-row tile t of the rows from row0
    // on, k = 32 sub + 8 (lane / 16) .. + 7.
    static __device__ __forceinline__ bf16x8 frag(const uint8_t* lds, int row0, int t, int sub) {
        const int r = threadIdx.x % 16, g = threadIdx.x / 16 % 4;
        if constexpr (!ACROSS) {
            const int row = row0 + (FIRST ? a_row(t, r) : t * 16 + r);
            return *reinterpret_cast<const bf16x8*>(lds + row * kRowBytes +
                                                    ((sub * 4 + g) ^ key(row)) * 16);
        } else {
            // (lane 4 i + j of 16 gives the place of columns 4 j .. 4 j + 3 of line i, and gets
            // column 4 i + j of the four lines)
            const int row = row0 + (FIRST ? a_row(t, 4 * (r % 4)) : t * 16 + 4 * (r % 4));
            const int k = 32 * sub + 8 * g + r / 4;
            const int at = k * kRowBytes + ((row * 2) ^ key_across(k));
            typedef __attribute__((address_space(3))) i16x4 lds4;
            union {
                i16x4 h[2];
                bf16x8 all;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(lds + at));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(lds + at + 4 * kRowBytes));
            return u.all;
        }
    }

    // 16 codes for each lane: pieces 4 half + (lane / 16) of its row.
    static __device__ __forceinline__ u32x4 codes(const uint8_t* lds, int row0, int t, int half) {
        const int r = threadIdx.x % 16, g = threadIdx.x / 16 % 4;
        const int row = row0 + (FIRST ? a_row(t, r) : t * 16 + r);
        return *reinterpret_cast<const u32x4*>(lds + row * kRowBytes +
                                               ((half * 4 + g) ^ key(row)) * 16);
    }
};

// ---- the order of the tiles --------------------------------------------------

// Workgroups are dealt to the eight XCDs in turn.  Each XCD takes a run of
// neighbouring items, whose operands its L2 then holds once: bands of up to
// eight tiles of the shorter side, walked along the longer one.
struct Items {
    int64_t m_tiles, n_tiles, tiles, end, at, step;

    __device__ Items(int64_t m, int64_t n, int tm, int tn, int slices) {
        m_tiles = (m + tm - 1) / tm;
        n_tiles = (n + tn - 1) / tn;
        tiles = m_tiles * n_tiles;
        const int64_t all = tiles * slices;
        const int64_t run = (all + 7) / 8, x = blockIdx.x % 8;
        step = gridDim.x / 8;
        end = run * (x + 1) < all ? run * (x + 1) : all;
        at = run * x + blockIdx.x / 8;
    }
    __device__ bool left() const { return at < end; }
    __device__ void next() { at += step; }
    __device__ void place(int64_t* mt, int64_t* nt, int* slice) const {
        *slice = static_cast<int>(at / tiles);
        const int64_t t = at % tiles;
        const bool n_short = n_tiles <= m_tiles;
        const int64_t few = n_short ? n_tiles : m_tiles, many = n_short ? m_tiles : n_tiles;
        const int64_t band = t / (8 * many), in = t % (8 * many);
        const int64_t wide = few - band * 8 < 8 ? few - band * 8 : 8;
        const int64_t s = band * 8 + in % wide, l = in / wide;
        *mt = n_short ? l : s;
        *nt = n_short ? s : l;
    }
};

constexpr int kTileGroups = 256;          // one workgroup a CU

inline unsigned product_grid(int64_t m, int64_t n, int tm, int tn, int slices, int groups) {
    const int64_t all = ((m + tm - 1) / tm) * ((n + tn - 1) / tn) * slices;
    const int64_t up = (all + 7) / 8 * 8;
    return static_cast<unsigned>(up < groups ? (up < 8 ? 8 : up) : groups);
}

// ---- the product -------------------------------------------------------------

// Where a wave's sums are: element i of acc[t][u] is C[n][m] with
//   m = m0 + 32 (t/2) + 8 (lane/16) + 4 (t%2) + i,   n = n0 + 16 u + lane%16.
struct Place {
    int64_t m0, n0;                       // of the wave
    int64_t m, n;                         // ends of the product
    int slice;
};

template <class Via, bool SA, bool SB, int TM, int TN, int WM, int WN, class Epilogue>
__global__ __launch_bounds__(kTileThreads, 2) void k_product(ProductArgs a, Epilogue e) {
    static_assert(WM * WN == kTileWaves, "");
    constexpr int kMT = TM / WM / 16, kNT = TN / WN / 16;
    typedef Side<Via, SA, TM, true> SideA;
    typedef Side<Via, SB, TN, false> SideB;
    constexpr int kStep = SideA::kStep;
    __shared__ __attribute__((aligned(128))) uint8_t lds[2][SideA::kBytes + SideB::kBytes];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN * (TM / WM), wn = wave % WN * (TN / WN);
    if (a.count != nullptr) (a.count_is_k ? a.k : a.n) = *a.count;
    const int64_t per_slice = ((a.k + a.slices - 1) / a.slices + kStep - 1) / kStep * kStep;

    struct Cursor {
        Items items;
        int64_t mt, nt, k0, k1;
        int slice;
    };
    auto enter = [&](Cursor& c) {
        if (!c.items.left()) return;
        c.items.place(&c.mt, &c.nt, &c.slice);
        c.k0 = c.slice * per_slice;
        c.k1 = c.k0 + per_slice < a.k ? c.k0 + per_slice : a.k;
    };
    Cursor in{Items(a.m, a.n, TM, TN, a.slices), 0, 0, 0, 0, 0};
    enter(in);
    Cursor out = in;
    SideA sa;
    SideB sb;
    // The step at `in` into registers; then on to the next one.
    bool held = false;
    auto fetch = [&] {
        held = in.items.left();
        if (!held) return;
        sa.load(a.a, a.lda, in.mt * TM, a.m, in.k0, in.k1);
        sb.load(a.b, a.ldb, in.nt * TN, a.n, in.k0, in.k1);
        in.k0 += kStep;
        if (in.k0 >= in.k1) {
            in.items.next();
            enter(in);
        }
    };
    auto put = [&](uint8_t* to) {
        if (!held) return;
        sa.put(to);
        sb.put(to + SideA::kBytes);
    };
    int buf = 0;
    fetch();
    put(lds[0]);
    fetch();
    __syncthreads();
    while (out.items.left()) {
        f32x4 acc[kMT][kNT] = {};
        typename Epilogue::template Steps<kNT> steps;
        const Place at{out.mt * TM + wm, out.nt * TN + wn, a.m, a.n, out.slice};
        steps.enter(e, at, out.k0);
        do {
            const uint8_t* la = lds[buf];
            const uint8_t* lb = la + SideA::kBytes;
            if constexpr (Via::kPlanes == 3) {
                bf16x8 vb[3][kNT];
                for (int p = 0; p < 3; ++p)
                    for (int u = 0; u < kNT; ++u)
                        vb[p][u] = SideB::frag(lb + p * SideB::kPlaneBytes, wn, u, 0);
#pragma unroll
                for (int t = 0; t < kMT; ++t) {
                    if (t == kMT / 2) {
                        put(lds[buf ^ 1]);
                        fetch();
                    }
                    bf16x8 va[3];
                    for (int p = 0; p < 3; ++p)
                        va[p] = SideA::frag(la + p * SideA::kPlaneBytes, wm, t, 0);
                    // the smallest products first
                    constexpr int pa[6] = {0, 2, 1, 0, 1, 0}, pb[6] = {2, 0, 1, 1, 0, 0};
                    for (int q = 0; q < 6; ++q)
                        for (int u = 0; u < kNT; ++u)
                            acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                va[pa[q]], vb[pb[q]][u], acc[t][u], 0, 0, 0);
                }
            } else if constexpr (sizeof(typename Via::elem) == 2) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s == 1) {
                        put(lds[buf ^ 1]);
                        fetch();
                    }
                    bf16x8 vb[kNT];
                    for (int u = 0; u < kNT; ++u) vb[u] = SideB::frag(lb, wn, u, s);
#pragma unroll
                    for (int t = 0; t < kMT; ++t) {
                        const bf16x8 va = SideA::frag(la, wm, t, s);
                        for (int u = 0; u < kNT; ++u)
                            acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, vb[u],
                                                                                acc[t][u], 0, 0, 0);
                    }
                }
            } else {
                steps.template product<SideA, SideB, kMT>(la, lb, wm, wn, acc, [&] {
                    put(lds[buf ^ 1]);
                    fetch();
                });
            }
            __syncthreads();
            buf ^= 1;
            out.k0 += kStep;
        } while (out.k0 < out.k1);
        e.template finish<kMT, kNT>(acc, at);
        out.items.next();
        enter(out);
    }
}

// An epilogue whose operands need nothing at each step.
struct NoSteps {
    template <int NT> struct Steps {
        template <class E> __device__ void enter(const E&, const Place&, int64_t) {}
    };
};

// The eight neighbouring sums of pair p of tiles.
template <int MT, int NT>
__device__ __forceinline__ void eight(const f32x4 (&acc)[MT][NT], int p, int u, float* v) {
    for (int i = 0; i < 4; ++i) {
        v[i] = acc[2 * p][u][i];
        v[4 + i] = acc[2 * p + 1][u][i];
    }
}

// C written out, a row of M for each n.
template <typename Y> struct StoreTile : NoSteps {
    Y* y;
    int64_t ld;
    StoreTile(void* to, int64_t l) : y(static_cast<Y*>(to)), ld(l) {}
    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x4 (&acc)[MT][NT], const Place& at) const {
        const int lane = threadIdx.x % kWave;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int64_t n = at.n0 + u * 16 + lane % 16;
            if (n >= at.n) continue;
            for (int p = 0; p < MT / 2; ++p) {
                float v[8];
                eight(acc, p, u, v);
                store8(y + n * ld, at.m0 + p * 32 + lane / 16 * 8, at.m, v);
            }
        }
    }
};

}  // namespace dlk
