// A tiled matrix product on the matrix cores, shared by the output head's
// kernels over many tokens (headloss.hip, e4m3.hip):
//
//   C[n][m] = sum over k of A(m, k) B(n, k),    m < M, n < N, k < K
//
// with the tile of sums handed to an epilogue while it is in registers.  A
// workgroup of eight waves keeps TM x TN sums (32 x 32 for each matrix
// instruction) and steps along k; its way through its tiles is one pipeline, so
// that a tile's epilogue has the next tile's first steps under way.
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

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;
constexpr int kSquare = 32;              // rows and columns of a matrix instruction's result

struct ProductArgs {
    const void* a;
    int64_t lda;
    const void* b;
    int64_t ldb;
    int64_t m, n, k;
    int slices;                          // parts of k, each with sums of its own
    const int* count;                    // or nullptr: the number of rows that n (or k) stands for
    bool count_is_k;
    int items, most;                     // or 0: cut by cut_of into these, for that number
};

// Parts of k for a product of `tiles` tiles of 256 x 256, `most` at most, so that there are as
// many as `items` of them in all.
__host__ __device__ inline int cut_of(int64_t tiles, int items, int most) {
    const int64_t n = items / (tiles > 1 ? tiles : 1);
    return static_cast<int>(n < 1 ? 1 : n > most ? most : n);
}
// At least 256 of k in each, and no more than the sums' memory is worth (20 rows x 50,304 x 128
// in fp32: 345 us with up to 16, 211 with 32, 150 with 64; 200 x 5000 x 256 in bf16, without the
// least length, 100, 101 and 110).
inline int most_of(int64_t k) { return static_cast<int>(k < 512 ? 1 : k / 256 > 64 ? 64 : k / 256); }
__host__ __device__ inline int64_t tiles_of(int64_t rows) { return (rows + 255) / 256; }

// ---- one operand -------------------------------------------------------------

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

// One operand's side of a step: ROWS rows (m or n) by STEP_BYTES of each along k.
// FIRST: operand A, whose rows a lane's sums run along (see m_row below; PAIRS: over two tiles).
template <class Via, bool ACROSS, int ROWS, bool FIRST, bool PAIRS, int STEP_BYTES> struct Side {
    typedef typename Via::elem T;
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    static constexpr int kStep = STEP_BYTES / static_cast<int>(sizeof(T));
    static constexpr int kLine = (ACROSS ? ROWS : kStep) / kPer;     // pieces in a line of memory
    static constexpr int kLines = ACROSS ? kStep : ROWS;
    static constexpr int kMine = kLine * kLines / kTileThreads;
    static constexpr int kApart = kTileThreads / kLine;              // lines between a thread's
    static constexpr int kHeld = Via::kPlanes == 3 ? 2 : static_cast<int>(sizeof(T));
    static constexpr int kRowBytes = (ACROSS ? ROWS : kStep) * kHeld;
    static constexpr int kPlaneBytes = kRowBytes * kLines;
    static constexpr int kBytes = kPlaneBytes * Via::kPlanes;
    static_assert(kMine >= 1 && kMine * kTileThreads == kLine * kLines, "");

    // ---- through registers: any alignment, any element type

    u32x4 v[kMine];
    const T* at;                                                     // this thread's first piece
    int64_t ld, apart, lines, wide;                                  // (of what is left from here)

    // Rows row0 .. row0 + ROWS - 1 of `rows`, and k from k0 up to k1.
    __device__ __forceinline__ void enter(const void* p, int64_t ld_, int64_t row0, int64_t rows,
                                          int64_t k0, int64_t k1) {
        const int c = threadIdx.x % kLine * kPer, l = threadIdx.x / kLine;
        ld = ld_;
        apart = kApart * ld;
        lines = ACROSS ? k1 - k0 : rows - row0;
        wide = ACROSS ? rows - row0 : k1 - k0;
        at = static_cast<const T*>(p) + (ACROSS ? k0 * ld + row0 : row0 * ld + k0) + l * ld + c;
    }
    // Whether all of the step's pieces are inside.
    __device__ __forceinline__ bool whole() const { return lines >= kLines && wide >= kLine * kPer; }
    __device__ __forceinline__ void load() {
        for (int j = 0; j < kMine; ++j)
            v[j] = *reinterpret_cast<const typename Raw<T>::any*>(at + j * apart);
    }
    // The pieces of a step that is not whole: 0 outside.
    __device__ __forceinline__ void load_some() {
        const int c = threadIdx.x % kLine * kPer, l = threadIdx.x / kLine;
        for (int j = 0; j < kMine; ++j) {
            const T* q = at + j * apart;
            v[j] = u32x4{};
            if (l + j * kApart >= lines) continue;
            if (c + kPer <= wide) {
                v[j] = *reinterpret_cast<const typename Raw<T>::any*>(q);
            } else if (c < wide) {
                const int n = static_cast<int>(wide) - c;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    constexpr int kIn = 4 / static_cast<int>(sizeof(T));
                    uint32_t e = 0;
                    __builtin_memcpy(&e, q + i, sizeof(T));
                    e <<= i % kIn * 8 * static_cast<int>(sizeof(T)) % 32;
                    for (int k = 0; k < 4; ++k) v[j][k] |= i / kIn == k ? e : 0;
                }
            }
        }
    }
    // On to the next step.
    __device__ __forceinline__ void onward() {
        at += ACROSS ? kStep * ld : kStep;
        (ACROSS ? lines : wide) -= kStep;
    }
    // The pieces p, which a step's load() left, to LDS.
    __device__ __forceinline__ void put(uint8_t* lds, const u32x4 (&p)[kMine]) const {
        for (int j = 0; j < kMine; ++j) put(lds, j, p[j]);
    }
    __device__ __forceinline__ void put(uint8_t* lds, int j, const u32x4& p) const {
        const int c = threadIdx.x % kLine, line = threadIdx.x / kLine + j * kApart;
        if constexpr (Via::kPlanes == 1) {
            const int to = line * kRowBytes +
                           (ACROSS ? (c * 16) ^ key_across(line) : (c ^ key(line)) * 16);
            *reinterpret_cast<u32x4*>(lds + to) = p;
        } else {
            const int to = line * kRowBytes +
                           (ACROSS ? (c * 8) ^ key_across(line)
                                   : ((c >> 1) ^ key(line)) * 16 + (c & 1) * 8);
            uint32_t q[3][2];
            for (int i = 0; i < 2; ++i) {
                float x = __uint_as_float(p[2 * i]), y = __uint_as_float(p[2 * i + 1]);
                for (int h = 0; h < 3; ++h) {
                    typedef float f32x2 __attribute__((ext_vector_type(2)));
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    q[h][i] = __builtin_bit_cast(
                        uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
                    x -= __uint_as_float(q[h][i] << 16);
                    y -= __uint_as_float(q[h][i] & 0xFFFF0000u);
                }
            }
            for (int h = 0; h < 3; ++h)
                *reinterpret_cast<u32x2*>(lds + h * kPlaneBytes + to) = u32x2{q[h][0], q[h][1]};
        }
    }

    // ---- straight into LDS: rows at multiples of 16 bytes, as far as `direct` below allows
    //
    // 64 lanes' pieces are neighbours in LDS: each lane asks for the piece that belongs in its
    // place.  The buffer's bounds turn what lies outside into zeros without a branch, at the
    // end of k by an offset past them; what a piece holds past the end of the other side
    // belongs to rows of the result that nobody looks at.
    struct Direct {
        const uint8_t *matrix, *base;     // base: of the step, the same for all lanes
        uint32_t offset[kMine];           // of this thread's pieces, in bytes
        int row_bytes;
        uint32_t bound;                   // bytes of all rows, or of a line that is across k
        int lines, wide;                  // what is left

        static __device__ __forceinline__ int piece() {
            const int c = threadIdx.x % kLine, l = threadIdx.x / kLine;
            static_assert(ACROSS ? kApart % 4 == 0 : kApart % 32 == 0, "one key for each j");
            return c ^ (ACROSS ? key_across(l) / 16 : key(l));
        }
        __device__ __forceinline__ void start(const void* p, int64_t ld) {
            matrix = base = static_cast<const uint8_t*>(p);
            bound = 0;
            row_bytes = static_cast<int>(ld * static_cast<int64_t>(sizeof(T)));
            for (int j = 0; j < kMine; ++j)
                offset[j] = (threadIdx.x / kLine + j * kApart) * static_cast<uint32_t>(row_bytes) +
                            piece() * 16;
        }
        __device__ __forceinline__ void enter(int64_t row0, int64_t rows, int64_t k0, int64_t k1) {
            const int64_t r = rows - row0 < ROWS ? rows - row0 : ROWS;
            const int64_t k = k1 > k0 ? k1 - k0 : 0;
            base = matrix +
                   (ACROSS ? k0 * row_bytes + row0 * static_cast<int64_t>(sizeof(T))
                           : row0 * row_bytes + k0 * static_cast<int64_t>(sizeof(T)));
            lines = static_cast<int>(ACROSS ? k : r);
            wide = static_cast<int>(k);
            // (a line's bytes, whole pieces, are at most row_bytes)
            bound = ACROSS ? static_cast<uint32_t>(r * static_cast<int64_t>(sizeof(T)) + 15) / 16 * 16
                           : static_cast<uint32_t>(r) * static_cast<uint32_t>(row_bytes);
        }
        // Nothing more to load: zeros from here on.
        __device__ __forceinline__ void stop() { lines = wide = 0; }
        __device__ __forceinline__ void load(uint8_t* lds, int wave) {
            typedef __attribute__((address_space(3))) void lds_any;
            uint8_t* to = lds + wave * (kWave * 16);
            // Bytes from the step's first to its last (along k, to the end of its last row: the
            // offsets see to the end of k).
            uint32_t bytes = bound;
            if constexpr (ACROSS) {
                const int n = __builtin_elementwise_min(lines, kLines);
                bytes = n > 0 ? (n - 1) * row_bytes + bound : 0;
            }
            __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(base), 0, bytes, 0x00020000);
            for (int j = 0; j < kMine; ++j) {
                uint32_t o = offset[j];
                if constexpr (!ACROSS) o = piece() * kPer < wide ? o : 0xFFFFFFF0u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_any*)(to + j * (kTileThreads * 16)),
                                                         16, o, 0, 0, 0);
            }
            base += ACROSS ? kStep * static_cast<int64_t>(row_bytes)
                           : kStep * static_cast<int64_t>(sizeof(T));
            if (ACROSS) lines -= kStep;
            else wide -= kStep;
        }
    };

    // ---- in LDS

    // The 16-byte piece of row `row` that holds its piece c is at piece c ^ key(row).  A
    // 128-bit read takes 16 lanes at a time, 0-3 12-15 20-23 24-27 and 4-7 8-11 16-19 28-31 of
    // each 32: with the keys, and with A's orders of rows too, they meet 64 different banks.
    static __device__ __forceinline__ int key(int row) {
        const int four = FIRST && PAIRS ? row >> 2 & 3 : row >> 3 & 3;
        return kRowBytes == 128 ? (row >> 1 & 1) | four << 1 : four;
    }
    // Across k, 32 lanes read 8 bytes of four lines, two halves of a 64-byte window in each, or
    // with PAIRS two of 32 bytes, 64 apart.
    static __device__ __forceinline__ int key_across(int k) {
        return FIRST && PAIRS ? (k & 1) << 5 | (k & 2) << 6 : (k & 3) << 6;
    }

    // The matrix instruction leaves a lane rows 8 i + 4 (lane/32) .. + 3 of its column.  The
    // first operand's rows in the order that makes them 16 neighbours, or 32 in a pair of
    // tiles: row r of tile t is this one of the wave's.
    static __device__ __forceinline__ int m_row(int t, int r) {
        if constexpr (!FIRST) return t * 32 + r;
        if constexpr (PAIRS)
            return t / 2 * 64 + t % 2 * 16 + r / 4 % 2 * 32 + 4 * (r / 8) + r % 4;
        return t * 32 + r / 4 % 2 * 16 + 4 * (r / 8) + r % 4;
    }

    // 8 elements of k for each lane: row `lane % 32` of 32-row tile t of the rows from row0
    // on, k = 16 sub + 8 (lane / 32) .. + 7.
    static __device__ __forceinline__ bf16x8 frag(const uint8_t* lds, int row0, int t, int sub) {
        const int lane = threadIdx.x % kWave;
        if constexpr (!ACROSS) {
            // (the key is that of tile 0's row: 16, 32 or 64 rows further on it is the same)
            const int row = m_row(0, lane % 32);
            return *reinterpret_cast<const bf16x8*>(
                lds + (row0 + m_row(t, 0)) * kRowBytes + row * kRowBytes +
                ((sub * 2 + lane / 32) ^ key(row)) * 16);
        } else {
            // (lane 4 i + j of 16 gives the place of columns 4 j .. 4 j + 3 of line i, and gets
            // column 4 i + j of the four lines)
            const int row = row0 + m_row(t, lane / 16 % 2 * 16 + 4 * (lane % 4));
            const int k = 16 * sub + 8 * (lane / 32) + lane % 16 / 4;
            const int from = k * kRowBytes + ((row * 2) ^ key_across(k));
            typedef __attribute__((address_space(3))) i16x4 lds4;
            union {
                i16x4 h[2];
                bf16x8 all;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(lds + from));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(lds + from + 4 * kRowBytes));
            return u.all;
        }
    }

    // Piece `c` of each lane's row of codes.
    static __device__ __forceinline__ u32x4 codes(const uint8_t* lds, int row0, int t, int c) {
        const int row = m_row(0, threadIdx.x % 32);
        return *reinterpret_cast<const u32x4*>(lds + (row0 + m_row(t, 0)) * kRowBytes +
                                               row * kRowBytes + (c ^ key(row)) * 16);
    }
};

// What is the same for all lanes, as a scalar (divisions leave it in vector registers).
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t scalar(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// A scalar as if it were new: what is derived from it (a division's reciprocal) is worked
// out here each time, rather than held in registers through the loops.
__device__ __forceinline__ int afresh(int v) {
    asm volatile("" : "+s"(v));
    return v;
}

// ---- the order of the tiles --------------------------------------------------

// Workgroups are dealt to the eight XCDs in turn.  Each XCD takes a run of
// neighbouring whole tiles, whose operands its L2 then holds once: bands of up to
// eight tiles of the shorter side, walked along the longer one.  What is left of the
// longer side past its last whole tile comes at the end, dealt over all XCDs, so that it
// does not cost a whole turn more.  (Fewer than 2^31 items: 32 bits count them.)
struct Items {
    int few, many, each, run, end, len;   // len: of k, a slice
    bool n_short;

    __device__ Items(int m, int n, int k, int tm, int tn, int slices, int step_k) {
        const int m_tiles = (m + tm - 1) / tm, n_tiles = (n + tn - 1) / tn;
        n_short = n_tiles <= m_tiles;
        few = n_short ? n_tiles : m_tiles;
        many = n_short ? m / tm : n / tn;
        const int all = few * many * slices;
        const int edge = few * ((n_short ? m_tiles : n_tiles) - many) * slices;
        const int x = blockIdx.x % 8;
        each = (all + 7) / 8;
        const int from = each * x < all ? each * x : all;
        run = all - from < each ? all - from : each;
        end = run + (edge + 7 - x) / 8;
        len = scalar(((k + slices - 1) / slices + step_k - 1) / step_k * step_k);
    }
    static __device__ int first() { return blockIdx.x / 8; }
    static __device__ int step() { return gridDim.x / 8; }
    __device__ void place(int at, int* mt, int* nt, int* slice) const {
        const int x = blockIdx.x % 8;
        int s, l;
        if (at < run) {
            const int i = each * x + at, tiles = afresh(few * many), eight = afresh(8 * many);
            *slice = i / tiles;
            const int t = i % tiles, band = t / eight, in = t % eight;
            const int wide = few - band * 8 < 8 ? few - band * 8 : 8;
            s = band * 8 + in % wide;
            l = in / wide;
        } else {
            const int i = (at - run) * 8 + x, each_slice = afresh(few);
            *slice = i / each_slice;
            s = i % each_slice;
            l = many;
        }
        *slice = scalar(*slice);
        *mt = scalar(n_short ? l : s);
        *nt = scalar(n_short ? s : l);
    }
    // Steps of k of a slice: one at least, whose sums are then zeros.
    __device__ int turns(int k, int slice, int step_k) const {
        const int64_t left = k - static_cast<int64_t>(slice) * len;
        const int n = left < len ? static_cast<int>(left) : len;
        return n <= step_k ? 1 : (n + step_k - 1) / step_k;
    }
};

// What the products are of, in 32 bits where these are enough (fewer than 2^31 items, rows
// and columns): the loops below have few scalar registers to spare.
struct Extent {
    int m, n, k, slices;
    __device__ explicit Extent(const ProductArgs& a)
        : m(static_cast<int>(a.m)), n(static_cast<int>(a.n)), k(static_cast<int>(a.k)),
          slices(a.slices) {
        if (a.count != nullptr) (a.count_is_k ? k : n) = scalar(*a.count);
        if (a.items != 0) slices = scalar(cut_of(tiles_of(m) * tiles_of(n), a.items, a.most));
    }
};

constexpr int kTileGroups = 256;          // one workgroup a CU

inline unsigned product_grid(int64_t m, int64_t n, int tm, int tn, int slices, int groups) {
    const int64_t all = ((m + tm - 1) / tm) * ((n + tn - 1) / tn) * slices;
    const int64_t up = (all + 7) / 8 * 8;
    return static_cast<unsigned>(up < groups ? (up < 8 ? 8 : up) : groups);
}

// ---- the product -------------------------------------------------------------

// Where a wave's sums are: element i of acc[t][u] is C[n][m] with n = n0 + 32 u + lane%32 and
//   m = m0 + 64 (t/2) + 32 (lane/32) + 16 (t%2) + i       (pairs of tiles), or
//   m = m0 + 16 (lane/32) + i                             (one tile a wave).
struct Place {
    int64_t m0, n0;                       // of the wave
    int64_t m, n;                         // ends of the product
    int slice;
};

template <int N> struct Count {
    static constexpr int value = N;
};

// How a step's products are made: kSubs times, every row tile of A with all of B's.
// A's pieces are read kAhead row tiles (no more than a round's) before their use, B's (into the
// next of kSlots) for the next time round.
template <class Epilogue, int MT, int NT, int SUBS> struct Bf16Math {
    static constexpr int kSubs = SUBS, kAhead = MT > 3 ? 3 : 1, kSlots = 2;
    typedef bf16x8 A;
    struct B {
        bf16x8 v[NT];
    };
    __device__ __forceinline__ void enter(const Epilogue&, const Place&) {}
    __device__ __forceinline__ void step() {}
    __device__ __forceinline__ void take(const B&) {}
    template <class S> __device__ __forceinline__ A read_a(const uint8_t* l, int w, int t, int sub) {
        return S::frag(l, w, t, sub);
    }
    template <class S> __device__ __forceinline__ B read_b(const uint8_t* l, int w, int sub) {
        B b;
        for (int u = 0; u < NT; ++u) b.v[u] = S::frag(l, w, u, sub);
        return b;
    }
    __device__ __forceinline__ void multiply(const A& a, const B& b, f32x16 (&acc)[NT]) {
        for (int u = 0; u < NT; ++u)
            acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b.v[u], acc[u], 0, 0, 0);
    }
};

template <class Epilogue, int MT, int NT, int SUBS> struct SplitMath {
    static constexpr int kSubs = SUBS, kAhead = 1, kSlots = 2;
    struct A {
        bf16x8 p[3];
    };
    struct B {
        bf16x8 v[3][NT];
    };
    __device__ __forceinline__ void enter(const Epilogue&, const Place&) {}
    __device__ __forceinline__ void step() {}
    __device__ __forceinline__ void take(const B&) {}
    template <class S> __device__ __forceinline__ A read_a(const uint8_t* l, int w, int t, int sub) {
        A a;
        for (int p = 0; p < 3; ++p) a.p[p] = S::frag(l + p * S::kPlaneBytes, w, t, sub);
        return a;
    }
    template <class S> __device__ __forceinline__ B read_b(const uint8_t* l, int w, int sub) {
        B b;
        for (int p = 0; p < 3; ++p)
            for (int u = 0; u < NT; ++u) b.v[p][u] = S::frag(l + p * S::kPlaneBytes, w, u, sub);
        return b;
    }
    __device__ __forceinline__ void multiply(const A& a, const B& b, f32x16 (&acc)[NT]) {
        // the smallest products first
        constexpr int pa[6] = {0, 2, 1, 0, 1, 0}, pb[6] = {2, 0, 1, 1, 0, 0};
#pragma unroll
        for (int q = 0; q < 6; ++q)
            for (int u = 0; u < NT; ++u)
                acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[pa[q]], b.v[pb[q]][u], acc[u],
                                                                 0, 0, 0);
    }
};

// Through registers.  The next step's 16-byte pieces are under way from memory to registers
// while this step's products run, and are put into the other one of two LDS buffers beside
// them: a step costs one barrier and no wait that its products do not cover.  Binary32's way
// to LDS has some 35 vector instructions a piece (its three planes): these are spread between
// the products, five after each, from copies of the pieces, whose registers take the step
// after at once (all of a step's at a time, halfway through its products: 3.85 ms for 2048 x
// 73760 x 2048, so 3.40; of which the conversions are 0.27).  Other types' pieces, whose
// products leave no registers for copies, go halfway.
constexpr int kStepBytes = 128;

template <class Via, bool SA, bool SB, int TM, int TN, int WM, int WN, class Epilogue,
          template <class, int, int, int> class Math>
__global__ __launch_bounds__(kTileThreads, 2) void k_product(ProductArgs a, Epilogue e) {
    static_assert(WM * WN == kTileWaves, "");
    constexpr int kMT = TM / WM / kSquare, kNT = TN / WN / kSquare;
    typedef Side<Via, SA, TM, true, kMT % 2 == 0, kStepBytes> SideA;
    typedef Side<Via, SB, TN, false, false, kStepBytes> SideB;
    constexpr bool kSpread = Via::kPlanes == 3;
    // (a sub-step is 32 bytes of what LDS holds)
    typedef Math<Epilogue, kMT, kNT, SideA::kStep * SideA::kHeld / 32> Made;
    constexpr int kStep = SideA::kStep, kGroups = Made::kSubs * kMT, kAhead = Made::kAhead;
    static_assert(kMT >= 1 && kNT >= 1 && kGroups % (kAhead + 1) == 0 && kGroups > kAhead &&
                      kAhead <= kMT && Made::kSubs % Made::kSlots == 0, "");
    __shared__ __attribute__((aligned(128))) uint8_t lds[2][SideA::kBytes + SideB::kBytes];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN * (TM / WM), wn = wave % WN * (TN / WN);
    const Extent x(a);
    const Items items(x.m, x.n, x.k, TM, TN, x.slices, kStep);
    int in_at = Items::first(), in_turns = 0;
    SideA sa;
    SideB sb;
    auto aim = [&] {
        if (in_at >= items.end) return;
        int mt, nt, slice;
        items.place(in_at, &mt, &nt, &slice);
        in_turns = items.turns(x.k, slice, kStep);
        const int64_t k0 = static_cast<int64_t>(slice) * items.len;
        const int64_t k1 = k0 + items.len < x.k ? k0 + items.len : x.k;
        sa.enter(a.a, a.lda, static_cast<int64_t>(mt) * TM, x.m, k0, k1);
        sb.enter(a.b, a.ldb, static_cast<int64_t>(nt) * TN, x.n, k0, k1);
    };
    aim();
    // The step at `in` into registers; then on to the next one.
    bool held = false;
    auto fetch = [&] {
        held = in_at < items.end;
        if (!held) return;
        // (one branch for both: where ways join, the compiler waits for all that either has
        // under way before it uses a register of theirs again)
        if (sa.whole() && sb.whole()) {
            sa.load();
            sb.load();
        } else {
            sa.load_some();
            sb.load_some();
        }
        sa.onward();
        sb.onward();
        if (--in_turns == 0) {
            in_at += Items::step();
            aim();
        }
    };
    auto put = [&](uint8_t* to) {
        if (!held) return;
        sa.put(to, sa.v);
        sb.put(to + SideA::kBytes, sb.v);
    };
    int buf = 0;
    fetch();
    put(lds[0]);
    fetch();
    __syncthreads();
    for (int item = Items::first(); item < items.end; item += Items::step()) {
        int mt, nt, slice;
        items.place(item, &mt, &nt, &slice);
        int turns = items.turns(x.k, slice, kStep);
        f32x16 acc[kMT][kNT] = {};
        const Place at{static_cast<int64_t>(mt) * TM + wm, static_cast<int64_t>(nt) * TN + wn, x.m,
                       x.n, slice};
        Made made;
        made.enter(e, at);
        typename Made::A va[kAhead + 1];
        typename Made::B vb[Made::kSlots];
        vb[0] = made.template read_b<SideB>(lds[buf] + SideA::kBytes, wn, 0);
#pragma unroll
        for (int g = 0; g < kAhead; ++g) va[g] = made.template read_a<SideA>(lds[buf], wm, g % kMT, g / kMT);
#pragma clang loop unroll(disable)
        do {
            const uint8_t *l = lds[buf], *next = lds[buf ^ 1];
            made.step();
            u32x4 pa[SideA::kMine], pb[SideB::kMine];
            if constexpr (kSpread) {
                for (int j = 0; j < SideA::kMine; ++j) pa[j] = sa.v[j];
                for (int j = 0; j < SideB::kMine; ++j) pb[j] = sb.v[j];
                fetch();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int sub = g / kMT, h = g + kAhead;
                if (!kSpread && g == kGroups / 2) {
                    put(lds[buf ^ 1]);
                    fetch();
                }
                if (g % kMT == 0) made.take(vb[sub % Made::kSlots]);
                // All of this step has been read, and the next one is in LDS.  (After a
                // tile's last step these are the next tile's, and not used.)
                if (h == kGroups) __syncthreads();
                if (h % kMT == 0)
                    vb[h / kMT % Made::kSlots] = made.template read_b<SideB>(
                        (h < kGroups ? l : next) + SideA::kBytes, wn, h / kMT % Made::kSubs);
                va[h % (kAhead + 1)] = made.template read_a<SideA>(
                    h < kGroups ? l : next, wm, h % kMT, h / kMT % Made::kSubs);
                __builtin_amdgcn_sched_barrier(0);
                made.multiply(va[g % (kAhead + 1)], vb[sub % Made::kSlots], acc[g % kMT]);
                if constexpr (kSpread) {
                    // (a step that is not there leaves what nobody reads)
                    constexpr int kOver = kGroups - kAhead, kA = SideA::kMine, kAll = kA + SideB::kMine;
#pragma unroll
                    for (int q = 0; q < kAll; ++q) {
                        if (q * kOver / kAll != g) continue;
                        if (q < kA) sa.put(lds[buf ^ 1], q, pa[q]);
                        else sb.put(lds[buf ^ 1] + SideA::kBytes, q - kA, pb[q - kA]);
                    }
                    // one product, then what the vector unit does while it runs
#pragma unroll
                    for (int i = 0; i < 6 * kNT; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            buf ^= 1;
        } while (--turns > 0);
        e.template finish<kMT, kNT>(acc, at);
    }
}

// Straight to LDS, whole 128-byte lines of memory at a time (half lines cost as many
// requests to L2, and were slower).  No registers are held meanwhile, and LDS holds five
// units, one operand's 32 KB of a step each, in turn A B A B A: while a step's products run,
// the next step's two are there or nearly so and A of the step after it is under way, and
// when they are done their places take that step's B and the next A.  So A, which is
// taken to be the operand that comes from far (weights), has the time of two to three steps to
// come, B (tokens, read by many) that of one to two.  The loop has no branch but those to
// the next tile, so that the compiler can count the reads that are under way.
constexpr int kUnits = 5, kUnitBytes = 32768;

template <class Via, bool SA, bool SB, int TM, int TN, int WM, int WN, class Epilogue,
          template <class, int, int, int> class Math>
__global__ __launch_bounds__(kTileThreads, 2) void k_product_direct(ProductArgs a, Epilogue e) {
    static_assert(WM * WN == kTileWaves, "");
    constexpr int kMT = TM / WM / kSquare, kNT = TN / WN / kSquare;
    typedef Side<Via, SA, TM, true, kMT % 2 == 0, kStepBytes> SideA;
    typedef Side<Via, SB, TN, false, false, kStepBytes> SideB;
    typedef Math<Epilogue, kMT, kNT, 4> Made;
    constexpr int kStep = SideA::kStep, kGroups = Made::kSubs * kMT, kAhead = Made::kAhead;
    constexpr int kLoads = SideA::kMine;                             // of a unit, each thread's
    static_assert(SideA::kBytes == kUnitBytes && SideB::kBytes == kUnitBytes, "");
    static_assert(kGroups % (kAhead + 1) == 0 && kGroups > kAhead + 1 && kAhead <= kMT &&
                      Made::kSubs % Made::kSlots == 0, "");
    __shared__ __attribute__((aligned(128))) uint8_t lds[kUnits * kUnitBytes];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN * (TM / WM), wn = wave % WN * (TN / WN);
    const Extent x(a);
    const Items items(x.m, x.n, x.k, TM, TN, x.slices, kStep);
    typename SideA::Direct sa;
    typename SideB::Direct sb;
    sa.start(a.a, a.lda);
    sb.start(a.b, a.ldb);
    // To the item at `at`, for one side.
    auto aim = [&](int at, auto& side, bool first) {
        int turns = INT32_MAX;
        if (at < items.end) {
            int mt, nt, slice;
            items.place(at, &mt, &nt, &slice);
            turns = items.turns(x.k, slice, kStep);
            const int64_t k0 = static_cast<int64_t>(slice) * items.len;
            const int64_t k1 = k0 + items.len < x.k ? k0 + items.len : x.k;
            if (first) side.enter(static_cast<int64_t>(mt) * TM, x.m, k0, k1);
            else side.enter(static_cast<int64_t>(nt) * TN, x.n, k0, k1);
        } else {
            side.stop();
        }
        // (so that the compiler knows of no scalar load under way in the loop below, beside
        // which it could not count LDS reads)
        __builtin_amdgcn_s_waitcnt(0xC07F);
        return turns;
    };
    int a_at = Items::first(), b_at = a_at;
    int a_turns = aim(a_at, sa, true), b_turns = aim(b_at, sb, false);
    // On to the next items where that is due: before a step's products, whose block of
    // instructions is then not cut.
    auto onward = [&] {
        if (a_turns == 0) a_turns = aim(a_at += Items::step(), sa, true);
        if (b_turns == 0) b_turns = aim(b_at += Items::step(), sb, false);
    };
    // Sends for the next unit of an operand.
    auto fetch_a = [&](int place) {
        sa.load(lds + place, wave);
        --a_turns;
    };
    auto fetch_b = [&](int place) {
        sb.load(lds + place, wave);
        --b_turns;
    };
    auto after = [](int place, int units) {
        const int p = place + units * kUnitBytes;
        return p >= kUnits * kUnitBytes ? p - kUnits * kUnitBytes : p;
    };
    // All but the last `late` units sent for are in LDS, for every wave, and what every wave
    // has asked LDS for so far it has.
    auto meet = [&](auto late) {
        constexpr int n = decltype(late)::value * kLoads;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4 << 14) | 0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    fetch_a(0);
    fetch_b(kUnitBytes);
    onward();
    fetch_a(2 * kUnitBytes);
    fetch_b(3 * kUnitBytes);
    onward();
    fetch_a(4 * kUnitBytes);
    meet(Count<3>{});
    int at_a = 0, at_b = kUnitBytes;
    for (int item = Items::first(); item < items.end; item += Items::step()) {
        int mt, nt, slice;
        items.place(item, &mt, &nt, &slice);
        int turns = items.turns(x.k, slice, kStep);
        f32x16 acc[kMT][kNT] = {};
        const Place at{static_cast<int64_t>(mt) * TM + wm, static_cast<int64_t>(nt) * TN + wn, x.m,
                       x.n, slice};
        Made made;
        made.enter(e, at);
        typename Made::A va[kAhead + 1];
        typename Made::B vb[Made::kSlots];
        vb[0] = made.template read_b<SideB>(lds + at_b, wn, 0);
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
            va[g] = made.template read_a<SideA>(lds + at_a, wm, g % kMT, g / kMT);
        auto turn = [&](auto first) {
            onward();
            made.step();
            const int next_a = after(at_a, 2), next_b = after(at_b, 2);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int sub = g / kMT, h = g + kAhead;
                if (g % kMT == 0) made.take(vb[sub % Made::kSlots]);
                // An epilogue's loads and stores are counted with the units: the first time
                // after it all have to be in.
                if (h == kGroups) meet(Count<decltype(first)::value ? 0 : 1>{});
                // (after a tile's last step these are the next tile's, and not used)
                if (h % kMT == 0)
                    vb[h / kMT % Made::kSlots] = made.template read_b<SideB>(
                        lds + (h < kGroups ? at_b : next_b), wn, h / kMT % Made::kSubs);
                va[h % (kAhead + 1)] = made.template read_a<SideA>(
                    lds + (h < kGroups ? at_a : next_a), wm, h % kMT, h / kMT % Made::kSubs);
                __builtin_amdgcn_sched_barrier(0);
                made.multiply(va[g % (kAhead + 1)], vb[sub % Made::kSlots], acc[g % kMT]);
                __builtin_amdgcn_sched_barrier(0);
                // this step has been read by all: its places are free
                if (h == kGroups) fetch_b(at_a);
                if (kAhead > 1 ? h == kGroups + 1 : h == kGroups) fetch_a(at_b);
            }
            at_a = next_a;
            at_b = next_b;
        };
        turn(Count<1>{});
#pragma clang loop unroll(disable)
        while (--turns > 0) turn(Count<0>{});
        e.template finish<kMT, kNT>(acc, at);
    }
    // (LDS is this workgroup's until all that was sent for has come)
    __builtin_amdgcn_s_waitcnt(0x0F70);
}

// (8192^3 of codes with a bf16 result, straight against through registers: 0.47 and 1.10 ms, or
// 1.00 with one operand of odd rows; 2048 tokens x 73,760 x 2048 in bf16: 0.53 and 0.74.)
//
// Whether an operand can go straight to LDS: rows at multiples of 16 bytes, offsets within a
// tile in 31 bits, and whole pieces of `along` elements (0: whatever a line's last piece holds
// past its end may be read).
inline bool direct(const void* p, int64_t ld, int64_t esize, int64_t along) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * esize % 16 == 0 &&
           along * esize % 16 == 0 && ld * esize < int64_t(1) << 23;
}

// ---- epilogues ---------------------------------------------------------------

// The lane, worked out where it is asked for: what an epilogue derives from it would
// otherwise be held in registers through the products.
__device__ __forceinline__ int lane_here() {
    int lane = static_cast<int>(threadIdx.x) % kWave;
    asm volatile("" : "+v"(lane));
    return lane;
}

// A lane's sums of column u as runs of neighbours: run p of MT/2 (32 each), or the one of 16,
// from row run_at(p) on.
template <int MT> constexpr int kRun = MT == 1 ? 16 : 32;
template <int MT> constexpr int kRuns = MT == 1 ? 1 : MT / 2;
template <int MT> __device__ __forceinline__ int run_at(int p, int lane) {
    return MT == 1 ? lane / 32 * 16 : p * 64 + lane / 32 * 32;
}
template <int MT, int NT>
__device__ __forceinline__ float in_run(const f32x16 (&acc)[MT][NT], int p, int u, int i) {
    return acc[p * 2 + i / 16][u][i % 16];
}

// Four 16-byte pieces of each of four neighbouring lanes, exchanged: lane j gets as its piece s
// piece j of lane s.
__device__ __forceinline__ void exchange(u32x4 (&c)[4], int lane) {
    auto swap = [](u32x4& low, u32x4& high, bool upper, auto other) {
        for (int d = 0; d < 4; ++d) {
            const uint32_t t = other(upper ? low[d] : high[d]);
            low[d] = upper ? t : low[d];
            high[d] = upper ? high[d] : t;
        }
    };
    auto next = [](uint32_t v) { return dpp<0xB1>(v); };                 // lanes 1 0 3 2
    auto second = [](uint32_t v) { return dpp<0x4E>(v); };               // lanes 2 3 0 1
    swap(c[0], c[1], lane & 1, next);
    swap(c[2], c[3], lane & 1, next);
    swap(c[0], c[2], lane & 2, second);
    swap(c[1], c[3], lane & 2, second);
}

// A run of N of a lane's values, value(0) ..., into row n of C, from column m on.  Lanes hold a
// row each, and 64 bytes of it are four lanes' business: they exchange pieces, so that each
// store is of whole 64-byte segments (a lane's own 16 bytes at a time, four times the
// requests, took up to a quarter of the products' time).  ADD: to what is there before.
template <int N, bool ADD, typename Y, class Value>
__device__ __forceinline__ void write_run(Y* y, int64_t ld, int64_t n, int64_t n_end, int64_t m,
                                          int64_t m_end, int lane, Value value) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(Y));
    if (N % (4 * kPer) == 0 && __all(m + N <= m_end)) {
        Y* at = y + (n - lane % 4) * ld + m + lane % 4 * kPer;
#pragma unroll
        for (int q = 0; q < N / (4 * kPer); ++q) {
            u32x4 c[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float w[kPer];
                for (int i = 0; i < kPer; ++i) w[i] = value((4 * q + s) * kPer + i);
                c[s] = __builtin_bit_cast(u32x4, Vec<Y>::pack(w));
                __builtin_amdgcn_sched_barrier(0);          // (few values at a time in registers)
            }
            exchange(c, lane);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (n - lane % 4 + s >= n_end) continue;
                Y* to = at + s * ld + 4 * q * kPer;
                if constexpr (ADD) {
                    float a[kPer], b[kPer];
                    Vec<Y>::unpack(Vec<Y>::load(to), a);
                    Vec<Y>::unpack(__builtin_bit_cast(typename Vec<Y>::raw, c[s]), b);
                    for (int i = 0; i < kPer; ++i) a[i] += b[i];
                    Vec<Y>::store(to, Vec<Y>::pack(a));
                } else {
                    Vec<Y>::store(to, __builtin_bit_cast(typename Vec<Y>::raw, c[s]));
                }
            }
        }
        return;
    }
    if (n >= n_end) return;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        float w[8];
        for (int k = 0; k < 8; ++k) w[k] = value(i + k);
        if (ADD) {
            float a[8];
            load8(y + n * ld, m + i, m_end, a);
            for (int k = 0; k < 8; ++k) w[k] += a[k];
        }
        store8(y + n * ld, m + i, m_end, w);
    }
}

// C written out, a row of M for each n.
template <typename Y> struct StoreTile {
    Y* y;
    int64_t ld;
    StoreTile(void* to, int64_t l) : y(static_cast<Y*>(to)), ld(l) {}
    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x16 (&acc)[MT][NT], const Place& at) const {
        const int lane = lane_here();
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int p = 0; p < kRuns<MT>; ++p)
                write_run<kRun<MT>, false>(y, ld, at.n0 + u * kSquare + lane % kSquare, at.n,
                                           at.m0 + run_at<MT>(p, lane), at.m, lane,
                                           [&](int i) { return in_run(acc, p, u, i); });
    }
};

}  // namespace dlk
