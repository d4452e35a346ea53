// Log probabilities of given tokens straight from the head's inputs, and their
// gradients, without the logits.
//
//   l = x E^T ; m = max l ; S = sum exp(l - m)
//   log p_t = (l_t - m) - log S ;  H = log S - sum exp(l - m)(l - m) / S
//   d = a (delta_t - p) - b p (log p + H) ;  dx = d E ;  dE = d^T x
//
// Forward: E's product with x tile by tile (tiles.h), from whose registers a wave leaves the
// m, S and sum of a span of the vocabulary for each token, joined by a second launch.  2048
// tokens x 73760 x 2048 in bf16: 0.54 ms, 1.14 PFLOP/s, of which 13 us join the parts; the
// matrix cores' power bounds it (a loop of nothing but these instructions reaches 1.8).  In
// fp32, six bf16 products for one: 3.3 ms, 187 TFLOP/s.  Up to 32 tokens read E once, straight
// into registers (few.h): one token 69 us, 4.4 TB/s; 33 tokens in tiles of 128 take 84.
//
// Backward: the rows that have a part are gathered first, so that a product has as many
// columns as there are of them (a masked-token loss has targets at its masked positions only);
// then the logits again, piece by piece of the vocabulary, d in memory, and its two products.
// 2048 rows, all with a target, x 73760 x 2048 in bf16: 1.92 ms for 1.86 TFLOP.  A piece is
// 128 MB of d: here 96 x 8 tiles, three whole turns of the 256 workgroups (with 72 MB 0.6 in
// 100 more, with 48 17, with 256 3; other sizes fall between turns with any of them, and a
// width of 128 took 8 in 100 less with 256).  Rows of at most 128 numbers keep d in registers
// (narrow.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "dlhead.h"
#include "few.h"
#include "head.h"
#include "head_device.h"
#include "narrow.h"
#include "tiles.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// What is known of a span of the vocabulary for one token: the largest logit m, the
// sum of exp(l - m) without one largest element's own 1, and the sum of
// exp(l - m)(l - m).
template <typename F> struct PartOf {
    float m;
    F rest, dot;

    static __device__ __forceinline__ PartOf none() { return PartOf{-__builtin_inff(), 0, 0}; }
    // None of a span's tokens has a probability (nor is there a NaN).
    __device__ __forceinline__ bool nothing() const {
        return m == -__builtin_inff() && rest == rest;
    }
    template <typename G> __device__ __forceinline__ void add(const PartOf<G>& q) {
        if (q.nothing()) return;
        PartOf p{q.m, q.rest, q.dot};
        if (nothing()) {
            *this = p;
            return;
        }
        if (p.m > m) {
            const PartOf t = *this;
            *this = p;
            p = t;
        }
        const float d = p.m - m, w = exp_of(d);
        rest += w * (1 + p.rest);
        // (w is 0 where d is -infinity)
        dot += w > 0 || w != w ? w * (p.dot + d * (1 + p.rest)) : 0;
    }
};
// Of a span; and of many, one after the other, in binary64: equal terms round the same way
// at each addition, and 2^28 tokens' in one chain of binary32 came out 4e-4 off.
typedef PartOf<float> Part;
typedef PartOf<double> Total;

__device__ __forceinline__ Part part_of(const Total& t) {
    return Part{t.m, static_cast<float>(t.rest), static_cast<float>(t.dot)};
}

// ---- forward -----------------------------------------------------------------

struct StatsTile {
    Part* parts;                          // one row of `rows` for each wave's span
    int64_t rows;
    const int64_t* targets;               // or nullptr
    float* at_target;                     // the targets' logits

    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x16 (&acc)[MT][NT], const Place& at) const {
        constexpr int kMine = MT * 16;                     // of a token's logits in this lane
        const int lane = lane_here();
        const int64_t left = at.m - at.m0;                 // of the vocabulary from here on
        if (left <= 0) return;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int64_t n = at.n0 + u * kSquare + lane % kSquare;
            float v[kMine];
            for (int q = 0; q < kMine; ++q) v[q] = in_run(acc, q / 32, u, q % 32);
            // element q of v is token m0 + 64 (q/32) + 32 (lane/32) + q%32
            const int first = lane / 32 * 32;
            if (left < MT * 32)
                for (int q = 0; q < kMine; ++q)
                    if (q / 32 * 64 + first + q % 32 >= left) v[q] = -__builtin_inff();
            if (targets != nullptr) {
                const int64_t t = n < at.n ? targets[n] - at.m0 : -1;
                const bool mine = t >= 0 && t < MT * 32 && t < left && t / 32 % 2 == lane / 32;
                if (__any(mine)) {
                    float l = 0;
                    for (int q = 0; q < kMine; ++q)
                        if (q / 32 * 64 + first + q % 32 == t) l = v[q];
                    if (mine) at_target[n] = l;
                }
            }
            float m = v[0];
            for (int q = 1; q < kMine; ++q) m = fmaxf(m, v[q]);
            m = fmaxf(m, __shfl_xor(m, 32));
            const float from = m == -__builtin_inff() ? 0.0f : m;
            float s = 0, dot = 0;
            for (int q = 0; q < kMine; ++q) {
                const float d = v[q] - from, x = exp_of(d);
                s += x;
                // (a masked token's d is -infinity and its x 0, of which the product is to be 0)
                dot = __builtin_fmaf(x, fmaxf(d, -0x1.fffffep+127f), dot);
            }
            s += __shfl_xor(s, 32);
            dot += __shfl_xor(dot, 32);
            float rest = s - 1;
            // a nearly certain token: the others' sum by itself, with all its digits
            if (__any(s < 1.5f)) {
                float r = 0, same = 0;
                for (int q = 0; q < kMine; ++q) {
                    const bool top = v[q] == m;
                    same += top ? 1.0f : 0.0f;
                    r += top ? 0.0f : exp_of(v[q] - from);
                }
                r += __shfl_xor(r, 32);
                same += __shfl_xor(same, 32);
                if (s < 1.5f) rest = r + (same - 1);
            }
            if (lane < 32 && n < at.n)
                parts[at.m0 / (MT * 32) * rows + n] = Part{m, rest, dot};
        }
    }
};

// The same for a few tokens: a thread meets one token's logits, some rows of the vocabulary
// in turn, and leaves a part for all of the workgroup's.
struct StatsFew {
    static constexpr bool kRowsFirst = false;
    Part* parts;                          // one row of `rows` for each workgroup
    int64_t rows;
    const int64_t* targets;               // or nullptr
    float* at_target;
    Total mine;

    __device__ __forceinline__ void begin() { mine = Total::none(); }
    __device__ __forceinline__ void value(float l, int64_t row, int v) {
        if (targets != nullptr && targets[v] == row) at_target[v] = l;
        // (one of +infinity or NaN makes the sum NaN, one of -infinity has no part in it)
        mine.add(Part{l, l == -__builtin_inff() ? 0.0f : l - l, 0});
    }
    __device__ __forceinline__ void end(float* lds, int count) {
        const int tokens = count <= 16 ? 16 : 32;
        Part* all = reinterpret_cast<Part*>(lds);
        Part part = part_of(mine);
        __syncthreads();
        all[threadIdx.x] = part;
        for (int n = kFewThreads / 2; n >= tokens; n /= 2) {
            __syncthreads();
            if (static_cast<int>(threadIdx.x) < n) {
                part.add(all[threadIdx.x + n]);
                all[threadIdx.x] = part;
            }
        }
        if (static_cast<int>(threadIdx.x) < count) parts[blockIdx.x * rows + threadIdx.x] = part;
    }
};

// The row's results from its spans' parts: 16 rows a workgroup, 64 threads each.  (All of a
// thread's in binary64, rather than its runs of 256: 0.6 us more for one row of 256 parts.)
constexpr int kJoinRows = 16, kJoinParts = 64, kJoinRun = 256;

__global__ __launch_bounds__(kJoinRows * kJoinParts) void k_join(
    const Part* parts, int n_parts, int64_t rows, int64_t vocab, const int64_t* targets,
    const float* at_target, float* logprobs, float* entropy, float* stats) {
    __shared__ Part lds[kJoinParts][kJoinRows];
    const int r = threadIdx.x % kJoinRows, g = threadIdx.x / kJoinRows;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinRows + r;
    const int64_t safe = row < rows ? row : rows - 1;
    Part all = Part::none();
    Total before = Total::none();         // what came before the last kJoinRun or fewer
    for (int p = g, run = 0; p < n_parts; p += 4 * kJoinParts) {
        Part q[4];
        for (int k = 0; k < 4; ++k)
            q[k] = p + k * kJoinParts < n_parts ? parts[(p + k * kJoinParts) * rows + safe]
                                               : Part::none();
        for (int k = 0; k < 4; ++k) all.add(q[k]);
        if ((run += 4) < kJoinRun) continue;
        before.add(all);
        all = Part::none();
        run = 0;
    }
    if (!before.nothing()) {
        before.add(all);
        all = part_of(before);
    }
    lds[g][r] = all;
    for (int h = kJoinParts / 2; h > 0; h /= 2) {
        __syncthreads();
        if (g < h) {
            all.add(lds[g + h][r]);
            lds[g][r] = all;
        }
    }
    if (g != 0 || row >= rows) return;
    const bool nothing = all.nothing();
    const float m = all.m, log_s = nothing ? 0.0f : log1pf(all.rest);
    if (stats != nullptr) {
        stats[2 * row] = m;
        stats[2 * row + 1] = log_s;
    }
    if (entropy != nullptr)
        entropy[row] = nothing ? 0.0f : log_s - all.dot / (1 + all.rest);
    if (logprobs != nullptr) {
        const int64_t t = targets[row];
        float lp = 0.0f;
        if (t >= vocab) lp = __uint_as_float(0x7FC00000u);
        else if (t >= 0) lp = nothing ? m : (at_target[row] - m) - log_s;
        logprobs[row] = lp;
    }
}

// ---- backward ----------------------------------------------------------------

// What the gradient in a row's logits needs beside them.
struct __attribute__((aligned(16))) RowTerms {
    float m, log_s, a, b, entropy;
    int32_t target;                       // or -1
    int32_t pad[2];
};

// The rows that have a part in the gradients, in order: those with a target, or all
// if there is a gradient of the entropies.  And their largest weight: what the products
// multiply is dlogits in units of it, so that where all weights are one (a mean's), a
// target's 1 - p is near 1 and not rounded from a number that none of bf16's is near to.
// One workgroup.
constexpr int kSelectThreads = 1024;

struct Selected {
    int count;
    float unit;
};

__global__ __launch_bounds__(kSelectThreads) void k_select(const int64_t* targets,
                                                           const float* dlogprobs,
                                                           const float* dentropy, int64_t rows,
                                                           int* index, int* where, Selected* to) {
    __shared__ int waves[2][kSelectThreads / kWave];
    __shared__ uint32_t most[kSelectThreads / kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    int before = 0;
    uint32_t unit = 0;
    for (int64_t r0 = 0, turn = 0; r0 < rows; r0 += kSelectThreads, ++turn) {
        const int64_t row = r0 + threadIdx.x;
        const bool has = row < rows && targets[row] >= 0;
        const bool in = has || (row < rows && dentropy != nullptr);
        auto weigh = [&](float w) {
            const uint32_t b = abs_bits(w);
            unit = b < 0x7F800000u ? Max{}(unit, b) : unit;
        };
        if (has) weigh(dlogprobs[row]);
        if (in && dentropy != nullptr) weigh(dentropy[row]);
        const uint64_t votes = __ballot(in);
        if (lane == 0) waves[turn % 2][wave] = __popcll(votes);
        __syncthreads();
        int at = before;
        for (int w = 0; w < kSelectThreads / kWave; ++w) {
            const int c = waves[turn % 2][w];
            if (w < wave) at += c;
            before += c;
        }
        at += __popcll(votes & ((uint64_t(1) << lane) - 1));
        if (in) index[at] = static_cast<int>(row);
        if (row < rows) where[row] = in ? at : -1;
    }
    unit = wave_reduce(unit, Max{});
    if (lane == 0) most[wave] = unit;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 0; w < kSelectThreads / kWave; ++w) unit = Max{}(unit, most[w]);
    // (one below 2^-100, whose quotients might not be numbers, is no unit)
    const float u = __uint_as_float(unit);
    *to = Selected{before, u >= 0x1p-100f ? u : 1.0f};
}

struct GatherArgs {
    const void* x;
    int64_t ldx, rows, vocab;
    int width;
    const int64_t* targets;
    const float* stats;
    const float* entropy;                 // or nullptr
    const float* dlogprobs;
    const float* dentropy;                // or nullptr
    const int* index;
    const Selected* selected;
    void* to;
    int64_t ldto;
    RowTerms* terms;                      // or nullptr: narrow ones, kNarrowTerms x rows
    float* narrow;
    void* p;                              // dlogits of a piece, and where its last one's rows end
    int64_t ldp, p_end;
};

template <typename T> __global__ __launch_bounds__(256) void k_gather(GatherArgs a) {
    const int n = a.selected->count;
    const float unit = a.selected->unit;
    for (int64_t j = blockIdx.x; j < n; j += gridDim.x) {
        const int64_t row = a.index[j];
        const T* from = static_cast<const T*>(a.x) + row * a.ldx;
        T* to = static_cast<T*>(a.to) + j * a.ldto;
        for (int c = threadIdx.x * 8; c < a.width; c += 256 * 8) {
            float v[8];
            load8(from, c, a.width, v);
            store8(to, c, a.width, v);
        }
        // (zeros up to a multiple of 8: the products with dlogits read that far)
        if (a.terms != nullptr && threadIdx.x < 8 && a.p_end + threadIdx.x < a.ldp)
            static_cast<T*>(a.p)[j * a.ldp + a.p_end + threadIdx.x] = from_f32<T>(0.0f);
        if (threadIdx.x == 0) {
            const int64_t t = a.targets[row];
            RowTerms r{};
            r.m = a.stats[2 * row];
            r.log_s = a.stats[2 * row + 1];
            r.a = t < 0 ? 0.0f : t >= a.vocab ? __uint_as_float(0x7FC00000u) : a.dlogprobs[row] / unit;
            r.b = a.dentropy != nullptr ? a.dentropy[row] / unit : 0.0f;
            r.entropy = a.dentropy != nullptr ? a.entropy[row] : 0.0f;
            r.target = t < 0 || t >= a.vocab ? -1 : static_cast<int32_t>(t);
            if (a.terms != nullptr) {
                a.terms[j] = r;
            } else {
                const float m = r.m == -__builtin_inff() ? 0.0f : r.m;
                const float base = (m + r.log_s) * kLog2e, other = -r.b * kLn2;
                // (what log2(p) of the largest logit lacks)
                const float lack = -r.log_s * kLog2e - __builtin_fmaf(m, kLog2e, -base);
                const float of_h = other * lack - r.b * r.entropy;
                const float terms[kNarrowTerms] = {
                    base, -r.a, __int_as_float(r.target), m, r.log_s, of_h - r.a, other, of_h};
                for (int k = 0; k < kNarrowTerms; ++k) a.narrow[k * a.rows + j] = terms[k];
            }
        }
    }
}

// The gradient in the logits of a piece of the vocabulary.
template <typename T, bool ENTROPY> struct GradTile {
    const RowTerms* terms;
    T* out;
    int64_t ld;
    int64_t first;                        // token that the piece begins with

    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x16 (&acc)[MT][NT], const Place& at) const {
        const int lane = lane_here();
        if (at.m - at.m0 <= 0) return;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int64_t n = at.n0 + u * kSquare + lane % kSquare;
            const RowTerms r = terms[n < at.n ? n : at.n - 1];
            const int64_t far = r.target - first - at.m0;
            const int t = r.target < 0 || far < 0 || far >= MT * 32 ? -1 : static_cast<int>(far);
            // (a row of masked tokens only: their log probabilities are the logits)
            const float from = r.m == -__builtin_inff() ? 0.0f : r.m;
            auto gradient = [&](float l, bool target) {
                float lp = (l - from) - r.log_s;
                if ((ENTROPY || target) && lp > kCertain) lp = -r.log_s;
                const float x = exp_of(lp);
                const float h = ENTROPY && x > 0 ? r.b * x * (lp + r.entropy) : 0.0f;
                // (1 - p of the target keeps its digits)
                return x != x ? x : -r.a * (target ? expm1f(lp) : x) - h;
            };
#pragma unroll
            for (int p = 0; p < kRuns<MT>; ++p) {
                const int mine = run_at<MT>(p, lane);
                float of_target = 0;
                if (__any(t >= mine && t < mine + 32)) {
                    float l = 0;
                    for (int i = 0; i < 32; ++i) l = t == mine + i ? in_run(acc, p, u, i) : l;
                    of_target = gradient(l, true);
                }
                write_run<32, false>(out, ld, n, at.n, at.m0 + mine, at.m, lane, [&](int i) {
                    const float d = gradient(in_run(acc, p, u, i), false);
                    return t == mine + i ? of_target : d;
                });
            }
        }
    }
};

// Sums of dx in binary32, a matrix of rows x width for each slice of the vocabulary,
// added up over its pieces.
struct SumTile {
    float* sums;
    int64_t ld;
    bool first;

    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x16 (&acc)[MT][NT], const Place& at) const {
        const int lane = lane_here();
        float* to = sums + at.slice * at.n * ld;
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int p = 0; p < kRuns<MT>; ++p) {
                const int64_t n = at.n0 + u * kSquare + lane % kSquare;
                const int64_t m = at.m0 + run_at<MT>(p, lane);
                auto value = [&](int i) { return in_run(acc, p, u, i); };
                if (first) write_run<32, false>(to, ld, n, at.n, m, at.m, lane, value);
                else write_run<32, true>(to, ld, n, at.n, m, at.m, lane, value);
            }
    }
};

// The slices' sums together, in the inputs' units: row i of out from row where[i] of the sums
// (0 if that is -1), or with no `where` from row i.  With `where`, slices are as many as
// cut_of gives for the selected rows' tiles, m_tiles for each 256 of them.
struct Slices {
    const float* sums;
    int64_t ld;
    int number, items, most, m_tiles;
};

// What they leave out of the product: columns `from` to `to`, eight at most, of d, and as many
// rows of e.
template <typename T> struct Rest {
    const T* d;
    int64_t ldd;
    const T* e;
    int64_t lde, from, to;
};

template <typename T>
__global__ __launch_bounds__(256) void k_join_slices(Slices a, int64_t rows, int width,
                                                     const int* where, const Selected* selected,
                                                     T* out, int64_t ldo, Rest<T> rest) {
    const float unit = selected->unit;
    const float* sums = a.sums;
    const int64_t lds = a.ld, apart = where != nullptr ? selected->count : rows;
    const int slices = where != nullptr
                           ? cut_of(tiles_of(selected->count) * a.m_tiles, a.items, a.most)
                           : a.number;
    const int per = (width + 7) / 8;                       // groups of eight columns
    const int64_t all = rows * per;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < all; i += gridDim.x * int64_t(256)) {
        const int64_t row = i / per, c = i % per * 8;
        const int64_t at = where != nullptr ? where[row] : row;
        float v[8] = {};
        if (at >= 0) {
            load8(sums + at * lds, c, width, v);
            for (int s = 1; s < slices; ++s) {
                float w[8];
                load8(sums + (s * apart + at) * lds, c, width, w);
                for (int k = 0; k < 8; ++k) v[k] += w[k];
            }
            if (rest.from < rest.to) {
                float d[8];
                load8(rest.d + at * rest.ldd, rest.from, rest.to, d);
                for (int j = 0; j < 8; ++j) {
                    if (rest.from + j >= rest.to) break;
                    float w[8];
                    load8(rest.e + (rest.from + j) * rest.lde, c, width, w);
                    for (int k = 0; k < 8; ++k) v[k] += d[j] * w[k];
                }
            }
            for (int k = 0; k < 8; ++k) v[k] *= unit;
        }
        store8(out + row * ldo, c, width, v);
    }
}

// C written out in the inputs' units.
template <typename T> struct UnitTile {
    T* y;
    int64_t ld;
    const Selected* selected;             // or nullptr

    template <int MT, int NT>
    __device__ __forceinline__ void finish(const f32x16 (&acc)[MT][NT], const Place& at) const {
        const int lane = lane_here();
        const float unit = selected != nullptr ? selected->unit : 1.0f;
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int p = 0; p < kRuns<MT>; ++p)
                write_run<32, false>(y, ld, at.n0 + u * kSquare + lane % kSquare, at.n,
                                     at.m0 + run_at<MT>(p, lane), at.m, lane,
                                     [&](int i) { return in_run(acc, p, u, i) * unit; });
    }
};

// ---- plans -------------------------------------------------------------------

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Rows of the vocabulary that a wave leaves one part of.
constexpr int kSpan = 128, kSpanSplit = 64;

// Up to so many tokens go in tiles of their own.
constexpr int kSomeTokens = 128;

int span_of(int64_t rows, int64_t esize) {
    return esize == 2 && rows > kSomeTokens ? kSpan : kSpanSplit;
}

struct Backward {
    int64_t piece, pieces;                // of the vocabulary; the last takes the rest
    int64_t ld_p, ld_x, ld_s;
    int items, most, slices;              // of the vocabulary for dx (of all rows: fewer have more)
    int slices_e;                         // of the rows for dembed
    int64_t widest;                       // piece
    int64_t index, where, selected, terms, x, p, sums, sums_e, bytes;      // places in the workspace
};

int items_of(int64_t tiles) { return static_cast<int>(tiles > 128 ? tiles : 256); }

// Rows of sums that the slices of up to `rows` rows need.
int64_t slice_rows(int64_t rows, int items, int most, int64_t m_tiles) {
    const int64_t all = items / m_tiles, cut = most * tiles_of(rows);
    return 256 * (all < cut ? all : cut);
}

constexpr int64_t kPieceBytes = int64_t(128) << 20, kNarrowPiece = int64_t(1) << 18;

Backward backward_plan(int64_t rows, int64_t vocab, int64_t width, int64_t esize) {
    Backward b{};
    int64_t most = kPieceBytes / (rows * esize) / 256 * 256;
    most = most < 2048 ? 2048 : most;
    b.pieces = (vocab + most - 1) / most;
    b.piece = b.pieces == 1 ? vocab : vocab / b.pieces / 256 * 256;
    if (b.piece == 0) {
        b.piece = vocab;
        b.pieces = 1;
    }
    b.widest = vocab - (b.pieces - 1) * b.piece;
    b.ld_p = up(b.widest, 8);
    b.ld_x = up(width, 8);
    b.ld_s = up(width, 4);
    // Products of few tiles are cut along k, so that every CU has some (333 rows x 73,760 x 2048
    // in bf16: 2.60 ms whole, 0.59 in 16).
    const int64_t m_tiles = tiles_of(width), tiles = m_tiles * tiles_of(rows);
    b.items = items_of(tiles);
    b.most = most_of(b.piece);
    b.slices = cut_of(tiles, b.items, b.most);
    const int64_t tiles_e = m_tiles * tiles_of(b.widest);
    b.slices_e = cut_of(tiles_e, items_of(tiles_e), most_of(rows));
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    b.index = take(4 * rows);
    b.where = take(4 * rows);
    b.selected = take(sizeof(Selected));
    b.terms = take(static_cast<int64_t>(sizeof(RowTerms)) * rows);
    b.x = take(rows * b.ld_x * esize);
    b.p = take(rows * b.ld_p * esize);
    b.sums = take(slice_rows(rows, b.items, b.most, m_tiles) * b.ld_s * 4);
    b.sums_e = b.slices_e == 1 ? at : take(b.slices_e * b.widest * b.ld_s * 4);
    b.bytes = at;
    return b;
}

// The same for rows of 128 numbers at most, whose products take no more time than the gradient
// in the logits takes to be written and read twice.
struct Narrow {
    int64_t ld_x, ld_s, piece;            // of the vocabulary, for dembed
    int items, most, slices_e;            // as above
    int64_t index, where, selected, terms, x, sums, bytes;
};

Narrow narrow_plan(int64_t rows, int64_t vocab, int64_t width) {
    Narrow b{};
    b.ld_x = up(width, 8);
    b.ld_s = up(width, 4);
    b.piece = vocab < kNarrowPiece ? vocab : kNarrowPiece;
    b.items = items_of(tiles_of(rows));
    b.most = most_of(vocab);
    b.slices_e = cut_of(tiles_of(b.piece), items_of(tiles_of(b.piece)), most_of(rows));
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    b.index = take(4 * rows);
    b.where = take(4 * rows);
    b.selected = take(sizeof(Selected));
    b.terms = take(4 * kNarrowTerms * rows);
    b.x = take(2 * rows * b.ld_x);
    const int64_t of_x = slice_rows(rows, b.items, b.most, 1), of_e = b.slices_e * b.piece;
    b.sums = take((of_x > of_e ? of_x : of_e) * b.ld_s * 4);
    b.bytes = at;
    return b;
}

// bf16: 256 x 256 tiles; binary32, whose three planes fill the LDS: 256 x 128.  `along_a`,
// `along_b`: elements of the operands' last lines in memory that have to be whole pieces of 16
// bytes to go straight to LDS; 0 for those of the workspace, which holds what follows.
template <typename T, bool SA, bool SB, class E>
hipError_t product_of(const ProductArgs& a, const E& e, hipStream_t s, int64_t along_a,
                      int64_t along_b) {
    const dim3 block(kTileThreads);
    // Tiles of 128 x 128, where half of a larger one or more would be empty and few tokens mean
    // few tiles (forward, bf16 and fp32: 100 tokens x 2000 x 512 33 us against 40 and 60 against
    // 86; 33 x 73,760 x 2048 84 against 105, 128 of them 299 against 311).  Not for products
    // across the embedding, with its bytes to bring (dx of 20 x 73,760 x 2048 in fp32: 50 us
    // more).
    if constexpr (!SA && !SB) {
        if (a.n <= kSomeTokens) {
            typedef std::conditional_t<sizeof(T) == 2, ViaBf16, ViaSplit> Via;
            const dim3 grid(product_grid(a.m, a.n, 128, 128, a.slices,
                                         sizeof(T) == 2 ? 2 * kTileGroups : kTileGroups));
            if constexpr (sizeof(T) == 2)
                k_product<Via, SA, SB, 128, 128, 2, 4, E, Bf16Math><<<grid, block, 0, s>>>(a, e);
            else
                k_product<Via, SA, SB, 128, 128, 2, 4, E, SplitMath><<<grid, block, 0, s>>>(a, e);
            return hipGetLastError();
        }
    }
    if constexpr (sizeof(T) == 2) {
        const dim3 grid(product_grid(a.m, a.n, 256, 256, a.slices, kTileGroups));
        if (direct(a.a, a.lda, 2, along_a) && direct(a.b, a.ldb, 2, along_b))
            k_product_direct<ViaBf16, SA, SB, 256, 256, 2, 4, E, Bf16Math>
                <<<grid, block, 0, s>>>(a, e);
        else
            k_product<ViaBf16, SA, SB, 256, 256, 2, 4, E, Bf16Math><<<grid, block, 0, s>>>(a, e);
    } else {
        k_product<ViaSplit, SA, SB, 256, 128, 4, 2, E, SplitMath>
            <<<dim3(product_grid(a.m, a.n, 256, 128, a.slices, kTileGroups)), block, 0, s>>>(a, e);
    }
    return hipGetLastError();
}

constexpr int kFewTokens = 32, kFewGroups = 256;

template <typename T> hipError_t forward(const HeadArgs& a, hipStream_t s) {
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    float* at_target = reinterpret_cast<float*>(ws);
    Part* parts = reinterpret_cast<Part*>(ws + up(4 * a.rows, 256));
    int n_parts = 0;
    hipError_t st;
    if (a.rows <= kFewTokens) {
        const FewArgs f{a.embed, a.lde, a.vocab, a.width, a.x, a.ldx, static_cast<int>(a.rows),
                        nullptr, nullptr};
        const StatsFew e{parts, a.rows, a.targets, at_target, {}};
        constexpr bool kHalf = sizeof(T) == 2;
        typedef std::conditional_t<kHalf, FewBf16<8>, FewSplit<4>> Src;
        st = a.rows <= 16 ? few<Src, 1, kHalf ? 2 : 1>(f, e, kFewGroups, s, &n_parts)
                          : few<Src, 2, 1>(f, e, kFewGroups, s, &n_parts);
    } else {
        const StatsTile e{parts, a.rows, a.targets, at_target};
        const ProductArgs p{a.embed, a.lde, a.x, a.ldx, a.vocab, a.rows, a.width, 1, nullptr,
                            false, 0, 0};
        const int span = span_of(a.rows, sizeof(T));
        n_parts = static_cast<int>((a.vocab + span - 1) / span);
        st = product_of<T, false, false>(p, e, s, a.width, a.width);
    }
    if (st != hipSuccess) return st;
    k_join<<<dim3(static_cast<unsigned>((a.rows + kJoinRows - 1) / kJoinRows)),
             dim3(kJoinRows * kJoinParts), 0, s>>>(parts, n_parts, a.rows, a.vocab, a.targets,
                                                   at_target, a.logprobs, a.entropy, a.stats);
    return hipGetLastError();
}

template <typename T>
hipError_t join_slices(const Slices& a, int64_t rows, int64_t width, const int* where,
                       const Selected* selected, T* out, int64_t ldo, hipStream_t s,
                       const Rest<T>& rest = {}) {
    const int64_t blocks = (rows * ((width + 7) / 8) + 255) / 256;
    k_join_slices<T><<<dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s>>>(
        a, rows, static_cast<int>(width), where, selected, out, ldo, rest);
    return hipGetLastError();
}

// The rows that take part, and the largest weight; then their inputs and terms.
template <typename T> hipError_t collect(const HeadBackwardArgs& a, const GatherArgs& g, int* index,
                                         int* where, Selected* selected, hipStream_t s) {
    k_select<<<dim3(1), dim3(kSelectThreads), 0, s>>>(a.targets, a.dlogprobs, a.dentropy, a.rows,
                                                      index, where, selected);
    if (const hipError_t st = hipGetLastError(); st != hipSuccess) return st;
    const unsigned walkers = static_cast<unsigned>(a.rows < 2048 ? a.rows : 2048);
    k_gather<T><<<dim3(walkers), dim3(256), 0, s>>>(g);
    return hipGetLastError();
}

hipError_t narrow_backward(const HeadBackwardArgs& a, hipStream_t s) {
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const Narrow b = narrow_plan(a.rows, a.vocab, a.width);
    int* index = reinterpret_cast<int*>(ws + b.index);
    int* where = reinterpret_cast<int*>(ws + b.where);
    Selected* selected = reinterpret_cast<Selected*>(ws + b.selected);
    float* terms = reinterpret_cast<float*>(ws + b.terms);
    bf16* x = reinterpret_cast<bf16*>(ws + b.x);
    float* sums = reinterpret_cast<float*>(ws + b.sums);
    const int width = static_cast<int>(a.width);
    const bool few = a.rows <= kFewTokens, h = a.dentropy != nullptr;
    const GatherArgs g{a.x,     a.ldx,     a.rows,      a.vocab,    width, a.targets,
                       a.stats, a.entropy, a.dlogprobs, a.dentropy, index, selected,
                       x,       b.ld_x,    nullptr,     terms,      nullptr, 0, 0};
    hipError_t st = collect<bf16>(a, g, index, where, selected, s);
    if (st != hipSuccess) return st;
    const bf16* embed = static_cast<const bf16*>(a.embed);
    static_assert(kNarrowStill == 256, "tiles_of counts them");
    if (a.dx != nullptr) {
        const NarrowArgs k{x,       b.ld_x,           a.rows, embed,           a.lde, a.vocab, width,
                           b.items, b.most, &selected->count, 0, {terms, a.rows}, sums, b.ld_s};
        const auto to_lds = [&](auto straight) {
            constexpr bool kStraight = decltype(straight)::value;
            return !h ? k_narrow<true, false, false, kStraight>
                   : few ? k_narrow<true, true, true, kStraight>
                         : k_narrow<true, true, false, kStraight>;
        };
        (direct(embed, a.lde, 2, a.width) ? to_lds(std::true_type{}) : to_lds(std::false_type{}))
            <<<dim3(static_cast<unsigned>(slice_rows(a.rows, b.items, b.most, 1) / 256)),
               dim3(kTileThreads), 0, s>>>(k);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        st = join_slices<bf16>({sums, b.ld_s, 0, b.items, b.most, 1}, a.rows, a.width, where,
                               selected, static_cast<bf16*>(a.dx), a.lddx, s);
        if (st != hipSuccess) return st;
    }
    if (a.dembed == nullptr) return hipSuccess;
    for (int64_t v0 = 0; v0 < a.vocab; v0 += b.piece) {
        const int64_t n = a.vocab - v0 < b.piece ? a.vocab - v0 : b.piece;
        const NarrowArgs k{embed + v0 * a.lde, a.lde, n, x, b.ld_x, a.rows, width,
                           b.slices_e, 0, &selected->count, v0, {terms, a.rows}, sums, b.ld_s};
        (!h ? k_narrow<false, false, false, true>
         : few ? k_narrow<false, true, true, true> : k_narrow<false, true, false, true>)
            <<<dim3(static_cast<unsigned>(tiles_of(n) * b.slices_e)), dim3(kTileThreads), 0, s>>>(k);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        st = join_slices<bf16>({sums, b.ld_s, b.slices_e, 0, 0, 0}, n, a.width, nullptr, selected,
                               static_cast<bf16*>(a.dembed) + v0 * a.ldde, a.ldde, s);
        if (st != hipSuccess) return st;
    }
    return hipSuccess;
}

template <typename T> hipError_t backward(const HeadBackwardArgs& a, hipStream_t s) {
    if (a.rows == 0) {
        const ProductArgs none{nullptr, 0, nullptr, 0, a.width, a.vocab, 0, 1, nullptr, false, 0, 0};
        return product_of<T, true, true>(
            none, UnitTile<T>{static_cast<T*>(a.dembed), a.ldde, nullptr}, s, 0, 0);
    }
    if constexpr (sizeof(T) == 2)
        // (0.56 ms against the general form's 1.21 for 8191 tokens x 50304 x 128, 0.48 against
        // 1.04 with a width of 16, 0.079 against 0.149 for 100 tokens, 0.040 against 0.067 for
        // 100 x 1000)
        if (a.width <= kNarrow && a.width % 8 == 0) return narrow_backward(a, s);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const Backward b = backward_plan(a.rows, a.vocab, a.width, sizeof(T));
    int* index = reinterpret_cast<int*>(ws + b.index);
    int* where = reinterpret_cast<int*>(ws + b.where);
    Selected* selected = reinterpret_cast<Selected*>(ws + b.selected);
    const int* count = &selected->count;
    RowTerms* terms = reinterpret_cast<RowTerms*>(ws + b.terms);
    T* x = reinterpret_cast<T*>(ws + b.x);
    T* p = reinterpret_cast<T*>(ws + b.p);
    float* sums = reinterpret_cast<float*>(ws + b.sums);
    float* sums_e = reinterpret_cast<float*>(ws + b.sums_e);
    const GatherArgs g{a.x,       a.ldx,      a.rows, a.vocab, static_cast<int>(a.width),
                       a.targets, a.stats,    a.entropy, a.dlogprobs, a.dentropy,
                       index,     selected,   x,      b.ld_x,  terms, nullptr,
                       p,         b.ld_p,     b.widest};
    hipError_t st = collect<T>(a, g, index, where, selected, s);
    if (st != hipSuccess) return st;
    Rest<T> rest{};
    for (int64_t i = 0; i < b.pieces; ++i) {
        const int64_t v0 = i * b.piece;
        const int64_t n = i + 1 < b.pieces ? b.piece : a.vocab - v0;
        const T* embed = static_cast<const T*>(a.embed) + v0 * a.lde;
        const ProductArgs lp{embed, a.lde, x, b.ld_x, n, a.rows, a.width, 1, count, false, 0, 0};
        if (a.dentropy != nullptr) {
            const GradTile<T, true> e{terms, p, b.ld_p, v0};
            st = product_of<T, false, false>(lp, e, s, a.width, a.width);
        } else {
            const GradTile<T, false> e{terms, p, b.ld_p, v0};
            st = product_of<T, false, false>(lp, e, s, a.width, a.width);
        }
        if (st != hipSuccess) return st;
        if (a.dx != nullptr) {
            // (p's rows end in zeros up to whole pieces; a row of the embedding that ends inside a
            // piece is read on into the next one, but the last of all has none: up to eight rows
            // are left for the join, where nothing is read so too, for the same results)
            int64_t end = n;
            if (sizeof(T) == 2 && i + 1 == b.pieces && a.width % 8 != 0) {
                end = (n - 1) / 8 * 8;
                rest = Rest<T>{p, b.ld_p, embed, a.lde, end, n};
            }
            const ProductArgs dp{embed, a.lde, p, b.ld_p, a.width, a.rows, end, b.slices, count,
                                 false, b.items, b.most};
            const SumTile e{sums, b.ld_s, i == 0};
            if ((st = product_of<T, true, false>(dp, e, s, 0, 0)) != hipSuccess) return st;
        }
        if (a.dembed != nullptr) {
            T* to = static_cast<T*>(a.dembed) + v0 * a.ldde;
            const ProductArgs ep{x, b.ld_x, p, b.ld_p, a.width, n, a.rows, b.slices_e, count, true, 0, 0};
            if (b.slices_e == 1) {
                const UnitTile<T> e{to, a.ldde, selected};
                st = product_of<T, true, true>(ep, e, s, 0, 0);
            } else {
                const SumTile e{sums_e, b.ld_s, true};
                st = product_of<T, true, true>(ep, e, s, 0, 0);
                if (st == hipSuccess)
                    st = join_slices<T>({sums_e, b.ld_s, b.slices_e, 0, 0, 0}, n, a.width, nullptr,
                                        selected, to, a.ldde, s);
            }
            if (st != hipSuccess) return st;
        }
    }
    if (a.dx == nullptr) return hipSuccess;
    return join_slices<T>(
        {sums, b.ld_s, 0, b.items, b.most, static_cast<int>(tiles_of(a.width))}, a.rows, a.width,
        where, selected, static_cast<T*>(a.dx), a.lddx, s, rest);
}

}  // namespace

int64_t head_workspace_bytes(int64_t rows, int64_t vocab, int64_t width, int dtype,
                             bool with_backward) {
    const int64_t span = span_of(rows, dtype == DL_BF16 ? 2 : 4);
    const int64_t parts = rows <= kFewTokens ? kFewGroups : (vocab + span - 1) / span;
    const int64_t fwd =
        up(4 * rows, 256) + up(parts * rows * static_cast<int64_t>(sizeof(Part)), 256);
    if (!with_backward) return fwd;
    int64_t bwd = backward_plan(rows, vocab, width, dtype == DL_BF16 ? 2 : 4).bytes;
    if (dtype == DL_BF16 && width <= kNarrow) {
        const int64_t narrow = narrow_plan(rows, vocab, width).bytes;
        bwd = bwd > narrow ? bwd : narrow;
    }
    return fwd > bwd ? fwd : bwd;
}

hipError_t head_logprobs(const HeadArgs& a, int dtype, hipStream_t s) {
    return dtype == DL_BF16 ? forward<bf16>(a, s) : forward<float>(a, s);
}

hipError_t head_logprobs_backward(const HeadBackwardArgs& a, int dtype, hipStream_t s) {
    return dtype == DL_BF16 ? backward<bf16>(a, s) : backward<float>(a, s);
}

}  // namespace dlk
