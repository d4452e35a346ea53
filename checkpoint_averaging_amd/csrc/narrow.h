// Gradients of log probabilities where rows are of 128 bf16 numbers at most: the gradient in
// the logits goes from the registers that hold the logits straight into its product, and no
// part of it through memory.
//
//   l = still . moving ;  p = exp(l - m - log S) ;  d = -a (p - delta_t) - b p (log p + H)
//   sums = sum over the moving rows of d times them
//
// for dx (tokens still, the vocabulary moving past them) and for dembed (the other way
// round).  A wave holds 32 still rows in registers, whole, and 32 x 128 sums.  Of moving rows
// LDS has units of 128, four in turn, sent for three units ahead; each is read along its
// rows for the logits and across them for the sums.  The first product leaves a lane 16 of
// 32 moving rows in its column, which is what the second one takes of its own operand if the
// rows are counted in that order.  d is rounded to bf16 for it, as the general form's is.
//
// 8191 tokens x 50304 x 128: dx 0.21 ms, dembed 0.29 (with an entropy's gradient 0.23 and
// 0.28), 0.21 TFLOP each: 0.64 to 1 PFLOP/s, which the exponentials and conversions between
// the products bound (some 8 vector instructions an element beside its two matrix
// instructions' share).  Through memory the gradient in the logits was 824 MB written and
// twice read, and the two and its own product took 1.1 ms.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "head_device.h"
#include "tiles.h"

namespace dlk {

constexpr int kNarrow = 128;             // elements of a row, with zeros from its width on
constexpr int kNarrowStill = kTileWaves * kSquare, kNarrowUnit = 128;
constexpr int kNarrowRing = 4, kNarrowBytes = kNarrowUnit * kNarrow * 2;
constexpr int kNarrowTerms = 8;

// A token whose log probability comes out above this has the row's largest logit, m: its log
// probability is -log S.  (Formed from a logit that is summed in another order than the
// forward pass's, it would lose all digits of a 1 - p, or of a log p + H, that are below the
// logit's last place.)
constexpr float kCertain = -0.25f;

// A row's terms, an array of `rows` for each: (m + log S) log2(e), -a, its target (or -1),
// m (0 if that is -infinity), log S; and, with a gradient b of the entropies, -a - b H,
// -b log(2) and -b H: d = p (one + other log2(p)) + a delta_t.
//
// The first is one binary32 number, so log2(p) = l log2(e) less it is off by up to three
// roundings of the logit's own size (the general form subtracts m first), the same for all of
// a row.  p moves by as much, relatively; from log p + H it is taken out: -b H has what is
// missing in log2(p) added, times -b log(2).
struct NarrowTerms {
    const float* of;
    int64_t rows;
    __device__ __forceinline__ float get(int term, int64_t row) const {
        return of[term * rows + row];
    }
};

struct NarrowArgs {
    const bf16* still;
    int64_t ld_still, still_rows;
    const bf16* moving;
    int64_t ld_moving, moving_rows;
    int width;
    int slices;                           // of the moving rows; with tokens still, cut_of's items
    int most;                             // and most
    const int* count;                     // of the tokens
    int64_t first;                        // token id of the vocabulary's first row here
    NarrowTerms terms;
    float* sums;                          // still_rows x ld for each slice
    int64_t ld;
};

// The 16-byte piece c of a row is at c ^ key(row): 16 lanes' reads along rows (rows 0-3 12-15
// 20-23 24-27 of 32 at a time, or the others), and 32 lanes' of 64 bytes of four neighbouring
// rows, meet all banks.
__device__ __forceinline__ int narrow_key(int row) { return (row & 3) << 2 | (row >> 2 & 3); }

// FEW: the forward pass was a few tokens', whose logits are summed in another order.
// STRAIGHT: the moving rows go to LDS straight; otherwise, at any alignment, through
// registers, with the same results (dx of 8191 tokens x 50304 x 128: 255 us for 216).
template <bool TOKENS_STILL, bool ENTROPY, bool FEW, bool STRAIGHT>
__global__ __launch_bounds__(kTileThreads, 2) void k_narrow(NarrowArgs a) {
    constexpr float kLog2e = 0x1.715476p+0f;
    constexpr int kSubs = kNarrow / 16, kWide = kNarrow / kSquare, kMine = kNarrowBytes / 16 / kTileThreads;
    constexpr int kLoads = kMine + (TOKENS_STILL ? 0 : 2);
    __shared__ __attribute__((aligned(128))) uint8_t lds[kNarrowRing][kNarrowBytes];
    __shared__ float lds_terms[TOKENS_STILL ? 1 : kNarrowRing][8][kNarrowUnit];
    const int lane = threadIdx.x % kWave, half = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int count = *a.count;
    const int slices = scalar(TOKENS_STILL ? cut_of(tiles_of(count), a.slices, a.most)
                                           : a.slices);
    const int slice = scalar(static_cast<int>(blockIdx.x) % slices);
    const int still_rows = TOKENS_STILL ? count : static_cast<int>(a.still_rows);
    const int moving_rows = TOKENS_STILL ? static_cast<int>(a.moving_rows) : count;
    const int n0 = scalar(static_cast<int>(blockIdx.x) / slices) * kNarrowStill;
    if (n0 >= still_rows) return;
    const int len = scalar((moving_rows + slices * kNarrowUnit - 1) / (slices * kNarrowUnit)) *
                    kNarrowUnit;
    const int from = slice * len;
    const int rows = moving_rows - from < len ? (moving_rows > from ? moving_rows - from : 0) : len;
    const int units = (rows + kNarrowUnit - 1) / kNarrowUnit;
    // this lane's column
    const int n = n0 + wave * kSquare + lane % kSquare;
    const bool there = n < still_rows;

    // ---- the way of the moving rows to LDS: rows that are not there are zeros
    const int64_t row_bytes = a.ld_moving * 2;
    const int line = threadIdx.x / 16, piece = threadIdx.x % 16 ^ narrow_key(line);
    uint32_t offset[kMine];
    for (int j = 0; j < kMine; ++j)
        offset[j] = piece * 8 < a.width
                        ? (line + j * 32) * static_cast<uint32_t>(row_bytes) + piece * 16
                        : 0xFFFFFFF0u;
    const uint8_t* base = reinterpret_cast<const uint8_t*>(a.moving) +
                          from * row_bytes;
    const float* term_base = a.terms.of + from;
    const uint32_t term_offset = static_cast<uint32_t>(threadIdx.x % kNarrowUnit) * 4;
    // (a wave's places are of half of a term)
    const float* term_of = term_base + wave / 2 * a.terms.rows;
    int left = rows;                      // not sent for yet
    auto fetch = [&](int slot) {
        if constexpr (!STRAIGHT) {
            static_assert(TOKENS_STILL, "their terms' way is straight");
            u32x4 v[kMine];
            for (int j = 0; j < kMine; ++j) {
                v[j] = u32x4{};
                if (line + j * 32 < left && piece * 8 < a.width)
                    v[j] = *reinterpret_cast<const Raw<bf16>::any*>(
                        base + (line + j * 32) * row_bytes + piece * 16);
            }
            for (int j = 0; j < kMine; ++j)
                *reinterpret_cast<u32x4*>(lds[slot] + (j * kTileThreads + threadIdx.x) * 16) = v[j];
            base += kNarrowUnit * row_bytes;
            left -= kNarrowUnit;
            return;
        }
        typedef __attribute__((address_space(3))) void lds_any;
        const int have = __builtin_elementwise_max(__builtin_elementwise_min(left, kNarrowUnit), 0);
        __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(base), 0, static_cast<uint32_t>(have * row_bytes), 0x00020000);
        for (int j = 0; j < kMine; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (lds_any*)(lds[slot] + wave * (kWave * 16) + j * (kTileThreads * 16)), 16,
                offset[j], 0, 0, 0);
        base += kNarrowUnit * row_bytes;
        if constexpr (!TOKENS_STILL) {
            float* to = &lds_terms[slot][0][0] + wave * kWave;
            __amdgpu_buffer_rsrc_t t = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<float*>(term_of), 0, have * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t, (lds_any*)to, 4, term_offset, 0, 0, 0);
            t = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(term_of + 4 * a.terms.rows), 0,
                                                  wave < (ENTROPY ? 8 : 2) ? have * 4 : 0, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t, (lds_any*)(to + 4 * kNarrowUnit), 4,
                                                     term_offset, 0, 0, 0);
            term_of += kNarrowUnit;
        }
        left -= kNarrowUnit;
    };

    // ---- the still rows
    bf16x8 still[kSubs];
    for (int s = 0; s < kSubs; ++s) {
        const int k = s * 16 + half * 8;
        u32x4 v{};
        if (there && k < a.width)
            v = *reinterpret_cast<const Raw<bf16>::any*>(a.still + n * a.ld_still + k);
        still[s] = __builtin_bit_cast(bf16x8, v);
    }
    float base2 = 0, mine = 0, top = 0, log_s = 0, one = 0, other = 0, of_h = 0;
    int target = -1;
    if constexpr (TOKENS_STILL) {
        if (there) {
            base2 = a.terms.get(0, n);
            mine = a.terms.get(1, n);
            target = __float_as_int(a.terms.get(2, n)) - from;
            top = a.terms.get(3, n);
            log_s = a.terms.get(4, n);
            if constexpr (ENTROPY) {
                one = a.terms.get(5, n);
                other = a.terms.get(6, n);
                of_h = a.terms.get(7, n);
            }
        }
    }
    const int id = static_cast<int>(a.first) + n;             // of this lane's row of the vocabulary
    __builtin_amdgcn_s_waitcnt(0x0070);                       // (none of these counts below)

    // log2(p) of a logit, and what p is multiplied by in d.  (A still token's -a alone is a
    // factor of its sums.)
    auto power = [&](float l, float base) { return __builtin_fmaf(l, kLog2e, -base); };
    // (log2(p) is -infinity where p is 0)
    auto weight = [](float log2p, float f0, float f1) {
        return __builtin_fmaf(f1, fmaxf(log2p, -0x1p+100f), f0);
    };

    // Moving row `row` of a slot along its width, and four of them across it: columns of tile w.
    auto along = [&](const uint8_t* l, int row, int sub) {
        return *reinterpret_cast<const bf16x8*>(l + row * (kNarrow * 2) +
                                                ((sub * 2 + half) ^ narrow_key(row)) * 16);
    };
    auto across = [&](const uint8_t* l, int row, int w) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const int line4 = row + lane % 16 / 4, c = w * 64 + lane / 16 % 2 * 32 + lane % 4 * 8;
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4*)(l + line4 * (kNarrow * 2) + (c ^ narrow_key(line4) * 16)));
    };

    f32x16 acc[kWide] = {};
    for (int u = 0; u < kNarrowRing - 1; ++u) fetch(u);
    for (int u = 0; u < units; ++u) {
        constexpr int kOut = (kNarrowRing - 2) * kLoads;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((kOut & 15) | (kOut >> 4 << 14) | 0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fetch((u + kNarrowRing - 1) % kNarrowRing);
        const int slot = u % kNarrowRing;
        const uint8_t* l = lds[slot];
#pragma unroll 1
        for (int pair = 0; pair < kNarrowUnit / 64; ++pair) {
            f32x16 s[2] = {};
            for (int sub = 0; sub < kSubs; ++sub)
                for (int t = 0; t < 2; ++t)
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        along(l, pair * 64 + t * 32 + lane % 32, sub), still[sub], s[t], 0, 0, 0);
            bf16x8 d[2][2];
            for (int t = 0; t < 2; ++t) {
                const int row0 = pair * 64 + t * 32;          // of the unit
                // element i is of row row0 + 8 (i / 4) + 4 half + i % 4
                float v[16];
                // (looked for there only: 58 us for 53 of dx, and 43 for 40 of dembed, for 20
                // tokens x 50,304 x 128; 8 to 12 in 100 more for 8191)
                if constexpr (FEW) {
                    float e[16], most = kCertain * kLog2e;
                    for (int i = 0; i < 16; ++i) {
                        const int r = row0 + 8 * (i / 4) + 4 * half + i % 4;
                        e[i] = power(s[t][i], TOKENS_STILL ? base2 : lds_terms[slot][0][r]);
                        // (rows past the end are zeros, which are not looked for)
                        if (TOKENS_STILL ? there : u * kNarrowUnit + r < rows)
                            most = fmaxf(most, e[i]);
                    }
                    if (__any(most > kCertain * kLog2e))
                        for (int i = 0; i < 16; ++i) {
                            const int r = row0 + 8 * (i / 4) + 4 * half + i % 4;
                            const float m = TOKENS_STILL ? top : lds_terms[slot][3][r];
                            s[t][i] = e[i] > kCertain * kLog2e ? m : s[t][i];
                        }
                }
                if constexpr (TOKENS_STILL) {
                    for (int i = 0; i < 16; ++i) {
                        const float e = power(s[t][i], base2);
                        v[i] = __builtin_amdgcn_exp2f(e);
                        if constexpr (ENTROPY) v[i] *= weight(e, one, other);
                    }
                    const int at = target - u * kNarrowUnit - row0;
                    if (__any(at >= 0 && at < 32)) {
                        for (int i = 0; i < 16; ++i)
                            if (at == 8 * (i / 4) + 4 * half + i % 4) {
                                // (with ENTROPY a certain token's logit is m itself here)
                                const float lp = (s[t][i] - top) - log_s;
                                const float less = expm1f(!ENTROPY && lp > kCertain ? -log_s : lp);
                                if constexpr (ENTROPY) {
                                    const float e = power(s[t][i], base2);
                                    v[i] = mine * less + __builtin_amdgcn_exp2f(e) *
                                                             weight(e, of_h, other);
                                } else {
                                    v[i] = less;
                                }
                            }
                    }
                } else {
                    const auto& terms = lds_terms[slot];
                    f32x4 w[4];
                    for (int q = 0; q < 4; ++q) {
                        const int r = row0 + 8 * q + 4 * half;
                        const f32x4 b = *reinterpret_cast<const f32x4*>(&terms[0][r]);
                        w[q] = *reinterpret_cast<const f32x4*>(&terms[ENTROPY ? 5 : 1][r]);
                        f32x4 f{};
                        if constexpr (ENTROPY) f = *reinterpret_cast<const f32x4*>(&terms[6][r]);
                        for (int j = 0; j < 4; ++j) {
                            const float e = power(s[t][4 * q + j], b[j]);
                            v[4 * q + j] = __builtin_amdgcn_exp2f(e);
                            if constexpr (ENTROPY) w[q][j] = weight(e, w[q][j], f[j]);
                        }
                    }
                    // -a of the targets more; where p is near 1, and little is left of both, the
                    // two by themselves
                    const int near = __float_as_int(terms[2][row0 + lane % 32]) - (id - lane % 32);
                    const bool hits = __any(near >= 0 && near < 32);
                    uint32_t certain = 0;
                    if (hits) {
                        for (int i = 0; i < 16; ++i) {
                            const int r = row0 + 8 * (i / 4) + 4 * half + i % 4;
                            const bool hit = __float_as_int(terms[2][r]) == id;
                            certain |= hit && v[i] > 1 - 0x1p-6f ? 1u << i : 0;
                            if constexpr (ENTROPY) {
                                v[i] = __builtin_fmaf(v[i], w[i / 4][i % 4], hit ? -terms[1][r] : 0);
                            } else {
                                v[i] = (v[i] - (hit ? 1.0f : 0.0f)) * w[i / 4][i % 4];
                            }
                        }
                        if (__any(certain != 0)) {
                            for (int i = 0; i < 16; ++i) {
                                const int r = row0 + 8 * (i / 4) + 4 * half + i % 4;
                                if (!(certain >> i & 1)) continue;
                                v[i] = terms[1][r] * expm1f(-terms[4][r]);
                                if constexpr (ENTROPY) {
                                    const float e = power(s[t][i], terms[0][r]);
                                    v[i] += __builtin_amdgcn_exp2f(e) *
                                            weight(e, terms[7][r], terms[6][r]);
                                }
                            }
                        }
                    } else {
                        for (int i = 0; i < 16; ++i) v[i] *= w[i / 4][i % 4];
                    }
                }
                // (zeros stand for rows past the end, but what becomes of them need not be finite)
                const int end = rows - u * kNarrowUnit - row0;
                if (end < 32)
                    for (int i = 0; i < 16; ++i)
                        if (8 * (i / 4) + 4 * half + i % 4 >= end) v[i] = 0;
                for (int h = 0; h < 2; ++h)
                    for (int i = 0; i < 8; ++i) d[t][h][i] = static_cast<__bf16>(v[8 * h + i]);
            }
            for (int t = 0; t < 2; ++t)
                for (int h = 0; h < 2; ++h)
                    for (int w = 0; w < kWide; ++w) {
                        // eight rows of k for each half of the wave: those d's elements are of
                        const int row = pair * 64 + t * 32 + h * 16 + half * 4;
                        union {
                            i16x4 part[2];
                            bf16x8 all;
                        } e;
                        e.part[0] = across(l, row, w);
                        e.part[1] = across(l, row + 8, w);
                        acc[w] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e.all, d[t][h], acc[w], 0, 0, 0);
                    }
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);   // (LDS is this workgroup's until all has come)
    if (!there) return;
    float* to = a.sums + (static_cast<int64_t>(slice) * still_rows + n) * a.ld;
    for (int w = 0; w < kWide; ++w)
        for (int q = 0; q < 4; ++q) {
            const int c = w * kSquare + 8 * q + 4 * half;
            if (c >= a.width) continue;
            f32x4 v;
            for (int j = 0; j < 4; ++j) v[j] = acc[w][4 * q + j] * (TOKENS_STILL && !ENTROPY ? mine : 1.0f);
            *reinterpret_cast<f32x4*>(to + c) = v;
        }
}

}  // namespace dlk
