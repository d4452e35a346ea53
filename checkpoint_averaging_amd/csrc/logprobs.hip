// Log probabilities of given tokens, entropy and the most likely alternatives
// of each row of logits, and their gradient.
//
// With m the row's largest element, d = l - m and e = exp(d):
//   log p = d - log S, S = sum e ;  H = log S - sum(e d) / S
// One pass keeps S and t = sum(e d) against a running maximum.  Where S is below
// 1.5 there is one maximum and S = 1 + R; log S is then log1p(R), so that a
// nearly certain token's log probability and entropy keep their digits.  R
// comes from the threads' sums but for the one that the maximum's own 1 went
// through: its elements (one 256th of the row) are read once more.
//
// The pass is bound by the logits' bytes, with some ten instructions and one
// exponential (four instructions' time) an element close behind: 2048 x 73760
// bf16 54 us (5.6 TB/s; a plain read of them takes 50), fp32 92 us (6.5 TB/s),
// 777 x 50277 fp32 with five alternatives 34 us.  One row is a chain of
// latencies: 10 us with eight alternatives, in 16 parts and two kernels, 13 us in
// one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlhead.h"
#include "head.h"
#include "head_device.h"

#pragma clang fp contract(off)

namespace dlk {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kUnroll = 4;          // 16-byte loads a thread has under way
constexpr int kTogether = 2;        // of these, vectors whose maximum is taken together
// Vectors of a row that the threads' sums go through before they start anew: 64
// turns of kUnroll loads, so no row of fewer than 262144 elements does.
constexpr uint32_t kRun = 64 * kUnroll * kThreads;
constexpr int64_t kMaxGrid = 1 << 20;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.40282347e38f;
constexpr float kFar = -1e4f;       // exp of this and of anything below is 0
constexpr int kMaxParts = 16;
constexpr int kAdded = 1024;        // most candidates added between two looks at the list
constexpr int kList = kAdded + 256; // candidates held at once (see choose)
constexpr int kKeys = 256;          // maxima that bound the alternatives

// Logits of more than this stream past the 256 MB Infinity Cache without a
// stay in it (2048 x 73760 bf16, 302 MB: 57 us, 61 us with ordinary loads);
// fewer may be there still, or be wanted again by the backward pass (180 x
// 73760 fp32, 53 MB: 15 us, 20 us non-temporally).  Alternatives are read
// again, so their rows are loaded in the ordinary way.
constexpr int64_t kNontemporalMin = int64_t(192) << 20;

template <int N> struct Count {
    static constexpr int value = N;
    __device__ constexpr operator int() const { return N; }
};

// exp(d) for d <= 0; NaN stays NaN.  The product with log2(e) is rounded once, so
// a term is off by some |d| 2^-23 of itself beside the exponential's own last
// place: terms far below the maximum, which weigh little in S.  (Log
// probabilities of 2048 x 73760 come out 3e-8 off, root mean square, as by torch's
// operations in fp32; entropies 5e-8.)
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7FC00000u); }
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }

// Statistics of some elements of a row.  r is the sum without the (single)
// maximum, where S is below 1.5.
struct Stats {
    float m, s, r, t;

    static __device__ __forceinline__ Stats none() { return Stats{kLowest, 0.0f, 0.0f, 0.0f}; }

    // The same elements against a maximum m2 >= m.
    __device__ __forceinline__ Stats at(float m2) const {
        const float d = fmaxf(m - m2, kFar), a = exp_of(d);
        return m == m2 ? *this : Stats{m2, a * s, a * s, a * (t + d * s)};
    }
    // The statistics (without r) of these elements and of others.
    __device__ __forceinline__ Stats with(const Stats& o) const {
        const float m2 = fmaxf(m, o.m);
        const Stats p = at(m2), q = o.at(m2);
        return Stats{m2, p.s + q.s, 0.0f, p.t + q.t};
    }
    // The statistics of 16 neighbouring lanes, or of the wave (without r), in one.
    __device__ __forceinline__ Stats of_lanes() const {
        const Stats q = at(lanes_reduce<16>(m, Max{}));
        return Stats{q.m, lanes_reduce<16>(q.s, Sum{}), lanes_reduce<16>(q.r, Sum{}),
                     lanes_reduce<16>(q.t, Sum{})};
    }
    __device__ __forceinline__ Stats of_wave() const {
        const Stats q = at(wave_reduce(m, Max{}));
        return Stats{q.m, wave_sum(q.s), 0.0f, wave_sum(q.t)};
    }
    __device__ __forceinline__ bool nothing() const { return s == 0.0f; }
    __device__ __forceinline__ bool nearly_certain() const { return s < 1.5f && s > 0.0f; }
    __device__ __forceinline__ float log_sum() const {
        return nothing() ? 0.0f : nearly_certain() ? log1pf(r) : logf(s);
    }
};

// A thread's running statistics.  The first maximum is the lowest finite value:
// an element of -infinity then adds exp(-infinity) = 0, one of +infinity or NaN
// turns S into NaN.
//
// Equal terms round the same way at each addition, so that a chain of them shows
// at its full length (150001 logits of two values, 586 a thread in one chain: log
// S 9e-6 off; 2^30 of them: 3e-3).  Up to 16 elements are therefore added to each
// other first, and their sum to the thread's, which starts anew after kRun: 9e-7
// and 2e-6.
struct Running {
    float m, s, t;

    static __device__ __forceinline__ Running none() { return Running{kLowest, 0.0f, 0.0f}; }

    // Moves the maximum up to m2 > m: every element seen is below it.  The
    // distance is cut off where its exponential is 0, or 0 * infinity would
    // make a NaN of it.
    template <bool ENTROPY> __device__ __forceinline__ void raise(float m2) {
        const float d = fmaxf(m - m2, kFar), a = exp_of(d);
        if constexpr (ENTROPY) t = a * (t + d * s);
        s *= a;
        m = m2;
    }
    // Adds N elements that are not above the maximum.
    template <bool ENTROPY, int N> __device__ __forceinline__ void add(const float* l) {
        float gs, gt;
        for (int i = 0; i < N; ++i) {
            const float d = l[i] - m, e = exp_of(d);
            gs = i == 0 ? e : gs + e;
            if constexpr (ENTROPY) {
                const float f = fmaxf(d, kFar);
                gt = i == 0 ? e * f : __builtin_fmaf(e, f, gt);
            }
        }
        s += gs;
        if constexpr (ENTROPY) t += gt;
    }
    __device__ __forceinline__ Stats stats() const { return Stats{m, s, 0.0f, t}; }
};

// The order of alternatives as whole numbers: larger logits first, NaN before
// all, and in a full key equal ones by the lower index.  0 is below every
// key, ~0 above.
__device__ __forceinline__ uint32_t order_of(float l) {
    const float v = l + 0.0f;                 // -0 as 0
    const uint32_t b = __float_as_uint(v);
    return v != v ? 0xFFFFFFFFu : (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t i) {
    return (static_cast<uint64_t>(order) << 32) | (0x7FFFFFFFu - i);
}
__device__ __forceinline__ int64_t index_of(uint64_t key) {
    return 0x7FFFFFFFu - static_cast<uint32_t>(key);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((u >> 31) != 0 ? (u == 0xFFFFFFFFu ? u : u & 0x7FFFFFFFu) : ~u);
}

// log p of one logit under the row's statistics.
__device__ __forceinline__ float logprob_of(float l, const Stats& st, float log_sum) {
    return st.nothing() ? minus_inf() : (l - st.m) - log_sum;
}

struct TopLds {
    uint64_t list[kList];
    uint64_t best[DL_MAX_TOP];
    uint32_t key[kKeys];
    int cand[kKeys];
    int count, cands;
    uint32_t least;
};

// best[0..k) = the k largest of the `count` distinct keys of list[], largest
// first; 0 where there are fewer.  An element's place is the number of larger
// ones, counted four keys at a time (list[count..] is filled up with 0).
__device__ __forceinline__ void rank_select(TopLds& s, int count, int k) {
    const int padded = (count + 3) / 4 * 4;
    if (threadIdx.x < static_cast<unsigned>(padded - count)) s.list[count + threadIdx.x] = 0;
    if (threadIdx.x < static_cast<unsigned>(k)) s.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t q = s.list[i];
        int rank = 0;
        for (int j = 0; j < padded; j += 4) {
            ulonglong2 o[2];
            for (int u = 0; u < 2; ++u)
                o[u] = *reinterpret_cast<const ulonglong2*>(&s.list[j + 2 * u]);
            for (int u = 0; u < 2; ++u) rank += (o[u].x > q) + (o[u].y > q);
        }
        if (rank < k) s.best[rank] = q;
    }
    __syncthreads();
}

// A lower bound of the k-th largest of the 256 numbers key[]: its upper BITS
// bits, from the highest down.  A bit belongs to it if k numbers reach it; the
// scalar unit counts them from a compare's mask.  The first wave finds it for
// all (the others' vector units are left to other workgroups).
template <int BITS> __device__ __forceinline__ uint32_t kth_bound(TopLds& s, int k) {
    static_assert(kKeys == 4 * kWave, "four numbers a lane");
    if (threadIdx.x < kWave) {
        const uint4 q = reinterpret_cast<const uint4*>(s.key)[threadIdx.x];
        uint32_t t = 0;
        for (int bit = 31; bit >= 32 - BITS; --bit) {
            const uint32_t u = t | (1u << bit);
            const int c = __popcll(__ballot(q.x >= u)) + __popcll(__ballot(q.y >= u)) +
                          __popcll(__ballot(q.z >= u)) + __popcll(__ballot(q.w >= u));
            if (c >= k) t = u;
        }
        if (threadIdx.x == 0) s.least = t;
    }
    __syncthreads();
    return s.least;
}

// best[0..k) of the elements [0, n) of l, whose index in the row is `first`
// more, from the threads' own statistics of a pass in which thread t took the
// vectors t, t + kThreads, ...
//
// The k-th largest of the threads' maxima is a lower bound of the k-th largest
// element, and only threads whose maximum reaches it hold elements that do:
// about k threads' vectors are read once more (out of a cache), spread over
// all threads.  Elements that reach the bound go to a list; where more might
// overflow it, the list is cut to its k largest, whose last then is a bound
// too (rows of many equal or ordered elements).
template <typename T>
__device__ __forceinline__ void choose(TopLds& s, const T* l, uint32_t n, uint32_t first, int k,
                                       const Stats& mine) {
    constexpr int NV = Vec<T>::n;
    static_assert(kThreads == kKeys && kThreads * 4 == kAdded, "");
    const int tid = threadIdx.x;
    uint32_t key = 0;                         // no elements
    if (static_cast<uint32_t>(tid * NV) < n)
        key = mine.s != mine.s ? 0xFF800000u  // NaN or +infinity: at least +infinity
              : mine.nothing() ? 0x007FFFFFu  // -infinity
                               : order_of(mine.m);
    s.key[tid] = key;
    if (tid == 0) s.count = s.cands = 0;
    __syncthreads();
    const uint32_t least = kth_bound<sizeof(T) == 2 ? 16 : 20>(s, k);
    if (key >= least) s.cand[atomicAdd(&s.cands, 1)] = tid;
    __syncthreads();
    const uint32_t cands = s.cands;
    const uint32_t vectors = (n + NV - 1) / NV;
    const uint32_t steps = (vectors + kThreads - 1) / kThreads;
    const uint32_t total = steps * cands;
    auto load = [&](uint32_t p, uint32_t& at) {
        typename Vec<T>::raw r{};
        at = n;
        if (p < total) at = (p / cands * kThreads + s.cand[p % cands]) * NV;
        if (at + NV <= n) {
            r = Vec<T>::load(l + at);
        } else if (at < n) {                              // the row's last, partial vector
            float x[NV];
            for (int i = 0; i < NV; ++i) x[i] = at + i < n ? to_f32(l[at + i]) : 0.0f;
            r = Vec<T>::pack(x);
        }
        return r;
    };
    uint32_t at;
    typename Vec<T>::raw r = load(tid, at);
    uint64_t bound = 0;
#pragma unroll 1
    for (uint32_t p0 = 0; p0 < total; p0 += kThreads) {
        uint32_t next_at;
        const typename Vec<T>::raw next = load(p0 + kThreads + tid, next_at);
#pragma unroll 1
        for (int h = 0; h < NV / 4; ++h) {                  // kAdded elements between two looks
            float x[4];
            Vec<T>::unpack4(r, h, x);
            for (int i = 0; i < 4; ++i) {
                const uint32_t o = order_of(x[i]), e = at + 4 * h + i;
                if (e < n && o >= least) {
                    const uint64_t q = key_of(o, first + e);
                    if (q > bound) s.list[atomicAdd(&s.count, 1)] = q;
                }
            }
            __syncthreads();
            const int count = s.count;
            __syncthreads();                                // read by all before more is added
            if (count > kList - kAdded) {
                rank_select(s, count, k);
                if (tid < k) s.list[tid] = s.best[tid];
                bound = s.best[k - 1];
                if (tid == 0) s.count = k;
                __syncthreads();
            }
        }
        r = next;
        at = next_at;
    }
    rank_select(s, s.count, k);
}

// What a row is split into: `parts` workgroups of `chunk` elements each.
//
// Up to 256 rows, one for each CU, are split into parts of at least 4096
// elements that a second kernel joins, if they are long enough to win its 3 us
// back (one row of 40000 bf16: 5.2 us in parts, 7.1 us whole; of 10000: 5.0 us,
// 3.8 us).  From 257 rows on a row is one workgroup's: 256 x 50304 in two parts
// and 257 whole are 12.5 and 14.0 us in fp32, 11.2 and 10.3 us in bf16 (with 20
// alternatives 18.5 and 19.9, 16.7 and 15.8).
struct Split {
    uint32_t parts, chunk;
};

Split split_of(int64_t rows, int64_t vocab) {
    int64_t parts = rows <= 256 && vocab >= 24 * 1024 ? 512 / rows : 1;
    parts = parts < kMaxParts ? parts : kMaxParts;
    const int64_t most = (vocab + 4095) / 4096;
    parts = parts < most ? parts : most;
    const int64_t chunk = ((vocab + parts - 1) / parts + 7) / 8 * 8;
    return Split{static_cast<uint32_t>((vocab + chunk - 1) / chunk), static_cast<uint32_t>(chunk)};
}

// A part's results in the workspace: its statistics, then its best keys.
__host__ __device__ inline int64_t part_bytes(int k) { return 16 + 8 * static_cast<int64_t>(k); }

template <bool TOP>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t row, const Stats& st,
                                          float target_logit, int64_t target,
                                          const uint64_t* best) {
    const float log_sum = st.log_sum();
    if (threadIdx.x == 0) {
        if (a.logprobs != nullptr)
            a.logprobs[row] = target < 0 ? 0.0f
                              : target >= a.vocab ? nan_f()
                                                  : logprob_of(target_logit, st, log_sum);
        if (a.entropy != nullptr)
            a.entropy[row] = st.nothing() ? 0.0f : log_sum - st.t / st.s;
        if (a.stats != nullptr) {
            a.stats[2 * row] = st.nothing() ? minus_inf() : st.m;
            a.stats[2 * row + 1] = log_sum;
        }
    }
    if constexpr (TOP) {
        if (threadIdx.x < static_cast<unsigned>(a.top_k)) {
            const uint64_t q = best[threadIdx.x];
            a.top_ids[row * a.top_k + threadIdx.x] = index_of(q);
            a.top_logprobs[row * a.top_k + threadIdx.x] = logprob_of(logit_of(q), st, log_sum);
        }
    }
}

// R of a nearly certain row (or part), from the threads' own statistics
// `mine`: the single maximum's thread counts by its elements, read again.
template <typename T>
__device__ __forceinline__ float rest_of(float* lds, int* owner, const T* l, uint32_t n,
                                         const Stats& mine, const Stats& row) {
    constexpr int NV = Vec<T>::n;
    const int tid = threadIdx.x;
    const bool owns = mine.s > 0.0f && mine.m == row.m;
    if (owns) *owner = tid;                   // one thread: two would make S 2
    __syncthreads();
    float r = owns ? 0.0f : mine.s * exp_of(fmaxf(mine.m - row.m, kFar));
    const uint32_t steps = (n + kThreads * NV - 1) / (kThreads * NV);
    for (uint32_t j = tid; j < steps; j += kThreads) {
        const uint32_t at = (j * kThreads + *owner) * NV;
        for (uint32_t i = at; i < at + NV && i < n; ++i) {
            const float x = to_f32(l[i]);
            if (x != row.m) r += exp_of(x - row.m);
        }
    }
    r = wave_sum(r);
    if (tid % kWave == 0) lds[tid / kWave] = r;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// One workgroup a part of a row; with one part a row, the results themselves.
// Eight workgroups a CU (64 vector registers, 80 scalar ones): 2048 rows are
// then under way at once (2048 x 73760 bf16 with 20 alternatives: 78 us, 86 us
// with six).
template <typename T, bool ENTROPY, bool TOP, bool NT>
__global__ __launch_bounds__(kThreads, 8) void k_logprobs(LogprobsArgs a, uint32_t parts, uint32_t chunk) {
    constexpr int NV = Vec<T>::n;
    typedef typename Vec<T>::raw raw;
    __shared__ Stats lds[kWaves];
    __shared__ float lds_r[kWaves];
    __shared__ int owner;
    __shared__ char top_lds[TOP ? sizeof(TopLds) : 1] __attribute__((aligned(16)));
    const int tid = threadIdx.x;
    // At most 256 rows are in parts, so jobs, and all indices within a row (below
    // 2^31), are whole numbers of 32 bits.
    const uint32_t jobs = static_cast<uint32_t>(a.rows) * parts;
    for (uint32_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const uint32_t r0 = job / parts;
        const int64_t row = r0;
        const uint32_t first = (job - r0 * parts) * chunk;
        const uint32_t left = static_cast<uint32_t>(a.vocab) - first;
        const uint32_t n = left < chunk ? left : chunk;
        const T* whole = static_cast<const T*>(a.logits) + row * a.ld;
        const T* l = whole + first;
        int64_t target = -1;
        float target_logit = 0;
        if (parts == 1 && a.targets != nullptr) {
            target = a.targets[row];
            if (target >= 0 && target < a.vocab) target_logit = to_f32(whole[target]);
        }
        Running run = Running::none();
        Stats before = Stats::none();             // of the runs before this one
        const uint32_t full = n / NV;             // whole vectors
        uint32_t v = tid;
        auto max_of = [&](const raw& r) {
            float x[NV], mx = kLowest;
            Vec<T>::unpack(r, x);
            for (int i = 0; i < NV; ++i) mx = fmaxf(mx, x[i]);
            return mx;
        };
        // The maximum is looked at once for kTogether vectors; mx is the first one's.
        auto take = [&](const raw* r, float mx, auto count) {
            constexpr int kElems = decltype(count)::value * NV;
            float x[kElems];
            for (int u = 0; u < count; ++u) Vec<T>::unpack(r[u], x + u * NV);
            for (int i = NV; i < kElems; ++i) mx = fmaxf(mx, x[i]);
            if (mx > run.m) {
                // (no instruction: keeps the branch, as the few instructions of a seldom
                // raise are a tenth of the pass where every group does them)
                __asm__("" : "+v"(mx));
                run.template raise<ENTROPY>(mx);
            }
            run.template add<ENTROPY, kElems>(x);
        };
        uint32_t end = full < kRun ? full : kRun;
        for (;;) {
            for (; v + (kUnroll - 1) * kThreads < end; v += kUnroll * kThreads) {
                // The last two loads go out once the first has come (777 x 50304 fp32: 25
                // us, 27 us with all four at once; 2048 x 73760: 91 us, 89 us).
                raw r[kUnroll];
                float first;
                for (int u = 0; u < kUnroll; ++u) {
                    if (u == kTogether) __builtin_amdgcn_sched_barrier(0);
                    r[u] = Vec<T>::template load<NT>(l + static_cast<size_t>(v + u * kThreads) * NV);
                    if (u == kTogether - 1) first = max_of(r[0]);
                }
                for (int u = 0; u < kUnroll; u += kTogether)
                    take(r + u, u == 0 ? first : max_of(r[u]), Count<kTogether>{});
            }
            if (end == full) break;
            before = before.with(run.stats());
            run = Running::none();
            end = full - end < kRun ? full : end + kRun;
        }
        for (; v < full; v += kThreads) {
            const raw r = Vec<T>::load(l + static_cast<size_t>(v) * NV);
            take(&r, max_of(r), Count<1>{});
        }
        if (v == full) {                          // the row's last, partial vector
            for (uint32_t i = full * NV; i < n; ++i) {
                const float x = to_f32(l[i]);
                if (x > run.m) run.template raise<ENTROPY>(x);
                run.template add<ENTROPY, 1>(&x);
            }
        }
        const Stats mine = full <= kRun ? run.stats() : before.with(run.stats());
        Stats st = mine.of_wave();
        if (tid % kWave == 0) lds[tid / kWave] = st;
        __syncthreads();
        {
            const float m = fmaxf(fmaxf(lds[0].m, lds[1].m), fmaxf(lds[2].m, lds[3].m));
            const Stats q0 = lds[0].at(m), q1 = lds[1].at(m), q2 = lds[2].at(m), q3 = lds[3].at(m);
            st = Stats{m, (q0.s + q1.s) + (q2.s + q3.s), 0.0f, (q0.t + q1.t) + (q2.t + q3.t)};
        }
        if (st.nearly_certain()) st.r = rest_of<T>(lds_r, &owner, l, n, mine, st);
        const uint64_t* best = nullptr;
        if constexpr (TOP) {
            TopLds& s = *reinterpret_cast<TopLds*>(top_lds);
            choose<T>(s, l, n, first, a.top_k, mine);
            best = s.best;
        }
        if (parts == 1) {
            write_row<TOP>(a, row, st, target_logit, target, best);
        } else {
            char* w = static_cast<char*>(a.workspace) + static_cast<int64_t>(job) * part_bytes(a.top_k);
            if (tid == 0) *reinterpret_cast<Stats*>(w) = st;
            if constexpr (TOP)
                if (tid < a.top_k) reinterpret_cast<uint64_t*>(w + 16)[tid] = best[tid];
        }
        __syncthreads();
    }
}

// Joins the parts of a row.  Every part's best keys are sorted; the first
// ceil(k / parts) of each are at least k keys, so the k-th largest of them
// bounds the row's k-th from below and few keys are left to be ranked.  All
// loads are under way before the first is used: a chain of them is what this
// kernel's time is made of.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a, int parts) {
    constexpr int kHeld = kMaxParts * DL_MAX_TOP / kThreads;
    __shared__ char top_lds[TOP ? sizeof(TopLds) : 1] __attribute__((aligned(16)));
    const int tid = threadIdx.x, held = tid % kMaxParts, k = a.top_k;
    const int64_t bytes = part_bytes(k);
    const int64_t row = blockIdx.x;
    const char* w = static_cast<const char*>(a.workspace) + row * parts * bytes;
    int64_t target = -1;
    float target_logit = 0;
    if (a.targets != nullptr) target = a.targets[row];
    Stats st = Stats::none();
    if (held < parts) st = *reinterpret_cast<const Stats*>(w + held * bytes);
    uint64_t key[kHeld];
    uint32_t head = 0;
    if constexpr (TOP) {
        const int heads = (k + parts - 1) / parts;       // parts * heads < parts + k
        if (tid < parts * heads)
            head = static_cast<uint32_t>(
                reinterpret_cast<const uint64_t*>(w + tid / heads * bytes + 16)[tid % heads] >>
                32);
        for (int u = 0; u < kHeld; ++u) {
            const int i = tid + u * kThreads;
            key[u] = i < parts * k
                         ? reinterpret_cast<const uint64_t*>(w + i / k * bytes + 16)[i % k]
                         : 0;
        }
    }
    if (target >= 0 && target < a.vocab)
        target_logit = to_f32((static_cast<const T*>(a.logits) + row * a.ld)[target]);
    static_assert(kMaxParts == 16, "");
    st = st.of_lanes();
    const uint64_t* best = nullptr;
    if constexpr (TOP) {
        TopLds& s = *reinterpret_cast<TopLds*>(top_lds);
        s.key[tid] = head;
        if (tid == 0) s.count = 0;
        __syncthreads();
        const uint32_t least = kth_bound<sizeof(T) == 2 ? 16 : 20>(s, k);
        for (int u = 0; u < kHeld; ++u)
            if (key[u] != 0 && static_cast<uint32_t>(key[u] >> 32) >= least)
                s.list[atomicAdd(&s.count, 1)] = key[u];
        __syncthreads();
        rank_select(s, s.count, k);
        best = s.best;
    }
    write_row<TOP>(a, row, st, target_logit, target, best);
}

// The gradient: elementwise, one exponential each, bound by the bytes in and
// out.  It is written past the caches, which leaves them to the logits that the
// forward pass has read (333 x 50304 fp32, both passes: 38 us, 47 us with
// ordinary stores).  Elements of a row in chunks of kThreads * kBackUnroll
// vectors.
constexpr int kBackUnroll = 2;

template <typename T, bool ENTROPY>
__global__ __launch_bounds__(kThreads) void k_logprobs_backward(LogprobsBackwardArgs a) {
    constexpr int NV = Vec<T>::n;
    typedef typename Vec<T>::raw raw;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const T* l = static_cast<const T*>(a.logits) + row * a.ld;
        T* dl = static_cast<T*>(a.dlogits) + row * a.ldd;
        const int64_t t = a.targets[row];
        // a row with nothing unmasked: every log p is -infinity
        const float m = a.stats[2 * row] == minus_inf() ? 0.0f : a.stats[2 * row];
        const float log_sum = a.stats[2 * row + 1];
        const float g = t < 0 ? 0.0f : t >= a.vocab ? nan_f() : a.dlogprobs[row];
        const float b = ENTROPY ? a.dentropy[row] : 0.0f;
        const float h = ENTROPY ? a.entropy[row] : 0.0f;
        auto one = [&](float x) {
            const float lp = (x - m) - log_sum, p = exp_of(lp);
            float c = g;
            if constexpr (ENTROPY) c += b * (fmaxf(lp, kFar) + h);
            return -(c * p);
        };
        auto of_target = [&](float x) {
            const float lp = (x - m) - log_sum, p = exp_of(lp);
            float d = -g * expm1f(lp);
            if constexpr (ENTROPY) d -= b * (fmaxf(lp, kFar) + h) * p;
            return d;
        };
        const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kBackUnroll) + threadIdx.x;
        const int64_t full = a.vocab / NV;
        raw r[kBackUnroll];
        for (int u = 0; u < kBackUnroll; ++u)
            if (v0 + u * kThreads < full)
                r[u] = Vec<T>::load(l + (v0 + u * kThreads) * NV);
        for (int u = 0; u < kBackUnroll; ++u) {
            const int64_t v = v0 + u * kThreads, at = v * NV;
            if (v < full) {
                float x[NV], d[NV];
                Vec<T>::unpack(r[u], x);
                for (int i = 0; i < NV; ++i) d[i] = one(x[i]);
                if (t >= at && t < at + NV)
                    for (int i = 0; i < NV; ++i)
                        if (at + i == t) d[i] = of_target(x[i]);
                Vec<T>::template store<true>(dl + at, Vec<T>::pack(d));
            } else if (v == full) {
                for (int64_t i = at; i < a.vocab; ++i) {
                    const float x = to_f32(l[i]);
                    dl[i] = from_f32<T>(i == t ? of_target(x) : one(x));
                }
            }
        }
    }
}

template <typename T, bool ENTROPY, bool TOP>
hipError_t launch(const LogprobsArgs& a, hipStream_t s) {
    const Split sp = split_of(a.rows, a.vocab);
    const int64_t jobs = a.rows * sp.parts;
    const dim3 grid(static_cast<unsigned>(jobs < kMaxGrid ? jobs : kMaxGrid)), block(kThreads);
    if (!TOP && a.rows * a.vocab * static_cast<int64_t>(sizeof(T)) >= kNontemporalMin)
        k_logprobs<T, ENTROPY, TOP, !TOP><<<grid, block, 0, s>>>(a, sp.parts, sp.chunk);
    else
        k_logprobs<T, ENTROPY, TOP, false><<<grid, block, 0, s>>>(a, sp.parts, sp.chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || sp.parts == 1) return e;
    k_logprobs_join<T, TOP>
        <<<dim3(static_cast<unsigned>(a.rows)), dim3(kThreads), 0, s>>>(a, static_cast<int>(sp.parts));
    return hipGetLastError();
}

template <typename T> hipError_t dispatch(const LogprobsArgs& a, hipStream_t s) {
    if (a.entropy != nullptr)
        return a.top_k > 0 ? launch<T, true, true>(a, s) : launch<T, true, false>(a, s);
    return a.top_k > 0 ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

template <typename T> hipError_t backward(const LogprobsBackwardArgs& a, hipStream_t s) {
    const int64_t per = static_cast<int64_t>(kThreads) * kBackUnroll * Vec<T>::n;
    const dim3 grid(static_cast<unsigned>((a.vocab + per - 1) / per),
                    static_cast<unsigned>(a.rows < 65535 ? a.rows : 65535)),
        block(kThreads);
    if (a.dentropy != nullptr) k_logprobs_backward<T, true><<<grid, block, 0, s>>>(a);
    else k_logprobs_backward<T, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top_k) {
    const Split sp = split_of(rows, vocab);
    return sp.parts == 1 ? 0 : rows * sp.parts * part_bytes(top_k);
}

hipError_t logprobs(const LogprobsArgs& a, int dtype, hipStream_t s) {
    return dtype == DL_F32 ? dispatch<float>(a, s) : dispatch<bf16>(a, s);
}

hipError_t logprobs_backward(const LogprobsBackwardArgs& a, int dtype, hipStream_t s) {
    return dtype == DL_F32 ? backward<float>(a, s) : backward<bf16>(a, s);
}

}  // namespace dlk
