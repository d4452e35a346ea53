// Log probabilities of given tokens, entropy and the most likely alternatives
// of each row of logits, and their gradient.
//
// With m the row's largest element, d = l - m and e = exp(d):
//   log p = d - log S, S = sum e ;  H = log S - sum(e d) / S
// One pass keeps, against a running maximum, S, the sum R of every e below 1
// and t = sum(e d).  Where S is below 1.5 there is one maximum and S = 1 + R, so
// log S = log1p(R): a nearly certain token's log probability and entropy keep
// their digits, which log(1 + R) would lose.
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
constexpr int64_t kMaxGrid = 1 << 20;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.40282347e38f;
constexpr float kFar = -1e4f;       // exp of this and of anything below is 0
constexpr int kMaxParts = 32;
constexpr int kList = kThreads * 8 + kThreads;   // candidates held at once (see choose)

// exp(d) for d <= 0; NaN stays NaN.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7FC00000u); }
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }

// Running statistics of the elements seen so far.  The first maximum is the
// lowest finite value: an element of -infinity then adds exp(-infinity) = 0,
// one of +infinity or NaN turns S into NaN.
struct Stats {
    float m, s, r, t;

    static __device__ __forceinline__ Stats none() { return Stats{kLowest, 0.0f, 0.0f, 0.0f}; }

    // Moves the maximum up to m2 > m: every element seen is below it.  The
    // distance is cut off where its exponential is 0, or 0 * infinity would
    // make a NaN of it.
    __device__ __forceinline__ void raise(float m2) {
        const float d = fmaxf(m - m2, kFar), a = exp_of(d);
        t = a * (t + d * s);
        s *= a;
        r = s;
        m = m2;
    }
    // Adds an element that is not above the maximum.
    template <bool ENTROPY> __device__ __forceinline__ void add(float l) {
        const float d = l - m, e = exp_of(d);
        s += e;
        r += __builtin_amdgcn_fractf(e);      // e if below 1, 0 at the maximum itself
        if constexpr (ENTROPY) t = __builtin_fmaf(e, fmaxf(d, kFar), t);
    }
    __device__ __forceinline__ void merge(Stats o) {
        if (o.m > m) raise(o.m);
        else if (m > o.m) o.raise(m);
        s += o.s;
        r += o.r;
        t += o.t;
    }
    __device__ __forceinline__ Stats shuffled(int o) const {
        Stats q;
        q.m = __shfl_xor(m, o);
        q.s = __shfl_xor(s, o);
        q.r = __shfl_xor(r, o);
        q.t = __shfl_xor(t, o);
        return q;
    }
    __device__ __forceinline__ bool nothing() const { return s == 0.0f; }
    __device__ __forceinline__ float log_sum() const {
        if (nothing()) return 0.0f;
        return s < 1.5f ? log1pf(r) : logf(s);
    }
};

// The order of alternatives as whole numbers: larger logits first, NaN before
// all, and in a full key equal ones by the lower index.  0 is below every
// key, ~0 above.
__device__ __forceinline__ uint32_t order_of(float l) {
    const float v = l + 0.0f;                 // -0 as 0
    const uint32_t b = __float_as_uint(v);
    return v != v ? 0xFFFFFFFFu : (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(uint32_t order, int64_t i) {
    return (static_cast<uint64_t>(order) << 32) | (0x7FFFFFFFu - static_cast<uint32_t>(i));
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
    uint32_t key[kThreads];
    int cand[kThreads];
    int count, cands;
    uint32_t least;
};

// best[0..k) = the k largest of the `count` distinct keys of list[], largest
// first; 0 where there are fewer.  An element's place is the number of larger
// ones.
__device__ __forceinline__ void rank_select(TopLds& s, int count, int k) {
    if (threadIdx.x < static_cast<unsigned>(k)) s.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t q = s.list[i];
        int rank = 0;
        for (int j = 0; j < count; ++j) rank += s.list[j] > q;
        if (rank < k) s.best[rank] = q;
    }
    __syncthreads();
}

// best[0..k) of the elements [0, n) of l, whose index in the row is `first`
// more, from the threads' own statistics of a pass in which thread t took the
// vectors t, t + kThreads, ...
//
// The k-th largest of the threads' maxima is a lower bound of the k-th largest
// element, and only threads whose maximum reaches it hold elements that do:
// about k threads' vectors are read once more (out of a cache), spread over
// all threads.  Elements that reach the bound go to a list; when a round may
// overflow it, the list is cut to its k largest, whose last then is a bound
// too (rows of many equal or ordered elements).
template <typename T>
__device__ __forceinline__ void choose(TopLds& s, const T* l, int64_t n, int64_t first, int k,
                                       const Stats& mine) {
    constexpr int NV = Vec<T>::n;
    const int tid = threadIdx.x;
    // The thread's maximum, rounded down to make room for its number: distinct keys.
    uint32_t key = 0;                         // no elements
    if (static_cast<int64_t>(tid) * NV < n)
        key = mine.s != mine.s ? 0xFF800000u  // NaN or +infinity: at least +infinity
              : mine.nothing() ? 0x007FFFFFu  // -infinity
                               : order_of(mine.m);
    key = (key & ~0xFFu) | static_cast<uint32_t>(tid);
    s.key[tid] = key;
    if (tid == 0) s.count = s.cands = 0;
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < kThreads; j += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(&s.key[j]);
        rank += (q.x > key) + (q.y > key) + (q.z > key) + (q.w > key);
    }
    if (rank == k - 1) s.least = key & ~0xFFu;
    __syncthreads();
    const uint32_t least = s.least;
    if ((key & ~0xFFu) >= least) s.cand[atomicAdd(&s.cands, 1)] = tid;
    __syncthreads();
    const uint32_t cands = s.cands;
    // (fewer than 2^31 / NV vectors, so whole numbers of 32 bits hold these)
    const uint32_t vectors = static_cast<uint32_t>((n + NV - 1) / NV);
    const uint32_t steps = (vectors + kThreads - 1) / kThreads;
    uint64_t bound = 0;
    for (uint32_t p0 = 0; p0 < steps * cands; p0 += kThreads) {
        const uint32_t p = p0 + tid;
        if (p < steps * cands) {
            const int64_t at = static_cast<int64_t>(p / cands * kThreads + s.cand[p % cands]) * NV;
            if (at < n) {
                float x[NV];
                if (at + NV <= n) {
                    Vec<T>::unpack(*reinterpret_cast<const typename Vec<T>::raw*>(l + at), x);
                } else {
                    for (int i = 0; i < NV; ++i) x[i] = at + i < n ? to_f32(l[at + i]) : 0.0f;
                }
                for (int i = 0; i < NV; ++i) {
                    const uint32_t o = order_of(x[i]);
                    const uint64_t q = key_of(o, first + at + i);
                    if (at + i < n && o >= least && q > bound) s.list[atomicAdd(&s.count, 1)] = q;
                }
            }
        }
        __syncthreads();
        const int count = s.count;
        __syncthreads();                      // read by all before the next round adds to it
        if (count > kList - kThreads * NV) {
            rank_select(s, count, k);
            if (tid < k) s.list[tid] = s.best[tid];
            bound = s.best[k - 1];
            if (tid == 0) s.count = k;
            __syncthreads();
        }
    }
    rank_select(s, s.count, k);
}

// What a row is split into: `parts` workgroups of `chunk` elements each.
struct Split {
    int parts;
    int64_t chunk;
};

Split split_of(int64_t rows, int64_t vocab) {
    const int64_t least = 4096;
    int64_t parts = (1024 + rows - 1) / rows;
    parts = parts < kMaxParts ? parts : kMaxParts;
    const int64_t most = (vocab + least - 1) / least;
    parts = parts < most ? parts : most;
    const int64_t chunk = ((vocab + parts - 1) / parts + 7) / 8 * 8;
    return Split{static_cast<int>((vocab + chunk - 1) / chunk), chunk};
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

// One workgroup a part of a row; with one part a row, the results themselves.
template <typename T, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobsArgs a, int parts, int64_t chunk) {
    constexpr int NV = Vec<T>::n;
    typedef typename Vec<T>::raw raw;
    __shared__ Stats lds[kWaves];
    __shared__ char top_lds[TOP ? sizeof(TopLds) : 1] __attribute__((aligned(16)));
    const int tid = threadIdx.x;
    for (int64_t job = blockIdx.x; job < a.rows * parts; job += gridDim.x) {
        const int64_t row = job / parts;
        const int part = static_cast<int>(job - row * parts);
        const int64_t first = part * chunk;
        const int64_t n = a.vocab - first < chunk ? a.vocab - first : chunk;
        const T* whole = static_cast<const T*>(a.logits) + row * a.ld;
        const T* l = whole + first;
        int64_t target = -1;
        float target_logit = 0;
        if (parts == 1 && a.targets != nullptr) {
            target = a.targets[row];
            if (target >= 0 && target < a.vocab) target_logit = to_f32(whole[target]);
        }
        Stats st = Stats::none();
        const int64_t full = n / NV;              // whole vectors
        int64_t v = tid;
        auto take = [&](const raw& r) {
            float x[NV];
            Vec<T>::unpack(r, x);
            float mx = x[0];
            for (int i = 1; i < NV; ++i) mx = fmaxf(mx, x[i]);
            if (mx > st.m) st.raise(mx);
            for (int i = 0; i < NV; ++i) st.template add<ENTROPY>(x[i]);
        };
        for (; v + (kUnroll - 1) * kThreads < full; v += kUnroll * kThreads) {
            raw r[kUnroll];
            for (int u = 0; u < kUnroll; ++u)
                r[u] = *reinterpret_cast<const raw*>(l + (v + u * kThreads) * NV);
            for (int u = 0; u < kUnroll; ++u) take(r[u]);
        }
        for (; v < full; v += kThreads) take(*reinterpret_cast<const raw*>(l + v * NV));
        if (v == full) {                          // the row's last, partial vector
            for (int64_t i = full * NV; i < n; ++i) {
                const float x = to_f32(l[i]);
                if (x > st.m) st.raise(x);
                st.template add<ENTROPY>(x);
            }
        }
        const Stats mine = st;
        for (int o = kWave / 2; o > 0; o >>= 1) st.merge(st.shuffled(o));
        if (tid % kWave == 0) lds[tid / kWave] = st;
        __syncthreads();
        st = lds[0];
        for (int w = 1; w < kWaves; ++w) st.merge(lds[w]);
        const uint64_t* best = nullptr;
        if constexpr (TOP) {
            TopLds& s = *reinterpret_cast<TopLds*>(top_lds);
            choose<T>(s, l, n, first, a.top_k, mine);
            best = s.best;
        }
        if (parts == 1) {
            write_row<TOP>(a, row, st, target_logit, target, best);
        } else {
            char* w = static_cast<char*>(a.workspace) + job * part_bytes(a.top_k);
            if (tid == 0) *reinterpret_cast<Stats*>(w) = st;
            if constexpr (TOP)
                if (tid < a.top_k) reinterpret_cast<uint64_t*>(w + 16)[tid] = best[tid];
        }
        __syncthreads();
    }
}

// Joins the parts of a row.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a, int parts) {
    __shared__ char top_lds[TOP ? sizeof(TopLds) : 1] __attribute__((aligned(16)));
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* w = static_cast<const char*>(a.workspace) + row * parts * part_bytes(a.top_k);
        int64_t target = -1;
        float target_logit = 0;
        if (a.targets != nullptr) {
            target = a.targets[row];
            if (target >= 0 && target < a.vocab)
                target_logit = to_f32((static_cast<const T*>(a.logits) + row * a.ld)[target]);
        }
        Stats st = *reinterpret_cast<const Stats*>(w);
        for (int p = 1; p < parts; ++p)
            st.merge(*reinterpret_cast<const Stats*>(w + p * part_bytes(a.top_k)));
        const uint64_t* best = nullptr;
        if constexpr (TOP) {
            TopLds& s = *reinterpret_cast<TopLds*>(top_lds);
            const int k = a.top_k;
            for (int i = tid; i < parts * k; i += kThreads)
                s.list[i] = reinterpret_cast<const uint64_t*>(w + i / k * part_bytes(k) + 16)[i % k];
            __syncthreads();
            rank_select(s, parts * k, k);
            best = s.best;
        }
        write_row<TOP>(a, row, st, target_logit, target, best);
        __syncthreads();
    }
}

// Elements of a row in chunks of kThreads * kBackUnroll vectors.
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
                r[u] = *reinterpret_cast<const raw*>(l + (v0 + u * kThreads) * NV);
        for (int u = 0; u < kBackUnroll; ++u) {
            const int64_t v = v0 + u * kThreads, at = v * NV;
            if (v < full) {
                float x[NV], d[NV];
                Vec<T>::unpack(r[u], x);
                for (int i = 0; i < NV; ++i) d[i] = one(x[i]);
                if (t >= at && t < at + NV)
                    for (int i = 0; i < NV; ++i)
                        if (at + i == t) d[i] = of_target(x[i]);
                *reinterpret_cast<raw*>(dl + at) = Vec<T>::pack(d);
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
    const dim3 block(kThreads);
    k_logprobs<T, ENTROPY, TOP><<<dim3(static_cast<unsigned>(jobs < kMaxGrid ? jobs : kMaxGrid)),
                                  block, 0, s>>>(a, sp.parts, sp.chunk);
    if (sp.parts > 1) {
        if (hipError_t e = hipGetLastError()) return e;
        k_logprobs_join<T, TOP><<<dim3(static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid)),
                                  block, 0, s>>>(a, sp.parts);
    }
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
