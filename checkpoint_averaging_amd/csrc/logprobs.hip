// Log probabilities of given tokens, entropy and the most likely alternatives
// of each row of logits, and their gradient.
//
// With m the row's largest element, d = l - m and e = exp(d):
//   log p = d - log S, S = sum e ;  H = log S - sum(e d) / S
// One pass keeps, against a running maximum, S, the sum R of every e below 1
// and t = sum(e d).  The number of elements equal to the maximum is S - R, so
// where there is one, log S = log1p(R): a nearly certain token's log
// probability and entropy keep their digits, which log(1 + R) would lose.
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
constexpr int64_t kMaxGrid = 1 << 20;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.40282347e38f;
constexpr float kFar = -1e4f;       // exp of this and of anything below is 0

// exp(d) for d <= 0; NaN stays NaN.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

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
    __device__ __forceinline__ void add(float l) {
        if (l > m) raise(l);
        const float d = l - m, e = exp_of(d);
        s += e;
        r += __builtin_amdgcn_fractf(e);      // e if below 1, 0 at the maximum itself
        t += e * fmaxf(d, kFar);
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
        const float ones = rintf(s - r);
        return ones == 1.0f ? log1pf(r) : logf(ones + r);
    }
};

// The order of alternatives: larger logits first, NaN before all, equal ones
// by the lower index.  0 is below every key, ~0 above.
template <typename T> __device__ __forceinline__ uint64_t key_of(T l, int64_t i) {
    const float v = to_f32(l) + 0.0f;         // -0 as 0
    const uint32_t b = __float_as_uint(v);
    const uint32_t u = v != v ? 0xFFFFFFFFu : (b >> 31) != 0 ? ~b : b | 0x80000000u;
    return (static_cast<uint64_t>(u) << 32) | (0x7FFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int64_t index_of(uint64_t key) {
    return 0x7FFFFFFFu - static_cast<uint32_t>(key);
}

// log p of one logit under the row's statistics.
__device__ __forceinline__ float logprob_of(float l, const Stats& st, float log_sum) {
    if (st.nothing()) return __uint_as_float(0xFF800000u);
    return (l - st.m) - log_sum;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobsArgs a) {
    __shared__ Stats lds_s[kWaves];
    __shared__ uint64_t lds_k[kWaves];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* l = static_cast<const T*>(a.logits) + row * a.ld;
    Stats st = Stats::none();
    for (int64_t i = threadIdx.x; i < a.vocab; i += kThreads) st.add(to_f32(l[i]));
    for (int o = kWave / 2; o > 0; o >>= 1) st.merge(st.shuffled(o));
    if (threadIdx.x % kWave == 0) lds_s[threadIdx.x / kWave] = st;
    __syncthreads();
    st = lds_s[0];
    for (int w = 1; w < kWaves; ++w) st.merge(lds_s[w]);
    const float log_sum = st.log_sum();
    if (threadIdx.x == 0) {
        if (a.logprobs != nullptr) {
            const int64_t t = a.targets[row];
            a.logprobs[row] = t < 0 ? 0.0f
                              : t >= a.vocab ? __uint_as_float(0x7FC00000u)
                                             : logprob_of(to_f32(l[t]), st, log_sum);
        }
        if (a.entropy != nullptr)
            a.entropy[row] = st.nothing() ? 0.0f : log_sum - st.t / st.s;
        if (a.stats != nullptr) {
            a.stats[2 * row] = st.nothing() ? __uint_as_float(0xFF800000u) : st.m;
            a.stats[2 * row + 1] = log_sum;
        }
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
        uint64_t best = 0;
        for (int64_t i = threadIdx.x; i < a.vocab; i += kThreads) {
            const uint64_t q = key_of(l[i], i);
            if (q < last && q > best) best = q;
        }
        for (int o = kWave / 2; o > 0; o >>= 1) {
            const uint64_t q = __shfl_xor(static_cast<unsigned long long>(best), o);
            best = q > best ? q : best;
        }
        __syncthreads();
        if (threadIdx.x % kWave == 0) lds_k[threadIdx.x / kWave] = best;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) best = lds_k[w] > best ? lds_k[w] : best;
        last = best;
        if (threadIdx.x == 0) {
            const int64_t id = index_of(best);
            a.top_ids[row * a.top_k + k] = id;
            a.top_logprobs[row * a.top_k + k] = logprob_of(to_f32(l[id]), st, log_sum);
        }
    }
    __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_backward(LogprobsBackwardArgs a) {
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const T* l = static_cast<const T*>(a.logits) + row * a.ld;
    T* dl = static_cast<T*>(a.dlogits) + row * a.ldd;
    const float m = a.stats[2 * row], log_sum = a.stats[2 * row + 1];
    const int64_t t = a.targets[row];
    const bool nothing = m == __uint_as_float(0xFF800000u);
    float g = t < 0 ? 0.0f : a.dlogprobs[row];
    if (t >= a.vocab) g = __uint_as_float(0x7FC00000u);
    const float b = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
    const float h = a.dentropy != nullptr ? a.entropy[row] : 0.0f;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= a.vocab) continue;
    const float lp = nothing ? __uint_as_float(0xFF800000u) : (to_f32(l[i]) - m) - log_sum;
    const float p = exp_of(lp);
    float d = i == t ? -g * expm1f(lp) : -g * p;
    d -= b * p * (fmaxf(lp, kFar) + h);
    dl[i] = from_f32<T>(d);
    }
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t, int64_t, int) { return 0; }

hipError_t logprobs(const LogprobsArgs& a, int dtype, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid)), block(kThreads);
    if (dtype == DL_F32) k_logprobs<float><<<grid, block, 0, s>>>(a);
    else k_logprobs<bf16><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t logprobs_backward(const LogprobsBackwardArgs& a, int dtype, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.vocab + kThreads - 1) / kThreads),
                    static_cast<unsigned>(a.rows < 32768 ? a.rows : 32768)),
        block(kThreads);
    if (dtype == DL_F32) k_logprobs_backward<float><<<grid, block, 0, s>>>(a);
    else k_logprobs_backward<bf16><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dlk
