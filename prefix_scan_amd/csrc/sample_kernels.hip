// sample_kernels.hip -- one token from each row of logits.
//
// The kept tokens are a prefix of the row in order of falling logit, so they
// are known by the key K of the last one and how many of the tokens equal to
// it (by rising index) are in.  top_k and top_p each find such a cut by
// digits: a histogram of the keys' top digit (counts for top_k, weights for
// top_p) tells which digit the cut falls in, and the next digit is looked at
// among the keys that share it.  No row is sorted.
//
// Weights are e^((x - M) / T) in 64 bits, held as 64-bit fixed point: sums
// (by LDS atomics, by waves, in any order) are exact, so the cut and the
// drawn token depend on the inputs alone.
#include "sample.hpp"

namespace libscan {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct Row {
    float temperature, top_p, min_p, u;
    int32_t top_k;
};

__device__ __forceinline__ Row row_of(const sample_args_t &a, uint64_t r)
{
    Row p;
    p.temperature = a.temperatures ? a.temperatures[r] : a.temperature;
    p.top_p = a.top_ps ? a.top_ps[r] : a.top_p;
    p.min_p = a.min_ps ? a.min_ps[r] : a.min_p;
    p.top_k = a.top_ks ? a.top_ks[r] : a.top_k;
    p.u = a.u[r];
    return p;
}

// Order-preserving u32 of a logit; 0 for what is never kept (NaN, -inf).
// Both zeros have one key.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (!(x > -__builtin_inff()))
        return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The weight of a key against the largest logit: 0 <= w <= 1, 1 at the top.
struct Weigh {
    double top, over_t, one;     // M, 1 / T's divisor, the fixed-point one
    float t;
    __device__ __forceinline__ double real(uint32_t key) const
    {
        const double x = (double)logit_of(key);
        if (x == top)            // also +inf
            return 1.0;
        return exp((x - top) / over_t);
    }
    __device__ __forceinline__ uint64_t fixed(double w) const { return (uint64_t)ceil(w * one); }
};

__device__ __forceinline__ uint64_t wave_sum64(uint64_t x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        x += __shfl_xor((unsigned long long)x, d);
    return x;
}

__device__ __forceinline__ uint64_t wave_incl64(uint64_t x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t y = __shfl_up((unsigned long long)x, d);
        if ((int)(threadIdx.x & 63) >= d)
            x += y;
    }
    return x;
}

struct Shared {
    unsigned long long hist[256];
    unsigned long long part[kWaves];
    unsigned long long best[kWaves];
    unsigned long long word;
    uint32_t digit, count;
    int token;
};

__device__ __forceinline__ uint64_t block_sum64(uint64_t x, Shared &s)
{
    x = wave_sum64(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        s.part[threadIdx.x / 64] = x;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        t += s.part[w];
    return t;
}

// A cut: keys above `key` are in, and `ties` of those equal to it.
struct Cut {
    uint32_t key, ties;
};

template <class T>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(const sample_args_t a, int shift)
{
    __shared__ Shared s;
    const uint64_t r = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + (int64_t)r * a.row_stride;
    const uint32_t n = (uint32_t)a.vocab;
    const Row p = row_of(a, r);
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;

    // The largest logit and its lowest index.
    unsigned long long best = 0;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t k = key_of((float)x[i]);
        const unsigned long long c = ((unsigned long long)k << 32) | (0xFFFFFFFFu - i);
        if (k && c > best)
            best = c;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const unsigned long long o = __shfl_xor(best, d);
        best = o > best ? o : best;
    }
    if (lane == 0)
        s.best[wave] = best;
    __syncthreads();
    best = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        best = s.best[w] > best ? s.best[w] : best;
    const bool greedy = !(p.temperature > 0.f);
    if (best == 0 || greedy) {
        if (threadIdx.x == 0) {
            a.tokens[r] = best ? (int32_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
            if (a.logprobs)
                a.logprobs[r] = best ? 0.f : -__builtin_inff();
            if (a.kept)
                a.kept[r] = best ? 1 : 0;
        }
        return;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    Weigh wt;
    wt.top = (double)logit_of(top_key);
    wt.over_t = (double)p.temperature;
    wt.one = (double)(1ull << shift);
    const double min_w = p.min_p > 0.f ? (p.min_p < 1.f ? (double)p.min_p : 1.0) : 0.0;

    Cut cut = {0u, 0u};
    // top_k: the key of the k-th token.
    if (p.top_k > 0 && (uint32_t)p.top_k < n) {
        uint32_t prefix = 0, need = (uint32_t)p.top_k;
        bool all = false;
        for (int b = 24; b >= 0 && !all; b -= 8) {
            __syncthreads();
            if (threadIdx.x < 256)
                s.hist[threadIdx.x] = 0;
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
                const uint32_t k = key_of((float)x[i]);
                if (k && (b == 24 || (k >> (b + 8)) == prefix))
                    atomicAdd(&s.hist[(k >> b) & 255], 1ull);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t above = 0;
                int d = 255;
                for (; d >= 0; --d) {
                    if (above + s.hist[d] >= need)
                        break;
                    above += (uint32_t)s.hist[d];
                }
                s.digit = (uint32_t)d;          // -1: fewer than k tokens in all
                s.count = above;
            }
            __syncthreads();
            if ((int)s.digit < 0) {
                all = true;
            } else {
                need -= s.count;
                prefix = (prefix << 8) | s.digit;
            }
        }
        if (!all)
            cut = {prefix, need};
    }

    // What the cut and min_p leave, and its weight.
    const double cut_w = cut.key ? wt.real(cut.key) : 0.0;
    const uint64_t tie_weight = cut.key && cut_w >= min_w ? cut.ties * wt.fixed(cut_w) : 0;
    const bool nucleus = p.top_p < 1.f;
    if (nucleus) {
        uint64_t sum = 0;
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t k = key_of((float)x[i]);
            if (k > cut.key) {
                const double w = wt.real(k);
                if (w >= min_w)
                    sum += wt.fixed(w);
            }
        }
        const uint64_t total = block_sum64(sum, s) + tie_weight;
        const double want = p.top_p > 0.f ? ceil((double)p.top_p * (double)total) : 1.0;
        uint64_t need = want < 1.0 ? 1 : (uint64_t)want;
        if (need > total)
            need = total;
        uint32_t prefix = 0;
        for (int b = 24; b >= 0; b -= 8) {
            __syncthreads();
            if (threadIdx.x < 256)
                s.hist[threadIdx.x] = 0;
            __syncthreads();
            if (threadIdx.x == 0 && tie_weight && (b == 24 || (cut.key >> (b + 8)) == prefix))
                atomicAdd(&s.hist[(cut.key >> b) & 255], (unsigned long long)tie_weight);
            for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
                const uint32_t k = key_of((float)x[i]);
                if (k > cut.key && (b == 24 || (k >> (b + 8)) == prefix)) {
                    const double w = wt.real(k);
                    if (w >= min_w)
                        atomicAdd(&s.hist[(k >> b) & 255], (unsigned long long)wt.fixed(w));
                }
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                uint64_t above = 0;
                int d = 255;
                for (; d > 0; --d) {
                    if (above + s.hist[d] >= need)
                        break;
                    above += s.hist[d];
                }
                s.digit = (uint32_t)d;
                s.word = above;
            }
            __syncthreads();
            need -= s.word;
            prefix = (prefix << 8) | s.digit;
        }
        const uint64_t each = wt.fixed(wt.real(prefix));
        cut = {prefix, (uint32_t)((need + each - 1) / each)};
    }

    // Every wave has a contiguous part of the row: its ties before it, then
    // the kept weight before it, then the token.
    const uint32_t per = (n + kWaves * 64 - 1) / (kWaves * 64) * 64;
    const uint32_t lo = wave * per < n ? wave * per : n, hi = lo + per < n ? lo + per : n;
    uint32_t ties = 0;
    if (cut.key) {
        for (uint32_t i = lo; i < hi; i += 64) {
            const uint32_t k = i + lane < hi ? key_of((float)x[i + lane]) : 0u;
            ties += __popcll(__ballot(k == cut.key));
        }
    }
    __syncthreads();
    if (lane == 0)
        s.part[wave] = ties;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w)
        before += (uint32_t)s.part[w];
    const auto kept_weight = [&](uint32_t i, uint32_t &rank, bool &in) -> uint64_t {
        const uint32_t k = i + lane < hi ? key_of((float)x[i + lane]) : 0u;
        const uint64_t same = __ballot(cut.key && k == cut.key);
        const uint32_t mine = rank + __popcll(same & ((1ull << lane) - 1));
        rank += __popcll(same);
        in = k > cut.key || (cut.key && k == cut.key && mine < cut.ties);
        if (!in)
            return 0;
        const double w = wt.real(k);
        in = w >= min_w;
        return in ? wt.fixed(w) : 0;
    };
    uint64_t sum = 0;
    uint32_t held = 0, rank = before;
    for (uint32_t i = lo; i < hi; i += 64) {
        bool in;
        sum += kept_weight(i, rank, in);
        held += in;
    }
    sum = wave_sum64(sum);
    const uint64_t count = block_sum64(held, s);
    __syncthreads();
    if (lane == 0)
        s.part[wave] = sum;
    __syncthreads();
    uint64_t total = 0, base = 0;
    for (int w = 0; w < kWaves; ++w) {
        base += w < wave ? s.part[w] : 0;
        total += s.part[w];
    }
    const double uz = p.u > 0.f ? (double)p.u * (double)total : 0.0;
    uint64_t want = uz < (double)total ? (uint64_t)uz : total - 1;
    if (want > total - 1)
        want = total - 1;
    if (base <= want && want < base + sum) {
        rank = before;
        for (uint32_t i = lo; i < hi; i += 64) {
            bool in;
            const uint64_t w = kept_weight(i, rank, in);
            const uint64_t incl = base + wave_incl64(w);
            const uint64_t hit = __ballot(incl > want);
            if (hit) {
                if (lane == __ffsll((unsigned long long)hit) - 1) {
                    a.tokens[r] = (int32_t)(i + lane);
                    if (a.logprobs) {
                        const double d = wt.real(key_of((float)x[i + lane])) == 1.0
                                             ? 0.0 : ((double)(float)x[i + lane] - wt.top) / wt.over_t;
                        a.logprobs[r] = (float)(d - log((double)total / wt.one));
                    }
                }
                break;
            }
            base = __shfl((unsigned long long)incl, 63);
        }
    }
    if (threadIdx.x == 0 && a.kept)
        a.kept[r] = (int32_t)count;
}

}  // namespace

size_t sample_body_bytes(uint64_t, uint64_t) { return 0; }

hipError_t launch_sample(const sample_args_t &a, void *, hipStream_t stream)
{
    int bits = 0;
    while ((1ull << bits) < a.vocab)
        ++bits;
    const unsigned rows = (unsigned)a.rows;
    switch (a.dtype) {
    case LIBSCAN_F32: sample_row_kernel<float><<<rows, kThreads, 0, stream>>>(a, 62 - bits); break;
    case LIBSCAN_BF16: sample_row_kernel<__bf16><<<rows, kThreads, 0, stream>>>(a, 62 - bits); break;
    default: sample_row_kernel<_Float16><<<rows, kThreads, 0, stream>>>(a, 62 - bits); break;
    }
    return hipGetLastError();
}

}  // namespace libscan
