// sample_kernels.hip -- one token from each row of logits.
//
// The kept tokens are a prefix of the row in order of falling logit, so they
// are known by the last one: its key (the logit in an order-preserving u32)
// and its index, the largest kept one of that key.  No row is sorted, and a
// row is read three times at most before its token is drawn:
//
//   max      the largest logit M and its lowest index; with a small top_k, a
//            maximum of each lane's share of the row too.  The k-th largest
//            of those is no larger than the k-th largest logit, so what lies
//            below it is out and the histogram is not needed;
//   hist     for other cuts, a histogram over 2048 bins of M - x (64 to a
//            binade, so that they are fine where the weight is, whatever the
//            logits' scale): counts for top_k, weights for top_p;
//   collect  the bin that the cut falls in is known; what lies above it is
//            in, and its weight is summed by blocks of the row; the bin's own
//            tokens go to a list.  With top_k, all that lies above goes to
//            the list too;
//   draw     one workgroup a row finds the cut in the list by digits (of the
//            key, then of the index among equal keys), and the token by
//            digits of its index, or by the blocks' sums and a second look
//            at one block.
// A row is cut into parts over `max`, `hist` and `collect`, so that few long
// rows fill the GPU too.  A list that would be too long (thousands of equal
// logits at the cut, or top_k in the thousands) is not used: `draw` takes the
// digits over the row itself.
//
// What bounds it, at 512 bf16 rows of 150001 (154 MB, 23 us of reading) with
// all kinds of cuts: max 28 us (5.5 TB/s, memory), hist 65 and collect 64 (the
// issue of instructions: ten 64-bit ones a weight and as many 32-bit ones a
// logit), draw 39.  One row of 32000: 3, 5, 8 and 12 us, the latency of four
// kernels that depend on each other.
//
// Weights are 2^((x - M) log2 e / T) in 64 bits, held as 64-bit fixed point:
// sums (by LDS and global atomics, in any order) are exact, so the cut and
// the drawn token depend on the inputs alone.
#include "sample.hpp"

#include "device_common.hpp"

#include <type_traits>

namespace libscan {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kList = 8192;            // longest list of a row
constexpr uint32_t kBuf = 1024;             // entries a workgroup gathers before it appends them
constexpr uint32_t kMaxima = 2048;          // most of a row
constexpr uint32_t kMaxBlocks = 1024;       // of a row
constexpr uint32_t kHeld = 2048;            // longest list that `draw` holds in LDS, with its weights
constexpr unsigned long long kIn = 1ull << 63;      // of a held weight: min_p leaves the token

struct Setting {
    float temperature, top_p, min_p, u;
    int32_t top_k;
};

__device__ __forceinline__ Setting setting_of(const sample_args_t &a, uint64_t r)
{
    Setting p;
    p.temperature = a.temperatures ? a.temperatures[r] : a.temperature;
    p.top_p = a.top_ps ? a.top_ps[r] : a.top_p;
    p.min_p = a.min_ps ? a.min_ps[r] : a.min_p;
    p.top_k = a.top_ks ? a.top_ks[r] : a.top_k;
    p.u = a.u[r];
    return p;
}

// How a row is cut: kFew is a top_k that the lanes' maxima bound.  Against the
// histogram, top_k 1, 50 and 900: 36, 47 and 62 us, not 46, 57 and 69, for 48
// rows of 128000; 82, 89 and 122, not 125, 138 and 174, for 512 of 150001; one
// row of 32000 takes the same either way (22, 27 and 37).  Past half as many
// as there are maxima the bound lets too much through.
enum { kAll, kFew, kTopK, kNucleus };

__device__ __forceinline__ int cut_of(const Setting &p, uint32_t n, uint32_t maxima)
{
    if (p.top_k > 0 && (uint32_t)p.top_k < n)
        return (uint32_t)p.top_k <= maxima / 2 ? kFew : kTopK;
    return p.top_p < 1.f ? kNucleus : kAll;
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

// M - x is exact or rounded the same way for all, so bins never cross keys.
__device__ __forceinline__ uint32_t bin_of(float top, float x)
{
    const float d = x == top ? 0.f : top - x;
    const int b = (int)(__float_as_uint(d) >> 17) - ((127 - 10) << 6);
    return (uint32_t)(b < 0 ? 0 : b > (int)kBins - 1 ? (int)kBins - 1 : b);
}

// The smallest logit in bins 0 .. bin: logits from it on are in them.  For
// all lanes of a wave alike.
__device__ __forceinline__ float from_bin(float top, uint32_t bin)
{
    uint32_t in = key_of(top), out = 0x007FFFFFu;       // -inf's key
    if (bin >= kBins - 1)
        return -3.402823466e38f;
    // Mostly within a step of the top less the bin's far end.
    const uint32_t near = key_of(top - __uint_as_float((bin + 1 + ((127 - 10) << 6)) << 17));
    if (near > out + 1 && near + 2 < in) {
        const bool a = bin_of(top, logit_of(near - 1)) <= bin, b = bin_of(top, logit_of(near)) <= bin,
                   c = bin_of(top, logit_of(near + 1)) <= bin, d = bin_of(top, logit_of(near + 2)) <= bin;
        if (!a && d)
            return logit_of(b ? near : c ? near + 1 : near + 2);
    }
#pragma unroll 1
    while (in - out > 1) {
        const uint32_t mid = out + (in - out) / 2;
        if (bin_of(top, logit_of(mid)) <= bin)
            in = mid;
        else
            out = mid;
    }
    return logit_of(in);
}

// Weights.  w = 2^y with y = (x - M) log2 e / T is 2^e times entry i of a table
// of 2^(i / 512) times a cubic of the 2^-10 that are left.  The cubic is 2^-46
// off, and so is 1 / T, rounded, times what does not round to zero (y of 52).  The
// exponent goes into the table's entry, so that one product and sum rounds it
// to the fixed-point word.  Ten 64-bit operations a weight, which bound a pass
// over rows without a cut: 512 x 150001 logits take 113 us.
constexpr int kPowers = 512;
enum { kPlain, kMin, kInfinite };

// The table, times the fixed-point one.
__device__ __forceinline__ void fill_powers(double *t, int shift)
{
    for (int i = threadIdx.x; i < kPowers; i += kThreads)
        t[i] = ldexp(exp2((double)i / kPowers), shift);
}

struct Weigh {
    double top, by, one;         // M, 512 log2 e / T, the fixed-point one
    double least;                // min_p, times one
    float floor;                 // logits below this weigh nothing, and count as this one
    bool top_only;               // M = +inf: only its equals weigh
    const double *pow;

    __device__ __forceinline__ Weigh(int shift, float temperature, float min_p, float most_likely,
                                     const double *powers)
    {
        pow = powers;
        top = (double)most_likely;
        one = (double)(1ull << shift);
        top_only = most_likely == __builtin_inff();
        // e^-111 < 2^-149, the least min_p there is.
        floor = most_likely - 111.f * temperature;
        if (!(floor < most_likely))
            floor = logit_of(key_of(most_likely) - 1);
        by = kPowers * 1.4426950408889634074 / (double)temperature;
        const double most = kPowers * 1000.0 / (top - (double)floor);
        by = by < most ? by : most;
        least = min_p > 0.f ? (min_p < 1.f ? (double)min_p : 1.0) * one : 0.0;
    }
    // The weight of a logit, in fixed point (one <= 2^51): 2^-45 of it off, and
    // half a unit by its rounding to a word; and whether min_p leaves it.  HOW:
    // no min_p, one, or M = +inf; without a branch, so that several go through
    // at a time.
    template <int HOW>
    __device__ __forceinline__ uint64_t fixed(float x, bool &in) const
    {
        if constexpr (HOW == kInfinite) {
            in = x == __builtin_inff() || least == 0.0;
            return x == __builtin_inff() ? (uint64_t)one : 0;
        }
        const double d = (double)fmaxf(x, floor) - top;
        const double magic = 6755399441055744.0;               // 1.5 * 2^52
        const double t = __builtin_fma(d, by, magic);
        const int k = (int)(uint32_t)__double_as_longlong(t);
        const double r = __builtin_fma(d, by, magic - t);      // 512ths that are left
        constexpr double c = 0.6931471805599453094 / kPowers;
        double p = __builtin_fma(r, c * c * c / 6, c * c / 2);
        p = __builtin_fma(p, r, c);
        p = __builtin_fma(p, r, 1.0);
        // Exponents of 160 below the table's at least.
        const double scale = __longlong_as_double(__double_as_longlong(pow[k & (kPowers - 1)]) +
                                                  ((int64_t)(k >> 9) << 52));
        in = HOW == kPlain || scale * p >= least;
        const double w = __builtin_fma(scale, p, 4503599627370496.0);
        return (uint64_t)__double_as_longlong(w) & 0xFFFFFFFFFFFFFull;
    }
    // f(HOW) for this row's.
    template <class F>
    __device__ __forceinline__ void how(F f) const
    {
        const int h = __builtin_amdgcn_readfirstlane(top_only ? kInfinite : least > 0.0 ? kMin : kPlain);
        if (h == kPlain)
            f(std::integral_constant<int, kPlain>());
        else if (h == kMin)
            f(std::integral_constant<int, kMin>());
        else
            f(std::integral_constant<int, kInfinite>());
    }
};

// For whole waves.
__device__ __forceinline__ uint64_t wave_sum64(uint64_t x)
{
    const uint64_t t = wave_incl64_add(x);
    return (uint64_t)__builtin_amdgcn_readlane((uint32_t)(t >> 32), 63) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)t, 63);
}

// A row in granules of 8 logits, counted from the 16-byte boundary at or
// before its start, so that all but the first and the last are whole
// 16-byte loads wherever the row starts.
template <class T>
struct RowOf {
    const T *x;
    uint32_t n, skew;
    __device__ __forceinline__ RowOf(const sample_args_t &a, uint64_t r)
        : x(static_cast<const T *>(a.logits) + (int64_t)r * a.row_stride), n((uint32_t)a.vocab)
    {
        skew = (uint32_t)((uintptr_t)x & 15) / (uint32_t)sizeof(T);
    }
    // Index of a granule's first logit (negative in the first one, maybe).
    __device__ __forceinline__ int64_t first(uint32_t granule) const { return (int64_t)granule * 8 - skew; }
    // Eight logits as they lie in memory; outside the row -inf.
    struct Raw {
        T v[8] __attribute__((aligned(16)));
    };
    __device__ __forceinline__ Raw raw(uint32_t granule) const
    {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const int64_t i = first(granule);
        Raw r;
        if (i >= 0 && i + 8 <= (int64_t)n) {
            u32x4 t[sizeof(T) / 2];
#pragma unroll
            for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                t[h] = reinterpret_cast<const u32x4 *>(x + i)[h];
            __builtin_memcpy(&r, t, sizeof(r));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r.v[e] = i + e >= 0 && i + e < (int64_t)n ? x[i + e] : (T)-__builtin_inff();
        }
        return r;
    }
    __device__ __forceinline__ void load(uint32_t granule, float (&v)[8]) const
    {
        const Raw r = raw(granule);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = (float)r.v[e];
    }
    // f(granule, logits) for `count` wave steps from the one at `from` on, each
    // read while the four before are looked at.
    template <class F>
    __device__ __forceinline__ void steps(uint32_t from, uint32_t count, F f) const
    {
        constexpr uint32_t AHEAD = 4;
        const uint32_t lane = threadIdx.x & 63;
        Raw r[AHEAD];
#pragma unroll
        for (uint32_t j = 0; j < AHEAD; ++j)
            if (j < count)
                r[j] = raw((from + j) * 64 + lane);
        for (uint32_t i = 0; i < count; i += AHEAD) {
#pragma unroll
            for (uint32_t j = 0; j < AHEAD; ++j) {
                if (i + j < count) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = (float)r[j].v[e];
                    if (i + j + AHEAD < count)
                        r[j] = raw((from + i + j + AHEAD) * 64 + lane);
                    f((from + i + j) * 64 + lane, v);
                }
            }
        }
    }
};

// How rows are cut.  A wave step is 64 granules; blocks of `steps` of them
// have a sum of kept weights each, and a wave has `blocks` blocks.
struct BinCut;

struct Geometry {
    uint32_t parts, blocks, steps, row_blocks, list;
    uint32_t maxima, share;       // maxima of a row, and lanes that have one together
    uint32_t halves;              // 2: a lane has one of each half of its steps
    int shift;
    uint64_t row0;
    // scratch, rows from row0 on
    unsigned long long *best;     // [rows][parts]
    float *tops;                  // [rows][maxima]
    unsigned long long *hist;     // [rows][kBins]
    unsigned long long *sums;     // [rows][row_blocks]
    unsigned long long *entries;  // [rows][list]: key, index
    uint32_t *counts;             // [rows][row_blocks]
    uint32_t *length;             // [rows]
    BinCut *cut;                  // [rows]
};

__device__ __forceinline__ unsigned long long best_of(const Geometry &g, uint32_t row, int lane)
{
    unsigned long long best = 0;
    for (uint32_t i = lane; i < g.parts; i += 64) {
        const unsigned long long o = g.best[(uint64_t)row * g.parts + i];
        best = o > best ? o : best;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const unsigned long long o = __shfl_xor(best, d);
        best = o > best ? o : best;
    }
    return best;
}

__device__ __forceinline__ Weigh weigh_of(const Geometry &g, const Setting &p, float top, const double *pow)
{
    return Weigh(g.shift, p.temperature, p.min_p, top, pow);
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ unsigned long long s_best[kWaves];
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    const int kind = cut_of(setting_of(a, g.row0 + row), x.n, g.maxima);
    if (kind == kTopK || kind == kNucleus)
        for (uint32_t i = part * kThreads + threadIdx.x; i < kBins; i += g.parts * kThreads)
            g.hist[(uint64_t)row * kBins + i] = 0;
    if (part == 0 && threadIdx.x == 0)
        g.length[row] = 0;
    const uint32_t per = g.blocks * g.steps, from = (part * kWaves + wave) * per;
    float top = -__builtin_inff(), half_top = -__builtin_inff();
    uint32_t at = 0;
    const auto look = [&](uint32_t granule, const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (v[e] > top) {
                top = v[e];
                at = (uint32_t)x.first(granule) + e;
            }
    };
    float *tops = g.tops + (uint64_t)row * g.maxima;
    if (kind == kFew && g.halves == 2) {
        x.steps(from, per / 2, look);
        half_top = top;
        const uint32_t half_at = at;
        top = -__builtin_inff();
        x.steps(from + per / 2, per - per / 2, look);
        const uint32_t to = ((part * kWaves + wave) * 64 + lane) * 2;
        tops[to] = half_top;
        tops[to + 1] = top;
        if (half_top >= top) {           // the lower index of equal ones
            top = half_top;
            at = half_at;
        }
    } else {
        x.steps(from, per, look);
        if (kind == kFew) {
            float of_share = top;
            for (uint32_t d = 1; d < g.share; d <<= 1)
                of_share = fmaxf(of_share, __shfl_xor(of_share, d));
            if (lane % g.share == 0)
                tops[((part * kWaves + wave) * 64 + lane) / g.share] = of_share;
        }
    }
    unsigned long long best = top > -__builtin_inff()
                                  ? (unsigned long long)key_of(top) << 32 | (0xFFFFFFFFu - at) : 0ull;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const unsigned long long o = __shfl_xor(best, d);
        best = o > best ? o : best;
    }
    if (lane == 0)
        s_best[wave] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            best = s_best[w] > best ? s_best[w] : best;
        g.best[(uint64_t)row * g.parts + part] = best;
    }
}

// Weight a row's nucleus has to reach.
__device__ __forceinline__ uint64_t nucleus_of(const Setting &p, uint64_t total)
{
    const double want = p.top_p > 0.f ? ceil((double)p.top_p * (double)total) : 1.0;
    const uint64_t need = want < 1.0 ? 1 : (uint64_t)want;
    return need > total ? total : need;
}

struct BinCut {
    uint32_t bin;                // bins below it are in; kBins: all are
    uint64_t above, total;       // of the histogram: in bins below, in all
    uint64_t in_bin;
};

struct BinShared {
    unsigned long long part[kWaves];
    BinCut cut;
};

// Where the cut falls in a histogram.  For a workgroup.
template <class Word>
__device__ __forceinline__ BinCut bin_cut(const Word *hist, const Setting &p, int kind, BinShared &s)
{
    constexpr int PER = kBins / kThreads;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    uint64_t h[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        h[i] = hist[threadIdx.x * PER + i];
        sum += h[i];
    }
    const uint64_t incl = wave_incl64_add(sum);
    if (lane == 63)
        s.part[wave] = incl;
    __syncthreads();
    uint64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? s.part[w] : 0;
        total += s.part[w];
    }
    const uint64_t need = kind != kNucleus ? (uint64_t)p.top_k : nucleus_of(p, total);
    if (threadIdx.x == 0)
        s.cut = BinCut{kBins, total, total, 0};
    __syncthreads();
    if (before < need && need <= before + sum) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < need && need <= before + h[i])
                s.cut = BinCut{threadIdx.x * PER + i, before, total, h[i]};
            before += h[i];
        }
    }
    __syncthreads();
    return s.cut;
}

// What a workgroup puts on its row's list: together in LDS first, so that the
// row's counter is asked once.
struct ListBuf {
    unsigned long long entry[kBuf];
    uint32_t count, valid;       // places given out; those that were used from the start on

    __device__ __forceinline__ void clear()
    {
        if (threadIdx.x == 0) {
            count = 0;
            valid = kBuf;
        }
    }

    // Lanes' entries: bits of `mine` say which of v's a lane has.  For a wave.
    __device__ __forceinline__ void add(const Geometry &g, uint32_t row, uint32_t mine, const float (&v)[8],
                                        uint32_t first)
    {
        const int lane = threadIdx.x & 63;
        uint32_t total = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            total += __popcll(__ballot(mine >> e & 1));
        uint32_t at = 0;
        if (lane == 0)
            at = atomicAdd(&count, total);
        at = __builtin_amdgcn_readfirstlane(at);
        const bool fits = at + total <= kBuf;
        if (!fits) {             // straight to the row
            if (lane == 0) {
                atomicMin(&valid, at);
                at = atomicAdd(&g.length[row], total);
            }
            at = __builtin_amdgcn_readfirstlane(at);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t takers = __ballot(mine >> e & 1);
            if (mine >> e & 1) {
                const uint32_t to = at + __popcll(takers & lanemask_lt());
                const unsigned long long t = (unsigned long long)key_of(v[e]) << 32 | (first + e);
                if (fits)
                    entry[to] = t;
                else if (to < g.list)
                    g.entries[(uint64_t)row * g.list + to] = t;
            }
            at += __popcll(takers);
        }
    }

    // For the workgroup, with a barrier before.
    __device__ __forceinline__ void flush(const Geometry &g, uint32_t row)
    {
        const uint32_t n = count < valid ? count : valid;
        if (n == 0)
            return;
        if (threadIdx.x == 0)
            base = atomicAdd(&g.length[row], n);
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < n; i += kThreads)
            if (base + i < g.list)
                g.entries[(uint64_t)row * g.list + base + i] = entry[i];
    }
    uint32_t base;
};

template <class T>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const sample_args_t a, const Geometry g)
{
    // Counts, or weights: one of them, at a word or two for a bin.
    __shared__ unsigned long long s_hist[kBins];
    uint32_t *const s_count = reinterpret_cast<uint32_t *>(s_hist);
    __shared__ double s_pow[kPowers];
    __shared__ BinShared s_bins;
    __shared__ ListBuf s_list;
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    const Setting p = setting_of(a, g.row0 + row);
    const int cut = cut_of(p, x.n, g.maxima);
    if (cut == kAll || !(p.temperature > 0.f))
        return;
    const unsigned long long best = best_of(g, row, lane);
    if (best == 0)
        return;
    for (uint32_t i = threadIdx.x; i < kBins; i += kThreads)
        s_hist[i] = 0;
    fill_powers(s_pow, g.shift);
    __syncthreads();
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s_pow);
    const uint32_t per = g.blocks * g.steps, from = (part * kWaves + wave) * per;
    if (cut == kFew) {
        // top_k of the maxima, and so of the logits, are no smaller than the
        // last of the bin that the top_k-th maximum is in.
        s_list.clear();
        for (uint32_t i = threadIdx.x; i < g.maxima; i += kThreads) {
            const float v = g.tops[(uint64_t)row * g.maxima + i];
            if (v > -__builtin_inff())
                atomicAdd(&s_count[bin_of(top, v)], 1u);
        }
        __syncthreads();
        const float least_in = from_bin(top, bin_cut(s_count, p, cut, s_bins).bin);
        x.steps(from, per, [&](uint32_t granule, const float (&v)[8]) {
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mine |= (uint32_t)(v[e] >= least_in) << e;
            if (__any(mine))
                s_list.add(g, row, mine, v, (uint32_t)x.first(granule));
        });
        __syncthreads();
        s_list.flush(g, row);
        return;
    }
    if (cut == kTopK)
        x.steps(from, per, [&](uint32_t, const float (&v)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v[e] > -__builtin_inff())
                    atomicAdd(&s_count[bin_of(top, v[e])], 1u);
        });
    else
        w.how([&](auto how) {
            x.steps(from, per, [&](uint32_t, const float (&v)[8]) {
                uint64_t weight[8];
                bool in[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    weight[e] = w.template fixed<how.value>(v[e], in[e]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (v[e] > -__builtin_inff() && in[e] && weight[e])
                        atomicAdd(&s_hist[bin_of(top, v[e])], (unsigned long long)weight[e]);
            });
        });
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kBins; i += kThreads)
        if (const unsigned long long h = cut == kTopK ? (unsigned long long)s_count[i] : s_hist[i])
            atomicAdd(&g.hist[(uint64_t)row * kBins + i], h);
}

// Whether a row under top_k has its whole prefix in the list.
__device__ __forceinline__ bool listed(const Geometry &g, const BinCut &c)
{
    return c.above + c.in_bin <= g.list;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_collect_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ BinShared s_bins;
    __shared__ double s_pow[kPowers];
    __shared__ ListBuf s_list;
    __shared__ float s_few[kWaves][256];
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    const Setting p = setting_of(a, g.row0 + row);
    const int kind = cut_of(p, x.n, g.maxima);
    if (kind == kFew || !(p.temperature > 0.f))
        return;
    const unsigned long long best = best_of(g, row, lane);
    if (best == 0)
        return;
    fill_powers(s_pow, g.shift);
    s_list.clear();
    BinCut cut = {kBins, 0, 0, 0};
    if (kind != kAll) {
        cut = bin_cut(g.hist + (uint64_t)row * kBins, p, kind, s_bins);
        if (part == 0 && threadIdx.x == 0)
            g.cut[row] = cut;
        if (kind == kTopK && !listed(g, cut))
            return;
    } else {
        __syncthreads();
    }
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s_pow);
    const uint32_t first_block = (part * kWaves + wave) * g.blocks;
    // From `sure` on a logit is in; from `maybe` on it goes to the list.
    const float least_logit = -3.402823466e38f;
    float sure = least_logit, maybe = least_logit;
    if (kind != kAll) {
        maybe = from_bin(top, cut.bin);
        sure = kind == kTopK || cut.bin == 0 ? __builtin_inff() : from_bin(top, cut.bin - 1);
    }
    const bool all_sure = kind == kNucleus && cut.bin == 0 ? false : kind != kTopK;
    uint64_t sum = 0;
    uint32_t count = 0, step = 0, block = first_block;
    const uint32_t blocks = first_block < g.row_blocks
                                ? (g.row_blocks - first_block < g.blocks ? g.row_blocks - first_block : g.blocks)
                                : 0;
    w.how([&](auto how) {
        x.steps(first_block * g.steps, blocks * g.steps, [&](uint32_t granule, const float (&v)[8]) {
            const int64_t first = x.first(granule);
            if (all_sure) {
                // What is in is few or all: few are put together first, and
                // weighed by full waves.
                uint32_t in = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    in |= (uint32_t)(v[e] >= sure) << e;
                uint32_t total = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    total += __popcll(__ballot(in >> e & 1));
                if (total > 256) {
                    uint64_t weight[8];
                    bool held[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        weight[e] = w.template fixed<how.value>(v[e], held[e]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        held[e] = held[e] && v[e] >= sure;
                        sum += held[e] ? weight[e] : 0;
                        count += held[e];
                    }
                } else if (total) {
                    float *const few = s_few[wave];
                    uint32_t at = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t takers = __ballot(in >> e & 1);
                        if (in >> e & 1)
                            few[at + __popcll(takers & lanemask_lt())] = v[e];
                        at += __popcll(takers);
                    }
                    for (uint32_t j = lane; j < total; j += 64) {
                        bool held;
                        const uint64_t weight = w.template fixed<how.value>(few[j], held);
                        sum += held ? weight : 0;
                        count += held;
                    }
                }
            }
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mine |= (uint32_t)(v[e] >= maybe && !(v[e] >= sure && all_sure)) << e;
            if (kind != kAll && __any(mine))
                s_list.add(g, row, mine, v, (uint32_t)first);
            if (++step == g.steps) {             // a block's end
                if (kind != kTopK) {
                    sum = wave_sum64(sum);
                    count = wave_sum(count);
                    if (lane == 0) {
                        g.sums[(uint64_t)row * g.row_blocks + block] = sum;
                        g.counts[(uint64_t)row * g.row_blocks + block] = count;
                    }
                }
                sum = 0;
                count = step = 0;
                ++block;
            }
        });
    });
    __syncthreads();
    s_list.flush(g, row);
}

// ---------------------------------------------------------------------------
// draw
// ---------------------------------------------------------------------------

// The last kept token: keys above are in, and of those equal to it the ones
// at index `last` and before.
struct Cut {
    uint32_t key, last;
    __device__ __forceinline__ bool in(uint32_t k, uint32_t i) const
    {
        return k > key || (k == key && i <= last);
    }
};

// Words that share a digit meet in its counter: lanes have eight between them.
constexpr int kCopies = 8;

struct DrawShared {
    unsigned long long hist[256][kCopies];
    unsigned long long part[kWaves];
    unsigned long long need, found;
    uint32_t digit;
    uint32_t vary;
    double pow[kPowers];
    union {
        unsigned long long sums[kMaxBlocks];      // once the list is done with
        struct {
            unsigned long long entry[kHeld], weight[kHeld];
        } list;
    };
};

__device__ __forceinline__ uint64_t block_sum64(uint64_t x, DrawShared &s)
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

// The 32-bit word at which amounts, summed over entries in rising (or, DOWN,
// falling) order of it, reach `need`, which then is what that word itself
// has to give; `each(f)` calls f(word, amount) for the entries, in any order.
// `found`: what the entries of the word amount to.  Words differ from `like`
// in bits of `vary` only: digits without such bits are not looked at.
template <bool DOWN, class Each>
__device__ __forceinline__ uint32_t select_word(Each each, uint32_t like, uint32_t vary, uint64_t &need,
                                                uint64_t &found, DrawShared &s)
{
    const int lane = threadIdx.x & 63;
    uint32_t prefix = 0;
    for (int b = 24; b >= 0; b -= 8) {
        if (b && (vary >> b & 255) == 0) {
            prefix = prefix << 8 | (like >> b & 255);
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            (&s.hist[0][0])[threadIdx.x + i * kThreads] = 0;
        __syncthreads();
        each([&](uint32_t word, uint64_t amount) {
            if (b == 24 || (word >> (b + 8)) == prefix)
                atomicAdd(&s.hist[(word >> b) & 255][threadIdx.x % kCopies], (unsigned long long)amount);
        });
        __syncthreads();
        {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                sum += s.hist[threadIdx.x][(i + threadIdx.x) % kCopies];
            s.hist[threadIdx.x][0] = sum;
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            uint64_t h[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 4 * lane + i;
                h[i] = s.hist[DOWN ? 255 - d : d][0];
                sum += h[i];
            }
            const uint64_t incl = wave_incl64_add(sum);
            uint64_t before = incl - sum;
            if (before < need && need <= incl) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before < need && need <= before + h[i]) {
                        s.digit = (uint32_t)(DOWN ? 255 - (4 * lane + i) : 4 * lane + i);
                        s.need = need - before;
                        s.found = h[i];
                        break;
                    }
                    before += h[i];
                }
            }
        }
        __syncthreads();
        prefix = prefix << 8 | s.digit;
        need = s.need;
        found = s.found;
    }
    return prefix;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ DrawShared s;
    const uint32_t row = blockIdx.x;
    const uint64_t r = g.row0 + row;
    const RowOf<T> x(a, r);
    const Setting p = setting_of(a, r);
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const int kind = cut_of(p, x.n, g.maxima);
    // Read at once: what follows is a chain.
    const BinCut bins = kind == kAll || kind == kFew ? BinCut{kBins, 0, 0, 0} : g.cut[row];
    const uint32_t listed_n = kind == kAll ? 0 : g.length[row];
    constexpr int PER = kMaxBlocks / kThreads;
    uint64_t block_sum[PER];
    uint32_t block_count[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t b = threadIdx.x + i * kThreads;
        const bool any = (kind == kAll || kind == kNucleus) && b < g.row_blocks;
        block_sum[i] = any ? g.sums[(uint64_t)row * g.row_blocks + b] : 0;
        block_count[i] = any ? g.counts[(uint64_t)row * g.row_blocks + b] : 0;
    }
    const unsigned long long best = best_of(g, row, lane);
    if (best == 0 || !(p.temperature > 0.f)) {
        if (threadIdx.x == 0) {
            a.tokens[r] = best ? (int32_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
            if (a.logprobs)
                a.logprobs[r] = best ? 0.f : -__builtin_inff();
            if (a.kept)
                a.kept[r] = best ? 1 : 0;
        }
        return;
    }
    fill_powers(s.pow, g.shift);
    __syncthreads();
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s.pow);
    // Is what has to be looked at in the list, or is it the row?
    const bool whole = kind == kTopK ? !listed(g, bins) : listed_n > g.list;
    const bool top_k = kind == kTopK || kind == kFew;
    const bool here = !whole && listed_n <= kHeld;
    const unsigned long long *entries = g.entries + (uint64_t)row * g.list;
    const uint32_t granules = (x.n + x.skew + 7) / 8;
    const auto weight_of = [&](uint32_t key, bool &in) -> uint64_t {
        uint64_t v = 0;
        w.how([&](auto how) { v = w.template fixed<how.value>(logit_of(key), in); });
        return in ? v : 0;
    };
    // Keys of what is looked at differ from `like` in these bits.
    uint32_t like = 0, vary = 0xFFFFFFFFu;
    if (here && listed_n) {
        like = (uint32_t)(entries[0] >> 32);
        if (threadIdx.x == 0)
            s.vary = 0;
        __syncthreads();
        uint32_t own = 0;
        for (uint32_t i = threadIdx.x; i < listed_n; i += kThreads) {
            const unsigned long long t = entries[i];
            bool in;
            const uint64_t v = weight_of((uint32_t)(t >> 32), in);
            s.list.entry[i] = t;
            s.list.weight[i] = v | (in ? kIn : 0);
            own |= (uint32_t)(t >> 32) ^ like;
        }
#pragma unroll
        for (int d = 32; d; d >>= 1)
            own |= __shfl_xor(own, d);
        if (lane == 0 && own)
            atomicOr(&s.vary, own);
        __syncthreads();
        vary = s.vary;
    }
    // f(key, index, weight(in)) for every token that is looked at.
    const auto each_entry = [&](auto f) {
        if (here) {
            for (uint32_t i = threadIdx.x; i < listed_n; i += kThreads) {
                const unsigned long long t = s.list.entry[i];
                f((uint32_t)(t >> 32), (uint32_t)t, [&](bool &in) -> uint64_t {
                    const unsigned long long v = s.list.weight[i];
                    in = v >= kIn;
                    return v & ~kIn;
                });
            }
        } else if (whole) {
            for (uint32_t i = threadIdx.x; i < granules; i += kThreads) {
                float v[8];
                x.load(i, v);
                const uint32_t first = (uint32_t)x.first(i);
#pragma unroll 1
                for (int e = 0; e < 8; ++e)
                    if (const uint32_t k = key_of(v[e]))
                        f(k, first + e, [&](bool &in) { return weight_of(k, in); });
            }
        } else {
            for (uint32_t i = threadIdx.x; i < listed_n; i += kThreads) {
                const unsigned long long t = entries[i];
                const uint32_t k = (uint32_t)(t >> 32);
                f(k, (uint32_t)t, [&](bool &in) { return weight_of(k, in); });
            }
        }
    };
    const uint32_t index_bits = x.n > 1 ? 0xFFFFFFFFu >> __clz(x.n - 1) : 0;
    // The index of the `need`-th token of a key.
    const auto last_of = [&](uint32_t key, uint64_t need) {
        uint64_t found;
        return select_word<false>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i, auto) {
                    if (k == key)
                        f(i, 1);
                });
            },
            0, index_bits, need, found, s);
    };

    Cut cut = {0, 0};
    // kFew: the maxima are of top_k lanes at least, and a row is listed whole
    // where it has not so many.
    if (top_k && (kind == kFew ? listed_n : bins.total) > (uint32_t)p.top_k) {
        uint64_t need = (uint64_t)p.top_k, found;
        cut.key = select_word<true>(
            [&](auto f) { each_entry([&](uint32_t k, uint32_t, auto) { f(k, 1); }); }, like, vary, need,
            found, s);
        cut.last = need == found ? 0xFFFFFFFFu : last_of(cut.key, need);
    }
    if (p.top_p < 1.f) {
        uint64_t need;
        if (kind == kNucleus && !whole) {
            need = nucleus_of(p, bins.total) - bins.above;
        } else {
            uint64_t sum = 0;
            each_entry([&](uint32_t k, uint32_t i, auto weight) {
                bool in;
                if (cut.in(k, i))
                    sum += weight(in);
            });
            need = nucleus_of(p, block_sum64(sum, s));
        }
        uint64_t found;
        const uint32_t key = select_word<true>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i, auto weight) {
                    bool in;
                    if (cut.in(k, i))
                        f(k, weight(in));
                });
            },
            like, vary, need, found, s);
        bool in;
        const uint64_t each = weight_of(key, in);
        if (found > (need - 1) / each * each + each)       // not all of the key's
            cut.last = last_of(key, (need + each - 1) / each);
        else if (key != cut.key)
            cut.last = 0xFFFFFFFFu;
        cut.key = key;
    }

    // The token: where the kept weight, in index order, passes u of its sum.
    const auto place_of_u = [&](uint64_t total) -> uint64_t {
        const double uz = p.u > 0.f ? (double)p.u * (double)total : 0.0;
        const uint64_t want = uz < (double)total ? (uint64_t)uz : total - 1;
        return want > total - 1 ? total - 1 : want;
    };
    const auto answer = [&](uint32_t i, uint64_t total) {
        i = i < x.n ? i : x.n - 1;           // logits that change under the call
        a.tokens[r] = (int32_t)i;
        if (a.logprobs) {
            const float v = (float)x.x[i];
            const double d = v == top ? 0.0 : ((double)v - (double)top) / (double)p.temperature;
            a.logprobs[r] = (float)(d - log((double)total / w.one));
        }
    };
    uint64_t kept = 0;
    if (top_k && !whole) {
        uint64_t sum = 0;
        each_entry([&](uint32_t k, uint32_t i, auto weight) {
            if (cut.in(k, i)) {
                bool in;
                sum += weight(in);
                kept += in;
            }
        });
        const uint64_t total = block_sum64(sum, s);
        kept = block_sum64(kept, s);
        uint64_t need = place_of_u(total) + 1, found;
        const uint32_t token = select_word<false>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i, auto weight) {
                    bool in;
                    if (cut.in(k, i))
                        f(i, weight(in));
                });
            },
            0, index_bits, need, found, s);
        if (threadIdx.x == 0) {
            answer(token, total);
            if (a.kept)
                a.kept[r] = (int32_t)kept;
        }
        return;
    }

    // By blocks: what `collect` summed, and the list's part of each.  A held
    // list's kept tokens wait in registers while the sums take its place.
    const uint32_t step = g.steps * 64;          // granules of a block
    constexpr int OWN = kHeld / kThreads;
    uint32_t own_block[OWN];
    uint64_t own_weight[OWN];
    if (here) {
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const uint32_t at = threadIdx.x + j * kThreads;
            own_weight[j] = 0;
            own_block[j] = 0;
            if (at < listed_n) {
                const unsigned long long t = s.list.entry[at], v = s.list.weight[at];
                if (cut.in((uint32_t)(t >> 32), (uint32_t)t)) {
                    own_weight[j] = v & ~kIn;
                    own_block[j] = ((uint32_t)t + x.skew) / 8 / step;
                    kept += v >= kIn;
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t b = threadIdx.x + i * kThreads;
        s.sums[b] = whole ? 0 : block_sum[i];
        kept += whole ? 0 : block_count[i];
    }
    __syncthreads();
    if (here) {
#pragma unroll
        for (int j = 0; j < OWN; ++j)
            if (own_weight[j])
                atomicAdd(&s.sums[own_block[j]], (unsigned long long)own_weight[j]);
    } else if (kind != kAll) {
        each_entry([&](uint32_t k, uint32_t i, auto weight) {
            if (!cut.in(k, i))
                return;
            bool in;
            const uint64_t v = weight(in);
            kept += in;
            if (v)
                atomicAdd(&s.sums[(i + x.skew) / 8 / step], (unsigned long long)v);
        });
    }
    kept = block_sum64(kept, s);
    if (threadIdx.x == 0 && a.kept)
        a.kept[r] = (int32_t)kept;
    uint64_t h[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        h[i] = s.sums[threadIdx.x * PER + i];
        sum += h[i];
    }
    const uint64_t total = block_sum64(sum, s);
    const uint64_t want = place_of_u(total);
    const uint64_t incl = wave_incl64_add(sum);
    __syncthreads();
    if (lane == 63)
        s.part[wave] = incl;
    __syncthreads();
    uint64_t before = incl - sum;
    for (int v = 0; v < wave; ++v)
        before += s.part[v];
    if (before <= want && want < before + sum) {
        for (int i = 0; i < PER; ++i) {
            if (before <= want && want < before + h[i]) {
                s.digit = threadIdx.x * PER + i;
                s.need = want - before;
            }
            before += h[i];
        }
    }
    __syncthreads();
    // The block again, in its order, a wave step a wave.
    uint64_t left = s.need;
    const uint32_t from = s.digit * step;
    for (uint32_t i = 0; i < g.steps; i += kWaves) {
        const uint32_t granule = from + (i + wave) * 64 + lane;
        const uint32_t first = (uint32_t)x.first(granule);
        float v[8];
        uint64_t own[8], mine = 0;
        bool in[8];
        if (i + wave < g.steps) {
            x.load(granule, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = -__builtin_inff();
        }
        w.how([&](auto how) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                own[e] = w.template fixed<how.value>(v[e], in[e]);
        });
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t k = key_of(v[e]);
            own[e] = k && in[e] && cut.in(k, first + e) ? own[e] : 0;
            mine += own[e];
        }
        const uint64_t upto = wave_incl64_add(mine);
        __syncthreads();
        if (lane == 63)
            s.part[wave] = upto;
        __syncthreads();
        uint64_t at = upto - mine, all = 0;
#pragma unroll
        for (int v_ = 0; v_ < kWaves; ++v_) {
            at += v_ < wave ? s.part[v_] : 0;
            all += s.part[v_];
        }
        if (at <= left && left < at + mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (at <= left && left < at + own[e])
                    answer(first + e, total);
                at += own[e];
            }
        }
        if (left < all)
            return;
        left -= all;
    }
}

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Cuts rows of `vocab`, `rows` of them at a time, and lays out the scratch.
struct Layout {
    Geometry g;
    uint64_t batch;
    size_t bytes;
};

Layout layout_of(uint64_t rows, uint64_t vocab, void *body)
{
    Layout l = {};
    Geometry &g = l.g;
    int bits = 0;
    while ((1ull << bits) < vocab)
        ++bits;
    // Sums of all weights stay below 2^62.
    g.shift = 62 - bits < 51 ? 62 - bits : 51;
    const uint64_t waves = (vocab + 7 + 511) / 512;              // wave steps
    g.steps = (uint32_t)((waves + kMaxBlocks - 1) / kMaxBlocks);
    if (g.steps < 4 && waves >= 256)             // a block's sum costs about as much as a step
        g.steps = 4;
    g.row_blocks = (uint32_t)((waves + g.steps - 1) / g.steps);
    g.list = (uint32_t)(vocab < kList ? (vocab ? vocab : 1) : kList);
    const size_t fixed = kBins * 8 + (size_t)g.row_blocks * 12 + (size_t)g.list * 8 + 64 * kWaves * 8 + kMaxima * 4;
    // Rows at a time: 256 MiB of scratch, or 1024 rows.
    uint64_t most = ((size_t)1 << 28) / fixed;
    most = most < 1024 ? 1024 : most > 32768 ? 32768 : most;
    l.batch = rows < most ? rows : most;
    // Parts: about eight workgroups a compute unit over all rows.
    const uint64_t want = l.batch ? 2048 / l.batch : 1;
    uint64_t parts = (g.row_blocks + kWaves - 1) / kWaves;
    parts = parts < want ? parts : want;
    parts = parts > 64 ? 64 : parts < 1 ? 1 : parts;
    g.blocks = (uint32_t)((g.row_blocks + parts * kWaves - 1) / (parts * kWaves));
    g.parts = (g.row_blocks + g.blocks * kWaves - 1) / (g.blocks * kWaves);
    g.share = 1;
    while (g.parts * kThreads / g.share > kMaxima && g.share < 64)
        g.share *= 2;
    g.halves = g.parts * kThreads * 2 <= kMaxima && g.blocks * g.steps >= 8 ? 2 : 1;
    g.maxima = g.parts * kThreads * g.halves / g.share;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = body ? static_cast<char *>(body) + at : nullptr;
        at += align256(bytes * l.batch);
        return p;
    };
    g.best = reinterpret_cast<unsigned long long *>(take(g.parts * 8));
    g.tops = reinterpret_cast<float *>(take(g.maxima * 4));
    g.hist = reinterpret_cast<unsigned long long *>(take(kBins * 8));
    g.sums = reinterpret_cast<unsigned long long *>(take(g.row_blocks * 8));
    g.entries = reinterpret_cast<unsigned long long *>(take((size_t)g.list * 8));
    g.counts = reinterpret_cast<uint32_t *>(take(g.row_blocks * 4));
    g.length = reinterpret_cast<uint32_t *>(take(4));
    g.cut = reinterpret_cast<BinCut *>(take(sizeof(BinCut)));
    l.bytes = at;
    return l;
}

template <class T>
hipError_t run_sample(const sample_args_t &a, void *body, hipStream_t stream)
{
    Layout l = layout_of(a.rows, a.vocab, body);
    for (uint64_t row0 = 0; row0 < a.rows; row0 += l.batch) {
        l.g.row0 = row0;
        const unsigned rows = (unsigned)(a.rows - row0 < l.batch ? a.rows - row0 : l.batch);
        const dim3 grid(l.g.parts, rows);
        // A row can only be cut if something says so for it.
        const bool cut = a.top_ks || a.top_ps || (a.top_k > 0 && (uint64_t)a.top_k < a.vocab) ||
                         a.top_p < 1.f;
        sample_max_kernel<T><<<grid, kThreads, 0, stream>>>(a, l.g);
        if (cut)
            sample_hist_kernel<T><<<grid, kThreads, 0, stream>>>(a, l.g);
        sample_collect_kernel<T><<<grid, kThreads, 0, stream>>>(a, l.g);
        sample_draw_kernel<T><<<rows, kThreads, 0, stream>>>(a, l.g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

size_t sample_body_bytes(uint64_t rows, uint64_t vocab) { return layout_of(rows, vocab, nullptr).bytes; }

hipError_t launch_sample(const sample_args_t &a, void *body, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: return run_sample<float>(a, body, stream);
    case LIBSCAN_BF16: return run_sample<__bf16>(a, body, stream);
    default: return run_sample<_Float16>(a, body, stream);
    }
}

}  // namespace libscan
