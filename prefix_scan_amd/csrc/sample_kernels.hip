// sample_kernels.hip -- one token from each row of logits.
//
// The kept tokens are a prefix of the row in order of falling logit, so they
// are known by the last one: its key (the logit in an order-preserving u32)
// and its index, the largest kept one of that key.  No row is sorted, and a
// row is read three times at most:
//
//   max      the largest logit M and its lowest index;
//   hist     where there is a cut, a histogram over 2048 bins of M - x (64 to
//            a binade, so that they are fine where the weight is, whatever
//            the logits' scale): counts for top_k, weights for top_p;
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
// Weights are 2^((x - M) log2 e / T) in 64 bits, held as 64-bit fixed point:
// sums (by LDS and global atomics, in any order) are exact, so the cut and
// the drawn token depend on the inputs alone.
#include "sample.hpp"

namespace libscan {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kList = 8192;            // longest list of a row
constexpr uint32_t kWaveBuf = 768;          // entries a wave gathers before it appends them
constexpr uint32_t kMaxBlocks = 1024;       // of a row

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

// What a row does with its bins.
enum { kAll, kTopK, kNucleus };

__device__ __forceinline__ int cut_of(const Setting &p, uint32_t n)
{
    if (p.top_k > 0 && (uint32_t)p.top_k < n)
        return kTopK;
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

// 2^(i / 64), for 2^y = 2^(i / 64) 2^r: |r| <= 1 / 128 leaves a polynomial of
// the fifth degree 2^-53 off.
__device__ __forceinline__ void fill_powers(double *t)
{
    if (threadIdx.x < 64)
        t[threadIdx.x] = exp2((double)threadIdx.x / 64.0);
}

struct Weigh {
    double top, by, one;         // M, log2 e / T, the fixed-point one
    const double *pow;
    // The weight of a logit against the largest: 0 <= w <= 1, 1 at the top.
    __device__ __forceinline__ double real(float x) const
    {
        const double d = (double)x - top;
        double y = (double)x == top ? 0.0 : d * by;            // also +inf
        y = y >= -1100.0 ? y : -1100.0;                        // also inf - inf
        const double magic = 6755399441055744.0;               // 1.5 * 2^52
        const double t = __builtin_fma(y, 64.0, magic);
        const int k = (int)(uint32_t)__double_as_longlong(t);
        const double r = __builtin_fma(t - magic, -1.0 / 64.0, y) * 0.693147180559945309417;
        double p = __builtin_fma(r, 1.0 / 120.0, 1.0 / 24.0);
        p = __builtin_fma(p, r, 1.0 / 6.0);
        p = __builtin_fma(p, r, 0.5);
        p = __builtin_fma(p, r, 1.0);
        p = __builtin_fma(p, r, 1.0);
        return __builtin_amdgcn_ldexp(pow[k & 63] * p, k >> 6);
    }
    // To the nearest; one <= 2^51.
    __device__ __forceinline__ uint64_t fixed(double w) const
    {
        const double t = __builtin_fma(w, one, 4503599627370496.0);
        return (uint64_t)__double_as_longlong(t) & 0xFFFFFFFFFFFFFull;
    }
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
    // What lies outside the row reads as -inf.
    __device__ __forceinline__ void load(uint32_t granule, float (&v)[8]) const
    {
        const int64_t i = first(granule);
        if (i >= 0 && i + 8 <= (int64_t)n) {
            typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
            constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
                const vec t = *reinterpret_cast<const vec *>(x + i + h * V);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    v[h * V + e] = (float)t[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = i + e >= 0 && i + e < (int64_t)n ? (float)x[i + e] : -__builtin_inff();
        }
    }
};

// How rows are cut.  A wave step is 64 granules; blocks of `steps` of them
// have a sum of kept weights each, and a wave has `blocks` blocks.
struct Geometry {
    uint32_t parts, blocks, steps, row_blocks, list;
    int shift;
    uint64_t row0;
    // scratch, rows from row0 on
    unsigned long long *best;     // [rows][parts]
    unsigned long long *hist;     // [rows][kBins]
    unsigned long long *sums;     // [rows][row_blocks]
    unsigned long long *entries;  // [rows][list]: key, index
    uint32_t *counts;             // [rows][row_blocks]
    uint32_t *length;             // [rows]
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
    return Weigh{(double)top, 1.4426950408889634074 / (double)p.temperature, (double)(1ull << g.shift), pow};
}

__device__ __forceinline__ double least_weight(const Setting &p)
{
    return p.min_p > 0.f ? (p.min_p < 1.f ? (double)p.min_p : 1.0) : 0.0;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ unsigned long long s_best[kWaves];
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    if (cut_of(setting_of(a, g.row0 + row), x.n) != kAll)
        for (uint32_t i = part * kThreads + threadIdx.x; i < kBins; i += g.parts * kThreads)
            g.hist[(uint64_t)row * kBins + i] = 0;
    if (part == 0 && threadIdx.x == 0)
        g.length[row] = 0;
    const uint32_t per = g.blocks * g.steps, from = (part * kWaves + wave) * per;
    float top = -__builtin_inff();
    uint32_t at = 0;
#pragma unroll 4
    for (uint32_t i = 0; i < per; ++i) {
        const uint32_t granule = (from + i) * 64 + lane;
        const int64_t first = x.first(granule);
        if (first >= (int64_t)x.n)
            break;
        float v[8];
        x.load(granule, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (v[e] > top) {
                top = v[e];
                at = (uint32_t)(first + e);
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

template <class T>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ unsigned long long s_hist[kBins];
    __shared__ double s_pow[64];
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    const Setting p = setting_of(a, g.row0 + row);
    const int cut = cut_of(p, x.n);
    if (cut == kAll || !(p.temperature > 0.f))
        return;
    const unsigned long long best = best_of(g, row, lane);
    if (best == 0)
        return;
    for (uint32_t i = threadIdx.x; i < kBins; i += kThreads)
        s_hist[i] = 0;
    fill_powers(s_pow);
    __syncthreads();
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s_pow);
    const double least = least_weight(p);
    const uint32_t per = g.blocks * g.steps, from = (part * kWaves + wave) * per;
#pragma unroll 2
    for (uint32_t i = 0; i < per; ++i) {
        const uint32_t granule = (from + i) * 64 + lane;
        if (x.first(granule) >= (int64_t)x.n)
            break;
        float v[8];
        x.load(granule, v);
        if (cut == kTopK) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v[e] > -__builtin_inff())
                    atomicAdd(&s_hist[bin_of(top, v[e])], 1ull);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v[e] > -__builtin_inff()) {
                    const double r = w.real(v[e]);
                    if (r >= least)
                        atomicAdd(&s_hist[bin_of(top, v[e])], (unsigned long long)w.fixed(r));
                }
        }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kBins; i += kThreads)
        if (s_hist[i])
            atomicAdd(&g.hist[(uint64_t)row * kBins + i], s_hist[i]);
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

// Where the cut falls in a row's histogram.  For a workgroup.
__device__ __forceinline__ BinCut bin_cut(const Geometry &g, uint32_t row, const Setting &p, int kind,
                                          BinShared &s)
{
    constexpr int PER = kBins / kThreads;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    uint64_t h[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        h[i] = g.hist[(uint64_t)row * kBins + threadIdx.x * PER + i];
        sum += h[i];
    }
    const uint64_t incl = wave_incl64(sum);
    if (lane == 63)
        s.part[wave] = incl;
    __syncthreads();
    uint64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? s.part[w] : 0;
        total += s.part[w];
    }
    const uint64_t need = kind == kTopK ? (uint64_t)p.top_k : nucleus_of(p, total);
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

// Whether a row under top_k has its whole prefix in the list.
__device__ __forceinline__ bool listed(const Geometry &g, const BinCut &c)
{
    return c.above + c.in_bin <= g.list;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_collect_kernel(const sample_args_t a, const Geometry g)
{
    __shared__ BinShared s_bins;
    __shared__ double s_pow[64];
    __shared__ unsigned long long s_buf[kWaves][kWaveBuf];
    const uint32_t row = blockIdx.y, part = blockIdx.x;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const RowOf<T> x(a, g.row0 + row);
    const Setting p = setting_of(a, g.row0 + row);
    if (!(p.temperature > 0.f))
        return;
    const unsigned long long best = best_of(g, row, lane);
    if (best == 0)
        return;
    fill_powers(s_pow);
    const int kind = cut_of(p, x.n);
    BinCut cut = {kBins, 0, 0, 0};
    if (kind != kAll) {
        cut = bin_cut(g, row, p, kind, s_bins);
        if (kind == kTopK && !listed(g, cut))
            return;
    } else {
        __syncthreads();
    }
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s_pow);
    const double least = least_weight(p);
    const uint32_t first_block = (part * kWaves + wave) * g.blocks;
    unsigned long long *entries = g.entries + (uint64_t)row * g.list;
    uint32_t held = 0;           // of the wave's buffer
    const auto append = [&]() {
        uint32_t to = 0;
        if (lane == 0)
            to = atomicAdd(&g.length[row], held);
        to = __shfl(to, 0);
        for (uint32_t i = lane; i < held; i += 64)
            if (to + i < g.list)
                entries[to + i] = s_buf[wave][i];
        held = 0;
    };
    for (uint32_t b = first_block; b < first_block + g.blocks && b < g.row_blocks; ++b) {
        uint64_t sum = 0;
        uint32_t count = 0;
        for (uint32_t i = 0; i < g.steps; ++i) {
            const uint32_t granule = (b * g.steps + i) * 64 + lane;
            const int64_t first = x.first(granule);
            float v[8];
            x.load(granule, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool live = v[e] > -__builtin_inff();
                const uint32_t bin = live ? bin_of(top, v[e]) : kBins;
                if (kind != kTopK && live && bin < cut.bin) {
                    const double r = w.real(v[e]);
                    if (r >= least) {
                        sum += w.fixed(r);
                        ++count;
                    }
                }
                const bool take = live && (bin == cut.bin || (kind == kTopK && bin < cut.bin));
                const uint64_t takers = __ballot(take);
                if (takers) {
                    if (take)
                        s_buf[wave][held + __popcll(takers & ((1ull << lane) - 1))] =
                            (unsigned long long)key_of(v[e]) << 32 | (uint32_t)(first + e);
                    held += __popcll(takers);
                }
            }
            if (held > kWaveBuf - 512)
                append();
        }
        if (kind != kTopK) {
            sum = wave_sum64(sum);
            count = (uint32_t)wave_sum64(count);
            if (lane == 0) {
                g.sums[(uint64_t)row * g.row_blocks + b] = sum;
                g.counts[(uint64_t)row * g.row_blocks + b] = count;
            }
        }
    }
    if (held)
        append();
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

struct DrawShared {
    BinShared bins;
    unsigned long long hist[256];
    unsigned long long part[kWaves];
    unsigned long long need, found;
    uint32_t digit;
    double pow[64];
    unsigned long long sums[kMaxBlocks];
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
// `found`: what the entries of the word amount to.
template <bool DOWN, class Each>
__device__ __forceinline__ uint32_t select_word(Each each, uint64_t &need, uint64_t &found, DrawShared &s)
{
    const int lane = threadIdx.x & 63;
    uint32_t prefix = 0;
    for (int b = 24; b >= 0; b -= 8) {
        __syncthreads();
        s.hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](uint32_t word, uint64_t amount) {
            if (b == 24 || (word >> (b + 8)) == prefix)
                atomicAdd(&s.hist[(word >> b) & 255], (unsigned long long)amount);
        });
        __syncthreads();
        if (threadIdx.x < 64) {
            uint64_t h[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 4 * lane + i;
                h[i] = s.hist[DOWN ? 255 - d : d];
                sum += h[i];
            }
            const uint64_t incl = wave_incl64(sum);
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
    fill_powers(s.pow);
    const int kind = cut_of(p, x.n);
    BinCut bins = {kBins, 0, 0, 0};
    if (kind != kAll)
        bins = bin_cut(g, row, p, kind, s.bins);
    else
        __syncthreads();
    const float top = logit_of((uint32_t)(best >> 32));
    const Weigh w = weigh_of(g, p, top, s.pow);
    const double least = least_weight(p);
    const uint32_t listed_n = kind == kAll ? 0 : g.length[row];
    // Is what has to be looked at in the list, or is it the row?
    const bool whole = kind == kTopK ? !listed(g, bins) : listed_n > g.list;
    const unsigned long long *entries = g.entries + (uint64_t)row * g.list;
    const uint32_t granules = (x.n + x.skew + 7) / 8;
    const auto each_entry = [&](auto f) {
        if (whole) {
            for (uint32_t i = threadIdx.x; i < granules; i += kThreads) {
                float v[8];
                x.load(i, v);
                const uint32_t first = (uint32_t)x.first(i);
#pragma unroll 1
                for (int e = 0; e < 8; ++e)
                    if (const uint32_t k = key_of(v[e]))
                        f(k, first + e);
            }
        } else {
            for (uint32_t i = threadIdx.x; i < listed_n; i += kThreads) {
                const unsigned long long t = entries[i];
                f((uint32_t)(t >> 32), (uint32_t)t);
            }
        }
    };
    const auto weight_of = [&](uint32_t key, bool &in) -> uint64_t {
        const double v = w.real(logit_of(key));
        in = v >= least;
        return in ? w.fixed(v) : 0;
    };
    // The index of the `need`-th token of a key.
    const auto last_of = [&](uint32_t key, uint64_t need) {
        uint64_t found;
        return select_word<false>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i) {
                    if (k == key)
                        f(i, 1);
                });
            },
            need, found, s);
    };

    Cut cut = {0, 0};
    if (kind == kTopK && bins.total > (uint32_t)p.top_k) {
        uint64_t need = (uint64_t)p.top_k, found;
        cut.key = select_word<true>(
            [&](auto f) { each_entry([&](uint32_t k, uint32_t) { f(k, 1); }); }, need, found, s);
        cut.last = need == found ? 0xFFFFFFFFu : last_of(cut.key, need);
    }
    if (p.top_p < 1.f) {
        uint64_t need;
        if (kind == kNucleus && !whole) {
            need = nucleus_of(p, bins.total) - bins.above;
        } else {
            uint64_t sum = 0;
            each_entry([&](uint32_t k, uint32_t i) {
                bool in = cut.in(k, i);
                if (in)
                    sum += weight_of(k, in);
            });
            need = nucleus_of(p, block_sum64(sum, s));
        }
        uint64_t found;
        const uint32_t key = select_word<true>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i) {
                    bool in = cut.in(k, i);
                    if (in)
                        f(k, weight_of(k, in));
                });
            },
            need, found, s);
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
        a.tokens[r] = (int32_t)i;
        if (a.logprobs) {
            const float v = (float)x.x[i];
            const double d = v == top ? 0.0 : ((double)v - (double)top) / (double)p.temperature;
            a.logprobs[r] = (float)(d - log((double)total / w.one));
        }
    };
    uint64_t kept = 0;
    if (kind == kTopK && !whole) {
        uint64_t sum = 0;
        each_entry([&](uint32_t k, uint32_t i) {
            bool in = cut.in(k, i);
            if (in) {
                sum += weight_of(k, in);
                kept += in;
            }
        });
        const uint64_t total = block_sum64(sum, s);
        kept = block_sum64(kept, s);
        uint64_t need = place_of_u(total) + 1, found;
        const uint32_t token = select_word<false>(
            [&](auto f) {
                each_entry([&](uint32_t k, uint32_t i) {
                    bool in = cut.in(k, i);
                    if (in)
                        f(i, weight_of(k, in));
                });
            },
            need, found, s);
        if (threadIdx.x == 0) {
            answer(token, total);
            if (a.kept)
                a.kept[r] = (int32_t)kept;
        }
        return;
    }

    // By blocks: what `collect` summed, and the list's part of each.
    const uint32_t step = g.steps * 64;          // granules of a block
    for (uint32_t b = threadIdx.x; b < g.row_blocks; b += kThreads) {
        s.sums[b] = whole ? 0 : g.sums[(uint64_t)row * g.row_blocks + b];
        kept += whole ? 0 : g.counts[(uint64_t)row * g.row_blocks + b];
    }
    __syncthreads();
    if (kind != kAll)
        each_entry([&](uint32_t k, uint32_t i) {
            bool in = cut.in(k, i);
            if (!in)
                return;
            const uint64_t v = weight_of(k, in);
            kept += in;
            if (v)
                atomicAdd(&s.sums[(i + x.skew) / 8 / step], (unsigned long long)v);
        });
    kept = block_sum64(kept, s);
    if (threadIdx.x == 0 && a.kept)
        a.kept[r] = (int32_t)kept;
    constexpr int PER = kMaxBlocks / kThreads;
    uint64_t h[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t b = threadIdx.x * PER + i;
        h[i] = b < g.row_blocks ? s.sums[b] : 0;
        sum += h[i];
    }
    const uint64_t total = block_sum64(sum, s);
    const uint64_t want = place_of_u(total);
    const uint64_t incl = wave_incl64(sum);
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
    // The block again, in its order, by the first wave.
    if (wave)
        return;
    uint64_t left = s.need;
    const uint32_t from = s.digit * step;
    for (uint32_t i = 0; i < g.steps; ++i) {
        const uint32_t granule = from + i * 64 + lane;
        const uint32_t first = (uint32_t)x.first(granule);
        float v[8];
        uint64_t own[8], mine = 0;
        x.load(granule, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t k = key_of(v[e]);
            bool in = k && cut.in(k, first + e);
            own[e] = in ? weight_of(k, in) : 0;
            mine += own[e];
        }
        const uint64_t upto = wave_incl64(mine);
        if (__ballot(upto > left)) {
            uint64_t at = upto - mine;
            if (at <= left && left < upto) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (at <= left && left < at + own[e])
                        answer(first + e, total);
                    at += own[e];
                }
            }
            return;
        }
        left -= __shfl((unsigned long long)upto, 63);
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
    g.row_blocks = (uint32_t)((waves + g.steps - 1) / g.steps);
    g.list = (uint32_t)(vocab < kList ? (vocab ? vocab : 1) : kList);
    const size_t fixed = kBins * 8 + (size_t)g.row_blocks * 12 + (size_t)g.list * 8 + 64 * kWaves * 8;
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
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char *p = body ? static_cast<char *>(body) + at : nullptr;
        at += align256(bytes * l.batch);
        return p;
    };
    g.best = reinterpret_cast<unsigned long long *>(take(g.parts * 8));
    g.hist = reinterpret_cast<unsigned long long *>(take(kBins * 8));
    g.sums = reinterpret_cast<unsigned long long *>(take(g.row_blocks * 8));
    g.entries = reinterpret_cast<unsigned long long *>(take((size_t)g.list * 8));
    g.counts = reinterpret_cast<uint32_t *>(take(g.row_blocks * 4));
    g.length = reinterpret_cast<uint32_t *>(take(4));
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
