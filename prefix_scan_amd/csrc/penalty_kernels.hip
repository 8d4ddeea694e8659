// penalty_kernels.hip -- repetition, presence and frequency penalties, biases
// and masks on rows of logits, in one pass.
//
// A workgroup has C logits of one row.  Those that the row's past tokens and
// biases name are a few of them: a bit each in LDS, whose rank among the bits
// is the logit's slot.  How often a token was there and which of its biases
// is the last are found by slot (whole numbers, so their order plays no part),
// then each slot's logit is worked out, one a thread, and the row goes out with
// the slots' logits and the mask.  Logits that nothing touches go out as they
// came; in place only what changes is written.
//
// Bound: waiting (69% of the waves' time; vector instructions are 18 of 61 us)
// for the steps before, which every workgroup of a row goes through with all of
// the row's lists.  256 rows of 150001 bf16 with 3000 tokens, 12 biases and 20
// masks: 61 us with 16384 logits a workgroup, 73 with 8192; with 10 tokens and
// nothing else 42, the copy alone 23.  With 384 slots, so that a compute unit
// holds four workgroups rather than three, 61 to 64.  With a count in LDS for
// every logit (4096 a workgroup) 82, and with each named logit put in its place
// among a thread's registers 106.
#include "penalty.hpp"
#include "device_common.hpp"
#include "rows_io.hpp"

namespace libscan {

namespace {

constexpr int kSlots = 1024;                    // named logits that are worked on at once
constexpr uint32_t kInPrompt = 0x80000000u;      // besides the count of what was written since

struct List {
    const int32_t *tokens;
    uint32_t len;
    uint64_t first;                              // where it starts among all rows' packed elements
};

__device__ __forceinline__ List list_of(const penalty_list_t &l, uint64_t r)
{
    if (!l.tokens)
        return List{nullptr, 0, 0};
    if (!l.ends)
        return List{l.tokens + (int64_t)r * l.row_stride, (uint32_t)l.count, 0};
    uint64_t lo = r ? l.ends[r - 1] : 0, hi = l.ends[r];
    hi = hi < l.count ? hi : l.count;
    lo = lo < hi ? lo : hi;
    return List{l.tokens + lo, (uint32_t)(hi - lo), lo};
}

template <int W, int S, int P, bool BIAS>
struct Shared {
    uint32_t bits[W];                 // named logits
    uint32_t rank[W + 1];             // how many there are before each word's
    uint32_t wave[16];
    uint32_t times[S];                // of each slot: how often its token was there; then its new logit
    uint32_t bias[BIAS ? S : 1];      // one more than its last bias's place in the list, or 0
    uint16_t place[S];
    piece_t row[P];                   // the logits as they came, then as they go out
};

constexpr int kBatch = 4;                         // tokens of a thread that are under way at once

// f(place, index in the list) for those of a list's tokens that lie among the
// `many` logits from c0 on.  (Vocabularies end below 2^31, and so negative
// tokens lie behind every place.)
template <int kThreads, class F>
__device__ __forceinline__ void each_here(const List &l, uint32_t tid, uint32_t c0, uint32_t many, F f)
{
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < l.len; j0 += kBatch * kThreads) {
        uint32_t i[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t j = j0 + u * kThreads + tid;
            i[u] = j < l.len ? (uint32_t)l.tokens[j] - c0 : ~0u;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i[u] < many)
                f(i[u], j0 + u * kThreads + tid);
    }
}

// A piece with minus infinity for the elements whose bit is set.
template <class T>
__device__ __forceinline__ piece_t shut_out(piece_t x, uint32_t shut)
{
    float all[kPiece<T>];
#pragma unroll
    for (int e = 0; e < kPiece<T>; ++e)
        all[e] = -__builtin_inff();
    const piece_t closed = Unpack<T>::pack(all);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const auto on = [&](int e) { return 0u - (shut >> e & 1); };
        const uint32_t which = kPiece<T> == 4 ? on(d) : (on(2 * d) & 0xFFFFu) | (on(2 * d + 1) & 0xFFFF0000u);
        x[d] = (x[d] & ~which) | (closed[d] & which);
    }
    return x;
}

template <class T, int kThreads, int kPieces, bool BIAS>
__global__ __launch_bounds__(kThreads, kThreads == 512 ? 4 : 2) void penalize_kernel(penalty_args_t p)
{
    constexpr int V = kPiece<T>, C = kThreads * V * kPieces, W = C / 32, S = C < kSlots ? C : kSlots;
    static_assert(W <= kThreads && C <= 65536 && V <= 32, "a thread a word; places of 16 bits");
    __shared__ Shared<W, S, kThreads * kPieces, BIAS> s;
    T *const row = reinterpret_cast<T *>(s.row);
    const uint64_t chunks = (p.vocab + C - 1) / C, all = p.rows * chunks;
    const bool in_place = p.logits == p.out;
    const piece_t none = {0, 0, 0, 0};
    for (uint64_t w = blockIdx.x; w < all; w += gridDim.x) {
        const uint64_t r = w / chunks;
        const uint32_t c0 = (uint32_t)(w % chunks) * C;
        uint32_t tid = threadIdx.x;
        const uint32_t many = p.vocab - c0 < C ? (uint32_t)p.vocab - c0 : C;
        const T *const from = static_cast<const T *>(p.logits) + (int64_t)r * p.row_stride + c0;
        T *const to = static_cast<T *>(p.out) + (int64_t)r * p.out_stride + c0;
        const auto place = [&](int q) { return (q * kThreads + tid) * V; };
        const auto left = [&](uint32_t i) { return i < many ? (int)(many - i < (uint32_t)V ? many - i : V) : 0; };
        const auto slot_of = [&](uint32_t i) {
            return s.rank[i / 32] + __popc(s.bits[i / 32] & ((1u << (i % 32)) - 1));
        };

        piece_t raw[kPieces];
        if (!in_place) {
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                raw[q] = left(place(q)) ? load_piece<T>(from + place(q), left(place(q))) : none;
        }
        const List past = list_of(p.past, r);
        const List bias = BIAS ? list_of(p.bias, r) : List{nullptr, 0, 0};
        const float *const values =
            !BIAS ? nullptr : p.bias_values + (p.bias.ends ? (int64_t)bias.first : (int64_t)r * p.bias_stride);
        const int64_t prompts = p.prompts ? p.prompts[r] : 0;
        const uint32_t prompt = prompts > 0 ? prompts < (int64_t)~0u ? (uint32_t)prompts : ~0u : 0;
        const int64_t grammar = !p.mask ? -1 : p.mask_slots ? p.mask_slots[r] : (int64_t)r;
        float rep = p.repetitions ? p.repetitions[r] : p.repetition;
        float presence = p.presences ? p.presences[r] : p.presence;
        float frequency = p.frequencies ? p.frequencies[r] : p.frequency;
        const uint32_t *const mask =
            grammar >= 0 && (uint64_t)grammar < p.masks ? p.mask + grammar * p.mask_stride + c0 / 32 : nullptr;
        uint32_t allowed[kPieces];
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
            allowed[q] = mask && left(place(q)) ? mask[place(q) / 32] >> (place(q) % 32) : ~0u;
        rep = rep > 0.f ? rep : 1.f;
        presence = presence == presence ? presence : 0.f;
        frequency = frequency == frequency ? frequency : 0.f;

        // The thread's number is read anew for each step: places and addresses are
        // kept from one to the next otherwise, and spill.
        const auto anew = [&]() {
            __syncthreads();
            asm volatile("" : "+v"(tid));
        };

        if (tid < W)
            s.bits[tid] = 0;
        __syncthreads();
        const auto name = [&](uint32_t i, uint32_t) { atomicOr(&s.bits[i / 32], 1u << (i % 32)); };
        each_here<kThreads>(past, tid, c0, many, name);
        if (BIAS)
            each_here<kThreads>(bias, tid, c0, many, name);
        if (!in_place) {
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                s.row[q * kThreads + tid] = raw[q];
        }
        anew();
        uint32_t bits = tid < W ? s.bits[tid] : 0, sum = wave_incl_add((uint32_t)__popc(bits));
        if (tid % 64 == 63)
            s.wave[tid / 64] = sum;
        __syncthreads();
        for (uint32_t v = 0; v < tid / 64; ++v)
            sum += s.wave[v];
        if (tid < W)
            s.rank[tid + 1] = sum;
        if (tid == 0)
            s.rank[0] = 0;
        __syncthreads();
        const uint32_t named = s.rank[W];
        // Words [w0, w1): as many as there are slots for, mostly all.
        for (uint32_t w0 = 0; w0 < (uint32_t)W;) {
            const uint32_t base = s.rank[w0];
            uint32_t w1 = W;
            if (named - base > (uint32_t)S) {
                uint32_t past_it = W;
                w1 = w0 + 1;
                while (past_it - w1 > 1) {
                    const uint32_t mid = w1 + (past_it - w1) / 2;
                    if (s.rank[mid] - base <= (uint32_t)S)
                        w1 = mid;
                    else
                        past_it = mid;
                }
            }
            const uint32_t n = s.rank[w1] - base;
            if (n != 0) {
                for (uint32_t k = tid; k < n; k += kThreads) {
                    s.times[k] = 0;
                    if (BIAS)
                        s.bias[k] = 0;
                }
                if (tid >= w0 && tid < w1) {
                    uint32_t k = s.rank[tid] - base;
                    for (uint32_t b = bits; b != 0; b &= b - 1)
                        s.place[k++] = (uint16_t)(tid * 32 + __builtin_ctz(b));
                }
                anew();
                each_here<kThreads>(past, tid, c0, many, [&](uint32_t i, uint32_t j) {
                    const uint32_t k = slot_of(i) - base;
                    if (k >= n)
                        return;
                    if (j >= prompt)
                        atomicAdd(&s.times[k], 1u);
                    else
                        atomicOr(&s.times[k], kInPrompt);
                });
                if (BIAS) {
                    each_here<kThreads>(bias, tid, c0, many, [&](uint32_t i, uint32_t j) {
                        const uint32_t k = slot_of(i) - base;
                        if (k < n)
                            atomicMax(&s.bias[k], j + 1);
                    });
                }
                anew();
                for (uint32_t k = tid; k < n; k += kThreads) {
                    const uint32_t times = s.times[k], since = times & ~kInPrompt, b = BIAS ? s.bias[k] : 0;
                    const uint32_t i = s.place[k];
                    float y = (float)(in_place ? from[i] : row[i]);
                    const float more = BIAS && b ? values[b - 1] : 0.f;
                    if (times) {
                        y = y > 0.f ? y / rep : y * rep;
                        y -= since ? __builtin_fmaf(frequency, (float)since, presence) : 0.f;
                    }
                    if (BIAS && b)
                        y += more;
                    if (!in_place)
                        row[i] = (T)y;
                    else if (!mask || (mask[i / 32] >> (i % 32) & 1))
                        to[i] = (T)y;
                }
            }
            anew();
            w0 = w1;
        }
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const uint32_t i = place(q), shut = ~allowed[q] & ((1u << V) - 1);
            const int m = left(i);
            if (m == 0)
                continue;
            if (!in_place || shut == (1u << V) - 1) {
                piece_t x = in_place ? none : s.row[q * kThreads + tid];
                if (mask)
                    x = shut_out<T>(x, shut);
                store_piece<T>(to + i, x, m);
            } else if (shut != 0) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < m && (shut >> e & 1))
                        to[i + e] = (T)-__builtin_inff();
            }
        }
        anew();
    }
}

template <class T, int kThreads, int kPieces>
hipError_t run_penalize(const penalty_args_t &a, hipStream_t stream)
{
    constexpr int C = kThreads * kPieces * kPiece<T>;
    const uint64_t all = a.rows * ((a.vocab + C - 1) / C);
    const unsigned grid = (unsigned)(all < (1u << 22) ? all : 1u << 22);
    if (a.bias.tokens)
        penalize_kernel<T, kThreads, kPieces, true><<<grid, kThreads, 0, stream>>>(a);
    else
        penalize_kernel<T, kThreads, kPieces, false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

// Workgroups of 512 threads and 16384 logits (f32: 8192), or of 256 and 2048 (1024)
// where the large ones would be fewer than 512, two a compute unit.  Each goes
// through all of its row's list, so that large ones do less in all; small ones are
// more, which counts where lists are long and rows few.  bf16, vocabulary of 32000,
// us by small and by large workgroups, lists of 1000 | of 32768 tokens:
//     16 rows, 32 large workgroups      7.3  7.4 |   80  186
//     64 rows, 128                      7.4  7.6 |  153  189
//    128 rows, 256                     12.6  8.1 |  267  295
//    192 rows, 384                     14.8  9.1 |  309  299
//    256 rows, 512                     20.3 10.1 |  449  330
//   1024 rows, 2048                    72.1 32.4 | 1626  994
// (f32 and 150001 logits alike.)  Between 256 and 512 short lists would gain by the
// large ones and long lists of few rows lose.
template <class T>
hipError_t size_penalize(const penalty_args_t &a, hipStream_t stream)
{
    constexpr uint64_t C = 512 * 4 * kPiece<T>;
    return a.rows * ((a.vocab + C - 1) / C) < 512 ? run_penalize<T, 256, 1>(a, stream)
                                                  : run_penalize<T, 512, 4>(a, stream);
}

}  // namespace

hipError_t launch_penalize(const penalty_args_t &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: return size_penalize<float>(a, stream);
    case LIBSCAN_BF16: return size_penalize<__bf16>(a, stream);
    default: return size_penalize<_Float16>(a, stream);
    }
}

}  // namespace libscan
