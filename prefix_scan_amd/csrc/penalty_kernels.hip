// penalty_kernels.hip -- repetition, presence and frequency penalties, biases
// and masks on rows of logits, in one pass.
//
// A workgroup has C logits of one row.  It counts the row's past tokens among
// them in LDS (whole numbers, so their order plays no part), notes for each
// the last bias that names it, and goes over the logits once.  Rows that
// nothing touches are copied as they are.
//
// Bound: memory, the logits' bytes once in and once out.  Every workgroup of
// a row reads the row's past tokens: more logits a workgroup read them less
// often, fewer fill the GPU with few rows.
#include "penalty.hpp"
#include "rows_io.hpp"

namespace libscan {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInPrompt = 0x80000000u;      // besides the count of what was written since

struct List {
    const int32_t *tokens;
    uint64_t len, first;                         // first: where it starts among all rows' packed elements
};

__device__ __forceinline__ List list_of(const penalty_list_t &l, uint64_t r)
{
    if (!l.tokens)
        return List{nullptr, 0, 0};
    if (!l.ends)
        return List{l.tokens + (int64_t)r * l.row_stride, l.count, 0};
    uint64_t lo = r ? l.ends[r - 1] : 0, hi = l.ends[r];
    hi = hi < l.count ? hi : l.count;
    lo = lo < hi ? lo : hi;
    return List{l.tokens + lo, hi - lo, lo};
}

template <class T, int C, bool BIAS>
__global__ __launch_bounds__(kThreads) void penalize_kernel(penalty_args_t p)
{
    constexpr int V = kPiece<T>, kPieces = C / (kThreads * V), kBatch = 4;
    static_assert(kPieces * kThreads * V == C, "whole pieces");
    __shared__ __align__(16) uint32_t s_times[C];
    __shared__ __align__(16) uint32_t s_bias[BIAS ? C : 4];
    const uint64_t chunks = (p.vocab + C - 1) / C, all = p.rows * chunks;
    const bool in_place = p.logits == p.out;
    const piece_t none = {0, 0, 0, 0};
    for (uint64_t w = blockIdx.x; w < all; w += gridDim.x) {
        const uint64_t r = w / chunks, c0 = w % chunks * C;
        const uint32_t many = p.vocab - c0 < C ? (uint32_t)(p.vocab - c0) : C;
        const T *const from = static_cast<const T *>(p.logits) + (int64_t)r * p.row_stride + c0;
        T *const to = static_cast<T *>(p.out) + (int64_t)r * p.out_stride + c0;
        const auto left = [&](uint32_t i) { return i < many ? (int)(many - i < (uint32_t)V ? many - i : V) : 0; };

        piece_t raw[kPieces];
        if (!in_place) {
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const uint32_t i = (q * kThreads + threadIdx.x) * V;
                raw[q] = left(i) ? load_piece<T>(from + i, left(i)) : none;
            }
        }
        for (uint32_t i = threadIdx.x; i < C / 4; i += kThreads) {
            reinterpret_cast<piece_t *>(s_times)[i] = none;
            if (BIAS)
                reinterpret_cast<piece_t *>(s_bias)[i] = none;
        }
        __syncthreads();
        const List past = list_of(p.past, r);
        const int64_t prompt = p.prompts ? p.prompts[r] : 0;
        for (uint64_t j0 = threadIdx.x; j0 < past.len; j0 += kBatch * kThreads) {
            int32_t t[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                t[u] = j0 + u * kThreads < past.len ? past.tokens[j0 + u * kThreads] : -1;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint64_t i = (uint64_t)(int64_t)t[u] - c0;
                if (t[u] >= 0 && i < many) {
                    if ((int64_t)(j0 + u * kThreads) >= prompt)
                        atomicAdd(&s_times[i], 1u);
                    else
                        atomicOr(&s_times[i], kInPrompt);
                }
            }
        }
        const float *values = nullptr;
        if (BIAS) {
            const List bias = list_of(p.bias, r);
            values = p.bias_values + (p.bias.ends ? (int64_t)bias.first : (int64_t)r * p.bias_stride);
            for (uint64_t j = threadIdx.x; j < bias.len; j += kThreads) {
                const int32_t t = bias.tokens[j];
                const uint64_t i = (uint64_t)(int64_t)t - c0;
                if (t >= 0 && i < many)
                    atomicMax(&s_bias[i], (uint32_t)j + 1);
            }
        }
        float rep = p.repetitions ? p.repetitions[r] : p.repetition;
        float presence = p.presences ? p.presences[r] : p.presence;
        float frequency = p.frequencies ? p.frequencies[r] : p.frequency;
        rep = rep > 0.f ? rep : 1.f;
        presence = presence == presence ? presence : 0.f;
        frequency = frequency == frequency ? frequency : 0.f;
        const uint32_t *mask = nullptr;
        if (p.mask) {
            const int64_t slot = p.mask_slots ? p.mask_slots[r] : (int64_t)r;
            if (slot >= 0 && (uint64_t)slot < p.masks)
                mask = p.mask + slot * p.mask_stride + c0 / 32;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const uint32_t i = (q * kThreads + threadIdx.x) * V;
            const int n = left(i);
            if (n == 0)
                continue;
            uint32_t times[V], bias[V], any = 0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                times[e] = s_times[i + e];
                bias[e] = BIAS ? s_bias[i + e] : 0;
                any |= times[e] | bias[e];
            }
            const uint32_t allowed = mask ? mask[i / 32] >> (i % 32) : ~0u;
            if (any == 0 && (~allowed & ((1u << n) - 1)) == 0) {
                if (!in_place)
                    store_piece<T>(to + i, raw[q], n);
                continue;
            }
            const piece_t x = in_place ? load_piece<T>(from + i, n) : raw[q];
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = Unpack<T>::get(x, e);
                if (times[e]) {
                    const uint32_t since = times[e] & ~kInPrompt;
                    y[e] = y[e] > 0.f ? y[e] / rep : y[e] * rep;
                    y[e] -= since ? __builtin_fmaf(frequency, (float)since, presence) : 0.f;
                }
                if (BIAS && bias[e])
                    y[e] += values[bias[e] - 1];
                if (!(allowed >> e & 1))
                    y[e] = -__builtin_inff();
            }
            store_piece<T>(to + i, Unpack<T>::pack(y), n);
        }
        __syncthreads();
    }
}

template <class T, int C>
hipError_t run_penalize(const penalty_args_t &a, hipStream_t stream)
{
    const uint64_t all = a.rows * ((a.vocab + C - 1) / C);
    const unsigned grid = (unsigned)(all < (1u << 23) ? all : 1u << 23);
    if (a.bias.tokens)
        penalize_kernel<T, C, true><<<grid, kThreads, 0, stream>>>(a);
    else
        penalize_kernel<T, C, false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T>
hipError_t size_penalize(const penalty_args_t &a, hipStream_t stream)
{
    return a.rows * ((a.vocab + 4095) / 4096) < 1024 ? run_penalize<T, 2048>(a, stream)
                                                     : run_penalize<T, 4096>(a, stream);
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
