// gatescan_tile.hpp -- the kernel of the gated recurrence and of its gradient
// (gatescan.hpp has the formulas), on one tile a workgroup.
//
// A thread has R tokens, one after another, of 16 bytes of channels; eight
// lanes share a row, so that each load of a wave is eight whole lines.  The
// threads scan their tokens, one wave chains the groups of a channel through
// LDS, takes the carry from the tiles before and hands every group its own,
// and the threads go over their tokens once more from there.
//
// Bound: memory.  Rows are read and written once (descriptors of the carry
// add 1.5 KB to a tile of 48 KB and more).  Tiles are drawn from a ticket
// in the order of their place in their lines, all lines' first tiles first: a
// tile waits only on tiles that were drawn before it.
#pragma once

#include "device_common.hpp"
#include "gatescan.hpp"
#include "linattn.hpp"
#include "rows_io.hpp"

namespace libscan {

// a and 1 - a of a gate.  e^x is 2^(x log2 e) with what that product's rounding
// left put back (log2 e in two parts), so that it is good to about one step at
// any x; past 200 of 0 the power has long been 0 or infinite.  Near a = 1 the
// smaller of a and 1 - a is computed and the other is 1 less it: a state's
// memory is 1 / (1 - a) tokens long, and each step's error counts that often.
__device__ __forceinline__ float gate_exp(float x)
{
    x = x > 200.f ? 200.f : x;
    x = x < -200.f ? -200.f : x;
    const float hi = 1.44269502f, lo = 1.92596299e-8f;
    const float t = x * hi;
    const float rest = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    // rest is below 2^-16: 2^rest = 1 + rest ln 2.
    return __builtin_fmaf(p, p < __builtin_inff() ? rest * 0.693147182f : 0.f, p);
}

struct Gate {
    float a, rest;       // a, 1 - a
};

template <int FORM>
__device__ __forceinline__ Gate gate_of(float g)
{
    if (FORM == GATESCAN_DECAY)
        return Gate{g, 1.f - g};
    if (FORM == GATESCAN_SIGMOID) {
        const float e = gate_exp(-__builtin_fabsf(g)), d = 1.f + e;
        float r = __builtin_amdgcn_rcpf(d);
        r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
        const float small = e * r, large = 1.f - small;
        return g < 0.f ? Gate{small, large} : Gate{large, small};
    }
    // 1 - e^g from its series near 0 (eight terms: 0.35^8 / 9! is below 2^-30).
    float s = __builtin_fmaf(g, 1.f / 40320.f, 1.f / 5040.f);
    s = __builtin_fmaf(s, g, 1.f / 720.f);
    s = __builtin_fmaf(s, g, 1.f / 120.f);
    s = __builtin_fmaf(s, g, 1.f / 24.f);
    s = __builtin_fmaf(s, g, 1.f / 6.f);
    s = __builtin_fmaf(s, g, 0.5f);
    s = __builtin_fmaf(s * g, g, g);
    const float p = gate_exp(g);
    return __builtin_fabsf(g) < 0.35f ? Gate{1.f + s, -s} : Gate{p, 1.f - p};
}

// A product of gates that has left the floats counts as the smallest of them,
// not as zero, unless one of its factors is zero: an infinite state stays one.
__device__ __forceinline__ float kept_product(float A, bool zero)
{
    return A == 0.f && !zero ? __builtin_copysignf(1.40129846e-45f, A) : A;
}

template <class T, int FORM, bool BLEND, bool GRAD>
__global__ __launch_bounds__(kGateThreads, 4) void gatescan_kernel(GateArgs p)
{
    typedef Unpack<T> U;
    constexpr int V = kPiece<T>, C = kGateLanes * V, G = kGateGroups;
    constexpr int R = gate_rows(sizeof(T) == 4 ? LIBSCAN_F32 : LIBSCAN_BF16, GRAD), TT = G * R;
    static_assert(C <= 64 && G <= C, "one wave chains the groups");
    __shared__ __align__(16) float s_a[G][C], s_h[G][C];
    __shared__ uint32_t s_reset[G];
    __shared__ int32_t s_first[TT], s_last[TT];     // the sequence that starts / ends at a token, or -1
    __shared__ uint32_t s_ticket[2], s_seq;

    const int tid = threadIdx.x, lane8 = tid % kGateLanes, group = tid / kGateLanes;
    const bool chained = p.tiles > 1;
    uint32_t at = blockIdx.x, tag = 0;
    if (chained) {
        if (tid == 0) {
            const TileTicket t = draw_ticket(p.ticket, p.chains * p.tiles);
            s_ticket[0] = t.tile;
            s_ticket[1] = t.tag;
        }
        __syncthreads();
        at = __builtin_amdgcn_readfirstlane(s_ticket[0]);
        tag = __builtin_amdgcn_readfirstlane(s_ticket[1]);
    }
    const uint32_t k = at / p.chains, chain = at % p.chains;
    const uint32_t seq = chain / p.blocks;
    const uint64_t c0 = (uint64_t)(chain % p.blocks) * C + lane8 * V;
    const int n = c0 < p.width ? (int)(p.width - c0 < (uint64_t)V ? p.width - c0 : V) : 0;

    // Tokens [0, end) are in sequences; the tile has places [k TT, k TT + TT) in
    // the sweep's order, the thread R from `place` on.
    uint64_t end = p.tokens;
    if (p.ends) {
        const uint64_t last = p.ends[p.seqs - 1];
        end = last < end ? last : end;
    }
    const uint64_t tile0 = (uint64_t)k * TT;
    const uint64_t place = tile0 + (uint64_t)group * R;
    const auto token = [&](int r) -> int64_t {
        const int64_t x = (int64_t)(place + r);
        return GRAD ? (int64_t)p.tokens - 1 - x : x;
    };
    const auto inside = [&](int r) { const int64_t t = token(r); return t >= 0 && t < (int64_t)end; };
    const auto row = [&](const GateRows &s, int64_t t) {
        return static_cast<const T *>(s.p) + (int64_t)seq * s.seq + t * s.tok + c0;
    };

    // All of the thread's rows are asked for at once.
    const bool whole = inside(0) && inside(R - 1);
    piece_t rg[R], rx[R], rd[R], rh[R];
    const piece_t none = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rg[r] = rx[r] = rd[r] = rh[r] = none;
        if (n > 0 && (whole || inside(r))) {
            const int64_t t = token(r);
            rg[r] = load_piece<T>(row(p.gate, t), n);
            if (!GRAD || BLEND)
                rx[r] = load_piece<T>(row(p.x, t), n);
            if (GRAD) {
                rd[r] = load_piece<T>(row(p.dout, t), n);
                if (t > 0)
                    rh[r] = load_piece<T>(row(p.h, t - 1), n);
            }
        }
    }

    // Where sequences start and end among the tile's tokens.
    uint32_t firsts = 0, lasts = 0;      // the thread's, a bit a token
    const int64_t tok0 = GRAD ? (int64_t)p.tokens - (int64_t)(tile0 + TT) : (int64_t)tile0;   // lowest token
    if (p.ends) {
        for (int i = tid; i < TT; i += kGateThreads)
            s_first[i] = s_last[i] = -1;
        if (tid < 64) {
            // Sequences that start at tok0 or later, and the one before them.
            const uint32_t s = tok0 > 0 ? first_above(p.ends, p.seqs, (uint64_t)tok0 - 1) : 0;
            if (tid == 0)
                s_seq = s;
        }
        __syncthreads();
        const bool top = GRAD ? k == 0 : k == p.tiles - 1;      // what lies past the rows is the last tile's
        for (uint32_t s = s_seq + tid;; s += kGateThreads) {
            bool more = s < p.seqs;
            uint64_t first = 0, len = 0;
            if (more) {
                run_of(p.ends, p.tokens, s, &first, &len);
                more = top || (int64_t)first < tok0 + TT;
            }
            if (more && len) {
                if ((int64_t)first >= tok0 && (int64_t)first < tok0 + TT)
                    s_first[first - tok0] = (int32_t)s;
                const int64_t l = (int64_t)(first + len) - 1;
                if (l >= tok0 && l < tok0 + TT)
                    s_last[l - tok0] = (int32_t)s;
            } else if (more && p.state_out && (int64_t)first >= tok0) {
                // An empty sequence passes its state (or its gradient) through.
                const float *from = GRAD ? p.last : p.first;
                const uint64_t b0 = (uint64_t)(chain % p.blocks) * C;
                for (uint64_t c = b0; c < b0 + C && c < p.width; ++c)
                    p.state_out[s * p.width + c] = from ? from[s * p.width + c] : 0.f;
            }
            if (__syncthreads_count(more) < kGateThreads)
                break;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (inside(r)) {
                firsts |= (s_first[token(r) - tok0] >= 0 ? 1u : 0u) << r;
                lasts |= (s_last[token(r) - tok0] >= 0 ? 1u : 0u) << r;
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            firsts |= (token(r) == 0 ? 1u : 0u) << r;
            lasts |= (token(r) == (int64_t)end - 1 ? 1u : 0u) << r;
        }
    }
    const auto out_at = [&](int i, int64_t t) {
        return static_cast<T *>(p.out[i]) + (int64_t)seq * p.out_seq[i] + t * p.out_tok[i] + c0;
    };
    // Rows that are in no sequence.  A tile of nothing else is done: no tile
    // with tokens looks back to it.
    const auto clear = [&](int r) {
        const int64_t t = token(r);
        if (p.clear && n > 0 && t >= 0 && t < (int64_t)p.tokens) {
            store_piece<T>(out_at(0, t), none, n);
            if (GRAD)
                store_piece<T>(out_at(1, t), none, n);
        }
    };
    if ((tok0 > 0 ? tok0 : 0) >= (int64_t)end) {
        for (int r = 0; r < R; ++r)
            clear(r);
        // Equal sequences of no tokens pass their states through.
        if (!p.ends && p.state_out && group == 0 && n > 0) {
            float v[V] = {};
            const float *from = GRAD ? p.last : p.first;
            if (from)
                load_floats<V>(from + seq * p.width + c0, n, v);
            store_floats<V>(p.state_out + seq * p.width + c0, n, v);
        }
        return;
    }
    const auto seq_of = [&](const int32_t *marks, int r) -> uint64_t {
        return p.ends ? (uint64_t)(uint32_t)marks[token(r) - tok0] : seq;
    };
    const uint32_t resets = GRAD ? lasts : firsts;       // where the sweep starts anew
    // A wave without starts, ends and rows outside takes the short way.
    const bool plain = !__any(!whole || (firsts | lasts) != 0);

    // The thread's own tokens: (A, H) of each channel.
    float A[V], H[V];
    bool zero[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        A[e] = 1.f;
        H[e] = 0.f;
        zero[e] = false;
    }
    float fa[GRAD ? 1 : R][V], fb[GRAD ? 1 : R][V];      // forward: a and b, kept for the second pass
    (void)fa;
    (void)fb;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (!plain && !inside(r)) {
            if (!GRAD) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    fa[r][e] = 1.f;
                    fb[r][e] = 0.f;
                }
            }
            continue;
        }
        const bool reset = !plain && (resets >> r & 1) != 0;
        float from[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            from[e] = 0.f;
        if (reset) {
            const float *s = GRAD ? p.last : p.first;
            if (s)
                load_floats<V>(s + seq_of(GRAD ? s_last : s_first, r) * p.width + c0, n, from);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Gate w = gate_of<FORM>(U::get(rg[r], e));
            if (GRAD) {
                const float d = U::get(rd[r], e);
                H[e] = w.a * ((reset ? from[e] : H[e]) + d);
            } else {
                const float x = U::get(rx[r], e), b = BLEND ? w.rest * x : x;
                // A sequence's first token takes in the state before it.
                fa[r][e] = w.a;
                H[e] = __builtin_fmaf(w.a, reset ? from[e] : H[e], b);
                fb[r][e] = reset ? H[e] : b;
            }
            A[e] = reset ? 0.f : A[e] * w.a;
            zero[e] |= w.a == 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        s_a[group][lane8 * V + e] = kept_product(A[e], zero[e]);
#pragma unroll
    for (int e = 0; e < V; ++e)
        s_h[group][lane8 * V + e] = H[e];
    if (lane8 == 0)
        s_reset[group] = resets;
    __syncthreads();

    // One lane a channel: the tile's pair, the carry, and each group's.
    if (tid < C) {
        const uint64_t anew = __ballot(tid < G && s_reset[tid % G] != 0);
        // The first tile of the line that has tokens starts a sequence.
        const uint32_t k0 = GRAD && p.ends ? (uint32_t)((p.tokens - end) / TT) : 0;
        uint64_t *const mine = p.desc + ((uint64_t)at * 2) * C + tid;      // A; H is C further on
        float carry = 0.f;
        if (chained) {
            float a = 1.f, h = 0.f;
            bool none_zero = true;
#pragma unroll 8
            for (int g = 0; g < G; ++g) {
                const float ga = s_a[g][tid], gh = s_h[g][tid];
                if (anew >> g & 1) {
                    a = 0.f;
                    h = gh;
                } else {
                    a *= ga;
                    h = __builtin_fmaf(ga, h, gh);
                }
                none_zero = none_zero && ga != 0.f;
            }
            const bool known = anew != 0 || k <= k0;
            const auto word = [&](uint32_t status, float v) {
                return (uint64_t)(tag | status) << 32 | __builtin_bit_cast(uint32_t, v);
            };
            const auto put = [&](uint64_t *to, uint64_t w) {
                __hip_atomic_store(to, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            };
            const auto get = [&](uint32_t tile, int half) {
                return __hip_atomic_load(p.desc + ((uint64_t)(tile * p.chains + chain) * 2 + half) * C + tid,
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            };
            const auto status = [&](uint64_t w) {
                const uint32_t hi = (uint32_t)(w >> 32);
                return (hi & ~3u) == tag ? hi & 3u : 0u;
            };
            const auto value = [&](uint64_t w) { return __builtin_bit_cast(float, (uint32_t)w); };
            if (known) {
                put(mine + C, word(kStatusPrefix, h));
            } else {
                put(mine, word(kStatusAgg, kept_product(a, !none_zero)));
                put(mine + C, word(kStatusAgg, h));
            }
            if (k > k0) {
                // The nearest tile whose chained value is there, among the
                // last kWindow, with the pairs of all between.
                constexpr int kStep = 4, kWindow = 32;
                uint64_t wa[kStep], wh[kStep];
                int found = -1;
                while (found < 0) {
                    for (int b = 0; b < kWindow && found < 0; b += kStep) {
                        bool ready = true;
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            const uint32_t back = (uint32_t)(b + i) < k - k0 ? b + i : k - k0 - 1;
                            wh[i] = get(k - 1 - back, 1);
                            wa[i] = b == 0 ? get(k - 1 - back, 0) : 0;
                        }
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            if (found < 0 && ready) {
                                if (__all(status(wh[i]) == kStatusPrefix))
                                    found = b + i;
                                else
                                    ready = __all(status(wh[i]) != 0 && (b != 0 || status(wh[i]) == kStatusPrefix ||
                                                                         status(wa[i]) != 0));
                            }
                        }
                        if (!ready)
                            break;
                    }
                    if (found < 0)
                        __builtin_amdgcn_s_sleep(1);
                }
                if (found < kStep) {
#pragma unroll
                    for (int i = kStep - 1; i >= 0; --i) {
                        if (i <= found)
                            carry = status(wh[i]) == kStatusPrefix
                                        ? value(wh[i])
                                        : __builtin_fmaf(value(wa[i]), carry, value(wh[i]));
                    }
                } else {
                    for (int b = found; b >= 0; b -= kStep) {
                        bool ready = false;
                        while (!ready) {
                            ready = true;
#pragma unroll
                            for (int i = 0; i < kStep; ++i) {
                                const uint32_t tile = k - 1 - (b - i > 0 ? b - i : 0);
                                wh[i] = get(tile, 1);
                                wa[i] = get(tile, 0);
                            }
#pragma unroll
                            for (int i = 0; i < kStep; ++i)
                                ready = ready && status(wh[i]) != 0 &&
                                        (status(wh[i]) == kStatusPrefix || status(wa[i]) != 0);
                            ready = __all(ready);
                        }
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            if (b - i >= 0)
                                carry = status(wh[i]) == kStatusPrefix
                                            ? value(wh[i])
                                            : __builtin_fmaf(value(wa[i]), carry, value(wh[i]));
                        }
                    }
                }
                if (!known)
                    put(mine + C, word(kStatusPrefix, __builtin_fmaf(kept_product(a, !none_zero), carry, h)));
            }
        }
#pragma unroll 8
        for (int g = 0; g < G; ++g) {
            const float ga = s_a[g][tid], gh = s_h[g][tid];
            s_h[g][tid] = carry;
            carry = anew >> g & 1 ? gh : __builtin_fmaf(ga, carry, gh);
        }
    }
    __syncthreads();

    // Once more over the thread's tokens, from what enters them.
#pragma unroll
    for (int e = 0; e < V; ++e)
        H[e] = s_h[group][lane8 * V + e];
    if (n == 0)
        return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t t = token(r);
        if (!plain && !inside(r)) {
            clear(r);
            continue;
        }
        const bool reset = !plain && (resets >> r & 1) != 0;
        if (!GRAD) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                H[e] = reset ? fb[r][e] : __builtin_fmaf(fa[r][e], H[e], fb[r][e]);
            store_piece<T>(out_at(0, t), U::pack(H), n);
            if (!plain && (lasts >> r & 1) && p.state_out)
                store_floats<V>(p.state_out + seq_of(s_last, r) * p.width + c0, n, H);
            continue;
        }
        const bool starts = !plain && (firsts >> r & 1) != 0;
        if (reset) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                H[e] = 0.f;
            if (p.last)
                load_floats<V>(p.last + seq_of(s_last, r) * p.width + c0, n, H);
        }
        float before[V], dg[V], dx[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            before[e] = U::get(rh[r], e);
        if (starts) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                before[e] = 0.f;
            if (p.first)
                load_floats<V>(p.first + seq_of(s_first, r) * p.width + c0, n, before);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Gate w = gate_of<FORM>(U::get(rg[r], e));
            const float dh = U::get(rd[r], e) + H[e];
            H[e] = w.a * dh;
            dx[e] = BLEND ? dh * w.rest : dh;
            const float da = dh * (BLEND ? before[e] - U::get(rx[r], e) : before[e]);
            dg[e] = FORM == GATESCAN_DECAY ? da : FORM == GATESCAN_LOG ? da * w.a : da * (w.a * w.rest);
        }
        store_piece<T>(out_at(0, t), U::pack(dg), n);
        store_piece<T>(out_at(1, t), U::pack(dx), n);
        if (starts && p.state_out)
            store_floats<V>(p.state_out + seq_of(s_first, r) * p.width + c0, n, H);
    }
}

template <class T, bool GRAD>
hipError_t launch_gate_tiles(const GateArgs &a, hipStream_t stream)
{
    const unsigned grid = a.chains * a.tiles;
#define LIBSCAN_GATE(FORM)                                                                        \
    if (a.form == FORM) {                                                                         \
        if (a.blend)                                                                              \
            gatescan_kernel<T, FORM, true, GRAD><<<grid, kGateThreads, 0, stream>>>(a);           \
        else                                                                                      \
            gatescan_kernel<T, FORM, false, GRAD><<<grid, kGateThreads, 0, stream>>>(a);          \
    }
    LIBSCAN_GATE(GATESCAN_DECAY)
    LIBSCAN_GATE(GATESCAN_LOG)
    LIBSCAN_GATE(GATESCAN_SIGMOID)
#undef LIBSCAN_GATE
    return hipGetLastError();
}

}  // namespace libscan
