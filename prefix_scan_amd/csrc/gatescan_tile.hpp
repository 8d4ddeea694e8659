// gatescan_tile.hpp -- the kernel of the gated recurrence and of its gradient
// (gatescan.hpp has the formulas).
//
// A thread has R tokens, one after another, of 16 bytes of channels; eight
// lanes share a row, so that each load of a wave is eight whole lines.  Per
// tile,
//   1. the threads scan their tokens and leave a pair for each channel in LDS;
//   2. one wave, a lane a channel, chains the pairs of the tile's groups, looks
//      back for what enters the tile and publishes what leaves it;
//   3. the threads go over their tokens once more from what enters them, and
//      store.
//
// Bound: memory, or with few lines the chain of carries.  Rows are read and
// written once (descriptors of the carry add 1.5 KB to a tile of 48 KB and
// more).  A workgroup draws one tile, from one of eight counters that each have
// a share of the lines that lie side by side, in the order of the tiles' place
// in their lines: a tile waits only on tiles that were drawn before it.  One
// word's draws are served 12 ns apart, and a tile of 48 KB takes 7: from one
// ticket 8 x 4096 x 2048 bf16 took 118 us, from eight counters 87, where a copy
// of the same tiles takes 69 to 78 and the bytes at the card's best rate 60.
// (With a load before the draw's atomic, a second trip to memory that
// everything else waits for, 157; with several tiles a draw, one after
// another, 109, as each waits for the one before.)  A line's carry takes 0.16 us a
// tile: one to eight lines of 1025 tiles 164 to 198 us.  Of 16 such lines (131073 x
// 1024) 64 tiles each fit on the card at once, and a tile is there for 15 us from its
// draw to its last store: 234 us.
//
// Both paths are in one kernel, which has the registers of the other path: 128 with
// 16 spilled (forward, 16 bits), 64 to 87 (f32), 30 to 76 (gradients; log of 16 bits
// 122, 205 with blend).  The whole tiles' path alone takes 87 to 101 (forward) and
// 90 to 128 (gradients), of which log with blend of 16 bits spills two or three.
//
// Rows of whole tiles are read and written past what the caches keep.  8 x 4096 x
// 2048 bf16 takes 89 us so, 88 with stores like any others and 99 with loads like
// any others too, its gradient 151, 136 and 157; with a kernel after it that reads
// the outputs 132, 127 and 146 (gradient 215, 210 and 215).  32 x 128 x 8192, which
// the caches hold, 39, 40 and 33, and 63, 60 and 54 with that kernel: there the
// marks cost more than they save.
#pragma once

#include "device_common.hpp"
#include "gatescan.hpp"
#include "linattn.hpp"
#include "rows_io.hpp"

namespace libscan {

// a and 1 - a of a gate.  e^x is 2^(x log2 e).  For f32 rows what that
// product's rounding left is put back (log2 e in two parts), so that it is
// good to about one step at any x; 16-bit rows are rounded to 2^-9 and 2^-12
// of themselves, and an error of x 2^-24 in e^x is left in.  Near a = 1 the
// smaller of a and 1 - a is computed and the other is 1 less it, for all rows:
// a state's memory is 1 / (1 - a) tokens long, and each step's error counts
// that often.
template <bool FINE>
__device__ __forceinline__ float gate_exp(float x)
{
    const float hi = 1.44269502f, lo = 1.92596299e-8f;
    const float t = x * hi, p = __builtin_amdgcn_exp2f(t);
    if (!FINE)
        return p;
    // rest is below 2^-16: 2^rest = 1 + rest ln 2.  Nothing is put back to 0
    // and infinity, where rest may be NaN.
    const float rest = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
    return p > 0.f && p < __builtin_inff() ? __builtin_fmaf(p, rest * 0.693147182f, p) : p;
}

struct Gate {
    float a, rest;       // a, 1 - a
};

template <int FORM, bool FINE>
__device__ __forceinline__ Gate gate_of(float g)
{
    if (FORM == GATESCAN_DECAY)
        return Gate{g, 1.f - g};
    if (FORM == GATESCAN_SIGMOID) {
        const float e = gate_exp<FINE>(-__builtin_fabsf(g)), d = 1.f + e;
        float r = __builtin_amdgcn_rcpf(d);
        if (FINE)
            r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
        const float small = e * r, large = 1.f - small;
        return g < 0.f ? Gate{small, large} : Gate{large, small};
    }
    const float p = gate_exp<FINE>(g);
    if (!FINE) {
        // 1 - e^g from its series near 0 (0.1^6 / 6! is below 2^-29).
        float s = __builtin_fmaf(g, 1.f / 120.f, 1.f / 24.f);
        s = __builtin_fmaf(s, g, 1.f / 6.f);
        s = __builtin_fmaf(s, g, 0.5f);
        s = __builtin_fmaf(s * g, g, g);
        return __builtin_fabsf(g) < 0.1f ? Gate{1.f + s, -s} : Gate{p, 1.f - p};
    }
    // Eight terms: 0.35^8 / 9! is below 2^-30.
    float s = __builtin_fmaf(g, 1.f / 40320.f, 1.f / 5040.f);
    s = __builtin_fmaf(s, g, 1.f / 720.f);
    s = __builtin_fmaf(s, g, 1.f / 120.f);
    s = __builtin_fmaf(s, g, 1.f / 24.f);
    s = __builtin_fmaf(s, g, 1.f / 6.f);
    s = __builtin_fmaf(s, g, 0.5f);
    s = __builtin_fmaf(s * g, g, g);
    return __builtin_fabsf(g) < 0.35f ? Gate{1.f + s, -s} : Gate{p, 1.f - p};
}

// The product of two products of gates.  One that has left the floats counts
// as the smallest of them, not as zero, unless a factor is zero: an infinite
// state stays infinite.
template <bool SIGNED>
__device__ __forceinline__ float kept_product(float a, float b)
{
    const float least = __builtin_fminf(__builtin_fminf(__builtin_fabsf(a), __builtin_fabsf(b)), 1.40129846e-45f);
    const float p = a * b, q = __builtin_fmaxf(__builtin_fabsf(p), least);
    return SIGNED ? __builtin_copysignf(q, p) : q;
}

template <class T, int FORM, bool BLEND, bool GRAD>
struct GateTile {
    typedef Unpack<T> U;
    static constexpr int V = kPiece<T>, C = kGateLanes * V, G = kGateGroups;
    static constexpr int R = gate_rows(sizeof(T) == 4 ? LIBSCAN_F32 : LIBSCAN_BF16, GRAD), TT = G * R;
    static constexpr bool FINE = sizeof(T) == 4;
    // Of any tile: a thread has four channels of some tokens.
    static constexpr int kParts = kGateThreads * 4 / C, kTokens = TT / kParts;
    static_assert(C <= 64 && kParts <= G && G <= 32 && G % 8 == 0 && kParts % 8 == 0, "one wave chains the groups");

    // Pieces that a thread keeps of a tile.
    static constexpr int kStash = GRAD ? 3 * R + (BLEND ? R : 1) : R * V / 2;

    struct Shared {
        // Each group's pair, then that of all groups before it in the tile.
        alignas(16) float a[G][C];
        alignas(16) float h[G][C];
        alignas(16) float carry[C];                  // what enters the tile
        piece_t kept[kStash][64];
        uint32_t reset[kParts];                      // whether the sweep starts anew in a part
        uint32_t k, line, seq;
        int32_t first[TT], last[TT];                 // the sequence that starts / ends at a token, or -1
    };

    // The call's arguments, in the kernel's own memory.
    typedef const __attribute__((address_space(4))) GateArgs Args;

    Args *p;
    Shared &s;
    uint64_t end;                // tokens [0, end) are in sequences
    uint32_t k, line;            // the tile: its place in its line
    int64_t low;                 // its lowest token (below 0 where a gradient's last tile reaches past them)

    __device__ __forceinline__ GateTile(Shared &shared, uint32_t k_, uint32_t line_) : s(shared), k(k_), line(line_)
    {
        p = (Args *)__builtin_amdgcn_kernarg_segment_ptr();
        end = p->tokens;
        if (p->ends) {
            const uint64_t last = p->ends[p->seqs - 1];
            end = last < end ? last : end;
        }
        low = GRAD ? (int64_t)p->tokens - (int64_t)(k + 1) * TT : (int64_t)k * TT;
    }

    // The token at one of the tile's places in the sweep's order.
    __device__ __forceinline__ int64_t token(int at) const { return GRAD ? low + (TT - 1 - at) : low + at; }

    // Where the line's channels start.
    __device__ __forceinline__ uint64_t column() const { return (uint64_t)(line % p->blocks) * C; }

    template <class Rows>
    __device__ __forceinline__ const T *row(const Rows &from, int64_t t) const
    {
        return static_cast<const T *>(from.p) + (int64_t)(line / p->blocks) * from.seq + t * from.tok +
               (int64_t)column();
    }
    __device__ __forceinline__ T *out_row(int which, int64_t t) const
    {
        return static_cast<T *>(p->out[which]) + (int64_t)(line / p->blocks) * p->out_seq[which] +
               t * p->out_tok[which] + (int64_t)column();
    }

    // Where sequences start and end among the tile's tokens, and whether any
    // does; the states of empty ones are passed through by the tiles at whose
    // tokens they lie.
    __device__ __forceinline__ bool mark()
    {
        const int tid = threadIdx.x;
        for (int i = tid; i < TT; i += kGateThreads)
            s.first[i] = s.last[i] = -1;
        if (tid < 64) {
            // Sequences that start at `low` or later, and the one before them.
            const uint32_t from = low > 0 ? first_above(p->ends, p->seqs, (uint64_t)low - 1) : 0;
            if (tid == 0)
                s.seq = from;
        }
        __syncthreads();
        const bool top = GRAD ? k == 0 : k == p->tiles - 1;      // what lies past the rows is the last tile's
        for (uint32_t q = s.seq + tid;; q += kGateThreads) {
            bool more = q < p->seqs;
            uint64_t first = 0, len = 0;
            if (more) {
                run_of(p->ends, p->tokens, q, &first, &len);
                more = top || (int64_t)first < low + TT;
            }
            if (more && len) {
                if ((int64_t)first >= low && (int64_t)first < low + TT)
                    s.first[first - low] = (int32_t)q;
                const int64_t l = (int64_t)(first + len) - 1;
                if (l >= low && l < low + TT)
                    s.last[l - low] = (int32_t)q;
            }
            if (p->state_out) {
                const int lane = tid % 64;
                const float *const from = GRAD ? p->last : p->first;
                uint64_t empty = __ballot(more && len == 0 && (int64_t)first >= low);
                while (empty) {
                    const uint32_t which = q - lane + (uint32_t)__builtin_ctzll(empty);
                    empty &= empty - 1;
                    const uint64_t c = column() + lane;
                    if (lane < C && c < p->width)
                        p->state_out[which * p->width + c] = from ? from[which * p->width + c] : 0.f;
                }
            }
            if (__syncthreads_count(more) < kGateThreads)
                break;
        }
        bool any = false;
        for (int i = tid; i < TT; i += kGateThreads)
            any |= s.first[i] >= 0 || s.last[i] >= 0;
        return __syncthreads_or(any) != 0;
    }

    // From dh of a token, h before it and its x: the gradients, and what goes on.
    __device__ __forceinline__ static float grad_of(const Gate &w, float dh, float before, float x, float *dg, float *dx)
    {
        *dx = BLEND ? dh * w.rest : dh;
        const float da = dh * (BLEND ? before - x : before);
        *dg = FORM == GATESCAN_DECAY ? da : FORM == GATESCAN_LOG ? da * w.a : da * (w.a * w.rest);
        return w.a * dh;
    }

    // ---- Whole tiles: no sequence starts or ends in them (but for equal    ----
    // ---- sequences' own ends, whose states the carry takes in), and every ----
    // ---- lane has all of its channels or none.                            ----

    // The same for all threads.
    __device__ __forceinline__ bool whole() const
    {
        // (A packed batch's first token starts a sequence, so that low > 0 there.)
        return low >= 0 && low + TT <= (int64_t)end && p->width % V == 0;
    }

    struct Pieces {
        piece_t g[R], d[R];                              // gate; x, or dout in the gradient
        piece_t h[GRAD ? R : 1], x[GRAD && BLEND ? R : 1];
    };
    template <class Rows>
    __device__ __forceinline__ void load_rows(const Rows &from, int lane8, int64_t first,
                                              piece_t (&to)[R]) const
    {
        const int64_t step = GRAD ? -from.tok : from.tok;
        const T *at = row(from, first) + lane8 * V;
#pragma unroll
        for (int r = 0; r < R; ++r, at += step)
            to[r] = load_piece_past(at);
    }

    // The forward pass's outputs a token earlier; in place of those before the
    // first token, which are its state, its own.
    template <class To>
    __device__ __forceinline__ void load_before(int lane8, int64_t first, To &to) const
    {
        const int64_t tok = p->h.tok;
        const T *at = row(p->h, first - 1) + lane8 * V;
#pragma unroll
        for (int r = 0; r < R; ++r, at -= tok)
            to[r] = load_piece_past(r == R - 1 && first == R - 1 ? at + tok : at);
    }

    // 1. of a tile, from its rows; the forward pass keeps a and b for 3.
    struct Kept {
        float a[GRAD ? 1 : R][V], b[GRAD ? 1 : R][V];
    };
    __device__ __forceinline__ void scan(const Pieces &x, Kept &keep, int lane8, int group) const
    {
        float A[V], H[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            A[e] = 1.f;
            H[e] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const Gate w = gate_of<FORM, FINE>(U::get(x.g[r], e));
                if (GRAD) {
                    H[e] = w.a * (H[e] + U::get(x.d[r], e));
                } else {
                    const float v = U::get(x.d[r], e);
                    keep.a[r][e] = w.a;
                    keep.b[r][e] = BLEND ? w.rest * v : v;
                    H[e] = __builtin_fmaf(w.a, H[e], keep.b[r][e]);
                }
                A[e] *= w.a;
            }
            // Row by row: moved behind all rows' gates, the sums need more registers
            // (sigmoid with blend of f32 128 with 13 spilled, not 87 and none).
#pragma unroll
            for (int e = 0; e < V; ++e)
                asm volatile("" : "+v"(A[e]), "+v"(H[e]));
            __builtin_amdgcn_sched_barrier(0);
        }
        bool gone = false;
#pragma unroll
        for (int e = 0; e < V; ++e)
            gone |= A[e] == 0.f;
        if (__any(gone)) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                A[e] = 1.f;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    A[e] = kept_product<FORM == GATESCAN_DECAY>(
                        A[e], GRAD ? gate_of<FORM, FINE>(U::get(x.g[r], e)).a : keep.a[GRAD ? 0 : r][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            s.a[group][lane8 * V + e] = A[e];
#pragma unroll
        for (int e = 0; e < V; ++e)
            s.h[group][lane8 * V + e] = H[e];
    }

    // 3. of a forward tile.
    __device__ __forceinline__ void finish(const Kept &keep, int lane8, int group, bool any) const
    {
        float H[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            H[e] = __builtin_fmaf(s.a[group][lane8 * V + e], s.carry[lane8 * V + e], s.h[group][lane8 * V + e]);
        T *to = out_row(0, low + group * R) + lane8 * V;
        if (any) {
            const int64_t step = p->out_tok[0];
#pragma unroll
            for (int r = 0; r < R; ++r, to += step) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    H[e] = __builtin_fmaf(keep.a[GRAD ? 0 : r][e], H[e], keep.b[GRAD ? 0 : r][e]);
                store_piece_past(to, U::pack(H));
                __builtin_amdgcn_sched_barrier(0);
            }
            if (p->state_out && !p->ends && group == G - 1 && low + TT == (int64_t)end)
                store_floats<V>(p->state_out + (line / p->blocks) * p->width + column() + lane8 * V, V, H);
        }
    }

    __device__ __forceinline__ void stream_whole()
    {
        const int lane8 = threadIdx.x % kGateLanes, group = threadIdx.x / kGateLanes;
        const int64_t first = token(group * R);
        const bool mine = column() + lane8 * V < p->width;
        Pieces x = {};
        if (mine) {
            load_rows(p->gate, lane8, first, x.g);
            load_rows(GRAD ? p->dout : p->x, lane8, first, x.d);
        }
        if constexpr (!GRAD) {
            Kept keep;
            scan(x, keep, lane8, group);
            __syncthreads();
            if (threadIdx.x < 64) {
                stash(keep);
                carry(G, 0);
                unstash(keep);
            }
            __syncthreads();
            finish(keep, lane8, group, mine);
        } else {
            if (mine) {
                if constexpr (BLEND)
                    load_rows(p->x, lane8, first, x.x);
                load_before(lane8, first, x.h);
            }
            Kept none;
            scan(x, none, lane8, group);
            __syncthreads();
            if (threadIdx.x < 64) {
                stash(x);
                carry(G, 0);
                unstash(x);
            }
            __syncthreads();
            float H[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                H[e] = __builtin_fmaf(s.a[group][lane8 * V + e], s.carry[lane8 * V + e],
                                      s.h[group][lane8 * V + e]);
            if (!mine)
                return;
            T *to = out_row(0, first) + lane8 * V, *to1 = out_row(1, first) + lane8 * V;
            const int64_t step = -p->out_tok[0], step1 = -p->out_tok[1];
            const uint64_t of = (line / p->blocks) * p->width + column() + lane8 * V;      // in states
#pragma unroll
            for (int r = 0; r < R; ++r, to += step, to1 += step1) {
                float dg[V], dx[V], before[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    before[e] = U::get(x.h[r], e);
                if (r == R - 1 && first == R - 1) {          // the first token of all
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        before[e] = 0.f;
                    if (p->first)
                        load_floats<V>(p->first + of, V, before);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const Gate w = gate_of<FORM, FINE>(U::get(x.g[r], e));
                    H[e] = grad_of(w, U::get(x.d[r], e) + H[e], before[e], BLEND ? U::get(x.x[BLEND ? r : 0], e) : 0.f,
                                   &dg[e], &dx[e]);
                }
                store_piece_past(to, U::pack(dg));
                store_piece_past(to1, U::pack(dx));
                __builtin_amdgcn_sched_barrier(0);
            }
            if (p->state_out && first == R - 1)
                store_floats<V>(p->state_out + of, V, H);
        }
    }

    // What the carrying wave's threads keep of their tile, in LDS while they
    // carry: kept in registers beside the carry, 14 to 126 of them spill.
    template <class X>
    __device__ __forceinline__ void stash(const X &x) const
    {
        static_assert(sizeof(X) <= sizeof(s.kept[0]) * kStash, "room for it");
        const piece_t *const from = reinterpret_cast<const piece_t *>(&x);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(X) / 16); ++i)
            s.kept[i][threadIdx.x % 64] = from[i];
    }
    template <class X>
    __device__ __forceinline__ void unstash(X &x) const
    {
        // By an address that says nothing of what was stored there.
        uint32_t lane = threadIdx.x % 64;
        asm volatile("" : "+v"(lane)::"memory");
        piece_t *const to = reinterpret_cast<piece_t *>(&x);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(X) / 16); ++i)
            to[i] = s.kept[i][lane];
    }

    // ---- Any tile ----

    // A thread's four channels of a line, from `c` on: at the width's end they
    // overlap the four before, whose values they have as well.  n: how many
    // there are, 4 unless the line has fewer, or 0.
    __device__ __forceinline__ void four_of(int *c, int *n) const
    {
        const uint64_t rest = p->width - column();
        const int left = rest < (uint64_t)C ? (int)rest : C;
        *c = threadIdx.x % (C / 4) * 4;
        *n = *c >= left ? 0 : left < 4 ? left : 4;
        if (*n == 4 && *c > left - 4)
            *c = left - 4;
    }

    // Rows of one tensor: the thread's first token's, and the way to its next.
    struct Walk {
        const T *at;
        int64_t step;
    };
    template <class Rows>
    __device__ __forceinline__ Walk walk(const Rows &from, int c, int64_t t) const
    {
        return Walk{row(from, t) + c, GRAD ? -from.tok : from.tok};
    }

    __device__ __forceinline__ void stream_any()
    {
        const int part = threadIdx.x / (C / 4);
        int c, n;
        four_of(&c, &n);
        const int64_t at = (int64_t)column() + c, width = (int64_t)p->width;
        // The thread's places and, by their distance from `low`, its tokens; of
        // the tile's, those in [lo, hi) are in sequences.
        const int lo = low < 0 ? (int)-low : 0, hi = (int64_t)end - low < TT ? (int)((int64_t)end - low) : TT;
        const auto index = [&](int u) { return GRAD ? TT - 1 - (part * kTokens + u) : part * kTokens + u; };
        const int64_t t0 = low + index(0);
        uint32_t in = 0, firsts = 0, lasts = 0;      // a bit a token
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const int i = index(u);
            const bool inside = n > 0 && i >= lo && i < hi;
            in |= (inside ? 1u : 0u) << u;
            if (p->ends) {
                firsts |= (inside && s.first[i] >= 0 ? 1u : 0u) << u;
                lasts |= (inside && s.last[i] >= 0 ? 1u : 0u) << u;
            }
        }
        if (!p->ends) {
            // Equal sequences: at their ends' distances alone.
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
                firsts |= ((int64_t)index(u) == -low ? 1u : 0u) << u;
                lasts |= ((int64_t)index(u) == (int64_t)end - 1 - low ? 1u : 0u) << u;
            }
            firsts &= in;
            lasts &= in;
        }
        const uint32_t resets = GRAD ? lasts : firsts;       // where the sweep starts anew
        // The states of the sequence that starts (ends) at a place.
        const auto place_of = [&](const int32_t *marks, int u) {
            return (p->ends ? (int64_t)marks[index(u)] : (int64_t)(line / p->blocks)) * width + at;
        };
        const auto state_at = [&](const float *of, const int32_t *marks, int u, float (&to)[4]) {
            const Four<float> v = of ? load_four(of + place_of(marks, u), n) : Four<float>{};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[e] = v.get(e);
        };
        const int32_t *const marks = GRAD ? s.last : s.first;
        const float *const entering = GRAD ? p->last : p->first;

        Four<T> g[kTokens], d[kTokens], x[GRAD && BLEND ? kTokens : 1], h[GRAD ? kTokens : 1];
        (void)x;
        (void)h;
        const auto load = [&](Walk from, auto &to, uint32_t which) {
#pragma unroll
            for (int u = 0; u < kTokens; ++u, from.at += from.step) {
                to[u] = Four<T>{};
                if (which >> u & 1)
                    to[u] = load_four(from.at, n);
            }
        };
        load(walk(p->gate, c, t0), g, in);
        load(walk(GRAD ? p->dout : p->x, c, t0), d, in);
        if constexpr (GRAD) {
            if constexpr (BLEND)
                load(walk(p->x, c, t0), x, in);
            load(walk(p->h, c, t0 - 1), h, in & ~firsts);
        }
        float A[4], H[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            A[e] = 1.f;
            H[e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (!(in >> u & 1))
                continue;
            if (resets >> u & 1)
                state_at(entering, marks, u, H);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Gate w = gate_of<FORM, FINE>(g[u].get(e));
                const float v = d[u].get(e);
                H[e] = GRAD ? w.a * (H[e] + v) : __builtin_fmaf(w.a, H[e], BLEND ? w.rest * v : v);
                A[e] = kept_product<FORM == GATESCAN_DECAY>(A[e], w.a);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                asm volatile("" : "+v"(A[e]), "+v"(H[e]));
        }
        if (n > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s.a[part][c + e] = A[e];
                s.h[part][c + e] = H[e];
            }
        }
        if (threadIdx.x % (C / 4) == 0)          // a line's first channel is one of the width's
            s.reset[part] = resets != 0;
        __syncthreads();
        const uint32_t anew = parts_anew();
        if (threadIdx.x < 64)
            carry(kParts, anew);
        __syncthreads();
        if (n == 0)
            return;
        const bool started = (anew & ((1u << part) - 1)) != 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            H[e] = started ? s.h[part][c + e] : __builtin_fmaf(s.a[part][c + e], s.carry[c + e], s.h[part][c + e]);
        T *to = out_row(0, t0) + c, *to1 = out_row(GRAD ? 1 : 0, t0) + c;
        const int64_t step = GRAD ? -p->out_tok[0] : p->out_tok[0], step1 = GRAD ? -p->out_tok[1] : 0;
#pragma unroll
        for (int u = 0; u < kTokens; ++u, to += step, to1 += step1) {
            float out[2][4] = {}, before[4];
            if (in >> u & 1) {
                if (resets >> u & 1)
                    state_at(entering, marks, u, H);
                if constexpr (GRAD) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        before[e] = h[u].get(e);
                    if (firsts >> u & 1)
                        state_at(p->first, s.first, u, before);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Gate w = gate_of<FORM, FINE>(g[u].get(e));
                    const float v = d[u].get(e);
                    if constexpr (GRAD)
                        H[e] = grad_of(w, v + H[e], before[e], BLEND ? x[BLEND ? u : 0].get(e) : 0.f, &out[0][e],
                                       &out[1][e]);
                    else
                        out[0][e] = H[e] = __builtin_fmaf(w.a, H[e], BLEND ? w.rest * v : v);
                }
                if (p->state_out && ((GRAD ? firsts : lasts) >> u & 1))
                    store_four(p->state_out + place_of(GRAD ? s.first : s.last, u), Four<float>::of(H), n);
            } else if (!past_end(index(u))) {
                continue;
            }
            store_four(to, Four<T>::of(out[0]), n);
            if constexpr (GRAD)
                store_four(to1, Four<T>::of(out[1]), n);
        }
    }
    // Whether a place's row is in no sequence and to be cleared.
    __device__ __forceinline__ bool past_end(int index) const
    {
        return p->clear && low + index >= (int64_t)end && low + index < (int64_t)p->tokens;
    }
    __device__ __forceinline__ uint32_t parts_anew() const
    {
        const uint32_t lane = threadIdx.x % 64;
        return (uint32_t)__ballot(lane < (uint32_t)kParts && s.reset[lane % kParts] != 0);
    }

    // A tile without tokens: none with any looks back to it.  Equal sequences of
    // no tokens pass their states through.
    __device__ __forceinline__ bool idle() const { return (low > 0 ? low : 0) >= (int64_t)end; }
    __device__ __forceinline__ void stream_idle() const
    {
        const int part = threadIdx.x / (C / 4);
        int c, n;
        four_of(&c, &n);
        if (n == 0)
            return;
        for (int i = part * kTokens; i < (part + 1) * kTokens; ++i) {
            if (past_end(i)) {
                store_four(out_row(0, low + i) + c, Four<T>{}, n);
                if (GRAD)
                    store_four(out_row(1, low + i) + c, Four<T>{}, n);
            }
        }
        if (!p->ends && p->state_out && part == 0) {
            const float *const from = GRAD ? p->last : p->first;
            const uint64_t of = (line / p->blocks) * p->width + column() + c;
            store_four(p->state_out + of, from ? load_four(from + of, n) : Four<float>{}, n);
        }
    }

    // 2., by one wave: the groups' pairs, the tile's carry.  anew: the groups in
    // which the sweep starts anew, a bit each.
    __device__ __forceinline__ void carry(int groups, uint32_t anew)
    {
        const uint32_t tag = p->tag;
        const int lane = threadIdx.x % 64;
        if (lane >= C)
            return;
        // The first tile of the line that has tokens starts a sequence, and
        // equal sequences' states enter there.
        const uint32_t k0 = GRAD && p->ends ? (uint32_t)((p->tokens - end) / TT) : 0;
        // The nearest tiles' words: asked for before the groups are chained, as
        // mostly a tile shortly before is through by then.
        Window<4> w;
        if (k > k0)
            w = window<4>(k0, lane);
        float in = 0.f, a = 1.f, h = 0.f;
        // (Eight at a time: one by one each read of LDS waits for the write before it.)
        for (int g0 = 0; g0 < groups; g0 += 8) {
            float ga[8], gh[8], ea[8], eh[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                ga[u] = s.a[g0 + u][lane];
                gh[u] = s.h[g0 + u][lane];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                ea[u] = a;
                eh[u] = h;
                h = __builtin_fmaf(ga[u], h, gh[u]);
                a = kept_product<FORM == GATESCAN_DECAY>(a, ga[u]);
            }
            if (anew >> g0 & 0xFF) {
                h = eh[0];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    eh[u] = h;
                    h = anew >> (g0 + u) & 1 ? gh[u] : __builtin_fmaf(ga[u], h, gh[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                s.a[g0 + u][lane] = ea[u];
                s.h[g0 + u][lane] = eh[u];
            }
        }
        uint64_t *const mine = p->desc + ((uint64_t)(k * p->chains + line) * 2) * C + lane;      // A; H is C on
        if (k > k0 && !nearest(w, tag, &in)) {
            if (anew != 0) {
                send(mine + C, tag | kStatusPrefix, h);
            } else {
                send(mine, tag | kStatusAgg, a);
                send(mine + C, tag | kStatusAgg, h);
            }
            for (;;) {
                if (p->far ? nearest(window<kGateWindow>(k0, lane), tag, &in)
                           : nearest(window<4>(k0, lane), tag, &in))
                    break;
            }
            if (anew == 0)
                send(mine + C, tag | kStatusPrefix, __builtin_fmaf(a, in, h));
        } else if (p->tiles > 1) {
            if (k <= k0)
                in = entering(lane);
            send(mine + C, tag | kStatusPrefix, anew != 0 ? h : __builtin_fmaf(a, in, h));
        } else {
            in = entering(lane);
        }
        s.carry[lane] = in;
    }

    // What enters the first tile of equal sequences.
    __device__ __forceinline__ float entering(int lane) const
    {
        const float *const state = GRAD ? p->last : p->first;
        const uint64_t c = column() + lane;
        return !p->ends && state && c < p->width ? state[(line / p->blocks) * p->width + c] : 0.f;
    }

    // The words of the N tiles before this one (of the line's first, where there are fewer).
    template <int N>
    struct Window {
        uint64_t a[N], h[N];
    };
    template <int N>
    __device__ __forceinline__ Window<N> window(uint32_t k0, int lane) const
    {
        Window<N> w;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t tile = k > k0 + u ? k - 1 - u : k0;
            w.h[u] = fetch(tile, 1, lane);
            w.a[u] = fetch(tile, 0, lane);
        }
        return w;
    }
    // What enters this tile, if the window has a chained value and all pairs after it.
    template <int N>
    __device__ __forceinline__ static bool nearest(const Window<N> &w, uint32_t tag, float *in)
    {
        uint32_t chained = 0, ready = 0;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t st = status(w.h[u], tag);
            chained |= (uint32_t)__all(st == kStatusPrefix) << u;
            ready |= (uint32_t)__all(st == kStatusPrefix || (st != 0 && status(w.a[u], tag) != 0)) << u;
        }
        const uint32_t first = chained & (0u - chained);
        if (chained == 0 || (~ready & (first - 1)) != 0)
            return false;
        float x = 0.f;
#pragma unroll
        for (int u = N - 1; u >= 0; --u)
            if (1u << u <= first)
                x = advance(x, w.a[u], w.h[u], tag);
        *in = x;
        return true;
    }

    __device__ __forceinline__ static void send(uint64_t *to, uint32_t head, float v)
    {
        __hip_atomic_store(to, (uint64_t)head << 32 | __builtin_bit_cast(uint32_t, v), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ uint64_t fetch(uint32_t tile, int half, int lane) const
    {
        return __hip_atomic_load(p->desc + ((uint64_t)(tile * p->chains + line) * 2 + half) * C + lane,
                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ static uint32_t status(uint64_t w, uint32_t tag)
    {
        const uint32_t hi = (uint32_t)(w >> 32);
        return (hi & ~3u) == tag ? hi & 3u : 0u;
    }
    __device__ __forceinline__ static float value(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)w); }
    // One tile further: its chained value, or its pair on top of what enters it.
    __device__ __forceinline__ static float advance(float in, uint64_t wa, uint64_t wh, uint32_t tag)
    {
        return status(wh, tag) == kStatusPrefix ? value(wh) : __builtin_fmaf(value(wa), in, value(wh));
    }

    __device__ __forceinline__ void run()
    {
        if (!(p->ends && mark()) && whole())
            stream_whole();
        else if (idle())
            stream_idle();
        else
            stream_any();
    }
};

// The next number of a counter {tag, count}, mostly by one atomic.  One with
// another launch's tag starts anew.
__device__ __forceinline__ uint32_t gate_draw(uint64_t *counter, uint32_t tag)
{
    uint64_t seen = __hip_atomic_fetch_add(counter, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((uint32_t)(seen >> 32) == tag)
        return (uint32_t)seen;
    ++seen;
    while ((uint32_t)(seen >> 32) != tag) {
        if (__hip_atomic_compare_exchange_strong(counter, &seen, (uint64_t)tag << 32 | 1, __ATOMIC_RELAXED,
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
            return 0;
    }
    return (uint32_t)__hip_atomic_fetch_add(counter, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <class T, int FORM, bool BLEND, bool GRAD>
__global__ __launch_bounds__(kGateThreads, 4) void gatescan_kernel(GateArgs p)
{
    typedef GateTile<T, FORM, BLEND, GRAD> Tile;
    __shared__ typename Tile::Shared s;
    uint32_t k = 0, line = blockIdx.x;               // lines of one tile wait for nothing
    if (p.tiles > 1) {
        if (threadIdx.x == 0) {
            // There are as many tiles as workgroups, so one of the counters has one.
            // (Workgroups go to the dies in turn, and so a die has a counter's lines.)
            uint32_t set = blockIdx.x % kGateSets;
            for (;; set = (set + 1) % kGateSets) {
                const uint32_t from = gate_set(p.chains, set), many = gate_set(p.chains, set + 1) - from;
                if (many == 0)
                    continue;
                const uint32_t n = gate_draw(p.counters + set * kGateCounterStride, p.tag);
                if (n < many * p.tiles) {
                    s.k = n / many;
                    s.line = from + n % many;
                    break;
                }
            }
        }
        __syncthreads();
        k = __builtin_amdgcn_readfirstlane(s.k);
        line = __builtin_amdgcn_readfirstlane(s.line);
    }
    Tile(s, k, line).run();
}

template <class T, bool GRAD>
hipError_t launch_gate_tiles(const GateArgs &a, hipStream_t stream)
{
#define LIBSCAN_GATE(FORM)                                                                        \
    if (a.form == FORM) {                                                                         \
        if (a.blend)                                                                              \
            gatescan_kernel<T, FORM, true, GRAD><<<a.chains * a.tiles, kGateThreads, 0, stream>>>(a);        \
        else                                                                                      \
            gatescan_kernel<T, FORM, false, GRAD><<<a.chains * a.tiles, kGateThreads, 0, stream>>>(a);       \
    }
    LIBSCAN_GATE(GATESCAN_DECAY)
    LIBSCAN_GATE(GATESCAN_LOG)
    LIBSCAN_GATE(GATESCAN_SIGMOID)
#undef LIBSCAN_GATE
    return hipGetLastError();
}

}  // namespace libscan
