// linattn_kernels.hip -- linear attention with a decay for each head: the
// sweep in 32-bit matrix products (every type), the scan of segment states,
// and the sum of shared heads' gradients.  linattn.hpp has the mathematics.
//
// The sweep.  A workgroup of D / 32 waves (D = 64 or 128) has one segment of
// one sequence and head and D columns of the outputs; each wave owns 32
// columns n and keeps its m x 32 part of the state Z in accumulators for the
// whole segment.  It takes 32 tokens at a time: with A, B, C the chunk's rows
//
//   out = (p^(i+1-shift)) A Z + ((A B^T) o mask p^(i-j)) C
//   Z  <- p^32 Z + B^T (p^(31+shift-j) C)
//
// so the state is read and written once a segment and every row of a, b and
// c is read once.  All products are v_mfma_f32_32x32x2_f32.  An accumulator
// register r holds row 8 (r / 4) + 4 (lane / 32) + r % 4 of column lane % 32;
// taking the contraction's tokens (or m) in that same order makes Z's
// accumulators the second operand of A Z as they stand.
//
// The chunk is causal by selection, not by multiplication: a masked pair is
// zero whatever the product was.  A value that is not finite would still
// reach earlier rows as 0 * inf, so a chunk with one in C is taken again one
// token at a time.
#include "linattn.hpp"

#include "../../include/libscan.h"

namespace libscan {

namespace {

template <class T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }

template <class T>
struct Vec16 {
    static constexpr int kN = 16 / (int)sizeof(T);
    typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
};

__device__ __forceinline__ bool not_finite(float x)
{
    return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u;
}

// Rows [0, cnt) of a chunk into LDS as floats, zeros in the rest of its
// ROWS x WP.  Returns whether the thread saw a value that is not finite.
template <class T, bool VEC, int ROWS, int WP, int LD, int THREADS>
__device__ __forceinline__ bool load_rows(const T *base, int64_t step, int cnt, int width,
                                          float (*dst)[LD])
{
    bool bad = false;
    if (VEC) {
        constexpr int V = Vec16<T>::kN, PER = WP / V;
        for (int i = threadIdx.x; i < ROWS * PER; i += THREADS) {
            const int r = i / PER, c = i % PER * V;
            float x[V];
            if (r < cnt && c < width) {
                const auto t = *reinterpret_cast<const typename Vec16<T>::type *>(base + r * step + c);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] = to_f32(t[e]);
                    bad |= not_finite(x[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<f32x4 *>(&dst[r][c + e]) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
        }
    } else {
        for (int i = threadIdx.x; i < ROWS * WP; i += THREADS) {
            const int r = i / WP, c = i % WP;
            float x = 0.f;
            if (r < cnt && c < width)
                x = to_f32(base[r * step + c]);
            bad |= not_finite(x);
            dst[r][c] = x;
        }
    }
    return bad;
}

// STATES: only the segment's own contribution to the state, into set.seg.
template <class T, int D, bool VEC, bool STATES>
__global__ __launch_bounds__(D * 2) void sweep_f32_kernel(const SweepSet set)
{
    constexpr int NW = D / 32, THREADS = D * 2, C = 32, LD = D + 4, MT = D / 32;
    __shared__ __align__(16) float s_a[STATES ? 1 : C][LD];
    __shared__ __align__(16) float s_b[C][LD];
    __shared__ __align__(16) float s_c[C][LD];
    __shared__ __align__(16) float s_p[STATES ? 1 : NW][C][C + 4];
    __shared__ float s_pw[C + 2], s_pl[C + 2];        // powers of the decay: hi, lo

    const Sweep &sw = set.s[blockIdx.z];
    const uint32_t head = blockIdx.y;
    Place pl;
    if (!place_of(set, blockIdx.x, &pl))
        return;
    if (STATES && pl.last)
        return;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    const float g = set.log_decay[head];
    if (threadIdx.x < C + 2) {
        const Power p = decay_power(g, (double)threadIdx.x);
        s_pw[threadIdx.x] = p.hi;
        s_pl[threadIdx.x] = p.lo;
    }

    const int m = sw.m, n = sw.n, col = wave * 32 + l32;
    const uint64_t sh = (uint64_t)pl.seq * set.heads + head;
    float *seg = set.seg + (((uint64_t)blockIdx.z * set.items + blockIdx.x) * set.heads + head) *
                               (D * D) + wave * (MT * 16 * 64) + lane;
    f32x16 z[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            z[mt][r] = 0.f;
    if (!STATES) {
        if (pl.lo)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    z[mt][r] = seg[(mt * 16 + r) * 64];
        if (sw.state_in && col < n) {
            const Power w = decay_power(g, (double)pl.lo);
            const float *st = sw.state_in + sh * ((uint64_t)m * n) + col * sw.state_n;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = mt * 32 + 8 * (r / 4) + 4 * half + r % 4;
                    if (row < m)
                        z[mt][r] += decayed(st[row * sw.state_m], w);
                }
        }
    }

    uint64_t single = 0;           // tokens below this one are taken one at a time
    for (uint64_t at = pl.lo; at < pl.hi;) {
        const uint64_t left = pl.hi - at;
        int cnt = at < single ? 1 : (int)(left < C ? left : C);
        for (;;) {
            const int64_t dir = sw.rev ? -1 : 1;
            const uint64_t tok = pl.first + (sw.rev ? pl.len - 1 - at : at);
            if (!STATES)
                load_rows<T, VEC, C, D, LD, THREADS>(row_ptr<T>(sw.a, pl.seq, tok, head),
                                                     dir * sw.a.tok, cnt, m, s_a);
            load_rows<T, VEC, C, D, LD, THREADS>(row_ptr<T>(sw.b, pl.seq, tok, head),
                                                 dir * sw.b.tok, cnt, m, s_b);
            const bool bad = load_rows<T, VEC, C, D, LD, THREADS>(
                row_ptr<T>(sw.c, pl.seq, tok, head), dir * sw.c.tok, cnt, n, s_c);
            if (!__syncthreads_or(!STATES && bad && cnt > 1))
                break;
            single = at + cnt;
            cnt = 1;
        }

        if (!STATES) {
            // Pairs: wave w contracts its 32 of the m columns for all of them.
            f32x16 acc;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[r] = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int at4 = wave * 32 + 8 * q + 4 * half;
                const f32x4 bv = *reinterpret_cast<const f32x4 *>(&s_b[l32][at4]);
                const f32x4 av = *reinterpret_cast<const f32x4 *>(&s_a[l32][at4]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bv[e], av[e], acc, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4 *>(&s_p[wave][l32][8 * q + 4 * half]) =
                    f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};

            // What the rows read of the state.
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[r] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 av =
                        *reinterpret_cast<const f32x4 *>(&s_a[l32][mt * 32 + 8 * q + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(av[e], z[mt][4 * q + e], acc, 0, 0, 0);
                }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[r] *= s_pw[8 * (r / 4) + 4 * half + r % 4 + 1 - sw.shift];
            __syncthreads();

            // What they read of the chunk's own tokens.
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j0 = 8 * q + 4 * half;
                f32x4 pv = *reinterpret_cast<const f32x4 *>(&s_p[0][l32][j0]);
#pragma unroll
                for (int w = 1; w < NW; ++w)
                    pv += *reinterpret_cast<const f32x4 *>(&s_p[w][l32][j0]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + e;
                    const float p = j <= l32 ? pv[e] * (sw.pair_scale * s_pw[l32 - j]) : 0.f;
                    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(p, s_c[j][col], acc, 0, 0, 0);
                }
            }
            if (col < n) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int i = 8 * (r / 4) + 4 * half + r % 4;
                    if (i < cnt) {
                        const uint64_t t = pl.first + (sw.rev ? pl.len - 1 - at - i : at + i);
                        const int64_t o = (int64_t)pl.seq * sw.out_seq + (int64_t)t * sw.out_tok +
                                          (int64_t)head * sw.out_head + col;
                        const float x = acc[r] * sw.out_scale;
                        if (sw.out_f32)
                            static_cast<float *>(sw.out)[o] = x;
                        else
                            static_cast<T *>(sw.out)[o] = (T)x;
                    }
                }
            }
        }

        // The state past this chunk.
        const Power whole = {s_pw[cnt], s_pl[cnt]};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                z[mt][r] = decayed(z[mt][r], whole);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 8 * q + 4 * half + e;
                const float w = j < cnt ? sw.pair_scale * s_pw[cnt - 1 + sw.shift - j] : 0.f;
                const float cv = w * s_c[j][col];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    z[mt] = __builtin_amdgcn_mfma_f32_32x32x2f32(s_b[j][mt * 32 + l32], cv, z[mt], 0, 0, 0);
            }
        at += cnt;
        __syncthreads();
    }

    if (STATES) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                seg[(mt * 16 + r) * 64] = z[mt][r];
    } else if (sw.state_out && pl.last && col < n) {
        float *st = sw.state_out + sh * ((uint64_t)m * n) + col * sw.state_n;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = mt * 32 + 8 * (r / 4) + 4 * half + r % 4;
                if (row < m)
                    st[row * sw.state_m] = z[mt][r];
            }
    }
}

// The exclusive scan of a sequence's segment states, (l, S) o (r, U) =
// (l r, r S + U), each thread four elements of the state: segment s is left
// with what its tokens read of the segments before it.
template <int D>
__global__ __launch_bounds__(256) void segment_scan_kernel(const SweepSet set)
{
    const uint32_t head = blockIdx.y;
    constexpr uint32_t PARTS = D * D / 1024;
    const uint32_t sweep = blockIdx.z, seq = blockIdx.x / PARTS;
    const uint64_t L = set.seg_len;
    uint64_t first = 0, len = set.tokens, item = 0;
    if (!set.ends) {
        item = (uint64_t)seq * ((set.tokens + L - 1) / L);
    } else {
        run_of(set.ends, set.tokens, seq, &first, &len);
        if (len <= L)
            return;
        for (uint32_t i0 = 0; i0 < seq; i0 += 64) {
            const uint32_t i = i0 + (threadIdx.x & 63);
            uint32_t n = 0;
            if (i < seq) {
                uint64_t f, l;
                run_of(set.ends, set.tokens, i, &f, &l);
                n = l ? (uint32_t)((l + L - 1) / L) : 1u;
            }
            item += __shfl(wave_incl_u32(n), 63);
        }
    }
    const uint64_t segs = (len + L - 1) / L;
    if (item + segs > set.items)        // ends that no batch of this many tokens has
        return;
    const Power w = decay_power(set.log_decay[head], (double)L);
    f32x4 *p = reinterpret_cast<f32x4 *>(
                   set.seg + (((uint64_t)sweep * set.items + item) * set.heads + head) * (D * D)) +
               blockIdx.x % PARTS * 256 + threadIdx.x;
    const uint64_t step = (uint64_t)set.heads * (D * D) / 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    constexpr int AHEAD = 8;            // loads in flight ahead of the chain
    for (uint64_t s = 0; s < segs; s += AHEAD) {
        f32x4 own[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)      // the last segment left no sum
            own[i] = s + i + 1 < segs ? p[(s + i) * step] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (s + i < segs) {
                p[(s + i) * step] = sum;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = decayed(sum[e], w) + own[i][e];
            }
    }
}

// dst = the sum over each `share` consecutive heads of src, in order.
template <class T>
__global__ __launch_bounds__(256) void head_sum_kernel(const HeadSum h)
{
    const uint64_t per = (uint64_t)h.heads * h.width;
    const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= h.seqs * h.tokens * per)
        return;
    const uint64_t row = i / per, head = i % per / h.width;
    const int c = (int)(i % h.width);
    const float *src = h.src + (row * h.heads + head) * h.share * h.width + c;
    float x = 0.f;
    for (uint32_t k = 0; k < h.share; ++k)
        x += src[(uint64_t)k * h.width];
    T *dst = static_cast<T *>(const_cast<void *>(h.dst.p));
    dst[(int64_t)(row / h.tokens) * h.dst.seq + (int64_t)(row % h.tokens) * h.dst.tok +
        (int64_t)head * h.dst.head + c] = (T)x;
}

// Single tokens.  A workgroup has COLS = 4 LPR (or LPR) columns of one row's
// and head's state: LPR lanes cover a row of them, 256 / LPR rows at a time,
// so every load and store is 16 bytes a lane and the whole slab is in flight
// at once.  Each thread adds up its rows' part of the output; the row groups
// are added in LDS in a fixed order.
template <class T, int V, int LPR>
__global__ __launch_bounds__(256) void step_kernel(const StepArgs a)
{
    constexpr int COLS = LPR * V, GROUPS = 256 / LPR;
    __shared__ float s_q[kLinattnWidth], s_k[kLinattnWidth];
    __shared__ float s_o[GROUPS][COLS];
    const uint32_t row = blockIdx.x, head = blockIdx.y;
    const int c0 = blockIdx.z * COLS, lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int col = c0 + lane * V;
    T *out = static_cast<T *>(const_cast<void *>(a.out.p)) + (int64_t)row * a.out.seq +
             (int64_t)head * a.out.head;
    const int64_t slot = a.slots ? (int64_t)a.slots[row] : (int64_t)row;
    if (slot < 0 || (uint64_t)slot >= a.pool) {       // an idle row
        if (threadIdx.x < COLS && c0 + (int)threadIdx.x < a.dv)
            out[c0 + threadIdx.x] = (T)0.f;
        return;
    }
    const T *q = row_ptr<T>(a.q, row, 0, head), *k = row_ptr<T>(a.k, row, 0, head);
    const T *v = row_ptr<T>(a.v, row, 0, head);
    if ((int)threadIdx.x < a.dk) {
        s_q[threadIdx.x] = to_f32(q[threadIdx.x]) * a.scale;
        s_k[threadIdx.x] = to_f32(k[threadIdx.x]);
    }
    const Power w = decay_power(a.log_decay[head], 1.0);
    const uint64_t base = ((uint64_t)slot * a.heads + head) * ((uint64_t)a.dk * a.dv) + col;
    const float *src = a.state + base;
    float *dst = a.state_out + base;
    float vv[V], o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        vv[e] = col + e < a.dv ? to_f32(v[col + e]) : 0.f;
        o[e] = 0.f;
    }
    __syncthreads();
    if (col < a.dv) {
#pragma unroll 4
        for (int r = group; r < a.dk; r += GROUPS) {
            float x[V];
            if (V == 4)
                *reinterpret_cast<f32x4 *>(x) = *reinterpret_cast<const f32x4 *>(src + (int64_t)r * a.dv);
            else
                x[0] = src[(int64_t)r * a.dv];
            const float kr = s_k[r], qr = s_q[r];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[e] = decayed(x[e], w) + kr * vv[e];
                o[e] += qr * x[e];
            }
            if (V == 4)
                *reinterpret_cast<f32x4 *>(dst + (int64_t)r * a.dv) = *reinterpret_cast<f32x4 *>(x);
            else
                dst[(int64_t)r * a.dv] = x[0];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        s_o[group][lane * V + e] = o[e];
    __syncthreads();
    if (threadIdx.x < COLS && c0 + (int)threadIdx.x < a.dv) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
            x += s_o[i][threadIdx.x];
        out[c0 + threadIdx.x] = (T)x;
    }
}

template <class T, int D>
void run_sweeps(const SweepSet &set, hipStream_t stream)
{
    const dim3 grid(set.items, set.heads, (unsigned)set.count);
    if (set.seg_len) {
        if (set.aligned)
            sweep_f32_kernel<T, D, true, true><<<grid, D * 2, 0, stream>>>(set);
        else
            sweep_f32_kernel<T, D, false, true><<<grid, D * 2, 0, stream>>>(set);
        launch_segment_scan(set, D, stream);
    }
    if (set.aligned)
        sweep_f32_kernel<T, D, true, false><<<grid, D * 2, 0, stream>>>(set);
    else
        sweep_f32_kernel<T, D, false, false><<<grid, D * 2, 0, stream>>>(set);
}

template <class T>
void run_step(const StepArgs &a, hipStream_t stream)
{
    const bool aligned = (((uintptr_t)a.state | (uintptr_t)a.state_out) & 15) == 0;
    const unsigned v = a.dv % 4 == 0 && aligned ? 4 : 1;
    const auto blocks = [&](int cols) { return (unsigned)((a.dv + cols - 1) / cols); };
    // Narrow slabs where whole ones would leave compute units idle.
    const bool narrow = (uint64_t)a.rows * a.heads < 512;
    if (v == 4) {
        if (narrow)
            step_kernel<T, 4, 8><<<dim3(a.rows, a.heads, blocks(32)), 256, 0, stream>>>(a);
        else
            step_kernel<T, 4, 32><<<dim3(a.rows, a.heads, blocks(128)), 256, 0, stream>>>(a);
    } else {
        step_kernel<T, 1, 32><<<dim3(a.rows, a.heads, blocks(32)), 256, 0, stream>>>(a);
    }
}

}  // namespace

size_t linattn_state_floats(int width) { return width <= 64 ? 64 * 64 : 128 * 128; }

uint64_t linattn_seg_len(uint64_t tokens, bool ragged, uint32_t seqs, uint32_t heads, int sweeps)
{
    // Equal shares of the tokens for 1024 workgroups, in whole chunks, but
    // not so short that the states outweigh the rows.
    const uint64_t rows = ragged ? tokens : tokens * seqs;
    uint64_t share = (rows * heads * (uint64_t)sweeps + 1023) / 1024;
    share = (share + 63) / 64 * 64;
    if (share < 256)
        share = 256;
    return tokens > share ? share : 0;
}

uint64_t linattn_items(uint64_t tokens, bool ragged, uint32_t seqs, uint64_t seg_len)
{
    if (!seg_len)
        return seqs;
    return ragged ? seqs + tokens / seg_len : seqs * ((tokens + seg_len - 1) / seg_len);
}

void launch_segment_scan(const SweepSet &set, int width, hipStream_t stream)
{
    const dim3 grid((unsigned)(width * width / 1024) * set.seqs, set.heads, (unsigned)set.count);
    if (width == 64)
        segment_scan_kernel<64><<<grid, 256, 0, stream>>>(set);
    else
        segment_scan_kernel<128><<<grid, 256, 0, stream>>>(set);
}

hipError_t launch_sweeps(const SweepSet &set, hipStream_t stream)
{
    int width = 0;
    for (int i = 0; i < set.count; ++i) {
        width = set.s[i].m > width ? set.s[i].m : width;
        width = set.s[i].n > width ? set.s[i].n : width;
    }
    width = width <= 64 ? 64 : 128;
    if (set.dtype != LIBSCAN_F32)
        launch_sweeps_split(set, width, stream);
    else if (width == 64)
        run_sweeps<float, 64>(set, stream);
    else
        run_sweeps<float, 128>(set, stream);
    return hipGetLastError();
}

hipError_t launch_head_sum(const HeadSum &h, hipStream_t stream)
{
    const uint64_t n = h.seqs * h.tokens * h.heads * (uint64_t)h.width;
    if (n == 0)
        return hipSuccess;
    const unsigned blocks = (unsigned)((n + 255) / 256);
    switch (h.dtype) {
    case LIBSCAN_F32: head_sum_kernel<float><<<blocks, 256, 0, stream>>>(h); break;
    case LIBSCAN_BF16: head_sum_kernel<__bf16><<<blocks, 256, 0, stream>>>(h); break;
    default: head_sum_kernel<_Float16><<<blocks, 256, 0, stream>>>(h); break;
    }
    return hipGetLastError();
}

hipError_t launch_linattn_step(const StepArgs &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: run_step<float>(a, stream); break;
    case LIBSCAN_BF16: run_step<__bf16>(a, stream); break;
    default: run_step<_Float16>(a, stream); break;
    }
    return hipGetLastError();
}

}  // namespace libscan
