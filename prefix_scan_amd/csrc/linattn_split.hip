// linattn_split.hip -- the sweep of linattn.hpp for bf16 and f16 rows, in
// bf16 matrix products (v_mfma_f32_32x32x16_bf16) with 32-bit sums.
//
// A workgroup of D / 32 waves (D = 64 or 128) has one segment of one sequence
// and head; wave w owns 32 columns n and keeps its m x 32 part of the state Z
// in 32-bit accumulators for the whole segment.  It takes C = 64 tokens at a
// time; with A, B, C the chunk's rows
//
//   out^T = Z^T A^T (p^(i+1-shift)) + C^T ((A B^T) o mask p^(i-j))^T
//   Z    <- p^64 Z + B^T (p^(63+shift-j) C)
//
// so the state is read and written once a segment and every row of a, b and
// c is read once.  The rows of chunk t + 1 are on their way in registers
// while chunk t is computed from LDS.
//
// How exact.  A bf16 operand is one bf16 part, an f16 one the exact sum of
// two (so that neither scores nor states can overflow f16).  The products
// that feed the 16-bit outputs round their computed operand (scores, state)
// to as many parts: one rounding of 2^-8 for bf16, of 2^-16 for f16.  The
// state itself is a 32-bit sum of p^.. C split into three parts, exact to
// 24 bits, times the exact B; where no state is asked for, and it is only
// read through a rounding to the rows' own precision, two parts (2^-16) do.
//
// Layouts.  An operand lane holds 8 consecutive k of row lane % 32, k from
// 8 (lane / 32); an accumulator register r holds row 8 (r / 4) + 4 (lane /
// 32) + r % 4 of column lane % 32.  C and B are read down their columns by
// transposing LDS loads; for B these fetch the middle two of every four
// groups of 4 columns the other way round, which makes the accumulators of Z
// hold 8 consecutive m a lane: the second operand of Z^T A^T as they stand.
#include "linattn.hpp"

#include "../../include/libscan.h"

namespace libscan {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int C = 64;                   // tokens of a chunk

template <class T>
struct In;
template <>
struct In<__bf16> {
    static constexpr int kParts = 1;
    static constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
};
template <>
struct In<_Float16> {
    static constexpr int kParts = 2;
    static constexpr uint32_t kExp = 0x7C007C00u, kOne = 0x04000400u;
};

__device__ __forceinline__ float low16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats' upper halves in one word: both cut to bf16.
__device__ __forceinline__ uint32_t cut_pair(float a, float b)
{
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

__device__ __forceinline__ uint32_t round_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

__device__ __forceinline__ float above(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }

// What is left of x past its part h, and nothing where x is not finite.
__device__ __forceinline__ float rest(float x, float h)
{
    return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? 0.f : x - h;
}

// Eight floats in P parts, each rounded to nearest from what the ones before
// it left.
template <int P, bool FINITE>
__device__ __forceinline__ void parts_of(const float *x, u32x4 *out)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (p + 1 == P) {
                out[p][e] = round_pair(a, b);
            } else if (FINITE) {
                out[p][e] = cut_pair(a, b);
                a -= above(a);
                b -= above(b);
            } else {
                const uint32_t w = round_pair(a, b);
                out[p][e] = w;
                a = rest(a, low16(w));
                b = rest(b, high16(w));
            }
        }
    }
}

// This thread's 16 bytes of rows [0, cnt) of a chunk, zeros past them.
template <class T, bool VEC, int W, int THREADS, int N>
__device__ __forceinline__ void fetch(u32x4 (&r)[N], const T *base, int64_t step, int cnt, int width)
{
    constexpr int PER = W / 8, RS = THREADS / PER;
    static_assert(N == C / RS, "a chunk of C rows");
    const int row0 = threadIdx.x / PER, col = threadIdx.x % PER * 8;
    const T *p = base + row0 * step + col;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        r[k] = u32x4{0, 0, 0, 0};
        if (row0 + k * RS < cnt && col < width) {
            if (VEC) {
                r[k] = *reinterpret_cast<const u32x4 *>(p);
            } else {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < width)
                        r[k][e / 2] |= (uint32_t)h[e] << (16 * (e & 1));
            }
        }
        p += RS * step;
    }
}

// The fetched rows into LDS, split into parts.
template <class T, int W, int THREADS, int N, int LD>
__device__ __forceinline__ void stage(const u32x4 (&r)[N], __bf16 (*dst)[C][LD])
{
    constexpr int PER = W / 8, RS = THREADS / PER;
    const int row0 = threadIdx.x / PER, col = threadIdx.x % PER * 8;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (In<T>::kParts == 1) {
            *reinterpret_cast<u32x4 *>(&dst[0][row0 + k * RS][col]) = r[k];
        } else {
            typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
            const f16x8 h = __builtin_bit_cast(f16x8, r[k]);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = (float)h[e];
            u32x4 p[In<T>::kParts];
            parts_of<In<T>::kParts, false>(x, p);
#pragma unroll
            for (int i = 0; i < In<T>::kParts; ++i)
                *reinterpret_cast<u32x4 *>(&dst[i][row0 + k * RS][col]) = p[i];
        }
    }
}

template <class T, int N>
__device__ __forceinline__ bool any_not_finite(const u32x4 (&r)[N])
{
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bad |= ((r[k][e] & In<T>::kExp) + In<T>::kOne) & 0x80008000u;
    return bad != 0;
}

// Eight rows down 16 columns: p is this lane's place in the first four.
template <int LD>
__device__ __forceinline__ u32x4 column_frag(const __bf16 *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
    const u32x2 b = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * LD)));
    return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int D, int IP, bool STATES>
struct Lds {
    static constexpr int LD = D + 16;      // 16 B apart in bank: rows and columns both read clean
    static constexpr int LP = C + 8;
    union {
        __bf16 a[STATES ? 1 : IP][STATES ? 1 : C][LD];
        __bf16 o[STATES ? 1 : D / 32][STATES ? 1 : C][32];      // a wave's outputs, once a is read
    };
    __bf16 b[IP][C][LD];
    __bf16 c[IP][C][LD];
    __bf16 p[STATES ? 1 : IP][STATES ? 1 : C][LP];
    float pw[C + 8], pl[C + 8];            // powers of the decay: hi, lo
    float pair[C + 32];                    // pair_scale p^d at 31 + d
    float wt[C];                           // pair_scale p^(cnt-1+shift-j)
    int bad[2];
};

// STATES: only the segment's own contribution to the state, into set.seg.
// WP: parts of the decayed rows that the state sums.
template <class T, int D, bool VEC, int WP, bool STATES>
__global__ __launch_bounds__(D * 2, In<T>::kParts == 1 ? 2 : 1) void sweep_split_kernel(const SweepSet set)
{
    constexpr int NW = D / 32, THREADS = D * 2, MT = D / 32, IP = In<T>::kParts;
    constexpr int N = C * D / 8 / THREADS;
    typedef Lds<D, IP, STATES> S;
    __shared__ __align__(16) S s;

    const Sweep &sw = set.s[blockIdx.z];
    const uint32_t head = blockIdx.y;
    Place pl;
    if (!place_of(set, blockIdx.x, &pl))
        return;
    if (STATES && pl.last)
        return;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    const float g = set.log_decay[head];
    for (int i = threadIdx.x; i < C + 2; i += THREADS) {
        const Power p = decay_power(g, (double)i);
        s.pw[i] = p.hi;
        s.pl[i] = p.lo;
    }
    if (threadIdx.x < C + 31) {
        const int d = (int)threadIdx.x - 31;
        s.pair[threadIdx.x] = d >= 0 ? sw.pair_scale * decay_power(g, (double)d).hi : 0.f;
    }
    if (threadIdx.x < 2)
        s.bad[threadIdx.x] = 0;

    const int m = sw.m, n = sw.n, col = wave * 32 + l32;
    const uint64_t sh = (uint64_t)pl.seq * set.heads + head;
    float *seg = set.seg + (((uint64_t)blockIdx.z * set.items + blockIdx.x) * set.heads + head) *
                               (D * D) + wave * (MT * 16 * 64) + lane;
    // z[mt][r]: row 32 mt + 16 (r / 8) + 8 half + r % 8 of column col.
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
                    const int row = mt * 32 + 16 * (r / 8) + 8 * half + r % 8;
                    if (row < m)
                        z[mt][r] += decayed(st[row * sw.state_m], w);
                }
        }
    }

    const int64_t dir = sw.rev ? -1 : 1;
    const T *pa = row_ptr<T>(sw.a, pl.seq, 0, head), *pb = row_ptr<T>(sw.b, pl.seq, 0, head),
            *pc = row_ptr<T>(sw.c, pl.seq, 0, head);
    u32x4 ra[STATES ? 1 : N], rb[N], rc[N];
    const auto fetch_chunk = [&](uint64_t at, int cnt) {
        const int64_t tok = (int64_t)(pl.first + (sw.rev ? pl.len - 1 - at : at));
        if constexpr (!STATES)
            fetch<T, VEC, D, THREADS>(ra, pa + tok * sw.a.tok, dir * sw.a.tok, cnt, m);
        fetch<T, VEC, D, THREADS>(rb, pb + tok * sw.b.tok, dir * sw.b.tok, cnt, m);
        fetch<T, VEC, D, THREADS>(rc, pc + tok * sw.c.tok, dir * sw.c.tok, cnt, n);
    };

    // The scores' tile of this wave (rows ti, columns tj of the 2 x 2; the
    // fourth is all masked).  With two waves the first has both on the diagonal.
    const int ti = NW == 4 ? (wave != 0) : wave, tj = NW == 4 ? wave == 2 : 0;
    // Places of this lane in column reads: row (of 16) and column.
    const int trow = 8 * half + (lane & 15) / 4, tcol = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const int tswap = 16 * ((lane >> 4) & 1) + 4 * ((lane & 3) == 1 ? 2 : (lane & 3) == 2 ? 1 : lane & 3);

    uint64_t at = pl.lo, single = 0;   // tokens below `single` are taken one at a time
    int cnt = pl.hi - at < C ? (int)(pl.hi - at) : C, cnt_wt = -1, turn = 0;
    fetch_chunk(at, cnt);
    while (at < pl.hi) {
        __syncthreads();
        if constexpr (!STATES)
            stage<T, D, THREADS>(ra, s.a);
        stage<T, D, THREADS>(rb, s.b);
        stage<T, D, THREADS>(rc, s.c);
        if (__any(any_not_finite<T>(rc)) && lane == 0)
            s.bad[turn] = 1;
        if (cnt != cnt_wt) {
            if (threadIdx.x < C) {
                const int j = threadIdx.x;
                s.wt[j] = j < cnt ? sw.pair_scale * s.pw[cnt - 1 + sw.shift - j] : 0.f;
            }
            cnt_wt = cnt;
        }
        __syncthreads();
        const bool bad = s.bad[turn] != 0;
        turn ^= 1;
        if (threadIdx.x == 0)
            s.bad[turn] = 0;
        if (bad && cnt > 1) {          // again, one token at a time
            single = at + cnt;
            cnt = 1;
            fetch_chunk(at, cnt);
            continue;
        }
        const uint64_t next = at + cnt;
        const uint64_t left = pl.hi - next;
        const int next_cnt = left == 0 ? 0 : next < single ? 1 : (int)(left < C ? left : C);
        if (next_cnt)
            fetch_chunk(next, next_cnt);

        f32x16 o[2];
        if constexpr (!STATES) {
            // Scores, transposed: a lane has token i of its tile and four
            // consecutive j at a time.
            if (wave < 3) {
#pragma unroll
                for (int k = 0; k < (NW == 4 ? 1 : 2); ++k) {
                    if (k && wave)
                        break;
                    const int it = ti + k, jt = tj + k;
                    f32x16 acc;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        acc[r] = 0.f;
#pragma unroll
                    for (int q = 0; q < 2 * MT; ++q) {
                        u32x4 af[IP], bf[IP];
#pragma unroll
                        for (int p = 0; p < IP; ++p) {
                            af[p] = *reinterpret_cast<const u32x4 *>(&s.a[p][32 * it + l32][16 * q + 8 * half]);
                            bf[p] = *reinterpret_cast<const u32x4 *>(&s.b[p][32 * jt + l32][16 * q + 8 * half]);
                        }
#pragma unroll
                        for (int x = 0; x < IP; ++x)
#pragma unroll
                            for (int y = 0; x + y < IP; ++y)
                                acc = mma(bf[x], af[y], acc);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = 32 * (ti - tj) + l32 - (8 * q + 4 * half + e);
                            x[e] = acc[4 * q + e] * s.pair[31 + d];
                            if (d < 0)
                                x[e] = 0.f;
                        }
#pragma unroll
                        for (int p = 0; p < IP; ++p) {
                            const u32x2 w = {round_pair(x[0], x[1]), round_pair(x[2], x[3])};
                            *reinterpret_cast<u32x2 *>(&s.p[p][32 * it + l32][32 * jt + 8 * q + 4 * half]) = w;
                            if (p + 1 < IP) {
                                x[0] = rest(x[0], low16(w[0]));
                                x[1] = rest(x[1], high16(w[0]));
                                x[2] = rest(x[2], low16(w[1]));
                                x[3] = rest(x[3], high16(w[1]));
                            }
                        }
                    }
                }
            }

            // What the rows read of the state.
#pragma unroll
            for (int it = 0; it < 2; ++it)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[it][r] = 0.f;
#pragma unroll
            for (int q = 0; q < 2 * MT; ++q) {
                float x[8];
                u32x4 zf[IP];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = z[q / 2][8 * (q % 2) + e];
                parts_of<IP, false>(x, zf);
#pragma unroll
                for (int it = 0; it < 2; ++it)
#pragma unroll
                    for (int y = 0; y < IP; ++y) {
                        const u32x4 af = *reinterpret_cast<const u32x4 *>(
                            &s.a[y][32 * it + l32][16 * q + 8 * half]);
#pragma unroll
                        for (int w = 0; w + y < IP; ++w)
                            o[it] = mma(zf[w], af, o[it]);
                    }
            }
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const float w = s.pw[32 * it + l32 + 1 - sw.shift];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[it][r] *= w;
            }
            __syncthreads();
        }

        // What they read of the chunk's own tokens, and the state past it.
        const Power whole = {s.pw[cnt], s.pl[cnt]};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                z[mt][r] = decayed(z[mt][r], whole);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u32x4 cf[IP];
#pragma unroll
            for (int p = 0; p < IP; ++p)
                cf[p] = column_frag<S::LD>(&s.c[p][16 * q + trow][32 * wave + tcol]);
            if constexpr (!STATES) {
#pragma unroll
                for (int it = q / 2; it < 2; ++it)
#pragma unroll
                    for (int y = 0; y < IP; ++y) {
                        const u32x4 pf = *reinterpret_cast<const u32x4 *>(
                            &s.p[y][32 * it + l32][16 * q + 8 * half]);
#pragma unroll
                        for (int x = 0; x + y < IP; ++x)
                            o[it] = mma(cf[x], pf, o[it]);
                    }
            }
            if (bad)
                continue;
            float x[8];
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&s.wt[16 * q + 8 * half]);
            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&s.wt[16 * q + 8 * half + 4]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = e & 1 ? high16(cf[0][e / 2]) : low16(cf[0][e / 2]);
#pragma unroll
                for (int p = 1; p < IP; ++p)
                    x[e] += e & 1 ? high16(cf[p][e / 2]) : low16(cf[p][e / 2]);
                x[e] *= e < 4 ? w0[e] : w1[e - 4];
            }
            u32x4 xf[WP];
            parts_of<WP, true>(x, xf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int y = 0; y < IP; ++y) {
                    const u32x4 bf = column_frag<S::LD>(&s.b[y][16 * q + trow][32 * mt + tswap]);
#pragma unroll
                    for (int p = 0; p + y < WP; ++p)
                        z[mt] = mma(bf, xf[p], z[mt]);
                }
        }
        if (bad) {                     // one token, with a value that is not finite
            float v = 0.f;
#pragma unroll
            for (int p = 0; p < IP; ++p)
                v += (float)s.c[p][0][col];
            v *= s.wt[0];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float b = 0.f;
#pragma unroll
                    for (int p = 0; p < IP; ++p)
                        b += (float)s.b[p][0][mt * 32 + 16 * (r / 8) + 8 * half + r % 8];
                    z[mt][r] = __builtin_fmaf(b, v, z[mt][r]);
                }
        }

        if constexpr (!STATES) {
            const uint64_t t0 = pl.first + (sw.rev ? pl.len - 1 - at : at);
            const int64_t row0 = (int64_t)pl.seq * sw.out_seq + (int64_t)t0 * sw.out_tok +
                                 (int64_t)head * sw.out_head + wave * 32;
            const int64_t step = dir * sw.out_tok;
            if (sw.out_f32) {          // partial gradients of shared heads: dense, so aligned
                float *out = static_cast<float *>(sw.out) + row0;
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const int i = 32 * it + l32;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 y;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = o[it][4 * q + e] * sw.out_scale;
                        const int c0 = 8 * q + 4 * half;
                        if (i >= cnt || wave * 32 + c0 >= n)
                            continue;
                        if (n % 4 == 0) {
                            *reinterpret_cast<f32x4 *>(out + i * step + c0) = y;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (wave * 32 + c0 + e < n)
                                    out[i * step + c0 + e] = y[e];
                        }
                    }
                }
            } else {
                // Through LDS, in 16-byte pieces that trade places by row.
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const int i = 32 * it + l32;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        T y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = (T)(o[it][4 * q + e] * sw.out_scale);
                        u32x2 w;
                        __builtin_memcpy(&w, y, 8);
                        *reinterpret_cast<u32x2 *>(&s.o[wave][i][8 * (q ^ ((i >> 2) & 3)) + 4 * half]) = w;
                    }
                }
                T *out = static_cast<T *>(sw.out) + row0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = 16 * k + lane / 4, q = lane & 3;
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(&s.o[wave][i][8 * (q ^ ((i >> 2) & 3))]);
                    if (i < cnt && wave * 32 + 8 * q < n) {
                        T *to = out + i * step + 8 * q;
                        if (sw.out_aligned) {
                            *reinterpret_cast<u32x4 *>(to) = w;
                        } else {
                            uint16_t *h = reinterpret_cast<uint16_t *>(to);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (wave * 32 + 8 * q + e < n)
                                    h[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
            }
        }
        at = next;
        cnt = next_cnt;
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
                const int row = mt * 32 + 16 * (r / 8) + 8 * half + r % 8;
                if (row < m)
                    st[row * sw.state_m] = z[mt][r];
            }
    }
}

template <class T, int D, bool VEC, int WP>
void run_split(const SweepSet &set, hipStream_t stream)
{
    const dim3 grid(set.items, set.heads, (unsigned)set.count);
    if (set.seg_len) {
        sweep_split_kernel<T, D, VEC, WP, true><<<grid, D * 2, 0, stream>>>(set);
        launch_segment_scan(set, D, stream);
    }
    sweep_split_kernel<T, D, VEC, WP, false><<<grid, D * 2, 0, stream>>>(set);
}

template <class T, int D>
void split_of(const SweepSet &set, hipStream_t stream)
{
    bool states = false;
    for (int i = 0; i < set.count; ++i)
        states |= set.s[i].state_out != nullptr;
    if (set.aligned && states)
        run_split<T, D, true, 3>(set, stream);
    else if (set.aligned)
        run_split<T, D, true, 2>(set, stream);
    else if (states)
        run_split<T, D, false, 3>(set, stream);
    else
        run_split<T, D, false, 2>(set, stream);
}

}  // namespace

void launch_sweeps_split(const SweepSet &set, int width, hipStream_t stream)
{
    if (set.dtype == LIBSCAN_BF16) {
        if (width <= 64)
            split_of<__bf16, 64>(set, stream);
        else
            split_of<__bf16, 128>(set, stream);
    } else {
        if (width <= 64)
            split_of<_Float16, 64>(set, stream);
        else
            split_of<_Float16, 128>(set, stream);
    }
}

}  // namespace libscan
