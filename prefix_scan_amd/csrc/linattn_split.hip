// linattn_split.hip -- the sweep of linattn.hpp in 16-bit matrix products
// (v_mfma_f32_16x16x32) with 32-bit sums.
//
// A workgroup of D / 16 waves (D = 64 or 128) has one segment of one sequence
// and head; wave w owns 16 columns n and keeps its m x 16 part of the state Z
// in 32-bit accumulators for the whole segment.  It takes C tokens at a time
// (64; 32 for f32 rows); with A, B, C the chunk's rows
//
//   out^T = Z^T A^T (p^(i+1-shift)) + C^T ((A B^T) o mask p^(i-j))^T
//   Z    <- p^C Z + B^T (p^(C-1+shift-j) C)
//
// so the state is read and written once a segment and every row of a, b and
// c is read once.  The rows of chunk t + 1 are on their way in registers
// while chunk t is computed from LDS.  16 columns a wave keep it at 128
// registers, so that four waves a SIMD hide each other's waits: 4 x 4096
// tokens of 32 heads of 128 took 166 us with 32 columns a wave and half as
// many waves, 130 with these, when bf16's scores and state were one part (and
// 150 now; in segments, whose states are another 62).  Up to five vector
// registers and 38 scalar ones are spilled all the same, in the 16-bit kinds
// of 128.
//
// What bounds it.  That sweep moves 590 MB in 150 us, 3.9 TB/s (a copy: 6.8),
// with 1.2 of 2.6 wave cycles waiting: each wave reads all rows of a and b
// from LDS for its 16 columns, 512 bytes for each 16 x 16 x 32 product, and a
// chunk's memory reads, LDS reads and products follow each other within a
// workgroup; the two workgroups of a compute unit overlap them in part.  With
// one part, the gradients' sweeps of 8 x 2048 x 16 took 197 us even with no
// rows read or written; of those, 17 to 52 went with any one of the four
// steps, and 58 stayed without all of them.
//
// How exact.  An operand is one or more 16-bit parts whose products are
// summed in 32 bits:
//   bf16 rows  are one part.  Scores and the state that a row reads are two,
//              16 bits; the decayed rows that the state sums are three, 24
//              bits, or two where no final state is asked for and the state
//              is only read in two.  One part each, 2^-8, is seen in the
//              outputs: 2.35e-3 from 64 bits in root mean square, where their
//              own rounding, and two parts, are 1.66e-3.  It took 186, 432
//              and 195 us, not 206, 467 and 228, for 4 x 4096 x 32 and
//              65537 x 16 forward and the gradients of 8 x 2048 x 16.
//   f16 rows   are one part of f16.  Scores, state and decayed rows leave
//              f16's range, so they are scaled by powers of two and back in 32
//              bits: each row of scores by its own largest (no row sees what
//              another holds), the state by the largest of a wave's 16 columns,
//              the decayed rows by the largest of those whose b is not zeros.
//              They are two parts each: 2^-22 of a number, or 2^-40 of what it
//              is scaled by where that is more.  The rows' scales cost a
//              barrier and a second look at the scores: 226 us for 37 prompts
//              of 600 tokens on average, 24 heads, 203 with one scale a chunk,
//              which loses ordinary rows beside large ones.
//   f32 rows   are three bf16 parts, 24 bits, as are scores, state and
//              decayed rows; of the nine products the six above 2^-24 are
//              taken, at a rate 2.7 times the 32-bit products'.
//
// Layouts.  An operand lane holds 8 k of row lane % 16; an accumulator
// register r holds row 4 (lane / 16) + r of column lane % 16.  C and B are
// read down their columns by transposing LDS loads.  k runs in the order
// that two tiles' accumulators have it, over the m and over the tokens of
// every 32: lane group g has 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3.  So
// the accumulators of Z are the operand of Z^T A^T as they stand, and the
// column reads of b and c go through 16 rows on end.  Rows of a and of the
// scores are stored in that order.  Rows of a, b and c are 16 elements longer
// than they need be, those of the scores trade places by row: no read meets a
// bank twice.  The 8-byte writes of a's rows and of the scores do: two rows of
// a share their banks, and scores reach half of them (11.9 million cycles of
// the sweep above, about 20 us of a compute unit's).
//
// The chunk is causal by selection, not by multiplication: a masked pair is
// zero whatever the product was.  A value of c that is not finite would still
// reach earlier rows as 0 * inf, so a chunk with one is taken again one token
// at a time; those of a and b reach no other row's scores.
#include "linattn.hpp"

#include "../../include/libscan.h"
#include "device_common.hpp"

namespace libscan {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Parts of a row's elements, and of scores and the state where they are
// multiplied.
template <class T>
struct In;
template <>
struct In<__bf16> {
    static constexpr int kParts = 1, kMade = 2, kChunk = 64;
    static constexpr bool kScaled = false;
};
template <>
struct In<_Float16> {
    static constexpr int kParts = 1, kMade = 2, kChunk = 64;
    static constexpr bool kScaled = true;
};
template <>
struct In<float> {
    static constexpr int kParts = 3, kMade = 3, kChunk = 32;
    static constexpr bool kScaled = false;
};

__device__ __forceinline__ float low16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float above(float x) { return high16(__float_as_uint(x)); }

template <bool F16>
__device__ __forceinline__ float value16(uint32_t w, int high)
{
    if constexpr (F16)
        return (float)__builtin_bit_cast(f16x2, w)[high];
    else
        return high ? high16(w) : low16(w);
}

// a's and b's lower, and upper, halves in one word.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Two floats, both cut to bf16.
__device__ __forceinline__ uint32_t cut_pair(float a, float b)
{
    return high_halves(__float_as_uint(a), __float_as_uint(b));
}

template <bool F16>
__device__ __forceinline__ uint32_t round_pair(float a, float b)
{
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// What is left of x past its part h; some number where x is not finite, so
// that the parts' sum stays what x is.
template <bool F16, bool FINITE>
__device__ __forceinline__ float rest(float x, float h)
{
    constexpr float most = F16 ? 32768.f : 0x1p126f;
    if constexpr (FINITE)
        return x - h;
    return __builtin_amdgcn_fmed3f(x - h, -most, most);
}

// Two floats in P parts: bf16 ones are cut but for the last, which is rounded
// to nearest from what they left; f16 ones are rounded.
template <int P, bool F16, bool FINITE>
__device__ __forceinline__ void parts_of_pair(float a, float b, uint32_t *out)
{
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (p + 1 == P || F16) {
            out[p] = round_pair<F16>(a, b);
            if (p + 1 < P) {
                a = rest<F16, FINITE>(a, value16<F16>(out[p], 0));
                b = rest<F16, FINITE>(b, value16<F16>(out[p], 1));
            }
        } else {
            out[p] = cut_pair(a, b);
            a = rest<F16, FINITE>(a, above(a));
            b = rest<F16, FINITE>(b, above(b));
        }
    }
}

template <int P, bool F16, bool FINITE>
__device__ __forceinline__ void parts_of(const float *x, u32x4 *out)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t w[P];
        parts_of_pair<P, F16, FINITE>(x[2 * e], x[2 * e + 1], w);
#pragma unroll
        for (int p = 0; p < P; ++p)
            out[p][e] = w[p];
    }
}

template <bool F16>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The same number, which the compiler takes for a new one: what follows from
// it stays where it is, instead of in registers all through the loop.
__device__ __forceinline__ int afresh(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// A number that all lanes have, in a scalar register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ uint64_t uniform64(uint64_t x)
{
    return (uint64_t)uniform((uint32_t)(x >> 32)) << 32 | uniform((uint32_t)x);
}

__device__ __forceinline__ float uniform_float(float x) { return __uint_as_float(uniform(__float_as_uint(x))); }

__device__ __forceinline__ double uniform_double(double x)
{
    return __longlong_as_double((int64_t)uniform64((uint64_t)__double_as_longlong(x)));
}

// Eight elements of a row, as fetched.
template <class T>
struct Unit {
    u32x4 w[sizeof(T) / 2];
};

// A tensor's rows of one sequence and head.
template <class T>
struct Lines {
    const T *p;                  // of the sequence's first token
    int64_t tok;
    __device__ __forceinline__ Lines(const Rows &r, uint64_t seq, uint64_t first, uint32_t head)
        : p(row_ptr<T>(r, seq, first, head)), tok(r.tok)
    {
    }
};

// This thread's units of the rows of cnt tokens from the one at `at` on, back
// where REV; zeros past them.  A whole chunk's addresses are a scalar and a
// lane's 32 bits (the host sees to it that those hold them).
template <class T, bool VEC, int W, int THREADS, int N>
__device__ __forceinline__ void fetch(Unit<T> (&r)[N], const Lines<T> &from, uint64_t at, bool rev, int cnt,
                                      int width)
{
    constexpr int PER = W / 8, RS = THREADS / PER, H = (int)sizeof(T) / 2, C = In<T>::kChunk;
    static_assert(N == C / RS, "a chunk of rows");
    if (VEC && cnt == C) {
        const char *base = reinterpret_cast<const char *>(from.p + (int64_t)(rev ? at - (C - 1) : at) * from.tok);
        const int64_t step = (rev ? -RS : RS) * from.tok * (int64_t)sizeof(T);
        const uint32_t tid = afresh((int)threadIdx.x), row = tid / PER, col = tid % PER * 8;
        const uint32_t place = ((rev ? C - 1 - row : row) * (uint32_t)from.tok + col) * (uint32_t)sizeof(T);
        if (width == W) {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    r[k].w[h] = *reinterpret_cast<const u32x4 *>(base + k * step + place + 16 * h);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    r[k].w[h] = u32x4{0, 0, 0, 0};
                    if ((int)col + 4 * h < width)
                        r[k].w[h] = *reinterpret_cast<const u32x4 *>(base + k * step + place + 16 * h);
                }
        }
        return;
    }
    const int tid = afresh((int)threadIdx.x), row0 = tid / PER, col = tid % PER * 8;
    const int64_t step = rev ? -from.tok : from.tok;
    const T *p = from.p + (int64_t)at * from.tok + row0 * step + col;
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int h = 0; h < H; ++h)
            r[k].w[h] = u32x4{0, 0, 0, 0};
        if (row0 + k * RS < cnt && col < width) {
            if (VEC) {
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (h == 0 || col + 4 < width)
                        r[k].w[h] = reinterpret_cast<const u32x4 *>(p)[h];
            } else if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < width)
                        r[k].w[e / 4][e % 4] = __float_as_uint(p[e]);
            } else {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < width)
                        r[k].w[0][e / 2] |= (uint32_t)h[e] << (16 * (e & 1));
            }
        }
        p += RS * step;
    }
}

// The fetched rows into LDS, in parts; PERMUTED in the order of k.
template <class T, bool PERMUTED, int W, int THREADS, int N, int CH, int LD>
__device__ __forceinline__ void stage(const Unit<T> (&r)[N], uint16_t (*dst)[CH][LD])
{
    constexpr int PER = W / 8, RS = THREADS / PER;
    // f32 rows leave registers for the addresses.
    const int tid = sizeof(T) == 4 ? (int)threadIdx.x : afresh((int)threadIdx.x);
    const int row0 = tid / PER, unit = tid % PER;
    const int col = PERMUTED ? unit / 4 * 32 + (unit & 1) * 16 + (unit & 2) * 2 : unit * 8;
    const auto put = [&](int part, int row, u32x4 w) {
        uint16_t *p = &dst[part][row][col];
        if (PERMUTED) {
            *reinterpret_cast<u32x2 *>(p) = u32x2{w[0], w[1]};
            *reinterpret_cast<u32x2 *>(p + 8) = u32x2{w[2], w[3]};
        } else {
            *reinterpret_cast<u32x4 *>(p) = w;
        }
    };
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (sizeof(T) == 2) {
            put(0, row0 + k * RS, r[k].w[0]);
        } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = __uint_as_float(r[k].w[e / 4][e % 4]);
            u32x4 p[3];
            parts_of<3, false, false>(x, p);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                put(i, row0 + k * RS, p[i]);
        }
    }
}

template <class T, int N>
__device__ __forceinline__ bool any_not_finite(const Unit<T> (&r)[N])
{
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = r[k].w[h][e];
                if constexpr (sizeof(T) == 4)
                    bad |= (w & 0x7F800000u) + 0x00800000u;
                else if constexpr (In<T>::kScaled)
                    bad |= (w & 0x7C007C00u) + 0x04000400u;
                else
                    bad |= (w & 0x7F807F80u) + 0x00800080u;
            }
    return (bad & (sizeof(T) == 4 ? 0x80000000u : 0x80008000u)) != 0;
}

// The largest of a wave's numbers.
__device__ __forceinline__ uint32_t wave_most(uint32_t x)
{
    const auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    x = larger(x, dpp<kDppRowShr1, 0xF>(x));
    x = larger(x, dpp<kDppRowShr2, 0xF>(x));
    x = larger(x, dpp<kDppRowShr4, 0xF>(x));
    x = larger(x, dpp<kDppRowShr8, 0xF>(x));
    x = larger(x, dpp<kDppRowBcast15, 0xA>(x));
    x = larger(x, dpp<kDppRowBcast31, 0xC>(x));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The largest exponent that a decayed row of c has among this thread's rows of
// f16: |x| < 2^(the returned - 140).  Rows whose b is zeros add nothing to the
// state and do not count.  pw: the power of the chunk's first row, those of
// the next before it.
template <class T, int W, int THREADS, int N>
__device__ __forceinline__ int decayed_exponent(const Unit<T> (&b)[N], const Unit<T> (&c)[N], const float *pw,
                                                float scale, int cnt)
{
    constexpr int PER = W / 8, RS = THREADS / PER;
    const int tid = afresh((int)threadIdx.x), row0 = tid / PER, lane = tid & 63;
    int most = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t any = 0, lo = 0, hi = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            any |= b[k].w[0][e];
            const uint32_t l = c[k].w[0][e] & 0x7FFFu, h = c[k].w[0][e] & 0x7FFF0000u;
            lo = l > lo ? l : lo;
            hi = h > hi ? h : hi;
        }
        const uint64_t rows = __ballot((any & 0x7FFF7FFFu) != 0) >> (lane / PER * PER);
        const uint32_t top = lo > hi >> 16 ? lo : hi >> 16;
        const int row = row0 + k * RS;
        if ((rows & ((1u << PER) - 1)) != 0 && top != 0 && row < cnt) {
            const int e = (int)(top >> 10) + (int)(__float_as_uint(scale * pw[-row]) >> 23 & 255);
            most = e > most ? e : most;
        }
    }
    return most;
}

// LDS by its own pointers: a lane's place plus a constant, which the
// instruction adds.
typedef __attribute__((address_space(3))) uint16_t lds_u16;

// Eight rows down 16 columns, in the order of k: p is this lane's place in
// the first four of them.
template <int LD>
__device__ __forceinline__ u32x4 column_frag(lds_u16 *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
    const u32x2 b = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * LD)));
    return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ u32x4 row_frag(lds_u16 *p)
{
    return *(const __attribute__((address_space(3))) u32x4 *)p;
}

// The same of a row that is not stored in the order of k.
__device__ __forceinline__ u32x4 row_frag_of(lds_u16 *p)
{
    typedef const __attribute__((address_space(3))) u32x2 lds_u32x2;
    const u32x2 a = *(lds_u32x2 *)p, b = *(lds_u32x2 *)(p + 16);
    return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ float power2(int e)
{
    return __builtin_amdgcn_ldexpf(1.f, e < -126 ? -126 : e > 126 ? 126 : e);
}

// The power of two that takes a row's scores, the largest of them with the bits
// `most`, to below 2^15.  Not past 2^40: scores below 2^-26 lie below f16's
// outputs whatever the rows of c are.
__device__ __forceinline__ int row_scale(uint32_t most)
{
    const int e = (int)(most >> 23);
    return e == 255 ? 0 : e < 101 ? 40 : 141 - e;
}

// This lane's row and four of the 16 columns from `first` of each tile.
template <class T, int IT>
__device__ __forceinline__ void put_out(const f32x4 *o, T *out, int64_t tok, uint64_t at, bool rev, int cnt,
                                        int first, int n, bool aligned)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    const int lane = afresh((int)threadIdx.x & 63), c0 = lane / 16 * 4, row = lane & 15;
    out += first;
    if (aligned && cnt == 16 * IT) {
        char *base = reinterpret_cast<char *>(out + (int64_t)(rev ? at - (16 * IT - 1) : at) * tok);
        const int64_t step = (rev ? -16 : 16) * tok * (int64_t)sizeof(T);
        const uint32_t place = (uint32_t)(rev ? 16 * IT - 1 - row : row) * (uint32_t)tok + c0;
        if (first + c0 < n) {
#pragma unroll
            for (int it = 0; it < IT; ++it)
                *reinterpret_cast<t4 *>(base + it * step + place * (uint32_t)sizeof(T)) =
                    __builtin_convertvector(o[it], t4);
        }
        return;
    }
    const int64_t step = rev ? -tok : tok;
    T *to = out + (int64_t)at * tok + row * step + c0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (16 * it + row < cnt && first + c0 + e < n)
                to[e] = (T)o[it][e];
        to += 16 * step;
    }
}

// A chunk's outputs in LDS, whole rows in pieces of 16 bytes that trade places
// by row, so that neither columns nor rows meet a bank twice.
template <class T, int D>
struct OutRows {
    static constexpr int V = 16 / (int)sizeof(T), PIECES = D / V;
    T x[In<T>::kChunk][D];
    __device__ __forceinline__ T *at(int row, int piece) { return &x[row][(piece ^ (row & (PIECES - 1))) * V]; }
};

template <class T, int D, int IT>
__device__ __forceinline__ void hold_rows(OutRows<T, D> &s, const f32x4 *o, int wave, int l16, int g4)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    constexpr int V = 16 / (int)sizeof(T);
    const int c0 = wave * 16 + 4 * g4;
#pragma unroll
    for (int it = 0; it < IT; ++it)
        *reinterpret_cast<t4 *>(s.at(16 * it + l16, c0 / V) + c0 % V) = __builtin_convertvector(o[it], t4);
}

// From there to memory, 16 bytes a lane.
template <class T, int D, int THREADS>
__device__ __forceinline__ void put_rows(OutRows<T, D> &s, T *out, int64_t tok, uint64_t at, bool rev, int cnt,
                                         int n, bool whole)
{
    constexpr int C = In<T>::kChunk, V = OutRows<T, D>::V, PER = OutRows<T, D>::PIECES, RS = THREADS / PER;
    const int tid = afresh((int)threadIdx.x), row0 = tid / PER, piece = tid % PER, col = piece * V;
    if (whole && cnt == C) {
        char *base = reinterpret_cast<char *>(out + (int64_t)(rev ? at - (C - 1) : at) * tok);
        const int64_t step = (rev ? -RS : RS) * tok * (int64_t)sizeof(T);
        const uint32_t place =
            ((uint32_t)(rev ? C - 1 - row0 : row0) * (uint32_t)tok + (uint32_t)col) * (uint32_t)sizeof(T);
        if (col < n) {
#pragma unroll
            for (int k = 0; k < C / RS; ++k)
                *reinterpret_cast<u32x4 *>(base + k * step + place) =
                    *reinterpret_cast<const u32x4 *>(s.at(row0 + k * RS, piece));
        }
        return;
    }
    const int64_t step = rev ? -tok : tok;
    T *to = out + (int64_t)at * tok + row0 * step + col;
#pragma unroll
    for (int k = 0; k < C / RS; ++k) {
        const T *x = s.at(row0 + k * RS, piece);
        if (row0 + k * RS < cnt) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (col + e < n)
                    to[e] = x[e];
        }
        to += RS * step;
    }
}

template <class T, int D, bool STATES>
struct Lds {
    static constexpr int C = In<T>::kChunk, IP = In<T>::kParts, OP = In<T>::kMade;
    static constexpr int LD = D + 16, LP = C == 64 ? 64 : C + 16;
    __device__ static constexpr int swap(int row) { return C == 64 ? (row >> 1 & 3) << 1 : 0; }
    alignas(16) uint16_t a[STATES ? 1 : IP][STATES ? 1 : C][LD];
    alignas(16) uint16_t b[IP][C][LD];
    uint16_t c[IP][C][LD];
    alignas(16) uint16_t p[STATES ? 1 : OP][STATES ? 1 : C][LP];
    float pw[C + 4], pl[C + 4];            // powers of the decay: hi, lo
    float pair[C + 16];                    // pair_scale out_scale p^d at 16 + d, 0 for d < 0
    float wt[C];                           // pair_scale p^(cnt-1+shift-j)
    int bad[2];
    int top[2];                            // f16: decayed_exponent of the chunk
    uint32_t most[In<T>::kScaled && !STATES ? C : 1];   // bits of each row's largest score
    // A chunk's outputs take the place of its rows of a, which have been read by
    // then: room of their own would leave one workgroup a compute unit.
    __device__ __forceinline__ OutRows<T, D> &outputs()
    {
        static_assert(STATES || sizeof(OutRows<T, D>) <= sizeof(a), "outputs within a's rows");
        return *reinterpret_cast<OutRows<T, D> *>(&a[0][0][0]);
    }
};

// STATES: only the segment's own contribution to the state, into set.seg.
// WP: parts of the decayed rows that the state sums.
template <class T, int D, bool VEC, int WP, bool STATES>
__global__ __launch_bounds__(D * 4, sizeof(T) == 4 && !STATES ? 2 : 4) void sweep_split_kernel(const SweepSet set)
{
    constexpr int C = In<T>::kChunk, IP = In<T>::kParts, OP = In<T>::kMade;
    constexpr int NW = D / 16, THREADS = D * 4, KK = D / 32, IT = C / 16, KS = C / 32;
    constexpr int N = C * D / 8 / THREADS;
    constexpr bool F16 = In<T>::kScaled;
    // Whether columns and rows past the widths are left out.  bf16 rows have no
    // registers for the branches.
    constexpr bool SKIP = sizeof(T) == 4 || F16;
    typedef Lds<T, D, STATES> S;
    __shared__ __align__(16) S s;

    // Of a gradient's three sweeps over the same rows, two read the same ones
    // at the same time: they follow each other on one of the 8 dies (blocks
    // go round them), so that its cache has the rows for all.
    uint32_t sweep = 0, item = blockIdx.x, head = blockIdx.y;
    if (set.count > 1) {
        const uint64_t units = (uint64_t)gridDim.x * set.heads, n = units / 8 * 8 * set.count;
        const uint64_t b = item + gridDim.x * (head + (uint64_t)set.heads * blockIdx.z);
        uint64_t unit;
        if (b < n) {
            sweep = (uint32_t)(b / 8 % set.count);
            unit = b / 8 / set.count * 8 + b % 8;
        } else {
            sweep = (uint32_t)((b - n) % set.count);
            unit = units / 8 * 8 + (b - n) / set.count;
        }
        item = (uint32_t)(unit % gridDim.x);
        head = (uint32_t)(unit / gridDim.x);
    } else if (set.ends) {
        // Sequences differ in length: each one's heads go round the dies, so
        // that these have equal shares.  37 prompts of 600 tokens on average,
        // 24 heads, f16: 204 us; 220 to 320 by items, as their number has it.
        const uint64_t b = blockIdx.x + (uint64_t)gridDim.x * blockIdx.y;
        item = uniform((uint32_t)(b / set.heads));
        head = uniform((uint32_t)(b % set.heads));
    }
    const Sweep &sw = set.s[sweep];
    // Rows past the last end: each item has some of them; mostly there are none.
    const auto clear_rest = [&]() {
        if (STATES || !set.clear_from || sw.out_f32)
            return;
        T *const out = static_cast<T *>(sw.out) + (int64_t)head * sw.out_head;
        for (uint64_t t = *set.clear_from + (uint64_t)item; t < set.tokens; t += gridDim.x)
            if ((int)threadIdx.x < sw.n)
                out[(int64_t)t * sw.out_tok + threadIdx.x] = (T)0.f;
    };
    Place pl;
    if (!place_of(set, item, STATES, &pl)) {
        clear_rest();
        return;
    }
    pl.seq = uniform(pl.seq);
    pl.first = uniform64(pl.first);
    pl.len = uniform64(pl.len);
    pl.lo = uniform64(pl.lo);
    pl.hi = uniform64(pl.hi);
    pl.slot0 = uniform(pl.slot0);
    pl.last = pl.hi == pl.len;
    const int wave = uniform(threadIdx.x / 64);
    const int lane = threadIdx.x & 63, g4 = lane >> 4, l16 = lane & 15;
    const float g = set.log_decay[head];
    const int m = sw.m, n = sw.n;
    const bool rev = sw.rev;
    const Lines<T> la(sw.a, pl.seq, pl.first, head), lb(sw.b, pl.seq, pl.first, head),
        lc(sw.c, pl.seq, pl.first, head);
    Unit<T> ra[STATES ? 1 : N], rb[N], rc[N];
    const auto fetch_a = [&](uint64_t at, int cnt) {
        if constexpr (!STATES)
            fetch<T, VEC, D, THREADS>(ra, la, rev ? pl.len - 1 - at : at, rev, cnt, m);
    };
    const auto fetch_b = [&](uint64_t at, int cnt) {
        fetch<T, VEC, D, THREADS>(rb, lb, rev ? pl.len - 1 - at : at, rev, cnt, m);
    };
    const auto fetch_c = [&](uint64_t at, int cnt) {
        fetch<T, VEC, D, THREADS>(rc, lc, rev ? pl.len - 1 - at : at, rev, cnt, n);
    };
    const auto fetch_chunk = [&](uint64_t at, int cnt) {
        fetch_a(at, cnt);
        fetch_b(at, cnt);
        fetch_c(at, cnt);
    };
    uint64_t at = pl.lo, single = 0;   // tokens below `single` are taken one at a time
    int cnt = pl.hi - at < C ? (int)(pl.hi - at) : C, cnt_wt = -1, turn = 0;
    double whole = 1.0, drift = 1.0;   // p^cnt; what the factors so far left of it
    fetch_chunk(at, cnt);
    for (int i = threadIdx.x; i < C + 17; i += THREADS) {
        const int d = i - 16;
        const Power p = d >= 0 ? decay_power(g, (double)d) : Power{0.f, 0.f};
        if (d < C)
            s.pair[i] = sw.pair_scale * sw.out_scale * p.hi;
        if (d >= 0) {
            s.pw[d] = p.hi;
            s.pl[d] = p.lo;
        }
    }
    if (threadIdx.x < 2)
        s.bad[threadIdx.x] = s.top[threadIdx.x] = 0;
    if constexpr (!STATES)                  // the scores' upper corner stays zero
        for (int i = threadIdx.x; i < OP * C * S::LP / 8; i += THREADS)
            reinterpret_cast<u32x4 *>(&s.p[0][0][0])[i] = u32x4{0, 0, 0, 0};

    const int col = wave * 16 + l16;
    const bool active = wave * 16 < n;      // whether the wave has columns
    const uint64_t sh = (uint64_t)pl.seq * set.heads + head;
    // Two tiles of 16 rows: z[kk][u][r] is row 32 kk + 16 u + 4 g4 + r of column col.
    f32x4 z[KK][2];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u)
            z[kk][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto seg_of = [&](uint32_t slot) {
        return set.seg + (((uint64_t)sweep * set.slots + slot) * set.heads + head) * (D * D) +
               (wave * KK * 64 + lane) * 8;
    };
    if (!STATES && active) {
        if (pl.lo) {
            // The scan's result, or the scan itself where segments are few.
            const bool few = pl.len <= kFewSegments * set.seg_len;
            const uint32_t before = (uint32_t)(pl.lo / set.seg_len);
            const Power w = decay_power(g, (double)set.seg_len);
            for (uint32_t k = few ? 0 : before - 1; k < before; ++k) {
                const float *seg = seg_of(pl.slot0 + k);
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const f32x4 t = *reinterpret_cast<const f32x4 *>(seg + kk * 512 + 4 * u);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            z[kk][u][r] = decayed(z[kk][u][r], w) + t[r];
                    }
            }
        }
        if (sw.state_in && col < n) {
            const Power w = decay_power(g, (double)pl.lo);
            const float *st = sw.state_in + sh * ((uint64_t)m * n) + col * sw.state_n;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int row = kk * 32 + e / 4 * 16 + 4 * g4 + e % 4;
                    if (row < m)
                        z[kk][e / 4][e % 4] += decayed(st[row * sw.state_m], w);
                }
        }
    }
    // f16: z holds the state times 2^sigma.  top_of_z: the exponent of the
    // largest number that is finite in it.
    int sigma = 0;
    const auto top_of_z = [&]() {
        uint32_t own = 0;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = __float_as_uint(z[kk][e / 4][e % 4]) & 0x7FFFFFFFu;
                own = x > own ? x : own;
            }
        own = wave_most(own);
        if (own >= 0x7F800000u) {
            own = 0;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t x = __float_as_uint(z[kk][e / 4][e % 4]) & 0x7FFFFFFFu;
                    own = x > own && x < 0x7F800000u ? x : own;
                }
            own = wave_most(own);
        }
        return (int)(own >> 23);
    };

    const int64_t out0 = (int64_t)pl.seq * sw.out_seq + (int64_t)pl.first * sw.out_tok +
                         (int64_t)head * sw.out_head;
    // This lane's places: along the rows of a, b and the scores, and down the
    // columns of b and c.
    lds_u16 *const arow = (lds_u16 *)&s.a[0][0][0] + l16 * S::LD + 8 * g4;
    lds_u16 *const bcol = (lds_u16 *)&s.b[0][0][0] + (4 * g4 + l16 / 4) * S::LD + 4 * (l16 & 3);
    lds_u16 *const ccol = (lds_u16 *)&s.c[0][0][0] + (4 * g4 + l16 / 4) * S::LD + 4 * (l16 & 3) + wave * 16;

    while (at < pl.hi) {
        __syncthreads();
        if constexpr (!STATES)
            stage<T, true, D, THREADS>(ra, s.a);
        stage<T, false, D, THREADS>(rb, s.b);
        stage<T, false, D, THREADS>(rc, s.c);
        if (__any(any_not_finite(rc)) && lane == 0)
            s.bad[turn] = 1;
        if constexpr (F16) {
            const int top = (int)wave_most((uint32_t)decayed_exponent<T, D, THREADS>(
                rb, rc, &s.pw[cnt - 1 + sw.shift], sw.pair_scale, cnt));
            if (lane == 0)
                atomicMax(&s.top[turn], top);
            if (!STATES && threadIdx.x < C)
                s.most[threadIdx.x] = 0;
        }
        if (cnt != cnt_wt) {
            const int j = afresh((int)threadIdx.x);
            if (j < C)
                s.wt[j] = j < cnt ? sw.pair_scale * s.pw[cnt - 1 + sw.shift - j] : 0.f;
            cnt_wt = cnt;
            whole = uniform_double((double)s.pw[cnt] + (double)s.pl[cnt]);
        }
        __syncthreads();
        const bool bad = uniform(s.bad[turn]) != 0;
        const int top = F16 ? (int)uniform(s.top[turn]) : 0;
        turn ^= 1;
        if (threadIdx.x == 0)
            s.bad[turn] = s.top[turn] = 0;
        if (bad && cnt > 1) {          // again, one token at a time
            single = at + cnt;
            cnt = 1;
            fetch_chunk(at, cnt);
            continue;
        }
        const uint64_t next = at + cnt;
        const uint64_t left = pl.hi - next;
        const int next_cnt = left == 0 ? 0 : next < single ? 1 : (int)(left < C ? left : C);
        // The next chunk's rows are asked for between the steps: all at once they
        // fill the queue to memory, and the waves stand still for a third of the
        // chunk's time.
        if (next_cnt) {
            fetch_a(next, next_cnt);
            if constexpr (STATES) {
                fetch_b(next, next_cnt);
                fetch_c(next, next_cnt);
            }
        }

        int top_z = 0;
        f32x4 o[IT];
        if constexpr (!STATES) {
            // Scores, transposed: a lane has token i and four consecutive j.
            const int own = afresh(lane), oi = own & 15, og = own / 16;
            lds_u16 *const brow = (lds_u16 *)&s.b[0][0][0] + oi * S::LD + 4 * og;
            constexpr int TILES = IT * (IT + 1) / 2;
            const auto row_of = [](int x) { return x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3; };
            const auto scores = [&](int x) {
                const int it = row_of(x), jt = x - it * (it + 1) / 2;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    if (SKIP && kk * 32 >= m)
                        break;
                    u32x4 af[IP], bf[IP];
#pragma unroll
                    for (int p = 0; p < IP; ++p) {
                        af[p] = row_frag(arow + (p * C + 16 * it) * S::LD + 32 * kk);
                        bf[p] = row_frag_of(brow + (p * C + 16 * jt) * S::LD + 32 * kk);
                    }
#pragma unroll
                    for (int u = 0; u < IP; ++u)
#pragma unroll
                        for (int v = 0; u + v < IP; ++v)
                            acc = mma<F16>(bf[u], af[v], acc);
                }
                const int d0 = 16 * (it - jt) + oi - 4 * og;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[e] *= s.pair[16 + d0 - e];
                    if (d0 - e < 0)
                        acc[e] = 0.f;
                }
                return acc;
            };
            // This lane's four of a tile, in each part.
            const auto place = [&](int p, int x) {
                const int it = row_of(x), jt = x - it * (it + 1) / 2;
                return reinterpret_cast<u32x2 *>(
                    &s.p[p][16 * it + oi][((4 * (jt / 2) + og) ^ S::swap(oi)) * 8 + 4 * (jt & 1)]);
            };
            const auto put_scores = [&](int x, f32x4 y) {
                uint32_t w0[OP], w1[OP];
                parts_of_pair<OP, F16, false>(y[0], y[1], w0);
                parts_of_pair<OP, F16, false>(y[2], y[3], w1);
#pragma unroll
                for (int p = 0; p < OP; ++p)
                    *place(p, x) = u32x2{w0[p], w1[p]};
            };
            if constexpr (F16) {
                // Each row by its own power of two, so that it has what it would
                // have without the others.  Until that is known the scores' 32
                // bits wait in the places of the two parts: in registers over
                // the barrier they cost spills.
#pragma unroll 1
                for (int x = wave; x < TILES; x += NW) {
                    const f32x4 y = scores(x);
                    uint32_t b[4], most = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        b[e] = __float_as_uint(y[e]);
                        most = (b[e] & 0x7FFFFFFFu) > most ? b[e] & 0x7FFFFFFFu : most;
                    }
                    atomicMax(&s.most[16 * row_of(x) + oi], most);
                    *place(0, x) = u32x2{low_halves(b[0], b[1]), low_halves(b[2], b[3])};
                    *place(1, x) = u32x2{high_halves(b[0], b[1]), high_halves(b[2], b[3])};
                }
                __syncthreads();
#pragma unroll 1
                for (int x = wave; x < TILES; x += NW) {
                    const u32x2 lo = *place(0, x), hi = *place(1, x);
                    const f32x4 y = {__uint_as_float(low_halves(lo[0], hi[0])),
                                     __uint_as_float(high_halves(lo[0], hi[0])),
                                     __uint_as_float(low_halves(lo[1], hi[1])),
                                     __uint_as_float(high_halves(lo[1], hi[1]))};
                    put_scores(x, y * power2(row_scale(s.most[16 * row_of(x) + oi])));
                }
            } else {
#pragma unroll 1
                for (int x = wave; x < TILES; x += NW)
                    put_scores(x, scores(x));
            }

            if (next_cnt)
                fetch_b(next, next_cnt);

            // What the rows read of the state.
#pragma unroll
            for (int it = 0; it < IT; ++it)
                o[it] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (!SKIP || active) {
                // f16: the state by the power of two that takes it to below 2^15.
                int tau = 0;
                if constexpr (F16) {
                    top_z = top_of_z();
                    tau = 141 - top_z;
                }
                const float by = F16 ? power2(tau) : 1.f;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    if (SKIP && kk * 32 >= m)
                        break;
                    float x[8];
                    u32x4 zf[OP];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = F16 ? z[kk][e / 4][e % 4] * by : z[kk][e / 4][e % 4];
                    parts_of<OP, F16, false>(x, zf);
#pragma unroll
                    for (int it = 0; it < IT; ++it)
#pragma unroll
                        for (int v = 0; v < IP; ++v) {
                            const u32x4 af = row_frag(arow + (v * C + 16 * it) * S::LD + 32 * kk);
#pragma unroll
                            for (int u = 0; u + v < OP; ++u)
                                o[it] = mma<F16>(zf[u], af, o[it]);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    float w = s.pw[16 * it + oi + 1 - sw.shift] * sw.out_scale;
                    if constexpr (F16)
                        w = w * power2(-tau) * power2(-sigma) * power2(row_scale(s.most[16 * it + oi]));
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[it][r] *= w;
                }
            }
            if (next_cnt)
                fetch_c(next, next_cnt);
            __syncthreads();
        }

        // What they read of the chunk's own tokens.
        if constexpr (!STATES) {
            const uint64_t tok = rev ? pl.len - 1 - at : at;
            if (!SKIP || active) {
                const int own = afresh(lane);
                lds_u16 *const prow = (lds_u16 *)&s.p[0][0][0] + (own & 15) * S::LP;
                const int piece = (own / 16) ^ S::swap(own & 15);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    u32x4 cf[IP];
#pragma unroll
                    for (int p = 0; p < IP; ++p)
                        cf[p] = column_frag<S::LD>(ccol + (p * C + 32 * ks) * S::LD);
#pragma unroll
                    for (int it = 2 * ks; it < IT; ++it)
#pragma unroll
                        for (int v = 0; v < OP; ++v) {
                            const u32x4 pf = row_frag(prow + (v * C + 16 * it) * S::LP + (piece ^ (4 * ks)) * 8);
#pragma unroll
                            for (int u = 0; u < IP && u + v < OP; ++u)
                                o[it] = mma<F16>(cf[u], pf, o[it]);
                        }
                }
                if constexpr (F16) {
#pragma unroll
                    for (int it = 0; it < IT; ++it)
                        o[it] *= power2(-row_scale(s.most[16 * it + (own & 15)]));
                }
                if (sizeof(T) == 2 && sw.out_f32)
                    put_out<float, IT>(o, static_cast<float *>(sw.out) + out0, sw.out_tok, tok, rev, cnt,
                                       wave * 16, n, sw.out_whole);
                else
                    hold_rows<T, D, IT>(s.outputs(), o, wave, l16, g4);
            }
            if (!(sizeof(T) == 2 && sw.out_f32)) {
                __syncthreads();
                put_rows<T, D, THREADS>(s.outputs(), static_cast<T *>(sw.out) + out0, sw.out_tok, tok, rev,
                                        cnt, n, sw.out_whole);
            }
        }
        // The state past the chunk.
        if (!SKIP || active) {
            // The state is decayed by floats whose product follows p^(tokens)
            // itself: the rounding of one is made up for by the next.  Of a
            // subnormal one, whose reciprocal may be infinite, nothing is left.
            const double exact = whole * drift;
            float decay = (float)exact;
            drift = decay >= 0x1p-126f && decay < __builtin_inff()
                        ? 1.0 + (exact - (double)decay) * (double)__builtin_amdgcn_rcpf(decay)
                        : 1.0;
            drift = uniform_double(drift);
            float by = 1.f;
            if constexpr (F16) {
                // The decayed rows to below 2^15, and the state to below 2^100.
                if constexpr (STATES)
                    top_z = top_of_z();
                int to = 155 - top;
                to = to < -100 ? -100 : to > 100 ? 100 : to;
                to = to < sigma + 226 - top_z ? to : sigma + 226 - top_z;
                decay = decay * power2(to) * power2(-sigma);
                sigma = to;
                by = power2(sigma);
            }
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        z[kk][u][r] *= decay;
#pragma unroll 1
            for (int ks = 0; ks < KS; ++ks) {
                u32x4 cf[IP];
#pragma unroll
                for (int p = 0; p < IP; ++p)
                    cf[p] = column_frag<S::LD>(ccol + (p * C + 32 * ks) * S::LD);
                float x[8];
                const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&s.wt[32 * ks + 4 * g4]);
                const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&s.wt[32 * ks + 16 + 4 * g4]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = value16<F16>(cf[0][e / 2], e & 1);
#pragma unroll
                    for (int p = 1; p < IP; ++p)
                        x[e] += value16<F16>(cf[p][e / 2], e & 1);
                    x[e] *= e < 4 ? w0[e] : w1[e - 4];
                    if constexpr (F16)
                        x[e] *= by;
                }
                u32x4 xf[WP];
                // f16: powers past 2^98, or not finite, are not scaled down.
                if (bad || (F16 && top >= 255)) {
                    parts_of<WP, F16, false>(x, xf);
                } else {
                    // Rows that do not count may be past f16, and meet zeros of b.
                    if constexpr (F16)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = __builtin_amdgcn_fmed3f(x[e], -32768.f, 32768.f);
                    parts_of<WP, F16, true>(x, xf);
                }
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    if (SKIP && kk * 32 >= m)
                        break;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int v = 0; v < IP; ++v) {
                            const u32x4 bf =
                                column_frag<S::LD>(bcol + (v * C + 32 * ks) * S::LD + 32 * kk + 16 * u);
#pragma unroll
                            for (int p = 0; p + v < WP; ++p)
                                z[kk][u] = mma<F16>(bf, xf[p], z[kk][u]);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }

        at = next;
        cnt = next_cnt;
    }

    clear_rest();
    if (!active)
        return;
    if constexpr (F16) {
        const float by = power2(-sigma);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                z[kk][u] *= by;
    }
    if (STATES) {
        float *seg = seg_of(pl.slot0 + (uint32_t)(pl.lo / set.seg_len));
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                *reinterpret_cast<f32x4 *>(seg + kk * 512 + 4 * u) = z[kk][u];
    } else if (sw.state_out && pl.last && col < n) {
        float *st = sw.state_out + sh * ((uint64_t)m * n) + col * sw.state_n;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = kk * 32 + e / 4 * 16 + 4 * g4 + e % 4;
                if (row < m)
                    st[row * sw.state_m] = z[kk][e / 4][e % 4];
            }
    }
}

template <class T, int D, bool VEC, int WP>
void run_split(const SweepSet &set, hipStream_t stream)
{
    const dim3 grid(set.items, set.heads, (unsigned)set.count);
    if (set.slots) {
        const dim3 cut(set.slots, set.heads, (unsigned)set.count);
        sweep_split_kernel<T, D, VEC, WP, true><<<cut, D * 4, 0, stream>>>(set);
        if (set.tokens > kFewSegments * set.seg_len)
            launch_segment_scan(set, D, stream);
    }
    sweep_split_kernel<T, D, VEC, WP, false><<<grid, D * 4, 0, stream>>>(set);
}

// Parts of the decayed rows: see "How exact".
template <class T, int D, bool VEC>
void split_of(const SweepSet &set, hipStream_t stream)
{
    if constexpr (sizeof(T) == 4) {
        run_split<T, D, VEC, 3>(set, stream);
    } else if constexpr (In<T>::kScaled) {
        run_split<T, D, VEC, 2>(set, stream);
    } else {
        bool states = false;
        for (int i = 0; i < set.count; ++i)
            states |= set.s[i].state_out != nullptr;
        if (states)
            run_split<T, D, VEC, 3>(set, stream);
        else
            run_split<T, D, VEC, 2>(set, stream);
    }
}

template <class T>
void split_by_width(const SweepSet &set, int width, hipStream_t stream)
{
    if (width == 64 && set.aligned)
        split_of<T, 64, true>(set, stream);
    else if (width == 64)
        split_of<T, 64, false>(set, stream);
    else if (set.aligned)
        split_of<T, 128, true>(set, stream);
    else
        split_of<T, 128, false>(set, stream);
}

}  // namespace

void launch_sweeps_split(const SweepSet &set, int width, hipStream_t stream)
{
    switch (set.dtype) {
    case LIBSCAN_F32: return split_by_width<float>(set, width, stream);
    case LIBSCAN_BF16: return split_by_width<__bf16>(set, width, stream);
    default: return split_by_width<_Float16>(set, width, stream);
    }
}

}  // namespace libscan
