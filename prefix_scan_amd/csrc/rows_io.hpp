// rows_io.hpp -- rows of f32, bf16 and f16 elements, 16 bytes of a lane at a
// time, as floats.
//
// A piece is whole (one access of 16 bytes, at any alignment of the element:
// the memory system splits what crosses a line) or cut short by the row's end.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libscan {

typedef uint32_t piece_t __attribute__((ext_vector_type(4)));

template <class T>
constexpr int kPiece = 16 / (int)sizeof(T);      // elements of a piece

// The first n elements at `at` (all, for n >= kPiece), zeros behind them.  A
// piece cut short is put together of 8, 4 and 2 bytes.
template <class T>
__device__ __forceinline__ piece_t load_piece(const T *at, int n)
{
    piece_t r = {0, 0, 0, 0};
    if (n >= kPiece<T>) {
        __builtin_memcpy(&r, at, sizeof(r));
        return r;
    }
    const uint16_t *from = reinterpret_cast<const uint16_t *>(at);
    const int units = n > 0 ? n * (int)(sizeof(T) / 2) : 0;   // of two bytes
    uint32_t one = 0, two[2] = {0, 0};
    if (units & 4) {
        __builtin_memcpy(two, from, 8);
        r[0] = two[0];
        r[1] = two[1];
        from += 4;
    }
    if (units & 2) {
        __builtin_memcpy(&one, from, 4);
        r[0] = units & 4 ? r[0] : one;
        r[2] = units & 4 ? one : 0;
        from += 2;
    }
    if (sizeof(T) == 2 && (units & 1)) {
        const uint32_t last = *from;
        r[0] = units < 2 ? last : r[0];
        r[1] = (units & 6) == 2 ? last : r[1];
        r[2] = (units & 6) == 4 ? last : r[2];
        r[3] = (units & 6) == 6 ? last : 0;
    }
    return r;
}

template <class T>
__device__ __forceinline__ void store_piece(T *at, piece_t r, int n)
{
    if (n >= kPiece<T>) {
        __builtin_memcpy(at, &r, sizeof(r));
        return;
    }
    uint16_t *to = reinterpret_cast<uint16_t *>(at);
    const int units = n > 0 ? n * (int)(sizeof(T) / 2) : 0;
    if (units & 4) {
        const uint32_t two[2] = {r[0], r[1]};
        __builtin_memcpy(to, two, 8);
        to += 4;
    }
    if (units & 2) {
        const uint32_t one = units & 4 ? r[2] : r[0];
        __builtin_memcpy(to, &one, 4);
        to += 2;
    }
    if (sizeof(T) == 2 && (units & 1))
        *to = (uint16_t)(units < 2 ? r[0] : (units & 6) == 2 ? r[1] : (units & 6) == 4 ? r[2] : r[3]);
}

// Whole pieces that are read or written once, past what the caches keep.
typedef uint32_t loose_t __attribute__((ext_vector_type(4), aligned(2)));

template <class T>
__device__ __forceinline__ piece_t load_piece_past(const T *at)
{
    return __builtin_nontemporal_load(reinterpret_cast<const loose_t *>(at));
}

template <class T>
__device__ __forceinline__ void store_piece_past(T *at, piece_t r)
{
    __builtin_nontemporal_store((loose_t)r, reinterpret_cast<loose_t *>(at));
}

typedef float pair_f32 __attribute__((ext_vector_type(2)));
typedef __bf16 pair_bf16 __attribute__((ext_vector_type(2)));
typedef _Float16 pair_f16 __attribute__((ext_vector_type(2)));

template <class T>
struct Unpack;

template <>
struct Unpack<float> {
    __device__ static __forceinline__ float get(const piece_t &r, int e)
    {
        const uint32_t w = r[e];        // a vector's element is no lvalue to cast from
        return __builtin_bit_cast(float, w);
    }
    __device__ static __forceinline__ piece_t pack(const float (&f)[4])
    {
        piece_t r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = __builtin_bit_cast(uint32_t, f[e]);
        return r;
    }
};

template <>
struct Unpack<__bf16> {
    __device__ static __forceinline__ float get(const piece_t &r, int e)
    {
        const uint32_t w = r[e / 2];
        return __builtin_bit_cast(float, e & 1 ? w & 0xFFFF0000u : w << 16);
    }
    __device__ static __forceinline__ piece_t pack(const float (&f)[8])
    {
        piece_t r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = __builtin_bit_cast(
                uint32_t, __builtin_convertvector((pair_f32){f[2 * e], f[2 * e + 1]}, pair_bf16));
        return r;
    }
};

template <>
struct Unpack<_Float16> {
    __device__ static __forceinline__ float get(const piece_t &r, int e)
    {
        return (float)__builtin_bit_cast(pair_f16, (uint32_t)r[e / 2])[e & 1];
    }
    __device__ static __forceinline__ piece_t pack(const float (&f)[8])
    {
        piece_t r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = __builtin_bit_cast(
                uint32_t, __builtin_convertvector((pair_f32){f[2 * e], f[2 * e + 1]}, pair_f16));
        return r;
    }
};

// Four elements, of 8 or 16 bytes, the first n of them.
template <class T>
struct Four {
    uint32_t w[sizeof(T)] = {};
    __device__ __forceinline__ float get(int e) const
    {
        piece_t r = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i)
            r[i] = w[i];
        return Unpack<T>::get(r, e);
    }
    __device__ static __forceinline__ Four of(const float (&f)[4])
    {
        float g[kPiece<T>] = {f[0], f[1], f[2], f[3]};
        const piece_t r = Unpack<T>::pack(g);
        Four x;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i)
            x.w[i] = r[i];
        return x;
    }
};

template <class T>
__device__ __forceinline__ Four<T> load_four(const T *at, int n)
{
    Four<T> x;
    if (n >= 4) {
        __builtin_memcpy(x.w, at, sizeof(x.w));
        return x;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        if (e < n) {
            if (sizeof(T) == 4)
                x.w[e] = reinterpret_cast<const uint32_t *>(at)[e];
            else
                x.w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(at)[e] << (16 * (e & 1));
        }
    }
    return x;
}

template <class T>
__device__ __forceinline__ void store_four(T *at, const Four<T> &x, int n)
{
    if (n >= 4) {
        __builtin_memcpy(at, x.w, sizeof(x.w));
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        if (e < n) {
            if (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(at)[e] = x.w[e];
            else
                reinterpret_cast<uint16_t *>(at)[e] = (uint16_t)(x.w[e / 2] >> (16 * (e & 1)));
        }
    }
}

// V consecutive floats (states), the first n of them.
template <int V>
__device__ __forceinline__ void load_floats(const float *at, int n, float (&f)[V])
{
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
        const piece_t r = load_piece<float>(at + 4 * q, n - 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[4 * q + e] = Unpack<float>::get(r, e);
    }
}

template <int V>
__device__ __forceinline__ void store_floats(float *at, int n, const float (&f)[V])
{
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
        store_piece<float>(at + 4 * q, Unpack<float>::pack({f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]}),
                           n - 4 * q);
}

}  // namespace libscan
