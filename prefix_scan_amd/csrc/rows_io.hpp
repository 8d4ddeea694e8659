// rows_io.hpp -- rows of f32, bf16 and f16 elements, 16 bytes of a lane at a
// time, as floats.
//
// A piece is whole (one access of 16 bytes, at any alignment of the element:
// the memory system splits what crosses a line) or cut short by the row's end
// (element by element).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libscan {

typedef uint32_t piece_t __attribute__((ext_vector_type(4)));

template <class T>
constexpr int kPiece = 16 / (int)sizeof(T);      // elements of a piece

// The first n elements at `at` (all, for n >= kPiece), zeros behind them.
template <class T>
__device__ __forceinline__ piece_t load_piece(const T *at, int n)
{
    piece_t r = {0, 0, 0, 0};
    if (n >= kPiece<T>) {
        __builtin_memcpy(&r, at, sizeof(r));
        return r;
    }
#pragma unroll
    for (int e = 0; e < kPiece<T>; ++e) {
        if (e < n) {
            if (sizeof(T) == 4) {
                r[e & 3] = reinterpret_cast<const uint32_t *>(at)[e];
            } else {
                const uint32_t w = reinterpret_cast<const uint16_t *>(at)[e];
                r[(e / 2) & 3] |= w << (16 * (e & 1));
            }
        }
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
#pragma unroll
    for (int e = 0; e < kPiece<T>; ++e) {
        if (e < n) {
            if (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(at)[e] = r[e & 3];
            else
                reinterpret_cast<uint16_t *>(at)[e] = (uint16_t)(r[(e / 2) & 3] >> (16 * (e & 1)));
        }
    }
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
