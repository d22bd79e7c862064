// Shared parts of the kernels that norm rows: pieces of 8 consecutive values a lane, and their sums.
#pragma once

#include "layer.h"

namespace m3 {

constexpr int kNV = 8;    // consecutive values of a lane

// 8 values at any element: global memory takes loads and stores of 8 or 16 bytes there, in one
// instruction each, which rows of odd lengths (VEC false) use up to their last piece.
template <typename T> struct Loose8 { typedef T type __attribute__((ext_vector_type(8), aligned(sizeof(T)))); };

// 8 values of a row from column c on; zeros behind the row's end
template <typename T, bool VEC>
__device__ __forceinline__ void load8(float (&o)[kNV], const T *row, int c, int n) {
    if constexpr (VEC) {
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                const bf16x8 v = *(const bf16x8 *)(row + c);
#pragma unroll
                for (int e = 0; e < 8; e++) o[e] = to_f(v[e]);
            } else {
                const f32x4 a = *(const f32x4 *)(row + c), b = *(const f32x4 *)(row + c + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    o[e] = a[e];
                    o[e + 4] = b[e];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = 0.f;
        }
    } else if (c + 8 <= n) {
        const typename Loose8<T>::type v = *(const typename Loose8<T>::type *)(row + c);
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = to_f(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = c + e < n ? to_f(row[c + e]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int c, int n, const float (&o)[kNV]) {
    if constexpr (VEC) {
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                bf16x8 v;
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = from_f<bf16>(o[e]);
                *(bf16x8 *)(row + c) = v;
            } else {
                *(f32x4 *)(row + c) = f32x4{o[0], o[1], o[2], o[3]};
                *(f32x4 *)(row + c + 4) = f32x4{o[4], o[5], o[6], o[7]};
            }
        }
    } else if (c + 8 <= n) {
        typename Loose8<T>::type v;
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = from_f<T>(o[e]);
        *(typename Loose8<T>::type *)(row + c) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (c + e < n) row[c + e] = from_f<T>(o[e]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x141>(v);    // half-row mirror: the other quad of 8
    v += dpp_move<0x140>(v);    // row mirror: the other 8 of 16
    return sum_across_rows(v);
}
// Squares leave fp32's range long before the values do: a row whose mean square + eps is no number of
// [2^-98, infinity) is summed again with its values times a power of two, `row_scale` of that mean, which
// brings every finite row back inside, whatever its length (2^25 at most): below, 2^25 squares of a mean of 2^-98 scaled by
// 2^200 add up to 2^127, and one least subnormal value alone, squared and scaled, has a mean of 2^-123. At 2^-98
// unscaled squares that are subnormal or lost are 2^-28 of the mean at most.
constexpr float kLeastMean = 0x1p-98f;
__device__ __forceinline__ bool in_range(float mean) { return mean >= kLeastMean && mean < INFINITY; }
__device__ __forceinline__ float row_scale(float mean) { return mean < kLeastMean ? 0x1p100f : 0x1p-80f; }

// 8 values as loaded, converted where they are used: the next row's loads are in flight while a row is
// worked on.
template <typename T> struct Raw8 { typedef T type __attribute__((ext_vector_type(8), aligned(16))); };
template <typename T, bool VEC>
__device__ __forceinline__ typename Raw8<T>::type raw8(const T *row, int c, int n) {
    typename Raw8<T>::type v;
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = from_f<T>(0.f);
    if constexpr (VEC) {
        if (c < n) v = *(const typename Raw8<T>::type *)(row + c);
    } else if (c + 8 <= n) {
        v = *(const typename Loose8<T>::type *)(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (c + e < n) v[e] = row[c + e];
    }
    return v;
}

}  // namespace m3
