// Shared device helpers of the layer operators (short convolution, selective scan, residual RMS norm).
#pragma once

#include "m3_common.h"

namespace m3 {

// Four consecutive elements of a token array as one load (8 bytes of bf16, 16 of fp32).
template <typename T> struct QuadOf;
template <> struct QuadOf<float> { typedef f32x4 type; };
template <> struct QuadOf<bf16> { typedef bf16x4 type; };
template <typename T> using quad = typename QuadOf<T>::type;

// How a kernel reads rows of token arrays in fours. ALIGNED: rows of a multiple of 4 elements, every
// quad aligned to its size. ANY: rows of 4 elements or more, any length and alignment (global memory
// takes a load of 8 or 16 bytes at any element); the quad that crosses a row's end is loaded from
// its last 4 elements and shifted. ONE: rows of any length, element by element.
enum Access { ONE, ANY, ALIGNED };
// How the rows of B and C are read, N elements of a token and group: N may be below 4 where a lane holds
// all states of a channel.
constexpr Access states_access(Access acc, int lpc) { return acc == ANY && lpc == 1 ? ONE : acc; }

// A token number that is the same for all lanes, in a scalar register and unknown to the compiler, which
// would otherwise carry each lane's 64-bit addresses from tile to tile and add to every one of them.
__device__ __forceinline__ int64_t scalar_token(int t) {
    t = __builtin_amdgcn_readfirstlane(t);
    asm("" : "+s"(t));
    return t;
}

template <typename T> struct LooseQuad { typedef T type __attribute__((ext_vector_type(4), aligned(sizeof(T)))); };

// Elements c0 .. c0 + 3 of row t behind `base` (rows of n elements, `row` apart). Places behind a row's
// end get other elements of the row or zero; their results are never stored. `base` is the same for
// all lanes and the offset has 32 bits, so that the load takes the address from scalar registers and
// an offset that does not change from tile to tile.
template <typename T, Access ACC>
__device__ __forceinline__ quad<T> load_quad(const T *base, int t, int64_t row, int c0, int n) {
    quad<T> v;
    const uint32_t r = t * (uint32_t)row;
    if constexpr (ACC == ALIGNED) {
        v = *(const quad<T> *)((const char *)base + (r + min(c0, n - 4)) * (uint32_t)sizeof(T));
    } else if constexpr (ACC == ANY) {
        typedef typename LooseQuad<T>::type loose;
        const int at = min(c0, n - 4), over = c0 - at;
        v = *(const loose *)((const char *)base + (r + at) * (uint32_t)sizeof(T));
        if (over & 1) v = quad<T>{v[1], v[2], v[3], from_f<T>(0.f)};
        if (over & 2) v = quad<T>{v[2], v[3], from_f<T>(0.f), from_f<T>(0.f)};
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            v[e] = *(const T *)((const char *)base + (r + min(c0 + e, n - 1)) * (uint32_t)sizeof(T));
    }
    return v;
}
template <typename T, Access ACC>
__device__ __forceinline__ void store_quad(T *base, int t, int64_t row, int c0, int n, f32x4 v) {
    T *to = (T *)((char *)base + (uint32_t)(t * (uint32_t)row + c0) * (uint32_t)sizeof(T));
    if (ACC == ALIGNED ? c0 < n : ACC == ANY && c0 + 4 <= n) {
        quad<T> o;
#pragma unroll
        for (int e = 0; e < 4; e++) o[e] = from_f<T>(v[e]);
        if (ACC == ALIGNED) *(quad<T> *)to = o;
        else *(typename LooseQuad<T>::type *)to = o;
    } else if (ACC != ALIGNED) {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (c0 + e < n) to[e] = from_f<T>(v[e]);
    }
}

// e^v, log(1 + e^v) and 1 / (1 + e^-v) on the hardware's exp2, log2 and reciprocal (about one unit
// in the last place each). log1p adds what 1 + e^v rounded away, over 1 + e^v (log(u + c) = log u +
// c / u for a c far below u): the step sizes of a layer lie where that is most of the value.
__device__ __forceinline__ float exp_hw(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }
__device__ __forceinline__ float softplus_hw(float v) {
    const float w = exp_hw(v), u = 1.f + w, c = w - (u - 1.f);
    const float l = fmaf(__builtin_amdgcn_logf(u), 0.69314718056f, c * __builtin_amdgcn_rcpf(u));
    return v > 20.f ? v : l;
}
__device__ __forceinline__ float sigmoid_hw(float v) { return __builtin_amdgcn_rcpf(1.f + exp_hw(-v)); }

// One wave's LDS traffic is in order: the barrier only keeps the compiler from moving accesses
// across it.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// DPP move into the lanes of `BANKS` (4-lane banks of every 16-lane row) of `keep`; the other lanes keep.
template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_into(float keep, float from) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(keep), __float_as_int(from), CTRL, 0xF, BANKS, false));
}

// K values a lane, summed over each group of K consecutive lanes; lane i of a group gets the sum of
// value i. Every level halves the values: a lane keeps the half that its bit names and hands the
// other half to the lane across, so K values cost about 3 (K - 1) operations instead of K log2(K)
// additions and K selections.
template <int K>
__device__ __forceinline__ float transpose_sum(float (&p)[K], int lane) {
    static_assert(K == 1 || K == 2 || K == 4 || K == 8 || K == 16, "groups inside a 16-lane row");
    if constexpr (K >= 2) {
        const bool odd = lane & 1;
#pragma unroll
        for (int i = 0; i < K / 2; i++) {
            const float keep = odd ? p[2 * i + 1] : p[2 * i], send = odd ? p[2 * i] : p[2 * i + 1];
            p[i] = keep + dpp_move<0xB1>(send);                 // lane ^ 1
        }
    }
    if constexpr (K >= 4) {
        const bool up = lane & 2;
#pragma unroll
        for (int i = 0; i < K / 4; i++) {
            const float keep = up ? p[2 * i + 1] : p[2 * i], send = up ? p[2 * i] : p[2 * i + 1];
            p[i] = keep + dpp_move<0x4E>(send);                 // lane ^ 2
        }
    }
    if constexpr (K >= 8) {
#pragma unroll
        for (int i = 0; i < K / 8; i++) {                       // lane ^ 4: shifts by 4 into alternate banks
            const float a = p[2 * i], b = p[2 * i + 1];
            p[i] = dpp_into<0x104, 0x5>(b, a) + dpp_into<0x114, 0xA>(a, b);
        }
    }
    if constexpr (K >= 16) {                                    // lane ^ 8: a rotation of the row by 8
        const float a = p[0], b = p[1];
        p[0] = dpp_into<0x128, 0x3>(b, a) + dpp_into<0x128, 0xC>(a, b);
    }
    return p[0];
}

// Sequence s of a packed batch: its tokens [a, b), entries clamped to [0, total].
__device__ __forceinline__ void packed_bounds(const int32_t *cu, int s, int total, int &a, int &b) {
    a = min(max(cu[s], 0), total);
    b = min(max(cu[s + 1], a), total);
}

}  // namespace m3
