// Cache of recurrent states in 8 or 4 bits: states taken from a slot pool into cache entries, and back.
//
//   scale = max(max |value| of a block / top, 2^-126),  q = round(value / scale),  value = q scale
//
// One pass: a lane holds 8 consecutive values, a block 4 to 32 consecutive lanes, so that a block's largest value
// needs no memory. HBM-bound.
#include "layer.h"

namespace m3 {

struct CacheParams {
    void *h;
    uint8_t *q;
    float *scale;
    const int32_t *slots, *entries;
    int64_t q_row;                  // bytes of an entry
    int32_t values, block, blocks, pieces, nslots, nentries;
};

constexpr int kCacheLane = 8, kCachePiece = 256 * kCacheLane;    // values of a lane, of a workgroup

constexpr float cache_top(int kind) { return kind == MAMBA3_CACHE_E4M3 ? 448.f : kind == MAMBA3_CACHE_INT8 ? 127.f : 7.f; }

template <typename T> struct Eight { typedef T type __attribute__((ext_vector_type(8), aligned(sizeof(T)))); };
typedef uint32_t loose2 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t loose1 __attribute__((ext_vector_type(1), aligned(1)));

// The row of this workgroup: its slot and entry, false where either is out of range
__device__ __forceinline__ bool cache_row(const CacheParams &p, int k, int64_t &slot, int64_t &entry) {
    slot = p.slots ? p.slots[k] : k;
    entry = p.entries ? p.entries[k] : k;
    return slot >= 0 && slot < p.nslots && entry >= 0 && entry < p.nentries;
}

// The quotient rounded to fp32, as a division does: from the rounded reciprocal two corrections by the remainder,
// which a fused multiply-add gives exactly, settle the last place. Values and scale are brought up by a power
// of two where the remainder would be subnormal.
__device__ __forceinline__ float cache_quotient(float v, float scale, float r) {
    float q = v * r;
    q = fmaf(fmaf(-scale, q, v), r, q);
    return fmaf(fmaf(-scale, q, v), r, q);
}

template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_state_store(CacheParams p) {
    const int k = blockIdx.x / p.pieces, c = (blockIdx.x % p.pieces) * kCachePiece + threadIdx.x * kCacheLane;
    int64_t slot, entry;
    if (!cache_row(p, k, slot, entry)) return;
    const T *h = (const T *)p.h + slot * p.values;
    float v[kCacheLane];
    if (c + kCacheLane <= p.values) {
        const typename Eight<T>::type x = *(const typename Eight<T>::type *)(h + c);
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) v[e] = to_f(x[e]);
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) v[e] = c + e < p.values ? to_f(h[c + e]) : 0.f;
    }
    // magnitudes compare as integers, infinities and NaNs above all numbers
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kCacheLane; e++) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    for (int o = 1; o < p.block / kCacheLane; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    const float top = __uint_as_float(m);
    float scale = fmaxf(top / cache_top(KIND), 0x1p-126f);
    if (m >= 0x7f800000u) scale = NAN;
    const float up = scale < 0x1p-60f ? 0x1p64f : 1.f, s = scale * up, r = 1.f / s;
    float q[kCacheLane];
#pragma unroll
    for (int e = 0; e < kCacheLane; e++) {
        q[e] = cache_quotient(v[e] * up, s, r);
        if (KIND != MAMBA3_CACHE_E4M3) q[e] = fminf(fmaxf(rintf(q[e]), -cache_top(KIND)), cache_top(KIND));
    }
    if (c >= p.values) return;
    if (c % p.block == 0) p.scale[entry * p.blocks + c / p.block] = scale;
    uint32_t w[2] = {0, 0};
    if constexpr (KIND == MAMBA3_CACHE_E4M3) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            int t = 0;
            t = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * j], q[4 * j + 1], t, false);
            t = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * j + 2], q[4 * j + 3], t, true);
            w[j] = (uint32_t)t;
        }
    } else if constexpr (KIND == MAMBA3_CACHE_INT8) {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) w[e >> 2] |= ((uint32_t)(int)q[e] & 255u) << (8 * (e & 3));
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) w[0] |= ((uint32_t)(int)q[e] & 15u) << (4 * e);
    }
    constexpr int PER = KIND == MAMBA3_CACHE_INT4 ? 2 : 1;      // values of a byte
    uint8_t *to = p.q + entry * p.q_row + c / PER;
    if (c + kCacheLane <= p.values) {
        if constexpr (PER == 2) *(loose1 *)to = loose1{w[0]};
        else *(loose2 *)to = loose2{w[0], w[1]};
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane / PER; e++)
            if (c + e * PER < p.values) to[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}

template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_state_load(CacheParams p) {
    const int k = blockIdx.x / p.pieces, c = (blockIdx.x % p.pieces) * kCachePiece + threadIdx.x * kCacheLane;
    int64_t slot, entry;
    if (!cache_row(p, k, slot, entry) || c >= p.values) return;
    constexpr int PER = KIND == MAMBA3_CACHE_INT4 ? 2 : 1;
    const uint8_t *from = p.q + entry * p.q_row + c / PER;
    const float scale = p.scale[entry * p.blocks + c / p.block];
    uint32_t w[2] = {0, 0};
    const bool whole = c + kCacheLane <= p.values;
    if (whole) {
        if constexpr (PER == 2) {
            w[0] = (*(const loose1 *)from)[0];
        } else {
            const loose2 b = *(const loose2 *)from;
            w[0] = b[0];
            w[1] = b[1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane / PER; e++)
            if (c + e * PER < p.values) w[e >> 2] |= (uint32_t)from[e] << (8 * (e & 3));
    }
    float v[kCacheLane];
    if constexpr (KIND == MAMBA3_CACHE_E4M3) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
            v[4 * j] = a[0];
            v[4 * j + 1] = a[1];
            v[4 * j + 2] = b[0];
            v[4 * j + 3] = b[1];
        }
    } else if constexpr (KIND == MAMBA3_CACHE_INT8) {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) v[e] = (float)(int8_t)(w[e >> 2] >> (8 * (e & 3)));
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) v[e] = (float)((int32_t)(w[0] << (28 - 4 * e)) >> 28);
    }
    T *h = (T *)p.h + slot * p.values;
    if (whole) {
        typename Eight<T>::type o;
#pragma unroll
        for (int e = 0; e < kCacheLane; e++) o[e] = from_f<T>(v[e] * scale);
        *(typename Eight<T>::type *)(h + c) = o;
    } else {
#pragma unroll
        for (int e = 0; e < kCacheLane; e++)
            if (c + e < p.values) h[c + e] = from_f<T>(v[e] * scale);
    }
}

int64_t state_cache_workgroups(const mamba3_state_cache_args *a) {
    return (int64_t)a->n * (((int64_t)a->values + kCachePiece - 1) / kCachePiece);
}

template <typename T, int KIND>
static void cache_go(const CacheParams &p, bool store, const dim3 grid, hipStream_t st) {
    if (store) hipLaunchKernelGGL((k_state_store<T, KIND>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((k_state_load<T, KIND>), grid, dim3(256), 0, st, p);
}

mamba3_status launch_state_cache(const mamba3_state_cache_args *a, bool store, hipStream_t st) {
    CacheParams p{};
    p.h = a->h; p.q = (uint8_t *)a->q; p.scale = a->scale;
    p.slots = a->slots; p.entries = a->entries;
    p.values = a->values; p.block = a->block;
    p.blocks = (a->values + a->block - 1) / a->block;
    p.pieces = (a->values + kCachePiece - 1) / kCachePiece;
    p.nslots = a->nslots; p.nentries = a->nentries;
    p.q_row = a->kind == MAMBA3_CACHE_INT4 ? ((int64_t)a->values + 1) / 2 : a->values;
    const dim3 grid((uint32_t)state_cache_workgroups(a));
    const bool f32 = a->dtype == MAMBA3_F32;
#define M3_GO(KIND)                                           \
    do {                                                      \
        if (f32) cache_go<float, KIND>(p, store, grid, st);   \
        else cache_go<bf16, KIND>(p, store, grid, st);        \
    } while (0)
    if (a->kind == MAMBA3_CACHE_E4M3) M3_GO(MAMBA3_CACHE_E4M3);
    else if (a->kind == MAMBA3_CACHE_INT8) M3_GO(MAMBA3_CACHE_INT8);
    else M3_GO(MAMBA3_CACHE_INT4);
#undef M3_GO
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
