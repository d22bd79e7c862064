// Cache of recurrent states in 8 or 4 bits: states taken from a slot pool into cache entries, and back.
//
//   scale = max(max |value| of a block / top, 2^-126),  q = round(value / scale),  value = q scale
//
// One pass: a lane holds 16 bytes of consecutive values, a block 4 to 64 consecutive lanes, so that a block's largest
// value needs no memory. HBM-bound; a workgroup's index and load latencies are a good part of its life, which two
// pieces with their loads together share (64 states of 262144 fp32 values to 8 bits and back, with 1, 2, 4 pieces
// 43.8, 39.6, 41.8 us, 152 MB; 8 values a lane, 32 bytes apart, 40.4). Read back from 4 bits 15.9 us, 78 MB: 4.9 TB/s,
// a large copy's rate (a call among others 17).
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

constexpr int kCachePieces = 2;       // pieces of a workgroup
// Values of a lane, 16 bytes of them, and of a piece of a workgroup's
template <typename T> constexpr int cache_lane() { return 16 / sizeof(T); }
template <typename T> constexpr int cache_piece() { return 256 * cache_lane<T>(); }

constexpr float cache_top(int kind) { return kind == MAMBA3_CACHE_E4M3 ? 448.f : kind == MAMBA3_CACHE_INT8 ? 127.f : 7.f; }

template <typename T> struct CacheLane { typedef T type __attribute__((ext_vector_type(cache_lane<T>()), aligned(sizeof(T)))); };
// A lane's bytes at any place: 2, 4 or 8
template <int BYTES> struct CacheBytes;
template <> struct CacheBytes<2> { typedef uint16_t type __attribute__((aligned(1))); };
template <> struct CacheBytes<4> { typedef uint32_t type __attribute__((aligned(1))); };
template <> struct CacheBytes<8> { typedef uint64_t type __attribute__((aligned(1))); };

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

// A lane's q times their scale, in place, so that their rounding to the states' type is one of the exact product (of 31 bits
// at most). To bf16 the fp32 product stands for it but where that is the middle of two bf16: there an fp32 next to
// it on the product's side does, odd where it is not exact. (64 states of 262144 bf16 values to int8
// and back with every product in 64 bits 26.6 us, so 24.2, rounded by way of fp32 alone 23.6.)
template <typename T>
__device__ __forceinline__ void cache_products(float (&v)[cache_lane<T>()], float scale) {
    constexpr int L = cache_lane<T>();
    float q[L];
    bool middle = false;
#pragma unroll
    for (int e = 0; e < L; e++) {
        q[e] = v[e];
        v[e] *= scale;
        if (sizeof(T) == 2) middle |= (__float_as_uint(v[e]) & 0xffffu) == 0x8000u;
    }
    if (middle)
#pragma unroll
        for (int e = 0; e < L; e++) {
            const double exact = (double)q[e] * (double)scale;
            if ((double)v[e] != exact)
                v[e] = __uint_as_float((__float_as_uint(v[e]) - (fabs((double)v[e]) > fabs(exact) ? 1u : 0u)) | 1u);
        }
}

// A lane's values from value c of a state on; zeros behind its end
template <typename T>
__device__ __forceinline__ typename CacheLane<T>::type cache_values(const T *h, int c, int values) {
    constexpr int L = cache_lane<T>();
    typename CacheLane<T>::type x;
    if (c + L <= values) {
        x = *(const typename CacheLane<T>::type *)(h + c);
    } else {
#pragma unroll
        for (int e = 0; e < L; e++) x[e] = c + e < values ? h[c + e] : from_f<T>(0.f);
    }
    return x;
}

// A workgroup has kCachePieces pieces of a state, all of their loads in flight together.
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_state_store(CacheParams p) {
    constexpr int L = cache_lane<T>(), PIECE = cache_piece<T>(), U = kCachePieces;
    const int k = blockIdx.x / p.pieces, c0 = (blockIdx.x % p.pieces) * (U * PIECE) + threadIdx.x * L;
    int64_t slot, entry;
    if (!cache_row(p, k, slot, entry)) return;
    const T *h = (const T *)p.h + slot * p.values;
    typename CacheLane<T>::type x[U];
#pragma unroll
    for (int u = 0; u < U; u++) x[u] = cache_values(h, c0 + u * PIECE, p.values);
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = c0 + u * PIECE;
        float v[L], q[L];
        // magnitudes compare as integers, infinities and NaNs above all numbers
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < L; e++) {
            v[e] = to_f(x[u][e]);
            m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        for (int o = 1; o < p.block / L; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        const float top = __uint_as_float(m);
        float scale = fmaxf(top / cache_top(KIND), 0x1p-126f);
        if (m >= 0x7f800000u) scale = NAN;
        const float up = scale < 0x1p-60f ? 0x1p64f : 1.f, s = scale * up, r = 1.f / s;
#pragma unroll
        for (int e = 0; e < L; e++) {
            q[e] = cache_quotient(v[e] * up, s, r);
            if (KIND != MAMBA3_CACHE_E4M3) q[e] = fminf(fmaxf(rintf(q[e]), -cache_top(KIND)), cache_top(KIND));
        }
        if (c >= p.values) return;
        if (c % p.block == 0) p.scale[entry * p.blocks + c / p.block] = scale;
        uint32_t w[2] = {0, 0};
        if constexpr (KIND == MAMBA3_CACHE_E4M3) {
#pragma unroll
            for (int e = 0; e < L; e += 4) {
                const int low = __builtin_amdgcn_cvt_pk_fp8_f32(q[e], q[e + 1], 0, false);
                w[e >> 2] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[e + 2], q[e + 3], low, true);
            }
        } else if constexpr (KIND == MAMBA3_CACHE_INT8) {
#pragma unroll
            for (int e = 0; e < L; e++) w[e >> 2] |= ((uint32_t)(int)q[e] & 255u) << (8 * (e & 3));
        } else {
#pragma unroll
            for (int e = 0; e < L; e++) w[0] |= ((uint32_t)(int)q[e] & 15u) << (4 * e);
        }
        constexpr int PER = KIND == MAMBA3_CACHE_INT4 ? 2 : 1;      // values of a byte
        typedef typename CacheBytes<L / PER>::type bytes;
        uint8_t *to = p.q + entry * p.q_row + c / PER;
        if (c + L <= p.values) {
            *(bytes *)to = (bytes)((uint64_t)w[1] << 32 | w[0]);
        } else {
#pragma unroll
            for (int e = 0; e < L / PER; e++)
                if (c + e * PER < p.values) to[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
        }
    }
}

template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_state_load(CacheParams p) {
    constexpr int L = cache_lane<T>(), PIECE = cache_piece<T>(), U = kCachePieces, PER = KIND == MAMBA3_CACHE_INT4 ? 2 : 1;
    typedef typename CacheBytes<L / PER>::type bytes;
    const int k = blockIdx.x / p.pieces, c0 = (blockIdx.x % p.pieces) * (U * PIECE) + threadIdx.x * L;
    int64_t slot, entry;
    if (!cache_row(p, k, slot, entry)) return;
    uint64_t raw[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = c0 + u * PIECE;
        const uint8_t *from = p.q + entry * p.q_row + c / PER;
        raw[u] = 0;
        scale[u] = c < p.values ? p.scale[entry * p.blocks + c / p.block] : 0.f;
        if (c + L <= p.values) {
            raw[u] = *(const bytes *)from;
        } else {
#pragma unroll
            for (int e = 0; e < L / PER; e++)
                if (c + e * PER < p.values) raw[u] |= (uint64_t)from[e] << (8 * e);
        }
    }
    T *h = (T *)p.h + slot * p.values;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = c0 + u * PIECE;
        const uint32_t w[2] = {(uint32_t)raw[u], (uint32_t)(raw[u] >> 32)};
        float v[L];
        if constexpr (KIND == MAMBA3_CACHE_E4M3) {
#pragma unroll
            for (int e = 0; e < L; e += 4) {
                const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[e >> 2], false);
                const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[e >> 2], true);
                v[e] = a[0];
                v[e + 1] = a[1];
                v[e + 2] = b[0];
                v[e + 3] = b[1];
            }
        } else if constexpr (KIND == MAMBA3_CACHE_INT8) {
#pragma unroll
            for (int e = 0; e < L; e++) v[e] = (float)(int8_t)(w[e >> 2] >> (8 * (e & 3)));
        } else {
#pragma unroll
            for (int e = 0; e < L; e++) v[e] = (float)((int32_t)(w[0] << (28 - 4 * e)) >> 28);
        }
        cache_products<T>(v, scale[u]);
        if (c + L <= p.values) {
            typename CacheLane<T>::type o;
#pragma unroll
            for (int e = 0; e < L; e++) o[e] = from_f<T>(v[e]);
            *(typename CacheLane<T>::type *)(h + c) = o;
        } else {
#pragma unroll
            for (int e = 0; e < L; e++)
                if (c + e < p.values) h[c + e] = from_f<T>(v[e]);
        }
    }
}

// Values of a workgroup
static int cache_span(int32_t dtype) { return kCachePieces * (dtype == MAMBA3_F32 ? cache_piece<float>() : cache_piece<bf16>()); }

int64_t state_cache_workgroups(const mamba3_state_cache_args *a) {
    const int64_t span = cache_span(a->dtype);
    return a->n * ((a->values + span - 1) / span);
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
    const int span = cache_span(a->dtype);
    p.pieces = (a->values + span - 1) / span;
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
