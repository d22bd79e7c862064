// Shared parts of the selective scan's forward and backward kernels.
//
// A wave holds CW = 64 / LPC channels, LPC consecutive lanes a channel with NPL states each
// (N <= NPL * LPC; states behind N stay zero). Lane l: channel l / LPC, states (l % LPC) * NPL ..
#pragma once

#include "layer.h"

namespace m3 {

constexpr int kSelWaves = 4;         // waves of a workgroup; each works by itself on CW channels
constexpr int kSelTile = 16;         // tokens staged at once

struct SelParams {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    const float *h_in;
    void *y;
    float *h_out;
    int64_t x_row, dt_row, B_row, C_row, z_row;   // elements from one token to the next
    const int32_t *cu;       // packed batches, or NULL
    int32_t nseq;            // sequences (padded: the batch)
    int32_t seqlen, total;   // tokens of a padded sequence, tokens of the batch
    int32_t dim, dpg, N, G;  // channels, channels of a B/C group, states a channel, groups
    int32_t tiles;           // workgroups that cover a group's channels
    int32_t softplus;
    float *ckpt;             // the states before every tile of a row (the backward's first pass), or NULL
};

// A row of tokens that one workgroup walks: [t0, t1) of sequence seq.
struct SelRow {
    int t0, t1, seq;
};

__device__ __forceinline__ SelRow sel_row(const SelParams &p, int r) {
    SelRow o;
    o.seq = r;
    if (p.cu) {
        packed_bounds(p.cu, r, p.total, o.t0, o.t1);
    } else {
        o.t0 = r * p.seqlen;
        o.t1 = o.t0 + p.seqlen;
    }
    return o;
}

// Tokens between two stored states: as many as the backward keeps in registers (64 states a lane).
template <int NPL> constexpr int kSelStored = 64 / NPL;
// The stored states of a row that starts at token t0 begin at this index (a row of len tokens takes
// ceil(len / every) of them, at most len / every + 1, so that rows never overlap).
__device__ __forceinline__ int64_t stored_base(const SelRow &row, int every) { return row.t0 / every + row.seq; }
// The lane's place in stored state k: workgroup column gt of `per`, four states of 64 lanes together.
__device__ __forceinline__ int64_t stored_at(int64_t k, int per, int gt, int wave, int lane, int npl) {
    return (((k * per + gt) * kSelWaves + wave) * (npl / 4)) * 256 + lane * 4;
}

// NPL states of a channel from / to a row of N states, n0 the lane's first. VEC: N is a multiple of 4
// and the row 16-byte aligned.
template <int NPL, bool VEC>
__device__ __forceinline__ void load_states(float (&h)[NPL], const float *row, int n0, int N) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (n0 + i < N) v = *(const f32x4 *)(row + n0 + i);
#pragma unroll
            for (int e = 0; e < 4; e++) h[i + e] = v[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; i++) h[i] = n0 + i < N ? row[n0 + i] : 0.f;
    }
}
template <int NPL, bool VEC>
__device__ __forceinline__ void store_states(const float (&h)[NPL], float *row, int n0, int N) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4)
            if (n0 + i < N) *(f32x4 *)(row + n0 + i) = f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            if (n0 + i < N) row[n0 + i] = h[i];
    }
}

// The lane arrangement of N states: as few lanes a channel as leave 4 or 8 states a lane.
#define M3_SEL_DISPATCH(N, CALL)              \
    do {                                      \
        if ((N) <= 4) CALL(4, 1);             \
        else if ((N) <= 8) CALL(4, 2);        \
        else if ((N) <= 16) CALL(4, 4);       \
        else if ((N) <= 32) CALL(8, 4);       \
        else if ((N) <= 64) CALL(8, 8);       \
        else CALL(8, 16);                     \
    } while (0)

SelParams sel_params(const mamba3_selective_scan_args *a);
bool sel_vec(const SelParams &p, int64_t es);
// Enqueue the scan that writes p.ckpt and no outputs.
void launch_sel_stored(const SelParams &p, int32_t dtype, bool vec, hipStream_t st);

}  // namespace m3
