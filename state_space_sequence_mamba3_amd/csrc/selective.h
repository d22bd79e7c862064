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
    // Rows: a sequence each (nseg 1), or its segments of seg_tokens tokens: nseg a sequence of a padded
    // batch, or those of the table of a packed one.
    int32_t rows, nseg, seg_tokens;
    const int4 *table;       // t0, t1, sequence (-1: no segment), 1 first | 2 last of its sequence
    const int32_t *seq_row;  // [nseq + 1] a sequence's first row in the table
    float *seg_h;            // [rows][D][N] a segment's last state from zero, then the state entering it
    float *seg_s;            // [rows][D] the sum of a segment's steps
    // the backward's first pass
    const void *dy;
    int64_t dy_row;
    float *seg_g;            // [rows][D][N] the segment's share of the gradient that enters the one before,
                             // then the gradient that enters the segment at its end
    float *ckpt;             // the states before every tile of a row
    float *ckpt_s;           // the sums of the steps before them (segments only)
};

// A row of tokens that one workgroup walks: [t0, t1) of sequence seq.
struct SelRow {
    int t0, t1, seq;
    bool first, last;
};

__device__ __forceinline__ SelRow sel_row_of(const SelParams &p, int r) {
    SelRow o;
    o.first = o.last = true;
    if (p.table) {
        const int4 e = p.table[r];
        o.t0 = e.x;
        o.t1 = e.y;
        o.seq = e.z;
        o.first = e.w & 1;
        o.last = e.w & 2;
    } else if (p.cu) {
        o.seq = r;
        packed_bounds(p.cu, r, p.total, o.t0, o.t1);
    } else {
        const int k = r % p.nseg, a = r / p.nseg * p.seqlen;
        o.seq = r / p.nseg;
        o.t0 = a + min(k * p.seg_tokens, p.seqlen);
        o.t1 = min(o.t0 + min(p.seg_tokens, p.seqlen), a + p.seqlen);
        o.first = k == 0;
        o.last = k == p.nseg - 1;
    }
    return o;
}

// The same, in scalar registers
__device__ __forceinline__ SelRow sel_row(const SelParams &p, int r) {
    SelRow o = sel_row_of(p, r);
    o.t0 = __builtin_amdgcn_readfirstlane(o.t0);
    o.t1 = __builtin_amdgcn_readfirstlane(o.t1);
    o.seq = __builtin_amdgcn_readfirstlane(o.seq);
    o.first = __builtin_amdgcn_readfirstlane(o.first);
    o.last = __builtin_amdgcn_readfirstlane(o.last);
    return o;
}

// Tokens between two states that the backward's first pass stores: its second pass computes the states
// and decays between them again and keeps both in registers, 4 or 8 of each a lane and token.
constexpr int kSelStored = 8;
// The stored states of row r begin at this index (a row of len tokens takes ceil(len / every) of them,
// at most len / every + 1, so that rows, which lie in the order of their tokens, never overlap).
__device__ __forceinline__ int64_t stored_base(int t0, int r, int every) { return (int64_t)t0 / every + r; }
// The lane's place in stored state k: workgroup column gt of `per`, four states of 64 lanes together.
__device__ __forceinline__ int64_t stored_at(int64_t k, int per, int gt, int wave, int lane, int npl) {
    return (((k * per + gt) * kSelWaves + wave) * (npl / 4)) * 256 + lane * 4;
}

// 2^v h, v the exponent of many steps together. A state may grow (s A > 0) by more than fp32's range while h
// is zero or tiny: two factors of 2^(v/2), held finite, give h 2^v wherever that is in range, and zero for
// zero.
__device__ __forceinline__ float carried(float v, float h) {
    const float e = fminf(__builtin_amdgcn_exp2f(0.5f * v), 3.40282347e38f);
    return h * e * e;
}

// NPL states of a channel from / to a row of N states, n0 the lane's first. VEC: N is a multiple of 4
// and the row 16-byte aligned; else a row's last one to three states are taken one by one.
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
        for (int i = 0; i < NPL; i += 4) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (n0 + i + 4 <= N) {
                v = *(const LooseQuad<float>::type *)(row + n0 + i);
            } else {
#pragma unroll
                for (int e = 0; e < 3; e++)
                    if (n0 + i + e < N) v[e] = row[n0 + i + e];
            }
#pragma unroll
            for (int e = 0; e < 4; e++) h[i + e] = v[e];
        }
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
        for (int i = 0; i < NPL; i += 4) {
            if (n0 + i + 4 <= N) {
                *(LooseQuad<float>::type *)(row + n0 + i) = f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < 3; e++)
                    if (n0 + i + e < N) row[n0 + i + e] = h[i + e];
            }
        }
    }
}

// The lane arrangement of N states: as few lanes a channel as leave 4 or 8 states a lane. The backward
// keeps the states and decays of 8 tokens, and with 8 states a lane that takes more than 256
// registers, one wave a SIMD at half its rate: it takes 4 a lane up to 64 states (see k_selbwd for what
// that leaves).
#define M3_SEL_DISPATCH(N, CALL)              \
    do {                                      \
        if ((N) <= 4) CALL(4, 1);             \
        else if ((N) <= 8) CALL(4, 2);        \
        else if ((N) <= 16) CALL(4, 4);       \
        else if ((N) <= 32) CALL(8, 4);       \
        else if ((N) <= 64) CALL(8, 8);       \
        else CALL(8, 16);                     \
    } while (0)
#define M3_SELBWD_DISPATCH(N, CALL)           \
    do {                                      \
        if ((N) <= 4) CALL(4, 1);             \
        else if ((N) <= 8) CALL(4, 2);        \
        else if ((N) <= 16) CALL(4, 4);       \
        else if ((N) <= 32) CALL(4, 8);       \
        else if ((N) <= 64) CALL(4, 16);      \
        else CALL(8, 16);                     \
    } while (0)

// Lanes a channel and states a lane of the arrangement above.
inline void sel_shape(int N, bool back, int &npl, int &lpc) {
#define M3_GO(NPL, LPC) npl = NPL, lpc = LPC
    if (back) M3_SELBWD_DISPATCH(N, M3_GO);
    else M3_SEL_DISPATCH(N, M3_GO);
#undef M3_GO
}

SelParams sel_params(const mamba3_selective_scan_args *a);
Access sel_access(const SelParams &p, int64_t es);
// Rows of a call (p.rows, nseg, seg_tokens): whole sequences, or segments where those leave the GPU
// empty. True if segments; they need seg_bytes of workspace for the parts that `sel_segments` lays out.
bool sel_plan(SelParams &p, bool back);
// Workgroups of the backward's last launch: dB and dC, and the sums over rows.
inline int64_t sel_reduce_blocks(const SelParams &p) { return ((int64_t)p.total * p.G * 2 * p.N + 255) / 256; }
inline int64_t sel_sum_blocks(const SelParams &p) { return ((int64_t)p.dim * (p.N + 2) + 255) / 256; }
size_t sel_segment_bytes(const SelParams &p);
void sel_segments(SelParams &p, char *ws);
// Enqueue: a packed batch's segment table; the scan that writes p.ckpt (and segments' ends) and no
// outputs; the chain over the segments of a sequence, forward and (p.seg_g) backward.
void launch_sel_table(const SelParams &p, hipStream_t st);
void launch_sel_stored(const SelParams &p, int32_t dtype, Access acc, hipStream_t st);
void launch_sel_chain(const SelParams &p, const float *dh_out, hipStream_t st);

}  // namespace m3
