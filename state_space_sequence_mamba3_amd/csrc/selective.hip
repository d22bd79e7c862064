// Selective scan over whole sequences and its one-token step.
//
// Per sequence, channel d (B/C group g = d / (D/G)) and state n:
//   dt' = softplus(dt_t + bias_d)  (or dt_t + bias_d)
//   h_t[d,n] = exp(dt' A[d,n]) h_{t-1}[d,n] + dt' x_t[d] B_t[g,n]
//   y_t[d]   = (sum_n C_t[g,n] h_t[d,n] + D_d x_t[d]) SiLU(z_t[d])
// The decay differs for every channel and state, so nothing of it is a matrix product: the work is
// an exponential (two issue slots), two products and two fused adds for every token, channel and
// state, on the vector unit. Where N is 16 that is 96 slots for 8 bytes of bf16, so the vector
// unit and not the memory bounds the scan.
#include "selective.h"

namespace m3 {

// LDS of one wave: B and C rows and the pairs (dt', dt' x) of a tile's tokens in fp32, and its y.
template <int NP, int CW>
struct SelLds {
    float B[kSelTile][NP], C[kSelTile][NP];
    float u[kSelTile][CW][2];
    float y[kSelTile][CW];
};

// One workgroup: kSelWaves * CW channels of one group over one sequence's tokens, in tiles of 16.
// A tile's inputs are loaded into registers while the tile before is worked on (4 channels of one
// token a lane, so that a wave's load covers whole 32-byte pieces and the four waves of a
// workgroup whole 128-byte lines), prepared there (softplus, dt' x, fp32) and laid into the wave's
// own LDS; the recurrence then reads them as broadcasts. No wave waits for another.
//
// STORE: the backward's first pass. No outputs; the states before every kSelStored tokens go to p.ckpt.
template <typename T, int NPL, int LPC, bool VEC, bool STORE>
__global__ __launch_bounds__(64 * kSelWaves) void k_selscan(SelParams p) {
    constexpr int CW = 64 / LPC, NP = NPL * LPC, TT = kSelTile;
    constexpr int XQ = TT * CW / 4, XE = (XQ + 63) / 64;      // quads of a channel tile, and of a lane
    constexpr int BQ = TT * NP / 4, BE = (BQ + 63) / 64;
    __shared__ SelLds<NP, CW> lds[kSelWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    SelLds<NP, CW> &S = lds[wave];
    const int per = p.tiles * p.G;
    const int r = blockIdx.x / per, gt = blockIdx.x % per, g = gt / p.tiles;
    const int c0 = ((gt % p.tiles) * kSelWaves + wave) * CW;  // the wave's first channel in its group
    if (c0 >= p.dpg) return;
    const SelRow row = sel_row(p, r);
    const int ch = lane / LPC, sub = lane % LPC, n0 = sub * NPL;
    const bool real = c0 + ch < p.dpg;
    const int d = g * p.dpg + min(c0 + ch, p.dpg - 1);        // the lane's channel in the recurrence

    float A2[NPL], h[NPL];
    load_states<NPL, VEC>(A2, p.A + (int64_t)d * p.N, n0, p.N);
#pragma unroll
    for (int i = 0; i < NPL; i++) A2[i] *= kLog2e;
#pragma unroll
    for (int i = 0; i < NPL; i++) h[i] = 0.f;
    if (p.h_in) load_states<NPL, VEC>(h, p.h_in + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);

    // the lane's quads of a tile: token xt, channels xc .. xc + 3 of the group
    int xt[XE], xc[XE], bt[BE], bn[BE];
    f32x4 biasv[XE], Dv[XE];
#pragma unroll
    for (int i = 0; i < XE; i++) {
        const int q = min(lane + 64 * i, XQ - 1);
        xt[i] = q / (CW / 4);
        xc[i] = c0 + q % (CW / 4) * 4;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int dd = g * p.dpg + min(xc[i] + e, p.dpg - 1);
            biasv[i][e] = p.bias ? p.bias[dd] : 0.f;
            Dv[i][e] = p.D ? p.D[dd] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < BE; i++) {
        const int q = min(lane + 64 * i, BQ - 1);
        bt[i] = q / (NP / 4);
        bn[i] = q % (NP / 4) * 4;
    }
    const T *x = (const T *)p.x + g * p.dpg, *dt = (const T *)p.dt + g * p.dpg;
    const T *z = p.z && !STORE ? (const T *)p.z + g * p.dpg : nullptr;
    const T *B = (const T *)p.B + g * p.N, *C = (const T *)p.C + g * p.N;
    T *y = (T *)p.y + g * p.dpg;

    quad<T> rx[XE], rd[XE], rz[XE], rB[BE], rC[BE];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < XE; i++) {
            const int64_t t = min(t0 + xt[i], row.t1 - 1);
            rx[i] = load_quad<T, VEC>(x + t * p.x_row, xc[i], p.dpg);
            rd[i] = load_quad<T, VEC>(dt + t * p.dt_row, xc[i], p.dpg);
            if (z) rz[i] = load_quad<T, VEC>(z + t * p.z_row, xc[i], p.dpg);
        }
#pragma unroll
        for (int i = 0; i < BE; i++) {
            const int64_t t = min(t0 + bt[i], row.t1 - 1);
            rB[i] = load_quad<T, VEC>(B + t * p.B_row, bn[i], p.N);
            if (!STORE) rC[i] = load_quad<T, VEC>(C + t * p.C_row, bn[i], p.N);
        }
    };
    const int64_t stored = stored_base(row, kSelStored<NPL>);
    if (row.t0 < row.t1) fetch(row.t0);
    for (int t0 = row.t0; t0 < row.t1; t0 += TT) {
        f32x4 xv[XE], zv[XE];
#pragma unroll
        for (int i = 0; i < XE; i++) {
            f32x4 u[2];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                xv[i][e] = to_f(rx[i][e]);
                zv[i][e] = z ? to_f(rz[i][e]) : 0.f;
                float s = to_f(rd[i][e]) + biasv[i][e];
                if (p.softplus) s = softplus_hw(s);
                // a step of 0 behind the sequence's end keeps the state
                const bool in = t0 + xt[i] < row.t1;
                u[e >> 1][2 * (e & 1)] = in ? s : 0.f;
                u[e >> 1][2 * (e & 1) + 1] = in ? s * xv[i][e] : 0.f;
            }
            if (XQ % 64 == 0 || lane + 64 * i < XQ) {
                f32x4 *to = (f32x4 *)&S.u[xt[i]][xc[i] - c0][0];
                to[0] = u[0];
                to[1] = u[1];
            }
        }
#pragma unroll
        for (int i = 0; i < BE; i++) {
            if (BQ % 64 == 0 || lane + 64 * i < BQ) {
                f32x4 b, c;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    // places behind the last state or token hold zero, whatever lies there
                    const bool in = bn[i] + e < p.N && t0 + bt[i] < row.t1;
                    b[e] = in ? to_f(rB[i][e]) : 0.f;
                    c[e] = in && !STORE ? to_f(rC[i][e]) : 0.f;
                }
                *(f32x4 *)&S.B[bt[i]][bn[i]] = b;
                if (!STORE) *(f32x4 *)&S.C[bt[i]][bn[i]] = c;
            }
        }
        wave_lds_fence();
        if (t0 + TT < row.t1) fetch(t0 + TT);
#pragma unroll
        for (int tg = 0; tg < TT; tg += LPC) {
            float part[LPC];
#pragma unroll
            for (int j = 0; j < LPC; j++) {
                const int t = tg + j;
                if (STORE && t % kSelStored<NPL> == 0 && t0 + t < row.t1) {
                    float *to = p.ckpt + stored_at(stored + (t0 - row.t0 + t) / kSelStored<NPL>, per, gt, wave, lane, NPL);
#pragma unroll
                    for (int i = 0; i < NPL; i += 4)
                        *(f32x4 *)(to + i * 64) = f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]};
                }
                const float s = S.u[t][ch][0], u = S.u[t][ch][1];
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < NPL; i++) {
                    const float a = __builtin_amdgcn_exp2f(s * A2[i]);
                    h[i] = a * h[i] + u * S.B[t][n0 + i];
                    if (!STORE) acc += h[i] * S.C[t][n0 + i];
                }
                part[j] = acc;
            }
            if (!STORE) S.y[tg + sub][ch] = transpose_sum<LPC>(part, lane);
        }
        wave_lds_fence();
        if (STORE) continue;
#pragma unroll
        for (int i = 0; i < XE; i++) {
            const int t = t0 + xt[i];
            if ((XQ % 64 == 0 || lane + 64 * i < XQ) && t < row.t1) {
                f32x4 v = *(const f32x4 *)&S.y[xt[i]][xc[i] - c0];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[e] += Dv[i][e] * xv[i][e];
                    if (z) v[e] *= zv[i][e] * sigmoid_hw(zv[i][e]);
                }
                store_quad<T, VEC>(y + (int64_t)t * p.dim, xc[i], p.dpg, v);
            }
        }
        wave_lds_fence();
    }
    if (!STORE && p.h_out && real) store_states<NPL, VEC>(h, p.h_out + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);
}

// One token: LPC lanes a channel as in the scan; the states stream through once.
struct SelStepParams {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    float *h;
    void *y;
    int64_t x_row, dt_row, B_row, C_row, z_row;
    const int32_t *slots;
    int32_t nslots, dim, dpg, N, softplus;
};

template <typename T, int NPL, int LPC, bool VEC>
__global__ __launch_bounds__(256) void k_selstep(SelStepParams p, int tiles) {
    constexpr int CB = 256 / LPC;                       // channels of a workgroup
    const int b = blockIdx.x / tiles, d = (blockIdx.x % tiles) * CB + threadIdx.x / LPC;
    const int sub = threadIdx.x % LPC, n0 = sub * NPL;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nslots) return;       // inactive row (uniform across the workgroup)
    }
    if (d >= p.dim) return;                             // whole channels: a channel's lanes stay together
    float *hs = p.h + (slot * p.dim + d) * p.N;
    float h[NPL], A2[NPL];
    load_states<NPL, VEC>(h, hs, n0, p.N);
    load_states<NPL, VEC>(A2, p.A + (int64_t)d * p.N, n0, p.N);
    const int g = d / p.dpg;
    const T *B = (const T *)p.B + b * p.B_row + g * p.N, *C = (const T *)p.C + b * p.C_row + g * p.N;
    const float x = to_f(((const T *)p.x)[b * p.x_row + d]);
    float s = to_f(((const T *)p.dt)[b * p.dt_row + d]) + (p.bias ? p.bias[d] : 0.f);
    float Bv[NPL], Cv[NPL];
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
        const quad<T> bq = load_quad<T, VEC>(B, n0 + i, p.N), cq = load_quad<T, VEC>(C, n0 + i, p.N);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            Bv[i + e] = n0 + i + e < p.N ? to_f(bq[e]) : 0.f;
            Cv[i + e] = n0 + i + e < p.N ? to_f(cq[e]) : 0.f;
        }
    }
    if (p.softplus) s = softplus_hw(s);
    const float u = s * x;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        h[i] = exp_hw(s * A2[i]) * h[i] + u * Bv[i];
        acc += h[i] * Cv[i];
    }
    store_states<NPL, VEC>(h, hs, n0, p.N);
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) acc += __shfl_xor(acc, o, 64);
    if (sub == 0) {
        float v = acc + (p.D ? p.D[d] * x : 0.f);
        if (p.z) {
            const float z = to_f(((const T *)p.z)[b * p.z_row + d]);
            v *= z * sigmoid_hw(z);
        }
        ((T *)p.y)[(int64_t)b * p.dim + d] = from_f<T>(v);
    }
}

namespace {

int64_t dense(int64_t row, int64_t n) { return row ? row : n; }

bool quads(const void *q, int64_t row, int64_t es) { return ((uintptr_t)q % (4 * es)) == 0 && row % 4 == 0; }

}  // namespace

SelParams sel_params(const mamba3_selective_scan_args *a) {
    SelParams p{};
    const int64_t gn = (int64_t)a->ngroups * a->dstate;
    p.x = a->x; p.dt = a->dt; p.B = a->B; p.C = a->C; p.z = a->z;
    p.A = a->A; p.D = a->D; p.bias = a->dt_bias; p.h_in = a->h_in;
    p.y = a->y; p.h_out = a->h_out;
    p.x_row = dense(a->x_row, a->dim);
    p.dt_row = dense(a->dt_row, a->dim);
    p.z_row = dense(a->z_row, a->dim);
    p.B_row = dense(a->B_row, gn);
    p.C_row = dense(a->C_row, gn);
    p.cu = a->cu_seqlens;
    p.nseq = a->cu_seqlens ? a->nseq : a->batch;
    p.seqlen = a->seqlen;
    p.total = (int32_t)((int64_t)a->batch * a->seqlen);
    p.dim = a->dim; p.dpg = a->dim / a->ngroups; p.N = a->dstate; p.G = a->ngroups;
    p.softplus = a->dt_softplus;
    return p;
}

// Whether every row can be read in quads: channels of a group and states in fours, rows and
// pointers aligned to a quad. Otherwise every element is loaded by itself.
bool sel_vec(const SelParams &p, int64_t es) {
    return p.dpg % 4 == 0 && p.N % 4 == 0 && quads(p.x, p.x_row, es) && quads(p.dt, p.dt_row, es) &&
           quads(p.B, p.B_row, es) && quads(p.C, p.C_row, es) && quads(p.z, p.z_row, es) && quads(p.y, p.dim, es);
}

template <typename T, bool STORE>
static void scan_go(const SelParams &p0, bool vec, hipStream_t st) {
    SelParams p = p0;
#define M3_GO(NPL, LPC)                                                                                        \
    do {                                                                                                       \
        p.tiles = (p.dpg + kSelWaves * (64 / LPC) - 1) / (kSelWaves * (64 / LPC));                             \
        const dim3 grid((uint32_t)p.nseq * p.tiles * p.G);                                                     \
        if (vec) hipLaunchKernelGGL((k_selscan<T, NPL, LPC, true, STORE>), grid, dim3(64 * kSelWaves), 0, st, p);     \
        else hipLaunchKernelGGL((k_selscan<T, NPL, LPC, false, STORE>), grid, dim3(64 * kSelWaves), 0, st, p);        \
    } while (0)
    M3_SEL_DISPATCH(p.N, M3_GO);
#undef M3_GO
}

mamba3_status launch_selective_scan(const mamba3_selective_scan_args *a, hipStream_t st) {
    const SelParams p = sel_params(a);
    if (a->dtype == MAMBA3_F32) scan_go<float, false>(p, sel_vec(p, 4), st);
    else scan_go<bf16, false>(p, sel_vec(p, 2), st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

size_t selective_workspace_bytes(const mamba3_selective_scan_args *a) {
    (void)a;
    return 0;
}

void launch_sel_stored(const SelParams &p, int32_t dtype, bool vec, hipStream_t st) {
    if (dtype == MAMBA3_F32) scan_go<float, true>(p, vec, st);
    else scan_go<bf16, true>(p, vec, st);
}

template <typename T>
static void step_go(const mamba3_selective_step_args *a, const SelStepParams &p, hipStream_t st) {
    const int64_t es = sizeof(T);
    const bool vec = p.N % 4 == 0 && quads(p.B, p.B_row, es) && quads(p.C, p.C_row, es);
#define M3_GO(NPL, LPC)                                                                                        \
    do {                                                                                                       \
        const int tiles = (p.dim + 256 / LPC - 1) / (256 / LPC);                                               \
        const dim3 grid((uint32_t)a->batch * tiles);                                                           \
        if (vec) hipLaunchKernelGGL((k_selstep<T, NPL, LPC, true>), grid, dim3(256), 0, st, p, tiles);         \
        else hipLaunchKernelGGL((k_selstep<T, NPL, LPC, false>), grid, dim3(256), 0, st, p, tiles);            \
    } while (0)
    M3_SEL_DISPATCH(p.N, M3_GO);
#undef M3_GO
}

mamba3_status launch_selective_step(const mamba3_selective_step_args *a, hipStream_t st) {
    SelStepParams p{};
    const int64_t gn = (int64_t)a->ngroups * a->dstate;
    p.x = a->x; p.dt = a->dt; p.B = a->B; p.C = a->C; p.z = a->z;
    p.A = a->A; p.D = a->D; p.bias = a->dt_bias; p.h = a->h; p.y = a->y;
    p.x_row = dense(a->x_row, a->dim);
    p.dt_row = dense(a->dt_row, a->dim);
    p.z_row = dense(a->z_row, a->dim);
    p.B_row = dense(a->B_row, gn);
    p.C_row = dense(a->C_row, gn);
    p.slots = a->slots; p.nslots = a->nslots;
    p.dim = a->dim; p.dpg = a->dim / a->ngroups; p.N = a->dstate; p.softplus = a->dt_softplus;
    if (a->dtype == MAMBA3_F32) step_go<float>(a, p, st);
    else step_go<bf16>(a, p, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
