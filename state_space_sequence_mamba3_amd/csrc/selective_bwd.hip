// Backward of the selective scan. With r_t = dy_t SiLU(z_t) and, per channel d and state n,
//   g_t = C_t r_t + a_{t+1} g_{t+1}                        (a_t = exp(s_t A), g carries dh_out at the end)
//   dC_t = sum_d r_t h_t,  dB_t = sum_d g_t u_t,           (u_t = s_t x_t)
//   du_t = sum_n g_t B_t,  ds_t = du_t x_t + sum_n g_t a_t h_{t-1} A,   dA = sum_t g_t a_t h_{t-1} s_t
//   dx_t = du_t s_t + D r_t,  ddt_t = ds_t softplus'(dt_t + bias),  dz_t = dy_t y_t SiLU'(z_t)
//
// The forward pass keeps nothing: a first pass (k_selscan's STORE form) writes the state before every 8
// tokens in fp32, and this pass walks those pieces backwards. A piece's states and decays are computed again
// and stay in registers while its tokens are taken in reverse.
//
// Workspace, a token and channel: N' / 2 bytes of states (N' = N rounded up to 4, 8, .. 128), and 8 N / c bytes of
// dB and dC's sums over the c channels of a workgroup (256, 128, 64, 32, 16, 16): 2.1, 4.5, 10, 24, 64, 128 bytes at
// N = 4, 8, .. 128, where a bf16 token array has 2 (segments add half a byte and their states). Both are written
// and read once.
//
// Up to N = 16 the vector unit bounds it: about 20 issue slots for every token, channel and state.
// 8 x 2048 tokens of 4096 channels at N = 16, bf16: 1.14 ms, of which 0.22 the states, 0.89 this pass
// (the vector unit 86 % busy, two waves a SIMD) and 0.03 the sums over workgroups. Pieces of 16 tokens took
// 342 registers, one wave a SIMD and 0.4 ms more; the matrix unit's fp32 products for the sums over
// channels take their cycles from the vector unit and cost 0.35 ms.
// Two waves a SIMD are left at N = 9 .. 32 only (88 % busy at 32; fp32 at N = 17 .. 32 with 4 to 10 registers spilled).
// Below, tiles of 16 tokens of 64 and 32 channels a wave take 294 to 458 registers; above, the staged tiles leave room in
// the LDS for one workgroup a CU (105 KB at N = 33 .. 64; 102 at 65 .. 128, with 410 registers and more). One wave a
// SIMD keeps the vector unit 57 % (N = 4), 59 (8), 52 (64) and 42 (128) busy; at 128 LDS bank conflicts take a
// third of the cycles besides. The same tokens at N = 4, 8, 32, 64, 128: 0.67, 0.97, 2.37, 7.5, 19.7 ms; fp32 at
// 4 .. 128: 0.86, 1.09, 1.24, 2.47, 7.7, 19.2.
#include <type_traits>

#include "selective.h"

namespace m3 {

struct SelBwdParams {
    SelParams f;
    const float *dh_out;
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *dbias, *dh_in;
    float *part_bc;     // [G * tiles][total][2][N]: dB and dC of one workgroup's channels
    float *part_a;      // [rows][D][N]
    float *part_d;      // [rows][2][D]: dD, ddt_bias
};

template <int NP, int CW, int TT>
struct SelBwdLds {
    float B[TT][NP], C[TT][NP];
    float u[TT][CW][4];                 // s, u, r
    float y[TT][CW], du[TT][CW], ds[TT][CW];
    float bc[2][TT][2][NP];             // the wave's dB and dC, two tiles' buffers
};

// One level of the sum over the channels of a wave: pairs of values, BIT the lane bit that is summed
// over and that then names the value of the pair.
template <int BIT>
__device__ __forceinline__ float pair_sum(float a, float b, int lane) {
    if constexpr (BIT == 5) {
        const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(v[0]) + __uint_as_float(v[1]);
    } else if constexpr (BIT == 4) {
        const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(v[0]) + __uint_as_float(v[1]);
    } else if constexpr (BIT == 3) {
        return dpp_into<0x128, 0x3>(b, a) + dpp_into<0x128, 0xC>(a, b);
    } else if constexpr (BIT == 2) {
        return dpp_into<0x104, 0x5>(b, a) + dpp_into<0x114, 0xA>(a, b);
    } else {
        const bool up = lane >> BIT & 1;
        const float keep = up ? b : a, send = up ? a : b;
        return keep + dpp_move<BIT == 1 ? 0x4E : 0xB1>(send);
    }
}
// V values summed over the lane bits 5 .. LOW; of the V >> (6 - LOW) left, lane l's value f is number
// f << (6 - LOW) | (bit 5 of l, bit 4 of l << 1, ..).
template <int V, int BIT, int LOW>
__device__ __forceinline__ void channel_sum(float (&p)[V], int lane) {
    if constexpr (BIT >= LOW) {
        static_assert(V >> (6 - LOW) >= 1, "a value left for every lane");
#pragma unroll
        for (int i = 0; i < V >> (6 - BIT); i++) p[i] = pair_sum<BIT>(p[2 * i], p[2 * i + 1], lane);
        channel_sum<V, BIT - 1, LOW>(p, lane);
    }
}
// The value number that lane l holds in p[0] after channel_sum
template <int LOW>
__device__ __forceinline__ int channel_value(int lane) {
    int v = 0;
#pragma unroll
    for (int b = 5; b >= LOW; b--) v |= (lane >> b & 1) << (5 - b);
    return v;
}

template <int LPC> constexpr int kLow = LPC == 1 ? 0 : LPC == 2 ? 1 : LPC == 4 ? 2 : LPC == 8 ? 3 : 4;

// The workgroups and their channels are k_selscan's; its four waves keep step, because dB and dC are
// summed over them before they leave the workgroup.
template <typename T, int NPL, int LPC, Access ACC>
__global__ __launch_bounds__(64 * kSelWaves, LPC >= 4 && NPL == 4 ? 2 : 1) void k_selbwd(SelBwdParams q) {
    constexpr int CW = 64 / LPC, NP = NPL * LPC, SUB = kSelStored, TT = 64 / NPL, NSUB = TT / SUB;
    constexpr int XQ = TT * CW / 4, XE = (XQ + 63) / 64;
    constexpr int BQ = TT * NP / 4, BE = (BQ + 63) / 64;
    constexpr int LOW = kLow<LPC>;
    constexpr int GS = LPC < SUB ? LPC : SUB;                     // tokens of one transposed sum
    constexpr int VT = 2 * NPL;                                 // values a token to sum over channels
    constexpr int TV = (1 << (6 - LOW)) > VT ? (1 << (6 - LOW)) / VT : 1;   // tokens of one channel sum
    constexpr int V = VT * TV;
    __shared__ SelBwdLds<NP, CW, TT> lds[kSelWaves];
    const SelParams &p = q.f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    SelBwdLds<NP, CW, TT> &S = lds[wave];
    const int per = p.tiles * p.G;
    const int rw = blockIdx.x / per, gt = blockIdx.x % per, g = gt / p.tiles;
    const int c0 = ((gt % p.tiles) * kSelWaves + wave) * CW;
    const SelRow row = sel_row(p, rw);
    if (row.seq < 0) return;
    const int ch = lane / LPC, sub = lane % LPC, n0 = sub * NPL;
    const bool real = c0 + ch < p.dpg;
    const int d = g * p.dpg + min(c0 + ch, p.dpg - 1);

    float A[NPL], G[NPL], dA[NPL];
    load_states<NPL, ACC == ALIGNED>(A, p.A + (int64_t)d * p.N, n0, p.N);
#pragma unroll
    for (int i = 0; i < NPL; i++) G[i] = dA[i] = 0.f;
    // lanes behind the group's last channel repeat it with no gradient: they add nothing to dB and dC
    if (!real) {
    } else if (p.seg_g) load_states<NPL, ACC == ALIGNED>(G, p.seg_g + ((int64_t)rw * p.dim + d) * p.N, n0, p.N);
    else if (q.dh_out) load_states<NPL, ACC == ALIGNED>(G, q.dh_out + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);

    float most = A[0], least = A[0];                            // of the lane's states
#pragma unroll
    for (int i = 1; i < NPL; i++) {
        most = fmaxf(most, A[i]);
        least = fminf(least, A[i]);
    }
    float H[NPL];                                               // the state that enters the segment
#pragma unroll
    for (int i = 0; i < NPL; i++) H[i] = 0.f;
    if (p.seg_h) load_states<NPL, ACC == ALIGNED>(H, p.seg_h + ((int64_t)rw * p.dim + d) * p.N, n0, p.N);

    int xt[XE], xc[XE], bt[BE], bn[BE];
    f32x4 biasv[XE], Dv[XE], dDv[XE], dbv[XE];
#pragma unroll
    for (int i = 0; i < XE; i++) {
        const int k = min(lane + 64 * i, XQ - 1);
        xt[i] = k / (CW / 4);
        xc[i] = c0 + k % (CW / 4) * 4;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int dd = g * p.dpg + min(xc[i] + e, p.dpg - 1);
            biasv[i][e] = p.bias ? p.bias[dd] : 0.f;
            Dv[i][e] = p.D ? p.D[dd] : 0.f;
            dDv[i][e] = dbv[i][e] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < BE; i++) {
        const int k = min(lane + 64 * i, BQ - 1);
        bt[i] = k / (NP / 4);
        bn[i] = k % (NP / 4) * 4;
    }
    const T *x = (const T *)p.x + g * p.dpg, *dt = (const T *)p.dt + g * p.dpg;
    const T *z = p.z ? (const T *)p.z + g * p.dpg : nullptr, *dy = (const T *)p.dy + g * p.dpg;
    const T *B = (const T *)p.B + g * p.N, *C = (const T *)p.C + g * p.N;
    const int64_t stored = stored_base(row.t0, rw, SUB);

    quad<T> rx[XE], rd[XE], rz[XE], ry[XE], rB[BE], rC[BE];
    float h0n[NSUB][NPL], s0n[NSUB];
#pragma unroll
    for (int b = 0; b < NSUB; b++) s0n[b] = 0.f;
    // the tile from t0 on (tokens behind the row's last repeat it)
    auto fetch = [&](int t0) {
        const int64_t at = scalar_token(t0);
        const T *x0 = x + at * p.x_row, *d0 = dt + at * p.dt_row, *z0 = z + at * p.z_row, *y0 = dy + at * p.dy_row,
                *B0 = B + at * p.B_row, *C0 = C + at * p.C_row;
        auto load = [&](auto tail) {
            constexpr bool TAIL = decltype(tail)::value;
#pragma unroll
            for (int i = 0; i < XE; i++) {
                const int t = TAIL ? min(xt[i], row.t1 - 1 - t0) : xt[i];
                rx[i] = load_quad<T, ACC>(x0, t, p.x_row, xc[i], p.dpg);
                rd[i] = load_quad<T, ACC>(d0, t, p.dt_row, xc[i], p.dpg);
                if (z) rz[i] = load_quad<T, ACC>(z0, t, p.z_row, xc[i], p.dpg);
                ry[i] = load_quad<T, ACC>(y0, t, p.dy_row, xc[i], p.dpg);
            }
#pragma unroll
            for (int i = 0; i < BE; i++) {
                const int t = TAIL ? min(bt[i], row.t1 - 1 - t0) : bt[i];
                rB[i] = load_quad<T, states_access(ACC, LPC)>(B0, t, p.B_row, bn[i], p.N);
                rC[i] = load_quad<T, states_access(ACC, LPC)>(C0, t, p.C_row, bn[i], p.N);
            }
        };
        if (t0 + TT <= row.t1) load(std::integral_constant<bool, false>());
        else load(std::integral_constant<bool, true>());
#pragma unroll
        for (int b = 0; b < NSUB; b++) {
            if (t0 + b * SUB >= row.t1) continue;
            const int64_t k = stored + (t0 - row.t0) / SUB + b;
            const float *from = p.ckpt + stored_at(k, per, gt, wave, lane, NPL);
            if (p.seg_h) s0n[b] = p.ckpt_s[((k * per + gt) * kSelWaves + wave) * CW + ch];
#pragma unroll
            for (int i = 0; i < NPL; i += 4) {
                const f32x4 v = *(const f32x4 *)(from + i * 64);
#pragma unroll
                for (int e = 0; e < 4; e++) h0n[b][i + e] = v[e];
            }
        }
    };
    const int last = row.t0 + (row.t1 - row.t0 - 1) / TT * TT;   // the last tile's first token
    if (row.t0 < row.t1) fetch(last);
    int buf = 0;
    for (int t0 = last; t0 >= row.t0 && row.t0 < row.t1; t0 -= TT, buf ^= 1) {
        f32x4 xv[XE], zv[XE], ov[XE], rv[XE], sv[XE], gv[XE];   // x, z, dy, r, s, softplus'
        float h0s[NSUB][NPL];
#pragma unroll
        for (int b = 0; b < NSUB; b++)
#pragma unroll
            for (int i = 0; i < NPL; i++)       // a segment's states were stored as from zero
                h0s[b][i] = !real ? 0.f : p.seg_h ? h0n[b][i] + __builtin_amdgcn_exp2f(s0n[b] * (A[i] * kLog2e)) * H[i] : h0n[b][i];
        if (p.seg_h && real) {
            bool far = false;
#pragma unroll
            for (int b = 0; b < NSUB; b++) far |= fmaxf(s0n[b] * most, s0n[b] * least) > 88.f;
            if (far) {                          // (states that grow: see `carried`)
#pragma unroll
                for (int b = 0; b < NSUB; b++)
#pragma unroll
                    for (int i = 0; i < NPL; i++)
                        h0s[b][i] = h0n[b][i] + carried(s0n[b] * (A[i] * kLog2e), H[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < XE; i++) {
            const bool in = t0 + xt[i] < row.t1;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                xv[i][e] = to_f(rx[i][e]);
                zv[i][e] = z ? to_f(rz[i][e]) : 0.f;
                // behind the sequence's end: a step of 0 and no gradient hand everything on unchanged
                const float o = in && xc[i] + e < p.dpg ? to_f(ry[i][e]) : 0.f;
                ov[i][e] = o;
                const float raw = to_f(rd[i][e]) + biasv[i][e];
                const float s = p.softplus ? softplus_hw(raw) : raw;
                gv[i][e] = p.softplus ? sigmoid_hw(raw) : 1.f;
                sv[i][e] = in ? s : 0.f;
                rv[i][e] = !in ? 0.f : z ? o * zv[i][e] * sigmoid_hw(zv[i][e]) : o;
            }
            if (XQ % 64 == 0 || lane + 64 * i < XQ) {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    *(f32x4 *)&S.u[xt[i]][xc[i] - c0 + e][0] =
                        f32x4{sv[i][e], in ? sv[i][e] * xv[i][e] : 0.f, rv[i][e], 0.f};
            }
        }
#pragma unroll
        for (int i = 0; i < BE; i++) {
            if (BQ % 64 == 0 || lane + 64 * i < BQ) {
                f32x4 b, c;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const bool in = bn[i] + e < p.N && t0 + bt[i] < row.t1;
                    b[e] = in ? to_f(rB[i][e]) : 0.f;
                    c[e] = in ? to_f(rC[i][e]) : 0.f;
                }
                *(f32x4 *)&S.B[bt[i]][bn[i]] = b;
                *(f32x4 *)&S.C[bt[i]][bn[i]] = c;
            }
        }
        wave_lds_fence();
        if (t0 > row.t0) fetch(t0 - TT);
#pragma unroll 1
        for (int b0 = NSUB > 1 && t0 + SUB < row.t1 ? SUB : 0; b0 >= 0; b0 -= SUB) {
            float hs[SUB][NPL], as[SUB][NPL], h0[NPL];
#pragma unroll
            for (int i = 0; i < NPL; i++) h0[i] = b0 ? h0s[NSUB - 1][i] : h0s[0][i];
#pragma unroll
            for (int tg = 0; tg < SUB; tg += GS) {
                float part[GS];
#pragma unroll
                for (int j = 0; j < GS; j++) {
                    const int t = tg + j;
                    const float s = S.u[b0 + t][ch][0], u = S.u[b0 + t][ch][1];
                    float acc = 0.f;
#pragma unroll
                    for (int i = 0; i < NPL; i++) {
                        const float a = __builtin_amdgcn_exp2f(s * (A[i] * kLog2e));
                        as[t][i] = a;
                        hs[t][i] = a * (t ? hs[t ? t - 1 : 0][i] : h0[i]) + u * S.B[b0 + t][n0 + i];
                        acc += hs[t][i] * S.C[b0 + t][n0 + i];
                    }
                    part[j] = acc;
                }
                float v = transpose_sum<GS>(part, lane);
                if constexpr (LPC > GS) v += dpp_move<0x128>(v);
                S.y[b0 + tg + sub % GS][ch] = v;
            }
#pragma unroll
            for (int tg = SUB - GS; tg >= 0; tg -= GS) {
                float pu[GS], ps[GS];
#pragma unroll
                for (int j = GS - 1; j >= 0; j--) {
                    const int t = tg + j;
                    const float s = S.u[b0 + t][ch][0], u = S.u[b0 + t][ch][1], r = S.u[b0 + t][ch][2];
                    float du = 0.f, ds = 0.f;
#pragma unroll
                    for (int i = 0; i < NPL; i++) {
                        G[i] += r * S.C[b0 + t][n0 + i];
                        du += G[i] * S.B[b0 + t][n0 + i];
                        const float ga = G[i] * as[t][i];
                        const float w = ga * (t ? hs[t ? t - 1 : 0][i] : h0[i]);
                        dA[i] += w * s;
                        ds += w * A[i];
                        as[t][i] = u * G[i];            // dB's share, in the decay's place
                        hs[t][i] = r * hs[t][i];        // dC's, in the state's
                        G[i] = ga;
                    }
                    pu[j] = du;
                    ps[j] = ds;
                }
                float v = transpose_sum<GS>(pu, lane), w = transpose_sum<GS>(ps, lane);
                if constexpr (LPC > GS) {
                    v += dpp_move<0x128>(v);
                    w += dpp_move<0x128>(w);
                }
                S.du[b0 + tg + sub % GS][ch] = v;
                S.ds[b0 + tg + sub % GS][ch] = w;
            }
            // dB and dC: the sum over the wave's channels
#pragma unroll
            for (int tb = 0; tb < SUB; tb += TV) {
                float vals[V];
#pragma unroll
                for (int t = 0; t < TV; t++)
#pragma unroll
                    for (int i = 0; i < NPL; i++) {
                        vals[t * VT + i] = as[tb + t][i];
                        vals[t * VT + NPL + i] = hs[tb + t][i];
                    }
                channel_sum<V, 5, LOW>(vals, lane);
#pragma unroll
                for (int f = 0; f < (V >> (6 - LOW)); f++) {
                    const int k = f << (6 - LOW) | channel_value<LOW>(lane);
                    const int t = b0 + tb + k / VT, which = k % VT / NPL, i = k % NPL;
                    S.bc[buf][t][which][n0 + i] = vals[f];
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < TT * 2 * NP; i += 64 * kSelWaves) {
            const int t = i / (2 * NP), which = i / NP % 2, n = i % NP;
            if (t0 + t < row.t1 && n < p.N) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kSelWaves; w++) s += lds[w].bc[buf][t][which][n];
                q.part_bc[(((int64_t)gt * p.total + t0 + t) * 2 + which) * p.N + n] = s;
            }
        }
#pragma unroll
        for (int i = 0; i < XE; i++) {
            const int t = t0 + xt[i];
            if ((XQ % 64 == 0 || lane + 64 * i < XQ) && t < row.t1) {
                const f32x4 y = *(const f32x4 *)&S.y[xt[i]][xc[i] - c0], du = *(const f32x4 *)&S.du[xt[i]][xc[i] - c0],
                            ds = *(const f32x4 *)&S.ds[xt[i]][xc[i] - c0];
                f32x4 ox, od, oz;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    ox[e] = du[e] * sv[i][e] + Dv[i][e] * rv[i][e];
                    od[e] = (du[e] * xv[i][e] + ds[e]) * gv[i][e];
                    const float sg = sigmoid_hw(zv[i][e]);
                    oz[e] = ov[i][e] * (y[e] + Dv[i][e] * xv[i][e]) * (sg + zv[i][e] * sg * (1.f - sg));
                    dDv[i][e] += rv[i][e] * xv[i][e];
                    dbv[i][e] += od[e];
                }
                const int64_t at = scalar_token(t0) * p.dim + g * p.dpg;
                store_quad<T, ACC>((T *)q.dx + at, xt[i], p.dim, xc[i], p.dpg, ox);
                store_quad<T, ACC>((T *)q.ddt + at, xt[i], p.dim, xc[i], p.dpg, od);
                if (q.dz) store_quad<T, ACC>((T *)q.dz + at, xt[i], p.dim, xc[i], p.dpg, oz);
            }
        }
        wave_lds_fence();
    }
    if (real) {
        store_states<NPL, ACC == ALIGNED>(dA, q.part_a + ((int64_t)rw * p.dim + d) * p.N, n0, p.N);
        if (q.dh_in && row.first) store_states<NPL, ACC == ALIGNED>(G, q.dh_in + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);
    }
    // dD and ddt_bias: the sum over the lanes that hold the same channels (token lanes), in LDS
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; k++) {
        wave_lds_fence();
        float *flat = &S.u[0][0][0];                    // [TT][CW]
#pragma unroll
        for (int i = 0; i < XE; i++)
            if (XQ % 64 == 0 || lane + 64 * i < XQ) *(f32x4 *)(flat + xt[i] * CW + xc[i] - c0) = k ? dbv[i] : dDv[i];
        wave_lds_fence();
        if (lane < CW && c0 + lane < p.dpg) {
            float s = 0.f;
            for (int t = 0; t < TT; t++) s += flat[t * CW + lane];
            q.part_d[((int64_t)rw * 2 + k) * p.dim + g * p.dpg + c0 + lane] = s;
        }
    }
}

// The sums over workgroups: dB and dC over a group's channel tiles, dA, dD and ddt_bias over the rows.
template <typename T>
__global__ __launch_bounds__(256) void k_selbwd_reduce(SelBwdParams q, int bc_blocks) {
    const SelParams &p = q.f;
    if ((int)blockIdx.x < bc_blocks) {
        const int64_t n = (int64_t)p.total * p.G * 2 * p.N;
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;      // [G][total][2][N]
        if (i >= n) return;
        const int64_t each = (int64_t)p.total * 2 * p.N, g = i / each, o = i % each;
        const int64_t t = o / (2 * p.N), which = o / p.N % 2, m = o % p.N;
        if (p.cu && (t < p.cu[0] || t >= p.cu[p.nseq])) return;       // a token of no sequence
        float s = 0.f;
#pragma unroll 8
        for (int k = 0; k < p.tiles; k++) s += q.part_bc[(g * p.tiles + k) * each + o];
        ((T *)(which ? q.dC : q.dB))[(t * p.G + g) * p.N + m] = from_f<T>(s);
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - bc_blocks) * 256 + threadIdx.x, dn = (int64_t)p.dim * p.N;
    const int rows = p.table ? p.seq_row[p.nseq] : p.rows;     // (the table's rows behind hold nothing)
    float s = 0.f;
    if (i < dn) {
#pragma unroll 8
        for (int r = 0; r < rows; r++) s += q.part_a[r * dn + i];
        q.dA[i] = s;
    } else if (i < dn + 2 * p.dim) {
        const int64_t k = i - dn;
#pragma unroll 8
        for (int r = 0; r < rows; r++) s += q.part_d[(int64_t)r * 2 * p.dim + k];
        if (k < p.dim) {
            if (q.dD) q.dD[k] = s;
        } else if (q.dbias) {
            q.dbias[k - p.dim] = s;
        }
    }
}

namespace {

struct SelWs {
    size_t seg, seg_g, ckpt, ckpt_s, bc, a, d, total;
};
SelWs sel_ws(const SelParams &p, bool segments) {
    SelWs w{};
    int npl, lpc;
    sel_shape(p.N, true, npl, lpc);
    const int64_t per = (int64_t)p.tiles * p.G, stored = p.total / kSelStored + p.rows;
    auto al = [](int64_t v) { return (size_t)((v + 255) / 256 * 256); };
    size_t o = 0;
    w.seg = o; o += segments ? sel_segment_bytes(p) : 0;
    w.seg_g = o; o += segments ? al((int64_t)p.rows * p.dim * p.N * 4) : 0;
    w.ckpt = o; o += al(stored * per * kSelWaves * 64 * npl * 4);
    w.ckpt_s = o; o += segments ? al(stored * per * kSelWaves * (64 / lpc) * 4) : 0;
    w.bc = o; o += al(per * p.total * 2 * p.N * 4);
    w.a = o; o += al((int64_t)p.rows * p.dim * p.N * 4);
    w.d = o; o += al((int64_t)p.rows * 2 * p.dim * 4);
    w.total = o;
    return w;
}

template <typename T>
void bwd_go(SelBwdParams &q, Access acc, hipStream_t st) {
    SelParams &p = q.f;
#define M3_GO(NPL, LPC)                                                                                             \
    do {                                                                                                            \
        const dim3 grid((uint32_t)p.rows * p.tiles * p.G);                                                          \
        const dim3 block(64 * kSelWaves);                                                                           \
        if (acc == ALIGNED) hipLaunchKernelGGL((k_selbwd<T, NPL, LPC, ALIGNED>), grid, block, 0, st, q);            \
        else if (acc == ANY) hipLaunchKernelGGL((k_selbwd<T, NPL, LPC, ANY>), grid, block, 0, st, q);               \
        else hipLaunchKernelGGL((k_selbwd<T, NPL, LPC, ONE>), grid, block, 0, st, q);                               \
    } while (0)
    if (p.rows > 0) M3_SELBWD_DISPATCH(p.N, M3_GO);
#undef M3_GO
    const int64_t bc = sel_reduce_blocks(p), a = sel_sum_blocks(p);
    hipLaunchKernelGGL((k_selbwd_reduce<T>), dim3((uint32_t)(bc + a)), dim3(256), 0, st, q, (int)bc);
}

}  // namespace

size_t selective_bwd_workspace_bytes(const mamba3_selective_scan_bwd_args *b) {
    SelParams p = sel_params(&b->fwd);
    const bool segments = sel_plan(p, true);
    return sel_ws(p, segments).total;
}

mamba3_status launch_selective_scan_bwd(const mamba3_selective_scan_bwd_args *b, hipStream_t st) {
    SelBwdParams q{};
    q.f = sel_params(&b->fwd);
    SelParams &p = q.f;
    p.y = nullptr;
    p.h_out = nullptr;
    const bool segments = sel_plan(p, true);
    const SelWs w = sel_ws(p, segments);
    char *ws = (char *)b->workspace;
    if (segments) {
        sel_segments(p, ws + w.seg);
        p.seg_g = (float *)(ws + w.seg_g);
        p.ckpt_s = (float *)(ws + w.ckpt_s);
    }
    p.ckpt = (float *)(ws + w.ckpt);
    q.part_bc = (float *)(ws + w.bc);
    q.part_a = (float *)(ws + w.a);
    q.part_d = (float *)(ws + w.d);
    p.dy = b->dy;
    p.dy_row = b->dy_row ? b->dy_row : p.dim;
    q.dh_out = b->dh_out;
    q.dx = b->dx; q.ddt = b->ddt; q.dB = b->dB; q.dC = b->dC; q.dz = b->dz;
    q.dA = b->dA; q.dD = b->dD; q.dbias = b->ddt_bias; q.dh_in = b->dh_in;
    const int64_t es = b->fwd.dtype == MAMBA3_BF16 ? 2 : 4;
    auto quads = [&](const void *a, int64_t row) { return ((uintptr_t)a % (4 * es)) == 0 && row % 4 == 0; };
    Access acc = sel_access(p, es);
    if (acc == ALIGNED && !(quads(p.dy, p.dy_row) && quads(q.dx, 0) && quads(q.ddt, 0) && quads(q.dz, 0))) acc = ANY;
    if (p.rows > 0) {
        launch_sel_table(p, st);
        launch_sel_stored(p, b->fwd.dtype, acc, st);
        if (segments) launch_sel_chain(p, b->dh_out, st);
    }
    if (b->fwd.dtype == MAMBA3_F32) bwd_go<float>(q, acc, st);
    else bwd_go<bf16>(q, acc, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
