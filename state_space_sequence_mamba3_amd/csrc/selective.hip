// Selective scan over whole sequences and its one-token step.
//
// Per sequence, channel d (B/C group g = d / (D/G)) and state n:
//   dt' = softplus(dt_t + bias_d)  (or dt_t + bias_d)
//   h_t[d,n] = exp(dt' A[d,n]) h_{t-1}[d,n] + dt' x_t[d] B_t[g,n]
//   y_t[d]   = (sum_n C_t[g,n] h_t[d,n] + D_d x_t[d]) SiLU(z_t[d])
// The decay differs for every channel and state, so nothing of it is a matrix product: the work is
// an exponential (two issue slots), two products and two fused adds for every token, channel and
// state, on the vector unit. Where N is 16 that is 96 slots for 8 bytes of bf16, so the vector
// unit and not the memory bounds the scan: 8 x 4096 tokens of 4096 channels at N = 16 take 0.58 ms
// (1.86 TB/s of what has to move; the vector unit 87 % busy, two waves a SIMD), one sequence of 32768
// tokens of 2048 channels in 32 segments 0.44 ms (0.19 first pass, 0.01 chain, 0.24 scan; saturated).
// More states cost in proportion: 8 x 2048 tokens of 4096 channels, bf16, at N = 4, 8, 16, 32, 64, 128 take 0.26, 0.25,
// 0.30, 0.52, 1.03, 2.18 ms; fp32 the same from N = 16 on but for N = 128, whose 260 registers leave one wave
// a SIMD (3.26 ms).
// The step streams the states: 256 x 4096 channels in 30 us, 4.76 TB/s (27 with states that some cache still
// holds; then 38 with 15 states, whose rows are taken in unaligned fours and a rest, 45 state by state).
#include <cmath>
#include <type_traits>

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
// LPC lanes hold a channel: with one lane a channel there would be no sums over lanes, but a quarter
// of the waves at N = 16, and one wave alone on its SIMD issues every second slot only.
// A tile's inputs are loaded into registers while the tile before is worked on (4 channels of one
// token a lane, so that a wave's load covers whole 32-byte pieces and the four waves of a
// workgroup whole 128-byte lines), prepared there (softplus, dt' x, fp32) and laid into the wave's
// own LDS; the recurrence then reads them as broadcasts. No wave waits for another.
//
// FULL writes y and h_out. PART is a segment's first pass: its last state from a zero state and the sum
// of its steps, no outputs. STORE is the backward's first pass: the states before every kSelStored
// tokens; STORE_PART the same for segments, with PART's results and the segment's share of the
// gradient that flows on to the one before it, sum_t (prod_{s <= t} a_s) C_t r_t.
enum SelMode { FULL, PART, STORE, STORE_PART };

template <typename T, int NPL, int LPC, Access ACC, int MODE>
__global__ __launch_bounds__(64 * kSelWaves) void k_selscan(SelParams p) {
    constexpr int CW = 64 / LPC, NP = NPL * LPC, TT = kSelTile;
    constexpr int XQ = TT * CW / 4, XE = (XQ + 63) / 64;      // quads of a channel tile, and of a lane
    constexpr int BQ = TT * NP / 4, BE = (BQ + 63) / 64;
    __shared__ SelLds<NP, CW> lds[kSelWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    SelLds<NP, CW> &S = lds[wave];
    const int per = p.tiles * p.G;
    const int r = blockIdx.x / per, gt = blockIdx.x % per, g = gt / p.tiles;
    const int c0 = ((gt % p.tiles) * kSelWaves + wave) * CW;  // the wave's first channel in its group
    if (c0 >= p.dpg) return;
    const SelRow row = sel_row(p, r);
    if (row.seq < 0 || (MODE == PART && row.last)) return;    // (nothing takes up a last segment's end)
    constexpr bool CKPT = MODE == STORE || MODE == STORE_PART, ENDS = MODE == PART || MODE == STORE_PART;
    constexpr bool NEEDC = MODE == FULL || MODE == STORE_PART;
    const int ch = lane / LPC, sub = lane % LPC, n0 = sub * NPL;
    const bool real = c0 + ch < p.dpg;
    const int d = g * p.dpg + min(c0 + ch, p.dpg - 1);        // the lane's channel in the recurrence

    float A2[NPL], h[NPL];
    load_states<NPL, ACC == ALIGNED>(A2, p.A + (int64_t)d * p.N, n0, p.N);
#pragma unroll
    for (int i = 0; i < NPL; i++) A2[i] *= kLog2e;
#pragma unroll
    for (int i = 0; i < NPL; i++) h[i] = 0.f;
    if (MODE == FULL && p.seg_h) load_states<NPL, ACC == ALIGNED>(h, p.seg_h + ((int64_t)r * p.dim + d) * p.N, n0, p.N);
    else if (!ENDS && p.h_in) load_states<NPL, ACC == ALIGNED>(h, p.h_in + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);
    float sum = 0.f, prod[NPL], share[NPL];             // of the steps; of the decays; see STORE_PART
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        prod[i] = 1.f;
        share[i] = 0.f;
    }

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
    const T *z = p.z && NEEDC ? (const T *)p.z + g * p.dpg : nullptr;
    const T *dy = (const T *)p.dy + g * p.dpg;
    const T *B = (const T *)p.B + g * p.N, *C = (const T *)p.C + g * p.N;
    T *y = (T *)p.y + g * p.dpg;

    quad<T> rx[XE], rd[XE], rz[XE], ry[XE], rB[BE], rC[BE];
    // the tile from t0 on; TAIL: it may end behind the row's last token, whose inputs are repeated then
    // (inlined by force: a call would take the captured registers through scratch memory, which it did with
    // 3 states: 4 x 2048 tokens of 4096 channels 908 us instead of 166)
    auto fetch = [&](int t0, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        const int64_t at = scalar_token(t0);
        const T *x0 = x + at * p.x_row, *d0 = dt + at * p.dt_row, *z0 = z + at * p.z_row, *y0 = dy + at * p.dy_row,
                *B0 = B + at * p.B_row, *C0 = C + at * p.C_row;
#pragma unroll
        for (int i = 0; i < XE; i++) {
            const int t = TAIL ? min(xt[i], row.t1 - 1 - t0) : xt[i];
            rx[i] = load_quad<T, ACC>(x0, t, p.x_row, xc[i], p.dpg);
            rd[i] = load_quad<T, ACC>(d0, t, p.dt_row, xc[i], p.dpg);
            if (z) rz[i] = load_quad<T, ACC>(z0, t, p.z_row, xc[i], p.dpg);
            if (MODE == STORE_PART) ry[i] = load_quad<T, ACC>(y0, t, p.dy_row, xc[i], p.dpg);
        }
#pragma unroll
        for (int i = 0; i < BE; i++) {
            const int t = TAIL ? min(bt[i], row.t1 - 1 - t0) : bt[i];
            rB[i] = load_quad<T, states_access(ACC, LPC)>(B0, t, p.B_row, bn[i], p.N);
            if (NEEDC) rC[i] = load_quad<T, states_access(ACC, LPC)>(C0, t, p.C_row, bn[i], p.N);
        }
    };
    const std::integral_constant<bool, false> whole_tile;
    const std::integral_constant<bool, true> last_tile;
    auto fetch_next = [&](int t0) __attribute__((always_inline)) {
        if (t0 + TT <= row.t1) fetch(t0, whole_tile);
        else if (t0 < row.t1) fetch(t0, last_tile);
    };
    const int64_t stored = stored_base(row.t0, r, kSelStored);
    auto tile = [&](int t0, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        const int left = TAIL ? row.t1 - t0 : TT;           // the tile's tokens
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
                const bool in = !TAIL || xt[i] < left;
                u[e >> 1][2 * (e & 1)] = in ? s : 0.f;
                u[e >> 1][2 * (e & 1) + 1] = in ? s * xv[i][e] : 0.f;
            }
            if (XQ % 64 == 0 || lane + 64 * i < XQ) {
                f32x4 *to = (f32x4 *)&S.u[xt[i]][xc[i] - c0][0];
                to[0] = u[0];
                to[1] = u[1];
                if (MODE == STORE_PART) {                   // r = dy SiLU(z), in y's place
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        v[e] = to_f(ry[i][e]);
                        if (z) v[e] *= zv[i][e] * sigmoid_hw(zv[i][e]);
                        v[e] = !TAIL || xt[i] < left ? v[e] : 0.f;
                    }
                    *(f32x4 *)&S.y[xt[i]][xc[i] - c0] = v;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < BE; i++) {
            if (BQ % 64 == 0 || lane + 64 * i < BQ) {
                f32x4 b, c;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    b[e] = to_f(rB[i][e]);
                    c[e] = NEEDC ? to_f(rC[i][e]) : 0.f;
                }
                if (TAIL || p.N != NP) {
                    // places behind the last state or token hold zero, whatever lies there
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const bool in = bn[i] + e < p.N && (!TAIL || bt[i] < left);
                        b[e] = in ? b[e] : 0.f;
                        c[e] = in ? c[e] : 0.f;
                    }
                }
                *(f32x4 *)&S.B[bt[i]][bn[i]] = b;
                if (NEEDC) *(f32x4 *)&S.C[bt[i]][bn[i]] = c;
            }
        }
        wave_lds_fence();
        fetch_next(t0 + TT);
        // The operands of PF tokens come from LDS while the PF before are worked on (the prompt above: 622
        // us without, 583 with; four at once cost the long one a wave a SIMD).
        constexpr int PF = 2;
        struct Ops {
            float s, u, r;
            f32x4 b[NPL / 4], c[NPL / 4];
        } op[2][PF];
        auto operands = [&](int t, Ops &o) __attribute__((always_inline)) {
            o.s = S.u[t][ch][0];
            o.u = S.u[t][ch][1];
            if (MODE == STORE_PART) o.r = S.y[t][ch];
#pragma unroll
            for (int i = 0; i < NPL / 4; i++) {
                o.b[i] = *(const f32x4 *)&S.B[t][n0 + 4 * i];
                if (NEEDC) o.c[i] = *(const f32x4 *)&S.C[t][n0 + 4 * i];
            }
        };
#pragma unroll
        for (int k = 0; k < PF; k++) operands(k, op[0][k]);
        float part[LPC];
#pragma unroll
        for (int t = 0; t < TT; t++) {
            if (t % PF == 0) {
                if (t + PF < TT) {
#pragma unroll
                    for (int k = 0; k < PF; k++) operands(t + PF + k, op[(t / PF + 1) & 1][k]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            const Ops &o = op[t / PF & 1][t % PF];
            if (CKPT && t % kSelStored == 0 && t < left) {
                const int64_t k = stored + (t0 - row.t0 + t) / kSelStored;
                float *to = p.ckpt + stored_at(k, per, gt, wave, lane, NPL);
#pragma unroll
                for (int i = 0; i < NPL; i += 4)
                    *(f32x4 *)(to + i * 64) = f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]};
                if (MODE == STORE_PART && sub == 0)
                    p.ckpt_s[((k * per + gt) * kSelWaves + wave) * CW + ch] = sum;
            }
            if (ENDS) sum += o.s;
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; i++) {
                const float a = __builtin_amdgcn_exp2f(o.s * A2[i]);
                h[i] = a * h[i] + o.u * o.b[i / 4][i % 4];
                if (MODE == FULL) acc += h[i] * o.c[i / 4][i % 4];
                if (MODE == STORE_PART) {
                    prod[i] *= a;
                    share[i] += prod[i] * (o.r * o.c[i / 4][i % 4]);
                }
            }
            part[t % LPC] = acc;
            if (MODE == FULL && t % LPC == LPC - 1) S.y[t - (LPC - 1) + sub][ch] = transpose_sum<LPC>(part, lane);
        }
        wave_lds_fence();
        if (MODE != FULL) return;
        T *y0 = y + scalar_token(t0) * p.dim;
#pragma unroll
        for (int i = 0; i < XE; i++) {
            if ((XQ % 64 == 0 || lane + 64 * i < XQ) && (!TAIL || xt[i] < left)) {
                f32x4 v = *(const f32x4 *)&S.y[xt[i]][xc[i] - c0];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[e] += Dv[i][e] * xv[i][e];
                    if (z) v[e] *= zv[i][e] * sigmoid_hw(zv[i][e]);
                }
                store_quad<T, ACC>(y0, xt[i], p.dim, xc[i], p.dpg, v);
            }
        }
        wave_lds_fence();
    };
    fetch_next(row.t0);
    int t0 = row.t0;
    for (; t0 + TT <= row.t1; t0 += TT) tile(t0, whole_tile);
    if (t0 < row.t1) tile(t0, last_tile);
    if (!real) return;
    if (MODE == FULL && p.h_out && row.last)
        store_states<NPL, ACC == ALIGNED>(h, p.h_out + ((int64_t)row.seq * p.dim + d) * p.N, n0, p.N);
    if (ENDS) {
        store_states<NPL, ACC == ALIGNED>(h, p.seg_h + ((int64_t)r * p.dim + d) * p.N, n0, p.N);
        if (sub == 0) p.seg_s[(int64_t)r * p.dim + d] = sum;
    }
    if (MODE == STORE_PART) {
        // decays above one whose product left fp32's range: the share from the last token on, which is in
        // range wherever the gradient is
        bool over = false;
#pragma unroll
        for (int i = 0; i < NPL; i++) over |= !(prod[i] < INFINITY);
        if (over) {
#pragma unroll
            for (int i = 0; i < NPL; i++) share[i] = 0.f;
            const int c = d - g * p.dpg;
            for (int64_t t = row.t1 - 1; t >= row.t0; t--) {
                float s = to_f(dt[t * p.dt_row + c]) + (p.bias ? p.bias[d] : 0.f), r = to_f(dy[t * p.dy_row + c]);
                if (p.softplus) s = softplus_hw(s);
                if (z) {
                    const float zt = to_f(z[t * p.z_row + c]);
                    r *= zt * sigmoid_hw(zt);
                }
#pragma unroll
                for (int i = 0; i < NPL; i++) {
                    const float ct = n0 + i < p.N ? to_f(C[t * p.C_row + n0 + i]) : 0.f;
                    share[i] = __builtin_amdgcn_exp2f(s * A2[i]) * (share[i] + r * ct);
                }
            }
        }
    }
    if (MODE == STORE_PART) store_states<NPL, ACC == ALIGNED>(share, p.seg_g + ((int64_t)r * p.dim + d) * p.N, n0, p.N);
}

// The segments of a packed batch in the order of their tokens, one at least a sequence; entries behind
// the last have no sequence. One workgroup.
constexpr int kSelTabThreads = 256;
__global__ __launch_bounds__(kSelTabThreads) void k_seltable(SelParams p, int4 *table, int32_t *seq_row) {
    __shared__ int wsum[kSelTabThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t carry = 0;
    for (int s0 = 0; s0 < p.nseq; s0 += kSelTabThreads) {
        const int s = s0 + tid;
        int a = 0, b = 0, n = 0;
        if (s < p.nseq) {
            packed_bounds(p.cu, s, p.total, a, b);
            n = max(1, (b - a + p.seg_tokens - 1) / p.seg_tokens);
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o, 64);
            if (lane >= o) incl += v;
        }
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kSelTabThreads / 64; w++) {
            before += w < wave ? wsum[w] : 0;
            all += wsum[w];
        }
        // (a table whose entries decrease may count more rows than there are: none lies outside)
        const int64_t first = min(carry + before + incl - n, (int64_t)p.rows);
        if (s < p.nseq) seq_row[s] = (int)first;
        for (int k = 0; k < n && first + k < p.rows; k++)
            table[first + k] = make_int4(a + k * p.seg_tokens, (int)min((int64_t)a + (int64_t)(k + 1) * p.seg_tokens, (int64_t)b),
                                         s, (k == 0 ? 1 : 0) | (k == n - 1 ? 2 : 0));
        carry = min(carry + all, (int64_t)p.rows);
        __syncthreads();
    }
    if (tid == 0) seq_row[p.nseq] = (int)carry;
    for (int64_t r = carry + tid; r < p.rows; r += kSelTabThreads) table[r] = make_int4(0, 0, -1, 0);
}

// The chain over a sequence's segments, a thread for each channel and state: the state that enters a
// segment replaces its own end in seg_h, H_{k+1} = exp(A sum_k) H_k + U_k (see `carried`); the gradient that enters it at
// its end replaces its share in seg_g, G_{k-1} = exp(A sum_k) G_k + V_k from dh_out on. Loads of eight
// segments are in flight together.
constexpr int kSelChain = 8;
__global__ __launch_bounds__(256) void k_selchain(SelParams p, const float *dh_out) {
    const int64_t dn = (int64_t)p.dim * p.N, blocks = (dn + 255) / 256;
    const int s = (int)(blockIdx.x / blocks);
    const int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x;
    if (i >= dn) return;
    const int64_t d = i / p.N;
    const int r0 = p.table ? p.seq_row[s] : s * p.nseg, r1 = p.table ? p.seq_row[s + 1] : r0 + p.nseg;
    const float A2 = p.A[i] * kLog2e;
    if (blockIdx.y == 0) {
        float H = p.h_in ? p.h_in[s * dn + i] : 0.f;
        for (int r = r0; r < r1; r += kSelChain) {
            float U[kSelChain], S[kSelChain];
#pragma unroll
            for (int k = 0; k < kSelChain; k++) {
                const int64_t q = min(r + k, r1 - 1);
                const bool in = r + k < r1 - 1;             // (a last segment's end is not there)
                U[k] = in ? p.seg_h[q * dn + i] : 0.f;
                S[k] = in ? p.seg_s[q * p.dim + d] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kSelChain; k++)
                if (r + k < r1) {
                    p.seg_h[(int64_t)(r + k) * dn + i] = H;
                    H = carried(S[k] * A2, H) + U[k];
                }
        }
    } else {
        float G = dh_out ? dh_out[s * dn + i] : 0.f;
        for (int r = r1 - 1; r >= r0; r -= kSelChain) {
            float V[kSelChain], S[kSelChain];
#pragma unroll
            for (int k = 0; k < kSelChain; k++) {
                const int64_t q = max(r - k, r0);
                V[k] = p.seg_g[q * dn + i];
                S[k] = p.seg_s[q * p.dim + d];
            }
#pragma unroll
            for (int k = 0; k < kSelChain; k++)
                if (r - k >= r0) {
                    p.seg_g[(int64_t)(r - k) * dn + i] = G;
                    G = carried(S[k] * A2, G) + V[k];
                }
        }
    }
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

template <typename T, int NPL, int LPC, Access ACC>
__global__ __launch_bounds__(256) void k_selstep(SelStepParams p, int tiles) {
    constexpr int CB = 256 / LPC;                       // channels of a workgroup
    const int b = blockIdx.x / tiles, d = (blockIdx.x % tiles) * CB + threadIdx.x / LPC;
    const int sub = threadIdx.x % LPC, n0 = sub * NPL;
    if (d >= p.dim) return;                             // whole channels: a channel's lanes stay together
    // what does not wait for the slot first: a step is a few memory latencies long
    float h[NPL], A2[NPL];
    load_states<NPL, ACC == ALIGNED>(A2, p.A + (int64_t)d * p.N, n0, p.N);
    const int g = d / p.dpg;
    const T *B = (const T *)p.B + b * p.B_row + g * p.N, *C = (const T *)p.C + b * p.C_row + g * p.N;
    const float x = to_f(((const T *)p.x)[b * p.x_row + d]), D = p.D ? p.D[d] : 0.f;
    const float z = p.z ? to_f(((const T *)p.z)[b * p.z_row + d]) : 0.f;
    float s = to_f(((const T *)p.dt)[b * p.dt_row + d]) + (p.bias ? p.bias[d] : 0.f);
    float Bv[NPL], Cv[NPL];
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
        const quad<T> bq = load_quad<T, states_access(ACC, LPC)>(B, 0, 0, n0 + i, p.N), cq = load_quad<T, states_access(ACC, LPC)>(C, 0, 0, n0 + i, p.N);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            Bv[i + e] = n0 + i + e < p.N ? to_f(bq[e]) : 0.f;
            Cv[i + e] = n0 + i + e < p.N ? to_f(cq[e]) : 0.f;
        }
    }
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nslots) return;       // inactive row (uniform across the workgroup)
    }
    float *hs = p.h + (slot * p.dim + d) * p.N;
    load_states<NPL, ACC == ALIGNED>(h, hs, n0, p.N);
    if (p.softplus) s = softplus_hw(s);
    const float u = s * x;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        h[i] = exp_hw(s * A2[i]) * h[i] + u * Bv[i];
        acc += h[i] * Cv[i];
    }
    store_states<NPL, ACC == ALIGNED>(h, hs, n0, p.N);
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) acc += __shfl_xor(acc, o, 64);
    if (sub == 0) {
        float v = acc + D * x;
        if (p.z) v *= z * sigmoid_hw(z);
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

// How the rows can be read: a group's channels and the states are the rows' lengths.
Access sel_access(const SelParams &p, int64_t es) {
    const bool al = p.dpg % 4 == 0 && p.N % 4 == 0 && quads(p.x, p.x_row, es) && quads(p.dt, p.dt_row, es) &&
           quads(p.B, p.B_row, es) && quads(p.C, p.C_row, es) && quads(p.z, p.z_row, es) && quads(p.y, p.dim, es);
    return al ? ALIGNED : p.dpg >= 4 ? ANY : ONE;
}

template <typename T, int MODE>
static void scan_go(const SelParams &p, Access acc, hipStream_t st) {
#define M3_GO(NPL, LPC)                                                                                          \
    do {                                                                                                         \
        const dim3 grid((uint32_t)p.rows * p.tiles * p.G);                                                       \
        const dim3 block(64 * kSelWaves);                                                                        \
        if (acc == ALIGNED) hipLaunchKernelGGL((k_selscan<T, NPL, LPC, ALIGNED, MODE>), grid, block, 0, st, p);  \
        else if (acc == ANY) hipLaunchKernelGGL((k_selscan<T, NPL, LPC, ANY, MODE>), grid, block, 0, st, p);     \
        else hipLaunchKernelGGL((k_selscan<T, NPL, LPC, ONE, MODE>), grid, block, 0, st, p);                     \
    } while (0)
    if constexpr (MODE >= STORE) M3_SELBWD_DISPATCH(p.N, M3_GO);
    else M3_SEL_DISPATCH(p.N, M3_GO);
#undef M3_GO
}

// A wave's instructions issue every second slot at best when it is alone on its SIMD, so fewer than
// 256 workgroups (one a CU, one wave a SIMD) run at less than half the vector unit's rate. Segments cost
// a first pass of about two thirds of the scan and the chain, and pay below that; the backward has its
// first pass anyway. Sequences of 2048 tokens and 4096 channels (64 workgroups each), whole and in segments:
// forward 1 204 and 76 us, 3 206 and 182, 4 211 and 234, 8 314 and 437; backward 4 834 and 688, 6 1145 and
// 1141. Segments are as long as leave 1024 workgroups of the forward (four a CU; 512 of the backward,
// whose registers allow two), sqrt(2/3 of the sequence) and 64 tokens at least: no workgroup waits for a
// place. Packed sequences are of unknown lengths, and the longest one decides when nothing else is left to
// run: they are cut below 1024 workgroups, into pieces of their mean length at most (random lengths, forward: 6
// sequences 581 and 356 us, 12 745 and 670, 16 792 and 780, 20 888 and 1036).
bool sel_plan(SelParams &p, bool back) {
    int npl, lpc;
    sel_shape(p.N, back, npl, lpc);
    const int cw = kSelWaves * (64 / lpc);
    p.tiles = (p.dpg + cw - 1) / cw;
    p.rows = p.nseq;
    p.nseg = 1;
    p.seg_tokens = p.seqlen;
    const int64_t per = (int64_t)p.tiles * p.G;
    if (p.nseq == 0 || p.nseq * per >= (p.cu ? 1024 : back ? 384 : 256)) return false;
    const int64_t most = (back ? 512 : 1024) / per;                   // rows in all
    const int64_t cut = p.cu ? std::max<int64_t>(most - p.nseq, p.nseq) : most / p.nseq;   // of these by length
    if (cut < 2) return false;
    const int64_t tokens = p.cu ? p.total : p.seqlen;
    // a token of a lone wave takes about 0.2 us in the two passes and a segment 0.15 us in the chain:
    // segments of sqrt(2/3 tokens) balance the two (one sequence of 65536 tokens and 64 channels in
    // 1024, 313 segments: 281, 118 us)
    const int64_t least = std::max<int64_t>((int64_t)std::sqrt(tokens * (2. / 3.)), 64);
    const int64_t len = (std::max((tokens + cut - 1) / cut, least) + 15) / 16 * 16;
    if (len >= tokens) return false;
    p.seg_tokens = (int32_t)len;
    if (p.cu) {
        p.rows = (int32_t)(p.nseq + (tokens + len - 1) / len);
    } else {
        p.nseg = (int32_t)((tokens + len - 1) / len);
        p.rows = p.nseq * p.nseg;
    }
    return true;
}

static int64_t chain_blocks(const SelParams &p) { return ((int64_t)p.dim * p.N + 255) / 256; }
// Workgroups that cover the channels of one row of a step
static int64_t step_tiles(int dim, int N) {
    int npl, lpc;
    sel_shape(N, false, npl, lpc);
    return (dim + 256 / lpc - 1) / (256 / lpc);
}

static size_t al256(int64_t v) { return (size_t)((v + 255) / 256 * 256); }

size_t sel_segment_bytes(const SelParams &p) {
    return al256((int64_t)p.rows * p.dim * p.N * 4) + al256((int64_t)p.rows * p.dim * 4) +
           (p.cu ? al256((int64_t)p.rows * 16) + al256(((int64_t)p.nseq + 1) * 4) : 0);
}

void sel_segments(SelParams &p, char *ws) {
    p.seg_h = (float *)ws;
    ws += al256((int64_t)p.rows * p.dim * p.N * 4);
    p.seg_s = (float *)ws;
    ws += al256((int64_t)p.rows * p.dim * 4);
    if (p.cu) {
        p.table = (const int4 *)ws;
        p.seq_row = (const int32_t *)(ws + al256((int64_t)p.rows * 16));
    }
}

void launch_sel_table(const SelParams &p, hipStream_t st) {
    if (p.table)
        hipLaunchKernelGGL(k_seltable, dim3(1), dim3(kSelTabThreads), 0, st, p, (int4 *)p.table, (int32_t *)p.seq_row);
}

void launch_sel_chain(const SelParams &p, const float *dh_out, hipStream_t st) {
    hipLaunchKernelGGL(k_selchain, dim3((uint32_t)(chain_blocks(p) * p.nseq), p.seg_g ? 2 : 1), dim3(256), 0, st, p, dh_out);
}

mamba3_status launch_selective_scan(const mamba3_selective_scan_args *a, hipStream_t st) {
    SelParams p = sel_params(a);
    const bool segments = sel_plan(p, false), f32 = a->dtype == MAMBA3_F32;
    const Access acc = sel_access(p, f32 ? 4 : 2);
    if (segments) {
        sel_segments(p, (char *)a->workspace);
        launch_sel_table(p, st);
        if (f32) scan_go<float, PART>(p, acc, st);
        else scan_go<bf16, PART>(p, acc, st);
        launch_sel_chain(p, nullptr, st);
    }
    if (f32) scan_go<float, FULL>(p, acc, st);
    else scan_go<bf16, FULL>(p, acc, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

int64_t selective_workgroups(const mamba3_selective_scan_args *a, bool back) {
    SelParams p = sel_params(a);
    const bool segments = sel_plan(p, back);
    int64_t n = (int64_t)p.rows * p.tiles * p.G;
    if (segments) n = std::max(n, chain_blocks(p) * p.nseq);
    return back ? std::max(n, sel_reduce_blocks(p) + sel_sum_blocks(p)) : n;
}

int64_t selective_step_workgroups(const mamba3_selective_step_args *a) { return (int64_t)a->batch * step_tiles(a->dim, a->dstate); }

size_t selective_workspace_bytes(const mamba3_selective_scan_args *a) {
    SelParams p = sel_params(a);
    return sel_plan(p, false) ? sel_segment_bytes(p) : 0;
}

void launch_sel_stored(const SelParams &p, int32_t dtype, Access acc, hipStream_t st) {
    const bool f32 = dtype == MAMBA3_F32;
    if (p.seg_h) {
        if (f32) scan_go<float, STORE_PART>(p, acc, st);
        else scan_go<bf16, STORE_PART>(p, acc, st);
    } else {
        if (f32) scan_go<float, STORE>(p, acc, st);
        else scan_go<bf16, STORE>(p, acc, st);
    }
}

template <typename T>
static void step_go(const mamba3_selective_step_args *a, const SelStepParams &p, hipStream_t st) {
    const int64_t es = sizeof(T);
    const bool al = p.N % 4 == 0 && quads(p.B, p.B_row, es) && quads(p.C, p.C_row, es);
#define M3_GO(NPL, LPC)                                                                                        \
    do {                                                                                                       \
        const int tiles = (int)step_tiles(p.dim, p.N);                                                         \
        const dim3 grid((uint32_t)a->batch * tiles);                                                           \
        if (al) hipLaunchKernelGGL((k_selstep<T, NPL, LPC, ALIGNED>), grid, dim3(256), 0, st, p, tiles);       \
        else hipLaunchKernelGGL((k_selstep<T, NPL, LPC, ANY>), grid, dim3(256), 0, st, p, tiles);              \
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
