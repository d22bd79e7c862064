// Backward of the gated linear recurrence.
//
//   G_t = r_t + a_{t+1} G_{t+1},  r = dy SiLU(z)                     (dh_out at a sequence's end)
//   dv = u G,  dx = dv sigmoid(i),  di = dv x sigmoid'(i),  dz = dy h SiLU'(z)
//   decay   q = G a la (h_{t-1} - v a / u),  la = log a:  dgate = q (1 - s),  dw = sigmoid(w) / softplus(w) sum q
//   forget  q = G (h_{t-1} - v) (1 - s):                  dgate = q (1 - l) s, dl = sum q     (s = sigmoid(g))
//
// la / u tends to zero where the gate closes and u does, so q needs no case but u = 0 (or 1 - a^2 subnormal).
// Every run of W K tokens is a workgroup's by itself, with the tokens in registers: k_gate_part reads the
// inputs for the runs' (P, H, E), k_gate_chain turns them into the state that enters a run and the gradient that
// enters it from behind, and k_gate_bwd reads the inputs again, joins its waves' shares of the run in both
// directions, and goes over its tokens forwards for the states and backwards for the gradients. Nothing walks a
// sequence, so that one long sequence fills the GPU as a batch does, for a second read of the inputs.
//
// 8 x 2048 tokens of 4096 channels, decay, i, bf16: 326 us (k_gate_part 128, k_gate_chain 13, k_gate_bwd 185,
// k_gate_reduce 5), 1.55 GB, 4.8 TB/s: HBM-bound with the inputs read twice; read once the floor would be 193. A
// token's gradient needs the state from before its run and the gradient from behind it: the first read is for these. (A
// forward that kept its runs' states, 4 bytes a channel every 32 tokens, would save the states' part of it; it keeps
// nothing.) Runs walked by k_gate_bwd with the next tokens' loads in flight spilled; six waves a SIMD, sequences grouped for
// the last-level cache, and a first pass of one wave a run or with a prefetch were all slower.
#include <algorithm>

#include "gated.h"

namespace m3 {

// A workgroup's waves, a wave's tokens. 8 x 2048 tokens of 4096 channels: 325 us; 4 and 4 344, 16 and 4 442, 8 and 8
// (two waves a SIMD) 424; 1024 of 4096: 31.1, 34.7, 35.0, 33.3.
constexpr int kGateBwdWaves = 8, kGateBwdTokens = 4;
constexpr int kGateBwdOccupancy = 4;                      // waves a SIMD: two workgroups a CU
// Rows join those around them by themselves, without k_gate_chain and its launch, where a sequence has at most 32 and
// all are at most 2048 workgroups: 512 tokens of 1024 channels 22.4 us (with the chain 24.7), 4 x 512 of 2048 30.5 (32.9),
// 1024 of 4096 31.1 (32.4). Reading the others' runs in every row costs more with more of them: 8 x 1024 of 4096, 8192
// workgroups, 182 (172); 8 x 2048 of 4096 399 (325), 2048 of 4096 56.6 (50.1).
constexpr int kGateAlone = 32, kGateAloneGroups = 2048;

template <typename T, int V, int FORM, bool IG, bool ZG>
__global__ __launch_bounds__(64 * kGateBwdWaves, kGateBwdOccupancy) void k_gate_bwd(GateParams p) {
    constexpr int W = kGateBwdWaves, K = kGateBwdTokens;
    __shared__ piece32<V> join[3][W][64], around[4][W][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the last runs first: they were read last and may still lie in the cache
    const int r = p.first - (int)(blockIdx.x / p.tiles);
    const GateRow row = gate_row(p, r);
    const int c = (blockIdx.x % p.tiles * 64 + lane) * V, cc = min(c, p.dim - V);
    const int64_t o = (int64_t)r * p.dim + cc;
    if (row.seq < 0 || row.t0 >= row.t1) {              // no tokens: nothing but a row of partial sums
        if (wave == 0 && c < p.dim) {
#pragma unroll
            for (int e = 0; e < V; e++) {
                if (p.part) p.part[o + e] = 0.f;
                if (p.alone && p.dh_in && row.seq >= 0) {
                    const int64_t h = (int64_t)row.seq * p.dim + cc + e;
                    p.dh_in[h] = p.dh_out ? p.dh_out[h] : 0.f;
                }
            }
        }
        return;
    }
    const uint32_t at = cc * (uint32_t)sizeof(T);
    const int t = row.t0 + wave * K, n = min(row.t1 - t, K);        // the wave's tokens, or none
    GateRaw<T, V, FORM, IG, K> raw;
    piece<T, V> rd[K], rz[ZG ? K : 1];
    raw.template fetch<false>(p, t, row.t1, at);
    fetch_rows<T, V, K>(rd, p.dy, p.dy_row, t, row.t1, at);
    if constexpr (ZG) fetch_rows<T, V, K>(rz, p.z, p.z_row, t, row.t1, at);
    float c0[V], c1[V], s[V], g[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        c0[e] = p.channel[cc + e];
        c1[e] = gate_second<FORM>(c0[e]);
        const int64_t h = (int64_t)row.seq * p.dim + cc + e;
        s[e] = !p.alone ? p.H[o + e] : p.h_in ? p.h_in[h] : 0.f;
        g[e] = !p.alone ? p.E[o + e] : p.dh_out ? p.dh_out[h] : 0.f;
    }
    if (p.alone) {
        share_runs<V, W>(p, p.H, r - row.k, 1, row.k, cc, wave, around);
        share_runs<V, W>(p, p.E, r - row.k + row.n - 1, -1, row.n - 1 - row.k, cc, wave, around + 2);
    }
    // Of every token what both directions need: a, b = u v (then h_{t-1} less q's second term), r, and the factors of
    // G in dx, di, q and dgate. They take 64 registers, and computing them again would take a third more
    // operations.
    float a[K][V], h[K][V], d[K][V], fx[K][V], fi[K][V], fq[K][V], fh[K][V], fg[K][V], P[V], H[V], E[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        P[e] = 1.f;
        H[e] = E[e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; k++)
        if (k < n)
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float x = to_f(raw.x[k][e]);
                float sg, ng, si = 1.f, ni = 0.f, u;
                sigmoids(to_f(raw.g[k][e]), sg, ng);
                if (IG) sigmoids(to_f(raw.i[k][e]), si, ni);
                const float v = x * si;
                if constexpr (FORM == MAMBA3_GATE_DECAY) {
                    const float la = c0[e] * sg;
                    a[k][e] = __builtin_amdgcn_exp2f(c1[e] * sg);
                    const float w = one_minus_square(la, a[k][e]), i = w >= 0x1p-126f ? __builtin_amdgcn_rsqf(w) : 0.f;
                    u = w * i;
                    fq[k][e] = a[k][e] * la;
                    fh[k][e] = v * (a[k][e] * i);
                    fg[k][e] = ng;
                } else {
                    u = c1[e] * ng;
                    a[k][e] = fmaf(c1[e], sg, c0[e]);
                    fq[k][e] = ng;
                    fh[k][e] = v;
                    fg[k][e] = c1[e] * sg;
                }
                h[k][e] = u * v;
                fx[k][e] = u * si;
                if (IG) fi[k][e] = h[k][e] * ni;
                d[k][e] = to_f(rd[k][e]);
                if constexpr (ZG) {
                    const float z = to_f(rz[k][e]);
                    d[k][e] *= z * sigmoid_hw(z);
                }
                P[e] *= a[k][e];
                H[e] = fmaf(a[k][e], H[e], h[k][e]);
                E[e] = fmaf(P[e], d[k][e], E[e]);
            }
    join[0][wave][lane] = to_piece<V>(P);
    join[1][wave][lane] = to_piece<V>(H);
    join[2][wave][lane] = to_piece<V>(E);
    __syncthreads();
    if (p.alone) {
        join_runs<V, W>(s, around);
        join_runs<V, W>(g, around + 2);
        if (row.k == 0 && p.dh_in && wave == 0 && c < p.dim)
#pragma unroll
            for (int e = 0; e < V; e++) p.dh_in[(int64_t)row.seq * p.dim + cc + e] = fmaf(p.P[o + e], g[e], p.E[o + e]);
    }
#pragma unroll
    for (int w = 0; w < W - 1; w++)
        if (w < wave) {
            const piece32<V> A = join[0][w][lane], B = join[1][w][lane];
#pragma unroll
            for (int e = 0; e < V; e++) s[e] = fmaf(A[e], s[e], B[e]);
        }
#pragma unroll
    for (int w = W - 1; w > 0; w--)
        if (w > wave) {
            const piece32<V> A = join[0][w][lane], B = join[2][w][lane];
#pragma unroll
            for (int e = 0; e < V; e++) g[e] = fmaf(A[e], g[e], B[e]);
        }
#pragma unroll
    for (int k = 0; k < K; k++)
        if (k < n) {
            float dz[V];
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float was = s[e] - fh[k][e];
                s[e] = fmaf(a[k][e], s[e], h[k][e]);
                h[k][e] = was;
                if constexpr (ZG) {
                    const float v = to_f(rz[k][e]), q = sigmoid_hw(v);
                    dz[e] = to_f(rd[k][e]) * s[e] * (q * fmaf(v, 1.f - q, 1.f));
                }
            }
            if (ZG && p.dz && c < p.dim) store_piece<T, V>(p.dz, (int64_t)(t + k) * p.dim, at, dz);
        }
    float dw[V];
#pragma unroll
    for (int e = 0; e < V; e++) dw[e] = 0.f;
#pragma unroll
    for (int k = K - 1; k >= 0; k--)
        if (k < n) {
            float dx[V], di[V], dg[V];
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float G = d[k][e] + g[e], q = G * fq[k][e] * h[k][e];
                dw[e] += q;
                dx[e] = G * fx[k][e];
                dg[e] = q * fg[k][e];
                if (IG) di[e] = G * fi[k][e];
                g[e] = a[k][e] * G;
            }
            if (c < p.dim) {
                const int64_t to = (int64_t)(t + k) * p.dim;
                store_piece<T, V>(p.dx, to, at, dx);
                store_piece<T, V>(p.dgate, to, at, dg);
                if (IG && p.di) store_piece<T, V>(p.di, to, at, di);
            }
        }
    if (!p.part) return;
    __syncthreads();                                    // (the joins are read)
    join[0][wave][lane] = to_piece<V>(dw);
    __syncthreads();
    if (wave || c >= p.dim) return;
#pragma unroll
    for (int w = 1; w < W; w++) {
        const piece32<V> other = join[0][w][lane];
#pragma unroll
        for (int e = 0; e < V; e++) dw[e] += other[e];
    }
#pragma unroll
    for (int e = 0; e < V; e++) p.part[o + e] = dw[e];
}

// dweight from the runs' partial sums: 16 channels a workgroup, 16 threads over the rows of each.
template <int FORM>
__global__ __launch_bounds__(256) void k_gate_reduce(GateParams p, float *dweight) {
    __shared__ float red[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, c = blockIdx.x * 16 + x;
    float s = 0.f;
    if (c < p.dim) {
#pragma unroll 8
        for (int i = y; i < p.rows; i += 16) s += p.part[(int64_t)i * p.dim + c];
    }
    red[y][x] = s;
    __syncthreads();
    if (y || c >= p.dim) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += red[i][x];
    if constexpr (FORM == MAMBA3_GATE_DECAY) {
        // sigmoid(w) / softplus(w): 1 - e^w / 2 .. where both are e^w (a NaN passes the choice, not a minimum)
        const float w = p.weight[c], e = exp_full(w > 80.f ? 80.f : w);
        const float u = 1.f + e, l = fmaf(__builtin_amdgcn_logf(u), 0.69314718056f, (e - (u - 1.f)) * __builtin_amdgcn_rcpf(u));
        s *= w > 20.f ? 1.f / w : e < 0x1p-12f ? 1.f - 0.5f * e : e / (u * l);
    }
    dweight[c] = s;
}

namespace {

GateParams bwd_plan(const mamba3_gated_scan_bwd_args *b) {
    const mamba3_gated_scan_args *a = &b->fwd;
    GateParams p = gate_params(a);
    p.dy = b->dy;
    p.dh_out = b->dh_out;
    p.dy_row = b->dy_row ? b->dy_row : a->dim;
    p.dx = b->dx; p.dgate = b->dgate; p.di = b->di; p.dz = b->dz;
    p.dh_in = b->dh_in;
    p.seg_tokens = kGateBwdWaves * kGateBwdTokens;
    // (at least one run a sequence, also of a sequence without tokens)
    p.nseg = std::max((p.seqlen + p.seg_tokens - 1) / p.seg_tokens, 1);
    const int64_t runs = ((int64_t)p.total + p.seg_tokens - 1) / p.seg_tokens;
    const int64_t rows = p.cu ? p.nseq + runs : (int64_t)p.nseq * p.nseg;
    p.alone = (p.cu ? runs : p.nseg) <= kGateAlone && rows * p.tiles <= kGateAloneGroups;
    p.rows = (int32_t)std::min<int64_t>(rows, INT32_MAX);      // (more are refused for their workgroups)
    if (p.cu) p.nseg = 0;
    return p;
}

template <typename T>
void bwd_go(GateParams p, int form, hipStream_t st) {
    dim3 grid((uint32_t)((int64_t)p.rows * p.tiles));
#define M3_GO(V, FORM, IG, ZG) \
    hipLaunchKernelGGL((k_gate_part<T, V, FORM, IG, ZG, true, 4>), grid, dim3(256), 0, st, p)
    M3_GATE_DISPATCH(p, form, M3_GO);
#undef M3_GO
    launch_gate_chain(p, st);
    const int part = (int)(gate_most(64 * kGateBwdWaves) / p.tiles);                  // rows of a launch
    for (p.first = p.rows - 1; p.first >= 0; p.first -= part) {
        grid.x = (uint32_t)(std::min((int64_t)part, (int64_t)p.first + 1) * p.tiles);
#define M3_GO(V, FORM, IG, ZG) \
    hipLaunchKernelGGL((k_gate_bwd<T, V, FORM, IG, ZG>), grid, dim3(64 * kGateBwdWaves), 0, st, p)
        M3_GATE_DISPATCH(p, form, M3_GO);
#undef M3_GO
    }
}

}  // namespace

size_t gated_scan_bwd_workspace_bytes(const mamba3_gated_scan_bwd_args *b) {
    const GateParams p = bwd_plan(b);
    return p.rows ? gate_run_bytes(p, true) : 0;
}

int64_t gated_scan_bwd_workgroups(const mamba3_gated_scan_bwd_args *b) {
    const GateParams p = bwd_plan(b);
    return std::max((int64_t)p.rows * p.tiles, (int64_t)p.nseq * ((p.dim + 63) / 64));
}

mamba3_status launch_gated_scan_bwd(const mamba3_gated_scan_bwd_args *b, hipStream_t st) {
    GateParams p = bwd_plan(b);
    const int form = b->fwd.form;
    gate_runs(p, (char *)b->workspace, true);
    if (!b->dweight) p.part = nullptr;
    if (p.rows) {
        launch_gate_table(p, st);
        if (b->fwd.dtype == MAMBA3_F32) bwd_go<float>(p, form, st);
        else bwd_go<bf16>(p, form, st);
    }
    if (b->dweight) {
        const dim3 grid((uint32_t)((p.dim + 15) / 16));
        if (form == MAMBA3_GATE_DECAY) hipLaunchKernelGGL(k_gate_reduce<MAMBA3_GATE_DECAY>, grid, dim3(256), 0, st, p, b->dweight);
        else hipLaunchKernelGGL(k_gate_reduce<MAMBA3_GATE_FORGET>, grid, dim3(256), 0, st, p, b->dweight);
    }
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
