// Gated linear recurrence with one state a channel: whole sequences and one token.
//
//   h_t = a_t h_{t-1} + u_t v_t,  v = sigmoid(i) x,  y = h SiLU(z)
//   decay   a = exp(-rate softplus(w) sigmoid(g)), u = sqrt(1 - a^2)
//   forget  a = l + (1 - l) sigmoid(g),            u = 1 - a
//
// A few bytes and some 30 to 50 operations an element, so HBM-bound with the vector unit not far behind.
// A workgroup walks a row of tokens in rounds of W K tokens (W waves, K consecutive tokens each): the
// tokens' a and b = u v stay in registers while the waves exchange their runs' (P, H) through LDS with one
// barrier a round, every wave joins all of them in order (so that all carry the same state) and goes
// over its tokens again from the state that enters them: every input is read once. The next round's loads are
// in flight meanwhile. Where whole sequences are too few workgroups to fill the GPU they run in one pass
// over short runs (gated_pass.hip), or as segments: k_gate_part reads the inputs for the segments' (P, H), a row
// joins those before it or k_gate_chain does for all, and the walk starts from the states that enter the segments.
//
// 8 x 4096 tokens of 4096 channels, decay, i, bf16: 209 us a call among others, 1075 MB, 5.1 TB/s (a large copy runs at
// 4.88), the vector unit 77 % busy; in traces of single calls medians of 212 to 240, as the GPU's clocks go. A step of
// 256 x 4096 from slots takes 6.0 us, of 4 x 2048 3.8: a few memory latencies.
#include <algorithm>

#include "gated.h"
#include "selective.h"

namespace m3 {

template <typename T, int V, int FORM, bool IG, bool ZG, int W>
__global__ __launch_bounds__(64 * W) void k_gated(GateParams p) {
    constexpr int K = sizeof(T) == 2 ? 8 : 4;
    __shared__ piece32<V> join[2][2][W][64];
    const int r = blockIdx.x / p.tiles, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GateRow row = gate_row(p, r);
    if (row.seq < 0) return;
    const int c = (blockIdx.x % p.tiles * 64 + lane) * V, cc = min(c, p.dim - V);
    const uint32_t at = cc * (uint32_t)sizeof(T);
    GateRaw<T, V, FORM, IG, K> raw;
    piece<T, V> rz[ZG ? K : 1];
    auto fetch = [&](int64_t t64) {          // the wave's tokens from t on, if there are any
        if (t64 >= row.t1) return;
        const int t = (int)t64;
        if (t + K <= row.t1) raw.template fetch<true>(p, t, row.t1, at);
        else raw.template fetch<false>(p, t, row.t1, at);
        if constexpr (ZG) fetch_rows<T, V, K>(rz, p.z, p.z_row, t, row.t1, at);
    };
    fetch((int64_t)row.t0 + wave * K);
    float c0[V], c1[V], h[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        gate_channel<FORM>(p, cc + e, c0[e], c1[e]);
        // (of rows that join those before them, from k_gate_part: in place the sequence's last row overwrites h_in)
        const int from = p.alone ? r - row.k + row.n - 1 : r;
        h[e] = !p.h_in && (p.alone || !p.H) ? 0.f : p.H ? p.H[(int64_t)from * p.dim + cc + e] : p.h_in[(int64_t)row.seq * p.dim + cc + e];
    }
    int turn = 0;
    if (p.alone && row.k > 0) {                          // (the same for the workgroup)
        share_runs<V, W>(p, p.H, r - row.k, 1, row.k, cc, wave, join[1]);
        __syncthreads();
        join_runs<V, W>(h, join[1]);                     // (join[1] is written again behind the next barrier)
    }
    for (int64_t t = row.t0; t < row.t1; t += W * K, turn ^= 1) {
        const int mine = (int)min((int64_t)row.t1 - (t + wave * K), (int64_t)K);     // the wave's tokens, or none
        float a[K][V], b[K][V], P[V], H[V];
#pragma unroll
        for (int k = 0; k < K; k++) raw.open(k, c0, c1, a[k], b[k]);
        if (mine < K) {
#pragma unroll
            for (int k = 0; k < K; k++)
                if (k >= mine)
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        a[k][e] = 1.f;
                        b[k][e] = 0.f;
                    }
        }
        piece<T, V> z[ZG ? K : 1];
#pragma unroll
        for (int k = 0; k < (ZG ? K : 0); k++) z[k] = rz[k];
        fetch(t + W * K + wave * K);
#pragma unroll
        for (int e = 0; e < V; e++) {
            P[e] = a[0][e];
            H[e] = b[0][e];
#pragma unroll
            for (int k = 1; k < K; k++) {
                P[e] *= a[k][e];
                H[e] = fmaf(a[k][e], H[e], b[k][e]);
            }
        }
        join[turn][0][wave][lane] = to_piece<V>(P);
        join[turn][1][wave][lane] = to_piece<V>(H);
        __syncthreads();
        float s[V];
#pragma unroll
        for (int w = 0; w < W; w++) {
            if (w == wave)
#pragma unroll
                for (int e = 0; e < V; e++) s[e] = h[e];
            const piece32<V> A = join[turn][0][w][lane], B = join[turn][1][w][lane];
#pragma unroll
            for (int e = 0; e < V; e++) h[e] = fmaf(A[e], h[e], B[e]);
        }
        auto out = [&](int k) {
            float y[V];
#pragma unroll
            for (int e = 0; e < V; e++) {
                s[e] = fmaf(a[k][e], s[e], b[k][e]);
                y[e] = s[e];
                if constexpr (ZG) {
                    const float v = to_f(z[k][e]);
                    y[e] *= v * sigmoid_hw(v);
                }
            }
            if (c < p.dim) store_piece<T, V>(p.y, (t + wave * K + k) * p.dim, at, y);
        };
        if (mine >= K) {
#pragma unroll
            for (int k = 0; k < K; k++) out(k);
        } else {
#pragma unroll
            for (int k = 0; k < K; k++)
                if (k < mine) out(k);
        }
    }
    if (row.k == row.n - 1 && p.h_out && wave == 0 && c < p.dim)
#pragma unroll
        for (int e = 0; e < V; e++) p.h_out[(int64_t)row.seq * p.dim + cc + e] = h[e];
}

// The runs of a sequence joined: the state that enters each in place of H, and the gradient that enters
// it at its end in place of E, a workgroup for 64 channels of a sequence with 16 waves on consecutive runs.
// The gradient that enters the sequence's start is dh_in.
constexpr int kChainWaves = 16, kChainLoads = 8;
__global__ __launch_bounds__(64 * kChainWaves) void k_gate_chain(GateParams p) {
    __shared__ float join[2][kChainWaves][64];
    const int blocks = (p.dim + 63) / 64, s = p.first + blockIdx.x / blocks;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = blockIdx.x % blocks * 64 + lane, cc = min(c, p.dim - 1);
    int r0 = s * p.nseg, r1 = r0 + p.nseg;
    if (p.table) {
        r0 = p.seq_row[s];
        r1 = p.seq_row[s + 1];
    } else if (p.cu) {                                   // up to 64 sequences: every lane counts the rows of one
        int n = 0;
        if (lane < p.nseq) {
            int a, b;
            packed_bounds(p.cu, lane, p.total, a, b);
            n = max(1, (b - a + p.seg_tokens - 1) / p.seg_tokens);
        }
        int upto = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d, 64);
            if (lane >= d) upto += v;
        }
        // (decreasing entries may count more rows than there are)
        r1 = min(__builtin_amdgcn_readlane(upto, s), p.rows);
        r0 = min(r1, __builtin_amdgcn_readlane(upto, s) - __builtin_amdgcn_readlane(n, s));
    }
    const int share = (r1 - r0 + kChainWaves - 1) / kChainWaves;
    // (the gradient's runs are counted from the last)
    const bool back = blockIdx.y;
    float *X = back ? p.E : p.H;
    const int begin = min(wave * share, r1 - r0), end = min(begin + share, r1 - r0);
    auto index = [&](int k) { return (int64_t)(back ? r1 - 1 - k : r0 + k) * p.dim + cc; };
    float A = 1.f, B = 0.f;
    for (int k = begin; k < end; k += kChainLoads) {
        float a[kChainLoads], b[kChainLoads];
#pragma unroll
        for (int j = 0; j < kChainLoads; j++) {
            const int64_t q = index(min(k + j, end - 1));
            a[j] = p.P[q];
            b[j] = X[q];
        }
#pragma unroll
        for (int j = 0; j < kChainLoads; j++)
            if (k + j < end) {
                A *= a[j];
                B = fmaf(a[j], B, b[j]);
            }
    }
    join[0][wave][lane] = A;
    join[1][wave][lane] = B;
    __syncthreads();
    const float *first = back ? p.dh_out : p.h_in;
    float v = first ? first[(int64_t)s * p.dim + cc] : 0.f;
    for (int w = 0; w < wave; w++) v = fmaf(join[0][w][lane], v, join[1][w][lane]);
    if (c < p.dim)
        for (int k = begin; k < end; k += kChainLoads) {
            float a[kChainLoads], b[kChainLoads];
#pragma unroll
            for (int j = 0; j < kChainLoads; j++) {
                const int64_t q = index(min(k + j, end - 1));
                a[j] = p.P[q];
                b[j] = X[q];
            }
#pragma unroll
            for (int j = 0; j < kChainLoads; j++)
                if (k + j < end) {
                    X[index(k + j)] = v;
                    v = fmaf(a[j], v, b[j]);
                }
        }
    // (waves behind the last run hold the join of all of them, as the last does)
    if (back && p.dh_in && wave == kChainWaves - 1 && c < p.dim) p.dh_in[(int64_t)s * p.dim + c] = v;
}

// One token, four channels a thread
struct GateStepParams {
    const void *x, *gate, *i, *z;
    const float *weight;
    float *h;
    void *y;
    int64_t x_row, gate_row, i_row, z_row;
    const int32_t *slots;
    uint32_t n, quads;          // threads, those of a row
    int32_t nslots, dim;
    float rate;
};

template <typename T, int FORM>
__global__ __launch_bounds__(256) void k_gate_step(GateStepParams p) {
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;
    if (at >= p.n) return;
    const int b = at / p.quads, c = at % p.quads * 4, n = min(4, p.dim - c);
    // what does not wait for the slot first: a step is a few memory latencies long
    float x[4], g[4], i[4], z[4], w[4], h[4];
    auto load = [&](float (&o)[4], const void *base, int64_t row) {
        const T *q = (const T *)base + b * row + c;
        if (n == 4) {
            const piece<T, 4> v = *(const piece<T, 4> *)q;
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = to_f(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = e < n ? to_f(q[e]) : 0.f;
        }
    };
    auto load32 = [&](float (&o)[4], const float *q) {
        if (n == 4) {
            const piece<float, 4> v = *(const piece<float, 4> *)q;
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = e < n ? q[e] : 0.f;
        }
    };
    const int64_t slot = p.slots ? p.slots[b] : b;
    load(g, p.gate, p.gate_row);
    load(x, p.x, p.x_row);
    if (p.i) load(i, p.i, p.i_row);
    if (p.z) load(z, p.z, p.z_row);
#pragma unroll
    for (int e = 0; e < 4; e++) w[e] = 0.f;
    if (p.weight) load32(w, p.weight + c);
    if (p.slots && (slot < 0 || slot >= p.nslots)) return;
    float *hp = p.h + slot * p.dim + c;
    load32(h, hp);
    float y[4];
    GateParams q{};
    q.weight = w;
    q.rate = p.rate;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        float c0, c1, a, u;
        gate_channel<FORM>(q, e, c0, c1);
        gate_open<FORM>(g[e], c0, c1, a, u);
        float v = u * x[e];
        if (p.i) v *= sigmoid_hw(i[e]);
        h[e] = fmaf(a, h[e], v);
        y[e] = h[e];
        if (p.z) y[e] *= z[e] * sigmoid_hw(z[e]);
    }
    T *yp = (T *)p.y + (int64_t)b * p.dim + c;
    if (n == 4) {
        piece<float, 4> o;
        piece<T, 4> s;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            o[e] = h[e];
            s[e] = from_f<T>(y[e]);
        }
        *(piece<float, 4> *)hp = o;
        *(piece<T, 4> *)yp = s;
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (e < n) {
                hp[e] = h[e];
                yp[e] = from_f<T>(y[e]);
            }
    }
}

GateParams gate_params(const mamba3_gated_scan_args *a) {
    GateParams p{};
    p.x = a->x; p.gate = a->gate; p.i = a->i; p.z = a->z;
    p.weight = a->weight; p.h_in = a->h_in; p.y = a->y; p.h_out = a->h_out;
    p.x_row = a->x_row ? a->x_row : a->dim;
    p.gate_row = a->gate_row ? a->gate_row : a->dim;
    p.i_row = a->i_row ? a->i_row : a->dim;
    p.z_row = a->z_row ? a->z_row : a->dim;
    p.cu = a->cu_seqlens;
    p.nseq = a->cu_seqlens ? a->nseq : a->batch;
    p.seqlen = a->seqlen;
    p.total = a->batch * a->seqlen;
    p.dim = a->dim;
    const int channels = gate_two(a->dim) ? 128 : 64;
    p.tiles = (a->dim + channels - 1) / channels;
    p.rate = a->rate;
    p.rows = p.nseq;
    p.nseg = 1;
    p.seg_tokens = p.seqlen;
    return p;
}

namespace {

size_t al256(int64_t v) { return (size_t)((v + 255) / 256 * 256); }
constexpr int kGateAlone = 64;
constexpr int64_t kGatePass = 1 << 22;

// Whole sequences, or runs where those leave less than a workgroup a CU and are longer than two rounds of 16 waves.
// PASS (gated_pass.hip) reads every input once and needs two launches, but a sequence's runs wait for each other:
// about 2 us for every 1024 tokens, which 1024 channels of bf16 hide. SEGMENTS takes the others: segments of a
// multiple of 32 tokens (a round of four waves) that give 1024 workgroups, as long as a row can join those before it
// by itself (up to 64); else of a multiple of 128 (a round of 16 waves), which leave fewer to join.
// In us, decay form with i, bf16: one sequence of 512 tokens of 1024 channels whole 29.7, segments of 128 19.3, by
// this rule 17.3; 2048 of 4096 101, 39.6, 32.3, pass 29.3; 1024 of 4096 segments 21.6, pass 19.6; 4096 of 4096 58.5,
// pass 46.9; 32768 of 1024 115, pass 83; 65536 of 256 68, pass 126. Rows that join up to 0, 32, 64, 128 others by
// themselves: 2048 of 1024 24.5, 19.6, 18.0, 19.7; 8192 of 256 24.1, 22.9, 20.5, 21.6; 4 x 2048 of 512 20.0, 18.3, 18.5, 19.6.
enum Plan { WHOLE, SEGMENTS, PASS };
Plan fwd_plan(GateParams &p, bool f32) {
    const int64_t whole = (int64_t)p.nseq * p.tiles, tokens = p.cu ? p.total : p.seqlen;
    const int64_t run = gate_pass_tokens(f32);
    // Packed sequences differ in length, and whole the longest is the call's time: PASS up to 1536 workgroups, too. 20
    // sequences of 820 tokens on average of 4096 channels whole 177 us, so 139; 64 of 328 of 2048 128, 102; 60 of 1000 of
    // 4096 (1920 workgroups) 436, 459. (Up to 64 sequences: their rows are counted without a table.)
    const bool packed = p.cu && p.nseq <= 64 && whole < 1536 && p.total >= (int64_t)p.nseq * 2 * run;
    if (p.nseq == 0 || (whole >= (p.cu ? 512 : 256) && !packed) || tokens <= 256) return WHOLE;
    const int64_t cut = std::max<int64_t>(1024 / (p.cu ? p.tiles : whole), 2);
    auto length = [&](int64_t unit) { return ((tokens + cut - 1) / cut + unit - 1) / unit * unit; };
    auto count = [&](int64_t len) { return (tokens + len - 1) / len; };
    int64_t len = length(32);
    if (count(len) > kGateAlone) len = length(128);
    // (its workgroups have 1024 threads, and all are one launch: the runs' numbers are its own)
    const int64_t runs = p.cu ? p.nseq + count(run) : p.nseq * count(run);
    const bool pass = (!p.cu || p.nseq <= 64) && (int64_t)p.total * p.dim >= kGatePass && (p.cu ? 1 : (int64_t)p.nseq) * p.dim >= 1024 &&
                      runs * p.tiles <= gate_most(1024);
    if (!pass && whole >= 512) return WHOLE;
    if (pass) len = run;
    if (len >= tokens) return WHOLE;
    p.seg_tokens = (int32_t)len;
    p.nseg = (int32_t)count(len);
    p.rows = p.cu ? p.nseq + p.nseg : p.nseq * p.nseg;
    p.alone = p.nseg <= kGateAlone;                     // (of a packed sequence, at most)
    if (p.cu) p.nseg = 0;
    return pass ? PASS : SEGMENTS;
}

template <typename T>
void part_go(const GateParams &p, int form, hipStream_t st) {
    const dim3 grid((uint32_t)((int64_t)p.rows * p.tiles));
    // (as many waves as the scan has, see scan_go)
#define M3_GO(V, FORM, IG, ZG)                                                                                     \
    do {                                                                                                           \
        if (p.seg_tokens < 128) hipLaunchKernelGGL((k_gate_part<T, V, FORM, IG, false, false, 4>), grid, dim3(256), 0, st, p); \
        else hipLaunchKernelGGL((k_gate_part<T, V, FORM, IG, false, false, 16>), grid, dim3(1024), 0, st, p);      \
    } while (0)
    M3_GATE_DISPATCH(p, form, M3_GO);
#undef M3_GO
}

template <typename T>
void scan_go(const GateParams &p, int form, hipStream_t st) {
    const int64_t groups = (int64_t)p.rows * p.tiles;
    // 16 waves a row where there are few, or where packed sequences differ, so that the longest ends sooner; 4 where
    // a row is less than a round of 16. 40 x 400 tokens of 4096 channels, 4 waves 118 us, 16 150; packed 60 sequences of
    // 1000 on average 575 and 436, 40 of 200 103 and 94; 24 of 60 24 and 33, 100 of 60 of 1024 channels 28 and 38.
    const bool ragged = p.cu && p.nseg == 1 && p.nseq;
    const bool narrow = ragged ? groups >= 2048 || p.total / p.nseq < 128 : groups >= 1024 || p.seg_tokens < 128;
    const dim3 grid((uint32_t)groups);
#define M3_GO(V, FORM, IG, ZG)                                                                              \
    do {                                                                                                    \
        if (narrow)                                                                                         \
            hipLaunchKernelGGL((k_gated<T, V, FORM, IG, ZG, 4>), grid, dim3(64 * 4), 0, st, p);             \
        else hipLaunchKernelGGL((k_gated<T, V, FORM, IG, ZG, 16>), grid, dim3(64 * 16), 0, st, p);          \
    } while (0)
    M3_GATE_DISPATCH(p, form, M3_GO);
#undef M3_GO
}

}  // namespace

// Rows of packed sequences that no wave can count by itself
static bool gate_has_table(const GateParams &p) { return p.cu && p.nseg != 1 && p.nseq > 64; }

static size_t gate_table_bytes(const GateParams &p) {
    return gate_has_table(p) ? al256((int64_t)p.rows * 16) + al256(((int64_t)p.nseq + 1) * 4) : 0;
}
size_t gate_run_bytes(const GateParams &p, bool back) {
    return (back ? 4 : 2) * al256((int64_t)p.rows * p.dim * 4) + (back ? al256((int64_t)p.dim * 4) : 0) +
           gate_table_bytes(p);
}

char *gate_runs(GateParams &p, char *ws, bool back) {
    const size_t n = al256((int64_t)p.rows * p.dim * 4);
    p.P = (float *)ws;
    p.H = (float *)(ws += n);
    if (back) {
        p.E = (float *)(ws += n);
        p.part = (float *)(ws += n);
        p.channel = (float *)(ws += n);
        ws += al256((int64_t)p.dim * 4);
    } else {
        ws += n;
    }
    if (gate_has_table(p)) {
        p.table = (const int4 *)ws;
        p.seq_row = (const int32_t *)(ws + al256((int64_t)p.rows * 16));
        ws += gate_table_bytes(p);
    }
    return ws;
}

// The table is the selective scan's: the runs of a packed batch in the order of their tokens.
void launch_gate_table(const GateParams &p, hipStream_t st) {
    if (!p.table) return;
    SelParams q{};
    q.cu = p.cu;
    q.nseq = p.nseq;
    q.total = p.total;
    q.rows = p.rows;
    q.seg_tokens = p.seg_tokens;
    q.table = p.table;
    q.seq_row = p.seq_row;
    launch_sel_table(q, st);
}

static int64_t chain_blocks(const GateParams &p) { return (int64_t)p.nseq * ((p.dim + 63) / 64); }

void launch_gate_chain(GateParams p, hipStream_t st) {
    if (p.alone) return;
    const int64_t blocks = (p.dim + 63) / 64, part = gate_most(2 * 64 * kChainWaves) / blocks;     // sequences of a launch
    for (int64_t s = 0; s < p.nseq; s += part) {
        p.first = (int32_t)s;
        const dim3 grid((uint32_t)(std::min<int64_t>(part, p.nseq - s) * blocks), p.E ? 2 : 1);
        hipLaunchKernelGGL(k_gate_chain, grid, dim3(64 * kChainWaves), 0, st, p);
    }
}

mamba3_status launch_gated_scan(const mamba3_gated_scan_args *a, hipStream_t st) {
    GateParams p = gate_params(a);
    const bool f32 = a->dtype == MAMBA3_F32;
    const Plan plan = fwd_plan(p, f32);
    if (plan == PASS) {                                 // (at most 64 packed sequences: no table)
        launch_gate_pass(p, a->dtype, a->form, (char *)a->workspace, st);
        return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
    }
    if (plan == SEGMENTS) {
        gate_runs(p, (char *)a->workspace, false);
        launch_gate_table(p, st);
        if (f32) part_go<float>(p, a->form, st);
        else part_go<bf16>(p, a->form, st);
        launch_gate_chain(p, st);
    }
    if (f32) scan_go<float>(p, a->form, st);
    else scan_go<bf16>(p, a->form, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

size_t gated_scan_workspace_bytes(const mamba3_gated_scan_args *a) {
    GateParams p = gate_params(a);
    const Plan plan = fwd_plan(p, a->dtype == MAMBA3_F32);
    return plan == PASS ? gate_pass_bytes(p) : plan == SEGMENTS ? gate_run_bytes(p, false) : 0;
}

int64_t gated_scan_workgroups(const mamba3_gated_scan_args *a) {
    GateParams p = gate_params(a);
    const Plan plan = fwd_plan(p, a->dtype == MAMBA3_F32);
    const int64_t n = (int64_t)p.rows * p.tiles;
    if (plan == PASS) return std::max(n, (int64_t)(gate_pass_bytes(p) + 4095) / 4096);
    return std::max(n, plan == SEGMENTS ? chain_blocks(p) : 0);
}

int64_t gated_step_workgroups(const mamba3_gated_step_args *a) {
    return ((int64_t)a->batch * (((int64_t)a->dim + 3) / 4) + 255) / 256;
}

mamba3_status launch_gated_step(const mamba3_gated_step_args *a, hipStream_t st) {
    GateStepParams p{};
    p.x = a->x; p.gate = a->gate; p.i = a->i; p.z = a->z;
    p.weight = a->weight; p.h = a->h; p.y = a->y;
    p.x_row = a->x_row ? a->x_row : a->dim;
    p.gate_row = a->gate_row ? a->gate_row : a->dim;
    p.i_row = a->i_row ? a->i_row : a->dim;
    p.z_row = a->z_row ? a->z_row : a->dim;
    p.slots = a->slots; p.nslots = a->nslots; p.dim = a->dim; p.rate = a->rate;
    p.quads = (a->dim + 3) / 4;
    p.n = a->batch * p.quads;      // (below 2^32: fewer than 2^24 workgroups)
    const dim3 grid((uint32_t)gated_step_workgroups(a));
    const bool decay = a->form == MAMBA3_GATE_DECAY;
    if (a->dtype == MAMBA3_F32) {
        if (decay) hipLaunchKernelGGL((k_gate_step<float, MAMBA3_GATE_DECAY>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_gate_step<float, MAMBA3_GATE_FORGET>), grid, dim3(256), 0, st, p);
    } else {
        if (decay) hipLaunchKernelGGL((k_gate_step<bf16, MAMBA3_GATE_DECAY>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_gate_step<bf16, MAMBA3_GATE_FORGET>), grid, dim3(256), 0, st, p);
    }
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
