// Short causal convolution (width 2..8) over every channel by itself, with SiLU: whole sequences,
// their backward, and one token with the state in place.
//
// Two products a tap and a byte or two a product: HBM-bound, so the kernels stream. A thread holds
// V consecutive channels (16 bytes of a token row) and walks kTok tokens of the flat token axis with
// the last W - 1 inputs in registers; its rows are loaded together before they are worked on. The W
// - 1 rows before a thread's first token are read twice (mostly from the caches): 3 of 16 at width 4.
// Sequence starts inside a thread's tokens reset the registers to conv_in's rows (a branch that is
// uniform across the wave, which shares its tokens). Rows of any length and alignment are read in the
// same pieces: a row's last thread takes the last V channels, some of them its neighbour's too, which
// both write alike (16384 tokens of 4095 channels, bf16: 63 us and 119 backward; channel by channel 80
// and 142; 4096 channels 55 and 112). The step, whose states are in place, cannot read a channel twice and
// goes channel by channel unless dim is a multiple of 4 (15.8 us for 1024 x 4095, 15.3 for 4096).
//
// 8 x 4096 tokens of 4096 channels, width 4, bf16: 112 us, 4.8 TB/s of what has to move (a large copy runs at
// 4.94); the backward of 16384 x 4096 packed tokens 105 us, 3.8 TB/s; a step of 128 rows 4.1 us by itself.
// Registers grow with the width, and eight channels a thread of bf16 leave four waves a SIMD at width 2, two at 4
// to 6, one at 7 and 8 (266 registers): 16384 x 4096 take 46, 48, 55, 62, 64, 82 and 94 us at width 2 .. 8 (fp32, four
// channels a thread, 99 .. 108 for twice the bytes), the backward 84, 87, 100, 106, 132, 142, 157 (fp32 181 .. 206).
#include <algorithm>
#include <type_traits>

#include "layer.h"

namespace m3 {

struct ConvParams {
    const void *x, *conv_in, *dy, *dconv_out;
    const float *w, *bias;
    void *y, *conv_out, *dx, *dconv_in;
    float *part;                        // partial sums of dweight and dbias: [blocks][W + 1][dim]
    int64_t x_row, dy_row;
    const int32_t *cu;
    int32_t nseq, seqlen, total, dim, silu;
    int32_t main_blocks, chan_blocks;   // workgroups that walk tokens; those that cover the channels
};

constexpr int kTok = 16;                // tokens of a thread

// The sequence that holds token t, and its tokens [a, b). Tokens before the first sequence count as one
// of their own with number -1; those behind the last have no end.
struct SeqAt {
    int s, a, b;
};
// The tokens [first, second) that belong to sequences.
__device__ __forceinline__ int2 live_tokens(const ConvParams &p) {
    if (!p.cu) return make_int2(0, p.total);
    return make_int2(min(max(p.cu[0], 0), p.total), min(max(p.cu[p.nseq], 0), p.total));
}
__device__ __forceinline__ SeqAt seq_of(const ConvParams &p, int t) {
    SeqAt q;
    if (!p.cu) {
        q.s = t / p.seqlen;
        q.a = q.s * p.seqlen;
        q.b = q.a + p.seqlen;
        return q;
    }
    if (t < p.cu[0]) {
        q.s = -1;
        q.a = t;
        q.b = min(p.cu[0], p.total);
        return q;
    }
    int lo = 0, hi = p.nseq - 1;        // the last sequence that starts at or before t
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (p.cu[m] <= t) lo = m;
        else hi = m - 1;
    }
    q.s = lo;
    packed_bounds(p.cu, lo, p.total, q.a, q.b);
    return q;
}
__device__ __forceinline__ SeqAt bounds_of(const ConvParams &p, int s) {
    SeqAt q;
    q.s = s;
    if (p.cu) {
        packed_bounds(p.cu, s, p.total, q.a, q.b);
    } else {
        q.a = s * p.seqlen;
        q.b = q.a + p.seqlen;
    }
    return q;
}
// The sequence after token t reached the end of q (the next one that is not empty).
__device__ __forceinline__ void next_seq(const ConvParams &p, int t, SeqAt &q) {
    while (t >= q.b) {
        if (q.s + 1 >= p.nseq) {        // behind the last sequence
            q.a = t;
            q.b = INT32_MAX;
            return;
        }
        q = bounds_of(p, q.s + 1);
    }
    q.a = min(q.a, t);
}

// V elements of a row as one load: global memory takes one of 8 or 16 bytes at any element.
template <typename T, int V> struct RawVec { typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T)))); };
template <typename T> struct RawVec<T, 1> { typedef T type; };

// V elements of a row, as fp32
template <typename T, int V>
__device__ __forceinline__ void load_vec(float (&o)[V], const T *row) {
    if constexpr (V == 1) {
        o[0] = to_f(row[0]);
    } else {
        const typename RawVec<T, V>::type v = *(const typename RawVec<T, V>::type *)row;
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = to_f(v[e]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *row, const float (&o)[V]) {
    if constexpr (V == 1) {
        row[0] = from_f<T>(o[0]);
    } else {
        typename RawVec<T, V>::type v;
#pragma unroll
        for (int e = 0; e < V; e++) v[e] = from_f<T>(o[e]);
        *(typename RawVec<T, V>::type *)row = v;
    }
}
template <typename T, int V>
__device__ __forceinline__ float raw_f(const typename RawVec<T, V>::type &v, int e) {
    if constexpr (V == 1) return to_f(v);
    else return to_f(v[e]);
}

// Input tau of sequence q, channels c ..: its token, or a row of conv_in before the start.
template <typename T, int W, int V>
__device__ __forceinline__ void hist_vec(const ConvParams &p, const SeqAt &q, int tau, int c, float (&o)[V]) {
    const int j = W - 1 + tau - q.a;
    if (tau >= q.a) {
        load_vec<T, V>(o, (const T *)p.x + (int64_t)tau * p.x_row + c);
    } else if (p.conv_in && j >= 0 && q.s >= 0) {
        load_vec<T, V>(o, (const T *)p.conv_in + ((int64_t)q.s * (W - 1) + j) * p.dim + c);
    } else {
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = 0.f;
    }
}

// conv_out: element i of [S, W-1, D]
template <typename T, int W>
__device__ __forceinline__ void conv_state(const ConvParams &p, int64_t i) {
    const int c = (int)(i % p.dim), j = (int)(i / p.dim % (W - 1)), s = (int)(i / p.dim / (W - 1));
    const SeqAt q = bounds_of(p, s);
    float o[1];
    hist_vec<T, W, 1>(p, q, q.b - (W - 1) + j, c, o);
    ((T *)p.conv_out)[i] = from_f<T>(o[0]);
}

// 4 waves, each with its own tokens, the same 64 * V channels; the blocks behind the main ones write
// conv_out.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void k_conv(ConvParams p) {
    if ((int)blockIdx.x >= p.main_blocks) {
        const int64_t n = (int64_t)p.nseq * (W - 1) * p.dim;
        const int64_t i = (int64_t)(blockIdx.x - p.main_blocks) * 256 + threadIdx.x;
        if (i < n) conv_state<T, W>(p, i);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int from = (int)(blockIdx.x % p.chan_blocks) * 64 * V + lane * V;
    const int64_t first = ((int64_t)(blockIdx.x / p.chan_blocks) * 4 + wave) * kTok;
    if (first >= p.total || from >= p.dim) return;
    const int c = min(from, p.dim - V);  // a row's last thread: its last V channels, some also its neighbour's
    const int t0 = __builtin_amdgcn_readfirstlane((int)first);
    const T *x = (const T *)p.x + c;
    typename RawVec<T, V>::type raw[kTok];
#pragma unroll
    for (int i = 0; i < kTok; i++)
        raw[i] = *(const typename RawVec<T, V>::type *)(x + (int64_t)min(t0 + i, p.total - 1) * p.x_row);
    const int2 live = live_tokens(p);
    SeqAt q = seq_of(p, t0);
    next_seq(p, t0, q);
    float w[W][V], bias[V], win[W][V];   // win[j]: input t - W + 1 + j
#pragma unroll
    for (int e = 0; e < V; e++) {
        bias[e] = p.bias ? p.bias[c + e] : 0.f;
#pragma unroll
        for (int j = 0; j < W; j++) w[j][e] = p.w[(int64_t)(c + e) * W + j];
    }
#pragma unroll
    for (int j = 1; j < W; j++) hist_vec<T, W, V>(p, q, t0 - W + j, c, win[j]);
    // INSIDE: the thread's tokens lie in one sequence, and nothing is asked of each
    auto walk = [&](auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
#pragma unroll
        for (int i = 0; i < kTok; i++) {
            const int t = t0 + i;
            if (!INSIDE) {
                if (t >= live.y) break;
                if (t >= q.b) {
                    next_seq(p, t, q);
#pragma unroll
                    for (int j = 1; j < W; j++) hist_vec<T, W, V>(p, q, t - W + j, c, win[j]);
                }
            }
            float o[V];
#pragma unroll
            for (int e = 0; e < V; e++) {
#pragma unroll
                for (int j = 0; j + 1 < W; j++) win[j][e] = win[j + 1][e];
                win[W - 1][e] = raw_f<T, V>(raw[i], e);
                float v = bias[e];
#pragma unroll
                for (int j = 0; j < W; j++) v += w[j][e] * win[j][e];
                o[e] = p.silu ? v * sigmoid_hw(v) : v;
            }
            if (INSIDE || t >= live.x) store_vec<T, V>((T *)p.y + (int64_t)t * p.dim + c, o);
        }
    };
    if (q.s >= 0 && t0 + kTok <= min(q.b, live.y)) walk(std::integral_constant<bool, true>());
    else walk(std::integral_constant<bool, false>());
}

// SiLU's derivative at v
__device__ __forceinline__ float silu_grad(float v) {
    const float s = sigmoid_hw(v);
    return s + v * s * (1.f - s);
}

// dconv_in, element i of [S, W-1, D]: place k of the history reaches the outputs 0 .. k.
template <typename T, int W>
__device__ __forceinline__ void conv_state_grad(const ConvParams &p, int64_t i) {
    const int c = (int)(i % p.dim), k = (int)(i / p.dim % (W - 1)), s = (int)(i / p.dim / (W - 1));
    const SeqAt q = bounds_of(p, s);
    const int len = q.b - q.a;
    float g = 0.f;
    for (int t = 0; t <= k && t < len; t++) {
        float v = p.bias ? p.bias[c] : 0.f, h[1];
        for (int j = 0; j < W; j++) {
            hist_vec<T, W, 1>(p, q, q.a + t - W + 1 + j, c, h);
            v += p.w[(int64_t)c * W + j] * h[0];
        }
        const float dy = to_f(((const T *)p.dy)[(int64_t)(q.a + t) * p.dy_row + c]);
        g += p.w[(int64_t)c * W + k - t] * (p.silu ? dy * silu_grad(v) : dy);
    }
    if (k >= len && p.dconv_out)
        g += to_f(((const T *)p.dconv_out)[((int64_t)s * (W - 1) + k - len) * p.dim + c]);
    ((T *)p.dconv_in)[i] = from_f<T>(g);
}

// The backward walks kTokBwd tokens plus the W - 1 behind them: with e_t = dy_t act'(p_t),
// dx_tau = sum_j w[j] e_{tau + W - 1 - j}, so dx of a token is complete W - 1 tokens later and waits
// in registers until then. dweight's and dbias' sums over a workgroup's tokens go to `part`. Four
// channels a thread (8 bytes of bf16) leave three waves a SIMD. Tokens are taken in fours whose loads are in flight while
// the four before are worked on; INSIDE: the walk and its W - 1 neighbours on both sides lie in one
// sequence, which leaves no branch in it.
constexpr int kTokBwd = 32;

template <typename T, int W, int V>
struct ConvWalk {
    typedef typename RawVec<T, V>::type raw;
    float w[W][V], bias[V], win[W][V], pend[W][V];   // pend[j]: dx of token t - W + 1 + j so far
    float dw[W][V], db[V];

    template <bool INSIDE>
    __device__ __forceinline__ void run(const ConvParams &p, SeqAt q, int t0, int t1, int c) {
        constexpr int U = 4;
        const T *x = (const T *)p.x + c, *dy = (const T *)p.dy + c;
        const int end = t1 + W - 1;
        const int2 live = live_tokens(p);
        raw rx[U], rd[U];
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int64_t k = min(t + u, p.total - 1);
                rx[u] = *(const raw *)(x + k * p.x_row);
                rd[u] = *(const raw *)(dy + k * p.dy_row);
            }
        };
        fetch(t0);
        for (int tb = t0; tb < end; tb += U) {
            raw cx[U], cd[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                cx[u] = rx[u];
                cd[u] = rd[u];
            }
            if (tb + U < end) fetch(tb + U);
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int t = tb + u;
                if (t >= end) break;
                float e_t[V];
#pragma unroll
                for (int e = 0; e < V; e++) {
#pragma unroll
                    for (int j = 0; j + 1 < W; j++) pend[j][e] = pend[j + 1][e];
                    pend[W - 1][e] = 0.f;
                }
                if (INSIDE || t < p.total) {
                    if (!INSIDE && t >= q.b) {
                        next_seq(p, t, q);
#pragma unroll
                        for (int j = 1; j < W; j++) hist_vec<T, W, V>(p, q, t - W + j, c, win[j]);
                    }
#pragma unroll
                    for (int e = 0; e < V; e++) {
#pragma unroll
                        for (int j = 0; j + 1 < W; j++) win[j][e] = win[j + 1][e];
                        win[W - 1][e] = raw_f<T, V>(cx[u], e);
                        e_t[e] = INSIDE || (t >= live.x && t < live.y) ? raw_f<T, V>(cd[u], e) : 0.f;
                        if (p.silu) {
                            float v = bias[e];
#pragma unroll
                            for (int j = 0; j < W; j++) v += w[j][e] * win[j][e];
                            e_t[e] *= silu_grad(v);
                        }
                    }
                    const int pos = t - q.a;
#pragma unroll
                    for (int j = 0; j < W; j++)
                        if (INSIDE || pos >= W - 1 - j) {     // tap j's input is a token of this sequence
#pragma unroll
                            for (int e = 0; e < V; e++) pend[j][e] += w[j][e] * e_t[e];
                        }
                    if (t < t1 && (INSIDE || (t >= live.x && t < live.y))) {
#pragma unroll
                        for (int e = 0; e < V; e++) {
                            db[e] += e_t[e];
#pragma unroll
                            for (int j = 0; j < W; j++) dw[j][e] += e_t[e] * win[j][e];
                        }
                        const int k = t - q.b + (W - 1);      // the token's row of conv_out, if it has one
                        if (!INSIDE && p.dconv_out && k >= 0 && q.s >= 0) {
                            float o[V];
                            load_vec<T, V>(o, (const T *)p.dconv_out + ((int64_t)q.s * (W - 1) + k) * p.dim + c);
#pragma unroll
                            for (int e = 0; e < V; e++) pend[W - 1][e] += o[e];
                        }
                    }
                }
                const int tau = t - (W - 1);
                if (tau >= t0 && (INSIDE || (tau >= live.x && tau < live.y))) store_vec<T, V>((T *)p.dx + (int64_t)tau * p.dim + c, pend[0]);
            }
        }
    }
};

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvParams p) {
    if ((int)blockIdx.x >= p.main_blocks) {
        const int64_t n = (int64_t)p.nseq * (W - 1) * p.dim;
        const int64_t i = (int64_t)(blockIdx.x - p.main_blocks) * 256 + threadIdx.x;
        if (i < n) conv_state_grad<T, W>(p, i);
        return;
    }
    __shared__ float red[4][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c0 = (int)(blockIdx.x % p.chan_blocks) * 64 * V, from = c0 + lane * V;
    const int c = min(from, p.dim - V);  // as in the forward; a channel of two threads has equal sums in both
    const int blk = blockIdx.x / p.chan_blocks;
    const int64_t first = ((int64_t)blk * 4 + wave) * kTokBwd;
    ConvWalk<T, W, V> k;
#pragma unroll
    for (int e = 0; e < V; e++) {
        k.db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; j++) k.dw[j][e] = 0.f;
    }
    if (first < p.total && from < p.dim) {
        const int t0 = __builtin_amdgcn_readfirstlane((int)first);
        const int t1 = min(t0 + kTokBwd, p.total);
        SeqAt q = seq_of(p, t0);
        next_seq(p, t0, q);
#pragma unroll
        for (int e = 0; e < V; e++) {
            k.bias[e] = p.bias ? p.bias[c + e] : 0.f;
#pragma unroll
            for (int j = 0; j < W; j++) {
                k.w[j][e] = p.w[(int64_t)(c + e) * W + j];
                k.pend[j][e] = 0.f;
            }
        }
#pragma unroll
        for (int j = 1; j < W; j++) hist_vec<T, W, V>(p, q, t0 - W + j, c, k.win[j]);
        if (t0 - (W - 1) >= q.a && t1 + W - 1 <= q.b && t1 + W - 1 <= p.total) k.template run<true>(p, q, t0, t1, c);
        else k.template run<false>(p, q, t0, t1, c);
    }
    // the four waves' sums, in order
#pragma unroll
    for (int j = 0; j <= W; j++) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; e++)
            if (from < p.dim && c + e >= c0) red[wave][c - c0 + e] = j < W ? k.dw[j < W ? j : 0][e] : k.db[e];
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * V; i += 256)
            if (c0 + i < p.dim)
                p.part[((int64_t)blk * (W + 1) + j) * p.dim + c0 + i] =
                    (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
    }
}

// dweight [D, W] and dbias [D] from the partial sums of `blocks` workgroups: 16 columns of [W + 1][D] a
// workgroup, 16 threads over the rows of each.
__global__ __launch_bounds__(256) void k_conv_reduce(const float *part, int blocks, int dim, int W, float *dweight,
                                                     float *dbias) {
    __shared__ float red[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, n = dim * (W + 1), i = blockIdx.x * 16 + x;
    float s = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int b = y; b < blocks; b += 16) s += part[(int64_t)b * n + i];
    }
    red[y][x] = s;
    __syncthreads();
    if (y || i >= n) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k++) s += red[k][x];
    const int j = i / dim, c = i % dim;
    if (j < W) dweight[(int64_t)c * W + j] = s;
    else if (dbias) dbias[c] = s;
}

struct ConvStepParams {
    const void *x;
    const float *w, *bias;
    void *conv, *y;
    const int32_t *slots;
    int64_t x_row;
    int32_t batch, nslots, dim, silu;
};

// One token. Four channels a thread: 16-byte pieces of bf16 (eight channels, 32 weights a thread) took 21.5
// us at 1024 x 4096 where these take 15.2.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void k_conv_step(ConvStepParams p, int chan_blocks) {
    const int b = blockIdx.x / chan_blocks, c = ((int)(blockIdx.x % chan_blocks) * 256 + threadIdx.x) * V;
    if (c >= p.dim) return;
    // what does not wait for the slot first: a step is a few memory latencies long
    float w[V * W], bias[V], h[W][V], o[V];
    const float *wp = p.w + (int64_t)c * W;
#pragma unroll
    for (int i = 0; i < V * W; i++) w[i] = wp[i];
#pragma unroll
    for (int e = 0; e < V; e++) bias[e] = p.bias ? p.bias[c + e] : 0.f;
    load_vec<T, V>(h[W - 1], (const T *)p.x + b * p.x_row + c);
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nslots) return;
    }
    T *st = (T *)p.conv + slot * (W - 1) * p.dim + c;
#pragma unroll
    for (int j = 0; j + 1 < W; j++) load_vec<T, V>(h[j], st + (int64_t)j * p.dim);
#pragma unroll
    for (int e = 0; e < V; e++) {
        float v = bias[e];
#pragma unroll
        for (int j = 0; j < W; j++) v += w[e * W + j] * h[j][e];
        o[e] = p.silu ? v * sigmoid_hw(v) : v;
    }
#pragma unroll
    for (int j = 0; j + 1 < W; j++) store_vec<T, V>(st + (int64_t)j * p.dim, h[j + 1]);
    store_vec<T, V>((T *)p.y + (int64_t)b * p.dim + c, o);
}

namespace {

ConvParams conv_params(const mamba3_conv_args *a) {
    ConvParams p{};
    p.x = a->x; p.conv_in = a->conv_in; p.w = a->weight; p.bias = a->bias;
    p.y = a->y; p.conv_out = a->conv_out;
    p.x_row = a->x_row ? a->x_row : a->dim;
    p.cu = a->cu_seqlens;
    p.nseq = a->cu_seqlens ? a->nseq : a->batch;
    p.seqlen = a->seqlen;
    p.total = (int32_t)((int64_t)a->batch * a->seqlen);
    p.dim = a->dim; p.silu = a->silu;
    return p;
}

int64_t token_blocks(int64_t total, int tok) { return (total + 4 * tok - 1) / (4 * tok); }

// Channels of a thread: 16 bytes forward and 8 backward of bf16, 16 of fp32; single ones in rows of fewer.
int conv_vec(int dtype, int dim, bool back) {
    const int v = dtype == MAMBA3_F32 || back ? 4 : 8;
    return dim >= v ? v : 1;
}
int step_vec(int dim) { return dim % 4 == 0 ? 4 : 1; }
// Workgroups that walk tokens, and those of the states behind them
int64_t main_blocks(int64_t total, int dim, int v, bool back) {
    return token_blocks(total, back ? kTokBwd : kTok) * ((dim + 64 * v - 1) / (64 * v));
}
int64_t state_blocks(int64_t nseq, int width, int dim) { return (nseq * (width - 1) * dim + 255) / 256; }
int64_t step_blocks(int dim) { return (dim + 256 * step_vec(dim) - 1) / (256 * step_vec(dim)); }

#define M3_CONV_WIDTHS(W, CALL)     \
    switch (W) {                    \
        case 2: CALL(2); break;     \
        case 3: CALL(3); break;     \
        case 4: CALL(4); break;     \
        case 5: CALL(5); break;     \
        case 6: CALL(6); break;     \
        case 7: CALL(7); break;     \
        default: CALL(8); break;    \
    }

template <typename T, int V, bool BACK>
void conv_go(ConvParams p, int width, hipStream_t st) {
    p.chan_blocks = (p.dim + 64 * V - 1) / (64 * V);
    p.main_blocks = (int32_t)main_blocks(p.total, p.dim, V, BACK);
    const bool state = BACK ? p.dconv_in != nullptr : p.conv_out != nullptr;
    const int64_t extra = state ? state_blocks(p.nseq, width, p.dim) : 0;
    const dim3 grid((uint32_t)(p.main_blocks + extra));
    if (grid.x == 0) return;
#define M3_GO(W)                                                                                        \
    if constexpr (BACK) hipLaunchKernelGGL((k_conv_bwd<T, W, V>), grid, dim3(256), 0, st, p);           \
    else hipLaunchKernelGGL((k_conv<T, W, V>), grid, dim3(256), 0, st, p)
    M3_CONV_WIDTHS(width, M3_GO)
#undef M3_GO
}

template <typename T, int V>
void conv_step_go(const ConvStepParams &p, int width, hipStream_t st) {
    const int chan_blocks = (int)step_blocks(p.dim);
    const dim3 grid((uint32_t)((int64_t)p.batch * chan_blocks));
#define M3_GO(W) hipLaunchKernelGGL((k_conv_step<T, W, V>), grid, dim3(256), 0, st, p, chan_blocks)
    M3_CONV_WIDTHS(width, M3_GO)
#undef M3_GO
}

}  // namespace

int64_t conv_workgroups(const mamba3_conv_args *a, bool back) {
    const int64_t total = (int64_t)a->batch * a->seqlen, nseq = a->cu_seqlens ? a->nseq : a->batch;
    const int64_t walk = main_blocks(total, a->dim, conv_vec(a->dtype, a->dim, back), back) +
                         state_blocks(nseq, a->width, a->dim);
    return std::max(walk, back ? ((int64_t)a->dim * (a->width + 1) + 15) / 16 : 0);
}

int64_t conv_step_workgroups(const mamba3_conv_step_args *a) { return (int64_t)a->batch * step_blocks(a->dim); }

mamba3_status launch_conv(const mamba3_conv_args *a, hipStream_t st) {
    const ConvParams p = conv_params(a);
    const bool one = conv_vec(a->dtype, p.dim, false) == 1;
    if (a->dtype == MAMBA3_F32) {
        if (one) conv_go<float, 1, false>(p, a->width, st);
        else conv_go<float, 4, false>(p, a->width, st);
    } else {
        if (one) conv_go<bf16, 1, false>(p, a->width, st);
        else conv_go<bf16, 8, false>(p, a->width, st);
    }
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

size_t conv_bwd_workspace_bytes(const mamba3_conv_bwd_args *b) {
    const int64_t total = (int64_t)b->fwd.batch * b->fwd.seqlen;
    return (size_t)(token_blocks(total, kTokBwd) * (b->fwd.width + 1) * b->fwd.dim * 4);
}

mamba3_status launch_conv_bwd(const mamba3_conv_bwd_args *b, hipStream_t st) {
    const mamba3_conv_args *a = &b->fwd;
    ConvParams p = conv_params(a);
    p.dy = b->dy; p.dconv_out = b->dconv_out; p.dx = b->dx; p.dconv_in = b->dconv_in;
    p.dy_row = b->dy_row ? b->dy_row : a->dim;
    p.part = (float *)b->workspace;
    const bool one = conv_vec(a->dtype, p.dim, true) == 1;
    if (a->dtype == MAMBA3_F32) {
        if (one) conv_go<float, 1, true>(p, a->width, st);
        else conv_go<float, 4, true>(p, a->width, st);
    } else {
        if (one) conv_go<bf16, 1, true>(p, a->width, st);
        else conv_go<bf16, 4, true>(p, a->width, st);
    }
    const int64_t n = (int64_t)p.dim * (a->width + 1);
    hipLaunchKernelGGL(k_conv_reduce, dim3((uint32_t)((n + 15) / 16)), dim3(256), 0, st, p.part,
                       (int)token_blocks(p.total, kTokBwd), p.dim, a->width, b->dweight, b->dbias);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

mamba3_status launch_conv_step(const mamba3_conv_step_args *a, hipStream_t st) {
    ConvStepParams p{};
    p.x = a->x; p.w = a->weight; p.bias = a->bias; p.conv = a->conv; p.y = a->y;
    p.slots = a->slots; p.nslots = a->nslots;
    p.x_row = a->x_row ? a->x_row : a->dim;
    p.batch = a->batch; p.dim = a->dim; p.silu = a->silu;
    const bool one = step_vec(p.dim) == 1;
    if (a->dtype == MAMBA3_F32) {
        if (one) conv_step_go<float, 1>(p, a->width, st);
        else conv_step_go<float, 4>(p, a->width, st);
    } else {
        if (one) conv_step_go<bf16, 1>(p, a->width, st);
        else conv_step_go<bf16, 4>(p, a->width, st);
    }
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
