// Shared parts of the gated linear recurrence's forward and backward kernels.
//
// A wave holds 64 V consecutive channels, V a lane (2 but where gate_two says 1, so that a token's load is 4 bytes of
// bf16 or 8 of fp32 a lane, at any element), and K consecutive tokens of each in registers.
// The recurrence over a run of tokens is h -> P h + H with P the product of their decays and H their
// state from zero; the gradient's, from its end to its start, is g -> P g + E with the same P. Runs are joined in
// order: (P2 P1, P2 H1 + H2) and (P1 P2, E1 + P1 E2).
#pragma once

#include <type_traits>

#include "layer.h"

namespace m3 {

struct GateParams {
    const void *x, *gate, *i, *z, *dy;
    const float *weight, *h_in, *dh_out;
    void *y, *dx, *dgate, *di, *dz;
    float *h_out, *dh_in;
    int64_t x_row, gate_row, i_row, z_row, dy_row;    // elements from one token to the next
    const int32_t *cu;          // packed batches, or NULL
    int32_t nseq;               // sequences (padded: the batch)
    int32_t seqlen, total;      // tokens of a padded sequence, tokens of the batch
    int32_t dim, tiles;         // channels, workgroups that cover them
    float rate;
    // Rows of tokens that a workgroup takes: a sequence each (nseg 1), or its runs of seg_tokens tokens, nseg
    // of them in a padded sequence and as many as it needs in a packed one (nseg 0).
    int32_t rows, nseg, seg_tokens;
    int32_t alone;              // whether a row joins the runs around it itself, without k_gate_chain
    int32_t first;              // the launch's first row (k_gate_bwd, which goes down from it) or sequence (k_gate_chain)
    const int4 *table;          // the rows of a packed batch of more than 64 sequences, t0, t1, sequence (-1: no run)
    const int32_t *seq_row;     // [nseq + 1] a sequence's first row in the table
    float *P;                   // [rows][D] a run's product of decays
    float *H;                   // [rows][D] its last state from zero (after k_gate_chain: the state entering it); `alone`,
                                // forwards, h_in in the place of a sequence's last run
    float *E;                   // [rows][D] its share of the gradient that enters the run before (after: the one entering it)
    float *channel;             // [D] the channels' first constants, for the backward's second pass
    float *part;                // [rows][D] partial sums of dweight
    // One pass over the inputs (gated_pass.hip): what the runs publish
    uint64_t *runs, *checkpoints;
    uint32_t *counter;
};

// A row: its tokens, its sequence (-1: no row), its place among the sequence's rows and how many those are
struct GateRow {
    int t0, t1, seq, k, n;
};

// Row r, in scalar registers. Every lane of the wave takes part.
__device__ __forceinline__ GateRow gate_row(const GateParams &p, int r) {
    GateRow o;
    if (!p.cu) {
        o.seq = r / p.nseg;
        o.k = r % p.nseg;
        o.n = p.nseg;
        const int a = o.seq * p.seqlen;
        o.t0 = a + (int)min((int64_t)o.k * p.seg_tokens, (int64_t)p.seqlen);
        o.t1 = (int)min((int64_t)o.t0 + p.seg_tokens, (int64_t)a + p.seqlen);
    } else if (p.nseg == 1) {
        o.seq = r;
        o.k = 0;
        o.n = 1;
        packed_bounds(p.cu, r, p.total, o.t0, o.t1);
    } else if (p.table) {
        const int4 e = p.table[r];
        o.t0 = e.x;
        o.t1 = e.y;
        o.seq = e.z;
        const int s = max(e.z, 0), first = p.seq_row[s];
        o.k = r - first;
        o.n = p.seq_row[s + 1] - first;
    } else {
        // up to 64 sequences: every lane counts the rows of one
        const int s = threadIdx.x & 63;
        int a = 0, b = 0, n = 0;
        if (s < p.nseq) {
            packed_bounds(p.cu, s, p.total, a, b);
            n = max(1, (b - a + p.seg_tokens - 1) / p.seg_tokens);
        }
        int before = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(before, d, 64);
            if (s >= d) before += v;
        }
        before -= n;
        const uint64_t mine = __ballot(r >= before && r < before + n);
        const int from = mine ? __builtin_ctzll(mine) : 0;
        o.seq = mine ? from : -1;
        o.k = r - __builtin_amdgcn_readlane(before, from);
        // (decreasing entries may count more rows than there are)
        o.n = min(__builtin_amdgcn_readlane(n, from), p.rows - (r - o.k));
        o.t1 = __builtin_amdgcn_readlane(b, from);
        o.t0 = (int)min((int64_t)__builtin_amdgcn_readlane(a, from) + (int64_t)o.k * p.seg_tokens, (int64_t)o.t1);
        o.t1 = (int)min((int64_t)o.t0 + p.seg_tokens, (int64_t)o.t1);
    }
    o.t0 = __builtin_amdgcn_readfirstlane(o.t0);
    o.t1 = __builtin_amdgcn_readfirstlane(o.t1);
    o.seq = __builtin_amdgcn_readfirstlane(o.seq);
    o.k = __builtin_amdgcn_readfirstlane(o.k);
    o.n = __builtin_amdgcn_readfirstlane(o.n);
    return o;
}

// Whether a lane takes two channels. With an odd count the last lane takes the last two, one of which is the lane's before
// too: both compute and write the same, and no other workgroup does (which might read a state that this one replaced).
// 8 x 2048 tokens of 4095 channels, decay, i, bf16, with one channel a lane 164 us and backward 445; with two 144 and 397
// (4096 channels 117 and 325).
__host__ __device__ inline bool gate_two(int dim) { return dim % 2 == 0 || (dim > 1 && dim % 128 != 1); }

// V elements of a token, at any element: global memory takes loads and stores of 4 and 8 bytes there.
template <typename T, int V> struct PieceOf { typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T)))); };
template <typename T, int V> using piece = typename PieceOf<T, V>::type;

// The token's address is the same for all lanes and stays in scalar registers, the lane's offset has 32 bits.
template <typename T, int V>
__device__ __forceinline__ piece<T, V> load_piece(const void *base, int64_t elements, uint32_t lane_bytes) {
    return *(const piece<T, V> *)((const char *)((const T *)base + elements) + lane_bytes);
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(void *base, int64_t elements, uint32_t lane_bytes, const float (&v)[V]) {
    piece<T, V> o;
#pragma unroll
    for (int e = 0; e < V; e++) o[e] = from_f<T>(v[e]);
    *(piece<T, V> *)((char *)((T *)base + elements) + lane_bytes) = o;
}

// V floats of a lane in LDS
template <int V> struct Piece32Of { typedef float type __attribute__((ext_vector_type(V))); };
template <int V> using piece32 = typename Piece32Of<V>::type;
template <int V> __device__ __forceinline__ piece32<V> to_piece(const float (&v)[V]) {
    piece32<V> o;
#pragma unroll
    for (int e = 0; e < V; e++) o[e] = v[e];
    return o;
}

// e^v to an ulp or so for any v: what the product v log2(e) rounds away is put back. (Below -150, where e^v is zero, the
// product of a v far out would be infinite, and what it rounds away no number; a choice, which keeps a NaN.)
__device__ __forceinline__ float exp_full(float v) {
    v = v < -150.f ? -150.f : v;
    const float hi = v * kLog2e, lo = fmaf(v, kLog2e, -hi) + v * 1.92596299e-8f;
    const float e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e, lo * 0.69314718056f, e);
}

// A channel's constants. Decay: c0 = -rate softplus(w), c1 = c0 log2(e). Forget: c0 = l, c1 = 1 - l.
// softplus is taken exactly: an error in it is one of every decay of the channel, and adds up over the
// length of its memory.
template <int FORM> __device__ __forceinline__ float gate_second(float c0) {
    return FORM == MAMBA3_GATE_DECAY ? c0 * kLog2e : 1.f - c0;
}
template <int FORM>
__device__ __forceinline__ void gate_channel(const GateParams &p, int c, float &c0, float &c1) {
    if constexpr (FORM == MAMBA3_GATE_DECAY) {
        // (a choice and no minimum, which would take a NaN for 30)
        const float w = p.weight[c], e = exp_full(w > 30.f ? 30.f : w), u = 1.f + e, r = e - (u - 1.f);
        const float l = fmaf(__builtin_amdgcn_logf(u), 0.69314718056f, r * __builtin_amdgcn_rcpf(u));
        // below 2^-12 the logarithm of 1 + e is e - e^2 / 2, which log2 of a number next to 1 is not
        const float soft = w > 20.f ? w : e < 0x1p-12f ? fmaf(-0.5f * e, e, e) : l;
        // (kept finite: zero, a decay or a sigmoid, times an infinity would be no number)
        const float c = -p.rate * soft;
        c0 = c < -0x1p126f ? -0x1p126f : c;
    } else {
        c0 = p.weight ? p.weight[c] : 0.f;
    }
    c1 = gate_second<FORM>(c0);
}

// sigmoid(v) and 1 - sigmoid(v), both to their relative precision (e^-v leaves fp32's range below -88, where the
// sigmoid is zero)
__device__ __forceinline__ void sigmoids(float v, float &s, float &n) {
    const float e = exp_hw(-v);
    s = __builtin_amdgcn_rcpf(1.f + e);
    n = s > 0.f ? e * s : 1.f;
}

// 1 - e^{2 y} for y <= 0: a polynomial where the difference would cancel (fitted to (1 - e^{2 y}) / y on
// [-1/8, 0] with -2 at zero, within 2^-28 of it), the difference elsewhere
__device__ __forceinline__ float one_minus_square(float y, float a) {
    float s = fmaf(y, -0.24096550f, -0.66400212f);
    s = fmaf(y, s, -1.33322310f);
    s = fmaf(y, s, -1.99999857f);
    s = fmaf(y, s, -2.f);
    return y > -0.125f ? y * s : fmaf(-a, a, 1.f);
}

// A token's decay and what its input is taken by
template <int FORM>
__device__ __forceinline__ void gate_open(float g, float c0, float c1, float &a, float &u) {
    if constexpr (FORM == MAMBA3_GATE_DECAY) {
        const float s = sigmoid_hw(g);
        a = __builtin_amdgcn_exp2f(c1 * s);
        u = __builtin_amdgcn_sqrtf(one_minus_square(c0 * s, a));
    } else {
        float s, n;
        sigmoids(g, s, n);
        u = c1 * n;
        a = fmaf(c1, s, c0);
    }
}

// The rows of tokens t .. t + K - 1. WHOLE: all of them are before `end`, and a row's address is the one before it
// plus their distance; else those from `end` on are the one before it.
template <typename T, int V, int K, bool WHOLE = false>
__device__ __forceinline__ void fetch_rows(piece<T, V> (&o)[K], const void *base, int64_t row, int t, int end, uint32_t lane) {
    if constexpr (WHOLE) {
        const char *q = (const char *)((const T *)base + (int64_t)t * row);
#pragma unroll
        for (int k = 0; k < K; k++) {
            asm("" : "+s"(q));                           // (not K distances carried in scalar registers)
            o[k] = *(const piece<T, V> *)(q + lane);
            q += row * (int64_t)sizeof(T);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; k++) o[k] = load_piece<T, V>(base, (int64_t)min(t + k, end - 1) * row, lane);
    }
}

template <typename T, int V, int FORM, bool IG, int K>
struct GateRaw {
    piece<T, V> x[K], g[K], i[IG ? K : 1];

    // tokens t .. t + K - 1, those from `end` on as the one before it
    template <bool WHOLE>
    __device__ __forceinline__ void fetch(const GateParams &p, int t, int end, uint32_t lane) {
        fetch_rows<T, V, K, WHOLE>(g, p.gate, p.gate_row, t, end, lane);
        fetch_rows<T, V, K, WHOLE>(x, p.x, p.x_row, t, end, lane);
        if constexpr (IG) fetch_rows<T, V, K, WHOLE>(i, p.i, p.i_row, t, end, lane);
    }
    __device__ __forceinline__ void open(int k, const float (&c0)[V], const float (&c1)[V], float (&a)[V], float (&b)[V]) const {
#pragma unroll
        for (int e = 0; e < V; e++) {
            float u;
            gate_open<FORM>(to_f(g[k][e]), c0[e], c1[e], a[e], u);
            b[e] = u * to_f(x[k][e]);
            if (IG) b[e] *= sigmoid_hw(to_f(i[k][e]));
        }
    }
};

// The runs' P and H, and with BACK their E. A workgroup has a run of 64 V channels, W waves with
// consecutive shares of its tokens.
template <typename T, int V, int FORM, bool IG, bool ZG, bool BACK, int W>
__global__ __launch_bounds__(64 * W) void k_gate_part(GateParams p) {
    constexpr int K = sizeof(T) == 2 ? 8 : 4;
    __shared__ float join[3][W][V][64];
    const int r = blockIdx.x / p.tiles, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GateRow row = gate_row(p, r);
    const int c = (blockIdx.x % p.tiles * 64 + lane) * V, cc = min(c, p.dim - V);
    uint32_t at = cc * (uint32_t)sizeof(T);
    float c0[V], c1[V], P[V], H[V], E[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        gate_channel<FORM>(p, cc + e, c0[e], c1[e]);
        P[e] = 1.f;
        H[e] = E[e] = 0.f;
    }
    if (BACK && r == 0 && wave == 0 && c < p.dim)
#pragma unroll
        for (int e = 0; e < V; e++) p.channel[cc + e] = c0[e];
    if (row.seq < 0) return;
    if (!BACK && row.k == row.n - 1) {          // nothing takes up a last run's end: its place is the sequence's first state's
        if (p.alone && p.h_in && wave == 0 && c < p.dim)
#pragma unroll
            for (int e = 0; e < V; e++) p.H[(int64_t)r * p.dim + cc + e] = p.h_in[(int64_t)row.seq * p.dim + cc + e];
        return;
    }
    const int share = ((row.t1 - row.t0 + W - 1) / W + K - 1) / K * K;
    const int begin = (int)min((int64_t)row.t0 + (int64_t)wave * share, (int64_t)row.t1);
    const int end = (int)min((int64_t)begin + share, (int64_t)row.t1);
    // (a lane's offset that is unknown to the compiler, which would otherwise carry 64-bit addresses of every array)
    auto tokens = [&](auto whole, int t) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(whole)::value;
        GateRaw<T, V, FORM, IG, K> raw;
        piece<T, V> rd[BACK ? K : 1], rz[BACK && ZG ? K : 1];
        asm("" : "+v"(at));
        raw.template fetch<WHOLE>(p, t, end, at);
        if constexpr (BACK) fetch_rows<T, V, K, WHOLE>(rd, p.dy, p.dy_row, t, end, at);
        if constexpr (BACK && ZG) fetch_rows<T, V, K, WHOLE>(rz, p.z, p.z_row, t, end, at);
        __builtin_amdgcn_sched_barrier(0);               // all loads before the first token
#pragma unroll
        for (int k = 0; k < K; k++) {
            if (!WHOLE && t + k >= end) break;
            float a[V], b[V];
            raw.open(k, c0, c1, a, b);
#pragma unroll
            for (int e = 0; e < V; e++) {
                P[e] *= a[e];
                H[e] = fmaf(a[e], H[e], b[e]);
                if constexpr (BACK) {
                    float d = to_f(rd[k][e]);
                    if constexpr (ZG) {
                        const float z = to_f(rz[k][e]);
                        d *= z * sigmoid_hw(z);
                    }
                    E[e] = fmaf(P[e], d, E[e]);
                }
            }
        }
    };
    int t = begin;
    for (; t + K <= end; t += K) tokens(std::integral_constant<bool, true>(), t);
    if (t < end) tokens(std::integral_constant<bool, false>(), t);
#pragma unroll
    for (int e = 0; e < V; e++) {
        join[0][wave][e][lane] = P[e];
        join[1][wave][e][lane] = H[e];
        if (BACK) join[2][wave][e][lane] = E[e];
    }
    __syncthreads();
    if (wave || c >= p.dim) return;
#pragma unroll
    for (int w = 1; w < W; w++)
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float a = join[0][w][e][lane];
            if (BACK) E[e] = fmaf(P[e], join[2][w][e][lane], E[e]);
            H[e] = fmaf(a, H[e], join[1][w][e][lane]);
            P[e] *= a;
        }
    const int64_t o = (int64_t)r * p.dim + cc;
#pragma unroll
    for (int e = 0; e < V; e++) {
        p.P[o + e] = P[e];
        p.H[o + e] = H[e];
        if (BACK) p.E[o + e] = E[e];
    }
}

// The waves' shares of `count` rows on one side of row r (those from row `first` on, `step` apart, in the order in
// which they are joined), left in LDS: join[0] the products, join[1] the sums. The caller's barrier, then join_runs.
template <int V, int W>
__device__ __forceinline__ void share_runs(const GateParams &p, const float *X, int first, int step, int count, int cc, int wave,
                                           piece32<V> (*join)[W][64]) {
    const int lane = threadIdx.x & 63, share = (count + W - 1) / W;
    const int begin = min(wave * share, count), end = min(begin + share, count);
    float A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        A[e] = 1.f;
        B[e] = 0.f;
    }
    for (int k = begin; k < end; k++) {
        const int64_t q = (int64_t)(first + k * step) * p.dim + cc;
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float a = p.P[q + e];
            A[e] *= a;
            B[e] = fmaf(a, B[e], X[q + e]);
        }
    }
    join[0][wave][lane] = to_piece<V>(A);
    join[1][wave][lane] = to_piece<V>(B);
}
template <int V, int W>
__device__ __forceinline__ void join_runs(float (&v)[V], const piece32<V> (*join)[W][64]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int w = 0; w < W; w++) {
        const piece32<V> A = join[0][w][lane], B = join[1][w][lane];
#pragma unroll
        for (int e = 0; e < V; e++) v[e] = fmaf(A[e], v[e], B[e]);
    }
}

// Template arguments from a call's values: V, FORM, IG, ZG
#define M3_GATE_DISPATCH(p, form, CALL)                                        \
    do {                                                                       \
        const bool two_ = gate_two((p).dim), ig_ = (p).i, zg_ = (p).z;          \
        if ((form) == MAMBA3_GATE_DECAY) {                                     \
            if (two_) M3_GATE_D2(2, MAMBA3_GATE_DECAY, CALL);                  \
            else M3_GATE_D2(1, MAMBA3_GATE_DECAY, CALL);                       \
        } else {                                                               \
            if (two_) M3_GATE_D2(2, MAMBA3_GATE_FORGET, CALL);                 \
            else M3_GATE_D2(1, MAMBA3_GATE_FORGET, CALL);                      \
        }                                                                      \
    } while (0)
#define M3_GATE_D2(V, FORM, CALL)                                              \
    do {                                                                       \
        if (ig_ && zg_) CALL(V, FORM, true, true);                             \
        else if (ig_) CALL(V, FORM, true, false);                              \
        else if (zg_) CALL(V, FORM, false, true);                              \
        else CALL(V, FORM, false, false);                                      \
    } while (0)

// Workgroups of a launch: below 2^32 threads. A call may have 2^24 workgroups, so those of more than 256 threads go in parts.
constexpr int64_t gate_most(int threads) { return ((1LL << 32) - 1) / threads; }

GateParams gate_params(const mamba3_gated_scan_args *a);
// The parts of a call's workspace that the runs take, and the table's launch
size_t gate_run_bytes(const GateParams &p, bool back);
char *gate_runs(GateParams &p, char *ws, bool back);
void launch_gate_table(const GateParams &p, hipStream_t st);
void launch_gate_chain(GateParams p, hipStream_t st);
// The scan in one pass over runs of gate_pass_tokens tokens, and its workspace
int gate_pass_tokens(bool f32);
size_t gate_pass_bytes(const GateParams &p);
void launch_gate_pass(GateParams p, int32_t dtype, int form, char *ws, hipStream_t st);

}  // namespace m3
