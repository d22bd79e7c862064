// Gated linear recurrence of few long sequences in one pass over the inputs.
//
// A workgroup has a run of W K tokens of 64 V channels with all of its operands in registers. It publishes the
// run's product of decays and its state from zero, takes the state that enters it from the runs before it, and
// writes its outputs: every input is read once, where segments in two passes (gated.hip) read all but z twice.
// The state that enters run k is joined from the last checkpoint, the state behind every 8th run, and the
// published pairs of the up to 7 runs after that, in order: a fixed sequence of operations, whatever the timing.
//
// 32768 tokens of 2048 channels, bf16, with i, from a state (110 us at the rate of a large copy): 124 us, in
// two passes 167; six packed sequences of 16384 tokens of 4096 140, 218 in two passes; 2048 of 4096 29.3, 32.3. 16 waves
// and checkpoints every 8 runs: every 4 132 us, every 16 127; 8 waves (runs of 64 tokens, 16 to a checkpoint) 138,
// 4 waves 230. What is above the copy's time is the chain of checkpoints, one memory latency for 1024 tokens.
//
// Waiting. Runs are handed out by a counter, in an order in which every run a workgroup waits for has a smaller
// number: its workgroup has started, holds its CU until it ends, and waits only for still smaller ones, so the
// smallest unfinished one never waits and every wait ends. (A wait gives up after kPassPolls polls all the
// same and goes on with NaN, and a number behind the last ends, so that a workspace that another call overwrites neither
// hangs the GPU nor leads out of the arrays.) A
// published word is one 64-bit store that carries its own validity: a kernel fills the words with ones before,
// which no published word is. So no fence is needed, and nothing but these words crosses workgroups.
#include <algorithm>

#include "gated.h"

namespace m3 {

constexpr int kPassWaves = 16, kPassGroup = 8, kPassPolls = 1 << 20;

__global__ __launch_bounds__(256) void k_gate_clear(uint4 *words, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) words[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

__device__ __forceinline__ uint32_t plain_bits(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }
__device__ __forceinline__ void publish(uint64_t *to, float low, float high) {
    __hip_atomic_store(to, (uint64_t)plain_bits(high) << 32 | plain_bits(low), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void await(const uint64_t *from, float &low, float &high) {
    uint64_t v = 0x7fc000007fc00000ull;
    for (int i = 0; i < kPassPolls; i++) {
        const uint64_t now = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (now != ~0ull) {
            v = now;
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    low = __uint_as_float((uint32_t)v);
    high = __uint_as_float((uint32_t)(v >> 32));
}

template <typename T, int V, int FORM, bool IG, bool ZG>
__global__ __launch_bounds__(64 * kPassWaves, 8) void k_gate_pass(GateParams p) {
    constexpr int W = kPassWaves, K = sizeof(T) == 2 ? 8 : 4;
    __shared__ piece32<V> join[2][W][64], before[2][kPassGroup][64];
    __shared__ uint32_t number;
    if (threadIdx.x == 0) number = atomicAdd(p.counter, 1u) + 1u;       // (from ones on)
    __syncthreads();
    const uint32_t mine = __builtin_amdgcn_readfirstlane(number);
    if (mine >= gridDim.x) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // a padded batch's sequences side by side, a packed batch's rows in their order
    const int q = mine / p.tiles, tile = mine % p.tiles;
    const int r = p.cu ? q : q % p.nseq * p.nseg + q / p.nseq;
    const GateRow row = gate_row(p, r);
    if (row.seq < 0) return;
    const int c = (tile * 64 + lane) * V, cc = min(c, p.dim - V);
    uint32_t at = cc * (uint32_t)sizeof(T);
    const int t = row.t0 + wave * K, n = min(row.t1 - t, K);
    GateRaw<T, V, FORM, IG, K> raw;
    piece<T, V> rz[ZG ? K : 1];
    if (n == K) {
        raw.template fetch<true>(p, t, row.t1, at);
        if constexpr (ZG) fetch_rows<T, V, K, true>(rz, p.z, p.z_row, t, row.t1, at);
    } else if (n > 0) {
        raw.template fetch<false>(p, t, row.t1, at);
        if constexpr (ZG) fetch_rows<T, V, K>(rz, p.z, p.z_row, t, row.t1, at);
    }
    float c0[V], c1[V], s[V], a[K][V], b[K][V], P[V], H[V];
#pragma unroll
    for (int e = 0; e < V; e++) {
        gate_channel<FORM>(p, cc + e, c0[e], c1[e]);
        s[e] = p.h_in ? p.h_in[(int64_t)row.seq * p.dim + cc + e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; k++) raw.open(k, c0, c1, a[k], b[k]);
    if (n < K) {
#pragma unroll
        for (int k = 0; k < K; k++)
            if (k >= n)
#pragma unroll
                for (int e = 0; e < V; e++) {
                    a[k][e] = 1.f;
                    b[k][e] = 0.f;
                }
    }
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
    join[0][wave][lane] = to_piece<V>(P);
    join[1][wave][lane] = to_piece<V>(H);
    // h_in is here before anything is published: the last run may write h_out in its place
#pragma unroll
    for (int e = 0; e < V; e++) asm volatile("" : "+v"(s[e]));
    __syncthreads();
    // the whole run, published by the first wave unless a checkpoint stands for it or nothing follows
    const int place = row.k % kPassGroup, group = row.k - place;
    const bool follows = row.k < row.n - 1, checkpoint = place == kPassGroup - 1;
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < W; w++) {
            const piece32<V> A = join[0][w][lane], B = join[1][w][lane];
#pragma unroll
            for (int e = 0; e < V; e++) {
                H[e] = fmaf(A[e], H[e], B[e]);
                P[e] *= A[e];
            }
        }
        if (follows && !checkpoint && c < p.dim)
#pragma unroll
            for (int e = 0; e < V; e++) publish(p.runs + (int64_t)r * p.dim + cc + e, P[e], H[e]);
    }
    if (row.k > 0) {                                     // (the same for the workgroup)
        // a wave's share of what comes before: every W-th run of the group, the checkpoint by the last wave
        for (int j = wave; j < place; j += W) {
            float A[V], B[V];
#pragma unroll
            for (int e = 0; e < V; e++) await(p.runs + (int64_t)(r - place + j) * p.dim + cc + e, A[e], B[e]);
            before[0][j][lane] = to_piece<V>(A);
            before[1][j][lane] = to_piece<V>(B);
        }
        // (a sequence's checkpoints lie from its first row / 8 + its number on: no two share one)
        const int64_t first = (r - row.k) / kPassGroup + row.seq;
        if (wave == W - 1 && group > 0) {
            float A[V], B[V];
#pragma unroll
            for (int e = 0; e < V; e++) await(p.checkpoints + (first + group / kPassGroup - 1) * p.dim + cc + e, A[e], B[e]);
            before[0][kPassGroup - 1][lane] = to_piece<V>(A);
        }
        __syncthreads();
        if (group > 0) {
            const piece32<V> S = before[0][kPassGroup - 1][lane];
#pragma unroll
            for (int e = 0; e < V; e++) s[e] = S[e];
        }
        for (int j = 0; j < place; j++) {
            const piece32<V> A = before[0][j][lane], B = before[1][j][lane];
#pragma unroll
            for (int e = 0; e < V; e++) s[e] = fmaf(A[e], s[e], B[e]);
        }
    }
    if (wave == 0 && c < p.dim) {
        const int64_t first = (r - row.k) / kPassGroup + row.seq;
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float h = fmaf(P[e], s[e], H[e]);
            if (follows && checkpoint) publish(p.checkpoints + (first + group / kPassGroup) * p.dim + cc + e, h, 0.f);
            if (!follows && p.h_out) p.h_out[(int64_t)row.seq * p.dim + cc + e] = h;
        }
    }
#pragma unroll
    for (int w = 0; w < W - 1; w++)
        if (w < wave) {
            const piece32<V> A = join[0][w][lane], B = join[1][w][lane];
#pragma unroll
            for (int e = 0; e < V; e++) s[e] = fmaf(A[e], s[e], B[e]);
        }
    auto out = [&](int k) {
        float y[V];
#pragma unroll
        for (int e = 0; e < V; e++) {
            s[e] = fmaf(a[k][e], s[e], b[k][e]);
            y[e] = s[e];
            if constexpr (ZG) {
                const float v = to_f(rz[k][e]);
                y[e] *= v * sigmoid_hw(v);
            }
        }
        if (c < p.dim) store_piece<T, V>(p.y, (int64_t)(t + k) * p.dim, at, y);
    };
    if (n >= K) {
#pragma unroll
        for (int k = 0; k < K; k++) out(k);
    } else {
#pragma unroll
        for (int k = 0; k < K; k++)
            if (k < n) out(k);
    }
}

namespace {

template <typename T>
void pass_go(const GateParams &p, int form, hipStream_t st) {
    const dim3 grid((uint32_t)((int64_t)p.rows * p.tiles));
#define M3_GO(V, FORM, IG, ZG) \
    hipLaunchKernelGGL((k_gate_pass<T, V, FORM, IG, ZG>), grid, dim3(64 * kPassWaves), 0, st, p)
    M3_GATE_DISPATCH(p, form, M3_GO);
#undef M3_GO
}

size_t al256(int64_t v) { return (size_t)((v + 255) / 256 * 256); }
// Words that are cleared: the runs', the checkpoints', the counter
int64_t run_bytes(const GateParams &p) { return al256((int64_t)p.rows * p.dim * 8); }
int64_t checkpoint_bytes(const GateParams &p) { return al256(((int64_t)p.rows / kPassGroup + p.nseq + 1) * p.dim * 8); }

}  // namespace

int gate_pass_tokens(bool f32) { return kPassWaves * (f32 ? 4 : 8); }
size_t gate_pass_bytes(const GateParams &p) { return run_bytes(p) + checkpoint_bytes(p) + 256; }

void launch_gate_pass(GateParams p, int32_t dtype, int form, char *ws, hipStream_t st) {
    p.runs = (uint64_t *)ws;
    p.checkpoints = (uint64_t *)(ws + run_bytes(p));
    p.counter = (uint32_t *)(ws + run_bytes(p) + checkpoint_bytes(p));
    const int64_t n = (run_bytes(p) + checkpoint_bytes(p) + 256) / 16;
    hipLaunchKernelGGL(k_gate_clear, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, st, (uint4 *)ws, n);
    if (dtype == MAMBA3_F32) pass_go<float>(p, form, st);
    else pass_go<bf16>(p, form, st);
}

}  // namespace m3
