// Group norm of rows with an activation or gate, and its backward; a group's statistics are its row's own.
//
//   t = x or x SiLU(z),  n = (t - mean) / sqrt(var + eps),  v = n w + b,  y = v, SiLU(v) or v SiLU(z)
//   dt = r (dn - mean(dn) - n mean(dn n)),  dn = w dv,  dw = sum over rows of dv n,  db = sum of dv
//   (without the mean: n = t / sqrt(mean(t^2) + eps), and dt without mean(dn))
//
// Some 10 to 30 operations a value, so HBM-bound: rows are read once and kept in registers between their sums
// and their outputs, and a workgroup walks rows of the same columns with the next row's loads in flight, so that
// weights and, backwards, the sums over rows stay in registers too. A lane holds 8 consecutive values. Groups of up
// to 512 values take as many lanes as hold them (a power of two), several groups a wave, and sum inside
// the vector unit; longer ones take 2, 4, 8 or 16 waves.
//
// 32768 x 2048, 16 groups, gated, bf16: 80 us, 5.0 TB/s (a large copy runs at 4.88); its backward 138 us, 4.85 TB/s;
// 128 x 4096 in groups of 512 3.6 us. 2^25 values in groups of 64 37 us and 73 backward, of 512 38 and 74, of 600
// (two waves, 59 % of their lanes) 56 and 97, of 1024 43 and 78, of 4096 44 and 101, of 8192 51 and 110; of 4 (half a
// lane each) 82 and 137, of 100 54 and 107, of 513 75 and 123, where pieces cross groups and rows start at any value.
//
// The mean is taken off before squares are summed, and what its rounding left (the mean of the differences)
// once more, in the same sums as the squares: a group far from zero keeps its precision.
#include <algorithm>

#include "norm.h"

namespace m3 {

struct GnParams {
    const void *x, *z, *dy;
    const float *w, *b;
    void *y, *dx, *dz;
    float *part;                // [row blocks][2][dim] partial sums of dweight and dbias
    int64_t rows, x_row, z_row, dy_row;
    int32_t dim, groups, size;  // channels, groups, channels of a group
    int32_t lanes, tiles;       // lanes of a group (of one wave), workgroups that cover a row
    int32_t center;
    float eps, inv;             // 1 / size
};

constexpr bool gn_gated(int act) { return act == MAMBA3_GN_GATE || act == MAMBA3_GN_PREGATE; }

// Sums over a group, for every lane of it: over `lanes` consecutive lanes, or over the workgroup's WPG waves.
// `red`: two rows of LDS, used in turn, so that one barrier a sum is enough.
template <int WPG, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int lanes, float (*red)[N][16], int &turn) {
    if constexpr (WPG == 1) {
        auto add = [&](auto move) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = move(v[i]);
        };
        if (lanes > 1) add([](float a) { return a + dpp_move<0xB1>(a); });
        if (lanes > 2) add([](float a) { return a + dpp_move<0x4E>(a); });
        if (lanes > 4) add([](float a) { return a + dpp_move<0x141>(a); });
        if (lanes > 8) add([](float a) { return a + dpp_move<0x140>(a); });
        if (lanes > 32) {
            add([](float a) { return sum_across_rows(a); });
        } else if (lanes > 16) {
            add([](float a) {
                const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false, false);
                return __uint_as_float(s[0]) + __uint_as_float(s[1]);
            });
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) {
            v[i] = wave_sum(v[i]);
            if ((threadIdx.x & 63) == 0) red[turn][i][threadIdx.x >> 6] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < WPG; w++) v[i] += red[turn][i][w];
        }
        turn ^= 1;
    }
}

__device__ __forceinline__ float silu_of(float v, float s) { return v * s; }
__device__ __forceinline__ float dsilu_of(float v, float s) { return s * fmaf(v, 1.f - s, 1.f); }

// A lane's place: its group's first column, its own first value in the group, the group's values (0: no group)
struct GnLane {
    int col, c, n;
};

// A lane's 8 values of a row; those behind its group's end are not zero unless VEC. Rows of 8 values or more are
// read in full pieces at any element: one that crosses the row's end is taken from its last 8 values and shifted.
template <typename T, bool VEC>
__device__ __forceinline__ typename Raw8<T>::type gn_raw(const T *row, const GnLane &l, int dim) {
    if constexpr (VEC) {
        return raw8<T, true>(row + l.col, l.c, l.n);
    } else {
        typename Raw8<T>::type v;
        if (dim < kNV) return raw8<T, false>(row + l.col, l.c, l.n);
        const int from = min(l.col + l.c, dim - kNV), over = l.col + l.c - from;
        v = *(const typename Loose8<T>::type *)(row + from);
        if (over) {                                      // by 4, 2 and 1 values
            if constexpr (sizeof(T) == 2) {
                typedef uint32_t words __attribute__((ext_vector_type(4)));
                words u = __builtin_bit_cast(words, v);
                if (over & 4) u = words{u[2], u[3], 0, 0};
                if (over & 2) u = words{u[1], u[2], u[3], 0};
                if (over & 1)
                    u = words{u[0] >> 16 | u[1] << 16, u[1] >> 16 | u[2] << 16, u[2] >> 16 | u[3] << 16, u[3] >> 16};
                v = __builtin_bit_cast(typename Raw8<T>::type, u);
            } else {
                typedef typename Raw8<T>::type values;
                if (over & 4) v = values{v[4], v[5], v[6], v[7], 0, 0, 0, 0};
                if (over & 2) v = values{v[2], v[3], v[4], v[5], v[6], v[7], 0, 0};
                if (over & 1) v = values{v[1], v[2], v[3], v[4], v[5], v[6], v[7], 0};
            }
        }
        return v;
    }
}
// fp32 rows of dim values (weights and partial sums)
template <bool VEC>
__device__ __forceinline__ void gn_floats(float (&o)[kNV], const float *row, const GnLane &l, int dim) {
    const auto v = gn_raw<float, VEC>(row, l, dim);
#pragma unroll
    for (int e = 0; e < kNV; e++) o[e] = l.c + e < l.n ? v[e] : 0.f;
}
// The lane's values that its group has: 8, or the last one to seven as pieces of 4, 2 and 1.
template <typename T, bool VEC>
__device__ __forceinline__ void gn_store(T *row, const GnLane &l, const float (&o)[kNV]) {
    if constexpr (VEC) {
        store8<T, true>(row + l.col, l.c, l.n, o);
    } else {
        T *to = row + l.col + l.c;
        const int n = l.n - l.c;
        if (n >= kNV) {
            store8<T, false>(to, 0, kNV, o);
        } else if (n > 0) {
            typedef T four __attribute__((ext_vector_type(4), aligned(sizeof(T))));
            typedef T two __attribute__((ext_vector_type(2), aligned(sizeof(T))));
            four low = {from_f<T>(o[0]), from_f<T>(o[1]), from_f<T>(o[2]), from_f<T>(o[3])};
            const four high = {from_f<T>(o[4]), from_f<T>(o[5]), from_f<T>(o[6]), from_f<T>(o[7])};
            if (n & 4) {
                *(four *)to = low;
                to += 4;
                low = high;
            }
            if (n & 2) {
                *(two *)to = two{low[0], low[1]};
                to += 2;
                low[0] = low[2];
            }
            if (n & 1) *to = low[0];
        }
    }
}
template <int WPG>
__device__ __forceinline__ GnLane gn_lane(const GnParams &p, int tile) {
    GnLane l;
    const int lane = WPG == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int g = WPG == 1 ? tile * (64 / p.lanes) + lane / p.lanes : tile;
    l.c = (WPG == 1 ? lane % p.lanes : lane) * kNV;
    l.n = g < p.groups ? p.size : 0;
    l.col = g < p.groups ? g * p.size : 0;
    return l;
}

// t -> t - mean (in place, times a power of two where squares would leave fp32's range), and 1 / deviation of
// it. Returns that power. Where most of the differences is what the mean's rounding left (a group of equal values far from
// zero), the squares' mean less that of the differences has no digits, may be negative and says nothing of the values'
// size: the differences are the group from then on, until their mean is within the deviation. Each time it falls
// by 2^-20 or so: groups next to the end of fp32's range need up to eight rounds with eps 1e-5, twelve with the least one.
constexpr int kGnRounds = 16;
template <int WPG>
__device__ __forceinline__ float gn_stats(const GnParams &p, const GnLane &l, float (&t)[kNV], float &r,
                                          float (*red)[2][16], int &turn) {
    float k = 1.f;
    for (int round = 1;; round++) {
        float d[kNV], s[2] = {0.f, 0.f};
        if (p.center) {
#pragma unroll
            for (int e = 0; e < kNV; e++) s[0] += t[e];
            group_sums<WPG, 2>(s, p.lanes, red, turn);
            const float mean = s[0] * p.inv;
#pragma unroll
            for (int e = 0; e < kNV; e++) d[e] = l.c + e < l.n ? t[e] - mean : 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < kNV; e++) d[e] = t[e];
        }
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            s[0] += d[e];
            s[1] = fmaf(d[e], d[e], s[1]);
        }
        group_sums<WPG, 2>(s, p.lanes, red, turn);
        const float rest = p.center ? s[0] * p.inv : 0.f;
        const float mean = fmaf(s[1], p.inv, -rest * rest) + p.eps * k * k;
        // (scaled down, a group without deviation has lost eps: in its own size it has it)
        const bool rough = rest * rest > mean || (k < 1.f && mean < kLeastMean);
        const bool again = l.n && round < kGnRounds && (rough || (k == 1.f && !in_range(mean)));
        if (WPG == 1 ? !__any(again) : !again) {         // (the same for all lanes of a group)
            r = __builtin_amdgcn_rsqf(mean);
#pragma unroll
            for (int e = 0; e < kNV; e++) t[e] = l.c + e < l.n ? d[e] - rest : 0.f;
            return k;
        }
        if (again) {
            const float by = rough ? (k > 1.f ? 0x1p-100f : k < 1.f ? 0x1p80f : 1.f) : row_scale(mean);
            // (differences where they are small, values where their sums are too large)
            const bool take = rough || mean < kLeastMean;
#pragma unroll
            for (int e = 0; e < kNV; e++) t[e] = (take ? d[e] : t[e]) * by;
            k = rough ? 1.f : by;
        }
    }
}

template <typename T, int ACT, int WPG, bool VEC>
__global__ __launch_bounds__(WPG == 1 ? 256 : 64 * WPG) void k_gn(GnParams p) {
    __shared__ float red[2][2][16];
    constexpr int RPW = WPG == 1 ? 4 : 1;                // rows of a workgroup at once
    const GnLane l = gn_lane<WPG>(p, blockIdx.x % p.tiles);
    const int64_t step = (int64_t)(gridDim.x / p.tiles) * RPW;
    int64_t row = (int64_t)(blockIdx.x / p.tiles) * RPW + (WPG == 1 ? threadIdx.x >> 6 : 0);
    typename Raw8<T>::type rx, rz;
    auto fetch = [&](int64_t i) {
        rx = gn_raw<T, VEC>((const T *)p.x + i * p.x_row, l, p.dim);
        if (gn_gated(ACT)) rz = gn_raw<T, VEC>((const T *)p.z + i * p.z_row, l, p.dim);
    };
    if (row < p.rows) fetch(row);
    float w[kNV], b[kNV];
#pragma unroll
    for (int e = 0; e < kNV; e++) {
        w[e] = 1.f;
        b[e] = 0.f;
    }
    if (p.w) gn_floats<VEC>(w, p.w, l, p.dim);
    if (p.b) gn_floats<VEC>(b, p.b, l, p.dim);
    int turn = 0;
    for (; row < p.rows; row += step) {
        float t[kNV], f[kNV], r;
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            const bool in = VEC || l.c + e < l.n;        // (VEC: zeros behind the group's end)
            t[e] = in ? to_f(rx[e]) : 0.f;
            if constexpr (gn_gated(ACT)) {
                const float z = to_f(rz[e]);
                f[e] = z * sigmoid_hw(z);
                if (ACT == MAMBA3_GN_PREGATE) t[e] = in ? t[e] * f[e] : 0.f;
            }
        }
        if (row + step < p.rows) fetch(row + step);
        gn_stats<WPG>(p, l, t, r, red, turn);
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            float v = fmaf(t[e] * r, w[e], b[e]);
            if (ACT == MAMBA3_GN_SILU) v *= sigmoid_hw(v);
            if (ACT == MAMBA3_GN_GATE) v *= f[e];
            t[e] = v;
        }
        gn_store<T, VEC>((T *)p.y + row * p.dim, l, t);
    }
}

// Four waves a SIMD where that spills little: rows of odd lengths (groups of 100 bf16 values 133 -> 107 us), not fp32
// in whole pieces (groups of 2048 140 -> 149). Groups of 16 waves have no choice, 1024 threads are four waves a SIMD: of
// the 128 registers that leaves, whole pieces of bf16 spill 10 with a gate, of fp32 31 and, gated before, 22.
template <typename T, int ACT, int WPG, bool VEC>
__global__ __launch_bounds__(WPG == 1 ? 256 : 64 * WPG, sizeof(T) == 2 || !VEC ? 4 : 1) void k_gn_bwd(GnParams p) {
    __shared__ float red[2][2][16];
    __shared__ float4 join[WPG == 1 ? 4 * 256 : 1];
    constexpr int RPW = WPG == 1 ? 4 : 1;
    const GnLane l = gn_lane<WPG>(p, blockIdx.x % p.tiles);
    const int64_t rb = blockIdx.x / p.tiles, step = (int64_t)(gridDim.x / p.tiles) * RPW;
    int64_t row = rb * RPW + (WPG == 1 ? threadIdx.x >> 6 : 0);
    typename Raw8<T>::type rx, rz, rd;
    auto fetch = [&](int64_t i) {
        rx = gn_raw<T, VEC>((const T *)p.x + i * p.x_row, l, p.dim);
        rd = gn_raw<T, VEC>((const T *)p.dy + i * p.dy_row, l, p.dim);
        if (gn_gated(ACT)) rz = gn_raw<T, VEC>((const T *)p.z + i * p.z_row, l, p.dim);
    };
    if (row < p.rows) fetch(row);
    float w[kNV], b[kNV], dw[kNV], db[kNV];
#pragma unroll
    for (int e = 0; e < kNV; e++) {
        w[e] = 1.f;
        b[e] = dw[e] = db[e] = 0.f;
    }
    if (p.w) gn_floats<VEC>(w, p.w, l, p.dim);
    if (p.b) gn_floats<VEC>(b, p.b, l, p.dim);
    int turn = 0;
    for (; row < p.rows; row += step) {
        float t[kNV], d[kNV], r;
        typename Raw8<T>::type cx = rx, cz = rz;
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            const bool in = VEC || l.c + e < l.n;        // (VEC: zeros behind the group's end)
            t[e] = in ? to_f(rx[e]) : 0.f;
            d[e] = in ? to_f(rd[e]) : 0.f;
            if (ACT == MAMBA3_GN_PREGATE) {
                const float z = to_f(rz[e]);
                t[e] = in ? t[e] * (z * sigmoid_hw(z)) : 0.f;
            }
        }
        if (row + step < p.rows) fetch(row + step);
        const float k = gn_stats<WPG>(p, l, t, r, red, turn);
        float dz[kNV], s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            t[e] *= r;                                   // n
            if (ACT == MAMBA3_GN_SILU) {
                const float v = fmaf(t[e], w[e], b[e]);
                d[e] *= dsilu_of(v, sigmoid_hw(v));
            }
            if (ACT == MAMBA3_GN_GATE) {
                const float z = to_f(cz[e]), q = sigmoid_hw(z);
                dz[e] = d[e] * fmaf(t[e], w[e], b[e]) * dsilu_of(z, q);
                d[e] = VEC || l.c + e < l.n ? d[e] * silu_of(z, q) : 0.f;
            }
            db[e] += d[e];
            dw[e] = fmaf(d[e], t[e], dw[e]);
            d[e] *= w[e];
            s[0] += d[e];
            s[1] = fmaf(d[e], t[e], s[1]);
        }
        group_sums<WPG, 2>(s, p.lanes, red, turn);
        const float first = p.center ? s[0] * p.inv : 0.f, second = s[1] * p.inv, rk = r * k;
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            d[e] = rk * (d[e] - first - t[e] * second);
            if (ACT == MAMBA3_GN_PREGATE) {
                const float z = to_f(cz[e]), q = sigmoid_hw(z);
                dz[e] = d[e] * to_f(cx[e]) * dsilu_of(z, q);
                d[e] *= silu_of(z, q);
            }
        }
        gn_store<T, VEC>((T *)p.dx + row * p.dim, l, d);
        if (gn_gated(ACT) && p.dz) gn_store<T, VEC>((T *)p.dz + row * p.dim, l, dz);
    }
    if (!p.part) return;
    // one row of partial sums a workgroup: with several rows at once, those of its waves in order
    if constexpr (WPG == 1) {
        const int at = threadIdx.x;
        join[at] = make_float4(dw[0], dw[1], dw[2], dw[3]);
        join[256 + at] = make_float4(dw[4], dw[5], dw[6], dw[7]);
        join[512 + at] = make_float4(db[0], db[1], db[2], db[3]);
        join[768 + at] = make_float4(db[4], db[5], db[6], db[7]);
        __syncthreads();
        if (at >= 64) return;
#pragma unroll
        for (int v = 1; v < 4; v++) {
            const float4 a0 = join[at + 64 * v], a1 = join[256 + at + 64 * v];
            const float4 b0 = join[512 + at + 64 * v], b1 = join[768 + at + 64 * v];
            dw[0] += a0.x; dw[1] += a0.y; dw[2] += a0.z; dw[3] += a0.w;
            dw[4] += a1.x; dw[5] += a1.y; dw[6] += a1.z; dw[7] += a1.w;
            db[0] += b0.x; db[1] += b0.y; db[2] += b0.z; db[3] += b0.w;
            db[4] += b1.x; db[5] += b1.y; db[6] += b1.z; db[7] += b1.w;
        }
    }
    gn_store<float, VEC>(p.part + rb * 2 * p.dim, l, dw);
    gn_store<float, VEC>(p.part + (rb * 2 + 1) * p.dim, l, db);
}

// dweight (blockIdx.y 0) and dbias from `n` rows of partial sums: 16 columns a workgroup, 16 threads over the rows of
// each.
__global__ __launch_bounds__(256) void k_gn_reduce(const float *part, int n, int dim, float *dw, float *db) {
    __shared__ float red[16][17];
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, c = blockIdx.x * 16 + x;
    float s = 0.f;
    if (c < dim) {
#pragma unroll 8
        for (int i = y; i < n; i += 16) s += part[((int64_t)i * 2 + blockIdx.y) * dim + c];
    }
    red[y][x] = s;
    __syncthreads();
    if (y || c >= dim) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += red[i][x];
    out[c] = s;
}

namespace {

bool wide(const void *q, int64_t row, int64_t es) { return ((uintptr_t)q & 15u) == 0 && row * es % 16 == 0; }
int gn_waves(int size) { return size <= 512 ? 1 : size <= 1024 ? 2 : size <= 2048 ? 4 : size <= 4096 ? 8 : 16; }

GnParams gn_params(const mamba3_groupnorm_args *a) {
    GnParams p{};
    p.x = a->x; p.z = a->z; p.w = a->weight; p.b = a->bias; p.y = a->y;
    p.rows = a->rows; p.dim = a->dim; p.groups = a->groups; p.size = a->dim / a->groups;
    p.x_row = a->x_row ? a->x_row : a->dim;
    p.z_row = a->z_row ? a->z_row : a->dim;
    p.center = a->center;
    p.eps = a->eps;
    p.inv = (float)(1.0 / p.size);
    p.lanes = 1;
    while (p.lanes < 64 && p.lanes * kNV < p.size) p.lanes *= 2;
    p.tiles = gn_waves(p.size) == 1 ? (p.groups + 64 / p.lanes - 1) / (64 / p.lanes) : p.groups;
    return p;
}

// Workgroups that share the rows: 16 waves a CU for the backward, each of whose workgroups leaves partial sums, and
// twice that for the forward
int64_t gn_row_blocks(const GnParams &p, bool back) {
    const int w = gn_waves(p.size);
    const int64_t most = std::max<int64_t>((back ? 4096 : 8192) / (w == 1 ? 4 : w) / p.tiles, 1);
    return std::min<int64_t>(w == 1 ? (p.rows + 3) / 4 : p.rows, most);
}

template <typename T, int ACT, int WPG>
void gn_launch(const GnParams &p, bool vec, bool back, hipStream_t st) {
    const dim3 grid((uint32_t)(gn_row_blocks(p, back) * p.tiles)), block(WPG == 1 ? 256 : 64 * WPG);
    if (back) {
        if (vec) hipLaunchKernelGGL((k_gn_bwd<T, ACT, WPG, true>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((k_gn_bwd<T, ACT, WPG, false>), grid, block, 0, st, p);
    } else {
        if (vec) hipLaunchKernelGGL((k_gn<T, ACT, WPG, true>), grid, block, 0, st, p);
        else hipLaunchKernelGGL((k_gn<T, ACT, WPG, false>), grid, block, 0, st, p);
    }
}
template <typename T, int ACT>
void gn_act(const GnParams &p, bool vec, bool back, hipStream_t st) {
    const int w = gn_waves(p.size);
    if (w == 1) gn_launch<T, ACT, 1>(p, vec, back, st);
    else if (w == 2) gn_launch<T, ACT, 2>(p, vec, back, st);
    else if (w == 4) gn_launch<T, ACT, 4>(p, vec, back, st);
    else if (w == 8) gn_launch<T, ACT, 8>(p, vec, back, st);
    else gn_launch<T, ACT, 16>(p, vec, back, st);
}
template <typename T>
void gn_go(const GnParams &p, int act, bool vec, bool back, hipStream_t st) {
    if (act == MAMBA3_GN_NONE) gn_act<T, MAMBA3_GN_NONE>(p, vec, back, st);
    else if (act == MAMBA3_GN_SILU) gn_act<T, MAMBA3_GN_SILU>(p, vec, back, st);
    else if (act == MAMBA3_GN_GATE) gn_act<T, MAMBA3_GN_GATE>(p, vec, back, st);
    else gn_act<T, MAMBA3_GN_PREGATE>(p, vec, back, st);
}

}  // namespace

mamba3_status launch_groupnorm(const mamba3_groupnorm_args *a, hipStream_t st) {
    const GnParams p = gn_params(a);
    const int64_t es = a->dtype == MAMBA3_BF16 ? 2 : 4;
    const bool vec = p.size % 8 == 0 && wide(p.x, p.x_row, es) && wide(p.z, p.z_row, es) && wide(p.y, p.dim, es) &&
                     wide(p.w, p.dim, 4) && wide(p.b, p.dim, 4);
    if (a->dtype == MAMBA3_F32) gn_go<float>(p, a->act, vec, false, st);
    else gn_go<bf16>(p, a->act, vec, false, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

size_t groupnorm_bwd_workspace_bytes(const mamba3_groupnorm_bwd_args *b) {
    if (!b->dweight && !b->dbias) return 0;
    return (size_t)gn_row_blocks(gn_params(&b->fwd), true) * 2 * b->fwd.dim * 4;
}

mamba3_status launch_groupnorm_bwd(const mamba3_groupnorm_bwd_args *b, hipStream_t st) {
    const mamba3_groupnorm_args *a = &b->fwd;
    GnParams p = gn_params(a);
    const int64_t es = a->dtype == MAMBA3_BF16 ? 2 : 4;
    p.dy = b->dy;
    p.dy_row = b->dy_row ? b->dy_row : a->dim;
    p.dx = b->dx;
    p.dz = b->dz;
    p.part = b->dweight || b->dbias ? (float *)b->workspace : nullptr;
    const bool vec = p.size % 8 == 0 && wide(p.x, p.x_row, es) && wide(p.z, p.z_row, es) && wide(p.dy, p.dy_row, es) &&
                     wide(p.dx, p.dim, es) && wide(p.dz, p.dim, es) && wide(p.w, p.dim, 4) && wide(p.b, p.dim, 4);
    if (p.rows > 0) {
        if (a->dtype == MAMBA3_F32) gn_go<float>(p, a->act, vec, true, st);
        else gn_go<bf16>(p, a->act, vec, true, st);
    }
    if (b->dweight || b->dbias)
        hipLaunchKernelGGL(k_gn_reduce, dim3((p.dim + 15) / 16, 2), dim3(256), 0, st, (const float *)b->workspace,
                           (int)gn_row_blocks(p, true), p.dim, b->dweight, b->dbias);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
