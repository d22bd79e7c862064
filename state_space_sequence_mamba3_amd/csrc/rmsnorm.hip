// RMS norm of rows with the residual's addition, its 8-bit output with scales, and its backward.
//
//   s = x + residual,  v = s rsqrt(mean(s^2) + eps) w,  q = round(v / scale)
//   ds = dresidual_out + r (w dy - sh mean(w dy sh)),  dw = sum over rows of dy sh   (sh = r s)
//
// A few operations a value, so HBM-bound: every row is read once, kept in registers as fp32 between its
// sum and its outputs (rows of more than 8192 values are read twice), and everything a row needs
// is written in the same pass. A lane holds 8 consecutive values, so a wave's load covers 1 KB of
// bf16, and a scale's block of 32 .. 256 values lies in 4 .. 32 consecutive lanes.
//
// 32768 x 2048, bf16 with an fp32 residual: 138 us, 5.84 TB/s (a large copy runs at 4.94); its backward 209 us,
// 5.13 TB/s; 128 x 2048 to e4m3 in blocks of 128 4.4 us. 32768 x 2048 with a bf16 residual: 93 us, to 8 bits 88 to
// 98 (e4m3 or int8, any block), with y too 105 to 112.
// Rows above 8192 values: 2048 x 16384 104 us and 206 backward (79 and 53 % of the copy rate), for the second read and
// dweight's third (51 us); 4096 x 8200 104 and 261, where dweight's 129 workgroups leave half the CUs idle (91 us).
#include <type_traits>

#include "layer.h"

namespace m3 {

constexpr int kNV = 8;    // consecutive values of a lane

struct NormParams {
    const void *x, *res, *dy, *dres;     // (backward: x is s)
    const float *w;
    void *res_out, *y, *q, *dx;
    float *scale, *part, *dw;
    int64_t rows, x_row, dy_row;
    int32_t dim, qtype, qblock, nblocks;
    float eps;
};

// 8 values at any element: global memory takes loads and stores of 8 or 16 bytes there, in one
// instruction each, which rows of odd lengths (VEC false) use up to their last piece.
template <typename T> struct Loose8 { typedef T type __attribute__((ext_vector_type(8), aligned(sizeof(T)))); };

// 8 values of a row from column c on; zeros behind the row's end
template <typename T, bool VEC>
__device__ __forceinline__ void load8(float (&o)[kNV], const T *row, int c, int n) {
    if constexpr (VEC) {
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                const bf16x8 v = *(const bf16x8 *)(row + c);
#pragma unroll
                for (int e = 0; e < 8; e++) o[e] = to_f(v[e]);
            } else {
                const f32x4 a = *(const f32x4 *)(row + c), b = *(const f32x4 *)(row + c + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    o[e] = a[e];
                    o[e + 4] = b[e];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = 0.f;
        }
    } else if (c + 8 <= n) {
        const typename Loose8<T>::type v = *(const typename Loose8<T>::type *)(row + c);
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = to_f(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = c + e < n ? to_f(row[c + e]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int c, int n, const float (&o)[kNV]) {
    if constexpr (VEC) {
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                bf16x8 v;
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = from_f<bf16>(o[e]);
                *(bf16x8 *)(row + c) = v;
            } else {
                *(f32x4 *)(row + c) = f32x4{o[0], o[1], o[2], o[3]};
                *(f32x4 *)(row + c + 4) = f32x4{o[4], o[5], o[6], o[7]};
            }
        }
    } else if (c + 8 <= n) {
        typename Loose8<T>::type v;
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = from_f<T>(o[e]);
        *(typename Loose8<T>::type *)(row + c) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (c + e < n) row[c + e] = from_f<T>(o[e]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x141>(v);    // half-row mirror: the other quad of 8
    v += dpp_move<0x140>(v);    // row mirror: the other 8 of 16
    return sum_across_rows(v);
}
// The larger of two values, NaN if either is (a NaN in a block shows in its scale).
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }

// The sum over the WPR waves that share a row (every lane gets it).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; i++) v += red[i];
    }
    return v;
}
template <int WPR>
__device__ __forceinline__ float row_max(float v, float *red) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max_nan(v, __shfl_xor(v, o, 64));
    if constexpr (WPR > 1) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < WPR; i++) v = max_nan(v, red[i]);
    }
    return v;
}

// Squares leave fp32's range long before the values do: a row whose mean square + eps is no number of
// [2^-80, infinity) is summed again with its values times a power of two, `row_scale` of that mean, which
// brings every finite row back inside.
constexpr float kLeastMean = 0x1p-80f;
__device__ __forceinline__ bool in_range(float mean) { return mean >= kLeastMean && mean < INFINITY; }
__device__ __forceinline__ float row_scale(float mean) { return mean < kLeastMean ? 0x1p100f : 0x1p-80f; }

constexpr float kTinyScale = 1.17549435e-38f;   // 2^-126: a block of zeros divides by it

// q = round(v / scale). One Newton step makes the quotient by the reciprocal the correctly rounded
// one in all but rare cases, so q is the nearest 8-bit value of the true quotient.
__device__ __forceinline__ float quotient(float v, float scale, float r) {
    const float q = v * r;
    const float f = fmaf(fmaf(-scale, q, v), r, q);
    return f == f ? f : q;      // infinities: the correction is not a number where the quotient is
}
template <bool VEC>
__device__ __forceinline__ void store_q(const NormParams &p, int64_t row, int c, const float (&v)[kNV], float scale) {
    if (c >= p.dim) return;
    const float r = 1.f / scale;
    uint32_t w[2] = {0, 0};
    if (p.qtype == MAMBA3_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            int t = 0;
            t = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h], scale, r), quotient(v[4 * h + 1], scale, r), t, false);
            t = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * h + 2], scale, r), quotient(v[4 * h + 3], scale, r), t, true);
            w[h] = (uint32_t)t;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kNV; e++) {
            const float f = fminf(fmaxf(rintf(quotient(v[e], scale, r)), -127.f), 127.f);
            w[e >> 2] |= ((uint32_t)(int)f & 255u) << (8 * (e & 3));
        }
    }
    uint8_t *q = (uint8_t *)p.q + row * p.dim + c;
    if constexpr (VEC) {
        *(uint2 *)q = make_uint2(w[0], w[1]);
    } else if (c + 8 <= p.dim) {
        typedef uint32_t loose __attribute__((ext_vector_type(2), aligned(1)));
        *(loose *)q = loose{w[0], w[1]};
    } else {
#pragma unroll
        for (int e = 0; e < kNV; e++)
            if (c + e < p.dim) q[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}

// WPR waves share a row (a workgroup holds 4 / WPR rows); NCH > 0: a lane keeps NCH pieces of 8
// values in registers; NCH = 0: rows of any length, read again for the outputs.
template <typename T, typename RT, int WPR, int NCH, bool VEC>
__global__ __launch_bounds__(256) void k_norm(NormParams p) {
    __shared__ float red[4];
    constexpr int STEP = WPR * 64 * kNV;
    const int64_t row = WPR == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= p.rows) return;                       // (whole waves; WPR = 4: never)
    const int t = WPR == 4 ? threadIdx.x : threadIdx.x & 63;
    const T *x = (const T *)p.x + row * p.x_row;
    const RT *res = p.res ? (const RT *)p.res + row * p.dim : nullptr;
    RT *ro = p.res_out ? (RT *)p.res_out + row * p.dim : nullptr;
    const int nch = NCH ? NCH : (p.dim + STEP - 1) / STEP;
    float keep[NCH ? NCH : 1][kNV];
    auto sum_of = [&](int c, float (&s)[kNV]) {
        load8<T, VEC>(s, x, c, p.dim);
        if (res) {
            float r[kNV];
            load8<RT, VEC>(r, res, c, p.dim);
#pragma unroll
            for (int e = 0; e < kNV; e++) s[e] += r[e];
        }
    };
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < nch; i++) {
        float(&s)[kNV] = keep[NCH ? i : 0];
        sum_of(i * STEP + t * kNV, s);
#pragma unroll
        for (int e = 0; e < kNV; e++) ss += s[e] * s[e];
    }
    const float mean = row_sum<WPR>(ss, red) / (float)p.dim + p.eps;
    float rms = __builtin_amdgcn_rsqf(mean);
    if (!in_range(mean)) {                           // (the same for all lanes of the row)
        const float k = row_scale(mean);
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < nch; i++) {
            float(&s)[kNV] = keep[NCH ? i : 0];
            if constexpr (NCH == 0) sum_of(i * STEP + t * kNV, s);
#pragma unroll
            for (int e = 0; e < kNV; e++) ss += s[e] * k * (s[e] * k);
        }
        rms = __builtin_amdgcn_rsqf(row_sum<WPR>(ss, red) / (float)p.dim + p.eps * k * k) * k;
    }
    const bool one = p.q && p.nblocks == 1;          // one scale a row
    const float qmax = p.qtype == MAMBA3_E4M3 ? 448.f : 127.f;
    auto normed = [&](int c, const float (&s)[kNV], float (&v)[kNV]) {
        float w[kNV];
        if (p.w) load8<float, VEC>(w, p.w, c, p.dim);
#pragma unroll
        for (int e = 0; e < kNV; e++) v[e] = s[e] * rms * (p.w ? w[e] : 1.f);
    };
    float whole = 1.f;
    if (one) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < nch; i++) {
            const int c = i * STEP + t * kNV;
            float s[kNV], v[kNV];
            if constexpr (NCH == 0) sum_of(c, s);
            normed(c, NCH ? keep[NCH ? i : 0] : s, v);
#pragma unroll
            for (int e = 0; e < kNV; e++) m = max_nan(m, c + e < p.dim ? fabsf(v[e]) : 0.f);
        }
        const float top = row_max<WPR>(m, red) / qmax;
        whole = top < kTinyScale ? kTinyScale : top;
        if (t == 0) p.scale[row] = whole;
    }
#pragma unroll
    for (int i = 0; i < nch; i++) {
        const int c = i * STEP + t * kNV;
        float again[kNV], v[kNV];
        if constexpr (NCH == 0) sum_of(c, again);
        const float(&s)[kNV] = NCH ? keep[NCH ? i : 0] : again;
        if (ro) store8<RT, VEC>(ro, c, p.dim, s);
        normed(c, s, v);
        if (p.y) store8<T, VEC>((T *)p.y + row * p.dim, c, p.dim, v);
        if (p.q) {
            float sc = whole;
            if (!one) {
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < kNV; e++) m = max_nan(m, c + e < p.dim ? fabsf(v[e]) : 0.f);
                for (int o = 1; o < p.qblock / kNV; o <<= 1) m = max_nan(m, __shfl_xor(m, o, 64));
                sc = m / qmax;
                sc = sc < kTinyScale ? kTinyScale : sc;
                if (c < p.dim && c % p.qblock == 0) p.scale[row * p.nblocks + c / p.qblock] = sc;
            }
            store_q<VEC>(p, row, c, v, sc);
        }
    }
}

// 8 values as loaded, converted where they are used: the next row's loads are in flight while a row is
// worked on.
template <typename T> struct Raw8 { typedef T type __attribute__((ext_vector_type(8), aligned(16))); };
template <typename T, bool VEC>
__device__ __forceinline__ typename Raw8<T>::type raw8(const T *row, int c, int n) {
    typename Raw8<T>::type v;
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = from_f<T>(0.f);
    if constexpr (VEC) {
        if (c < n) v = *(const typename Raw8<T>::type *)(row + c);
    } else if (c + 8 <= n) {
        v = *(const typename Loose8<T>::type *)(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (c + e < n) v[e] = row[c + e];
    }
    return v;
}
// Two sums over the waves of a row, with one barrier: `red` is the row's half of two, used in turn.
template <int WPR>
__device__ __forceinline__ void row_sums(float &a, float &b, float2 *red) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; i++) {
            a += red[i].x;
            b += red[i].y;
        }
    }
}

// Backward. WPR waves share a row, 8 values a lane (1, 4, 8 or 16 waves: rows of up to 512, 2048, 4096
// and 8192 values; WPR = 1: four rows a workgroup); a workgroup walks several rows, so that dweight's
// partial sums stay in registers. LONG: rows of any length, read twice, and k_norm_dw for dweight.
template <typename T, typename RT, int WPR, bool LONG, bool VEC>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void k_norm_bwd(NormParams p) {
    constexpr int STEP = WPR * 64 * kNV;
    __shared__ float2 red[2][WPR];
    __shared__ float4 join[WPR == 1 ? 2 * 256 : 1];
    const int t = WPR > 1 ? threadIdx.x : threadIdx.x & 63;
    const int64_t first = WPR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t step = (int64_t)gridDim.x * (WPR > 1 ? 1 : 4);
    const int nch = LONG ? (p.dim + STEP - 1) / STEP : 1;
    typename Raw8<RT>::type rs, rr;
    typename Raw8<T>::type rd;
    auto fetch = [&](int64_t row, int i) {
        const int c = i * STEP + t * kNV;
        rs = raw8<RT, VEC>((const RT *)p.x + row * p.dim, c, p.dim);
        rd = raw8<T, VEC>((const T *)p.dy + row * p.dy_row, c, p.dim);
        if (p.dres) rr = raw8<RT, VEC>((const RT *)p.dres + row * p.dim, c, p.dim);
    };
    float w[kNV], dw[kNV];
    auto weigh = [&](int i) {
        if (p.w) {
            load8<float, VEC>(w, p.w, i * STEP + t * kNV, p.dim);
        } else {
#pragma unroll
            for (int e = 0; e < kNV; e++) w[e] = 1.f;
        }
    };
    weigh(0);
#pragma unroll
    for (int e = 0; e < kNV; e++) dw[e] = 0.f;
    int turn = 0;
    bool odd = false;                                // a row whose mean is out of range (see in_range)
    auto walk = [&](auto scaled) __attribute__((always_inline)) {
        constexpr bool SCALED = decltype(scaled)::value;
        if (!LONG && first < p.rows) fetch(first, 0);
        for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
            float ks[kNV], kd[kNV], kr[kNV];
            float ss = 0.f, sd = 0.f;
            auto unpack = [&]() {
#pragma unroll
                for (int e = 0; e < kNV; e++) {
                    ks[e] = to_f(rs[e]);
                    kd[e] = to_f(rd[e]);
                    kr[e] = p.dres ? to_f(rr[e]) : 0.f;
                }
            };
            for (int i = 0; i < nch; i++) {
                if (LONG) {
                    fetch(row, i);
                    weigh(i);
                }
                unpack();
#pragma unroll
                for (int e = 0; e < kNV; e++) {
                    ss += ks[e] * ks[e];
                    sd += ks[e] * w[e] * kd[e];
                }
            }
            if (!LONG && row + step < p.rows) fetch(row + step, 0);
            row_sums<WPR>(ss, sd, red[turn]);
            const float mean = ss / (float)p.dim + p.eps;
            const bool in = in_range(mean);
            float root, r;
            if constexpr (SCALED) {
                if (in) continue;                    // (the same for all lanes of the row)
                const float k = row_scale(mean);
                ss = sd = 0.f;
                for (int i = 0; i < nch; i++) {
                    if (LONG) {
                        fetch(row, i);
                        weigh(i);
                        unpack();
                    }
#pragma unroll
                    for (int e = 0; e < kNV; e++) {
                        ss += ks[e] * k * (ks[e] * k);
                        sd += ks[e] * k * w[e] * kd[e];
                    }
                }
                row_sums<WPR>(ss, sd, red[turn ^ 1]);    // (its last readers are before the barrier above)
                if (WPR > 1) __syncthreads();            // the next row writes this half
                root = __builtin_amdgcn_rsqf(ss / (float)p.dim + p.eps * k * k);
                r = root * k;
            } else {
                odd |= !in;
                root = in ? __builtin_amdgcn_rsqf(mean) : 0.f;
                r = root;
                sd = in ? sd : 0.f;
            }
            const float m = sd / (float)p.dim * root;                       // ds = r (w dy - m sh)
            if (LONG && t == 0 && p.part) p.part[row] = r;
            for (int i = 0; i < nch; i++) {
                const int c = i * STEP + t * kNV;
                float o[kNV];
                if (LONG) {
                    fetch(row, i);
                    weigh(i);
                    unpack();
                }
#pragma unroll
                for (int e = 0; e < kNV; e++) {
                    const float sh = ks[e] * r;
                    o[e] = kr[e] + r * (w[e] * kd[e] - m * sh);
                    if (!LONG) dw[e] += kd[e] * sh;
                }
                if (p.res_out) store8<RT, VEC>((RT *)p.res_out + row * p.dim, c, p.dim, o);
                if (p.dx) store8<T, VEC>((T *)p.dx + row * p.dim, c, p.dim, o);
            }
        }
    };
    // Rows out of range pass with r = 0, which leaves dres as it was and adds nothing to dweight, and are
    // taken in a walk of their own: a branch for them among the others cost 5 % (4096 x 8192 bf16 56 -> 59 us).
    walk(std::integral_constant<bool, false>());
    if (odd) walk(std::integral_constant<bool, true>());
    if (LONG || !p.part) return;
    // one row of partial sums a workgroup: with a wave a row, those of its four waves in order
    if constexpr (WPR == 1) {
        join[2 * threadIdx.x] = make_float4(dw[0], dw[1], dw[2], dw[3]);
        join[2 * threadIdx.x + 1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
        __syncthreads();
        if (threadIdx.x >= 64) return;
#pragma unroll
        for (int v = 1; v < 4; v++) {
            const float4 a = join[2 * (t + 64 * v)], b = join[2 * (t + 64 * v) + 1];
            dw[0] += a.x; dw[1] += a.y; dw[2] += a.z; dw[3] += a.w;
            dw[4] += b.x; dw[5] += b.y; dw[6] += b.z; dw[7] += b.w;
        }
    }
    store8<float, VEC>(p.part + (int64_t)blockIdx.x * p.dim, t * kNV, p.dim, dw);
}

// dweight from `n` rows of partial sums: 16 columns a workgroup, 16 threads over the rows of each.
__global__ __launch_bounds__(256) void k_norm_reduce(const float *part, int n, int dim, float *dw) {
    __shared__ float red[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, c = blockIdx.x * 16 + x;
    float s = 0.f;
    if (c < dim) {
#pragma unroll 8
        for (int i = y; i < n; i += 16) s += part[(int64_t)i * dim + c];
    }
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) s += red[i][x];
        dw[c] = s;
    }
}

// dweight of long rows: 64 columns a workgroup over all rows, with the rows' 1 / rms from k_norm_bwd.
template <typename T, typename RT>
__global__ __launch_bounds__(256) void k_norm_dw(NormParams p) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < p.dim) {
#pragma unroll 8
        for (int64_t i = wave; i < p.rows; i += 4)
            s += to_f(((const T *)p.dy)[i * p.dy_row + c]) * (to_f(((const RT *)p.x)[i * p.dim + c]) * p.part[i]);
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < p.dim) p.dw[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

namespace {

bool wide(const void *q, int64_t row, int64_t es) { return ((uintptr_t)q & 15u) == 0 && row * es % 16 == 0; }

// One wave a row needs no barrier, four spread few rows over more of the GPU. In us, one wave and four, bf16
// with a bf16 residual: 256 x 1024 4.2 and 3.8, 2048 x 1024 5.3 and 5.3, 8192 x 1024 12.4 and 14.0; at 2048
// values a row, where one wave holds 32 a lane, 256 rows 5.4 and 3.9, 2048 8.3 and 7.0, 32768 107 and 94.
bool one_wave(int64_t rows, int dim) { return dim <= 512 || (dim <= 1024 && rows >= 2048); }

// The backward's waves a row, and its workgroups: 16 waves a CU for all (each workgroup leaves a row of
// partial sums).
int bwd_waves(int dim) { return dim <= 512 ? 1 : dim <= 2048 ? 4 : dim <= 4096 ? 8 : dim <= 8192 ? 16 : 4; }
int64_t bwd_blocks(int64_t rows, int dim) {
    const int w = bwd_waves(dim);
    return std::min<int64_t>(w == 1 ? (rows + 3) / 4 : rows, w <= 4 ? 1024 : 4096 / w);
}

template <typename T, typename RT, int WPR, int NCH>
void norm_launch(const NormParams &p, bool vec, hipStream_t st) {
    const int64_t per = 4 / WPR;
    const dim3 grid((uint32_t)((p.rows + per - 1) / per));
    if (vec) hipLaunchKernelGGL((k_norm<T, RT, WPR, NCH, true>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((k_norm<T, RT, WPR, NCH, false>), grid, dim3(256), 0, st, p);
}

template <typename T, typename RT>
void norm_go(const NormParams &p, bool vec, hipStream_t st) {
    if (one_wave(p.rows, p.dim)) {
        if (p.dim <= 512) norm_launch<T, RT, 1, 1>(p, vec, st);
        else norm_launch<T, RT, 1, 2>(p, vec, st);
    } else if (p.dim <= 2048) {
        norm_launch<T, RT, 4, 1>(p, vec, st);
    } else if (p.dim <= 4096) {
        norm_launch<T, RT, 4, 2>(p, vec, st);
    } else if (p.dim <= 8192) {
        norm_launch<T, RT, 4, 4>(p, vec, st);
    } else {
        norm_launch<T, RT, 4, 0>(p, vec, st);
    }
}

template <typename T, typename RT, int WPR, bool LONG>
void bwd_launch(const NormParams &p, bool vec, hipStream_t st) {
    const dim3 grid((uint32_t)bwd_blocks(p.rows, p.dim)), block(WPR == 1 ? 256 : 64 * WPR);
    if (vec) hipLaunchKernelGGL((k_norm_bwd<T, RT, WPR, LONG, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_norm_bwd<T, RT, WPR, LONG, false>), grid, block, 0, st, p);
}

template <typename T, typename RT>
void norm_bwd_go(const NormParams &p, bool vec, hipStream_t st) {
    if (p.dim > 8192) bwd_launch<T, RT, 4, true>(p, vec, st);
    else if (p.dim <= 512) bwd_launch<T, RT, 1, false>(p, vec, st);
    else if (p.dim <= 2048) bwd_launch<T, RT, 4, false>(p, vec, st);
    else if (p.dim <= 4096) bwd_launch<T, RT, 8, false>(p, vec, st);
    else bwd_launch<T, RT, 16, false>(p, vec, st);
}

template <typename T, typename RT>
void dw_go(const NormParams &p, hipStream_t st) {
    hipLaunchKernelGGL((k_norm_dw<T, RT>), dim3((p.dim + 63) / 64), dim3(256), 0, st, p);
}

}  // namespace

mamba3_status launch_rmsnorm(const mamba3_rmsnorm_args *a, hipStream_t st) {
    NormParams p{};
    const int64_t es = a->dtype == MAMBA3_BF16 ? 2 : 4, rs = a->residual_dtype == MAMBA3_BF16 ? 2 : 4;
    p.x = a->x; p.res = a->residual; p.w = a->weight;
    p.res_out = a->residual_out; p.y = a->y; p.q = a->q; p.scale = a->qscale;
    p.rows = a->rows; p.dim = a->dim; p.x_row = a->x_row ? a->x_row : a->dim;
    p.qtype = a->qtype;
    const bool whole = a->qblock == 0 || a->qblock >= a->dim;
    p.qblock = whole ? a->dim : a->qblock;
    p.nblocks = whole ? 1 : (a->dim + a->qblock - 1) / a->qblock;
    p.eps = a->eps;
    const bool vec = a->dim % 8 == 0 && wide(p.x, p.x_row, es) && wide(p.res, p.dim, rs) && wide(p.w, p.dim, 4) &&
                     wide(p.res_out, p.dim, rs) && wide(p.y, p.dim, es) && ((uintptr_t)p.q & 7u) == 0;
    if (a->dtype == MAMBA3_F32) norm_go<float, float>(p, vec, st);
    else if (a->residual_dtype == MAMBA3_F32) norm_go<bf16, float>(p, vec, st);
    else norm_go<bf16, bf16>(p, vec, st);
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

size_t rmsnorm_bwd_workspace_bytes(const mamba3_rmsnorm_bwd_args *b) {
    if (!b->dweight) return 0;
    // rows longer than the registers leave their 1 / rms instead
    return (size_t)(b->dim > 8192 ? b->rows * 4 : bwd_blocks(b->rows, b->dim) * b->dim * 4);
}

mamba3_status launch_rmsnorm_bwd(const mamba3_rmsnorm_bwd_args *b, hipStream_t st) {
    NormParams p{};
    const int64_t es = b->dtype == MAMBA3_BF16 ? 2 : 4, rs = b->residual_dtype == MAMBA3_BF16 ? 2 : 4;
    p.x = b->s; p.dy = b->dy; p.dres = b->dresidual_out; p.w = b->weight;
    p.res_out = b->dresidual; p.dx = b->dx; p.dw = b->dweight;
    p.part = b->dweight ? (float *)b->workspace : nullptr;
    p.rows = b->rows; p.dim = b->dim; p.dy_row = b->dy_row ? b->dy_row : b->dim;
    p.eps = b->eps;
    const bool vec = b->dim % 8 == 0 && wide(p.x, p.dim, rs) && wide(p.dy, p.dy_row, es) && wide(p.dres, p.dim, rs) &&
                     wide(p.w, p.dim, 4) && wide(p.res_out, p.dim, rs) && wide(p.dx, p.dim, es);
    if (p.rows > 0) {
        if (b->dtype == MAMBA3_F32) norm_bwd_go<float, float>(p, vec, st);
        else if (b->residual_dtype == MAMBA3_F32) norm_bwd_go<bf16, float>(p, vec, st);
        else norm_bwd_go<bf16, bf16>(p, vec, st);
    }
    if (b->dweight) {
        if (b->dim <= 8192) {
            hipLaunchKernelGGL(k_norm_reduce, dim3((b->dim + 15) / 16), dim3(256), 0, st, p.part,
                               (int)bwd_blocks(b->rows, b->dim), b->dim, b->dweight);
        } else if (b->dtype == MAMBA3_F32) {
            dw_go<float, float>(p, st);
        } else if (b->residual_dtype == MAMBA3_F32) {
            dw_go<bf16, float>(p, st);
        } else {
            dw_go<bf16, bf16>(p, st);
        }
    }
    return hipGetLastError() == hipSuccess ? MAMBA3_OK : MAMBA3_EHIP;
}

}  // namespace m3
