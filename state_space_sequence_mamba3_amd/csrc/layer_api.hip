// C ABI of the layer operators: host-side validation and dispatch. Every check runs before any HIP
// call, so an error status means nothing was enqueued.
#include <algorithm>
#include <cmath>

#include "m3_common.h"

namespace {

constexpr int64_t kMaxBlocks = (1 << 24) - 1;   // HIP: threads of a launch below 2^32, 256 a workgroup

// One array of a call: its address range and what is known of it.
struct Arr {
    const void *p;
    int64_t bytes;
    int align;
    bool need;      // a required pointer
};

Arr rows_of(const void *p, int64_t tokens, int64_t row, int64_t n, int64_t es, bool need) {
    return {p, tokens > 0 ? ((tokens - 1) * (row ? row : n) + n) * es : 0, (int)es, need && tokens > 0};
}
Arr dense_of(const void *p, int64_t n, int64_t es, bool need, int align = 0) {
    return {p, n * es, align ? align : (int)es, need && n > 0};
}

bool overlap(const Arr &a, const Arr &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const char *x = (const char *)a.p, *y = (const char *)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

// Required pointers, alignments, and every output against every input and every other output.
// in_place: an (input, output) pair that may be the same array.
template <int NI, int NO>
mamba3_status check_arrays(const Arr (&in)[NI], const Arr (&out)[NO], int same_in = -1, int same_out = -1) {
    for (const Arr &a : in)
        if (a.need && !a.p) return MAMBA3_EINVAL;
    for (const Arr &a : out)
        if (a.need && !a.p) return MAMBA3_EINVAL;
    for (const Arr &a : in)
        if (a.p && (uintptr_t)a.p % a.align) return MAMBA3_EALIGN;
    for (const Arr &a : out)
        if (a.p && (uintptr_t)a.p % a.align) return MAMBA3_EALIGN;
    for (int i = 0; i < NO; i++) {
        for (int j = 0; j < NI; j++) {
            if (i == same_out && j == same_in && in[j].p == out[i].p) continue;
            if (overlap(out[i], in[j])) return MAMBA3_EINVAL;
        }
        for (int j = i + 1; j < NO; j++)
            if (overlap(out[i], out[j])) return MAMBA3_EINVAL;
    }
    return MAMBA3_OK;
}

// A caller's workspace: large enough, 256-byte aligned, apart from every array.
template <int NI, int NO>
mamba3_status check_workspace(const void *ws, size_t bytes, size_t need, const Arr (&in)[NI], const Arr (&out)[NO]) {
    if (bytes < need || (need > 0 && !ws) || (bytes > 0 && !ws)) return MAMBA3_EWORKSPACE;
    if ((uintptr_t)ws & 255u) return MAMBA3_EALIGN;
    const Arr w{ws, (int64_t)bytes, 1, false};
    for (const Arr &a : in)
        if (overlap(w, a)) return MAMBA3_EINVAL;
    for (const Arr &a : out)
        if (overlap(w, a)) return MAMBA3_EINVAL;
    return MAMBA3_OK;
}

bool dtype_ok(int32_t t) { return t == MAMBA3_F32 || t == MAMBA3_BF16; }
int64_t esize(int32_t t) { return t == MAMBA3_BF16 ? 2 : 4; }
bool flag(int32_t f) { return f == 0 || f == 1; }
// (rows of at most 2^25 elements: a tile's 16 rows are addressed by 32 bits of bytes)
bool row_ok(int64_t row, int64_t n) { return n <= (1 << 25) && (row == 0 || (row >= n && row <= (1 << 25))); }

// batch, seqlen, cu_seqlens and nseq of a whole-sequence call; S the sequences, T the tokens
mamba3_status check_batch(int32_t batch, int32_t seqlen, const int32_t *cu, int32_t nseq, int64_t *S, int64_t *T) {
    if (batch < 0 || seqlen < 0) return MAMBA3_EINVAL;
    if (cu && (batch != 1 || nseq < 1)) return MAMBA3_EINVAL;
    if ((uintptr_t)cu & 3u) return MAMBA3_EALIGN;
    *S = cu ? nseq : batch;
    *T = (int64_t)batch * seqlen;
    return *T <= (1 << 30) ? MAMBA3_OK : MAMBA3_EINVAL;   // (token numbers, and some past the end, in 32 bits)
}

// ---- convolution ----
mamba3_status conv_shape(const mamba3_conv_args *a, bool back, int64_t *S, int64_t *T) {
    if (!a) return MAMBA3_EINVAL;
    if (!dtype_ok(a->dtype) || !flag(a->silu) || a->dim < 1 || a->width < 1 || !row_ok(a->x_row, a->dim))
        return MAMBA3_EINVAL;
    const mamba3_status st = check_batch(a->batch, a->seqlen, a->cu_seqlens, a->nseq, S, T);
    if (st != MAMBA3_OK) return st;
    if (a->width < 2 || a->width > 8) return MAMBA3_EUNSUPPORTED;
    return m3::conv_workgroups(a, back) <= kMaxBlocks ? MAMBA3_OK : MAMBA3_EINVAL;
}

}  // namespace

extern "C" {

mamba3_status mamba3_conv_validate(const mamba3_conv_args *a) {
    int64_t S, T;
    const mamba3_status st = conv_shape(a, false, &S, &T);
    if (st != MAMBA3_OK) return st;
    const int64_t es = esize(a->dtype), D = a->dim, W = a->width;
    const Arr in[] = {rows_of(a->x, T, a->x_row, D, es, true), dense_of(a->weight, D * W, 4, true),
                      dense_of(a->bias, D, 4, false), dense_of(a->conv_in, S * (W - 1) * D, es, false),
                      dense_of(a->cu_seqlens, a->cu_seqlens ? S + 1 : 0, 4, false)};
    const Arr out[] = {dense_of(a->y, T * D, es, true), dense_of(a->conv_out, S * (W - 1) * D, es, false)};
    return check_arrays(in, out);
}

mamba3_status mamba3_conv_fwd(const mamba3_conv_args *a, void *stream) {
    const mamba3_status st = mamba3_conv_validate(a);
    return st != MAMBA3_OK ? st : m3::launch_conv(a, (hipStream_t)stream);
}

size_t mamba3_conv_bwd_workspace_size(const mamba3_conv_bwd_args *b) {
    int64_t S, T;
    return b && conv_shape(&b->fwd, true, &S, &T) == MAMBA3_OK ? m3::conv_bwd_workspace_bytes(b) : 0;
}

mamba3_status mamba3_conv_bwd_validate(const mamba3_conv_bwd_args *b) {
    int64_t S, T;
    if (!b) return MAMBA3_EINVAL;
    const mamba3_conv_args *a = &b->fwd;
    mamba3_status st = conv_shape(a, true, &S, &T);
    if (st != MAMBA3_OK) return st;
    if (!row_ok(b->dy_row, a->dim) || (b->dconv_in && !a->conv_in)) return MAMBA3_EINVAL;
    const int64_t es = esize(a->dtype), D = a->dim, W = a->width;
    const Arr in[] = {rows_of(a->x, T, a->x_row, D, es, true), dense_of(a->weight, D * W, 4, true),
                      dense_of(a->bias, D, 4, false), dense_of(a->conv_in, S * (W - 1) * D, es, false),
                      dense_of(a->cu_seqlens, a->cu_seqlens ? S + 1 : 0, 4, false),
                      rows_of(b->dy, T, b->dy_row, D, es, true), dense_of(b->dconv_out, S * (W - 1) * D, es, false)};
    const Arr out[] = {dense_of(b->dx, T * D, es, true), dense_of(b->dweight, D * W, 4, true),
                       dense_of(b->dbias, D, 4, false), dense_of(b->dconv_in, S * (W - 1) * D, es, false)};
    if ((st = check_arrays(in, out)) != MAMBA3_OK) return st;
    return check_workspace(b->workspace, b->workspace_bytes, m3::conv_bwd_workspace_bytes(b), in, out);
}

mamba3_status mamba3_conv_bwd(const mamba3_conv_bwd_args *b, void *stream) {
    const mamba3_status st = mamba3_conv_bwd_validate(b);
    return st != MAMBA3_OK ? st : m3::launch_conv_bwd(b, (hipStream_t)stream);
}

mamba3_status mamba3_conv_step_validate(const mamba3_conv_step_args *a) {
    if (!a) return MAMBA3_EINVAL;
    if (!dtype_ok(a->dtype) || !flag(a->silu) || a->batch < 0 || a->dim < 1 || a->width < 1 ||
        !row_ok(a->x_row, a->dim) || (a->slots && a->nslots < 0))
        return MAMBA3_EINVAL;
    if (a->width < 2 || a->width > 8) return MAMBA3_EUNSUPPORTED;
    if (m3::conv_step_workgroups(a) > kMaxBlocks) return MAMBA3_EINVAL;
    const int64_t es = esize(a->dtype), D = a->dim, W = a->width, b = a->batch;
    const Arr in[] = {rows_of(a->x, b, a->x_row, D, es, true), dense_of(a->weight, D * W, 4, true),
                      dense_of(a->bias, D, 4, false), dense_of(a->slots, a->slots ? b : 0, 4, false)};
    const Arr out[] = {dense_of(a->y, b * D, es, true),
                       dense_of(a->conv, (a->slots ? a->nslots : b) * (W - 1) * D, es, true)};
    return check_arrays(in, out);
}

mamba3_status mamba3_conv_step(const mamba3_conv_step_args *a, void *stream) {
    const mamba3_status st = mamba3_conv_step_validate(a);
    if (st != MAMBA3_OK || a->batch == 0) return st;
    return m3::launch_conv_step(a, (hipStream_t)stream);
}

// ---- selective scan ----
static mamba3_status sel_shape(const mamba3_selective_scan_args *a, bool back, int64_t *S, int64_t *T) {
    if (!a) return MAMBA3_EINVAL;
    if (!dtype_ok(a->dtype) || !flag(a->dt_softplus) || a->dim < 1 || a->dstate < 1 || a->ngroups < 1 ||
        a->dim % a->ngroups)
        return MAMBA3_EINVAL;
    const int64_t gn = (int64_t)a->ngroups * a->dstate;
    if (!row_ok(a->x_row, a->dim) || !row_ok(a->dt_row, a->dim) || !row_ok(a->z_row, a->dim) || !row_ok(a->B_row, gn) ||
        !row_ok(a->C_row, gn) || gn > INT32_MAX)
        return MAMBA3_EINVAL;
    const mamba3_status st = check_batch(a->batch, a->seqlen, a->cu_seqlens, a->nseq, S, T);
    if (st != MAMBA3_OK) return st;
    if (a->dstate > 128) return MAMBA3_EUNSUPPORTED;
    return m3::selective_workgroups(a, back) <= kMaxBlocks ? MAMBA3_OK : MAMBA3_EINVAL;
}

size_t mamba3_selective_scan_workspace_size(const mamba3_selective_scan_args *a) {
    int64_t S, T;
    return sel_shape(a, false, &S, &T) == MAMBA3_OK ? m3::selective_workspace_bytes(a) : 0;
}

mamba3_status mamba3_selective_scan_validate(const mamba3_selective_scan_args *a) {
    int64_t S, T;
    mamba3_status st = sel_shape(a, false, &S, &T);
    if (st != MAMBA3_OK) return st;
    const int64_t es = esize(a->dtype), D = a->dim, N = a->dstate, gn = a->ngroups * N;
    const Arr in[] = {rows_of(a->x, T, a->x_row, D, es, true), rows_of(a->dt, T, a->dt_row, D, es, true),
                      rows_of(a->z, T, a->z_row, D, es, false), rows_of(a->B, T, a->B_row, gn, es, true),
                      rows_of(a->C, T, a->C_row, gn, es, true), dense_of(a->A, D * N, 4, true, 16),
                      dense_of(a->D, D, 4, false), dense_of(a->dt_bias, D, 4, false),
                      dense_of(a->h_in, S * D * N, 4, false, 16),
                      dense_of(a->cu_seqlens, a->cu_seqlens ? S + 1 : 0, 4, false)};
    const Arr out[] = {dense_of(a->y, T * D, es, true), dense_of(a->h_out, S * D * N, 4, false, 16)};
    if ((st = check_arrays(in, out, 8, 1)) != MAMBA3_OK) return st;
    return check_workspace(a->workspace, a->workspace_bytes, m3::selective_workspace_bytes(a), in, out);
}

mamba3_status mamba3_selective_scan_fwd(const mamba3_selective_scan_args *a, void *stream) {
    const mamba3_status st = mamba3_selective_scan_validate(a);
    if (st != MAMBA3_OK) return st;
    if ((a->cu_seqlens ? a->nseq : a->batch) == 0) return MAMBA3_OK;
    return m3::launch_selective_scan(a, (hipStream_t)stream);
}

size_t mamba3_selective_scan_bwd_workspace_size(const mamba3_selective_scan_bwd_args *b) {
    int64_t S, T;
    return b && sel_shape(&b->fwd, true, &S, &T) == MAMBA3_OK ? m3::selective_bwd_workspace_bytes(b) : 0;
}

mamba3_status mamba3_selective_scan_bwd_validate(const mamba3_selective_scan_bwd_args *b) {
    int64_t S, T;
    if (!b) return MAMBA3_EINVAL;
    const mamba3_selective_scan_args *a = &b->fwd;
    mamba3_status st = sel_shape(a, true, &S, &T);
    if (st != MAMBA3_OK) return st;
    if (!row_ok(b->dy_row, a->dim) || (b->dz && !a->z)) return MAMBA3_EINVAL;
    const int64_t es = esize(a->dtype), D = a->dim, N = a->dstate, gn = a->ngroups * N;
    const Arr in[] = {rows_of(a->x, T, a->x_row, D, es, true), rows_of(a->dt, T, a->dt_row, D, es, true),
                      rows_of(a->z, T, a->z_row, D, es, false), rows_of(a->B, T, a->B_row, gn, es, true),
                      rows_of(a->C, T, a->C_row, gn, es, true), dense_of(a->A, D * N, 4, true, 16),
                      dense_of(a->D, D, 4, false), dense_of(a->dt_bias, D, 4, false),
                      dense_of(a->h_in, S * D * N, 4, false, 16),
                      dense_of(a->cu_seqlens, a->cu_seqlens ? S + 1 : 0, 4, false),
                      rows_of(b->dy, T, b->dy_row, D, es, true), dense_of(b->dh_out, S * D * N, 4, false, 16)};
    const Arr out[] = {dense_of(b->dx, T * D, es, true), dense_of(b->ddt, T * D, es, true),
                       dense_of(b->dB, T * gn, es, true), dense_of(b->dC, T * gn, es, true),
                       dense_of(b->dz, T * D, es, false), dense_of(b->dA, D * N, 4, true),
                       dense_of(b->dD, D, 4, false), dense_of(b->ddt_bias, D, 4, false),
                       dense_of(b->dh_in, S * D * N, 4, false, 16)};
    if ((st = check_arrays(in, out)) != MAMBA3_OK) return st;
    return check_workspace(b->workspace, b->workspace_bytes, m3::selective_bwd_workspace_bytes(b), in, out);
}

mamba3_status mamba3_selective_scan_bwd(const mamba3_selective_scan_bwd_args *b, void *stream) {
    const mamba3_status st = mamba3_selective_scan_bwd_validate(b);
    return st != MAMBA3_OK ? st : m3::launch_selective_scan_bwd(b, (hipStream_t)stream);
}

mamba3_status mamba3_selective_step_validate(const mamba3_selective_step_args *a) {
    if (!a) return MAMBA3_EINVAL;
    if (!dtype_ok(a->dtype) || !flag(a->dt_softplus) || a->batch < 0 || a->dim < 1 || a->dstate < 1 ||
        a->ngroups < 1 || a->dim % a->ngroups || (a->slots && a->nslots < 0))
        return MAMBA3_EINVAL;
    const int64_t es = esize(a->dtype), D = a->dim, N = a->dstate, gn = a->ngroups * N, b = a->batch;
    if (!row_ok(a->x_row, D) || !row_ok(a->dt_row, D) || !row_ok(a->z_row, D) || !row_ok(a->B_row, gn) ||
        !row_ok(a->C_row, gn) || gn > INT32_MAX)
        return MAMBA3_EINVAL;
    if (N > 128) return MAMBA3_EUNSUPPORTED;
    if (m3::selective_step_workgroups(a) > kMaxBlocks) return MAMBA3_EINVAL;
    const Arr in[] = {rows_of(a->x, b, a->x_row, D, es, true), rows_of(a->dt, b, a->dt_row, D, es, true),
                      rows_of(a->z, b, a->z_row, D, es, false), rows_of(a->B, b, a->B_row, gn, es, true),
                      rows_of(a->C, b, a->C_row, gn, es, true), dense_of(a->A, D * N, 4, true, 16),
                      dense_of(a->D, D, 4, false), dense_of(a->dt_bias, D, 4, false),
                      dense_of(a->slots, a->slots ? b : 0, 4, false)};
    const Arr out[] = {dense_of(a->y, b * D, es, true),
                       dense_of(a->h, (a->slots ? a->nslots : b) * D * N, 4, b > 0, 16)};
    return check_arrays(in, out);
}

mamba3_status mamba3_selective_step(const mamba3_selective_step_args *a, void *stream) {
    const mamba3_status st = mamba3_selective_step_validate(a);
    if (st != MAMBA3_OK || a->batch == 0) return st;
    return m3::launch_selective_step(a, (hipStream_t)stream);
}

// ---- RMS norm ----
static mamba3_status norm_shape(int64_t rows, int32_t dim, int32_t dtype, int32_t rtype, float eps, int64_t row) {
    if (rows < 0 || rows > kMaxBlocks || dim < 1 || !dtype_ok(dtype) || !dtype_ok(rtype) || !row_ok(row, dim))
        return MAMBA3_EINVAL;
    if (!(eps >= 0.f && std::isfinite(eps))) return MAMBA3_EINVAL;
    return rtype == MAMBA3_F32 || dtype == MAMBA3_BF16 ? MAMBA3_OK : MAMBA3_EUNSUPPORTED;
}

mamba3_status mamba3_rmsnorm_validate(const mamba3_rmsnorm_args *a) {
    if (!a) return MAMBA3_EINVAL;
    const mamba3_status st = norm_shape(a->rows, a->dim, a->dtype, a->residual_dtype, a->eps, a->x_row);
    if (st != MAMBA3_OK) return st;
    // (empty arrays may have no address)
    if (a->rows > 0 && ((a->q == nullptr) != (a->qscale == nullptr) || (!a->q && !a->y))) return MAMBA3_EINVAL;
    int64_t blocks = 0;
    if (a->q) {
        if ((a->qtype != MAMBA3_E4M3 && a->qtype != MAMBA3_INT8) || a->qblock < 0) return MAMBA3_EINVAL;
        const bool whole = a->qblock == 0 || a->qblock >= a->dim;
        if (!whole && a->qblock != 32 && a->qblock != 64 && a->qblock != 128 && a->qblock != 256)
            return MAMBA3_EUNSUPPORTED;
        blocks = whole ? 1 : (a->dim + a->qblock - 1) / a->qblock;
    }
    const int64_t es = esize(a->dtype), rs = esize(a->residual_dtype), M = a->rows * a->dim;
    const Arr in[] = {rows_of(a->x, a->rows, a->x_row, a->dim, es, true), dense_of(a->residual, M, rs, false),
                      dense_of(a->weight, a->dim, 4, false)};
    const Arr out[] = {dense_of(a->residual_out, M, rs, false), dense_of(a->y, M, es, false),
                       dense_of(a->q, a->q ? M : 0, 1, false), dense_of(a->qscale, a->rows * blocks, 4, false)};
    return check_arrays(in, out, 1, 0);
}

mamba3_status mamba3_rmsnorm_fwd(const mamba3_rmsnorm_args *a, void *stream) {
    const mamba3_status st = mamba3_rmsnorm_validate(a);
    if (st != MAMBA3_OK || a->rows == 0) return st;
    return m3::launch_rmsnorm(a, (hipStream_t)stream);
}

size_t mamba3_rmsnorm_bwd_workspace_size(const mamba3_rmsnorm_bwd_args *b) {
    return b && norm_shape(b->rows, b->dim, b->dtype, b->residual_dtype, b->eps, b->dy_row) == MAMBA3_OK
               ? m3::rmsnorm_bwd_workspace_bytes(b)
               : 0;
}

mamba3_status mamba3_rmsnorm_bwd_validate(const mamba3_rmsnorm_bwd_args *b) {
    if (!b) return MAMBA3_EINVAL;
    mamba3_status st = norm_shape(b->rows, b->dim, b->dtype, b->residual_dtype, b->eps, b->dy_row);
    if (st != MAMBA3_OK) return st;
    if (b->rows > 0 && !b->dx && !b->dresidual) return MAMBA3_EINVAL;
    const int64_t es = esize(b->dtype), rs = esize(b->residual_dtype), M = b->rows * b->dim;
    const Arr in[] = {dense_of(b->s, M, rs, true), rows_of(b->dy, b->rows, b->dy_row, b->dim, es, true),
                      dense_of(b->dresidual_out, M, rs, false), dense_of(b->weight, b->dim, 4, false)};
    const Arr out[] = {dense_of(b->dx, M, es, false), dense_of(b->dresidual, M, rs, false),
                       dense_of(b->dweight, b->dim, 4, false)};
    if ((st = check_arrays(in, out, 2, 1)) != MAMBA3_OK) return st;
    return check_workspace(b->workspace, b->workspace_bytes, m3::rmsnorm_bwd_workspace_bytes(b), in, out);
}

mamba3_status mamba3_rmsnorm_bwd(const mamba3_rmsnorm_bwd_args *b, void *stream) {
    const mamba3_status st = mamba3_rmsnorm_bwd_validate(b);
    return st != MAMBA3_OK ? st : m3::launch_rmsnorm_bwd(b, (hipStream_t)stream);
}

}  // extern "C"
