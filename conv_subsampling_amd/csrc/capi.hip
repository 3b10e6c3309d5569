// The library's C ABI (declared in include/dwconv.h): host-side argument
// validation, the thread-local error message, and dispatch to the kernel
// launchers.  Nothing here allocates, frees or synchronises.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "../../include/dwconv.h"
#include "launch.h"
#include "scratch.h"

#ifndef DW1D_BF16_VEC
#define DW1D_BF16_VEC 4  // bf16 channels per lane access in the 1-D kernel
#endif

namespace {

thread_local char g_err[512] = "";

dw_status fail(dw_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

dw_status ok() {
    g_err[0] = '\0';
    return DW_OK;
}

dw_status from_hip(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(DW_ERR_HIP, "%s: HIP launch failed: %s", what, hipGetErrorString(e));
}

// The 2-D kernels: a 3x3 kernel, stride 2, and the paddings
// dwconv2d_pads_supported accepts.
dw_status check_geometry_2d(const char* fn, int64_t KH, int64_t KW, int64_t stride, int64_t pt0, int64_t pt1,
                            int64_t pf0, int64_t pf1) {
    if (KH < 1 || KW < 1 || stride < 1 || pt0 < 0 || pt1 < 0 || pf0 < 0 || pf1 < 0)
        return fail(DW_ERR_INVALID_ARG, "%s: kernel %lldx%lld, stride %lld, pads (%lld, %lld, %lld, %lld) are not a "
                    "valid geometry", fn, (long long)KH, (long long)KW, (long long)stride, (long long)pt0,
                    (long long)pt1, (long long)pf0, (long long)pf1);
    if (KH != 3 || KW != 3 || stride != 2 || !dw::dwconv2d_pads_supported(pt0, pt1, pf0, pf1))
        return fail(DW_ERR_UNSUPPORTED, "%s: implemented for a 3x3 kernel, stride 2, padding 1 or 2 before and 0 to 2 "
                    "after on each axis (got %lldx%lld, stride %lld, pads (%lld, %lld, %lld, %lld))", fn,
                    (long long)KH, (long long)KW, (long long)stride, (long long)pt0, (long long)pt1,
                    (long long)pf0, (long long)pf1);
    return DW_OK;
}

// True when every extent is positive: a tensor with these extents holds
// elements.  (Multiplying the extents could overflow.)
template <typename... I>
bool nonempty(I... n) {
    return ((n > 0) && ...);
}

// Whether every extent is below dw::kMaxExtent (the launchers' size checks
// add extents together and need that bound; larger ones cannot fit anyway).
template <typename... I>
bool extents_ok(I... n) {
    return ((n < dw::kMaxExtent) && ...);
}

dw_status too_large(const char* fn) { return fail(DW_ERR_UNSUPPORTED, "%s: sizes too large for one launch", fn); }

bool geometry_ok_2d(int64_t KH, int64_t KW, int64_t stride, int64_t pt0, int64_t pt1, int64_t pf0, int64_t pf1) {
    return KH == 3 && KW == 3 && stride == 2 && dw::dwconv2d_pads_supported(pt0, pt1, pf0, pf1);
}

dw_status check_pad(const char* fn, dw_pad pad) {
    if (pad != DW_PAD_SYMMETRIC && pad != DW_PAD_CAUSAL)
        return fail(DW_ERR_INVALID_ARG, "%s: unknown pad mode %d", fn, (int)pad);
    return DW_OK;
}

dw_status check_dtype(const char* fn, dw_dtype dtype) {
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    return DW_OK;
}

// A dropout probability, and the generator's state where it drops anything.
dw_status check_dropout(const char* fn, double p, const uint64_t* rng) {
    if (!(p >= 0.0 && p < 1.0))
        return fail(DW_ERR_INVALID_ARG, "%s: dropout probability %g is not in [0, 1)", fn, p);
    if (p > 0.0 && !rng) return fail(DW_ERR_INVALID_ARG, "%s: rng must not be NULL when p > 0", fn);
    return DW_OK;
}

// The block operators' workspaces: large enough, and aligned for their vector
// and direct loads.
dw_status check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
    if (need && (!workspace || bytes < need))
        return fail(DW_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn, workspace ? bytes : (size_t)0, need);
    if (need && (uintptr_t)workspace % 16 != 0)
        return fail(DW_ERR_INVALID_ARG, "%s: the workspace must start on a multiple of 16 bytes", fn);
    return DW_OK;
}

dw_status check_norm_sizes(const char* fn, int64_t B, int64_t T, int64_t C) {
    if (B < 0 || T < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!dw::dwnorm_width_supported(C))
        return fail(DW_ERR_UNSUPPORTED, "%s: rows of C=%lld columns have no kernel (at most 8192)", fn, (long long)C);
    if (!extents_ok(B, T) || !dw::product_below(dw::kMaxExtent, {B, T})) return too_large(fn);
    return DW_OK;
}

dw_status dropout(const char* fn, const void* x, const void* residual, void* y, const uint64_t* rng, int64_t rows,
                  int64_t C, double p, float alpha, dw_dtype dtype, void* stream) {
    if (rows < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    dw_status s = check_dtype(fn, dtype);
    if (s == DW_OK) s = check_dropout(fn, p, rng);
    if (s != DW_OK) return s;
    if (rows == 0 || C == 0) return ok();
    if (!extents_ok(C) || !dw::dwdrop_fits(rows, C)) return too_large(fn);
    if (!x || !y) return fail(DW_ERR_INVALID_ARG, "%s: the input and the output must not be NULL", fn);
    return from_hip(dw::launch_dwdrop(x, residual, y, p > 0.0 ? rng : nullptr, rows, C, p, alpha, dtype == DW_BF16,
                                      (hipStream_t)stream), fn);
}

bool strides_ok(const dw_strides& s) { return s.item >= 0 && s.frame >= 0 && s.head >= 0; }

dw::AttnStride stride_of(const dw_strides& s) { return {s.item, s.frame, s.head}; }

// Offsets inside [n items][t frames][h heads] stay far below 2^63.
bool strides_fit(const dw_strides& s, int64_t n, int64_t t, int64_t h) {
    const int64_t far = (int64_t)1 << 58;
    return dw::product_below(far, {n, s.item}) && dw::product_below(far, {t + 256, s.frame}) &&
           dw::product_below(far, {h, s.head});
}

// A table without a map or the other way round; the table of no heads may be NULL.
bool half_a_bias(const dw_attn* a, const void* table, const int32_t* map) {
    return !table != !map && (table || !a || a->H != 0);
}

// The problem as the launchers take it.
dw_status check_attn(const char* fn, const dw_attn* a, bool bias, dw::AttnShape* s) {
    if (!a) return fail(DW_ERR_INVALID_ARG, "%s: shape must not be NULL", fn);
    if (a->B < 0 || a->Tq < 0 || a->Tk < 0 || a->H < 0 || a->Hkv < 0 || a->D < 0)
        return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!strides_ok(a->q) || !strides_ok(a->k) || !strides_ok(a->v))
        return fail(DW_ERR_INVALID_ARG, "%s: negative stride", fn);
    const dw_status t = check_dtype(fn, a->dtype);
    if (t != DW_OK) return t;
    if (a->H > 0 && (a->Hkv < 1 || a->H % a->Hkv != 0))
        return fail(DW_ERR_INVALID_ARG, "%s: H=%lld is not a multiple of Hkv=%lld", fn, (long long)a->H, (long long)a->Hkv);
    if (!(a->scale > 0.0f)) return fail(DW_ERR_INVALID_ARG, "%s: scale must be positive", fn);
    if (bias && (a->buckets < 1 || a->reach < 1))
        return fail(DW_ERR_INVALID_ARG, "%s: a bias needs at least one bucket and a reach of one frame", fn);
    if (a->D > dw::kAttnMaxHead)
        return fail(DW_ERR_UNSUPPORTED, "%s: heads of D=%lld have no kernel (at most 128)", fn, (long long)a->D);
    if (bias && a->reach > dw::kAttnMaxReach)
        return fail(DW_ERR_UNSUPPORTED, "%s: a reach of %lld frames has no kernel (at most 1024)", fn, (long long)a->reach);
    if (bias && !extents_ok(a->buckets)) return too_large(fn);
    if (!extents_ok(a->B, a->H, a->Hkv) || a->Tq > dw::kAttnMaxFrames || a->Tk > dw::kAttnMaxFrames ||
        !strides_fit(a->q, a->B, a->Tq, a->H) || !strides_fit(a->k, a->B, a->Tk, a->Hkv) ||
        !strides_fit(a->v, a->B, a->Tk, a->Hkv))
        return too_large(fn);
    const int64_t none = dw::kNoLimit;
    s->B = a->B, s->Tq = a->Tq, s->Tk = a->Tk, s->H = a->H, s->Hkv = a->Hkv, s->D = a->D;
    s->q = stride_of(a->q), s->k = stride_of(a->k), s->v = stride_of(a->v);
    s->dq = stride_of(a->dq), s->dk = stride_of(a->dk), s->dv = stride_of(a->dv);
    s->buckets = bias ? a->buckets : 0, s->reach = bias ? a->reach : 0;
    s->left = a->left < 0 || a->left > none ? none : a->left;
    s->right = a->right < 0 || a->right > none ? none : a->right;
    s->scale = a->scale;
    if (!dw::dwattn_fits(*s)) return too_large(fn);
    return DW_OK;
}

// How often p divides n, which is left without it.
int take_out(int64_t p, int64_t* n) {
    int e = 0;
    for (; *n % p == 0; *n /= p) ++e;
    return e;
}

// floor(m log(n/e) / log(reach/e)) for n >= e.  The quotient is a whole number
// k exactly where n^m e^k = reach^k e^m, which the exponents of the primes
// decide (a divisor that is no prime finds its primes taken out before it);
// elsewhere long double tells the floor.
int64_t log_steps(int64_t n, int64_t e, int64_t reach, int64_t m) {
    const long double t = m * (logl((long double)n / e) / logl((long double)reach / e));
    const int64_t k = llroundl(t);
    if (fabsl(t - k) > 1e-6L) return (int64_t)floorl(t);
    bool equal = true;
    for (int64_t p = 2, a = n, b = e, c = reach; p <= reach; ++p) {
        const int64_t of_n = take_out(p, &a), of_e = take_out(p, &b), of_reach = take_out(p, &c);
        equal = equal && m * of_n + k * of_e == k * of_reach + m * of_e;
    }
    return equal ? k : (int64_t)floorl(t);
}

}  // namespace

extern "C" {

int dw_abi_version(void) { return DW_ABI_VERSION; }

const char* dw_last_error(void) { return g_err; }

dw_status dwconv1d_fwd(const void* x, const void* w, const void* bias, const int32_t* lengths,
                       void* y, int64_t B, int64_t T, int64_t C, int64_t K,
                       dw_pad pad, dw_dtype dtype, void* stream) {
    const char* fn = "dwconv1d_fwd";
    if (B < 0 || T < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size (B=%lld T=%lld C=%lld)", fn, (long long)B, (long long)T, (long long)C);
    if (K < 1) return fail(DW_ERR_INVALID_ARG, "%s: kernel width K=%lld must be >= 1", fn, (long long)K);
    if (pad != DW_PAD_SYMMETRIC && pad != DW_PAD_CAUSAL) return fail(DW_ERR_INVALID_ARG, "%s: unknown pad mode %d", fn, (int)pad);
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (B == 0 || T == 0 || C == 0) return ok();
    if (!extents_ok(B, T, C, K)) return too_large(fn);
    if (!x || !w || !y) return fail(DW_ERR_INVALID_ARG, "%s: x, w and y must not be NULL", fn);
    if (x == y) return fail(DW_ERR_INVALID_ARG, "%s: y must not alias x", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    const void* ptrs[4] = {x, w, bias, y};
    const int vec = dw::pick_vec(C, es, ptrs, 4, dtype == DW_BF16 ? DW1D_BF16_VEC : 4);
    if (!dw::dwconv1d_fwd_fits(B, T, C, K, es, vec))
        return fail(DW_ERR_UNSUPPORTED, "%s: sizes too large for one launch (B=%lld T=%lld C=%lld K=%lld)", fn, (long long)B, (long long)T, (long long)C, (long long)K);
    const int64_t pL = pad == DW_PAD_CAUSAL ? K - 1 : (K - 1) / 2;
    return from_hip(dw::launch_dwconv1d_fwd(x, w, bias, lengths, y, B, T, C, K, pL, dtype == DW_BF16, vec,
                                            (hipStream_t)stream), fn);
}

dw_status dwconv1d_stream_fwd(const void* x, const void* w, const void* bias, const int32_t* lengths,
                              const void* cache_in, void* y, void* cache_out, int64_t B, int64_t Tc, int64_t C,
                              int64_t K, dw_dtype dtype, void* stream) {
    const char* fn = "dwconv1d_stream_fwd";
    if (B < 0 || Tc < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (K < 1) return fail(DW_ERR_INVALID_ARG, "%s: kernel width K=%lld must be >= 1", fn, (long long)K);
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (B == 0 || C == 0) return ok();
    if (!extents_ok(B, Tc, C, K)) return too_large(fn);
    const bool has_cache = K > 1;
    if ((!x && Tc > 0) || !w || (!y && Tc > 0) || (has_cache && (!cache_in || !cache_out)))
        return fail(DW_ERR_INVALID_ARG, "%s: x, w, y and the caches must not be NULL (unless empty)", fn);
    if (has_cache && cache_in == (const void*)cache_out)
        return fail(DW_ERR_INVALID_ARG, "%s: cache_out must be a different buffer from cache_in", fn);
    if (Tc > 0 && (x == (const void*)y || (has_cache && (y == cache_in || y == (const void*)cache_out))))
        return fail(DW_ERR_INVALID_ARG, "%s: y must not alias x or a cache", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    const void* ptrs[6] = {x, w, bias, y, cache_in, cache_out};
    const int vec = dw::pick_vec(C, es, ptrs, 6, dw::dwconv1d_stream_max_vec(K, dtype == DW_BF16));
    if (!dw::dwconv1d_stream_fits(B, Tc, C, K, es, vec)) return too_large(fn);
    return from_hip(dw::launch_dwconv1d_stream(x, w, bias, lengths, cache_in, y, cache_out, B, Tc, C, K,
                                               dtype == DW_BF16, vec, (hipStream_t)stream), fn);
}

size_t dwconv1d_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t K) {
    if (B < 0 || T < 0 || C < 0 || !dw::dwconv1d_bwd_supported(K)) return 0;
    if (!extents_ok(B, T, C) || !dw::dwconv1d_bwd_fits(B, T, C, K, 2)) return 0;
    return dw::dwconv1d_bwd_workspace(B, T, C, K);
}

dw_status dwconv1d_bwd(const void* x, const void* w, const int32_t* lengths, const void* dy, void* dx, float* dw_,
                       float* db, void* workspace, size_t workspace_bytes, int64_t B, int64_t T, int64_t C,
                       int64_t K, dw_pad pad, dw_dtype dtype, void* stream) {
    const char* fn = "dwconv1d_bwd";
    if (B < 0 || T < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (K < 1) return fail(DW_ERR_INVALID_ARG, "%s: kernel width K=%lld must be >= 1", fn, (long long)K);
    if (pad != DW_PAD_SYMMETRIC && pad != DW_PAD_CAUSAL) return fail(DW_ERR_INVALID_ARG, "%s: unknown pad mode %d", fn, (int)pad);
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (!dw::dwconv1d_bwd_supported(K))
        return fail(DW_ERR_UNSUPPORTED, "%s: kernel width K=%lld has no backward kernel (3, 4, 5, 7, 9, 15, 31)", fn, (long long)K);
    const bool want_wb = dw_ || db;
    if (!dx && !want_wb) return ok();
    if (C == 0) return ok();
    if ((!x && nonempty(B, T)) || (!dy && nonempty(B, T)) || !w)
        return fail(DW_ERR_INVALID_ARG, "%s: x, w and dy must not be NULL (unless empty)", fn);
    if (dx && (dx == x || dx == dy)) return fail(DW_ERR_INVALID_ARG, "%s: dx must not alias x or dy", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    if (!extents_ok(B, T, C) || !dw::dwconv1d_bwd_fits(B, T, C, K, es)) return too_large(fn);
    if (want_wb) {
        const size_t need = dw::dwconv1d_bwd_workspace(B, T, C, K);
        if (!workspace || workspace_bytes < need)
            return fail(DW_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn, workspace ? workspace_bytes : (size_t)0, need);
    }
    const void* ptrs[4] = {x, w, dy, dx};
    const int vec = dw::pick_vec(C, es, ptrs, 4, dw::dwconv1d_bwd_max_vec(K, dtype == DW_BF16));
    return from_hip(dw::launch_dwconv1d_bwd(x, w, lengths, dy, dx, dw_, db, workspace, B, T, C, K,
                                            pad == DW_PAD_CAUSAL, dtype == DW_BF16, vec, (hipStream_t)stream), fn);
}

dw_status dwsub_fused_fwd_ex(const void* x, const void* w0, const void* b0, const void* w1, const void* b1,
                             const int32_t* lengths, void* y, int64_t B, int64_t T, int64_t F, int64_t C,
                             dw_pad pad, dw_dtype dtype, void* stream) {
    const char* fn = "dwsub_fused_fwd";
    if (B < 0 || T < 0 || F < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    const dw_status ps = check_pad(fn, pad);
    if (ps != DW_OK) return ps;
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    const bool causal = pad == DW_PAD_CAUSAL;
    if (!extents_ok(B, T, F, C)) return too_large(fn);
    const dw::FrontDims fd = dw::front_dims(T, F, causal ? 1 : 0);
    if (B == 0 || fd.T2 == 0 || fd.F2 == 0 || C == 0) return ok();
    if ((!x && nonempty(T, F)) || !w0 || !w1 || !y)
        return fail(DW_ERR_INVALID_ARG, "%s: x, w0, w1 and y must not be NULL", fn);
    if (x == (const void*)y) return fail(DW_ERR_INVALID_ARG, "%s: y must not alias x", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    if (!dw::dwsub_fused_fwd_fits(B, T, F, C, causal, es)) return too_large(fn);
    return from_hip(dw::launch_dwsub_fused_fwd(x, w0, b0, w1, b1, lengths, y, B, T, F, C, causal, dtype == DW_BF16,
                                               (hipStream_t)stream), fn);
}

dw_status dwsub_fused_fwd(const float* x, const float* w0, const float* b0, const float* w1, const float* b1,
                          const int32_t* lengths, float* y, int64_t B, int64_t T, int64_t F, int64_t C,
                          void* stream) {
    return dwsub_fused_fwd_ex(x, w0, b0, w1, b1, lengths, y, B, T, F, C, DW_PAD_SYMMETRIC, DW_F32, stream);
}

size_t dwsub_fused_bwd_workspace_bytes_ex(int64_t B, int64_t T, int64_t F, int64_t C, dw_pad pad) {
    if (B < 0 || T < 0 || F < 0 || C < 0 || (pad != DW_PAD_SYMMETRIC && pad != DW_PAD_CAUSAL)) return 0;
    if (!extents_ok(B, T, F, C) || !dw::dwsub_fused_bwd_fits(B, T, F, C, pad == DW_PAD_CAUSAL, 2)) return 0;
    return dw::dwsub_fused_bwd_workspace(B, T, F, C, pad == DW_PAD_CAUSAL);
}

size_t dwsub_fused_bwd_workspace_bytes(int64_t B, int64_t T, int64_t F, int64_t C) {
    return dwsub_fused_bwd_workspace_bytes_ex(B, T, F, C, DW_PAD_SYMMETRIC);
}

dw_status dwsub_fused_bwd_ex(const void* x, const void* w0, const void* b0, const void* w1, const int32_t* lengths,
                             const void* dy, float* dw0, float* db0, float* dw1, float* db1, void* workspace,
                             size_t workspace_bytes, int64_t B, int64_t T, int64_t F, int64_t C, dw_pad pad,
                             dw_dtype dtype, void* stream) {
    const char* fn = "dwsub_fused_bwd";
    if (B < 0 || T < 0 || F < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    const dw_status ps = check_pad(fn, pad);
    if (ps != DW_OK) return ps;
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    const bool causal = pad == DW_PAD_CAUSAL;
    if (!dw0 && !db0 && !dw1 && !db1) return ok();
    if (C == 0) return ok();
    if (!extents_ok(B, T, F, C)) return too_large(fn);
    const dw::FrontDims fd = dw::front_dims(T, F, causal ? 1 : 0);
    if ((!x && nonempty(B, T, F)) || (!dy && nonempty(B, fd.T2, fd.F2, C)) || !w0 || !w1)
        return fail(DW_ERR_INVALID_ARG, "%s: x, w0, w1 and dy must not be NULL (unless empty)", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    if (!dw::dwsub_fused_bwd_fits(B, T, F, C, causal, es)) return too_large(fn);
    const size_t need = dw::dwsub_fused_bwd_workspace(B, T, F, C, causal);
    if (!workspace || workspace_bytes < need)
        return fail(DW_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                    workspace ? workspace_bytes : (size_t)0, need);
    return from_hip(dw::launch_dwsub_fused_bwd(x, w0, b0, w1, lengths, dy, dw0, db0, dw1, db1, workspace, B, T, F, C,
                                               causal, dtype == DW_BF16, (hipStream_t)stream), fn);
}

dw_status dwsub_fused_bwd(const float* x, const float* w0, const float* b0, const float* w1,
                          const int32_t* lengths, const float* dy, float* dw0, float* db0, float* dw1, float* db1,
                          void* workspace, size_t workspace_bytes, int64_t B, int64_t T, int64_t F, int64_t C,
                          void* stream) {
    return dwsub_fused_bwd_ex(x, w0, b0, w1, lengths, dy, dw0, db0, dw1, db1, workspace, workspace_bytes, B, T, F, C,
                              DW_PAD_SYMMETRIC, DW_F32, stream);
}

dw_status dwconv2d_fwd_ex(const void* x, const void* w, const void* bias, const int32_t* lengths, void* y,
                          int64_t B, int64_t T, int64_t F, int64_t C, int64_t KH, int64_t KW, int64_t stride,
                          int64_t pad_t0, int64_t pad_t1, int64_t pad_f0, int64_t pad_f1, dw_dtype dtype,
                          void* stream) {
    const char* fn = "dwconv2d_fwd";
    if (B < 0 || T < 0 || F < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    const dw_status gs = check_geometry_2d(fn, KH, KW, stride, pad_t0, pad_t1, pad_f0, pad_f1);
    if (gs != DW_OK) return gs;
    if (!extents_ok(B, T, F, C)) return too_large(fn);
    const dw::Conv2dGeom g = dw::conv2d_geom(T, F, C, pad_t0, pad_t1, pad_f0, pad_f1);
    if (B == 0 || g.To == 0 || g.Fo == 0 || C == 0) return ok();
    if ((!x && nonempty(T, F)) || !w || !y) return fail(DW_ERR_INVALID_ARG, "%s: x, w and y must not be NULL", fn);
    if (x == (const void*)y) return fail(DW_ERR_INVALID_ARG, "%s: y must not alias x", fn);
    const int es = dtype == DW_BF16 ? 2 : 4;
    const void* ptrs[4] = {x, w, bias, y};
    const int vec = dw::pick_vec(C, es, ptrs, 4, dtype == DW_BF16 ? 8 : 4);
    if (!dw::dwconv2d_fits(B, g, es)) return too_large(fn);
    return from_hip(dw::launch_dwconv2d_fwd(x, w, bias, lengths, y, B, g, dtype == DW_BF16, vec,
                                            (hipStream_t)stream), fn);
}

dw_status dwconv2d_fwd(const float* x, const float* w, const float* bias, const int32_t* lengths, float* y,
                       int64_t B, int64_t T, int64_t F, int64_t C, int64_t KH, int64_t KW, int64_t stride,
                       int64_t pad, void* stream) {
    return dwconv2d_fwd_ex(x, w, bias, lengths, y, B, T, F, C, KH, KW, stride, pad, pad, pad, pad, DW_F32, stream);
}

size_t dwconv2d_bwd_workspace_bytes_ex(int64_t B, int64_t T, int64_t F, int64_t C, int64_t KH, int64_t KW,
                                       int64_t stride, int64_t pad_t0, int64_t pad_t1, int64_t pad_f0,
                                       int64_t pad_f1) {
    if (B < 0 || T < 0 || F < 0 || C < 0 || !geometry_ok_2d(KH, KW, stride, pad_t0, pad_t1, pad_f0, pad_f1)) return 0;
    if (!extents_ok(B, T, F, C)) return 0;
    const dw::Conv2dGeom g = dw::conv2d_geom(T, F, C, pad_t0, pad_t1, pad_f0, pad_f1);
    if (!dw::dwconv2d_fits(B, g, 2)) return 0;
    return dw::dwconv2d_bwd_workspace(B, g);
}

size_t dwconv2d_bwd_workspace_bytes(int64_t B, int64_t T, int64_t F, int64_t C, int64_t KH, int64_t KW,
                                    int64_t stride, int64_t pad) {
    return dwconv2d_bwd_workspace_bytes_ex(B, T, F, C, KH, KW, stride, pad, pad, pad, pad);
}

// The conv2d backward's checks and launch.  With use_scratch, the fp64
// partials go to the library's own per-device scratch array (allocation-free
// entry point) instead of the caller's workspace.
static dw_status dwconv2d_bwd_impl(const char* fn, const void* x, const void* w, const int32_t* lengths,
                                   const void* dy, void* dx, float* dw_, float* db, void* workspace,
                                   size_t workspace_bytes, bool use_scratch, int64_t B, int64_t T, int64_t F,
                                   int64_t C, int64_t KH, int64_t KW, int64_t stride, int64_t pad_t0,
                                   int64_t pad_t1, int64_t pad_f0, int64_t pad_f1, dw_dtype dtype, void* stream) {
    if (B < 0 || T < 0 || F < 0 || C < 0) return fail(DW_ERR_INVALID_ARG, "%s: negative size", fn);
    if (dtype != DW_F32 && dtype != DW_BF16) return fail(DW_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    const dw_status gs = check_geometry_2d(fn, KH, KW, stride, pad_t0, pad_t1, pad_f0, pad_f1);
    if (gs != DW_OK) return gs;
    if (!extents_ok(B, T, F, C)) return too_large(fn);
    const dw::Conv2dGeom g = dw::conv2d_geom(T, F, C, pad_t0, pad_t1, pad_f0, pad_f1);
    if ((!x && nonempty(B, T, F, C)) || (!dy && nonempty(B, g.To, g.Fo, C)) || (!w && C > 0))
        return fail(DW_ERR_INVALID_ARG, "%s: x, w and dy must not be NULL (unless empty)", fn);
    if (dx && (dx == x || dx == dy)) return fail(DW_ERR_INVALID_ARG, "%s: dx must not alias x or dy", fn);
    const bool want_wb = dw_ || db;
    const int es = dtype == DW_BF16 ? 2 : 4;
    if (!dw::dwconv2d_fits(B, g, es)) return too_large(fn);
    if (want_wb) {
        const size_t need = dw::dwconv2d_bwd_workspace(B, g);
        if (use_scratch) {
            if (need > dw::kScratchBytes)
                return fail(DW_ERR_UNSUPPORTED, "%s: dw and db need %zu bytes of scratch, more than the %zu bytes "
                            "this allocation-free entry point holds (C = %lld; at most about 800 channels fit)", fn,
                            need, dw::kScratchBytes, (long long)C);
        } else if (!workspace || workspace_bytes < need) {
            return fail(DW_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                        workspace ? workspace_bytes : (size_t)0, need);
        }
    }
    if (!dx && !want_wb) return ok();
    if (C == 0) return ok();
    if (use_scratch && want_wb) {
        const hipError_t e = dw::scratch_on_current_device(&workspace);
        if (e != hipSuccess)
            return fail(DW_ERR_HIP, "%s: the device address of the library's scratch array: %s", fn,
                        hipGetErrorString(e));
    }
    // An empty batch or item still defines dw = 0 and db = 0; the launcher
    // writes those zeros when there is nothing to reduce.
    const void* ptrs[4] = {x, w, dy, dx};
    const int vec = dw::pick_vec(C, es, ptrs, 4, dtype == DW_BF16 ? 8 : 4);
    return from_hip(dw::launch_dwconv2d_bwd(x, w, lengths, dy, dx, dw_, db, workspace, B, g, dtype == DW_BF16, vec,
                                            (hipStream_t)stream), fn);
}

dw_status dwconv2d_bwd_ex(const void* x, const void* w, const int32_t* lengths, const void* dy, void* dx,
                          float* dw_, float* db, void* workspace, size_t workspace_bytes, int64_t B, int64_t T,
                          int64_t F, int64_t C, int64_t KH, int64_t KW, int64_t stride, int64_t pad_t0,
                          int64_t pad_t1, int64_t pad_f0, int64_t pad_f1, dw_dtype dtype, void* stream) {
    return dwconv2d_bwd_impl("dwconv2d_bwd", x, w, lengths, dy, dx, dw_, db, workspace, workspace_bytes, false, B, T,
                             F, C, KH, KW, stride, pad_t0, pad_t1, pad_f0, pad_f1, dtype, stream);
}

dw_status dwconv2d_bwd_noalloc(const void* x, const void* w, const int32_t* lengths, const void* dy, void* dx,
                               float* dw_, float* db, int64_t B, int64_t T, int64_t F, int64_t C, int64_t KH,
                               int64_t KW, int64_t stride, int64_t pad_t0, int64_t pad_t1, int64_t pad_f0,
                               int64_t pad_f1, dw_dtype dtype, void* stream) {
    return dwconv2d_bwd_impl("dwconv2d_bwd_noalloc", x, w, lengths, dy, dx, dw_, db, nullptr, 0, true, B, T, F, C,
                             KH, KW, stride, pad_t0, pad_t1, pad_f0, pad_f1, dtype, stream);
}

dw_status dwconv2d_bwd(const float* x, const float* w, const int32_t* lengths, const float* dy, float* dx,
                       float* dw_, float* db, void* workspace, size_t workspace_bytes, int64_t B, int64_t T,
                       int64_t F, int64_t C, int64_t KH, int64_t KW, int64_t stride, int64_t pad,
                       void* stream) {
    return dwconv2d_bwd_ex(x, w, lengths, dy, dx, dw_, db, workspace, workspace_bytes, B, T, F, C, KH, KW, stride,
                           pad, pad, pad, pad, DW_F32, stream);
}

dw_status dwdrop_fwd(const void* x, const void* residual, void* y, const uint64_t* rng, int64_t rows, int64_t C,
                     double p, float alpha, dw_dtype dtype, void* stream) {
    return dropout("dwdrop_fwd", x, residual, y, rng, rows, C, p, alpha, dtype, stream);
}

dw_status dwdrop_bwd(const void* dy, void* dx, const uint64_t* rng, int64_t rows, int64_t C, double p, float alpha,
                     dw_dtype dtype, void* stream) {
    return dropout("dwdrop_bwd", dy, nullptr, dx, rng, rows, C, p, alpha, dtype, stream);
}

dw_status dwnorm_fwd(const void* x, const void* residual, const void* gamma, const void* beta, const int32_t* lengths,
                     const uint64_t* rng, void* y, void* sum, float* mean, float* rstd, int64_t B, int64_t T,
                     int64_t C, float eps, float alpha, double p, dw_dtype dtype, void* stream) {
    const char* fn = "dwnorm_fwd";
    dw_status s = check_norm_sizes(fn, B, T, C);
    if (s == DW_OK) s = check_dtype(fn, dtype);
    if (s == DW_OK) s = check_dropout(fn, p, rng);
    if (s != DW_OK) return s;
    if (!(eps >= 0.0f)) return fail(DW_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    if (B == 0 || T == 0 || C == 0) return ok();
    if (!dw::dwnorm_fwd_fits(B * T, C)) return too_large(fn);
    if (!x || !y) return fail(DW_ERR_INVALID_ARG, "%s: x and y must not be NULL", fn);
    if (y == sum) return fail(DW_ERR_INVALID_ARG, "%s: y must not alias sum", fn);
    return from_hip(dw::launch_dwnorm_fwd(x, residual, gamma, beta, lengths, p > 0.0 ? rng : nullptr, y, sum, mean,
                                          rstd, B, T, C, eps, alpha, p, dtype == DW_BF16, (hipStream_t)stream), fn);
}

size_t dwnorm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C) {
    if (B < 0 || T < 0 || C < 0 || !dw::dwnorm_width_supported(C)) return 0;
    if (!extents_ok(B, T) || !dw::product_below(dw::kMaxExtent, {B, T})) return 0;
    return dw::dwnorm_bwd_workspace(B, T, C);
}

dw_status dwnorm_bwd(const void* sum, const void* gamma, const int32_t* lengths, const float* mean, const float* rstd,
                     const void* dy, const void* dsum, const uint64_t* rng, void* dx, void* dres, float* dgamma,
                     float* dbeta, void* workspace, size_t workspace_bytes, int64_t B, int64_t T, int64_t C,
                     float alpha, double p, dw_dtype dtype, void* stream) {
    const char* fn = "dwnorm_bwd";
    dw_status s = check_norm_sizes(fn, B, T, C);
    if (s == DW_OK) s = check_dtype(fn, dtype);
    if (s == DW_OK) s = check_dropout(fn, p, rng);
    if (s != DW_OK) return s;
    const bool params = dgamma || dbeta;
    if ((!dx && !dres && !params) || C == 0) return ok();
    if (nonempty(B, T) && (!sum || !mean || !rstd || !dy))
        return fail(DW_ERR_INVALID_ARG, "%s: sum, mean, rstd and dy must not be NULL (unless empty)", fn);
    if (dx && dx == dres) return fail(DW_ERR_INVALID_ARG, "%s: dx must not alias dres", fn);
    if (params) {
        const dw_status w = check_workspace(fn, workspace, workspace_bytes, dw::dwnorm_bwd_workspace(B, T, C));
        if (w != DW_OK) return w;
    }
    return from_hip(dw::launch_dwnorm_bwd(sum, gamma, lengths, mean, rstd, dy, dsum, p > 0.0 ? rng : nullptr, dx, dres,
                                          dgamma, dbeta, workspace, B, T, C, alpha, p, dtype == DW_BF16,
                                          (hipStream_t)stream), fn);
}

dw_status dwattn_rel_buckets(int32_t* map, int64_t buckets, int64_t reach, int bidirectional) {
    const char* fn = "dwattn_rel_buckets";
    const int64_t per = bidirectional ? buckets / 2 : buckets, e = per / 2;
    if (!map) return fail(DW_ERR_INVALID_ARG, "%s: map must not be NULL", fn);
    if (buckets < 1 || per < 1) return fail(DW_ERR_INVALID_ARG, "%s: fewer than one bucket a direction", fn);
    if (buckets > 65536) return fail(DW_ERR_UNSUPPORTED, "%s: over 65536 buckets", fn);
    if (reach < 1 || reach <= e)
        return fail(DW_ERR_INVALID_ARG, "%s: the reach must be past the %lld distances with a bucket each", fn, (long long)e);
    if (reach > dw::kAttnMaxReach) return fail(DW_ERR_UNSUPPORTED, "%s: a reach over 1024 frames", fn);
    for (int64_t n = 0; n <= reach; ++n) {
        int64_t b = n;
        if (n >= e) {
            const int64_t k = e > 0 ? log_steps(n, e, reach, per - e) : 0;
            b = e + (k < per - e ? k : per - e - 1);
        }
        map[reach - n] = (int32_t)b;
        if (n > 0) map[reach + n] = (int32_t)(bidirectional ? per + b : 0);
    }
    return ok();
}

size_t dwattn_fwd_workspace_bytes(const dw_attn* shape) {
    dw::AttnShape s;
    if (check_attn("dwattn_fwd_workspace_bytes", shape, false, &s) != DW_OK) return 0;
    return dw::dwattn_fwd_fits(s) ? dw::dwattn_fwd_workspace(s) : 0;
}

dw_status dwattn_fwd(const dw_attn* shape, const void* q, const void* k, const void* v, const void* table,
                     const int32_t* map, const int32_t* q_lengths, const int32_t* k_lengths, const int32_t* q_pos,
                     void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "dwattn_fwd";
    if (half_a_bias(shape, table, map)) return fail(DW_ERR_INVALID_ARG, "%s: a bias needs both its table and its map", fn);
    dw::AttnShape s;
    const dw_status c = check_attn(fn, shape, table != nullptr, &s);
    if (c != DW_OK) return c;
    if (!nonempty(s.B, s.Tq, s.H, s.D)) return ok();
    if (!dw::dwattn_fwd_fits(s)) return too_large(fn);
    if (!q || !out || (s.Tk > 0 && (!k || !v)))
        return fail(DW_ERR_INVALID_ARG, "%s: q, k, v and out must not be NULL (unless empty)", fn);
    if (out == q || out == k || out == v) return fail(DW_ERR_INVALID_ARG, "%s: out must not alias an input", fn);
    const dw_status w = check_workspace(fn, workspace, workspace_bytes, dw::dwattn_fwd_workspace(s));
    if (w != DW_OK) return w;
    const dw::AttnPtrs p = {q, k, v, table, map, q_lengths, k_lengths, q_pos};
    return from_hip(dw::launch_dwattn_fwd(p, s, out, lse, workspace, shape->dtype == DW_BF16, (hipStream_t)stream), fn);
}

size_t dwattn_bwd_workspace_bytes(const dw_attn* shape) {
    dw::AttnShape s;
    if (!shape || check_attn("dwattn_bwd_workspace_bytes", shape, shape->buckets > 0, &s) != DW_OK) return 0;
    const int elem = shape->dtype == DW_BF16 ? 2 : 4;
    return dw::dwattn_bwd_fits(s, elem) ? dw::dwattn_bwd_workspace(s, elem) : 0;
}

dw_status dwattn_bwd(const dw_attn* shape, const void* q, const void* k, const void* v, const void* table,
                     const int32_t* map, const int32_t* q_lengths, const int32_t* k_lengths, const int32_t* q_pos,
                     const void* out, const float* lse, const void* dout, void* dq, void* dk, void* dv, float* dtable,
                     void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "dwattn_bwd";
    if (half_a_bias(shape, table, map)) return fail(DW_ERR_INVALID_ARG, "%s: a bias needs both its table and its map", fn);
    if (dtable && !table) return fail(DW_ERR_INVALID_ARG, "%s: dtable needs a table", fn);
    dw::AttnShape s;
    const dw_status c = check_attn(fn, shape, table != nullptr, &s);
    if (c != DW_OK) return c;
    if (!strides_ok(shape->dq) || !strides_ok(shape->dk) || !strides_ok(shape->dv))
        return fail(DW_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (!dw::dwattn_bwd_fits(s, shape->dtype == DW_BF16 ? 2 : 4) || (dq && !strides_fit(shape->dq, s.B, s.Tq, s.H)) || (dk && !strides_fit(shape->dk, s.B, s.Tk, s.Hkv)) ||
        (dv && !strides_fit(shape->dv, s.B, s.Tk, s.Hkv)))
        return too_large(fn);
    if ((!dq && !dk && !dv && !dtable) || (s.H == 0 && (s.Hkv == 0 || (!dk && !dv)))) return ok();
    if (!dtable && (s.B == 0 || s.D == 0)) return ok();
    if (nonempty(s.B, s.Tq, s.H) && (!lse || (s.D > 0 && (!q || !out || !dout))))
        return fail(DW_ERR_INVALID_ARG, "%s: q, out, lse and dout must not be NULL (unless empty)", fn);
    if (nonempty(s.B, s.Tk, s.Hkv, s.D) && (!k || !v))
        return fail(DW_ERR_INVALID_ARG, "%s: k and v must not be NULL (unless empty)", fn);
    for (const void* o : {(const void*)dq, (const void*)dk, (const void*)dv})
        if (o && (o == q || o == k || o == v || o == out || o == dout))
            return fail(DW_ERR_INVALID_ARG, "%s: a gradient must not alias an input", fn);
    if ((dq && (dq == dk || dq == dv)) || (dk && dk == dv))
        return fail(DW_ERR_INVALID_ARG, "%s: the gradients must not alias each other", fn);
    const dw_status w =
        check_workspace(fn, workspace, workspace_bytes, dw::dwattn_bwd_workspace(s, shape->dtype == DW_BF16 ? 2 : 4));
    if (w != DW_OK) return w;
    const dw::AttnPtrs p = {q, k, v, table, map, q_lengths, k_lengths, q_pos};
    return from_hip(dw::launch_dwattn_bwd(p, s, out, lse, dout, dq, dk, dv, dtable, workspace, shape->dtype == DW_BF16,
                                          (hipStream_t)stream), fn);
}

}  // extern "C"
