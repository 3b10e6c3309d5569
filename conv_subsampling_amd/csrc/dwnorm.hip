// Layer norm over the last axis of [B][T][C] with the residual add and the
// dropout of a pre-norm block in front of it, its backward pass, and dropout
// by itself.
//
//   s = residual + alpha * drop(x);  y = (s - mean) * rstd * gamma + beta
//
// The statistics are those of the unrounded s.  A row lives in registers from
// its load to its store: LANES neighbouring lanes hold it as NG groups of 8
// columns each (WAVES > 1: a workgroup holds one row), so the mean and the
// variance are two passes over registers and memory sees each tensor once.
//
// All of it is bound by memory.  Measured against the 5.19 TB/s of a large copy,
// kernels in a row under the profiler: forward of [16,750,1024] bf16 with residual
// and dropout (87 MB over its valid frames) 16.4 us, 5.3 TB/s (float 34.4, 5.0;
// float [32,1500,512] 67.4, 5.1); backward with both
// residual gradients (106 MB) 24 to 26 us, 4.1 to 4.5 TB/s, and 3.9 us for the
// weights' sums.
#include "launch.h"
#include "rowops.h"

namespace dw {

constexpr int kNormThreads = 256, kNormWaves = kNormThreads / 64;
constexpr int64_t kNormMaxWidth = 8192;  // what a workgroup's registers hold of one row
constexpr int64_t kNormBwdBlocks = 512;  // workgroups (and partial rows) of the backward at most

struct NormFwd {
    const void *x, *residual, *gamma, *beta;
    const int32_t* lengths;
    const uint64_t* rng;
    void *y, *sum;
    float *mean, *rstd;
    uint32_t rows, T;
    int32_t C;
    float eps, alpha, keep_scale;
    uint32_t threshold;
};

struct NormBwd {
    const void *s, *gamma, *dy, *dsum;
    const int32_t* lengths;
    const float *mean, *rstd;
    const uint64_t* rng;
    void *dx, *dres;
    float* partial;  // [gridDim.x][2][C]: sums of dy * xhat and of dy; NULL: not wanted
    uint32_t rows, T;
    int32_t C;
    float alpha, keep_scale;
    uint32_t threshold;
};

__device__ __forceinline__ bool row_live(const int32_t* lengths, uint32_t row, uint32_t T) {
    if (!lengths) return true;
    const uint32_t b = row / T;
    return (int32_t)(row - b * T) < lengths[b];
}

// The sum of v over the lanes that hold the row.
template <int LANES, int WAVES>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
    v = lane_sum<LANES>(v);
    if constexpr (WAVES > 1) {
        __syncthreads();
        if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += scratch[w];
    }
    return v;
}

template <typename S, bool TAIL, int LANES, int NG, int WAVES>
__global__ __launch_bounds__(kNormThreads) void norm_fwd_kernel(const NormFwd a) {
    constexpr int kHolders = LANES * WAVES;  // lanes that hold one row
    __shared__ float scratch[WAVES];
    const uint32_t row = blockIdx.x * (uint32_t)(kNormThreads / kHolders) + threadIdx.x / kHolders;
    if (WAVES == 1 && row >= a.rows) return;  // WAVES > 1: the grid is exactly the rows
    const int lane = threadIdx.x % kHolders, C = a.C;
    const int64_t base = (int64_t)row * C;
    S* y = (S*)a.y + base;
    S* sum = a.sum ? (S*)a.sum + base : nullptr;
    if (!row_live(a.lengths, row, a.T)) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int col = (j * kHolders + lane) * kGroup;
            store_group<S, TAIL>(y, col, C, vzero<kGroup>());
            if (sum) store_group<S, TAIL>(sum, col, C, vzero<kGroup>());
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = 0.0f;
            if (a.rstd) a.rstd[row] = 0.0f;
        }
        return;
    }
    RawGroup<S> xr[NG], rr[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j)
        xr[j] = load_group<S, TAIL>((const S*)a.x + base, (j * kHolders + lane) * kGroup, C);
    if (a.residual) {
#pragma unroll
        for (int j = 0; j < NG; ++j)
            rr[j] = load_group<S, TAIL>((const S*)a.residual + base, (j * kHolders + lane) * kGroup, C);
    }
    Vf<kGroup> v[NG];
    if (a.rng) {
        const DropKeys keys = drop_keys(a.rng);
        const uint64_t groups = ((uint32_t)C + kGroup - 1) / kGroup;
#pragma unroll
        for (int j = 0; j < NG; ++j)
            v[j] = drop_group(widen<S>(xr[j]), philox(row * groups + j * kHolders + lane, keys), a.threshold,
                              a.alpha * a.keep_scale);
    } else {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            v[j] = widen<S>(xr[j]);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) v[j].v[e] *= a.alpha;
        }
    }
    if (a.residual) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const Vf<kGroup> r = widen<S>(rr[j]);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) v[j].v[e] += r.v[e];
        }
    }
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        if (sum) store_group<S, TAIL>(sum, (j * kHolders + lane) * kGroup, C, v[j]);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) t += v[j].v[e];
    }
    const float width = (float)C;
    const float mean = row_sum<LANES, WAVES>(t, scratch) / width;
    t = 0.0f;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const int col = (j * kHolders + lane) * kGroup;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            const bool in = TAIL ? col + e < C : col < C;
            v[j].v[e] = in ? v[j].v[e] - mean : 0.0f;
            t += v[j].v[e] * v[j].v[e];
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<LANES, WAVES>(t, scratch) / width + a.eps);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const int col = (j * kHolders + lane) * kGroup;
        Vf<kGroup> o;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) o.v[e] = v[j].v[e] * rstd;
        if (a.gamma) {
            const Vf<kGroup> g = widen<S>(load_group<S, TAIL>((const S*)a.gamma, col, C));
#pragma unroll
            for (int e = 0; e < kGroup; ++e) o.v[e] *= g.v[e];
        }
        if (a.beta) {
            const Vf<kGroup> b = widen<S>(load_group<S, TAIL>((const S*)a.beta, col, C));
#pragma unroll
            for (int e = 0; e < kGroup; ++e) o.v[e] += b.v[e];
        }
        store_group<S, TAIL>(y, col, C, o);
    }
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// At most kNormBwdBlocks workgroups take the rows in turn.  256, 512, 768, 1024
// and 2048 of them, with the sums of their partials, us from cold memory: bf16
// [16,750,1024] 41 39 39 42 44, [32,1500,512] 92 68 65 68 74, [8,1500,256] 21 19 18 19
// 23, [16,750,2048] 72 72 74 74 79, [16,750,4096] 117 120 123 135 149; float
// [16,750,1024] 70 69 69 72 75, [4,1500,4096] 120 122 129 135 147.  Fewer leave memory
// waiting, more write more partial sums.  A row loaded ahead gained nothing.
// One workgroup takes rows first, first + stride, ...; each lane keeps the
// weight gradients of its own columns in fp32 registers over them (a few tens
// of rows), the workgroup adds its waves in order and writes one partial row,
// and norm_param_reduce adds those in fp64 in order: no atomics, so repeated
// calls agree bit for bit.
template <typename S, bool TAIL, int LANES, int NG, int WAVES>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(const NormBwd a) {
    constexpr int kHolders = LANES * WAVES, kRows = kNormThreads / kHolders;
    __shared__ float scratch[WAVES];
    __shared__ float column[WAVES == 1 ? 2 * LANES * NG * kGroup : 1];
    const int lane = threadIdx.x % kHolders, C = a.C;
    const float width = (float)C;
    DropKeys keys = {};
    if (a.rng) keys = drop_keys(a.rng);
    const uint64_t groups = ((uint32_t)C + kGroup - 1) / kGroup;
    Vf<kGroup> gamma[NG], dg[NG], db[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        dg[j] = db[j] = vzero<kGroup>();
        if (a.gamma) {
            gamma[j] = widen<S>(load_group<S, TAIL>((const S*)a.gamma, (j * kHolders + lane) * kGroup, C));
        } else {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) gamma[j].v[e] = 1.0f;
        }
    }
    for (uint64_t first = (uint64_t)blockIdx.x * kRows; first < a.rows; first += (uint64_t)gridDim.x * kRows) {
        const uint64_t at = first + threadIdx.x / kHolders;
        if (WAVES == 1 && at >= a.rows) break;  // WAVES > 1: one row per workgroup, always in range
        const uint32_t row = (uint32_t)at;
        const int64_t base = (int64_t)row * C;
        S* dx = a.dx ? (S*)a.dx + base : nullptr;
        S* dres = a.dres ? (S*)a.dres + base : nullptr;
        if (!row_live(a.lengths, row, a.T)) {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int col = (j * kHolders + lane) * kGroup;
                if (dx) store_group<S, TAIL>(dx, col, C, vzero<kGroup>());
                if (dres) store_group<S, TAIL>(dres, col, C, vzero<kGroup>());
            }
            continue;
        }
        RawGroup<S> sr[NG], dyr[NG], dsr[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int col = (j * kHolders + lane) * kGroup;
            sr[j] = load_group<S, TAIL>((const S*)a.s + base, col, C);
            dyr[j] = load_group<S, TAIL>((const S*)a.dy + base, col, C);
        }
        if (a.dsum) {
#pragma unroll
            for (int j = 0; j < NG; ++j)
                dsr[j] = load_group<S, TAIL>((const S*)a.dsum + base, (j * kHolders + lane) * kGroup, C);
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        Vf<kGroup> xh[NG], g[NG];
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const Vf<kGroup> s = widen<S>(sr[j]), dy = widen<S>(dyr[j]);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                // columns past C hold dy = 0, so they add nothing to any sum
                xh[j].v[e] = (s.v[e] - mean) * rstd;
                g[j].v[e] = dy.v[e] * gamma[j].v[e];
                dg[j].v[e] += dy.v[e] * xh[j].v[e];
                db[j].v[e] += dy.v[e];
                t0 += g[j].v[e];
                t1 += g[j].v[e] * xh[j].v[e];
            }
        }
        t0 = row_sum<LANES, WAVES>(t0, scratch) / width;
        t1 = row_sum<LANES, WAVES>(t1, scratch) / width;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int col = (j * kHolders + lane) * kGroup;
            Vf<kGroup> ds;
#pragma unroll
            for (int e = 0; e < kGroup; ++e) ds.v[e] = rstd * (g[j].v[e] - t0 - xh[j].v[e] * t1);
            if (a.dsum) {
                const Vf<kGroup> d = widen<S>(dsr[j]);
#pragma unroll
                for (int e = 0; e < kGroup; ++e) ds.v[e] += d.v[e];
            }
            if (dres) store_group<S, TAIL>(dres, col, C, ds);
            if (dx) {
                if (a.rng) {
                    ds = drop_group(ds, philox(row * groups + j * kHolders + lane, keys), a.threshold,
                                    a.alpha * a.keep_scale);
                } else {
#pragma unroll
                    for (int e = 0; e < kGroup; ++e) ds.v[e] *= a.alpha;
                }
                store_group<S, TAIL>(dx, col, C, ds);
            }
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * C;
    if constexpr (WAVES == 1) {
        constexpr int kCols = LANES * NG * kGroup;
        for (int w = 0; w < kNormWaves; ++w) {
            if (threadIdx.x / 64 == w) {
#pragma unroll
                for (int j = 0; j < NG; ++j) {
#pragma unroll
                    for (int e = 0; e < kGroup; ++e) {
                        float u = dg[j].v[e], v = db[j].v[e];
#pragma unroll
                        for (int m = LANES; m < 64; m *= 2) {  // the wave's other rows
                            u += __shfl_xor(u, m);
                            v += __shfl_xor(v, m);
                        }
                        const int at = (j * LANES + lane) * kGroup + e;
                        if (threadIdx.x % 64 < LANES) {
                            column[at] = w ? column[at] + u : u;
                            column[kCols + at] = w ? column[kCols + at] + v : v;
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < C; c += kNormThreads) {
            out[c] = column[c];
            out[C + c] = column[kCols + c];
        }
    } else {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int col = (j * kHolders + lane) * kGroup;
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                if (col + e < C) {
                    out[col + e] = dg[j].v[e];
                    out[C + col + e] = db[j].v[e];
                }
            }
        }
    }
}

// 3 to 4 us, a launch and two rounds of loads: column sums of the [P][2][C] partials: 16 sub-rows x 64 columns a workgroup,
// sub-row q adding partials q, q + 16, ... in fp64, then the sub-rows in order.
constexpr int kParamCols = 64, kParamRows = 16;

__global__ __launch_bounds__(kParamCols* kParamRows) void norm_param_reduce(
    const float* __restrict__ partial, float* __restrict__ dgamma, float* __restrict__ dbeta, int32_t C, int32_t P) {
    __shared__ double acc[kParamRows][kParamCols];
    const int lane = threadIdx.x % kParamCols, sub = threadIdx.x / kParamCols;
    const int64_t ncol = 2 * (int64_t)C, col = (int64_t)blockIdx.x * kParamCols + lane;
    double s = 0.0;
    if (col < ncol) {
#pragma unroll 8
        for (int32_t r = sub; r < P; r += kParamRows) s += partial[r * ncol + col];
    }
    acc[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= ncol) return;
    double t = acc[0][lane];
#pragma unroll
    for (int q = 1; q < kParamRows; ++q) t += acc[q][lane];
    float* out = col < C ? dgamma : dbeta;
    if (out) out[col < C ? col : col - C] = (float)t;
}

// ---------------------------------------------------------------------------
// Dropout by itself: y = residual + alpha * drop(x).  Bound by memory: the
// generator's 20 wide multiplies serve 8 elements and hide behind the loads.
// [16,750,4096] bf16 (197 MB) takes 33.2 us, 5.9 TB/s; float [32,1500,512], the
// same bytes, 33.9 us; with a residual (295 MB) 48.1 and 48.8 us, 6.1 TB/s.
// ---------------------------------------------------------------------------
struct Drop {
    const void *x, *residual;
    void* y;
    const uint64_t* rng;
    uint64_t groups;  // in all
    uint32_t per_row;
    int32_t C;
    float scale;
    uint32_t threshold;
};

constexpr int kDropThreads = 256, kDropGroups = 4;  // groups a thread holds, so that its loads are in flight together

template <typename S, bool TAIL>
__global__ __launch_bounds__(kDropThreads) void drop_kernel(const Drop a) {
    const uint64_t first = (uint64_t)blockIdx.x * (kDropThreads * kDropGroups) + threadIdx.x;
    int64_t base[kDropGroups];
    int col[kDropGroups];
    RawGroup<S> xr[kDropGroups], rr[kDropGroups];
#pragma unroll
    for (int j = 0; j < kDropGroups; ++j) {
        const uint64_t g = first + j * kDropThreads;
        if constexpr (TAIL) {
            const uint64_t row = a.groups >> 32 ? g / a.per_row : (uint32_t)g / a.per_row;
            base[j] = (int64_t)row * a.C;
            col[j] = g < a.groups ? (int)(g - row * a.per_row) * kGroup : a.C;
        } else {  // whole groups lie end to end: one of them is a row of its own
            base[j] = (int64_t)g * kGroup;
            col[j] = g < a.groups ? 0 : a.C;
        }
        xr[j] = load_group<S, TAIL>((const S*)a.x + base[j], col[j], a.C);
    }
    if (a.residual) {
#pragma unroll
        for (int j = 0; j < kDropGroups; ++j)
            rr[j] = load_group<S, TAIL>((const S*)a.residual + base[j], col[j], a.C);
    }
    DropKeys keys = {};
    if (a.rng) keys = drop_keys(a.rng);
#pragma unroll
    for (int j = 0; j < kDropGroups; ++j) {
        Vf<kGroup> v = widen<S>(xr[j]);
        if (a.rng) {
            v = drop_group(v, philox(first + j * kDropThreads, keys), a.threshold, a.scale);
        } else {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) v.v[e] *= a.scale;
        }
        if (a.residual) {
            const Vf<kGroup> r = widen<S>(rr[j]);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) v.v[e] += r.v[e];
        }
        store_group<S, TAIL>((S*)a.y + base[j], col[j], a.C, v);
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
uint32_t drop_threshold(double p) {
    const double t = p * 65536.0 + 0.5;
    return t >= 65535.0 ? 65535u : (uint32_t)t;
}

static float keep_scale(double p) { return (float)(65536.0 / (65536.0 - (double)drop_threshold(p))); }

bool dwnorm_width_supported(int64_t C) { return C <= kNormMaxWidth; }

// A row of C columns held by LANES lanes of WAVES waves, NG groups each.
template <bool T, int L, int G, int W>
struct NormForm {
    static constexpr bool TAIL = T;
    static constexpr int LANES = L, NG = G, WAVES = W;
};

// Calls f with the narrowest form that holds a row of C: rows up to 512
// columns share a wave or fill it, wider ones take more groups per lane, and
// past 2048 columns a workgroup holds the row.
template <bool TAIL, typename F>
static hipError_t with_norm_form(int64_t C, F&& f) {
    if (C <= 64) return f(NormForm<TAIL, 8, 1, 1>());
    if (C <= 128) return f(NormForm<TAIL, 16, 1, 1>());
    if (C <= 256) return f(NormForm<TAIL, 32, 1, 1>());
    if (C <= 512) return f(NormForm<TAIL, 64, 1, 1>());
    if (C <= 1024) return f(NormForm<TAIL, 64, 2, 1>());
    if (C <= 2048) return f(NormForm<TAIL, 64, 4, 1>());
    if (C <= 4096) return f(NormForm<TAIL, 64, 2, 4>());
    return f(NormForm<TAIL, 64, 4, 4>());
}

template <typename F>
static hipError_t with_norm_form_any(int64_t C, F&& f) {
    return C % kGroup ? with_norm_form<true>(C, f) : with_norm_form<false>(C, f);
}

static int64_t norm_rows_per_block(int64_t C) {
    return C <= 64 ? 32 : C <= 128 ? 16 : C <= 256 ? 8 : C <= 2048 ? 4 : 1;
}

bool dwnorm_fwd_fits(int64_t rows, int64_t C) {
    const int64_t per = norm_rows_per_block(C);
    return grid_of_256_fits((rows + per - 1) / per);
}

hipError_t launch_dwnorm_fwd(const void* x, const void* residual, const void* gamma, const void* beta,
                             const int32_t* lengths, const uint64_t* rng, void* y, void* sum, float* mean,
                             float* rstd, int64_t B, int64_t T, int64_t C, float eps, float alpha, double p, bool bf16,
                             hipStream_t stream) {
    const NormFwd a = {x, residual, gamma, beta, lengths, rng, y, sum, mean, rstd, (uint32_t)(B * T), (uint32_t)T,
                       (int32_t)C, eps, alpha, keep_scale(p), drop_threshold(p)};
    const int64_t per = norm_rows_per_block(C);
    const dim3 grid((uint32_t)((B * T + per - 1) / per));
    return with_norm_form_any(C, [&](auto form) {
        using N = decltype(form);
        if (bf16)
            hipLaunchKernelGGL((norm_fwd_kernel<uint16_t, N::TAIL, N::LANES, N::NG, N::WAVES>), grid,
                               dim3(kNormThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((norm_fwd_kernel<float, N::TAIL, N::LANES, N::NG, N::WAVES>), grid, dim3(kNormThreads),
                               0, stream, a);
        return hipGetLastError();
    });
}

static int64_t norm_bwd_blocks(int64_t rows, int64_t C) {
    const int64_t per = norm_rows_per_block(C), blocks = (rows + per - 1) / per;
    return blocks < kNormBwdBlocks ? blocks : kNormBwdBlocks;
}

size_t dwnorm_bwd_workspace(int64_t B, int64_t T, int64_t C) {
    return (size_t)norm_bwd_blocks(B * T, C) * 2 * (size_t)C * sizeof(float);
}

hipError_t launch_dwnorm_bwd(const void* s, const void* gamma, const int32_t* lengths, const float* mean,
                             const float* rstd, const void* dy, const void* dsum, const uint64_t* rng, void* dx,
                             void* dres, float* dgamma, float* dbeta, void* workspace, int64_t B, int64_t T, int64_t C,
                             float alpha, double p, bool bf16, hipStream_t stream) {
    const bool params = dgamma || dbeta;
    const NormBwd a = {s, gamma, dy, dsum, lengths, mean, rstd, rng, dx, dres, params ? (float*)workspace : nullptr,
                       (uint32_t)(B * T), (uint32_t)T, (int32_t)C, alpha, keep_scale(p), drop_threshold(p)};
    const int64_t blocks = norm_bwd_blocks(B * T, C);
    if (blocks > 0) {
        const hipError_t e = with_norm_form_any(C, [&](auto form) {
            using N = decltype(form);
            if (bf16)
                hipLaunchKernelGGL((norm_bwd_kernel<uint16_t, N::TAIL, N::LANES, N::NG, N::WAVES>),
                                   dim3((uint32_t)blocks), dim3(kNormThreads), 0, stream, a);
            else
                hipLaunchKernelGGL((norm_bwd_kernel<float, N::TAIL, N::LANES, N::NG, N::WAVES>),
                                   dim3((uint32_t)blocks), dim3(kNormThreads), 0, stream, a);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (!params) return hipSuccess;
    hipLaunchKernelGGL(norm_param_reduce, dim3((uint32_t)((2 * C + kParamCols - 1) / kParamCols)),
                       dim3(kParamCols * kParamRows), 0, stream, (const float*)workspace, dgamma, dbeta, (int32_t)C,
                       (int32_t)blocks);
    return hipGetLastError();
}

static int64_t drop_blocks(int64_t rows, int64_t C) {
    const int64_t groups = rows * ((C + kGroup - 1) / kGroup), per = kDropThreads * kDropGroups;
    return (groups + per - 1) / per;
}

bool dwdrop_fits(int64_t rows, int64_t C) {
    return product_below((int64_t)1 << 60, {rows, C + kGroup}) && grid_of_256_fits(drop_blocks(rows, C));
}

hipError_t launch_dwdrop(const void* x, const void* residual, void* y, const uint64_t* rng, int64_t rows, int64_t C,
                         double p, float alpha, bool bf16, hipStream_t stream) {
    const int64_t per_row = (C + kGroup - 1) / kGroup;
    const bool tail = C % kGroup != 0;
    const Drop a = {x, residual, y, rng, (uint64_t)(rows * per_row), (uint32_t)per_row, tail ? (int32_t)C : kGroup,
                    alpha * keep_scale(p), drop_threshold(p)};
    const dim3 grid((uint32_t)drop_blocks(rows, C)), block(kDropThreads);
    if (bf16 && tail) hipLaunchKernelGGL((drop_kernel<uint16_t, true>), grid, block, 0, stream, a);
    if (bf16 && !tail) hipLaunchKernelGGL((drop_kernel<uint16_t, false>), grid, block, 0, stream, a);
    if (!bf16 && tail) hipLaunchKernelGGL((drop_kernel<float, true>), grid, block, 0, stream, a);
    if (!bf16 && !tail) hipLaunchKernelGGL((drop_kernel<float, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace dw
