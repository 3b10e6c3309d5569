// A gated linear recurrence over the frames of [B][T][C], channel by channel,
// and its backward pass.
//
//   w = scale * softplus(decay) * sigmoid(r),  a = exp(-w)
//   h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(g) x
//
// The state moves by d = 1 - a = -expm1(-w), taken without cancellation:
// h <- (h - d h) + u, u = sqrt(d (2 - d)) sigmoid(g) x, the bracket one fused
// operation.  A decay near 1 thus keeps its digits, as does one near 0, and
// products of decays are exponentials of sums of w.
//
// Frames in parallel: a run of frames maps the state h before it to P h + H
// behind it, and runs compose.  A thread takes 4 channels of FR frames, in
// registers; 4 threads along the frames share a wave and exchange (P, H) by
// lane swaps, the 4 waves of a workgroup through LDS, so that a workgroup moves
// through its frames in tiles of 16 * FR and memory sees each tensor once.
// Where items and channels make too few workgroups, the frames are shared out
// in chunks: a first kernel finds each chunk's (P, H), a second starts from
// what those before it leave.
#include "launch.h"
#include "rowops.h"
#include "quad.h"

namespace dw {

constexpr int kScanThreads = 256;
constexpr int kScanLanes = 16;                                // threads across the channels
constexpr int kScanRows = kScanThreads / kScanLanes;          // and along frames, or items
constexpr int kScanCols = kScanLanes * kQuad;                 // channels of a workgroup
constexpr int kScanFwdRun = 8, kScanBwdRun = 4;               // frames of a thread in a tile
constexpr int64_t kScanBlocks = 512;                          // workgroups that fill the GPU

struct ScanArgs {
    const void *x, *r, *g, *yin, *dy;
    const float* decay;
    const int32_t* lengths;
    const float* start;   // the state (backward: its gradient) that enters the first (last) frame, NULL: zero
    void *y, *dx, *dr, *dg;
    const float* h0;      // backward: the state before the first frame
    float *end, *copy;    // what leaves the last (first) frame; a copy of `start` beside the summaries
    float* summary;       // [2][B][chunks][C]: P, then H
    double* partial;      // backward: [row blocks][C], sums for ddecay
    FrameStride xs, rs, gs, ys, dys, dxs, drs, dgs;
    int64_t B, T, chunk;  // frames of a chunk, whole tiles
    int32_t C, col_blocks, chunks;
    float scale;
};

// What a phase of the work does: all frames of an item in one go; a chunk's
// (P, H) alone; a chunk from the state that the summaries before it give.
enum { kScanWhole = 0, kScanSummary = 1, kScanJoin = 2 };

struct Decay {
    float d, w;  // 1 - a, -log a
};

// 1 - exp(-w): a series where the difference would cancel (its first left out
// term is 2^-24.4 of it at w = 1/8), the exponential beyond (off by 2^-21 at most).
__device__ __forceinline__ float one_minus_exp(float w) {
    const float series = w * (1.0f + w * (-0.5f + w * (0.16666667f + w * (-0.041666668f + w * 0.0083333333f))));
    const float direct = 1.0f - __builtin_amdgcn_exp2f(w * -1.44269504f);
    return w < 0.125f ? series : direct;
}

__device__ __forceinline__ float softplus(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

// scale * softplus(decay), finite so that a closed gate is a decay of 1.
__device__ __forceinline__ float decay_rate(float decay, float scale) {
    const float k = scale * softplus(decay);
    return k > 1e30f ? 1e30f : k;
}

// sigmoid(v) / softplus(v), 1 in the limit where both underflow.
__device__ __forceinline__ float softplus_slope(float v) {
    return v < -16.0f ? 1.0f : 1.0f / ((1.0f + expf(-v)) * softplus(v));
}

struct Run {
    float p[kQuad], h[kQuad];  // state behind = p * state before + h
};

// The value of the wave's four rows of 16 lanes, in all lanes.
__device__ __forceinline__ void wave_rows(float v, float out[4]) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const auto e = __builtin_amdgcn_permlane32_swap(s[0], s[0], false, false);  // rows 0, 0, 2, 2
    const auto o = __builtin_amdgcn_permlane32_swap(s[1], s[1], false, false);  // rows 1, 1, 3, 3
    out[0] = __uint_as_float(e[0]);
    out[1] = __uint_as_float(o[0]);
    out[2] = __uint_as_float(e[1]);
    out[3] = __uint_as_float(o[1]);
}

// From the threads' runs of one tile, in their order along it (REVERSE: last
// first), and the state `carry` that enters the tile: the state that enters each
// thread's run, and in `carry` the one that leaves the tile.  `total`, if given,
// is composed with the tile's P.
template <int SEGS, bool REVERSE>
__device__ __forceinline__ void enter_runs(const Run& run, float carry[kQuad], float in[kQuad], float* total,
                                           float (*lds)[2][kScanCols]) {
    if constexpr (SEGS == 1) {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            in[e] = carry[e];
            carry[e] = run.h[e] + run.p[e] * carry[e];
            if (total) total[e] *= run.p[e];
        }
        return;
    }
    const int row = threadIdx.x / kScanLanes % 4;
    float p[kQuad][4], h[kQuad][4];
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        wave_rows(run.p[e], p[e]);
        wave_rows(run.h[e], h[e]);
    }
    if constexpr (SEGS > 4) {
        const int wave = threadIdx.x / 64, col = threadIdx.x % kScanLanes * kQuad;
        if (row == 0) {
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                float ph = p[e][0], hh = h[e][0];
                if constexpr (REVERSE) {
                    ph = p[e][3], hh = h[e][3];
#pragma unroll
                    for (int q = 2; q >= 0; --q) hh = h[e][q] + p[e][q] * hh, ph *= p[e][q];
                } else {
#pragma unroll
                    for (int q = 1; q < 4; ++q) hh = h[e][q] + p[e][q] * hh, ph *= p[e][q];
                }
                lds[wave][0][col + e] = ph;
                lds[wave][1][col + e] = hh;
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            float state = carry[e], mine = carry[e];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int at = REVERSE ? 3 - q : q;
                if (at == wave) mine = state;
                state = lds[at][1][col + e] + lds[at][0][col + e] * state;
                if (total) total[e] *= lds[at][0][col + e];
            }
            carry[e] = state;
            in[e] = mine;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) in[e] = carry[e];
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        float state = in[e], mine = in[e];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int at = REVERSE ? 3 - q : q;
            if (at == row) mine = state;
            state = h[e][at] + p[e][at] * state;
            if (SEGS <= 4 && total) total[e] *= p[e][at];
        }
        in[e] = mine;
        if constexpr (SEGS <= 4) carry[e] = state;
    }
}

// Where a thread works.
struct ScanPlace {
    int64_t b, first, last;  // item, frames [first, last) of its workgroup's chunk
    int64_t len;             // valid frames of the item
    int chunk, seg, col, have;
};

template <int SEGS, int PHASE>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a) {
    ScanPlace p;
    const int row = threadIdx.x / kScanLanes;
    const uint32_t rest = blockIdx.x / (uint32_t)a.col_blocks;
    p.col = (int)(blockIdx.x - rest * a.col_blocks) * kScanCols + threadIdx.x % kScanLanes * kQuad;
    p.have = a.C - p.col;
    if (p.have <= 0) p.col = 0;  // past the last channel: loads what is there, stores nothing
    p.seg = row % SEGS;
    if constexpr (PHASE == kScanWhole) {
        p.chunk = 0;
        p.b = (int64_t)rest * (kScanRows / SEGS);
        if constexpr (SEGS == 4) p.b += __builtin_amdgcn_readfirstlane(row / SEGS);  // one item a wave
        if constexpr (SEGS == 1) p.b += row;
        p.first = 0, p.last = a.T;
    } else {
        const uint32_t b = rest / (uint32_t)a.chunks;
        p.b = b;
        p.chunk = (int)(rest - b * a.chunks);
        p.first = p.chunk * a.chunk;
        p.last = p.first + a.chunk < a.T ? p.first + a.chunk : a.T;
    }
    p.len = p.b < a.B ? item_length(a.lengths, p.b, a.T) : 0;
    return p;
}

// One thread's FR frames of a tensor in the tile from frame t0 on; frames at or
// past the length (`valid` of the tile's are below it, at least one) read the
// last valid one and become `dead` (the bits of one stored value).
template <typename S, bool TAIL, int FR>
__device__ __forceinline__ void load_run(quad_raw<S> out[FR], const void* base, const FrameStride& s,
                                         const ScanPlace& p, int64_t t0, int valid, bool full, uint32_t dead) {
    const S* tile = (const S*)base + p.b * s.item + t0 * s.frame;
    const int at = p.seg * FR;
    const uint32_t fs = (uint32_t)s.frame;
    if (full) {
#pragma unroll
        for (int f = 0; f < FR; ++f) out[f] = load_quad<S, TAIL>(tile + (uint32_t)(f * fs) + (at * fs + p.col), p.have);
        return;
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int t = at + f < valid ? at + f : valid - 1;
        out[f] = load_quad<S, TAIL>(tile + ((uint32_t)t * fs + p.col), p.have);
        if (at + f >= valid) {
#pragma unroll
            for (int e = 0; e < (int)(sizeof(quad_raw<S>) / 4); ++e) out[f][e] = dead;
        }
    }
}

// The frame's values, zeros past the length; frames at or past `rows` are not
// the tile's.
template <typename S, bool TAIL, int FR>
__device__ __forceinline__ void store_frame(void* base, const FrameStride& s, const ScanPlace& p, int64_t t0, int f,
                                            int valid, int rows, const Vf<kQuad>& v) {
    const int t = p.seg * FR + f;
    if (t >= rows) return;
    S* tile = (S*)base + p.b * s.item + t0 * s.frame;
    store_quad<S, TAIL>(tile + ((uint32_t)t * (uint32_t)s.frame + p.col), p.have, t < valid ? v : vzero<kQuad>());
}

template <typename S>
constexpr uint32_t closed_gate() {  // -infinity, in each stored value
    return sizeof(S) == 4 ? 0xff800000u : 0xff80ff80u;
}

__device__ __forceinline__ Vf<kQuad> load_state(const float* base, int64_t row, int32_t C, const ScanPlace& p) {
    return base ? widen_quad<float>(load_quad<float, true>(base + row * C + p.col, p.have)) : vzero<kQuad>();
}

template <typename S, bool TAIL, int SEGS, int FR, int PHASE>
__global__ __launch_bounds__(kScanThreads) void scan_fwd_kernel(const ScanArgs a) {
    constexpr int kTileFrames = SEGS * FR;
    __shared__ float lds[2][4][2][kScanCols];
    const ScanPlace p = scan_place<SEGS, PHASE>(a);
    if (p.b >= a.B) return;  // SEGS < 16, where no thread waits for another wave
    float rate[kQuad], carry[kQuad], total[kQuad];
    {
        const Vf<kQuad> decay = load_state(a.decay, 0, a.C, p), h0 = load_state(a.start, p.b, a.C, p);
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            rate[e] = decay_rate(decay.v[e], a.scale);
            carry[e] = PHASE == kScanSummary ? 0.0f : h0.v[e];
            total[e] = 1.0f;
        }
        if (PHASE == kScanSummary && p.chunk == 0 && p.seg == 0 && p.have > 0)
            store_quad<float, true>(a.copy + p.b * a.C + p.col, p.have, h0);
    }
    const int64_t plane = a.B * a.chunks * (int64_t)a.C;
    if constexpr (PHASE == kScanJoin) {
        for (int c = 0; c < p.chunk; ++c) {
            const Vf<kQuad> P = load_state(a.summary, p.b * a.chunks + c, a.C, p);
            const Vf<kQuad> H = load_state(a.summary + plane, p.b * a.chunks + c, a.C, p);
#pragma unroll
            for (int e = 0; e < kQuad; ++e) carry[e] = H.v[e] + P.v[e] * carry[e];
        }
    }
    int turn = 0;
    for (int64_t t0 = p.first; t0 < p.last; t0 += kTileFrames) {
        const int64_t left = p.len - t0, size = p.last - t0;
        const int rows = size < kTileFrames ? (int)size : kTileFrames;
        const int valid = left < 0 ? 0 : left < rows ? (int)left : rows;
        Vf<kQuad> y[FR] = {};
        if (valid > 0) {
            quad_raw<S> xr[FR], rr[FR], gr[FR];
            const bool full = valid == kTileFrames;
            load_run<S, TAIL, FR>(rr, a.r, a.rs, p, t0, valid, full, closed_gate<S>());
            load_run<S, TAIL, FR>(xr, a.x, a.xs, p, t0, valid, full, 0);
            load_run<S, TAIL, FR>(gr, a.g, a.gs, p, t0, valid, full, 0);
            float d[FR][kQuad], u[FR][kQuad];
            Run run;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                float w = 0.0f, h = 0.0f;
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    const float wf = rate[e] * sigmoid_of<S>(quad_at<S>(rr[f], e));
                    const float df = one_minus_exp(wf);
                    const float m = __builtin_amdgcn_sqrtf(df * (2.0f - df));
                    d[f][e] = df;
                    u[f][e] = m * (sigmoid_of<S>(quad_at<S>(gr[f], e)) * quad_at<S>(xr[f], e));
                    w += wf;
                    h = __builtin_fmaf(-df, h, h) + u[f][e];
                }
                run.p[e] = __builtin_amdgcn_exp2f(w * -1.44269504f);
                run.h[e] = h;
            }
            float in[kQuad];
            enter_runs<SEGS, false>(run, carry, in, PHASE == kScanSummary ? total : nullptr, lds[turn]);
            turn ^= 1;
            if constexpr (PHASE != kScanSummary) {
#pragma unroll
                for (int e = 0; e < kQuad; ++e) {
                    float h = in[e];
#pragma unroll
                    for (int f = 0; f < FR; ++f) y[f].v[e] = h = __builtin_fmaf(-d[f][e], h, h) + u[f][e];
                }
            }
        }
        if constexpr (PHASE != kScanSummary) {
            if (p.have > 0) {
#pragma unroll
                for (int f = 0; f < FR; ++f) store_frame<S, TAIL, FR>(a.y, a.ys, p, t0, f, valid, rows, y[f]);
            }
        }
    }
    if (p.seg != 0 || p.have <= 0) return;
    Vf<kQuad> end, P;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) end.v[e] = carry[e], P.v[e] = total[e];
    if constexpr (PHASE == kScanSummary) {
        const int64_t at = (p.b * a.chunks + p.chunk) * a.C + p.col;
        store_quad<float, true>(a.summary + at, p.have, P);
        store_quad<float, true>(a.summary + plane + at, p.have, end);
    } else if (a.end && p.last == a.T) {
        store_quad<float, true>(a.end + p.b * a.C + p.col, p.have, end);
    }
}

// Backwards in time, G_t = dy_t + a_{t+1} G_{t+1}: the runs hand a_t G_t on to
// the frames before them.
template <typename S, bool TAIL, int SEGS, int FR, int PHASE>
__global__ __launch_bounds__(kScanThreads) void scan_bwd_kernel(const ScanArgs a) {
    constexpr int kTileFrames = SEGS * FR;
    __shared__ float lds[2][4][2][kScanCols];
    __shared__ float column[kScanRows][kScanCols];
    const ScanPlace p = scan_place<SEGS, PHASE>(a);
    const bool item = p.b < a.B;
    float rate[kQuad], carry[kQuad], total[kQuad], sum[kQuad];
    const Vf<kQuad> decay = load_state(a.decay, 0, a.C, p);
    const Vf<kQuad> start = item ? load_state(a.start, p.b, a.C, p) : vzero<kQuad>();
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        rate[e] = decay_rate(decay.v[e], a.scale);
        carry[e] = PHASE == kScanSummary ? 0.0f : start.v[e];
        total[e] = 1.0f;
        sum[e] = 0.0f;
    }
    if (PHASE == kScanSummary && p.chunk == 0 && p.seg == 0 && p.have > 0)
        store_quad<float, true>(a.copy + p.b * a.C + p.col, p.have, start);
    const int64_t plane = a.B * a.chunks * (int64_t)a.C;
    if constexpr (PHASE == kScanJoin) {
        for (int c = a.chunks - 1; c > p.chunk; --c) {
            const Vf<kQuad> P = load_state(a.summary, p.b * a.chunks + c, a.C, p);
            const Vf<kQuad> H = load_state(a.summary + plane, p.b * a.chunks + c, a.C, p);
#pragma unroll
            for (int e = 0; e < kQuad; ++e) carry[e] = H.v[e] + P.v[e] * carry[e];
        }
    }
    int turn = 0;
    const int64_t tiles = item ? (p.last - p.first + kTileFrames - 1) / kTileFrames : 0;
    for (int64_t i = tiles - 1; i >= 0; --i) {
        const int64_t t0 = p.first + i * kTileFrames;
        const int64_t left = p.len - t0, size = p.last - t0;
        const int rows = size < kTileFrames ? (int)size : kTileFrames;
        const int valid = left < 0 ? 0 : left < rows ? (int)left : rows;
        Vf<kQuad> dx[FR] = {}, dr[FR] = {}, dg[FR] = {};
        if (valid > 0) {
            quad_raw<S> rr[FR], dyr[FR], xr[FR], gr[FR];
            Vf<kQuad> before[FR];
            const bool full = valid == kTileFrames;
            load_run<S, TAIL, FR>(rr, a.r, a.rs, p, t0, valid, full, closed_gate<S>());
            load_run<S, TAIL, FR>(dyr, a.dy, a.dys, p, t0, valid, full, 0);
            if constexpr (PHASE != kScanSummary) {
                load_run<S, TAIL, FR>(xr, a.x, a.xs, p, t0, valid, full, 0);
                load_run<S, TAIL, FR>(gr, a.g, a.gs, p, t0, valid, full, 0);
                // the state before each frame: what the forward stored for the one in front of it
                const S* y = (const S*)a.yin + p.b * a.ys.item + t0 * a.ys.frame;
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    const int t = p.seg * FR + f;
                    if (f == 0 && p.seg == 0 && t0 == 0) {
                        before[f] = load_state(a.h0, p.b, a.C, p);
                    } else {
                        const int at = (t < valid ? t : valid) - 1;  // -1: the tile before
                        before[f] = widen_quad<S>(load_quad<S, TAIL>(y + (at * (int64_t)a.ys.frame + p.col), p.have));
                    }
                }
            }
            float d[FR][kQuad], w[FR][kQuad];
            Run run;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                float sw = 0.0f, c = 0.0f;
#pragma unroll
                for (int f = FR - 1; f >= 0; --f) {
                    const float wf = rate[e] * sigmoid_of<S>(quad_at<S>(rr[f], e));
                    const float df = one_minus_exp(wf);
                    w[f][e] = wf;
                    d[f][e] = df;
                    const float G = quad_at<S>(dyr[f], e) + c;
                    c = __builtin_fmaf(-df, G, G);
                    sw += wf;
                }
                run.p[e] = __builtin_amdgcn_exp2f(sw * -1.44269504f);
                run.h[e] = c;
            }
            float in[kQuad];
            enter_runs<SEGS, true>(run, carry, in, PHASE == kScanSummary ? total : nullptr, lds[turn]);
            turn ^= 1;
            if constexpr (PHASE != kScanSummary) {
#pragma unroll
                for (int e = 0; e < kQuad; ++e) {
                    float c = in[e];
#pragma unroll
                    for (int f = FR - 1; f >= 0; --f) {
                        const float G = quad_at<S>(dyr[f], e) + c;
                        const float x = quad_at<S>(xr[f], e), s = sigmoid_of<S>(quad_at<S>(rr[f], e));
                        const float gate = sigmoid_of<S>(quad_at<S>(gr[f], e));
                        const float z = d[f][e] * (2.0f - d[f][e]);                       // 1 - a^2 = m^2
                        const float rs = __builtin_amdgcn_rsqf(z > 1e-37f ? z : 1e-37f);  // w / m is 0 where w is
                        const float ix = gate * x;
                        const float open = G * (z * rs);
                        const float q = G * w[f][e] * (ix * (1.0f - z) * rs - before[f].v[e] * (1.0f - d[f][e]));
                        c = __builtin_fmaf(-d[f][e], G, G);
                        dx[f].v[e] = open * gate;
                        dg[f].v[e] = open * ix * (1.0f - gate);
                        dr[f].v[e] = q * (1.0f - s);
                        sum[e] += p.seg * FR + f < valid ? q : 0.0f;
                    }
                }
            }
        }
        if constexpr (PHASE != kScanSummary) {
            if (p.have > 0) {
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    if (a.dx) store_frame<S, TAIL, FR>(a.dx, a.dxs, p, t0, f, valid, rows, dx[f]);
                    if (a.dr) store_frame<S, TAIL, FR>(a.dr, a.drs, p, t0, f, valid, rows, dr[f]);
                    if (a.dg) store_frame<S, TAIL, FR>(a.dg, a.dgs, p, t0, f, valid, rows, dg[f]);
                }
            }
        }
    }
    if (item && p.seg == 0 && p.have > 0) {
        Vf<kQuad> end, P;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) end.v[e] = carry[e], P.v[e] = total[e];
        if constexpr (PHASE == kScanSummary) {
            const int64_t at = (p.b * a.chunks + p.chunk) * a.C + p.col;
            store_quad<float, true>(a.summary + at, p.have, P);
            store_quad<float, true>(a.summary + plane + at, p.have, end);
        } else if (a.end && p.first == 0) {
            store_quad<float, true>(a.end + p.b * a.C + p.col, p.have, end);
        }
    }
    if constexpr (PHASE != kScanSummary) {
        if (!a.partial) return;
        const int row = threadIdx.x / kScanLanes, lane = threadIdx.x % kScanLanes;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) column[row][lane * kQuad + e] = sum[e];
        __syncthreads();
        if (row != 0) return;
        double* out = a.partial + (int64_t)(blockIdx.x / (uint32_t)a.col_blocks) * a.C + p.col;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            double t = 0.0;
            for (int q = 0; q < kScanRows; ++q) t += column[q][lane * kQuad + e];
            if (e < p.have) out[e] = t * softplus_slope(decay.v[e]);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
// segs: threads along the frames of an item in a workgroup; run: frames of each
// in a tile.  chunks > 1: the frames are shared out.
struct ScanPlan {
    int segs, run;
    int64_t chunks, chunk, row_blocks, col_blocks;
};

static ScanPlan scan_plan(const ScanShape& s, int run) {
    ScanPlan p = {};
    p.run = s.T == 1 ? 1 : run;
    p.segs = s.T <= run ? 1 : s.T <= 4 * run ? 4 : 16;
    p.col_blocks = (s.C + kScanCols - 1) / kScanCols;
    p.chunks = 1;
    p.chunk = s.T;
    const int64_t tile = 16 * run, tiles = (s.T + tile - 1) / tile, per = kScanRows / p.segs;
    p.row_blocks = (s.B + per - 1) / per;
    const int64_t blocks = p.row_blocks * p.col_blocks;
    if (p.segs == 16 && blocks > 0 && blocks * 2 <= kScanBlocks && tiles >= 4) {
        const int64_t most = tiles / 2, want = kScanBlocks / blocks;
        const int64_t each = (tiles + (want < most ? want : most) - 1) / (want < most ? want : most);
        p.chunk = each * tile;
        p.chunks = (tiles + each - 1) / each;
        p.row_blocks *= p.chunks;
    }
    return p;
}

bool dwscan_fits(const ScanShape& s) {
    if (!product_below((int64_t)1 << 58, {s.B, s.T, s.C})) return false;
    for (const int run : {kScanFwdRun, kScanBwdRun}) {
        const ScanPlan p = scan_plan(s, run);
        if (!product_below((int64_t)1 << 24, {p.row_blocks, p.col_blocks})) return false;
    }
    return true;
}

static size_t scan_join_bytes(const ScanShape& s, const ScanPlan& p) {
    if (p.chunks == 1) return 0;
    const size_t bytes = (size_t)(s.B * (2 * p.chunks + 1) * s.C) * sizeof(float);
    return (bytes + 15) / 16 * 16;
}

static int64_t scan_partial_rows(const ScanPlan& p) {
    const int64_t chunks = partial_reduce_chunks(p.row_blocks);
    return p.row_blocks + (chunks > 1 ? chunks : 1);
}

size_t dwscan_fwd_workspace(const ScanShape& s) { return scan_join_bytes(s, scan_plan(s, kScanFwdRun)); }

size_t dwscan_bwd_workspace(const ScanShape& s) {
    const ScanPlan p = scan_plan(s, kScanBwdRun);
    return scan_join_bytes(s, p) + (size_t)(scan_partial_rows(p) * s.C) * sizeof(double);
}

static ScanArgs scan_args(const ScanPtrs& p, const ScanShape& s, const ScanPlan& plan, void* workspace) {
    ScanArgs a = {};
    a.x = p.x, a.r = p.r, a.g = p.g, a.decay = p.decay, a.lengths = p.lengths;
    a.xs = s.x, a.rs = s.r, a.gs = s.g, a.ys = s.y;
    a.dys = s.dy, a.dxs = s.dx, a.drs = s.dr, a.dgs = s.dg;
    a.B = s.B, a.T = s.T, a.C = (int32_t)s.C, a.scale = s.scale;
    a.chunk = plan.chunk, a.chunks = (int32_t)plan.chunks, a.col_blocks = (int32_t)plan.col_blocks;
    if (plan.chunks > 1) {
        a.summary = (float*)workspace;
        a.copy = a.summary + 2 * s.B * plan.chunks * s.C;
    }
    return a;
}

template <bool BACK, typename S, bool TAIL, int SEGS, int FR, int PHASE>
static hipError_t launch_scan_phase(const ScanArgs& a, dim3 grid, hipStream_t stream) {
    if constexpr (BACK)
        hipLaunchKernelGGL((scan_bwd_kernel<S, TAIL, SEGS, FR, PHASE>), grid, dim3(kScanThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((scan_fwd_kernel<S, TAIL, SEGS, FR, PHASE>), grid, dim3(kScanThreads), 0, stream, a);
    return hipGetLastError();
}

template <bool BACK, typename S, bool TAIL>
static hipError_t launch_scan_form(const ScanPlan& plan, ScanArgs a, hipStream_t stream) {
    constexpr int kRun = BACK ? kScanBwdRun : kScanFwdRun;
    const dim3 grid((uint32_t)(plan.row_blocks * plan.col_blocks));
    if (plan.chunks > 1) {
        const hipError_t e = launch_scan_phase<BACK, S, TAIL, 16, kRun, kScanSummary>(a, grid, stream);
        if (e != hipSuccess) return e;
        a.start = a.copy;  // what leaves may be written over what entered
        return launch_scan_phase<BACK, S, TAIL, 16, kRun, kScanJoin>(a, grid, stream);
    }
    if (plan.run == 1) return launch_scan_phase<BACK, S, TAIL, 1, 1, kScanWhole>(a, grid, stream);
    if (plan.segs == 1) return launch_scan_phase<BACK, S, TAIL, 1, kRun, kScanWhole>(a, grid, stream);
    if (plan.segs == 4) return launch_scan_phase<BACK, S, TAIL, 4, kRun, kScanWhole>(a, grid, stream);
    return launch_scan_phase<BACK, S, TAIL, 16, kRun, kScanWhole>(a, grid, stream);
}

template <bool BACK>
static hipError_t launch_scan(const ScanPlan& plan, const ScanArgs& a, bool bf16, hipStream_t stream) {
    const bool tail = a.C % kQuad != 0;
    if (bf16 && tail) return launch_scan_form<BACK, uint16_t, true>(plan, a, stream);
    if (bf16) return launch_scan_form<BACK, uint16_t, false>(plan, a, stream);
    if (tail) return launch_scan_form<BACK, float, true>(plan, a, stream);
    return launch_scan_form<BACK, float, false>(plan, a, stream);
}

hipError_t launch_dwscan_fwd(const ScanPtrs& p, const ScanShape& s, void* y, float* h_last, void* workspace, bool bf16,
                             hipStream_t stream) {
    const ScanPlan plan = scan_plan(s, kScanFwdRun);
    ScanArgs a = scan_args(p, s, plan, workspace);
    a.start = p.h0, a.y = y, a.end = h_last;
    return launch_scan<false>(plan, a, bf16, stream);
}

hipError_t launch_dwscan_bwd(const ScanPtrs& p, const ScanShape& s, const void* y, const void* dy, const float* dh_last,
                             void* dx, void* dr, void* dg, float* ddecay, float* dh0, void* workspace, bool bf16,
                             hipStream_t stream) {
    const ScanPlan plan = scan_plan(s, kScanBwdRun);
    ScanArgs a = scan_args(p, s, plan, workspace);
    a.start = dh_last, a.h0 = p.h0, a.yin = y, a.dy = dy, a.dx = dx, a.dr = dr, a.dg = dg, a.end = dh0;
    double* rows = (double*)((char*)workspace + scan_join_bytes(s, plan));
    a.partial = ddecay ? rows : nullptr;
    if (plan.row_blocks > 0) {
        const hipError_t e = launch_scan<true>(plan, a, bf16, stream);
        if (e != hipSuccess) return e;
    }
    if (!ddecay) return hipSuccess;
    RowOutputs out = {};
    out.n = 1;
    out.p[0] = ddecay, out.first[0] = 0, out.count[0] = 1;
    return launch_partial_reduce(rows, plan.row_blocks, 1, s.C, rows + plan.row_blocks * s.C, out, stream);
}

}  // namespace dw
