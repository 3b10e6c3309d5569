// Root mean square norm of each head of queries and keys with a weight for each
// element, and the rotation of its element pairs by the frame's position, in
// one pass; the same for the gradients.
//
//   n = x * rsqrt(mean(x^2) + eps) * gamma;  (n_i, n_j) turned by f = position * freq
//
// A head of D elements is ceil(D/2) pairs: the rotated ones in their order, then
// the rest two by two.  A lane holds 4 pairs, so a rotation never leaves its
// lane, and 4, 8 or 16 neighbouring lanes (a team) hold a head.  A team takes
// heads of one frame, whose cosines and sines it forms once: the angle in
// turns, reduced in 64 bits, then a float polynomial on [-1, 1].
//
// Bound by memory.  12000 frames of 8 + 8 heads of 128 in bf16: forward 86.8 MB in
// 18.6 us (4.7 TB/s; a large copy reaches 5.1), about 19 vector operations an element,
// which take 9 us of issue slots; gradients 124.5 MB in 29 us and 4 us for the
// sum of the gammas' partial rows, 32 together.  Two heads of both tensors in
// flight (134 registers, three waves a SIMD, so all workgroups at once); with four
// 40 us, with one 33, with the next two read ahead 33.  One frame of 64 items
// takes 11.5 us, which is the host's call and launch: the kernel is 6, a chain of
// loads, the angle's 64-bit reduction and two sums across a team.
#include "launch.h"
#include "rowops.h"
#include "quad.h"

namespace dw {

constexpr int kRopeThreads = 256;
constexpr int kRopeFly = 4;                 // heads whose loads are in flight together
// Workgroups (and partial rows) of the backward at most.  8 + 8 heads of 128 in bf16, us
// with at most 768, 1024 and 2048: 12000 frames 34.3, 34.2, 34.4, 16000 44.1, 48.7, 48.8,
// 22000 55.0, 55.0, 58.7, 32000 84.1, 91.2, 84.9: 768 are in flight together, and 769 to
// 1024 in one turn run a round and a rest.
constexpr int64_t kRopeBwdBlocks = 1024;

struct RopeStride {
    int64_t item, frame, head;
};

struct RopeArgs {
    const void *q, *k, *v, *q_gamma, *k_gamma, *dq_out, *dk_out;
    const double* freq;
    const int32_t *lengths, *pos, *place;
    void *q_out, *k_out, *v_out;  // backward: dq, dk
    float* partial;               // backward: [gridDim.x][2][D], NULL: not wanted
    RopeStride qs, ks, vs, qos, kos, vos, dqs, dks;
    int64_t S;
    uint64_t frames;  // B * T
    uint32_t T, split;
    int32_t H, Hkv, D, R;
    float eps;
};

// How a lane's 4 pairs lie in a head.  kWhole and kTail: each of its two quads is 4
// neighbouring elements, so vector accesses serve it: halves, the pairs' firsts
// and their seconds (a lane that is not rotated pairs the two quads of its 8
// elements in a row); neighbours, 8 elements in a row.  kTail: the head may end
// inside a quad (gradients of [9,1197,32+8 heads of 50] bf16, neighbours, 59 us;
// 144 element by element).  kLoose: each element has a place of its own, D standing
// for none (heads of 50 turned whole, halves: 177 us; [16,750,8+8 heads of 44] 38 and 68).
constexpr int kLoose = 0, kWhole = 1, kTail = 2;

template <int PACKED, bool HALVES>
struct PairMap {
    int at[2][kQuad];
    int first;  // the lane's first pair

    __device__ __forceinline__ PairMap(int lane, int D, int R) {
        first = lane * kQuad;
        const bool apart = HALVES && first < R / 2;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            const int p = first + e;
            if constexpr (PACKED != kLoose && HALVES) {
                at[0][e] = apart ? p : 2 * first + e;
                at[1][e] = apart ? p + R / 2 : 2 * first + kQuad + e;
            } else {
                const bool halves = HALVES && p < R / 2;
                at[0][e] = halves ? p : 2 * p;
                at[1][e] = halves ? p + R / 2 : 2 * p + 1;
            }
            at[0][e] = min(D, at[0][e]);
            at[1][e] = min(D, at[1][e]);
        }
    }

    // not kLoose: the first elements of the two quads as they lie in memory
    __device__ __forceinline__ int quad(int h) const { return HALVES ? at[h][0] : 2 * first + h * kQuad; }
};

template <typename S>
struct HeadRaw {
    quad_raw<S> q[2];
};

struct Head {
    f32x4 a, b;  // the pairs' first and second elements
};

// A head from its first element on; `on` is false for a head past the last.
template <typename S, int PACKED, bool HALVES>
__device__ __forceinline__ HeadRaw<S> load_head(const S* head, const PairMap<PACKED, HALVES>& m, int D, bool on) {
    HeadRaw<S> r = {};
    if constexpr (PACKED != kLoose) {
        if (on && 2 * m.first < D) {
            r.q[0] = load_quad<S, PACKED == kTail>(head + m.quad(0), D - m.quad(0));
            r.q[1] = load_quad<S, PACKED == kTail>(head + m.quad(1), D - m.quad(1));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                if (on && m.at[h][e] < D) {
                    if constexpr (sizeof(S) == 4)
                        r.q[h][e] = __float_as_uint(head[m.at[h][e]]);
                    else
                        r.q[h][e / 2] |= (uint32_t)head[m.at[h][e]] << (16 * (e & 1));
                }
            }
        }
    }
    return r;
}

template <typename S, int PACKED, bool HALVES>
__device__ __forceinline__ Head widen_head(const HeadRaw<S>& r, const PairMap<PACKED, HALVES>& m) {
    const Vf<kQuad> xv = widen_quad<S>(r.q[0]), yv = widen_quad<S>(r.q[1]);
    const f32x4 x = {xv.v[0], xv.v[1], xv.v[2], xv.v[3]}, y = {yv.v[0], yv.v[1], yv.v[2], yv.v[3]};
    if constexpr (PACKED != kLoose && !HALVES) return {{x[0], x[2], y[0], y[2]}, {x[1], x[3], y[1], y[3]}};
    return {x, y};
}

template <typename S, int PACKED, bool HALVES>
__device__ __forceinline__ void store_head(S* head, const PairMap<PACKED, HALVES>& m, int D, Head h) {
    if constexpr (PACKED != kLoose) {
        if (2 * m.first >= D) return;
        Vf<kQuad> x = {{h.a[0], h.a[1], h.a[2], h.a[3]}}, y = {{h.b[0], h.b[1], h.b[2], h.b[3]}};
        if constexpr (!HALVES) {
            x = {{h.a[0], h.b[0], h.a[1], h.b[1]}};
            y = {{h.a[2], h.b[2], h.a[3], h.b[3]}};
        }
        store_quad<S, PACKED == kTail>(head + m.quad(0), D - m.quad(0), x);
        store_quad<S, PACKED == kTail>(head + m.quad(1), D - m.quad(1), y);
    } else {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            if constexpr (sizeof(S) == 4) {
                if (m.at[0][e] < D) head[m.at[0][e]] = h.a[e];
                if (m.at[1][e] < D) head[m.at[1][e]] = h.b[e];
            } else {
                const uint32_t pair = pack_bf16x2(h.a[e], h.b[e]);
                if (m.at[0][e] < D) head[m.at[0][e]] = (uint16_t)pair;
                if (m.at[1][e] < D) head[m.at[1][e]] = (uint16_t)(pair >> 16);
            }
        }
    }
}

// The weights of the lane's elements; ones where there is no gamma, 0 past the head.
template <typename S, int PACKED, bool HALVES>
__device__ __forceinline__ Head load_gamma(const void* gamma, const PairMap<PACKED, HALVES>& m, int D) {
    if (gamma) return widen_head<S>(load_head<S>((const S*)gamma, m, D, true), m);
    return {f32x4(1.0f), f32x4(1.0f)};
}

struct Turns {
    float c[kQuad], s[kQuad];
};

// cos and sin of position * freq for the lane's 4 pairs; 1 and 0 for those that
// are not rotated.  In half turns the product is off by a few 2^-53 of itself,
// and what is left of it after the whole turns is exact in float to 2^-24 of a
// half turn.
__device__ __forceinline__ Turns turns_of(const double* freq, int64_t position, int first, int R) {
    Turns t;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        t.c[e] = 1.0f;
        t.s[e] = 0.0f;
        if (first + e < R / 2) {
            const double half = (double)position * freq[first + e] * 0.31830988618379067154;  // 1 / pi
            sincospif((float)(half - 2.0 * rint(0.5 * half)), &t.s[e], &t.c[e]);
        }
    }
    return t;
}

// The team's frame and its share of the heads.
struct RopeTeam {
    int64_t b, t, position;
    bool live;
};

__device__ __forceinline__ RopeTeam rope_frame(const RopeArgs& a, uint64_t frame) {
    RopeTeam f;
    f.b = (int64_t)(frame >> 32 ? frame / a.T : (uint32_t)frame / a.T);
    f.t = (int64_t)(frame - (uint64_t)f.b * a.T);
    f.live = !a.lengths || f.t < a.lengths[f.b];
    f.position = f.t + (a.pos ? a.pos[f.b] : 0);
    return f;
}

// Zeros for the heads of a frame past its length.
template <typename S, int PACKED, bool HALVES>
__device__ __forceinline__ void zero_heads(S* out, int64_t os, int32_t heads, uint32_t from, uint32_t step,
                                           const PairMap<PACKED, HALVES>& m, int D) {
    for (uint32_t h = from; h < (uint32_t)heads; h += step) store_head<S>(out + (int64_t)h * os, m, D, Head{});
}

// x: the heads of one frame; out: where they go.
template <typename S, int PACKED, bool HALVES, int LANES>
__device__ __forceinline__ void rope_heads(const S* x, int64_t xs, S* out, int64_t os, int32_t heads, uint32_t from,
                                           uint32_t step, const PairMap<PACKED, HALVES>& m, Head gamma,
                                           const Turns& turn, int D, float eps) {
    const float inv_d = 1.0f / (float)D;
    const int64_t x_step = step * xs, o_step = step * os;  // one head of the team's to the next
    x += from * xs;
    out += from * os;
    for (uint32_t h0 = from; h0 < (uint32_t)heads; h0 += kRopeFly * step, x += kRopeFly * x_step, out += kRopeFly * o_step) {
        HeadRaw<S> raw[kRopeFly];
#pragma unroll
        for (int j = 0; j < kRopeFly; ++j)
            raw[j] = load_head<S>(x + j * x_step, m, D, h0 + j * step < (uint32_t)heads);
#pragma unroll
        for (int j = 0; j < kRopeFly; ++j) {
            const uint32_t h = h0 + j * step;
            Head v = widen_head<S>(raw[j], m);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) sum += v.a[e] * v.a[e] + v.b[e] * v.b[e];
            const float rstd = __builtin_amdgcn_rsqf(lane_sum<LANES>(sum) * inv_d + eps);
            Head o;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                const float p = v.a[e] * rstd * gamma.a[e], q = v.b[e] * rstd * gamma.b[e];
                o.a[e] = p * turn.c[e] - q * turn.s[e];
                o.b[e] = q * turn.c[e] + p * turn.s[e];
            }
            if (h < (uint32_t)heads) store_head<S>(out + j * o_step, m, D, o);
        }
    }
}

template <typename S, int PACKED, bool HALVES, int LANES>
__global__ __launch_bounds__(kRopeThreads) void rope_fwd_kernel(const RopeArgs a) {
    constexpr int kTeams = kRopeThreads / LANES;
    const int lane = threadIdx.x % LANES, D = a.D;
    const uint64_t team = (uint64_t)blockIdx.x * kTeams + threadIdx.x / LANES;
    const uint64_t frame = team >> 32 ? team / a.split : (uint32_t)team / a.split;
    if (frame >= a.frames) return;
    const uint32_t part = (uint32_t)(team - frame * a.split);
    const RopeTeam f = rope_frame(a, frame);
    const PairMap<PACKED, HALVES> m(lane, D, a.R);
    const S* q = (const S*)a.q + f.b * a.qs.item + f.t * a.qs.frame;
    S* q_out = (S*)a.q_out + f.b * a.qos.item + f.t * a.qos.frame;
    // the first heads of k and v go to the teams behind those that hold the last of q
    const uint32_t from = (part + a.split - (uint32_t)a.H % a.split) % a.split;
    const uint32_t v_from = (from + a.split - (uint32_t)a.Hkv % a.split) % a.split;
    int64_t to = f.t;
    bool keys = a.Hkv > 0;
    if (a.place && keys) {  // a cache: only valid frames that fall into it
        to += a.place[f.b];
        keys = f.live && to >= 0 && to < a.S;
    }
    S* k_out = (S*)a.k_out + f.b * a.kos.item + to * a.kos.frame;
    S* v_out = (S*)a.v_out + f.b * a.vos.item + to * a.vos.frame;
    if (!f.live) {
        zero_heads<S>(q_out, a.qos.head, a.H, part, a.split, m, D);
        if (!keys) return;
        zero_heads<S>(k_out, a.kos.head, a.Hkv, from, a.split, m, D);
        if (a.v) zero_heads<S>(v_out, a.vos.head, a.Hkv, v_from, a.split, m, D);
        return;
    }
    const Turns turn = turns_of(a.freq, f.position, m.first, a.R);
    if (a.H > 0)
        rope_heads<S, PACKED, HALVES, LANES>(q, a.qs.head, q_out, a.qos.head, a.H, part, a.split, m,
                                             load_gamma<S>(a.q_gamma, m, D), turn, D, a.eps);
    if (!keys) return;
    rope_heads<S, PACKED, HALVES, LANES>((const S*)a.k + f.b * a.ks.item + f.t * a.ks.frame, a.ks.head, k_out,
                                         a.kos.head, a.Hkv, from, a.split, m, load_gamma<S>(a.k_gamma, m, D), turn, D,
                                         a.eps);
    if (!a.v) return;
    const S* v = (const S*)a.v + f.b * a.vs.item + f.t * a.vs.frame;
    for (uint32_t h = v_from; h < (uint32_t)a.Hkv; h += a.split)
        store_head<S>(v_out + (int64_t)h * a.vos.head, m, D,
                      widen_head<S>(load_head<S>(v + (int64_t)h * a.vs.head, m, D, true), m));
}

// Gradients of one frame's heads; dg takes the sums of u * xh.
template <typename S, int PACKED, bool HALVES, int LANES>
__device__ __forceinline__ void rope_grads(const S* x, int64_t xs, const S* dout, int64_t ds, S* dx, int64_t os,
                                           int32_t heads, uint32_t from, uint32_t step,
                                           const PairMap<PACKED, HALVES>& m, Head gamma, const Turns& turn,
                                           int D, float eps, Head& dg) {
    constexpr int kFly = kRopeFly / 2;  // two tensors each
    const float inv_d = 1.0f / (float)D;
    const int64_t x_step = step * xs, d_step = step * ds, o_step = step * os;
    x += from * xs;
    dout += from * ds;
    if (dx) dx += from * os;
    for (uint32_t h0 = from; h0 < (uint32_t)heads; h0 += kFly * step) {
        HeadRaw<S> xr[kFly], dr[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const uint32_t h = h0 + j * step;
            const bool on = h < (uint32_t)heads;
            xr[j] = load_head<S>(x + j * x_step, m, D, on);
            dr[j] = load_head<S>(dout + j * d_step, m, D, on);
        }
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const uint32_t h = h0 + j * step;
            Head v = widen_head<S>(xr[j], m), d = widen_head<S>(dr[j], m);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) sum += v.a[e] * v.a[e] + v.b[e] * v.b[e];
            // 0 where no head was loaded: with eps = 0 its zeros would have no norm
            const float mean = lane_sum<LANES>(sum) * inv_d;
            const float rstd = h < (uint32_t)heads ? __builtin_amdgcn_rsqf(mean + eps) : 0.0f;
            Head g;
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                const float p = d.a[e] * turn.c[e] + d.b[e] * turn.s[e];  // turned back
                const float q = d.b[e] * turn.c[e] - d.a[e] * turn.s[e];
                v.a[e] *= rstd;
                v.b[e] *= rstd;
                dg.a[e] += p * v.a[e];
                dg.b[e] += q * v.b[e];
                g.a[e] = p * gamma.a[e];
                g.b[e] = q * gamma.b[e];
                dot += g.a[e] * v.a[e] + g.b[e] * v.b[e];
            }
            dot = lane_sum<LANES>(dot) * inv_d;
#pragma unroll
            for (int e = 0; e < kQuad; ++e) {
                g.a[e] = rstd * (g.a[e] - v.a[e] * dot);
                g.b[e] = rstd * (g.b[e] - v.b[e] * dot);
            }
            if (dx && h < (uint32_t)heads) store_head<S>(dx + j * o_step, m, D, g);
        }
        x += kFly * x_step;
        dout += kFly * d_step;
        if (dx) dx += kFly * o_step;
    }
}

// Teams take frames (and parts of their heads) in turn and keep the gammas'
// gradients of their own elements in registers; a workgroup adds its teams in a
// fixed order and writes one partial row.
template <typename S, int PACKED, bool HALVES, int LANES>
__global__ __launch_bounds__(kRopeThreads) void rope_bwd_kernel(const RopeArgs a) {
    constexpr int kTeams = kRopeThreads / LANES, kWaves = kRopeThreads / 64;
    __shared__ float column[kWaves][2][2 * kQuad * LANES];
    const int lane = threadIdx.x % LANES, D = a.D;
    const PairMap<PACKED, HALVES> m(lane, D, a.R);
    const Head q_gamma = load_gamma<S>(a.q_gamma, m, D), k_gamma = load_gamma<S>(a.k_gamma, m, D);
    Head dg[2] = {};
    for (uint64_t team = (uint64_t)blockIdx.x * kTeams + threadIdx.x / LANES; team < a.frames * a.split;
         team += (uint64_t)gridDim.x * kTeams) {
        const uint64_t frame = team >> 32 ? team / a.split : (uint32_t)team / a.split;
        const uint32_t part = (uint32_t)(team - frame * a.split);
        const RopeTeam f = rope_frame(a, frame);
        const uint32_t from = (part + a.split - (uint32_t)a.H % a.split) % a.split;
        S* dq = a.q_out ? (S*)a.q_out + f.b * a.dqs.item + f.t * a.dqs.frame : nullptr;
        S* dk = a.k_out ? (S*)a.k_out + f.b * a.dks.item + f.t * a.dks.frame : nullptr;
        if (!f.live) {
            if (dq) zero_heads<S>(dq, a.dqs.head, a.H, part, a.split, m, D);
            if (dk) zero_heads<S>(dk, a.dks.head, a.Hkv, from, a.split, m, D);
            continue;
        }
        const Turns turn = turns_of(a.freq, f.position, m.first, a.R);
        if (a.H > 0)
            rope_grads<S, PACKED, HALVES, LANES>((const S*)a.q + f.b * a.qs.item + f.t * a.qs.frame, a.qs.head,
                                                 (const S*)a.dq_out + f.b * a.qos.item + f.t * a.qos.frame, a.qos.head,
                                                 dq, a.dqs.head, a.H, part, a.split, m, q_gamma, turn, D, a.eps, dg[0]);
        if (a.Hkv > 0)
            rope_grads<S, PACKED, HALVES, LANES>((const S*)a.k + f.b * a.ks.item + f.t * a.ks.frame, a.ks.head,
                                                 (const S*)a.dk_out + f.b * a.kos.item + f.t * a.kos.frame, a.kos.head,
                                                 dk, a.dks.head, a.Hkv, from, a.split, m, k_gamma, turn, D, a.eps, dg[1]);
    }
    if (!a.partial) return;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            float u = dg[n].a[e], w = dg[n].b[e];
#pragma unroll
            for (int x = LANES; x < 64; x *= 2) {  // the wave's other teams
                u += __shfl_xor(u, x);
                w += __shfl_xor(w, x);
            }
            if (threadIdx.x % 64 < LANES) {
                column[threadIdx.x / 64][n][lane * 2 * kQuad + e] = u;
                column[threadIdx.x / 64][n][lane * 2 * kQuad + kQuad + e] = w;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x >= 2 * LANES) return;
    const int n = threadIdx.x / LANES;
    float* out = a.partial + ((int64_t)blockIdx.x * 2 + n) * D;
    Head total = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
            total.a[e] += column[w][n][lane * 2 * kQuad + e];
            total.b[e] += column[w][n][lane * 2 * kQuad + kQuad + e];
        }
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        if (m.at[0][e] < D) out[m.at[0][e]] = total.a[e];
        if (m.at[1][e] < D) out[m.at[1][e]] = total.b[e];
    }
}

// Column sums of the [P][2][D] partials in fp64: 64 sub-rows x 16 columns a
// workgroup, sub-row q adding partials q, q + 64, ..., then the sub-rows in
// order, 16 at a time.
constexpr int kGammaCols = 16, kGammaRows = 64, kGammaParts = 4;

__global__ __launch_bounds__(kGammaCols* kGammaRows) void rope_gamma_reduce(const float* __restrict__ partial,
                                                                           float* __restrict__ dq_gamma,
                                                                           float* __restrict__ dk_gamma, int32_t D,
                                                                           int32_t P) {
    __shared__ double acc[kGammaRows][kGammaCols];
    const int lane = threadIdx.x % kGammaCols, sub = threadIdx.x / kGammaCols, ncol = 2 * D;
    const int col = blockIdx.x * kGammaCols + lane;
    double s = 0.0;
    if (col < ncol) {
#pragma unroll 8
        for (int32_t r = sub; r < P; r += kGammaRows) s += partial[(int64_t)r * ncol + col];
    }
    acc[sub][lane] = s;
    __syncthreads();
    constexpr int kEach = kGammaRows / kGammaParts;
    if (sub < kGammaParts) {
        s = 0.0;
#pragma unroll
        for (int q = 0; q < kEach; ++q) s += acc[sub * kEach + q][lane];
    }
    __syncthreads();
    if (sub < kGammaParts) acc[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= ncol) return;
#pragma unroll
    for (int q = 1; q < kGammaParts; ++q) s += acc[q][lane];
    float* out = col < D ? dq_gamma : dk_gamma;
    if (out) out[col < D ? col : col - D] = (float)s;
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static int rope_lanes(int64_t D) { return D <= 32 ? 4 : D <= 64 ? 8 : 16; }

// Teams that share a frame's heads: one where the frames alone fill the GPU
// (its cosines then serve all heads), else as many as there are heads.  8 + 8 heads of
// 128, 1 and 2 teams a frame, and this rule, us: bf16 4000 frames 11.3, 10.5 and 14.7,
// 8000 14.1, 13.9 and 15.9, 12000 18.4, 18.5 and 18.5 (float 16.5, 13.4 and 14.4, 28.8, 22.6 and
// 22.5, 43.3, 34.4 and 34.6), gradients 4000 20.3, 20.7 and 21.8, 8000 25.5, 27.9 and 28.1,
// 12000 34.3, 35.9 and 34.2 (750 workgroups are in flight together, 1500 are not).
// One team loses in float forward, several in bf16 at 4000 and 8000 frames.
static int64_t rope_split(const RopeShape& s, bool backward) {
    const int64_t heads = s.H > s.Hkv ? s.H : s.Hkv, lanes = s.B * s.T * rope_lanes(s.D);
    const int64_t enough = backward ? 128 * 1024 : 256 * 1024;
    int64_t n = 1;
    while (n < heads && n < 64 && lanes * n < enough) n *= 2;
    return n;
}

static int64_t rope_blocks(const RopeShape& s, bool backward) {
    const int64_t per = kRopeThreads / rope_lanes(s.D), teams = s.B * s.T * rope_split(s, backward);
    return (teams + per - 1) / per;
}

bool dwrope_fits(const RopeShape& s) {
    return product_below((int64_t)1 << 40, {s.B, s.T}) && grid_of_256_fits(rope_blocks(s, false));
}

template <int P, bool H, int L>
struct RopeForm {
    static constexpr bool HALVES = H;
    static constexpr int PACKED = P, LANES = L;
};

template <int P, bool H, typename F>
static hipError_t with_rope_lanes(int64_t D, F&& f) {
    if (D <= 32) return f(RopeForm<P, H, 4>());
    if (D <= 64) return f(RopeForm<P, H, 8>());
    return f(RopeForm<P, H, 16>());
}

// Quads of neighbouring elements serve a lane where its 4 pairs all are rotated
// or none is: always with neighbours, with halves where R is a multiple of 8.
template <typename F>
static hipError_t with_rope_form(const RopeShape& s, F&& f) {
    if (s.halves && s.R % 8 != 0) return with_rope_lanes<kLoose, true>(s.D, f);
    if (s.D % 8 == 0) return s.halves ? with_rope_lanes<kWhole, true>(s.D, f) : with_rope_lanes<kWhole, false>(s.D, f);
    return s.halves ? with_rope_lanes<kTail, true>(s.D, f) : with_rope_lanes<kTail, false>(s.D, f);
}

static RopeStride rope_stride(const AttnStride& s) { return {s.item, s.frame, s.head}; }

static RopeArgs rope_args(const RopePtrs& p, const RopeShape& s, bool backward) {
    RopeArgs a = {};
    a.q = p.q, a.k = p.k, a.q_gamma = p.q_gamma, a.k_gamma = p.k_gamma;
    a.freq = p.freq, a.lengths = p.lengths, a.pos = p.pos;
    a.qs = rope_stride(s.q), a.ks = rope_stride(s.k), a.vs = rope_stride(s.v);
    a.qos = rope_stride(s.q_out), a.kos = rope_stride(s.k_out), a.vos = rope_stride(s.v_out);
    a.dqs = rope_stride(s.dq), a.dks = rope_stride(s.dk);
    a.S = s.S, a.frames = (uint64_t)(s.B * s.T), a.T = (uint32_t)s.T, a.split = (uint32_t)rope_split(s, backward);
    a.H = (int32_t)s.H, a.Hkv = (int32_t)s.Hkv, a.D = (int32_t)s.D, a.R = (int32_t)s.R;
    a.eps = s.eps;
    return a;
}

hipError_t launch_dwrope_fwd(const RopePtrs& p, const RopeShape& s, const void* v, const int32_t* place, void* q_out,
                             void* k_out, void* v_out, bool bf16, hipStream_t stream) {
    RopeArgs a = rope_args(p, s, false);
    a.v = v, a.place = place, a.q_out = q_out, a.k_out = k_out, a.v_out = v_out;
    const dim3 grid((uint32_t)rope_blocks(s, false));
    return with_rope_form(s, [&](auto form) {
        using N = decltype(form);
        if (bf16)
            hipLaunchKernelGGL((rope_fwd_kernel<uint16_t, N::PACKED, N::HALVES, N::LANES>), grid, dim3(kRopeThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((rope_fwd_kernel<float, N::PACKED, N::HALVES, N::LANES>), grid, dim3(kRopeThreads), 0,
                               stream, a);
        return hipGetLastError();
    });
}

// As many as take equal turns.
static int64_t rope_bwd_blocks(const RopeShape& s) {
    const int64_t blocks = rope_blocks(s, true), turns = (blocks + kRopeBwdBlocks - 1) / kRopeBwdBlocks;
    return turns > 1 ? (blocks + turns - 1) / turns : blocks;
}

size_t dwrope_bwd_workspace(const RopeShape& s) {
    return (size_t)rope_bwd_blocks(s) * 2 * (size_t)s.D * sizeof(float);
}

hipError_t launch_dwrope_bwd(const RopePtrs& p, const RopeShape& s, const void* dq_out, const void* dk_out, void* dq,
                             void* dk, float* dq_gamma, float* dk_gamma, void* workspace, bool bf16,
                             hipStream_t stream) {
    RopeArgs a = rope_args(p, s, true);
    a.dq_out = dq_out, a.dk_out = dk_out, a.q_out = dq, a.k_out = dk;
    const bool params = dq_gamma || dk_gamma;
    a.partial = params ? (float*)workspace : nullptr;
    const int64_t blocks = rope_bwd_blocks(s);
    if (blocks > 0) {
        const hipError_t e = with_rope_form(s, [&](auto form) {
            using N = decltype(form);
            if (bf16)
                hipLaunchKernelGGL((rope_bwd_kernel<uint16_t, N::PACKED, N::HALVES, N::LANES>), dim3((uint32_t)blocks),
                                   dim3(kRopeThreads), 0, stream, a);
            else
                hipLaunchKernelGGL((rope_bwd_kernel<float, N::PACKED, N::HALVES, N::LANES>), dim3((uint32_t)blocks),
                                   dim3(kRopeThreads), 0, stream, a);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (!params) return hipSuccess;
    hipLaunchKernelGGL(rope_gamma_reduce, dim3((uint32_t)((2 * s.D + kGammaCols - 1) / kGammaCols)),
                       dim3(kGammaCols * kGammaRows), 0, stream, (const float*)workspace, dq_gamma, dk_gamma,
                       (int32_t)s.D, (int32_t)blocks);
    return hipGetLastError();
}

}  // namespace dw
