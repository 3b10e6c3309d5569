// Self-attention with a learned relative position bias by buckets: forward.
//
//   S_ij = scale * q_i . k_j + bias[j - i - pos],  out_i = sum_j softmax_j(S_ij) v_j
//
// One pass over the keys with the running maximum and sum of a softmax.  A
// workgroup of four waves owns 32 * QW queries of one head: with QW = 4 each
// wave owns 32 queries and all share the tiles of 64 keys; with QW = 1 (few
// queries: streaming, short utterances) the waves share 32 queries and divide
// tiles of 128 keys, and their results are joined in LDS.  Where even that
// leaves compute units idle, the key axis is split over workgroups, whose
// results attn_join adds.
//
// What bounds it, and what it measured (kernels in a row under the profiler;
// among other work, at a higher clock, the calls take 43 and 110 us):
//   bf16 [16,750,8x128], lengths 750 to 398: 46 to 49 us, 22.4 GFLOP of valid
//     pairs, 470 TFLOP/s.  A run over one key tile takes 22 us of that; at 47 us
//     in all, leaving out most of either product saved 6 to 7 us, the weights 3,
//     the bias 4, the loads of the tiles 8: no one unit fills it.  At
//     [4,3000,8x128], all frames valid, 188 us, 786 TFLOP/s.
//   float, causal [8,1500,8x64]: 126 to 129 us, 11.6 GFLOP, 91 TFLOP/s in the six
//     bf16 products that stand for each; each wave splits its own operands.
//   bf16, 8 frames of 64 streams over 391 keys: 11 us; one frame of 4 streams
//     over 6000 keys: 14 us and 3.8 us for the join, several times what their
//     bytes take: few tiles a workgroup, so latency.
// For [16,750,8x128], when it took 51 us: all of a tile's operands read ahead,
// two workgroups a compute unit, 62 us; tiles of 64 keys, 61 us.
#include "attn.h"

namespace dw {

struct AttnFwd : AttnArgs {
    void* out;     // [B][Tq][H][D]
    float* lse;    // [B][H][Tq] or NULL
    float* part;   // splits > 1: [splits][B * H * Tq][D4] unnormalised sums, then [splits][B * H * Tq][2] maxima and sums
    int32_t splits, nqb;
};

// The scores are kept in units of log2.  The running maximum follows the true
// one only when that has grown by more than kSlack: the weights then stay
// below 2^kSlack, and most tiles need no rescaling of the accumulators.
constexpr float kSlack = 8.0f;

// A flat bias up to this rides on the multiply that scales the scores.  In the
// sum of a larger one and a score, which the running maximum follows, the score
// may vanish, and a weight taken from both apart would pass 2^kSlack by as much
// as the score (here the sum still has 2^-8 of it); that bias is added to the
// scores first, as a looked-up one is.
constexpr float kRides = 65536.0f;

// Keys of a tile, its buffers, and the waves per SIMD that its registers are to
// allow.
template <typename S, int DP, int QW, bool DMA>
struct FwdShape {
    static constexpr int BN = QW == 1 ? 128 : QW == 2 || sizeof(S) * DP <= 128 ? 64 : 32;
    static constexpr int kBuffers = QW == 1 && !DMA ? 1 : 2;
    static constexpr int kWaves = (QW == 1 && DP > 64) || (sizeof(S) == 4 && DP > 96) ? 1 : QW == 4 && DMA && sizeof(S) == 2 ? 3 : 2;
    using Tiles = TilePair<S, DP, BN, kBuffers, DMA>;
};

// PACKED: the query heads that share a key head lie side by side in the columns
// (column c is query c % Tq of the group's head c / Tq), so that their keys are
// read and multiplied once; the bias is then there for each of them.
template <typename S, int DP, int QW, bool DMA, bool PACKED = false>
__global__ __launch_bounds__(kAttnThreads, (FwdShape<S, DP, QW, DMA>::kWaves)) void attn_fwd_kernel(const AttnFwd a) {
    static_assert(!PACKED || QW == 1, "the heads of a group share one tile of queries");
    using F = FwdShape<S, DP, QW, DMA>;
    constexpr int KW = 4 / QW, BN = F::BN, KT = BN / kTile / KW, NC = DP / 16, ND = DP / 32;
    typedef Tile<S, DP> T;
    extern __shared__ __align__(16) char smem[];
    float* bias = (float*)(smem + F::Tiles::kAllBytes);
    const int lane = threadIdx.x % 64, wave = wave_of_block(), half = lane / 32;
    const int wq = wave % QW, wk = wave / QW;

    const int heads = PACKED ? a.Hkv : a.H, group = a.H / a.Hkv;
    const AttnPlace place(blockIdx.x, a.nqb * a.splits, a.B * heads, a.left == kNoLimit && a.right != kNoLimit);
    const int split = place.block % a.splits, qb = place.block / a.splits;
    const int head = place.pair % heads, b = a.nqb > 1 ? item_of_rank(a, place.pair / heads) : place.pair / heads;
    const int hk = PACKED ? head : head / group;
    const AttnItem item(a, b);
    const int i0 = qb * (kTile * QW), iw = i0 + wq * kTile;
    const int member = PACKED ? lane % 32 / a.Tq : 0;  // of the group
    const int i = PACKED ? lane % 32 - member * a.Tq : iw + lane % 32, h = PACKED ? hk * group + member : head;
    const bool mine_to_write = PACKED ? member < group : i < a.Tq, live = mine_to_write && i < item.nq;

    // this lane's keys: [mine0, mine0 + mine)
    const int mine0 = item.first_key(a, i);
    const int mine1 = item.last_key(a, i);
    const uint32_t mine = live && mine1 >= mine0 ? mine1 - mine0 + 1 : 0;

    // the workgroup's keys, and this split's share of them
    int j0 = 0, j1 = 0;
    if (i0 < item.nq) {
        const int ilast = min(i0 + kTile * QW, item.nq) - 1;
        j0 = item.first_key(a, i0);
        j1 = item.last_key(a, ilast) + 1;
    }
    const int tiles = j1 > j0 ? (j1 - j0 + BN - 1) / BN : 0, share = (tiles + a.splits - 1) / a.splits;
    const int t0 = min(split * share, tiles), t1 = min(t0 + share, tiles);
    // the wave's keys, for the tiles that it can pass over or take unmasked
    const int iwl = min(iw + (PACKED ? a.Tq : kTile), item.nq) - 1;
    const int some0 = item.first_key(a, iw), some1 = iw < item.nq ? item.last_key(a, iwl) : -1;
    const int all0 = item.first_key(a, iwl), all1 = iw < item.nq ? item.last_key(a, iw) : -1;

    const int64_t j00 = j0 + t0 * BN;
    typename F::Tiles kv(smem, (const S*)a.k + b * a.ks.item + hk * a.ks.head + j00 * a.ks.frame, a.ks.frame,
                         (const S*)a.v + b * a.vs.item + hk * a.vs.head + j00 * a.vs.frame, a.vs.frame, a.D,
                         min(j1, j0 + t1 * BN) - (int)j00);

    const BiasFill<S> filler(a);
    if (t0 < t1) kv.start(0);
    Frag<S> q[NC];
    {
        const S* row = (const S*)a.q + b * a.qs.item + (int64_t)(live ? i : 0) * a.qs.frame + h * a.qs.head;
#pragma unroll
        for (int c = 0; c < NC; ++c) q[c] = to_frag<S>(load_group<S, !DMA>(row, 16 * c + 8 * half, live ? a.D : 0));
    }
    const int nbias = 2 * a.R + 1 + 2 * kBiasMargin;
    if constexpr (PACKED) {
        for (int m = 0; m < group; ++m) filler.fill(a, hk * group + m, bias + m * nbias);
    } else {
        filler.fill(a, h, bias);
    }
    // this lane's head's bias, from the place of its query
    const float* my_bias = bias + min(member, group - 1) * nbias;
    const int column = PACKED ? i : lane % 32;
    if (F::kBuffers == 2 && t0 < t1) kv.finish(0);
#pragma unroll
    for (int c = 0; c < NC; ++c) arrived(q[c]);
    f32x16 o[ND] = {};
    float top = -__builtin_inff(), sum = 0.0f;
    for (int t = 0; t < t1 - t0; ++t) {
        kv.enter(t, t + 1 < t1 - t0);
        const S* kt = kv.x_of(t);
        const S* vt = kv.y_of(t);
#pragma unroll
        for (int u = 0; u < KT; ++u) {
            const int row0 = (wk * KT + u) * kTile, j = (int)j00 + t * BN + row0;
            if (j > some1 || j + kTile <= some0) continue;
            // The tile's operands are read ahead of their use: the keys before
            // the first product, the first half of the values before the softmax
            // (as many as leave three waves a SIMD their registers).
            Frag<S> k[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) k[c] = T::rows(kt, row0, c, lane);
            __builtin_amdgcn_sched_barrier(0);
            f32x16 s = {};
#pragma unroll
            for (int c = 0; c < NC; ++c) s = mma(k[c], q[c], s);
            constexpr bool kAhead = sizeof(S) == 2;  // float's values would take twice the registers
            Frag<S> v[ND];
            if (kAhead) {
#pragma unroll
                for (int d = 0; d < ND; ++d) v[d] = T::columns(vt, row0, d, lane);
            }
            products_done(s);
            const int base = j - iw - item.pos32;
            const Span span = span_of(base, a.R);
            const bool edge = j < all0 || j + kTile - 1 > all1;
            // s becomes the weights exp2(scale2 * s + bias - top).  The flat
            // bias of a tile past the map's reach rides on the multiply
            // (scale2 > 0, so the largest score is that of the largest
            // product); a looked-up or a huge one is added first, the latter
            // from the map's repeated ends.
            float factor = a.scale2, flat = 0.0f;
            bool look = a.table && span == Span::kNear;
            if (a.table && span != Span::kNear) {
                flat = my_bias[span == Span::kLow ? 0 : nbias - 1];
                look = __any(fabsf(flat) > kRides);
            }
            if (look) {
                const int at = max(-a.R - kTile + 1, min(base, a.R + kTile - 1));
                const float* f = my_bias + (at + a.R + kBiasMargin + 4 * half - column);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale2, f[acc_row(r, 0)]);
                factor = 1.0f;
                flat = 0.0f;
            }
            if (edge) {
                const uint32_t at = j + 4 * half - mine0;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = at + acc_row(r, 0) < mine ? s[r] : -__builtin_inff();
            }
            float m = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) m = fmaxf(m, s[r]);
            m = fmaf(fmaxf(m, swap_halves(m)), factor, flat);
            if (__any(m > top + kSlack)) {
                m = fmaxf(m, top);
                const float f = m == -__builtin_inff() ? 1.0f : exp2_fast(top - m);
                sum *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[d][r] *= f;
                top = m;
            }
            flat -= top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = exp2_fast(fmaf(s[r], factor, flat));
                sum += s[r];
            }
            const Frag<S> p[2] = {to_frag<S>(s, 0), to_frag<S>(s, 1)};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    o[d] = mma(kAhead && c == 0 ? v[d] : T::columns(vt, row0 + 16 * c, d, lane), p[c], o[d]);
        }
        kv.leave(t, t + 1 < t1 - t0);
    }
    products_done(o);
    sum += swap_halves(sum);

    // Join the waves that share queries: wave wk of them takes every KW-th run
    // of 32 head elements.
    constexpr int NJ = (ND + KW - 1) / KW;
    if constexpr (KW > 1) {
        float* opart = (float*)smem;                          // [4][ND * 16][64]
        float* stat = (float*)(smem + 4 * ND * 16 * 64 * 4);  // [4][2][32]
        static_assert(4 * ND * 16 * 64 * 4 + 4 * 2 * 32 * 4 <= F::Tiles::kAllBytes, "the tiles' room holds the join");
        __syncthreads();
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) opart[((wave * ND + d) * 16 + r) * 64 + lane] = o[d][r];
        if (half == 0) {
            stat[wave * 64 + lane] = top;
            stat[wave * 64 + 32 + lane] = sum;
        }
        __syncthreads();
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < KW; ++w) m = fmaxf(m, stat[(w * QW + wq) * 64 + lane % 32]);
        float f[KW];
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            f[w] = m == -__builtin_inff() ? 0.0f : exp2_fast(stat[(w * QW + wq) * 64 + lane % 32] - m);
            sum += f[w] * stat[(w * QW + wq) * 64 + 32 + lane % 32];
        }
        top = m;
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
            const int d = wk + n * KW;
            if (d >= ND) break;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) v += f[w] * opart[(((w * QW + wq) * ND + d) * 16 + r) * 64 + lane];
                o[n][r] = v;
            }
        }
    }
    if (!mine_to_write) return;
    if (!live) {  // its columns went along with the others'
        top = -__builtin_inff();
        sum = 0.0f;
#pragma unroll
        for (int n = 0; n < NJ; ++n) o[n] = f32x16{};
    }
    const int64_t row = ((int64_t)b * a.H + h) * a.Tq + i;
    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // a row without keys is zero; NaN stays
#pragma unroll
    for (int n = 0; n < NJ; ++n) {
        const int d0 = 32 * (wk + n * KW) + 4 * half;
        if (wk + n * KW >= ND) break;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float v[4] = {o[n][4 * g], o[n][4 * g + 1], o[n][4 * g + 2], o[n][4 * g + 3]};
            if (a.splits > 1) {
                const int64_t rows = (int64_t)a.B * a.H * a.Tq;
                const int D4 = (a.D + 3) / 4 * 4;
                store4<float>(a.part + (split * rows + row) * D4, d0 + 8 * g, D4, v[0], v[1], v[2], v[3]);
            } else {
                store4<S>((S*)a.out + (((int64_t)b * a.Tq + i) * a.H + h) * a.D, d0 + 8 * g, a.D, v[0] * inv, v[1] * inv,
                          v[2] * inv, v[3] * inv);
            }
        }
    }
    if (half == 0 && wk == 0) {
        if (a.splits > 1) {
            const int64_t rows = (int64_t)a.B * a.H * a.Tq;
            float* stat = a.part + a.splits * rows * ((a.D + 3) / 4 * 4) + (split * rows + row) * 2;
            stat[0] = top;
            stat[1] = sum;
        } else if (a.lse) {
            a.lse[row] = sum == 0.0f ? -__builtin_inff() : (top + log2f(sum)) * kLn2;
        }
    }
}

// Joins the splits of the key axis: one thread takes 4 head elements of a row,
// kJoin splits' loads in flight together (3.8 us for 8 splits, nearly all of it
// latency; one after the other 10 us).
constexpr int kJoin = 8;

template <typename S>
__global__ __launch_bounds__(kAttnThreads) void attn_join(const AttnFwd a) {
    const int D4 = (a.D + 3) / 4;
    const int64_t rows = (int64_t)a.B * a.H * a.Tq, at = (int64_t)blockIdx.x * kAttnThreads + threadIdx.x;
    if (at >= rows * D4) return;
    const int64_t row = at / D4;
    const int d = (int)(at - row * D4);
    const float* stat = a.part + a.splits * rows * D4 * 4;
    float m = -__builtin_inff(), sum = 0.0f;
    f32x4 o = {};
    for (int s0 = 0; s0 < a.splits; s0 += kJoin) {  // kJoin splits' loads are in flight together
        float top[kJoin], part[kJoin];
        f32x4 v[kJoin];
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const int64_t s = min(s0 + k, a.splits - 1);
            top[k] = stat[(s * rows + row) * 2];
            part[k] = stat[(s * rows + row) * 2 + 1];
            v[k] = *reinterpret_cast<const f32x4*>(a.part + ((s * rows + row) * D4 + d) * 4);
        }
        float next = m;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) next = fmaxf(next, top[k]);
        const float ref = next == -__builtin_inff() ? 0.0f : next, f = exp2_fast(m - ref);
        sum *= f;
        o *= f;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const float g = s0 + k < a.splits ? exp2_fast(top[k] - ref) : 0.0f;
            sum += g * part[k];
            o += g * v[k];
        }
        m = next;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
    const int64_t i = row % a.Tq, bh = row / a.Tq;
    S* out = (S*)a.out + (((bh / a.H) * a.Tq + i) * a.H + bh % a.H) * a.D;
    store4<S>(out, 4 * d, a.D, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (d == 0 && a.lse) a.lse[row] = sum == 0.0f ? -__builtin_inff() : (m + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------------
// Launch plan
// ---------------------------------------------------------------------------
static int64_t part_floats(const AttnShape& s, int splits) {
    return splits > 1 ? splits * s.B * s.H * s.Tq * ((s.D + 3) / 4 * 4 + 2) : 0;
}

size_t dwattn_fwd_workspace(const AttnShape& s) {
    return (size_t)part_floats(s, fwd_plan(s).splits) * sizeof(float);
}

bool dwattn_fits(const AttnShape& s) {
    // workgroups of the narrowest tiles, and the rows
    const int64_t q32 = (s.Tq + 31) / 32, k32 = (s.Tk + 31) / 32;
    return product_below(kMaxExtent, {s.B, s.H, q32}) && product_below(kMaxExtent, {s.B, s.H, k32}) &&
           product_below(kMaxExtent, {s.B, s.H, s.Tq});
}

bool dwattn_fwd_fits(const AttnShape& s) {
    const FwdPlan p = fwd_plan(s);
    // splits are for a few hundred workgroups of at most 32 queries, so the join's threads are few
    return grid_of_256_fits(s.B * (p.packed ? s.Hkv : s.H) * p.nqb * p.splits);
}

template <typename S, int DP, int QW, bool DMA, bool PACKED = false>
static hipError_t launch_fwd(const AttnFwd& a, hipStream_t stream) {
    using F = FwdShape<S, DP, QW, DMA>;
    const int biases = PACKED ? a.H / a.Hkv : 1, lds = F::Tiles::kAllBytes + (a.table ? biases * attn_bias_bytes(a.R) : 0);
    hipLaunchKernelGGL((attn_fwd_kernel<S, DP, QW, DMA, PACKED>),
                       dim3((uint32_t)(a.B * (PACKED ? a.Hkv : a.H)) * a.nqb * a.splits), dim3(kAttnThreads), lds, stream, a);
    return hipGetLastError();
}

template <typename S>
static hipError_t fwd_of_type(const AttnFwd& a, const FwdPlan& plan, hipStream_t stream) {
    const bool direct = direct_fits(a.k, a.ks, a.D, sizeof(S)) && direct_fits(a.v, a.vs, a.D, sizeof(S));
    const AttnForm f = fwd_form(plan, a.D, sizeof(S), direct);
    const hipError_t e = with_head_width(a.D, [&](auto dp) {
        constexpr bool kNarrow = fwd_narrow(dp.value, sizeof(S));
        return f.packed && f.direct   ? launch_fwd<S, dp.value, 1, kNarrow, true>(a, stream)
               : f.packed             ? launch_fwd<S, dp.value, 1, false, true>(a, stream)
               : f.own == 1 && f.direct ? launch_fwd<S, dp.value, 1, kNarrow>(a, stream)
               : f.own == 1           ? launch_fwd<S, dp.value, 1, false>(a, stream)
               : f.own == 2 && f.direct ? launch_fwd<S, dp.value, 2, true>(a, stream)
               : f.own == 2           ? launch_fwd<S, dp.value, 2, false>(a, stream)
               : f.direct             ? launch_fwd<S, dp.value, 4, true>(a, stream)
                                      : launch_fwd<S, dp.value, 4, false>(a, stream);
    });
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t threads = (int64_t)a.B * a.H * a.Tq * ((a.D + 3) / 4);
    hipLaunchKernelGGL(attn_join<S>, dim3((uint32_t)((threads + kAttnThreads - 1) / kAttnThreads)), dim3(kAttnThreads), 0,
                       stream, a);
    return hipGetLastError();
}

hipError_t launch_dwattn_fwd(const AttnPtrs& p, const AttnShape& s, void* out, float* lse, void* workspace, bool bf16,
                             hipStream_t stream) {
    const FwdPlan plan = fwd_plan(s);
    AttnFwd a;
    (AttnArgs&)a = attn_args(p, s);
    a.out = out;
    a.lse = lse;
    a.part = (float*)workspace;
    a.splits = plan.splits;
    a.nqb = (int32_t)plan.nqb;
    return bf16 ? fwd_of_type<uint16_t>(a, plan, stream) : fwd_of_type<float>(a, plan, stream);
}

}  // namespace dw
