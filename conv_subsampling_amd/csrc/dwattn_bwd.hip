// Self-attention with a learned relative position bias by buckets: gradients.
//
//   P_ij = exp(S_ij - lse_i),  delta_i = dout_i . out_i
//   dS   = P * (dout v^T - delta)
//   dv   = P^T dout,  dk = scale * dS^T q,  dq = scale * dS k,  dbias[r] = sum of dS over the pairs r apart
//
// Nothing of the [Tq][Tk] maps goes to memory: two kernels recompute P, one
// for the side that each owns, so that every sum is taken by one wave in a
// fixed order and there are no atomics.
//   attn_dq_kernel   a wave owns 32 queries and streams the keys: dq, delta
//                    (for the other kernel), and the sums of dS by distance
//   attn_dkv_kernel  a wave owns 32 keys and streams the queries of every
//                    head that shares them: dk and dv
// attn_dbias_rows and attn_dtable then add the sums by distance over the
// workgroups and into buckets, in fp64.
#include "attn.h"

namespace dw {

struct AttnBwd : AttnArgs {
    const void *out, *dout;  // [B][Tq][H][D]
    const float* lse;        // [B][H][Tq]
    float* delta;            // [B][H][Tq]
    void *dq, *dk, *dv;
    AttnStride dqs, dks, dvs;
    float* dist;  // [H][B * nqb][2 R + 1] sums of dS by distance; NULL: not wanted
    int32_t nqb, nkb;
};

constexpr int kBwdOwned = 4 * kTile;  // queries or keys a workgroup owns
constexpr int kDiag = 36;             // row stride of the square that the diagonals are read from

// exp(S - lse) of a query that has keys; lse = -inf marks one that has none,
// whose weights are zero.
__device__ __forceinline__ float lse_or_inf(float lse) {
    return lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
}


// Orders a wave's LDS accesses before and after it: lanes read what other
// lanes of their wave wrote.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Streamed frames of a tile (two tiles of each tensor are in LDS).
template <typename S, int DP>
constexpr int kBwdRows = sizeof(S) * DP <= 128 ? 64 : 32;

template <typename S, int DP, bool DMA>
__global__ __launch_bounds__(kAttnThreads, (DP > 64 && (sizeof(S) == 4 || !DMA) ? 1 : 2)) void attn_dq_kernel(const AttnBwd a) {
    constexpr int BN = kBwdRows<S, DP>, KT = BN / kTile, NC = DP / 16, ND = DP / 32;
    typedef Tile<S, DP> T;
    extern __shared__ __align__(16) char smem[];
    float* bias = (float*)(smem + 4 * T::bytes(BN));
    const int nbias = 2 * a.R + 1 + 2 * kBiasMargin;
    const int lane = threadIdx.x % 64, wave = wave_of_block(), half = lane / 32;
    float* square = bias + (nbias + 3) / 4 * 4 + wave * kTile * kDiag;                      // a tile of dS
    float* sums = bias + (nbias + 3) / 4 * 4 + 4 * kTile * kDiag + wave * nbias;            // by distance, of this wave

    const AttnPlace place(blockIdx.x, a.nqb, a.B * a.H, a.left == kNoLimit && a.right != kNoLimit);
    const int qb = place.block, h = place.pair % a.H, b = item_of_rank(a, place.pair / a.H);
    const AttnItem item(a, b);
    const int i0 = qb * kBwdOwned, iw = i0 + wave * kTile, i = iw + lane % 32;
    const bool live = i < item.nq;
    const BiasFill<S> filler(a);
    if (a.dist)
        for (int x = lane; x < nbias; x += 64) sums[x] = 0.0f;

    Frag<S> q[NC], g[NC];
    float delta = 0.0f, lse2 = __builtin_inff();
    {
        const S* row = (const S*)a.q + b * a.qs.item + (int64_t)(live ? i : 0) * a.qs.frame + h * a.qs.head;
        const int64_t at = (((int64_t)b * a.Tq + (live ? i : 0)) * a.H + h) * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = 16 * c + 8 * half, D = live ? a.D : 0;
            const RawGroup<S> gr = load_group<S, !DMA>((const S*)a.dout + at, d, D);
            q[c] = to_frag<S>(load_group<S, !DMA>(row, d, D));
            g[c] = to_frag<S>(gr);
            const Vf<kGroup> x = widen<S>(gr), o = widen<S>(load_group<S, !DMA>((const S*)a.out + at, d, D));
#pragma unroll
            for (int e = 0; e < kGroup; ++e) delta = fmaf(x.v[e], o.v[e], delta);
        }
        delta += swap_halves(delta);
        const int64_t stat = ((int64_t)b * a.H + h) * a.Tq + i;
        if (live) lse2 = lse_or_inf(a.lse[stat]);
        if (half == 0 && i < a.Tq) a.delta[stat] = delta;
    }
    if (!a.dq && !a.dist) return;
    filler.fill(a, h, bias);
    const int mine0 = item.first_key(a, i), mine1 = item.last_key(a, i);
    const uint32_t mine = live && mine1 >= mine0 ? mine1 - mine0 + 1 : 0;
    int j0 = 0, j1 = 0;
    if (i0 < item.nq) {
        j0 = item.first_key(a, i0);
        j1 = item.last_key(a, min(i0 + kBwdOwned, item.nq) - 1) + 1;
    }
    const int iwl = min(iw + kTile, item.nq) - 1;
    const int some0 = item.first_key(a, iw), some1 = iw < item.nq ? item.last_key(a, iwl) : -1;
    const int all0 = item.first_key(a, iwl), all1 = iw + kTile <= item.nq ? item.last_key(a, iw) : -1;

    const S* kbase = (const S*)a.k + b * a.ks.item + (int64_t)(h / (a.H / a.Hkv)) * a.ks.head;
    const S* vbase = (const S*)a.v + b * a.vs.item + (int64_t)(h / (a.H / a.Hkv)) * a.vs.head;
    TileLoad<S, DP, BN, DMA> kl, vl;
    kl.setup(a.ks.frame, a.D);
    vl.setup(a.vs.frame, a.D);
    auto ktile_of = [&](int t) { return (S*)(smem + (t & 1) * 2 * T::bytes(BN)); };
    auto vtile_of = [&](int t) { return (S*)((char*)ktile_of(t) + T::bytes(BN)); };
    auto start = [&](int t) {
        const int64_t j = j0 + t * BN;
        kl.start(kbase + j * a.ks.frame, a.ks.frame, j1 - (int)j, a.D, ktile_of(t));
        vl.start(vbase + j * a.vs.frame, a.vs.frame, j1 - (int)j, a.D, vtile_of(t));
    };
    auto finish = [&](int t) {
        kl.finish(ktile_of(t));
        vl.finish(vtile_of(t));
    };
    const int tiles = j1 > j0 ? (j1 - j0 + BN - 1) / BN : 0;
    if (tiles) {
        start(0);
        finish(0);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) arrived(q[c]), arrived(g[c]);
    asm volatile("" : "+v"(lse2), "+v"(delta));
    f32x16 acc[ND] = {};
    float low = 0.0f, high = 0.0f;  // sums of dS past the map's reach
    for (int t = 0; t < tiles; ++t) {
        wave_loads_done();
        __syncthreads();
        if (t + 1 < tiles) start(t + 1);
        const S* ktile = ktile_of(t);
        const S* vtile = vtile_of(t);
        const int jt = j0 + t * BN;
#pragma unroll
        for (int u = 0; u < KT; ++u) {
            const int row0 = u * kTile, j = jt + row0;
            if (j > some1 || j + kTile <= some0) continue;
            f32x16 s = {}, ds = {};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                s = mma(T::rows(ktile, row0, c, lane), q[c], s);
                ds = mma(T::rows(vtile, row0, c, lane), g[c], ds);
            }
            products_done<S>();
            const int base = j - iw - item.pos32;
            const Span span = span_of(base, a.R);
            if (a.table && span == Span::kNear) {
                const float* p = bias + (base + a.R + kBiasMargin + 4 * half - lane % 32);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = exp2_fast(fmaf(s[r], a.scale2, p[acc_row(r, 0)]) - lse2);
            } else {
                const float flat = a.table ? bias[span == Span::kLow ? 0 : nbias - 1] : 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = exp2_fast(fmaf(s[r], a.scale2, flat) - lse2);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) ds[r] = s[r] * (ds[r] - delta);
            if (j < all0 || j + kTile - 1 > all1) {
                const uint32_t at = j + 4 * half - mine0;
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = at + acc_row(r, 0) < mine ? ds[r] : 0.0f;
            }
            if (a.dist) {
                if (span == Span::kNear) {
                    // The 63 diagonals of the tile: rows are queries in the
                    // square, and lane x reads column (x + row) mod 32, which
                    // is the diagonal x up to the wrap and x - 32 after it.
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        *reinterpret_cast<f32x4*>(square + (lane % 32) * kDiag + 8 * n + 4 * half) =
                            f32x4{ds[4 * n], ds[4 * n + 1], ds[4 * n + 2], ds[4 * n + 3]};
                    wave_lds_fence();
                    float up = 0.0f, down = 0.0f;
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        const int row = 16 * half + n, col = lane % 32 + row;
                        const float x = square[row * kDiag + col % 32];
                        up += col < 32 ? x : 0.0f;
                        down += col < 32 ? 0.0f : x;
                    }
                    up += swap_halves(up);
                    down += swap_halves(down);
                    float* p = sums + base + a.R + kBiasMargin + lane % 32;
                    if (half == 0) *p += up;
                    else p[-32] += down;
                    wave_lds_fence();
                } else {
                    float t = 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) t += ds[r];
                    if (span == Span::kLow) low += t;
                    else high += t;
                }
            }
            if (a.dq) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const Frag<S> p = to_frag<S>(ds, k);
#pragma unroll
                    for (int d = 0; d < ND; ++d) acc[d] = mma(T::columns(ktile, row0 + 16 * k, d, lane), p, acc[d]);
                }
            }
        }
        if (t + 1 < tiles) finish(t + 1);
    }
    products_done<S>();
    if (a.dq && i < a.Tq) {
        S* row = (S*)a.dq + b * a.dqs.item + (int64_t)i * a.dqs.frame + h * a.dqs.head;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                store4<S>(row, 32 * d + 8 * n + 4 * half, a.D, acc[d][4 * n] * a.scale, acc[d][4 * n + 1] * a.scale,
                          acc[d][4 * n + 2] * a.scale, acc[d][4 * n + 3] * a.scale);
    }
    if (!a.dist) return;
    low = lane_sum<64>(low);
    high = lane_sum<64>(high);
    if (lane == 0) {
        sums[0] += low;
        sums[nbias - 1] += high;
    }
    __syncthreads();
    const float* all = bias + (nbias + 3) / 4 * 4 + 4 * kTile * kDiag;
    float* to = a.dist + (((int64_t)h * a.B + b) * a.nqb + qb) * (2 * a.R + 1);
    for (int x = threadIdx.x; x < 2 * a.R + 1; x += kAttnThreads) {
        // the margins stand for the ends
        const int from = x == 0 ? 0 : x + kBiasMargin, till = x == 2 * a.R ? nbias : x + kBiasMargin + 1;
        float t = 0.0f;
        for (int y = from; y < till; ++y)
            t += (all[y] + all[nbias + y]) + (all[2 * nbias + y] + all[3 * nbias + y]);
        to[x] = t;
    }
}

// Sums by distance of one head over all workgroups, [H][2 R + 1] doubles: 16
// sub-rows x 64 distances, each sub-row every 16th workgroup, then in order.
constexpr int kDistCols = 64, kDistRows = 16;

__global__ __launch_bounds__(kDistCols* kDistRows) void attn_dbias_rows(const float* __restrict__ dist,
                                                                      double* __restrict__ total, int32_t n,
                                                                      int32_t parts) {
    __shared__ double acc[kDistRows][kDistCols];
    const int lane = threadIdx.x % kDistCols, sub = threadIdx.x / kDistCols, x = blockIdx.x * kDistCols + lane;
    const float* from = dist + (int64_t)blockIdx.y * parts * n;
    double s = 0.0;
    if (x < n) {
#pragma unroll 4
        for (int32_t r = sub; r < parts; r += kDistRows) s += from[(int64_t)r * n + x];
    }
    acc[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || x >= n) return;
    double t = acc[0][lane];
#pragma unroll
    for (int q = 1; q < kDistRows; ++q) t += acc[q][lane];
    total[(int64_t)blockIdx.y * n + x] = t;
}

// dtable[bucket][h]: each wave takes a bucket and adds the distances in it.
__global__ __launch_bounds__(kAttnThreads) void attn_dtable(const double* __restrict__ total,
                                                           const int32_t* __restrict__ map, float* __restrict__ dtable,
                                                           int32_t n, int32_t NB, int32_t H) {
    const int h = blockIdx.y, lane = threadIdx.x % 64;
    const int bucket = blockIdx.x * (kAttnThreads / 64) + threadIdx.x / 64;
    if (bucket >= NB) return;
    double s = 0.0;
    for (int x = lane; x < n; x += 64) {
        int m = map[x];
        m = m < 0 ? 0 : m >= NB ? NB - 1 : m;
        s += m == bucket ? total[(int64_t)h * n + x] : 0.0;
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m);
    if (lane == 0) dtable[(int64_t)bucket * H + h] = (float)s;
}

// ---------------------------------------------------------------------------
template <typename S, int DP, bool DMA>
__global__ __launch_bounds__(kAttnThreads, (DP > 64 || sizeof(S) == 4 ? 1 : 2)) void attn_dkv_kernel(const AttnBwd a) {
    constexpr int BQ = kBwdRows<S, DP>, QT = BQ / kTile, NC = DP / 16, ND = DP / 32;
    typedef Tile<S, DP> T;
    extern __shared__ __align__(16) char smem[];
    float* stats = (float*)(smem + 4 * T::bytes(BQ));  // of two tiles: [2][2][BQ], lse in units of log2, then delta
    float* bias = stats + 4 * BQ;
    const int nbias = 2 * a.R + 1 + 2 * kBiasMargin;
    const int lane = threadIdx.x % 64, wave = wave_of_block(), half = lane / 32;

    const AttnPlace place(blockIdx.x, a.nkb, a.B * a.Hkv, a.right == kNoLimit && a.left != kNoLimit);
    const int kb = place.block, hk = place.pair % a.Hkv, b = item_of_rank(a, place.pair / a.Hkv), group = a.H / a.Hkv;
    const AttnItem item(a, b);
    const int j0 = kb * kBwdOwned, jw = j0 + wave * kTile, j = jw + lane % 32;
    const bool live = j < item.nk;

    Frag<S> k[NC], v[NC];
    {
        const S* kr = (const S*)a.k + b * a.ks.item + (int64_t)(live ? j : 0) * a.ks.frame + hk * a.ks.head;
        const S* vr = (const S*)a.v + b * a.vs.item + (int64_t)(live ? j : 0) * a.vs.frame + hk * a.vs.head;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            k[c] = to_frag<S>(load_group<S, !DMA>(kr, 16 * c + 8 * half, live ? a.D : 0));
            v[c] = to_frag<S>(load_group<S, !DMA>(vr, 16 * c + 8 * half, live ? a.D : 0));
        }
    }
    const int mine0 = item.first_query(a, j), mine1 = item.last_query(a, j);
    const uint32_t mine = live && mine1 >= mine0 ? mine1 - mine0 + 1 : 0;
    int i0 = 0, i1 = 0;
    if (j0 < item.nk) {
        i0 = item.first_query(a, j0);
        i1 = item.last_query(a, min(j0 + kBwdOwned, item.nk) - 1) + 1;
    }
    const int jwl = min(jw + kTile, item.nk) - 1;
    const int some0 = item.first_query(a, jw), some1 = jw < item.nk ? item.last_query(a, jwl) : -1;
    const int all0 = item.first_query(a, jwl), all1 = jw + kTile <= item.nk ? item.last_query(a, jw) : -1;

    f32x16 dk[ND] = {}, dv[ND] = {};
    for (int n = 0; n < group; ++n) {
        const int h = hk * group + n;
        __syncthreads();  // the head before is done with the tiles and its bias
        const BiasFill<S> filler(a);
        const S* qbase = (const S*)a.q + b * a.qs.item + h * a.qs.head;
        const S* gbase = (const S*)a.dout + ((int64_t)b * a.Tq * a.H + h) * a.D;
        const int64_t gstride = (int64_t)a.H * a.D, srow = ((int64_t)b * a.H + h) * a.Tq;
        TileLoad<S, DP, BQ, DMA> ql, gl;
        ql.setup(a.qs.frame, a.D);
        gl.setup(gstride, a.D);
        float row_lse = 0.0f, row_delta = 0.0f;
        auto qtile_of = [&](int t) { return (S*)(smem + (t & 1) * 2 * T::bytes(BQ)); };
        auto gtile_of = [&](int t) { return (S*)((char*)qtile_of(t) + T::bytes(BQ)); };
        auto start = [&](int t) {
            const int64_t i = i0 + t * BQ;
            const bool mine = threadIdx.x < BQ && i + threadIdx.x < i1;
            row_lse = mine ? a.lse[srow + i + threadIdx.x] : -__builtin_inff();
            row_delta = mine ? a.delta[srow + i + threadIdx.x] : 0.0f;
            ql.start(qbase + i * a.qs.frame, a.qs.frame, i1 - (int)i, a.D, qtile_of(t));
            gl.start(gbase + i * gstride, gstride, i1 - (int)i, a.D, gtile_of(t));
        };
        auto finish = [&](int t) {
            ql.finish(qtile_of(t));
            gl.finish(gtile_of(t));
            if (threadIdx.x < BQ) {
                stats[(t & 1) * 2 * BQ + threadIdx.x] = lse_or_inf(row_lse);
                stats[(t & 1) * 2 * BQ + BQ + threadIdx.x] = row_delta;
            }
        };
        const int tiles = i1 > i0 ? (i1 - i0 + BQ - 1) / BQ : 0;
        if (tiles) start(0);
        filler.fill(a, h, bias);
        if (tiles) finish(0);
#pragma unroll
        for (int c = 0; c < NC; ++c) arrived(k[c]), arrived(v[c]);
        for (int t = 0; t < tiles; ++t) {
            wave_loads_done();
            __syncthreads();
            if (t + 1 < tiles) start(t + 1);
            const S* qtile = qtile_of(t);
            const S* gtile = gtile_of(t);
            const float* stat = stats + (t & 1) * 2 * BQ;
            const int it = i0 + t * BQ;
#pragma unroll
            for (int u = 0; u < QT; ++u) {
                const int row0 = u * kTile, i = it + row0;
                if (i > some1 || i + kTile <= some0) continue;
                f32x16 s = {}, ds = {};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    s = mma(T::rows(qtile, row0, c, lane), k[c], s);
                    ds = mma(T::rows(gtile, row0, c, lane), v[c], ds);
                }
                products_done<S>();
                // distance of the tile's first key and first query; along the registers it falls
                const int base = jw - i - item.pos32;
                const Span span = span_of(base, a.R);
                f32x4 lse2[4], delta[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    lse2[r] = *reinterpret_cast<const f32x4*>(stat + row0 + 8 * r + 4 * half);
                    delta[r] = *reinterpret_cast<const f32x4*>(stat + BQ + row0 + 8 * r + 4 * half);
                }
                if (a.table && span == Span::kNear) {
                    const float* p = bias + (base + a.R + kBiasMargin - 4 * half + lane % 32);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = exp2_fast(fmaf(s[r], a.scale2, p[-acc_row(r, 0)]) - lse2[r / 4][r % 4]);
                } else {
                    const float flat = a.table ? bias[span == Span::kLow ? 0 : nbias - 1] : 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = exp2_fast(fmaf(s[r], a.scale2, flat) - lse2[r / 4][r % 4]);
                }
                if (i < all0 || i + kTile - 1 > all1) {
                    const uint32_t at = i + 4 * half - mine0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = at + acc_row(r, 0) < mine ? s[r] : 0.0f;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = s[r] * (ds[r] - delta[r / 4][r % 4]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const Frag<S> p = to_frag<S>(s, c), g = to_frag<S>(ds, c);
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        dv[d] = mma(T::columns(gtile, row0 + 16 * c, d, lane), p, dv[d]);
                        dk[d] = mma(T::columns(qtile, row0 + 16 * c, d, lane), g, dk[d]);
                    }
                }
            }
            if (t + 1 < tiles) finish(t + 1);
        }
    }
    products_done<S>();
    if (j >= a.Tk) return;
    S* kr = a.dk ? (S*)a.dk + b * a.dks.item + (int64_t)j * a.dks.frame + hk * a.dks.head : nullptr;
    S* vr = a.dv ? (S*)a.dv + b * a.dvs.item + (int64_t)j * a.dvs.frame + hk * a.dvs.head : nullptr;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int at = 32 * d + 8 * n + 4 * half;
            if (kr)
                store4<S>(kr, at, a.D, dk[d][4 * n] * a.scale, dk[d][4 * n + 1] * a.scale, dk[d][4 * n + 2] * a.scale,
                          dk[d][4 * n + 3] * a.scale);
            if (vr) store4<S>(vr, at, a.D, dv[d][4 * n], dv[d][4 * n + 1], dv[d][4 * n + 2], dv[d][4 * n + 3]);
        }
    }
}

// ---------------------------------------------------------------------------
static int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

static int64_t query_blocks(const AttnShape& s) { return (s.Tq + kBwdOwned - 1) / kBwdOwned; }

// delta, then the sums by distance: of the workgroups, and in all.
static int64_t delta_bytes(const AttnShape& s) { return round16(s.B * s.H * s.Tq * (int64_t)sizeof(float)); }
static int64_t dist_bytes(const AttnShape& s) {
    return round16(s.H * s.B * query_blocks(s) * (2 * s.reach + 1) * (int64_t)sizeof(float));
}

size_t dwattn_bwd_workspace(const AttnShape& s) {
    const int64_t total = s.reach ? s.H * (2 * s.reach + 1) * (int64_t)sizeof(double) : 0;
    return (size_t)(delta_bytes(s) + (s.reach ? dist_bytes(s) : 0) + total);
}

template <typename S, int DP>
static hipError_t launch_bwd(const AttnBwd& a, hipStream_t stream) {
    constexpr int kRows = kBwdRows<S, DP>;
    const int nbias = a.table ? 2 * a.R + 1 + 2 * kBiasMargin : 0;
    if (a.nqb > 0) {
        const int lds = 4 * Tile<S, DP>::bytes(kRows) + (nbias + 3) / 4 * 16 +
                        (a.dist ? 4 * kTile * kDiag * 4 + 4 * nbias * 4 : 0);
        const bool dma = dma_fits<S>(a.k, a.ks, a.D) && dma_fits<S>(a.v, a.vs, a.D);
        hipLaunchKernelGGL((dma ? attn_dq_kernel<S, DP, true> : attn_dq_kernel<S, DP, false>),
                           dim3((uint32_t)(a.B * a.H) * a.nqb), dim3(kAttnThreads), lds, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.nkb > 0 && (a.dk || a.dv)) {
        const int lds = 4 * Tile<S, DP>::bytes(kRows) + 4 * kRows * 4 + nbias * 4;
        const AttnStride rows = {(int64_t)a.Tq * a.H * a.D, (int64_t)a.H * a.D, a.D};
        const bool dma = dma_fits<S>(a.q, a.qs, a.D) && dma_fits<S>(a.dout, rows, a.D);
        hipLaunchKernelGGL((dma ? attn_dkv_kernel<S, DP, true> : attn_dkv_kernel<S, DP, false>),
                           dim3((uint32_t)(a.B * a.Hkv) * a.nkb), dim3(kAttnThreads), lds, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_dwattn_bwd(const AttnPtrs& p, const AttnShape& s, const void* out, const float* lse, const void* dout,
                             void* dq, void* dk, void* dv, float* dtable, void* workspace, bool bf16,
                             hipStream_t stream) {
    AttnBwd a;
    (AttnArgs&)a = attn_args(p, s);
    a.out = out, a.lse = lse, a.dout = dout;
    a.dq = dq, a.dk = dk, a.dv = dv;
    a.dqs = s.dq, a.dks = s.dk, a.dvs = s.dv;
    a.nqb = (int32_t)query_blocks(s);
    a.nkb = (int32_t)((s.Tk + kBwdOwned - 1) / kBwdOwned);
    char* at = (char*)workspace;
    a.delta = (float*)at;
    at += delta_bytes(s);
    a.dist = dtable ? (float*)at : nullptr;
    double* total = (double*)(at + dist_bytes(s));
    if (s.B > 0) {
        const hipError_t e = with_head_width(s.D, [&](auto dp) {
            return bf16 ? launch_bwd<uint16_t, dp.value>(a, stream) : launch_bwd<float, dp.value>(a, stream);
        });
        if (e != hipSuccess) return e;
    }
    if (!dtable) return hipSuccess;
    const int32_t n = 2 * a.R + 1;
    hipLaunchKernelGGL(attn_dbias_rows, dim3((n + kDistCols - 1) / kDistCols, a.H), dim3(kDistCols * kDistRows), 0, stream,
                       a.dist, total, n, (int32_t)(s.B * a.nqb));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attn_dtable, dim3((a.NB + 3) / 4, a.H), dim3(kAttnThreads), 0, stream, total, p.buckets, dtable, n,
                       a.NB, a.H);
    return hipGetLastError();
}

}  // namespace dw
