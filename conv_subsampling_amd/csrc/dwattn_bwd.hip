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
// As in the forward, a workgroup's four waves own 128 frames (OW = 4), or where
// those make too few workgroups 64 or 32, the waves that share frames dividing
// the streamed tiles and adding their sums in LDS.  attn_dtable then adds the
// sums by distance over the workgroups and into buckets, in fp64.
//
// Seven products instead of the five that a pass with atomics would take: the
// two done twice keep the sums' order the same in every call.
// Measured, kernels in a row under the profiler, bf16 [16,750,8x128], lengths 750
// to 398 (56 GFLOP as five products): dq with the sums by distance 110 us, dk
// and dv 100 us, the table 6.6 us.  The matrix units are busy for a sixth of
// that; the rest is a run over one tile, which nothing overlaps, and the
// arithmetic between the products.  With a reach over 191 a compute unit holds
// one of dq's workgroups and not two (200: 123 us).
// float [3,333,4x50]: dq 27 to 31 us, dk and dv 41 to 45, the table 5, on so few
// workgroups that most compute units have none.
#include "attn.h"

namespace dw {

struct AttnBwd : AttnArgs {
    const void *out, *dout;  // [B][Tq][H][D]
    const float* lse;        // [B][H][Tq]
    float* stat;             // [B][H][3][Tq]: lse in units of log2 (inf where there are no keys), delta, one over the sum where lse lacks it (else 0)
    void *dq, *dk, *dv;
    AttnStride dqs, dks, dvs;
    float* dist;  // [H][B * nqb][2 R + 1] sums of dS by distance; NULL: not wanted
    int32_t nqb, nkb;
};

// exp(S - lse) of a query that has keys; lse = -inf marks one that has none,
// whose weights are zero.
__device__ __forceinline__ float lse_or_inf(float lse) {
    if (lse == -__builtin_inff()) return __builtin_inff();
    const float most = 3.0e38f;  // as the biases are held
    return fabsf(lse) < __builtin_inff() ? __builtin_amdgcn_fmed3f(lse * kLog2e, -most, most) : lse;
}

// lse = maximum + log(sum) holds the logarithm to 2^-24 of the whole.  Beyond
// this magnitude (in units of log2; a weight is off by 1e-4 there, and a row of
// nothing but masks of -1e9 or of the type's lowest value absorbs the logarithm
// altogether) the maximum stands in its place, and one over the sum apart.
constexpr float kHeavy = 1024.0f;
__device__ __forceinline__ bool heavy(float lse2) { return fabsf(lse2) > kHeavy && fabsf(lse2) < __builtin_inff(); }

// The maximum of a lane's row of scores (in units of log2, as the kernels
// compute them) and one over the sum of its weights over it, by one wave from
// memory: keys first to last are those that any of its 32 queries may see, from
// mine0 on `mine` of them are the lane's own.  Rare, so short and not fast.
template <typename S, int DP>
__device__ __forceinline__ void heavy_row(const AttnArgs& a, const AttnItem& item, int b, int h, int i, const Frag<S> (&q)[DP / 16],
                                        int first, int last, int mine0, uint32_t mine, float& top, float& weight) {
    const int lane = threadIdx.x % 64, half = lane / 32, hk = h / (a.H / a.Hkv);
    const S* keys = (const S*)a.k + b * a.ks.item + hk * a.ks.head;
    float sum = 0.0f;
    top = -__builtin_inff();
    for (int j = first; j <= last; j += kTile) {
        const int at = j + lane % 32;
        f32x16 s = {}, s_small = {};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c)
            mma_apart(to_frag<S>(load_group<S, true>(keys + (int64_t)min(at, last) * a.ks.frame, 16 * c + 8 * half,
                                                     at <= last ? a.D : 0)), q[c], s, s_small);
        if constexpr (sizeof(S) == 4) {
            products_done(s, s_small);
            s += s_small;
        } else {
            products_done(s);
        }
        float m = top;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int key = j + acc_row(r, half);
            const int x = min(max(key - i - item.pos32, -a.R), a.R) + a.R + kBiasMargin;
            const float bias = a.table ? BiasFill<S>::value(a, h, BiasFill<S>::map_at(a, x)) : 0.0f;
            s[r] = (uint32_t)(key - mine0) < mine ? fmaf(s[r], a.scale2, bias) : -__builtin_inff();
            m = fmaxf(m, s[r]);
        }
        m = fmaxf(m, swap_halves(m));
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        sum *= exp2_fast(top - ref);
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += exp2_fast(s[r] - ref);
        top = m;
    }
    sum += swap_halves(sum);
    weight = 1.0f / sum;
    if (sum == 0.0f) top = __builtin_inff(), weight = 1.0f;  // no keys, whatever lse says
}


// from[at] of every lane into LDS at to[at], zero for at >= count; the lanes of
// a wave have 64 neighbouring `at`.
__device__ __forceinline__ void load_lds_floats(const float* from, int count, int at, float* to) {
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)to +
                         __builtin_amdgcn_readfirstlane(at / 64) * 256;
    load_to_lds<4>(from, count > 0 ? (uint32_t)count * 4 : 0, at * 4, lds);
}

// Orders a wave's LDS accesses before and after it: lanes read what other
// lanes of their wave wrote.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename S, int DP, int OW>
struct BwdShape {
    static constexpr int ROWS = bwd_rows(DP, sizeof(S), OW), kBuffers = bwd_buffers(DP, sizeof(S), OW);
    template <bool DMA>
    using Tiles = TilePair<S, DP, ROWS, kBuffers, DMA && kBuffers == 2>;
};

// Adds acc over the waves that share owned frames (wave = part * OW + owner);
// run n of `out` is then the sum of run part + n * KW of 32 head elements.
template <int OW, int ND>
__device__ __forceinline__ void add_waves(char* smem, f32x16 (&acc)[ND], int lane, int wave) {
    constexpr int KW = 4 / OW;
    if constexpr (KW > 1) {
        float* all = (float*)smem;  // [4][ND * 16][64]
        __syncthreads();
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) all[((wave * ND + d) * 16 + r) * 64 + lane] = acc[d][r];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (ND + KW - 1) / KW; ++n) {
            const int d = wave / OW + n * KW;
            if (d >= ND) break;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) v += all[(((w * OW + wave % OW) * ND + d) * 16 + r) * 64 + lane];
                acc[n][r] = v;
            }
        }
    }
}

// The runs of 32 head elements that this wave has after add_waves, times scale.
template <typename S, int OW, int ND>
__device__ __forceinline__ void store_runs(S* row, const f32x16 (&acc)[ND], int D, float scale, int half, int wave) {
    constexpr int KW = 4 / OW;
#pragma unroll
    for (int n = 0; n < (ND + KW - 1) / KW; ++n) {
        const int d = wave / OW + n * KW;
        if (d >= ND) break;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            store4<S>(row, 32 * d + 8 * g + 4 * half, D, acc[n][4 * g] * scale, acc[n][4 * g + 1] * scale,
                      acc[n][4 * g + 2] * scale, acc[n][4 * g + 3] * scale);
    }
}

template <typename S, int DP, int OW, bool DMA>
__global__ __launch_bounds__(kAttnThreads, ((sizeof(S) == 4 && !DMA) || (DP > 64 && (sizeof(S) == 4 || !DMA)) ? 1 : 2)) void attn_dq_kernel(const AttnBwd a) {
    typedef BwdShape<S, DP, OW> Shape;
    typedef typename Shape::template Tiles<DMA> Tiles;
    typedef Tile<S, DP> T;
    constexpr int KW = 4 / OW, BN = Shape::ROWS, KT = BN / kTile / KW, NC = DP / 16, ND = DP / 32;
    static_assert(KW == 1 || 4 * ND * 16 * 64 * 4 <= Tiles::kAllBytes, "the tiles' room holds the waves' sums");
    extern __shared__ __align__(16) char smem[];
    float* bias = (float*)(smem + Tiles::kAllBytes);
    const int nbias = 2 * a.R + 1 + 2 * kBiasMargin;
    const int lane = threadIdx.x % 64, wave = wave_of_block(), half = lane / 32;
    float* square = bias + (nbias + 3) / 4 * 4 + wave * kTile * kDiag;                      // a tile of dS
    float* sums = bias + (nbias + 3) / 4 * 4 + 4 * kTile * kDiag + wave * nbias;            // by distance, of this wave

    const AttnPlace place(blockIdx.x, a.nqb, a.B * a.H, a.left == kNoLimit && a.right != kNoLimit);
    const int qb = place.block, h = place.pair % a.H, b = item_of_rank(a, place.pair / a.H);
    const AttnItem item(a, b);
    const int wk = wave / OW, i0 = qb * OW * kTile, iw = i0 + wave % OW * kTile, i = iw + lane % 32;
    const bool live = i < item.nq;
    const BiasFill<S> filler(a);
    if (a.dist) {
        for (int x = lane; x < nbias; x += 64) sums[x] = 0.0f;
        for (int x = lane; x < kTile * kDiag; x += 64) square[x] = 0.0f;
    }

    Frag<S> q[NC], g[NC];
    float delta = 0.0f, lse2 = __builtin_inff(), weight = 1.0f;
    const int mine0 = item.first_key(a, i), mine1 = item.last_key(a, i);
    const uint32_t mine = live && mine1 >= mine0 ? mine1 - mine0 + 1 : 0;
    const int iwl = min(iw + kTile, item.nq) - 1;
    const int some0 = item.first_key(a, iw), some1 = iw < item.nq ? item.last_key(a, iwl) : -1;
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
        float apart = 0.0f;
        if (__any(heavy(lse2))) {
            float top, w;
            heavy_row<S, DP>(a, item, b, h, i, q, some0, some1, mine0, mine, top, w);
            if (heavy(lse2)) lse2 = top, weight = apart = w;
        }
        if (half == 0 && wk == 0 && i < a.Tq) {
            const int64_t head = ((int64_t)b * a.H + h) * 3 * a.Tq;
            a.stat[head + i] = lse2;
            a.stat[head + a.Tq + i] = delta;
            a.stat[head + 2 * (int64_t)a.Tq + i] = apart;
        }
        delta *= weight;
    }
    if (!a.dq && !a.dist) return;
    int j0 = 0, j1 = 0;
    if (i0 < item.nq) {
        j0 = item.first_key(a, i0);
        j1 = item.last_key(a, min(i0 + OW * kTile, item.nq) - 1) + 1;
    }
    const int all0 = item.first_key(a, iwl), all1 = iw + kTile <= item.nq ? item.last_key(a, iw) : -1;

    const int hk = h / (a.H / a.Hkv);
    Tiles kv(smem, (const S*)a.k + b * a.ks.item + hk * a.ks.head + (int64_t)j0 * a.ks.frame, a.ks.frame,
             (const S*)a.v + b * a.vs.item + hk * a.vs.head + (int64_t)j0 * a.vs.frame, a.vs.frame, a.D, j1 - j0);
    const int tiles = j1 > j0 ? (j1 - j0 + BN - 1) / BN : 0;
    if (tiles) kv.start(0);
    filler.fill(a, h, bias);
    if (tiles && Shape::kBuffers == 2) kv.finish(0);
#pragma unroll
    for (int c = 0; c < NC; ++c) arrived(q[c]), arrived(g[c]);
    asm volatile("" : "+v"(lse2), "+v"(delta));
    f32x16 acc[ND] = {};
    float low = 0.0f, high = 0.0f;  // sums of dS past the map's reach
    for (int t = 0; t < tiles; ++t) {
        kv.enter(t, t + 1 < tiles);
        const S* ktile = kv.x_of(t);
        const S* vtile = kv.y_of(t);
        const int jt = j0 + t * BN;
#pragma unroll
        for (int u = 0; u < KT; ++u) {
            const int row0 = (wk * KT + u) * kTile, j = jt + row0;
            if (j > some1 || j + kTile <= some0) continue;
            f32x16 s = {}, ds = {}, s_small = {}, ds_small = {};
            // float's widest heads take one sum after the other: four at once leave no registers ([8,375,8x128] 124 us
            // so and 137 us side by side, [16,375,8x64] 109 and 105)
            constexpr bool kInTurn = sizeof(S) == 4 && DP > 64;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                mma_apart(T::rows(ktile, row0, c, lane), q[c], s, s_small);
                if (!kInTurn) mma_apart(T::rows(vtile, row0, c, lane), g[c], ds, ds_small);
            }
            if constexpr (sizeof(S) == 4) {
                products_done(s, s_small);
                s += s_small;
                if constexpr (kInTurn) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) mma_apart(T::rows(vtile, row0, c, lane), g[c], ds, ds_small);
                }
                products_done(ds, ds_small);
                ds += ds_small;
            } else {
                products_done(s, ds);
            }
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
            for (int r = 0; r < 16; ++r) ds[r] = s[r] * fmaf(ds[r], weight, -delta);
            if (j < all0 || j + kTile - 1 > all1) {
                const uint32_t at = j + 4 * half - mine0;
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = at + acc_row(r, 0) < mine ? ds[r] : 0.0f;
            }
            if (a.dist) {
                if (span == Span::kNear) {
                    // The 63 diagonals of the tile: query i writes its 32 keys
                    // from place 31 - i of its row of the square, so that a
                    // column holds one distance, and the places that no tile
                    // writes stay zero.
                    float* to = square + (lane % 32) * (kDiag - 1) + 31 + 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) to[acc_row(r, 0)] = ds[r];
                    wave_lds_fence();
                    float t[4] = {};
#pragma unroll
                    for (int n = 0; n < kTile; ++n) t[n % 4] += square[n * kDiag + lane];
                    if (lane < kDiag - 1) sums[base + a.R + kBiasMargin - 31 + lane] += (t[0] + t[1]) + (t[2] + t[3]);
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
        kv.leave(t, t + 1 < tiles);
    }
    products_done(acc);
    if (a.dq) {
        add_waves<OW, ND>(smem, acc, lane, wave);
        if (i < a.Tq)
            store_runs<S, OW, ND>((S*)a.dq + b * a.dqs.item + (int64_t)i * a.dqs.frame + h * a.dqs.head, acc, a.D, a.scale,
                                  half, wave);
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

// 5 to 6 us, two rounds of dependent loads and a launch.
// dtable[bucket][h]: a workgroup lists the distances of its bucket and adds
// their sums over the parts (items and query blocks), in an order that the
// sizes and the map fix: each thread every 256th, then lanes, then waves.
__global__ __launch_bounds__(kAttnThreads) void attn_dtable(const float* __restrict__ dist,
                                                           const int32_t* __restrict__ map, float* __restrict__ dtable,
                                                           int32_t n, int32_t parts, int32_t NB, int32_t H) {
    constexpr int kMost = 2 * kAttnMaxReach + 1, kSteps = (kMost + kAttnThreads - 1) / kAttnThreads;
    __shared__ int16_t list[kMost];
    __shared__ int found[kSteps][4];
    __shared__ double waves[4];
    const int bucket = blockIdx.x / H, h = blockIdx.x % H, lane = threadIdx.x % 64, wave = wave_of_block();
    uint64_t mask[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int x = threadIdx.x + k * kAttnThreads;
        int m = x < n ? map[x] : -1;
        m = x >= n ? -1 : m < 0 ? 0 : m >= NB ? NB - 1 : m;
        mask[k] = __ballot(m == bucket);
        if (lane == 0) found[k][wave] = __popcll(mask[k]);
    }
    __syncthreads();
    int count = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w == wave && mask[k] >> lane & 1)
                list[count + __popcll(mask[k] & ((1ull << lane) - 1))] = (int16_t)(threadIdx.x + k * kAttnThreads);
            count += found[k][w];
        }
    }
    __syncthreads();
    double s = 0.0;
    const float* from = dist + (int64_t)h * parts * n;
    const uint32_t each = count, all = each * (uint32_t)parts;
#pragma unroll 8
    for (uint32_t at = threadIdx.x; at < all; at += kAttnThreads) {
        const uint32_t part = at / each;
        s += from[(int64_t)part * n + list[at - part * each]];
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m);
    if (lane == 0) waves[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) dtable[(int64_t)bucket * H + h] = (float)(waves[0] + waves[1] + waves[2] + waves[3]);
}

template <typename S, int DP>
constexpr bool kValuesInLds = bwd_values_in_lds(DP, sizeof(S));
template <typename S, int DP>
constexpr int kValuesBytes = kValuesInLds<S, DP> ? 4 * (DP / 16) * 64 * 16 : 0;

template <typename S, int DP, int OW, bool DMA>
__global__ __launch_bounds__(kAttnThreads, (sizeof(S) == 4 || (!DMA && DP > 32) ? 1 : 2)) void attn_dkv_kernel(const AttnBwd a) {
    typedef BwdShape<S, DP, OW> Shape;
    typedef typename Shape::template Tiles<DMA> Tiles;
    typedef Tile<S, DP> T;
    constexpr int KW = 4 / OW, BQ = Shape::ROWS, QT = BQ / kTile / KW, NC = DP / 16, ND = DP / 32;
    extern __shared__ __align__(16) char smem[];
    u32x4* values = (u32x4*)(smem + Tiles::kAllBytes);
    float* stats = (float*)(smem + Tiles::kAllBytes + kValuesBytes<S, DP>);  // of two tiles: [2][3][BQ], as a.stat
    float* bias = stats + 6 * BQ;
    const int nbias = 2 * a.R + 1 + 2 * kBiasMargin;
    const int lane = threadIdx.x % 64, wave = wave_of_block(), half = lane / 32;

    const AttnPlace place(blockIdx.x, a.nkb, a.B * a.Hkv, a.right == kNoLimit && a.left != kNoLimit);
    const int kb = place.block, hk = place.pair % a.Hkv, b = item_of_rank(a, place.pair / a.Hkv), group = a.H / a.Hkv;
    const AttnItem item(a, b);
    const int wk = wave / OW, j0 = kb * OW * kTile, jw = j0 + wave % OW * kTile, j = jw + lane % 32;
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
        if constexpr (kValuesInLds<S, DP>) {
#pragma unroll
            for (int c = 0; c < NC; ++c) values[(wave * NC + c) * 64 + lane] = v[c].r;
        }
    }
    auto value = [&](int c) {
        if constexpr (kValuesInLds<S, DP>)
            return Frag<S>{values[(wave * NC + c) * 64 + lane]};
        else
            return v[c];
    };
    const int mine0 = item.first_query(a, j), mine1 = item.last_query(a, j);
    const uint32_t mine = live && mine1 >= mine0 ? mine1 - mine0 + 1 : 0;
    int i0 = 0, i1 = 0;
    if (j0 < item.nk) {
        i0 = item.first_query(a, j0);
        i1 = item.last_query(a, min(j0 + OW * kTile, item.nk) - 1) + 1;
    }
    const int jwl = min(jw + kTile, item.nk) - 1;
    const int some0 = item.first_query(a, jw), some1 = jw < item.nk ? item.last_query(a, jwl) : -1;
    const int all0 = item.first_query(a, jwl), all1 = jw + kTile <= item.nk ? item.last_query(a, jw) : -1;

    f32x16 dk[ND] = {}, dv[ND] = {};
    for (int n = 0; n < group; ++n) {
        const int h = hk * group + n;
        __syncthreads();  // the head before is done with the tiles and its bias
        const BiasFill<S> filler(a);
        const int64_t gstride = (int64_t)a.H * a.D;
        Tiles qg(smem, (const S*)a.q + b * a.qs.item + h * a.qs.head + (int64_t)i0 * a.qs.frame, a.qs.frame,
                 (const S*)a.dout + (((int64_t)b * a.Tq + i0) * a.H + h) * a.D, gstride, a.D, i1 - i0);
        // the tile's statistics, one float a lane: the first waves take lse, the next delta and so on
        const float* stat_rows = a.stat + ((int64_t)b * a.H + h) * 3 * a.Tq + i0;
        auto start_stats = [&](int t) {
            constexpr int kEach = BQ < 64 ? 64 : BQ;
            const int at = threadIdx.x % kEach;
#pragma unroll
            for (int row = 0; row < 3; row += kAttnThreads / kEach) {
                const int which = row + __builtin_amdgcn_readfirstlane(threadIdx.x / kEach);
                if (which < 3 && at < BQ)
                    load_lds_floats(stat_rows + (int64_t)which * a.Tq + t * BQ, i1 - i0 - t * BQ, at,
                                    stats + ((t & 1) * 3 + which) * BQ);
            }
        };
        const int tiles = i1 > i0 ? (i1 - i0 + BQ - 1) / BQ : 0;
        if (tiles) {
            qg.start(0);
            start_stats(0);
        }
        filler.fill(a, h, bias);
        if (tiles && Shape::kBuffers == 2) qg.finish(0);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            arrived(k[c]);
            if (!kValuesInLds<S, DP>) arrived(v[c]);
        }
        for (int t = 0; t < tiles; ++t) {
            qg.enter(t, t + 1 < tiles);
            if (t + 1 < tiles) start_stats(t + 1);
            const S* qtile = qg.x_of(t);
            const S* gtile = qg.y_of(t);
            const float* stat = stats + (t & 1) * 3 * BQ;
            const int it = i0 + t * BQ;
#pragma unroll
            for (int u = 0; u < QT; ++u) {
                const int row0 = (wk * QT + u) * kTile, i = it + row0;
                if (i > some1 || i + kTile <= some0) continue;
                f32x16 s = {}, ds = {};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    s = mma(T::rows(qtile, row0, c, lane), k[c], s);
                    ds = mma(T::rows(gtile, row0, c, lane), value(c), ds);
                    if (kValuesInLds<S, DP> && c % 2) __builtin_amdgcn_sched_barrier(0);
                }
                products_done(s, ds);
                // distance of the tile's first key and first query; along the registers it falls
                const int base = jw - i - item.pos32;
                const Span span = span_of(base, a.R);
                f32x4 row[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) row[r] = *reinterpret_cast<const f32x4*>(stat + row0 + 8 * r + 4 * half);
                auto lse2 = [&](int r) { return row[r / 4][r % 4]; };
                if (a.table && span == Span::kNear) {
                    const float* p = bias + (base + a.R + kBiasMargin - 4 * half + lane % 32);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = exp2_fast(fmaf(s[r], a.scale2, p[-acc_row(r, 0)]) - lse2(r));
                } else {
                    const float flat = a.table ? bias[span == Span::kLow ? 0 : nbias - 1] : 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = exp2_fast(fmaf(s[r], a.scale2, flat) - lse2(r));
                }
                if (__any(stat[2 * BQ + row0 + lane % 32] != 0.0f)) {  // scores reach a maximum only up to their rounding
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        row[r] = *reinterpret_cast<const f32x4*>(stat + 2 * BQ + row0 + 8 * r + 4 * half);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = row[r / 4][r % 4] != 0.0f ? fminf(s[r], 1.0f) * row[r / 4][r % 4] : s[r];
                }
                if (i < all0 || i + kTile - 1 > all1) {
                    const uint32_t at = i + 4 * half - mine0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = at + acc_row(r, 0) < mine ? s[r] : 0.0f;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) row[r] = *reinterpret_cast<const f32x4*>(stat + BQ + row0 + 8 * r + 4 * half);
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = s[r] * (ds[r] - row[r / 4][r % 4]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const Frag<S> p = to_frag<S>(s, c), g = to_frag<S>(ds, c);
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        dv[d] = mma(T::columns(gtile, row0 + 16 * c, d, lane), p, dv[d]);
                        dk[d] = mma(T::columns(qtile, row0 + 16 * c, d, lane), g, dk[d]);
                        if (kValuesInLds<S, DP> && d % 2) __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            qg.leave(t, t + 1 < tiles);
        }
    }
    products_done(dk);
    products_done(dv);
    const bool out = j < a.Tk;
    if (a.dk) {
        add_waves<OW, ND>(smem, dk, lane, wave);
        if (out)
            store_runs<S, OW, ND>((S*)a.dk + b * a.dks.item + (int64_t)j * a.dks.frame + hk * a.dks.head, dk, a.D, a.scale,
                                  half, wave);
    }
    if (a.dv) {
        add_waves<OW, ND>(smem, dv, lane, wave);
        if (out)
            store_runs<S, OW, ND>((S*)a.dv + b * a.dvs.item + (int64_t)j * a.dvs.frame + hk * a.dvs.head, dv, a.D, 1.0f,
                                  half, wave);
    }
}

// ---------------------------------------------------------------------------
// Launch plan
// ---------------------------------------------------------------------------
static int64_t blocks_of(int64_t frames, int ow) { return (frames + ow * kTile - 1) / (ow * kTile); }

static int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Three statistics of each query, then the workgroups' sums by distance.
static int64_t stat_bytes(const AttnShape& s) { return round16(s.B * s.H * s.Tq * 3 * (int64_t)sizeof(float)); }

bool dwattn_bwd_fits(const AttnShape& s, int elem_bytes) {
    const int64_t nqb = blocks_of(s.Tq, owned(s, elem_bytes, true)), nkb = blocks_of(s.Tk, owned(s, elem_bytes, false));
    if (!grid_of_256_fits(s.B * s.H * nqb) || !grid_of_256_fits(s.B * s.Hkv * nkb)) return false;
    // the workgroups' sums by distance of one head, counted in 31 bits, and a workgroup for each entry of the table
    return s.reach == 0 || (product_below(kMaxExtent, {s.B, (s.Tq + kTile - 1) / kTile, 2 * s.reach + 1}) &&
                            grid_of_256_fits(s.buckets * s.H));
}

// Enough for any context: one limited on one side may own fewer queries a workgroup.
size_t dwattn_bwd_workspace(const AttnShape& s, int elem_bytes) {
    AttnShape all = s, causal = s;
    all.left = all.right = causal.left = kNoLimit;
    causal.right = 0;
    int64_t blocks = 0;
    for (const AttnShape& c : {all, causal}) {
        const int64_t n = blocks_of(s.Tq, owned(c, elem_bytes, true));
        blocks = n > blocks ? n : blocks;
    }
    return (size_t)(stat_bytes(s) + (s.reach ? s.H * s.B * blocks * (2 * s.reach + 1) * (int64_t)sizeof(float) : 0));
}

template <typename S, int DP, int OW>
static hipError_t launch_dq(const AttnBwd& a, int lds, hipStream_t stream) {
    constexpr bool kDirect = BwdShape<S, DP, OW>::kBuffers == 2;
    const bool fits = direct_fits(a.k, a.ks, a.D, sizeof(S)) && direct_fits(a.v, a.vs, a.D, sizeof(S));
    hipLaunchKernelGGL((bwd_form(OW, a.D, sizeof(S), fits).direct ? attn_dq_kernel<S, DP, OW, kDirect>
                                                                  : attn_dq_kernel<S, DP, OW, false>),
                       dim3((uint32_t)(a.B * a.H) * a.nqb), dim3(kAttnThreads), lds, stream, a);
    return hipGetLastError();
}

template <typename S, int DP, int OW>
static hipError_t launch_dkv(const AttnBwd& a, int lds, hipStream_t stream) {
    constexpr bool kDirect = BwdShape<S, DP, OW>::kBuffers == 2;
    const AttnStride rows = {(int64_t)a.Tq * a.H * a.D, (int64_t)a.H * a.D, a.D};
    const bool fits = direct_fits(a.q, a.qs, a.D, sizeof(S)) && direct_fits(a.dout, rows, a.D, sizeof(S));
    hipLaunchKernelGGL((bwd_form(OW, a.D, sizeof(S), fits).direct ? attn_dkv_kernel<S, DP, OW, kDirect>
                                                                  : attn_dkv_kernel<S, DP, OW, false>),
                       dim3((uint32_t)(a.B * a.Hkv) * a.nkb), dim3(kAttnThreads), lds, stream, a);
    return hipGetLastError();
}

template <typename S, int DP>
static hipError_t launch_bwd(const AttnBwd& a, const AttnShape& s, int oq, int ok, hipStream_t stream) {
    if (a.nqb > 0 && a.H > 0) {
        const int lds = bwd_lds(s, sizeof(S), oq, true);
        // Tiles of 128 float keys of the widest heads leave no room for the square at all.
        constexpr int kLeast = bwd_tile_bytes(DP, sizeof(S), 1) + kSquareBytes > kLdsBytes ? 2 : 1;
        const hipError_t e = oq == 4   ? launch_dq<S, DP, 4>(a, lds, stream)
                             : oq == 2 ? launch_dq<S, DP, 2>(a, lds, stream)
                                       : launch_dq<S, DP, kLeast>(a, lds, stream);
        if (e != hipSuccess) return e;
    }
    if (a.nkb > 0 && (a.dk || a.dv)) {
        const int lds = bwd_lds(s, sizeof(S), ok, false);
        return ok == 4   ? launch_dkv<S, DP, 4>(a, lds, stream)
               : ok == 2 ? launch_dkv<S, DP, 2>(a, lds, stream)
                         : launch_dkv<S, DP, 1>(a, lds, stream);
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
    const int oq = owned(s, bf16 ? 2 : 4, true), ok = owned(s, bf16 ? 2 : 4, false);
    a.nqb = (int32_t)blocks_of(s.Tq, oq);
    a.nkb = (int32_t)blocks_of(s.Tk, ok);
    a.stat = (float*)workspace;
    a.dist = dtable ? (float*)((char*)workspace + stat_bytes(s)) : nullptr;
    if (s.B > 0) {
        const hipError_t e = with_head_width(s.D, [&](auto dp) {
            return bf16 ? launch_bwd<uint16_t, dp.value>(a, s, oq, ok, stream)
                        : launch_bwd<float, dp.value>(a, s, oq, ok, stream);
        });
        if (e != hipSuccess) return e;
    }
    if (!dtable || s.H == 0) return hipSuccess;
    hipLaunchKernelGGL(attn_dtable, dim3(a.NB * a.H), dim3(kAttnThreads), 0, stream, a.dist, p.buckets, dtable, 2 * a.R + 1,
                       (int32_t)(s.B * a.nqb), a.NB, a.H);
    return hipGetLastError();
}

}  // namespace dw
