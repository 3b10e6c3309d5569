// SiLU and GLU of the conv module, and a checkpoint of their input in 8 bits
// from which the backward pass runs.
//
// x = q * 2^(code - 127) with |q| <= 127 in groups of 32 columns.  The scale is a
// power of two, so both directions are exact but for the one rounding of q, the
// kept value is itself a bf16, and a group costs one byte.  A lane takes 8
// columns; the 4 lanes of a quad hold a group and find its largest magnitude by
// two lane permutations.
//
// Bound by memory.  With lengths of half to all of the frames: [16,750,2 x 1024]
// bf16 GLU forward with the checkpoint 19 us and gradients 18 us for 87 MB each (37
// together, 4.7 TB/s; a large copy reaches 5.1); [16,750,4096] SiLU gradients and
// activation 62 us for 311 MB (5.0 TB/s).  19 to 33 vector operations an element
// take half to two thirds of that time in issue slots, beside it.
#include "launch.h"
#include "rowops.h"

namespace dw {

constexpr int kActThreads = 256;
constexpr int kActGroup = 32;                    // columns that share a scale
constexpr int kActLanes = kActGroup / kGroup;    // lanes that hold them

// n / d for n < 2^31 by one multiplication: (mulhi(n, m) + n) >> l with
// 2^(l-1) < d <= 2^l and m = floor(2^32 (2^l - d) / d) + 1.
struct Divisor {
    uint32_t d, m, l;
};

static Divisor divisor(uint32_t d) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    return {d, (uint32_t)(((((uint64_t)1 << l) - d) << 32) / d + 1), l};
}

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& by) { return (__umulhi(n, by.m) + n) >> by.l; }

struct ActArgs {
    const void *x, *dy;
    const int32_t* lengths;
    void *y, *dx;
    int8_t* kept;
    uint8_t* codes;
    uint64_t units;   // lanes' pieces in all
    Divisor per_row;  // of a row, a multiple of 4
    Divisor T;
    int32_t C;
};

// open = 1 / (1 + exp(-v)) and shut = 1 - open, without cancellation.  The smaller of
// them is kept below 2^-126 too, from where the activation's input lifts it back into the range.  float:
// exp(-|v|), within a few units in the last place.  bf16: the exponent is one rounded product (off by |v|
// 2^-24 of the result), and all is taken 2^24 higher.
struct ActGate {
    float open, shut;
};

template <typename S>
__device__ __forceinline__ ActGate act_gate(float v) {
    if constexpr (sizeof(S) == 4) {
        const float e = expf(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + e);
        return {v < 0.0f ? e * r : r, v < 0.0f ? r : e * r};
    } else {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(fabsf(v), -1.44269504f, 24.0f));
        const float r = __builtin_amdgcn_rcpf(0x1p24f + e), less = e * r, more = r * 0x1p24f;
        return {v < 0.0f ? less : more, v < 0.0f ? more : less};
    }
}

typedef u32x2 bytes8 __attribute__((aligned(1)));

// The largest of the quad's four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xf, 0xf, true));  // quad_perm [1,0,3,2]
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xf, 0xf, true));  // quad_perm [2,3,0,1]
}

// Codes of 1 to 248 (magnitudes past 127 * 2^121 are kept as that: 128 times the
// scale would be infinite): with top = f * 2^k, 1 <= f < 2, the scale is 2^(k - 6) where
// f <= 127/64 and twice that elsewhere; adding 2^23 - 127/128 * 2^23 - 1 to the
// bits carries into the exponent exactly there.
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
    if (top >= 0x7f800000u) return 255u;
    const int e = (int)((top + 0x1ffffu) >> 23) - 6;
    return e < 1 ? 1u : e > 248 ? 248u : (uint32_t)e;
}

// Keeps 8 columns (zeros past the row's end) and, by the quad's first lane, the
// code of their group (0 in a row past its length).
template <bool TAIL>
__device__ __forceinline__ void keep_group(const Vf<kGroup>& v, int8_t* row, uint8_t* code_row, int col, int C,
                                           bool live) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) top = max(top, __float_as_uint(v.v[e]) & 0x7fffffffu);
    const uint32_t code = scale_code(quad_max(top));
    const float inverse = __uint_as_float((254u - code) << 23);  // code 255: its values are not used
    u32x2 q = {0u, 0u};
    if (code != 255u) {
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
            q[e / 4] |= ((uint32_t)(int)rintf(__builtin_amdgcn_fmed3f(v.v[e] * inverse, -127.0f, 127.0f)) & 0xffu)
                        << (8 * (e % 4));
    }
    if (col + kGroup <= C) {
        *reinterpret_cast<bytes8*>(row + col) = q;
    } else if (TAIL && col < C) {
#pragma unroll
        for (int e = 0; e < kGroup - 1; ++e)
            if (col + e < C) row[col + e] = (int8_t)(q[e / 4] >> (8 * (e % 4)));
    }
    if (col % kActGroup == 0 && col < C) code_row[col / kActGroup] = live ? (uint8_t)code : 0;
}

struct KeptRaw {
    u32x2 q;
    uint32_t code;
};

template <bool TAIL>
__device__ __forceinline__ KeptRaw load_kept(const int8_t* row, const uint8_t* code_row, int col, int C) {
    KeptRaw r = {{0u, 0u}, 0u};
    if (col < C) r.code = code_row[col / kActGroup];
    if (col + kGroup <= C) {
        r.q = *reinterpret_cast<const bytes8*>(row + col);
    } else if (TAIL && col < C) {
#pragma unroll
        for (int e = 0; e < kGroup - 1; ++e)
            if (col + e < C) r.q[e / 4] |= (uint32_t)(uint8_t)row[col + e] << (8 * (e % 4));
    }
    return r;
}

// Code 255 is the bits of infinity, and infinity times the kept zero a NaN.
__device__ __forceinline__ Vf<kGroup> widen_kept(const KeptRaw& r) {
    const float scale = __uint_as_float(r.code << 23);
    Vf<kGroup> v;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) v.v[e] = (float)(int8_t)(r.q[e / 4] >> (8 * (e % 4))) * scale;
    return v;
}

// One lane's piece of a row: 8 columns of each part.
struct ActPiece {
    uint64_t row;
    int col;   // C for a piece past the last
    bool live;
};

__device__ __forceinline__ ActPiece act_piece(const ActArgs& a, uint64_t unit) {
    ActPiece p = {0, a.C, false};
    if (unit >= a.units) return p;
    if (a.units >> 31) {
        p.row = unit / a.per_row.d;
        p.col = (int)(unit - p.row * a.per_row.d) * kGroup;
    } else {
        const uint32_t row = divide((uint32_t)unit, a.per_row);
        p.row = row;
        p.col = (int)((uint32_t)unit - row * a.per_row.d) * kGroup;
    }
    p.live = true;
    if (a.lengths) {
        const uint64_t b = p.row >> 31 ? p.row / a.T.d : divide((uint32_t)p.row, a.T);
        p.live = (int64_t)(p.row - b * a.T.d) < a.lengths[b];
    }
    return p;
}

template <typename S, bool TAIL, int ACT>
__global__ __launch_bounds__(kActThreads) void act_fwd_kernel(const ActArgs a) {
    constexpr int kParts = ACT == 2 ? 2 : 1, kPieces = ACT == 2 ? 2 : 4;
    const int C = a.C;
    const int64_t W = (int64_t)kParts * C, codes = kParts * (int64_t)((C + kActGroup - 1) / kActGroup);
    const uint64_t first = (uint64_t)blockIdx.x * (kActThreads * kPieces) + threadIdx.x;
    ActPiece p[kPieces];
    RawGroup<S> raw[kPieces][kParts];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        p[j] = act_piece(a, first + j * kActThreads);
#pragma unroll
        for (int h = 0; h < kParts; ++h)
            raw[j][h] = load_group<S, TAIL>((const S*)a.x + p[j].row * W + h * (int64_t)C, p[j].live ? p[j].col : C, C);
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int col = p[j].col;
        Vf<kGroup> v[kParts];
#pragma unroll
        for (int h = 0; h < kParts; ++h) v[h] = widen<S>(raw[j][h]);
        if (a.y) {
            Vf<kGroup> o = v[0];
            if constexpr (ACT != 0) {
#pragma unroll
                for (int e = 0; e < kGroup; ++e) o.v[e] *= act_gate<S>(v[kParts - 1].v[e]).open;
            }
            store_group<S, TAIL>((S*)a.y + p[j].row * C, col, C, o);  // 0 past the length: x reads as 0 there
        }
        if (a.kept) {
#pragma unroll
            for (int h = 0; h < kParts; ++h)
                keep_group<TAIL>(v[h], a.kept + p[j].row * W + h * (int64_t)C,
                                 a.codes + p[j].row * codes + h * (codes / kParts), col, C, p[j].live);
        }
    }
}

template <typename S, bool TAIL, int ACT>
__global__ __launch_bounds__(kActThreads) void act_bwd_kernel(const ActArgs a) {
    constexpr int kParts = ACT == 2 ? 2 : 1, kPieces = ACT == 2 ? 2 : 4;
    const int C = a.C;
    const int64_t W = (int64_t)kParts * C, codes = kParts * (int64_t)((C + kActGroup - 1) / kActGroup);
    const uint64_t first = (uint64_t)blockIdx.x * (kActThreads * kPieces) + threadIdx.x;
    ActPiece p[kPieces];
    KeptRaw raw[kPieces][kParts];
    RawGroup<S> dyr[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        p[j] = act_piece(a, first + j * kActThreads);
        const int from = p[j].live ? p[j].col : C;
#pragma unroll
        for (int h = 0; h < kParts; ++h)
            raw[j][h] = load_kept<TAIL>(a.kept + p[j].row * W + h * (int64_t)C,
                                        a.codes + p[j].row * codes + h * (codes / kParts), from, C);
        dyr[j] = load_group<S, TAIL>((const S*)a.dy + p[j].row * C, a.dx ? from : C, C);
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int col = p[j].col;
        const Vf<kGroup> x = widen_kept(raw[j][0]), dy = widen<S>(dyr[j]);
        Vf<kGroup> y = x, dx = dy;
        if constexpr (ACT == 1) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                const ActGate s = act_gate<S>(x.v[e]);
                y.v[e] = x.v[e] * s.open;
                dx.v[e] = dy.v[e] * (s.open + y.v[e] * s.shut);
            }
        }
        if constexpr (ACT == 2) {
            const Vf<kGroup> gate = widen_kept(raw[j][kParts - 1]);
            Vf<kGroup> db;
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                const ActGate s = act_gate<S>(gate.v[e]);
                y.v[e] = x.v[e] * s.open;
                dx.v[e] = dy.v[e] * s.open;
                db.v[e] = dx.v[e] * x.v[e] * s.shut;
            }
            if (a.dx) store_group<S, TAIL>((S*)a.dx + p[j].row * W + C, col, C, db);
        }
        if (a.dx) store_group<S, TAIL>((S*)a.dx + p[j].row * W, col, C, dx);
        if (a.y) store_group<S, TAIL>((S*)a.y + p[j].row * C, col, C, y);
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static int64_t act_per_row(int64_t C) { return (C + kActGroup - 1) / kActGroup * kActLanes; }

static int64_t act_blocks(int64_t rows, int64_t C, int act) {
    const int64_t per = kActThreads * (act == 2 ? 2 : 4);
    return (rows * act_per_row(C) + per - 1) / per;
}

bool dwact_fits(int64_t rows, int64_t C, int act) {
    return product_below((int64_t)1 << 60, {rows, C + kActGroup}) && grid_of_256_fits(act_blocks(rows, C, act));
}

template <typename S, bool TAIL, int ACT>
static void launch_act_kernel(bool backward, const ActArgs& a, dim3 grid, hipStream_t stream) {
    if (backward)
        hipLaunchKernelGGL((act_bwd_kernel<S, TAIL, ACT>), grid, dim3(kActThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((act_fwd_kernel<S, TAIL, ACT>), grid, dim3(kActThreads), 0, stream, a);
}

template <typename S, int ACT>
static void launch_act_width(bool backward, const ActArgs& a, dim3 grid, hipStream_t stream) {
    if (a.C % kGroup)
        launch_act_kernel<S, true, ACT>(backward, a, grid, stream);
    else
        launch_act_kernel<S, false, ACT>(backward, a, grid, stream);
}

template <typename S>
static void launch_act_kind(int act, bool backward, const ActArgs& a, dim3 grid, hipStream_t stream) {
    if (act == 0) launch_act_width<S, 0>(backward, a, grid, stream);
    if (act == 1) launch_act_width<S, 1>(backward, a, grid, stream);
    if (act == 2) launch_act_width<S, 2>(backward, a, grid, stream);
}

static hipError_t launch_act(int act, bool backward, ActArgs a, int64_t B, bool bf16, hipStream_t stream) {
    const int64_t rows = B * a.T.d;
    a.per_row = divisor((uint32_t)act_per_row(a.C));
    a.units = (uint64_t)rows * a.per_row.d;
    const dim3 grid((uint32_t)act_blocks(rows, a.C, act));
    if (bf16)
        launch_act_kind<uint16_t>(act, backward, a, grid, stream);
    else
        launch_act_kind<float>(act, backward, a, grid, stream);
    return hipGetLastError();
}

hipError_t launch_dwact_fwd(int act, const void* x, const int32_t* lengths, void* y, int8_t* kept, uint8_t* codes,
                            int64_t B, int64_t T, int64_t C, bool bf16, hipStream_t stream) {
    const ActArgs a = {x, nullptr, lengths, y, nullptr, kept, codes, 0, {}, divisor((uint32_t)T), (int32_t)C};
    return launch_act(act, false, a, B, bf16, stream);
}

hipError_t launch_dwact_bwd(int act, const int8_t* kept, const uint8_t* codes, const int32_t* lengths, const void* dy,
                            void* dx, void* y, int64_t B, int64_t T, int64_t C, bool bf16, hipStream_t stream) {
    const ActArgs a = {nullptr, dy, lengths, y, dx, const_cast<int8_t*>(kept), const_cast<uint8_t*>(codes), 0, {},
                       divisor((uint32_t)T), (int32_t)C};
    return launch_act(act, true, a, B, bf16, stream);
}

}  // namespace dw
