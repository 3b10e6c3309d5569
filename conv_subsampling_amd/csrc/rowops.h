// Device helpers of the row-wise operators (layer norm, dropout): 8-element
// groups of a row, sums over the lanes that share a row, and the
// counter-based dropout generator.
#pragma once

#include "common.h"

namespace dw {

constexpr int kGroup = 8;  // consecutive columns a lane holds together

// Eight stored columns as loaded: one 16-byte access of bf16, two of float.
template <typename S>
struct RawGroup {
    static constexpr int N = sizeof(S) / 2;
    u32x4 r[N];
};

// A row starts wherever its width puts it, so the vector accesses are declared
// with the alignment of one element: gfx950 takes unaligned global accesses,
// and an aligned one costs the same through this type.
template <typename S>
struct ElemAligned;
template <>
struct ElemAligned<float> {
    typedef u32x4 vec __attribute__((aligned(4)));
};
template <>
struct ElemAligned<uint16_t> {
    typedef u32x4 vec __attribute__((aligned(2)));
};

// Columns [col, col + 8) of a row of C; columns at or past C read as zero.
// TAIL: C is not a multiple of 8, so one group of the row is partial.
template <typename S, bool TAIL>
__device__ __forceinline__ RawGroup<S> load_group(const S* row, int col, int C) {
    RawGroup<S> g = {};
    if (col + kGroup <= C) {
        typedef typename ElemAligned<S>::vec vec;
        const vec* p = reinterpret_cast<const vec*>(row + col);
#pragma unroll
        for (int i = 0; i < RawGroup<S>::N; ++i) g.r[i] = p[i];
    } else if (TAIL && col < C) {
#pragma unroll
        for (int e = 0; e < kGroup - 1; ++e) {
            if (col + e < C) {
                if constexpr (sizeof(S) == 4)
                    g.r[e / 4][e % 4] = __float_as_uint(row[col + e]);
                else
                    g.r[0][e / 2] |= (uint32_t)row[col + e] << (16 * (e & 1));
            }
        }
    }
    return g;
}

template <typename S>
__device__ __forceinline__ Vf<kGroup> widen(const RawGroup<S>& g) {
    Vf<kGroup> v;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
        if constexpr (sizeof(S) == 4)
            v.v[e] = __uint_as_float(g.r[e / 4][e % 4]);
        else
            v.v[e] = (e & 1) ? bf16_hi(g.r[0][e / 2]) : bf16_lo(g.r[0][e / 2]);
    }
    return v;
}

// Rounds to the storage type (nearest even) and writes the columns below C.
template <typename S, bool TAIL>
__device__ __forceinline__ void store_group(S* row, int col, int C, const Vf<kGroup>& v) {
    RawGroup<S> g;
#pragma unroll
    for (int e = 0; e < kGroup; e += 2) {
        if constexpr (sizeof(S) == 4) {
            g.r[e / 4][e % 4] = __float_as_uint(v.v[e]);
            g.r[e / 4][e % 4 + 1] = __float_as_uint(v.v[e + 1]);
        } else {
            g.r[0][e / 2] = pack_bf16x2(v.v[e], v.v[e + 1]);
        }
    }
    if (col + kGroup <= C) {
        typedef typename ElemAligned<S>::vec vec;
        vec* p = reinterpret_cast<vec*>(row + col);
#pragma unroll
        for (int i = 0; i < RawGroup<S>::N; ++i) p[i] = g.r[i];
    } else if (TAIL && col < C) {
#pragma unroll
        for (int e = 0; e < kGroup - 1; ++e) {
            if (col + e < C) {
                if constexpr (sizeof(S) == 4)
                    row[col + e] = v.v[e];
                else
                    row[col + e] = (uint16_t)(g.r[0][e / 2] >> (16 * (e & 1)));
            }
        }
    }
}

// Sum over the LANES (a power of two) neighbouring lanes that share a row,
// given to each of them.  Within 16 lanes the partners come by DPP (the quad
// permutations, then the mirrors, whose lanes hold equal sums by then), across
// them by the row and half swaps: no LDS access.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
    if constexpr (LANES >= 2) v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
    if constexpr (LANES >= 4) v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
    if constexpr (LANES >= 8) v = dpp_add<0x141>(v);  // half mirror: the other quad of 8
    if constexpr (LANES >= 16) v = dpp_add<0x140>(v);  // mirror: the other 8 of 16
    if constexpr (LANES >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (LANES >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return v;
}

// The dropout generator: Philox4x32 with 10 rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).  The key is the
// caller's 64-bit seed; the counter is the 64-bit index of a group of 8
// columns (row * ceil(C / 8) + column / 8) and the caller's 64-bit stream.
// Column e of the group takes half word e of the 128 bits (low half of a word
// first), so one evaluation serves one 16-byte access of bf16, and the mask
// depends on neither the storage type nor the launch.  16 bits resolve p to
// 2^-16; the scale of the kept values uses the resolved probability, so the
// expectation is exact.
struct DropKeys {
    uint32_t k0, k1, s0, s1;
};

__device__ __forceinline__ DropKeys drop_keys(const uint64_t* rng) {
    const uint64_t seed = rng[0], stream = rng[1];
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)stream, (uint32_t)(stream >> 32)};
}

__device__ __forceinline__ u32x4 philox(uint64_t group, const DropKeys& keys) {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = keys.s0, c3 = keys.s1;
    uint32_t k0 = keys.k0, k1 = keys.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// v[e] * scale where the element's 16 bits reach the threshold, else 0.
__device__ __forceinline__ Vf<kGroup> drop_group(const Vf<kGroup>& v, u32x4 bits, uint32_t threshold, float scale) {
    Vf<kGroup> o;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
        const uint32_t h = (e & 1) ? bits[e / 2] >> 16 : bits[e / 2] & 0xffffu;
        o.v[e] = h >= threshold ? v.v[e] * scale : 0.0f;
    }
    return o;
}

}  // namespace dw
