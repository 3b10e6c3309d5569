// Four neighbouring columns of a row, as the operator over heads loads and stores
// them (8 bytes of bf16, 16 of float).
#pragma once

#include "rowops.h"

namespace dw {

constexpr int kQuad = 4;

// Rows start wherever their strides put them, so the accesses are declared with
// the alignment of one element, as in rowops.h.
template <typename S>
struct QuadRaw;
template <>
struct QuadRaw<float> {
    typedef u32x4 type;
    typedef u32x4 access __attribute__((aligned(4)));
};
template <>
struct QuadRaw<uint16_t> {
    typedef u32x2 type;
    typedef u32x2 access __attribute__((aligned(2)));
};
template <typename S>
using quad_raw = typename QuadRaw<S>::type;

// have: columns of the row from p on; those at or past it read as zero.
// TAIL: it may be under four.
template <typename S, bool TAIL>
__device__ __forceinline__ quad_raw<S> load_quad(const S* p, int have) {
    quad_raw<S> q = {};
    if (!TAIL || have >= kQuad) {
        q = *reinterpret_cast<const typename QuadRaw<S>::access*>(p);
    } else {
#pragma unroll
        for (int e = 0; e < kQuad - 1; ++e) {
            if (e < have) {
                if constexpr (sizeof(S) == 4)
                    q[e] = __float_as_uint(p[e]);
                else
                    q[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
            }
        }
    }
    return q;
}

template <typename S>
__device__ __forceinline__ float quad_at(const quad_raw<S>& q, int e) {
    if constexpr (sizeof(S) == 4)
        return __uint_as_float(q[e]);
    else
        return (e & 1) ? bf16_hi(q[e / 2]) : bf16_lo(q[e / 2]);
}

template <typename S>
__device__ __forceinline__ Vf<kQuad> widen_quad(const quad_raw<S>& q) {
    Vf<kQuad> v;
#pragma unroll
    for (int e = 0; e < kQuad; ++e) v.v[e] = quad_at<S>(q, e);
    return v;
}

// Rounds to the storage type (nearest even).
template <typename S, bool TAIL>
__device__ __forceinline__ void store_quad(S* p, int have, const Vf<kQuad>& v) {
    quad_raw<S> q;
    if constexpr (sizeof(S) == 4) {
#pragma unroll
        for (int e = 0; e < kQuad; ++e) q[e] = __float_as_uint(v.v[e]);
    } else {
        q[0] = pack_bf16x2(v.v[0], v.v[1]);
        q[1] = pack_bf16x2(v.v[2], v.v[3]);
    }
    if (!TAIL || have >= kQuad) {
        *reinterpret_cast<typename QuadRaw<S>::access*>(p) = q;
    } else {
#pragma unroll
        for (int e = 0; e < kQuad - 1; ++e) {
            if (e < have) {
                if constexpr (sizeof(S) == 4)
                    p[e] = v.v[e];
                else
                    p[e] = (uint16_t)(q[e / 2] >> (16 * (e & 1)));
            }
        }
    }
}

}  // namespace dw
