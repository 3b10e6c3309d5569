// The attention's launch plan: sizes, and the form of each kernel that they and
// the operands' alignment ask for.  Host code alone, so that a CPU test can ask
// which forms a shape takes.
#pragma once

#include <stdint.h>

namespace dw {

struct AttnStride {
    int64_t item, frame, head;  // in elements
};

constexpr int32_t kNoLimit = 1 << 30;        // a context without a limit
constexpr int64_t kAttnMaxFrames = 1 << 28;  // sums of frames and positions stay in 32 bits
constexpr int64_t kAttnMaxHead = 128;        // what a wave's accumulators hold
constexpr int64_t kAttnMaxReach = 1024;      // of the bias map: what LDS holds beside the tiles

struct AttnShape {
    int64_t B, Tq, Tk, H, Hkv, D;
    AttnStride q, k, v, dq, dk, dv;
    int64_t buckets, reach, left, right;  // left, right: at most kNoLimit
    float scale;
};

constexpr int kTile = 32;        // owned and streamed frames of one matrix tile
constexpr int kBiasMargin = 64;  // entries beyond the map's ends: a tile that touches it reads without a clamp
constexpr int kDiag = 64;        // row of the square in which the diagonals of a tile lie in columns
constexpr int64_t kUnits = 256;  // compute units
constexpr int kLdsBytes = 160 * 1024;

inline int attn_bias_bytes(int32_t R) { return (2 * R + 1 + 2 * kBiasMargin) * 4; }

// 16-byte chunks from one row of a tile to the next.
constexpr int tile_slots(int chunks, int elem_bytes) { return chunks + (chunks == 16 && elem_bytes == 2 ? 3 : 1); }

// The padded width that holds a head of D.
inline int head_width(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 96 ? 96 : 128; }

// What direct loads ask of a tensor: whole groups of 8 elements, aligned 16-byte
// chunks, frames that do not overlap, and a tile's offsets in 31 bits.
inline bool direct_fits(const void* base, const AttnStride& s, int64_t D, int elem_bytes) {
    const int64_t chunk = 16 / elem_bytes;
    return (uintptr_t)base % 16 == 0 && D % 8 == 0 && s.item % chunk == 0 && s.frame % chunk == 0 &&
           s.head % chunk == 0 && s.frame >= D && s.frame <= ((int64_t)1 << 29) / 256;
}

// The instance of a kernel that a call takes.
struct AttnForm {
    int dp, own;          // padded head width; owned frames of a workgroup, in units of 32
    bool direct, packed;  // loads straight into LDS; the heads of a group side by side
};

struct FwdPlan {
    int qw, splits;
    bool packed;
    int64_t nqb;
};

// 128 queries a workgroup read each key tile once for four waves, so they are
// taken where they make workgroups enough; next 64, whose two pairs of waves
// divide the keys; and with the fewest queries 32, the keys then being split
// over workgroups until each compute unit has one.  The plan goes by the sizes
// alone (lengths are on the device).
//
// From 128 queries to 64, measured over the batch, lengths from the whole to
// half: the times cross at 290 to 380 workgroups of 128 (bf16 [B,750,8x128],
// 128 and 64 queries: B = 6 33 and 29 us, 8 36 and 41, 15 44 and 63), 380 to 430
// ([B,375,8x64]: B = 16 16.8 and 16.3, 24 20 and 25) and 430 to 480
// ([B,750,8x50]), for float at 290 to 380 ([B,750,8x64]: B = 6 62 and 45, 8 66 and
// 67, 16 97 and 110), and for its widest heads they lie within 8% of each other from
// 170 to 400; so from 1.5 a compute unit on.  Under a causal mask, whose last
// workgroups have the most keys, they cross at 1000 (bf16 [B,1500,4x64]: B = 16
// 37 and 35, 24 40 and 47), 1100 (float [B,1500,8x64]: B = 9 137 and 113, 12 134 and
// 154) and, of three blocks an item, 580 and 700 ([B,300,8x64]): from 4 a unit on.
//
// From 64 queries to 32: of heads over 64, of which a unit takes one workgroup of
// 32, at 100 to 150 workgroups of 64 (bf16 [B,750,8x128], 64 and 32 queries: B = 1
// 19 and 19, 2 20 and 35; float [B,375,8x128]: B = 2 33 and 30, 3 33 and 33, 5 34 and
// 63); of narrower ones at about 250 (bf16 [B,750,8x64]: B = 2 16 and 14, 3 16 and 16).
//
// Twice as many splits cost the join more than they save (16 frames over 20000
// keys, 8 heads: 18 and 21 us).  The splits, and the workspace with them, do not
// depend on the bias.
constexpr int64_t kPackedBias = 16 * 1024;  // bytes of LDS for a group's biases beside the widest tiles

inline FwdPlan fwd_plan(const AttnShape& s) {
    const bool causal = s.left == kNoLimit && s.right != kNoLimit;
    const int64_t for4 = causal ? 4 * kUnits : kUnits * 3 / 2, for2 = s.D > 64 ? kUnits / 2 : kUnits;
    FwdPlan p;
    auto blocks_of = [&](int64_t queries) { return s.B * s.H * ((s.Tq + queries - 1) / queries); };
    p.qw = s.Tq > 32 && blocks_of(128) >= for4 ? 4 : s.Tq > 32 && blocks_of(64) >= for2 ? 2 : 1;
    const int64_t queries = 32 * p.qw;
    p.nqb = (s.Tq + queries - 1) / queries;
    p.splits = 1;
    const int64_t group = s.Hkv ? s.H / s.Hkv : 1;
    const bool could = p.qw == 1 && group > 1 && group * s.Tq <= kTile;
    p.packed = could && group * (s.reach ? attn_bias_bytes((int)s.reach) : 0) <= kPackedBias;
    if (p.qw == 1) {
        int64_t span = s.Tk;
        if (s.left < kNoLimit && s.right < kNoLimit) {
            const int64_t window = s.left + s.right + queries;
            span = window < 1 ? 1 : window < span ? window : span;
        }
        const int64_t blocks = could ? s.B * s.Hkv : blocks_of(32), tiles = (span + 127) / 128;
        int64_t n = kUnits / (blocks ? blocks : 1);
        n = n < tiles ? n : tiles;
        p.splits = (int)(n < 1 ? 1 : n > 64 ? 64 : n);
    }
    return p;
}

// Two buffers of 128 keys leave room for two workgroups a compute unit.
constexpr bool fwd_narrow(int dp, int elem_bytes) { return dp * elem_bytes <= 128; }

inline AttnForm fwd_form(const FwdPlan& p, int64_t D, int elem_bytes, bool direct) {
    const int dp = head_width(D);
    return {dp, p.qw, direct && (p.qw > 1 || fwd_narrow(dp, elem_bytes)), p.packed};
}

// Streamed frames of a tile of the gradients' kernels and its buffers: float rows
// over 64 wide leave room for one buffer beside the sums by distance.
constexpr int bwd_rows(int dp, int elem_bytes, int own) {
    return own == 1 ? 128 : own == 2 || elem_bytes * dp <= 128 ? 64 : 32;
}
constexpr int bwd_buffers(int dp, int elem_bytes, int own) {
    return own == 1 || (own == 2 && elem_bytes == 4 && dp > 64) ? 1 : 2;
}

// Wide bf16 heads leave no room for all of a wave's operands and sums in the
// registers of two waves a SIMD: its values then wait in LDS, in the order in
// which the lanes read them (16 bytes a lane).
constexpr bool bwd_values_in_lds(int dp, int elem_bytes) { return elem_bytes == 2 && dp > 64; }

constexpr int bwd_tile_bytes(int dp, int elem_bytes, int own) {
    return 2 * bwd_buffers(dp, elem_bytes, own) * bwd_rows(dp, elem_bytes, own) *
           tile_slots(dp * elem_bytes / 16, elem_bytes) * 16;
}
constexpr int kSquareBytes = 4 * kTile * kDiag * 4;  // a tile of dS for each wave, beside the tiles of the dq kernel

inline int padded_bias(const AttnShape& s) { return s.reach ? (2 * (int)s.reach + 1 + 2 * kBiasMargin + 3) / 4 * 4 : 0; }

// Bytes of LDS of a workgroup that owns 32 * ow queries or keys of heads of DP.
inline int bwd_lds(const AttnShape& s, int elem_bytes, int ow, bool queries) {
    const int dp = head_width(s.D), tiles = bwd_tile_bytes(dp, elem_bytes, ow), bias = padded_bias(s) * 4;
    const int values = bwd_values_in_lds(dp, elem_bytes) ? 4 * (dp / 16) * 64 * 16 : 0;
    return tiles + bias + (queries ? kSquareBytes + 4 * bias : values + 6 * bwd_rows(dp, elem_bytes, ow) * 4);
}

// Frames a workgroup owns, in units of 32: fewer where more would leave compute
// units without one, if LDS holds the tiles.  dq, then dk/dv, in us over the batch:
//   128 and 64 frames  bf16 [B,750,8x128]    B = 2 51, 38; 55, 35    4 52, 63; 56, 55    8 58, 93; 60, 81
//                      bf16 [B,375,8x64]     B = 8 30, 29; 20, 16   12 32, 44; 21, 25
//                      float [B,375,8x64]    B = 6 56, 46; 57, 35    8 56, 67; 57, 58   16 65, 104; 86, 91
//                      float [B,375,8x128]   B = 6 97, 75; 97, 82    8 97, 122; 97, 141
//                      bf16 causal [B,1000,8x64]  B = 6 48, 48; 40, 32  8 50, 55; 40, 39  12 61, 78; 51, 55
//   64 and 32 frames   bf16 [B,750,8x128]    B = 2 38, 67; 35, 52
//                      bf16 [B,375,8x64]     B = 2 26, 23; 14, 14    4 25, 26; 14, 25
//                      float [B,375,8x64]    B = 2 39, 35; 35, 26    4 39, 61; 35, 47
// The first cross at 150 to 200 workgroups of 128, of bf16 heads up to 64, whose
// workgroups of 64 a unit holds more of, at 270, and at up to twice that under a
// causal mask; the second between 96 and 192 workgroups of 64.
inline int owned(const AttnShape& s, int elem_bytes, bool queries) {
    const int64_t pairs = s.B * (queries ? s.H : s.Hkv), frames = queries ? s.Tq : s.Tk;
    const bool narrow = elem_bytes == 2 && s.D <= 64, one_sided = (s.left == kNoLimit) != (s.right == kNoLimit);
    const int64_t for4 = (narrow ? kUnits : kUnits * 3 / 4) * (one_sided ? 2 : 1), for2 = kUnits / 2;
    int ow = pairs * ((frames + 127) / 128) >= for4 ? 4 : pairs * ((frames + 63) / 64) >= for2 ? 2 : 1;
    while (ow < 4 && bwd_lds(s, elem_bytes, ow, queries) > kLdsBytes) ow *= 2;
    return ow;
}

inline AttnForm bwd_form(int own, int64_t D, int elem_bytes, bool direct) {
    const int dp = head_width(D);
    return {dp, own, direct && bwd_buffers(dp, elem_bytes, own) == 2, false};
}

}  // namespace dw
