// Shared pieces of the attention kernels (forward, gradients): arguments,
// matrix fragments, tiles in LDS, the relative position bias and the masks.
//
// Every product runs on 32x32 matrix instructions with the OWNED axis (the
// queries in the forward and in dq, the keys in dk and dv) in the columns, so
// that a lane holds one row of the softmax and its neighbour 32 lanes away the
// rest of it:
//   columns: owned index lane % 32
//   rows:    streamed index 8 * (r / 4) + 4 * (lane / 32) + r % 4 of register r
// The next product contracts over those rows.  A contraction may take its
// index in any order as long as both operands agree, so the probabilities go
// from the accumulator registers straight into the next instruction's operand,
// and it is the other operand that is read from LDS in that order (transposed).
#pragma once

#include "launch.h"
#include "rowops.h"

#include <type_traits>

namespace dw {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ int wave_of_block() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// BYTES (16 or 4) a lane from the buffer's byte off into LDS at lds plus BYTES
// times the lane, without a register between.  Inline assembly, without a result
// register, because the compiler would else wait for the load before any LDS
// read; nothing else in these kernels takes its operand from m0.  A build without
// optimisation keeps uniform values in vector registers, which the assembly
// cannot take: it has the compiler's own form, with its waits.
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t bytes, uint32_t off, uint32_t lds) {
    static_assert(BYTES == 16 || BYTES == 4, "the widths that the kernels use");
#ifdef __OPTIMIZE__
    const uint64_t at = (uint64_t)base;
    const u32x4 rsrc = {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, (uint32_t)kBufferFlags};
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(lds), "v"(off), "s"(rsrc) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :: "s"(lds), "v"(off), "s"(rsrc) : "memory");
#else
    const rsrc_t from = make_rsrc(base, bytes);
    auto* to = (__attribute__((address_space(3))) void*)(uintptr_t)lds;
    if constexpr (BYTES == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 16, off, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 4, off, 0, 0, 0);
#endif
}

// The 16-deep operand of one 32x32 product: 8 values a lane, of the streamed
// depth 8 * (lane / 32) + e.
template <typename S>
struct Frag;
template <>
struct Frag<uint16_t> {
    u32x4 r;
};
// float32 as three bf16 parts of 8 significant bits each, whose sum is the value
// exactly: the first cut off (so that nothing overflows), the second rounded (so
// that the third, and the products left out below, have either sign).
template <>
struct Frag<float> {
    u32x4 part[3];
};

__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x16 c) {
    return mma(a.r, b.r, c);
}

// float32 keeps its 24 bits: the six products of parts that can reach 2^-22 of
// the whole, smallest first; the three left out are at most 2^-22 of it together,
// of either sign, where rounding a product to float32 is 2^-24.  Six bf16
// products take 192 cycles of the matrix units where eight float ones take 512.
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
    c = mma(a.part[2], b.part[0], c);
    c = mma(a.part[0], b.part[2], c);
    c = mma(a.part[1], b.part[1], c);
    c = mma(a.part[1], b.part[0], c);
    c = mma(a.part[0], b.part[1], c);
    return mma(a.part[0], b.part[0], c);
}

// The same with the small products summed apart, so that the large sum is
// rounded once for each 16 of its depth and not six times.  For the scores and
// weights' gradients that the table's gradient adds up: its terms cancel, and
// its error fell from 1.1e-6 to 3.2e-7 of it ([3,333,4x50]).
__device__ __forceinline__ void mma_apart(const Frag<float>& a, const Frag<float>& b, f32x16& c, f32x16& small) {
    small = mma(a.part[2], b.part[0], small);
    small = mma(a.part[0], b.part[2], small);
    small = mma(a.part[1], b.part[1], small);
    small = mma(a.part[1], b.part[0], small);
    small = mma(a.part[0], b.part[1], small);
    c = mma(a.part[0], b.part[0], c);
}

__device__ __forceinline__ void mma_apart(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x16& c, f32x16&) {
    c = mma(a, b, c);
}

__device__ __forceinline__ Frag<float> split(const float (&v)[8]) {
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float x = v[e], y = v[e + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            // the high halves of both, cut off (the third part fits) or rounded
            const uint32_t pair = p == 1 ? pack_bf16x2(x, y)
                                         : __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302);
            f.part[p][e / 2] = pair;
            x -= bf16_lo(pair);
            y -= bf16_hi(pair);
        }
    }
    return f;
}

// Stands between a run of products and the first arithmetic on their sums: the
// wait states that a vector instruction has to keep from the product whose
// result it reads (8 passes + 4).  The compiler counts them too, but where two
// paths of different length lead from the products to a read it was seen to go by
// the longer one (7 states on the other, gfx950 at -O3).  The sums pass through
// the wait, because products, which have no other effect, else move past it.
__device__ __forceinline__ void products_done(f32x16& a) { asm volatile("s_nop 11" : "+v"(a)); }
__device__ __forceinline__ void products_done(f32x16& a, f32x16& b) { asm volatile("s_nop 11" : "+v"(a), "+v"(b)); }
template <int N>
__device__ __forceinline__ void products_done(f32x16 (&a)[N]) {
    static_assert(N <= 4, "runs of 32 head elements");
    if constexpr (N == 1) products_done(a[0]);
    if constexpr (N == 2) products_done(a[0], a[1]);
    if constexpr (N == 3) asm volatile("s_nop 11" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]));
    if constexpr (N == 4) asm volatile("s_nop 11" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
}

// Accumulator registers 8k .. 8k + 7 as the operand of the next product,
// rounded to the storage type (bf16: the matrix instruction takes no wider
// operand; the sums of a softmax are taken before the rounding).
template <typename S>
__device__ __forceinline__ Frag<S> to_frag(const f32x16& c, int k) {
    Frag<S> f;
    if constexpr (sizeof(S) == 4) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c[8 * k + e];
        f = split(v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f.r[e] = pack_bf16x2(c[8 * k + 2 * e], c[8 * k + 2 * e + 1]);
    }
    return f;
}

// Waits here for an operand that was loaded from memory.  Left to its first use
// inside the loop over tiles, the wait would hold up that loop's own loads.
__device__ __forceinline__ void arrived(Frag<uint16_t>& f) { asm volatile("" : "+v"(f.r)); }
__device__ __forceinline__ void arrived(Frag<float>& f) {
    asm volatile("" : "+v"(f.part[0]), "+v"(f.part[1]), "+v"(f.part[2]));
}

template <typename S>
__device__ __forceinline__ Frag<S> to_frag(const RawGroup<S>& g) {
    Frag<S> f;
    if constexpr (sizeof(S) == 4) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(g.r[e / 4][e % 4]);
        f = split(v);
    } else {
        f.r = g.r[0];
    }
    return f;
}

// ---------------------------------------------------------------------------
// A tile of frames x DP head elements in LDS.  A row is a whole number of
// 16-byte chunks and a pad that puts the rows that one instruction touches on
// different banks: eight neighbouring rows for a 16-byte read, four for a
// transposing one.  Measured, sixteen waves reading: 16-byte reads take 2.7
// cycles with these pads as from linear addresses (25 without one at 128 bf16
// elements), transposing reads 3.2 (4.7 there with one chunk of pad).
template <typename S, int DP>
struct Tile {
    static constexpr int kChunks = DP * (int)sizeof(S) / 16;
    static constexpr int kSlots = tile_slots(kChunks, sizeof(S));
    static constexpr int kStride = kSlots * 16 / (int)sizeof(S);
    static constexpr int kGroups = DP / kGroup;  // 8-element groups of a row

    static constexpr int bytes(int rows) { return rows * kSlots * 16; }

    // Operand whose rows are frames row0 + lane % 32 and whose depth is the
    // 16 head elements from 16 * c.
    static __device__ __forceinline__ Frag<S> rows(const S* t, int row0, int c, int lane) {
        const S* p = t + (row0 + lane % 32) * kStride + 16 * c + 8 * (lane / 32);
        Frag<S> f;
        if constexpr (sizeof(S) == 4) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            f = split(v);
        } else {
            f.r = *reinterpret_cast<const u32x4*>(p);
        }
        return f;
    }

    // Operand whose rows are head elements 32 * d + lane % 32 and whose depth
    // is the 16 frames from row0, in the order of the accumulator's registers:
    // frames 4 * (lane / 32) + e, then 8 + 4 * (lane / 32) + e - 4.  bf16: one
    // transposing read brings lane i of 16 the i-th column of four rows, whose
    // 4-element pieces the 16 lanes address.
    static __device__ __forceinline__ Frag<S> columns(const S* t, int row0, int d, int lane) {
        Frag<S> f;
        if constexpr (sizeof(S) == 4) {
            const S* p = t + (row0 + 4 * (lane / 32)) * kStride + 32 * d + lane % 32;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[((e / 4) * 8 + e % 4) * kStride];
            f = split(v);
        } else {
            const S* p = t + (row0 + 4 * (lane / 32) + lane % 16 / 4) * kStride + 32 * d + 16 * (lane / 16 % 2) +
                         4 * (lane % 4);
            typedef __attribute__((address_space(3))) s16x4* lds;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + 8 * kStride));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            f.r = u32x4{a.x, a.y, b.x, b.y};
        }
        return f;
    }
};

// A workgroup's share of a tile on its way from memory to LDS through
// registers: start() reads, finish() writes.  Rows from `live` on and head
// elements from D on become zero and are not read.
template <typename S, int DP, int ROWS>
struct TileRegs {
    static constexpr int kTotal = ROWS * Tile<S, DP>::kGroups;
    static constexpr int N = (kTotal + kAttnThreads - 1) / kAttnThreads;
    RawGroup<S> g[N];

    __device__ __forceinline__ void setup(int64_t, int) {}

    __device__ __forceinline__ void start(const S* base, int64_t frame, int live, int D, S*) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + n * kAttnThreads;
            const int row = at / Tile<S, DP>::kGroups, col = at % Tile<S, DP>::kGroups * kGroup;
            g[n] = load_group<S, true>(base + row * frame, col, row < live && at < kTotal ? D : 0);
        }
    }

    __device__ __forceinline__ void finish(S* tile) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + n * kAttnThreads;
            const int row = at / Tile<S, DP>::kGroups, col = at % Tile<S, DP>::kGroups * kGroup;
            if (kTotal % kAttnThreads != 0 && at >= kTotal) continue;
            u32x4* p = reinterpret_cast<u32x4*>(tile + row * Tile<S, DP>::kStride + col);
#pragma unroll
            for (int i = 0; i < RawGroup<S>::N; ++i) p[i] = g[n].r[i];
        }
    }
};

// The same without registers: loads that write LDS themselves, 16 bytes a lane
// to the wave's LDS address (m0) plus 16 times the lane.  A lane works out once
// which row and chunk its place in the tile is; lanes on a pad sit out.  The
// buffer ends at the last live row, so what lies past it arrives as zero.
// start() returns with the loads in flight: a wait for them and a barrier come
// before the tile is read.
template <typename S, int DP, int ROWS>
struct TileDma {
    static constexpr int kTotal = ROWS * Tile<S, DP>::kSlots;
    static constexpr int N = (kTotal + kAttnThreads - 1) / kAttnThreads;
    static constexpr uint32_t kSkip = 0xffffffffu, kZero = 0xfffffff0u;
    uint32_t off[N];

    __device__ __forceinline__ void setup(int64_t frame, int D) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + n * kAttnThreads;
            const int row = at / Tile<S, DP>::kSlots, chunk = at % Tile<S, DP>::kSlots;
            off[n] = at >= kTotal || chunk >= Tile<S, DP>::kChunks ? kSkip
                     : chunk * 16 >= D * (int)sizeof(S)             ? kZero
                                                        : (uint32_t)(row * frame * (int)sizeof(S)) + chunk * 16;
        }
    }

    __device__ __forceinline__ void start(const S* base, int64_t frame, int live, int D, S* tile) {
        const uint32_t bytes =
            live > 0 ? (uint32_t)((((live < ROWS ? live : ROWS) - 1) * frame + D) * (int)sizeof(S)) : 0;
        const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)tile +
                             wave_of_block() * 1024;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (off[n] != kSkip) load_to_lds<16>(base, bytes, off[n], lds + n * kAttnThreads * 16);
        }
    }

    __device__ __forceinline__ void finish(S*) const {}
};

__device__ __forceinline__ void wave_loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The tiles of two tensors (keys and values, or queries and output gradients),
// with two buffers each (tile t + 1 on its way while tile t is used) or one (its
// registers hold tile t + 1).  A third and fourth buffer, with counted waits, made
// no kernel faster: loads are not what the tiles wait for.
template <typename S, int DP, int ROWS, int BUFFERS, bool DMA>
struct TilePair {
    using Load = std::conditional_t<DMA, TileDma<S, DP, ROWS>, TileRegs<S, DP, ROWS>>;
    static_assert(BUFFERS == 2 || !DMA, "direct loads write the tile while the one before is in use");
    static constexpr int kBytes = Tile<S, DP>::bytes(ROWS), kAllBytes = 2 * BUFFERS * kBytes;
    Load x, y;
    char* at;
    const S *xbase, *ybase;
    int64_t xframe, yframe;
    int D, total;  // head elements, frames

    __device__ __forceinline__ TilePair(char* at, const S* xbase, int64_t xframe, const S* ybase, int64_t yframe, int D,
                                        int total)
        : at(at), xbase(xbase), ybase(ybase), xframe(xframe), yframe(yframe), D(D), total(total) {
        x.setup(xframe, D);
        y.setup(yframe, D);
    }

    __device__ __forceinline__ S* x_of(int t) const { return (S*)(at + (BUFFERS == 2 && (t & 1) ? 2 * kBytes : 0)); }
    __device__ __forceinline__ S* y_of(int t) const { return (S*)((char*)x_of(t) + kBytes); }

    __device__ __forceinline__ void start(int t) {
        const int64_t from = (int64_t)t * ROWS;
        x.start(xbase + from * xframe, xframe, total - (int)from, D, x_of(t));
        y.start(ybase + from * yframe, yframe, total - (int)from, D, y_of(t));
    }

    __device__ __forceinline__ void finish(int t) const {
        x.finish(x_of(t));
        y.finish(y_of(t));
    }

    // Everything before tile t is used: its loads are in, and every wave is
    // done with the buffer that the next tile's loads write, which start here.
    __device__ __forceinline__ void enter(int t, bool more) {
        if (BUFFERS == 1) {
            __syncthreads();
            finish(t);
        }
        wave_loads_done();
        __syncthreads();
        if (more) start(t + 1);
    }

    // After tile t was used.
    __device__ __forceinline__ void leave(int t, bool more) const {
        if (BUFFERS == 2 && more) finish(t + 1);
    }
};

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
struct AttnArgs {
    const void *q, *k, *v, *table;
    const int32_t *buckets, *q_lengths, *k_lengths, *q_pos;
    AttnStride qs, ks, vs;
    int32_t B, Tq, Tk, H, Hkv, D;
    int32_t NB, R;         // buckets of the table, reach of the map
    int32_t left, right;   // kNoLimit: none
    float scale, scale2;   // of the scores, and times log2(e)
};

inline AttnArgs attn_args(const AttnPtrs& p, const AttnShape& s) {
    AttnArgs a;
    a.q = p.q, a.k = p.k, a.v = p.v, a.table = p.table;
    a.buckets = p.buckets, a.q_lengths = p.q_lengths, a.k_lengths = p.k_lengths, a.q_pos = p.q_pos;
    a.qs = s.q, a.ks = s.k, a.vs = s.v;
    a.B = (int32_t)s.B, a.Tq = (int32_t)s.Tq, a.Tk = (int32_t)s.Tk;
    a.H = (int32_t)s.H, a.Hkv = (int32_t)s.Hkv, a.D = (int32_t)s.D;
    a.NB = (int32_t)s.buckets, a.R = (int32_t)s.reach;
    a.left = (int32_t)s.left, a.right = (int32_t)s.right;
    a.scale = s.scale, a.scale2 = s.scale * kLog2e;
    return a;
}

// Calls f with the padded head width that holds D.
template <typename F>
hipError_t with_head_width(int64_t D, F&& f) {
    switch (head_width(D)) {
        case 32: return f(std::integral_constant<int, 32>());
        case 64: return f(std::integral_constant<int, 64>());
        case 96: return f(std::integral_constant<int, 96>());
        default: return f(std::integral_constant<int, 128>());
    }
}

// The workgroup's place: its block of owned frames and its (item, head) pair.
// Workgroups go round the XCDs, and a pair's blocks share its keys and values
// in one XCD's L2, so whole pairs are dealt to the XCDs in turn (in turn, not in
// runs: an XCD then gets short and long items alike).  Pairs beyond a multiple
// of the XCDs are dealt block by block.  longest_last: a block's work grows with
// its index, so the last blocks of all pairs go first and the short ones fill up.
struct AttnPlace {
    uint32_t block, pair;
    __device__ __forceinline__ AttnPlace(uint32_t id, uint32_t blocks, uint32_t pairs, bool longest_last) {
        const uint32_t each = pairs / kNumXcd, even = each * kNumXcd;
        if (id < even * blocks) {
            const uint32_t slot = id / kNumXcd;
            pair = (longest_last ? slot % each : slot / blocks) * kNumXcd + id % kNumXcd;
            block = longest_last ? blocks - 1 - slot / each : slot % blocks;
        } else {
            pair = id / blocks;
            block = id % blocks;
        }
    }
};

// The item with the rank-th most work.  The workgroups of a padded batch start
// in this order, so that the long ones run beside short ones and not after them.
__device__ __forceinline__ int item_of_rank(const AttnArgs& a, int rank) {
    if (a.B == 1 || a.B > 64 || (!a.q_lengths && !a.k_lengths)) return rank;
    const int lane = threadIdx.x % 64, b = lane < a.B ? lane : 0;
    const float work = (float)item_length(a.q_lengths, b, a.Tq) * (float)item_length(a.k_lengths, b, a.Tk);
    int mine = 0;
    for (int m = 0; m < a.B; ++m) {
        const float other = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(work), m));
        mine += other > work || (other == work && m < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.B && mine == rank));
}

// One item's valid frames and the position of its first query on the key axis.
struct AttnItem {
    int32_t nq, nk;
    int64_t pos;
    int32_t pos32;  // pos where it can matter: beyond, every distance is past the map's reach on the same side

    __device__ __forceinline__ AttnItem(const AttnArgs& a, int b)
        : nq((int32_t)item_length(a.q_lengths, b, a.Tq)), nk((int32_t)item_length(a.k_lengths, b, a.Tk)),
          pos(a.q_pos ? a.q_pos[b] : 0) {
        const int64_t far = (int64_t)1 << 29;
        pos32 = (int32_t)(pos < -far ? -far : pos > far ? far : pos);
    }

    // Keys [first, last] that queries i0 .. i1 may see between them.
    __device__ __forceinline__ int32_t first_key(const AttnArgs& a, int32_t i0) const {
        const int64_t j = a.left == kNoLimit ? 0 : i0 + pos - a.left;
        return (int32_t)(j < 0 ? 0 : j > nk ? nk : j);
    }
    __device__ __forceinline__ int32_t last_key(const AttnArgs& a, int32_t i1) const {
        const int64_t j = a.right == kNoLimit ? nk - 1 : i1 + pos + a.right;
        return (int32_t)(j < -1 ? -1 : j > nk - 1 ? nk - 1 : j);
    }
    // Queries [first, last] that see a key of j0 .. j1.
    __device__ __forceinline__ int32_t first_query(const AttnArgs& a, int32_t j0) const {
        const int64_t i = a.right == kNoLimit ? 0 : j0 - pos - a.right;
        return (int32_t)(i < 0 ? 0 : i > nq ? nq : i);
    }
    __device__ __forceinline__ int32_t last_query(const AttnArgs& a, int32_t j1) const {
        const int64_t i = a.left == kNoLimit ? nq - 1 : j1 - pos + a.left;
        return (int32_t)(i < -1 ? -1 : i > nq - 1 ? nq - 1 : i);
    }
};

// The head's bias for every distance -R .. R in units of log2, with the ends
// repeated kBiasMargin times on both sides.  A table may hold its type's lowest
// or largest value: times log2(e) that must stay a number, so that rows which
// hold nothing else still weigh their keys alike.  Bucket numbers are held to
// the table.
// The constructor reads the map (the first entries of each thread), fill() the
// table: what is read in between is in flight with the map.
template <typename S>
struct BiasFill {
    static constexpr int kFirst = 3;
    int bucket[kFirst];

    static __device__ __forceinline__ int map_at(const AttnArgs& a, int x) {
        int rel = x - kBiasMargin;
        rel = rel < 0 ? 0 : rel > 2 * a.R ? 2 * a.R : rel;
        const int b = a.buckets[rel];
        return b < 0 ? 0 : b >= a.NB ? a.NB - 1 : b;
    }

    static __device__ __forceinline__ float value(const AttnArgs& a, int h, int b) {
        const float t = to_f32(((const S*)a.table)[(int64_t)b * a.H + h]);
        const float v = t * kLog2e, most = 3.0e38f;
        return fabsf(t) < __builtin_inff() ? __builtin_amdgcn_fmed3f(v, -most, most) : v;
    }

    __device__ __forceinline__ explicit BiasFill(const AttnArgs& a) {
        if (!a.table) return;
#pragma unroll
        for (int k = 0; k < kFirst; ++k) bucket[k] = map_at(a, threadIdx.x + k * kAttnThreads);
    }

    __device__ __forceinline__ void fill(const AttnArgs& a, int h, float* bias) const {
        if (!a.table) return;
        const int n = 2 * a.R + 1 + 2 * kBiasMargin;
#pragma unroll
        for (int k = 0; k < kFirst; ++k) {
            const int x = threadIdx.x + k * kAttnThreads;
            if (x < n) bias[x] = value(a, h, bucket[k]);
        }
        for (int x = threadIdx.x + kFirst * kAttnThreads; x < n; x += kAttnThreads) bias[x] = value(a, h, map_at(a, x));
    }
};

// The distance key - query of a tile's first key and first query says what the
// tile's bias is: past the map's reach on either side one value, else looked up.
enum class Span { kLow, kNear, kHigh };
__device__ __forceinline__ Span span_of(int base, int R) {
    return base + (kTile - 1) <= -R ? Span::kLow : base - (kTile - 1) >= R ? Span::kHigh : Span::kNear;
}

__device__ __forceinline__ float swap_halves(float v) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(threadIdx.x & 32 ? s[0] : s[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Row of register r of a 32x32 accumulator in lanes of half h.
__device__ __forceinline__ constexpr int acc_row(int r, int half) { return 8 * (r / 4) + 4 * half + r % 4; }

// Four neighbouring head elements d .. d + 3 of one frame.
template <typename S>
__device__ __forceinline__ void store4(S* row, int d, int D, float v0, float v1, float v2, float v3) {
    const float v[4] = {v0, v1, v2, v3};
    if (d + 4 <= D) {
        if constexpr (sizeof(S) == 4) {
            typedef f32x4 vec __attribute__((aligned(4)));
            *reinterpret_cast<vec*>(row + d) = f32x4{v0, v1, v2, v3};
        } else {
            typedef u32x2 vec __attribute__((aligned(2)));
            *reinterpret_cast<vec*>(row + d) = u32x2{pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (d + e < D) {
                if constexpr (sizeof(S) == 4)
                    row[d + e] = v[e];
                else
                    row[d + e] = (uint16_t)bf16_bits_rne(v[e]);
            }
        }
    }
}

}  // namespace dw
