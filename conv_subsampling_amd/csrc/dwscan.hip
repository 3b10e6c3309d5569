// A gated linear recurrence over the frames of [B][T][C], channel by channel,
// and its backward pass.
//
//   w = scale * softplus(decay) * sigmoid(r),  a = exp(-w)
//   h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(g) x
//
// Where a > 1/2 the state moves by d = 1 - a = -expm1(-w), taken without
// cancellation: h <- (h - d h) + u, u = sqrt(d (2 - d)) sigmoid(g) x, the bracket
// one fused operation; elsewhere h <- a h + u.  A decay near 1 thus keeps its
// digits, as does one near 0, down to 2^-126, and products of decays are
// exponentials of sums of w.
//
// Frames in parallel: a run of frames maps the state h before it to P h + H
// behind it, and runs compose.  A thread takes 2 channels of FR frames, in
// registers; the 2 threads along the frames that share a wave exchange (P, H)
// by a lane swap, the 4 waves of a workgroup through LDS, so a workgroup does a
// tile of 8 * FR frames and memory sees each tensor once.
//
// Tiles of one item are joined in one of two ways.  Where items and channels
// make workgroups enough, a workgroup goes through the tiles of its chain (an
// item's 64 channels) in turn.  Elsewhere every tile has a workgroup of its
// own, which publishes the (P, H) of its tile and composes those of the tiles
// before it, in their order, so results repeat bit for bit.  Tiles are given
// out by a counter for each chain: whoever waits for a tile waits for a
// workgroup that has started, and that one waits for earlier ones alone.
//
// Bound by memory in float, by memory and vector operations side by side in bf16
// (about 50 operations an element, 6 of them transcendental, 95 in the gradients;
// lengths of half to all):
// bf16 [16,750,1024] 81 MB in 26.9 us a call, 15 of them issue slots (3.0 TB/s; a
// large copy reaches 5.1, the loads and stores alone take 18 us), float [2,6001,512]
// 89 MB in 23.5 (3.8 TB/s), all of [32,1500,512] 393 MB in 86.2 (4.6 TB/s).  Gradients
// bf16 [16,750,1024] 168 MB in 51.0 (3.3 TB/s, 25 us of issue slots), float
// [32,1500,512] 787 MB in 170 (4.6 TB/s).  One frame of 64 items takes 8.7 us, which is
// the host's call; the kernel is 3.5.
#include "launch.h"
#include "rowops.h"

namespace dw {

constexpr int kScanThreads = 256, kScanWaves = kScanThreads / 64;
constexpr int kScanPair = 2;                                  // channels of a thread
constexpr int kScanLanes = 32;                                // threads across the channels
constexpr int kScanRows = kScanThreads / kScanLanes;          // and along frames, or items
constexpr int kScanCols = kScanLanes * kScanPair;             // channels of a workgroup
constexpr int kScanRun = 8, kScanLongRun = 16;                // frames of a thread in a tile
constexpr int kScanGroup = 16;                                // tiles whose composition is published too
constexpr int kScanTicket = 32;                               // words from one chain's counter to the next: a cache line
// Polls of a lane for its words, about a microsecond each.  A word that is read
// belongs to a workgroup that has started and waits for earlier ones alone, so it
// comes within microseconds.  Only where the workspace is overwritten meanwhile
// (two calls at once on one, which is not allowed) does it not: then the wait ends, a
// ticket past the last tile ends its workgroup, and nothing is written outside the
// call's tensors, but what is in them is undefined: NaN behind a wait that ended,
// anything in tiles that no workgroup took and in the sums of ddecay over them.
constexpr int kScanPolls = 1 << 16;

struct ScanArgs {
    const void *x, *r, *g, *yin, *dy;
    const float* decay;
    const int32_t* lengths;
    const float* start;   // the state (backward: its gradient) that enters the first (last) frame, NULL: zero
    void *y, *dx, *dr, *dg;
    const float* h0;      // backward: the state before the first frame
    float* end;           // what leaves the last (first) frame
    uint32_t* tickets;    // [chains][kScanTicket]: tiles given out
    uint64_t* words;      // [chains][tiles + tiles / kScanGroup][kScanCols]: published (P, H)
    double* partial;      // backward: [row blocks][C], sums for ddecay
    FrameStride xs, rs, gs, ys, dys, dxs, drs, dgs;
    int64_t B, T;
    int32_t C, col_blocks, tiles;
    float scale;
};

// ---------------------------------------------------------------------------
// Two neighbouring channels
// ---------------------------------------------------------------------------
template <typename S>
struct PairRaw;
template <>
struct PairRaw<float> {
    typedef u32x2 type;
    typedef u32x2 access __attribute__((aligned(4)));
};
template <>
struct PairRaw<uint16_t> {
    typedef uint32_t type;
    typedef uint32_t access __attribute__((aligned(2)));
};
template <typename S>
using pair_raw = typename PairRaw<S>::type;

// have: channels from p on; TAIL: it may be one.  STREAM: read without claiming a
// place in the caches.  The gradients read so what a training step reads for the
// last time, us without and with: bf16 [32,1500,512] 113.5 and 108.1, float 186.0
// and 176.2, between the kernels that write dy and read their results 184.9 and
// 178.2, 412.7 and 372.6.  The forward loses by it in bf16 ([16,750,1024] 29.0 and
// 31.8, [32,1500,512] 55.5 and 55.6; float 43.4 and 43.1, 86.1 and 77.6).
template <typename S, bool TAIL, bool STREAM>
__device__ __forceinline__ pair_raw<S> load_pair(const S* p, int have) {
    typedef typename PairRaw<S>::access access;
    if (!TAIL || have >= kScanPair) {
        if constexpr (STREAM)
            return __builtin_nontemporal_load(reinterpret_cast<const access*>(p));
        else
            return *reinterpret_cast<const access*>(p);
    }
    pair_raw<S> q = {};
    if (have == 1) {
        if constexpr (sizeof(S) == 4)
            q[0] = __float_as_uint(p[0]);
        else
            q = p[0];
    }
    return q;
}

template <typename S>
__device__ __forceinline__ float pair_at(const pair_raw<S>& q, int e) {
    if constexpr (sizeof(S) == 4)
        return __uint_as_float(q[e]);
    else
        return e ? bf16_hi(q) : bf16_lo(q);
}

// Rounded to the storage type (nearest even).
template <typename S>
__device__ __forceinline__ pair_raw<S> pack_pair(f32x2 v) {
    if constexpr (sizeof(S) == 4)
        return u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])};
    else
        return pack_bf16x2(v[0], v[1]);
}

// Into the caches: what reads it next gains more (bf16 [32,1500,512], forward and
// one reader 84.5 us against 86.6 without, gradients and readers 172.1 against
// 177.0) than a call by itself loses (52.4 against 50.5).
template <typename S, bool TAIL>
__device__ __forceinline__ void store_pair(S* p, int have, pair_raw<S> q) {
    if (!TAIL || have >= kScanPair) {
        *reinterpret_cast<typename PairRaw<S>::access*>(p) = q;
    } else if (have == 1) {
        if constexpr (sizeof(S) == 4)
            p[0] = __uint_as_float(q[0]);
        else
            p[0] = (uint16_t)q;
    }
}

// ---------------------------------------------------------------------------
// The step's functions
// ---------------------------------------------------------------------------
// exp(-v).  float: the rounding of the exponent's product, and what the constant
// leaves out, come back as a factor (bounded, so that infinite exponents stay what
// they are): off by 4 2^-24 of itself.  bf16: one rounded product, off by up to |v| 2^-24, which
// its inputs' own 2^-9 hide.
template <typename S>
__device__ __forceinline__ float exp_minus(float v) {
    const float t = v * -1.44269502f, p = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(S) == 2) return p;
    const float left = __builtin_fmaf(v, -1.92596299e-8f, __builtin_fmaf(v, -1.44269502f, -t));
    return p * __builtin_fmaf(__builtin_amdgcn_fmed3f(left, -1.0f, 1.0f), 0.69314718f, 1.0f);
}

// 1 / (1 + exp(-v)), given the exponential.  Results below 2^-126 are zero.
__device__ __forceinline__ float sigmoid_of(float e) { return __builtin_amdgcn_rcpf(1.0f + e); }

template <typename S>
__device__ __forceinline__ float sigmoid(float v) {
    return sigmoid_of(exp_minus<S>(v));
}

// 1 - sigmoid(v) = exp(-v) sigmoid(v), without cancellation.  Where the gate is zero, so
// is this, which then scales nothing but zeros.
__device__ __forceinline__ float shut_of(float e, float open) { return fminf(e, 0x1p126f) * open; }

// What the decay a = 2^-v (v = w / log 2) does to a state, as the one of 1 - a and a
// that a float holds without loss of digits: d = 1 - a where a > 1/2, a polynomial in
// v (off by 2.2 2^-24 of d with its roundings), and -a elsewhere (-0: a decay of 0).
__device__ __forceinline__ float decay_factor(float v) {
    const float d = v * (0.69314718f + v * (-0.24022606f + v * (0.055498954f + v * (-0.0095962733f + v * (0.0012907785f + v * -0.00011458035f)))));
    return v < 1.0f ? d : -__builtin_amdgcn_exp2f(-v);
}

__device__ __forceinline__ bool is_decay(float k) { return (int32_t)__float_as_uint(k) < 0; }

// a h
__device__ __forceinline__ float decayed(float k, float h) { return __builtin_fmaf(-k, h, is_decay(k) ? 0.0f : h); }

// 1 - a^2
__device__ __forceinline__ float lost_power(float k) { return __builtin_fmaf(-k, k, is_decay(k) ? 1.0f : 2.0f * k); }

// log(1 + exp(v)): 2 atanh(e / (2 + e)) where e is small (left out: 2^-28 of it),
// v itself where it is large.
__device__ __forceinline__ float softplus(float v) {
    const float e = expf(v), z = e / (2.0f + e), z2 = z * z;
    const float small = 2.0f * z * (1.0f + z2 * (0.33333333f + z2 * (0.2f + z2 * 0.14285714f)));
    return v > 20.0f ? v : e < 0.25f ? small : logf(1.0f + e);
}

// scale * softplus(decay) / log 2, finite so that a closed gate is a decay of 1.
__device__ __forceinline__ float decay_rate(float decay, float scale) {
    const float k = scale * softplus(decay) * 1.44269504f;
    return k > 1e30f ? 1e30f : k;
}

// sigmoid(v) / softplus(v), 1 in the limit where both underflow.
__device__ __forceinline__ float softplus_slope(float v) {
    return v < -16.0f ? 1.0f : 1.0f / ((1.0f + expf(-v)) * softplus(v));
}

// ---------------------------------------------------------------------------
// Runs and their composition
// ---------------------------------------------------------------------------
struct Run {
    f32x2 p, h;  // state behind = p * state before + h
};

__device__ __forceinline__ Run compose(const Run& first, const Run& then) {
    return {first.p * then.p, then.p * first.h + then.h};
}

__device__ __forceinline__ f32x2 through(const Run& run, f32x2 state) { return run.p * state + run.h; }

// The value of the wave's two rows of 32 lanes, in all lanes.
__device__ __forceinline__ void wave_rows(float v, float& low, float& high) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    low = __uint_as_float(s[0]);
    high = __uint_as_float(s[1]);
}

struct TileRuns {
    Run before;  // this thread's part of the tile that comes before its run
    Run all;     // the whole tile
};

// Composes the runs of the threads along the frames (REVERSE: last first).
template <int SEGS, bool REVERSE>
__device__ __forceinline__ TileRuns tile_runs(const Run& run, float (*lds)[2][kScanCols]) {
    const Run one = {f32x2(1.0f), f32x2(0.0f)};
    if constexpr (SEGS == 1) return {one, run};
    Run low, high;
#pragma unroll
    for (int e = 0; e < kScanPair; ++e) {
        float l, h;
        wave_rows(run.p[e], l, h);
        low.p[e] = l, high.p[e] = h;
        wave_rows(run.h[e], l, h);
        low.h[e] = l, high.h[e] = h;
    }
    const Run &first = REVERSE ? high : low, &second = REVERSE ? low : high;
    const bool upper = threadIdx.x % 64 >= kScanLanes, later = REVERSE ? !upper : upper;
    Run before = {later ? first.p : one.p, later ? first.h : one.h};
    const Run wave = compose(first, second);
    if constexpr (SEGS == 2) return {before, wave};
    const int at = threadIdx.x / 64, col = threadIdx.x % kScanLanes * kScanPair;
    if (!upper) {
        *(f32x2*)&lds[at][0][col] = wave.p;
        *(f32x2*)&lds[at][1][col] = wave.h;
    }
    __syncthreads();
    Run all = one, mine = one;
#pragma unroll
    for (int q = 0; q < kScanWaves; ++q) {
        const int w = REVERSE ? kScanWaves - 1 - q : q;
        const Run next = {*(const f32x2*)&lds[w][0][col], *(const f32x2*)&lds[w][1][col]};
        if (w == at) mine = all;
        all = q ? compose(all, next) : next;
    }
    return {compose(mine, before), all};
}

// A published (P, H): P is a product of decays, so its sign bit is free to say
// that the word holds something (cleared words are 0).  One 64-bit access at
// device scope, which passes the XCDs' own L2 caches, needs no order among words.
__device__ __forceinline__ void publish(uint64_t* word, float p, float h) {
    const uint64_t v = (uint64_t)__float_as_uint(h) << 32 | __float_as_uint(p) | 0x80000000u;
    __hip_atomic_store(word, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint64_t peek(const uint64_t* word) {
    return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What `count` published words in a row compose to, for each thread's channels.
// Each of the 4 waves takes a quarter of them, a lane for each channel; the
// quarters are composed in order.  Every word read here belongs to a workgroup
// that has started.
__device__ __forceinline__ Run fold_words(const uint64_t* words, int count, float (*lds)[2][kScanCols]) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int each = (count + kScanWaves - 1) / kScanWaves;
    const int first = wave * each, last = first + each < count ? first + each : count;
    float p = 1.0f, h = 0.0f;
    int polls = kScanPolls;  // in all
    constexpr int kFly = 4;  // reads in flight together
    for (int k = first; k < last; k += kFly) {
        uint64_t v[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) v[j] = k + j < last ? peek(words + (int64_t)(k + j) * kScanCols + lane) : 0;
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            if (k + j >= last) break;
            for (; (uint32_t)v[j] == 0 && polls > 0; --polls) {
                __builtin_amdgcn_s_sleep(1);
                v[j] = peek(words + (int64_t)(k + j) * kScanCols + lane);
            }
            const bool there = (uint32_t)v[j] != 0;
            const float wp = there ? __uint_as_float((uint32_t)v[j] & 0x7fffffffu) : __builtin_nanf("");
            p *= wp;
            h = wp * h + __uint_as_float((uint32_t)(v[j] >> 32));
        }
    }
    lds[wave][0][lane] = p;
    lds[wave][1][lane] = h;
    __syncthreads();
    const int col = threadIdx.x % kScanLanes * kScanPair;
    Run all = {*(const f32x2*)&lds[0][0][col], *(const f32x2*)&lds[0][1][col]};
#pragma unroll
    for (int q = 1; q < kScanWaves; ++q)
        all = compose(all, {*(const f32x2*)&lds[q][0][col], *(const f32x2*)&lds[q][1][col]});
    return all;
}

// ---------------------------------------------------------------------------
// Where a thread works, and its loads and stores
// ---------------------------------------------------------------------------
struct ScanPlace {
    int64_t b;       // item
    int64_t len;     // its valid frames
    uint32_t chain;  // of the workgroup: item (or items) and column block
    uint32_t lane;   // the thread's first channel within the workgroup's 64
    int seg, first, have;  // first: the workgroup's first channel
};

template <int SEGS>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a, uint32_t chain) {
    ScanPlace p;
    const int row = threadIdx.x / kScanLanes;
    const uint32_t rest = chain / (uint32_t)a.col_blocks;
    p.chain = chain;
    p.first = (int)(chain - rest * a.col_blocks) * kScanCols;
    p.lane = threadIdx.x % kScanLanes * kScanPair;
    p.have = a.C - p.first - (int)p.lane;
    if (p.have <= 0) p.lane = 0;  // past the last channel: loads what is there, stores nothing
    p.seg = row % SEGS;
    p.b = (int64_t)rest * (kScanRows / SEGS);
    if constexpr (SEGS == 2) p.b += __builtin_amdgcn_readfirstlane(row / SEGS);  // one item a wave
    if constexpr (SEGS == 1) p.b += row;
    p.len = p.b < a.B ? item_length(a.lengths, p.b, a.T) : 0;
    return p;
}

// A thread's frames of a tensor in the tile that starts at `tile`: a uniform
// base for each frame and one 32-bit offset (a frame's stride is below 2^23
// elements).  Frames at or past the length (`valid` of the tile's are below it,
// at least one) read the last valid one.
template <typename S, bool TAIL, bool STREAM, int FR>
__device__ __forceinline__ void load_run(pair_raw<S> out[FR], const void* base, const FrameStride& s,
                                         const ScanPlace& p, int64_t t0, int valid, bool full) {
    const char* tile = (const char*)((const S*)base + p.b * s.item + t0 * s.frame + p.first);
    const uint32_t step = (uint32_t)s.frame * (uint32_t)sizeof(S), lane = p.lane * (uint32_t)sizeof(S);
    const uint32_t at = p.seg * FR * step + lane;
    if (full) {
#pragma unroll
        for (int f = 0; f < FR; ++f) out[f] = load_pair<S, TAIL, STREAM>((const S*)(tile + (uint32_t)f * step + at), p.have);
    } else {
        const uint32_t most = (uint32_t)(valid - 1) * step + lane;
#pragma unroll
        for (int f = 0; f < FR; ++f) out[f] = load_pair<S, TAIL, STREAM>((const S*)(tile + min(at + f * step, most)), p.have);
    }
}

// The frames before those, one earlier each; frame 0 reads itself in place of the
// one before it.
template <typename S, bool TAIL, bool STREAM, int FR>
__device__ __forceinline__ void load_before(pair_raw<S> out[FR], const void* base, const FrameStride& s,
                                            const ScanPlace& p, int64_t t0, int valid, bool full) {
    if (t0 > 0) return load_run<S, TAIL, STREAM, FR>(out, base, s, p, t0 - 1, valid, full);
    const char* tile = (const char*)((const S*)base + p.b * s.item + p.first);
    const uint32_t step = (uint32_t)s.frame * (uint32_t)sizeof(S), lane = p.lane * (uint32_t)sizeof(S);
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int t = min(p.seg * FR + f, valid);
        out[f] = load_pair<S, TAIL, STREAM>((const S*)(tile + ((t > 0 ? t - 1 : 0) * step + lane)), p.have);
    }
}

// What the frames at or past the length become: the bits of two stored values.
template <typename S, int FR>
__device__ __forceinline__ void mask_run(pair_raw<S> out[FR], const ScanPlace& p, int valid, uint32_t dead) {
#pragma unroll
    for (int f = 0; f < FR; ++f)
        if (p.seg * FR + f >= valid) out[f] = dead;
}

// Writes a thread's frames of the tile: zeros past the length, none at or past
// `rows`.
template <typename S, bool TAIL, int FR>
__device__ __forceinline__ void store_run(void* base, const FrameStride& s, const ScanPlace& p, int64_t t0, int valid,
                                          int rows, bool full, const pair_raw<S> v[FR]) {
    if (p.have <= 0) return;
    char* tile = (char*)((S*)base + p.b * s.item + t0 * s.frame + p.first);
    const uint32_t step = (uint32_t)s.frame * (uint32_t)sizeof(S);
    const uint32_t at = p.seg * FR * step + p.lane * (uint32_t)sizeof(S);
    if (full) {
#pragma unroll
        for (int f = 0; f < FR; ++f) store_pair<S, TAIL>((S*)(tile + (uint32_t)f * step + at), p.have, v[f]);
    } else {
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            const int t = p.seg * FR + f;
            pair_raw<S> q = {};
            if (t < valid) q = v[f];
            if (t < rows) store_pair<S, TAIL>((S*)(tile + (uint32_t)f * step + at), p.have, q);
        }
    }
}

// Whether a workgroup goes through several tiles in turn: the other forms are for
// sequences of one tile at most, and for linked tiles.
template <int SEGS, int FR, bool LINKED>
constexpr bool scan_loops() {
    return !LINKED && SEGS == kScanRows && FR == kScanRun;
}

template <typename S>
constexpr uint32_t closed_gate() {  // -infinity, in each stored value
    return sizeof(S) == 4 ? 0xff800000u : 0xff80ff80u;
}

__device__ __forceinline__ f32x2 load_state(const float* base, int64_t row, int32_t C, const ScanPlace& p) {
    const int64_t at = row * C + p.first + p.lane;
    f32x2 v = {0.0f, 0.0f};
    if (base && p.have > 0) v[0] = base[at];
    if (base && p.have > 1) v[1] = base[at + 1];
    return v;
}

__device__ __forceinline__ void store_state(float* base, int64_t row, int32_t C, const ScanPlace& p, f32x2 v) {
    const int64_t at = row * C + p.first + p.lane;
    if (p.have > 0) base[at] = v[0];
    if (p.have > 1) base[at + 1] = v[1];
}

// What a workgroup finds out once for all its threads: the tile that it takes of
// its chain, in the order of the chain, and the decays of its 64 channels.
struct ScanShared {
    float decay[kScanCols], rate[kScanCols];
    int ticket;
};

template <bool LINKED>
__device__ __forceinline__ void begin_scan(const ScanArgs& a, const ScanPlace& p, ScanShared& s) {
    if (LINKED && threadIdx.x == 0)
        s.ticket = (int)__hip_atomic_fetch_add(a.tickets + (int64_t)p.chain * kScanTicket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (threadIdx.x / 64 == 1) {
        const int lane = threadIdx.x % 64;
        const float decay = p.first + lane < a.C ? a.decay[p.first + lane] : 0.0f;
        s.decay[lane] = decay;
        s.rate[lane] = decay_rate(decay, a.scale);
    }
    __syncthreads();
}

// The frames of a tile.
struct TileSpan {
    int64_t t0;
    int rows, valid;  // those of the sequence, those below the length
    bool full;
};

__device__ __forceinline__ TileSpan tile_span(const ScanArgs& a, const ScanPlace& p, int64_t tile, int frames) {
    TileSpan s;
    s.t0 = tile * frames;
    const int64_t left = p.len - s.t0, size = a.T - s.t0;
    s.rows = size < frames ? (int)size : frames;
    s.valid = left < 0 ? 0 : left < s.rows ? (int)left : s.rows;
    s.full = s.valid == frames;
    return s;
}

// The first row of threads publishes a run of the workgroup's 64 channels.
__device__ __forceinline__ void publish_run(uint64_t* words, const Run& run) {
    if (threadIdx.x >= kScanLanes) return;
#pragma unroll
    for (int e = 0; e < kScanPair; ++e) publish(words + threadIdx.x * kScanPair + e, run.p[e], run.h[e]);
}

// The state that enters a tile whose runs are known, and `carry`, the one that
// leaves it (LINKED: both 0 unless `wanted`).  Where tiles are linked, the chain's first one takes up
// the state that enters the chain and hands it on in its word, so nothing reads
// that state after the last tile has written its own.  The last tile of 16
// publishes what they compose to: tile `at` reads at / 16 such words and those
// of its own group.
template <bool LINKED>
__device__ __forceinline__ f32x2 enter_tile(const ScanArgs& a, const ScanPlace& p, const Run& all, int at, bool wanted,
                                            f32x2& carry, float (*lds)[kScanWaves][2][kScanCols]) {
    const f32x2 zero = {0.0f, 0.0f};
    if constexpr (!LINKED) {
        const f32x2 in = carry;
        carry = through(all, carry);
        return in;
    }
    const int group = at / kScanGroup, of_group = at % kScanGroup;
    uint64_t* words = a.words + (int64_t)p.chain * (a.tiles + a.tiles / kScanGroup) * kScanCols;
    uint64_t* groups = words + (int64_t)a.tiles * kScanCols;
    if (at == 0) {
        const f32x2 in = carry;
        carry = through(all, carry);
        publish_run(words, {zero, carry});
        return in;
    }
    publish_run(words + (int64_t)at * kScanCols, all);
    const bool closes = of_group == kScanGroup - 1;
    if (!wanted && !closes) return zero;
    Run before = {f32x2(1.0f), zero};
    if (of_group > 0) before = fold_words(words + (int64_t)group * kScanGroup * kScanCols, of_group, lds[0]);
    if (closes) publish_run(groups + (int64_t)group * kScanCols, compose(before, all));
    if (!wanted) return zero;
    if (group > 0) before = compose(fold_words(groups, group, lds[1]), before);
    carry = through(all, before.h);  // the first tile's word has P = 0: H is the state
    return before.h;
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <typename S, bool TAIL, int SEGS, int FR, bool LINKED>
__global__ __launch_bounds__(kScanThreads) void scan_fwd_kernel(const ScanArgs a) {
    constexpr int kTileFrames = SEGS * FR;
    __shared__ float lds[LINKED ? 3 : 2][kScanWaves][2][kScanCols];
    __shared__ ScanShared shared;
    const uint32_t chains = LINKED ? gridDim.x / (uint32_t)a.tiles : 0;
    const ScanPlace p = scan_place<SEGS>(a, LINKED ? blockIdx.x % chains : blockIdx.x);
    begin_scan<LINKED>(a, p, shared);
    if (p.b >= a.B) return;  // SEGS < 8, where no thread waits for another wave from here on
    int tile = LINKED ? __builtin_amdgcn_readfirstlane(shared.ticket) : 0;
    if (LINKED && tile >= a.tiles) return;  // given out by another call on this workspace
    const int end = scan_loops<SEGS, FR, LINKED>() ? a.tiles : tile + 1;
    const f32x2 rate = *(const f32x2*)&shared.rate[p.lane];
    f32x2 carry = tile == 0 ? load_state(a.start, p.b, a.C, p) : f32x2(0.0f);
    int turn = 0;
    for (; tile < end; ++tile) {
        const TileSpan span = tile_span(a, p, tile, kTileFrames);
        const int valid = span.valid;
        f32x2 k[FR], u[FR];
        Run all = {f32x2(1.0f), f32x2(0.0f)}, before = all;
        if (valid > 0) {
            pair_raw<S> xr[FR], rr[FR], gr[FR];
            load_run<S, TAIL, false, FR>(rr, a.r, a.rs, p, span.t0, valid, span.full);
            load_run<S, TAIL, false, FR>(gr, a.g, a.gs, p, span.t0, valid, span.full);
            load_run<S, TAIL, false, FR>(xr, a.x, a.xs, p, span.t0, valid, span.full);
            if (!span.full) {  // a decay of 1 and no input
                mask_run<S, FR>(rr, p, valid, closed_gate<S>());
                mask_run<S, FR>(xr, p, valid, 0);
            }
            f32x2 w = {0.0f, 0.0f}, h = w;
#pragma unroll
            for (int f = 0; f < FR; ++f) {
#pragma unroll
                for (int e = 0; e < kScanPair; ++e) {
                    const float wf = rate[e] * sigmoid<S>(pair_at<S>(rr[f], e));
                    const float kf = decay_factor(wf);
                    const float m = __builtin_amdgcn_sqrtf(lost_power(kf));
                    const float uf = m * (sigmoid<S>(pair_at<S>(gr[f], e)) * pair_at<S>(xr[f], e));
                    k[f][e] = kf;
                    u[f][e] = uf;
                    w[e] += wf;
                    h[e] = decayed(kf, h[e]) + uf;
                }
            }
            const Run run = {{__builtin_amdgcn_exp2f(-w[0]), __builtin_amdgcn_exp2f(-w[1])}, h};
            const TileRuns t = tile_runs<SEGS, false>(run, lds[turn]);
            turn ^= 1;
            all = t.all;
            before = t.before;
        }
        const bool wanted = valid > 0 || (a.end && tile == a.tiles - 1);
        f32x2 h = through(before, enter_tile<LINKED>(a, p, all, tile, wanted, carry, lds + 1));
        pair_raw<S> y[FR] = {};
        if (valid > 0) {
#pragma unroll
            for (int f = 0; f < FR; ++f) {
#pragma unroll
                for (int e = 0; e < kScanPair; ++e) h[e] = decayed(k[f][e], h[e]) + u[f][e];
                y[f] = pack_pair<S>(h);
            }
        }
        store_run<S, TAIL, FR>(a.y, a.ys, p, span.t0, valid, span.rows, span.full, y);
    }
    if (a.end && end >= a.tiles && p.seg == 0) store_state(a.end, p.b, a.C, p, carry);
}

// ---------------------------------------------------------------------------
// Backward in time, G_t = dy_t + a_{t+1} G_{t+1}: the runs hand a_t G_t on to
// the frames before them.
// ---------------------------------------------------------------------------
//
// Waves that share a SIMD at least: linked tiles 3 (168 registers; bf16 takes 135,
// [16,750,1024] 58.9 us against 61.1 with 4, [2,6001,512] 39.0 and 40.9; float spills 7,
// and 86.5 against 90.2 with 2, [8,375,1024] 28.4 and 33.2, [2,6001,512] 55.1 and 53.3), in
// turn 2 (bf16 176 registers, 180 us for [16,1500,2048] against 182 with 3; float 217).
constexpr int scan_bwd_waves(bool linked) { return linked ? 3 : 2; }

template <typename S, bool TAIL, int SEGS, int FR, bool LINKED>
__global__ __launch_bounds__(kScanThreads, scan_bwd_waves(LINKED)) void scan_bwd_kernel(const ScanArgs a) {
    constexpr int kTileFrames = SEGS * FR;
    __shared__ float lds[LINKED ? 3 : 2][kScanWaves][2][kScanCols];
    __shared__ float column[kScanRows][kScanCols];
    __shared__ ScanShared shared;
    const uint32_t chains = LINKED ? gridDim.x / (uint32_t)a.tiles : 0;
    const ScanPlace p = scan_place<SEGS>(a, LINKED ? blockIdx.x % chains : blockIdx.x);
    const bool item = p.b < a.B;
    begin_scan<LINKED>(a, p, shared);
    pair_raw<S> rr[FR], dyr[FR], xr[FR], gr[FR], prev[FR];
    // A step by itself, which the compiler does not join with what is made of them: in
    // turn bf16 [16,1500,2048] 180 us and 182, [64,200,512] 36.6 and 37.2, float alike.
    const auto load = [&](const TileSpan& s) {
        if (s.valid <= 0) return;
        load_run<S, TAIL, true, FR>(rr, a.r, a.rs, p, s.t0, s.valid, s.full);
        load_run<S, TAIL, true, FR>(dyr, a.dy, a.dys, p, s.t0, s.valid, s.full);
        load_run<S, TAIL, true, FR>(xr, a.x, a.xs, p, s.t0, s.valid, s.full);
        load_run<S, TAIL, true, FR>(gr, a.g, a.gs, p, s.t0, s.valid, s.full);
        // the state before each frame: what the forward stored for the one in front of it
        load_before<S, TAIL, true, FR>(prev, a.yin, a.ys, p, s.t0, s.valid, s.full);
    };
    constexpr bool kSeveral = LINKED || scan_loops<SEGS, FR, LINKED>();
    int at = LINKED ? __builtin_amdgcn_readfirstlane(shared.ticket) : 0;  // in the order of the chain: the last tile is first
    if (LINKED && at >= a.tiles) return;  // given out by another call on this workspace
    const int end = LINKED ? at + 1 : !item ? 0 : scan_loops<SEGS, FR, LINKED>() ? a.tiles : 1;
    const int row = LINKED ? (int)(p.chain / (uint32_t)a.col_blocks) * a.tiles + at : (int)(p.chain / (uint32_t)a.col_blocks);
    const f32x2 rate = *(const f32x2*)&shared.rate[p.lane];
    f32x2 unrate;  // w * unrate is the gate
#pragma unroll
    for (int e = 0; e < kScanPair; ++e) unrate[e] = __builtin_amdgcn_rcpf(fmaxf(rate[e], 0x1p-126f));
    f32x2 carry = item && at == 0 ? load_state(a.start, p.b, a.C, p) : f32x2(0.0f), sum = {0.0f, 0.0f};
    int turn = 0;
    for (; at < end; ++at) {
        const TileSpan span = tile_span(a, p, kSeveral ? a.tiles - 1 - at : 0, kTileFrames);
        const int valid = span.valid;
        load(span);
        f32x2 k[FR], w[FR];
        Run all = {f32x2(1.0f), f32x2(0.0f)}, before = all;
        if (valid > 0) {
            if (!span.full) {  // a decay of 1 and no gradient
                mask_run<S, FR>(rr, p, valid, closed_gate<S>());
                mask_run<S, FR>(dyr, p, valid, 0);
            }
            f32x2 sw = {0.0f, 0.0f}, c = sw;
#pragma unroll
            for (int f = FR - 1; f >= 0; --f) {
#pragma unroll
                for (int e = 0; e < kScanPair; ++e) {
                    const float wf = rate[e] * sigmoid<S>(pair_at<S>(rr[f], e));
                    w[f][e] = wf;
                    k[f][e] = decay_factor(wf);
                    c[e] = decayed(k[f][e], pair_at<S>(dyr[f], e) + c[e]);
                    sw[e] += wf;
                }
            }
            const Run run = {{__builtin_amdgcn_exp2f(-sw[0]), __builtin_amdgcn_exp2f(-sw[1])}, c};
            const TileRuns t = tile_runs<SEGS, true>(run, lds[turn]);
            turn ^= 1;
            all = t.all;
            before = t.before;
        }
        const bool wanted = valid > 0 || (a.end && at == a.tiles - 1);
        f32x2 c = through(before, enter_tile<LINKED>(a, p, all, at, wanted, carry, lds + 1));
        if (valid > 0) {
            const bool start = span.t0 == 0 && p.seg == 0;
            const f32x2 h0 = start ? load_state(a.h0, p.b, a.C, p) : f32x2(0.0f);
#pragma unroll
            for (int f = FR - 1; f >= 0; --f) {
                f32x2 dx, dr, dg;
#pragma unroll
                for (int e = 0; e < kScanPair; ++e) {
                    const float G = pair_at<S>(dyr[f], e) + c[e];
                    const float eg = exp_minus<S>(pair_at<S>(gr[f], e)), gate = sigmoid_of(eg);
                    // again, rather than kept: float [32,1500,512] linked 168 us, 176 with it in registers
                    // ([16,750,1024] 88 and 94; in turn [16,1500,2048] 331 and 330, bf16 181 and 180)
                    const float er = exp_minus<S>(pair_at<S>(rr[f], e));
                    const float h = f == 0 && start ? h0[e] : pair_at<S>(prev[f], e);
                    const float kf = k[f][e], z = lost_power(kf);                           // 1 - a^2 = m^2
                    const float rs = __builtin_amdgcn_rsqf(z > 0x1p-126f ? z : 0x1p-126f);  // m = z rs, 0 where z is
                    const float a2 = is_decay(kf) ? kf * kf : 1.0f - z;
                    dx[e] = G * (z * rs) * gate;
                    const float t = dx[e] * pair_at<S>(xr[f], e);
                    dg[e] = t * shut_of(eg, gate);
                    c[e] = decayed(kf, G);
                    // G i x a^2 / m = t a^2 / m^2
                    const float q = w[f][e] * (t * (a2 * (rs * rs)) - c[e] * h);
                    dr[e] = 0.69314718f * q * shut_of(er, w[f][e] * unrate[e]);
                    sum[e] += span.full || p.seg * FR + f < valid ? q : 0.0f;
                }
                xr[f] = pack_pair<S>(dx);  // the gradients take their inputs' places
                rr[f] = pack_pair<S>(dr);
                gr[f] = pack_pair<S>(dg);
            }
        }
        if (a.dx) store_run<S, TAIL, FR>(a.dx, a.dxs, p, span.t0, valid, span.rows, span.full, xr);
        if (a.dr) store_run<S, TAIL, FR>(a.dr, a.drs, p, span.t0, valid, span.rows, span.full, rr);
        if (a.dg) store_run<S, TAIL, FR>(a.dg, a.dgs, p, span.t0, valid, span.rows, span.full, gr);
    }
    if (a.end && end >= a.tiles && item && p.seg == 0) store_state(a.end, p.b, a.C, p, carry);
    if (!a.partial) return;
    const int mine = threadIdx.x / kScanLanes, lane = threadIdx.x % kScanLanes;
#pragma unroll
    for (int e = 0; e < kScanPair; ++e) column[mine][lane * kScanPair + e] = 0.69314718f * sum[e];
    __syncthreads();
    if (mine != 0) return;
    double* out = a.partial + (int64_t)row * a.C + p.first + p.lane;
#pragma unroll
    for (int e = 0; e < kScanPair; ++e) {
        double t = 0.0;
        for (int q = 0; q < kScanRows; ++q) t += column[q][lane * kScanPair + e];
        if (e < p.have) out[e] = t * softplus_slope(shared.decay[p.lane + e]);
    }
}

// Nothing taken, nothing published.
__global__ __launch_bounds__(kScanThreads) void scan_clear_kernel(u32x4* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kScanThreads)
        p[i] = u32x4(0u);
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
// segs: threads along the frames of an item in a workgroup; run: frames of each
// in a tile; linked: a workgroup for each tile.
struct ScanPlan {
    int segs, run;
    bool linked;
    int64_t tiles, row_blocks, col_blocks;  // row_blocks: of one column block, tiles among them where linked
};

// Runs of 16 frames (forward only: the gradients' would not leave registers for
// two waves a SIMD) make one tile of up to 128 frames, and in longer sequences
// halve the words that a tile reads of those before it; with 8, sequences waste
// less where they end.  us for 16 and 8: bf16 [16,750,1024] with lengths of half
// to all 29.3 and 27.0, [64,750,256] 29.0 and 27.3.  Two sequences of 512 channels, all
// valid: 1000 to 2000 frames alike (14.1), 4000 bf16 16.7 and 14.8, float 19.9 and 18.9,
// 6001 20.5 and 20.1, 23.8 and 25.6, one of 20000 32.0 and 29.9, 43.3 and 44.6; with
// lengths 6001 19.5 and 20.1, 22.6 and 24.4, 20000 in its first half 23.1 and 23.3, 26.6 and
// 28.4.  One bound serves both types: float gains by it from 6000 frames on, bf16 does
// not, and around 4000 both lose a microsecond or two.
//
// Linked or in turn, us: 256 chains, [16,750,1024] bf16 31 and 35, float 44 and 57;
// 512 chains, [16,1500,2048] bf16 102 and 100, float 164 and 158, [32,330,1024] 28 and
// 26.  Gradients: [16,1500,2048] bf16 190 and 181, float 337 and 330, [32,330,1024] 55
// and 52.  One chain a CU, all of one length, is near in turn (bf16 [16,750,1024] 58.9 and
// 59.3, float 87.4 and 86.5), but not with lengths of half to all (51 and 57), nor are
// a few more chains (320, [20,750,1024], 69 and 90, float 104 and 127) or fewer (192,
// [24,1500,512], 84 and 105).
// Up to 4 tiles in turn save the launch that clears the words: calls of [8,256,512]
// bf16 14.9 and 11.2, [1,200,64] 15.0 and 11.1 (gradients 23.2 and 22.0, 23.1 and 21.0);
// float [8,256,512] loses by it (15.2 and 16.4, gradients 23.8 and 27.9), [1,200,64] does
// not (15.0 and 13.4, 23.3 and 24.1).
static ScanPlan scan_plan(const ScanShape& s, bool backward) {
    ScanPlan p = {};
    const int64_t one = kScanRows * kScanRun;
    p.col_blocks = (s.C + kScanCols - 1) / kScanCols;
    const bool many = s.B * p.col_blocks >= 512;
    p.run = s.T == 1 ? 1 : kScanRun;
    if (!backward && s.T > one && (s.T <= 2 * one || (!many && s.T > 1024))) p.run = kScanLongRun;
    p.segs = s.T <= p.run ? 1 : s.T <= 2 * p.run ? 2 : kScanRows;
    p.tiles = (s.T + p.segs * p.run - 1) / (p.segs * p.run);
    const int64_t per = kScanRows / p.segs;
    p.row_blocks = (s.B + per - 1) / per;
    p.linked = p.tiles > 4 && !many;
    if (p.linked) p.row_blocks *= p.tiles;
    return p;
}

static int64_t scan_chains(const ScanPlan& p) { return p.row_blocks / p.tiles * p.col_blocks; }

bool dwscan_fits(const ScanShape& s) {
    if (!product_below((int64_t)1 << 58, {s.B, s.T, s.C})) return false;
    for (const bool backward : {false, true}) {
        const ScanPlan p = scan_plan(s, backward);
        if (!product_below((int64_t)1 << 24, {p.row_blocks, p.col_blocks})) return false;
    }
    return true;
}

// Tickets and words of a linked plan.
static size_t scan_ticket_bytes(const ScanPlan& p) {
    return p.linked ? (size_t)(scan_chains(p) * kScanTicket) * sizeof(uint32_t) : 0;
}

static size_t scan_link_bytes(const ScanPlan& p) {
    if (!p.linked) return 0;
    return scan_ticket_bytes(p) + (size_t)(scan_chains(p) * (p.tiles + p.tiles / kScanGroup) * kScanCols) * sizeof(uint64_t);
}

static int64_t scan_partial_rows(const ScanPlan& p) {
    const int64_t chunks = partial_reduce_chunks(p.row_blocks);
    return p.row_blocks + (chunks > 1 ? chunks : 1);
}

size_t dwscan_fwd_workspace(const ScanShape& s) { return scan_link_bytes(scan_plan(s, false)); }

size_t dwscan_bwd_workspace(const ScanShape& s) {
    const ScanPlan p = scan_plan(s, true);
    return scan_link_bytes(p) + (size_t)(scan_partial_rows(p) * s.C) * sizeof(double);
}

static ScanArgs scan_args(const ScanPtrs& p, const ScanShape& s, const ScanPlan& plan, void* workspace) {
    ScanArgs a = {};
    a.x = p.x, a.r = p.r, a.g = p.g, a.decay = p.decay, a.lengths = p.lengths;
    a.xs = s.x, a.rs = s.r, a.gs = s.g, a.ys = s.y;
    a.dys = s.dy, a.dxs = s.dx, a.drs = s.dr, a.dgs = s.dg;
    a.B = s.B, a.T = s.T, a.C = (int32_t)s.C, a.scale = s.scale;
    a.col_blocks = (int32_t)plan.col_blocks, a.tiles = (int32_t)plan.tiles;
    if (plan.linked) {
        a.tickets = (uint32_t*)workspace;
        a.words = (uint64_t*)((char*)workspace + scan_ticket_bytes(plan));
    }
    return a;
}

template <bool BACK, typename S, bool TAIL, int SEGS, int FR, bool LINKED>
static hipError_t launch_scan_kernel(const ScanPlan& plan, const ScanArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)(plan.row_blocks * plan.col_blocks));
    if constexpr (BACK)
        hipLaunchKernelGGL((scan_bwd_kernel<S, TAIL, SEGS, FR, LINKED>), grid, dim3(kScanThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((scan_fwd_kernel<S, TAIL, SEGS, FR, LINKED>), grid, dim3(kScanThreads), 0, stream, a);
    return hipGetLastError();
}

template <bool BACK, typename S, bool TAIL>
static hipError_t launch_scan_form(const ScanPlan& plan, const ScanArgs& a, hipStream_t stream) {
    if (plan.linked) {
        const int64_t n = (int64_t)(scan_link_bytes(plan) / sizeof(u32x4)), blocks = (n + kScanThreads - 1) / kScanThreads;
        hipLaunchKernelGGL(scan_clear_kernel, dim3((uint32_t)(blocks < 1024 ? blocks : 1024)), dim3(kScanThreads), 0,
                           stream, (u32x4*)a.tickets, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if constexpr (!BACK) {
            if (plan.run == kScanLongRun)
                return launch_scan_kernel<BACK, S, TAIL, kScanRows, kScanLongRun, true>(plan, a, stream);
        }
        return launch_scan_kernel<BACK, S, TAIL, kScanRows, kScanRun, true>(plan, a, stream);
    }
    if (plan.run == 1) return launch_scan_kernel<BACK, S, TAIL, 1, 1, false>(plan, a, stream);
    if (plan.segs == 1) return launch_scan_kernel<BACK, S, TAIL, 1, kScanRun, false>(plan, a, stream);
    if (plan.segs == 2) return launch_scan_kernel<BACK, S, TAIL, 2, kScanRun, false>(plan, a, stream);
    if constexpr (!BACK) {
        if (plan.run == kScanLongRun)
            return launch_scan_kernel<BACK, S, TAIL, kScanRows, kScanLongRun, false>(plan, a, stream);
    }
    return launch_scan_kernel<BACK, S, TAIL, kScanRows, kScanRun, false>(plan, a, stream);
}

template <bool BACK>
static hipError_t launch_scan(const ScanPlan& plan, const ScanArgs& a, bool bf16, hipStream_t stream) {
    const bool tail = a.C % kScanPair != 0;
    if (bf16 && tail) return launch_scan_form<BACK, uint16_t, true>(plan, a, stream);
    if (bf16) return launch_scan_form<BACK, uint16_t, false>(plan, a, stream);
    if (tail) return launch_scan_form<BACK, float, true>(plan, a, stream);
    return launch_scan_form<BACK, float, false>(plan, a, stream);
}

hipError_t launch_dwscan_fwd(const ScanPtrs& p, const ScanShape& s, void* y, float* h_last, void* workspace, bool bf16,
                             hipStream_t stream) {
    const ScanPlan plan = scan_plan(s, false);
    ScanArgs a = scan_args(p, s, plan, workspace);
    a.start = p.h0, a.y = y, a.end = h_last;
    return launch_scan<false>(plan, a, bf16, stream);
}

hipError_t launch_dwscan_bwd(const ScanPtrs& p, const ScanShape& s, const void* y, const void* dy, const float* dh_last,
                             void* dx, void* dr, void* dg, float* ddecay, float* dh0, void* workspace, bool bf16,
                             hipStream_t stream) {
    const ScanPlan plan = scan_plan(s, true);
    ScanArgs a = scan_args(p, s, plan, workspace);
    a.start = dh_last, a.h0 = p.h0, a.yin = y, a.dy = dy, a.dx = dx, a.dr = dr, a.dg = dg, a.end = dh0;
    double* rows = (double*)((char*)workspace + scan_link_bytes(plan));
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
