// kv_attend.hpp -- argument block and tile arithmetic of the attention kernels.
#pragma once

#include "common.hpp"
#include "kv.hpp"

namespace tpl {
namespace kv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// A row's reference for its exponentials moves only when a score exceeds it
// by this many powers of two, so that most tiles leave the accumulators as
// they are; weights reach 2^8 then, far from any type's end.
constexpr float kSlack = 8.0f;
// Weights that are multiplied as fp16 numbers have a reference this much under
// the largest score: they reach 2^15, and the ones that fp16 can no longer
// hold are under 2^-32 of the largest instead of 2^-25.  100000 tokens of the
// latter are 0.3 % of a row's sum, which counts them all.
template <typename V>
__device__ constexpr float lift() { return std::is_same<V, Fp16>::value ? 7.0f : 0.0f; }

struct AttendArgs {
    tpl_kv_cache c;
    tpl_kv_batch g;
    tpl_kv_query a;
    int* counters;     // workspace: parts of a row tile that are there, zero between calls
    float* parts;      // workspace: partial results
    FastDiv div_page, div_block, div_group;
    float factor;      // scale * log2 e
    int32_t group;     // query heads that share one of the cache
    int32_t cap;       // tokens that a table row can hold
    // Split kernel (few rows a sequence)
    int32_t few;       // it takes sequences of at most this many rows (new tokens * group)
    int32_t shares;    // its workgroups for each set of heads
    int32_t heads_log; // a workgroup takes 1 << heads_log of the cache's heads
    // Tile kernel (many rows a sequence)
    int32_t tile_rows;     // 128 or 256
    int32_t tile_tokens;   // new tokens of a row tile
    int32_t tiles;         // bound on the row tiles, grid order
    int32_t splits;        // parts of each tile's tokens
    float* tile_parts;
};

// Where a token stands that is not there: beyond every position.
constexpr int kNowhere = 0x7fffff00;

// The tokens that a range of rows sees, as groups of 16 consecutive tokens:
// first `na` groups from token 0 (the sinks, where they lie before the
// window), then groups from `lo` on.
struct Span {
    int na, lo, n;
    __device__ __forceinline__ int base(int t) const { return t < na ? t * 16 : lo + (t - na) * 16; }
};

__device__ __forceinline__ Span span_of(const AttendArgs& p, int first_pos, int last_pos) {
    Span s;
    s.na = 0;
    s.lo = 0;
    int hi = last_pos + 1;
    hi = hi < p.cap ? hi : p.cap;
    if (p.a.window > 0 && first_pos >= p.a.window) {
        const int lo = first_pos - p.a.window + 1;
        const int sink = p.a.sinks < lo ? p.a.sinks : lo;
        const int na = (sink + 15) >> 4, from = lo >> 4;
        if (na < from) {
            s.na = na;
            s.lo = from * 16;
        }
    }
    const int end = (hi + 15) >> 4, from = s.lo >> 4;
    // Pages beyond the table's width are not there: the sinks end at hi too.
    if (s.na > end) s.na = end;
    s.n = s.na + (end > from ? end - from : 0);
    return s;
}

// A number that no kernel of the call writes, at an address that is the same
// in every lane: by the scalar path.
template <typename X>
__device__ __forceinline__ X scalar(const X* p) {
    return *(const __attribute__((address_space(4))) X*)(uintptr_t)p;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Maximum and sum of a value over lanes that differ in bit 4 or 5.
__device__ __forceinline__ float2 swap32(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];   // a bit cast of a vector's element itself reads its first
    return make_float2(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float2 swap16(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const u32x2 r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return make_float2(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float max32(float x) { const float2 r = swap32(x); return fmaxf(r.x, r.y); }
__device__ __forceinline__ float max16(float x) { const float2 r = swap16(x); return fmaxf(r.x, r.y); }
__device__ __forceinline__ float sum32(float x) { const float2 r = swap32(x); return r.x + r.y; }
__device__ __forceinline__ float sum16(float x) { const float2 r = swap16(x); return r.x + r.y; }

// A number that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return ((uint64_t)hi << 32) | lo;
}

// Groups of 16 tokens of a split kernel's step where its 4 waves, 2 groups
// each, are on one head.
constexpr int kStepGroups = 8;

struct FewSeq {
    Seq s;
    Span span;
    int tiles;      // row tiles
    int steps;      // steps of one row tile, at least 1
    __device__ __forceinline__ uint64_t all() const { return (uint64_t)tiles * (uint32_t)steps; }
};

template <int ROWS>
__device__ __forceinline__ FewSeq few_seq(const AttendArgs& p, int b) {
    FewSeq f;
    f.s = read_seq(p.g, b);
    const int64_t rows = (int64_t)f.s.n * p.group;
    if (rows > p.few) f.s.n = 0;
    f.tiles = f.s.n ? (int)((rows + ROWS - 1) / ROWS) : 0;
    f.span = span_of(p, f.s.length - f.s.n, f.s.length - 1);
    const int log = 3 - p.heads_log;   // kStepGroups a wave's share of them
    f.steps = (f.span.n + (1 << log) - 1) >> log;
    if (f.steps < 1) f.steps = 1;
    return f;
}

__device__ __forceinline__ FewSeq uniform(FewSeq f) {
    f.s.row0 = uniform(f.s.row0);
    f.s.n = uniform(f.s.n);
    f.s.length = uniform(f.s.length);
    f.span.na = uniform(f.span.na);
    f.span.lo = uniform(f.span.lo);
    f.span.n = uniform(f.span.n);
    f.tiles = uniform(f.tiles);
    f.steps = uniform(f.steps);
    return f;
}

__device__ __forceinline__ FewSeq from_lane(FewSeq f, int lane) {
    f.s.row0 = __builtin_amdgcn_readlane(f.s.row0, lane);
    f.s.n = __builtin_amdgcn_readlane(f.s.n, lane);
    f.s.length = __builtin_amdgcn_readlane(f.s.length, lane);
    f.span.na = __builtin_amdgcn_readlane(f.span.na, lane);
    f.span.lo = __builtin_amdgcn_readlane(f.span.lo, lane);
    f.span.n = __builtin_amdgcn_readlane(f.span.n, lane);
    f.tiles = __builtin_amdgcn_readlane(f.tiles, lane);
    f.steps = __builtin_amdgcn_readlane(f.steps, lane);
    return f;
}

// Steps of a share: an equal part of them all, but no less than keeps the
// joining of a tile's parts (8 at a time) short beside its steps.  An average
// sequence of n steps takes about c + n / (8 c) of a step's time with c a
// share, least at c = sqrt(n / 8).
__device__ __forceinline__ int share_of(const AttendArgs& p, int total) {
    const int equal = (int)(((uint32_t)total + (uint32_t)p.shares - 1) / (uint32_t)p.shares);
    const int short_ = (int)__builtin_sqrtf((float)total / (float)(p.g.batch * 8)) + 1;
    return equal > short_ ? equal : short_;
}

// The batch's steps in order: every workgroup sums them for itself (one
// load's latency for up to 256 sequences, and no barrier for up to 64).
// Gives the total, the size of a share, and the sequence that this share
// begins in (-1: none) with that sequence's own first step.  More steps than
// 31 bits hold can only be counted for sequences that claim one another's
// rows (the host refuses sizes that allow them otherwise): nothing is done.
template <int ROWS>
__device__ __forceinline__ int locate(const AttendArgs& p, int share, int* at_b, FewSeq* at_seq, int* at_step, int* chunk) {
    __shared__ uint64_t sums[4];
    __shared__ int found_step, found_b;
    __shared__ FewSeq found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool alone = p.g.batch <= 64;   // every wave counts them all
    const int per = alone ? 1 : (p.g.batch + 255) / 256, me = alone ? lane : tid;
    uint64_t mine = 0;
    FewSeq f = {};
    for (int i = 0; i < per; ++i) {
        const int b = me * per + i;
        if (b < p.g.batch) {
            f = few_seq<ROWS>(p, b);
            mine += f.all();
        }
    }
    uint64_t run = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    uint64_t total, before = run - mine;
    if (alone) {
        total = __shfl(run, 63);
    } else {
        if (lane == 63) sums[wave] = run;
        if (tid == 0) found_b = -1;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += sums[w];
            total += sums[w];
        }
    }
    total = uniform(total);
    *at_b = -1;
    *at_step = *chunk = 0;
    if (total == 0 || total > 0x7fffffffu) return 0;
    *chunk = uniform(share_of(p, (int)total));
    const uint64_t c = (uint64_t)share * (uint32_t)*chunk;
    const bool here = mine && before <= c && c < before + mine;
    if (alone) {
        const uint64_t m = __ballot(here);
        if (m) {
            const int from = __builtin_ctzll(m);
            *at_b = from;
            *at_seq = from_lane(f, from);
            *at_step = __builtin_amdgcn_readlane((int)before, from);
        }
        return (int)total;
    }
    if (here) {
        int b = tid;
        for (int i = 0; per > 1 && i < per; ++i) {
            b = tid * per + i;
            if (b >= p.g.batch) break;
            f = few_seq<ROWS>(p, b);
            if (c < before + f.all()) break;
            before += f.all();
        }
        found = f;
        found_b = b;
        found_step = (int)before;
    }
    __syncthreads();
    // The same in every lane, which the compiler has to be told for what
    // follows from them to stay in scalar registers.
    *at_b = uniform(found_b);
    *at_seq = uniform(found);
    *at_step = uniform(found_step);
    return (int)total;
}

// The sequence that row tile x of the tile kernel belongs to: sequence b's
// tiles are numbered from starts[b] / tile_tokens + b on, and of those in
// order whose numbers begin at or before x it is the last.  64 are looked at
// together, with all that is needed of them, so that it is known after one
// load's latency.  b is -1 where there is none.
struct TileSeq {
    int b;
    Seq s;
};

__device__ __forceinline__ TileSeq tile_seq(const AttendArgs& p, int x) {
    const int lane = threadIdx.x & 63;
    TileSeq t = {-1, {0, 0, 0}};
    for (int b0 = 0; b0 < p.g.batch; b0 += 64) {
        const int bb = b0 + lane < p.g.batch ? b0 + lane : p.g.batch - 1;
        const Seq s = read_seq(p.g, bb);
        const uint64_t m = __ballot(b0 + lane < p.g.batch && s.n > 0 && s.row0 / p.tile_tokens + bb <= x);
        if (m) {
            const int from = 63 - __builtin_clzll(m);
            t.b = b0 + from;
            t.s.row0 = __builtin_amdgcn_readlane(s.row0, from);
            t.s.n = __builtin_amdgcn_readlane(s.n, from);
            t.s.length = __builtin_amdgcn_readlane(s.length, from);
        }
    }
    return t;
}

// Part of a row tile that one workgroup of the split kernel leaves: rows of
// 16 * dc sums, then each row's reference and sum of weights.
TPL_HD constexpr int few_part_floats(int dc, int mr) { return mr * 16 * (16 * dc + 2); }

// The split kernel's workgroups that a CU holds at once: two of its waves a
// SIMD as far as 256 registers allow, else one.  The grid is that many for
// every CU, so that equal shares end together.  Three a CU measured 3 to 20 %
// slower (more parts to join), and holding the next step's loads in registers
// as well gained nothing: two waves a SIMD keep HBM busy.
TPL_HD constexpr int few_blocks(bool held8, int dc, int mr) {
    return 4 * dc * (held8 ? 1 : 2) + 6 * mr * dc <= 200 ? 2 : 1;
}

hipError_t launch_few(const AttendArgs& p, int dc, int mr, hipStream_t st);
hipError_t launch_tile(const AttendArgs& p, int dk, bool join, hipStream_t st);

TPL_HD int tile_part_floats(int dk, int rows) { return rows * (dk + 2); }

}  // namespace kv
}  // namespace tpl
