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
    // Sequences that share their first tokens (the kernels' SHARED forms).
    tpl_kv_groups s;
    int32_t prefix;        // groups' rows and the tokens they share, not sequences
    int32_t direct;        // sequences' rows and all their tokens, the shared ones too; otherwise those have been taken before:
    int32_t before_splits; // in this many parts of each row
    float* before;         // [before_splits][tokens][heads][dim], weights' sums not yet divided by
    float2* before_ml;     // [before_splits][tokens][heads]: a row's reference and sum of weights
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

// A sequence's groups of 16 tokens where its first `cut` tokens are another's:
// those that hold them, in that one's pages, and those that hold tokens
// cut .. end - 1, in its own.  Where the cut lies inside 16 tokens both have a
// group there.
__device__ __forceinline__ Span span_cut(int cut, int end, bool first, bool own) {
    Span s;
    s.na = first ? (cut + 15) >> 4 : 0;
    s.lo = cut & ~15;
    s.n = s.na + (own && end > s.lo ? ((end + 15) >> 4) - (cut >> 4) : 0);
    return s;
}

// Group g of the sequences that share their first tokens, and their number:
// its rows, which are those of its sequences, and as its length the tokens
// that they share.  One that is not in order has no rows.
struct Group {
    int first, end;   // sequences
    Seq s;
};

__device__ __forceinline__ Group read_group(const AttendArgs& p, int g) {
    Group x;
    x.first = p.s.groups[g];
    x.end = p.s.groups[g + 1];
    const int shared = p.s.shared[g];
    x.s = Seq{0, 0, 0};
    if (x.first < 0 || x.end <= x.first || x.end > p.g.batch || shared < 1 || shared > p.cap) return x;
    const int row0 = p.g.starts[x.first], end = p.g.starts[x.end];
    if (row0 >= 0 && end > row0 && end <= p.g.tokens) x.s = Seq{row0, end - row0, shared};
    return x;
}

// How many of sequence b's first tokens are its group's, and the sequence that
// has them: none and itself where b has to look for itself.  Its group is the
// last of those in order that begin at or before it.
struct Common {
    int row, cut;
};

__device__ __forceinline__ Common common_of(const AttendArgs& p, int b, const Seq& s) {
    int lo = 0, hi = p.s.count;   // groups[lo] <= b, as far as they are in order
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.s.groups[mid] <= b)
            lo = mid;
        else
            hi = mid;
    }
    const Group g = read_group(p, lo);
    const bool ok = g.s.n > 0 && g.first <= b && b < g.end && s.n > 0 && g.s.row0 <= s.row0 && s.row0 + s.n <= g.s.row0 + g.s.n &&
                    g.s.length <= s.length - s.n;
    return ok ? Common{g.first, g.s.length} : Common{b, 0};
}

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
    int row;        // SHARED: the row of the table that names its first tokens,
    int cut;        // SHARED: how many those are
    __device__ __forceinline__ uint64_t all() const { return (uint64_t)tiles * (uint32_t)steps; }
};

// What the split kernel takes in turn: sequences, or groups of them.
template <bool SHARED>
__device__ __forceinline__ int few_items(const AttendArgs& p) { return SHARED && p.prefix ? p.s.count : p.g.batch; }

template <int ROWS, bool SHARED>
__device__ __forceinline__ FewSeq few_seq(const AttendArgs& p, int b) {
    FewSeq f;
    f.row = b;
    f.cut = 0;
    if (SHARED && p.prefix) {
        const Group g = read_group(p, b);
        f.s = g.s;
        f.row = g.first;
        f.cut = g.s.length;
    } else {
        f.s = read_seq(p.g, b);
    }
    const int64_t rows = (int64_t)f.s.n * p.group;
    if (rows > p.few) f.s.n = 0;
    f.tiles = f.s.n ? (int)((rows + ROWS - 1) / ROWS) : 0;
    if constexpr (SHARED) {
        if (!p.prefix) {
            const Common c = common_of(p, b, f.s);
            f.row = c.row;
            f.cut = c.cut;
        }
        f.span = span_cut(f.cut, f.s.length < p.cap ? f.s.length : p.cap, p.prefix || p.direct, !p.prefix);
    } else {
        f.span = span_of(p, f.s.length - f.s.n, f.s.length - 1);
    }
    const int log = 3 - p.heads_log;   // kStepGroups a wave's share of them
    f.steps = (f.span.n + (1 << log) - 1) >> log;
    if (f.steps < 1) f.steps = 1;
    return f;
}

template <bool SHARED>
__device__ __forceinline__ FewSeq uniform(FewSeq f) {
    f.s.row0 = uniform(f.s.row0);
    f.s.n = uniform(f.s.n);
    f.s.length = uniform(f.s.length);
    f.span.na = uniform(f.span.na);
    f.span.lo = uniform(f.span.lo);
    f.span.n = uniform(f.span.n);
    f.tiles = uniform(f.tiles);
    f.steps = uniform(f.steps);
    if constexpr (SHARED) {
        f.row = uniform(f.row);
        f.cut = uniform(f.cut);
    }
    return f;
}

template <bool SHARED>
__device__ __forceinline__ FewSeq from_lane(FewSeq f, int lane) {
    f.s.row0 = __builtin_amdgcn_readlane(f.s.row0, lane);
    f.s.n = __builtin_amdgcn_readlane(f.s.n, lane);
    f.s.length = __builtin_amdgcn_readlane(f.s.length, lane);
    f.span.na = __builtin_amdgcn_readlane(f.span.na, lane);
    f.span.lo = __builtin_amdgcn_readlane(f.span.lo, lane);
    f.span.n = __builtin_amdgcn_readlane(f.span.n, lane);
    f.tiles = __builtin_amdgcn_readlane(f.tiles, lane);
    f.steps = __builtin_amdgcn_readlane(f.steps, lane);
    if constexpr (SHARED) {
        f.row = __builtin_amdgcn_readlane(f.row, lane);
        f.cut = __builtin_amdgcn_readlane(f.cut, lane);
    }
    return f;
}

// Steps of a share: an equal part of them all, but no less than keeps the
// joining of a tile's parts (8 at a time) short beside its steps.  An average
// sequence of n steps takes about c + n / (8 c) of a step's time with c a
// share, least at c = sqrt(n / 8).
__device__ __forceinline__ int share_of(const AttendArgs& p, int items, int total) {
    const int equal = (int)(((uint32_t)total + (uint32_t)p.shares - 1) / (uint32_t)p.shares);
    const int short_ = (int)__builtin_sqrtf((float)total / (float)(items * 8)) + 1;
    return equal > short_ ? equal : short_;
}

// Measured (8 heads of 128 in e4m3, shared tokens and own ones together): 64
// sequences of up to 1024 of their own, 8 steps for 5, 58 -> 49 us; 128 of up to
// 800 86 -> 77; 256 of up to 200 87 -> 75; 64 of up to 4000, 32 steps for 18, 106
// -> 108.  Directly, 4 sequences of 530: 12.3 -> 13.1.
constexpr int kEven = 8;

// The batch's steps in order: every workgroup sums them for itself (one
// load's latency for up to 256 sequences, and no barrier for up to 64).
// Gives the total, the size of a share, and the sequence that this share
// begins in (-1: none) with that sequence's own first step.  More steps than
// 31 bits hold can only be counted for sequences that claim one another's
// rows (the host refuses sizes that allow them otherwise): nothing is done.
// `even`: steps that each row tile is counted with, 0: its own.
template <int ROWS, bool SHARED>
__device__ __forceinline__ int locate(const AttendArgs& p, int share, int* at_b, FewSeq* at_seq, int* at_step, int* chunk, int* even) {
    __shared__ uint64_t sums[4];
    __shared__ int tile_sums[4], longest[4];
    __shared__ int found_step, found_b;
    __shared__ FewSeq found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int items = few_items<SHARED>(p);
    const bool alone = items <= 64;   // every wave counts them all
    const int per = alone ? 1 : (items + 255) / 256, me = alone ? lane : tid;
    uint64_t mine = 0;
    int tiles = 0, steps = 0;   // SHARED: row tiles, and the most steps of one
    FewSeq f = {};
    for (int i = 0; i < per; ++i) {
        const int b = me * per + i;
        if (b < items) {
            f = few_seq<ROWS, SHARED>(p, b);
            mine += f.all();
            if constexpr (SHARED) {
                tiles += f.tiles;
                if (f.tiles && f.steps > steps) steps = f.steps;
            }
        }
    }
    uint64_t run = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    int run_tiles = tiles, all_tiles = 0, tiles_before = 0;
    if constexpr (SHARED) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(run_tiles, d), x = __shfl_xor(steps, d);
            if (lane >= d) run_tiles += o;
            if (x > steps) steps = x;
        }
        tiles_before = run_tiles - tiles;
        all_tiles = __shfl(run_tiles, 63);
    }
    uint64_t total, before = run - mine;
    if (alone) {
        total = __shfl(run, 63);
    } else {
        if (lane == 63) sums[wave] = run;
        if (SHARED && lane == 63) tile_sums[wave] = run_tiles, longest[wave] = steps;
        if (tid == 0) found_b = -1;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += sums[w];
            total += sums[w];
        }
        if constexpr (SHARED) {
            all_tiles = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < wave) tiles_before += tile_sums[w];
                all_tiles += tile_sums[w];
                if (longest[w] > steps) steps = longest[w];
            }
        }
    }
    total = uniform(total);
    *at_b = -1;
    *at_step = *chunk = *even = 0;
    if (total == 0 || total > 0x7fffffffu) return 0;
    *chunk = uniform(share_of(p, items, (int)total));
    if (SHARED && !p.prefix && !p.direct) {
        // Sequences' own tokens, taken to be few: whole row tiles a share, each
        // counted with the most steps that one has, where no share becomes kEven
        // steps longer.  No tile is then in parts that wait for one another, and
        // none begins twice.
        const int n = uniform(all_tiles), most = uniform(steps), each = uniform((int)((uint32_t)(n + p.shares - 1) / (uint32_t)p.shares));
        if ((int64_t)each * most <= *chunk + kEven && (int64_t)n * most <= 0x7fffffff) {
            *even = most;
            *chunk = each * most;
            total = (uint64_t)(n * most);
            mine = (uint64_t)(tiles * most);
            before = (uint64_t)(tiles_before * most);
            f.steps = most;
        }
    }
    const uint64_t c = (uint64_t)share * (uint32_t)*chunk;
    const bool here = mine && before <= c && c < before + mine;
    if (alone) {
        const uint64_t m = __ballot(here);
        if (m) {
            const int from = __builtin_ctzll(m);
            *at_b = from;
            *at_seq = from_lane<SHARED>(f, from);
            *at_step = __builtin_amdgcn_readlane((int)before, from);
        }
        return (int)total;
    }
    if (here) {
        int b = tid;
        for (int i = 0; per > 1 && i < per; ++i) {
            b = tid * per + i;
            if (b >= items) break;
            f = few_seq<ROWS, SHARED>(p, b);
            if (SHARED && *even) f.steps = *even;
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
    *at_seq = uniform<SHARED>(found);
    *at_step = uniform(found_step);
    return (int)total;
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
hipError_t launch_few_shared(const AttendArgs& p, int dc, int mr, hipStream_t st);
hipError_t launch_tile_shared(const AttendArgs& p, int dk, bool join, hipStream_t st);

TPL_HD int tile_part_floats(int dk, int rows) { return rows * (dk + 2); }

}  // namespace kv
}  // namespace tpl
