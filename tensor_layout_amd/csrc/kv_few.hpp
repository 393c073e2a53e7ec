// kv_few.hpp -- attention of a few rows a sequence (decoding, drafts) to a
// paged cache.
//
// out = sum_j w_j v_j / sum_j w_j, w_j = 2^(x_j - m), x = scale log2(e) q k,
// with one running reference m a row.
//
// Bound: HBM bytes of the cache, read once; for short caches the chain of
// dependent reads (lengths, table, keys, parts).  So the token axis is split:
// a head's work is counted in steps of 128 tokens of one (sequence, row
// tile), and every workgroup takes an equal share of consecutive steps of one
// head, whatever the sequences' lengths are.  Of a step each of 4 waves takes
// 32 tokens straight from HBM into registers: nothing is staged in LDS,
// because no other wave needs the same values.  Row tiles that end inside a
// share leave a part, and the last workgroup of a tile to do so joins its
// parts: no second launch.
//
// Where heads lie next to each other in a token's row (128 bytes each), HBM
// gives its rate only if a row's heads are read at about the same time from
// one die: workgroups of one share's heads are dealt to one die in a row (64
// windows of 1024 tokens 32 -> 23 us, drafts 65 -> 50 us), and where shares
// are so long that these drift apart, a workgroup takes two heads (64
// sequences of up to 8192 tokens 174 -> 155 us; with pages laid out by head
// it takes 140 us).
//
// Measured on an MI355X: that batch at 4.6 TB/s (154 us), in bf16 instead of
// e4m3 at 5.2 TB/s (275 us), in e4m3 with heads of 256 at 4.7 TB/s (301 us);
// two sequences of 131009 tokens, 64 heads on 8, pages by head, at 4.7 TB/s
// (115 us); a batch of 64 even ones by head at 5.5 TB/s (a large copy: 5.2).
//
// Layout.  S^T = K Q^T with 16 tokens as the rows of a 16x16x32 product:
// lane (r = lane % 16, g = lane / 16) holds channels of token r, and its part
// of the result is tokens 4 g .. 4 g + 3 of query row r.  Two such results
// are, as they lie, the second operand of O^T = V^T P^T (8 consecutive k
// slots a lane), if V's slots name the same tokens; so weights never leave
// their lane.  For V^T a lane reads DC consecutive channels of its 8 tokens
// and exchanges halves within the lane (v_perm); product t takes channel
// r * DC + t, which spreads the head's channels over products in an order
// that only the final store has to know.
//
// SHARED: sequences in groups whose first `cut` tokens lie in the pages of the
// group's first row of the table.  A softmax over two ranges of tokens is the
// join of each range's (m, sum w, sum w v), so one launch may take a group's
// rows over its shared tokens (p.prefix: the group is the sequence, and leaves
// these three) and the next each sequence's own tokens, starting from them in
// place of zeros.  Directly, one launch takes both ranges, a step in one only.
// 64 sequences behind 4096 shared tokens, up to 1024 of their own, 8 heads of 128
// in e4m3: 46 us, 20 of them for the shared (a copy of all bytes: 15); what bounds
// both is the chain of reads (lengths, groups, table, keys), of which a workgroup
// has few steps to hide.  Reading the first step's keys before the shared tokens'
// results, which takes 130 registers more, was slower (by 2 us).
#pragma once

#include "kv_attend.hpp"

namespace tpl {
namespace kv {

template <int BYTES>
struct Chunk {
    uint32_t w[BYTES / 4];
};

template <int BYTES>
__device__ __forceinline__ Chunk<BYTES> load_chunk(const uint8_t* p) {
    Chunk<BYTES> c;
    if constexpr (BYTES == 4) {
        c.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 12) {
        const u32x3 v = *reinterpret_cast<const u32x3*>(p);
        c.w[0] = v[0], c.w[1] = v[1], c.w[2] = v[2];
    } else if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(p + 16 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) c.w[4 * i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 8; ++i) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(p + 8 * i);
            c.w[2 * i] = v[0], c.w[2 * i + 1] = v[1];
        }
    }
    return c;
}

// 16 tokens of the cache, as a wave holds them.
template <bool HELD8, int DC>
struct Tile {
    static constexpr int KL = HELD8 ? DC / 4 : DC / 2;   // 16-byte loads of a key row
    u32x4 k[KL];
    Chunk<HELD8 ? DC : 2 * DC> v[4];
    float ks, vs;
    int base;     // first token, or a number beyond every position
    int lo, hi;   // SHARED: its tokens that count
};

// Where a group of 16 tokens lies: its page's table entry, its first token's
// place in the page, and that token (beyond every position past the span).
struct Place {
    int entry, slot, base, lo, hi;
};

// `first` names the pages of the span's first na groups, which end before token `cut`.
template <bool SHARED>
__device__ __forceinline__ Place place_of(const AttendArgs& p, const int32_t* pages, const int32_t* first, int cut, const Span& span, int t) {
    Place x;
    if constexpr (SHARED) {
        const bool own = (t < span.n ? t : span.n - 1) >= span.na;
        pages = own ? pages : first;
        x.lo = own ? cut : 0;
        x.hi = own ? kNowhere : cut - 1;
    }
    const int base = span.base(t < span.n ? t : span.n - 1);
    const int pg = (int)fdiv((uint32_t)base, p.div_page);
    x.entry = scalar(pages + pg);
    x.slot = base - pg * p.c.page;
    x.base = t < span.n ? base : kNowhere;
    return x;
}

// One head's keys, values and scales.
struct Head {
    const uint8_t *k, *v;
    const float *ks, *vs;
};

// Loads without a branch, so that they are in flight together: a group that
// is not there reads page 0 and stands beyond every position; lanes beyond
// the head's channels read its first ones.
template <bool HELD8, int DC, bool SHARED>
__device__ __forceinline__ void load_tile(const AttendArgs& p, const Head& h, Place at, Tile<HELD8, DC>& x) {
    constexpr int W = HELD8 ? 1 : 2;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const bool there = (uint32_t)at.entry < (uint32_t)p.c.pages;
    const uint32_t where = there ? at.entry : 0, slot = at.slot;
    x.base = there ? at.base : kNowhere;
    if constexpr (SHARED) x.lo = at.lo, x.hi = at.hi;
    const uint8_t* k = h.k + (uint64_t)where * (uint32_t)(p.c.k_page * W) + slot * (uint32_t)(p.c.k_token * W);
    const uint8_t* v = h.v + (uint64_t)where * (uint32_t)(p.c.v_page * W) + slot * (uint32_t)(p.c.v_token * W);
    x.ks = x.vs = 1.0f;
    if constexpr (HELD8) {
        const uint32_t blk = fdiv(slot, p.div_block);
        const float ks = scalar(h.ks + (uint64_t)where * (uint32_t)p.c.ks_page + blk * (uint32_t)p.c.ks_block);
        const float vs = scalar(h.vs + (uint64_t)where * (uint32_t)p.c.vs_page + blk * (uint32_t)p.c.vs_block);
        // Page 0 may hold nothing, and its scales anything: a product with
        // them would show in rows that do not see it.
        x.ks = there ? ks : 1.0f;
        x.vs = there ? vs : 1.0f;
    }
    const uint32_t kr = r * (uint32_t)(p.c.k_token * W);
#pragma unroll
    for (int i = 0; i < x.KL; ++i) {
        const uint32_t ch = HELD8 ? i * 64 + g * 16 : i * 32 + g * 8;
        x.k[i] = *reinterpret_cast<const u32x4*>(k + (uint32_t)(kr + (ch < (uint32_t)p.c.dim ? ch : 0) * W));
    }
    const uint32_t vc = (r * DC < p.c.dim ? r * DC : 0) * W;
#pragma unroll
    for (int e = 0; e < 4; ++e) x.v[e] = load_chunk<DC * W>(v + (uint32_t)(vc + (g * 4 + e) * (uint32_t)(p.c.v_token * W)));
}

// Channels t of 4 tokens as 2 words of two tokens each.
template <typename V, bool HELD8, int DC>
__device__ __forceinline__ u32x2 column(const Chunk<HELD8 ? DC : 2 * DC> (&v)[4], int t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (HELD8)
            w[e] = (t & 2) ? V::template from_e4m3<true>(v[e].w[t >> 2]) : V::template from_e4m3<false>(v[e].w[t >> 2]);
        else
            w[e] = v[e].w[t >> 1];
    }
    const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
    return u32x2{__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel)};
}

// Two numbers of a part, written through to where workgroups on other dies
// see them, and read from there.
__device__ __forceinline__ void leave2(float* p, float a, float b) {
    const uint64_t w = (uint64_t)__builtin_bit_cast(uint32_t, b) << 32 | __builtin_bit_cast(uint32_t, a);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 take2(const float* p) {
    const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, (uint32_t)w), __builtin_bit_cast(float, (uint32_t)(w >> 32)));
}

template <typename T, bool HELD8, int DC, int MR, bool SHARED>
__global__ void __launch_bounds__(256, few_blocks(HELD8, DC, MR)) k_few(AttendArgs p) {
    typedef typename T::one one;
    typedef typename T::x8 x8;
    // Weights and values are multiplied in the cache's type.  An e4m3 value's
    // scale is folded into its weight, which needs bf16's range.  A bf16 weight
    // goes in as the sum of two numbers, which keep 15 or 16 bits, so that its
    // rounding does not show beside the output's: HBM hides the second product
    // (64 sequences of up to 8192 tokens: 154 us with it and 153 to 154 without).
    // Where 64 rows make a step long (8 drafts of 8 heads: 115 against 107 us)
    // a bf16 output is left with weights of its own 8 bits, as an fp16 one of an
    // fp16 cache is with weights of its own 11.
    typedef typename std::conditional<HELD8, Bf16, T>::type V;
    constexpr bool kTwo = std::is_same<V, Bf16>::value && (MR <= 2 || std::is_same<T, Fp16>::value);
    typedef typename std::conditional<HELD8, E4m3, T>::type H;   // what the cache holds
    constexpr int KS = DC / 2;           // key products of a row
    constexpr int ROWS = MR * 16;
    constexpr int HALVES = DC > 8 ? 2 : 1, DCH = DC / HALVES, PITCH = 16 * DCH + 4;
    __shared__ float obuf[4][16][PITCH];
    __shared__ float mbuf[4][ROWS], lbuf[4][ROWS];
    __shared__ int arrived;

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b;
    int seq_step, chunk, even;
    // Its heads, this wave's among them and its place among their waves.
    const int hw = 1 << p.heads_log, sets = p.c.kv_heads >> p.heads_log;
    // Workgroups are dealt to the 8 dies in turn: the same share of all heads
    // goes to one die, one after the other.
    const int by8 = blockIdx.x >> 3, share = by8 / sets * 8 + (blockIdx.x & 7), h0 = by8 % sets << p.heads_log;
    const int id = share * sets + (h0 >> p.heads_log);
    if (share >= p.shares) return;
    const int wd = wave & (hw - 1), wt = wave >> p.heads_log, h = h0 + wd;
    FewSeq f;
    const int total = locate<ROWS, SHARED>(p, share, &b, &f, &seq_step, &chunk, &even);
    const int win = p.a.window ? p.a.window : 0x7fffffff;
    // Whether a row at `at` sees token j of a group, both ends of rows given;
    // whether all rows see its 16 tokens.
    auto sees = [&](const auto& x, int j, int at, int last) {
        if constexpr (SHARED)
            return (j <= at) & (j >= x.lo) & (j <= x.hi);
        else
            return (j <= at) & ((last - j < win) | (j < p.a.sinks));
    };
    auto all_see = [&](const auto& x, int first_at, int last_at) {
        if constexpr (SHARED)
            return (x.base <= first_at - 15) & (x.base >= x.lo) & (x.base <= x.hi - 15);
        else
            return (x.base <= first_at - 15) & ((last_at - x.base < win) | (x.base + 15 < p.a.sinks));
    };
    const bool flat = SHARED && p.prefix;   // all rows see as far as the last shared token
    if (b < 0) return;
    int c = share * chunk;
    const int cend = chunk < total - c ? c + chunk : total;
    if (c >= cend) return;

    while (c < cend) {
        const int off = c - seq_step, all = (int)f.all();
        if (off >= all) {
            seq_step += all;
            if (++b >= few_items<SHARED>(p)) return;
            f = uniform<SHARED>(few_seq<ROWS, SHARED>(p, b));
            if (SHARED && even) f.steps = even;
            continue;
        }
        const int rt = uniform((int)((uint32_t)off / (uint32_t)f.steps));
        const int s0 = uniform(off - rt * f.steps), tile_at = seq_step + rt * f.steps;
        const int s1 = uniform(f.steps - s0 < cend - c ? f.steps : s0 + (cend - c));
        const int rows = f.s.n * p.group - rt * ROWS;   // of this tile, may exceed ROWS
        const int first = flat ? f.s.length - 1 : f.s.length - f.s.n;
        const int32_t* pages = p.g.table + b * p.g.table_row;
        const int32_t* first_pages = SHARED ? p.g.table + f.row * p.g.table_row : pages;
        const int pmin = flat ? first : uniform(first + (int)fdiv((uint32_t)(rt * ROWS), p.div_group));
        const int lastrow = rt * ROWS + (rows < ROWS ? rows : ROWS) - 1;
        const int pmax = flat ? first : uniform(first + (int)fdiv((uint32_t)lastrow, p.div_group));

        x8 q[MR][KS];
        int pos[MR];
        f32x4 o[MR][DC];
        float m[MR], l[MR];
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
            const int row = mr * 16 + r;
            const bool there = row < rows;
            const int i = (int)fdiv((uint32_t)(rt * ROWS + row), p.div_group);
            const int head = h * p.group + rt * ROWS + row - i * p.group;
            pos[mr] = there ? flat ? first : first + i : -1;
            const one* src = (const one*)p.a.q + (there ? (f.s.row0 + i) * p.a.q_token + head * p.a.q_head : 0);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int ch = HELD8 ? (k >> 1) * 64 + g * 16 + (k & 1) * 8 : k * 32 + g * 8;
                u32x4 w = {0, 0, 0, 0};
                if (there && ch < p.c.dim) w = *reinterpret_cast<const u32x4*>(src + ch);
                q[mr][k] = __builtin_bit_cast(x8, w);
            }
            m[mr] = neg_inf();
            l[mr] = 0.0f;
#pragma unroll
            for (int t = 0; t < DC; ++t) o[mr][t] = f32x4{0, 0, 0, 0};
        }

        // What the rows found among the shared tokens, as if they had been the
        // first ones here: the tile's first share takes it, each wave some of
        // the parts, two at a time.
        if constexpr (SHARED) {
            if (f.cut > 0 && s0 == 0 && !p.direct && !flat) {
                constexpr int AT_ONCE = MR * DC <= 8 ? 2 : 1;
                const int step = 4 >> p.heads_log;
#pragma unroll
                for (int mr = 0; mr < MR; ++mr) {
                    const int row = mr * 16 + r;
                    if (row >= rows) continue;
                    const int i = (int)fdiv((uint32_t)(rt * ROWS + row), p.div_group);
                    const int head = h * p.group + rt * ROWS + row - i * p.group;
                    const int64_t part = (int64_t)p.g.tokens * p.a.heads, at = (int64_t)(f.s.row0 + i) * p.a.heads + head;
#pragma unroll 1
                    for (int k = wt; k < p.before_splits; k += AT_ONCE * step) {
                        float2 ml[AT_ONCE];
                        f32x4 v[AT_ONCE][DC];
#pragma unroll
                        for (int d = 0; d < AT_ONCE; ++d) {
                            const int kk = k + d * step < p.before_splits ? k + d * step : k;
                            ml[d] = p.before_ml[kk * part + at];
                            if (d && k + d * step >= p.before_splits) ml[d].x = neg_inf();
                            const float* y = p.before + (kk * part + at) * p.c.dim;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int t = 0; t < DC / 4; ++t) {
                                    const int ch = (g * 4 + e) * DC + t * 4;
                                    v[d][e * (DC / 4) + t] = *reinterpret_cast<const f32x4*>(y + (ch < p.c.dim ? ch : 0));
                                }
                        }
#pragma unroll
                        for (int d = 0; d < AT_ONCE; ++d) {
                            if (ml[d].x == neg_inf()) continue;
                            const float top = fmaxf(m[mr], ml[d].x);
                            const float c0 = m[mr] == neg_inf() ? 0.0f : exp2_(m[mr] - top), c1 = exp2_(ml[d].x - top);
                            l[mr] *= c0;
                            if (g == 0) l[mr] += ml[d].y * c1;   // a lane's sum is of its own tokens
                            m[mr] = top;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int t = 0; t < DC; ++t) o[mr][t][e] = o[mr][t][e] * c0 + v[d][e * (DC / 4) + (t >> 2)][t & 3] * c1;
                        }
                    }
                }
            }
        }

        constexpr int W = HELD8 ? 1 : 2;
        const Head hd = {(const uint8_t*)p.c.k + h * p.c.k_head * W, (const uint8_t*)p.c.v + h * p.c.v_head * W,
                         p.c.k_scale + h * p.c.ks_head, p.c.v_scale + h * p.c.vs_head};
        auto places = [&](Place (&at)[2], int s) {
            const int t = s * (kStepGroups >> p.heads_log) + wt * 2;
            at[0] = place_of<SHARED>(p, pages, first_pages, f.cut, f.span, t);
            at[1] = place_of<SHARED>(p, pages, first_pages, f.cut, f.span, t + 1);
        };
        bool left_out = false;
        auto step = [&](Tile<HELD8, DC> (&x)[2]) {
            if (p.c.dim < 16 * DC) {   // what lanes read beyond the head's channels meets the queries' zeros
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < x[u].KL; ++i)
                        if ((HELD8 ? i * 64 + g * 16 : i * 32 + g * 8) >= p.c.dim) x[u].k[i] = u32x4{0, 0, 0, 0};
            }
            f32x4 sc[MR][2];
            float f2[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int mr = 0; mr < MR; ++mr) sc[mr][u] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    u32x4 w;
                    if constexpr (HELD8) {
                        const uint32_t a = x[u].k[k >> 1][(k & 1) * 2], d = x[u].k[k >> 1][(k & 1) * 2 + 1];
                        w = u32x4{T::template from_e4m3<false>(a), T::template from_e4m3<true>(a),
                                  T::template from_e4m3<false>(d), T::template from_e4m3<true>(d)};
                    } else {
                        w = x[u].k[k];
                    }
                    const x8 kk = __builtin_bit_cast(x8, w);
#pragma unroll
                    for (int mr = 0; mr < MR; ++mr) sc[mr][u] = T::mfma16(kk, q[mr][k], sc[mr][u]);
                }
                const int base = x[u].base;
                // A masked score is minus infinity times this: it must not be zero.
                f2[u] = HELD8 ? fmaxf(p.factor * x[u].ks, 1.17549435e-38f) : p.factor;
                const bool full = all_see(x[u], pmin, pmax);
                if (!full) {
                    // Rows that do not see a token multiply its values with
                    // zeros, which an infinity or NaN among them would show:
                    // such values are left out here, and added at the end to
                    // the rows that do see them.
                    if (pmin != pmax) {
                        bool some = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < (int)(sizeof(x[u].v[i]) / 4); ++k) some |= clear_bad<H>(x[u].v[i].w[k]);
                        if (some) left_out = true;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = base + g * 4 + i;
#pragma unroll
                        for (int mr = 0; mr < MR; ++mr)
                            sc[mr][u][i] = sees(x[u], j, pos[mr], pos[mr]) ? sc[mr][u][i] : neg_inf();
                        // A token that no row sees weighs nothing, whatever its place holds.
                        if (!sees(x[u], j, pmax, pmin))
#pragma unroll
                            for (int k = 0; k < (int)(sizeof(x[u].v[i]) / 4); ++k) x[u].v[i].w[k] = 0;
                    }
                }
            }

            u32x4 w[MR], w2[MR];
#pragma unroll
            for (int mr = 0; mr < MR; ++mr) {
                float top = neg_inf();
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    top = fmaxf(top, f2[u] * fmaxf(fmaxf(sc[mr][u][0], sc[mr][u][1]), fmaxf(sc[mr][u][2], sc[mr][u][3])));
                top -= lift<V>();
                if (__any(top > m[mr] + kSlack)) {
                    top = max16(max32(fmaxf(top, m[mr])));
                    const float a = top == neg_inf() ? 1.0f : exp2_(m[mr] - top);
                    m[mr] = top;
                    l[mr] *= a;
#pragma unroll
                    for (int t = 0; t < DC; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mr][t][i] *= a;
                }
                const float ref = m[mr] == neg_inf() ? 0.0f : m[mr];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[i] = exp2_(__builtin_fmaf(sc[mr][u][i], f2[u], -ref));
                        l[mr] += e[i];
                        if constexpr (HELD8) e[i] *= x[u].vs;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = e[2 * i], b = e[2 * i + 1];
                        uint32_t x = pack2<V>(a, b);
                        if constexpr (kTwo && !HELD8) {
                            // A bf16 value may be infinite: what is left of a
                            // weight over zero has to be over zero too, so the
                            // first number is cut off instead of rounded and
                            // the second made larger by 2^-20 of the weight.
                            x = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
                            w2[mr][u * 2 + i] = pack2<V>(__builtin_fmaf(a, 1.0f + 0x1p-20f, -lo16<V>(x)),
                                                         __builtin_fmaf(b, 1.0f + 0x1p-20f, -hi16<V>(x)));
                        } else if constexpr (kTwo) {
                            w2[mr][u * 2 + i] = pack2<V>(a - lo16<V>(x), b - hi16<V>(x));
                        }
                        w[mr][u * 2 + i] = x;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < DC; ++t) {
                const u32x2 a0 = column<V, HELD8, DC>(x[0].v, t), a1 = column<V, HELD8, DC>(x[1].v, t);
                const auto vv = __builtin_bit_cast(typename V::x8, (u32x4{a0[0], a0[1], a1[0], a1[1]}));
#pragma unroll
                for (int mr = 0; mr < MR; ++mr) {
                    o[mr][t] = V::mfma16(vv, __builtin_bit_cast(typename V::x8, w[mr]), o[mr][t]);
                    if constexpr (kTwo) o[mr][t] = V::mfma16(vv, __builtin_bit_cast(typename V::x8, w2[mr]), o[mr][t]);
                }
            }
        };

        if (s0 * (kStepGroups >> p.heads_log) + wt * 2 < f.span.n) {
            Place at[2];
            places(at, s0);
            for (int s = s0; s < s1; ++s) {
                Tile<HELD8, DC> x[2];
                load_tile<HELD8, DC, SHARED>(p, hd, at[0], x[0]);
                load_tile<HELD8, DC, SHARED>(p, hd, at[1], x[1]);
                places(at, s + 1);   // the table's entries for the next step
                step(x);
                if (SHARED && (s + 1) * (kStepGroups >> p.heads_log) >= f.span.n) break;   // a tile's share may be longer
            }
        }

        if (__any(left_out)) {
#pragma unroll 1
            for (int s = s0; s < s1; ++s)
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int t = s * (kStepGroups >> p.heads_log) + wt * 2 + u;
                    if (t >= f.span.n) break;
                    const Place x = place_of<SHARED>(p, pages, first_pages, f.cut, f.span, t);
                    if ((uint32_t)x.entry >= (uint32_t)p.c.pages) continue;
                    if (all_see(x, pmin, pmax)) continue;
#pragma unroll 1
                    for (int j = 0; j < 16; ++j) {
                        const uint8_t* from = hd.v + (uint64_t)(uint32_t)x.entry * (uint32_t)(p.c.v_page * W) +
                                              (uint32_t)(x.slot + j) * (uint32_t)(p.c.v_token * W);
                        const int tok = x.base + j;
                        int g4 = g * 4, dim = p.c.dim;
                        asm volatile("" : "+v"(g4), "+s"(dim));   // no comparison is to be held in registers throughout
#pragma unroll
                        for (int t2 = 0; t2 < DC; ++t2)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int ch = (g4 + i) * DC + t2;
                                const float v = ch < dim ? value_at<H>(from + ch * W) : 0.0f;
                                if (!(__builtin_fabsf(v) < __builtin_inff()))
#pragma unroll
                                    for (int mr = 0; mr < MR; ++mr)
                                        if (sees(x, tok, pos[mr], pos[mr])) o[mr][t2][i] += v;
                            }
                    }
                }
        }

        // The sums of a head's waves join under their largest reference.
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
            l[mr] = sum16(sum32(l[mr]));
            // Scores that are no numbers pass a maximum by.  Where there were
            // no others the sum tells them from a row that saw nothing: any
            // reference then keeps them for the output.
            if (m[mr] == neg_inf() && l[mr] != l[mr]) m[mr] = 0.0f;
            if (g == 0) {
                mbuf[wave][mr * 16 + r] = m[mr];
                lbuf[wave][mr * 16 + r] = l[mr];
            }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == f.steps;
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
            float top = neg_inf();
            for (int i = wd; i < 4; i += hw) top = fmaxf(top, mbuf[i][mr * 16 + r]);
            const float a = m[mr] == neg_inf() ? 0.0f : exp2_(m[mr] - top);
            const int orow = mr * 16 + (tid >> 4), oc = tid & 15;
            const bool there = orow < rows;
            const int oi = (int)fdiv((uint32_t)(rt * ROWS + orow), p.div_group);
#pragma unroll
            for (int half = 0; half < HALVES; ++half) {
                if (mr + half) __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < DCH; ++t) obuf[wave][r][(g * 4 + i) * DCH + t] = m[mr] == neg_inf() ? 0.0f : o[mr][half * DCH + t][i] * a;
                __syncthreads();
                if (!there) continue;
                for (int d = 0; d < hw; ++d) {
                    float otop = neg_inf(), osum = 0.0f, y[DCH];
                    for (int i = d; i < 4; i += hw) otop = fmaxf(otop, mbuf[i][orow]);
#pragma unroll
                    for (int t = 0; t < DCH; ++t) y[t] = 0.0f;
                    for (int i = d; i < 4; i += hw) {
                        osum += mbuf[i][orow] == neg_inf() ? 0.0f : lbuf[i][orow] * exp2_(mbuf[i][orow] - otop);
#pragma unroll
                        for (int t = 0; t < DCH; ++t) y[t] += obuf[i][tid >> 4][oc * DCH + t];
                    }
                    if (flat && whole) {
                        const int head = (h0 + d) * p.group + rt * ROWS + orow - oi * p.group;
                        const int64_t at = (int64_t)(f.s.row0 + oi) * p.a.heads + head;
                        if (oc * DC < p.c.dim)
#pragma unroll
                            for (int t = 0; t < DCH; t += 2)
                                *reinterpret_cast<float2*>(p.before + at * p.c.dim + oc * DC + half * DCH + t) = make_float2(y[t], y[t + 1]);
                        if (oc == 0 && half == 0) p.before_ml[at] = make_float2(otop, osum);
                    } else if (whole) {
                        const int head = (h0 + d) * p.group + rt * ROWS + orow - oi * p.group;
                        const float inv = osum == 0.0f ? 0.0f : 1.0f / osum;
                        one* out = (one*)p.a.out + (f.s.row0 + oi) * p.a.o_token + head * p.a.o_head + oc * DC + half * DCH;
                        if (oc * DC < p.c.dim)
#pragma unroll
                            for (int t = 0; t < DCH; t += 2)
                                *reinterpret_cast<uint32_t*>(out + t) = pack2<T>(osum == 0.0f ? 0.0f : y[t] * inv, osum == 0.0f ? 0.0f : y[t + 1] * inv);
                        if (p.a.lse && oc == 0 && half == 0)
                            p.a.lse[(f.s.row0 + oi) * p.a.l_token + head * p.a.l_head] =
                                osum == 0.0f ? neg_inf() : (otop + __builtin_log2f(osum)) * kLn2;
                    } else {
                        float* part = p.parts + (((uint64_t)(uint32_t)id * 2 + (s0 ? 0 : 1)) * hw + d) * few_part_floats(DC, MR);
#pragma unroll
                        for (int t = 0; t < DCH; t += 2) leave2(part + orow * (16 * DC) + oc * DC + half * DCH + t, y[t], y[t + 1]);
                        if (oc == 0 && half == 0) leave2(part + ROWS * 16 * DC + orow * 2, otop, osum);
                    }
                }
            }
        }
        c += s1 - s0;
        if (whole) {
            __syncthreads();
            continue;
        }

        // A part is left.  The workgroup that leaves the last one of its row
        // tile joins them, in their order: whichever it is, the sum is the
        // same.  Parts are counted at the tile's first workgroup, in a number
        // that is zero again afterwards.
        const int w0 = uniform((int)((uint32_t)tile_at / (uint32_t)chunk));
        const int np = uniform((int)((uint32_t)(tile_at + f.steps - 1) / (uint32_t)chunk)) - w0 + 1;
        int* counter = p.counters + w0 * sets + (h0 >> p.heads_log);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's part is out
        __syncthreads();
        if (tid == 0) arrived = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (uniform(arrived) != np - 1) continue;
        if (tid == 0) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // 16 threads a row and head; the parts some at a time, so that their
        // reads, which go past this die's L2, wait for one another once.
        constexpr int AT_ONCE = DC <= 8 ? 8 : 4;
        const int nrow = rows < ROWS ? rows : ROWS, oc = tid & 15;
#pragma unroll 1
        for (int z = tid >> 4; z < nrow * hw; z += 16) {
            const int d = z / nrow, row = z - d * nrow;
            float top = neg_inf(), sum = 0.0f, y[DC];
#pragma unroll
            for (int t = 0; t < DC; ++t) y[t] = 0.0f;
#pragma unroll 1
            for (int i0 = 0; i0 < np; i0 += AT_ONCE) {
                float2 ml[AT_ONCE], v[AT_ONCE][DC / 2];
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    const int i = i0 + k < np ? i0 + k : np - 1;
                    const uint64_t w = (uint32_t)((w0 + i) * sets + (h0 >> p.heads_log));
                    const float* part = p.parts + ((w * 2 + (i ? 0 : 1)) * hw + d) * few_part_floats(DC, MR);
                    ml[k] = take2(part + ROWS * 16 * DC + row * 2);
#pragma unroll
                    for (int t = 0; t < DC / 2; ++t) v[k][t] = take2(part + row * 16 * DC + oc * DC + t * 2);
                    if (i0 + k >= np) ml[k].x = neg_inf();
                }
                float next = top;
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) next = fmaxf(next, ml[k].x);
                const float c0 = top == neg_inf() ? 0.0f : exp2_(top - next);
                sum *= c0;
#pragma unroll
                for (int t = 0; t < DC; ++t) y[t] *= c0;
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k) {
                    if (ml[k].x == neg_inf()) continue;   // nothing in it: no product, which an infinity would show
                    const float a = exp2_(ml[k].x - next);
                    sum += ml[k].y * a;
#pragma unroll
                    for (int t = 0; t < DC / 2; ++t) {
                        y[2 * t] += v[k][t].x * a;
                        y[2 * t + 1] += v[k][t].y * a;
                    }
                }
                top = next;
            }
            const int i = (int)fdiv((uint32_t)(rt * ROWS + row), p.div_group);
            const int head = (h0 + d) * p.group + rt * ROWS + row - i * p.group;
            if (flat) {
                const int64_t at = (int64_t)(f.s.row0 + i) * p.a.heads + head;
                if (oc * DC < p.c.dim)
#pragma unroll
                    for (int t = 0; t < DC; t += 4)
                        *reinterpret_cast<f32x4*>(p.before + at * p.c.dim + oc * DC + t) = f32x4{y[t], y[t + 1], y[t + 2], y[t + 3]};
                if (oc == 0) p.before_ml[at] = make_float2(top, sum);
                continue;
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            one* out = (one*)p.a.out + (f.s.row0 + i) * p.a.o_token + head * p.a.o_head + oc * DC;
            if (oc * DC < p.c.dim)
#pragma unroll
                for (int t = 0; t < DC; t += 2)
                    *reinterpret_cast<uint32_t*>(out + t) = pack2<T>(sum == 0.0f ? 0.0f : y[t] * inv, sum == 0.0f ? 0.0f : y[t + 1] * inv);
            if (p.a.lse && oc == 0)
                p.a.lse[(f.s.row0 + i) * p.a.l_token + head * p.a.l_head] =
                    sum == 0.0f ? neg_inf() : (top + __builtin_log2f(sum)) * kLn2;
        }
    }
}

template <typename T, bool HELD8, int DC, int MR, bool SHARED>
static hipError_t go(const AttendArgs& p, hipStream_t st) {
    k_few<T, HELD8, DC, MR, SHARED><<<(unsigned)((p.shares + 7) / 8 * 8 * (p.c.kv_heads >> p.heads_log)), 256, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, bool HELD8, int DC, bool SHARED>
static hipError_t go_mr(const AttendArgs& p, int mr, hipStream_t st) {
    if (mr == 1) return go<T, HELD8, DC, 1, SHARED>(p, st);
    if constexpr (DC <= 8) {   // 64 rows of longer heads would not fit a lane's registers
        if (mr == 4) return go<T, HELD8, DC, 4, SHARED>(p, st);
    }
    return go<T, HELD8, DC, 2, SHARED>(p, st);
}

template <typename T, bool HELD8, bool SHARED>
static hipError_t go_dc(const AttendArgs& p, int dc, int mr, hipStream_t st) {
    switch (dc) {
    case 4: return go_mr<T, HELD8, 4, SHARED>(p, mr, st);
    case 8: return go_mr<T, HELD8, 8, SHARED>(p, mr, st);
    case 12: return go_mr<T, HELD8, 12, SHARED>(p, mr, st);
    default: return go_mr<T, HELD8, 16, SHARED>(p, mr, st);
    }
}

template <bool SHARED>
static hipError_t go_few(const AttendArgs& p, int dc, int mr, hipStream_t st) {
    const bool held8 = p.c.type == TPL_KV_E4M3;
    if (p.a.type == TPL_KV_BF16)
        return held8 ? go_dc<Bf16, true, SHARED>(p, dc, mr, st) : go_dc<Bf16, false, SHARED>(p, dc, mr, st);
    return held8 ? go_dc<Fp16, true, SHARED>(p, dc, mr, st) : go_dc<Fp16, false, SHARED>(p, dc, mr, st);
}

}  // namespace kv
}  // namespace tpl
