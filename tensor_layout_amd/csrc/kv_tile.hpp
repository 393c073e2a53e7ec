// kv_tile.hpp -- attention of many rows a sequence (prompts and their chunks)
// to a paged cache.
//
// The formulas are those of kv_few.hpp.  Bound: the matrix units and the
// exponentials.  A workgroup of 4 waves takes 128 query rows, one of 8 takes
// 256 (the query heads of one cache head, token by token: they share keys and
// values, and a row tile ends at one diagonal), 32 rows a wave, and walks
// over the cache 64 tokens at a time.  Keys and values are brought into LDS
// as 16-bit numbers (an e4m3 value is converted once for all rows), the
// values transposed on the way, so that both products read whole 16-byte
// operands:
//
//   S^T = K Q^T    32x32x16: lane (row r = lane % 32, half h = lane / 32)
//                  gets tokens 8 i + 4 h .. + 3 of query row r,
//   O^T = V^T P^T  whose second operand these are as they lie, if a slot
//                  group of V^T holds tokens 4 h .. 4 h + 3 and 8 + 4 h ..
//                  8 + 4 h + 3 of each 16 (V is stored in that order).
//
// So weights stay in their lanes, a row's maximum needs one exchange of
// halves, and rescaling is a product with a lane's own number.
//
// Measured on an MI355X (a matrix product of 8192^3 in bf16 runs at 1240
// TFLOP/s): a prompt of 8192 tokens, 32 heads of 128 on 8 in e4m3, 566 us,
// 970 TFLOP/s (555 to 592 us from card to card).  Steps there, on one card:
// two waves a SIMD instead of one 1400 -> 752 us; no short-circuit conditions,
// which had cost registers, 737; products in groups whose operands are read
// one group ahead, the weights' arithmetic beside them and the scores of the
// next step before the values of this one 604; keys' halves apart in LDS 598;
// 8 waves that share a step 572; their products first 3 % less again.  What is
// left is vector arithmetic: about 265 instructions a wave and step beside 32
// matrix products, 49 % of the vector units' time and 43 % of the matrix
// units', which hardly overlap further with two waves a SIMD.  With 64
// channels a head there are 16 products beside about 315 vector instructions,
// and the values of a step are transposed by half of the waves: two prompts of
// up to 8000 tokens under a window of 1024, 16 heads of 64 in fp16, 152 us,
// 50 % of the vector units' time and 19 % of the matrix units'.
//
// SHARED: as in kv_few.hpp; with p.prefix the row tiles are those of a group,
// every row sees all shared tokens, and parts (m, sum w, sum w v) are left for
// the launch over the sequences' own tokens.  256 samples of one prompt of 32768
// tokens, 64 heads of 128 on 8 in e4m3: 293 us of 325 (275 GFLOP, 940 TFLOP/s),
// 49 % and 44 % of the vector and matrix units' time.  64 of one of 4096: 20 us in
// 16 parts of 4 steps, 9 % and 5 %: waits for pages, keys and each other.
#pragma once

#include "kv_attend.hpp"

namespace tpl {
namespace kv {

constexpr int kTokens = 64;    // tokens of a step
constexpr int kInfo = 128;     // 16-token groups whose pages are looked up at a time

// The row tile x: its sequence (or group of them), how many of its first tokens
// are another's, and the row of the table that names those.
struct TileAt {
    int b, row, cut;
    Seq s;
};

template <bool SHARED>
__device__ __forceinline__ TileAt tile_at(const AttendArgs& p, int x) {
    TileAt t;
    t.cut = 0;
    if (SHARED && p.prefix) {
        // Groups are numbered as sequences are.
        const int lane = threadIdx.x & 63;
        t.b = t.row = -1;
        t.s = Seq{0, 0, 0};
        for (int g0 = 0; g0 < p.s.count; g0 += 64) {
            const Group g = read_group(p, g0 + lane < p.s.count ? g0 + lane : p.s.count - 1);
            const uint64_t m = __ballot(g0 + lane < p.s.count && g.s.n > 0 && g.s.row0 / p.tile_tokens + g0 + lane <= x);
            if (m) {
                const int from = 63 - __builtin_clzll(m);
                t.b = g0 + from;
                t.row = __builtin_amdgcn_readlane(g.first, from);
                t.s.row0 = __builtin_amdgcn_readlane(g.s.row0, from);
                t.s.n = __builtin_amdgcn_readlane(g.s.n, from);
                t.s.length = t.cut = __builtin_amdgcn_readlane(g.s.length, from);
            }
        }
        return t;
    }
    const TileSeq q = seq_of_tile(p.g, p.tile_tokens, x);
    t.b = t.row = q.b;
    t.s = q.s;
    if constexpr (SHARED) {
        if (t.b >= 0) {
            const Common c = common_of(p, t.b, t.s);
            t.row = uniform(c.row);
            t.cut = uniform(c.cut);
        }
    }
    return t;
}

template <typename T, bool HELD8, int D, int WAVES, bool SHARED>
__global__ void __launch_bounds__(WAVES * 64, D <= 128 ? 2 : 1) k_tile(AttendArgs p) {
    typedef typename T::one one;
    typedef typename T::x8 x8;
    // Weights are multiplied in the cache's type, with an e4m3 value's scale in
    // bf16.  One 16-bit number each, an error of half a step of the output's
    // type at most; two, as kv_few.hpp takes, cost a prompt of 8192 tokens 813
    // against 590 us (e4m3) and 953 against 590 (16 bit), and are taken only
    // where the output keeps 11 bits and the weight would keep 8.  The sum takes
    // weights before their rounding: after it, so that equal values cancel
    // exactly, it cost 3 % of that prompt and made no random output more exact.
    typedef typename std::conditional<HELD8, Bf16, T>::type V;
    constexpr bool kTwo = HELD8 && std::is_same<T, Fp16>::value;
    constexpr int W = HELD8 ? 1 : 2;
    typedef typename std::conditional<HELD8, E4m3, T>::type H;   // what the cache holds
    constexpr int KS = D / 16, NT = D / 32;
    constexpr int AHEAD = 1;   // groups of products (see below) that operands are read ahead; 2 and 3 gained nothing
    // Rows of K padded by 16 bytes: an odd number of 16-byte units, so that
    // 16 lanes reading a column of it reach all banks.  Rows of V^T are 128
    // bytes, their 16-byte units exchanged by the row's number: both the
    // reads (rows next to each other, one unit) and the writes (rows 8 apart)
    // then spread over the banks.
    constexpr int KP = D * 2 + 16, KB = kTokens * KP, VB = D * kTokens * 2;
    constexpr int THREADS = WAVES * 64;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (KB + VB)];   // two steps' keys, then values
    // Two halves, looked up in turn.
    __shared__ const uint8_t *gk[2 * kInfo], *gv[2 * kInfo];
    __shared__ int gbase[2 * kInfo];
    // Of a key's scale its product with the scores' factor.  Of a value's
    // scale the power of two goes in where the values are converted; what is
    // left of it, 1 to under 2, multiplies the weights: its logarithm is
    // added in the exponent, and its reciprocal brings the weights' sum back.
    __shared__ __attribute__((aligned(16))) float gks[2 * kInfo], gvs[2 * kInfo], glg[2 * kInfo], grv[2 * kInfo];
    // A bit a group: all of it is seen by all of the tile's rows.
    __shared__ uint64_t gfull[2 * kInfo / 64];
    __shared__ int left_out;   // whether put_v left out values that are no finite numbers

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Heads next to each other in the grid lie on different dies, a head's
    // tiles on one, which keeps its keys and values in that die's L2; later
    // tiles, which see more, begin first.
    const int h = blockIdx.x % p.c.kv_heads;
    const int rest = blockIdx.x / p.c.kv_heads;
    const int split = rest % p.splits;
    const int x = p.tiles - 1 - rest / p.splits;
    const TileAt mine = tile_at<SHARED>(p, x);
    const int b = mine.b, cut = mine.cut;
    const Seq s = mine.s;
    if (b < 0) return;
    if ((int64_t)s.n * p.group <= p.few) return;
    const int t0 = (x - s.row0 / p.tile_tokens - b) * p.tile_tokens;   // the tile's first new token
    if (t0 < 0 || t0 >= s.n) return;
    const int tn = s.n - t0 < p.tile_tokens ? s.n - t0 : p.tile_tokens;
    const int rows = tn * p.group;
    const bool flat = SHARED && p.prefix;   // all rows see as far as the last shared token
    const int pmin = flat ? s.length - 1 : s.length - s.n + t0, pmax = flat ? pmin : pmin + tn - 1;
    const Span span = SHARED ? span_cut(cut, pmax + 1 < p.cap ? pmax + 1 : p.cap, true, !flat) : span_of(p, pmin, pmax);
    const int32_t* pages = p.g.table + b * p.g.table_row;
    const int32_t* first_pages = SHARED ? p.g.table + mine.row * p.g.table_row : pages;
    const int win = p.a.window ? p.a.window : 0x7fffffff;
    // Group t's tokens that count: its first ones are another's up to the cut.
    struct Range {
        int lo, hi;
    };
    auto range_of = [&](int t) { return Range{SHARED && t >= span.na ? cut : 0, SHARED && t < span.na ? cut - 1 : kNowhere}; };
    // Whether a row at `at` sees token j, both ends of rows given; whether all
    // or any of them see the 16 from `base` on.
    auto sees = [&](Range rg, int j, int at, int last) {
        if constexpr (SHARED)
            return (j <= at) & (j >= rg.lo) & (j <= rg.hi);
        else
            return (j <= at) & ((last - j < win) | (j < p.a.sinks));
    };
    auto whole16 = [&](Range rg, int base, int first_at, int last_at) {
        if constexpr (SHARED)
            return (base <= first_at - 15) & (base >= rg.lo) & (base <= rg.hi - 15);
        else
            return (base <= first_at - 15) & ((last_at - base < win) | (base + 15 < p.a.sinks));
    };
    auto some16 = [&](int base, int first_at, int last_at) {
        if constexpr (SHARED)
            return base <= last_at;
        else
            return (base <= last_at) & ((first_at - base - 15 < win) | (base < p.a.sinks));
    };

    const int row = wave * 32 + r;
    const bool there = row < rows;
    const int qi = (int)fdiv((uint32_t)row, p.div_group);
    const int head = h * p.group + row - qi * p.group;
    const int pos = there ? flat ? pmin : pmin + qi : -1;
    // Positions of this wave's rows.
    const int wfirst = wave * 32, wlast = (wave * 32 + 31 < rows ? wave * 32 + 31 : rows - 1);
    const bool wany = wfirst < rows;
    const int wmin = flat ? pmin : pmin + (int)fdiv((uint32_t)wfirst, p.div_group);
    const int wmax = !wany ? -1 : flat ? pmin : pmin + (int)fdiv((uint32_t)wlast, p.div_group);

    x8 q[KS];
    {
        const one* src = (const one*)p.a.q + (there ? (s.row0 + t0 + qi) * p.a.q_token + head * p.a.q_head : 0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            // The 8 channels that unit k * 2 + hh of a row of keys in LDS holds.
            // Of e4m3 keys the first halves of every 16 channels lie before the
            // second ones, so that lanes write units next to each other.
            const int unit = k * 2 + hh;
            const int ch = !HELD8 ? unit * 8 : unit < D / 16 ? unit * 16 : unit * 16 - D + 8;
            u32x4 w = {0, 0, 0, 0};
            if (there && ch < p.c.dim) w = *reinterpret_cast<const u32x4*>(src + ch);
            q[k] = __builtin_bit_cast(x8, w);
        }
    }
    f32x16 o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;
    float m = neg_inf(), l = 0.0f;

    const int all = (span.n + 3) >> 2;   // steps of 64 tokens
    const int per = (all + p.splits - 1) / p.splits;
    const int st0 = split * per, st1 = st0 + per < all ? st0 + per : all;

    // What a thread brings: KN 16-byte pieces of keys; VN units of 4 tokens by
    // 8 channels of values.
    constexpr int PIECES = D * W / 16, KN = (kTokens * PIECES + THREADS - 1) / THREADS;
    constexpr int CH8 = D / 8, VN = (kTokens / 4 * CH8 + THREADS - 1) / THREADS;
    typedef typename std::conditional<HELD8, u32x2, u32x4>::type VPiece;
    u32x4 kreg[KN];
    VPiece vreg[VN][4];
#pragma unroll
    for (int i = 0; i < KN; ++i) kreg[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < VN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) vreg[i][e] = VPiece{};

    // Where the next groups lie, their first tokens and scales.  A group
    // whose page is not there stands beyond every position; its loads go to
    // page 0.
    auto look_up = [&](int group0) {
        const int t = group0 + tid, to = t & (2 * kInfo - 1);
        if (tid >= kInfo) return;
        int where = -1, base = 0, slot = 0;
        float ks = 0.0f, vs = 0.0f;
        if (t < span.n) {
            base = span.base(t);
            const int pg = (int)fdiv((uint32_t)base, p.div_page);
            where = (SHARED && t < span.na ? first_pages : pages)[pg];
            if (where >= p.c.pages) where = -1;
            if (where >= 0) slot = base - pg * p.c.page;
            if (HELD8 && where >= 0) {
                const int blk = (int)fdiv((uint32_t)slot, p.div_block);
                ks = p.c.k_scale[where * p.c.ks_page + h * p.c.ks_head + blk * p.c.ks_block];
                vs = p.c.v_scale[where * p.c.vs_page + h * p.c.vs_head + blk * p.c.vs_block];
            }
        }
        base = where < 0 ? kNowhere : base;
        gbase[to] = base;
        const uint64_t seen = __ballot(whole16(range_of(t), base, pmin, pmax));
        if (lane == 0) gfull[to >> 6] = seen;
        where = where < 0 ? 0 : where;
        gk[to] = (const uint8_t*)p.c.k + (where * p.c.k_page + slot * p.c.k_token + h * p.c.k_head) * W;
        gv[to] = (const uint8_t*)p.c.v + (where * p.c.v_page + slot * p.c.v_token + h * p.c.v_head) * W;
        // A masked score is minus infinity times this: it must not be zero.
        gks[to] = HELD8 ? fmaxf(ks * p.factor, 1.17549435e-38f) : p.factor;
        if constexpr (HELD8) {
            vs = vs < 1.17549435e-38f ? 1.17549435e-38f : vs;
            const float rest = scale_rest(vs);
            gvs[to] = vs;
            glg[to] = rest == 1.0f ? 0.0f : __builtin_log2f(rest);
            grv[to] = 1.0f / rest;
        }
    };
    // Lanes beyond the head's channels read its first ones: those of keys are
    // cleared before they meet the queries' zeros, those of values only reach
    // sums that nothing stores.
    auto all_see = [&](int step) {
        const uint64_t m = gfull[(step >> 4) & (2 * kInfo / 64 - 1)];
        const uint32_t half = (step & 8) ? (uint32_t)(m >> 32) : (uint32_t)m;
        return ((__builtin_amdgcn_readfirstlane(half) >> ((step & 7) * 4)) & 15) == 15;
    };
    auto fetch_k = [&](int step) {
        const int g0 = (step * 4) & (2 * kInfo - 1);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int id = i * THREADS + tid, tok = id / PIECES, ch = (id - tok * PIECES) * (16 / W);
            if (KN * THREADS == kTokens * PIECES || id < kTokens * PIECES)
                kreg[i] = *reinterpret_cast<const u32x4*>(gk[g0 + (tok >> 4)] + ((tok & 15) * (int)p.c.k_token + (ch < p.c.dim ? ch : 0)) * W);
        }
    };
    auto fetch_v = [&](int step) {
        const int g0 = (step * 4) & (2 * kInfo - 1);
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int id = i * THREADS + tid, quad = id / CH8, ch = (id - quad * CH8) * 8;
            if (VN * THREADS == kTokens / 4 * CH8 || id < kTokens / 4 * CH8) {
                const uint8_t* v = gv[g0 + (quad >> 2)] + ((quad & 3) * 4 * (int)p.c.v_token + (ch < p.c.dim ? ch : 0)) * W;
#pragma unroll
                for (int e = 0; e < 4; ++e) vreg[i][e] = *reinterpret_cast<const VPiece*>(v + e * (int)p.c.v_token * W);
            }
        }
    };
    // Addresses in LDS are built from the step's buffer, so that they are
    // computed where they are used instead of held in registers throughout.
    auto put_k = [&](int at) {
        if (p.c.dim < D)
#pragma unroll
            for (int i = 0; i < KN; ++i)
                if ((i * THREADS + tid) % PIECES * (16 / W) >= p.c.dim) kreg[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int id = i * THREADS + tid, tok = id / PIECES, pc = id - tok * PIECES;
            if (KN * THREADS == kTokens * PIECES || id < kTokens * PIECES) {
                if constexpr (HELD8) {
                    u32x4 a, d;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[2 * k] = T::template from_e4m3<false>(kreg[i][k]);
                        a[2 * k + 1] = T::template from_e4m3<true>(kreg[i][k]);
                        d[2 * k] = T::template from_e4m3<false>(kreg[i][k + 2]);
                        d[2 * k + 1] = T::template from_e4m3<true>(kreg[i][k + 2]);
                    }
                    *reinterpret_cast<u32x4*>(lds + at + tok * KP + pc * 16) = a;
                    *reinterpret_cast<u32x4*>(lds + at + tok * KP + D + pc * 16) = d;
                } else {
                    *reinterpret_cast<u32x4*>(lds + at + tok * KP + pc * 16) = kreg[i];
                }
            }
        }
    };
    auto put_v = [&](int step, int buf) {
        const int g0 = (step * 4) & (2 * kInfo - 1);
        if (!all_see(step)) {   // a token that no row sees weighs nothing, whatever its place holds
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const int quad = (i * THREADS + tid) / CH8 % (kTokens / 4);
                const int j = gbase[g0 + (quad >> 2)] + (quad & 3) * 4;
                const Range rg = range_of(step * 4 + (quad >> 2));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!sees(rg, j + e, pmax, pmin)) vreg[i][e] = VPiece{};
                // Rows that do not see a token multiply its values with zeros,
                // which an infinity or NaN among them would show: such values
                // are left out here, and added at the end to the rows that do
                // see them.
                const int gb = j - (quad & 3) * 4;
                if (whole16(rg, gb, pmin, pmax)) continue;   // all rows see these 16
                bool some = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int k = 0; k < (int)(sizeof(VPiece) / 4); ++k) {
                        uint32_t w = vreg[i][e][k];
                        some |= clear_bad<H>(w);
                        vreg[i][e][k] = w;
                    }
                if (some) left_out = 1;
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int id = i * THREADS + tid, quad = id / CH8, c8 = id - quad * CH8;
            if (VN * THREADS == kTokens / 4 * CH8 || id < kTokens / 4 * CH8) {
                // Of each 16 tokens: pair 0 holds quads 0 and 2, pair 1 quads 1 and 3.
                const int pair = (quad >> 2) * 2 + (quad & 1), half = (quad >> 1) & 1;
                // The scale's power of two goes in with the conversion.
                const float vs = HELD8 ? gvs[g0 + (quad >> 2)] : 1.0f;
                const int at = buf + c8 * 1024 + half * 8 + ((pair ^ ((c8 & 1) * 4) ^ (c8 & 7)) << 4);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (HELD8)
                            w[e] = (t & 2) ? bf16_from_e4m3<true>(vreg[i][e][t >> 2], vs) : bf16_from_e4m3<false>(vreg[i][e][t >> 2], vs);
                        else
                            w[e] = vreg[i][e][t >> 1];
                    }
                    const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
                    *reinterpret_cast<u32x2*>(lds + (at ^ ((t >> 1) << 4)) + t * 128) =
                        u32x2{__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel)};
                }
            }
        }
    };
    f32x16 sc[2];
    f32x16 sn[2];
    // The products go in groups of NT: four groups of key products (32 tokens,
    // half of the channels), four of value products (16 tokens).  A group's
    // operands are read while the one before it is multiplied.
    struct Part {
        u32x4 w[NT];
    };
    auto read_k = [&](Part& f, int at, int g) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            f.w[i] = *reinterpret_cast<const u32x4*>(lds + at + ((g >> 1) * 32 + r) * KP + ((g & 1) * NT + i) * 32 + hh * 16);
    };
    auto mul_k = [&](const Part& f, int g) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const u32x4 w = f.w[i];
            if ((g & 1) == 0 && i == 0) {
                f32x16 zero;
#pragma unroll
                for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
                sn[g >> 1] = T::mfma32(__builtin_bit_cast(x8, w), q[0], zero);
            } else {
                sn[g >> 1] = T::mfma32(__builtin_bit_cast(x8, w), q[(g & 1) * NT + i], sn[g >> 1]);
            }
        }
    };
    auto read_v = [&](Part& f, int vat, int z) {
#pragma unroll
        for (int t = 0; t < NT; ++t) f.w[t] = *reinterpret_cast<const u32x4*>(lds + (vat ^ (((z * 2) ^ ((t & 1) * 4)) << 4)) + t * 4096);
    };
    // Whether a step is seen by all of the wave's rows whole, by none at all.
    auto sight = [&](int step, bool& full, bool& any) {
        const int g0 = (step * 4) & (2 * kInfo - 1);
        full = true, any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int base = __builtin_amdgcn_readfirstlane(gbase[g0 + i]);
            full = full & whole16(range_of(step * 4 + i), base, wmin, wmax);
            any = any | some16(base, wmin, wmax);
        }
    };
    auto mask = [&](int step) {
        const int g0 = (step * 4) & (2 * kInfo - 1);
#pragma unroll
        for (int z = 0; z < 4; ++z) {   // 16 tokens; `d` tokens back from the row lies the lane's first
            const int base = __builtin_amdgcn_readfirstlane(gbase[g0 + z]);
            const Range rg = range_of(step * 4 + z);
            const int last = SHARED && rg.hi < pos ? rg.hi : pos;
            const int d = last - base - hh * 4;
            // The last `w` tokens up to there are seen.
            const uint32_t w = !SHARED ? (uint32_t)win : last < rg.lo ? 0u : (uint32_t)(last - rg.lo + 1);
            const int sk = p.a.sinks - base - hh * 4;
            if (!SHARED && base < p.a.sinks) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = (i >> 2) * 8 + (i & 3);
                    if (!(((uint32_t)(d - t) < w) | ((t < sk) & (t <= d)))) sc[z >> 1][(z & 1) * 8 + i] = neg_inf();
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = (i >> 2) * 8 + (i & 3);
                    if (!((uint32_t)(d - t) < w)) sc[z >> 1][(z & 1) * 8 + i] = neg_inf();
                }
            }
        }
    };

    // The steps' pipeline: while step st's weights are taken and multiplied
    // with its values, step st + 1's scores are already under way (independent
    // matrix products to fill the exponentials' time), its values and step
    // st + 2's keys are brought into LDS, and what follows is being read.
    bool any = false;   // of the step at hand
    if (tid == 0) left_out = 0;
    if (st0 < st1) {
        look_up((st0 * 4) & ~(kInfo - 1));
        if ((st0 * 4 & (kInfo - 1)) + 16 > kInfo) look_up((st0 * 4 & ~(kInfo - 1)) + kInfo);
        __syncthreads();
        fetch_k(st0);
        fetch_v(st0);
        put_k(0);
        put_v(st0, 2 * KB);
        if (st0 + 1 < st1) fetch_k(st0 + 1);
        __syncthreads();
        bool full;
        sight(st0, full, any);
        {
            Part f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                read_k(f, 0, g);
                mul_k(f, g);
            }
            sc[0] = sn[0];
            sc[1] = sn[1];
        }
        if (!full) mask(st0);
        if (st0 + 1 < st1) {
            put_k(KB);
            fetch_v(st0 + 1);
            if (st0 + 2 < st1) fetch_k(st0 + 2);
        }
        __syncthreads();
    }
    for (int st = st0; st < st1; ++st) {
        const int odd = (st - st0) & 1;
        const int kat = odd ? 0 : KB;                     // step st + 1's keys
        const int vat0 = 2 * KB + (odd ? VB : 0);         // step st's values
        const int vat = vat0 + r * 128 + ((hh ^ (((r >> 1) ^ (r >> 3)) & 7)) << 4);
        const int gi = (st * 4) & (2 * kInfo - 1);
        const bool more = st + 1 < st1;
        bool full = true, next = more;
        if (more && !all_see(st + 1)) sight(st + 1, full, next);
        if (any | next) {
            Part f[AHEAD + 1];
            // The order of the groups: weights of 16 tokens are ready before
            // their values' products, and what is left of the weights goes
            // beside each.
            auto read = [&](int at) {
                Part& operand = f[at % (AHEAD + 1)];
                switch (at) {
                case 0: case 1: case 2: return read_k(operand, kat, at);
                case 4: return read_k(operand, kat, 3);
                case 3: return read_v(operand, vat, 0);
                default: return read_v(operand, vat, at - 4);
                }
            };
#pragma unroll
            for (int at = 0; at < AHEAD; ++at) read(at);
            f32x4 f2, lg, rv;
            if constexpr (HELD8) {
                f2 = *reinterpret_cast<const f32x4*>(gks + gi);
                lg = *reinterpret_cast<const f32x4*>(glg + gi);
                rv = *reinterpret_cast<const f32x4*>(grv + gi);
            } else {
                f2 = f32x4{p.factor, p.factor, p.factor, p.factor};
            }
            float top = neg_inf();
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                float t = neg_inf();
#pragma unroll
                for (int i = 0; i < 8; ++i) t = fmaxf(t, sc[z >> 1][(z & 1) * 8 + i]);
                top = fmaxf(top, t * f2[z]);
            }
            top -= lift<V>();
            if (__any(top > m + kSlack)) {
                top = max32(fmaxf(top, m));
                const float a = top == neg_inf() ? 1.0f : exp2_(m - top);
                m = top;
                l *= a;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[t][i] *= a;
            }
            const float ref = m == neg_inf() ? 0.0f : m;
            u32x4 w[4], w2[4];
            // Weights of 4 of a lane's 8 tokens of 16.
            auto weigh = [&](int z, int half) {
                float e[4];
                const float c = HELD8 ? lg[z] - ref : -ref;
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = exp2_(__builtin_fmaf(sc[z >> 1][(z & 1) * 8 + half * 4 + i], f2[z], c));
                const float s4 = (e[0] + e[1]) + (e[2] + e[3]);
                if constexpr (HELD8)
                    l = __builtin_fmaf(s4, rv[z], l);
                else
                    l += s4;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = pack2<V>(e[2 * i], e[2 * i + 1]);
                    w[z][half * 2 + i] = x;
                    if constexpr (kTwo) w2[z][half * 2 + i] = pack2<V>(e[2 * i] - lo16<V>(x), e[2 * i + 1] - hi16<V>(x));
                }
            };
            auto mul_v = [&](const Part& f, int z) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 x = f.w[t];
                    o[t] = V::mfma32(__builtin_bit_cast(typename V::x8, x), __builtin_bit_cast(typename V::x8, w[z]), o[t]);
                    if constexpr (kTwo) o[t] = V::mfma32(__builtin_bit_cast(typename V::x8, x), __builtin_bit_cast(typename V::x8, w2[z]), o[t]);
                }
            };
            // Of two waves a SIMD the one in its products goes first: 583 -> 566 us
            // for the prompt above; with 4 waves a workgroup it cost 1 %.
            if constexpr (WAVES == 8) __builtin_amdgcn_s_setprio(3);
#pragma unroll
            for (int at = 0; at < 8; ++at) {
                const Part& operand = f[at % (AHEAD + 1)];
                __builtin_amdgcn_sched_barrier(0);
                if (at + AHEAD < 8) read(at + AHEAD);
                if (at < 3 || at == 4)
                    mul_k(operand, at < 3 ? at : 3);
                else
                    mul_v(operand, at == 3 ? 0 : at - 4);
                if (at < 6) weigh(at >> 1, at & 1);
                if (at == 6) weigh(3, 0), weigh(3, 1);
            }
            if constexpr (WAVES == 8) __builtin_amdgcn_s_setprio(0);
            sc[0] = sn[0];
            sc[1] = sn[1];
            if (!full) mask(st + 1);
        }
        any = next;
        if (more) {
            put_v(st + 1, 2 * KB + (odd ? 0 : VB));
            if (st + 2 < st1) {
                put_k(odd ? KB : 0);
                fetch_v(st + 2);
                if (st + 3 < st1) fetch_k(st + 3);
            }
            if (((st + 4) * 4 & (kInfo - 1)) == 0 && st + 4 < st1) look_up((st + 4) * 4);
        }
        __syncthreads();
    }

    if (left_out) {
#pragma unroll 1
        for (int t = st0 * 4; t < st1 * 4 && t < span.n; ++t) {
            const int base = span.base(t), pg = (int)fdiv((uint32_t)base, p.div_page);
            const int where = (SHARED && t < span.na ? first_pages : pages)[pg];
            const Range rg = range_of(t);
            if (where < 0 || where >= p.c.pages) continue;
            if (whole16(rg, base, pmin, pmax)) continue;   // all see it: nothing left out
#pragma unroll 1
            for (int j = base; j < base + 16; ++j) {
                if (!sees(rg, j, pos, pos)) continue;
                const uint8_t* from = (const uint8_t*)p.c.v + (where * p.c.v_page + (j - pg * p.c.page) * p.c.v_token + h * p.c.v_head) * W;
                int h4 = hh * 4, dim = p.c.dim;
                asm volatile("" : "+v"(h4), "+s"(dim));   // no comparison is to be held in registers throughout
#pragma unroll
                for (int u = 0; u < NT; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int ch = u * 32 + (i >> 2) * 8 + h4 + (i & 3);
                        const float v = ch < dim ? value_at<H>(from + ch * W) : 0.0f;
                        if (!(__builtin_fabsf(v) < __builtin_inff())) o[u][i] += v;
                    }
            }
        }
    }

    l = sum32(l);
    if (m == neg_inf() && l != l) m = 0.0f;   // scores that are no numbers, not a row that saw nothing
    // The row again, from the thread's number, rather than held throughout.
    int again = threadIdx.x;
    asm volatile("" : "+v"(again));
    const int orow = (again >> 6) * 32 + (again & 31), oh = again >> 5 & 1;
    if (orow >= rows) return;
    const int oi = (int)fdiv((uint32_t)orow, p.div_group), ohead = h * p.group + orow - oi * p.group;
    if (flat) {
        const int64_t at = ((int64_t)split * p.g.tokens + s.row0 + t0 + oi) * p.a.heads + ohead;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int ch = t * 32 + i * 2 + oh * 4;
                if (ch < p.c.dim)
                    *reinterpret_cast<f32x4*>(p.before + at * p.c.dim + ch) = f32x4{o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]};
            }
        if (oh == 0) p.before_ml[at] = make_float2(m, l);
        return;
    }
    if (p.splits > 1) {
        float* part = p.tile_parts + ((uint64_t)(x * p.c.kv_heads + h) * p.splits + split) * tile_part_floats(D, p.tile_rows);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<f32x4*>(part + ((t * 8 + i / 2 + oh) * p.tile_rows + orow) * 4) =
                    m == neg_inf() ? f32x4{0, 0, 0, 0} : f32x4{o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]};
        if (oh == 0) {
            part[p.tile_rows * D + orow] = m;
            part[p.tile_rows * D + p.tile_rows + orow] = l;
        }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    one* out = (one*)p.a.out + (s.row0 + t0 + oi) * p.a.o_token + ohead * p.a.o_head;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int ch = t * 32 + i * 2 + oh * 4;
            if (ch < p.c.dim) {
                u32x2 w = {0, 0};
                if (l != 0.0f) w = u32x2{pack2<T>(o[t][i] * inv, o[t][i + 1] * inv), pack2<T>(o[t][i + 2] * inv, o[t][i + 3] * inv)};
                *reinterpret_cast<u32x2*>(out + ch) = w;
            }
        }
    if (p.a.lse && oh == 0)
        p.a.lse[(s.row0 + t0 + oi) * p.a.l_token + ohead * p.a.l_head] = l == 0.0f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
}

// Joins a row tile's parts, in their order.  A part is kept by 4 channels,
// then rows: threads next to each other write and read rows next to each
// other.
constexpr int kJoinBlocks = 8;   // of a row tile

template <typename T, int D, bool SHARED>
__global__ void __launch_bounds__(256) k_tile_join(AttendArgs p) {
    typedef typename T::one one;
    const int h = blockIdx.x % p.c.kv_heads, x = blockIdx.x / p.c.kv_heads;
    const TileSeq mine = seq_of_tile(p.g, p.tile_tokens, x);   // the groups' launch is not joined
    const int b = mine.b;
    const Seq s = mine.s;
    if (b < 0) return;
    if ((int64_t)s.n * p.group <= p.few) return;
    const int t0 = (x - s.row0 / p.tile_tokens - b) * p.tile_tokens;
    if (t0 < 0 || t0 >= s.n) return;
    const int tn = s.n - t0 < p.tile_tokens ? s.n - t0 : p.tile_tokens;
    const float* base = p.tile_parts + (uint64_t)(x * p.c.kv_heads + h) * p.splits * tile_part_floats(D, p.tile_rows);
    constexpr int AT_ONCE = 4;
    const int rows = tn * p.group, quads = p.c.dim / 4;
    for (int item = blockIdx.y * 256 + threadIdx.x; item < p.tile_rows * quads; item += kJoinBlocks * 256) {
        const int q = item / p.tile_rows, row = item - q * p.tile_rows;
        if (row >= rows) continue;
        float top = neg_inf(), sum = 0.0f;
        f32x4 y = {0, 0, 0, 0};
        for (int i0 = 0; i0 < p.splits; i0 += AT_ONCE) {
            float m[AT_ONCE], l[AT_ONCE], next = top;
            f32x4 v[AT_ONCE];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const float* part = base + (uint64_t)(i0 + k < p.splits ? i0 + k : p.splits - 1) * tile_part_floats(D, p.tile_rows);
                m[k] = part[p.tile_rows * D + row];
                l[k] = part[p.tile_rows * D + p.tile_rows + row];
                v[k] = *reinterpret_cast<const f32x4*>(part + item * 4);
                if (i0 + k >= p.splits) m[k] = neg_inf();
                next = fmaxf(next, m[k]);
            }
            const float c0 = top == neg_inf() ? 0.0f : exp2_(top - next);
            sum *= c0;
            y *= c0;
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                if (m[k] == neg_inf()) continue;   // nothing in it: no product, which an infinity would show
                const float a = exp2_(m[k] - next);
                sum += l[k] * a;
                y += v[k] * a;
            }
            top = next;
        }
        const int qi = (int)fdiv((uint32_t)row, p.div_group), head = h * p.group + row - qi * p.group;
        const float inv = 1.0f / sum;
        u32x2 w = {0, 0};
        if (sum != 0.0f) w = u32x2{pack2<T>(y[0] * inv, y[1] * inv), pack2<T>(y[2] * inv, y[3] * inv)};
        *reinterpret_cast<u32x2*>((one*)p.a.out + (s.row0 + t0 + qi) * p.a.o_token + head * p.a.o_head + q * 4) = w;
        if (p.a.lse && q == 0)
            p.a.lse[(s.row0 + t0 + qi) * p.a.l_token + head * p.a.l_head] = sum == 0.0f ? neg_inf() : (top + __builtin_log2f(sum)) * kLn2;
    }
}

template <typename T, bool HELD8, int D, bool SHARED>
static hipError_t go(const AttendArgs& p, bool join, hipStream_t st) {
    if (join)
        k_tile_join<T, D, SHARED><<<dim3((unsigned)(p.tiles * p.c.kv_heads), kJoinBlocks), 256, 0, st>>>(p);
    else if (D <= 128 && p.tile_rows == 256)
        k_tile<T, HELD8, D <= 128 ? D : 128, 8, SHARED><<<(unsigned)(p.tiles * p.c.kv_heads * p.splits), 512, 0, st>>>(p);
    else
        k_tile<T, HELD8, D, 4, SHARED><<<(unsigned)(p.tiles * p.c.kv_heads * p.splits), 256, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, bool HELD8, bool SHARED>
static hipError_t go_d(const AttendArgs& p, int dk, bool join, hipStream_t st) {
    switch (dk) {
    case 64: return go<T, HELD8, 64, SHARED>(p, join, st);
    case 96: return go<T, HELD8, 96, SHARED>(p, join, st);
    case 128: return go<T, HELD8, 128, SHARED>(p, join, st);
    case 192: return go<T, HELD8, 192, SHARED>(p, join, st);
    default: return go<T, HELD8, 256, SHARED>(p, join, st);
    }
}

template <bool SHARED>
static hipError_t go_tile(const AttendArgs& p, int dk, bool join, hipStream_t st) {
    const bool held8 = p.c.type == TPL_KV_E4M3;
    if (p.a.type == TPL_KV_BF16)
        return held8 ? go_d<Bf16, true, SHARED>(p, dk, join, st) : go_d<Bf16, false, SHARED>(p, dk, join, st);
    return held8 ? go_d<Fp16, true, SHARED>(p, dk, join, st) : go_d<Fp16, false, SHARED>(p, dk, join, st);
}

}  // namespace kv
}  // namespace tpl
