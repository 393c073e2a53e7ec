// kv_append.hip -- rotation of new keys and queries to their positions and
// their writing, with the values, into the pages of a key/value cache.
//
// y[c] = x[c] cos a - x[c'] sin a, y[c'] = x[c'] cos a + x[c] sin a for the
// pair (c, c') of a head, a = position * inv_freq.  For an e4m3 cache a block
// of tokens of one head is scaled by the least power of two s with
// max |y| <= 448 s, and y / s is rounded once.
//
// Bound: HBM bytes for prompts (each input read and each output written
// once), the call's own latency for single tokens.  Workgroups are told apart
// by a group of tokens (those of one block: they share scales) and by what
// they do: keys, where a wave takes a head at a time, values, which need no
// angles, and queries, which need no scales and go 8 tokens at a time.  A
// lane holds 8 channels, so a wave reads 64 / (dim / 8) whole rows; up to 4
// such reads are under way at once.  A workgroup takes the cosines and sines
// it needs once, in LDS, in 64 bits, while its first rows are on their way.
//
// Measured on an MI355X (HBM copies run at 5.1 to 5.2 TB/s): 65536 tokens of
// 16 + 16 + 16 heads of 64 into a 16-bit cache 156 us, 5.2 TB/s; three prompts
// of up to 4093 tokens, 28 + 4 + 4 heads of 128, e4m3 in blocks of 64: 51 us,
// 3.4 TB/s (before keys, values and queries had workgroups of their own 16 us
// more, with one row under way at a time 31); one token, 32 + 8 + 8 heads of
// 128: 4.8 us; 256 single tokens of the same heads: 8.0 us.
#include "kv.hpp"

namespace tpl {
namespace kv {

struct AppendArgs {
    tpl_kv_cache c;
    tpl_kv_batch g;
    tpl_kv_new a;
    int32_t unit;       // tokens of a group: the block, or kGroup where blocks bear no scale
    int32_t by_token;   // grid.x: 1 a group for each row that begins one, 0 numbered by sequence
    // grid.y: ky workgroups for the keys, ky for the values, then the queries'
    // qt ranges of q_tokens tokens, each in slices of its rows.
    int32_t ky, qt, q_tokens, q_slices;
    int32_t sec_end[TPL_KV_MAX_AXES];
};

constexpr int kGroup = 16;
constexpr int kQueryTokens = 8;   // of a workgroup on the queries of longer groups

// cos and sin of an angle in 64 bits, rounded to 32.  The angle is brought
// into [-pi/4, pi/4] with pi/2 in two parts (a product of up to 31 bits times
// the first is exact inside the fused multiply-add); the Taylor series end
// where the next term is under 2^-44, far below a 32-bit rounding.
__device__ __forceinline__ float2 cos_sin(double angle) {
    const double n = __builtin_rint(angle * 0.63661977236758134308);   // 2 / pi
    double r = __builtin_fma(-n, 1.57079632679489655800, angle);
    r = __builtin_fma(-n, 6.12323399573676603587e-17, r);
    const double z = r * r;
    double s = 1.0 / 6227020800.0;
    s = __builtin_fma(s, z, -1.0 / 39916800.0);
    s = __builtin_fma(s, z, 1.0 / 362880.0);
    s = __builtin_fma(s, z, -1.0 / 5040.0);
    s = __builtin_fma(s, z, 1.0 / 120.0);
    s = __builtin_fma(s, z, -1.0 / 6.0);
    s = __builtin_fma(s * z, r, r);
    double c = -1.0 / 87178291200.0;
    c = __builtin_fma(c, z, 1.0 / 479001600.0);
    c = __builtin_fma(c, z, -1.0 / 3628800.0);
    c = __builtin_fma(c, z, 1.0 / 40320.0);
    c = __builtin_fma(c, z, -1.0 / 720.0);
    c = __builtin_fma(c, z, 1.0 / 24.0);
    c = __builtin_fma(c, z, -0.5);
    c = __builtin_fma(c, z, 1.0);
    // |n| is under 2^53 and r is no number where the angle is none.
    const int q = (int)((int64_t)n & 3);
    const double cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
    return make_float2((float)((q == 1 || q == 2) ? -cc : cc), (float)((q & 2) ? -ss : ss));
}

// How channels turn: not at all; with the one half the rotated channels away,
// where that half is a multiple of 4 (kQuads) or not (kSingles); with the
// next one (kPairs).
enum Mode { kStill, kQuads, kSingles, kPairs };

// 8 channels of a row from `ch`, and for kQuads their partners, 4 at a time,
// which lie on one side of the half.
template <int MODE>
struct Raw {
    u32x4 own;
    u32x2 other[MODE == kQuads ? 2 : 1];
};

template <typename T, int MODE>
__device__ __forceinline__ Raw<MODE> load_raw(const typename T::one* row, int ch, int half) {
    Raw<MODE> r;
    r.own = *reinterpret_cast<const u32x4*>(row + ch);
    if constexpr (MODE == kQuads) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = ch + 4 * j;
            const int partner = c < half ? c + half : c < 2 * half ? c - half : c;
            r.other[j] = *reinterpret_cast<const u32x2*>(row + partner);
        }
    }
    return r;
}

// (cos, sin) of a row's pairs, taken where they are asked for: what stands for
// a row of the workgroup's table where there is none.
struct Taken {
    const AppendArgs& p;
    int row, index;   // of the token: its row, and its place in its sequence
    __device__ __forceinline__ float2 operator[](int f) const {
        int pos = index;
        if (p.a.positions) {
            int axis = 0;
#pragma unroll
            for (int k = 0; k < TPL_KV_MAX_AXES - 1; ++k) axis += (k + 1 < p.a.axes && f >= p.sec_end[k]) ? 1 : 0;
            pos = p.a.positions[axis * p.a.positions_row + row];
        }
        return cos_sin((double)pos * (double)p.a.inv_freq[f]);
    }
};

// The channels, rotated.  `cs`: the row's (cos, sin) by pair.  Products are
// rounded before they are added, as the formula's plain evaluation does, so
// that a block's maximum does not depend on which of the two products a fused
// multiply-add would keep whole.
template <typename T, int MODE, int FROM, typename Angles>
__device__ __forceinline__ void rotate(const Raw<FROM>& r, const typename T::one* row, int ch, int half, Angles cs,
                                       float (&y)[8]) {
#pragma clang fp contract(off)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = r.own[i];
        y[2 * i] = lo16<T>(w);
        y[2 * i + 1] = hi16<T>(w);
    }
    if constexpr (MODE == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ch + 2 * i < 2 * half) {
                const float2 t = cs[(ch >> 1) + i];
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = a * t.x - b * t.y;
                y[2 * i + 1] = b * t.x + a * t.y;
            }
        }
    } else if constexpr (MODE == kQuads) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = ch + 4 * j;
            if (c < 2 * half) {
                const bool first = c < half;
                const uint32_t sign = first ? 0x80000000u : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = r.other[j][i >> 1];
                    const float b = (i & 1) ? hi16<T>(w) : lo16<T>(w);
                    const float2 t = cs[(first ? c : c - half) + i];
                    const float sn = t.y;
                    const float x = y[4 * j + i] * t.x, z = b * __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, sn) ^ sign);
                    y[4 * j + i] = x + z;
                }
            }
        }
    } else if constexpr (MODE == kSingles) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = ch + i;
            if (c < 2 * half) {
                const bool first = c < half;
                const float b = (float)row[first ? c + half : c - half];
                const float2 t = cs[first ? c : c - half];
                const float x = y[i] * t.x, z = b * t.y;
                y[i] = first ? x - z : x + z;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(typename T::one* p, const float y[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<T>(y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<u32x4*>(p) = w;
}

__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

// y / s as 8 e4m3 values.  Where s is a power of two (every scale this kernel
// sets) the quotient is a shift of the exponent; another writer's scale
// takes the division.  The conversion gives NaN for NaN; infinities, which
// are rare and known (`bad`), are made such.
__device__ __forceinline__ u32x2 held8(const float y[8], float s, bool bad) {
    float h[8];
    const uint32_t bits = __builtin_bit_cast(uint32_t, s);
    if ((bits & 0x007fffffu) == 0 && bits != 0) {
        const int e = 127 - (int)(bits >> 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __builtin_amdgcn_ldexpf(y[i], e);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = y[i] / s;
    }
    if (bad)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = finite(h[i]) ? h[i] : __builtin_nanf("");
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(h[4 * i], h[4 * i + 1], 0, false);
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(h[4 * i + 2], h[4 * i + 3], v, true);
    }
    return w;
}

// The least power of two that brings amax to 448 = 0.875 * 2^9 or under.
__device__ __forceinline__ float scale_of(float amax) {
    const float part = __builtin_amdgcn_frexp_mantf(amax);
    int e = __builtin_amdgcn_frexp_expf(amax);
    e = e - 9 + (part > 0.875f ? 1 : 0);
    e = amax == 0.0f ? -126 : (e < -126 ? -126 : (e > 127 ? 127 : e));
    return __builtin_amdgcn_ldexpf(1.0f, e);
}

// U: rows of a lane whose loads are under way at once.  TABLE: the angles of
// all tokens of a group fit the workgroup's LDS.  Where they do not (blocks of
// over 128 tokens at 128 channels) those of keys, and of by_token's queries,
// are taken for each head and pass anew, which bounds the call: the three
// prompts named above take 320 us in blocks of 256 tokens, 64 in blocks of 128.
template <typename T, bool HELD8, int U, int MODE, bool TABLE>
__global__ void __launch_bounds__(256, TABLE ? 4 : 2) k_append(AppendArgs p) {
    typedef typename T::one one;
    constexpr int WAVES = 4;
    extern __shared__ float2 table[];
    const tpl_kv_cache& c = p.c;
    const tpl_kv_batch& g = p.g;
    const tpl_kv_new& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = blockIdx.x, unit = p.unit;

    // The sequence of this group: 64 are looked at together, with all that is
    // needed of them, so that it is known after one load's latency; of those in
    // order it is the last that has the row, or whose groups' numbers begin at
    // or before this one.  A row's sequence is first looked for at the row's
    // own number and before: most sequences of a batch of rows have one each.
    int b = -1;
    Seq s = {0, 0, 0};
    auto look = [&](int b0) {
        const int bb = b0 + lane < g.batch ? b0 + lane : g.batch - 1;
        const Seq x = read_seq(g, bb);
        const bool there = b0 + lane < g.batch && x.n > 0 &&
                           (p.by_token ? (x.row0 <= id && id < x.row0 + x.n) : (x.row0 / unit + 2 * bb <= id));
        const uint64_t m = __ballot(there);
        if (m) {
            const int from = 63 - __builtin_clzll(m);
            b = b0 + from;
            s.row0 = __builtin_amdgcn_readlane(x.row0, from);
            s.n = __builtin_amdgcn_readlane(x.n, from);
            s.length = __builtin_amdgcn_readlane(x.length, from);
        }
        return m != 0;
    };
    const int near = id < g.batch ? id : g.batch - 1;
    if (!p.by_token || !look(near > 63 ? near - 63 : 0))
        for (int b0 = 0; b0 < g.batch; b0 += 64)
            if (look(b0) && p.by_token) break;
    if (b < 0) return;
    const int first = s.length - s.n;   // index of the sequence's first new token
    int i0;                             // index of the group's first token
    if (p.by_token) {
        i0 = first + id - s.row0;
        if (id >= s.row0 + s.n || (id != s.row0 && i0 % unit != 0)) return;
    } else {
        const int64_t blk = first / unit + (int64_t)id - (s.row0 / unit + 2 * b);
        const int64_t x = blk * unit;
        if (x >= s.length) return;
        i0 = x > first ? (int)x : first;
    }
    const int had = i0 % unit;
    const int count = s.length - i0 > unit - had ? unit - had : s.length - i0;
    const int row0 = s.row0 + i0 - first;
    const int pg = i0 / c.page, slot = i0 - pg * c.page;
    const int where = pg < g.width ? g.table[b * g.table_row + pg] : -1;

    const int cpr = c.dim >> 3, rpw = 64 / cpr;
    const int lr = lane / cpr, ch = (lane - lr * cpr) * 8;
    const bool mine = lr < rpw;
    const int pairs = MODE == kStill ? 0 : a.rot >> 1;

    // A wave's task: a head's keys, or its values.  Rows t0 + lr, + rpw, ...
    // are loaded together: past the last one, and in lanes that have no row,
    // the last one again, so that nothing branches.  The first of them are on
    // their way while the angles are taken.
    const bool keys = (int)blockIdx.y < p.ky, queries = (int)blockIdx.y >= 2 * p.ky;
    const int h = (blockIdx.y - (keys ? 0 : p.ky)) * WAVES + wave;
    const int qy = blockIdx.y - 2 * p.ky, slice = qy / p.qt, from = queries ? (qy - slice * p.qt) * p.q_tokens : 0;
    const int to_ = queries && from + p.q_tokens < count ? from + p.q_tokens : count;   // tokens whose angles it needs
    if (from >= count) return;
    Raw<MODE> raw[U];
    auto load = [&](int t0) __attribute__((always_inline)) {
        const one* x = keys ? (const one*)a.k + row0 * a.k_token + h * a.k_head : (const one*)a.v + row0 * a.v_token + h * a.v_head;
        const int64_t xs = keys ? a.k_token : a.v_token;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = t0 + u * rpw + lr;
            raw[u] = load_raw<T, MODE>(x + (i < count ? i : count - 1) * xs, mine ? ch : 0, pairs);
        }
    };
    if (!queries && h < c.kv_heads) load(0);

    if (pairs && (TABLE ? keys || queries : queries && !p.by_token)) {
        for (int i = threadIdx.x; i < (to_ - from) * pairs; i += 64 * WAVES) {
            const int u = i / pairs, f = i - u * pairs, t = from + u;
            int pos = i0 + t;
            if (a.positions) {
                int axis = 0;
#pragma unroll
                for (int k = 0; k < TPL_KV_MAX_AXES - 1; ++k) axis += (k + 1 < a.axes && f >= p.sec_end[k]) ? 1 : 0;
                pos = a.positions[axis * a.positions_row + row0 + t];
            }
            table[i] = cos_sin((double)pos * (double)a.inv_freq[f]);
        }
        __syncthreads();
    }
    auto write = [&](auto mode, auto is_key) __attribute__((always_inline)) {
        constexpr int M = decltype(mode)::value;   // MODE for keys, kStill for values
        constexpr bool key = decltype(is_key)::value;
        const one* x = key ? (const one*)a.k + row0 * a.k_token + h * a.k_head : (const one*)a.v + row0 * a.v_token + h * a.v_head;
        const int64_t xs = key ? a.k_token : a.v_token;
        const int64_t to = key ? where * c.k_page + slot * c.k_token + h * c.k_head
                               : where * c.v_page + slot * c.v_token + h * c.v_head;
        const int64_t ts = key ? c.k_token : c.v_token;
        float y[U][8];
        auto turned = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = t0 + u * rpw + lr, j = i < count ? i : count - 1;
                if constexpr (TABLE)
                    rotate<T, M>(raw[u], x + j * xs, mine ? ch : 0, pairs, table + j * pairs, y[u]);
                else
                    rotate<T, M>(raw[u], x + j * xs, mine ? ch : 0, pairs, Taken{p, row0 + j, i0 + j}, y[u]);
            }
        };
        if constexpr (!HELD8) {
            one* d = (one*)(key ? c.k : c.v) + to;
            for (int t0 = 0; t0 < count; t0 += U * rpw) {
                if (t0) load(t0);
                turned(t0);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (mine && t0 + u * rpw + lr < count) store8<T>(d + (t0 + u * rpw + lr) * ts + ch, y[u]);
            }
        } else {
            float* at = key ? c.k_scale + where * c.ks_page + h * c.ks_head + (slot / c.block) * c.ks_block
                            : c.v_scale + where * c.vs_page + h * c.vs_head + (slot / c.block) * c.vs_block;
            uint8_t* d = (uint8_t*)(key ? c.k : c.v) + to;
            float old = 0.0f;
            if (had) old = *at;
            // A maximum passes over NaN by itself.  An infinity shows in it,
            // and has it taken again over the finite ones.
            float amax = 0.0f;
            for (int t0 = 0; t0 < count; t0 += U * rpw) {
                if (t0) load(t0);
                turned(t0);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, __builtin_fabsf(y[u][i]));
            }
#pragma unroll
            for (int m = 32; m; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
            const bool bad = !finite(amax);
            if (bad) {
                amax = 0.0f;
                for (int t = lr; t < count; t += rpw) {
                    if (!mine) break;
                    float z[8];
                    if constexpr (TABLE)
                        rotate<T, M>(load_raw<T, M>(x + t * xs, ch, pairs), x + t * xs, ch, pairs, table + t * pairs, z);
                    else
                        rotate<T, M>(load_raw<T, M>(x + t * xs, ch, pairs), x + t * xs, ch, pairs, Taken{p, row0 + t, i0 + t}, z);
#pragma unroll
                    for (int i = 0; i < 8; ++i) amax = finite(z[i]) ? fmaxf(amax, __builtin_fabsf(z[i])) : amax;
                }
#pragma unroll
                for (int m = 32; m; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
            }
            float sc = scale_of(amax);
            if (had) {
                const float grown = fmaxf(old, sc);
                if (grown != old) {   // the tokens that the block holds, under the larger scale
                    const float ratio = old / grown;
                    for (int t = lr - had; t < 0; t += rpw) {
                        if (!mine) break;
                        u32x2* w = reinterpret_cast<u32x2*>(d + t * ts + ch);
                        const u32x2 o = *w;
                        float z[8];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            z[4 * i] = __builtin_amdgcn_cvt_f32_fp8(o[i], 0) * ratio;
                            z[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(o[i], 1) * ratio;
                            z[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(o[i], 2) * ratio;
                            z[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(o[i], 3) * ratio;
                        }
                        *w = held8(z, 1.0f, false);
                    }
                }
                sc = grown;
            }
            // Where one batch of loads holds the whole group (single tokens,
            // most blocks of 16), its rows are still there; else they come
            // again, out of the caches.
            for (int t0 = 0; t0 < count; t0 += U * rpw) {
                if (count > U * rpw) {
                    load(t0);
                    turned(t0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (mine && t0 + u * rpw + lr < count)
                        *reinterpret_cast<u32x2*>(d + (t0 + u * rpw + lr) * ts + ch) = held8(y[u], sc, bad);
            }
            if (lane == 0) *at = sc;
        }
    };
    if (!queries) {
        if (where < 0 || where >= c.pages) return;
        if (h >= c.kv_heads) return;
        if (keys)
            write(std::integral_constant<int, MODE>(), std::true_type());
        else
            write(std::integral_constant<int, kStill>(), std::false_type());
        return;
    }

    // The queries: rows of (token, head).  A row is read and written by one
    // wave in one step, reads first, so q_out may be q itself.
    const int rows = (to_ - from) * a.heads, stride = p.q_slices * WAVES * rpw;
    for (int r0 = (slice * WAVES + wave) * rpw; r0 < rows; r0 += stride * U) {
        Raw<MODE> w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * stride + lr < rows ? r0 + u * stride + lr : rows - 1;
            const int t = r / a.heads, hq = r - t * a.heads;
            w[u] = load_raw<T, MODE>((const one*)a.q + (row0 + from + t) * a.q_token + hq * a.q_head, mine ? ch : 0, pairs);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * stride + lr;
            if (mine && r < rows) {
                const int t = r / a.heads, hq = r - t * a.heads;
                const one* x = (const one*)a.q + (row0 + from + t) * a.q_token + hq * a.q_head;
                float y[8];
                if constexpr (TABLE)
                    rotate<T, MODE>(w[u], x, ch, pairs, table + t * pairs, y);
                else if (p.by_token)
                    rotate<T, MODE>(w[u], x, ch, pairs, Taken{p, row0 + from + t, i0 + from + t}, y);
                else
                    rotate<T, MODE>(w[u], x, ch, pairs, table + t * pairs, y);
                store8<T>((one*)a.q_out + (row0 + from + t) * a.o_token + hq * a.o_head + ch, y);
            }
        }
    }
}

template <typename T, bool HELD8, int MODE>
static void launch_u(const AppendArgs& p, int u, dim3 grid, size_t lds, hipStream_t st) {
    if (u == 1)
        k_append<T, HELD8, 1, MODE, true><<<grid, 256, lds, st>>>(p);
    else if (u == 2)
        k_append<T, HELD8, 2, MODE, true><<<grid, 256, lds, st>>>(p);
    else
        k_append<T, HELD8, 4, MODE, true><<<grid, 256, lds, st>>>(p);
}

template <typename T, bool HELD8>
static hipError_t launch_mode(const AppendArgs& p, int u, dim3 grid, size_t lds, hipStream_t st) {
    if (!p.a.inv_freq)
        launch_u<T, HELD8, kStill>(p, u, grid, lds, st);
    else if (p.a.interleaved)
        launch_u<T, HELD8, kPairs>(p, u, grid, lds, st);
    else if (p.a.rot % 8 == 0)
        launch_u<T, HELD8, kQuads>(p, u, grid, lds, st);
    else
        launch_u<T, HELD8, kSingles>(p, u, grid, lds, st);
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_long(const AppendArgs& p, dim3 grid, size_t lds, hipStream_t st) {
    if (p.a.interleaved)
        k_append<T, true, 1, kPairs, false><<<grid, 256, lds, st>>>(p);
    else
        k_append<T, true, 1, kSingles, false><<<grid, 256, lds, st>>>(p);
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_append(const AppendArgs& p, int u, dim3 grid, size_t lds, hipStream_t st) {
    return p.c.type == TPL_KV_E4M3 ? launch_mode<T, true>(p, u, grid, lds, st) : launch_mode<T, false>(p, u, grid, lds, st);
}

static int append_impl(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_new* a, hipStream_t st) {
    if (!c || !g || !a) return fail_status(TPL_E_ARG, "cache, batch and arguments must not be NULL");
    if (const char* why = check_cache(c)) return fail_status(TPL_E_ARG, why);
    if (const char* why = check_batch(*c, g)) return fail_status(TPL_E_ARG, why);
    if (a->type != TPL_KV_BF16 && a->type != TPL_KV_FP16)
        return fail_status(TPL_E_DTYPE, "keys, values and queries must be bf16 or fp16");
    if (c->type != TPL_KV_E4M3 && c->type != a->type)
        return fail_status(TPL_E_DTYPE, "a 16-bit cache holds the type of its keys and values");
    if (a->inv_freq) {
        if (a->rot < 2 || a->rot > c->dim || (a->rot & 1))
            return fail_status(TPL_E_ARG, "rotated channels must be an even number, 2 .. dim");
        if (a->axes < 1 || a->axes > TPL_KV_MAX_AXES) return fail_status(TPL_E_ARG, "positions must have 1 .. 4 axes");
        if (a->axes > 1) {
            if (!a->positions) return fail_status(TPL_E_ARG, "sections need positions");
            int64_t sum = 0;
            for (int i = 0; i < a->axes; ++i) {
                if (a->sections[i] < 0) return fail_status(TPL_E_ARG, "sections must be >= 0");
                sum += a->sections[i];
            }
            if (sum != a->rot / 2) return fail_status(TPL_E_ARG, "sections must add up to the rotated pairs");
        }
    }
    if (a->q && (a->heads < 1 || a->heads > 65535)) return fail_status(TPL_E_ARG, "heads must be 1 .. 65535");
    if (g->batch == 0 || g->tokens == 0) return TPL_OK;
    if (!a->k || !a->v) return fail_status(TPL_E_ARG, "k and v must not be NULL");
    if (a->q && !a->q_out) return fail_status(TPL_E_ARG, "q needs q_out");
    if (!aligned16(a->k, a->k_token, a->k_head, 2) || !aligned16(a->v, a->v_token, a->v_head, 2) ||
        (a->q && (!aligned16(a->q, a->q_token, a->q_head, 2) || !aligned16(a->q_out, a->o_token, a->o_head, 2))))
        return fail_status(TPL_E_LAYOUT, "k, v, q and q_out must start, and their rows and heads lie, on 16 bytes");

    AppendArgs p;
    p.c = *c;
    p.g = *g;
    p.a = *a;
    if (!a->inv_freq) p.a.rot = 0;
    p.unit = c->type == TPL_KV_E4M3 ? c->block : kGroup;
    int end = 0;
    for (int i = 0; i < TPL_KV_MAX_AXES; ++i) {
        end += (a->inv_freq && a->axes > 1 && i < a->axes) ? a->sections[i] : 0;
        p.sec_end[i] = end;
    }
    // A sequence's groups are numbered from starts / unit + 2 b on, which
    // leaves room for the two that its ends may cut; where there are more
    // such numbers than rows (single tokens), each row asks whether it
    // begins a group.
    const int64_t numbered = g->tokens / p.unit + 2 * (int64_t)g->batch;
    p.by_token = g->tokens <= numbered ? 1 : 0;
    const int64_t gx = p.by_token ? g->tokens : numbered;
    // Rows under way at once: one where most groups are single tokens, else as
    // many as a group's tokens fill.
    const int rpw = 64 / (c->dim / 8);
    const int u = p.by_token ? 1 : p.unit > 2 * rpw ? 4 : 2;
    // A head a wave; the queries of single tokens in slices of a row a wave,
    // those of longer groups by kQueryTokens tokens, or by 4 times as many
    // where a block's would be more workgroups than grid.y takes.
    p.ky = (c->kv_heads + 3) / 4;
    p.qt = 1, p.q_tokens = p.unit, p.q_slices = 0;
    if (a->q && p.by_token) p.q_slices = (int)((a->heads + 4 * (int64_t)rpw - 1) / (4 * rpw));
    if (a->q && !p.by_token) {
        p.q_tokens = p.unit <= 32768 * kQueryTokens ? kQueryTokens : 4 * kQueryTokens;
        p.qt = (p.unit + p.q_tokens - 1) / p.q_tokens, p.q_slices = 1;
    }
    const int64_t gy = 2 * p.ky + p.qt * p.q_slices;
    // The table of angles: a group's tokens are no more than there are.  Over
    // 64 KiB only queries of longer groups have one.
    const int64_t angle = p.a.rot / 2 * (int64_t)sizeof(float2);
    int64_t lds = (p.unit < g->tokens ? p.unit : g->tokens) * angle;
    const bool fits = lds <= 64 * 1024;
    if (!fits) lds = a->q && !p.by_token ? p.q_tokens * angle : 0;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    hipError_t e;
    if (a->type == TPL_KV_BF16)
        e = fits ? launch_append<Bf16>(p, u, grid, (size_t)lds, st) : launch_long<Bf16>(p, grid, (size_t)lds, st);
    else
        e = fits ? launch_append<Fp16>(p, u, grid, (size_t)lds, st) : launch_long<Fp16>(p, grid, (size_t)lds, st);
    if (e != hipSuccess) return fail_status(TPL_E_HIP, std::string("HIP launch failed: ") + hipGetErrorString(e));
    return TPL_OK;
}

}  // namespace kv
}  // namespace tpl

extern "C" int tpl_kv_append(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_new* args,
                             hipStream_t stream) {
    try {
        return tpl::kv::append_impl(cache, batch, args, stream);
    } catch (...) {
        return TPL_E_ARG;
    }
}
