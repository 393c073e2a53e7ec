// kv_tile.hip -- attention of many rows a sequence (prompts and their chunks)
// to a paged cache.
//
// The formulas are those of kv_few.hip.  Bound: the matrix units and the
// exponentials.  A workgroup of 4 waves takes 128 query rows (the query heads
// of one cache head, token by token: they share keys and values, and a row
// tile ends at one diagonal), 32 rows a wave, and walks over the cache 64
// tokens at a time.  Keys and values are brought into LDS as 16-bit numbers
// (an e4m3 value is converted once for 128 rows), the values transposed on
// the way, so that both products read whole 16-byte operands:
//
//   S^T = K Q^T    32x32x16: lane (row r = lane % 32, half h = lane / 32)
//                  gets tokens 8 i + 4 h .. + 3 of query row r,
//   O^T = V^T P^T  whose second operand these are as they lie, if a slot
//                  group of V^T holds tokens 4 h .. 4 h + 3 and 8 + 4 h ..
//                  8 + 4 h + 3 of each 16 (V is stored in that order).
//
// So weights stay in their lanes, a row's maximum needs one exchange of
// halves, and rescaling is a product with a lane's own number.
#include "kv_attend.hpp"

namespace tpl {
namespace kv {

constexpr int kTokens = 64;    // tokens of a step
constexpr int kInfo = 256;     // 16-token groups whose pages are looked up at a time

template <typename T, bool HELD8, int D>
__global__ void __launch_bounds__(256) k_tile(AttendArgs p) {
    typedef typename T::one one;
    typedef typename T::x8 x8;
    typedef typename std::conditional<HELD8, Bf16, T>::type V;   // as in kv_few.hip
    constexpr bool kTwo = HELD8 && std::is_same<T, Fp16>::value;
    constexpr int W = HELD8 ? 1 : 2;
    constexpr int KS = D / 16, NT = D / 32;
    // Rows of K padded by 16 bytes: an odd number of 16-byte units, so that
    // 16 lanes reading a column of it reach all banks.
    constexpr int KP = D * 2 + 16;
    __shared__ __attribute__((aligned(16))) uint8_t ldsk[kTokens * KP];
    __shared__ __attribute__((aligned(16))) uint8_t ldsv[D * kTokens * 2];
    __shared__ int gpage[kInfo], gbase[kInfo];
    __shared__ float gks[kInfo], gvs[kInfo];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Heads next to each other in the grid lie on different dies, a head's
    // tiles on one, which keeps its keys and values in that die's L2; later
    // tiles, which see more, begin first.
    const int h = blockIdx.x % p.c.kv_heads;
    const int rest = blockIdx.x / p.c.kv_heads;
    const int split = rest % p.splits;
    const int x = p.tiles - 1 - rest / p.splits;
    // Sequence b's tiles are numbered from starts[b] / tile_tokens + b.
    int before = 0;
    for (int b0 = 0; b0 < p.g.batch; b0 += 64) {
        const int bb = b0 + lane;
        before += __builtin_popcountll(__ballot(bb < p.g.batch && p.g.starts[bb] / p.tile_tokens + bb <= x));
    }
    if (before == 0) return;
    const int b = before - 1;
    const Seq s = read_seq(p.g, b);
    if ((int64_t)s.n * p.group <= p.few) return;
    const int t0 = (x - s.row0 / p.tile_tokens - b) * p.tile_tokens;   // the tile's first new token
    if (t0 < 0 || t0 >= s.n) return;
    const int tn = s.n - t0 < p.tile_tokens ? s.n - t0 : p.tile_tokens;
    const int rows = tn * p.group;
    const int pmin = s.length - s.n + t0, pmax = pmin + tn - 1;
    const Span span = span_of(p, pmin, pmax);
    const int32_t* pages = p.g.table + b * p.g.table_row;

    const int row = wave * 32 + r;
    const bool there = row < rows;
    const int qi = (int)fdiv((uint32_t)row, p.div_group);
    const int head = h * p.group + row - qi * p.group;
    const int pos = there ? pmin + qi : -1;
    // Positions of this wave's rows.
    const int wfirst = wave * 32, wlast = (wave * 32 + 31 < rows ? wave * 32 + 31 : rows - 1);
    const bool wany = wfirst < rows;
    const int wmin = pmin + (int)fdiv((uint32_t)wfirst, p.div_group);
    const int wmax = wany ? pmin + (int)fdiv((uint32_t)wlast, p.div_group) : -1;

    x8 q[KS];
    {
        const one* src = (const one*)p.a.q + (there ? (s.row0 + t0 + qi) * p.a.q_token + head * p.a.q_head : 0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int ch = k * 16 + hh * 8;
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
    constexpr int PIECES = D * W / 16, KN = (kTokens * PIECES + 255) / 256;
    constexpr int CH8 = D / 8, VN = (kTokens / 4 * CH8 + 255) / 256;
    u32x4 kreg[KN];
    typedef typename std::conditional<HELD8, u32x2, u32x4>::type VPiece;
    VPiece vreg[VN][4];

    auto look_up = [&](int group0) {   // pages, first tokens and scales of the next groups
        const int t = group0 + tid;
        int where = -1, base = 0;
        float ks = 0.0f, vs = 0.0f;
        if (t < span.n) {
            base = span.base(t);
            const int pg = (int)fdiv((uint32_t)base, p.div_page);
            where = pages[pg];
            if (where >= p.c.pages) where = -1;
            if (HELD8 && where >= 0) {
                const int blk = (int)fdiv((uint32_t)(base - pg * p.c.page), p.div_block);
                ks = p.c.k_scale[where * p.c.ks_page + h * p.c.ks_head + blk * p.c.ks_block];
                vs = p.c.v_scale[where * p.c.vs_page + h * p.c.vs_head + blk * p.c.vs_block];
            }
        }
        gpage[tid] = where;
        gbase[tid] = where < 0 ? 0x7fffff00 : base;
        gks[tid] = HELD8 ? ks * p.factor : p.factor;
        gvs[tid] = vs;
    };
    auto fetch = [&](int step) {
        const int g0 = (step * 4) & (kInfo - 1);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int id = i * 256 + tid, tok = id / PIECES, ch = (id - tok * PIECES) * (16 / W);
            kreg[i] = u32x4{0, 0, 0, 0};
            if (id < kTokens * PIECES && ch < p.c.dim) {
                const int g = g0 + (tok >> 4), where = gpage[g];
                if (where >= 0) {
                    const int base = gbase[g];
                    const int slot = base - (int)fdiv((uint32_t)base, p.div_page) * p.c.page + (tok & 15);
                    kreg[i] = *reinterpret_cast<const u32x4*>(
                        (const uint8_t*)p.c.k + (where * p.c.k_page + slot * p.c.k_token + h * p.c.k_head + ch) * W);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int id = i * 256 + tid, quad = id / CH8, ch = (id - quad * CH8) * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e) vreg[i][e] = VPiece{};
            if (id < kTokens / 4 * CH8 && ch < p.c.dim) {
                const int g = g0 + (quad >> 2), where = gpage[g];
                if (where >= 0) {
                    const int base = gbase[g];
                    const int slot = base - (int)fdiv((uint32_t)base, p.div_page) * p.c.page + (quad & 3) * 4;
                    const uint8_t* v = (const uint8_t*)p.c.v + (where * p.c.v_page + slot * p.c.v_token + h * p.c.v_head + ch) * W;
                    const int j = base + (quad & 3) * 4;
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // a token that no row sees weighs nothing, whatever its place holds
                        if (j + e <= pmax && (p.a.window == 0 || pmin - (j + e) < p.a.window || j + e < p.a.sinks))
                            vreg[i][e] = *reinterpret_cast<const VPiece*>(v + e * p.c.v_token * W);
                }
            }
        }
    };
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int id = i * 256 + tid, tok = id / PIECES, pc = id - tok * PIECES;
            if (id < kTokens * PIECES) {
                if constexpr (HELD8) {
                    u32x4 a, d;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[2 * k] = T::template from_e4m3<false>(kreg[i][k]);
                        a[2 * k + 1] = T::template from_e4m3<true>(kreg[i][k]);
                        d[2 * k] = T::template from_e4m3<false>(kreg[i][k + 2]);
                        d[2 * k + 1] = T::template from_e4m3<true>(kreg[i][k + 2]);
                    }
                    *reinterpret_cast<u32x4*>(ldsk + tok * KP + pc * 32) = a;
                    *reinterpret_cast<u32x4*>(ldsk + tok * KP + pc * 32 + 16) = d;
                } else {
                    *reinterpret_cast<u32x4*>(ldsk + tok * KP + pc * 16) = kreg[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int id = i * 256 + tid, quad = id / CH8, c8 = id - quad * CH8;
            if (id < kTokens / 4 * CH8) {
                // Of each 16 tokens: pair 0 holds quads 0 and 2, pair 1 quads 1 and 3.
                const int pair = (quad >> 2) * 2 + (quad & 1), half = (quad >> 1) & 1;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (HELD8)
                            w[e] = (t & 2) ? V::template from_e4m3<true>(vreg[i][e][t >> 2]) : V::template from_e4m3<false>(vreg[i][e][t >> 2]);
                        else
                            w[e] = vreg[i][e][t >> 1];
                    }
                    const uint32_t sel = (t & 1) ? 0x07060302u : 0x05040100u;
                    const int d = c8 * 8 + t, col = pair ^ (((d >> 1) ^ (d >> 3)) & 7);
                    *reinterpret_cast<u32x2*>(ldsv + d * 128 + col * 16 + half * 8) =
                        u32x2{__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel)};
                }
            }
        }
    };

    if (st0 < st1) {
        look_up((st0 * 4) & ~(kInfo - 1));
        __syncthreads();
        fetch(st0);
    }
    for (int st = st0; st < st1; ++st) {
        put();
        const int gi = (st * 4) & (kInfo - 1);
        // This step's groups, before the next ones may replace them.
        int base[4];
        float f2[4], vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base[i] = __builtin_amdgcn_readfirstlane(gbase[gi + i]);
            f2[i] = gks[gi + i];
            vs[i] = gvs[gi + i];
        }
        __syncthreads();
        if (st + 1 < st1) {
            if (((st + 1) * 4 & (kInfo - 1)) == 0) {
                look_up((st + 1) * 4);
                __syncthreads();
            }
            fetch(st + 1);
        }
        bool full = true, any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            full = full && base[i] <= wmin - 15 && (p.a.window == 0 || wmax - base[i] < p.a.window || base[i] + 15 < p.a.sinks);
            any = any || (base[i] <= wmax && (p.a.window == 0 || wmin - base[i] - 15 < p.a.window || base[i] < p.a.sinks));
        }
        if (any) {
            f32x16 sc[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[u][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const x8 kk = *reinterpret_cast<const x8*>(ldsk + (u * 32 + r) * KP + k * 32 + hh * 16);
                    sc[u] = T::mfma32(kk, q[k], sc[u]);
                }
            }
            if (full) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[u][i] *= f2[u * 2 + (i >> 3)];
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = base[u * 2 + (i >> 3)] + ((i >> 2) & 1) * 8 + hh * 4 + (i & 3);
                        sc[u][i] = sees(p, pos, j) ? sc[u][i] * f2[u * 2 + (i >> 3)] : neg_inf();
                    }
            }
            float top = neg_inf();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[u][i]);
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
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int z = 0; z < 2; ++z) {   // 16 tokens
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        e[i] = exp2_(sc[u][z * 8 + i] - ref);
                        l += e[i];
                        if constexpr (HELD8) e[i] *= vs[u * 2 + z];
                    }
                    u32x4 w, w2;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[i] = pack2<V>(e[2 * i], e[2 * i + 1]);
                        if constexpr (kTwo) w2[i] = pack2<V>(e[2 * i] - lo16<V>(w[i]), e[2 * i + 1] - hi16<V>(w[i]));
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int d = t * 32 + r, pair = (u * 2 + z) * 2 + hh;
                        const auto vv = *reinterpret_cast<const typename V::x8*>(
                            ldsv + d * 128 + ((pair ^ (((d >> 1) ^ (d >> 3)) & 7)) * 16));
                        o[t] = V::mfma32(vv, __builtin_bit_cast(typename V::x8, w), o[t]);
                        if constexpr (kTwo) o[t] = V::mfma32(vv, __builtin_bit_cast(typename V::x8, w2), o[t]);
                    }
                }
        }
        __syncthreads();
    }

    l = sum32(l);
    if (!there) return;
    if (p.splits > 1) {
        float* part = p.tile_parts + ((uint64_t)(x * p.c.kv_heads + h) * p.splits + split) * tile_part_floats(D);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<f32x4*>(part + row * D + t * 32 + i * 2 + hh * 4) =
                    m == neg_inf() ? f32x4{0, 0, 0, 0} : f32x4{o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]};
        if (hh == 0) {
            part[kTileRows * D + row] = m;
            part[kTileRows * D + kTileRows + row] = l;
        }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    one* out = (one*)p.a.out + (s.row0 + t0 + qi) * p.a.o_token + head * p.a.o_head;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int ch = t * 32 + i * 2 + hh * 4;
            if (ch < p.c.dim) {
                u32x2 w = {0, 0};
                if (l != 0.0f) w = u32x2{pack2<T>(o[t][i] * inv, o[t][i + 1] * inv), pack2<T>(o[t][i + 2] * inv, o[t][i + 3] * inv)};
                *reinterpret_cast<u32x2*>(out + ch) = w;
            }
        }
    if (p.a.lse && hh == 0)
        p.a.lse[(s.row0 + t0 + qi) * p.a.l_token + head * p.a.l_head] = l == 0.0f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
}

// Joins a row tile's parts, in their order: a wave a row at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_tile_join(AttendArgs p) {
    typedef typename T::one one;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = blockIdx.x % p.c.kv_heads, x = blockIdx.x / p.c.kv_heads;
    int before = 0;
    for (int b0 = 0; b0 < p.g.batch; b0 += 64) {
        const int bb = b0 + lane;
        before += __builtin_popcountll(__ballot(bb < p.g.batch && p.g.starts[bb] / p.tile_tokens + bb <= x));
    }
    if (before == 0) return;
    const int b = before - 1;
    const Seq s = read_seq(p.g, b);
    if ((int64_t)s.n * p.group <= p.few) return;
    const int t0 = (x - s.row0 / p.tile_tokens - b) * p.tile_tokens;
    if (t0 < 0 || t0 >= s.n) return;
    const int tn = s.n - t0 < p.tile_tokens ? s.n - t0 : p.tile_tokens;
    const float* base = p.tile_parts + (uint64_t)(x * p.c.kv_heads + h) * p.splits * tile_part_floats(D);
    for (int row = blockIdx.y * 4 + wave; row < tn * p.group; row += gridDim.y * 4) {
        float top = neg_inf();
        for (int i = 0; i < p.splits; ++i) top = fmaxf(top, base[i * tile_part_floats(D) + kTileRows * D + row]);
        float sum = 0.0f, y[D / 64 + 1];
#pragma unroll
        for (int k = 0; k < D / 64 + 1; ++k) y[k] = 0.0f;
        for (int i = 0; i < p.splits; ++i) {
            const float* part = base + i * tile_part_floats(D);
            const float mp = part[kTileRows * D + row];
            if (mp == neg_inf()) continue;
            const float a = exp2_(mp - top);
            sum += part[kTileRows * D + kTileRows + row] * a;
#pragma unroll
            for (int k = 0; k < D / 64 + 1; ++k)
                if (k * 64 + lane < D) y[k] += part[row * D + k * 64 + lane] * a;
        }
        const int qi = (int)fdiv((uint32_t)row, p.div_group), head = h * p.group + row - qi * p.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        one* out = (one*)p.a.out + (s.row0 + t0 + qi) * p.a.o_token + head * p.a.o_head;
#pragma unroll
        for (int k = 0; k < D / 64 + 1; ++k)
            if (k * 64 + lane < p.c.dim && k * 64 + lane < D) out[k * 64 + lane] = (one)(sum == 0.0f ? 0.0f : y[k] * inv);
        if (p.a.lse && lane == 0)
            p.a.lse[(s.row0 + t0 + qi) * p.a.l_token + head * p.a.l_head] = sum == 0.0f ? neg_inf() : (top + __builtin_log2f(sum)) * kLn2;
    }
}

template <typename T, bool HELD8, int D>
static hipError_t go(const AttendArgs& p, bool join, hipStream_t st) {
    if (join)
        k_tile_join<T, D><<<dim3((unsigned)(p.tiles * p.c.kv_heads), 4), 256, 0, st>>>(p);
    else
        k_tile<T, HELD8, D><<<(unsigned)(p.tiles * p.c.kv_heads * p.splits), 256, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, bool HELD8>
static hipError_t go_d(const AttendArgs& p, int dk, bool join, hipStream_t st) {
    switch (dk) {
    case 64: return go<T, HELD8, 64>(p, join, st);
    case 96: return go<T, HELD8, 96>(p, join, st);
    case 128: return go<T, HELD8, 128>(p, join, st);
    case 192: return go<T, HELD8, 192>(p, join, st);
    default: return go<T, HELD8, 256>(p, join, st);
    }
}

hipError_t launch_tile(const AttendArgs& p, int dk, bool join, hipStream_t st) {
    const bool held8 = p.c.type == TPL_KV_E4M3;
    if (p.a.type == TPL_KV_BF16) return held8 ? go_d<Bf16, true>(p, dk, join, st) : go_d<Bf16, false>(p, dk, join, st);
    return held8 ? go_d<Fp16, true>(p, dk, join, st) : go_d<Fp16, false>(p, dk, join, st);
}

}  // namespace kv
}  // namespace tpl
