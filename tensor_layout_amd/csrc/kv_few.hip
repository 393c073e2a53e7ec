// kv_few.hip -- attention of a few rows a sequence (decoding, drafts) to a
// paged cache.
//
// out = sum_j w_j v_j / sum_j w_j, w_j = 2^(x_j - m), x = scale log2(e) q k,
// with one running reference m a row.
//
// Bound: HBM bytes of the cache, read once.  So the token axis is split: the
// batch's work is counted in steps of 128 tokens of one (sequence, head, row
// tile), and every workgroup takes an equal share of consecutive steps,
// whatever the sequences' lengths are.  Of a step each of 4 waves takes 32
// tokens straight from HBM into registers: nothing is staged in LDS, because
// no other wave needs the same values.
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
};

template <bool HELD8, int DC>
__device__ __forceinline__ void load_tile(const AttendArgs& p, const int32_t* pages, const Span& span, int t, int h,
                                          Tile<HELD8, DC>& x) {
    constexpr int W = HELD8 ? 1 : 2;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    x.base = 0x7fffff00;
    x.ks = x.vs = 0.0f;
#pragma unroll
    for (int i = 0; i < x.KL; ++i) x.k[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < (int)(sizeof(x.v[e]) / 4); ++i) x.v[e].w[i] = 0;
    if (t >= span.n) return;
    const int base = span.base(t);
    const int pg = (int)fdiv((uint32_t)base, p.div_page), slot = base - pg * p.c.page;
    const int where = pages[pg];
    if (where < 0 || where >= p.c.pages) return;
    x.base = base;
    const uint8_t* k = (const uint8_t*)p.c.k + (where * p.c.k_page + slot * p.c.k_token + h * p.c.k_head) * W;
    const uint8_t* v = (const uint8_t*)p.c.v + (where * p.c.v_page + slot * p.c.v_token + h * p.c.v_head) * W;
    if constexpr (HELD8) {
        const int blk = (int)fdiv((uint32_t)slot, p.div_block);
        x.ks = p.c.k_scale[where * p.c.ks_page + h * p.c.ks_head + blk * p.c.ks_block];
        x.vs = p.c.v_scale[where * p.c.vs_page + h * p.c.vs_head + blk * p.c.vs_block];
    }
    const uint8_t* kl = k + r * p.c.k_token * W;
#pragma unroll
    for (int i = 0; i < x.KL; ++i) {
        const int ch = HELD8 ? i * 64 + g * 16 : i * 32 + g * 8;
        if (ch < p.c.dim) x.k[i] = *reinterpret_cast<const u32x4*>(kl + ch * W);
    }
    if (r * DC < p.c.dim) {
        const uint8_t* vl = v + r * DC * W;
#pragma unroll
        for (int e = 0; e < 4; ++e) x.v[e] = load_chunk<DC * W>(vl + (g * 4 + e) * p.c.v_token * W);
    }
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

template <typename T, bool HELD8, int DC, int MR>
__global__ void __launch_bounds__(256) k_few(AttendArgs p) {
    typedef typename T::one one;
    typedef typename T::x8 x8;
    // Weights and values are multiplied in the cache's type.  An e4m3 value's
    // scale is folded into its weight, which needs bf16's range; where the
    // output keeps 11 bits the weight goes in as the sum of two bf16 numbers.
    typedef typename std::conditional<HELD8, Bf16, T>::type V;
    constexpr bool kTwo = HELD8 && std::is_same<T, Fp16>::value;
    constexpr int KS = DC / 2;           // key products of a row
    constexpr int ROWS = MR * 16;
    constexpr int HALVES = DC > 8 ? 2 : 1, DCH = DC / HALVES, PITCH = 16 * DCH + 4;
    __shared__ float obuf[4][16][PITCH];
    __shared__ float mbuf[4][ROWS], lbuf[4][ROWS];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b;
    uint64_t seq_step, chunk;
    const uint64_t total = locate<ROWS>(p, false, 0, &b, &seq_step, &chunk);
    uint64_t c = (uint64_t)blockIdx.x * chunk;
    uint64_t cend = c + chunk < total ? c + chunk : total;
    if (c >= cend || b < 0) return;

    while (c < cend) {
        FewSeq f = few_seq<ROWS>(p, b);
        const uint64_t off = c - seq_step, all = f.all(p);
        if (off >= all) {
            seq_step += all;
            if (++b >= p.g.batch) return;
            continue;
        }
        const int unit = (int)(off / (uint32_t)f.steps);
        const int s0 = (int)(off - (uint64_t)unit * (uint32_t)f.steps);
        const int s1 = (uint64_t)(f.steps - s0) < cend - c ? f.steps : s0 + (int)(cend - c);
        const int rt = unit / p.c.kv_heads, h = unit - rt * p.c.kv_heads;
        const int rows = f.s.n * p.group - rt * ROWS;   // of this tile, may exceed ROWS
        const int first = f.s.length - f.s.n;
        const int32_t* pages = p.g.table + b * p.g.table_row;
        const int pmin = first + (int)fdiv((uint32_t)(rt * ROWS), p.div_group);
        const int lastrow = rt * ROWS + (rows < ROWS ? rows : ROWS) - 1;
        const int pmax = first + (int)fdiv((uint32_t)lastrow, p.div_group);

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
            pos[mr] = there ? first + i : -1;
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

        for (int s = s0; s < s1; ++s) {
            const int t0 = s * kStepGroups + wave * 2;
            if (t0 >= f.span.n) break;
            Tile<HELD8, DC> x[2];
            load_tile<HELD8, DC>(p, pages, f.span, t0, h, x[0]);
            load_tile<HELD8, DC>(p, pages, f.span, t0 + 1, h, x[1]);

            f32x4 sc[MR][2];
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
                const float f2 = HELD8 ? p.factor * x[u].ks : p.factor;
                const bool full = base <= pmin - 15 &&
                                  (p.a.window == 0 || pmax - base < p.a.window || base + 15 < p.a.sinks);
                if (full) {
#pragma unroll
                    for (int mr = 0; mr < MR; ++mr)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[mr][u][i] *= f2;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = base + g * 4 + i;
#pragma unroll
                        for (int mr = 0; mr < MR; ++mr)
                            sc[mr][u][i] = sees(p, pos[mr], j) ? sc[mr][u][i] * f2 : neg_inf();
                        // A token that no row sees weighs nothing, whatever its place holds.
                        if (!(j <= pmax && (p.a.window == 0 || pmin - j < p.a.window || j < p.a.sinks)))
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
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[mr][u][i]);
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
                        e[i] = exp2_(sc[mr][u][i] - ref);
                        l[mr] += e[i];
                        if constexpr (HELD8) e[i] *= x[u].vs;
                    }
                    w[mr][u * 2] = pack2<V>(e[0], e[1]);
                    w[mr][u * 2 + 1] = pack2<V>(e[2], e[3]);
                    if constexpr (kTwo) {
                        w2[mr][u * 2] = pack2<V>(e[0] - lo16<V>(w[mr][u * 2]), e[1] - hi16<V>(w[mr][u * 2]));
                        w2[mr][u * 2 + 1] = pack2<V>(e[2] - lo16<V>(w[mr][u * 2 + 1]), e[3] - hi16<V>(w[mr][u * 2 + 1]));
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
        }

        // The four waves' sums join under the largest reference.
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
            l[mr] = sum16(sum32(l[mr]));
            if (g == 0) {
                mbuf[wave][mr * 16 + r] = m[mr];
                lbuf[wave][mr * 16 + r] = l[mr];
            }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == f.steps;
        float* part = p.parts + ((uint64_t)blockIdx.x * 2 + (s0 ? 0 : 1)) * few_part_floats<DC, MR>();
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
            const int row = mr * 16 + r;
            float top = neg_inf();
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, mbuf[i][row]);
            const float a = m[mr] == neg_inf() ? 0.0f : exp2_(m[mr] - top);
            const int orow = mr * 16 + (tid >> 4), oc = tid & 15;
            float otop = neg_inf(), osum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) otop = fmaxf(otop, mbuf[i][orow]);
#pragma unroll
            for (int i = 0; i < 4; ++i) osum += mbuf[i][orow] == neg_inf() ? 0.0f : lbuf[i][orow] * exp2_(mbuf[i][orow] - otop);
            const bool there = orow < rows;
            const int oi = (int)fdiv((uint32_t)(rt * ROWS + orow), p.div_group);
            const int head = h * p.group + rt * ROWS + orow - oi * p.group;
            const float inv = osum == 0.0f ? 0.0f : 1.0f / osum;
#pragma unroll
            for (int half = 0; half < HALVES; ++half) {
                if (mr + half) __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < DCH; ++t) obuf[wave][r][(g * 4 + i) * DCH + t] = m[mr] == neg_inf() ? 0.0f : o[mr][half * DCH + t][i] * a;
                __syncthreads();
                if (there && oc * DC < p.c.dim) {
                    float y[DCH];
#pragma unroll
                    for (int t = 0; t < DCH; ++t) {
                        y[t] = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[t] += obuf[i][tid >> 4][oc * DCH + t];
                    }
                    if (whole) {
                        one* out = (one*)p.a.out + (f.s.row0 + oi) * p.a.o_token + head * p.a.o_head + oc * DC + half * DCH;
#pragma unroll
                        for (int t = 0; t < DCH; t += 2)
                            *reinterpret_cast<uint32_t*>(out + t) = pack2<T>(osum == 0.0f ? 0.0f : y[t] * inv, osum == 0.0f ? 0.0f : y[t + 1] * inv);
                    } else {
                        float* out = part + orow * (16 * DC) + oc * DC + half * DCH;
#pragma unroll
                        for (int t = 0; t < DCH; ++t) out[t] = y[t];
                    }
                }
                if (there && oc == 0 && half == 0) {
                    if (whole) {
                        if (p.a.lse)
                            p.a.lse[(f.s.row0 + oi) * p.a.l_token + head * p.a.l_head] =
                                osum == 0.0f ? neg_inf() : (otop + __builtin_log2f(osum)) * kLn2;
                    } else {
                        part[ROWS * 16 * DC + orow] = otop;
                        part[ROWS * 16 * DC + ROWS + orow] = osum;
                    }
                }
            }
        }
        __syncthreads();
        c += s1 - s0;
    }
}

// Joins the parts of row tiles that more than one workgroup took: a wave a
// row, 64 lanes over its channels, the parts in their order.
template <typename T, int DC, int MR>
__global__ void __launch_bounds__(256) k_few_join(AttendArgs p) {
    typedef typename T::one one;
    constexpr int ROWS = MR * 16, PER = DC / 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bb = blockIdx.x / p.c.kv_heads, h = blockIdx.x - bb * p.c.kv_heads;
    int b;
    uint64_t seq_step, chunk;
    locate<ROWS>(p, true, bb, &b, &seq_step, &chunk);
    const FewSeq f = few_seq<ROWS>(p, bb);
    const int row = blockIdx.y * 4 + wave;
    for (int rt = 0; rt < f.tiles; ++rt) {
        if (rt * ROWS + row >= f.s.n * p.group) break;
        const uint64_t c0 = seq_step + ((uint64_t)rt * p.c.kv_heads + h) * (uint32_t)f.steps;
        const uint64_t w0 = c0 / chunk, w1 = (c0 + f.steps - 1) / chunk;
        if (w0 == w1) continue;
        const int np = (int)(w1 - w0) + 1;
        const float* base = p.parts + w0 * 2 * few_part_floats<DC, MR>();
        float top = neg_inf();
        for (int i = lane; i < np; i += 64) {
            const float* part = base + ((uint64_t)i * 2 + (i ? 0 : 1)) * few_part_floats<DC, MR>();
            top = fmaxf(top, part[ROWS * 16 * DC + row]);
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        float sum = 0.0f, y[PER];
#pragma unroll
        for (int t = 0; t < PER; ++t) y[t] = 0.0f;
#pragma unroll 4
        for (int i = 0; i < np; ++i) {
            const float* part = base + ((uint64_t)i * 2 + (i ? 0 : 1)) * few_part_floats<DC, MR>();
            const float mp = part[ROWS * 16 * DC + row];
            const float a = mp == neg_inf() ? 0.0f : exp2_(mp - top);
            sum += part[ROWS * 16 * DC + ROWS + row] * a;
            if (lane * PER < p.c.dim)
#pragma unroll
                for (int t = 0; t < PER; ++t) {
                    const float o = part[row * 16 * DC + lane * PER + t];
                    y[t] += mp == neg_inf() ? 0.0f : o * a;
                }
        }
        const int i = (int)fdiv((uint32_t)(rt * ROWS + row), p.div_group);
        const int head = h * p.group + rt * ROWS + row - i * p.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        one* out = (one*)p.a.out + (f.s.row0 + i) * p.a.o_token + head * p.a.o_head + lane * PER;
        if (lane * PER < p.c.dim)
#pragma unroll
            for (int t = 0; t < PER; ++t) out[t] = (one)(sum == 0.0f ? 0.0f : y[t] * inv);
        if (p.a.lse && lane == 0)
            p.a.lse[(f.s.row0 + i) * p.a.l_token + head * p.a.l_head] =
                sum == 0.0f ? neg_inf() : (top + __builtin_log2f(sum)) * kLn2;
    }
}

template <typename T, bool HELD8, int DC, int MR>
static hipError_t go(const AttendArgs& p, int join, hipStream_t st) {
    k_few<T, HELD8, DC, MR><<<p.workers, 256, 0, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !join) return e;
    k_few_join<T, DC, MR><<<dim3((unsigned)(p.g.batch * p.c.kv_heads), MR * 4), 256, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, bool HELD8, int DC>
static hipError_t go_mr(const AttendArgs& p, int mr, int join, hipStream_t st) {
    if (mr == 1) return go<T, HELD8, DC, 1>(p, join, st);
    if constexpr (DC <= 8) {   // 64 rows of longer heads would not fit a lane's registers
        if (mr == 4) return go<T, HELD8, DC, 4>(p, join, st);
    }
    return go<T, HELD8, DC, 2>(p, join, st);
}

template <typename T, bool HELD8>
static hipError_t go_dc(const AttendArgs& p, int dc, int mr, int join, hipStream_t st) {
    switch (dc) {
    case 4: return go_mr<T, HELD8, 4>(p, mr, join, st);
    case 8: return go_mr<T, HELD8, 8>(p, mr, join, st);
    case 12: return go_mr<T, HELD8, 12>(p, mr, join, st);
    default: return go_mr<T, HELD8, 16>(p, mr, join, st);
    }
}

hipError_t launch_few(const AttendArgs& p, int dc, int mr, int join, hipStream_t st) {
    const bool held8 = p.c.type == TPL_KV_E4M3;
    if (p.a.type == TPL_KV_BF16) return held8 ? go_dc<Bf16, true>(p, dc, mr, join, st) : go_dc<Bf16, false>(p, dc, mr, join, st);
    return held8 ? go_dc<Fp16, true>(p, dc, mr, join, st) : go_dc<Fp16, false>(p, dc, mr, join, st);
}

}  // namespace kv
}  // namespace tpl
