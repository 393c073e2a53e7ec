// linear_chunk.hip -- linear attention of many new tokens a sequence: chunks of
// 64 tokens through the matrix units.
//
// With l = exp(decay), i and j a chunk's tokens from 0 on and S the state before it
//
//   out_i = l^(i+1) q_i S + sum_{j <= i} l^(i-j) (q_i k_j) v_j
//   S'    = l^n S + sum_j l^(n-1-j) k_j v_j^T
//
// A workgroup takes one head of one sequence (or of a segment of it) and walks
// over its chunks with the state in registers, 32 value channels a wave.  Queries,
// keys and values stand in LDS as they lie in memory, and every product of
// 32x32x16 reads them from there or has its operand in registers already:
//
//   P^T = K Q^T      its result (column i, rows j) is, with decay and mask, the
//                    second operand of
//   O^T = V^T P^T    where V^T's operands come by transposing reads of LDS, 4
//                    tokens of a channel each, in the order of P^T's rows;
//   O^T += S^T Q^T   the state's registers (column: value channel, rows: key
//                    channels) are S^T's operand as they lie, if Q's operand
//                    names key channels in the same order;
//   S += K^T (w V)   K^T by transposing reads, w V from the registers of V^T.
//
// So neither the state nor the outputs pass through LDS.  P is computed once
// for all waves, a block of 32x32 each, and handed over in LDS as operands.
//
// Roundings: P, S and w V are fp32 numbers and go into the products as the sum
// of two 16-bit ones (16 or 22 bits): outputs are rounded to 8 or 11.  States
// stay, so where the pool's are made bf16's w V is the sum of three (24).  In fp16 each is brought near 2^14 by a
// power of two before, so that nothing leaves that type's range.
//
// A value that is no finite number would reach earlier rows of its chunk as its
// product with a weight of zero: such a chunk is taken token by token.
//
// Where whole sequences are too few for the CUs a sequence goes in segments:
// what each adds (k_chunk, kState), the states before each (k_scan), then the
// outputs (kOutput).
//
// Bound: HBM bytes for long sequences of many; here the vector and matrix units,
// whose work does not overlap.  Measured on an MI355X: a prompt of 8192 tokens,
// 32 heads of 128 by 128 in bf16, 42 us for the segments' states, 12 for the
// scan, 78 for the outputs (a copy of the bytes: 52).  Each left out by itself,
// the last loses 18 us with the products into the state, 11 with those of states
// and queries, 11 with P, 10 with the writing and 9 with the reading.  Vector and
// matrix instructions take 38 % and 21 % of its time, 1100 of the former and 78 of
// the latter a wave and chunk.  Steps: no scratch memory (its reads wait behind
// the next chunk's) and operands by 16 tokens 133 -> 82 us; two parts of the
// weighted values 82 -> 77.  Not faster: 8 waves of 16 channels (95 us), pieces
// exchanged in LDS so that little conflicts (96), rows in LDS further apart (80 to
// 84), the order of products and vector work set by hand (82 to 88).
#include "linear.hpp"

namespace tpl {
namespace linear {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// 4 numbers of a column: of 16 lanes each 4 name a row's 16 columns, and lane l
// of them gets column l of the 4 rows.
__device__ __forceinline__ u32x2 read_column(const uint16_t* p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
    return __builtin_bit_cast(u32x2, v);
}

__device__ __forceinline__ float max_swap32(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float max_wave(float x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
    return max_swap32(x);
}

// The power of two that brings a largest magnitude to 2^14 .. 2^15 (one under
// 2^-27 not that far: sums that are multiplied by it beside have to stay in
// range), and its reciprocal.
struct Scale {
    float up, down;
};
__device__ __forceinline__ float inverse2(float x) {   // of a power of two
    return __builtin_bit_cast(float, (254u << 23) - __builtin_bit_cast(uint32_t, x));
}
__device__ __forceinline__ Scale scale_of(float most) {
    int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23 & 255);   // 127 + its exponent
    e = e < 100 ? 100 : e > 254 ? 254 : e;
    const float down = __builtin_bit_cast(float, (uint32_t)(e - 14) << 23);
    return Scale{inverse2(down), down};
}

// Two numbers as 16-bit ones, and what those leave of them: the part that is
// taken first may be rounded any way, so that fp16 takes the one instruction
// that rounds both towards zero (two parts keep 21 bits at least).
template <typename T>
__device__ __forceinline__ uint32_t part2(float& a, float& b) {
    if constexpr (std::is_same<T, kv::Fp16>::value) {
        const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
        a = __builtin_fmaf((float)h[0], -1.0f, a);
        b = __builtin_fmaf((float)h[1], -1.0f, b);
        return __builtin_bit_cast(uint32_t, h);
    } else {
        const uint32_t x = pack2<T>(a, b);
        a -= lo16<T>(x), b -= hi16<T>(x);
        return x;
    }
}
// Two numbers as the sum of two 16-bit ones each.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = part2<T>(a, b);
    if constexpr (std::is_same<T, kv::Fp16>::value)
        lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    else
        lo = pack2<T>(a, b);
}

// The sequence that segment x belongs to (see seq_of_tile of kv.hpp).
struct At {
    int b;
    Rows s;
};
__device__ __forceinline__ At seq_of_segment(const LinearArgs& p, int x) {
    const int lane = threadIdx.x & 63;
    At t = {-1, {0, 0}};
    for (int b0 = 0; b0 < p.g.batch; b0 += 64) {
        const int bb = b0 + lane < p.g.batch ? b0 + lane : p.g.batch - 1;
        const Rows s = rows_of(p.g, bb);
        const uint64_t m = __ballot(b0 + lane < p.g.batch && s.n > 0 && s.row0 / p.segment + bb <= x);
        if (m) {
            const int from = 63 - __builtin_clzll(m);
            t.b = b0 + from;
            t.s.row0 = __builtin_amdgcn_readlane(s.row0, from);
            t.s.n = __builtin_amdgcn_readlane(s.n, from);
        }
    }
    return t;
}

template <typename T, int NK, int WAVES, int MODE>
__global__ void __launch_bounds__(WAVES * 64, NK <= 4 ? 2 : 1) k_chunk(LinearArgs p) {
    typedef typename T::one one;
    typedef typename T::x8 x8;
    constexpr bool kScaled = std::is_same<T, kv::Fp16>::value;
    constexpr int THREADS = WAVES * 64, DK = NK * 32, VC = WAVES * 32;
    // A chunk is read while the one before it is at work, where that leaves the
    // state its registers.
    constexpr bool kAhead = NK <= 4;
    // Rows padded by 16 bytes: 32 rows' pieces at one place reach all banks.
    constexpr int QP = DK + 8, VP = VC + 8;
    constexpr int QUERIES = MODE == kState ? 0 : kChunk * QP, BLOCKS = MODE == kState ? 0 : 3;
    __shared__ __attribute__((aligned(16))) uint16_t lds[QUERIES + kChunk * QP + kChunk * VP];
    __shared__ u32x4 pbuf[BLOCKS + 1][2][2][64];   // block, part, product, lane
    __shared__ float pdown[BLOCKS + 1][64];
    __shared__ __attribute__((aligned(16))) float weight[kChunk];   // l^(n-1-j)
    __shared__ __attribute__((aligned(16))) _Float16 weight16[kChunk];
    __shared__ int bad;
    uint16_t *qs = lds, *ks = lds + QUERIES, *vs = ks + kChunk * QP;

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sl = blockIdx.x % p.slices, rest = blockIdx.x / p.slices, h = rest % p.p.heads, unit = rest / p.p.heads;
    int b, row0, n;
    if constexpr (MODE == kWhole) {
        const Rows s = rows_of(p.g, unit);
        b = unit, row0 = s.row0, n = s.n;
        if (n == 0 || n <= p.few) return;
    } else {
        const At t = seq_of_segment(p, unit);
        if (t.b < 0 || t.s.n <= p.few) return;
        const int t0 = (unit - t.s.row0 / p.segment - t.b) * p.segment;
        if (t0 < 0 || t0 >= t.s.n) return;
        b = t.b, row0 = t.s.row0 + t0, n = t.s.n - t0 < p.segment ? t.s.n - t0 : p.segment;
    }
    const float g2 = decay_of(p, h);
    const int kh = h / p.share;
    const int dv0 = sl * VC;   // the workgroup's value channels; this wave's: 32 from dv0 + wave * 32 on
    const int dvw = dv0 + wave * 32;
    const bool active = dvw < p.p.value_dim;
    const one* gq = (const one*)p.a.q + (int64_t)row0 * p.a.q_token + kh * p.a.q_head;
    const one* gk = (const one*)p.a.k + (int64_t)row0 * p.a.k_token + kh * p.a.k_head;
    const one* gv = (const one*)p.a.v + (int64_t)row0 * p.a.v_token + h * p.a.v_head + dv0;
    one* go = (one*)p.a.out + (int64_t)row0 * p.a.o_token + h * p.a.o_head;

    // The state: register i of block kb is key channel kb * 32 + 8 (i / 4) + 4 hh + i % 4 of value channel dvw + r.
    f32x16 S[NK];
    const float* from = nullptr;
    int64_t s_key = p.p.value_dim;
    float* mine = p.parts + ((int64_t)unit * p.p.heads + h) * p.p.key_dim * p.p.value_dim;
    if constexpr (MODE == kWhole) from = source_of(p, b, h), s_key = p.p.s_key;
    if constexpr (MODE == kOutput) from = mine;
#pragma unroll
    for (int kb = 0; kb < NK; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int ch = kb * 32 + (i >> 2) * 8 + hh * 4 + (i & 3);
            S[kb][i] = 0.0f;
            if (MODE != kState && from && ch < p.p.key_dim && dvw + r < p.p.value_dim) S[kb][i] = from[ch * s_key + dvw + r];
        }

    // What a thread brings: pieces of 8 channels, always the same ones, of every
    // KR-th (VR-th) token; threads that do not fill a row more bring none.
    constexpr int KPR = DK / 8, KR = THREADS / KPR, KN = (kChunk + KR - 1) / KR;
    constexpr int VPR = VC / 8, VR = THREADS / VPR, VN = (kChunk + VR - 1) / VR;
    const int ktok = tid / KPR, kch = (tid - ktok * KPR) * 8, vtok = tid / VPR, vch = (tid - vtok * VPR) * 8;
    const bool kput = ktok < KR, vput = vtok < VR;   // it has a place in LDS
    const bool kmine = kput && kch < p.p.key_dim, vmine = vput && dv0 + vch < p.p.value_dim;
    // The host keeps 64 rows within 2^31 bytes.
    const uint32_t qoff = ((uint32_t)ktok * (uint32_t)p.a.q_token + kch) * 2, koff = ((uint32_t)ktok * (uint32_t)p.a.k_token + kch) * 2;
    const uint32_t voff = ((uint32_t)vtok * (uint32_t)p.a.v_token + vch) * 2;
    u32x4 qreg[MODE == kState ? 1 : KN], kreg[KN], vreg[VN];
    auto fetch = [&](int t, int count) {   // zeros beyond the chunk's tokens and the head's channels
        const char *bq = (const char*)(gq + t * p.a.q_token), *bk = (const char*)(gk + t * p.a.k_token), *bv = (const char*)(gv + t * p.a.v_token);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const bool there = kmine && ktok + i * KR < count;
            kreg[i] = u32x4{0, 0, 0, 0};
            if (there) kreg[i] = *reinterpret_cast<const u32x4*>(bk + i * KR * p.a.k_token * 2 + koff);
            if constexpr (MODE != kState) {
                qreg[i] = u32x4{0, 0, 0, 0};
                if (there) qreg[i] = *reinterpret_cast<const u32x4*>(bq + i * KR * p.a.q_token * 2 + qoff);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            vreg[i] = u32x4{0, 0, 0, 0};
            if (vmine && vtok + i * VR < count) vreg[i] = *reinterpret_cast<const u32x4*>(bv + i * VR * p.a.v_token * 2 + voff);
        }
    };
    auto put = [&](int count) {
        bool some = false;
#pragma unroll
        for (int i = 0; i < KN; ++i)
            if (kput && (KR * KN == kChunk || ktok + i * KR < kChunk)) {
                *reinterpret_cast<u32x4*>(ks + (ktok + i * KR) * QP + kch) = kreg[i];
                if constexpr (MODE != kState) *reinterpret_cast<u32x4*>(qs + (ktok + i * KR) * QP + kch) = qreg[i];
            }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            if constexpr (MODE != kState) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w = vreg[i][e];
                    some |= kv::clear_bad<T>(w);
                }
            }
            if (vput && (VR * VN == kChunk || vtok + i * VR < kChunk)) *reinterpret_cast<u32x4*>(vs + (vtok + i * VR) * VP + vch) = vreg[i];
        }
        if (some && count > 1) bad = 1;
        if (tid < kChunk) {
            const float w = tid < count ? exp2_(g2 * (float)(count - 1 - tid)) : 0.0f;
            weight[tid] = w;
            if constexpr (kScaled) weight16[tid] = (_Float16)w;
        }
    };

    if (tid == 0) bad = 0;
    __syncthreads();
    int t = 0, count = n < kChunk ? n : kChunk, single = 0;   // tokens before `single` are taken one by one
    if (kAhead) fetch(0, count);
    while (t < n) {
        if (!kAhead) fetch(t, count);
        put(count);
        __syncthreads();
        if (MODE != kState && bad && count > 1) {
            __syncthreads();
            if (tid == 0) bad = 0;
            single = t + count;
            count = 1;
            if (kAhead) fetch(t, 1);
            __syncthreads();
            continue;
        }
        const int here = t, now = count;
        t += count;
        count = t < single ? 1 : n - t < kChunk ? n - t : kChunk;
        if (kAhead && t < n) fetch(t, count);

        f32x16 o[2];
        float into[2];   // what the state's part of the outputs is multiplied with
        if constexpr (MODE != kState) {
            // P^T's blocks: rows of j = 0 and columns of i = 0, of j = 0 and i = 1, of j = 1 and i = 1.
#pragma unroll 1
            for (int blk = wave; blk < 3; blk += WAVES) {
                const int jb = blk >> 1, ib = (blk + 1) >> 1;
                f32x16 x;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll
                for (int s = 0; s < NK * 2; ++s) {
                    const u32x4 kw = *reinterpret_cast<const u32x4*>(ks + (jb * 32 + r) * QP + s * 16 + hh * 8);
                    const u32x4 qw = *reinterpret_cast<const u32x4*>(qs + (ib * 32 + r) * QP + s * 16 + hh * 8);
                    x = T::mfma32(__builtin_bit_cast(x8, kw), __builtin_bit_cast(x8, qw), x);
                }
                const int d0 = (ib - jb) * 32 + r - hh * 4;   // i - j of register 0
                float most = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = d0 - (i >> 2) * 8 - (i & 3);
                    x[i] = d < 0 ? 0.0f : x[i] * exp2_(g2 * (float)d);
                    if constexpr (kScaled) most = fmaxf(most, __builtin_fabsf(x[i]));
                }
                if constexpr (kScaled) {
                    const Scale sc = scale_of(max_swap32(most));
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= sc.up;
                    pdown[blk][lane] = sc.down;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    u32x4 hi, lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a, c;
                        split2<T>(x[s * 8 + i * 2], x[s * 8 + i * 2 + 1], a, c);
                        hi[i] = a, lo[i] = c;
                    }
                    pbuf[blk][0][s][lane] = hi;
                    pbuf[blk][1][s][lane] = lo;
                }
            }
            // What the state before the chunk gives (waves beyond the head's
            // value channels bring rows and blocks of P only).
#pragma unroll
            for (int ib = 0; ib < 2; ++ib)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[ib][i] = 0.0f;
            if (active) {
            Scale sc = {1.0f, 1.0f};
            if constexpr (kScaled) {
                float most = 0.0f;
#pragma unroll
                for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) most = fmaxf(most, __builtin_fabsf(S[kb][i]));
                most = max_wave(most);
                if (!(most < __builtin_inff())) {   // an infinity says nothing of the other channels
                    most = 0.0f;
#pragma unroll
                    for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float x = __builtin_fabsf(S[kb][i]);
                            most = fmaxf(most, x < __builtin_inff() ? x : 0.0f);
                        }
                    most = max_wave(most);
                }
                sc = scale_of(most);
            }
#pragma unroll
            for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    u32x4 hi, lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a, c;
                        split2<T>(S[kb][s * 8 + i * 2] * sc.up, S[kb][s * 8 + i * 2 + 1] * sc.up, a, c);
                        hi[i] = a, lo[i] = c;
                    }
#pragma unroll
                    for (int ib = 0; ib < 2; ++ib) {
                        const uint16_t* q = qs + (ib * 32 + r) * QP + kb * 32 + s * 16 + hh * 4;
                        const u32x2 q0 = *reinterpret_cast<const u32x2*>(q), q1 = *reinterpret_cast<const u32x2*>(q + 8);
                        const x8 qw = __builtin_bit_cast(x8, (u32x4{q0[0], q0[1], q1[0], q1[1]}));
                        o[ib] = T::mfma32(__builtin_bit_cast(x8, hi), qw, o[ib]);
                        o[ib] = T::mfma32(__builtin_bit_cast(x8, lo), qw, o[ib]);
                    }
                }
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) {
                into[ib] = exp2_(g2 * (float)(ib * 32 + r + 1)) * sc.down;
                if constexpr (!kScaled)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[ib][i] *= into[ib];
            }
            }
            __syncthreads();   // P is there
        }

        // Values, transposed: of 16 tokens those at 4 hh .. + 3 and 8 + 4 hh .. + 3.
        const int trow = hh * 4 + ((lane & 15) >> 2), tcol = (lane >> 4 & 1) * 16 + (lane & 3) * 4;
        auto column16 = [&](const uint16_t* base, int pitch, int z) {
            const u32x2 a = read_column(base + (z * 16 + trow) * pitch + tcol), c = read_column(base + (z * 16 + 8 + trow) * pitch + tcol);
            return u32x4{a[0], a[1], c[0], c[1]};
        };
        if constexpr (MODE != kState) {
            if (active) {
            // A block of P^T with its 32 tokens' values, on top of what is there
            // (brought to the block's power of two, from the one before).
            u32x4 vt[2];
#pragma unroll
            for (int blk = 0; blk < 3; ++blk) {
                const int jb = blk >> 1, ib = (blk + 1) >> 1;
                if (blk != 1) vt[0] = column16(vs + wave * 32, VP, jb * 2), vt[1] = column16(vs + wave * 32, VP, jb * 2 + 1);
                if constexpr (kScaled) {
                    const float up = blk < 2 ? into[ib] * inverse2(pdown[blk][lane]) : pdown[1][lane] * inverse2(pdown[2][lane]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[ib][i] *= up;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        o[ib] = T::mfma32(__builtin_bit_cast(x8, vt[s]), __builtin_bit_cast(x8, pbuf[blk][part][s][lane]), o[ib]);
            }
            const float last[2] = {kScaled ? pdown[0][lane] * p.a.scale : p.a.scale, kScaled ? pdown[2][lane] * p.a.scale : p.a.scale};
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) {
                const int tok = ib * 32 + r;
                if (tok >= now) continue;
                one* to = go + (here + tok) * p.a.o_token + dvw + hh * 4;
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    if (dvw + a * 8 < p.p.value_dim)
                        *reinterpret_cast<u32x2*>(to + a * 8) =
                            u32x2{pack2<T>(o[ib][a * 4] * last[ib], o[ib][a * 4 + 1] * last[ib]),
                                  pack2<T>(o[ib][a * 4 + 2] * last[ib], o[ib][a * 4 + 3] * last[ib])};
            }
            }
        }

        if (active && (MODE != kOutput || t < n)) {
            const float keep = exp2_(g2 * (float)now);
            // The weighted values of 16 tokens.
            auto weighted = [&](int z, float (&w)[8]) {
                const u32x4 v = column16(vs + wave * 32, VP, z);
                const f32x4 a = *reinterpret_cast<const f32x4*>(weight + z * 16 + hh * 4);
                const f32x4 c = *reinterpret_cast<const f32x4*>(weight + z * 16 + 8 + hh * 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i * 2] = lo16<T>(v[i]) * a[i * 2], w[i * 2 + 1] = hi16<T>(v[i]) * a[i * 2 + 1];
                    w[i * 2 + 4] = lo16<T>(v[i + 2]) * c[i * 2], w[i * 2 + 5] = hi16<T>(v[i + 2]) * c[i * 2 + 1];
                }
            };
            Scale sc = {1.0f, 1.0f};
            if constexpr (kScaled) {
                // A value channel's own, as a column of the state has one lane
                // pair; how large the largest is in 16 bits tells its power of
                // two (which leaves a binade for that).
                kv::f16x2 most = {0, 0};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const u32x4 v = column16(vs + wave * 32, VP, z);
                    const u32x2 a = *reinterpret_cast<const u32x2*>(weight16 + z * 16 + hh * 4), c = *reinterpret_cast<const u32x2*>(weight16 + z * 16 + 8 + hh * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const kv::f16x2 x = __builtin_bit_cast(kv::f16x2, v[i] & 0x7fff7fffu) * __builtin_bit_cast(kv::f16x2, (uint32_t)(i < 2 ? a[i] : c[i - 2]));
                        most = __builtin_elementwise_max(most, x);
                    }
                }
                sc = scale_of(max_swap32(fmaxf((float)most[0], (float)most[1])));
            }
            const float first = keep * sc.up;
#pragma unroll
            for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[kb][i] *= first;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                float w[8];
                weighted(z, w);
                // In bf16 three parts where the state is kept: two would leave it
                // 2^-18 off.
                constexpr int PARTS = kScaled || MODE == kOutput ? 2 : 3;
                u32x4 part[PARTS];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a = w[i * 2] * sc.up, c = w[i * 2 + 1] * sc.up;
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) part[k][i] = part2<T>(a, c);
                }
#pragma unroll
                for (int kb = 0; kb < NK; ++kb) {
                    const x8 kt = __builtin_bit_cast(x8, column16(ks + kb * 32, QP, z));
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) S[kb] = T::mfma32(kt, __builtin_bit_cast(x8, part[k]), S[kb]);
                }
            }
            if constexpr (kScaled) {
#pragma unroll
                for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[kb][i] *= sc.down;
            }
        }
        __syncthreads();   // the chunk's LDS is free
    }

    // The lane again, so that no address is held throughout.
    int again = threadIdx.x;
    asm volatile("" : "+v"(again));
    const int dv = dvw + (again & 31), key0 = (again >> 5 & 1) * 4;
    float* to = nullptr;
    if constexpr (MODE == kWhole) to = state_at(p, p.g.slots[b], h);
    if constexpr (MODE == kState) to = mine;
    if (to && dv < p.p.value_dim)
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int ch = kb * 32 + (i >> 2) * 8 + key0 + (i & 3);
                if (ch < p.p.key_dim) to[ch * s_key + dv] = S[kb][i];
            }
}

// From what each segment adds to what stands before it, and the sequence's
// last state.
__global__ void __launch_bounds__(256) k_scan(LinearArgs p) {
    const int h = blockIdx.x % p.p.heads, b = blockIdx.x / p.p.heads;
    const Rows s = rows_of(p.g, b);
    if (s.n == 0 || s.n <= p.few) return;
    const int quads = p.p.value_dim / 4, i = blockIdx.y * 256 + threadIdx.x;
    const int key = i / quads, c = (i - key * quads) * 4;
    if (key >= p.p.key_dim) return;
    const float g2 = decay_of(p, h);
    const int64_t state = (int64_t)p.p.key_dim * p.p.value_dim, next = state * p.p.heads;
    float* at = p.parts + (int64_t)(s.row0 / p.segment + b) * next + h * state + key * p.p.value_dim + c;
    const float* from = source_of(p, b, h);
    f32x4 x = {0, 0, 0, 0};
    if (from) x = *reinterpret_cast<const f32x4*>(from + key * p.p.s_key + c);
    const int count = (s.n + p.segment - 1) / p.segment;
    const float keep = exp2_(g2 * (float)p.segment);
    constexpr int AHEAD = 4;   // segments' parts under way
    f32x4 y[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) y[k] = k < count ? *reinterpret_cast<const f32x4*>(at + k * next) : f32x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < count; k0 += AHEAD)
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int seg = k0 + k;
            if (seg >= count) break;
            const f32x4 added = y[k];
            if (seg + AHEAD < count) y[k] = *reinterpret_cast<const f32x4*>(at + (seg + AHEAD) * next);
            *reinterpret_cast<f32x4*>(at + seg * next) = x;
            const float f = seg + 1 < count ? keep : exp2_(g2 * (float)(s.n - seg * p.segment));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __builtin_fmaf(x[e], f, added[e]);
        }
    float* to = state_at(p, p.g.slots[b], h);
    if (to) *reinterpret_cast<f32x4*>(to + key * p.p.s_key + c) = x;
}

// Waves of a workgroup: 2, each with 32 of up to 64 value channels, or 4 (for
// up to 128, and where 2 would have to hold too much of a chunk on its way).
int chunk_waves(int key_dim, int value_dim) { return value_dim <= 64 && key_dim <= 96 ? 2 : 4; }
int chunk_slices(int key_dim, int value_dim) {
    const int w = chunk_waves(key_dim, value_dim) * 32;
    return (value_dim + w - 1) / w;
}

template <typename T, int NK, int WAVES>
static hipError_t go_mode(const LinearArgs& p, int mode, unsigned grid, hipStream_t st) {
    if (mode == kWhole)
        k_chunk<T, NK, WAVES, kWhole><<<grid, WAVES * 64, 0, st>>>(p);
    else if (mode == kState)
        k_chunk<T, NK, WAVES, kState><<<grid, WAVES * 64, 0, st>>>(p);
    else
        k_chunk<T, NK, WAVES, kOutput><<<grid, WAVES * 64, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, int NK>
static hipError_t go_waves(const LinearArgs& p, int mode, unsigned grid, hipStream_t st) {
    if constexpr (NK <= 3) {
        if (chunk_waves(p.p.key_dim, p.p.value_dim) == 2) return go_mode<T, NK, 2>(p, mode, grid, st);
    }
    return go_mode<T, NK, 4>(p, mode, grid, st);
}

template <typename T>
static hipError_t go_keys(const LinearArgs& p, int mode, unsigned grid, hipStream_t st) {
    const int d = p.p.key_dim;
    if (d <= 32) return go_waves<T, 1>(p, mode, grid, st);
    if (d <= 64) return go_waves<T, 2>(p, mode, grid, st);
    if (d <= 96) return go_waves<T, 3>(p, mode, grid, st);
    if (d <= 128) return go_waves<T, 4>(p, mode, grid, st);
    if (d <= 192) return go_waves<T, 6>(p, mode, grid, st);
    return go_waves<T, 8>(p, mode, grid, st);
}

hipError_t launch_chunk(const LinearArgs& p, int mode, int64_t units, hipStream_t st) {
    const unsigned grid = (unsigned)(units * p.p.heads * p.slices);
    return p.a.type == TPL_KV_BF16 ? go_keys<kv::Bf16>(p, mode, grid, st) : go_keys<kv::Fp16>(p, mode, grid, st);
}

hipError_t launch_scan(const LinearArgs& p, hipStream_t st) {
    const int64_t n = (int64_t)p.p.key_dim * (p.p.value_dim / 4);
    k_scan<<<dim3((unsigned)(p.g.batch * p.p.heads), (unsigned)((n + 255) / 256)), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace linear
}  // namespace tpl
