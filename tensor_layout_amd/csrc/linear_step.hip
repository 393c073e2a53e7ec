// linear_step.hip -- linear attention of few new tokens a sequence (decoding,
// drafts): the recurrence itself.
//
// Bound: HBM bytes of the states, each read and written once.  A workgroup
// takes one head of one sequence, or a slice of its value channels, and holds
// that part of the state in registers: a thread 4 value channels of every
// ROWS-th key channel, so that a wave's reads lie next to each other.  All of
// a thread's reads are under way before the first is used.  Keys, queries and
// values of TOK tokens (one, or 4 where a sequence may have more) stand in LDS as
// fp32; a token costs two fused products a state's number, and the sums over key
// channels are joined over lanes and waves.
//
// Measured on an MI355X (a large copy: 4.9 to 5.2 TB/s): one token of 128
// sequences, 32 heads of 128 by 128, 541 MB, 108 us (5.0 TB/s); one of a
// single sequence, 16 heads, 4.1 us.  Steps there: LDS for one
// token instead of 16 (49 KB a workgroup let 3 stand on a CU) and registers
// instead of the compiler's wide vectors 163 -> 108 us.  With 128 value channels
// a workgroup instead of 64: 109; with 32: 110.
#include "linear.hpp"

namespace tpl {
namespace linear {

template <typename T, int COLS, int NP, int TOK>
__global__ void __launch_bounds__(256) k_step(LinearArgs p) {
    typedef typename T::one one;
    constexpr int ROWS = 256 / COLS, SLICE = COLS * 4, DK = NP * ROWS;   // key channels of a pass; value channels; key channels
    __shared__ float ks[TOK][DK], qs[TOK][DK];
    __shared__ float part[TOK][4][SLICE];

    const int slices = (p.p.value_dim + SLICE - 1) / SLICE;
    const int sl = blockIdx.x % slices, rest = blockIdx.x / slices, h = rest % p.p.heads, b = rest / p.p.heads;
    const Rows s = rows_of(p.g, b);
    if (s.n == 0 || s.n > p.few) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = tid % COLS, row = tid / COLS, dv = sl * SLICE + col * 4;
    const bool there = dv < p.p.value_dim;

    f32x4 S[NP];
    const float* from = source_of(p, b, h);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int r = row + i * ROWS;
        S[i] = f32x4{0, 0, 0, 0};
        if (from && there && r < p.p.key_dim) S[i] = *reinterpret_cast<const f32x4*>(from + r * p.p.s_key + dv);
    }
    const float keep = exp2_(decay_of(p, h));
    const int kh = h / p.share;

    for (int t0 = 0; t0 < s.n; t0 += TOK) {
        const int n = s.n - t0 < TOK ? s.n - t0 : TOK;
        const int64_t row0 = s.row0 + t0;
        if (t0) __syncthreads();
        // Zeros beyond the head's channels, where states are zero too.
        for (int i = tid; i < n * (DK / 2); i += 256) {
            const int t = i / (DK / 2), ch = (i - t * (DK / 2)) * 2;
            uint32_t kw = 0, qw = 0;
            if (ch < p.p.key_dim) {
                kw = *reinterpret_cast<const uint32_t*>((const one*)p.a.k + (row0 + t) * p.a.k_token + kh * p.a.k_head + ch);
                qw = *reinterpret_cast<const uint32_t*>((const one*)p.a.q + (row0 + t) * p.a.q_token + kh * p.a.q_head + ch);
            }
            ks[t][ch] = lo16<T>(kw), ks[t][ch + 1] = hi16<T>(kw);
            qs[t][ch] = lo16<T>(qw), qs[t][ch + 1] = hi16<T>(qw);
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            u32x2 vw = {0, 0};
            if (there) vw = *reinterpret_cast<const u32x2*>((const one*)p.a.v + (row0 + t) * p.a.v_token + h * p.a.v_head + dv);
            const float v[4] = {lo16<T>(vw[0]), hi16<T>(vw[0]), lo16<T>(vw[1]), hi16<T>(vw[1])};
            float o[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float k = ks[t][row + i * ROWS], q = qs[t][row + i * ROWS];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[i][e] = __builtin_fmaf(S[i][e], keep, k * v[e]);
                    o[e] = __builtin_fmaf(q, S[i][e], o[e]);
                }
            }
#pragma unroll
            for (int d = COLS; d < 64; d <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], d);
            if (lane < COLS) *reinterpret_cast<f32x4*>(&part[t][wave][col * 4]) = f32x4{o[0], o[1], o[2], o[3]};
        }
        __syncthreads();
        for (int i = tid; i < n * (SLICE / 2); i += 256) {
            const int t = i / (SLICE / 2), c = (i - t * (SLICE / 2)) * 2;
            if (sl * SLICE + c >= p.p.value_dim) continue;
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                y[e] = ((part[t][0][c + e] + part[t][1][c + e]) + (part[t][2][c + e] + part[t][3][c + e])) * p.a.scale;
            *reinterpret_cast<uint32_t*>((one*)p.a.out + (row0 + t) * p.a.o_token + h * p.a.o_head + sl * SLICE + c) = pack2<T>(y[0], y[1]);
        }
    }

    float* to = state_at(p, p.g.slots[b], h);
    if (!to || !there) return;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int r = row + i * ROWS;
        if (r < p.p.key_dim) *reinterpret_cast<f32x4*>(to + r * p.p.s_key + dv) = S[i];
    }
}

template <typename T, int COLS, int TOK>
static hipError_t go(const LinearArgs& p, hipStream_t st) {
    constexpr int ROWS = 256 / COLS;
    const int64_t grid = (int64_t)p.g.batch * p.p.heads * ((p.p.value_dim + COLS * 4 - 1) / (COLS * 4));
    switch ((p.p.key_dim + 63) / 64) {   // key channels up to the next multiple of 64
    case 1: k_step<T, COLS, 64 / ROWS, TOK><<<(unsigned)grid, 256, 0, st>>>(p); break;
    case 2: k_step<T, COLS, 128 / ROWS, TOK><<<(unsigned)grid, 256, 0, st>>>(p); break;
    case 3: k_step<T, COLS, 192 / ROWS, TOK><<<(unsigned)grid, 256, 0, st>>>(p); break;
    default: k_step<T, COLS, 256 / ROWS, TOK><<<(unsigned)grid, 256, 0, st>>>(p); break;
    }
    return hipGetLastError();
}

template <typename T, int COLS>
static hipError_t go_tokens(const LinearArgs& p, hipStream_t st) {
    return p.g.tokens <= p.g.batch ? go<T, COLS, 1>(p, st) : go<T, COLS, 4>(p, st);
}

hipError_t launch_step(const LinearArgs& p, bool narrow, hipStream_t st) {
    if (p.a.type == TPL_KV_BF16) return narrow ? go_tokens<kv::Bf16, 8>(p, st) : go_tokens<kv::Bf16, 16>(p, st);
    return narrow ? go_tokens<kv::Fp16, 8>(p, st) : go_tokens<kv::Fp16, 16>(p, st);
}

}  // namespace linear
}  // namespace tpl
