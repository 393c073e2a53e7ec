// kv_read.hip -- tokens of a paged cache as packed rows of 16-bit keys and
// values.
//
// x = held * scale in 32 bits, rounded once (nothing is rounded where the
// scale is a power of two, as append's are, and x a normal number of the
// rows' type); a 16-bit cache's values go through bit for bit.
//
// Bound: HBM bytes, each read and written once.  A workgroup takes up to
// `rows` consecutive tokens of one sequence; where they lie is looked up once
// for all their heads and kept in LDS, then every thread moves 8 channels at a
// time, kAtOnce loads under way before the first is used.
//
// Measured on an MI355X (a large copy: 4.9 to 5.2 TB/s): 102000 tokens of 8
// heads of 128 out of an e4m3 cache, 641 MB, 122 us (5.3 TB/s); 45000 of 5 heads
// of 80 out of an fp16 one, 145 MB, 33 us (4.4 TB/s); 41 tokens 4.1 us, one launch.
#include <climits>

#include "common.hpp"
#include "kv.hpp"

namespace tpl {
namespace kv {

constexpr int kMaxRows = 32;   // tokens of a workgroup
constexpr int kAtOnce = 4;     // pieces of 8 channels that a thread has under way

struct ReadArgs {
    tpl_kv_cache c;
    tpl_kv_batch g;
    tpl_kv_rows a;
    FastDiv div_page, div_block, div_row, div_head;   // of pieces: a row's, a head's
    int32_t cap;    // tokens that a table row can hold
    int32_t rows;   // of a tile
    int32_t first;  // what blockIdx.y = 0 reads: 0 keys, 1 values
};

template <typename T, bool HELD8>
__global__ void __launch_bounds__(256) k_read(ReadArgs p) {
    constexpr int W = HELD8 ? 1 : 2;
    typedef typename std::conditional<HELD8, u32x2, u32x4>::type Piece;
    // Of each row its page's and its place's offset in the pool (bytes) and in
    // the scales, or -1.
    __shared__ int64_t at[kMaxRows], scale_at[kMaxRows];

    const bool values = blockIdx.y + p.first;
    const TileSeq mine = seq_of_tile(p.g, p.rows, blockIdx.x);
    if (mine.b < 0) return;
    const Seq s = mine.s;
    const int t0 = ((int)blockIdx.x - s.row0 / p.rows - mine.b) * p.rows;   // the tile's first row in its sequence
    if (t0 < 0 || t0 >= s.n) return;
    const int n = s.n - t0 < p.rows ? s.n - t0 : p.rows;
    const int tid = threadIdx.x;
    if (tid < n) {
        const int pos = s.length - s.n + t0 + tid;
        const int pg = (int)fdiv((uint32_t)pos, p.div_page), slot = pos - pg * p.c.page;
        const int where = pos < p.cap ? p.g.table[mine.b * p.g.table_row + pg] : -1;
        const bool there = (uint32_t)where < (uint32_t)p.c.pages;
        at[tid] = there ? (values ? where * p.c.v_page + slot * p.c.v_token : where * p.c.k_page + slot * p.c.k_token) * W : -1;
        if constexpr (HELD8) {
            const int blk = (int)fdiv((uint32_t)slot, p.div_block);
            scale_at[tid] = !there ? 0 : values ? where * p.c.vs_page + blk * p.c.vs_block : where * p.c.ks_page + blk * p.c.ks_block;
        }
    }
    __syncthreads();

    const uint8_t* from = (const uint8_t*)(values ? p.c.v : p.c.k);
    const float* scales = values ? p.c.v_scale : p.c.k_scale;
    const int64_t head_in = (values ? p.c.v_head : p.c.k_head) * W, head_sc = values ? p.c.vs_head : p.c.ks_head;
    const int64_t head_out = values ? p.a.v_head : p.a.k_head, row_out = values ? p.a.v_token : p.a.k_token;
    uint16_t* to = (uint16_t*)(values ? p.a.v : p.a.k) + (s.row0 + t0) * row_out;
    const int pieces = n * (int)p.div_row.d;
    for (int i0 = tid; i0 < pieces; i0 += 256 * kAtOnce) {
        Piece x[kAtOnce];
        float sc[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * 256;
            x[u] = Piece{};
            sc[u] = 0.0f;
            if (i >= pieces) continue;
            const int row = (int)fdiv((uint32_t)i, p.div_row), c = i - row * (int)p.div_row.d;
            const int head = (int)fdiv((uint32_t)c, p.div_head), ch = (c - head * (int)p.div_head.d) * 8;
            const int64_t o = at[row];
            if (o < 0) continue;
            x[u] = *reinterpret_cast<const Piece*>(from + o + head * head_in + ch * W);
            if constexpr (HELD8) sc[u] = scales[scale_at[row] + head * head_sc];
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * 256;
            if (i >= pieces) continue;
            const int row = (int)fdiv((uint32_t)i, p.div_row), c = i - row * (int)p.div_row.d;
            const int head = (int)fdiv((uint32_t)c, p.div_head), ch = (c - head * (int)p.div_head.d) * 8;
            u32x4 y;
            if constexpr (HELD8) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(x[u][k], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(x[u][k], true);
                    const float a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1];
                    y[2 * k] = pack2<T>(a0 * sc[u], a1 * sc[u]);
                    y[2 * k + 1] = pack2<T>(b0 * sc[u], b1 * sc[u]);
                }
            } else {
                y = x[u];
            }
            *reinterpret_cast<u32x4*>(to + row * row_out + head * head_out + ch) = y;
        }
    }
}

// Whether rows or heads of a result lie over one another.
static bool overlap(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head) {
    token = tokens > 1 ? token < 0 ? -token : token : INT64_MAX;
    head = heads > 1 ? head < 0 ? -head : head : INT64_MAX;
    if (token < dim || head < dim) return true;
    if (token == INT64_MAX || head == INT64_MAX) return false;
    return token >= head ? (token - dim) / head < heads - 1 : (head - dim) / token < tokens - 1;
}

static int read_impl(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_rows* a, hipStream_t st) {
    if (!c || !g || !a) return fail_status(TPL_E_ARG, "cache, batch and rows must not be NULL");
    if (const char* why = check_cache(c)) return fail_status(TPL_E_ARG, why);
    if (const char* why = check_batch(*c, g)) return fail_status(TPL_E_ARG, why);
    if (a->type != TPL_KV_BF16 && a->type != TPL_KV_FP16) return fail_status(TPL_E_DTYPE, "rows must be bf16 or fp16");
    if (c->type != TPL_KV_E4M3 && c->type != a->type) return fail_status(TPL_E_DTYPE, "a 16-bit cache is read as the type it holds");
    if (g->batch == 0 || g->tokens == 0) return TPL_OK;
    if (!a->k && !a->v) return fail_status(TPL_E_ARG, "k and v must not both be NULL");
    if (a->k == a->v) return fail_status(TPL_E_ARG, "k and v must not be one tensor");
    if ((a->k && !aligned16(a->k, a->k_token, a->k_head, 2)) || (a->v && !aligned16(a->v, a->v_token, a->v_head, 2)))
        return fail_status(TPL_E_LAYOUT, "k and v must start, and their rows and heads lie, on 16 bytes");
    if ((a->k && overlap(g->tokens, c->kv_heads, c->dim, a->k_token, a->k_head)) ||
        (a->v && overlap(g->tokens, c->kv_heads, c->dim, a->v_token, a->v_head)))
        return fail_status(TPL_E_LAYOUT, "rows and heads of k and v must not lie over one another");
    ReadArgs p;
    p.c = *c;
    p.g = *g;
    p.a = *a;
    const int head = c->dim / 8, row = head * c->kv_heads;
    p.div_page = make_fastdiv((uint32_t)c->page);
    p.div_block = make_fastdiv((uint32_t)(c->type == TPL_KV_E4M3 ? c->block : c->page));
    p.div_row = make_fastdiv((uint32_t)row);
    p.div_head = make_fastdiv((uint32_t)head);
    p.cap = g->width * c->page;
    p.first = a->k ? 0 : 1;
    // As many tokens as give every thread its kAtOnce pieces once.  8 heads of
    // 128: 8 tokens a workgroup; 102000 tokens 122 us, with 4 150, with 32 127;
    // 500 tokens 4.4 us, with 1 4.9, with 32 7.0.
    p.rows = 256 * kAtOnce / row;
    p.rows = p.rows < 1 ? 1 : p.rows > kMaxRows ? kMaxRows : p.rows;
    const dim3 grid((unsigned)(g->tokens / p.rows + g->batch), a->k && a->v ? 2 : 1);
    if (c->type != TPL_KV_E4M3)
        k_read<Bf16, false><<<grid, 256, 0, st>>>(p);
    else if (a->type == TPL_KV_BF16)
        k_read<Bf16, true><<<grid, 256, 0, st>>>(p);
    else
        k_read<Fp16, true><<<grid, 256, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail_status(TPL_E_HIP, std::string("HIP launch failed: ") + hipGetErrorString(e));
    return TPL_OK;
}

}  // namespace kv
}  // namespace tpl

extern "C" int tpl_kv_read(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_rows* rows, hipStream_t stream) {
    try {
        return tpl::kv::read_impl(cache, batch, rows, stream);
    } catch (...) {
        return TPL_E_ARG;
    }
}
