// kv_attend.hip -- attention to a paged key/value cache: checks of arguments,
// choice of the kernels, C entry points.
#include <climits>

#include "kv_attend.hpp"

namespace tpl {
namespace kv {

constexpr int kCUs = 256;
constexpr int kCounters = TPL_KV_COUNTERS / 4;   // at least the split kernel's workgroups

bool aligned16(const void* p, int64_t s0, int64_t s1, int bytes) {
    return ((uintptr_t)p & 15) == 0 && (s0 * bytes) % 16 == 0 && (s1 * bytes) % 16 == 0;
}

const char* check_cache(const tpl_kv_cache* c) {
    if (c->type != TPL_KV_BF16 && c->type != TPL_KV_FP16 && c->type != TPL_KV_E4M3)
        return "a cache holds bf16, fp16 or e4m3";
    if (!c->k || !c->v) return "cache pools must not be NULL";
    if (c->pages < 1 || c->pages > INT_MAX) return "a cache must have at least one page";
    if (c->dim < 16 || c->dim > 256 || c->dim % 16) return "dim must be a multiple of 16, at most 256";
    if (c->kv_heads < 1 || c->kv_heads > kCounters) return "kv_heads must be 1 .. 1024";
    if (c->page < 16 || c->page % 16 || c->page > (1 << 20)) return "page must be a multiple of 16 tokens, at most 2^20";
    const int w = c->type == TPL_KV_E4M3 ? 1 : 2;
    for (int64_t x : {c->k_token, c->v_token, c->k_page, c->v_page, c->ks_page, c->vs_page, c->ks_block, c->vs_block})
        if (x > ((int64_t)1 << 40) || x < -((int64_t)1 << 40)) return "strides must be under 2^40";
    if (c->type == TPL_KV_E4M3) {
        if (!c->k_scale || !c->v_scale) return "an e4m3 cache needs its scales";
        if (c->block < 16 || c->block % 16 || c->page % c->block)
            return "block must be a multiple of 16 tokens and divide the page";
    }
    if (!aligned16(c->k, c->k_token, c->k_head, w) || !aligned16(c->v, c->v_token, c->v_head, w) ||
        (c->k_page * w) % 16 || (c->v_page * w) % 16)
        return "cache pools must start, and their pages, tokens and heads lie, on 16 bytes";
    // Offsets inside a page, and its size, are 32-bit numbers in the kernels.
    const int64_t in_page[] = {c->k_token * w * c->page, c->v_token * w * c->page, c->k_token, c->v_token};
    for (int64_t x : in_page)
        if (x < 0 || x > INT_MAX) return "a page's tokens must lie within 2^31 bytes";
    const int64_t page_of[] = {c->k_page * w, c->v_page * w};
    for (int64_t x : page_of)
        if (x < 0 || x > UINT32_MAX) return "pages must lie at most 2^32 bytes apart";
    if (c->type == TPL_KV_E4M3) {
        const int64_t s[] = {c->ks_page, c->vs_page, c->ks_block * c->page, c->vs_block * c->page};
        for (int64_t x : s)
            if (x < 0 || x > INT_MAX) return "a page's scales must lie within 2^31 elements";
    }
    return nullptr;
}

const char* check_batch(const tpl_kv_cache& c, const tpl_kv_batch* g) {
    if (g->batch < 0 || g->tokens < 0 || g->width < 0) return "batch, tokens and width must be >= 0";
    if (g->batch > (1 << 20)) return "batch must be at most 2^20";
    if (g->tokens > (1 << 28)) return "tokens must be at most 2^28";
    if ((int64_t)g->width * c.page > kMaxLength) return "a table row must not name more than 2^30 tokens";
    if (g->batch && (!g->starts || !g->lengths || (g->width && !g->table)))
        return "table, starts and lengths must not be NULL";
    return nullptr;
}

struct Choice {
    bool few, tile;
    int dc, mr, dk;
    int64_t few_bytes, tile_bytes;   // of parts
    // The counters come first in every workspace, also in one for a call that
    // counts nothing: the next call on it may, and has to find them zero.
    int64_t bytes() const { return few_bytes + tile_bytes > 0 ? kCounters * 4 + few_bytes + tile_bytes : 0; }
};

static const char* choose(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_query* a, AttendArgs& p, Choice& q,
                          int* status) {
    *status = TPL_E_ARG;
    if (!c || !g || !a) return "cache, batch and arguments must not be NULL";
    if (const char* why = check_cache(c)) return why;
    if (const char* why = check_batch(*c, g)) return why;
    if (a->type != TPL_KV_BF16 && a->type != TPL_KV_FP16) {
        *status = TPL_E_DTYPE;
        return "queries must be bf16 or fp16";
    }
    if (c->type != TPL_KV_E4M3 && c->type != a->type) {
        *status = TPL_E_DTYPE;
        return "a 16-bit cache holds the type of its queries";
    }
    if (a->heads < 1 || a->heads % c->kv_heads) return "heads must be a multiple of the cache's";
    if (!(a->scale > 0.0f) || !(a->scale < __builtin_inff())) return "scale must be a finite number over zero";
    if (a->window < 0 || a->sinks < 0) return "window and sinks must be >= 0";
    if (a->window > kMaxLength || a->sinks > kMaxLength) return "window and sinks must be at most 2^30";
    p.c = *c;
    p.g = *g;
    p.a = *a;
    if (c->type != TPL_KV_E4M3) p.c.block = c->page;
    if (a->window == 0) p.a.sinks = 0;
    p.counters = nullptr;
    p.parts = p.tile_parts = nullptr;
    p.group = a->heads / c->kv_heads;
    p.cap = g->width * c->page;
    p.factor = a->scale * kLog2e;
    p.div_page = make_fastdiv((uint32_t)c->page);
    p.div_block = make_fastdiv((uint32_t)p.c.block);
    p.div_group = make_fastdiv((uint32_t)p.group);
    q.few = q.tile = false;
    q.few_bytes = q.tile_bytes = 0;
    if (g->batch == 0 || g->tokens == 0) return nullptr;
    const int64_t rows = (int64_t)g->tokens * p.group;   // no sequence has more
    if (rows > INT_MAX) return "tokens * heads / kv_heads must be under 2^31";

    // Which kernel takes a sequence goes by its rows, which only the device
    // knows; the host leaves a kernel out where no sequence can need it, and
    // where there are no more rows than sequences (decoding) or only one
    // sequence lets one kernel take whatever there is.
    const int limit = 64;
    if (p.group > 128 || rows <= limit || (g->batch > 1 && g->tokens <= g->batch)) {
        q.few = true;
        p.few = INT_MAX;
    } else if (g->batch == 1) {
        q.tile = true;
        p.few = 0;
    } else {
        q.few = q.tile = true;
        p.few = limit;
    }
    if (q.few) {
        // 16 lanes hold dc channels each: 12 only where those are whole lanes (144 and 192 channels).
        q.dc = c->dim <= 64 ? 4 : c->dim <= 128 ? 8 : c->dim <= 192 && c->dim % 12 == 0 ? 12 : 16;
        // Rows of a tile: those of an average sequence, or of a decoding one
        // where the average is a prompt's.
        int64_t mean = (rows + g->batch - 1) / g->batch;
        if (mean > limit) mean = p.group;
        q.mr = mean <= 16 ? 1 : mean <= 32 || q.dc > 8 ? 2 : 4;
        // No more shares than steps there can be.
        const int64_t tiles = (rows + q.mr * 16 - 1) / (q.mr * 16) + g->batch;
        const int64_t most = tiles * (((int64_t)p.cap + 31) / 32 + 1);
        // Two heads a workgroup where they lie next to each other within 256
        // bytes and a share is long: it then reads whole 256 bytes of a token.
        // 64 sequences of up to 8192 tokens (64 steps a share at most): 155
        // against 174 us; 24 of them (24 steps): 65 against 72.  At 16 steps,
        // where the parts that are left weigh more, it goes both ways: 8 of up
        // to 16384 58 against 62, 2 of up to 65536 63 against 60, 32 of up to
        // 4096 46 against 49 with a row each and 48 against 46 with four.
        // Under a window of 1024, 64 of them (8 steps): 28 against 22 us.
        int64_t seen = p.cap;
        if (a->window && (int64_t)a->window + a->sinks < seen) seen = (int64_t)a->window + a->sinks;
        const int64_t blocks = kCUs * few_blocks(c->type == TPL_KV_E4M3, q.dc, q.mr);
        const int w = c->type == TPL_KV_E4M3 ? 1 : 2;
        p.heads_log = c->kv_heads % 2 == 0 && c->k_head * w < 256 && c->k_head < c->k_token && c->v_head < c->v_token &&
                      g->batch * (seen / 128) * c->kv_heads >= 24 * blocks ? 1 : 0;
        int64_t shares = blocks / (c->kv_heads >> p.heads_log);
        if (most > INT_MAX) return "tokens and table are too large together";
        if (shares > most) shares = most;
        p.shares = shares < 1 ? 1 : (int)shares;
        q.few_bytes = (int64_t)p.shares * c->kv_heads * 2 * few_part_floats(q.dc, q.mr) * 4;
    }
    if (q.tile) {
        q.dk = c->dim <= 64 ? 64 : c->dim <= 96 ? 96 : c->dim <= 128 ? 128 : c->dim <= 192 ? 192 : 256;
        // Row tiles of 256 (8 waves that share a step's keys and values) where
        // they still give every CU two, else of 128.  One prompt of 8192
        // tokens, 32 heads of 128: 572 against 598 us; a chunk of 1024 tokens
        // (128 tiles of 256): 169 against 139 us.  Under a window larger tiles
        // see more that most of their rows do not (window 1024: 178 against
        // 158 us), and longer heads do not fit 8 waves' registers.
        const bool large = q.dk <= 128 && a->window == 0 && rows / 256 * c->kv_heads >= 2 * kCUs;
        p.tile_rows = large ? 256 : 128;
        p.tile_tokens = p.tile_rows / p.group;
        const int64_t tiles = (int64_t)g->tokens / p.tile_tokens + g->batch;
        const int64_t units = tiles * c->kv_heads;
        int64_t most = p.cap;
        if (a->window && (int64_t)a->window + a->sinks + p.tile_tokens < most) most = (int64_t)a->window + a->sinks + p.tile_tokens;
        most = (most + 511) / 512;
        int64_t splits = 2 * kCUs / units;
        if (splits > most) splits = most;
        if (splits > 32) splits = 32;
        if (splits < 1) splits = 1;
        p.tiles = (int)tiles;
        p.splits = (int)splits;
        if (units * splits > INT_MAX) return "too many row tiles";
        if (splits > 1) q.tile_bytes = units * splits * tile_part_floats(q.dk, p.tile_rows) * 4;
    }
    return nullptr;
}

static int attend_impl(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_query* a, void* ws, int64_t ws_bytes,
                       hipStream_t st) {
    AttendArgs p;
    Choice q;
    int status;
    if (const char* why = choose(c, g, a, p, q, &status)) return fail_status(status, why);
    if (!q.few && !q.tile) return TPL_OK;
    if (!a->q || !a->out) return fail_status(TPL_E_ARG, "q and out must not be NULL");
    if (!aligned16(a->q, a->q_token, a->q_head, 2) || !aligned16(a->out, a->o_token, a->o_head, 2))
        return fail_status(TPL_E_LAYOUT, "q and out must start, and their rows and heads lie, on 16 bytes");
    if (q.bytes() > 0 && (!ws || ((uintptr_t)ws & 15))) return fail_status(TPL_E_ARG, "workspace must lie on 16 bytes");
    if (ws_bytes < q.bytes()) return fail_status(TPL_E_ARG, "workspace is too small");
    p.counters = (int*)ws;
    p.parts = (float*)((char*)ws + kCounters * 4);
    p.tile_parts = (float*)((char*)p.parts + q.few_bytes);
    hipError_t e = hipSuccess;
    if (q.tile) e = launch_tile(p, q.dk, false, st);
    if (e == hipSuccess && q.few) e = launch_few(p, q.dc, q.mr, st);
    if (e == hipSuccess && q.tile && p.splits > 1) e = launch_tile(p, q.dk, true, st);
    if (e != hipSuccess) return fail_status(TPL_E_HIP, std::string("HIP launch failed: ") + hipGetErrorString(e));
    return TPL_OK;
}

}  // namespace kv
}  // namespace tpl

extern "C" {

int tpl_kv_attend(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_query* args, void* workspace,
                  int64_t workspace_bytes, hipStream_t stream) {
    try {
        return tpl::kv::attend_impl(cache, batch, args, workspace, workspace_bytes, stream);
    } catch (...) {
        return TPL_E_ARG;
    }
}

int64_t tpl_kv_attend_workspace(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_query* args) {
    try {
        tpl::kv::AttendArgs p;
        tpl::kv::Choice q;
        int status;
        if (const char* why = tpl::kv::choose(cache, batch, args, p, q, &status)) {
            tpl::fail_status(status, why);
            return -1;
        }
        return q.bytes();
    } catch (...) {
        return -1;
    }
}

}  // extern "C"
