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

// The split kernel's sizes for `items` sequences (or groups) of `rows` rows in
// all, of which it takes those of up to `limit`.
static const char* plan_few(AttendArgs& p, Choice& q, int64_t rows, int64_t items, int limit, bool pairs) {
    // 16 lanes hold dc channels each: 12 only where those are whole lanes (144 and 192 channels).
    q.dc = p.c.dim <= 64 ? 4 : p.c.dim <= 128 ? 8 : p.c.dim <= 192 && p.c.dim % 12 == 0 ? 12 : 16;
    // Rows of a tile: those of an average sequence, or of a decoding one
    // where the average is a prompt's.
    int64_t mean = (rows + items - 1) / items;
    if (mean > limit) mean = p.group;
    q.mr = mean <= 16 ? 1 : mean <= 32 || q.dc > 8 ? 2 : 4;
    // No more shares than steps there can be.
    const int64_t tiles = (rows + q.mr * 16 - 1) / (q.mr * 16) + items;
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
    if (p.a.window && (int64_t)p.a.window + p.a.sinks < seen) seen = (int64_t)p.a.window + p.a.sinks;
    const int64_t blocks = kCUs * few_blocks(p.c.type == TPL_KV_E4M3, q.dc, q.mr);
    const int w = p.c.type == TPL_KV_E4M3 ? 1 : 2;
    p.heads_log = pairs && p.c.kv_heads % 2 == 0 && p.c.k_head * w < 256 && p.c.k_head < p.c.k_token && p.c.v_head < p.c.v_token &&
                  items * (seen / 128) * p.c.kv_heads >= 24 * blocks ? 1 : 0;
    int64_t shares = blocks / (p.c.kv_heads >> p.heads_log);
    if (most > INT_MAX) return "tokens and table are too large together";
    if (shares > most) shares = most;
    p.shares = shares < 1 ? 1 : (int)shares;
    q.few_bytes = (int64_t)p.shares * p.c.kv_heads * 2 * few_part_floats(q.dc, q.mr) * 4;
    return nullptr;
}

// The tile kernel's.
static const char* plan_tile(AttendArgs& p, Choice& q, int64_t rows, int64_t items) {
    q.dk = p.c.dim <= 64 ? 64 : p.c.dim <= 96 ? 96 : p.c.dim <= 128 ? 128 : p.c.dim <= 192 ? 192 : 256;
    // Row tiles of 256 (8 waves that share a step's keys and values) where
    // they still give every CU two, else of 128.  One prompt of 8192
    // tokens, 32 heads of 128: 572 against 598 us; a chunk of 1024 tokens
    // (128 tiles of 256): 169 against 139 us.  Under a window larger tiles
    // see more that most of their rows do not (window 1024: 178 against
    // 158 us), and longer heads do not fit 8 waves' registers.
    const bool large = q.dk <= 128 && p.a.window == 0 && rows / 256 * p.c.kv_heads >= 2 * kCUs;
    p.tile_rows = large ? 256 : 128;
    p.tile_tokens = p.tile_rows / p.group;
    const int64_t tiles = (int64_t)p.g.tokens / p.tile_tokens + items;
    const int64_t units = tiles * p.c.kv_heads;
    int64_t most = p.cap;
    if (p.a.window && (int64_t)p.a.window + p.a.sinks + p.tile_tokens < most) most = (int64_t)p.a.window + p.a.sinks + p.tile_tokens;
    most = (most + 511) / 512;
    int64_t splits = 2 * kCUs / units;
    if (splits > most) splits = most;
    if (splits > 32) splits = 32;
    if (splits < 1) splits = 1;
    p.tiles = (int)tiles;
    p.splits = (int)splits;
    if (units * splits > INT_MAX) return "too many row tiles";
    if (splits > 1) q.tile_bytes = units * splits * tile_part_floats(q.dk, p.tile_rows) * 4;
    return nullptr;
}

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
    p.s = tpl_kv_groups{};
    p.prefix = p.direct = p.before_splits = 0;
    p.before = nullptr;
    p.before_ml = nullptr;
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
    if (q.few)
        if (const char* why = plan_few(p, q, rows, g->batch, limit, true)) return why;
    if (q.tile) return plan_tile(p, q, rows, g->batch);
    return nullptr;
}

static int check_query(const tpl_kv_query* a, void* ws, int64_t ws_bytes, int64_t need) {
    if (!a->q || !a->out) return fail_status(TPL_E_ARG, "q and out must not be NULL");
    if (!aligned16(a->q, a->q_token, a->q_head, 2) || !aligned16(a->out, a->o_token, a->o_head, 2))
        return fail_status(TPL_E_LAYOUT, "q and out must start, and their rows and heads lie, on 16 bytes");
    if (need > 0 && (!ws || ((uintptr_t)ws & 15))) return fail_status(TPL_E_ARG, "workspace must lie on 16 bytes");
    if (ws_bytes < need) return fail_status(TPL_E_ARG, "workspace is too small");
    return TPL_OK;
}

static int attend_impl(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_query* a, void* ws, int64_t ws_bytes,
                       hipStream_t st) {
    AttendArgs p;
    Choice q;
    int status;
    if (const char* why = choose(c, g, a, p, q, &status)) return fail_status(status, why);
    if (!q.few && !q.tile) return TPL_OK;
    if (const int bad = check_query(a, ws, ws_bytes, q.bytes())) return bad;
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

// Sequences that share tokens, in one of two ways.
//
// Two launches: groups' rows over the tokens that they share, whose results stay
// in 32 bits in the workspace, then sequences' rows over their own tokens, which
// begin from those results.
//
// Directly: each sequence's rows over the shared tokens and its own.
struct SharedChoice {
    Choice q1, q2;
    int64_t few_bytes, rows;   // of both launches' parts; rows * heads of the results between them
    int64_t bytes;
};

// The tile kernel's sizes for groups' rows over their shared tokens.  All tiles
// of a group see the same tokens, so that nothing but the ends of rounds over
// the CUs speaks against row tiles of 256: they are taken from 512 rows a group
// on (256 samples of 32768 tokens, 2048 rows for each of 8 heads, in 4 parts:
// 318 against 363 us with tiles of 128; 256 rows over 4096 tokens 62 against 59).
// The number of parts is what the model below finds best, in steps of a workgroup
// with a CU to itself (3.5 us): rounds of workgroups, of which two on a CU take
// 1.5 times as long, each two steps' time to begin and end, and the writing and
// reading of what a part leaves of every row.  With 8, 16 and 32 parts: 64
// sequences behind 4096 tokens, 256 rows for each of 8 heads, 48, 46 and 53 us; 16
// behind 8192 47, 35 and 32; 24 behind 16000 105, 75 and 65; 256 behind 4096 74,
// 98 and 162.
static const char* plan_prefix_tile(AttendArgs& p, Choice& q, int64_t rows, int64_t groups) {
    q.dk = p.c.dim <= 64 ? 64 : p.c.dim <= 96 ? 96 : p.c.dim <= 128 ? 128 : p.c.dim <= 192 ? 192 : 256;
    const int64_t mean = (rows + groups - 1) / groups;
    const bool large = q.dk <= 128 && mean >= 512;
    p.tile_rows = large ? 256 : 128;
    p.tile_tokens = p.tile_rows / p.group;
    const int64_t per = (int64_t)p.tile_tokens * p.group, units = groups * ((mean + per - 1) / per) * p.c.kv_heads;
    const int64_t steps = ((int64_t)p.cap + 63) / 64;
    const bool pairs = !large && q.dk <= 128;   // two workgroups fit a CU
    const double part = (double)rows * p.c.kv_heads * p.c.dim * 8.0 / 14e6;   // bytes to and from memory, of a step's time
    double least = 1e300;
    for (int s = 1; s <= 64 && (s == 1 || s * 2 <= steps); ++s) {
        const int64_t n = units * s, slots = pairs ? 2 * kCUs : kCUs, rest = n % slots;
        const double rounds = (pairs ? 1.5 : 1.0) * (double)(n / slots) + (rest == 0 ? 0.0 : rest <= kCUs ? 1.0 : 1.5);
        const double cost = rounds * (double)((steps + s - 1) / s + 2) + part * s;
        if (cost < least) least = cost, p.splits = s;
    }
    const int64_t tiles = (int64_t)p.g.tokens / p.tile_tokens + groups;
    if (tiles * p.c.kv_heads * p.splits > INT_MAX) return "too many row tiles";
    p.tiles = (int)tiles;
    return nullptr;
}

static const char* choose_shared(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_groups* s, const tpl_kv_query* a,
                                 AttendArgs& p1, AttendArgs& p2, SharedChoice& x, int* status) {
    if (!s) {
        *status = TPL_E_ARG;
        return "groups must not be NULL";
    }
    if (const char* why = choose(c, g, a, p2, x.q2, status)) return why;
    if (a->window || a->sinks) return "sequences that share tokens have no window and no sinks";
    if (s->count < 0 || s->count > (1 << 20)) return "groups must be 0 .. 2^20";
    x.bytes = x.q2.bytes();
    x.few_bytes = x.q2.few_bytes;
    x.rows = 0;
    x.q1 = Choice{};
    if (s->count == 0 || (!x.q2.few && !x.q2.tile)) return nullptr;
    if (!s->groups || !s->shared) return "groups and shared must not be NULL";
    p2.s = *s;
    // Directly where an average sequence fills a row tile by itself: its
    // products over the shared tokens are as many either way (16 questions of
    // 300 tokens behind 2048, 8 heads a cache's: 242 against 290 us).  And
    // where all sequences' reading of whole rows of the table comes to 96 MiB
    // at most, which the caches beside HBM give in less time than a second
    // launch with its chain of reads takes (e4m3, 8 heads of 128; directly
    // against in two launches: 4 sequences of 530 tokens 12 against 22 us, 4 of
    // 8200 24 against 34, 64 of 530 18 against 25, 16 of 2200, 72 MB, 25 against
    // 26, 16 of 4200, 138 MB, 33 against 29, 64 of 1800 42 against 31; 256 of
    // 500, 262 MB, 50 against 53).
    const int64_t rows = (int64_t)g->tokens * p2.group, w = c->type == TPL_KV_E4M3 ? 1 : 2;
    const int64_t tiles = (rows + g->batch * 16 - 1) / ((int64_t)g->batch * 16);   // of 16 rows, of an average sequence
    const double once = (double)(g->batch * tiles * c->kv_heads) * (double)(c->dim * 2 * w) * p2.cap;
    if (rows >= (int64_t)g->batch * 128 || once <= 0x1.8p26) {
        p2.direct = 1;
        return nullptr;
    }
    p1 = p2;
    p1.prefix = 1;
    // A group of up to 16 rows goes through the split kernel; with 32 and 64
    // rows that took 72 and 47 us where row tiles take 67 and 32 (8 sequences of
    // 32200 tokens, 16 of 2200).
    if (p1.group > 128 || rows <= (int64_t)s->count * 16) {
        x.q1.few = true;
        p1.few = INT_MAX;
        if (const char* why = plan_few(p1, x.q1, rows, s->count, 64, true)) return why;
        p1.before_splits = 1;
    } else {
        x.q1.tile = true;
        p1.few = 0;
        if (const char* why = plan_prefix_tile(p1, x.q1, rows, s->count)) return why;
        p1.before_splits = p1.splits;
    }
    // Sequences' own tokens are taken to be few: one kernel for all of them, a
    // head a workgroup.
    x.q2 = Choice{};
    x.q2.few = true;
    p2.few = INT_MAX;
    if (const char* why = plan_few(p2, x.q2, rows, g->batch, 64, false)) return why;
    p2.before_splits = p1.before_splits;
    x.few_bytes = x.q1.few_bytes > x.q2.few_bytes ? x.q1.few_bytes : x.q2.few_bytes;
    x.rows = (int64_t)p1.before_splits * g->tokens * a->heads;
    x.bytes = kCounters * 4 + x.few_bytes + x.rows * (c->dim * 4 + 8);
    return nullptr;
}

static int attend_shared_impl(const tpl_kv_cache* c, const tpl_kv_batch* g, const tpl_kv_groups* s, const tpl_kv_query* a, void* ws,
                              int64_t ws_bytes, hipStream_t st) {
    AttendArgs p1, p2;
    SharedChoice x;
    int status;
    if (const char* why = choose_shared(c, g, s, a, p1, p2, x, &status)) return fail_status(status, why);
    if (!x.q2.few && !x.q2.tile) return TPL_OK;
    if (s->count == 0) return attend_impl(c, g, a, ws, ws_bytes, st);
    if (const int bad = check_query(a, ws, ws_bytes, x.bytes)) return bad;
    p2.counters = (int*)ws;
    p2.parts = (float*)((char*)ws + kCounters * 4);
    p2.tile_parts = (float*)((char*)p2.parts + x.few_bytes);
    hipError_t e = hipSuccess;
    if (!p2.direct) {
        p1.counters = p2.counters;
        p1.parts = p2.parts;
        p1.before = p2.before = p2.tile_parts;
        p1.before_ml = p2.before_ml = (float2*)(p1.before + x.rows * c->dim);
        e = x.q1.tile ? launch_tile_shared(p1, x.q1.dk, false, st) : launch_few_shared(p1, x.q1.dc, x.q1.mr, st);
    }
    if (e == hipSuccess && x.q2.tile) e = launch_tile_shared(p2, x.q2.dk, false, st);
    if (e == hipSuccess && x.q2.few) e = launch_few_shared(p2, x.q2.dc, x.q2.mr, st);
    if (e == hipSuccess && x.q2.tile && p2.splits > 1) e = launch_tile_shared(p2, x.q2.dk, true, st);
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

int tpl_kv_attend_shared(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_groups* groups,
                         const tpl_kv_query* args, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    try {
        return tpl::kv::attend_shared_impl(cache, batch, groups, args, workspace, workspace_bytes, stream);
    } catch (...) {
        return TPL_E_ARG;
    }
}

int64_t tpl_kv_attend_shared_workspace(const tpl_kv_cache* cache, const tpl_kv_batch* batch, const tpl_kv_groups* groups,
                                       const tpl_kv_query* args) {
    try {
        tpl::kv::AttendArgs p1, p2;
        tpl::kv::SharedChoice x;
        int status;
        if (const char* why = tpl::kv::choose_shared(cache, batch, groups, args, p1, p2, x, &status)) {
            tpl::fail_status(status, why);
            return -1;
        }
        return x.bytes;
    } catch (...) {
        return -1;
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
