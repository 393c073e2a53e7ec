// linear.hip -- linear attention with a decay for each head: checks of
// arguments, choice of the kernels, C entry points.
#include <climits>

#include "linear.hpp"

namespace tpl {
namespace linear {

constexpr int kCUs = 256;

struct Choice {
    bool step, whole, parts;   // kernels: token by token; chunks, whole sequences or segments of them
    bool narrow;
    int64_t segments, bytes;
};

static bool lies16(const void* p, int64_t s0, int64_t s1, int bytes) { return kv::aligned16(p, s0, s1, bytes); }

static const char* choose(const tpl_linear_pool* c, const tpl_linear_batch* g, const tpl_linear_new* a, LinearArgs& p, Choice& q,
                          int* status) {
    *status = TPL_E_ARG;
    q = Choice{};
    if (!c || !g || !a) return "pool, batch and arguments must not be NULL";
    if (!c->state || !c->decay) return "state and decay must not be NULL";
    if (c->slots < 1 || c->slots > INT_MAX) return "a pool must have at least one slot";
    if (c->heads < 1 || c->heads > 65535) return "heads must be 1 .. 65535";
    if (c->key_dim < 16 || c->key_dim > 256 || c->key_dim % 16 || c->value_dim < 16 || c->value_dim > 256 || c->value_dim % 16)
        return "dims must be multiples of 16, at most 256";
    for (int64_t x : {c->s_slot, c->s_head, c->s_key})
        if (x > ((int64_t)1 << 40) || x < -((int64_t)1 << 40)) return "strides must be under 2^40";
    if (!lies16(c->state, c->s_slot, c->s_head, 4) || (c->s_key * 4) % 16) return "states must lie on 16 bytes";
    if (g->batch < 0 || g->tokens < 0) return "batch and tokens must be >= 0";
    if (g->batch > (1 << 20)) return "batch must be at most 2^20";
    if (g->tokens > (1 << 28)) return "tokens must be at most 2^28";
    if (g->batch && (!g->slots || !g->starts)) return "slots and starts must not be NULL";
    if (a->type != TPL_KV_BF16 && a->type != TPL_KV_FP16) {
        *status = TPL_E_DTYPE;
        return "q, k and v must be bf16 or fp16";
    }
    if (a->key_heads < 1 || c->heads % a->key_heads) return "heads must be a multiple of the keys'";
    if (!(a->scale > -__builtin_inff()) || !(a->scale < __builtin_inff())) return "scale must be a finite number";
    p.p = *c;
    p.g = *g;
    p.a = *a;
    p.parts = nullptr;
    p.share = c->heads / a->key_heads;
    p.slices = chunk_slices(c->key_dim, c->value_dim);
    p.segment = kChunk;
    p.few = kFew;
    if (g->batch == 0 || g->tokens == 0) return nullptr;

    // Which kernel takes a sequence goes by its rows, which only the device
    // knows; the host leaves out one that no sequence can need, and where there
    // are no more rows than sequences (decoding) or one sequence lets one
    // kernel take whatever there is.
    if (g->tokens <= kFew || (g->batch > 1 && g->tokens <= g->batch)) {
        q.step = true;
        p.few = INT_MAX;
    } else if (g->batch == 1) {
        p.few = 0;
    } else {
        q.step = true;
    }
    const int64_t heads = (int64_t)g->batch * c->heads;
    if (q.step) {
        // Slices of 64 value channels, or of 32 where those would leave CUs
        // without work: 4 sequences of 16 heads of 128 take 4.5 us in slices of 32
        // and 5.1 in ones of 64, 128 of 32 heads 110 and 108.
        q.narrow = heads * ((c->value_dim + 63) / 64) < 2 * kCUs;
        if (heads * ((c->value_dim + 31) / 32) > INT_MAX) return "batch * heads is too large";
    }
    if (p.few != INT_MAX) {
        const int64_t units = heads * p.slices;
        // Whole sequences, or segments of them: as many as the model below finds
        // best, in units of a chunk by a workgroup that has its SIMDs to itself.
        // A workgroup takes its chunks and two more's time to begin and end; two
        // waves a SIMD, as many as up to 128 key channels allow, take 1.6 times
        // as long; segments take keys and values twice, 1.3 times the work, and
        // the scan; sequences of unlike lengths end apart, which is counted as a
        // tenth.  Measured, whole and in the segments that are chosen: a prompt of
        // 8192 tokens, 32 heads of 128, 713 and 131 us (16 of them; 8: 143, 12:
        // 146, 24: 150); 4 of 2000 190 and 144 (4; 2: 189, 8: 156); 8 of 4000,
        // whole, 375 (2: 471, 3: 463); 24 of up to 4000, 12 heads of 64 by 96, 317
        // and 264 (3).
        const int64_t slots = kCUs * 8 / chunk_waves(c->key_dim, c->value_dim), chunks = (g->tokens / g->batch + kChunk - 1) / kChunk;
        const auto rounds = [&](int64_t n) {
            const int64_t half = slots / 2;
            if (c->key_dim > 128) return (double)((n + half - 1) / half);
            const int64_t rest = n % slots;
            return 1.6 * (double)(n / slots) + (rest == 0 ? 0.0 : rest <= half ? 1.0 : 1.6);
        };
        double least = 1.1 * rounds(units) * (double)(chunks + 2);
        int64_t segments = 1;
        for (int64_t n = 2; n * 3 <= chunks * 2 && units * n < 8 * slots; ++n) {
            const double cost = 1.3 * rounds(units * n) * (double)((chunks + n - 1) / n + 2) + 2.0 * (double)(units * n) / (double)slots;
            if (cost < least) least = cost, segments = n;
        }
        if (segments > 1) {
            const int64_t segment = (chunks + segments - 1) / segments * kChunk;
            q.parts = true;
            p.segment = (int)segment;
            q.segments = g->tokens / segment + g->batch;
            q.bytes = q.segments * c->heads * c->key_dim * c->value_dim * 4;
            if (q.segments * c->heads * p.slices > INT_MAX) return "tokens * heads is too large";
        } else {
            q.whole = true;
            if (units > INT_MAX) return "batch * heads is too large";
        }
    }
    return nullptr;
}

static int attend_impl(const tpl_linear_pool* c, const tpl_linear_batch* g, const tpl_linear_new* a, void* ws, int64_t ws_bytes,
                       hipStream_t st) {
    LinearArgs p;
    Choice q;
    int status;
    if (const char* why = choose(c, g, a, p, q, &status)) return fail_status(status, why);
    if (!q.step && !q.whole && !q.parts) return TPL_OK;
    if (!a->q || !a->k || !a->v || !a->out) return fail_status(TPL_E_ARG, "q, k, v and out must not be NULL");
    if (!lies16(a->q, a->q_token, a->q_head, 2) || !lies16(a->k, a->k_token, a->k_head, 2) || !lies16(a->v, a->v_token, a->v_head, 2) ||
        !lies16(a->out, a->o_token, a->o_head, 2))
        return fail_status(TPL_E_LAYOUT, "q, k, v and out must start, and their rows and heads lie, on 16 bytes");
    // A chunk's rows have 32-bit offsets in the kernels.
    for (int64_t x : {a->q_token, a->k_token, a->v_token})
        if (g->tokens > 1 && (x < 0 || x > (INT_MAX >> 7))) return fail_status(TPL_E_LAYOUT, "rows of q, k and v must lie under 2^24 elements apart");
    if (q.bytes > 0 && (!ws || ((uintptr_t)ws & 15))) return fail_status(TPL_E_ARG, "workspace must lie on 16 bytes");
    if (ws_bytes < q.bytes) return fail_status(TPL_E_ARG, "workspace is too small");
    p.parts = (float*)ws;
    hipError_t e = hipSuccess;
    if (q.whole) e = launch_chunk(p, kWhole, g->batch, st);
    if (q.parts) {
        e = launch_chunk(p, kState, q.segments, st);
        if (e == hipSuccess) e = launch_scan(p, st);
        if (e == hipSuccess) e = launch_chunk(p, kOutput, q.segments, st);
    }
    if (e == hipSuccess && q.step) e = launch_step(p, q.narrow, st);
    if (e != hipSuccess) return fail_status(TPL_E_HIP, std::string("HIP launch failed: ") + hipGetErrorString(e));
    return TPL_OK;
}

}  // namespace linear
}  // namespace tpl

extern "C" {

int tpl_linear_attend(const tpl_linear_pool* pool, const tpl_linear_batch* batch, const tpl_linear_new* args, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream) {
    try {
        return tpl::linear::attend_impl(pool, batch, args, workspace, workspace_bytes, stream);
    } catch (...) {
        return TPL_E_ARG;
    }
}

int64_t tpl_linear_attend_workspace(const tpl_linear_pool* pool, const tpl_linear_batch* batch, const tpl_linear_new* args) {
    try {
        tpl::linear::LinearArgs p;
        tpl::linear::Choice q;
        int status;
        if (const char* why = tpl::linear::choose(pool, batch, args, p, q, &status)) {
            tpl::fail_status(status, why);
            return -1;
        }
        return q.bytes;
    } catch (...) {
        return -1;
    }
}

}  // extern "C"
