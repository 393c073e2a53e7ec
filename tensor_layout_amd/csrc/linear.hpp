// linear.hpp -- argument block and the reading of batches of the linear
// attention kernels.
#pragma once

#include "../../include/tpl_linear.h"
#include "common.hpp"
#include "kv.hpp"

namespace tpl {
namespace linear {

using kv::f32x4;
using kv::f32x16;
using kv::hi16;
using kv::lo16;
using kv::pack2;
using kv::u32x2;
using kv::u32x4;

// A sequence of up to this many new tokens goes token by token.  64 sequences, 32
// heads of 128 by 128: of 4 tokens 68 us that way and 79 in a chunk, of 8 81 and
// 79, of 16 111 and 82.  At 8 the two are even, and the recurrence is exact to fp32.
constexpr int kFew = 8;
constexpr int kChunk = 64;   // tokens that longer ones take together

struct LinearArgs {
    tpl_linear_pool p;
    tpl_linear_batch g;
    tpl_linear_new a;
    float* parts;        // workspace: states [segments][heads][key_dim][value_dim]
    int32_t few;         // the token-by-token kernel takes sequences of at most this many rows
    int32_t share;       // heads that read one of the keys'
    int32_t slices;      // workgroups of a head, by value channels
    int32_t segment;     // tokens of a segment
};

// A sequence's rows; none where they are not in order.
struct Rows {
    int row0, n;
};

__device__ __forceinline__ Rows rows_of(const tpl_linear_batch& g, int b) {
    const int r = g.starts[b], e = g.starts[b + 1];
    return r >= 0 && e > r && e <= g.tokens ? Rows{r, e - r} : Rows{0, 0};
}

// A state in the pool; nullptr where the number is not one of its slots.
__device__ __forceinline__ float* state_at(const LinearArgs& p, int slot, int head) {
    return slot >= 0 && slot < p.p.slots ? p.p.state + slot * p.p.s_slot + head * p.p.s_head : nullptr;
}
__device__ __forceinline__ const float* source_of(const LinearArgs& p, int b, int head) {
    return state_at(p, p.g.sources ? p.g.sources[b] : p.g.slots[b], head);
}

// The logarithm to base 2 of a head's decay: at most zero, and finite, so that
// a decay to nothing leaves exp2(0 * it) at one.  No number stays none.
__device__ __forceinline__ float decay_of(const LinearArgs& p, int head) {
    const float d = p.p.decay[head];
    return d != d ? d : fmaxf(fminf(d, 0.0f) * 1.44269504088896340736f, -1.0e6f);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

hipError_t launch_step(const LinearArgs& p, bool narrow, hipStream_t st);
enum { kWhole = 0, kState = 1, kOutput = 2 };   // what launch_chunk does with its sequences or segments
hipError_t launch_chunk(const LinearArgs& p, int mode, int64_t units, hipStream_t st);
hipError_t launch_scan(const LinearArgs& p, hipStream_t st);
int chunk_waves(int key_dim, int value_dim);    // of a workgroup
int chunk_slices(int key_dim, int value_dim);   // workgroups of a head

}  // namespace linear
}  // namespace tpl
