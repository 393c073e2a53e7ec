// kv.hpp -- what the paged key/value cache kernels share: argument blocks,
// 16-bit and e4m3 conversions, and the reading of a batch's device arrays.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>
#include <type_traits>

#include "../../include/tpl_kv.h"

namespace tpl {

int fail_status(int status, const std::string& why);   // kernels.hip

namespace kv {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The two 16-bit types: their vectors, matrix instructions and conversions.
// e4m3 converts to either without rounding (4 significant bits, 2^-9 .. 448).
struct Bf16 {
    typedef __bf16 one;
    typedef bf16x2 x2;
    typedef bf16x8 x8;
    static __device__ __forceinline__ f32x4 mfma16(x8 a, x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
};

struct Fp16 {
    typedef _Float16 one;
    typedef f16x2 x2;
    typedef f16x8 x8;
    static __device__ __forceinline__ f32x4 mfma16(x8 a, x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    }
};

// e4m3 times a scale's power of two, as bf16: nothing is rounded while the
// product stays a normal number.  scale_rest is what the power of two leaves
// of a normal scale over zero: 1 to under 2, and 1 for every scale that
// tpl_kv_append sets.
template <bool HI>
__device__ __forceinline__ uint32_t bf16_from_e4m3(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
}
__device__ __forceinline__ float scale_rest(float scale) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, scale) & 0x007fffffu) | 0x3f800000u);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typename T::x2 r;
    r[0] = (typename T::one)a;
    r[1] = (typename T::one)b;
    return __builtin_bit_cast(uint32_t, r);
}

// Clears the values of a word that are no finite numbers; whether there were
// any.  An exponent of all ones (for e4m3, which has no infinities, the code
// of all ones) carries into the sign's place when one is added to it.
struct E4m3 {};
template <typename H>
__device__ __forceinline__ bool clear_bad(uint32_t& w) {
    constexpr bool e4 = std::is_same<H, E4m3>::value, bf = std::is_same<H, Bf16>::value;
    constexpr uint32_t ones = e4 ? 0x7f7f7f7fu : bf ? 0x7f807f80u : 0x7c007c00u, unit = e4 ? 0x01010101u : bf ? 0x00800080u : 0x04000400u;
    const uint32_t top = e4 ? 0x80808080u : 0x80008000u;
    const uint32_t bad = ((w & ones) + unit) & top;
    if (bad) w &= ~((bad >> (e4 ? 7 : 15)) * (e4 ? 0xffu : 0xffffu));
    return bad != 0;
}

template <typename T>
__device__ __forceinline__ float lo16(uint32_t w) { return (float)__builtin_bit_cast(typename T::x2, w)[0]; }
template <typename T>
__device__ __forceinline__ float hi16(uint32_t w) { return (float)__builtin_bit_cast(typename T::x2, w)[1]; }

// One value of a cache, for the rare cases that ask for it alone.
template <typename H>
__device__ __forceinline__ float value_at(const uint8_t* p) {
    if constexpr (std::is_same<H, E4m3>::value) {
        return __builtin_amdgcn_cvt_f32_fp8(*p, 0);
    } else {
        return lo16<H>(*reinterpret_cast<const uint16_t*>(p));
    }
}

// Tokens of a sequence: far enough from 2^31 that sums of positions and tile
// offsets stay 32-bit numbers.
constexpr int kMaxLength = 1 << 30;

// A sequence of the batch as its device arrays give it; one that is not in
// order (see tpl_kv.h) has no new tokens.
struct Seq {
    int row0;    // its first row
    int n;       // new tokens
    int length;  // tokens with them
};

__device__ __forceinline__ Seq ordered(int row0, int end, int length, int tokens) {
    const bool ok = row0 >= 0 && end > row0 && end <= tokens && length >= end - row0 && length <= kMaxLength;
    return ok ? Seq{row0, end - row0, length} : Seq{0, 0, 0};
}

__device__ __forceinline__ Seq read_seq(const tpl_kv_batch& g, int b) {
    return ordered(g.starts[b], g.starts[b + 1], g.lengths[b], g.tokens);
}

// The sequence that row tile x belongs to, where a tile has up to `per` rows:
// sequence b's tiles are numbered from starts[b] / per + b on, and of those in
// order whose numbers begin at or before x it is the last.  64 are looked at
// together, with all that is needed of them, so that it is known after one
// load's latency.  b is -1 where there is none.
struct TileSeq {
    int b;
    Seq s;
};

__device__ __forceinline__ TileSeq seq_of_tile(const tpl_kv_batch& g, int per, int x) {
    const int lane = threadIdx.x & 63;
    TileSeq t = {-1, {0, 0, 0}};
    for (int b0 = 0; b0 < g.batch; b0 += 64) {
        const int bb = b0 + lane < g.batch ? b0 + lane : g.batch - 1;
        const Seq s = read_seq(g, bb);
        const uint64_t m = __ballot(b0 + lane < g.batch && s.n > 0 && s.row0 / per + bb <= x);
        if (m) {
            const int from = 63 - __builtin_clzll(m);
            t.b = b0 + from;
            t.s.row0 = __builtin_amdgcn_readlane(s.row0, from);
            t.s.n = __builtin_amdgcn_readlane(s.n, from);
            t.s.length = __builtin_amdgcn_readlane(s.length, from);
        }
    }
    return t;
}

// What the operators check alike (kv_attend.hip).
const char* check_cache(const tpl_kv_cache* c);
const char* check_batch(const tpl_kv_cache& c, const tpl_kv_batch* g);
bool aligned16(const void* p, int64_t s0, int64_t s1, int bytes);

}  // namespace kv
}  // namespace tpl
