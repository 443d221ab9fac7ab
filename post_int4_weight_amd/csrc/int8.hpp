// Shared device code of the int8 serving operators (linear_int8.hip,
// kv_cache.hip, attention_int8.hip): the quantization rule, and ragged
// batches.
#pragma once

#include "common.hpp"

#include <float.h>
#include <algorithm>

namespace ptq {

// ------------------------------------------------------ quantization rule --
// One scale S for a set of values with largest magnitude a: S = a / 127, code
// = rint(x / S) in [-127, 127]. S below FLT_MIN is stored as 0 (all codes 0):
// 1 / S is then always finite. A NaN or an infinity among the values makes S
// NaN, so what was stored with it reads as NaN instead of as a finite wrong
// value. The division by S is a product with 1 / S (one division per set, not
// one per value): it differs from the quotient by two roundings, 5e-6 of a
// code step at code 40.
// `amax` carries a NaN through (amax_acc).
__device__ __forceinline__ float int8_scale(float amax) {
    const float s = __fdiv_rn(amax, 127.0f);
    if (!(s <= FLT_MAX)) return __builtin_nanf("");
    return s < FLT_MIN ? 0.0f : s;
}
__device__ __forceinline__ float int8_inverse(float s) { return s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f; }
// The codes of 4 values, low byte first. Adding 3 * 2^22 to a product of at most
// 2^22 rounds it to a whole number, half to even, and leaves that number's low
// byte in the sum's. |x inv| <= 127 (1 + 2^-22) for every x of the set, so
// nothing needs clamping; the product has its own rounding (no fma).
__device__ __forceinline__ uint32_t int8_code4(float x0, float x1, float x2, float x3, float inv) {
#pragma clang fp contract(off)
    const float magic = 12582912.0f;
    const uint32_t a = __float_as_uint(x0 * inv + magic), b = __float_as_uint(x1 * inv + magic);
    const uint32_t c = __float_as_uint(x2 * inv + magic), d = __float_as_uint(x3 * inv + magic);
    return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}
__device__ __forceinline__ uint2 int8_code8(const float (&v)[8], float inv) {
    return make_uint2(int8_code4(v[0], v[1], v[2], v[3], inv), int8_code4(v[4], v[5], v[6], v[7], inv));
}
// max(|x|, a) that keeps a NaN of either
__device__ __forceinline__ float amax_acc(float a, float x) {
    const float m = fabsf(x);
    return (m > a || m != m) ? m : a;
}

// 8 consecutive elements of a row as floats
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 a = *(const uint4*)p;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

// 4 or 2 consecutive elements
__device__ __forceinline__ void load_n(const float* p, float (&v)[2]) {
    const float2 a = *(const float2*)p;
    v[0] = a.x; v[1] = a.y;
}
__device__ __forceinline__ void load_n(const uint16_t* p, float (&v)[4]) {
    const uint2 a = *(const uint2*)p;
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// float -> bf16, to nearest even, a NaN stays one (v_cvt_pk_bf16_f32)
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    union { bf16x2 h; uint32_t w; } u;
    u.h = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
    return u.w;
}
__device__ __forceinline__ uint32_t bf16_of(float f) { return bf16_pair(f, 0.f) & 0xffffu; }
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) { *(float4*)p = make_float4(a, b, c, d); }
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
    *(uint2*)p = make_uint2(bf16_pair(a, b), bf16_pair(c, d));
}

// ----------------------------------------------------------- ragged batch --
// Sequence b of a ragged batch owns rows offsets[b] .. offsets[b + 1], and has
// a number starts[b] of its own. A grid that cannot know the offsets on the
// host numbers its work units so that sequence b has units
// first(b) = floor(offsets[b] mul / div) + extra b .. first(b + 1): at least as
// many as it needs, the spare ones exit. The wave that looks a unit up reads
// 64 sequences at once, everything it needs of them in one round of loads.
// Offsets are clamped to [0, rows], so a wrong one cannot lead outside the
// caller's tensors.
struct Ragged {
    const int32_t* offsets;
    const int32_t* starts;
    int batch;
    int64_t rows;
};

struct RaggedUnit {
    int b;                 // the sequence: the last one with first(b) <= w
    int64_t off, rows;     // its rows
    int start;             // starts[b]
    int64_t local;         // w - first(b)
};

__device__ __forceinline__ RaggedUnit ragged_find(const Ragged& g, int64_t w, int mul, int div, int extra) {
    const int lane = threadIdx.x & 63;
    auto clamp = [&](int o) { return (int)(o < 0 ? 0 : (o > g.rows ? g.rows : o)); };
    RaggedUnit u{};
    for (int b0 = 0; b0 < g.batch; b0 += 64) {
        const int i = std::min(b0 + lane, g.batch - 1);
        const int o = clamp(g.offsets[i]), n = clamp(g.offsets[i + 1]), st = g.starts[i];
        const int64_t first = (int64_t)o * mul / div + (int64_t)extra * i;
        const uint64_t vote = __ballot(b0 + lane < g.batch && first <= w);
        if (!vote) break;
        const int at = 63 - __builtin_clzll(vote);
        u.b = b0 + at;
        u.off = __builtin_amdgcn_readlane(o, at);
        u.rows = std::max(__builtin_amdgcn_readlane(n, at) - (int)u.off, 0);
        u.start = __builtin_amdgcn_readlane(st, at);
        u.local = w - (u.off * mul / div + (int64_t)extra * u.b);
        if (at != 63) break;
    }
    return u;
}

}  // namespace ptq
