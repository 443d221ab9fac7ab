// Shared device code of attention over the int8 cache (attention_int8.hip,
// attention_tree.hip).
#pragma once

#include "int8.hpp"

namespace ptq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int TK = 64;       // tokens per step of a wave
constexpr float PSHIFT = 8.f;   // p up to 2^8: fp16 keeps 11 bits down to 2^-22 of the largest
// The reference m of a row follows its maximum only when that exceeds it by
// 2^LAZY (fp16 has the room): most steps leave the output accumulators alone.
constexpr float LAZY = 6.f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 8 codes -> fp16: bytes offset to unsigned go under the exponent of 1024,
// and 1024 + 128 comes off again (exact)
__device__ __forceinline__ f16x8 half8(uint32_t a, uint32_t b) {
    const uint32_t u = a ^ 0x80808080u, v = b ^ 0x80808080u, e = 0x64646464u;
    union { uint32_t w[4]; f16x2 h[4]; f16x8 x; } r;
    r.w[0] = __builtin_amdgcn_perm(e, u, 0x04010400u);
    r.w[1] = __builtin_amdgcn_perm(e, u, 0x04030402u);
    r.w[2] = __builtin_amdgcn_perm(e, v, 0x04010400u);
    r.w[3] = __builtin_amdgcn_perm(e, v, 0x04030402u);
    const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) r.h[k] -= off;
    return r.x;
}

constexpr float LOG2_RV_MIN = -60;   // below it a block adds nothing to the output (w underflows), only to the sum

// the larger of x in this lane and in lane ^ 32
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    float larger;      // fmaxf would make both canonical first
    asm("v_max_f32 %0, %1, %2" : "=v"(larger) : "v"(r[0]), "v"(r[1]));
    return larger;
}

}  // namespace ptq
