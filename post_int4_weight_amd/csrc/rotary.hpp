// Rotary positions, shared by rotary.hip and kv_cache.hip: the pairs of a head
// turn by the angle position * frequency.
//
// The angle is formed in fp64, in quarters of a turn, and reduced there: a
// position of 10^6 at frequency 1 keeps 2^-33 of a turn, where fp32 would keep
// 2^-4 of a radian. What is left lies within half a quarter, and its sine and
// cosine are Taylor sums in fp32 (first omitted terms 7e-12 and 1.2e-10): each is
// within 2^-23 + 2^-51 |angle| of the true value, the latter for the roundings of
// the angle in fp64 (2^-23 alone up to 10^8 radians, 2.7 times that near 2^31).
#pragma once

#include "int8.hpp"

namespace ptq {

// How the pairs (a, b) lie in a head of which the first 2 n channels turn.
enum PairLayout {
    PAIR_HALVES = 0,      // (i, i + n), n a multiple of 8: both are whole chunks of 8 channels
    PAIR_NEIGHBOURS = 1,  // (2 i, 2 i + 1)
    PAIR_ANY_HALVES = 2   // (i, i + n), any n: element by element
};

struct RotaryArgs {
    const double* freq;       // [n], radians per position
    const int32_t* positions; // of each row, or null (kv_cache.hip: the slot's own)
    int n;                    // pairs
    float magnitude;          // factor of the turned channels
};

inline PairLayout pair_layout(int n, int interleaved) {
    return interleaved ? PAIR_NEIGHBOURS : n % 8 == 0 ? PAIR_HALVES : PAIR_ANY_HALVES;
}

// cosine and sine, times the magnitude, of position * freq
__device__ __forceinline__ float2 turn_of(double position, double freq, float magnitude) {
    const double t = position * (freq * 0.63661977236758134308);      // quarters
    const double q = __builtin_rint(t);
    const float x = (float)((t - q) * 1.57079632679489661923), y = x * x;
    float sn = fmaf(y, -2.50521084e-8f, 2.75573192e-6f);      // -1 / 11!, 1 / 9!
    sn = fmaf(y, sn, -1.98412698e-4f);
    sn = fmaf(y, sn, 8.33333333e-3f);
    sn = fmaf(y, sn, -1.66666667e-1f);
    sn = fmaf(x * y, sn, x);
    float cs = fmaf(y, -2.75573192e-7f, 2.48015873e-5f);      // -1 / 10!, 1 / 8!
    cs = fmaf(y, cs, -1.38888889e-3f);
    cs = fmaf(y, cs, 4.16666667e-2f);
    cs = fmaf(y, cs, -0.5f);
    cs = fmaf(y, cs, 1.f);
    // q modulo 4: the low bits of q + 1.5 2^52 (an angle of 2^51 quarters has no place in a turn any more)
    const uint32_t k = (uint32_t)__double2loint(q + 6755399441055744.0);
    const float c = k & 1 ? sn : cs, s = k & 1 ? cs : sn;
    const uint32_t neg_c = ((k + 1) << 30) & 0x80000000u, neg_s = (k << 30) & 0x80000000u;
    return make_float2(__uint_as_float(__float_as_uint(c) ^ neg_c) * magnitude, __uint_as_float(__float_as_uint(s) ^ neg_s) * magnitude);
}

// the turned pair (a, b)
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = a;
    a = fmaf(x, c, -(b * s));
    b = fmaf(b, c, x * s);
}

// Elements 0 .. n - 1 of 8 from anywhere; storing leaves the first ones out
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, float (&v)[8]) {
    if (n >= 8) {
        struct { alignas(16) T x[8]; } w;
        __builtin_memcpy(&w, p, sizeof(w));
        load8(w.x, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? load_as_float(p, k) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int skip, int n, const float (&v)[8]) {
    if (n >= 8 && skip == 0) {
        struct { alignas(16) T x[8]; } w;
        store8(w.x, v);
        __builtin_memcpy(p, &w, sizeof(w));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k >= skip && k < n) store1(p + k, v[k]);
    }
}

}  // namespace ptq
