// Rotary positions, shared by rotary.hip and kv_cache.hip: the pairs of a head
// turn by the angle position * frequency.
//
// The angle is formed in fp64, in turns, and reduced there: a position of 10^6
// at frequency 1 keeps 2^-33 of a turn, where fp32 would keep 2^-4 of a radian.
// What is left lies within an eighth of a turn of a multiple of a quarter, and
// its sine and cosine are Taylor sums in fp32 (first omitted terms 7e-12 and
// 1.2e-10): each is within 2^-23 of the true value.
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

__device__ __forceinline__ void turn_of(int position, double freq, float magnitude, float& c, float& s) {
    const double turns = (double)position * (freq * 0.15915494309189533577);
    const double quarters = 4.0 * (turns - __builtin_rint(turns));      // in [-2, 2], exact
    const double q = __builtin_rint(quarters);
    const float x = (float)((quarters - q) * 1.57079632679489661923), y = x * x;
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
    const int k = (int)q & 3;
    c = (k & 1 ? sn : cs) * ((k == 1 || k == 2) ? -magnitude : magnitude);
    s = (k & 1 ? cs : sn) * (k >= 2 ? -magnitude : magnitude);
}

// the turned pair (a, b)
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = a;
    a = fmaf(x, c, -(b * s));
    b = fmaf(b, c, x * s);
}

// Two chunks of 8 channels of a head, a and b, that hold 8 pairs from pair i0
// on: pair k is (a[k], b[k]), or neighbours within a, then within b. Pairs from
// n on stay as they are, whatever they hold.
template <int LAYOUT>
__device__ __forceinline__ void turn_chunks(const RotaryArgs& r, int position, int i0, float (&a)[8], float (&b)[8]) {
    static_assert(LAYOUT != PAIR_ANY_HALVES, "has no chunks");
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (i0 + k >= r.n) break;
        float c, s;
        turn_of(position, r.freq[i0 + k], r.magnitude, c, s);
        if constexpr (LAYOUT == PAIR_HALVES) {
            turn_pair(a[k], b[k], c, s);
        } else {
            float (&x)[8] = k < 4 ? a : b;
            turn_pair(x[2 * k & 7], x[(2 * k & 7) + 1], c, s);
        }
    }
}

}  // namespace ptq
