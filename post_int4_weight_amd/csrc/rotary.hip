// Rotary positions on the heads of each token (arithmetic in rotary.hpp):
//   y_a = m (x_a cos t - x_b sin t), y_b = m (x_b cos t + x_a sin t),
//   t = position * frequency of the pair; channels past the pairs are copied.
//
// A thread takes 16 channels of a token, 8 pairs or 16 channels past them, in
// HEADS heads: the 8 sines and cosines (about 30 instructions each) are formed
// once and all loads go out before them. Neighbouring threads take neighbouring
// channels, then heads, then tokens, so that a wave reads whole stretches of a row
// (with heads in another dimension of the grid: 124 us where it takes 96). What
// bounds it is memory: 16384 tokens, 64 heads of 128, bf16: 96 us, 5.6 TB/s, a copy
// of them 101; neighbours as pairs 102, halves of 45 pairs 131. A single head of
// 200000 tokens, whose sines no other shares: 31 us, 3.3 TB/s. For a few tokens
// (64, 32 heads) it is the launch: 3 us of the kernel, 8 of the call.
#include "rotary.hpp"

namespace ptq {
namespace {

template <typename T>
struct ApplyArgs {
    RotaryArgs r;
    const T* X; int64_t ldx;
    T* Y; int64_t ldy;
    unsigned total;           // threads: rows x groups x items
    int heads, dim;
    int turning, items;       // items of a token that turn, and all that are written
    int groups;               // of heads: group g has heads g, g + groups, ..
};

template <typename T, int LAYOUT, int HEADS>
__global__ __launch_bounds__(256) void rotary_kernel(ApplyArgs<T> a) {
    const unsigned at = blockIdx.x * 256u + threadIdx.x;
    if (at >= a.total) return;
    const int item = (int)(at % (unsigned)a.items), group = (int)(at / (unsigned)a.items % (unsigned)a.groups);
    const unsigned row = at / (unsigned)a.items / (unsigned)a.groups;
    const T* X = a.X + row * a.ldx;
    T* Y = a.Y + row * a.ldy;
    const bool turns = item < a.turning;
    // Channels of the item: n_a of them from c_a on, n_b from c_b on. Where the last ones of halves of any size, or of
    // channels past the pairs, are fewer than 8, the item takes the 8 that end there: `again` of its pairs are another's.
    int i0 = 8 * item, again = 0, c_a, c_b, n_a = 8, n_b = 8;
    if (turns && LAYOUT != PAIR_NEIGHBOURS) {
        if (LAYOUT == PAIR_ANY_HALVES) {
            again = std::max(0, std::min(i0, i0 + 8 - a.r.n));
            i0 -= again;
            n_a = n_b = std::min(8, a.r.n);
        }
        c_a = i0, c_b = i0 + a.r.n;
    } else {
        c_a = LAYOUT == PAIR_NEIGHBOURS ? 16 * item : 2 * a.r.n + 16 * (item - a.turning);
        c_b = c_a + 8;
        if (c_b >= a.dim) n_b = 0;
        if (LAYOUT == PAIR_ANY_HALVES) {
            n_a = std::min(8, a.dim - 2 * a.r.n);
            c_a = std::min(c_a, a.dim - n_a), c_b = std::min(c_b, a.dim - 8);
        }
    }
    const int pairs = std::min(8, a.r.n - i0);
    double f[8], position = 0.;
    if (turns) {
        position = (double)a.r.positions[row];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = a.r.freq[i0 + std::min(k, pairs - 1)];
    }
    float x[HEADS][2][8];
    int64_t head[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        head[h] = (int64_t)std::min(group + h * a.groups, a.heads - 1) * a.dim;      // past the last head: that one again
        if constexpr (LAYOUT == PAIR_ANY_HALVES) {
            load_some(X + head[h] + c_a, n_a, x[h][0]);
            load_some(X + head[h] + c_b, n_b, x[h][1]);
        } else {
            load8(X + head[h] + c_a, x[h][0]);
            load8(X + head[h] + (n_b ? c_b : c_a), x[h][1]);
        }
    }
    if (turns) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (LAYOUT != PAIR_HALVES && k >= pairs) break;
            const float2 t = turn_of(position, f[k], a.r.magnitude);
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                if constexpr (LAYOUT == PAIR_NEIGHBOURS)
                    turn_pair(x[h][k >> 2][2 * k & 7], x[h][k >> 2][(2 * k & 7) + 1], t.x, t.y);
                else
                    turn_pair(x[h][0][k], x[h][1][k], t.x, t.y);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if (group + h * a.groups >= a.heads) break;
        if constexpr (LAYOUT == PAIR_ANY_HALVES) {
            // in place, the pairs that are another's may have turned before they were loaded
            const int skip = a.X == a.Y ? again : 0;
            store_some(Y + head[h] + c_a, skip, n_a, x[h][0]);
            store_some(Y + head[h] + c_b, skip, n_b, x[h][1]);
        } else {
            store8(Y + head[h] + c_a, x[h][0]);
            if (n_b) store8(Y + head[h] + c_b, x[h][1]);
        }
    }
}

template <typename T, int LAYOUT>
int launch(ApplyArgs<T> a, int64_t rows, hipStream_t st) {
    constexpr int MANY = 4;
    const int64_t units = rows * a.items;
    const bool few = units * cdiv(a.heads, MANY) < 256 * 1024;      // not one wave for each SIMD
    a.groups = few ? a.heads : (int)cdiv(a.heads, MANY);
    // a launch of 2^32 threads or more wraps without an error
    if (units > (((int64_t)1 << 32) - 256) / a.groups) {
        set_error("rotary_apply: rows = %lld with %d heads of %d channels are too many for a launch", (long long)rows,
                  a.heads, a.dim);
        return PTQ_EINVAL;
    }
    a.total = (unsigned)(units * a.groups);
    const dim3 grid((unsigned)cdiv((int64_t)a.total, 256));
    if (few)
        hipLaunchKernelGGL((rotary_kernel<T, LAYOUT, 1>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((rotary_kernel<T, LAYOUT, MANY>), grid, dim3(256), 0, st, a);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

template <typename T>
int launch_layout(const T* X, int64_t ldx, T* Y, int64_t ldy, int64_t rows, int heads, int dim, const RotaryArgs& r,
                  int layout, hipStream_t st) {
    const bool in_place = X == Y;      // channels past the pairs are there already
    ApplyArgs<T> a{r, X, ldx, Y, ldy, 0, heads, dim, 0, 0, 0};
    a.turning = (int)cdiv(r.n, 8);
    a.items = in_place ? a.turning : (int)(layout == PAIR_NEIGHBOURS ? cdiv(dim, 16) : a.turning + cdiv(dim - 2 * r.n, 16));
    switch (layout) {
        case PAIR_HALVES: return launch<T, PAIR_HALVES>(a, rows, st);
        case PAIR_NEIGHBOURS: return launch<T, PAIR_NEIGHBOURS>(a, rows, st);
        default: return launch<T, PAIR_ANY_HALVES>(a, rows, st);
    }
}

}  // namespace

int launch_rotary(const void* X, int64_t ldx, void* Y, int64_t ldy, int dtype, int64_t rows, int heads, int dim,
                  const Rotary& p, const int32_t* positions, hipStream_t st) {
    if (rows == 0) return PTQ_OK;
    const RotaryArgs r{p.freq, positions, p.n, p.magnitude};
    const int layout = pair_layout(p.n, p.interleaved);
    return dtype == PTQ_F32 ? launch_layout((const float*)X, ldx, (float*)Y, ldy, rows, heads, dim, r, layout, st)
                            : launch_layout((const uint16_t*)X, ldx, (uint16_t*)Y, ldy, rows, heads, dim, r, layout, st);
}

}  // namespace ptq
