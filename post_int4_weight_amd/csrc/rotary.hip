// Rotary positions on the heads of each token (arithmetic in rotary.hpp):
//   y_a = m (x_a cos t - x_b sin t), y_b = m (x_b cos t + x_a sin t),
//   t = position * frequency of the pair; channels past the pairs are copied.
//
// A thread takes 16 channels of a token, 8 pairs or 16 channels past them, in
// HEADS heads: the 8 sines and cosines (about 900 cycles a wave) are formed once
// and all loads go out before them. What bounds it is memory, and for a few
// tokens the launch.
#include "rotary.hpp"

namespace ptq {
namespace {

template <typename T>
struct ApplyArgs {
    RotaryArgs r;
    const T* X; int64_t ldx;
    T* Y; int64_t ldy;
    int64_t rows;
    int heads, dim;
    int turning, items;       // items of a token that turn, and all that are written
};

template <typename T, int LAYOUT, int HEADS>
__global__ __launch_bounds__(256) void rotary_kernel(ApplyArgs<T> a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / a.items;
    if (row >= a.rows) return;
    const int item = (int)(at % a.items), h0 = blockIdx.y * HEADS;
    const T* X = a.X + row * a.ldx + (int64_t)h0 * a.dim;
    T* Y = a.Y + row * a.ldy + (int64_t)h0 * a.dim;
    const bool turns = item < a.turning;
    // channels of the item: n_a of them from c_a on, n_b from c_b on (8, or fewer at the end)
    int i0 = 8 * item, c_a = i0, c_b = i0 + a.r.n, n_a = 8, n_b = 8;
    if (!turns || LAYOUT == PAIR_NEIGHBOURS) {
        c_a = LAYOUT == PAIR_NEIGHBOURS ? 16 * item : 2 * a.r.n + 16 * (item - a.turning);
        c_b = c_a + 8;
        if (LAYOUT == PAIR_ANY_HALVES) n_a = std::min(8, a.dim - c_a);
        n_b = std::max(0, std::min(8, a.dim - c_b));      // 0 or 8 where chunks are whole
    } else if (LAYOUT == PAIR_ANY_HALVES) {
        n_a = n_b = std::min(8, a.r.n - i0);
    }
    const int position = a.r.positions[row];
    if constexpr (LAYOUT == PAIR_ANY_HALVES) {
        for (int k = 0; k < n_a; ++k) {
            float c = 1.f, s = 0.f;
            if (turns) turn_of(position, a.r.freq[i0 + k], a.r.magnitude, c, s);
            for (int h = 0; h < HEADS && h0 + h < a.heads; ++h) {
                const T* x = X + h * a.dim;
                T* y = Y + h * a.dim;
                float u = load_as_float(x, c_a + k), v = k < n_b ? load_as_float(x, c_b + k) : 0.f;
                if (turns) turn_pair(u, v, c, s);
                store1(y + c_a + k, u);
                if (k < n_b) store1(y + c_b + k, v);
            }
        }
        return;
    } else {
        float x[HEADS][2][8];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const int64_t d = (int64_t)std::min(h, a.heads - 1 - h0) * a.dim;      // past the last head: that one again
            load8(X + d + c_a, x[h][0]);
            load8(X + d + (n_b ? c_b : c_a), x[h][1]);
        }
        if (turns) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (LAYOUT == PAIR_NEIGHBOURS && i0 + k >= a.r.n) break;
                float c, s;
                turn_of(position, a.r.freq[i0 + k], a.r.magnitude, c, s);
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    if constexpr (LAYOUT == PAIR_HALVES)
                        turn_pair(x[h][0][k], x[h][1][k], c, s);
                    else
                        turn_pair(x[h][k >> 2][2 * k & 7], x[h][k >> 2][(2 * k & 7) + 1], c, s);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            if (h0 + h >= a.heads) break;
            store8(Y + h * a.dim + c_a, x[h][0]);
            if (n_b) store8(Y + h * a.dim + c_b, x[h][1]);
        }
    }
}

template <typename T, int LAYOUT>
int launch(const ApplyArgs<T>& a, hipStream_t st) {
    constexpr int MANY = 4;
    const int64_t threads = cdiv(a.rows * a.items, 256) * 256;
    const bool few = threads * cdiv(a.heads, MANY) < 256 * 1024;      // not one wave for each SIMD
    const int64_t groups = few ? a.heads : cdiv(a.heads, MANY);
    // a launch of 2^32 threads or more wraps without an error
    if (threads > (((int64_t)1 << 32) - 1) / groups) {
        set_error("rotary_apply: rows = %lld with %d heads of %d channels are too many for a launch", (long long)a.rows,
                  a.heads, a.dim);
        return PTQ_EINVAL;
    }
    const dim3 grid((unsigned)(threads / 256), (unsigned)groups);
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
    ApplyArgs<T> a{r, X, ldx, Y, ldy, rows, heads, dim, 0, 0};
    a.turning = (int)cdiv(r.n, 8);
    a.items = in_place ? a.turning : (int)(layout == PAIR_NEIGHBOURS ? cdiv(dim, 16) : a.turning + cdiv(dim - 2 * r.n, 16));
    switch (layout) {
        case PAIR_HALVES: return launch<T, PAIR_HALVES>(a, st);
        case PAIR_NEIGHBOURS: return launch<T, PAIR_NEIGHBOURS>(a, st);
        default: return launch<T, PAIR_ANY_HALVES>(a, st);
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
