// Softmax attention of a ragged batch of queries over the int8 block cache
// (layout in kv_cache.hip):
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
//   k_j = S_k[block(j)] c_j,  v_j = S_v[block(j)] c'_j
//
// Arithmetic. Codes are exact in fp16, so both products run on the fp16
// matrix cores: q is scaled by a power of two that brings its largest element
// to [8, 16) (a bf16 q is then exact; an fp32 q is split into two fp16 terms),
// S_k and the softmax scale multiply the fp32 sums, and S_v multiplies the
// probabilities: w_j = p_j S_v[block(j)] / R in fp16 (two terms for fp32
// queries), R the row's running maximum of S_v over the blocks it attends to, so
// w_j <= p_j whatever the scales are, and a block that a window or the diagonal
// hides from a row, which may hold anything, has no part in the row's rounding.
// Sums, maxima and the output accumulate in fp32.
#include "attention.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace ptq {
namespace {

constexpr int TR = ATTN_ROWS;     // query rows (tokens x grouped heads) of a tile

struct AttnArgs {
    Ragged g;
    const int32_t* table; int64_t width;      // g.starts: the lengths
    int heads, kv_heads, group, dim, bs, bs_log2;
    int64_t num_blocks;
    const int8_t* k; const int8_t* v; const float* ks; const float* vs;
    const void* Q; int64_t ldq;
    void* O; int64_t ldo;
    float* lse;                    // [rows, heads] or null
    float scale2;                  // softmax scale * log2(e)
    int causal; int64_t window;
    const int32_t* parents;        // trees only
    int nsplit;
    float* part; float* part_lse;  // [nsplit][rows * heads][dim], [nsplit][rows * heads]
};

// One tile of query rows: flat rows f0 .. f0 + TR of sequence b, flat row =
// token * group + head within the group.
struct Tile {
    int b;
    int64_t off;           // first row (token) of the sequence
    int rows;              // flat rows of the sequence
    int f0;
    int64_t len;           // keys of the sequence
    int64_t pos0;          // position of the sequence's first query token
    int it0, it1;          // steps of TK tokens with a key that some row of the tile attends to
    int64_t lo_max, hi_min;   // steps within [lo_max, hi_min) need no mask
    int64_t hi;            // end of the keys any row attends to
    bool over;             // longer than its row of the table can hold: NaN
};

__device__ __forceinline__ int64_t row_lo(const AttnArgs& a, int64_t pos) {
    return a.window > 0 ? std::max<int64_t>(0, pos - a.window + 1) : 0;
}
__device__ __forceinline__ int64_t row_hi(const AttnArgs& a, int64_t pos, int64_t len) {
    return a.causal ? std::min<int64_t>(std::max<int64_t>(pos + 1, 0), len) : len;
}

__device__ __forceinline__ bool find_tile(const AttnArgs& a, int64_t unit, int tr, Tile& t) {
    const RaggedUnit u = ragged_find(a.g, unit, a.group, tr, 1);
    t.b = u.b;
    t.off = u.off;
    const int64_t n = u.rows, rows = n * a.group, f0 = u.local * tr;
    if (n <= 0 || f0 >= rows) return false;
    t.rows = (int)rows;
    t.f0 = (int)f0;
    t.len = std::max(u.start, 0);
    t.pos0 = t.len - n;
    t.over = t.len > a.width * a.bs;
    t.len = std::min<int64_t>(t.len, a.width * a.bs);
    const int64_t first = t.pos0 + f0 / a.group;
    const int64_t last = t.pos0 + std::min<int64_t>(f0 + tr - 1, rows - 1) / a.group;
    t.lo_max = row_lo(a, last);
    t.hi_min = row_hi(a, first, t.len);
    t.hi = row_hi(a, last, t.len);
    const int64_t lo = row_lo(a, first);
    t.it0 = (int)(lo / TK);
    t.it1 = t.hi > lo ? (int)((t.hi + TK - 1) / TK) : t.it0;
    return true;
}

// The same of a sequence whose last rows are the nodes of a tree: all see the keys before it (a window may hide the first),
// and what a row sees from hi_min on is in its line.
__device__ __forceinline__ bool find_tree_tile(const AttnArgs& a, int64_t unit, int tr, Tile& t) {
    const RaggedUnit u = find_longest_first(a.g, (unsigned)unit, a.group, tr);
    t.b = u.b;
    t.off = u.off;
    const int64_t n = u.rows, rows = n * a.group, f0 = u.local * tr;
    if (n <= 0 || f0 >= rows) return false;
    t.rows = (int)rows;
    t.f0 = (int)f0;
    t.len = std::max(u.start, 0);
    t.over = t.len > a.width * a.bs || t.len < n || n > NODES;
    t.pos0 = std::max<int64_t>(t.len - n, 0);
    t.lo_max = a.window > 0 ? std::max<int64_t>(0, t.pos0 + n - a.window) : 0;
    t.hi_min = t.pos0;
    t.hi = std::min(t.pos0 + std::min<int64_t>(f0 + tr - 1, rows - 1) / a.group + 1, t.len);
    const int64_t lo = a.window > 0 ? std::max<int64_t>(0, t.pos0 - a.window + 1) : 0;
    t.it0 = (int)(lo / TK);
    t.it1 = t.over ? t.it0 : (int)((t.hi + TK - 1) / TK);
    return true;
}

// Steps of a split of a tile of tr rows: an even share, but not so few that
// the start of a workgroup and the join would outweigh them.
constexpr int min_steps(int tr) { return tr == TR ? 8 : 4; }
__device__ __forceinline__ int split_steps(const Tile& t, int nsplit, int tr) {
    const int n = t.it1 - t.it0;
    return std::max(min_steps(tr), (n + nsplit - 1) / nsplit);
}

// One query row in fp16 terms: scaled by the power of two that brings its
// largest element to [8, 16), negated for a negative softmax scale (scores
// then grow with what the sums give). `at(c)`: first channel of fragment c.
// The row is shared by the lanes that differ in the bits from GROUP up.
// Returns the factor of the scores, in units of log2.
template <typename T, int NC, int GROUP, int NT, typename F>
__device__ __forceinline__ float load_query(const T* p, float scale2, f16x8 (&q)[NT][NC], F&& at) {
    float x[NC][8];
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        load8(p + at(c), x[c]);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[c][k]));
    }
#pragma unroll
    for (int o = GROUP; o < 64; o *= 2) m = fmaxf(m, __shfl_xor(m, o, 64));
    const int field = std::min(257 - (int)(__float_as_uint(m) >> 23), 253);
    const float up = __uint_as_float((uint32_t)field << 23);
    const float sign = scale2 < 0.f ? -up : up;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float y = x[c][k] * sign;
            q[0][c][k] = (_Float16)y;
            if constexpr (NT == 2) q[1][c][k] = (_Float16)(y - (float)q[0][c][k]);
        }
    return fabsf(scale2) * __uint_as_float((uint32_t)(254 - field) << 23);
}

// Few query rows, long caches: the scores are computed transposed,
// S^T = K Q^T (tokens x rows), so a lane ends up with 16 scores of one query
// row, and the probabilities are already the operand of O^T = V^T P^T: nothing
// goes through LDS but the join of the waves. The tokens of a step are dealt
// to operand rows so that lane group lg holds tokens 16 lg .. 16 lg + 15 (row r
// of score block t is token 16 (r / 4) + 4 t + r % 4): V comes as one
// 16-byte load per channel, and a lane's tokens lie in one block of the cache
// (its size is a multiple of 16), so a lane needs one S_k and one S_v a step.
// The waves of a workgroup take every NW-th step; block ids come a step early.
// What bounds it is memory: each step's 16 KB (D = 128) are requested at once,
// and the other waves of the CU work meanwhile: a SIMD holds four at D = 64 (111
// + 16 registers), two at 128 (159 + 32 of bf16, 175 + 32 of fp32 queries), one
// at 256 (256 + 76, 256 + 108), where nothing is in flight while it computes. 64
// sequences of 100 .. 16000 keys, 64 query heads on 8, D = 128: 227 us, 4.7
// TB/s. 16 sequences of 100 .. 4000 keys, 16 on 4, D = 256: 34 us, 2.0 TB/s.
template <int D>
struct StepCodes {
    uint4 k[4][D / 64], v[D / 16];
    float sk, sv;
};

//
// TREE: the queries are the nodes of trees of drafted tokens (attention_tree.hip).
template <typename T, int D, int NW, bool TREE>
__global__ __launch_bounds__(64 * NW) void attention_rows_kernel(AttnArgs a) {
    constexpr int NT = sizeof(T) == 4 ? 2 : 1;    // fp16 terms of q and of the probabilities
    constexpr int NC = D / 32;                    // 32-deep steps of q.k
    const int split = (int)(blockIdx.x % (unsigned)a.nsplit);
    const int64_t tile = blockIdx.x / (unsigned)a.nsplit;
    const int h = (int)(tile % a.kv_heads);
    Tile tl;
    if (!(TREE ? find_tree_tile(a, tile / a.kv_heads, TR, tl) : find_tile(a, tile / a.kv_heads, TR, tl))) return;
    const int per = split_steps(tl, a.nsplit, TR);
    const int s0 = tl.it0 + split * per, s1 = std::min(s0 + per, tl.it1);
    if (split > 0 && s0 >= s1) return;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int f = std::min(tl.f0 + li, tl.rows - 1);
    const int64_t token = tl.off + f / a.group;
    const int qh = h * a.group + f % a.group;
    const int64_t pos = tl.pos0 + f / a.group;
    int my_lo = 0, my_hi = 0;
    if constexpr (!TREE) my_lo = (int)row_lo(a, pos), my_hi = (int)row_hi(a, pos, tl.len);
    // lines of the tile's nodes, where this split has keys of the tree or a window asks for depths
    __shared__ TreeLines<TREE ? TR : 1> lines_of;
    const int first_node = tl.f0 / a.group;
    const bool lines = TREE && !tl.over && (a.window > 0 || (int64_t)s1 * TK > tl.pos0);
    constexpr int PN = (NODES + 64 * NW - 1) / (64 * NW);
    int up[PN];
    if constexpr (TREE)
        if (lines)
#pragma unroll
            for (int i = 0; i < PN; ++i)
                up[i] = a.parents[tl.off + std::min((int)threadIdx.x + 64 * NW * i, tl.rows / a.group - 1)];

    const int32_t* table = a.table + (int64_t)tl.b * a.width;
    const int64_t pool = (int64_t)a.bs * D, stride = (int64_t)a.kv_heads * pool;      // codes of a (block, head), of a block
    const int8_t* kp = a.k + (int64_t)h * pool;
    const int8_t* vp = a.v + (int64_t)h * pool;
    const int end = (int)tl.hi, bmask = a.bs - 1;
    const int kgrp = 16 * (li >> 2), vgrp = 16 * lg;      // this lane's tokens of a step: rows of K, columns of V
    // block of position p: one without a valid id, and positions past the keys, stand for some other block of the
    // pool, whose codes are as good as any (the scale says NaN, or the mask leaves them out)
    auto entry = [&](int p) { return table[std::min(p, end - 1) >> a.bs_log2]; };
    auto ok = [&](int id) { return (unsigned)id < (unsigned)a.num_blocks; };
    int idk = 0, idv = 0;                                 // of the step to load next
    auto ids = [&](int it) {
        idk = entry(it * TK + kgrp);
        idv = entry(it * TK + vgrp);
    };
    auto load = [&](int it, StepCodes<D>& c) {
        const int tk = it * TK + kgrp, tv = it * TK + vgrp;
        const int8_t* p = kp + (ok(idk) ? idk : 0) * stride + (((tk & bmask) + (li & 3)) * D + 16 * lg);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < D / 64; ++e) c.k[t][e] = *(const uint4*)(p + 4 * t * D + 64 * e);
        const int bv = ok(idv) ? idv : 0;
        const int8_t* q = vp + bv * stride + (li * a.bs + (tv & bmask));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) c.v[i] = *(const uint4*)(q + 16 * i * a.bs);
        const int64_t at = (int64_t)bv * a.kv_heads + h;
        c.sk = a.ks[at];
        c.sv = a.vs[at];
        if (!ok(idv)) c.sk = c.sv = __builtin_nanf("");
        if (TREE && !(c.sk < INFINITY)) c.sk = __builtin_nanf("");
        if (!(c.sv < INFINITY)) c.sv = __builtin_nanf("");     // times codes of one sign it would stay infinite
        if (tv >= end) c.sk = c.sv = 0.f;
    };

    // q: operand column li, channels 64 (c / 2) + 16 lg + 8 (c % 2) + 0..7 of step c
    f16x8 q[NT][NC];
    f32x4 acc[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float qs = 0.f, m = -INFINITY, l = tl.over ? __builtin_nanf("") : 0.f, R = 0.f, rcp_R = 0.f;

    auto work = [&](int it, const StepCodes<D>& c) {
        // scores
        f32x4 s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const f16x8 k0 = half8(c.k[t][e].x, c.k[t][e].y), k1 = half8(c.k[t][e].z, c.k[t][e].w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[n][2 * e], s[t], 0, 0, 0);
                    s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[n][2 * e + 1], s[t], 0, 0, 0);
                }
            }
        }
        const float ck = c.sk * qs;
        const int tv = it * TK + vgrp;
        const bool whole = it * TK >= tl.lo_max && (int64_t)it * TK + TK <= tl.hi_min;   // no row masks anything here
        const int r_lo = my_lo - tv, r_hi = my_hi - tv;
        uint32_t seen = 0xffffu;
        if constexpr (TREE)
            if (!whole) seen = seen16(lines_of.line[f / a.group - first_node], tv, (int)tl.pos0, my_lo);
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = s[t][i] * ck;
                if (TREE ? !(seen >> (4 * t + i) & 1) : !whole && (4 * t + i < r_lo || 4 * t + i >= r_hi)) x = -INFINITY;
                s[t][i] = x;
                top = fmaxf(top, x);
            }
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // R: largest finite S_v of the row's blocks so far
        float big = c.sv < INFINITY && (TREE ? seen != 0 : whole || (r_lo < 16 && r_hi > 0)) ? c.sv : 0.f;
        big = fmaxf(big, __shfl_xor(big, 16, 64));
        big = fmaxf(big, __shfl_xor(big, 32, 64));
        if (__any(top > m + LAZY || big > R)) {
            const float m_new = !TREE || top > m + LAZY ? fmaxf(m, top) : m;      // a tree's rows each by itself
            float fall = m_new == m ? 1.f : exp2_fast(m - m_new);
            m = m_new;
            l *= fall;
            if (big > R) {
                rcp_R = big < FLT_MIN ? 0.f : __fdiv_rn(1.f, big);
                fall *= R * rcp_R;
                R = big;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] *= fall;
        }
        const float m_sub = (m == -INFINITY ? 0.f : m) - PSHIFT, rv = c.sv * rcp_R;
        f16x8 w[NT][2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float p0 = exp2_fast(s[t][i] - m_sub), p1 = exp2_fast(s[t][i + 1] - m_sub);
                l += p0;
                l += p1;
                f32x2 y = {p0 * rv, p1 * rv};
                if (!whole) {      // S_v of a block that is not this row's may be NaN
                    if (TREE ? !(seen >> (4 * t + i) & 1) : 4 * t + i < r_lo || 4 * t + i >= r_hi) y[0] = 0.f;
                    if (TREE ? !(seen >> (4 * t + i + 1) & 1) : 4 * t + i + 1 < r_lo || 4 * t + i + 1 >= r_hi) y[1] = 0.f;
                }
                const f16x2 x = __builtin_convertvector(y, f16x2);
                const int e = 4 * (t & 1) + i;
                w[0][t >> 1][e] = x[0];
                w[0][t >> 1][e + 1] = x[1];
                if constexpr (NT == 2) {
                    const f16x2 z = __builtin_convertvector((f32x2{y[0] - (float)x[0], y[1] - (float)x[1]}), f16x2);
                    w[1][t >> 1][e] = z[0];
                    w[1][t >> 1][e + 1] = z[1];
                }
            }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const f16x8 v0 = half8(c.v[i].x, c.v[i].y), v1 = half8(c.v[i].z, c.v[i].w);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[n][0], acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[n][1], acc[i], 0, 0, 0);
            }
        }
    };

    int it = s0 + wave;
    if (it < s1) ids(it);
    constexpr bool EARLY = TREE && D <= 128;      // the first keys are on their way while lines are built
    StepCodes<D> first;
    if constexpr (EARLY)
        if (it < s1) load(it, first);
    qs = load_query<T, NC, 16>((const T*)a.Q + token * a.ldq + (int64_t)qh * D, a.scale2, q,
                               [&](int c) { return 64 * (c / 2) + 16 * lg + 8 * (c % 2); });
    if constexpr (TREE)
        if (lines) {
            const int count = std::min(tl.f0 + TR - 1, tl.rows - 1) / a.group - first_node + 1;
            build_lines<64 * NW>(lines_of, up, tl.rows / a.group, first_node, count, a.window, (int)threadIdx.x);
            const int depth = lines_of.level[f / a.group - first_node];
            if (depth < 0) l = __builtin_nanf("");
            my_lo = first_key((int)tl.pos0, depth, a.window);
        }
    if constexpr (EARLY)
        if (it < s1) {
            if (it + NW < s1) ids(it + NW);
            work(it, first);
            it += NW;
        }
    for (; it < s1; it += NW) {
        StepCodes<D> c;
        load(it, c);
        if (it + NW < s1) ids(it + NW);
        work(it, c);
    }

    // join the waves: factors to the common maximum, then sums through LDS
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    __shared__ float sm[NW][TR], sl[NW][TR];
    constexpr int DP = D * NW <= 512 ? D : 512 / NW;      // channels that go through LDS at a time
    __shared__ __attribute__((aligned(16))) float so[NW][TR][DP + 4];
    if (lg == 0) {
        sm[wave][li] = m;
        sl[wave][li] = l;
    }
    __syncthreads();
    float M = sm[0][li];
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w][li]);
    const float M0 = M == -INFINITY ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) L += sl[w][li] * exp2_fast(sm[w][li] - M0);
    const float mine = (R > 0.f ? R : 1.f) * exp2_fast(m - M0) / (L == 0.f ? 1.f : L);
    const bool split_out = a.nsplit > 1;
    const int64_t nflat = a.g.rows * a.heads;
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DP) {
        if (d0) __syncthreads();
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            const f32x4 x = acc[d0 / 16 + i];
            *(f32x4*)&so[wave][li][16 * i + 4 * lg] = f32x4{x[0] * mine, x[1] * mine, x[2] * mine, x[3] * mine};
        }
        __syncthreads();
        for (int c = threadIdx.x; c < TR * (DP / 4); c += 64 * NW) {
            const int r = c / (DP / 4), d = 4 * (c % (DP / 4)), fr = tl.f0 + r;
            if (fr >= tl.rows) continue;
            f32x4 o = *(const f32x4*)&so[0][r][d];
#pragma unroll
            for (int w = 1; w < NW; ++w) o += *(const f32x4*)&so[w][r][d];
            const int64_t row = tl.off + fr / a.group;
            const int head = h * a.group + fr % a.group;
            if (split_out)
                *(f32x4*)(a.part + (split * nflat + row * a.heads + head) * D + d0 + d) = o;
            else
                store4((T*)a.O + row * a.ldo + (int64_t)head * D + d0 + d, o[0], o[1], o[2], o[3]);
        }
    }
    if (wave == 0 && lg == 0 && tl.f0 + li < tl.rows && (split_out || a.lse)) {
        // L carries 2^PSHIFT
        const float lse2 = L == 0.f ? -INFINITY : M0 - PSHIFT + __log2f(L);
        const int64_t at = token * a.heads + qh;
        if (split_out)
            a.part_lse[split * nflat + at] = lse2;
        else
            a.lse[at] = lse2 * 0.6931471805599453f;
    }
}

// Many query rows: 32 rows a wave, WAVES waves on the same keys. K and V go
// through LDS once per workgroup, converted to fp16 on the way (a wave that
// converted its own operands would spend more on that than on the products).
// S^T = K Q^T and O^T = V^T P^T as above, on 32x32x16 products: operand row r
// of a block of 32 tokens is token 16 (r / 4 % 2) + 4 (r / 8) + r % 4, so lane
// half hf holds tokens 16 hf .. 16 hf + 15, again in one block of the cache:
// one S_k and one S_v per lane and score block, which go into the exponent,
// w = 2^(s ck - m + log2 rv), and the sum of p takes 1 / rv once per 16 values.
//
// What bounds it (D = 128): a product holds the SIMD's vector pipe for 24 of its
// 32 cycles' worth, so products and the 8 vector instructions that go with each
// of them (scale, exponential, sum, rounding of its share of probabilities,
// maxima, conversion of the codes) come to about 40 cycles, and the fragment a
// product reads takes LDS another 32. All three being near, a wave must never
// wait with only one other on its SIMD: three blocks are in work at a time, the
// products give the scores of block n + 1 and the output of block n - 1 while
// the exponentials of block n run between them, and everything else of a step
// (fetching and staging the next ones, its only barrier, the head of the next
// block) lies between products, too. A fragment is read AHEAD products early.
// Measured, 4 prompts of 2000 .. 4096 tokens over 5000 keys, 32 query heads on
// 8: 661 .. 691 us on three cards, about 42% of the matrix cycles; phases one
// after the other were 785 where this order was 652. 64
// rows a wave halve the LDS reads, but then one wave a SIMD has to issue
// everything, and a sixth more of it to move accumulators between register
// files: 917 us against 773 on the same card. Fragments 6 products early, or
// wave priorities, change it by 1%.
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {      // f(integral_constant<int, I>) for I = B .. E - 1, in order
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// x is computed here: without this the compiler moves the sums and maxima of a
// block behind its products, and every probability stays in a register till then
__device__ __forceinline__ void pin(float& x) { asm volatile("" : "+v"(x)); }

template <int QUAD_PERM>
__device__ __forceinline__ float swap_lanes(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), QUAD_PERM, 0xf, 0xf, true));
}

// Rows of K are in the order of the operand's rows, and 16 bytes longer than
// their values: 16 neighbours touch every bank, and an operand fragment is one
// lane address and a constant.
template <int D>
struct TileLds {
    static constexpr int KROW = 2 * D + 16, VROW = 2 * TK + 16;       // bytes of a token of K, of a channel of V
    static constexpr int K_BYTES = TK * KROW, V_BYTES = D * VROW;
    static constexpr int V_AT = 2 * K_BYTES, BYTES = V_AT + 3 * V_BYTES;
    // operand row of a token of a step
    __host__ __device__ static constexpr int k_row(int token) {
        return (token & ~31) | (token >> 2 & 3) << 3 | (token >> 4 & 1) << 2 | (token & 3);
    }
};

//
// TREE: the queries are the nodes of trees of drafted tokens (attention_tree.hip);
// steps with keys of the tree take their masks from the nodes' lines.
template <typename T, int D, int WAVES, bool TREE>
__global__ __launch_bounds__(64 * WAVES) void attention_tile_kernel(AttnArgs a) {
    constexpr int NT = sizeof(T) == 4 ? 2 : 1;
    constexpr bool PIPE = NT == 1;                 // two terms of everything would not fit the registers
    constexpr int AHEAD = 3;
    constexpr int NTH = 64 * WAVES, NC = D / 16, ND = D / 32;
    constexpr int NCH = TK * D / 16;               // 16-byte chunks of K, and of V, in a step
    static_assert(NCH % 64 == 0 && NCH <= NTH, "one chunk of each a thread");
    using L = TileLds<D>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    // of step it, at (it - s0) % 4: S_k of the lane half's group in either block, then log2 S_v of them (NaN: S_v is
    // not finite); the largest finite S_v, negative if one is not finite
    __shared__ __attribute__((aligned(16))) float ssc[4][2][4], sbig[4];
    __shared__ float ssv[4][2][2];      // S_v of them, 0 if it is not finite

    const int split = (int)(blockIdx.x % (unsigned)a.nsplit);
    const int64_t tile = blockIdx.x / (unsigned)a.nsplit;
    const int h = (int)(tile % a.kv_heads);
    Tile tl;
    // later tiles of a sequence have more keys: they go first
    const int64_t unit = TREE ? tile / a.kv_heads : gridDim.x / (unsigned)a.nsplit / a.kv_heads - 1 - tile / a.kv_heads;
    if (!(TREE ? find_tree_tile(a, unit, 32 * WAVES, tl) : find_tile(a, unit, 32 * WAVES, tl))) return;
    const int per = split_steps(tl, a.nsplit, 32 * WAVES);
    const int s0 = __builtin_amdgcn_readfirstlane(tl.it0 + split * per);
    const int s1 = __builtin_amdgcn_readfirstlane(std::min(s0 + per, tl.it1));
    if (split > 0 && s0 >= s1) return;

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int li = lane & 31, hf = lane >> 5;
    const bool idle = tl.f0 + 32 * wave >= tl.rows;     // no row of this wave: it only helps staging
    const int f = std::min(tl.f0 + 32 * wave + li, tl.rows - 1);
    const int64_t token = tl.off + f / a.group;
    const int qh = h * a.group + f % a.group;
    const int64_t pos = tl.pos0 + f / a.group;
    // keys of this lane's row (of a tree's node: the first, and the end of those before the tree); the wave's rows have
    // none from w_max on
    int my_lo = 0, my_hi = (int)tl.pos0;
    bool broken = tl.over;
    const int first_node = tl.f0 / a.group;
    __shared__ TreeLines<TREE ? 32 * WAVES : 1> lines_of;
    if constexpr (TREE) {
        if (!tl.over && (a.window > 0 || (int64_t)s1 * TK > tl.pos0)) {
            const int n = tl.rows / a.group;
            int up[1];
            static_assert(NODES <= NTH, "a node a thread");
            up[0] = a.parents[tl.off + std::min(t, n - 1)];
            const int count = std::min(tl.f0 + 32 * WAVES - 1, tl.rows - 1) / a.group - first_node + 1;
            build_lines<NTH>(lines_of, up, n, first_node, count, a.window, t);
            const int depth = lines_of.level[f / a.group - first_node];
            broken = depth < 0;
            my_lo = first_key((int)tl.pos0, depth, a.window);
        }
    } else {
        my_lo = (int)row_lo(a, pos), my_hi = (int)row_hi(a, pos, tl.len);
    }
    const int fb = std::min(tl.f0 + 32 * wave + 31, tl.rows - 1);
    const int64_t last_pos = tl.pos0 + fb / a.group;
    const int w_max = idle ? 0 : __builtin_amdgcn_readfirstlane((int)(TREE ? last_pos + 1 : row_hi(a, last_pos, tl.len)));

    f16x8 q[NT][NC];
    const float qs = load_query<T, NC, 32>((const T*)a.Q + token * a.ldq + (int64_t)qh * D, a.scale2, q,
                                           [&](int c) { return 16 * c + 8 * hf; });

    f32x16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    // ref, limit: what m comes down to for the exponents, the score from which it moves
    float m = -INFINITY, ref = -PSHIFT, limit = -INFINITY, l = broken ? __builtin_nanf("") : 0.f;
    float R = 0.f, log2_R = 0.f, poison = 0.f;

    // Staging: one 16-byte chunk of K (16 channels of a token) and one of V (16 tokens of a channel) per thread and
    // step. A wave's chunks lie in one block of the cache, of K because its tokens are neighbours, of V by the way the
    // chunks are dealt: gpr = chunks of a channel that are neighbours in a block. So ids and addresses of blocks are
    // scalar. The ids of a step's four groups are requested a step before the codes they lead to, in lanes 0 .. 3 of
    // every quad, and looked at only then: a wait in between would wait for the codes requested before them, too.
    const int32_t* table = a.table + (int64_t)tl.b * a.width;
    const int64_t pool = (int64_t)a.bs * D, stride = (int64_t)a.kv_heads * pool;
    const int8_t* kp = a.k + (int64_t)h * pool;
    const int8_t* vp = a.v + (int64_t)h * pool;
    const int end = __builtin_amdgcn_readfirstlane((int)tl.hi), bmask = a.bs - 1;
    const bool stages = NCH >= NTH || wave < NCH / 64;       // waves past the chunks have none
    const int ktok = t / (D / 16), gpr = std::min(a.bs, TK) / 16, nblk = 4 / gpr;
    const int vblk = wave % nblk, vd = (wave / nblk) * (64 / gpr) + lane / gpr, vgrp = vblk * gpr + lane % gpr;
    const unsigned koff = (unsigned)((ktok & bmask) * D + 16 * (t % (D / 16)));
    const unsigned voff = (unsigned)(vd * a.bs + ((16 * vgrp) & bmask));
    const int kgrp = wave * 64 / (D / 16) / 16 % 4, vfirst = vblk * gpr;      // a group of the wave's chunks' block
    auto entries = [&](int it) {
        const unsigned p = std::min((unsigned)it * TK + 16 * (lane & 3), (unsigned)end - 1);     // it is past the end, too
        return *(const int32_t*)((const char*)table + (p >> a.bs_log2 << 2));
    };
    // a block without a valid id, and positions past the keys, stand for some other block of the pool, whose codes
    // are as good as any (the scale says NaN, or the mask leaves them out)
    auto valid = [&](int id) { return (unsigned)id < (unsigned)a.num_blocks ? id : 0; };
    auto base = [&](const int8_t* from, int ids, int group) {
        return from + (int64_t)valid(__builtin_amdgcn_readlane(ids, group)) * stride;
    };
    int ids2 = 0, ids3 = 0;         // of steps it + 2, it + 3
    uint4 rk, rv_;
    float sk_r, sv_r;
    auto fetch_k = [&](int it, int ids) {
        if (stages) rk = *(const uint4*)(base(kp, ids, kgrp) + ((it * TK) & bmask) * D + koff);
    };
    auto fetch_v = [&](int it, int ids) {
        if (stages) rv_ = *(const uint4*)(base(vp, ids, vfirst) + ((it * TK) & bmask) + voff);
    };
    auto fetch_scales = [&](int ids) {
        if (wave == 0) {
            const int64_t at = (int64_t)valid(ids) * a.kv_heads + h;
            sk_r = a.ks[at];
            sv_r = a.vs[at];
        }
    };
    const int kto = L::k_row(ktok) * L::KROW + 32 * (t % (D / 16));
    const int vto = L::V_AT + vd * L::VROW + 32 * vgrp;
    auto stage_k = [&](int at, int half) {    // at: offset of the buffer
        if (stages) *(f16x8*)(smem + at + kto + 16 * half) = half ? half8(rk.z, rk.w) : half8(rk.x, rk.y);
    };
    auto stage_v = [&](int at, int half) {
        if (stages) *(f16x8*)(smem + at + vto + 16 * half) = half ? half8(rv_.z, rv_.w) : half8(rv_.x, rv_.y);
    };
    auto stage_scales = [&](int it, int ids) {
        if (wave == 0 && lane < 4) {
            const bool past = (unsigned)it * TK + 16 * lane >= (unsigned)end, known = (unsigned)ids < (unsigned)a.num_blocks;
            const float sk = past ? 0.f : known && (!TREE || sk_r < INFINITY) ? sk_r : __builtin_nanf("");
            const float sv = past || !known ? 0.f : sv_r;
            const bool bad = !(sv < INFINITY);
            float* to = ssc[(it - s0) & 3][lane & 1] + (lane >> 1);
            to[0] = sk;
            to[2] = bad ? __builtin_nanf("") : __builtin_amdgcn_logf(sv);     // v_log_f32: base 2
            float big = bad ? 0.f : sv;
            ssv[(it - s0) & 3][lane & 1][lane >> 1] = big;
            big = fmaxf(big, swap_lanes<0xB1>(big));        // quad_perm [1, 0, 3, 2]
            big = fmaxf(big, swap_lanes<0x4E>(big));        // quad_perm [2, 3, 0, 1]
            const bool any_bad = __ballot(bad) != 0;
            if (lane == 0) sbig[(it - s0) & 3] = any_bad ? -big : big;
        }
    };
    // buffers of K of this step and the next, of V of the last step, this one and the next
    int k0 = 0, k1 = L::K_BYTES, vm = 2 * L::V_BYTES, v0 = 0, v1 = L::V_BYTES;

    // operand fragments of this lane
    const int kfrom = li * L::KROW + 16 * hf, vfrom = L::V_AT + li * L::VROW + 32 * hf;
    auto k_frag = [&](int at, int u, int c) {       // tokens 32 u .., channels 16 c ..
        return *(const f16x8*)(smem + at + kfrom + 32 * u * L::KROW + 32 * c);
    };
    auto v_frag = [&](int at, int u, int j) {       // product j of a block: channels 32 (j % ND) .., tokens 16 hf + 8 (j / ND) ..
        return *(const f16x8*)(smem + at + vfrom + 32 * (j % ND) * L::VROW + 64 * u + 16 * (j / ND));
    };

    auto clear = [&](f32x16& x) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = 0.f;
    };
    auto top_of = [&](const f32x16& s, float& top, int r) {
        top = r ? fmaxf(fmaxf(top, s[r]), s[r + 1]) : fmaxf(s[0], s[1]);
        pin(top);
    };
    auto scores = [&](int at, int u, f32x16& s, float& top) __attribute__((always_inline)) {
        clear(s);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const f16x8 k = k_frag(at, u, c);
#pragma unroll
            for (int n = 0; n < NT; ++n) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[n][c], s, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 16; r += 2) top_of(s, top, r);
    };
    using Probs = f16x8[NT][2];
    auto output = [&](int at, int u, const Probs& w) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2 * ND; ++j) {
            const f16x8 v = v_frag(at, u, j);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[j % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[n][j / ND], acc[j % ND], 0, 0, 0);
        }
    };
    auto forget = [&](Probs& w) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) w[n][k][e] = (_Float16)0.f;
    };
    // A row moves to another reference when its largest score mx exceeds limit or S_v of a block it attends to exceeds R.
    // What was pending at the old references is in acc already. Blocks that all rows attend to are compared with all_R, a
    // scalar that no row's R is below: with R itself the bf16 kernel spills 47 registers. As bits, so that a negative one
    // of sbig is large, too.
    unsigned all_R = 0;
    auto move = [&](float mx, float big) __attribute__((always_inline)) {
        const float m_new = !TREE || mx > limit ? fmaxf(m, mx) : m;      // a tree's rows each by itself
        float fall = m_new == m ? 1.f : exp2_fast(m - m_new);
        m = m_new;
        ref = (m == -INFINITY ? 0.f : m) - PSHIFT;
        limit = m + LAZY;
        l *= fall;
        if (big > R) {
            fall *= big < FLT_MIN ? 0.f : __fdiv_rn(R, big);
            R = big;
            log2_R = big < FLT_MIN ? 0.f : __builtin_amdgcn_logf(big);
        }
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][r] *= fall;
    };
    auto scales_of = [&](int it) { return *(const f32x4*)ssc[(it - s0) & 3][hf]; };
    auto big_of = [&](int it) { return sbig[(it - s0) & 3]; };
    auto bits = [](float big) { return (unsigned)__builtin_amdgcn_readfirstlane(__float_as_uint(big)); };
    auto log2_rv = [&](float log2_sv) { return fmaxf(log2_sv - log2_R, LOG2_RV_MIN); };      // of NaN, too
    // two probabilities of block (it, u), into w and sum; in(r): whether the row attends to key r of the lane's 16
    auto pair = [&](auto masked, const f32x16& s, float ck, float off, int r, Probs& w, float& sum, auto&& in) {
        f32x2 e;
        e[0] = exp2_fast(fmaf(s[r], ck, -off));
        e[1] = exp2_fast(fmaf(s[r + 1], ck, -off));
        if constexpr (decltype(masked)::value) {     // S_v of a block that is not this row's may be NaN
            if (!in(r)) e[0] = 0.f;
            if (!in(r + 1)) e[1] = 0.f;
        }
        sum += e[0];
        sum += e[1];
        pin(sum);
        const f16x2 x = __builtin_convertvector(e, f16x2);
        w[0][r >> 3][r & 7] = x[0];
        w[0][r >> 3][(r & 7) + 1] = x[1];
        if constexpr (NT == 2) {
            const f32x2 rest = {e[0] - (float)x[0], e[1] - (float)x[1]};
            const f16x2 y = __builtin_convertvector(rest, f16x2);
            w[1][r >> 3][r & 7] = y[0];
            w[1][r >> 3][(r & 7) + 1] = y[1];
        }
    };

    // one block by itself: steps that some row of the tile masks, and fp32 queries
    auto plain_block = [&](auto masked, int it, int u) __attribute__((always_inline)) {
        f32x16 s;
        float top;
        scores(k0, u, s, top);
        const f32x4 sc = scales_of(it);
        float ck = sc[u] * qs;
        const int g0 = it * TK + 32 * u + 16 * hf, lo = my_lo - g0, hi = my_hi - g0;
        uint32_t seen = 0;
        if constexpr (TREE && decltype(masked)::value)
            seen = seen16(lines_of.line[f / a.group - first_node], g0, (int)tl.pos0, my_lo);
        auto in = [&](int r) { return TREE ? (seen >> r & 1) != 0 : r >= lo && r < hi; };
        if constexpr (decltype(masked)::value) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = in(r) ? s[r] * ck : -INFINITY;
            ck = 1.f;
#pragma unroll
            for (int r = 0; r < 16; r += 2) top_of(s, top, r);
        }
        const float mx = max_halves(top * ck);
        const bool mine = !decltype(masked)::value || (TREE ? seen != 0 : lo < 16 && hi > 0);
        const float big = max_halves(mine ? ssv[(it - s0) & 3][hf][u] : 0.f);
        if (__any(mx > limit || big > R)) move(mx, big);
        if (mine && sc[2 + u] != sc[2 + u]) poison = sc[2 + u];
        const float lr = log2_rv(sc[2 + u]), off = ref - lr;
        Probs w;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 16; r += 2) pair(masked, s, ck, off, r, w, sum, in);
        l += sum * exp2_fast(-lr);
        output(v0, u, w);
    };
    // What a block needs to know before its exponentials: S_k, the largest score of each row, whether a row has to move
    struct Head {
        float ck, mx, lr, off;
        unsigned big;
        bool moves;
    };
    auto head_of = [&](float sk, float lv, unsigned big, float top, bool first) {
        Head h;
        h.ck = sk * qs;
        h.mx = max_halves(top * h.ck);
        h.big = big;
        h.moves = (first && big > all_R) || __any(h.mx > limit);      // S_v's are the step's
        h.lr = log2_rv(lv);
        h.off = ref - h.lr;
        return h;
    };
    // Block u of a step with scales sc, scores s and head h, next to the scores of the block after it (K at nk, block nu;
    // into sn, topn) and the output of the block before it (V at pv, block pu, probabilities wp); its own go to w. pre:
    // the first fragments, then those of the block after (K at nk2, block nu2). at_slot: what else goes between products
    // head: of the next block, once its maxima are known
    auto piped_block = [&](auto uc, const f32x4& sc, Head& h, const f32x16& s, f32x16& sn, f16x8 (&pre)[AHEAD], int nk, int nu,
                           int pv, int pu, int nk2, int nu2, Probs& wp, Probs& w, auto at_slot,
                           auto next_head) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value, N = NC + 2 * ND, PER = 16 / N;      // values a product
        if (h.moves) {
            output(pv, pu, wp);
            forget(wp);
            move(h.mx, fabsf(__uint_as_float(h.big)));
            all_R = std::max(all_R, h.big & 0x7fffffffu);
            if (u == 0 && sc[2] + sc[3] != sc[2] + sc[3]) poison = __builtin_nanf("");
            h.lr = log2_rv(sc[2 + u]);
            h.off = ref - h.lr;
        }
        f16x8 fr[N];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) fr[j] = pre[j];
        float sum = 0.f, topn = 0.f, e[16];
        auto add_up = [&](auto jc) {           // values PER j .. of the last slot
            constexpr int r0 = PER * decltype(jc)::value;
#pragma unroll
            for (int r = r0; r < r0 + PER; ++r) {
                sum = r ? sum + e[r] : e[r];
                if (r & 1) {
                    const f16x2 x = __builtin_convertvector((f32x2{e[r - 1], e[r]}), f16x2);
                    w[0][r >> 3][(r & 7) - 1] = x[0];
                    w[0][r >> 3][r & 7] = x[1];
                }
            }
            pin(sum);
        };
        static_for<0, N>([&](auto jc) {
            constexpr int j = decltype(jc)::value, J = j + AHEAD;
            if constexpr (J < NC) fr[J] = k_frag(nk, nu, J);
            else if constexpr (J < N) fr[J] = v_frag(pv, pu, J - NC);
            else pre[J - N] = k_frag(nk2, nu2, J - N);
            if constexpr (j == 0) clear(sn);
            if constexpr (j < NC) {
                sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[j], q[0][j], sn, 0, 0, 0);
            } else {
                constexpr int i = (j - NC) % ND, k = (j - NC) / ND;
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[j], wp[0][k], acc[i], 0, 0, 0);
            }
#pragma unroll
            for (int r = PER * j; r < PER * (j + 1); ++r) e[r] = exp2_fast(fmaf(s[r], h.ck, -h.off));
            if constexpr (j > 0) add_up(std::integral_constant<int, j - 1>{});
            at_slot(jc);
            // the new scores are complete a product after their last one
            constexpr int FROM = NC + 1, LAST = N - 2;
            if constexpr (j >= FROM && j < LAST)
                static_for<8 * (j - FROM) / (LAST - FROM), 8 * (j + 1 - FROM) / (LAST - FROM)>([&](auto pc) {
                    top_of(sn, topn, 2 * decltype(pc)::value);
                });
            if constexpr (j == N - 1) {
                add_up(jc);
                l += sum * exp2_fast(-h.lr);
                h = next_head(topn);
            }
        });
    };

    if (s0 < s1) {
        const int ids0 = entries(s0), ids1 = entries(s0 + 1);
        fetch_k(s0, ids0);
        fetch_v(s0, ids0);
        fetch_scales(ids0);
        for (int half : {0, 1}) {
            stage_k(k0, half);
            stage_v(v0, half);
        }
        stage_scales(s0, ids0);
        fetch_k(s0 + 1, ids1);
        fetch_scales(ids1);
        for (int half : {0, 1}) stage_k(k1, half);
        stage_scales(s0 + 1, ids1);
        // what a step finds: K of it and it + 1, V of it, scales of it and it + 1 in LDS; K of it + 2, V of it + 1 and
        // scales of it + 2 on their way (past the last step: of some block, into a buffer that nobody reads)
        ids2 = entries(s0 + 2);
        ids3 = entries(s0 + 3);
        fetch_k(s0 + 2, ids2);
        fetch_v(s0 + 1, ids1);
        fetch_scales(ids2);
        __syncthreads();
        auto next_scales = [&](int it) {
            stage_scales(it + 2, ids2);
            fetch_scales(ids3);
        };
        auto next_ids = [&](int it) {
            ids2 = ids3;
            ids3 = entries(it + 4);
        };
        auto rotate = [&] {
            const int k = k0, v = vm;
            k0 = k1;
            k1 = k;
            vm = v0;
            v0 = v1;
            v1 = v;
        };
        auto plain_step = [&](auto masked, int it) __attribute__((always_inline)) {
            for (int half : {0, 1}) stage_v(v1, half);
            fetch_v(it + 2, ids2);
            if (!decltype(masked)::value || it * TK < w_max) {
                plain_block(masked, it, 0);
                plain_block(masked, it, 1);
            }
            __syncthreads();
            for (int half : {0, 1}) stage_k(k0, half);
            fetch_k(it + 3, ids3);
            next_scales(it);
            next_ids(it);
            rotate();
        };
        // steps that some row of the tile masks (the start of windows, the diagonal) go through loops of their own
        int it = s0;
        const int whole = std::min(__builtin_amdgcn_readfirstlane((int)((tl.lo_max + TK - 1) / TK)), s1);
        const int last = std::min(__builtin_amdgcn_readfirstlane((int)(tl.hi_min / TK)), s1);
        for (; it < whole; ++it) plain_step(std::true_type{}, it);
        if constexpr (PIPE) {
            if (it < last) {
                f32x16 sa, sb;
                f16x8 pre[AHEAD];
                Probs wa, wb;
                float top;
                scores(k0, 0, sa, top);
                forget(wb);
                int pv = v0;        // nothing before the first block: zero probabilities on any V that is there
                f32x4 sc = scales_of(it), sc_next;
                float big_next;
                Head h = head_of(sc[0], sc[2], bits(big_of(it)), top, true);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) pre[j] = k_frag(k0, 1, j);
                for (; it < last; ++it) {
                    // K of this step is not read after product NC - 1, what the last step staged is not before the last
                    // AHEAD products: the barrier goes in between. Past the first slot a wave reads NC more fragments up
                    // to there, all but the last AHEAD of them for products that are issued: with at most AHEAD accesses
                    // to LDS open, and those in order, what it staged has landed and what others may overwrite is read.
                    // (Waiting for all of them, 64 channels: 459 us against 451.)
                    static_assert(NC >= AHEAD, "fragments read between a step's staging and the barrier");
                    piped_block(std::integral_constant<int, 0>{}, sc, h, sa, sb, pre, k0, 1, pv, 1, k1, 0, wb, wa,
                        [&](auto slot) {
                            if constexpr (decltype(slot)::value == 0) __builtin_amdgcn_sched_barrier(0);
                            if constexpr (decltype(slot)::value == NC) {
                                asm volatile("" ::: "memory");
                                __builtin_amdgcn_sched_barrier(0);
                                __builtin_amdgcn_s_waitcnt(0xc07f | AHEAD << 8);      // lgkmcnt
                                __builtin_amdgcn_s_barrier();
                                __builtin_amdgcn_sched_barrier(0);
                                asm volatile("" ::: "memory");
                            }
                        },
                        [&](float topn) { return head_of(sc[1], sc[3], 0, topn, false); });
                    piped_block(std::integral_constant<int, 1>{}, sc, h, sb, sa, pre, k1, 0, v0, 0, k1, 1, wa, wb,
                        [&](auto slot) {
                            constexpr int j = decltype(slot)::value * 16 / (NC + 2 * ND);       // of 16, or every second
                            if constexpr (j == 0) {
                                sc_next = scales_of(it + 1);
                                big_next = big_of(it + 1);
                            }
                            if constexpr (j == 2) stage_k(k0, 0);
                            if constexpr (j == 4) stage_k(k0, 1), fetch_k(it + 3, ids3);
                            if constexpr (j == 6) stage_v(v1, 0);
                            if constexpr (j == 8) stage_v(v1, 1), fetch_v(it + 2, ids2);
                            if constexpr (j == 10) next_scales(it);
                            if constexpr (j == 12) next_ids(it);
                        },
                        [&](float topn) { return head_of(sc_next[0], sc_next[2], bits(big_next), topn, true); });
                    sc = sc_next;
                    rotate();
                    pv = vm;
                }
                output(pv, 1, wb);
                __syncthreads();
            }
        } else {
            for (; it < last; ++it) plain_step(std::false_type{}, it);
        }
        for (; it < s1; ++it) plain_step(std::true_type{}, it);
    }
    if (idle) return;

    l += __shfl_xor(l, 32, 64);
    if (tl.f0 + 32 * wave + li >= tl.rows) return;
    poison += __shfl_xor(poison, 32, 64);
    const float mine = (R > 0.f ? R : 1.f) / (l == 0.f ? 1.f : l) + poison;
    const bool split_out = a.nsplit > 1;
    const int64_t nflat = a.g.rows * a.heads, at = token * a.heads + qh;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int d = 32 * i + 8 * b + 4 * hf;
            const f32x4 o = {acc[i][4 * b] * mine, acc[i][4 * b + 1] * mine, acc[i][4 * b + 2] * mine,
                             acc[i][4 * b + 3] * mine};
            if (split_out)
                *(f32x4*)(a.part + (split * nflat + at) * D + d) = o;
            else
                store4((T*)a.O + token * a.ldo + (int64_t)qh * D + d, o[0], o[1], o[2], o[3]);
        }
    if (hf == 0 && (split_out || a.lse)) {
        const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) - PSHIFT + __log2f(l);
        if (split_out)
            a.part_lse[split * nflat + at] = lse2;
        else
            a.lse[at] = lse2 * 0.6931471805599453f;
    }
}

// Join of the splits: 16 rows a workgroup, 16 threads a row; tr: rows of the
// tiles that were split. A join that reads one split after the other waits for
// memory each time: 1 query over 16000 keys, 63 splits, 47.8 us in all, 21.8
// with JB splits at a time.
template <typename T, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int tr) {
    const int64_t part = blockIdx.x % (unsigned)(tr / TR), tile = blockIdx.x / (unsigned)(tr / TR);
    const int h = (int)(tile % a.kv_heads);
    Tile tl;
    if (!find_tile(a, tile / a.kv_heads, tr, tl)) return;
    const int per = split_steps(tl, a.nsplit, tr);
    const int n = std::max(1, (tl.it1 - tl.it0 + per - 1) / per);    // split 0 is always written
    const int r = threadIdx.x / 16, c = threadIdx.x % 16, f = tl.f0 + (int)part * TR + r;
    if (f >= tl.rows) return;
    const int64_t row = tl.off + f / a.group, nflat = a.g.rows * a.heads;
    const int head = h * a.group + f % a.group;
    const int64_t at = row * a.heads + head;
    // JB splits at a time, all their loads at once
    constexpr int JB = 8;
    float M = -INFINITY, M0 = 0.f, L = 0.f;
    f32x4 o[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < n; s += JB) {
        float lse[JB];
        f32x4 v[JB][D / 64];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int64_t from = std::min(s + j, n - 1) * nflat + at;
            lse[j] = s + j < n ? a.part_lse[from] : -INFINITY;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) v[j][i] = *(const f32x4*)(a.part + from * D + 64 * i + 4 * c);
        }
        const float before = M;
#pragma unroll
        for (int j = 0; j < JB; ++j) M = fmaxf(M, lse[j]);
        M0 = M == -INFINITY ? 0.f : M;
        const float fall = exp2_fast(before - M0);
        L *= fall;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) o[i] *= fall;
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const float w = exp2_fast(lse[j] - M0);
            L += w;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) o[i] += (s + j < n ? w : 0.f) * v[j][i];
        }
    }
    const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        store4((T*)a.O + row * a.ldo + (int64_t)head * D + 64 * i + 4 * c, o[i][0] * inv, o[i][1] * inv,
                   o[i][2] * inv, o[i][3] * inv);
    if (a.lse && c == 0) a.lse[at] = L == 0.f ? -INFINITY : (M0 + __log2f(L)) * 0.6931471805599453f;
}

int64_t tile_units(int64_t rows, int64_t batch, int group, int tr) { return rows * group / tr + batch; }

// Waves of a tile: two per SIMD. At 256 channels the output and query
// fragments of 32 rows leave no registers for the rest: those go through
// attention_rows_kernel whatever the number of rows.
constexpr int TILE_WAVES = ATTN_TILE / 32;

// The choice of an AttnPlan. Lengths are not known here: keys is the most there
// may be, and every sequence but one is taken to end half way through a tile.
int64_t likely_tiles(int64_t rows, int64_t batch, int group, int tr) {
    return std::max<int64_t>({1, batch, cdiv(rows * group, tr) + (batch - 1) / 2});
}
// As long as the longest sequence there can be: none (and positions less a window stay far from 2^63).
int64_t bounded_window(int64_t window, int block, int64_t width) { return window >= width * block ? 0 : window; }
int64_t most_keys(int64_t rows, int64_t batch, int block, int64_t width, int64_t window) {
    const int64_t keys = width * block;
    return window > 0 ? std::min(keys, window + cdiv(rows, std::max<int64_t>(batch, 1))) : keys;
}
// Tiles, one workgroup on a CU at a time: splits as long as all run at once. 1
// sequence of 512 queries on 8 kv heads over 4000 keys: 59 us with the 256
// workgroups that 4 splits make, 78 with 2 splits, 77 with 8.
// Few rows: splits of 32 steps up to 1536 workgroups (64 sequences of 100 ..
// 16000 keys on 8 heads: 227 us with 3 splits, 243 with 2, 259 with 1), and
// shorter ones only up to 512 (16 sequences of 100 .. 8000 keys: 34.8 us with 4
// splits, 38.2 with 8, 51.5 with 16; 128 sequences of 100 .. 4000 keys: 124 with
// 1, 136 with 2).
// Up to 2048 keys eight waves share a tile instead, and there is no join: 1000
// keys 14.3 us, split 19; 16 sequences of 2000 keys 20.9 and 25.3. At 4000 keys
// of one sequence it is 29 against 19.
AttnPlan plan(int64_t rows, int64_t batch, int heads, int kv_heads, int dim, int64_t keys, bool tiles) {
    AttnPlan p;
    p.tr = tiles ? ATTN_TILE : TR;
    const int64_t units = likely_tiles(rows, batch, heads / kv_heads, p.tr) * kv_heads;
    const int64_t want = tiles ? 256 / units : std::max(512 / units, std::min(1536 / units, cdiv(keys, 32 * TK)));
    const int64_t most = std::min<int64_t>(cdiv(keys, 8 * TK), 64);
    p.nsplit = (int)std::max<int64_t>(1, std::min(want, most));
    p.nw = 4;
    if (!tiles && dim <= 128 && p.nsplit > 1 && keys <= 2048) {
        p.nw = 8;
        p.nsplit = 1;
    }
    return p;
}
// Microseconds that either kernel takes, fitted to both kernels' times at 2 ..
// 512 queries on 1000 .. 16000 keys, 64 and 128 channels: a start, and steps of
// 64 keys, 4 at a time on a CU or one. At 8 sequences on 8 kv heads of 4 query
// heads over 2000 keys: 16 queries 22.7 us with few rows at a time and 34.6 with
// tiles, 32 queries 39.3 and 38.7, 64 queries 73.6 and 53.1.
// fp32 queries take twice the products in both kernels, and the same rule: over
// 192 sizes each of 2 .. 512 queries on 1024 .. 16000 keys the choice is 0.7%
// slower than the better kernel in the mean, for bf16 and for fp32, 23% and 19%
// at worst (8 sequences of 32 heads of 64 on 8: 128 queries on 1024 keys bf16,
// few rows 38.2 us where tiles take 31.1; 64 on 4096 fp32, tiles 86.7, few rows
// 73.1). Above that fp32 tiles win as bf16 ones do: 8 sequences of 512 queries
// of 16 heads of 128 on 2 over 16000 keys, 874 us against 1668.
bool use_tiles(int64_t rows, int64_t batch, int heads, int kv_heads, int dim, int64_t keys) {
    if (dim > 128) return false;
    const int group = heads / kv_heads;
    const double steps = (double)keys / TK * kv_heads * dim / 128;
    const double few = 18 + 1.85 / 1024 * steps * likely_tiles(rows, batch, group, TR);
    const double many = 38 + 2.1 / 256 * steps * likely_tiles(rows, batch, group, ATTN_TILE);
    return many < few;
}

template <typename T, int D>
int launch(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    const int tr = p.tr;
    const int64_t units = tile_units(a.g.rows, a.g.batch, a.group, tr) * a.kv_heads;
    const dim3 grid((unsigned)(units * a.nsplit));
    if constexpr (D <= 128) {
        if (tr != TR) {
            static PerDevice ready;    // more than 64 KB of LDS
            PTQ_TRY(allow_lds(ready, (const void*)attention_tile_kernel<T, D, TILE_WAVES, false>, TileLds<D>::BYTES));
            hipLaunchKernelGGL((attention_tile_kernel<T, D, TILE_WAVES, false>), grid, dim3(64 * TILE_WAVES), TileLds<D>::BYTES, st,
                               a);
        } else if (p.nw == 8) {
            hipLaunchKernelGGL((attention_rows_kernel<T, D, 8, false>), grid, dim3(512), 0, st, a);
        } else {
            hipLaunchKernelGGL((attention_rows_kernel<T, D, 4, false>), grid, dim3(256), 0, st, a);
        }
    } else {
        hipLaunchKernelGGL((attention_rows_kernel<T, D, 4, false>), grid, dim3(256), 0, st, a);
    }
    PTQ_LAUNCH_CHECK();
    if (a.nsplit > 1) {
        hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3((unsigned)(units * (tr / TR))), dim3(256), 0, st, a, tr);
        PTQ_LAUNCH_CHECK();
    }
    return PTQ_OK;
}

template <typename T>
int launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
    switch (a.dim) {
        case 64: return launch<T, 64>(a, p, st);
        case 128: return launch<T, 128>(a, p, st);
        default: return launch<T, 256>(a, p, st);
    }
}

}  // namespace

size_t attention_int8_ws_bytes(int64_t rows, int64_t batch, int heads, int kv_heads, int dim, int block,
                               int64_t width) {
    // a window makes the splits fewer, and may choose few rows at a time where the whole length would choose tiles
    const int64_t keys = most_keys(rows, batch, block, width, 0);
    int n = plan(rows, batch, heads, kv_heads, dim, keys, false).nsplit;
    if (use_tiles(rows, batch, heads, kv_heads, dim, keys))
        n = std::max(n, plan(rows, batch, heads, kv_heads, dim, keys, true).nsplit);
    return attention_int8_part_bytes(n, rows, heads, dim);
}

size_t attention_int8_part_bytes(int nsplit, int64_t rows, int heads, int dim) {
    if (nsplit == 1) return 0;
    Sizer z;
    z.take<float>((size_t)nsplit * rows * heads * dim);
    z.take<float>((size_t)nsplit * rows * heads);
    return z.bytes();
}

AttnPlan attention_int8_plan(int64_t rows, int64_t batch, int heads, int kv_heads, int dim, int block, int64_t width,
                             int64_t window) {
    const int64_t keys = most_keys(rows, batch, block, width, bounded_window(window, block, width));
    return plan(rows, batch, heads, kv_heads, dim, keys, use_tiles(rows, batch, heads, kv_heads, dim, keys));
}

int run_attention_int8(const AttnPlan& p, const KVCacheInt8& c, const RaggedRows& r, int dtype, const void* Q,
                       int64_t ldq, int heads, float scale, int causal, int64_t window, void* O, int64_t ldo,
                       float* lse, void* ws, size_t ws_bytes, hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    window = bounded_window(window, c.block, r.width);
    AttnArgs a{};
    a.g.offsets = r.offsets; a.g.starts = r.starts; a.g.batch = (int)r.batch; a.g.rows = r.rows;
    a.table = r.table; a.width = r.width;
    a.heads = heads; a.kv_heads = c.heads; a.group = heads / c.heads;
    a.dim = c.dim; a.bs = c.block; a.bs_log2 = __builtin_ctz((unsigned)c.block); a.num_blocks = c.num_blocks;
    a.k = c.k; a.v = c.v; a.ks = c.k_scales; a.vs = c.v_scales;
    a.Q = Q; a.ldq = ldq; a.O = O; a.ldo = ldo; a.lse = lse;
    a.scale2 = (float)(scale * 1.4426950408889634);
    a.causal = causal; a.window = window;
    a.nsplit = p.nsplit;
    if (a.nsplit > 1) {
        Arena ar(ws, ws_bytes);
        a.part = ar.take<float>((size_t)a.nsplit * r.rows * heads * c.dim);
        a.part_lse = ar.take<float>((size_t)a.nsplit * r.rows * heads);
    }
    return dtype == PTQ_F32 ? launch_dim<float>(a, p, st) : launch_dim<uint16_t>(a, p, st);
}

namespace {

template <typename T, int D>
int launch_tree(const AttnArgs& a, int tr, int nw, hipStream_t st) {
    const dim3 grid((unsigned)(tile_units(a.g.rows, a.g.batch, a.group, tr) * a.kv_heads * a.nsplit));
    if constexpr (D <= 128) {
        if (tr == ATTN_TILE) {
            static PerDevice ready;    // more than 64 KB of LDS
            PTQ_TRY(allow_lds(ready, (const void*)attention_tile_kernel<T, D, TILE_WAVES, true>, TileLds<D>::BYTES));
            hipLaunchKernelGGL((attention_tile_kernel<T, D, TILE_WAVES, true>), grid, dim3(64 * TILE_WAVES),
                               TileLds<D>::BYTES, st, a);
            PTQ_LAUNCH_CHECK();
            return PTQ_OK;
        }
        if (nw == 8) {
            hipLaunchKernelGGL((attention_rows_kernel<T, D, 8, true>), grid, dim3(512), 0, st, a);
            PTQ_LAUNCH_CHECK();
            return PTQ_OK;
        }
    }
    hipLaunchKernelGGL((attention_rows_kernel<T, D, 4, true>), grid, dim3(256), 0, st, a);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

template <typename T>
int launch_tree(const AttnArgs& a, int tr, int nw, hipStream_t st) {
    switch (a.dim) {
        case 64: return launch_tree<T, 64>(a, tr, nw, st);
        case 128: return launch_tree<T, 128>(a, tr, nw, st);
        default: return launch_tree<T, 256>(a, tr, nw, st);
    }
}

}  // namespace

int launch_attention_tree_rows(const TreeArgs& t, int dtype, int dim, int tr, int nw, hipStream_t st) {
    AttnArgs a{};
    a.g = t.g;
    a.table = t.table; a.width = t.width;
    a.heads = t.heads; a.kv_heads = t.kv_heads; a.group = t.group;
    a.dim = dim; a.bs = t.bs; a.bs_log2 = t.bs_log2; a.num_blocks = t.num_blocks;
    a.k = t.k; a.v = t.v; a.ks = t.ks; a.vs = t.vs;
    a.Q = t.Q; a.ldq = t.ldq; a.O = t.O; a.ldo = t.ldo; a.lse = t.lse;
    a.scale2 = t.scale2;
    a.causal = 1; a.window = t.window; a.parents = t.parents;
    a.nsplit = t.nsplit; a.part = t.part; a.part_lse = t.part_lse;
    return dtype == PTQ_F32 ? launch_tree<float>(a, tr, nw, st) : launch_tree<uint16_t>(a, tr, nw, st);
}

}  // namespace ptq
