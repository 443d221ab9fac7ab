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

// ------------------------------------------------------------------ trees --
struct TreeArgs {
    Ragged g;                             // g.starts: the lengths
    const int32_t* parents;
    const int32_t* table; int64_t width;
    int heads, kv_heads, group, bs, bs_log2;
    int64_t num_blocks;
    const int8_t* k; const int8_t* v; const float* ks; const float* vs;
    const void* Q; int64_t ldq;
    void* O; int64_t ldo;
    float* lse;                    // [rows, heads] or null
    float scale2;                  // softmax scale * log2(e)
    int64_t window;
    int nsplit;
    float* part; float* part_lse;  // [nsplit][rows * heads][dim], [nsplit][rows * heads]
};
// The kernels of attention_int8.hip, by tiles of tr = ATTN_ROWS rows (nw waves: 4, or 8 up to 128 channels) or of
// ATTN_TILE (up to 128 channels): write O and lse, or the splits' parts.
int launch_attention_tree_rows(const TreeArgs& a, int dtype, int dim, int tr, int nw, hipStream_t st);

// Unit w of the tiles of tr rows of each sequence, those of the longest sequence
// first: workgroups start in their order, and the longest, started last, would be
// waited for alone (16 trees over 500 .. 8000 keys: 112 us as they come, 91 so; 64
// over 100 .. 16000: 1309 and 1193). Up to 64 sequences, one a lane; more, and those
// whose workgroups all start at once, are taken as they come.
__device__ __forceinline__ RaggedUnit find_longest_first(const Ragged& g, unsigned w, int group, int tr) {
    if (g.batch == 1 || g.batch > 64 || gridDim.x <= 256) return ragged_find(g, w, group, tr, 1);
    const int lane = threadIdx.x & 63, i = std::min(lane, g.batch - 1);
    auto clamp = [&](int o) { return (int)(o < 0 ? 0 : (o > g.rows ? g.rows : o)); };
    const int o = clamp(g.offsets[i]), n = clamp(g.offsets[i + 1]), len = g.starts[i];
    const int tiles = lane < g.batch ? (int)(((int64_t)std::max(n - o, 0) * group + tr - 1) / tr) : 0;
    int rank = lane < g.batch ? 0 : lane;
    for (int j = 0; j < g.batch; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        if (lane < g.batch) rank += other > len || (other == len && j < lane);
    }
    const int which = __builtin_amdgcn_ds_permute(4 * rank, lane), mine = __builtin_amdgcn_ds_permute(4 * rank, tiles);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int x = __shfl_up(upto, d, 64);
        if (lane >= d) upto += x;
    }
    const int at = 63 - __builtin_clzll(__ballot(lane < g.batch && (unsigned)(upto - mine) <= w) | 1);
    RaggedUnit u;
    u.b = __builtin_amdgcn_readlane(which, at);
    u.off = __builtin_amdgcn_readlane(o, u.b);
    u.rows = std::max(__builtin_amdgcn_readlane(n, u.b) - (int)u.off, 0);
    u.start = __builtin_amdgcn_readlane(len, u.b);
    u.local = w - (unsigned)__builtin_amdgcn_readlane(upto - mine, at);
    return u;
}

// What the nodes of a tile of ROWS query rows attend to, of keys in the order of
// a sequence: a line of bits for each node, 64 ones for keys before the tree, a
// bit for each node (its ancestors and itself), 64 zeros.
constexpr int NODES = TREE_NODES;
constexpr int LINE_WORDS = 2 + NODES / 32 + 2;

template <int ROWS>
struct TreeLines {
    uint32_t line[ROWS][LINE_WORDS + 1];      // an odd stride
    int16_t parent[NODES];
    int16_t level[ROWS];                      // depth of a node, negative: no valid way up
};

// All NTH threads, t of them this one: nodes first .. first + count of a tree of n; up[i]: parents[t + i NTH], requested
// before. A window > 0 leaves out ancestors window levels up and more.
template <int NTH, int ROWS, int PN>
__device__ __forceinline__ void build_lines(TreeLines<ROWS>& s, const int (&up)[PN], int n, int first, int count,
                                            int64_t window, int t) {
#pragma unroll
    for (int i = 0; i < PN; ++i)
        if (t + i * NTH < n) s.parent[t + i * NTH] = (int16_t)(up[i] >= -1 && up[i] < NODES ? up[i] : NODES);
    for (int i = t; i < count * LINE_WORDS; i += NTH) s.line[i / LINE_WORDS][i % LINE_WORDS] = i % LINE_WORDS < 2 ? ~0u : 0u;
    __syncthreads();
    if (t < count) {
        // ancestors come in falling order: a word is done when the walk leaves it
        int j = first + t, depth = 0, word = j >> 5;
        uint32_t bits = 0;
        bool fine = true;
        while (true) {
            const int p = s.parent[j];
            if (j >> 5 != word) {
                s.line[t][2 + word] = bits;
                word = j >> 5;
                bits = 0;
            }
            if (window <= 0 || depth < window) bits |= 1u << (j & 31);
            if (p >= j) fine = false;
            if (p >= j || p < 0) break;
            j = p;
            ++depth;
        }
        s.line[t][2 + word] = bits;
        s.level[t] = (int16_t)(fine ? depth : -1);
    }
    __syncthreads();
}

// Which of the 16 keys from key on (of which the tree's begin at base, the row's at lo <= base) a row with this line
// attends to. Where all 16 lie before the tree there need be no lines.
__device__ __forceinline__ uint32_t seen16(const uint32_t* line, int key, int base, int lo) {
    const int o = std::min(std::max(key - base, -64) + 64, 32 * (LINE_WORDS - 2));      // the last two words are 0
    const uint32_t* w = line + (o >> 5);
    uint32_t seen = (uint32_t)((((uint64_t)w[1] << 32 | w[0]) >> (o & 31)) & 0xffffu);
    if (key + 16 <= base) seen = 0xffffu;
    if (key < lo) seen &= lo - key < 16 ? 0xffffu << (lo - key) : 0u;
    return seen;
}

// First key of a node at this depth, of those before the tree
__device__ __forceinline__ int first_key(int base, int depth, int64_t window) {
    return window > 0 ? (int)std::min<int64_t>(base, std::max<int64_t>(0, base + std::max(depth, 0) - window + 1)) : 0;
}

}  // namespace ptq
