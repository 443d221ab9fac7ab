// Softmax attention of trees of drafted tokens over the int8 block cache
// (layout in kv_cache.hip): the last n keys of a sequence are the nodes of a
// tree, its queries are theirs. Node i attends to every key before the tree and
// to its ancestors and itself,
//
//   o_i = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q_i.k_j - m)
//   k_j = S_k[block(j)] c_j,  v_j = S_v[block(j)] c'_j
//
// Arithmetic, the same in all kernels of trees. Both products run on the fp16
// matrix cores, where the codes of K and V are exact. A row of q is scaled by a
// power of two and held in one fp16 term (bf16: elements of at least 2^-20 of the
// largest are exact) or in two (fp32: off by 2^-22 of themselves or by 2^-28 of the
// largest), w_j = p_j S_v[block(j)] / R in one (11 bits, which is below bf16's
// rounding of the output) or in two, R the running maximum of S_v over the blocks
// that the row attends to. Maxima, sums and the output accumulate in fp32. Scores
// as int8 products of K's codes as they lie, with q in whole numbers of steps, need
// no conversion of K, but one large channel then costs the others their bits (40
// nodes over 2000 keys, D = 128, a channel 300 times larger: outputs off by 4.3e-3
// instead of 1.7e-3, of fp32 by 4e-5 instead of 6e-7), and they were hardly faster:
// 16 trees over 500 .. 8000 keys 97 us where these take 94, the chosen kernels of
// 167 shapes 0.5% in the mean.
#include "attention.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace ptq {
namespace {

constexpr int ROWS = ATTN_TREE_ROWS;            // query rows (nodes x grouped heads) of a tile

// One tile of query rows: flat rows f0 .. f0 + tr of sequence b, flat row =
// node * group + head within the group.
struct TreeTile {
    int b;
    int64_t off;           // first row of the sequence
    int nodes, rows;       // nodes, and flat rows, of the sequence
    int f0;
    int base, end;         // keys before the tree; end of the keys that a row of the tile attends to
    int it0, it1;          // steps of tk keys that some row of the tile attends to
    bool bad;              // longer than its row of the table can hold, or more nodes than a line has: NaN
};

template <bool LONGEST_FIRST>
__device__ __forceinline__ bool find_tile(const TreeArgs& a, unsigned unit, int tr, int tk, TreeTile& t) {
    const RaggedUnit u = LONGEST_FIRST ? find_longest_first(a.g, unit, a.group, tr) : ragged_find(a.g, unit, a.group, tr, 1);
    t.b = u.b;
    t.off = u.off;
    const int64_t rows = u.rows * a.group, f0 = u.local * tr;      // below 2^25 (rows x heads)
    if (u.rows <= 0 || f0 >= rows) return false;
    t.nodes = (int)u.rows;
    t.rows = (int)rows;
    t.f0 = (int)f0;
    const int len = std::max(u.start, 0);
    t.base = std::max(len - t.nodes, 0);
    t.bad = len > a.width * a.bs || len < t.nodes || t.nodes > NODES;
    t.end = std::min(t.base + std::min(t.f0 + tr - 1, t.rows - 1) / a.group + 1, len);
    const int lo = a.window > 0 ? (int)std::max<int64_t>(0, t.base - a.window + 1) : 0;      // of the root, the lowest
    t.it0 = lo / tk;
    t.it1 = t.bad ? t.it0 : (int)(((unsigned)t.end + tk - 1) / tk);
    return true;
}

// Steps of a split of a tile: an even share, but not so few that the start of a
// workgroup and the join would outweigh them.
__device__ __forceinline__ int split_steps(const TreeTile& t, int nsplit, int least = 4) {
    return std::max(least, (t.it1 - t.it0 + nsplit - 1) / nsplit);
}

// One query row: 32 channels of it for each of the NC pairs of fragments, as they come from memory.
template <typename T, int NC>
struct QueryRow {
    static constexpr int WORDS = 16 * sizeof(T) / 16;      // 16-byte words of 16 channels
    uint4 raw[NC][WORDS];
    // lane half hf holds channels 32 c + 16 hf .. + 15: 8 of fragment 2 c, 8 of 2 c + 1; the lanes that differ in bit 5
    // share the row
    __device__ __forceinline__ void load(const T* p) {
        const int hf = (threadIdx.x >> 5) & 1;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int w = 0; w < WORDS; ++w) raw[c][w] = *(const uint4*)(p + 32 * c + 16 * hf + w * (16 / sizeof(T)));
    }
    __device__ __forceinline__ void values(int e, float (&x)[8]) const { load8((const T*)&raw[e / 2][e % 2 * (WORDS / 2)], x); }
    // In NT fp16 terms, scaled by the power of two that brings the largest element to [8, 16), negated for a negative softmax
    // scale; returns the factor with which they stand for the row times that scale, in units of log2. A row with a NaN or an
    // infinity gets the factor NaN.
    template <int NT>
    __device__ __forceinline__ float terms(float scale2, f16x8 (&q)[NT][2 * NC]) {
        uint32_t size = 0;      // |x| as bits, in the order of the values: a NaN's are the largest
#pragma unroll
        for (int e = 0; e < 2 * NC; ++e) {
            float x[8];
            values(e, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) size = std::max(size, __float_as_uint(x[k]) & 0x7fffffffu);
        }
        size = std::max(size, (uint32_t)__shfl_xor((int)size, 32, 64));
        const int field = std::min(257 - (int)(size >> 23), 253);
        const float up = __uint_as_float((uint32_t)field << 23 | (scale2 < 0.f ? 0x80000000u : 0u));
#pragma unroll
        for (int e = 0; e < 2 * NC; ++e) {
            float x[8];
            values(e, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float y = x[k] * up;
                q[0][e][k] = (_Float16)y;
                if constexpr (NT == 2) q[1][e][k] = (_Float16)(y - (float)q[0][e][k]);
            }
        }
        const float back = __uint_as_float((uint32_t)(254 - field) << 23);
        return size < 0x7f800000u ? fabsf(scale2) * back : __builtin_nanf("");
    }
};

// A workgroup takes a tile of 32 query rows of one kv head, and its NW waves every
// NW-th step of 64 keys (32 where 64 do not fit the registers of the waves that a
// SIMD shall hold). Scores are computed transposed, S^T = K Q^T, so that a lane
// ends up with scores of one row and the probabilities are already the operand of
// O^T = V^T P^T: operand row r of a block of 32 keys is key
// 16 (r / 4 % 2) + 4 (r / 8) + r % 4, so lane half hf holds keys 16 hf .. 16 hf +
// 15, in one block of the cache: one S_k and one S_v a lane.
//
// A wave copies the codes of a step into a part of LDS of its own, as they are and
// whole rows at a time, and copies the next step over it when it has read it; the
// other waves of the SIMD work meanwhile, and nothing waits for another wave until
// the join. What bounds it: for few rows memory (16 trees of 8 nodes over 4000
// keys, 32 heads on 8, D = 128: 41 us, the cache's 131 MB at 3.2 TB/s), with more
// tiles on the same keys the vector instructions of the exponentials and of the
// conversion of K and V. Tiles of 64 and 128 rows that share a step among waves were 1%
// faster in the mean over 1700 shapes, and taken out; from about 300 rows a kv
// head on, the tiles of 256 rows of attention_int8.hip win, and for few rows and
// keys its tiles of 16, whose keys go straight into registers.
template <typename T>
constexpr int blocks_of(int dim) { return dim <= (sizeof(T) == 4 ? 64 : 128) ? 2 : 1; }
constexpr int waves_of(int dim) { return dim <= 128 ? 2 : 1; }

// Chunks of 16 bytes in LDS, C a row: chunk c of row r lies at c ^ swizzle(r), so that the same chunk of 16 neighbours is
// in all 64 banks.
template <int C>
__device__ __forceinline__ int swizzle(int r) {
    return (r / (16 / C)) & (C - 1);
}

// Codes of a step in LDS: K in the order of the operand's rows, chunks of 16 channels, and V in chunks of 16 keys of a
// channel.
template <int D, int U>
struct TreeCodes {
    uint4 k[32 * U][D / 16];
    uint4 v[D][2 * U];
};

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;
// 16 bytes a lane from `from` into LDS at to + 16 lane (`to` the same for the wave); done when vmcnt says so
__device__ __forceinline__ void copy16(const void* from, void* to) {
    __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
}

template <typename T, int D, int NW>
__global__ __launch_bounds__(64 * NW, waves_of(D)) void attention_tree_kernel(TreeArgs a) {
    constexpr int U = blocks_of<T>(D), TK = 32 * U;
    constexpr int NT = sizeof(T) == 4 ? 2 : 1;    // fp16 terms of q and of the probabilities
    constexpr int NC = D / 32, NTH = 64 * NW;
    constexpr bool FOLD = NT == 1;       // S_v / R goes into the exponent
    __shared__ TreeLines<ROWS> lines_of;

    const int split = (int)(blockIdx.x % (unsigned)a.nsplit);
    const unsigned tile = blockIdx.x / (unsigned)a.nsplit;
    const int h = (int)(tile % (unsigned)a.kv_heads);
    TreeTile tl;
    if (!find_tile<true>(a, tile / (unsigned)a.kv_heads, ROWS, TK, tl)) return;
    const int per = split_steps(tl, a.nsplit);
    const int s0 = tl.it0 + split * per, s1 = std::min(s0 + per, tl.it1);
    if (split > 0 && s0 >= s1) return;

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int li = lane & 31, hf = lane >> 5;
    const int first_node = tl.f0 / a.group;
    auto row_of = [&](int i) { return std::min(tl.f0 + i, tl.rows - 1); };
    const int node = row_of(li) / a.group;
    const int32_t* table = a.table + (int64_t)tl.b * a.width;
    const unsigned pool = (unsigned)a.bs * D, stride = (unsigned)a.kv_heads * pool;      // codes of a (block, head), of a block
    const int8_t* kp = a.k + (int64_t)h * pool;
    const int8_t* vp = a.v + (int64_t)h * pool;
    const int end = tl.end, bmask = a.bs - 1;
    // block of position p: one without a valid id, and positions past the keys, stand for some other block of the
    // pool, whose codes are as good as any (the scale says NaN, or the mask leaves them out)
    auto entry = [&](int p) __attribute__((always_inline)) { return table[std::min(p, end - 1) >> a.bs_log2]; };
    auto ok = [&](int id) { return (unsigned)id < (unsigned)a.num_blocks; };
    auto place = [&](int id, int off) __attribute__((always_inline)) { return (uint64_t)(ok(id) ? (unsigned)id : 0u) * stride + (unsigned)off; };
    auto scale_at = [&](int id) { return (uint64_t)(ok(id) ? (unsigned)id : 0u) * (unsigned)a.kv_heads + (unsigned)h; };
    // infinite scales, too, count as NaN: times codes of one sign they would stay infinite
    auto clean = [&](float s, int id, int p) { return p >= end ? 0.f : ok(id) && s < INFINITY ? s : __builtin_nanf(""); };
    auto key_of_row = [](int r) { return 16 * (r >> 2 & 1) + 4 * (r >> 3) + (r & 3); };      // r < 32

    // what the rest waits for is requested first, and answered in that order: parents, the query row, the first keys
    const bool lines = !tl.bad && (a.window > 0 || s1 * TK > tl.base);
    constexpr int PN = NODES / NTH + (NODES % NTH != 0);
    int up[PN];
    if (lines)
#pragma unroll
        for (int i = 0; i < PN; ++i) up[i] = a.parents[tl.off + std::min(t + i * NTH, tl.nodes - 1)];
    QueryRow<T, NC> row;
    row.load((const T*)a.Q + (tl.off + node) * a.ldq + (int64_t)(h * a.group + row_of(li) % a.group) * D);

    // this wave's part of LDS, and the copies of one step into it
    constexpr int KC = D / 16, VC = 2 * U;      // chunks of a row of K, groups of 16 keys of a channel of V
    using Codes = TreeCodes<D, U>;
    __shared__ __attribute__((aligned(16))) unsigned char own[NW * sizeof(Codes)];
    Codes& codes = ((Codes*)own)[wave];
    float rsk[U], rsv[U];
    int ids_of[U];
    const bool one_block = a.bs >= TK;      // a step lies in one block of the cache: addresses are scalar
    auto copy = [&](int it) __attribute__((always_inline)) {
        constexpr int KI = 32 * U * KC / 64, VI = D * VC / 64;      // copies of 64 chunks
        auto krow = [&](int i) { return (i * 64 + lane) / KC; };
        auto koff = [&](int i) {      // from the first key of a step in one block
            return ((krow(i) & ~31) + key_of_row(krow(i) & 31)) * D + 16 * ((lane % KC) ^ swizzle<KC>(krow(i)));
        };
        const int vd = lane / VC, vg = (lane % VC) ^ swizzle<VC>(vd);      // 64 / VC channels a copy, a multiple of 16
        const int voff = vd * a.bs + 16 * vg;
        if (one_block) {
            const int id = __builtin_amdgcn_readfirstlane(entry(it * TK)), from = (it * TK) & bmask;
            const int8_t* kb = kp + place(id, from * D);
            const int8_t* vb = vp + place(id, from);
#pragma unroll
            for (int i = 0; i < KI; ++i)
                copy16(kb + (unsigned)koff(i), (char*)codes.k + 1024 * i);
#pragma unroll
            for (int i = 0; i < VI; ++i)
                copy16(vb + (unsigned)(voff + i * (64 / VC) * a.bs), (char*)codes.v + 1024 * i);
#pragma unroll
            for (int u = 0; u < U; ++u) ids_of[u] = id;
            rsk[0] = a.ks[scale_at(id)];
            rsv[0] = a.vs[scale_at(id)];
            if constexpr (U == 2) rsk[1] = rsk[0], rsv[1] = rsv[0];
            return;
        }
        // blocks of 16 keys each
        const int id0 = entry(it * TK), id1 = entry(it * TK + 16);
        const int id2 = U == 1 ? 0 : entry(it * TK + 32), id3 = U == 1 ? 0 : entry(it * TK + 48);
        const int idv = entry(it * TK + 16 * vg);
        ids_of[0] = hf ? id1 : id0;
        if constexpr (U == 2) ids_of[1] = hf ? id3 : id2;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int key = key_of_row(krow(i) & 31);
            const int id = i * 64 / KC < 32 ? (key & 16 ? id1 : id0) : (key & 16 ? id3 : id2);      // rows of one 32
            const int p = it * TK + (krow(i) & ~31) + key;
            copy16(kp + place(id, (p & bmask) * D + 16 * ((lane % KC) ^ swizzle<KC>(krow(i)))), (char*)codes.k + 1024 * i);
        }
        const int8_t* from = vp + place(idv, vd * a.bs + ((it * TK + 16 * vg) & bmask));
#pragma unroll
        for (int i = 0; i < VI; ++i)
            copy16(from + i * (64 / VC) * a.bs, (char*)codes.v + 1024 * i);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rsk[u] = a.ks[scale_at(ids_of[u])];
            rsv[u] = a.vs[scale_at(ids_of[u])];
        }
    };
    if (s0 + wave < s1) copy(s0 + wave);

    // lines of the tile's nodes, where this split has keys of the tree or a window asks for depths
    int lo = 0;
    bool broken = tl.bad;
    if (lines) {
        const int count = std::min(tl.f0 + ROWS - 1, tl.rows - 1) / a.group - first_node + 1;
        build_lines<NTH>(lines_of, up, tl.nodes, first_node, count, a.window, t);
        const int depth = lines_of.level[node - first_node];
        broken = depth < 0;
        lo = first_key(tl.base, depth, a.window);
    }
    const int lo_max = a.window > 0 ? (int)std::max<int64_t>(0, tl.base + (int64_t)tl.nodes - a.window) : 0;   // of the deepest row
    // steps that no row masks: [whole, last)
    const int whole = std::min(__builtin_amdgcn_readfirstlane((lo_max + TK - 1) / TK), s1);
    const int last = std::min(__builtin_amdgcn_readfirstlane(tl.base / TK), s1);

    f16x8 q[NT][2 * NC];
    f32x16 acc[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    // ref: what the scores' maximum m stands for in the exponents
    float m = -INFINITY, l = broken ? __builtin_nanf("") : 0.f, R = 0.f, rcp_R = 0.f, log2_R = 0.f, poison = 0.f;
    const float qs = row.template terms<NT>(a.scale2, q);

    auto work = [&](auto masked, int it) __attribute__((always_inline)) {
        constexpr bool MASK = decltype(masked)::value;
        float sk[U], sv[U], lv[U];      // S_k, S_v and log2 S_v of the lane's keys of each block
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tv = it * TK + 32 * u + 16 * hf;
            sk[u] = clean(rsk[u], ids_of[u], tv);
            sv[u] = clean(rsv[u], ids_of[u], tv);
            lv[u] = FOLD ? __builtin_amdgcn_logf(sv[u]) : 0.f;
        }
        f32x16 s[U];
        uint32_t seen[U];
        float ck[U], top = -INFINITY, big = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                const uint4 k = codes.k[32 * u + li][(2 * e + hf) ^ swizzle<KC>(li)];
                const f16x8 k0 = half8(k.x, k.y), k1 = half8(k.z, k.w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k0, q[n][2 * e], s[u], 0, 0, 0);
                    s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k1, q[n][2 * e + 1], s[u], 0, 0, 0);
                }
            }
            ck[u] = sk[u] * qs;
            seen[u] = 0xffffu;
            if constexpr (MASK) {
                seen[u] = seen16(lines_of.line[node - first_node], it * TK + 32 * u + 16 * hf, tl.base, lo);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[u][r] = seen[u] >> r & 1 ? s[u][r] * ck[u] : -INFINITY;
                ck[u] = 1.f;
            }
            float most = s[u][0];
#pragma unroll
            for (int r = 1; r < 16; ++r) most = fmaxf(most, s[u][r]);
            top = fmaxf(top, most * ck[u]);
            // R: largest finite S_v of the row's blocks so far
            if (sv[u] < INFINITY && (!MASK || seen[u])) big = fmaxf(big, sv[u]);
            if (FOLD && sv[u] != sv[u] && (!MASK || seen[u])) poison = sv[u];
        }
        top = max_halves(top);
        big = max_halves(big);
        if (__any(top > m + LAZY || big > R)) {
            // each row by itself: what one row sees changes no other row's roundings
            float fall = 1.f;
            if (top > m + LAZY) {
                fall = exp2_fast(m - top);
                m = top;
                l *= fall;
            }
            if (big > R) {
                rcp_R = big < FLT_MIN ? 0.f : __fdiv_rn(1.f, big);
                fall *= R * rcp_R;
                R = big;
                log2_R = big < FLT_MIN ? 0.f : __builtin_amdgcn_logf(big);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][r] *= fall;
        }
        const float m_sub = (m == -INFINITY ? 0.f : m) - PSHIFT;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float rv = sv[u] * rcp_R, lr = FOLD ? fmaxf(lv[u] - log2_R, LOG2_RV_MIN) : 0.f;      // of NaN, too
            const float off = m_sub - lr;
            float sum = 0.f;
            f16x8 w[NT][2];
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                f32x2 y;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float p = exp2_fast(fmaf(s[u][r + k], ck[u], -off));
                    const bool in = !MASK || (seen[u] >> (r + k) & 1);      // S_v of a block that is not this row's may be NaN
                    if constexpr (FOLD) {
                        if (!in) p = 0.f;
                        sum += p;
                        y[k] = p;
                    } else {
                        sum += p;
                        y[k] = in ? p * rv : 0.f;
                    }
                }
                const f16x2 x = __builtin_convertvector(y, f16x2);
                w[0][r >> 3][r & 7] = x[0];
                w[0][r >> 3][(r & 7) + 1] = x[1];
                if constexpr (NT == 2) {
                    const f16x2 z = __builtin_convertvector((f32x2{y[0] - (float)x[0], y[1] - (float)x[1]}), f16x2);
                    w[1][r >> 3][r & 7] = z[0];
                    w[1][r >> 3][(r & 7) + 1] = z[1];
                }
            }
            l += FOLD ? sum * exp2_fast(-lr) : sum;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint4 v = codes.v[32 * i + li][(2 * u + hf) ^ swizzle<VC>(li)];
                const f16x8 v0 = half8(v.x, v.y), v1 = half8(v.z, v.w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, w[n][0], acc[i], 0, 0, 0);
                    acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w[n][1], acc[i], 0, 0, 0);
                }
            }
        }
    };
    auto step = [&](auto masked, int it) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt = 0: the copies have landed
        asm volatile("" ::: "memory");
        work(masked, it);
        __builtin_amdgcn_s_waitcnt(0xc07f);      // lgkmcnt = 0: everything has been read
        asm volatile("" ::: "memory");
        if (it + NW < s1) copy(it + NW);
    };
    int it = s0 + wave;
    for (; it < whole; it += NW) step(std::true_type{}, it);
    for (; it < last; it += NW) step(std::false_type{}, it);
    for (; it < s1; it += NW) step(std::true_type{}, it);

    l += __shfl_xor(l, 32, 64);
    if (FOLD) poison += __shfl_xor(poison, 32, 64);
    // this lane's row is worked out again: its registers are the loop's
    int again = li;
    asm volatile("" : "+v"(again));
    const int f = row_of(again), qh = h * a.group + f % a.group;
    const bool there = tl.f0 + again < tl.rows;
    const int64_t token = tl.off + f / a.group;
    const bool split_out = a.nsplit > 1;
    const int64_t nflat = a.g.rows * a.heads, at = token * a.heads + qh;
    // join the waves: factors to the common maximum, then sums through LDS
    __shared__ float sm[NW][ROWS], sl[NW][ROWS];
    if (hf == 0) {
        sm[wave][li] = m;
        sl[wave][li] = l;
    }
    __syncthreads();
    float M = sm[0][li];
#pragma unroll
    for (int g = 1; g < NW; ++g) M = fmaxf(M, sm[g][li]);
    const float M0 = M == -INFINITY ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int g = 0; g < NW; ++g) L += sl[g][li] * exp2_fast(sm[g][li] - M0);
    const float mine = (R > 0.f ? R : 1.f) * exp2_fast(m - M0) / (L == 0.f ? 1.f : L) + poison;
    constexpr int JC = sizeof(own) >= sizeof(float) * NW * ROWS * 68 ? 64 : 32;      // channels at a time
    static_assert(sizeof(own) >= sizeof(float) * NW * ROWS * (JC + 4), "the join goes where the keys were");
    float(*so)[ROWS][JC + 4] = (float(*)[ROWS][JC + 4])own;      // behind the barrier above
#pragma unroll
    for (int i0 = 0; i0 < NC; i0 += JC / 32) {
        if (i0) __syncthreads();
#pragma unroll
        for (int i = 0; i < JC / 32; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f32x16& x = acc[i0 + i];
                *(f32x4*)&so[wave][li][32 * i + 8 * b + 4 * hf] =
                    f32x4{x[4 * b] * mine, x[4 * b + 1] * mine, x[4 * b + 2] * mine, x[4 * b + 3] * mine};
            }
        __syncthreads();
        for (int c = t; c < ROWS * JC / 4; c += NTH) {
            const int r = c / (JC / 4), d = 4 * (c % (JC / 4)), fr = tl.f0 + r;
            if (fr >= tl.rows) continue;
            f32x4 o = *(const f32x4*)&so[0][r][d];
#pragma unroll
            for (int g = 1; g < NW; ++g) o += *(const f32x4*)&so[g][r][d];
            const int64_t row = tl.off + fr / a.group;
            const int head = h * a.group + fr % a.group;
            if (split_out)
                *(f32x4*)(a.part + (split * nflat + row * a.heads + head) * D + 32 * i0 + d) = o;
            else
                store4((T*)a.O + row * a.ldo + (int64_t)head * D + 32 * i0 + d, o[0], o[1], o[2], o[3]);
        }
    }
    if (wave == 0 && hf == 0 && there && (split_out || a.lse)) {
        // L carries 2^PSHIFT
        const float lse2 = L == 0.f ? -INFINITY : M0 - PSHIFT + __log2f(L);
        if (split_out)
            a.part_lse[split * nflat + at] = lse2;
        else
            a.lse[at] = lse2 * 0.6931471805599453f;
    }
}

// Join of the splits: 16 rows a workgroup, 16 threads a row, JB splits at a
// time with all their loads at once; tr: rows of the tiles that were split.
template <typename T, int D, int tr>
__global__ __launch_bounds__(256) void attention_tree_join_kernel(TreeArgs a) {
    constexpr int TK = tr == ROWS ? 32 * blocks_of<T>(D) : ptq::TK;
    const unsigned part = blockIdx.x % (unsigned)(tr / 16), tile = blockIdx.x / (unsigned)(tr / 16);
    const int h = (int)(tile % (unsigned)a.kv_heads);
    TreeTile tl;
    if (!find_tile<false>(a, tile / (unsigned)a.kv_heads, tr, TK, tl)) return;
    const int per = split_steps(tl, a.nsplit, tr == ATTN_ROWS ? 8 : 4);
    const int n = std::max(1, (tl.it1 - tl.it0 + per - 1) / per);    // split 0 is always written
    const int r = threadIdx.x / 16, c = threadIdx.x % 16, f = tl.f0 + (int)part * 16 + r;
    if (f >= tl.rows) return;
    const int64_t row = tl.off + f / a.group, nflat = a.g.rows * a.heads;
    const int head = h * a.group + f % a.group;
    const int64_t at = row * a.heads + head;
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

template <typename T, int D>
int launch(const TreeArgs& a, const TreePlan& p, hipStream_t st) {
    const int64_t units = tile_units(a.g.rows, a.g.batch, a.group, p.tr) * a.kv_heads;
    const dim3 grid((unsigned)(units * a.nsplit)), join((unsigned)(units * (p.tr / 16)));
    if (p.tr != ROWS) {
        PTQ_TRY(launch_attention_tree_rows(a, sizeof(T) == 4 ? PTQ_F32 : PTQ_BF16, D, p.tr, p.nw, st));
        if (a.nsplit > 1) {
            if (p.tr == ATTN_ROWS)
                hipLaunchKernelGGL((attention_tree_join_kernel<T, D, ATTN_ROWS>), join, dim3(256), 0, st, a);
            else if constexpr (D <= 128)
                hipLaunchKernelGGL((attention_tree_join_kernel<T, D, ATTN_TILE>), join, dim3(256), 0, st, a);
            PTQ_LAUNCH_CHECK();
        }
        return PTQ_OK;
    }
    if (D <= 128 && p.nw == 8) {
        if constexpr (D <= 128) hipLaunchKernelGGL((attention_tree_kernel<T, D, 8>), grid, dim3(512), 0, st, a);
    } else {
        hipLaunchKernelGGL((attention_tree_kernel<T, D, 4>), grid, dim3(256), 0, st, a);
    }
    PTQ_LAUNCH_CHECK();
    if (a.nsplit > 1) {
        hipLaunchKernelGGL((attention_tree_join_kernel<T, D, ROWS>), join, dim3(256), 0, st, a);
        PTQ_LAUNCH_CHECK();
    }
    return PTQ_OK;
}

template <typename T>
int launch_dim(const TreeArgs& a, int dim, const TreePlan& p, hipStream_t st) {
    switch (dim) {
        case 64: return launch<T, 64>(a, p, st);
        case 128: return launch<T, 128>(a, p, st);
        default: return launch<T, 256>(a, p, st);
    }
}

}  // namespace

size_t attention_tree_part_bytes(int nsplit, int64_t rows, int heads, int dim) {
    if (nsplit == 1) return 0;
    Sizer z;
    z.take<float>((size_t)nsplit * rows * heads * dim);
    z.take<float>((size_t)nsplit * rows * heads);
    return z.bytes();
}

// The choice of a TreePlan: the least of estimated times, in microseconds,
//   start + rounds (first + steps each) + [join + bytes of the parts],
// fitted to 750 shapes with all their plans (1 .. 64 sequences of 1 .. 64 nodes, 1
// .. 8 kv heads, groups of 1 .. 8, 64 .. 16000 keys, half of them ragged). Over 670
// others like them the choice is 3.6% slower than the best plan in the mean, 12% at
// nine shapes of ten, 44% at worst. Without one of the kernels the best plan would
// be slower in the mean by 5.7% (tiles of 16 rows: 1 tree of 16 nodes over 1000 keys
// 15.3 us, of 32 rows 18.6), 3.8% (of 32), 2.4% (32 rows by four waves) and 0.4% (of
// 256, which more rows a sequence need: 8 trees of 200 .. 512 nodes, 4 heads a
// group, over 500 .. 8000 keys: 295 us). Lengths are not known here: keys is the
// most there may be, and every sequence is taken to have the mean number of rows. A
// round is as many workgroups as the card holds.
TreePlan attention_tree_plan(int64_t rows, int64_t batch, int heads, int kv_heads, int dim, int dtype, int block,
                             int64_t width, int64_t window) {
    const int64_t group = heads / kv_heads, most = width * block;
    const int64_t keys = window > 0 && window < most ? std::min(most, window + cdiv(rows, batch)) : most;
    const int64_t each = cdiv(rows * group, batch);
    const bool f32 = dtype == PTQ_F32, wide = dim > 128;
    const int d = dim == 64 ? 0 : dim == 128 ? 1 : 2;
    struct Kind {
        int tr, nw;
        double start, first, step[2][3];      // step: bf16, fp32 at 64, 128, 256 channels
        int slots[3], least;                  // workgroups at once, steps of a split at least
    };
    const Kind kinds[] = {
        {ATTN_ROWS, 4, 5.0, wide ? 6.1 : 6.7, {{1.55, 2.0, 3.8}, {1.8, 2.15, 4.0}}, {1024, 512, 256}, 8},
        {ATTN_ROWS, 8, 6.1, 6.0, {{1.8, 2.6, 0}, {2.05, 3.15, 0}}, {512, 256, 0}, 8},
        {ROWS, 4, 7.1, wide ? 8.0 : 4.8, {{1.5, 2.25, 2.1}, {1.8, 1.55, 2.6}}, {512, 512, 256}, 4},
        {ROWS, 8, 6.2, 6.5, {{1.75, 2.8, 0}, {2.1, 2.1, 0}}, {256, 256, 0}, 4},
        {ATTN_TILE, 8, 7.8, 3.8, {{1.35, 1.8, 0}, {1.8, 2.75, 0}}, {256, 256, 0}, 4},
    };
    TreePlan best{};
    double least = 0;
    for (const Kind& k : kinds) {
        if (k.nw == 8 && wide) continue;
        const int tk = k.tr == ROWS ? 32 * (f32 ? blocks_of<float>(dim) : blocks_of<uint16_t>(dim)) : TK;
        const int steps = (int)std::max<int64_t>(1, cdiv(keys, tk)), waves = k.tr == ATTN_TILE ? 1 : k.nw;
        const double tiles = (double)(batch * cdiv(each, k.tr) * kv_heads);
        for (int ns = 1; ns <= 64 && (ns == 1 || ns * 4 <= steps); ns += std::max(1, ns / 4)) {
            const int per = std::max(k.least, (steps + ns - 1) / ns), mine = (std::min(per, steps) + waves - 1) / waves;
            const double full = tiles * ((steps + per - 1) / per) / k.slots[d];
            const double rounds = std::max(1., (full + std::ceil(full)) / 2);
            const double time = k.start + rounds * (k.first + k.step[f32][d] * mine) +
                                (ns == 1 ? 0. : 3.1 + 0.37e-6 * ns * (double)rows * heads * dim * 8);
            if (best.nsplit == 0 || time < least) {
                least = time;
                best = TreePlan{k.tr, k.nw, ns};
            }
        }
    }
    return best;
}

int run_attention_tree(const TreePlan& p, const KVCacheInt8& c, const RaggedRows& r, const int32_t* parents, int dtype,
                       const void* Q, int64_t ldq, int heads, float scale, int64_t window, void* O, int64_t ldo,
                       float* lse, void* ws, size_t ws_bytes, hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    TreeArgs a{};
    a.g.offsets = r.offsets; a.g.starts = r.starts; a.g.batch = (int)r.batch; a.g.rows = r.rows;
    a.parents = parents;
    a.table = r.table; a.width = r.width;
    a.heads = heads; a.kv_heads = c.heads; a.group = heads / c.heads;
    a.bs = c.block; a.bs_log2 = __builtin_ctz((unsigned)c.block); a.num_blocks = c.num_blocks;
    a.k = c.k; a.v = c.v; a.ks = c.k_scales; a.vs = c.v_scales;
    a.Q = Q; a.ldq = ldq; a.O = O; a.ldo = ldo; a.lse = lse;
    a.scale2 = (float)(scale * 1.4426950408889634);
    a.window = window >= r.width * c.block ? 0 : window;      // as long as the longest sequence there can be: none
    a.nsplit = p.nsplit;
    if (a.nsplit > 1) {
        Arena ar(ws, ws_bytes);
        a.part = ar.take<float>((size_t)a.nsplit * r.rows * heads * c.dim);
        a.part_lse = ar.take<float>((size_t)a.nsplit * r.rows * heads);
    }
    return dtype == PTQ_F32 ? launch_dim<float>(a, c.dim, p, st) : launch_dim<uint16_t>(a, c.dim, p, st);
}

}  // namespace ptq
