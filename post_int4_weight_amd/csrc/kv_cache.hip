// Keys and values in an int8 cache of blocks of tokens: quantized as they are
// written, and read back.
//
// The cache is a pool of blocks. Per (block, head): k codes [bs][D], v codes
// [D][bs] and one scale each. Values are stored with a token's neighbours
// next to each other because attention contracts over tokens: 16 tokens of
// one channel are then one 16-byte load of a matrix-core operand.
// Position p of sequence b is slot p % bs of block block_table[b][p / bs].
//
// Write: S = max(S_old, max |new| / 127), S_old counting only where the block
// holds earlier positions of the sequence; when S grows, those codes are
// recoded, rint(c (S_old / S)), and the new values get rint(x / S)
// ("int8.hpp"). One workgroup owns a (block, head) pair, so nothing is
// summed or raced over, and the same call twice leaves the same cache.
#include "int8.hpp"

#include <algorithm>

namespace ptq {
namespace {

// The blocks one workgroup works on: unit w of the ragged batch.
struct BlockSpan {
    int b;            // sequence
    int64_t p0;       // first position of the block
    int lo, hi;       // slots [lo, hi) belong to rows of the call
    int64_t row0;     // row of slot 0 (slot lo is the first real one)
    int32_t id;       // block of the pool, -1: none
};

// false: a spare unit
__device__ __forceinline__ bool find_block(const Ragged& g, const int32_t* starts, const int32_t* table,
                                           int64_t width, int64_t num_blocks, int bs, int64_t unit, BlockSpan& s) {
    int64_t j;
    s.b = ragged_find(g, unit, 1, bs, 2, &j);
    const int64_t o = ragged_offset(g, s.b), n = ragged_offset(g, s.b + 1) - o;
    if (n <= 0) return false;
    const int64_t given = starts[s.b], start = given < 0 ? 0 : given;
    const int64_t at = start / bs + j;
    s.p0 = at * bs;
    if (s.p0 >= start + n) return false;
    s.lo = (int)std::max<int64_t>(start - s.p0, 0);
    s.hi = (int)std::min<int64_t>(start + n - s.p0, bs);
    s.row0 = o + s.p0 - start;
    s.id = (at < width && given >= 0) ? table[s.b * width + at] : -1;
    if (s.id < 0 || s.id >= num_blocks) s.id = -1;
    return true;
}

struct CacheArgs {
    Ragged g;
    const int32_t* starts; const int32_t* table; int64_t width;
    int heads, dim, bs;
    int64_t num_blocks;
    int8_t* codes[2];        // k, v
    float* scales[2];
};

constexpr int KEEP = 4;      // chunks of 8 values a thread holds

// codes of 8 values, low bytes first
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k >> 2] |= (uint32_t)(uint8_t)int8_code(v[k], inv) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) r |= (uint32_t)(uint8_t)(int)rintf((float)(int8_t)(w >> (8 * k)) * ratio) << (8 * k);
    return r;
}

// grid (units, heads, 2): z = 0 keys, 1 values. blockDim.x * KEEP chunks cover a block.
template <typename T>
__global__ __launch_bounds__(1024) void kv_write_kernel(CacheArgs a, const T* __restrict__ K, int64_t ldk,
                                                        const T* __restrict__ V, int64_t ldv) {
    extern __shared__ __attribute__((aligned(16))) unsigned char image[];   // values: [dim][bs + 16]
    __shared__ float red[16];
    BlockSpan s;
    if (!find_block(a.g, a.starts, a.table, a.width, a.num_blocks, a.bs, blockIdx.x, s) || s.id < 0) return;
    const bool val = blockIdx.z == 1;
    const int h = blockIdx.y, t = threadIdx.x, nt = blockDim.x;
    const T* X = val ? V : K;
    const int64_t ld = val ? ldv : ldk;
    const int cpr = a.dim / 8, nch = a.bs * cpr;
    float keep[KEEP][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int c = t + i * nt, slot = c / cpr;
        if (c < nch && slot >= s.lo && slot < s.hi) {
            load8(X + (s.row0 + slot) * ld + (int64_t)h * a.dim + 8 * (c % cpr), keep[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) m = amax_acc(m, keep[i][k]);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = amax_acc(m, __shfl_xor(m, off, 64));
    if ((t & 63) == 0) red[t >> 6] = m;
    float* scale = a.scales[val] + (int64_t)s.id * a.heads + h;
    const float S_old = s.lo > 0 ? *scale : 0.f;
    __syncthreads();
    m = 0.f;
    for (int w = 0; w < nt / 64; ++w) m = amax_acc(m, red[w]);
    float S = int8_scale(m);
    if (S_old >= S || S_old != S_old) S = S_old;
    const float inv = int8_inverse(S);
    const float ratio = S > S_old ? S_old * inv : 1.f;
    const bool recode = s.lo > 0 && ratio != 1.f;
    if (t == 0) *scale = S;
    int8_t* codes = a.codes[val] + ((int64_t)s.id * a.heads + h) * a.bs * a.dim;
    if (!val) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = t + i * nt, slot = c / cpr;
            if (c >= nch) break;
            uint2* p = (uint2*)(codes + 8 * c);
            if (slot >= s.lo && slot < s.hi) {
                *p = codes8(keep[i], inv);
            } else if (slot < s.lo && recode) {
                const uint2 w = *p;
                *p = make_uint2(recode4(w.x, ratio), recode4(w.y, ratio));
            }
        }
        return;
    }
    // values: the new codes go through LDS into channel-major order, then
    // 16 slots of a channel at a time into the block
    const int pitch = a.bs + 16;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int c = t + i * nt, slot = c / cpr;
        if (c < nch && slot >= s.lo && slot < s.hi) {
            const uint2 w = codes8(keep[i], inv);
            unsigned char* p = image + 8 * (c % cpr) * pitch + slot;
#pragma unroll
            for (int k = 0; k < 8; ++k) p[k * pitch] = (unsigned char)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
        }
    }
    __syncthreads();
    const int seg = a.bs / 16;
    for (int c = t; c < a.dim * seg; c += nt) {
        const int d = c / seg, s0 = 16 * (c % seg);
        uint4* p = (uint4*)(codes + d * a.bs + s0);
        uint4 w = *(const uint4*)(image + d * pitch + s0);
        if (s.lo > s0 || s.hi < s0 + 16) {       // not all of it is new
            if (s.hi <= s0 || (s.lo >= s0 + 16 && !recode)) continue;
            uint4 old = *p;
            uint32_t* n = (uint32_t*)&w;
            uint32_t* o = (uint32_t*)&old;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t keepmask = 0, oldmask = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int slot = s0 + 4 * q + k;
                    if (slot >= s.lo && slot < s.hi) keepmask |= 0xffu << (8 * k);
                    if (slot < s.lo) oldmask |= 0xffu << (8 * k);
                }
                const uint32_t r = recode ? ((recode4(o[q], ratio) & oldmask) | (o[q] & ~oldmask)) : o[q];
                n[q] = (n[q] & keepmask) | (r & ~keepmask);
            }
        }
        *p = w;
    }
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    *(uint4*)p = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                            bf16_pair(v[6], v[7]));
}

template <typename T>
__global__ __launch_bounds__(256) void kv_read_kernel(CacheArgs a, T* __restrict__ K, int64_t ldk,
                                                      T* __restrict__ V, int64_t ldv) {
    extern __shared__ __attribute__((aligned(16))) unsigned char image[];   // values: [dim][bs + 16]
    BlockSpan s;
    if (!find_block(a.g, a.starts, a.table, a.width, a.num_blocks, a.bs, blockIdx.x, s)) return;
    const bool val = blockIdx.z == 1;
    const int h = blockIdx.y, t = threadIdx.x, nt = blockDim.x;
    T* X = val ? V : K;
    const int64_t ld = val ? ldv : ldk;
    const float S = s.id >= 0 ? a.scales[val][(int64_t)s.id * a.heads + h] : __builtin_nanf("");
    const int8_t* codes = a.codes[val] + ((int64_t)std::max(s.id, 0) * a.heads + h) * a.bs * a.dim;
    const bool have = s.id >= 0;
    const int pitch = a.bs + 16, cpr = a.dim / 8;
    if (val && have) {
        const int seg = a.bs / 16;
        for (int c = t; c < a.dim * seg; c += nt) {
            const int d = c / seg, s0 = 16 * (c % seg);
            *(uint4*)(image + d * pitch + s0) = *(const uint4*)(codes + d * a.bs + s0);
        }
        __syncthreads();
    }
    for (int c = t + s.lo * cpr; c < s.hi * cpr; c += nt) {
        const int slot = c / cpr, d0 = 8 * (c % cpr);
        uint2 w = make_uint2(0u, 0u);
        if (have && !val) w = *(const uint2*)(codes + 8 * c);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int8_t q = (have && val) ? (int8_t)image[(d0 + k) * pitch + slot]
                                           : (int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
            v[k] = (float)q * S;
        }
        store8(X + (s.row0 + slot) * ld + (int64_t)h * a.dim + d0, v);
    }
}

CacheArgs cache_args(const KVCacheInt8& c, const RaggedRows& r) {
    CacheArgs a{};
    a.g.offsets = r.offsets; a.g.batch = (int)r.batch; a.g.rows = r.rows;
    a.starts = r.starts; a.table = r.table; a.width = r.width;
    a.heads = c.heads; a.dim = c.dim; a.bs = c.block; a.num_blocks = c.num_blocks;
    a.codes[0] = c.k; a.codes[1] = c.v;
    a.scales[0] = c.k_scales; a.scales[1] = c.v_scales;
    return a;
}

// units of ragged_find(mul = 1, div = bs, extra = 2)
dim3 block_grid(const KVCacheInt8& c, const RaggedRows& r) {
    return dim3((unsigned)(r.rows / c.block + 2 * r.batch), (unsigned)c.heads, 2);
}

}  // namespace

int launch_kv_write(const KVCacheInt8& c, const RaggedRows& r, int dtype, const void* K, int64_t ldk, const void* V,
                    int64_t ldv, hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    const CacheArgs a = cache_args(c, r);
    const int nt = std::max(64, c.block * c.dim / (8 * KEEP));
    const int lds = c.dim * (c.block + 16);
    if (dtype == PTQ_F32)
        hipLaunchKernelGGL(kv_write_kernel<float>, block_grid(c, r), dim3(nt), lds, st, a, (const float*)K, ldk,
                           (const float*)V, ldv);
    else
        hipLaunchKernelGGL(kv_write_kernel<uint16_t>, block_grid(c, r), dim3(nt), lds, st, a, (const uint16_t*)K, ldk,
                           (const uint16_t*)V, ldv);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

int launch_kv_read(const KVCacheInt8& c, const RaggedRows& r, int dtype, void* K, int64_t ldk, void* V, int64_t ldv,
                   hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    const CacheArgs a = cache_args(c, r);
    const int lds = c.dim * (c.block + 16);
    if (dtype == PTQ_F32)
        hipLaunchKernelGGL(kv_read_kernel<float>, block_grid(c, r), dim3(256), lds, st, a, (float*)K, ldk, (float*)V,
                           ldv);
    else
        hipLaunchKernelGGL(kv_read_kernel<uint16_t>, block_grid(c, r), dim3(256), lds, st, a, (uint16_t*)K, ldk,
                           (uint16_t*)V, ldv);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

}  // namespace ptq
