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
__device__ __forceinline__ bool find_block(const Ragged& g, const int32_t* table, int64_t width, int64_t num_blocks,
                                           int bs, int64_t unit, BlockSpan& s) {
    const RaggedUnit u = ragged_find(g, unit, 1, bs, 2);
    if (u.rows <= 0) return false;
    const int64_t start = std::max(u.start, 0), at = start / bs + u.local;
    s.b = u.b;
    s.p0 = at * bs;
    if (s.p0 >= start + u.rows) return false;
    s.lo = (int)std::max<int64_t>(start - s.p0, 0);
    s.hi = (int)std::min<int64_t>(start + u.rows - s.p0, bs);
    s.row0 = u.off + s.p0 - start;
    s.id = (at < width && u.start >= 0) ? table[s.b * width + at] : -1;
    if (s.id >= num_blocks) s.id = -1;
    return true;
}

struct CacheArgs {
    Ragged g;
    const int32_t* table; int64_t width;
    int heads, dim, bs;
    int64_t num_blocks;
    int8_t* codes[2];        // k, v
    float* scales[2];
};

__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) r |= (uint32_t)(uint8_t)(int)rintf((float)(int8_t)(w >> (8 * k)) * ratio) << (8 * k);
    return r;
}

// Both kernels give a thread 16 NV codes of one (block, head): of K 2 NV chunks
// of 8 channels of a token, per = bs dim / (16 NV) chunks apart; of V NV
// channels of 16 tokens, so that a row of the input (or output) and 16 slots
// of the block are both whole accesses and the codes change order in registers.
// NV = 4, or 2 where fp32 values are held until the block's maximum is known
// (64 of them took 115 registers a thread, and the write 29 us where NV = 2
// takes 16.5: 61 prompts, 12 heads of 64).
// What bounds both is memory, and for a few tokens their own latency: 16 chunked
// prompts of 1000 .. 4099 tokens, 8 heads of 128, bf16: 109 us, 4.6 TB/s; 16
// such sequences read back: 108 us, 5.0 TB/s; one token appended to each of 64
// sequences: 6 us. With NV = 2 the bf16 write took 118 us.
// Threads of a workgroup: `per` for each head, as many heads as make 256.
template <typename T>
constexpr int write_nv() { return sizeof(T) == 4 ? 2 : 4; }
constexpr int READ_NV = 4;
struct HeadThreads {
    int h, q;            // head, thread within the head
    int quad, seg;       // V: channels NV quad .., slots 16 seg ..
};
template <int NV>
__device__ __forceinline__ HeadThreads head_threads(const CacheArgs& a, int per) {
    HeadThreads x;
    const int t = threadIdx.x;
    x.h = blockIdx.y * (blockDim.x / per) + t / per;
    x.q = t % per;
    x.quad = x.q % (a.dim / NV);
    x.seg = x.q / (a.dim / NV);
    return x;
}

// grid (units, groups of heads, 2): z = 0 keys, 1 values
template <typename T>
__global__ __launch_bounds__(sizeof(T) == 4 ? 1024 : 512) void kv_write_kernel(CacheArgs a, int per, const T* __restrict__ K, int64_t ldk,
                                                       const T* __restrict__ V, int64_t ldv) {
    constexpr int NV = write_nv<T>();
    __shared__ float red[16];
    BlockSpan s;
    if (!find_block(a.g, a.table, a.width, a.num_blocks, a.bs, blockIdx.x, s) || s.id < 0) return;
    const bool val = blockIdx.z == 1;
    const HeadThreads x = head_threads<NV>(a, per);
    const bool live = x.h < a.heads;
    const int64_t ld = val ? ldv : ldk;
    const T* X = (val ? V : K) + s.row0 * ld + (int64_t)std::min(x.h, a.heads - 1) * a.dim;
    const int cpr = a.dim / 8;
    // all loads at once: a slot that is not the call's reads the nearest one that is (the maximum is the same)
    float v[16 * NV];      // K: [chunk][channel], V: [slot][channel]
    if (!val) {
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) {
            const int c = x.q + i * per, slot = std::min(std::max(c / cpr, s.lo), s.hi - 1);
            load8(X + slot * ld + 8 * (c % cpr), *(float (*)[8])&v[8 * i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int slot = std::min(std::max(16 * x.seg + i, s.lo), s.hi - 1);
            load_n(X + slot * ld + NV * x.quad, *(float (*)[NV])&v[NV * i]);
        }
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16 * NV; ++i) m = amax_acc(m, v[i]);
    float* scale = a.scales[val] + (int64_t)s.id * a.heads + x.h;
    const float S_old = live && s.lo > 0 ? *scale : 0.f;
    for (int off = (per < 64 ? per : 64) / 2; off > 0; off >>= 1) m = amax_acc(m, __shfl_xor(m, off, 64));
    if (per > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        const int first = threadIdx.x / per * (per / 64);
        m = 0.f;
        for (int w = 0; w < per / 64; ++w) m = amax_acc(m, red[first + w]);
    }
    if (!live) return;
    float S = int8_scale(m);
    if (S_old >= S || S_old != S_old) S = S_old;
    const float inv = int8_inverse(S);
    const float ratio = S > S_old ? S_old * inv : 1.f;
    const bool recode = s.lo > 0 && ratio != 1.f;
    if (x.q == 0) *scale = S;
    int8_t* codes = a.codes[val] + ((int64_t)s.id * a.heads + x.h) * a.bs * a.dim;
    if (!val) {
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) {
            const int c = x.q + i * per, slot = c / cpr;
            uint2* p = (uint2*)(codes + 8 * c);
            if (slot >= s.lo && slot < s.hi) {
                *p = int8_code8(*(float (*)[8])&v[8 * i], inv);
            } else if (slot < s.lo && recode) {
                const uint2 w = *p;
                *p = make_uint2(recode4(w.x, ratio), recode4(w.y, ratio));
            }
        }
        return;
    }
    const int s0 = 16 * x.seg;
    const bool all = s.lo <= s0 && s.hi >= s0 + 16;
    if (s.hi <= s0 || (s.lo >= s0 + 16 && !recode)) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint4* p = (uint4*)(codes + (NV * x.quad + k) * a.bs + s0);
        uint32_t n[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            n[q] = int8_code4(v[(4 * q) * NV + k], v[(4 * q + 1) * NV + k], v[(4 * q + 2) * NV + k], v[(4 * q + 3) * NV + k], inv);
        if (!all) {      // slots before lo keep their codes, at the new scale; those from hi on their bytes
            const uint4 w = *p;
            const uint32_t old[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t fresh = 0, held = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int slot = s0 + 4 * q + e;
                    if (slot >= s.lo && slot < s.hi) fresh |= 0xffu << (8 * e);
                    if (slot < s.lo) held |= 0xffu << (8 * e);
                }
                const uint32_t o = recode ? (recode4(old[q], ratio) & held) | (old[q] & ~held) : old[q];
                n[q] = (n[q] & fresh) | (o & ~fresh);
            }
        }
        *p = make_uint4(n[0], n[1], n[2], n[3]);
    }
}

// byte k of w as a number, times S
__device__ __forceinline__ float value_of(uint32_t w, int k, float S) { return (float)(int8_t)(w >> (8 * k)) * S; }

template <typename T>
__global__ __launch_bounds__(512) void kv_read_kernel(CacheArgs a, int per, T* __restrict__ K, int64_t ldk,
                                                      T* __restrict__ V, int64_t ldv) {
    BlockSpan s;
    if (!find_block(a.g, a.table, a.width, a.num_blocks, a.bs, blockIdx.x, s)) return;
    const bool val = blockIdx.z == 1, have = s.id >= 0;
    const HeadThreads x = head_threads<READ_NV>(a, per);
    if (x.h >= a.heads) return;
    const int64_t ld = val ? ldv : ldk, at = (int64_t)(have ? s.id : 0) * a.heads + x.h;
    T* X = (val ? V : K) + s.row0 * ld + (int64_t)x.h * a.dim;
    const int8_t* codes = a.codes[val] + at * a.bs * a.dim;
    const float S = have ? a.scales[val][at] : __builtin_nanf("");
    if (!val) {
        const int cpr = a.dim / 8;
        uint2 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = have ? *(const uint2*)(codes + 8 * (x.q + i * per)) : make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = x.q + i * per, slot = c / cpr;
            if (slot < s.lo || slot >= s.hi) continue;
            T* p = X + slot * ld + 8 * (c % cpr);
            if constexpr (sizeof(T) == 2) {
                *(uint4*)p = make_uint4(bf16_pair(value_of(w[i].x, 0, S), value_of(w[i].x, 1, S)),
                                        bf16_pair(value_of(w[i].x, 2, S), value_of(w[i].x, 3, S)),
                                        bf16_pair(value_of(w[i].y, 0, S), value_of(w[i].y, 1, S)),
                                        bf16_pair(value_of(w[i].y, 2, S), value_of(w[i].y, 3, S)));
            } else {
                store4(p, value_of(w[i].x, 0, S), value_of(w[i].x, 1, S), value_of(w[i].x, 2, S), value_of(w[i].x, 3, S));
                store4(p + 4, value_of(w[i].y, 0, S), value_of(w[i].y, 1, S), value_of(w[i].y, 2, S), value_of(w[i].y, 3, S));
            }
        }
        return;
    }
    uint4 w[4];          // 16 slots of each channel
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = have ? *(const uint4*)(codes + (4 * x.quad + k) * a.bs + 16 * x.seg) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t c[4] = {((const uint32_t*)&w[0])[q], ((const uint32_t*)&w[1])[q], ((const uint32_t*)&w[2])[q],
                               ((const uint32_t*)&w[3])[q]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int slot = 16 * x.seg + 4 * q + e;
            if (slot >= s.lo && slot < s.hi)
                store4(X + slot * ld + 4 * x.quad, value_of(c[0], e, S), value_of(c[1], e, S), value_of(c[2], e, S),
                       value_of(c[3], e, S));
        }
    }
}

CacheArgs cache_args(const KVCacheInt8& c, const RaggedRows& r) {
    CacheArgs a{};
    a.g.offsets = r.offsets; a.g.starts = r.starts; a.g.batch = (int)r.batch; a.g.rows = r.rows;
    a.table = r.table; a.width = r.width;
    a.heads = c.heads; a.dim = c.dim; a.bs = c.block; a.num_blocks = c.num_blocks;
    a.codes[0] = c.k; a.codes[1] = c.v;
    a.scales[0] = c.k_scales; a.scales[1] = c.v_scales;
    return a;
}

// units of ragged_find(mul = 1, div = bs, extra = 2) x groups of heads x {K, V}, and the threads of a workgroup
struct Launch {
    dim3 grid, block;
    int per;
};
int block_launch(const char* fn, const KVCacheInt8& c, const RaggedRows& r, int nv, Launch& l) {
    l.per = c.block * c.dim / (16 * nv);
    const int nt = std::max(l.per, std::min(256, (int)cdiv((int64_t)l.per * c.heads, 64) * 64));
    const int64_t units = r.rows / c.block + 2 * r.batch;
    // a launch of 2^32 threads or more wraps without an error: only some of its workgroups run
    if (units > (((int64_t)1 << 32) - 1) / nt) {
        set_error("%s: rows = %lld, batch = %lld: %lld workgroups of %d threads are too many for a launch", fn,
                  (long long)r.rows, (long long)r.batch, (long long)units, nt);
        return PTQ_EINVAL;
    }
    l.block = dim3((unsigned)nt);
    l.grid = dim3((unsigned)units, (unsigned)cdiv(c.heads, nt / l.per), 2);
    return PTQ_OK;
}

}  // namespace

int launch_kv_write(const KVCacheInt8& c, const RaggedRows& r, int dtype, const void* K, int64_t ldk, const void* V,
                    int64_t ldv, hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    const CacheArgs a = cache_args(c, r);
    Launch l;
    PTQ_TRY(block_launch("kv_cache_write_int8", c, r, dtype == PTQ_F32 ? write_nv<float>() : write_nv<uint16_t>(), l));
    if (dtype == PTQ_F32)
        hipLaunchKernelGGL(kv_write_kernel<float>, l.grid, l.block, 0, st, a, l.per, (const float*)K, ldk, (const float*)V,
                           ldv);
    else
        hipLaunchKernelGGL(kv_write_kernel<uint16_t>, l.grid, l.block, 0, st, a, l.per, (const uint16_t*)K, ldk,
                           (const uint16_t*)V, ldv);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

int launch_kv_read(const KVCacheInt8& c, const RaggedRows& r, int dtype, void* K, int64_t ldk, void* V, int64_t ldv,
                   hipStream_t st) {
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    const CacheArgs a = cache_args(c, r);
    Launch l;
    PTQ_TRY(block_launch("kv_cache_read_int8", c, r, READ_NV, l));
    if (dtype == PTQ_F32)
        hipLaunchKernelGGL(kv_read_kernel<float>, l.grid, l.block, 0, st, a, l.per, (float*)K, ldk, (float*)V, ldv);
    else
        hipLaunchKernelGGL(kv_read_kernel<uint16_t>, l.grid, l.block, 0, st, a, l.per, (uint16_t*)K, ldk, (uint16_t*)V,
                           ldv);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

}  // namespace ptq
