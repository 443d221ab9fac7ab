// Linear layer on int8 codes:
//
//   Y[t][o] = (sum_j c[t][j] w[o][j]) sx[t] sw[o] + bias[o]
//
// with w the int8 codes [out, in] of a quantizer (one scale per output
// channel: group_size = in) and c, sx the codes and scales of the activations,
// quantized token by token (quantize_tokens_int8; "int8.hpp" has the rule).
// The sums are exact: products of int8 in int32, in < 131072.
// Measured: 1 token, 4096 x 4096: 6.8 us; 37 tokens, 8192 x 28672: 43 us, the
// codes at 5.4 TB/s; 8192 tokens, 8192 x 8192: 413 .. 425 us, the product alone
// 362 .. 385 us, 2.9 .. 3.0 POP/s.
#include "int8.hpp"

#include <algorithm>
#include <type_traits>

namespace ptq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int KT = 128;        // codes per row and stage of the product
constexpr int NXCD = 8;

// ------------------------------------------------------------------ tokens --
// One workgroup per token. The row is read once: a thread keeps up to 4 chunks
// of 8 values in registers between the maximum and the codes (rows of up to
// 32768 values with 1024 threads; longer ones are read again for the rest).
constexpr int QKEEP = 4;

template <typename T, bool SMOOTH>
__global__ __launch_bounds__(1024) void quantize_tokens_kernel(const T* __restrict__ X, int64_t ldx, int in, int shift,
                                                               const float* __restrict__ s, int8_t* __restrict__ codes,
                                                               int64_t ldc, float* __restrict__ scales) {
    const int64_t row = blockIdx.x;
    const T* x = X + row * ldx;
    const int nch = in / 8, t = threadIdx.x, nt = blockDim.x;
    auto chunk = [&](int c, float (&v)[8]) {
        load8(x + 8 * c, v);
        if (SMOOTH) {
            float d[8];
            load8(s + 8 * c, d);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __fdiv_rn(v[k], d[k]);
        }
    };
    float keep[QKEEP][8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < QKEEP; ++i) {
        const int c = t + i * nt;
        if (c < nch) {
            chunk(c, keep[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) a = amax_acc(a, keep[i][k]);
        }
    }
    for (int c = t + QKEEP * nt; c < nch; c += nt) {
        float v[8];
        chunk(c, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) a = amax_acc(a, v[k]);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) a = amax_acc(a, __shfl_xor(a, off, 64));
    __shared__ float red[16];
    if ((t & 63) == 0) red[t >> 6] = a;
    __syncthreads();
    a = 0.f;
    for (int w = 0; w < nt / 64; ++w) a = amax_acc(a, red[w]);
    const float S = int8_scale(a), inv = int8_inverse(S);
    if (t == 0) scales[row] = S;
    int8_t* out = codes + row * ldc;
    const int whole = in / KT * (KT / 8);     // the last stage's codes move up by shift, zeros go before them
    auto store = [&](int c, const float (&v)[8]) {
        *(uint2*)(out + 8 * c + (c >= whole ? shift : 0)) = int8_code8(v, inv);
    };
#pragma unroll
    for (int i = 0; i < QKEEP; ++i) {
        const int c = t + i * nt;
        if (c < nch) store(c, keep[i]);
    }
    for (int c = t + QKEEP * nt; c < nch; c += nt) {
        float v[8];
        chunk(c, v);
        store(c, v);
    }
    if (t < shift / 8) *(uint2*)(out + 8 * (whole + t)) = make_uint2(0u, 0u);
}

// ----------------------------------------------------------------- product --
struct Int8GemmArgs {
    const int8_t* W; int64_t ldw; int64_t out;    // rows of the MFMA's first operand
    const int8_t* C; int64_t ldc; int64_t rows;   // and of its second
    int in;
    const float* sw; const float* sx; const float* bias;
    void* Y; int64_t ldy; int y_dtype;
    int nsplit; int* part;     // shares of the depth, their int32 sums [split][tile][value / 4][thread][4]
};

// Accumulators of v_mfma_i32_16x16x64_i8: lane l supplies row l % 16 of each
// operand and the 16 consecutive codes at 16 (l / 16) of the 64-deep step;
// register r of lane l holds W row 4 (l / 16) + r, token l % 16, so a lane
// stores 4 consecutive outputs of one token.
__device__ __forceinline__ void store_out(const Int8GemmArgs& g, int64_t o, int64_t token, i32x4 acc) {
    if (token >= g.rows) return;
    const float sx = g.sx[token];
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (o + r < g.out) y[r] = (float)acc[r] * (sx * g.sw[o + r]) + (g.bias ? g.bias[o + r] : 0.f);
    const int64_t at = token * g.ldy + o;
    if (g.y_dtype == PTQ_F32) {
        float* p = (float*)g.Y + at;
        if (o + 4 <= g.out && ((uintptr_t)p & 15u) == 0) {
            *(float4*)p = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (o + r < g.out) p[r] = y[r];
        }
    } else {
        uint16_t* p = (uint16_t*)g.Y + at;
        if (o + 4 <= g.out && ((uintptr_t)p & 7u) == 0) {
            *(uint2*)p = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (o + r < g.out) p[r] = (uint16_t)bf16_of(y[r]);
        }
    }
}

// 16 codes at k of a row; 0 past `in` (a multiple of 8) and for rows that are not there
__device__ __forceinline__ uint4 load_codes(const int8_t* P, int64_t ld, int64_t r, int64_t rows, int64_t k, int in) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && k < in) {
        const int8_t* p = P + r * ld + k;
        const uint2 a = *(const uint2*)p;
        v.x = a.x;
        v.y = a.y;
        if (k + 16 <= in) {
            const uint2 b = *(const uint2*)(p + 8);
            v.z = b.x;
            v.w = b.y;
        }
    }
    return v;
}

// 16 codes at an address that is a multiple of 8 (one 16-byte load)
struct __attribute__((aligned(8))) Codes16 {
    uint32_t w[4];
};
__device__ __forceinline__ i32x4 load_codes16(const int8_t* p) {
    const Codes16 c = *(const Codes16*)p;
    return i32x4{(int)c.w[0], (int)c.w[1], (int)c.w[2], (int)c.w[3]};
}

// ---- few tokens: the weights are read once, straight into operand registers.
// A workgroup owns 16 outputs; its 16 waves share the depth in runs of KT, one
// after another, so that together they read whole stretches of each row. Each
// wave reads the tokens' codes (which stay in L2, or LDS) next to the weights.
// The int32 partial sums meet in LDS.
constexpr int FW = 16, FUN = 2;      // waves; runs of a wave in flight

// the weights of runs s, s + FW, ... of this lane
__device__ __forceinline__ void load_runs(const int8_t* w, int s, i32x4 (&fw)[FUN][2]) {
#pragma unroll
    for (int u = 0; u < FUN; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) fw[u][e] = load_codes16(w + (int64_t)(s + u * FW) * KT + 64 * e);
}

// fw holds the first runs if there are FUN whole ones; codes(k): the lane's 16 codes at k, with k + 16 <= the
// codes' own end for whole runs, and tail(k) the same anywhere
template <typename F, typename G>
__device__ __forceinline__ i32x4 sum_runs(const int8_t* w, int in, int wave, int lg, i32x4 (&fw)[FUN][2], F&& codes, G&& tail) {
    i32x4 acc = i32x4{0, 0, 0, 0};
    const int full = in / KT;
    int s = wave;
    while (s + (FUN - 1) * FW < full) {
        i32x4 fc[FUN][2];
#pragma unroll
        for (int u = 0; u < FUN; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) fc[u][e] = codes((s + u * FW) * KT + 64 * e);
#pragma unroll
        for (int u = 0; u < FUN; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][e], fc[u][e], acc, 0, 0, 0);
        s += FUN * FW;
        if (s + (FUN - 1) * FW < full) load_runs(w, s, fw);
    }
    for (; s * KT < in; s += FW) {       // the last runs, the ragged one among them
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = s * KT + 64 * e;
            const uint4 x = load_codes(w - 16 * lg, 0, 0, 1, k + 16 * lg, in);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{(int)x.x, (int)x.y, (int)x.z, (int)x.w}, tail(k), acc, 0, 0, 0);
        }
    }
    return acc;
}

__global__ __launch_bounds__(64 * FW) void matmul_int8_few_kernel(Int8GemmArgs g, unsigned strips) {
    __shared__ __attribute__((aligned(16))) i32x4 part[FW][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, lg = lane >> 4;
    const int64_t o0 = (int64_t)(blockIdx.x % strips) * 16, r0 = (int64_t)(blockIdx.x / strips) * 16;
    const int8_t* w = g.W + std::min<int64_t>(o0 + li, g.out - 1) * g.ldw + 16 * lg;
    const int8_t* c = g.C + std::min<int64_t>(r0 + li, g.rows - 1) * g.ldc + 16 * lg;
    i32x4 fw[FUN][2];
    if (wave + (FUN - 1) * FW < g.in / KT) load_runs(w, wave, fw);
    part[wave][lane] = sum_runs(w, g.in, wave, lg, fw, [&](int k) { return load_codes16(c + k); },
                                [&](int k) {
                                    const uint4 x = load_codes(c - 16 * lg, 0, 0, 1, k + 16 * lg, g.in);
                                    return i32x4{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
                                });
    __syncthreads();
    if (wave) return;
    i32x4 sum = part[0][lane];
#pragma unroll
    for (int v = 1; v < FW; ++v) sum += part[v][lane];
    store_out(g, o0 + 4 * lg, r0 + li, sum);
}

// The same with the tokens quantized in every workgroup, while its first
// weights are on their way: one launch instead of two, for up to 16 tokens of
// up to FUSED_MOST values together (their codes stay in LDS). 2^RL >= rows: the waves that share a row are FW / 2^RL.
constexpr int FUSED_MOST = 65536, FKEEP = FUSED_MOST / 8 / (64 * FW);
__host__ __device__ inline int fused_pitch(int in) { return (in + KT - 1) / KT * KT + 16; }   // rows start on different banks

template <typename T, bool SMOOTH>
__global__ __launch_bounds__(64 * FW) void linear_int8_few_kernel(Int8GemmArgs g, const T* __restrict__ X, int64_t ldx,
                                                                  const float* __restrict__ s, int rl) {
    extern __shared__ __attribute__((aligned(16))) unsigned char codes[];
    __shared__ __attribute__((aligned(16))) i32x4 part[FW][64];
    __shared__ float red[FW], sx[FW];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, lg = lane >> 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16;
    const int8_t* w = g.W + std::min<int64_t>(o0 + li, g.out - 1) * g.ldw + 16 * lg;
    i32x4 fw[FUN][2];
    if (wave + (FUN - 1) * FW < g.in / KT) load_runs(w, wave, fw);

    const int wpr = FW >> rl, row = wave / wpr, nch = g.in / 8, pitch = fused_pitch(g.in);
    const bool have = row < g.rows;
    float keep[FKEEP][8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < FKEEP; ++i) {
        const int c = (wave % wpr + i * wpr) * 64 + lane;
        if (have && c < nch) {
            load8(X + row * ldx + 8 * c, keep[i]);
            if (SMOOTH) {
                float d[8];
                load8(s + 8 * c, d);
#pragma unroll
                for (int k = 0; k < 8; ++k) keep[i][k] = __fdiv_rn(keep[i][k], d[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) a = amax_acc(a, keep[i][k]);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) a = amax_acc(a, __shfl_xor(a, off, 64));
    if (lane == 0) red[wave] = a;
    __syncthreads();
    a = 0.f;
    for (int v = 0; v < wpr; ++v) a = amax_acc(a, red[row * wpr + v]);
    const float S = int8_scale(a), inv = int8_inverse(S);
    if (lane == 0 && wave % wpr == 0) sx[row] = S;
    if (have) {
        unsigned char* out = codes + row * pitch;
#pragma unroll
        for (int i = 0; i < FKEEP; ++i) {
            const int c = (wave % wpr + i * wpr) * 64 + lane;
            if (c < nch) *(uint2*)(out + 8 * c) = int8_code8(keep[i], inv);
        }
        if (wave % wpr == 0 && nch + lane < (pitch - 16) / 8) *(uint2*)(out + 8 * (nch + lane)) = make_uint2(0u, 0u);
    }
    __syncthreads();
    const unsigned char* c = codes + std::min(li, (int)g.rows - 1) * pitch + 16 * lg;
    auto at = [&](int k) { return *(const i32x4*)(c + k); };
    part[wave][lane] = sum_runs(w, g.in, wave, lg, fw, at, at);
    __syncthreads();
    if (wave) return;
    i32x4 sum = part[0][lane];
#pragma unroll
    for (int v = 1; v < FW; ++v) sum += part[v][lane];
    g.sx = sx;
    store_out(g, o0 + 4 * lg, li, sum);
}

// ---- many tokens: tiles of TO outputs x TT tokens, WO x WT waves, stages of
// KT codes copied straight into LDS (16 bytes a lane, no registers), two
// stages in flight. Staged rows are 128 bytes; the 16-byte chunk c of row r
// sits in slot c ^ ((r >> 1) & 7), so the 16 rows that an operand fetch reads
// at one chunk touch every bank; the copy puts it there by choosing which
// chunk each lane fetches. Rows past the end repeat the last one (their
// outputs are dropped). The ragged end of `in` goes through registers, checked.
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ int slot(int r, int c) { return r * KT + 16 * (c ^ ((r >> 1) & 7)); }

// f(integral_constant<int, I>) for I = B .. E - 1, in order
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// 16 bytes a lane from resource r at voff + soff into LDS at base + 16 lane
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, unsigned char* base, unsigned voff, unsigned soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)base, 16, voff, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_copies() {   // vmcnt <= N, lgkmcnt = 0
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Tiles in the order they are taken: strips of 8 tiles of outputs, column by
// column, and a contiguous share of that for each XCD (workgroup b runs on
// XCD b % 8), whose L2 then serves about 8 x 4 tiles' operands at a time.
__device__ __forceinline__ bool tile_of(unsigned b, int to, int tt, int& o, int& r) {
    const int n = to * tt, per = (n + NXCD - 1) / NXCD;
    const int i = (int)(b % NXCD) * per + (int)(b / NXCD);
    if ((int)(b / NXCD) >= per || i >= n) return false;
    const int strip = i / (8 * tt), left = std::min(8, to - 8 * strip), j = i - strip * 8 * tt;
    o = 8 * strip + j % left;
    r = j / left;
    return true;
}

// Outputs of 16 tokens x 16 WA outputs of a wave, from accumulators to rows of
// Y through the wave's own piece of LDS: a row is then written in whole
// stretches (the accumulators hold 4 outputs of one token a lane: 8 bytes in
// bf16), by single elements where Y's rows are not aligned.
template <int WA>
constexpr int rows_bytes() { return 16 * (16 * WA + 4) * 4; }

template <int WA, typename F>
__device__ __forceinline__ void store_rows(const Int8GemmArgs& g, int64_t o0, int64_t r0, unsigned char* lds, F&& acc) {
    constexpr int OW = 16 * WA, PITCH = OW + 4;
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    int* S = (int*)lds;
#pragma unroll
    for (int a = 0; a < WA; ++a) *(i32x4*)(S + li * PITCH + 16 * a + 4 * lg) = acc(a);
    __builtin_amdgcn_wave_barrier();
    const int rows = (int)std::min<int64_t>(16, g.rows - r0);
    const int e = g.y_dtype == PTQ_F32 ? 4 : 2;
    if (((uintptr_t)g.Y | (uint64_t)g.ldy * e) % (4 * e) == 0 && o0 + OW <= g.out) {
        constexpr int PR = OW / 4, RI = 64 / PR;      // lanes per row, rows at a time
        const int o = 4 * (lane % PR);
        float sw[4], bias[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sw[k] = g.sw[o0 + o + k];
            bias[k] = g.bias ? g.bias[o0 + o + k] : 0.f;
        }
#pragma unroll
        for (int r = lane / PR; r < 16; r += RI) {
            if (r >= rows) break;
            const i32x4 x = *(const i32x4*)(S + r * PITCH + o);
            const float sx = g.sx[r0 + r];
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = (float)x[k] * (sx * sw[k]) + bias[k];
            const int64_t at = (r0 + r) * g.ldy + o0 + o;
            if (e == 4) *(float4*)((float*)g.Y + at) = make_float4(y[0], y[1], y[2], y[3]);
            else *(uint2*)((uint16_t*)g.Y + at) = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
        }
    } else {
        constexpr int PR = OW < 64 ? OW : 64, RI = 64 / PR;
        for (int o = lane % PR; o < OW; o += PR) {
            if (o0 + o >= g.out) break;
            const float sw = g.sw[o0 + o], bias = g.bias ? g.bias[o0 + o] : 0.f;
#pragma unroll 4
            for (int r = lane / PR; r < rows; r += RI) {
                const float y = (float)S[r * PITCH + o] * (g.sx[r0 + r] * sw) + bias;
                const int64_t at = (r0 + r) * g.ldy + o0 + o;
                if (e == 4) ((float*)g.Y)[at] = y;
                else ((uint16_t*)g.Y)[at] = (uint16_t)bf16_of(y);
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
}

// The tokens' codes come in stages of their own (see tile_ldc): whole stages
// of KT, then, where `in` leaves a rest, one with the last KT codes of the row
// of which those that an earlier stage had are zero. The weights' last stage
// then simply starts at in - KT: no access needs a check. in >= KT.
template <int TO, int TT, int WO, int WT, int NST>
__global__ __launch_bounds__(64 * WO * WT, 1) void matmul_int8_tile_kernel(Int8GemmArgs g, int tiles_o, int tiles_t) {
    constexpr int NW = WO * WT, WA = TO / WO / 16, WB = TT / WT / 16;
    constexpr int PW = TO / 8 / NW, PC = TT / 8 / NW;      // copies of 8 rows per wave and stage
    constexpr int STAGE = (TO + TT) * KT;
    constexpr int NM = WA * WB, NR = WA + WB, NL = PW + PC;
    static_assert(PW * 8 * NW == TO && PC * 8 * NW == TT && NST >= 2, "tile shape");
    static_assert(NW * rows_bytes<WA>() <= NST * STAGE, "epilogue fits the stages");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    int to, tt;
    if (!tile_of(blockIdx.x, tiles_o, tiles_t, to, tt)) return;
    const int64_t o0 = (int64_t)to * TO, r0 = (int64_t)tt * TT;
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wo = (wave / WT) * (TO / WO), wt = (wave % WT) * (TT / WT);
    const int li = lane & 15, lg = lane >> 4;

    // byte offsets of this lane's copies from the tile's first row
    __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)(g.W + o0 * g.ldw), (short)0, 0x7fffffff, 0x00020000);
    __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc((void*)(g.C + r0 * g.ldc), (short)0, 0x7fffffff, 0x00020000);
    unsigned vw[PW], vc[PC];
#pragma unroll
    for (int q = 0; q < PW; ++q) {
        const int r = 8 * (wave * PW + q) + (lane >> 3);
        vw[q] = (unsigned)(std::min<int64_t>(r, g.out - 1 - o0) * g.ldw + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
    }
#pragma unroll
    for (int q = 0; q < PC; ++q) {
        const int r = 8 * (wave * PC + q) + (lane >> 3);
        vc[q] = (unsigned)(std::min<int64_t>(r, g.rows - 1 - r0) * g.ldc + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
    }
    const int stages = (g.in + KT - 1) / KT;
    auto copy_one = [&](int s, int buf, auto qc) {
        constexpr int q = decltype(qc)::value;
        unsigned char* base = smem + buf * STAGE;
        if constexpr (q < PW) copy16(rw, base + (wave * PW + q) * 1024, vw[q], (unsigned)std::min(s * KT, g.in - KT));
        else copy16(rc, base + TO * KT + (wave * PC + q - PW) * 1024, vc[q - PW], (unsigned)(s * KT));
    };

    i32x4 acc[WA][WB];
#pragma unroll
    for (int a = 0; a < WA; ++a)
#pragma unroll
        for (int b = 0; b < WB; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    // Pipeline over the two 64-deep halves of a stage: the fragments of the
    // next half are read while this half's products run. The barrier sits
    // before a stage's second half, whose fragments are in registers by then:
    // past it the next stage has landed for every wave, and this stage's
    // buffer takes the copies of the stage NST later.
    i32x4 fw[2][WA], fc[2][WB];
    auto read_one = [&](int buf, int half, int set, int q) {
        const unsigned char* S = smem + buf * STAGE;
        if (q == 0) fw[set][0] = *(const i32x4*)(S + slot(wo + li, 4 * half + lg));
        else if (q <= WB) fc[set][q - 1] = *(const i32x4*)(S + TO * KT + slot(wt + 16 * (q - 1) + li, 4 * half + lg));
        else fw[set][q - WB] = *(const i32x4*)(S + slot(wo + 16 * (q - WB) + li, 4 * half + lg));
    };
    auto mfma_one = [&](int set, int i) {
        acc[i / WB][i % WB] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[set][i / WB], fc[set][i % WB], acc[i / WB][i % WB], 0, 0, 0);
    };
    // this split's stages: an even share
    const int first = (int)((int64_t)stages * blockIdx.y / g.nsplit), last = (int)((int64_t)stages * (blockIdx.y + 1) / g.nsplit);
#pragma unroll
    for (int s = 0; s < NST; ++s) static_for<0, NL>([&](auto q) { copy_one(std::min(first + s, last - 1), s, q); });
    wait_copies<(NST - 1) * NL>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int q = 0; q < NR; ++q) read_one(0, 0, 0, q);
    int buf = 0;
    for (int s = first; s < last; ++s) {
        const int after = buf + 1 == NST ? 0 : buf + 1;
#pragma unroll
        for (int q = 0; q < NR; ++q) read_one(buf, 1, 1, q);
#pragma unroll
        for (int i = 0; i < NM; ++i) mfma_one(0, i);
#pragma unroll
        for (int i = 0; i < NR && i < NM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if constexpr (NM > NR) __builtin_amdgcn_sched_group_barrier(0x008, NM - NR, 0);
        __builtin_amdgcn_sched_barrier(0);
        wait_copies<(NST - 2) * NL>();
        __builtin_amdgcn_s_barrier();
        // past the last stage the copies repeat it into the free buffer
        const int next = std::min(s + NST, last - 1);
        static_for<0, NM>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            mfma_one(1, i);
            if constexpr (i < NR) read_one(after, 0, 0, i);
            static_for<i * NL / NM, (i + 1) * NL / NM>([&](auto q) { copy_one(next, buf, q); });
            __builtin_amdgcn_sched_barrier(0);
        });
        static_for<NM, NR>([&](auto q) { read_one(after, 0, 0, decltype(q)::value); });
        buf = after;
    }
    wait_copies<0>();
    if (g.nsplit > 1) {
        i32x4* p = (i32x4*)g.part + ((int64_t)blockIdx.y * tiles_o * tiles_t + (int64_t)tt * tiles_o + to) * (TO * TT / 4) + t;
#pragma unroll
        for (int b = 0; b < WB; ++b)
#pragma unroll
            for (int a = 0; a < WA; ++a) p[(b * WA + a) * (64 * NW)] = acc[a][b];
        return;
    }
    __syncthreads();
    unsigned char* mine = smem + wave * rows_bytes<WA>();
#pragma unroll
    for (int b = 0; b < WB; ++b)
        if (r0 + wt + 16 * b < g.rows) store_rows<WA>(g, o0 + wo, r0 + wt + 16 * b, mine, [&](int a) { return acc[a][b]; });
}

// Sum of the splits of a tile, 16 tokens of each wave at a time.
template <int TO, int TT, int WO, int WT>
__global__ __launch_bounds__(64 * WO * WT) void matmul_int8_join_kernel(Int8GemmArgs g, int tiles_o, int tiles_t) {
    constexpr int NW = WO * WT, WA = TO / WO / 16, WB = TT / WT / 16;
    __shared__ __attribute__((aligned(16))) unsigned char lds[NW * rows_bytes<WA>()];
    const int b = blockIdx.x % WB, tile = blockIdx.x / WB, t = threadIdx.x, wave = t >> 6;
    const int64_t o0 = (int64_t)(tile % tiles_o) * TO + (wave / WT) * (TO / WO);
    const int64_t r0 = (int64_t)(tile / tiles_o) * TT + (wave % WT) * (TT / WT) + 16 * b;
    if (r0 >= g.rows) return;
    const int64_t step = (int64_t)tiles_o * tiles_t * (TO * TT / 4);
    const i32x4* p = (const i32x4*)g.part + (int64_t)tile * (TO * TT / 4) + b * WA * (64 * NW) + t;
    i32x4 sum[WA];
#pragma unroll
    for (int a = 0; a < WA; ++a) sum[a] = p[a * (64 * NW)];
    for (int s = 1; s < g.nsplit; ++s)
#pragma unroll
        for (int a = 0; a < WA; ++a) sum[a] += p[s * step + a * (64 * NW)];
    store_rows<WA>(g, o0, r0, lds + wave * rows_bytes<WA>(), [&](int a) { return sum[a]; });
}

// f(part) for parts of the product, of whole tiles of to x tt, that a launch with one workgroup of that many threads a
// tile takes (it has to have fewer than 2^32): one part, but for billions of outputs.
template <typename F>
void for_parts(const Int8GemmArgs& g, int to, int tt, int threads, F&& f) {
    const int64_t most = ((int64_t)1 << 31) / threads, e = g.y_dtype == PTQ_F32 ? 4 : 2;
    const int64_t no = std::min(cdiv(g.out, to), most), step_o = no * to, step_t = std::max<int64_t>(1, most / no) * tt;
    for (int64_t r = 0; r < g.rows; r += step_t)
        for (int64_t o = 0; o < g.out; o += step_o) {
            Int8GemmArgs part = g;
            part.W += o * g.ldw;
            part.sw += o;
            if (g.bias) part.bias += o;
            part.out = std::min(g.out - o, step_o);
            if (g.C) part.C += r * g.ldc;
            if (g.sx) part.sx += r;
            part.rows = std::min(g.rows - r, step_t);
            part.Y = (char*)g.Y + (r * g.ldy + o) * e;
            f(part);
        }
}

void launch_few(const Int8GemmArgs& g, hipStream_t st) {
    for_parts(g, 16, 16, 64 * FW, [&](const Int8GemmArgs& part) {
        const int64_t strips = cdiv(part.out, 16);
        hipLaunchKernelGGL(matmul_int8_few_kernel, dim3((unsigned)(strips * cdiv(part.rows, 16))), dim3(64 * FW), 0, st,
                           part, (unsigned)strips);
    });
}

// ceil(log2(rows)) if the fused kernel takes them, else -1
int fused_rows_log2(int64_t rows, int64_t in) {
    if (rows > 16) return -1;
    const int rl = rows <= 1 ? 0 : rows <= 2 ? 1 : rows <= 4 ? 2 : rows <= 8 ? 3 : 4;
    return (in << rl) <= FUSED_MOST ? rl : -1;
}

template <typename T, bool SMOOTH>
int launch_fused(const Int8GemmArgs& g, const T* X, int64_t ldx, const float* s, int rl, hipStream_t st) {
    static PerDevice ready;
    PTQ_TRY(allow_lds(ready, (const void*)linear_int8_few_kernel<T, SMOOTH>, 128 * 1024));
    for_parts(g, 16, 16, 64 * FW, [&](const Int8GemmArgs& part) {      // up to 16 tokens: parts of the outputs
        hipLaunchKernelGGL((linear_int8_few_kernel<T, SMOOTH>), dim3((unsigned)cdiv(part.out, 16)), dim3(64 * FW),
                           (unsigned)(part.rows * fused_pitch(part.in)), st, part, X, ldx, s, rl);
    });
    return PTQ_OK;
}

template <int TO, int TT, int WO, int WT, int NST>
int launch_tile(const Int8GemmArgs& g, hipStream_t st) {
    constexpr int lds = NST * (TO + TT) * KT;
    static PerDevice ready;
    PTQ_TRY(allow_lds(ready, (const void*)matmul_int8_tile_kernel<TO, TT, WO, WT, NST>, lds));
    constexpr int joins = TT / WT / 16;             // workgroups of the join for each of the product's
    for_parts(g, TO, TT, 64 * WO * WT * (g.nsplit > 1 ? joins : 1), [&](const Int8GemmArgs& part) {
        const int64_t to = cdiv(part.out, TO), tt = cdiv(part.rows, TT);
        hipLaunchKernelGGL((matmul_int8_tile_kernel<TO, TT, WO, WT, NST>),
                           dim3((unsigned)(cdiv(to * tt, NXCD) * NXCD), part.nsplit), dim3(64 * WO * WT), lds, st, part,
                           (int)to, (int)tt);
        if (part.nsplit > 1)
            hipLaunchKernelGGL((matmul_int8_join_kernel<TO, TT, WO, WT>), dim3((unsigned)(to * tt * joins)),
                               dim3(64 * WO * WT), 0, st, part, (int)to, (int)tt);
    });
    return PTQ_OK;
}

// Codes of a caller with a ragged `in`, put into stages (tile_ldc).
__global__ __launch_bounds__(256) void stage_codes_kernel(const int8_t* __restrict__ A, int64_t lda, int64_t rows, int in,
                                                          int8_t* __restrict__ C, int64_t ldc) {
    const int whole = in / KT * KT, shift = (int)ldc - in, nch = (int)(ldc / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * nch; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / nch;
        const int at = 8 * (int)(i % nch), k = at < whole ? at : at - shift;
        uint2 v = make_uint2(0u, 0u);
        if (at < whole || k >= whole) v = *(const uint2*)(A + r * lda + k);
        *(uint2*)(C + r * ldc + at) = v;
    }
}

template <typename T>
void launch_tokens(const T* X, int64_t rows, int in, int64_t ldx, const float* s, int8_t* codes, int64_t ldc, int shift,
                   float* scales, hipStream_t st) {
    const int nt = in <= 8192 ? 256 : in <= 16384 ? 512 : 1024;
    if (s)
        hipLaunchKernelGGL((quantize_tokens_kernel<T, true>), dim3((unsigned)rows), dim3(nt), 0, st, X, ldx, in, shift, s,
                           codes, ldc, scales);
    else
        hipLaunchKernelGGL((quantize_tokens_kernel<T, false>), dim3((unsigned)rows), dim3(nt), 0, st, X, ldx, in, shift,
                           s, codes, ldc, scales);
}

int launch_quantize(const void* X, int x_dtype, int64_t rows, int64_t in, int64_t ldx, const float* s, int8_t* codes,
                    int64_t ldc, int shift, float* scales, hipStream_t st) {
    constexpr int64_t MOST = (int64_t)1 << 21;      // rows of a launch, which has fewer than 2^32 threads
    for (int64_t r = 0; r < rows; r += MOST) {
        const int64_t n = std::min(rows - r, MOST);
        if (x_dtype == PTQ_F32)
            launch_tokens((const float*)X + r * ldx, n, (int)in, ldx, s, codes + r * ldc, ldc, shift, scales + r, st);
        else
            launch_tokens((const uint16_t*)X + r * ldx, n, (int)in, ldx, s, codes + r * ldc, ldc, shift, scales + r, st);
        PTQ_LAUNCH_CHECK();
    }
    return PTQ_OK;
}

// Tile shapes; us: time of a stage of one workgroup per CU. Rings are as deep
// as 160 KB of LDS allow for one workgroup a CU from 128 x 128 on (128, 144 and
// 128 KB), and for two below (60 to 80 KB each): small tiles wait for their
// copies, so 5 stages against 3 at 64 x 64: 4096 x 4096 weights, 200 tokens
// 10.8 against 14.4 us; 8 against 2 at 32 x 32.
struct Shape {
    int to, tt;
    float us;
};
constexpr Shape SHAPES[] = {{256, 256, 2.55f}, {128, 256, 1.47f}, {128, 128, 1.38f},
                            {64, 64, 0.449f},  {64, 32, 0.336f},  {32, 32, 0.193f}};
static_assert(sizeof(SHAPES) / sizeof(SHAPES[0]) == INT8_SHAPES, "a launch for each shape");

// Row stride of the tokens' codes in stages.
int64_t tile_ldc(int64_t in) { return cdiv(in, KT) * KT; }

size_t part_elems(const Int8Plan& p, int64_t rows, int64_t out) {
    if (p.few || p.nsplit == 1) return 0;
    const Shape s = SHAPES[p.shape];
    return (size_t)p.nsplit * cdiv(out, s.to) * cdiv(rows, s.tt) * s.to * s.tt;
}

// C: the tokens' codes as the plan wants them (in stages for tiles)
int run_product(const Int8Plan& p, const int8_t* C, int64_t ldc, const float* sx, int64_t rows, const int8_t* B, int64_t ldb,
                const float* sw, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y, int64_t ldy, int* part,
                hipStream_t st) {
    Int8GemmArgs g{};
    g.W = B; g.ldw = ldb; g.out = out;
    g.C = C; g.ldc = ldc; g.rows = rows;
    g.in = (int)in;
    g.sw = sw; g.sx = sx; g.bias = bias;
    g.Y = Y; g.ldy = ldy; g.y_dtype = y_dtype;
    g.nsplit = p.nsplit; g.part = part;
    if (p.few) {
        launch_few(g, st);
    } else {
        switch (p.shape) {
            case 0: PTQ_TRY((launch_tile<256, 256, 4, 2, 2>(g, st))); break;
            case 1: PTQ_TRY((launch_tile<128, 256, 2, 4, 3>(g, st))); break;
            case 2: PTQ_TRY((launch_tile<128, 128, 2, 2, 4>(g, st))); break;
            case 3: PTQ_TRY((launch_tile<64, 64, 2, 2, 5>(g, st))); break;
            case 4: PTQ_TRY((launch_tile<64, 32, 2, 2, 5>(g, st))); break;
            default: PTQ_TRY((launch_tile<32, 32, 2, 2, 8>(g, st)));
        }
    }
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

}  // namespace

// The streaming kernel serves up to 16 tokens on weights of up to 2^25 codes
// (4096 x 4096, 1 token: 6.2 us against 6.9 for 32 x 32 tiles; 8192 x 8192, 8
// tokens: 16.0 against 14.6) and depths below one stage. Otherwise the shape
// and the split with the least estimate: workgroups per CU times the stages of
// one, at least the weights at 3.88 TB/s, and for splits 5 us and the partial
// sums written and read at 2.04 TB/s. The constants are fitted to 4107 timings
// of 170 products, 1 to 4096 tokens, 255 x 2056 to 28672 x 8192 weights; the
// choice is 0.8% slower than the best of each in the mean, 14% at worst (512
// tokens, 5003 x 4104: 34.4 against 30.3 us).
Int8Plan matmul_int8_plan(int64_t rows, int64_t out, int64_t in) {
    Int8Plan p{in < KT || (rows <= 16 && out * in <= ((int64_t)1 << 25)), 0, 1};
    if (p.few) return p;
    const int64_t stages = cdiv(in, KT);
    double least = 1e300;
    for (int k = 0; k < INT8_SHAPES; ++k) {
        const Shape& h = SHAPES[k];
        const int64_t tiles = cdiv(out, h.to) * cdiv(rows, h.tt);
        for (int ns : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (ns > 1 && (stages < 4 * ns || tiles * ns > 2048)) break;
            double us = std::max((double)cdiv(tiles * ns, 256) * cdiv(stages, ns) * h.us, out * in / 3.88e6);
            if (ns > 1) us += 5.0 + (double)tiles * ns * h.to * h.tt * 8 / 2.04e6;
            if (us < least) {
                least = us;
                p.shape = k;
                p.nsplit = ns;
            }
        }
    }
    return p;
}

int launch_quantize_tokens_int8(const void* X, int x_dtype, int64_t rows, int64_t in, int64_t ldx, const float* s,
                                int8_t* codes, int64_t ldc, float* scales, hipStream_t st) {
    return launch_quantize(X, x_dtype, rows, in, ldx, s, codes, ldc, 0, scales, st);
}

size_t matmul_int8_ws_bytes(const Int8Plan& p, int64_t rows, int64_t out, int64_t in) {
    Sizer z;
    z.take<int>(part_elems(p, rows, out));
    if (!p.few && in % KT) z.take<int8_t>((size_t)(rows * tile_ldc(in)));
    return z.bytes();
}

int run_matmul_int8(const Int8Plan& p, const int8_t* A, int64_t lda, const float* a_scales, int64_t rows,
                    const int8_t* B, int64_t ldb, const float* b_scales, int64_t out, int64_t in, const float* bias,
                    int y_dtype, void* Y, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
    Arena a(ws, ws_bytes);
    int* part = a.take<int>(part_elems(p, rows, out));
    if (!p.few && in % KT) {
        const int64_t ldc = tile_ldc(in);
        int8_t* c = a.take<int8_t>((size_t)(rows * ldc));
        hipLaunchKernelGGL(stage_codes_kernel, dim3((unsigned)std::min<int64_t>(cdiv(rows * ldc, 2048), 8192)), dim3(256), 0,
                           st, A, lda, rows, (int)in, c, ldc);
        PTQ_LAUNCH_CHECK();
        A = c;
        lda = ldc;
    }
    return run_product(p, A, lda, a_scales, rows, B, ldb, b_scales, out, in, bias, y_dtype, Y, ldy, part, st);
}

size_t linear_int8_ws_bytes(int64_t rows, int64_t out, int64_t in) {
    Sizer z;
    z.take<int8_t>((size_t)(rows * tile_ldc(in)));
    z.take<float>((size_t)rows);
    z.take<int>(part_elems(matmul_int8_plan(rows, out, in), rows, out));
    return z.bytes();
}

int run_linear_int8(const void* X, int x_dtype, int64_t rows, int64_t ldx, const float* s, const int8_t* codes,
                    int64_t ldb, const float* scales, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y,
                    int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
    const Int8Plan p = matmul_int8_plan(rows, out, in);
    Arena a(ws, ws_bytes);
    const int64_t ldc = tile_ldc(in);
    int8_t* c = a.take<int8_t>((size_t)(rows * ldc));
    float* sx = a.take<float>((size_t)rows);
    int* part = a.take<int>(part_elems(p, rows, out));
    const int rl = p.few ? fused_rows_log2(rows, in) : -1;
    if (rl >= 0) {
        Int8GemmArgs g{};
        g.W = codes; g.ldw = ldb; g.out = out;
        g.rows = rows; g.in = (int)in;
        g.sw = scales; g.bias = bias;
        g.Y = Y; g.ldy = ldy; g.y_dtype = y_dtype;
        if (x_dtype == PTQ_F32)
            PTQ_TRY(s ? (launch_fused<float, true>(g, (const float*)X, ldx, s, rl, st))
                      : (launch_fused<float, false>(g, (const float*)X, ldx, s, rl, st)));
        else
            PTQ_TRY(s ? (launch_fused<uint16_t, true>(g, (const uint16_t*)X, ldx, s, rl, st))
                      : (launch_fused<uint16_t, false>(g, (const uint16_t*)X, ldx, s, rl, st)));
        PTQ_LAUNCH_CHECK();
        return PTQ_OK;
    }
    PTQ_TRY(launch_quantize(X, x_dtype, rows, in, ldx, s, c, ldc, p.few ? 0 : (int)(ldc - in), sx, st));
    return run_product(p, c, ldc, sx, rows, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy, part, st);
}

}  // namespace ptq
