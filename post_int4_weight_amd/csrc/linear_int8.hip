// Linear layer on int8 codes:
//
//   Y[t][o] = (sum_j c[t][j] w[o][j]) sx[t] sw[o] + bias[o]
//
// with w the int8 codes [out, in] of a quantizer (one scale per output
// channel: group_size = in) and c, sx the codes and scales of the activations,
// quantized token by token (quantize_tokens_int8; "int8.hpp" has the rule).
// The sums are exact: products of int8 in int32, in < 131072.
#include "int8.hpp"

#include <algorithm>

namespace ptq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ tokens --
// One workgroup per token. The row is read once: a thread keeps up to 4 chunks
// of 8 values in registers between the maximum and the codes (rows of up to
// 32768 values with 1024 threads; longer ones are read again for the rest).
constexpr int QKEEP = 4;

template <typename T, bool SMOOTH>
__global__ __launch_bounds__(1024) void quantize_tokens_kernel(const T* __restrict__ X, int64_t ldx, int in, int pad,
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
    auto store = [&](int c, const float (&v)[8]) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k >> 2] |= (uint32_t)(uint8_t)int8_code(v[k], inv) << (8 * (k & 3));
        *(uint2*)(out + 8 * c) = make_uint2(w[0], w[1]);
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
    for (int c = nch + t; c < pad / 8; c += nt) *(uint2*)(out + 8 * c) = make_uint2(0u, 0u);
}

// ----------------------------------------------------------------- product --
struct Int8GemmArgs {
    const int8_t* W; int64_t ldw; int64_t out;    // rows of the MFMA's first operand
    const int8_t* C; int64_t ldc; int64_t rows;   // and of its second
    int in;
    const float* sw; const float* sx; const float* bias;
    void* Y; int64_t ldy; int y_dtype;
};

// Accumulators of v_mfma_i32_16x16x64_i8: lane l supplies row l % 16 of each
// operand and the 16 consecutive codes at 16 (l / 16) of the 64-deep step;
// register r of lane l holds W row 4 (l / 16) + r, token l % 16, so a lane
// stores 4 consecutive outputs of one token.
__device__ __forceinline__ void store4(const Int8GemmArgs& g, int64_t o, int64_t token, i32x4 acc) {
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

// Tile of TB x TB (outputs x tokens), 4 waves of 2 x 2, KT codes per stage,
// staged through registers with every access checked: any sizes, strides of
// any multiple of 8. 16-byte chunks of a staged row are XOR-swizzled by
// (row >> 1) & 7 (128-byte rows: 16 rows at one chunk then touch every bank).
constexpr int TB = 128, KT = 128, CH = KT / 16;

__device__ __forceinline__ int swz(int r, int c) { return r * KT + 16 * (c ^ ((r >> 1) & 7)); }

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

__global__ __launch_bounds__(256) void matmul_int8_kernel(Int8GemmArgs g) {
    __shared__ __attribute__((aligned(16))) unsigned char smem[2 * TB * KT];
    unsigned char* const sw = smem;
    unsigned char* const sc = smem + TB * KT;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t tiles = cdiv(g.out, TB);
    const int64_t o0 = (blockIdx.x % tiles) * TB, r0 = (blockIdx.x / tiles) * TB;
    const int wo = (wave >> 1) * (TB / 2), wr = (wave & 1) * (TB / 2);
    const int li = lane & 15, lg = lane >> 4;
    i32x4 acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    constexpr int PER = TB * CH / 256;
    uint4 vw[PER], vc[PER];
    auto load = [&](int k0) {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int idx = t + 256 * q, r = idx / CH, c = idx % CH;
            vw[q] = load_codes(g.W, g.ldw, o0 + r, g.out, k0 + 16 * c, g.in);
            vc[q] = load_codes(g.C, g.ldc, r0 + r, g.rows, k0 + 16 * c, g.in);
        }
    };
    load(0);
    for (int k0 = 0; k0 < g.in; k0 += KT) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int idx = t + 256 * q, r = idx / CH, c = idx % CH;
            *(uint4*)(sw + swz(r, c)) = vw[q];
            *(uint4*)(sc + swz(r, c)) = vc[q];
        }
        __syncthreads();
        if (k0 + KT < g.in) load(k0 + KT);
#pragma unroll
        for (int kk = 0; kk < KT / 64; ++kk) {
            i32x4 fw[4], fc[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                fw[a] = *(const i32x4*)(sw + swz(wo + 16 * a + li, 4 * kk + lg));
                fc[a] = *(const i32x4*)(sc + swz(wr + 16 * a + li, 4 * kk + lg));
            }
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[a], fc[b], acc[a][b], 0, 0, 0);
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) store4(g, o0 + wo + 16 * a + 4 * lg, r0 + wr + 16 * b + li, acc[a][b]);
}

template <typename T>
void launch_tokens(const T* X, int64_t rows, int in, int64_t ldx, const float* s, int8_t* codes, int64_t ldc, int pad,
                   float* scales, hipStream_t st) {
    const int nt = in <= 8192 ? 256 : in <= 16384 ? 512 : 1024;
    if (s)
        hipLaunchKernelGGL((quantize_tokens_kernel<T, true>), dim3((unsigned)rows), dim3(nt), 0, st, X, ldx, in, pad, s,
                           codes, ldc, scales);
    else
        hipLaunchKernelGGL((quantize_tokens_kernel<T, false>), dim3((unsigned)rows), dim3(nt), 0, st, X, ldx, in, pad,
                           s, codes, ldc, scales);
}

}  // namespace

int launch_quantize_tokens_int8(const void* X, int x_dtype, int64_t rows, int64_t in, int64_t ldx, const float* s,
                                int8_t* codes, int64_t ldc, int64_t pad, float* scales, hipStream_t st) {
    if (rows == 0) return PTQ_OK;
    if (x_dtype == PTQ_F32)
        launch_tokens((const float*)X, rows, (int)in, ldx, s, codes, ldc, (int)pad, scales, st);
    else
        launch_tokens((const uint16_t*)X, rows, (int)in, ldx, s, codes, ldc, (int)pad, scales, st);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

size_t matmul_int8_ws_bytes(int64_t rows, int64_t out, int64_t in) {
    (void)rows; (void)out; (void)in;
    return 0;
}

int run_matmul_int8(const int8_t* A, int64_t lda, const float* a_scales, int64_t rows, const int8_t* B, int64_t ldb,
                    const float* b_scales, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y,
                    int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
    (void)ws; (void)ws_bytes;
    if (rows == 0 || out == 0) return PTQ_OK;
    Int8GemmArgs g{};
    g.W = B; g.ldw = ldb; g.out = out;
    g.C = A; g.ldc = lda; g.rows = rows;
    g.in = (int)in;
    g.sw = b_scales; g.sx = a_scales; g.bias = bias;
    g.Y = Y; g.ldy = ldy; g.y_dtype = y_dtype;
    hipLaunchKernelGGL(matmul_int8_kernel, dim3((unsigned)(cdiv(out, TB) * cdiv(rows, TB))), dim3(256), 0, st,
                       g);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

// The tokens' codes are padded with zeros to whole stages of the product.
int64_t linear_int8_ldc(int64_t in) { return cdiv(in, KT) * KT; }

size_t linear_int8_ws_bytes(int64_t rows, int64_t out, int64_t in) {
    Sizer z;
    z.take<int8_t>((size_t)(rows * linear_int8_ldc(in)));
    z.take<float>((size_t)rows);
    z.take<char>(matmul_int8_ws_bytes(rows, out, in));
    return z.bytes();
}

int run_linear_int8(const void* X, int x_dtype, int64_t rows, int64_t ldx, const float* s, const int8_t* codes,
                    int64_t ldb, const float* scales, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y,
                    int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
    if (rows == 0 || out == 0) return PTQ_OK;
    Arena a(ws, ws_bytes);
    const int64_t ldc = linear_int8_ldc(in);
    int8_t* c = a.take<int8_t>((size_t)(rows * ldc));
    float* sx = a.take<float>((size_t)rows);
    const size_t mb = matmul_int8_ws_bytes(rows, out, in);
    char* mw = a.take<char>(mb);
    PTQ_TRY(launch_quantize_tokens_int8(X, x_dtype, rows, in, ldx, s, c, ldc, ldc, sx, st));
    return run_matmul_int8(c, ldc, sx, rows, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy, mw, mb, st);
}

}  // namespace ptq
