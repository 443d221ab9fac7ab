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
#include <type_traits>

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

constexpr int KT = 128;        // codes per row and stage
constexpr int NXCD = 8;

// ---- few tokens: the weights are read once, straight into operand registers.
// A workgroup owns 16 NA outputs; its waves share the depth in runs of KT, one
// after another, so that together they read whole stretches of each row. Up
// to 16 TM tokens: each wave reads their codes (which stay in L2) next to the
// weights. The int32 partial sums meet in LDS.
template <int NA, int TM, int WAVES, int UN>
__global__ __launch_bounds__(64 * WAVES) void matmul_int8_few_kernel(Int8GemmArgs g) {
    __shared__ __attribute__((aligned(16))) i32x4 part[WAVES][NA * TM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, lg = lane >> 4;
    const int64_t o0 = (int64_t)blockIdx.x * (16 * NA);
    const int8_t* w[NA];
    const int8_t* c[TM];
#pragma unroll
    for (int a = 0; a < NA; ++a) w[a] = g.W + std::min<int64_t>(o0 + 16 * a + li, g.out - 1) * g.ldw + 16 * lg;
#pragma unroll
    for (int b = 0; b < TM; ++b) c[b] = g.C + std::min<int64_t>(16 * b + li, g.rows - 1) * g.ldc + 16 * lg;
    i32x4 acc[NA][TM];
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    const int full = g.in / KT;               // whole runs
    int s = wave;
    for (; s + (UN - 1) * WAVES < full; s += UN * WAVES) {
        i32x4 fw[UN][NA][2], fc[UN][TM][2];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t k = (int64_t)(s + u * WAVES) * KT;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int a = 0; a < NA; ++a) fw[u][a][e] = load_codes16(w[a] + k + 64 * e);
#pragma unroll
                for (int b = 0; b < TM; ++b) fc[u][b][e] = load_codes16(c[b] + k + 64 * e);
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int a = 0; a < NA; ++a)
#pragma unroll
                    for (int b = 0; b < TM; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][a][e], fc[u][b][e], acc[a][b], 0, 0, 0);
    }
    for (; s * KT < g.in; s += WAVES) {       // the last runs, the ragged one among them
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t k = (int64_t)s * KT + 64 * e;
            i32x4 fw[NA], fc[TM];
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                const uint4 x = load_codes(w[a] - 16 * lg, 0, 0, 1, k + 16 * lg, g.in);
                fw[a] = i32x4{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
            }
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                const uint4 x = load_codes(c[b] - 16 * lg, 0, 0, 1, k + 16 * lg, g.in);
                fc[b] = i32x4{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
            }
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int b = 0; b < TM; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[a], fc[b], acc[a][b], 0, 0, 0);
        }
    }
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) part[wave][a * TM + b][lane] = acc[a][b];
    __syncthreads();
    for (int q = wave; q < NA * TM; q += WAVES) {
        const int a = q / TM, b = q % TM;
        i32x4 sum = part[0][q][lane];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) sum += part[v][q][lane];
        store4(g, o0 + 16 * a + 4 * lg, 16 * b + li, sum);
    }
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

template <int TO, int TT, int WO, int WT>
__global__ __launch_bounds__(64 * WO * WT, 1) void matmul_int8_tile_kernel(Int8GemmArgs g, int tiles_o, int tiles_t) {
    constexpr int NW = WO * WT, WA = TO / WO / 16, WB = TT / WT / 16;
    constexpr int PW = TO / 8 / NW, PC = TT / 8 / NW;      // copies of 8 rows per wave and stage
    constexpr int STAGE = (TO + TT) * KT;
    constexpr int NM = WA * WB, NR = WA + WB, NL = PW + PC;
    static_assert(PW * 8 * NW == TO && PC * 8 * NW == TT && NM >= NR && NL <= NM, "tile shape");
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
    auto copy_one = [&](int s, int buf, auto qc) {
        constexpr int q = decltype(qc)::value;
        unsigned char* base = smem + buf * STAGE;
        if constexpr (q < PW) copy16(rw, base + (wave * PW + q) * 1024, vw[q], (unsigned)(s * KT));
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
    // buffer takes the copies of the stage after that.
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
    const int full = g.in / KT;
    if (full > 0) {
#pragma unroll
        for (int s = 0; s < 2; ++s) static_for<0, NL>([&](auto q) { copy_one(std::min(s, full - 1), s, q); });
        wait_copies<NL>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int q = 0; q < NR; ++q) read_one(0, 0, 0, q);
        for (int s = 0; s < full; ++s) {
            const int buf = s & 1;
#pragma unroll
            for (int q = 0; q < NR; ++q) read_one(buf, 1, 1, q);
#pragma unroll
            for (int i = 0; i < NM; ++i) mfma_one(0, i);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            if constexpr (NM > NR) __builtin_amdgcn_sched_group_barrier(0x008, NM - NR, 0);
            __builtin_amdgcn_sched_barrier(0);
            wait_copies<0>();
            __builtin_amdgcn_s_barrier();
            // past the last stage the copies repeat it into the free buffer
            const int next = std::min(s + 2, full - 1);
            static_for<0, NM>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                mfma_one(1, i);
                if constexpr (i < NR) read_one(buf ^ 1, 0, 0, i);
                static_for<i * NL / NM, (i + 1) * NL / NM>([&](auto q) { copy_one(next, buf, q); });
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        wait_copies<0>();
    }
    if (full * KT < g.in) {
        __syncthreads();
        for (int c = t; c < (TO + TT) * 8; c += 64 * NW) {
            const int r = c / 8, k = c % 8;
            const uint4 v = r < TO ? load_codes(g.W, g.ldw, o0 + r, g.out, full * KT + 16 * k, g.in)
                                   : load_codes(g.C, g.ldc, r0 + r - TO, g.rows, full * KT + 16 * k, g.in);
            *(uint4*)(smem + slot(r, k)) = v;
        }
        __syncthreads();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int q = 0; q < NR; ++q) read_one(0, half, 0, q);
#pragma unroll
            for (int i = 0; i < NM; ++i) mfma_one(0, i);
        }
    }
#pragma unroll
    for (int a = 0; a < WA; ++a)
#pragma unroll
        for (int b = 0; b < WB; ++b) store4(g, o0 + wo + 16 * a + 4 * lg, r0 + wt + 16 * b + li, acc[a][b]);
}

template <int NA, int TM, int WAVES, int UN>
void launch_few(const Int8GemmArgs& g, hipStream_t st) {
    hipLaunchKernelGGL((matmul_int8_few_kernel<NA, TM, WAVES, UN>), dim3((unsigned)cdiv(g.out, 16 * NA)),
                       dim3(64 * WAVES), 0, st, g);
}

template <int TO, int TT, int WO, int WT>
int launch_tile(const Int8GemmArgs& g, hipStream_t st) {
    constexpr int lds = 2 * (TO + TT) * KT;
    static bool ready = false;
    if (!ready) {
        PTQ_HIP(hipFuncSetAttribute((const void*)matmul_int8_tile_kernel<TO, TT, WO, WT>,
                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds));
        ready = true;
    }
    const int64_t to = cdiv(g.out, TO), tt = cdiv(g.rows, TT);
    hipLaunchKernelGGL((matmul_int8_tile_kernel<TO, TT, WO, WT>), dim3((unsigned)(cdiv(to * tt, NXCD) * NXCD)),
                       dim3(64 * WO * WT), lds, st, g, (int)to, (int)tt);
    return PTQ_OK;
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
    if (rows <= 16) launch_few<1, 1, 16, 2>(g, st);
    else if (rows <= 32) launch_few<1, 2, 16, 2>(g, st);
    else if (rows <= 48) launch_few<2, 3, 8, 2>(g, st);
    else if (rows <= 64) launch_few<2, 4, 8, 2>(g, st);
    else if (cdiv(rows, 256) * cdiv(out, 256) >= 200) PTQ_TRY((launch_tile<256, 256, 4, 2>(g, st)));
    else PTQ_TRY((launch_tile<128, 128, 2, 2>(g, st)));
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
