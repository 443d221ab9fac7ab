// C ABI of the int8 serving operators (declared in include/ptq.h): argument
// checks, before any HIP call, and the calls into linear_int8.hip,
// kv_cache.hip and attention_int8.hip.
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "ptq_testing.h"

namespace ptq {
namespace {

#define REFUSE(...)              \
    do {                         \
        set_error(__VA_ARGS__);  \
        return PTQ_EINVAL;       \
    } while (0)

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool dtype_ok(int t) { return t == PTQ_BF16 || t == PTQ_F32; }
int64_t elems16(int dtype) { return dtype == PTQ_BF16 ? 8 : 4; }

// int32 sums of `in` products of int8 (at most 2^14 each)
constexpr int64_t MAX_IN = ((int64_t)1 << 17) - 8;
constexpr int64_t MAX_LD = (int64_t)1 << 22;      // 256 rows of codes within 32-bit offsets
constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 1;

int check_sizes(const char* fn, int64_t rows, int64_t in) {
    if (rows < 0 || rows > MAX_ROWS) REFUSE("%s: rows = %lld outside [0, 2^31)", fn, (long long)rows);
    if (in < 8 || in % 8 || in > MAX_IN)
        REFUSE("%s: in = %lld must be a multiple of 8 in [8, %lld]", fn, (long long)in, (long long)MAX_IN);
    return PTQ_OK;
}

// a [rows, in] bf16 or fp32 operand whose rows are 16-byte aligned
int check_float_rows(const char* fn, const char* name, const void* X, int dtype, int64_t in, int64_t ld) {
    if (!dtype_ok(dtype)) REFUSE("%s: dtype of %s = %d is neither PTQ_BF16 nor PTQ_F32", fn, name, dtype);
    if (!X) REFUSE("%s: %s is NULL", fn, name);
    if (!aligned16(X)) REFUSE("%s: %s is not 16-byte aligned", fn, name);
    if (ld < in || ld % elems16(dtype))
        REFUSE("%s: row stride %lld of %s: at least %lld and rows 16-byte aligned", fn, (long long)ld, name,
               (long long)in);
    return PTQ_OK;
}

int check_codes(const char* fn, const char* name, const void* p, int64_t in, int64_t ld) {
    if (!p) REFUSE("%s: %s is NULL", fn, name);
    if (!aligned16(p)) REFUSE("%s: %s is not 16-byte aligned", fn, name);
    if (ld < in || ld % 8 || ld > MAX_LD)
        REFUSE("%s: row stride %lld of %s: a multiple of 8 in [%lld, %lld]", fn, (long long)ld, name, (long long)in,
               (long long)MAX_LD);
    return PTQ_OK;
}

int check_product(const char* fn, const int8_t* B, int64_t ldb, const float* b_scales, int64_t out, int64_t in,
                  int y_dtype, const void* Y, int64_t ldy) {
    PTQ_TRY(check_codes(fn, "codes", B, in, ldb));
    if (!b_scales) REFUSE("%s: scales is NULL", fn);
    if (!dtype_ok(y_dtype)) REFUSE("%s: dtype of Y = %d is neither PTQ_BF16 nor PTQ_F32", fn, y_dtype);
    if (!Y) REFUSE("%s: Y is NULL", fn);
    if (!aligned16(Y)) REFUSE("%s: Y is not 16-byte aligned", fn);
    if (ldy < out) REFUSE("%s: row stride %lld of Y < out = %lld", fn, (long long)ldy, (long long)out);
    return PTQ_OK;
}

int check_out(const char* fn, int64_t rows, int64_t out) {
    if (out < 0 || out > MAX_ROWS) REFUSE("%s: out = %lld outside [0, 2^31)", fn, (long long)out);
    // the product's launch has at most one workgroup per 16 x 16 outputs
    if (cdiv(rows, 16) * cdiv(out, 16) > MAX_ROWS) REFUSE("%s: rows x out too large", fn);
    return PTQ_OK;
}

int check_cache(const char* fn, const KVCacheInt8& c) {
    if (c.heads < 1 || c.heads > 65535) REFUSE("%s: kv_heads = %d outside [1, 65535]", fn, c.heads);
    if (c.dim != 64 && c.dim != 128 && c.dim != 256) REFUSE("%s: head_dim = %d not in {64, 128, 256}", fn, c.dim);
    if (c.block != 16 && c.block != 32 && c.block != 64 && c.block != 128)
        REFUSE("%s: block_size = %d not in {16, 32, 64, 128}", fn, c.block);
    if (c.num_blocks < 0 || c.num_blocks > MAX_ROWS)
        REFUSE("%s: num_blocks = %lld outside [0, 2^31)", fn, (long long)c.num_blocks);
    return PTQ_OK;
}

int check_cache_pointers(const char* fn, const KVCacheInt8& c) {
    if (!c.k || !c.v || !c.k_scales || !c.v_scales) REFUSE("%s: a cache pointer is NULL", fn);
    if (!aligned16(c.k) || !aligned16(c.v)) REFUSE("%s: k_codes or v_codes is not 16-byte aligned", fn);
    return PTQ_OK;
}

int check_ragged(const char* fn, const RaggedRows& r, const char* starts, int heads) {
    if (r.rows < 0 || r.batch < 0 || r.width < 0)
        REFUSE("%s: rows, batch and table_width must not be negative", fn);
    // launches count work units of at least one row and head in 32 bits (attention: at most one workgroup of 256 threads
    // for 16 rows and one for each sequence, or half as many of 512, so below 2^32 threads)
    if ((r.rows + 2 * r.batch) > MAX_ROWS / (64 * (int64_t)heads))
        REFUSE("%s: rows = %lld, batch = %lld too large for %d heads", fn, (long long)r.rows, (long long)r.batch, heads);
    if (r.width > MAX_ROWS / 128) REFUSE("%s: table_width = %lld too large", fn, (long long)r.width);
    if (r.rows > 0 && r.batch > 0) {
        if (!r.offsets) REFUSE("%s: offsets is NULL", fn);
        if (!r.starts) REFUSE("%s: %s is NULL", fn, starts);
        if (r.width > 0 && !r.table) REFUSE("%s: block_table is NULL", fn);
    }
    return PTQ_OK;
}

// matmul_int8 with the plan given, or chosen
int matmul(const char* fn, const Int8Plan* given, const int8_t* A, int64_t lda, const float* a_scales, int64_t rows,
           const int8_t* codes, int64_t ldb, const float* scales, int64_t out, int64_t in, const float* bias,
           int y_dtype, void* Y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    PTQ_TRY(check_sizes(fn, rows, in));
    PTQ_TRY(check_out(fn, rows, out));
    if (rows == 0 || out == 0) return PTQ_OK;
    PTQ_TRY(check_codes(fn, "A", A, in, lda));
    if (!a_scales) REFUSE("%s: a_scales is NULL", fn);
    PTQ_TRY(check_product(fn, codes, ldb, scales, out, in, y_dtype, Y, ldy));
    const Int8Plan p = given ? *given : matmul_int8_plan(rows, out, in);
    const size_t need = matmul_int8_ws_bytes(p, rows, out, in);
    if (need && (!workspace || workspace_bytes < need)) {
        set_error("%s: workspace %zu bytes, need %zu", fn, workspace ? workspace_bytes : (size_t)0, need);
        return PTQ_EWORKSPACE;
    }
    if (need && !aligned16(workspace)) REFUSE("%s: workspace is not 16-byte aligned", fn);
    return run_matmul_int8(p, A, lda, a_scales, rows, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy, workspace,
                           workspace_bytes, (hipStream_t)stream);
}

// attention_int8_cache with the plan given, or chosen
int attention(const char* fn, const AttnPlan* given, const KVCacheInt8& c, const RaggedRows& r, int dtype,
              const void* Q, int64_t ldq, int heads, float scale, int causal, int64_t window, void* O, int64_t ldo,
              float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    PTQ_TRY(check_cache(fn, c));
    if (heads < 1 || heads > 65535 || heads % c.heads)
        REFUSE("%s: heads = %d must be a multiple of kv_heads = %d, at most 65535", fn, heads, c.heads);
    PTQ_TRY(check_ragged(fn, r, "seq_lens", heads));
    if (!std::isfinite(scale)) REFUSE("%s: scale is not finite", fn);
    if (causal != 0 && causal != 1) REFUSE("%s: causal = %d is neither 0 nor 1", fn, causal);
    if (window < 0) REFUSE("%s: window = %lld < 0", fn, (long long)window);
    if (window > 0 && !causal) REFUSE("%s: a window needs causal = 1", fn);
    if (r.rows == 0 || r.batch == 0) return PTQ_OK;
    PTQ_TRY(check_cache_pointers(fn, c));
    if (c.num_blocks < 1) REFUSE("%s: num_blocks = 0", fn);
    const int64_t n = (int64_t)heads * c.dim;
    PTQ_TRY(check_float_rows(fn, "Q", Q, dtype, n, ldq));
    PTQ_TRY(check_float_rows(fn, "O", O, dtype, n, ldo));
    const AttnPlan p =
        given ? *given : attention_int8_plan(r.rows, r.batch, heads, c.heads, c.dim, c.block, r.width, window);
    const size_t need = given ? attention_int8_part_bytes(p.nsplit, r.rows, heads, c.dim)
                              : attention_int8_ws_bytes(r.rows, r.batch, heads, c.heads, c.dim, c.block, r.width);
    if (need && (!workspace || workspace_bytes < need)) {
        set_error("%s: workspace %zu bytes, need %zu", fn, workspace ? workspace_bytes : (size_t)0, need);
        return PTQ_EWORKSPACE;
    }
    if (need && !aligned16(workspace)) REFUSE("%s: workspace is not 16-byte aligned", fn);
    return run_attention_int8(p, c, r, dtype, Q, ldq, heads, scale, causal, window, O, ldo, lse, workspace,
                              workspace_bytes, (hipStream_t)stream);
}

}  // namespace
}  // namespace ptq

using namespace ptq;

extern "C" {

int quantize_tokens_int8(const void* X, int x_dtype, int64_t rows, int64_t in, int64_t ldx, const float* s,
                         int8_t* codes, int64_t ldc, float* scales, void* stream) {
    const char* fn = "quantize_tokens_int8";
    PTQ_TRY(check_sizes(fn, rows, in));
    if (rows == 0) return PTQ_OK;
    PTQ_TRY(check_float_rows(fn, "X", X, x_dtype, in, ldx));
    if (s && !aligned16(s)) REFUSE("%s: s is not 16-byte aligned", fn);
    PTQ_TRY(check_codes(fn, "codes", codes, in, ldc));
    if (!scales) REFUSE("%s: scales is NULL", fn);
    return launch_quantize_tokens_int8(X, x_dtype, rows, in, ldx, s, codes, ldc, scales, (hipStream_t)stream);
}

size_t matmul_int8_workspace_bytes(int64_t rows, int64_t out, int64_t in) {
    return rows > 0 && out > 0 && in > 0 ? matmul_int8_ws_bytes(matmul_int8_plan(rows, out, in), rows, out, in) : 0;
}

int matmul_int8(const int8_t* A, int64_t lda, const float* a_scales, int64_t rows, const int8_t* codes, int64_t ldb,
                const float* scales, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y, int64_t ldy,
                void* workspace, size_t workspace_bytes, void* stream) {
    return matmul("matmul_int8", nullptr, A, lda, a_scales, rows, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy,
                  workspace, workspace_bytes, stream);
}

int ptq_test_matmul_int8_plan(int64_t rows, int64_t out, int64_t in, int* shape, int* nsplit) {
    if (rows < 1 || out < 1 || in < 8 || in % 8 || in > MAX_IN || !shape || !nsplit)
        REFUSE("ptq_test_matmul_int8_plan: bad arguments");
    const Int8Plan p = matmul_int8_plan(rows, out, in);
    *shape = p.few ? -1 : p.shape;
    *nsplit = p.nsplit;
    return PTQ_OK;
}

size_t ptq_test_matmul_int8_workspace_bytes(int shape, int nsplit, int64_t rows, int64_t out, int64_t in) {
    return rows > 0 && out > 0 && in > 0 && shape < INT8_SHAPES
               ? matmul_int8_ws_bytes(Int8Plan{shape < 0, std::max(shape, 0), nsplit}, rows, out, in)
               : 0;
}

int ptq_test_matmul_int8(int shape, int nsplit, const int8_t* A, int64_t lda, const float* a_scales, int64_t rows,
                         const int8_t* codes, int64_t ldb, const float* scales, int64_t out, int64_t in,
                         const float* bias, int y_dtype, void* Y, int64_t ldy, void* workspace, size_t workspace_bytes,
                         void* stream) {
    const char* fn = "ptq_test_matmul_int8";
    // a tile holds whole stages of 128, and a share of the depth one at least
    if (shape < -1 || shape >= INT8_SHAPES || nsplit < 1 || nsplit > 16 ||
        (shape < 0 ? nsplit > 1 : in < 128 || nsplit > cdiv(in, 128)))
        REFUSE("%s: shape = %d, nsplit = %d", fn, shape, nsplit);
    const Int8Plan p{shape < 0, std::max(shape, 0), nsplit};
    return matmul(fn, &p, A, lda, a_scales, rows, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy, workspace,
                  workspace_bytes, stream);
}

size_t linear_int8_workspace_bytes(int64_t rows, int64_t out, int64_t in) {
    return rows > 0 && out > 0 && in > 0 ? linear_int8_ws_bytes(rows, out, in) : 0;
}

int linear_int8(const void* X, int x_dtype, int64_t rows, int64_t ldx, const float* s, const int8_t* codes,
                int64_t ldb, const float* scales, int64_t out, int64_t in, const float* bias, int y_dtype, void* Y,
                int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "linear_int8";
    PTQ_TRY(check_sizes(fn, rows, in));
    PTQ_TRY(check_out(fn, rows, out));
    if (rows == 0 || out == 0) return PTQ_OK;
    PTQ_TRY(check_float_rows(fn, "X", X, x_dtype, in, ldx));
    if (s && !aligned16(s)) REFUSE("%s: s is not 16-byte aligned", fn);
    PTQ_TRY(check_product(fn, codes, ldb, scales, out, in, y_dtype, Y, ldy));
    const size_t need = linear_int8_ws_bytes(rows, out, in);
    if (!workspace || workspace_bytes < need) {
        set_error("%s: workspace %zu bytes, need %zu", fn, workspace ? workspace_bytes : (size_t)0, need);
        return PTQ_EWORKSPACE;
    }
    if (!aligned16(workspace)) REFUSE("%s: workspace is not 16-byte aligned", fn);
    return run_linear_int8(X, x_dtype, rows, ldx, s, codes, ldb, scales, out, in, bias, y_dtype, Y, ldy, workspace,
                           workspace_bytes, (hipStream_t)stream);
}

int kv_cache_write_int8(int8_t* k_codes, int8_t* v_codes, float* k_scales, float* v_scales, int64_t num_blocks,
                        int kv_heads, int head_dim, int block_size, const void* K, int64_t ldk, const void* V,
                        int64_t ldv, int dtype, int64_t rows, const int32_t* offsets, const int32_t* starts,
                        int64_t batch, const int32_t* block_table, int64_t table_width, void* stream) {
    const char* fn = "kv_cache_write_int8";
    const KVCacheInt8 c{k_codes, v_codes, k_scales, v_scales, num_blocks, kv_heads, head_dim, block_size};
    const RaggedRows r{rows, batch, offsets, starts, block_table, table_width};
    PTQ_TRY(check_cache(fn, c));
    PTQ_TRY(check_ragged(fn, r, "starts", kv_heads));
    if (rows == 0 || batch == 0) return PTQ_OK;
    PTQ_TRY(check_cache_pointers(fn, c));
    const int64_t n = (int64_t)kv_heads * head_dim;
    PTQ_TRY(check_float_rows(fn, "K", K, dtype, n, ldk));
    PTQ_TRY(check_float_rows(fn, "V", V, dtype, n, ldv));
    return launch_kv_write(c, r, dtype, K, ldk, V, ldv, (hipStream_t)stream);
}

int kv_cache_read_int8(const int8_t* k_codes, const int8_t* v_codes, const float* k_scales, const float* v_scales,
                       int64_t num_blocks, int kv_heads, int head_dim, int block_size, void* K, int64_t ldk, void* V,
                       int64_t ldv, int dtype, int64_t rows, const int32_t* offsets, const int32_t* starts,
                       int64_t batch, const int32_t* block_table, int64_t table_width, void* stream) {
    const char* fn = "kv_cache_read_int8";
    const KVCacheInt8 c{const_cast<int8_t*>(k_codes), const_cast<int8_t*>(v_codes), const_cast<float*>(k_scales),
                        const_cast<float*>(v_scales), num_blocks, kv_heads, head_dim, block_size};
    const RaggedRows r{rows, batch, offsets, starts, block_table, table_width};
    PTQ_TRY(check_cache(fn, c));
    PTQ_TRY(check_ragged(fn, r, "starts", kv_heads));
    if (rows == 0 || batch == 0) return PTQ_OK;
    PTQ_TRY(check_cache_pointers(fn, c));
    const int64_t n = (int64_t)kv_heads * head_dim;
    PTQ_TRY(check_float_rows(fn, "K", K, dtype, n, ldk));
    PTQ_TRY(check_float_rows(fn, "V", V, dtype, n, ldv));
    return launch_kv_read(c, r, dtype, K, ldk, V, ldv, (hipStream_t)stream);
}

size_t attention_int8_cache_workspace_bytes(int64_t rows, int64_t batch, int heads, int kv_heads, int head_dim,
                                            int block_size, int64_t table_width) {
    const KVCacheInt8 c{nullptr, nullptr, nullptr, nullptr, 0, kv_heads, head_dim, block_size};
    if (check_cache("attention_int8_cache_workspace_bytes", c) != PTQ_OK || rows <= 0 || batch <= 0 ||
        heads < kv_heads || heads % kv_heads || table_width < 0)
        return 0;
    return attention_int8_ws_bytes(rows, batch, heads, kv_heads, head_dim, block_size, table_width);
}

int attention_int8_cache(const void* Q, int64_t ldq, void* O, int64_t ldo, float* lse, int dtype, int64_t rows,
                         int heads, const int32_t* offsets, const int32_t* seq_lens, int64_t batch,
                         const int32_t* block_table, int64_t table_width, const int8_t* k_codes, const int8_t* v_codes,
                         const float* k_scales, const float* v_scales, int64_t num_blocks, int kv_heads, int head_dim,
                         int block_size, float scale, int causal, int64_t window, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const KVCacheInt8 c{const_cast<int8_t*>(k_codes), const_cast<int8_t*>(v_codes), const_cast<float*>(k_scales),
                        const_cast<float*>(v_scales), num_blocks, kv_heads, head_dim, block_size};
    const RaggedRows r{rows, batch, offsets, seq_lens, block_table, table_width};
    return attention("attention_int8_cache", nullptr, c, r, dtype, Q, ldq, heads, scale, causal, window, O, ldo, lse,
                     workspace, workspace_bytes, stream);
}

int ptq_test_attention_int8_plan(int64_t rows, int64_t batch, int heads, int kv_heads, int head_dim, int block_size,
                                 int64_t table_width, int64_t window, int* tiles, int* waves, int* nsplit) {
    const char* fn = "ptq_test_attention_int8_plan";
    PTQ_TRY(check_cache(fn, KVCacheInt8{nullptr, nullptr, nullptr, nullptr, 0, kv_heads, head_dim, block_size}));
    if (rows < 1 || batch < 1 || heads < kv_heads || heads % kv_heads || table_width < 0 || window < 0 || !tiles ||
        !waves || !nsplit)
        REFUSE("%s: bad arguments", fn);
    const AttnPlan p = attention_int8_plan(rows, batch, heads, kv_heads, head_dim, block_size, table_width, window);
    *tiles = p.tr == ATTN_TILE;
    *waves = p.nw;
    *nsplit = p.nsplit;
    return PTQ_OK;
}

size_t ptq_test_attention_int8_workspace_bytes(int nsplit, int64_t rows, int heads, int head_dim) {
    return nsplit > 0 && rows > 0 && heads > 0 && head_dim > 0 ? attention_int8_part_bytes(nsplit, rows, heads, head_dim)
                                                               : 0;
}

int ptq_test_attention_int8_cache(int tiles, int waves, int nsplit, const void* Q, int64_t ldq, void* O, int64_t ldo,
                                  float* lse, int dtype, int64_t rows, int heads, const int32_t* offsets,
                                  const int32_t* seq_lens, int64_t batch, const int32_t* block_table,
                                  int64_t table_width, const int8_t* k_codes, const int8_t* v_codes,
                                  const float* k_scales, const float* v_scales, int64_t num_blocks, int kv_heads,
                                  int head_dim, int block_size, float scale, int causal, int64_t window,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "ptq_test_attention_int8_cache";
    if ((tiles != 0 && tiles != 1) || (tiles && head_dim > 128) || nsplit < 1 || nsplit > 64 ||
        (waves != 4 && (waves != 8 || tiles || nsplit > 1 || head_dim > 128)) || rows > 1 << 16 || batch > 1 << 10)
        REFUSE("%s: tiles = %d, waves = %d, nsplit = %d", fn, tiles, waves, nsplit);
    const KVCacheInt8 c{const_cast<int8_t*>(k_codes), const_cast<int8_t*>(v_codes), const_cast<float*>(k_scales),
                        const_cast<float*>(v_scales), num_blocks, kv_heads, head_dim, block_size};
    const RaggedRows r{rows, batch, offsets, seq_lens, block_table, table_width};
    const AttnPlan p{tiles ? ATTN_TILE : ATTN_ROWS, waves, nsplit};
    return attention(fn, &p, c, r, dtype, Q, ldq, heads, scale, causal, window, O, ldo, lse, workspace,
                     workspace_bytes, stream);
}

}  // extern "C"
