/*
 * ptq_testing.h — test hook of libptq.so (not part of the product API).
 *
 * Exposes the fp32 MFMA GEMM used inside stages 2 and 3 so its operand
 * layouts and triangle modes can be checked against a reference on their own:
 *
 *   C = alpha * op(A) op(B) + beta * C,   beta = beta_one ? 1 : 0
 *
 * layout_a: 0 = A row-major [M, K] (row stride lda), 1 = A stored [K, M].
 * layout_b: 0 = B row-major [K, N] (row stride ldb), 1 = B stored [N, K].
 * tri: 0 none; 1 A upper triangular (A[i][k] = 0 for k < i: those k are
 * skipped per row tile); 2 B upper (layout 0, B[k][j] = 0 for k > j);
 * 3 B upper stored [N][K] (entries with k < j are zero). upper_only: only
 * output tiles on or above the diagonal are written (128 x 128 tiles, or
 * 64 x 64 when the product has fewer than 1024 of 128 x 128): every entry
 * on or above the diagonal is, entries below it only inside diagonal tiles.
 * Device pointers; lda, ldb multiples of 4; asynchronous on `stream`.
 * Returns PTQ_OK, PTQ_EINVAL or PTQ_EHIP.
 */
#ifndef PTQ_TESTING_H
#define PTQ_TESTING_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

int ptq_test_gemm_f32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, int layout_a, const float* B,
                      int64_t ldb, int layout_b, float* C, int64_t ldc, float alpha, int beta_one, int tri,
                      int upper_only, void* stream);

/* The same product on the bf16 MFMA from three-term bf16 splits of A and B
 * (x = hi + mid + lo, six term products kept: fp32 GEMM accuracy), as used
 * for the large GEMMs of the U recursion. Output tiles are 256 x 256
 * (upper_only: tiles on or above the diagonal). The workspace (16-byte
 * aligned, size from the query) holds the split planes. Asynchronous.
 * Returns PTQ_OK, PTQ_EINVAL, PTQ_EWORKSPACE or PTQ_EHIP. */
size_t ptq_test_gemm_f32_split3_workspace_bytes(int64_t M, int64_t N, int64_t K);
int ptq_test_gemm_f32_split3(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, int layout_a,
                             const float* B, int64_t ldb, int layout_b, float* C, int64_t ldc, float alpha,
                             int beta_one, int tri, int upper_only, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Two independent products of the fp32 GEMM in one launch, as the U
 * recursion runs H11 -= R12 R12^T and T = R12 U22 at its small levels:
 * product 0 with B stored [N][K] (layout_b 1), product 1 with B row-major
 * [K][N] (layout_b 0), A row-major [M, K] for both, each with its own C,
 * alpha, beta, tri and upper_only as in ptq_test_gemm_f32. The results are
 * those of two ptq_test_gemm_f32 calls, bit for bit (when the two cannot
 * share a launch, two launches are made). Device pointers; K, lda, ldb
 * multiples of 4. Asynchronous. Returns PTQ_OK, PTQ_EINVAL or PTQ_EHIP. */
int ptq_test_gemm_f32_pair(int64_t M0, int64_t N0, int64_t K0, const float* A0, int64_t lda0, const float* B0,
                           int64_t ldb0, float* C0, int64_t ldc0, float alpha0, int beta_one0, int tri0,
                           int upper_only0, int64_t M1, int64_t N1, int64_t K1, const float* A1, int64_t lda1,
                           const float* B1, int64_t ldb1, float* C1, int64_t ldc1, float alpha1, int beta_one1,
                           int tri1, int upper_only1, void* stream);

/* matmul_int8 with the kernel given instead of chosen: shape -1 is the
 * streaming kernel (nsplit 1), 0 .. 5 are tiles of 256 x 256, 128 x 256,
 * 128 x 128, 64 x 64, 64 x 32 and 32 x 32 outputs x tokens (in >= 128), with
 * the depth in nsplit shares (at most 16, and ceil(in / 128)). _plan says what
 * matmul_int8 chooses. Returns PTQ_OK, PTQ_EINVAL, PTQ_EWORKSPACE or PTQ_EHIP. */
int ptq_test_matmul_int8_plan(int64_t rows, int64_t out, int64_t in, int* shape, int* nsplit);
size_t ptq_test_matmul_int8_workspace_bytes(int shape, int nsplit, int64_t rows, int64_t out, int64_t in);
int ptq_test_matmul_int8(int shape, int nsplit, const int8_t* A, int64_t lda, const float* a_scales, int64_t rows,
                         const int8_t* codes, int64_t ldb, const float* scales, int64_t out, int64_t in,
                         const float* bias, int y_dtype, void* Y, int64_t ldy, void* workspace,
                         size_t workspace_bytes, void* stream);

/* attention_int8_cache with the kernel given instead of chosen: tiles of 256
 * rows (1; head_dim up to 128) or few rows at a time (0), the waves of the
 * latter (4, or 8 with nsplit 1 and head_dim up to 128), and the splits of the
 * keys (1 .. 64). _plan says what attention_int8_cache chooses. Returns PTQ_OK,
 * PTQ_EINVAL, PTQ_EWORKSPACE or PTQ_EHIP. */
int ptq_test_attention_int8_plan(int64_t rows, int64_t batch, int heads, int kv_heads, int head_dim, int block_size,
                                 int64_t table_width, int64_t window, int* tiles, int* waves, int* nsplit);
size_t ptq_test_attention_int8_workspace_bytes(int nsplit, int64_t rows, int heads, int head_dim);
int ptq_test_attention_int8_cache(int tiles, int waves, int nsplit, const void* Q, int64_t ldq, void* O, int64_t ldo,
                                  float* lse, int dtype, int64_t rows, int heads, const int32_t* offsets,
                                  const int32_t* seq_lens, int64_t batch, const int32_t* block_table,
                                  int64_t table_width, const int8_t* k_codes, const int8_t* v_codes,
                                  const float* k_scales, const float* v_scales, int64_t num_blocks, int kv_heads,
                                  int head_dim, int block_size, float scale, int causal, int64_t window,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* attention_int8_tree with the kernel given instead of chosen: tiles of 256
 * query rows (1; head_dim up to 128, 8 waves), of 32 (0) or of 16 (2; 4 waves,
 * or 8 with head_dim up to 128), and the splits of the keys (1 .. 64). _plan says
 * what attention_int8_tree chooses. Returns PTQ_OK, PTQ_EINVAL, PTQ_EWORKSPACE or
 * PTQ_EHIP. */
int ptq_test_attention_tree_plan(int64_t rows, int64_t batch, int heads, int kv_heads, int head_dim, int dtype,
                                 int block_size, int64_t table_width, int64_t window, int* tiles, int* waves, int* nsplit);
size_t ptq_test_attention_tree_workspace_bytes(int nsplit, int64_t rows, int heads, int head_dim);
int ptq_test_attention_int8_tree(int tiles, int waves, int nsplit, const void* Q, int64_t ldq, void* O, int64_t ldo, float* lse,
                                 int dtype, int64_t rows, int heads, const int32_t* offsets, const int32_t* seq_lens,
                                 const int32_t* parents, int64_t batch, const int32_t* block_table,
                                 int64_t table_width, const int8_t* k_codes, const int8_t* v_codes,
                                 const float* k_scales, const float* v_scales, int64_t num_blocks, int kv_heads,
                                 int head_dim, int block_size, float scale, int64_t window, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* verify_drafts with the number of workgroups of a sequence given instead of
 * chosen: 1 .. 4. Returns PTQ_OK, PTQ_EINVAL, PTQ_EWORKSPACE or PTQ_EHIP. */
size_t ptq_test_verify_drafts_workspace_bytes(int shares, int64_t batch);
int ptq_test_verify_drafts(int shares, const void* target, int64_t ldt, const void* draft, int64_t ldd, int dtype,
                           int64_t rows, int64_t vocab, const int32_t* tokens, const int32_t* parents,
                           const int32_t* offsets, int64_t batch, const float* u, const float* r, int32_t* path,
                           int32_t* counts, int32_t* next, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PTQ_TESTING_H */
