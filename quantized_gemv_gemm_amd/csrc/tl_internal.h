// Internal declarations shared by the host API and the kernel translation units.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "tl.h"

namespace tl {

constexpr int kGroup = 128;   // weights per fp16 scale along K
constexpr int kHBlock = 1024; // Hadamard block width

// name of the last kernel launched by this host thread
void set_last_kernel(const char *name);

int64_t packed_words(int64_t N, int64_t K);
hipError_t launch_pack(const int8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                       uint32_t *packed, int8_t *q, float *row_scale, int32_t *invalid_count,
                       hipStream_t stream);

hipError_t launch_hadamard(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs,
                           float *xr, hipStream_t stream);

hipError_t launch_quant(const float *xr, int64_t T, int64_t K, int8_t *xq, float *tok_scale,
                        hipStream_t stream);

// Decode activation limbs in the GEMV workspace.  b <= 8: row-major rows, hi
// limbs [b][K + 16] then lo limbs [b][K + 16].  b > 8: the operand order of
// v_mfma_i32_16x16x64_i8, so that every operand load reads 1 KB contiguously:
// tokens in chunks of 16 (chunk c = t / 16 owns 32 K bytes at 32 K c); inside a
// chunk, for group g, 64-k half h and limb l, 64 lanes x 16 bytes, where lane
// r + 16 q holds A row r (token 16 c + 4 (r % 4) + r / 4) and
// k = 128 g + 32 q + 16 h + j.
// Limb scales: sigma[t][j] = |x|max / 32639 of token t's 1024-block j (the last
// block may be shorter), limb_blocks(K) per token, after the limbs.
constexpr int kLimbRowPad = 16;
constexpr int kTokChunk = 16;      // tokens per MFMA operand (and per GEMV grid row)
constexpr int kGemvMaxTokens = 64; // decode tokens per call
__host__ __device__ inline int64_t limb_chunks(int64_t b) { return (b + kTokChunk - 1) / kTokChunk; }
__host__ __device__ inline int limb_blocks(int64_t K) { return int((K + kHBlock - 1) / kHBlock); }
__host__ __device__ inline int64_t limb_region_bytes(int64_t b, int64_t K) {
  return b > 8 ? 32 * K * limb_chunks(b) : 2 * b * (K + kLimbRowPad);
}
__host__ __device__ inline int64_t limb_frag_offset(int t, int64_t k, int limb, int64_t K) {
  const int64_t g = k >> 7;
  const int kk = int(k & 127);
  const int tc = t & (kTokChunk - 1);
  const int row = 4 * (tc & 3) + (tc >> 2);
  return 32 * K * (t / kTokChunk) +
         (((((g * 2 + ((kk >> 4) & 1)) * 2 + limb) * 64 + row + 16 * (kk >> 5)) << 4) + (kk & 15));
}

size_t gemv_workspace_bytes(int64_t b, int64_t K, int64_t N);
// false when the weight-stream variant for (b, K, N) would not fit a compute unit
// (its LDS or workgroup size); the entry points then return TL_ERR_UNSUPPORTED
bool gemv_supported(int64_t b, int64_t K, int64_t N);
hipError_t launch_gemv_prepare(const float *xr, int64_t b, int64_t K, void *workspace,
                               hipStream_t stream);
hipError_t launch_gemv_main(const void *workspace, int64_t b, int64_t K, int64_t N,
                            const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                            hipStream_t stream);

// fused rotation -> GEMV limbs / int8 quantisation (k_rotq.hip)
bool fused_input_supported(int64_t K);
hipError_t launch_gemv_prepare_x(const uint16_t *x, int64_t b, int64_t K, const int8_t *signs,
                                 int8_t *xhi, int64_t Kp, float *sigma, hipStream_t stream);
hipError_t launch_quant_x(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs, int8_t *xq,
                          float *tok_scale, hipStream_t stream);
// the GEMV workspace carved for the fused prep (k_gemv.hip)
hipError_t launch_gemv_prepare_rotated(const uint16_t *x, int64_t b, int64_t K, const int8_t *signs,
                                       void *workspace, hipStream_t stream);

// rotation + limbs + GEMV in one launch for one or two tokens (k_gemv.hip)
bool gemv_rot_supported(int64_t b, int64_t K, int64_t N);
hipError_t launch_gemv_rot(const uint16_t *x, int64_t b, int64_t K, int64_t N, const int8_t *signs,
                           const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                           hipStream_t stream);

// decode GEMV against int8 activations (k_gemv.hip)
bool gemv_q8_supported(int64_t b, int64_t K, int64_t N);
hipError_t launch_gemv_q8(const int8_t *xq, const float *tok_scale, int64_t b, int64_t K, int64_t N,
                          const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                          hipStream_t stream);

// split-block rotation stages (k_split.hip)
hipError_t launch_hadamard_half(const uint16_t *x, int64_t T, int64_t ldx, const int8_t *signs,
                                double *u, hipStream_t stream);
hipError_t launch_hadamard_join(const double *u_lo, const double *u_hi, int64_t T, int half, float *xr,
                                int64_t ldxr, hipStream_t stream);

// measurement helper: a launch that only reads `bytes` (k_probe.hip)
hipError_t launch_read_probe(const void *src, size_t bytes, uint32_t *sink, hipStream_t stream);
hipError_t launch_mfma_probe(int random, int iters, uint32_t *sink, hipStream_t stream);

size_t gemm_workspace_bytes(int64_t M, int64_t K, int64_t N);
hipError_t launch_gemm(const int8_t *xq, const float *tok_scale, int64_t M, int64_t K, int64_t N,
                       const uint32_t *packed, const int8_t *q, const float *row_scale, void *y,
                       int y_dtype, int32_t *acc_out, void *workspace, hipStream_t stream);

// ---------------------------------------------------------------------------
// one step of speculative decoding over a paged cache
constexpr int kMaxRequests = TL_MAX_REQUESTS;
// Their prefix sums sit in LDS: behind what an attention kernel stages, and with its static
// variables (272 to 288 bytes by the compiler's report) within a compute unit's 160 KB.
constexpr size_t kLdsBytes = 160 * 1024, kStaticLds = 512;
constexpr size_t prefix_bytes(int R) { return size_t(R + 1) * 4; }
constexpr bool fits_lds(size_t staged) { return staged + prefix_bytes(kMaxRequests) + kStaticLds <= kLdsBytes; }

// attention (k_tree.hip)
struct TreeArgs {
  const uint16_t *q;         // bf16 [T, H * G, D], tokens ldq elements apart
  const char *k, *v;         // caches
  const float *k_scale, *v_scale;
  const int32_t *table, *q_start, *kv_lens;
  const uint64_t *tree_mask;
  uint16_t *out;             // bf16 [T, H * G, D]
  float *lse;                // f32 [T, H * G] or NULL
  float *part_o, *part_ml;   // workspace: partial sums, and their maximum and sum
  int32_t *borders;          // workspace: the items that workgroups share
  int64_t ldq;
  int T, R, H, G;            // tokens, requests, cache heads, query heads of each
  int pages, block_shift, table_width;
  int max_keys;              // table_width * block
  float scale;
};
size_t tree_workspace_bytes(int64_t max_nodes, int64_t group, int64_t D, bool e4m3);
hipError_t launch_tree_attention(TreeArgs a, int64_t D, bool e4m3, int64_t max_nodes, void *workspace,
                                 hipStream_t stream);

// block tables, slots, positions and tree masks (k_step.hip)
struct StepArgs {
  const int32_t *ctx_lens, *new_lens, *owned;
  int32_t *table;
  const int32_t *free_list, *free_head, *parents;
  int32_t *q_start, *kv_lens;
  int64_t *slots;
  int32_t *positions;
  uint64_t *tree_mask;
  int32_t *owned_out, *free_head_out;
  int64_t free_count;
  int T, R, table_width, block;
};
hipError_t launch_step_plan(const StepArgs &a, hipStream_t stream);

// cache rows (k_kv.hip)
struct WriteArgs {
  const uint16_t *q, *k, *v;  // bf16 [T, heads, D], tokens ldq / ldk / ldv elements apart
  const int64_t *slots;
  const int32_t *positions;
  const float *cos_sin;       // f32 [max_pos, rot]: cosines, then sines
  uint16_t *q_out;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int64_t ldq, ldk, ldv, slot_count;
  int T, Hq, H, rot, max_pos, block_shift;
};
hipError_t launch_kv_write(const WriteArgs &a, int64_t D, bool e4m3, hipStream_t stream);

struct CommitArgs {
  const int32_t *accepted, *path, *ctx_lens, *kv_lens, *table;
  char *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t *ctx_out;
  int64_t layer_tokens;       // pages * heads * block
  int R, L, H, pages, block_shift, table_width, path_width;
};
hipError_t launch_kv_commit(const CommitArgs &a, int64_t D, bool e4m3, hipStream_t stream);

// greedy check of drafted trees (k_verify.hip)
struct VerifyArgs {
  const void *logits;         // [T, V], rows ld elements apart
  const int32_t *draft, *parents, *q_start;
  int32_t *accepted, *path, *next, *target;
  uint64_t *best;             // workspace [T][parts]
  int64_t ld, V;
  int T, R, path_width, parts;
};
int verify_parts(int64_t T, int64_t V);
hipError_t launch_tree_verify(const VerifyArgs &a, bool f32, hipStream_t stream);

// whole layer from the raw input (tl_api.cpp): the checks that need no workspace,
// then the workspace checks and the launches on the path tl_linear_path names
size_t linear_scratch_bytes(int64_t T, int64_t K, int64_t N);
int linear_check(const uint16_t *x, int64_t T, int64_t K, int64_t N, const uint32_t *packed,
                 const uint16_t *scales, const int8_t *q, const float *row_scale, void *y, int y_dtype);
int linear_run(const uint16_t *x, int64_t T, int64_t K, int64_t N, const int8_t *signs,
               const uint32_t *packed, const uint16_t *scales, const int8_t *q, const float *row_scale,
               void *y, int y_dtype, void *workspace, size_t workspace_bytes, hipStream_t st);

}  // namespace tl
