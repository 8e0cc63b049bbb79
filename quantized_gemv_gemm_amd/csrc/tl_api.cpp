// Host side of the C ABI declared in include/tl.h: argument checks, then launches.
// Every check runs before any HIP call, so a rejected call touches neither the
// GPU nor the outputs.
#include <stdint.h>
#include <string.h>

#include "kv_layout.h"
#include "tl_internal.h"

namespace tl {
static thread_local const char *g_last_kernel = "";
static thread_local const char *g_last_error = "";
void set_last_kernel(const char *name) { g_last_kernel = name; }
}  // namespace tl

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  const void *p;
  size_t bytes;
};

bool overlap(Span a, Span b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// outputs must not overlap inputs or each other
bool any_alias(const Span *in, int nin, const Span *out, int nout) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (overlap(out[o], in[i])) return true;
    for (int j = o + 1; j < nout; ++j)
      if (overlap(out[o], out[j])) return true;
  }
  return false;
}

int from_hip(hipError_t e) {
  if (e == hipSuccess) return TL_OK;
  tl::g_last_error = hipGetErrorString(e);
  return TL_ERR_LAUNCH;
}

constexpr int64_t kMaxDim = int64_t(1) << 31;  // rows, tokens and K stay below 2^31
// keys of a request's table: the attention counts positions in 32 bits, and looks for the
// tiles of a segment 64 at a time, so up to 1024 positions past the last key
constexpr int64_t kMostKeys = kMaxDim - 4096;

// one step of speculative decoding over a paged cache
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <typename... P>
bool aligned_to(size_t n, P... p) {
  return (aligned(p, n) && ...);
}
template <typename... P>
bool any_null(P... p) {
  return (!p || ...);
}

bool count_ok(int64_t n) { return n >= 0 && n < kMaxDim; }
bool block_ok(int64_t block) { return block >= tl::kKvTile && block <= 4096 && (block & (block - 1)) == 0; }
int log2_of(int64_t n) { return __builtin_ctzll(uint64_t(n)); }
bool width_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

// sizes of a cache: 0 or a status
int check_cache(int cache_dtype, int64_t pages, int64_t H, int64_t block, int64_t D) {
  if (cache_dtype != TL_BF16 && cache_dtype != TL_E4M3) return TL_ERR_DTYPE;
  if (!width_ok(D) || !block_ok(block) || H < 1 || H > 65536 || pages < 1 || pages >= kMaxDim) return TL_ERR_SHAPE;
  if (pages > (int64_t(1) << 50) / (H * block * D)) return TL_ERR_SHAPE;
  return TL_OK;
}
size_t cache_bytes(int cache_dtype, int64_t tokens, int64_t D) { return size_t(tokens) * D * (cache_dtype == TL_BF16 ? 2 : 1); }

}  // namespace

extern "C" {

int tl_abi_version(void) { return TL_ABI_VERSION; }

const char *tl_status_string(int s) {
  switch (s) {
    case TL_OK: return "ok";
    case TL_ERR_NULLPTR: return "a required pointer is NULL";
    case TL_ERR_SHAPE: return "invalid shape (negative, too large, or not a required multiple)";
    case TL_ERR_ALIGN: return "pointer not 16-byte aligned";
    case TL_ERR_DTYPE: return "y_dtype must be TL_BF16 or TL_F32";
    case TL_ERR_LAUNCH: return "HIP runtime error during launch";
    case TL_ERR_UNSUPPORTED: return "no kernel variant for this request";
    case TL_ERR_WORKSPACE: return "workspace missing or too small";
    case TL_ERR_ALIAS: return "an output overlaps an input or another output";
    case TL_ERR_SCRATCH:
      return "request needs more scratch than the no-allocation entry point's static buffer holds";
    default: return "unknown status";
  }
}

const char *tl_last_kernel_name(void) { return tl::g_last_kernel; }

const char *tl_last_error_detail(void) { return tl::g_last_error; }

size_t tl_packed_bytes(int64_t N, int64_t K) {
  if (N < 0 || K <= 0 || K % tl::kGroup || N >= kMaxDim || K >= kMaxDim) return 0;
  return size_t(tl::packed_words(N, K)) * 4;
}

int tl_pack_weights(const int8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                    uint32_t *packed, int8_t *q, float *row_scale, int32_t *invalid_count,
                    void *stream) {
  if (N < 0 || K <= 0 || K % tl::kGroup || N >= kMaxDim || K >= kMaxDim) return TL_ERR_SHAPE;
  if (N == 0) return TL_OK;
  if (!codes || !scales || !packed || !q || !row_scale) return TL_ERR_NULLPTR;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(packed) || !aligned16(q) ||
      !aligned16(row_scale))
    return TL_ERR_ALIGN;
  const size_t G = size_t(K / tl::kGroup);
  Span in[] = {{codes, size_t(N) * K}, {scales, size_t(N) * G * 2}};
  Span out[] = {{packed, size_t(tl::packed_words(N, K)) * 4}, {q, size_t(N) * G}, {row_scale, size_t(N) * 4},
                {invalid_count, invalid_count ? 4u : 0u}};
  if (any_alias(in, 2, out, 4)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_pack(codes, scales, N, K, packed, q, row_scale, invalid_count,
                                  static_cast<hipStream_t>(stream)));
}

int tl_hadamard_blk(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs, float *xr,
                    void *stream) {
  if (T < 0 || K <= 0 || K % tl::kHBlock || T >= kMaxDim || K >= kMaxDim) return TL_ERR_SHAPE;
  if (T == 0) return TL_OK;
  if (!x || !xr) return TL_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(xr) || (signs && !aligned16(signs))) return TL_ERR_ALIGN;
  Span in[] = {{x, size_t(T) * K * 2}, {signs, signs ? size_t(K) : 0u}};
  Span out[] = {{xr, size_t(T) * K * 4}};
  if (any_alias(in, 2, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_hadamard(x, T, K, signs, xr, static_cast<hipStream_t>(stream)));
}

int tl_hadamard_half(const uint16_t *x, int64_t T, int64_t ldx, const int8_t *signs, double *u,
                     void *stream) {
  if (T < 0 || T >= kMaxDim || ldx < tl::kHBlock / 2 || ldx >= kMaxDim) return TL_ERR_SHAPE;
  if (T == 0) return TL_OK;
  if (!x || !u) return TL_ERR_NULLPTR;
  if (!aligned16(x) || ldx % 8 || !aligned16(u)) return TL_ERR_ALIGN;
  const size_t half = tl::kHBlock / 2;
  Span in[] = {{x, (size_t(T - 1) * ldx + half) * 2}, {signs, signs ? half : 0u}};
  Span out[] = {{u, size_t(T) * half * 8}};
  if (any_alias(in, 2, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_hadamard_half(x, T, ldx, signs, u, static_cast<hipStream_t>(stream)));
}

int tl_hadamard_join(const double *u_lo, const double *u_hi, int64_t T, int half, float *xr,
                     int64_t ldxr, void *stream) {
  if (T < 0 || T >= kMaxDim || ldxr < tl::kHBlock / 2 || ldxr >= kMaxDim || (half != 0 && half != 1))
    return TL_ERR_SHAPE;
  if (T == 0) return TL_OK;
  if (!u_lo || !u_hi || !xr) return TL_ERR_NULLPTR;
  if (!aligned16(u_lo) || !aligned16(u_hi) || !aligned16(xr) || ldxr % 4) return TL_ERR_ALIGN;
  const size_t hb = tl::kHBlock / 2;
  Span in[] = {{u_lo, size_t(T) * hb * 8}, {u_hi, size_t(T) * hb * 8}};
  Span out[] = {{xr, (size_t(T - 1) * ldxr + hb) * 4}};
  if (any_alias(in, 2, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_hadamard_join(u_lo, u_hi, T, half, xr, ldxr, static_cast<hipStream_t>(stream)));
}

size_t tl_gemv_workspace_size(int64_t b, int64_t K, int64_t N) {
  if (b < 0 || b > tl::kGemvMaxTokens || K <= 0 || K % tl::kGroup || N < 0) return 0;
  return tl::gemv_workspace_bytes(b, K, N);
}

namespace {
int check_gemv_shape(int64_t b, int64_t K, int64_t N, int64_t bmax = tl::kGemvMaxTokens) {
  if (b < 0 || b > bmax || N < 0 || K <= 0 || K % tl::kGroup || N >= kMaxDim || K >= kMaxDim)
    return TL_ERR_SHAPE;
  return TL_OK;
}
}  // namespace

int tl_gemv_prepare(const float *xr, int64_t b, int64_t K, void *workspace, size_t workspace_bytes,
                    void *stream) {
  if (int s = check_gemv_shape(b, K, 0)) return s;
  if (b == 0) return TL_OK;
  if (!xr) return TL_ERR_NULLPTR;
  const size_t need = tl::gemv_workspace_bytes(b, K, 0);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned16(xr) || !aligned16(workspace)) return TL_ERR_ALIGN;
  Span in[] = {{xr, size_t(b) * K * 4}};
  Span out[] = {{workspace, need}};
  if (any_alias(in, 1, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_gemv_prepare(xr, b, K, workspace, static_cast<hipStream_t>(stream)));
}

int tl_gemv_prepared(const void *workspace, size_t workspace_bytes, int64_t b, int64_t K, int64_t N,
                     const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                     void *stream) {
  if (int s = check_gemv_shape(b, K, N)) return s;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (b == 0 || N == 0) return TL_OK;
  if (!packed || !scales || !y) return TL_ERR_NULLPTR;
  const size_t need = tl::gemv_workspace_bytes(b, K, N);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(y) || !aligned16(workspace))
    return TL_ERR_ALIGN;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(b) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{workspace, need}, {packed, size_t(tl::packed_words(N, K)) * 4}, {scales, size_t(N) * G * 2}};
  Span out[] = {{y, ysz}};
  if (any_alias(in, 3, out, 1)) return TL_ERR_ALIAS;
  if (!tl::gemv_supported(b, K, N)) return TL_ERR_UNSUPPORTED;
  return from_hip(tl::launch_gemv_main(workspace, b, K, N, packed, scales, y, y_dtype,
                                       static_cast<hipStream_t>(stream)));
}

int tl_gemv_ternary(const float *xr, int64_t b, int64_t K, int64_t N, const uint32_t *packed,
                    const uint16_t *scales, void *y, int y_dtype, void *workspace,
                    size_t workspace_bytes, void *stream) {
  if (int s = check_gemv_shape(b, K, N)) return s;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (b == 0 || N == 0) return TL_OK;
  if (!xr || !packed || !scales || !y) return TL_ERR_NULLPTR;
  const size_t need = tl::gemv_workspace_bytes(b, K, N);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned16(xr) || !aligned16(packed) || !aligned16(scales) || !aligned16(y) ||
      !aligned16(workspace))
    return TL_ERR_ALIGN;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(b) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{xr, size_t(b) * K * 4}, {packed, size_t(tl::packed_words(N, K)) * 4}, {scales, size_t(N) * G * 2}};
  Span out[] = {{y, ysz}, {workspace, need}};
  if (any_alias(in, 3, out, 2)) return TL_ERR_ALIAS;
  if (!tl::gemv_supported(b, K, N)) return TL_ERR_UNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = tl::launch_gemv_prepare(xr, b, K, workspace, st);
  if (e != hipSuccess) return from_hip(e);
  return from_hip(tl::launch_gemv_main(workspace, b, K, N, packed, scales, y, y_dtype, st));
}

int tl_gemv_prepare_x(const uint16_t *x, int64_t b, int64_t K, const int8_t *signs,
                      void *workspace, size_t workspace_bytes, void *stream) {
  if (int s = check_gemv_shape(b, K, 0)) return s;
  if (K % tl::kHBlock) return TL_ERR_SHAPE;
  if (!tl::fused_input_supported(K)) return TL_ERR_UNSUPPORTED;
  if (b == 0) return TL_OK;
  if (!x) return TL_ERR_NULLPTR;
  const size_t need = tl::gemv_workspace_bytes(b, K, 0);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(workspace) || (signs && !aligned16(signs))) return TL_ERR_ALIGN;
  Span in[] = {{x, size_t(b) * K * 2}, {signs, signs ? size_t(K) : 0u}};
  Span out[] = {{workspace, need}};
  if (any_alias(in, 2, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_gemv_prepare_rotated(x, b, K, signs, workspace,
                                                  static_cast<hipStream_t>(stream)));
}

int tl_gemv_ternary_x(const uint16_t *x, int64_t b, int64_t K, int64_t N, const int8_t *signs,
                      const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                      void *workspace, size_t workspace_bytes, void *stream) {
  if (int s = check_gemv_shape(b, K, N)) return s;
  if (K % tl::kHBlock) return TL_ERR_SHAPE;
  if (!tl::fused_input_supported(K)) return TL_ERR_UNSUPPORTED;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (b == 0 || N == 0) return TL_OK;
  if (!x || !packed || !scales || !y) return TL_ERR_NULLPTR;
  const size_t need = tl::gemv_workspace_bytes(b, K, N);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(scales) || !aligned16(y) ||
      !aligned16(workspace) || (signs && !aligned16(signs)))
    return TL_ERR_ALIGN;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(b) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{x, size_t(b) * K * 2}, {signs, signs ? size_t(K) : 0u},
               {packed, size_t(tl::packed_words(N, K)) * 4}, {scales, size_t(N) * G * 2}};
  Span out[] = {{y, ysz}, {workspace, need}};
  if (any_alias(in, 4, out, 2)) return TL_ERR_ALIAS;
  if (!tl::gemv_rot_supported(b, K, N) && !tl::gemv_supported(b, K, N)) return TL_ERR_UNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (tl::gemv_rot_supported(b, K, N))
    return from_hip(tl::launch_gemv_rot(x, b, K, N, signs, packed, scales, y, y_dtype, st));
  hipError_t e = tl::launch_gemv_prepare_rotated(x, b, K, signs, workspace, st);
  if (e != hipSuccess) return from_hip(e);
  return from_hip(tl::launch_gemv_main(workspace, b, K, N, packed, scales, y, y_dtype, st));
}

int tl_quant_act_int8_x(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs, int8_t *xq,
                        float *tok_scale, void *stream) {
  if (T < 0 || K <= 0 || K % tl::kHBlock || T >= kMaxDim || K >= kMaxDim) return TL_ERR_SHAPE;
  if (!tl::fused_input_supported(K)) return TL_ERR_UNSUPPORTED;
  if (T == 0) return TL_OK;
  if (!x || !xq || !tok_scale) return TL_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(tok_scale) || (signs && !aligned16(signs)))
    return TL_ERR_ALIGN;
  Span in[] = {{x, size_t(T) * K * 2}, {signs, signs ? size_t(K) : 0u}};
  Span out[] = {{xq, size_t(T) * K}, {tok_scale, size_t(T) * 4}};
  if (any_alias(in, 2, out, 2)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_quant_x(x, T, K, signs, xq, tok_scale, static_cast<hipStream_t>(stream)));
}

int tl_gemv_ternary_q8(const int8_t *xq, const float *tok_scale, int64_t b, int64_t K, int64_t N,
                       const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                       void *stream) {
  if (int s = check_gemv_shape(b, K, N, tl::kTokChunk)) return s;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (b == 0 || N == 0) return TL_OK;
  if (!xq || !tok_scale || !packed || !scales || !y) return TL_ERR_NULLPTR;
  if (!aligned16(xq) || !aligned16(packed) || !aligned16(scales) || !aligned16(y)) return TL_ERR_ALIGN;
  if (!tl::gemv_q8_supported(b, K, N)) return TL_ERR_UNSUPPORTED;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(b) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{xq, size_t(b) * K}, {tok_scale, size_t(b) * 4}, {packed, size_t(tl::packed_words(N, K)) * 4},
               {scales, size_t(N) * G * 2}};
  Span out[] = {{y, ysz}};
  if (any_alias(in, 4, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_gemv_q8(xq, tok_scale, b, K, N, packed, scales, y, y_dtype,
                                     static_cast<hipStream_t>(stream)));
}

int tl_quant_act_int8(const float *xr, int64_t T, int64_t K, int8_t *xq, float *tok_scale,
                      void *stream) {
  if (T < 0 || K <= 0 || K % tl::kGroup || T >= kMaxDim || K >= kMaxDim) return TL_ERR_SHAPE;
  if (T == 0) return TL_OK;
  if (!xr || !xq || !tok_scale) return TL_ERR_NULLPTR;
  if (!aligned16(xr) || !aligned16(xq) || !aligned16(tok_scale)) return TL_ERR_ALIGN;
  Span in[] = {{xr, size_t(T) * K * 4}};
  Span out[] = {{xq, size_t(T) * K}, {tok_scale, size_t(T) * 4}};
  if (any_alias(in, 1, out, 2)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_quant(xr, T, K, xq, tok_scale, static_cast<hipStream_t>(stream)));
}

int tl_read_probe(const void *src, size_t bytes, uint32_t *sink, void *stream) {
  if (bytes < 16 || bytes % 16 || bytes / 16 / 512 > 0x7FFFFFFF) return TL_ERR_SHAPE;
  if (!src || !sink) return TL_ERR_NULLPTR;
  if (!aligned16(src) || !aligned16(sink)) return TL_ERR_ALIGN;
  Span in[] = {{src, bytes}};
  Span out[] = {{sink, 4}};
  if (any_alias(in, 1, out, 1)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_read_probe(src, bytes, sink, static_cast<hipStream_t>(stream)));
}

int tl_mfma_probe(int random_operands, int iters, uint32_t *sink, void *stream) {
  if (iters <= 0) return TL_ERR_SHAPE;
  if (!sink) return TL_ERR_NULLPTR;
  if (!aligned16(sink)) return TL_ERR_ALIGN;
  return from_hip(tl::launch_mfma_probe(random_operands ? 1 : 0, iters, sink, static_cast<hipStream_t>(stream)));
}

size_t tl_gemm_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || N < 0 || K <= 0 || K % tl::kGroup) return 0;
  return tl::gemm_workspace_bytes(M, K, N);
}

int tl_gemm_int8_rescale(const int8_t *xq, const float *tok_scale, int64_t M, int64_t K,
                         int64_t N, const uint32_t *packed, const int8_t *q,
                         const float *row_scale, void *y, int y_dtype, int32_t *acc_out,
                         void *workspace, size_t workspace_bytes, void *stream) {
  if (M < 0 || N < 0 || K <= 0 || K % tl::kGroup || K > 133120 || M >= kMaxDim || N >= kMaxDim)
    return TL_ERR_SHAPE;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (M == 0 || N == 0) return TL_OK;
  if (!xq || !tok_scale || !packed || !q || !row_scale || !y) return TL_ERR_NULLPTR;
  if (!aligned16(xq) || !aligned16(tok_scale) || !aligned16(packed) || !aligned16(q) ||
      !aligned16(row_scale) || !aligned16(y) || (acc_out && !aligned16(acc_out)) ||
      (workspace && !aligned16(workspace)))
    return TL_ERR_ALIGN;
  const size_t need = tl::gemm_workspace_bytes(M, K, N);
  if (need && (!workspace || workspace_bytes < need)) return TL_ERR_WORKSPACE;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(M) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{xq, size_t(M) * K}, {tok_scale, size_t(M) * 4}, {packed, size_t(tl::packed_words(N, K)) * 4},
               {q, size_t(N) * G}, {row_scale, size_t(N) * 4}};
  Span out[] = {{y, ysz}, {acc_out, acc_out ? size_t(M) * N * 4 : 0u}, {workspace, need}};
  if (any_alias(in, 5, out, 3)) return TL_ERR_ALIAS;
  return from_hip(tl::launch_gemm(xq, tok_scale, M, K, N, packed, q, row_scale, y, y_dtype,
                                  acc_out, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// whole layer from the raw input, path chosen by the token count
// ---------------------------------------------------------------------------
namespace {

constexpr size_t kLinCounters = 1024;  // the GEMM's split-K counters: kept at offset 0 for both paths

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct LinearLayout {
  int path;
  size_t gemm_ws;  // counters + partials (0: the GEMM runs unsplit)
  size_t xq, sx;   // offsets of the int8 path's activations and token scales
  size_t total;
};

LinearLayout linear_layout(int64_t T, int64_t K, int64_t N) {
  LinearLayout l{};
  l.path = tl_linear_path(T, K, N);
  if (l.path == TL_PATH_GEMV) {
    l.total = kLinCounters + tl::gemv_workspace_bytes(T, K, N);
  } else {
    l.gemm_ws = tl::gemm_workspace_bytes(T, K, N);
    l.xq = align256(l.gemm_ws > kLinCounters ? l.gemm_ws : kLinCounters);
    l.sx = l.xq + align256(size_t(T) * K);
    l.total = l.sx + align256(size_t(T) * 4);
  }
  return l;
}

}  // namespace

namespace tl {

size_t linear_scratch_bytes(int64_t T, int64_t K, int64_t N) { return linear_layout(T, K, N).total; }

int linear_check(const uint16_t *x, int64_t T, int64_t K, int64_t N, const uint32_t *packed,
                 const uint16_t *scales, const int8_t *q, const float *row_scale, void *y, int y_dtype) {
  if (T < 0 || N < 0 || K <= 0 || K % tl::kHBlock || T >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return TL_ERR_SHAPE;
  if (!tl::fused_input_supported(K)) return TL_ERR_UNSUPPORTED;
  if (y_dtype != TL_BF16 && y_dtype != TL_F32) return TL_ERR_DTYPE;
  if (T == 0 || N == 0) return TL_OK;
  if (!x || !packed || !scales || !q || !row_scale || !y) return TL_ERR_NULLPTR;
  return TL_OK;
}

int linear_run(const uint16_t *x, int64_t T, int64_t K, int64_t N, const int8_t *signs,
               const uint32_t *packed, const uint16_t *scales, const int8_t *q, const float *row_scale,
               void *y, int y_dtype, void *workspace, size_t workspace_bytes, hipStream_t st) {
  const LinearLayout l = linear_layout(T, K, N);
  if (!workspace || workspace_bytes < l.total) return TL_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(scales) || !aligned16(q) ||
      !aligned16(row_scale) || !aligned16(y) || !aligned16(workspace) || (signs && !aligned16(signs)))
    return TL_ERR_ALIGN;
  const size_t G = size_t(K / tl::kGroup);
  const size_t ysz = size_t(T) * N * (y_dtype == TL_F32 ? 4 : 2);
  Span in[] = {{x, size_t(T) * K * 2}, {signs, signs ? size_t(K) : 0u},
               {packed, size_t(tl::packed_words(N, K)) * 4}, {scales, size_t(N) * G * 2},
               {q, size_t(N) * G}, {row_scale, size_t(N) * 4}};
  Span out[] = {{y, ysz}, {workspace, l.total}};
  if (any_alias(in, 6, out, 2)) return TL_ERR_ALIAS;
  char *ws = static_cast<char *>(workspace);
  if (l.path == TL_PATH_GEMV && !tl::gemv_rot_supported(T, K, N) && !tl::gemv_supported(T, K, N))
    return TL_ERR_UNSUPPORTED;
  if (l.path == TL_PATH_GEMV) {
    if (tl::gemv_rot_supported(T, K, N))
      return from_hip(tl::launch_gemv_rot(x, T, K, N, signs, packed, scales, y, y_dtype, st));
    void *gw = ws + kLinCounters;
    hipError_t e = tl::launch_gemv_prepare_rotated(x, T, K, signs, gw, st);
    if (e != hipSuccess) return from_hip(e);
    return from_hip(tl::launch_gemv_main(gw, T, K, N, packed, scales, y, y_dtype, st));
  }
  int8_t *xq = reinterpret_cast<int8_t *>(ws + l.xq);
  float *sx = reinterpret_cast<float *>(ws + l.sx);
  hipError_t e = tl::launch_quant_x(x, T, K, signs, xq, sx, st);
  if (e != hipSuccess) return from_hip(e);
  return from_hip(tl::launch_gemm(xq, sx, T, K, N, packed, q, row_scale, y, y_dtype, nullptr,
                                  l.gemm_ws ? workspace : nullptr, st));
}

}  // namespace tl

extern "C" {

int tl_linear_path(int64_t T, int64_t K, int64_t N) {
  if (T <= tl::kTokChunk) return TL_PATH_GEMV;
  if (T > tl::kGemvMaxTokens) return TL_PATH_INT8;
  // 17..64 tokens: the GEMV runs one chunk of 16 tokens per grid row, each
  // streaming all N x K weights again, while the int8 path's time hardly grows
  // with T at this size; the GEMV stays ahead up to about 2^27 streamed weights
  // (qkv 5120 x 10240: two chunks; down 17408 x 5120 and gate_up 5120 x 34816:
  // none beyond the first).
  const int64_t streamed = tl::limb_chunks(T) * N * K;
  return streamed <= (int64_t(1) << 27) ? TL_PATH_GEMV : TL_PATH_INT8;
}

size_t tl_linear_workspace_size(int64_t T, int64_t K, int64_t N) {
  if (T < 0 || N < 0 || K <= 0 || K % tl::kHBlock || T >= kMaxDim || N >= kMaxDim) return 0;
  return linear_layout(T, K, N).total;
}

int tl_linear_apply(const uint16_t *x, int64_t T, int64_t K, int64_t N, const int8_t *signs,
                    const uint32_t *packed, const uint16_t *scales, const int8_t *q,
                    const float *row_scale, void *y, int y_dtype, void *workspace,
                    size_t workspace_bytes, void *stream) {
  if (int s = tl::linear_check(x, T, K, N, packed, scales, q, row_scale, y, y_dtype)) return s;
  if (T == 0 || N == 0) return TL_OK;
  return tl::linear_run(x, T, K, N, signs, packed, scales, q, row_scale, y, y_dtype, workspace,
                        workspace_bytes, static_cast<hipStream_t>(stream));
}

// ---------------------------------------------------------------------------
// one step of speculative decoding over a paged cache
int64_t tl_kv_offset(int which, int cache_dtype, int64_t H, int64_t D, int64_t block, int64_t page, int64_t head,
                     int64_t token, int64_t d) {
  if (page < 0 || page >= kMaxDim || check_cache(cache_dtype, page + 1, H, block, D)) return -1;
  if ((which != 0 && which != 1) || head < 0 || head >= H || token < 0 || token >= block || d < 0 || d >= D) return -1;
  const int es = cache_dtype == TL_BF16 ? 2 : 1, t = int(token & (tl::kKvTile - 1));
  const int in_tile = which ? tl::kv_tile_v(t, int(d), es) : tl::kv_tile_k(t, int(d), es);
  return ((page * H + head) * block + token - t) * D + in_tile;
}

int tl_step_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *owned, int64_t R, int32_t *table,
                 int64_t table_width, int64_t block, const int32_t *free_list, int64_t free_count,
                 const int32_t *free_head, const int32_t *parents, int64_t T, int32_t *q_start, int32_t *kv_lens,
                 int64_t *slots, int32_t *positions, uint64_t *tree_mask, int32_t *owned_out,
                 int32_t *free_head_out, void *stream) {
  if (R < 0 || R > tl::kMaxRequests || !count_ok(T) || !count_ok(free_count) || !block_ok(block)) return TL_ERR_SHAPE;
  if (table_width < 0 || table_width > (kMaxDim - 1) / block) return TL_ERR_SHAPE;
  if (any_null(free_head, q_start, free_head_out)) return TL_ERR_NULLPTR;
  if (R && (any_null(ctx_lens, new_lens, owned, kv_lens, owned_out) || (table_width && !table))) return TL_ERR_NULLPTR;
  if (T && (any_null(slots, positions) || (parents && !tree_mask))) return TL_ERR_NULLPTR;
  if (free_count && !free_list) return TL_ERR_NULLPTR;
  if (!aligned_to(4, ctx_lens, new_lens, owned, table, free_list, free_head, parents, q_start, kv_lens, positions,
                  owned_out, free_head_out) ||
      !aligned_to(8, slots, tree_mask))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, t4 = size_t(T) * 4;
  const bool tree = parents && T;
  Span in[] = {{ctx_lens, r4}, {new_lens, r4}, {owned, r4}, {free_list, size_t(free_count) * 4}, {free_head, 4},
               {parents, t4}};
  Span out[] = {{table, r4 * table_width}, {q_start, r4 + 4}, {kv_lens, r4}, {slots, 2 * t4}, {positions, t4},
                {tree ? tree_mask : nullptr, 2 * t4}, {owned_out, r4}, {free_head_out, 4}};
  if (any_alias(in, 6, out, 8)) return TL_ERR_ALIAS;
  tl::StepArgs a = {ctx_lens, new_lens, owned, table, free_list, free_head, parents, q_start, kv_lens, slots, positions,
                    tree ? tree_mask : nullptr, owned_out, free_head_out, free_count, int(T), int(R),
                    int(table_width), int(block)};
  return from_hip(tl::launch_step_plan(a, static_cast<hipStream_t>(stream)));
}

// both cache writers: what tl_kv_write takes, and the norms' arguments
namespace {
int kv_write(tl::WriteArgs a, int64_t T, int64_t H, int64_t D, int64_t Hq, int64_t axes, int64_t max_pos, int64_t rot,
             int cache_dtype, int64_t pages, int64_t block, bool norm, void *stream) {
  if (int s = check_cache(cache_dtype, pages, H, block, D)) return s;
  if (!count_ok(T) || a.ldk < H * D || a.ldv < H * D || a.ldk >= kMaxDim || a.ldv >= kMaxDim) return TL_ERR_SHAPE;
  if (a.q && (Hq < 1 || Hq > 65536 || a.q_head < D || a.q_head >= kMaxDim || a.ldq < (Hq - 1) * a.q_head + D ||
              a.ldq >= kMaxDim))
    return TL_ERR_SHAPE;
  if (a.cos_sin && (rot < 16 || rot % 16 || rot > D || max_pos < 1 || max_pos >= kMaxDim)) return TL_ERR_SHAPE;
  if (a.cos_sin && (axes < 1 || axes > 16)) return TL_ERR_SHAPE;
  if (norm && !(a.eps >= 0.0f && a.eps < __builtin_inff())) return TL_ERR_SHAPE;
  if (!tl::fits_grid(tl::kv_write_groups(T, H, a.q ? Hq : 0, D), 256)) return TL_ERR_SHAPE;
  if (T == 0) return TL_OK;
  const bool e4m3 = cache_dtype == TL_E4M3;
  if (any_null(a.k, a.v, a.slots, a.k_cache, a.v_cache) || (a.q && !a.q_out) || (a.cos_sin && !a.positions))
    return TL_ERR_NULLPTR;
  if (a.cos_sin && axes > 1 && !a.axis_of) return TL_ERR_NULLPTR;
  if (e4m3 && any_null(a.k_scale, a.v_scale)) return TL_ERR_NULLPTR;
  if (!aligned_to(16, a.k, a.v, a.q, a.q_out, a.cos_sin, a.k_cache, a.v_cache, a.q_weight, a.k_weight) || a.ldk % 8 ||
      a.ldv % 8 || (a.q && (a.ldq % 8 || a.q_head % 8)) || !aligned_to(8, a.slots) ||
      !aligned_to(4, a.positions, a.axis_of, a.k_scale, a.v_scale))
    return TL_ERR_ALIGN;
  const size_t kv = cache_bytes(cache_dtype, pages * H * block, D), sc = e4m3 ? size_t(pages) * H * block * 4 : 0;
  Span in[] = {{a.k, (size_t(T - 1) * a.ldk + H * D) * 2},
               {a.v, (size_t(T - 1) * a.ldv + H * D) * 2},
               {a.slots, size_t(T) * 8},
               {a.q, a.q ? (size_t(T - 1) * a.ldq + (Hq - 1) * a.q_head + D) * 2 : 0},
               {a.positions, a.cos_sin ? size_t(T) * axes * 4 : 0},
               {a.cos_sin, a.cos_sin ? size_t(max_pos) * rot * 4 : 0},
               {a.q_weight, a.q ? size_t(D) * 4 : 0},
               {a.k_weight, size_t(D) * 4},
               {a.axis_of, a.cos_sin ? size_t(rot) * 2 : 0}};
  Span out[] = {{a.k_cache, kv}, {a.v_cache, kv}, {a.k_scale, sc}, {a.v_scale, sc},
                {a.q_out, a.q ? size_t(T) * Hq * D * 2 : 0}};
  if (any_alias(in, 9, out, 5)) return TL_ERR_ALIAS;
  a.slot_count = pages * block;
  a.T = int(T);
  a.Hq = int(Hq);
  a.H = int(H);
  a.rot = a.cos_sin ? int(rot) : 0;
  a.max_pos = int(max_pos);
  a.block_shift = log2_of(block);
  a.axes = int(axes);
  return from_hip(tl::launch_kv_write(a, D, e4m3, norm, static_cast<hipStream_t>(stream)));
}
}  // namespace

int tl_kv_write(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int64_t *slots, int64_t T,
                int64_t H, int64_t D, const uint16_t *q, int64_t ldq, int64_t Hq, const int32_t *positions,
                const float *cos_sin, int64_t max_pos, int64_t rot, uint16_t *q_out, void *k_cache, void *v_cache,
                float *k_scale, float *v_scale, int cache_dtype, int64_t pages, int64_t block, void *stream) {
  tl::WriteArgs a = {q, k, v, slots, positions, cos_sin, q_out, k_cache, v_cache, k_scale, v_scale, ldq, ldk, ldv};
  a.q_head = D;
  return kv_write(a, T, H, D, Hq, 1, max_pos, rot, cache_dtype, pages, block, false, stream);
}

int tl_kv_write_norm(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int64_t *slots, int64_t T,
                     int64_t H, int64_t D, const uint16_t *q, int64_t ldq, int64_t q_head, int64_t Hq,
                     const float *q_weight, const float *k_weight, float eps, const int32_t *positions, int64_t axes,
                     const int32_t *axis_of, const float *cos_sin, int64_t max_pos, int64_t rot, uint16_t *q_out,
                     void *k_cache, void *v_cache, float *k_scale, float *v_scale, int cache_dtype, int64_t pages,
                     int64_t block, void *stream) {
  tl::WriteArgs a = {q, k, v, slots, positions, cos_sin, q_out, k_cache, v_cache, k_scale, v_scale, ldq, ldk, ldv};
  a.q_head = q_head;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.axis_of = axis_of;
  a.eps = eps;
  return kv_write(a, T, H, D, Hq, axes, max_pos, rot, cache_dtype, pages, block, true, stream);
}

size_t tl_tree_attention_workspace_size(int64_t max_nodes, int64_t G, int64_t D, int cache_dtype) {
  if (max_nodes < 1 || max_nodes >= kMaxDim || G < 1 || G > 64 || !width_ok(D)) return 0;
  if (cache_dtype != TL_BF16 && cache_dtype != TL_E4M3) return 0;
  return tl::tree_workspace_bytes(max_nodes, G, D, cache_dtype == TL_E4M3);
}

int tl_tree_attention(const uint16_t *q, int64_t ldq, int64_t T, int64_t H, int64_t G, int64_t D, const void *k_cache,
                      const void *v_cache, const float *k_scale, const float *v_scale, int cache_dtype,
                      int64_t pages, int64_t block, const int32_t *table, int64_t table_width, int64_t R,
                      const int32_t *q_start, const int32_t *kv_lens, const uint64_t *tree_mask, float scale,
                      int64_t max_nodes, uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
                      void *stream) {
  if (int s = check_cache(cache_dtype, pages, H, block, D)) return s;
  if (!count_ok(T) || R < 0 || R > tl::kMaxRequests || G < 1 || G > 64 || max_nodes < 1 || max_nodes >= kMaxDim)
    return TL_ERR_SHAPE;
  if (ldq < H * G * D || ldq >= kMaxDim || T * G >= kMaxDim) return TL_ERR_SHAPE;
  if (table_width < 0 || table_width > kMostKeys / block) return TL_ERR_SHAPE;
  if (!(scale > 0.0f && scale < __builtin_inff())) return TL_ERR_SHAPE;
  if (T == 0 || R == 0) return TL_OK;
  // the units of work the kernel counts stay below 2^31, whichever form it takes: 16 rows are
  // the fewest of a block
  if (double(H) * (double(T) * G / 16 + R) * (double(table_width) * block / 128 + 1) >= 2147483648.0) return TL_ERR_SHAPE;
  const bool e4m3 = cache_dtype == TL_E4M3;
  if (any_null(q, k_cache, v_cache, q_start, kv_lens, out) || (table_width && !table)) return TL_ERR_NULLPTR;
  if (e4m3 && any_null(k_scale, v_scale)) return TL_ERR_NULLPTR;
  const size_t need = tl::tree_workspace_bytes(max_nodes, G, D, e4m3);
  if (!workspace || workspace_bytes < need) return TL_ERR_WORKSPACE;
  if (!aligned_to(16, q, k_cache, v_cache, out, workspace) || ldq % 8 || !aligned_to(8, tree_mask) ||
      !aligned_to(4, table, q_start, kv_lens, lse) || (e4m3 && !aligned_to(16, k_scale, v_scale)))
    return TL_ERR_ALIGN;
  const size_t kv = cache_bytes(cache_dtype, pages * H * block, D), sc = e4m3 ? size_t(pages) * H * block * 4 : 0;
  Span in[] = {{q, (size_t(T - 1) * ldq + H * G * D) * 2}, {k_cache, kv}, {v_cache, kv}, {k_scale, sc}, {v_scale, sc},
               {table, size_t(R) * table_width * 4}, {q_start, size_t(R) * 4 + 4}, {kv_lens, size_t(R) * 4},
               {tree_mask, tree_mask ? size_t(T) * 8 : 0}};
  Span o[] = {{out, size_t(T) * H * G * D * 2}, {lse, lse ? size_t(T) * H * G * 4 : 0}, {workspace, need}};
  if (any_alias(in, 9, o, 3)) return TL_ERR_ALIAS;
  tl::TreeArgs a = {};
  a.q = q;
  a.k = static_cast<const char *>(k_cache);
  a.v = static_cast<const char *>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = table;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.tree_mask = tree_mask;
  a.out = out;
  a.lse = lse;
  a.ldq = ldq;
  a.T = int(T);
  a.R = int(R);
  a.H = int(H);
  a.G = int(G);
  a.pages = int(pages);
  a.block_shift = log2_of(block);
  a.table_width = int(table_width);
  a.max_keys = int(table_width * block);
  a.scale = scale;
  return from_hip(tl::launch_tree_attention(a, D, e4m3, max_nodes, workspace, static_cast<hipStream_t>(stream)));
}

size_t tl_tree_verify_workspace_size(int64_t T, int64_t V) {
  if (!count_ok(T) || V < 1 || V >= kMaxDim) return 0;
  return size_t(T) * tl::verify_parts(T, V) * 8;
}

int tl_tree_verify(const void *logits, int logits_dtype, int64_t ld, int64_t T, int64_t V, const int32_t *draft,
                   const int32_t *parents, const int32_t *q_start, int64_t R, int32_t *accepted, int32_t *path,
                   int64_t path_width, int32_t *next, int32_t *target, void *workspace, size_t workspace_bytes,
                   void *stream) {
  if (logits_dtype != TL_BF16 && logits_dtype != TL_F32) return TL_ERR_DTYPE;
  if (!count_ok(T) || R < 0 || R > tl::kMaxRequests || V < 1 || V >= kMaxDim || ld < V || ld >= kMaxDim) return TL_ERR_SHAPE;
  if (path_width < 1 || path_width > TL_TREE_NODES || T * tl::verify_parts(T, V) >= kMaxDim) return TL_ERR_SHAPE;
  if (T == 0 && R == 0) return TL_OK;
  if (!q_start || (T && any_null(logits, draft, parents, target)) || (R && any_null(accepted, path, next)))
    return TL_ERR_NULLPTR;
  const size_t need = tl_tree_verify_workspace_size(T, V), es = logits_dtype == TL_F32 ? 4 : 2;
  if (need && (!workspace || workspace_bytes < need)) return TL_ERR_WORKSPACE;
  if (!aligned_to(es, logits) || !aligned_to(16, workspace) ||
      !aligned_to(4, draft, parents, q_start, accepted, path, next, target))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, t4 = size_t(T) * 4;
  Span in[] = {{logits, T ? (size_t(T - 1) * ld + V) * es : 0}, {draft, t4}, {parents, t4}, {q_start, r4 + 4}};
  Span out[] = {{accepted, r4}, {path, r4 * path_width}, {next, r4}, {target, t4}, {workspace, need}};
  if (any_alias(in, 4, out, 5)) return TL_ERR_ALIAS;
  tl::VerifyArgs a = {logits, draft, parents, q_start, accepted, path, next, target, static_cast<uint64_t *>(workspace),
                      ld, V, int(T), int(R), int(path_width), tl::verify_parts(T, V)};
  return from_hip(tl::launch_tree_verify(a, logits_dtype == TL_F32, static_cast<hipStream_t>(stream)));
}

int tl_kv_commit(const int32_t *accepted, const int32_t *path, int64_t path_width, const int32_t *ctx_lens,
                 const int32_t *kv_lens, const int32_t *table, int64_t table_width, int64_t R, void *k_cache,
                 void *v_cache, float *k_scale, float *v_scale, int cache_dtype, int64_t L, int64_t pages, int64_t H,
                 int64_t block, int64_t D, int32_t *ctx_out, void *stream) {
  if (int s = check_cache(cache_dtype, pages, H, block, D)) return s;
  if (R < 0 || R > tl::kMaxRequests || L < 1 || L > 4096 || path_width < 1 || path_width > TL_TREE_NODES) return TL_ERR_SHAPE;
  if (table_width < 0 || table_width > (kMaxDim - 1) / block || L * R * H >= kMaxDim) return TL_ERR_SHAPE;
  if (pages > (int64_t(1) << 50) / (L * H * block * D)) return TL_ERR_SHAPE;
  if (R == 0) return TL_OK;
  const bool e4m3 = cache_dtype == TL_E4M3;
  if (any_null(accepted, path, ctx_lens, kv_lens, k_cache, v_cache, ctx_out) || (table_width && !table) ||
      (e4m3 && any_null(k_scale, v_scale)))
    return TL_ERR_NULLPTR;
  if (!aligned_to(16, k_cache, v_cache) ||
      !aligned_to(4, accepted, path, ctx_lens, kv_lens, table, k_scale, v_scale, ctx_out))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, tokens = size_t(L) * pages * H * block;
  const size_t kv = cache_bytes(cache_dtype, int64_t(tokens), D), sc = e4m3 ? tokens * 4 : 0;
  Span in[] = {{accepted, r4}, {path, r4 * path_width}, {ctx_lens, r4}, {kv_lens, r4}, {table, r4 * table_width}};
  Span out[] = {{k_cache, kv}, {v_cache, kv}, {k_scale, sc}, {v_scale, sc}, {ctx_out, r4}};
  if (any_alias(in, 5, out, 5)) return TL_ERR_ALIAS;
  tl::CommitArgs a = {accepted, path, ctx_lens, kv_lens, table, static_cast<char *>(k_cache),
                      static_cast<char *>(v_cache), k_scale, v_scale, ctx_out, pages * H * block, int(R), int(L),
                      int(H), int(pages), log2_of(block), int(table_width), int(path_width)};
  return from_hip(tl::launch_kv_commit(a, D, e4m3, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// layers that keep a state per request
namespace {
constexpr int64_t kMostState = int64_t(1) << 50;  // elements
bool requests_ok(int64_t T, int64_t R, int64_t states) {
  return count_ok(T) && R >= 0 && R <= tl::kMaxRequests && states >= 0 && states < kMaxDim;
}
bool delta_heads_ok(int64_t Hk, int64_t G, int64_t Dk, int64_t Dv) {
  return Hk >= 1 && G >= 1 && Hk <= 65535 && G <= 65535 && Hk * G <= 65535 && (Dk == 64 || Dk == 128) && Dv >= 16 &&
         Dv <= 65536 && Dv % 16 == 0;
}
bool distance_ok(int64_t ld, int64_t least) { return ld >= least && ld < kMaxDim; }
}  // namespace

int tl_short_conv(const uint16_t *x, int64_t ldx, int64_t T, int64_t C, const float *weight, int64_t taps,
                  const float *bias, const int32_t *q_start, const int32_t *kv_lens, const int32_t *state_slots,
                  int64_t R, const uint64_t *tree_mask, int64_t norm_heads, int64_t norm_dim, float eps,
                  uint16_t *state, int64_t states, uint16_t *out, int64_t ldo, void *stream) {
  if (!requests_ok(T, R, states) || C < 8 || C > (1 << 20) || C % 8 || taps < 2 || taps > 4) return TL_ERR_SHAPE;
  if (!distance_ok(ldx, C) || !distance_ok(ldo, C)) return TL_ERR_SHAPE;
  if (norm_heads < 0 || (norm_heads && (!width_ok(norm_dim) || norm_heads > C / norm_dim))) return TL_ERR_SHAPE;
  if (norm_heads && !(eps >= 0.0f && eps < __builtin_inff())) return TL_ERR_SHAPE;
  if (states > kMostState / (3 * C) || !tl::conv_fits_grid(T, R)) return TL_ERR_SHAPE;
  if (T == 0 || R == 0) return TL_OK;
  if (any_null(x, weight, q_start, kv_lens, state_slots, out) || (states && !state)) return TL_ERR_NULLPTR;
  if (!aligned_to(16, x, state, out, weight, bias) || ldx % 8 || ldo % 8 || !aligned_to(8, tree_mask) ||
      !aligned_to(4, q_start, kv_lens, state_slots))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, row = size_t(C) * 2;
  Span in[] = {{x, size_t(T - 1) * ldx * 2 + row}, {weight, size_t(C) * taps * 4}, {bias, bias ? size_t(C) * 4 : 0},
               {q_start, r4 + 4}, {kv_lens, r4}, {state_slots, r4}, {tree_mask, tree_mask ? size_t(T) * 8 : 0}};
  Span o[] = {{state, size_t(states) * (taps - 1) * row}, {out, size_t(T - 1) * ldo * 2 + row}};
  if (any_alias(in, 7, o, 2)) return TL_ERR_ALIAS;
  tl::ConvArgs a = {x, weight, bias, q_start, kv_lens, state_slots, tree_mask, state, out, ldx, ldo, states,
                    int(T), int(R), int(C), norm_heads ? int(norm_heads * norm_dim) : 0, int(norm_dim), eps};
  return from_hip(tl::launch_short_conv(a, taps, static_cast<hipStream_t>(stream)));
}

size_t tl_delta_rule_workspace_size(int64_t T, int64_t R, int64_t Hk, int64_t G, int64_t Dk, int64_t max_nodes,
                                    int tree) {
  if (!requests_ok(T, R, 0) || !delta_heads_ok(Hk, G, Dk, 16) || max_nodes < 1 || max_nodes >= kMaxDim) return 0;
  return tl::delta_workspace_bytes(T, R, Hk, G, Dk, max_nodes, tree != 0);
}

int tl_delta_rule(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                  const float *a, int64_t lda, const float *b, int64_t ldb, const float *a_log, const float *dt_bias,
                  int64_t T, int64_t Hk, int64_t G, int64_t Dk, int64_t Dv, const int32_t *q_start,
                  const int32_t *kv_lens, const int32_t *state_slots, int64_t R, const uint64_t *tree_mask, float scale,
                  float *state, int64_t states, int64_t max_nodes, uint16_t *out, void *workspace,
                  size_t workspace_bytes, void *stream) {
  if (!requests_ok(T, R, states) || !delta_heads_ok(Hk, G, Dk, Dv) || max_nodes < 1 || max_nodes >= kMaxDim)
    return TL_ERR_SHAPE;
  const int64_t Hv = Hk * G;
  if (!distance_ok(ldq, Hk * Dk) || !distance_ok(ldk, Hk * Dk) || !distance_ok(ldv, Hv * Dv) || !distance_ok(lda, Hv) ||
      !distance_ok(ldb, Hv))
    return TL_ERR_SHAPE;
  if (states > kMostState / (Hv * Dk * Dv) || !tl::delta_fits_grid(T, R, Hk, G, Dv, max_nodes, tree_mask != nullptr))
    return TL_ERR_SHAPE;
  if (!(scale > -__builtin_inff() && scale < __builtin_inff())) return TL_ERR_SHAPE;
  if (T == 0 || R == 0) return TL_OK;
  if (any_null(q, k, v, a, b, q_start, kv_lens, state_slots, out) || (states && !state) || !a_log != !dt_bias)
    return TL_ERR_NULLPTR;
  const size_t need = tl::delta_workspace_bytes(T, R, Hk, G, Dk, max_nodes, tree_mask != nullptr);
  if (need && (!workspace || workspace_bytes < need)) return TL_ERR_WORKSPACE;
  if (!aligned_to(16, q, k, v, state, out, workspace) || ldq % 8 || ldk % 8 || ldv % 8 || !aligned_to(8, tree_mask) ||
      !aligned_to(4, a, b, a_log, dt_bias, q_start, kv_lens, state_slots))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, h4 = size_t(Hv) * 4, last = size_t(T - 1);
  Span in[] = {{q, (last * ldq + Hk * Dk) * 2}, {k, (last * ldk + Hk * Dk) * 2}, {v, (last * ldv + Hv * Dv) * 2},
               {a, last * lda * 4 + h4}, {b, last * ldb * 4 + h4}, {a_log, a_log ? h4 : 0}, {dt_bias, a_log ? h4 : 0},
               {q_start, r4 + 4}, {kv_lens, r4}, {state_slots, r4}, {tree_mask, tree_mask ? size_t(T) * 8 : 0}};
  Span o[] = {{state, size_t(states) * Hv * Dk * Dv * 4}, {out, size_t(T) * Hv * Dv * 2}, {workspace, need}};
  if (any_alias(in, 11, o, 3)) return TL_ERR_ALIAS;
  tl::DeltaArgs d = {};
  d.q = q, d.k = k, d.v = v, d.a = a, d.b = b, d.a_log = a_log, d.dt_bias = dt_bias;
  d.q_start = q_start, d.kv_lens = kv_lens, d.slots = state_slots, d.tree_mask = tree_mask;
  d.state = state, d.out = out;
  d.ldq = ldq, d.ldk = ldk, d.ldv = ldv, d.lda = lda, d.ldb = ldb, d.state_count = states;
  d.T = int(T), d.R = int(R), d.Hk = int(Hk), d.G = int(G), d.Hv = int(Hv), d.Dv = int(Dv);
  d.scale = scale;
  d.L = 1;
  return from_hip(tl::launch_delta_rule(d, Dk, max_nodes, workspace, static_cast<hipStream_t>(stream)));
}

int tl_delta_commit(const int32_t *accepted, const int32_t *path, int64_t path_width, const int32_t *q_start,
                    const int32_t *kv_lens, const int32_t *state_slots, int64_t R, int64_t T, int64_t L,
                    const uint16_t *k, int64_t ldk, int64_t k_layer, const uint16_t *v, int64_t ldv, int64_t v_layer,
                    const float *a, int64_t lda, int64_t a_layer, const float *b, int64_t ldb, int64_t b_layer,
                    const float *a_log, const float *dt_bias, int64_t Hk, int64_t G, int64_t Dk, int64_t Dv,
                    float *state, int64_t states, const uint16_t *x, int64_t ldx, int64_t x_layer, int64_t C,
                    int64_t taps, uint16_t *conv_state, void *stream) {
  if (!requests_ok(T, R, states) || !delta_heads_ok(Hk, G, Dk, Dv) || L < 1 || L > 4096) return TL_ERR_SHAPE;
  if (path_width < 1 || path_width > TL_TREE_NODES) return TL_ERR_SHAPE;
  const int64_t Hv = Hk * G;
  if (!distance_ok(ldk, Hk * Dk) || !distance_ok(ldv, Hv * Dv) || !distance_ok(lda, Hv) || !distance_ok(ldb, Hv))
    return TL_ERR_SHAPE;
  if (x && (C < 8 || C > (1 << 20) || C % 8 || taps < 2 || taps > 4 || !distance_ok(ldx, C))) return TL_ERR_SHAPE;
  constexpr int64_t far = int64_t(1) << 45;              // of a layer from the next
  if (k_layer < 0 || v_layer < 0 || a_layer < 0 || b_layer < 0 || x_layer < 0 || k_layer > far || v_layer > far ||
      a_layer > far || b_layer > far || x_layer > far)
    return TL_ERR_SHAPE;
  if (states > kMostState / (L * Hv * Dk * Dv) || (x && states > kMostState / (L * 3 * C))) return TL_ERR_SHAPE;
  if (!tl::fits_grid(tl::delta_commit_groups(L, R, Hv, Dv, x ? C : 0), 256)) return TL_ERR_SHAPE;
  if (T == 0 || R == 0) return TL_OK;
  if (any_null(accepted, path, q_start, kv_lens, state_slots, k, v, a, b) || (states && !state) || !a_log != !dt_bias ||
      (x && states && !conv_state))
    return TL_ERR_NULLPTR;
  if (!aligned_to(16, k, v, state, x, conv_state) || ldk % 8 || ldv % 8 || k_layer % 8 || v_layer % 8 ||
      (x && (ldx % 8 || x_layer % 8)) || !aligned_to(4, accepted, path, q_start, kv_lens, state_slots, a, b, a_log, dt_bias))
    return TL_ERR_ALIGN;
  const size_t r4 = size_t(R) * 4, h4 = size_t(Hv) * 4, last = size_t(T - 1), m = size_t(L - 1);
  Span in[] = {{accepted, r4}, {path, r4 * path_width}, {q_start, r4 + 4}, {kv_lens, r4}, {state_slots, r4},
               {k, (m * k_layer + last * ldk + Hk * Dk) * 2}, {v, (m * v_layer + last * ldv + Hv * Dv) * 2},
               {a, (m * a_layer + last * lda) * 4 + h4}, {b, (m * b_layer + last * ldb) * 4 + h4},
               {a_log, a_log ? L * h4 : 0}, {dt_bias, a_log ? L * h4 : 0},
               {x, x ? (m * x_layer + last * ldx + C) * 2 : 0}};
  Span o[] = {{state, size_t(L) * states * Hv * Dk * Dv * 4}, {x ? conv_state : nullptr, size_t(L) * states * (taps - 1) * C * 2}};
  if (any_alias(in, 12, o, 2)) return TL_ERR_ALIAS;
  tl::DeltaArgs d = {};
  d.k = k, d.v = v, d.a = a, d.b = b, d.a_log = a_log, d.dt_bias = dt_bias;
  d.q_start = q_start, d.kv_lens = kv_lens, d.slots = state_slots;
  d.state = state;
  d.ldk = ldk, d.ldv = ldv, d.lda = lda, d.ldb = ldb, d.state_count = states;
  d.T = int(T), d.R = int(R), d.Hk = int(Hk), d.G = int(G), d.Hv = int(Hv), d.Dv = int(Dv);
  d.accepted = accepted, d.path = path, d.x = x, d.conv_state = conv_state;
  d.k_layer = k_layer, d.v_layer = v_layer, d.a_layer = a_layer, d.b_layer = b_layer, d.x_layer = x_layer, d.ldx = ldx;
  d.path_width = int(path_width), d.L = int(L), d.C = int(C), d.taps = int(taps);
  return from_hip(tl::launch_delta_commit(d, Dk, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
