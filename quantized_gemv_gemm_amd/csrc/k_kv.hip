// Rows of the paged K/V cache: a step's rows written (with the rotary embedding and, for
// an 8-bit cache, the quantisation), and accepted rows moved together.
//
// kv_write, with h = rot / 2 and (c, s) the table's row of the token's position:
//   x'[d] = x[d] c[d] - x[d + h] s[d],  x'[d + h] = x[d + h] c[d] + x[d] s[d]   (d < h)
//   x'[d] = x[d] (d >= rot), rounded to bf16, for q (to q_out) and k; v as it is;
//   e4m3: scale = max |x'| / 448, code = e4m3(x' / scale) for each token and head.
// kv_write_norm (NORM) takes x w / sqrt(mean of the head's x^2 + eps) in the place of x for q and
// k, an axis of positions for each pair of elements, and rounds only what it stores: an e4m3
// row's scale and codes are those of the f32 values.
// Products and sums are rounded one by one (no fused multiply-add) and the divisions are
// IEEE ones, so the codes are those of the plain formula.
//
// What bounds it is memory: 2 (Hq + 2 H) D bytes a token read, q_out and the cache rows
// written (8191 tokens, 32 + 2 x 8 heads of 128, into e4m3: 40 to 44 us, 4.3 to 4.7 TB/s,
// where a large copy reaches 4.9; 128 tokens of 256-wide heads 7.4 us, latency).  A thread holds 16 elements of a row: 8 and their 8 partners h further on, or
// 16 consecutive ones past rot; D / 16 neighbouring lanes hold a row, so its maximum is
// a few shuffles.  A K row's elements lie in 16-byte runs in the cache and are stored
// from registers.  V's run is 8 consecutive tokens of one d: a workgroup takes 16 tokens
// of one head through LDS and stores whole runs where the tokens' slots make them up
// (a prompt), and single elements elsewhere (a tree, a run's ragged ends).
#include "kv_layout.h"
#include "tl_device.h"

namespace tl {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;      // of a workgroup of the cache part
constexpr int kRun = 8;          // tokens of a run of V
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct Row16 {
  u32x4 a, b;  // bf16 elements lo .. lo + 7 and hi .. hi + 7
};

// The 16 elements that piece p (of D / 16) of a row holds begin at lo and hi.
__device__ __forceinline__ void piece(int p, int rot, int &lo, int &hi) {
  if (16 * p < rot) {
    lo = 8 * p;
    hi = lo + rot / 2;
  } else {
    lo = 16 * p;
    hi = lo + 8;
  }
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

__device__ __forceinline__ void rotate(Row16 &x, const float *cs, int h, int lo) {
  const float4 *c = reinterpret_cast<const float4 *>(cs + lo), *s = reinterpret_cast<const float4 *>(cs + h + lo);
  const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
  const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a0 = lo_bf16(x.a[e]), a1 = hi_bf16(x.a[e]), b0 = lo_bf16(x.b[e]), b1 = hi_bf16(x.b[e]);
    const int i = 2 * e;
    x.a[e] = pack2(a0 * cc[i] - b0 * ss[i], a1 * cc[i + 1] - b1 * ss[i + 1]);
    x.b[e] = pack2(b0 * cc[i] + a0 * ss[i], b1 * cc[i + 1] + a1 * ss[i + 1]);
  }
}

__device__ __forceinline__ const float *angles(const WriteArgs &a, int t) {
  const int pos = min(max(a.positions[t], 0), a.max_pos - 1);
  return a.cos_sin + int64_t(pos) * a.rot;
}

__device__ __forceinline__ float largest(const Row16 &x) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    m = fmaxf(fmaxf(m, fabsf(lo_bf16(x.a[e]))), fabsf(hi_bf16(x.a[e])));
    m = fmaxf(fmaxf(m, fabsf(lo_bf16(x.b[e]))), fabsf(hi_bf16(x.b[e])));
  }
  return m;
}

// four bf16 -> four e4m3 codes of x / scale
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float scale) {
  const bool some = scale > 0.0f;
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(some ? lo_bf16(w0) / scale : 0.0f, some ? hi_bf16(w0) / scale : 0.0f, 0, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(some ? lo_bf16(w1) / scale : 0.0f, some ? hi_bf16(w1) / scale : 0.0f, c, true);
  return uint32_t(c);
}

// A piece of a row in f32: elements lo .. lo + 7 and hi .. hi + 7.
struct Piece16 {
  float a[8], b[8];
};

__device__ __forceinline__ void load8(const float *from, float (&to)[8]) {
  const float4 x = reinterpret_cast<const float4 *>(from)[0], y = reinterpret_cast<const float4 *>(from)[1];
  to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w, to[4] = y.x, to[5] = y.y, to[6] = y.z, to[7] = y.w;
}

// Cosines and sines of `count` tokens from t0 on, [count][rot], to LDS: each pair's angle goes by
// its own axis of positions.  The workgroup passes a barrier before it reads them.
__device__ __forceinline__ void stage_angles(const WriteArgs &a, int t0, int count, float *to) {
  const int h = a.rot / 2;
  for (int u = threadIdx.x; u < count * h; u += kThreads) {
    const int i = u / h, d = u - i * h;
    const int32_t *at_t = a.positions + min(t0 + i, a.T - 1);
    int pos = at_t[0];
    if (a.axis_of && a.axes <= 3) {                      // asked for beside the axis, not after it
      const int axis = a.axis_of[d], second = at_t[a.axes > 1 ? a.T : 0], third = at_t[a.axes > 2 ? 2 * int64_t(a.T) : 0];
      pos = axis <= 0 || a.axes == 1 ? pos : axis == 1 || a.axes == 2 ? second : third;
    } else if (a.axis_of) {
      pos = at_t[int64_t(min(max(a.axis_of[d], 0), a.axes - 1)) * a.T];
    }
    pos = min(max(pos, 0), a.max_pos - 1);
    const float *at = a.cos_sin + int64_t(pos) * a.rot + d;
    to[i * a.rot + d] = at[0];
    to[i * a.rot + h + d] = at[h];
  }
}

// Piece p's elements of the weights, or ones.
struct Weight16 {
  float a[8], b[8];
};
__device__ __forceinline__ Weight16 weights(const float *weight, int lo, int hi) {
  Weight16 w;
  if (weight) {
    load8(weight + lo, w.a);
    load8(weight + hi, w.b);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w.a[e] = w.b[e] = 1.0f;
  }
  return w;
}

// Piece p of a row, normalised and turned by its token's staged angles.  The P lanes of a row
// call it together.
template <int P>
__device__ __forceinline__ Piece16 normed(const Row16 &x, const WriteArgs &a, const Weight16 &w, const float *angle, int p,
                                          int lo) {
  Piece16 y;
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y.a[2 * e] = lo_bf16(x.a[e]), y.a[2 * e + 1] = hi_bf16(x.a[e]);
    y.b[2 * e] = lo_bf16(x.b[e]), y.b[2 * e + 1] = hi_bf16(x.b[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = fmaf(y.a[e], y.a[e], fmaf(y.b[e], y.b[e], sum));
#pragma unroll
  for (int off = P / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  const float by = 1.0f / sqrtf(sum / float(16 * P) + a.eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y.a[e] = y.a[e] * by * w.a[e];
    y.b[e] = y.b[e] * by * w.b[e];
  }
  if (16 * p < a.rot) {                                  // pairs lo .. lo + 7
    float c[8], s[8];
    load8(angle + lo, c);
    load8(angle + a.rot / 2 + lo, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = y.a[e], v = y.b[e];
      y.a[e] = u * c[e] - v * s[e];
      y.b[e] = v * c[e] + u * s[e];
    }
  }
  return y;
}

__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  return u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}

// A magnitude's bits rise with it, and a NaN's are above infinity's: their maximum is NaN where an
// element is, and a row that is not finite does not pass for a row of zeros.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float scale) {
  const bool some = scale != 0.0f;                       // NaN too: its codes are NaN
  u32x2 o;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = some ? x[4 * e + j] / scale : 0.0f;
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
    o[e] = uint32_t(c);
  }
  return o;
}

// With norms, the angles of a workgroup's tokens are staged once, for all their heads, beside the
// rows and the weights: one after another the loads of a prompt took 98 us where this takes 70
// (8191 tokens, 24 + 2 x 4 heads of 256, three axes: 270 MB at 3.9 TB/s).  Four rows of q a
// thread, its weights kept in registers, took 74.
template <int D, bool E4M3, bool NORM>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(const WriteArgs a, int cache_groups) {
  constexpr int kAngles = kThreads / (D / 16);           // tokens whose angles have a place
  __shared__ __attribute__((aligned(16))) float s_angle[NORM ? kAngles * D : 4];
  constexpr int P = D / 16;                              // pieces (lanes) of a row
  constexpr int ES = E4M3 ? 1 : 2;
  const int tid = threadIdx.x, h = a.rot / 2;
  if (int(blockIdx.x) >= cache_groups) {                 // q
    if constexpr (NORM) {
      const int64_t rows = int64_t(a.T) * a.Hq, row0 = int64_t(blockIdx.x - cache_groups) * kAngles;
      const uint32_t heads = uint32_t(a.Hq), here = uint32_t(min(rows - row0, int64_t(kAngles)));
      const int p = tid % P, t0 = rows <= 0xFFFFFFFF ? int(uint32_t(row0) / heads) : int(row0 / a.Hq);
      const uint32_t first = uint32_t(row0 - int64_t(t0) * a.Hq);  // head of the group's first row
      const int tokens = int((first + here - 1) / heads) + 1;
      int lo, hi;
      piece(p, a.rot, lo, hi);
      const uint32_t at = first + min(uint32_t(tid / P), here - 1);  // past the last row it is the last one again
      const int token = int(at / heads);
      const uint16_t *src = a.q + int64_t(t0 + token) * a.ldq + int64_t(at - token * heads) * a.q_head;
      const Row16 x = {*reinterpret_cast<const u32x4 *>(src + lo), *reinterpret_cast<const u32x4 *>(src + hi)};
      const Weight16 w = weights(a.q_weight, lo, hi);
      if (a.rot) stage_angles(a, t0, tokens, s_angle);
      __syncthreads();
      const Piece16 y = normed<P>(x, a, w, s_angle + token * a.rot, p, lo);
      const int64_t row = row0 + tid / P;
      if (row < rows) {
        *reinterpret_cast<u32x4 *>(a.q_out + row * D + lo) = pack8(y.a);
        *reinterpret_cast<u32x4 *>(a.q_out + row * D + hi) = pack8(y.b);
      }
    } else {
      const int64_t row = int64_t(blockIdx.x - cache_groups) * (kThreads / P) + tid / P;
      if (row >= int64_t(a.T) * a.Hq) return;
      const int t = int(row / a.Hq), head = int(row - int64_t(t) * a.Hq), p = tid % P;
      int lo, hi;
      piece(p, a.rot, lo, hi);
      const uint16_t *src = a.q + t * a.ldq + int64_t(head) * D;
      Row16 x = {*reinterpret_cast<const u32x4 *>(src + lo), *reinterpret_cast<const u32x4 *>(src + hi)};
      if (16 * p < a.rot) rotate(x, angles(a, t), h, lo);
      uint16_t *dst = a.q_out + row * D;
      *reinterpret_cast<u32x4 *>(dst + lo) = x.a;
      *reinterpret_cast<u32x4 *>(dst + hi) = x.b;
    }
    return;
  }

  // K and V of 16 tokens of one head
  __shared__ __attribute__((aligned(16))) char v_rows[(kTokens + kRun - 1) * (D * ES + 4)];
  __shared__ int64_t s_slot[kTokens + kRun];             // [0]: the slot before the first token
  const int head = int(blockIdx.x) % a.H, t0 = int(blockIdx.x) / a.H * kTokens;
  if (tid < kTokens + kRun) {
    const int t = t0 + tid - 1;
    int64_t s = t >= 0 && t < a.T ? a.slots[t] : -1;
    s_slot[tid] = s >= 0 && s < a.slot_count ? s : -1;
  }
  // with norms, rows are asked for beside their slots, and for the first round of the loop below
  // before the barrier
  auto ask = [&](const uint16_t *rows, int64_t ld, int u, int lo, int hi) {
    const uint16_t *src = rows + int64_t(min(t0 + u / P, a.T - 1)) * ld + int64_t(head) * D;
    return Row16{*reinterpret_cast<const u32x4 *>(src + lo), *reinterpret_cast<const u32x4 *>(src + hi)};
  };
  Row16 first_v, first_k;
  if constexpr (NORM) {
    int lo, hi;
    piece(tid % P, a.rot, lo, hi);
    first_v = ask(a.v, a.ldv, tid, 16 * (tid % P), 16 * (tid % P) + 8);
    first_k = ask(a.k, a.ldk, tid, lo, hi);
    if (a.rot) stage_angles(a, t0, min(kTokens, a.T - t0), s_angle);
  }
  __syncthreads();
  const int mask = (1 << a.block_shift) - 1;
  // element offset of the tile that holds a slot of this head
  auto tile_of = [&](int64_t slot) {
    return ((((slot >> a.block_shift) * a.H + head) << a.block_shift) + (slot & mask & ~15)) * D;
  };
  auto scale_of = [&](int64_t slot) { return (((slot >> a.block_shift) * a.H + head) << a.block_shift) + (slot & mask); };

  constexpr int PITCH = D * ES + 4;                      // bytes of a row in LDS
  for (int u = tid; u < (kTokens + kRun - 1) * P; u += kThreads) {
    const int i = u / P, p = u % P, t = t0 + i;
    const int64_t slot = s_slot[i + 1];
    const bool live = t < a.T && slot >= 0;              // the lanes of a row agree
    // V: also the tokens that a run begun here goes on to
    Row16 x = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if constexpr (NORM) {
      x = u == tid ? first_v : ask(a.v, a.ldv, u, 16 * p, 16 * p + 8);
      if (!live) x = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    } else if (live) {
      const uint16_t *src = a.v + t * a.ldv + int64_t(head) * D + 16 * p;
      x = {*reinterpret_cast<const u32x4 *>(src), *reinterpret_cast<const u32x4 *>(src + 8)};
    }
    uint32_t *row = reinterpret_cast<uint32_t *>(v_rows + i * PITCH);
    if constexpr (E4M3) {
      float m = largest(x);
#pragma unroll
      for (int off = P / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
      const float scale = m / 448.0f;
      if (live && p == 0 && i < kTokens) a.v_scale[scale_of(slot)] = scale;
      row[4 * p + 0] = codes4(x.a[0], x.a[1], scale);
      row[4 * p + 1] = codes4(x.a[2], x.a[3], scale);
      row[4 * p + 2] = codes4(x.b[0], x.b[1], scale);
      row[4 * p + 3] = codes4(x.b[2], x.b[3], scale);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row[8 * p + e] = x.a[e];
        row[8 * p + 4 + e] = x.b[e];
      }
    }
    if (i >= kTokens) continue;                          // whole rows of lanes: the shuffles below agree
    Row16 k = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    int lo, hi;
    piece(p, a.rot, lo, hi);
    if constexpr (NORM) {
      k = u == tid ? first_k : ask(a.k, a.ldk, u, lo, hi);
    } else if (live) {
      const uint16_t *src = a.k + t * a.ldk + int64_t(head) * D;
      k = {*reinterpret_cast<const u32x4 *>(src + lo), *reinterpret_cast<const u32x4 *>(src + hi)};
      if (16 * p < a.rot) rotate(k, angles(a, t), h, lo);
    }
    const int in_tile = int(slot & 15);
    Piece16 y;
    if constexpr (NORM) {                                // rows past the last token are an existing token's
      y = normed<P>(k, a, weights(a.k_weight, lo, hi), s_angle + min(i, a.T - 1 - t0) * a.rot, p, lo);
      if constexpr (!E4M3) k = {pack8(y.a), pack8(y.b)};
    }
    if constexpr (E4M3 && NORM) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(max(m, magnitude(y.a[e])), magnitude(y.b[e]));
#pragma unroll
      for (int off = P / 2; off > 0; off >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), off, 64)));
      const float scale = __uint_as_float(m) / 448.0f;
      if (live) {
        if (p == 0) a.k_scale[scale_of(slot)] = scale;
        char *dst = static_cast<char *>(a.k_cache) + tile_of(slot);
        *reinterpret_cast<u32x2 *>(dst + kv_tile_k(in_tile, lo, 1)) = codes8(y.a, scale);
        *reinterpret_cast<u32x2 *>(dst + kv_tile_k(in_tile, hi, 1)) = codes8(y.b, scale);
      }
    } else if constexpr (E4M3) {
      float m = largest(k);
#pragma unroll
      for (int off = P / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
      const float scale = m / 448.0f;
      if (live) {
        if (p == 0) a.k_scale[scale_of(slot)] = scale;
        char *dst = static_cast<char *>(a.k_cache) + tile_of(slot);
        const u32x2 c0 = {codes4(k.a[0], k.a[1], scale), codes4(k.a[2], k.a[3], scale)};
        const u32x2 c1 = {codes4(k.b[0], k.b[1], scale), codes4(k.b[2], k.b[3], scale)};
        *reinterpret_cast<u32x2 *>(dst + kv_tile_k(in_tile, lo, 1)) = c0;
        *reinterpret_cast<u32x2 *>(dst + kv_tile_k(in_tile, hi, 1)) = c1;
      }
    } else if (live) {
      uint16_t *dst = static_cast<uint16_t *>(a.k_cache) + tile_of(slot);
      *reinterpret_cast<u32x4 *>(dst + kv_tile_k(in_tile, lo, 2)) = k.a;
      *reinterpret_cast<u32x4 *>(dst + kv_tile_k(in_tile, hi, 2)) = k.b;
    }
  }
  __syncthreads();

  // V from LDS: the first token of a run, or of what there is of one, stores it.  A run is
  // consecutive slots within one aligned 8 of them.
  constexpr int U = 16 / (kRun * ES);                    // d's (16 apart) of a 16-byte piece
  for (int u = tid; u < kTokens * D / U; u += kThreads) {
    const int i = u / (D / U), q = u % (D / U);          // token, piece of the run
    const int64_t slot = s_slot[i + 1];
    if (slot < 0 || (s_slot[i] >= 0 && s_slot[i] + 1 == slot && (slot & (kRun - 1)) != 0)) continue;
    int n = 1;                                           // on into the next workgroup's tokens if need be
    while (((slot + n) & (kRun - 1)) != 0 && s_slot[i + 1 + n] == slot + n) ++n;
    const int d = q / 16 * (16 * U) + q % 16;
    char *dst = static_cast<char *>(a.v_cache) + (tile_of(slot) + kv_tile_v(int(slot & 15), d, ES)) * ES;
    if (n == kRun) {
      u32x4 w;
      if constexpr (E4M3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t v = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v |= uint32_t(*reinterpret_cast<const uint8_t *>(v_rows + (i + 4 * (e & 1) + b) * PITCH + d + 16 * (e >> 1))) << (8 * b);
          w[e] = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = uint32_t(*reinterpret_cast<const uint16_t *>(v_rows + (i + 2 * e) * PITCH + 2 * d)) |
                 uint32_t(*reinterpret_cast<const uint16_t *>(v_rows + (i + 2 * e + 1) * PITCH + 2 * d)) << 16;
      }
      *reinterpret_cast<u32x4 *>(dst) = w;
    } else {
      for (int k = 0; k < n; ++k) {
        if constexpr (E4M3) {
          dst[k] = v_rows[(i + k) * PITCH + d];
          dst[k + 8] = v_rows[(i + k) * PITCH + d + 16];
        } else {
          reinterpret_cast<uint16_t *>(dst)[k] = *reinterpret_cast<const uint16_t *>(v_rows + (i + k) * PITCH + 2 * d);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Rows ctx + path[i] of a request go to ctx + i, as many as the path has.  A workgroup takes one layer, request
// and head, and the elements lie in threads' registers while they move, up to 4096 of V at
// a time: some d's of every row, all read before one is written, so paths may overlap
// their targets.  What bounds it is the chain of loads to the first row (lengths, path,
// page, row; 17 nodes of one layer 4.2 us) and, over many requests and layers, V's lines: a
// token's values are 2 (1) bytes of every 16, so moving one touches the lines of eight (64
// requests of 64 nodes, 16 layers of 4 256-wide e4m3 heads: 26 us).
template <int D, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_commit_kernel(const CommitArgs a) {
  constexpr int ES = E4M3 ? 1 : 2;
  constexpr int VN = 16, KN = VN * ES / 16 > 0 ? VN * ES / 16 : 1;  // registers of a pass: elements of V, pieces of K
  // of a move's source and target: the token, and its row's first byte in K and in V
  struct Place {
    int64_t token, k, v;
  };
  __shared__ Place s_src[kTreeNodes], s_dst[kTreeNodes];
  __shared__ int s_count;
  const int tid = threadIdx.x;
  int b = blockIdx.x;
  const int head = b % a.H;
  b /= a.H;
  const int r = b % a.R, layer = b / a.R;
  const int ctx = max(a.ctx_lens[r], 0), n = max(max(a.kv_lens[r], 0) - ctx, 0);  // not served: no new tokens
  const int block = 1 << a.block_shift;
  // a tree's accepted nodes as far as the path names them (a chain's lie where they belong)
  const int count = min(max(a.accepted[r], 0), n <= kTreeNodes ? min(n, a.path_width) : n);
  const int from = tid < a.path_width ? a.path[int64_t(r) * a.path_width + tid] : -1;
  if (tid == 0 && head == 0 && layer == 0) a.ctx_out[r] = ctx + count;
  if (n > kTreeNodes || count == 0) return;
  if (tid < 64) {
    int64_t src = -1, dst = -1;
    if (tid < count && from > tid && from < n) {
      auto token = [&](int pos) -> int64_t {
        const int page = pos >> a.block_shift;
        if (page >= a.table_width) return -1;
        const int id = a.table[int64_t(r) * a.table_width + page];
        if (uint32_t(id) >= uint32_t(a.pages)) return -1;
        return ((int64_t(id) * a.H + head) << a.block_shift) + (pos & (block - 1));
      };
      src = token(ctx + from);
      dst = token(ctx + tid);
    }
    const bool go = src >= 0 && dst >= 0;
    const uint64_t all = __ballot(go);
    const int at = __popcll(all & ((uint64_t(1) << tid) - 1));   // the moves, without gaps
    if (go) {
      const int64_t base = layer * a.layer_tokens;       // tokens before this layer's cache
      auto place = [&](int64_t tok) {
        const int64_t tile = (base + (tok & ~int64_t(15))) * (D * ES);
        return Place{base + tok, tile + kv_k_token(int(tok & 15)), tile + kv_v_token(int(tok & 15), ES)};
      };
      s_src[at] = place(src);
      s_dst[at] = place(dst);
    }
    if (tid == 0) s_count = __popcll(all);
  }
  __syncthreads();
  const int moves = s_count;
  if (moves == 0) return;

  int log_d = D == 64 ? 6 : D == 128 ? 7 : 8;            // d's of a pass, a power of two
  while (moves << log_d > VN * kThreads) --log_d;
  const int log_k = log_d + (E4M3 ? 0 : 1) - 4;          // 16-byte pieces of K
  for (int d0 = 0; d0 < D; d0 += 1 << log_d) {
    const int p0 = d0 * ES / 16;
    u32x4 k[KN];
    uint32_t v[VN];
    float ks = 0, vs = 0;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
      if (i * kThreads >= moves << log_k) break;         // uniform
      const int u = i * kThreads + tid, row = u >> log_k, p = p0 + u - (row << log_k);
      if (row < moves) k[i] = *reinterpret_cast<const u32x4 *>(a.k_cache + s_src[row].k + kv_k_piece(p));
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      if (i * kThreads >= moves << log_d) break;
      const int u = i * kThreads + tid, row = u >> log_d, d = d0 + u - (row << log_d);
      if (row < moves) {
        const char *p = a.v_cache + s_src[row].v + kv_v_element(d, ES);
        if constexpr (E4M3) v[i] = *reinterpret_cast<const uint8_t *>(p);
        else v[i] = *reinterpret_cast<const uint16_t *>(p);
      }
    }
    const bool scales = E4M3 && d0 == 0 && tid < moves;
    if (scales) {
      ks = a.k_scale[s_src[tid].token];
      vs = a.v_scale[s_src[tid].token];
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                  // every load has returned
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KN; ++i) {
      if (i * kThreads >= moves << log_k) break;
      const int u = i * kThreads + tid, row = u >> log_k, p = p0 + u - (row << log_k);
      if (row < moves) *reinterpret_cast<u32x4 *>(a.k_cache + s_dst[row].k + kv_k_piece(p)) = k[i];
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      if (i * kThreads >= moves << log_d) break;
      const int u = i * kThreads + tid, row = u >> log_d, d = d0 + u - (row << log_d);
      if (row < moves) {
        char *p = a.v_cache + s_dst[row].v + kv_v_element(d, ES);
        if constexpr (E4M3) *reinterpret_cast<uint8_t *>(p) = uint8_t(v[i]);
        else *reinterpret_cast<uint16_t *>(p) = uint16_t(v[i]);
      }
    }
    if (scales) {
      a.k_scale[s_dst[tid].token] = ks;
      a.v_scale[s_dst[tid].token] = vs;
    }
  }
}

int64_t cache_groups(int64_t T, int64_t H) { return (T + kTokens - 1) / kTokens * H; }

template <int D, bool E4M3, bool NORM>
hipError_t write_rows(const WriteArgs &a, hipStream_t stream) {
  const int64_t cache = cache_groups(a.T, a.H), all = kv_write_groups(a.T, a.H, a.q ? a.Hq : 0, D);
  if (!fits_grid(all, kThreads)) return hipErrorInvalidValue;
  (void)hipGetLastError();
  hipLaunchKernelGGL((kv_write_kernel<D, E4M3, NORM>), dim3(unsigned(all)), dim3(kThreads), 0, stream, a, int(cache));
  set_last_kernel(NORM ? E4M3 ? "kv_write_norm_e4m3" : "kv_write_norm_bf16" : E4M3 ? "kv_write_e4m3" : "kv_write_bf16");
  return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t commit_rows(const CommitArgs &a, hipStream_t stream) {
  const int64_t grid = int64_t(a.L) * a.R * a.H;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  (void)hipGetLastError();
  hipLaunchKernelGGL((kv_commit_kernel<D, E4M3>), dim3(unsigned(grid)), dim3(kThreads), 0, stream, a);
  set_last_kernel(E4M3 ? "kv_commit_e4m3" : "kv_commit_bf16");
  return hipGetLastError();
}

}  // namespace

template <bool E4M3>
static hipError_t write_of(const WriteArgs &a, int64_t D, bool norm, hipStream_t stream) {
  if (norm) {
    return D == 64    ? write_rows<64, E4M3, true>(a, stream)
           : D == 128 ? write_rows<128, E4M3, true>(a, stream)
                      : write_rows<256, E4M3, true>(a, stream);
  }
  return D == 64    ? write_rows<64, E4M3, false>(a, stream)
         : D == 128 ? write_rows<128, E4M3, false>(a, stream)
                    : write_rows<256, E4M3, false>(a, stream);
}

int64_t kv_write_groups(int64_t T, int64_t H, int64_t Hq, int64_t D) {
  const int64_t of_group = kThreads / (D / 16);          // rows of q
  return cache_groups(T, H) + (T * Hq + of_group - 1) / of_group;
}

hipError_t launch_kv_write(const WriteArgs &a, int64_t D, bool e4m3, bool norm, hipStream_t stream) {
  return e4m3 ? write_of<true>(a, D, norm, stream) : write_of<false>(a, D, norm, stream);
}

hipError_t launch_kv_commit(const CommitArgs &a, int64_t D, bool e4m3, hipStream_t stream) {
  if (e4m3) return D == 64 ? commit_rows<64, true>(a, stream) : D == 128 ? commit_rows<128, true>(a, stream) : commit_rows<256, true>(a, stream);
  return D == 64 ? commit_rows<64, false>(a, stream) : D == 128 ? commit_rows<128, false>(a, stream) : commit_rows<256, false>(a, stream);
}

}  // namespace tl
