// Rows of the paged K/V cache: a step's rows written (with the rotary embedding and, for
// an 8-bit cache, the quantisation), and accepted rows moved together.
//
// kv_write, with h = rot / 2 and (c, s) the table's row of the token's position:
//   x'[d] = x[d] c[d] - x[d + h] s[d],  x'[d + h] = x[d + h] c[d] + x[d] s[d]   (d < h)
//   x'[d] = x[d] (d >= rot), rounded to bf16, for q (to q_out) and k; v as it is;
//   e4m3: scale = max |x'| / 448, code = e4m3(x' / scale) for each token and head.
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

template <int D, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(const WriteArgs a, int cache_groups) {
  constexpr int P = D / 16;                              // pieces (lanes) of a row
  constexpr int ES = E4M3 ? 1 : 2;
  const int tid = threadIdx.x, h = a.rot / 2;
  if (int(blockIdx.x) >= cache_groups) {                 // q
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
    if (live) {
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
    if (live) {
      const uint16_t *src = a.k + t * a.ldk + int64_t(head) * D;
      k = {*reinterpret_cast<const u32x4 *>(src + lo), *reinterpret_cast<const u32x4 *>(src + hi)};
      if (16 * p < a.rot) rotate(k, angles(a, t), h, lo);
    }
    const int in_tile = int(slot & 15);
    if constexpr (E4M3) {
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

template <int D, bool E4M3>
hipError_t write_rows(const WriteArgs &a, hipStream_t stream) {
  const int64_t cache = (int64_t(a.T) + kTokens - 1) / kTokens * a.H;
  const int64_t q = a.q ? (int64_t(a.T) * a.Hq + kThreads / (D / 16) - 1) / (kThreads / (D / 16)) : 0;
  if (cache + q > 0x7FFFFFFF) return hipErrorInvalidValue;
  (void)hipGetLastError();
  hipLaunchKernelGGL((kv_write_kernel<D, E4M3>), dim3(unsigned(cache + q)), dim3(kThreads), 0, stream, a, int(cache));
  set_last_kernel(E4M3 ? "kv_write_e4m3" : "kv_write_bf16");
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

hipError_t launch_kv_write(const WriteArgs &a, int64_t D, bool e4m3, hipStream_t stream) {
  if (e4m3) return D == 64 ? write_rows<64, true>(a, stream) : D == 128 ? write_rows<128, true>(a, stream) : write_rows<256, true>(a, stream);
  return D == 64 ? write_rows<64, false>(a, stream) : D == 128 ? write_rows<128, false>(a, stream) : write_rows<256, false>(a, stream);
}

hipError_t launch_kv_commit(const CommitArgs &a, int64_t D, bool e4m3, hipStream_t stream) {
  if (e4m3) return D == 64 ? commit_rows<64, true>(a, stream) : D == 128 ? commit_rows<128, true>(a, stream) : commit_rows<256, true>(a, stream);
  return D == 64 ? commit_rows<64, false>(a, stream) : D == 128 ? commit_rows<128, false>(a, stream) : commit_rows<256, false>(a, stream);
}

}  // namespace tl
