// The gated delta rule.  Each request keeps for each value head a state S [Dk, Dv] in f32;
// token by token, with log decay g and step b,
//   S <- exp(g) S + k u^T,   u = b (v - exp(g) S^T k),   out = scale S^T q.
//
// Few tokens (delta_step_kernel): token by token, the state in registers.
//
// Many tokens and drafted trees: chunks of 64.  With D_i the sum of the log decays of token i
// and its ancestors (all before it, in a chain) and j running over i's ancestors,
//   u_i = b_i (v_i - exp(D_i) S^T k_i - sum_j exp(D_i - D_j) (k_i k_j) u_j),
// so U = T (V - exp(D) K S) with T = (I + A)^-1 diag(b), A_ij = b_i exp(D_i - D_j) k_i k_j, and
//   out_i = scale (exp(D_i) S^T q_i + sum_j P_ij u_j),  P_ij = exp(D_i - D_j) q_i k_j (j = i too),
//   S <- exp(D_last) S + sum_j k_j (exp(D_last - D_j) u_j)^T.
// T and P need no state: delta_prep_kernel makes them for all chunks at once, and
// delta_scan_kernel walks a request's chunks with 32 columns of a head's state in registers.
// Where a call's requests have one chunk each, delta_chunk_kernel does both in one launch.
//
// Products run on the bf16 matrix instructions.  q and k are bf16; an f32 operand is the sum
// of three bf16 parts of 8 bits each, cut off exactly (x = hi + mid + lo), and its products
// are added part by part in f32: S, u and the outputs are as exact as f32 products would make
// them, at three instructions (six for T or P times an f32 operand, without the terms below
// 2^-24) where f32 matrix instructions would take eight times the cycles.  (P, U and S^T q in
// two parts, 16 bits, spared 3 to 6 % of a call and left nothing of outputs whose terms
// cancel to 2^-17.)
//
// A product with a masked zero would still spread what is not finite to tokens that do not see
// it.  So tokens with such a k, g or b, and elements of v, count as zeros in the products, and
// the results of those that do see them, and the state, become NaN at the end.
#include <cstddef>
#include <type_traits>

#include "kv_layout.h"
#include "mixer_dev.h"

namespace tl {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kChunk = 64;          // tokens of a chunk: a tree's most
static_assert(kChunk == kTreeNodes, "a tree is one chunk");

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// the upper 16 bits of two floats
__device__ __forceinline__ uint32_t upper(float x, float y) {
  return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302);
}
__device__ __forceinline__ float below(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }

// log decay and step of token t and value head h
struct Gate {
  float g, b;
};
__device__ __forceinline__ Gate make_gate(const DeltaArgs &a, float x, float y, float a_log, float dt_bias) {
  if (!a.a_log) return {x, y};
  const float z = x + dt_bias;
  return {-expf(a_log) * (z > 20.0f ? z : log1pf(expf(z))), 1.0f / (1.0f + expf(-y))};
}
__device__ __forceinline__ Gate gate_of(const DeltaArgs &a, const float *pa, const float *pb, int64_t t, int h, int layer) {
  const int64_t at = int64_t(layer) * a.Hv + h;
  return make_gate(a, pa[t * a.lda + h], pb[t * a.ldb + h], a.a_log ? a.a_log[at] : 0.0f, a.a_log ? a.dt_bias[at] : 0.0f);
}

// ---------------------------------------------------------------------------
// Token by token.  256 threads take one request, head and 32 columns; a thread holds 4
// columns of Dk / 32 rows.  S^T k and S^T q of the old state are summed together: the new
// state's S^T q is exp(g) S^T q + (q k) u.  What 16 tokens bring is asked for at once, beside
// the state, and passes through LDS; a token then costs one barrier.  The state's bytes bound it
// (48 heads of 128 x 128: one token of each of 64 requests, 403 MB, 80 us; 4 branches through 48
// layers, 1.25 GB, 245 us, 5.1 TB/s), for few requests the latency (one token 5.4 us, each
// further one 0.8).
constexpr int kStepBatch = 16;

template <int DK>
struct alignas(16) StepShared {
  float k[kStepBatch][DK], q[kStepBatch][DK], v[kStepBatch][32], decay[kStepBatch], step[kStepBatch];
  float sum[2][4][8][12];
};
static_assert(alignof(StepShared<64>) >= 16 && offsetof(StepShared<64>, v) % 16 == 0 && offsetof(StepShared<64>, sum) % 16 == 0 &&
                  alignof(StepShared<128>) >= 16 && offsetof(StepShared<128>, v) % 16 == 0 && offsetof(StepShared<128>, sum) % 16 == 0,
              "read and written 16 bytes at a time");

// the sum over the lanes that differ in bits 3 to 5
__device__ __forceinline__ float sum_rows(float x) {
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xF, 0xF, true));  // row_ror:8
  const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

// tokens: the numbers in the request of the `count` tokens, or NULL for the first ones.  Every
// thread of the workgroup calls it; those that are not `on` only pass the barriers.
template <int DK, bool COMMIT>
__device__ __forceinline__ void step_request(const DeltaArgs &a, const Request &rq, int h, int layer, int col0, int count,
                                             const int *tokens, StepShared<DK> &lds, bool on) {
  constexpr int N = DK / 32, P = DK / 8;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6 & 3;
  const int col = col0 + 4 * (lane & 7), kh = h / a.G;
  const bool live = on && col < a.Dv;
  float *state = a.state + ((int64_t(layer) * a.state_count + rq.row) * a.Hv + h) * DK * a.Dv + col;
  f32x4 S[N];
  if (!rq.fresh && live) {
#pragma unroll
    for (int i = 0; i < N; ++i) S[i] = *reinterpret_cast<const f32x4 *>(state + int64_t(32 * i + 8 * wave + (lane >> 3)) * a.Dv);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) S[i] = f32x4{0, 0, 0, 0};
  }
  const uint16_t *pk = a.k + int64_t(layer) * a.k_layer + kh * DK, *pq = a.q + kh * DK;
  const uint16_t *pv = a.v + int64_t(layer) * a.v_layer + int64_t(h) * a.Dv + col0;
  const float *pa = a.a + int64_t(layer) * a.a_layer, *pb = a.b + int64_t(layer) * a.b_layer;
  for (int i0 = 0; i0 < count; i0 += kStepBatch) {
    const int here = min(kStepBatch, count - i0);
    auto token = [&](int j) { return int64_t(rq.first) + (tokens ? tokens[i0 + j] : i0 + j); };
    if (on) {
      Gate gate = {0.0f, 0.0f};
      if (tid < here) gate = gate_of(a, pa, pb, token(tid), h, layer);
      for (int u = tid; u < here * P * (COMMIT ? 1 : 2); u += kThreads) {
        const int w = u < here * P ? u : u - here * P, j = w / P, d = w % P * 8;
        const int64_t t = token(j);
        const u32x4 x = *reinterpret_cast<const u32x4 *>((u < here * P ? pk + t * a.ldk : pq + t * a.ldq) + d);
        f32x4 *to = reinterpret_cast<f32x4 *>((u < here * P ? lds.k[j] : lds.q[j]) + d);
        to[0] = f32x4{lo_bf16(x[0]), hi_bf16(x[0]), lo_bf16(x[1]), hi_bf16(x[1])};
        to[1] = f32x4{lo_bf16(x[2]), hi_bf16(x[2]), lo_bf16(x[3]), hi_bf16(x[3])};
      }
      const int j = tid >> 2 & (kStepBatch - 1), d = (tid & 3) * 8;
      if (tid >= kThreads - 4 * kStepBatch && j < here && col0 + d < a.Dv) {   // the last wave: the others have the gates and k
        const u32x4 x = *reinterpret_cast<const u32x4 *>(pv + token(j) * a.ldv + d);
        f32x4 *to = reinterpret_cast<f32x4 *>(lds.v[j] + d);
        to[0] = f32x4{lo_bf16(x[0]), hi_bf16(x[0]), lo_bf16(x[1]), hi_bf16(x[1])};
        to[1] = f32x4{lo_bf16(x[2]), hi_bf16(x[2]), lo_bf16(x[3]), hi_bf16(x[3])};
      }
      if (tid < here) {
        lds.decay[tid] = expf(gate.g);
        lds.step[tid] = gate.b;
      }
    }
    __syncthreads();
    for (int i = 0; i < here; ++i) {
      const float decay = lds.decay[i], step = lds.step[i];
      const f32x4 v = *reinterpret_cast<const f32x4 *>(lds.v[i] + 4 * (lane & 7));
      constexpr int SUMS = COMMIT ? 4 : 9;
      float kk[N], sum[12];
#pragma unroll
      for (int e = 0; e < 12; ++e) sum[e] = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int row = 32 * j + 8 * wave + (lane >> 3);
        kk[j] = lds.k[i][row];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = fmaf(S[j][e], kk[j], sum[e]);
        if constexpr (!COMMIT) {
          const float qq = lds.q[i][row];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[4 + e] = fmaf(S[j][e], qq, sum[4 + e]);
          sum[8] = fmaf(kk[j], qq, sum[8]);
        }
      }
#pragma unroll
      for (int e = 0; e < SUMS; ++e) sum[e] = sum_rows(sum[e]);
      auto &sums = lds.sum[i & 1];                       // the token before may still be read
      if (on && lane < 8)
#pragma unroll
        for (int e = 0; e < SUMS; e += 4)
          *reinterpret_cast<f32x4 *>(sums[wave][lane] + e) = f32x4{sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
      __syncthreads();
#pragma unroll
      for (int e = 0; e < SUMS; e += 4) {
        f32x4 x[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) x[w] = *reinterpret_cast<const f32x4 *>(sums[w][lane & 7] + e);
        x[0] = x[0] + x[1] + (x[2] + x[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[e + j] = x[0][j];
      }
      float u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = step * (v[e] - decay * sum[e]);
#pragma unroll
        for (int j = 0; j < N; ++j) S[j][e] = fmaf(kk[j], u[e], decay * S[j][e]);
      }
      if constexpr (!COMMIT) {
        if (tid < 8 && live) {
          float o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = a.scale * fmaf(sum[8], u[e], decay * sum[4 + e]);
          *reinterpret_cast<u32x2 *>(a.out + (token(i) * a.Hv + h) * a.Dv + col) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
        }
      }
    }
  }
  if (live) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<f32x4 *>(state + int64_t(32 * i + 8 * wave + (lane >> 3)) * a.Dv) = S[i];
  }
}

template <int DK, bool COMMIT>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(const DeltaArgs a, int conv_groups) {
  __shared__ StepShared<DK> lds;
  __shared__ int s_token[kTreeNodes];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blocks = (a.Dv + 31) / 32;
  int id = blockIdx.x;
  const bool conv = COMMIT && id >= a.L * a.R * a.Hv * blocks;
  int cb, h = 0;
  if (conv) {
    id -= a.L * a.R * a.Hv * blocks;
    cb = id % conv_groups;
    id /= conv_groups;
  } else {
    cb = id % blocks;
    id /= blocks;
    h = id % a.Hv;
    id /= a.Hv;
  }
  const int r = id % a.R, layer = id / a.R;
  const Request rq = request_of(a.q_start, a.kv_lens, a.slots, a.R, a.T, a.state_count, r);
  if (rq.r < 0 || rq.n <= 0) return;
  const int first = rq.first, n = rq.n;
  if constexpr (COMMIT) {
    if (rq.row < 0 || n > kTreeNodes) return;
    if (wave == 0) {
      const int most = min(a.accepted[r], a.path_width);   // entries, of which those that name a token count
      const int at = lane < most ? a.path[int64_t(r) * a.path_width + lane] : -1;
      const bool on = at >= 0 && at < n;
      const uint64_t all = __ballot(on);
      if (on) s_token[__popcll(all & ((uint64_t(1) << lane) - 1))] = at;
      if (lane == 0) s_count = __popcll(all);
    }
    __syncthreads();
    const int count = s_count;
    if (count == 0) return;
    if (conv) {                                          // the last rows of x along the branch
      const int c = (cb * kThreads + tid) * 8, W = a.taps;
      if (c >= a.C) return;
      uint16_t *st = a.conv_state + (int64_t(layer) * a.state_count + rq.row) * (W - 1) * a.C + c;
      const uint16_t *x = a.x + int64_t(layer) * a.x_layer + int64_t(first) * a.ldx + c;
      u32x4 next[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        next[j] = u32x4{0, 0, 0, 0};
        const int back = count - (W - 1) + j;
        if (j < W - 1) {
          if (back >= 0) next[j] = *reinterpret_cast<const u32x4 *>(x + int64_t(s_token[back]) * a.ldx);
          else if (!rq.fresh) next[j] = *reinterpret_cast<const u32x4 *>(st + int64_t(back + W - 1) * a.C);
        }
      }
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < W - 1) *reinterpret_cast<u32x4 *>(st + int64_t(j) * a.C) = next[j];
      return;
    }
    step_request<DK, true>(a, rq, h, layer, cb * 32, count, s_token, lds, true);
  } else {
    if (rq.row < 0) {
      const int col = cb * 32 + 4 * (lane & 7);
      if (col < a.Dv)
        for (int i = wave * 8 + (lane >> 3); i < n; i += 32)
          *reinterpret_cast<u32x2 *>(a.out + (int64_t(first + i) * a.Hv + h) * a.Dv + col) = u32x2{0, 0};
      return;
    }
    step_request<DK, false>(a, rq, h, 0, cb * 32, n, nullptr, lds, true);
  }
}

// ---------------------------------------------------------------------------
// Chunks.  The workspace holds, for each chunk and value head, T and P as the matrix
// instructions take their first operand, and the decays; for each chunk and key head, K, Q
// and K transposed in the same order.  (The scan's workgroups would else ask for rows that
// lie a token of all heads apart, in halves of lines and mostly in the same few channels of
// an L2: a call for 8191 tokens of 48 heads of 128 x 128 took 25 us longer, of 390.)  A
// 16x16x32 operand is 64 lanes of 16 bytes: lane 16 g + m holds row m, columns 8 g .. 8 g + 7
// of 32.  Its result's lane 16 g + m holds column m, rows 4 g .. 4 g + 3.  Rows
// are dealt to pairs of tiles so that a pair's results are the next product's second operand
// as they stand: row m of tile 2 s + p is token (or element of k)
//   32 s + 8 (m / 4) + 4 p + m % 4,
// and the lane's 4 + 4 values of a pair are the 8 consecutive ones 32 s + 8 g ...
__host__ __device__ constexpr int dealt(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }

constexpr int kTile = 1024;                              // bytes of an operand
// tile i of T or P has its columns of 32 up to s = i / 2: 6 operands for each part
__host__ __device__ constexpr int tri_at(int i, int s) { return (i < 2 ? i : 2 * (i - 1)) + s; }
constexpr int kTriangle = 6;
constexpr int kParts = 3;
// T lies in parts; P in f32, as two halves of a lane's 8 values: what a wave cuts for itself is
// a third less to write and to read
constexpr int kDecays = (kParts + 2) * kTriangle * kTile;  // behind T and P: three lists of 64
constexpr int kHeadBytes = kDecays + 3 * kChunk * 4;      // the third: exp(D_last) and a word of tokens
__host__ __device__ constexpr int key_bytes(int DK) { return 3 * kChunk * DK * 2; }

// the three bf16 parts of 8 floats, as an operand's lane holds them
__device__ __forceinline__ void cut(const float (&x)[8], u32x4 (&o)[kParts]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float p = x[2 * e], q = x[2 * e + 1];
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      o[part][e] = upper(p, q);
      p = below(p);
      q = below(q);
    }
  }
}

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight both(f32x4 x, f32x4 y) { return {{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}}; }
__device__ __forceinline__ void cut(const Eight &x, u32x4 (&o)[kParts]) { cut(x.v, o); }

// The part products of two f32 operands, smallest first: hi lo, mid mid, lo hi, hi mid, mid hi,
// hi hi.  What is below 2^-24 of the largest stays out.
constexpr int kPartProducts = 6, kOfFirst[kPartProducts] = {2, 1, 0, 1, 0, 0}, kOfSecond[kPartProducts] = {0, 1, 2, 0, 1, 0};

// What one lane wrote to LDS is there for the wave's other lanes (which need no barrier: a
// wave's LDS instructions are executed in order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A token's part of a chunk: what it sees, its gate, and D (a power of two's exponent) up to it
// and up to the last token.  Tokens whose gates are not finite are named in `lost` and count
// as ones that do nothing; of tokens past the n there is nothing.
struct Chunk64 {
  double total, end;
  float b;
  uint64_t seen, lost;
};
struct GateRow {
  float a, b, a_log, dt_bias;
  uint64_t seen;
};
__device__ __forceinline__ GateRow ask_gates(const DeltaArgs &a, int64_t t0, int n, int h, int lane, bool tree) {
  const int64_t t = t0 + min(lane, n - 1);
  GateRow x = {a.a[t * a.lda + h], a.b[t * a.ldb + h], 0.0f, 0.0f, ~uint64_t(0)};
  if (tree) x.seen = a.tree_mask[t];
  if (a.a_log) {
    x.a_log = a.a_log[h];
    x.dt_bias = a.dt_bias[h];
  }
  return x;
}
__device__ __forceinline__ Chunk64 sum_gates(const DeltaArgs &a, const GateRow &x, int n, int lane, bool tree) {
  Chunk64 c;
  Gate gate = make_gate(a, x.a, x.b, x.a_log, x.dt_bias);
  if (lane >= n) gate = {0.0f, 0.0f};
  const uint64_t own = uint64_t(1) << lane, upto = own | (own - 1);
  c.seen = lane < n ? (x.seen | own) & upto : 0;
  // exp of less is 0 either way, and sums of finite numbers can be subtracted
  if (gate.g < -1.0e4f) gate.g = -1.0e4f;
  const bool lost = !__builtin_isfinite(gate.g) || !__builtin_isfinite(gate.b);
  if (lost) gate = {0.0f, 0.0f};
  c.lost = __ballot(lost);
  c.b = gate.b;
  c.total = double(gate.g) * 1.4426950408889634;
  if (!tree) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double before = __shfl_up(c.total, off, 64);
      if (lane >= off) c.total += before;
    }
  } else {
    const uint64_t mine = __builtin_bit_cast(uint64_t, c.total);
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    for (int j0 = 0; j0 < n; j0 += 16) {                 // without branches, so that tokens overlap
      const int bits = int(uint32_t(c.seen >> j0));
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int on = bits << (31 - j) >> 31;
        const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(mine), j0 + j) & on;
        const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(mine >> 32), j0 + j) & on;
        sum[j & 3] += __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
      }
    }
    c.total = sum[0] + sum[1] + (sum[2] + sum[3]);
  }
  c.end = __shfl(c.total, n - 1, 64);
  return c;
}

// 8 values of k_i k_j and q_i k_j, j = j0 .., become those of A and P
__device__ __forceinline__ void weigh(float (&kk)[8], float (&qk)[8], int i, int j0, uint64_t seen, float step, double total,
                                      const double *totals) {
  const uint32_t bits = uint32_t(seen >> j0);            // i's own bit is its highest
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float decay = __builtin_amdgcn_exp2f(float(total - totals[j0 + e]));
    const bool on = bits >> e & 1;
    kk[e] = on && j0 + e < i ? step * decay * kk[e] : 0.0f;
    qk[e] = on ? decay * qk[e] : 0.0f;
  }
}

// Column m of (I + D)^-1 for a strictly lower block D of 16 rows
template <int PITCH>
__device__ __forceinline__ void solve_block(const float *D, int m, float (&t)[16]) {
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    f32x4 d[4];
#pragma unroll
    for (int y = 0; y < x; y += 4) d[y / 4] = *reinterpret_cast<const f32x4 *>(D + x * PITCH + y);
    float sum = x == m ? 1.0f : 0.0f;
#pragma unroll
    for (int y = 0; y < x; ++y) sum = fmaf(-d[y / 4][y & 3], t[y], sum);
    t[x] = sum;
    if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // four rows' reads at a time: registers
  }
}

// 8 values of T's row i, columns j0 .., with the steps, in parts
template <int PITCH>
__device__ __forceinline__ void solver_row(const float *A, const float *steps, int i, int j0, u32x4 (&o)[kParts]) {
  const f32x4 *row = reinterpret_cast<const f32x4 *>(A + i * PITCH + j0), *b = reinterpret_cast<const f32x4 *>(steps + j0);
  const f32x4 u[2] = {row[0], row[1]}, v[2] = {b[0], b[1]};
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = j0 + e <= i ? u[e >> 2][e & 3] * v[e >> 2][e & 3] : 0.0f;
  cut(x, o);
}

// An operand of K transposed, 32 tokens of elements dealt(p, m) of 32, from the tokens' two row
// tiles: times one-hot columns, which pick that element of every token.
__device__ __forceinline__ u32x4 transposed(u32x4 lower, u32x4 higher, int p, int m, int g) {
  u32x4 pick;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = dealt(p, m) - 8 * g - 2 * e;
    pick[e] = d == 0 ? 0x3F80u : d == 1 ? 0x3F800000u : 0u;
  }
  const f32x4 zero = {0, 0, 0, 0};
  const f32x4 x = mfma(lower, pick, zero), y = mfma(higher, pick, zero);
  return u32x4{upper(x[0], x[1]), upper(x[2], x[3]), upper(y[0], y[1]), upper(y[2], y[3])};
}

// One wave makes T and P of one chunk and value head, and for the first and last head of a key
// head K's and Q's operands; four heads share a workgroup, and waves never wait for each other.
// What it writes bounds it: 294 MB for 8191 tokens of 48 heads of 128 x 128 in 77 us.  All of K
// stays in registers as operands.  A lies in LDS; its diagonal blocks of 16 are solved column
// by column, a lane each (T_ii = (I + A_ii)^-1), and the blocks below follow by
// T_ij = -T_ii sum over k of A_ik T_kj on the f32 matrix instruction, whose steps take rows
// 4 g + c in the order in which results lie, so T's blocks are operands as they stand.
template <int DK>
__global__ __launch_bounds__(kThreads, 2) void delta_prep_kernel(const DeltaArgs a) {
  constexpr int NS = DK / 32, PITCH = kChunk + 4, WAVES = kThreads / 64;
  __shared__ __attribute__((aligned(16))) float s_A[WAVES][kChunk * PITCH];
  __shared__ double s_total[WAVES][kChunk];
  __shared__ __attribute__((aligned(16))) float s_b[WAVES][kChunk];
  __shared__ uint64_t s_seen[WAVES][kChunk];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
  const int number = blockIdx.x, h = int(blockIdx.y) * WAVES + wave, kh = h / a.G;
  int part;
  const Request rq = find_piece<kChunk>(a.q_start, a.kv_lens, a.slots, a.R, a.T, a.state_count, number, part);
  if (h >= a.Hv || rq.r < 0 || rq.row < 0) return;
  const int64_t t0 = int64_t(rq.first) + part * kChunk;
  const int n = min(kChunk, rq.n - part * kChunk);
  const bool tree = a.tree_mask && rq.n <= kTreeNodes;
  char *head = a.heads + (int64_t(number) * a.Hv + h) * kHeadBytes;
  float *A = s_A[wave];

  // Everything is asked for at once, the gates first.
  const GateRow row = ask_gates(a, t0, n, h, lane, tree);
  // rows of K and Q as operands: tile t's row m is token dealt(t, m); past the last one it is the last
  u32x4 k[4][NS], q[4][NS];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t i = t0 + min(dealt(t, m), n - 1);
    const uint16_t *pk = a.k + i * a.ldk + kh * DK + 8 * g, *pq = a.q + i * a.ldq + kh * DK + 8 * g;
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      k[t][c] = *reinterpret_cast<const u32x4 *>(pk + 32 * c);
      q[t][c] = *reinterpret_cast<const u32x4 *>(pq + 32 * c);
    }
  }
  const Chunk64 mine = sum_gates(a, row, n, lane, tree);
  uint64_t bad = mine.lost;                              // tokens whose k, g or b is not finite
  s_total[wave][lane] = mine.total;
  s_b[wave][lane] = mine.b;
  s_seen[wave][lane] = mine.seen;
#pragma unroll
  for (int t = 0; t < 4; ++t) {                          // an exponent of all ones is what is not finite
    u16x2 top = {0, 0};
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, k[t][c][e] & 0x7FFF7FFFu));
    uint64_t all = __ballot(top[0] >= 0x7F80u || top[1] >= 0x7F80u);
    if (all == 0) continue;
    all |= all >> 32;
    all |= all >> 16;
    for (int j = 0; j < 16; ++j) bad |= (all >> j & 1) << dealt(t, j);
    if (all >> m & 1)
#pragma unroll
      for (int c = 0; c < NS; ++c) k[t][c] = u32x4{0, 0, 0, 0};
  }
  {
    float *to = reinterpret_cast<float *>(head + kDecays);
    to[lane] = lane < n ? __builtin_amdgcn_exp2f(float(mine.total)) : 0.0f;
    to[kChunk + lane] = lane < n ? __builtin_amdgcn_exp2f(float(mine.end - mine.total)) : 0.0f;
    if (lane == 0) *reinterpret_cast<f32x4 *>(to + 2 * kChunk) =
        f32x4{__builtin_amdgcn_exp2f(float(mine.end)), 0.0f, __uint_as_float(uint32_t(bad)), __uint_as_float(uint32_t(bad >> 32))};
  }
  const int share = h % a.G;                             // the key head's operands, by its first and last value head
  u32x4 *keys = reinterpret_cast<u32x4 *>(a.keys + (int64_t(number) * a.Hk + kh) * key_bytes(DK)) + lane;
  if (share == 0) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int c = 0; c < NS; ++c) keys[(t * NS + c) * 64] = k[t][c];
    if (!tree)
#pragma unroll
      for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          keys[(8 * NS + t * 2 + s) * 64] = transposed(k[2 * s][t >> 1], k[2 * s + 1][t >> 1], t & 1, m, g);
  }
  if (share == a.G - 1)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int c = 0; c < NS; ++c) keys[((4 + t) * NS + c) * 64] = q[t][c];
  wave_sync();

  // (K K^T)^T and (Q K^T)^T: a lane holds token i = dealt(t, m) against 8 consecutive j's
  f32x4 *P = reinterpret_cast<f32x4 *>(head + kParts * kTriangle * kTile);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (32 * (t >> 1) >= n) break;                       // uniform
    const int i = dealt(t, m);
    const double upto_i = s_total[wave][i];
    const float step = s_b[wave][i];
    const uint64_t sees = s_seen[wave][i];
#pragma unroll
    for (int s = 0; s <= t >> 1; ++s) {
      float kk[8], qk[8];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          x = mfma(k[2 * s + p][c], k[t][c], x);
          y = mfma(k[2 * s + p][c], q[t][c], y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk[4 * p + e] = x[e];
          qk[4 * p + e] = y[e];
        }
      }
      weigh(kk, qk, i, 32 * s + 8 * g, sees, step, upto_i, s_total[wave]);
      f32x4 *to = reinterpret_cast<f32x4 *>(A + i * PITCH + 32 * s + 8 * g);
      to[0] = f32x4{kk[0], kk[1], kk[2], kk[3]};
      to[1] = f32x4{kk[4], kk[5], kk[6], kk[7]};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        P[(e * kTriangle + tri_at(t, s)) * 64 + lane] = f32x4{qk[4 * e], qk[4 * e + 1], qk[4 * e + 2], qk[4 * e + 3]};
    }
  }
  wave_sync();

  // T's diagonal blocks: lane 16 b + c solves column c of block b, row by row.  Tokens past the
  // last one are rows of A that nobody wrote where 32 of them are missing: their blocks stay out.
  const int tiles = n > 32 ? 4 : 2;
  if (g < tiles) {
    const float *D = A + 16 * g * PITCH + 16 * g;
    float t[16];
    solve_block<PITCH>(D, m, t);
    float *to = A + 16 * g * PITCH + 16 * g + m;
#pragma unroll
    for (int x = 0; x < 16; ++x) to[x * PITCH] = t[x];
  }
  wave_sync();
  f32x4 T[4][4];                                         // T[i][j][c]: row 16 i + 4 g + c, column 16 j + m
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) T[i][i][c] = i < tiles ? A[(16 * i + 4 * g + c) * PITCH + 16 * i + m] : 0.0f;
#pragma unroll
  for (int off = 1; off < 4; ++off) {
    if (off == 2 && tiles == 2) break;                   // uniform
#pragma unroll
    for (int i = off; i < 4; ++i) {
      if (i >= tiles) break;
      const int j = i - off;
      f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
      for (int b = j; b < i; ++b) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(A + (16 * i + m) * PITCH + 16 * b + 4 * g);
#pragma unroll
        for (int c = 0; c < 4; ++c) x = __builtin_amdgcn_mfma_f32_16x16x4f32(w[c], T[b][j][c], x, 0, 0, 0);
      }
      const f32x4 w = *reinterpret_cast<const f32x4 *>(A + (16 * i + m) * PITCH + 16 * i + 4 * g);
#pragma unroll
      for (int c = 0; c < 4; ++c) y = __builtin_amdgcn_mfma_f32_16x16x4f32(w[c], x[c], y, 0, 0, 0);
      T[i][j] = -y;
    }
  }
  wave_sync();
#pragma unroll
  for (int i = 1; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < i; ++j)
      if (i < tiles)
#pragma unroll
        for (int c = 0; c < 4; ++c) A[(16 * i + 4 * g + c) * PITCH + 16 * j + m] = T[i][j][c];
  wave_sync();
  u32x4 *to = reinterpret_cast<u32x4 *>(head);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (32 * (t >> 1) >= n) break;
    const int i = dealt(t, m);
#pragma unroll
    for (int s = 0; s <= t >> 1; ++s) {
      u32x4 part[kParts];
      solver_row<PITCH>(A, s_b[wave], i, 32 * s + 8 * g, part);
#pragma unroll
      for (int e = 0; e < kParts; ++e) to[(e * kTriangle + tri_at(t, s)) * 64 + lane] = part[e];
    }
  }
}

// A workgroup walks the chunks of one request, head and 32 columns.  Wave w of the first
// four takes row tile w of the chunk's tokens and of the state the tiles TP w .. (a pair for Dk
// 128, one for Dk 64), and goes the chain from one chunk's state to the next one's: K S, U, K^T U.
// Wave 4 + w makes the results of row tile w beside it.  The chain's latency bounds it: 8191
// tokens of 48 heads of 128 x 128 take 305 us, about 5100 cycles a chunk; its matrix
// instructions take 1728 of them a SIMD, its 312 LDS reads of 1 KB 2500 at 128 bytes a cycle, and
// its global loads some 700.  Requests of very different lengths wait for a place instead: a
// workgroup needs 8 waves of 182 registers or more, and a compute unit holds one.  Column m of
// tile c is column 2 m + c: a lane's columns are neighbours.
constexpr int kScanThreads = 512;

template <int DK>
__global__ __launch_bounds__(kScanThreads, 1) void delta_scan_kernel(const DeltaArgs a) {
  constexpr int NS = DK / 32, CT = 2, TP = DK / 64;      // column tiles of the workgroup, state tiles of a wave
  static_assert(TP == 1 || TP == 2, "a wave holds a pair of state tiles, or one of a pair");
  __shared__ __attribute__((aligned(16))) u32x4 s_S[3][CT][NS][64], s_R[3][CT][2][64], s_U[3][CT][2][64], s_W[3][CT][2][64];
  __shared__ uint32_t s_bad[16 * CT][2];                 // of each column: tokens whose v is not finite
  __shared__ int s_some;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int all_waves = __builtin_amdgcn_readfirstlane(tid >> 6), wave = all_waves & 3;  // uniform: barriers follow
  const int blocks = (a.Dv + 16 * CT - 1) / (16 * CT);
  // Workgroups go to the 8 L2s in turn: those of one key head, which read the same K, Q, T and P,
  // are 8 numbers apart.
  const int of_key = a.G * blocks, j = int(blockIdx.x) >> 3, key = j / of_key * 8 + (int(blockIdx.x) & 7);
  if (key >= a.R * a.Hk) return;
  const int r = key / a.Hk, kh = key - r * a.Hk, h = kh * a.G + j % of_key / blocks, cb = j % blocks;
  // a chain's state is NaN from such a token on, so the words need no clearing for later chunks
  if (tid < 32 * CT) s_bad[tid >> 1][tid & 1] = 0;
  if (tid == 0) s_some = 0;
  __syncthreads();
  const Request rq = request_of(a.q_start, a.kv_lens, a.slots, a.R, a.T, a.state_count, r);
  if (rq.r < 0 || rq.n <= 0) return;
  const int first = rq.first, n = rq.n, srow = rq.row;
  // Past the last column a lane repeats the work of another one, value for value.
  const int own_col = 16 * CT * cb + CT * m, col = own_col < a.Dv ? own_col : own_col - 16;
  auto store = [&](int64_t t, const float *o) {
    uint16_t *to = a.out + (t * a.Hv + h) * a.Dv + col;
    *reinterpret_cast<uint32_t *>(to) = pack_bf16(o[0], o[1]);
  };
  if (srow < 0) {
    const float zero[2] = {0.0f, 0.0f};
    for (int i = 4 * all_waves + g; i < n; i += 32) store(int64_t(first) + i, zero);
    return;
  }
  const bool tree = a.tree_mask && n <= kTreeNodes, fresh = rq.fresh;
  const int64_t number = int64_t(first) / kChunk + r;
  const int row0 = 32 * (wave >> 1) + 8 * g + 4 * (wave & 1), pairs = (wave >> 1) + 1;
  const int last = (n - 1) / kChunk;
  auto head_of = [&](int part) { return a.heads + ((number + part) * a.Hv + h) * kHeadBytes; };
  auto key_of = [&](int part) { return reinterpret_cast<const u32x4 *>(a.keys + ((number + part) * a.Hk + kh) * key_bytes(DK)) + lane; };
  // tokens that a column's results, and the state after them, must not have seen
  auto not_finite = [&](uint64_t bad, uint64_t (&gone)[CT]) {
#pragma unroll
    for (int c = 0; c < CT; ++c) gone[c] = bad | s_bad[CT * m + c][0] | uint64_t(s_bad[CT * m + c][1]) << 32;
  };
  auto word_of = [](const f32x4 &end) { return __float_as_uint(end[2]) | uint64_t(__float_as_uint(end[3])) << 32; };

  if (all_waves >= 4) {                                  // out = scale (exp(D) Q S + P U)
    u32x4 Q[NS];
    f32x4 P[2][2];
    f32x4 grown, end;
    auto fetch_row = [&](int part) {
      const u32x4 *from = key_of(part) + (4 + wave) * NS * 64;
#pragma unroll
      for (int s = 0; s < NS; ++s) Q[s] = from[s * 64];
      grown = *reinterpret_cast<const f32x4 *>(head_of(part) + kDecays + row0 * 4);
      end = *reinterpret_cast<const f32x4 *>(head_of(part) + kDecays + 2 * kChunk * 4);
    };
    auto fetch_weights = [&](int part) {
      const f32x4 *from = reinterpret_cast<const f32x4 *>(head_of(part)) + (kParts * kTriangle + tri_at(wave, 0)) * 64 + lane;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) P[s][e] = from[(e * kTriangle + (s < pairs ? s : 0)) * 64];
    };
    fetch_row(0);
    fetch_weights(0);
    auto chunk = [&](int part, auto whole) {
      constexpr bool more = decltype(whole)::value;
      const int64_t t0 = int64_t(first) + part * kChunk;
      const int here = more ? kChunk : n - part * kChunk;
      const bool rows = more || 32 * (wave >> 1) < here;
      const uint64_t bad = word_of(end);
      f32x4 o[CT];
      __syncthreads();
      if (rows) {
        u32x4 y[NS][CT][kParts];
#pragma unroll
        for (int c = 0; c < CT; ++c) o[c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int e = kParts - 1; e >= 0; --e)
#pragma unroll
            for (int c = 0; c < CT; ++c) y[s][c][e] = s_S[e][c][s][lane];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int e = kParts - 1; e >= 0; --e)
#pragma unroll
            for (int c = 0; c < CT; ++c) o[c] = mfma(Q[s], y[s][c][e], o[c]);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][e] *= grown[e];
      }
      __syncthreads();
      if constexpr (more) fetch_row(part + 1);
      __syncthreads();
      if (rows) {
        auto add = [&](auto two) {
          constexpr int N = decltype(two)::value ? 2 : 1;
#pragma unroll
          for (int s = 0; s < N; ++s) {
            u32x4 w[kParts], x[CT][kParts];
            cut(both(P[s][0], P[s][1]), w);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int e = 0; e < kParts; ++e) x[c][e] = s_U[e][c][s][lane];
#pragma unroll
            for (int j = 0; j < kPartProducts; ++j)
#pragma unroll
              for (int c = 0; c < CT; ++c) o[c] = mfma(w[kOfFirst[j]], x[c][kOfSecond[j]], o[c]);
          }
        };
        if (pairs == 2) add(std::true_type());
        else add(std::false_type());
#pragma unroll
        for (int c = 0; c < CT; ++c) o[c] *= a.scale;
        if (s_some || bad) {
          uint64_t gone[CT];
          not_finite(bad, gone);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = row0 + e;
            const uint64_t own = uint64_t(1) << j, upto = own | (own - 1);
            const uint64_t seen = tree ? ((j < here ? a.tree_mask[t0 + j] : 0) | own) & upto : upto;
#pragma unroll
            for (int c = 0; c < CT; ++c)
              if (seen & gone[c]) o[c][e] = __builtin_nanf("");
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x[2] = {o[0][e], o[1][e]};
          if (more || row0 + e < here) store(t0 + row0 + e, x);
        }
      }
      if constexpr (more) fetch_weights(part + 1);
    };
    for (int part = 0; part < last; ++part) chunk(part, std::true_type());
    chunk(last, std::false_type());
    return;
  }

  const int state_row = TP == 2 ? 32 * wave + 8 * g : 32 * (wave >> 1) + 8 * g + 4 * (wave & 1);
  float *state = a.state + ((int64_t(srow) * a.Hv + h) * DK + state_row) * a.Dv + col;
  f32x4 S[TP][CT];                                       // [p][c][e]: row state_row + 4 p + e
  if (!fresh) {
#pragma unroll
    for (int p = 0; p < TP; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[p][c][e] = state[int64_t(4 * p + e) * a.Dv + c];
  } else {
#pragma unroll
    for (int p = 0; p < TP; ++p)
#pragma unroll
      for (int c = 0; c < CT; ++c) S[p][c] = f32x4{0, 0, 0, 0};
  }

  // What a wave takes of a chunk.  Each piece is asked for as soon as the chunk before has used
  // it.  Rows past the last token are the last one's: nothing of theirs is kept.
  u32x4 K[NS], T[2][kParts], keys[TP][2];
  uint32_t V[4];                                         // two columns of a row
  f32x4 grown, left, end;                                // end: exp(D_last), nothing, a word of tokens
  const int vcol = h * a.Dv + col;
  const uint16_t *to_v[4];                               // this lane's rows of the chunk that is asked for next
  auto rows_of = [&](int part) {
    const int most = min(kChunk, n - part * kChunk) - 1;
    const int64_t t0 = int64_t(first) + part * kChunk;
#pragma unroll
    for (int e = 0; e < 4; ++e) to_v[e] = a.v + (t0 + min(row0 + e, most)) * a.ldv + vcol;
  };
  auto fetch_rows = [&](int part) {
    const u32x4 *from = key_of(part) + wave * NS * 64;
#pragma unroll
    for (int s = 0; s < NS; ++s) K[s] = from[s * 64];
#pragma unroll
    for (int e = 0; e < 4; ++e) V[e] = *reinterpret_cast<const uint32_t *>(to_v[e]);
    grown = *reinterpret_cast<const f32x4 *>(head_of(part) + kDecays + row0 * 4);
    end = *reinterpret_cast<const f32x4 *>(head_of(part) + kDecays + 2 * kChunk * 4);
  };
  // waves with one pair of columns bring it twice, so that all have asked for as much
  auto fetch_solver = [&](int part) {
    const u32x4 *from = reinterpret_cast<const u32x4 *>(head_of(part)) + tri_at(wave, 0) * 64 + lane;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < kParts; ++e) T[s][e] = from[(e * kTriangle + (s < pairs ? s : 0)) * 64];
    left = *reinterpret_cast<const f32x4 *>(head_of(part) + kDecays + (kChunk + row0) * 4);
  };
  auto fetch_keys = [&](int part) {
    const u32x4 *kt = key_of(part) + 8 * NS * 64;
#pragma unroll
    for (int p = 0; p < TP; ++p)
#pragma unroll
      for (int s = 0; s < 2; ++s) keys[p][s] = kt[((TP * wave + p) * 2 + s) * 64];
  };
  auto share_state = [&] {                               // S in parts, as the second operand
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if constexpr (TP == 2) {
        u32x4 o[3];
        cut(both(S[0][c], S[TP - 1][c]), o);
#pragma unroll
        for (int e = 0; e < 3; ++e) s_S[e][c][wave][lane] = o[e];
      } else {
        float x[4] = {S[0][c][0], S[0][c][1], S[0][c][2], S[0][c][3]};
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const u32x2 w = {upper(x[0], x[1]), upper(x[2], x[3])};
          reinterpret_cast<u32x2 *>(&s_S[e][c][wave >> 1][lane])[wave & 1] = w;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = below(x[j]);
        }
      }
    }
  };
  rows_of(0);
  fetch_rows(0);
  fetch_solver(0);
  share_state();
  // One chunk.  Those before the last are whole and ask for the next one's operands, without
  // branches around the loads: only then can each wait count what was asked for after it.
  auto chunk = [&](int part, auto whole) {
    constexpr bool more = decltype(whole)::value;
    const int here = more ? kChunk : n - part * kChunk;
    const bool rows = more || 32 * (wave >> 1) < here;   // this wave has tokens
    const float decay = end[0];
    const uint64_t bad = word_of(end);
    __syncthreads();
    if (rows) {
      f32x4 ks[CT];
      u32x4 y[NS][CT][3];
#pragma unroll
      for (int c = 0; c < CT; ++c) ks[c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 2; e >= 0; --e)
#pragma unroll
          for (int c = 0; c < CT; ++c) y[s][c][e] = s_S[e][c][s][lane];
      __builtin_amdgcn_sched_barrier(0);                 // every read on its way before the first product
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 2; e >= 0; --e)
#pragma unroll
          for (int c = 0; c < CT; ++c) ks[c] = mfma(K[s], y[s][c][e], ks[c]);
      // R = V - exp(D) K S
      float x[CT][4], sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const float v = c ? hi_bf16(V[e]) : lo_bf16(V[e]);
          sum += v;
          x[c][e] = fmaf(-grown[e], ks[c][e], v);
        }
      const uint64_t none = bad | (here < kChunk ? ~uint64_t(0) << (here & 63) : 0);
      if (none || __any(!__builtin_isfinite(sum))) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const bool off = none >> (row0 + e) & 1;
            if (!off && !__builtin_isfinite(c ? hi_bf16(V[e]) : lo_bf16(V[e]))) {
              atomicOr(&s_bad[CT * m + c][(row0 + e) >> 5], 1u << ((row0 + e) & 31));
              s_some = 1;
              x[c][e] = 0.0f;
            }
            if (off) x[c][e] = 0.0f;
          }
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const u32x2 w = {upper(x[c][0], x[c][1]), upper(x[c][2], x[c][3])};
          reinterpret_cast<u32x2 *>(&s_R[e][c][wave >> 1][lane])[wave & 1] = w;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[c][j] = below(x[c][j]);
        }
      }
    }
    if (more || !tree) fetch_keys(part);
    if constexpr (more) {
      if (n - part * kChunk >= 2 * kChunk) {             // the next chunk is whole
#pragma unroll
        for (int e = 0; e < 4; ++e) to_v[e] += kChunk * a.ldv;
      } else {
        rows_of(part + 1);
      }
      fetch_rows(part + 1);
    }
    __syncthreads();
    const bool some = s_some || bad;
    if (rows) {                                          // U = T R
      f32x4 u[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) u[c] = f32x4{0, 0, 0, 0};
      auto solve = [&](auto two) {
        constexpr int N = decltype(two)::value ? 2 : 1;
        u32x4 x[N][CT][3];
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
          for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int c = 0; c < CT; ++c) x[s][c][e] = s_R[e][c][s][lane];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kPartProducts; ++j)
#pragma unroll
          for (int s = 0; s < N; ++s)
#pragma unroll
            for (int c = 0; c < CT; ++c) u[c] = mfma(T[s][kOfFirst[j]], x[s][c][kOfSecond[j]], u[c]);
      };
      if (pairs == 2) solve(std::true_type());
      else solve(std::false_type());
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = u[c][e];
          y[e] = left[e] * u[c][e];
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const u32x2 z = {upper(y[0], y[1]), upper(y[2], y[3])};
          reinterpret_cast<u32x2 *>(&s_W[e][c][wave >> 1][lane])[wave & 1] = z;
          const u32x2 w = {upper(x[0], x[1]), upper(x[2], x[3])};
          reinterpret_cast<u32x2 *>(&s_U[e][c][wave >> 1][lane])[wave & 1] = w;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = below(x[j]);
            y[j] = below(y[j]);
          }
        }
      }
    }
    __syncthreads();
    if (!tree) {                                         // S = exp(D_last) S + K^T (exp(D_last - D) U)
      auto advance = [&](auto two) {
        constexpr int N = decltype(two)::value ? 2 : 1;
        u32x4 x[N][CT][3];
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
          for (int e = 2; e >= 0; --e)
#pragma unroll
            for (int c = 0; c < CT; ++c) x[s][c][e] = s_W[e][c][s][lane];
#pragma unroll
        for (int p = 0; p < TP; ++p)
#pragma unroll
          for (int c = 0; c < CT; ++c) S[p][c] *= decay;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
          for (int e = 2; e >= 0; --e)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int p = 0; p < TP; ++p) S[p][c] = mfma(keys[p][s], x[s][c][e], S[p][c]);
      };
      if (here > 32) advance(std::true_type());
      else advance(std::false_type());
      if (some) {
        uint64_t gone[CT];
        not_finite(bad, gone);
#pragma unroll
        for (int p = 0; p < TP; ++p)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            if (gone[c]) S[p][c] = S[p][c] + __builtin_nanf("");
      }
    }
    if constexpr (more) share_state();
    if constexpr (more) fetch_solver(part + 1);
  };
  for (int part = 0; part < last; ++part) chunk(part, std::true_type());
  chunk(last, std::false_type());
  if (!tree) {
#pragma unroll
    for (int p = 0; p < TP; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < CT; ++c) state[int64_t(4 * p + e) * a.Dv + c] = S[p][c][e];
  }
}

// Drafted trees, and chains of one chunk: a workgroup takes one request, value head and 128
// columns, makes T and P in LDS and uses them there, in one launch; a wave has 16 columns for
// all tokens, so K S, R and U stay in its registers from product to product.  A longer request
// of the call, a chain, goes token by token, its four blocks of 32 columns one after another
// (3.6 us a token).  Latency bounds it: a tree of 64 takes 15.8 us, ten steps behind barriers of
// 1000 to 3000 cycles each and the gates' sums, which one wave makes while seven wait; 16 of up to
// 64, with 48 heads, 35 us in one and a half rounds of two workgroups a compute unit, 69 MB.
constexpr int kFusedThreads = 512;

template <int DK, bool TREE>
__global__ __launch_bounds__(kFusedThreads, 4) void delta_chunk_kernel(const DeltaArgs a) {
  constexpr int NS = DK / 32, PITCH = kChunk + 4;
  struct Operands {
    u32x4 K[4][NS][64], QT[kParts * kTriangle * 64];    // K's; Q's, then T's
  };
  __shared__ Operands lds;
  auto &s_K = lds.K;
  auto &s_QT = lds.QT;
  __shared__ __attribute__((aligned(16))) float s_A[kChunk * PITCH];  // A, then T
  __shared__ u32x4 s_P[kParts * kTriangle * 64];
  __shared__ f32x4 s_T[kTriangle][64];                   // T's blocks below the diagonal, as results lie
  __shared__ double s_total[kChunk];
  __shared__ __attribute__((aligned(16))) float s_b[kChunk], s_grown[kChunk], s_left[kChunk];
  __shared__ uint64_t s_seen[kChunk], s_bad[5];
  static_assert(sizeof(lds.QT) >= sizeof(lds.K) && sizeof(lds) >= sizeof(StepShared<DK>), "Q fits where T is");
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blocks = (a.Dv + 127) / 128;
  int id = blockIdx.x;
  const int cb = id % blocks;
  id /= blocks;
  const int h = id % a.Hv, kh = h / a.G;
  const Request rq = request_of(a.q_start, a.kv_lens, a.slots, a.R, a.T, a.state_count, id / a.Hv);
  if (rq.r < 0 || rq.n <= 0) return;
  const int col0 = 128 * cb + 16 * wave, col = col0 < a.Dv ? col0 + m : m;
  const bool cols = col0 < a.Dv;                         // uniform
  uint16_t *out = a.out + (int64_t(rq.first) * a.Hv + h) * a.Dv + col;
  if (rq.row < 0) {
    if (cols)
      for (int i = g; i < rq.n; i += 4) out[i * int64_t(a.Hv) * a.Dv] = 0;
    return;
  }
  if (rq.n > kTreeNodes) {
    StepShared<DK> &step = reinterpret_cast<StepShared<DK> &>(lds);
    for (int c = 0; c < 128 && 128 * cb + c < a.Dv; c += 32)
      step_request<DK, false>(a, rq, h, 0, 128 * cb + c, rq.n, nullptr, step, tid < kThreads);
    return;
  }
  float *state = a.state + ((int64_t(rq.row) * a.Hv + h) * DK + 8 * g) * a.Dv + col;
  const int64_t t0 = rq.first;
  const int n = rq.n;
  const bool wide = n > 32;                              // else the tokens of tiles 2 and 3 are not there
  // K (four waves) and Q (the others) of row tile `rt`; past the last token it is the last one.
  const int rt = wave & 3;
  const bool stage = 32 * (rt >> 1) < n;
  GateRow gates;
  if (wave == 7) gates = ask_gates(a, t0, n, h, lane, TREE);
  u32x4 k[NS];
  if (stage) {
    const int64_t i = t0 + min(dealt(rt, m), n - 1);
    const uint16_t *from = (wave < 4 ? a.k + i * a.ldk : a.q + i * a.ldq) + kh * DK + 8 * g;
#pragma unroll
    for (int c = 0; c < NS; ++c) k[c] = *reinterpret_cast<const u32x4 *>(from + 32 * c);
  }
  if (wave == 7) {
    const Chunk64 x = sum_gates(a, gates, n, lane, TREE);
    s_total[lane] = x.total;
    s_b[lane] = x.b;
    s_seen[lane] = x.seen;
    s_grown[lane] = lane < n ? __builtin_amdgcn_exp2f(float(x.total)) : 0.0f;
    if (!TREE) s_left[lane] = lane < n ? __builtin_amdgcn_exp2f(float(x.end - x.total)) : 0.0f;
    if (lane == 0) s_bad[4] = x.lost;
  }
  if (stage) {
    if (wave < 4) {
      u16x2 top = {0, 0};                              // an exponent of all ones is what is not finite
#pragma unroll
      for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, k[c][e] & 0x7FFF7FFFu));
      uint64_t all = __ballot(top[0] >= 0x7F80u || top[1] >= 0x7F80u), bad = 0;
      if (all) {
        all |= all >> 32;
        all |= all >> 16;
        for (int j = 0; j < 16; ++j) bad |= (all >> j & 1) << dealt(rt, j);
        if (all >> m & 1)
#pragma unroll
          for (int c = 0; c < NS; ++c) k[c] = u32x4{0, 0, 0, 0};
      }
      if (lane == 0) s_bad[wave] = bad;
    }
    u32x4 *to = wave < 4 ? &s_K[rt][0][lane] : &s_QT[rt * NS * 64 + lane];
#pragma unroll
    for (int c = 0; c < NS; ++c) to[c * 64] = k[c];
  } else if (wave < 4 && lane == 0) {
    s_bad[wave] = 0;
  }
  __syncthreads();
  // The state comes while T is made: asked for beside K and Q it held them up (16 trees of up
  // to 64, 48 heads of 128 x 128: 1.7 us longer, of 35).
  f32x4 S[2 * NS];                                       // tile t, e: row 32 (t / 2) + 8 g + 4 (t % 2) + e
  if (cols && !rq.fresh) {
#pragma unroll
    for (int t = 0; t < 2 * NS; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = state[int64_t(32 * (t >> 1) + 4 * (t & 1) + e) * a.Dv];
  } else {
#pragma unroll
    for (int t = 0; t < 2 * NS; ++t) S[t] = f32x4{0, 0, 0, 0};
  }
  const uint64_t bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3] | s_bad[4];

  // A and P of row tile `wave`
  if (wave < 4 && 32 * (wave >> 1) < n) {
    u32x4 k[NS], q[NS];
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      k[c] = s_K[wave][c][lane];
      q[c] = s_QT[(wave * NS + c) * 64 + lane];
    }
    const int i = dealt(wave, m);
    for (int s = 0; s <= wave >> 1; ++s) {
      float kk[8], qk[8];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          const u32x4 kj = s_K[2 * s + p][c][lane];
          x = mfma(kj, k[c], x);
          y = mfma(kj, q[c], y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk[4 * p + e] = x[e];
          qk[4 * p + e] = y[e];
        }
      }
      weigh(kk, qk, i, 32 * s + 8 * g, s_seen[i], s_b[i], s_total[i], s_total);
      f32x4 *to = reinterpret_cast<f32x4 *>(s_A + i * PITCH + 32 * s + 8 * g);
      to[0] = f32x4{kk[0], kk[1], kk[2], kk[3]};
      to[1] = f32x4{kk[4], kk[5], kk[6], kk[7]};
      u32x4 x[kParts];
      cut(qk, x);
#pragma unroll
      for (int e = 0; e < kParts; ++e) s_P[(e * kTriangle + tri_at(wave, s)) * 64 + lane] = x[e];
    }
  }
  __syncthreads();

  // T: the diagonal blocks, a wave each, then those below, a diagonal after the other
  const int tiles = wide ? 4 : 2;
  if (wave < tiles) {
    float t[16];
    const float *D = s_A + 16 * wave * PITCH + 16 * wave;
    solve_block<PITCH>(D, m, t);
    wave_sync();
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (x >> 2 == g) s_A[(16 * wave + x) * PITCH + 16 * wave + m] = t[x];
  }
  __syncthreads();
  f32x4 own[3];
#pragma unroll
  for (int off = 1; off < 4; ++off) {
    if (off >= tiles) break;                           // uniform
    own[off - 1] = f32x4{0, 0, 0, 0};
    if (wave + off < tiles) {
      const int bi = wave + off, bj = wave;
      f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0}, first;
#pragma unroll
      for (int c = 0; c < 4; ++c) first[c] = s_A[(16 * bj + 4 * g + c) * PITCH + 16 * bj + m];
      for (int b = bj; b < bi; ++b) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(s_A + (16 * bi + m) * PITCH + 16 * b + 4 * g);
        const f32x4 u = b == bj ? first : s_T[b * (b - 1) / 2 + bj][lane];
#pragma unroll
        for (int c = 0; c < 4; ++c) x = __builtin_amdgcn_mfma_f32_16x16x4f32(w[c], u[c], x, 0, 0, 0);
      }
      const f32x4 w = *reinterpret_cast<const f32x4 *>(s_A + (16 * bi + m) * PITCH + 16 * bi + 4 * g);
#pragma unroll
      for (int c = 0; c < 4; ++c) y = __builtin_amdgcn_mfma_f32_16x16x4f32(w[c], x[c], y, 0, 0, 0);
      own[off - 1] = -y;
      s_T[bi * (bi - 1) / 2 + bj][lane] = -y;
    }
    __syncthreads();
  }
#pragma unroll
  for (int off = 1; off < 4; ++off)
    if (off < tiles && wave + off < tiles)
#pragma unroll
      for (int c = 0; c < 4; ++c) s_A[(16 * (wave + off) + 4 * g + c) * PITCH + 16 * wave + m] = own[off - 1][c];
  // K S and Q S of the wave's columns
  f32x4 R[4], o[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) R[t] = o[t] = f32x4{0, 0, 0, 0};
  if (cols) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u32x4 y[3];
      cut(both(S[2 * s], S[2 * s + 1]), y);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= 2 && !wide) break;                    // uniform
        const u32x4 k = s_K[t][s][lane], q = s_QT[(t * NS + s) * 64 + lane];
#pragma unroll
        for (int e = 2; e >= 0; --e) {
          R[t] = mfma(k, y[e], R[t]);
          o[t] = mfma(q, y[e], o[t]);
        }
      }
    }
  }
  uint16_t V[4][4];                                    // rows of the four tiles
  const int64_t ldv = a.ldv;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + e;
      V[t][e] = a.v[(t0 + min(i, n - 1)) * ldv + int64_t(h) * a.Dv + col];
    }
  __syncthreads();
  if (wave < 4 && 32 * (wave >> 1) < n) {
    const int i = dealt(wave, m);
    for (int s = 0; s <= wave >> 1; ++s) {
      u32x4 x[kParts];
      solver_row<PITCH>(s_A, s_b, i, 32 * s + 8 * g, x);
#pragma unroll
      for (int e = 0; e < kParts; ++e) s_QT[(e * kTriangle + tri_at(wave, s)) * 64 + lane] = x[e];
    }
  }
  // R = V - exp(D) K S, in parts; what must not be seen counts as zero
  uint64_t gone = bad;
  u32x4 x[2][3];
  if (cols) {
    const uint64_t none = bad | (n < kChunk ? ~uint64_t(0) << n : 0);
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= 2 && !wide) break;
      const f32x4 grown = *reinterpret_cast<const f32x4 *>(s_grown + 32 * (t >> 1) + 8 * g + 4 * (t & 1));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = bf16_bits_to_float(V[t][e]);
        sum += v;
        R[t][e] = fmaf(-grown[e], R[t][e], v);
        o[t][e] *= grown[e];
      }
    }
    if (none || __any(!__builtin_isfinite(sum))) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + e;
          const bool off = none >> i & 1, lost = !__builtin_isfinite(bf16_bits_to_float(V[t][e]));
          if (!off && lost) gone |= uint64_t(1) << i;
          if (off || lost) R[t][e] = 0.0f;
        }
      gone |= __shfl_xor(gone, 16, 64);                // a column's four lanes
      gone |= __shfl_xor(gone, 32, 64);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s == 0 || wide) cut(both(R[2 * s], R[2 * s + 1]), x[s]);
  }
  __syncthreads();
  if (cols) {
    f32x4 U[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      U[t] = f32x4{0, 0, 0, 0};
      if (t >= 2 && !wide) continue;
#pragma unroll
      for (int s = 0; s <= t >> 1; ++s) {
        u32x4 w[kParts];
#pragma unroll
        for (int e = 0; e < kParts; ++e) w[e] = s_QT[(e * kTriangle + tri_at(t, s)) * 64 + lane];
#pragma unroll
        for (int j = 0; j < kPartProducts; ++j) U[t] = mfma(w[kOfFirst[j]], x[s][kOfSecond[j]], U[t]);
      }
    }
    // out = scale (exp(D) Q S + P U)
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s == 0 || wide) {
        u32x4 u[kParts];
        cut(both(U[2 * s], U[2 * s + 1]), u);
#pragma unroll
        for (int t = 2 * s; t < 4; ++t) {
          if (t >= 2 && !wide) break;
          u32x4 w[kParts];
#pragma unroll
          for (int e = 0; e < kParts; ++e) w[e] = s_P[(e * kTriangle + tri_at(t, s)) * 64 + lane];
#pragma unroll
          for (int j = 0; j < kPartProducts; ++j) o[t] = mfma(w[kOfFirst[j]], u[kOfSecond[j]], o[t]);
        }
      }
    if (__any(gone != 0)) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (gone & s_seen[32 * (t >> 1) + 8 * g + 4 * (t & 1) + e]) o[t][e] = __builtin_nanf("");
    }
    const int64_t out_row = int64_t(a.Hv) * a.Dv;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= 2 && !wide) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + e;
        if (i < n) out[i * out_row] = uint16_t(pack_bf16(a.scale * o[t][e], 0.0f));
      }
    }
    if constexpr (!TREE) {                             // S = exp(D_last) S + K^T (exp(D_last - D) U)
      const float decay = s_grown[n - 1];
      u32x4 w[2][3];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s == 0 || wide) {
          const f32x4 *left = reinterpret_cast<const f32x4 *>(s_left + 32 * s + 8 * g);
          cut(both(left[0] * U[2 * s], left[1] * U[2 * s + 1]), w[s]);
        }
#pragma unroll
      for (int t = 0; t < 2 * NS; ++t) {
        float *to = state + int64_t(32 * (t >> 1) + 4 * (t & 1)) * a.Dv;
        f32x4 next = {0, 0, 0, 0};
        if (!rq.fresh)
#pragma unroll
          for (int e = 0; e < 4; ++e) next[e] = decay * to[int64_t(e) * a.Dv];
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (s == 0 || wide) {
            const u32x4 key = transposed(s_K[2 * s][t >> 1][lane], s_K[2 * s + 1][t >> 1][lane], t & 1, m, g);
#pragma unroll
            for (int e = 2; e >= 0; --e) next = mfma(key, w[s][e], next);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) to[int64_t(e) * a.Dv] = gone ? __builtin_nanf("") : next[e];
      }
    }
  }
}

// Which kernels take a call: token by token for few tokens, one launch for trees and chains
// of one chunk, chunks prepared beforehand for the rest.  Kernels, us, with states that come from
// memory (the calls go through 800 MB of them in turn):
//   48 heads of 128 x 128
//   chains of tokens       1     4     6     8    16    32    64
//   1 request:   step    6.0   8.2   9.8  11.2  17.5  30.7  57.4
//                chunk  12.9  13.0  13.1  13.1  13.2  13.4  17.9
//                scan   14.9  15.2  15.3  15.4  15.1  16.0  20.6
//   64 requests: step   79.4  93.6   118   155   260   464   874
//                chunk   125   129   128   129   133   138   180
//                scan    257   271   273   276   279   285   342
//   16 heads of 64 x 64
//   1 request:   step    5.2   7.1   8.5   9.9  15.1  26.5  49.4
//                chunk   9.6   9.6   9.7   9.8   9.8   9.7  12.4
//   64 requests: step   13.4  19.4  24.0  28.6  44.5  80.5   154
//                chunk  24.3  24.4  24.8  24.8  24.8  25.3  33.9
// Trees of 64 with 48 heads of 128 x 128 take 15.8 us for one request, 38 for 16, 152 for 64; in
// the scan's chunks 20, 86 and 313.  One form serves the whole call: 63 single tokens beside a
// chain of 512 take 285 us in the scan, where each alone takes 78 (step) and 44.
constexpr int64_t kStepTokens = 6;
enum class Form { kStep, kChunk, kScan };
Form form_of(int64_t max_nodes, bool tree) {
  if (!tree && max_nodes <= kStepTokens) return Form::kStep;
  return max_nodes <= kChunk ? Form::kChunk : Form::kScan;
}
size_t up(size_t n) { return (n + 255) / 256 * 256; }
int64_t chunks_of(int64_t T, int64_t R) { return T / kChunk + R; }

// Workgroups of a form's launch over all requests, heads and columns; of threads_of threads.
int64_t groups_of(Form form, int64_t R, int64_t Hk, int64_t G, int64_t Dv) {
  return form == Form::kStep    ? R * Hk * G * ((Dv + 31) / 32)
         : form == Form::kChunk ? R * Hk * G * ((Dv + 127) / 128)
                                : (R * Hk + 7) / 8 * 8 * G * ((Dv + 31) / 32);
}
int threads_of(Form form) { return form == Form::kStep ? kThreads : form == Form::kChunk ? kFusedThreads : kScanThreads; }

template <int DK>
hipError_t run(DeltaArgs a, Form form, hipStream_t stream) {
  (void)hipGetLastError();
  const dim3 grid(unsigned(groups_of(form, a.R, a.Hk, a.G, a.Dv))), threads(threads_of(form));
  if (form == Form::kStep) {
    hipLaunchKernelGGL((delta_step_kernel<DK, false>), grid, threads, 0, stream, a, 1);
    set_last_kernel("delta_step");
    return hipGetLastError();
  }
  if (form == Form::kChunk) {
    if (a.tree_mask) hipLaunchKernelGGL((delta_chunk_kernel<DK, true>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((delta_chunk_kernel<DK, false>), grid, threads, 0, stream, a);
    set_last_kernel(a.tree_mask ? "delta_tree" : "delta_chunk");
    return hipGetLastError();
  }
  hipLaunchKernelGGL((delta_prep_kernel<DK>), dim3(unsigned(chunks_of(a.T, a.R)), unsigned((a.Hv + 3) / 4)), dim3(kThreads), 0, stream, a);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((delta_scan_kernel<DK>), grid, threads, 0, stream, a);
  set_last_kernel("delta_scan");
  return hipGetLastError();
}

}  // namespace

size_t delta_workspace_bytes(int64_t T, int64_t R, int64_t Hk, int64_t G, int64_t Dk, int64_t max_nodes, bool tree) {
  if (form_of(max_nodes, tree) != Form::kScan) return 0;
  const size_t n = size_t(chunks_of(T, R));
  return up(n * size_t(Hk * G) * kHeadBytes) + n * size_t(Hk) * key_bytes(int(Dk));
}

bool delta_fits_grid(int64_t T, int64_t R, int64_t Hk, int64_t G, int64_t Dv, int64_t max_nodes, bool tree) {
  const Form form = form_of(max_nodes, tree);
  return fits_grid(groups_of(form, R, Hk, G, Dv), threads_of(form)) && (form != Form::kScan || fits_grid(chunks_of(T, R), kThreads));
}

hipError_t launch_delta_rule(DeltaArgs a, int64_t Dk, int64_t max_nodes, void *workspace, hipStream_t stream) {
  const Form form = form_of(max_nodes, a.tree_mask != nullptr);
  a.heads = static_cast<char *>(workspace);
  a.keys = a.heads + up(size_t(chunks_of(a.T, a.R)) * size_t(a.Hv) * kHeadBytes);
  return Dk == 64 ? run<64>(a, form, stream) : run<128>(a, form, stream);
}

static int64_t conv_groups_of(int64_t C) { return (C + 8 * kThreads - 1) / (8 * kThreads); }

int64_t delta_commit_groups(int64_t L, int64_t R, int64_t Hv, int64_t Dv, int64_t C) {
  return L * R * (Hv * ((Dv + 31) / 32) + conv_groups_of(C));
}

hipError_t launch_delta_commit(const DeltaArgs &a, int64_t Dk, hipStream_t stream) {
  const int64_t conv = a.x ? conv_groups_of(a.C) : 0, grid = delta_commit_groups(a.L, a.R, a.Hv, a.Dv, a.x ? a.C : 0);
  (void)hipGetLastError();
  if (Dk == 64) hipLaunchKernelGGL((delta_step_kernel<64, true>), dim3(unsigned(grid)), dim3(kThreads), 0, stream, a, int(conv));
  else hipLaunchKernelGGL((delta_step_kernel<128, true>), dim3(unsigned(grid)), dim3(kThreads), 0, stream, a, int(conv));
  set_last_kernel("delta_commit");
  return hipGetLastError();
}

}  // namespace tl
