// Attention of a step's tokens (drafted trees, single tokens or prompt chunks) over a
// paged K/V cache.
//
// For row (node, query head) and the keys it may see (the request's context, and in
// the tree its ancestors and itself):
//   o = sum_k exp(s_k - M) v_k / sum_k exp(s_k - M),  s_k = scale q.k,  M = max_k s_k
// in one pass with the running maximum and sum held in f32.
//
// Design.  Scores are computed transposed, S^T = K Q^T, with v_mfma_f32_16x16x32_bf16:
// 16 keys are the rows of A and 16 query rows the columns of B.  Two such products over
// 32 keys leave a lane with 8 consecutive keys of one query row (the cache's order of K
// rows sees to that), so the row's maximum, sum and rescale factor are plain per-lane
// scalars, and the probabilities are, as they lie, the B operand of O^T = V^T P^T.
// K and V go from memory straight into operand registers in 1 KB loads; LDS only joins
// the four waves of a workgroup.
//
// Work is cut into units of kUnitKeys keys of one (request, cache head, row block), and
// workgroup w of W takes units [w U / W, (w + 1) U / W): lengths live on the device, so
// the cut is made there, evenly whatever the lengths are, and the host never waits.
// An item that falls to several workgroups leaves partial sums in the workspace, which
// tree_combine_kernel adds in a fixed order.
//
// Two forms: `split` (few rows) gives the four waves of a workgroup the same rows and
// different keys; `share` (many rows) gives them different rows and the same keys.
//
// Rounding: q.k and p.v are sums of bf16 products in f32; the probabilities are
// rounded once to bf16 for the product with V (relative 2^-9 each, with errors of both
// signs), while their sum is taken before that rounding.
#include <type_traits>

#include "kv_layout.h"
#include "tl_device.h"

namespace tl {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepKeys = 32;                 // keys of one step of a wave: two tiles
constexpr int kUnitSteps = 4;
constexpr int kUnitKeys = kStepKeys * kUnitSteps;
constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxGrid = 512;
constexpr float kNegInf = -__builtin_inff();

// ---------------------------------------------------------------------------
// which units there are
struct Item {
  int r, h, b;         // request, cache head, row block
  int n, kv;           // the request's nodes and cache length (its nodes' keys among them)
  int units;           // of this item
  int at;              // unit inside the item
  int64_t first;       // global index of the item's first unit
};

__device__ __forceinline__ int request_nodes(const TreeArgs &a, int r) {
  const int lo = max(a.q_start[r], 0), hi = min(a.q_start[r + 1], a.T);
  return max(hi - lo, 0);
}
__device__ __forceinline__ int request_keys(const TreeArgs &a, int r) {
  return min(max(a.kv_lens[r], 0), a.max_keys);
}
__device__ __forceinline__ int row_blocks(int n, int G, int rows) { return int((int64_t(n) * G + rows - 1) / rows); }

// A request of up to 64 nodes has the same keys for every row block; a longer one is a
// chain, whose row block ends at its last node's own key.
__device__ __forceinline__ int block_keys(int n, int kv, int b, int G, int rows) {
  if (n <= kTreeNodes) return kv;
  const int last = int((min(int64_t(b + 1) * rows, int64_t(n) * G) - 1) / G);
  return max(kv - n + last + 1, 0);
}
__device__ __forceinline__ int block_units(int n, int kv, int b, int G, int rows) {
  return max((block_keys(n, kv, b, G, rows) + kUnitKeys - 1) / kUnitKeys, 1);
}

// pre[r] = units of the requests before r (R + 1 entries), by the whole workgroup.
__device__ __forceinline__ void unit_prefix(const TreeArgs &a, int rows, int *pre, int *red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.R + kThreads - 1) / kThreads, r0 = tid * per;
  int sum = 0;
  for (int j = 0; j < per; ++j) {  // the same count in every lane: the loop below needs them all
    const int r = r0 + j;
    int n = 0, kv = 0, units = 0;
    if (r < a.R) {
      n = request_nodes(a, r);
      kv = request_keys(a, r);
      if (n && n <= kTreeNodes) units = row_blocks(n, a.G, rows) * block_units(n, kv, 0, a.G, rows);
    }
    uint64_t longs = __ballot(n > kTreeNodes);
    while (longs) {
      const int src = __builtin_ctzll(longs);
      longs &= longs - 1;
      const int ln = __shfl(n, src, 64), lkv = __shfl(kv, src, 64), nb = row_blocks(ln, a.G, rows);
      int part = 0;
      for (int b = lane; b < nb; b += 64) part += block_units(ln, lkv, b, a.G, rows);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) part += __shfl_xor(part, off, 64);
      if (lane == src) units = part;
    }
    sum += units * a.H;
    if (r < a.R) pre[r + 1] = sum;  // within this thread so far
  }
  int run = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(run, off, 64);
    if (lane >= off) run += up;
  }
  if (lane == 63) red[wave] = run;
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  int before = run - sum;
  for (int w = 0; w < wave; ++w) before += red[w];
  for (int j = 0; j < per; ++j)
    if (r0 + j < a.R) pre[r0 + j + 1] += before;
  __syncthreads();
}

// The item that holds unit u < pre[R]; every lane of the wave takes part.
__device__ __forceinline__ Item locate(const TreeArgs &a, int rows, const int *pre, int u) {
  Item it;
  int lo = 0, hi = a.R;  // pre[lo] <= u < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid;
  }
  it.r = lo;
  it.n = request_nodes(a, lo);
  it.kv = request_keys(a, lo);
  const int per_head = (pre[lo + 1] - pre[lo]) / a.H, local = u - pre[lo];
  it.h = local / per_head;
  int v = local - it.h * per_head;
  if (it.n <= kTreeNodes) {
    it.units = block_units(it.n, it.kv, 0, a.G, rows);
    it.b = v / it.units;
    v -= it.b * it.units;
  } else {
    const int lane = threadIdx.x & 63, nb = row_blocks(it.n, a.G, rows);
    it.b = 0;
    it.units = 0;
    for (int base = 0; base < nb; base += 64) {
      const int mine = base + lane < nb ? block_units(it.n, it.kv, base + lane, a.G, rows) : 0;
      int run = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(run, off, 64);
        if (lane >= off) run += up;
      }
      const uint64_t past = __ballot(run > v);
      if (past) {
        const int at = __builtin_ctzll(past);
        v -= __shfl(run - mine, at, 64);
        it.units = __shfl(mine, at, 64);
        it.b = base + at;
        break;
      }
      v -= __shfl(run, 63, 64);
    }
  }
  it.at = v;
  it.first = u - v;
  return it;
}

// first unit of workgroup w of 2^grid_log
__device__ __forceinline__ int first_unit(int w, int total, int grid_log) {
  return int((int64_t(total) * w) >> grid_log);
}

// Workgroups are dealt to the eight XCDs in turn: workgroup indices are renamed so that
// an XCD gets neighbouring units, whose row blocks read the same keys from its own L2.
__device__ __forceinline__ int renamed(int id, int grid_log) {
  return ((id & 7) << (grid_log - 3)) + (id >> 3);
}

// ---------------------------------------------------------------------------
// registers
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}
// four e4m3 bytes -> four bf16 (exact)
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
}
__device__ __forceinline__ bf16x8 as_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  u32x4 v = {a, b, c, d};
  return __builtin_bit_cast(bf16x8, v);
}
// maximum and sum over the four lanes that share a query row (lane, lane ^ 16, ...)
__device__ __forceinline__ float row_max(float x) {
  auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// One step's K or V: two tiles as loaded.
template <int D, bool E4M3>
struct Tiles {
  static constexpr int C = E4M3 ? D / 32 : D / 16;  // 1 KB loads a step
  u32x4 w[C];

  // K: `at` is the lane's place in chunk 0 of its tile (lanes m < 8 the first tile, the
  // others the second); the second product's tokens are 8 places on
  template <int FROM = 0, int TO = C / 2>
  __device__ __forceinline__ void load_k(const char *at) {
#pragma unroll
    for (int c = FROM; c < TO; ++c) {
      w[2 * c] = *reinterpret_cast<const u32x4 *>(at + 1024 * c);
      w[2 * c + 1] = *reinterpret_cast<const u32x4 *>(at + 1024 * c + 128);
    }
  }
  // V: lanes g < 2 the first tile, the others the second
  __device__ __forceinline__ void load_v(const char *at) {
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = *reinterpret_cast<const u32x4 *>(at + 512 * c);
  }
  // the A operand of K: product t, 32 d's number j (of D / 32)
  __device__ __forceinline__ bf16x8 k_operand(int t, int j) const {
    if constexpr (!E4M3) {
      return __builtin_bit_cast(bf16x8, w[2 * j + t]);
    } else {
      const u32x4 x = w[2 * (j >> 1) + t];
      const uint32_t a = x[2 * (j & 1)], b = x[2 * (j & 1) + 1];
      return as_operand(e4m3_lo(a), e4m3_hi(a), e4m3_lo(b), e4m3_hi(b));
    }
  }
  // the A operand of V: 16 d's number j (of D / 16)
  __device__ __forceinline__ bf16x8 v_operand(int j) const {
    if constexpr (!E4M3) {
      return __builtin_bit_cast(bf16x8, w[j]);
    } else {
      const uint32_t a = w[j >> 1][2 * (j & 1)], b = w[j >> 1][2 * (j & 1) + 1];
      return as_operand(e4m3_lo(a), e4m3_hi(a), e4m3_lo(b), e4m3_hi(b));
    }
  }
  // V: zero all but the keys in `keep` (a bit for each of the lane's eight); their P is
  // zero, but 0 * NaN is not
  __device__ __forceinline__ void keep_keys(uint32_t keep) {
    uint32_t m[4];
    if constexpr (!E4M3) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m[e] = (keep >> (2 * e) & 1 ? 0xFFFFu : 0u) | (keep >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[e] |= keep >> (4 * e + i) & 1 ? 0xFFu << (8 * i) : 0u;
        m[e + 2] = m[e];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[c][e] &= m[e];
  }
  // V: whether the lane holds an infinity or NaN
  __device__ __forceinline__ bool not_finite() const {
    uint32_t bad = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) bad |= odd_bits(w[c][e]);
    return bad != 0;
  }
  // V: infinities and NaN to zero
  __device__ __forceinline__ void drop_not_finite() {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = odd_bits(w[c][e]);          // 0x8000 (0x80) of an element turns into all its bits
        w[c][e] &= ~(E4M3 ? (b >> 7) * 0xFFu : (b >> 15) * 0xFFFFu);
      }
  }

 private:
  // the top bit of every element that is not finite (e4m3 has no infinities; NaN is 0x7F with either sign)
  static __device__ __forceinline__ uint32_t odd_bits(uint32_t x) {
    return E4M3 ? ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  }
};

// element d = 16 j + i past a V tile's `at` (an e4m3 one as it stands, without its scale)
template <bool E4M3>
__device__ __forceinline__ float v_element(const char *at, int j, int i) {
  if constexpr (!E4M3) {
    return bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(at + 512 * j + 16 * i));
  } else {
    const uint32_t x = *reinterpret_cast<const uint8_t *>(at + 512 * (j >> 1) + 8 * (j & 1) + 16 * i);
    return bf16_bits_to_float(e4m3_lo(x) & 0xFFFFu);
  }
}

template <int D, int RT>
struct Rows {
  f32x4 o[D / 16][RT];  // lane (n, g): query row n of row tile t, d = 16 j + 4 g + i
  float m[RT], l[RT];   // running maximum (raw scores) and the lane's share of the sum
};

template <int D, bool E4M3, int RT, bool SHARE>
struct Variant {
  static constexpr int rows = 16 * RT * (SHARE ? kWaves : 1);
  // workgroups a compute unit holds, by registers: where it is one, 512 of them a lane
  static constexpr int occupancy = D * (E4M3 ? 1 : 2) * RT > 512 || D * RT > 256 || D * (E4M3 ? 1 : 2) > 256 ? 1 : 2;
  static constexpr int grid_log = occupancy == 1 ? 8 : 9;
};

// ---------------------------------------------------------------------------
template <int D, bool E4M3, int RT, bool SHARE>
__global__ __launch_bounds__(kThreads, (Variant<D, E4M3, RT, SHARE>::occupancy)) void tree_attention_kernel(const TreeArgs a) {
  constexpr int ROWS = Variant<D, E4M3, RT, SHARE>::rows;
  constexpr int QC = D / 32, OC = D / 16;
  // the four waves' sums are joined in rounds of at most 64 KB of LDS
  constexpr int ROUNDS = RT * D > 256 ? RT * D / 256 : 1;
  constexpr int JT = OC / ROUNDS;                      // 16-d tiles joined in a round
  constexpr int JW = JT / kWaves;                      // of which each wave finishes this many
  static_assert(JW * kWaves * ROUNDS == OC, "rounds");
  extern __shared__ __align__(16) char lds[];
  f32x4 *join = reinterpret_cast<f32x4 *>(lds);        // [wave][JT][RT][64] (split form only)
  float *stat = reinterpret_cast<float *>(lds + (SHARE ? 0 : kWaves * JT * RT * 1024));  // [wave][2][RT * 16]
  int *pre = reinterpret_cast<int *>(stat + (SHARE ? 0 : kWaves * 2 * RT * 16));
  __shared__ int red[kWaves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row16 = lane & 15, g = lane >> 4;
  constexpr int LOG = Variant<D, E4M3, RT, SHARE>::grid_log;
  const int w = renamed(blockIdx.x, LOG);
  unit_prefix(a, ROWS, pre, red);
  const int total = __builtin_amdgcn_readfirstlane(pre[a.R]);
  const int u_begin = first_unit(w, total, LOG), u_end = first_unit(w + 1, total, LOG);
  const float c2 = a.scale * 1.44269504088896340736f;  // scores to powers of two

  for (int u = u_begin; u < u_end;) {
    const Item it = locate(a, ROWS, pre, u);
    const int r = __builtin_amdgcn_readfirstlane(it.r), h = __builtin_amdgcn_readfirstlane(it.h);
    const int n = __builtin_amdgcn_readfirstlane(it.n), kv = __builtin_amdgcn_readfirstlane(it.kv);
    const int blk = __builtin_amdgcn_readfirstlane(it.b), units = __builtin_amdgcn_readfirstlane(it.units);
    const int at = __builtin_amdgcn_readfirstlane(it.at);
    const int take = min(units - at, u_end - u);
    const bool whole = take == units;
    const int slot = 2 * w + (u == u_begin ? 0 : 1);   // of this workgroup's partial sums
    u += take;

    // this wave's rows
    const bool flat = n <= kTreeNodes;
    const int ctx = kv - n;
    const int q0 = max(a.q_start[r], 0);
    const int row0 = blk * ROWS + (SHARE ? wave * 16 * RT : 0);
    bf16x8 q[QC][RT];
    uint64_t sees[RT];                                 // flat: nodes the row may see
    int node[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = row0 + 16 * t + row16;
      node[t] = row / a.G;
      const bool there = node[t] < n;
      const int64_t tok = q0 + (there ? node[t] : 0);
      sees[t] = 0;
      if (flat && there)
        sees[t] = a.tree_mask ? a.tree_mask[tok] : (~uint64_t(0) >> (63 - node[t]));
      const uint16_t *src = a.q + tok * a.ldq + int64_t(h * a.G + (there ? row - node[t] * a.G : 0)) * D;
#pragma unroll
      for (int j = 0; j < QC; ++j) {
        const int d = E4M3 ? 64 * (j >> 1) + 16 * g + 8 * (j & 1) : 32 * j + 8 * g;
        u32x4 v = *reinterpret_cast<const u32x4 *>(src + d);
        if (!there) v = u32x4{0, 0, 0, 0};
        q[j][t] = __builtin_bit_cast(bf16x8, v);
      }
    }
    // keys that all of the wave's rows see come first: below `clear` no mask is looked at
    const int clear = flat ? ctx : ctx + row0 / a.G + 1;
    const int key_end = block_keys(n, kv, blk, a.G, ROWS);

    Rows<D, RT> acc;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      acc.m[t] = kNegInf;
      acc.l[t] = 0.0f;
#pragma unroll
      for (int j = 0; j < OC; ++j) acc.o[j][t] = f32x4{0, 0, 0, 0};
    }

    // this wave's steps of the segment
    const int steps_end = min((at + take) * kUnitSteps, (key_end + kStepKeys - 1) / kStepKeys);
    int s0 = at * kUnitSteps, s1 = max(steps_end, s0);
    if (SHARE) {
      if (row0 >= n * a.G) s1 = s0;                    // a wave past the last row
    } else {
      const int len = s1 - s0, base = s0;
      s0 = base + len * wave / kWaves;
      s1 = base + len * (wave + 1) / kWaves;
    }
    const int shift = a.block_shift;                   // tokens of a page, as a power of two
    const int32_t *table = a.table + int64_t(r) * a.table_width;
    int page_base = (s0 * kStepKeys) >> shift;
    int page_ids = page_base + lane < a.table_width ? table[page_base + lane] : -1;

    // tile number 2 s + t: where it is, and how many of its keys there are
    auto place = [&](int s, int t, int64_t &tile, int &lim) {
      const int pos = s * kStepKeys + 16 * t;
      int page = (pos >> shift) - page_base;
      if (page >= 64) {                                // uniform
        page_base += page;
        page_ids = page_base + lane < a.table_width ? table[page_base + lane] : -1;
        page = 0;
      }
      int id = __builtin_amdgcn_readlane(page_ids, page);
      lim = min(max(key_end - pos, 0), 16);
      if (lim == 0 || uint32_t(id) >= uint32_t(a.pages)) {
        id = 0;
        lim = 0;
      }
      // in tokens: the cache's element offset is this times D
      tile = ((int64_t(id) * a.H + h) << shift) + (pos & ((1 << shift) - 1));
    };
    constexpr int ES = E4M3 ? 1 : 2;
    const int k_lane = 256 * g + 16 * (row16 & 7), v_lane = 256 * (g & 1) + 16 * row16;
    // one step, tokens at t0 and t1; the second form looks at masks, at keys that are not
    // there and at values that are not finite, the first knows that all rows see all keys
    auto step = [&](int s, int64_t t0, int64_t t1, [[maybe_unused]] int lim0, [[maybe_unused]] int lim1,
                    auto mask_tag) {
      constexpr bool MASKED = decltype(mask_tag)::value;
      Tiles<D, E4M3> kt, vt;
      // all loads are on their way before the first wait; where that takes too many
      // registers, K's second half and V take the place of K's first
      constexpr bool LATE_V = D * ES * RT > 512;
      const char *k_at = a.k + (row16 < 8 ? t0 : t1) * (D * ES) + k_lane;
      const char *v_at = a.v + (g < 2 ? t0 : t1) * (D * ES) + v_lane;
      if constexpr (LATE_V)
        kt.template load_k<0, D / 64>(k_at);
      else
        kt.load_k(k_at);
      f32x4 ks[2], vs[2];                              // e4m3: the scales of the lane's tokens
      if constexpr (E4M3) {
        const int64_t at = (g < 2 ? t0 : t1) + 8 * (g & 1);
        ks[0] = *reinterpret_cast<const f32x4 *>(a.k_scale + at);
        ks[1] = *reinterpret_cast<const f32x4 *>(a.k_scale + at + 4);
        vs[0] = *reinterpret_cast<const f32x4 *>(a.v_scale + at);
        vs[1] = *reinterpret_cast<const f32x4 *>(a.v_scale + at + 4);
      }
      if constexpr (!LATE_V) vt.load_v(v_at);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 sc[2][RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sc[0][t] = sc[1][t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < QC; ++j) {
        if (LATE_V && j == QC / 2) {
          __builtin_amdgcn_sched_barrier(0);
          kt.template load_k<D / 64, D / 32>(k_at);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 ka = kt.k_operand(i, j);
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[i][t] = mfma(ka, q[j][t], sc[i][t]);
        }
      }
      if constexpr (LATE_V) {
        __builtin_amdgcn_sched_barrier(0);
        vt.load_v(v_at);
      }
      if constexpr (E4M3) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[0][t][i] *= ks[0][i];
            sc[1][t][i] *= ks[1][i];
          }
      }
      [[maybe_unused]] const int pos = s * kStepKeys;
      [[maybe_unused]] uint32_t vis[RT];               // a bit for each of the lane's eight keys
      [[maybe_unused]] bool rare = false;
      [[maybe_unused]] uint32_t zero[RT];              // as vis: its probability is 0
      if constexpr (MASKED) {
        const int left = min(max((g < 2 ? lim0 : lim1) - 8 * (g & 1), 0), 8);
        const uint32_t have = (1u << left) - 1u;
        const int j0 = pos + 8 * g - ctx;              // the node of the lane's first key
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (flat) {
            vis[t] = j0 <= -8 ? 255u : j0 < 0 ? uint32_t(sees[t] << -j0) | ((1u << -j0) - 1u)
                                              : j0 < 64 ? uint32_t(sees[t] >> j0) : 0u;
          } else {
            vis[t] = (1u << min(max(node[t] - j0 + 1, 0), 8)) - 1u;
          }
          vis[t] &= have;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(vis[t] >> i & 1)) sc[i >> 2][t][i & 3] = kNegInf;
        }
        vt.keep_keys(have);
        bool odd = vt.not_finite();
        if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {                // what the scales of absent tokens hold is not used
            const float x = have >> i & 1 ? vs[i >> 2][i & 3] : 0.0f;
            const bool bad = !(fabsf(x) < __builtin_inff());
            odd |= bad;
            vs[i >> 2][i & 3] = bad ? 0.0f : x;
          }
        }
        rare = __any(odd);
        if (rare) vt.drop_not_finite();
      }

      bf16x8 p[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float top = fmaxf(fmaxf(fmaxf(sc[0][t][0], sc[0][t][1]), fmaxf(sc[0][t][2], sc[0][t][3])),
                          fmaxf(fmaxf(sc[1][t][0], sc[1][t][1]), fmaxf(sc[1][t][2], sc[1][t][3])));
        top = fmaxf(row_max(top), acc.m[t]);
        if (__any(top > acc.m[t])) {
          const float f = top > acc.m[t] ? __builtin_amdgcn_exp2f((acc.m[t] - top) * c2) : 1.0f;
          acc.l[t] *= f;
#pragma unroll
          for (int j = 0; j < OC; ++j) acc.o[j][t] *= f;
          acc.m[t] = top;
        }
        const float mc = top == kNegInf ? 0.0f : top * c2;
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i >> 2][t][i & 3], c2, -mc));
        acc.l[t] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        if constexpr (MASKED) {
          zero[t] = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) zero[t] |= uint32_t(e[i] == 0.0f) << i;
        }
        if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] *= vs[i >> 2][i & 3];
        }
        p[t] = as_operand(pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7]));
      }

#pragma unroll
      for (int j = 0; j < OC; ++j) {
        const bf16x8 va = vt.v_operand(j);
#pragma unroll
        for (int t = 0; t < RT; ++t) acc.o[j][t] = mfma(va, p[t], acc.o[j][t]);
      }
      if constexpr (MASKED) {
        // An infinity or NaN of a node that some rows do not see must not reach them
        // through 0 * inf: the products above went without it, and it is added key by
        // key where the row sees the key.
        if (rare)
          for (int kk = 0; kk < kStepKeys; ++kk) {
            const int token = kk & 15;
            if (token >= (kk < 16 ? lim0 : lim1)) continue;
            const int64_t at = kk < 16 ? t0 : t1;
            const char *tile = a.v + (at * D + kv_tile_v(token, 4 * g, ES)) * ES;
            const float scale = E4M3 ? a.v_scale[at + token] : 1.0f;
            const int from = row16 + 16 * (kk >> 3), e = kk & 7;
            float with[RT];                            // NaN: 0 * inf; 0: not seen
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              const int on = __shfl(int(vis[t]), from, 64) >> e & 1, none = __shfl(int(zero[t]), from, 64) >> e & 1;
              with[t] = !on ? 0.0f : none ? __builtin_nanf("") : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < OC; ++j) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float v = v_element<E4M3>(tile, j, i) * scale;
                const bool finite = fabsf(v) < __builtin_inff();
#pragma unroll
                for (int t = 0; t < RT; ++t) acc.o[j][t][i] += finite || with[t] == 0.0f ? 0.0f : with[t] * v;
              }
              __builtin_amdgcn_sched_barrier(0);       // few registers: the loop hardly ever runs
            }
          }
      }
    };
    // the keys that every row sees; from the first page that is not one, or the first node
    // on, the careful form
    int s = s0;
    int64_t t0, t1;
    int lim0, lim1;
    for (; s < s1; ++s) {
      place(s, 0, t0, lim0);
      place(s, 1, t1, lim1);
      if (s * kStepKeys + kStepKeys > clear || lim0 + lim1 < 32) break;
      step(s, t0, t1, 16, 16, std::false_type());
    }
    for (; s < s1; ++s) {
      place(s, 0, t0, lim0);
      place(s, 1, t1, lim1);
      step(s, t0, t1, lim0, lim1, std::true_type());
    }

    // ---- the segment's results
#pragma unroll
    for (int t = 0; t < RT; ++t) acc.l[t] = row_sum(acc.l[t]);
    float top[RT], total_l[RT];
    if constexpr (SHARE) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        top[t] = acc.m[t];
        total_l[t] = acc.l[t];
      }
    } else {
      __syncthreads();                                 // the last segment's readers are done
#pragma unroll
      for (int t = 0; t < RT; ++t)
        if (g == 0) {
          stat[(wave * 2 + 0) * RT * 16 + 16 * t + row16] = acc.m[t];
          stat[(wave * 2 + 1) * RT * 16 + 16 * t + row16] = acc.l[t];
        }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float mw[kWaves];
        top[t] = kNegInf;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          mw[v] = stat[(v * 2 + 0) * RT * 16 + 16 * t + row16];
          top[t] = fmaxf(top[t], mw[v]);
        }
        total_l[t] = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          const float f = mw[v] == top[t] ? 1.0f : __builtin_amdgcn_exp2f((mw[v] - top[t]) * c2);
          total_l[t] += f * stat[(v * 2 + 1) * RT * 16 + 16 * t + row16];
        }
        const float f = acc.m[t] == top[t] ? 1.0f : __builtin_amdgcn_exp2f((acc.m[t] - top[t]) * c2);
#pragma unroll
        for (int j = 0; j < OC; ++j) acc.o[j][t] *= f;
      }
    }

    // where the lane's values go: four d's of row n in each 16-d tile
    float inv[RT];
    int64_t to[RT];                                    // element offset of the row, in out or part_o
    bool there[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = row0 + 16 * t + row16;
      there[t] = node[t] < n;
      inv[t] = !whole || total_l[t] == 0.0f ? 0.0f : 1.0f / total_l[t];
      const int64_t line = whole ? int64_t(q0 + node[t]) * a.H * a.G + h * a.G + (row - node[t] * a.G)
                                 : int64_t(slot) * ROWS + row - blk * ROWS;
      to[t] = line * D + 4 * g;
      if (there[t] && g == 0 && (SHARE || wave == 0)) {
        if (!whole) {
          a.part_ml[2 * line] = top[t];
          a.part_ml[2 * line + 1] = total_l[t];
        } else if (a.lse) {
          a.lse[line] = top[t] == kNegInf
                            ? kNegInf
                            : (top[t] * c2 + __builtin_amdgcn_logf(total_l[t])) * 0.693147180559945309f;
        }
      }
    }
    auto put = [&](int j, int t, f32x4 v) {
      if (whole) {
        const uint2 o = {pack2(v[0] * inv[t], v[1] * inv[t]), pack2(v[2] * inv[t], v[3] * inv[t])};
        *reinterpret_cast<uint2 *>(a.out + to[t] + 16 * j) = o;
      } else {
        *reinterpret_cast<f32x4 *>(a.part_o + to[t] + 16 * j) = v;
      }
    };
    if constexpr (SHARE) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
        if (there[t]) {
          if (whole) {
#pragma unroll
            for (int j = 0; j < OC; ++j) put(j, t, acc.o[j][t]);
          } else {
#pragma unroll
            for (int j = 0; j < OC; ++j) put(j, t, acc.o[j][t]);
          }
        }
    } else {
#pragma unroll
      for (int round = 0; round < ROUNDS; ++round) {
        if (round) __syncthreads();
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int t = 0; t < RT; ++t) join[((wave * JT + j) * RT + t) * 64 + lane] = acc.o[round * JT + j][t];
        __syncthreads();
#pragma unroll
        for (int jj = 0; jj < JW; ++jj)
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int j = wave * JW + jj;
            f32x4 v = join[(j * RT + t) * 64 + lane];
#pragma unroll
            for (int x = 1; x < kWaves; ++x) v += join[((x * JT + j) * RT + t) * 64 + lane];
            if (there[t]) put(round * JT + j, t, v);
          }
      }
    }
  }
}

// Adds the partial sums of items that several workgroups share.  Workgroup w looks at
// the first unit of main workgroup w: it is the owner of the item if that is the first
// such border inside it.  blockIdx.y takes every gridDim.y-th row.
__global__ __launch_bounds__(kThreads) void tree_combine_kernel(const TreeArgs a, int rows, int D, int grid_log) {
  extern __shared__ __align__(16) char lds[];
  int *pre = reinterpret_cast<int *>(lds);
  __shared__ int red[kWaves];
  const int w = blockIdx.x;
  unit_prefix(a, rows, pre, red);
  const int total = pre[a.R], s = first_unit(w, total, grid_log);
  if (s == 0 || s >= total || s == first_unit(w + 1, total, grid_log)) return;
  int w0 = w - 1;                                      // the workgroup before that has any units
  while (first_unit(w0, total, grid_log) == s) --w0;
  const Item it = locate(a, rows, pre, s);
  const int u0 = int(it.first), u1 = u0 + it.units;
  if (s == u0 || first_unit(w0, total, grid_log) > u0) return;
  // parts: the end of workgroup w0, and the beginnings of w, w + 1, ... inside the item
  const int slot0 = 2 * w0 + (first_unit(w0, total, grid_log) == u0 ? 0 : 1);
  const float c2 = a.scale * 1.44269504088896340736f;
  const int threads_a_row = D / 4, lane = threadIdx.x % threads_a_row;
  const int per_pass = kThreads / threads_a_row;
  const int q0 = max(a.q_start[it.r], 0);
  for (int row = blockIdx.y * per_pass + threadIdx.x / threads_a_row; row < rows; row += gridDim.y * per_pass) {
    const int64_t all = int64_t(it.b) * rows + row;
    const int node = int(all / a.G);
    if (node >= it.n) continue;
    float top = a.part_ml[(int64_t(slot0) * rows + row) * 2];
    for (int x = w; x < int(gridDim.x) && first_unit(x, total, grid_log) < u1; ++x)
      if (first_unit(x, total, grid_log) < first_unit(x + 1, total, grid_log))
        top = fmaxf(top, a.part_ml[(int64_t(2 * x) * rows + row) * 2]);
    f32x4 o = {0, 0, 0, 0};
    float l = 0.0f;
    auto add = [&](int64_t slot) {
      const float m = a.part_ml[(slot * rows + row) * 2];
      const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c2);
      l += f * a.part_ml[(slot * rows + row) * 2 + 1];
      o += f * *reinterpret_cast<const f32x4 *>(a.part_o + (slot * rows + row) * D + 4 * lane);
    };
    add(slot0);
    for (int x = w; x < int(gridDim.x) && first_unit(x, total, grid_log) < u1; ++x)
      if (first_unit(x, total, grid_log) < first_unit(x + 1, total, grid_log)) add(2 * x);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = int64_t(q0 + node) * a.H * a.G + it.h * a.G + (all - int64_t(node) * a.G);
    const uint2 v = {pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv)};
    *reinterpret_cast<uint2 *>(a.out + at * D + 4 * lane) = v;
    if (a.lse && lane == 0)
      a.lse[at] = top == kNegInf ? kNegInf : (top * c2 + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
  }
}

template <int D, bool E4M3, int RT, bool SHARE>
hipError_t launch(const TreeArgs &a, const char *name, hipStream_t stream) {
  constexpr int ROWS = Variant<D, E4M3, RT, SHARE>::rows;
  constexpr int ROUNDS = RT * D > 256 ? RT * D / 256 : 1;
  constexpr size_t join = SHARE ? 0 : kWaves * (D / 16 / ROUNDS) * RT * 1024 + kWaves * 2 * RT * 16 * 4;
  const size_t prefix = size_t(a.R + 1) * 4;
  (void)hipGetLastError();
  constexpr int LOG = Variant<D, E4M3, RT, SHARE>::grid_log;
  hipLaunchKernelGGL((tree_attention_kernel<D, E4M3, RT, SHARE>), dim3(1 << LOG), dim3(kThreads), join + prefix, stream, a);
  hipLaunchKernelGGL(tree_combine_kernel, dim3(1 << LOG, 4), dim3(kThreads), prefix, stream, a, ROWS, D, LOG);
  set_last_kernel(name);
  return hipGetLastError();
}

// Rows of one cache head in the step's longest request decide the form: up to 32 rows
// every row sits in each wave and the waves split the keys; above, they share the keys.
// 2-byte elements of 256-wide heads leave registers for 16 rows a wave.
struct Form {
  bool share;
  int tiles;  // of 16 rows a wave
};
Form tree_form(int64_t rows, int64_t D, bool e4m3) {
  const int most = D == 256 && !e4m3 ? 1 : 2;
  return {rows > 32, rows <= 16 ? 1 : most};
}
int form_rows(Form f) { return 16 * f.tiles * (f.share ? kWaves : 1); }

template <int D, bool E4M3>
hipError_t pick(const TreeArgs &a, Form f, hipStream_t stream) {
  if (!f.share && f.tiles == 1)
    return launch<D, E4M3, 1, false>(a, E4M3 ? "tree_attention_e4m3_split16" : "tree_attention_bf16_split16", stream);
  if constexpr (D == 256 && !E4M3) {
    return launch<D, E4M3, 1, true>(a, "tree_attention_bf16_share64", stream);
  } else {
    if (f.share)
      return launch<D, E4M3, 2, true>(a, E4M3 ? "tree_attention_e4m3_share128" : "tree_attention_bf16_share128", stream);
    return launch<D, E4M3, 2, false>(a, E4M3 ? "tree_attention_e4m3_split32" : "tree_attention_bf16_split32", stream);
  }
}

}  // namespace

size_t tree_workspace_bytes(int64_t max_nodes, int64_t group, int64_t D, bool e4m3) {
  return size_t(2 * kMaxGrid) * form_rows(tree_form(max_nodes * group, D, e4m3)) * (D + 2) * 4;
}

hipError_t launch_tree_attention(TreeArgs a, int64_t D, bool e4m3, int64_t max_nodes, void *workspace,
                                 hipStream_t stream) {
  const Form f = tree_form(max_nodes * a.G, D, e4m3);
  a.part_o = static_cast<float *>(workspace);
  a.part_ml = a.part_o + int64_t(2 * kMaxGrid) * form_rows(f) * D;
  if (e4m3) return D == 64 ? pick<64, true>(a, f, stream) : D == 128 ? pick<128, true>(a, f, stream) : pick<256, true>(a, f, stream);
  return D == 64 ? pick<64, false>(a, f, stream) : D == 128 ? pick<128, false>(a, f, stream) : pick<256, false>(a, f, stream);
}

}  // namespace tl
