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
//
// Work is cut into units of kUnitKeys keys of one (request, cache head, row block), and
// workgroup w of W takes units [w U / W, (w + 1) U / W): lengths live on the device, so
// the cut is made there, evenly whatever the lengths are, and the host never waits.
// An item that falls to several workgroups leaves partial sums in the workspace, which
// tree_combine_kernel adds in a fixed order.
//
// Measured, main and joining launch: one token over 1000 keys 9.7 + 3.9 us; 4 trees of 8 over
// 131071 e4m3 keys, 8 heads of 128, 194 + 5.4 us (5.5 TB/s; reading alone reaches 5.9); 16
// trees of 64, 4 query heads, over up to 8192 bf16 keys 99 + 14 us (2.7 TB/s, 475 TFLOP/s),
// e4m3 140 + 7; 2 prompts of 2048 on 2048, 24 query heads of 256, 345 + 17 us in bf16 (855
// TFLOP/s; a large library product reaches 1205), 403 + 17 in e4m3.
//
// Two kernels.  `split` (few rows of a cache head): bound by the cache's bytes.  The
// four waves of a workgroup hold the same rows and take different keys; K and V go from
// memory straight into operand registers, and LDS only joins the waves' sums at the end.
// `share` (more rows): bound by the matrix cores and the exponentials.  The waves hold
// different rows and take the same keys, which are staged in LDS two or four steps deep, so
// that memory is read once for 64 or 128 rows.
//
// Rounding: q.k and p.v are sums of bf16 products in f32; the probabilities (in e4m3 times
// V's scale) are rounded once to bf16 for the product with V (off by 2^-8 of it at most, with
// errors of both signs), while their sum is taken before that rounding.  It is the one place
// between the inputs and the result with fewer than 32 bits, and what the matrix instruction
// takes: outputs are off by 0.0023 of their size in the mean square, where their own rounding
// to bf16 alone makes 0.0017.
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
constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 8;                            // of a running maximum, as a power of two

// ---------------------------------------------------------------------------
// which units there are
struct Item {
  int r, h, b;         // request, cache head, row block
  int n, kv;           // the request's nodes and length (its nodes' keys among them)
  int units;           // of this item
  int at;              // unit inside the item
  int64_t first;       // global index of the item's first unit
};

__device__ __forceinline__ int request_nodes(const TreeArgs &a, int r) {
  const int lo = max(a.q_start[r], 0), hi = min(a.q_start[r + 1], a.T);
  return max(hi - lo, 0);
}
__device__ __forceinline__ int request_keys(const TreeArgs &a, int r) { return max(a.kv_lens[r], 0); }
// (n G stays below 2^31)
__device__ __forceinline__ int row_blocks(int n, int G, int rows) { return (uint32_t(n) * G + rows - 1) / uint32_t(rows); }

// A request of up to 64 nodes has the same keys for every row block; a longer one is a
// chain, whose row block ends at its last node's own key.  A length may pass the table: the
// keys that the table has no page for are not there, whosever they are.
__device__ __forceinline__ int block_keys(const TreeArgs &a, int n, int kv, int b, int rows) {
  if (n <= kTreeNodes) return min(kv, a.max_keys);
  const int last = min(int((uint32_t(b + 1) * rows - 1) / uint32_t(a.G)), n - 1);
  return min(max(kv - n + last + 1, 0), a.max_keys);
}
__device__ __forceinline__ int block_units(const TreeArgs &a, int n, int kv, int b, int rows) {
  return max((block_keys(a, n, kv, b, rows) + kUnitKeys - 1) / kUnitKeys, 1);
}

// pre[r] = units of the requests before r (R + 1 entries), by a whole workgroup of NT
// threads.  Their sum stays below 2^31 because the requests' tokens do not overlap: where
// q_start falls there are no units at all.  Requests are dealt to the waves in turn.  A
// chain's blocks are counted by its own lane if they are few, else by the whole wave (64
// prompts of 100 tokens, all of them in one wave and that one counting each: 87 us of
// attention, of which 62 are left).
template <int NT>
__device__ __forceinline__ void unit_prefix(const TreeArgs &a, int rows, int *pre, int *red) {
  constexpr int kOwnBlocks = 16, WAVES = NT / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  bool falls = false;
  for (int base = 0; base < a.R; base += NT) {
    const int r = base + WAVES * lane + wave;
    int n = 0, kv = 0, nb = 0, units = 0;
    if (r < a.R) {
      falls |= a.q_start[r + 1] < a.q_start[r];
      n = request_nodes(a, r);
      kv = request_keys(a, r);
      nb = row_blocks(n, a.G, rows);
      if (n <= kTreeNodes) units = nb * block_units(a, n, kv, 0, rows);
      else if (nb <= kOwnBlocks)
        for (int b = 0; b < nb; ++b) units += block_units(a, n, kv, b, rows);
    }
    uint64_t longs = __ballot(n > kTreeNodes && nb > kOwnBlocks);
    while (longs) {
      const int src = __builtin_ctzll(longs);
      longs &= longs - 1;
      const int ln = __builtin_amdgcn_readlane(n, src), lkv = __builtin_amdgcn_readlane(kv, src);
      const int blocks = __builtin_amdgcn_readlane(nb, src);
      int part = 0;
      for (int b = lane; b < blocks; b += 64) part += block_units(a, ln, lkv, b, rows);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) part += __shfl_xor(part, off, 64);
      if (lane == src) units = part;
    }
    if (r < a.R) pre[r + 1] = units * a.H;
  }
  const bool bad = __syncthreads_or(falls);
  const int per = (a.R + NT - 1) / NT, r0 = tid * per;
  int sum = 0;
  for (int j = 0; j < per; ++j)
    if (r0 + j < a.R) pre[r0 + j + 1] = sum += bad ? 0 : pre[r0 + j + 1];  // within this thread so far
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
    it.units = block_units(a, it.n, it.kv, 0, rows);
    it.b = v / it.units;
    v -= it.b * it.units;
  } else {
    const int lane = threadIdx.x & 63, nb = row_blocks(it.n, a.G, rows);
    it.b = 0;
    it.units = 0;
    for (int base = 0; base < nb; base += 64) {
      const int mine = base + lane < nb ? block_units(a, it.n, it.kv, base + lane, rows) : 0;
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

// unit u, or the first of its item if that has `undivided` units at most
__device__ __forceinline__ int whole_from(const TreeArgs &a, int rows, const int *pre, int u, int undivided) {
  const Item it = locate(a, rows, pre, u);
  return __builtin_amdgcn_readfirstlane(it.units <= undivided ? int(it.first) : u);
}

// first unit of workgroup w of W (with fewer units than workgroups some have none)
__device__ __forceinline__ int first_unit(int w, int W, int total) { return int(int64_t(total) * w / W); }
// the workgroup that has unit u, with fewer units than workgroups: one each
__device__ __forceinline__ int only_unit(int u, int W, int total) { return ((u + 1) * W + total - 1) / total - 1; }

// Workgroups are dealt to the eight XCDs in turn: their indices are renamed so that an XCD
// gets neighbouring units, whose row blocks read the same keys from its own L2.
__device__ __forceinline__ int renamed(int id, int W) { return (id & 7) * (W >> 3) + (id >> 3); }

// What the joining kernel has to know of workgroup w's first unit: nothing (parts = 0)
// unless it is the first border between workgroups inside its item.
struct Border {
  int r, h, b, n;
  int slot0, parts;    // the item's partial sums: slot0, then the first ones of the workgroups
  int unit, total;     // that have `unit`, the units after it, ... of `total`
};
__device__ __forceinline__ Border border_of(const Item &it, int w, int W, int total) {
  const int unit = int(it.first) + it.at, u0 = int(it.first), u1 = u0 + it.units;
  Border d = {it.r, it.h, it.b, it.n, 0, 0, unit, total};
  if (it.at == 0) return d;
  const int last = total < W ? only_unit(unit - 1, W, total) : w - 1;  // the workgroup before
  const int before = total < W ? unit - 1 : first_unit(last, W, total);
  if (before > u0) return d;
  d.slot0 = 2 * last + (before == u0 ? 0 : 1);
  int end = u1 - unit;                                 // workgroups to the item's end
  if (total >= W) {
    int e = int(double(u1) * W / total);               // the first whose first unit is u1 or more, or one off
    while (first_unit(e, W, total) < u1) ++e;
    while (first_unit(e - 1, W, total) >= u1) --e;
    end = e - w;
  }
  d.parts = 1 + end;
  return d;
}
__device__ __forceinline__ int slot_of(const Border &d, int part, int w, int W) {
  if (part == 0) return d.slot0;
  return 2 * (d.total < W ? only_unit(d.unit + part - 1, W, d.total) : w + part - 1);
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
  __device__ __forceinline__ void load_k(const char *at) {
#pragma unroll
    for (int c = 0; c < C / 2; ++c) {
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
  // Scores count as powers of two (times scale / ln 2).  m: what the weights are relative to,
  // the running maximum within kSlack; past: how far above m a score may be; -inf (and m = 0)
  // before there is any.  l: the lane's share of the sum.
  float m[RT], past[RT], l[RT];
  __device__ __forceinline__ float top(int t) const { return past[t] < 0.0f ? kNegInf : m[t]; }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = 0.0f;
      past[t] = kNegInf;
      l[t] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][t] = f32x4{0, 0, 0, 0};
    }
  }
};

// A segment: the run of units of one item that a workgroup has; all values are uniform.
struct Segment {
  int r, h, n, kv, blk;
  int ctx, key_end, q0;
  int s0, s1;          // steps
  bool whole, flat;    // the whole item; <= 64 nodes
  int slot;            // of the partial sums
};
__device__ __forceinline__ Segment segment_of(const TreeArgs &a, const Item &it, int rows, int take, int slot) {
  Segment g;
  g.r = __builtin_amdgcn_readfirstlane(it.r);
  g.h = __builtin_amdgcn_readfirstlane(it.h);
  g.n = __builtin_amdgcn_readfirstlane(it.n);
  g.kv = __builtin_amdgcn_readfirstlane(it.kv);
  g.blk = __builtin_amdgcn_readfirstlane(it.b);
  const int at = __builtin_amdgcn_readfirstlane(it.at);
  g.whole = take == __builtin_amdgcn_readfirstlane(it.units);
  g.slot = slot;
  g.flat = g.n <= kTreeNodes;
  g.ctx = g.kv - g.n;
  g.key_end = block_keys(a, g.n, g.kv, g.blk, rows);
  g.q0 = max(a.q_start[g.r], 0);
  g.s0 = at * kUnitSteps;
  g.s1 = max(min((at + take) * kUnitSteps, (g.key_end + kStepKeys - 1) / kStepKeys), g.s0);
  return g;
}

// The rows of a wave: what they see, and their queries as B operands.
template <int D, bool E4M3, int RT>
struct Queries {
  bf16x8 q[D / 32][RT];
  uint64_t sees[RT];   // flat: nodes the row may see
  int node[RT];        // of query row (lane & 15) of row tile t; n or more: there is none

  __device__ __forceinline__ void load(const TreeArgs &a, const Segment &s, int row0, int row16, int g) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = row0 + 16 * t + row16;
      node[t] = row / a.G;
      const bool there = node[t] < s.n;
      const int64_t tok = s.q0 + (there ? node[t] : 0);
      // without a branch that lanes part at: the compiler has been seen to save registers that
      // are needed later at the end of one, before the lanes that stayed away are back
      uint64_t own = ~uint64_t(0) >> ((63 - node[t]) & 63);
      if (a.tree_mask) own = a.tree_mask[tok];         // uniform
      sees[t] = s.flat && there ? own : 0;
      const uint16_t *src = a.q + tok * a.ldq + int64_t(s.h * a.G + (there ? row - node[t] * a.G : 0)) * D;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int d = E4M3 ? 64 * (j >> 1) + 16 * g + 8 * (j & 1) : 32 * j + 8 * g;
        u32x4 v = *reinterpret_cast<const u32x4 *>(src + d);
        if (!there) v = u32x4{0, 0, 0, 0};
        q[j][t] = __builtin_bit_cast(bf16x8, v);
      }
    }
  }

  // which of the lane's eight keys from position `pos` on row tile t sees, if they are there
  __device__ __forceinline__ uint32_t visible(int t, const Segment &s, int pos) const {
    const int j0 = max(pos - s.ctx, -8);               // the node of the first key; further back all are seen
    if (s.flat)
      return (j0 <= -8 ? 255u : j0 < 0 ? uint32_t(sees[t] << -j0) | ((1u << -j0) - 1u)
                                       : j0 < 64 ? uint32_t(sees[t] >> j0) : 0u) & 255u;
    return (1u << min(max(node[t] - j0 + 1, 0), 8)) - 1u;
  }
};

// The tiles of a segment from a step on, in order: page numbers are held 64 at a time in a
// register's lanes, and looked at where a page begins.
struct Pages {
  const int32_t *table;
  int ids, base;       // page numbers base .. base + 63
  int pos;             // of the next tile
  int64_t tile;        // the last tile's first token in the cache; its elements are at D times this
  bool good;           // its page is one

  __device__ __forceinline__ void fetch(const TreeArgs &a, int lane) {
    ids = base + lane < a.table_width ? table[base + lane] : -1;
    asm volatile("" : "+v"(ids));                      // waited for here, not at every use
  }
  __device__ __forceinline__ void enter(const TreeArgs &a, const Segment &s, int lane) {
    int page = (pos >> a.block_shift) - base;
    if (page >= 64) {                                  // uniform
      base += page;
      fetch(a, lane);
      page = 0;
    }
    const int id = __builtin_amdgcn_readlane(ids, page);
    good = uint32_t(id) < uint32_t(a.pages);
    tile = (((good ? int64_t(id) : 0) * a.H + s.h) << a.block_shift) + (pos & ((1 << a.block_shift) - 1)) - 16;
  }
  __device__ __forceinline__ void begin(const TreeArgs &a, const Segment &s, int step, int lane) {
    table = a.table + int64_t(s.r) * a.table_width;
    pos = step * kStepKeys;
    base = pos >> a.block_shift;
    fetch(a, lane);
    enter(a, s, lane);
  }
  // the next tile, and how many of its keys there are (where there are none it is some
  // tile of the cache all the same)
  __device__ __forceinline__ int64_t next(const TreeArgs &a, const Segment &s, int lane, int &lim) {
    if (pos < s.key_end && (pos & ((1 << a.block_shift) - 1)) == 0) enter(a, s, lane);
    const int left = min(s.key_end - pos, 16);
    pos += 16;
    if (left > 0) tile += 16;
    lim = good && left > 0 ? left : 0;
    return left > 0 ? tile : s.h << a.block_shift;     // of page 0
  }
};

// The places of 64 tiles of a segment, a lane each: a step's are two readlanes, so that the
// scalar work between two steps is short.
struct Window {
  int first;           // tile of lane 0
  uint32_t lo, hi;     // first token in the cache (some tile of it where there is none)

  // fills it from tile `from` on, and gives the first of its tiles that lacks a key
  __device__ __forceinline__ int fill(const TreeArgs &a, const Segment &s, int from, int lane) {
    first = from;
    const int pos = (from + lane) * kKvTile, page = pos >> a.block_shift, mask = (1 << a.block_shift) - 1;
    int id = -1;
    if (pos < s.key_end && page < a.table_width) id = a.table[int64_t(s.r) * a.table_width + page];
    const bool good = uint32_t(id) < uint32_t(a.pages);
    const int64_t at = (((good ? int64_t(id) : 0) * a.H + s.h) << a.block_shift) + (good ? pos & mask : 0);
    lo = uint32_t(at);
    hi = uint32_t(at >> 32);
    const uint64_t lacks = __ballot(!good || pos + kKvTile > s.key_end);
    return lacks ? from + __builtin_ctzll(lacks) : 0x7FFFFFFF;
  }
  __device__ __forceinline__ int64_t tile(int i) const {  // i: uniform
    const int at = i - first;
    return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readlane(hi, at))) << 32 | uint32_t(__builtin_amdgcn_readlane(lo, at)));
  }
};

// e4m3: the scales of the lane's eight keys
struct Scales {
  f32x4 k[2], v[2];
  __device__ __forceinline__ void load(const TreeArgs &a, int64_t t0, int64_t t1, int g) {
    const int64_t at = (g < 2 ? t0 : t1) + 8 * (g & 1);
    k[0] = *reinterpret_cast<const f32x4 *>(a.k_scale + at);
    k[1] = *reinterpret_cast<const f32x4 *>(a.k_scale + at + 4);
    v[0] = *reinterpret_cast<const f32x4 *>(a.v_scale + at);
    v[1] = *reinterpret_cast<const f32x4 *>(a.v_scale + at + 4);
  }
  // absent keys' scales are not used; whether one of the others' is not finite (it counts as 0 then)
  __device__ __forceinline__ bool keep_v(uint32_t have) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = have >> i & 1 ? v[i >> 2][i & 3] : 0.0f;
      const bool bad = !(fabsf(x) < __builtin_inff());
      odd |= bad;
      v[i >> 2][i & 3] = bad ? 0.0f : x;
    }
    return odd;
  }
};

// The lane's keys that are there (a bit each) of two tiles with lim0 and lim1 keys.
__device__ __forceinline__ uint32_t present(int lim0, int lim1, int g) {
  const int left = min(max((g < 2 ? lim0 : lim1) - 8 * (g & 1), 0), 8);
  return (1u << left) - 1u;
}

// An operand of V (2-byte elements) without absent keys (a bit of `keep` for each of the
// eight) and without infinities and NaN, whose top bits are gathered in `odd`.
__device__ __forceinline__ bf16x8 clean(bf16x8 x, const uint32_t *keep, uint32_t &odd) {
  u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] &= keep[e];
    const uint32_t b = ((w[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    odd |= b;
    w[e] &= ~((b >> 15) * 0xFFFFu);
  }
  return __builtin_bit_cast(bf16x8, w);
}

// New scores, taken relative to the running maxima: e.  A row's new maximum is taken over,
// rescaling the sums, once it is past the old one by kSlack: weights up to 2^8 are as exact
// as those up to 1, and a maximum still creeps up for long after it is nearly reached (with
// the rescale at every rise a quarter of the steps over 8192 keys had one).  So a lane looks
// at its own eight scores alone, and the four lanes of a row meet only where one of them is
// past it.  (The comparison takes e, not the scores: the compiler passes what comes out of a
// matrix instruction through one more instruction each before it compares.)
template <int D, int RT>
__device__ __forceinline__ void relate(const f32x4 (&s0)[RT], const f32x4 (&s1)[RT], float c2, Rows<D, RT> &acc,
                                       float (&e)[RT][8]) {
  float top[RT];
  bool past = false;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[t][i] = __builtin_fmaf(s0[t][i], c2, -acc.m[t]);
      e[t][4 + i] = __builtin_fmaf(s1[t][i], c2, -acc.m[t]);
    }
    const float *x = e[t];
    top[t] = fmaxf(fmaxf(fmaxf(fmaxf(x[0], x[1]), x[2]), fmaxf(fmaxf(x[3], x[4]), x[5])), fmaxf(x[6], x[7]));
    past |= top[t] > acc.past[t];
  }
  if (!__any(past)) return;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float up = row_max(top[t]);
    const bool none = acc.past[t] < 0.0f, rise = up > (none ? kNegInf : 0.0f);
    const float by = rise ? up : 0.0f, f = none ? 1.0f : __builtin_amdgcn_exp2f(-by);
    acc.l[t] *= f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc.o[j][t] *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) e[t][i] -= by;
    acc.m[t] += by;
    if (rise) acc.past[t] = kSlack;
  }
}
// Relative scores of one row tile to weights: adds to the running sum, and gives the B
// operand of the second product.  zero: a bit for each key whose weight is 0.
template <int D, bool E4M3, int RT, bool MASKED>
__device__ __forceinline__ bf16x8 weigh(float (&e)[8], const f32x4 *vs, int t, Rows<D, RT> &acc, uint32_t &zero) {
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(e[i]);
  acc.l[t] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  if constexpr (MASKED) {
    zero = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) zero |= uint32_t(e[i] == 0.0f) << i;
  }
  if constexpr (E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] *= vs[i >> 2][i & 3];
  }
  return as_operand(pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7]));
}

// An infinity or NaN of a node that some rows do not see must not reach them through
// 0 * inf: the products go without such values, and this adds them key by key where the
// row sees the key.
template <int D, bool E4M3, int RT>
__device__ __forceinline__ void add_not_finite(const TreeArgs &a, int64_t t0, int64_t t1, int lim0, int lim1,
                                               const uint32_t *vis, const uint32_t *zero, int row16, int g,
                                               Rows<D, RT> &acc) {
  constexpr int ES = E4M3 ? 1 : 2;
  for (int kk = 0; kk < kStepKeys; ++kk) {
    const int token = kk & 15;
    if (token >= (kk < 16 ? lim0 : lim1)) continue;
    const int64_t at = kk < 16 ? t0 : t1;
    const char *tile = a.v + (at * D + kv_tile_v(token, 4 * g, ES)) * ES;
    const float scale = E4M3 ? a.v_scale[at + token] : 1.0f;
    const int from = row16 + 16 * (kk >> 3), e = kk & 7;
    float with[RT];                                    // NaN: 0 * inf; 0: not seen
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int on = __shfl(int(vis[t]), from, 64) >> e & 1, none = __shfl(int(zero[t]), from, 64) >> e & 1;
      with[t] = !on ? 0.0f : none ? __builtin_nanf("") : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = v_element<E4M3>(tile, j, i) * scale;
        const bool finite = fabsf(v) < __builtin_inff();
#pragma unroll
        for (int t = 0; t < RT; ++t) acc.o[j][t][i] += finite || with[t] == 0.0f ? 0.0f : with[t] * v;
      }
      __builtin_amdgcn_sched_barrier(0);               // few registers: the loop hardly ever runs
    }
  }
}

// Where a row's results go; `lead` lanes also store its maximum and sum, or its lse.
template <int D, int RT>
struct Results {
  float inv[RT];
  int64_t to[RT];                                      // element offset of the lane's d's, in out or part_o
  bool there[RT];

  __device__ __forceinline__ void begin(const TreeArgs &a, const Segment &s, int rows, int row0, int row16, int g,
                                        const int *node, const float *top, const float *sum, bool lead) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = row0 + 16 * t + row16;
      there[t] = node[t] < s.n;
      inv[t] = !s.whole || sum[t] == 0.0f ? 0.0f : 1.0f / sum[t];
      const int64_t line = s.whole ? int64_t(s.q0 + node[t]) * a.H * a.G + s.h * a.G + (row - node[t] * a.G)
                                   : int64_t(s.slot) * rows + row - s.blk * rows;
      to[t] = line * D + 4 * g;
      if (there[t] && g == 0 && lead) {
        if (!s.whole) {
          a.part_ml[2 * line] = top[t];
          a.part_ml[2 * line + 1] = sum[t];
        } else if (a.lse) {
          a.lse[line] = log_sum(top[t], sum[t]);
        }
      }
    }
  }
  // no key seen: a sum of 0, -inf + log 0.  Scores that are all NaN leave no maximum either,
  // but a sum that is NaN.
  static __device__ __forceinline__ float log_sum(float top, float sum) {
    return (top + __builtin_amdgcn_logf(sum)) * 0.693147180559945309f;
  }
  __device__ __forceinline__ void put(const TreeArgs &a, bool whole, int j, int t, f32x4 v) const {
    if (whole) {
      const uint2 o = {pack2(v[0] * inv[t], v[1] * inv[t]), pack2(v[2] * inv[t], v[3] * inv[t])};
      *reinterpret_cast<uint2 *>(a.out + to[t] + 16 * j) = o;
    } else {
      *reinterpret_cast<f32x4 *>(a.part_o + to[t] + 16 * j) = v;
    }
  }
};

// ---------------------------------------------------------------------------
// few rows: the waves of a workgroup take different keys
template <int D, bool E4M3, int RT>
struct Split {
  static constexpr int rows = 16 * RT;
  // workgroups a compute unit holds, by registers: where it is one, 512 of them a lane; a
  // third one where a step has least to load (64-wide e4m3, 16 trees of 64 over up to 8192
  // keys 92 -> 75 us, 64 of 4 over 500 27 -> 23; in bf16 16 trees of 8 go from 36 to 37)
  static constexpr int occupancy = D * (E4M3 ? 1 : 2) > 256 ? 1 : D == 64 && E4M3 ? 3 : 2;
  static constexpr int grid = 256 * occupancy;
  // the four waves' sums are joined through LDS, up to 64 KB
  static constexpr size_t lds = kWaves * (D / 16) * RT * 1024 + kWaves * 2 * RT * 16 * 4;
  static_assert(fits_lds(lds), "the most requests' prefix sums lie behind it");
};

template <int D, bool E4M3, int RT>
__global__ __launch_bounds__(kThreads, (Split<D, E4M3, RT>::occupancy)) void tree_split_kernel(const TreeArgs a) {
  using S = Split<D, E4M3, RT>;
  constexpr int ROWS = S::rows, QC = D / 32, OC = D / 16, JW = OC / kWaves, W = S::grid;
  constexpr int ES = E4M3 ? 1 : 2;
  extern __shared__ __align__(16) char lds[];
  f32x4 *join = reinterpret_cast<f32x4 *>(lds);        // [wave][OC][RT][64]
  float *stat = reinterpret_cast<float *>(lds + kWaves * OC * RT * 1024);  // [wave][2][RT * 16]
  int *pre = reinterpret_cast<int *>(stat + kWaves * 2 * RT * 16);
  __shared__ int red[kWaves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row16 = lane & 15, g = lane >> 4;
  unit_prefix<kThreads>(a, ROWS, pre, red);
  const int total = __builtin_amdgcn_readfirstlane(pre[a.R]);
  const int w = renamed(blockIdx.x, W);
  const int u_begin = first_unit(w, W, total), u_end = first_unit(w + 1, W, total);
  const float c2 = a.scale * 1.44269504088896340736f;  // scores to powers of two
  if (u_begin == u_end && threadIdx.x == 0) a.borders[8 * w + 5] = 0;

  for (int u = u_begin; u < u_end;) {
    const Item it = locate(a, ROWS, pre, u);
    if (u == u_begin && threadIdx.x == 0) reinterpret_cast<Border *>(a.borders)[w] = border_of(it, w, W, total);
    const int take = min(__builtin_amdgcn_readfirstlane(it.units - it.at), u_end - u);
    const Segment seg = segment_of(a, it, ROWS, take, 2 * w + (u == u_begin ? 0 : 1));
    u += take;
    const int row0 = seg.blk * ROWS;
    Queries<D, E4M3, RT> qs;
    qs.load(a, seg, row0, row16, g);
    // keys that all rows see come first: below `clear` no mask is looked at
    const int clear = seg.flat ? seg.ctx : seg.ctx + min(row0 / a.G + 1, seg.n);
    Rows<D, RT> acc;
    acc.clear();

    const int len = seg.s1 - seg.s0;                   // this wave's steps
    const int s1 = seg.s0 + len * (wave + 1) / kWaves;
    int s = seg.s0 + len * wave / kWaves;
    Pages pages;
    pages.begin(a, seg, s, lane);
    const int k_lane = 256 * g + 16 * (row16 & 7), v_lane = 256 * (g & 1) + 16 * row16;
    // one step, tokens at t0 and t1; the second form looks at masks, at keys that are not
    // there and at values that are not finite, the first knows that all rows see all keys
    auto step = [&](int64_t t0, int64_t t1, [[maybe_unused]] int lim0, [[maybe_unused]] int lim1, auto mask_tag) {
      constexpr bool MASKED = decltype(mask_tag)::value;
      Tiles<D, E4M3> kt, vt;
      Scales sl;
      // all loads are on their way before the first wait
      kt.load_k(a.k + (row16 < 8 ? t0 : t1) * (D * ES) + k_lane);
      if constexpr (E4M3) sl.load(a, t0, t1, g);
      vt.load_v(a.v + (g < 2 ? t0 : t1) * (D * ES) + v_lane);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 sc[2][RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sc[0][t] = sc[1][t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < QC; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 ka = kt.k_operand(i, j);
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[i][t] = mfma(ka, qs.q[j][t], sc[i][t]);
        }
      if constexpr (E4M3) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          sc[0][t] *= sl.k[0];
          sc[1][t] *= sl.k[1];
        }
      }
      [[maybe_unused]] uint32_t vis[RT];               // a bit for each of the lane's eight keys
      [[maybe_unused]] bool rare = false;
      if constexpr (MASKED) {
        const uint32_t have = present(lim0, lim1, g);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          vis[t] = qs.visible(t, seg, s * kStepKeys + 8 * g) & have;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(vis[t] >> i & 1)) sc[i >> 2][t][i & 3] = kNegInf;
        }
        vt.keep_keys(have);
        bool odd = vt.not_finite();
        if constexpr (E4M3) odd |= sl.keep_v(have);
        rare = __any(odd);
        if (rare) vt.drop_not_finite();
      }
      bf16x8 p[RT];
      uint32_t zero[RT];
      float e[RT][8];
      relate(sc[0], sc[1], c2, acc, e);
#pragma unroll
      for (int t = 0; t < RT; ++t) p[t] = weigh<D, E4M3, RT, MASKED>(e[t], sl.v, t, acc, zero[t]);
#pragma unroll
      for (int j = 0; j < OC; ++j) {
        const bf16x8 va = vt.v_operand(j);
#pragma unroll
        for (int t = 0; t < RT; ++t) acc.o[j][t] = mfma(va, p[t], acc.o[j][t]);
      }
      if constexpr (MASKED)
        if (rare) add_not_finite<D, E4M3, RT>(a, t0, t1, lim0, lim1, vis, zero, row16, g, acc);
    };
    // the keys that every row sees; from the first page that is not one, or the first node
    // on, the careful form
    int64_t t0, t1;
    int lim0, lim1;
    for (; s < s1; ++s) {
      t0 = pages.next(a, seg, lane, lim0);
      t1 = pages.next(a, seg, lane, lim1);
      if (s * kStepKeys + kStepKeys > clear || lim0 + lim1 < 32) break;
      step(t0, t1, 16, 16, std::false_type());
    }
    while (s < s1) {
      step(t0, t1, lim0, lim1, std::true_type());
      if (++s == s1) break;
      t0 = pages.next(a, seg, lane, lim0);
      t1 = pages.next(a, seg, lane, lim1);
    }

    // ---- the four waves' sums
    __syncthreads();                                   // the last segment's readers are done
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      acc.l[t] = row_sum(acc.l[t]);
      if (g == 0) {
        stat[(wave * 2 + 0) * RT * 16 + 16 * t + row16] = acc.top(t);
        stat[(wave * 2 + 1) * RT * 16 + 16 * t + row16] = acc.l[t];
      }
    }
    __syncthreads();
    float top[RT], sum[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float mw[kWaves];
      top[t] = kNegInf;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        mw[v] = stat[(v * 2 + 0) * RT * 16 + 16 * t + row16];
        top[t] = fmaxf(top[t], mw[v]);
      }
      sum[t] = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float f = mw[v] == top[t] ? 1.0f : __builtin_amdgcn_exp2f(mw[v] - top[t]);
        sum[t] += f * stat[(v * 2 + 1) * RT * 16 + 16 * t + row16];
      }
      const float f = acc.top(t) == top[t] ? 1.0f : __builtin_amdgcn_exp2f(acc.top(t) - top[t]);
#pragma unroll
      for (int j = 0; j < OC; ++j) acc.o[j][t] *= f;
    }
    Results<D, RT> res;
    res.begin(a, seg, ROWS, row0, row16, g, qs.node, top, sum, wave == 0);
#pragma unroll
    for (int j = 0; j < OC; ++j)
#pragma unroll
      for (int t = 0; t < RT; ++t) join[((wave * OC + j) * RT + t) * 64 + lane] = acc.o[j][t];
    __syncthreads();
#pragma unroll
    for (int jj = 0; jj < JW; ++jj)
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int j = wave * JW + jj;
        f32x4 v = join[(j * RT + t) * 64 + lane];
#pragma unroll
        for (int x = 1; x < kWaves; ++x) v += join[((x * OC + j) * RT + t) * 64 + lane];
        if (res.there[t]) res.put(a, seg.whole, j, t, v);
      }
  }
}

// ---------------------------------------------------------------------------
// many rows: the waves of a workgroup take different rows and share the keys through LDS
template <int D, bool E4M3, int RT>
struct Share {
  // Two workgroups of four waves a compute unit; 256-wide heads, whose steps are twice as
  // long in LDS and whose waves hold 16 rows, have one of eight, which reads memory once for
  // 128 rows (prompt chunk 380 -> 357 us; for 128-wide heads eight waves measured 113 -> 117).
  static constexpr int waves = D == 256 ? 8 : 4;
  static constexpr int threads = 64 * waves;
  static constexpr int rows = 16 * RT * waves;
  // waves a SIMD, by registers: a third one takes 64-wide heads, whose softmax is the longer
  // part of a step, from 396 us to 364 (a prompt of 8192, bf16) and from 550 to 481 (e4m3)
  static constexpr int occupancy = D == 64 ? 3 : 2;
  static constexpr int grid = 1024 * occupancy / waves;
  // Items of up to three units stay whole, with the workgroup that has their last one: the
  // partial sums of 128 rows, written and read again, cost more than a unit (64 trees over
  // 300 keys 59 -> 52 us, a prompt of 300 tokens 34 -> 27, 128-wide heads; eight trees over
  // 350 keys on average 33 -> 35).  With five, four prompts of 500 go from 57 to 42, but
  // eight trees over 350 from 35 to 40 and one over 512 from 22 to 35.
  static constexpr int undivided = 3;
  static constexpr int ring = D == 256 && E4M3 ? 2 : 4;  // steps on their way or in use
  static constexpr int tile = 16 * D * (E4M3 ? 1 : 2); // bytes of a tile in the cache
  static constexpr int units = tile / 1024;            // its 1 KB pieces
  // pieces a wave brings of a step's K and of its V; where there are fewer pieces than waves,
  // the first half of the waves bring K and the others V
  static constexpr bool halves = 2 * units < waves;
  static constexpr int mine = halves ? 1 : 2 * units / waves;
  // The second tile lies 128 bytes off a multiple of the first: lanes 0-7 and 8-15 read
  // one of K each, and would meet in the same 32 of the 64 banks.
  static constexpr int gap = 128;
  static constexpr int raw = 2 * tile + gap;           // bytes of a step of K, or of V, as the cache has it
  static constexpr int wide = 2 * 16 * D * 2 + gap;    // and as bf16
  static constexpr int scales = E4M3 ? waves * 256 : 0;  // of a step, a copy for each wave
  static constexpr size_t lds = ring * (2 * raw + scales) + (E4M3 ? 4 * wide : 0);
  static_assert(fits_lds(lds), "the most requests' prefix sums lie behind it");
  // loads of a wave for a step: what the waits count
  static constexpr int loads = (halves ? 1 : 2) * mine + (E4M3 ? 1 : 0);
};

// s_waitcnt vmcnt(N), the other counters free
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | 0x0F70);
}
// all waves: LDS writes done before are seen after; loads on their way go on
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
__device__ __forceinline__ void load_to_lds16(const char *from, char *to) {  // to: uniform; lane i writes at 16 i
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                   (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// The staging of steps.  K and V have a ring of `ring` steps in LDS, as the cache has them
// ([tile][16 D]), filled by loads that go to LDS directly.  e4m3 steps are widened to bf16
// (in a bf16 cache's order) a turn before they are used.
template <int D, bool E4M3, int RT>
struct Stage {
  using S = Share<D, E4M3, RT>;
  static constexpr int ES = E4M3 ? 1 : 2;
  char *lds;
  int wave, lane;

  __device__ __forceinline__ char *raw_k(int step) const { return lds + (step & (S::ring - 1)) * (2 * S::raw); }
  __device__ __forceinline__ char *raw_v(int step) const { return raw_k(step) + S::raw; }
  __device__ __forceinline__ char *wide_k(int step) const {
    return lds + S::ring * (2 * S::raw + S::scales) + (step & 1) * (2 * S::wide);
  }
  // this wave's scales of a step: [32] of K, [32] of V
  __device__ __forceinline__ char *marks(int step) const {
    return lds + S::ring * 2 * S::raw + (step & (S::ring - 1)) * S::scales + wave * 256;
  }
  __device__ __forceinline__ const char *use_k(int step) const { return E4M3 ? wide_k(step) : raw_k(step); }
  __device__ __forceinline__ const char *use_v(int step) const { return use_k(step) + (E4M3 ? S::wide : S::raw); }

  // this wave's first piece of K or V, or -1: it has none
  template <bool V>
  __device__ __forceinline__ int first() const {
    if constexpr (!S::halves) return wave * S::mine;
    const int p = V ? wave - S::waves / 2 : wave;
    return p >= 0 && p < S::waves / 2 ? p : -1;
  }
  // this wave's pieces of two tiles at t0 and t1
  template <bool V>
  __device__ __forceinline__ void bring(const char *cache, int64_t t0, int64_t t1, char *to) const {
    if (first<V>() < 0) return;
#pragma unroll
    for (int i = 0; i < S::mine; ++i) {
      const int p = first<V>() + i, of = p / S::units, c = p % S::units;
      load_to_lds16(cache + (of ? t1 : t0) * (D * ES) + 1024 * c + 16 * lane, to + of * S::gap + 1024 * p);
    }
  }
  __device__ __forceinline__ void bring(const TreeArgs &a, int step, int64_t t0, int64_t t1) const {
    bring<false>(a.k, t0, t1, raw_k(step));
    bring<true>(a.v, t0, t1, raw_v(step));
    if constexpr (E4M3) {
      const int64_t at = (lane & 16 ? t1 : t0) + (lane & 15);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)((lane < 32 ? a.k_scale : a.v_scale) + at),
          (__attribute__((address_space(3))) void *)marks(step), 4, 0, 0);
    }
  }
  // this wave's pieces of a step, as bf16; only its own loads need to have arrived
  template <bool V>
  __device__ __forceinline__ void widen(const char *from, char *to) const {
    if (first<V>() < 0) return;
#pragma unroll
    for (int i = 0; i < S::mine; ++i) {
      const int p = first<V>() + i, of = p / S::units, c = p % S::units;
      const u32x4 x = *reinterpret_cast<const u32x4 *>(from + of * S::gap + 1024 * p + 16 * lane);
      const u32x4 lo = {e4m3_lo(x[0]), e4m3_hi(x[0]), e4m3_lo(x[1]), e4m3_hi(x[1])};
      const u32x4 hi = {e4m3_lo(x[2]), e4m3_hi(x[2]), e4m3_lo(x[3]), e4m3_hi(x[3])};
      // K: 16 d's of a token are halves of two 32-d pieces; V: 8 tokens of two 16-d tiles,
      // of which a piece has four
      char *dst = to + of * (32 * D + S::gap) + 2048 * c + (V ? 1024 * (lane >> 5) + 16 * (lane & 31) : 16 * lane);
      *reinterpret_cast<u32x4 *>(dst) = lo;
      *reinterpret_cast<u32x4 *>(dst + (V ? 512 : 1024)) = hi;
    }
  }
  __device__ __forceinline__ void widen(int step) const {
    if constexpr (E4M3) {
      widen<false>(raw_k(step), wide_k(step));
      widen<true>(raw_v(step), wide_k(step) + S::wide);
    }
  }
  // until this wave's loads of a step have arrived, `later` further steps being on their way
  __device__ __forceinline__ void arrive(int later) const {
    if (S::ring > 2 && later >= 2) wait_loads<2 * S::loads>();
    else if (S::ring > 2 && later == 1) wait_loads<S::loads>();
    else wait_loads<0>();
  }
};

template <int D, bool E4M3, int RT>
__global__ __launch_bounds__((Share<D, E4M3, RT>::threads), (Share<D, E4M3, RT>::occupancy)) void tree_share_kernel(const TreeArgs a) {
  using S = Share<D, E4M3, RT>;
  using St = Stage<D, E4M3, RT>;
  constexpr int ROWS = S::rows, QC = D / 32, OC = D / 16, W = S::grid;
  static_assert(S::ring <= 4, "arrive() counts two later steps at most");
  static_assert(!S::halves || 4 * S::units == S::waves, "a wave brings whole pieces");
  extern __shared__ __align__(16) char lds[];
  int *pre = reinterpret_cast<int *>(lds + S::lds);
  __shared__ int red[S::waves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row16 = lane & 15, g = lane >> 4;
  const St st = {lds, wave, lane};
  unit_prefix<S::threads>(a, ROWS, pre, red);
  const int total = __builtin_amdgcn_readfirstlane(pre[a.R]);
  const int w = renamed(blockIdx.x, W);
  int u = first_unit(w, W, total), u_end = first_unit(w + 1, W, total);
  if (u < u_end) {
    if (u_end < total) u_end = whole_from(a, ROWS, pre, u_end, S::undivided);
    u = whole_from(a, ROWS, pre, u, S::undivided);
  }
  const int u_begin = u;
  const float c2 = a.scale * 1.44269504088896340736f;
  if (u == u_end && threadIdx.x == 0) a.borders[8 * w + 5] = 0;
  // operands in a step: K of 32 d's number j, tokens of product i; V of 16 d's number j
  const int k_lane = (row16 >> 3) * (32 * D + S::gap) + 256 * g + 16 * (row16 & 7);
  const int v_lane = (g >> 1) * (32 * D + S::gap) + 256 * (g & 1) + 16 * row16;

  while (u < u_end) {
    const Item it = locate(a, ROWS, pre, u);
    if (u == u_begin && threadIdx.x == 0) reinterpret_cast<Border *>(a.borders)[w] = border_of(it, w, W, total);
    const int take = min(__builtin_amdgcn_readfirstlane(it.units - it.at), u_end - u);
    const Segment seg = segment_of(a, it, ROWS, take, 2 * w + (u == u_begin ? 0 : 1));
    u += take;
    const int s1 = seg.s1;
    const int row0 = seg.blk * ROWS + wave * 16 * RT;
    const bool idle = row0 >= seg.n * a.G;             // a wave past the last row only helps to stage
    Queries<D, E4M3, RT> qs;
    qs.load(a, seg, row0, row16, g);
    Rows<D, RT> acc;
    acc.clear();

    // steps before `plain` are seen by all rows, and every key of theirs is there
    int plain = max(seg.flat ? seg.ctx : seg.ctx + min(row0 / a.G + 1, seg.n), 0) / kStepKeys;
    Window ahead;
    plain = min(plain, ahead.fill(a, seg, 2 * seg.s0, lane) >> 1);
    int issued = seg.s0;
    [[maybe_unused]] int ready = seg.s0;               // steps before are in LDS for all waves
    auto bring = [&]() {
      if (2 * issued - ahead.first >= 64) plain = min(plain, ahead.fill(a, seg, 2 * issued, lane) >> 1);
      st.bring(a, issued, ahead.tile(2 * issued), ahead.tile(2 * issued + 1));
      ++issued;
    };
    // what there is room for: all waves are done with the steps before this turn's
    auto refill = [&]() {
      if constexpr (E4M3) {
        if (issued < s1) bring();
      } else {
        while (issued < min(ready + 2, s1)) bring();
      }
    };
    lds_barrier();                                     // the last segment's readers are done
    for (int i = 0; i < (E4M3 ? S::ring - 1 : 2) && issued < s1; ++i) bring();
    if constexpr (E4M3) {
      if (seg.s0 < s1) {
        st.arrive(issued - 1 - seg.s0);
        st.widen(seg.s0);
      }
    }
    // One step.  Operands are read from LDS four at a time, the next four on their way
    // while four are multiplied, and V's first eight while the scores are weighed.
    // Later steps are begun to be brought while the first operands come.
    auto step = [&](int s, int64_t t0, int64_t t1, int lim0, int lim1, auto mask_tag) {
      constexpr bool MASKED = decltype(mask_tag)::value;
      const char *kb = st.use_k(s) + k_lane, *vb = st.use_v(s) + v_lane;
      bf16x8 f[2][4];
      f32x4 sc[2][RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) sc[0][t] = sc[1][t] = f32x4{0, 0, 0, 0};
      auto read_k = [&](int n, bf16x8 (&to)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = *reinterpret_cast<const bf16x8 *>(kb + 1024 * ((4 * n + i) >> 1) + 128 * (i & 1));
      };
      auto read_v = [&](int n, bf16x8 (&to)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = *reinterpret_cast<const bf16x8 *>(vb + 512 * (4 * n + i));
      };
      read_k(0, f[0]);
      if (QC > 2) read_k(1, f[1]);
      else read_v(0, f[1]);
      __builtin_amdgcn_sched_barrier(0);
      refill();
#pragma unroll
      for (int n = 0; n < QC / 2; ++n) {
        if (n > 0) {
          if (n + 1 < QC / 2) read_k(n + 1, f[~n & 1]);
          else read_v(0, f[~n & 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[i & 1][t] = mfma(f[n & 1][i], qs.q[2 * n + (i >> 1)][t], sc[i & 1][t]);
      }
      constexpr int at = (QC / 2) & 1;                 // where V's first four went
      if constexpr (OC > 4) read_v(1, f[~at & 1]);
      Scales sl;
      if constexpr (E4M3) {
        const f32x4 *sp = reinterpret_cast<const f32x4 *>(st.marks(s)) + 2 * g;
        sl.k[0] = sp[0];
        sl.k[1] = sp[1];
        sl.v[0] = sp[8];
        sl.v[1] = sp[9];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          sc[0][t] *= sl.k[0];
          sc[1][t] *= sl.k[1];
        }
      }
      [[maybe_unused]] uint32_t vis[RT], keep[4], odd = 0;
      if constexpr (MASKED) {
        const uint32_t have = present(lim0, lim1, g);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          vis[t] = qs.visible(t, seg, s * kStepKeys + 8 * g) & have;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(vis[t] >> i & 1)) sc[i >> 2][t][i & 3] = kNegInf;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          keep[e] = (have >> (2 * e) & 1 ? 0xFFFFu : 0u) | (have >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
        if constexpr (E4M3) odd = sl.keep_v(have);
      }
      bf16x8 p[RT];
      uint32_t zero[RT];
      float e[RT][8];
      relate(sc[0], sc[1], c2, acc, e);
#pragma unroll
      for (int t = 0; t < RT; ++t) p[t] = weigh<D, E4M3, RT, MASKED>(e[t], sl.v, t, acc, zero[t]);
#pragma unroll
      for (int n = 0; n < OC / 4; ++n) {
        if (n > 0 && n + 1 < OC / 4) read_v(n + 1, f[(n + 1 + at) & 1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bf16x8 va = f[(n + at) & 1][i];
          if constexpr (MASKED) va = clean(va, keep, odd);
#pragma unroll
          for (int t = 0; t < RT; ++t) acc.o[4 * n + i][t] = mfma(va, p[t], acc.o[4 * n + i][t]);
        }
      }
      if constexpr (MASKED)
        if (__any(odd != 0)) add_not_finite<D, E4M3, RT>(a, t0, t1, lim0, lim1, vis, zero, row16, g, acc);
    };
    // A turn: wait for the wave's own pieces; the barrier makes everybody's visible and says
    // that everybody is done with the steps before, whose places are filled again.  bf16
    // takes two steps a turn, with the next two on their way meanwhile (with one step a turn
    // and three on their way a tree batch took 113 us for 109, a prompt chunk 350 to 371 on
    // several cards for 348 to 363); e4m3 takes one, which is widened a turn before.
    auto turn = [&](int s, int64_t t0, int64_t t1, int lim0, int lim1, auto mask_tag) {
      if (E4M3 || s == ready) {
        if constexpr (!E4M3) wait_loads<0>();
        lds_barrier();
        ready = issued;
      }
      if (!idle) step(s, t0, t1, lim0, lim1, mask_tag);
      else refill();
      if constexpr (E4M3) {
        if (s + 1 < s1) {
          st.arrive(issued - 2 - s);
          st.widen(s + 1);
        }
      }
    };
    int s = seg.s0;
    while (s < min(plain, s1)) {
      turn(s, 0, 0, 16, 16, std::false_type());
      ++s;
    }
    // the rest with care: masks, keys that are not there, values that are not finite
    if (s < s1) {
      Pages now;
      now.begin(a, seg, s, lane);
      for (; s < s1; ++s) {
        int lim0, lim1;
        const int64_t t0 = now.next(a, seg, lane, lim0), t1 = now.next(a, seg, lane, lim1);
        turn(s, t0, t1, lim0, lim1, std::true_type());
      }
    }

#pragma unroll
    for (int t = 0; t < RT; ++t) {
      acc.l[t] = row_sum(acc.l[t]);
      acc.m[t] = acc.top(t);
    }
    Results<D, RT> res;
    res.begin(a, seg, ROWS, row0, row16, g, qs.node, acc.m, acc.l, true);
#pragma unroll
    for (int t = 0; t < RT; ++t)
      if (res.there[t]) {
        if (seg.whole) {
#pragma unroll
          for (int j = 0; j < OC; ++j) res.put(a, true, j, t, acc.o[j][t]);
        } else {
#pragma unroll
          for (int j = 0; j < OC; ++j) res.put(a, false, j, t, acc.o[j][t]);
        }
      }
  }
}

// ---------------------------------------------------------------------------
// Adds the partial sums of the items that several workgroups share.  blockIdx.x takes its
// share of the borders between the W main workgroups, of which those that are the first
// inside their item have parts to add; blockIdx.y takes some values of the item's rows.  A
// thread holds four neighbouring values, with four parts on their way at a time.  Where the
// items are few, so that each has many parts, GROUPS = 4 groups of threads take every
// fourth part: a long cache of few heads has over a hundred parts an item, and added in a
// row they took longer than the attention (one request, 4 heads, 65536 keys, 16 rows: 60 us
// in all with one group, 35 with four; sixteen trees over 8192 keys, two or three parts an
// item: 114 with one, 135 with four).
template <int GROUPS>
__global__ __launch_bounds__(GROUPS == 1 ? 256 : 512) void tree_combine_kernel(const TreeArgs a, int rows, int D, int W) {
  constexpr int kJoinGroup = GROUPS == 1 ? 256 : 512 / GROUPS;
  __shared__ f32x4 s_o[GROUPS][GROUPS == 1 ? 1 : kJoinGroup];
  __shared__ float2 s_ml[GROUPS][GROUPS == 1 ? 1 : kJoinGroup];
  const int lane = threadIdx.x & 63, group = threadIdx.x / kJoinGroup, me = threadIdx.x % kJoinGroup;
  const int value = blockIdx.y * (4 * kJoinGroup) + 4 * me, row = value / D, d = value - row * D;
  const Border *borders = reinterpret_cast<const Border *>(a.borders);
  const int end = W / gridDim.x * (blockIdx.x + 1);
  for (int base = W / gridDim.x * blockIdx.x; base < end; base += 64) {
    uint64_t owners = __ballot(base + lane < end && borders[base + lane].parts != 0);
    while (owners) {                                   // the same in every wave
      const int w = base + __builtin_ctzll(owners);
      owners &= owners - 1;
      const Border b = borders[w];
      const uint32_t all = uint32_t(b.b) * rows + row;
      const int node = all / uint32_t(a.G);
      const bool there = row < rows && node < b.n;
      float m = kNegInf, l = 0.0f;
      f32x4 o = {0, 0, 0, 0};
      for (int p = group; there && p < b.parts; p += 4 * GROUPS) {
        float2 ml[4];
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int part = min(p + i * GROUPS, b.parts - 1);
          const int64_t line = int64_t(slot_of(b, part, w, W)) * rows + row;
          ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * line);
          v[i] = *reinterpret_cast<const f32x4 *>(a.part_o + line * D + d);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p + i * GROUPS < b.parts) top = fmaxf(top, ml[i].x);
        const float keep = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
        l *= keep;
        o *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p + i * GROUPS < b.parts) {
            const float f = ml[i].x == top ? 1.0f : __builtin_amdgcn_exp2f(ml[i].x - top);
            l += f * ml[i].y;
            o += f * v[i];
          }
        m = top;
      }
      float top = m;
      if constexpr (GROUPS > 1) {
        s_o[group][me] = o;
        s_ml[group][me] = make_float2(m, l);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) top = fmaxf(top, s_ml[i][me].x);
        l = 0.0f;
        o = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          const float2 x = s_ml[i][me];
          const float f = x.x == top ? 1.0f : __builtin_amdgcn_exp2f(x.x - top);
          l += f * x.y;
          o += f * s_o[i][me];
        }
        __syncthreads();
      }
      if (group == 0 && there) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t at =
            int64_t(max(a.q_start[b.r], 0) + node) * a.H * a.G + b.h * a.G + int(all - uint32_t(node) * a.G);
        const uint2 x = {pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv)};
        *reinterpret_cast<uint2 *>(a.out + at * D + d) = x;
        if (a.lse && d == 0) a.lse[at] = Results<64, 1>::log_sum(top, l);
      }
    }
  }
}

void combine(const TreeArgs &a, int W, int rows, int D, hipStream_t stream) {
  const int64_t items = a.H * (int64_t(a.T) * a.G / rows + a.R);  // there can be
  if (8 * items > W) {
    hipLaunchKernelGGL(tree_combine_kernel<1>, dim3(W, rows * D / 1024), dim3(256), 0, stream, a, rows, D, W);
  } else {
    int X = 8;                                         // columns: a power of two, enough for each item
    while (X < items) X *= 2;
    hipLaunchKernelGGL(tree_combine_kernel<4>, dim3(X, rows * D / 512), dim3(512), 0, stream, a, rows, D, W);
  }
}

template <int D, bool E4M3, int RT>
hipError_t launch_split(const TreeArgs &a, const char *name, hipStream_t stream) {
  using S = Split<D, E4M3, RT>;
  (void)hipGetLastError();
  hipLaunchKernelGGL((tree_split_kernel<D, E4M3, RT>), dim3(S::grid), dim3(kThreads), S::lds + prefix_bytes(a.R),
                     stream, a);
  combine(a, S::grid, S::rows, D, stream);
  set_last_kernel(name);
  return hipGetLastError();
}

template <int D, bool E4M3, int RT>
hipError_t launch_share(const TreeArgs &a, const char *name, hipStream_t stream) {
  using S = Share<D, E4M3, RT>;
  (void)hipGetLastError();
  hipLaunchKernelGGL((tree_share_kernel<D, E4M3, RT>), dim3(S::grid), dim3(S::threads), S::lds + prefix_bytes(a.R),
                     stream, a);
  combine(a, S::grid, S::rows, D, stream);
  set_last_kernel(name);
  return hipGetLastError();
}

// Rows of one cache head in the step's longest request decide the form.  In the split form
// every row of a block sits in each wave and the waves split the keys; blocks of 16 or 32
// rows, of which several read the same keys.  In the share form they share the keys through
// LDS in blocks of 64 or 128 rows.  Split and share, us a call, 8 cache heads (16 requests
// over 8192 keys; 16 over 1024; one over 16384):
//   bf16   64-wide,  64 rows   53  59 | 20 26 | 19 25      128 rows   79  71 | 21 33 | 23 29
//   bf16  128-wide,  32 rows  111 108 | 28 28 | 26 25       64 rows  118 120 | 27 34 | 31 28
//                    48 rows  113 113 | 26 31 | 29 26       96 rows  234 127 | 40 42 | 36 31
//   bf16  256-wide,  32 rows  212 201 | 31 40 | 32 35       64 rows  405 208 | 54 45 | 38 38
//   e4m3   64-wide, 256 rows  154 142 | 39 41 | 33 40
//   e4m3  128-wide, 128 rows  119 133 | 29 50 | 30 39      256 rows  228 219 | 46 59 | 44 51
//   e4m3  256-wide,  32 rows  120 168 | 27 37 | 31 32       48 rows  239 177 | 40 40 | 38 34
// One request over 65536 keys, 128-wide bf16, 64 rows: 86 and 56 with 8 heads, 52 and 39 with 4.
// The rule knows rows, width and type alone, so each border is a balance of these columns:
// bf16 borders lie where many requests over long caches gain, and short caches lose up to a
// third there (64-wide, 128 rows: 33 for 21; 128-wide, 64 rows: 34 for 27); e4m3 ones lie
// where short caches gain, and long ones lose up to 8 % (64-wide, 256 rows: 154 for 142).  The
// longest request speaks for all of a call: a chunk of 512 tokens with 32 single tokens
// beside it, all over 8192 keys, takes 246 us in bf16 (in two calls 300) and 281 in e4m3 (235).
// A step widened to two bytes in LDS for each block costs e4m3 more than bytes read again,
// so its split form goes further.  256-wide heads leave the split form registers for 16
// rows a wave: 32 e4m3 ones are possible with all 512 registers of a lane (113 us for 119),
// but the compiler does not come through there without spilling.
struct Form {
  bool share;
  int tiles, waves;  // of 16 rows a wave; with different rows
};
Form tree_form(int64_t rows, int64_t D, bool e4m3) {
  if (rows <= (D == 256 ? 32 : e4m3 ? 256 : D == 64 ? 64 : 32)) return {false, rows <= 16 || D == 256 ? 1 : 2, 1};
  // 64 rows in blocks of 128 leave half the waves idle: 118 us for 115, over 1024 keys 38 for 35
  return {true, D == 256 || (rows <= 64 && D == 128) ? 1 : 2, D == 256 ? 8 : 4};
}
int form_rows(Form f) { return 16 * f.tiles * f.waves; }

template <int D, bool E4M3>
hipError_t pick(const TreeArgs &a, Form f, hipStream_t stream) {
  if (f.share) {
    if constexpr (D == 128 && !E4M3) {
      if (f.tiles == 1) return launch_share<D, E4M3, 1>(a, "tree_attention_bf16_share64", stream);
    }
    return launch_share<D, E4M3, D == 256 ? 1 : 2>(
        a, E4M3 ? "tree_attention_e4m3_share128" : "tree_attention_bf16_share128", stream);
  }
  if constexpr (D != 256) {
    if (f.tiles == 2)
      return launch_split<D, E4M3, 2>(a, E4M3 ? "tree_attention_e4m3_split32" : "tree_attention_bf16_split32", stream);
  }
  return launch_split<D, E4M3, 1>(a, E4M3 ? "tree_attention_e4m3_split16" : "tree_attention_bf16_split16", stream);
}

// the most workgroups a kernel for width D has
int64_t most_workgroups(int64_t D) { return D == 64 ? 768 : 512; }

}  // namespace

// partial sums of two segments a workgroup, then their maxima and sums, then the borders
size_t tree_workspace_bytes(int64_t max_nodes, int64_t group, int64_t D, bool e4m3) {
  const size_t W = most_workgroups(D);
  return 2 * W * form_rows(tree_form(max_nodes * group, D, e4m3)) * (D + 2) * 4 + W * sizeof(Border);
}

hipError_t launch_tree_attention(TreeArgs a, int64_t D, bool e4m3, int64_t max_nodes, void *workspace,
                                 hipStream_t stream) {
  const Form f = tree_form(max_nodes * a.G, D, e4m3);
  const int64_t lines = 2 * most_workgroups(D) * form_rows(f);
  a.part_o = static_cast<float *>(workspace);
  a.part_ml = a.part_o + lines * D;
  a.borders = reinterpret_cast<int32_t *>(a.part_ml + lines * 2);
  if (e4m3) return D == 64 ? pick<64, true>(a, f, stream) : D == 128 ? pick<128, true>(a, f, stream) : pick<256, true>(a, f, stream);
  return D == 64 ? pick<64, false>(a, f, stream) : D == 128 ? pick<128, false>(a, f, stream) : pick<256, false>(a, f, stream);
}

}  // namespace tl
