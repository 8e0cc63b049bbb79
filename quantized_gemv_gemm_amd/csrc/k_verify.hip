// Greedy check of drafted trees against the model's logits.
//
//   target(t) = the lowest index of the largest logit of row t
//   walk: node 0 is given; from node c go to the lowest node whose parent is c and whose
//   drafted token is target(c); accepted = nodes walked, next = target of the last one.
//
// What bounds it is reading the logits once (512 rows of 248320 in bf16: 42 us, 6.1 TB/s,
// where summing a large tensor reaches 5.9, and 4.8 for the walks; 17 rows in f32: 5.8 and
// 4.2 us).  Launch 1 cuts every row into `parts` so that
// a single tree also fills the chip.  A thread compares whole 16-byte loads: the largest of
// their 8 (4) values against its own, and keeps the load that holds it: about 3 operations
// a value, where comparing and remembering each one took 11 and was slower than the memory.
// The place inside the load is looked up once at the end.  Parts
// are joined by 64-bit keys (the logit in an order-preserving integer form above the
// complement of its index), so the largest key is the largest logit and, among equals, the
// lowest index.  -0 counts as +0.  A NaN is larger than every number: the largest
// magnitude, kept beside, tells a thread that it met one, and it looks again one by one.
// Launch 2 is a workgroup a request: its waves join the parts of the nodes, then one walks,
// lane = node, each step one ballot.
#include "kv_layout.h"
#include "tl_device.h"

namespace tl {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((u & 0x7FFFFFFFu) == 0) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// largest of two 16-bit numbers at once
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <bool F32>
struct Load16 {
  static constexpr int E = F32 ? 4 : 8;                  // values
  u32x4 w;
  __device__ __forceinline__ float value(int i) const {  // i: a constant
    if constexpr (F32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ float top() const {         // NaN passed over
    if constexpr (F32) return fmaxf(fmaxf(value(0), value(1)), fmaxf(value(2), value(3)));
    return fmaxf(fmaxf(fmaxf(value(0), value(1)), fmaxf(value(2), value(3))),
                 fmaxf(fmaxf(value(4), value(5)), fmaxf(value(6), value(7))));
  }
  // the largest magnitude, as bits, joined with one of other loads
  __device__ __forceinline__ uint32_t size(uint32_t before) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) before = max(before, w[i] & 0x7FFFFFFFu);
      else before = max_u16x2(before, w[i] & 0x7FFF7FFFu);
    }
    return before;
  }
  static __device__ __forceinline__ bool has_nan(uint32_t size) {
    if constexpr (F32) return size > 0x7F800000u;
    return (size & 0xFFFFu) > 0x7F80u || size >> 16 > 0x7F80u;
  }
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void row_best_kernel(const VerifyArgs a, int64_t part) {
  using L = Load16<F32>;
  constexpr int E = L::E;
  const int64_t row = blockIdx.x / a.parts;
  const int p = int(blockIdx.x - row * a.parts), tid = threadIdx.x;
  const char *base = static_cast<const char *>(a.logits) + row * a.ld * (F32 ? 4 : 2);
  // parts are counted from the row's first 16-byte border, up to E - 1 values in
  const int64_t skip = min(int64_t((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / (F32 ? 4 : 2), a.V);
  const int64_t lo = skip + p * part, hi = min(lo + part, a.V);  // part is a multiple of E
  const u32x4 *src = reinterpret_cast<const u32x4 *>(base + skip * (F32 ? 4 : 2));
  auto one = [&](int64_t i) {
    if constexpr (F32) return reinterpret_cast<const float *>(base)[i];
    else return bf16_bits_to_float(reinterpret_cast<const uint16_t *>(base)[i]);
  };
  auto key_of = [](float f, int64_t i) { return uint64_t(order_key(f)) << 32 | (0xFFFFFFFFu - uint32_t(i)); };

  const int64_t first = lo + int64_t(tid) * E;
  constexpr int64_t kStep = int64_t(kThreads) * E;
  float best = -__builtin_inff();
  int at = 0;                                            // number of the load with the best value, the first of equals
  L with = {};
  uint32_t size = 0;
  int64_t i = first;
  int n = 0;
  for (; i + 3 * kStep + E <= hi; i += 4 * kStep, n += 4) {  // four loads on their way
    L l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) l[j].w = __builtin_nontemporal_load(src + (i - skip + j * kStep) / E);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = l[j].top();
      const bool more = t > best || n + j == 0;
      at = more ? n + j : at;
#pragma unroll
      for (int e = 0; e < 4; ++e) with.w[e] = more ? l[j].w[e] : with.w[e];
      best = fmaxf(best, t);
      size = l[j].size(size);
    }
  }
  for (; i + E <= hi; i += kStep, ++n) {
    const L l = {src[(i - skip) / E]};
    const float t = l.top();
    if (t > best || n == 0) {
      at = n;
      with = l;
    }
    best = fmaxf(best, t);
    size = l.size(size);
  }
  uint64_t key = 0;                                      // below every logit's key
  auto better = [&](uint64_t k) { key = k > key ? k : key; };
  if (L::has_nan(size)) {                                // one by one
    for (int64_t j = first; j + E <= hi; j += kStep)
      for (int e = 0; e < E; ++e) better(key_of(one(j + e), j + e));
  } else if (n > 0) {
    const int64_t j = first + at * kStep;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (with.value(e) == best) better(key_of(best, j + e));
  }
  for (; i < hi; ++i) better(key_of(one(i), i));         // the last few: one thread has them
  if (p == 0 && tid == 0)
    for (int64_t j = 0; j < skip; ++j) better(key_of(one(j), j));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) better(__shfl_xor(key, off, 64));
  __shared__ uint64_t red[kThreads / 64];
  if ((tid & 63) == 0) red[tid >> 6] = key;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) better(red[w]);
    a.best[blockIdx.x] = key;
  }
}

constexpr int kMostParts = 64;  // a lane each

// targets of rows first + wave, + wave + 4, ... below `last`: to(row, target)
template <typename To>
__device__ __forceinline__ void row_targets(const VerifyArgs &a, int first, int last, int wave, int lane, To to) {
  constexpr int kWavesHere = kThreads / 64;
  for (int t = first + wave; t < last; t += 4 * kWavesHere) {  // four rows' loads on their way
    uint64_t best[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = t + j * kWavesHere;
      best[j] = row < last && lane < a.parts ? a.best[int64_t(row) * a.parts + lane] : 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = t + j * kWavesHere;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor(best[j], off, 64);
        best[j] = o > best[j] ? o : best[j];
      }
      if (lane == 0 && row < last) to(row, int(0xFFFFFFFFu - uint32_t(best[j])));
    }
  }
}

// workgroup r < R: request r; workgroup R: the rows that belong to no request
__global__ __launch_bounds__(kThreads) void tree_walk_kernel(const VerifyArgs a) {
  const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (r == a.R) {
    row_targets(a, max(a.q_start[a.R], 0), a.T, wave, lane, [&](int t, int v) { a.target[t] = v; });
    return;
  }
  __shared__ int s_target[kTreeNodes];
  const int first = min(max(a.q_start[r], 0), a.T), last = min(max(a.q_start[r + 1], first), a.T), n = last - first;
  int32_t *path = a.path + int64_t(r) * a.path_width;
  if (n > kTreeNodes) {                                  // a prompt: nothing was drafted
    row_targets(a, first, last, wave, lane, [&](int t, int v) {
      a.target[t] = v;
      if (t == last - 1) a.next[r] = v;
    });
    if (threadIdx.x < a.path_width) path[threadIdx.x] = -1;
    if (threadIdx.x == 0) a.accepted[r] = n;
    return;
  }
  int draft = -1, up = -1;
  if (wave == 0 && lane < n) {
    up = a.parents[first + lane];
    draft = a.draft[first + lane];
  }
  row_targets(a, first, last, wave, lane, [&](int t, int v) { s_target[t - first] = v; });
  __syncthreads();
  if (wave) return;
  const bool there = lane < n;
  const int target = there ? s_target[lane] : -1;
  if (there) a.target[first + lane] = target;
  if (up < 0 || up >= lane || lane == 0) up = -1;
  int cur = n ? 0 : -1, count = 0, at = -1;              // at: the node that lane i's place on the path holds
  while (cur >= 0) {                                     // uniform; rises, so at most n rounds
    if (lane == count) at = cur;
    ++count;
    const int want = __shfl(target, cur, 64);
    const uint64_t fit = __ballot(there && up == cur && draft == want);
    const int next = fit ? __builtin_ctzll(fit) : -1;
    if (next < 0) {
      if (lane == 0) a.next[r] = want;
      break;
    }
    cur = next;
  }
  if (lane == 0) {
    a.accepted[r] = count;
    if (n == 0) a.next[r] = -1;
  }
  if (lane < a.path_width) path[lane] = lane < count ? at : -1;
}

}  // namespace

// Rows in enough parts for eight workgroups a compute unit, each of at least 4096 logits.
int verify_parts(int64_t T, int64_t V) {
  const int64_t wanted = T > 0 ? (2048 + T - 1) / T : 1, most = (V + 4095) / 4096;
  int64_t p = wanted < most ? wanted : most;
  p = p < 1 ? 1 : p > kMostParts ? kMostParts : p;
  return int(p);
}

hipError_t launch_tree_verify(const VerifyArgs &a, bool f32, hipStream_t stream) {
  (void)hipGetLastError();
  const int64_t part = ((a.V + a.parts - 1) / a.parts + 7) / 8 * 8;
  const dim3 grid(unsigned(int64_t(a.T) * a.parts));
  if (a.T) {
    if (f32) hipLaunchKernelGGL(row_best_kernel<true>, grid, dim3(kThreads), 0, stream, a, part);
    else hipLaunchKernelGGL(row_best_kernel<false>, grid, dim3(kThreads), 0, stream, a, part);
  }
  hipLaunchKernelGGL(tree_walk_kernel, dim3(unsigned(a.R + 1)), dim3(kThreads), 0, stream, a);
  set_last_kernel("tree_verify");
  return hipGetLastError();
}

}  // namespace tl
