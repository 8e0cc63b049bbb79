// Greedy check of drafted trees against the model's logits.
//
//   target(t) = the lowest index of the largest logit of row t
//   walk: node 0 is given; from node c go to the lowest node whose parent is c and whose
//   drafted token is target(c); accepted = nodes walked, next = target of the last one.
//
// What bounds it is reading the logits once.  Launch 1 cuts every row into `parts` so
// that a single tree also fills the chip; a thread keeps one running maximum as a 64-bit
// key (the logit in an order-preserving integer form above the complement of its index),
// so the largest key is the largest logit and, among equals, the lowest index, in any
// order of comparison.  -0 counts as +0, and a NaN as larger than every number.
// Launch 2 is a wavefront a request: lane = node, each step of the walk one ballot.
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

__device__ __forceinline__ void better(uint32_t &key, uint32_t &at, uint32_t k, uint32_t i) {
  if (k > key) {  // a thread meets its indices in rising order: the first of equals stays
    key = k;
    at = i;
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void row_best_kernel(const VerifyArgs a, int64_t part) {
  const int64_t row = blockIdx.x / a.parts;
  const int p = int(blockIdx.x - row * a.parts), tid = threadIdx.x;
  constexpr int E = F32 ? 4 : 8;                         // elements of a 16-byte load
  const char *base = static_cast<const char *>(a.logits) + row * a.ld * (F32 ? 4 : 2);
  // parts are counted from the row's first 16-byte border, up to E - 1 elements in
  const int64_t skip = min(int64_t((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / (F32 ? 4 : 2), a.V);
  const int64_t lo = skip + p * part, hi = min(lo + part, a.V);  // part is a multiple of E
  uint32_t key = 0, at = 0;                              // below every logit's key
  auto look = [&](u32x4 w, int64_t i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (F32) {
        better(key, at, order_key(__uint_as_float(w[e])), uint32_t(i + e));
      } else {
        better(key, at, order_key(__uint_as_float(w[e] << 16)), uint32_t(i + 2 * e));
        better(key, at, order_key(__uint_as_float(w[e] & 0xFFFF0000u)), uint32_t(i + 2 * e + 1));
      }
    }
  };
  auto look_one = [&](int64_t i) {
    float f;
    if constexpr (F32) f = reinterpret_cast<const float *>(base)[i];
    else f = bf16_bits_to_float(reinterpret_cast<const uint16_t *>(base)[i]);
    better(key, at, order_key(f), uint32_t(i));
  };
  if (p == 0 && tid == 0)
    for (int64_t i = 0; i < skip; ++i) look_one(i);
  const u32x4 *src = reinterpret_cast<const u32x4 *>(base + skip * (F32 ? 4 : 2));
  int64_t i = lo + int64_t(tid) * E;
  constexpr int64_t kStep = int64_t(kThreads) * E;
  for (; i + 3 * kStep + E <= hi; i += 4 * kStep) {      // four loads in flight
    u32x4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __builtin_nontemporal_load(src + (i - skip + j * kStep) / E);
#pragma unroll
    for (int j = 0; j < 4; ++j) look(w[j], i + j * kStep);
  }
  for (; i + E <= hi; i += kStep) look(src[(i - skip) / E], i);
  for (; i < hi; ++i) look_one(i);                       // the last few: one thread has them
  uint64_t best = uint64_t(key) << 32 | (0xFFFFFFFFu - at);
  if (key == 0) best = 0;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor(best, off, 64);
    best = o > best ? o : best;
  }
  __shared__ uint64_t red[kThreads / 64];
  if ((tid & 63) == 0) red[tid >> 6] = best;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) best = red[w] > best ? red[w] : best;
    a.best[blockIdx.x] = best;
  }
}

__device__ __forceinline__ int row_target(const VerifyArgs &a, int t) {
  uint64_t best = 0;
  for (int p = 0; p < a.parts; ++p) {
    const uint64_t o = a.best[int64_t(t) * a.parts + p];
    best = o > best ? o : best;
  }
  return int(0xFFFFFFFFu - uint32_t(best));
}

// workgroup r < R: request r; workgroup R: the rows that belong to no request
__global__ __launch_bounds__(64) void tree_walk_kernel(const VerifyArgs a) {
  const int r = blockIdx.x, lane = threadIdx.x;
  if (r == a.R) {
    for (int t = max(a.q_start[a.R], 0) + lane; t < a.T; t += 64) a.target[t] = row_target(a, t);
    return;
  }
  const int first = min(max(a.q_start[r], 0), a.T), last = min(max(a.q_start[r + 1], first), a.T), n = last - first;
  int32_t *path = a.path + int64_t(r) * a.path_width;
  if (n > kTreeNodes) {                                  // a prompt: nothing was drafted
    for (int i = lane; i < n; i += 64) {
      const int v = row_target(a, first + i);
      a.target[first + i] = v;
      if (i == n - 1) a.next[r] = v;
    }
    if (lane < a.path_width) path[lane] = -1;
    if (lane == 0) a.accepted[r] = n;
    return;
  }
  const bool there = lane < n;
  int target = -1, draft = -1, up = -1;
  if (there) {
    up = a.parents[first + lane];
    draft = a.draft[first + lane];
    target = row_target(a, first + lane);
    a.target[first + lane] = target;
  }
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

// Rows in enough parts for four workgroups a compute unit, each of at least 4096 logits.
int verify_parts(int64_t T, int64_t V) {
  const int64_t wanted = T > 0 ? (1024 + T - 1) / T : 1, most = (V + 4095) / 4096;
  const int64_t p = wanted < most ? wanted : most;
  return int(p < 1 ? 1 : p);
}

hipError_t launch_tree_verify(const VerifyArgs &a, bool f32, hipStream_t stream) {
  (void)hipGetLastError();
  const int64_t part = ((a.V + a.parts - 1) / a.parts + 7) / 8 * 8;
  const dim3 grid(unsigned(int64_t(a.T) * a.parts));
  if (a.T) {
    if (f32) hipLaunchKernelGGL(row_best_kernel<true>, grid, dim3(kThreads), 0, stream, a, part);
    else hipLaunchKernelGGL(row_best_kernel<false>, grid, dim3(kThreads), 0, stream, a, part);
  }
  hipLaunchKernelGGL(tree_walk_kernel, dim3(unsigned(a.R + 1)), dim3(64), 0, stream, a);
  set_last_kernel("tree_verify");
  return hipGetLastError();
}

}  // namespace tl
