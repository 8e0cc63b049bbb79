// Device helpers of the operators that keep a state per request (short_conv, delta_rule).
#pragma once

#include "tl_device.h"

namespace tl {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// What a workgroup has to know of a request: its first token and their number, the row of its
// state (-1: it is not served), and whether it has just begun.
struct Request {
  int r, first, n, row;
  bool fresh;
};
constexpr Request kNoRequest = {-1, 0, 0, -1, false};

__device__ __forceinline__ Request request_at(int r, int lo, int hi, int kv, int slot, int64_t states) {
  return {r, lo, hi - lo, kv > 0 && slot >= 0 && slot < states ? slot : -1, kv <= hi - lo};
}

// Request r, or none (r = -1) where the starts do not rise from 0 or more to T or less.  All
// threads of the workgroup call it and get the same answer; up to 64 requests each wave looks at
// all starts for itself, with one round of loads and no barrier.
__device__ __forceinline__ Request request_of(const int32_t *q_start, const int32_t *kv_lens, const int32_t *slots, int R,
                                              int T, int64_t states, int r) {
  const Request q = request_at(r, q_start[r], q_start[r + 1], kv_lens[r], slots[r], states);
  bool bad = false;
  const int step = R <= 64 ? 64 : int(blockDim.x);
  for (int j = R <= 64 ? threadIdx.x & 63 : threadIdx.x; j < R; j += step) {
    const int lo = q_start[j], hi = q_start[j + 1];
    bad |= lo < 0 || hi < lo || hi > T;
  }
  const bool any = R <= 64 ? __any(bad) : __syncthreads_or(bad);
  return any ? kNoRequest : q;
}

// Requests cut into pieces of P tokens.  Piece c of request r has the number
// q_start[r] / P + r + c: no two pieces share one, and all are below T / P + R, which the
// host knows without the lengths.  Returns the piece's request (r = -1 if no piece has this
// number, or the starts do not rise) and its place in it.
template <int P>
__device__ __forceinline__ Request find_piece(const int32_t *q_start, const int32_t *kv_lens, const int32_t *slots, int R,
                                              int T, int64_t states, int number, int &part) {
  Request q = kNoRequest;
  if (R <= 64) {
    const int r = threadIdx.x & 63;
    int lo = 0, hi = 0, kv = 0, slot = -1;
    if (r < R) lo = q_start[r], hi = q_start[r + 1], kv = kv_lens[r], slot = slots[r];
    const bool bad = r < R && (lo < 0 || hi < lo || hi > T);
    const uint64_t at = __ballot(r < R && lo / P + r <= number);
    if (__any(bad) || at == 0) return q;
    const int from = 63 - __clzll(at);
    auto of = [&](int x) { return __builtin_amdgcn_readlane(x, from); };
    q = request_at(from, of(lo), of(hi), of(kv), of(slot), states);
  } else {
    int before = 0;
    bool bad = false;
    for (int r0 = 0; r0 < R; r0 += int(blockDim.x)) {
      const int r = r0 + threadIdx.x;
      bool counts = false;
      if (r < R) {
        const int lo = q_start[r], hi = q_start[r + 1];
        bad |= lo < 0 || hi < lo || hi > T;
        counts = lo / P + r <= number;
      }
      before += __syncthreads_count(counts);
    }
    if (__syncthreads_or(bad) || before == 0) return q;
    const int r = before - 1;
    q = request_at(r, q_start[r], q_start[r + 1], kv_lens[r], slots[r], states);
  }
  part = number - (q.first / P + q.r);
  return int64_t(part) * P < q.n ? q : kNoRequest;
}

}  // namespace tl
