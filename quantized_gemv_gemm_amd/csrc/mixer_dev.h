// Device helpers of the operators that keep a state per request (short_conv, delta_rule).
#pragma once

#include "tl_device.h"

namespace tl {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMixerThreads = 256;

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// Whether the requests' starts rise from 0 or more to T or less.  All threads of the
// workgroup call it and get the same answer.
__device__ __forceinline__ bool starts_rise(const int32_t *q_start, int R, int T) {
  bool bad = false;
  for (int r = threadIdx.x; r < R; r += kMixerThreads) {
    const int lo = q_start[r], hi = q_start[r + 1];
    bad |= lo < 0 || hi < lo || hi > T;
  }
  return !__syncthreads_or(bad);
}

// Requests cut into pieces of P tokens.  Piece c of request r has the number
// q_start[r] / P + r + c: no two pieces share one, and all are below T / P + R, which the
// host knows without the lengths.
struct Piece {
  int r, first, n, part;  // request (-1: no piece has this number), its tokens, the piece's place
};
template <int P>
__device__ __forceinline__ Piece find_piece(const int32_t *q_start, int R, int T, int number) {
  int before = 0;
  bool bad = false;
  for (int r0 = 0; r0 < R; r0 += kMixerThreads) {
    const int r = r0 + threadIdx.x;
    bool counts = false;
    if (r < R) {
      const int lo = q_start[r], hi = q_start[r + 1];
      bad |= lo < 0 || hi < lo || hi > T;
      counts = lo / P + r <= number;
    }
    before += __syncthreads_count(counts);
  }
  if (__syncthreads_or(bad) || before == 0) return {-1, 0, 0, 0};
  const int r = before - 1, first = q_start[r], n = q_start[r + 1] - first, part = number - (first / P + r);
  if (int64_t(part) * P >= n) return {-1, 0, 0, 0};
  return {r, first, n, part};
}

// The row of a request's state, or -1 if the request is not served.
__device__ __forceinline__ int state_row(const int32_t *kv_lens, const int32_t *slots, int64_t count, int r) {
  const int s = slots[r];
  return kv_lens[r] > 0 && s >= 0 && s < count ? s : -1;
}

}  // namespace tl
