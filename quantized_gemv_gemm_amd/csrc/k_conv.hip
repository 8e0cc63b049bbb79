// The short causal convolution of a layer that keeps a state: for each channel c and token t
//   y = bias[c] + sum over j < W of w[c, W - 1 - j] x[j tokens back, c],   y <- y / (1 + exp(-y)),
// and the first norm_heads heads of D channels are divided by sqrt(sum of their y^2 + eps).
// "j tokens back" goes along the request (a chain) or along the tree's branch, and past the
// step's first token into the request's state: its last W - 1 rows of x, the oldest first.
//
// A thread holds 8 neighbouring channels of a run of tokens; D / 8 neighbouring lanes hold a head.
// A run keeps the last W - 1 rows in registers, so that each row of x is read once, but for the
// W - 1 before a run; a tree's tokens gather theirs along the branch. Memory bounds it: 8191
// tokens of 10240 channels and 4 taps move 336 MB in 76 us, 4.4 TB/s; without any arithmetic
// between the loads and the stores the same kernel took 75. A prompt's results are stored past
// the L2, which is worth 3 of 82 us where the convolution runs alone. With the delta rule's
// preparation behind it, which reads them, it is not: 70 + 76 us, against 67 + 74 with plain stores.
#include "kv_layout.h"
#include "mixer_dev.h"

namespace tl {
namespace {

constexpr int kThreads = 256;

struct Row8 {
  float v[8];
};
__device__ __forceinline__ Row8 widen(u32x4 w) {
  Row8 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.v[2 * e] = lo_bf16(w[e]);
    x.v[2 * e + 1] = hi_bf16(w[e]);
  }
  return x;
}

// RUN tokens of a run, AHEAD of its rows on their way together
template <int W, int RUN, int AHEAD>
__global__ __launch_bounds__(kThreads) void short_conv_kernel(const ConvArgs a) {
  int part;
  const Request p = find_piece<RUN>(a.q_start, a.kv_lens, a.slots, a.R, a.T, a.state_count, int(blockIdx.x), part);
  if (p.r < 0) return;
  const int c0 = (int(blockIdx.y) * kThreads + threadIdx.x) * 8;
  if (c0 >= a.C) return;                                 // heads are whole: their lanes agree
  const int i0 = part * RUN, count = min(RUN, p.n - i0);
  uint16_t *out = a.out + int64_t(p.first + i0) * a.ldo + c0;
  if (p.row < 0) {
    for (int i = 0; i < count; ++i) *reinterpret_cast<u32x4 *>(out + int64_t(i) * a.ldo) = u32x4{0, 0, 0, 0};
    return;
  }
  const bool tree = a.tree_mask && p.n <= kTreeNodes, fresh = p.fresh;
  uint16_t *state = a.state + int64_t(p.row) * (W - 1) * a.C + c0;
  const uint16_t *x = a.x + int64_t(p.first) * a.ldx + c0;
  auto load_row = [&](int at) -> u32x4 {                 // token `at`, or for at < 0 the state's row at + W - 1
    if (at < 0 && fresh) return u32x4{0, 0, 0, 0};
    return *reinterpret_cast<const u32x4 *>(at >= 0 ? x + int64_t(at) * a.ldx : state + int64_t(at + W - 1) * a.C);
  };
  float w[W][8], bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bias[e] = a.bias ? a.bias[c0 + e] : 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = a.weight[int64_t(c0 + e) * W + j];
  }
  auto finish = [&](float (&y)[8], int i) {              // SiLU, the head's length, rounding
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * y[e]));
      sum = fmaf(y[e], y[e], sum);
    }
    if (c0 < a.norm_channels) {
      for (int off = a.norm_dim / 16; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
      const float by = 1.0f / sqrtf(sum + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= by;
    }
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack_bf16(y[2 * e], y[2 * e + 1]);
    u32x4 *to = reinterpret_cast<u32x4 *>(out + int64_t(i) * a.ldo);
    if (RUN > 16) __builtin_nontemporal_store(o, to);    // a prompt's rows do not stay in the L2 until they are read
    else *to = o;
  };
  if (tree) {
    for (int i = 0; i < count; ++i) {
      const uint64_t word = a.tree_mask[p.first + i0 + i];
      u32x4 raw[W];
      int at = i0 + i;
#pragma unroll
      for (int j = W - 1; j >= 0; --j) {
        raw[j] = load_row(at);
        if (at > 0) {                                    // the nearest ancestor, or the row before the step
          const uint64_t less = word & ((uint64_t(1) << at) - 1);
          at = less ? 63 - __clzll(less) : -1;
        } else {
          --at;
        }
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const Row8 r = widen(raw[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(w[j][e], r.v[e], y[e]);
      }
      finish(y, i);
    }
    return;
  }
  Row8 rows[W - 1 + AHEAD];                             // the last W - 1 rows, and the next ones
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j] = widen(load_row(i0 - (W - 1) + j));
  for (int i = 0; i < count; i += AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) rows[W - 1 + u] = widen(load_row(min(i0 + i + u, p.n - 1)));
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (i + u >= count) break;                         // uniform
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(w[j][e], rows[u + j].v[e], y[e]);
      finish(y, i + u);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j] = rows[AHEAD + j];
  }
  if (i0 == 0) {                                         // the thread that has read the old rows
    u32x4 next[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) next[j] = load_row(p.n - (W - 1) + j);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<u32x4 *>(state + int64_t(j) * a.C) = next[j];
  }
}

template <int W, int RUN, int AHEAD>
hipError_t launch(const ConvArgs &a, hipStream_t stream) {
  const int64_t pieces = int64_t(a.T) / RUN + a.R;
  (void)hipGetLastError();
  hipLaunchKernelGGL((short_conv_kernel<W, RUN, AHEAD>), dim3(unsigned(pieces), unsigned((a.C + 8 * kThreads - 1) / (8 * kThreads))),
                     dim3(kThreads), 0, stream, a);
  set_last_kernel("short_conv");
  return hipGetLastError();
}

// The longest run that leaves two workgroups for each compute unit: long ones read fewer rows
// twice and the weights less often, short ones have fewer rows to wait for.  One request of
// 10240 channels, us, with runs of 4, 16, 32 and 64 tokens: 64 tokens 6.3, 14.3, 23.9, 43; 1024
// 16.6, 18.2, 26, 46; 2048 25.8, 22.2, 27.8, 47; 4096 68, 52, 36, 49; 8191 131, 84, 81, 77.
template <int W>
hipError_t run(const ConvArgs &a, hipStream_t stream) {
  const int64_t groups = (a.C + 8 * kThreads - 1) / (8 * kThreads);
  auto fills = [&](int run) { return a.T / run * groups >= 512; };
  return fills(64)   ? launch<W, 64, 8>(a, stream)
         : fills(32) ? launch<W, 32, 8>(a, stream)
         : fills(16) ? launch<W, 16, 4>(a, stream)
                     : launch<W, 4, 4>(a, stream);
}

}  // namespace

// Shorter runs than 64 are taken only for tokens that 2^15 bounds.
bool conv_fits_grid(int64_t T, int64_t R) { return fits_grid(T / 64 + R, kThreads); }

hipError_t launch_short_conv(const ConvArgs &a, int64_t taps, hipStream_t stream) {
  return taps == 2 ? run<2>(a, stream) : taps == 3 ? run<3>(a, stream) : run<4>(a, stream);
}

}  // namespace tl
