// Block tables, slots, positions and tree masks of a step, from the request lengths.
//
// With bs tokens a page, request r owning owned[r] pages and F free pages from
// free_head on:
//   want  = ceil((ctx + new) / bs),  need = max(0, want - owned)   (0 if want > table width)
//   first = sum of need over the requests before r
//   room = all tokens up to r's last are among the T, or it has neither tokens nor need
//   served = room, want fits the table and (need = 0 or free_head + first + need <= F)
//   table[r, owned + j] = free_list[free_head + first + j]          (served, j < need)
//   slot  = table[r, pos / bs] * bs + pos % bs,  pos = ctx + i for the i-th new token
//   position = ctx + depth(i), mask = bits of i and its ancestors   (trees of <= 64 nodes)
// A request whose last tokens are past the T could not be attended to: its cache length
// would count rows that nobody writes.  Where room or pages end they end for all later
// requests that need any, so the pages that are granted are the first ones of the list.
//
// One launch.  What bounds it is latency: a few dependent loads, whatever the sizes are
// (one tree of 33 nodes 3.9 us, 512 requests with 68000 new tokens 8.6 us; a launch that
// does nothing takes 1.8).
// Every workgroup computes the two prefix sums over the requests for itself (R is small
// and sits in L2) and then takes its share of tokens, so no workgroup waits for another
// and no counter has to be cleared.  A tree is one wavefront: a lane holds a node, and
// six rounds of "my bits |= my parent's bits, my parent = my parent's parent" through
// lane shuffles reach all of 64 ancestors.
#include "kv_layout.h"
#include "tl_device.h"

namespace tl {
namespace {

constexpr int kThreads = 256;

struct Sums {
  int q;         // new tokens before r (saturated at T)
  int64_t need;  // pages before r
};

__device__ __forceinline__ int64_t pages_needed(const StepArgs &a, int ctx, int fresh, int owned, bool &fits) {
  const int64_t want = (int64_t(ctx) + fresh + a.block - 1) / a.block;
  fits = want <= a.table_width;
  return fits ? max(want - owned, int64_t(0)) : 0;
}

__global__ __launch_bounds__(kThreads) void step_plan_kernel(const StepArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int *q_pre = reinterpret_cast<int *>(lds);             // [R + 1]
  int *n_pre = q_pre + a.R + 1;                          // [R + 1], saturated above any free list
  __shared__ int64_t red[2 * kThreads / 64];
  __shared__ int granted;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kWavesHere = kThreads / 64;
  constexpr int64_t kMost = 0x7FFFFFFF;

  const int per = (a.R + kThreads - 1) / kThreads, r0 = tid * per;
  int64_t sq = 0, sn = 0;
  for (int j = 0; j < per && r0 + j < a.R; ++j) {
    bool fits;
    const int fresh = max(a.new_lens[r0 + j], 0);
    sq += fresh;
    sn += pages_needed(a, max(a.ctx_lens[r0 + j], 0), fresh, max(a.owned[r0 + j], 0), fits);
  }
  int64_t iq = sq, in = sn;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t uq = __shfl_up(iq, off, 64), un = __shfl_up(in, off, 64);
    if (lane >= off) {
      iq += uq;
      in += un;
    }
  }
  if (lane == 63) {
    red[wave] = iq;
    red[kWavesHere + wave] = in;
  }
  if (tid == 0) {
    granted = 0;
    q_pre[0] = n_pre[0] = 0;
  }
  __syncthreads();
  int64_t bq = iq - sq, bn = in - sn;
  for (int w = 0; w < wave; ++w) {
    bq += red[w];
    bn += red[kWavesHere + w];
  }
  const int64_t head = *a.free_head;
  const int64_t left = head < 0 ? 0 : max(a.free_count - head, int64_t(0));  // pages there are
  int mine = 0;
  for (int j = 0; j < per && r0 + j < a.R; ++j) {
    const int r = r0 + j;
    bool fits;
    const int fresh = max(a.new_lens[r], 0), ctx = max(a.ctx_lens[r], 0), owned = max(a.owned[r], 0);
    const int64_t need = pages_needed(a, ctx, fresh, owned, fits);
    bq += fresh;
    const bool room = bq <= a.T || (fresh == 0 && need == 0);
    const bool served = fits && room && (need == 0 || bn + need <= left);
    bn += need;
    q_pre[r + 1] = int(min(bq, int64_t(a.T)));
    n_pre[r + 1] = int(min(bn, kMost));
    if (served && need) mine = int(bn);
    if (blockIdx.x == 0) {
      a.q_start[r + 1] = int(min(bq, int64_t(a.T)));
      a.kv_lens[r] = served ? ctx + fresh : 0;
      a.owned_out[r] = owned + (served ? int(need) : 0);
    }
  }
  if (mine) atomicMax(&granted, mine);
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.q_start[0] = 0;
    *a.free_head_out = int(head) + granted;
  }

  // the new pages of the tables
  const int stride = gridDim.x * kThreads;
  for (int p = blockIdx.x * kThreads + tid; p < granted; p += stride) {
    int lo = 0, hi = a.R;                                // n_pre[lo] <= p < n_pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (n_pre[mid] <= p) lo = mid;
      else hi = mid;
    }
    a.table[int64_t(lo) * a.table_width + max(a.owned[lo], 0) + (p - n_pre[lo])] = a.free_list[head + p];
  }

  // slots, and the positions of chains
  for (int t = blockIdx.x * kThreads + tid; t < a.T; t += stride) {
    if (t >= q_pre[a.R]) {
      a.slots[t] = -1;
      a.positions[t] = 0;
      if (a.tree_mask) a.tree_mask[t] = 0;
      continue;
    }
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (q_pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int fresh = max(a.new_lens[lo], 0), ctx = max(a.ctx_lens[lo], 0), owned = max(a.owned[lo], 0);
    bool fits;
    const int64_t need = pages_needed(a, ctx, fresh, owned, fits);
    const int64_t pos = int64_t(ctx) + (t - q_pre[lo]);
    int64_t slot = -1;
    const bool room = int64_t(q_pre[lo]) + fresh <= a.T;
    if (fits && room && (need == 0 || n_pre[lo] + need <= left)) {
      const int64_t page = pos / a.block;
      const int id = page < owned ? a.table[int64_t(lo) * a.table_width + page]
                                  : a.free_list[head + n_pre[lo] + (page - owned)];
      if (id >= 0) slot = int64_t(id) * a.block + (pos - page * a.block);
    }
    a.slots[t] = slot;
    if (!a.tree_mask || fresh > kTreeNodes) {
      a.positions[t] = int(pos);
      if (a.tree_mask) a.tree_mask[t] = 0;
    }
  }

  // trees, a wavefront each
  if (!a.tree_mask) return;
  for (int r = blockIdx.x * kWavesHere + wave; r < a.R; r += gridDim.x * kWavesHere) {
    if (max(a.new_lens[r], 0) > kTreeNodes) continue;
    const int first = q_pre[r], n = q_pre[r + 1] - first, ctx = max(a.ctx_lens[r], 0);
    int up = lane < n ? a.parents[first + lane] : -1;
    if (up < 0 || up >= lane) up = -1;
    uint64_t bits = uint64_t(1) << lane;
#pragma unroll
    for (int round = 0; round < 6; ++round) {
      const int from = max(up, 0);
      const uint64_t theirs = __shfl(bits, from, 64);
      const int further = __shfl(up, from, 64);
      if (up >= 0) {
        bits |= theirs;
        up = further;
      }
    }
    if (lane < n) {
      a.tree_mask[first + lane] = bits;
      a.positions[first + lane] = ctx + __popcll(bits) - 1;
    }
  }
}

}  // namespace

hipError_t launch_step_plan(const StepArgs &a, hipStream_t stream) {
  // a thread a token, or a wavefront a tree, up to one workgroup a compute unit
  const int64_t groups = (int64_t(a.T) + kThreads - 1) / kThreads;
  const int64_t trees = a.tree_mask ? (a.R + kThreads / 64 - 1) / (kThreads / 64) : 0;
  int64_t grid = groups > trees ? groups : trees;
  grid = grid < 1 ? 1 : grid > 256 ? 256 : grid;
  (void)hipGetLastError();
  hipLaunchKernelGGL(step_plan_kernel, dim3(unsigned(grid)), dim3(kThreads), size_t(a.R + 1) * 8, stream, a);
  set_last_kernel("step_plan");
  return hipGetLastError();
}

}  // namespace tl
