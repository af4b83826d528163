// Plans of packed batches: from cu_seqlens on the device to the work lists of the
// forward and backward passes, without a host synchronisation.
//
// A sequence of length n has ceil(n / rows) tiles of `rows` rows. The persistent kernels
// deal a list out in snake order, which balances only a list whose heaviest entries
// come first, so the lists are sorted by cost: under causal masking tile t of a query
// list costs t + 1 and key block t costs (blocks - t); without it every tile costs its
// sequence's length. A counting sort over at most 1024 cost classes is enough (the
// order inside a class does not matter, and no result depends on the order of a list).
//
// One block of 1024 threads: a plan serves every layer that runs the batch. Bound by the
// latency of its passes over the lists: 9 to 11 us up to 32768 rows, 66 us for 2^20 rows in 8
// sequences, 211 us for 2^20 in 4096.
// Bounds that are not 0 = cu[0] <= cu[1] <= ... <= cu[nseq] <= total give empty
// lists and raise kDeviceIndexBit.
#include "fa_launch.h"
#include "fa_packed.h"
#include "sm103.cuh"

namespace fa {

__device__ unsigned int g_plan_status;

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 1024;

// Exclusive scan of one value per thread over the block; `total` gets the sum.
__device__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Last i with first[i] <= x, for first[0] = 0 <= ... <= first[n] and x < first[n].
__device__ int find_sequence(const int* first, int n, int x) {
  int lo = 0, hi = n;  // first[lo] <= x < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const int* cu, int nseq,
                                                        int total, int causal, uint8_t* plan,
                                                        PlanLayout lay) {
  __shared__ int warp_sums[32];
  __shared__ int bins[kBins];
  __shared__ int longest_seq;
  const int tid = threadIdx.x;
  PlanHead* head = reinterpret_cast<PlanHead*>(plan);
  grid_wait();
  grid_launch_dependents();

  int bad = 0;
  for (int i = tid; i < nseq; i += kThreads) bad |= cu[i] > cu[i + 1] ? 1 : 0;
  if (tid == 0) {
    bad |= (cu[0] != 0 || cu[nseq] > total) ? 1 : 0;
    longest_seq = 0;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      *head = PlanHead{kPlanMagic, total, nseq, total, 0, 0, 0, 0, {}};
      atomicOr(&g_plan_status, kDeviceIndexBit);
    }
    return;
  }

  // Tiles before each sequence, for the tiles of 256, 128, 64 and 32 rows.
  int* first = reinterpret_cast<int*>(plan + lay.off_scan);  // [4][nseq + 1]
  int tiles[4] = {0, 0, 0, 0}, longest = 0;
  for (int base = 0; base < nseq; base += kThreads) {
    const int i = base + tid;
    const int len = i < nseq ? cu[i + 1] - cu[i] : 0;
    longest = max(longest, len);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rows = plan_tile_rows(k);
      int sum;
      const int before = block_scan((len + rows - 1) / rows, warp_sums, sum);
      if (i < nseq) first[k * (nseq + 1) + i] = tiles[k] + before;
      tiles[k] += sum;
    }
  }
  atomicMax(&longest_seq, longest);
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) first[k * (nseq + 1) + nseq] = tiles[k];
    *head = PlanHead{kPlanMagic, total, nseq, cu[nseq], tiles[0], tiles[1], tiles[2], tiles[3], {}};
  }
  __syncthreads();
  const int* first128 = first + (nseq + 1);

  for (int list = 0; list < kPlanLists; ++list) {
    const int rows = plan_tile_rows(list);
    const int* mine = list == kKeyList ? first128 : first + list * (nseq + 1);
    const int n = mine[nseq];
    PlanTile* out = reinterpret_cast<PlanTile*>(plan + lay.off[list]);
    const int most = (longest_seq + rows - 1) / rows;
    int shift = 0;
    while ((most >> shift) >= kBins) ++shift;
    auto entry = [&](int i, int& bin) {
      const int s = find_sequence(mine, nseq, i);
      const int start = cu[s], len = cu[s + 1] - start, tile = i - mine[s];
      const int all = mine[s + 1] - mine[s];
      // in tiles, 1 <= cost <= most
      const int cost = !causal ? all : list == kKeyList ? all - tile : tile + 1;
      bin = (most - cost) >> shift;
      return make_int4(start, len, tile, first128[s] * kWorkspaceRowAlign);
    };
    bins[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      int bin;
      entry(i, bin);
      atomicAdd(&bins[bin], 1);
    }
    __syncthreads();
    int sum;
    const int at = block_scan(bins[tid], warp_sums, sum);
    bins[tid] = at;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      int bin;
      const PlanTile e = entry(i, bin);
      out[atomicAdd(&bins[bin], 1)] = e;
    }
    __syncthreads();
  }
}
static_assert(kBins == kThreads, "one cost class per thread in the scan");
static_assert(kWorkspaceRowAlign == 128, "workspace rows are counted in 128-row tiles");

}  // namespace

cudaError_t launch_packed_plan(const int* cu_seqlens, int nseq, int total, int causal, void* plan,
                               cudaStream_t s) {
  return launch_early(plan_kernel, 1, kThreads, 0, s, cu_seqlens, nseq, total, causal,
                      static_cast<uint8_t*>(plan), plan_layout(nseq, total));
}

cudaError_t plan_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_plan_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_plan_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
