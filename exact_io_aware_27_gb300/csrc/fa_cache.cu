// Rows of new keys and values into a paged cache: token t of request i goes to cache
// position starts[i] + t - cu_seqlens[i], which is row (position mod page) of page
// table[i, position / page].
//
// Memory bound: every row is read once and written once, 16 bytes a thread. A block
// takes kTokens tokens: its first threads look the tokens' places up (a binary search
// over the bounds, then the table), then all threads copy, K and V of up to four
// chunks in flight each. A place out of range is not written and raises
// kDeviceIndexBit; so do bounds that are not 0 = cu[0] <= ... <= cu[nseq] <= total, which
// the other threads look at meanwhile, each block at its share. Whatever the bounds are, a
// row goes only to a request in whose bounds it lies.
#include "fa_decode.h"
#include "fa_launch.h"
#include "sm103.cuh"

namespace fa {

__device__ unsigned int g_append_status;

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;

struct AppendParams {
  const uint4 *K, *V;
  long long ldk, ldv;  // 16-byte units
  const int *cu, *starts, *table;
  uint4 *Kc, *Vc;
  int total, nseq, Hkv, per_row, max_pages, num_pages, page, page_shift;  // per_row: d / 8
};

__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  __shared__ long long place[kTokens];  // first 16-byte unit of the token's row of head 0
  const int per = p.Hkv * p.per_row;    // 16-byte units of a token
  const long long head = (long long)p.page * p.per_row;  // units from head to head
  grid_wait();
  grid_launch_dependents();
  if (threadIdx.x >= 32) {  // the threads that have no token to look up
    constexpr int n = kThreads - 32;
    const int me = threadIdx.x - 32;
    bool bad = false;
    for (long long i = (long long)blockIdx.x * n + me; i < p.nseq; i += (long long)gridDim.x * n)
      bad |= p.cu[i] > p.cu[i + 1];
    if (blockIdx.x == 0 && me == 0) bad |= p.cu[0] != 0 || p.cu[p.nseq] > p.total;
    if (bad) atomicOr(&g_append_status, kDeviceIndexBit);
  }
  for (long long t0 = (long long)blockIdx.x * kTokens; t0 < p.total;
       t0 += (long long)gridDim.x * kTokens) {
    if (threadIdx.x < kTokens) {
      const int t = (int)t0 + threadIdx.x;
      long long at = -1;
      if (t < p.total && t < p.cu[p.nseq]) {  // rows behind the last request are skipped
        int lo = 0, hi = p.nseq;  // t < cu[hi]; cu[lo] <= t, or lo = 0
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.cu[mid] <= t)
            lo = mid;
          else
            hi = mid;
        }
        const long long pos = (long long)p.starts[lo] + t - p.cu[lo];
        int page = -1;
        if (p.starts[lo] >= 0 && p.cu[lo] <= t && p.cu[lo] >= 0 &&
            pos < (long long)p.max_pages << p.page_shift)
          page = p.table[(long long)lo * p.max_pages + (pos >> p.page_shift)];
        if (page >= 0 && page < p.num_pages)
          at = ((long long)page * p.Hkv << p.page_shift) * p.per_row +
               (pos & (p.page - 1)) * p.per_row;
        else
          atomicOr(&g_append_status, kDeviceIndexBit);
      }
      place[threadIdx.x] = at;
    }
    __syncthreads();
    const int n = kTokens * per;
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * kThreads) {
      uint4 k[4], v[4];
      long long to[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kThreads;
        const int tok = i / per, c = i - tok * per;
        to[u] = i < n ? place[tok] : -1;
        if (to[u] >= 0) {
          const int h = c / p.per_row;
          to[u] += h * head + (c - h * p.per_row);
          k[u] = ld_stream16(p.K + (t0 + tok) * p.ldk + c);
          v[u] = ld_stream16(p.V + (t0 + tok) * p.ldv + c);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (to[u] >= 0) {
          p.Kc[to[u]] = k[u];
          p.Vc[to[u]] = v[u];
        }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  AppendParams p;
  p.K = static_cast<const uint4*>(a.K);
  p.V = static_cast<const uint4*>(a.V);
  p.ldk = a.ldk / 8;
  p.ldv = a.ldv / 8;
  p.cu = a.cu_seqlens;
  p.starts = a.starts;
  p.table = a.table;
  p.Kc = static_cast<uint4*>(a.Kc);
  p.Vc = static_cast<uint4*>(a.Vc);
  p.total = a.total;
  p.nseq = a.nseq;
  p.Hkv = a.Hkv;
  p.per_row = a.d / 8;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.page = a.page;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  const unsigned blocks = (unsigned)ceil_div(a.total, kTokens);
  return launch_early(append_kernel, blocks, kThreads, 0, s, p);
}

cudaError_t append_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_append_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_append_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
