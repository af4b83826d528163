// The backward pass over packed sequences: the gradient kernel (fa_backward.cuh) over
// Q, dO [total, Hq, d] and K, V [total, Hkv, d], and its preprocess kernel.
//
// Blocks are 128-row tiles of the sequences, from the plan's lists. A key block of a
// key/value head runs over the queries of all Hq / Hkv query heads that read it, so
// that dK and dV are summed on chip, in a fixed order, and written once. The statistics
// -D and -L * log2(e) lie in a workspace in which every sequence starts on a multiple of
// 128 rows: TMA copies of fp32 rows have to start on 16-byte boundaries, which a
// sequence's first row in the packed tensors need not do.
#include "fa_backward.cuh"
#include "fa_launch.h"
#include "fa_packed.cuh"

namespace fa {

__device__ unsigned int g_packed_bwd_status;

namespace {

struct PackedBwd {
  struct Params {
    const uint8_t* plan;
    long long off_kv, off_q;  // the lists' places in the plan
    __nv_bfloat16 *dQ, *dK, *dV;
    long long lddq, lddk, lddv;
    const float *nD, *nL2;
    long long ws_rows;
    int total, nseq, Hq, Hkv, per_kv, causal, kgroup, qgroup, fill, trigger;
  };
  struct View {
    const Params& p;
    int tiles, covered;
  };
  struct KvItem {
    PlanTile s;  // sequence start, length, tile, first workspace row
    int hk;
  };
  struct QItem {
    PlanTile s;
    int h;
  };
  static constexpr bool kEarly = true;
  static constexpr bool kForeignTail = true;
  FA_DEV static unsigned int* status() { return &g_packed_bwd_status; }
  FA_DEV static bool trigger(const Params& p) { return p.trigger; }
  FA_DEV static View view(const Params& p) {
    const PlanHead* head = reinterpret_cast<const PlanHead*>(p.plan);
    const bool ok = plan_matches(head, p.total, p.nseq, status());
    return {p, ok ? head->tiles128 : 0, ok ? head->covered : p.total};
  }
  FA_DEV static int causal(const View& g) { return g.p.causal; }
  FA_DEV static int heads(const View& g) { return g.p.per_kv; }
  FA_DEV static int kv_items(const View& g) { return g.tiles * g.p.Hkv; }
  FA_DEV static int q_items(const View& g) { return g.tiles * g.p.Hq; }

  FA_DEV static KvItem kv_item(const View& g, int i) {
    int rank, hk;
    grouped_tile(i, g.p.Hkv, g.tiles, g.p.kgroup, rank, hk);
    return {__ldg(reinterpret_cast<const PlanTile*>(g.p.plan + g.p.off_kv) + rank), hk};
  }
  FA_DEV static int first_key(const KvItem& it) { return it.s.z * 128; }
  FA_DEV static int rows(const View&, const KvItem& it) { return it.s.y; }
  FA_DEV static int keys(const View&, const KvItem& it) { return it.s.y; }
  FA_DEV static int kv_halves(const View& g, const KvItem& it, int& q_first) {
    q_first = g.p.causal ? it.s.z * 128 : 0;
    return (it.s.y - q_first + 63) / 64;
  }
  FA_DEV static void load_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                               const View&, const KvItem& it) {
    tma_load_3d(dst, map, f, col, it.hk, it.s.x + it.s.z * 128);
  }
  FA_DEV static void load_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                  const View& g, const KvItem& it, int hd, int q) {
    tma_load_3d(dst, map, f, col, it.hk * g.p.per_kv + hd, it.s.x + q);
  }
  FA_DEV static void load_stats(void* dst, const CUtensorMap* map, uint64_t* f, const View& g,
                                const KvItem& it, int hd, int q) {
    tma_load_2d(dst, map, f, it.s.w + q, it.hk * g.p.per_kv + hd);
  }
  template <int D>
  FA_DEV static void store_keys(const View& g, const KvItem& it, int w, int warp, uint32_t col,
                                float mul, uint8_t* stage, const CUtensorMap* map, int d) {
    const int key = it.s.z * 128 + warp * 32;
    packed_rows_store<D>(col, mul, stage, map, it.hk, it.s.x + key, it.s.y - key, 0, d,
                         w == 0 ? g.p.dV : g.p.dK, w == 0 ? g.p.lddv : g.p.lddk);
  }
  template <int D>
  FA_DEV static void zero_key(const View&, const KvItem&, int, int, int) {}  // every key is seen

  FA_DEV static QItem q_item(const View& g, int i) {
    int rank, h;
    grouped_tile(i, g.p.Hq, g.tiles, g.p.qgroup, rank, h);
    return {__ldg(reinterpret_cast<const PlanTile*>(g.p.plan + g.p.off_q) + rank), h};
  }
  FA_DEV static int first_query(const QItem& it) { return it.s.z * 128; }
  FA_DEV static int keys(const View&, const QItem& it) { return it.s.y; }
  FA_DEV static int key_blocks(const View& g, const QItem& it) {
    return g.p.causal ? it.s.z + 1 : (it.s.y + 127) / 128;
  }
  FA_DEV static void load_block_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                        const View&, const QItem& it, int row) {
    tma_load_3d(dst, map, f, col, it.h, it.s.x + it.s.z * 128 + row);
  }
  FA_DEV static void load_block_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                     const View& g, const QItem& it, int key) {
    tma_load_3d(dst, map, f, col, it.h / g.p.per_kv, it.s.x + key);
  }
  FA_DEV static void query_stats(const View& g, const QItem& it, int r, float& nl2, float& nd) {
    const size_t row = (size_t)it.h * g.p.ws_rows + it.s.w + it.s.z * 128 + r;
    nl2 = g.p.nL2[row];
    nd = g.p.nD[row];
  }
  template <int NCOL>
  FA_DEV static void store_queries(const View& g, const QItem& it, int warp, uint32_t tcol,
                                   float mul, uint8_t* stage, const CUtensorMap* map, int col0,
                                   int d) {
    const int q = it.s.z * 128 + warp * 32;
    packed_rows_store<NCOL>(tcol, mul, stage, map, it.h, it.s.x + q, it.s.y - q, col0, d, g.p.dQ,
                            g.p.lddq);
  }
  // Rows that no sequence covers, where the caller asked for zeros.
  FA_DEV static void finish(const View& g, int d) {
    const Params& p = g.p;
    const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long nt = (long long)gridDim.x * blockDim.x;
    if (p.fill & 1) zero_rows(p.dQ, g.covered, p.total, p.Hq * d, p.lddq, t, nt);
    if (p.fill & 2) zero_rows(p.dK, g.covered, p.total, p.Hkv * d, p.lddk, t, nt);
    if (p.fill & 4) zero_rows(p.dV, g.covered, p.total, p.Hkv * d, p.lddv, t, nt);
  }
};

// -D = -rowsum(dO o O) and -L * log2(e) of one 128-row tile and head per block step;
// rows past the sequence's end get 0 and -inf, so that P is exactly 0 there. Bound by
// reading O and dO from HBM: D / 8 lanes per row, 16 bytes of each per lane, four rows
// in flight per lane before any arithmetic.
template <int D>
__global__ void __launch_bounds__(256) packed_preprocess_kernel(
    const __nv_bfloat16* __restrict__ O, const __nv_bfloat16* __restrict__ dO,
    const float* __restrict__ L, const uint8_t* __restrict__ plan, long long off_kv,
    float* __restrict__ ws_nD, float* __restrict__ ws_nL2, long long ws_rows, int total, int nseq,
    int Hq, int d, int trigger) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPB = 256 / LPR;    // rows per block step
  constexpr int U = 4;              // steps in flight
  static_assert(128 % (RPB * U) == 0, "whole rounds of steps per tile");
  __shared__ float sums[128];
  grid_wait();
  if (trigger) grid_launch_dependents();
  const PlanHead* head = reinterpret_cast<const PlanHead*>(plan);
  if (!plan_matches(head, total, nseq, &g_packed_bwd_status)) return;
  const long long pairs = (long long)head->tiles128 * Hq;
  const int sub = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  for (long long i = blockIdx.x; i < pairs; i += gridDim.x) {
    const int e = (int)(i / Hq), h = (int)(i - (long long)e * Hq);
    const PlanTile s = __ldg(reinterpret_cast<const PlanTile*>(plan + off_kv) + e);
    const int valid = s.y - s.z * 128;  // rows of this tile
    const size_t row0 = (size_t)s.x + (size_t)s.z * 128;
#pragma unroll
    for (int base = 0; base < 128; base += RPB * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = base + u * RPB + r0;
        a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < valid && 8 * sub < d) {
          const size_t at = ((row0 + r) * Hq + h) * d;
          a[u] = reinterpret_cast<const uint4*>(O + at)[sub];
          b[u] = reinterpret_cast<const uint4*>(dO + at)[sub];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float acc = bf16_lo(a[u].x) * bf16_lo(b[u].x) + bf16_hi(a[u].x) * bf16_hi(b[u].x) +
                    bf16_lo(a[u].y) * bf16_lo(b[u].y) + bf16_hi(a[u].y) * bf16_hi(b[u].y) +
                    bf16_lo(a[u].z) * bf16_lo(b[u].z) + bf16_hi(a[u].z) * bf16_hi(b[u].z) +
                    bf16_lo(a[u].w) * bf16_lo(b[u].w) + bf16_hi(a[u].w) * bf16_hi(b[u].w);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (sub == 0) sums[base + u * RPB + r0] = acc;
      }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      const int r = threadIdx.x;
      const size_t w = (size_t)h * ws_rows + s.w + s.z * 128 + r;
      ws_nD[w] = -sums[r];
      ws_nL2[w] = r < valid ? -L[(size_t)h * total + row0 + r] * kLog2e : -INFINITY;
    }
    __syncthreads();
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <int D>
cudaError_t launch_packed_bwd_d(const PackedBwdArgs& a, cudaStream_t stream) {
  const PlanLayout lay = plan_layout(a.nseq, a.total);
  const long long ws_rows = packed_ws_rows(a.nseq, a.total);
  const int sms = sm_count();
  const long long pairs = lay.cap[kKeyList] * a.Hq;
  cudaError_t e = launch_early(
      packed_preprocess_kernel<D>, (unsigned)(pairs < 8LL * sms ? pairs : 8LL * sms), 256, 0, stream,
      static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO), a.L,
      static_cast<const uint8_t*>(a.plan), (long long)lay.off[kKeyList], a.ws_nD, a.ws_nL2, ws_rows,
      a.total, a.nseq, a.Hq, a.d, pairs < sms ? 1 : 0);
  if (e != cudaSuccess) return e;

  CUtensorMap mq, mk, mv, mdo, ml2, md, mdq, mdk, mdv;
  const long long ldo = (long long)a.Hq * a.d;
  const cuuint64_t dims[2] = {(cuuint64_t)ws_rows, (cuuint64_t)a.Hq};
  const cuuint64_t strides[1] = {(cuuint64_t)ws_rows * 4};
  const cuuint32_t box[2] = {64, 1};
  if (make_bf16_packed_map(&mq, a.Q, a.total, a.Hq, a.d, a.ldq, 64) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mk, a.K, a.total, a.Hkv, a.d, a.ldk, 128) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mv, a.V, a.total, a.Hkv, a.d, a.ldv, 128) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mdo, a.dO, a.total, a.Hq, a.d, ldo, 64) != CUDA_SUCCESS ||
      encode_tensor_map(&ml2, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.ws_nL2, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
      encode_tensor_map(&md, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.ws_nD, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdq, a.dQ, a.total, a.Hq, a.d, a.lddq) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdk, a.dK, a.total, a.Hkv, a.d, a.lddk) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdv, a.dV, a.total, a.Hkv, a.d, a.lddv) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  BwdParams p;
  p.d = a.d;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  PackedBwd::Params g;
  g.plan = static_cast<const uint8_t*>(a.plan);
  g.off_kv = (long long)lay.off[kKeyList];
  g.off_q = (long long)lay.off[1];
  g.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  g.dK = static_cast<__nv_bfloat16*>(a.dK);
  g.dV = static_cast<__nv_bfloat16*>(a.dV);
  g.lddq = a.lddq;
  g.lddk = a.lddk;
  g.lddv = a.lddv;
  g.nD = a.ws_nD;
  g.nL2 = a.ws_nL2;
  g.ws_rows = ws_rows;
  g.total = a.total;
  g.nseq = a.nseq;
  g.Hq = a.Hq;
  g.Hkv = a.Hkv;
  g.per_kv = a.Hq / a.Hkv;
  g.causal = a.causal;
  g.fill = a.fill;
  const int tiles = ceil_div(a.total, 128);
  g.kgroup = heads_per_group(a.Hkv, tiles);
  g.qgroup = round_up(heads_per_group(a.Hq, tiles), g.per_kv);
  constexpr int smem = BwdSmem<D>::BYTES;
  e = cudaFuncSetAttribute(bwd_kernel<D, PackedBwd>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  const long long items = pairs + lay.cap[kKeyList] * a.Hkv;
  g.trigger = items < sms;  // see launch_as
  return launch_early(bwd_kernel<D, PackedBwd>, (unsigned)(items < sms ? items : sms),
                      KvCfg<D>::THREADS, smem, stream, mq, mk, mv, mdo, ml2, md, mdq, mdk, mdv, p, g);
}

}  // namespace

cudaError_t launch_packed_backward(const PackedBwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_packed_bwd_d<128>(a, s) : launch_packed_bwd_d<64>(a, s);
}

cudaError_t packed_bwd_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_bwd_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_packed_bwd_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
