// The dense backward pass: the preprocess kernel and the gradient kernel
// (fa_backward.cuh) over [BH, n|m, d] tensors.
#include "fa_backward.cuh"

namespace fa {

__device__ unsigned int g_bwd_status;

namespace {

struct DenseBwd {
  struct Params {
    __nv_bfloat16 *dK, *dV;
    const float *nD, *nL2;
    int n, m, n_pad, BH, causal, ktiles, kgroup, qtiles, qgroup, n_kv, n_dq;
  };
  using View = const Params&;
  struct KvItem {
    int ks, bh;  // first key, head
  };
  struct QItem {
    int q0, bh;  // first query, head
  };
  static constexpr bool kEarly = false;
  static constexpr bool kHeads = false, kListed = false;
  static constexpr bool kForeignTail = false;  // TMA reads zeros past a head's rows
  FA_DEV static View view(const Params& g) { return g; }
  FA_DEV static unsigned int* status() { return &g_bwd_status; }
  FA_DEV static int causal(const Params& g) { return g.causal; }
  // Each list is dealt in snake order; the query blocks in reverse CTA order, so that
  // the CTAs left with one key block more get no query block more.
  FA_DEV static int kv_count(const Params& g, int c, int P) { return snake_count(g.n_kv, c, P); }
  FA_DEV static int q_count(const Params& g, int c, int P) {
    return snake_count(g.n_dq, P - 1 - c, P);
  }
  FA_DEV static void finish(const Params&, int) {}

  // Key blocks near 0 carry the most work under causal masking: the launch order puts
  // rank 0 first, heads a group at a time so that the blocks in flight share L2.
  FA_DEV static int kv_rank(const Params&, int, int, int) { return 0; }
  FA_DEV static int q_rank(const Params&, int, int, int) { return 0; }
  FA_DEV static KvItem kv_item(const Params& g, int t, int, int c, int P) {
    int ktile, bh;
    grouped_tile(snake_item(t, c, P), g.BH, g.ktiles, g.kgroup, ktile, bh);
    return {ktile * 128, bh};
  }
  FA_DEV static int first_key(const KvItem& it) { return it.ks; }
  FA_DEV static int rows(const Params& g, const KvItem&) { return g.n; }
  FA_DEV static int keys(const Params& g, const KvItem&) { return g.m; }
  // Whole 128-query blocks, from the first with a query q >= ks.
  FA_DEV static int kv_halves(const Params& g, const KvItem& it, int& q_first) {
    const int i0 = g.causal ? it.ks / 128 : 0;
    q_first = i0 * 128;
    return 2 * max(0, (g.n + 127) / 128 - i0);
  }
  FA_DEV static int kv_part(const Params&, const KvItem&, int per, int& first) {
    first = 0;
    return per;
  }
  FA_DEV static void load_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                               const Params&, const KvItem& it) {
    tma_load_3d(dst, map, f, col, it.ks, it.bh);
  }
  FA_DEV static void load_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                  const Params&, const KvItem& it, int, int q) {
    tma_load_3d(dst, map, f, col, q, it.bh);
  }
  FA_DEV static void load_stats(void* dst, const CUtensorMap* map, uint64_t* f, const Params&,
                                const KvItem& it, int, int q) {
    tma_load_2d(dst, map, f, q, it.bh);
  }
  template <int D>
  FA_DEV static void store_keys(const Params& g, const KvItem& it, int, int warp, uint32_t col,
                                float mul, uint8_t* stage, const CUtensorMap* map, int d) {
    tmem_rows_store<D>(col, mul, stage, map, 0, it.ks + warp * 32, g.m, it.bh, d);
  }
  template <int D>
  FA_DEV static void zero_key(const Params& g, const KvItem& it, int w, int key, int d) {
    __nv_bfloat16* const out = w == 0 ? g.dV : g.dK;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      if (8 * c < d) reinterpret_cast<uint4*>(out + ((size_t)it.bh * g.m + key) * d)[c] = z;
  }

  // Under causal masking the last query blocks see the most keys: the launch order
  // puts them first.
  FA_DEV static QItem q_item(const Params& g, int t, int, int c, int P) {
    int rank, bh;
    grouped_tile(snake_item(t, P - 1 - c, P), g.BH, g.qtiles, g.qgroup, rank, bh);
    return {(g.causal ? g.qtiles - 1 - rank : rank) * 128, bh};
  }
  FA_DEV static int first_query(const QItem& it) { return it.q0; }
  FA_DEV static int keys(const Params& g, const QItem&) { return g.m; }
  FA_DEV static int key_blocks(const Params& g, const QItem& it) {
    const int nkb = (g.m + 127) / 128;
    return g.causal ? min(nkb, min(it.q0 + 127, g.n - 1) / 128 + 1) : nkb;  // keys k <= q
  }
  FA_DEV static void load_block_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                        const Params&, const QItem& it, int row) {
    tma_load_3d(dst, map, f, col, it.q0 + row, it.bh);
  }
  FA_DEV static void load_block_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                     const Params&, const QItem& it, int key) {
    tma_load_3d(dst, map, f, col, key, it.bh);
  }
  FA_DEV static void query_stats(const Params& g, const QItem& it, int r, float& nl2, float& nd) {
    const size_t row = (size_t)it.bh * g.n_pad + it.q0 + r;  // < n_pad always
    nl2 = g.nL2[row];
    nd = g.nD[row];
  }
  template <int NCOL>
  FA_DEV static void store_queries(const Params& g, const QItem& it, int warp, uint32_t tcol,
                                   float mul, uint8_t* stage, const CUtensorMap* map, int col0,
                                   int d) {
    tmem_rows_store<NCOL>(tcol, mul, stage, map, col0, it.q0 + warp * 32, g.n, it.bh, d - col0);
  }
};

// ================================================================== preprocess
// Each warp step covers RPW consecutive workspace rows (head bh, query q <
// n_pad), LPR lanes per row, one 16-byte load of O and of dO per lane:
// -D = -sum_c dO*O and -L * log2(e). Rows q >= n get -D = 0 and -inf, so that
// recomputed probabilities there are exactly 0. A warp takes U steps at a time
// and issues all their loads before any arithmetic (memory-level parallelism:
// the kernel is bound by reading O and dO from HBM).
template <int D>
__global__ void __launch_bounds__(256) preprocess_kernel(const __nv_bfloat16* __restrict__ O,
                                                         const __nv_bfloat16* __restrict__ dO,
                                                         const float* __restrict__ L,
                                                         float* __restrict__ ws_nD,
                                                         float* __restrict__ ws_nL2, int n,
                                                         int n_pad, int d, long long rows) {
  constexpr int LPR = D / 8;     // lanes per row (8 bf16 per lane)
  constexpr int RPW = 32 / LPR;  // rows per warp step
  constexpr int U = 4;           // warp steps in flight
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPR;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long base = ((long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RPW * U;
       base < rows; base += warps * RPW * U) {
    // base is a multiple of RPW * U, which divides n_pad: the U * RPW rows of this
    // iteration are queries q0 .. q0 + U * RPW - 1 of one head
    const long long bh = base / n_pad;
    const int q0 = (int)(base - bh * n_pad) + lane / LPR;
    const __nv_bfloat16* o_head = O + (size_t)bh * n * d;
    const __nv_bfloat16* do_head = dO + (size_t)bh * n * d;
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + u * RPW;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);  // zero products for rows and lanes past the data
      if (q < n && 8 * sub < d) {
        a[u] = reinterpret_cast<const uint4*>(o_head + (size_t)q * d)[sub];
        b[u] = reinterpret_cast<const uint4*>(do_head + (size_t)q * d)[sub];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + u * RPW;
      float acc = bf16_lo(a[u].x) * bf16_lo(b[u].x) + bf16_hi(a[u].x) * bf16_hi(b[u].x) +
                  bf16_lo(a[u].y) * bf16_lo(b[u].y) + bf16_hi(a[u].y) * bf16_hi(b[u].y) +
                  bf16_lo(a[u].z) * bf16_lo(b[u].z) + bf16_hi(a[u].z) * bf16_hi(b[u].z) +
                  bf16_lo(a[u].w) * bf16_lo(b[u].w) + bf16_hi(a[u].w) * bf16_hi(b[u].w);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if (sub == 0) {
        const size_t r = (size_t)bh * n_pad + q;
        ws_nD[r] = -acc;
        ws_nL2[r] = (q < n) ? -L[(size_t)bh * n + q] * kLog2e : -INFINITY;
      }
    }
  }
}

template <int D>
cudaError_t launch_bwd_d(const BwdArgs& a, bool with_kv, bool with_dq, cudaStream_t stream) {
  using KC = KvCfg<D>;
  using QC = QCfg<D>;
  static_assert(KC::BQ == QC::BM && KC::BN == QC::BN, "the passes share the tensor maps");
  static_assert(KC::THREADS == QC::THREADS, "the passes share the launch");
  CUtensorMap mq, mk, mv, mdo, ml2, md, mdq, mdk, mdv;
  // Q and dO, -L2 and -D travel in 64-row pieces; K and V in 128-row tiles.
  // Rows of d values; the 64-column boxes read zeros past d.
  if (make_bf16_head_map(&mq, a.Q, a.BH, a.n, a.d, 64) != CUDA_SUCCESS ||
      make_bf16_head_map(&mk, a.K, a.BH, a.m, a.d, KC::BN) != CUDA_SUCCESS ||
      make_bf16_head_map(&mv, a.V, a.BH, a.m, a.d, KC::BN) != CUDA_SUCCESS ||
      make_bf16_head_map(&mdo, a.dO, a.BH, a.n, a.d, 64) != CUDA_SUCCESS ||
      make_f32_row_map(&ml2, a.ws_nL2, a.BH, a.n_pad, 64) != CUDA_SUCCESS ||
      make_f32_row_map(&md, a.ws_nD, a.BH, a.n_pad, 64) != CUDA_SUCCESS ||
      make_bf16_store_map(&mdq, a.dQ, a.BH, a.n, a.d) != CUDA_SUCCESS ||
      make_bf16_store_map(&mdk, a.dK, a.BH, a.m, a.d) != CUDA_SUCCESS ||
      make_bf16_store_map(&mdv, a.dV, a.BH, a.m, a.d) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  BwdParams p;
  p.d = a.d;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  DenseBwd::Params g;
  g.dK = static_cast<__nv_bfloat16*>(a.dK);
  g.dV = static_cast<__nv_bfloat16*>(a.dV);
  g.nD = a.ws_nD;
  g.nL2 = a.ws_nL2;
  g.n = a.n;
  g.m = a.m;
  g.n_pad = a.n_pad;
  g.BH = a.BH;
  g.causal = a.causal;
  g.ktiles = ceil_div(a.m, KC::BN);
  g.kgroup = heads_per_group(a.BH, g.ktiles);
  g.qtiles = ceil_div(a.n, QC::BM);
  g.qgroup = heads_per_group(a.BH, g.qtiles);
  g.n_kv = with_kv ? g.ktiles * a.BH : 0;
  g.n_dq = with_dq ? g.qtiles * a.BH : 0;
  constexpr int smem = BwdSmem<D>::BYTES;
  cudaError_t e =
      cudaFuncSetAttribute(bwd_kernel<D, DenseBwd>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int grid = g.n_kv + g.n_dq < sms ? g.n_kv + g.n_dq : sms;
  bwd_kernel<D, DenseBwd><<<(unsigned)grid, KC::THREADS, smem, stream>>>(
      mq, mk, mv, mdo, ml2, md, mdq, mdk, mdv, p, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_preprocess(const BwdArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.BH * a.n_pad;
  const bool wide = a.d > 64;
  // 4 warp steps of 2 (d > 64) or 4 rows per warp, 8 warps a block, at most one
  // full-occupancy wave (8 blocks of 256 threads per SM); grid-stride beyond.
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long rows_per_block = (wide ? 2 : 4) * 4 * 8;
  long long blocks = (rows + rows_per_block - 1) / rows_per_block;
  if (blocks > 8LL * sms) blocks = 8LL * sms;
  const int grid = (int)(blocks < 1 ? 1 : blocks);
  if (wide)
    preprocess_kernel<128><<<grid, 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO), a.L,
        a.ws_nD, a.ws_nL2, a.n, a.n_pad, a.d, rows);
  else
    preprocess_kernel<64><<<grid, 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO), a.L,
        a.ws_nD, a.ws_nL2, a.n, a.n_pad, a.d, rows);
  return cudaGetLastError();
}

// Head dimensions up to 64 run the 64-column kernels, larger ones the 128-column
// kernels (columns past d read as zeros).
cudaError_t launch_bwd_dkdv(const BwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_bwd_d<128>(a, true, false, s) : launch_bwd_d<64>(a, true, false, s);
}

cudaError_t launch_bwd_dq(const BwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_bwd_d<128>(a, false, true, s) : launch_bwd_d<64>(a, false, true, s);
}

cudaError_t launch_bwd_main(const BwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_bwd_d<128>(a, true, true, s) : launch_bwd_d<64>(a, true, true, s);
}

cudaError_t bwd_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_bwd_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_bwd_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
