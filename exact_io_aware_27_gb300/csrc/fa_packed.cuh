// Device helpers of the passes over packed sequences.
#pragma once

#include "fa_packed.h"
#include "sm103.cuh"

namespace fa {
namespace {

// Entries of a plan's list, or 0 (and kDeviceIndexBit in `status`) for a plan that
// was not made for these sizes: its entries would not be rows of these tensors.
FA_DEV bool plan_matches(const PlanHead* h, int total, int nseq, unsigned int* status) {
  if (h->magic == kPlanMagic && h->total == total && h->nseq == nseq) return true;
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kDeviceIndexBit);
  return false;
}

// tmem_rows_store for rows of a packed tensor [rows, H, d]: NCOL columns of this
// warp's 32 TMEM lanes, times `mul`, to columns [col0, d). Lane i is head h + i % heads
// (heads = 1 << head_shift) of row row0 + i / heads; the first `valid` lanes are stored
// (valid may be <= 0 or above 32). A full piece leaves through the staging buffers and TMA; a
// piece that ends inside its 32 rows, where the next row belongs to another sequence,
// is written lane by lane (`out` is the tensor, `ld` its row stride). BUFS: staging buffers
// of 2 KB.
template <int NCOL, int BUFS = 2>
FA_DEV void packed_rows_store(uint32_t tcol, float mul, uint8_t* stage, const CUtensorMap* map,
                              int h, int row0, int valid, int col0, int d, __nv_bfloat16* out,
                              long long ld, int head_shift = 0) {
  if (valid <= 0) return;  // warp-uniform
  const int valid_cols = d - col0;
  const int lane = threadIdx.x & 31;
  const bool full = valid >= 32;
  if (full) {
    if (lane == 0) bulk_wait_read<0>();  // copies of an earlier call
    __syncwarp();
  }
#pragma unroll
  for (int c = 0; c < NCOL / 32; ++c) {
    if (32 * c >= valid_cols) break;  // warp-uniform
    uint32_t o[32];
    tmem_ld32(tcol + 32 * c, o);
    tmem_ld_wait();
    reg_fence32(o);
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = pack_bf16(__uint_as_float(o[2 * e]) * mul, __uint_as_float(o[2 * e + 1]) * mul);
    if (!full) {
      if (lane < valid) {
        const int at = h + (lane & ((1 << head_shift) - 1));
        uint4* dst = reinterpret_cast<uint4*>(out + (row0 + (lane >> head_shift)) * ld +
                                              (long long)at * d + col0 + 32 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (32 * c + 8 * k < valid_cols)
            dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      continue;
    }
    uint8_t* buf = stage + c % BUFS * 2048;
    if (c >= BUFS) {  // the copy of piece c - BUFS has read this buffer
      if (lane == 0) bulk_wait_read<BUFS - 1>();
      __syncwarp();
    }
    const uint32_t row = smem_u32(buf) + lane * 64;
    const uint32_t sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      st_shared_v4(row + (((uint32_t)k ^ sw) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2],
                   w[4 * k + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, buf, col0 + 32 * c, h, row0);
      bulk_commit();
    }
  }
}

// Zeros rows [first, last) of a packed bf16 tensor (rows of `cols` values, `ld` from
// row to row; cols and ld multiples of 8), by thread `t` of `nt` over the grid.
FA_DEV void zero_rows(__nv_bfloat16* x, long long first, long long last, int cols, long long ld,
                      long long t, long long nt) {
  const int per = cols / 8;
  for (long long i = t; i < (last - first) * per; i += nt) {
    const long long r = i / per;
    reinterpret_cast<uint4*>(x + (first + r) * ld)[i - r * per] = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace
}  // namespace fa
