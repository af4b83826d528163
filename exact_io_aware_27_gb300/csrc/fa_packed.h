// Plans of packed batches (sequences one after another in one tensor), shared by
// the plan kernel and the passes that read a plan.
#pragma once

#include "fa_internal.h"

namespace fa {

// One entry of a plan's work lists: a tile of one sequence.
//   x  first row of the sequence in the packed tensors
//   y  length of the sequence
//   z  tile within the sequence
//   w  first workspace row of the sequence (a multiple of kWorkspaceRowAlign)
using PlanTile = int4;

// The plan's first 64 bytes, written by the plan kernel.
constexpr int kPlanMagic = 0x50415131;
struct PlanHead {
  int magic;        // kPlanMagic
  int total, nseq;  // the sizes the plan was made for
  int covered;      // rows the sequences cover; the rest of the tensors belongs to none
  int tiles256;     // entries of the list of 256-row tiles
  int tiles128;     // entries of each list of 128-row tiles
  int tiles64, tiles32;
  int pad[8];
};
static_assert(sizeof(PlanHead) == 64, "the lists start 64 bytes into a plan");

// A plan's lists: tiles of 256 >> i rows for i = 0..3, the last rows of a sequence (the
// most expensive under causal masking) first; and the 128-row key blocks, the first rows
// first. Each holds at most total / tile + nseq entries.
constexpr int kPlanLists = 5, kKeyList = 4;
__host__ __device__ constexpr int plan_tile_rows(int list) { return list == kKeyList ? 128 : 256 >> list; }
struct PlanLayout {
  long long cap[kPlanLists];
  size_t off[kPlanLists], off_scan, bytes;
};
inline PlanLayout plan_layout(int nseq, int total) {
  PlanLayout l;
  size_t at = sizeof(PlanHead);
  for (int i = 0; i < kPlanLists; ++i) {
    l.cap[i] = (long long)total / plan_tile_rows(i) + nseq;
    l.off[i] = at;
    at += (size_t)l.cap[i] * sizeof(PlanTile);
  }
  l.off_scan = at;
  l.bytes = at + ((size_t)nseq + 1) * 4 * sizeof(int);
  l.bytes = (l.bytes + 15) / 16 * 16;
  return l;
}

// bf16 [rows, H, d] with `ld` elements from row to row, as boxes of 64 columns x
// box_heads heads x box_rows rows with 128-byte swizzle (loads), or of 32 columns x
// box_heads heads x 32 / box_heads rows with 64-byte swizzle (stores).
CUresult make_bf16_packed_map(CUtensorMap* map, const void* base, int rows, int H, int d,
                              long long ld, int box_rows, int box_heads = 1);
CUresult make_bf16_packed_store_map(CUtensorMap* map, void* base, int rows, int H, int d,
                                    long long ld, int box_heads = 1);

struct PackedFwdArgs {
  const void *Q, *K, *V;
  long long ldq, ldk, ldv;  // elements from row to row
  void* O;
  float* L;
  const void* plan;
  int total, nseq, Hq, Hkv, d, causal, fill;
  float scale;
};
// Backward workspace: -D and -L * log2(e), fp32 [Hq, packed_ws_rows] each; a
// sequence's rows start at its tiles' PlanTile::w.
inline long long packed_ws_rows(int nseq, int total) {
  return plan_layout(nseq, total).cap[kKeyList] * kWorkspaceRowAlign;
}
struct PackedBwdArgs {
  const void *Q, *K, *V, *O, *dO;
  const float* L;
  long long ldq, ldk, ldv;
  void *dQ, *dK, *dV;
  long long lddq, lddk, lddv;
  float *ws_nD, *ws_nL2;
  const void* plan;
  int total, nseq, Hq, Hkv, d, causal, fill;
  float scale;
};
cudaError_t launch_packed_backward(const PackedBwdArgs& a, cudaStream_t s);
cudaError_t packed_bwd_read_status(unsigned int* out);
cudaError_t launch_packed_plan(const int* cu_seqlens, int nseq, int total, int causal, void* plan,
                               cudaStream_t s);
cudaError_t launch_packed_forward(const PackedFwdArgs& a, cudaStream_t s);
cudaError_t plan_read_status(unsigned int* out);
cudaError_t packed_read_status(unsigned int* out);

}  // namespace fa
