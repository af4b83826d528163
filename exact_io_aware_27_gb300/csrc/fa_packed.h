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

// The gradient kernel's work on key blocks: all queries of one, or a range of their
// 64-query halves.
struct BwdItem {
  PlanTile s;
  int head;
  int first, halves;
  int slot;  // a part: where its sums go; else -1
};
// A key block whose parts' sums, in slots [slot, slot + parts), are joined.
struct BwdJoin {
  PlanTile s;
  int head, slot, parts, pad;
};
// How the gradient kernel's items are dealt to its CTAs where key blocks are split (see
// fa_packed_backward.cu); split_tiles = 0 where none is. A list's item of row t for CTA c
// is number t P + rank, with a rank per CTA and 1 << shift rows.
constexpr int kMaxBwdCtas = 192;  // ranks are bytes
struct BwdDealHead {
  int parts;        // entries of the table of parts, the first items of the key blocks' list
  int split_tiles;  // the plan's first key tiles, which they hold
  int joins;        // split key blocks
  int shifts;       // of the key blocks' list, and << 8 of the query blocks'
  int4 cta[kMaxBwdCtas];  // its key blocks and query blocks, its first rank of those, and
                          // in which row of ranks they start
};
// A key block is split where it has more than 5/3 hc halves, into ceil(halves / hc) parts,
// with hc = max(kMinPart, 6/5 of the batch's halves / kPartShare): a fifth more than what
// one of 152 SMs gets of the dK/dV pass, which takes some 60 % of the time. With W halves
// in the batch, W / hc <= 5/6 kPartShare and there are at most 8/5 W / hc parts.
constexpr int kMinPart = 16, kPartShare = 152, kMaxParts = 256;
static_assert(kMaxParts >= 8 * kPartShare / 6, "every part has a slot");
// The deal and the join cost some 5 us: batches whose key blocks are not likely to have
// more halves than this are not split.
constexpr int kSplitFrom = 32;
constexpr size_t kPartBytes128 = 2 * 128 * 128 * 4;  // dV and dK of a key block, fp32, d = 128

// Backward workspace: -D and -L * log2(e), fp32 [Hq, rows] each (a sequence's rows start at
// its tiles' PlanTile::w), the deal's head, the split key blocks, the parts, the ranks and
// the parts' sums.
struct PackedBwdLayout {
  long long rows;
  size_t nD, nL2, head, joins, items, ranks, parts, bytes;
  int slots;
};
inline PackedBwdLayout packed_bwd_layout(int nseq, int total, int Hq) {
  const long long cap = plan_layout(nseq, total).cap[kKeyList];
  PackedBwdLayout l;
  l.rows = cap * kWorkspaceRowAlign;
  // A batch has at most cap key blocks of ceil(total / 64) halves per query head.
  const long long halves = ceil_div(total, 64);
  const long long most = cap * Hq * halves * 2 / kMinPart;
  l.slots = halves * Hq <= kSplitFrom ? 0 : (int)(most < kMaxParts ? most : kMaxParts);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = (at + n + 127) / 128 * 128;
    return here;
  };
  l.nD = take((size_t)l.rows * Hq * 4);
  l.nL2 = take((size_t)l.rows * Hq * 4);
  l.head = take(sizeof(BwdDealHead));
  l.joins = take(kMaxParts / 2 * sizeof(BwdJoin));
  l.items = take(kMaxParts * sizeof(BwdItem));
  l.ranks = take((size_t)cap * Hq * 2 + kMaxParts + 4 * kMaxBwdCtas);
  l.parts = take((size_t)l.slots * kPartBytes128);
  l.bytes = at;
  return l;
}
struct PackedBwdArgs {
  const void *Q, *K, *V, *O, *dO;
  const float* L;
  long long ldq, ldk, ldv;
  void *dQ, *dK, *dV;
  long long lddq, lddk, lddv;
  void* workspace;
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
