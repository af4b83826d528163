// Norms of queries and keys with the position rotation, on their own and on the way into
// a paged cache (bf16 or 4 bits): arguments of the launches.
#pragma once

#include "fa.h"
#include "fa_internal.h"

namespace fa {

struct RopeArgs {  // of Q or of K; strides in elements
  const void *Q, *K;
  void *Qo, *Ko;
  long long ldq, ldk, ldqo, ldko;
  const int* positions;
  int total, Hq, Hkv, d;
  fa_rope how;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

struct RopeBackwardArgs {
  const void *dQo, *dKo, *Q, *K;  // Q or K NULL where it has no weight
  void *dQ, *dK;
  long long lddqo, lddko, ldq, ldk, lddq, lddk;
  const int* positions;
  float *dwq, *dwk, *partial;
  int total, Hq, Hkv, d;
  fa_rope how;
};
// Bytes of partial sums of the weights' gradients.
size_t rope_workspace_bytes(int d);
cudaError_t launch_rope_backward(const RopeBackwardArgs& a, cudaStream_t s);
cudaError_t rope_read_status(unsigned int* out);

// Rows of requests at cache positions.
struct PlaceArgs {
  const int *cu_seqlens, *starts, *table;
  int total, nseq, max_pages, num_pages, Hkv, d, page;
};
struct RopeAppendArgs {
  PlaceArgs at;
  const void *Q, *K, *V;  // Q may be NULL
  void* Qo;
  long long ldq, ldk, ldv;
  void *Kc, *Vc;  // bf16 caches, or
  void* cache4;   // the cache in 4 bits
  int Hq, fill;
  fa_rope how;
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s);

struct Cache4ReadArgs {
  PlaceArgs at;
  const void* cache;
  void *K, *V;  // bf16 [total, Hkv, d], dense
  int fill;
};
cudaError_t launch_cache4_read(const Cache4ReadArgs& a, cudaStream_t s);
cudaError_t rope_append_read_status(unsigned int* out);

struct Decode4Args {
  const void *Q, *cache;
  const int *table, *lens;
  void* O;
  float* L;
  void* workspace;
  int B, Hq, Hkv, d, max_pages, num_pages, page;
  float scale;
};
size_t decode4_workspace_bytes(int B, int Hq, int Hkv, int d, int capacity);
cudaError_t launch_decode4(const Decode4Args& a, cudaStream_t s);
cudaError_t decode4_read_status(unsigned int* out);

}  // namespace fa
