// The paged cache and decode attention behind a shared prefix: arguments and the
// workspace that its three kernels share.
#pragma once

#include "fa_internal.h"

namespace fa {

// Caches are bf16 [pages, Hkv, page, d], page a power of two.
constexpr int kMinPage = 16, kMaxPage = 1024;
constexpr int kMaxBatch = 8192;

struct AppendArgs {
  const void *K, *V;
  long long ldk, ldv;
  const int *cu_seqlens, *starts, *table;
  void *Kc, *Vc;
  int total, nseq, Hkv, d, max_pages, num_pages, page;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s);
cudaError_t append_read_status(unsigned int* out);

struct DecodeArgs {
  const void *Q, *Kc, *Vc;
  const int *prefix_pages, *prefix_len, *table, *lens;
  void* O;
  float* L;
  void* workspace;
  int B, Hq, Hkv, d, prefix_cap, max_pages, num_pages, page;  // prefix_cap: pages
  float scale;
};
// Bytes of workspace for at most prefix_cap shared and own_cap own keys a request.
size_t decode_workspace_bytes(int B, int Hq, int Hkv, int d, int prefix_cap, int own_cap);
cudaError_t launch_prefix_decode(const DecodeArgs& a, cudaStream_t s);
cudaError_t prefix_read_status(unsigned int* out);

}  // namespace fa
