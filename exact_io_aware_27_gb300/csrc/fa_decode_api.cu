// Host side of the paged-cache entry points of include/fa.h: argument checks.
#include "fa_check.h"
#include "fa_decode.h"

namespace fa {

namespace {

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxSequences = 65535;
constexpr long long kMaxRowStride = 1LL << 30;  // elements
constexpr long long kMaxKeys = 1LL << 30;       // keys a table row can name

// The cache's sizes: FA_OK or the status to return.
int check_cache(int num_pages, int Hkv, int page, int d) {
  if (num_pages < 1 || Hkv < 1 || Hkv > 65535) return FA_ERR_INVALID_ARG;
  if (page < kMinPage || page > kMaxPage || (page & (page - 1)) != 0) return FA_ERR_INVALID_ARG;
  if ((long long)num_pages * Hkv > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED_HEAD_DIM;
  return FA_OK;
}

size_t cache_bytes(int num_pages, int Hkv, int page, int d) {
  return (size_t)num_pages * Hkv * page * d * 2;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_append(const void* K, const void* V, long long k_stride, long long v_stride,
                    int total, const int* cu_seqlens, const int* starts, int nseq,
                    const int* block_table, int max_pages, void* K_cache, void* V_cache,
                    int num_pages, int Hkv, int page, int d, void* stream) {
  int rc = check_cache(num_pages, Hkv, page, d);
  if (rc != FA_OK) return rc;
  if (total < 1 || total > kMaxRows || nseq < 1 || nseq > kMaxSequences || max_pages < 1 ||
      (long long)max_pages * page > kMaxKeys)
    return FA_ERR_INVALID_ARG;
  if (!K || !V || !cu_seqlens || !starts || !block_table || !K_cache || !V_cache)
    return FA_ERR_INVALID_ARG;
  for (long long ld : {k_stride, v_stride})
    if (ld < (long long)Hkv * d || ld % 8 != 0 || ld > kMaxRowStride) return FA_ERR_INVALID_ARG;
  for (const void* p : {K, V, static_cast<const void*>(K_cache), static_cast<const void*>(V_cache)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  for (const int* p : {cu_seqlens, starts, block_table})
    if (!is_aligned(p, 4)) return FA_ERR_MISALIGNED;
  const size_t width = (size_t)Hkv * d * 2, cache = cache_bytes(num_pages, Hkv, page, d);
  const Rows ins[] = {rows_of(K, total, width, (size_t)k_stride * 2),
                      rows_of(V, total, width, (size_t)v_stride * 2),
                      bytes_of(cu_seqlens, ((size_t)nseq + 1) * 4), bytes_of(starts, (size_t)nseq * 4),
                      bytes_of(block_table, (size_t)nseq * max_pages * 4)};
  const Rows outs[] = {bytes_of(K_cache, cache), bytes_of(V_cache, cache)};
  for (const Rows& o : outs)
    for (const Rows& i : ins)
      if (rows_overlap(o, i)) return FA_ERR_INVALID_ARG;
  if (rows_overlap(outs[0], outs[1])) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  AppendArgs a;
  a.K = K;
  a.V = V;
  a.ldk = k_stride;
  a.ldv = v_stride;
  a.cu_seqlens = cu_seqlens;
  a.starts = starts;
  a.table = block_table;
  a.Kc = K_cache;
  a.Vc = V_cache;
  a.total = total;
  a.nseq = nseq;
  a.Hkv = Hkv;
  a.d = d;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page = page;
  return launch_cache_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                  : FA_ERR_CUDA;
}

static int check_decode(int B, int Hq, int Hkv, int d) {
  if (B < 1 || B > kMaxBatch || Hq < 1 || Hq > 65535 || Hkv < 1 || Hq % Hkv != 0 ||
      Hq / Hkv > 128 || (long long)B * Hq > 0x7fffffffLL)
    return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED_HEAD_DIM;
  return FA_OK;
}

size_t fa_prefix_workspace_bytes(int B, int Hq, int Hkv, int d, int prefix_capacity,
                                 int own_capacity) {
  if (check_decode(B, Hq, Hkv, d) != FA_OK || prefix_capacity < 0 || prefix_capacity > kMaxKeys ||
      own_capacity < 0 || own_capacity > kMaxKeys)
    return 0;
  return decode_workspace_bytes(B, Hq, Hkv, d, prefix_capacity, own_capacity);
}

int fa_prefix_decode(const void* Q, const void* K_cache, const void* V_cache,
                     const int* prefix_pages, int num_prefix_pages, const int* prefix_len,
                     const int* block_table, int max_pages, const int* lens, int B, int Hq,
                     int Hkv, int d, int num_pages, int page, float scale, void* O, float* L,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(num_pages, Hkv, page, d);
  if (rc != FA_OK) return rc;
  if ((rc = check_decode(B, Hq, Hkv, d)) != FA_OK) return rc;
  if ((rc = check_scale_value(scale)) != FA_OK) return rc;
  if (num_prefix_pages < 0 || (long long)num_prefix_pages * page > kMaxKeys || max_pages < 0 ||
      (long long)max_pages * page > kMaxKeys)
    return FA_ERR_INVALID_ARG;
  // the kernels count steps of 128 shared and 64 own keys in 32 bits
  const long long groups = (long long)Hkv * ((Hq / Hkv + 15) / 16);
  const int tile = 128 / (Hq / Hkv);
  if ((long long)((B + 2 * tile - 1) / (2 * tile)) * Hkv *
              (((long long)num_prefix_pages * page + 127) / 128) > 0x7fffffffLL ||
      groups * B * (((long long)max_pages * page + 63) / 64) > 0x7fffffffLL)
    return FA_ERR_INVALID_ARG;
  if (!Q || !K_cache || !V_cache || !lens || !O || !L || !workspace) return FA_ERR_INVALID_ARG;
  if ((num_prefix_pages > 0 && (!prefix_pages || !prefix_len)) || (max_pages > 0 && !block_table))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {Q, K_cache, V_cache, static_cast<const void*>(O),
                        static_cast<const void*>(workspace)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(prefix_pages), static_cast<const void*>(prefix_len),
                        static_cast<const void*>(block_table), static_cast<const void*>(lens),
                        static_cast<const void*>(L)})
    if (!is_aligned(p, 4)) return FA_ERR_MISALIGNED;
  const size_t need =
      decode_workspace_bytes(B, Hq, Hkv, d, num_prefix_pages * page, max_pages * page);
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const size_t qn = (size_t)B * Hq * d * 2, cache = cache_bytes(num_pages, Hkv, page, d);
  const Rows ins[] = {bytes_of(Q, qn), bytes_of(K_cache, cache), bytes_of(V_cache, cache),
                      bytes_of(prefix_pages, prefix_pages ? (size_t)num_prefix_pages * 4 : 0),
                      bytes_of(prefix_len, prefix_len ? 4 : 0),
                      bytes_of(block_table, block_table ? (size_t)B * max_pages * 4 : 0),
                      bytes_of(lens, (size_t)B * 4)};
  const Rows outs[] = {bytes_of(O, qn), bytes_of(L, (size_t)B * Hq * 4), bytes_of(workspace, need)};
  for (const Rows& o : outs)
    for (const Rows& i : ins)
      if (rows_overlap(o, i)) return FA_ERR_INVALID_ARG;
  for (int x = 0; x < 3; ++x)
    for (int y = x + 1; y < 3; ++y)
      if (rows_overlap(outs[x], outs[y])) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  DecodeArgs a;
  a.Q = Q;
  a.Kc = K_cache;
  a.Vc = V_cache;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.table = block_table;
  a.lens = lens;
  a.O = O;
  a.L = L;
  a.workspace = workspace;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.prefix_cap = num_prefix_pages;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page = page;
  a.scale = scale;
  return launch_prefix_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                   : FA_ERR_CUDA;
}

}  // extern "C"
