// Host side of the entry points of include/fa.h between projection and attention (norm and
// rotation) and of the cache in 4 bits: argument checks.
#include "fa_cache4.cuh"
#include "fa_check.h"
#include "fa_decode.h"
#include "fa_rope.h"

namespace fa {

namespace {

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxSequences = 65535;
constexpr long long kMaxRowStride = 1LL << 30;  // elements
constexpr long long kMaxKeys = 1LL << 30;       // keys a table row can name

int check_heads(int H, int d) {
  if (H < 1 || H > 65535) return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED_HEAD_DIM;
  return FA_OK;
}
int check_how(const fa_rope* h, int d) {
  if (!h || !std::isfinite(h->eps) || h->eps < 0.f) return FA_ERR_INVALID_ARG;
  if (h->cos_sin && (h->positions < 1 || h->rot < 8 || h->rot > d || h->rot % 8 != 0))
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(h->q_weight, 8) || !is_aligned(h->k_weight, 8) || !is_aligned(h->cos_sin, 16))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}
bool stride_ok(long long ld, int H, int d) {
  return ld >= (long long)H * d && ld % 8 == 0 && ld <= kMaxRowStride;
}
// What `how` points to, as inputs.
struct HowRows {
  Rows r[3];
};
HowRows rows_of_how(const fa_rope* h, int d) {
  return {{bytes_of(h->q_weight, h->q_weight ? (size_t)d * 2 : 0),
           bytes_of(h->k_weight, h->k_weight ? (size_t)d * 2 : 0),
           bytes_of(h->cos_sin, h->cos_sin ? (size_t)h->positions * h->rot * 4 : 0)}};
}
bool any_overlap(const Rows* outs, int nout, const Rows* ins, int nin) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (rows_overlap(outs[o], ins[i])) return true;
    for (int i = o + 1; i < nout; ++i)
      if (rows_overlap(outs[o], outs[i])) return true;
  }
  return false;
}
int from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

int check_cache(int num_pages, int Hkv, int page, int d) {
  if (num_pages < 1) return FA_ERR_INVALID_ARG;
  const int rc = check_heads(Hkv, d);
  if (rc != FA_OK) return rc;
  if (page < kMinPage || page > kMaxPage || (page & (page - 1)) != 0) return FA_ERR_INVALID_ARG;
  if ((long long)num_pages * Hkv > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  return FA_OK;
}
size_t cache4_bytes(int num_pages, int Hkv, int page, int d) {
  return (size_t)num_pages * Hkv * page * fa_cache4_row_bytes(d);
}
int check_place(const int* cu, const int* starts, const int* table, int total, int nseq,
                int max_pages, int page) {
  if (total < 1 || total > kMaxRows || nseq < 1 || nseq > kMaxSequences || max_pages < 1 ||
      (long long)max_pages * page > kMaxKeys || !cu || !starts || !table)
    return FA_ERR_INVALID_ARG;
  for (const int* p : {cu, starts, table})
    if (!is_aligned(p, 4)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// fa_rope_append into Kc and Vc, or fa_cache4_append into cache4.
int append(const void* Q, const void* K, const void* V, long long q_stride, long long k_stride,
           long long v_stride, int total, int Hq, const int* cu, const int* starts, int nseq,
           const int* table, int max_pages, const fa_rope* how, void* Qo, int fill, void* Kc,
           void* Vc, void* cache4, int num_pages, int Hkv, int page, int d, void* stream) {
  int rc = check_cache(num_pages, Hkv, page, d);
  if (rc != FA_OK) return rc;
  if ((rc = check_place(cu, starts, table, total, nseq, max_pages, page)) != FA_OK) return rc;
  if (Hq < 0 || Hq > 65535 || (Hq > 0) != (Q != nullptr) || (Hq > 0) != (Qo != nullptr))
    return FA_ERR_INVALID_ARG;
  if (!K || !V || (cache4 ? Kc || Vc : !Kc || !Vc)) return FA_ERR_INVALID_ARG;
  if ((rc = check_how(how, d)) != FA_OK) return rc;
  if ((fill & ~1) != 0 || (Hq > 0 && !stride_ok(q_stride, Hq, d)) ||
      !stride_ok(k_stride, Hkv, d) || !stride_ok(v_stride, Hkv, d))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {Q, K, V, static_cast<const void*>(Qo), static_cast<const void*>(Kc),
                        static_cast<const void*>(Vc), static_cast<const void*>(cache4)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  const size_t qw = (size_t)Hq * d * 2, kw = (size_t)Hkv * d * 2;
  const HowRows h = rows_of_how(how, d);
  const Rows ins[] = {rows_of(Q, Q ? total : 0, qw, (size_t)q_stride * 2),
                      rows_of(K, total, kw, (size_t)k_stride * 2),
                      rows_of(V, total, kw, (size_t)v_stride * 2),
                      bytes_of(cu, ((size_t)nseq + 1) * 4),
                      bytes_of(starts, (size_t)nseq * 4),
                      bytes_of(table, (size_t)nseq * max_pages * 4),
                      h.r[0],
                      h.r[1],
                      h.r[2]};
  const size_t rows = (size_t)num_pages * Hkv * page;
  const Rows outs[] = {bytes_of(Qo, Qo ? (size_t)total * qw : 0),
                       cache4 ? bytes_of(cache4, cache4_bytes(num_pages, Hkv, page, d))
                              : bytes_of(Kc, rows * d * 2),
                       bytes_of(Vc, Vc ? rows * d * 2 : 0)};
  if (any_overlap(outs, 3, ins, 9)) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  RopeAppendArgs a;
  a.at = {cu, starts, table, total, nseq, max_pages, num_pages, Hkv, d, page};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.Qo = Qo;
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.ldv = v_stride;
  a.Kc = Kc;
  a.Vc = Vc;
  a.cache4 = cache4;
  a.Hq = Hq;
  a.fill = fill;
  a.how = *how;
  return from_cuda(launch_rope_append(a, static_cast<cudaStream_t>(stream)));
}

int check_decode4(int B, int Hq, int Hkv, int d) {
  if (B < 1 || B > kMaxBatch || Hq < 1 || Hq > 65535 || Hkv < 1 || Hq % Hkv != 0 ||
      Hq / Hkv > 128 || (long long)B * Hq > 0x7fffffffLL)
    return FA_ERR_INVALID_ARG;
  return check_heads(Hkv, d);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_qk_norm_rope(const void* Q, const void* K, long long q_stride, long long k_stride,
                    int total, int Hq, int Hkv, int d, const int* positions, const fa_rope* how,
                    void* Qo, void* Ko, long long qo_stride, long long ko_stride, void* stream) {
  int rc;
  if ((rc = check_heads(Hq, d)) != FA_OK || (rc = check_heads(Hkv, d)) != FA_OK) return rc;
  if ((rc = check_how(how, d)) != FA_OK) return rc;
  if (total < 1 || total > kMaxRows || !Q || !K || !Qo || !Ko || (how->cos_sin && !positions) ||
      !stride_ok(q_stride, Hq, d) || !stride_ok(qo_stride, Hq, d) ||
      !stride_ok(k_stride, Hkv, d) || !stride_ok(ko_stride, Hkv, d))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {Q, K, static_cast<const void*>(Qo), static_cast<const void*>(Ko)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  if (!is_aligned(positions, 4)) return FA_ERR_MISALIGNED;
  const size_t qw = (size_t)Hq * d * 2, kw = (size_t)Hkv * d * 2;
  const HowRows h = rows_of_how(how, d);
  const bool q_in_place = Q == Qo && q_stride == qo_stride;
  const bool k_in_place = K == Ko && k_stride == ko_stride;
  const Rows q = rows_of(Q, total, qw, (size_t)q_stride * 2);
  const Rows k = rows_of(K, total, kw, (size_t)k_stride * 2);
  const Rows outs[] = {rows_of(Qo, total, qw, (size_t)qo_stride * 2),
                       rows_of(Ko, total, kw, (size_t)ko_stride * 2)};
  const Rows ins[] = {bytes_of(positions, how->cos_sin ? (size_t)total * 4 : 0), h.r[0], h.r[1],
                      h.r[2]};
  if (any_overlap(outs, 2, ins, 4) || (!q_in_place && rows_overlap(outs[0], q)) ||
      rows_overlap(outs[0], k) || (!k_in_place && rows_overlap(outs[1], k)) ||
      rows_overlap(outs[1], q))
    return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  RopeArgs a;
  a.Q = Q;
  a.K = K;
  a.Qo = Qo;
  a.Ko = Ko;
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.ldqo = qo_stride;
  a.ldko = ko_stride;
  a.positions = positions;
  a.total = total;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.how = *how;
  return from_cuda(launch_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_workspace_bytes(int Hq, int Hkv, int d) {
  if (check_heads(Hq, d) != FA_OK || check_heads(Hkv, d) != FA_OK) return 0;
  return rope_workspace_bytes(d);
}

int fa_qk_norm_rope_backward(const void* dQo, const void* dKo, long long dqo_stride,
                             long long dko_stride, const void* Q, const void* K,
                             long long q_stride, long long k_stride, int total, int Hq, int Hkv,
                             int d, const int* positions, const fa_rope* how, void* dQ, void* dK,
                             long long dq_stride, long long dk_stride, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int rc;
  if ((rc = check_heads(Hq, d)) != FA_OK || (rc = check_heads(Hkv, d)) != FA_OK) return rc;
  if ((rc = check_how(how, d)) != FA_OK) return rc;
  const bool wq = how->q_weight != nullptr, wk = how->k_weight != nullptr;
  if (total < 1 || total > kMaxRows || !dQo || !dKo || !dQ || !dK ||
      (how->cos_sin && !positions) || (wq && (!Q || !dq_weight)) || (wk && (!K || !dk_weight)) ||
      ((wq || wk) && !workspace))
    return FA_ERR_INVALID_ARG;
  if (!stride_ok(dqo_stride, Hq, d) || !stride_ok(dq_stride, Hq, d) ||
      (wq && !stride_ok(q_stride, Hq, d)) || !stride_ok(dko_stride, Hkv, d) ||
      !stride_ok(dk_stride, Hkv, d) || (wk && !stride_ok(k_stride, Hkv, d)))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {dQo, dKo, wq ? Q : nullptr, wk ? K : nullptr, static_cast<const void*>(dQ),
                        static_cast<const void*>(dK),
                        wq || wk ? static_cast<const void*>(workspace) : nullptr})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  for (const void* p :
       {static_cast<const void*>(positions), static_cast<const void*>(wq ? dq_weight : nullptr),
        static_cast<const void*>(wk ? dk_weight : nullptr)})
    if (!is_aligned(p, 4)) return FA_ERR_MISALIGNED;
  const size_t need = wq || wk ? rope_workspace_bytes(d) : 0;
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const size_t qw = (size_t)Hq * d * 2, kw = (size_t)Hkv * d * 2;
  const HowRows h = rows_of_how(how, d);
  const Rows ins[] = {rows_of(dQo, total, qw, (size_t)dqo_stride * 2),
                      rows_of(dKo, total, kw, (size_t)dko_stride * 2),
                      rows_of(Q, wq ? total : 0, qw, (size_t)q_stride * 2),
                      rows_of(K, wk ? total : 0, kw, (size_t)k_stride * 2),
                      bytes_of(positions, how->cos_sin ? (size_t)total * 4 : 0),
                      h.r[0],
                      h.r[1],
                      h.r[2]};
  const Rows outs[] = {rows_of(dQ, total, qw, (size_t)dq_stride * 2),
                       rows_of(dK, total, kw, (size_t)dk_stride * 2),
                       bytes_of(dq_weight, wq ? (size_t)d * 4 : 0),
                       bytes_of(dk_weight, wk ? (size_t)d * 4 : 0), bytes_of(workspace, need)};
  if (any_overlap(outs, 5, ins, 8)) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  RopeBackwardArgs a;
  a.dQo = dQo;
  a.dKo = dKo;
  a.Q = Q;
  a.K = K;
  a.dQ = dQ;
  a.dK = dK;
  a.lddqo = dqo_stride;
  a.lddko = dko_stride;
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.lddq = dq_stride;
  a.lddk = dk_stride;
  a.positions = positions;
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  a.partial = static_cast<float*>(workspace);
  a.total = total;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.how = *how;
  return from_cuda(launch_rope_backward(a, static_cast<cudaStream_t>(stream)));
}

int fa_rope_append(const void* Q, const void* K, const void* V, long long q_stride,
                   long long k_stride, long long v_stride, int total, int Hq,
                   const int* cu_seqlens, const int* starts, int nseq, const int* block_table,
                   int max_pages, const fa_rope* how, void* Qo, int fill, void* K_cache,
                   void* V_cache, int num_pages, int Hkv, int page, int d, void* stream) {
  if (!K_cache || !V_cache) return FA_ERR_INVALID_ARG;
  return append(Q, K, V, q_stride, k_stride, v_stride, total, Hq, cu_seqlens, starts, nseq,
                block_table, max_pages, how, Qo, fill, K_cache, V_cache, nullptr, num_pages, Hkv,
                page, d, stream);
}

size_t fa_cache4_row_bytes(int d) {
  return d < 8 || d > 128 || d % 8 != 0 ? 0 : (size_t)groups4(d) * (kBlock4 / kRows4);
}

int fa_cache4_append(const void* Q, const void* K, const void* V, long long q_stride,
                     long long k_stride, long long v_stride, int total, int Hq,
                     const int* cu_seqlens, const int* starts, int nseq, const int* block_table,
                     int max_pages, const fa_rope* how, void* Qo, int fill, void* cache,
                     int num_pages, int Hkv, int page, int d, void* stream) {
  if (!cache) return FA_ERR_INVALID_ARG;
  return append(Q, K, V, q_stride, k_stride, v_stride, total, Hq, cu_seqlens, starts, nseq,
                block_table, max_pages, how, Qo, fill, nullptr, nullptr, cache, num_pages, Hkv,
                page, d, stream);
}

int fa_cache4_read(const void* cache, int num_pages, int Hkv, int page, int d,
                   const int* cu_seqlens, const int* starts, int nseq, const int* block_table,
                   int max_pages, int total, void* K, void* V, int fill, void* stream) {
  int rc = check_cache(num_pages, Hkv, page, d);
  if (rc != FA_OK) return rc;
  if ((rc = check_place(cu_seqlens, starts, block_table, total, nseq, max_pages, page)) != FA_OK)
    return rc;
  if (!cache || !K || !V || (fill & ~1) != 0) return FA_ERR_INVALID_ARG;
  for (const void* p : {cache, static_cast<const void*>(K), static_cast<const void*>(V)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  const size_t bytes = (size_t)total * Hkv * d * 2;
  const Rows ins[] = {bytes_of(cache, cache4_bytes(num_pages, Hkv, page, d)),
                      bytes_of(cu_seqlens, ((size_t)nseq + 1) * 4),
                      bytes_of(starts, (size_t)nseq * 4),
                      bytes_of(block_table, (size_t)nseq * max_pages * 4)};
  const Rows outs[] = {bytes_of(K, bytes), bytes_of(V, bytes)};
  if (any_overlap(outs, 2, ins, 4)) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  Cache4ReadArgs a;
  a.at = {cu_seqlens, starts, block_table, total, nseq, max_pages, num_pages, Hkv, d, page};
  a.cache = cache;
  a.K = K;
  a.V = V;
  a.fill = fill;
  return from_cuda(launch_cache4_read(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_cache4_workspace_bytes(int B, int Hq, int Hkv, int d, int capacity) {
  if (check_decode4(B, Hq, Hkv, d) != FA_OK || capacity < 0 || capacity > kMaxKeys) return 0;
  return decode4_workspace_bytes(B, Hq, Hkv, d, capacity);
}

int fa_cache4_decode(const void* Q, const void* cache, const int* block_table, int max_pages,
                     const int* lens, int B, int Hq, int Hkv, int d, int num_pages, int page,
                     float scale, void* O, float* L, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int rc = check_cache(num_pages, Hkv, page, d);
  if (rc != FA_OK) return rc;
  if ((rc = check_decode4(B, Hq, Hkv, d)) != FA_OK) return rc;
  if ((rc = check_scale_value(scale)) != FA_OK) return rc;
  if (max_pages < 0 || (long long)max_pages * page > kMaxKeys) return FA_ERR_INVALID_ARG;
  // the kernels count chunks of keys in 32 bits
  if ((long long)Hkv * ((Hq / Hkv + 7) / 8) * B * (((long long)max_pages * page + 63) / 64) >
      0x7fffffffLL)
    return FA_ERR_INVALID_ARG;
  if (!Q || !cache || !lens || !O || !L || !workspace || (max_pages > 0 && !block_table))
    return FA_ERR_INVALID_ARG;
  for (const void* p :
       {Q, cache, static_cast<const void*>(O), static_cast<const void*>(workspace)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(lens),
                        static_cast<const void*>(L)})
    if (!is_aligned(p, 4)) return FA_ERR_MISALIGNED;
  const size_t need = decode4_workspace_bytes(B, Hq, Hkv, d, max_pages * page);
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const size_t qn = (size_t)B * Hq * d * 2;
  const Rows ins[] = {bytes_of(Q, qn), bytes_of(cache, cache4_bytes(num_pages, Hkv, page, d)),
                      bytes_of(block_table, block_table ? (size_t)B * max_pages * 4 : 0),
                      bytes_of(lens, (size_t)B * 4)};
  const Rows outs[] = {bytes_of(O, qn), bytes_of(L, (size_t)B * Hq * 4), bytes_of(workspace, need)};
  if (any_overlap(outs, 3, ins, 4)) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  Decode4Args a;
  a.Q = Q;
  a.cache = cache;
  a.table = block_table;
  a.lens = lens;
  a.O = O;
  a.L = L;
  a.workspace = workspace;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page = page;
  a.scale = scale;
  return from_cuda(launch_decode4(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
