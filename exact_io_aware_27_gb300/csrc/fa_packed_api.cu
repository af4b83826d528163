// Host side of the packed-sequence entry points of include/fa.h: argument checks and
// tensor maps.
#include "fa_check.h"
#include "fa_packed.h"

namespace fa {

namespace {

int packed_map(CUtensorMap* map, const void* base, int rows, int H, int d, long long ld,
               cuuint32_t cols, cuuint32_t box_heads, cuuint32_t box_rows,
               CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {cols, box_heads, box_rows};
  return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                           dims, strides, box, swizzle);
}

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxSequences = 65535;
constexpr long long kMaxRowStride = 1LL << 30;  // elements

int check_plan_sizes(int nseq, int total) {
  if (nseq < 1 || nseq > kMaxSequences || total < 1 || total > kMaxRows)
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int check_heads(int nseq, int total, int Hq, int Hkv, int d) {
  if (Hq < 1 || Hkv < 1 || Hq > 65535 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED_HEAD_DIM;
  // work items are counted in 32 bits
  if (plan_layout(nseq, total).cap[kKeyList] * Hq > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

bool bad_stride(long long ld, int H, int d) {
  return ld < (long long)H * d || ld % 8 != 0 || ld > kMaxRowStride;
}

Rows rows16(const void* p, int rows, int H, int d, long long ld) {
  return rows_of(p, rows, (size_t)H * d * 2, (size_t)ld * 2);
}

}  // namespace

CUresult make_bf16_packed_map(CUtensorMap* map, const void* base, int rows, int H, int d,
                              long long ld, int box_rows, int box_heads) {
  return (CUresult)packed_map(map, base, rows, H, d, ld, 64, (cuuint32_t)box_heads,
                              (cuuint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

CUresult make_bf16_packed_store_map(CUtensorMap* map, void* base, int rows, int H, int d,
                                    long long ld, int box_heads) {
  return (CUresult)packed_map(map, base, rows, H, d, ld, 32, (cuuint32_t)box_heads,
                              (cuuint32_t)(32 / box_heads), CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_packed_plan_bytes(int nseq, int total) {
  if (check_plan_sizes(nseq, total) != FA_OK) return 0;
  return plan_layout(nseq, total).bytes;
}

int fa_packed_plan(const int* cu_seqlens, int nseq, int total, int causal, void* plan,
                   size_t plan_bytes, void* stream) {
  int rc = check_plan_sizes(nseq, total);
  if (rc != FA_OK) return rc;
  if (!cu_seqlens || !plan) return FA_ERR_INVALID_ARG;
  if (!is_aligned(cu_seqlens, 4) || !is_aligned(plan, 16)) return FA_ERR_MISALIGNED;
  const size_t need = plan_layout(nseq, total).bytes;
  if (plan_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  if (rows_overlap(bytes_of(plan, need), bytes_of(cu_seqlens, ((size_t)nseq + 1) * 4)))
    return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  return launch_packed_plan(cu_seqlens, nseq, total, causal ? 1 : 0, plan,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_packed_forward(const void* Q, const void* K, const void* V, long long q_stride,
                      long long k_stride, long long v_stride, int total, int Hq, int Hkv, int d,
                      int causal, float scale, const void* plan, int nseq, void* O, float* L,
                      int fill, void* stream) {
  int rc = check_plan_sizes(nseq, total);
  if (rc != FA_OK) return rc;
  if ((rc = check_heads(nseq, total, Hq, Hkv, d)) != FA_OK) return rc;
  if ((rc = check_scale_value(scale)) != FA_OK) return rc;
  if (!Q || !K || !V || !plan || !O || !L || (fill & ~3)) return FA_ERR_INVALID_ARG;
  if (bad_stride(q_stride, Hq, d) || bad_stride(k_stride, Hkv, d) || bad_stride(v_stride, Hkv, d))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {Q, K, V, plan, static_cast<const void*>(O)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  if (!is_aligned(L, 4)) return FA_ERR_MISALIGNED;
  const Rows ins[] = {rows16(Q, total, Hq, d, q_stride), rows16(K, total, Hkv, d, k_stride),
                      rows16(V, total, Hkv, d, v_stride),
                      bytes_of(plan, plan_layout(nseq, total).bytes)};
  const Rows outs[] = {rows16(O, total, Hq, d, (long long)Hq * d),
                       bytes_of(L, (size_t)Hq * total * 4)};
  for (const Rows& o : outs)
    for (const Rows& i : ins)
      if (rows_overlap(o, i)) return FA_ERR_INVALID_ARG;
  if (rows_overlap(outs[0], outs[1])) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  PackedFwdArgs a;
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.ldv = v_stride;
  a.O = O;
  a.L = L;
  a.plan = plan;
  a.total = total;
  a.nseq = nseq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.causal = causal ? 1 : 0;
  a.fill = fill;
  a.scale = scale;
  return launch_packed_forward(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                    : FA_ERR_CUDA;
}

size_t fa_packed_workspace_bytes(int nseq, int total, int Hq) {
  if (check_plan_sizes(nseq, total) != FA_OK || check_heads(nseq, total, Hq, 1, 8) != FA_OK)
    return 0;
  return packed_bwd_layout(nseq, total, Hq).bytes;
}

int fa_packed_backward(const void* Q, const void* K, const void* V, long long q_stride,
                       long long k_stride, long long v_stride, const void* O, const float* L,
                       const void* dO, int total, int Hq, int Hkv, int d, int causal, float scale,
                       const void* plan, int nseq, void* dQ, void* dK, void* dV,
                       long long dq_stride, long long dk_stride, long long dv_stride, int fill,
                       void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_plan_sizes(nseq, total);
  if (rc != FA_OK) return rc;
  if ((rc = check_heads(nseq, total, Hq, Hkv, d)) != FA_OK) return rc;
  if ((rc = check_scale_value(scale)) != FA_OK) return rc;
  if (!Q || !K || !V || !O || !L || !dO || !plan || !dQ || !dK || !dV || !workspace || (fill & ~7))
    return FA_ERR_INVALID_ARG;
  if (bad_stride(q_stride, Hq, d) || bad_stride(k_stride, Hkv, d) || bad_stride(v_stride, Hkv, d) ||
      bad_stride(dq_stride, Hq, d) || bad_stride(dk_stride, Hkv, d) || bad_stride(dv_stride, Hkv, d))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {Q, K, V, O, dO, plan, static_cast<const void*>(dQ),
                        static_cast<const void*>(dK), static_cast<const void*>(dV),
                        static_cast<const void*>(workspace)})
    if (!is_aligned(p, 16)) return FA_ERR_MISALIGNED;
  if (!is_aligned(L, 4)) return FA_ERR_MISALIGNED;
  const size_t need = fa_packed_workspace_bytes(nseq, total, Hq);
  if (workspace_bytes < need) return FA_ERR_WORKSPACE_TOO_SMALL;
  const Rows ins[] = {rows16(Q, total, Hq, d, q_stride), rows16(K, total, Hkv, d, k_stride),
                      rows16(V, total, Hkv, d, v_stride),
                      rows16(O, total, Hq, d, (long long)Hq * d),
                      rows16(dO, total, Hq, d, (long long)Hq * d),
                      bytes_of(L, (size_t)Hq * total * 4),
                      bytes_of(plan, plan_layout(nseq, total).bytes)};
  const Rows outs[] = {rows16(dQ, total, Hq, d, dq_stride), rows16(dK, total, Hkv, d, dk_stride),
                       rows16(dV, total, Hkv, d, dv_stride), bytes_of(workspace, need)};
  for (const Rows& o : outs)
    for (const Rows& i : ins)
      if (rows_overlap(o, i)) return FA_ERR_INVALID_ARG;
  for (int x = 0; x < 4; ++x)
    for (int y = x + 1; y < 4; ++y)
      if (rows_overlap(outs[x], outs[y])) return FA_ERR_INVALID_ARG;
  if ((rc = require_device()) != FA_OK) return rc;
  PackedBwdArgs a;
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.O = O;
  a.dO = dO;
  a.L = L;
  a.ldq = q_stride;
  a.ldk = k_stride;
  a.ldv = v_stride;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  a.lddq = dq_stride;
  a.lddk = dk_stride;
  a.lddv = dv_stride;
  a.workspace = workspace;
  a.plan = plan;
  a.total = total;
  a.nseq = nseq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.causal = causal ? 1 : 0;
  a.fill = fill;
  a.scale = scale;
  return launch_packed_backward(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

}  // extern "C"
