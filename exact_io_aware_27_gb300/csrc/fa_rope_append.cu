// Rows of new keys and values into a paged cache, bf16 or 4 bits, with the queries' and keys'
// norm and rotation (fa_rope.cuh) on the way, and rows of the cache in 4 bits back as bf16.
//
// Token t of request i goes to cache position starts[i] + t - cu_seqlens[i], which is row
// (position mod page) of page table[i, position / page] and turns by that position's angles.
// Bound by memory: every row is read once and written once. A warp takes a few heads of one
// token; Q's heads, K's and V's are chunks of one grid, so that a decode step's tokens are
// one short launch. Indices are checked as in fa_cache.cu: a place out of range is not written
// and raises kDeviceIndexBit, and so do bounds that break the rule.
#include "fa_cache4.cuh"
#include "fa_launch.h"
#include "fa_rope.cuh"

namespace fa {

__device__ unsigned int g_rope_append_status;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // rows of a lane in flight

struct Place {
  const int *cu, *starts, *table;
  int total, nseq, max_pages, num_pages, Hkv, page, page_shift;
};

FA_DEV void bad_index() { atomicOr(&g_rope_append_status, kDeviceIndexBit); }

// Whether the bounds break the rule, looked at by thread `me` of `all`.
FA_DEV void check_bounds(const Place& p, long long me, long long all) {
  bool bad = false;
  for (long long i = me; i < p.nseq; i += all) bad |= p.cu[i] > p.cu[i + 1];
  if (me == 0) bad |= p.cu[0] != 0 || p.cu[p.nseq] > p.total;
  if (bad) bad_index();
}

// The request in whose bounds row t lies and the row's position; request -1 behind the last
// one, -2 (reported) where it has no position. The warp searches 32 bounds at a time.
struct Token {
  int request;
  long long pos;
};
FA_DEV Token token_of(const Place& p, int t) {
  const int lane = threadIdx.x & 31;
  if (t >= p.cu[p.nseq]) return {-1, 0};
  int lo = 0, hi = p.nseq;  // the last i of [lo, hi) with cu[i] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned under = __ballot_sync(0xffffffffu, i < hi && p.cu[i] <= t);
    if (under == 0) break;  // bounds that break the rule
    lo += (31 - __clz(under)) * step;
    hi = min(hi, lo + step);
  }
  const int from = p.cu[lo], start = p.starts[lo];
  const long long pos = (long long)start + t - from;
  if (from < 0 || from > t || t >= p.cu[lo + 1] || start < 0) {
    if (lane == 0) bad_index();
    return {-2, 0};
  }
  return {lo, pos};
}
// The page that holds the token's position, or -1 (reported).
FA_DEV int page_of(const Place& p, const Token& k) {
  if (k.pos < (long long)p.max_pages << p.page_shift) {
    const int page = p.table[(long long)k.request * p.max_pages + (k.pos >> p.page_shift)];
    if ((unsigned)page < (unsigned)p.num_pages) return page;
  }
  if ((threadIdx.x & 31) == 0) bad_index();
  return -1;
}

struct AppendParams {
  Place at;
  const __nv_bfloat16 *Q, *K, *V, *wq, *wk;
  __nv_bfloat16 *Qo, *Kc, *Vc;
  uint8_t* cache4;
  long long ldq, ldk, ldv;
  RopeHow how;
  int Hq, q_chunks, kv_chunks, fill;
};

// A row's group of up to 64 channels in 4 bits: the pair, and the codes of the lane's eight
// channels (A in bits 0 .. 15, B above). Every lane of the row takes part. A group with a value
// that is not finite, or whose range is not, is held as NaN.
struct Codes {
  uint32_t pair[2];  // of each group
  uint32_t code;
};
// x to the nearest of the 16 values, of a tie to the even one. The quotient is off by 2^-23
// at most; a remainder on the other side of half a step says so, and exactly half is a tie.
// `up`: a power of two that a very small scale, whose inverse would be infinite, is times.
FA_DEV uint32_t code_of(float x, float lo, float up, float scale, float inv) {
  const float a = (x - lo) * up;
  float c = fminf(fmaxf(rintf(a * inv), 0.f), 15.f);
  const float r2 = 2.f * fmaf(-c, scale, a);
  const bool odd = ((int)c & 1) != 0;
  if (c < 15.f && (r2 > scale || (odd && r2 == scale))) c += 1.f;
  if (c > 0.f && (r2 < -scale || (odd && r2 == -scale))) c -= 1.f;
  return (uint32_t)c;
}
template <int W, int G>
FA_DEV Codes quantize8(const float (&x)[8], const RopeLane& at) {
  Codes out;
  out.code = 0;
  float lo[2], scale[2], up[2], inv[2];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const bool a = at.in && at.a / 64 == j, b = at.in && at.b / 64 == j;
    float mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < 4 ? !a : !b) continue;
      mn = fminf(mn, x[i]);
      mx = fmaxf(mx, x[i]);
      zero += x[i] * 0.f;  // NaN where x is not finite
    }
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      zero += __shfl_xor_sync(0xffffffffu, zero, o);
    }
    lo[j] = __bfloat162float(__float2bfloat16_rn(mn)) + zero;
    const float range = mx - lo[j];
    scale[j] = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(fmaxf(range, 0.f), 15.f)));
    if (!(range < INFINITY) || !(fabsf(lo[j]) < INFINITY)) scale[j] = lo[j] = NAN;
    out.pair[j] = pack_bf16(scale[j], lo[j]);
    up[j] = scale[j] < 0x1p-100f ? 0x1p100f : 1.f;
    scale[j] *= up[j];
    inv[j] = __fdiv_rn(1.f, scale[j]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = G == 1 ? 0 : (i < 4 ? at.a : at.b) >> 6;
    const float s = j ? scale[G - 1] : scale[0];
    if (s > 0.f)
      out.code |= code_of(x[i], j ? lo[G - 1] : lo[0], j ? up[G - 1] : up[0], s,
                          j ? inv[G - 1] : inv[0])
                  << (4 * i);
  }
  return out;
}

// FOUR: the cache in 4 bits.
template <int W, bool FOUR>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int R = 32 / W, G = W == 16 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % W;
  const int y = (int)blockIdx.y;
  const int kind = y < p.q_chunks ? 0 : y < p.q_chunks + p.kv_chunks ? 1 : 2;  // Q, K, V
  const int chunk = y - (kind > 0 ? p.q_chunks : 0) - (kind > 1 ? p.kv_chunks : 0);
  const int h0 = chunk * kUnroll * R + lane / W;
  const int heads = kind == 0 ? p.Hq : p.at.Hkv, d = p.how.d;
  const __nv_bfloat16* const x_of = kind == 0 ? p.Q : kind == 1 ? p.K : p.V;
  const __nv_bfloat16* const weight = kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr;
  const long long ld = kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv;
  const RopeLane at = rope_lane(p.how, l, kind < 2);
  grid_wait();
  grid_launch_dependents();
  if (kind == 1 && chunk == 0)
    check_bounds(p.at, (long long)blockIdx.x * kThreads + threadIdx.x,
                 (long long)gridDim.x * kThreads);
  float w[8];
  load_weight(w, weight, at);
  for (int t = (int)blockIdx.x * kWarps + warp; t < p.at.total; t += (int)gridDim.x * kWarps) {
    uint2 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      a[u] = b[u] = make_uint2(0, 0);
      const int h = h0 + u * R;
      if (h < heads && at.in) {
        const __nv_bfloat16* row = x_of + (long long)t * ld + h * d;
        a[u] = ld_stream8(row + at.a);
        b[u] = ld_stream8(row + at.b);
      }
    }
    const Token token = token_of(p.at, t);
    bool ok = token.request >= 0;
    int page = 0;
    if (ok && kind > 0) {
      page = page_of(p.at, token);
      ok = page >= 0;
    }
    if (ok && p.how.rot > 0 && token.pos >= p.how.positions) {
      if (lane == 0) bad_index();
      ok = false;
    }
    if (!ok) {
      if (kind != 0 || !p.fill) continue;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * R;
        if (h >= heads || !at.in) continue;
        __nv_bfloat16* row = p.Qo + ((long long)t * heads + h) * d;
        *reinterpret_cast<uint2*>(row + at.a) = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(row + at.b) = make_uint2(0, 0);
      }
      continue;
    }
    const int pos = (int)token.pos, in_page = pos & (p.at.page - 1);
    Angles g{};
    if (kind < 2) g = rope_angles(p.how, at, l, pos);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * R;
      if (h - lane / W >= heads) break;  // warp-uniform
      float x[8];
      unpack8(x, a[u], b[u]);
      if (weight) norm8<W>(x, w, p.how);
      if (kind < 2) turn8(x, p.how, at, g, 1.f);
      const bool in = h < heads && at.in;
      if (kind == 0 || !FOUR) {
        if (!in) continue;
        __nv_bfloat16* row =
            kind == 0 ? p.Qo + ((long long)t * heads + h) * d
                      : (kind == 1 ? p.Kc : p.Vc) +
                            ((((long long)page * heads + h) << p.at.page_shift) + in_page) * d;
        *reinterpret_cast<uint2*>(row + at.a) = pack4(x);
        *reinterpret_cast<uint2*>(row + at.b) = pack4(x + 4);
      } else {
        const Codes c = quantize8<W, G>(x, at);
        if (!in) continue;
        uint32_t* const block = reinterpret_cast<uint32_t*>(
            p.cache4 + ((((long long)page * heads + h) << p.at.page_shift) + (in_page & ~15)) *
                           (G * kBlock4 / kRows4));
        const int r = in_page & 15;
        if (kind == 1) {
          uint16_t* const half = reinterpret_cast<uint16_t*>(block);
          half[2 * k_word4(G, r, at.a >> 6, (at.a >> 3) & 7) + ((at.a >> 2) & 1)] =
              (uint16_t)c.code;
          half[2 * k_word4(G, r, at.b >> 6, (at.b >> 3) & 7) + ((at.b >> 2) & 1)] =
              (uint16_t)(c.code >> 16);
        } else {
          block[v_word4(G, r, at.a >> 6, (at.a >> 3) & 7)] = c.code;
        }
        if (l < G) block[pair_word4(G, r, kind - 1, l)] = c.pair[G == 2 && l ? 1 : 0];
      }
    }
  }
}

struct ReadParams {
  Place at;
  const uint8_t* cache;
  __nv_bfloat16 *K, *V;
  int d, fill;
};

// A lane turns one word of eight codes into 16 bytes: 16 lanes take K and V of a row of G = 1,
// 32 of G = 2. Sixteen tokens a block, so that most of a cache block's sectors, which the rows
// of V share, are used from L1.
template <int G>
__global__ void __launch_bounds__(512) cache4_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int LANES = 16 * G, R = 32 / LANES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES;
  const int kv = l / (8 * G), j = l / 8 % G, word = l % 8, c0 = 64 * j + 8 * word;
  grid_wait();
  grid_launch_dependents();
  check_bounds(p.at, (long long)blockIdx.x * 512 + threadIdx.x, (long long)gridDim.x * 512);
  const int t = (int)blockIdx.x * 16 + warp;
  if (t >= p.at.total) return;
  __nv_bfloat16* const out = (kv ? p.V : p.K) + (long long)t * p.at.Hkv * p.d + c0;
  const Token token = token_of(p.at, t);
  const int page = token.request >= 0 ? page_of(p.at, token) : -1;
  if (page < 0) {
    if (p.fill && c0 < p.d)
      for (int h = lane / LANES; h < p.at.Hkv; h += R)
        *reinterpret_cast<uint4*>(out + h * p.d) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int in_page = (int)token.pos & (p.at.page - 1), r = in_page & 15;
  const int at = kv ? v_word4(G, r, j, word) : k_word4(G, r, j, word);
  const int pair_at = pair_word4(G, r, kv, j);
#pragma unroll 4
  for (int h = lane / LANES; h < p.at.Hkv; h += R) {
    const uint32_t* block = reinterpret_cast<const uint32_t*>(
        p.cache + ((((long long)page * p.at.Hkv + h) << p.at.page_shift) + (in_page & ~15)) *
                      (G * kBlock4 / kRows4));
    const uint32_t code = block[at], pair = block[pair_at];
    const float scale = bf16_lo(pair), lo = bf16_hi(pair);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pack_bf16(fmaf((float)(code >> (8 * i) & 15), scale, lo),
                       fmaf((float)(code >> (8 * i + 4) & 15), scale, lo));
    if (c0 < p.d) *reinterpret_cast<uint4*>(out + h * p.d) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

Place place_of(const PlaceArgs& a) {
  Place p;
  p.cu = a.cu_seqlens;
  p.starts = a.starts;
  p.table = a.table;
  p.total = a.total;
  p.nseq = a.nseq;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.Hkv = a.Hkv;
  p.page = a.page;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  return p;
}

struct Append {
  AppendParams& p;
  bool four;
  cudaStream_t stream;
  template <int W>
  cudaError_t run() const {
    const int per = kUnroll * (32 / W);
    p.q_chunks = p.Q ? ceil_div(p.Hq, per) : 0;
    p.kv_chunks = ceil_div(p.at.Hkv, per);
    return launch_early(four ? rope_append_kernel<W, true> : rope_append_kernel<W, false>,
                        dim3((unsigned)ceil_div(p.at.total, kWarps),
                             (unsigned)(p.q_chunks + 2 * p.kv_chunks)),
                        kThreads, 0, stream, p);
  }
};

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  AppendParams p{};
  p.at = place_of(a.at);
  p.Q = static_cast<const __nv_bfloat16*>(a.Q);
  p.K = static_cast<const __nv_bfloat16*>(a.K);
  p.V = static_cast<const __nv_bfloat16*>(a.V);
  p.wq = static_cast<const __nv_bfloat16*>(a.how.q_weight);
  p.wk = static_cast<const __nv_bfloat16*>(a.how.k_weight);
  p.Qo = static_cast<__nv_bfloat16*>(a.Qo);
  p.Kc = static_cast<__nv_bfloat16*>(a.Kc);
  p.Vc = static_cast<__nv_bfloat16*>(a.Vc);
  p.cache4 = static_cast<uint8_t*>(a.cache4);
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.how = rope_how(a.how, a.at.d);
  p.Hq = a.Hq;
  p.fill = a.fill;
  return with_lanes(a.at.d, Append{p, a.cache4 != nullptr, s});
}

cudaError_t launch_cache4_read(const Cache4ReadArgs& a, cudaStream_t s) {
  ReadParams p;
  p.at = place_of(a.at);
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.K = static_cast<__nv_bfloat16*>(a.K);
  p.V = static_cast<__nv_bfloat16*>(a.V);
  p.d = a.at.d;
  p.fill = a.fill;
  return launch_early(groups4(p.d) == 2 ? cache4_read_kernel<2> : cache4_read_kernel<1>,
                      dim3((unsigned)ceil_div(p.at.total, 16)), 512, 0, s, p);
}

cudaError_t rope_append_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_append_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_rope_append_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
