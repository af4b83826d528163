// Rows of new keys and values into a paged cache, bf16 or 4 bits, with the queries' and keys'
// norm and rotation (fa_rope.cuh) on the way, and rows of the cache in 4 bits back as bf16.
//
// Token t of request i goes to cache position starts[i] + t - cu_seqlens[i], which is row
// (position mod page) of page table[i, position / page] and turns by that position's angles.
// Bound by memory: every row is read once and written once. A warp takes a few heads of Q, K or
// V of one token after another, all warps side by side, and looks a request up only where
// another one begins. 32768 rows of 32/8 heads, d = 128, into the bf16 cache: 137 us (805 MB,
// 5.9 TB/s, 87 % of the measured copy rate). Into the cache in 4 bits the codes cost about as many
// instructions as norm and rotation together: 8192 rows 49 us (177 MB, 26 at the copy rate). No
// unit is at its limit there (67 % of the issue slots, 47 % of the ALU's); a pass over two rows
// is one chain of sums, exchanges, extremes and quotients, and 20 warps an SM do not hide it (of
// 6.6 cycles from one instruction of a warp to its next, 1.7 are latencies of a fixed length,
// 1.2 lost to another warp, 0.8 shuffles and shared memory, 0.7 a busy pipe, 0.6 memory). Indices are checked as in fa_cache.cu: a place out of range is not written and
// raises kDeviceIndexBit, and so do bounds that break the rule.
#include "fa_cache4.cuh"
#include "fa_launch.h"
#include "fa_rope.cuh"

namespace fa {

__device__ unsigned int g_rope_append_status;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Passes of a warp's lanes over the rows of an item, stages of a warp's ring.
constexpr int kPasses = 4, kStages = 3;
constexpr int kStage = 512 * kPasses + kAngleBytes;
// Blocks on an SM, as many as the registers allow; 4 bits want 120.
constexpr int kPerSm = 6, kPerSm4 = 5;

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

// Where rows go. A warp meets them in order, so that most lie in the request of the one before.
struct Cursor {
  int request = -1;    // of the row: -1 behind the last request, -2 without a place (reported)
  int end = 0;         // of the request's rows
  long long shift = 0; // from row to position

  // Moves on to row t. The search looks at 32 bounds at a time.
  FA_DEV void to(const Place& p, int t) {
    if (request >= 0 && t < end) return;
    const int lane = threadIdx.x & 31;
    request = -1;
    if (t >= p.cu[p.nseq]) return;
    int lo = 0, hi = p.nseq;  // the last i of [lo, hi) with cu[i] <= t
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const unsigned under = __ballot_sync(0xffffffffu, i < hi && p.cu[i] <= t);
      if (under == 0) break;  // bounds that break the rule
      lo += (31 - __clz(under)) * step;
      hi = min(hi, lo + step);
    }
    const int from = uniform(p.cu[lo]), start = uniform(p.starts[lo]);
    end = uniform(p.cu[lo + 1]);
    request = uniform(lo);
    shift = (long long)start - from;
    if (from < 0 || from > t || t >= end || start < 0) {
      if (lane == 0) bad_index();
      request = -2;
    }
  }
};
// The page that holds position pos of a request, as the table has it, or -1.
FA_DEV int table_page(const Place& p, int request, long long pos) {
  const long long index = pos >> p.page_shift;
  return index < p.max_pages ? p.table[(long long)request * p.max_pages + index] : -1;
}
FA_DEV bool page_ok(const Place& p, int page) {
  if ((unsigned)page < (unsigned)p.num_pages) return true;
  if ((threadIdx.x & 31) == 0) bad_index();
  return false;
}

struct AppendSide {  // Q, K or V
  const __nv_bfloat16 *x, *w;
  __nv_bfloat16* y;  // Qo or a bf16 cache
  long long ld;
  int heads, chunks;
};
struct AppendParams {
  Place at;
  AppendSide side[3];
  Deal deal;  // of the chunks of Q's heads, K's and V's of each token
  uint8_t* cache4;
  RopeHow how;
  int fill;
};

// Chunks of a token: Q's, then K's, then V's (kinds 0, 1, 2).
FA_DEV int kind_of(const AppendParams& p, int c) {
  return c < p.side[0].chunks ? 0 : c < p.side[0].chunks + p.side[1].chunks ? 1 : 2;
}
FA_DEV int chunk_of(const AppendParams& p, int c) {  // within the kind
  if (c >= p.side[0].chunks) c -= p.side[0].chunks;
  else return c;
  return c >= p.side[1].chunks ? c - p.side[1].chunks : c;
}

FA_DEV float min_nan(float a, float b, float c) {  // NaN if one is
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
FA_DEV float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Eight neighbouring channels of a group in 4 bits, of N rows side by side; SAME lanes have the
// group. A group with a value that is not finite, or whose range is not, is held as NaN.
//
// Quotients are a product with an inverse, and one correction by the remainder: off by far
// less than half a step of fp32, so that they round as the exact quotients do, and a tie
// between two codes, which is a number of few bits, comes out exactly.
struct Codes {
  uint32_t pair, code;
};
template <int SAME, int N>
FA_DEV void quantize8(Codes (&out)[N], const float (&x)[N][8], bool in) {
  float lo[N], hi[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    lo[n] = min_nan(min_nan(x[n][0], x[n][1], x[n][2]), x[n][3], x[n][4]);
    hi[n] = max_nan(max_nan(x[n][0], x[n][1], x[n][2]), x[n][3], x[n][4]);
    lo[n] = min_nan(min_nan(lo[n], x[n][5], x[n][6]), x[n][7], x[n][7]);
    hi[n] = max_nan(max_nan(hi[n], x[n][5], x[n][6]), x[n][7], x[n][7]);
    if (!in) {
      lo[n] = INFINITY;
      hi[n] = -INFINITY;
    }
  }
#pragma unroll
  for (int o = SAME / 2; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      lo[n] = min_nan(lo[n], lo[n], __shfl_xor_sync(0xffffffffu, lo[n], o));
      hi[n] = max_nan(hi[n], hi[n], __shfl_xor_sync(0xffffffffu, hi[n], o));
    }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float least = __bfloat162float(__float2bfloat16_rn(lo[n]));
    const float range = hi[n] - least, span = max_nan(range, 0.f, 0.f);
    constexpr float k15 = 1.f / 15.f;
    const float fifteenth = fmaf(fmaf(-15.f, span * k15, span), k15, span * k15);
    float scale = __bfloat162float(__float2bfloat16_rn(fifteenth));
    if (!(range < INFINITY) || !(fabsf(least) < INFINITY)) scale = least = NAN;
    out[n].pair = pack_bf16(scale, least);
    // A power of two keeps the inverse of a very small scale finite; codes are 0 where it is 0.
    const float up = scale < 0x1p-100f ? 0x1p100f : 1.f;
    scale *= up;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    if (!(scale > 0.f)) inv = 0.f;
    const uint64_t up2 = both(up), from = both(-least * up), inv2 = both(inv), down = both(-scale);
    // 1.5 2^23 + e is a number whose lowest bits are e's nearest integer; sixteen times the sum
    // of those before and it are the codes so far, and a constant that wraps around.
    uint32_t code = 0;
#pragma unroll
    for (int i = 6; i >= 0; i -= 2) {
      const uint64_t a = ffma2(f2pack(x[n][i], x[n][i + 1]), up2, from), q = fmul2(a, inv2);
      float e0, e1;
      f2unpack(ffma2(ffma2(q, down, a), inv2, q), e0, e1);
      e0 = fminf(fmaxf(e0, 0.f), 15.f) + 12582912.f;
      e1 = fminf(fmaxf(e1, 0.f), 15.f) + 12582912.f;
      code = (code * 16u + __float_as_uint(e1)) * 16u + __float_as_uint(e0);
    }
    // 0x4b400000 (1.5 2^23) times 1 + 16 + ... + 16^7 modulo 2^32
    out[n].code = code - 0x4b400000u * 0x11111111u;
  }
}

// FOUR: the cache in 4 bits. An item is kPasses * 32 / W heads of one token;
// requests and pages are looked up and angles copied two items ahead.
template <int W, bool INTER, bool FOUR>
__global__ void __launch_bounds__(kThreads, FOUR ? kPerSm4 : kPerSm)
    rope_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int R = 32 / W, U = kPasses, S = kStages, G = W == 16 ? 2 : 1;
  __shared__ __align__(16) uint8_t rings[kWarps * S * kStage];
  __shared__ float4 natural[FOUR ? kWarps : 1][128];  // 2 R rows in fp32, channels in order
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, l = lane % W, seg = lane / W;
  const int d = p.how.d;
  const Piece mine = piece_of(p.deal, (int)blockIdx.x * kWarps + warp);
  const uint32_t ring = smem_u32(rings) + warp * S * kStage, row = 2 * d;
  // where a lane's channels lie in a row that is turned and in one that is not
  const RopeLane at_turned = rope_lane(p.how, l, true), at_plain = rope_lane(p.how, l, false);
  grid_wait();
  Item next = mine.first, it = next;
  Cursor cur;
  struct Where {
    int pos, page;  // pos -1: no place; page as the table has it
  } where[S];       // of the items from the one worked on
  int put = 0;      // items whose copies are issued
  uint32_t to = ring;
  auto issue = [&]() {
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) where[k] = where[k + 1];
    if (put < mine.items) {
      const int kind = kind_of(p, next.chunk);
      const AppendSide& s = p.side[kind];
      const int t = next.token, h = chunk_of(p, next.chunk) * U * R;
      copy_async<U>(to, s.x + (long long)t * s.ld + h * d, min(U * R, s.heads - h) * 2 * d, lane);
      cur.to(p.at, t);
      Where& w = where[S - 1];
      const long long pos = t + cur.shift;
      w.pos = cur.request >= 0 ? (int)min(pos, 0x7fffffffLL) : -1;
      w.page = w.pos >= 0 && kind > 0 ? table_page(p.at, cur.request, pos) : 0;
      if (w.pos == 0x7fffffff || (p.how.rot && w.pos >= p.how.positions)) {
        if (lane == 0) bad_index();
        w.pos = -1;
      }
      if (p.how.rot && kind < 2 && w.pos >= 0)
        copy_async<1>(to + 512 * U, p.how.cos_sin + (size_t)w.pos * p.how.rot, 4 * p.how.rot, lane);
      next.advance(p.deal);
      if (++put == mine.items) grid_launch_dependents();
    }
    cp_async_commit();
    to = to == ring + (S - 1) * kStage ? ring : to + kStage;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  check_bounds(p.at, (long long)blockIdx.x * kThreads + threadIdx.x,
               (long long)gridDim.x * kThreads);
  uint32_t stage = ring;
  for (int i = 0; i < mine.items; ++i, it.advance(p.deal)) {
    cp_async_wait<S - 2>();
    __syncwarp();  // the stage has landed for every lane, and the last one is read
    issue();
    const int kind = kind_of(p, it.chunk);
    const AppendSide& s = p.side[kind];
    const int heads = s.heads, t = it.token, h0 = chunk_of(p, it.chunk) * U * R + seg;
    const int pos = where[0].pos, page = where[0].page;
    const bool norm = s.w != nullptr;
    const RopeLane at = kind < 2 ? at_turned : at_plain;
    const uint32_t rows = stage + seg * row;
    Turn turn{};
    if (kind < 2)
      turn = rope_turn(rope_angles(stage + 512 * U, p.how, at, l), load_weight<INTER>(s.w, at));
    stage = stage == ring + (S - 1) * kStage ? ring : stage + kStage;
    if (pos < 0 || (kind > 0 && !page_ok(p.at, page))) {
      if (kind == 0 && p.fill) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h0 + u * R < heads && at.in) {
            __nv_bfloat16* const out = s.y + ((long long)t * heads + h0 + u * R) * d;
            *reinterpret_cast<uint2*>(out + at.a) = make_uint2(0, 0);
            *reinterpret_cast<uint2*>(out + at.b) = make_uint2(0, 0);
          }
      }
    } else if (kind == 0 || !FOUR) {
      // of head h0, and from head to head of this token
      __nv_bfloat16* const out =
          kind == 0 ? s.y + ((long long)t * heads + h0) * d
                    : s.y + ((((long long)page * heads + h0) << p.at.page_shift) +
                             (pos & (p.at.page - 1))) * d;
      const long long step = kind == 0 ? d : (long long)d << p.at.page_shift;
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        if (h0 - seg + u * R >= heads) break;  // warp-uniform
        if (kind < 2) {
          Pairs y[2];
          norm_and_turn<W, INTER, 2>(y, rows + u * R * row, R * row, turn, norm, p.how, at);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (h0 + (u + k) * R < heads && at.in)
              store_row<INTER>(out + (u + k) * R * step, y[k], at);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (h0 + (u + k) * R < heads && at.in) {
              const uint32_t from = rows + (u + k) * R * row;
              *reinterpret_cast<uint2*>(out + (u + k) * R * step + at.a) =
                  ld_shared8(from + 2 * at.a);
              *reinterpret_cast<uint2*>(out + (u + k) * R * step + at.b) =
                  ld_shared8(from + 2 * at.b);
            }
        }
      }
    } else {
      const int in_page = pos & (p.at.page - 1), r = in_page & 15, j = l >> 3;
      uint8_t* const block =
          p.cache4 + ((((long long)page * heads + h0) << p.at.page_shift) + (in_page & ~15)) *
                         (G * kBlock4 / kRows4);
      const long long step = (long long)(G * kBlock4 / kRows4) << p.at.page_shift;
      const int word = kind == 1 ? k_word4(G, r, j, l & 7) : v_word4(G, r, j, l & 7);
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        if (h0 - seg + u * R >= heads) break;  // warp-uniform
        float x[2][8];
        if (kind == 1) {
          Pairs y[2];
          norm_and_turn<W, INTER, 2>(y, rows + u * R * row, R * row, turn, norm, p.how, at);
          channels<INTER>(y[0], x[0]);
          channels<INTER>(y[1], x[1]);
          if (!INTER && p.how.rot > 0) {  // channels 8 l .. 8 l + 7 from the lanes that have them
            float* const to = reinterpret_cast<float*>(natural[warp]) + seg * 8 * W;
            __syncwarp();
            if (at.in) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                *reinterpret_cast<float4*>(to + 256 * k + at.a) =
                    make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
                *reinterpret_cast<float4*>(to + 256 * k + at.b) =
                    make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float4 a = *reinterpret_cast<const float4*>(to + 256 * k + 8 * l);
              const float4 b = *reinterpret_cast<const float4*>(to + 256 * k + 8 * l + 4);
              x[k][0] = a.x, x[k][1] = a.y, x[k][2] = a.z, x[k][3] = a.w;
              x[k][4] = b.x, x[k][5] = b.y, x[k][6] = b.z, x[k][7] = b.w;
            }
          }
        } else {
          channels<false>(row_of<false>(rows + u * R * row, at), x[0]);
          channels<false>(row_of<false>(rows + (u + 1) * R * row, at), x[1]);
        }
        Codes code[2];
        quantize8<(W < 8 ? W : 8), 2>(code, x, at.in);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (h0 + (u + k) * R < heads && at.in) {
            uint32_t* const words = reinterpret_cast<uint32_t*>(block + (u + k) * R * step);
            words[word] = code[k].code;
            if ((l & 7) == 0) words[pair_word4(G, r, kind - 1, j)] = code[k].pair;
          }
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

// A word of eight codes as eight values in bf16.
FA_DEV uint4 values8(uint32_t code, uint32_t pair) {
  const float scale = bf16_lo(pair), lo = bf16_hi(pair);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16(fmaf((float)(code >> (8 * i) & 15), scale, lo),
                     fmaf((float)(code >> (8 * i + 4) & 15), scale, lo));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// A warp takes a head of 16 rows of `total`, and of those the runs that lie in one block of the
// cache: it reads the block's words in their order and writes eight channels a lane, 128 bytes
// of four rows at a time. Neighbouring warps take the heads of the same rows, so that whole
// rows leave together (70700 rows, 8 heads, d = 128: 64 us, 378 MB, 5.9 TB/s; with the heads of
// a row one after another in a warp 74).
template <int G>
__global__ void __launch_bounds__(kThreads) cache4_read_kernel(const __grid_constant__ ReadParams p) {
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int w = lane & 7, q = lane >> 3;  // word of a group; row of four
  grid_wait();
  grid_launch_dependents();
  check_bounds(p.at, (long long)blockIdx.x * kThreads + threadIdx.x,
               (long long)gridDim.x * kThreads);
  const long long all = (long long)((p.at.total + 15) / 16) * p.at.Hkv;
  for (long long i = (long long)blockIdx.x * kWarps + warp; i < all;
       i += (long long)gridDim.x * kWarps) {
    const int t0 = (int)(i / p.at.Hkv) * 16, t1 = min(t0 + 16, p.at.total);
    const int h = (int)(i % p.at.Hkv);
    Cursor cur;
    for (int t = t0; t < t1;) {
      cur.to(p.at, t);
      const long long pos = t + cur.shift;
      const int page = cur.request >= 0 ? table_page(p.at, cur.request, pos) : -1;
      if (cur.request < 0 || !page_ok(p.at, page)) {
        if (p.fill && 8 * lane < p.d) {
          const long long to = ((long long)t * p.at.Hkv + h) * p.d + 8 * lane;
          *reinterpret_cast<uint4*>(p.K + to) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(p.V + to) = make_uint4(0, 0, 0, 0);
        }
        ++t;
        continue;
      }
      const int in_page = (int)pos & (p.at.page - 1), r0 = in_page & 15;
      const int n = min(min(16 - r0, cur.end - t), t1 - t);  // rows r0 .. r0 + n - 1 of the block
      const uint32_t* const block = reinterpret_cast<const uint32_t*>(
          p.cache + ((((long long)page * p.at.Hkv + h) << p.at.page_shift) + (in_page & ~15)) *
                        (G * kBlock4 / kRows4));
      uint32_t k[4][G], kp[4][G], vp[4][G];
      uint4 v[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        v[j] = *reinterpret_cast<const uint4*>(block + v_word4(G, 2 * q, j, w));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          k[i][j] = block[k_word4(G, 4 * i + q, j, w)];
          kp[i][j] = block[pair_word4(G, 4 * i + q, 0, j)];
          // V's four words are of rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9
          vp[i][j] = block[pair_word4(G, 2 * q + (i & 1) + 8 * (i >> 1), 1, j)];
        }
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int c = 64 * j + 8 * w;
        const uint32_t words[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        if (c >= p.d) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rk = 4 * i + q - r0, rv = 2 * q + (i & 1) + 8 * (i >> 1) - r0;
          if (rk >= 0 && rk < n)
            *reinterpret_cast<uint4*>(p.K + ((long long)(t + rk) * p.at.Hkv + h) * p.d + c) =
                values8(k[i][j], kp[i][j]);
          if (rv >= 0 && rv < n)
            *reinterpret_cast<uint4*>(p.V + ((long long)(t + rv) * p.at.Hkv + h) * p.d + c) =
                values8(words[i], vp[i][j]);
        }
      }
      t += n;
    }
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
  template <int W, bool INTER>
  cudaError_t run() const {
    const int per = kPasses * (32 / W);
    int chunks = 0;
    for (int i = 0; i < 3; ++i) {
      p.side[i].chunks = ceil_div(p.side[i].heads, per);
      chunks += p.side[i].chunks;
    }
    const long long need = ((long long)p.at.total * chunks + kWarps - 1) / kWarps;
    const int most = sm_count() * (four ? kPerSm4 : kPerSm), blocks = (int)(need < most ? need : most);
    p.deal = deal(p.at.total, chunks, blocks, kWarps);
    return launch_early(four ? rope_append_kernel<W, INTER, true> : rope_append_kernel<W, INTER, false>,
                        dim3((unsigned)blocks), kThreads, 0, stream, p);
  }
};

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  AppendParams p{};
  p.at = place_of(a.at);
  const void *const x[3] = {a.Q, a.K, a.V}, *const w[3] = {a.how.q_weight, a.how.k_weight, nullptr};
  void* const y[3] = {a.Qo, a.Kc, a.Vc};
  const long long ld[3] = {a.ldq, a.ldk, a.ldv};
  for (int i = 0; i < 3; ++i) {
    p.side[i].x = static_cast<const __nv_bfloat16*>(x[i]);
    p.side[i].w = static_cast<const __nv_bfloat16*>(w[i]);
    p.side[i].y = static_cast<__nv_bfloat16*>(y[i]);
    p.side[i].ld = ld[i];
    p.side[i].heads = i == 0 ? a.Hq : a.at.Hkv;
  }
  p.cache4 = static_cast<uint8_t*>(a.cache4);
  p.how = rope_how(a.how, a.at.d);
  p.fill = a.fill;
  return with_lanes(p.how, Append{p, a.cache4 != nullptr, s});
}

cudaError_t launch_cache4_read(const Cache4ReadArgs& a, cudaStream_t s) {
  ReadParams p;
  p.at = place_of(a.at);
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.K = static_cast<__nv_bfloat16*>(a.K);
  p.V = static_cast<__nv_bfloat16*>(a.V);
  p.d = a.at.d;
  p.fill = a.fill;
  const long long warps = (long long)ceil_div(p.at.total, 16) * p.at.Hkv;
  const long long blocks = (warps + kWarps - 1) / kWarps;
  return launch_early(groups4(p.d) == 2 ? cache4_read_kernel<2> : cache4_read_kernel<1>,
                      dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), kThreads, 0, s, p);
}

cudaError_t rope_append_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_append_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_rope_append_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
