// A head's row of d channels, divided by its root mean square and turned by its position's
// angles, by a few lanes of a warp.
//
// Eight channels a lane, as two pieces of four (A and B): W = 1 .. 16 lanes share a row, and a
// warp takes 32 / W rows. A lane's channels are chosen so that a pair that is turned together
// lies in one lane: with pairs (i, i + rot / 2) piece A is four channels of the first half
// and B the four that belong to them in the second; with pairs (2 i, 2 i + 1), and behind
// channel rot, A and B are neighbours. Either way the lane's four pairs are turned by angles
// 4 l .. 4 l + 3. Only the sums over a row go through shuffles.
#pragma once

#include <atomic>

#include "fa_rope.h"
#include "sm103.cuh"

namespace fa {

// Lanes of a row: the power of two that holds d / 8.
inline int rope_lanes(int d) {
  int w = 1;
  while (w * 8 < d) w *= 2;
  return w;
}

struct RopeHow {
  const float* cos_sin;
  int positions, rot, interleaved, d;
  float eps, inv_d;
};
// A value that is the same in all lanes, as one that the compiler knows to be: it then takes
// uniform registers for it and what follows from it.
FA_DEV int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// SMs of the current device, asked for once.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}
inline RopeHow rope_how(const fa_rope& h, int d) {
  RopeHow r;
  r.cos_sin = h.cos_sin;
  r.positions = h.positions;
  r.rot = h.cos_sin ? h.rot : 0;
  r.interleaved = h.interleaved;
  r.d = d;
  r.eps = h.eps;
  r.inv_d = 1.f / (float)d;
  return r;
}

struct RopeLane {
  int a, b;        // first channels of its pieces
  bool in, turns;  // it has channels; they are turned
};
// `turned`: whether the row is turned at all (values are not).
FA_DEV RopeLane rope_lane(const RopeHow& h, int l, bool turned) {
  RopeLane r;
  r.in = 8 * l < h.d;
  r.turns = turned && 8 * l < h.rot;
  const bool halves = r.turns && !h.interleaved;
  r.a = halves ? 4 * l : 8 * l;
  r.b = halves ? h.rot / 2 + 4 * l : 8 * l + 4;
  return r;
}

// A lane's eight channels in fp32 as four packed pairs: a[i] and b[i] hold the first and second
// channels of the pairs 2 i and 2 i + 1 that are turned together. INTER: those are neighbours.
struct Pairs {
  uint64_t a[2], b[2];
};
template <bool INTER>
FA_DEV Pairs unpack_pairs(uint2 A, uint2 B) {
  Pairs p;
  if (INTER) {
    p.a[0] = f2pack(bf16_lo(A.x), bf16_lo(A.y));
    p.b[0] = f2pack(bf16_hi(A.x), bf16_hi(A.y));
    p.a[1] = f2pack(bf16_lo(B.x), bf16_lo(B.y));
    p.b[1] = f2pack(bf16_hi(B.x), bf16_hi(B.y));
  } else {
    p.a[0] = f2pack(bf16_lo(A.x), bf16_hi(A.x));
    p.a[1] = f2pack(bf16_lo(A.y), bf16_hi(A.y));
    p.b[0] = f2pack(bf16_lo(B.x), bf16_hi(B.x));
    p.b[1] = f2pack(bf16_lo(B.y), bf16_hi(B.y));
  }
  return p;
}
// The channels of pieces A (x[0 .. 3]) and B.
template <bool INTER>
FA_DEV void channels(const Pairs& p, float (&x)[8]) {
  if (INTER) {
    f2unpack(p.a[0], x[0], x[2]);
    f2unpack(p.b[0], x[1], x[3]);
    f2unpack(p.a[1], x[4], x[6]);
    f2unpack(p.b[1], x[5], x[7]);
  } else {
    f2unpack(p.a[0], x[0], x[1]);
    f2unpack(p.a[1], x[2], x[3]);
    f2unpack(p.b[0], x[4], x[5]);
    f2unpack(p.b[1], x[6], x[7]);
  }
}
FA_DEV uint2 pack4(const float* x) {
  return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
FA_DEV Pairs times(const Pairs& x, uint64_t f) {
  return {{fmul2(x.a[0], f), fmul2(x.a[1], f)}, {fmul2(x.b[0], f), fmul2(x.b[1], f)}};
}
FA_DEV Pairs times(const Pairs& x, const Pairs& y) {
  return {{fmul2(x.a[0], y.a[0]), fmul2(x.a[1], y.a[1])},
          {fmul2(x.b[0], y.b[0]), fmul2(x.b[1], y.b[1])}};
}
FA_DEV Pairs plus(const Pairs& x, const Pairs& y, const Pairs& z) {  // x y + z
  return {{ffma2(x.a[0], y.a[0], z.a[0]), ffma2(x.a[1], y.a[1], z.a[1])},
          {ffma2(x.b[0], y.b[0], z.b[0]), ffma2(x.b[1], y.b[1], z.b[1])}};
}
FA_DEV float dot(const Pairs& x, const Pairs& y) {
  uint64_t v = fmul2(x.a[0], y.a[0]);
  v = ffma2(x.a[1], y.a[1], v);
  v = ffma2(x.b[0], y.b[0], v);
  v = ffma2(x.b[1], y.b[1], v);
  float lo, hi;
  f2unpack(v, lo, hi);
  return lo + hi;
}
FA_DEV uint64_t both(float x) { return f2pack(x, x); }
// 1 / sqrt(x), 2^-22 off at most.
FA_DEV float inverse_root(float x) {
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A warp's rows on their way through shared memory: a ring of stages, each a token's chunk of
// heads, 512 bytes for every pass of the warp's lanes over 32 / W rows, and the angles of its
// position. Rows that are behind the heads hold anything.
constexpr int kAngleBytes = 512;
// Copies `bytes` (at most 512 N) from src to shared memory in the background.
template <int N>
FA_DEV void copy_async(uint32_t to, const void* src, int bytes, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = 16 * lane + 512 * i;
    if (at < bytes) cp_async16(to + at, static_cast<const uint8_t*>(src) + at, 16);
  }
}
FA_DEV float4 ld_shared16f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
FA_DEV uint2 ld_shared8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

template <bool INTER>
FA_DEV void store_row(__nv_bfloat16* row, const Pairs& p, const RopeLane& at) {
  float x[8];
  channels<INTER>(p, x);
  *reinterpret_cast<uint2*>(row + at.a) = pack4(x);
  *reinterpret_cast<uint2*>(row + at.b) = pack4(x + 4);
}

template <bool INTER>
FA_DEV Pairs row_of(uint32_t row, const RopeLane& at) {
  uint2 a = make_uint2(0, 0), b = a;  // a lane without channels adds nothing to its row's sums
  if (at.in) {
    a = ld_shared8(row + 2 * at.a);
    b = ld_shared8(row + 2 * at.b);
  }
  return unpack_pairs<INTER>(a, b);
}

// Sums over the W lanes of a row, of N rows side by side.
template <int W, int N>
FA_DEV void row_sums(float (&v)[N]) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// The lane's angles: cosines and sines of its four pairs, from a position's row of the table in
// shared memory.
struct Angles {
  uint64_t c[2], s[2];
};
FA_DEV Angles rope_angles(uint32_t row, const RopeHow& h, const RopeLane& at, int l) {
  Angles g;
  g.c[0] = g.c[1] = both(1.f);
  g.s[0] = g.s[1] = both(0.f);
  if (at.turns) {
    const float4 c = ld_shared16f(row + 16 * l), s = ld_shared16f(row + 2 * h.rot + 16 * l);
    g.c[0] = f2pack(c.x, c.y);
    g.c[1] = f2pack(c.z, c.w);
    g.s[0] = f2pack(s.x, s.y);
    g.s[1] = f2pack(s.z, s.w);
  }
  return g;
}
// Weight and rotation in one: a' = a ca + b sb, b' = b cb + a sa.
struct Turn {
  uint64_t ca[2], sb[2], cb[2], sa[2];
};
FA_DEV Turn rope_turn(const Angles& g, const Pairs& w) {
  Turn t;
  const uint64_t minus = both(-1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t.ca[i] = fmul2(w.a[i], g.c[i]);
    t.sa[i] = fmul2(w.a[i], g.s[i]);
    t.cb[i] = fmul2(w.b[i], g.c[i]);
    t.sb[i] = fmul2(fmul2(w.b[i], g.s[i]), minus);
  }
  return t;
}
FA_DEV Pairs turned(const Pairs& x, const Turn& t, bool turns) {
  Pairs y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y.a[i] = fmul2(x.a[i], t.ca[i]);
    y.b[i] = fmul2(x.b[i], t.cb[i]);
    if (turns) {
      y.a[i] = ffma2(x.b[i], t.sb[i], y.a[i]);
      y.b[i] = ffma2(x.a[i], t.sa[i], y.b[i]);
    }
  }
  return y;
}
// The rotation back, by the angles alone.
FA_DEV Pairs turned_back(const Pairs& y, const Angles& g, bool turns) {
  if (!turns) return y;
  Pairs x;
  const uint64_t minus = both(-1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.a[i] = ffma2(y.b[i], g.s[i], fmul2(y.a[i], g.c[i]));
    x.b[i] = ffma2(y.a[i], fmul2(g.s[i], minus), fmul2(y.b[i], g.c[i]));
  }
  return x;
}
// N rows of a stage, `step` bytes from row to row, normed (if so; the weight is in `t`) and turned.
template <int W, bool INTER, int N>
FA_DEV void norm_and_turn(Pairs (&y)[N], uint32_t row, uint32_t step, const Turn& t, bool norm,
                          const RopeHow& h, const RopeLane& at) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Pairs x = row_of<INTER>(row + i * step, at);
    if (norm) v[i] = dot(x, x);
    y[i] = turned(x, t, at.turns);
  }
  if (!norm) return;
  row_sums<W, N>(v);
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = times(y[i], both(inverse_root(v[i] * h.inv_d + h.eps)));
}
// The lane's weights, ones without a weight.
template <bool INTER>
FA_DEV Pairs load_weight(const __nv_bfloat16* weight, const RopeLane& at) {
  const uint32_t one = weight ? 0u : 0x3f803f80u;
  uint2 a = make_uint2(one, one), b = a;
  if (weight && at.in) {
    a = *reinterpret_cast<const uint2*>(weight + at.a);
    b = *reinterpret_cast<const uint2*>(weight + at.b);
  }
  return unpack_pairs<INTER>(a, b);
}

// Items (chunks of heads of a token, in order) dealt to the warps of `blocks` thread blocks in
// turn, so that neighbouring warps work on neighbouring rows: pieces of the items' axis, a
// token's chunks in one warp, took 20 % longer. The warps that take part are a number without a
// common divisor with a token's chunks, so that each meets all of a token's chunks, which
// may cost more or less, in turn.
struct Deal {
  int blocks, workers, chunks;  // chunks of a token
  long long items;
  int tokens, rest;             // a round's items: whole tokens, and chunks
};
inline Deal deal(long long tokens, int chunks, int blocks, int warps) {
  Deal d;
  d.blocks = blocks;
  d.chunks = chunks;
  d.items = tokens * chunks;
  d.workers = blocks * warps;
  auto divisor = [](int a, int b) {
    while (b) {
      const int r = a % b;
      a = b;
      b = r;
    }
    return a;
  };
  if (d.items > d.workers)
    while (d.workers > 1 && divisor(d.workers, chunks) != 1) --d.workers;
  d.tokens = d.workers / chunks;
  d.rest = d.workers % chunks;
  return d;
}
// An item, and the same warp's next.
struct Item {
  int token, chunk;
  FA_DEV void advance(const Deal& d) {
    token += d.tokens;
    chunk += d.rest;
    if (chunk >= d.chunks) {
      chunk -= d.chunks;
      ++token;
    }
  }
};
struct Piece {
  Item first;
  int items;
};
// The share of warp `me` of all.
FA_DEV Piece piece_of(const Deal& d, int me) {
  Piece p;
  p.first.token = me / d.chunks;
  p.first.chunk = me - p.first.token * d.chunks;
  p.items = me < d.workers && me < d.items ? (int)((d.items - me - 1) / d.workers) + 1 : 0;
  return p;
}

// Thread blocks of each of N kinds: `most` in all, shared out by items, one at least where there
// is an item, and no more than there are items for.
template <int N>
void share_blocks(int (&blocks)[N], const long long (&items)[N], int most, int warps) {
  long long all = 0;
  for (int i = 0; i < N; ++i) all += items[i];
  for (int i = 0; i < N; ++i) {
    const long long need = (items[i] + warps - 1) / warps;
    long long b = all > 0 ? (long long)((double)most * items[i] / all) : 0;
    if (b < 1) b = 1;
    blocks[i] = (int)(b < need ? b : need);
  }
}

// f.run<W, INTER>() for the lanes of a row of d channels.
template <class F>
cudaError_t with_lanes(const RopeHow& h, const F& f) {
  const bool inter = h.rot > 0 && h.interleaved;
  switch (rope_lanes(h.d)) {
    case 1: return inter ? f.template run<1, true>() : f.template run<1, false>();
    case 2: return inter ? f.template run<2, true>() : f.template run<2, false>();
    case 4: return inter ? f.template run<4, true>() : f.template run<4, false>();
    case 8: return inter ? f.template run<8, true>() : f.template run<8, false>();
    default: return inter ? f.template run<16, true>() : f.template run<16, false>();
  }
}

}  // namespace fa
