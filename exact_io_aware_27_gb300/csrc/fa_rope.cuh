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

FA_DEV uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p)
               : "memory");
  return v;
}
// Channels A (x[0..3]) and B (x[4..7]) of a row.
FA_DEV void unpack8(float (&x)[8], uint2 a, uint2 b) {
  x[0] = bf16_lo(a.x);
  x[1] = bf16_hi(a.x);
  x[2] = bf16_lo(a.y);
  x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(b.x);
  x[5] = bf16_hi(b.x);
  x[6] = bf16_lo(b.y);
  x[7] = bf16_hi(b.y);
}
FA_DEV uint2 pack4(const float* x) {
  return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

template <int W>
FA_DEV float row_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's angles at position `pos`: cosines and sines of its four pairs.
struct Angles {
  float4 c, s;
};
FA_DEV Angles rope_angles(const RopeHow& h, const RopeLane& at, int l, int pos) {
  Angles g;
  g.c = make_float4(1.f, 1.f, 1.f, 1.f);
  g.s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at.turns) {
    const float* row = h.cos_sin + (size_t)pos * h.rot;
    g.c = *reinterpret_cast<const float4*>(row + 4 * l);
    g.s = *reinterpret_cast<const float4*>(row + h.rot / 2 + 4 * l);
  }
  return g;
}
FA_DEV void turn(float& a, float& b, float c, float s) {
  const float x = a * c - b * s;
  b = b * c + a * s;
  a = x;
}
// The lane's pairs turned (sign = -1: back).
FA_DEV void turn8(float (&x)[8], const RopeHow& h, const RopeLane& at, const Angles& g,
                  float sign) {
  if (!at.turns) return;
  if (h.interleaved) {
    turn(x[0], x[1], g.c.x, sign * g.s.x);
    turn(x[2], x[3], g.c.y, sign * g.s.y);
    turn(x[4], x[5], g.c.z, sign * g.s.z);
    turn(x[6], x[7], g.c.w, sign * g.s.w);
  } else {
    turn(x[0], x[4], g.c.x, sign * g.s.x);
    turn(x[1], x[5], g.c.y, sign * g.s.y);
    turn(x[2], x[6], g.c.z, sign * g.s.z);
    turn(x[3], x[7], g.c.w, sign * g.s.w);
  }
}
// x / root mean square, times the weight w; every lane of a row takes part.
template <int W>
FA_DEV void norm8(float (&x)[8], const float (&w)[8], const RopeHow& h) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += x[i] * x[i];
  const float r = rsqrtf(row_sum<W>(s) * h.inv_d + h.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
}
FA_DEV void load_weight(float (&w)[8], const __nv_bfloat16* weight, const RopeLane& at) {
  uint2 a = make_uint2(0, 0), b = a;
  if (weight && at.in) {
    a = *reinterpret_cast<const uint2*>(weight + at.a);
    b = *reinterpret_cast<const uint2*>(weight + at.b);
  }
  unpack8(w, a, b);
}

// f.run<W>() for the lanes of a row of d channels.
template <class F>
cudaError_t with_lanes(int d, const F& f) {
  switch (rope_lanes(d)) {
    case 1: return f.template run<1>();
    case 2: return f.template run<2>();
    case 4: return f.template run<4>();
    case 8: return f.template run<8>();
    default: return f.template run<16>();
  }
}

}  // namespace fa
