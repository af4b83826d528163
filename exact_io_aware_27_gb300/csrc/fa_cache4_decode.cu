// Decode attention over the paged cache in 4 bits (fa_cache4.cuh): one new token for each of B
// requests over its own keys.
//
//   split kernel  the keys of all (row tile, key/value head, request) units lie end to end in
//                 chunks, each unit behind two steps for its start and end, and every worker
//                 takes an even piece of that axis (Split), whatever the lengths. A worker is a
//                 block with chunks of 128 keys, 32 of them per warp, or, where there are many
//                 units, a warp with chunks of 32. A unit that lies in one piece is finished
//                 there; else each piece gives a part (o, e) as in fa_prefix.cu.
//   join kernel   joins the parts, and fills the rows of requests without keys.
//
// Warp-level products (16 x 8 x 16) with the keys as the 16 rows and the queries of a
// key/value head as the 8 columns, so that the few queries of grouped heads fill them:
//   S = K Q^T      = sum over groups of scale (q . code) + min (sum q), in fp32
//   O^T = V^T P^T  = (P scale) . code, and P min, summed in fp32
// A code alone in the lowest four bits of a 16-bit number is, read as fp16, code 2^-24, and in
// the next four code 2^-20: two logical operations and half a shift turn two codes into
// operands, exactly, without an addition. Q is brought to a largest value of 256 to 512 by a
// power of two for each query, and P scale, rounded to fp16, is taken relative to a reference
// that follows its largest values, as the softmax's own reference follows the scores: what
// loses bits is below 2^-14 of the largest term, and off by 2^-25 of it at most. The two groups
// have references of their own, since they are outputs of their own: with one for both, a group
// whose values were 2^20 times smaller than the other's was off by percents.
// Each warp has a ring of two stages of 32 keys, two bulk copies each; the values of a run (a
// unit, or the part of it in a worker's piece) that are the same in all lanes are told to be so
// (uniform()), which takes them out of the registers that the products need. That, and 32 keys
// at a time instead of 16, is what 12 warps an SM with 168 registers each allow (d > 64, up to 8
// queries; pieces of blocks spill 32 bytes, single warps none). With 16 queries it is 8 warps
// of 254 registers, and 32 to 64 bytes spilled.
//
// Bound by chains of dependent instructions with few warps to hide them, just before memory:
// about 520 a warp for 32 keys (d = 128), 176 of them to take codes apart. No unit is at its
// limit (55 % of the issue slots, 56 % of the ALU's, 27 % of the products'); of the 4.9 cycles
// from one instruction of a warp to its next, 1.3 are latencies of a fixed length, 0.8 lost to
// another warp, 0.7 a busy pipe, and 0.4 waits for memory. 256 requests of up to 8192 keys, 32/8
// heads, d = 128 (1.2 GB): 203 us, 5.9 TB/s, 87 % of the measured copy rate; with all keys in L2
// it takes as long. The first form, 16 keys a step with the codes as bf16 values 128 + code,
// took 385 us. 32 requests of up to 4096 keys (73 MB): 23.7 us, of which 3.5 until the first keys
// are there, 13 at that rate, and the rest the ends of units and the join.
#include "fa_cache4.cuh"
#include "fa_decode.h"
#include "fa_launch.h"
#include "fa_rope.cuh"
#include "fa_split.cuh"

namespace fa {

__device__ unsigned int g_decode4_status;

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kRescale = 8.f;  // the reference maximum moves when passed by 2^8
// P scale in units of a reference, of each query and group: it moves when passed by kMost, a
// number that fp16 still has. Its inverse is held: at most kMostInverse, which fp32 still has
// times a weight (2^8, or 2^16 where the scores' own rounding is a step of that size), and no less
// than the least normal number, with which P scale, 2^140 at most, is one that fp16 has.
constexpr float kMost = 4096.f, kMostInverse = 0x1p110f, kLeastInverse = 0x1p-126f;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;              // keys of a warp's stage: two blocks of the cache
constexpr int kChunk = kKeys * kWarps;  // keys of a block's step
// Steps that a unit's start and end count as, besides (1000 requests of up to 1000 keys, 8/2
// heads, d = 128, on whole blocks: 50 us; with 1 step 53, with 3 51; on single warps 3 are as
// good as 2).
constexpr int kRunSteps = 2;
// From so many units on, each warp has its own: a unit's start and end cost a warp what they cost
// a block, and there is nothing to join between warps. With fewer, pieces of a unit are so many
// that joining them costs more (d = 128; 128 units of up to 4096 keys: 18 us with blocks, 20 with
// warps; 256: 23 and 23; 2000 of up to 1000 keys: 50 and 43; 8000 of up to 500: 111 and 74).
constexpr int kSoloUnits = 320;
constexpr int kMaxSms = 160;         // slots are reserved for this many SMs

// Blocks of the split kernel per SM at most, by the registers: 12 warps of 168, or 8 of more for
// two tiles of queries.
constexpr int per_sm(int NT) { return NT == 1 ? 3 : 2; }
// A unit of at most so many chunks is one block's, where all units find a block at once: then
// nothing is joined, and a call is one launch (2 requests of up to 300 keys, 8/2 heads, d = 64:
// 3.9 us in a graph, with two launches 6).
constexpr int kWholeChunks = 8;

struct Sizes {
  int B, Hq, Hkv, per_kv, d;
  int tile;        // queries of a tile, 8 or 16
  int row_tiles;   // tiles of a key/value head's queries
  int slot_rows;
  bool solo;       // a worker of the split is a warp, not a block
  int chunk;       // keys of a step
  int workers;     // of the split
  long long units, steps;  // steps of all units, at most
  float *o, *e;    // [slot][slot_rows][d], [slot][slot_rows]
  int* first;      // [B + 1] steps before each request
};

Sizes sizes_of(int B, int Hq, int Hkv, int d, int capacity) {
  Sizes s{};
  s.B = B;
  s.Hq = Hq;
  s.Hkv = Hkv;
  s.per_kv = Hq / Hkv;
  s.d = d;
  // A tile of 16 queries takes 1.75 times as long as one of 8 (64 requests of up to 8192 keys,
  // 4 x 16 heads, d = 128: 55 us against 63; of 2 x 20 heads, two tiles against three: 53
  // against 49).
  s.tile = 7 * ceil_div(s.per_kv, 16) < 4 * ceil_div(s.per_kv, 8) ? 16 : 8;
  s.row_tiles = ceil_div(s.per_kv, s.tile);
  s.slot_rows = s.per_kv < s.tile ? s.per_kv : s.tile;
  s.units = (long long)Hkv * s.row_tiles * B;
  auto steps = [&](int chunk) {
    return capacity ? s.units * (((long long)capacity + chunk - 1) / chunk + kRunSteps) : 0;
  };
  s.solo = s.units >= kSoloUnits && steps(kKeys) <= 0x7fffffff;  // counted in 32 bits
  s.chunk = s.solo ? kKeys : kChunk;
  s.steps = steps(s.chunk);
  return s;
}
size_t lay_out(Sizes* s, void* base) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = p + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  // no fewer for more keys, with which warps may not be counted any longer
  const size_t workers = (size_t)kMaxSms * per_sm(1) * (s->units >= kSoloUnits ? kWarps : 1);
  const size_t slots = 2 * ((size_t)s->steps < workers ? (size_t)s->steps : workers);
  s->o = reinterpret_cast<float*>(take(slots * s->slot_rows * s->d * 4));
  s->e = reinterpret_cast<float*>(take(slots * s->slot_rows * 4));
  s->first = reinterpret_cast<int*>(take(((size_t)s->B + 1) * 4));
  return at;
}

struct DecodeParams {
  Sizes s;
  const __nv_bfloat16* Q;
  const uint8_t* cache;
  const int *table, *lens;
  __nv_bfloat16* O;
  float* L;
  int max_pages, num_pages, page_shift;
  float scale_log2;
};

FA_DEV int keys_of(const DecodeParams& p, int b) {
  return max(0, min(p.lens[b], p.max_pages << p.page_shift));
}
// Steps of a unit of so many keys.
FA_DEV int steps_of(int keys, int chunk) {
  return keys > 0 ? (keys + chunk - 1) / chunk + kRunSteps : 0;
}

// The workers' pieces of all units, of so many steps for each tile of queries. A warp's has
// kLeastSteps, so that a long request among short ones is not in more parts than the keys are
// worth (one of 131072 keys among 320: 40 us; without a least piece 47, and with 8 steps 32, but
// 300 requests of up to 1000 keys, 8/2 heads, 21 instead of 20).
constexpr unsigned kLeastSteps = 4;
FA_DEV Split split_of(const Sizes& s, int steps) {
  const unsigned all = (unsigned)(s.Hkv * s.row_tiles) * (unsigned)steps;
  const unsigned most = (unsigned)s.workers;
  return Split(all, s.solo ? min(most, (all + kLeastSteps - 1) / kLeastSteps) : most);
}

template <int G, int NT>
struct Cfg {
  static constexpr int BLOCK = G * kBlock4;
  static constexpr int STAGE = 2 * BLOCK;
  static constexpr int STAGES = 2;
  static constexpr int ROWS = 8 * NT;      // queries of a tile
  static constexpr int D = 64 * G;
  static constexpr int RINGS = kWarps * STAGES * STAGE;
  static constexpr int PARTS = kWarps * ROWS * D * 4;
  static constexpr int BYTES = RINGS + PARTS;  // then first[B + 1]
};

// A lane's part of a stage, where `mine`: `bytes` (a multiple of 16) from global to shared memory,
// both 16-byte aligned, counted on `bar`, or an arrival alone where there is no source.
// Predicated, without branches.
FA_DEV void bulk_load(bool mine, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\tsetp.ne.u32 p, %0, 0;\n\tsetp.ne.and.u64 q, %2, 0, p;\n\t"
      "setp.eq.and.u64 r, %2, 0, p;\n\t"
      "@r mbarrier.arrive.shared::cta.b64 _, [%4];\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %3;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2], %3, [%4];"
      "\n\t}" ::"r"((uint32_t)mine),
      "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
FA_DEV uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// Codes e of the halves of a word in fp16, times 2^-24 (e even) or 2^-20.
FA_DEV uint32_t codes(uint32_t w, int e) {
  return (e < 2 ? w : w >> 8) & (e & 1 ? 0x00f000f0u : 0x000f000fu);
}
FA_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
FA_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
FA_DEV void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 1 / x, 2^-23 off at most. Exact quotients call a routine with registers of its own: with them
// the two ends of a unit took 1.5 us longer (32 requests of up to 4096 keys, 32/8 heads, d = 128:
// 25.5 us against 23.5), and d > 64 spilled.
FA_DEV float about_inverse(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The power of two at or below x, at least 2^-118.
FA_DEV float power_of_two(float x) {
  return fmaxf(__uint_as_float(__float_as_uint(x) & 0x7f800000u), 0x1p-118f);
}
// An 8 x 8 matrix of 16-bit values, a row of it in four lanes, transposed.
FA_DEV uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A stage's words of one lane: 16 keys of K (rows g and g + 8), of V (rows 2 t, 2 t + 1, 2 t + 8,
// 2 t + 9), and the pairs of rows g and g + 8.
template <int G>
struct Words {
  uint32_t k[2][2 * G], v[G][4], pair[2][2 * G];
  FA_DEV void load(uint32_t stage, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      if constexpr (G == 2) {
        const uint4 a = ld_shared16(stage + 4 * k_word4(G, r, 0, 2 * t));
        const uint4 b = ld_shared16(stage + 4 * pair_word4(G, r, 0, 0));
        k[h][0] = a.x, k[h][1] = a.y, k[h][2] = a.z, k[h][3] = a.w;
        pair[h][0] = b.x, pair[h][1] = b.y, pair[h][2] = b.z, pair[h][3] = b.w;
      } else {
        const uint2 a = ld_shared8(stage + 4 * k_word4(G, r, 0, 2 * t));
        const uint2 b = ld_shared8(stage + 4 * pair_word4(G, r, 0, 0));
        k[h][0] = a.x, k[h][1] = a.y;
        pair[h][0] = b.x, pair[h][1] = b.y;
      }
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const uint4 a = ld_shared16(stage + 4 * v_word4(G, 2 * t, j, g));
      v[j][0] = a.x, v[j][1] = a.y, v[j][2] = a.z, v[j][3] = a.w;
    }
  }
};

// The queries of a tile and their running softmax over the keys that a warp has seen. Lane
// (g, t) has columns (queries) 2 t and 2 t + 1 of every 8 x 8 accumulator. Scores are in units
// of a query's own: c is what makes them exponents of 2. Queries so large that c has no room in
// fp32 (2^24 of it are the codes') are raised: their scores are kRaise times as large, c as
// much smaller.
constexpr float kRaise = 0x1p64f;
template <int G, int NT>
struct Tile {
  uint32_t q[NT][G][4][2];  // every second pair divided by 16
  float qs[NT][G][2];       // sums of a query over a group, times 2^-24
  float c[NT][2];
  unsigned raised[NT];      // bit 4 r: query r is
  float o[NT][G][4][4];     // channels 64 j + 8 g + 2 i + (e / 2), query 2 t + e % 2
  float z[NT][G][2];        // sums of P min, of this lane's keys
  // reference, what is added to scores (minus it, or 0 if there is none yet), weight sum of this
  // lane's keys, and the score that moves the reference
  float m[NT][2], ref[NT][2], l[NT][2], top[NT][2];
  float v_inv[NT][G][2];  // o is in units of its inverse

  // The lane's part of the queries' rows.
  struct Raw {
    uint4 w[NT][G][2];
    FA_DEV void load(const __nv_bfloat16* Q, int rows, int d, int lane) {
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c0 = 64 * j + 16 * t + 8 * u, row = 8 * n + g;
            w[n][j][u] = make_uint4(0, 0, 0, 0);
            if (row < rows && c0 < d) w[n][j][u] = *reinterpret_cast<const uint4*>(Q + row * d + c0);
          }
    }
  };
  FA_DEV void start(const Raw& raw, float scale_log2, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 (&w)[G][2] = raw.w[n];
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          for (uint32_t x : {w[j][u].x, w[j][u].y, w[j][u].z, w[j][u].w})
            most = fmaxf(most, fmaxf(fabsf(bf16_lo(x)), fabsf(bf16_hi(x))));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // 2^-8 of the query's power of two; an infinite entry stays one
      const float unit = most < INFINITY ? power_of_two(most) * 0x1p-8f : 1.f;
      // 2^-e from 2^e
      const float inv = __uint_as_float(0x7f000000u - __float_as_uint(unit));
      float to_log2 = unit * 0x1p24f * scale_log2;
      const bool raise = !(to_log2 < 0x1p120f);
      if (raise) to_log2 = unit * (0x1p24f / kRaise) * scale_log2;
      raised[n] = __ballot_sync(0xffffffffu, raise);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t x[4] = {w[j][u].x, w[j][u].y, w[j][u].z, w[j][u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // channels e and e + 4
            float a = e & 1 ? bf16_hi(x[e / 2]) : bf16_lo(x[e / 2]);
            float b = e & 1 ? bf16_hi(x[2 + e / 2]) : bf16_lo(x[2 + e / 2]);
            a *= inv;
            b *= inv;
            sum += a + b;
            q[n][j][2 * u + e / 2][e & 1] =
                e & 1 ? pack_f16(a * 0.0625f, b * 0.0625f) : pack_f16(a, b);
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= raise ? 0x1p-24f * kRaise : 0x1p-24f;
        qs[n][j][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        qs[n][j][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][j][i][e] = 0.f;
        z[n][j][0] = z[n][j][1] = 0.f;
        v_inv[n][j][0] = v_inv[n][j][1] = kMostInverse;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // never 0, which would make -infinity times it NaN
        c[n][e] = fmaxf(__shfl_sync(0xffffffffu, to_log2, 8 * t + 4 * e), 0x1p-149f);
        m[n][e] = top[n][e] = -INFINITY;
        ref[n][e] = l[n][e] = 0.f;
      }
    }
  }

  // The first `keys` of a stage's two blocks, side by side: one block's chain of products,
  // weights and products leaves half of the issue slots empty.
  FA_DEV void step(const Words<G> (&w)[2], int keys, int lane) {
    const int g = lane >> 2;
    float s[2][NT][4], sv[2][2][G], mv[2][2][G], acc[2][NT][G][4];
    // The products of a sum one after another wait for each other: four sums in turn.
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint32_t w0 = w[k].k[0][2 * j + x / 2], w1 = w[k].k[1][2 * j + x / 2];
          const int e = 2 * (x & 1);
          const uint32_t a[4] = {codes(w0, e), codes(w1, e), codes(w0, e + 1), codes(w1, e + 1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (x == 0)
              mma_f16_first(acc[k][n][j], a, q[n][j][x][0], q[n][j][x][1]);
            else
              mma_f16(acc[k][n][j], a, q[n][j][x][0], q[n][j][x][1]);
          }
        }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (raised[n] != 0) {  // warp-uniform
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float by = raised[n] >> (8 * (lane & 3) + 4 * (i & 1)) & 1 ? kRaise : 1.f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < G; ++j) acc[k][n][j][i] *= by;
        }
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = i >> 1;
          s[k][n][i] = fmaf(bf16_lo(w[k].pair[h][0]), acc[k][n][0][i],
                            bf16_hi(w[k].pair[h][0]) * qs[n][0][i & 1]);
#pragma unroll
          for (int j = 1; j < G; ++j)
            s[k][n][i] = fmaf(bf16_lo(w[k].pair[h][j]), acc[k][n][j][i],
                              fmaf(bf16_hi(w[k].pair[h][j]), qs[n][j][i & 1], s[k][n][i]));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < G; ++j) {
          sv[k][h][j] = bf16_lo(w[k].pair[h][G + j]);
          mv[k][h][j] = bf16_hi(w[k].pair[h][G + j]);
        }
    }
    if (keys < kKeys) {  // what lies behind the keys may be anything
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (g + 8 * h + 16 * k >= keys) {
#pragma unroll
            for (int n = 0; n < NT; ++n) s[k][n][2 * h] = s[k][n][2 * h + 1] = -INFINITY;
#pragma unroll
            for (int j = 0; j < G; ++j) sv[k][h][j] = mv[k][h][j] = 0.f;
          }
    }
    bool over = false;
    float high[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        high[n][e] = max3f(fmaxf(s[0][n][e], s[0][n][2 + e]), s[1][n][e], s[1][n][2 + e]);
        over |= high[n][e] > top[n][e];
      }
    if (__any_sync(0xffffffffu, over)) {
      float f[NT][2], was[NT][G][2];
      bool shrinks = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = high[n][e];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[n][e]);
          f[n][e] = x == -INFINITY ? 1.f : ex2((m[n][e] - x) * c[n][e]);
          const bool met = m[n][e] > -INFINITY;
          m[n][e] = x;
          ref[n][e] = x == -INFINITY ? 0.f : -x;
          top[n][e] = x + kRescale * about_inverse(c[n][e]);
          l[n][e] *= f[n][e];
          const float grow = about_inverse(f[n][e]);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            z[n][j][e] *= f[n][e];
            // o shrinks with its unit, and by itself where the unit may not
            was[n][j][e] = v_inv[n][j][e];
            v_inv[n][j][e] = fminf(was[n][j][e] * grow, kMostInverse);
            shrinks |= met && v_inv[n][j][e] == kMostInverse;
          }
        }
      if (__any_sync(0xffffffffu, shrinks)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < G; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float g = f[n][e] * v_inv[n][j][e] * about_inverse(was[n][j][e]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[n][j][i][e] *= g;
                o[n][j][i][2 + e] *= g;
              }
            }
      }
    }
    // P, and P scale in o's units
    float p[2][NT][4], ps[2][NT][G][4], most = 0.f;
    auto scaled = [&]() {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < G; ++j)
              f2unpack(fmul2(fmul2(f2pack(p[k][n][2 * h], p[k][n][2 * h + 1]),
                                   f2pack(v_inv[n][j][0], v_inv[n][j][1])),
                             f2pack(sv[k][h][j], sv[k][h][j])),
                       ps[k][n][j][2 * h], ps[k][n][j][2 * h + 1]);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // The difference first: beside a large reference times c, rounded, the product of the same
        // score with c may be off by any power of two.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[2];
          f2unpack(fmul2(fadd2(f2pack(s[k][n][2 * h], s[k][n][2 * h + 1]),
                               f2pack(ref[n][0], ref[n][1])),
                         f2pack(c[n][0], c[n][1])),
                   x[0], x[1]);
          p[k][n][2 * h] = ex2(x[0]);
          p[k][n][2 * h + 1] = ex2(x[1]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[n][e] += p[k][n][e] + p[k][n][2 + e];
#pragma unroll
          for (int j = 0; j < G; ++j)
            z[n][j][e] = fmaf(p[k][n][e], mv[k][0][j], fmaf(p[k][n][2 + e], mv[k][1][j], z[n][j][e]));
        }
      }
    scaled();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < G; ++j) {
          most = max3f(most, ps[k][n][j][0], ps[k][n][j][1]);
          most = max3f(most, ps[k][n][j][2], ps[k][n][j][3]);
        }
    if (__any_sync(0xffffffffu, most > kMost)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              x = max3f(x, p[k][n][e] * sv[k][0][j], p[k][n][2 + e] * sv[k][1][j]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fminf(fmaxf(about_inverse(x), kLeastInverse), v_inv[n][j][e]);
            const float f = x * about_inverse(v_inv[n][j][e]);
            v_inv[n][j][e] = x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[n][j][i][e] *= f;
              o[n][j][i][2 + e] *= f;
            }
          }
      scaled();
    }
    uint32_t b[2][NT][G][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            b[k][n][j][h] = transpose8(pack_f16(ps[k][n][j][2 * h], ps[k][n][j][2 * h + 1]));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t (&v)[4] = w[k].v[j];
        const uint32_t two[2][2] = {
            {__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410)},
            {__byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w0 = two[i / 2][0], w1 = two[i / 2][1];
          const int e = 2 * (i & 1);
          const uint32_t a[4] = {codes(w0, e), codes(w0, e + 1), codes(w1, e), codes(w1, e + 1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(o[n][j][i], a, b[k][n][j][0], b[k][n][j][1]);
        }
      }
  }

  // The sums over the lanes that share a query, in plain units.
  FA_DEV void finish() {
    auto all = [](float v) {
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      return v + __shfl_xor_sync(0xffffffffu, v, 16);
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] = all(l[n][e]);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float add = all(z[n][j][e]), unit = about_inverse(v_inv[n][j][e]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // even channels came times 2^-24, odd ones 2^-20
            o[n][j][i][e] = fmaf(o[n][j][i][e] * 0x1p24f, unit, add);
            o[n][j][i][2 + e] = fmaf(o[n][j][i][2 + e] * 0x1p20f, unit, add);
          }
        }
      }
  }

  // The first `rows` rows as they are: O and L of a whole unit, or o and e of a part. A lane has
  // eight neighbouring channels of each group.
  FA_DEV void write(int rows, int d, int lane, bool whole, __nv_bfloat16* O, float* part,
                    float* stat) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * t + e;
        if (row >= rows) continue;
        const float sum = l[n][e], top = m[n][e] * c[n][e] + lg2(sum);
        const float inv = whole || sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const int col = 64 * j + 8 * g;
          if (col >= d) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = o[n][j][i][e] * inv;
            v[2 * i + 1] = o[n][j][i][2 + e] * inv;
          }
          if (whole) {
            *reinterpret_cast<uint4*>(O + row * d + col) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7]));
          } else {
            float4* const to = reinterpret_cast<float4*>(part + row * d + col);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        if (g == 0) stat[row] = whole ? top * kLn2 : top;
      }
  }

  // Rows [0, 8 NT) of o as floats [row][64 G]: two channels at a time, pair x of every four
  // at x ^ (row % 8 / 2), which puts a half warp's stores into different banks.
  FA_DEV void store(float* part, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(part + (8 * n + 2 * t + e) * 64 * G + 64 * j + 8 * g +
                                       2 * (i ^ t)) =
                make_float2(o[n][j][i][e], o[n][j][i][2 + e]);
  }
  // Columns c .. c + 3 (c a multiple of 4) of a row that store() wrote.
  FA_DEV static float4 fetch(const float* part, int row, int c) {
    const int t = (row & 7) >> 1, x = (c & 7) / 2;
    const float* at = part + row * 64 * G + (c & ~7);
    const float2 a = *reinterpret_cast<const float2*>(at + 2 * (x ^ t));
    const float2 b = *reinterpret_cast<const float2*>(at + 2 * ((x + 1) ^ t));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

FA_DEV float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }  // of a part

// A block takes a piece of the split (kPieces) or a unit (kWhole), 32 keys of each chunk a warp,
// or each warp takes a piece by itself (kSolo).
enum Mode { kPieces, kWhole, kSolo };
template <int G, int NT, Mode MODE>
__global__ void __launch_bounds__(kThreads, per_sm(NT))
    decode4_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<G, NT>;
  constexpr bool WHOLE = MODE == kWhole, SOLO = MODE == kSolo;
  constexpr int CHUNK = SOLO ? kKeys : kChunk;
  extern __shared__ __align__(128) uint8_t smem4[];
  __shared__ uint64_t full[kWarps][C::STAGES];
  __shared__ float2 stats[kWarps][C::ROWS];  // a warp's reference and weight sum
  __shared__ int warp_sums[kWarps];
  __shared__ uint32_t abort_flag, never;
  const Sizes& s = p.s;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  float* const parts = reinterpret_cast<float*>(smem4 + C::RINGS);
  int* const first = reinterpret_cast<int*>(smem4 + (SOLO ? C::RINGS : C::BYTES));

  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[warp][i], 2);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = never = 0;
  __syncthreads();
  grid_wait();
  grid_launch_dependents();

  // neighbouring pieces on different SMs
  const int me = SOLO ? warp * (int)gridDim.x + (int)blockIdx.x : (int)blockIdx.x;
  const int shift = SOLO ? 0 : kKeys * warp;  // of the warp's keys in a chunk
  int steps = 0;  // of one (head, row tile)
  int before = 0;  // up to 32 requests: steps before request `lane`, in every warp by itself
  const bool few = s.B <= 32;
  unsigned x_begin = 0, x_end = 0;
  if constexpr (!WHOLE) {
    // Steps before each request: an exclusive scan of the lengths, of neighbouring ones by a
    // thread each.
    const int per = few ? 1 : (s.B + kThreads - 1) / kThreads;
    const int b0 = few ? lane : (int)threadIdx.x * per;
    int n = 0;
    bool bad = false;
#pragma unroll 8
    for (int i = 0; i < per; ++i) {
      const int len = b0 + i < s.B ? p.lens[b0 + i] : 0;
      bad |= len < 0 || len > p.max_pages << p.page_shift;
      n += steps_of(max(0, min(len, p.max_pages << p.page_shift)), CHUNK);
    }
    if (bad && blockIdx.x == 0) atomicOr(&g_decode4_status, kDeviceIndexBit);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    before = x - n;
    steps = __shfl_sync(0xffffffffu, x, 31);
    if (!few) {
      if (lane == 31) warp_sums[warp] = x;
      __syncthreads();
      steps = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        steps += warp_sums[w];
      }
      int at = before;
#pragma unroll 8
      for (int i = 0; i < per; ++i) {
        if (b0 + i < s.B) {
          first[b0 + i] = at;
          if (blockIdx.x == 0) s.first[b0 + i] = at;
          at += steps_of(keys_of(p, b0 + i), CHUNK);
        }
      }
      if (threadIdx.x == 0) {
        first[s.B] = steps;
        if (blockIdx.x == 0) s.first[s.B] = steps;
      }
      __syncthreads();
    }
    steps = uniform(steps);
    const Split sp = split_of(s, steps);
    if (me >= sp.workers) return;
    x_begin = (unsigned)uniform((int)sp.start(me));
    x_end = (unsigned)uniform((int)sp.start(me + 1));
  }
  // Steps before request b, at most B.
  auto first_of = [&](int b) {
    int f = steps;
    if (!few)
      f = first[b];
    else if (b < s.B)
      f = __shfl_sync(0xffffffffu, before, b);
    return uniform(f);
  };

  // A run of steps of one unit: chunks c0 .. c1 - 1 of its keys.
  struct Run {
    int b, ht, len, c0, c1;
    unsigned x1;  // the end of its steps
    int begins, ends;  // the unit
  };
  auto run_of = [&](int ht, int b, unsigned x) {  // from step x on
    Run r;
    const unsigned u0 = (unsigned)(ht * steps + first_of(b));
    const unsigned u1 = (unsigned)(ht * steps + first_of(b + 1));
    r.b = uniform(b);
    r.ht = uniform(ht);
    r.x1 = (unsigned)uniform((int)min(u1, x_end));
    r.c0 = uniform(max(0, (int)(x - u0) - kRunSteps));
    r.c1 = uniform(max(0, (int)(r.x1 - u0) - kRunSteps));
    r.begins = uniform(x == u0);
    r.ends = uniform(r.x1 == u1);
    r.len = uniform(keys_of(p, b));
    return r;
  };
  auto first_run = [&]() {
    if constexpr (WHOLE) {
      Run r;
      r.ht = me / s.B;
      r.b = me - r.ht * s.B;
      r.len = uniform(keys_of(p, r.b));
      r.c0 = 0;
      r.c1 = (r.len + CHUNK - 1) / CHUNK;
      r.x1 = 0;
      r.begins = r.ends = true;
      return r;
    }
    const int ht = (int)(x_begin / (unsigned)steps), in = (int)(x_begin - (unsigned)(ht * steps));
    int lo = 0, hi = s.B;  // the last request with steps before it that are no more than `in`
    if (few) {
      lo = 31 - __clz(__ballot_sync(0xffffffffu, lane < s.B && before <= in));
    } else {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= in)
          lo = mid;
        else
          hi = mid;
      }
    }
    return run_of(ht, uniform(lo), x_begin);
  };
  auto next_run = [&](const Run& r) {  // r.x1 < x_end
    int ht = r.ht, b = r.b + 1;
    for (;;) {  // requests without keys have no steps
      if (b == s.B) {
        b = 0;
        ++ht;
      }
      if (first_of(b + 1) > first_of(b)) return run_of(ht, b, r.x1);
      ++b;
    }
  };

  // Stages of a run in which this warp has keys.
  auto stages_of = [&](const Run& r) {
    const int key = r.c0 * CHUNK + shift;
    return min(r.c1 - r.c0, max(0, r.len - key + CHUNK - 1) / CHUNK);
  };

  const uint32_t ring = smem_u32(smem4) + warp * C::STAGES * C::STAGE;
  const uint32_t bars = smem_u32(&full[warp][0]);
  const WaitCtx wait{&abort_flag, &g_decode4_status};
  // ---- the issuing side, up to STAGES stages ahead of the products: lanes 2 i and 2 i + 1 have
  // the addresses of the two blocks of stage i of the next 16, and issue their copies.
  Run ir = first_run();
  const Run ir_first = ir;
  if constexpr (WHOLE) {
    const int len = p.lens[ir.b];
    if ((len < 0 || len > p.max_pages << p.page_shift) && threadIdx.x == 0)
      atomicOr(&g_decode4_status, kDeviceIndexBit);
  }
  int ij = 0, i_stages = stages_of(ir);  // stages of the run that lanes have had, and all
  int i_at = 0, i_end = 0;               // of the 16
  int i_stage = 0, issued = 0;
  bool more = true;
  const uint8_t* src = nullptr;
  auto refill = [&]() {
    while (ij == i_stages) {
      if (ir.x1 == x_end) {
        more = false;
        return;
      }
      ir = next_run(ir);
      i_stages = stages_of(ir);
      ij = 0;
    }
    const int key = (ir.c0 + ij + (lane >> 1)) * CHUNK + shift + kRows4 * (lane & 1);
    src = nullptr;
    if (ij + (lane >> 1) < i_stages && key < ir.len) {
      int page = p.table[(size_t)ir.b * p.max_pages + (key >> p.page_shift)];
      if ((unsigned)page >= (unsigned)p.num_pages) {
        atomicOr(&g_decode4_status, kDeviceIndexBit);
        page = 0;
      }
      const int hk = ir.ht / s.row_tiles, in = key & ((1 << p.page_shift) - 1);
      src = p.cache + ((((size_t)page * s.Hkv + hk) << p.page_shift) + in) * (C::BLOCK / kRows4);
    }
    i_at = 0;
    i_end = min(16, i_stages - ij);
    ij += i_end;
  };
  auto issue = [&]() {
    if (i_at == i_end) refill();
    if (!more) return;
    bulk_load(lane >> 1 == i_at, ring + i_stage * C::STAGE + (lane & 1) * C::BLOCK, src, C::BLOCK,
              bars + 8 * i_stage);
    i_stage = i_stage + 1 == C::STAGES ? 0 : i_stage + 1;
    ++issued;
    ++i_at;
  };
  __syncwarp();  // the barriers are initialised
#pragma unroll
  for (int i = 0; i < C::STAGES; ++i) issue();

  // ---- the products
  int stage = 0, used = 0;
  uint32_t phase = 0;
  bool alive = true;
  Tile<G, NT> tile;
  typename Tile<G, NT>::Raw raw;
  Run r = ir_first;
  int rows;
  size_t row0;
  auto load_queries = [&]() {  // of run r
    const int hk = r.ht / s.row_tiles, rt = r.ht - hk * s.row_tiles;
    rows = min(8 * NT, s.per_kv - rt * 8 * NT);
    row0 = (size_t)r.b * s.Hq + hk * s.per_kv + rt * 8 * NT;
    raw.load(p.Q + row0 * s.d, rows, s.d, lane);
  };
  load_queries();
  if constexpr (WHOLE) {
    if (r.len == 0) {
      for (int i = threadIdx.x; i < rows * (s.d / 8); i += kThreads)
        reinterpret_cast<uint4*>(p.O + row0 * s.d)[i] = make_uint4(0, 0, 0, 0);
      if (threadIdx.x < rows) p.L[row0 + threadIdx.x] = -INFINITY;
      return;
    }
  }
  for (;;) {
    tile.start(raw, p.scale_log2, lane);
    int keys = r.len - (r.c0 * CHUNK + shift);  // from the stage on
    for (int j = stages_of(r); j > 0; --j, keys -= CHUNK) {
      if (alive) alive = warp_wait(&full[warp][stage], phase, wait);
      if (!alive) break;
      const uint32_t at = ring + stage * C::STAGE;
      ++used;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      Words<G> w[2];
      w[0].load(at, lane);
      w[1].load(at + C::BLOCK, lane);
      __syncwarp();  // every lane has read the stage: it may be filled again
      issue();
      tile.step(w, keys, lane);
    }
    tile.finish();
    const bool whole = r.begins && r.ends, last = r.x1 == x_end;
    const unsigned slot = 2u * (unsigned)me + (r.begins ? 1u : 0u);  // Split::slot
    const int done_rows = rows;
    const size_t done_row0 = row0;
    if constexpr (SOLO) {
      if (!last) {  // the next run's queries come while this one's results go
        r = next_run(r);
        load_queries();
      }
      if (whole)
        tile.write(done_rows, s.d, lane, true, p.O + done_row0 * s.d, (float*)nullptr,
                   p.L + done_row0);
      else
        tile.write(done_rows, s.d, lane, false, (__nv_bfloat16*)nullptr,
                   s.o + (size_t)slot * s.slot_rows * s.d, s.e + (size_t)slot * s.slot_rows);
      if (last) break;
      continue;
    }
    tile.store(parts + warp * C::ROWS * C::D, lane);
    if (lane < 4) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          stats[warp][8 * n + 2 * lane + e] =
              make_float2(tile.m[n][e] * tile.c[n][e], tile.l[n][e]);
    }
    if (!last) {  // the next run's queries come while this one's parts are joined
      r = next_run(r);
      load_queries();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < done_rows * (C::D / 4); i += kThreads) {
      const int row = i / (C::D / 4), c = (i - row * (C::D / 4)) * 4;
      if (c >= s.d) continue;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stats[k][row].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = stats[k][row];
        const float f = ex2(ml.x - ref);
        const float4 v = Tile<G, NT>::fetch(parts + k * C::ROWS * C::D, row, c);
        sum += f * ml.y;
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if (whole) {
        const float inv = 1.f / sum;
        *reinterpret_cast<uint2*>(p.O + (done_row0 + row) * s.d + c) = make_uint2(
            pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (c == 0) p.L[done_row0 + row] = (top + lg2(sum)) * kLn2;
      } else {
        const float inv = inverse(sum);
        const size_t at = (size_t)slot * s.slot_rows + row;
        *reinterpret_cast<float4*>(s.o + at * s.d + c) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (c == 0) s.e[at] = top + lg2(sum);
      }
    }
    if (last) break;
    __syncthreads();  // the parts are read
  }
  // After a wait that ran out: the copies in flight land before the block's memory is given up.
  const WaitCtx drain{&never, &g_decode4_status};
  while (used < issued) {
    warp_wait(&full[warp][stage], phase, drain);
    ++used;
    if (++stage == C::STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// A row (request, query head) is joined by one warp, or by kJoinWarps where there are few rows or
// the row has more than kAlone parts (a request much longer than the others; one of 131072 keys
// among 320, a key/value head of 8 queries: 40 us for the call, with a warp for each row 245).
// Rows of a block are gridDim.x apart, so that such a request's are many blocks' work. Lane i
// looks up part i's e, and the warp adds the parts up, four columns a lane, of which the first 6
// or 16 are on their way beside e: the kernel is a chain of waits for memory, about 3 us behind
// the split kernel. Rows that the split kernel has finished are left alone.
constexpr int kJoinWarps = 8, kAlone = 32;

// What a row's parts come to, for one warp of WARPS: sum_i w_i o_i and sum_i w_i (this lane's),
// w_i = 2^(e_i - ref).
struct Joined {
  float ref, sum;
  float4 acc;
};
template <int WARPS, int U>  // U parts on their way at a time
FA_DEV Joined join_parts(const Sizes& s, int in, int w0, int parts, int mine, int lane) {
  // Part i of the row in s.o and s.e.
  auto place = [&](int i) {
    return (size_t)Split::slot(0, 0, parts, w0, i) * s.slot_rows + in % s.tile;
  };
  const bool has = 4 * lane < s.d;
  Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int base = mine; base < parts; base += 32 * WARPS) {
    const int i = base + lane * WARPS;
    const float e = i < parts ? s.e[place(i)] : -INFINITY;
    const int n = min(32, (parts - base + WARPS - 1) / WARPS);  // lanes with a part
    float4 v[U];
    auto load = [&](int j) {  // the first ones on their way beside e
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j + u < n && has)
          v[u] = reinterpret_cast<const float4*>(s.o + place(base + (j + u) * WARPS) * s.d)[lane];
      }
    };
    load(0);
    float top = e;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float next = fmaxf(r.ref, top);
    const float back = r.ref == next ? 1.f : ex2(r.ref - next);  // 0 on the first round
    r.ref = next;
    const float weight = i < parts ? ex2(e - (r.ref == -INFINITY ? 0.f : r.ref)) : 0.f;
    r.sum = r.sum * back + weight;
    r.acc.x *= back;
    r.acc.y *= back;
    r.acc.z *= back;
    r.acc.w *= back;
    for (int j = 0; j < n; j += U) {
      if (j > 0) load(j);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = __shfl_sync(0xffffffffu, weight, (j + u) & 31);
        if (j + u >= n) break;
        r.acc.x += w * v[u].x;
        r.acc.y += w * v[u].y;
        r.acc.z += w * v[u].z;
        r.acc.w += w * v[u].w;
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) r.sum += __shfl_xor_sync(0xffffffffu, r.sum, x);
  return r;
}

FA_DEV void write_row(const DecodeParams& p, int row, int lane, const Joined& r) {
  const float inv = 1.f / r.sum;
  if (4 * lane < p.s.d)
    reinterpret_cast<uint2*>(p.O + (size_t)row * p.s.d)[lane] =
        make_uint2(pack_bf16(r.acc.x * inv, r.acc.y * inv),
                   pack_bf16(r.acc.z * inv, r.acc.w * inv));
  if (lane == 0) p.L[row] = (r.ref + lg2(r.sum)) * kLn2;
}

template <int WARPS>  // of a row
__global__ void __launch_bounds__(32 * kJoinWarps, WARPS == 1 ? 4 : 2)
    join4_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ float4 sums[kJoinWarps][32];
  __shared__ float2 stats[kJoinWarps];
  __shared__ int4 many[kJoinWarps];  // row, head's query, first worker and parts of a warp's row
  const Sizes& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = WARPS == 1 ? warp * gridDim.x + blockIdx.x : blockIdx.x;
  const bool mine = (WARPS == 1 || warp == 0) && row < s.B * s.Hq;
  const int b = min(row / s.Hq, s.B - 1), hq = min(row - b * s.Hq, s.Hq - 1);
  const int hk = hq / s.per_kv, in = hq - hk * s.per_kv, ht = hk * s.row_tiles + in / s.tile;
  // The lengths are the call's inputs: they were written before the split kernel, which launched
  // this one, had started, so that the parts are found while that kernel runs. Many requests'
  // lengths take longer to sum up than to read from where the split kernel puts their sums.
  int f0 = 0, f1 = 0, steps = 0;
  if (s.B <= 256) {
    for (int i = lane; i < s.B; i += 32) {
      const int n = steps_of(keys_of(p, i), s.chunk);
      steps += n;
      if (i < b) f0 += n;
      if (i == b) f1 = n;
    }
    steps = __reduce_add_sync(0xffffffffu, steps);
    f0 = __reduce_add_sync(0xffffffffu, f0);
    f1 = __reduce_add_sync(0xffffffffu, f1) + f0;
    grid_wait();
  } else {
    grid_wait();
    steps = s.first[s.B];
    f0 = s.first[b];
    f1 = s.first[b + 1];
  }
  grid_launch_dependents();
  int w0 = 0, parts = 1;  // 1: nothing to join
  if (f0 < f1) {
    const Split sp = split_of(s, steps);
    w0 = sp.owner((unsigned)(ht * steps + f0));
    parts = sp.owner((unsigned)(ht * steps + f1) - 1u) - w0 + 1;
  } else if (mine) {
    if (4 * lane < s.d)
      reinterpret_cast<uint2*>(p.O + (size_t)row * s.d)[lane] = make_uint2(0, 0);
    if (lane == 0) p.L[row] = -INFINITY;
  }

  // A row joined by the block; every thread calls.
  auto join = [&](int row, int in, int w0, int parts) {
    Joined r = join_parts<kJoinWarps, WARPS == 1 ? 6 : 16>(s, in, w0, parts, warp, lane);
    sums[warp][lane] = r.acc;
    if (lane == 0) stats[warp] = make_float2(r.ref, r.sum);
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, stats[w].x);
    r = {top, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      // a warp without parts has reference -inf and adds nothing
      const float f = w < parts ? ex2(stats[w].x - (top == -INFINITY ? 0.f : top)) : 0.f;
      const float4 v = sums[w][lane];
      r.acc.x += f * v.x;
      r.acc.y += f * v.y;
      r.acc.z += f * v.z;
      r.acc.w += f * v.w;
      r.sum += f * stats[w].y;
    }
    write_row(p, row, lane, r);
  };
  if (WARPS > 1) {
    if (parts > 1) join(row, in, w0, parts);  // the block's row
    return;
  }
  const bool alone = parts <= kAlone;
  if (lane == 0) many[warp] = make_int4(row, in, w0, mine && !alone ? parts : 0);
  if (mine && alone && parts > 1)
    write_row(p, row, lane, join_parts<1, 6>(s, in, w0, parts, 0, lane));
  if (!__syncthreads_or(mine && !alone)) return;
  for (int w = 0; w < kJoinWarps; ++w) {
    const int4 m = many[w];
    if (m.w == 0) continue;
    join(m.x, m.y, m.z, m.w);
    __syncthreads();
  }
}

// Bytes of the kernel's shared memory that are not dynamic, at most.
constexpr int kStatic = 1024;

template <int G, int NT>
cudaError_t launch(const Decode4Args& a, cudaStream_t stream) {
  using C = Cfg<G, NT>;
  DecodeParams p;
  p.s = sizes_of(a.B, a.Hq, a.Hkv, a.d, a.max_pages * a.page);
  lay_out(&p.s, a.workspace);
  const int count = sm_count(), sms = count < kMaxSms ? count : kMaxSms;
  const int fixed = p.s.solo ? C::RINGS : C::BYTES, smem = fixed + (a.B + 1) * 4;
  // As many blocks as fit (an SM has 227 KB for them, and 1 KB of each is the system's), and no
  // more than the capacities can keep busy.
  const int fit = 227 * 1024 / (smem + kStatic + 1024), most = fit < per_sm(NT) ? fit : per_sm(NT);
  const long long need = p.s.solo ? (p.s.steps + kWarps - 1) / kWarps : p.s.steps;
  const int blocks = need == 0 ? 1 : (int)(need < sms * most ? need : sms * most);
  p.s.workers = p.s.solo ? blocks * kWarps : blocks;
  p.Q = static_cast<const __nv_bfloat16*>(a.Q);
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.table = a.table;
  p.lens = a.lens;
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.L = a.L;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  p.scale_log2 = a.scale * kLog2e;
  const bool whole =
      ceil_div(a.max_pages * a.page, kChunk) <= kWholeChunks && p.s.units <= sms * per_sm(NT);
  auto kernel = whole      ? decode4_kernel<G, NT, kWhole>
                : p.s.solo ? decode4_kernel<G, NT, kSolo>
                           : decode4_kernel<G, NT, kPieces>;
  const int dynamic = whole ? C::BYTES : smem;
  cudaError_t e = cudaSuccess;
  if (dynamic + kStatic > 48 * 1024)  // what a block may have of both without asking
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::BYTES + (kMaxBatch + 1) * 4);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(whole ? p.s.units : blocks);
  e = launch_early(kernel, dim3(grid), kThreads, dynamic, stream, p);
  if (e != cudaSuccess || whole) return e;
  const int rows = a.B * a.Hq;
  // A warp per row once there is a row for every fourth warp slot of the GPU's SMs.
  return rows >= sms * 4
             ? launch_early(join4_kernel<1>, dim3((unsigned)ceil_div(rows, kJoinWarps)),
                            32 * kJoinWarps, 0, stream, p)
             : launch_early(join4_kernel<kJoinWarps>, dim3((unsigned)rows), 32 * kJoinWarps, 0,
                            stream, p);
}

}  // namespace

size_t decode4_workspace_bytes(int B, int Hq, int Hkv, int d, int capacity) {
  Sizes s = sizes_of(B, Hq, Hkv, d, capacity);
  return lay_out(&s, nullptr);
}

cudaError_t launch_decode4(const Decode4Args& a, cudaStream_t s) {
  const bool two = sizes_of(a.B, a.Hq, a.Hkv, a.d, 0).tile == 16;
  if (a.d > 64) return two ? launch<2, 2>(a, s) : launch<2, 1>(a, s);
  return two ? launch<1, 2>(a, s) : launch<1, 1>(a, s);
}

cudaError_t decode4_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_decode4_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_decode4_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
