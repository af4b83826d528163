// Decode attention behind a shared prefix: one new token for each of B requests, whose
// keys are the prefix that all of them share and then their own, both in pages of a
// cache. Per query row the keys are split into parts, each part gives
//   o = softmax over its keys times V,   e = log2 sum 2^(s * scale * log2(e))
// and the parts are joined exactly: O = sum 2^(e - M) o / sum 2^(e - M), M = max e. A part
// whose scores are all minus infinity (a key with an infinite entry, or a product that
// overflows) has e = -inf and o = 0: it adds nothing to the others.
//
//   prefix kernel  the shared keys, once for all requests: the query rows of all
//                  requests and of the query heads of one key/value head are the rows
//                  of one matrix product, so that K and V are read once for 256 rows.
//                  This is the forward kernel (fa_forward.cuh, tcgen05) with rows
//                  (request, query head), non-causal, keys from pages.
//   shared kernel  the same for at most 16 or 32 rows, with the own kernel's products.
//   own kernel     each request's own keys. Hq / Hkv rows share a key, far fewer than a
//                  tcgen05 tile has: bound by reading the keys from HBM, so the
//                  products are warp-level ones of 16 rows and every warp streams its
//                  own keys through a private ring of shared memory.
//   join kernel    joins the parts of each row, prefix and own.
//   whole kernel   instead of them all, for small calls.
//
// These kernels split their keys evenly, whatever the lengths: the blocks of all (row
// group, key/value head) units are laid end to end and worker c of P takes the c-th of
// P equal pieces of that axis (Split). A worker's piece covers whole units and at most
// two partial ones, so the parts need one slot per unit and two per worker. Lengths are
// read on the device; nothing depends on the order in which workers finish.
#include "fa_decode.h"
#include "fa_forward.cuh"
#include "fa_launch.h"

namespace fa {

__device__ unsigned int g_prefix_status;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMaxSms = 160;       // slots are reserved for this many thread blocks
constexpr int kOwnWarps = 4;       // warps of a thread block of the own kernel
// Thread blocks of the own kernel per SM: 128 KB of keys in flight on each, above the
// latency-bandwidth product of an SM's share of HBM, for either row size.
constexpr int kOwnPerSmWide = 2, kOwnPerSmNarrow = 4;
constexpr int kOwnChunk = 64;      // keys per step of the own keys' split
constexpr int kMinPrefixBlocks = 2;  // 128-key blocks a prefix worker takes at least

// `total` steps (below 2^31) dealt to at most `most` workers in contiguous pieces that
// differ by one step at most; the longer pieces come first.
struct Split {
  unsigned total, base, longer;
  int workers;
  FA_DEV Split(unsigned steps, unsigned most) : total(steps) {
    workers = (int)min(steps, most);
    base = workers > 0 ? steps / (unsigned)workers : 0u;
    longer = steps - base * (unsigned)workers;
  }
  FA_DEV unsigned start(int w) const { return (unsigned)w * base + min((unsigned)w, longer); }
  // The worker whose piece holds step x (0 <= x < total).
  FA_DEV int owner(unsigned x) const {
    const unsigned in_longer = longer * (base + 1);
    return (int)(x < in_longer ? x / (base + 1) : longer + (x - in_longer) / base);
  }
  // The slot of a unit's part number `part` of `parts` (its first worker is `first`):
  // unit's own slot, or the worker's slot for the unit that starts in its piece and goes
  // on (odd) or came from the piece before (even).
  FA_DEV static unsigned slot(unsigned unit, unsigned units, int parts, int first, int part) {
    return parts == 1 ? unit : units + 2u * (unsigned)(first + part) + (part == 0 ? 1u : 0u);
  }
};

// Sizes that the three kernels agree on.
struct DecodeSizes {
  int B, Hq, Hkv, per_kv, d;
  int per_tile;       // requests per 128-row tile of the prefix kernel
  int pairs;          // tile pairs
  int pair_rows;      // rows of a prefix slot
  int row_tiles;      // 16-row tiles of a key/value head's rows in the own kernel
  int own_rows;       // rows of an own slot
  int own_per_sm;     // thread blocks of the own kernel per SM
  int sms, prefix_workers, own_blocks;  // blocks launched of the prefix and own kernels
  int prefix_step_ns, own_chunk_ns;     // see prefix_share
  unsigned units_magic;                 // ceil(2^32 / (pairs * Hkv))
  float *prefix_o, *prefix_e;  // [slot][pair_rows][d], [slot][pair_rows]
  float *own_o, *own_e;        // [slot][own_rows][d], [slot][own_rows]
  int* first;                  // [B + 1] own chunks before each request
};

// Lays the workspace out for prefixes of at most `prefix_cap` and own parts of at most
// `own_cap` keys (a worker without steps has no slots); returns its bytes.
size_t lay_out(DecodeSizes* s, void* base, int prefix_cap, int own_cap) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = p + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  auto slots = [](size_t units, size_t steps_each, size_t workers) {
    const size_t steps = units * steps_each;
    return steps == 0 ? 0 : units + 2 * (steps < workers ? steps : workers);
  };
  const size_t pslots = slots((size_t)s->pairs * s->Hkv, ((size_t)prefix_cap + 127) / 128, kMaxSms);
  const size_t oslots = slots((size_t)s->Hkv * s->row_tiles * s->B,
                              ((size_t)own_cap + kOwnChunk - 1) / kOwnChunk,
                              (size_t)kMaxSms * s->own_per_sm * kOwnWarps);
  s->prefix_o = reinterpret_cast<float*>(take(pslots * s->pair_rows * s->d * 4));
  s->prefix_e = reinterpret_cast<float*>(take(pslots * s->pair_rows * 4));
  s->own_o = reinterpret_cast<float*>(take(oslots * s->own_rows * s->d * 4));
  s->own_e = reinterpret_cast<float*>(take(oslots * s->own_rows * 4));
  s->first = reinterpret_cast<int*>(take(((size_t)s->B + 1) * 4));
  return at;
}

DecodeSizes sizes_of(int B, int Hq, int Hkv, int d) {
  DecodeSizes s{};
  s.B = B;
  s.Hq = Hq;
  s.Hkv = Hkv;
  s.per_kv = Hq / Hkv;
  s.d = d;
  s.per_tile = 128 / s.per_kv;
  s.pairs = ceil_div(B, 2 * s.per_tile);
  s.pair_rows = (B < 2 * s.per_tile ? B : 2 * s.per_tile) * s.per_kv;
  s.row_tiles = ceil_div(s.per_kv, 16);
  s.own_rows = s.per_kv < 16 ? s.per_kv : 16;
  s.own_per_sm = d > 64 ? kOwnPerSmWide : kOwnPerSmNarrow;
  return s;
}

// The prefix's length, at most what the listed pages hold.
FA_DEV int prefix_keys(const int* prefix_len, int cap) {
  const int n = prefix_len ? *prefix_len : 0;
  return max(0, min(n, cap));
}
// Thread blocks of the prefix kernel that get work, for a prefix of `blocks` 128-key
// blocks and `chunks` chunks of own keys per head and row tile. The two kernels run side
// by side, a prefix block on an SM of its own and the own kernel's on the others, so the
// SMs are shared out in proportion to the work: a prefix step of 128 keys takes an SM
// 2.4 us (two row tiles) or 1.5 us (one), 0.5 us less for d <= 64, 8 d ns in the shared
// kernel, and a chunk of own keys 4 d ns (their bytes at 65 GB/s). All kernels compute this
// from the same integers, in few divisions: it stands at the start of each, and one more
// costs a call half a microsecond.
// 256 requests behind 8192 keys (32/8 heads, d = 128, up to 2048 own): 183 us, against
// 226 us with every SM for the one kernel and then for the other.
FA_DEV int prefix_share(const DecodeSizes& s, int blocks, int chunks) {
  const unsigned steps = (unsigned)(s.pairs * s.Hkv) * (unsigned)blocks;
  if (steps == 0) return 0;
  const int most = (int)min((unsigned)s.prefix_workers,
                            (steps + kMinPrefixBlocks - 1) / kMinPrefixBlocks);
  if (chunks == 0) return most;
  const unsigned long long a = (unsigned long long)steps * (unsigned)s.prefix_step_ns;
  const unsigned long long both = a + (unsigned long long)(s.Hkv * s.row_tiles) *
                                          (unsigned)chunks * (unsigned)s.own_chunk_ns;
  // to 24 bits, for a 32-bit division
  const int shift = max(0, 40 - __clzll((long long)both));
  const unsigned part = (unsigned)(a >> shift), all = (unsigned)(both >> shift);
  const int top = min(most, s.sms - 1);
  const int n = max(1, min((int)(((unsigned)s.sms * part + all / 2) / all), top));
  // Whole blocks a unit where that is near: fewer parts. Else an even number: SMs come in
  // pairs, and a pair of which one half has a prefix block and the other own ones is slower
  // (in the case above 32 blocks take 181 us, 34 187, 31 or 33 196).
  const int units = s.pairs * s.Hkv;
  const int m = (int)__umulhi((unsigned)(n + units / 2), s.units_magic) * units;  // n / units
  if (m > 0 && (m & 1) == 0 && m <= top && abs(m - n) * 8 <= min(n, s.sms - n)) return m;
  return n > 1 ? n & ~1 : n;
}
FA_DEV Split prefix_split(const DecodeSizes& s, int blocks, int share) {
  return Split((unsigned)(s.pairs * s.Hkv) * (unsigned)blocks, (unsigned)share);
}
// Thread blocks of the own kernel that get work.
FA_DEV int own_share(const DecodeSizes& s, int share) {
  return min(s.own_blocks, s.own_per_sm * (s.sms - share));
}
FA_DEV Split own_split(const DecodeSizes& s, int chunks, int share) {
  return Split((unsigned)(s.Hkv * s.row_tiles) * (unsigned)chunks,
               (unsigned)(own_share(s, share) * kOwnWarps));
}
// 1 / l for a part's sum l of weights, 0 for a part without a finite score.
FA_DEV float part_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
// Own chunks of a request whose table row holds `cap` keys.
FA_DEV int own_chunks(int len, int cap) {
  return (max(0, min(len, cap)) + kOwnChunk - 1) / kOwnChunk;
}

// ================================================================== prefix kernel
struct PrefixParams {
  DecodeSizes s;
  const int *pages, *len, *lens;
  int cap, own_cap;                      // keys
  int page, page_shift, box, num_pages;  // box: rows of a TMA copy
};

// ONE_TILE: all rows of a key/value head fit one 128-row tile (so there is one pair, and
// its second tile is empty): both softmax groups work on that tile, each on every other
// 64 keys.
template <bool ONE_TILE>
struct Prefix {
  using Params = PrefixParams;
  struct View {
    const Params& p;
    int keys, blocks;
    Split split;
  };
  struct Item {
    int pair, hk, k0, m;  // tile pair, head, first key, keys
    unsigned slot;
  };
  static constexpr bool kSplit = true, kAlternate = ONE_TILE, kEarly = true;
  static constexpr bool kForeignTail = true;
  FA_DEV static unsigned int* status() { return &g_prefix_status; }
  FA_DEV static bool trigger(const Params&) { return true; }  // for the own kernel
  FA_DEV static View view(const Params& p) {
    const int n = *p.len;
    int chunks = 0;  // each warp on its own; read beside n
    for (int b = threadIdx.x & 31; b < p.s.B; b += 32)
      chunks += own_chunks(p.lens[b], p.own_cap);
    chunks = __reduce_add_sync(0xffffffffu, chunks);
    if ((n < 0 || n > p.cap) && blockIdx.x == 0 && threadIdx.x == 0)
      atomicOr(status(), kDeviceIndexBit);
    const int keys = max(0, min(n, p.cap)), blocks = (keys + 127) / 128;
    return {p, keys, blocks, prefix_split(p.s, blocks, prefix_share(p.s, blocks, chunks))};
  }
  FA_DEV static int segments(const View& g, int cta, int) {
    if (cta >= g.split.workers) return 0;
    const unsigned a = g.split.start(cta), b = g.split.start(cta + 1), n = (unsigned)g.blocks;
    return (int)((a % n + (b - a) + n - 1) / n);
  }
  FA_DEV static Item segment(const View& g, int cta, int, int j) {
    const unsigned a = g.split.start(cta), b = g.split.start(cta + 1);
    const unsigned unit = a / (unsigned)g.blocks + (unsigned)j, u0 = unit * (unsigned)g.blocks;
    const unsigned x0 = max(a, u0), x1 = min(b, u0 + (unsigned)g.blocks);
    Item it;
    it.pair = (int)(unit / (unsigned)g.p.s.Hkv);
    it.hk = (int)unit - it.pair * g.p.s.Hkv;
    it.k0 = (int)(x0 - u0) * 128;
    it.m = min(g.keys, (int)(x1 - u0) * 128) - it.k0;
    const unsigned units = (unsigned)(g.p.s.pairs * g.p.s.Hkv);
    it.slot = x1 - x0 == (unsigned)g.blocks ? unit
                                            : units + 2u * (unsigned)cta + (x0 == u0 ? 1u : 0u);
    return it;
  }
  FA_DEV static int steps(const View& g, const Item& it, int t) {
    const int halves = (it.m + 63) / 64;
    if (ONE_TILE) return (halves + 1 - t) / 2;
    return (2 * it.pair + t) * g.p.s.per_tile < g.p.s.B ? halves : 0;
  }
  // The first request of tile t.
  FA_DEV static int request(const View& g, const Item& it, int t) {
    return (2 * it.pair + (ONE_TILE ? 0 : t)) * g.p.s.per_tile;
  }
  FA_DEV static int keys(const View&, const Item& it) { return it.m; }
  FA_DEV static constexpr int causal(const View&) { return 0; }
  FA_DEV static int query(const View&, const Item&, int, int) { return 0; }
  template <class C>
  FA_DEV static uint32_t tile_bytes(const View& g) {
    return (uint32_t)(g.p.s.per_tile * g.p.s.per_kv) * 128u * C::KCH;
  }
  // Rows (request, query head of the key/value head): the rows past per_tile * per_kv of
  // a tile keep what the buffer held; nothing of them is stored.
  FA_DEV static void load_q(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                            const View& g, const Item& it, int t) {
    tma_load_4d(dst, map, f, col, 0, it.hk, request(g, it, t));
  }
  // Copies of `box` rows (a page or 128 keys) of a block; pages wholly past the item's
  // keys are not read.
  FA_DEV static int boxes(const View& g, const Item& it, int block) {
    return (min(128, it.m - block * 128) + g.p.box - 1) / g.p.box;
  }
  template <class C>
  FA_DEV static uint32_t block_bytes(const View& g, const Item& it, int block) {
    return (uint32_t)(boxes(g, it, block) * g.p.box) * 256u * C::KCH;
  }
  // The pages of a block's copies.
  struct Place {
    int page[8];
  };
  FA_DEV static Place place(const View& g, const Item& it, int block) {
    Place at;
    const int n = boxes(g, it, block), key0 = it.k0 + block * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      at.page[i] = i < n ? g.p.pages[(key0 + i * g.p.box) >> g.p.page_shift] : 0;
    return at;
  }
  template <class C>
  FA_DEV static void load_kv(uint8_t* kdst, uint8_t* vdst, const CUtensorMap* mk,
                             const CUtensorMap* mv, uint64_t* f, const View& g, const Item& it,
                             int block, const Place& at) {
    const int n = boxes(g, it, block), key0 = it.k0 + block * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= n) break;
      int page = at.page[i];
      if ((unsigned)page >= (unsigned)g.p.num_pages) {
        atomicOr(status(), kDeviceIndexBit);
        page = 0;
      }
      const int row = (key0 + i * g.p.box) & (g.p.page - 1), plane = page * g.p.s.Hkv + it.hk;
#pragma unroll
      for (int c = 0; c < C::KCH; ++c) {
        tma_load_3d(kdst + c * C::CHUNK + i * g.p.box * 128, mk, f, c * 64, row, plane);
        tma_load_3d(vdst + c * C::CHUNK + i * g.p.box * 128, mv, f, c * 64, row, plane);
      }
    }
  }
  // Writes columns [c0, c0 + NCOL) of a warp's 32 rows of a part, fp32 [pair_rows, d]:
  // 16 columns at a time through 2 KB of shared memory (16-byte piece k of row r at
  // k ^ ((r >> 1) & 3)), so that a row's 64 bytes leave together. `fetch(c, v)` gives this
  // lane's columns c .. c + 15; `rows` of the 32 rows are written.
  template <int NCOL, class F>
  FA_DEV static void write_part(float* out, int rows, int c0, int d, int lane, uint8_t* stage,
                                F fetch) {
#pragma unroll
    for (int c = 0; c < NCOL; c += 16) {
      if (c0 + c >= d) break;  // warp-uniform
      float v[16];
      fetch(c0 + c, v);
      __syncwarp();  // the previous piece has been read
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), k = lane & 3;
        const float4 x =
            *reinterpret_cast<const float4*>(stage + r * 64 + ((k ^ ((r >> 1) & 3)) << 4));
        if (r < rows && c0 + c + 4 * k < d)
          *reinterpret_cast<float4*>(out + (size_t)r * d + c0 + c + 4 * k) = x;
      }
    }
  }
  // Rows of tile t that hold a request's query head, and its first row in a slot.
  FA_DEV static int tile_rows(const View& g, const Item& it, int t) {
    return min(g.p.s.per_tile, g.p.s.B - request(g, it, t)) * g.p.s.per_kv;
  }
  // The part's o and e of one warp's 32 rows.
  template <int D>
  FA_DEV static void store(const View& g, const Item& it, int t, int warp, int lane, uint32_t ocol,
                           float m_ref, float l, uint8_t* stage, const CUtensorMap*, int d) {
    const DecodeSizes& s = g.p.s;
    const int rows = tile_rows(g, it, t) - warp * 32;
    if (rows <= 0) return;  // warp-uniform
    const size_t at = (size_t)it.slot * s.pair_rows + t * s.per_tile * s.per_kv + warp * 32;
    const float inv = part_inverse(l);
    write_part<D>(s.prefix_o + at * d, rows, 0, d, lane, stage, [&](int c, float (&v)[16]) {
      uint32_t x[16];
      tmem_ld16(ocol + c, x);
      tmem_ld_wait();
      reg_fence16(x);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(x[e]) * inv;
    });
    if (lane < rows) s.prefix_e[at + lane] = m_ref + lg2(l);
  }
  // The same from the two halves of the keys: (m, l) = s0 with O in columns ocol, s1 with
  // O in ocol + D (nothing there where `second` is false). Group t writes half of the
  // columns.
  template <int D>
  FA_DEV static void store_joined(const View& g, const Item& it, int t, int warp, int lane,
                                  uint32_t ocol, float2 s0, float2 s1, bool second,
                                  uint8_t* stage, const CUtensorMap*, int d) {
    const DecodeSizes& s = g.p.s;
    const int rows = tile_rows(g, it, 0) - warp * 32;
    if (rows <= 0) return;  // warp-uniform
    const size_t at = (size_t)it.slot * s.pair_rows + warp * 32;
    const float top = second ? fmaxf(s0.x, s1.x) : s0.x;
    const float ref = top == -INFINITY ? 0.f : top;
    float f0 = ex2(s0.x - ref), f1 = second ? ex2(s1.x - ref) : 0.f;
    const float l = second ? s0.y * f0 + s1.y * f1 : s0.y * f0;
    if (l != 0.f) {  // else both are 0
      f0 /= l;
      f1 /= l;
    }
    write_part<D / 2>(s.prefix_o + at * d, rows, t * (D / 2), d, lane, stage,
                      [&](int c, float (&v)[16]) {
                        uint32_t x[16], y[16];
                        tmem_ld16(ocol + c, x);
                        if (second) tmem_ld16(ocol + D + c, y);
                        tmem_ld_wait();
                        reg_fence16(x);
                        if (second) reg_fence16(y);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                          v[e] = __uint_as_float(x[e]) * f0;
                          if (second) v[e] += __uint_as_float(y[e]) * f1;
                        }
                      });
    if (t == 0 && lane < rows) s.prefix_e[at + lane] = ref + lg2(l);
  }
  FA_DEV static void idle_warps(const View&, int, int, int) {}
};

// ================================================================== row tiles
// 16 query rows of one request and key/value head (rows past the group's are zeros) in
// one warp, with their output and statistics: rows lane / 4 and lane / 4 + 8 of each
// fragment, columns 8 n + 2 (lane % 4) + {0, 1}.
template <int D>
struct RowTile {
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float m0, m1, l0, l1;

  // The first `rows` rows, row r at src + at(r).
  template <class F>
  FA_DEV void load(const __nv_bfloat16* src, F at, int rows, int d) {
    const int lane = threadIdx.x & 31, qr = lane >> 2, qc = (lane & 3) * 2;
    const int last = max(rows - 1, 0);
    const __nv_bfloat16 *row0 = src + at(min(qr, last)), *row1 = src + at(min(qr + 8, last));
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = qr + (e & 1) * 8, col = kk * 16 + (e >> 1) * 8 + qc;
        q[kk][e] = row < rows && col < d
                       ? *reinterpret_cast<const unsigned int*>((e & 1 ? row1 : row0) + col)
                       : 0u;
      }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }

  // One stage of 16 keys (K at kb, V at vb in shared memory, D * 2 bytes a key, 16-byte
  // piece j of key r at j ^ (r % 8)), of which the first `keys` count.
  FA_DEV void step(uint32_t kb, uint32_t vb, int keys, float scale_log2) {
    const int lane = threadIdx.x & 31, qc = (lane & 3) * 2;
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};  // keys 0..7, 8..15
    {
      const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b[4];
        ldmatrix_x4(b, kb + row * (2 * D) + (((kk * 2 + half) ^ (row & 7)) << 4));
        mma_16816(sa, q[kk], b[0], b[1]);
        mma_16816(sb, q[kk], b[2], b[3]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sa[e] *= scale_log2;
      sb[e] *= scale_log2;
    }
    if (keys < 16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (qc + (e & 1) >= keys) sa[e] = -INFINITY;
        if (8 + qc + (e & 1) >= keys) sb[e] = -INFINITY;
      }
    }
    float x0 = fmaxf(fmaxf(sa[0], sa[1]), fmaxf(sb[0], sb[1]));
    float x1 = fmaxf(fmaxf(sa[2], sa[3]), fmaxf(sb[2], sb[3]));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    // The reference maximum moves only when a row passes it by 2^8 (as in the forward
    // kernel): most steps need no rescaling.
    if (__any_sync(0xffffffffu, x0 > m0 + kRescaleThreshold || x1 > m1 + kRescaleThreshold)) {
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float c0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0);
      const float c1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= c0;
        o[n][1] *= c0;
        o[n][2] *= c1;
        o[n][3] *= c1;
      }
    }
    const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sa[e] = ex2(sa[e] - u0);
      sb[e] = ex2(sb[e] - u0);
      sa[2 + e] = ex2(sa[2 + e] - u1);
      sb[2 + e] = ex2(sb[2 + e] - u1);
    }
    l0 += (sa[0] + sa[1]) + (sb[0] + sb[1]);
    l1 += (sa[2] + sa[3]) + (sb[2] + sb[3]);
    // P in bf16 (the products' operand type), l from the values before rounding
    const uint32_t pa[4] = {pack_bf16(sa[0], sa[1]), pack_bf16(sa[2], sa[3]),
                            pack_bf16(sb[0], sb[1]), pack_bf16(sb[2], sb[3])};
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      ldmatrix_x4_trans(b, vb + row * (2 * D) + (((n * 2 + half) ^ (row & 7)) << 4));
      mma_16816(o[2 * n], pa, b[0], b[1]);
      mma_16816(o[2 * n + 1], pa, b[2], b[3]);
    }
  }

  // The rows' sums over the four lanes that share a row.
  FA_DEV void finish() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  }
};

// Copies a stage in the background: rows [0, keys) of K and V from row `row0` of the
// caches (rows of d values), zeros behind them and behind column d.
template <int D>
FA_DEV void load_stage(uint32_t dst, const __nv_bfloat16* Kc, const __nv_bfloat16* Vc, size_t row0,
                       int keys, int d) {
  constexpr int PPR = D / 8;  // 16-byte pieces of a row
  const int lane = threadIdx.x & 31, first = lane / PPR, piece = lane % PPR;
#pragma unroll
  for (int i = 0; i < 16 * PPR / 32; ++i) {
    const int r = first + i * (32 / PPR);
    const bool in = r < keys && 8 * piece < d;
    const size_t at = in ? (row0 + r) * d + 8 * piece : 0;
    const uint32_t to = dst + r * (2 * D) + ((piece ^ (r & 7)) << 4);
    cp_async16(to, Kc + at, in ? 16 : 0);
    cp_async16(to + 16 * 2 * D, Vc + at, in ? 16 : 0);
  }
}

// ================================================================== own kernel
struct OwnParams {
  DecodeSizes s;
  const __nv_bfloat16 *Q, *Kc, *Vc;
  const int *table, *lens, *prefix_len;
  int prefix_cap, max_pages, num_pages, page_shift;  // prefix_cap: keys
  float scale_log2;
};

template <int D>
struct OwnCfg {
  static constexpr int ROW = D * 2;          // bytes of a key
  static constexpr int KEYS = 16;            // keys of a ring stage
  static constexpr int STAGES = 3;
  static constexpr int PART = KEYS * ROW;    // K or V of a stage
  static constexpr int STAGE = 2 * PART;
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int RINGS = kOwnWarps * WARP;  // then first[B + 1]
};

// Length of request b's own keys, at most what its table row holds.
FA_DEV int own_keys(const OwnParams& p, int b) {
  return max(0, min(p.lens[b], p.max_pages << p.page_shift));
}

// Pages are read 16 keys at a time (a page holds a multiple of 16): per stage 16 rows of
// K and of V, 16-byte piece j of row r at j ^ (r % 8), which ldmatrix reads without bank
// conflicts. Three stages a warp keep two in flight.
template <int D>
__global__ void __launch_bounds__(32 * kOwnWarps) own_kernel(const __grid_constant__ OwnParams p) {
  using C = OwnCfg<D>;
  extern __shared__ __align__(128) uint8_t smem_own[];
  __shared__ int warp_sums[kOwnWarps];
  grid_launch_dependents();
  int* first = reinterpret_cast<int*>(smem_own + C::RINGS);
  const DecodeSizes& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kThreads = 32 * kOwnWarps;

  // Chunks before each request (exclusive scan of the lengths).
  const int shared_keys = prefix_keys(p.prefix_len, p.prefix_cap);  // in flight with them
  int run = 0;
  for (int b0 = 0; b0 < s.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < s.B) {
      const int len = p.lens[b];
      if ((len < 0 || len > p.max_pages << p.page_shift) && blockIdx.x == 0)
        atomicOr(&g_prefix_status, kDeviceIndexBit);
      n = own_chunks(len, p.max_pages << p.page_shift);
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = run, sum = 0;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      sum += warp_sums[w];
    }
    if (b < s.B) first[b] = before + x - n;
    run += sum;
    __syncthreads();
  }
  if (threadIdx.x == 0) first[s.B] = run;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= s.B; b += kThreads) s.first[b] = first[b];

  const int chunks = run;  // of one (head, row tile)
  const unsigned units = (unsigned)(s.Hkv * s.row_tiles * s.B);
  const int share = prefix_share(s, (shared_keys + 127) / 128, chunks);
  const Split sp = own_split(s, chunks, share);
  // The first workers on different SMs; the blocks past the share get none.
  const int active = own_share(s, share);
  const int me = (int)blockIdx.x < active ? warp * active + (int)blockIdx.x : sp.workers;
  if (me >= sp.workers) {  // no barrier of the block follows
    grid_wait();
    return;
  }
  const unsigned x_end = sp.start(me + 1), x_begin = sp.start(me);

  // A run of chunks of one unit.
  struct Run {
    int b, ht, key, key_end, len;  // request, head and row tile, keys [key, key_end)
    unsigned x0, x1, u0, u1;       // this run's steps, the unit's steps
  };
  auto run_at = [&](unsigned x) {
    Run r;
    r.ht = (int)(x / (unsigned)chunks);
    const int in = (int)(x - (unsigned)(r.ht * chunks));
    int lo = 0, hi = s.B;  // first[lo] <= in < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= in)
        lo = mid;
      else
        hi = mid;
    }
    r.b = lo;
    r.u0 = (unsigned)(r.ht * chunks + first[lo]);
    r.u1 = (unsigned)(r.ht * chunks + first[lo + 1]);
    r.x0 = x;
    r.x1 = min(r.u1, x_end);
    r.len = own_keys(p, lo);
    r.key = (int)(x - r.u0) * kOwnChunk;
    r.key_end = min(r.len, (int)(r.x1 - r.u0) * kOwnChunk);
    return r;
  };

  const uint32_t ring = smem_u32(smem_own) + warp * C::WARP;
  // ---- the issuing side: runs STAGES - 1 stages ahead of the products
  Run ir = run_at(x_begin);
  int i_page = 0, i_at = 32;  // pages of 32 stages, one per lane; the next of them
  bool i_more = true;
  int i_stage = 0;
  const size_t head_rows = (size_t)1 << p.page_shift;
  auto issue = [&]() {
    if (i_more) {
      if (i_at == 32) {
        const int key = ir.key + lane * C::KEYS;
        int page = 0;
        if (key < ir.key_end)
          page = p.table[(size_t)ir.b * p.max_pages + (key >> p.page_shift)];
        if ((unsigned)page >= (unsigned)p.num_pages) {
          atomicOr(&g_prefix_status, kDeviceIndexBit);
          page = 0;
        }
        i_page = page;
        i_at = 0;
      }
      const int page = __shfl_sync(0xffffffffu, i_page, i_at);
      const int hk = ir.ht / s.row_tiles;
      const size_t row0 = ((size_t)page * s.Hkv + hk) * head_rows + (ir.key & (head_rows - 1));
      load_stage<D>(ring + i_stage * C::STAGE, p.Kc, p.Vc, row0, ir.key_end - ir.key, s.d);
      ++i_at;
      ir.key += C::KEYS;
      if (ir.key >= ir.key_end) {
        if (ir.x1 < x_end) {
          ir = run_at(ir.x1);
          i_at = 32;
        } else {
          i_more = false;
        }
      }
    }
    i_stage = i_stage + 1 == C::STAGES ? 0 : i_stage + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) issue();

  // ---- the products
  const int qr = lane >> 2, qc = (lane & 3) * 2;  // row and first column of a fragment
  int stage = 0;
  RowTile<D> tile;
  for (unsigned x = x_begin; x < x_end;) {
    const Run r = run_at(x);
    x = r.x1;
    const int hk = r.ht / s.row_tiles, rt = r.ht - hk * s.row_tiles;
    const int rows = min(16, s.per_kv - rt * 16);
    tile.load(p.Q + ((size_t)r.b * s.Hq + hk * s.per_kv + rt * 16) * s.d,
              [&](int row) { return row * s.d; }, rows, s.d);
    for (int key = r.key; key < r.key_end; key += C::KEYS) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();  // the stage has landed for every lane, and the last one is read
      issue();
      const uint32_t kb = ring + stage * C::STAGE;
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      tile.step(kb, kb + C::PART, r.key_end - key, p.scale_log2);
    }
    tile.finish();
    const unsigned unit = (unsigned)(r.ht * s.B + r.b);
    const unsigned slot = r.x0 == r.u0 && r.x1 == r.u1
                              ? unit
                              : units + 2u * (unsigned)me + (r.x0 == r.u0 ? 1u : 0u);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = qr + 8 * e;
      if (row >= rows) continue;
      const float inv = part_inverse(e ? tile.l1 : tile.l0);
      float* out = s.own_o + ((size_t)slot * s.own_rows + row) * s.d;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        if (8 * n < s.d)
          *reinterpret_cast<float2*>(out + 8 * n + qc) =
              make_float2(tile.o[n][2 * e] * inv, tile.o[n][2 * e + 1] * inv);
      if ((lane & 3) == 0)
        s.own_e[(size_t)slot * s.own_rows + row] =
            e ? tile.m1 + lg2(tile.l1) : tile.m0 + lg2(tile.l0);
    }
  }
  cp_async_wait<0>();
  // This kernel needs nothing of the prefix kernel, beside which it may run, but it
  // completes after it: the join kernel waits for this one.
  grid_wait();
}

// ================================================================== whole kernel
// Small calls, where three kernels' latency would be most of the time: a cluster of one
// to eight thread blocks per request and row tile takes all of its keys, the prefix's and
// its own, 16 at a time in turn by the warps, and joins the warps' parts through the
// cluster's shared memory. The prefix is read again for every request, from L2 but for
// the first. A warp's stage takes about 0.85 us (the latency of a copy over the two in
// flight), so that few requests want many blocks each.
struct WholeParams {
  DecodeSizes s;
  const __nv_bfloat16 *Q, *Kc, *Vc;
  const int *pages, *prefix_len, *table, *lens;
  __nv_bfloat16* O;
  float* L;
  int prefix_cap, max_pages, num_pages, page_shift;  // prefix_cap: keys
  int cluster;                                        // blocks of a cluster
  float scale_log2;
};
constexpr int kWholeWarps = 8;
// Floats from row to row of outputs in shared memory: eight rows' fragments, 32 bytes of
// each, lie in different banks.
template <int D>
constexpr int kPartPitch = D + 8;
template <int D>
struct WholeCfg {
  static constexpr int STAGES = 3;
  static constexpr int STAGE = 2 * 16 * 2 * D;
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int BYTES = kWholeWarps * WARP;
  static_assert(BYTES >= (kWholeWarps + 1) * 16 * kPartPitch<D> * 4,
                "the rings hold the outputs at the end");
};

// Joins `n` parts of a row's four columns c .. c + 3: stat(i) gives part i's (m, l) and
// value(i) its four columns, both relative to m. Returns the joined m and l: (-inf, 0)
// where no part has a finite score, so that a further join gives them no say in its maximum.
template <class S, class V>
FA_DEV float2 join_parts(int n, float4& acc, S stat, V value) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) m = fmaxf(m, stat(i).x);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= n) break;
    const float2 ml = stat(i);
    const float4 x = value(i);
    const float f = ex2(ml.x - ref);
    l += f * ml.y;
    acc.x += f * x.x;
    acc.y += f * x.y;
    acc.z += f * x.z;
    acc.w += f * x.w;
  }
  return make_float2(m, l);
}

template <int D>
__global__ void __launch_bounds__(32 * kWholeWarps)
    whole_kernel(const __grid_constant__ WholeParams p) {
  using C = WholeCfg<D>;
  extern __shared__ __align__(128) uint8_t smem_whole[];
  __shared__ float2 stats[kWholeWarps][16];  // a warp's m and l per row
  __shared__ float2 joined[16];              // this block's
  const DecodeSizes& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / p.cluster, rank = blockIdx.x - unit * p.cluster;
  const int b = unit % s.B, ht = unit / s.B;
  const int hk = ht / s.row_tiles, rt = ht - hk * s.row_tiles;
  const int rows = min(16, s.per_kv - rt * 16);
  const int own_cap = p.max_pages << p.page_shift;
  grid_wait();
  grid_launch_dependents();
  const int len = p.lens[b], plen = p.prefix_len ? *p.prefix_len : 0;
  if (len < 0 || len > own_cap || plen < 0 || plen > p.prefix_cap)
    if (threadIdx.x == 0) atomicOr(&g_prefix_status, kDeviceIndexBit);
  const int own = max(0, min(len, own_cap)), shared = max(0, min(plen, p.prefix_cap));
  const int p_steps = (shared + 15) / 16, steps = p_steps + (own + 15) / 16;

  // This warp's steps me, me + all, ...
  const int me = rank * kWholeWarps + warp, all = p.cluster * kWholeWarps;
  const int mine = max(0, (steps - me + all - 1) / all);
  const uint32_t ring = smem_u32(smem_whole) + warp * C::WARP;
  const size_t head_rows = (size_t)1 << p.page_shift;
  auto keys_of = [&](int i, int& key) {  // step i's first key in its list, and its keys
    key = i < p_steps ? 16 * i : 16 * (i - p_steps);
    return min(16, (i < p_steps ? shared : own) - key);
  };
  int ids = 0;  // pages of this warp's steps 32 k .. 32 k + 31, one per lane
  auto issue = [&](int j) {
    if (j < mine) {
      if ((j & 31) == 0) {
        const int i = me + (j + lane) * all;
        ids = 0;
        if (j + lane < mine) {
          int key;
          keys_of(i, key);
          ids = *(i < p_steps ? p.pages + (key >> p.page_shift)
                              : p.table + (size_t)b * p.max_pages + (key >> p.page_shift));
          if ((unsigned)ids >= (unsigned)p.num_pages) {
            atomicOr(&g_prefix_status, kDeviceIndexBit);
            ids = 0;
          }
        }
      }
      const int page = __shfl_sync(0xffffffffu, ids, j & 31);
      int key;
      const int n = keys_of(me + j * all, key);
      load_stage<D>(ring + (j % C::STAGES) * C::STAGE, p.Kc, p.Vc,
                    ((size_t)page * s.Hkv + hk) * head_rows + (key & (head_rows - 1)), n, s.d);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < C::STAGES - 1; ++j) issue(j);
  RowTile<D> tile;
  tile.load(p.Q + ((size_t)b * s.Hq + hk * s.per_kv + rt * 16) * s.d,
            [&](int row) { return row * s.d; }, rows, s.d);
  for (int j = 0; j < mine; ++j) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();  // the stage has landed for every lane, and the last one is read
    issue(j + C::STAGES - 1);
    int key;
    const int n = keys_of(me + j * all, key);
    const uint32_t kb = ring + (j % C::STAGES) * C::STAGE;
    tile.step(kb, kb + C::STAGE / 2, n, p.scale_log2);
  }
  tile.finish();
  cp_async_wait<0>();
  __syncthreads();  // every ring is read: they hold the outputs now

  constexpr int PITCH = kPartPitch<D>;
  float* part = reinterpret_cast<float*>(smem_whole);  // [warp][row][PITCH]
  const int qr = lane >> 2, qc = (lane & 3) * 2;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float* out = part + (warp * 16 + qr + 8 * e) * PITCH;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(out + 8 * n + qc) =
          make_float2(tile.o[n][2 * e], tile.o[n][2 * e + 1]);
    if ((lane & 3) == 0)
      stats[warp][qr + 8 * e] = e ? make_float2(tile.m1, tile.l1) : make_float2(tile.m0, tile.l0);
  }
  __syncthreads();
  // The block's warps, then the cluster's blocks; those with keys come first.
  float* const mid = part + kWholeWarps * 16 * PITCH;  // [row][PITCH] of this block
  const int warps_in = min(kWholeWarps, max(0, steps - rank * kWholeWarps));
  const int blocks_in = min(p.cluster, (steps + kWholeWarps - 1) / kWholeWarps);
  auto write = [&](int r, int c, float4 acc, float2 ml, bool any) {
    const float inv = any ? 1.f / ml.y : 0.f;
    const size_t row = (size_t)b * s.Hq + hk * s.per_kv + rt * 16 + r;
    *reinterpret_cast<uint2*>(p.O + row * s.d + c) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (c == 0) p.L[row] = any ? (ml.x + lg2(ml.y)) * kLn2 : -INFINITY;
  };
  for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kWholeWarps) {
    const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
    float4 acc;
    const float2 ml = join_parts(
        warps_in, acc, [&](int w) { return stats[w][r]; },
        [&](int w) { return *reinterpret_cast<const float4*>(part + (w * 16 + r) * PITCH + c); });
    if (p.cluster == 1) {
      if (c < s.d) write(r, c, acc, ml, steps > 0);
    } else {
      *reinterpret_cast<float4*>(mid + r * PITCH + c) = acc;
      if (c == 0) joined[r] = ml;
    }
  }
  if (p.cluster == 1) return;
  cluster_sync();  // every block's rows are written
  for (int i = rank * 32 * kWholeWarps + threadIdx.x; i < rows * (D / 4);
       i += p.cluster * 32 * kWholeWarps) {
    const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
    if (c >= s.d) continue;
    float4 acc;
    const float2 ml = join_parts(
        blocks_in, acc, [&](int k) { return cluster_ld2(cluster_map(smem_u32(&joined[r]), k)); },
        [&](int k) { return cluster_ld4(cluster_map(smem_u32(mid + r * PITCH + c), k)); });
    write(r, c, acc, ml, steps > 0);
  }
  cluster_sync();  // no block leaves while its rows are read
}

// ================================================================== shared kernel
// The prefix kernel's work for few rows a key/value head, where a 128-row tile
// would be mostly empty and one SM's chain of scores, softmax and product, not the keys'
// way from HBM, sets the time (one request, 32/8 heads, d = 128, behind 100000 keys: 66 us,
// 6.2 TB/s, against 82 us with the tiles; 16 requests, 8/8 heads, behind 20000: 21.5 and
// 30.1). With d = 128 it takes 16 rows only: two row tiles a warp fill the registers, and a
// unit's start and end take 3 us longer than the 128-row tile's. Eight warps take a worker's
// piece, 16 keys each of every 128, and each streams its keys through a ring of its own, as
// in the own kernel; at the end of a unit they join their parts in shared memory. Same
// pieces, slots and parts.
struct SharedParams {
  DecodeSizes s;
  const __nv_bfloat16 *Q, *Kc, *Vc;
  const int *pages, *len, *lens;
  int cap, own_cap, num_pages, page_shift;  // capacities in keys
  float scale_log2;
};
constexpr int kSharedWarps = 8;
template <int D>
constexpr int kSharedTiles = D == 64 ? 2 : 1;  // row tiles of a warp at most
template <int D>
struct SharedCfg {
  static constexpr int ROWS = 16 * kSharedTiles<D>;
  static constexpr int STAGE = 2 * 16 * 2 * D;
  static constexpr int STAGES = 192 * 1024 / (kSharedWarps * STAGE);
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int BYTES = kSharedWarps * WARP;
  static_assert(BYTES >= kSharedWarps * ROWS * kPartPitch<D> * 4,
                "the rings hold the outputs");
};

template <int D, int TILES>
__global__ void __launch_bounds__(32 * kSharedWarps, 1)
    shared_kernel(const __grid_constant__ SharedParams p) {
  using C = SharedCfg<D>;
  extern __shared__ __align__(128) uint8_t smem_shared[];
  __shared__ float2 stats[kSharedWarps][C::ROWS];  // a warp's m and l per row
  const DecodeSizes& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  grid_launch_dependents();  // the own kernel
  const int n = *p.len;
  int chunks = 0;  // each warp on its own; read beside n
  for (int b = lane; b < s.B; b += 32) chunks += own_chunks(p.lens[b], p.own_cap);
  chunks = __reduce_add_sync(0xffffffffu, chunks);
  if ((n < 0 || n > p.cap) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(&g_prefix_status, kDeviceIndexBit);
  const int keys = max(0, min(n, p.cap)), blocks = (keys + 127) / 128;
  const Split split = prefix_split(s, blocks, prefix_share(s, blocks, chunks));
  const int cta = (int)blockIdx.x;
  if (cta >= split.workers) return;

  const int rows = s.B * s.per_kv;  // one pair: a unit is a head
  const uint32_t ring = smem_u32(smem_shared) + warp * C::WARP;
  const size_t head_rows = (size_t)1 << p.page_shift;
  const unsigned end = split.start(cta + 1);
  for (unsigned x = split.start(cta); x < end;) {
    const unsigned hk = x / (unsigned)blocks, u0 = hk * (unsigned)blocks;
    const unsigned x1 = min(end, u0 + (unsigned)blocks);
    const int k0 = (int)(x - u0) * 128, k1 = min(keys, (int)(x1 - u0) * 128);
    const int stages = (int)(x1 - x);
    int ids = 0;  // pages of this warp's stages 32 k .. 32 k + 31, one per lane
    auto issue = [&](int j) {
      if (j < stages) {
        const int key = k0 + 128 * j + 16 * warp;
        if ((j & 31) == 0) {
          const int mine = key + 128 * lane;
          ids = 0;
          if (mine < k1) ids = p.pages[mine >> p.page_shift];
          if ((unsigned)ids >= (unsigned)p.num_pages) {
            atomicOr(&g_prefix_status, kDeviceIndexBit);
            ids = 0;
          }
        }
        const int page = __shfl_sync(0xffffffffu, ids, j & 31);
        load_stage<D>(ring + (j % C::STAGES) * C::STAGE, p.Kc, p.Vc,
                      ((size_t)page * s.Hkv + hk) * head_rows + (key & (head_rows - 1)), k1 - key,
                      s.d);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < C::STAGES - 1; ++j) issue(j);
    RowTile<D> tile[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
      tile[t].load(p.Q + (size_t)hk * s.per_kv * s.d,
                   [&](int r) {
                     const int b = (16 * t + r) / s.per_kv;
                     return ((size_t)b * s.Hq + (16 * t + r - b * s.per_kv)) * s.d;
                   },
                   rows - 16 * t, s.d);
    for (int j = 0; j < stages; ++j) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();  // the stage has landed for every lane, and the last one is read
      issue(j + C::STAGES - 1);
      const int count = k1 - (k0 + 128 * j + 16 * warp);
      if (count <= 0) break;  // the last stage
      const uint32_t kb = ring + (j % C::STAGES) * C::STAGE;
#pragma unroll
      for (int t = 0; t < TILES; ++t) tile[t].step(kb, kb + C::STAGE / 2, count, p.scale_log2);
    }
    cp_async_wait<0>();
    __syncthreads();  // every ring is read: they hold the outputs now

    constexpr int PITCH = kPartPitch<D>;
    float* part = reinterpret_cast<float*>(smem_shared);  // [warp][row][PITCH]
    const int qr = lane >> 2, qc = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      tile[t].finish();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * t + qr + 8 * e;
        float* out = part + (warp * C::ROWS + row) * PITCH;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(out + 8 * i + qc) =
              make_float2(tile[t].o[i][2 * e], tile[t].o[i][2 * e + 1]);
        if ((lane & 3) == 0)
          stats[warp][row] = e ? make_float2(tile[t].m1, tile[t].l1)
                               : make_float2(tile[t].m0, tile[t].l0);
      }
    }
    __syncthreads();
    const int warps_in = min(kSharedWarps, (k1 - k0 + 15) / 16);
    const unsigned slot = x == u0 && x1 == u0 + (unsigned)blocks
                              ? hk
                              : (unsigned)s.Hkv + 2u * (unsigned)cta + (x == u0 ? 1u : 0u);
    for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kSharedWarps) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      float4 acc;
      const float2 ml = join_parts(
          warps_in, acc, [&](int w) { return stats[w][r]; },
          [&](int w) {
            return *reinterpret_cast<const float4*>(part + (w * C::ROWS + r) * PITCH + c);
          });
      const float inv = part_inverse(ml.y);
      const size_t at = (size_t)slot * s.pair_rows + r;
      if (c < s.d)
        *reinterpret_cast<float4*>(s.prefix_o + at * s.d + c) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (c == 0) s.prefix_e[at] = ml.x + lg2(ml.y);
    }
    x = x1;
    if (x < end) __syncthreads();  // the outputs are read: the rings may be filled again
  }
}

// ================================================================== join kernel
struct JoinParams {
  DecodeSizes s;
  const int *prefix_len, *lens;
  int prefix_cap, own_cap;  // keys
  __nv_bfloat16* O;
  float* L;
};

// A row (request, query head) is joined by one warp, or by kJoinWarps where there are
// too few rows to fill the GPU and each has many parts. Lane j of a warp looks up every
// 32nd part (its slot and e); then the warp adds the parts up, four columns a lane and
// four or eight parts in flight (fewer where many rows share the registers): the kernel
// is bound by the latency of these loads. A row
// without keys gets O = 0, L = -inf.
constexpr int kJoinWarps = 8;
template <int WARPS>  // of a row
__global__ void __launch_bounds__(32 * kJoinWarps, WARPS == 1 ? 4 : 1)
    join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float4 sums[kJoinWarps][32];
  __shared__ float2 stats[kJoinWarps];  // a warp's reference and weight sum
  const DecodeSizes& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = WARPS == 1 ? blockIdx.x * kJoinWarps + warp : blockIdx.x;
  const int mine = WARPS == 1 ? 0 : warp;  // this warp of the row's
  const int b = min(row / s.Hq, s.B - 1), hq = min(row - b * s.Hq, s.Hq - 1);
  const int hk = hq / s.per_kv, in = hq - hk * s.per_kv;

  // Parts of the prefix, then of the request's own keys. The lengths are the call's inputs:
  // they were written before the own kernel started, which launched this one, so that the
  // parts are found while that kernel runs (1.2 us). Many requests' lengths take longer
  // to sum up than to read from where the own kernel puts their sums.
  const int blocks = (prefix_keys(p.prefix_len, p.prefix_cap) + 127) / 128;
  int f0 = 0, f1 = 0, chunks = 0;
  if (s.B <= 256) {
    for (int i = lane; i < s.B; i += 32) {
      const int n = own_chunks(p.lens[i], p.own_cap);
      chunks += n;
      if (i < b) f0 += n;
      if (i == b) f1 = n;
    }
    chunks = __reduce_add_sync(0xffffffffu, chunks);
    f0 = __reduce_add_sync(0xffffffffu, f0);
    f1 = __reduce_add_sync(0xffffffffu, f1) + f0;
  } else {
    grid_wait();
    chunks = s.first[s.B];
    f0 = s.first[b];
    f1 = s.first[b + 1];
  }
  const int share = prefix_share(s, blocks, chunks);
  int pparts = 0, pfirst = 0;
  const int pair = b / (2 * s.per_tile);
  const unsigned punit = (unsigned)(pair * s.Hkv + hk);
  if (blocks > 0) {
    const Split sp = prefix_split(s, blocks, share);
    pfirst = sp.owner(punit * (unsigned)blocks);
    pparts = sp.owner((punit + 1) * (unsigned)blocks - 1) - pfirst + 1;
  }
  const int prow = (b - pair * 2 * s.per_tile) * s.per_kv + in;
  const int ht = hk * s.row_tiles + in / 16;
  int oparts = 0, ofirst = 0;
  if (f1 > f0) {
    const Split sp = own_split(s, chunks, share);
    ofirst = sp.owner((unsigned)(ht * chunks + f0));
    oparts = sp.owner((unsigned)(ht * chunks + f1) - 1u) - ofirst + 1;
  }
  const unsigned punits = (unsigned)(s.pairs * s.Hkv);
  const unsigned ounits = (unsigned)(s.Hkv * s.row_tiles * s.B);
  const int parts = pparts + oparts;
  grid_wait();
  grid_launch_dependents();
  if (row >= s.B * s.Hq) return;  // WARPS == 1 only: no barrier follows

  float ref = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < parts; base += 32 * WARPS) {
    const int i = base + lane * WARPS + mine;
    const float* o = nullptr;
    float e = -INFINITY;
    if (i < pparts) {
      const size_t at = (size_t)Split::slot(punit, punits, pparts, pfirst, i) * s.pair_rows + prow;
      o = s.prefix_o + at * s.d;
      e = s.prefix_e[at];
    } else if (i < parts) {
      const unsigned slot =
          Split::slot((unsigned)(ht * s.B + b), ounits, oparts, ofirst, i - pparts);
      const size_t at = (size_t)slot * s.own_rows + in % 16;
      o = s.own_o + at * s.d;
      e = s.own_e[at];
    }
    float top = e;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float next = fmaxf(ref, top);
    const float back = ref == next ? 1.f : ex2(ref - next);  // 0 on the first round
    ref = next;
    const float weight = o ? ex2(e - (ref == -INFINITY ? 0.f : ref)) : 0.f;
    sum = sum * back + weight;  // this lane's parts
    acc.x *= back;
    acc.y *= back;
    acc.z *= back;
    acc.w *= back;
    const int n = min(32, (parts - base - mine + WARPS - 1) / WARPS);  // lanes with a part
    constexpr int U = WARPS == 1 ? 4 : 8;
    for (int j = 0; j < n; j += U) {
      float4 v[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* src = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (j + u) & 31));
        w[u] = __shfl_sync(0xffffffffu, weight, (j + u) & 31);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j + u < n && 4 * lane < s.d) v[u] = reinterpret_cast<const float4*>(src)[lane];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u >= n) break;
        acc.x += w[u] * v[u].x;
        acc.y += w[u] * v[u].y;
        acc.z += w[u] * v[u].z;
        acc.w += w[u] * v[u].w;
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (WARPS > 1) {
    sums[warp][lane] = acc;
    if (lane == 0) stats[warp] = make_float2(ref, sum);
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, stats[w].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      // a warp without parts has reference -inf and adds nothing
      const float f = w < parts ? ex2(stats[w].x - (top == -INFINITY ? 0.f : top)) : 0.f;
      const float4 v = sums[w][lane];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
      sum += f * stats[w].y;
    }
    ref = top;
  }
  const float inv = parts > 0 ? 1.f / sum : 0.f;
  if (4 * lane < s.d)
    reinterpret_cast<uint2*>(p.O + (size_t)row * s.d)[lane] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0) p.L[row] = parts > 0 ? (ref + lg2(sum)) * kLn2 : -INFINITY;
}

int decode_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms < kMaxSms ? sms : kMaxSms;
}

// Blocks per unit with which the whole kernel is expected to beat the three kernels, or
// 0 where it is not, from the capacities (the lengths are known on the device only). Both
// forms were timed at 72 points (8, 2 and 1 key/value heads of 4, 4 and 16 rows, 1 to 64
// requests, 64 to 8000 shared and 64 to 2048 own keys); in ns they fit
//   whole   1500 + waves (3000 + stages t), t = 850 (d > 64) or 460 for a warp's stage of
//           16 keys, + 1000 for a cluster, and 1 per 9000 bytes at least
//   three   11000 (9000 with the shared kernel) + 1 per 6000 bytes, every key read once,
//           + 2 per row joined
// to about 15 %; over 64 other points the form taken was 0.5 % slower than the better one.
// The two take 6.0 and 12.3 us for 16 requests of 2 x 4 heads, d = 64, behind 1024 keys
// with 512 own, and 58 and 26 us for 16 requests of 8 x 4 heads, d = 128, behind 8000 keys
// with 128 own.
template <int D>
unsigned whole_cluster(const DecodeSizes& s, int prefix_cap, int own_cap, int sms) {
  const long long keys = (long long)prefix_cap + own_cap;
  const long long units = (long long)s.Hkv * s.row_tiles * s.B;
  const long long per_block = 16 * kWholeWarps;  // keys of a stage of all warps
  // A cluster of eight needs eight free SMs of one GPC: no more than half of the SMs.
  int c = 1;
  while (c < 8 && 2 * c * units <= (c == 4 ? sms / 2 : sms) && keys >= 2 * c * per_block) c *= 2;
  const long long stages = (keys + c * per_block - 1) / (c * per_block);
  if (stages > 64 || units * c > 0x7fffffffLL) return 0;
  const long long slots = (long long)sms * (D == 128 ? 1 : 2);
  const long long waves = (units * c + slots - 1) / slots;
  const long long bytes = 4LL * s.d;  // K and V of one key
  long long whole = 1500 + waves * (3000 + stages * (D == 128 ? 850 : 460)) + (c > 1 ? 1000 : 0);
  if (whole < units * keys * bytes / 9000) whole = units * keys * bytes / 9000;
  const bool few = s.B * s.per_kv <= SharedCfg<D>::ROWS;
  const long long three = (few ? 9000 : 11000) +
                          (long long)s.Hkv * (prefix_cap + (long long)s.B * own_cap) * bytes / 6000 +
                          2LL * s.B * s.Hq;
  return whole <= three ? (unsigned)c : 0;
}

template <int D>
cudaError_t launch_decode_d(const DecodeArgs& a, cudaStream_t stream) {
  using C = FwdCfg<D>;
  DecodeSizes s = sizes_of(a.B, a.Hq, a.Hkv, a.d);
  lay_out(&s, a.workspace, a.prefix_cap * a.page, a.max_pages * a.page);
  const int sms = decode_sms();
  // No more blocks than the capacities can keep busy.
  const long long prefix_steps = (long long)s.pairs * s.Hkv * ceil_div(a.prefix_cap * a.page, 128);
  const long long own_steps =
      (long long)s.Hkv * s.row_tiles * s.B * ceil_div(a.max_pages * a.page, kOwnChunk);
  auto least = [](long long x, long long y) { return (unsigned)(x < y ? x : y); };
  const unsigned prefix_grid = least(sms, prefix_steps);
  const unsigned own_grid = least(sms * s.own_per_sm, own_steps > 0 ? own_steps : 1);
  s.sms = sms;
  s.prefix_workers = (int)prefix_grid;
  s.own_blocks = (int)own_grid;
  const int rows = a.B * s.per_kv;  // of a key/value head
  const bool few = rows <= SharedCfg<D>::ROWS;
  s.prefix_step_ns = few ? 8 * a.d : (a.B <= s.per_tile ? 1500 : 2400) - (D == 64 ? 500 : 0);
  s.units_magic = (unsigned)((0x100000000ull + s.pairs * s.Hkv - 1) / (unsigned)(s.pairs * s.Hkv));
  s.own_chunk_ns = 4 * a.d;
  int shift = 0;
  while ((1 << shift) < a.page) ++shift;
  cudaError_t e;
  const int cap = a.prefix_cap << shift;
  // One launch where it is expected to take less time than the three kernels.
  const unsigned cluster = whole_cluster<D>(s, cap, a.max_pages * a.page, sms);
  if (cluster > 0) {
    WholeParams w;
    w.s = s;
    w.Q = static_cast<const __nv_bfloat16*>(a.Q);
    w.Kc = static_cast<const __nv_bfloat16*>(a.Kc);
    w.Vc = static_cast<const __nv_bfloat16*>(a.Vc);
    w.pages = a.prefix_pages;
    w.prefix_len = a.prefix_cap > 0 ? a.prefix_len : nullptr;
    w.table = a.table;
    w.lens = a.lens;
    w.O = static_cast<__nv_bfloat16*>(a.O);
    w.L = a.L;
    w.prefix_cap = cap;
    w.max_pages = a.max_pages;
    w.num_pages = a.num_pages;
    w.page_shift = shift;
    w.cluster = (int)cluster;
    w.scale_log2 = a.scale * kLog2e;
    e = cudaFuncSetAttribute(whole_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WholeCfg<D>::BYTES);
    if (e != cudaSuccess) return e;
    return launch_as(whole_kernel<D>, (unsigned)(s.Hkv * s.row_tiles * s.B) * cluster,
                     32 * kWholeWarps, WholeCfg<D>::BYTES, stream, true, cluster, w);
  }
  if (a.prefix_cap > 0 && few) {
    SharedParams h;
    h.s = s;
    h.Q = static_cast<const __nv_bfloat16*>(a.Q);
    h.Kc = static_cast<const __nv_bfloat16*>(a.Kc);
    h.Vc = static_cast<const __nv_bfloat16*>(a.Vc);
    h.pages = a.prefix_pages;
    h.len = a.prefix_len;
    h.lens = a.lens;
    h.cap = cap;
    h.own_cap = a.max_pages << shift;
    h.num_pages = a.num_pages;
    h.page_shift = shift;
    h.scale_log2 = a.scale * kLog2e;
    auto kernel = rows <= 16 ? shared_kernel<D, 1> : shared_kernel<D, kSharedTiles<D>>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SharedCfg<D>::BYTES);
    if (e != cudaSuccess) return e;
    e = launch_early(kernel, prefix_grid, 32 * kSharedWarps, SharedCfg<D>::BYTES, stream, h);
    if (e != cudaSuccess) return e;
  } else if (a.prefix_cap > 0) {
    PrefixParams g;
    g.s = s;
    g.pages = a.prefix_pages;
    g.len = a.prefix_len;
    g.lens = a.lens;
    g.cap = cap;
    g.own_cap = a.max_pages << shift;
    g.page = a.page;
    g.page_shift = shift;
    g.box = a.page < 128 ? a.page : 128;
    g.num_pages = a.num_pages;
    CUtensorMap mq, mk, mv;
    const cuuint64_t qd[4] = {(cuuint64_t)a.d, (cuuint64_t)s.per_kv, (cuuint64_t)a.Hkv,
                              (cuuint64_t)a.B};
    const cuuint64_t qs[3] = {(cuuint64_t)a.d * 2, (cuuint64_t)s.per_kv * a.d * 2,
                              (cuuint64_t)a.Hq * a.d * 2};
    const cuuint32_t qb[4] = {64, (cuuint32_t)s.per_kv, 1, (cuuint32_t)s.per_tile};
    if (encode_tensor_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.Q), qd, qs,
                          qb, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
        make_bf16_head_map(&mk, a.Kc, a.num_pages * a.Hkv, a.page, a.d, g.box) != CUDA_SUCCESS ||
        make_bf16_head_map(&mv, a.Vc, a.num_pages * a.Hkv, a.page, a.d, g.box) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    FwdParams p;
    p.d = a.d;
    p.scale_log2 = a.scale * kLog2e;
    const bool one_tile = a.B <= s.per_tile;
    auto kernel = one_tile ? fwd_kernel<D, Prefix<true>> : fwd_kernel<D, Prefix<false>>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_early(kernel, prefix_grid, C::THREADS, C::SMEM, stream, mq, mk, mv, mk, p, g);
    if (e != cudaSuccess) return e;
  }
  OwnParams op;
  op.s = s;
  op.Q = static_cast<const __nv_bfloat16*>(a.Q);
  op.Kc = static_cast<const __nv_bfloat16*>(a.Kc);
  op.Vc = static_cast<const __nv_bfloat16*>(a.Vc);
  op.table = a.table;
  op.lens = a.lens;
  op.prefix_len = a.prefix_cap > 0 ? a.prefix_len : nullptr;
  op.prefix_cap = cap;
  op.max_pages = a.max_pages;
  op.num_pages = a.num_pages;
  op.page_shift = shift;
  op.scale_log2 = a.scale * kLog2e;
  const int own_smem = OwnCfg<D>::RINGS + (a.B + 1) * 4;
  e = cudaFuncSetAttribute(own_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           OwnCfg<D>::RINGS + (kMaxBatch + 1) * 4);
  if (e != cudaSuccess) return e;
  // Beside the prefix kernel, which has waited for what comes before it in the stream.
  e = launch_as(own_kernel<D>, own_grid, 32 * kOwnWarps, own_smem, stream, a.prefix_cap > 0, 1, op);
  if (e != cudaSuccess) return e;
  JoinParams jp;
  jp.s = s;
  jp.prefix_len = a.prefix_cap > 0 ? a.prefix_len : nullptr;
  jp.prefix_cap = cap;
  jp.lens = a.lens;
  jp.own_cap = a.max_pages << shift;
  jp.O = static_cast<__nv_bfloat16*>(a.O);
  jp.L = a.L;
  // A warp per row once there is a row for every fourth warp slot of the GPU's SMs.
  const int joined = a.B * a.Hq;
  return joined >= sms * 4
             ? launch_early(join_kernel<1>, (unsigned)ceil_div(joined, kJoinWarps),
                            32 * kJoinWarps, 0, stream, jp)
             : launch_early(join_kernel<kJoinWarps>, (unsigned)joined, 32 * kJoinWarps, 0, stream,
                            jp);
}

}  // namespace

size_t decode_workspace_bytes(int B, int Hq, int Hkv, int d, int prefix_cap, int own_cap) {
  DecodeSizes s = sizes_of(B, Hq, Hkv, d);
  return lay_out(&s, nullptr, prefix_cap, own_cap);
}

cudaError_t launch_prefix_decode(const DecodeArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_decode_d<128>(a, s) : launch_decode_d<64>(a, s);
}

cudaError_t prefix_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_prefix_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
