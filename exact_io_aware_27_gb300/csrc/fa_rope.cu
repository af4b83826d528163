// Norms of queries and keys for each head with the position rotation in the same pass, and
// their gradients.
//
//   forward   n = x r, r = (mean x^2 + eps)^-1/2;  u = n o w;  y = R u
//             R turns pairs of channels: (a, b) -> (a c - b s, b c + a s)
//   backward  g = R^T dy;  dw = sum over rows of g o n
//             dx = r (g o w - n mean(g o w o n))
//
// Bound by memory: a row is read once and written once (forward), or dy and x read and dx
// written (backward), and everything between stays in registers (fa_rope.cuh). 16384 rows of
// 32/8 heads, d = 128, norm and rotation: forward 53 us (336 MB, 6.3 TB/s, 93 % of the measured
// copy rate), backward 80 us (503 MB, 6.3 TB/s), with the sums of dw over the blocks 140 us
// together. Both took 179 us with a block per eight rows and loads into registers: the registers
// that hide the loads' way are then the limit.
#include "fa_launch.h"
#include "fa_rope.cuh"

namespace fa {

__device__ unsigned int g_rope_status;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Passes of a warp's lanes over the rows of an item, and stages of a warp's ring: four KB a warp
// are on their way, 96 or 80 KB on an SM.
constexpr int kPasses = 4, kForwardStages = 3, kBackwardStages = 2;
constexpr int kForwardStage = 512 * kPasses + kAngleBytes;
constexpr int kBackwardStage = 2 * 512 * kPasses + kAngleBytes;  // dy's rows, x's, angles
// Blocks: as many as the registers allow to be resident, six or five on an SM.
constexpr int kMaxSms = 160;  // partial sums are reserved for this many
constexpr int kForwardPerSm = 6, kBackwardPerSm = 5;

// One of the two tensors, Q or K.
struct Side {
  const __nv_bfloat16 *x, *dy, *w;
  __nv_bfloat16* y;  // y, or dx
  long long ldx, lddy, ldy;
  int heads;
  Deal deal;
};

struct RopeParams {
  Side q, k;
  RopeHow how;
  const int* positions;
  float* partial;  // backward: [blocks][d], Q's blocks first
};

// The position of a row, as it stands in `positions`; 0 where nothing is turned.
FA_DEV int position_of(const RopeParams& p, int t) { return p.how.rot ? p.positions[t] : 0; }
// Whether the table has it (else it is reported).
FA_DEV bool position_ok(const RopeParams& p, int pos, int lane) {
  if (p.how.rot == 0 || (unsigned)pos < (unsigned)p.how.positions) return true;
  if (lane == 0) atomicOr(&g_rope_status, kDeviceIndexBit);
  return false;
}
FA_DEV void load_angles(const RopeParams& p, uint32_t to, int pos, int lane) {
  if (p.how.rot && (unsigned)pos < (unsigned)p.how.positions)
    copy_async<1>(to, p.how.cos_sin + (size_t)pos * p.how.rot, 4 * p.how.rot, lane);
}

// An item is kPasses * 32 / W heads of one row; the first blocks take Q's, the others K's.
// Positions are read an item before the angles that they choose are copied. The stream's next
// kernel may start once all rows are on their way: earlier, its blocks take SMs from this one's
// (training 16384 rows, 32/8 heads, d = 128: 236 us against 145), at the end it comes 4 us later.
template <int W, bool INTER>
__global__ void __launch_bounds__(kThreads, kForwardPerSm)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int R = 32 / W, U = kPasses, S = kForwardStages;
  __shared__ __align__(16) uint8_t rings[kWarps * S * kForwardStage];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, l = lane % W, seg = lane / W;
  const bool is_q = (int)blockIdx.x < p.q.deal.blocks;
  const Side& s = is_q ? p.q : p.k;
  const int d = p.how.d, heads = s.heads;
  const Piece mine =
      piece_of(s.deal, ((int)blockIdx.x - (is_q ? 0 : p.q.deal.blocks)) * kWarps + warp);
  const uint32_t ring = smem_u32(rings) + warp * S * kForwardStage, row = 2 * d;
  const RopeLane at = rope_lane(p.how, l, true);
  grid_wait();
  if (mine.items > 0) {
    Item in = mine.first;
    int put = 0;                  // items whose copies are issued
    int pos[S];                   // of the items from the one worked on
    int ahead = position_of(p, in.token);
    uint32_t to = ring;
    auto issue = [&]() {
      pos[S - 1] = ahead;
      if (put < mine.items) {
        const int h = in.chunk * U * R;
        copy_async<U>(to, s.x + (long long)in.token * s.ldx + h * d, min(U * R, heads - h) * 2 * d,
                      lane);
        load_angles(p, to + 512 * U, ahead, lane);
        in.advance(s.deal);
        if (++put < mine.items)
          ahead = position_of(p, in.token);
        else
          grid_launch_dependents();
      }
      cp_async_commit();
      to = to == ring + (S - 1) * kForwardStage ? ring : to + kForwardStage;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
#pragma unroll
      for (int k = 0; k + 1 < S; ++k) pos[k] = pos[k + 1];
      issue();
    }
    const bool norm = s.w != nullptr;
    const Pairs w = load_weight<INTER>(s.w, at);
    Item it = mine.first;
    uint32_t stage = ring;
    for (int i = 0; i < mine.items; ++i, it.advance(s.deal)) {
      cp_async_wait<S - 2>();
      __syncwarp();  // the stage has landed for every lane, and the last one is read
#pragma unroll
      for (int k = 0; k + 1 < S; ++k) pos[k] = pos[k + 1];
      issue();
      if (position_ok(p, pos[0], lane)) {
        const uint32_t rows = stage + seg * row;
        const Turn turn = rope_turn(rope_angles(stage + 512 * U, p.how, at, l), w);
        const int h0 = it.chunk * U * R + seg;
        __nv_bfloat16* const out = s.y + (long long)it.token * s.ldy + h0 * d;
#pragma unroll
        for (int u = 0; u < U; u += 2) {
          if (h0 - seg + u * R >= heads) break;  // warp-uniform
          Pairs y[2];
          norm_and_turn<W, INTER, 2>(y, rows + u * R * row, R * row, turn, norm, p.how, at);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (h0 + (u + k) * R < heads && at.in)
              store_row<INTER>(out + (u + k) * R * d, y[k], at);
        }
      }
      stage = stage == ring + (S - 1) * kForwardStage ? ring : stage + kForwardStage;
    }
  }
}

// The same division of the work: a lane sums its channels' part of dw over all its rows, a block
// over its lanes, in a fixed order, and reduce_kernel over the blocks.
template <int W, bool INTER>
__global__ void __launch_bounds__(kThreads, kBackwardPerSm)
    rope_backward_kernel(const __grid_constant__ RopeParams p) {
  constexpr int R = 32 / W, U = kPasses;
  static_assert(kBackwardStages == 2, "one stage is worked on, one is on its way");
  __shared__ __align__(16) uint8_t rings[kWarps * 2 * kBackwardStage];
  __shared__ float sums[kWarps][8 * W];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, l = lane % W, seg = lane / W;
  const bool is_q = (int)blockIdx.x < p.q.deal.blocks;
  const Side& s = is_q ? p.q : p.k;
  const int d = p.how.d, heads = s.heads;
  const Piece mine =
      piece_of(s.deal, ((int)blockIdx.x - (is_q ? 0 : p.q.deal.blocks)) * kWarps + warp);
  const uint32_t ring = smem_u32(rings) + warp * 2 * kBackwardStage, row = 2 * d;
  const RopeLane at = rope_lane(p.how, l, true);
  const bool norm = s.w != nullptr;
  grid_wait();
  const Pairs w = load_weight<INTER>(s.w, at);
  Pairs dw = {{0, 0}, {0, 0}};
  if (mine.items > 0) {
    Item in = mine.first;
    int put = 0;  // items whose copies are issued
    int ahead = position_of(p, in.token), next = 0;
    uint32_t stage = ring, other = ring + kBackwardStage;
    auto issue = [&](uint32_t to) {
      next = ahead;
      if (put < mine.items) {
        const int h = in.chunk * U * R, bytes = min(U * R, heads - h) * 2 * d;
        copy_async<U>(to, s.dy + (long long)in.token * s.lddy + h * d, bytes, lane);
        if (norm)
          copy_async<U>(to + 512 * U, s.x + (long long)in.token * s.ldx + h * d, bytes, lane);
        load_angles(p, to + 1024 * U, ahead, lane);
        in.advance(s.deal);
        if (++put < mine.items)
          ahead = position_of(p, in.token);
        else
          grid_launch_dependents();
      }
      cp_async_commit();
    };
    issue(stage);
    Item it = mine.first;
    for (int i = 0; i < mine.items; ++i, it.advance(s.deal)) {
      const int pos = next;
      cp_async_wait<0>();
      __syncwarp();  // the stage has landed for every lane, and the other one is read
      issue(other);
      if (position_ok(p, pos, lane)) {
        const uint32_t rows = stage + seg * row;
        const Angles g = rope_angles(stage + 1024 * U, p.how, at, l);
        const int h0 = it.chunk * U * R + seg;
        __nv_bfloat16* const out = s.y + (long long)it.token * s.ldy + h0 * d;
#pragma unroll
        for (int u0 = 0; u0 < U; u0 += 2) {
          if (h0 - seg + u0 * R >= heads) break;  // warp-uniform
          Pairs y[2], x[2];
          float sum[4];  // of x^2, then of g o w o x
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t from = rows + (u0 + k) * R * row;
            y[k] = turned_back(row_of<INTER>(from, at), g, at.turns);
            if (norm) {
              x[k] = row_of<INTER>(from + 512 * U, at);
              sum[k] = dot(x[k], x[k]);
              sum[2 + k] = dot(times(y[k], w), x[k]);
            }
          }
          if (norm) {
            row_sums<W, 4>(sum);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float r = inverse_root(sum[k] * p.how.inv_d + p.how.eps);
              const Pairs n = times(x[k], both(r));
              if (h0 + (u0 + k) * R < heads) dw = plus(y[k], n, dw);  // else it is anything
              y[k] = plus(times(y[k], w), {{both(r), both(r)}, {both(r), both(r)}},
                          times(n, both(-sum[2 + k] * r * r * p.how.inv_d)));
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (h0 + (u0 + k) * R < heads && at.in)
              store_row<INTER>(out + (u0 + k) * R * d, y[k], at);
        }
      }
      const uint32_t swap = stage;
      stage = other;
      other = swap;
    }
  }
  if (!norm) return;
  float mine_dw[8];
  channels<INTER>(dw, mine_dw);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = W; o < 32; o <<= 1) mine_dw[i] += __shfl_xor_sync(0xffffffffu, mine_dw[i], o);
  if (lane < W && at.in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sums[warp][at.a + i] = mine_dw[i];
      sums[warp][at.b + i] = mine_dw[4 + i];
    }
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < d) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i][c];
    p.partial[(size_t)blockIdx.x * d + c] = v;
  }
}

struct ReduceParams {
  const float* partial;
  float *dwq, *dwk;
  int d, q_rows, k_rows;  // partial rows of Q, then of K
};
// A block adds up 32 channels of one of the two.
__global__ void __launch_bounds__(1024) reduce_kernel(const __grid_constant__ ReduceParams p) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const bool is_q = blockIdx.y == 0;
  float* const out = is_q ? p.dwq : p.dwk;
  const int rows = is_q ? p.q_rows : p.k_rows, c = (int)blockIdx.x * 32 + lane;
  const float* from = p.partial + (is_q ? 0 : (size_t)p.q_rows * p.d);
  grid_wait();
  grid_launch_dependents();
  if (!out) return;
  float v = 0.f;
  if (c < p.d) {
#pragma unroll 16
    for (int r = row; r < rows; r += 32) v += from[(size_t)r * p.d + c];
  }
  sums[row][lane] = v;
  __syncthreads();
  v = sums[lane][row];  // this warp's channel: a lane per row
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int mine = (int)blockIdx.x * 32 + row;
  if (lane == 0 && mine < p.d) out[mine] = v;
}

Side side(const void* x, const void* dy, const void* w, void* y, long long ldx, long long lddy,
          long long ldy, int heads) {
  Side s;
  s.x = static_cast<const __nv_bfloat16*>(x);
  s.dy = static_cast<const __nv_bfloat16*>(dy);
  s.w = static_cast<const __nv_bfloat16*>(w);
  s.y = static_cast<__nv_bfloat16*>(y);
  s.ldx = ldx;
  s.lddy = lddy;
  s.ldy = ldy;
  s.heads = heads;
  return s;
}

// Deals both sides' items; returns the blocks of both.
int deal_sides(RopeParams& p, int total, int d, int per_sm) {
  const int sms = sm_count(), per = kPasses * (32 / rope_lanes(d));
  const int cq = ceil_div(p.q.heads, per), ck = ceil_div(p.k.heads, per);
  int blocks[2];
  share_blocks<2>(blocks, {(long long)total * cq, (long long)total * ck},
                  (sms < kMaxSms ? sms : kMaxSms) * per_sm, kWarps);
  p.q.deal = deal(total, cq, blocks[0], kWarps);
  p.k.deal = deal(total, ck, blocks[1], kWarps);
  return blocks[0] + blocks[1];
}

struct Forward {
  const RopeParams& p;
  int blocks;
  cudaStream_t stream;
  template <int W, bool INTER>
  cudaError_t run() const {
    return launch_early(rope_kernel<W, INTER>, dim3((unsigned)blocks), kThreads, 0, stream, p);
  }
};
struct Backward {
  const RopeParams& p;
  int blocks;
  cudaStream_t stream;
  template <int W, bool INTER>
  cudaError_t run() const {
    return launch_early(rope_backward_kernel<W, INTER>, dim3((unsigned)blocks), kThreads, 0,
                        stream, p);
  }
};

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p{};
  p.q = side(a.Q, nullptr, a.how.q_weight, a.Qo, a.ldq, 0, a.ldqo, a.Hq);
  p.k = side(a.K, nullptr, a.how.k_weight, a.Ko, a.ldk, 0, a.ldko, a.Hkv);
  p.how = rope_how(a.how, a.d);
  p.positions = a.positions;
  const int blocks = deal_sides(p, a.total, a.d, kForwardPerSm);
  return with_lanes(p.how, Forward{p, blocks, s});
}

size_t rope_workspace_bytes(int d) {
  return (size_t)(kMaxSms * kBackwardPerSm + 2) * d * sizeof(float);
}

cudaError_t launch_rope_backward(const RopeBackwardArgs& a, cudaStream_t s) {
  RopeParams p{};
  p.q = side(a.Q, a.dQo, a.how.q_weight, a.dQ, a.ldq, a.lddqo, a.lddq, a.Hq);
  p.k = side(a.K, a.dKo, a.how.k_weight, a.dK, a.ldk, a.lddko, a.lddk, a.Hkv);
  p.how = rope_how(a.how, a.d);
  p.positions = a.positions;
  p.partial = a.partial;
  const int blocks = deal_sides(p, a.total, a.d, kBackwardPerSm);
  cudaError_t e = with_lanes(p.how, Backward{p, blocks, s});
  if (e != cudaSuccess || (!a.how.q_weight && !a.how.k_weight)) return e;
  ReduceParams r;
  r.partial = a.partial;
  r.dwq = a.how.q_weight ? a.dwq : nullptr;
  r.dwk = a.how.k_weight ? a.dwk : nullptr;
  r.d = a.d;
  r.q_rows = p.q.deal.blocks;
  r.k_rows = p.k.deal.blocks;
  return launch_early(reduce_kernel, dim3((unsigned)ceil_div(a.d, 32), 2), 1024, 0, s, r);
}

cudaError_t rope_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
