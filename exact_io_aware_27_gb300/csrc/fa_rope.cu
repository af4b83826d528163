// Norms of queries and keys for each head with the position rotation in the same pass, and
// their gradients.
//
//   forward   n = x r, r = (mean x^2 + eps)^-1/2;  u = n o w;  y = R u
//             R turns pairs of channels: (a, b) -> (a c - b s, b c + a s)
//   backward  g = R^T dy;  dw = sum over rows of g o n
//             dx = r (g o w - n mean(g o w o n))
//
// Bound by memory: a row is read once and written once (forward), or dy and x read and dx
// written (backward), and everything between stays in registers (fa_rope.cuh).
#include "fa_launch.h"
#include "fa_rope.cuh"

namespace fa {

__device__ unsigned int g_rope_status;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // rows of a lane in flight

// One of the two tensors, Q or K.
struct Side {
  const __nv_bfloat16 *x, *dy, *w;
  __nv_bfloat16* y;       // y, or dx
  long long ldx, lddy, ldy;
  int heads, chunks;      // chunks of kUnroll * 32 / W heads
};

struct RopeParams {
  Side q, k;
  RopeHow how;
  const int* positions;
  int total;
  float* partial;  // backward: [2][blocks][d]
};

// The position of row t, or -1 (reported) where the table has none.
FA_DEV int position_of(const RopeParams& p, int t) {
  if (p.how.rot == 0) return 0;
  const int pos = p.positions[t];
  if ((unsigned)pos < (unsigned)p.how.positions) return pos;
  atomicOr(&g_rope_status, kDeviceIndexBit);
  return -1;
}

// A warp takes kUnroll * 32 / W heads of one row t; blockIdx.y counts Q's chunks of heads, then
// K's.
template <int W>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int R = 32 / W;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % W;
  const bool is_q = (int)blockIdx.y < p.q.chunks;
  const Side& s = is_q ? p.q : p.k;
  const int h0 = ((int)blockIdx.y - (is_q ? 0 : p.q.chunks)) * kUnroll * R + lane / W;
  const RopeLane at = rope_lane(p.how, l, true);
  grid_wait();
  grid_launch_dependents();
  float w[8];
  load_weight(w, s.w, at);
  for (int t = (int)blockIdx.x * kWarps + warp; t < p.total; t += (int)gridDim.x * kWarps) {
    const int pos = position_of(p, t);
    uint2 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      a[u] = b[u] = make_uint2(0, 0);
      const int h = h0 + u * R;
      if (h < s.heads && at.in) {
        const __nv_bfloat16* row = s.x + (long long)t * s.ldx + h * p.how.d;
        a[u] = ld_stream8(row + at.a);
        b[u] = ld_stream8(row + at.b);
      }
    }
    if (pos < 0) continue;
    const Angles g = rope_angles(p.how, at, l, pos);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * R;
      if (h - lane / W >= s.heads) break;  // warp-uniform
      float x[8];
      unpack8(x, a[u], b[u]);
      if (s.w) norm8<W>(x, w, p.how);
      turn8(x, p.how, at, g, 1.f);
      if (h < s.heads && at.in) {
        __nv_bfloat16* row = s.y + (long long)t * s.ldy + h * p.how.d;
        *reinterpret_cast<uint2*>(row + at.a) = pack4(x);
        *reinterpret_cast<uint2*>(row + at.b) = pack4(x + 4);
      }
    }
  }
}

// The same division of the work, by persistent blocks: a lane sums its channels' part of dw over
// all its rows, a block over its lanes, in a fixed order, and reduce_kernel over the blocks.
template <int W>
__global__ void __launch_bounds__(kThreads)
    rope_backward_kernel(const __grid_constant__ RopeParams p) {
  constexpr int R = 32 / W;
  __shared__ float sums[kWarps][8 * W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % W;
  const bool is_q = (int)blockIdx.y < p.q.chunks;
  const Side& s = is_q ? p.q : p.k;
  const int h0 = ((int)blockIdx.y - (is_q ? 0 : p.q.chunks)) * kUnroll * R + lane / W;
  const RopeLane at = rope_lane(p.how, l, true);
  grid_wait();
  grid_launch_dependents();
  float w[8], dw[8];
  load_weight(w, s.w, at);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  for (int t = (int)blockIdx.x * kWarps + warp; t < p.total; t += (int)gridDim.x * kWarps) {
    const int pos = position_of(p, t);
    uint2 a[kUnroll], b[kUnroll], xa[kUnroll], xb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      a[u] = b[u] = xa[u] = xb[u] = make_uint2(0, 0);
      const int h = h0 + u * R;
      if (h < s.heads && at.in) {
        const __nv_bfloat16* row = s.dy + (long long)t * s.lddy + h * p.how.d;
        a[u] = ld_stream8(row + at.a);
        b[u] = ld_stream8(row + at.b);
        if (s.w) {
          row = s.x + (long long)t * s.ldx + h * p.how.d;
          xa[u] = ld_stream8(row + at.a);
          xb[u] = ld_stream8(row + at.b);
        }
      }
    }
    if (pos < 0) continue;
    const Angles g = rope_angles(p.how, at, l, pos);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * R;
      if (h - lane / W >= s.heads) break;  // warp-uniform
      float y[8];
      unpack8(y, a[u], b[u]);
      turn8(y, p.how, at, g, -1.f);
      if (s.w) {
        float x[8];
        unpack8(x, xa[u], xb[u]);
        float xx = 0.f, dot = 0.f;  // sums of x^2 and of g o w o x
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xx += x[i] * x[i];
          dot += y[i] * w[i] * x[i];
        }
        xx = row_sum<W>(xx);
        dot = row_sum<W>(dot);
        const float r = rsqrtf(xx * p.how.inv_d + p.how.eps);
        const float back = dot * r * r * p.how.inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[i] += y[i] * (x[i] * r);
          y[i] = r * (y[i] * w[i] - x[i] * back);
        }
      }
      if (h < s.heads && at.in) {
        __nv_bfloat16* row = s.y + (long long)t * s.ldy + h * p.how.d;
        *reinterpret_cast<uint2*>(row + at.a) = pack4(y);
        *reinterpret_cast<uint2*>(row + at.b) = pack4(y + 4);
      }
    }
  }
  if (!s.w) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = W; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
  if (lane < W && at.in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sums[warp][at.a + i] = dw[i];
      sums[warp][at.b + i] = dw[4 + i];
    }
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < p.how.d) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i][c];
    p.partial[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * p.how.d + c] = v;
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
#pragma unroll 4
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

int chunks_of(int heads, int d) { return ceil_div(heads, kUnroll * (32 / rope_lanes(d))); }

Side side(const void* x, const void* dy, const void* w, void* y, long long ldx, long long lddy,
          long long ldy, int heads, int d) {
  Side s;
  s.x = static_cast<const __nv_bfloat16*>(x);
  s.dy = static_cast<const __nv_bfloat16*>(dy);
  s.w = static_cast<const __nv_bfloat16*>(w);
  s.y = static_cast<__nv_bfloat16*>(y);
  s.ldx = ldx;
  s.lddy = lddy;
  s.ldy = ldy;
  s.heads = heads;
  s.chunks = chunks_of(heads, d);
  return s;
}

// Blocks per chunk of the backward kernel: six on each SM in all, so that every warp has rows
// in flight while its neighbours reduce.
constexpr int kBackwardBlocks = 6 * 152;
int backward_blocks(int Hq, int Hkv, int d) {
  const int n = chunks_of(Hq, d) + chunks_of(Hkv, d);
  return n < kBackwardBlocks ? kBackwardBlocks / n : 1;
}

struct Forward {
  const RopeParams& p;
  cudaStream_t stream;
  template <int W>
  cudaError_t run() const {
    const int blocks = ceil_div(p.total, kWarps);
    return launch_early(rope_kernel<W>, dim3((unsigned)blocks, (unsigned)(p.q.chunks + p.k.chunks)),
                        kThreads, 0, stream, p);
  }
};
struct Backward {
  const RopeParams& p;
  int blocks;
  cudaStream_t stream;
  template <int W>
  cudaError_t run() const {
    return launch_early(rope_backward_kernel<W>,
                        dim3((unsigned)blocks, (unsigned)(p.q.chunks + p.k.chunks)), kThreads, 0,
                        stream, p);
  }
};

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p{};
  p.q = side(a.Q, nullptr, a.how.q_weight, a.Qo, a.ldq, 0, a.ldqo, a.Hq, a.d);
  p.k = side(a.K, nullptr, a.how.k_weight, a.Ko, a.ldk, 0, a.ldko, a.Hkv, a.d);
  p.how = rope_how(a.how, a.d);
  p.positions = a.positions;
  p.total = a.total;
  return with_lanes(a.d, Forward{p, s});
}

size_t rope_workspace_bytes(int Hq, int Hkv, int d) {
  const size_t n = (size_t)chunks_of(Hq, d) + chunks_of(Hkv, d);
  return n * backward_blocks(Hq, Hkv, d) * d * sizeof(float);
}

cudaError_t launch_rope_backward(const RopeBackwardArgs& a, cudaStream_t s) {
  RopeParams p{};
  p.q = side(a.Q, a.dQo, a.how.q_weight, a.dQ, a.ldq, a.lddqo, a.lddq, a.Hq, a.d);
  p.k = side(a.K, a.dKo, a.how.k_weight, a.dK, a.ldk, a.lddko, a.lddk, a.Hkv, a.d);
  p.how = rope_how(a.how, a.d);
  p.positions = a.positions;
  p.total = a.total;
  p.partial = a.partial;
  const int most = backward_blocks(a.Hq, a.Hkv, a.d), need = ceil_div(a.total, kWarps);
  const int blocks = need < most ? need : most;
  cudaError_t e = with_lanes(a.d, Backward{p, blocks, s});
  if (e != cudaSuccess || (!a.how.q_weight && !a.how.k_weight)) return e;
  ReduceParams r;
  r.partial = a.partial;
  r.dwq = a.how.q_weight ? a.dwq : nullptr;
  r.dwk = a.how.k_weight ? a.dwk : nullptr;
  r.d = a.d;
  r.q_rows = p.q.chunks * blocks;
  r.k_rows = p.k.chunks * blocks;
  return launch_early(reduce_kernel, dim3((unsigned)ceil_div(a.d, 32), 2), 1024, 0, s, r);
}

cudaError_t rope_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
