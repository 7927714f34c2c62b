// The feed-forward block for at most eight tokens (a decoded token, a handful of
// streams): two matrix-vector-like products that do nothing but stream the weights.
//
// Bound by reading the weights from HBM once.  No shared memory on their way: with
// m16n8k16 the weight's rows are M and the tokens N, and because the order of K is
// free as long as both operands agree, a lane takes 8 consecutive K-elements (16
// bytes) of its row for two MMA steps.  A warp's load then covers 64 contiguous bytes
// of 8 rows, the warps of a block take consecutive pieces of the same 16 rows, and
// each lane keeps kDepth steps (2 x 16 bytes each) in flight.  The partial sums of the
// warps meet in shared memory, in warp order.  One block per 8 ffn columns (8 rows of
// Wg and the same 8 of Wu fill the 16) or per 16 output columns, so the blocks are
// small and spread evenly; against tiles of 256 rows (pair_gemm.cu) nothing has to be
// split along K and joined by another launch.
// Measured for one token, 4096/14336: 38 us for 235 MB of Wg and Wu (6.2 TB/s, 0.92 of
// the copy rate), 19 us for 117 MB of Wd.  Many blocks with two steps in flight beat
// fewer with four or eight for the first (38 against 43 and 40 us); the second, with few
// blocks, wants 16 warps of four (19 against 23 with eight, 20 with eight warps).
#include "dmuon.h"
#include "act.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "train.h"

namespace dm {
namespace {

DM_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool GLU, int WARPS, int kDepth>
__global__ void __launch_bounds__(WARPS * 32) thin_kernel(const ThinArgs g) {
  __shared__ float red[WARPS][16][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = lane >> 2;            // MMA rows `row` and `row` + 8, and the token
  const int quad = (lane & 3) * 8;      // this lane's K-elements within a step of 32
  // kGlu: rows of gate, then the same rows of up; else 16 rows of the weight.  Rows
  // past the end repeat the last one; their sums are not written.
  const long long first = (long long)blockIdx.x * (GLU ? 8 : 16);
  const long long r0 = min(first + row, g.cols - 1ll);
  const long long r1 = GLU ? r0 : min(first + 8 + row, g.cols - 1ll);
  const __nv_bfloat16* wa = g.w0 + r0 * g.w_ld + quad;
  const __nv_bfloat16* wb = (GLU ? g.w1 : g.w0) + r1 * g.w_ld + quad;
  const __nv_bfloat16* x = g.x + (long long)row * g.x_ld + quad;
  const bool token = row < g.tokens;
  const int steps = (g.k + 31) / 32;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // the first launch of a call must see what came before it; the second's weights
  // were complete by then (the first lets it start only after its own wait), so their
  // loads need not wait for the first's results
  if (GLU) {
    grid_wait();
    grid_launch_dependents();
  }
  float c[4] = {0.f, 0.f, 0.f, 0.f};
  bool waited = GLU;
  for (int s0 = warp; s0 < steps; s0 += kDepth * WARPS) {
    uint4 a[kDepth], b[kDepth], t[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int k = (s0 + d * WARPS) * 32;
      const bool in = k + quad < g.k;  // k is a multiple of 8: a lane's piece is in or out
      a[d] = in ? __ldcs(reinterpret_cast<const uint4*>(wa + k)) : zero;
      b[d] = in ? __ldcs(reinterpret_cast<const uint4*>(wb + k)) : zero;
    }
    if (!waited) {
      grid_wait();
      waited = true;
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int k = (s0 + d * WARPS) * 32;
      t[d] = token && k + quad < g.k ? *reinterpret_cast<const uint4*>(x + k) : zero;
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      mma16816(c, a[d].x, b[d].x, a[d].y, b[d].y, t[d].x, t[d].y);
      mma16816(c, a[d].z, b[d].z, a[d].w, b[d].w, t[d].z, t[d].w);
    }
  }
  if (!waited) grid_wait();
  const int n = (lane & 3) * 2;  // tokens of this lane's sums
  red[warp][row][n] = c[0];
  red[warp][row][n + 1] = c[1];
  red[warp][row + 8][n] = c[2];
  red[warp][row + 8][n + 1] = c[3];
  __syncthreads();
  constexpr int kOut = GLU ? 8 : 16;  // columns this block writes
  const int i = threadIdx.x % kOut, tok = threadIdx.x / kOut;
  const long long col = first + i;
  if (tok >= g.tokens || tok >= 8 || col >= g.cols) return;
  float v = 0.f, u = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    v += red[w][i][tok];
    if (GLU) u += red[w][i + 8][tok];
  }
  if (GLU) {
    if (g.gate != nullptr) {
      g.gate[tok * g.cols + col] = __float2bfloat16_rn(v);
      g.up[tok * g.cols + col] = __float2bfloat16_rn(u);
    }
    v = (g.act == DMUON_ACT_SILU   ? act_value<DMUON_ACT_SILU>(v)
         : g.act == DMUON_ACT_GELU ? act_value<DMUON_ACT_GELU>(v)
                                   : act_value<DMUON_ACT_GELU_TANH>(v)) *
        u;
  }
  g.out[tok * g.out_ld + col] = __float2bfloat16_rn(v);
}

}  // namespace

cudaError_t launch_thin(const ThinArgs& g, bool glu, cudaStream_t s) {
  if (glu)
    return launch_dependent(thin_kernel<true, 8, 2>, unsigned((g.cols + 7) / 8), 256u, s, g);
  return launch_dependent(thin_kernel<false, 16, 4>, unsigned((g.cols + 15) / 16), 512u, s, g);
}

}  // namespace dm
