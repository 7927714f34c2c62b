// One token of linear attention for each of many streams:
//   S <- a S + k v^T,   out = scale q S
// Bound by reading and writing the fp32 states (8 bytes an element) once: 0.2 products a
// byte.  A column of S meets only its own element of v and out, so the columns are cut into
// pieces of 32 (128 bytes of a row), a block takes the key_dim rows of one piece, all its
// loads in flight at once, and no block waits for another.  8 lanes hold a row, 16 rows at a
// time; the 16 sums of a column meet by shuffles and through shared memory, in that order.
// Measured, 250 streams of 32 heads of 128 x 128: 155 us a pass, 6.8 TB/s, the copy rate; one stream 3.8 us,
// a launch's latency.
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

constexpr int kThreads = 128, kCols = 32, kRowsAtOnce = kThreads / 8;
constexpr int kPasses = 128 / kRowsAtOnce;

__global__ void __launch_bounds__(kThreads) linattn_step_kernel(const __grid_constant__ LinStepArgs g,
                                                                int pieces) {
  __shared__ float sq[128], sk[128], part[kThreads / 32][kCols], decay[2];
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int b = blockIdx.x;
  const int piece = b % pieces;
  b /= pieces;
  const int head = b % g.heads, row = b / g.heads;
  const long long slot = g.slot != nullptr ? (long long)g.slot[row] : row;
  if (slot < 0 || slot >= g.slots) return;
  if (g.slot != nullptr) {
    // the first row of a slot takes all of them
    int before = 0;
    for (int r = tid; r < row; r += kThreads) before |= g.slot[r] == slot;
    if (__syncthreads_or(before)) return;
  }
  const int c0 = piece * kCols + (lane & 7) * 4, r0 = tid >> 3;
  const bool in = c0 < g.dv;
  const float log_decay = g.log_decay[head];
  const long long at = ((slot * g.heads + head) * g.dk + r0) * g.dv + c0;
  const long long step = (long long)kRowsAtOnce * g.dv;
  float4 st[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
    st[p] = in && r0 + p * kRowsAtOnce < g.dk
                ? __ldcs(reinterpret_cast<const float4*>(g.state + at + p * step))
                : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = row; r < g.rows;) {
    if (tid < g.dk) {
      sq[tid] = __bfloat162float(g.q.p[r * g.q.ts + head * g.q.hs + tid]);
      sk[tid] = __bfloat162float(g.k.p[r * g.k.ts + head * g.k.hs + tid]);
    }
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
      const __nv_bfloat16* vp = g.v.p + r * g.v.ts + head * g.v.hs + c0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __bfloat162float(vp[i]);
    }
    // a and, of a slow head, what its rounding drops: over thousands of steps an error with one sign
    // would add up (8000 of log_decay -1e-6: 3e-4 of the state).  a rounded down, so that the rest of
    // an infinity has its sign.  By one thread, with all loads on their way: 250 streams 155 us, 164
    // to 177 by each.
    if (tid == kThreads - 1) {
      const float e = expm1f(log_decay);
      float a = expf(log_decay), rest = 0.f;
      if (log_decay <= 0.f && e > -0.4375f) {
        a = 1.f + e;
        rest = e - (a - 1.f);  // exact
        if (rest < 0.f) {
          a -= 0x1p-24f;
          rest += 0x1p-24f;
        }
      }
      decay[0] = a;
      decay[1] = rest;
    }
    __syncthreads();
    // k v is exact; what is left of a joins it, as a state that decays by less than its last bit
    // would else stay as it is
    const float a = decay[0], rest = decay[1];
    auto stepped = [&](float x, float kv) { return fmaf(a, x, rest > 0.f ? fmaf(rest, x, kv) : kv); };
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = r0 + p * kRowsAtOnce;
      if (i < g.dk) {
        const float k = sk[i], q = sq[i];
        st[p].x = stepped(st[p].x, k * v[0]);
        st[p].y = stepped(st[p].y, k * v[1]);
        st[p].z = stepped(st[p].z, k * v[2]);
        st[p].w = stepped(st[p].w, k * v[3]);
        o[0] = fmaf(q, st[p].x, o[0]);
        o[1] = fmaf(q, st[p].y, o[1]);
        o[2] = fmaf(q, st[p].z, o[2]);
        o[3] = fmaf(q, st[p].w, o[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], 8);
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], 16);
    }
    if (lane < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][lane * 4 + i] = o[i];
    }
    __syncthreads();
    if (tid < kCols && piece * kCols + tid < g.dv) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) sum += part[w][tid];
      g.out.p[r * g.out.ts + head * g.out.hs + piece * kCols + tid] =
          __float2bfloat16_rn(g.scale * sum);
    }
    if (g.slot == nullptr) break;
    int next = g.rows;
    for (int n = r + 1 + tid; n < g.rows && next == g.rows; n += kThreads)
      if (g.slot[n] == slot) next = n;
    next = __reduce_min_sync(0xffffffffu, next);
    __shared__ int nexts[kThreads / 32];
    if (lane == 0) nexts[warp] = next;
    __syncthreads();
    r = min(min(nexts[0], nexts[1]), min(nexts[2], nexts[3]));
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
    if (in && r0 + p * kRowsAtOnce < g.dk)
      __stcs(reinterpret_cast<float4*>(g.new_state + at + p * step), st[p]);
}

}  // namespace

cudaError_t launch_linattn_step(const LinStepArgs& g, cudaStream_t s) {
  const int pieces = (g.dv + kCols - 1) / kCols;
  return launch_dependent(linattn_step_kernel, unsigned((long long)g.rows * g.heads * pieces),
                          unsigned(kThreads), s, g, pieces);
}

}  // namespace dm
