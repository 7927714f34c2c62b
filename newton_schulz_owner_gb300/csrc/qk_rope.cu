// Root-mean-square norm of every query and key head, its gains, and the rotation by
// position, forward and backward, in one pass over the heads.
//
// Bound by HBM: 4 bytes an element forward (read and write bf16), 6 backward.  A head is
// spread over LANES lanes of a warp, 8 elements each, as two runs of four: in the split form
// the runs are elements 4l .. 4l + 3 of each half of the rotated part, so that a lane holds
// both sides of its pairs and nothing but the sums of squares crosses lanes; in the
// interleaved form, and past the rotated part, they are neighbours.
//
// Angles.  t = position * inv_freq radians is needed modulo a turn only, and in fp32 a
// position of 10^5 would leave a third of the digits.  f / 2 pi as a 64-bit fraction of a turn
// times the position, modulo 2^64, is exact but for the fraction's rounding (2^-53 of it): the
// top 32 bits are the angle.  A lane forms its four fractions once and keeps them over all its
// tokens; a token's four sines and cosines serve all heads that the lane takes of it.
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

template <bool VEC>
DM_DEV void load4(const __nv_bfloat16* p, float (&v)[4]) {
  if (VEC) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __bfloat162float(p[i]);
  }
}
template <bool VEC>
DM_DEV void store4(__nv_bfloat16* p, const float (&v)[4]) {
  if (VEC) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}

// The lane's share of a head.
struct Share {
  int a, b;      // first elements of its two runs
  bool in;       // it has elements
  bool turned;   // they are rotated
};
template <bool ILV>
DM_DEV Share share_of(int l, int dim, int rotary) {
  Share s;
  s.in = 8 * l < dim;
  s.turned = 8 * l < rotary;
  if (!ILV && s.turned) {
    s.a = 4 * l;
    s.b = rotary / 2 + 4 * l;
  } else {
    s.a = 8 * l;
    s.b = 8 * l + 4;
  }
  return s;
}

// The four angles of a lane as fractions of a turn per position, in 2^-64.
struct Turns {
  unsigned long long f[4];
  float bad[4];  // 0, or NaN for a frequency that is not finite
};
DM_DEV Turns turns_of(const float* inv_freq, int l, bool turned) {
  Turns t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    double f = turned ? double(inv_freq[4 * l + i]) * 0.15915494309189533577 : 0.0;
    f -= floor(f);
    t.bad[i] = float(f - f);
    t.f[i] = static_cast<unsigned long long>(f * 18446744073709551616.0);
  }
  return t;
}
DM_DEV void angles(const Turns& t, int position, float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long at = t.f[i] * static_cast<unsigned long long>((long long)position);
    const float half_turns = float(int(at >> 32)) * 4.656612873077393e-10f + t.bad[i];
    sincospif(half_turns, &s[i], &c[i]);
  }
}

// (a, b) of a lane turned by its angles (back: by minus them).
template <bool ILV, bool BACK>
DM_DEV void turn(float (&a)[4], float (&b)[4], const float (&c)[4], const float (&s0)[4]) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = BACK ? -s0[i] : s0[i];
  if (ILV) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * c[i] - y * s[i];
      a[2 * i + 1] = x * s[i] + y * c[i];
      const float u = b[2 * i], v = b[2 * i + 1];
      b[2 * i] = u * c[2 + i] - v * s[2 + i];
      b[2 * i + 1] = u * s[2 + i] + v * c[2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * c[i] - y * s[i];
      b[i] = x * s[i] + y * c[i];
    }
  }
}

template <int LANES>
DM_DEV float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

DM_DEV float square_sum(const float (&a)[4], const float (&b)[4]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
  return s;
}

template <int LANES, bool ILV, bool VEC, bool BACK>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs g) {
  constexpr int kGroups = 32 / LANES;  // heads that a warp takes at once
  constexpr int kDepth = BACK ? 2 : 4;  // and how many times it loads before it computes
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
  const Share sh = share_of<ILV>(l, g.dim, g.rotary);
  const Turns turns = turns_of(g.inv_freq, l, sh.turned);
  const float inv_dim = 1.f / float(g.dim);
  float wa[2][4], wb[2][4], da[2][4], db[2][4];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool has = g.w[x] != nullptr && sh.in && g.heads[x] > 0;
      wa[x][i] = has ? __bfloat162float(g.w[x][sh.a + i]) : 1.f;
      wb[x][i] = has ? __bfloat162float(g.w[x][sh.b + i]) : 1.f;
      da[x][i] = db[x][i] = 0.f;
    }
  const long long units = (long long)g.tokens * g.parts;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * kWarps) {
    const int t = int(u / g.parts), part = int(u - (long long)t * g.parts);
    float c[4], s[4];
    if (g.rotary > 0) angles(turns, g.position[t], c, s);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const __nv_bfloat16* xin = g.x[x].p + t * g.x[x].ts;
      const __nv_bfloat16* dyin = BACK ? g.dy[x].p + t * g.dy[x].ts : nullptr;
      __nv_bfloat16* out = g.out[x].p + t * g.out[x].ts;
      // every lane of the warp goes round equally often: the sums cross lanes
      for (int h0 = part * kGroups * kDepth; h0 < g.heads[x]; h0 += g.parts * kGroups * kDepth) {
        float a[kDepth][4], b[kDepth][4], ga[kDepth][4], gb[kDepth][4];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int h = h0 + d * kGroups + group;
          const bool has = sh.in && h < g.heads[x];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[d][i] = b[d][i] = ga[d][i] = gb[d][i] = 0.f;
          if (has) {
            load4<VEC>(xin + h * g.x[x].hs + sh.a, a[d]);
            load4<VEC>(xin + h * g.x[x].hs + sh.b, b[d]);
            if (BACK) {
              load4<VEC>(dyin + h * g.dy[x].hs + sh.a, ga[d]);
              load4<VEC>(dyin + h * g.dy[x].hs + sh.b, gb[d]);
            }
          }
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int h = h0 + d * kGroups + group;
          const bool has = sh.in && h < g.heads[x];
          const float r = rsqrtf(group_sum<LANES>(square_sum(a[d], b[d])) * inv_dim + g.eps);
          if (!BACK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[d][i] = a[d][i] * r * wa[x][i];
              b[d][i] = b[d][i] * r * wb[x][i];
            }
            if (sh.turned) turn<ILV, false>(a[d], b[d], c, s);
          } else {
            if (sh.turned) turn<ILV, true>(ga[d], gb[d], c, s);
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[d][i] *= r;  // n
              b[d][i] *= r;
              if (has) {
                da[x][i] = fmaf(ga[d][i], a[d][i], da[x][i]);
                db[x][i] = fmaf(gb[d][i], b[d][i], db[x][i]);
              }
              ga[d][i] *= wa[x][i];
              gb[d][i] *= wb[x][i];
              m = fmaf(ga[d][i], a[d][i], fmaf(gb[d][i], b[d][i], m));
            }
            m = group_sum<LANES>(m) * inv_dim;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[d][i] = r * fmaf(-a[d][i], m, ga[d][i]);
              b[d][i] = r * fmaf(-b[d][i], m, gb[d][i]);
            }
          }
          if (has) {
            store4<VEC>(out + h * g.out[x].hs + sh.a, a[d]);
            store4<VEC>(out + h * g.out[x].hs + sh.b, b[d]);
          }
        }
      }
    }
  }
  if (BACK && g.partial != nullptr) {
    // the block's sums, its groups one after another
    constexpr int kBlockGroups = kWarps * kGroups;
    __shared__ float sums[kBlockGroups][2 * LANES * 8];
    float* mine = sums[(threadIdx.x >> 5) * kGroups + group];
    if (sh.in) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mine[x * g.dim + sh.a + i] = da[x][i];
          mine[x * g.dim + sh.b + i] = db[x][i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.dim; i += kThreads) {
      float v = 0.f;
#pragma unroll 8
      for (int k = 0; k < kBlockGroups; ++k) v += sums[k][i];
      g.partial[(long long)blockIdx.x * 2 * g.dim + i] = v;
    }
  }
}

// The gains' gradients: the blocks' sums added in a fixed order, 32 elements to a block.
__global__ void __launch_bounds__(1024) rope_gains_kernel(const float* partial, int blocks, int dim,
                                                          __nv_bfloat16* dw_q,
                                                          __nv_bfloat16* dw_k) {
  __shared__ float sums[32][33];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (i < 2 * dim)
    for (int b = row; b < blocks; b += 32) v += partial[(long long)b * 2 * dim + i];
  sums[row][lane] = v;
  __syncthreads();
  v = sums[lane][row];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  const int at = blockIdx.x * 32 + row;
  if (lane != 0 || at >= 2 * dim) return;
  __nv_bfloat16* dw = at < dim ? dw_q : dw_k;
  if (dw != nullptr) dw[at < dim ? at : at - dim] = __float2bfloat16_rn(v);
}

using RopeKernel = void (*)(RopeArgs);
template <int LANES>
RopeKernel kernel_of(bool back, bool ilv, bool vec) {
  if (back)
    return ilv ? (vec ? rope_kernel<LANES, true, true, true> : rope_kernel<LANES, true, false, true>)
               : (vec ? rope_kernel<LANES, false, true, true>
                      : rope_kernel<LANES, false, false, true>);
  return ilv ? (vec ? rope_kernel<LANES, true, true, false> : rope_kernel<LANES, true, false, false>)
             : (vec ? rope_kernel<LANES, false, true, false>
                    : rope_kernel<LANES, false, false, false>);
}

}  // namespace

cudaError_t launch_rope(RopeArgs& g, bool backward, bool interleaved, bool vec, int sms,
                        cudaStream_t s) {
  int lanes = 4;  // of a head, a power of two
  while (lanes * 8 < g.dim) lanes *= 2;
  const RopeKernel k = lanes == 4    ? kernel_of<4>(backward, interleaved, vec)
                       : lanes == 8  ? kernel_of<8>(backward, interleaved, vec)
                       : lanes == 16 ? kernel_of<16>(backward, interleaved, vec)
                                     : kernel_of<32>(backward, interleaved, vec);
  // A token to a warp, unless that leaves warps of the GPU idle: then its heads are shared.
  const int most = g.heads[0] > g.heads[1] ? g.heads[0] : g.heads[1];
  const int at_once = 32 / lanes * (backward ? 2 : 4);
  const int max_parts = (most + at_once - 1) / at_once;
  const long long full = (long long)sms * 8 * kWarps;
  g.parts = 1;
  while (g.parts < max_parts && (long long)g.tokens * g.parts < full) ++g.parts;
  long long blocks = ((long long)g.tokens * g.parts + kWarps - 1) / kWarps;
  const long long resident = (long long)sms * 8;
  if (blocks > resident) blocks = resident;
  if (blocks > kRopeBlocks) blocks = kRopeBlocks;
  if (blocks > 0) {
    const cudaError_t e = launch_dependent(k, unsigned(blocks), unsigned(kThreads), s, g);
    if (e != cudaSuccess) return e;
  }
  if (g.partial == nullptr) return cudaSuccess;
  return launch_dependent(rope_gains_kernel, unsigned((2 * g.dim + 31) / 32), 1024u, s,
                          (const float*)g.partial, int(blocks), g.dim, g.dw[0], g.dw[1]);
}

}  // namespace dm
