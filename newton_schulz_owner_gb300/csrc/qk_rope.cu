// Root-mean-square norm of every query and key head, its gains, and the rotation by
// position, forward and backward, in one pass over the heads.
//
// Bound by HBM: 4 bytes an element forward (read and write bf16), 6 backward.  A head is
// spread over LANES lanes of a warp, 8 elements each, as four pairs: in the split form elements
// 4l .. 4l + 3 of each half of the rotated part, in the interleaved form (and past the rotated
// part) eight neighbours.  Both sides of a pair lie in one lane, so that only the sums of squares
// cross lanes.  A warp loads all heads that it takes of a token before it computes on the first.
//
// What limits it besides is issuing: with 130 instructions for 2 x 128 elements of a head a warp left
// HBM idle half the time.  Hence pairs go two at a time (fma.rn.f32x2), and the gains are folded
// into the sines and cosines once per token:
//   n_a w_a cos - n_b w_b sin = r (x_a (w_a cos) - x_b (w_b sin))
// Measured, 8192 tokens of 64 heads of 128: 44 us forward (6.1 TB/s, 0.90 of the copy rate; 111
// with one element at a time), 73 us backward (5.5 TB/s, 0.81; 148 so).  With twice as many registers a
// thread as forward it has half the warps to wait for memory with, hence the next chunk is brought to L2
// while one is computed (79 us without; 77 two chunks ahead).
//
// Angles.  t = position * inv_freq radians is needed modulo a turn only, and in fp32 a
// position of 10^5 would leave a third of the digits.  inv_freq / 2 pi as a 64-bit fraction of a
// turn (an exact 24 x 128-bit product, cut) times the position, modulo 2^64, has an error of
// 2^-33 turns at most; its top 32 bits are the angle.
#include "f32x2.cuh"
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

// ------------------------------------------------------------------ a lane's share of a head
// Four pairs (x, y), two to a word of each.
struct Pairs {
  F2 x[2], y[2];
};
struct Raw {  // eight bf16: the lane's two runs of four
  uint2 a, b;
};
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

template <bool VEC>
DM_DEV uint2 load4(const __nv_bfloat16* p) {
  if (VEC) return *reinterpret_cast<const uint2*>(p);
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  return make_uint2(uint32_t(h[0]) | uint32_t(h[1]) << 16, uint32_t(h[2]) | uint32_t(h[3]) << 16);
}
template <bool VEC>
DM_DEV void store4(__nv_bfloat16* p, uint2 v) {
  if (VEC) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    h[0] = uint16_t(v.x);
    h[1] = uint16_t(v.x >> 16);
    h[2] = uint16_t(v.y);
    h[3] = uint16_t(v.y >> 16);
  }
}
template <bool ILV>
DM_DEV Pairs unpack(const Raw& r) {
  Pairs p;
  if (ILV) {
    p.x[0] = f2(bf16_lo(r.a.x), bf16_lo(r.a.y));
    p.y[0] = f2(bf16_hi(r.a.x), bf16_hi(r.a.y));
    p.x[1] = f2(bf16_lo(r.b.x), bf16_lo(r.b.y));
    p.y[1] = f2(bf16_hi(r.b.x), bf16_hi(r.b.y));
  } else {
    p.x[0] = f2(bf16_lo(r.a.x), bf16_hi(r.a.x));
    p.x[1] = f2(bf16_lo(r.a.y), bf16_hi(r.a.y));
    p.y[0] = f2(bf16_lo(r.b.x), bf16_hi(r.b.x));
    p.y[1] = f2(bf16_lo(r.b.y), bf16_hi(r.b.y));
  }
  return p;
}
// The eight values in the order of the lane's elements.
template <bool ILV>
DM_DEV void in_order(const Pairs& p, float (&v)[8]) {
  float x[4], y[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f2_split(p.x[i], x[2 * i], x[2 * i + 1]);
    f2_split(p.y[i], y[2 * i], y[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[ILV ? 2 * i : i] = x[i];
    v[ILV ? 2 * i + 1 : i + 4] = y[i];
  }
}
template <bool ILV, bool VEC>
DM_DEV void store(__nv_bfloat16* p, const Share& sh, const Pairs& v) {
  float o[8];
  in_order<ILV>(v, o);
  store4<VEC>(p + sh.a, make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])));
  store4<VEC>(p + sh.b, make_uint2(pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])));
}

// ------------------------------------------------------------------ angles
// inv_freq radians as a fraction of a turn in 2^-64 (whole turns dropped).
DM_DEV unsigned long long turn_of(float inv_freq) {
  // 2^128 / 2 pi
  constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  const uint32_t bits = __float_as_uint(inv_freq);
  const int expo = int(bits >> 23) & 255;
  unsigned long long m = bits & 0x7FFFFFu;
  if (expo != 0) m |= 0x800000u;
  // |f| = m 2^(e - 150), so the fraction is m (2^128 / 2 pi) 2^(e - 214) modulo 2^64
  const int shift = 214 - (expo == 0 ? 1 : expo);
  const unsigned long long w0 = m * kLo, c = __umul64hi(m, kLo), lo = m * kHi;
  const unsigned long long w1 = lo + c, w2 = __umul64hi(m, kHi) + (w1 < lo ? 1 : 0);
  unsigned long long f;
  if (shift >= 192) f = 0;
  else if (shift >= 128) f = w2 >> (shift - 128);
  else if (shift > 64) f = w1 >> (shift - 64) | w2 << (128 - shift);
  else if (shift == 64) f = w1;
  else if (shift > 0) f = w0 >> shift | w1 << (64 - shift);
  else f = shift > -64 ? w0 << -shift : 0;
  return (bits >> 31) != 0 ? 0ull - f : f;
}

// Sines and cosines of a lane's four angles; one and zero where nothing turns.
DM_DEV void angles(const float* inv_freq, int l, bool turned, int position, F2 (&c)[2], F2 (&s)[2]) {
  float co[4], si[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    co[i] = 1.f;
    si[i] = 0.f;
    if (turned) {
      const float f = inv_freq[4 * l + i];
      const unsigned long long at = turn_of(f) * static_cast<unsigned long long>((long long)position);
      // a frequency that is no number leaves none
      sincospif(fmaf(float(int(at >> 32)), 4.656612873077393e-10f, f - f), &si[i], &co[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[i] = f2(co[2 * i], co[2 * i + 1]);
    s[i] = f2(si[2 * i], si[2 * i + 1]);
  }
}

template <int LANES>
DM_DEV float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
DM_DEV float dot(const Pairs& a, const Pairs& b) {
  F2 t = mul2(a.x[0], b.x[0]);
  t = fma2(a.x[1], b.x[1], t);
  t = fma2(a.y[0], b.y[0], t);
  t = fma2(a.y[1], b.y[1], t);
  float lo, hi;
  f2_split(t, lo, hi);
  return lo + hi;
}

// A lane's gains.
template <bool ILV, bool VEC>
DM_DEV Pairs gains(const __nv_bfloat16* w, const Share& sh) {
  Raw r{make_uint2(0x3F803F80u, 0x3F803F80u), make_uint2(0x3F803F80u, 0x3F803F80u)};
  if (w != nullptr && sh.in) {
    r.a = load4<VEC>(w + sh.a);
    r.b = load4<VEC>(w + sh.b);
  }
  return unpack<ILV>(r);
}

// ------------------------------------------------------------------ kernels
// A chunk is kGroups * kDepth heads of queries or keys; a warp takes `per` chunks of a token.
template <int LANES>
struct Chunk {
  static constexpr int kGroups = 32 / LANES, kDepth = 4, kHeads = kGroups * kDepth;
};
constexpr int kBlocks = 7, kGradBlocks = 4;  // resident on an SM

template <int LANES, bool ILV, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ RopeArgs g) {
  using C = Chunk<LANES>;
  const int lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
  const Share sh = share_of<ILV>(l, g.dim, g.rotary);
  const unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = int(u / unsigned(g.parts)), part = int(u - unsigned(t) * unsigned(g.parts));
  grid_launch_dependents();
  grid_wait();
  if (t >= g.tokens) return;
  const float inv_dim = 1.f / float(g.dim);
  const int q_chunks = (g.heads[0] + C::kHeads - 1) / C::kHeads;
  const int chunks = q_chunks + (g.heads[1] + C::kHeads - 1) / C::kHeads;
  const int position = g.rotary > 0 ? g.position[t] : 0;
  F2 c[2], s[2];
  bool fresh = true;
  for (int n = part * g.per; n < min(chunks, (part + 1) * g.per); ++n) {
    const int x = n >= q_chunks ? 1 : 0;
    const int h0 = (n - x * q_chunks) * C::kHeads + group;
    const __nv_bfloat16* in = g.x[x].p + t * g.x[x].ts + h0 * g.x[x].hs;
    __nv_bfloat16* out = g.out[x].p + t * g.out[x].ts + h0 * g.out[x].hs;
    const long long in_step = C::kGroups * g.x[x].hs, out_step = C::kGroups * g.out[x].hs;
    const int left = sh.in ? (g.heads[x] - h0 + C::kGroups - 1) / C::kGroups : 0;  // heads from h0 on
    Raw raw[C::kDepth];
#pragma unroll
    for (int d = 0; d < C::kDepth; ++d, in += in_step) {
      raw[d] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
      if (d < left) {
        raw[d].a = load4<VEC>(in + sh.a);
        raw[d].b = load4<VEC>(in + sh.b);
      }
    }
    if (fresh) angles(g.inv_freq, l, sh.turned, position, c, s);
    fresh = false;
    const Pairs w = gains<ILV, VEC>(g.w[x], sh);
    Pairs wc, ws;  // x_out = r (x wc.x - y ws.y), y_out = r (x ws.x + y wc.y)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wc.x[i] = mul2(w.x[i], c[i]);
      wc.y[i] = mul2(w.y[i], c[i]);
      ws.x[i] = mul2(w.x[i], s[i]);
      ws.y[i] = negate2(mul2(w.y[i], s[i]));
    }
#pragma unroll
    for (int d = 0; d < C::kDepth; ++d, out += out_step) {
      const Pairs v = unpack<ILV>(raw[d]);
      const float r = rsqrtf(fmaf(group_sum<LANES>(dot(v, v)), inv_dim, g.eps));
      const F2 rr = f2(r, r);
      Pairs o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o.x[i] = mul2(rr, fma2(v.x[i], wc.x[i], mul2(v.y[i], ws.y[i])));
        o.y[i] = mul2(rr, fma2(v.x[i], ws.x[i], mul2(v.y[i], wc.y[i])));
      }
      if (d < left) store<ILV, VEC>(out, sh, o);
    }
  }
}

// Brings a lane's part of a chunk of heads to L2: by one lane of eight, whose elements share a line.
template <int LANES>
DM_DEV void fetch_ahead(const Heads& h, const Share& sh, int l, int t, int h0, int heads) {
  using C = Chunk<LANES>;
  if ((l & 7) != 0 || !sh.in) return;
  const __nv_bfloat16* p = h.p + t * h.ts + h0 * h.hs + 8 * l;
#pragma unroll
  for (int d = 0; d < C::kDepth; ++d)
    if (h0 + d * C::kGroups < heads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p + d * C::kGroups * h.hs));
}

// Gradients; where they are wanted (partial) the gains' too: a block sums its own, for rope_gains_kernel.
template <int LANES, bool ILV, bool VEC>
__global__ void __launch_bounds__(kThreads, kGradBlocks) rope_grad_kernel(const __grid_constant__ RopeArgs g) {
  using C = Chunk<LANES>;
  const int lane = threadIdx.x & 31, l = lane % LANES, group = lane / LANES;
  const Share sh = share_of<ILV>(l, g.dim, g.rotary);
  grid_launch_dependents();
  grid_wait();
  const float inv_dim = 1.f / float(g.dim);
  const int q_chunks = (g.heads[0] + C::kHeads - 1) / C::kHeads;
  const int chunks = q_chunks + (g.heads[1] + C::kHeads - 1) / C::kHeads;
  Pairs dw[2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[x].x[i] = dw[x].y[i] = 0;
  const unsigned units = unsigned(g.tokens) * unsigned(g.parts);
  for (unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const int t = int(u / unsigned(g.parts)), part = int(u - unsigned(t) * unsigned(g.parts));
    const int position = g.rotary > 0 ? g.position[t] : 0;
    F2 c[2], s[2], minus_s[2];
    angles(g.inv_freq, l, sh.turned, position, c, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) minus_s[i] = negate2(s[i]);
    const int end = min(chunks, (part + 1) * g.per);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Pairs w = gains<ILV, VEC>(g.heads[x] > 0 ? g.w[x] : nullptr, sh);
      const long long in_step = C::kGroups * g.x[x].hs, dy_step = C::kGroups * g.dy[x].hs,
                      out_step = C::kGroups * g.out[x].hs;
#pragma unroll 1
      for (int n = x == 0 ? part * g.per : max(part * g.per, q_chunks);
           n < (x == 0 ? min(end, q_chunks) : end); ++n) {
        const int h0 = (n - x * q_chunks) * C::kHeads + group;
        const __nv_bfloat16* in = g.x[x].p + t * g.x[x].ts + h0 * g.x[x].hs;
        const __nv_bfloat16* dy = g.dy[x].p + t * g.dy[x].ts + h0 * g.dy[x].hs;
        __nv_bfloat16* out = g.out[x].p + t * g.out[x].ts + h0 * g.out[x].hs;
        const int left = sh.in ? (g.heads[x] - h0 + C::kGroups - 1) / C::kGroups : 0;
        Raw raw[C::kDepth], grad[C::kDepth];
#pragma unroll
        for (int d = 0; d < C::kDepth; ++d, in += in_step, dy += dy_step) {
          raw[d] = grad[d] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
          if (d < left) {
            raw[d].a = load4<VEC>(in + sh.a);
            raw[d].b = load4<VEC>(in + sh.b);
            grad[d].a = load4<VEC>(dy + sh.a);
            grad[d].b = load4<VEC>(dy + sh.b);
          }
        }
        {
          // the next chunk, of this token or of the warp's next one
          int t1 = t, n1 = n + 1;
          if (n1 >= end) {
            const unsigned u1 = u + gridDim.x * kWarps;
            t1 = u1 < units ? int(u1 / unsigned(g.parts)) : -1;
            n1 = int(u1 - unsigned(t1) * unsigned(g.parts)) * g.per;
          }
          if (t1 >= 0) {
            const int x1 = n1 >= q_chunks ? 1 : 0, h1 = (n1 - x1 * q_chunks) * C::kHeads + group;
            fetch_ahead<LANES>(x1 ? g.x[1] : g.x[0], sh, l, t1, h1, x1 ? g.heads[1] : g.heads[0]);
            fetch_ahead<LANES>(x1 ? g.dy[1] : g.dy[0], sh, l, t1, h1, x1 ? g.heads[1] : g.heads[0]);
          }
        }
#pragma unroll
        for (int d = 0; d < C::kDepth; ++d, out += out_step) {
          Pairs v = unpack<ILV>(raw[d]);
          const Pairs z = unpack<ILV>(grad[d]);
          // (of an absent head 1: with eps = 0 its root would be infinite)
          const float square = fmaf(group_sum<LANES>(dot(v, v)), inv_dim, g.eps);
          const float r = rsqrtf(d < left ? square : 1.f);
          const F2 rr = f2(r, r);
          Pairs gw;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const F2 gx = fma2(z.x[i], c[i], mul2(z.y[i], s[i]));
            const F2 gy = fma2(z.y[i], c[i], mul2(z.x[i], minus_s[i]));
            v.x[i] = mul2(v.x[i], rr);  // n
            v.y[i] = mul2(v.y[i], rr);
            dw[x].x[i] = fma2(gx, v.x[i], dw[x].x[i]);
            dw[x].y[i] = fma2(gy, v.y[i], dw[x].y[i]);
            gw.x[i] = mul2(gx, w.x[i]);
            gw.y[i] = mul2(gy, w.y[i]);
          }
          const float m = -group_sum<LANES>(dot(gw, v)) * inv_dim;
          const F2 mm = f2(m, m);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            v.x[i] = mul2(rr, fma2(v.x[i], mm, gw.x[i]));
            v.y[i] = mul2(rr, fma2(v.y[i], mm, gw.y[i]));
          }
          if (d < left) store<ILV, VEC>(out, sh, v);
        }
      }
    }
  }
  if (g.partial == nullptr) return;
  // the block's sums, its groups one after another
  constexpr int kBlockGroups = kWarps * C::kGroups;
  __shared__ float sums[kBlockGroups][2 * LANES * 8];
  float* mine = sums[(threadIdx.x >> 5) * C::kGroups + group];
  if (sh.in) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v[8];
      in_order<ILV>(dw[x], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mine[x * g.dim + sh.a + i] = v[i];
        mine[x * g.dim + sh.b + i] = v[i + 4];
      }
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
#pragma unroll 8
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
    return ilv ? (vec ? rope_grad_kernel<LANES, true, true> : rope_grad_kernel<LANES, true, false>)
               : (vec ? rope_grad_kernel<LANES, false, true> : rope_grad_kernel<LANES, false, false>);
  return ilv ? (vec ? rope_kernel<LANES, true, true> : rope_kernel<LANES, true, false>)
             : (vec ? rope_kernel<LANES, false, true> : rope_kernel<LANES, false, false>);
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
  // Chunks of a warp share their token's sines; but with few tokens more warps of one chunk each
  // fill the GPU (8192 tokens of 64 heads of 128, an earlier kernel: 52 us with 2 chunks to a warp, 48 with
  // 8, which is 44 now; backward 82 with 2, 75 with 4, 73 with 8; 777 of 32: 5.1 with one, 6.2 with 2).  Backward, blocks stay and take
  // token after token, so that the gains' sums meet once a block (88 us with twice the blocks that
  // fit, 82 with as many).
  const int heads = 32 / lanes * 4;
  const int chunks = (g.heads[0] + heads - 1) / heads + (g.heads[1] + heads - 1) / heads;
  g.per = (long long)g.tokens * chunks > (long long)sms * 56 ? 8 : 1;
  g.parts = (chunks + g.per - 1) / g.per;
  const long long units = (long long)g.tokens * g.parts;
  long long blocks = (units + kWarps - 1) / kWarps;
  if (backward && blocks > (long long)sms * kGradBlocks) blocks = (long long)sms * kGradBlocks;
  if (backward && blocks > kRopeBlocks) blocks = kRopeBlocks;
  if (blocks > 0) {
    const cudaError_t e = launch_dependent(k, unsigned(blocks), unsigned(kThreads), s, g);
    if (e != cudaSuccess) return e;
  }
  if (g.partial == nullptr) return cudaSuccess;
  return launch_dependent(rope_gains_kernel, unsigned((2 * g.dim + 31) / 32), 1024u, s,
                          (const float*)g.partial, int(blocks), g.dim, g.dw[0], g.dw[1]);
}

}  // namespace dm
