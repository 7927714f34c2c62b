// Memory-bound kernels of the training-side operators: activations in 8 bits,
// row copies, and the per-token parts of the cross entropy.  Each streams its
// tensors once; offsets are 64-bit.
#include "act8.cuh"
#include "dmuon.h"
#include "launch.h"
#include "shift.cuh"
#include "train.h"

#include <cuda_fp16.h>

namespace dm {
namespace {

constexpr int kThreads = 256;
constexpr int kVecCols = kThreads * 8;  // columns a block covers, 8 per thread

DM_DEV void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}
DM_DEV uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
DM_DEV float load1(const void* p, long long i) {
  return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}
template <bool BF16>
DM_DEV void load8(const void* p, long long i, bool vec, int n, float (&f)[8]) {
  if (vec && n >= 8) {
    if (BF16) {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), f);
    } else {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = q[0], b = q[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? load1<BF16>(p, i + k) : 0.f;
  }
}

// Eight values of a block in 8 bits; the block's other values are in the three
// lanes beside (all lanes of the warp take part).
template <bool BF16>
DM_DEV uint2 act8_pack(const float (&v)[8], float& s) {
  float top = 0.f, bad = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    top = fmaxf(top, fabsf(v[k]));
    bad = fmaf(v[k], 0.f, bad);  // NaN once a value is not finite
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  s = act8_scale(top, bad == 0.f);
  uint32_t w[2] = {0u, 0u};
  if (bad == 0.f && s > 0.f) {
    const float r = __fdiv_rn(1.f, s);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k >> 2] |= (BF16 ? act8_code_bf16(v[k], r) : act8_code_f32(v[k], s)) << (8 * (k & 3));
  }
  return make_uint2(w[0], w[1]);
}
DM_DEV void act8_unpack(const uint2& q, float s, float (&f)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = s * act8_int(w[k >> 2], k & 3);
}
template <bool BF16>
DM_DEV void store8(void* out, long long at, bool vec, int n, const float (&f)[8]) {
  if (vec && n >= 8) {
    if (BF16) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) = pack8(f);
    } else {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      q[0] = make_float4(f[0], f[1], f[2], f[3]);
      q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) {
        if (BF16) static_cast<__nv_bfloat16*>(out)[at + k] = __float2bfloat16_rn(f[k]);
        else static_cast<float*>(out)[at + k] = f[k];
      }
  }
}

// Any shape and pitch: a block covers kVecCols columns of one row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_save_kernel(long long cols, unsigned tiles,
                                                             const void* x, long long ld,
                                                             bool vec_in, bool vec_out,
                                                             signed char* codes,
                                                             __nv_bfloat16* scales) {
  grid_launch_dependents();
  grid_wait();
  const long long row = blockIdx.x / tiles;
  const long long c0 = (long long)(blockIdx.x - unsigned(row) * tiles) * kVecCols + threadIdx.x * 8;
  const int n = c0 < cols ? int(min(8ll, cols - c0)) : 0;
  float v[8], s;
  load8<BF16>(x, row * ld + c0, vec_in, n, v);
  const uint2 w = act8_pack<BF16>(v, s);
  if (n == 0) return;
  signed char* dst = codes + row * cols + c0;
  if (vec_out && n >= 8) {
    *reinterpret_cast<uint2*>(dst) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) dst[k] = (signed char)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
  }
  if ((threadIdx.x & 3) == 0)
    scales[row * ((cols + kActBlock - 1) / kActBlock) + c0 / kActBlock] = __float2bfloat16_rn(s);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_load_kernel(long long cols, unsigned tiles,
                                                             const signed char* codes,
                                                             const __nv_bfloat16* scales,
                                                             void* out, long long ld, bool vec_in,
                                                             bool vec_out) {
  grid_launch_dependents();
  grid_wait();
  const long long row = blockIdx.x / tiles;
  const long long c0 = (long long)(blockIdx.x - unsigned(row) * tiles) * kVecCols + threadIdx.x * 8;
  if (c0 >= cols) return;
  const int n = int(min(8ll, cols - c0));
  const float s = __bfloat162float(scales[row * ((cols + kActBlock - 1) / kActBlock) + c0 / kActBlock]);
  const signed char* src = codes + row * cols + c0;
  float f[8];
  if (vec_in && n >= 8) {
    act8_unpack(*reinterpret_cast<const uint2*>(src), s, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? s * float(src[k]) : 0.f;
  }
  store8<BF16>(out, row * ld + c0, vec_out, n, f);
}

// Contiguous rows of whole blocks: the matrix is one run of blocks, and a thread
// keeps kUnits 16-byte loads in flight.
constexpr int kUnits = 4;
template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_save_flat_kernel(long long units, const void* x,
                                                                  uint2* codes,
                                                                  __nv_bfloat16* scales) {
  grid_launch_dependents();
  grid_wait();
  const long long u0 = (long long)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  float v[kUnits][8];
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    load8<BF16>(x, (u0 + k * kThreads) * 8, true, u0 + k * kThreads < units ? 8 : 0, v[k]);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const long long u = u0 + k * kThreads;
    float s;
    const uint2 w = act8_pack<BF16>(v[k], s);
    if (u < units) {
      codes[u] = w;
      if ((threadIdx.x & 3) == 0) scales[u / 4] = __float2bfloat16_rn(s);
    }
  }
}
template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_load_flat_kernel(long long units,
                                                                  const uint2* codes,
                                                                  const __nv_bfloat16* scales,
                                                                  void* out) {
  grid_launch_dependents();
  grid_wait();
  const long long u0 = (long long)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  uint2 q[kUnits];
  float s[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const long long u = u0 + k * kThreads;
    if (u < units) {
      q[k] = codes[u];
      s[k] = __bfloat162float(scales[u / 4]);
    }
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const long long u = u0 + k * kThreads;
    if (u < units) {
      float f[8];
      act8_unpack(q[k], s[k], f);
      store8<BF16>(out, u * 8, true, 8, f);
    }
  }
}

DM_DEV bool live_target(const long long* target, long long row, long long vocab) {
  if (target == nullptr) return true;
  const long long t = target[row];
  return t >= 0 && t < vocab;
}

// The largest finite |grad_loss| of the tokens that have a target (1 if that is 0), by one
// block.  An infinite one stays infinite relative to it and spoils only its own token's
// gradients, which an infinite scale would spread over all.
DM_DEV void grad_scale(const CopyArgs& g) {
  __shared__ float top[kThreads / 32];
  float m = 0.f;
#pragma unroll 4
  for (long long t = threadIdx.x; t < g.tokens; t += kThreads)
    if (live_target(g.target, t, g.vocab)) {
      const float f = fabsf(g.grad_loss[t]);
      if (f < INFINITY) m = fmaxf(m, f);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, top[w]);
    *g.grad_scale = m > 0.f ? m : 1.f;
  }
}

// Up to CopyArgs::kMost matrices to rows that TMA can read, one launch.  A thread
// moves 8 columns; the threads run through rows and columns alike, so that narrow
// matrices fill them too.  src == nullptr: zeros.
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const __grid_constant__ CopyArgs g) {
  grid_launch_dependents();
  grid_wait();
  if (g.grad_loss != nullptr && blockIdx.x + 1 == gridDim.x) {  // an extra block
    grad_scale(g);
    return;
  }
  int m = 0;
  while (m + 1 < g.n && blockIdx.x >= g.mat[m + 1].block_begin) ++m;
  const CopyArgs::Mat& M = g.mat[m];
  const unsigned per_row = unsigned((M.cols + 7) / 8);
  const unsigned long long u0 =
      (unsigned long long)(blockIdx.x - M.block_begin) * (4 * kThreads) + threadIdx.x;
  const unsigned long long units = (unsigned long long)M.rows * per_row;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long u = u0 + k * kThreads;
    if (u >= units) return;
    const long long row = units <= 0xFFFFFFFFull ? (long long)(unsigned(u) / per_row)
                                                 : (long long)(u / per_row);
    const long long c0 = ((long long)u - row * per_row) * 8;
    const int n = int(min(8ll, M.cols - c0));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (M.src != nullptr && (m > 0 || live_target(g.target, row, g.vocab))) {
      const __nv_bfloat16* p = M.src + row * M.src_ld + c0;
      // the words around eight elements of an inner row lie inside the matrix
      if (n == 8 && (M.src_vec || (row > 0 && row + 1 < M.rows))) {
        uint4 q[1];
        load_shifted<1>(p, q);
        v = q[0];
      } else {
        float f[8];
        load8<true>(p, 0, false, n, f);
        v = pack8(f);
      }
    }
    __nv_bfloat16* d = M.dst + row * M.dst_ld + c0;
    if (M.dst_vec && n == 8) {
      *reinterpret_cast<uint4*>(d) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) reinterpret_cast<uint16_t*>(d)[j] = uint16_t(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// lse and loss from the groups' maxima and sums.  A block takes `tb` tokens (a power
// of two up to 32, few when there are few tokens, so that the groups spread over
// many blocks): lane % tb is the token, everything else strides over the groups
// with four loads in flight.  Partial results join in a fixed order.
//
// With M and S the maximum and sum of all entries but the target, and z the target's
// logit, loss = log(1 + S exp(M - z)): a sure token's keeps its relative accuracy, since
// nothing small is added to 1 before the logarithm (log1p).  What then decides is the
// error of z, a sum of one sign as large as it gets, so z is summed here again without
// one: the products are exact in fp32, each addition's rounding error is kept
// (two_sum) and added at the end.  That reads hidden and one row of the head per token,
// while the product before still runs (both are older than it).  One token of 4096 x
// 128256 whose loss is 0.005: relative error 1.1e-6; 3.6e-5 with the product's logit and a
// sum that holds the target's 1.
constexpr int kRowThreads = 1024;
DM_DEV void two_sum(float a, float b, float& sum, float& err) {
  sum = __fadd_rn(a, b);
  const float t = __fsub_rn(sum, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(sum, t)), __fsub_rn(b, t));
}
DM_DEV void add_exactly(float2& z, float v) {
  float e;
  two_sum(z.x, v, z.x, e);
  z.y = __fadd_rn(z.y, e);
}
DM_DEV float2 join_lanes(float2 z) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, z.x, o), y = __shfl_xor_sync(0xffffffffu, z.y, o);
    add_exactly(z, x);
    z.y = __fadd_rn(z.y, y);
  }
  return z;
}
// Part `part` of `parts` of a row of hidden times a row of the head, in every lane.
DM_DEV float2 target_logit(const XentRows& r, long long row, long long target, int part, int parts,
                           int lane) {
  const __nv_bfloat16 *h = r.hidden + row * r.hidden_ld, *w = r.weight + target * r.weight_ld;
  const int whole = r.k / 8 * 8;
  float2 z = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int c = (part * 32 + lane) * 8; c < whole; c += parts * 256) {
    float a[8], b[8];
    unpack8(*reinterpret_cast<const uint4*>(h + c), a);
    unpack8(*reinterpret_cast<const uint4*>(w + c), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) add_exactly(z, __fmul_rn(a[j], b[j]));
  }
  if (part == 0 && whole + lane < r.k)
    add_exactly(z, __fmul_rn(__bfloat162float(h[whole + lane]), __bfloat162float(w[whole + lane])));
  return join_lanes(z);
}
// maximum and sum of up to N pairs; pairs at the common maximum add as they are, so
// that a NaN beside an infinity stays
DM_DEV float weigh(float m, float s, float top) {
  return m == top ? s : s * exp2f((m - top) * 1.44269504f);
}
DM_DEV void join(float& m, float& s, float pm, float ps) {
  const float top = fmaxf(m, pm);
  s = weigh(m, s, top) + weigh(pm, ps, top);
  m = top;
}
__global__ void __launch_bounds__(kRowThreads) xent_rows_kernel(const XentRows r, int tb) {
  __shared__ float sm[kRowThreads / 32][32], ss[kRowThreads / 32][32];
  __shared__ float2 zt[kRowThreads / 32];
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int parts = 32 / tb;  // warps that share a target's logit
  {
    const long long row = (long long)blockIdx.x * tb + w / parts;
    if (row < r.tokens && live_target(r.target, row, r.vocab)) {
      const float2 z = target_logit(r, row, r.target[row], w % parts, parts, lane);
      if (lane == 0) zt[w] = z;
    }
  }
  grid_wait();
  const long long row = (long long)blockIdx.x * tb + (lane & (tb - 1));
  const bool in = row < r.tokens;
  const long long groups = (r.vocab + r.group - 1) / r.group;
  const int step = kRowThreads / tb;
  float m = -INFINITY, s = 0.f;
  if (in)
    for (long long g = w * (32 / tb) + lane / tb; g < groups; g += 4 * step) {
      float2 p[4];
      float top = m;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = g + k * step < groups ? r.group_stat[(g + k * step) * r.stat_ld + row]
                                     : make_float2(-INFINITY, 0.f);
        top = fmaxf(top, p[k].x);
      }
      s = weigh(m, s, top);
#pragma unroll
      for (int k = 0; k < 4; ++k) s += weigh(p[k].x, p[k].y, top);
      m = top;
    }
  for (int o = tb; o < 32; o <<= 1)
    join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
  sm[w][lane] = m;
  ss[w][lane] = s;
  __syncthreads();
  // warp w joins the warps' results of token w of the block: lane = warp
  if (w >= tb) return;
  m = sm[lane][w];
  s = ss[lane][w];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
  const long long t = (long long)blockIdx.x * tb + w;
  float2 z = join_lanes(t < r.tokens && lane < parts ? zt[w * parts + lane]
                                                     : make_float2(0.f, 0.f));
  if (lane != 0 || t >= r.tokens) return;
  if (!live_target(r.target, t, r.vocab)) {
    r.loss[t] = r.lse[t] = 0.f;
    return;
  }
  // an infinite logit has no rounding error, and one of +infinity no loss
  if (!(fabsf(z.x) < INFINITY)) z.y = 0.f;
  const float d = z.x < INFINITY ? (m - z.x) - z.y : __int_as_float(0x7fc00000);
  if (d <= 0.f) {
    const float loss = log1pf(s * expf(d));
    r.loss[t] = loss;
    r.lse[t] = z.x + (z.y + loss);
  } else {
    const float ls = logf(s + expf(-d));
    r.loss[t] = d + ls;
    r.lse[t] = m + ls;
  }
}

// G = grad_loss / scale * (exp(z - lse) - [entry is the target]).  kXentScale exp(z - m)
// comes in fp16: 2^-11 of an entry's G beside the 2^-8 of rounding it to bf16 here, down to
// 2^-29 of its group's largest, and 2^-40 of that one's G below.  At the target the
// difference to 1 is taken as expm1(-loss).  With equal weights (a mean) grad_loss / scale
// is 1, and the -1 of an unlikely target is exact; the scale is put back in fp32 where the
// products are written.
// A block takes kGradCols columns of one row, four 16-byte loads in flight a thread.
constexpr int kGradCols = 4 * kVecCols;
__global__ void __launch_bounds__(kThreads) xent_grad_kernel(const XentRows r, uint4* e,
                                                             long long e_ld, unsigned tiles) {
  grid_launch_dependents();
  grid_wait();
  const long long row = blockIdx.x / tiles;
  const long long c0 = (long long)(blockIdx.x - unsigned(row) * tiles) * kGradCols + threadIdx.x * 8;
  uint4* p = e + (row * e_ld + c0) / 8;
  uint4 q[4];
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long c = c0 + k * kVecCols;
    if (c < r.vocab) {
      q[k] = p[k * kThreads];
      m[k] = r.group_stat[(unsigned(c) / unsigned(r.group)) * r.stat_ld + row].x;
    }
  }
  const long long t = r.target[row];
  const bool live = t >= 0 && t < r.vocab;
  const float gl = live ? r.grad_loss[row] / *r.grad_scale : 0.f, lse = r.lse[row];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long c = c0 + k * kVecCols;
    if (c >= r.vocab) break;
    if (!live) {
      p[k * kThreads] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const float f = gl * (1.f / kXentScale) * exp2f((m[k] - lse) * 1.44269504f);
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[2 * j] = x.x * f;
      v[2 * j + 1] = x.y * f;
    }
    if (t >= c && t < c + 8) {
      const float at = gl * expm1f(-r.loss[row]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j == t) v[j] = at;
    }
    p[k * kThreads] = pack8(v);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
long long tiles_of(long long cols) { return (cols + kVecCols - 1) / kVecCols; }

}  // namespace

cudaError_t launch_act8_save(long long rows, long long cols, const void* x, long long ld,
                             bool bf16, signed char* codes, __nv_bfloat16* scales,
                             cudaStream_t s) {
  const bool vin = aligned16(x) && ld % 8 == 0;
  const bool vout = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  if (vin && vout && ld == cols && cols % kActBlock == 0) {
    const long long units = rows * cols / 8;
    return launch_dependent(bf16 ? act8_save_flat_kernel<true> : act8_save_flat_kernel<false>,
                            unsigned((units + kThreads * kUnits - 1) / (kThreads * kUnits)),
                            kThreads, s, units, x, reinterpret_cast<uint2*>(codes), scales);
  }
  const unsigned tiles = unsigned(tiles_of(cols));
  return launch_dependent(bf16 ? act8_save_kernel<true> : act8_save_kernel<false>,
                          unsigned(rows) * tiles, kThreads, s, cols, tiles, x, ld, vin, vout, codes,
                          scales);
}

cudaError_t launch_act8_load(long long rows, long long cols, const signed char* codes,
                             const __nv_bfloat16* scales, void* out, long long ld, bool bf16,
                             cudaStream_t s) {
  const bool vin = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  const bool vout = aligned16(out) && ld % 8 == 0;
  if (vin && vout && ld == cols && cols % kActBlock == 0) {
    const long long units = rows * cols / 8;
    return launch_dependent(bf16 ? act8_load_flat_kernel<true> : act8_load_flat_kernel<false>,
                            unsigned((units + kThreads * kUnits - 1) / (kThreads * kUnits)),
                            kThreads, s, units, reinterpret_cast<const uint2*>(codes), scales, out);
  }
  const unsigned tiles = unsigned(tiles_of(cols));
  return launch_dependent(bf16 ? act8_load_kernel<true> : act8_load_kernel<false>,
                          unsigned(rows) * tiles, kThreads, s, cols, tiles, codes, scales, out, ld,
                          vin, vout);
}

cudaError_t launch_copy_rows(CopyArgs& g, cudaStream_t s) {
  unsigned blocks = 0;
  for (int m = 0; m < g.n; ++m) {
    CopyArgs::Mat& M = g.mat[m];
    M.block_begin = blocks;
    M.src_vec = aligned16(M.src) && M.src_ld % 8 == 0;
    M.dst_vec = aligned16(M.dst) && M.dst_ld % 8 == 0;
    const long long units = M.rows * ((M.cols + 7) / 8);
    blocks += unsigned((units + 4 * kThreads - 1) / (4 * kThreads));
  }
  if (g.grad_loss != nullptr) ++blocks;
  if (blocks == 0) return cudaSuccess;
  return launch_dependent(copy_rows_kernel, blocks, unsigned(kThreads), s, g);
}

cudaError_t launch_xent_rows(const XentRows& r, cudaStream_t s) {
  int tb = 32;
  while (tb > 1 && r.tokens < 152ll * tb) tb >>= 1;
  return launch_dependent(xent_rows_kernel, unsigned((r.tokens + tb - 1) / tb), kRowThreads, s, r,
                          tb);
}

cudaError_t launch_xent_grad(const XentRows& r, void* e, long long e_ld, cudaStream_t s) {
  const unsigned tiles = unsigned((r.vocab + kGradCols - 1) / kGradCols);
  return launch_dependent(xent_grad_kernel, unsigned(r.tokens) * tiles, kThreads, s, r,
                          static_cast<uint4*>(e), e_ld, tiles);
}

}  // namespace dm
