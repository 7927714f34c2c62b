// Memory-bound kernels of the training-side operators: activations in 8 bits,
// row copies, and the per-token parts of the cross entropy.  Each streams its
// tensors once; offsets are 64-bit.
#include "act8.cuh"
#include "dmuon.h"
#include "launch.h"
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

// Four neighbouring lanes hold a block: 8 values each.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_save_kernel(long long cols, long long tiles,
                                                             const void* x, long long ld,
                                                             bool vec_in, bool vec_out,
                                                             signed char* codes,
                                                             __nv_bfloat16* scales) {
  const long long row = blockIdx.x / tiles;
  const long long c0 = (blockIdx.x - row * tiles) * kVecCols + threadIdx.x * 8;
  const int n = c0 < cols ? int(min(8ll, cols - c0)) : 0;
  float v[8];
  load8<BF16>(x, row * ld + c0, vec_in, n, v);
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    top = fmaxf(top, fabsf(v[k]));
    finite = finite && fabsf(v[k]) <= 3.402823466e38f;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    finite = __shfl_xor_sync(0xffffffffu, int(finite), o) && finite;
  }
  if (n == 0) return;
  const float s = act8_scale(top, finite);
  const bool live = finite && s > 0.f;
  const float r = BF16 && live ? __fdiv_rn(1.f, s) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (live) w[k >> 2] |= (BF16 ? act8_code_bf16(v[k], r) : act8_code_f32(v[k], s)) << (8 * (k & 3));
  signed char* dst = codes + row * cols + c0;
  if (vec_out && n >= 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) dst[k] = (signed char)(w[k >> 2] >> (8 * (k & 3)));
  }
  if ((threadIdx.x & 3) == 0)
    scales[row * ((cols + kActBlock - 1) / kActBlock) + c0 / kActBlock] = __float2bfloat16_rn(s);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) act8_load_kernel(long long cols, long long tiles,
                                                             const signed char* codes,
                                                             const __nv_bfloat16* scales,
                                                             void* out, long long ld, bool vec_in,
                                                             bool vec_out) {
  const long long row = blockIdx.x / tiles;
  const long long c0 = (blockIdx.x - row * tiles) * kVecCols + threadIdx.x * 8;
  if (c0 >= cols) return;
  const int n = int(min(8ll, cols - c0));
  const float s = __bfloat162float(scales[row * ((cols + kActBlock - 1) / kActBlock) + c0 / kActBlock]);
  const signed char* src = codes + row * cols + c0;
  float f[8];
  if (vec_in && n >= 8) {
    const uint2 q = *reinterpret_cast<const uint2*>(src);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = s * float((signed char)(w[k >> 2] >> (8 * (k & 3))));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? s * float(src[k]) : 0.f;
  }
  const long long at = row * ld + c0;
  if (vec_out && n >= 8) {
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

DM_DEV bool live_target(const long long* target, long long row, long long vocab) {
  if (target == nullptr) return true;
  const long long t = target[row];
  return t >= 0 && t < vocab;
}

// src == nullptr: zeros.
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(long long cols, long long tiles,
                                                             const __nv_bfloat16* src,
                                                             long long src_ld,
                                                             __nv_bfloat16* dst, long long dst_ld,
                                                             const long long* target,
                                                             long long vocab, bool vec_in,
                                                             bool vec_out) {
  const long long row = blockIdx.x / tiles;
  const long long c0 = (blockIdx.x - row * tiles) * kVecCols + threadIdx.x * 8;
  if (c0 >= cols) return;
  const int n = int(min(8ll, cols - c0));
  float f[8] = {};
  if (src != nullptr && live_target(target, row, vocab))
    load8<true>(src, row * src_ld + c0, vec_in, n, f);
  __nv_bfloat16* d = dst + row * dst_ld + c0;
  if (vec_out && n >= 8) {
    *reinterpret_cast<uint4*>(d) = pack8(f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) d[k] = __float2bfloat16_rn(f[k]);
  }
}

__global__ void __launch_bounds__(1024) grad_scale_kernel(const float* grad_loss,
                                                          const long long* target,
                                                          long long tokens, long long vocab,
                                                          float* scale) {
  __shared__ float top[32];
  float m = 0.f;
  for (long long t = threadIdx.x; t < tokens; t += 1024)
    if (live_target(target, t, vocab)) m = fmaxf(m, fabsf(grad_loss[t]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = top[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (threadIdx.x == 0) *scale = m > 0.f ? m : 1.f;
  }
}

// One block per 32 tokens: 8 warps share the groups, lane = token.
__global__ void __launch_bounds__(kThreads) xent_rows_kernel(const XentRows r) {
  __shared__ float sm[8][32], ss[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * 32 + lane;
  const bool in = row < r.tokens;
  const long long groups = (r.vocab + kXentGroup - 1) / kXentGroup;
  // running maximum and sum of exponentials relative to it
  float m = -INFINITY, s = 0.f;
  if (in)
    for (long long g = w; g < groups; g += 8) {
      const float2 p = r.group_stat[g * r.stat_ld + row];
      if (p.x > m) {
        s = s * exp2f((m - p.x) * 1.44269504f) + p.y;
        m = p.x;
      } else {
        // groups with the same infinity keep their sum, so that a NaN in it stays
        s += p.x == m ? p.y : p.y * exp2f((p.x - m) * 1.44269504f);
      }
    }
  sm[w][lane] = m;
  ss[w][lane] = s;
  __syncthreads();
  if (w != 0 || !in) return;
  m = sm[0][lane];
#pragma unroll
  for (int k = 1; k < 8; ++k) m = fmaxf(m, sm[k][lane]);
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    s += sm[k][lane] == m ? ss[k][lane] : ss[k][lane] * exp2f((sm[k][lane] - m) * 1.44269504f);
  const bool live = live_target(r.target, row, r.vocab);
  const float ls = logf(s);
  r.loss[row] = live ? (m - r.target_logit[row]) + ls : 0.f;
  r.lse[row] = live ? m + ls : 0.f;
}

// G = grad_loss / scale * (exp(z - lse) - [entry is the target]).  exp(z - m)
// comes in fp16, whose 11 bits leave the one rounding to bf16 here the only one
// that shows; at the target the difference to 1 is taken as expm1(-loss).  With
// equal weights (a mean) grad_loss / scale is 1, and the -1 of an unlikely target
// is exact; the scale is put back in fp32 where the products are written.
__global__ void __launch_bounds__(kThreads) xent_grad_kernel(const XentRows r, uint4* e,
                                                             long long e_ld, long long tiles) {
  const long long row = blockIdx.x / tiles;
  const long long c0 = (blockIdx.x - row * tiles) * kVecCols + threadIdx.x * 8;
  if (c0 >= r.vocab) return;
  uint4* p = e + (row * e_ld + c0) / 8;
  const long long t = r.target[row];
  if (t < 0 || t >= r.vocab) {
    *p = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const float gl = r.grad_loss[row] / *r.grad_scale;
  const float f = gl * exp2f((r.group_stat[(c0 / kXentGroup) * r.stat_ld + row].x - r.lse[row]) *
                             1.44269504f);
  const uint4 q = *p;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
    v[2 * k] = x.x * f;
    v[2 * k + 1] = x.y * f;
  }
  if (t >= c0 && t < c0 + 8) {
    const float at = gl * expm1f(-r.loss[row]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + k == t) v[k] = at;
  }
  *p = pack8(v);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
long long tiles_of(long long cols) { return (cols + kVecCols - 1) / kVecCols; }

}  // namespace

cudaError_t launch_act8_save(long long rows, long long cols, const void* x, long long ld,
                             bool bf16, signed char* codes, __nv_bfloat16* scales,
                             cudaStream_t s) {
  const long long tiles = tiles_of(cols);
  const bool vin = aligned16(x) && ld % 8 == 0;
  const bool vout = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  const unsigned grid = unsigned(rows * tiles);
  if (bf16)
    act8_save_kernel<true><<<grid, kThreads, 0, s>>>(cols, tiles, x, ld, vin, vout, codes, scales);
  else
    act8_save_kernel<false><<<grid, kThreads, 0, s>>>(cols, tiles, x, ld, vin, vout, codes, scales);
  return counted(cudaGetLastError());
}

cudaError_t launch_act8_load(long long rows, long long cols, const signed char* codes,
                             const __nv_bfloat16* scales, void* out, long long ld, bool bf16,
                             cudaStream_t s) {
  const long long tiles = tiles_of(cols);
  const bool vin = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  const bool vout = aligned16(out) && ld % 8 == 0;
  const unsigned grid = unsigned(rows * tiles);
  if (bf16)
    act8_load_kernel<true><<<grid, kThreads, 0, s>>>(cols, tiles, codes, scales, out, ld, vin, vout);
  else
    act8_load_kernel<false><<<grid, kThreads, 0, s>>>(cols, tiles, codes, scales, out, ld, vin, vout);
  return counted(cudaGetLastError());
}

cudaError_t launch_copy_rows(long long rows, long long cols, const __nv_bfloat16* src,
                             long long src_ld, __nv_bfloat16* dst, long long dst_ld,
                             const long long* target, long long vocab, cudaStream_t s) {
  const long long tiles = tiles_of(cols);
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  copy_rows_kernel<<<unsigned(rows * tiles), kThreads, 0, s>>>(
      cols, tiles, src, src_ld, dst, dst_ld, target, vocab, aligned16(src) && src_ld % 8 == 0,
      aligned16(dst) && dst_ld % 8 == 0);
  return counted(cudaGetLastError());
}

cudaError_t launch_zero_rows(long long rows, long long cols, __nv_bfloat16* dst, long long ld,
                             cudaStream_t s) {
  return launch_copy_rows(rows, cols, nullptr, 8, dst, ld, nullptr, 0, s);
}

cudaError_t launch_grad_scale(const float* grad_loss, const long long* target, long long tokens,
                              long long vocab, float* scale, cudaStream_t s) {
  grad_scale_kernel<<<1, 1024, 0, s>>>(grad_loss, target, tokens, vocab, scale);
  return counted(cudaGetLastError());
}

cudaError_t launch_xent_rows(const XentRows& r, cudaStream_t s) {
  xent_rows_kernel<<<unsigned((r.tokens + 31) / 32), kThreads, 0, s>>>(r);
  return counted(cudaGetLastError());
}

cudaError_t launch_xent_grad(const XentRows& r, void* e, long long e_ld, cudaStream_t s) {
  const long long tiles = tiles_of(r.vocab);
  xent_grad_kernel<<<unsigned(r.tokens * tiles), kThreads, 0, s>>>(r, static_cast<uint4*>(e), e_ld,
                                                                   tiles);
  return counted(cudaGetLastError());
}

}  // namespace dm
