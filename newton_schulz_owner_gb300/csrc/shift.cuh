// Unaligned runs of bytes through aligned 16-byte loads.
#pragma once
#include "ptx.cuh"

namespace dm {

// 16 N bytes at p from the N + 1 aligned 16-byte words around them (N words when p is
// aligned).  The caller makes sure that those words may be read.
template <int N>
DM_DEV void load_shifted(const void* p, uint4 (&out)[N]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const unsigned skip = unsigned(at & 15u);
  const uint4* q = reinterpret_cast<const uint4*>(at - skip);
  if (skip == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __ldcs(q + i);
    return;
  }
  uint32_t w[4 * N + 4];
#pragma unroll
  for (int i = 0; i <= N; ++i) {
    const uint4 v = __ldcs(q + i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  const unsigned word = skip / 4, bits = (skip & 3u) * 8u;
  uint32_t o[4 * N];
#pragma unroll
  for (int k = 0; k < 4 * N; ++k) {
    uint32_t a = w[k], b = w[k + 1];
#pragma unroll
    for (int s = 1; s < 4; ++s)
      if (word == unsigned(s)) {
        a = w[k + s];
        b = k + s + 1 < 4 * N + 4 ? w[k + s + 1] : 0u;
      }
    o[k] = __funnelshift_r(a, b, bits);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

}  // namespace dm
