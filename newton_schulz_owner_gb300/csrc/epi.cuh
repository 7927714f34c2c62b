// Epilogue pieces shared by the tensor-core kernels: 32 x 32 bf16 chunks staged
// in shared memory in the layout of the TMA 64-byte swizzle, and the record of a
// bounded wait that gave up.
#pragma once
#include "dmuon.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace dm {

constexpr int kEpiBufBytes = 32 * 32 * 2;  // one 32 x 32 bf16 epilogue chunk
// After a bounded wait gives up, wait this long before leaving so that copies
// and MMAs already issued to this CTA's shared memory / TMEM have landed.
constexpr long long kAbortSettleCycles = 400000;

DM_DEV void raise_abort(int* err, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicCAS(err, 0, int(DMUON_ERR_TIMEOUT));
}

DM_DEV uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

// 16-byte unit u of row i of a chunk sits at byte i*64 + ((u ^ ((i >> 1) & 3)) << 4).
DM_DEV uint32_t epi_off(int row, int unit) {
  return uint32_t(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
}

DM_DEV void epi_store_row(uint32_t buf, int row, const float (&o)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    st_shared_v4(buf + epi_off(row, u), pack_bf16x2(o[8 * u], o[8 * u + 1]),
                 pack_bf16x2(o[8 * u + 2], o[8 * u + 3]), pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                 pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
}

DM_DEV void epi_load_row(uint32_t buf, int row, float (&x)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t w[4];
    ld_shared_v4(buf + epi_off(row, u), w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
      x[8 * u + 2 * k] = f.x;
      x[8 * u + 2 * k + 1] = f.y;
    }
  }
}

// Element (row, col) of a chunk buffer.
DM_DEV void epi_store_elem(uint32_t buf, int row, int col, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  st_shared_b16(buf + epi_off(row, col >> 3) + uint32_t((col & 7) * 2),
                *reinterpret_cast<const uint16_t*>(&b));
}

}  // namespace dm
