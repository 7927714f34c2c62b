// Products of the training-side operators on CTA pairs, with fused epilogues.
//
// One launch runs one to three products C = A B (fp32 accumulation of bf16
// operands) whose epilogue is a template parameter (LinEpi):
//   kLinStore    C = bf16(acc); over several launches through an fp32 sum
//   kLinGlu      gate = x Wg^T and up = x Wu^T of the same 128 ffn columns in
//                one accumulator; writes h = act(gate) * up and what backward
//                needs of gate and up
//   kLinGluGrad  acc = dh = dy Wd; with the kept gate and up it writes
//                dgate = dh * up * act'(gate), dup = dh * act(gate) and
//                h = act(gate) * up again
//   kLinXent     acc = logits of 256 tokens x 256 vocabulary entries; writes,
//                per token and group of 128 entries, max m and sum of
//                exp(z - m), the target's logit, and exp(z - m) itself in fp16
//                when gradients are wanted
// Each operand is K-major (rows of K) or MN-major (rows of M or N), a template
// parameter, so no operand is ever transposed in memory.
//
// The products are bound by the tensor cores, so the unit of work is the one
// that needs the least operand traffic per MMA: a 256 x 256 tile on a pair of
// SMs (tcgen05.mma.cta_group::2, M = N = 256, K = 16), each CTA staging its 128
// rows of A and its 128 columns of B by TMA, 128 K-elements (64 KB) per stage,
// three stages.  Warp 0 loads, one thread of warp 1 in the leader issues the
// MMAs, warps 2-9 run the epilogue on one of two 256-column TMEM accumulators
// while the next tile accumulates in the other.  kLinGlu puts Wg's 128 rows in
// the first CTA's B half and Wu's in the second's, which leaves gate and up of
// an element in the same TMEM lane, 128 columns apart.
//
// Tiles are handed out statically.  With T tiles on P pairs the last wave fills
// only T mod P pairs; its tiles are split along K into parts that fill the
// wave, the parts' fp32 accumulators go to the workspace, and the warp that
// arrives last at a part of a tile adds them in order (so the result does not
// depend on which one was last) and runs the epilogue.
#include "act8.cuh"
#include "dmuon.h"
#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "train.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dm {
namespace {

constexpr int kTile = 256;                 // tile rows and columns (CTA pair)
constexpr int kHalf = 128;                 // one CTA's rows of A / columns of B
constexpr int kK = 128;                    // K-elements per stage
constexpr int kStages = 3;
constexpr int kOpBytes = kHalf * kK * 2;   // 32 KB: one CTA's share of an operand
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kPairTx = 2 * kStageBytes;   // both CTAs' loads land on the leader's barrier
constexpr int kAtom = kOpBytes / 2;        // one TMA box: 64 K x 128 rows, or 64 MN x 128 K
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kAccCols = 256;
constexpr int kEpiBytes = kEpiWarps * 2 * kEpiBufBytes;
constexpr int kBarBytes = 512;
constexpr size_t kSmemBytes = size_t(kStages) * kStageBytes + kEpiBytes + 1024 + kBarBytes;
static_assert(kSmemBytes <= 232448, "dynamic shared memory above the per-block limit");

// Tiles of a product are walked in strips of kStrip tile rows, columns outer,
// rows inner: the pairs then work on about 8 row panels and 9 column panels at
// a time, close to the fewest panels that 76 tiles can share.
constexpr int kStrip = 8;

// The tensor core's accumulation rounds toward zero, so a sum of K products loses
// up to K/16 * 2^-25 of its size.  That is far below bf16 for an output that is
// rounded to it, but not for the fp32 losses: the logits are accumulated in runs
// of kRun stages (512 K-elements), each drained and added in registers, rounded
// to nearest.  The drains hide behind the next run's MMAs.
constexpr int kRun = 4;

// Split parts a launch may have, and the size of one.
constexpr int kMaxParts = 152;
constexpr size_t kPartFloats = size_t(kTile) * kTile;

struct Unit {
  int prob, ti, tj;
  int kb_lo, kb_hi;  // K blocks of this unit
  int q, part;       // split tile (0-based) and part; q < 0: a whole tile
};

DM_DEV Unit decode_unit(const LinArgs& g, int u) {
  Unit U;
  int t = u;
  U.q = -1;
  U.part = 0;
  if (u >= g.full_tiles) {
    const int r = u - g.full_tiles;
    U.q = r / g.split;
    U.part = r - U.q * g.split;
    t = g.full_tiles + U.q;
  }
  int p = 0;
  while (p + 1 < g.n_prob && t >= g.prob[p + 1].tile_begin) ++p;
  const LinProblem& P = g.prob[p];
  U.prob = p;
  const int local = t - P.tile_begin;
  const int per = kStrip * P.tiles_n;
  const int strip = local / per;
  const int rows = min(kStrip, P.tiles_m - strip * kStrip);
  const int r = local - strip * per;
  U.tj = r / rows;
  U.ti = strip * kStrip + (r - U.tj * rows);
  const int kb = P.kb0 + P.kb1;
  U.kb_lo = 0;
  U.kb_hi = kb;
  if (U.q >= 0) {
    U.kb_lo = int((long long)kb * U.part / g.split);
    U.kb_hi = int((long long)kb * (U.part + 1) / g.split);
  }
  return U;
}

// ------------------------------------------------------------------ roles
template <int EPI, bool A_MN, bool B_MN>
DM_DEV void producer(const LinArgs& g, uint32_t rank, uint8_t* sA, uint8_t* sB,
                     uint64_t* full_bar, uint64_t* empty_bar, volatile int* abort_flag) {
  const uint32_t leader_full = mapa_shared(smem_u32(full_bar), 0);
  const int clusters = int(cluster_count_x());
  int stage = 0;
  uint32_t phase = 0;
  for (int u = int(cluster_id_x()); u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    const LinProblem& P = g.prob[U.prob];
    const int row0 = U.ti * kTile + int(rank) * kHalf;
    const int col0 = EPI == kLinGlu ? U.tj * kHalf : U.tj * kTile + int(rank) * kHalf;
    for (int kb = U.kb_lo; kb < U.kb_hi; ++kb) {
      const bool second = EPI != kLinGlu && kb >= P.kb0;
      const CUtensorMap* mapA = &g.maps[second ? P.a1 : P.a0];
      const CUtensorMap* mapB =
          &g.maps[EPI == kLinGlu ? (rank == 0 ? P.b0 : P.b1) : (second ? P.b1 : P.b0)];
      const int k0 = (second ? kb - P.kb0 : kb) * kK;
      if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) {
        raise_abort(g.err, abort_flag);
        return;
      }
      if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], kPairTx);
      const uint32_t bar = leader_full + uint32_t(stage) * 8u;
      uint8_t* a = sA + stage * kOpBytes;
      uint8_t* b = sB + stage * kOpBytes;
      // rows, columns and K past the tensors' ends read as zeros
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (A_MN) tma_load_2d_pair(a + h * kAtom, mapA, bar, row0 + h * 64, k0);
        else tma_load_2d_pair(a + h * kAtom, mapA, bar, k0 + h * 64, row0);
        if (B_MN) tma_load_2d_pair(b + h * kAtom, mapB, bar, col0 + h * 64, k0);
        else tma_load_2d_pair(b + h * kAtom, mapB, bar, k0 + h * 64, col0);
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

template <int EPI, bool A_MN, bool B_MN>
DM_DEV void mma_issuer(const LinArgs& g, uint8_t* sA, uint8_t* sB, uint64_t* full_bar,
                       uint64_t* empty_bar, uint64_t* tfull, uint64_t* tempty,
                       uint64_t* drain_bar, uint32_t tmem_base, volatile int* abort_flag) {
  constexpr uint32_t idesc = idesc_bf16(kTile, kTile, A_MN, B_MN);
  // K-major: two 64-element panels 16 KB apart, 32 bytes per K step inside a
  // 128-byte row, 8-row groups 1 KB apart.  MN-major: 64-element atoms 16 KB
  // apart (LBO), 8-row K groups 1 KB apart (SBO), 2 KB per K step.
  const uint64_t a_desc = sdesc_sw128(smem_u32(sA), A_MN ? kAtom : 16, 1024);
  const uint64_t b_desc = sdesc_sw128(smem_u32(sB), B_MN ? kAtom : 16, 1024);
  const int clusters = int(cluster_count_x());
  int stage = 0;
  uint32_t phase = 0;
  int it = 0;  // accumulators handed to the epilogue so far
  bool ok = true;
  for (int u = int(cluster_id_x()); ok && u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    for (int lo = U.kb_lo; ok && lo < U.kb_hi; ++it) {
      const int hi = EPI == kLinXent ? min(lo + kRun, U.kb_hi) : U.kb_hi;
      const int acc = it & 1;
      const uint32_t aph = uint32_t(it >> 1) & 1u;
      if (!mbar_wait_cluster(&tempty[acc], aph ^ 1u, abort_flag)) {
        raise_abort(g.err, abort_flag);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + uint32_t(acc * kAccCols);
      for (int kb = lo; kb < hi; ++kb) {
        if (!mbar_wait_cluster(&full_bar[stage], phase, abort_flag)) {
          raise_abort(g.err, abort_flag);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = a_desc + uint64_t(stage * (kOpBytes >> 4));
        const uint64_t bd = b_desc + uint64_t(stage * (kOpBytes >> 4));
#pragma unroll
        for (int k = 0; k < kK / 16; ++k) {
          const uint64_t ao = A_MN
                                  ? uint64_t(k) * (2048u >> 4)
                                  : uint64_t(k >> 2) * (kAtom >> 4) + uint64_t(k & 3) * (32u >> 4);
          const uint64_t bo = B_MN
                                  ? uint64_t(k) * (2048u >> 4)
                                  : uint64_t(k >> 2) * (kAtom >> 4) + uint64_t(k & 3) * (32u >> 4);
          umma_bf16_pair(d, ad + ao, bd + bo, idesc, (kb > lo || k > 0) ? 1u : 0u);
        }
        umma_commit_pair(&empty_bar[stage], 0x3);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      umma_commit_pair(&tfull[acc], 0x3);
      lo = hi;
    }
  }
  // every issued MMA must finish before TMEM and shared memory go away
  umma_commit_pair(drain_bar, 0x1);
  (void)mbar_wait(drain_bar, 0, nullptr);
}

// ------------------------------------------------------------------ epilogue
// act(x) and, for the gradient, act'(x), in fp32.
DM_DEV float act_value(int act, float x) {
  if (act == DMUON_ACT_SILU) return x * __fdividef(1.f, 1.f + __expf(-x));
  if (act == DMUON_ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678f));
  return 0.5f * x * (1.f + tanhf(0.79788456f * fmaf(0.044715f * x * x, x, x)));
}
DM_DEV void act_both(int act, float x, float& a, float& da) {
  if (act == DMUON_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-x));
    a = x * s;
    da = s * fmaf(x, 1.f - s, 1.f);
  } else if (act == DMUON_ACT_GELU) {
    const float phi = 0.5f * (1.f + erff(x * 0.70710678f));
    a = x * phi;
    da = fmaf(x * 0.39894228f, __expf(-0.5f * x * x), phi);
  } else {
    const float t = tanhf(0.79788456f * fmaf(0.044715f * x * x, x, x));
    const float half = 0.5f * (1.f + t);
    a = x * half;
    da = fmaf(0.5f * x * (1.f - t * t), 0.79788456f * fmaf(0.134145f * x, x, 1.f), half);
  }
}

// 32 values of one row, as bf16, at dst: 16-byte stores where allowed.
DM_DEV void store_row32(__nv_bfloat16* dst, int n, bool vec, const float (&v)[32]) {
  if (vec && n >= 32) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      reinterpret_cast<uint4*>(dst)[u] =
          make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                     pack_bf16x2(v[8 * u + 4], v[8 * u + 5]),
                     pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) dst[j] = __float2bfloat16_rn(v[j]);
  }
}

DM_DEV void unpack8(const uint4& q, float* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}

// One row's block of 32 values in 8 bits; values past n are not written.
DM_DEV void store_act8(signed char* codes, __nv_bfloat16* scale, int n, bool vec,
                       const float (&v)[32]) {
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < n) {
      top = fmaxf(top, fabsf(v[j]));
      finite = finite && fabsf(v[j]) <= 3.402823466e38f;
    }
  const float s = act8_scale(top, finite);
  const bool live = finite && s > 0.f;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    uint32_t p = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (live && j + k < n) p |= act8_code_f32(v[j + k], s) << (8 * k);
    }
    w[j / 4] = p;
  }
  if (vec && n >= 32) {
    reinterpret_cast<uint4*>(codes)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(codes)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) codes[j] = (signed char)(w[j / 4] >> (8 * (j & 3)));
  }
  *scale = __float2bfloat16_rn(s);
}

// 32 kept values of one row (columns c0 .. c0 + 31, n of them inside).
DM_DEV void load_kept(const LinArgs& g, const void* base, const __nv_bfloat16* scales, int row,
                      int c0, int n, float (&v)[32]) {
  if (g.keep == kKeepBf16) {
    const __nv_bfloat16* p =
        static_cast<const __nv_bfloat16*>(base) + (long long)row * g.ffn + c0;
    if (g.kept_vec && n >= 32) {
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u] = reinterpret_cast<const uint4*>(p)[u];
#pragma unroll
      for (int u = 0; u < 4; ++u) unpack8(q[u], v + 8 * u);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = j < n ? __bfloat162float(p[j]) : 0.f;
    }
  } else {
    const signed char* p = static_cast<const signed char*>(base) + (long long)row * g.ffn + c0;
    const int blocks = (g.ffn + kActBlock - 1) / kActBlock;
    const float s = __bfloat162float(scales[(long long)row * blocks + c0 / kActBlock]);
    if (g.kept_vec && n >= 32) {
      const uint4 q[2] = {reinterpret_cast<const uint4*>(p)[0],
                          reinterpret_cast<const uint4*>(p)[1]};
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = s * float((signed char)(w[j / 4] >> (8 * (j & 3))));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = j < n ? s * float(p[j]) : 0.f;
    }
  }
}

template <int EPI>
DM_DEV void epilogue(const LinArgs& g, uint32_t rank, uint64_t* tfull, uint64_t* tempty,
                     uint32_t epi_smem, uint32_t tmem_base, volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;          // TMEM lane quarter this warp may read
  const int h = (warp - 2) >> 2;   // which half of the tile's columns
  const int ew = warp - 2;
  const uint32_t buf0 = epi_smem + uint32_t(ew * 2 * kEpiBufBytes);
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
  const int clusters = int(cluster_count_x());
  const int r_loc = int(rank) * kHalf + q * 32;
  int stored = 0;  // chunks staged so far (their buffers alternate)

  // Write a 32 x 32 chunk (rows rg0.., columns c0..) of an output with m rows
  // and n columns: through shared memory by TMA, which drops what lies outside.
  auto put_raw = [&](int map, const uint32_t (&w)[16], int c0, int rg0) {
    const uint32_t buf = buf0 + uint32_t((stored++ & 1) * kEpiBufBytes);
    if (lane == 0) bulk_wait_read<1>();  // the store that last read this buffer
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      st_shared_v4(buf + epi_off(lane, u), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&g.maps[map], buf, c0, rg0);
      bulk_commit();
    }
  };
  auto put = [&](int map, const float (&o)[32], int c0, int rg0) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
    put_raw(map, w, c0, rg0);
  };

  int it = 0;
  for (int u = int(cluster_id_x()); u < g.total_units; u += clusters, ++it) {
    const Unit U = decode_unit(g, u);
    const LinProblem& P = g.prob[U.prob];
    const int acc = it & 1;
    const uint32_t aph = uint32_t(it >> 1) & 1u;
    int w = 1;
    if (lane == 0) w = mbar_wait_cluster(&tfull[acc], aph, abort_flag) ? 1 : 0;
    w = __shfl_sync(0xffffffffu, w, 0);
    if (!w) {
      if (lane == 0) raise_abort(g.err, abort_flag);
      break;
    }
    tc_fence_after();
    const uint32_t t_acc = tmem_base + uint32_t(acc * kAccCols) + (uint32_t(q * 32) << 16);
    // this warp's four accumulator chunks: first tile column of chunk k
    auto chunk_col = [&](int k) {
      return EPI == kLinGlu ? (k >> 1) * kHalf + h * 64 + (k & 1) * 32 : h * 128 + k * 32;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty + uint32_t(acc) * 8u);
    };
    const float* parts = nullptr;  // this warp's first part, when the sum comes from the workspace
    if (U.q >= 0) {
      const size_t mine = (size_t(rank) * kEpiWarps + ew) * 4096;
      float* dst = g.partial + size_t(U.q * g.split + U.part) * kPartFloats + mine;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        float v[32];
        tmem_ld32(t_acc + uint32_t(chunk_col(k)), v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) dst[(k * 32 + j) * 32 + lane] = v[j];
      }
      release();
      __threadfence();
      __syncwarp();
      int* counter = g.arrived + (U.q * 2 + int(rank)) * kEpiWarps + ew;
      int before = 0;
      if (lane == 0) before = atomicAdd(counter, 1);
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != g.split - 1) continue;
      if (lane == 0) *counter = 0;  // ready for the next launch
      __threadfence();
      parts = g.partial + size_t(U.q) * g.split * kPartFloats + mine;
    }
    auto load_acc = [&](int k, float (&v)[32]) {
      if (parts == nullptr) {
        __syncwarp();
        tmem_ld32(t_acc + uint32_t(chunk_col(k)), v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __ldcg(parts + (k * 32 + j) * 32 + lane);
        for (int p = 1; p < g.split; ++p) {
          const float* src = parts + size_t(p) * kPartFloats;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += __ldcg(src + (k * 32 + j) * 32 + lane);
        }
      }
    };
    const int rg0 = U.ti * kTile + r_loc;
    const int r = rg0 + lane;

    if constexpr (EPI == kLinStore) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int c0 = U.tj * kTile + chunk_col(k);
        if (c0 >= P.n) break;
        float v[32];
        load_acc(k, v);
        if (g.sum != nullptr) {
          float* sp = g.sum + (long long)r * P.n + c0;
          const bool vec = (P.n & 3) == 0 && c0 + 32 <= P.n;
          if (g.sum_read && r < P.m) {
            if (vec) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(sp + j);
                v[j] += f.x; v[j + 1] += f.y; v[j + 2] += f.z; v[j + 3] += f.w;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c0 + j < P.n) v[j] += sp[j];
            }
          }
          if (g.sum_write) {
            if (r < P.m) {
              if (vec) {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                  *reinterpret_cast<float4*>(sp + j) =
                      make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (c0 + j < P.n) sp[j] = v[j];
              }
            }
            continue;
          }
        }
        if (g.scale != nullptr) {
          const float f = *g.scale;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= f;
        }
        if (P.c_map >= 0) put(P.c_map, v, c0, rg0);
        else if (r < P.m) store_row32(P.c + (long long)r * P.c_ld + c0, P.n - c0, false, v);
      }
    } else if constexpr (EPI == kLinGlu) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int c0 = U.tj * kHalf + chunk_col(k);
        if (c0 >= P.n) break;
        float a[32], b[32];
        load_acc(k, a);
        load_acc(k + 2, b);
        if (g.keep == kKeepBf16) {
          if (g.kept_vec) {
            put(g.map_gate, a, c0, rg0);
            put(g.map_up, b, c0, rg0);
          } else if (r < P.m) {
            const long long at = (long long)r * g.ffn + c0;
            store_row32(static_cast<__nv_bfloat16*>(g.gate) + at, P.n - c0, false, a);
            store_row32(static_cast<__nv_bfloat16*>(g.up) + at, P.n - c0, false, b);
          }
        } else if (g.keep == kKeepAct8 && r < P.m) {
          const long long at = (long long)r * g.ffn + c0;
          const long long sa =
              (long long)r * ((g.ffn + kActBlock - 1) / kActBlock) + c0 / kActBlock;
          store_act8(static_cast<signed char*>(g.gate) + at, g.gate_scale + sa, P.n - c0,
                     g.kept_vec != 0, a);
          store_act8(static_cast<signed char*>(g.up) + at, g.up_scale + sa, P.n - c0,
                     g.kept_vec != 0, b);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = act_value(g.act, a[j]) * b[j];
        put(P.c_map, a, c0, rg0);
      }
    } else if constexpr (EPI == kLinGluGrad) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int c0 = U.tj * kTile + chunk_col(k);
        if (c0 >= P.n) break;
        float v[32], ga[32], up[32];
        if (r < P.m) {
          load_kept(g, g.gate, g.gate_scale, r, c0, P.n - c0, ga);
          load_kept(g, g.up, g.up_scale, r, c0, P.n - c0, up);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ga[j] = up[j] = 0.f;
        }
        load_acc(k, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float a, da;
          act_both(g.act, ga[j], a, da);
          const float dh = v[j];
          ga[j] = dh * up[j] * da;  // dgate
          up[j] *= a;               // h
          v[j] = dh * a;            // dup
        }
        put(P.c_map, ga, c0, rg0);
        put(g.map_dup, v, c0, rg0);
        put(g.map_h, up, c0, rg0);
      }
    }
    if (parts == nullptr) release();
  }
  // stores complete, and stop reading shared memory, before the CTA exits
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

// Logits of 32 tokens x 128 vocabulary entries per warp, in registers.
DM_DEV void epilogue_xent(const LinArgs& g, uint32_t rank, uint64_t* tfull, uint64_t* tempty,
                          uint32_t epi_smem, uint32_t tmem_base, volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, h = (warp - 2) >> 2, ew = warp - 2;
  const uint32_t buf0 = epi_smem + uint32_t(ew * 2 * kEpiBufBytes);
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
  const int clusters = int(cluster_count_x());
  const LinProblem& P = g.prob[0];
  int it = 0;
  bool ok = true;
  for (int u = int(cluster_id_x()); ok && u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    const int rg0 = U.ti * kTile + int(rank) * kHalf + q * 32;
    const int r = rg0 + lane;
    const int g0 = U.tj * kTile + h * kXentGroup;  // first vocabulary entry of the group
    float z[kXentGroup];
#pragma unroll
    for (int j = 0; j < kXentGroup; ++j) z[j] = 0.f;
#pragma unroll 1
    for (int lo = U.kb_lo; lo < U.kb_hi; lo += kRun, ++it) {
      const int acc = it & 1;
      int w = 1;
      if (lane == 0) w = mbar_wait_cluster(&tfull[acc], uint32_t(it >> 1) & 1u, abort_flag) ? 1 : 0;
      w = __shfl_sync(0xffffffffu, w, 0);
      if (!w) {
        if (lane == 0) raise_abort(g.err, abort_flag);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t = tmem_base + uint32_t(acc * kAccCols + h * kXentGroup) +
                         (uint32_t(q * 32) << 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v[16];
        tmem_ld16(t + uint32_t(k * 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) z[k * 16 + j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty + uint32_t(acc) * 8u);
    }
    if (!ok || g0 >= P.n) continue;
    const int n = P.n - g0;  // entries of the group that exist, if below 128
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kXentGroup; ++j)
      if (j < n) m = fmaxf(m, z[j]);
    const long long t = r < P.m ? g.target[r] : -1;
    const int d = t >= g0 && t < g0 + kXentGroup && t < P.n ? int(t - g0) : -1;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int j = k * 32; j < k * 32 + 32; ++j) {
        if (j == d) g.target_logit[r] = z[j];
        z[j] = j < n ? exp2f((z[j] - m) * 1.44269504f) : 0.f;
        s += z[j];
      }
      if (P.c_map >= 0 && k * 32 < n) {
        const uint32_t buf = buf0 + uint32_t((k & 1) * kEpiBufBytes);
        if (lane == 0) bulk_wait_read<1>();  // the store that last read this buffer
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 p = __floats2half2_rn(z[k * 32 + 8 * i + 2 * j], z[k * 32 + 8 * i + 2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t*>(&p);
          }
          st_shared_v4(buf + epi_off(lane, i), o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&g.maps[P.c_map], buf, g0 + k * 32, rg0);
          bulk_commit();
        }
      }
    }
    if (r < P.m) g.group_stat[(long long)(g0 / kXentGroup) * g.stat_ld + r] = make_float2(m, s);
  }
  // stores complete, and stop reading shared memory, before the CTA exits
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1) pair_gemm_kernel(const __grid_constant__ LinArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kOpBytes;
  uint8_t* sE = sB + kStages * kOpBytes;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(sE + kEpiBytes);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* tfull = empty_bar + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain_bar = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);    // leader: its expect_tx; both CTAs' copies add bytes
      mbar_init(&empty_bar[s], 1);   // the leader's commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);               // the leader's commit
      mbar_init(&tempty[a], 2 * kEpiWarps);  // leader: every epilogue warp of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (threadIdx.x == 0) {
    producer<EPI, A_MN, B_MN>(g, rank, sA, sB, full_bar, empty_bar, abort_flag);
  } else if (threadIdx.x == 32) {
    if (rank == 0)
      mma_issuer<EPI, A_MN, B_MN>(g, sA, sB, full_bar, empty_bar, tfull, tempty, drain_bar,
                                  tmem_base, abort_flag);
  } else if (warp >= 2) {
    if constexpr (EPI == kLinXent)
      epilogue_xent(g, rank, tfull, tempty, smem_u32(sE), tmem_base, abort_flag);
    else
      epilogue<EPI>(g, rank, tfull, tempty, smem_u32(sE), tmem_base, abort_flag);
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag != 0) {
    const long long t0 = clock64();
    while (clock64() - t0 < kAbortSettleCycles) {
    }
  }
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

using Kernel = void (*)(LinArgs);
Kernel kernel_for(int epi, bool a_mn, bool b_mn) {
  switch (epi) {
    case kLinGlu: return !a_mn && !b_mn ? pair_gemm_kernel<kLinGlu, false, false> : nullptr;
    case kLinGluGrad: return !a_mn && b_mn ? pair_gemm_kernel<kLinGluGrad, false, true> : nullptr;
    case kLinXent: return !a_mn && !b_mn ? pair_gemm_kernel<kLinXent, false, false> : nullptr;
    case kLinStore:
      if (!a_mn) return b_mn ? pair_gemm_kernel<kLinStore, false, true>
                             : pair_gemm_kernel<kLinStore, false, false>;
      return b_mn ? pair_gemm_kernel<kLinStore, true, true> : nullptr;
    default: return nullptr;
  }
}

}  // namespace

size_t lin_partial_bytes() { return kMaxParts * kPartFloats * sizeof(float); }
size_t lin_arrived_bytes() { return kMaxParts * 2 * kEpiWarps * sizeof(int); }

cudaError_t lin_prepare() {
  const struct { int epi; bool a, b; } all[] = {
      {kLinGlu, false, false},   {kLinGluGrad, false, true}, {kLinXent, false, false},
      {kLinStore, false, false}, {kLinStore, false, true},   {kLinStore, true, true}};
  for (const auto& k : all) {
    const cudaError_t e = cudaFuncSetAttribute(kernel_for(k.epi, k.a, k.b),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(kSmemBytes));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

void lin_schedule(LinArgs& g, bool may_split, int clusters) {
  int tiles = 0, kb = 0;
  for (int p = 0; p < g.n_prob; ++p) {
    g.prob[p].tile_begin = tiles;
    tiles += g.prob[p].tiles_m * g.prob[p].tiles_n;
    const int k = g.prob[p].kb0 + g.prob[p].kb1;
    kb = p == 0 || k < kb ? k : kb;
  }
  g.full_tiles = g.total_units = tiles;
  g.split = 1;
  const int rest = tiles % clusters;
  if (!may_split || rest == 0) return;
  // Time of the last wave in K blocks (about 0.55 us each): a part costs its
  // blocks plus about 4 for filling the pipeline and writing its accumulator,
  // and the warp that joins S parts reads them at about 2 blocks each.
  long long best = kb;
  for (int s = 2; s * rest <= kMaxParts && 2 * s <= kb; ++s) {
    const long long waves = ((long long)rest * s + clusters - 1) / clusters;
    const long long cost = waves * ((kb + s - 1) / s + 4) + 2 * s;
    if (cost < best) {
      best = cost;
      g.split = s;
    }
  }
  if (g.split > 1) {
    g.full_tiles = tiles - rest;
    g.total_units = g.full_tiles + rest * g.split;
  }
}

cudaError_t launch_lin(const LinArgs& g, int epi, bool a_mn, bool b_mn, int max_clusters,
                       cudaStream_t s) {
  if (g.total_units <= 0) return cudaSuccess;
  const Kernel k = kernel_for(epi, a_mn, b_mn);
  if (k == nullptr) return cudaErrorInvalidValue;
  const int clusters = g.total_units < max_clusters ? g.total_units : max_clusters;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(2 * clusters), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return counted(cudaLaunchKernelEx(&cfg, k, g));
}

}  // namespace dm
