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
//                exp(z - m) without the target, and kXentScale exp(z - m) itself
//                in fp16 when gradients are wanted
// Each operand is K-major (rows of K) or MN-major (rows of M or N), a template
// parameter, so no operand is ever transposed in memory.
//
// Two orientations (template parameter SWAP).  Plainly, the tokens are M and a
// tile holds 256 of them.  Swapped, the weight's rows are M and the tokens are N,
// and a tile holds `nt` tokens, a multiple of 32 chosen to fit: with few tokens the
// launch streams the weights at the memory's rate instead of multiplying padding
// (a stage is then 16 KB of weights and nt/2 token rows, and up to ten fit), and a
// ragged count wastes less of its last tile.  The accumulator's lanes are then
// the weight's rows; each 32 x 32 chunk is turned in shared memory, and from there
// on both orientations share the epilogue code: a lane holds one token.
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
// wave; the parts' fp32 accumulators go to the workspace, and a second, fully
// parallel launch adds them in order and runs the epilogue on the sums.  (Letting
// the last arriving CTA of a tile do that in the first launch serialises the reads:
// dx of 301 tokens, 1536/8960, took 46 us that way and takes 22 + 4 this way.)
//
// Measured alone on one GB300 (2070 MHz, before the power cap bites): gate and up of
// 8192 tokens, 4096/14336, 0.99 ms (1.94 PFLOP/s; cuBLAS's best product 1.90), the
// down projection 0.50 ms; sustained, the backward's products run at 1.70 to 1.76
// PFLOP/s (cuBLAS sustained 1.73).
#include "act.cuh"
#include "act8.cuh"
#include "dmuon.h"
#include "epi.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "shift.cuh"
#include "train.h"

#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dm {
namespace {

constexpr int kTile = 256;                 // tile rows and columns (CTA pair)
constexpr int kHalf = 128;                 // one CTA's rows of A / columns of B
constexpr int kMaxStages = 10;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kAccCols = 256;
constexpr int kBarBytes = 512;
// Stages and, for each epilogue warp, 4 KB in which chunks are turned or wait to be
// stored; kLinGluGrad takes 32 KB less of stages and gives each warp another 4 KB, for
// the gate's and up's chunks on their way in.
__host__ __device__ constexpr int stage_area(int epi) { return (epi == kLinGluGrad ? 160 : 192) << 10; }
__host__ __device__ constexpr int warp_bytes(int epi) { return epi == kLinGluGrad ? 8192 : 4096; }
constexpr size_t kSmemBytes = size_t(224 << 10) + 1024 + kBarBytes;
static_assert(stage_area(kLinStore) + kEpiWarps * warp_bytes(kLinStore) == 224 << 10 &&
                  stage_area(kLinGluGrad) + kEpiWarps * warp_bytes(kLinGluGrad) == 224 << 10,
              "shared memory layout");
static_assert(kSmemBytes <= 232448, "dynamic shared memory above the per-block limit");
static_assert((2 * kMaxStages + 4 + 1 + 8) * 8 + 8 <= kBarBytes, "barrier area too small");

// Tiles of a product are walked in strips of kStrip tile rows, columns outer,
// rows inner: the pairs then work on about 8 row panels and 9 column panels at
// a time, close to the fewest panels that 76 tiles can share.
constexpr int kStrip = 8;

// The tensor core's accumulation rounds toward zero, so a sum of K terms of one sign
// comes out short: of 2^20, 3.1e-3 to 5.4e-3 of the sum were missing, which is K * 2^-28.4
// to K * 2^-27.5.  Below K = 2^18 that is at most a third of rounding an output to bf16
// (longer sums are cut, train_api.cu), but not for the fp32 losses: the logits are
// accumulated in runs of
// 512 K-elements, each drained and added in registers, rounded to nearest (error of
// 777 tokens' losses against 64 bits 2.7e-6 without, 3.6e-7 with, and 1.0e-7 with the
// target's logit, a sum of one sign, summed apart in xent_rows_kernel; fp32 products on
// the CUDA cores 6e-7).  The drains hide behind the next run's MMAs: 1% of the time.
constexpr int kRunElems = 512;

// Workspace of the split parts.
constexpr size_t kPartialBytes = size_t(40) << 20;

// A stage: K-elements, this CTA's 128 rows of A and its half of B's columns (128,
// or nt/2 tokens).  Plainly 128 K-elements, which halves the barrier round trips;
// swapped, where the bytes in flight bound the rate at which weights stream, 64, so
// that a smaller part of the stages is being consumed (and for kLinGluGrad, whose
// stages have 160 KB).
template <int EPI, bool SWAP>
struct Stage {
  static constexpr int k = lin_stage_k(EPI, SWAP);
  static constexpr int a_bytes = kHalf * k * 2;
  static constexpr int panels = k / 64;  // spans of a 128-byte swizzled row
  static DM_DEV int b_rows(const LinArgs& g) { return SWAP ? g.nt / 2 : kHalf; }
  static DM_DEV int bytes(const LinArgs& g) { return a_bytes + b_rows(g) * k * 2; }
  static DM_DEV int count(const LinArgs& g) {
    return SWAP ? g.stages : stage_area(EPI) / (2 * a_bytes);
  }
};

struct Unit {
  int prob, ti, tj;
  int kb_lo, kb_hi;  // K blocks of this unit
  int q, part;       // split tile (0-based) and part; q < 0: a whole tile
};

// n / d with d's magic number (lin_magic), n < 2^31: the epilogue decodes a tile per
// few thousand cycles, and hardware division would take a third of that.
DM_DEV int divide(int n, int d, unsigned magic) {
  int q = int(__umulhi(unsigned(n), magic));
  const int r = n - q * d;
  if (r < 0) --q;
  else if (r >= d) ++q;
  return q;
}

DM_DEV Unit decode_unit(const LinArgs& g, int u) {
  Unit U;
  int t = u;
  U.q = -1;
  U.part = 0;
  if (u >= g.full_tiles) {
    const int r = u - g.full_tiles;
    U.q = divide(r, g.split, g.split_magic);
    U.part = r - U.q * g.split;
    t = g.full_tiles + U.q;
  }
  int p = 0;
  while (p + 1 < g.n_prob && t >= g.prob[p + 1].tile_begin) ++p;
  const LinProblem& P = g.prob[p];
  U.prob = p;
  const int local = t - P.tile_begin;
  const int per = kStrip * P.tiles_n;
  const int strip = divide(local, per, P.strip_magic);
  const int r = local - strip * per;
  const int rows = min(kStrip, P.tiles_m - strip * kStrip);
  U.tj = rows == kStrip ? r / kStrip : divide(r, rows, P.last_magic);
  U.ti = strip * kStrip + (r - U.tj * rows);
  const int kb = P.kb0 + P.kb1;
  U.kb_lo = 0;
  U.kb_hi = kb;
  if (U.q >= 0) {
    U.kb_lo = divide(kb * U.part, g.split, g.split_magic);
    U.kb_hi = divide(kb * (U.part + 1), g.split, g.split_magic);
  }
  return U;
}

// ------------------------------------------------------------------ roles
template <int EPI, bool A_MN, bool B_MN, bool SWAP>
DM_DEV void producer(const LinArgs& g, uint32_t rank, uint8_t* sStage, uint64_t* full_bar,
                     uint64_t* empty_bar, volatile int* abort_flag) {
  const uint32_t leader_full = mapa_shared(smem_u32(full_bar), 0);
  const int clusters = int(cluster_count_x());
  using St = Stage<EPI, SWAP>;
  const int stages = St::count(g), bytes = St::bytes(g), brows = St::b_rows(g);
  constexpr int a_box = St::k * 128;  // 64 MN-elements of k rows, or (two panels) 128 rows
  int stage = 0;
  uint32_t phase = 0;
  bool started = false;
  for (int u = int(cluster_id_x()); u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    const LinProblem& P = g.prob[U.prob];
    // kLinGlu: a plain tile's B half is the gate's (first CTA) or the up's rows; a
    // swapped tile's A share is 64 rows of each
    const int row0 = SWAP && EPI == kLinGlu ? U.ti * kHalf + int(rank) * 64
                                            : U.ti * kTile + int(rank) * kHalf;
    const int col0 = SWAP ? U.tj * g.nt + int(rank) * brows
                          : (EPI == kLinGlu ? U.tj * kHalf : U.tj * kTile + int(rank) * kHalf);
    // A's or B's share of K block kb into stage s; rows, columns and K past the tensors'
    // ends read as zeros
    auto load = [&](int kb, int s, bool a_too, bool b_too) {
      const bool second = EPI != kLinGlu && kb >= P.kb0;
      const bool tail = A_MN && B_MN && kb == P.kb0 - 1;
      const CUtensorMap* mapA = &g.maps[second || tail ? P.a1 : P.a0];
      const CUtensorMap* mapB = &g.maps[EPI == kLinGlu && !SWAP ? (rank == 0 ? P.b0 : P.b1)
                                                                : (second || tail ? P.b1 : P.b0)];
      const int k0 = (second ? kb - P.kb0 : kb) * St::k;
      const uint32_t bar = leader_full + uint32_t(s) * 8u;
      uint8_t* a = sStage + s * bytes;
      uint8_t* b = a + St::a_bytes;
      if (A_MN && a_too) {
        tma_load_2d_pair(a, mapA, bar, row0, k0);
        tma_load_2d_pair(a + a_box, mapA, bar, row0 + 64, k0);
      }
      if (B_MN && b_too) {
        tma_load_2d_pair(b, mapB, bar, col0, k0);
        tma_load_2d_pair(b + a_box, mapB, bar, col0 + 64, k0);
      }
#pragma unroll
      for (int h = 0; h < St::panels; ++h) {
        if (!A_MN && a_too) {
          if (SWAP && EPI == kLinGlu) {
            tma_load_2d_pair(a + h * 16384, &g.maps[P.a0], bar, k0 + h * 64, row0);
            tma_load_2d_pair(a + h * 16384 + 8192, &g.maps[P.a1], bar, k0 + h * 64, row0);
          } else {
            tma_load_2d_pair(a + h * 16384, mapA, bar, k0 + h * 64, row0);
          }
        }
        if (!B_MN && b_too) tma_load_2d_pair(b + h * brows * 128, mapB, bar, k0 + h * 64, col0);
      }
    };
    auto expect = [&](int kb, int s) {
      if (rank == 0)
        mbar_arrive_expect_tx(&full_bar[s], uint32_t(A_MN && B_MN && kb == P.kb0 - 1
                                                         ? 8 * 128 * g.k_tail
                                                         : 2 * bytes));
    };
    int kb = U.kb_lo;
    if (!(A_MN && B_MN) && !started) {
      // the weights of the first stages, then what the launch before may still write
      started = true;
      const int n = g.early == kEarlyWeights ? min(stages, U.kb_hi - U.kb_lo) : 0;
      for (int s = 0; s < n; ++s) {
        expect(kb + s, s);
        load(kb + s, s, SWAP, !SWAP);
      }
      grid_wait();
      for (int s = 0; s < n; ++s) load(kb + s, s, !SWAP, SWAP);
      kb += n;
      if (n == stages) phase = 1;
      else stage = n;
    }
    for (; kb < U.kb_hi; ++kb) {
      if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) {
        raise_abort(g.err, abort_flag);
        return;
      }
      expect(kb, stage);
      load(kb, stage, true, true);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

template <int EPI, bool A_MN, bool B_MN, bool SWAP>
DM_DEV void mma_issuer(const LinArgs& g, uint8_t* sStage, uint64_t* full_bar, uint64_t* empty_bar,
                       uint64_t* tfull, uint64_t* tempty, uint64_t* drain_bar, uint32_t tmem_base,
                       volatile int* abort_flag) {
  const uint32_t idesc = idesc_bf16(kTile, SWAP ? g.nt : kTile, A_MN, B_MN);
  // K-major: 64-element panels, 32 bytes per K step inside a 128-byte row, 8-row
  // groups 1 KB apart.  MN-major: 64-element atoms of the stage's K rows apart (LBO),
  // 8-row K groups 1 KB apart (SBO), 2 KB per K step.  Shared-memory addresses stay
  // below 256 KB, so adding to the start-address field never carries out of it.
  using St = Stage<EPI, SWAP>;
  constexpr int atom = St::k * 128;
  const uint64_t a_desc = sdesc_sw128(smem_u32(sStage), A_MN ? atom : 16, 1024);
  const uint64_t b_desc = sdesc_sw128(smem_u32(sStage) + St::a_bytes, B_MN ? atom : 16, 1024);
  const uint32_t step = uint32_t(St::bytes(g)) >> 4;
  const uint32_t b_panel = uint32_t(St::b_rows(g)) * 128u >> 4;
  const int stages = St::count(g);
  const int clusters = int(cluster_count_x());
  int stage = 0;
  uint32_t phase = 0;
  int it = 0;  // accumulators handed to the epilogue so far
  bool ok = true;
  for (int u = int(cluster_id_x()); ok && u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    const int last = g.prob[U.prob].kb0 - 1;
    for (int lo = U.kb_lo; ok && lo < U.kb_hi; ++it) {
      const int hi = EPI == kLinXent ? min(lo + kRunElems / St::k, U.kb_hi) : U.kb_hi;
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
        const uint64_t ad = a_desc + uint64_t(uint32_t(stage) * step);
        const uint64_t bd = b_desc + uint64_t(uint32_t(stage) * step);
        const int k_rows = A_MN && B_MN && kb == last ? g.k_tail : St::k;
#pragma unroll
        for (int k = 0; k < St::k / 16; ++k) {
          if (A_MN && B_MN && k * 16 >= k_rows) break;
          const uint64_t ao = A_MN
                                  ? uint64_t(k) * (2048u >> 4)
                                  : uint64_t(k >> 2) * (16384u >> 4) + uint64_t(k & 3) * (32u >> 4);
          const uint64_t bo = B_MN ? uint64_t(k) * (2048u >> 4)
                                   : uint64_t(uint32_t(k >> 2) * b_panel) + uint64_t(k & 3) * (32u >> 4);
          umma_bf16_pair(d, ad + ao, bd + bo, idesc, (kb > lo || k > 0) ? 1u : 0u);
        }
        umma_commit_pair(&empty_bar[stage], 0x3);
        if (++stage == stages) {
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
// a <- act(a) * b
template <int ACT>
DM_DEV void glu32(float (&a)[32], const float (&b)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) a[j] = act_value<ACT>(a[j]) * b[j];
}
// From dh, gate and up: v <- dup, ga <- dgate, up <- h
template <int ACT>
DM_DEV void glu_grad16(float* v, float (&ga)[16], float (&up)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float a, da;
    act_both<ACT>(ga[j], a, da);
    const float dh = v[j];
    ga[j] = dh * up[j] * da;
    up[j] *= a;
    v[j] = dh * a;
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

// One row's block of 32 fp32 values in 8 bits; values past n count as zeros.  The
// quotient is taken with the scale's rounded reciprocal: within 2e-5 of a step, far
// below what the accumulation of the values leaves uncertain.
DM_DEV float act8_block(float (&v)[32], int n, uint32_t (&w)[8]) {
  if (n < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j >= n) v[j] = 0.f;
  }
  float top = 0.f, bad = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    top = fmaxf(top, fabsf(v[j]));
    bad = fmaf(v[j], 0.f, bad);  // NaN once a value is not finite
  }
  const float s = act8_scale(top, bad == 0.f);
  const float r = bad == 0.f && s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = act8_code_fast(bad == 0.f ? v[4 * j + k] : 0.f, r);
    w[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
  return s;
}

// 32 kept values of one row (columns c0 .. c0 + 31, n of them inside), as stored.
struct Kept {
  uint4 q[4];
  float scale;
};
// From rows that are not 16-byte aligned.  `inner`: neither the first nor the last row,
// so that the aligned words around a whole piece of it lie inside the tensor.
DM_DEV void fetch_kept(const LinArgs& g, const void* base, const __nv_bfloat16* scales, int row,
                       int c0, int n, bool inner, Kept& k) {
  const long long at = (long long)row * g.ffn + c0;
  if (g.keep == kKeepBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (inner && n >= 32) {
      load_shifted<4>(p, k.q);
      return;
    }
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = (2 * j < n ? uint32_t(p[2 * j]) : 0u) |
             (2 * j + 1 < n ? uint32_t(p[2 * j + 1]) << 16 : 0u);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      k.q[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at;
    const int blocks = (g.ffn + kActBlock - 1) / kActBlock;
    k.scale = __bfloat162float(scales[(long long)row * blocks + c0 / kActBlock]);
    if (inner && n >= 32) {
      uint4 t[2];
      load_shifted<2>(p, t);
      k.q[0] = t[0];
      k.q[1] = t[1];
      return;
    }
    uint32_t w[8] = {};
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) w[j / 4] |= uint32_t(p[j]) << (8 * (j & 3));
    k.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    k.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
DM_DEV void kept_values(const LinArgs& g, const Kept& k, int half, float (&v)[16]) {
  if (g.keep == kKeepBf16) {
    unpack8(k.q[2 * half], v);
    unpack8(k.q[2 * half + 1], v + 8);
  } else {
    const uint32_t w[4] = {k.q[half].x, k.q[half].y, k.q[half].z, k.q[half].w};
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = k.scale * act8_int(w[j / 4], j & 3);
  }
}

// A 32 x 32 fp32 chunk in a warp's 4 KB of shared memory, turned: lane i writes
// element j of its row to word (j, i ^ j), lane j reads back (j, i ^ j) for every
// i.  Both touch 32 banks per instruction.
DM_DEV void turn_write(float* buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) buf[j * 32 + (lane ^ j)] = v[j];
}
DM_DEV void turn_read(const float* buf, int lane, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = buf[lane * 32 + (i ^ lane)];
}

// A swapped kLinGlu chunk has gate in the TMEM lanes of one warp and up in those of
// another, which hands its part over: `ready` and `taken` are mbarriers that one
// lane of the giving and of the receiving warp arrives on.
struct Handover {
  uint64_t *ready, *taken;
  uint32_t parity;
};

// Where an epilogue warp's 32 x 32 chunks lie.  Chunk k (0..3) sits at the
// accumulator's columns 32 col(k).. and the warp's quarter of the TMEM lanes; it holds
// the output's rows row(k).. and columns c(k)...
template <int EPI, bool SWAP>
struct Chunks {
  const LinArgs& g;
  const LinProblem& P;
  int ti, tj, rank, q, h, chunks;
  DM_DEV Chunks(const LinArgs& g_, const Unit& U, int rank_, int q_, int h_)
      : g(g_), P(g_.prob[U.prob]), ti(U.ti), tj(U.tj), rank(rank_), q(q_), h(h_),
        chunks(SWAP ? g_.nt / 32 : kAccCols / 32) {}
  DM_DEV int col(int k) const {
    if (SWAP) return 2 * k + h;
    return EPI == kLinGlu ? (k >> 1) * 4 + h * 2 + (k & 1) : h * 4 + k;
  }
  DM_DEV int row(int k) const {
    return SWAP ? tj * g.nt + col(k) * 32 : ti * kTile + rank * kHalf + q * 32;
  }
  DM_DEV int c(int k) const {
    if (SWAP)
      return EPI == kLinGlu ? ti * kHalf + rank * 64 + (q & 1) * 32
                            : ti * kTile + rank * kHalf + q * 32;
    return EPI == kLinGlu ? tj * kHalf + h * 64 + (k & 1) * 32 : tj * kTile + (h * 4 + k) * 32;
  }
  static constexpr int count = EPI == kLinGlu && !SWAP ? 2 : 4;  // chunks to write (if inside)
  DM_DEV bool inside(int k) const {
    return k < count && col(k) < chunks && row(k) < P.rows && c(k) < P.cols;
  }
};

// A split tile's part: the raw accumulator, for the joining launch.
template <int EPI, bool SWAP>
DM_DEV void store_part(const Chunks<EPI, SWAP>& G, const Unit& U, uint32_t t_acc, int lane) {
  float* dst = G.g.partial +
               size_t(U.q * G.g.split + U.part) * (size_t(G.chunks) * 32 * kTile) + lane;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int col = G.col(k);
    if (col >= G.chunks) break;
    float v[32];
    __syncwarp();
    tmem_ld32(t_acc + uint32_t(col * 32), v);
    tmem_ld_wait();
    float* p = dst + ((size_t(G.rank) * G.chunks + col) * 4 + G.q) * 1024;
#pragma unroll
    for (int j = 0; j < 32; ++j) p[j * 32] = v[j];
  }
}

template <int EPI, bool SWAP>
DM_DEV void epilogue(const LinArgs& g, uint32_t rank, uint64_t* tfull, uint64_t* tempty,
                     uint8_t* epi, uint64_t* pair_bar, uint32_t tmem_base,
                     volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;          // TMEM lane quarter this warp may read
  const int h = (warp - 2) >> 2;   // which half of the tile's columns (swapped: of its chunks)
  const int ew = warp - 2;
  // two 2 KB chunks to be stored; swapped, also the 4 KB in which a chunk is turned
  float* turn = reinterpret_cast<float*>(epi + ew * warp_bytes(kLinStore));
  const uint32_t buf0 = smem_u32(turn);
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
  const int clusters = int(cluster_count_x());
  int stored = 0;  // chunks staged so far (their buffers alternate)
  const int pair = h * 2 + (q & 1);
  Handover ho{pair_bar + 2 * pair, pair_bar + 2 * pair + 1, 0u};
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    int w = 1;
    if (lane == 0) {
      w = mbar_wait(bar, parity, abort_flag) ? 1 : 0;
      if (!w) raise_abort(g.err, abort_flag);
    }
    return __shfl_sync(0xffffffffu, w, 0) != 0;
  };
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  // kLinStore, plain: 32 x 64 chunks in the warp's 4 KB (128-byte rows: half the TMA
  // requests of 32 x 32 ones)
  auto put_wide = [&](int map, const uint32_t (&w)[32], int c0, int rg0) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u)
      st_shared_v4(buf0 + uint32_t(lane * 128 + ((u ^ (lane & 7)) << 4)), w[4 * u], w[4 * u + 1],
                   w[4 * u + 2], w[4 * u + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&g.maps[map], buf0, c0, rg0);
      bulk_commit();
    }
  };

  // Write a 32 x 32 chunk (rows rg0.., columns c0..) of an output through shared
  // memory by TMA, which drops what lies outside.
  auto put_packed = [&](int map, const uint32_t (&w)[16], int c0, int rg0) {
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
  // Where rows are not 16-byte aligned TMA cannot write them: the chunk still goes
  // through shared memory, and the warp writes it row by row, 64 bytes at a time.
  auto put_plain = [&](__nv_bfloat16* dst, long long ld, const float (&o)[32], int c0, int rg0,
                       int rows, int n) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
    epi_store_row(buf0, lane, o);
    __syncwarp();
    const int last = min(32, rows - rg0);
    dst += (long long)rg0 * ld + c0 + lane;
    if (lane < n)
      for (int i = 0; i < last; ++i)
        reinterpret_cast<uint16_t*>(dst)[i * ld] = ld_shared_b16(
            buf0 + epi_off(i, lane >> 3) + uint32_t((lane & 7) * 2));
    __syncwarp();
  };
  auto put = [&](int map, const float (&o)[32], int c0, int rg0) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
    put_packed(map, w, c0, rg0);
  };
  // and one in 8 bits: the codes by TMA too (32-byte rows; written by the lanes, they
  // would be 64 scattered pieces), the scales as they are
  auto put_act8 = [&](int map, void* codes, __nv_bfloat16* scales, float (&o)[32], int c0, int rg0,
                      int n, bool in) {
    uint32_t w[8];
    const float s = act8_block(o, n, w);
    const long long row = rg0 + lane;
    if (in)
      scales[row * ((g.ffn + kActBlock - 1) / kActBlock) + c0 / kActBlock] = __float2bfloat16_rn(s);
    if (g.kept_vec) {
      const uint32_t buf = buf0 + uint32_t((stored++ & 1) * kEpiBufBytes);
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
      st_shared_v4(buf + uint32_t(lane * 32), w[0], w[1], w[2], w[3]);
      st_shared_v4(buf + uint32_t(lane * 32 + 16), w[4], w[5], w[6], w[7]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&g.maps[map], buf, c0, rg0);
        bulk_commit();
      }
    } else {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      st_shared_v4(buf0 + uint32_t(lane * 32), w[0], w[1], w[2], w[3]);
      st_shared_v4(buf0 + uint32_t(lane * 32 + 16), w[4], w[5], w[6], w[7]);
      __syncwarp();
      const unsigned rows = __popc(__ballot_sync(0xffffffffu, in));
      signed char* dst = static_cast<signed char*>(codes) + (long long)rg0 * g.ffn + c0 + lane;
      const signed char* src = reinterpret_cast<const signed char*>(turn) + lane;
      if (lane < n)
        for (unsigned i = 0; i < rows; ++i) dst[(long long)i * g.ffn] = src[i * 32];
      __syncwarp();
    }
  };

  int it = 0;
  for (int u = int(cluster_id_x()); u < g.total_units; u += clusters, ++it) {
    const Unit U = decode_unit(g, u);
    const LinProblem& P = g.prob[U.prob];
    const int acc = it & 1;
    const uint32_t aph = uint32_t(it >> 1) & 1u;
    const Chunks<EPI, SWAP> G(g, U, int(rank), q, h);
    int w = 1;
    if (lane == 0) w = mbar_wait_cluster(&tfull[acc], aph, abort_flag) ? 1 : 0;
    w = __shfl_sync(0xffffffffu, w, 0);
    if (!w) {
      if (lane == 0) raise_abort(g.err, abort_flag);
      break;
    }
    tc_fence_after();
    const uint32_t t_acc = tmem_base + uint32_t(acc * kAccCols) + (uint32_t(q * 32) << 16);
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_tempty + uint32_t(acc) * 8u);
    };
    if (U.q >= 0) {
      store_part(G, U, t_acc, lane);
      release();
      continue;
    }
    // accumulator chunk k with the TMEM's lanes: a lane holds a row of the tile
    auto load_raw = [&](int k, float (&v)[32]) {
      __syncwarp();
      tmem_ld32(t_acc + uint32_t(G.col(k) * 32), v);
      tmem_ld_wait();
    };
    // and with one output row per lane
    auto load_acc = [&](int k, float (&v)[32]) {
      load_raw(k, v);
      if (SWAP) {
        if (lane == 0) bulk_wait_read<0>();  // no store still reads the buffer
        __syncwarp();
        turn_write(turn, lane, v);
        __syncwarp();
        turn_read(turn, lane, v);
        __syncwarp();
      }
    };

    if constexpr (EPI == kLinStore && !SWAP) {
      if (g.sum == nullptr && P.c_map >= 0) {
        const float f = g.scale != nullptr ? *g.scale : 1.f;
        const bool second = G.inside(2);
#pragma unroll 1
        for (int k = 0; k < 4; k += 2) {
          if (!G.inside(k)) break;
          uint32_t w[32];
          __syncwarp();
          float v0[32], v1[32];
          tmem_ld32(t_acc + uint32_t(G.col(k) * 32), v0);
          tmem_ld32(t_acc + uint32_t(G.col(k) * 32 + 32), v1);
          tmem_ld_wait();
          // the accumulator is free as soon as it is in registers
          if (k == 2 || !second) release();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            w[j] = pack_bf16x2(v0[2 * j] * f, v0[2 * j + 1] * f);
            w[16 + j] = pack_bf16x2(v1[2 * j] * f, v1[2 * j + 1] * f);
          }
          put_wide(P.c_map, w, G.c(k), G.row(k));
        }
        if (!G.inside(0)) release();
        continue;
      }
    }
    bool dead = false;
#pragma unroll 1
    for (int k = 0; k < G.count; ++k) {
      if (!G.inside(k)) break;
      const int c0 = G.c(k), rg0 = G.row(k), r = rg0 + lane, n = P.cols - c0;
      if constexpr (EPI == kLinStore) {
        float v[32];
        load_acc(k, v);
        if (!SWAP && g.sum != nullptr) {
          float* sp = g.sum + P.sum_at + (long long)r * P.cols + c0;
          const bool vec = (P.cols & 3) == 0 && n >= 32;
          if (g.sum_read && r < P.rows) {
            if (vec) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(sp + j);
                v[j] += f.x; v[j + 1] += f.y; v[j + 2] += f.z; v[j + 3] += f.w;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < n) v[j] += sp[j];
            }
          }
          if (g.sum_write) {
            if (r < P.rows) {
              if (vec) {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                  *reinterpret_cast<float4*>(sp + j) =
                      make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (j < n) sp[j] = v[j];
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
        if (SWAP && P.c_map >= 0) put(P.c_map, v, c0, rg0);
        else put_plain(P.c, P.c_ld, v, c0, rg0, P.rows, n);
      } else {  // kLinGlu
        float a[32], b[32];
        if (SWAP) {
          // gate's rows are the TMEM lanes of quarters 0 and 1, up's those of 2 and 3, whose
          // warp turns its chunk for the other one
          if (q >= 2) {
            load_raw(k, a);
            turn_write(turn, lane, a);
            arrive_warp(ho.ready);
            dead = !wait_warp(ho.taken, ho.parity);
            ho.parity ^= 1u;
            if (dead) break;
            continue;
          }
          load_acc(k, a);
          dead = !wait_warp(ho.ready, ho.parity);
          ho.parity ^= 1u;
          if (dead) break;
          // quarter q's warp is number (q + 2) % 4 of its half: the partner's is number q
          turn_read(reinterpret_cast<const float*>(epi + (h * 4 + q) * warp_bytes(EPI)), lane, b);
          arrive_warp(ho.taken);
        } else {
          load_acc(k, a);
          load_acc(k + 2, b);
        }
        if (g.keep == kKeepBf16) {
          if (g.kept_vec) {
            put(g.map_gate, a, c0, rg0);
            put(g.map_up, b, c0, rg0);
          } else {
            put_plain(static_cast<__nv_bfloat16*>(g.gate), g.ffn, a, c0, rg0, P.rows, n);
            put_plain(static_cast<__nv_bfloat16*>(g.up), g.ffn, b, c0, rg0, P.rows, n);
          }
        } else if (g.keep == kKeepAct8) {
          put_act8(g.map_gate, g.gate, g.gate_scale, a, c0, rg0, n, r < P.rows);
          put_act8(g.map_up, g.up, g.up_scale, b, c0, rg0, n, r < P.rows);
        }
        // one loop per activation: the three side by side in one loop overflow the
        // instruction cache
        if (g.act == DMUON_ACT_SILU) glu32<DMUON_ACT_SILU>(a, b);
        else if (g.act == DMUON_ACT_GELU) glu32<DMUON_ACT_GELU>(a, b);
        else glu32<DMUON_ACT_GELU_TANH>(a, b);
        put(P.c_map, a, c0, rg0);
      }
    }
    if (dead) break;
    release();
  }
  // stores complete, and stop reading shared memory, before the CTA exits
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

// kLinGluGrad.  The kept gate and up of a chunk come in by TMA, a chunk ahead, and the
// three outputs leave by TMA.  (With lanes reading their own rows from global memory the
// loads took 17000 of a tile's 45000 cycles, and reading and writing 8 rows x 64 bytes an
// instruction was no better: 86 us against 59 for 2048 tokens, 1536/8960.)  Rows that
// are not 16-byte aligned are read by the lanes.
template <bool SWAP>
DM_DEV void epilogue_grad(const LinArgs& g, uint32_t rank, uint64_t* tfull, uint64_t* tempty,
                          uint8_t* epi, uint64_t* kept_bars, uint32_t tmem_base,
                          volatile int* abort_flag) {
  using Geo = Chunks<kLinGluGrad, SWAP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, h = (warp - 2) >> 2, ew = warp - 2;
  float* turn = reinterpret_cast<float*>(epi + ew * warp_bytes(kLinGluGrad));
  const uint32_t buf0 = smem_u32(turn), kept0 = buf0 + 4096u;
  uint64_t* kept_bar = kept_bars + ew;
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
  const int clusters = int(cluster_count_x());
  const bool act8 = g.keep == kKeepAct8, vec = g.kept_vec != 0;
  const int blocks = (g.ffn + kActBlock - 1) / kActBlock;
  int stored = 0;
  uint32_t kept_parity = 0;
  bool fetched = false;  // a chunk's gate and up are on their way

  // every lane is done with what the buffer held
  auto fetch = [&](const Geo& G, int k) {
    if (!vec || !G.inside(k)) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(kept_bar, act8 ? 2048u : 4096u);
      tma_load_2d_u32(kept0, &g.maps[g.map_gate], smem_u32(kept_bar), G.c(k), G.row(k));
      tma_load_2d_u32(kept0 + 2048u, &g.maps[g.map_up], smem_u32(kept_bar), G.c(k), G.row(k));
    }
    fetched = true;
  };
  auto read_kept = [&](Kept& kg, Kept& ku) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (act8 && i >= 2) break;
      const uint32_t at = kept0 + (act8 ? uint32_t(lane * 32 + i * 16) : epi_off(lane, i));
      ld_shared_v4(at, kg.q[i].x, kg.q[i].y, kg.q[i].z, kg.q[i].w);
      ld_shared_v4(at + 2048u, ku.q[i].x, ku.q[i].y, ku.q[i].z, ku.q[i].w);
    }
    __syncwarp();
  };
  auto put = [&](int map, const uint32_t (&w)[16], int c0, int rg0) {
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

  int it = 0;
  for (int u = int(cluster_id_x()); u < g.total_units; u += clusters, ++it) {
    const Unit U = decode_unit(g, u);
    const Geo G(g, U, int(rank), q, h);
    const LinProblem& P = G.P;
    const int acc = it & 1;
    if (U.q < 0 && !fetched) fetch(G, 0);
    // block scales, as stored: a plain tile's four of a row lie side by side
    uint2 scale4[2] = {};
    const bool four = act8 && vec && !SWAP && blocks % 4 == 0 && G.inside(0);
    if (four && U.q < 0 && G.row(0) + lane < P.rows) {
      const long long at = (long long)(G.row(0) + lane) * blocks + G.c(0) / kActBlock;
      scale4[0] = *reinterpret_cast<const uint2*>(g.gate_scale + at);
      scale4[1] = *reinterpret_cast<const uint2*>(g.up_scale + at);
    }
    int w = 1;
    if (lane == 0) w = mbar_wait_cluster(&tfull[acc], uint32_t(it >> 1) & 1u, abort_flag) ? 1 : 0;
    w = __shfl_sync(0xffffffffu, w, 0);
    if (!w) {
      if (lane == 0) raise_abort(g.err, abort_flag);
      break;
    }
    tc_fence_after();
    const uint32_t t_acc = tmem_base + uint32_t(acc * kAccCols) + (uint32_t(q * 32) << 16);
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_tempty + uint32_t(acc) * 8u);
    };
    if (U.q >= 0) {
      store_part(G, U, t_acc, lane);
      release();
      continue;
    }
    bool dead = false;
#pragma unroll 1
    for (int k = 0; k < 4 && G.inside(k); ++k) {
      const int c0 = G.c(k), rg0 = G.row(k), r = rg0 + lane, n = P.cols - c0;
      Kept kg{}, ku{};
      if (vec) {
        int kw = 1;
        if (lane == 0) {
          kw = mbar_wait(kept_bar, kept_parity, abort_flag) ? 1 : 0;
          if (!kw) raise_abort(g.err, abort_flag);
        }
        dead = __shfl_sync(0xffffffffu, kw, 0) == 0;
        if (dead) break;
        kept_parity ^= 1u;
        read_kept(kg, ku);
        if (four) {
          const uint32_t sg = k & 2 ? scale4[0].y : scale4[0].x;
          const uint32_t su = k & 2 ? scale4[1].y : scale4[1].x;
          kg.scale = __uint_as_float(k & 1 ? sg & 0xFFFF0000u : sg << 16);
          ku.scale = __uint_as_float(k & 1 ? su & 0xFFFF0000u : su << 16);
        } else if (act8 && r < P.rows) {
          const long long at = (long long)r * blocks + c0 / kActBlock;
          kg.scale = __bfloat162float(g.gate_scale[at]);
          ku.scale = __bfloat162float(g.up_scale[at]);
        }
        fetched = false;
        if (G.inside(k + 1)) {
          fetch(G, k + 1);
        } else if (u + clusters < g.total_units) {
          const Unit N = decode_unit(g, u + clusters);
          if (N.q < 0) fetch(Geo(g, N, int(rank), q, h), 0);
        }
      } else if (r < P.rows) {
        const bool inner = r > 0 && r + 1 < P.rows;
        fetch_kept(g, g.gate, g.gate_scale, r, c0, n, inner, kg);
        fetch_kept(g, g.up, g.up_scale, r, c0, n, inner, ku);
      }
      float v[32];
      __syncwarp();
      tmem_ld32(t_acc + uint32_t(G.col(k) * 32), v);
      tmem_ld_wait();
      if (!G.inside(k + 1)) release();  // the accumulator is in registers
      if (SWAP) {
        if (lane == 0) bulk_wait_read<0>();  // no store still reads the buffer
        __syncwarp();
        turn_write(turn, lane, v);
        __syncwarp();
        turn_read(turn, lane, v);
        __syncwarp();
      }
      // in halves of 16 columns, packed as they are done, to stay within the registers
      uint32_t pg[16], pd[16], ph[16];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float ga[16], up[16];
        kept_values(g, kg, half, ga);
        kept_values(g, ku, half, up);
        float* vh = v + 16 * half;
        if (g.act == DMUON_ACT_SILU) glu_grad16<DMUON_ACT_SILU>(vh, ga, up);
        else if (g.act == DMUON_ACT_GELU) glu_grad16<DMUON_ACT_GELU>(vh, ga, up);
        else glu_grad16<DMUON_ACT_GELU_TANH>(vh, ga, up);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          pg[8 * half + j] = pack_bf16x2(ga[2 * j], ga[2 * j + 1]);
          pd[8 * half + j] = pack_bf16x2(vh[2 * j], vh[2 * j + 1]);
          ph[8 * half + j] = pack_bf16x2(up[2 * j], up[2 * j + 1]);
        }
      }
      put(P.c_map, pg, c0, rg0);
      put(g.map_dup, pd, c0, rg0);
      put(g.map_h, ph, c0, rg0);
    }
    if (dead) break;
    if (!G.inside(0)) release();
  }
  // a fetch that nobody waited for (after an abort) must land before the CTA exits
  if (fetched && lane == 0) (void)mbar_wait(kept_bar, kept_parity, nullptr, kAbortSettleCycles);
  // stores complete, and stop reading shared memory, before the CTA exits
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

// Logits of the cross entropy, accumulated in registers over runs of K.  A group of
// vocabulary entries (128 plainly: the columns of a lane; 32 swapped: the lanes of
// a warp) shares its maximum m: exp(z - m) = 2^((z - m) log2 e).  A token's target takes
// no part (its logit counts as -infinity): the loss of a token that is sure of it is the
// weight of the others, which would be lost beside the target's 1.  m is at least the
// lowest finite number, so that a group whose logits are all -infinity weighs nothing.
constexpr float kLowest = -3.40282347e38f;
template <bool SWAP>
DM_DEV void epilogue_xent(const LinArgs& g, uint32_t rank, uint64_t* tfull, uint64_t* tempty,
                          uint8_t* epi, uint32_t tmem_base, volatile int* abort_flag) {
  constexpr float kLog2e = 1.44269504f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, h = (warp - 2) >> 2, ew = warp - 2;
  float* turn = reinterpret_cast<float*>(epi + ew * warp_bytes(kLinStore));
  const uint32_t buf0 = smem_u32(turn);
  const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
  const int clusters = int(cluster_count_x());
  const int chunks = SWAP ? g.nt / 32 : kAccCols / 32;
  const LinProblem& P = g.prob[0];
  int it = 0;
  bool ok = true;

  // swapped: 32 exponentials of one token, entries c0 .., to the workspace in fp16
  auto put = [&](const float* e, int c0, int rg0) {
    const uint32_t buf = buf0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 p = __floats2half2_rn(e[8 * i + 2 * j] * kXentScale,
                                            e[8 * i + 2 * j + 1] * kXentScale);
        o[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      st_shared_v4(buf + epi_off(lane, i), o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&g.maps[P.c_map], buf, c0, rg0);
      bulk_commit();
    }
  };

  for (int u = int(cluster_id_x()); ok && u < g.total_units; u += clusters) {
    const Unit U = decode_unit(g, u);
    float z[kXentGroup];
#pragma unroll
    for (int j = 0; j < kXentGroup; ++j) z[j] = 0.f;
#pragma unroll 1
    for (int lo = U.kb_lo; lo < U.kb_hi; lo += kRunElems / Stage<kLinXent, SWAP>::k, ++it) {
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
      const uint32_t t = tmem_base + uint32_t(acc * kAccCols) + (uint32_t(q * 32) << 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = SWAP ? (2 * (k >> 1) + h) * 32 + (k & 1) * 16 : h * kXentGroup + k * 16;
        if (!SWAP || 2 * (k >> 1) + h < chunks) {
          float v[16];
          tmem_ld16(t + uint32_t(col), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) z[k * 16 + j] += v[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_tempty + uint32_t(acc) * 8u);
    }
    if (!ok) break;
    if constexpr (!SWAP) {
      const int rg0 = U.ti * kTile + int(rank) * kHalf + q * 32, r = rg0 + lane;
      const int g0 = U.tj * kTile + h * kXentGroup;  // first vocabulary entry of the group
      if (g0 >= P.cols || rg0 >= P.rows) continue;
      const long long t = r < P.rows ? g.target[r] : -1;
      const int d = t >= g0 && t < g0 + kXentGroup && t < P.cols ? int(t - g0) : -1;
      if (__any_sync(0xffffffffu, d >= 0)) {
#pragma unroll
        for (int j = 0; j < kXentGroup; ++j)
          if (j == d) z[j] = -INFINITY;
      }
      const int n = P.cols - g0;
      if (n < kXentGroup) {  // entries past the vocabulary weigh nothing
#pragma unroll
        for (int j = 0; j < kXentGroup; ++j)
          if (j >= n) z[j] = -INFINITY;
      }
      float m = fmaxf(z[0], kLowest);
#pragma unroll
      for (int j = 1; j < kXentGroup; ++j) m = fmaxf(m, z[j]);
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = k * 32; j < k * 32 + 32; ++j) {
          z[j] = ex2((z[j] - m) * kLog2e);
          s += z[j];
        }
        // 64 entries of each token at a time: 128-byte rows
        if (P.c_map >= 0 && (k & 1) && (k - 1) * 32 < n) {
          if (lane == 0) bulk_wait_read<0>();  // the store that last read the buffer
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 p = __floats2half2_rn(z[(k - 1) * 32 + 8 * i + 2 * j] * kXentScale,
                                                  z[(k - 1) * 32 + 8 * i + 2 * j + 1] * kXentScale);
              o[j] = *reinterpret_cast<const uint32_t*>(&p);
            }
            st_shared_v4(buf0 + uint32_t(lane * 128 + ((i ^ (lane & 7)) << 4)), o[0], o[1], o[2],
                         o[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&g.maps[P.c_map], buf0, g0 + (k - 1) * 32, rg0);
            bulk_commit();
          }
        }
      }
      if (r < P.rows)
        g.group_stat[(long long)(g0 / kXentGroup) * g.stat_ld + r] = make_float2(m, s);
    } else {
      const int c0 = U.ti * kTile + int(rank) * kHalf + q * 32;
      if (c0 >= P.cols) continue;
      const int n = P.cols - c0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rg0 = U.tj * g.nt + (2 * k + h) * 32, r = rg0 + lane;
        if (2 * k + h < chunks && rg0 < P.rows) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = z[k * 32 + j];
          if (P.c_map >= 0 && lane == 0) bulk_wait_read<0>();  // no store still reads the buffer
          __syncwarp();
          turn_write(turn, lane, v);
          __syncwarp();
          if (r < P.rows) {  // the target, in the word from which this lane reads it
            const unsigned long long d = (unsigned long long)(g.target[r] - c0);
            if (d < 32) st_shared_f32(buf0 + uint32_t(lane * 32 + (int(d) ^ lane)) * 4u, -INFINITY);
          }
          turn_read(turn, lane, v);
          __syncwarp();
          if (n < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j >= n) v[j] = -INFINITY;
          }
          float m = fmaxf(v[0], kLowest);
#pragma unroll
          for (int j = 1; j < 32; ++j) m = fmaxf(m, v[j]);
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[j] = ex2((v[j] - m) * kLog2e);
            s += v[j];
          }
          if (P.c_map >= 0) put(v, c0, rg0);
          if (r < P.rows) g.group_stat[(long long)(c0 / 32) * g.stat_ld + r] = make_float2(m, s);
        }
      }
    }
  }
  // stores complete, and stop reading shared memory, before the CTA exits
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

template <int EPI, bool A_MN, bool B_MN, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1) pair_gemm_kernel(const __grid_constant__ LinArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sEpi = smem + stage_area(EPI);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(sEpi + kEpiWarps * warp_bytes(EPI));
  uint64_t* empty_bar = full_bar + kMaxStages;
  uint64_t* tfull = empty_bar + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain_bar = tempty + 2;
  // ready and taken of four warp pairs (kLinGlu), or one per epilogue warp (kLinGluGrad)
  uint64_t* pair_bar = drain_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pair_bar + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
  const uint32_t rank = cluster_rank();
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kLinMaps && int(threadIdx.x) - 64 < g.n_maps)
    prefetch_tensormap(&g.maps[threadIdx.x - 64]);
  if (threadIdx.x == 0) {
    for (int b = 0; b < 8; ++b) mbar_init(&pair_bar[b], 1);  // one lane of a warp
    for (int s = 0; s < kMaxStages; ++s) {
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
  // What follows reads what earlier launches wrote.  The next launch may start once this
  // one is past its wait: then every launch but this one is complete, which lets it read
  // ahead of its own wait (LinEarly) what this one does not write.  The epilogue's warps
  // always wait, so that a launch ends after those before it.  (1 to 3% of a pass with
  // fewer than 1000 tokens: loss and gradients of 300, 1536 x 151936, 450 -> 440 us.)
  if (g.early == kEarlyNone || threadIdx.x >= 64) {
    grid_wait();
    grid_launch_dependents();
  }

  if (warp == 0) {
    if (elect_one())
      producer<EPI, A_MN, B_MN, SWAP>(g, rank, smem, full_bar, empty_bar, abort_flag);
  } else if (warp == 1) {
    if (rank == 0 && elect_one())
      mma_issuer<EPI, A_MN, B_MN, SWAP>(g, smem, full_bar, empty_bar, tfull, tempty, drain_bar,
                                        tmem_base, abort_flag);
  } else if (warp >= 2) {
    if constexpr (EPI == kLinXent)
      epilogue_xent<SWAP>(g, rank, tfull, tempty, sEpi, tmem_base, abort_flag);
    else if constexpr (EPI == kLinGluGrad)
      epilogue_grad<SWAP>(g, rank, tfull, tempty, sEpi, pair_bar, tmem_base, abort_flag);
    else
      epilogue<EPI, SWAP>(g, rank, tfull, tempty, sEpi, pair_bar, tmem_base, abort_flag);
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

// ------------------------------------------------------------------ joining split tiles
// A block of 256 threads takes one 32 x 32 chunk of a split tile (kLinGlu: gate's
// and up's), adds the parts in order, turns it if need be, and runs the epilogue
// with eight consecutive columns of a row per thread of its first half.  Bound by
// the latency of reading the parts (from L2, mostly): a thread keeps its four
// elements of eight parts in flight.
constexpr int kJoinThreads = 256;
DM_DEV float load_part(const float* p) {  // not moved: eight parts' loads go out together
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
DM_DEV void sum_parts(const float* p, size_t stride, int split, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.f;
  int s = 0;
  for (; s + 8 <= split; s += 8) {
    float t[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) t[k][j] = load_part(p + (s + k) * stride + j * 32);
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += t[k][j];
  }
  float t[8][4];
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (s + k < split) {
#pragma unroll
      for (int j = 0; j < 4; ++j) t[k][j] = load_part(p + (s + k) * stride + j * 32);
    }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (s + k < split) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += t[k][j];
    }
}
DM_DEV void store_row8(__nv_bfloat16* dst, int n, bool vec, const float (&v)[8]) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) dst[j] = __float2bfloat16_rn(v[j]);
  }
}
// Eight values of a 32-value block (its four threads are neighbours in a warp; all
// lanes of the warp take part).
DM_DEV void store_act8_part(signed char* codes, __nv_bfloat16* scale, int n, bool vec, bool write,
                            bool first, const float (&v)[8]) {
  float top = 0.f, bad = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = j < n ? v[j] : 0.f;
    top = fmaxf(top, fabsf(x));
    bad = fmaf(x, 0.f, bad);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (!write || n <= 0) return;
  const float s = act8_scale(top, bad == 0.f);
  const float r = bad == 0.f && s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j >> 2] |= (act8_code_fast(bad == 0.f ? v[j] : 0.f, r) & 0xFFu) << (8 * (j & 3));
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) codes[j] = (signed char)(w[j >> 2] >> (8 * (j & 3)));
  }
  if (first) *scale = __float2bfloat16_rn(s);
}

template <int EPI>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ LinArgs g) {
  __shared__ float t0[32][33], t1[EPI == kLinGlu ? 32 : 1][33];
  grid_launch_dependents();
  grid_wait();
  const int chunks = g.swap ? g.nt / 32 : kAccCols / 32;
  // chunk of the tile: CTA of the pair, column chunk, TMEM lane quarter
  const int cols = EPI == kLinGlu && !g.swap ? chunks / 2 : chunks;
  const int quarters = EPI == kLinGlu && g.swap ? 2 : 4;
  int b = int(blockIdx.x);
  const int q = b % quarters;
  b /= quarters;
  const int rank = b & 1;
  b >>= 1;
  const int col = b % cols;
  b /= cols;  // split tile
  const Unit U = decode_unit(g, g.full_tiles + b * g.split);
  const LinProblem& P = g.prob[U.prob];
  int row0, c0;
  if (g.swap) {
    row0 = U.tj * g.nt + col * 32;
    c0 = EPI == kLinGlu ? U.ti * kHalf + rank * 64 + q * 32 : U.ti * kTile + rank * kHalf + q * 32;
  } else {
    row0 = U.ti * kTile + rank * kHalf + q * 32;
    c0 = (EPI == kLinGlu ? U.tj * kHalf : U.tj * kTile) + col * 32;
  }
  if (row0 >= P.rows || c0 >= P.cols) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t stride = size_t(chunks) * 32 * kTile;
  const float* base = g.partial + size_t(b) * g.split * stride + warp * 128 + lane;
  auto chunk_at = [&](int cc, int qq) { return ((size_t(rank) * chunks + cc) * 4 + qq) * 1024; };
  float sv[4], su[4];
  sum_parts(base + chunk_at(col, q), stride, g.split, sv);
  if (EPI == kLinGlu)
    sum_parts(base + (g.swap ? chunk_at(col, q + 2) : chunk_at(col + cols, q)), stride, g.split, su);
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // sv[j]: TMEM lane `lane`, column 4 warp + j
    const int i = g.swap ? warp * 4 + j : lane, k = g.swap ? lane : warp * 4 + j;
    t0[i][k] = sv[j];
    if (EPI == kLinGlu) t1[i][k] = su[j];
  }
  __syncthreads();
  if (threadIdx.x >= 128) return;
  float v[8], u[8];
  const int tr = threadIdx.x >> 2, tc = (threadIdx.x & 3) * 8;
  const int r = row0 + tr, c = c0 + tc, n = P.cols - c;
  const bool in = r < P.rows;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = t0[tr][tc + j];
    if (EPI == kLinGlu) u[j] = t1[tr][tc + j];
  }
  const bool vec = P.c_map >= 0;
  if (EPI == kLinStore) {
    if (!in || n <= 0) return;
    if (g.sum != nullptr) {
      float* sp = g.sum + P.sum_at + (long long)r * P.cols + c;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          if (g.sum_read) v[j] += sp[j];
          if (g.sum_write) sp[j] = v[j];
        }
      if (g.sum_write) return;
    }
    if (g.scale != nullptr) {
      const float f = *g.scale;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f;
    }
    store_row8(P.c + (long long)r * P.c_ld + c, n, vec, v);
  } else if (EPI == kLinGlu) {
    const long long at = (long long)r * g.ffn + c;
    if (g.keep == kKeepBf16 && in) {
      store_row8(static_cast<__nv_bfloat16*>(g.gate) + at, n, g.kept_vec != 0, v);
      store_row8(static_cast<__nv_bfloat16*>(g.up) + at, n, g.kept_vec != 0, u);
    } else if (g.keep == kKeepAct8) {
      const long long sa = (long long)r * ((g.ffn + kActBlock - 1) / kActBlock) + c0 / kActBlock;
      store_act8_part(static_cast<signed char*>(g.gate) + at, g.gate_scale + sa, n,
                      g.kept_vec != 0, in, tc == 0, v);
      store_act8_part(static_cast<signed char*>(g.up) + at, g.up_scale + sa, n, g.kept_vec != 0,
                      in, tc == 0, u);
    }
    if (!in || n <= 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = g.act == DMUON_ACT_SILU   ? act_value<DMUON_ACT_SILU>(v[j])
                      : g.act == DMUON_ACT_GELU ? act_value<DMUON_ACT_GELU>(v[j])
                                                : act_value<DMUON_ACT_GELU_TANH>(v[j]);
      v[j] = a * u[j];
    }
    store_row8(P.c + (long long)r * P.c_ld + c, n, true, v);
  } else {  // kLinGluGrad
    if (!in || n <= 0) return;
    const long long at = (long long)r * g.ffn + c;
    float ga[8], up[8];
    if (g.keep == kKeepBf16) {
      const __nv_bfloat16* pg = static_cast<const __nv_bfloat16*>(g.gate) + at;
      const __nv_bfloat16* pu = static_cast<const __nv_bfloat16*>(g.up) + at;
      if (g.kept_vec && n >= 8) {
        unpack8(*reinterpret_cast<const uint4*>(pg), ga);
        unpack8(*reinterpret_cast<const uint4*>(pu), up);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ga[j] = j < n ? __bfloat162float(pg[j]) : 0.f;
          up[j] = j < n ? __bfloat162float(pu[j]) : 0.f;
        }
      }
    } else {
      const long long sa = (long long)r * ((g.ffn + kActBlock - 1) / kActBlock) + c / kActBlock;
      const float sg = __bfloat162float(g.gate_scale[sa]), su = __bfloat162float(g.up_scale[sa]);
      const signed char* pg = static_cast<const signed char*>(g.gate) + at;
      const signed char* pu = static_cast<const signed char*>(g.up) + at;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ga[j] = j < n ? sg * float(pg[j]) : 0.f;
        up[j] = j < n ? su * float(pu[j]) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, da;
      if (g.act == DMUON_ACT_SILU) act_both<DMUON_ACT_SILU>(ga[j], a, da);
      else if (g.act == DMUON_ACT_GELU) act_both<DMUON_ACT_GELU>(ga[j], a, da);
      else act_both<DMUON_ACT_GELU_TANH>(ga[j], a, da);
      const float dh = v[j];
      ga[j] = dh * up[j] * da;
      up[j] *= a;
      v[j] = dh * a;
    }
    const long long to = (long long)r * P.c_ld + c;
    store_row8(P.c + to, n, true, ga);
    store_row8(g.dup + to, n, true, v);
    store_row8(g.h + to, n, true, up);
  }
}

using Kernel = void (*)(LinArgs);
Kernel kernel_for(int epi, bool a_mn, bool b_mn, bool swap) {
  if (swap) {
    if (b_mn) return nullptr;
    switch (epi) {
      case kLinGlu: return a_mn ? nullptr : pair_gemm_kernel<kLinGlu, false, false, true>;
      case kLinGluGrad: return a_mn ? pair_gemm_kernel<kLinGluGrad, true, false, true> : nullptr;
      case kLinXent: return a_mn ? nullptr : pair_gemm_kernel<kLinXent, false, false, true>;
      case kLinStore:
        return a_mn ? pair_gemm_kernel<kLinStore, true, false, true>
                    : pair_gemm_kernel<kLinStore, false, false, true>;
      default: return nullptr;
    }
  }
  switch (epi) {
    case kLinGlu: return !a_mn && !b_mn ? pair_gemm_kernel<kLinGlu, false, false, false> : nullptr;
    case kLinGluGrad:
      return !a_mn && b_mn ? pair_gemm_kernel<kLinGluGrad, false, true, false> : nullptr;
    case kLinXent:
      return !a_mn && !b_mn ? pair_gemm_kernel<kLinXent, false, false, false> : nullptr;
    case kLinStore:
      if (!a_mn) return b_mn ? pair_gemm_kernel<kLinStore, false, true, false>
                             : pair_gemm_kernel<kLinStore, false, false, false>;
      return b_mn ? pair_gemm_kernel<kLinStore, true, true, false> : nullptr;
    default: return nullptr;
  }
}

}  // namespace

size_t lin_partial_bytes() { return kPartialBytes; }

cudaError_t lin_prepare() {
  for (int epi = kLinStore; epi <= kLinXent; ++epi)
    for (int v = 0; v < 8; ++v) {
      const Kernel k = kernel_for(epi, (v & 1) != 0, (v & 2) != 0, (v & 4) != 0);
      if (k == nullptr) continue;
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 int(kSmemBytes));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

// Swapped where that saves a tenth of the padded rows: at 7/8 of them a block of
// 4096/14336 measured 7% faster with 448 tokens and 1% with 224 (1536/8960: 1% and 10%
// slower, backward 2% faster and the same); at all of them both are within 2% of the other.
// The cross entropy's epilogue costs more swapped, once a tile, while what swapping saves
// grows with K: with several token tiles it breaks even at K (256 - nt) = 150e3 (320 tokens:
// K = 1024 76 us against 69, 1536 138 both ways, 2560 173 against 193), with one, where the
// weights' way from memory hides most of either, at 250e3 to 330e3.  Up to 32 tokens it wins
// throughout (one token, K = 1536: 92 us against 127).
bool lin_swaps(long long tokens, int epi, long long k, int* nt) {
  const long long plain = (tokens + kTile - 1) / kTile;  // tiles of 256 tokens, either way
  const long long fit = ((tokens + plain - 1) / plain + 31) / 32 * 32;
  *nt = int(fit);
  if (epi == kLinXent)
    return tokens <= kXentSwapTokens &&
           (fit <= 32 || k * (kTile - fit) >= (plain == 1 ? 300000 : 160000));
  return fit * 10 < kTile * 9;
}

// floor(2^32 / d) or one more: the quotient's estimate is off by one at most.
static unsigned lin_magic(int d) {
  return d <= 1 ? 0xFFFFFFFFu : unsigned((0x100000000ull + unsigned(d) - 1) / unsigned(d));
}

void lin_schedule(LinArgs& g, int epi, int clusters) {
  int tiles = 0, kb = 0;
  for (int p = 0; p < g.n_prob; ++p) {
    g.prob[p].tile_begin = tiles;
    tiles += g.prob[p].tiles_m * g.prob[p].tiles_n;
    const int k = g.prob[p].kb0 + g.prob[p].kb1;
    kb = p == 0 || k < kb ? k : kb;
    g.prob[p].strip_magic = lin_magic(kStrip * g.prob[p].tiles_n);
    g.prob[p].last_magic = lin_magic(g.prob[p].tiles_m % kStrip);
  }
  if (g.swap) {
    g.stages = stage_area(epi) / ((kHalf + g.nt / 2) * lin_stage_k(epi, true) * 2);
    if (g.stages > kMaxStages) g.stages = kMaxStages;
  }
  g.full_tiles = g.total_units = tiles;
  g.split = 1;
  g.split_magic = lin_magic(1);
  const int rest = tiles % clusters;
  if (epi == kLinXent || rest == 0) return;
  // Microseconds of the last wave.  Per 128 K-elements a pair moves 64 KB plus 256
  // bytes per column of its tile through each SM's shared memory (in by TMA, out to the
  // tensor core) at about 243 GB/s: 0.54 for 256 columns.  With few tokens the weights'
  // way from HBM takes longer, 0.75 shared by the token tiles that use them.  A part
  // costs about 0.3 more (the pipeline stays filled from one to the next); joining costs
  // a launch (3) and the parts' way to L2 and back (5 TB/s).
  const int cols = g.swap ? g.nt : kTile;
  double t_kb = (65536 + 256.0 * cols) / 243e3;
  if (g.swap) t_kb = std::max(t_kb, 0.75 / g.prob[0].tiles_n);
  t_kb *= lin_stage_k(epi, g.swap != 0) / 128.0;
  const double part = double(cols) * kTile * sizeof(float);
  double best = kb * t_kb + 0.3;
  for (int s = 2; rest * s * part <= double(kPartialBytes) && 2 * s <= kb; ++s) {
    const int waves = (rest * s + clusters - 1) / clusters;
    const double cost = waves * ((kb + s - 1) / s * t_kb + 0.3) + 3 + 2 * rest * s * part / 5e6;
    if (cost < best) {
      best = cost;
      g.split = s;
    }
  }
  g.split_magic = lin_magic(g.split);
  if (g.split > 1) {
    g.full_tiles = tiles - rest;
    g.total_units = g.full_tiles + rest * g.split;
  }
}

cudaError_t launch_lin(const LinArgs& g, int epi, bool a_mn, bool b_mn, int max_clusters,
                       cudaStream_t s) {
  if (g.total_units <= 0) return cudaSuccess;
  const Kernel k = kernel_for(epi, a_mn, b_mn, g.swap != 0);
  if (k == nullptr) return cudaErrorInvalidValue;
  const int clusters = g.total_units < max_clusters ? g.total_units : max_clusters;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(2 * clusters), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = counted(cudaLaunchKernelEx(&cfg, k, g));
  if (e != cudaSuccess || g.split == 1) return e;
  const int chunks = (g.swap ? g.nt : kAccCols) / 32;
  const int tiles = (g.total_units - g.full_tiles) / g.split;
  const int blocks = tiles * 2 * chunks * (epi == kLinGlu ? 2 : 4);
  return launch_dependent(epi == kLinStore ? join_kernel<kLinStore>
                          : epi == kLinGlu ? join_kernel<kLinGlu>
                                           : join_kernel<kLinGluGrad>,
                          unsigned(blocks), unsigned(kJoinThreads), s, g);
}

}  // namespace dm
