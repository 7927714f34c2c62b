// Linear attention with a decay for each head over packed sequences: one kernel for the forward
// pass and for each gradient.
//
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,   a = exp(log_decay)
//
// A block of 128 tokens of a sequence, i and j counted from its start, L of them live, S_0 the
// state that enters it:
//   o_i = scale [ sum_{j <= i} a^{i-j} (q_i . k_j) v_j  +  a^{i+1} q_i S_0 ]
//   S_L = a^L S_0 + sum_j a^{L-1-j} k_j v_j^T
// No power of a is negative, so nothing overflows however fast a head forgets.  The same with
// time running backwards (j >= i, a^{L-1-i} at the state, a^{j+1} at the keys) gives the
// gradients: with g = scale dout, dq is this of (g, v, k) along time, dk of (v, g, q) and dv of
// (k, q, g) against it, the states transposed or not.
//
// Four tcgen05 products a block, M = 128: scores Q K^T, weighted scores (bf16, in TMEM) times V,
// Q times the state (bf16, in shared memory), and (a^{L-1-j} k_j)^T V, whose fp32 result is added
// to the fp32 state that 256 threads keep in registers -- rounded to nearest there, where a sum
// that stayed in the tensor core over thousands of tokens would be truncated.  Tiles are [token]
// [64 elements] with the 128-byte swizzle; the same tile is a K-major operand where the sum runs
// over the head's elements and an MN-major one where it runs over tokens, so nothing is
// transposed.  Keys take their decay in place once the scores have read them.
//
// A cluster of up to 8 CTAs shares a sequence of a head: each first sums the states of its own
// stretch alone (keys and values), the stretches' states go through memory, each CTA combines
// those before its own, and then sweeps its stretch (keys and values from L2 for the most part).
#include "dmuon.h"
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

constexpr int kStateWarps = 8, kOutWarps = 8;
constexpr int kThreads = (kStateWarps + kOutWarps + 2) * 32;
constexpr int kLoadWarp = kStateWarps + kOutWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kMaxStages = 4;
constexpr int kSmemBytes = 232448;
constexpr int kMiscBytes = 1024;  // barriers and powers of the decay
constexpr uint32_t kTmemCols = 512;
// TMEM columns: scores (then the weighted ones), the block's own state, two parts of the output
constexpr uint32_t kColScore = 0, kColState = 128, kColInner = 256, kColOuter = 384;
constexpr long long kAbortSettleCycles = 2000000;

// DK, DV: head sizes padded to 64 or 128 (TMA fills with zeros).
template <int DK, int DV>
struct Tiles {
  static constexpr int k = kMixBlock * DK * 2, v = kMixBlock * DV * 2;
  static constexpr int q = DK > DV ? k : v;  // also holds the output on its way out
  static constexpr int stage = q + k + v;
  static constexpr int state = DK * DV * 2;
  static constexpr int fit = (kSmemBytes - 1024 - kMiscBytes - state) / stage;
  static constexpr int stages = fit < kMaxStages ? fit : kMaxStages;
  static_assert(stages >= 2, "two stages must fit");
  static constexpr int bytes = 1024 + kMiscBytes + state + stages * stage;
};

struct Bars {
  uint64_t full[kMaxStages];   // a stage's loads
  uint64_t empty[kMaxStages];  // its products, and its output gone
  uint64_t score;              // scores in TMEM
  uint64_t weighted;           // weighted scores in TMEM
  uint64_t keys;               // keys decayed, rows past the end cleared
  uint64_t half;               // the state's first product (exact states)
  uint64_t low;                // the keys' low parts in shared memory
  uint64_t block_state;        // the block's state in TMEM
  uint64_t entry;              // the entering state in shared memory
  uint64_t out;                // both parts of the output in TMEM
  uint32_t tmem;
  int abort;
};

DM_DEV void raise_abort(int* err, volatile int* flag) {
  *flag = 1;
  atomicExch(err, DMUON_ERR_TIMEOUT);
}
// Wait of a whole warp (or one thread); false: gave up.
DM_DEV bool await(uint64_t* bar, uint32_t parity, int* err, volatile int* flag) {
  if (mbar_wait(bar, parity, flag)) return true;
  raise_abort(err, flag);
  return false;
}

// A sequence's blocks in the order of the sweep.
struct Span {
  int begin, len, blocks, lo, hi;  // lo .. hi: this CTA's
  bool against;
  DM_DEV int place(int m) const { return against ? blocks - 1 - m : m; }
  DM_DEV int row(int m) const { return begin + place(m) * kMixBlock; }
  DM_DEV int live(int m) const { return min(kMixBlock, len - place(m) * kMixBlock); }
  // tokens of blocks 0 .. m - 1 of the sweep
  DM_DEV int before(int m) const {
    return against ? len - min(len, (blocks - m) * kMixBlock) : min(len, m * kMixBlock);
  }
};
DM_DEV Span span_of(const LinAttnArgs& g, int seq, int rank) {
  Span s;
  int b = 0, e = g.tokens;
  if (g.offsets != nullptr) {
    b = min(max(g.offsets[seq], 0), g.tokens);
    e = min(max(g.offsets[seq + 1], 0), g.tokens);
  }
  s.begin = b;
  s.len = max(e - b, 0);
  s.blocks = (s.len + kMixBlock - 1) / kMixBlock;
  const int per = (s.blocks + g.split - 1) / g.split;
  s.lo = min(rank * per, s.blocks);
  s.hi = min(s.lo + per, s.blocks);
  s.against = g.against != 0;
  return s;
}

DM_DEV uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
DM_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
DM_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ------------------------------------------------------------------ loads
template <int DK, int DV>
DM_DEV void load_role(const LinAttnArgs& g, const Span& sp, int head, bool first_pass, uint8_t* smem,
                      Bars* bars, volatile int* flag) {
  using T = Tiles<DK, DV>;
  int it = 0;
  for (int pass = first_pass ? 0 : 1; pass < 2; ++pass)
    for (int m = sp.lo; m < sp.hi; ++m, ++it) {
      const int s = it % T::stages;
      if (!await(&bars->empty[s], ((it / T::stages) & 1) ^ 1, g.err, flag)) return;
      uint8_t* q = smem + s * T::stage;
      uint8_t *k = q + T::q, *v = k + T::k;
      const int row = sp.row(m);
      uint64_t* bar = &bars->full[s];
      mbar_arrive_expect_tx(bar, uint32_t(T::k + T::v + (pass != 0 ? T::k : 0)));
#pragma unroll
      for (int p = 0; p < DK / 64; ++p) {
        if (pass != 0) tma_load_3d(q + p * 16384, &g.q, bar, p * 64, head, row);
        tma_load_3d(k + p * 16384, &g.k, bar, p * 64, head, row);
      }
#pragma unroll
      for (int p = 0; p < DV / 64; ++p) tma_load_3d(v + p * 16384, &g.v, bar, p * 64, head, row);
    }
}

// ------------------------------------------------------------------ products
template <int DK, int DV>
DM_DEV void mma_role(const LinAttnArgs& g, const Span& sp, bool first_pass, uint8_t* smem,
                     uint8_t* state, Bars* bars, volatile int* flag) {
  using T = Tiles<DK, DV>;
  const uint32_t tmem = bars->tmem;
  const bool exact = g.state_out != nullptr;
  constexpr uint32_t id_score = idesc_bf16(128, 128, false, false);
  constexpr uint32_t id_inner = idesc_bf16(128, DV, false, true);
  constexpr uint32_t id_state = idesc_bf16(128, DV, true, true);
  // (a^..k)^T V, rows of K in steps of 16 tokens.  With 64 key elements the upper half of the
  // 128 rows reads what follows the tile; those lanes of the result are not used.
  auto block_state = [&](uint32_t k, uint32_t v, bool accumulate) {
    const uint64_t a = sdesc_sw128(k, 16384, 1024), b = sdesc_sw128(v, 16384, 1024);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      umma_bf16(tmem + kColState, a + uint64_t(j) * 128, b + uint64_t(j) * 128, id_state,
                accumulate || j > 0);
  };
  int it = 0, swept = 0;
  for (int pass = first_pass ? 0 : 1; pass < 2; ++pass)
    for (int m = sp.lo; m < sp.hi; ++m, ++it) {
      const int s = it % T::stages;
      const uint32_t q = smem_u32(smem) + s * T::stage, k = q + T::q, v = k + T::k;
      if (!await(&bars->full[s], (it / T::stages) & 1, g.err, flag)) return;
      if (pass == 1) {
        // the last block's weighted scores have been read (no order is promised between
        // products of unlike shape); its output is on its way meanwhile
        if (swept > 0 && !await(&bars->out, (swept - 1) & 1, g.err, flag)) return;
        tc_fence_after();
        const uint64_t a = sdesc_sw128(q, 16, 1024), b = sdesc_sw128(k, 16, 1024);
#pragma unroll
        for (int j = 0; j < DK / 16; ++j) {
          const uint64_t at = uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2;
          umma_bf16(tmem + kColScore, a + at, b + at, id_score, j > 0);
        }
        umma_commit(&bars->score);
      }
      if (!await(&bars->keys, it & 1, g.err, flag)) return;
      tc_fence_after();
      block_state(k, v, false);
      umma_commit(exact ? &bars->half : &bars->block_state);
      if (pass == 1) {
        if (!await(&bars->weighted, swept & 1, g.err, flag)) return;
        tc_fence_after();
        const uint64_t b = sdesc_sw128(v, 16384, 1024);
#pragma unroll
        for (int j = 0; j < 8; ++j)  // 8 columns of weighted scores a step, in two halves
          umma_bf16_ts(tmem + kColInner, tmem + kColScore + (j >> 2) * 64 + (j & 3) * 8,
                       b + uint64_t(j) * 128, id_inner, j > 0);
        if (!await(&bars->entry, swept & 1, g.err, flag)) return;
        tc_fence_after();
        const uint64_t a = sdesc_sw128(q, 16, 1024);
        const uint64_t e = sdesc_sw128(smem_u32(state), DK * 128, 1024);
#pragma unroll
        for (int j = 0; j < DK / 16; ++j)
          umma_bf16(tmem + kColOuter, a + uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2,
                    e + uint64_t(j) * 128, id_inner, j > 0);
        umma_commit(&bars->out);
        ++swept;
      }
      if (exact) {
        if (!await(&bars->low, it & 1, g.err, flag)) return;
        tc_fence_after();
        block_state(k, v, true);
        umma_commit(&bars->block_state);
      }
      umma_commit(&bars->empty[s]);
      if (pass == 0) mbar_arrive_n(&bars->empty[s], kOutWarps);
    }
}

// ------------------------------------------------------------------ states
// Thread (warp w, lane) keeps row 32 (w % 4) + lane of the state, columns DV / 2 (w / 4) on.
template <int DK, int DV>
struct StateRole {
  static constexpr int kCols = DV / 2;
  using T = Tiles<DK, DV>;
  const LinAttnArgs& g;
  const Span& sp;
  Bars* bars;
  volatile int* flag;
  const float* power;
  uint8_t* smem;
  uint8_t* entry;
  int item, tid, lane, row, col;
  float st[kCols];

  DM_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kCols; ++i) st[i] = 0.f;
  }
  DM_DEV void read_initial() {
    zero();
    if (g.state_in == nullptr || row >= g.dk) return;
    const float* p = g.state_in + (long long)item * g.dk * g.dv + (long long)row * g.st_row;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (col + i < g.dv) st[i] = g.in_scale * p[(long long)(col + i) * g.st_col];
  }
  DM_DEV void write_final() {
    if (row >= g.dk) return;
    float* p = g.state_out + (long long)item * g.dk * g.dv + (long long)row * g.st_row;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (col + i < g.dv) p[(long long)(col + i) * g.st_col] = g.out_scale * st[i];
  }
  // Rank r's state alone, four columns at a time so that a warp's rows lie together.
  DM_DEV float4* local(int rank) const {
    return reinterpret_cast<float4*>(g.local) +
           ((size_t)item * g.split + rank) * (kMixLocalBytes / 16) + (col / 4) * 128 + row;
  }
  DM_DEV void publish(int rank) {
    float4* p = local(rank);
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      __stcg(p + i * 128, make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]));
  }
  // S before this CTA's stretch, from those before it.
  DM_DEV void gather(int rank, float log_decay) {
    zero();
    const int per = (sp.blocks + g.split - 1) / g.split;
    for (int r = 0; r < rank; ++r) {
      const int n = sp.before(min((r + 1) * per, sp.blocks)) - sp.before(min(r * per, sp.blocks));
      const float f = n == 0 ? 1.f : expf(log_decay * float(n));
      const float4* p = local(r);
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 x = __ldcg(p + i * 128);
        st[4 * i] = fmaf(f, st[4 * i], x.x);
        st[4 * i + 1] = fmaf(f, st[4 * i + 1], x.y);
        st[4 * i + 2] = fmaf(f, st[4 * i + 2], x.z);
        st[4 * i + 3] = fmaf(f, st[4 * i + 3], x.w);
      }
    }
  }
  // The state as the operand of Q S: rows of 64 bf16, 128-byte swizzle.
  DM_DEV void write_entry() {
    if (row >= DK) return;
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) {
      const int c = col + i * 8;
      const uint32_t at = smem_u32(entry) + (c >> 6) * (DK * 128) + row * 128 +
                          ((((c & 63) >> 3) ^ (row & 7)) << 4);
      st_shared_v4(at, pack_bf16(st[8 * i], st[8 * i + 1]), pack_bf16(st[8 * i + 2], st[8 * i + 3]),
                   pack_bf16(st[8 * i + 4], st[8 * i + 5]), pack_bf16(st[8 * i + 6], st[8 * i + 7]));
    }
  }
  static constexpr int kUnits = kMixBlock * DK / 8 / (kStateWarps * 32);  // 16 bytes each
  DM_DEV float key_weight(int j, int live) const {
    return j >= live ? 0.f : power[sp.against ? j + 1 : live - 1 - j];
  }
  // Keys times their decay, in place; the part that bf16 drops to low[] if EXACT.  Rows past the
  // end hold another sequence's tokens, or anything: they become zeros, here and in V.
  template <bool EXACT>
  DM_DEV void decay_keys(uint8_t* k, uint8_t* v, int live, uint32_t (&low)[EXACT ? kUnits * 4 : 1]) {
    const uint32_t base = smem_u32(k);
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = tid + n * kStateWarps * 32;
      const int j = (u >> 3) & (kMixBlock - 1);
      const float w = key_weight(j, live);
      uint32_t x[4];
      ld_shared_v4(base + u * 16, x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = j < live ? bf16_lo(x[i]) * w : 0.f, b = j < live ? bf16_hi(x[i]) * w : 0.f;
        x[i] = pack_bf16(a, b);
        if constexpr (EXACT) low[n * 4 + i] = pack_bf16(a - bf16_lo(x[i]), b - bf16_hi(x[i]));
      }
      st_shared_v4(base + u * 16, x[0], x[1], x[2], x[3]);
    }
    if (live < kMixBlock) {
#pragma unroll
      for (int n = 0; n < kMixBlock * DV / 8 / (kStateWarps * 32); ++n) {
        const int u = tid + n * kStateWarps * 32;
        if (((u >> 3) & (kMixBlock - 1)) >= live) st_shared_v4(smem_u32(v) + u * 16, 0, 0, 0, 0);
      }
    }
  }
  DM_DEV void announce(uint64_t* bar) {  // shared-memory writes, to the tensor core
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  // Add block m, in stage s, to the state.
  template <bool EXACT>
  DM_DEV bool add_block(int m, int s, int it) {
    uint8_t* k = smem + s * T::stage + T::q;
    const int live = sp.live(m);
    uint32_t low[EXACT ? kUnits * 4 : 1];
    decay_keys<EXACT>(k, k + T::k, live, low);
    announce(&bars->keys);
    if constexpr (EXACT) {
      if (!await(&bars->half, it & 1, g.err, flag)) return false;
#pragma unroll
      for (int n = 0; n < kUnits; ++n)
        st_shared_v4(smem_u32(k) + (tid + n * kStateWarps * 32) * 16, low[4 * n], low[4 * n + 1],
                     low[4 * n + 2], low[4 * n + 3]);
      announce(&bars->low);
    }
    if (!await(&bars->block_state, it & 1, g.err, flag)) return false;
    tc_fence_after();
    const float f = power[live];
    const uint32_t at = bars->tmem + (uint32_t(row & ~31) << 16) + kColState + col;
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
      float x[16];
      tmem_ld16(at + c * 16, x);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        st[c * 16 + i] = row < g.dk ? fmaf(f, st[c * 16 + i], x[i]) : 0.f;
    }
    tc_fence_before();
    return true;
  }
  template <bool EXACT>
  DM_DEV void run(bool first_pass, int rank, float log_decay) {
    int it = 0;
    bool ok = true;
    if (g.split == 1 || (rank == 0 && first_pass)) read_initial();
    else zero();
    if (first_pass) {
      for (int m = sp.lo; ok && m < sp.hi; ++m, ++it) {
        const int s = it % T::stages;
        ok = await(&bars->full[s], (it / T::stages) & 1, g.err, flag) && add_block<EXACT>(m, s, it);
      }
      publish(rank);
    }
    if (g.split > 1) {
      // before the barrier: afterwards the last CTA may write the final state over it
      if (rank == 0) read_initial();
      cluster_arrive();
      cluster_wait();
      if (rank > 0) gather(rank, log_decay);
    }
    int swept = 0;
    for (int m = sp.lo; ok && m < sp.hi; ++m, ++it, ++swept) {
      const int s = it % T::stages;
      if (swept > 0 && !await(&bars->out, (swept - 1) & 1, g.err, flag)) break;
      write_entry();
      announce(&bars->entry);
      ok = await(&bars->full[s], (it / T::stages) & 1, g.err, flag) &&
           await(&bars->score, swept & 1, g.err, flag) && add_block<EXACT>(m, s, it);
    }
    if (EXACT && rank == g.split - 1) write_final();
  }
};

// ------------------------------------------------------------------ scores and outputs
// Thread (warp w, lane) has row 32 (w % 4) + lane of the scores and of the output, columns
// 64 (w / 4) on of the scores and DV / 2 (w / 4) on of the output.
template <int DK, int DV>
DM_DEV void out_role(const LinAttnArgs& g, const Span& sp, int head, bool first_pass,
                     const float* power, uint8_t* smem, Bars* bars, volatile int* flag) {
  using T = Tiles<DK, DV>;
  const int w = int(threadIdx.x >> 5) - kStateWarps, lane = threadIdx.x & 31;
  const int quarter = w & 3, half = w >> 2, row = quarter * 32 + lane;
  const uint32_t lanes = bars->tmem + (uint32_t(quarter * 32) << 16);
  int it = first_pass ? sp.hi - sp.lo : 0, swept = 0;
  for (int m = sp.lo; m < sp.hi; ++m, ++it, ++swept) {
    const int live = sp.live(m);
    if (!await(&bars->score, swept & 1, g.err, flag)) break;
    tc_fence_after();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j0 = half * 64 + b * 32;
      uint32_t p[16];
      // nothing on this side of the diagonal, or past the last live column
      const bool none = sp.against ? j0 + 31 < quarter * 32 || j0 >= live : j0 > quarter * 32 + 31;
      if (none) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0;
      } else {
        float x[32];
        tmem_ld32(lanes + kColScore + j0, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = j0 + i, gap = sp.against ? j - row : row - j;
          x[i] = gap >= 0 && j < live ? x[i] * power[max(gap, 0)] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      }
      tmem_st16(lanes + kColScore + half * 64 + b * 16, p);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->weighted);

    const int s = it % T::stages;
    const float f = row < live ? power[sp.against ? live - 1 - row : row + 1] : 0.f;
    if (!await(&bars->out, swept & 1, g.err, flag)) break;
    tc_fence_after();
    const int first = sp.row(m) + quarter * 32;
    const int rows = live - quarter * 32;  // of this warp that exist
#pragma unroll
    for (int b = 0; b < DV / 64; ++b) {
      const int c = half * (DV / 2) + b * 32;
      float x[32], y[32];
      tmem_ld32(lanes + kColInner + c, x);
      tmem_ld32(lanes + kColOuter + c, y);
      tmem_ld_wait();
      const uint32_t tile = smem_u32(smem) + s * T::stage + (w * (DV / 64) + b) * 2048;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = i * 8 + e * 2;
          o[e] = pack_bf16(g.scale * fmaf(f, y[n], x[n]), g.scale * fmaf(f, y[n + 1], x[n + 1]));
        }
        st_shared_v4(tile + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), o[0], o[1], o[2], o[3]);
      }
      if (rows >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && c < g.dv) tma_store_3d(&g.o, tile, c, head, first);
      } else {
        // the end of a sequence: what lies behind it is not this one's to write
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int r = (lane >> 2) + n * 8, i = lane & 3;
          if (r < rows && c + i * 8 < g.dv) {
            uint4 o;
            ld_shared_v4(tile + r * 64 + ((i ^ ((r >> 1) & 3)) << 4), o.x, o.y, o.z, o.w);
            *reinterpret_cast<uint4*>(g.out.p + (first + r) * g.out.ts + head * g.out.hs + c +
                                      i * 8) = o;
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      bulk_commit();
      bulk_wait_read<0>();
      mbar_arrive(&bars->empty[s]);
    }
    __syncwarp();
  }
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) mix_kernel(const __grid_constant__ LinAttnArgs g) {
  extern __shared__ uint8_t smem_raw[];
  using T = Tiles<DK, DV>;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* state = smem + T::stages * T::stage;
  Bars* bars = reinterpret_cast<Bars*>(state + T::state);
  float* power = reinterpret_cast<float*>(bars + 1);
  static_assert(sizeof(Bars) + (kMixBlock + 1) * sizeof(float) <= kMiscBytes, "");
  volatile int* flag = &bars->abort;

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
  const int item = int(blockIdx.x) / g.split, rank = int(blockIdx.x) - item * g.split;
  const int seq = item / g.heads, head = item - seq * g.heads;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], kOutWarps + 1);
    }
    mbar_init(&bars->score, 1);
    mbar_init(&bars->weighted, kOutWarps);
    mbar_init(&bars->keys, kStateWarps);
    mbar_init(&bars->half, 1);
    mbar_init(&bars->low, kStateWarps);
    mbar_init(&bars->block_state, 1);
    mbar_init(&bars->entry, kStateWarps);
    mbar_init(&bars->out, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && elect_one()) {
    prefetch_tensormap(&g.q);
    prefetch_tensormap(&g.k);
    prefetch_tensormap(&g.v);
    prefetch_tensormap(&g.o);
  }
  grid_wait();
  grid_launch_dependents();
  const float log_decay = g.log_decay[head];
  if (threadIdx.x <= kMixBlock)
    power[threadIdx.x] = threadIdx.x == 0 ? 1.f : expf(log_decay * float(threadIdx.x));
  const Span sp = span_of(g, seq, rank);
  // the CTAs of a cluster but the last sum their stretches' states first
  const bool first_pass = rank + 1 < g.split;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp < kStateWarps) {
    StateRole<DK, DV> r{g, sp, bars, flag, power, smem, state, item, int(threadIdx.x),
                        int(threadIdx.x & 31), int((warp & 3) * 32 + (threadIdx.x & 31)),
                        int(warp >> 2) * (DV / 2)};
    if (g.state_out != nullptr) r.template run<true>(first_pass, rank, log_decay);
    else r.template run<false>(first_pass, rank, log_decay);
  } else {
    if (g.split > 1) cluster_arrive();  // the state's warps wait for their kind only
    if (warp < kLoadWarp) {
      out_role<DK, DV>(g, sp, head, first_pass, power, smem, bars, flag);
    } else if (warp == kLoadWarp) {
      if (elect_one()) load_role<DK, DV>(g, sp, head, first_pass, smem, bars, flag);
    } else if (elect_one()) {
      mma_role<DK, DV>(g, sp, first_pass, smem, state, bars, flag);
    }
    __syncwarp();
    if (g.split > 1) cluster_wait();
  }
  __syncthreads();
  if (*flag != 0) {
    // given up: copies and products in flight must land before memory goes away
    const long long t0 = clock64();
    while (clock64() - t0 < kAbortSettleCycles) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(bars->tmem, kTmemCols);
  }
}

using MixKernel = void (*)(LinAttnArgs);
MixKernel kernel_for(int dk, int dv, int* smem) {
  if (dk <= 64) {
    *smem = dv <= 64 ? Tiles<64, 64>::bytes : Tiles<64, 128>::bytes;
    return dv <= 64 ? mix_kernel<64, 64> : mix_kernel<64, 128>;
  }
  *smem = dv <= 64 ? Tiles<128, 64>::bytes : Tiles<128, 128>::bytes;
  return dv <= 64 ? mix_kernel<128, 64> : mix_kernel<128, 128>;
}

}  // namespace

cudaError_t linattn_prepare() {
  for (int i = 0; i < 4; ++i) {
    int smem = 0;
    const MixKernel k = kernel_for(i & 1 ? 128 : 64, i & 2 ? 128 : 64, &smem);
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_linattn(const LinAttnArgs& g, cudaStream_t s) {
  int smem = 0;
  const MixKernel k = kernel_for(g.dk, g.dv, &smem);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((long long)g.sequences * g.heads * g.split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(g.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.split > 1 ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, k, g));
}

}  // namespace dm
