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
// A cluster of up to 8 CTAs takes the whole packed batch of a head (or a run of its sequences),
// cut evenly into stretches of blocks wherever sequences begin and end.  A CTA whose last sequence
// goes on in the next one's stretch first sums that sequence's share of the state alone (keys and
// values), the shares go to the CTAs behind it through memory, and then each CTA sweeps its
// stretch, keys and values coming from L2 the second time.  Long batches go in rounds of at most
// kRoundBlocks blocks a CTA, so that a round's keys and values stay in L2.
#include "dmuon.h"
#include "f32x2.cuh"
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

// Warps: states, weighted scores, outputs, loads and products (two of the last four idle: register
// shares are given to whole warpgroups).
constexpr int kStateWarps = 8, kWeighWarps = 8, kOutWarps = 4, kOtherWarps = 4;
constexpr int kWeighWarp = kStateWarps, kOutWarp = kWeighWarp + kWeighWarps;
constexpr int kLoadWarp = kOutWarp + kOutWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kThreads = (kStateWarps + kWeighWarps + kOutWarps + kOtherWarps) * 32;
// Registers of a thread at launch, and what each kind takes: the shares add up to what the block
// was launched with.
constexpr int kRegs = 80, kStateRegs = 120, kWeighRegs = 64, kOutRegs = 64, kOtherRegs = 48;
static_assert(kStateWarps * kStateRegs + kWeighWarps * kWeighRegs + kOutWarps * kOutRegs +
                      kOtherWarps * kOtherRegs == kThreads / 32 * kRegs, "");
constexpr int kMaxStages = 4;
constexpr int kSmemBytes = 232448;
constexpr int kMiscBytes = 1536;  // barriers and powers of the decay
constexpr uint32_t kTmemCols = 512;
// TMEM columns: scores (then the weighted ones), the block's own state, two parts of the output
constexpr uint32_t kColScore = 0, kColState = 128, kColInner = 256, kColOuter = 384;
constexpr long long kAbortSettleCycles = 2000000;
constexpr int kRoundBlocks = 8;

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

struct Shared {
  uint64_t full[kMaxStages];   // a stage's loads
  uint64_t empty[kMaxStages];  // its products, and its output gone
  uint64_t score;              // scores in TMEM
  uint64_t weighted;           // weighted scores in TMEM
  uint64_t keys[2];            // keys decayed, rows past the end cleared: of even and odd blocks, as
                               // the states' warps may be one ahead of the products there
  uint64_t half;               // the state's first product (exact states)
  uint64_t low;                // the keys' low parts in shared memory
  uint64_t block_state[2];     // the block's state in TMEM
  uint64_t entry;              // the entering state in shared memory
  uint64_t spent;              // weighted scores read
  uint64_t out;                // both parts of the output in TMEM
  uint64_t taken;              // and out of it again
  uint64_t put;                // this CTA's share of the round in memory
  uint64_t shares;             // the round's shares of all CTAs of the cluster
  uint32_t tmem;
  int abort;
  int place[6];                // what locate() found
  int sums[kThreads / 32];
  alignas(16) float fall[96];        // what weigh() needs of the powers of a
  float power_[32 + kMixBlock + 1];  // a^n, n = -32 .. 128; zeros below 0
};
static_assert(sizeof(Shared) <= kMiscBytes, "");

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

// ------------------------------------------------------------------ the packed batch
struct Extent {
  int begin, len, blocks;
};
DM_DEV Extent extent_of(const LinAttnArgs& g, int seq) {
  int b = 0, e = g.tokens;
  if (g.offsets != nullptr) {
    b = min(max(g.offsets[seq], 0), g.tokens);
    e = min(max(g.offsets[seq + 1], 0), g.tokens);
  }
  const int len = max(e - b, 0);
  return {b, len, (len + kMixBlock - 1) / kMixBlock};
}

// A block of the batch, in the order of the sweep (along time, or against it from the last
// sequence's end on): number m of sequence seq.
struct Cursor {
  int seq, m;
  Extent x;
  DM_DEV int place(const LinAttnArgs& g) const { return g.against ? x.blocks - 1 - m : m; }
  DM_DEV int row(const LinAttnArgs& g) const { return x.begin + place(g) * kMixBlock; }
  DM_DEV int live(const LinAttnArgs& g) const { return min(kMixBlock, x.len - place(g) * kMixBlock); }
  // tokens of the sequence's first n blocks of the sweep
  DM_DEV int before(const LinAttnArgs& g, int n) const {
    return g.against ? x.len - min(x.len, (x.blocks - n) * kMixBlock) : min(x.len, n * kMixBlock);
  }
  // n blocks on (past the batch's end: any block)
  DM_DEV void skip(const LinAttnArgs& g, int n) {
    while (n >= x.blocks - m) {
      n -= x.blocks - m;
      m = 0;
      do {
        seq += g.against ? -1 : 1;
        if (seq < 0 || seq >= g.sequences) {
          seq = 0;
          x = Extent{0, 0, 0x7FFFFFFF};
          break;
        }
        x = extent_of(g, seq);
      } while (x.blocks == 0);
    }
    m += n;
  }
};

// What a CTA does: stretches of `per` blocks, one in each round, of the nb blocks that its cluster
// takes.
struct Work {
  int nb, per, rounds, rank;
  Cursor start;  // the first round's
};
// Blocks of all sequences are numbered in their order; sequences are dealt to the clusters of a
// head by the block that they start with, and the blocks of a cluster evenly to its CTAs.  Every
// thread counts the blocks of a run of sequences.
DM_DEV Work divide(const LinAttnArgs& g, int rank, int nb) {
  Work w;
  w.nb = nb;
  w.rank = rank;
  w.rounds = g.split == 1 ? 1 : max(1, (nb + g.split * kRoundBlocks - 1) / (g.split * kRoundBlocks));
  w.per = (nb + g.split * w.rounds - 1) / (g.split * w.rounds);
  w.start.seq = 0;
  w.start.m = 0;
  w.start.x = Extent{0, 0, 0x7FFFFFFF};
  return w;
}
// The same for at most 32 sequences, one to a lane: every warp finds its own.
DM_DEV Work locate_few(const LinAttnArgs& g, int group, int rank) {
  const int lane = int(threadIdx.x) & 31;
  Extent x{0, 0, 0};
  if (lane < g.sequences) x = extent_of(g, lane);
  int first = x.blocks;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, first, d);
    if (lane >= d) first += v;
  }
  const int total = __shfl_sync(0xffffffffu, first, 31);
  first -= x.blocks;
  int lo = 0, hi = total;
  if (g.groups > 1) {
    const int a = int((long long)total * group / g.groups), b = int((long long)total * (group + 1) / g.groups);
    lo = __reduce_min_sync(0xffffffffu, x.blocks > 0 && first >= a ? first : total);
    hi = __reduce_min_sync(0xffffffffu, x.blocks > 0 && first >= b ? first : total);
  }
  Work w = divide(g, rank, hi - lo);
  const int i = min(rank * w.per, w.nb);
  if (i < w.nb) {
    const int flat = g.against ? hi - 1 - i : lo + i;
    const unsigned has = __ballot_sync(0xffffffffu, first <= flat && flat < first + x.blocks);
    const int s = __ffs(has) - 1;
    w.start.seq = s;
    w.start.x.begin = __shfl_sync(0xffffffffu, x.begin, s);
    w.start.x.len = __shfl_sync(0xffffffffu, x.len, s);
    w.start.x.blocks = __shfl_sync(0xffffffffu, x.blocks, s);
    const int m = flat - __shfl_sync(0xffffffffu, first, s);
    w.start.m = g.against ? w.start.x.blocks - 1 - m : m;
  }
  return w;
}
DM_DEV Work locate(const LinAttnArgs& g, int group, int rank, Shared* sh) {
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int run = (g.sequences + kThreads - 1) / kThreads;
  const int s0 = min(tid * run, g.sequences), s1 = min(s0 + run, g.sequences);
  int mine = 0;
  for (int s = s0; s < s1; ++s) mine += extent_of(g, s).blocks;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sh->sums[warp] = upto;
  __syncthreads();
  int first = upto - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) first += sh->sums[w];
    total += sh->sums[w];
  }
  if (tid == 0) sh->place[0] = sh->place[1] = total;
  __syncthreads();
  int lo = 0, hi = total;
  if (g.groups > 1) {
    const int cut[2] = {int((long long)total * group / g.groups),
                        int((long long)total * (group + 1) / g.groups)};
    int at = first;
    for (int s = s0; s < s1; ++s) {
      const int n = extent_of(g, s).blocks;
#pragma unroll
      for (int i = 0; i < 2; ++i)  // the first start of a (non-empty) sequence from the cut on
        if (n > 0 && at >= cut[i]) atomicMin(&sh->place[i], at);
      at += n;
    }
    __syncthreads();
    lo = sh->place[0];
    hi = sh->place[1];
  }
  Work w = divide(g, rank, hi - lo);
  const int i = min(rank * w.per, w.nb);
  const int flat = g.against ? hi - 1 - i : lo + i;
  if (i < w.nb) {
    int at = first;
    for (int s = s0; s < s1; ++s) {
      const int n = extent_of(g, s).blocks;
      if (at <= flat && flat < at + n) {
        sh->place[2] = s;
        sh->place[3] = g.against ? n - 1 - (flat - at) : flat - at;
      }
      at += n;
    }
    __syncthreads();
    w.start.seq = sh->place[2];
    w.start.m = sh->place[3];
    w.start.x = extent_of(g, w.start.seq);
  }
  return w;
}

// A CTA's part of a round: n blocks from `at` on, before them the last `ahead` of those, from
// `share` on, for the state that they leave to the next CTA.
struct Round {
  int lo, n, ahead;
  Cursor at, share;
};
DM_DEV void fill_round(const LinAttnArgs& g, const Work& w, Round& r) {
  r.n = max(0, min(w.per, w.nb - r.lo));
  r.ahead = 0;
  if (w.rank + 1 < g.split && r.n > 0) {
    r.share = r.at;
    r.share.skip(g, r.n - 1);
    if (r.share.m + 1 < r.share.x.blocks) {
      r.ahead = min(r.share.m + 1, r.n);
      r.share.m -= r.ahead - 1;
    }
  }
}
DM_DEV Round first_round(const LinAttnArgs& g, const Work& w) {
  Round r;
  r.lo = w.rank * w.per;
  r.at = w.start;
  fill_round(g, w, r);
  return r;
}
DM_DEV void next_round(const LinAttnArgs& g, const Work& w, Round& r) {
  if (r.lo + g.split * w.per < w.nb) r.at.skip(g, g.split * w.per);
  r.lo += g.split * w.per;
  fill_round(g, w, r);
}

// ------------------------------------------------------------------ loads
template <int DK, int DV>
DM_DEV void load_role(const LinAttnArgs& g, const Work& w, int head, uint8_t* smem, Shared* sh) {
  using T = Tiles<DK, DV>;
  volatile int* flag = &sh->abort;
  int it = 0;
  auto load = [&](int row, bool queries) {
    const int s = it % T::stages;
    if (!await(&sh->empty[s], ((it / T::stages) & 1) ^ 1, g.err, flag)) return false;
    uint8_t* q = smem + s * T::stage;
    uint8_t *k = q + T::q, *v = k + T::k;
    uint64_t* bar = &sh->full[s];
    mbar_arrive_expect_tx(bar, uint32_t(T::k + T::v + (queries ? T::k : 0)));
#pragma unroll
    for (int p = 0; p < DK / 64; ++p) {
      if (queries) tma_load_3d(q + p * 16384, &g.q, bar, p * 64, head, row);
      tma_load_3d(k + p * 16384, &g.k, bar, p * 64, head, row);
    }
#pragma unroll
    for (int p = 0; p < DV / 64; ++p) tma_load_3d(v + p * 16384, &g.v, bar, p * 64, head, row);
    ++it;
    return true;
  };
  Round r = first_round(g, w);
  for (int round = 0; round < w.rounds; ++round) {
    Cursor c = r.share;
    for (int i = 0; i < r.ahead; ++i, ++c.m)
      if (!load(c.row(g), false)) return;
    c = r.at;
    for (int i = 0; i < r.n; ++i, c.skip(g, 1))
      if (!load(c.row(g), true)) return;
    next_round(g, w, r);
  }
}

// ------------------------------------------------------------------ products
template <int DK, int DV>
DM_DEV void mma_role(const LinAttnArgs& g, const Work& w, uint8_t* smem, uint8_t* state, Shared* sh) {
  using T = Tiles<DK, DV>;
  volatile int* flag = &sh->abort;
  const uint32_t tmem = sh->tmem;
  const bool exact = g.exact != 0;
  constexpr uint32_t id_score = idesc_bf16(128, 128, false, false);
  constexpr uint32_t id_inner = idesc_bf16(128, DV, false, true);
  constexpr uint32_t id_state = idesc_bf16(128, DV, true, true);
  // (a^..k)^T V, rows of K in steps of 16 tokens.  With 64 key elements the upper half of the
  // 128 rows reads what follows the tile; those lanes of the result are not used.
  auto block_state = [&](uint32_t to, uint32_t k, uint32_t v, bool accumulate) {
    const uint64_t a = sdesc_sw128(k, 16384, 1024), b = sdesc_sw128(v, 16384, 1024);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      umma_bf16(tmem + to, a + uint64_t(j) * 128, b + uint64_t(j) * 128, id_state,
                accumulate || j > 0);
  };
  int it = 0, swept = 0;
  // ahead of the sweep: the state alone, into two places in turn
  auto share = [&]() {
    const int s = it % T::stages;
    const uint32_t q = smem_u32(smem) + s * T::stage, k = q + T::q, v = k + T::k;
    if (!await(&sh->full[s], (it / T::stages) & 1, g.err, flag)) return false;
    if (!await(&sh->keys[it & 1], it >> 1 & 1, g.err, flag)) return false;
    tc_fence_after();
    const uint32_t to = (it & 1) != 0 ? kColInner : kColState;
    block_state(to, k, v, false);
    if (exact) block_state(to, q, v, true);  // the keys' low parts lie where queries would
    umma_commit(&sh->block_state[it & 1]);
    umma_commit(&sh->empty[s]);
    mbar_arrive_n(&sh->empty[s], kOutWarps);
    ++it;
    return true;
  };
  auto block = [&]() {
    const int s = it % T::stages;
    const uint32_t q = smem_u32(smem) + s * T::stage, k = q + T::q, v = k + T::k;
    if (!await(&sh->full[s], (it / T::stages) & 1, g.err, flag)) return false;
    // the last block's weighted scores have been read (no order is promised between products of
    // unlike shape); its output is on its way meanwhile
    if (swept > 0 && !await(&sh->spent, (swept - 1) & 1, g.err, flag)) return false;
    tc_fence_after();
    {
      const uint64_t a = sdesc_sw128(q, 16, 1024), b = sdesc_sw128(k, 16, 1024);
#pragma unroll
      for (int j = 0; j < DK / 16; ++j) {
        const uint64_t at = uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2;
        umma_bf16(tmem + kColScore, a + at, b + at, id_score, j > 0);
      }
      umma_commit(&sh->score);
    }
    if (!await(&sh->keys[it & 1], it >> 1 & 1, g.err, flag)) return false;
    tc_fence_after();
    block_state(kColState, k, v, false);
    umma_commit(exact ? &sh->half : &sh->block_state[it & 1]);
    if (!await(&sh->weighted, swept & 1, g.err, flag)) return false;
    if (swept > 0 && !await(&sh->taken, (swept - 1) & 1, g.err, flag)) return false;
    tc_fence_after();
    {
      const uint64_t b = sdesc_sw128(v, 16384, 1024);
#pragma unroll
      for (int j = 0; j < 8; ++j)  // 8 columns of weighted scores a step, in two halves
        umma_bf16_ts(tmem + kColInner, tmem + kColScore + (j >> 2) * 64 + (j & 3) * 8,
                     b + uint64_t(j) * 128, id_inner, j > 0);
      umma_commit(&sh->spent);
    }
    if (!await(&sh->entry, swept & 1, g.err, flag)) return false;
    tc_fence_after();
    {
      const uint64_t a = sdesc_sw128(q, 16, 1024);
      const uint64_t e = sdesc_sw128(smem_u32(state), DK * 128, 1024);
#pragma unroll
      for (int j = 0; j < DK / 16; ++j)
        umma_bf16(tmem + kColOuter, a + uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2,
                  e + uint64_t(j) * 128, id_inner, j > 0);
      umma_commit(&sh->out);
    }
    if (exact) {
      if (!await(&sh->low, swept & 1, g.err, flag)) return false;
      tc_fence_after();
      block_state(kColState, k, v, true);
      umma_commit(&sh->block_state[it & 1]);
    }
    umma_commit(&sh->empty[s]);
    ++swept;
    ++it;
    return true;
  };
  Round r = first_round(g, w);
  for (int round = 0; round < w.rounds; ++round) {
    // the last output of the round before, read by then, makes room for every other share
    if (r.ahead > 0 && swept > 0 && !await(&sh->taken, (swept - 1) & 1, g.err, flag)) return;
    for (int i = 0; i < r.ahead; ++i)
      if (!share()) return;
    for (int i = 0; i < r.n; ++i)
      if (!block()) return;
    next_round(g, w, r);
  }
}

// ------------------------------------------------------------------ states
// Thread (warp w, lane) keeps row 32 (w % 4) + lane of the state, columns DV / 2 (w / 4) on.
template <int DK, int DV>
struct StateRole {
  static constexpr int kCols = DV / 2, kThreadsHere = kStateWarps * 32;
  static constexpr int kUnits = kMixBlock * DK / 8 / kThreadsHere;  // 16 bytes of keys each
  using T = Tiles<DK, DV>;
  const LinAttnArgs& g;
  const Work& w;
  Shared* sh;
  uint8_t* smem;
  uint8_t* entry;
  float log_decay;
  int head, cluster, tid, lane, row, col;
  F2 st[kCols / 2];
  float full_weight[4];  // of this thread's four rows of keys in a whole block

  DM_DEV const float* power() const { return sh->power_ + 32; }
  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  DM_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) st[i] = 0;
  }
  DM_DEV long long state_at(int seq) const {
    return ((long long)seq * g.heads + head) * g.dk * g.dv + (long long)row * g.st_row;
  }
  DM_DEV void read_initial(int seq) {
    zero();
    if (g.state_in == nullptr || row >= g.dk) return;
    const float* p = g.state_in + state_at(seq);
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const int c = col + 2 * i;
      if (c < g.dv)
        st[i] = f2(g.in_scale * p[(long long)c * g.st_col], g.in_scale * p[(long long)(c + 1) * g.st_col]);
    }
  }
  DM_DEV void write_final(int seq) {
    if (row >= g.dk) return;
    float* p = g.state_out + state_at(seq);
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const int c = col + 2 * i;
      float a, b;
      f2_split(st[i], a, b);
      if (c < g.dv) {
        p[(long long)c * g.st_col] = g.out_scale * a;
        p[(long long)(c + 1) * g.st_col] = g.out_scale * b;
      }
    }
  }
  // A state in the workspace, four columns at a time so that a warp's rows lie together.  Slots of
  // a CTA: its share of even and of odd rounds (the last CTA's: what the round leaves to the
  // next), and a copy of a sequence's first state.
  DM_DEV float4* slot(int rank, int which) const {
    return reinterpret_cast<float4*>(g.local) +
           (((size_t)cluster * g.split + rank) * kMixSlots + which) * (kMixLocalBytes / 16) +
           (col / 4) * 128 + row;
  }
  DM_DEV void put(float4* p) {
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      float4 v;
      f2_split(st[2 * i], v.x, v.y);
      f2_split(st[2 * i + 1], v.z, v.w);
      __stcg(p + i * 128, v);
    }
  }
  // st <- f st + what lies there
  DM_DEV void take(const float4* p, float f) {
    const F2 ff = f2(f, f);
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      const float4 v = __ldcg(p + i * 128);
      st[2 * i] = fma2(ff, st[2 * i], f2(v.x, v.y));
      st[2 * i + 1] = fma2(ff, st[2 * i + 1], f2(v.z, v.w));
    }
  }
  // The state before this CTA's stretch of a round, inside sequence c.seq: what the rounds before
  // left, and the shares of the CTAs before it.
  DM_DEV void gather(const Cursor& c, int round) {
    zero();
    const int base = round * g.split * w.per;              // sweep's number of the round's first block
    const int start = base + w.rank * w.per - c.m;          // and of the sequence's
    int from = 0;
    if (start < base) take(slot(g.split - 1, round & 1), 1.f);
    else from = (start - base) / w.per;
    for (int r = from; r < w.rank; ++r) {
      const int n0 = max(base + r * w.per - start, 0), n1 = base + (r + 1) * w.per - start;
      take(slot(r, round & 1), expf(log_decay * float(c.before(g, n1) - c.before(g, n0))));
    }
  }
  // The state as the operand of Q S: rows of 64 bf16, 128-byte swizzle.
  DM_DEV void write_entry() {
    if (row < DK) {
      const uint32_t at = smem_u32(entry) + row * 128;
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i) {
        const int c = col + i * 8;
        st_shared_v4(at + (c >> 6) * (DK * 128) + ((((c & 63) >> 3) ^ (row & 7)) << 4),
                     pack_bf16(st[4 * i]), pack_bf16(st[4 * i + 1]), pack_bf16(st[4 * i + 2]),
                     pack_bf16(st[4 * i + 3]));
      }
    }
    announce(&sh->entry);
  }
  DM_DEV void announce(uint64_t* bar) {  // shared-memory writes, to the tensor core
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  // The thread's unit n of the keys, its token
  DM_DEV int token_of(int n) const { return ((tid >> 3) + 32 * n) & (kMixBlock - 1); }
  DM_DEV float key_weight(int j, int live) const {
    return j >= live ? 0.f : power()[g.against ? j + 1 : live - 1 - j];
  }
  // Keys of block `it` times their decay, in place; what bf16 drops of them (EXACT) to low[], or
  // (TO_QUERIES) to where the stage's queries would lie.  Rows past the end hold another sequence's
  // tokens, or anything: they become zeros, here and in V.
  template <bool EXACT, bool TO_QUERIES, bool WHOLE>
  DM_DEV void decay_keys(int it, int live, uint32_t (&low)[EXACT && !TO_QUERIES ? kUnits * 4 : 1]) {
    const uint32_t stage = smem_u32(smem) + (it % T::stages) * T::stage + tid * 16;
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const uint32_t at = stage + T::q + n * kThreadsHere * 16;
      const int j = token_of(n);
      const float f = WHOLE ? full_weight[n & 3] : key_weight(j, live);
      const F2 ff = f2(f, f);
      uint32_t x[4], y[4];
      ld_shared_v4(at, x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 v = WHOLE || j < live ? mul2(bf16_pair(x[i]), ff) : 0;
        x[i] = pack_bf16(v);
        y[i] = EXACT ? pack_bf16(add2(v, negate2(bf16_pair(x[i])))) : 0;
        if constexpr (EXACT && !TO_QUERIES) low[n * 4 + i] = y[i];
      }
      st_shared_v4(at, x[0], x[1], x[2], x[3]);
      if (EXACT && TO_QUERIES) st_shared_v4(at - T::q, y[0], y[1], y[2], y[3]);
    }
    if (!WHOLE) {
#pragma unroll
      for (int n = 0; n < kMixBlock * DV / 8 / kThreadsHere; ++n)
        if (token_of(n) >= live) st_shared_v4(stage + T::q + T::k + n * kThreadsHere * 16, 0, 0, 0, 0);
    }
  }
  template <bool EXACT, bool TO_QUERIES>
  DM_DEV void keys(int it, int live, uint32_t (&low)[EXACT && !TO_QUERIES ? kUnits * 4 : 1]) {
    if (live == kMixBlock) decay_keys<EXACT, TO_QUERIES, true>(it, live, low);
    else decay_keys<EXACT, TO_QUERIES, false>(it, live, low);
    announce(&sh->keys[it & 1]);
  }
  // Block `it`, of `live` tokens, joins the state.
  DM_DEV bool add_block(int it, int live, uint32_t from) {
    if (!wait(&sh->block_state[it & 1], it >> 1)) return false;
    tc_fence_after();
    const float f = power()[live];
    const F2 ff = f2(f, f);
    const uint32_t at = sh->tmem + (uint32_t(row & ~31) << 16) + from + col;
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
      float x[16];
      tmem_ld16(at + c * 16, x);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 8; ++i) st[c * 8 + i] = fma2(ff, st[c * 8 + i], f2(x[2 * i], x[2 * i + 1]));
    }
    if (row >= g.dk) zero();  // of keys past the head's size: 0 times an infinity of V may be there
    tc_fence_before();
    return true;
  }
  DM_DEV bool loaded(int it) { return wait(&sh->full[it % T::stages], it / T::stages); }
  // The share of this round is in memory (or was not asked for): tell the cluster.
  DM_DEV bool arrive(int round) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->put);
    if (tid < 32) {
      if (!wait(&sh->put, round)) return false;
      if (tid < g.split) mbar_arrive_cluster(mapa_shared(smem_u32(&sh->shares), uint32_t(tid)));
      __syncwarp();
    }
    return true;
  }
  DM_DEV bool all_arrived(int round) {
    if (mbar_wait_cluster(&sh->shares, round & 1, &sh->abort)) return true;
    raise_abort(g.err, &sh->abort);
    return false;
  }
  // This CTA's share, from the start of its last sequence or of its stretch: each block's keys while
  // the product of the block before runs.
  template <bool EXACT>
  DM_DEV bool sum_share(const Round& r, int& it) {
    Cursor c = r.share;
    uint32_t none[1];
    int before = 0;
    for (int i = 0; i <= r.ahead; ++i, ++c.m) {
      int live = 0;
      if (i < r.ahead) {
        live = c.live(g);
        if (!loaded(it + i)) return false;
        keys<EXACT, true>(it + i, live, none);
      }
      if (i > 0 && !add_block(it + i - 1, before, ((it + i - 1) & 1) != 0 ? kColInner : kColState))
        return false;
      before = live;
    }
    it += r.ahead;
    return true;
  }
  template <bool EXACT>
  DM_DEV void run() {
#pragma unroll
    for (int n = 0; n < 4; ++n) full_weight[n] = key_weight(token_of(n), kMixBlock);
    zero();
    const bool over = g.state_in != nullptr && g.state_in == g.state_out;
    int it = 0, swept = 0;
    bool ok = true;
    Round r = first_round(g, w);
    for (int round = 0; ok && round < w.rounds; ++round) {
      bool kept = false;
      if (r.ahead > 0) {
        if (r.share.m == 0) {
          read_initial(r.share.seq);
          // another CTA may write the final state over it before this one's sweep is there
          if (over) put(slot(w.rank, 2));
          kept = over;
        } else {
          zero();
        }
        ok = sum_share<EXACT>(r, it);
        put(slot(w.rank, round & 1));
      }
      if (g.split > 1) ok = arrive(round) && ok;
      Cursor c = r.at;
      for (int i = 0; ok && i < r.n; ++i, c.skip(g, 1), ++it, ++swept) {
        const int live = c.live(g);
        uint32_t low[EXACT ? kUnits * 4 : 1];
        ok = loaded(it) && wait(&sh->score, swept);
        if (!ok) break;
        keys<EXACT, false>(it, live, low);
        if (i == 0 && g.split > 1) {
          ok = all_arrived(round);
          if (!ok) break;
          if (c.m > 0) gather(c, round);
        }
        if (c.m == 0) {
          if (kept && c.seq == r.share.seq) {
            zero();
            take(slot(w.rank, 2), 0.f);
          } else {
            read_initial(c.seq);
          }
        }
        ok = swept == 0 || wait(&sh->out, swept - 1);
        if (!ok) break;
        write_entry();
        if constexpr (EXACT) {
          ok = wait(&sh->half, swept);
          if (!ok) break;
          const uint32_t k = smem_u32(smem) + (it % T::stages) * T::stage + T::q + tid * 16;
#pragma unroll
          for (int n = 0; n < kUnits; ++n)
            st_shared_v4(k + n * kThreadsHere * 16, low[4 * n], low[4 * n + 1], low[4 * n + 2],
                         low[4 * n + 3]);
          announce(&sh->low);
        }
        ok = add_block(it, live, kColState);
        if (g.state_out != nullptr && c.m + 1 == c.x.blocks) write_final(c.seq);
      }
      if (r.n == 0 && g.split > 1) ok = ok && all_arrived(round);
      if (w.rank + 1 == g.split && round + 1 < w.rounds) put(slot(w.rank, (round + 1) & 1));
      next_round(g, w, r);
    }
  }
  // Sequences without tokens: their states pass through.
  DM_DEV void pass_through(int first, int stride) {
    for (int s = first; s < g.sequences; s += stride) {
      if (extent_of(g, s).blocks != 0) continue;
      read_initial(s);
      write_final(s);
    }
  }
};

// ------------------------------------------------------------------ weighted scores
// Thread (warp w, lane) has row 32 (w % 4) + lane of the scores, columns 64 (w / 4) on.
//
// Weights a^(i - j) of 32 columns from j0 = 32 b on, rows 32 q + lane: nothing above the diagonal;
// at b = q one weight of its own per lane and column; below, with D = 32 (q - b), a^lane times
// a^(D - jj), which all lanes share: four columns' come with one broadcast load.  Against time the
// same turned: a^(31 - lane) a^(D - 31 + jj), D = 32 (b - q).
struct WeighRole {
  const LinAttnArgs& g;
  const Work& w;
  Shared* sh;
  int warp, lane;

  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  // Columns j0 .. j0 + 31 of x, weighted, to p.
  template <bool AGAINST>
  DM_DEV void weigh(const float (&x)[32], int q, int j0, int live, F2 own, uint32_t (&p)[16]) {
    const int b = j0 >> 5;
    if (b == q || (AGAINST && j0 + 32 > live)) {
      const int row = q * 32 + lane;
      const float* t = sh->power_ + 32 + (AGAINST ? j0 - row : row - j0);
      // columns that row sees, a bit each
      uint32_t see = b == q ? (AGAINST ? 0xFFFFFFFFu << lane : 0xFFFFFFFFu >> (31 - lane)) : 0xFFFFFFFFu;
      if (AGAINST && j0 + 32 > live) see &= 0xFFFFFFFFu >> (j0 + 32 - live);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float u = x[2 * i] * t[AGAINST ? 2 * i : -2 * i];
        const float v = x[2 * i + 1] * t[AGAINST ? 2 * i + 1 : -2 * i - 1];
        p[i] = pack_bf16((see >> (2 * i) & 1) != 0 ? u : 0.f, (see >> (2 * i + 1) & 1) != 0 ? v : 0.f);
      }
    } else {
      const int at = AGAINST ? 32 * (b - q) - 32 : 96 - 32 * (q - b);
      const float4* t = reinterpret_cast<const float4*>(sh->fall + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = t[i];
        p[2 * i] = pack_bf16(mul2(mul2(f2(x[4 * i], x[4 * i + 1]), own), f2(f.x, f.y)));
        p[2 * i + 1] = pack_bf16(mul2(mul2(f2(x[4 * i + 2], x[4 * i + 3]), own), f2(f.z, f.w)));
      }
    }
  }
  template <bool AGAINST>
  DM_DEV bool block(int live, int swept, F2 own) {
    const int q = warp & 3, c0 = (warp >> 2) * 64;
    const uint32_t at = sh->tmem + (uint32_t(q * 32) << 16) + kColScore + c0;
    if (!wait(&sh->score, swept)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      const int j0 = c0 + n * 32;
      uint32_t p[16];
      if (AGAINST ? j0 + 31 < q * 32 || j0 >= live : j0 > q * 32) {
        // nothing on this side of the diagonal
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0;
      } else {
        float x[32];
        tmem_ld32(at + n * 32, x);
        tmem_ld_wait();
        weigh<AGAINST>(x, q, j0, live, own, p);
      }
      tmem_st16(at + n * 16, p);  // two to a column, where scores were read already
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->weighted);
    return true;
  }
  DM_DEV void run() {
    int swept = 0;
    bool ok = true;
    const float f = sh->power_[32 + (g.against ? 31 - lane : lane)];
    const F2 own = f2(f, f);
    Round r = first_round(g, w);
    for (int round = 0; ok && round < w.rounds; ++round) {
      Cursor c = r.at;
      for (int i = 0; ok && i < r.n; ++i, c.skip(g, 1), ++swept) {
        const int live = c.live(g);
        ok = g.against ? block<true>(live, swept, own) : block<false>(live, swept, own);
      }
      next_round(g, w, r);
    }
  }
};

// ------------------------------------------------------------------ outputs
// Thread (warp w, lane) has row 32 w + lane.
template <int DK, int DV>
struct OutRole {
  using T = Tiles<DK, DV>;
  const LinAttnArgs& g;
  const Work& w;
  Shared* sh;
  uint8_t* smem;
  int head, warp, lane;

  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  DM_DEV bool block(int row0, int live, int it, int swept) {
    const int row = warp * 32 + lane, s = it % T::stages;
    const float f = row < live ? sh->power_[32 + (g.against ? live - 1 - row : row + 1)] : 0.f;
    const F2 fs = f2(f * g.scale, f * g.scale), ss = f2(g.scale, g.scale);
    const uint32_t at = sh->tmem + (uint32_t(warp * 32) << 16);
    // 32 columns to a piece of 2 KB, rows of 64 bytes
    const uint32_t tile = smem_u32(smem) + s * T::stage + warp * (DV / 32) * 2048 + lane * 64;
    if (!wait(&sh->out, swept)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int n = 0; n < DV / 16; ++n) {
      float x[16], y[16];
      tmem_ld16(at + kColInner + n * 16, x);
      tmem_ld16(at + kColOuter + n * 16, y);
      tmem_ld_wait();
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = pack_bf16(fma2(fs, f2(y[2 * e], y[2 * e + 1]), mul2(ss, f2(x[2 * e], x[2 * e + 1]))));
      const uint32_t to = tile + (n >> 1) * 2048;
      const int swizzle = (lane >> 1) & 3;
      st_shared_v4(to + (((2 * (n & 1)) ^ swizzle) << 4), o[0], o[1], o[2], o[3]);
      st_shared_v4(to + (((2 * (n & 1) + 1) ^ swizzle) << 4), o[4], o[5], o[6], o[7]);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->taken);
    const int first = row0 + warp * 32;
    const int rows = live - warp * 32;  // of this warp that exist
    if (rows >= 32) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int n = 0; n < DV / 32; ++n)
          if (n * 32 < g.dv) tma_store_3d(&g.o, tile + n * 2048, n * 32, head, first);
        bulk_commit();
        bulk_wait_read<0>();
      }
    } else {
      // the end of a sequence: what lies behind it is not this one's to write
      __syncwarp();
      const uint32_t base = tile - lane * 64;
      for (int u = lane; u < 32 * (DV / 8); u += 32) {
        const int r = u / (DV / 8), n = u % (DV / 8);
        if (r < rows && n * 8 < g.dv) {
          uint4 o;
          ld_shared_v4(base + (n >> 2) * 2048 + r * 64 + (((n & 3) ^ ((r >> 1) & 3)) << 4), o.x, o.y,
                       o.z, o.w);
          *reinterpret_cast<uint4*>(g.out.p + (first + r) * g.out.ts + head * g.out.hs + n * 8) = o;
        }
      }
      __syncwarp();
    }
    if (lane == 0) mbar_arrive(&sh->empty[s]);
    __syncwarp();
    return true;
  }
  DM_DEV void run() {
    int it = 0, swept = 0;
    bool ok = true;
    Round r = first_round(g, w);
    for (int round = 0; ok && round < w.rounds; ++round) {
      it += r.ahead;
      Cursor c = r.at;
      for (int i = 0; ok && i < r.n; ++i, c.skip(g, 1), ++it, ++swept)
        ok = block(c.row(g), c.live(g), it, swept);
      next_round(g, w, r);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) mix_kernel(const __grid_constant__ LinAttnArgs g) {
  extern __shared__ uint8_t smem_raw[];
  using T = Tiles<DK, DV>;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* state = smem + T::stages * T::stage;
  Shared* sh = reinterpret_cast<Shared*>(state + T::state);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
  const int cluster = int(blockIdx.x) / g.split, rank = int(blockIdx.x) - cluster * g.split;
  const int group = cluster / g.heads, head = cluster - group * g.heads;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kOutWarps + 1);
    }
    mbar_init(&sh->score, 1);
    mbar_init(&sh->weighted, kWeighWarps);
    mbar_init(&sh->spent, 1);
    mbar_init(&sh->taken, kOutWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->keys[i], kStateWarps);
      mbar_init(&sh->block_state[i], 1);
    }
    mbar_init(&sh->put, kStateWarps);
    mbar_init(&sh->half, 1);
    mbar_init(&sh->low, kStateWarps);
    mbar_init(&sh->entry, kStateWarps);
    mbar_init(&sh->out, 1);
    mbar_init(&sh->shares, uint32_t(g.split));
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh->tmem, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && elect_one()) {
    prefetch_tensormap(&g.q);
    prefetch_tensormap(&g.k);
    prefetch_tensormap(&g.v);
    prefetch_tensormap(&g.o);
  }
  if (g.split > 1) cluster_sync();  // barriers of all CTAs stand before one arrives on another's
  grid_wait();
  grid_launch_dependents();
  const float log_decay = g.log_decay[head];
  if (threadIdx.x < 32 + kMixBlock + 1) {
    const int n = int(threadIdx.x) - 32;
    sh->power_[threadIdx.x] = n < 0 ? 0.f : n == 0 ? 1.f : expf(log_decay * float(n));
  }
  if (threadIdx.x < 96)
    sh->fall[threadIdx.x] = expf(log_decay * float(g.against ? threadIdx.x + 1 : 96 - threadIdx.x));
  const Work w = g.sequences <= 32 ? locate_few(g, group, rank) : locate(g, group, rank, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp < kStateWarps) {
    regs_inc<kStateRegs>();
    StateRole<DK, DV> r{g, w, sh, smem, state, log_decay, head, cluster, int(threadIdx.x),
                        int(threadIdx.x & 31), int((warp & 3) * 32 + (threadIdx.x & 31)),
                        int(warp >> 2) * (DV / 2)};
    if (g.exact) r.template run<true>();
    else r.template run<false>();
    if (g.state_out != nullptr) r.pass_through(group * g.split + rank, g.groups * g.split);
  } else if (warp < kOutWarp) {
    regs_dec<kWeighRegs>();
    WeighRole r{g, w, sh, warp - kWeighWarp, int(threadIdx.x & 31)};
    r.run();
  } else if (warp < kLoadWarp) {
    regs_dec<kOutRegs>();
    OutRole<DK, DV> r{g, w, sh, smem, head, warp - kOutWarp, int(threadIdx.x & 31)};
    r.run();
  } else {
    regs_dec<kOtherRegs>();
    if (warp == kLoadWarp && elect_one()) load_role<DK, DV>(g, w, head, smem, sh);
    if (warp == kMmaWarp && elect_one()) mma_role<DK, DV>(g, w, smem, state, sh);
    __syncwarp();
  }
  __syncthreads();
  if (*const_cast<volatile int*>(&sh->abort) != 0) {
    // given up: copies and products in flight must land before memory goes away
    const long long t0 = clock64();
    while (clock64() - t0 < kAbortSettleCycles) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(sh->tmem, kTmemCols);
  }
  if (g.split > 1) cluster_sync();  // no CTA leaves while another may still arrive on its barrier
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
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes a{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
    if (e != cudaSuccess) return e;
    // launched with fewer, the states' warps would wait for theirs forever
    if (a.numRegs != kRegs) return cudaErrorInvalidKernelImage;
  }
  return cudaSuccess;
}

cudaError_t launch_linattn(const LinAttnArgs& g, cudaStream_t s) {
  int smem = 0;
  const MixKernel k = kernel_for(g.dk, g.dv, &smem);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(g.groups * g.heads * g.split), 1, 1);
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
