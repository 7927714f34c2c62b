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
// Three operands are rounded to bf16 because the tensor core takes them so: weighted scores, the state
// that enters a block and the decayed keys.  Outputs and gradients are 0.0026 from 64 bits by it, where
// rounding the result alone gives 0.0017.  A second part of each would take a product and a pass of its
// own: the keys' costs a fifth (152 heads of 5120 tokens: 125 us, 150 with it), and is taken where a
// state is an output, which then keeps 16 bits of every term.
//
// A cluster of up to 8 CTAs takes the whole packed batch of a head (or a run of its sequences), cut
// evenly into stretches of blocks wherever sequences begin and end.  A CTA whose last sequence goes
// on in the next one's stretch first sums that sequence's share of the state alone (keys and
// values), the shares go to the CTAs behind it through memory, and then each CTA sweeps its
// stretch.  (Sharing again and again, in rounds short enough for keys and values to stay in L2, was
// slower the shorter the rounds: 65536 tokens of 32 heads 829 us in rounds of 12 blocks a CTA, 797
// of 16, 747 of 64, 738 in one, which is 675 to 690 now.)  Where that would leave a CTA to a head,
// or a head's gradient, and SMs without one or a last wave of few, sequences are instead dealt
// whole to all SMs (deal()).
//
// Bound, with a head to each SM, by HBM and by the SM's shared memory at once: of the 5500 cycles
// of a block of 128 x 128 heads about 2450 go to the warps' reads and writes there, 1800 to
// operands of products, 1000 to copies, and little else can run beside them; the tensor cores are
// busy for 30%. 152 heads of 5120 tokens take 125 us, 6.4 TB/s of q, k, v and out, 0.94 of the copy
// rate (150 us where a final state is written, 74 us of 64 elements: 5.4 TB/s).  With fewer heads,
// keys and values are read twice and not all SMs take part: 8192 tokens of 32 heads 85 us (40 at
// the copy rate), 65536 tokens with states 675 to 690 (318).  Where a final state is written,
// the warps of a CTA load and store spilled registers about 300 times a block, next to never
// elsewhere.  The gradients of 8192 tokens of 32 heads in 5 sequences take 149 us
// (69), dealt: 44 to 49 blocks to each SM, 3.1 us a block.
#include "dmuon.h"
#include "f32x2.cuh"
#include "mix.h"
#include "ptx.cuh"

namespace dm {
namespace {

// Warps: states, weighted scores, outputs, then loads and two that issue products (one of the last
// four idles: register shares are given to whole warpgroups).
constexpr int kStateWarps = 8, kWeighWarps = 8, kOutWarps = 4, kOtherWarps = 4;
constexpr int kWeighWarp = kStateWarps, kOutWarp = kWeighWarp + kWeighWarps;
constexpr int kLoadWarp = kOutWarp + kOutWarps, kStateMmaWarp = kLoadWarp + 1,
              kOutMmaWarp = kLoadWarp + 2;
constexpr int kThreads = (kStateWarps + kWeighWarps + kOutWarps + kOtherWarps) * 32;
// Registers of a thread at launch, and what each kind takes: the shares add up to what the block
// was launched with.  (Exact states keep more at hand; the others gain 1 to 4% by the weights'.)
constexpr int kRegs = 80, kOutRegs = 64, kOtherRegs = 48;
__host__ __device__ constexpr int state_regs(bool exact) { return exact ? 120 : 112; }
__host__ __device__ constexpr int weigh_regs(bool exact) { return exact ? 64 : 72; }
static_assert(kStateWarps * state_regs(false) + kWeighWarps * weigh_regs(false) + kOutWarps * kOutRegs +
                      kOtherWarps * kOtherRegs == kThreads / 32 * kRegs, "");
static_assert(kStateWarps * state_regs(true) + kWeighWarps * weigh_regs(true) + kOutWarps * kOutRegs +
                      kOtherWarps * kOtherRegs == kThreads / 32 * kRegs, "");
constexpr int kMaxStages = 4;
constexpr int kSmemBytes = 232448;
constexpr int kMiscBytes = 2048;  // barriers and powers of the decay
constexpr uint32_t kTmemCols = 512;
// TMEM columns: scores (then the weighted ones), the block's own state, two parts of the output
constexpr uint32_t kColScore = 0, kColState = 128, kColInner = 256, kColOuter = 384;
constexpr long long kAbortSettleCycles = 2000000;

// DK, DV: head sizes padded to 64 or 128 (TMA fills with zeros).
template <int DK, int DV>
struct Tiles {
  static constexpr int k = kMixBlock * DK * 2, v = kMixBlock * DV * 2;
  static constexpr int q = k > v ? k : v;  // also holds the output on its way out
  static constexpr int stage = q + k + v;
  static constexpr int state = k;  // the entering state, or before it the keys' low parts
  static constexpr int fit = (kSmemBytes - 1024 - kMiscBytes - state) / stage;
  static constexpr int stages = fit < kMaxStages ? fit : kMaxStages;
  static_assert(stages >= 2, "two stages must fit");
  static constexpr int bytes = 1024 + kMiscBytes + state + stages * stage;
};

// What the warps need of a block, in the order of the CTA's work: written with its loads.
enum BlockKind {
  kSweep = 1,  // swept; without it only summed, for the CTAs behind this one
  kFirst = 2,  // of its kind
  kLast = 4,
  kEnd = 8,    // no block: all are done
  kAbove = 16  // which of two numbers decays the state over a whole one
};
struct Block {
  int kind, row, live;       // first token, tokens
  int seq, m, blocks, len;   // number m of a sequence's blocks in the order of the sweep, its tokens
  int it;                    // number among the CTA's blocks
};
constexpr int kRing = 8;  // more than stages and the warps' distances from the loads together

struct Shared {
  uint64_t full[kMaxStages];   // a stage's keys and values are there
  uint64_t empty[kMaxStages];  // and have been read
  uint64_t q_full[kMaxStages], q_empty[kMaxStages];  // its queries; its output has left their place
  uint64_t score;              // scores in TMEM
  uint64_t weighted;           // weighted scores in TMEM
  uint64_t keys[2];            // keys of the first and last 64 tokens decayed, rows past the end cleared
  uint64_t block_state;        // the block's state in TMEM
  uint64_t entry;              // the entering state in shared memory (and values past the end cleared)
  uint64_t outer;              // queries times that state in TMEM
  uint64_t out;                // and the other part of the output; the weighted scores are read
  uint64_t taken;              // and out of it again
  uint64_t put;                // this CTA's share in memory
  uint64_t shares;             // those of all CTAs of the cluster
  Block block[kRing];          // by number
  Block sweep[kRing];          // the swept ones by theirs
  uint32_t tmem;
  int abort;
  union {
    struct {
      int place[6];            // what locate() found
      int sums[kThreads / 32];
    };
    int list[kMixDealt];       // sequences that the CTA was dealt: 32 pair + sequence, or -1
  };
  alignas(16) float fall[96];        // what weigh() needs of the powers of a
  float near_[64];                   // scale a^n, n = -32 .. 31; zeros below 0
  uint32_t key[kMixBlock + 1];       // key_scale a^n as the sum of two bf16
  float whole[2];                    // the fp32 numbers below and above a^128,
  uint32_t above;                    // and how often a block takes the latter, in 2^-32
};
static_assert(sizeof(Shared) <= kMiscBytes, "");

// a^n; 1 for n = 0 however fast the head forgets.
DM_DEV float power_of(float log_decay, int n) { return n == 0 ? 1.f : expf(log_decay * float(n)); }
DM_DEV bool gave_up(int* err, volatile int* flag) {
  *flag = 1;
  atomicExch(err, DMUON_ERR_TIMEOUT);
  return false;
}
DM_DEV bool await_long(uint64_t* bar, uint32_t parity, int* err, volatile int* flag) {
  return mbar_wait(bar, parity, flag) || gave_up(err, flag);
}
// Wait of a whole warp (or one thread); false: gave up.
DM_DEV bool await(uint64_t* bar, uint32_t parity, int* err, volatile int* flag) {
  return __builtin_expect(mbar_try_wait(smem_u32(bar), parity), 1) ||
         await_long(bar, parity, err, flag);
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
};
// n blocks on (past the batch's end: any block)
DM_DEV Cursor skipped(const LinAttnArgs& g, Cursor c, int n) {
  while (n >= c.x.blocks - c.m) {
    n -= c.x.blocks - c.m;
    c.m = 0;
    do {
      c.seq += g.against ? -1 : 1;
      if (c.seq < 0 || c.seq >= g.sequences) {
        c.seq = 0;
        c.x = Extent{0, 0, 0x7FFFFFFF};
        break;
      }
      c.x = extent_of(g, c.seq);
    } while (c.x.blocks == 0);
  }
  c.m += n;
  return c;
}
// What a CTA does: n blocks from `start` on, of the nb blocks that its cluster takes in stretches of
// `per`.
struct Work {
  int nb, per, n, rank;
  Cursor start;
};
// Blocks of all sequences are numbered in their order; sequences are dealt to the clusters of a
// head by the block that they start with, and the blocks of a cluster evenly to its CTAs.  Every
// thread counts the blocks of a run of sequences.
DM_DEV Work divide(const LinAttnArgs& g, int rank, int nb) {
  Work w;
  w.nb = nb;
  w.rank = rank;
  w.per = (nb + g.split - 1) / g.split;
  w.n = max(0, min(w.per, nb - rank * w.per));
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
  const int i = rank * w.per;
  if (w.n > 0) {
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
#pragma unroll 1
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
#pragma unroll 1
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
  const int i = rank * w.per;
  const int flat = g.against ? hi - 1 - i : lo + i;
  if (w.n > 0) {
    int at = first;
#pragma unroll 1
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

// Sequences of all heads and sweeps ("pairs"), dealt whole to `ctas` CTAs: the longest sequence's of all
// pairs first, each to the CTA with the least to do so far, then the next one's.  CTAs with equally
// much to do are runs of their numbers, a lane each: one at first, and one more for every sequence at
// most.  The first warp of each CTA deals for all; list: what its own gets.
DM_DEV void deal(const LinAttnArgs& g, int pairs, int ctas, int* list) {
  constexpr int kStart = 1;  // blocks' time that a sequence takes besides
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = int(threadIdx.x) & 31, cta = int(blockIdx.x);
  list[lane] = -1;
  __syncwarp();
  const int blocks = lane < g.sequences ? extent_of(g, lane).blocks : 0;
  int place = 0;  // among the sequences
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int other = __shfl_sync(kAll, blocks, i);
    place += other > blocks || (other == blocks && i < lane);
  }
  auto sum_upto = [&](int v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v += u;
    }
    return v;
  };
  int runs = 1, first = 0, count = lane == 0 ? ctas : 0, load = 0, left = kMixDealt;
#pragma unroll 1
  for (int n = 0; n < g.sequences; ++n) {
    const int s = __ffs(__ballot_sync(kAll, place == n)) - 1;
    const int cost = __shfl_sync(kAll, blocks, s) + kStart;
    if (cost == kStart) break;
    // sequences of a CTA of the run that start before `level`, and of all
    auto taken = [&](int level) { return level > load ? min((level - load + cost - 1) / cost, left) : 0; };
    auto total = [&](int level) { return __reduce_add_sync(kAll, count * taken(level)); };
    int lo = __reduce_min_sync(kAll, count > 0 ? load : 0x7FFFFFFF);
    int hi = __reduce_max_sync(kAll, count > 0 ? load : 0) + (pairs / ctas + 1) * cost;
    if (total(hi) < pairs) hi += pairs * cost;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (total(mid) >= pairs) hi = mid;
      else lo = mid;
    }
    // those that start before lo, and as many that start there as are left
    int takes = taken(lo);
    const int able = taken(hi) > takes ? count : 0;
    const int rest = pairs - __reduce_add_sync(kAll, count * takes);
    int more = min(max(rest - (sum_upto(able) - able), 0), able);
    const unsigned cut = __ballot_sync(kAll, more > 0 && more < count);
    if (cut != 0) {  // the one run of which some do
      const int from = __ffs(cut) - 1;
      const int m = __shfl_sync(kAll, more, from), f = __shfl_sync(kAll, first, from),
                c = __shfl_sync(kAll, count, from), l = __shfl_sync(kAll, load, from),
                e = __shfl_sync(kAll, left, from), t = __shfl_sync(kAll, takes, from);
      if (lane == from) count = m;
      if (lane == runs) {
        first = f + m;
        count = c - m;
        load = l;
        left = e;
        takes = t;
        more = 0;
      }
      ++runs;
    }
    takes += more > 0;
    const int pair = sum_upto(count * takes) - count * takes + (cta - first) * takes;
    if (cta >= first && cta < first + count)
      for (int i = 0; i < takes; ++i) list[kMixDealt - left + i] = 32 * (pair + i) + s;
    load += takes * cost;
    left -= takes;
  }
}

// ------------------------------------------------------------------ loads
// The one walk through the batch: the CTA's stretch from its last sequence on, if that goes on in
// the next CTA's, and then the whole stretch.
template <int DK, int DV>
DM_DEV void load_role(const LinAttnArgs& g, const Work& w, int head, bool again, uint8_t* smem,
                      Shared* sh) {
  using T = Tiles<DK, DV>;
  volatile int* flag = &sh->abort;
  int it = 0, swept = 0;
  // A slow head multiplies its state by a^128 thousands of times, and an error of 2^-25 with one sign
  // would add up (2^20 tokens, log_decay -1e-6: 7e-5 of the state).  So whole blocks take the fp32
  // numbers below and above a^128 in turn, as often as their mean asks for: the product of any run of
  // them is within 2^-23.
  const uint32_t above = sh->above;
  auto load = [&](const Cursor& c, int kind) {
    const int s = it % T::stages;
    const uint32_t parity = ((it / T::stages) & 1) ^ 1;
    uint8_t* q = smem + s * T::stage;
    uint8_t *k = q + T::q, *v = k + T::k;
    const Block b{kind | (uint32_t(c.m + 1) * above < above ? kAbove : 0), c.row(g), c.live(g), c.seq, c.m,
                  c.x.blocks, c.x.len, it};
    sh->block[it % kRing] = b;
    if (kind & kSweep) sh->sweep[swept++ % kRing] = b;
    if (!await(&sh->empty[s], parity, g.err, flag)) return false;
    if (kind & kEnd) {
      mbar_arrive(&sh->full[s]);
    } else {
      mbar_arrive_expect_tx(&sh->full[s], uint32_t(T::k + T::v));
#pragma unroll
      for (int p = 0; p < DK / 64; ++p)
        tma_load_3d(k + p * 16384, &g.k, &sh->full[s], p * 64, head, b.row);
#pragma unroll
      for (int p = 0; p < DV / 64; ++p)
        tma_load_3d(v + p * 16384, &g.v, &sh->full[s], p * 64, head, b.row);
    }
    if (!await(&sh->q_empty[s], parity, g.err, flag)) return false;
    if (kind & kSweep) {
      mbar_arrive_expect_tx(&sh->q_full[s], uint32_t(T::k));
#pragma unroll
      for (int p = 0; p < DK / 64; ++p)
        tma_load_3d(q + p * 16384, &g.q, &sh->q_full[s], p * 64, head, b.row);
    } else {
      mbar_arrive(&sh->q_full[s]);
    }
    ++it;
    return true;
  };
  Cursor at = w.start;
  if (w.rank + 1 < g.split && w.n > 0) {
    Cursor c = skipped(g, at, w.n - 1);
    if (c.m + 1 < c.x.blocks) {
      const int ahead = min(c.m + 1, w.n);
      c.m -= ahead - 1;
#pragma unroll 1
      for (int i = 0; i < ahead; ++i, ++c.m)
        if (!load(c, (i == 0 ? kFirst : 0) | (i + 1 == ahead ? kLast : 0))) return;
    }
  }
#pragma unroll 1
  for (int i = 0; i < w.n; ++i) {
    if (!load(at, kSweep | (i == 0 ? kFirst : 0))) return;
    if (i + 1 < w.n) at = skipped(g, at, 1);
  }
  if (!load(at, kEnd) || !again) return;
  // all of the stages have been read: what arrives on their barriers has
#pragma unroll 1
  for (int i = max(0, it - 1 - T::stages); i < it - 1; ++i) {
    const int s = i % T::stages;
    if (!await(&sh->empty[s], (i / T::stages) & 1, g.err, flag)) return;
    if (!await(&sh->q_empty[s], (i / T::stages) & 1, g.err, flag)) return;
  }
}

// ------------------------------------------------------------------ products
// Two threads issue them, as issuing takes about as long as computing: one the blocks' own states,
// one the rest.  (A third for the scores alone: 140 us where two took 131, 152 heads of 5120
// tokens; scores in two TMEM buffers, the next ones multiplied while these are weighted: 143.)
template <int DK, int DV, bool EXACT>
DM_DEV void state_mma_role(const LinAttnArgs& g, uint8_t* smem, uint8_t* state, Shared* sh) {
  using T = Tiles<DK, DV>;
  volatile int* flag = &sh->abort;
  constexpr uint32_t id = idesc_bf16(128, DV, true, true);
  const uint32_t to = sh->tmem + kColState;
  // (a^..k)^T V, rows of K in steps of 16 tokens.  With 64 key elements the upper half of the
  // 128 rows reads what follows the tile; those lanes of the result are not used.
  auto product = [&](uint32_t k, uint32_t v, int half, bool accumulate) {
    const uint64_t a = sdesc_sw128(k, 16384, 1024) + uint64_t(half) * 512,
                   b = sdesc_sw128(v, 16384, 1024) + uint64_t(half) * 512;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      umma_bf16(to, a + uint64_t(j) * 128, b + uint64_t(j) * 128, id, accumulate || j > 0);
  };
#pragma unroll 1
  for (int it = 0;; ++it) {
    const int s = it % T::stages;
    const uint32_t q = smem_u32(smem) + s * T::stage, k = q + T::q, v = k + T::k;
    if (!await(&sh->full[s], (it / T::stages) & 1, g.err, flag)) return;
    const int kind = sh->block[it % kRing].kind;
    if (kind & kEnd) return;
    // the keys' low parts lie where queries would, or the state that enters did
    const uint32_t low = kind & kSweep ? smem_u32(state) : q;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // the last block's state is added by then
      if (!await(&sh->keys[half], it & 1, g.err, flag)) return;
      tc_fence_after();
      product(k, v, half, half > 0);
      if (EXACT) product(low, v, half, true);
    }
    umma_commit(&sh->block_state);
    umma_commit(&sh->empty[s]);
    if (!(kind & kSweep)) {  // in the place of the output's warps
#pragma unroll
      for (int n = 0; n < kOutWarps; ++n) umma_commit(&sh->q_empty[s]);
    }
  }
}
template <int DK, int DV>
DM_DEV void out_mma_role(const LinAttnArgs& g, uint8_t* smem, uint8_t* state, Shared* sh) {
  using T = Tiles<DK, DV>;
  volatile int* flag = &sh->abort;
  const uint32_t tmem = sh->tmem;
  constexpr uint32_t id_score = idesc_bf16(128, 128, false, false);
  constexpr uint32_t id_out = idesc_bf16(128, DV, false, true);
  const uint64_t ed = sdesc_sw128(smem_u32(state), DK * 128, 1024);
  int swept = 0;
#pragma unroll 1
  for (int it = 0;; ++it) {
    const int s = it % T::stages;
    const uint32_t q = smem_u32(smem) + s * T::stage, k = q + T::q, v = k + T::k;
    const uint64_t qd = sdesc_sw128(q, 16, 1024), kd = sdesc_sw128(k, 16, 1024);
    if (!await(&sh->full[s], (it / T::stages) & 1, g.err, flag)) return;
    const int kind = sh->block[it % kRing].kind;
    if (kind & kEnd) {
      if (swept > 0) (void)await(&sh->outer, (swept - 1) & 1, g.err, flag);
      return;
    }
    if (!await(&sh->q_full[s], (it / T::stages) & 1, g.err, flag)) return;
    if (!(kind & kSweep)) {
      mbar_arrive(&sh->empty[s]);  // waited for all the same: a wait misses no phase
      continue;
    }
    // the last block's weighted scores have been read (no order is promised between products of
    // unlike shape)
    if (swept > 0 && !await(&sh->out, (swept - 1) & 1, g.err, flag)) return;
    tc_fence_after();
#pragma unroll
    for (int j = 0; j < DK / 16; ++j) {
      const uint64_t at = uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2;
      umma_bf16(tmem + kColScore, qd + at, kd + at, id_score, j > 0);
    }
    umma_commit(&sh->score);
    mbar_arrive(&sh->score);  // and with it what lies in sh->sweep, seen by this thread
    // the state's part while the scores are weighted
    if (swept > 0 && !await(&sh->taken, (swept - 1) & 1, g.err, flag)) return;
    if (!await(&sh->entry, swept & 1, g.err, flag)) return;
    tc_fence_after();
#pragma unroll
    for (int j = 0; j < DK / 16; ++j)
      umma_bf16(tmem + kColOuter, qd + uint64_t(j >> 2) * 1024 + uint64_t(j & 3) * 2,
                ed + uint64_t(j) * 128, id_out, j > 0);
    umma_commit(&sh->outer);
    if (!await(&sh->weighted, swept & 1, g.err, flag)) return;
    tc_fence_after();
    const uint64_t vd = sdesc_sw128(v, 16384, 1024);
#pragma unroll
    for (int j = 0; j < 8; ++j)  // 8 columns of weighted scores a step, in two halves
      umma_bf16_ts(tmem + kColInner, tmem + kColScore + (j >> 2) * 64 + (j & 3) * 8,
                   vd + uint64_t(j) * 128, id_out, j > 0);
    umma_commit(&sh->out);
    mbar_arrive(&sh->out);
    umma_commit(&sh->empty[s]);
    ++swept;
  }
}

// ------------------------------------------------------------------ states
// Thread (warp w, lane) keeps row 32 (w % 4) + lane of the state, columns DV / 2 (w / 4) on.
template <int DK, int DV, bool EXACT>
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

  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  DM_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) st[i] = 0;
  }
  DM_DEV long long state_at(int seq) const { return ((long long)seq * g.heads + head) * g.dk * g.dv; }
  // A caller's state: four elements of a row at a time, or (transposed) one, rows side by side.
  DM_DEV void read_initial(int seq) {
    if (g.state_in == nullptr || row >= g.dk) return;
    const float* p = g.state_in + state_at(seq) + row * g.st_row + col * g.st_col;
    if (g.st_col == 1) {
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i)
        if (col + 4 * i < g.dv) {
          const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
          st[2 * i] = f2(v.x, v.y);
          st[2 * i + 1] = f2(v.z, v.w);
        }
    } else {
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i, p += 2 * g.st_col)
        if (col + 2 * i < g.dv) st[i] = f2(p[0], p[g.st_col]);
    }
  }
  DM_DEV void write_final(int seq) {  // of the gradients' sweeps only dv's has one: never transposed
    if (row >= g.dk) return;
    float* p = g.state_out + state_at(seq) + row * g.st_row + col;
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      float4 v;
      f2_split(st[2 * i], v.x, v.y);
      f2_split(st[2 * i + 1], v.z, v.w);
      if (col + 4 * i < g.dv) *reinterpret_cast<float4*>(p + 4 * i) = v;
    }
  }
  // A state in the workspace, four columns at a time so that a warp's rows lie together.  Slots of
  // a CTA: its share, and a copy of the first state of the sequence that it begins and others end.
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
  // A final state may be written over the first one while other CTAs have yet to read that.
  DM_DEV bool over() const { return g.split > 1 && g.state_in != nullptr && g.state_in == g.state_out; }
  DM_DEV void keep_initial(int seq) {
    float4* to = slot(w.rank, 1);
    const float* p = g.state_in + state_at(seq) + row * g.st_row + col * g.st_col;
#pragma unroll 1
    for (int i = 0; i < kCols / 4; ++i, p += 4 * g.st_col) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < g.dk && col + 4 * i < g.dv)
        v = make_float4(p[0], p[g.st_col], p[2 * g.st_col], p[3 * g.st_col]);
      __stcg(to + i * 128, v);
    }
  }
  // tokens of the first n of a sequence's blocks in the order of the sweep
  DM_DEV int before(const Block& b, int n) const {
    return g.against ? b.len - min(b.len, (b.blocks - n) * kMixBlock) : min(b.len, n * kMixBlock);
  }
  // The state before block b: a sequence's first state, and for a CTA that begins inside the
  // sequence the shares of the CTAs before it.
  DM_DEV void enter(const Block& b, bool first, int share_seq) {
    const bool inside = first && b.m > 0;
    const int start = w.rank * w.per - b.m;  // sweep's number of the sequence's first block
    const int from = inside ? start / w.per : w.rank;
    zero();
    const float4* p = nullptr;
    if (over() && (inside || b.seq == share_seq)) p = slot(from, 1);
    else read_initial(b.seq);
    // lane r: the decay over rank r's part of the sequence
    const int n0 = max(lane * w.per - start, 0), n1 = (lane + 1) * w.per - start;
    const float decay =
        lane >= from && lane < w.rank ? expf(log_decay * float(before(b, n1) - before(b, n0))) : 0.f;
    constexpr int kPart = 4;  // of 4 columns each, so that several ranks' loads are in flight
#pragma unroll
    for (int i0 = 0; i0 < kCols / 4; i0 += kPart) {
      if (p != nullptr) {
#pragma unroll
        for (int i = i0; i < i0 + kPart; ++i) {
          const float4 v = __ldcg(p + i * 128);
          st[2 * i] = f2(v.x, v.y);
          st[2 * i + 1] = f2(v.z, v.w);
        }
      }
#pragma unroll 2
      for (int r = from; r < w.rank; ++r) {
        const float f = __shfl_sync(0xffffffffu, decay, r);
        const F2 ff = f2(f, f);
        const float4* q = slot(r, 0);
#pragma unroll
        for (int i = i0; i < i0 + kPart; ++i) {
          const float4 v = __ldcg(q + i * 128);
          st[2 * i] = fma2(ff, st[2 * i], f2(v.x, v.y));
          st[2 * i + 1] = fma2(ff, st[2 * i + 1], f2(v.z, v.w));
        }
      }
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
  DM_DEV uint32_t key_weight(int j, int live) const {
    return j >= live ? 0u : sh->key[g.against ? j + 1 : live - 1 - j];
  }
  // Keys of block `it` times their decay, in place; what bf16 drops of them (EXACT) to `low`.  The
  // decay is kept as a sum of two bf16 numbers, so that k a = k a_0 + k a_1 is rounded like an fp32
  // product, two elements at a time, and what its rounding drops comes with two more products.
  // Rows past the end hold another sequence's tokens, or anything: they become zeros.
  DM_DEV void keys(int it, int live, uint32_t low) {
    const uint32_t stage = smem_u32(smem) + (it % T::stages) * T::stage + tid * 16;
    low += tid * 16;
    // tokens 0 .. 63, then the rest: the products of the first half start while the second is made
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      constexpr int kBatch = kUnits / 2;  // loads in flight: two tokens, in one or two panels
      uint32_t x[kBatch][4];
      auto unit = [&](int b) { return (half * 2 + (b & 1) + (b >> 1) * 4) * kThreadsHere * 16; };
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        ld_shared_v4(stage + T::q + unit(b), x[b][0], x[b][1], x[b][2], x[b][3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = token_of(half * 2 + e);
        const uint32_t w = key_weight(j, live), mask = j < live ? 0xFFFFFFFFu : 0u;
        const uint32_t w0 = __byte_perm(w, 0, 0x1010), w1 = __byte_perm(w, 0, 0x3232);
#pragma unroll
        for (int b = e; b < kBatch; b += 2) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t k = x[b][i] & mask;
            x[b][i] = bf16_fma2(k, w0, bf16_mul2(k, w1));
            if (EXACT) y[i] = bf16_fma2(k, w1, bf16_fma2(k, w0, x[b][i] ^ 0x80008000u));
          }
          st_shared_v4(stage + T::q + unit(b), x[b][0], x[b][1], x[b][2], x[b][3]);
          if (EXACT) st_shared_v4(low + unit(b), y[0], y[1], y[2], y[3]);
        }
      }
      announce(&sh->keys[half]);
    }
  }
  // Rows of values past a sequence's end become zeros, too.
  DM_DEV void clear_values(const Block& b) {
    if (__builtin_expect(b.live == kMixBlock, 1)) return;
    const uint32_t at = smem_u32(smem) + (b.it % T::stages) * T::stage + T::q + T::k + tid * 16;
#pragma unroll 1
    for (int n = 0; n < kMixBlock * DV / 8 / kThreadsHere; ++n)
      if (token_of(n) >= b.live) st_shared_v4(at + n * kThreadsHere * 16, 0, 0, 0, 0);
  }
  DM_DEV bool block_done(int it) { return wait(&sh->block_state, it); }
  // A block joins the state.
  DM_DEV void add_block(const Block& b) {
    tc_fence_after();
    const float f = b.live == kMixBlock ? sh->whole[(b.kind & kAbove) != 0] : expf(log_decay * float(b.live));
    const F2 ff = f2(f, f);
    const uint32_t at = sh->tmem + (uint32_t(row & ~31) << 16) + kColState + col;
    float x[2][16];
    tmem_ld16(at, x[0]);
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
      tmem_ld_wait();
      if (c + 1 < kCols / 16) tmem_ld16(at + (c + 1) * 16, x[(c + 1) & 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st[c * 8 + i] = fma2(ff, st[c * 8 + i], f2(x[c & 1][2 * i], x[c & 1][2 * i + 1]));
    }
    if (row >= g.dk) zero();  // of keys past the head's size: 0 times an infinity of V may be there
    tc_fence_before();
  }
  // This CTA's share is in memory (or it has none): tell the cluster.
  DM_DEV bool arrive() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->put);
    if (tid < 32) {
      if (!wait(&sh->put, 0)) return false;
      if (tid < g.split) mbar_arrive_cluster(mapa_shared(smem_u32(&sh->shares), uint32_t(tid)));
      __syncwarp();
    }
    return true;
  }
  DM_DEV bool all_arrived() {
    return mbar_wait_cluster(&sh->shares, 0, &sh->abort) || gave_up(g.err, &sh->abort);
  }
  // What a block needs before its keys, ahead of the sweep and in it.
  DM_DEV bool begin_share(const Block& b) {
    if (b.kind & kFirst) {
      if (over() && b.m == 0) keep_initial(b.seq);
      zero();
    }
    clear_values(b);
    // the low parts go where queries would be, once the output before them has left
    return wait(&sh->q_full[b.it % T::stages], b.it / T::stages);
  }
  DM_DEV bool begin_sweep(const Block& b, int swept, int share_seq) {
    const bool first = (b.kind & kFirst) != 0;
    if (__builtin_expect(b.m == 0 || first, 0)) {
      if (first && b.m > 0 && !all_arrived()) return false;
      enter(b, first, share_seq);
    }
    clear_values(b);
    // The scores are there, so the last block's products are done and with them (exact: since its
    // low parts were read) the place of the state that enters is free.
    if (!wait(&sh->score, swept)) return false;
    write_entry();
    return !EXACT || wait(&sh->outer, swept);  // the low parts take that place
  }
  DM_DEV void run() {
    zero();
    int swept = 0, share_seq = -1;
    if (!wait(&sh->full[0], 0)) return;
    Block b = sh->block[0];
    if (g.split > 1 && (b.kind & (kEnd | kSweep)) != 0 && !arrive()) return;  // it has no share
#pragma unroll 1
    for (int it = 0; (b.kind & kEnd) == 0; ++it) {
      const int s = it % T::stages, s1 = (it + 1) % T::stages;
      const bool sweep = (b.kind & kSweep) != 0;
      if (__builtin_expect(sweep, 1)) {
        if (!begin_sweep(b, swept, share_seq)) return;
        ++swept;
      } else {
        if (!begin_share(b)) return;
        share_seq = b.seq;
      }
      keys(it, b.live, sweep ? smem_u32(entry) : smem_u32(smem) + s * T::stage);
      // while the product runs, the next block
      if (!wait(&sh->full[s1], (it + 1) / T::stages)) return;
      const Block next = sh->block[(it + 1) % kRing];
      if (!block_done(it)) return;
      add_block(b);
      if (EXACT && __builtin_expect(sweep && g.state_out != nullptr && b.m + 1 == b.blocks, 0))
        write_final(b.seq);
      if (__builtin_expect((b.kind & kLast) != 0, 0)) {
        put(slot(w.rank, 0));
        if (!arrive()) return;
      }
      b = next;
    }
  }
  // Sequences without tokens: their states pass through.
  DM_DEV void pass_through(int first, int stride) {
#pragma unroll 1
    for (int s = first; s < g.sequences; s += stride) {
      if (extent_of(g, s).blocks != 0) continue;
      const long long at = state_at(s);
#pragma unroll 1
      for (int i = tid; i < g.dk * g.dv; i += kThreadsHere)
        g.state_out[at + i] = g.state_in == nullptr ? 0.f : g.state_in[at + i];
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
  float log_decay;
  int warp, lane;

  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  // Columns j0 .. j0 + 31 of x, weighted, to p.
  template <bool AGAINST>
  DM_DEV void weigh(const float (&x)[32], int q, int j0, int live, F2 own, uint32_t (&p)[16]) {
    const int b = j0 >> 5;
    if (b == q) {
      const float* t = sh->near_ + 32 + (AGAINST ? -lane : lane);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        p[i] = pack_bf16(x[2 * i] * t[AGAINST ? 2 * i : -2 * i],
                         x[2 * i + 1] * t[AGAINST ? 2 * i + 1 : -2 * i - 1]);
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
    if (b == q || (AGAINST && j0 + 32 > live)) {
      // columns that the row sees, a bit each: whatever the others hold becomes 0
      uint32_t see = b != q ? 0xFFFFFFFFu : AGAINST ? 0xFFFFFFFFu << lane : 0xFFFFFFFFu >> (31 - lane);
      if (AGAINST && j0 + 32 > live) see &= 0xFFFFFFFFu >> (j0 + 32 - live);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // two bits to a mask of two halves
        const uint32_t two = see >> (2 * i) & 3u;
        p[i] &= (two & 1u) * 0xFFFFu + (two >> 1) * 0xFFFF0000u;
      }
    }
  }
  template <bool AGAINST>
  DM_DEV bool block(int swept, F2 own) {
    const int q = warp & 3, c0 = (warp >> 2) * 64;
    const uint32_t at = sh->tmem + (uint32_t(q * 32) << 16) + kColScore + c0;
    if (!wait(&sh->score, swept)) return false;
    tc_fence_after();
    const int live = sh->sweep[swept % kRing].live;
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
    const float f = g.scale * power_of(log_decay, g.against ? 31 - lane : lane);
    const F2 own = f2(f, f);
    const int n = w.n;
    if (g.against) {
#pragma unroll 1
      for (int swept = 0; swept < n && block<true>(swept, own); ++swept) {
      }
    } else {
#pragma unroll 1
      for (int swept = 0; swept < n && block<false>(swept, own); ++swept) {
      }
    }
  }
};

// ------------------------------------------------------------------ outputs
// Thread (warp w, lane) has row 32 w + lane.  The weighted scores carry the scale already.
template <int DK, int DV>
struct OutRole {
  using T = Tiles<DK, DV>;
  const LinAttnArgs& g;
  const Work& w;
  Shared* sh;
  uint8_t* smem;
  float log_decay;
  int head, warp, lane;
  float whole;  // weight of a whole block

  DM_DEV bool wait(uint64_t* bar, int n) { return await(bar, n & 1, g.err, &sh->abort); }
  // of the entering state in the thread's row of a block of `live` tokens
  DM_DEV float weight(int live) const {
    const int row = warp * 32 + lane;
    return row < live ? g.state_scale * power_of(log_decay, g.against ? live - 1 - row : row + 1) : 0.f;
  }
  // The store of the last block has left stage s.
  DM_DEV void release(int s) {
    if (lane == 0) {
      bulk_wait_read<0>();
      mbar_arrive(&sh->q_empty[s]);
    }
  }
  DM_DEV bool block(int swept) {
    if (!wait(&sh->out, swept)) return false;
    tc_fence_after();
    const Block& b = sh->sweep[swept % kRing];
    const int live = b.live, row0 = b.row, s = b.it % T::stages;
    const float f = __builtin_expect(live == kMixBlock, 1) ? whole : weight(live);
    const F2 ff = f2(f, f);
    const uint32_t at = sh->tmem + (uint32_t(warp * 32) << 16);
    // 32 columns to a piece of 2 KB, rows of 64 bytes
    const uint32_t tile = smem_u32(smem) + s * T::stage + warp * (DV / 32) * 2048 + lane * 64;
#pragma unroll 1
    for (int n = 0; n < DV / 16; ++n) {
      float x[16], y[16];
      tmem_ld16(at + kColInner + n * 16, x);
      tmem_ld16(at + kColOuter + n * 16, y);
      tmem_ld_wait();
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = pack_bf16(fma2(ff, f2(y[2 * e], y[2 * e + 1]), f2(x[2 * e], x[2 * e + 1])));
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
    // TMA reads what was written, or (all rows or some past the end) writes queries over it
    fence_proxy_async_smem();
    if (__builtin_expect(rows >= 32, 1)) {
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int n = 0; n < DV / 32; ++n)
          if (n * 32 < g.dv) tma_store_3d(&g.o, tile + n * 2048, n * 32, head, first);
        bulk_commit();
      }
    } else {
      // the end of a sequence: what lies behind it is not this one's to write
      __syncwarp();
      const uint32_t base = tile - lane * 64;
#pragma unroll 1
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
    release(s);
    return true;
  }
  DM_DEV void run() {
    const int n = w.n;
    whole = weight(kMixBlock);
#pragma unroll 1
    for (int swept = 0; swept < n && block(swept); ++swept) {
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
};

// All warps, each from its own branch.
DM_DEV void sync_roles() { asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory"); }

template <int DK, int DV, bool EXACT>
__global__ void __launch_bounds__(kThreads, 1) mix_kernel(const __grid_constant__ LinAttnSweeps sweeps) {
  extern __shared__ uint8_t smem_raw[];
  using T = Tiles<DK, DV>;
  // the state's tile, the stages (of which products read when they run past that tile's end), the rest
  uint8_t* state = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t* smem = state + T::state;
  Shared* sh = reinterpret_cast<Shared*>(smem + T::stages * T::stage);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
  const int split = sweeps.sweep[0].split, heads = sweeps.sweep[0].heads, ctas = sweeps.deal;
  const int cluster = ctas > 0 ? 0 : int(blockIdx.x) / split, rank = int(blockIdx.x) - cluster * split;
  const int of_sweep = sweeps.sweep[0].groups * heads;
  const LinAttnArgs* at = &sweeps.sweep[cluster / of_sweep];
  const int group = cluster % of_sweep / heads;
  int head = cluster % of_sweep - group * heads;
  auto init_barriers = [&]() {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 2);
      mbar_init(&sh->q_full[s], 1);
      mbar_init(&sh->q_empty[s], kOutWarps);
    }
    mbar_init(&sh->keys[0], kStateWarps);
    mbar_init(&sh->keys[1], kStateWarps);
    mbar_init(&sh->block_state, 1);
    mbar_init(&sh->score, 2);
    mbar_init(&sh->weighted, kWeighWarps);
    mbar_init(&sh->outer, 1);
    mbar_init(&sh->entry, kStateWarps);
    mbar_init(&sh->out, 2);
    mbar_init(&sh->taken, kOutWarps);
    mbar_init(&sh->put, kStateWarps);
    mbar_init(&sh->shares, uint32_t(split));
    fence_barrier_init();
  };
  if (threadIdx.x == 0) {
    sh->abort = 0;
    init_barriers();
  }
  if (warp == kOutMmaWarp) {
    tmem_alloc(&sh->tmem, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && elect_one()) {
    prefetch_tensormap(&at->q);
    prefetch_tensormap(&at->k);
    prefetch_tensormap(&at->v);
    prefetch_tensormap(&at->o);
  }
  if (split > 1) cluster_sync();  // barriers of all CTAs stand before one arrives on another's
  grid_wait();
  grid_launch_dependents();
  Work w;
  if (ctas > 0) {
    if (warp == 0) deal(*at, sweeps.count * heads, ctas, sh->list);
    __syncthreads();
  } else {
    w = at->sequences <= 32 ? locate_few(*at, group, rank) : locate(*at, group, rank, sh);
  }
  float log_decay = 0.f;
  auto begin = [&](int unit) {
    if (ctas > 0) {
      const int u = sh->list[unit];
      const int pair = max(u, 0) >> 5, sweep = pair / heads;
      at = &sweeps.sweep[sweep];
      head = pair - sweep * heads;
      w.start.seq = u & 31;
      w.start.m = 0;
      w.start.x = u < 0 ? Extent{0, 0, 0x7FFFFFFF} : extent_of(*at, u & 31);
      w.nb = w.per = w.n = u < 0 ? 0 : w.start.x.blocks;
      w.rank = 0;
    }
    const LinAttnArgs& g = *at;
    log_decay = g.log_decay[head];
    const int t = int(threadIdx.x);
    if (t <= kMixBlock) {
      const float f = g.key_scale * power_of(log_decay, t), high = bf16_lo(pack_bf16(f, f));
      sh->key[t] = pack_bf16(high, f - high);
    } else if (t < kMixBlock + 1 + 64) {
      const int n = t - kMixBlock - 1 - 32;
      sh->near_[n + 32] = n < 0 ? 0.f : g.scale * power_of(log_decay, n);
    } else if (t < kMixBlock + 1 + 64 + 96) {
      const int n = t - kMixBlock - 1 - 64;
      sh->fall[n] = expf(log_decay * float(g.against ? n + 1 : 96 - n));
    } else if (t == kMixBlock + 1 + 64 + 96) {
      // a^128 = 1 + e = f + rest, exactly; a rounding below 0.57 does not outlast a few blocks
      const float z = log_decay * float(kMixBlock), e = expm1f(z);
      float f = 1.f + e, above = 0.f;
      if (z <= 0.f && f > 0.57f) {
        const float rest = e - (f - 1.f);
        if (rest < 0.f) f -= 0x1p-24f;
        above = fminf((rest < 0.f ? rest + 0x1p-24f : rest) * 0x1p56f, 0x1.fffffep31f);
      } else {
        f = expf(z);
      }
      sh->whole[0] = f;
      sh->whole[1] = f + 0x1p-24f;
      sh->above = uint32_t(above);
    }
  };
  begin(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Between sequences that a CTA was dealt everything stops, and starts as in a new launch.
  auto more = [&](int unit) { return ctas > 0 && unit < kMixDealt && sh->list[unit] >= 0; };
  auto next = [&](int unit) {
    if (!more(unit)) return false;
    tc_fence_before();
    sync_roles();
    if (*const_cast<volatile int*>(&sh->abort) != 0) return false;
    if (threadIdx.x == 0) {
      for (uint64_t* bar = sh->full; bar <= &sh->shares; ++bar) mbar_inval(bar);
      init_barriers();
    }
    begin(unit);
    sync_roles();
    tc_fence_after();
    return true;
  };
  int unit = 0;
  if (warp < kStateWarps) {
    regs_inc<state_regs(EXACT)>();
    do {
      StateRole<DK, DV, EXACT> r{*at, w, sh, smem, state, log_decay, head, cluster, int(threadIdx.x),
                                 int(threadIdx.x & 31), int((warp & 3) * 32 + (threadIdx.x & 31)),
                                 int(warp >> 2) * (DV / 2)};
      r.run();
      if (EXACT && ctas == 0 && at->state_out != nullptr)
        r.pass_through(group * split + rank, at->groups * split);
    } while (next(++unit));
  } else if (warp < kOutWarp) {
    regs_dec<weigh_regs(EXACT)>();
    do {
      WeighRole r{*at, w, sh, log_decay, warp - kWeighWarp, int(threadIdx.x & 31)};
      r.run();
    } while (next(++unit));
  } else if (warp < kLoadWarp) {
    regs_dec<kOutRegs>();
    do {
      OutRole<DK, DV> r{*at, w, sh, smem, log_decay, head, warp - kOutWarp, int(threadIdx.x & 31)};
      r.run();
    } while (next(++unit));
  } else {
    regs_dec<kOtherRegs>();
    do {
      if (warp == kLoadWarp && elect_one()) load_role<DK, DV>(*at, w, head, more(unit + 1), smem, sh);
      if (warp == kStateMmaWarp && elect_one()) state_mma_role<DK, DV, EXACT>(*at, smem, state, sh);
      if (warp == kOutMmaWarp && elect_one()) out_mma_role<DK, DV>(*at, smem, state, sh);
      __syncwarp();
    } while (next(++unit));
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
  if (warp == kOutMmaWarp) {
    tc_fence_after();
    tmem_dealloc(sh->tmem, kTmemCols);
  }
  if (split > 1) cluster_sync();  // no CTA leaves while another may still arrive on its barrier
}

using MixKernel = void (*)(LinAttnSweeps);
template <int DK, int DV>
MixKernel kernel_of(bool exact, int* smem) {
  *smem = Tiles<DK, DV>::bytes;
  return exact ? mix_kernel<DK, DV, true> : mix_kernel<DK, DV, false>;
}
MixKernel kernel_for(int dk, int dv, bool exact, int* smem) {
  if (dk <= 64) return dv <= 64 ? kernel_of<64, 64>(exact, smem) : kernel_of<64, 128>(exact, smem);
  return dv <= 64 ? kernel_of<128, 64>(exact, smem) : kernel_of<128, 128>(exact, smem);
}

}  // namespace

cudaError_t linattn_prepare(int (&fit)[kMixMaxSplit + 1]) {
  for (int i = 0; i < 8; ++i) {
    int smem = 0;
    const MixKernel k = kernel_for(i & 1 ? 128 : 64, i & 2 ? 128 : 64, (i & 4) != 0, &smem);
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes a{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
    if (e != cudaSuccess) return e;
    // launched with fewer, the states' warps would wait for theirs forever
    if (a.numRegs != kRegs) return cudaErrorInvalidKernelImage;
    if (i > 0) continue;  // one CTA to an SM in all of them, so as many clusters fit
    fit[0] = 0;
    for (int split = 1; split <= kMixMaxSplit; ++split) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(unsigned(split), 1, 1);
      cfg.blockDim = dim3(kThreads, 1, 1);
      cfg.dynamicSmemBytes = size_t(smem);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(split);
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit[split], k, &cfg);
      if (e != cudaSuccess) return e;
      if (fit[split] < 1) return cudaErrorInvalidConfiguration;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_linattn(const LinAttnSweeps& g, cudaStream_t s) {
  const LinAttnArgs& one = g.sweep[0];
  int smem = 0;
  const MixKernel k = kernel_for(one.dk, one.dv, one.exact != 0, &smem);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(g.deal > 0 ? g.deal : g.count * one.groups * one.heads * one.split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(one.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = one.split > 1 ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, k, g));
}

}  // namespace dm
