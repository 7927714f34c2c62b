// C ABI of the training-side operators: argument checks, workspace layout, tensor
// maps and launch sequences.  See include/dmuon.h.
#include "dmuon.h"
#include "launch.h"
#include "train.h"

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <mutex>

namespace dm {
namespace {

constexpr size_t kHdrBytes = 256;  // workspace header: device error word
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTokens = int64_t(1) << 22, kMaxDim = int64_t(1) << 19,
                  kMaxVocab = int64_t(1) << 22;
// Gradients of the logits are formed for as many tokens at a time as fit here
// (a multiple of 256, at least 256); the loss alone keeps no logits and only
// bounds the group statistics.
constexpr size_t kLogitBytes = size_t(2200) << 20;
constexpr int64_t kLossTokens = 16384;
// The tensor core's truncation takes up to K * 2^-27.5 of a sum of one sign (pair_gemm.cu).
// Sums over tokens are cut at 2^16 of them (2^20 at once: 5.4e-3 of a weight gradient
// missing, more than its rounding to bf16; of 2^16, a sixteenth of that), the parts added in
// fp32.  A sum over more than 2^18 vocabulary entries is cut into parts of at most 2^17;
// usual vocabularies stay whole (152064: up to 8e-4, a fifth of the rounding).
constexpr int64_t kSumTokens = 1 << 16, kVocabWhole = 1 << 18, kVocabPart = 1 << 17;

using bf16 = __nv_bfloat16;

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Row pitch of what the workspace holds: whole 128-byte lines, so that a box row of a
// TMA copy touches one (with rows of 16-byte multiples only, 390 us against 304 for the
// logits of 2443 tokens, 2259 x 50119).
int64_t pitch(int64_t v) { return (v + 63) / 64 * 64; }
int64_t up32(int64_t v) { return (v + 31) / 32 * 32; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool all_aligned(size_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

// Ready the current device: the products' shared memory opt-in, once.
int device_ready(int* max_clusters) {
  int d = 0, sms = 0;
  const int st = library_device(&d, &sms, max_clusters);
  if (st != DMUON_OK) return st;
  static std::mutex mu;
  static bool ready[kMaxDevices] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (!ready[d]) {
    if (lin_prepare() != cudaSuccess) return DMUON_ERR_CUDA;
    ready[d] = true;
  }
  return DMUON_OK;
}

// Hands out 256-byte aligned pieces of a workspace (base may be null: sizes only).
struct Carve {
  unsigned char* base;
  size_t used = 0;
  explicit Carve(void* b) : base(static_cast<unsigned char*>(b)) {}
  template <typename T>
  T* take(size_t bytes) {
    T* p = base == nullptr ? nullptr : reinterpret_cast<T*>(base + used);
    used = align_up(used + bytes, 256);
    return p;
  }
};

// The part of every workspace that the products use.
struct ProductSpace {
  int* err;
  float* partial;
};
ProductSpace take_product_space(Carve& c) {
  ProductSpace s;
  s.err = c.take<int>(kHdrBytes);
  s.partial = c.take<float>(lin_partial_bytes());
  return s;
}

// One launch under construction.
struct Launch {
  LinArgs g{};
  int n_maps = 0;
  int k_box = 128;  // K rows in a box of an MN-major weight: a stage's
  bool ok = true;

  explicit Launch(const ProductSpace& s, LinEarly early = kEarlyNone) {
    g.err = s.err;
    g.partial = s.partial;
    g.early = early;
  }
  int map(const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols, int box_rows,
          CUtensorMapSwizzle swizzle, int elem = 2) {
    const TensorMapEncode enc = library_tensor_map_encoder();
    if (enc == nullptr || n_maps >= kLinMaps) {
      ok = false;
      return 0;
    }
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * cuuint64_t(elem)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)}, es[2] = {1, 1};
    ok = ok && enc(&g.maps[n_maps],
                   elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    return n_maps++;
  }
  // An operand stored as `rows` rows of `cols` contiguous elements; whether it is
  // K-major or MN-major, a box is 64 columns x 128 rows (swapped: half the tile's
  // tokens, the stage's 64 K rows of an MN-major weight, 64 rows each of gate and up).
  int operand(const bf16* p, int64_t cols, int64_t rows, int64_t ld, int box_rows = 128) {
    return map(p, cols, rows, ld, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  int output(const bf16* p, int64_t cols, int64_t rows, int64_t ld, bool wide = false) {
    return wide ? map(p, cols, rows, ld, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B)
                : map(p, cols, rows, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  int output_codes(const void* p, int64_t cols, int64_t rows) {
    return map(p, cols, rows, cols, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE, 1);
  }
  LinProblem& problem(int epi, int64_t rows, int64_t cols, int64_t k0, int64_t k1) {
    const int k = lin_stage_k(epi, g.swap != 0);
    LinProblem& P = g.prob[g.n_prob++];
    P.rows = int(rows);
    P.cols = int(cols);
    P.tiles_m = int(ceil_div(rows, 256));
    P.tiles_n = int(ceil_div(cols, 256));
    P.kb0 = int(ceil_div(k0, k));
    P.kb1 = int(ceil_div(k1, k));
    P.c_map = -1;
    return P;
  }
  // A weight gradient: rows x cols = left^T right, summed over the tokens.  A box takes
  // TMA as long for rows past the tensor's end as for rows inside, so the last K block has
  // maps of its own, with just its rows (5 tokens, 3584 x 152064: 212 us with boxes of 128
  // rows, 167 with 16).
  struct TokenOperand {
    int body, tail;
  };
  TokenOperand token_operand(const bf16* p, int64_t cols, int64_t tokens, int64_t ld) {
    g.k_tail = int(ceil_div((tokens - 1) % 128 + 1, 16) * 16);
    const int tail = operand(p, cols, tokens, ld, g.k_tail);
    return {tokens <= 128 || g.k_tail == 128 ? tail : operand(p, cols, tokens, ld), tail};
  }
  LinProblem& weight_problem(int64_t rows, int64_t cols, int64_t tokens, TokenOperand left,
                             TokenOperand right) {
    LinProblem& P = problem(kLinStore, rows, cols, tokens, 0);
    P.a0 = left.body;
    P.a1 = left.tail;
    P.b0 = right.body;
    P.b1 = right.tail;
    return P;
  }
  // One part of a sum over several launches, kept in `sum` from the first to the last.
  void part_of(LinProblem& P, float* sum, bool first, bool last) {
    if (first && last) return;
    if (g.sum == nullptr) g.sum = sum;
    P.sum_at = sum - g.sum;
    g.sum_read = !first;
    g.sum_write = !last;
  }
  // A product tokens x weight, swapped where that fits the token count better.  A part of a
  // sum stays plain (300,000 entries of 1536, 129 tokens: 585 us against 573): a running sum in
  // the swapped epilogue would cost every product that has none (37 tokens through 1536/8960:
  // 28.8 -> 29.0 us).
  LinProblem& token_problem(int epi, int64_t tokens, int64_t cols, int cols_per_tile, int64_t k0,
                            int64_t k1, bool part = false) {
    int nt = 0;
    if (!part && lin_swaps(tokens, epi, k0 + k1, &nt)) {
      g.swap = 1;
      g.nt = nt;
    }
    k_box = lin_stage_k(epi, g.swap != 0);
    LinProblem& P = problem(epi, tokens, cols, k0, k1);
    P.tiles_n = int(ceil_div(cols, cols_per_tile));
    if (g.swap) {
      P.tiles_m = P.tiles_n;
      P.tiles_n = int(ceil_div(tokens, nt));
    }
    return P;
  }
  // Operands of a token product: the tokens' rows of K, and the weight (rows of K,
  // or for a weight read along its other axis rows of the output's columns).
  void operands(LinProblem& P, const bf16* tok, int64_t k, int64_t tok_ld, const bf16* w,
                int64_t w_cols, int64_t w_rows, int64_t w_ld, bool k_major, bool second = false) {
    const int t = operand(tok, k, P.rows, tok_ld, g.swap ? g.nt / 2 : 128);
    const int m = operand(w, w_cols, w_rows, w_ld, k_major ? 128 : k_box);
    (second ? P.a1 : P.a0) = g.swap ? m : t;
    (second ? P.b1 : P.b0) = g.swap ? t : m;
  }
  // The kept gate and up, read and written in 32 x 32 chunks.
  void kept_maps(const dmuon_ffn_shape& s) {
    if (!g.kept_vec) return;
    const bool codes = g.keep == kKeepAct8;
    for (int i = 0; i < 2; ++i) {
      const void* p = i == 0 ? g.gate : g.up;
      (i == 0 ? g.map_gate : g.map_up) =
          codes ? output_codes(p, s.ffn, s.tokens)
                : output(static_cast<const bf16*>(p), s.ffn, s.tokens, s.ffn);
    }
  }
  // C: TMA where its rows allow it, plain stores otherwise.
  void store_to(LinProblem& P, bf16* c, int64_t ld, bool store_epilogue = true) {
    P.c = c;
    P.c_ld = ld;
    if (aligned(c, 16) && ld % 8 == 0)
      P.c_map = output(c, P.cols, P.rows, ld, store_epilogue && !g.swap);
  }
  // Run a token product; the weight's K is contiguous (k_major) or its columns are.
  int run_token(int epi, bool k_major, int clusters, cudaStream_t s) {
    return g.swap ? run(epi, !k_major, false, clusters, s) : run(epi, false, !k_major, clusters, s);
  }
  int run(int epi, bool a_mn, bool b_mn, int clusters, cudaStream_t s) {
    if (!ok) return DMUON_ERR_CUDA;
    g.n_maps = n_maps;
    lin_schedule(g, epi, clusters);
    return launch_lin(g, epi, a_mn, b_mn, clusters, s) == cudaSuccess ? DMUON_OK : DMUON_ERR_CUDA;
  }
};

// A bf16 matrix as TMA can read it: where it lies, or (noted in `c`) copied to `copy`.
struct Readable {
  const bf16* p;
  int64_t ld;
};
Readable readable(CopyArgs& c, const void* p, int64_t rows, int64_t cols, int64_t ld, bf16* copy) {
  const bf16* src = static_cast<const bf16*>(p);
  if (aligned(src, 16) && ld % 8 == 0) return {src, ld};
  c.add(src, ld, copy, pitch(cols), rows, cols);
  return {copy, pitch(cols)};
}
int run_copies(CopyArgs& c, cudaStream_t s) {
  return c.n == 0 || launch_copy_rows(c, s) == cudaSuccess ? DMUON_OK : DMUON_ERR_CUDA;
}

// ------------------------------------------------------------------ feed-forward block
bool ffn_shape_ok(const dmuon_ffn_shape* s) {
  return s != nullptr && s->tokens >= 0 && s->tokens <= kMaxTokens && s->hidden >= 1 &&
         s->hidden <= kMaxDim && s->ffn >= 1 && s->ffn <= kMaxDim &&
         s->activation >= DMUON_ACT_SILU && s->activation <= DMUON_ACT_GELU_TANH &&
         s->save >= DMUON_SAVE_NONE && s->save <= DMUON_SAVE_ACT8;
}

struct FfnSpace {
  ProductSpace ps;
  bf16 *x, *dy, *h, *dgate, *dup, *w_gate, *w_up, *w_down;
  float* sum[3];
  size_t bytes;
};
FfnSpace ffn_space(const dmuon_ffn_shape& s, bool backward, void* ws) {
  Carve c(ws);
  FfnSpace f{};
  const size_t t = size_t(s.tokens), dp = size_t(pitch(s.hidden)), fp = size_t(pitch(s.ffn));
  f.ps = take_product_space(c);
  f.x = c.take<bf16>(t * dp * 2);
  f.h = c.take<bf16>(t * fp * 2);
  if (backward) {
    f.dy = c.take<bf16>(t * dp * 2);
    f.dgate = c.take<bf16>(t * fp * 2);
    f.dup = c.take<bf16>(t * fp * 2);
    if (s.tokens > kSumTokens)
      for (float*& sum : f.sum) sum = c.take<float>(size_t(s.ffn) * size_t(s.hidden) * 4);
  }
  if (s.hidden % 8 != 0) {
    f.w_gate = c.take<bf16>(size_t(s.ffn) * dp * 2);
    f.w_up = c.take<bf16>(size_t(s.ffn) * dp * 2);
  }
  if (s.ffn % 8 != 0) f.w_down = c.take<bf16>(size_t(s.hidden) * fp * 2);
  f.bytes = c.used;
  return f;
}

struct FfnWeights {
  Readable gate, up, down;
};
FfnWeights ffn_weights(CopyArgs& c, const dmuon_ffn_shape& s, const FfnSpace& f, const void* wg,
                       const void* wu, const void* wd) {
  return {readable(c, wg, s.ffn, s.hidden, s.hidden, f.w_gate),
          readable(c, wu, s.ffn, s.hidden, s.hidden, f.w_up),
          readable(c, wd, s.hidden, s.ffn, s.ffn, f.w_down)};
}

// saved[] = {gate, up} in bf16, or {gate codes, gate scales, up codes, up scales}
bool saved_ok(int save, void* const* saved) {
  const int n = save == DMUON_SAVE_NONE ? 0 : save == DMUON_SAVE_BF16 ? 2 : 4;
  if (n == 0) return true;
  if (saved == nullptr) return false;
  for (int i = 0; i < n; ++i)
    if (saved[i] == nullptr) return false;
  return true;
}
void use_saved(LinArgs& g, const dmuon_ffn_shape& s, void* const* saved) {
  g.act = s.activation;
  g.keep = s.save == DMUON_SAVE_BF16 ? kKeepBf16 : s.save == DMUON_SAVE_ACT8 ? kKeepAct8 : kKeepNone;
  g.ffn = int(s.ffn);
  if (g.keep == kKeepBf16) {
    g.gate = saved[0];
    g.up = saved[1];
    g.kept_vec = s.ffn % 8 == 0 && aligned(g.gate, 16) && aligned(g.up, 16);
  } else if (g.keep == kKeepAct8) {
    g.gate = saved[0];
    g.gate_scale = static_cast<bf16*>(saved[1]);
    g.up = saved[2];
    g.up_scale = static_cast<bf16*>(saved[3]);
    g.kept_vec = s.ffn % 16 == 0 && aligned(g.gate, 16) && aligned(g.up, 16) &&
                 aligned(g.gate_scale, 8) && aligned(g.up_scale, 8);
  }
}

// Every bf16 element at an even address; weights at 16 bytes where rows allow TMA.
int ffn_alignment(const dmuon_ffn_shape& s, const void* wg, const void* wu, const void* wd,
                  void* const* saved, std::initializer_list<const void*> others) {
  if (!all_aligned(2, {wg, wu, wd}) || !all_aligned(2, others)) return DMUON_ERR_ALIGNMENT;
  if (s.save == DMUON_SAVE_BF16 && !all_aligned(2, {saved[0], saved[1]})) return DMUON_ERR_ALIGNMENT;
  if (s.save == DMUON_SAVE_ACT8 && !all_aligned(2, {saved[1], saved[3]})) return DMUON_ERR_ALIGNMENT;
  if (s.hidden % 8 == 0 && (!aligned(wg, 16) || !aligned(wu, 16))) return DMUON_ERR_ALIGNMENT;
  if (s.ffn % 8 == 0 && !aligned(wd, 16)) return DMUON_ERR_ALIGNMENT;
  return DMUON_OK;
}

// Whether two bf16 matrices of one size may share an element.
bool overlap(const void* a, int64_t a_ld, const void* b, int64_t b_ld, int64_t rows, int64_t cols) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  if (pa + (uintptr_t(rows - 1) * uintptr_t(a_ld) + uintptr_t(cols)) * 2 <= pb ||
      pb + (uintptr_t(rows - 1) * uintptr_t(b_ld) + uintptr_t(cols)) * 2 <= pa)
    return false;
  if (rows == 1 || a_ld != b_ld) return true;
  // rows of one pitch: columns may lie side by side
  const int64_t apart = (int64_t(pb) - int64_t(pa)) / 2 % a_ld;
  const int64_t at = apart < 0 ? apart + a_ld : apart;
  return at < cols || at + cols > a_ld;
}

int ffn_forward(const dmuon_ffn_shape& s, const void* x, int64_t x_ld, const void* wg,
                const void* wu, const void* wd, void* y, int64_t y_ld, void* const* saved,
                void* ws, cudaStream_t st) {
  int clusters = 0;
  int e = device_ready(&clusters);
  if (e != DMUON_OK) return e;
  const FfnSpace f = ffn_space(s, false, ws);
  const int64_t fp = pitch(s.ffn);
  CopyArgs copies{};
  const FfnWeights w = ffn_weights(copies, s, f, wg, wu, wd);
  const Readable xr = readable(copies, x, s.tokens, s.hidden, x_ld, f.x);
  e = run_copies(copies, st);
  if (e != DMUON_OK) return e;
  // Few tokens: weights streamed without tiles: eight tokens through 4096/14336 59 us, one
  // 56, against 73 with tiles (with 16 or 32, sharing the weights' registers among more
  // tokens, 89 and 138 against 73; 1536/8960, eight, 24 against 29).  8-bit blocks span more columns
  // than a block computes.
  if (s.tokens <= kThinTokens && s.hidden % 8 == 0 && s.ffn % 8 == 0 &&
      s.save != DMUON_SAVE_ACT8) {
    ThinArgs a{};
    a.x = xr.p;
    a.x_ld = xr.ld;
    a.w0 = w.gate.p;
    a.w1 = w.up.p;
    a.w_ld = w.gate.ld;
    a.out = f.h;
    a.out_ld = fp;
    if (s.save == DMUON_SAVE_BF16) {
      a.gate = static_cast<bf16*>(saved[0]);
      a.up = static_cast<bf16*>(saved[1]);
    }
    a.tokens = int(s.tokens);
    a.k = int(s.hidden);
    a.cols = int(s.ffn);
    a.act = s.activation;
    ThinArgs b{};
    b.x = f.h;
    b.x_ld = fp;
    b.w0 = w.down.p;
    b.w_ld = w.down.ld;
    b.out = static_cast<bf16*>(y);
    b.out_ld = y_ld;
    b.tokens = a.tokens;
    b.k = int(s.ffn);
    b.cols = int(s.hidden);
    return launch_thin(a, true, st) == cudaSuccess && launch_thin(b, false, st) == cudaSuccess
               ? DMUON_OK
               : DMUON_ERR_CUDA;
  }
  {
    Launch L(f.ps);
    LinProblem& P = L.token_problem(kLinGlu, s.tokens, s.ffn, 128, s.hidden, 0);
    const int t = L.operand(xr.p, s.hidden, s.tokens, xr.ld, L.g.swap ? L.g.nt / 2 : 128);
    const int gate = L.operand(w.gate.p, s.hidden, s.ffn, w.gate.ld, L.g.swap ? 64 : 128);
    const int up = L.operand(w.up.p, s.hidden, s.ffn, w.up.ld, L.g.swap ? 64 : 128);
    P.a0 = L.g.swap ? gate : t;
    P.a1 = up;
    P.b0 = L.g.swap ? t : gate;
    P.b1 = up;
    L.store_to(P, f.h, fp, false);
    use_saved(L.g, s, saved);
    L.kept_maps(s);
    e = L.run_token(kLinGlu, true, clusters, st);
    if (e != DMUON_OK) return e;
  }
  Launch L(f.ps, kEarlyWeights);
  LinProblem& P = L.token_problem(kLinStore, s.tokens, s.hidden, 256, s.ffn, 0);
  L.operands(P, f.h, s.ffn, fp, w.down.p, s.ffn, s.hidden, w.down.ld, true);
  L.store_to(P, static_cast<bf16*>(y), y_ld);
  return L.run_token(kLinStore, true, clusters, st);
}

int ffn_backward(const dmuon_ffn_shape& s, const void* dy, int64_t dy_ld, const void* x,
                 int64_t x_ld, const void* wg, const void* wu, const void* wd,
                 void* const* saved, void* dx, int64_t dx_ld, void* dwg, void* dwu, void* dwd,
                 void* ws, cudaStream_t st) {
  int clusters = 0;
  int e = device_ready(&clusters);
  if (e != DMUON_OK) return e;
  if (s.tokens == 0) {  // sums over no token
    CopyArgs zeros{};
    zeros.add(nullptr, 8, static_cast<bf16*>(dwg), s.hidden, s.ffn, s.hidden);
    zeros.add(nullptr, 8, static_cast<bf16*>(dwu), s.hidden, s.ffn, s.hidden);
    zeros.add(nullptr, 8, static_cast<bf16*>(dwd), s.ffn, s.hidden, s.ffn);
    return run_copies(zeros, st);
  }
  const FfnSpace f = ffn_space(s, true, ws);
  const int64_t fp = pitch(s.ffn);
  CopyArgs copies{};
  const FfnWeights w = ffn_weights(copies, s, f, wg, wu, wd);
  const Readable xr = readable(copies, x, s.tokens, s.hidden, x_ld, f.x);
  const Readable dyr = readable(copies, dy, s.tokens, s.hidden, dy_ld, f.dy);
  e = run_copies(copies, st);
  if (e != DMUON_OK) return e;
  {  // dh = dy Wd, and from it dgate, dup and h
    Launch L(f.ps);
    LinProblem& P = L.token_problem(kLinGluGrad, s.tokens, s.ffn, 256, s.hidden, 0);
    L.operands(P, dyr.p, s.hidden, dyr.ld, w.down.p, s.ffn, s.hidden, w.down.ld, false);
    L.store_to(P, f.dgate, fp, false);
    L.g.dup = f.dup;
    L.g.h = f.h;
    L.g.map_dup = L.output(f.dup, s.ffn, s.tokens, fp);
    L.g.map_h = L.output(f.h, s.ffn, s.tokens, fp);
    use_saved(L.g, s, saved);
    L.kept_maps(s);
    e = L.run_token(kLinGluGrad, false, clusters, st);
    if (e != DMUON_OK) return e;
  }
  {  // dx = dgate Wg + dup Wu
    Launch L(f.ps, kEarlyWeights);
    LinProblem& P = L.token_problem(kLinStore, s.tokens, s.hidden, 256, s.ffn, s.ffn);
    L.operands(P, f.dgate, s.ffn, fp, w.gate.p, s.hidden, s.ffn, w.gate.ld, false);
    L.operands(P, f.dup, s.ffn, fp, w.up.p, s.hidden, s.ffn, w.up.ld, false, true);
    L.store_to(P, static_cast<bf16*>(dx), dx_ld);
    e = L.run_token(kLinStore, false, clusters, st);
    if (e != DMUON_OK) return e;
  }
  // dWg = dgate^T x, dWu = dup^T x, dWd = dy^T h
  const bf16* left[3] = {f.dgate, f.dup, dyr.p};
  bf16* out[3] = {static_cast<bf16*>(dwg), static_cast<bf16*>(dwu), static_cast<bf16*>(dwd)};
  for (int64_t t0 = 0; t0 < s.tokens; t0 += kSumTokens) {
    const int64_t t = std::min(kSumTokens, s.tokens - t0);
    Launch L(f.ps, kEarlyAll);
    const Launch::TokenOperand ox = L.token_operand(xr.p + t0 * xr.ld, s.hidden, t, xr.ld),
                               oh = L.token_operand(f.h + t0 * fp, s.ffn, t, fp);
    for (int i = 0; i < 3; ++i) {
      const int64_t m = i < 2 ? s.ffn : s.hidden, n = i < 2 ? s.hidden : s.ffn;
      const int64_t ld = i < 2 ? fp : dyr.ld;
      const Launch::TokenOperand ol = L.token_operand(left[i] + t0 * ld, m, t, ld);
      LinProblem& P = L.weight_problem(m, n, t, ol, i < 2 ? ox : oh);
      L.store_to(P, out[i], n);
      L.part_of(P, f.sum[i], t0 == 0, t0 + t == s.tokens);
    }
    e = L.run(kLinStore, true, true, clusters, st);
    if (e != DMUON_OK) return e;
  }
  return DMUON_OK;
}

// ------------------------------------------------------------------ cross entropy
bool xent_shape_ok(const dmuon_xent_shape* s) {
  return s != nullptr && s->tokens >= 0 && s->tokens <= kMaxTokens && s->hidden >= 1 &&
         s->hidden <= kMaxDim && s->vocab >= 1 && s->vocab <= kMaxVocab;
}

// Tokens worked on at a time.
int64_t xent_piece(const dmuon_xent_shape& s, bool grads) {
  int64_t most = kLossTokens;
  if (grads)
    most = std::min(kSumTokens,
                    std::max<int64_t>(256, int64_t(kLogitBytes / (size_t(pitch(s.vocab)) * 2)) /
                                               256 * 256));
  return std::min(s.tokens, most);
}

struct XentSpace {
  ProductSpace ps;
  bf16 *hidden, *weight, *e;
  float* grad_scale;
  float2* stat;
  float *sum, *hidden_sum;
  int64_t piece;
  size_t bytes;
};
XentSpace xent_space(const dmuon_xent_shape& s, bool grads, void* ws) {
  Carve c(ws);
  XentSpace x{};
  const size_t dp = size_t(pitch(s.hidden));
  x.piece = xent_piece(s, grads);
  x.ps = take_product_space(c);
  x.hidden = c.take<bf16>(size_t(s.tokens) * dp * 2);
  x.grad_scale = c.take<float>(4);
  // swapped products have four times the groups, over at most kXentSwapTokens tokens
  x.stat = c.take<float2>(
      std::max(size_t(ceil_div(s.vocab, kXentGroup)) * size_t(up32(x.piece)),
               size_t(ceil_div(s.vocab, kXentGroupSwap)) *
                   size_t(std::min<int64_t>(up32(x.piece), kXentSwapTokens))) * sizeof(float2));
  if (s.hidden % 8 != 0) x.weight = c.take<bf16>(size_t(s.vocab) * dp * 2);
  if (grads) {
    x.e = c.take<bf16>(size_t(x.piece) * size_t(pitch(s.vocab)) * 2);
    if (x.piece < s.tokens) x.sum = c.take<float>(size_t(s.vocab) * size_t(s.hidden) * 4);
    if (s.vocab > kVocabWhole)
      x.hidden_sum = c.take<float>(size_t(x.piece) * size_t(s.hidden) * 4);
  }
  x.bytes = c.used;
  return x;
}

int xent(const dmuon_xent_shape& s, const void* hidden, int64_t h_ld, const void* weight,
         const int64_t* target, const float* grad_loss, float* loss, float* lse, void* dhidden,
         int64_t dh_ld, void* dweight, void* ws, cudaStream_t st) {
  const bool grads = grad_loss != nullptr;
  int clusters = 0;
  int e = device_ready(&clusters);
  if (e != DMUON_OK) return e;
  const XentSpace x = xent_space(s, grads, ws);
  const int64_t vp = pitch(s.vocab);
  const long long* tgt = reinterpret_cast<const long long*>(target);
  CopyArgs copies{};
  Readable h;
  if (grads) {
    // masked rows become zeros, so that nothing they hold (NaN of padding, say)
    // reaches the weight's gradient, which sums over rows
    copies.target = tgt;
    copies.vocab = s.vocab;
    copies.grad_loss = grad_loss;
    copies.tokens = s.tokens;
    copies.grad_scale = x.grad_scale;
    h = {x.hidden, pitch(s.hidden)};
    copies.add(static_cast<const bf16*>(hidden), h_ld, x.hidden, h.ld, s.tokens, s.hidden);
  } else {
    h = readable(copies, hidden, s.tokens, s.hidden, h_ld, x.hidden);
  }
  const Readable w = readable(copies, weight, s.vocab, s.hidden, s.hidden, x.weight);
  e = run_copies(copies, st);
  if (e != DMUON_OK) return e;
  for (int64_t t0 = 0; t0 < s.tokens; t0 += x.piece) {
    const int64_t n = std::min(x.piece, s.tokens - t0);
    const bf16* hp = h.p + t0 * h.ld;
    XentRows R{};
    R.tokens = n;
    R.vocab = s.vocab;
    R.target = tgt + t0;
    R.grad_loss = grads ? grad_loss + t0 : nullptr;
    R.grad_scale = x.grad_scale;
    R.hidden = hp;
    R.hidden_ld = h.ld;
    R.weight = w.p;
    R.weight_ld = w.ld;
    R.k = int(s.hidden);
    R.group_stat = x.stat;
    R.stat_ld = up32(n);
    R.loss = loss + t0;
    R.lse = lse + t0;
    {
      Launch L(x.ps);
      LinProblem& P = L.token_problem(kLinXent, n, s.vocab, 256, s.hidden, 0);
      L.operands(P, hp, s.hidden, h.ld, w.p, s.hidden, s.vocab, w.ld, true);
      if (grads) P.c_map = L.output(x.e, s.vocab, n, vp, !L.g.swap);
      L.g.target = tgt + t0;
      L.g.group_stat = x.stat;
      L.g.stat_ld = R.stat_ld;
      R.group = L.g.swap ? kXentGroupSwap : kXentGroup;
      e = L.run_token(kLinXent, true, clusters, st);
      if (e != DMUON_OK) return e;
    }
    if (launch_xent_rows(R, st) != cudaSuccess) return DMUON_ERR_CUDA;
    if (!grads) continue;
    if (launch_xent_grad(R, x.e, vp, st) != cudaSuccess) return DMUON_ERR_CUDA;
    // dhidden = G W
    const int64_t cuts = s.vocab > kVocabWhole ? ceil_div(s.vocab, kVocabPart) : 1;
    const int64_t span = pitch(ceil_div(s.vocab, cuts));
    for (int64_t v0 = 0; v0 < s.vocab; v0 += span) {
      const int64_t k = std::min(span, s.vocab - v0);
      Launch L(x.ps, kEarlyWeights);
      LinProblem& P = L.token_problem(kLinStore, n, s.hidden, 256, k, 0, cuts > 1);
      L.operands(P, x.e + v0, k, vp, w.p + v0 * w.ld, s.hidden, k, w.ld, false);
      L.store_to(P, static_cast<bf16*>(dhidden) + t0 * dh_ld, dh_ld);
      L.part_of(P, x.hidden_sum, v0 == 0, v0 + k == s.vocab);
      L.g.scale = x.grad_scale;
      e = L.run_token(kLinStore, false, clusters, st);
      if (e != DMUON_OK) return e;
    }
    // dweight += G^T h, in fp32 over the pieces
    Launch L(x.ps, kEarlyAll);
    LinProblem& P = L.weight_problem(s.vocab, s.hidden, n, L.token_operand(x.e, s.vocab, n, vp),
                                     L.token_operand(hp, s.hidden, n, h.ld));
    L.store_to(P, static_cast<bf16*>(dweight), s.hidden);
    L.g.scale = x.grad_scale;
    L.part_of(P, x.sum, t0 == 0, t0 + n == s.tokens);
    e = L.run(kLinStore, true, true, clusters, st);
    if (e != DMUON_OK) return e;
  }
  return DMUON_OK;
}

}  // namespace
}  // namespace dm

extern "C" {

using namespace dm;

int dmuon_act8_save(int64_t rows, int64_t cols, const void* x, int64_t x_ld, int x_dt,
                    int8_t* codes, void* scales, cudaStream_t stream) {
  if (rows < 0 || cols < 0 || (x_dt != DMUON_F32 && x_dt != DMUON_BF16))
    return DMUON_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return DMUON_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr || x_ld < cols)
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(x, x_dt == DMUON_BF16 ? 2 : 4) || !aligned(scales, 2)) return DMUON_ERR_ALIGNMENT;
  if (ceil_div(cols, 2048) > INT32_MAX / rows) return DMUON_ERR_UNSUPPORTED;
  int clusters = 0;
  const int st = device_ready(&clusters);
  if (st != DMUON_OK) return st;
  return launch_act8_save(rows, cols, x, x_ld, x_dt == DMUON_BF16,
                          reinterpret_cast<signed char*>(codes), static_cast<bf16*>(scales),
                          stream) == cudaSuccess
             ? DMUON_OK
             : DMUON_ERR_CUDA;
}

int dmuon_act8_load(int64_t rows, int64_t cols, const int8_t* codes, const void* scales,
                    void* out, int64_t out_ld, int out_dt, cudaStream_t stream) {
  if (rows < 0 || cols < 0 || (out_dt != DMUON_F32 && out_dt != DMUON_BF16))
    return DMUON_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return DMUON_OK;
  if (out == nullptr || codes == nullptr || scales == nullptr || out_ld < cols)
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(out, out_dt == DMUON_BF16 ? 2 : 4) || !aligned(scales, 2))
    return DMUON_ERR_ALIGNMENT;
  if (ceil_div(cols, 2048) > INT32_MAX / rows) return DMUON_ERR_UNSUPPORTED;
  int clusters = 0;
  const int st = device_ready(&clusters);
  if (st != DMUON_OK) return st;
  return launch_act8_load(rows, cols, reinterpret_cast<const signed char*>(codes),
                          static_cast<const bf16*>(scales), out, out_ld, out_dt == DMUON_BF16,
                          stream) == cudaSuccess
             ? DMUON_OK
             : DMUON_ERR_CUDA;
}

size_t dmuon_ffn_workspace_bytes(const dmuon_ffn_shape* shape, int backward) {
  if (!ffn_shape_ok(shape)) return 0;
  return ffn_space(*shape, backward != 0, nullptr).bytes;
}

int dmuon_ffn_forward(const dmuon_ffn_shape* shape, const void* x, int64_t x_ld,
                      const void* w_gate, const void* w_up, const void* w_down, void* y,
                      int64_t y_ld, void* const* saved, void* workspace, size_t ws_bytes,
                      cudaStream_t stream) {
  if (!ffn_shape_ok(shape)) return DMUON_ERR_INVALID_ARG;
  if (shape->tokens == 0) return DMUON_OK;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr ||
      workspace == nullptr || x_ld < shape->hidden || y_ld < shape->hidden ||
      !saved_ok(shape->save, saved))
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return DMUON_ERR_ALIGNMENT;
  const int st = ffn_alignment(*shape, w_gate, w_up, w_down, saved, {x, y});
  if (st != DMUON_OK) return st;
  if (ws_bytes < dmuon_ffn_workspace_bytes(shape, 0)) return DMUON_ERR_WORKSPACE;
  return ffn_forward(*shape, x, x_ld, w_gate, w_up, w_down, y, y_ld, saved, workspace, stream);
}

int dmuon_ffn_backward(const dmuon_ffn_shape* shape, const void* dy, int64_t dy_ld, const void* x,
                       int64_t x_ld, const void* w_gate, const void* w_up, const void* w_down,
                       void* const* saved, void* dx, int64_t dx_ld, void* dw_gate, void* dw_up,
                       void* dw_down, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!ffn_shape_ok(shape) || shape->save == DMUON_SAVE_NONE) return DMUON_ERR_INVALID_ARG;
  if (w_gate == nullptr || w_up == nullptr || w_down == nullptr || dw_gate == nullptr ||
      dw_up == nullptr || dw_down == nullptr || workspace == nullptr)
    return DMUON_ERR_INVALID_ARG;
  if (shape->tokens > 0 &&
      (dy == nullptr || x == nullptr || dx == nullptr || dy_ld < shape->hidden ||
       x_ld < shape->hidden || dx_ld < shape->hidden || !saved_ok(shape->save, saved)))
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return DMUON_ERR_ALIGNMENT;
  const dmuon_ffn_shape& sh = *shape;
  void* const none[4] = {};
  const int st = sh.tokens > 0 ? ffn_alignment(sh, w_gate, w_up, w_down, saved,
                                               {dy, x, dx, dw_gate, dw_up, dw_down})
                               : ffn_alignment(sh, w_gate, w_up, w_down, none,
                                               {dw_gate, dw_up, dw_down});
  if (st != DMUON_OK) return st;
  if (ws_bytes < dmuon_ffn_workspace_bytes(shape, 1)) return DMUON_ERR_WORKSPACE;
  // dx is written before, and while, the weight gradients read dy and x
  if (sh.tokens > 0 && (overlap(dx, dx_ld, dy, dy_ld, sh.tokens, sh.hidden) ||
                        overlap(dx, dx_ld, x, x_ld, sh.tokens, sh.hidden)))
    return DMUON_ERR_INVALID_ARG;
  return ffn_backward(*shape, dy, dy_ld, x, x_ld, w_gate, w_up, w_down, saved, dx, dx_ld, dw_gate,
                      dw_up, dw_down, workspace, stream);
}

size_t dmuon_xent_workspace_bytes(const dmuon_xent_shape* shape, int grads) {
  if (!xent_shape_ok(shape)) return 0;
  // one for gradients serves the loss alone too, which takes more tokens at a time (a vast
  // vocabulary's group statistics of 16384 tokens outweigh what gradients keep)
  const size_t loss = xent_space(*shape, false, nullptr).bytes;
  return grads != 0 ? std::max(loss, xent_space(*shape, true, nullptr).bytes) : loss;
}

int dmuon_xent(const dmuon_xent_shape* shape, const void* hidden, int64_t hidden_ld,
               const void* weight, const int64_t* target, const float* grad_loss, float* loss,
               float* lse, void* dhidden, int64_t dhidden_ld, void* dweight, void* workspace,
               size_t ws_bytes, cudaStream_t stream) {
  if (!xent_shape_ok(shape) || weight == nullptr || workspace == nullptr)
    return DMUON_ERR_INVALID_ARG;
  const bool grads = grad_loss != nullptr || dhidden != nullptr || dweight != nullptr;
  if (grads && dweight == nullptr) return DMUON_ERR_INVALID_ARG;
  if (shape->tokens > 0) {
    if (hidden == nullptr || target == nullptr || loss == nullptr || lse == nullptr ||
        hidden_ld < shape->hidden)
      return DMUON_ERR_INVALID_ARG;
    if (grads && (grad_loss == nullptr || dhidden == nullptr || dhidden_ld < shape->hidden))
      return DMUON_ERR_INVALID_ARG;
  }
  if (!aligned(workspace, 256) || !aligned(weight, shape->hidden % 8 == 0 ? 16 : 2) ||
      !aligned(dweight, 2))
    return DMUON_ERR_ALIGNMENT;
  if (shape->tokens > 0 &&
      (!all_aligned(2, {hidden, dhidden}) || !all_aligned(4, {loss, lse, grad_loss}) ||
       !aligned(target, 8)))
    return DMUON_ERR_ALIGNMENT;
  if (ws_bytes < dmuon_xent_workspace_bytes(shape, grads ? 1 : 0)) return DMUON_ERR_WORKSPACE;
  if (shape->tokens == 0 && grads) {
    int clusters = 0;
    const int st = device_ready(&clusters);
    if (st != DMUON_OK) return st;
    CopyArgs zeros{};
    zeros.add(nullptr, 8, static_cast<bf16*>(dweight), shape->hidden, shape->vocab, shape->hidden);
    return run_copies(zeros, stream);
  }
  if (shape->tokens == 0) return DMUON_OK;
  return xent(*shape, hidden, hidden_ld, weight, target, grad_loss, loss, lse, dhidden, dhidden_ld,
              dweight, workspace, stream);
}

}  // extern "C"
