// C ABI of the operators that mix tokens: argument checks, tensor maps and launch sequences.
// See include/dmuon.h.
#include "dmuon.h"
#include "launch.h"
#include "mix.h"
#include "train.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

namespace dm {
namespace {

constexpr size_t kHdrBytes = 256;  // workspace header: device error word
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTokens = int64_t(1) << 22, kMaxHeads = int64_t(1) << 16,
                  kMaxSequences = int64_t(1) << 16;

using bf16 = __nv_bfloat16;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Ready the current device, once: the kernels' shared memory opt-in, and how many clusters fit.
struct Device {
  int sms;
  int fit[kMixMaxSplit + 1];
};
int device_ready(Device* device) {
  int d = 0, clusters = 0, sms = 0;
  const int st = library_device(&d, &sms, &clusters);
  if (st != DMUON_OK) return st;
  static std::mutex mu;
  static bool ready[kMaxDevices] = {};
  static Device known[kMaxDevices];
  std::lock_guard<std::mutex> lk(mu);
  if (!ready[d]) {
    if (linattn_prepare(known[d].fit) != cudaSuccess) return DMUON_ERR_CUDA;
    known[d].sms = sms;
    ready[d] = true;
  }
  *device = known[d];
  return DMUON_OK;
}

// ------------------------------------------------------------------ tensors of heads
// A tensor's rows with strides that also hold where there is one token or one head only.
struct Rows {
  uintptr_t p;
  int64_t tokens, heads, dim, ts, hs;
  uintptr_t end() const {
    return p + uintptr_t((tokens - 1) * ts + (heads - 1) * hs + dim) * 2;
  }
};
// Fills r; false: a null pointer, or rows that may overlap.
bool rows_of(const dmuon_heads* h, int64_t tokens, int64_t heads, int64_t dim, Rows* r) {
  if (h == nullptr || h->data == nullptr) return false;
  constexpr int64_t kMost = int64_t(1) << 38;  // of a stride, in elements
  *r = Rows{reinterpret_cast<uintptr_t>(h->data), tokens, heads, dim, h->token_stride,
            h->head_stride};
  if (heads == 1) r->hs = dim;
  if (tokens == 1) r->ts = heads == 1 ? dim : r->hs;
  if (r->hs < dim || r->ts < dim || r->hs > kMost || r->ts > kMost) return false;
  if (tokens == 1 || heads == 1) return true;
  return r->ts >= (heads - 1) * r->hs + dim || r->hs >= (tokens - 1) * r->ts + dim;
}
// Whether two tensors of the same tokens (heads and dims may differ) may share an element.
bool overlap(const Rows& a, const Rows& b) {
  if (a.end() <= b.p || b.end() <= a.p) return false;
  // a stride over one row is any stride that neither's row passes
  if ((a.tokens > 1 && a.ts != b.ts) || (a.heads > 1 && b.heads > 1 && a.hs != b.hs)) return true;
  const int64_t ts = a.tokens > 1 ? a.ts : int64_t(1) << 40,
                hs = a.heads > 1 ? a.hs : b.heads > 1 ? b.hs : std::max(a.dim, b.dim);
  // parts of one packed tensor: b's place against a's as whole strides, outer and inner, and a
  // rest.  Element (t, h, x) of a is (t', h', x') of b where
  //   apart = (t - t') ts + (h - h') hs + (x - x')
  const int64_t apart = (int64_t(b.p) - int64_t(a.p)) / 2;
  const bool by_token = ts >= hs;
  const int64_t s1 = by_token ? ts : hs, s2 = by_token ? hs : ts;
  const int64_t a1 = by_token ? a.tokens : a.heads, b1 = by_token ? b.tokens : b.heads;
  const int64_t a2 = by_token ? a.heads : a.tokens, b2 = by_token ? b.heads : b.tokens;
  auto floor_div = [](int64_t x, int64_t y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
  const int64_t k1 = floor_div(apart, s1);
  for (int64_t i = k1; i <= k1 + 1; ++i) {
    if (i <= -b1 || i >= a1) continue;
    const int64_t rest = apart - i * s1, k2 = floor_div(rest, s2);
    for (int64_t j = k2; j <= k2 + 1; ++j) {
      if (j <= -b2 || j >= a2) continue;
      const int64_t x = rest - j * s2;
      if (x < a.dim && -x < b.dim) return true;
    }
  }
  return false;
}
bool same(const Rows& a, const Rows& b) {
  return a.p == b.p && (a.tokens == 1 || a.ts == b.ts) && (a.heads == 1 || a.hs == b.hs);
}
bool rows_aligned(const Rows& r, size_t bytes) {
  return r.p % bytes == 0 && r.ts * 2 % int64_t(bytes) == 0 && r.hs * 2 % int64_t(bytes) == 0;
}
Heads device_heads(const Rows& r) { return {reinterpret_cast<bf16*>(r.p), r.ts, r.hs}; }

// ------------------------------------------------------------------ norms and rotation
bool qk_shape_ok(const dmuon_qk_shape* s) {
  return s != nullptr && s->tokens >= 0 && s->tokens <= kMaxTokens && s->q_heads >= 1 &&
         s->q_heads <= kMaxHeads && s->k_heads >= 0 && s->k_heads <= kMaxHeads &&
         s->head_dim >= 8 && s->head_dim <= 256 && s->head_dim % 8 == 0 && s->rotary_dim >= 0 &&
         s->rotary_dim <= s->head_dim && s->rotary_dim % 8 == 0 && s->eps >= 0.f &&
         std::isfinite(s->eps);
}
size_t qk_workspace(const dmuon_qk_shape& s) {
  return kHdrBytes + size_t(kRopeBlocks) * 2 * size_t(s.head_dim) * sizeof(float);
}

// Forward (dout null) and backward.
int qk_norm_rope(const dmuon_qk_shape* shape, const dmuon_heads* const x[2],
                 const dmuon_heads* const dout[2], const dmuon_heads* const out[2],
                 const void* const w[2], const float* inv_freq, const int32_t* position,
                 void* const dw[2], float* partial, cudaStream_t st) {
  const dmuon_qk_shape& s = *shape;
  const int64_t heads[2] = {s.q_heads, s.k_heads};
  if (s.rotary_dim > 0 && (inv_freq == nullptr || (position == nullptr && s.tokens > 0)))
    return DMUON_ERR_INVALID_ARG;
  const bool backward = partial != nullptr;
  RopeArgs g{};
  bool vec = true;
  Rows xr[2], dr[2], orow[2];
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0 || s.tokens == 0) continue;
    if (!rows_of(x[i], s.tokens, heads[i], s.head_dim, &xr[i]) ||
        !rows_of(out[i], s.tokens, heads[i], s.head_dim, &orow[i]) ||
        (backward && !rows_of(dout[i], s.tokens, heads[i], s.head_dim, &dr[i])))
      return DMUON_ERR_INVALID_ARG;
  }
  if (!aligned(w[0], 2) || !aligned(w[1], 2) || !aligned(inv_freq, 4) || !aligned(position, 4) ||
      !aligned(dw[0], 2) || !aligned(dw[1], 2))
    return DMUON_ERR_ALIGNMENT;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0 || s.tokens == 0) continue;
    if (xr[i].p % 2 != 0 || orow[i].p % 2 != 0 || (backward && dr[i].p % 2 != 0))
      return DMUON_ERR_ALIGNMENT;
    vec = vec && rows_aligned(xr[i], 8) && rows_aligned(orow[i], 8) &&
          (!backward || rows_aligned(dr[i], 8));
    g.x[i] = device_heads(xr[i]);
    g.out[i] = device_heads(orow[i]);
    if (backward) g.dy[i] = device_heads(dr[i]);
    vec = vec && aligned(w[i], 8);
  }
  // an output is its own input, or apart from every input and the other output
  if (s.tokens > 0) {
    for (int i = 0; i < 2; ++i) {
      if (heads[i] == 0) continue;
      for (int j = 0; j < 2; ++j) {
        if (heads[j] == 0) continue;
        if (backward) {
          if (overlap(orow[i], xr[j])) return DMUON_ERR_INVALID_ARG;
          if (!(i == j && same(orow[i], dr[j])) && overlap(orow[i], dr[j]))
            return DMUON_ERR_INVALID_ARG;
        } else if (!(i == j && same(orow[i], xr[j])) && overlap(orow[i], xr[j])) {
          return DMUON_ERR_INVALID_ARG;
        }
        if (i < j && overlap(orow[i], orow[j])) return DMUON_ERR_INVALID_ARG;
      }
    }
  }
  if (s.tokens == 0 && !backward) return DMUON_OK;
  // a warp takes 4 heads at least
  if (s.tokens * (ceil_div(heads[0], 4) + ceil_div(heads[1], 4)) > INT32_MAX)
    return DMUON_ERR_UNSUPPORTED;
  Device device;
  const int e = device_ready(&device);
  if (e != DMUON_OK) return e;
  for (int i = 0; i < 2; ++i) {
    g.w[i] = static_cast<const bf16*>(w[i]);
    g.dw[i] = static_cast<bf16*>(dw[i]);
    g.heads[i] = int(heads[i]);
  }
  g.inv_freq = inv_freq;
  g.position = position;
  g.tokens = int(s.tokens);
  g.dim = int(s.head_dim);
  g.rotary = int(s.rotary_dim);
  g.eps = s.eps;
  g.partial = dw[0] != nullptr || dw[1] != nullptr ? partial : nullptr;
  return launch_rope(g, backward, s.interleaved != 0, vec, device.sms, st) == cudaSuccess
             ? DMUON_OK
             : DMUON_ERR_CUDA;
}

// ------------------------------------------------------------------ linear attention
bool linattn_shape_ok(const dmuon_linattn_shape* s) {
  return s != nullptr && s->tokens >= 0 && s->tokens <= kMaxTokens && s->sequences >= 1 &&
         s->sequences <= kMaxSequences && s->heads >= 1 && s->heads <= kMaxHeads &&
         s->key_dim >= 8 && s->key_dim <= 128 && s->key_dim % 8 == 0 && s->value_dim >= 8 &&
         s->value_dim <= 128 && s->value_dim % 8 == 0 && std::isfinite(s->scale) &&
         std::isfinite(1.f / s->scale) && s->sequences * s->heads <= (int64_t(1) << 27);
}
// States of the call: of so many sequences, or slots.
struct States {
  uintptr_t p, bytes;
  States(const float* at, const dmuon_linattn_shape& s, int64_t n)
      : p(reinterpret_cast<uintptr_t>(at)),
        bytes(at == nullptr ? 0 : uintptr_t(n) * uintptr_t(s.heads * s.key_dim * s.value_dim) * 4) {}
  bool meets(uintptr_t from, uintptr_t to) const { return bytes > 0 && p < to && from < p + bytes; }
  bool meets(const Rows& r) const { return meets(r.p, r.end()); }
  // Written states are the read ones or lie apart from them.
  bool beside(const States& read) const { return p == read.p || !meets(read.p, read.p + read.bytes); }
};

// How a head's packed batch is shared: `groups` clusters of `split` CTAs, or whole sequences of all heads
// and sweeps dealt to `deal` CTAs.
struct Share {
  int groups, split, deal;
};
// Microseconds, measured with 128 elements to a head and taken for fewer, too (a block of 64 takes
// 1.9): a block takes 3 (exact states 3.8), 1.5 more (2) where a CTA sums its share ahead; a launch
// 6, sharing 5.  Clusters of a size that the GPU's groups of SMs do not divide into run fewer at a
// time (gradients of 8192 tokens of 8 heads: 24 clusters of 6 111 us, of 4 77).
Share choose_share(const dmuon_linattn_shape& s, int sweeps, bool exact, const Device& device) {
  const int64_t blocks = s.tokens / kMixBlock + std::min(s.sequences, s.tokens);  // at most
  const double one = double(blocks) / double(s.sequences);
  const double sweep = exact ? 3.8 : 3.0, ahead = exact ? 2.0 : 1.5;
  Share best{1, 1, 0};
  double least = 0, whole = 0;
  for (int64_t groups = 1; groups <= s.sequences && groups <= 64; ++groups) {
    const int64_t clusters = sweeps * s.heads * groups;
    for (int split = 1; split <= kMixMaxSplit; ++split) {
      if (groups * split > blocks && groups * split > 1) break;
      if (split > 1 && clusters * split > kMixMaxCtas) break;
      // clusters end where sequences do: the largest has about half a sequence more than its part
      const double part = double(blocks) / groups + (groups > 1 ? one / 2 : 0.0);
      const double stretch = std::ceil(part / split);
      // what a CTA sums ahead: its last sequence, about half of one of many
      const double summed = split == 1 ? 0.0 : s.sequences > split ? std::min(stretch, one / 2) : stretch;
      const double cost = double(ceil_div(clusters, device.fit[split])) *
                          (stretch * sweep + summed * ahead + 6 + (split > 1 ? 5 : 0));
      if (whole == 0) whole = cost;  // a CTA to a head
      if (least == 0 || cost < least) {
        best = {int(groups), split, 0};
        least = cost;
      }
    }
    if (clusters >= device.sms) break;
  }
  // Dealing whole sequences: the longest of n, cut at random, is H_n / n of the batch; each takes 4
  // us to begin, and with all SMs busy a block takes longer.  (Gradients of 8192 tokens of 32 heads
  // in 5 sequences: a CTA to a head and gradient 180 us, dealt 149; of 4096 tokens of 28 heads, 3
  // CTAs to each 110 to 124, dealt 79 to 84, but in 2 equal sequences 87 and 93; 8192 of 40 heads
  // in 30 sequences 250 and 312.)  Not where one long sequence among short ones would lose much by
  // it.
  const int64_t pairs = sweeps * s.heads, ctas = std::min(int64_t(device.sms), pairs * s.sequences);
  if (whole <= 1.25 * least && !exact && s.sequences > 1 && s.sequences < 32 &&
      pairs * s.sequences <= ctas * (kMixDealt / 2)) {
    double longest = 0;
    for (int64_t i = 1; i <= s.sequences; ++i) longest += one / double(i);
    const double each = std::max(longest, double(blocks * pairs) / double(ctas));
    const double begun = std::ceil(double(pairs * s.sequences) / double(ctas));
    if (1.2 * (each * sweep + begun * 4 + 6) < least) best = {1, 1, int(ctas)};
  }
  return best;
}
// The workspace serves any way to share any number of tokens and sequences up to the shape's.
size_t linattn_workspace(const dmuon_linattn_shape& s) {
  const int64_t ctas = std::min(3 * s.sequences * s.heads * kMixMaxSplit, kMixMaxCtas);
  return kHdrBytes + size_t(ctas) * kMixSlots * kMixLocalBytes;
}

bool tile_map(CUtensorMap* m, const Rows& r, bool output = false) {
  const TensorMapEncode enc = library_tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(r.dim), cuuint64_t(r.heads), cuuint64_t(r.tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(r.hs) * 2, cuuint64_t(r.ts) * 2};
  const cuuint32_t box[3] = {output ? 32u : 64u, 1, output ? 32u : unsigned(kMixBlock)}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, reinterpret_cast<void*>(r.p), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             output ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One sweep: out of (q, k, v), key width q.dim, value width v.dim.
struct Sweep {
  const Rows *q, *k, *v, *out;
  bool against;
  const float* state_in;
  float* state_out;
  bool transposed;  // the caller's state is (value, key)
  bool scaled;      // and scale times the sum
};
int run_sweeps(const dmuon_linattn_shape& s, const Sweep* w, int sweeps, const float* log_decay,
               const int32_t* offsets, const Device& device, void* ws, cudaStream_t st) {
  bool exact = false;
  for (int i = 0; i < sweeps; ++i) exact = exact || w[i].state_out != nullptr;
  const Share share = choose_share(s, sweeps, exact, device);
  LinAttnSweeps all{};
  all.count = sweeps;
  all.deal = share.deal;
  for (int i = 0; i < sweeps; ++i, ++w) {
    LinAttnArgs& g = all.sweep[i];
    if (!tile_map(&g.q, *w->q) || !tile_map(&g.k, *w->k) || !tile_map(&g.v, *w->v) ||
        !tile_map(&g.o, *w->out, true))
      return DMUON_ERR_CUDA;
    g.log_decay = log_decay;
    g.offsets = offsets;
    g.sequences = int(s.sequences);
    g.heads = int(s.heads);
    g.tokens = int(s.tokens);
    g.dk = int(w->q->dim);
    g.dv = int(w->v->dim);
    g.scale = s.scale;
    g.against = w->against;
    g.state_in = w->state_in;
    g.state_out = w->state_out;
    g.key_scale = w->scaled ? s.scale : 1.f;
    g.state_scale = w->scaled ? 1.f : s.scale;
    g.st_row = w->transposed ? 1 : g.dv;
    g.st_col = w->transposed ? g.dk : 1;
    g.out = device_heads(*w->out);
    g.groups = share.groups;
    g.split = share.split;
    g.exact = exact;
    g.err = static_cast<int*>(ws);
    g.local = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kHdrBytes);
  }
  return launch_linattn(all, st) == cudaSuccess ? DMUON_OK : DMUON_ERR_CUDA;
}

// Rows of a tensor of the call, checked; `status` keeps the first failure.
Rows checked(const dmuon_heads* h, const dmuon_linattn_shape& s, int64_t dim, int* status) {
  Rows r{};
  if (!rows_of(h, s.tokens, s.heads, dim, &r)) *status = DMUON_ERR_INVALID_ARG;
  else if (*status == DMUON_OK && !rows_aligned(r, 16)) *status = DMUON_ERR_ALIGNMENT;
  return r;
}
int check_common(const dmuon_linattn_shape* s, const float* log_decay, const int32_t* offsets,
                 const float* a, const float* b, void* ws, size_t ws_bytes) {
  if (!linattn_shape_ok(s) || log_decay == nullptr || ws == nullptr ||
      (offsets == nullptr && s->sequences != 1))
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !aligned(log_decay, 4) || !aligned(offsets, 4) || !aligned(a, 16) ||
      !aligned(b, 16))
    return DMUON_ERR_ALIGNMENT;
  if (ws_bytes < linattn_workspace(*s)) return DMUON_ERR_WORKSPACE;
  return DMUON_OK;
}

}  // namespace
}  // namespace dm

using namespace dm;

extern "C" {

int dmuon_qk_norm_rope(const dmuon_qk_shape* shape, const dmuon_heads* q, const dmuon_heads* k,
                       const void* w_q, const void* w_k, const float* inv_freq,
                       const int32_t* position, const dmuon_heads* q_out,
                       const dmuon_heads* k_out, cudaStream_t stream) {
  if (!qk_shape_ok(shape)) return DMUON_ERR_INVALID_ARG;
  const dmuon_heads *x[2] = {q, k}, *none[2] = {}, *out[2] = {q_out, k_out};
  const void* w[2] = {w_q, w_k};
  void* dw[2] = {};
  return qk_norm_rope(shape, x, none, out, w, inv_freq, position, dw, nullptr, stream);
}

size_t dmuon_qk_norm_rope_workspace_bytes(const dmuon_qk_shape* shape) {
  return qk_shape_ok(shape) ? qk_workspace(*shape) : 0;
}

int dmuon_qk_norm_rope_backward(const dmuon_qk_shape* shape, const dmuon_heads* dq_out,
                                const dmuon_heads* dk_out, const dmuon_heads* q,
                                const dmuon_heads* k, const void* w_q, const void* w_k,
                                const float* inv_freq, const int32_t* position,
                                const dmuon_heads* dq, const dmuon_heads* dk, void* dw_q,
                                void* dw_k, void* workspace, size_t ws_bytes,
                                cudaStream_t stream) {
  if (!qk_shape_ok(shape) || workspace == nullptr) return DMUON_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return DMUON_ERR_ALIGNMENT;
  if (ws_bytes < qk_workspace(*shape)) return DMUON_ERR_WORKSPACE;
  const dmuon_heads *x[2] = {q, k}, *dout[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
  const void* w[2] = {w_q, w_k};
  void* dw[2] = {dw_q, shape->k_heads > 0 ? dw_k : nullptr};
  float* partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kHdrBytes);
  return qk_norm_rope(shape, x, dout, out, w, inv_freq, position, dw, partial, stream);
}

size_t dmuon_linattn_workspace_bytes(const dmuon_linattn_shape* shape, int backward) {
  (void)backward;
  return linattn_shape_ok(shape) ? linattn_workspace(*shape) : 0;
}

int dmuon_linattn_forward(const dmuon_linattn_shape* shape, const dmuon_heads* q,
                          const dmuon_heads* k, const dmuon_heads* v, const float* log_decay,
                          const int32_t* offsets, const float* state, float* final_state,
                          const dmuon_heads* out, void* workspace, size_t ws_bytes,
                          cudaStream_t stream) {
  int e = check_common(shape, log_decay, offsets, state, final_state, workspace, ws_bytes);
  if (e != DMUON_OK) return e;
  const dmuon_linattn_shape& s = *shape;
  if (s.tokens == 0 && final_state == nullptr) return DMUON_OK;
  // without tokens the states still pass through: a tensor of one token that no sequence has
  dmuon_linattn_shape one = s;
  dmuon_heads dummy{workspace, s.heads * 128, 128};
  if (s.tokens == 0) {
    one.tokens = 1;
    q = k = v = out = &dummy;
  }
  const Rows qr = checked(q, one, s.key_dim, &e), kr = checked(k, one, s.key_dim, &e),
             vr = checked(v, one, s.value_dim, &e), orow = checked(out, one, s.value_dim, &e);
  if (e != DMUON_OK) return e;
  const States first(state, s, s.sequences), last(final_state, s, s.sequences);
  if (!last.beside(first)) return DMUON_ERR_INVALID_ARG;
  if (s.tokens > 0) {
    if (overlap(orow, qr) || overlap(orow, kr) || overlap(orow, vr) || first.meets(orow))
      return DMUON_ERR_INVALID_ARG;
    for (const Rows* r : {&qr, &kr, &vr, &orow})
      if (last.meets(*r)) return DMUON_ERR_INVALID_ARG;
  }
  Device device;
  e = device_ready(&device);
  if (e != DMUON_OK) return e;
  const Sweep w{&qr, &kr, &vr, &orow, false, state, final_state, false, false};
  return run_sweeps(s, &w, 1, log_decay, offsets, device, workspace, stream);
}

int dmuon_linattn_backward(const dmuon_linattn_shape* shape, const dmuon_heads* dout,
                           const dmuon_heads* q, const dmuon_heads* k, const dmuon_heads* v,
                           const float* log_decay, const int32_t* offsets, const float* state,
                           const float* dfinal_state, const dmuon_heads* dq,
                           const dmuon_heads* dk, const dmuon_heads* dv, float* dstate,
                           void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int e = check_common(shape, log_decay, offsets, state, dfinal_state, workspace, ws_bytes);
  if (e != DMUON_OK) return e;
  if (!aligned(dstate, 16)) return DMUON_ERR_ALIGNMENT;
  const dmuon_linattn_shape& s = *shape;
  if (s.tokens == 0 && dstate == nullptr) return DMUON_OK;
  dmuon_linattn_shape one = s;
  dmuon_heads dummy{workspace, s.heads * 128, 128};
  if (s.tokens == 0) {
    one.tokens = 1;
    dout = q = k = v = dq = dk = dv = &dummy;
  }
  const Rows dor = checked(dout, one, s.value_dim, &e), qr = checked(q, one, s.key_dim, &e),
             kr = checked(k, one, s.key_dim, &e), vr = checked(v, one, s.value_dim, &e),
             dqr = checked(dq, one, s.key_dim, &e), dkr = checked(dk, one, s.key_dim, &e),
             dvr = checked(dv, one, s.value_dim, &e);
  if (e != DMUON_OK) return e;
  const States first(state, s, s.sequences), dlast(dfinal_state, s, s.sequences),
      dfirst(dstate, s, s.sequences);
  if (!dfirst.beside(dlast)) return DMUON_ERR_INVALID_ARG;
  // the scale is a factor of q and dout then, on their way to the states' gradients: a range in which
  // elements up to 2^63 do not overflow by it
  if ((dfinal_state != nullptr || dstate != nullptr) &&
      !(std::fabs(s.scale) >= 0x1p-64f && std::fabs(s.scale) <= 0x1p64f))
    return DMUON_ERR_UNSUPPORTED;
  if (s.tokens > 0) {
    for (const Rows* o : {&dqr, &dkr, &dvr}) {
      if (first.meets(*o) || dlast.meets(*o)) return DMUON_ERR_INVALID_ARG;
      for (const Rows* i : {&dor, &qr, &kr, &vr})
        if (overlap(*o, *i)) return DMUON_ERR_INVALID_ARG;
    }
    for (const Rows* r : {&dor, &qr, &kr, &vr, &dqr, &dkr, &dvr})
      if (dfirst.meets(*r)) return DMUON_ERR_INVALID_ARG;
    if (overlap(dqr, dkr) || overlap(dqr, dvr) || overlap(dkr, dvr)) return DMUON_ERR_INVALID_ARG;
  }
  Device device;
  e = device_ready(&device);
  if (e != DMUON_OK) return e;
  // The states' gradients hold the scale, dout and q as they are read do not.
  const bool scaled = dfinal_state != nullptr || dstate != nullptr;
  const Sweep sweeps[3] = {{&dor, &vr, &kr, &dqr, false, state, nullptr, true, false},
                           {&vr, &dor, &qr, &dkr, true, dfinal_state, nullptr, true, scaled},
                           {&kr, &qr, &dor, &dvr, true, dfinal_state, dstate, false, scaled}};
  if (s.tokens == 0) return run_sweeps(s, sweeps + 2, 1, log_decay, offsets, device, workspace, stream);
  // The three side by side fill the GPU without cutting sequences as finely (8192 tokens of 32
  // heads in 5 sequences: 149 us; with dstate, in two launches with keys kept to 16 bits, 285).
  // Apart where dv's sweep is another kernel, or writes dstate, perhaps over the dfinal_state that
  // dk's reads.
  const bool apart = dstate != nullptr || (s.key_dim <= 64) != (s.value_dim <= 64);
  e = run_sweeps(s, sweeps, apart ? 2 : 3, log_decay, offsets, device, workspace, stream);
  if (e != DMUON_OK || !apart) return e;
  return run_sweeps(s, sweeps + 2, 1, log_decay, offsets, device, workspace, stream);
}

int dmuon_linattn_step(const dmuon_linattn_shape* shape, const dmuon_heads* q,
                       const dmuon_heads* k, const dmuon_heads* v, const float* log_decay,
                       const int32_t* slot, int64_t slots, const float* state, float* new_state,
                       const dmuon_heads* out, cudaStream_t stream) {
  if (!linattn_shape_ok(shape) || log_decay == nullptr || slots < 0) return DMUON_ERR_INVALID_ARG;
  const dmuon_linattn_shape& s = *shape;
  if (s.tokens == 0) return DMUON_OK;
  if (state == nullptr || new_state == nullptr || (slot == nullptr && slots < s.tokens))
    return DMUON_ERR_INVALID_ARG;
  if (!aligned(state, 16) || !aligned(new_state, 16) || !aligned(log_decay, 4) || !aligned(slot, 4))
    return DMUON_ERR_ALIGNMENT;
  LinStepArgs g{};
  Rows qr, kr, vr, orow;
  if (!rows_of(q, s.tokens, s.heads, s.key_dim, &qr) ||
      !rows_of(k, s.tokens, s.heads, s.key_dim, &kr) ||
      !rows_of(v, s.tokens, s.heads, s.value_dim, &vr) ||
      !rows_of(out, s.tokens, s.heads, s.value_dim, &orow))
    return DMUON_ERR_INVALID_ARG;
  for (const Rows* r : {&qr, &kr, &vr, &orow})
    if (r->p % 2 != 0) return DMUON_ERR_ALIGNMENT;
  if (s.tokens * s.heads * ceil_div(s.value_dim, 32) > INT32_MAX) return DMUON_ERR_UNSUPPORTED;
  if (overlap(orow, qr) || overlap(orow, kr) || overlap(orow, vr)) return DMUON_ERR_INVALID_ARG;
  const int64_t reached = std::min(slots, int64_t(1) << 31);  // by int32 slots
  const States before(state, s, reached), after(new_state, s, reached);
  if (!after.beside(before) || before.meets(orow)) return DMUON_ERR_INVALID_ARG;
  for (const Rows* r : {&qr, &kr, &vr, &orow})
    if (after.meets(*r)) return DMUON_ERR_INVALID_ARG;
  Device device;
  const int e = device_ready(&device);
  if (e != DMUON_OK) return e;
  g.q = device_heads(qr);
  g.k = device_heads(kr);
  g.v = device_heads(vr);
  g.out = device_heads(orow);
  g.log_decay = log_decay;
  g.slot = slot;
  g.slots = slots;
  g.state = state;
  g.new_state = new_state;
  g.rows = int(s.tokens);
  g.heads = int(s.heads);
  g.dk = int(s.key_dim);
  g.dv = int(s.value_dim);
  g.scale = s.scale;
  return launch_linattn_step(g, stream) == cudaSuccess ? DMUON_OK : DMUON_ERR_CUDA;
}

}  // extern "C"
