// Tables and host-side launchers of the training-side operators: the gated
// feed-forward block, softmax cross entropy over a vocabulary, and activations
// kept in 8 bits.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"

namespace dm {

// ------------------------------------------------------------------ shared with dmuon_api.cu
// Status of the current device (DMUON_OK when it is usable), its SM count and
// how many CTA pairs of the product kernels fit on it at once.
int library_device(int* device, int* sms, int* max_clusters);
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                     const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncode library_tensor_map_encoder();

// ------------------------------------------------------------------ tensor-core products
// Elements of one 8-bit activation block (they share a bf16 scale).
constexpr int kActBlock = 32;
// Vocabulary entries whose exponentials share a reference maximum (plain and
// swapped orientation).
constexpr int kXentGroup = 128, kXentGroupSwap = 32;
// Exponentials wait in fp16 times this, the largest power of two that keeps 1 finite: 11 bits
// down to 2^-29 of their group's largest (e^-20; without it 2^-14, e^-9.7), 2^-40 absolute
// below.
constexpr float kXentScale = 32768.f;
// The most tokens for which the logits run swapped (a workspace is sized by it).
constexpr int kXentSwapTokens = 1024;

// What a product's epilogue does with the fp32 accumulator.
enum LinEpi {
  kLinStore = 0,    // C = bf16(acc), optionally through an fp32 running sum
  kLinGlu = 1,      // h = act(gate) * up, gate / up kept as asked
  kLinGluGrad = 2,  // acc = dh: dgate, dup and h from the kept gate / up
  kLinXent = 3      // logits: group maxima and sums, exponentials kept as asked
};
// What a product may load while the launch before it still runs.
enum LinEarly {
  kEarlyNone = 0,     // nothing: a call's first product
  kEarlyWeights = 1,  // the weight operand
  kEarlyAll = 2       // weight gradients: both operands are older than that launch
};
enum LinKeep { kKeepNone = 0, kKeepBf16 = 1, kKeepAct8 = 2 };

// K-elements of a pipeline stage, the unit of kb0 and kb1.
__host__ __device__ constexpr int lin_stage_k(int epi, bool swap) {
  return swap || epi == kLinGluGrad ? 64 : 128;
}
constexpr int kLinMaps = 13;     // tensor maps of one launch
constexpr int kLinProblems = 3;  // products of one launch

struct LinProblem {
  int rows, cols;        // output extent (rows: tokens, except for weight gradients)
  int tiles_m, tiles_n;  // tile grid of the product (swapped: m counts columns, n rows)
  int kb0, kb1;          // K blocks from the first and the second operand pair
  int tile_begin;        // first tile of this product in the launch
  unsigned strip_magic, last_magic;  // division by the tiles of a strip, by the last strip's rows
  int a0, b0, a1, b1;    // operand maps (kLinGlu: gate's weight b0, up's b1; swapped a0, a1;
                         // weight gradients: a1, b1 for the last K block)
  int c_map;             // output map, or -1: c is written with plain stores
  __nv_bfloat16* c;
  long long c_ld;
  long long sum_at;      // where its running sum starts in LinArgs::sum
};

struct LinArgs {
  CUtensorMap maps[kLinMaps];
  LinProblem prob[kLinProblems];
  int n_prob, n_maps;
  int swap, nt, stages;  // swapped orientation: tokens per tile, pipeline stages
  int early;             // LinEarly
  int k_tail;            // weight gradients: tokens in the last K block (a multiple of 16)
  int full_tiles;        // tiles computed whole; the rest in `split` parts along K
  int split;
  unsigned split_magic;
  int total_units;       // full_tiles + split * (tiles - full_tiles)
  float* partial;        // fp32 parts of the split tiles
  int* err;
  // kLinStore, plain: fp32 running sums over launches (row pitch = cols of the product).  One
  // address for all products: testing one of each product's own costs 0.3 us a launch.
  float* sum;
  int sum_read, sum_write;  // add what a sum holds; write there instead of C
  const float* scale;    // C = scale * acc (device scalar), or null
  // kLinGlu / kLinGluGrad
  int act, keep;
  int ffn;
  int kept_vec;          // rows of the kept tensors allow 16-byte access
  void *gate, *up;                          // bf16 values or 8-bit codes
  __nv_bfloat16 *gate_scale, *up_scale;     // 8-bit block scales
  int map_gate, map_up;                     // their maps, 32 x 32 boxes (kept_vec)
  int map_dup, map_h;                       // kLinGluGrad: output maps beside c_map (dgate)
  __nv_bfloat16 *dup, *h;                   // and their tensors (pitch c_ld)
  // kLinXent
  const long long* target;
  float2* group_stat;    // (max logit, sum of exp(logit - that)) per [group][token], the
                         // token's target left out
  long long stat_ld;     // pitch of a group
};

size_t lin_partial_bytes();
cudaError_t lin_prepare();  // once per device
// Split the tiles of the last, partly filled wave along K (sets full_tiles ..
// total_units from the products' tile counts).
void lin_schedule(LinArgs& g, int epi, int clusters);
// Whether a product over `tokens` rows and k K-elements runs swapped, and its tokens per tile.
bool lin_swaps(long long tokens, int epi, long long k, int* nt);
cudaError_t launch_lin(const LinArgs& g, int epi, bool a_mn, bool b_mn, int max_clusters,
                       cudaStream_t s);

// Launch a kernel that may start while the one before it in the stream still runs
// (it calls grid_wait() before it writes, or reads what that one writes).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned blocks, unsigned threads,
                             cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

// ------------------------------------------------------------------ few tokens
constexpr int kThinTokens = 8;
struct ThinArgs {
  const __nv_bfloat16 *x, *w0, *w1;  // w1: up's weight
  long long x_ld, w_ld, out_ld;
  __nv_bfloat16 *out, *gate, *up;    // gate, up: kept projections (contiguous) or null
  int tokens, k, cols, act;
};
// out = x w0^T, or act(x w0^T) * (x w1^T); k a multiple of 8, rows 16-byte aligned.
cudaError_t launch_thin(const ThinArgs& g, bool glu, cudaStream_t s);

// ------------------------------------------------------------------ memory-bound kernels
cudaError_t launch_act8_save(long long rows, long long cols, const void* x, long long ld,
                             bool bf16, signed char* codes, __nv_bfloat16* scales,
                             cudaStream_t s);
cudaError_t launch_act8_load(long long rows, long long cols, const signed char* codes,
                             const __nv_bfloat16* scales, void* out, long long ld, bool bf16,
                             cudaStream_t s);
// Copies of bf16 matrices (src null: zeros), one launch; with `target`, rows of the
// first whose target lies outside [0, vocab) become zeros; with `grad_loss` also the
// scale that the gradients of the logits are formed relative to.
struct CopyArgs {
  static constexpr int kMost = 5;
  struct Mat {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    long long rows, cols, src_ld, dst_ld;
    unsigned block_begin;
    int src_vec, dst_vec;  // 16-byte aligned rows
  };
  Mat mat[kMost];
  int n;
  const long long* target;
  long long vocab;
  const float* grad_loss;  // of `tokens` tokens
  long long tokens;
  float* grad_scale;       // out: largest |grad_loss| of tokens with a target, 1 if 0
  void add(const __nv_bfloat16* src, long long src_ld, __nv_bfloat16* dst, long long dst_ld,
           long long rows, long long cols) {
    Mat& M = mat[n++];
    M.src = src;
    M.dst = dst;
    M.rows = rows;
    M.cols = cols;
    M.src_ld = src_ld;
    M.dst_ld = dst_ld;
  }
};
cudaError_t launch_copy_rows(CopyArgs& g, cudaStream_t s);
struct XentRows {
  long long tokens, vocab;
  const long long* target;
  const float* grad_loss;   // null: no gradients
  const float* grad_scale;  // G is formed of grad_loss / *grad_scale
  const __nv_bfloat16 *hidden, *weight;  // rows of k elements, 16-byte aligned
  long long hidden_ld, weight_ld;
  int k;
  const float2* group_stat;  // as LinArgs
  long long stat_ld;
  int group;                // vocabulary entries per group
  float *loss, *lse;
};
cudaError_t launch_xent_rows(const XentRows& r, cudaStream_t s);
// Exponentials (fp16) to gradients of the logits (bf16), in place.
cudaError_t launch_xent_grad(const XentRows& r, void* e, long long e_ld, cudaStream_t s);

}  // namespace dm
