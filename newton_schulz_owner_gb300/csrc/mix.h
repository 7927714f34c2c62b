// Host-side launchers of the operators that mix tokens: the norms and rotation of query
// and key heads, and linear attention with a decay for each head.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "train.h"

namespace dm {

// Rows of heads: element (t, h, i) at p[t * ts + h * hs + i].
struct Heads {
  __nv_bfloat16* p;
  long long ts, hs;
};

// ------------------------------------------------------------------ norms and rotation
struct RopeArgs {
  // [0]: queries, [1]: keys.  Forward: x -> out.  Backward: x and dy -> out = dx.
  Heads x[2], dy[2], out[2];
  const __nv_bfloat16* w[2];
  const float* inv_freq;
  const int32_t* position;
  int tokens, heads[2], dim, rotary;
  float eps;
  int per, parts;             // chunks of heads that a warp takes, warps of a token
  float* partial;             // backward: sums of the gains' gradients, one row per block
  __nv_bfloat16* dw[2];       // or null
};
constexpr int kRopeBlocks = 1216;  // most blocks of a backward launch
// vec: every row lies at an 8-byte address.
cudaError_t launch_rope(RopeArgs& g, bool backward, bool interleaved, bool vec, int sms,
                        cudaStream_t s);

// ------------------------------------------------------------------ linear attention
// One sweep over every sequence, along time or against it (mix_kernel in linattn.cu), with
// a = exp(log_decay):
//   along:    S_t = a S_{t-1} + k_t v_t^T,      out_t = scale q_t S_t       state_out = S behind the last
//   against:  R_t = R_{t+1} + k_t v_t^T,        out_t = scale q_t R_t,
//             then decayed on its way to t - 1:  R_t <- a R_t               state_out = R before the first
// state_in and state_out are what the sweep keeps: S, or with key_scale = scale, scale S (R alike).
struct LinAttnArgs {
  CUtensorMap q, k, v, o;     // loads: 64 x 1 x 128 boxes; o: stores of 32 x 1 x 32
  const float* log_decay;
  const int32_t* offsets;
  int sequences, heads, tokens, dk, dv;
  float scale;
  int against;
  const float* state_in;      // or null
  float* state_out;           // or null
  // The state kept is S or R itself (1 and scale), or scale times it (scale and 1): what the keys are
  // multiplied by on the way to it, and the queries' product with it on its way out.
  float key_scale, state_scale;
  int st_row, st_col;         // element strides of a state (row: the keys' side)
  Heads out;
  int groups;                 // runs that a head's sequences are cut into, a cluster each
  int split;                  // CTAs of a cluster
  int exact;                  // keys are kept to 16 bits in the state
  float* local;               // states on the way from CTA to CTA
  int* err;
};
constexpr int kMixBlock = 128;   // tokens taken at a time
constexpr int kMixMaxSplit = 8;
constexpr size_t kMixLocalBytes = size_t(128) * 128 * 4;  // of a state
constexpr int kMixSlots = 2;            // states of a CTA in the workspace
constexpr int64_t kMixMaxCtas = 320;    // of a launch whose sequences are shared
// Once per device: shared memory opt-in; fit[n] is how many clusters of n CTAs run at once.
cudaError_t linattn_prepare(int (&fit)[kMixMaxSplit + 1]);
// Sweeps of one launch: of the same sizes (padded to 64 or 128), sharing and precision.
struct LinAttnSweeps {
  LinAttnArgs sweep[3];
  int count;
  int deal;  // CTAs that all sequences of all heads and sweeps are dealt to whole, 0: not dealt
};
constexpr int kMixDealt = 32;  // most sequences that a CTA is dealt
cudaError_t launch_linattn(const LinAttnSweeps& g, cudaStream_t s);

struct LinStepArgs {
  Heads q, k, v, out;
  const float* log_decay;
  const int32_t* slot;
  long long slots;
  const float* state;
  float* new_state;
  int rows, heads, dk, dv;
  float scale;
};
cudaError_t launch_linattn_step(const LinStepArgs& g, cudaStream_t s);

}  // namespace dm
