// loss.h -- launch arguments of the training objectives (token_loss.cu,
// router_loss.cu), shared with their host entry points (loss_api.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

// moe_status of the current device (MOE_OK: compute capability 10.3), checked once per
// device; its SM count in sms_out unless null.
int device_status(int* sms_out);

// Logits types, as moe_dtype in include/moe_nvfp4.h.
enum LossDtype { kF32 = 0, kBf16 = 1, kF16 = 2 };

// Objectives over a row of vocabulary logits.
enum TokenLossMode { kPolicy = 0, kDistill = 1 };  // kPolicy without adv: logp alone

constexpr int kMaxTeacher = 256;     // teacher slots per row
constexpr int kMaxVocab = 1 << 18;   // logits per row

struct TokenLossArgs {
  int N, V;
  int64_t ld, ld_grad;      // row strides in elements
  const void* logits;       // [N][V]
  void* dlogits;            // [N][V], or null: losses only
  const float* row_weight;  // [N] upstream gradient of each row's loss, or null: 1
  float* row_loss;          // [N], or null
  float* logp;              // [N], or null
  float tau, inv_tau;       // temperature and its reciprocal
  float c2;                 // log2(e) / tau: exp(x / tau) = 2^(x c2)
  int ids64;                // actions / teacher ids are int64
  // kPolicy
  const void* actions;      // [N]
  const float* old_logp;
  const float* adv;         // or null: log-probabilities only
  const float* ref_logp;    // or null
  float clip_lo, clip_hi;   // bounds of the probability ratio
  float kl_coef;
  // kDistill
  int k;
  const void* t_ids;        // [N][k]
  const void* t_logits;     // [N][k]
  int t_dtype;
  const float* t_lse;       // [N] log-sum-exp of the teacher's whole row over tau, or null
};

// Roles of the long rows' kernel that its self-test makes leave.
enum LongRole { kConsumers = 0, kProducer = 1, kGather = 2, kFinish = 3 };
struct LeaveArgs {
  int role, rank, row;  // from this row of cluster 0 on, in the block of this rank
};

cudaError_t launch_token_loss(const TokenLossArgs& a, int mode, int dtype, cudaStream_t s);
// Blocks a row of V logits is divided among; 0: a short row.
int token_loss_cluster(int V, int dtype);
// The policy gradient of long bf16 rows by kLeaveClusters clusters, a role of which leaves.
constexpr int kLeaveClusters = 4;
cudaError_t launch_token_loss_leave(const TokenLossArgs& a, const LeaveArgs& leave,
                                    cudaStream_t s);

struct RouterLossArgs {
  int T, E, K, S;
  int64_t ld, ld_grad;
  const void* logits;         // [T][E]
  const void* ids;            // [T][K]
  int ids64;
  const uint8_t* mask;        // [T], 0 = row left out; or null
  const int32_t* offsets;     // [S+1] first row of each sequence; or null (S == 1, all rows)
  float balance_coef, z_coef;
  float* losses;              // [2] balance, z
  int32_t* counts;            // [S][E]
  int32_t* tokens;            // [S+1] live rows per sequence, then their sum
  void* ws;
  // gradient
  const float* loss_grad;     // [2] upstream gradients of losses, or null: 1
  const float* topk_w;        // [T][K] routing scores and
  const float* d_topk_w;      // [T][K] their upstream gradients, or null
  void* dlogits;              // [T][E]
  bool aligned;               // rows are whole 16-byte vectors
  bool counts_aligned;        // as are the counts'
};

size_t router_loss_ws_bytes(int T, int E, int S);
cudaError_t launch_router_loss(const RouterLossArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_router_loss_grad(const RouterLossArgs& a, int dtype, cudaStream_t s);

// One logit as float.
template <int DT>
struct LogitType;
template <>
struct LogitType<kF32> {
  using type = float;
};
template <>
struct LogitType<kBf16> {
  using type = uint16_t;
};
template <>
struct LogitType<kF16> {
  using type = uint16_t;
};

}  // namespace moe
