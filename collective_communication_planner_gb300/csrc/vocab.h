// Operators over vocabulary-parallel logits: launch arguments and limits.
#pragma once

#include "internal.h"

namespace tccl {

constexpr int kMaxTop = 128;

// A [rows, vocab] matrix of logits cut by columns over `used` rank buffers.
struct VocabArgs {
  BasePtrs<kMaxRanks> p;  // src: logits, dst: gradients (gradient calls)
  uint32_t* sm_mask;
  uint64_t rows;
  uint64_t src_stride, dst_stride;  // elements from a row to the next
  uint32_t vocab, shard;
  int nranks;
  int used;         // ranks that hold valid columns
  float inv_temp;   // 1 / temperature
  float exp2_scale; // log2(e) / temperature
};

struct LogProbsArgs {
  VocabArgs v;
  const int64_t* tokens;
  float *log_probs, *entropy, *stats;
  float* top_log_probs;
  int64_t* top_ids;
  int top_k;
};

struct LogProbsGradArgs {
  VocabArgs v;
  const int64_t* tokens;
  const float *stats, *entropy, *d_log_probs, *d_entropy;
};

struct DistillArgs {
  VocabArgs v;
  const int64_t* ids;
  const void* teacher;
  const float* teacher_lse;
  float *loss, *stats;        // forward: outputs (stats may be null)
  const float* weights;       // with a gradient
  const float* saved;         // gradient alone: the forward's stats
  int top_k;
  int teacher_bf16;
};

int launch_log_probs(int dtype, const LogProbsArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream);
int launch_log_probs_grad(int dtype, const LogProbsGradArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream);
int launch_distill(int dtype, const DistillArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream);
int launch_distill_grad(int dtype, const DistillArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream);

}  // namespace tccl
