// Operators over vocabulary-parallel logits: launch arguments and limits.
#pragma once

#include "internal.h"

namespace tccl {

constexpr int kMaxTop = 128;

// How the row kernels walk a row. Every rank's segment of a row is cut into
// 16-byte vectors plus edge elements, with the same number of vectors in
// every full segment, so that one index runs over the vectors of all ranks.
struct VocabCut {
  uint32_t full, last; // vectors of a full segment, of the last one
  uint32_t divisor;    // full, but at least 1
  uint32_t vectors;    // vectors of a row
  uint32_t edge;       // edge elements of a full segment
  uint32_t edges;      // edge elements of a row
  // a step of `threads` vectors in (segment, vector) form
  uint32_t step_seg, step_vec;
};

// A [rows, vocab] matrix of logits cut by columns over `used` rank buffers.
struct VocabArgs {
  BasePtrs<kMaxRanks> p;  // src: logits, dst: gradients (gradient calls)
  uint32_t* sm_mask;
  uint64_t rows;
  uint64_t src_stride, dst_stride;  // elements from a row to the next
  uint32_t vocab, shard;
  int nranks;
  int used;         // ranks that hold valid columns
  int aligned;      // every row of every buffer starts on a 16-byte boundary
  float inv_temp;   // 1 / temperature
  float exp2_scale; // log2(e) / temperature
  VocabCut cut;
};

struct LogProbsArgs {
  VocabArgs v;
  const int64_t* tokens;
  float *log_probs, *entropy, *stats;
  float* top_log_probs;
  int64_t* top_ids;
  int top_k;
  int batches;      // batches of vectors a thread takes of its slice
  int batch_shift;  // 2^batch_shift batches share one stored maximum
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

struct VocabLaunch {
  int sm_count, cap;
  void* stream;
  int ctas, threads;  // out
};

// Each returns a cudaError_t as int.
int launch_log_probs(int dtype, LogProbsArgs& a, VocabLaunch& l);
int launch_log_probs_grad(int dtype, LogProbsGradArgs& a, VocabLaunch& l);
int launch_distill(int dtype, DistillArgs& a, VocabLaunch& l);
int launch_distill_grad(int dtype, DistillArgs& a, VocabLaunch& l);

}  // namespace tccl
