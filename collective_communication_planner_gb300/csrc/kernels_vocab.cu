// Operators over vocabulary-parallel logits: log probabilities with entropy
// and top alternatives, distillation, and their gradients.
#include <cfloat>
#include <cmath>

#include "dispatch.cuh"
#include "vocab.h"

namespace tccl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

// 2^d: results below 2^-126 are 0, which is exact enough for a term of a sum
// whose largest term is 1
__device__ __forceinline__ float exp2_ftz(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d));
  return e;
}

template <int DT>
__device__ __forceinline__ float load_one(const void* p, uint64_t i) {
  if (DT == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void store_one(void* p, uint64_t i, float x) {
  if (DT == kBF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<float*>(p)[i] = x;
}

template <int DT>
__device__ __forceinline__ float logit(const VocabArgs& v, uint64_t t, uint32_t j) {
  return load_one<DT>(v.p.src[j / v.shard], t * v.src_stride + j % v.shard);
}

// Part of a row's softmax: the maximum m, s = sum 2^((x - m) c) and
// u = sum 2^((x - m) c) (x - m), c = log2(e) / temperature. No element: m = -inf.
struct Part {
  float m = -INFINITY, s = 0.f, u = 0.f;
  __device__ __forceinline__ void rescale(float to, float c) {
    if (m == ninf()) return;
    const float d = m - to, f = exp2_ftz(d * c);
    // terms that vanish beside 2^0 go before their (possibly infinite)
    // distance meets a product
    u = f == 0.f ? 0.f : f * (u + s * d);
    s *= f;
  }
  __device__ __forceinline__ void join(Part o, float c) {
    const float to = (o.m > m || o.m != o.m) ? o.m : m;
    rescale(to, c);
    o.rescale(to, c);
    m = to;
    s += o.s;
    u += o.u;
  }
  __device__ __forceinline__ void add(float x, float c) {
    if (x == ninf()) return;
    Part o;
    o.m = x;
    o.s = 1.f;
    o.u = 0.f;
    join(o, c);
  }
};

__device__ __forceinline__ Part shfl_xor(const Part& a, int o) {
  Part b;
  b.m = __shfl_xor_sync(0xFFFFFFFFu, a.m, o);
  b.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
  b.u = __shfl_xor_sync(0xFFFFFFFFu, a.u, o);
  return b;
}

// every thread of the block gets the joined part, joined in the same order
__device__ Part block_join(Part a, float c, Part* slots) {
  for (int o = 16; o > 0; o >>= 1) {
    Part b = shfl_xor(a, o);
    // the lower lane's part first, so both lanes compute the same bits
    if (threadIdx.x & o) {
      b.join(a, c);
      a = b;
    } else {
      a.join(b, c);
    }
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = a;
  __syncthreads();
  Part r = slots[0];
  for (int w = 1; w < kThreads / 32; ++w) r.join(slots[w], c);
  return r;
}

template <int DT>
__device__ Part row_part(const VocabArgs& v, uint64_t t, Part* slots) {
  Part a;
  for (uint32_t j = threadIdx.x; j < v.vocab; j += kThreads) a.add(logit<DT>(v, t, j), v.exp2_scale);
  return block_join(a, v.exp2_scale, slots);
}

// (value, column) as one number that orders alternatives: larger values
// first, the lower column first among equals. -inf is no alternative: 0.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t j) {
  if (!(x > ninf())) return 0;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as 0
  const uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return static_cast<uint64_t>(o) << 32 | (0xFFFFFFFFu - j);
}

__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

__device__ uint64_t block_max(uint64_t k, uint64_t* slots) {
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t b = __shfl_xor_sync(0xFFFFFFFFu, k, o);
    k = b > k ? b : k;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = k;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) k = slots[w] > k ? slots[w] : k;
  return k;
}

// log of the sum of 2^d terms, and log probabilities from a row's part
__device__ __forceinline__ float log_sum(const Part& a) { return a.m == ninf() ? 0.f : logf(a.s); }
__device__ __forceinline__ float log_prob(float x, const Part& a, float log_s, float inv_temp) {
  return x == ninf() && a.s == a.s ? x : (x - a.m) * inv_temp - log_s;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) log_probs_kernel(const __grid_constant__ LogProbsArgs a) {
  __shared__ Part parts[kThreads / 32];
  __shared__ uint64_t keys[kThreads / 32];
  if (threadIdx.x == 0) dev::record_sm(a.v.sm_mask);
  const VocabArgs& v = a.v;
  for (uint64_t t = blockIdx.x; t < v.rows; t += gridDim.x) {
    const int64_t token = a.tokens ? a.tokens[t] : 0;
    const bool scored = token >= 0 && token < v.vocab;
    Part r;
    if (scored) r = row_part<DT>(v, t, parts);
    const bool bad = !(r.s <= FLT_MAX);
    const float ls = log_sum(r);
    if (threadIdx.x == 0) {
      if (a.log_probs)
        a.log_probs[t] = scored ? log_prob(logit<DT>(v, t, static_cast<uint32_t>(token)), r, ls, v.inv_temp) : 0.f;
      if (a.entropy) a.entropy[t] = r.m == ninf() ? 0.f : ls - v.inv_temp * (r.u / r.s);
      if (a.stats) {
        a.stats[2 * t] = scored ? r.m : 0.f;
        a.stats[2 * t + 1] = ls;
      }
    }
    uint64_t last = ~0ull;
    for (int i = 0; i < a.top_k; ++i) {
      uint64_t best = 0;
      if (scored && !bad && last) {
        for (uint32_t j = threadIdx.x; j < v.vocab; j += kThreads) {
          const uint64_t k = key_of(logit<DT>(v, t, j), j);
          if (k < last && k > best) best = k;
        }
        best = block_max(best, keys);
      }
      last = best;
      if (threadIdx.x == 0) {
        const uint64_t o = t * a.top_k + i;
        a.top_ids[o] = best ? static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
        a.top_log_probs[o] = best ? log_prob(key_value(best), r, ls, v.inv_temp)
                                  : (scored && bad ? __int_as_float(0x7fc00000) : ninf());
      }
    }
  }
}

// writes g(j) to every column of row t, zeros in the padding
template <int DT, typename F>
__device__ void write_row(const VocabArgs& v, uint64_t t, bool zero, F g) {
  for (int r = 0; r < v.nranks; ++r)
    for (uint32_t c = threadIdx.x; c < v.shard; c += kThreads) {
      const uint32_t j = r * v.shard + c;
      float y = 0.f;
      if (!zero && j < v.vocab) y = g(load_one<DT>(v.p.src[r], t * v.src_stride + c), j);
      store_one<DT>(v.p.dst[r], t * v.dst_stride + c, y);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) log_probs_grad_kernel(const __grid_constant__ LogProbsGradArgs a) {
  if (threadIdx.x == 0) dev::record_sm(a.v.sm_mask);
  const VocabArgs& v = a.v;
  for (uint64_t t = blockIdx.x; t < v.rows; t += gridDim.x) {
    const int64_t token = a.tokens[t];
    const float m = a.stats[2 * t], ls = a.stats[2 * t + 1];
    const float da = a.d_log_probs[t], db = a.d_entropy ? a.d_entropy[t] : 0.f;
    const float h = db != 0.f ? a.entropy[t] : 0.f;
    const bool zero = token < 0 || token >= v.vocab || (da == 0.f && db == 0.f) || m == ninf();
    write_row<DT>(v, t, zero, [&](float x, uint32_t j) {
      const float lp = (x - m) * v.inv_temp - ls;
      const float p = exp2_ftz(lp * 1.44269504f);
      float y = p == 0.f ? 0.f : -p * (da + db * (lp + h));
      if (j == token) y += da;
      return y * v.inv_temp;
    });
  }
}

// The teacher's entries of row t: q per entry (0: empty) and log q, in shared
// memory; returns Q.
struct Teacher {
  float q[kMaxTop], log_q[kMaxTop];
  int64_t id[kMaxTop];
};

__device__ float read_teacher(const DistillArgs& a, uint64_t t, Teacher* s) {
  __syncthreads();
  if (threadIdx.x < a.top_k) {
    const uint64_t o = t * a.top_k + threadIdx.x;
    const int64_t id = a.ids[o];
    const bool has = id >= 0 && id < a.v.vocab;
    s->id[threadIdx.x] = has ? id : -1;
    const float x = a.teacher_bf16 ? load_one<kBF16>(a.teacher, o) : load_one<kF32>(a.teacher, o);
    s->log_q[threadIdx.x] = has ? x * a.v.inv_temp : ninf();
  }
  __syncthreads();
  float top = ninf(), lse = 0.f, total = 0.f;
  if (a.teacher_lse) {
    lse = a.teacher_lse[t];
  } else {
    for (int k = 0; k < a.top_k; ++k) top = fmaxf(top, s->log_q[k]);
    float sum = 0.f;
    for (int k = 0; k < a.top_k; ++k) sum += top == ninf() ? 0.f : expf(s->log_q[k] - top);
    lse = top == ninf() ? 0.f : top + logf(sum);
  }
  for (int k = 0; k < a.top_k; ++k) total += expf(s->log_q[k] - lse);
  __syncthreads();
  if (threadIdx.x < a.top_k) {
    const float lq = s->log_q[threadIdx.x] - lse;
    s->log_q[threadIdx.x] = lq;
    s->q[threadIdx.x] = expf(lq);
  }
  __syncthreads();
  return total;
}

template <int DT>
__device__ void distill_grad_row(const DistillArgs& a, uint64_t t, const Teacher& s, float total,
                                 float w, float m, float ls) {
  const VocabArgs& v = a.v;
  write_row<DT>(v, t, w == 0.f || total == 0.f || m == ninf(), [&](float x, uint32_t j) {
    float q = 0.f;
    for (int k = 0; k < a.top_k; ++k)
      if (s.id[k] == j) q += s.q[k];
    return w * v.inv_temp * (total * exp2_ftz(((x - m) * v.inv_temp - ls) * 1.44269504f) - q);
  });
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ Part parts[kThreads / 32];
  __shared__ Teacher s;
  if (threadIdx.x == 0) dev::record_sm(a.v.sm_mask);
  const VocabArgs& v = a.v;
  for (uint64_t t = blockIdx.x; t < v.rows; t += gridDim.x) {
    const float total = read_teacher(a, t, &s);
    const Part r = row_part<DT>(v, t, parts);
    const float ls = log_sum(r);
    if (threadIdx.x == 0) {
      float loss = 0.f;
      for (int k = 0; k < a.top_k; ++k)
        if (!(s.q[k] <= 0.f))
          loss += s.q[k] * (s.log_q[k] - log_prob(logit<DT>(v, t, static_cast<uint32_t>(s.id[k])), r, ls, v.inv_temp));
      a.loss[t] = loss;
      if (a.stats) {
        a.stats[2 * t] = r.m;
        a.stats[2 * t + 1] = ls;
      }
    }
    if (a.weights) {
      __syncthreads();  // the loss reads the logits before an in-place gradient replaces them
      distill_grad_row<DT>(a, t, s, total, a.weights[t], r.m, ls);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ Teacher s;
  if (threadIdx.x == 0) dev::record_sm(a.v.sm_mask);
  for (uint64_t t = blockIdx.x; t < a.v.rows; t += gridDim.x) {
    const float total = read_teacher(a, t, &s);
    distill_grad_row<DT>(a, t, s, total, a.weights[t], a.saved[2 * t], a.saved[2 * t + 1]);
  }
}

template <typename Args>
int launch(void (*bf16)(Args), void (*f32)(Args), int dtype, const Args& a, int sm_count, int cap,
           int* ctas, int* threads, void* stream) {
  uint64_t grid = static_cast<uint64_t>(sm_count) * 8;
  if (grid > a.v.rows) grid = a.v.rows;
  if (cap > 0 && grid > static_cast<uint64_t>(cap)) grid = cap;
  *ctas = static_cast<int>(grid);
  *threads = kThreads;
  (dtype == kBF16 ? bf16 : f32)<<<static_cast<unsigned>(grid), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_log_probs(int dtype, const LogProbsArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream) {
  return launch<LogProbsArgs>(log_probs_kernel<kBF16>, log_probs_kernel<kF32>, dtype, a, sm_count, cap, ctas, threads, stream);
}

int launch_log_probs_grad(int dtype, const LogProbsGradArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream) {
  return launch<LogProbsGradArgs>(log_probs_grad_kernel<kBF16>, log_probs_grad_kernel<kF32>, dtype, a, sm_count, cap, ctas, threads, stream);
}

int launch_distill(int dtype, const DistillArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream) {
  return launch<DistillArgs>(distill_kernel<kBF16>, distill_kernel<kF32>, dtype, a, sm_count, cap, ctas, threads, stream);
}

int launch_distill_grad(int dtype, const DistillArgs& a, int sm_count, int cap, int* ctas, int* threads, void* stream) {
  return launch<DistillArgs>(distill_grad_kernel<kBF16>, distill_grad_kernel<kF32>, dtype, a, sm_count, cap, ctas, threads, stream);
}

}  // namespace tccl
