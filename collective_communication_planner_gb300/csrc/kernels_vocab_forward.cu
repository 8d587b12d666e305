// Forward passes over vocabulary-parallel logits: log probabilities with
// entropy and top alternatives, and the distillation loss.
#include "vocab_device.cuh"

namespace tccl {
namespace {

using namespace vocab;

constexpr int kThreads = 256;
constexpr int kMaxEntries = 64;    // stored chunk maxima per thread
constexpr int kMaxWork = 512;      // of them looked at again for alternatives
constexpr int kMaxCandidates = 1024;
constexpr int kForwardCluster = 8;

// The smallest bf16 number that is not below x, as its bits.
__device__ __forceinline__ uint16_t bf16_above(float x) {
  const uint32_t b = __float_as_uint(x);
  return static_cast<uint16_t>((b & 0x80000000u) ? b >> 16 : (b + 0xFFFFu) >> 16);
}

// The statistics of a row over the cluster. With TOP, the maximum of every
// 2^shift chunks is kept in `tops` for the alternatives, and thread_max set.
template <int DT, bool ENTROPY, bool TOP>
__device__ __forceinline__ Stats row_stats(const VocabArgs& v, const Segments& seg, uint32_t lo, uint32_t hi,
                                           uint32_t cta, uint32_t ctas, JoinSlots& slots, int& phase,
                                           uint16_t* tops, int shift, float& thread_max) {
  int chunk = 0;
  float entry = kClamp;
  Part a = scan_row<DT, ENTROPY, false>(v, seg, lo, hi, cta == 0, StreamLoad(), [&](float top) {
    if (!TOP) return;
    entry = fmaxf(entry, top);
    tops[(chunk >> shift) * kThreads + threadIdx.x] = bf16_above(entry);
    if ((++chunk & ((1 << shift) - 1)) == 0) entry = kClamp;
  });
  thread_max = a.m;
  a = row_join(a, v.exp2_scale, slots, phase, ctas);
  if (fabsf(a.m) < -kClamp) return stats_of(a, v.exp2_scale);
  return slow_stats<DT>(v, seg, lo, hi, slots, phase, cta, ctas);
}

// ---------------------------------------------------------------- alternatives
// A value and its column as one number that orders alternatives: larger
// values first, the lower column first among equals. 0: no alternative (-inf).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as 0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t column) {
  if (!(x > -INFINITY)) return 0;
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xFFFFFFFFu - column);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  return order_value(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int64_t key_column(uint64_t k) {
  return static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

// One warp: a value that at least k of the threads' maxima (as orders) reach,
// and not many more. Bisection: a comparison of all pairs of maxima instead
// took 1300 instructions a warp, and most of a decode batch's time.
__device__ __forceinline__ float warp_threshold(const uint32_t* order, int k) {
  constexpr int N = kThreads / 32;
  uint32_t mine[N], least = 0xFFFFFFFFu, most = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mine[i] = order[i * 32 + (threadIdx.x & 31)];
    least = min(least, mine[i]);
    most = max(most, mine[i]);
  }
  uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, least), hi = __reduce_max_sync(0xFFFFFFFFu, most);
  // lo is reached by at least k; nothing above hi is reached at all
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += mine[i] >= mid;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (n < k) {
      hi = mid - 1;
      continue;
    }
    lo = mid;
    if (n <= k + k / 8) break;
  }
  return order_value(lo);
}

struct TopSlots {
  uint64_t candidate[kMaxCandidates];
  uint64_t sorted[kMaxTop];
  uint32_t order[kThreads];  // every thread's maximum
  uint32_t work[kMaxWork];   // entry * kThreads + thread
  int candidates, works;
  float threshold;
  int found;
};

__device__ __forceinline__ void offer(TopSlots& t, float x, uint32_t column) {
  const uint64_t k = key_of(x, column);
  if (!k) return;
  const int i = atomicAdd(&t.candidates, 1);
  if (i < kMaxCandidates) t.candidate[i] = k;
}

// The best k of the first n candidates, sorted, into t.sorted; t.found of
// them. Keys differ, so a key's place is the number of larger ones. All threads.
__device__ void sort_candidates(TopSlots& t, int n, int k) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = t.candidate[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += t.candidate[j] > mine;
    if (place < k) t.sorted[place] = mine;
  }
  if (threadIdx.x == 0) t.found = min(n, k);
  __syncthreads();
}

// The same for any row, one element a thread and step: keeps the best k so far
// and drops what is below the k-th whenever the list is nearly full.
template <int DT>
__device__ __noinline__ void select_by_scan(const VocabArgs& v, const Segments& seg, uint32_t lo, uint32_t hi,
                                            bool edges, TopSlots& t, int k) {
  constexpr int K = Elem<DT>::kVec;
  __syncthreads();
  if (threadIdx.x == 0) t.candidates = 0;
  uint64_t floor_key = 0;
  const auto prune = [&](bool last) {
    __syncthreads();
    const int n = t.candidates;
    if (!last && n <= kMaxCandidates - kThreads) {
      __syncthreads();  // nobody adds before everybody has read
      return;
    }
    sort_candidates(t, n, k);
    if (!last) {
      if (t.found == k) floor_key = t.sorted[k - 1];
      for (int i = threadIdx.x; i < t.found; i += kThreads) t.candidate[i] = t.sorted[i];
      if (threadIdx.x == 0) t.candidates = t.found;
      __syncthreads();
    }
  };
  const auto take = [&](bool on, float x, uint32_t column) {
    if (on && key_of(x, column) > floor_key) offer(t, x, column);
    prune(false);
  };
  __syncthreads();
  ChunkWalk w(v.cut, lo + threadIdx.x / 32);
  for (uint32_t i = lo; i < hi; i += kThreads / 32, w.next(v.cut, v.step)) {
    for (int k = 0; k < kBatch; ++k) {
      const bool on = w.index < hi && w.vector() + k * 32 < w.vectors(v);
      const uint32_t col = on ? seg.head[w.seg] + (w.vector() + k * 32) * K : 0;
      for (int j = 0; j < K; ++j)
        take(on, on ? load_one<DT>(seg.at<DT>(w.seg, col + j)) : 0.f, w.seg * v.shard + col + j);
    }
  }
  for (uint32_t e0 = 0; edges && e0 < v.cut.edges; e0 += kThreads) {
    const uint32_t e = e0 + threadIdx.x;
    const bool on = e < v.cut.edges;
    uint32_t es = 0, col = 0;
    if (on) edge_at<DT>(v, seg, e, es, col);
    take(on, on ? load_one<DT>(seg.at<DT>(es, col)) : 0.f, es * v.shard + col);
  }
  prune(true);
}

// The best k columns among this CTA's chunks [lo, hi) and edge elements,
// sorted, in t.sorted[0 .. t.found). A value that k of the threads' maxima
// reach is at most the k-th largest element, so only the lanes' shares of
// chunks whose maximum reaches it are read again.
template <int DT>
__device__ void select_top(const VocabArgs& v, const Segments& seg, uint32_t lo, uint32_t hi, bool edges,
                           TopSlots& t, int k, const uint16_t* tops, int shift,
                           float thread_max, bool slow) {
  constexpr int K = Elem<DT>::kVec;
  if (slow) {  // the maxima were clamped
    select_by_scan<DT>(v, seg, lo, hi, edges, t, k);
    return;
  }
  t.order[threadIdx.x] = order_of(thread_max);
  if (threadIdx.x == 0) t.candidates = t.works = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float found = warp_threshold(t.order, k);
    if (threadIdx.x == 0) t.threshold = found;
  }
  __syncthreads();
  const float threshold = t.threshold;
  const auto reaches = [&](float x) { return x >= threshold && x > kClamp; };
  const int warps = kThreads / 32, warp = threadIdx.x / 32;
  const int chunks = lo + warp < hi ? (hi - lo - warp + warps - 1) / warps : 0;
  const int entries = (chunks + (1 << shift) - 1) >> shift;
  for (int i = 0; i < entries; ++i) {
    if (reaches(__uint_as_float(static_cast<uint32_t>(tops[i * kThreads + threadIdx.x]) << 16))) {
      const int n = atomicAdd(&t.works, 1);
      if (n < kMaxWork) t.work[n] = i * kThreads + threadIdx.x;
    }
  }
  for (uint32_t e = threadIdx.x; edges && e < v.cut.edges; e += kThreads) {
    uint32_t es, col;
    edge_at<DT>(v, seg, e, es, col);
    const float x = load_one<DT>(seg.at<DT>(es, col));
    if (reaches(x)) offer(t, x, es * v.shard + col);
  }
  __syncthreads();
  if (t.works <= kMaxWork) {
    const int per = kBatch << shift, items = t.works * per;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const uint32_t job = t.work[i / per], thread = job % kThreads;
      const uint32_t chunk = lo + ((job / kThreads << shift) + i % per / kBatch) * warps + thread / 32;
      if (chunk >= hi) continue;
      const ChunkWalk w(v.cut, chunk);
      const uint32_t vec = w.part * kChunkVectors + i % kBatch * 32 + thread % 32;
      if (vec >= w.vectors(v)) continue;
      const uint32_t col = seg.head[w.seg] + vec * K;
      Vec<DT> x;
      x.set(dev::ld_global_v4(seg.at<DT>(w.seg, col)));
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (reaches(x.get(j))) offer(t, x.get(j), w.seg * v.shard + col + j);
    }
  }
  __syncthreads();
  const int n = t.candidates;
  bool whole = t.works > kMaxWork || n > kMaxCandidates;
  if (!whole && n < k) {
    // fewer than k columns above the clamp: there may be some below it
    bool below = false;
    each_element<DT>(v, seg, lo, hi, edges, [&](float x) { below = below || (x <= kClamp && x > -INFINITY); });
    whole = __syncthreads_or(below);
  }
  if (whole) select_by_scan<DT>(v, seg, lo, hi, edges, t, k);
  else sort_candidates(t, n, k);
}

struct ClusterTop {
  uint64_t list[kForwardCluster][kMaxTop];
  uint64_t count[kForwardCluster];
  int place[kMaxTop];
};

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 5) log_probs_kernel(const __grid_constant__ LogProbsArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Segments seg;
  __shared__ JoinSlots slots;
  TopSlots* top = reinterpret_cast<TopSlots*>(dynamic);
  ClusterTop* both = reinterpret_cast<ClusterTop*>(dynamic + sizeof(TopSlots));
  const VocabArgs& v = a.v;
  const uint32_t ctas = cluster_size(), cta = cluster_rank();
  uint16_t* tops = reinterpret_cast<uint16_t*>(dynamic + sizeof(TopSlots) + (ctas > 1 ? sizeof(ClusterTop) : 0));
  const uint32_t per = (v.cut.chunks + ctas - 1) / ctas;
  const uint32_t lo = min(v.cut.chunks, cta * per), hi = min(v.cut.chunks, lo + per);
  start(ctas);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  int phase = 0;
  for (uint64_t t = blockIdx.x / ctas; t < v.rows; t += gridDim.x / ctas) {
    const int64_t token = a.tokens ? a.tokens[t] : 0;
    const bool scored = token >= 0 && token < v.vocab;  // the same in every thread of the cluster
    Stats st{0.f, 0.f, 0.f};
    float x = 0.f, thread_max = 0.f;
    if (scored) {
      __syncthreads();  // the last row's segments are done with
      set_segments<DT>(v, t, seg);
      __syncthreads();
      if (a.tokens && threadIdx.x == 0)
        x = load_one<DT>(seg.at_column<DT>(v, static_cast<uint32_t>(token)));
      st = row_stats<DT, true, TOP>(v, seg, lo, hi, cta, ctas, slots, phase, tops, a.entry_shift, thread_max);
    }
    if (threadIdx.x == 0 && cta == 0) {
      if (a.tokens) a.log_probs[t] = scored ? st.log_prob(x, v.inv_temp) : 0.f;
      if (a.entropy) a.entropy[t] = st.entropy;
      if (a.stats) {
        a.stats[2 * t] = st.max;
        a.stats[2 * t + 1] = st.log2_s * kLn2;
      }
    }
    if (!TOP) continue;
    const int k = a.top_k;
    float* out_lp = a.top_log_probs + t * k;
    int64_t* out_id = a.top_ids + t * k;
    int found = 0;
    if (scored && !st.bad() && !st.empty()) {
      select_top<DT>(v, seg, lo, hi, cta == 0, *top, k, tops, a.entry_shift, thread_max,
                     !(fabsf(st.max) < -kClamp));
      const int mine = top->found;
      if (ctas == 1) {
        found = mine;
        for (int i = threadIdx.x; i < mine; i += kThreads) {
          out_lp[i] = st.log_prob(key_value(top->sorted[i]), v.inv_temp);
          out_id[i] = key_column(top->sorted[i]);
        }
      } else {
        // every CTA gets every CTA's sorted list and places its own keys by
        // the number of larger ones in each list
        for (int i = threadIdx.x; i < mine * static_cast<int>(ctas); i += kThreads)
          remote_store(remote(&both->list[cta][i / ctas], i % ctas), top->sorted[i / ctas]);
        if (threadIdx.x < ctas) remote_store(remote(&both->count[cta], threadIdx.x), static_cast<uint64_t>(mine));
        if (threadIdx.x < k) both->place[threadIdx.x] = 0;
        cluster_barrier();
        for (int i = threadIdx.x; i < mine * static_cast<int>(ctas); i += kThreads) {
          const uint64_t key = top->sorted[i / ctas];
          const uint64_t* list = both->list[i % ctas];
          int l = 0, h = static_cast<int>(both->count[i % ctas]);
          while (l < h) {
            const int mid = (l + h) / 2;
            if (list[mid] > key) l = mid + 1;
            else h = mid;
          }
          if (l) atomicAdd(&both->place[i / ctas], l);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < mine; i += kThreads) {
          const int place = both->place[i];
          if (place >= k) continue;
          out_lp[place] = st.log_prob(key_value(top->sorted[i]), v.inv_temp);
          out_id[place] = key_column(top->sorted[i]);
        }
        for (uint32_t q = 0; q < ctas; ++q) found += static_cast<int>(both->count[q]);
      }
    }
    if (cta == 0)
      for (int i = found + threadIdx.x; i < k; i += kThreads) {
        out_lp[i] = scored && st.bad() ? NAN : -INFINITY;
        out_id[i] = -1;
      }
  }
}

// ---------------------------------------------------------------- distillation
template <int DT>
__global__ void __launch_bounds__(kThreads, 5) distill_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ Segments seg;
  __shared__ JoinSlots slots;
  __shared__ Entries entries;
  const VocabArgs& v = a.v;
  const uint32_t ctas = cluster_size(), cta = cluster_rank();
  const uint32_t per = (v.cut.chunks + ctas - 1) / ctas;
  const uint32_t lo = min(v.cut.chunks, cta * per), hi = min(v.cut.chunks, lo + per);
  start(ctas);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  int phase = 0;
  for (uint64_t t = blockIdx.x / ctas; t < v.rows; t += gridDim.x / ctas) {
    __syncthreads();  // the last row's segments are done with
    set_segments<DT>(v, t, seg);
    __syncthreads();
    const bool mine = cta == 0 && threadIdx.x < 32;
    if (mine) {
      const TeacherRow q = read_teacher(a, t);
      uint32_t x[kMaxTop / 32];
      load_named<DT>(v, t, q, x);
      set_entries<DT>(q, x, a.top_k, entries, [](uint32_t) { return false; });
    }
    float unused;
    const Stats st = row_stats<DT, false, false>(v, seg, lo, hi, cta, ctas, slots, phase, nullptr, 0, unused);
    if (mine) store_loss(a, t, entries, st);
  }
}

// CTAs of one row: as many as keep every SM at no more than four, but none
// whose slice is less than one chunk of every warp.
int cluster_for(const VocabArgs& v, const VocabLaunch& l) {
  int c = 1;
  while (c < kForwardCluster && v.rows * c * 2 <= static_cast<uint64_t>(l.sm_count) * 4 &&
         v.cut.chunks >= static_cast<uint32_t>(2 * c * kThreads / 32) && (l.cap <= 0 || 2 * c <= l.cap))
    c *= 2;
  return c;
}

uint64_t grid_for(const VocabArgs& v, const VocabLaunch& l, int cluster) {
  uint64_t rows = v.rows;
  if (l.cap > 0 && rows * cluster > static_cast<uint64_t>(l.cap)) rows = l.cap / cluster;
  // far more rows than fit at once: a bounded grid takes the rest in turn
  const uint64_t most = static_cast<uint64_t>(1) << 20;
  return (rows < most ? rows : most) * cluster;
}

template <int DT, bool TOP>
int launch_log_probs_t(LogProbsArgs& a, VocabLaunch& l) {
  set_cut<DT>(a.v, 0);
  const int c = cluster_for(a.v, l);
  size_t smem = 0;
  a.entry_shift = 0;
  if (TOP) {
    const uint32_t per = (a.v.cut.chunks + c - 1) / c, warps = kThreads / 32, most = (per + warps - 1) / warps;
    while (((most + (1u << a.entry_shift) - 1) >> a.entry_shift) > kMaxEntries) ++a.entry_shift;
    const uint32_t entries = (most + (1u << a.entry_shift) - 1) >> a.entry_shift;
    smem = sizeof(TopSlots) + (c > 1 ? sizeof(ClusterTop) : 0) + sizeof(uint16_t) * kThreads * entries;
    const cudaError_t e = cudaFuncSetAttribute(log_probs_kernel<DT, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  return launch_rows(log_probs_kernel<DT, TOP>, a, l, grid_for(a.v, l, c), kThreads, c, smem);
}

template <int DT>
int launch_distill_t(DistillArgs& a, VocabLaunch& l) {
  set_cut<DT>(a.v, 0);
  const int c = cluster_for(a.v, l);
  return launch_rows(distill_kernel<DT>, a, l, grid_for(a.v, l, c), kThreads, c, 0);
}

}  // namespace

int launch_log_probs(int dtype, LogProbsArgs& a, VocabLaunch& l) {
  if (dtype == kBF16) return a.top_k ? launch_log_probs_t<kBF16, true>(a, l) : launch_log_probs_t<kBF16, false>(a, l);
  return a.top_k ? launch_log_probs_t<kF32, true>(a, l) : launch_log_probs_t<kF32, false>(a, l);
}

int launch_distill(int dtype, DistillArgs& a, VocabLaunch& l) {
  if (a.weights) return vocab::launch_distill_step(dtype, a, l);
  return dtype == kBF16 ? launch_distill_t<kBF16>(a, l) : launch_distill_t<kF32>(a, l);
}

}  // namespace tccl
