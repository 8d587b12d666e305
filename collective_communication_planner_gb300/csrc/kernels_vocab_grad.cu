// Gradients of vocabulary-parallel log probabilities and of distillation, the
// latter also in one pass with its loss.
#include "vocab_device.cuh"

namespace tccl {
namespace {

using namespace vocab;

constexpr int kThreads = 256;
constexpr uint64_t kKeepBytes = 52ull << 20;  // rows that L2 keeps between two reads

// The segments of the current row for a gradient: where the logits and the
// gradient start, and the first element of the body, which starts on a 16-byte
// boundary of the gradient. Where the logits do not, a vector is put together
// from two aligned ones, and the body leaves both ends of the segment enough
// elements that those lie within it.
struct GradSegments : Segments {
  char* dst[kMaxRanks];
  template <int DT>
  __device__ __forceinline__ char* to(uint32_t seg, uint32_t col) const {
    return dst[seg] + static_cast<uint64_t>(col) * Elem<DT>::kBytes;
  }
};

template <int DT>
__device__ __forceinline__ uint32_t head_of(const char* dst) {
  return static_cast<uint32_t>(-reinterpret_cast<uintptr_t>(dst) & 15) / Elem<DT>::kBytes + Elem<DT>::kVec;
}

template <int DT>
__device__ __forceinline__ void set_segments(const VocabArgs& v, uint64_t t, GradSegments& s) {
  if (threadIdx.x < v.used) {
    s.src[threadIdx.x] = static_cast<const char*>(v.p.src[threadIdx.x]) + t * v.src_stride * Elem<DT>::kBytes;
    char* dst = static_cast<char*>(v.p.dst[threadIdx.x]) + t * v.dst_stride * Elem<DT>::kBytes;
    s.dst[threadIdx.x] = dst;
    s.head[threadIdx.x] = v.aligned ? 0 : head_of<DT>(dst);
  }
}

// One row's gradient y = p (scale + slope log2 p); columns that a token or a
// teacher's entry names get their own term afterwards.
// log2 p = x c - (max c + log2_s): the subtrahend is rounded once (hi), so
// that it takes one fused operation an element, and what the rounding lost is
// made up for in scale and slope. A row whose maximum is not within
// (-2^100, 2^100) is not `fast`: (x - max) c - log2_s then.
struct RowGrad {
  float max, c, log2_s, hi, scale, slope, fast_scale, fast_slope;
  bool zero, fast;

  __device__ __forceinline__ void set(const VocabArgs& v, float m, float log2_sum, float to_scale, float to_slope) {
    max = m;
    c = v.exp2_scale;
    log2_s = log2_sum;
    fast = fabsf(m) < -kClamp;
    scale = to_scale;
    slope = to_slope;
    const float mc = __fmul_rn(m, c);
    hi = __fadd_rn(mc, log2_s);
    // max c + log2_s - hi: the product's rounding, and the sum's (two-sum)
    const float back = __fsub_rn(hi, mc);
    const float lost = __fadd_rn(__fadd_rn(__fsub_rn(mc, __fsub_rn(hi, back)), __fsub_rn(log2_s, back)),
                                 __fmaf_rn(m, c, -mc));
    const float f = exp2_ftz(-lost);
    fast_scale = f * __fmaf_rn(-slope, lost, scale);
    fast_slope = f * slope;
  }
  __device__ __forceinline__ float one(float x) const {
    const float l = fast ? __fmaf_rn(x, c, -hi) : (x - max) * c - log2_s, p = exp2_ftz(l);
    const float s = fast ? fast_slope : slope, o = fast ? fast_scale : scale;
    // a masked place: 0 whatever its distance
    return p == 0.f ? 0.f : p * (s == 0.f ? o : __fmaf_rn(s, l, o));
  }
  template <bool SLOPE>
  __device__ __forceinline__ f32x2 two(f32x2 x) const {
    const f32x2 l = fma2(x, pack(c, c), pack(-hi, -hi));
    const f32x2 p = exp2x2(l);
    if (!SLOPE) return mul2(p, pack(fast_scale, fast_scale));
    return mul2(p, fma2(pack(fast_slope, fast_slope), l, pack(fast_scale, fast_scale)));
  }
};

// The gradient of a vector of the row. A named column's own term is not in it:
// a branch for it here would keep the vectors of a chunk from overlapping
// (GB300, 4096 x 131072 bf16: 452 us with it, 314 without).
template <int DT, bool SLOPE>
__device__ __forceinline__ uint4 grad_of(const RowGrad& g, Vec<DT>& x) {
  Vec<DT> y;
  if (g.fast) {
    if (SLOPE) x.clamp();  // a masked place: 0 times a finite distance
#pragma unroll
    for (int i = 0; i < Vec<DT>::kPairs; ++i) y.put_pair(i, g.two<SLOPE>(x.pair(i)));
  } else {
#pragma unroll
    for (int i = 0; i < Vec<DT>::kPairs; ++i) y.put_pair(i, pack(g.one(x.get(2 * i)), g.one(x.get(2 * i + 1))));
  }
  return y.out();
}

// The gradient of this warp's chunks of [lo, hi) of the row. In place a lane
// reads a vector before it replaces it, and no other lane reads it: the
// buffers are equally aligned then.
template <int DT, bool SLOPE>
__device__ __forceinline__ void store_chunks(const VocabArgs& v, const GradSegments& s, const RowGrad& g, uint32_t lo,
                                             uint32_t hi) {
  for (ChunkWalk w(v.cut, lo + (threadIdx.x >> 5)); w.index < hi; w.next(v.cut)) {
    Vec<DT> x[kBatch];
    const uint32_t first = w.vector(), end = w.vectors(v), head = s.head[w.seg];
    load_chunk<DT, true>(v, s.at<DT>(w.seg, head), w, x, StreamLoad());
    char* to = s.to<DT>(w.seg, head) + static_cast<uint64_t>(first) * 16;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (first + k * 32 >= end) break;
      dev::st_global_v4(to + k * 512, grad_of<DT, SLOPE>(g, x[k]));
    }
  }
}

template <int DT>
__device__ __forceinline__ void zero_chunks(const VocabArgs& v, const GradSegments& s, uint32_t lo, uint32_t hi) {
  for (ChunkWalk w(v.cut, lo + (threadIdx.x >> 5)); w.index < hi; w.next(v.cut)) {
    const uint32_t first = w.vector(), end = w.vectors(v);
    char* to = s.to<DT>(w.seg, s.head[w.seg]) + static_cast<uint64_t>(first) * 16;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (first + k * 32 < end) dev::st_global_v4(to + k * 512, make_uint4(0, 0, 0, 0));
  }
}

// The edge elements of the row, by CTA 0 of the row's, and the zeros of its
// padding columns, shared by all of them.
template <int DT>
__device__ __forceinline__ void store_edges(const VocabArgs& v, const GradSegments& s, const RowGrad& g, uint64_t t,
                                            uint32_t cta, uint32_t ctas) {
  for (uint32_t e = threadIdx.x; cta == 0 && e < v.cut.edges; e += blockDim.x) {
    uint32_t seg, col;
    edge_at<DT>(v, s, e, seg, col);
    store_one<DT>(s.to<DT>(seg, col), g.zero ? 0.f : g.one(load_one<DT>(s.at<DT>(seg, col))));
  }
  const uint32_t all = v.nranks * v.shard;
  for (uint32_t j = v.vocab + cta * blockDim.x + threadIdx.x; j < all; j += ctas * blockDim.x) {
    const uint32_t r = j / v.shard;
    store_one<DT>(static_cast<char*>(v.p.dst[r]) + (t * v.dst_stride + (j - r * v.shard)) * Elem<DT>::kBytes, 0.f);
  }
}

// Work item b of a call is part b % parts of row b / parts: an equal share of its chunks.
struct Item {
  uint64_t row;
  uint32_t part, lo, hi;
  __device__ __forceinline__ Item(const VocabArgs& v, uint64_t b, uint32_t parts) {
    row = b >> 32 ? b / parts : static_cast<uint32_t>(b) / parts;
    part = static_cast<uint32_t>(b - row * parts);
    const uint32_t per = (v.cut.chunks + parts - 1) / parts;
    lo = min(v.cut.chunks, part * per);
    hi = min(v.cut.chunks, lo + per);
  }
};


// the chunk that a column of row t is in, or kEdge
constexpr uint32_t kEdge = 0xFFFFFFFFu;
template <int DT>
__device__ __forceinline__ uint32_t chunk_of(const VocabArgs& v, uint64_t t, uint32_t column) {
  const uint32_t seg = column / v.shard, col = column - seg * v.shard;
  const char* dst = static_cast<const char*>(v.p.dst[seg]) + t * v.dst_stride * Elem<DT>::kBytes;
  const uint32_t head = v.aligned ? 0 : head_of<DT>(dst);
  const uint32_t vectors = seg + 1 == v.used ? v.cut.last : v.cut.full, vec = (col - head) / Elem<DT>::kVec;
  if (col < head || vec >= vectors) return kEdge;
  return seg * v.cut.per_segment + vec / kChunkVectors;
}

// whether a CTA that has chunks [lo, hi) of row t, and with `edges` the edge
// elements, has a column
template <int DT>
__device__ __forceinline__ bool has_column(const VocabArgs& v, uint64_t t, uint32_t column, uint32_t lo, uint32_t hi,
                                           bool edges) {
  const uint32_t chunk = chunk_of<DT>(v, t, column);
  return chunk == kEdge ? edges : chunk >= lo && chunk < hi;
}

template <int DT>
__device__ __forceinline__ float read_column(const VocabArgs& v, uint64_t t, uint32_t column) {
  const uint32_t seg = column / v.shard;
  return load_one<DT>(static_cast<const char*>(v.p.src[seg]) +
                      (t * v.src_stride + column - seg * v.shard) * Elem<DT>::kBytes);
}
template <int DT>
__device__ __forceinline__ void write_column(const VocabArgs& v, uint64_t t, uint32_t column, float y) {
  const uint32_t seg = column / v.shard;
  store_one<DT>(static_cast<char*>(v.p.dst[seg]) + (t * v.dst_stride + column - seg * v.shard) * Elem<DT>::kBytes, y);
}

template <int DT, bool SLOPE>
__global__ void __launch_bounds__(kThreads, 5) log_probs_grad_kernel(const __grid_constant__ LogProbsGradArgs a) {
  __shared__ GradSegments seg;
  const VocabArgs& v = a.v;
  start(1);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  for (uint64_t b = blockIdx.x; b < v.rows * v.parts; b += gridDim.x) {
    const Item it(v, b, v.parts);
    const uint64_t t = it.row;
    set_segments<DT>(v, t, seg);  // the last item's are done with: the barrier below
    const int64_t token = a.tokens[t];
    const float da = a.d_log_probs[t], db = SLOPE ? a.d_entropy[t] : 0.f, m = a.stats[2 * t];
    const float ls = a.stats[2 * t + 1], h = SLOPE && db != 0.f ? a.entropy[t] : 0.f;
    RowGrad g;
    // log p in base 2: log p = ln 2 log2 p
    g.set(v, m, ls * kLog2e, -(da + db * h) * v.inv_temp, -db * v.inv_temp * kLn2);
    g.zero = token < 0 || token >= v.vocab || (da == 0.f && db == 0.f) || m == -INFINITY;
    // thread 0 gives the token's column its own term after the body's stores;
    // it reads the logit first, since an in-place gradient replaces it
    const uint32_t column = static_cast<uint32_t>(token);
    const bool named = threadIdx.x == 0 && !g.zero && has_column<DT>(v, t, column, it.lo, it.hi, it.part == 0);
    const float x = named ? read_column<DT>(v, t, column) : 0.f;
    __syncthreads();
    if (g.zero) zero_chunks<DT>(v, seg, it.lo, it.hi);
    else store_chunks<DT, SLOPE>(v, seg, g, it.lo, it.hi);
    store_edges<DT>(v, seg, g, t, it.part, v.parts);
    __syncthreads();
    if (named) write_column<DT>(v, t, column, g.one(x) + da * v.inv_temp);
  }
}

// ---------------------------------------------------------------- distillation
// The teacher's columns that fall to this CTA, in entry order: after the
// body's stores those columns get their own value.
struct Named {
  int32_t column[kMaxTop];
  float q[kMaxTop], x[kMaxTop];
  float total;
  int count;
};

// Warp 0 keeps the entries of the row whose column is in chunks [lo, hi), or,
// with `edges`, an edge element, in entry order, with the logits there, since an
// in-place gradient replaces them.
template <int DT>
__device__ __forceinline__ void keep_named(const VocabArgs& v, uint64_t t, const TeacherRow& r, Named& n, uint32_t lo,
                                           uint32_t hi, bool edges) {
  int count = 0;
#pragma unroll
  for (int i = 0; i < kMaxTop / 32; ++i) {
    const bool here = r.column[i] >= 0 && has_column<DT>(v, t, r.column[i], lo, hi, edges);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, here);
    if (here) {
      const int at = count + __popc(mask & ((1u << (threadIdx.x & 31)) - 1));
      n.column[at] = r.column[i];
      n.q[at] = r.q[i];
      n.x[at] = read_column<DT>(v, t, r.column[i]);
    }
    count += __popc(mask);
  }
  if ((threadIdx.x & 31) == 0) {
    n.count = count;
    n.total = r.total;
  }
}

// after a barrier behind the body's stores
template <int DT>
__device__ __forceinline__ void store_named(const VocabArgs& v, uint64_t t, const Named& n, const RowGrad& g, float weight) {
  const int i = threadIdx.x;
  if (i >= n.count) return;
  const int32_t column = n.column[i];
  float q = 0.f;
  for (int j = 0; j < n.count; ++j) {
    if (n.column[j] != column) continue;
    if (j < i) return;  // an earlier entry names it too and does this
    q += n.q[j];
  }
  write_column<DT>(v, t, column, g.one(n.x[i]) - q * weight);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 5) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ GradSegments seg;
  __shared__ Named named;
  const VocabArgs& v = a.v;
  start(1);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  for (uint64_t b = blockIdx.x; b < v.rows * v.parts; b += gridDim.x) {
    const Item it(v, b, v.parts);
    const uint64_t t = it.row;
    const float w = a.weights[t] * v.inv_temp, m = a.saved[2 * t], ls = a.saved[2 * t + 1];
    bool zero = w == 0.f || m == -INFINITY;
    __syncthreads();  // the last item's segments and columns are done with
    set_segments<DT>(v, t, seg);
    if (!zero && threadIdx.x < 32) keep_named<DT>(v, t, read_teacher(a, t), named, it.lo, it.hi, it.part == 0);
    __syncthreads();
    zero = zero || named.total == 0.f;
    RowGrad g;
    g.set(v, m, ls * kLog2e, w * named.total, 0.f);
    g.zero = zero;
    if (zero) zero_chunks<DT>(v, seg, it.lo, it.hi);
    else store_chunks<DT, false>(v, seg, g, it.lo, it.hi);
    store_edges<DT>(v, seg, g, t, it.part, v.parts);
    if (!zero) {
      __syncthreads();
      store_named<DT>(v, t, named, g, w);
    }
  }
}

constexpr int kStepCluster = 8;
constexpr int kStepCtasPerSm = 5;

// Loss and gradient in one call: a cluster of CTAs sums up a row, joins its
// statistics through distributed shared memory and reads it again, from L2,
// for the gradient.
template <int DT>
__global__ void __launch_bounds__(kThreads, kStepCtasPerSm) distill_step_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ GradSegments seg;
  __shared__ Named named;
  __shared__ LossSlots loss;
  __shared__ JoinSlots slots;
  const VocabArgs& v = a.v;
  const uint32_t ctas = cluster_size(), cta = cluster_rank();
  const uint32_t per = (v.cut.chunks + ctas - 1) / ctas;
  const uint32_t lo = min(v.cut.chunks, cta * per), hi = min(v.cut.chunks, lo + per);
  start(ctas);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  int phase = 0;
  const float c = v.exp2_scale;
  for (uint64_t t = blockIdx.x / ctas; t < v.rows; t += gridDim.x / ctas) {
    __syncthreads();  // the last row's segments and columns are done with
    set_segments<DT>(v, t, seg);
    __syncthreads();
    if (threadIdx.x < 32) {
      const TeacherRow q = read_teacher(a, t);
      keep_named<DT>(v, t, q, named, lo, hi, cta == 0);
      if (cta == 0) set_loss<DT>(v, seg, q, loss);
    }
    Part p = scan_row<DT, false, true>(v, seg, lo, hi, cta == 0, KeepLoad(), [](float) {});
    p = row_join(p, c, slots, phase, ctas);
    const bool fast = fabsf(p.m) < -kClamp;
    const Stats st = fast ? stats_of(p, c) : slow_stats<DT>(v, seg, lo, hi, slots, phase, cta, ctas);
    if (cta == 0 && threadIdx.x < 32) store_loss(a, t, loss, st);
    const float w = a.weights[t] * v.inv_temp;
    RowGrad g;
    g.set(v, st.max, st.log2_s, w * named.total, 0.f);
    g.zero = w == 0.f || named.total == 0.f || st.empty();
    // An in-place gradient may be written from here on: past the join's
    // barrier a CTA reads its own columns only, each before it replaces it.
    if (g.zero) zero_chunks<DT>(v, seg, lo, hi);
    else store_chunks<DT, false>(v, seg, g, lo, hi);
    store_edges<DT>(v, seg, g, t, cta, ctas);
    if (!g.zero) {
      __syncthreads();
      store_named<DT>(v, t, named, g, w);
    }
  }
}

template <int DT, typename Args>
int launch_parts(void (*kernel)(Args), Args& a, VocabLaunch& l) {
  VocabArgs& v = a.v;
  set_cut<DT>(v, 2);
  // an item is at most eight chunks a warp; fewer where that leaves SMs
  // without four items
  constexpr uint32_t kWarps = kThreads / 32;
  uint32_t deep = 8;
  while (deep > 1 && v.rows * ((v.cut.chunks + deep * kWarps - 1) / (deep * kWarps)) < static_cast<uint64_t>(l.sm_count) * 4)
    deep /= 2;
  v.parts = v.cut.chunks > deep * kWarps ? (v.cut.chunks + deep * kWarps - 1) / (deep * kWarps) : 1;
  uint64_t grid = v.rows * v.parts;
  const uint64_t most = l.cap > 0 ? static_cast<uint64_t>(l.cap) : static_cast<uint64_t>(1) << 30;
  if (grid > most) grid = most;
  return launch_rows(kernel, a, l, grid, kThreads, 1, 0);
}

template <int DT>
int launch_step_t(DistillArgs& a, VocabLaunch& l) {
  VocabArgs& v = a.v;
  set_cut<DT>(v, 2);
  // CTAs of a row: few enough rows at once for L2 to keep them between the two
  // reads, or as many as the SMs take of few rows; every warp gets a chunk
  const uint64_t row_bytes = static_cast<uint64_t>(v.vocab) * Elem<DT>::kBytes;
  const uint64_t resident = static_cast<uint64_t>(l.sm_count) * kStepCtasPerSm;
  const auto kept = [&](int c) { return (v.rows < resident / c ? v.rows : resident / c) * row_bytes; };
  int c = 1;
  while (c < kStepCluster && v.cut.chunks >= static_cast<uint32_t>(2 * c * kThreads / 32) &&
         (l.cap <= 0 || 2 * c <= l.cap) && (v.rows * 2 * c <= resident || kept(c) > kKeepBytes))
    c *= 2;
  uint64_t rows = v.rows;
  if (l.cap > 0 && rows * c > static_cast<uint64_t>(l.cap)) rows = l.cap / c;
  const uint64_t most = static_cast<uint64_t>(1) << 27;
  return launch_rows(distill_step_kernel<DT>, a, l, (rows < most ? rows : most) * c, kThreads, c, 0);
}

}  // namespace

int launch_log_probs_grad(int dtype, LogProbsGradArgs& a, VocabLaunch& l) {
  if (dtype == kBF16)
    return launch_parts<kBF16>(a.d_entropy ? log_probs_grad_kernel<kBF16, true> : log_probs_grad_kernel<kBF16, false>, a, l);
  return launch_parts<kF32>(a.d_entropy ? log_probs_grad_kernel<kF32, true> : log_probs_grad_kernel<kF32, false>, a, l);
}

int launch_distill(int dtype, DistillArgs& a, VocabLaunch& l) {
  if (!a.weights) return vocab::launch_distill_forward(dtype, a, l);
  return dtype == kBF16 ? launch_step_t<kBF16>(a, l) : launch_step_t<kF32>(a, l);
}

int launch_distill_grad(int dtype, DistillArgs& a, VocabLaunch& l) {
  return dtype == kBF16 ? launch_parts<kBF16>(distill_grad_kernel<kBF16>, a, l)
                        : launch_parts<kF32>(distill_grad_kernel<kF32>, a, l);
}

}  // namespace tccl
