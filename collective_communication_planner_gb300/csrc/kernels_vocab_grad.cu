// Gradients of vocabulary-parallel log probabilities and of distillation, the
// latter also in one pass with its loss.
#include "vocab_device.cuh"

namespace tccl {
namespace {

using namespace vocab;

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // vectors a thread holds

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
__device__ __forceinline__ void set_segments(const VocabArgs& v, uint64_t t, GradSegments& s) {
  if (threadIdx.x < v.used) {
    s.src[threadIdx.x] = static_cast<const char*>(v.p.src[threadIdx.x]) + t * v.src_stride * Elem<DT>::kBytes;
    char* dst = static_cast<char*>(v.p.dst[threadIdx.x]) + t * v.dst_stride * Elem<DT>::kBytes;
    s.dst[threadIdx.x] = dst;
    const uint32_t gap = static_cast<uint32_t>(-reinterpret_cast<uintptr_t>(dst) & 15) / Elem<DT>::kBytes;
    s.head[threadIdx.x] = v.aligned ? 0 : gap + Elem<DT>::kVec;
  }
}

// sixteen bytes from an address that is aligned to its elements only
__device__ __forceinline__ uint4 load_any(const char* at) {
  const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 15);
  if (m == 0) return dev::ld_global_v4(at);
  const uint4 a = dev::ld_global_v4(at - m), b = dev::ld_global_v4(at - m + 16);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (m & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (m & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t bits = (m & 3) * 8;
  uint4 r;
  r.x = __funnelshift_r(w[0], w[1], bits);
  r.y = __funnelshift_r(w[1], w[2], bits);
  r.z = __funnelshift_r(w[2], w[3], bits);
  r.w = __funnelshift_r(w[3], w[4], bits);
  return r;
}

// One row's gradient y = p (scale + slope log2 p), plus `hot` at `token`,
// where p = 2^((x - max) c - log2_s).
struct RowGrad {
  float max, c, log2_s, scale, slope, hot;
  uint32_t token;
  bool zero, fast;

  __device__ __forceinline__ void set(const VocabArgs& v, float m, float log_s) {
    max = m;
    c = v.exp2_scale;
    log2_s = log_s * kLog2e;
    slope = hot = 0.f;
    token = 0xFFFFFFFFu;
    fast = fabsf(m) < -kClamp;
  }
  __device__ __forceinline__ float one(float x, uint32_t column) const {
    const float l = (x - max) * c - log2_s, p = exp2_ftz(l);
    // a masked place: 0 whatever its distance
    float y = p == 0.f ? 0.f : p * (slope == 0.f ? scale : __fmaf_rn(slope, l, scale));
    if (column == token) y += hot;
    return y;
  }
  template <bool SLOPE>
  __device__ __forceinline__ f32x2 two(f32x2 x) const {
    const f32x2 l = fma2(add2(x, pack(-max, -max)), pack(c, c), pack(-log2_s, -log2_s));
    const f32x2 p = exp2x2(l);
    if (!SLOPE) return mul2(p, pack(scale, scale));
    return mul2(p, fma2(pack(slope, slope), l, pack(scale, scale)));
  }
};

// The gradient of N vectors already in registers (clamped where the row is
// `fast`), stored; the vectors a thread holds are Walk's from `first`.
template <int DT, int N, bool SLOPE>
__device__ __forceinline__ void store_vectors(const VocabArgs& v, const GradSegments& s, const RowGrad& g,
                                              Vec<DT> (&x)[N], uint32_t first, uint32_t hi) {
  constexpr int K = Elem<DT>::kVec;
  Walk w(v.cut, first);
#pragma unroll
  for (int k = 0; k < N; ++k, w.next(v.cut)) {
    if (w.index >= hi) break;
    const uint32_t col = s.head[w.seg] + w.vec * K;
    const uint32_t hot = g.token - (w.seg * v.shard + col);
    Vec<DT> y;
    if (g.fast) {
      f32x2 r[Vec<DT>::kPairs];
#pragma unroll
      for (int i = 0; i < Vec<DT>::kPairs; ++i) r[i] = g.two<SLOPE>(x[k].pair(i));
      if (hot < K) {
#pragma unroll
        for (int i = 0; i < Vec<DT>::kPairs; ++i)
          if (i == hot / 2) r[i] = add2(r[i], hot & 1 ? pack(0.f, g.hot) : pack(g.hot, 0.f));
      }
#pragma unroll
      for (int i = 0; i < Vec<DT>::kPairs; ++i) y.put_pair(i, r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < Vec<DT>::kPairs; ++i)
        y.put_pair(i, pack(g.one(x[k].get(2 * i), w.seg * v.shard + col + 2 * i),
                           g.one(x[k].get(2 * i + 1), w.seg * v.shard + col + 2 * i + 1)));
    }
    dev::st_global_v4(s.to<DT>(w.seg, col), y.out());
  }
}

template <int DT, int N>
__device__ __forceinline__ void load_vectors(const VocabArgs& v, const GradSegments& s, Vec<DT> (&x)[N],
                                             uint32_t first, uint32_t hi) {
  Walk w(v.cut, first);
#pragma unroll
  for (int k = 0; k < N; ++k, w.next(v.cut)) {
    x[k].set_empty();
    if (w.index >= hi) continue;
    const char* at = s.at<DT>(w.seg, s.head[w.seg] + w.vec * Elem<DT>::kVec);
    x[k].set(v.aligned ? dev::ld_global_v4(at) : load_any(at));
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
    store_one<DT>(s.to<DT>(seg, col), g.zero ? 0.f : g.one(load_one<DT>(s.at<DT>(seg, col)), seg * v.shard + col));
  }
  const uint32_t all = v.nranks * v.shard;
  for (uint32_t j = v.vocab + cta * blockDim.x + threadIdx.x; j < all; j += ctas * blockDim.x) {
    const uint32_t r = j / v.shard;
    store_one<DT>(static_cast<char*>(v.p.dst[r]) + (t * v.dst_stride + (j - r * v.shard)) * Elem<DT>::kBytes, 0.f);
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_zeros(const VocabArgs& v, const GradSegments& s, uint32_t first, uint32_t hi) {
  Walk w(v.cut, first);
#pragma unroll
  for (int k = 0; k < N; ++k, w.next(v.cut))
    if (w.index < hi)
      dev::st_global_v4(s.to<DT>(w.seg, s.head[w.seg] + w.vec * Elem<DT>::kVec), make_uint4(0, 0, 0, 0));
}

// Pieces of rows: CTA b takes piece b % pieces of row b / pieces.
template <int DT, bool SLOPE>
__global__ void __launch_bounds__(kThreads) log_probs_grad_kernel(const __grid_constant__ LogProbsGradArgs a) {
  __shared__ GradSegments seg;
  const VocabArgs& v = a.v;
  const uint32_t pieces = max(1u, (v.cut.vectors + kThreads * kVecs - 1) / (kThreads * kVecs));
  start(1);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  for (uint64_t b = blockIdx.x; b < v.rows * pieces; b += gridDim.x) {
    const uint64_t t = b / pieces;
    const uint32_t piece = static_cast<uint32_t>(b - t * pieces), first = piece * kThreads * kVecs + threadIdx.x;
    __syncthreads();  // the last piece's segments are done with
    set_segments<DT>(v, t, seg);
    const int64_t token = a.tokens[t];
    const float da = a.d_log_probs[t], db = SLOPE ? a.d_entropy[t] : 0.f;
    RowGrad g;
    g.set(v, a.stats[2 * t], a.stats[2 * t + 1]);
    g.zero = token < 0 || token >= v.vocab || (da == 0.f && db == 0.f) || g.max == -INFINITY;
    g.scale = -da * v.inv_temp;
    if (SLOPE && db != 0.f) {
      // log p in base 2: log p = ln 2 log2 p
      g.scale = -(da + db * a.entropy[t]) * v.inv_temp;
      g.slope = -db * v.inv_temp * kLn2;
    }
    g.hot = da * v.inv_temp;
    g.token = static_cast<uint32_t>(token);
    __syncthreads();
    if (g.zero) {
      store_zeros<DT, kVecs>(v, seg, first, v.cut.vectors);
    } else {
      Vec<DT> x[kVecs];
      load_vectors<DT, kVecs>(v, seg, x, first, v.cut.vectors);
      if (SLOPE && g.fast)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) x[k].clamp();
      store_vectors<DT, kVecs, SLOPE>(v, seg, g, x, first, v.cut.vectors);
    }
    store_edges<DT>(v, seg, g, t, piece, pieces);
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

// Warp 0 keeps the entries of the row whose column belongs to vectors
// [lo, hi), or, for CTA `cta` of `ctas`, to its edge elements. Reads the
// logits there, since an in-place gradient replaces them.
template <int DT>
__device__ __forceinline__ void keep_named(const VocabArgs& v, const GradSegments& s, const TeacherRow& r, Named& n,
                                           uint32_t lo, uint32_t hi, uint32_t cta) {
  constexpr int K = Elem<DT>::kVec;
  int count = 0;
#pragma unroll
  for (int i = 0; i < kMaxTop / 32; ++i) {
    bool here = false;
    uint32_t seg = 0, col = 0;
    if (r.column[i] >= 0) {
      seg = r.column[i] / v.shard;
      col = r.column[i] - seg * v.shard;
      const uint32_t vec = (col - s.head[seg]) / K;  // huge before the head
      const uint32_t vectors = seg + 1 == v.used ? v.cut.last : v.cut.full;
      if (col < s.head[seg] || vec >= vectors) here = cta == 0;
      else here = seg * v.cut.full + vec >= lo && seg * v.cut.full + vec < hi;
    }
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, here);
    if (here) {
      const int at = count + __popc(mask & ((1u << (threadIdx.x & 31)) - 1));
      n.column[at] = r.column[i];
      n.q[at] = r.q[i];
      n.x[at] = load_one<DT>(s.at<DT>(seg, col));
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
__device__ __forceinline__ void store_named(const VocabArgs& v, const GradSegments& s, const Named& n, RowGrad g,
                                            float weight) {
  const int i = threadIdx.x;
  if (i >= n.count) return;
  const int32_t column = n.column[i];
  float q = 0.f;
  for (int j = 0; j < n.count; ++j) {
    if (n.column[j] != column) continue;
    if (j < i) return;  // an earlier entry names it too and does this
    q += n.q[j];
  }
  const uint32_t seg = column / v.shard, col = column - seg * v.shard;
  g.hot = -q * weight;
  g.token = column;
  store_one<DT>(s.to<DT>(seg, col), g.one(n.x[i], column));
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ GradSegments seg;
  __shared__ Named named;
  const VocabArgs& v = a.v;
  const uint32_t pieces = max(1u, (v.cut.vectors + kThreads * kVecs - 1) / (kThreads * kVecs));
  start(1);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  for (uint64_t b = blockIdx.x; b < v.rows * pieces; b += gridDim.x) {
    const uint64_t t = b / pieces;
    const uint32_t piece = static_cast<uint32_t>(b - t * pieces);
    const uint32_t lo = piece * kThreads * kVecs, first = lo + threadIdx.x;
    const uint32_t hi = min(v.cut.vectors, lo + kThreads * kVecs);
    __syncthreads();  // the last piece's segments and columns are done with
    set_segments<DT>(v, t, seg);
    const float w = a.weights[t] * v.inv_temp;
    RowGrad g;
    g.set(v, a.saved[2 * t], a.saved[2 * t + 1]);
    g.zero = w == 0.f || g.max == -INFINITY;
    __syncthreads();
    Vec<DT> x[kVecs];
    if (!g.zero) {
      load_vectors<DT, kVecs>(v, seg, x, first, hi);
      if (threadIdx.x < 32) keep_named<DT>(v, seg, read_teacher(a, t), named, lo, hi, piece);
    }
    __syncthreads();
    if (!g.zero) {
      g.scale = w * named.total;
      g.zero = named.total == 0.f;
    }
    if (g.zero) store_zeros<DT, kVecs>(v, seg, first, hi);
    else store_vectors<DT, kVecs, false>(v, seg, g, x, first, hi);
    store_edges<DT>(v, seg, g, t, piece, pieces);
    if (!g.zero) {
      __syncthreads();
      store_named<DT>(v, seg, named, g, w);
    }
  }
}

constexpr int kStepThreads = 512;
constexpr int kStepCluster = 8;

// Loss and gradient in one call: a cluster of CTAs holds a row in registers,
// joins its statistics through distributed shared memory and writes the
// gradient, so that a logit is read once. A row that is longer than the
// cluster's registers (or its CTAs, under a cap) is taken in several tiles and
// read a second time for the gradient.
template <int DT>
__global__ void __launch_bounds__(kStepThreads, 2) distill_step_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ GradSegments seg;
  __shared__ Named named;
  __shared__ LossSlots loss;
  __shared__ JoinSlots slots;
  const VocabArgs& v = a.v;
  const uint32_t ctas = cluster_size(), cta = cluster_rank();
  const uint32_t tile = blockDim.x * kVecs, tiles = max(1u, (v.cut.vectors + tile * ctas - 1) / (tile * ctas));
  const uint32_t lo = min(v.cut.vectors, cta * tile * tiles), hi = min(v.cut.vectors, lo + tile * tiles);
  start(ctas);
  if (threadIdx.x == 0) dev::record_sm(v.sm_mask);
  int phase = 0;
  const float c = v.exp2_scale;
  for (uint64_t t = blockIdx.x / ctas; t < v.rows; t += gridDim.x / ctas) {
    __syncthreads();  // the last row's segments and columns are done with
    set_segments<DT>(v, t, seg);
    __syncthreads();
    Vec<DT> x[kVecs];
    load_vectors<DT, kVecs>(v, seg, x, lo + threadIdx.x, hi);
    if (threadIdx.x < 32) {
      const TeacherRow q = read_teacher(a, t);
      keep_named<DT>(v, seg, q, named, lo, hi, cta);
      if (cta == 0) set_loss<DT>(v, seg, q, loss);
    }
    // the thread's maximum so far, and the sum relative to it
    Part p{kClamp, 0.f, 0.f};
    for (uint32_t i = 0;;) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) x[k].clamp();
      const float top = batch_max<DT, kVecs>(x);
      if (top > p.m) rebase(p, top, c);
      const float r = __fmul_rn(p.m, c);
      f32x2 s[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
#pragma unroll
        for (int j = 0; j < Vec<DT>::kPairs; ++j)
          s[j & 1] = add2(s[j & 1], exp2x2(fma2(x[k].pair(j), pack(c, c), pack(-r, -r))));
      float s0, s1, s2, s3;
      unpack(s[0], s0, s1);
      unpack(s[1], s2, s3);
      p.s += (s0 + s1) + (s2 + s3);
      if (++i == tiles) break;
      load_vectors<DT, kVecs>(v, seg, x, lo + i * tile + threadIdx.x, hi);
    }
    for (uint32_t e = threadIdx.x; cta == 0 && e < v.cut.edges; e += blockDim.x) {
      uint32_t es, ec;
      edge_at<DT>(v, seg, e, es, ec);
      const float y = max_f32(load_one<DT>(seg.at<DT>(es, ec)), kClamp);
      if (y > p.m) rebase(p, y, c);
      p.s += exp2_ftz(__fmaf_rn(y, c, -__fmul_rn(p.m, c)));
    }
    p = row_join(p, c, slots, phase, ctas);
    const bool fast = fabsf(p.m) < -kClamp;
    const Stats st = fast ? stats_of(p, c) : slow_stats<DT>(v, seg, lo, hi, slots, phase, cta, ctas);
    if (cta == 0 && threadIdx.x < 32) store_loss(a, t, loss, st);
    const float w = a.weights[t] * v.inv_temp;
    RowGrad g;
    g.set(v, st.max, 0.f);
    g.log2_s = st.log2_s;
    g.scale = w * named.total;
    g.zero = w == 0.f || named.total == 0.f || st.empty();
    // An in-place gradient may be written from here on: past the join's
    // barrier a CTA reads its own columns only, each before it replaces it.
    for (uint32_t i = 0; i < tiles; ++i) {
      const uint32_t first = lo + i * tile + threadIdx.x;
      if (g.zero) {
        store_zeros<DT, kVecs>(v, seg, first, hi);
        continue;
      }
      // one tile is still in registers, but clamped
      if (tiles > 1 || !fast) load_vectors<DT, kVecs>(v, seg, x, first, hi);
      store_vectors<DT, kVecs, false>(v, seg, g, x, first, hi);
    }
    store_edges<DT>(v, seg, g, t, cta, ctas);
    if (!g.zero) {
      __syncthreads();
      store_named<DT>(v, seg, named, g, w);
    }
  }
}

template <typename Args>
int launch_pieces(void (*kernel)(Args), const Args& a, VocabLaunch& l) {
  const VocabArgs& v = a.v;
  const uint64_t pieces = v.cut.vectors ? (v.cut.vectors + kThreads * kVecs - 1) / (kThreads * kVecs) : 1;
  uint64_t grid = v.rows * pieces;
  const uint64_t most = l.cap > 0 ? static_cast<uint64_t>(l.cap) : static_cast<uint64_t>(1) << 30;
  if (grid > most) grid = most;
  return launch_rows(kernel, a, l, grid, kThreads, 1, 0);
}

template <int DT>
int launch_step_t(DistillArgs& a, VocabLaunch& l) {
  // the smallest cluster whose registers hold a row, then the smallest CTAs
  set_cut<DT>(a.v, kStepThreads, 2);
  const uint32_t n = a.v.cut.vectors;
  int c = 1;
  while (c < kStepCluster && static_cast<uint32_t>(c * kStepThreads * kVecs) < n && (l.cap <= 0 || 2 * c <= l.cap)) c *= 2;
  const uint32_t per = (n + c * kVecs - 1) / (c * kVecs);
  const int threads = per >= kStepThreads ? kStepThreads : per <= 128 ? 128 : static_cast<int>((per + 31) / 32 * 32);
  set_cut<DT>(a.v, threads, 2);
  uint64_t rows = a.v.rows;
  if (l.cap > 0 && rows * c > static_cast<uint64_t>(l.cap)) rows = l.cap / c;
  const uint64_t most = static_cast<uint64_t>(1) << 27;
  return launch_rows(distill_step_kernel<DT>, a, l, (rows < most ? rows : most) * c, threads, c, 0);
}

}  // namespace

int launch_log_probs_grad(int dtype, LogProbsGradArgs& a, VocabLaunch& l) {
  if (dtype == kBF16) {
    set_cut<kBF16>(a.v, kThreads, 2);
    return launch_pieces(a.d_entropy ? log_probs_grad_kernel<kBF16, true> : log_probs_grad_kernel<kBF16, false>, a, l);
  }
  set_cut<kF32>(a.v, kThreads, 2);
  return launch_pieces(a.d_entropy ? log_probs_grad_kernel<kF32, true> : log_probs_grad_kernel<kF32, false>, a, l);
}

int launch_distill(int dtype, DistillArgs& a, VocabLaunch& l) {
  if (!a.weights) return vocab::launch_distill_forward(dtype, a, l);
  return dtype == kBF16 ? launch_step_t<kBF16>(a, l) : launch_step_t<kF32>(a, l);
}

int launch_distill_grad(int dtype, DistillArgs& a, VocabLaunch& l) {
  if (dtype == kBF16) {
    set_cut<kBF16>(a.v, kThreads, 2);
    return launch_pieces(distill_grad_kernel<kBF16>, a, l);
  }
  set_cut<kF32>(a.v, kThreads, 2);
  return launch_pieces(distill_grad_kernel<kF32>, a, l);
}

}  // namespace tccl
