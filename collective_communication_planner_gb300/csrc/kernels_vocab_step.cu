// Distillation with its gradient in one call.
#include "vocab_grad.cuh"

namespace tccl {
namespace {

using namespace vocab;

constexpr int kWarps = 8;  // that stream, at the most; one more reads the teacher's entries
constexpr int kThreads = (kWarps + 1) * 32;
constexpr uint64_t kKeepBytes = 52ull << 20;  // rows that L2 keeps between two reads
constexpr int kStepCluster = 8;
constexpr int kStepCtasPerSm = 4;

// Loss and gradient in one call: a cluster of CTAs sums up a row, joins its
// statistics through distributed shared memory and reads it again, from L2,
// for the gradient. Short and few rows, and rows of many odd segments; long ones
// take the ring. What bounds it is latency: a row is read, joined and read again,
// and only other rows fill the gaps. 4096 x 16384 bf16 55 us against 40 of memory
// traffic that cannot be saved; 4 x 131072 7.4 us.
template <int DT>
__global__ void __launch_bounds__(kThreads, kStepCtasPerSm) distill_step_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ GradSegments seg;
  __shared__ Entries named;
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
    const float w = a.weights[t] * v.inv_temp;
    if (threadIdx.x >= v.step.warps * 32) {
      const TeacherRow q = read_teacher(a, t);
      uint32_t x[kMaxTop / 32];
      load_named<DT>(v, t, q, x);
      set_entries<DT>(q, x, a.top_k, named, [&](uint32_t column) {
        return has_column<DT>(v, t, column, lo, hi, cta == 0);
      });
    }
    Part p = scan_row<DT, false, true>(v, seg, lo, hi, cta == 0, KeepLoad(), [](float, const Vec<DT>(&)[kBatch]) {});
    p = row_join(p, c, slots, phase, v.step.warps, ctas);
    const Stats st = joined_stats<DT>(p, v, seg, lo, hi, slots, phase, cta, ctas);
    if (cta == 0 && threadIdx.x >= v.step.warps * 32) store_loss(a, t, named, st);
    RowGrad g;
    g.set(v, st.max, st.log2_s, w * named.total, 0.f);
    g.zero = w == 0.f || named.total == 0.f || st.empty();
    // An in-place gradient may be written from here on: past the join's
    // barrier a CTA reads its own columns only, each before it replaces it.
    if (g.zero) zero_chunks<DT>(v, seg, first_chunk(v, lo, hi), hi, v.step);
    else store_chunks<DT, false>(v, seg, g, lo, hi);
    store_edges<DT>(v, seg, g, t, cta, ctas);
    if (!g.zero) {
      __syncthreads();
      for (int i = threadIdx.x; i < named.count; i += blockDim.x) store_named<DT>(v, t, named, g, w, i);
    }
  }
}

template <int DT>
int launch_step_t(DistillArgs& a, VocabLaunch& l) {
  VocabArgs& v = a.v;
  set_cut<DT>(v, v.together ? 0 : 2);
  // CTAs of a row: few enough rows at once for L2 to keep them between the two
  // reads, or as many as the SMs take of few rows; every warp gets a chunk.
  // GB300: 4096 x 131039 bf16 over 16 ranks with one CTA a row 461 us, rows within
  // 104 / 52 / 26 MB (2, 4 and 8 CTAs) 446 / 443 / 597; 128 x 131072 with 1 / 4 / 8
  // 20.1 / 15.2 / 20.2; 64 rows with 1 / 8 19.1 / 10.9.
  const uint64_t row_bytes = static_cast<uint64_t>(v.vocab) * Elem<DT>::kBytes;
  const uint64_t resident = static_cast<uint64_t>(l.sm_count) * kStepCtasPerSm;
  const auto kept = [&](int c) { return (v.rows < resident / c ? v.rows : resident / c) * row_bytes; };
  int c = 1;
  while (c < kStepCluster && v.cut.chunks >= static_cast<uint32_t>(2 * c * kWarps) &&
         (l.cap <= 0 || 2 * c <= l.cap) && (v.rows * 2 * c <= resident || kept(c) > kKeepBytes))
    c *= 2;
  // Many short rows: fewer warps, so that more rows are in flight. 4096 rows bf16,
  // so / with eight: 1000 columns 15.2 / 35.9 us, 4096 27.1 / 41.1, 16384 55.0 / 62.2.
  int warps = kWarps;
  const bool many = v.rows >= static_cast<uint64_t>(l.sm_count) * 4;
  while (warps > 1 && many && v.cut.chunks <= static_cast<uint32_t>(warps) * 2) warps /= 2;
  uint64_t rows = v.rows;
  if (l.cap > 0 && rows * c > static_cast<uint64_t>(l.cap)) rows = l.cap / c;
  const uint64_t most = static_cast<uint64_t>(1) << 27;
  return launch_rows(distill_step_kernel<DT>, a, l, (rows < most ? rows : most) * c, (warps + 1) * 32, c, 0,
                     warps);
}

}  // namespace

namespace vocab {
int launch_distill_step(int dtype, DistillArgs& a, VocabLaunch& l) {
  if (plan_distill_ring(dtype, a, l)) return launch_distill_ring(dtype, a, l);
  return dtype == kBF16 ? launch_step_t<kBF16>(a, l) : launch_step_t<kF32>(a, l);
}
}  // namespace vocab

}  // namespace tccl
