// ef_distill_loss, ef_distill_grad, ef_distill_loss_grad: distillation from
// row packets.
//
// Statistics are relative to a row's largest logits, a for the student and b
// for the packet: exp((x - a) / tau) = 2^((x - a) c), c = log2(e) / tau.  The
// difference is taken before the product, so rows of very large or very low
// logits keep their digits, and log(p / q) is formed from relative
// quantities, never from two log-sum-exps of full size.
#include "ef_rows.cuh"

namespace ef {
namespace {

constexpr int kThreads = 256;

struct DistillArgs {
  const void* logits;
  int64_t stride;
  int vocab, k;
  const float* values;
  const int32_t* indices;
  const int32_t* counts;
  const float* tail;
  const float* stats_in;
  const float* row_grad;
  float c, inv_tau;
  float* loss;
  float* stats;
  void* grad;
  int64_t grad_stride;
};

// LOSS: compute the row's statistics (else read them from stats_in).
template <typename T, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a) {
  __shared__ float red[32];
  __shared__ int32_t idx[EF_MAX_ROW_PACKET];
  __shared__ float sx[EF_MAX_ROW_PACKET];  // student
  __shared__ float tx[EF_MAX_ROW_PACKET];  // teacher
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  T* g = GRAD ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
  const int tid = threadIdx.x, vocab = a.vocab;
  const float c = a.c;
  const float w = GRAD ? (a.row_grad ? a.row_grad[row] : 1.0f) * a.inv_tau : 0.0f;
  if (!LOSS && w == 0.0f) {
    for (int v = tid; v < vocab; v += kThreads) g[v] = from_f32<T>(0.0f);
    return;
  }
  int n = a.counts ? min(max(a.counts[row], 0), a.k) : a.k;
  bool bad = false;
  for (int j = tid; j < n; j += kThreads) {
    const int32_t i = a.indices[row * a.k + j];
    const int32_t before = j > 0 ? a.indices[row * a.k + j - 1] : -1;
    const bool ok = i > before && i >= 0 && i < vocab;
    bad |= !ok;
    idx[j] = i;
    sx[j] = ok ? to_f32(x[i]) : kNegInf;
    tx[j] = sx[j] == kNegInf ? kNegInf : a.values[row * a.k + j];
  }
  if (__syncthreads_or(bad)) {
    const float nan = __int_as_float(0x7FFFFFFF);
    if (LOSS && tid == 0) {
      a.loss[row] = nan;
      if (a.stats)
        for (int q = 0; q < 6; ++q) a.stats[row * 6 + q] = nan;
    }
    if (GRAD)
      for (int v = tid; v < vocab; v += kThreads) g[v] = from_f32<T>(w == 0.0f ? 0.0f : nan);
    return;
  }
  auto in_packet = [&](int v) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (idx[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    return lo < n && idx[lo] == v ? lo : -1;
  };

  // the largest logits (0 where there are none), the log-sum-exps relative to
  // them, and the two masses outside the packet
  float top, top_t, l_off, l_all, l_t, p_off, q_off;
  if (LOSS) {
    float m = kNegInf, ms = kNegInf, mt = kNegInf;
    for (int v = tid; v < vocab; v += kThreads)
      if (in_packet(v) < 0) m = fmaxf(m, to_f32(x[v]));
    for (int j = tid; j < n; j += kThreads) {
      ms = fmaxf(ms, sx[j]);
      mt = fmaxf(mt, tx[j]);
    }
    const float m_off = block_max(m, red);
    top = finite_ref(fmaxf(block_max(ms, red), m_off));
    mt = block_max(mt, red);
    top_t = finite_ref(mt);
    float s = 0.0f;
    const float ref = finite_ref(m_off);
    for (int v = tid; v < vocab; v += kThreads)
      if (in_packet(v) < 0) s += exp2_fast((to_f32(x[v]) - ref) * c);
    s = block_sum(s, red);
    const bool has_off = s != 0.0f;
    l_off = has_off ? fmaf(ref - top, a.inv_tau, logf(s)) : kNegInf;
    const float tail = a.tail && has_off ? fmaf(-top_t, a.inv_tau, a.tail[row]) : kNegInf;
    // reference of the teacher's sum: its largest term
    const float rt = finite_ref(fmaxf(mt == kNegInf ? kNegInf : 0.0f, tail));
    float es = 0.0f, et = 0.0f;
    for (int j = tid; j < n; j += kThreads) {
      es += exp2f((sx[j] - top) * c);
      et += expf(fmaf(tx[j] - top_t, a.inv_tau, -rt));
    }
    const float sum_s = block_sum(es, red) + expf(l_off);
    const float sum_t = block_sum(et, red) + expf(tail - rt);
    l_all = sum_s != 0.0f ? logf(sum_s) : kNegInf;
    l_t = sum_t != 0.0f ? rt + logf(sum_t) : kNegInf;
    p_off = exp_diff(tail, l_t);
    q_off = exp_diff(l_off, l_all);
    const float gap = l_t - l_all;
    float acc = 0.0f;
    for (int j = tid; j < n; j += kThreads) {
      const float y = tx[j] - top_t, p = exp_diff(y * a.inv_tau, l_t);
      if (p != 0.0f) acc += p * fmaf(y - (sx[j] - top), a.inv_tau, -gap);
    }
    acc = block_sum(acc, red);
    if (p_off != 0.0f) acc += p_off * ((tail - l_off) - gap);
    if (tid == 0) {
      a.loss[row] = l_t == kNegInf ? 0.0f : acc;
      if (a.stats) {
        float* o = a.stats + row * 6;
        o[0] = top;
        o[1] = l_off;
        o[2] = l_all;
        o[3] = top_t;
        o[4] = l_t;
        o[5] = p_off;
      }
    }
  } else {
    const float* o = a.stats_in + row * 6;
    top = o[0];
    l_off = o[1];
    l_all = o[2];
    top_t = o[3];
    l_t = o[4];
    p_off = o[5];
    q_off = exp_diff(l_off, l_all);
  }
  if (!GRAD) return;
  __syncthreads();
  const bool dead = w == 0.0f || l_t == kNegInf;
  // a NaN in either log-sum-exp shows in every entry
  const float poison = 0.0f * (l_t + l_all);
  const float coef = w * (q_off - p_off) + poison;
  for (int v = tid; v < vocab; v += kThreads) {
    const float s = to_f32(x[v]);
    float d = 0.0f;
    if (!dead && s != kNegInf) {
      const int j = in_packet(v);
      d = j >= 0 ? w * (exp_diff((s - top) * a.inv_tau, l_all) -
                        exp_diff((tx[j] - top_t) * a.inv_tau, l_t)) + poison
                 : coef * exp_diff((s - top) * a.inv_tau, l_off);
    }
    g[v] = from_f32<T>(d);
  }
}

ef_status check_packets(const void* logits, int size, int64_t rows, int64_t vocab, int32_t k,
                        const float* values, const int32_t* indices, const int32_t* counts) {
  if ((!logits && vocab > 0) || (k > 0 && (!values || !indices))) return EF_ERR_NULL;
  if (!aligned_to(logits, size) || !aligned4(values) || !aligned4(indices) || !aligned4(counts))
    return EF_ERR_ALIGN;
  (void)rows;
  return EF_OK;
}

ef_status check_grad(const void* logits, int size, int64_t rows, int64_t vocab, int64_t stride,
                     const void* grad, int64_t grad_stride) {
  if (grad_stride < vocab || grad_stride > (1ll << 40)) return EF_ERR_SIZE;
  if (!grad && vocab > 0) return EF_ERR_NULL;
  if (!aligned_to(grad, size)) return EF_ERR_ALIGN;
  if (grad == logits && grad_stride == stride) return EF_OK;
  if (overlaps(grad, rows_bytes(rows, vocab, grad_stride, size), logits,
               rows_bytes(rows, vocab, stride, size)))
    return EF_ERR_ALIAS;
  return EF_OK;
}

template <bool LOSS, bool GRAD>
ef_status launch(int32_t dtype, int64_t rows, float tau, DistillArgs a, void* stream) {
  DeviceInfo dev;
  const ef_status st = current_device(&dev);
  if (st != EF_OK) return st;
  a.c = (float)(1.4426950408889634074 / (double)tau);
  a.inv_tau = 1.0f / tau;
  with_dtype(dtype, [&](auto t) {
    launch_pdl(distill_kernel<decltype(t), LOSS, GRAD>, dim3((unsigned)rows), dim3(kThreads), 0,
               static_cast<cudaStream_t>(stream), a);
  });
  return check_launch();
}

}  // namespace
}  // namespace ef

extern "C" {

ef_status ef_distill_loss(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                          int64_t row_stride, int32_t k, const float* values,
                          const int32_t* indices, const int32_t* counts, const float* tail,
                          float tau, float* out_loss, float* out_stats, void* stream) {
  using namespace ef;
  ef_status st = check_rows(dtype, rows, vocab, row_stride, k, tau);
  if (st != EF_OK) return st;
  if (rows == 0) return EF_OK;
  const int size = dtype_size(dtype);
  st = check_packets(logits, size, rows, vocab, k, values, indices, counts);
  if (st != EF_OK) return st;
  if (!out_loss) return EF_ERR_NULL;
  if (!aligned4(tail) || !aligned4(out_loss) || !aligned4(out_stats)) return EF_ERR_ALIGN;
  const size_t r = (size_t)rows;
  const Span spans[] = {{logits, rows_bytes(rows, vocab, row_stride, size), false},
                        {values, r * k * 4, false}, {indices, r * k * 4, false},
                        {counts, r * 4, false}, {tail, r * 4, false},
                        {out_loss, r * 4, true}, {out_stats, r * 24, true}};
  if (any_overlap(spans, 7)) return EF_ERR_ALIAS;
  DistillArgs a = {};
  a.logits = logits, a.stride = row_stride, a.vocab = (int)vocab, a.k = k;
  a.values = values, a.indices = indices, a.counts = counts, a.tail = tail;
  a.loss = out_loss, a.stats = out_stats;
  return launch<true, false>(dtype, rows, tau, a, stream);
}

ef_status ef_distill_grad(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                          int64_t row_stride, int32_t k, const float* values,
                          const int32_t* indices, const int32_t* counts, float tau,
                          const float* stats, const float* row_grad, void* grad,
                          int64_t grad_stride, void* stream) {
  using namespace ef;
  ef_status st = check_rows(dtype, rows, vocab, row_stride, k, tau);
  if (st != EF_OK) return st;
  if (rows == 0) return EF_OK;
  const int size = dtype_size(dtype);
  st = check_packets(logits, size, rows, vocab, k, values, indices, counts);
  if (st != EF_OK) return st;
  if (!stats) return EF_ERR_NULL;
  if (!aligned4(stats) || !aligned4(row_grad)) return EF_ERR_ALIGN;
  st = check_grad(logits, size, rows, vocab, row_stride, grad, grad_stride);
  if (st != EF_OK) return st;
  const size_t r = (size_t)rows;
  const Span spans[] = {{grad, rows_bytes(rows, vocab, grad_stride, size), true},
                        {values, r * k * 4, false}, {indices, r * k * 4, false},
                        {counts, r * 4, false}, {stats, r * 24, false}, {row_grad, r * 4, false}};
  if (any_overlap(spans, 6)) return EF_ERR_ALIAS;
  DistillArgs a = {};
  a.logits = logits, a.stride = row_stride, a.vocab = (int)vocab, a.k = k;
  a.values = values, a.indices = indices, a.counts = counts, a.stats_in = stats;
  a.row_grad = row_grad, a.grad = grad, a.grad_stride = grad_stride;
  return launch<false, true>(dtype, rows, tau, a, stream);
}

ef_status ef_distill_loss_grad(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, int32_t k, const float* values,
                               const int32_t* indices, const int32_t* counts, const float* tail,
                               float tau, const float* row_grad, float* out_loss, void* grad,
                               int64_t grad_stride, void* stream) {
  using namespace ef;
  ef_status st = check_rows(dtype, rows, vocab, row_stride, k, tau);
  if (st != EF_OK) return st;
  if (rows == 0) return EF_OK;
  const int size = dtype_size(dtype);
  st = check_packets(logits, size, rows, vocab, k, values, indices, counts);
  if (st != EF_OK) return st;
  if (!out_loss) return EF_ERR_NULL;
  if (!aligned4(tail) || !aligned4(out_loss) || !aligned4(row_grad)) return EF_ERR_ALIGN;
  st = check_grad(logits, size, rows, vocab, row_stride, grad, grad_stride);
  if (st != EF_OK) return st;
  const size_t r = (size_t)rows;
  const Span spans[] = {{grad, rows_bytes(rows, vocab, grad_stride, size), true},
                        {out_loss, r * 4, true}, {values, r * k * 4, false},
                        {indices, r * k * 4, false}, {counts, r * 4, false},
                        {tail, r * 4, false}, {row_grad, r * 4, false}};
  const Span in_loss[] = {{logits, rows_bytes(rows, vocab, row_stride, size), false},
                          {out_loss, r * 4, true}};
  if (any_overlap(spans, 7) || any_overlap(in_loss, 2)) return EF_ERR_ALIAS;
  DistillArgs a = {};
  a.logits = logits, a.stride = row_stride, a.vocab = (int)vocab, a.k = k;
  a.values = values, a.indices = indices, a.counts = counts, a.tail = tail;
  a.row_grad = row_grad, a.loss = out_loss, a.grad = grad, a.grad_stride = grad_stride;
  return launch<true, true>(dtype, rows, tau, a, stream);
}

}  // extern "C"
