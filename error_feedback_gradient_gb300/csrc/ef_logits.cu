// ef_logits_topk: the k largest logits of every row as a packet, and the
// log-sum-exp of the rest.
//
// One CTA per row.  The k-th largest key is found bit by bit (32 counting
// passes over the row), ties are cut at a position found the same way, and
// the row is then emitted in order.
#include "ef_rows.cuh"

namespace ef {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_topk_kernel(
    const T* __restrict__ logits, int vocab, int64_t stride, int k, float c, float inv_tau,
    float* __restrict__ out_values, int32_t* __restrict__ out_indices,
    int32_t* __restrict__ out_counts, float* __restrict__ out_tail) {
  __shared__ uint32_t scan[33];
  __shared__ float red[32];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T* x = logits + row * stride;
  const int tid = threadIdx.x;

  // count of keys >= T among live entries
  auto count = [&](auto pred) {
    uint32_t n = 0;
    for (int v = tid; v < vocab; v += kThreads) n += pred(order_key(to_f32(x[v])), v) ? 1u : 0u;
    uint32_t total;
    block_excl_scan(n, scan, &total);
    return total;
  };
  const uint32_t live = count([](uint32_t key, int) { return key > kKeyNegInf; });
  const uint32_t want = min((uint32_t)k, live);
  // the want-th largest key (everything is > key when want = 0)
  uint32_t cut = 0xFFFFFFFFu;
  int last = -1;  // ties at `cut` are taken up to this position
  if (want > 0) {
    cut = 0;
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = cut | (1u << b);
      if (count([t](uint32_t key, int) { return key >= t; }) >= want) cut = t;
    }
    const uint32_t need = want - count([cut](uint32_t key, int) { return key > cut; });
    int lo = 0, hi = vocab - 1;  // smallest position with `need` ties up to it
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (count([=](uint32_t key, int v) { return key == cut && v <= mid; }) >= need) hi = mid;
      else lo = mid + 1;
    }
    last = lo;
  }
  auto taken = [&](uint32_t key, int v) {
    return want > 0 && (key > cut || (key == cut && v <= last));
  };

  // packet, in order
  uint32_t base = 0;
  if (want > 0) {
    for (int v0 = 0; v0 < vocab; v0 += kThreads) {
      const int v = v0 + tid;
      const float f = v < vocab ? to_f32(x[v]) : 0.0f;
      const bool take = v < vocab && taken(order_key(f), v);
      uint32_t total;
      const uint32_t pos = base + block_excl_scan(take ? 1u : 0u, scan, &total);
      if (take) {
        out_values[row * k + pos] = f;
        out_indices[row * k + pos] = v;
      }
      base += total;
    }
  }
  for (int j = (int)want + tid; j < k; j += kThreads) {
    out_values[row * k + j] = 0.0f;
    out_indices[row * k + j] = -1;
  }
  if (tid == 0) out_counts[row] = (int32_t)want;
  if (out_tail == nullptr) return;

  float m = kNegInf;
  for (int v = tid; v < vocab; v += kThreads) {
    const float f = to_f32(x[v]);
    if (!taken(order_key(f), v)) m = fmaxf(m, f);
  }
  m = finite_ref(block_max(m, red));
  float s = 0.0f;
  for (int v = tid; v < vocab; v += kThreads) {
    const float f = to_f32(x[v]);
    if (!taken(order_key(f), v)) s += exp2_fast((f - m) * c);
  }
  s = block_sum(s, red);
  if (tid == 0) out_tail[row] = s == 0.0f ? kNegInf : fmaf(m, inv_tau, log2f(s) * kLn2);
}

}  // namespace
}  // namespace ef

extern "C" {

ef_status ef_logits_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, int32_t k, float tau, float* out_values,
                         int32_t* out_indices, int32_t* out_counts, float* out_tail,
                         void* stream) {
  using namespace ef;
  ef_status st = check_rows(dtype, rows, vocab, row_stride, k, tau);
  if (st != EF_OK) return st;
  if (rows == 0) return EF_OK;
  const int size = dtype_size(dtype);
  if ((!logits && vocab > 0) || !out_counts || (k > 0 && (!out_values || !out_indices)))
    return EF_ERR_NULL;
  if (!aligned_to(logits, size) || !aligned4(out_values) || !aligned4(out_indices) ||
      !aligned4(out_counts) || !aligned4(out_tail))
    return EF_ERR_ALIGN;
  const Span spans[] = {{logits, rows_bytes(rows, vocab, row_stride, size), false},
                        {out_values, (size_t)rows * k * 4, true},
                        {out_indices, (size_t)rows * k * 4, true},
                        {out_counts, (size_t)rows * 4, true},
                        {out_tail, (size_t)rows * 4, true}};
  if (any_overlap(spans, 5)) return EF_ERR_ALIAS;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != EF_OK) return st;
  const float c = (float)(1.4426950408889634074 / (double)tau);
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    launch_pdl(logits_topk_kernel<T>, dim3((unsigned)rows), dim3(kThreads), 0,
               static_cast<cudaStream_t>(stream), static_cast<const T*>(logits), (int)vocab,
               row_stride, (int)k, c, 1.0f / tau, out_values, out_indices, out_counts, out_tail);
  });
  return check_launch();
}

}  // extern "C"
