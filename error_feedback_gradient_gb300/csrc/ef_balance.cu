// ef_balance_loss, ef_balance_grad, ef_balance_loss_grad: a router's balance
// loss, its per-expert counts and its gradient.
//
// One CTA per segment: it counts the ids, then a warp takes a token at a
// time, each lane a fixed set of experts.
#include "ef_rows.cuh"

namespace ef {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegBatch = 256;  // segments per launch
constexpr int kPerLane = EF_MAX_EXPERTS / 32;

struct SegBatch {
  int64_t off[kSegBatch + 1];
};

struct BalanceArgs {
  const void* logits;
  int64_t stride;
  int experts, k;
  const int32_t* ids;
  const uint8_t* mask;
  float alpha, beta;
  WsHeader* ws;
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  const int32_t* counts_in;
  const int32_t* tokens_in;
  const float* seg_grad;
  void* grad;
  int64_t grad_stride;
};

template <typename T, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kThreads) balance_kernel(BalanceArgs a, SegBatch seg, int first) {
  __shared__ int32_t cnt[EF_MAX_EXPERTS];
  __shared__ float f[EF_MAX_EXPERTS];
  __shared__ float part[EF_MAX_EXPERTS];
  __shared__ float red[32];
  __shared__ int32_t n_tok;
  pdl_wait();
  const int s = first + (int)blockIdx.x, E = a.experts, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = seg.off[blockIdx.x], t1 = seg.off[blockIdx.x + 1];
  if (tid == 0) n_tok = 0;
  for (int e = tid; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  if (LOSS) {
    int n = 0;
    for (int64_t t = t0 + tid; t < t1; t += kThreads) n += !a.mask || a.mask[t] ? 1 : 0;
    atomicAdd(&n_tok, n);
    for (int64_t i = t0 * a.k + tid; i < t1 * a.k; i += kThreads) {
      const int32_t e = a.ids[i];
      if (e >= 0 && e < E && (!a.mask || a.mask[i / a.k])) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
  } else {
    for (int e = tid; e < E; e += kThreads) cnt[e] = a.counts_in[(int64_t)s * E + e];
    if (tid == 0) n_tok = a.tokens_in[s];
    __syncthreads();
  }
  const float inv_n = n_tok > 0 ? 1.0f / (float)n_tok : 0.0f;
  const float scale = (float)E / (float)a.k * inv_n;
  for (int e = tid; e < E; e += kThreads) {
    f[e] = (float)cnt[e] * scale;
    part[e] = 0.0f;
  }
  __syncthreads();
  const float w = GRAD ? (a.seg_grad ? a.seg_grad[s] : 1.0f) * inv_n : 0.0f;
  float acc[kPerLane] = {};
  float z2 = 0.0f;
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    const T* z = static_cast<const T*>(a.logits) + t * a.stride;
    T* g = GRAD ? static_cast<T*>(a.grad) + t * a.grad_stride : nullptr;
    if (a.mask && !a.mask[t]) {
      if (GRAD)
        for (int e = lane; e < E; e += 32) g[e] = from_f32<T>(0.0f);
      continue;
    }
    float p[kPerLane];
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      p[i] = e < E ? to_f32(z[e]) : kNegInf;
      m = fmaxf(m, p[i]);
    }
    m = finite_ref(warp_max(m));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) sum += p[i] = exp2f((p[i] - m) * 1.4426950408889634f);
    sum = warp_sum(sum);
    const bool none = sum == 0.0f;
    const float inv = none ? 0.0f : 1.0f / sum;
    const float lse = none ? 0.0f : fmaf(log2f(sum), kLn2, m);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      p[i] *= inv;
      acc[i] += p[i];
      dot += e < E ? p[i] * f[e] : 0.0f;
    }
    z2 += lse * lse;
    if (GRAD) {
      dot = warp_sum(dot);
      const float base = 2.0f * a.beta * lse;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const int e = lane + 32 * i;
        if (e < E) g[e] = from_f32<T>(w * p[i] * (a.alpha * (f[e] - dot) + base));
      }
    }
  }
  if (!LOSS) return;
  if (s == 0 && tid == 0) a.ws->status = EF_OK;
  for (int q = 0; q < kWarps; ++q) {  // the warps in order
    if (warp == q)
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (lane + 32 * i < E) part[lane + 32 * i] += acc[i];
    __syncthreads();
  }
  float b = 0.0f;
  for (int e = tid; e < E; e += kThreads) b += f[e] * part[e];
  b = block_sum(b, red);
  z2 = block_sum(lane == 0 ? z2 : 0.0f, red);
  for (int e = tid; e < E; e += kThreads) a.counts[(int64_t)s * E + e] = cnt[e];
  if (tid == 0) {
    a.tokens[s] = n_tok;
    a.loss[s] = n_tok > 0 ? (a.alpha * b + (a.beta != 0.0f ? a.beta * z2 : 0.0f)) * inv_n : 0.0f;
  }
}

ef_status check_common(int32_t dtype, int64_t tokens, int32_t experts, int64_t stride, int32_t k,
                       int32_t nseg, const int64_t* off, float alpha, float beta) {
  if (dtype_size(dtype) == 0) return EF_ERR_ARG;
  if (tokens < 0 || tokens >= (1ll << 31) || experts < 1 || experts > EF_MAX_EXPERTS ||
      stride < experts || stride > (1ll << 40))
    return EF_ERR_SIZE;
  if (k < 1 || k > EF_MAX_EXPERTS) return EF_ERR_K;
  if (nseg < 1) return EF_ERR_SEGMENTS;
  if (!off) return EF_ERR_NULL;
  if (off[0] != 0 || off[nseg] != tokens) return EF_ERR_SEGMENTS;
  for (int32_t s = 0; s < nseg; ++s)
    if (off[s] > off[s + 1]) return EF_ERR_SEGMENTS;
  if (!std::isfinite(alpha) || !std::isfinite(beta)) return EF_ERR_ARG;
  return EF_OK;
}

// The buffers of a call; those it does not use are NULL in `a`.
ef_status check_buffers(const BalanceArgs& a, int size, int64_t tokens, int32_t nseg, bool loss,
                        bool grad, const void* ws, size_t ws_bytes, size_t need) {
  if (tokens > 0 && (!a.logits || (loss && !a.ids) || (grad && !a.grad))) return EF_ERR_NULL;
  if (loss && (!a.loss || !a.counts || !a.tokens)) return EF_ERR_NULL;
  if (!loss && (!a.counts_in || !a.tokens_in)) return EF_ERR_NULL;
  if (!aligned_to(a.logits, size) || !aligned_to(a.grad, size) || !aligned4(a.ids) ||
      !aligned4(a.loss) || !aligned4(a.counts) || !aligned4(a.tokens) || !aligned4(a.counts_in) ||
      !aligned4(a.tokens_in) || !aligned4(a.seg_grad))
    return EF_ERR_ALIGN;
  if (grad && (a.grad_stride < a.experts || a.grad_stride > (1ll << 40))) return EF_ERR_SIZE;
  if (loss && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need))
    return EF_ERR_WORKSPACE;
  const size_t table = (size_t)nseg * a.experts * 4, seg = (size_t)nseg * 4, t = (size_t)tokens;
  const bool in_place = a.grad == a.logits && a.grad_stride == a.stride;
  const Span spans[] = {
      {in_place ? nullptr : a.logits, rows_bytes(tokens, a.experts, a.stride, size), false},
      {a.grad, rows_bytes(tokens, a.experts, a.grad_stride, size), true},
      {a.ids, t * a.k * 4, false}, {a.mask, t, false}, {a.seg_grad, seg, false},
      {a.counts_in, table, false}, {a.tokens_in, seg, false}, {a.counts, table, true},
      {a.tokens, seg, true}, {a.loss, seg, true}, {loss ? ws : nullptr, need, true}};
  return any_overlap(spans, 11) ? EF_ERR_ALIAS : EF_OK;
}

size_t workspace_bytes_for() { return sizeof(WsHeader); }

template <bool LOSS, bool GRAD>
ef_status launch(int32_t dtype, const BalanceArgs& a, int32_t nseg, const int64_t* off,
                 void* stream) {
  DeviceInfo dev;
  ef_status st = current_device(&dev);
  if (st != EF_OK) return st;
  for (int32_t first = 0; first < nseg; first += kSegBatch) {
    const int n = nseg - first < kSegBatch ? nseg - first : kSegBatch;
    SegBatch b;
    for (int i = 0; i <= n; ++i) b.off[i] = off[first + i];
    with_dtype(dtype, [&](auto t) {
      launch_pdl(balance_kernel<decltype(t), LOSS, GRAD>, dim3((unsigned)n), dim3(kThreads), 0,
                 static_cast<cudaStream_t>(stream), a, b, (int)first);
    });
    st = check_launch();
    if (st != EF_OK) return st;
  }
  return EF_OK;
}

}  // namespace
}  // namespace ef

extern "C" {

ef_status ef_balance_workspace_size(int64_t tokens, int32_t experts, int32_t k, int32_t nseg,
                                    const int64_t* h_seg_offsets, size_t* bytes) {
  if (!bytes) return EF_ERR_NULL;
  const ef_status st = ef::check_common(EF_DTYPE_F32, tokens, experts, experts, k, nseg,
                                        h_seg_offsets, 0.0f, 0.0f);
  if (st != EF_OK) return st;
  *bytes = ef::workspace_bytes_for();
  return EF_OK;
}

ef_status ef_balance_loss(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                          int64_t row_stride, const int32_t* ids, int32_t k, const uint8_t* mask,
                          int32_t nseg, const int64_t* h_seg_offsets, float alpha, float beta,
                          float* out_loss, int32_t* out_counts, int32_t* out_tokens,
                          void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ef;
  ef_status st = check_common(dtype, tokens, experts, row_stride, k, nseg, h_seg_offsets, alpha,
                              beta);
  if (st != EF_OK) return st;
  BalanceArgs a = {};
  a.logits = logits, a.stride = row_stride, a.experts = experts, a.k = k, a.ids = ids;
  a.mask = mask, a.alpha = alpha, a.beta = beta;
  a.loss = out_loss, a.counts = out_counts, a.tokens = out_tokens;
  a.ws = static_cast<WsHeader*>(workspace);
  st = check_buffers(a, dtype_size(dtype), tokens, nseg, true, false, workspace, workspace_bytes,
                     workspace_bytes_for());
  if (st != EF_OK) return st;
  return launch<true, false>(dtype, a, nseg, h_seg_offsets, stream);
}

ef_status ef_balance_grad(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                          int64_t row_stride, int32_t k, const uint8_t* mask, int32_t nseg,
                          const int64_t* h_seg_offsets, float alpha, float beta,
                          const int32_t* counts, const int32_t* token_counts,
                          const float* seg_grad, void* grad, int64_t grad_stride, void* stream) {
  using namespace ef;
  ef_status st = check_common(dtype, tokens, experts, row_stride, k, nseg, h_seg_offsets, alpha,
                              beta);
  if (st != EF_OK) return st;
  BalanceArgs a = {};
  a.logits = logits, a.stride = row_stride, a.experts = experts, a.k = k;
  a.mask = mask, a.alpha = alpha, a.beta = beta;
  a.counts_in = counts, a.tokens_in = token_counts, a.seg_grad = seg_grad;
  a.grad = grad, a.grad_stride = grad_stride;
  st = check_buffers(a, dtype_size(dtype), tokens, nseg, false, true, nullptr, 0, 0);
  if (st != EF_OK) return st;
  return launch<false, true>(dtype, a, nseg, h_seg_offsets, stream);
}

ef_status ef_balance_loss_grad(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                               int64_t row_stride, const int32_t* ids, int32_t k,
                               const uint8_t* mask, int32_t nseg, const int64_t* h_seg_offsets,
                               float alpha, float beta, const float* seg_grad, float* out_loss,
                               int32_t* out_counts, int32_t* out_tokens, void* grad,
                               int64_t grad_stride, void* workspace, size_t workspace_bytes,
                               void* stream) {
  using namespace ef;
  ef_status st = check_common(dtype, tokens, experts, row_stride, k, nseg, h_seg_offsets, alpha,
                              beta);
  if (st != EF_OK) return st;
  BalanceArgs a = {};
  a.logits = logits, a.stride = row_stride, a.experts = experts, a.k = k, a.ids = ids;
  a.mask = mask, a.alpha = alpha, a.beta = beta, a.seg_grad = seg_grad;
  a.loss = out_loss, a.counts = out_counts, a.tokens = out_tokens;
  a.ws = static_cast<WsHeader*>(workspace);
  a.grad = grad, a.grad_stride = grad_stride;
  st = check_buffers(a, dtype_size(dtype), tokens, nseg, true, true, workspace, workspace_bytes,
                     workspace_bytes_for());
  if (st != EF_OK) return st;
  return launch<true, true>(dtype, a, nseg, h_seg_offsets, stream);
}

}  // extern "C"
