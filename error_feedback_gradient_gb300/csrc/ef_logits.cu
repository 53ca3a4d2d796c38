// ef_logits_topk: the k largest logits of every row as a packet, and the
// log-sum-exp of the rest, in one pass over the logits.
//
// A bound first: cut a row into groups; the k-th largest of the groups'
// maxima is at most the k-th largest element (k groups hold one at least that
// large each).  With G groups and the largest elements spread over them, about
// -G ln(1 - k / G) elements reach that bound: little more than k where k is
// well below G.  Those are the candidates; the packet is picked from them, and
// everything below the bound goes into the sum at once.
#include "ef_rows.cuh"

namespace ef {
namespace {

// Maxima that keep a NaN, so that the element is found among the candidates.
template <typename T>
struct NanMax;
template <>
struct NanMax<float> {
  using P = float;
  static __device__ __forceinline__ P none() { return kNegInf; }
  static __device__ __forceinline__ P of(P a, P b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  static __device__ __forceinline__ P slot(const uint4& r) {
    return of(of(__uint_as_float(r.x), __uint_as_float(r.y)),
              of(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  static __device__ __forceinline__ float value(P a) { return a; }
  static __device__ __forceinline__ bool reaches(P a, float t) { return !(a < t); }
};
template <typename P2, typename E>
struct NanMax16 {
  using P = P2;
  static __device__ __forceinline__ P of(P a, P b) { return __hmax2_nan(a, b); }
  static __device__ __forceinline__ P slot(const uint4& r) {
    return of(of(reinterpret_cast<const P&>(r.x), reinterpret_cast<const P&>(r.y)),
              of(reinterpret_cast<const P&>(r.z), reinterpret_cast<const P&>(r.w)));
  }
  static __device__ __forceinline__ float value(P a) {
    return NanMax<float>::of(to_f32(a.x), to_f32(a.y));
  }
  static __device__ __forceinline__ bool reaches(P a, float t) { return !(value(a) < t); }
};
template <>
struct NanMax<__nv_bfloat16> : NanMax16<__nv_bfloat162, __nv_bfloat16> {
  static __device__ __forceinline__ P none() { return __float2bfloat162_rn(kNegInf); }
};
template <>
struct NanMax<__half> : NanMax16<__half2, __half> {
  static __device__ __forceinline__ P none() { return __float2half2_rn(kNegInf); }
};

// The value of a key (a NaN key gives a NaN).
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct TopkArgs {
  const void* logits;
  int64_t stride;
  int vocab, k;
  float c, inv_tau;
  float* values;
  int32_t* indices;
  int32_t* counts;
  float* tail;
};

// ---------------------------------------------------------------------------
// Any row, by the whole CTA: the k-th largest key is found bit by bit, ties
// are cut at a position found the same way, and the row is emitted in order.
// Some sixty passes over the row; taken where more elements reach the bound
// than the candidates' list holds (a row of equal logits, for one).
// ---------------------------------------------------------------------------

template <typename T>
__device__ __noinline__ void plain_row(const TopkArgs& a, int64_t row, uint32_t* scan,
                                       float* red) {
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  const int tid = threadIdx.x, threads = blockDim.x, vocab = a.vocab, k = a.k;
  auto count = [&](auto pred) {
    uint32_t n = 0;
    for (int v = tid; v < vocab; v += threads) n += pred(order_key(to_f32(x[v])), v) ? 1u : 0u;
    uint32_t total;
    block_excl_scan(n, scan, &total);
    return total;
  };
  const uint32_t live = count([](uint32_t key, int) { return key > kKeyNegInf; });
  const uint32_t want = min((uint32_t)k, live);
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
  uint32_t base = 0;
  for (int v0 = 0; v0 < vocab && want > 0; v0 += threads) {
    const int v = v0 + tid;
    const float f = v < vocab ? to_f32(x[v]) : 0.0f;
    const bool take = v < vocab && taken(order_key(f), v);
    uint32_t total;
    const uint32_t pos = base + block_excl_scan(take ? 1u : 0u, scan, &total);
    if (take) {
      a.values[row * k + pos] = f;
      a.indices[row * k + pos] = v;
    }
    base += total;
  }
  for (int j = (int)want + tid; j < k; j += threads) {
    a.values[row * k + j] = 0.0f;
    a.indices[row * k + j] = -1;
  }
  if (tid == 0) a.counts[row] = (int32_t)want;
  if (a.tail == nullptr) return;
  float m = kNegInf;
  for (int v = tid; v < vocab; v += threads) {
    const float f = to_f32(x[v]);
    if (!taken(order_key(f), v)) m = fmaxf(m, f);
  }
  m = finite_ref(block_max(m, red));
  float s = 0.0f;
  for (int v = tid; v < vocab; v += threads) {
    const float f = to_f32(x[v]);
    if (!taken(order_key(f), v)) s += exp2_fast((f - m) * a.c);
  }
  s = block_sum(s, red);
  if (tid == 0) a.tail[row] = s == 0.0f ? kNegInf : fmaf(m, a.inv_tau, log2_fast(s) * kLn2);
}

// ---------------------------------------------------------------------------
// One warp's selections.  Both narrow a threshold bit by bit between a lower
// and an upper key.
// ---------------------------------------------------------------------------

// A key t with at least k of keys[0..n) at or above it, and not many more:
// the search stops at k + k / 8 + 4.  Returns 0 if there are fewer than k keys
// above -Inf.
__device__ __forceinline__ uint32_t warp_bound(const uint32_t* keys, int n, int k) {
  const int lane = (int)lane_id();
  uint32_t hi = 0, lo = 0xFFFFFFFFu;
  int live = 0;
  for (int i = lane; i < n; i += 32) {
    const uint32_t q = keys[i];
    hi = max(hi, q);
    lo = min(lo, q);
    live += q > kKeyNegInf ? 1 : 0;
  }
  hi = __reduce_max_sync(kFull, hi);
  lo = max(__reduce_min_sync(kFull, lo), kKeyNegInf + 1);
  if (__reduce_add_sync(kFull, live) < k) return 0;
  // t keeps count(t) >= k
  uint32_t t = lo;
  const int most = k + k / 8 + 4;
  const uint32_t differ = hi ^ lo;
  if (differ != 0) {
    const int top = 31 - __clz(differ);
    t = lo & ~((2u << top) - 1u);  // the common prefix: every key is at or above it
    for (int b = top; b >= 0; --b) {
      const uint32_t mid = t | (1u << b);
      int c = 0;
      for (int i = lane; i < n; i += 32) c += keys[i] >= mid ? 1 : 0;
      c = __reduce_add_sync(kFull, c);
      if (c >= k) {
        t = mid;
        if (c <= most) break;
      }
    }
    t = max(t, lo);
  }
  // the smallest key that is at or above it: a value of the row
  uint32_t snap = 0xFFFFFFFFu;
  for (int i = lane; i < n; i += 32)
    if (keys[i] >= t) snap = min(snap, keys[i]);
  return __reduce_min_sync(kFull, snap);
}

constexpr int kBuckets = 512;

// The candidates' packet.  `key`, `idx`: n candidates in any order; `okey`,
// `oidx`: room for as many; `bucket`: kBuckets words.  Writes the row's packet
// and its tail, (m, s) being the sum over the elements that are no candidates.
__device__ __forceinline__ void warp_emit(const TopkArgs& a, int64_t row, int n,
                                          uint32_t* key, int32_t* idx, uint32_t* okey,
                                          int32_t* oidx, uint32_t* bucket, float m, float s) {
  const int lane = (int)lane_id(), k = a.k;
  // in ascending order of position: counted into buckets of neighbouring
  // positions, each bucket's few sorted among themselves
  const int bits = 32 - __clz(max(a.vocab - 1, 1));
  const int shift = max(bits - 9, 0);
  constexpr int kPer = kBuckets / 32;
#pragma unroll
  for (int q = 0; q < kPer; ++q) bucket[q * 32 + lane] = 0;
  __syncwarp();
  for (int i = lane; i < n; i += 32) atomicAdd(&bucket[idx[i] >> shift], 1u);
  __syncwarp();
  uint32_t cnt[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    cnt[q] = bucket[lane * kPer + q];
    sum += cnt[q];
  }
  uint32_t base = warp_incl_scan(sum) - sum;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    bucket[lane * kPer + q] = base;  // the bucket's first place; then its next one
    base += cnt[q];
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const uint32_t at = atomicAdd(&bucket[idx[i] >> shift], 1u);
    okey[at] = key[i];
    oidx[at] = idx[i];
  }
  __syncwarp();
  // bucket b now holds its end, its start is bucket b - 1's end
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    uint32_t kv = 0, to = 0;
    int32_t iv = 0;
    if (i < n) {
      kv = okey[i];
      iv = oidx[i];
      const int b = iv >> shift;
      const uint32_t from = b > 0 ? bucket[b - 1] : 0u, end = bucket[b];
      to = from;
      if (end - from > 1)
        for (uint32_t q = from; q < end; ++q) to += oidx[q] < iv ? 1u : 0u;
    }
    if (i < n) {
      key[to] = kv;
      idx[to] = iv;
    }
  }
  __syncwarp();
  // the k-th largest key, and how many of its ties belong to the packet
  const int want = min(k, n);
  uint32_t cut = 0;
  int need = 0;
  if (n > k && k > 0) {
    uint32_t hi = 0, lo = 0xFFFFFFFFu;
    for (int i = lane; i < n; i += 32) {
      hi = max(hi, key[i]);
      lo = min(lo, key[i]);
    }
    hi = __reduce_max_sync(kFull, hi);
    lo = __reduce_min_sync(kFull, lo);
    cut = lo;
    int at = n;  // keys at or above cut
    if (hi != lo) {
      const int top = 31 - __clz(hi ^ lo);
      cut = lo & ~((2u << top) - 1u);
      for (int b = top; b >= 0 && at != k; --b) {
        const uint32_t mid = cut | (1u << b);
        int c = 0;
        for (int i = lane; i < n; i += 32) c += key[i] >= mid ? 1 : 0;
        c = __reduce_add_sync(kFull, c);
        if (c >= k) {
          cut = mid;
          at = c;
        }
      }
    }
    if (at == k) {
      need = n;  // every key at or above it is taken
    } else {
      int above = 0;
      for (int i = lane; i < n; i += 32) above += key[i] > cut ? 1 : 0;
      need = k - __reduce_add_sync(kFull, above);
    }
  } else {
    need = k > 0 ? n : 0;
    if (k == 0) cut = 0xFFFFFFFFu;
  }
  int out = 0, ties = 0;
  float m2 = kNegInf;  // candidates that are left out
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t kv = i < n ? key[i] : 0u;
    const bool tie = i < n && kv == cut;
    const unsigned tied = __ballot_sync(kFull, tie);
    const bool take =
        i < n && k > 0 && (kv > cut || (tie && ties + __popc(tied & lanemask_lt()) < need));
    const unsigned mask = __ballot_sync(kFull, take);
    if (take) {
      const int pos = out + __popc(mask & lanemask_lt());
      a.values[row * k + pos] = key_value(kv);
      a.indices[row * k + pos] = idx[i];
    }
    // what is left out keeps its key, what is taken becomes -Inf
    if (i < n) {
      if (take) key[i] = kKeyNegInf;
      else m2 = fmaxf(m2, key_value(kv));
    }
    out += __popc(mask);
    ties += __popc(tied);
  }
  for (int j = want + lane; j < k; j += 32) {
    a.values[row * k + j] = 0.0f;
    a.indices[row * k + j] = -1;
  }
  if (lane == 0) a.counts[row] = want;
  if (a.tail == nullptr) return;
  __syncwarp();
  m2 = fmaxf(warp_max(m2), m);
  const float ref = finite_ref(m2);
  float s2 = 0.0f;
  for (int i = lane; i < n; i += 32) s2 += exp2_fast((key_value(key[i]) - ref) * a.c);
  s2 = warp_sum(s2);
  if (m != kNegInf) s2 += s * exp2_fast((m - ref) * a.c);
  else s2 += s;  // 0, or NaN
  if (lane == 0) a.tail[row] = s2 == 0.0f ? kNegInf : fmaf(ref, a.inv_tau, log2_fast(s2) * kLn2);
}

// ---------------------------------------------------------------------------
// A persistent grid; a CTA takes one row after another, in chunks that its
// workers hold in registers.  Two more warps: the first has chunks copied to
// shared memory ahead of time and finds the bound from the workers' maxima, the
// second makes the packet of one row while the others read the next.  A row of
// several chunks keeps its maxima, so the bound rises from chunk to chunk.
// FINE: a group is a slot position (a few per thread) instead of a thread.
// ---------------------------------------------------------------------------

// (kSummed: two, by turns, so that a row's arrivals never meet the last row's)
enum TopkBarrier { kReady = 1, kMaxima, kBound, kSummed, kListFree = kSummed + 2 };

template <int WARPS, int NV, bool FINE>
struct TopkShape {
  static constexpr int kWorkers = WARPS - 2, kLanes = kWorkers * 32, kCap = kLanes * NV;
  static constexpr int kGroups = FINE ? kCap : kLanes;
};

// Shared memory in bytes: the chunk, the groups' keys, two lists of `cap`
// candidates (keys, positions) and the order's scratch.
__host__ __device__ constexpr size_t topk_smem(int slots, int groups, int cap) {
  return (size_t)slots * 16 + (size_t)groups * 4 + (size_t)cap * 24 + kBuckets * 4;
}

template <typename T, int WARPS, int NV, bool FINE>
__global__ void __launch_bounds__(WARPS * 32, 32 / WARPS)
    topk_stream(TopkArgs a, int64_t rows, int chunks, int per, int cap) {
  using S = Slot<T>;
  using M = NanMax<T>;
  using Sh = TopkShape<WARPS, NV, FINE>;
  constexpr int N = S::N, kThreads = WARPS * 32, kLanes = Sh::kLanes, kWorkers = Sh::kWorkers;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t scan[33];
  __shared__ float red[32];
  __shared__ float part_m[2][32], part_s[2][32];  // [kWorkers]: the row's ends
  __shared__ float bound_sh;
  __shared__ int lo_sh;
  __shared__ int count[2];
  __shared__ int again;
  __shared__ __align__(8) uint64_t full;
  uint4* buf = reinterpret_cast<uint4*>(smem);
  uint32_t* groups = reinterpret_cast<uint32_t*>(buf + Sh::kCap);
  uint32_t* lists = groups + Sh::kGroups;  // keys, positions; keys, positions
  uint32_t* order = lists + 4 * cap;       // keys, positions, buckets
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int vocab = a.vocab;
  const float c = a.c;
  const int64_t step = gridDim.x;

  if (tid == 0) {
    mbar_init(&full, 1);
    count[0] = count[1] = again = 0;
    fence_bulk();
  }
  if (warp < kWorkers) {
#pragma unroll
    for (int v = 0; v < NV; ++v) buf[v * kLanes + tid] = S::none();
    fence_bulk();
  }
  __syncthreads();
  pdl_wait();

  // adds a candidate
  auto push = [&](int turn, float f, int at) {
    const int i = atomicAdd(&count[turn], 1);
    if (i < cap) {
      lists[turn * 2 * cap + i] = order_key(f);
      lists[turn * 2 * cap + cap + i] = (uint32_t)at;
    }
  };

  if (warp < kWorkers) {
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += step, turn ^= 1) {
      typename M::P group[FINE ? NV : 1];
#pragma unroll
      for (int v = 0; v < (FINE ? NV : 1); ++v) group[v] = M::none();
      float run = kNegInf, s = 0.0f;  // the warp's maximum below the bound, the lane's sum
      for (int ch = 0; ch < chunks; ++ch) {
        bar_sync(kReady, kThreads - 32);
        const int lo = lo_sh;  // position of the chunk's first element
        uint4 raw[NV];
        typename M::P top[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          raw[v] = buf[v * kLanes + tid];
          top[v] = M::slot(raw[v]);
          if (FINE) {
            group[v] = M::of(group[v], top[v]);
            groups[v * kLanes + tid] = order_key(M::value(group[v]));
          } else {
            group[0] = M::of(group[0], top[v]);
          }
        }
        if (!FINE) groups[tid] = order_key(M::value(group[0]));
        __syncwarp();
        bar_arrive(kMaxima, kThreads - 32);
        bar_sync(kBound, kThreads - 32);
        const float t = bound_sh;
        SlotMax<T> below;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (M::reaches(top[v], t)) {
            float2 f[N / 2];
            S::unpack(raw[v], f);
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (!((e & 1 ? f[e / 2].y : f[e / 2].x) < t)) bits |= 1u << e;
            const int at = lo + (v * kLanes + tid) * N;
            for (uint32_t left = bits; left != 0; left &= left - 1) {
              const int e = __ffs(left) - 1;
              float x = f[0].x;
#pragma unroll
              for (int q = 1; q < N; ++q)
                if (q == e) x = q & 1 ? f[q / 2].y : f[q / 2].x;
              push(turn, x, at + e);
            }
            S::mask(raw[v], bits);
          }
          below.add(raw[v]);
        }
        const float m = warp_max(fmaxf(run, below.get())), ref = finite_ref(m);
        float2 sum = make_float2(0.0f, 0.0f);
        if (run != kNegInf) sum.x = s * exp2_fast((run - ref) * c);
        else sum.x = s;
        run = m;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float2 f[N / 2];
          S::add(raw[v], -ref, f);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            f[e] = mul2(f[e], make_float2(c, c));
            f[e].x = exp2_fast(f[e].x);
            f[e].y = exp2_fast(f[e].y);
            sum = add2(sum, f[e]);
          }
        }
        s = sum.x + sum.y;
      }
      s = warp_sum(s);
      if (lane == 0) {
        part_m[turn][warp] = run;
        part_s[turn][warp] = s;
      }
      __syncwarp();
      bar_arrive(kSummed + turn, kThreads);
    }
  } else if (warp == kWorkers) {
    // ------------------------------------------------ copies and bounds
    bool lost = false;
    uint32_t phase = 0;
    const auto start = [&](int64_t row, int ch) {
      const T* x = static_cast<const T*>(a.logits) + row * a.stride;
      const RowShape shape = S::shape(x, vocab);
      const int lo = min(ch * per, shape.slots), held = min(per, shape.slots - lo);
      if (lane == 0 && !lost) {
        mbar_expect(&full, (uint32_t)held * 16);
        if (held > 0)
          bulk_copy(buf, reinterpret_cast<const uint4*>(x + shape.head) + lo, (uint32_t)held * 16,
                    &full);
      }
    };
    if ((int64_t)blockIdx.x < rows) start(blockIdx.x, 0);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += step, turn ^= 1) {
      const T* x = static_cast<const T*>(a.logits) + row * a.stride;
      const RowShape shape = S::shape(x, vocab);
      const bool has_edge = lane < shape.edge;
      const int edge_at = S::edge_at(shape, lane);
      const T edge = has_edge ? x[edge_at] : from_f32<T>(kNegInf);
      for (int ch = 0; ch < chunks; ++ch) {
        if (!lost && !mbar_wait(&full, phase)) lost = true;
        phase ^= 1;
        lost = __any_sync(kFull, lost);
        const int lo = min(ch * per, shape.slots), held = min(per, shape.slots - lo);
        // slots past the chunk: -Inf, where another chunk or row had elements
        for (int q = held + lane; q < per; q += 32) buf[q] = S::none();
        if (lane == 0) lo_sh = shape.head + lo * N;
        if (ch == 0 && row != (int64_t)blockIdx.x && row != (int64_t)blockIdx.x + step) {
          // the list was the row's before the last one: wait until its packet is made
          __syncwarp();
          bar_sync(kListFree, 64);
        }
        if (ch == 0 && lane == 0) count[turn] = 0;
        __syncwarp();
        bar_sync(kReady, kThreads - 32);
        bar_sync(kMaxima, kThreads - 32);
        // the chunk is in registers
        const bool more = ch + 1 < chunks || row + step < rows;
        if (more) {
          fence_bulk();
          __syncwarp();
          if (ch + 1 < chunks) start(row, ch + 1);
          else start(row + step, 0);
          __syncwarp();
        }
        const uint32_t key = a.k > 0 ? warp_bound(groups, Sh::kGroups, a.k) : 0xFFFFFFFFu;
        // -Inf itself is never a candidate
        const float lowest = sizeof(T) == 2 && to_f32(from_f32<T>(1e30f)) > 1e38f ? -65504.0f
                                                                               : -3.402823466e38f;
        const float t = a.k == 0 ? __int_as_float(0x7F800000) : key == 0 ? lowest : key_value(key);
        if (lane == 0) bound_sh = t;
        if (ch == 0) {
          const float f = to_f32(edge);
          const bool take = has_edge && f != kNegInf && a.k > 0 && !(f < t);
          if (take) push(turn, f, edge_at);
          const float e = take ? kNegInf : f;
          const float m = warp_max(e);
          const float s = warp_sum(exp2_fast((e - finite_ref(m)) * c));
          if (lane == 0) {
            part_m[turn][kWorkers] = m;
            part_s[turn][kWorkers] = s;
          }
        }
        __syncwarp();
        bar_sync(kBound, kThreads - 32);
      }
      __syncwarp();
      if (lost && lane == 0) count[turn] = cap + 1;
      __syncwarp();
      bar_arrive(kSummed + turn, kThreads);
    }
  } else {
    // ------------------------------------------------ packets
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += step, turn ^= 1) {
      bar_sync(kSummed + turn, kThreads);
      const int n = count[turn];
      if (n > cap) {
        if (lane == 0) {
          a.counts[row] = -1;
          again = 1;
        }
      } else {
        const float mw = lane <= kWorkers ? part_m[turn][lane] : kNegInf;
        const float sw = lane <= kWorkers ? part_s[turn][lane] : 0.0f;
        const float m = warp_max(mw), ref = finite_ref(m);
        const float s = warp_sum(mw == kNegInf ? sw : sw * exp2_fast((mw - ref) * c));
        uint32_t* list = lists + turn * 2 * cap;
        warp_emit(a, row, n, list, reinterpret_cast<int32_t*>(list + cap), order,
                  reinterpret_cast<int32_t*>(order + cap), order + 2 * cap, m, s);
      }
      __syncwarp();
      // (for the row after the next one, where there is one)
      if (row + 2 * step < rows) bar_arrive(kListFree, 64);
    }
  }
  __syncthreads();
  if (!again) return;
  for (int64_t row = blockIdx.x; row < rows; row += step) {
    const int n = a.counts[row];
    __syncthreads();
    if (n == -1) plain_row<T>(a, row, scan, red);
    __syncthreads();
  }
}

// CTAs of a persistent kernel: as many as fit the device, at most `most`.
int64_t resident(int sms, int by_threads, size_t smem, int64_t most) {
  int fit = (int)(225 * 1024 / (smem + 2048));
  if (fit > by_threads) fit = by_threads;
  if (fit < 1) fit = 1;
  return (int64_t)sms * fit < most ? (int64_t)sms * fit : most;
}

template <typename T, int WARPS, int NV, bool FINE>
void launch_stream(const TopkArgs& a, int64_t rows, int sms, cudaStream_t s) {
  using Sh = TopkShape<WARPS, NV, FINE>;
  const auto kernel = topk_stream<T, WARPS, NV, FINE>;
  const int64_t slots = a.vocab / Slot<T>::N + 1;
  const int chunks = (int)((slots + Sh::kCap - 1) / Sh::kCap);
  const int per = (int)((slots + chunks - 1) / chunks);
  // candidates: about 1.1 k in a row's first chunk, 1.1 k / i in its i-th
  int deep = 4;
  while ((1 << (deep - 2)) < chunks) ++deep;
  int64_t cap = (int64_t)a.k * deep + 512;
  if (cap > a.vocab) cap = a.vocab;
  if (cap > 4096) cap = 4096;
  cap = (cap + 3) & ~3;
  const size_t smem = topk_smem(Sh::kCap, Sh::kGroups, (int)cap);
  if (smem > 48 * 1024)
    (void)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  const int64_t grid = resident(sms, 32 / WARPS, smem, rows);
  launch_pdl(kernel, dim3((unsigned)grid), dim3(WARPS * 32), smem, s, a, rows, chunks, per,
             (int)cap);
}

template <typename T>
void launch_typed(const TopkArgs& a, int64_t rows, int sms, cudaStream_t s) {
  const int64_t slots = a.vocab / Slot<T>::N + 1;
  // threads as groups while there are well over k of them
  if (slots <= TopkShape<4, 8, true>::kCap && a.k <= 256)
    launch_stream<T, 4, 8, true>(a, rows, sms, s);
  else if (slots <= TopkShape<8, 8, true>::kCap)
    launch_stream<T, 8, 8, true>(a, rows, sms, s);
  else if (a.k <= TopkShape<16, 9, false>::kGroups * 6 / 10)
    launch_stream<T, 16, 9, false>(a, rows, sms, s);
  else
    launch_stream<T, 16, 9, true>(a, rows, sms, s);
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
  TopkArgs a;
  a.logits = logits, a.stride = row_stride, a.vocab = (int)vocab, a.k = k;
  a.c = (float)(1.4426950408889634074 / (double)tau), a.inv_tau = 1.0f / tau;
  a.values = out_values, a.indices = out_indices, a.counts = out_counts, a.tail = out_tail;
  with_dtype(dtype, [&](auto t) {
    launch_typed<decltype(t)>(a, rows, dev.sms, static_cast<cudaStream_t>(stream));
  });
  return check_launch();
}

}  // extern "C"
