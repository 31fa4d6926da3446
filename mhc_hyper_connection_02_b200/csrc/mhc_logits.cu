// Log probabilities of given tokens (with entropy and top alternatives) and distillation from a
// teacher's top logits, over rows of logits, with their gradients.
//
// With c = log2(e) / temperature, m the row's maximum and d_v = (z_v - m) c, one walk over a row
// forms s = sum_v 2^d_v and u = sum_v 2^d_v d_v; then
//   ln p_v  = ln2 (d_v - log2 s),   entropy = ln2 (log2 s - u / s),
//   loss    = sum_k w_k (ln w_k - ln p_{i_k}), w the softmax of the teacher's K logits.
// Each thread carries a running maximum and rescales its sums when it grows; threads, then the CTAs
// of a cluster, join theirs on the common maximum. Sums are fp32 and joined in a fixed order.
//
// Gradients: with e_v = 2^d_v and p_v = e_v / s,
//   d_z_v = (g_lp (1[v = y] - p_v) - g_ent p_v (ln p_v + entropy)) / temperature
//   d_z_v = g (p_v - sum_{k: i_k = v} w_k) / temperature.
// Both are one pass: read a logit, write its gradient (which may take the logit's place).
//
// Masked logits: -infinity has p = 0 and adds nothing (its d is cut at kDCut before the product
// with p). The lowest finite value works like any other: where m c is large the
// difference z - m is formed first. A row of -infinity alone has s = 0: no distribution. A row with
// a NaN or a +infinity has s = NaN, which every output inherits.
#include <cooperative_groups.h>
#include <math.h>

#include "mhc.h"
#include "mhc_internal.h"
#include "mhc_rows.cuh"
#include "mhc_rows_host.h"

namespace mhc {

constexpr int kLgThreads = 256;
constexpr int kLgUnroll = 4;
constexpr int kLgTopMax = MHC_TOP_MAX;
constexpr int kLgCand = 1024;     // candidates for the top alternatives kept in shared memory
constexpr int kLgTeacherMax = MHC_DISTILL_MAX;
constexpr float kDCut = -200.0f;  // 2^-200 is zero in fp32: cutting d there keeps 0 * d finite
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float ex2(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d));
  return e;
}

// May d be formed as fma(z, c, -mc)? While mc's rounding stays far below one.
__device__ __forceinline__ bool small_mc(float mc) { return fabsf(mc) < 4194304.0f; }

// Factor exponent that takes sums on the maximum `from` to the maximum `to` (>= from).
__device__ __forceinline__ float shift_of(float from, float to, float c) {
  return from == -INFINITY ? -1000.0f : fmaxf((from - to) * c, -1000.0f);  // -inf: nothing summed
}

struct RowSums {
  float m, s, u;
};

// Rows of a cluster of C CTAs: CTA r takes the windows [r W, (r + 1) W) of the row.
struct RowPart {
  int off, n, first, last;  // windows [first, last) of the row's n elements
};

template <int DT>
__device__ __forceinline__ RowPart row_part(const void* row, int n, int rank, int ranks) {
  RowPart p;
  p.off = window_offset<DT>(row);
  p.n = n;
  const int ns = window_count<DT>(p.off, n);
  const int per = (ns + ranks - 1) / ranks;
  p.first = min(rank * per, ns);
  p.last = min(p.first + per, ns);
  return p;
}

// This thread's sums over its windows of the part: first + tid, + kLgThreads, .... The usual d is
// one fma, z c - mc with mc = m c rounded: every d is off by mc's rounding, which the end takes out
// again. Where mc overflows (the lowest finite values, or an infinity) d is (z - m) c.
template <int DT, bool kEnt>
__device__ __forceinline__ RowSums thread_sums(const typename Elem<DT>::raw* row, const RowPart& p,
                                               float c) {
  using E = Elem<DT>;
  constexpr int VE = E::kVec;
  RowSums r{-INFINITY, 0.f, 0.f};
  float mc = 0.f;
  for (int s0 = p.first + threadIdx.x; s0 < p.last; s0 += kLgThreads * kLgUnroll) {
    uint4 w[kLgUnroll];
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * kLgThreads;
      // past the part: a window of an empty row, all -infinity
      w[j] = load_window<DT>(row, s < p.last ? p.n : 0, p.off, s);
    }
    float tm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      float x[VE];
      E::unpack(w[j], x);
#pragma unroll
      for (int q = 0; q < VE; ++q) tm = fmaxf(tm, x[q]);
    }
    if (tm > r.m) {
      const float mcn = __fmul_rn(tm, c);
      float d = shift_of(r.m, tm, c);
      if (r.m != -INFINITY && small_mc(mc) && small_mc(mcn)) d = fmaxf(mc - mcn, -1000.0f);
      const float f = ex2(d);
      if constexpr (kEnt) r.u = f * fmaf(d, r.s, r.u);
      r.s *= f;
      r.m = tm;
      mc = mcn;
    }
    const bool usual = small_mc(mc);
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      float x[VE];
      E::unpack(w[j], x);
      float ts = 0.f, tu = 0.f;
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const float d = usual ? fmaf(x[q], c, -mc) : (x[q] - r.m) * c;
        const float e = ex2(d);
        ts += e;
        if constexpr (kEnt) tu = fmaf(e, fmaxf(d, kDCut), tu);
      }
      r.s += ts;
      if constexpr (kEnt) r.u += tu;
    }
  }
  if (small_mc(mc)) {  // from the rounded mc to m c itself
    const float d = -fmaf(r.m, c, -mc), f = r.m == -INFINITY ? 1.0f : ex2(d);
    if constexpr (kEnt)
      if (r.m != -INFINITY) r.u = f * fmaf(d, r.s, r.u);
    r.s *= f;
  }
  return r;
}

template <bool kEnt>
__device__ __forceinline__ RowSums rebase(RowSums r, float m, float c) {
  const float d = shift_of(r.m, m, c), f = ex2(d);
  if constexpr (kEnt) r.u = f * fmaf(d, r.s, r.u);
  r.s *= f;
  r.m = m;
  return r;
}

// The sums of the whole part from its threads', in every thread.
template <bool kEnt>
__device__ __forceinline__ RowSums block_sums(RowSums r, float c, float* red) {
  const float m = block_max<kLgThreads>(r.m, red);
  r = rebase<kEnt>(r, m, c);
  if constexpr (kEnt) {
    const float2 v = block_sum2<kLgThreads>(r.s, r.u, red);
    return {m, v.x, v.y};
  }
  return {m, block_sum<kLgThreads>(r.s, red), 0.f};
}

// The row's sums from the parts' (in shared memory of every CTA of the cluster), in rank order.
template <bool kEnt>
__device__ __forceinline__ RowSums cluster_sums(RowSums* mine, int ranks, float c) {
  if (ranks == 1) return *mine;
  auto cl = cooperative_groups::this_cluster();
  RowSums v[8];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < ranks) {
      v[k] = *cl.map_shared_rank(mine, k);
      m = fmaxf(m, v[k].m);
    }
  RowSums r{m, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < ranks) {
      const RowSums b = rebase<kEnt>(v[k], m, c);
      r.s += b.s;
      r.u += b.u;
    }
  return r;
}

// ------------------------------------------------------------------------------ top alternatives
//
// Keys order logits by value, then by the lower index: the value's bits mapped so that unsigned
// order is float order (-0 counts as +0), above the complement of the index. 0 is "none".

__device__ __forceinline__ uint32_t order_key(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long top_key(uint32_t order, int index) {
  return (static_cast<unsigned long long>(order) << 32) | (0xffffffffu - static_cast<uint32_t>(index));
}

struct TopShared {
  unsigned long long cand[kLgCand];
  unsigned long long list[kLgTopMax];
  unsigned long long warp_best[kLgThreads / 32];
  uint32_t key[kLgThreads];
  uint32_t threshold;
  int count;
  int scan[kLgThreads / 32];
};

// list[r] = the r-th largest of cand[0 .. n), r < K (the rest of the list stays as it is).
__device__ __forceinline__ void rank_select(TopShared& sh, int n, int K) {
  for (int i = threadIdx.x; i < n; i += kLgThreads) {
    const unsigned long long k = sh.cand[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
    if (r < K && k != 0) sh.list[r] = k;
  }
}

// Adds this thread's elements with keys above `bar` (or at it, unless `above`) to the candidates.
template <int DT>
__device__ __forceinline__ void collect(const typename Elem<DT>::raw* row, const RowPart& p,
                                        uint32_t own, uint32_t bar, bool above, TopShared& sh) {
  using E = Elem<DT>;
  if (own == 0 || own < bar || (above && own == bar)) return;
  for (int s0 = p.first + threadIdx.x; s0 < p.last; s0 += kLgThreads * kLgUnroll) {
    uint4 w[kLgUnroll];
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * kLgThreads;
      w[j] = load_window<DT>(row, s < p.last ? p.n : 0, p.off, s);
    }
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * kLgThreads;
      if (s >= p.last) break;
      float x[E::kVec];
      E::unpack(w[j], x);
#pragma unroll
      for (int q = 0; q < E::kVec; ++q) {
        const uint32_t k = order_key(x[q]);
        const int e = window_first<DT>(s, p.off) + q;
        if ((above ? k > bar : k >= bar) && e >= 0 && e < p.n) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kLgCand) sh.cand[at] = top_key(k, e);
        }
      }
    }
  }
}

// The part's K best into sh.list, in order. `m` is this thread's maximum.
//
// The K-th largest of the threads' maxima bounds the K-th largest element from below, and only
// threads whose maximum reaches it can hold an element that does: for logits in no special order
// about K threads walk their windows again, and a few more than K candidates are ranked. Where
// more candidates than fit reach the bound, those above it are taken first and the missing ones
// are the first elements equal to it (rows with long runs of one value: masked or constant rows);
// where even those above it do not fit, K rounds each find the next best element.
template <int DT>
__device__ __forceinline__ void top_of_part(const typename Elem<DT>::raw* row, const RowPart& p,
                                            float m, int K, TopShared& sh) {
  using E = Elem<DT>;
  constexpr int NW = kLgThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t own = p.first + tid < p.last ? order_key(m) : 0;
  __syncthreads();
  sh.key[tid] = own;
  if (tid < kLgTopMax) sh.list[tid] = 0;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  if (warp == 0) {
    uint32_t k[NW], prefix = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) k[i] = sh.key[i * 32 + lane];
    for (int bit = 31; bit >= 32 - E::kOrderBits; --bit) {
      const uint32_t trial = prefix | (1u << bit);
      unsigned n = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) n += k[i] >= trial;
      if (__reduce_add_sync(0xffffffffu, n) >= static_cast<unsigned>(K)) prefix = trial;
    }
    uint32_t lowest = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      if (k[i] >= prefix && k[i] < lowest) lowest = k[i];
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    if (lane == 0) sh.threshold = lowest;
  }
  __syncthreads();
  const uint32_t bar = sh.threshold;  // 0 when fewer than K threads hold elements
  collect<DT>(row, p, own, bar, false, sh);
  __syncthreads();
  int n = sh.count;
  if (n <= kLgCand) {
    rank_select(sh, n, K);
    __syncthreads();
    return;
  }
  __syncthreads();
  if (tid == 0) sh.count = 0;
  __syncthreads();
  collect<DT>(row, p, own, bar, true, sh);
  __syncthreads();
  n = sh.count;
  if (n <= kLgCand) {
    rank_select(sh, n, K);
    // The first K - n elements equal to the bar, in index order.
    int found = n;
    for (int base = p.first; base < p.last && found < K; base += kLgThreads) {
      const int s = base + tid;
      unsigned hits = 0;
      if (s < p.last) {
        float x[E::kVec];
        E::unpack(load_window<DT>(row, p.n, p.off, s), x);
#pragma unroll
        for (int q = 0; q < E::kVec; ++q) {
          const int e = window_first<DT>(s, p.off) + q;
          if (order_key(x[q]) == bar && e >= 0 && e < p.n) hits |= 1u << q;
        }
      }
      int before = __popc(hits);  // inclusive prefix over the warp, then the warps before
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = before;
      __syncthreads();
      int total = 0;
      int at = found + before - __popc(hits);
      for (int w = 0; w < NW; ++w) {
        if (w < warp) at += sh.scan[w];
        total += sh.scan[w];
      }
#pragma unroll
      for (int q = 0; q < E::kVec; ++q)
        if (hits & (1u << q)) {
          if (at < K) sh.list[at] = top_key(bar, window_first<DT>(s, p.off) + q);
          ++at;
        }
      found += total;
    }
    __syncthreads();
    return;
  }
  unsigned long long last = ~0ull;
  for (int r = 0; r < K; ++r) {
    unsigned long long best = 0;
    if (own >= bar)
      for (int s = p.first + tid; s < p.last; s += kLgThreads) {
        float x[E::kVec];
        E::unpack(load_window<DT>(row, p.n, p.off, s), x);
#pragma unroll
        for (int q = 0; q < E::kVec; ++q) {
          const int e = window_first<DT>(s, p.off) + q;
          const unsigned long long k = top_key(order_key(x[q]), e);
          if (e >= 0 && e < p.n && k < last && k > best) best = k;
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long v = __shfl_xor_sync(0xffffffffu, best, o);
      if (v > best) best = v;
    }
    __syncthreads();
    if (lane == 0) sh.warp_best[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w)
      if (sh.warp_best[w] > best) best = sh.warp_best[w];
    if (tid == 0) sh.list[r] = best;
    last = best;
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------ forward kernels

struct LogprobArgs {
  const void* logits;
  int64_t stride;
  const int64_t* targets;  // or null
  float* logprob;          // or null (with targets)
  float* entropy;          // or null
  int64_t* top_index;      // [T][K]
  float* top_logprob;      // [T][K]
  float* stats;            // [T][2] or null
  float c, inv_t;          // log2(e) / temperature, 1 / temperature
  int V, K, ranks;
};

// One cluster of `ranks` CTAs per row.
template <int DT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kLgThreads) logprob_kernel(const LogprobArgs a) {
  using E = Elem<DT>;
  __shared__ float red[2 * kLgThreads / 32];
  __shared__ RowSums part;
  __shared__ typename std::conditional<kTop, TopShared, int>::type sh_top;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x / a.ranks;
  const int rank = static_cast<int>(blockIdx.x - t * a.ranks);
  const auto* row = static_cast<const typename E::raw*>(a.logits) + t * a.stride;
  const RowPart p = row_part<DT>(row, a.V, rank, a.ranks);
  const RowSums own = thread_sums<DT, kEnt>(row, p, a.c);
  const RowSums mine = block_sums<kEnt>(own, a.c, red);
  if (threadIdx.x == 0) part = mine;
  if constexpr (kTop) top_of_part<DT>(row, p, own.m, a.K, sh_top);
  __syncthreads();
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();
  if (rank == 0) {
    const RowSums r = cluster_sums<kEnt>(&part, a.ranks, a.c);
    const float ls = logf(r.s);
    if (threadIdx.x == 0) {
      if (a.logprob) {
        const int64_t y = a.targets[t];
        float lp = 0.0f;  // no target
        if (y >= a.V)
          lp = NAN;
        else if (y >= 0)
          lp = r.s == 0.0f ? -INFINITY
                           : (E::to_f32(row[y]) - r.m) * a.inv_t - ls;
        a.logprob[t] = lp;
      }
      if constexpr (kEnt) a.entropy[t] = r.s == 0.0f ? 0.0f : ls - kLn2 * (r.u / r.s);
      if (a.stats) *reinterpret_cast<float2*>(a.stats + 2 * t) = make_float2(isnan(r.s) ? NAN : r.m, r.s);
    }
    if constexpr (kTop) {
      if (a.ranks > 1) {  // join the parts' lists
        auto cl = cooperative_groups::this_cluster();
        const int n = a.ranks * a.K;
        for (int i = threadIdx.x; i < n; i += kLgThreads)
          sh_top.cand[i] = cl.map_shared_rank(sh_top.list, i / a.K)[i % a.K];
        __syncthreads();
        rank_select(sh_top, n, a.K);
        __syncthreads();
      }
      const int k = threadIdx.x;
      if (k < a.K) {
        const unsigned long long key = sh_top.list[k];
        const int64_t v = 0xffffffffu - static_cast<uint32_t>(key);
        const float z = order_value(static_cast<uint32_t>(key >> 32));
        const bool dead = isnan(r.s);
        a.top_index[t * a.K + k] = dead ? -1 : v;
        a.top_logprob[t * a.K + k] =
            dead ? NAN : r.s == 0.0f ? -INFINITY : (z - r.m) * a.inv_t - ls;
      }
    }
  }
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();  // rank 0 has read this CTA's part
}

struct DistillArgs {
  const void* logits;
  int64_t stride;
  const int64_t* index;  // [T][K], negative: unused
  const void* teacher;   // [T][K]
  float* loss;
  float* weights;        // [T][K]
  float* stats;          // [T][2]
  float c, inv_t;
  int V, K, ranks, teacher_dtype;
};

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == 0) return Elem<0>::to_f32(static_cast<const uint16_t*>(p)[i]);
  if (dtype == 1) return Elem<1>::to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

template <int DT>
__global__ void __launch_bounds__(kLgThreads) distill_kernel(const DistillArgs a) {
  using E = Elem<DT>;
  constexpr int PER = kLgTeacherMax / kLgThreads;
  __shared__ float red[2 * kLgThreads / 32];
  __shared__ RowSums part;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x / a.ranks;
  const int rank = static_cast<int>(blockIdx.x - t * a.ranks);
  const auto* row = static_cast<const typename E::raw*>(a.logits) + t * a.stride;
  const RowPart p = row_part<DT>(row, a.V, rank, a.ranks);
  const RowSums mine = block_sums<false>(thread_sums<DT, false>(row, p, a.c), a.c, red);
  if (threadIdx.x == 0) part = mine;
  __syncthreads();
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();
  if (rank == 0) {
    const RowSums r = cluster_sums<false>(&part, a.ranks, a.c);
    const float ls = logf(r.s);
    // The teacher's softmax over its used entries.
    float g[PER], tm = -INFINITY;
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int k = threadIdx.x + i * kLgThreads;
      const int64_t v = k < a.K ? a.index[t * a.K + k] : -1;
      id[i] = v < 0 ? -1 : v >= a.V ? a.V : static_cast<int>(v);
      g[i] = id[i] < 0 ? -INFINITY : load_any(a.teacher, a.teacher_dtype, t * a.K + k);
      if (id[i] == a.V) g[i] = NAN;  // no such token: the row's loss and gradient say so
      tm = fmaxf(tm, g[i]);
    }
    tm = block_max<kLgThreads>(tm, red);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // tm = -infinity: nothing used; a NaN stays one
      g[i] = tm == -INFINITY && !isnan(g[i]) ? -INFINITY : (g[i] - tm) * a.c;
      sum += ex2(g[i]);
    }
    sum = block_sum<kLgThreads>(sum, red);
    const float tl2 = log2f(sum);
    float loss = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int k = threadIdx.x + i * kLgThreads;
      if (k >= a.K) continue;
      const float w = sum == 0.0f || id[i] < 0 ? 0.0f : ex2(g[i]) / sum;
      a.weights[t * a.K + k] = w;
      if (w != 0.0f) {
        const float lp = id[i] == a.V ? NAN
                         : r.s == 0.0f
                             ? -INFINITY
                             : (E::to_f32(row[id[i]]) - r.m) * a.inv_t - ls;
        loss = fmaf(w, kLn2 * (g[i] - tl2) - lp, loss);
      }
    }
    loss = block_sum<kLgThreads>(loss, red);
    if (threadIdx.x == 0) {
      a.loss[t] = loss;
      *reinterpret_cast<float2*>(a.stats + 2 * t) = make_float2(isnan(r.s) ? NAN : r.m, r.s);
    }
  }
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------------------------ gradient kernel

struct LogitGradArgs {
  const void* logits;
  int64_t stride;
  void* d_logits;
  int64_t d_stride;
  const float* stats;      // [T][2]
  const int64_t* targets;  // log probabilities: or null
  const float* d_logprob;  // or null
  const float* d_entropy;  // or null
  const float* entropy;
  const int64_t* index;    // distillation: [T][K]
  const float* weights;    // [T][K]
  const float* d_loss;
  float c, inv_t;
  int V, K, chunks;
};

constexpr int kLgRounds = 2;  // of kLgUnroll windows per thread and chunk
constexpr int kLgChunk = kLgThreads * kLgUnroll * kLgRounds;  // windows

template <int DT>
__device__ __forceinline__ void store_window(typename Elem<DT>::raw* out, int n, int e0,
                                             bool aligned, const float (&v)[Elem<DT>::kVec]) {
  using E = Elem<DT>;
  if (aligned && e0 >= 0 && e0 <= n - E::kVec) {
    st_stream(out + e0, E::pack(v));
  } else {
#pragma unroll
    for (int q = 0; q < E::kVec; ++q)
      if (e0 + q >= 0 && e0 + q < n) out[e0 + q] = E::from_f32(v[q]);
  }
}

// Coherent form of load_window: the gradient may take the logits' place.
template <int DT>
__device__ __forceinline__ uint4 load_window_rw(const typename Elem<DT>::raw* row, int n, int off,
                                                int s) {
  const int e0 = window_first<DT>(s, off);
  if (e0 >= 0 && e0 <= n - Elem<DT>::kVec) return ld_stream(row + e0);
  return load_window<DT>(row, n, off, s);
}

// One chunk of a row per CTA. kDistill: the dense term g p of every element, then the few teacher
// entries of the chunk once more, each formed in fp32 from its logit (read before any store).
template <int DT, bool kDistill, bool kEnt>
__global__ void __launch_bounds__(kLgThreads) logit_grad_kernel(const LogitGradArgs a) {
  using E = Elem<DT>;
  constexpr int VE = E::kVec;
  constexpr int PER = kLgTeacherMax / kLgThreads;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - t * a.chunks);
  const auto* row = static_cast<const typename E::raw*>(a.logits) + t * a.stride;
  auto* out = static_cast<typename E::raw*>(a.d_logits) + t * a.d_stride;
  const int n = a.V, off = window_offset<DT>(row);
  const bool aligned =
      ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int first = chunk * kLgChunk;
  const int last = min(first + kLgChunk, window_count<DT>(off, n));
  const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * t);
  const float m = st.x, mc = __fmul_rn(st.x, a.c), is = 1.0f / st.y;
  const bool usual = small_mc(mc);
  const float off_d = usual ? fmaf(m, a.c, -mc) : 0.0f;  // what every d of the loop is too large by

  float A, B = 0.f, at_target = 0.f;
  int target = -1;
  bool zero;
  // Distillation: this chunk's teacher entries (position, logit, summed weight).
  [[maybe_unused]] int pos[PER];
  [[maybe_unused]] float ez[PER], ew[PER];
  if constexpr (kDistill) {
    __shared__ int s_pos[kLgTeacherMax];
    __shared__ float s_w[kLgTeacherMax];
    __shared__ uint32_t s_seen[kLgChunk * VE / 32];
    __shared__ int s_twice;
    const int lo = window_first<DT>(first, off);  // of the chunk's first window
    for (int i = threadIdx.x; i < kLgChunk * VE / 32; i += kLgThreads) s_seen[i] = 0;
    if (threadIdx.x == 0) s_twice = 0;
    bool any = false, nan = false;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int k = threadIdx.x + i * kLgThreads;
      pos[i] = -1;
      if (k < a.K) {
        const int64_t v = a.index[t * a.K + k];
        const float w = a.weights[t * a.K + k];
        any |= w != 0.0f;
        nan |= isnan(w);
        int q = -1;
        if (v >= 0 && v < n && w != 0.0f) {
          const int r = static_cast<int>(v) - lo;
          if (r >= 0 && r < (last - first) * VE) q = r;
        }
        s_pos[k] = q;
        s_w[k] = w;
        pos[i] = q;
        ew[i] = w;
        if (q >= 0) {
          ez[i] = E::to_f32(row[lo + q]);
          if (atomicOr(&s_seen[q >> 5], 1u << (q & 31)) & (1u << (q & 31))) s_twice = 1;
        }
      }
    }
    any = __syncthreads_or(any);
    nan = __syncthreads_or(nan);
    if (s_twice) {  // an index given twice: its first entry adds up the weights, in entry order
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = threadIdx.x + i * kLgThreads;
        if (pos[i] < 0) continue;
        float w = 0.f;
        for (int j = 0; j < a.K; ++j) {
          if (s_pos[j] != pos[i]) continue;
          if (j < k) {
            pos[i] = -1;
            break;
          }
          w += s_w[j];
        }
        ew[i] = w;
      }
    }
    const float g = a.d_loss[t];
    zero = g == 0.0f || st.y == 0.0f || !any;
    at_target = g * a.inv_t;  // times each entry's weight
    A = nan ? NAN : at_target * is;
  } else {
    float glp = a.d_logprob ? a.d_logprob[t] : 0.0f;
    if (glp != 0.0f) {
      const int64_t y = a.targets[t];
      if (y < 0)
        glp = 0.0f;
      else if (y >= n)
        glp = NAN;
      else
        target = static_cast<int>(y);
    }
    at_target = glp * a.inv_t;
    A = -at_target * is;
    zero = glp == 0.0f;
    if constexpr (kEnt) {
      const float gent = a.d_entropy[t];
      const float k = a.inv_t * is * gent;
      A -= k * (a.entropy[t] - kLn2 * log2f(st.y));
      B = -k * kLn2;
      zero = zero && gent == 0.0f;
    }
    zero = zero || st.y == 0.0f;
  }
  // e and d as the loop forms them carry off_d: taken out of the row's constants instead.
  const float fa = ex2(-off_d) * fmaf(-B, off_d, A), fb = ex2(-off_d) * B;

  for (int s0 = first + threadIdx.x; s0 < last; s0 += kLgThreads * kLgUnroll) {
    uint4 w[kLgUnroll];
    if (!zero) {
#pragma unroll
      for (int j = 0; j < kLgUnroll; ++j) {
        const int s = s0 + j * kLgThreads;
        if (s < last) w[j] = load_window_rw<DT>(row, n, off, s);
      }
    }
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * kLgThreads;
      if (s >= last) break;
      const int e0 = window_first<DT>(s, off);
      float x[VE];
      if (zero) {
#pragma unroll
        for (int q = 0; q < VE; ++q) x[q] = 0.0f;
      } else {
        E::unpack(w[j], x);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const float d = usual ? fmaf(x[q], a.c, -mc) : (x[q] - m) * a.c;
          const float e = ex2(d);
          if constexpr (kEnt)
            x[q] = e * fmaf(fb, fmaxf(d, kDCut), fa);
          else
            x[q] = e * fa;
        }
        if constexpr (!kDistill) {
          const int at = target - e0;
          if (target >= 0 && at >= 0 && at < VE) {
#pragma unroll
            for (int q = 0; q < VE; ++q)
              if (q == at) x[q] += at_target;
          }
        }
      }
      store_window<DT>(out, n, e0, aligned, x);
    }
  }
  if constexpr (kDistill) {
    if (!zero) {
      __syncthreads();
      const int lo = window_first<DT>(first, off);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (pos[i] >= 0)
          out[lo + pos[i]] =
              E::from_f32(fmaf(ex2((ez[i] - m) * a.c), A, -at_target * ew[i]));
    }
  }
}

// ------------------------------------------------------------------------------ launches

namespace {

// CTAs per row: one while the rows alone fill the device; for few rows a cluster of up to eight
// shares each (every CTA keeping at least one round of windows).
int row_ranks(int64_t T, int V, int vec) {
  const int64_t want = 2 * static_cast<int64_t>(device_sm_count());
  int r = 1;
  while (r < 8 && T * r < want &&
         static_cast<int64_t>(V) / (2 * r) >= static_cast<int64_t>(vec) * kLgThreads)
    r *= 2;
  return r;
}

template <typename A>
int launch_rows(void (*kernel)(A), int64_t T, int ranks, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T * ranks));
  cfg.blockDim = dim3(kLgThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  note_launches(1);
  return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

template <int DT>
int launch_logprob(LogprobArgs a, int64_t T, cudaStream_t s) {
  a.ranks = row_ranks(T, a.V, Elem<DT>::kVec);
  auto kernel = a.entropy ? (a.K > 0 ? logprob_kernel<DT, true, true> : logprob_kernel<DT, true, false>)
                          : (a.K > 0 ? logprob_kernel<DT, false, true> : logprob_kernel<DT, false, false>);
  return launch_rows(kernel, T, a.ranks, s, a);
}

template <int DT>
int launch_distill(DistillArgs a, int64_t T, cudaStream_t s) {
  a.ranks = row_ranks(T, a.V, Elem<DT>::kVec);
  return launch_rows(distill_kernel<DT>, T, a.ranks, s, a);
}

template <int DT>
int launch_logit_grad(LogitGradArgs a, int64_t T, bool distill, cudaStream_t s) {
  // Windows of a row at its worst alignment.
  const int windows = (a.V + 2 * Elem<DT>::kVec - 2) / Elem<DT>::kVec;
  a.chunks = (windows + kLgChunk - 1) / kLgChunk;
  if (T * a.chunks > (int64_t(1) << 31) - 1) return MHC_ERR_INVALID_ARG;
  auto kernel = distill ? logit_grad_kernel<DT, true, false>
                : a.d_entropy ? logit_grad_kernel<DT, false, true>
                              : logit_grad_kernel<DT, false, false>;
  return launch_rows(kernel, T * a.chunks, 1, s, a);
}

bool temperature_ok(float t) {
  return t > 0.0f && isfinite(t) && isfinite(1.0f / t) && isfinite(1.44269504f / t) &&
         1.44269504f / t > 0.0f;
}
float exponent_scale(float t) { return static_cast<float>(1.4426950408889634 / t); }

#define MHC_BY_DTYPE(dtype, f, ...)                                       \
  ((dtype) == MHC_DTYPE_BF16  ? f<MHC_DTYPE_BF16>(__VA_ARGS__)            \
   : (dtype) == MHC_DTYPE_F16 ? f<MHC_DTYPE_F16>(__VA_ARGS__)             \
                              : f<MHC_DTYPE_F32>(__VA_ARGS__))

}  // namespace

}  // namespace mhc

extern "C" {

int mhc_token_logprobs(const void* logits, int64_t row_stride, int dtype, const int64_t* targets,
                       float temperature, float* logprob, float* entropy, int top,
                       int64_t* top_index, float* top_logprob, float* stats, int64_t T, int64_t V,
                       mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, V, row_stride) || !dtype_ok(dtype) || !temperature_ok(temperature) ||
      top < 0 || top > MHC_TOP_MAX || top > V)
    return MHC_ERR_INVALID_ARG;
  if (T > ((int64_t(1) << 31) - 1) / 8) return MHC_ERR_INVALID_ARG;
  if (T == 0) return MHC_OK;
  if (!logits || (!logprob != !targets) || (top > 0 && (!top_index || !top_logprob)))
    return MHC_ERR_INVALID_ARG;
  if (!logprob && !entropy && top == 0 && !stats) return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), nt = static_cast<size_t>(T) * 4;
  if (misaligned(logits, es) || misaligned(targets, 8) || misaligned(logprob, 4) ||
      misaligned(entropy, 4) || misaligned(stats, 8) ||
      (top > 0 && (misaligned(top_index, 8) || misaligned(top_logprob, 4))))
    return MHC_ERR_INVALID_ARG;
  const Range outs[5] = {{logprob, nt},
                         {entropy, nt},
                         {stats, 2 * nt},
                         {top > 0 ? top_index : nullptr, 2 * nt * top},
                         {top > 0 ? top_logprob : nullptr, nt * top}};
  const Range ins[2] = {{logits, row_bytes(T, V, row_stride, es)}, {targets, 2 * nt}};
  if (any_overlap(outs, 5, ins, 2)) return MHC_ERR_ALIAS;
  DeviceScope dev(logits);
  if (dev.status != MHC_OK) return dev.status;
  const LogprobArgs a{logits, row_stride, targets, logprob, entropy, top_index, top_logprob, stats,
                      exponent_scale(temperature), 1.0f / temperature, static_cast<int>(V), top, 1};
  return launched(
      MHC_BY_DTYPE(dtype, launch_logprob, a, T, reinterpret_cast<cudaStream_t>(stream)));
}

int mhc_token_logprobs_backward(const void* logits, int64_t row_stride, int dtype,
                                const int64_t* targets, float temperature, const float* stats,
                                const float* d_logprob, const float* d_entropy,
                                const float* entropy, void* d_logits, int64_t d_row_stride,
                                int64_t T, int64_t V, mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, V, row_stride) || !rows_ok(T, V, d_row_stride) || !dtype_ok(dtype) ||
      !temperature_ok(temperature))
    return MHC_ERR_INVALID_ARG;
  if (T == 0) return MHC_OK;
  if (!logits || !stats || !d_logits || (!d_logprob && !d_entropy) || (d_logprob && !targets) ||
      (d_entropy && !entropy))
    return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), nt = static_cast<size_t>(T) * 4;
  if (misaligned(logits, es) || misaligned(d_logits, es) || misaligned(stats, 8) ||
      misaligned(targets, 8) || misaligned(d_logprob, 4) || misaligned(d_entropy, 4) ||
      misaligned(entropy, 4))
    return MHC_ERR_INVALID_ARG;
  const Range out = {d_logits, row_bytes(T, V, d_row_stride, es)};
  const Range in = {logits, row_bytes(T, V, row_stride, es)};
  const Range rest[5] = {{stats, 2 * nt}, {targets, 2 * nt}, {d_logprob, nt}, {d_entropy, nt},
                         {entropy, nt}};
  const bool in_place = logits == d_logits && row_stride == d_row_stride;
  if ((!in_place && overlap(out, in)) || any_overlap(&out, 1, rest, 5)) return MHC_ERR_ALIAS;
  DeviceScope dev(logits);
  if (dev.status != MHC_OK) return dev.status;
  LogitGradArgs a{};
  a.logits = logits, a.stride = row_stride, a.d_logits = d_logits, a.d_stride = d_row_stride;
  a.stats = stats, a.targets = targets, a.d_logprob = d_logprob;
  a.d_entropy = d_entropy, a.entropy = entropy;
  a.c = exponent_scale(temperature), a.inv_t = 1.0f / temperature, a.V = static_cast<int>(V);
  return launched(
      MHC_BY_DTYPE(dtype, launch_logit_grad, a, T, false, reinterpret_cast<cudaStream_t>(stream)));
}

int mhc_distill_topk(const void* logits, int64_t row_stride, int dtype, const int64_t* index,
                     const void* teacher, int teacher_dtype, float temperature, float* loss,
                     float* weights, float* stats, int64_t T, int64_t V, int64_t K,
                     mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, V, row_stride) || !dtype_ok(dtype) || !dtype_ok(teacher_dtype) ||
      !temperature_ok(temperature) || K < 1 || K > MHC_DISTILL_MAX)
    return MHC_ERR_INVALID_ARG;
  if (T > ((int64_t(1) << 31) - 1) / 8) return MHC_ERR_INVALID_ARG;
  if (T == 0) return MHC_OK;
  if (!logits || !index || !teacher || !loss || !weights || !stats) return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), ts = dtype_size(teacher_dtype);
  const size_t nt = static_cast<size_t>(T) * 4, nk = static_cast<size_t>(T) * K;
  if (misaligned(logits, es) || misaligned(index, 8) || misaligned(teacher, ts) ||
      misaligned(loss, 4) || misaligned(weights, 4) || misaligned(stats, 8))
    return MHC_ERR_INVALID_ARG;
  const Range outs[3] = {{loss, nt}, {weights, 4 * nk}, {stats, 2 * nt}};
  const Range ins[3] = {{logits, row_bytes(T, V, row_stride, es)}, {index, 8 * nk},
                        {teacher, ts * nk}};
  if (any_overlap(outs, 3, ins, 3)) return MHC_ERR_ALIAS;
  DeviceScope dev(logits);
  if (dev.status != MHC_OK) return dev.status;
  const DistillArgs a{logits, row_stride, index, teacher, loss, weights, stats,
                      exponent_scale(temperature), 1.0f / temperature, static_cast<int>(V),
                      static_cast<int>(K), 1, teacher_dtype};
  return launched(
      MHC_BY_DTYPE(dtype, launch_distill, a, T, reinterpret_cast<cudaStream_t>(stream)));
}

int mhc_distill_topk_backward(const void* logits, int64_t row_stride, int dtype,
                              const int64_t* index, const float* weights, const float* stats,
                              const float* d_loss, float temperature, void* d_logits,
                              int64_t d_row_stride, int64_t T, int64_t V, int64_t K,
                              mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, V, row_stride) || !rows_ok(T, V, d_row_stride) || !dtype_ok(dtype) ||
      !temperature_ok(temperature) || K < 1 || K > MHC_DISTILL_MAX)
    return MHC_ERR_INVALID_ARG;
  if (T == 0) return MHC_OK;
  if (!logits || !index || !weights || !stats || !d_loss || !d_logits) return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), nt = static_cast<size_t>(T) * 4;
  const size_t nk = static_cast<size_t>(T) * K;
  if (misaligned(logits, es) || misaligned(d_logits, es) || misaligned(index, 8) ||
      misaligned(weights, 4) || misaligned(stats, 8) || misaligned(d_loss, 4))
    return MHC_ERR_INVALID_ARG;
  const Range out = {d_logits, row_bytes(T, V, d_row_stride, es)};
  const Range in = {logits, row_bytes(T, V, row_stride, es)};
  const Range rest[4] = {{index, 8 * nk}, {weights, 4 * nk}, {stats, 2 * nt}, {d_loss, nt}};
  const bool in_place = logits == d_logits && row_stride == d_row_stride;
  if ((!in_place && overlap(out, in)) || any_overlap(&out, 1, rest, 4)) return MHC_ERR_ALIAS;
  DeviceScope dev(logits);
  if (dev.status != MHC_OK) return dev.status;
  LogitGradArgs a{};
  a.logits = logits, a.stride = row_stride, a.d_logits = d_logits, a.d_stride = d_row_stride;
  a.stats = stats, a.index = index, a.weights = weights, a.d_loss = d_loss;
  a.c = exponent_scale(temperature), a.inv_t = 1.0f / temperature;
  a.V = static_cast<int>(V), a.K = static_cast<int>(K);
  return launched(
      MHC_BY_DTYPE(dtype, launch_logit_grad, a, T, true, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
