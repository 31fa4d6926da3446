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

constexpr int kLgUnroll = 4;
constexpr int kLgTopMax = MHC_TOP_MAX;
constexpr float kDCut = -200.0f;  // 2^-200 is zero in fp32: cutting d there keeps 0 * d finite
constexpr float kLn2 = 0.693147180559945309f;

// The hardware's base-2 exponential: relative error up to 2^-22, four times that of a rounded one, in
// every sum, weight and gradient here (fp32 outputs are off by about 1.5e-7 where plain fp32
// arithmetic's are by 5e-8). A more exact one takes several instructions more an element, in passes
// that issue slots bound next to memory. Results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d));
  return e;
}

__device__ __forceinline__ F2 ex2(F2 d) {
  const float2 v = split(d);
  return f2(ex2(v.x), ex2(v.y));
}
__device__ __forceinline__ F2 max2(F2 d, float lo) {
  const float2 v = split(d);
  return f2(fmaxf(v.x, lo), fmaxf(v.y, lo));
}

// May Elem's cut of the logits at -2^100 stand for the cut of d? Where c carries that value far
// below kDCut, but not to -infinity.
template <int DT>
__device__ __forceinline__ bool cut_ok(float c) {
  return !Elem<DT>::kCuts || (c > 1e-18f && c < 1e7f);
}

// May d be formed as fma(z, c, -mc)? While mc's rounding stays far below one.
__device__ __forceinline__ bool small_mc(float mc) { return fabsf(mc) < 4194304.0f; }

// Factor exponent that takes sums on the maximum `from` to the maximum `to` (>= from).
__device__ __forceinline__ float shift_of(float from, float to, float c) {
  return from == -INFINITY ? -1000.0f : fmaxf((from - to) * c, -1000.0f);  // -inf: nothing summed
}

// The same for a thread's running sums, which stand on what their d was formed with: the rounded mc
// where that is small, else m c itself. A change from one to the other takes mc's rounding, up to a
// quarter, out again or in.
__device__ __forceinline__ float shift_between(float from, float mc_from, float to, float mc_to,
                                               float c) {
  if (from == -INFINITY) return -1000.0f;
  if (small_mc(mc_from) && small_mc(mc_to)) return fmaxf(mc_from - mc_to, -1000.0f);
  float d = (from - to) * c;
  if (small_mc(mc_from)) d -= fmaf(from, c, -mc_from);
  if (small_mc(mc_to)) d += fmaf(to, c, -mc_to);
  return fmaxf(d, -1000.0f);
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

// Where a thread's maximum was met first, and the largest maximum of its other rounds.
struct ThreadBest {
  int round;     // first window of that round of kLgUnroll
  float second;
};

// This thread's sums over its windows of the part: first + tid, + NT, .... The usual d is one fma,
// z c - mc with mc = m c rounded: every d is off by mc's rounding, which the end takes out again.
// Where mc overflows (the lowest finite values, or an infinity) d is (z - m) c.
//
// ex2 runs at 16 a clock and SM: a warp's takes 8 of the 11 cycles that HBM's rate allows an element
// of bf16. The rest is therefore done on packed values (maximum, cut) and on pairs of fp32.
// T=8192, V=131072, bf16: 310 us, with entropy 319 us (6.9 and 6.7 TB/s) in a burst, without packed
// values and pairs 352 and 406 us. Under seconds of load they take 359 and 387 us, at the power cap
// and 1.55 GHz: ex2 by itself would take 290 us there, so it is not the bound alone.
template <int DT, int NT, bool kEnt>
__device__ __forceinline__ RowSums thread_sums(const typename Elem<DT>::raw* row, const RowPart& p,
                                               float c, ThreadBest& best) {
  using E = Elem<DT>;
  constexpr int VE = E::kVec;
  RowSums r{-INFINITY, 0.f, 0.f};
  best = {0, -INFINITY};
  F2 s2 = f2(0.f), u2 = f2(0.f);
  float mc = 0.f;
  const F2 c2 = f2(c);
  const bool cut = cut_ok<DT>(c);
  for (int s0 = p.first + threadIdx.x; s0 < p.last; s0 += NT * kLgUnroll) {
    uint4 w[kLgUnroll];
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * NT;
      // past the part: a window of an empty row, all -infinity
      w[j] = load_window<DT>(row, s < p.last ? p.n : 0, p.off, s);
    }
    const float tm = E::max_of(w);
    best.second = fmaxf(best.second, fminf(tm, r.m));
    if (tm > r.m) {
      best.round = s0;
      const float mcn = __fmul_rn(tm, c);
      const float d = shift_between(r.m, mc, tm, mcn, c);
      const F2 f = f2(ex2(d));
      if constexpr (kEnt) u2 = f * fma2(f2(d), s2, u2);
      s2 = f * s2;
      r.m = tm;
      mc = mcn;
    }
    if (small_mc(mc) && (!kEnt || cut)) {
      const F2 nmc = f2(-mc);
#pragma unroll
      for (int j = 0; j < kLgUnroll; ++j) {
        float x[VE];
        E::unpack(kEnt ? E::cut(w[j]) : w[j], x);
#pragma unroll
        for (int q = 0; q < VE; q += 2) {
          const F2 d = fma2(f2(x[q], x[q + 1]), c2, nmc);
          const F2 e = ex2(d);
          s2 = s2 + e;
          if constexpr (kEnt) u2 = fma2(e, E::kCuts ? d : max2(d, kDCut), u2);
        }
      }
    } else {
      const bool usual = small_mc(mc);
#pragma unroll
      for (int j = 0; j < kLgUnroll; ++j) {
        float x[VE];
        E::unpack(w[j], x);
#pragma unroll
        for (int q = 0; q < VE; q += 2) {
          F2 d;
          if (usual)
            d = fma2(f2(x[q], x[q + 1]), c2, f2(-mc));
          else
            d = f2((x[q] - r.m) * c, (x[q + 1] - r.m) * c);
          const F2 e = ex2(d);
          s2 = s2 + e;
          if constexpr (kEnt) u2 = fma2(e, max2(d, kDCut), u2);
        }
      }
    }
  }
  const float2 vs = split(s2), vu = split(u2);
  r.s = vs.x + vs.y;
  r.u = vu.x + vu.y;
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
template <int NT, bool kEnt>
__device__ __forceinline__ RowSums block_sums(RowSums r, float c, float* red) {
  const float m = block_max<NT>(r.m, red);
  r = rebase<kEnt>(r, m, c);
  if constexpr (kEnt) {
    const float2 v = block_sum2<NT>(r.s, r.u, red);
    return {m, v.x, v.y};
  }
  return {m, block_sum<NT>(r.s, red), 0.f};
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

template <int NT>
struct TopShared {
  // candidates; at least what the CTAs of a cluster join
  static constexpr int kCand = 4 * NT > 8 * kLgTopMax ? 4 * NT : 8 * kLgTopMax;
  unsigned long long cand[kCand];
  unsigned long long list[kLgTopMax];
  unsigned long long warp_best[NT / 32];
  // Maxima of groups of threads: enough that the K-th largest of them lets few elements through.
  static constexpr int kGroup = NT >= 256 ? 4 : NT >= 128 ? 2 : 1, kGroups = NT / kGroup;
  uint32_t key[kGroups];
  int round[NT], thread[NT];
  int count, rounds, threads;
  int scan[NT / 32];
};

// list[r] = the r-th largest of cand[0 .. n), r < K (the rest of the list stays as it is).
template <int NT>
__device__ __forceinline__ void rank_select(TopShared<NT>& sh, int n, int K) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const unsigned long long k = sh.cand[i];
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
    if (r < K && k != 0) sh.list[r] = k;
  }
}

// Adds the elements with keys from `least` on to the candidates. Only threads with a maximum that
// qualifies can hold one, and all but those whose second round qualifies too in one round of windows
// alone: the rounds and the threads are gathered, and the whole CTA walks them. Does nothing (returns
// false) where more than `most` threads qualify.
template <int DT, int NT>
__device__ __forceinline__ bool collect(const typename Elem<DT>::raw* row, const RowPart& p,
                                        uint32_t own, const ThreadBest& best, uint32_t least,
                                        int most, TopShared<NT>& sh) {
  using E = Elem<DT>;
  if (own >= least) {
    if (order_key(best.second) < least)
      sh.round[atomicAdd(&sh.rounds, 1)] = best.round;
    else
      sh.thread[atomicAdd(&sh.threads, 1)] = p.first + threadIdx.x;
  }
  __syncthreads();
  const int per = (p.last - p.first + NT - 1) / NT, rounds = kLgUnroll * sh.rounds;
  const int items = rounds + sh.threads * per;
  if (sh.rounds + sh.threads > most) return false;
  for (int i0 = threadIdx.x; i0 < items; i0 += NT * 2) {
    uint4 w[2];
    int at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = i0 + j * NT, h = (i - rounds) / per;
      at[j] = i < rounds  ? sh.round[i / kLgUnroll] + i % kLgUnroll * NT
              : i < items ? sh.thread[h] + (i - rounds - h * per) * NT
                          : p.last;
      w[j] = load_window<DT>(row, at[j] < p.last ? p.n : 0, p.off, at[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (at[j] >= p.last) continue;
      float x[E::kVec];
      E::unpack(w[j], x);
#pragma unroll
      for (int q = 0; q < E::kVec; ++q) {
        const uint32_t k = order_key(x[q]);
        const int e = window_first<DT>(at[j], p.off) + q;
        if (k >= least && e >= 0 && e < p.n) {
          const int to = atomicAdd(&sh.count, 1);
          if (to < TopShared<NT>::kCand) sh.cand[to] = top_key(k, e);
        }
      }
    }
  }
  __syncthreads();
  return true;
}

// The K-th largest of the groups' keys, in every lane of every warp; 0 when there are not as many.
template <int DT, int NT>
__device__ __forceinline__ uint32_t kth_key(const TopShared<NT>& sh, int K) {
  constexpr int M = TopShared<NT>::kGroups / 32;
  const int lane = threadIdx.x & 31;
  uint32_t k[M], prefix = 0;
#pragma unroll
  for (int i = 0; i < M; ++i) k[i] = sh.key[i * 32 + lane];
  for (int bit = 31; bit >= 32 - Elem<DT>::kOrderBits; --bit) {
    const uint32_t trial = prefix | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) n += __popc(__ballot_sync(0xffffffffu, k[i] >= trial));
    if (n >= K) prefix = trial;
    if (n == K) break;
  }
  uint32_t lowest = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < M; ++i)
    if (k[i] >= prefix && k[i] < lowest) lowest = k[i];
  return __reduce_min_sync(0xffffffffu, lowest);
}

// The part's K best into sh.list, in order. `m` is this thread's maximum.
//
// The K-th largest of the thread groups' maxima bounds the K-th largest element from below, and only
// threads whose maximum reaches it can hold an element that does: for logits in no special order
// a few more than K threads' windows are walked again, and a few more than K candidates are ranked.
// Where many more threads (rows with long runs of one value: masked or constant rows) or more
// candidates than fit reach the bound, those above it are taken first and the missing ones are the
// first elements equal to it; where even those above it do not fit, K rounds each find the next best
// element.
template <int DT, int NT>
__device__ __forceinline__ void top_of_part(const typename Elem<DT>::raw* row, const RowPart& p,
                                            float m, const ThreadBest& best, int K,
                                            TopShared<NT>& sh) {
  using E = Elem<DT>;
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t own = p.first + tid < p.last ? order_key(m) : 0;
  uint32_t of_group = own;
#pragma unroll
  for (int o = 1; o < TopShared<NT>::kGroup; o <<= 1)
    of_group = max(of_group, __shfl_xor_sync(0xffffffffu, of_group, o));
  __syncthreads();
  if (tid % TopShared<NT>::kGroup == 0) sh.key[tid / TopShared<NT>::kGroup] = of_group;
  if (tid < kLgTopMax) sh.list[tid] = 0;
  if (tid == 0) sh.count = 0, sh.rounds = 0, sh.threads = 0;
  __syncthreads();
  const uint32_t bar = kth_key<DT, NT>(sh, K);
  if (collect<DT, NT>(row, p, own, best, bar > 0 ? bar : 1, 2 * K + 32, sh)) {
    const int n = sh.count;
    if (n <= TopShared<NT>::kCand) {
      rank_select<NT>(sh, n, K);
      __syncthreads();
      return;
    }
  }
  __syncthreads();
  if (tid == 0) sh.count = 0, sh.rounds = 0, sh.threads = 0;
  __syncthreads();
  collect<DT, NT>(row, p, own, best, bar + 1, NT, sh);  // keys stay below 2^32 - 1
  const int n = sh.count;
  if (n <= TopShared<NT>::kCand) {
    rank_select<NT>(sh, n, K);
    // The first K - n elements equal to the bar, in index order.
    int found = n;
    for (int base = p.first; base < p.last && found < K; base += NT) {
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
      for (int s = p.first + tid; s < p.last; s += NT) {
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
  int64_t first;           // row of the launch's first cluster
  bool tail;               // of a split launch (RowSplit)
};

// The rows of a call in one launch or two. A row's CTA streams at a fixed rate, so where the rows
// fill the device a few times and a few are left over, those take as long as a full round. They go
// into a launch of their own, shared by clusters, that starts while the last full round runs: its
// CTAs start when every CTA of the first launch has started (and so has seen the launch before it
// finished), and wait for the first launch's end before their own.
__device__ __forceinline__ void begin_rows(bool tail) {
  if (!tail) pdl_wait();
  pdl_trigger();
}
__device__ __forceinline__ void end_rows(bool tail) {
  if (tail) pdl_wait();
}

// CTAs that an SM has to hold: at 1536 threads the plain form took 309 us instead of 317 us, with
// alternatives (whose second look at the windows wants registers) at 1280 threads 371 us instead of
// 408 us (T=8192, V=131072, bf16).
__host__ __device__ constexpr int logprob_ctas(int threads, bool top) {
  return threads > 32 ? (top ? 1280 : 1536) / threads : 1;
}

template <int DT, int NT, bool kEnt, bool kTop>
__global__ void __launch_bounds__(NT, logprob_ctas(NT, kTop)) logprob_kernel(const LogprobArgs a) {
  using E = Elem<DT>;
  __shared__ float red[2 * NT / 32];
  __shared__ RowSums part;
  __shared__ typename std::conditional<kTop, TopShared<NT>, int>::type sh_top;
  begin_rows(a.tail);
  const int rank = blockIdx.x % a.ranks;
  const int64_t t = a.first + blockIdx.x / a.ranks;
  const auto* row = static_cast<const typename E::raw*>(a.logits) + t * a.stride;
  const RowPart p = row_part<DT>(row, a.V, rank, a.ranks);
  ThreadBest best;
  const RowSums own = thread_sums<DT, NT, kEnt>(row, p, a.c, best);
  const RowSums mine = block_sums<NT, kEnt>(own, a.c, red);
  if (threadIdx.x == 0) part = mine;
  if constexpr (kTop) top_of_part<DT, NT>(row, p, own.m, best, a.K, sh_top);
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
        for (int i = threadIdx.x; i < n; i += NT)
          sh_top.cand[i] = cl.map_shared_rank(sh_top.list, i / a.K)[i % a.K];
        __syncthreads();
        rank_select<NT>(sh_top, n, a.K);
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
  end_rows(a.tail);
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
  int64_t first;
  bool tail;
};

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == 0) return Elem<0>::to_f32(static_cast<const uint16_t*>(p)[i]);
  if (dtype == 1) return Elem<1>::to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT, logprob_ctas(NT, false)) distill_kernel(const DistillArgs a) {
  using E = Elem<DT>;
  extern __shared__ float entries_f[];  // rank 0: [2][K]
  __shared__ float red[2 * NT / 32];
  __shared__ RowSums part;
  begin_rows(a.tail);
  const int rank = blockIdx.x % a.ranks;
  const int64_t t = a.first + blockIdx.x / a.ranks;
  const auto* row = static_cast<const typename E::raw*>(a.logits) + t * a.stride;
  const RowPart p = row_part<DT>(row, a.V, rank, a.ranks);
  ThreadBest best;
  const RowSums mine = block_sums<NT, false>(thread_sums<DT, NT, false>(row, p, a.c, best), a.c, red);
  if (threadIdx.x == 0) part = mine;
  __syncthreads();
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();
  if (rank == 0) {
    const RowSums r = cluster_sums<false>(&part, a.ranks, a.c);
    const float ls = logf(r.s);
    // The teacher's softmax over its used entries. Each thread keeps its entries' values in shared
    // memory (scaled teacher logits; student logits).
    float* gs = entries_f;
    float* zs = gs + a.K;
    float tm = -INFINITY;
    for (int k = threadIdx.x; k < a.K; k += NT) {
      const int64_t v = a.index[t * a.K + k];
      float g = -INFINITY, z = 0.0f;
      if (v >= a.V) {
        g = NAN;  // no such token: the row's loss and gradient say so
      } else if (v >= 0) {
        g = load_any(a.teacher, a.teacher_dtype, t * a.K + k);
        z = E::to_f32(row[v]);
      }
      gs[k] = g;
      zs[k] = z;
      tm = fmaxf(tm, g);
    }
    tm = block_max<NT>(tm, red);
    float sum = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) {
      // tm = -infinity: nothing used; a NaN stays one
      const float g = gs[k], d = tm == -INFINITY && !isnan(g) ? -INFINITY : (g - tm) * a.c;
      gs[k] = d;
      sum += ex2(d);
    }
    sum = block_sum<NT>(sum, red);
    const float tl2 = log2f(sum);
    float loss = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) {
      const float d = gs[k];
      const bool unused = isnan(sum) && a.index[t * a.K + k] < 0;  // else d = -infinity says so
      const float w = sum == 0.0f || unused ? 0.0f : ex2(d) / sum;
      a.weights[t * a.K + k] = w;
      if (w != 0.0f) {
        const float lp = r.s == 0.0f ? -INFINITY : (zs[k] - r.m) * a.inv_t - ls;
        loss = fmaf(w, kLn2 * (d - tl2) - lp, loss);
      }
    }
    loss = block_sum<NT>(loss, red);
    if (threadIdx.x == 0) {
      a.loss[t] = loss;
      *reinterpret_cast<float2*>(a.stats + 2 * t) = make_float2(isnan(r.s) ? NAN : r.m, r.s);
    }
  }
  if (a.ranks > 1) cooperative_groups::this_cluster().sync();
  end_rows(a.tail);
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

// The constants of a row's gradient: e (fb d + fa) with e = 2^d (kEnt; e fa otherwise).
struct GradRow {
  float c, m, mc, fa, fb;
  bool usual;  // d by one fma, and the bracket is formed before the product with e
};
template <int DT, bool kEnt>
__device__ __forceinline__ GradRow grad_row(float c, float m, float A, float B) {
  GradRow g;
  g.c = c, g.m = m, g.mc = __fmul_rn(m, c);
  g.usual = small_mc(g.mc) && (!kEnt || cut_ok<DT>(c));
  // A masked logit's e is 0: in the usual form its bracket has to stay finite at the lowest d that
  // the cuts leave, or the product would be NaN.
  if constexpr (kEnt)
    g.usual = g.usual && fmaf(fabsf(B), Elem<DT>::kCuts ? c * 0x1p100f : -kDCut, fabsf(A)) < 1e38f;
  // What every d of the usual form is too large by (see thread_sums): taken out of the constants.
  const float off = g.usual ? fmaf(m, c, -g.mc) : 0.0f;
  g.fa = ex2(-off) * fmaf(-B, off, A);
  g.fb = ex2(-off) * B;
  return g;
}

// A window's gradients without the terms of single elements.
template <int DT, bool kEnt, bool kUsual>
__device__ __forceinline__ void grad_window(uint4 w, const GradRow& g, float (&x)[Elem<DT>::kVec]) {
  using E = Elem<DT>;
  E::unpack(kEnt && kUsual ? E::cut(w) : w, x);
#pragma unroll
  for (int q = 0; q < E::kVec; q += 2) {
    F2 d;
    if constexpr (kUsual)
      d = fma2(f2(x[q], x[q + 1]), f2(g.c), f2(-g.mc));
    else
      d = f2((x[q] - g.m) * g.c, (x[q + 1] - g.m) * g.c);
    F2 e = ex2(d);
    if constexpr (kEnt && kUsual)
      e = e * fma2(f2(g.fb), E::kCuts ? d : max2(d, kDCut), f2(g.fa));
    else if constexpr (kEnt)
      e = fma2(e * max2(d, kDCut), f2(g.fb), e * f2(g.fa));
    else
      e = e * f2(g.fa);
    const float2 v = split(e);
    x[q] = v.x, x[q + 1] = v.y;
  }
}

// A chunk of a row: kLgRounds times kLgUnroll windows a thread. Twice as many windows took 3 % longer
// for wide rows (fewer, longer CTAs: their tail), half as many 4 to 9 % (a chunk's start).
constexpr int kLgRounds = 2;
// CTAs that an SM has to hold: 1536 threads, at 40 registers. The passes wait for memory, and with
// 1024 threads of 64 registers the distillation's took 376 us, with 1280 339 us, with these 331 us
// (T=4096, V=131072, bf16), although 24 to 60 bytes a thread of its entry then go to local memory.
constexpr int grad_ctas(int threads) { return threads > 32 ? 1536 / threads : 1; }
template <int DT, int NT>
struct GradChunk {
  using raw = typename Elem<DT>::raw;
  const raw* row;
  raw* out;
  int off, first, last;  // windows [first, last)
  bool aligned;
  __device__ __forceinline__ GradChunk(const LogitGradArgs& a, int64_t t, int chunk) {
    row = static_cast<const raw*>(a.logits) + t * a.stride;
    out = static_cast<raw*>(a.d_logits) + t * a.d_stride;
    off = window_offset<DT>(row);
    aligned = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    constexpr int per = NT * kLgUnroll * kLgRounds;
    first = chunk * per;
    last = min(first + per, window_count<DT>(off, a.V));
  }
  __device__ __forceinline__ void fetch(int n, int s0, uint4 (&w)[kLgUnroll]) const {
#pragma unroll
    for (int j = 0; j < kLgUnroll; ++j) {
      const int s = s0 + j * NT;
      if (s < last) w[j] = load_window_rw<DT>(row, n, off, s);
    }
  }
  // f(window, its first element, the values to store) forms the gradients of each of the thread's
  // windows, the first of which are in w.
  template <bool kRead, typename F>
  __device__ __forceinline__ void walk(int n, uint4 (&w)[kLgUnroll], F&& f) const {
    for (int s0 = first + threadIdx.x; s0 < last;) {
#pragma unroll
      for (int j = 0; j < kLgUnroll; ++j) {
        const int s = s0 + j * NT;
        if (s >= last) break;
        const int e0 = window_first<DT>(s, off);
        float x[Elem<DT>::kVec];
        f(w[j], e0, x);
        store_window<DT>(out, n, e0, aligned, x);
      }
      s0 += NT * kLgUnroll;
      if (kRead && s0 < last) fetch(n, s0, w);
    }
  }
  __device__ __forceinline__ void fill(int n, uint4 (&w)[kLgUnroll], float v) const {
    walk<false>(n, w, [&](const uint4&, int, float (&x)[Elem<DT>::kVec]) {
#pragma unroll
      for (int q = 0; q < Elem<DT>::kVec; ++q) x[q] = v;
    });
  }
};

// Gradient of log probability and entropy, a chunk per CTA. The first windows are read before
// anything else. Bound by HBM: T=8192, V=131072 bf16 625 us, 6.9 TB/s (read and written once).
template <int DT, int NT, bool kEnt>
__global__ void __launch_bounds__(NT, grad_ctas(NT)) logprob_grad_kernel(const LogitGradArgs a) {
  constexpr int VE = Elem<DT>::kVec;
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x / a.chunks;
  const GradChunk<DT, NT> ch(a, t, static_cast<int>(blockIdx.x - t * a.chunks));
  uint4 w[kLgUnroll];
  ch.fetch(a.V, ch.first + threadIdx.x, w);

  const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * t);
  const float is = 1.0f / st.y;
  float glp = a.d_logprob ? a.d_logprob[t] : 0.0f;
  int target = -VE;
  if (glp != 0.0f) {
    const int64_t y = a.targets[t];
    if (y < 0)
      glp = 0.0f;
    else if (y >= a.V)
      glp = NAN;
    else
      target = static_cast<int>(y);
  }
  const float at_target = glp * a.inv_t;
  float A = -at_target * is, B = 0.f;
  bool zero = glp == 0.0f;
  if constexpr (kEnt) {
    const float gent = a.d_entropy[t];
    const float k = a.inv_t * is * gent;
    A -= k * (a.entropy[t] - kLn2 * log2f(st.y));
    B = -k * kLn2;
    zero = zero && gent == 0.0f;
  }
  if (zero || st.y == 0.0f) {
    ch.fill(a.V, w, 0.0f);
    return;
  }
  const GradRow g = grad_row<DT, kEnt>(a.c, st.x, A, B);
  auto walk = [&](auto usual) {
    ch.template walk<true>(a.V, w, [&](const uint4& v, int e0, float (&x)[VE]) {
      grad_window<DT, kEnt, decltype(usual)::value>(v, g, x);
      const int at = target - e0;
      if (at >= 0 && at < VE) {
#pragma unroll
        for (int q = 0; q < VE; ++q)
          if (q == at) x[q] += at_target;
      }
    });
  };
  if (g.usual)
    walk(std::true_type{});
  else
    walk(std::false_type{});
}

// Gradient of the distillation loss, a chunk per CTA: the dense term g p of every element, then the
// few teacher entries of the chunk once more, each formed in fp32 from its logit. The entries are
// read along with the first windows and wait in registers, so that the dense walk need not wait for
// them; where it takes the logits' place, only its first store does. Two entries of one token are
// told by a bit per element of the chunk; only then are the entries compared (comparing them always
// took a tenth of the pass).
template <int DT, int NT>
__global__ void __launch_bounds__(NT, grad_ctas(NT)) distill_grad_kernel(const LogitGradArgs a) {
  using E = Elem<DT>;
  constexpr int VE = E::kVec;
  constexpr int kSeen = NT * kLgUnroll * kLgRounds * VE / 32;
  static_assert(kSeen % NT == 0, "whole words a thread");
  enum { kAny = 1, kNan = 2, kTwice = 4 };
  extern __shared__ int pos[];  // [K] positions in the chunk (or -1), weights, logits
  __shared__ uint32_t seen[kSeen];
  __shared__ int flags;
  float* const ws = reinterpret_cast<float*>(pos) + a.K;
  float* const zs = ws + a.K;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / a.chunks;
  const GradChunk<DT, NT> ch(a, t, static_cast<int>(blockIdx.x - t * a.chunks));
  uint4 w[kLgUnroll];
  ch.fetch(a.V, ch.first + tid, w);
  struct Entry {
    int at;  // position in the chunk, or -1
    float w, z;
  };
  auto read_entry = [&](int k) {
    const int64_t v = a.index[t * a.K + k];
    Entry e{-1, a.weights[t * a.K + k], 0.f};
    if (v >= 0 && v < a.V && e.w != 0.0f) {
      const int r = static_cast<int>(v) - window_first<DT>(ch.first, ch.off);
      if (r >= 0 && r < (ch.last - ch.first) * VE) e.at = r, e.z = E::to_f32(ch.row[v]);
    }
    return e;
  };
  auto keep_entry = [&](int k, const Entry& e) {
    pos[k] = e.at;
    ws[k] = e.w;
    zs[k] = e.z;
    int f = (e.w != 0.0f ? kAny : 0) | (isnan(e.w) ? kNan : 0);
    if (e.at >= 0) {
      const uint32_t bit = 1u << (e.at & 31);
      if (atomicOr(&seen[e.at >> 5], bit) & bit) f |= kTwice;
    }
    if (f) atomicOr(&flags, f);
  };
  Entry e{-1, 0.f, 0.f};
  if (tid < a.K) e = read_entry(tid);
#pragma unroll
  for (int i = 0; i < kSeen / NT; ++i) seen[i * NT + tid] = 0;
  if (tid == 0) flags = 0;
  if (a.K > NT || ch.row == ch.out) {
    __syncthreads();
    for (int k = tid + NT; k < a.K; k += NT) keep_entry(k, read_entry(k));
    if (tid < a.K) zs[tid] = e.z;
    __syncthreads();  // the entries' logits are read
  }

  const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * t);
  const float dl = a.d_loss[t];
  const float at_entry = dl * a.inv_t;  // times each entry's weight
  const float A = at_entry / st.y;
  if (dl == 0.0f || st.y == 0.0f) {
    ch.fill(a.V, w, 0.0f);
    return;
  }
  const GradRow g = grad_row<DT, false>(a.c, st.x, A, 0.0f);
  auto walk = [&](auto usual) {
    ch.template walk<true>(a.V, w, [&](const uint4& v, int, float (&x)[VE]) {
      grad_window<DT, false, decltype(usual)::value>(v, g, x);
    });
  };
  if (g.usual)
    walk(std::true_type{});
  else
    walk(std::false_type{});

  __syncthreads();  // seen and flags are clear, the dense terms stored
  if (tid < a.K) keep_entry(tid, e);
  __syncthreads();
  const int flag = flags;
  if ((flag & kNan) || !(flag & kAny)) {  // a weight without a value; no teacher's distribution
    ch.fill(a.V, w, (flag & kNan) ? NAN : 0.0f);
    return;
  }
  auto* const out = ch.out + window_first<DT>(ch.first, ch.off);
  for (int k = tid; k < a.K; k += NT) {
    const int at = pos[k];
    if (at < 0) continue;
    float sum = ws[k];
    bool is_first = true;
    if (flag & kTwice) {  // the first entry of a token adds up the weights, in entry order
      sum = 0.f;
      for (int j = 0; j < a.K; ++j)
        if (pos[j] == at) {
          is_first = is_first && j >= k;
          sum += ws[j];
        }
    }
    if (is_first)
      out[at] = E::from_f32(fmaf(ex2((zs[k] - st.x) * a.c), A, -at_entry * sum));
  }
}

// ------------------------------------------------------------------------------ launches

namespace {

// Threads of a CTA: about eight windows each for short rows, so that one warp, which needs no
// barrier, does a row of 1000 16-bit logits.
int row_threads(int V, int vec) {
  const int windows = (V + vec - 1) / vec;
  return windows <= 256 ? 32 : windows <= 2048 ? 128 : 256;
}

// CTAs per row: one while the rows alone fill the device; for few rows a cluster of up to eight
// shares each (every CTA keeping at least one round of windows).
int row_ranks(int64_t T, int V, int vec, int threads) {
  const int64_t want = 2 * static_cast<int64_t>(device_sm_count());
  int r = 1;
  while (r < 8 && T * r < want &&
         static_cast<int64_t>(V) / (2 * r) >= static_cast<int64_t>(vec) * threads)
    r *= 2;
  return r;
}

template <typename... A>
int launch_rows(void (*kernel)(A...), int64_t grid, int threads, int ranks, size_t smem,
                cudaStream_t s, const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a...);
  note_launches(1);
  return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

// f(threads as a constant).
template <typename F>
int by_threads(int threads, F&& f) {
  using std::integral_constant;
  return threads == 32    ? f(integral_constant<int, 32>{})
         : threads == 128 ? f(integral_constant<int, 128>{})
                          : f(integral_constant<int, 256>{});
}

// Launches a kernel of a cluster per row, in two parts where few rows are left over after full rounds
// of `ctas` CTAs an SM and a row is long (from 128 KB): 66 -> 61 us for T=1500, V=100003 bf16 with 5
// alternatives, but 51 -> 54 us for T=3000, V=30000. Few are up to a quarter of a round: in one launch
// and in two, for 1/32, 1/8, 1/4, 3/8 and 1/2 of a round left over after one round of V=131072 bf16
// 59 and 47, 61 and 51, 64 and 59, 68 and 68, 72 and 72 us; after three rounds 125 and 119, 127 and
// 121, 131 and 127, 133 and 135, 137 and 137 us; after one round of V=66001 35 and 31, 37 and 33, 41
// and 37, 41 and 41, 43 and 43 us.
template <typename A>
int launch_split(void (*kernel)(A), int64_t T, int vec, int threads, int ctas, size_t smem,
                 cudaStream_t s, A a) {
  const int64_t round = static_cast<int64_t>(device_sm_count()) * ctas;
  const int64_t left = T % round;
  const bool split = threads == 256 && a.V / vec >= 8192 && T > round && left > 0 &&
                     left * 4 <= round;
  const int64_t rows = split ? T - left : T;
  a.first = 0, a.tail = false;
  a.ranks = row_ranks(rows, a.V, vec, threads);
  const int st = launch_rows(kernel, rows * a.ranks, threads, a.ranks, smem, s, a);
  if (!split || st != MHC_OK) return st;
  a.first = rows, a.tail = true;
  a.ranks = row_ranks(left, a.V, vec, threads);
  return launch_rows(kernel, left * a.ranks, threads, a.ranks, smem, s, a);
}

template <int DT>
int launch_logprob(const LogprobArgs& a, int64_t T, cudaStream_t s) {
  const int threads = row_threads(a.V, Elem<DT>::kVec);
  return by_threads(threads, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    auto kernel = a.entropy ? (a.K > 0 ? logprob_kernel<DT, NT, true, true>
                                       : logprob_kernel<DT, NT, true, false>)
                            : (a.K > 0 ? logprob_kernel<DT, NT, false, true>
                                       : logprob_kernel<DT, NT, false, false>);
    return launch_split(kernel, T, Elem<DT>::kVec, NT, logprob_ctas(NT, a.K > 0), 0, s, a);
  });
}

template <int DT>
int launch_distill(const DistillArgs& a, int64_t T, cudaStream_t s) {
  const int threads = row_threads(a.V, Elem<DT>::kVec);
  return by_threads(threads, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    return launch_split(distill_kernel<DT, NT>, T, Elem<DT>::kVec, NT, logprob_ctas(NT, false),
                        static_cast<size_t>(a.K) * 8, s, a);
  });
}

template <int DT>
int launch_logit_grad(LogitGradArgs a, int64_t T, bool distill, cudaStream_t s) {
  // Windows of a row: one more than fill it where rows may begin anywhere in their first.
  constexpr int VE = Elem<DT>::kVec;
  const bool whole = aligned16(a.logits) && a.stride % VE == 0;
  const int windows = (a.V + (whole ? VE - 1 : 2 * VE - 2)) / VE;
  const int threads = windows <= 256 ? 32 : windows <= 1024 ? 128 : 256;
  const int chunk = threads * kLgUnroll * kLgRounds;
  a.chunks = (windows + chunk - 1) / chunk;
  const int64_t items = T * a.chunks;
  if (items > (int64_t(1) << 31) - 1) return MHC_ERR_INVALID_ARG;
  return by_threads(threads, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    auto kernel = distill       ? distill_grad_kernel<DT, NT>
                  : a.d_entropy ? logprob_grad_kernel<DT, NT, true>
                                : logprob_grad_kernel<DT, NT, false>;
    return launch_rows(kernel, items, NT, 1, distill ? static_cast<size_t>(a.K) * 12 : 0, s, a);
  });
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
                      exponent_scale(temperature), 1.0f / temperature, static_cast<int>(V), top, 1, 0, false};
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
                      static_cast<int>(K), 1, teacher_dtype, 0, false};
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
