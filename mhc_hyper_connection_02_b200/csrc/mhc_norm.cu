// Layer norm of rows (the layer input y a pre-map emits, the row a head emits) and its backward pass
// with the weights' gradients.
//
//   mean = sum(x) / H, var = sum((x - mean)^2) / H, rstd = 1 / sqrt(var + eps)
//   y    = (x - mean) * rstd * gamma + beta
//   xh   = (x - mean) * rstd, q = d_y * gamma
//   d_x  = rstd * (q - sum(q) / H - xh * sum(q * xh) / H)
//   d_gamma = sum_t d_y * xh, d_beta = sum_t d_y
//
// The variance is formed from the differences to the mean (a second walk over the row), not from
// sum(x^2) - mean^2, which loses every digit where |mean| is large against the deviation. All sums
// and statistics are fp32; y and d_x are rounded once. Sums over tokens are in a fixed order: each
// group of a CTA adds its tokens in order, the CTA its groups into a partial row of the workspace, and
// a second kernel adds the partial rows in order.
#include <math.h>

#include <initializer_list>

#include "mhc.h"
#include "mhc_internal.h"
#include "mhc_rows.cuh"
#include "mhc_rows_host.h"

namespace mhc {

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* gamma;  // or null: ones
  const void* beta;   // or null: zeros
  void* y;            // [T][H]
  float* mean;        // or null
  float* rstd;        // or null
  int64_t T;
  int H;
  float eps;
};

struct NormBwdArgs {
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* gamma;  // or null: ones
  const float* mean;
  const float* rstd;
  void* dx;           // [T][H]
  float* part;        // [blocks][2][H]: d_gamma, d_beta partial rows
  int64_t T;
  int H;
};

// ------------------------------------------------------------------------------ rows in registers
//
// A group of G threads holds a row: thread i of it the accesses i, i + G, ..., N of them, of VW
// elements each (16 bytes, or one element where the row's width, stride or address does not allow
// more). The row is read once; mean, variance and output come from the registers.

// Access of VW elements: 16 bytes kept packed until used, or one element.
template <int DT, int VW>
struct Chunk {
  using E = Elem<DT>;
  using raw = typename E::raw;
  typename std::conditional<VW == 1, raw, uint4>::type v;
  __device__ __forceinline__ void load(const raw* p) {
    if constexpr (VW == 1) v = *p; else v = ld_stream(p);
  }
  __device__ __forceinline__ void get(float (&x)[VW]) const {
    if constexpr (VW == 1) x[0] = E::to_f32(v); else E::unpack(v, x);
  }
  static __device__ __forceinline__ void put(raw* p, const float (&x)[VW]) {
    if constexpr (VW == 1) *p = E::from_f32(x[0]); else st_stream(p, E::pack(x));
  }
};

// VW weights at p (of the rows' type or fp32), through L1. wide: p is 32-byte aligned; eight fp32
// weights then come in one access (two of 16 bytes each touch every sector of the warp's span, which
// made the weights' L1 traffic the forward pass's bound).
template <int WT, int VW>
__device__ __forceinline__ void load_weights(const typename Elem<WT>::raw* p, bool wide,
                                             float (&g)[VW]) {
  using W = Elem<WT>;
  if constexpr (VW == 1) {
    g[0] = W::to_f32(__ldg(p));
  } else {
    if constexpr (WT == 2 && VW == 8) {
      if (wide) {
        asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(g[0]), "=f"(g[1]), "=f"(g[2]), "=f"(g[3]), "=f"(g[4]), "=f"(g[5]),
                       "=f"(g[6]), "=f"(g[7])
                     : "l"(p));
        return;
      }
    }
#pragma unroll
    for (int q = 0; q < VW; q += W::kVec) {
      float x[W::kVec];
      W::unpack(__ldg(reinterpret_cast<const uint4*>(p + q)), x);
#pragma unroll
      for (int k = 0; k < W::kVec; ++k) g[q + k] = x[k];
    }
  }
}
__device__ __forceinline__ bool aligned32(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

constexpr int kNormWarpRows = 4;  // rows per CTA of the one-warp-per-row forward form

// Forward. kWarp: a warp per K rows, no barrier; otherwise a CTA (G = blockDim.x threads) per K
// rows. Two rows at a time read the weights once and share each exchange between threads.
template <int DT, int WT, int VW, int N, int K, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kNormWarpRows : K == 2 ? 512 : 1024) norm_row_kernel(
    const NormArgs a) {
  using W = Elem<WT>;
  using C = Chunk<DT, VW>;
  using raw = typename C::raw;
  static_assert(K == 1 || K == 2, "one or two rows at a time");
  __shared__ float red[2][64];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = kWarp ? 32 : blockDim.x, tid = kWarp ? lane : threadIdx.x;
  const int64_t t0 =
      K * (kWarp ? blockIdx.x * int64_t(kNormWarpRows) + warp : static_cast<int64_t>(blockIdx.x));
  if (kWarp && t0 >= a.T) return;
  const int rows = K == 2 && t0 + 1 < a.T ? 2 : 1;
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  const auto* beta = static_cast<const typename W::raw*>(a.beta);
  const bool gw = aligned32(gamma), bw = aligned32(beta);
  const raw* x = static_cast<const raw*>(a.x) + t0 * a.x_stride;  // may be y: coherent loads
  raw* y = static_cast<raw*>(a.y) + t0 * a.H;
  const float fh = static_cast<float>(a.H);  // divided by: exact for rows of one value

  // Sums over the group, the same bits in every thread.
  auto total = [&](const float (&v)[K], int turn, float (&out)[K]) {
    if constexpr (K == 1) {
      out[0] = warp_sum(v[0]);
      if constexpr (!kWarp) {
        if (lane == 0) red[turn][warp] = out[0];
        __syncthreads();
        out[0] = warp_sum(lane < (G >> 5) ? red[turn][lane] : 0.0f);
      }
    } else {
      const float h = warp_sum_halves(v[0], v[1]);
      float2 p;
      if constexpr (kWarp) {
        p = join_halves(h);
      } else {
        if ((lane & 15) == 0) red[turn][2 * lane + warp] = h;
        __syncthreads();
        p = sum_of_warps(red[turn], G >> 5);
      }
      out[0] = p.x, out[1] = p.y;
    }
  };

  C c[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = (i * G + tid) * VW;
      if (h < a.H && k < rows) c[k][i].load(x + k * a.x_stride + h);
    }
  float s[K], mean[K], v[K], rstd[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    s[k] = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i * G + tid) * VW < a.H && k < rows) {
        float f[VW];
        c[k][i].get(f);
#pragma unroll
        for (int q = 0; q < VW; ++q) s[k] += f[q];
      }
  }
  total(s, 0, mean);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    mean[k] /= fh;
    v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i * G + tid) * VW < a.H && k < rows) {
        float f[VW];
        c[k][i].get(f);
#pragma unroll
        for (int q = 0; q < VW; ++q) {
          const float d = f[q] - mean[k];
          v[k] = fmaf(d, d, v[k]);
        }
      }
  }
  total(v, 1, rstd);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    rstd[k] = 1.0f / sqrtf(rstd[k] / fh + a.eps);
    if (tid == 0 && k < rows) {
      if (a.mean) a.mean[t0 + k] = mean[k];
      if (a.rstd) a.rstd[t0 + k] = rstd[k];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = (i * G + tid) * VW;
    if (h < a.H) {
      float g[VW], b[VW];
#pragma unroll
      for (int q = 0; q < VW; ++q) g[q] = 1.0f, b[q] = 0.0f;
      if (gamma) load_weights<WT, VW>(gamma + h, gw, g);
      if (beta) load_weights<WT, VW>(beta + h, bw, b);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k < rows) {
          float f[VW];
          c[k][i].get(f);
#pragma unroll
          for (int q = 0; q < VW; ++q) f[q] = fmaf((f[q] - mean[k]) * rstd[k], g[q], b[q]);
          C::put(y + k * static_cast<int64_t>(a.H) + h, f);
        }
    }
  }
}

// to[c] = the sum of sums[j n + c] over the groups j, in order (n floats each).
__device__ __forceinline__ void add_groups(const float* sums, int R, int n, float* to) {
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    float v = sums[c];
    for (int j = 1; j < R; ++j) v += sums[static_cast<size_t>(j) * n + c];
    to[c] = v;
  }
}

// ------------------------------------------------------------------------------ staged rows
//
// Rows of one or two arrays (x; x and d_y) staged in shared memory by 1-D bulk copies, K tokens to a
// stage; a group of G threads has S stages of its own and works on one at a time, and the barrier of
// its exchange of sums also tells its first warp that a stage has been read and takes the next copy.
//
// Rows that are not whole 16-byte windows (odd widths, strides or addresses): where a row begins in
// its first window (its phase) repeats every kVec tokens, so a CTA takes tokens of one class t mod
// kVec only. Then every row of an array has the same phase there, columns stay with their threads,
// and all accesses are whole windows. The output's phase sets the windows; an input of another phase
// (a gap between its rows) is read as two windows and shifted. The copies take whole windows too:
// what they read beside a row belongs to the rows before and after it (or the gap between) and is
// not used; only before the first token's row and behind the last one's, where the array ends, the
// row's own elements are read one by one.
constexpr int kStagesEach = 4;  // of a group, at most
template <int DT, int A, int K, bool kAligned>
struct RowRing {
  using E = Elem<DT>;
  using raw = typename E::raw;
  static constexpr int VE = E::kVec;
  const raw* base[A];
  int64_t stride[A];
  int off[A];         // phase of the class's rows
  int shift[A];       // against the output's phase
  // Tokens are below 2^31; a few stages beyond the last still fit 32 bits.
  uint32_t T;            // tokens of the class
  int64_t tokens;        // of all
  uint32_t first, step;  // in the class: the group's first, and from one stage to its next
  int H, classes, cls;
  int slot;           // windows of a row in a stage
  int n;              // windows of an output row
  uint4* masks;       // of the first and of the last one: the row's elements
  uint8_t* stages;
  uint64_t* full;
  float* stats;       // per stage: K pairs of mean and rstd (A = 2)
  const float* mean;  // of the class's tokens
  const float* rstd;
  int S;

  // Windows of a slot: those a row of n elements touches and, unaligned, one before and one after.
  static __host__ __device__ __forceinline__ int slot_windows(int n) {
    return kAligned ? n / VE : (n + 2 * VE - 2) / VE + 2;
  }
  __device__ __forceinline__ void init(int64_t all, int h, int C, int groups, int group,
                                       int stages_each, uint8_t* memory, uint64_t* bars,
                                       float* pairs = nullptr, const float* means = nullptr,
                                       const float* rstds = nullptr) {
    classes = kAligned ? 1 : C;
    cls = blockIdx.x % classes;
    const int rank = blockIdx.x / classes, ranks = gridDim.x / classes;
    tokens = all;
    T = static_cast<uint32_t>((tokens - cls + classes - 1) / classes);
    first = (group * ranks + rank) * K;
    step = ranks * K * groups;
    H = h, S = stages_each;
    slot = slot_windows(h);
    stages = memory + static_cast<size_t>(group * S) * stage_bytes();
    full = bars + group * S;
    if constexpr (A == 2) {
      stats = pairs + group * S * 2 * K;
      mean = means + cls, rstd = rstds + cls;
    }
  }
  // By one thread, before anything is copied.
  static __device__ __forceinline__ void init_barriers(uint64_t* bars, int n) {
    for (int i = 0; i < n; ++i) mbar_init(&bars[i], A);  // bulk copies; A = 2: and the statistics
    fence_mbarrier_init();
  }
  __device__ __forceinline__ void array(int i, const void* p, int64_t st, int out_off) {
    base[i] = static_cast<const raw*>(p) + cls * st;
    stride[i] = st * classes;
    off[i] = kAligned ? 0 : window_offset<DT>(base[i]);
    shift[i] = off[i] - out_off;
  }
  // The output's windows, for phase out_off; by all threads, before the CTA's next barrier.
  __device__ __forceinline__ void output(int out_off, uint4* two_masks) {
    n = kAligned ? H / VE : window_count<DT>(out_off, H);
    masks = two_masks;
    if (!kAligned && threadIdx.x < 2 * VE) {
      const int which = threadIdx.x / VE, q = threadIdx.x % VE;
      const int e = (which == 0 ? 0 : n - 1) * VE - out_off + q;
      reinterpret_cast<typename std::conditional<DT == 2, uint32_t, raw>::type*>(masks)[threadIdx.x] =
          e >= 0 && e < H ? ~0u : 0u;
    }
  }
  __device__ __forceinline__ int64_t token(uint32_t j) const {
    return cls + static_cast<int64_t>(j) * classes;
  }
  __device__ __forceinline__ int stage_bytes() const { return A * K * slot * 16; }
  __device__ __forceinline__ int rows(uint32_t j) const {
    return j + K <= T ? K : static_cast<int>(T - j);
  }
  __device__ __forceinline__ uint4* slot_at(int st, int r, int i) const {
    return reinterpret_cast<uint4*>(stages + static_cast<size_t>(st) * stage_bytes()) +
           (r * A + i) * slot;
  }

  // Starts the copy of the tokens j .. into a stage (one thread; shared out over the group's warps it
  // took 5 % longer), their statistics along with it. A stage that the class's last token does not
  // fill gets that token again.
  __device__ __forceinline__ void copy(int st, uint32_t j) const {
    // Rows where an array begins or ends: at either end of the class at most.
    if (!kAligned && (j == 0 || j + K >= T) &&
        (token(j) == 0 || token(min(j + K - 1, T - 1)) == tokens - 1)) {
      copy_ends(st, j);
    } else {
      uint32_t bytes = 0;
#pragma unroll
      for (int i = 0; i < A; ++i) bytes += windows(i);
      mbar_arrive_expect_tx(&full[st], bytes * (K * 16));
#pragma unroll
      for (int r = 0; r < K; ++r)
#pragma unroll
        for (int i = 0; i < A; ++i)
          bulk_g2s(slot_at(st, r, i) + (kAligned ? 0 : 1),
                   base[i] - off[i] + static_cast<int64_t>(min(j + r, T - 1)) * stride[i],
                   windows(i) * 16, &full[st]);
    }
    if constexpr (A == 2) {
#pragma unroll
      for (int r = 0; r < K; ++r) {
        const int64_t t = static_cast<int64_t>(min(j + r, T - 1)) * classes;
        async_copy4(&stats[(st * K + r) * 2], mean + t);
        async_copy4(&stats[(st * K + r) * 2 + 1], rstd + t);
      }
      async_copies_arrive(&full[st]);
    }
  }
  __device__ __forceinline__ int windows(int i) const {
    return kAligned ? H / VE : (off[i] + H + VE - 1) / VE;
  }
  // The same with rows that an array begins or ends with: only the windows that such a row fills,
  // and its other elements one by one. Those are stored before the arrival, which releases them to
  // whoever waits on the stage, and the fence puts them before copies that overwrite them later.
  __device__ __noinline__ void copy_ends(int st, uint32_t j) const {
    for (int turn = 0; turn < 2; ++turn) {  // elements and the sum of bytes, then the copies
      uint32_t bytes = 0;
      for (int r = 0; r < K; ++r)
        for (int i = 0; i < A; ++i) {
          const uint32_t at = min(j + r, T - 1);
          const raw* row = base[i] + static_cast<int64_t>(at) * stride[i];
          const int64_t t = token(at);
          const int from = t == 0 && off[i] > 0 ? 1 : 0;
          const int to = t == tokens - 1 ? (off[i] + H) / VE : windows(i);
          uint4* slot_of = slot_at(st, r, i) + 1;
          if (turn == 0) {
            bytes += (to - from) * 16;
            raw* elements = reinterpret_cast<raw*>(slot_of) + off[i];
            if (from > 0)
              for (int e = 0; e < VE - off[i]; ++e) elements[e] = row[e];
            for (int e = to * VE - off[i]; e < H; ++e) elements[e] = row[e];
          } else {
            bulk_g2s(slot_of + from, row - off[i] + from * VE, (to - from) * 16, &full[st]);
          }
        }
      if (turn == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&full[st], bytes);
      }
    }
  }
  // The first S stages.
  __device__ __forceinline__ void start() const {
    for (int i = 0; i < S && first + i * step < T; ++i) copy(i, first + i * step);
  }

  // Output window s of row r of array i; what lies outside the row comes back as zero.
  __device__ __forceinline__ uint4 window(int st, int r, int i, int s) const {
    const uint4* p = slot_at(st, r, i) + s;
    if constexpr (kAligned) {
      return *p;
    } else {
      uint4 w;
      if (shift[i] == 0) {
        w = p[1];
      } else {
        const int by = (shift[i] & (VE - 1)) * static_cast<int>(sizeof(raw));  // bytes
        if (shift[i] > 0) ++p;
        const uint4 lo = p[0], hi = p[1];
        uint32_t v[6] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y};
        uint32_t u[5];
        if (by & 8) {
          v[0] = lo.z, v[1] = lo.w, v[2] = hi.x, v[3] = hi.y, v[4] = hi.z, v[5] = hi.w;
        }
#pragma unroll
        for (int q = 0; q < 5; ++q) u[q] = (by & 4) ? v[q + 1] : v[q];
        const int bits = (by & 3) * 8;
        w = make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits),
                       __funnelshift_r(u[2], u[3], bits), __funnelshift_r(u[3], u[4], bits));
      }
      if (s == 0 || s == n - 1) {
        const uint4 m = masks[s == 0 ? 0 : 1];
        w = make_uint4(w.x & m.x, w.y & m.y, w.z & m.z, w.w & m.w);
      }
      return w;
    }
  }

  // After a wait that gave up in stage st: no copy into this CTA's shared memory may outlive it.
  __device__ __forceinline__ void drain(int st, uint32_t lap, uint32_t j, int ahead) const {
    for (int i = 0; i < ahead && j + i * step < T; ++i) {
      mbar_drain(&full[st], lap & 1, 131);
      if (++st == S) st = 0, ++lap;
    }
  }
};

// One weight per element of the windows, in fp32 (zero outside the row), the first and the second
// four of each window apart, so that a warp's 16-byte reads meet no bank twice.
template <int VE, typename W>
__device__ __forceinline__ void stage_weights(float* to, const typename W::raw* w, float otherwise,
                                              int H, int off, int n) {
  constexpr int U = 8;  // loads in flight
  for (int i0 = threadIdx.x; i0 < n * VE; i0 += U * blockDim.x) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = i0 + u * blockDim.x - off;
      v[u] = h < 0 || h >= H ? 0.0f : w ? W::to_f32(__ldg(w + h)) : otherwise;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * blockDim.x;
      if (i < n * VE) to[((i % VE) / 4 * n + i / VE) * 4 + i % 4] = v[u];
    }
  }
}
template <int VE>
__device__ __forceinline__ void staged_weights(const float* from, int n, int s, F2 (&g)[VE / 2]) {
#pragma unroll
  for (int q = 0; q < VE; q += 4) {
    const float4 v = reinterpret_cast<const float4*>(from)[q / 4 * n + s];
    g[q / 2] = f2(v.x, v.y);
    g[q / 2 + 1] = f2(v.z, v.w);
  }
}
template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& w, F2 (&v)[Elem<DT>::kVec / 2]) {
  float f[Elem<DT>::kVec];
  Elem<DT>::unpack(w, f);
#pragma unroll
  for (int q = 0; q < Elem<DT>::kVec / 2; ++q) v[q] = f2(f[2 * q], f[2 * q + 1]);
}
// Windows' output: whole ones at once; of those at a row's ends the elements in the row, which end
// or begin with the window, in at most three parts of 1, 2 and 4 elements.
template <int DT, bool kAligned>
__device__ __forceinline__ void put_window(typename Elem<DT>::raw* row, int H, int e0,
                                           const F2 (&v)[Elem<DT>::kVec / 2]) {
  using E = Elem<DT>;
  using raw = typename E::raw;
  constexpr int VE = E::kVec;
  float o[VE];
#pragma unroll
  for (int q = 0; q < VE / 2; ++q) {
    const float2 u = split(v[q]);
    o[2 * q] = u.x, o[2 * q + 1] = u.y;
  }
  const uint4 w = E::pack(o);
  raw* const to = row + e0;
  if (kAligned || (e0 >= 0 && e0 + VE <= H)) {
    st_stream(to, w);
  } else if constexpr (DT == 2) {
    const uint32_t f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e0 + q >= 0 && e0 + q < H) to[q] = __uint_as_float(f[q]);
  } else if (e0 < 0) {  // the last c elements of the window
    const int c = VE + e0;
    if (c & 1) to[VE - c] = static_cast<raw>((c & 4 ? (c & 2 ? w.x : w.y) : (c & 2 ? w.z : w.w)) >> 16);
    if (c & 2) *reinterpret_cast<uint32_t*>(to + (c & 4 ? 2 : 6)) = c & 4 ? w.y : w.w;
    if (c & 4) *reinterpret_cast<uint2*>(to + 4) = make_uint2(w.z, w.w);
  } else {  // the first c
    const int c = H - e0;
    if (c & 4) *reinterpret_cast<uint2*>(to) = make_uint2(w.x, w.y);
    if (c & 2) *reinterpret_cast<uint32_t*>(to + (c & 4)) = c & 4 ? w.z : w.x;
    if (c & 1)
      to[c - 1] = static_cast<raw>((c & 4 ? (c & 2 ? w.w : w.z) : (c & 2 ? w.y : w.x)) & 0xffffu);
  }
}

constexpr int kRingStages = 64;    // of all groups, at most
constexpr int kRingThreads = 512;  // of all groups, at most

// Forward of many rows that are not whole windows. x is read once and stays packed in registers.
// T=8192, H=3501 bf16: 43 us (2.6 TB/s), element by element 80 us; bound by the instructions of a
// group's warps, of which an SM holds 16.
template <int DT, int WT, int N, int K>
__global__ void __launch_bounds__(kRingThreads) norm_ring_kernel(const NormArgs a, int G, int R, int S,
                                                        int C) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  using raw = typename E::raw;
  constexpr int VE = E::kVec, P = VE / 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRingStages];
  __shared__ float red[2][2 * 32];
  const int warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  __shared__ uint4 masks[2];
  using Ring = RowRing<DT, 1, K, false>;
  __shared__ Ring plans[kRingThreads / 32];  // for the groups' copying threads: few registers
  if (threadIdx.x == 0) Ring::init_barriers(full, R * S);
  Ring rr;
  rr.init(a.T, a.H, C, R, group, S, ring, full);
  raw* const y0 = static_cast<raw*>(a.y) + static_cast<int64_t>(rr.cls) * a.H;
  const int off = window_offset<DT>(y0);
  rr.output(off, masks);
  const int n = rr.n;
  rr.array(0, a.x, a.x_stride, off);
  Ring& plan = plans[group];
  if (tid == 0) plan = rr;
  float* const gs = reinterpret_cast<float*>(ring + static_cast<size_t>(R * S) * rr.stage_bytes());
  float* const bs = gs + n * VE;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int nw = G >> 5, w0 = group * nw;
  if (tid == 0) plan.start();
  stage_weights<VE, W>(gs, static_cast<const typename W::raw*>(a.gamma), 1.0f, a.H, off, n);
  stage_weights<VE, W>(bs, static_cast<const typename W::raw*>(a.beta), 0.0f, a.H, off, n);
  __syncthreads();

  const float fh = static_cast<float>(a.H);
  int turn = 0;
  bool ok = true;
  auto total = [&](const float (&v)[K], float (&out)[K]) {  // over the group, which agrees on ok
    float sums[2] = {v[0], K == 2 ? v[K - 1] : 0.0f};
    const float part = warp_sums<2>(sums);
    if (G == 32) {
      ok = __all_sync(0xffffffffu, ok);
      share_sums<2>(part, sums);
    } else {
      put_warp_sums<2>(part, red[turn], warp);
      ok = !named_bar_or(group + 1, G, !ok);
      joined_sums<2>(red[turn], w0, nw, sums);
      turn ^= 1;
    }
    out[0] = sums[0];
    if (K == 2) out[K - 1] = sums[1];
  };
  int st = 0;
  uint32_t lap = 0;
  uint32_t j = rr.first;
  for (; j < rr.T; j += rr.step) {
    const int rows = rr.rows(j);
    ok = mbar_wait(&rr.full[st], lap & 1, 132);
    uint4 h[K][N];
    float s[K], mean[K], v[K], rstd[K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      F2 sum = f2(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = i * G + tid;
        h[r][i] = at < n ? rr.window(st, r, 0, at) : make_uint4(0, 0, 0, 0);
        F2 x[P];
        unpack_pairs<DT>(h[r][i], x);
#pragma unroll
        for (int q = 0; q < P; ++q) sum = sum + x[q];
      }
      const float2 u = split(sum);
      s[r] = u.x + u.y;
    }
    total(s, mean);
    if (!ok) break;
    if (G == 32) __syncwarp();
    if (tid == 0 && j + S * rr.step < rr.T) plan.copy(st, j + S * rr.step);
#pragma unroll
    for (int r = 0; r < K; ++r) {
      mean[r] /= fh;
      F2 sum = f2(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = i * G + tid, e0 = at * VE - off;
        if (at < n) {
          F2 x[P];
          unpack_pairs<DT>(h[r][i], x);
          if (e0 >= 0 && e0 + VE <= a.H) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
              const F2 d = x[q] + f2(-mean[r]);
              sum = fma2(d, d, sum);
            }
          } else {
#pragma unroll
            for (int q = 0; q < P; ++q) {
              const float2 u = split(x[q]);
              const int e = e0 + 2 * q;
              const F2 d = f2(e >= 0 && e < a.H ? u.x - mean[r] : 0.0f,
                              e + 1 >= 0 && e + 1 < a.H ? u.y - mean[r] : 0.0f);
              sum = fma2(d, d, sum);
            }
          }
        }
      }
      const float2 u = split(sum);
      v[r] = u.x + u.y;
    }
    total(v, rstd);
#pragma unroll
    for (int r = 0; r < K; ++r) {
      rstd[r] = 1.0f / sqrtf(rstd[r] / fh + a.eps);
      if (tid == 0 && r < rows) {
        const int64_t t = rr.token(j + r);
        if (a.mean) a.mean[t] = mean[r];
        if (a.rstd) a.rstd[t] = rstd[r];
      }
    }
    raw* const y = y0 + static_cast<int64_t>(j) * rr.classes * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 g[P], b[P];
        staged_weights<VE>(gs, n, at, g);
        staged_weights<VE>(bs, n, at, b);
#pragma unroll
        for (int r = 0; r < K; ++r) {
          if (r >= rows) break;
          F2 x[P];
          unpack_pairs<DT>(h[r][i], x);
#pragma unroll
          for (int q = 0; q < P; ++q)
            x[q] = fma2((x[q] + f2(-mean[r])) * f2(rstd[r]), g[q], b[q]);
          put_window<DT, false>(y + static_cast<int64_t>(r) * rr.classes * a.H, a.H, at * VE - off, x);
        }
      }
    }
    if (++st == S) st = 0, ++lap;
  }
  if (!ok && tid == 0) plan.drain(st, lap, j, S);
}

// Backward. A group reads the rows of a stage once (kHold: they stay packed in its registers) or
// twice, and exchanges the sums of K tokens at once. Each thread keeps its columns' gradient sums in
// registers over all its tokens: 16 columns at 512 threads an SM, which is what they and two held
// rows leave room for; with 8 columns at 1024 threads each warp's exchange costs as much for half the
// work (T=8192, H=7168 bf16: 110 us, where this form took 87 us before its later steps). All waits
// are bounded, and a group leaves its loop together.
//
// Now 68.5 us, 5.1 TB/s and 78 % of the copy rate; H=3501 57 us. The copies alone take 40 us: what
// bounds the pass is the latency of a warp's instructions (14 warps an SM, 46 % of issue slots used).
template <int DT, int WT, int N, int K, bool kHold, bool kAligned>
__global__ void __launch_bounds__(kRingThreads) norm_bwd_ring_kernel(const NormBwdArgs a, int G, int R,
                                                            int S, int C) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  using raw = typename E::raw;
  constexpr int VE = E::kVec, P = VE / 2;  // elements and pairs of a window
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRingStages];
  __shared__ float red[2][2 * K * 32];  // by turn: each warp's sums (joined_sums)
  const int warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  __shared__ __align__(8) float stats[kRingStages * 2 * K];
  __shared__ uint4 masks[2];
  using Ring = RowRing<DT, 2, K, kAligned>;
  // Unaligned, the groups' copying threads keep what they need here: few registers are free.
  __shared__ Ring plans[kAligned ? 1 : kRingThreads / 32];
  if (threadIdx.x == 0) Ring::init_barriers(full, R * S);
  Ring rr;
  rr.init(a.T, a.H, C, R, group, S, ring, full, stats, a.mean, a.rstd);
  raw* const dx0 = static_cast<raw*>(a.dx) + static_cast<int64_t>(rr.cls) * a.H;
  const int off = kAligned ? 0 : window_offset<DT>(dx0);
  rr.output(off, masks);
  const int n = rr.n;
  rr.array(0, a.x, a.x_stride, off);
  rr.array(1, a.dy, a.dy_stride, off);
  if (!kAligned && tid == 0) plans[group] = rr;
  auto plan = [&]() -> const Ring& {
    if constexpr (kAligned)
      return rr;
    else
      return plans[group];
  };
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int nw = G >> 5, w0 = group * nw;
  if (tid == 0) plan().start();
  // gamma: in registers, where they have room for it, or behind the stages.
  constexpr bool kOwn = kHold && kAligned;
  const auto* const gamma = static_cast<const typename W::raw*>(a.gamma);
  float* const gs = reinterpret_cast<float*>(ring + static_cast<size_t>(R * S) * rr.stage_bytes());
  [[maybe_unused]] F2 own[kOwn ? N : 1][P];
  if constexpr (kOwn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const int h = (i * G + tid) * VE + q;
        v[q] = h >= a.H ? 0.0f : gamma ? W::to_f32(__ldg(gamma + h)) : 1.0f;
      }
#pragma unroll
      for (int q = 0; q < P; ++q) own[i][q] = f2(v[2 * q], v[2 * q + 1]);
    }
  } else {
    stage_weights<VE, W>(gs, gamma, 1.0f, a.H, off, n);
  }
  auto weights = [&](int i, int at, F2 (&g)[P]) {
    if constexpr (kOwn) {
#pragma unroll
      for (int q = 0; q < P; ++q) g[q] = own[i][q];
    } else {
      staged_weights<VE>(gs, n, at, g);
    }
  };
  __syncthreads();
  constexpr int lag = kHold ? 0 : 1;  // the stage to copy into was read that many iterations ago

  const float per_h = 1.0f / static_cast<float>(a.H);
  F2 dg[N][P], db[N][P];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < P; ++q) dg[i][q] = f2(0.0f), db[i][q] = f2(0.0f);
  raw* dx = dx0 + static_cast<int64_t>(rr.first) * rr.classes * a.H;
  const int64_t dx_step = static_cast<int64_t>(rr.step) * rr.classes * a.H;
  int st = 0, turn = 0;
  uint32_t lap = 0;
  bool ok = true;
  uint32_t j = rr.first;
  for (; j < rr.T; j += rr.step, turn ^= 1) {
    const int rows = rr.rows(j);
    ok = mbar_wait(&rr.full[st], lap & 1, 130);
    F2 nm[K], fr[K];
    float rs[K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      const float2 v = reinterpret_cast<const float2*>(rr.stats)[st * K + r];
      nm[r] = f2(-v.x);
      rs[r] = v.y;
      fr[r] = f2(rs[r]);
    }
    const bool whole = K == 1 || rows == K;  // else the last row is there twice
    uint4 hx[K][N], hd[K][N];
    if constexpr (kHold) {
#pragma unroll
      for (int r = 0; r < K; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int at = i * G + tid;
          if (at < n) {
            hx[r][i] = rr.window(st, r, 0, at);
            hd[r][i] = rr.window(st, r, 1, at);
            if (r > 0 && !whole) hx[r][i] = hd[r][i] = make_uint4(0, 0, 0, 0);
          }
        }
    }
    F2 s1[K], s2[K];
#pragma unroll
    for (int r = 0; r < K; ++r) s1[r] = s2[r] = f2(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 g[P];
        weights(i, at, g);
#pragma unroll
        for (int r = 0; r < K; ++r) {
          F2 x[P], d[P];
          unpack_pairs<DT>(kHold ? hx[r][i] : rr.window(st, r, 0, at), x);
          unpack_pairs<DT>(kHold ? hd[r][i] : rr.window(st, r, 1, at), d);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const F2 u = d[q] * (x[q] + nm[r]);
            dg[i][q] = fma2(u, fr[r], dg[i][q]);
            db[i][q] = db[i][q] + d[q];
            s1[r] = fma2(d[q], g[q], s1[r]);
            s2[r] = fma2(u, g[q], s2[r]);  // sum(q (x - mean))
          }
        }
      }
    }
    float sums[2 * K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      const float2 u1 = split(s1[r]), u2 = split(s2[r]);
      sums[2 * r] = u1.x + u1.y;
      sums[2 * r + 1] = u2.x + u2.y;
    }
    const float part = warp_sums<2 * K>(sums);
    if (G == 32) {
      ok = __all_sync(0xffffffffu, ok);
      share_sums<2 * K>(part, sums);
    } else {
      put_warp_sums<2 * K>(part, red[turn], warp);
      ok = !named_bar_or(group + 1, G, !ok);
      joined_sums<2 * K>(red[turn], w0, nw, sums);
    }
    if (!ok) break;
    // Every thread has read this stage (kHold), or the one before for the last time.
    const uint32_t next = j + (S - lag) * rr.step;
    if (G == 32) __syncwarp();
    if (tid == 0 && (kHold || lap + st > 0) && next < rr.T)
      plan().copy(kHold ? st : st > 0 ? st - 1 : S - 1, next);
    // d_x = r d_y gamma - r c1 - (x - mean) r^2 c2 = r (d_y gamma) + ((x - mean) f + f0). x - mean is
    // formed first for every type: taken into f0 the mean's part would be off by 2^-24 |mean| r of
    // the last term, and a 16-bit row can have |mean| r above 10^4 (few values a step from the rest).
    F2 f0[K], fx[K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      const float f = -rs[r] * rs[r] * (rs[r] * sums[2 * r + 1] * per_h);
      fx[r] = f2(f);
      f0[r] = f2(-rs[r] * (sums[2 * r] * per_h));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 g[P];
        weights(i, at, g);
#pragma unroll
        for (int r = 0; r < K; ++r) {
          if (r > 0 && !whole) break;
          F2 x[P], d[P];
          unpack_pairs<DT>(kHold ? hx[r][i] : rr.window(st, r, 0, at), x);
          unpack_pairs<DT>(kHold ? hd[r][i] : rr.window(st, r, 1, at), d);
#pragma unroll
          for (int q = 0; q < P; ++q)
            x[q] = fma2(d[q] * g[q], fr[r], fma2(x[q] + nm[r], fx[r], f0[r]));
          put_window<DT, kAligned>(dx + static_cast<int64_t>(r) * rr.classes * a.H, a.H,
                                   at * VE - off, x);
        }
      }
    }
    dx += dx_step;
    if (++st == S) st = 0, ++lap;
  }
  // Stages with a copy, from the current one on (the first pass of !kHold has them all).
  if (!ok && tid == 0) plan().drain(st, lap, j, kHold || lap + st == 0 ? S : S - 1);
  if (!a.part) return;
  // The groups' sums, through the stages' memory (free: every group is done).
  __syncthreads();
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  float* to = R > 1 ? reinterpret_cast<float*>(ring) + static_cast<size_t>(group) * (2 * a.H) : part;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = i * G + tid, e0 = at * VE - off;
    if (at < n) {
      if (kAligned) {
#pragma unroll
        for (int q = 0; q < P; q += 2) {
          const float2 lo = split(dg[i][q]), hi = split(dg[i][q + 1]);
          *reinterpret_cast<float4*>(to + e0 + 2 * q) = make_float4(lo.x, lo.y, hi.x, hi.y);
          const float2 lb = split(db[i][q]), hb = split(db[i][q + 1]);
          *reinterpret_cast<float4*>(to + a.H + e0 + 2 * q) = make_float4(lb.x, lb.y, hb.x, hb.y);
        }
      } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
          const float2 u = split(dg[i][q]), v = split(db[i][q]);
          const int e = e0 + 2 * q;
          if (e >= 0 && e < a.H) to[e] = u.x, to[a.H + e] = v.x;
          if (e + 1 >= 0 && e + 1 < a.H) to[e + 1] = u.y, to[a.H + e + 1] = v.y;
        }
      }
    }
  }
  if (R == 1) return;
  __syncthreads();
  add_groups(reinterpret_cast<const float*>(ring), R, 2 * a.H, part);
}

// ------------------------------------------------------------------------------ any row

constexpr int kNormThreads = 256;

// Any H, stride and alignment: one CTA per row, three walks over the row (the second and third
// from L1 / L2).
template <int DT, int WT>
__global__ void __launch_bounds__(kNormThreads) norm_loop_kernel(const NormArgs a) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  __shared__ float red[kNormThreads / 32];
  pdl_wait();
  pdl_trigger();
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  const auto* beta = static_cast<const typename W::raw*>(a.beta);
  const float fh = static_cast<float>(a.H);  // divided by: exact for rows of one value
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    // x may be y (in place): plain loads, each element read by the thread that writes it.
    const auto* x = static_cast<const typename E::raw*>(a.x) + t * a.x_stride;
    auto* y = static_cast<typename E::raw*>(a.y) + t * a.H;
    float s = 0.f;
    for (int h = threadIdx.x; h < a.H; h += kNormThreads) s += E::to_f32(x[h]);
    const float mean = block_sum<kNormThreads>(s, red) / fh;
    float v = 0.f;
    for (int h = threadIdx.x; h < a.H; h += kNormThreads) {
      const float d = E::to_f32(x[h]) - mean;
      v = fmaf(d, d, v);
    }
    const float rstd = 1.0f / sqrtf(block_sum<kNormThreads>(v, red) / fh + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[t] = mean;
      if (a.rstd) a.rstd[t] = rstd;
    }
    for (int h = threadIdx.x; h < a.H; h += kNormThreads) {
      const float g = gamma ? W::to_f32(gamma[h]) : 1.0f;
      const float b = beta ? W::to_f32(beta[h]) : 0.0f;
      y[h] = E::from_f32(fmaf((E::to_f32(x[h]) - mean) * rstd, g, b));
    }
  }
}

template <int DT, int WT>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_dx_loop_kernel(const NormBwdArgs a) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  __shared__ float red[2 * kNormThreads / 32];
  pdl_wait();
  pdl_trigger();
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  const float fh = static_cast<float>(a.H);  // divided by: exact for rows of one value
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const auto* x = static_cast<const typename E::raw*>(a.x) + t * a.x_stride;
    const auto* dy = static_cast<const typename E::raw*>(a.dy) + t * a.dy_stride;
    auto* dx = static_cast<typename E::raw*>(a.dx) + t * a.H;
    const float mean = a.mean[t], rstd = a.rstd[t];
    float s1 = 0.f, s2 = 0.f;
    for (int h = threadIdx.x; h < a.H; h += kNormThreads) {
      const float q = E::to_f32(dy[h]) * (gamma ? W::to_f32(gamma[h]) : 1.0f);
      s1 += q;
      s2 = fmaf(q, (E::to_f32(x[h]) - mean) * rstd, s2);
    }
    const float2 s = block_sum2<kNormThreads>(s1, s2, red);
    const float c1 = s.x / fh, c2 = s.y / fh;
    for (int h = threadIdx.x; h < a.H; h += kNormThreads) {
      const float q = E::to_f32(dy[h]) * (gamma ? W::to_f32(gamma[h]) : 1.0f);
      const float xh = (E::to_f32(x[h]) - mean) * rstd;
      dx[h] = E::from_f32(rstd * (q - c1 - xh * c2));
    }
  }
}

// Partial rows of the weights' gradients for the loop form: block (i, j) adds tokens j, j + J, ...
// (J = gridDim.y) of columns i * 256 .. + 256.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_part_loop_kernel(const NormBwdArgs a) {
  using E = Elem<DT>;
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x * kNormThreads + threadIdx.x;
  if (h >= a.H) return;
  float dg = 0.f, db = 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const float g = E::to_f32(static_cast<const typename E::raw*>(a.dy)[t * a.dy_stride + h]);
    const float x = E::to_f32(static_cast<const typename E::raw*>(a.x)[t * a.x_stride + h]);
    dg = fmaf(g, (x - a.mean[t]) * a.rstd[t], dg);
    db += g;
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.H;
  p[h] = dg;
  p[a.H + h] = db;
}

// Partial rows of the weights' gradients: enough CTAs to fill the device, and no more than tokens.
// A device-independent bound keeps the workspace the same on every device.
constexpr int kNormPartRows = 296;

// Adds `rows` partial rows of n = 2H floats (V at a time) in a fixed order: thread (i, j) of a block
// adds the rows j, j + 32, ... of its columns, all in flight at once, then the 32 sums are added in
// order.
constexpr int kSumLanes = 16, kSumRows = 32;
template <int V>
__global__ void __launch_bounds__(kSumLanes* kSumRows) norm_bwd_sum_kernel(
    const float* __restrict__ part, int rows, int64_t H, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[kSumRows][kSumLanes * V + 1];
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x % kSumLanes, j = threadIdx.x / kSumLanes;
  const int64_t n = 2 * H, base = blockIdx.x * static_cast<int64_t>(kSumLanes * V);
  const int64_t c = base + i * V;
  float s[V];
#pragma unroll
  for (int q = 0; q < V; ++q) s[q] = 0.0f;
  if (c < n)
#pragma unroll
    for (int u = 0; u < (kNormPartRows + kSumRows - 1) / kSumRows; ++u) {
      const int r = j + u * kSumRows;
      if (r >= rows) break;
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(part + r * n + c);
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
      } else {
        s[0] += part[r * n + c];
      }
    }
#pragma unroll
  for (int q = 0; q < V; ++q) red[j][i * V + q] = s[q];
  __syncthreads();
  const int64_t at = base + threadIdx.x;
  if (threadIdx.x < kSumLanes * V && at < n) {
    float v = red[0][threadIdx.x];
#pragma unroll
    for (int r = 1; r < kSumRows; ++r) v += red[r][threadIdx.x];
    if (at < H) {
      if (dgamma) dgamma[at] = v;
    } else if (dbeta) {
      dbeta[at - H] = v;
    }
  }
}

namespace {

// One per token at most, or (classes of tokens, RowRing) seven more.
int norm_part_rows(int64_t T) {
  return static_cast<int>(T + 7 < kNormPartRows ? T + 7 : kNormPartRows);
}

unsigned row_grid(int64_t T) {
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  return static_cast<unsigned>(T < cap ? T : cap);
}

bool vector_rows(int vec, int64_t H, std::initializer_list<int64_t> strides,
                 std::initializer_list<const void*> arrays) {
  if (H % vec != 0) return false;
  for (const int64_t st : strides)
    if (st % vec != 0) return false;
  for (const void* p : arrays)
    if (!aligned16(p)) return false;
  return true;
}

int round32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

// Rows in registers: 16-byte accesses (VW elements), or single elements (VW = 1), which is for few
// rows and for those that the staged form does not take (shorter than two windows or too wide).
template <int DT, int WT, int VW>
cudaError_t norm_forward_rows(const NormArgs& a, cudaStream_t s, bool* done) {
  const int64_t n = a.H / VW;  // accesses of a row (VW divides H)
  *done = true;
  const bool few = a.T < 2 * device_sm_count();
  // A warp per row or two: no barrier.
  auto warps = [&](auto kernel, int rows) {
    rows *= kNormWarpRows;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((a.T + rows - 1) / rows)),
                      dim3(32 * kNormWarpRows), 0, s, a);
  };
  if (!few && n <= 32) return warps(norm_row_kernel<DT, WT, VW, 1, 2, true>, 2);
  if constexpr (VW > 1) {
    if (!few && n <= 64) return warps(norm_row_kernel<DT, WT, VW, 2, 2, true>, 2);
    if (!few && n <= 128) return warps(norm_row_kernel<DT, WT, VW, 4, 2, true>, 2);
    if (!few && n <= 256) return warps(norm_row_kernel<DT, WT, VW, 8, 1, true>, 1);
  }
  // A CTA per row; with few rows as many threads as the row has work for, with many two rows each
  // (T=8192, H=7168 bf16: 45 us, a row each 56 us).
  constexpr int M = VW == 1 ? 16 : 4;
  const int per = few && n <= 1024 ? 1 : few && n <= 2048 ? 2 : M;
  const int G = round32((n + per - 1) / per);
  if (G > 1024) {
    *done = false;
    return cudaSuccess;
  }
  if constexpr (VW > 1) {
    if (!few && G <= 512)
      return launch_pdl(norm_row_kernel<DT, WT, VW, M, 2, false>,
                        dim3(static_cast<unsigned>((a.T + 1) / 2)), dim3(G), 0, s, a);
  }
  auto k = per == 1   ? norm_row_kernel<DT, WT, VW, 1, 1, false>
           : per == 2 ? norm_row_kernel<DT, WT, VW, 2, 1, false>
                      : norm_row_kernel<DT, WT, VW, M, 1, false>;
  return launch_pdl(k, dim3(static_cast<unsigned>(a.T)), dim3(G), 0, s, a);
}

// CTAs of a backward kernel: one an SM (a device-independent bound keeps the workspace the same).
unsigned norm_bwd_grid(int64_t most) {
  const int64_t sms = device_sm_count() < kNormPartRows ? device_sm_count() : kNormPartRows;
  return static_cast<unsigned>(most < sms ? most : sms);
}

// How a staged kernel of A arrays is launched: windows per thread and tokens per stage are its
// template's.
struct RingPlan {
  int G, R, S, C;
  unsigned grid;
  size_t smem;
  bool ok;
};
template <int VE>
RingPlan ring_plan(int64_t T, int64_t H, int A, int per, int K, int weights, bool aligned,
                   bool sums, int least) {
  RingPlan p{};
  const int n = static_cast<int>(aligned ? H / VE : (H + 2 * VE - 2) / VE);
  p.G = round32((n + per - 1) / per);
  if (p.G > kRingThreads || H < 2 * VE) return p;
  p.R = kRingThreads / p.G;  // 16 single warps, or at most 8 groups with a named barrier each
  p.C = aligned ? 1 : VE;
  const size_t stage = static_cast<size_t>(A) * K * (aligned ? n : n + 2) * 16;
  const size_t w = static_cast<size_t>(weights) * n * VE * 4;  // staged weights
  const size_t limit = (aligned ? 224 : 220) * 1024;  // beside the kernels' static 3 or 6 KB
  if (w >= limit) return p;
  const size_t fit = (limit - w) / (stage * p.R);
  const size_t most_stages = kRingStages / p.R < kStagesEach ? kRingStages / p.R : kStagesEach;
  p.S = static_cast<int>(fit < most_stages ? fit : most_stages);
  if (p.S < least) return p;
  p.smem = p.R * p.S * stage + w;
  // the groups' sums may overwrite the stages and the weights behind them
  const size_t sum = sums && p.R > 1 ? static_cast<size_t>(p.R) * 2 * H * 4 : 0;
  if (p.smem < sum) p.smem = sum;
  const int64_t batches = (T + static_cast<int64_t>(p.C) * K - 1) / (static_cast<int64_t>(p.C) * K);
  const int64_t most = norm_bwd_grid(kNormPartRows) / p.C;
  p.grid = static_cast<unsigned>((batches < most ? batches : most) * p.C);
  p.ok = p.grid > 0;
  return p;
}

template <int DT, int WT>
cudaError_t norm_forward_ring(const NormArgs& a, cudaStream_t s, bool* done) {
  constexpr int VE = Elem<DT>::kVec, N = 16 / VE;
  const bool wide = (a.H + 2 * VE - 2) / VE > kRingThreads * N;
  const RingPlan p = ring_plan<VE>(a.T, a.H, 1, wide ? 2 * N : N, 2, 2, false, false, 2);
  auto k = wide ? norm_ring_kernel<DT, WT, 2 * N, 2> : norm_ring_kernel<DT, WT, N, 2>;
  *done = p.ok && ensure_smem_limit(reinterpret_cast<const void*>(k), static_cast<int>(p.smem));
  if (!*done) return cudaSuccess;
  return launch_pdl(k, dim3(p.grid), dim3(p.G * p.R), p.smem, s, a, p.G, p.R, p.S, p.C);
}

template <int DT, int WT>
int norm_forward(const NormArgs& a, cudaStream_t s) {
  constexpr int VE = Elem<DT>::kVec;
  bool done = false;
  cudaError_t e = cudaSuccess;
  if (vector_rows(VE, a.H, {a.x_stride}, {a.x, a.y, a.gamma, a.beta}))
    e = norm_forward_rows<DT, WT, VE>(a, s, &done);
  else if (a.T >= 2 * device_sm_count())
    e = norm_forward_ring<DT, WT>(a, s, &done);
  if (!done) e = norm_forward_rows<DT, WT, 1>(a, s, &done);
  if (!done)
    e = launch_pdl(norm_loop_kernel<DT, WT>, dim3(row_grid(a.T)), dim3(kNormThreads), 0, s, a);
  note_launches(1);
  return e == cudaSuccess ? 0 : MHC_ERR_CUDA;
}

// Launches the staged form and returns its number of partial rows, or 0 (nothing launched) where two
// stages of rows do not fit beside the weights (or rows are shorter than two windows).
template <int DT, int WT, bool kAligned>
int norm_backward_ring(const NormBwdArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VE = Elem<DT>::kVec, N = 16 / VE;  // windows of a thread that holds 16 columns
  constexpr int K = VE == 8 ? 2 : 1;
  const int n = static_cast<int>(kAligned ? a.H / VE : (static_cast<int64_t>(a.H) + 2 * VE - 2) / VE);
  const bool hold = n <= kRingThreads * N;
  const int per = hold ? N : 2 * N;
  const RingPlan p = ring_plan<VE>(a.T, a.H, 2, per, hold ? K : 1, hold && kAligned ? 0 : 1,
                                   kAligned, true,
                                   kAligned || hold ? 2 : 3);
  if (!p.ok) return 0;
  auto k = hold ? norm_bwd_ring_kernel<DT, WT, N, K, true, kAligned>
                : norm_bwd_ring_kernel<DT, WT, 2 * N, 1, false, kAligned>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(k), static_cast<int>(p.smem))) return 0;
  *e = launch_pdl(k, dim3(p.grid), dim3(p.G * p.R), p.smem, s, a, p.G, p.R, p.S, p.C);
  note_launches(1);
  return static_cast<int>(p.grid);
}

template <int DT, int WT>
int norm_backward(NormBwdArgs a, float* dgamma, float* dbeta, cudaStream_t s) {
  constexpr int VE = Elem<DT>::kVec;
  const bool params = dgamma || dbeta;
  if (!params) a.part = nullptr;
  cudaError_t e = cudaSuccess;
  int rows = 0;
  if (vector_rows(VE, a.H, {a.x_stride, a.dy_stride}, {a.x, a.dy, a.dx}))
    rows = norm_backward_ring<DT, WT, true>(a, s, &e);
  else
    rows = norm_backward_ring<DT, WT, false>(a, s, &e);
  if (rows == 0) {
    e = launch_pdl(norm_bwd_dx_loop_kernel<DT, WT>, dim3(row_grid(a.T)), dim3(kNormThreads), 0, s,
                   a);
    note_launches(1);
    if (e != cudaSuccess) return MHC_ERR_CUDA;
    if (params) {
      rows = norm_part_rows(a.T);
      e = launch_pdl(norm_bwd_part_loop_kernel<DT>,
                     dim3((a.H + kNormThreads - 1) / kNormThreads, rows), dim3(kNormThreads), 0, s,
                     a);
      note_launches(1);
    }
  }
  if (e != cudaSuccess) return MHC_ERR_CUDA;
  if (!params) return 0;
  const int v = a.H % 2 == 0 ? 4 : 1;  // 2H floats are whole 16-byte accesses, and so is every row
  e = launch_pdl(v == 4 ? norm_bwd_sum_kernel<4> : norm_bwd_sum_kernel<1>,
                 dim3(static_cast<unsigned>((2 * int64_t(a.H) + kSumLanes * v - 1) / (kSumLanes * v))),
                 dim3(kSumLanes * kSumRows), 0, s, static_cast<const float*>(a.part), rows,
                 int64_t(a.H), dgamma, dbeta);
  note_launches(1);
  return e == cudaSuccess ? 0 : MHC_ERR_CUDA;
}

// Weights are fp32 or of the rows' type.
template <typename F>
int norm_dispatch(int dtype, int w_dtype, F&& f) {
  using std::integral_constant;
  if (dtype == MHC_DTYPE_BF16)
    return w_dtype == MHC_DTYPE_F32
               ? f(integral_constant<int, 0>{}, integral_constant<int, 2>{})
               : f(integral_constant<int, 0>{}, integral_constant<int, 0>{});
  if (dtype == MHC_DTYPE_F16)
    return w_dtype == MHC_DTYPE_F32
               ? f(integral_constant<int, 1>{}, integral_constant<int, 2>{})
               : f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
}

}  // namespace

}  // namespace mhc

extern "C" {

int mhc_layer_norm(const void* x, int64_t x_stride, int dtype, const void* gamma, const void* beta,
                   int w_dtype, void* y, float* mean, float* rstd, int64_t T, int64_t H, float eps,
                   mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, H, x_stride) || !dtype_ok(dtype) || !(eps > 0.0f) || !isfinite(eps))
    return MHC_ERR_INVALID_ARG;
  if ((gamma || beta) && w_dtype != MHC_DTYPE_F32 && w_dtype != dtype) return MHC_ERR_INVALID_ARG;
  if (T == 0) return MHC_OK;
  if (!x || !y) return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), ws = dtype_size(w_dtype);
  if (misaligned(x, es) || misaligned(y, es) || (gamma && misaligned(gamma, ws)) ||
      (beta && misaligned(beta, ws)) || misaligned(mean, 4) || misaligned(rstd, 4))
    return MHC_ERR_INVALID_ARG;
  const size_t nx = row_bytes(T, H, x_stride, es), ny = row_bytes(T, H, H, es);
  const size_t nt = static_cast<size_t>(T) * 4, nw = static_cast<size_t>(H) * ws;
  const bool in_place = x == y && x_stride == H;
  if (!in_place && overlaps(x, nx, y, ny)) return MHC_ERR_ALIAS;
  const Range outs[3] = {{y, ny}, {mean, nt}, {rstd, nt}};
  const Range ins[2] = {{gamma, nw}, {beta, nw}};
  if (any_overlap(outs, 3, ins, 2) || any_overlap(outs + 1, 2, nullptr, 0) ||
      overlap(outs[1], {x, nx}) || overlap(outs[2], {x, nx}))
    return MHC_ERR_ALIAS;
  DeviceScope dev(x);
  if (dev.status != MHC_OK) return dev.status;
  const NormArgs a{x, x_stride, gamma, beta, y, mean, rstd, T, static_cast<int>(H), eps};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(norm_dispatch(dtype, (gamma || beta) ? w_dtype : int(MHC_DTYPE_F32),
                                [&](auto dt, auto wt) {
                                  return norm_forward<dt.value, wt.value>(a, s);
                                }));
}

size_t mhc_layer_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T <= 0 || !rows_ok(T, H, H)) return 0;
  const size_t b = static_cast<size_t>(norm_part_rows(T)) * 2 * static_cast<size_t>(H) * 4;
  return (b + 255) / 256 * 256;
}

int mhc_layer_norm_backward(const void* d_y, int64_t dy_stride, const void* x, int64_t x_stride,
                            int dtype, const void* gamma, int w_dtype, const float* mean,
                            const float* rstd, void* d_x, float* d_gamma, float* d_beta,
                            void* workspace, size_t workspace_bytes, int64_t T, int64_t H,
                            mhc_stream_t stream) {
  if (T < 0 || !rows_ok(T, H, x_stride) || !rows_ok(T, H, dy_stride) || !dtype_ok(dtype))
    return MHC_ERR_INVALID_ARG;
  if (gamma && w_dtype != MHC_DTYPE_F32 && w_dtype != dtype) return MHC_ERR_INVALID_ARG;
  if (misaligned(d_gamma, 4) || misaligned(d_beta, 4)) return MHC_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), ws = dtype_size(w_dtype);
  const size_t nh = static_cast<size_t>(H) * 4, nt = static_cast<size_t>(T) * 4;
  if (d_gamma && d_beta && overlaps(d_gamma, nh, d_beta, nh)) return MHC_ERR_ALIAS;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // the sums over no token are zero
    for (float* p : {d_gamma, d_beta}) {
      if (!p) continue;
      DeviceScope dev(p);
      if (dev.status != MHC_OK) return dev.status;
      if (cudaMemsetAsync(p, 0, nh, s) != cudaSuccess) return launched(MHC_ERR_CUDA);
    }
    return MHC_OK;
  }
  if (!d_y || !x || !mean || !rstd || !d_x) return MHC_ERR_INVALID_ARG;
  if (misaligned(d_y, es) || misaligned(x, es) || misaligned(d_x, es) ||
      (gamma && misaligned(gamma, ws)) || misaligned(mean, 4) || misaligned(rstd, 4))
    return MHC_ERR_INVALID_ARG;
  const size_t need = mhc_layer_norm_backward_workspace_bytes(T, H);
  if (workspace_bytes < need || !workspace) return MHC_ERR_WORKSPACE_TOO_SMALL;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MHC_ERR_INVALID_ARG;
  const Range outs[4] = {{d_x, row_bytes(T, H, H, es)}, {d_gamma, nh}, {d_beta, nh},
                         {workspace, need}};
  const Range ins[5] = {{d_y, row_bytes(T, H, dy_stride, es)}, {x, row_bytes(T, H, x_stride, es)},
                        {gamma, static_cast<size_t>(H) * ws}, {mean, nt}, {rstd, nt}};
  if (any_overlap(outs, 4, ins, 5)) return MHC_ERR_ALIAS;
  DeviceScope dev(x);
  if (dev.status != MHC_OK) return dev.status;
  const NormBwdArgs a{d_y, dy_stride, x, x_stride, gamma, mean, rstd, d_x,
                      static_cast<float*>(workspace), T, static_cast<int>(H)};
  return launched(norm_dispatch(dtype, gamma ? w_dtype : int(MHC_DTYPE_F32), [&](auto dt, auto wt) {
    return norm_backward<dt.value, wt.value>(a, d_gamma, d_beta, s);
  }));
}

}  // extern "C"
