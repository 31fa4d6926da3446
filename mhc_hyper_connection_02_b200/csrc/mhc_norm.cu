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
// CTA adds its tokens in order into a partial row of the workspace, and a second kernel adds the
// partial rows in order.
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
  // kRo: not written by this kernel (read-only path). kKeep: worth keeping in L1 (weights).
  __device__ __forceinline__ void load(const raw* p) {
    if constexpr (VW == 1) v = *p; else v = ld_stream(p);
  }
  __device__ __forceinline__ void load_ro(const raw* p) {
    if constexpr (VW == 1) v = __ldg(p); else v = ld_stream_ro(p);
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

// Backward for rows of any stride and alignment: d_x and the CTA's partial sums of the weights'
// gradients in one pass over x and d_y, element by element. A CTA holds R groups of G threads; group
// j of CTA i takes the tokens i R + j, + gridDim.x R, ..., and reads the next token's rows before it
// exchanges sums for this one. Each thread keeps its N columns' gradient sums in registers; with one
// column a thread (1024 threads a row) a row of 1001 took five times as long.
template <int DT, int WT, int N>
__global__ void __launch_bounds__(512) norm_bwd_row_kernel(const NormBwdArgs a, int G) {
  using W = Elem<WT>;
  using E = Elem<DT>;
  using raw = typename E::raw;
  extern __shared__ float group_sums[];  // [R][2][H] (R > 1)
  __shared__ float red[2][2 * 16];       // by turn: each warp's sums (joined_sums)
  pdl_wait();
  pdl_trigger();
  const int R = blockDim.x / G;
  const int warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  const int nw = G >> 5, w0 = group * nw;
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  const float fh = static_cast<float>(a.H);
  float dg[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t t = blockIdx.x * static_cast<int64_t>(R) + group;
  raw cx[N], cd[N];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t at) {
    const raw* x = static_cast<const raw*>(a.x) + at * a.x_stride;
    const raw* dy = static_cast<const raw*>(a.dy) + at * a.dy_stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = i * G + tid;
      if (h < a.H) cx[i] = __ldg(x + h), cd[i] = __ldg(dy + h);
    }
    mean = a.mean[at];
    rstd = a.rstd[at];
  };
  if (t < a.T) fetch(t);
  int turn = 0;
  for (; t < a.T; t += step, turn ^= 1) {
    float xh[N], q[N], sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = i * G + tid;
      if (h < a.H) {
        const float d = E::to_f32(cd[i]);
        xh[i] = (E::to_f32(cx[i]) - mean) * rstd;
        dg[i] = fmaf(d, xh[i], dg[i]);
        db[i] += d;
        q[i] = gamma ? d * W::to_f32(__ldg(gamma + h)) : d;
        sums[0] += q[i];
        sums[1] = fmaf(q[i], xh[i], sums[1]);
      }
    }
    const float r = rstd;
    if (t + step < a.T) fetch(t + step);
    const float part = warp_sums<2>(sums);
    if (G == 32) {
      share_sums<2>(part, sums);
    } else {
      put_warp_sums<2>(part, red[turn], warp);
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
      joined_sums<2>(red[turn], w0, nw, sums);
    }
    const float c1 = sums[0] / fh, c2 = sums[1] / fh;
    raw* dx = static_cast<raw*>(a.dx) + t * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = i * G + tid;
      if (h < a.H) dx[h] = E::from_f32(r * (q[i] - c1 - xh[i] * c2));
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  float* to = R > 1 ? group_sums + static_cast<size_t>(group) * 2 * a.H : part;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = i * G + tid;
    if (h < a.H) to[h] = dg[i], to[a.H + h] = db[i];
  }
  if (R == 1) return;
  __syncthreads();
  add_groups(group_sums, R, 2 * a.H, part);
}

// Backward for rows of 16-byte accesses. The tokens' rows of x and d_y are staged in shared memory
// by 1-D bulk copies, K tokens to a stage; a group of G threads has S stages of its own and works
// on one at a time. It reads the rows once (kHold: they stay packed in its registers) or twice, and
// exchanges the sums of K tokens at once; the barrier of that exchange also tells its first thread
// that a stage has been read and takes the next copy. Each thread keeps its columns' gradient sums
// in registers over all its tokens: 16 columns at 512 threads an SM, which is what they and two held
// rows leave room for. gamma is kept in shared memory in fp32, the first and the second four columns
// of each access apart, so that a warp's 16-byte reads meet no bank twice. All waits are bounded,
// and a group leaves its loop together.
constexpr int kRingStages = 64;  // of all groups, at most
template <int DT, int WT, int N, int K, bool kHold>
__global__ void __launch_bounds__(512) norm_bwd_ring_kernel(const NormBwdArgs a, int G, int R,
                                                            int S) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  using raw = typename E::raw;
  constexpr int VW = E::kVec, P = VW / 2;  // elements and pairs of an access
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRingStages];
  __shared__ float red[2][2 * K * 16];  // by turn: each warp's sums (joined_sums)
  const int row_bytes = a.H * static_cast<int>(sizeof(raw));
  const int stage_bytes = 2 * K * row_bytes;
  float* gs = reinterpret_cast<float*>(ring + static_cast<size_t>(R * S) * stage_bytes);
  const int n = a.H / VW;  // accesses of a row
  const int warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R * S; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  for (int h = threadIdx.x; h < a.H; h += blockDim.x)
    gs[((h % VW) / 4 * n + h / VW) * 4 + h % 4] = gamma ? W::to_f32(gamma[h]) : 1.0f;
  __syncthreads();

  // Group j of the CTA takes the tokens from ((i R + j) gridDim.x + blockIdx.x) K on, i = 0, 1, ....
  const int64_t step = static_cast<int64_t>(gridDim.x) * K * R;
  int64_t t = (static_cast<int64_t>(group) * gridDim.x + blockIdx.x) * K;
  uint64_t* const mine = full + group * S;
  uint8_t* const stages = ring + static_cast<size_t>(group * S) * stage_bytes;
  auto copy = [&](int st, int64_t at) {  // by the group's first thread
    uint8_t* to = stages + static_cast<size_t>(st) * stage_bytes;
    const int rows = at + K <= a.T ? K : static_cast<int>(a.T - at);
    mbar_arrive_expect_tx(&mine[st], 2u * rows * row_bytes);
    for (int r = 0; r < rows; ++r, to += 2 * row_bytes) {
      bulk_g2s(to, static_cast<const raw*>(a.x) + (at + r) * a.x_stride, row_bytes, &mine[st]);
      bulk_g2s(to + row_bytes, static_cast<const raw*>(a.dy) + (at + r) * a.dy_stride, row_bytes,
               &mine[st]);
    }
  };
  if (tid == 0)
    for (int i = 0; i < S && t + i * step < a.T; ++i) copy(i, t + i * step);
  const float fh = static_cast<float>(a.H);
  F2 dg[N][P], db[N][P];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < P; ++q) dg[i][q] = f2(0.0f), db[i][q] = f2(0.0f);
  auto weights = [&](int at, F2 (&g)[P]) {
#pragma unroll
    for (int q = 0; q < VW; q += 4) {
      const float4 v = reinterpret_cast<const float4*>(gs)[q / 4 * n + at];
      g[q / 2] = f2(v.x, v.y);
      g[q / 2 + 1] = f2(v.z, v.w);
    }
  };
  auto pairs = [&](const uint4& w, F2 (&v)[P]) {
    float f[VW];
    E::unpack(w, f);
#pragma unroll
    for (int q = 0; q < P; ++q) v[q] = f2(f[2 * q], f[2 * q + 1]);
  };
  float mean[K], rstd[K];
  auto stats = [&](int64_t t) {
#pragma unroll
    for (int r = 0; r < K; ++r)
      if (t + r < a.T) mean[r] = a.mean[t + r], rstd[r] = a.rstd[t + r];
  };
  const int nw = G >> 5, w0 = group * nw;
#pragma unroll
  for (int r = 0; r < K; ++r) mean[r] = rstd[r] = 0.0f;
  stats(t);
  int st = 0, turn = 0;
  uint32_t lap = 0;
  bool ok = true;
  for (; t < a.T; t += step, turn ^= 1) {
    F2 nm[K], fr[K];
    float rs[K];
#pragma unroll
    for (int r = 0; r < K; ++r) nm[r] = f2(-mean[r]), fr[r] = f2(rstd[r]), rs[r] = rstd[r];
    const int rows = t + K <= a.T ? K : static_cast<int>(a.T - t);
    ok = mbar_wait(&mine[st], lap & 1, 130);
    const uint4* const sx =
        reinterpret_cast<const uint4*>(stages + static_cast<size_t>(st) * stage_bytes);
    uint4 hx[K][N], hd[K][N];
    if constexpr (kHold) {
#pragma unroll
      for (int r = 0; r < K; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int at = i * G + tid;
          if (at < n && r < rows) {
            hx[r][i] = sx[2 * r * n + at];
            hd[r][i] = sx[(2 * r + 1) * n + at];
          } else {
            hx[r][i] = hd[r][i] = make_uint4(0, 0, 0, 0);
          }
        }
    }
    stats(t + step);
    F2 s1[K], s2[K];
#pragma unroll
    for (int r = 0; r < K; ++r) s1[r] = s2[r] = f2(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 g[P];
        weights(at, g);
#pragma unroll
        for (int r = 0; r < K; ++r) {
          F2 x[P], d[P];
          pairs(kHold ? hx[r][i] : sx[2 * r * n + at], x);
          pairs(kHold ? hd[r][i] : sx[(2 * r + 1) * n + at], d);
#pragma unroll
          for (int q = 0; q < P; ++q) {  // a row that is not there has d_y = 0
            const F2 xh = (x[q] + nm[r]) * fr[r], v = d[q] * g[q];
            dg[i][q] = fma2(d[q], xh, dg[i][q]);
            db[i][q] = db[i][q] + d[q];
            s1[r] = s1[r] + v;
            s2[r] = fma2(v, xh, s2[r]);
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
    if (kHold) {
      if (tid == 0 && t + S * step < a.T) copy(st, t + S * step);
    } else {
      if (tid == 0 && lap + st > 0 && t + (S - 1) * step < a.T)
        copy(st > 0 ? st - 1 : S - 1, t + (S - 1) * step);
    }
    // d_x = r v - r c1 - (x - mean) r^2 c2
    F2 f1[K], fx[K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      f1[r] = f2(-rs[r] * (sums[2 * r] / fh));
      fx[r] = f2(-rs[r] * rs[r] * (sums[2 * r + 1] / fh));
    }
    raw* dx = static_cast<raw*>(a.dx) + t * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 g[P];
        weights(at, g);
#pragma unroll
        for (int r = 0; r < K; ++r) {
          if (r >= rows) break;
          F2 x[P], d[P];
          pairs(kHold ? hx[r][i] : sx[2 * r * n + at], x);
          pairs(kHold ? hd[r][i] : sx[(2 * r + 1) * n + at], d);
          float o[VW];
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const float2 u = split(fma2(d[q] * g[q], fr[r], fma2(x[q] + nm[r], fx[r], f1[r])));
            o[2 * q] = u.x, o[2 * q + 1] = u.y;
          }
          st_stream(dx + static_cast<int64_t>(r) * a.H + at * VW, E::pack(o));
        }
      }
    }
    if (++st == S) st = 0, ++lap;
  }
  if (!ok && tid == 0) {  // no copy into this CTA's shared memory may outlive it
    const int ahead = kHold ? S : S - 1;  // stages with a copy from the current one on
    for (int i = 0; i < S && t + i * step < a.T; ++i) {
      if (i >= ahead && lap > 0) break;
      mbar_wait(&mine[st], lap & 1, 131);
      if (++st == S) st = 0, ++lap;
    }
  }
  if (!a.part) return;
  // The groups' sums, through the stages' memory (free: every group is done).
  __syncthreads();
  float4* part = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H);
  float4* to = R > 1 ? reinterpret_cast<float4*>(ring) + static_cast<size_t>(group) * (a.H / 2)
                     : part;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = i * G + tid;
    if (at < n) {
#pragma unroll
      for (int q = 0; q < P; q += 2) {
        const float2 lo = split(dg[i][q]), hi = split(dg[i][q + 1]);
        to[at * (VW / 4) + q / 2] = make_float4(lo.x, lo.y, hi.x, hi.y);
        const float2 lb = split(db[i][q]), hb = split(db[i][q + 1]);
        to[a.H / 4 + at * (VW / 4) + q / 2] = make_float4(lb.x, lb.y, hb.x, hb.y);
      }
    }
  }
  if (R == 1) return;
  __syncthreads();
  add_groups(reinterpret_cast<const float*>(ring), R, 2 * a.H, reinterpret_cast<float*>(part));
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

int norm_part_rows(int64_t T) { return static_cast<int>(T < kNormPartRows ? T : kNormPartRows); }

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

template <int DT, int WT, int VW>
cudaError_t norm_forward_rows(const NormArgs& a, cudaStream_t s, bool* done) {
  const int64_t n = a.H / VW;  // accesses of a row (VW divides H)
  constexpr int M = VW == 1 ? 16 : 4;  // of a thread, with many rows
  *done = true;
  const bool few = a.T < 2 * device_sm_count();
  if (!few && n <= 64 * M) {
    // A warp per row or two: no barrier.
    auto k = n <= 32       ? norm_row_kernel<DT, WT, VW, 1, 2, true>
             : n <= 64     ? norm_row_kernel<DT, WT, VW, 2, 2, true>
             : n <= 32 * M ? norm_row_kernel<DT, WT, VW, M, 2, true>
                           : norm_row_kernel<DT, WT, VW, 2 * M, 1, true>;
    const int rows = kNormWarpRows * (n <= 32 * M ? 2 : 1);
    return launch_pdl(k, dim3(static_cast<unsigned>((a.T + rows - 1) / rows)),
                      dim3(32 * kNormWarpRows), 0, s, a);
  }
  // A CTA per two rows; with few rows one each, and as many threads as the row has work for.
  const int per = few && n <= 1024 ? 1 : few && n <= 2048 ? 2 : M;
  const int G = round32((n + per - 1) / per);
  if (G <= 1024) {
    const bool two = per == M && !few && G <= 512;
    auto k = per == 1   ? norm_row_kernel<DT, WT, VW, 1, 1, false>
             : per == 2 ? norm_row_kernel<DT, WT, VW, 2, 1, false>
             : two      ? norm_row_kernel<DT, WT, VW, M, 2, false>
                        : norm_row_kernel<DT, WT, VW, M, 1, false>;
    const int64_t grid = two ? (a.T + 1) / 2 : a.T;
    return launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(G), 0, s, a);
  }
  *done = false;
  return cudaSuccess;
}

template <int DT, int WT>
int norm_forward(const NormArgs& a, cudaStream_t s) {
  constexpr int VE = Elem<DT>::kVec;
  bool done = false;
  cudaError_t e;
  if (vector_rows(VE, a.H, {a.x_stride}, {a.x, a.y, a.gamma, a.beta}))
    e = norm_forward_rows<DT, WT, VE>(a, s, &done);
  else
    e = norm_forward_rows<DT, WT, 1>(a, s, &done);
  if (!done)
    e = launch_pdl(norm_loop_kernel<DT, WT>, dim3(row_grid(a.T)), dim3(kNormThreads), 0, s, a);
  note_launches(1);
  return e == cudaSuccess ? 0 : MHC_ERR_CUDA;
}

// CTAs of a backward kernel: one an SM (a device-independent bound keeps the workspace the same).
unsigned norm_bwd_grid(int64_t most) {
  const int64_t sms = device_sm_count() < kNormPartRows ? device_sm_count() : kNormPartRows;
  return static_cast<unsigned>(most < sms ? most : sms);
}

// Launches the element-wise form and returns its number of partial rows, or 0 (nothing launched)
// where the row is too wide for it.
template <int DT, int WT>
int norm_backward_rows(const NormBwdArgs& a, cudaStream_t s, cudaError_t* e) {
  const int per = a.H <= 4096 ? 8 : 16;
  const int G = round32((a.H + per - 1) / per);
  if (G > 512) return 0;
  const int R = G == 32 ? 16 : 512 / G < 15 ? 512 / G : 15;
  const size_t smem = R > 1 ? static_cast<size_t>(R) * 2 * a.H * 4 : 0;
  auto k = per == 8 ? norm_bwd_row_kernel<DT, WT, 8> : norm_bwd_row_kernel<DT, WT, 16>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(k), static_cast<int>(smem))) return 0;
  const unsigned grid = norm_bwd_grid((a.T + R - 1) / R);
  *e = launch_pdl(k, dim3(grid), dim3(G * R), smem, s, a, G);
  note_launches(1);
  return static_cast<int>(grid);
}

// The staged form, likewise: rows of 16-byte accesses that fit twice beside gamma.
template <int DT, int WT>
int norm_backward_ring(const NormBwdArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VW = Elem<DT>::kVec, N = 16 / VW;  // accesses of a thread that holds 16 columns
  constexpr int K = VW == 8 ? 2 : 1;
  const int64_t n = a.H / VW;
  const bool hold = n <= 512 * N;
  const int per = hold ? (n <= 32 ? 1 : N) : 2 * N;
  const int G = round32((n + per - 1) / per);
  if (G > 512) return 0;
  const int R = G == 32 ? 16 : 512 / G < 15 ? 512 / G : 15;
  const size_t stage = 2 * static_cast<size_t>(a.H) * sizeof(typename Elem<DT>::raw) * (hold ? K : 1);
  const size_t weights = static_cast<size_t>(a.H) * 4, sums = R > 1 ? 2 * weights * R : 0;
  const size_t fit = (224 * 1024 - weights) / (stage * R);
  const int S = static_cast<int>(fit < kRingStages / 16 ? fit : kRingStages / 16);
  if (S < 2) return 0;
  // gamma lies behind the stages; the groups' sums may overwrite it
  const size_t used = R * S * stage + weights, smem = used > sums ? used : sums;
  auto k = !hold      ? norm_bwd_ring_kernel<DT, WT, 2 * N, 1, false>
           : per == 1 ? norm_bwd_ring_kernel<DT, WT, 1, K, true>
                      : norm_bwd_ring_kernel<DT, WT, N, K, true>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(k), static_cast<int>(smem))) return 0;
  const int rows = hold ? K : 1;
  const unsigned grid = norm_bwd_grid((a.T + rows - 1) / rows);
  *e = launch_pdl(k, dim3(grid), dim3(G * R), smem, s, a, G, R, S);
  note_launches(1);
  return static_cast<int>(grid);
}

template <int DT, int WT>
int norm_backward(NormBwdArgs a, float* dgamma, float* dbeta, cudaStream_t s) {
  constexpr int VE = Elem<DT>::kVec;
  const bool params = dgamma || dbeta;
  if (!params) a.part = nullptr;
  cudaError_t e = cudaSuccess;
  int rows = 0;
  if (vector_rows(VE, a.H, {a.x_stride, a.dy_stride}, {a.x, a.dy, a.dx, a.gamma}))
    rows = norm_backward_ring<DT, WT>(a, s, &e);
  if (rows == 0) rows = norm_backward_rows<DT, WT>(a, s, &e);
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
