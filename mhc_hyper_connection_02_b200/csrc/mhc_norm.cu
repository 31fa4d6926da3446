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

// Backward: d_x and the CTA's partial sums of the weights' gradients in one pass over x and d_y.
// A CTA holds R groups of G threads (R = blockDim.x / G; kWarp: G = 32); group j of CTA i takes the
// tokens i R + j, + gridDim.x R, ..., and reads the next token's rows before it works on this one's.
// Each thread keeps its columns' gradient sums in registers; at the end the groups add theirs up
// in order through shared memory.
constexpr int norm_bwd_threads(int vw, int n, bool warp) {
  return warp ? 256 : vw * n > 4 ? 512 : 1024;  // what the registers of 8 or 16 columns allow
}
template <int DT, int WT, int VW, int N, bool kWarp>
__global__ void __launch_bounds__(norm_bwd_threads(VW, N, kWarp)) norm_bwd_row_kernel(const NormBwdArgs a,
                                                                          int G) {
  using W = Elem<WT>;
  using C = Chunk<DT, VW>;
  using raw = typename C::raw;
  extern __shared__ float sums[];    // [2][H]: the groups' sums (R > 1)
  __shared__ float red[2][64];  // by turn: each warp's two sums (sum_of_warps)
  pdl_wait();
  pdl_trigger();
  if constexpr (kWarp) G = 32;
  const int R = blockDim.x / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  const float fh = static_cast<float>(a.H);
  float g[N][VW], dg[N][VW], db[N][VW];
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int q = 0; q < VW; ++q) g[i][q] = 1.0f, dg[i][q] = 0.0f, db[i][q] = 0.0f;
    const int h = (i * G + tid) * VW;
    if (gamma && h < a.H) load_weights<WT, VW>(gamma + h, aligned32(gamma), g[i]);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t t = blockIdx.x * static_cast<int64_t>(R) + group;
  C cx[N], cd[N];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = (i * G + tid) * VW;
      if (h < a.H) {
        cx[i].load_ro(static_cast<const raw*>(a.x) + at * a.x_stride + h);
        cd[i].load_ro(static_cast<const raw*>(a.dy) + at * a.dy_stride + h);
      }
    }
    mean = a.mean[at];
    rstd = a.rstd[at];
  };
  if (t < a.T) fetch(t);
  int turn = 0;
  for (; t < a.T; t += step, turn ^= 1) {
    float xh[N][VW], q[N][VW], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i * G + tid) * VW < a.H) {
        cx[i].get(xh[i]);
        cd[i].get(q[i]);
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          const float d = q[i][k];
          xh[i][k] = (xh[i][k] - mean) * rstd;
          dg[i][k] = fmaf(d, xh[i][k], dg[i][k]);
          db[i][k] += d;
          q[i][k] = d * g[i][k];
          s1 += q[i][k];
          s2 = fmaf(q[i][k], xh[i][k], s2);
        }
      }
    const float r = rstd;
    if (t + step < a.T) fetch(t + step);
    const float half = warp_sum_halves(s1, s2);
    float2 p;
    if constexpr (kWarp) {
      p = join_halves(half);
    } else {
      const int nw = G >> 5, w0 = group * nw;
      if ((lane & 15) == 0) red[turn][2 * lane + warp] = half;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
      p = sum_of_warps(red[turn] + w0, nw);
    }
    const float c1 = p.x / fh, c2 = p.y / fh;
    raw* dx = static_cast<raw*>(a.dx) + t * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = (i * G + tid) * VW;
      if (h < a.H) {
#pragma unroll
        for (int k = 0; k < VW; ++k) q[i][k] = r * (q[i][k] - c1 - xh[i][k] * c2);
        C::put(dx + h, q[i]);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  for (int j = 0; j < R; ++j) {
    if (j > 0) __syncthreads();
    if (group != j) continue;
    float* out = j == R - 1 ? part : sums;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = (i * G + tid) * VW;
      if (h < a.H) {
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          out[h + k] = j > 0 ? sums[h + k] + dg[i][k] : dg[i][k];
          out[a.H + h + k] = j > 0 ? sums[a.H + h + k] + db[i][k] : db[i][k];
        }
      }
    }
  }
}

// Backward for wide rows (16-byte accesses): as above, but the tokens' rows of x and d_y are staged
// in shared memory by 1-D bulk copies, several tokens ahead, and read from there twice instead of
// being held in registers, which go to the columns' gradient sums. gamma is kept in shared memory
// in fp32 (the first and the second four columns of each access apart, so that a warp's 16-byte
// reads meet no bank twice). The last warp's first lane issues the copies; all waits are bounded,
// and a group leaves its loop together (named_bar_or).
template <int DT, int WT, int N>
__global__ void __launch_bounds__(N == 4 ? 544 : 1024) norm_bwd_ring_kernel(const NormBwdArgs a, int G, int R,
                                                             int stages) {
  using E = Elem<DT>;
  using W = Elem<WT>;
  using raw = typename E::raw;
  constexpr int VW = E::kVec;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[8], empty[8];
  __shared__ float red[2][64];  // by turn: each warp's two sums (sum_of_warps)
  const int row_bytes = a.H * static_cast<int>(sizeof(raw));
  float* gs = reinterpret_cast<float*>(ring + static_cast<size_t>(stages) * 2 * row_bytes);
  const int n = a.H / VW;  // accesses of a row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / G, tid = threadIdx.x - group * G;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], G / 32);
    }
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();
  const auto* gamma = static_cast<const typename W::raw*>(a.gamma);
  for (int h = threadIdx.x; h < a.H; h += blockDim.x)
    gs[((h % VW) / 4 * n + h / VW) * 4 + h % 4] = gamma ? W::to_f32(gamma[h]) : 1.0f;
  __syncthreads();

  if (group >= R) {
    if (tid == 0) {
      int64_t issued = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < a.T && ok; t += gridDim.x, ++issued) {
        const int st = static_cast<int>(issued % stages);
        if (issued >= stages)
          ok = mbar_wait(&empty[st], static_cast<uint32_t>((issued / stages - 1) & 1), 130);
        if (!ok) break;
        uint8_t* to = ring + static_cast<size_t>(st) * 2 * row_bytes;
        mbar_arrive_expect_tx(&full[st], 2u * row_bytes);
        bulk_g2s(to, static_cast<const raw*>(a.x) + t * a.x_stride, row_bytes, &full[st]);
        bulk_g2s(to + row_bytes, static_cast<const raw*>(a.dy) + t * a.dy_stride, row_bytes,
                 &full[st]);
      }
      if (!ok)  // no copy into this CTA's shared memory may outlive it
        for (int i = 0; i < stages; ++i) {
          const int64_t k = issued / stages + (i < issued % stages ? 1 : 0);
          if (k > 0) mbar_wait(&full[i], static_cast<uint32_t>((k - 1) & 1), 131);
        }
    }
    return;
  }

  const float fh = static_cast<float>(a.H);
  constexpr int P = VW / 2;  // pairs of an access
  F2 dg[N][P], db[N][P];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < P; ++q) dg[i][q] = f2(0.0f), db[i][q] = f2(0.0f);
  // The access at `at` of the staged rows, in pairs: x - mean, d_y and d_y gamma.
  auto take = [&](const uint4* sx, const uint4* sd, int at, F2 neg_mean, F2 (&xm)[P], F2 (&d)[P],
                  F2 (&v)[P]) {
    float f[VW];
    E::unpack(sx[at], f);
#pragma unroll
    for (int q = 0; q < P; ++q) xm[q] = f2(f[2 * q], f[2 * q + 1]) + neg_mean;
    E::unpack(sd[at], f);
#pragma unroll
    for (int q = 0; q < P; ++q) d[q] = f2(f[2 * q], f[2 * q + 1]);
#pragma unroll
    for (int q = 0; q < VW; q += 4) {
      const float4 g = reinterpret_cast<const float4*>(gs)[q / 4 * n + at];
      v[q / 2] = d[q / 2] * f2(g.x, g.y);
      v[q / 2 + 1] = d[q / 2 + 1] * f2(g.z, g.w);
    }
  };
  int64_t k = group;
  int64_t t = blockIdx.x + k * static_cast<int64_t>(gridDim.x);
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  const int nw = G >> 5;
  float mean = 0.f, rstd = 0.f;
  if (t < a.T) mean = a.mean[t], rstd = a.rstd[t];
  int turn = 0;
  for (; t < a.T; t += step, k += R, turn ^= 1) {
    const int st = static_cast<int>(k % stages);
    const F2 neg_mean = f2(-mean);
    const float r = rstd;
    if (t + step < a.T) mean = a.mean[t + step], rstd = a.rstd[t + step];
    const bool ok = mbar_wait(&full[st], static_cast<uint32_t>((k / stages) & 1), 132);
    const uint4* sx = reinterpret_cast<const uint4*>(ring + static_cast<size_t>(st) * 2 * row_bytes);
    const uint4* sd = sx + n;
    F2 s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 xm[P], d[P], v[P];
        take(sx, sd, at, neg_mean, xm, d, v);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          const F2 xh = xm[q] * f2(r);
          dg[i][q] = fma2(d[q], xh, dg[i][q]);
          db[i][q] = db[i][q] + d[q];
          s1 = s1 + v[q];
          s2 = fma2(v[q], xh, s2);
        }
      }
    }
    const float2 u1 = split(s1), u2 = split(s2);
    const float half = warp_sum_halves(u1.x + u1.y, u2.x + u2.y);
    if ((lane & 15) == 0) red[turn][2 * lane + warp] = half;
    if (named_bar_or(group + 1, G, !ok)) break;
    const float2 p = sum_of_warps(red[turn] + group * nw, nw);
    // d_x = r v - r c1 - (x - mean) r^2 c2
    const F2 fr = f2(r), f1 = f2(-r * (p.x / fh)), fx = f2(-r * r * (p.y / fh));
    raw* dx = static_cast<raw*>(a.dx) + t * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
        F2 xm[P], d[P], v[P];
        take(sx, sd, at, neg_mean, xm, d, v);
        float o[VW];
#pragma unroll
        for (int q = 0; q < P; ++q) {
          const float2 u = split(fma2(v[q], fr, fma2(xm[q], fx, f1)));
          o[2 * q] = u.x, o[2 * q + 1] = u.y;
        }
        st_stream(dx + at * VW, E::pack(o));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (!a.part) return;
  // The groups' sums, in order: through the stages' memory (free: every group is done), each
  // access's first and second four columns apart as gamma's.
  float4* part = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H);
  float4* sums = reinterpret_cast<float4*>(ring);
  for (int j = 0; j < R; ++j) {
    if (R > 1) asm volatile("bar.sync 15, %0;" ::"r"(R * G) : "memory");
    if (group != j) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * G + tid;
      if (at < n) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int q = 0; q < P; q += 2) {
            const float2 lo = split(w == 0 ? dg[i][q] : db[i][q]);
            const float2 hi = split(w == 0 ? dg[i][q + 1] : db[i][q + 1]);
            float4 v = make_float4(lo.x, lo.y, hi.x, hi.y);
            float4* sum = sums + (w * (P / 2) + q / 2) * n + at;
            if (j > 0) {
              const float4 b = *sum;
              v = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
            }
            if (j < R - 1)
              *sum = v;
            else
              part[(w * a.H + at * VW) / 4 + q / 2] = v;
          }
      }
    }
  }
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

// Adds `rows` partial rows of n = 2H floats in a fixed order: 8 warps of a block take every eighth
// row of 32 columns, and the eight sums are added in order.
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const float* __restrict__ part, int rows,
                                                           int64_t H, float* __restrict__ dgamma,
                                                           float* __restrict__ dbeta) {
  __shared__ float red[8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = 2 * H, c = blockIdx.x * int64_t(32) + lane;
  float s = 0.f;
  if (c < n)
    for (int r = warp; r < rows; r += 8) s += part[r * n + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < n) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    if (c < H) {
      if (dgamma) dgamma[c] = s;
    } else if (dbeta) {
      dbeta[c - H] = s;
    }
  }
}

namespace {

// Partial rows of the weights' gradients: enough CTAs to fill the device, and no more than tokens.
// A device-independent bound keeps the workspace the same on every device.
constexpr int kNormPartRows = 296;

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
  *done = true;
  const bool few = a.T < 2 * device_sm_count();
  if (!few && n <= 256) {
    // A warp per row or two: no barrier.
    auto k = n <= 32    ? norm_row_kernel<DT, WT, VW, 1, 2, true>
             : n <= 64  ? norm_row_kernel<DT, WT, VW, 2, 2, true>
             : n <= 128 ? norm_row_kernel<DT, WT, VW, 4, 2, true>
                        : norm_row_kernel<DT, WT, VW, 8, 1, true>;
    const int rows = kNormWarpRows * (n <= 128 ? 2 : 1);
    return launch_pdl(k, dim3(static_cast<unsigned>((a.T + rows - 1) / rows)),
                      dim3(32 * kNormWarpRows), 0, s, a);
  }
  // A CTA per two rows; with few rows one each, and as many threads as the row has work for.
  const int per = few && n <= 1024 ? 1 : few && n <= 2048 ? 2 : 4;
  const int G = round32((n + per - 1) / per);
  if (G <= 1024) {
    auto k = per == 1   ? norm_row_kernel<DT, WT, VW, 1, 1, false>
             : per == 2 ? norm_row_kernel<DT, WT, VW, 2, 1, false>
             : few || G > 512 ? norm_row_kernel<DT, WT, VW, 4, 1, false>
                              : norm_row_kernel<DT, WT, VW, 4, 2, false>;
    const int64_t grid = per < 4 || few || G > 512 ? a.T : (a.T + 1) / 2;
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

// CTAs of a backward kernel: as many as are resident, no more than tokens or partial rows.
unsigned norm_bwd_grid(const void* kernel, int threads, size_t smem, int64_t groups_of_tokens) {
  int resident = 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, smem) !=
          cudaSuccess ||
      resident < 1)
    resident = 1;
  int64_t grid = static_cast<int64_t>(device_sm_count()) * resident;
  if (grid > kNormPartRows) grid = kNormPartRows;
  if (grid > groups_of_tokens) grid = groups_of_tokens;
  return static_cast<unsigned>(grid);
}

// Launches the register form and returns its number of partial rows, or 0 (nothing launched) where
// the row is too wide for it.
template <int DT, int WT, int VW>
int norm_backward_rows(const NormBwdArgs& a, cudaStream_t s, cudaError_t* e) {
  const int64_t n = a.H / VW;
  const bool warp = n <= 64;
  int per = 1;
  while (per < 4 && (warp ? n > 32 * per : n > norm_bwd_threads(VW, per, false) * per)) per *= 2;
  if (VW > 1 && per > 2) return 0;
  const int G = warp ? 32 : round32((n + per - 1) / per);
  if (G > norm_bwd_threads(VW, per, false)) return 0;
  const int R = warp ? 8 : G >= 256 ? 1 : G >= 160 ? 2 : G >= 96 ? 4 : 8;
  auto k = warp ? (per == 1 ? norm_bwd_row_kernel<DT, WT, VW, 1, true>
                            : norm_bwd_row_kernel<DT, WT, VW, 2, true>)
           : per == 1 ? norm_bwd_row_kernel<DT, WT, VW, 1, false>
           : per == 2 ? norm_bwd_row_kernel<DT, WT, VW, 2, false>
                      : norm_bwd_row_kernel<DT, WT, VW, (VW == 1 ? 4 : 1), false>;
  const size_t smem = R > 1 ? static_cast<size_t>(2) * a.H * 4 : 0;
  const unsigned grid =
      norm_bwd_grid(reinterpret_cast<const void*>(k), G * R, smem, (a.T + R - 1) / R);
  *e = launch_pdl(k, dim3(grid), dim3(G * R), smem, s, a, G);
  note_launches(1);
  return static_cast<int>(grid);
}

// The staged form, likewise: rows of 16-byte accesses.
template <int DT, int WT>
int norm_backward_ring(const NormBwdArgs& a, cudaStream_t s, cudaError_t* e) {
  const int64_t n = a.H / Elem<DT>::kVec;
  if (n > 512 * 4) return 0;
  const int per = n > 2 * 992 ? 4 : n > 330 ? 2 : 1;
  const int G = round32((n + per - 1) / per);
  const int R = per == 4 || G > 496 ? 1 : G > 330 ? 2 : 3;
  const size_t row = static_cast<size_t>(a.H) * sizeof(typename Elem<DT>::raw);
  const size_t limit = 224 * 1024 - static_cast<size_t>(a.H) * 4;
  const int stages = static_cast<int>(limit / (2 * row) < 8 ? limit / (2 * row) : 8);
  if (stages < 2) return 0;
  const size_t smem = stages * 2 * row + static_cast<size_t>(a.H) * 4;
  auto k = per == 1   ? norm_bwd_ring_kernel<DT, WT, 1>
           : per == 2 ? norm_bwd_ring_kernel<DT, WT, 2>
                      : norm_bwd_ring_kernel<DT, WT, 4>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(k), static_cast<int>(smem))) return 0;
  const unsigned grid =
      norm_bwd_grid(reinterpret_cast<const void*>(k), G * R + 32, smem, a.T);
  *e = launch_pdl(k, dim3(grid), dim3(G * R + 32), smem, s, a, G, R, stages);
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
  if (vector_rows(VE, a.H, {a.x_stride, a.dy_stride}, {a.x, a.dy, a.dx, a.gamma})) {
    if (a.H >= 2048) rows = norm_backward_ring<DT, WT>(a, s, &e);
    if (rows == 0) rows = norm_backward_rows<DT, WT, VE>(a, s, &e);
  } else {
    rows = norm_backward_rows<DT, WT, 1>(a, s, &e);
  }
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
  e = launch_pdl(norm_bwd_sum_kernel, dim3(static_cast<unsigned>((2 * int64_t(a.H) + 31) / 32)),
                 dim3(256), 0, s, static_cast<const float*>(a.part), rows, int64_t(a.H), dgamma,
                 dbeta);
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
