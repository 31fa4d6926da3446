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

template <int DT, int WT>
int norm_forward(const NormArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(norm_loop_kernel<DT, WT>, dim3(row_grid(a.T)),
                                   dim3(kNormThreads), 0, s, a);
  note_launches(1);
  return e == cudaSuccess ? 0 : MHC_ERR_CUDA;
}

template <int DT, int WT>
int norm_backward(const NormBwdArgs& a, float* dgamma, float* dbeta, cudaStream_t s) {
  cudaError_t e = launch_pdl(norm_bwd_dx_loop_kernel<DT, WT>, dim3(row_grid(a.T)),
                             dim3(kNormThreads), 0, s, a);
  note_launches(1);
  if (e != cudaSuccess) return MHC_ERR_CUDA;
  if (!dgamma && !dbeta) return 0;
  const int rows = norm_part_rows(a.T);
  e = launch_pdl(norm_bwd_part_loop_kernel<DT>, dim3((a.H + kNormThreads - 1) / kNormThreads, rows),
                 dim3(kNormThreads), 0, s, a);
  note_launches(1);
  if (e != cudaSuccess) return MHC_ERR_CUDA;
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
