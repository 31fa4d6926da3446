// Device-side helpers of the row operators (layer norm, token log probabilities, distillation):
// element types, 16-byte windows over rows of any alignment, and block reductions in a fixed order.
#pragma once

#include <cuda_fp16.h>

#include "mhc_device.cuh"

namespace mhc {

// Element types (the values of enum mhc_dtype). kVec elements fill 16 bytes.
template <int DT>
struct Elem;

template <>
struct Elem<0> {  // bf16
  using raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr int kOrderBits = 16;  // leading bits of order_key that tell values apart
  static constexpr raw kNegInf = 0xff80;
  static __device__ __forceinline__ float to_f32(raw v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ raw from_f32(float v) { return f32_to_bf16(v); }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = bf16_lo((&w.x)[q]);
      x[2 * q + 1] = bf16_hi((&w.x)[q]);
    }
  }
  // Each value at least -2^100 (a NaN stays one): finite, and below anything whose exponential
  // matters.
  static constexpr bool kCuts = true;
  static __device__ __forceinline__ uint4 cut(uint4 w) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"((&w.x)[q]) : "r"(0xf180f180u));
    return w;
  }
  // The largest of the windows' values, NaN apart.
  template <int N>
  static __device__ __forceinline__ float max_of(const uint4 (&w)[N]) {
    uint32_t m = w[0].x;
#pragma unroll
    for (int i = 1; i < 4 * N; ++i)
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"((&w[i / 4].x)[i % 4]));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

template <>
struct Elem<1> {  // fp16
  using raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr int kOrderBits = 19;
  static constexpr raw kNegInf = 0xfc00;
  static __device__ __forceinline__ float to_f32(raw v) {
    return __half2float(__ushort_as_half(v));
  }
  static __device__ __forceinline__ raw from_f32(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&(&w.x)[q]));
      x[2 * q] = f.x;
      x[2 * q + 1] = f.y;
    }
  }
  // -infinity and the lowest finite value are too near for a cut between them.
  static constexpr bool kCuts = false;
  static __device__ __forceinline__ uint4 cut(uint4 w) { return w; }
  template <int N>
  static __device__ __forceinline__ float max_of(const uint4 (&w)[N]) {
    uint32_t m = w[0].x;
#pragma unroll
    for (int i = 1; i < 4 * N; ++i)
      asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"((&w[i / 4].x)[i % 4]));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 h = __floats2half2_rn(x[2 * q], x[2 * q + 1]);
      (&w.x)[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return w;
  }
};

template <>
struct Elem<2> {  // fp32
  using raw = float;
  static constexpr int kVec = 4;
  static constexpr int kOrderBits = 32;
  static __device__ __forceinline__ float to_f32(raw v) { return v; }
  static __device__ __forceinline__ raw from_f32(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = __uint_as_float((&w.x)[q]);
  }
  static constexpr bool kCuts = false;
  static __device__ __forceinline__ uint4 cut(uint4 w) { return w; }
  template <int N>
  static __device__ __forceinline__ float max_of(const uint4 (&w)[N]) {
    float m = __uint_as_float(w[0].x);
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) m = fmaxf(m, __uint_as_float((&w[i / 4].x)[i % 4]));
    return m;
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// ------------------------------------------------------------------------------ windows
//
// A row of n elements at any element-aligned address is cut at the 16-byte boundaries of its
// addresses: window s holds elements s * kVec - off .. + kVec, where `off` elements of window 0
// (and the end of the last window) lie outside the row. Whole windows are read and written with
// one 16-byte access, the first and the last by single elements where the row does not fill them,
// so nothing outside the row is touched.

template <int DT>
__device__ __forceinline__ int window_offset(const void* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) /
                          sizeof(typename Elem<DT>::raw));
}
template <int DT>
__device__ __forceinline__ int window_count(int off, int n) {
  return (off + n + Elem<DT>::kVec - 1) / Elem<DT>::kVec;
}

// First element of window s (negative in a partial window 0).
template <int DT>
__device__ __forceinline__ int window_first(int s, int off) {
  return s * Elem<DT>::kVec - off;
}

// Window s; what lies outside the row (all of it past the last window) comes back as -infinity.
template <int DT>
__device__ __forceinline__ uint4 load_window(const typename Elem<DT>::raw* row, int n, int off,
                                             int s) {
  using E = Elem<DT>;
  const int e0 = window_first<DT>(s, off);
  if (e0 >= 0 && e0 <= n - E::kVec) return ld_stream_ro(row + e0);
  uint4 w;
  if constexpr (DT == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + j;
      (&w.x)[j] = (e >= 0 && e < n) ? __float_as_uint(row[e]) : 0xff800000u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + 2 * j;
      const uint32_t lo = (e >= 0 && e < n) ? row[e] : E::kNegInf;
      const uint32_t hi = (e + 1 >= 0 && e + 1 < n) ? row[e + 1] : E::kNegInf;
      (&w.x)[j] = lo | (hi << 16);
    }
  }
  return w;
}

// ------------------------------------------------------------------------------ async copies

// Four bytes global -> shared without a register; async_copies_arrive lets `bar` count one arrival
// once this thread's copies so far are there (an arrival its initial count includes).
__device__ __forceinline__ void async_copy4(void* smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void async_copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// ------------------------------------------------------------------------------ pairs
//
// Two fp32 operations in one instruction (each rounded as on its own): half the issue slots where
// a loop over elements is bound by them.

struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// ------------------------------------------------------------------------------ reductions

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Both sums in five exchanges: lanes 0-15 end with the sum of a, lanes 16-31 with that of b.
__device__ __forceinline__ float warp_sum_halves(float a, float b) {
  const bool high = (threadIdx.x & 16) != 0;
  float v = high ? b : a;
  v += __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// (sum of a, sum of b) in every lane, from warp_sum_halves' result.
__device__ __forceinline__ float2 join_halves(float v) {
  const float o = __shfl_xor_sync(0xffffffffu, v, 16);
  return (threadIdx.x & 16) != 0 ? make_float2(o, v) : make_float2(v, o);
}
// The pair of sums over nw warps from their halves in red[0 .. nw) and red[32 .. 32 + nw).
__device__ __forceinline__ float2 sum_of_warps(const float* red, int nw) {
  const int half = (threadIdx.x >> 4) & 1, l = threadIdx.x & 15;
  const float* r = red + 32 * half;
  float v = l < nw ? r[l] : 0.0f;
  if (l + 16 < nw) v += r[l + 16];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return join_halves(v);
}

// The same for M = 2 or 4 sums of up to 16 warps: lanes j 32 / M to (j + 1) 32 / M hold sum j ...
template <int M>
__device__ __forceinline__ float warp_sums(const float (&v)[M]) {
  if constexpr (M == 2) {
    return warp_sum_halves(v[0], v[1]);
  } else {
    const bool high = (threadIdx.x & 16) != 0, odd = (threadIdx.x & 8) != 0;
    float a = high ? v[2] : v[0], b = high ? v[3] : v[1];
    a += __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 16);
    float s = odd ? b : a;
    s += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
}
// ... which every lane gets all of,
template <int M>
__device__ __forceinline__ void share_sums(float s, float (&v)[M]) {
#pragma unroll
  for (int j = 0; j < M; ++j) v[j] = __shfl_sync(0xffffffffu, s, j * (32 / M));
}
// or which are put into red[16 M] ...
template <int M>
__device__ __forceinline__ void put_warp_sums(float s, float* red, int warp) {
  const int lane = threadIdx.x & 31;
  if (lane % (32 / M) == 0) red[lane / (32 / M) * 16 + warp] = s;
}
// and, after a barrier, joined over the warps w0 .. w0 + nw.
template <int M>
__device__ __forceinline__ void joined_sums(const float* red, int w0, int nw, float (&v)[M]) {
  constexpr int L = 32 / M;
  const int lane = threadIdx.x & 31, l = lane % L;
  const float* r = red + lane / L * 16 + w0;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; w += L)
    if (l + w < nw) s += r[l + w];
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  share_sums<M>(s, v);
}

// Block reductions of NT threads: an xor tree in each warp, then the warps in order, the same bits
// in every thread. `red` holds NT / 32 floats (2 NT / 32 for the pair); the leading barrier makes
// it safe to use one array for several reductions.
template <int NT>
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) v += red[w];
  return v;
}
template <int NT>
__device__ __forceinline__ float2 block_sum2(float a, float b, float* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red[2 * (threadIdx.x >> 5)] = a;
    red[2 * (threadIdx.x >> 5) + 1] = b;
  }
  __syncthreads();
  a = red[0];
  b = red[1];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) {
    a += red[2 * w];
    b += red[2 * w + 1];
  }
  return make_float2(a, b);
}

}  // namespace mhc
