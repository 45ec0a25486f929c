// Streaming one row of logits: its 16-byte body between an unaligned head and a ragged tail, and the softmax
// statistics (m, s), s = sum 2^((x - m) c) with c = log2(e) / T, that the distillation and verification
// kernels share.
//
// An accumulator starts at (-FLT_MAX, 0): a masked logit (-inf) then contributes 2^(-inf) = 0 instead of
// -inf - -inf, and a row without a finite logit ends with s = 0. NaN and +inf logits make s NaN (inf - inf),
// so `stats_valid` needs no test per element. The difference x - m is taken before the multiplication by c
// (not fused as x c - m c): the rounding of m c would shift every exponent of the row by the same amount.
#pragma once

#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "sfc_device.cuh"

namespace sfc {

constexpr float kLog2e = 1.4426950408889634f;

// log2(e) / T, finite for every T > 0 (a subnormal T would give +inf, and 0 * inf a NaN at the maximum).
__device__ __forceinline__ float exponent_scale(float T) { return fminf(kLog2e / T, FLT_MAX); }

__device__ __forceinline__ bool temperature_valid(float T) { return T > 0.f && T < INFINITY; }

template <int DT>
struct RowSpan {
  const unsigned char* row;
  int64_t V, nvec;
  int head;  // elements before the first 16-byte boundary

  __device__ __forceinline__ RowSpan(const void* base, int64_t offset, int64_t V_) : V(V_) {
    row = static_cast<const unsigned char*>(base) + offset * Elem<DT>::kBytes;
    const int to16 = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / Elem<DT>::kBytes;
    head = static_cast<int>(V < to16 ? V : to16);
    nvec = (V - head) / Elem<DT>::kVec;
  }
  __device__ __forceinline__ const uint4* body() const {
    return reinterpret_cast<const uint4*>(row + static_cast<int64_t>(head) * Elem<DT>::kBytes);
  }
  __device__ __forceinline__ int64_t tail() const { return head + nvec * Elem<DT>::kVec; }  // first tail element
  // Scalars outside the body (fewer than two vectors): the index of scalar i, for i < scalars().
  __device__ __forceinline__ int scalars() const { return head + static_cast<int>(V - tail()); }
  __device__ __forceinline__ int64_t scalar_index(int i) const { return i < head ? i : tail() + (i - head); }
  __device__ __forceinline__ float at(int64_t i) const { return Elem<DT>::load1(row, i); }
};

struct SoftmaxAcc {
  float m = -FLT_MAX, s = 0.f;

  __device__ __forceinline__ void add(float x, float c) {
    if (x > m) {
      s *= ex2_approx((m - x) * c);
      m = x;
    }
    s += ex2_approx((x - m) * c);
  }
  // One vector: a rescale only when its maximum is a new one.
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float vmax, float c) {
    if (vmax > m) {
      s *= ex2_approx((m - vmax) * c);
      m = vmax;
    }
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = ex2_approx((x[i] - m) * c);
#pragma unroll
    for (int w = N / 2; w > 0; w /= 2)  // a fixed tree
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] += e[i + w];
    s += e[0];
  }
  __device__ __forceinline__ void merge(float m2, float s2, float c) {
    const float mn = fmaxf(m, m2);
    s = s * ex2_approx((m - mn) * c) + s2 * ex2_approx((m2 - mn) * c);
    m = mn;
  }
};

// A finite maximum and a mass: false for rows with NaN or +inf logits (s is NaN) or without a finite one.
__device__ __forceinline__ bool stats_valid(float m, float s) { return s > 0.f && s < INFINITY && m < INFINITY; }

// The accumulators of the CTA's NT threads as one, the same bits in every thread: warp butterflies (each
// step is symmetric in its two operands), then the warps in order. `red` holds 2 NT / 32 floats; a barrier
// must separate two uses of it.
template <int NT>
__device__ __forceinline__ void block_merge(SoftmaxAcc& a, float c, float* red) {
  constexpr int NW = NT / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(kFull, a.m, o), s2 = __shfl_xor_sync(kFull, a.s, o);
    a.merge(m2, s2, c);
  }
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = a.m;
    red[NW + (threadIdx.x >> 5)] = a.s;
  }
  __syncthreads();
  float m = red[0];
  for (int w = 1; w < NW; ++w) m = fmaxf(m, red[w]);
  float s = 0.f;
  for (int w = 0; w < NW; ++w) s += red[NW + w] * ex2_approx((red[w] - m) * c);
  a.m = m;
  a.s = s;
}

// Sums over the CTA in a fixed order, the same bits in every thread. `red` holds K NT / 32 floats.
template <int NT, int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float* red) {
  constexpr int NW = NT / 32;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(kFull, v[k], o);
    if ((threadIdx.x & 31) == 0) red[k * NW + (threadIdx.x >> 5)] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = red[k * NW];
    for (int w = 1; w < NW; ++w) v[k] += red[k * NW + w];
  }
}

// This thread's share (vectors t, t + NT, ...) of the row's statistics.
template <int DT, int NT>
__device__ __forceinline__ SoftmaxAcc row_stats(const RowSpan<DT>& r, int64_t v0, int64_t v1, bool scalars, float c) {
  constexpr int VEC = Elem<DT>::kVec, U = 4;
  SoftmaxAcc a;
  const uint4* body = r.body();
  for (int64_t k0 = v0 + threadIdx.x; k0 < v1; k0 += NT * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = k0 + u * NT < v1 ? __ldg(body + k0 + u * NT) : Elem<DT>::neg_inf_vec();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[VEC];
      Elem<DT>::unpack(v[u], x);
      a.add(x, Elem<DT>::vmax(v[u]), c);
    }
  }
  if (scalars && static_cast<int>(threadIdx.x) < r.scalars()) a.add(r.at(r.scalar_index(threadIdx.x)), c);
  return a;
}

// Round once to the element type.
template <int DT>
struct Out;
template <>
struct Out<0> {
  __device__ __forceinline__ static void store1(unsigned char* row, int64_t i, float x) {
    reinterpret_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(x);
  }
  __device__ __forceinline__ static uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Out<1> {
  __device__ __forceinline__ static void store1(unsigned char* row, int64_t i, float x) {
    reinterpret_cast<float*>(row)[i] = x;
  }
  __device__ __forceinline__ static uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

}  // namespace sfc
