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

// The two halves of a cluster barrier (release / acquire).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The arrival of a cluster barrier that orders no memory, such as that of CTAs which have started.
__device__ __forceinline__ void cluster_arrive_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
// The arrival of a CTA whose first warp alone has stored what the other CTAs are to see behind the barrier: a release waits for
// all that its warp has in flight.
__device__ __forceinline__ void cluster_arrive_first_warp() {
  if (threadIdx.x < 32) {
    __syncwarp();
    cluster_arrive();
  } else {
    cluster_arrive_started();
  }
}

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

__device__ __forceinline__ uint64_t fmul_f2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float warp_max(float x) {  // one instruction (NaN only where all are)
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// 2^((x - m) c) of a vector's elements, two lanes of a packed instruction at a time: the pass over a row is bound by
// its instruction issue as much as by HBM. minus_m and c hold their value in both lanes.
template <int N>
__device__ __forceinline__ void exponentials(const float (&x)[N], uint64_t minus_m, uint64_t c, uint64_t (&e)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float a, b;
    unpack_f2(fmul_f2(fadd_f2(pack_f2(x[2 * i], x[2 * i + 1]), minus_m), c), a, b);
    e[i] = pack_f2(ex2_approx(a), ex2_approx(b));
  }
}

// The larger elements of two vectors.
template <int DT>
__device__ __forceinline__ uint4 larger(const uint4& a, const uint4& b) {
  auto word = [](uint32_t x, uint32_t y) {
    if constexpr (DT == 0) {
      const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
      return *reinterpret_cast<const uint32_t*>(&h);
    } else {
      return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
    }
  };
  return make_uint4(word(a.x, b.x), word(a.y, b.y), word(a.z, b.z), word(a.w, b.w));
}

// The statistics of what one thread has seen. The sum is held in two lanes. m is the true maximum: a reference that
// lies above it loses mass (2^((x - m) c) is flushed to 0), and so does the rescaling of a sum that grew far above its
// reference. Rows that are masked but for improbable tokens, and low temperatures, are such cases.
struct SoftmaxAcc {
  float m = -FLT_MAX;
  uint64_t s2 = 0;  // (0.f, 0.f)

  __device__ __forceinline__ void raise(float x, float c) {
    if (x > m) {
      const float f = ex2_approx((m - x) * c);
      s2 = fmul_f2(s2, pack_f2(f, f));
      m = x;
    }
  }
  __device__ __forceinline__ void add(float x, float c) {
    raise(x, c);
    s2 = fadd_f2(s2, pack_f2(ex2_approx((x - m) * c), 0.f));
  }
  // One vector: a rescale only when its maximum is a new one.
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float vmax, float c) {
    raise(vmax, c);
    add_below(x, c);
  }
  template <int N>
  __device__ __forceinline__ void add_below(const float (&x)[N], float c) {  // none of x is above m
    uint64_t e[N / 2];
    exponentials(x, pack_f2(-m, -m), pack_f2(c, c), e);
#pragma unroll
    for (int w = N / 4; w > 0; w /= 2)  // a fixed tree
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] = fadd_f2(e[i], e[i + w]);
    s2 = fadd_f2(s2, e[0]);
  }
  // U vectors. bf16: one maximum of all, which packed maxima make cheap (128 x 4 rows of 151936 verified in 98.4 us, with
  // one for each vector 99.3); f32: one for each, so that none waits for the others (32 x 4 rows of 129280 44.0 us, one
  // of all 45.1).
  template <int DT, int U>
  __device__ __forceinline__ void add(const uint4 (&v)[U], float c) {
    constexpr int G = DT == 0 ? U : 1;
#pragma unroll
    for (int g = 0; g < U; g += G) {
      uint4 top = v[g];
#pragma unroll
      for (int u = 1; u < G; ++u) top = larger<DT>(top, v[g + u]);
      raise(Elem<DT>::vmax(top), c);
#pragma unroll
      for (int u = 0; u < G; ++u) {
        float x[Elem<DT>::kVec];
        Elem<DT>::unpack(v[g + u], x);
        add_below(x, c);
      }
    }
  }
  __device__ __forceinline__ float sum() const {
    float a, b;
    unpack_f2(s2, a, b);
    return a + b;
  }
};

// Merged statistics: of a warp, a CTA, a row.
struct SoftmaxStats {
  float m, s;

  __device__ __forceinline__ void merge(float m2, float s2, float c) {
    const float mn = fmaxf(m, m2);
    s = s * ex2_approx((m - mn) * c) + s2 * ex2_approx((m2 - mn) * c);
    m = mn;
  }
};

// A finite reference and a mass: false for rows with NaN or +inf logits (s is NaN) or without a finite one.
__device__ __forceinline__ bool stats_valid(float m, float s) { return s > 0.f && s < INFINITY && m < INFINITY; }

__device__ __forceinline__ float warp_total(float x) {  // butterflies: the same bits in every lane
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// The warp's statistics: its maximum first, then each thread's sum rescaled once.
__device__ __forceinline__ SoftmaxStats warp_stats(const SoftmaxAcc& a, float c) {
  const float m = warp_max(a.m);
  return SoftmaxStats{m, warp_total(a.sum() * ex2_approx((a.m - m) * c))};
}
// Those of the CTA's warps, one in each lane (the lanes past them repeat the first with no mass).
template <int NT>
__device__ __forceinline__ SoftmaxStats merge_warps(const float2* red, float c) {
  const int lane = threadIdx.x & 31;
  const float2 v = red[lane < NT / 32 ? lane : 0];
  const float m = warp_max(v.x);
  return SoftmaxStats{m, warp_total(lane < NT / 32 ? v.y * ex2_approx((v.x - m) * c) : 0.f)};
}

// This thread's vectors of [v0, v1) of a row, every NT-th, U of them at a time. The first batch can be on its way
// before anything else of the row is known, and each later one is while the one before it is used.
template <int DT, int NT, int U>
struct RowStream {
  const uint4* body;
  int k, v1;
  uint4 v[U];

  __device__ __forceinline__ RowStream(const RowSpan<DT>& r, int v0, int v1_)
      : body(r.body()), k(v0 + static_cast<int>(threadIdx.x)), v1(v1_) {
    load(v, k);
  }
  __device__ __forceinline__ void load(uint4 (&w)[U], int at) const {
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = at + u * NT < v1 ? ld_once(body + at + u * NT) : Elem<DT>::neg_inf_vec();
  }
  // use(U vectors), in order, by whole warps; vectors past the end are -inf.
  template <class F>
  __device__ __forceinline__ void batches(F use) {
    while (k - static_cast<int>(threadIdx.x & 31) < v1) {
      uint4 next[U];
      load(next, k + NT * U);
      use(v);
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = next[u];
      k += NT * U;
    }
  }
  // use(vector, its index), the same by vectors; padding vectors (-inf) have an index >= v1.
  template <class F>
  __device__ __forceinline__ void each(F use) {
    batches([&](const uint4 (&w)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) use(w[u], k + u * NT);
    });
  }
};

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

// A vector of 16-bit elements to an address that lies `shift` > 0 bytes past a 16-byte boundary, by a whole warp whose
// lanes hold consecutive vectors, the active ones first: each lane joins the end of its neighbour's vector and the start
// of its own to one aligned store; only the warp's two ends are stored by elements. (By elements throughout, a bf16
// gradient that is shifted against its logits took 445 us at 1024 x 151936; so 205, aligned 138. For f32 elements
// by themselves are faster: 128 us against 140 at 512 x 129280.)
__device__ __forceinline__ void store_shifted(unsigned char* at, const uint4& w, int shift, bool active) {
  const int lane = threadIdx.x & 31;
  const unsigned on = __ballot_sync(kFull, active);
  uint32_t c[8] = {0u, 0u, 0u, 0u, w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __shfl_up_sync(kFull, c[4 + i], 1);
  const int from = 16 - shift, bits = (from & 3) * 8;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    switch (from >> 2) {  // uniform
      case 0: o[i] = __funnelshift_r(c[i], c[i + 1], bits); break;
      case 1: o[i] = __funnelshift_r(c[i + 1], c[i + 2], bits); break;
      case 2: o[i] = __funnelshift_r(c[i + 2], c[i + 3], bits); break;
      default: o[i] = __funnelshift_r(c[i + 3], c[i + 4], bits); break;
    }
  }
  if (!active) return;
  if (lane > 0) *reinterpret_cast<uint4*>(at - shift) = make_uint4(o[0], o[1], o[2], o[3]);
  const bool last = lane == 31 || !(on >> (lane + 1) & 1u);
  if (lane > 0 && !last) return;
  const int first_part = from / 2;  // elements before the next boundary
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < first_part ? lane == 0 : last)
      reinterpret_cast<uint16_t*>(at)[e] = static_cast<uint16_t>(e & 1 ? c[4 + e / 2] >> 16 : c[4 + e / 2]);
}

}  // namespace sfc
