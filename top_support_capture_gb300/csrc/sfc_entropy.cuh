// Softmax statistics of a row together with what its entropy needs, and the gradient that log-probabilities and the
// entropy pass to the logits. With d = (x - m) c, c = log2(e) / T, m the row's maximum:
//
//   s = sum 2^d,  w = sum 2^d d,  ln p = ln2 d - ln s,  H = -sum p ln p = ln s - ln2 w / s   (both parts are >= 0)
//   sum_i g_i dlnp_i/dx_j + h dH/dx_j = (g_j - p_j (G + h (ln p_j + H))) / T,   G = sum_i g_i
//
// A masked logit has d = -inf and p = 0; its products p d and p ln p are 0 because d is held above kFar there, where 2^d is
// 0 in 32 bits. The exponential itself takes the d that was not held, so that NaN and +inf logits reach s as in SoftmaxAcc.
#pragma once

#include "sfc_rows.cuh"

namespace sfc {

constexpr float kFar = -200.f;
constexpr float kLn2 = 0.6931471805599453f;

// Statistics of what one thread has seen, in two lanes each. m is the true maximum (see SoftmaxAcc).
struct EntropyAcc {
  float m = -FLT_MAX;
  uint64_t s2 = 0, w2 = 0;

  __device__ __forceinline__ void raise(float x, float c) {
    if (x > m) {
      const float d = fmaxf((m - x) * c, kFar), f = ex2_approx(d);
      const uint64_t f2 = pack_f2(f, f);
      w2 = fmul_f2(ffma_f2(pack_f2(d, d), s2, w2), f2);
      s2 = fmul_f2(s2, f2);
      m = x;
    }
  }
  template <int N>
  __device__ __forceinline__ void add_below(const float (&x)[N], float c) {  // none of x is above m
    const uint64_t minus_m = pack_f2(-m, -m), c2 = pack_f2(c, c);
    uint64_t e[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      float a, b;
      unpack_f2(fmul_f2(fadd_f2(pack_f2(x[2 * i], x[2 * i + 1]), minus_m), c2), a, b);
      e[i] = pack_f2(ex2_approx(a), ex2_approx(b));
      w2 = ffma_f2(e[i], pack_f2(fmaxf(a, kFar), fmaxf(b, kFar)), w2);
    }
#pragma unroll
    for (int w = N / 4; w > 0; w /= 2)  // a fixed tree
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] = fadd_f2(e[i], e[i + w]);
    s2 = fadd_f2(s2, e[0]);
  }
  __device__ __forceinline__ void add(float x, float c) {
    raise(x, c);
    const float d = (x - m) * c, e = ex2_approx(d);
    s2 = fadd_f2(s2, pack_f2(e, 0.f));
    w2 = fadd_f2(w2, pack_f2(e * fmaxf(d, kFar), 0.f));
  }
  // U vectors; bf16: one maximum of all of them (see SoftmaxAcc::add). Returns their maximum.
  template <int DT, int U>
  __device__ __forceinline__ float add(const uint4 (&v)[U], float c) {
    constexpr int G = DT == 0 ? U : 1;
    float most = -INFINITY;
#pragma unroll
    for (int g = 0; g < U; g += G) {
      uint4 top = v[g];
#pragma unroll
      for (int u = 1; u < G; ++u) top = larger<DT>(top, v[g + u]);
      const float x_top = Elem<DT>::vmax(top);
      most = fmaxf(most, x_top);
      raise(x_top, c);
#pragma unroll
      for (int u = 0; u < G; ++u) {
        float x[Elem<DT>::kVec];
        Elem<DT>::unpack(v[g + u], x);
        add_below(x, c);
      }
    }
    return most;
  }
};

// The sums of vectors whose logits are known to be near: none above m, |m c| <= kNearTop and |x c| <= kNear for all of them. The
// exponent is one fused step then, d' = x c - M with M = m c rounded: against another reference, which is off by M's rounding
// rho, at most half (2^24 and below have steps of 1), and which `finish` takes out again: 2^rho and its inverse are near 1, and
// w' - rho s' subtracts numbers of the size of half the mass. (Larger references do not do: from 2^31 on 2^rho may be infinite or
// 0.) kNear keeps every d' a number, so that none is held: its exponential is 0 long before.
constexpr float kNearTop = 0x1p24f, kNear = 1e18f;

struct NearAcc {
  uint64_t c2, minus_M2, s2 = 0, w2 = 0;

  __device__ __forceinline__ NearAcc(float m, float c) : c2(pack_f2(c, c)), minus_M2(pack_f2(-(m * c), -(m * c))) {}
  template <int DT>
  __device__ __forceinline__ void add(const uint4& v) {
    constexpr int N = Elem<DT>::kVec;
    float x[N];
    Elem<DT>::unpack(v, x);
    uint64_t e[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint64_t d = ffma_f2(pack_f2(x[2 * i], x[2 * i + 1]), c2, minus_M2);
      float a, b;
      unpack_f2(d, a, b);
      e[i] = pack_f2(ex2_approx(a), ex2_approx(b));
      w2 = ffma_f2(e[i], d, w2);
    }
#pragma unroll
    for (int w = N / 4; w > 0; w /= 2)  // a fixed tree
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] = fadd_f2(e[i], e[i + w]);
    s2 = fadd_f2(s2, e[0]);
  }
  __device__ __forceinline__ void finish(EntropyAcc& a, float m, float c) const {  // a has seen nothing before
    const float rho = fmaf(m, c, -(m * c)), f = ex2_approx(-rho);
    a.m = m;
    a.s2 = fmul_f2(s2, pack_f2(f, f));
    a.w2 = fmul_f2(ffma_f2(pack_f2(-rho, -rho), s2, w2), pack_f2(f, f));
  }
};

template <int DT>
__device__ __forceinline__ uint4 smaller(const uint4& a, const uint4& b) {  // element by element
  auto word = [](uint32_t x, uint32_t y) {
    if constexpr (DT == 0) {
      const __nv_bfloat162 h = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
      return *reinterpret_cast<const uint32_t*>(&h);
    } else {
      return __float_as_uint(fminf(__uint_as_float(x), __uint_as_float(y)));
    }
  };
  return make_uint4(word(a.x, b.x), word(a.y, b.y), word(a.z, b.z), word(a.w, b.w));
}
template <int DT>
__device__ __forceinline__ float vmin(const uint4& v) {
  float x[Elem<DT>::kVec];
  Elem<DT>::unpack(v, x);
#pragma unroll
  for (int i = 1; i < Elem<DT>::kVec; ++i) x[0] = fminf(x[0], x[i]);
  return x[0];
}

// One thread's share (every NT-th) of n vectors in shared memory; by whole warps. The extremes come first: the sums then have no
// rescaling and no step that waits for the one before. A warp takes one form of the sums (of threads that see nothing but a mask's
// fill beside others it would go through both). Returns whether each |x c| is at most kNear.
template <int DT, int NT>
__device__ __forceinline__ bool add_kept(EntropyAcc& a, const uint4* kept, int n, float c) {
  const int tid = threadIdx.x;
  float most = 0.f, least = 0.f;
  if (tid < n) {
    uint4 top = kept[tid], low = top;
#pragma unroll 4
    for (int k = tid + NT; k < n; k += NT) {
      const uint4 v = kept[k];
      top = larger<DT>(top, v);
      low = smaller<DT>(low, v);
    }
    most = Elem<DT>::vmax(top), least = vmin<DT>(low);
  }
  const bool near = fmaxf(fabsf(most * c), fabsf(least * c)) <= kNear;
  const bool short_form = __all_sync(kFull, near && fabsf(most * c) <= kNearTop);
  if (tid >= n) return true;
  if (short_form) {
    NearAcc sums(most, c);
#pragma unroll 4
    for (int k = tid; k < n; k += NT) sums.template add<DT>(kept[k]);
    sums.finish(a, most, c);
  } else {
    a.raise(most, c);
#pragma unroll 2
    for (int k = tid; k < n; k += NT) {
      float x[Elem<DT>::kVec];
      Elem<DT>::unpack(kept[k], x);
      a.add_below(x, c);
    }
  }
  return near;
}

__device__ __forceinline__ void prefetch_l2(const void* from, uint32_t bytes) {  // 16-byte aligned, a multiple of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// x - m over T, as divide(x - m); a difference of finite logits that passes the largest number is taken by halves.
template <class F>
__device__ __forceinline__ float below_max(float x, float m, F divide) {
  const float d = x - m;
  return d == -INFINITY && x > -INFINITY ? divide(0.5f * x - 0.5f * m) * 2.f : divide(d);
}

struct EntropyStats {
  float m, s, w;

  // In 32 bits: no log-probability of the row is smaller than ln s in size (z - max z <= 0), so the rounding is one of the result's.
  __device__ __forceinline__ float log_sum() const { return logf(s); }
  __device__ __forceinline__ float entropy(float ln_s) const { return fmaxf(ln_s - kLn2 * (w / s), 0.f); }
};

// The statistics that the lanes of a warp hold, merged: the same bits in every lane.
__device__ __forceinline__ EntropyStats merge_lanes(const EntropyStats& v, float c) {
  const float m = warp_max(v.m), d = fmaxf((v.m - m) * c, kFar), f = ex2_approx(d);
  return EntropyStats{m, warp_total(v.s * f), warp_total((v.w + d * v.s) * f)};
}
__device__ __forceinline__ EntropyStats merge_lanes(const EntropyAcc& a, float c) {
  float s, t, w, u;
  unpack_f2(a.s2, s, t);
  unpack_f2(a.w2, w, u);
  return merge_lanes(EntropyStats{a.m, s + t, w + u}, c);
}
// One thread's 16 bytes into another CTA's shared memory, counted by that CTA's barrier: the exchange of a cluster's
// statistics without the barrier of the whole cluster, whose release waits for all that its warps have in flight.
__device__ __forceinline__ void dsmem_send(uint32_t addr, const float4& v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}
// n <= 32 statistics in shared memory, merged by a whole warp (the lanes past them repeat the first with no mass).
__device__ __forceinline__ EntropyStats merge_shared(const float4* part, int n, float c) {
  const int lane = threadIdx.x & 31;
  const float4 v = part[lane < n ? lane : 0];
  return merge_lanes(EntropyStats{v.x, lane < n ? v.y : 0.f, lane < n ? v.z : 0.f}, c);
}

__device__ __forceinline__ float held(float x) {  // an overflow is held at the largest number; NaN stays
  return fabsf(x) == INFINITY ? copysignf(FLT_MAX, x) : x;
}
// The dense part of a row's gradient: 2^d (a + b d) = -p (G + h (ln p + H)) scale. Where G or h is large, b times the held d could
// overflow and meet an exponential of 0: a and b are then those of 2^-10 G and 2^-10 h, and the results are lifted by 2^10.
__device__ __forceinline__ bool large(float G, float h) { return !(fabsf(G) + fabsf(h) <= 0x1p100f); }  // (NaN among them)

struct RowGradient {
  float m, c, a, b;
  bool lifted;

  __device__ __forceinline__ RowGradient(const float4& v, bool lifted_) : m(v.x), c(v.y), a(v.z), b(v.w), lifted(lifted_) {}
  // G and h with the factor that is common to the row (an upstream gradient over T) multiplied in already.
  __device__ __forceinline__ RowGradient(float m_, float s, float ln_s, float H, float G, float h, float c_) : m(m_), c(c_) {
    lifted = large(G, h);
    if (lifted) G = held(G) * 0x1p-10f, h = held(h) * 0x1p-10f;
    const float inv_s = 1.f / s;
    a = -fmaf(h, H - ln_s, G) * inv_s;
    b = -h * kLn2 * inv_s;
  }
  __device__ __forceinline__ float at(float x) const {
    const float d = (x - m) * c, g = ex2_approx(d) * fmaf(fmaxf(d, kFar), b, a);
    return lifted ? held(g * 0x1p10f) : g;
  }
  template <int DT>
  __device__ __forceinline__ uint4 vector(const uint4& v) const {  // (not of a lifted row)
    constexpr int N = Elem<DT>::kVec;
    const uint64_t minus_m = pack_f2(-m, -m), c2 = pack_f2(c, c), a2 = pack_f2(a, a), b2 = pack_f2(b, b);
    float x[N];
    Elem<DT>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float d, e;
      unpack_f2(fmul_f2(fadd_f2(pack_f2(x[i], x[i + 1]), minus_m), c2), d, e);
      const uint64_t t = ffma_f2(pack_f2(fmaxf(d, kFar), fmaxf(e, kFar)), b2, a2);
      unpack_f2(fmul_f2(pack_f2(ex2_approx(d), ex2_approx(e)), t), x[i], x[i + 1]);
    }
    return Out<DT>::pack(x);
  }
  // A vector of a lifted row (see write_lifted).
  template <int DT>
  __device__ __forceinline__ uint4 lifted_vector(const uint4& v) const {
    float x[Elem<DT>::kVec];
    Elem<DT>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < Elem<DT>::kVec; ++i) x[i] = at(x[i]);
    return Out<DT>::pack(x);
  }
  // The same for logits that are near (see NearAcc), and moderate factors.
  struct Near {
    uint64_t c2, minus_M2, a2, b2;

    __device__ __forceinline__ explicit Near(const RowGradient& g) {
      // 2^d (a + b d) with d = d' - rho
      const float M = g.m * g.c, rho = fmaf(g.m, g.c, -M), f = ex2_approx(-rho), a = f * fmaf(-g.b, rho, g.a), b = f * g.b;
      c2 = pack_f2(g.c, g.c), minus_M2 = pack_f2(-M, -M), a2 = pack_f2(a, a), b2 = pack_f2(b, b);
    }
    template <int DT>
    __device__ __forceinline__ uint4 vector(const uint4& v) const {
      constexpr int N = Elem<DT>::kVec;
      float x[N];
      Elem<DT>::unpack(v, x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t d = ffma_f2(pack_f2(x[i], x[i + 1]), c2, minus_M2);
        float p, q;
        unpack_f2(d, p, q);
        unpack_f2(fmul_f2(pack_f2(ex2_approx(p), ex2_approx(q)), ffma_f2(d, b2, a2)), x[i], x[i + 1]);
      }
      return Out<DT>::pack(x);
    }
  };
  __device__ __forceinline__ bool moderate() const {
    return fabsf(m * c) <= kNearTop && fabsf(a) <= kNear && fabsf(b) <= kNear && !lifted;
  }
};

// One vector of a gradient row to `to`, which lies `shift` bytes past a 16-byte boundary; by whole warps (see store_shifted).
template <int DT>
__device__ __forceinline__ void store_vector(unsigned char* to, const uint4& w, int shift, bool active) {
  if (DT == 0 && shift != 0) {
    store_shifted(to, w, shift, active);
  } else if (active) {
    if (shift == 0) {
      *reinterpret_cast<uint4*>(to) = w;
    } else {
      uint32_t* four = reinterpret_cast<uint32_t*>(to);
      four[0] = w.x, four[1] = w.y, four[2] = w.z, four[3] = w.w;
    }
  }
}

// The vectors [v0, v1) of a lifted row's gradient, read again and written by a whole CTA, in a loop of its own: rows that hardly
// occur cost the others a uniform branch or two (2048 x 32000 bf16 46.7 us, without them 46.4; x 1000 6.7 and 6.5).
template <int DT, int NT>
__device__ __forceinline__ void write_lifted(const RowGradient& g, const RowSpan<DT>& row, unsigned char* out, int shift, int v0, int v1) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = v0 + static_cast<int>(threadIdx.x); i - lane < v1; i += NT)
    store_vector<DT>(out + static_cast<int64_t>(i) * 16, g.template lifted_vector<DT>(row.body()[min(i, v1 - 1)]), shift, i < v1);
}

}  // namespace sfc
