// Distillation of a student from a teacher's top logits: the loss of each row against a packed teacher
// distribution (a captured support and its log-probabilities, or raw top logits), and its gradient.
//
//   z = x / T, ln p = z - ln sum_V exp z;  t_i = exp(y_i), or softmax over the row's entries of y_i / T
//   loss = sum_i t_i (ln t_i - ln p_i),   dloss/dx_j = (tau p_j - t_j) / T,   tau = sum_i t_i
//
// One CTA per row: the statistics pass streams the row, the teacher's entries gather their logits, and the
// gradient pass reads the row again (from L2 where it still lies there) and writes tau p_j g / T everywhere;
// after a barrier the teacher's entries overwrite theirs with the whole gradient.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"

namespace sfc {
namespace {

struct DistillParams {
  const void* logits;
  int64_t row_stride, V;
  int32_t W;
  bool normalise;
  const float* temperature;
  const int32_t* ids;
  const float* values;
  const int32_t* lengths;
  const float* grad_loss;
  float* loss;
  float4* stats;  // out (forward) or in (backward)
  int32_t* row_status;
  unsigned char* grad;
  int64_t grad_stride;
};

constexpr int kThreads = 512;

// What the gradient needs of a row: its softmax (m, s) and its teacher's (y0, ty): t_i = exp((y_i - y0) a) / ty,
// tau. m is NaN on rows that pass no gradient on (no teacher entry, bad parameters).
struct RowTerms {
  float m, s, tau, y0, ty;
};

// Statistics as they are kept between the forward and the backward call: (m, s, tau, 0), or with normalised
// teachers (tau = 1) (m, s, y0, ty).
__device__ __forceinline__ float4 pack_terms(const RowTerms& t, bool normalise) {
  return normalise ? make_float4(t.m, t.s, t.y0, t.ty) : make_float4(t.m, t.s, t.tau, 0.f);
}
__device__ __forceinline__ RowTerms unpack_terms(const float4& v, bool normalise) {
  return normalise ? RowTerms{v.x, v.y, 1.f, v.z, v.w} : RowTerms{v.x, v.y, v.z, 0.f, 1.f};
}

template <int DT, bool FWD, bool BWD>
__global__ void __launch_bounds__(kThreads) distill_kernel(const __grid_constant__ DistillParams p) {
  constexpr int NW = kThreads / 32, VEC = Elem<DT>::kVec;
  __shared__ float red[6 * NW];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const float T = p.temperature[r];
  const int len = p.lengths[r];
  const int n = min(max(len, 0), p.W);
  const int32_t* ids = p.ids + r * p.W;
  const float* values = p.values + r * p.W;
  const RowSpan<DT> row(p.logits, r * p.row_stride, p.V);
  const float c = exponent_scale(T);
  const float ty_T = p.normalise ? T : 1.f;  // the teacher's temperature
  RowTerms q;
  bool live = true;  // the row has a teacher and passes its checks: uniform over the CTA
  if (FWD) {
    int status = len > p.W ? SFC_ROW_OVERFLOW : SFC_ROW_OK;
    float loss = 0.f;
    if (!temperature_valid(T) || len < 0) {
      status = SFC_ROW_BADPARAM;
    } else if (n > 0) {
      SoftmaxAcc a = row_stats<DT, kThreads>(row, 0, row.nvec, true, c);
      block_merge<kThreads>(a, c, red);
      q = RowTerms{a.m, a.s, 0.f, 0.f, 1.f};
      // the teacher's normaliser
      int bad = !stats_valid(a.m, a.s);
      if (p.normalise) {
        SoftmaxAcc ta;
        const float yc = exponent_scale(T);
        for (int j = tid; j < n; j += kThreads) ta.add(values[j], yc);
        block_merge<kThreads>(ta, yc, red + 2 * NW);
        q.y0 = ta.m;
        q.ty = ta.s;
        bad |= !stats_valid(ta.m, ta.s);
      }
      const float ln_ty = logf(q.ty);
      float sum[2] = {0.f, 0.f};  // tau, sum t (ln t - (x - m) / T)
      for (int j = tid; j < n; j += kThreads) {
        const int32_t id = ids[j];
        const bool in = id >= 0 && id < p.V;
        const float y = (values[j] - q.y0) / ty_T - ln_ty;
        const float x = row.at(in ? id : 0);
        bad |= !in || !(y < INFINITY);
        const float t = expf(y);
        sum[0] += t;
        if (t > 0.f) sum[1] += t * (y - (x - a.m) / T);
      }
      bad = __syncthreads_or(bad);
      block_sum<kThreads, 2>(sum, red + 4 * NW);
      q.tau = p.normalise ? 1.f : sum[0];
      loss = sum[1] + q.tau * logf(a.s);
      if (bad) status = SFC_ROW_BADPARAM;
    }
    live = status != SFC_ROW_BADPARAM && n > 0;
    if (!live) q.m = __int_as_float(0x7fc00000);
    if (tid == 0) {
      p.loss[r] = status == SFC_ROW_BADPARAM ? __int_as_float(0x7fc00000) : loss;
      if (p.row_status) p.row_status[r] = status;
      if (p.stats) p.stats[r] = pack_terms(q, p.normalise);
    }
  } else {
    q = unpack_terms(p.stats[r], p.normalise);
    live = q.m == q.m;
  }
  if (!BWD) return;
  unsigned char* grad = p.grad + r * p.grad_stride * Elem<DT>::kBytes;
  const float g = live ? p.grad_loss[r] / T : 0.f;
  const float k = live ? g * q.tau / q.s : 0.f;
  const float m = live ? q.m : 0.f;
  const bool same = ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(row.row)) & 15) == 0;
  if (!live) {
    for (int64_t i = tid; i < p.V; i += kThreads) Out<DT>::store1(grad, i, 0.f);
    return;
  }
  const uint4* body = row.body();
  uint4* out = reinterpret_cast<uint4*>(grad + static_cast<int64_t>(row.head) * Elem<DT>::kBytes);
  for (int64_t v = tid; v < row.nvec; v += kThreads) {
    float x[VEC];
    Elem<DT>::unpack(__ldg(body + v), x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = k * ex2_approx((x[e] - m) * c);
    if (same) {
      out[v] = Out<DT>::pack(x);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) Out<DT>::store1(grad, row.head + v * VEC + e, x[e]);
    }
  }
  if (tid < row.scalars()) {
    const int64_t i = row.scalar_index(tid);
    Out<DT>::store1(grad, i, k * ex2_approx((row.at(i) - m) * c));
  }
  __syncthreads();  // the dense values are written before the teacher's entries overwrite theirs
  const float ln_ty = logf(q.ty);
  for (int j = tid; j < n; j += kThreads) {
    const int32_t id = ids[j];
    if (id < 0 || id >= p.V) continue;
    const float t = expf((values[j] - q.y0) / ty_T - ln_ty);
    Out<DT>::store1(grad, id, k * ex2_approx((row.at(id) - m) * c) - t * g);
  }
}

int check(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* temperature,
          const int32_t* ids, const float* values, const int32_t* lengths, int32_t W, uint32_t flags) {
  if (!logits || !temperature || !ids || !values || !lengths) return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || row_stride < V) return SFC_EINVAL;
  if (W < 1 || W > SFC_MAX_PACKED_WIDTH) return SFC_EINVAL;
  if (flags & ~static_cast<uint32_t>(SFC_FLAG_NORMALISE_TEACHER)) return SFC_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SFC_BF16 ? 2 : 4)) return SFC_EINVAL;
  return SFC_OK;
}

// The gradient's array: element-aligned, rows that do not overlap, and no byte shared with the logits.
int check_grad(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* grad_loss,
               const void* grad, int64_t grad_stride) {
  const int64_t elt = dtype == SFC_BF16 ? 2 : 4;
  if (!grad_loss || !grad || grad_stride < V) return SFC_EINVAL;
  const uintptr_t g = reinterpret_cast<uintptr_t>(grad), l = reinterpret_cast<uintptr_t>(logits);
  if (g % elt) return SFC_EINVAL;
  const uintptr_t g_end = g + ((B - 1) * grad_stride + V) * elt, l_end = l + ((B - 1) * row_stride + V) * elt;
  return g < l_end && l < g_end ? SFC_EINVAL : SFC_OK;
}

template <bool FWD, bool BWD>
int launch(const DistillParams& p, int dtype, int64_t B, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(B);
  if (dtype == SFC_BF16)
    distill_kernel<0, FWD, BWD><<<grid, kThreads, 0, st>>>(p);
  else
    distill_kernel<1, FWD, BWD><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SFC_OK : SFC_ECUDA;
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_distill_forward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                   const float* temperature, const int32_t* teacher_ids, const float* teacher_values,
                                   const int32_t* lengths, int32_t packed_width, uint32_t flags, float* loss,
                                   float* row_stats, int32_t* row_status, void* stream) {
  const int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                            packed_width, flags);
  if (rc != SFC_OK) return rc;
  if (!loss || !row_status || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, nullptr, loss,
                             reinterpret_cast<float4*>(row_stats), row_status, nullptr, 0};
  return sfc::launch<true, false>(p, dtype, B, stream);
}

extern "C" int sfc_distill_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                    const float* temperature, const int32_t* teacher_ids, const float* teacher_values,
                                    const int32_t* lengths, int32_t packed_width, uint32_t flags,
                                    const float* row_stats, const float* grad_loss, void* grad_logits,
                                    int64_t grad_stride, void* stream) {
  int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                      packed_width, flags);
  if (rc == SFC_OK) rc = sfc::check_grad(logits, dtype, B, V, row_stride, grad_loss, grad_logits, grad_stride);
  if (rc != SFC_OK) return rc;
  if (!row_stats || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, grad_loss, nullptr,
                             const_cast<float4*>(reinterpret_cast<const float4*>(row_stats)), nullptr,
                             static_cast<unsigned char*>(grad_logits), grad_stride};
  return sfc::launch<false, true>(p, dtype, B, stream);
}

extern "C" int sfc_distill_forward_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                            const float* temperature, const int32_t* teacher_ids,
                                            const float* teacher_values, const int32_t* lengths,
                                            int32_t packed_width, uint32_t flags, const float* grad_loss, float* loss,
                                            int32_t* row_status, void* grad_logits, int64_t grad_stride,
                                            void* stream) {
  int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                      packed_width, flags);
  if (rc == SFC_OK) rc = sfc::check_grad(logits, dtype, B, V, row_stride, grad_loss, grad_logits, grad_stride);
  if (rc != SFC_OK) return rc;
  if (!loss || !row_status) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, grad_loss, loss, nullptr, row_status,
                             static_cast<unsigned char*>(grad_logits), grad_stride};
  return sfc::launch<true, true>(p, dtype, B, stream);
}
