// Gradient of the training-side replay (sfc_replay.cu): with lp_i = z_i - ln sum_S exp z_j, z = x / T, an
// upstream gradient g of the sampled token's log-probability and, where it is given, G_i of every member's,
//
//   dL/dx_i = (u_i - pi_i sum_S u) / T,   u_i = G_i + g [i = token],   pi_i = exp lp_i,   i in S
//   dL/dx_i = 0 outside S (the masked positions)
//
// The output is a dense row that is zero almost everywhere: the kernel is bound by writing it.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"

namespace sfc {
namespace {

struct ReplayBackwardParams {
  const void* logits;
  int64_t row_stride, V;
  int32_t W;
  const float* temperature;
  const int32_t* ids;
  const int32_t* lengths;
  const int32_t* tokens;
  const float* grad_token;
  const float* grad_entries;
  unsigned char* grad;
  int64_t grad_stride;
};

constexpr int kThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kThreads) replay_backward_kernel(const __grid_constant__ ReplayBackwardParams p) {
  constexpr int NW = kThreads / 32;
  __shared__ float2 red[NW];
  __shared__ float red_sum[NW];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const float T = p.temperature[r];
  const int n = p.lengths[r];
  const int32_t tok = p.tokens[r];
  const int32_t* ids = p.ids + r * p.W;
  const float* G = p.grad_entries ? p.grad_entries + r * p.W : nullptr;
  const unsigned char* row = static_cast<const unsigned char*>(p.logits) + r * p.row_stride * Elem<DT>::kBytes;
  const RowSpan<DT> out(p.grad, r * p.grad_stride, p.V);
  uint4* body = const_cast<uint4*>(out.body());
  unsigned char* grad = const_cast<unsigned char*>(out.row);
  for (int64_t v = tid; v < out.nvec; v += kThreads) body[v] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < out.scalars()) Out<DT>::store1(grad, out.scalar_index(tid), 0.f);
  // rows without a log-probability (their status says why) pass no gradient on
  if (!temperature_valid(T) || n < 1 || n > p.W) return;
  const float c = exponent_scale(T), g = p.grad_token[r];
  SoftmaxAcc a;
  float sum = 0.f;
  int bad = 0;
  for (int j = tid; j < n; j += kThreads) {
    const int32_t id = ids[j];
    const bool in = id >= 0 && id < p.V;
    bad |= !in;
    a.add(Elem<DT>::load1(row, in ? id : 0), c);
    sum += (G ? G[j] : 0.f) + (id == tok ? g : 0.f);
  }
  const SoftmaxStats st = block_stats<kThreads>(a, c, red);
  const float total = block_total<kThreads>(sum, red_sum);
  if (__syncthreads_or(bad) || !stats_valid(st.m, st.s)) return;  // the barrier also orders the zeros before the values
  const float k = total / st.s;
  for (int j = tid; j < n; j += kThreads) {
    const int32_t id = ids[j];
    const float u = (G ? G[j] : 0.f) + (id == tok ? g : 0.f);
    Out<DT>::store1(grad, id, (u - k * ex2_approx((Elem<DT>::load1(row, id) - st.m) * c)) / T);
  }
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_replay_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                   const float* temperature, const int32_t* support_ids, const int32_t* lengths,
                                   int32_t packed_width, const int32_t* tokens, const float* grad_token_logprob,
                                   const float* grad_support_logprobs, void* grad_logits, int64_t grad_stride,
                                   void* stream) {
  if (!logits || !temperature || !support_ids || !lengths || !tokens || !grad_token_logprob || !grad_logits)
    return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || row_stride < V || grad_stride < V) return SFC_EINVAL;
  if (packed_width < 1 || packed_width > SFC_MAX_PACKED_WIDTH) return SFC_EINVAL;
  const int64_t elt = dtype == SFC_BF16 ? 2 : 4;
  const uintptr_t g = reinterpret_cast<uintptr_t>(grad_logits), l = reinterpret_cast<uintptr_t>(logits);
  if (g % elt || l % elt) return SFC_EINVAL;
  if (g < l + ((B - 1) * row_stride + V) * elt && l < g + ((B - 1) * grad_stride + V) * elt) return SFC_EINVAL;
  const sfc::ReplayBackwardParams p{logits, row_stride, V, packed_width, temperature, support_ids, lengths, tokens,
                                    grad_token_logprob, grad_support_logprobs,
                                    static_cast<unsigned char*>(grad_logits), grad_stride};
  const unsigned grid = static_cast<unsigned>(B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SFC_BF16)
    sfc::replay_backward_kernel<0><<<grid, sfc::kThreads, 0, st>>>(p);
  else
    sfc::replay_backward_kernel<1><<<grid, sfc::kThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SFC_OK : SFC_ECUDA;
}
