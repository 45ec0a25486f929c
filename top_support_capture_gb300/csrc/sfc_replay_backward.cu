// Gradient of the training-side replay (sfc_replay.cu): with lp_i = z_i - ln sum_S exp z_j, z = x / T, an
// upstream gradient g of the sampled token's log-probability and, where it is given, G_i of every member's,
//
//   dL/dx_i = (u_i - pi_i sum_S u) / T,   u_i = G_i + g [i = token],   pi_i = exp lp_i,   i in S
//   dL/dx_i = 0 outside S (the masked positions)
//
// The output is a dense row that is zero almost everywhere: the kernel is bound by writing it. A row is cut over a
// thread-block cluster: each CTA clears its slice while its share of the support's logits is gathered, the cluster
// exchanges the softmax statistics and sum_S u (distributed shared memory), and after its barrier, which also orders
// the zeros, each CTA writes its share of the entries wherever in the row they lie. The first kHeld entries of a
// thread stay in registers in between.
//
// 512 x 151936 bf16, W = 1024: 37 us for 155 MB of rows and 30 MB of gathered logits (DRAM answers in 64 bytes), 0.74
// of the measured copy rate; 256 x 129280 f32, W = 8192: 46 us for 132 + 86 MB. One CTA per row: 42 and 95 us.
#include <cuda_runtime.h>

#include <algorithm>
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
  int32_t slices, per;  // CTAs a row, vectors a slice
};

constexpr int kThreads = 256, kHeld = 8, kMaxSlices = 8;
constexpr int64_t kSliceVectors = 8192, kFillCtas = 1216;

template <int DT>
__global__ void __launch_bounds__(kThreads) replay_backward_kernel(const __grid_constant__ ReplayBackwardParams p) {
  constexpr int NW = kThreads / 32;
  __shared__ float2 red[NW];
  __shared__ float red_u[NW];
  __shared__ float4 table[kMaxSlices];  // (m, s, sum u) of the CTAs
  const int tid = threadIdx.x, lane = tid & 31, S = p.slices, rank = blockIdx.y;
  const int64_t r = blockIdx.x;
  if (S > 1) cluster_arrive();  // its CTAs have started: waited for before the first store into another
  const float T = p.temperature[r];
  const int len = p.lengths[r];
  const int32_t tok = p.tokens[r];
  const float g = p.grad_token[r];
  // rows without a log-probability (their status says why) pass no gradient on
  const int n = temperature_valid(T) && len <= p.W ? max(len, 0) : 0;
  const int32_t* ids = p.ids + r * p.W;
  const float* G = p.grad_entries ? p.grad_entries + r * p.W : nullptr;
  const unsigned char* row = static_cast<const unsigned char*>(p.logits) + r * p.row_stride * Elem<DT>::kBytes;
  const float c = exponent_scale(T);
  const int first = rank * kThreads + tid, step = S * kThreads;
  int32_t id[kHeld];
  float x[kHeld], u[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e) id[e] = first + e * step < n ? ids[first + e * step] : -1;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const bool in = id[e] >= 0 && id[e] < p.V;
    x[e] = in ? Elem<DT>::load1(row, id[e]) : -INFINITY;
    u[e] = in && G ? G[first + e * step] : 0.f;
  }
  // the slice's zeros, while those travel
  const RowSpan<DT> out(p.grad, r * p.grad_stride, p.V);
  unsigned char* grad = const_cast<unsigned char*>(out.row);
  uint4* body = const_cast<uint4*>(out.body());
  const int nvec = static_cast<int>(out.nvec), v0 = min(rank * p.per, nvec), v1 = min(v0 + p.per, nvec);
#pragma unroll 4
  for (int v = v0 + tid; v < v1; v += kThreads) body[v] = make_uint4(0u, 0u, 0u, 0u);
  if (rank == 0 && tid < out.scalars()) Out<DT>::store1(grad, out.scalar_index(tid), 0.f);
  if (n == 0) {  // uniform over the cluster
    if (S > 1) cluster_wait();
    return;
  }
  SoftmaxAcc a;
  float total = 0.f;
  auto fold = [&](int32_t i, float v, float up) {
    if (i < 0 || i >= p.V) v = __int_as_float(0x7fc00000);  // an id outside the row: no gradient
    a.add(v, c);
    total += up + (i == tok ? g : 0.f);
  };
#pragma unroll
  for (int e = 0; e < kHeld; ++e)
    if (first + e * step < n) fold(id[e], x[e], u[e]);
  for (int j = first + kHeld * step; j < n; j += step) {
    const int32_t i = ids[j];
    fold(i, Elem<DT>::load1(row, i >= 0 && i < p.V ? i : 0), G ? G[j] : 0.f);
  }
  const SoftmaxStats w = warp_stats(a, c);
  total = warp_total(total);
  if (lane == 0) {
    red[tid >> 5] = make_float2(w.m, w.s);
    red_u[tid >> 5] = total;
  }
  __syncthreads();  // also orders the CTA's zeros
  SoftmaxStats st = merge_warps<kThreads>(red, c);
  total = warp_total(lane < NW ? red_u[lane] : 0.f);
  if (S > 1) {
    cluster_wait();
    if (tid < S) {
      const uint32_t to = dsmem_addr(&table[rank], tid);
      dsmem_st64(to, pack_f2(st.m, st.s));
      dsmem_st32(to + 8, __float_as_uint(total));
    }
    cluster_sync_all();
    st = SoftmaxStats{table[0].x, table[0].y};
    total = table[0].z;
    for (int k = 1; k < S; ++k) {
      st.merge(table[k].x, table[k].y, c);
      total += table[k].z;
    }
  }
  if (!stats_valid(st.m, st.s)) return;
  const float k = total / st.s;
  auto put = [&](int32_t i, float v, float up) {
    Out<DT>::store1(grad, i, (up + (i == tok ? g : 0.f) - k * ex2_approx((v - st.m) * c)) / T);
  };
#pragma unroll
  for (int e = 0; e < kHeld; ++e)
    if (first + e * step < n) put(id[e], x[e], u[e]);
  for (int j = first + kHeld * step; j < n; j += step) put(ids[j], Elem<DT>::load1(row, ids[j]), G ? G[j] : 0.f);
}

template <int DT>
cudaError_t start(ReplayBackwardParams p, int64_t B, cudaStream_t stream) {
  const int64_t vectors = p.V / Elem<DT>::kVec;
  // slices of about kSliceVectors (128 KB: 64 KB measured 41 us and 256 KB 37 us at 512 x 151936 bf16, 44 and 57 us at
  // 256 x 129280 f32), more where the rows are few
  const int64_t want = std::max((vectors + kSliceVectors - 1) / kSliceVectors, std::min((kFillCtas + B - 1) / B, vectors / 512));
  p.slices = static_cast<int32_t>(std::clamp<int64_t>(want, 1, kMaxSlices));
  p.per = static_cast<int32_t>((vectors + p.slices - 1) / p.slices + 7) & ~7;  // whole 128-byte lines
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B), static_cast<unsigned>(p.slices));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {1, static_cast<unsigned>(p.slices), 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, replay_backward_kernel<DT>, p);
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
                                    static_cast<unsigned char*>(grad_logits), grad_stride, 1, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((dtype == SFC_BF16 ? sfc::start<0>(p, B, st) : sfc::start<1>(p, B, st)) != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}
