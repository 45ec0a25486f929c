// Verification of drafted tokens against full target rows. Per request, with target rows t_0 .. t_n and draft
// rows d_0 .. d_{n-1} (n <= D drafts), p_j = softmax(t_j / T), q_j = softmax(d_j / T_d) or, without draft rows,
// certainty of the drafted token:
//
//   draft j is accepted while u_j q_j(x_j) < p_j(x_j), in order; a = the number accepted
//   the next token is drawn from max(p_a - q_a, 0) when a < n (from p_a where that leaves no mass), else from p_n
//
// so that the tokens are distributed as if they had been drawn from the target one by one (Leviathan et al.,
// "Fast Inference from Transformers via Speculative Decoding", 2023, theorem 1; Chen et al., 2023).
//
// Two launches: one CTA per row leaves its softmax statistics in the workspace, then one CTA per request walks
// the drafts and draws over the vocabulary at the position it stopped at.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"
#include "sfc_verify.cuh"

namespace sfc {
namespace {

struct RowStats {  // 16 bytes
  float m, s;
  int32_t argmax;  // greedy rows: the lowest id among the largest logits
  int32_t pad;
};

struct VerifyParams {
  const void* target;
  const void* draft;  // null: every draft is certain
  int64_t V, target_request, target_row, draft_request, draft_row;
  int32_t B, D;
  bool greedy_t0;
  const float* temperature;
  const float* draft_temperature;
  const int32_t* draft_tokens;
  const int32_t* num_drafts;
  const float* uniforms;
  RaceKey key;
  uint32_t row_offset;
  RowStats* stats;  // [B, 2 D + 1]: the target's rows, then the draft's
  VerifyOutputs out;

  __device__ __forceinline__ bool is_target(int j) const { return j <= D; }
  __device__ __forceinline__ bool usable(float T) const { return temperature_valid(T) || (greedy_t0 && T == 0.f); }
  __device__ __forceinline__ int drafts(int64_t b) const { return num_drafts ? num_drafts[b] : D; }
  __device__ __forceinline__ float temp(int64_t b, bool of_target) const { return of_target ? temperature[b] : draft_temperature[b]; }
};

template <int DT>
__device__ __forceinline__ RowSpan<DT> target_row(const VerifyParams& p, int64_t b, int j) {
  return RowSpan<DT>(p.target, b * p.target_request + j * p.target_row, p.V);
}
template <int DT>
__device__ __forceinline__ RowSpan<DT> draft_row(const VerifyParams& p, int64_t b, int j) {
  return RowSpan<DT>(p.draft, b * p.draft_request + j * p.draft_row, p.V);
}

constexpr int kThreads = 512;

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int NW = kThreads / 32;
  __shared__ float2 red[NW];
  __shared__ int lowest;
  const int rows = p.draft ? 2 * p.D + 1 : p.D + 1;
  const int64_t b = blockIdx.x / rows;
  const int i = static_cast<int>(blockIdx.x % rows);
  const bool of_target = p.is_target(i);
  const int j = of_target ? i : i - p.D - 1, n = p.drafts(b);
  const float T = p.temp(b, of_target);
  if (n < 0 || n > p.D || j > n || (!of_target && j == n) || !p.usable(T)) return;  // not part of the request
  const RowSpan<DT> row = of_target ? target_row<DT>(p, b, j) : draft_row<DT>(p, b, j);
  const float c = T == 0.f ? kLog2e : exponent_scale(T);
  const SoftmaxStats a = block_stats<kThreads>(row_stats<DT, kThreads>(row, 0, row.nvec, true, c), c, red);
  int arg = 0;
  if (T == 0.f) {
    if (threadIdx.x == 0) lowest = INT32_MAX;
    __syncthreads();
    int mine = INT32_MAX;
    for (int64_t k = threadIdx.x; k < p.V && mine == INT32_MAX; k += kThreads)
      if (row.at(k) == a.m) mine = static_cast<int>(k);
    atomicMin(&lowest, mine);
    __syncthreads();
    arg = lowest;
  }
  if (threadIdx.x == 0) p.stats[b * (2 * p.D + 1) + i] = RowStats{a.m, a.s, arg, 0};
}

// ln of the probability of token t, and the probability, in 64 bits: it is compared with a number next to it.
template <int DT>
__device__ __forceinline__ double log_prob(const RowSpan<DT>& row, const RowStats& st, float T, int32_t t) {
  if (T == 0.f) return t == st.argmax ? 0.0 : -INFINITY;
  return (static_cast<double>(row.at(t)) - st.m) / T - log(static_cast<double>(st.s));
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int NW = kThreads / 32;
  __shared__ float ratios[NW];
  __shared__ int32_t best_ids[NW];
  __shared__ int sh_a, sh_status;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x;
  const int n = p.drafts(b);
  const RowStats* stats = p.stats + b * (2 * p.D + 1);
  const float T = p.temperature[b], Td = p.draft ? p.draft_temperature[b] : 0.f;
  const int32_t* drafted = p.draft_tokens + b * p.D;
  float* lps = p.out.token_logprobs + b * (p.D + 1);
  int32_t* tokens = p.out.tokens + b * (p.D + 1);
  if (tid == 0) {
    int status = SFC_ROW_OK, a = 0;
    if (n < 0 || n > p.D || !p.usable(T) || (p.draft && n > 0 && !p.usable(Td))) status = SFC_ROW_BADPARAM;
    while (status == SFC_ROW_OK) {
      const RowStats st = stats[a];
      if (!stats_valid(st.m, st.s)) status = SFC_ROW_BADPARAM;
      if (a == n || status != SFC_ROW_OK) break;
      const int32_t t = drafted[a];
      const RowStats sd = p.draft ? stats[p.D + 1 + a] : RowStats{0.f, 1.f, 0, 0};
      if (t < 0 || t >= p.V || !stats_valid(sd.m, sd.s)) {
        status = SFC_ROW_BADPARAM;
        break;
      }
      const double lp = log_prob<DT>(target_row<DT>(p, b, a), st, T, t);
      const double q = p.draft ? exp(log_prob<DT>(draft_row<DT>(p, b, a), sd, Td, t)) : 1.0;
      if (!(p.uniforms[b * p.D + a] * q < exp(lp))) break;
      tokens[a] = t;
      lps[a] = static_cast<float>(lp);
      ++a;
    }
    sh_a = a;
    sh_status = status;
  }
  __syncthreads();
  const int a = sh_a;
  if (sh_status != SFC_ROW_OK) {
    for (int j = tid; j <= p.D; j += kThreads) p.out.refuse(b, p.D, j, sh_status);
    return;
  }
  const RowStats st = stats[a];
  const RowSpan<DT> row = target_row<DT>(p, b, a);
  int32_t token = st.argmax;
  if (T != 0.f) {
    const bool refused = a < n;
    const int32_t refused_token = refused ? drafted[a] : -1;
    const float c = exponent_scale(T), inv = 1.f / st.s;
    const bool with_q = refused && p.draft;
    const RowStats sd = with_q ? stats[p.D + 1 + a] : RowStats{0.f, 1.f, -1, 0};
    const RowSpan<DT> qrow = with_q ? draft_row<DT>(p, b, a) : row;
    const float cd = Td == 0.f ? 0.f : exponent_scale(Td), invd = 1.f / sd.s;
    const uint32_t counter_row = p.row_offset + static_cast<uint32_t>(b);
    RaceBest best;
    for (int pass = 0; pass < 2 && best.ratio == 0.f; ++pass) {  // the second: no residual mass
      RaceBest mine;
      for (int64_t quad = tid; 4 * quad < p.V; quad += kThreads) {
        const uint4 w4 = race_block(p.key, counter_row, static_cast<uint32_t>(quad));
        const uint32_t words[4] = {w4.x, w4.y, w4.z, w4.w};
        for (int e = 0; e < 4; ++e) {
          const int64_t i = 4 * quad + e;
          if (i >= p.V) break;
          float w = ex2_approx((row.at(i) - st.m) * c) * inv;
          if (pass == 0 && refused) {
            const float q = !p.draft ? (i == refused_token ? INFINITY : 0.f)
                            : Td == 0.f ? (i == sd.argmax ? 1.f : 0.f)
                                        : ex2_approx((qrow.at(i) - sd.m) * cd) * invd;
            w = fmaxf(w - q, 0.f);
          }
          mine.offer(w / race_wait(words[e]), static_cast<int32_t>(i));
        }
      }
      __syncthreads();
      best = block_best<kThreads>(mine, ratios, best_ids);
    }
    token = best.id;
  }
  for (int j = a + 1 + tid; j <= p.D; j += kThreads) {
    tokens[j] = -1;
    lps[j] = 0.f;
  }
  if (tid == 0) {
    tokens[a] = token;
    lps[a] = static_cast<float>(log_prob<DT>(row, st, T, token));
    p.out.accepted[b] = a;
    p.out.row_status[b] = SFC_ROW_OK;
  }
}

}  // namespace
}  // namespace sfc

extern "C" size_t sfc_verify_workspace_size(int64_t B, int32_t D, int64_t V, int dtype) {
  if (B < 1 || B > INT32_MAX || D < 1 || D > SFC_MAX_DRAFTS || V < 1 || V > INT32_MAX ||
      (dtype != SFC_BF16 && dtype != SFC_F32))
    return 0;
  return static_cast<size_t>(B) * (2 * D + 1) * sizeof(sfc::RowStats);
}

extern "C" int sfc_verify_drafts(const void* target_logits, const void* draft_logits, int dtype, int64_t B, int32_t D,
                                 int64_t V, int64_t target_request_stride, int64_t target_row_stride,
                                 int64_t draft_request_stride, int64_t draft_row_stride, const float* temperature,
                                 const float* draft_temperature, const int32_t* draft_tokens,
                                 const int32_t* num_drafts, const float* uniforms, uint64_t seed, uint64_t step,
                                 int64_t row_offset, uint32_t flags, int32_t* accepted, int32_t* tokens,
                                 float* token_logprobs, int32_t* row_status, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!target_logits || !temperature || !draft_tokens || !uniforms || !accepted || !tokens || !token_logprobs ||
      !row_status)
    return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || D < 1 || D > SFC_MAX_DRAFTS) return SFC_EINVAL;
  if (B * (2 * D + 1) > INT32_MAX) return SFC_EINVAL;  // the grid
  if (target_request_stride < 0 || target_row_stride < 0 || draft_request_stride < 0 || draft_row_stride < 0) return SFC_EINVAL;
  if (row_offset < 0 || row_offset + B > (int64_t{1} << 32)) return SFC_EINVAL;
  if (flags & ~static_cast<uint32_t>(SFC_FLAG_GREEDY_T0)) return SFC_EINVAL;
  const uintptr_t elt = dtype == SFC_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(target_logits) % elt || reinterpret_cast<uintptr_t>(draft_logits) % elt ||
      reinterpret_cast<uintptr_t>(workspace) % 16)
    return SFC_EINVAL;
  if (!workspace || workspace_bytes < sfc_verify_workspace_size(B, D, V, dtype)) return SFC_EWORKSPACE;
  const sfc::VerifyParams p{target_logits, draft_logits, V, target_request_stride, target_row_stride,
                            draft_request_stride, draft_row_stride, static_cast<int32_t>(B), D,
                            (flags & SFC_FLAG_GREEDY_T0) != 0, temperature,
                            draft_temperature ? draft_temperature : temperature, draft_tokens, num_drafts, uniforms,
                            sfc::RaceKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
                                         static_cast<uint32_t>(step), static_cast<uint32_t>(step >> 32)},
                            static_cast<uint32_t>(row_offset), static_cast<sfc::RowStats*>(workspace),
                            sfc::VerifyOutputs{accepted, tokens, token_logprobs, row_status}};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned rows = static_cast<unsigned>(B * (draft_logits ? 2 * D + 1 : D + 1)), reqs = static_cast<unsigned>(B);
  if (dtype == SFC_BF16) {
    sfc::verify_stats_kernel<0><<<rows, sfc::kThreads, 0, st>>>(p);
    sfc::verify_draw_kernel<0><<<reqs, sfc::kThreads, 0, st>>>(p);
  } else {
    sfc::verify_stats_kernel<1><<<rows, sfc::kThreads, 0, st>>>(p);
    sfc::verify_draw_kernel<1><<<reqs, sfc::kThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SFC_OK : SFC_ECUDA;
}
