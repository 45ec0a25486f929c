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
// Two launches, no CTA waits for another:
//  - Statistics: every row is cut into slices, one CTA each, ordered by position. A CTA leaves its slice's softmax
//    statistics in the request's block of the workspace; the last one at a position (an atomic ticket) merges them
//    and decides on the position's draft. A refusal raises the request's stop mark, and the CTAs of later positions
//    that have not started yet skip their rows: those do not matter.
//  - Draw: the vocabulary of each request is cut into slices that race at the position it stopped at (the two rows
//    come from L2 where they still lie there); the last slice merges, writes the outputs and returns the request's
//    block to zero.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"
#include "sfc_verify.cuh"

namespace sfc {
namespace {

constexpr int kStatThreads = 512, kDrawThreads = 256;
constexpr int64_t kStatCtas = 1216, kDrawCtas = 608;  // CTAs wanted: two waves of four a SM; one wave

struct RowStats {  // 16 bytes
  float m, s;
  int32_t argmax;  // greedy rows: the lowest id among the largest logits
  int32_t pad;
};

struct Decision {  // one position of a request, 48 bytes
  RowStats target, draft;
  int32_t code;  // kAccepted, kStopped (draw here) or kBad
  float lp;      // accepted: ln p of the draft
  int32_t pad[2];
};
constexpr int kAccepted = 1, kStopped = 2, kBad = 3;

struct BlockHeader {  // of a request's block
  uint32_t stop;      // kStopBase - (the lowest refused position so far), 0: none
  uint32_t draws;     // ticket of the draw
  uint32_t tickets[SFC_MAX_DRAFTS + 1];
  uint32_t pad;
};
constexpr uint32_t kStopBase = SFC_MAX_DRAFTS + 2;
static_assert(sizeof(Decision) % 16 == 0 && sizeof(BlockHeader) % 16 == 0, "blocks are cut into 16-byte pieces");

// How the work is cut, by sizes alone. At least `kMinVectors` 16-byte vectors a slice.
constexpr int kMaxStatSlices = 16, kMaxDrawSlices = 128, kMinVectors = 512;
struct Cut {
  int stat, draw;                                   // slices per row, per request
  int32_t rec_at, decision_at, best_at, block_bytes;  // a request's block: header, [2D+1][stat], [D+1], [draw]
};
Cut cut_of(int64_t B, int D, int64_t V, int elt) {
  const int64_t vectors = V * elt / 16, rows = B * (2 * D + 1);
  auto slices = [&](int64_t want, int most, int64_t least) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, vectors / least})));
  };
  Cut c;
  c.stat = slices((kStatCtas + rows - 1) / rows, kMaxStatSlices, kMinVectors);
  c.draw = slices((kDrawCtas + B - 1) / B, kMaxDrawSlices, 128);
  c.rec_at = sizeof(BlockHeader);
  c.decision_at = c.rec_at + (2 * D + 1) * c.stat * static_cast<int>(sizeof(RowStats));
  c.best_at = c.decision_at + (D + 1) * static_cast<int>(sizeof(Decision));
  c.block_bytes = (c.best_at + c.draw * static_cast<int>(sizeof(RaceBest)) + 15) & ~15;
  return c;
}

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
  unsigned char* blocks;
  Cut cut;
  VerifyOutputs out;

  __device__ __forceinline__ unsigned char* block(int64_t b) const { return blocks + b * cut.block_bytes; }
  __device__ __forceinline__ BlockHeader* header(int64_t b) const { return reinterpret_cast<BlockHeader*>(block(b)); }
  // Slice records of position j's row: the target's (j <= D), then the draft's.
  __device__ __forceinline__ RowStats* records(int64_t b, bool of_target, int j) const {
    return reinterpret_cast<RowStats*>(block(b) + cut.rec_at) + (of_target ? j : D + 1 + j) * cut.stat;
  }
  __device__ __forceinline__ Decision* decision(int64_t b, int j) const {
    return reinterpret_cast<Decision*>(block(b) + cut.decision_at) + j;
  }
  __device__ __forceinline__ RaceBest* bests(int64_t b) const { return reinterpret_cast<RaceBest*>(block(b) + cut.best_at); }
  __device__ __forceinline__ bool usable(float T) const { return temperature_valid(T) || (greedy_t0 && T == 0.f); }
  __device__ __forceinline__ int drafts(int64_t b) const { return num_drafts ? num_drafts[b] : D; }
  // Whether the request's parameters allow any work.
  __device__ __forceinline__ bool sound(int64_t b, int n) const {
    return n >= 0 && n <= D && usable(temperature[b]) && (!draft || n == 0 || usable(draft_temperature[b]));
  }
};

template <int DT>
__device__ __forceinline__ RowSpan<DT> target_row(const VerifyParams& p, int64_t b, int j) {
  return RowSpan<DT>(p.target, b * p.target_request + j * p.target_row, p.V);
}
template <int DT>
__device__ __forceinline__ RowSpan<DT> draft_row(const VerifyParams& p, int64_t b, int j) {
  return RowSpan<DT>(p.draft, b * p.draft_request + j * p.draft_row, p.V);
}

// ln of the probability of token t, and the probability, in 64 bits: it is compared with a number next to it.
template <int DT>
__device__ __forceinline__ double log_prob(const RowSpan<DT>& row, const RowStats& st, float T, int32_t t) {
  if (T == 0.f) return t == st.argmax ? 0.0 : -INFINITY;
  return (static_cast<double>(row.at(t)) - st.m) / T - log(static_cast<double>(st.s));
}

// A row's statistics from its slice records, by one warp (lane k: slice k).
__device__ __forceinline__ RowStats merge_records(const RowStats* rec, int slices, float c) {
  const int lane = threadIdx.x & 31;
  RowStats v{-FLT_MAX, 0.f, INT32_MAX, 0};
  if (lane < slices) {
    const uint4 w = __ldcg(reinterpret_cast<const uint4*>(rec + lane));
    v = RowStats{__uint_as_float(w.x), __uint_as_float(w.y), static_cast<int32_t>(w.z), 0};
  }
  const float m = warp_max(v.m);
  const float s = warp_total(v.s * ex2_approx((v.m - m) * c));
  const int arg = __reduce_min_sync(kFull, v.m == m ? v.argmax : INT32_MAX);
  return RowStats{m, s, arg, 0};
}

__device__ __forceinline__ float stat_scale(float T) { return T == 0.f ? kLog2e : exponent_scale(T); }

template <int DT>
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float2 red[kStatThreads / 32];
  __shared__ int lowest;
  __shared__ bool last;
  // block index: position, side, request, slice (the earliest positions first)
  const int S = p.cut.stat, sides = p.draft ? 2 : 1;
  unsigned i = blockIdx.x;
  const int slice = static_cast<int>(i % S);
  i /= S;
  const int64_t b = i % static_cast<unsigned>(p.B);
  i /= static_cast<unsigned>(p.B);
  const bool of_target = sides == 1 || i % 2 == 0;
  const int j = static_cast<int>(i / sides), n = p.drafts(b);
  BlockHeader* head = p.header(b);
  if (!p.sound(b, n) || j > n || (!of_target && j == n)) return;  // not part of the request
  const uint32_t stop = *reinterpret_cast<volatile uint32_t*>(&head->stop);
  // past a refusal (one vote: the mark may rise while the CTA's threads read it)
  if (__syncthreads_or(stop != 0 && static_cast<int>(kStopBase - stop) < j)) return;
  const float T = of_target ? p.temperature[b] : p.draft_temperature[b], c = stat_scale(T);
  const RowSpan<DT> row = of_target ? target_row<DT>(p, b, j) : draft_row<DT>(p, b, j);
  const int64_t per = (row.nvec + S - 1) / S, v0 = min(slice * per, row.nvec), v1 = min(v0 + per, row.nvec);
  const SoftmaxStats a = block_stats<kStatThreads>(row_stats<DT, kStatThreads>(row, v0, v1, slice == 0, c), c, red);
  int arg = 0;
  if (T == 0.f) {  // the slice's elements once more, for the lowest id of its maximum
    if (threadIdx.x == 0) lowest = INT32_MAX;
    __syncthreads();
    int mine = INT32_MAX;
    const int64_t e0 = row.head + v0 * Elem<DT>::kVec, e1 = row.head + v1 * Elem<DT>::kVec;
    for (int64_t k = e0 + threadIdx.x; k < e1 && mine == INT32_MAX; k += kStatThreads)
      if (row.at(k) == a.m) mine = static_cast<int>(k);
    if (slice == 0 && static_cast<int>(threadIdx.x) < row.scalars()) {
      const int64_t k = row.scalar_index(threadIdx.x);
      if (row.at(k) == a.m) mine = min(mine, static_cast<int>(k));
    }
    atomicMin(&lowest, mine);
    __syncthreads();
    arg = lowest;
  }
  if (threadIdx.x == 0) {
    p.records(b, of_target, j)[slice] = RowStats{a.m, a.s, arg, 0};
    __threadfence();
    const uint32_t all = static_cast<uint32_t>(S) * (p.draft && j < n ? 2u : 1u);
    last = atomicAdd(&head->tickets[j], 1u) == all - 1;
  }
  __syncthreads();
  if (!last || threadIdx.x >= 32) return;
  __threadfence();
  Decision d{};
  const float Tt = p.temperature[b];
  d.target = merge_records(p.records(b, true, j), S, stat_scale(Tt));
  d.draft = RowStats{0.f, 1.f, INT32_MAX, 0};
  const bool drafted = j < n;
  if (drafted && p.draft) d.draft = merge_records(p.records(b, false, j), S, stat_scale(p.draft_temperature[b]));
  if (threadIdx.x != 0) return;
  d.code = kStopped;
  if (!stats_valid(d.target.m, d.target.s) || !stats_valid(d.draft.m, d.draft.s)) d.code = kBad;
  if (drafted && d.code != kBad) {
    const int32_t t = p.draft_tokens[b * p.D + j];
    if (t < 0 || t >= p.V) {
      d.code = kBad;
    } else {
      const double lp = log_prob<DT>(target_row<DT>(p, b, j), d.target, Tt, t);
      const double q = p.draft ? exp(log_prob<DT>(draft_row<DT>(p, b, j), d.draft, p.draft_temperature[b], t)) : 1.0;
      if (p.uniforms[b * p.D + j] * q < exp(lp)) d.code = kAccepted;
      d.lp = static_cast<float>(lp);
    }
  }
  *p.decision(b, j) = d;
  if (d.code != kAccepted) atomicMax(&head->stop, kStopBase - static_cast<uint32_t>(j));
}

// Elements 8 g .. 8 g + 7 of a row; past its end: -inf.
template <int DT>
__device__ __forceinline__ void load8(const RowSpan<DT>& row, int64_t g, bool aligned, float (&x)[8]) {
  const int64_t i0 = 8 * g;
  if (aligned && i0 + 8 <= row.V) {
    const uint4* at = reinterpret_cast<const uint4*>(row.row + i0 * Elem<DT>::kBytes);
    if constexpr (DT == 0) {
      Elem<0>::unpack(__ldg(at), x);
    } else {
      float lo[4], hi[4];
      Elem<1>::unpack(__ldg(at), lo);
      Elem<1>::unpack(__ldg(at + 1), hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = i0 + e < row.V ? row.at(i0 + e) : -INFINITY;
  }
}

// The race over elements [8 g0, 8 g1). -ln u is estimated first (lg2, absolute error below 2^-22 times ln 2): only
// a weight that could beat the warp's best so far takes the exact logarithm and the division.
template <int DT, bool RESIDUAL>
__device__ __forceinline__ RaceBest race(const VerifyParams& p, const RowSpan<DT>& row, const RowSpan<DT>& qrow,
                                         const RowStats& st, const RowStats& sd, float c, float cd, int32_t certain,
                                         uint32_t counter_row, int64_t g0, int64_t g1) {
  RaceBest best;
  float bar = 0.f;  // of the warp
  const float inv = 1.f / st.s, invd = 1.f / sd.s;
  const bool aligned = (reinterpret_cast<uintptr_t>(row.row) & 15) == 0;
  const bool qaligned = (reinterpret_cast<uintptr_t>(qrow.row) & 15) == 0;
  const int lane = threadIdx.x & 31;
  for (int64_t base = g0 + (threadIdx.x & ~31); base < g1; base += kDrawThreads) {  // uniform over the warp
    const int64_t g = base + lane;
    float w[8];
    if (g < g1) {
      load8(row, g, aligned, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = ex2_approx((w[e] - st.m) * c) * inv;
      if (RESIDUAL) {
        if (certain >= 0) {
          const int64_t off = certain - 8 * g;
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = off == e ? 0.f : w[e];
        } else if (cd == 0.f) {  // a greedy draft
          const int64_t off = sd.argmax - 8 * g;
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = off == e ? fmaxf(w[e] - 1.f, 0.f) : w[e];
        } else {
          float q[8];
          load8(qrow, g, qaligned, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = fmaxf(w[e] - ex2_approx((q[e] - sd.m) * cd) * invd, 0.f);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float most = fmaxf(fmaxf(w[4 * h], w[4 * h + 1]), fmaxf(w[4 * h + 2], w[4 * h + 3]));
        if (!(most > bar * 0x1p-25f)) continue;  // E >= -ln(1 - 2^-24): no word can make it win
        const uint4 block = race_block(p.key, counter_row, static_cast<uint32_t>(2 * g + h));
        const uint32_t words[4] = {block.x, block.y, block.z, block.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = static_cast<float>(2u * (words[e] >> 9) + 1u) * 0x1p-24f;
          const float estimate = fmaf(__log2f(u), -0.693147f, -4e-7f) * 0.99999f;  // at most E
          if (w[4 * h + e] > bar * estimate) best.offer(w[4 * h + e] / -logf(u), static_cast<int32_t>(8 * g + 4 * h + e));
        }
      }
    }
    bar = warp_max(fmaxf(bar, best.ratio));
  }
  return best;
}

template <int DT>
__global__ void __launch_bounds__(kDrawThreads) verify_draw_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int NW = kDrawThreads / 32;
  __shared__ float ratios[NW];
  __shared__ int32_t best_ids[NW];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31, S = p.cut.draw;
  const int slice = static_cast<int>(blockIdx.x % static_cast<unsigned>(S));
  const int64_t b = blockIdx.x / static_cast<unsigned>(S);
  const int n = p.drafts(b);
  const bool sound = p.sound(b, n);
  int a = 0, code = kBad;
  if (sound) {  // the first position that was not accepted
    for (int j0 = 0; j0 <= n; j0 += 32) {
      const int mine = j0 + lane <= n ? __ldcg(&p.decision(b, j0 + lane)->code) : kBad;
      const unsigned open = __ballot_sync(kFull, mine != kAccepted);
      if (open) {
        a = j0 + __ffs(static_cast<int>(open)) - 1;
        code = __shfl_sync(kFull, mine, __ffs(static_cast<int>(open)) - 1);
        break;
      }
    }
  }
  const bool refused = a < n;
  const float T = p.temperature[b];
  const Decision* d = p.decision(b, a);
  const RowStats st = d->target, sd = d->draft;
  const RowSpan<DT> row = target_row<DT>(p, b, a);
  RaceBest best;
  if (code == kStopped && T != 0.f) {
    const int64_t groups = (p.V + 7) / 8, per = (groups + S - 1) / S;
    const int64_t g0 = min(slice * per, groups), g1 = min(g0 + per, groups);
    const float c = exponent_scale(T), Td = p.draft ? p.draft_temperature[b] : 0.f;
    const float cd = Td == 0.f ? 0.f : exponent_scale(Td);
    const uint32_t counter_row = p.row_offset + static_cast<uint32_t>(b);
    const int32_t certain = refused && !p.draft ? p.draft_tokens[b * p.D + a] : -1;
    RaceBest mine;
    if (refused)
      mine = race<DT, true>(p, row, p.draft ? draft_row<DT>(p, b, a) : row, st, sd, c, cd, certain, counter_row, g0, g1);
    else
      mine = race<DT, false>(p, row, row, st, sd, c, cd, -1, counter_row, g0, g1);
    best = block_best<kDrawThreads>(mine, ratios, best_ids);
  }
  if (tid == 0) {
    p.bests(b)[slice] = best;
    __threadfence();
    last = atomicAdd(&p.header(b)->draws, 1u) == static_cast<uint32_t>(S - 1);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  RaceBest mine;
  if (code == kStopped && T != 0.f) {
    for (int k = tid; k < S; k += kDrawThreads) {
      const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p.bests(b) + k));
      mine.offer(__uint_as_float(w.x), static_cast<int32_t>(w.y));
    }
    best = block_best<kDrawThreads>(mine, ratios, best_ids);
    if (best.ratio == 0.f) {  // no residual mass: from the target, by this CTA alone (next to never)
      mine = race<DT, false>(p, row, row, st, sd, exponent_scale(T), 0.f, -1, p.row_offset + static_cast<uint32_t>(b), 0,
                             (p.V + 7) / 8);
      __syncthreads();
      best = block_best<kDrawThreads>(mine, ratios, best_ids);
    }
  }
  const int32_t token = T == 0.f ? st.argmax : best.id;
  float* lps = p.out.token_logprobs + b * (p.D + 1);
  int32_t* tokens = p.out.tokens + b * (p.D + 1);
  for (int j = tid; j <= p.D; j += kDrawThreads) {
    if (code != kStopped) {
      p.out.refuse(b, p.D, j, SFC_ROW_BADPARAM);
    } else if (j == a) {
      tokens[a] = token;
      lps[a] = static_cast<float>(log_prob<DT>(row, st, T, token));
    } else {
      tokens[j] = j < a ? p.draft_tokens[b * p.D + j] : -1;
      lps[j] = j < a ? p.decision(b, j)->lp : 0.f;
    }
  }
  if (tid == 0 && code == kStopped) {
    p.out.accepted[b] = a;
    p.out.row_status[b] = SFC_ROW_OK;
  }
  __syncthreads();  // the block has been read
  uint4* words = reinterpret_cast<uint4*>(p.block(b));
  for (int k = tid; k < p.cut.block_bytes / 16; k += kDrawThreads) words[k] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace
}  // namespace sfc

extern "C" size_t sfc_verify_workspace_size(int64_t B, int32_t D, int64_t V, int dtype) {
  if (B < 1 || B > INT32_MAX || D < 1 || D > SFC_MAX_DRAFTS || V < 1 || V > INT32_MAX ||
      (dtype != SFC_BF16 && dtype != SFC_F32))
    return 0;
  return static_cast<size_t>(B) * sfc::cut_of(B, D, V, dtype == SFC_BF16 ? 2 : 4).block_bytes;
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
  const sfc::Cut cut = sfc::cut_of(B, D, V, dtype == SFC_BF16 ? 2 : 4);
  if (B * (2 * D + 2) * cut.stat > INT32_MAX || B * cut.draw > INT32_MAX) return SFC_EINVAL;  // the grids
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
                            static_cast<uint32_t>(row_offset), static_cast<unsigned char*>(workspace), cut,
                            sfc::VerifyOutputs{accepted, tokens, token_logprobs, row_status}};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned stat = static_cast<unsigned>(B * (D + 1) * (draft_logits ? 2 : 1) * cut.stat);
  const unsigned draw = static_cast<unsigned>(B * cut.draw);
  if (dtype == SFC_BF16) {
    sfc::verify_stats_kernel<0><<<stat, sfc::kStatThreads, 0, st>>>(p);
    sfc::verify_draw_kernel<0><<<draw, sfc::kDrawThreads, 0, st>>>(p);
  } else {
    sfc::verify_stats_kernel<1><<<stat, sfc::kStatThreads, 0, st>>>(p);
    sfc::verify_draw_kernel<1><<<draw, sfc::kDrawThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SFC_OK : SFC_ECUDA;
}
