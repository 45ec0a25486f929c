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
//  - Statistics: the two rows of every position are cut into slices, one CTA each, ordered by position. A CTA leaves
//    its slice's softmax statistics in the request's block of the workspace; the last one at a position (an atomic
//    ticket) merges them and decides on the position's draft. A refusal raises the request's stop mark; where the CTAs
//    are more than run at once (a row is one slice then), those of later positions that have not started yet skip their
//    rows: those do not matter.
//  - Draw: the vocabulary of each request is cut into slices that race at the position it stopped at (the two rows
//    come from L2 where they still lie there); the last slice merges, writes the outputs and returns the request's
//    block to zero.
// 64 requests x 4 drafts x 151936 bf16: 57 us as called. Profiled one by one from cold caches the statistics take 34
// (175 MB at 5.1 TB/s: what one wave of streaming CTAs reaches with its start and its end; a warp waits for memory in nine
// cycles of fourteen) and the draw 29. Of the draw's time the SMs have work in 70 % (576 CTAs in 608 places, uneven at the
// end), and one that has issues in 61 % of its cycles: 64 registers leave it 6.4 warps a scheduler, and of a warp's 10.4
// cycles an instruction 1.9 pass waiting for the one before (Philox is a chain of products), 1.2 for an arithmetic pipe, 1.1
// at a barrier. One request: 13.9 us, two chains of dependent steps (parameters, rows, merge, ticket, decision; decision,
// rows, race, ticket, outputs). Tried: the statistics in a launch for every two positions, the later ones skipping
// refused requests: 73 us, each launch adds more than it saves; slices of a third of a row in 2.3 waves: 59 us.
#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"
#include "sfc_verify.cuh"

namespace sfc {
namespace {

constexpr int kStatThreads = 512, kStatUnroll = 4, kDrawThreads = 256;
constexpr int64_t kSlots = 304;  // CTAs of statistics that a GB300 runs at once: two a SM
constexpr int64_t kDrawCtas = 608;  // of the draw, four a SM

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
constexpr int kMaxStatSlices = 32, kMaxDrawSlices = 128, kMinVectors = 512;
struct Cut {
  int stat, draw;                                     // slices per row, per request
  bool waves;                                         // more CTAs of statistics than run at once
  int32_t stat_per, draw_per;                         // vectors of a slice, groups of 8 elements of a slice
  int32_t rec_at, decision_at, best_at, block_bytes;  // a request's block: header, [2D+1][stat], [D+1], [draw]
};
Cut cut_of(int64_t B, int D, int64_t V, int elt) {
  const int64_t vectors = V * elt / 16, rows = B * (D + 1);
  auto slices = [&](int64_t want, int most, int64_t least) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, vectors / least})));
  };
  Cut c;
  c.stat = slices(kSlots / rows, kMaxStatSlices, kMinVectors);  // one wave where the rows allow
  c.draw = slices(kDrawCtas / B, kMaxDrawSlices, 128);
  const int64_t groups = (V + 7) / 8, per = (groups + c.draw - 1) / c.draw;
  c.draw_per = static_cast<int32_t>((per + kDrawThreads - 1) / kDrawThreads * kDrawThreads);  // a group for every thread
  c.draw = static_cast<int>((groups + c.draw_per - 1) / c.draw_per);
  c.waves = rows * c.stat > kSlots;
  c.stat_per = static_cast<int32_t>((vectors + c.stat - 1) / c.stat);
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
  int32_t D;
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

// ln of the probability of token t from its logit x, given the mass in 32 bits. What is emitted is taken in 32 bits (each of
// x - m, its quotient, ln s and the difference rounds once: 4e-8 relative in all against 64 bits, where one thread's 64-bit
// logarithm would cost a microsecond); what has to decide against a number next to it, in 64.
__device__ __forceinline__ float log_prob(float x, const RowStats& st, float T, int32_t t) {
  if (T == 0.f) return t == st.argmax ? 0.f : -INFINITY;
  return (x - st.m) / T - logf(st.s);
}
__device__ __noinline__ double log_prob_exact(float x, const RowStats& st, float T, int32_t t) {
  if (T == 0.f) return t == st.argmax ? 0.0 : -INFINITY;
  return (static_cast<double>(x) - st.m) / T - log(static_cast<double>(st.s));
}

// u q < p.
__device__ __forceinline__ bool accepts(float u, float x, const RowStats& st, float T, float y, const RowStats& sd,
                                        float Td, bool certain, int32_t t) {
  const float left = certain ? u : u * expf(log_prob(y, sd, Td, t)), right = expf(log_prob(x, st, T, t));
  if (fabsf(left - right) > 0x1p-14f * fmaxf(left, right) && right > 0x1p-100f) return left < right;
  return u * (certain ? 1.0 : exp(log_prob_exact(y, sd, Td, t))) < exp(log_prob_exact(x, st, T, t));
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

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float stat_scale(float T) { return T == 0.f ? kLog2e : exponent_scale(T); }

template <int DT>
__global__ void __launch_bounds__(kStatThreads, 2) verify_stats_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int VEC = Elem<DT>::kVec, NW = kStatThreads / 32;
  __shared__ float2 red[2 * NW];
  __shared__ int lowest[2];
  // grid: request, slice, position (the earliest first); a CTA takes its slice of both rows of a position
  const int S = p.cut.stat, slice = blockIdx.y, j = blockIdx.z;
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, n = p.drafts(b);
  BlockHeader* head = p.header(b);
  if (!p.cut.waves) launch_dependents();
  const RowSpan<DT> row = target_row<DT>(p, b, j);
  auto first = [&](const RowSpan<DT>& r) { return min(slice * p.cut.stat_per, static_cast<int>(r.nvec)); };
  auto end = [&](const RowSpan<DT>& r) { return min((slice + 1) * p.cut.stat_per, static_cast<int>(r.nvec)); };
  RowStream<DT, kStatThreads, kStatUnroll> stream(row, first(row), end(row));  // on its way while the parameters load
  if (!p.sound(b, n) || j > n) return;  // not part of the request
  if (p.cut.waves) {
    // past a refusal (one vote: the mark may rise while the CTA's threads read it)
    const uint32_t stop = *reinterpret_cast<volatile uint32_t*>(&head->stop);
    if (__syncthreads_or(stop != 0 && static_cast<int>(kStopBase - stop) < j)) return;
  }
  const bool drafted = j < n, certain = !p.draft, two = drafted && !certain;
  const float Tt = p.temperature[b], Td = certain ? 0.f : p.draft_temperature[b], ct = stat_scale(Tt), cd = stat_scale(Td);
  const RowSpan<DT> qrow = two ? draft_row<DT>(p, b, j) : row;
  // the draft's token and logits, on their way long before the decision
  const int32_t t = drafted ? p.draft_tokens[b * p.D + j] : 0;
  const bool in = t >= 0 && t < p.V;
  float u = 0.f, x = 0.f, y = 0.f;
  if (drafted && tid == 0) {
    u = p.uniforms[b * p.D + j];
    x = row.at(in ? t : 0);
    if (two) y = qrow.at(in ? t : 0);
  }
  // one side's statistics into the warp's place
  auto fold = [&](RowStream<DT, kStatThreads, kStatUnroll>& from, int side) {
    const RowSpan<DT>& r = side ? qrow : row;
    const float c = side ? cd : ct;
    SoftmaxAcc acc;
    from.batches([&](const uint4 (&v)[kStatUnroll]) { acc.template add<DT>(v, c); });
    if (slice == 0 && tid < r.scalars()) acc.add(r.at(r.scalar_index(tid)), c);
    const SoftmaxStats w = warp_stats(acc, c);
    if (lane == 0) red[side * NW + (tid >> 5)] = make_float2(w.m, w.s);
  };
  fold(stream, 0);
  if (two) {
    RowStream<DT, kStatThreads, kStatUnroll> from(qrow, first(qrow), end(qrow));
    fold(from, 1);
  }
  if (tid < 2) lowest[tid] = INT32_MAX;
  __syncthreads();
  const bool greedy = Tt == 0.f || (two && Td == 0.f);
  if (greedy) {  // the slice once more, for the lowest id of its maximum
    for (int side = Tt == 0.f ? 0 : 1; side < (two && Td == 0.f ? 2 : 1); ++side) {
      const RowSpan<DT>& r = side ? qrow : row;
      const float m = merge_warps<kStatThreads>(red + side * NW, side ? cd : ct).m;
      int mine = INT32_MAX;
      RowStream<DT, kStatThreads, kStatUnroll> from(r, first(r), end(r));
      from.each([&](const uint4& v, int at) {
        float x[VEC];
        Elem<DT>::unpack(v, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (x[e] == m && at < end(r)) mine = min(mine, r.head + at * VEC + e);
      });
      if (slice == 0 && tid < r.scalars()) {
        const int64_t k = r.scalar_index(tid);
        if (r.at(k) == m) mine = min(mine, static_cast<int>(k));
      }
      atomicMin(&lowest[side], mine);
    }
    __syncthreads();
  }
  if (tid >= 32) return;  // the first warp closes the slice, and the last slice's the position
  Decision d{};
  const SoftmaxStats at = merge_warps<kStatThreads>(red, ct);
  d.target = RowStats{at.m, at.s, lowest[0], 0};
  d.draft = RowStats{0.f, 1.f, INT32_MAX, 0};
  if (two) {
    const SoftmaxStats ad = merge_warps<kStatThreads>(red + NW, cd);
    d.draft = RowStats{ad.m, ad.s, lowest[1], 0};
  }
  if (S > 1) {
    int last = 0;
    if (lane == 0) {
      p.records(b, true, j)[slice] = d.target;
      if (two) p.records(b, false, j)[slice] = d.draft;
      __threadfence();
      last = atomicAdd(&head->tickets[j], 1u) == static_cast<uint32_t>(S - 1);
    }
    if (!__shfl_sync(kFull, last, 0)) return;
    __threadfence();
  }
  if (S > 1) {
    d.target = merge_records(p.records(b, true, j), S, ct);
    if (two) d.draft = merge_records(p.records(b, false, j), S, cd);
  }
  if (threadIdx.x != 0) return;
  d.code = kStopped;
  if (!in || !stats_valid(d.target.m, d.target.s) || !stats_valid(d.draft.m, d.draft.s)) {
    d.code = kBad;
  } else if (drafted) {
    if (accepts(u, x, d.target, Tt, y, d.draft, Td, certain, t)) d.code = kAccepted;
    d.lp = log_prob(x, d.target, Tt, t);
  }
  *p.decision(b, j) = d;
  if (d.code != kAccepted) atomicMax(&head->stop, kStopBase - static_cast<uint32_t>(j));
}

// Elements 8 g .. 8 g + 7 of a row as they lie in memory (16-byte loads where the row allows, else one by one);
// past its end: -inf.
template <int DT>
struct Eight {
  static constexpr int N = DT == 0 ? 1 : 2;
  uint4 v[N];

  __device__ __forceinline__ void load(const RowSpan<DT>& row, int64_t g, bool aligned) {
    const int64_t i0 = 8 * g;
    if (aligned && i0 + 8 <= row.V) {
      const uint4* at = reinterpret_cast<const uint4*>(row.row + i0 * Elem<DT>::kBytes);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = ld_once(at + k);
    } else {
      uint32_t w[4 * N];
#pragma unroll
      for (int k = 0; k < 4 * N; ++k) {
        if constexpr (DT == 0) {
          const uint32_t lo = i0 + 2 * k < row.V ? __float_as_uint(row.at(i0 + 2 * k)) : 0xFF800000u;
          const uint32_t hi = i0 + 2 * k + 1 < row.V ? __float_as_uint(row.at(i0 + 2 * k + 1)) : 0xFF800000u;
          w[k] = (lo >> 16) | hi;
        } else {
          w[k] = i0 + k < row.V ? __float_as_uint(row.at(i0 + k)) : 0xFF800000u;
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (DT == 0) {
      Elem<0>::unpack(v[0], x);
    } else {
      float lo[4], hi[4];
      Elem<1>::unpack(v[0], lo);
      Elem<1>::unpack(v[1], hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
    }
  }
};

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The race over elements [8 g0, 8 g1). E = -ln u is estimated from lg2 (absolute error below 2^-22); an element
// takes the exact logarithm and the division only if its weight, over the least E that the estimate allows, reaches
// the warp's bar. The bar is the best ratio so far, at first the largest that the estimates guarantee: about one
// element of a warp's first 256 passes, and ever fewer later. What is left is the noise itself: ten rounds for four
// elements.
template <int DT, bool RESIDUAL>
__device__ __forceinline__ RaceBest race(const VerifyParams& p, const RowSpan<DT>& row, const RowSpan<DT>& qrow,
                                         const RowStats& st, const RowStats& sd, float c, float cd, int32_t certain,
                                         uint32_t counter_row, int64_t g0, int64_t g1) {
  RaceBest best;
  float bar = 0.f;  // of the warp
  const float inv = 1.f / st.s, invd = 1.f / sd.s;
  const uint64_t m2 = pack_f2(-st.m, -st.m), c2 = pack_f2(c, c), inv2 = pack_f2(inv, inv);
  const uint64_t md2 = pack_f2(-sd.m, -sd.m), cd2 = pack_f2(cd, cd), invd2 = pack_f2(-invd, -invd);
  const bool aligned = (reinterpret_cast<uintptr_t>(row.row) & 15) == 0;
  const bool qaligned = (reinterpret_cast<uintptr_t>(qrow.row) & 15) == 0;
  const bool two = RESIDUAL && certain < 0 && cd != 0.f;
  const int lane = threadIdx.x & 31;
  Eight<DT> tx, qx;  // of the coming group
  if (g0 + threadIdx.x < g1) {
    tx.load(row, g0 + threadIdx.x, aligned);
    if (two) qx.load(qrow, g0 + threadIdx.x, qaligned);
  }
  for (int64_t base = g0 + (threadIdx.x & ~31); base < g1; base += kDrawThreads) {  // uniform over the warp
    const int64_t g = base + lane;
    float w[8], u[8], most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.f;
    if (g < g1) {
      float x[8];
      uint64_t e2[4];
      tx.values(x);
      exponentials(x, m2, c2, e2);
#pragma unroll
      for (int i = 0; i < 4; ++i) e2[i] = fmul_f2(e2[i], inv2);
      if (two) {
        uint64_t q2[4];
        qx.values(x);
        exponentials(x, md2, cd2, q2);
#pragma unroll
        for (int i = 0; i < 4; ++i) e2[i] = fadd_f2(e2[i], fmul_f2(q2[i], invd2));  // (fused, equal p and q would leave a rounding)
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack_f2(e2[i], w[2 * i], w[2 * i + 1]);
      if (g + kDrawThreads < g1) {
        tx.load(row, g + kDrawThreads, aligned);
        if (two) qx.load(qrow, g + kDrawThreads, qaligned);
      }
      if (RESIDUAL && !two) {  // all of the draft's mass on one token
        const int64_t off = (certain >= 0 ? certain : sd.argmax) - 8 * g;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = off == e ? w[e] - 1.f : w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, w[e]);
    }
    // E >= -ln(1 - 2^-24): where every weight is too small, no word can make one win
    if (!__any_sync(kFull, most > bar * 0x1p-25f)) continue;
    bool pass = false;
    float reach = 0.f;  // the largest ratio that is certain
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 block = race_block(p.key, counter_row, static_cast<uint32_t>(2 * g + h));
      const uint32_t words[4] = {block.x, block.y, block.z, block.w};
#pragma unroll
      for (int e = 4 * h; e < 4 * h + 4; ++e) {
        u[e] = race_unit(words[e - 4 * h]);
        const float l = lg2_approx(u[e]);
        pass |= w[e] > 0.f && w[e] >= bar * fmaf(l, -0.69314f, -4e-7f);
        if (bar == 0.f) reach = fmaxf(reach, w[e] * rcp_approx(fmaf(l, -0.69316f, 4e-7f)));
      }
    }
    if (!__any_sync(kFull, pass)) continue;
    if (bar == 0.f) bar = warp_max(reach) * 0.99999f;
    if (pass) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (w[e] > 0.f && w[e] >= bar * fmaf(lg2_approx(u[e]), -0.69314f, -4e-7f))
          best.offer(w[e] / -logf(u[e]), static_cast<int32_t>(8 * g + e));
      }
    }
    bar = fmaxf(bar, warp_max(best.ratio));
  }
  return best;
}

template <int DT>
__global__ void __launch_bounds__(kDrawThreads, 4) verify_draw_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int NW = kDrawThreads / 32;
  __shared__ float ratios[NW];
  __shared__ int32_t best_ids[NW];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31, S = p.cut.draw;
  const int slice = blockIdx.y;
  const int64_t b = blockIdx.x;
  const int n = p.drafts(b);
  const bool sound = p.sound(b, n);
  int a = 0, code = kBad;
  RowStats st{}, sd{};
  wait_for_primary();
  if (sound) {  // the first position that was not accepted, one position a lane
    for (int j0 = 0; j0 <= n; j0 += 32) {
      const uint4* at = reinterpret_cast<const uint4*>(p.decision(b, min(j0 + lane, n)));
      const uint4 w0 = __ldcg(at), w1 = __ldcg(at + 1), w2 = __ldcg(at + 2);
      const int mine = j0 + lane <= n ? static_cast<int>(w2.x) : kBad;
      const unsigned open = __ballot_sync(kFull, mine != kAccepted);
      if (open) {
        const int k = __ffs(static_cast<int>(open)) - 1;
        a = j0 + k;
        code = __shfl_sync(kFull, mine, k);
        auto take = [&](const uint4& w) {
          return RowStats{__uint_as_float(__shfl_sync(kFull, w.x, k)), __uint_as_float(__shfl_sync(kFull, w.y, k)),
                          static_cast<int32_t>(__shfl_sync(kFull, w.z, k)), 0};
        };
        st = take(w0);
        sd = take(w1);
        break;
      }
    }
  }
  const bool refused = a < n;
  const float T = p.temperature[b];
  const RowSpan<DT> row = target_row<DT>(p, b, a);
  RaceBest best;
  if (code == kStopped && T != 0.f) {
    const int64_t groups = (p.V + 7) / 8;
    const int64_t g0 = min(static_cast<int64_t>(slice) * p.cut.draw_per, groups), g1 = min(g0 + p.cut.draw_per, groups);
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
    if (best.ratio == 0.f) code = kBad;  // no winner (a sound row has one): there is no id to read the row at
  }
  const int32_t token = T == 0.f ? st.argmax : best.id;
  float* lps = p.out.token_logprobs + b * (p.D + 1);
  int32_t* tokens = p.out.tokens + b * (p.D + 1);
  for (int j = tid; j <= p.D; j += kDrawThreads) {
    if (code != kStopped) {
      p.out.refuse(b, p.D, j, SFC_ROW_BADPARAM);
    } else if (j == a) {
      tokens[a] = token;
      lps[a] = log_prob(row.at(token), st, T, token);
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

// Where all CTAs of the statistics run at once, the draw's start while they end (programmatic dependent launch) and
// wait for them before they read the workspace. (With more of them, the waiting CTAs took their places: 10 us slower
// at 64 x 4 x 151936.)
template <int DT>
cudaError_t start(const VerifyParams& p, dim3 stat, dim3 draw, cudaStream_t stream) {
  verify_stats_kernel<DT><<<stat, kStatThreads, 0, stream>>>(p);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = draw;
  cfg.blockDim = dim3(kDrawThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cut.waves ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<DT>, p);
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
  if (target_request_stride < 0 || target_row_stride < 0 || draft_request_stride < 0 || draft_row_stride < 0) return SFC_EINVAL;
  if (row_offset < 0 || row_offset + B > (int64_t{1} << 32)) return SFC_EINVAL;
  if (flags & ~static_cast<uint32_t>(SFC_FLAG_GREEDY_T0)) return SFC_EINVAL;
  const uintptr_t elt = dtype == SFC_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(target_logits) % elt || reinterpret_cast<uintptr_t>(draft_logits) % elt ||
      reinterpret_cast<uintptr_t>(workspace) % 16)
    return SFC_EINVAL;
  if (!workspace || workspace_bytes < sfc_verify_workspace_size(B, D, V, dtype)) return SFC_EWORKSPACE;
  const sfc::VerifyParams p{target_logits, draft_logits, V, target_request_stride, target_row_stride,
                            draft_request_stride, draft_row_stride, D,
                            (flags & SFC_FLAG_GREEDY_T0) != 0, temperature,
                            draft_temperature ? draft_temperature : temperature, draft_tokens, num_drafts, uniforms,
                            sfc::RaceKey(seed, step),
                            static_cast<uint32_t>(row_offset), static_cast<unsigned char*>(workspace), cut,
                            sfc::VerifyOutputs{accepted, tokens, token_logprobs, row_status}};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 stat(static_cast<unsigned>(B), static_cast<unsigned>(cut.stat), static_cast<unsigned>(D + 1));
  const dim3 draw(static_cast<unsigned>(B), static_cast<unsigned>(cut.draw));
  const cudaError_t err = dtype == SFC_BF16 ? sfc::start<0>(p, stat, draw, st) : sfc::start<1>(p, stat, draw, st);
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}
