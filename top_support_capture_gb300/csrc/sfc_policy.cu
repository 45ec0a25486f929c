// The clipped policy loss of each row's sampled token and its gradient, in one read of the logits. With lp, H the token's
// log-probability and the row's entropy over the whole vocabulary at T, rho = exp(lp - old):
//
//   loss = -min(rho A, clamp(rho, 1 - low, 1 + high) A) - w H,   or without old: loss = -A lp - w H
//   dloss/dlp = -rho A where the unclipped side is the smaller one (0 elsewhere), or -A
//   dloss/dx_j = (dloss/dlp (delta_jt - p_j) + w p_j (ln p_j + H)) / T          (sfc_entropy.cuh)
//
// A row is cut into slices, one CTA each, which form a cluster. A slice stays in shared memory between its two uses: one
// thread starts a bulk copy of it before anything else, and the wait for it is bounded (SFC_ROW_TIMEOUT). The CTAs exchange
// their statistics through distributed shared memory; each then works out the row's scalars for itself. The dense part of
// the gradient is written first, the token's entry over it after the CTA's barrier. Rows longer than a cluster's shared
// memory are read again.
//
// 2048 x 151936 bf16: 180 us, 1.02 of the measured copy rate (2 x 622 MB). The CTAs of a SM read, compute and write in turns, so
// what they issue and wait for counts as much as the bytes. The steps: sums that were rescaled as each vector raised the
// maximum, exponents in two steps and products held above -200 one by one 264 us; a later slice on its way to L2 meanwhile 260;
// the extremes of a thread's vectors first, so that the sums have no such step, 252; one fused step per exponent and no holding
// where the extremes allow it 230; the slices' statistics sent by stores that the receiver's barrier counts 180: a
// cluster barrier's release had every warp wait for all that it had in flight (a quarter of the warps' time).
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_entropy.cuh"
#include "sfc_host.cuh"

namespace sfc {
namespace {

struct PolicyParams {
  const void* logits;
  int64_t row_stride, V;
  const float* temperature;
  const int32_t* tokens;
  const float* old_logprobs;  // or null
  const float* advantages;
  float clip_low, clip_high, entropy_weight;
  const float* grad_loss;
  float* loss;
  float* logprobs;
  float* entropy;
  int32_t* row_status;
  unsigned char* grad;
  int64_t grad_stride;
  int32_t slices, per;  // CTAs a row, vectors a slice
  bool stall;           // test of the failure path: the copies are never started
};

constexpr int kMaxSlices = 8;       // the portable cluster size
constexpr int kKeepBytes = 212992;  // shared memory of one SM that keeps logits: 13 vectors for each of 1024 threads
constexpr uint32_t kStallPolls = 16;
constexpr float kLate = -1.f;  // in place of a mass: a copy did not arrive

// The bound of a wait for the other slices' statistics: above that of a slice for its own copy, which says so when it gives up. A
// CTA that hears nothing for so long (not expected to happen) looks at the whole row itself, so that a row's CTAs all come to the
// same outcome.
constexpr uint32_t kJoinPolls = 4 * kWaitPolls;

template <int DT>
__device__ __noinline__ float4 row_stats(const unsigned char* row, int64_t V, float c) {  // by a whole warp, in two passes
  const int lane = threadIdx.x & 31;
  float m = -FLT_MAX;
  for (int64_t i = lane; i < V; i += 32) m = fmaxf(m, Elem<DT>::load1(row, i));
  m = warp_max(m);
  double s = 0.0, w = 0.0;
  for (int64_t i = lane; i < V; i += 32) {
    const float d = (Elem<DT>::load1(row, i) - m) * c, e = ex2_approx(d);
    s += e;
    w += e * fmaxf(d, kFar);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o), w += __shfl_xor_sync(kFull, w, o);
  return make_float4(m, static_cast<float>(s), static_cast<float>(w), 0.f);
}

// KEEP: the slice's vectors lie in dynamic shared memory (16 bytes for each).
template <int DT, int NT, int MINB, bool KEEP>
__global__ void __launch_bounds__(NT, MINB) policy_kernel(const __grid_constant__ PolicyParams p) {
  constexpr int NW = NT / 32, VEC = Elem<DT>::kVec;
  constexpr int U = 4;  // vectors in flight per thread where they are not kept (and as many again)
  constexpr int kAhead = 76 * MINB;  // CTAs that a prefetch runs ahead: half of what runs at once
  extern __shared__ __align__(128) uint4 kept[];
  __shared__ uint64_t full, joined;  // the copy's arrival, that of the slices' statistics
  __shared__ float4 red[NW];
  __shared__ float4 table[kMaxSlices];  // (m, s, w) of the slices
  __shared__ float4 gradient;           // (m, c, a, b) of the row's
  __shared__ float slope_at_token;
  __shared__ bool lifted;
  __shared__ int outcome;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, S = p.slices, rank = blockIdx.y;
  const int64_t r = blockIdx.x;
  const RowSpan<DT> row(p.logits, r * p.row_stride, p.V);
  const uint4* body = row.body();
  const int nvec = static_cast<int>(row.nvec), v0 = min(rank * p.per, nvec), v1 = min(v0 + p.per, nvec), mine = v1 - v0;
  const bool scalar = rank == 0 && tid < row.scalars();
  if (tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&joined, 1);
    mbar_init_fence();
    if (KEEP && !p.stall) {  // on its way while the row's parameters load
      mbar_arrive_expect_tx(&full, mine * 16);
      if (mine > 0) bulk_load(kept, body + v0, mine * 16, &full);
    }
    mbar_arrive_expect_tx(&joined, S * sizeof(float4));
  }
  __syncthreads();                       // the barriers exist
  if (S > 1) cluster_arrive_started();  // waited for before the first store into another CTA
  const float T = p.temperature[r], A = p.advantages[r], old = p.old_logprobs ? p.old_logprobs[r] : 0.f, up = p.grad_loss[r];
  const int32_t token = p.tokens[r];
  const float c = exponent_scale(T);
  const float xt = token >= 0 && token < p.V ? row.at(token) : 0.f;
  const bool sound = temperature_valid(T) && token >= -1 && token < p.V && fabsf(A) < INFINITY && fabsf(old) < INFINITY;
  int status = sound ? SFC_ROW_OK : SFC_ROW_BADPARAM;
  bool live = sound && token >= 0, late = false;  // uniform over the row's CTAs
  bool near = false;  // this thread's kept logits lie within kNear
  if (live) {
    EntropyAcc a;
    if (KEEP) {
      late = !__all_sync(kFull, mbar_wait(&full, 0, p.stall ? kStallPolls : kWaitPolls));
      if (tid == 0 && r + kAhead / S < gridDim.x) {  // a later CTA's slice on its way to L2 while HBM would idle
        const RowSpan<DT> later(p.logits, (r + kAhead / S) * p.row_stride, p.V);
        const int vecs = static_cast<int>(later.nvec), at = min(rank * p.per, vecs), bytes = (min(at + p.per, vecs) - at) * 16;
        if (bytes > 0) prefetch_l2(later.body() + at, bytes);
      }
      if (!late) near = add_kept<DT, NT>(a, kept, mine, c);
    } else {
      RowStream<DT, NT, U> stream(row, v0, v1);
      stream.batches([&](const uint4(&v)[U]) { a.template add<DT, U>(v, c); });
    }
    if (scalar) a.add(row.at(row.scalar_index(tid)), c);
    const EntropyStats w = merge_lanes(a, c);
    if (lane == 0) red[wp] = make_float4(w.m, w.s, w.w, 0.f);
    if (KEEP) late = __syncthreads_or(late);
    else __syncthreads();
  }
  if (S > 1) cluster_wait();
  // the row's scalars, by one warp of each of its CTAs
  if (wp == 0) {
    const float nan = __int_as_float(0x7fc00000), inv_T = fminf(1.f / T, FLT_MAX);
    EntropyStats all{-FLT_MAX, kLate, 0.f};
    if (live) {
      if (!(KEEP && late)) all = merge_shared(red, NW, c);
      if (S > 1) {
        if (tid < S) dsmem_send(dsmem_addr(&table[rank], tid), make_float4(all.m, all.s, all.w, 0.f), dsmem_addr(&joined, tid));
        __syncwarp();
        if (__all_sync(kFull, mbar_wait(&joined, 0, kJoinPolls))) {
          late = __any_sync(kFull, table[lane < S ? lane : 0].y == kLate);
          all = merge_shared(table, S, c);
        } else if (!late) {
          const float4 v = row_stats<DT>(row.row, p.V, c);
          all = EntropyStats{v.x, v.y, v.z};
        }
      }
      live = stats_valid(all.m, all.s) && !late;
      if (!live) status = late ? SFC_ROW_TIMEOUT : SFC_ROW_BADPARAM;
    }
    float H = 0.f, lp = 0.f, ln_s = 0.f, loss = status < 0 ? nan : 0.f, slope = 0.f;  // slope: dloss/dlp
    if (live) {
      ln_s = all.log_sum();
      H = all.entropy(ln_s);
      const float z = below_max(xt, all.m, [&](float d) { return d * inv_T; });
      lp = z - ln_s;
      if (p.old_logprobs) {
        // lp - old with the quotient's remainder, and the near numbers subtracted first: rho is as exact as its exponent
        const float rest = z > -INFINITY ? fmaf(-z, T, xt - all.m) * inv_T : 0.f;
        const float rho = expf((z - old) - ln_s + rest), plain = rho * A;
        const float low = 1.f - p.clip_low, high = 1.f + p.clip_high;
        const bool active = A >= 0.f ? rho <= high : rho >= low;
        loss = active ? -plain : -(A >= 0.f ? high : low) * A;
        slope = active ? held(-plain) : 0.f;
      } else {
        loss = A == 0.f ? 0.f : -A * lp;
        slope = xt > -INFINITY ? -A : 0.f;  // a masked token's log-probability is the constant -inf
      }
      if (p.entropy_weight != 0.f) loss -= p.entropy_weight * H;
    }
    if (lane == 0) {
      const float scale = fabsf(up) < INFINITY ? held(up * inv_T) : up, g = held(slope * scale);
      if (live) {
        const RowGradient dense(all.m, all.s, ln_s, H, g, -p.entropy_weight * scale, c);
        gradient = make_float4(dense.m, dense.c, dense.a, dense.b);
        lifted = dense.lifted;
        slope_at_token = g;
      }
      outcome = live;
      if (rank == 0) {
        p.loss[r] = loss;
        p.logprobs[r] = status < 0 ? nan : lp;
        p.entropy[r] = status < 0 ? nan : H;
        p.row_status[r] = status;
      }
    }
  }
  __syncthreads();
  live = outcome;
  // nothing of the CTA's is still in flight when it ends
  if (KEEP && !live && tid == 0 && !p.stall) mbar_wait(&full, 0);
  const RowGradient dense(gradient, lifted);
  unsigned char* grad = p.grad + r * p.grad_stride * Elem<DT>::kBytes;
  unsigned char* out = grad + static_cast<int64_t>(row.head) * Elem<DT>::kBytes;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 15);
  auto put = [&](int at, const uint4& w) { store_vector<DT>(out + static_cast<int64_t>(at) * 16, w, shift, at < v1); };
  if (!live) {
    for (int i = v0 + tid; i - lane < v1; i += NT) put(i, make_uint4(0u, 0u, 0u, 0u));
  } else if (dense.lifted) {
    write_lifted<DT, NT>(dense, row, out, shift, v0, v1);
  } else if (KEEP && DT == 0 && shift != 0) {
    for (int i = tid; i - lane < mine; i += NT) put(v0 + i, dense.template vector<DT>(kept[min(i, mine - 1)]));
  } else if (KEEP && near && dense.moderate()) {
    const RowGradient::Near n(dense);
#pragma unroll 4
    for (int i = tid; i < mine; i += NT) put(v0 + i, n.template vector<DT>(kept[i]));
  } else if (KEEP) {
#pragma unroll 2
    for (int i = tid; i < mine; i += NT) put(v0 + i, dense.template vector<DT>(kept[i]));
  } else {
    RowStream<DT, NT, U> stream(row, v0, v1);
    stream.each([&](const uint4& w, int at) { put(at, dense.template vector<DT>(w)); });
  }
  if (scalar) {
    const int64_t i = row.scalar_index(tid);
    Out<DT>::store1(grad, i, live ? dense.at(row.at(i)) : 0.f);
  }
  if (live) {
    __syncthreads();  // the dense values are written before the token's overwrites its own
    const int64_t lo = row.head + static_cast<int64_t>(v0) * VEC, hi = row.head + static_cast<int64_t>(v1) * VEC;
    if (tid == 0 && ((token >= lo && token < hi) || (rank == 0 && (token < row.head || token >= row.tail()))))
      Out<DT>::store1(grad, token, dense.at(xt) + slope_at_token);
  }
}

template <int DT, int NT, int MINB, bool KEEP>
cudaError_t start(PolicyParams p, int64_t B, cudaStream_t stream) {
  auto kern = policy_kernel<DT, NT, MINB, KEEP>;
  const int64_t vectors = p.V / Elem<DT>::kVec;
  p.per = static_cast<int32_t>((vectors + p.slices - 1) / p.slices + 7) & ~7;  // whole 128-byte lines
  cudaLaunchConfig_t cfg = {};
  if (KEEP) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t err = allow_shared(kern, kKeepBytes / MINB, done);
    if (err != cudaSuccess) return err;
    cfg.dynamicSmemBytes = static_cast<size_t>(p.per) * 16;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(B), static_cast<unsigned>(p.slices));
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {1, static_cast<unsigned>(p.slices), 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT>
cudaError_t choose(PolicyParams& p, int64_t B, cudaStream_t stream) {
  const int64_t vectors = p.V / Elem<DT>::kVec;
  auto cut = [&](int64_t per) { return std::max<int64_t>(1, (vectors + per - 1) / per); };
  auto fits = [&](int64_t S) {
    p.slices = static_cast<int32_t>(std::min<int64_t>(S, kMaxSlices));
    return S <= kMaxSlices;
  };
  // Slices within their CTA's shared memory (in whole 128-byte lines): the smaller the CTAs the better, as long as a row fits a
  // cluster, since more of them take turns on a SM (2048 x 151936 bf16: six slices of 256 threads 180 us, three of 512 199;
  // 2048 x 50000: four of 128 63, two of 256 64, one of 512 70). Few rows: as many slices (two, four or eight) as there are places.
  int64_t fill = 1;
  while (fill < kMaxSlices && vectors >= 4096 * fill && 2 * fill * B <= 304) fill *= 2;
  if (fits(std::max(fill, cut(kKeepBytes / 8 / 16 - 8)))) return start<DT, 128, 8, true>(p, B, stream);
  if (fits(std::max(fill, cut(kKeepBytes / 4 / 16 - 8)))) return start<DT, 256, 4, true>(p, B, stream);
  if (fits(cut(kKeepBytes / 2 / 16 - 8))) return start<DT, 512, 2, true>(p, B, stream);
  if (fits(cut(kKeepBytes / 16 - 8))) return start<DT, 1024, 1, true>(p, B, stream);
  return start<DT, 512, 2, false>(p, B, stream);
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_policy_forward_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                           const float* temperature, const int32_t* tokens, const float* old_logprobs,
                                           const float* advantages, float clip_low, float clip_high, float entropy_weight,
                                           uint32_t flags, const float* grad_loss, float* loss, float* logprobs, float* entropy,
                                           int32_t* row_status, void* grad_logits, int64_t grad_stride, void* stream) {
  if (!logits || !temperature || !tokens || !advantages || !grad_loss || !loss || !logprobs || !entropy || !row_status || !grad_logits)
    return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || row_stride < V || grad_stride < V) return SFC_EINVAL;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f && clip_high < INFINITY) || !(fabsf(entropy_weight) < INFINITY))
    return SFC_EINVAL;
  if (flags & ~SFC_FLAG_TEST_STALL) return SFC_EINVAL;
  const int64_t elt = dtype == SFC_BF16 ? 2 : 4;
  const uintptr_t g = reinterpret_cast<uintptr_t>(grad_logits), l = reinterpret_cast<uintptr_t>(logits);
  if (g % elt || l % elt) return SFC_EINVAL;
  if (g < l + ((B - 1) * row_stride + V) * elt && l < g + ((B - 1) * grad_stride + V) * elt) return SFC_EINVAL;
  sfc::PolicyParams p{logits, row_stride, V, temperature, tokens, old_logprobs, advantages, clip_low, clip_high, entropy_weight,
                      grad_loss, loss, logprobs, entropy, row_status, static_cast<unsigned char*>(grad_logits), grad_stride, 1, 0,
                      (flags & SFC_FLAG_TEST_STALL) != 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((dtype == SFC_BF16 ? sfc::choose<0>(p, B, st) : sfc::choose<1>(p, B, st)) != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}
