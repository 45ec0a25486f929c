// Verification of drafted tokens over captured supports: the target's and the draft's filtered distributions as
// packed (id, log-probability) entries, as the decode step captures them. The rule is that of sfc_verify.cu with
// p_j and q_j zero outside the supports; a draft row of length 0 is a certain draft.
//
// One CTA per request, every step as wide as the CTA: its warps look the drafted tokens up in both supports, all
// positions at once, in 16-byte loads; each warp then has every decision (a lane a position); and the CTA draws over
// the target's support at the position it stopped at. The draft's entries of that position move to shared memory, and
// what they give a member is found through a hash table there (open addressing, 16-bit entry indices, at most half
// full). Latency bounds it, about ten dependent steps: 9.3 us for one request of 4 drafts at W = 1024, 30 us for 128 at
// W = 8192, where the request with the longest supports sets the end (its CTA works twice as long as the mean).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_host.cuh"
#include "sfc_verify.cuh"

namespace sfc {
namespace {

struct SupportRows {
  const int32_t* ids;
  const float* lps;
  const int32_t* lengths;
  int32_t W;
};

struct VerifySupportsParams {
  SupportRows target, draft;  // draft.ids null: every draft is certain
  int32_t D, table;           // slots of the hash table, a power of two
  const int32_t* draft_tokens;
  const int32_t* num_drafts;
  const float* uniforms;
  RaceKey key;
  uint32_t row_offset;
  VerifyOutputs out;
};

constexpr uint16_t kEmpty = 0xFFFFu;

__device__ __forceinline__ uint32_t slot_of(int32_t id, uint32_t mask) {
  return (static_cast<uint32_t>(id) * 0x9E3779B1u >> 15) & mask;  // Knuth's multiplicative hash
}

// The warp's search of ids[k0, k1) for t (k0 a multiple of 4): the lane that finds it leaves its log-probability.
__device__ __forceinline__ void find(const int32_t* ids, const float* lps, int k0, int k1, int32_t t, float* found) {
  const int lane = threadIdx.x & 31;
  int at = -1;
  if ((reinterpret_cast<uintptr_t>(ids) & 15) == 0) {
    const int4* four = reinterpret_cast<const int4*>(ids);
#pragma unroll 2
    for (int k = k0 + 4 * lane; k < k1; k += 128) {
      int4 v = make_int4(-1, -1, -1, -1);
      if (k + 4 <= k1) v = __ldg(four + k / 4);
      else {
        v.x = ids[k];
        if (k + 1 < k1) v.y = ids[k + 1];
        if (k + 2 < k1) v.z = ids[k + 2];
      }
      if (v.x == t) at = k;
      if (v.y == t) at = k + 1;
      if (v.z == t) at = k + 2;
      if (v.w == t) at = k + 3;
    }
  } else {
#pragma unroll 8
    for (int k = k0 + lane; k < k1; k += 32)
      if (ids[k] == t) at = k;
  }
  if (t >= 0 && at >= 0) *found = lps[at];
}

// The winner with its place in the row.
struct Drawn {
  RaceBest best;
  int at = 0;

  __device__ __forceinline__ void offer(float ratio, int32_t id, int k) {
    const float r = best.ratio;
    const int32_t i = best.id;
    best.offer(ratio, id);
    if (best.ratio != r || best.id != i) at = k;
  }
};

template <int NT>
__global__ void __launch_bounds__(NT) verify_supports_kernel(const __grid_constant__ VerifySupportsParams p) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) unsigned char shared[];  // [slots] entry indices, [draft.W] ids and probabilities
  uint16_t* table = reinterpret_cast<uint16_t*>(shared);
  int32_t* qids = reinterpret_cast<int32_t*>(shared + p.table * sizeof(uint16_t));
  float* qs = reinterpret_cast<float*>(qids + p.draft.W);
  __shared__ float lp_of[2][SFC_MAX_DRAFTS];  // of the drafted tokens: the target's, the draft's
  __shared__ float ratios[NW];
  __shared__ int32_t best_ids[NW], best_at[NW];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, D = p.D;
  const int64_t b = blockIdx.x;
  const int n = p.num_drafts ? p.num_drafts[b] : D;
  const int32_t* drafted = p.draft_tokens + b * D;
  const int32_t* tlen = p.target.lengths + b * (D + 1);
  const int32_t* dlen = p.draft.ids ? p.draft.lengths + b * D : nullptr;
  float* lps = p.out.token_logprobs + b * (D + 1);
  int32_t* tokens = p.out.tokens + b * (D + 1);
  const uint32_t mask = static_cast<uint32_t>(p.table) - 1;
  for (int k = tid; k < 2 * SFC_MAX_DRAFTS; k += NT) (&lp_of[0][0])[k] = -INFINITY;
  if (p.draft.ids)
    for (int k = tid; k < p.table / 2; k += NT) reinterpret_cast<uint32_t*>(table)[k] = 0xFFFFFFFFu;
  __syncthreads();
  // the look-ups: each row cut over `parts` warps
  const int looked = min(max(n, 0), D), rows = looked * (dlen ? 2 : 1);
  const int parts = max(1, NW / max(rows, 1));
  for (int i = wp; i < rows * parts; i += NW) {
    const int part = i / max(rows, 1), row = i - part * rows, side = row >= looked, j = row - side * looked;
    const SupportRows& of = side ? p.draft : p.target;
    const int len = min(max(side ? dlen[j] : tlen[j], 0), of.W);
    const int per = ((len + parts - 1) / parts + 127) & ~127, k0 = min(part * per, len), k1 = min(k0 + per, len);
    const int64_t at = (b * (side ? D : D + 1) + j) * of.W;
    find(of.ids + at, of.lps + at, k0, k1, drafted[j], &lp_of[side][j]);
  }
  __syncthreads();
  // the decisions, every warp for itself: code 0 goes on, kStop draws here, else the status plus kStatus
  constexpr int kStop = 1, kStatus = 16;
  int a = 0, code = kStatus + SFC_ROW_BADPARAM;
  if (n >= 0 && n <= D) {
    for (int j0 = 0; j0 <= n; j0 += 32) {
      const int j = j0 + lane;
      int mine = kStop;
      if (j <= n) {
        const int nt = tlen[j];
        if (nt < 1 || nt > p.target.W) {
          mine = kStatus + (nt < 1 ? SFC_ROW_BADPARAM : SFC_ROW_OVERFLOW);
        } else if (j < n) {
          const int nd = dlen ? dlen[j] : 0;
          const float lp = lp_of[0][j], lq = nd > 0 ? lp_of[1][j] : 0.f;  // no row: a certain draft
          if (drafted[j] < 0 || nd < 0) {
            mine = kStatus + SFC_ROW_BADPARAM;
          } else if (nd > p.draft.W) {
            mine = kStatus + SFC_ROW_OVERFLOW;
          } else if (!(lp < INFINITY) || !(lq < INFINITY)) {
            mine = kStatus + SFC_ROW_BADPARAM;
          } else {
            const float u = p.uniforms[b * D + j], left = u * expf(lq), right = expf(lp);
            bool accept = left < right;
            if (!(fabsf(left - right) > 0x1p-14f * fmaxf(left, right) && right > 0x1p-100f))  // too near: in 64 bits
              accept = u * exp(static_cast<double>(lq)) < exp(static_cast<double>(lp));
            if (accept) mine = 0;
          }
        }
      }
      const unsigned open = __ballot_sync(kFull, mine != 0);
      if (open) {
        const int k = __ffs(static_cast<int>(open)) - 1;
        a = j0 + k;
        code = __shfl_sync(kFull, mine, k);
        break;
      }
    }
  }
  if (code != kStop) {
    for (int j = tid; j <= D; j += NT) p.out.refuse(b, D, j, code - kStatus);
    return;
  }
  const bool refused = a < n;
  const int nt = tlen[a], nd = refused && dlen ? dlen[a] : 0;
  const int32_t* ids = p.target.ids + (b * (D + 1) + a) * p.target.W;
  const float* lp = p.target.lps + (b * (D + 1) + a) * p.target.W;
  int bad = 0;
  if (nd > 0) {
    const int32_t* from = p.draft.ids + (b * D + a) * p.draft.W;
    const float* from_lp = p.draft.lps + (b * D + a) * p.draft.W;
#pragma unroll 2
    for (int k = tid; k < nd; k += NT) {
      const int32_t id = from[k];
      const float l = from_lp[k];
      bad |= !(l < INFINITY);
      qids[k] = id;
      qs[k] = expf(l);
      // at most half full: an empty slot is found; ids that repeat take slots of their own
      for (uint32_t h = slot_of(id, mask);; h = (h + 1) & mask)
        if (atomicCAS(reinterpret_cast<unsigned short*>(table + h), kEmpty, static_cast<unsigned short>(k)) == kEmpty) break;
    }
    __syncthreads();
  }
  const int32_t refused_token = refused ? drafted[a] : -1;
  const uint32_t counter_row = p.row_offset + static_cast<uint32_t>(b);
  Drawn all;
  for (int pass = 0; pass < 2 && all.best.ratio == 0.f; ++pass) {  // the second: no residual mass
    Drawn mine;
    constexpr int E = 4;  // entries on their way at once
    for (int k0 = tid; k0 < nt; k0 += E * NT) {
      int32_t id[E];
      float l[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int k = k0 + e * NT;
        id[e] = k < nt ? ids[k] : 0;
        l[e] = k < nt ? lp[k] : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        bad |= id[e] < 0 || !(l[e] < INFINITY);
        float w = expf(l[e]);
        if (pass == 0 && refused && w > 0.f) {
          float q = 0.f;
          if (nd > 0) {
            for (uint32_t h = slot_of(id[e], mask); table[h] != kEmpty; h = (h + 1) & mask)
              if (qids[table[h]] == id[e]) {
                q = qs[table[h]];
                break;
              }
          } else if (id[e] == refused_token) {
            q = INFINITY;
          }
          w = fmaxf(w - q, 0.f);
        }
        if (!(w > 0.f)) continue;
        const uint4 block = race_block(p.key, counter_row, static_cast<uint32_t>(id[e]) >> 2);
        const uint32_t word = (id[e] & 2) ? ((id[e] & 1) ? block.w : block.z) : ((id[e] & 1) ? block.y : block.x);
        mine.offer(w / race_wait(word), id[e], k0 + e * NT);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float r = __shfl_xor_sync(kFull, mine.best.ratio, o);
      const int32_t i = __shfl_xor_sync(kFull, mine.best.id, o);
      const int k = __shfl_xor_sync(kFull, mine.at, o);
      mine.offer(r, i, k);
    }
    __syncthreads();
    if (lane == 0) {
      ratios[wp] = mine.best.ratio;
      best_ids[wp] = mine.best.id;
      best_at[wp] = mine.at;
    }
    __syncthreads();
    for (int w = 0; w < NW; ++w) all.offer(ratios[w], best_ids[w], best_at[w]);
  }
  bad = __syncthreads_or(bad);
  if (bad || all.best.ratio == 0.f) {  // a row without any mass has nothing to draw
    for (int j = tid; j <= D; j += NT) p.out.refuse(b, D, j, SFC_ROW_BADPARAM);
    return;
  }
  for (int j = tid; j <= D; j += NT) {
    tokens[j] = j < a ? drafted[j] : (j == a ? all.best.id : -1);
    lps[j] = j < a ? lp_of[0][j] : (j == a ? lp[all.at] : 0.f);
  }
  if (tid == 0) {
    p.out.accepted[b] = a;
    p.out.row_status[b] = SFC_ROW_OK;
  }
}

template <int NT>
cudaError_t start(const VerifySupportsParams& p, int64_t B, cudaStream_t stream) {
  constexpr int kMost = 2 * SFC_MAX_PACKED_WIDTH * 2 + SFC_MAX_PACKED_WIDTH * 8;  // 192 KB
  const int smem = p.draft.ids ? p.table * 2 + p.draft.W * 8 : 0;
  if (smem > 40 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t err = allow_shared(verify_supports_kernel<NT>, kMost, done);
    if (err != cudaSuccess) return err;
  }
  verify_supports_kernel<NT><<<static_cast<unsigned>(B), NT, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_verify_supports(const int32_t* target_ids, const float* target_logprobs,
                                   const int32_t* target_lengths, int32_t target_width, const int32_t* draft_ids,
                                   const float* draft_logprobs, const int32_t* draft_lengths, int32_t draft_width,
                                   int64_t B, int32_t D, const int32_t* draft_tokens, const int32_t* num_drafts,
                                   const float* uniforms, uint64_t seed, uint64_t step, int64_t row_offset,
                                   int32_t* accepted, int32_t* tokens, float* token_logprobs, int32_t* row_status,
                                   void* stream) {
  if (!target_ids || !target_logprobs || !target_lengths || !draft_tokens || !uniforms || !accepted || !tokens ||
      !token_logprobs || !row_status)
    return SFC_EINVAL;
  if (draft_ids && (!draft_logprobs || !draft_lengths || draft_width < 1 || draft_width > SFC_MAX_PACKED_WIDTH))
    return SFC_EINVAL;
  if (target_width < 1 || target_width > SFC_MAX_PACKED_WIDTH) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || D < 1 || D > SFC_MAX_DRAFTS) return SFC_EINVAL;
  if (row_offset < 0 || row_offset + B > (int64_t{1} << 32)) return SFC_EINVAL;
  int32_t table = 64;  // a power of two of at least twice the entries
  while (draft_ids && table < 2 * draft_width) table *= 2;
  const sfc::VerifySupportsParams p{
      sfc::SupportRows{target_ids, target_logprobs, target_lengths, target_width},
      sfc::SupportRows{draft_ids, draft_logprobs, draft_lengths, draft_ids ? draft_width : 0},
      D, table, draft_tokens, num_drafts, uniforms,
      sfc::RaceKey(seed, step),
      static_cast<uint32_t>(row_offset), sfc::VerifyOutputs{accepted, tokens, token_logprobs, row_status}};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // wide supports have more entries than a small CTA has threads: 128 x 4 at W = 8192 29.6 us with 1024 threads, 37.5
  // with 512, 60 with 256; 1 x 4 at W = 1024 9.3 us with 256, 9.5 with 512, 12.0 with 128
  const bool wide = std::max(target_width, draft_ids ? draft_width : 0) > 2048;
  if ((wide ? sfc::start<1024>(p, B, st) : sfc::start<256>(p, B, st)) != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}
