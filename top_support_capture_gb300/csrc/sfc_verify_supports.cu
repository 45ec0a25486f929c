// Verification of drafted tokens over captured supports: the target's and the draft's filtered distributions as
// packed (id, log-probability) entries, as the decode step captures them. The rule is that of sfc_verify.cu with
// p_j and q_j zero outside the supports; a draft row of length 0 is a certain draft.
//
// One CTA per request. Its warps look the drafted tokens up in both supports, all positions at once; thread 0
// walks the decisions; then the CTA draws over the target's support at the position it stopped at. What the draft
// gives a member is found through a hash table in shared memory (open addressing, 16-bit entry indices, at most
// half full), built from the draft's support of that position.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sfc.h"
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

constexpr int kThreads = 256;
constexpr uint16_t kEmpty = 0xFFFFu;

__device__ __forceinline__ uint32_t slot_of(int32_t id, uint32_t mask) {
  return (static_cast<uint32_t>(id) * 0x9E3779B1u >> 15) & mask;  // Knuth's multiplicative hash
}

// The log-probability of token t in a row of n entries (each lane's share of them, then the warp's): -inf where it
// is not a member.
__device__ __forceinline__ float find(const int32_t* ids, const float* lps, int n, int32_t t) {
  const int lane = threadIdx.x & 31;
  int at = -1;
  for (int k = lane; k < n; k += 32)
    if (ids[k] == t) at = k;
  at = __reduce_max_sync(kFull, at);
  return at < 0 ? -INFINITY : lps[at];
}

__global__ void __launch_bounds__(kThreads) verify_supports_kernel(const __grid_constant__ VerifySupportsParams p) {
  constexpr int NW = kThreads / 32;
  extern __shared__ uint16_t table[];
  __shared__ float lp_target[SFC_MAX_DRAFTS], lp_draft[SFC_MAX_DRAFTS];
  __shared__ float ratios[NW];
  __shared__ int32_t best_ids[NW];
  __shared__ int sh_a, sh_status;
  const int tid = threadIdx.x, wp = tid >> 5, D = p.D;
  const int64_t b = blockIdx.x;
  const int n = p.num_drafts ? p.num_drafts[b] : D;
  const int32_t* drafted = p.draft_tokens + b * D;
  const int32_t* tlen = p.target.lengths + b * (D + 1);
  const int32_t* dlen = p.draft.ids ? p.draft.lengths + b * D : nullptr;
  float* lps = p.out.token_logprobs + b * (D + 1);
  int32_t* tokens = p.out.tokens + b * (D + 1);
  const int looked = min(max(n, 0), D);
  for (int i = wp; i < 2 * looked; i += NW) {  // even: the target's rows, odd: the draft's
    const int j = i >> 1;
    const SupportRows& rows = (i & 1) ? p.draft : p.target;
    const int len = (i & 1) ? (dlen ? dlen[j] : 0) : tlen[j];
    const int64_t at = ((i & 1) ? b * D + j : b * (D + 1) + j) * rows.W;
    float lp = 0.f;  // a certain draft
    if (!(i & 1) || len > 0) lp = find(rows.ids + at, rows.lps + at, min(max(len, 0), rows.W), drafted[j]);
    if ((tid & 31) == 0) ((i & 1) ? lp_draft : lp_target)[j] = lp;
  }
  __syncthreads();
  if (tid == 0) {
    int a = 0, status = n < 0 || n > D ? SFC_ROW_BADPARAM : SFC_ROW_OK;
    while (status == SFC_ROW_OK) {
      if (tlen[a] < 1) status = SFC_ROW_BADPARAM;
      if (tlen[a] > p.target.W) status = SFC_ROW_OVERFLOW;
      if (a == n || status != SFC_ROW_OK) break;
      const float lp = lp_target[a], lq = lp_draft[a];
      if (drafted[a] < 0 || (dlen && dlen[a] < 0))
        status = SFC_ROW_BADPARAM;
      else if (dlen && dlen[a] > p.draft.W)
        status = SFC_ROW_OVERFLOW;
      else if (!(lp < INFINITY) || !(lq < INFINITY))
        status = SFC_ROW_BADPARAM;
      if (status != SFC_ROW_OK) break;
      // in 64 bits: compared with a number next to it
      if (!(p.uniforms[b * D + a] * exp(static_cast<double>(lq)) < exp(static_cast<double>(lp)))) break;
      tokens[a] = drafted[a];
      lps[a] = lp;
      ++a;
    }
    sh_a = a;
    sh_status = status;
  }
  __syncthreads();
  const int a = sh_a;
  if (sh_status != SFC_ROW_OK) {
    for (int j = tid; j <= D; j += kThreads) p.out.refuse(b, D, j, sh_status);
    return;
  }
  const bool refused = a < n;
  const int nt = tlen[a], nd = refused && dlen ? dlen[a] : 0;
  const int32_t* ids = p.target.ids + (b * (D + 1) + a) * p.target.W;
  const float* lp = p.target.lps + (b * (D + 1) + a) * p.target.W;
  const int32_t* qids = nd > 0 ? p.draft.ids + (b * D + a) * p.draft.W : nullptr;
  const float* qlp = nd > 0 ? p.draft.lps + (b * D + a) * p.draft.W : nullptr;
  const uint32_t mask = static_cast<uint32_t>(p.table) - 1;
  int bad = 0;
  if (nd > 0) {
    for (int k = tid; k < p.table; k += kThreads) table[k] = kEmpty;
    __syncthreads();
    for (int k = tid; k < nd; k += kThreads) {
      bad |= !(qlp[k] < INFINITY);
      // at most half full: an empty slot is found; ids that repeat take slots of their own
      for (uint32_t h = slot_of(qids[k], mask);; h = (h + 1) & mask)
        if (atomicCAS(reinterpret_cast<unsigned short*>(table + h), kEmpty, static_cast<unsigned short>(k)) == kEmpty) break;
    }
    __syncthreads();
  }
  const int32_t refused_token = refused ? drafted[a] : -1;
  const uint32_t counter_row = p.row_offset + static_cast<uint32_t>(b);
  RaceBest best;
  for (int pass = 0; pass < 2 && best.ratio == 0.f; ++pass) {  // the second: no residual mass
    RaceBest mine;
    for (int k = tid; k < nt; k += kThreads) {
      const int32_t id = ids[k];
      bad |= id < 0 || !(lp[k] < INFINITY);
      float w = expf(lp[k]);
      if (pass == 0 && refused) {
        float q = 0.f;
        if (nd > 0) {
          for (uint32_t h = slot_of(id, mask); table[h] != kEmpty; h = (h + 1) & mask)
            if (qids[table[h]] == id) {
              q = expf(qlp[table[h]]);
              break;
            }
        } else if (id == refused_token) {
          q = INFINITY;
        }
        w = fmaxf(w - q, 0.f);
      }
      if (!(w > 0.f)) continue;
      const uint4 block = race_block(p.key, counter_row, static_cast<uint32_t>(id) >> 2);
      const uint32_t word = (id & 2) ? ((id & 1) ? block.w : block.z) : ((id & 1) ? block.y : block.x);
      mine.offer(w / race_wait(word), id);
    }
    __syncthreads();
    best = block_best<kThreads>(mine, ratios, best_ids);
  }
  bad = __syncthreads_or(bad);
  if (bad || best.ratio == 0.f) {  // a row without any mass has nothing to draw
    for (int j = tid; j <= D; j += kThreads) p.out.refuse(b, D, j, SFC_ROW_BADPARAM);
    return;
  }
  for (int k = tid; k < nt; k += kThreads)
    if (ids[k] == best.id) lps[a] = lp[k];
  for (int j = a + 1 + tid; j <= D; j += kThreads) {
    tokens[j] = -1;
    lps[j] = 0.f;
  }
  if (tid == 0) {
    tokens[a] = best.id;
    p.out.accepted[b] = a;
    p.out.row_status[b] = SFC_ROW_OK;
  }
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
  const int smem = table * static_cast<int>(sizeof(uint16_t));  // at most 64 KB
  const sfc::VerifySupportsParams p{
      sfc::SupportRows{target_ids, target_logprobs, target_lengths, target_width},
      sfc::SupportRows{draft_ids, draft_logprobs, draft_lengths, draft_width},
      D, table, draft_tokens, num_drafts, uniforms,
      sfc::RaceKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(step),
                   static_cast<uint32_t>(step >> 32)},
      static_cast<uint32_t>(row_offset), sfc::VerifyOutputs{accepted, tokens, token_logprobs, row_status}};
  if (smem > 48 * 1024 && cudaFuncSetAttribute(sfc::verify_supports_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  sfc::verify_supports_kernel<<<static_cast<unsigned>(B), sfc::kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SFC_OK : SFC_ECUDA;
}
