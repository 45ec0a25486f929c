// Shared by the two verifications of drafted tokens: the race that draws the token after the last accepted
// draft, and the outputs.
//
// The race draws i with probability proportional to w_i as argmax w_i / E_i, E_i = -ln u_i. Its noise comes
// from Philox4x32-10 blocks at the counter (2^31 + i / 4, row, step lo, step hi), word i % 4: one block serves
// four neighbouring tokens, and since token ids are below 2^31 the counters never meet those of the decode
// step's race (token id, row, step), so a draft and its verification may share a seed and a step.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_device.cuh"

namespace sfc {

// The ten round keys and the step. They are made on the host and passed as kernel parameters, which the
// instructions take as constant operands: the schedule costs the kernels nothing.
struct RaceKey {
  uint32_t round[10][2];
  uint32_t step_lo, step_hi;

  RaceKey(uint64_t seed, uint64_t step) : step_lo(static_cast<uint32_t>(step)), step_hi(static_cast<uint32_t>(step >> 32)) {
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    for (auto& k : round) {
      k[0] = k0;
      k[1] = k1;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
  }
};

__device__ __forceinline__ uint4 race_block(const RaceKey& key, uint32_t row, uint32_t quad) {
  uint32_t c0 = 0x80000000u | quad, c1 = row, c2 = key.step_lo, c3 = key.step_hi;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ key.round[r][0];
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ key.round[r][1];
    c3 = static_cast<uint32_t>(p0);
  }
  return make_uint4(c0, c1, c2, c3);
}

// u = (2 (w >> 9) + 1) 2^-24, exact in float32 and never 0 or 1: the 23 bits as the fraction of a number in [1, 2),
// less 1 - 2^-24.
__device__ __forceinline__ float race_unit(uint32_t w) { return __uint_as_float(0x3F800000u | (w >> 9)) - 0x1.fffffep-1f; }

// E = -ln u of one word.
__device__ __forceinline__ float race_wait(uint32_t w) { return -logf(race_unit(w)); }

// The winner so far: the largest w / E, ties to the lowest id. No winner: ratio 0.
struct RaceBest {
  float ratio = 0.f;
  int32_t id = INT32_MAX;

  __device__ __forceinline__ void offer(float r, int32_t i) {
    if (r > ratio || (r == ratio && r > 0.f && i < id)) {
      ratio = r;
      id = i;
    }
  }
};

template <int NT>
__device__ __forceinline__ RaceBest block_best(RaceBest b, float* ratios, int32_t* ids) {
  constexpr int NW = NT / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float r = __shfl_xor_sync(kFull, b.ratio, o);
    const int32_t i = __shfl_xor_sync(kFull, b.id, o);
    b.offer(r, i);
  }
  if ((threadIdx.x & 31) == 0) {
    ratios[threadIdx.x >> 5] = b.ratio;
    ids[threadIdx.x >> 5] = b.id;
  }
  __syncthreads();
  RaceBest all;
  for (int w = 0; w < NW; ++w) all.offer(ratios[w], ids[w]);
  return all;
}

struct VerifyOutputs {
  int32_t* accepted;       // [B]
  int32_t* tokens;         // [B, D + 1]
  float* token_logprobs;   // [B, D + 1]
  int32_t* row_status;     // [B]

  // Position j of a request that failed its checks.
  __device__ __forceinline__ void refuse(int64_t b, int D, int j, int status) const {
    tokens[b * (D + 1) + j] = -1;
    token_logprobs[b * (D + 1) + j] = __int_as_float(0x7fc00000);
    if (j == 0) {
      accepted[b] = 0;
      row_status[b] = status;
    }
  }
};

}  // namespace sfc
