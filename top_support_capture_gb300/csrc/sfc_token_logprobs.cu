// Log-probabilities of given tokens over the whole vocabulary, with the row's entropy and its top alternatives, and their
// gradient (sfc_entropy.cuh has the formulas).
//
// The forward call reads the logits once. A row is cut into slices of 16-byte vectors, one CTA each, which form a cluster
// and exchange their statistics through distributed shared memory, merged in slice order.
//
// Top alternatives without a second pass: each thread already knows the maximum of what it has seen, and keeps those of its
// cells (32 elements or more) in shared memory. The K-th largest of the maxima of K or more disjoint groups of threads is a
// lower bound on the K-th largest logit, since each group has an element at least that large, and a tight one: with 128
// groups of randomly spread logits about K + K^2 / 256 elements reach it. Only the cells whose maximum reaches the bound
// have such elements: their vectors are read again (from L2, all at once over their warp's lanes), and what reaches the
// bound goes into a pool in shared memory, from which the K largest are ranked by counting. Of S slices each gives two
// bounds, the largest of the slices' K-th and the smallest of their ceil(K / S)-th; the larger one holds for the row. Where
// ties or a regular pattern overfill the pool or a warp's list of cells, the row's first CTA finds the K largest one by one
// instead (every thread holds its best, the winner's warp looks for its next): exact for any row.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_entropy.cuh"
#include "sfc_host.cuh"

namespace sfc {
namespace {

constexpr int kMaxSlices = 8;  // the portable cluster size
constexpr float kLate = -1.f;  // in place of a mass: a bounded wait gave up
constexpr int kGroups = 128;   // of threads; not fewer than SFC_MAX_TOP, not more than the smallest CTA
constexpr uint32_t kPool = 1024;
constexpr int kListed = 64;  // cells of a warp
constexpr int kCells = 24, kCellBytes = 32768;  // most of a thread (a mask's bits), of a CTA
static_assert(SFC_MAX_TOP <= kGroups && SFC_MAX_GIVEN <= kGroups, "");

struct ScoreParams {
  const void* logits;
  int64_t row_stride, V;
  const float* temperature;
  const int32_t* tokens;
  int32_t M, K;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  float4* stats;  // (m, s, H, 0) for the gradient, or null
  int32_t* row_status;
  int32_t slices, per;  // CTAs a row, vectors a slice
  int32_t shift;        // a cell holds 2^shift batches of a thread
};

__device__ __forceinline__ uint32_t dsmem_add(uint32_t addr, uint32_t n) {  // the counter's old value
  uint32_t v;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(addr), "r"(n) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t ld_volatile(const uint32_t* shared) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_addr(shared)) : "memory");
  return v;
}

template <int DT>
__device__ __forceinline__ uint64_t ckey_of(float x, int64_t id) {  // 0: not an alternative (-inf)
  return x > -INFINITY ? make_ckey(Keys<DT>::key(x), static_cast<uint32_t>(id)) : 0ull;
}

__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(kFull, k, o));
  return k;
}

// The sum of n over the lanes before this one, and over all.
__device__ __forceinline__ int warp_before(int n, int& total) {
  int upto = n;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int before = __shfl_up_sync(kFull, upto, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) upto += before;
  }
  total = __shfl_sync(kFull, upto, 31);
  return upto - n;
}

// The largest key below `limit` among the vectors first, first + step, ... below v1 (this lane's share of the work).
template <int DT>
__device__ __forceinline__ uint64_t best_below(const RowSpan<DT>& row, int first, int step, int v1, uint64_t limit) {
  constexpr int VEC = Elem<DT>::kVec;
  uint64_t best = 0;
  for (int k = first; k < v1; k += step) {
    float x[VEC];
    Elem<DT>::unpack(__ldg(row.body() + k), x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const uint64_t key = ckey_of<DT>(x[e], row.head + static_cast<int64_t>(k) * VEC + e);
      if (key < limit && key > best) best = key;
    }
  }
  return best;
}

template <int DT, int NT, int MINB>
__global__ void __launch_bounds__(NT, MINB) score_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int NW = NT / 32, VEC = Elem<DT>::kVec;
  constexpr int U = 4;  // vectors in flight per thread (and as many again)
  __shared__ float4 red[NW];
  __shared__ float4 table[kMaxSlices];   // (m, s, w) of the slices
  __shared__ float4 bounds[kMaxSlices];  // their K-th and ceil(K / S)-th group maxima
  __shared__ float4 joint;               // (m, s, w) of the row, the bound
  __shared__ uint64_t joined;            // the arrival of the slices' statistics
  __shared__ __align__(16) uint32_t groups[kGroups];  // keys of the groups' maxima, made different by their low bits
  __shared__ float cut[2];
  __shared__ uint64_t pool[kPool], winners[NW];
  __shared__ uint32_t list[NW][kListed], count;
  extern __shared__ float cells[];  // [cell][thread], where there are alternatives
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, S = p.slices, rank = blockIdx.y, K = p.K;
  const int64_t r = blockIdx.x;
  const RowSpan<DT> row(p.logits, r * p.row_stride, p.V);
  const int nvec = static_cast<int>(row.nvec), v0 = min(rank * p.per, nvec), v1 = min(v0 + p.per, nvec);
  RowStream<DT, NT, U> stream(row, v0, v1);
  if (S > 1) {
    if (tid == 0) {
      mbar_init(&joined, 1);
      mbar_init_fence();
      mbar_arrive_expect_tx(&joined, 2 * S * sizeof(float4));
    }
    __syncthreads();
    cluster_arrive_started();  // waited for before the first store into another CTA
  }
  const float T = p.temperature[r];
  const bool scalar = rank == 0 && tid < row.scalars();
  const float xs = scalar ? row.at(row.scalar_index(tid)) : -INFINITY;
  const int32_t token = rank == 0 && tid < p.M ? p.tokens[r * p.M + tid] : -1;
  const bool given = token >= 0 && token < p.V;
  const float xt = given ? row.at(token) : 0.f;
  if (tid == 0) count = 0;  // (of the first CTA: that of all)
  const float c = exponent_scale(T);
  EntropyAcc a;
  int batches = 0;
  const int of_cell = (1 << p.shift) - 1;
  float cell = -INFINITY;  // (a cell without a finite logit reaches no bound)
  stream.batches([&](const uint4(&v)[U]) {
    cell = fmaxf(cell, a.template add<DT, U>(v, c));
    if (K > 0 && (batches & of_cell) == of_cell) {
      cells[(batches >> p.shift) * NT + tid] = cell;
      cell = -INFINITY;
    }
    ++batches;
  });
  if (K > 0 && (batches & of_cell) != 0) cells[(batches >> p.shift) * NT + tid] = cell;
  if (scalar) a.add(xs, c);
  const EntropyStats mine = merge_lanes(a, c);
  if (lane == 0) red[wp] = make_float4(mine.m, mine.s, mine.w, 0.f);
  constexpr int Q = NT / kGroups;  // neighbouring threads of a group
  if (K > 0) {
    float g = a.m;
#pragma unroll
    for (int o = Q / 2; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(kFull, g, o));
    if (tid % Q == 0) groups[tid / Q] = (Keys<DT>::key(g) & ~(kGroups - 1u)) | (tid / Q);
  }
  const bool wrong = __syncthreads_or(token < -1 || token >= p.V) || !temperature_valid(T);
  EntropyStats all = merge_shared(red, NW, c);
  float2 own = make_float2(-FLT_MAX, -FLT_MAX);
  if (K > 0) {  // the group below K - 1 others has the K-th largest maximum; each of a group's threads compares a share
    const uint32_t key = groups[tid / Q];
    int above = 0;
#pragma unroll
    for (int i = 0; i < kGroups / 4 / Q; ++i) {
      const uint4 k = reinterpret_cast<const uint4*>(groups)[i * Q + tid % Q];
      above += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
    }
#pragma unroll
    for (int o = Q / 2; o > 0; o >>= 1) above += __shfl_xor_sync(kFull, above, o);
    const float value = Keys<DT>::value(key & ~(kGroups - 1u));
    if (above == K - 1) cut[0] = value;
    if (above == (K + S - 1) / S - 1) cut[1] = value;
    __syncthreads();
    own = make_float2(cut[0], cut[1]);
  }
  float bound = own.x;
  if (S > 1) {
    cluster_wait();
    if (wp == 0) {
      if (tid < S) {
        const uint32_t bar = dsmem_addr(&joined, tid);
        dsmem_send(dsmem_addr(&table[rank], tid), make_float4(all.m, all.s, all.w, 0.f), bar);
        dsmem_send(dsmem_addr(&bounds[rank], tid), make_float4(own.x, own.y, __uint_as_float(ld_volatile(&count)), 0.f), bar);
      }
      __syncwarp();
      if (__all_sync(kFull, mbar_wait(&joined, 0, 2 * kWaitPolls))) {
        all = merge_shared(table, S, c);
        float low = bounds[0].y;
        bound = bounds[0].x;
        for (int i = 1; i < S; ++i) {
          bound = fmaxf(bound, bounds[i].x);
          low = fminf(low, bounds[i].y);
        }
        if (lane == 0) joint = make_float4(all.m, all.s, all.w, fmaxf(bound, low));
      } else {  // the first CTA: SFC_ROW_TIMEOUT; without another's alternatives, it finds them all one by one
        if (lane == 0) joint = make_float4(-FLT_MAX, kLate, 0.f, 0.f);
        if (lane == 0 && K > 0) dsmem_add(dsmem_addr(&count, 0), kPool + 1);
      }
    }
    __syncthreads();
    all = EntropyStats{joint.x, joint.y, joint.z};
    bound = joint.w;
  }
  const bool valid = stats_valid(all.m, all.s), late = all.s == kLate;  // uniform over the cluster (but for waits that gave up)
  if (K > 0 && valid) {
    const uint32_t counter = S > 1 ? dsmem_addr(&count, 0) : smem_addr(&count);
    const uint32_t places = S > 1 ? dsmem_addr(pool, 0) : smem_addr(pool);
    // What the counter stood at came with the first CTA's statistics: places depend on that value, so that no CTA adds before it.
    auto add = [&](uint32_t n) { return S > 1 ? dsmem_add(counter, n) - __float_as_uint(bounds[0].z) : atomicAdd(&count, n); };
    auto place = [&](uint32_t at, float x, int64_t id) {
      if (at < kPool) dsmem_st64(places + at * 8, ckey_of<DT>(x, id));
    };
    // the warp's cells that reach the bound, then their vectors, one for each lane
    int listed = 0;
    if (__any_sync(kFull, a.m >= bound)) {
      uint32_t in = 0;
      const int of_thread = (batches + of_cell) >> p.shift;
#pragma unroll 8
      for (int i = 0; i < of_thread; ++i) in |= static_cast<uint32_t>(cells[i * NT + tid] >= bound) << i;
      int at = warp_before(__popc(in), listed);
      for (; in && at < kListed; in &= in - 1) list[wp][at++] = (__ffs(in) - 1) * NT + tid;
      __syncwarp();
    }
    if (listed > kListed) {
      if (lane == 0) add(kPool + 1);
      listed = 0;
    }
    const int vectors = listed << (p.shift + 2);
    static_assert(U == 4, "vectors of a batch");
    for (int i = lane; i - lane < vectors; i += 32) {
      const int of = list[wp][min(i, vectors - 1) >> (p.shift + 2)];
      const int at = v0 + of % NT + ((of / NT << (p.shift + 2)) + (i & ((4 << p.shift) - 1))) * NT;
      const uint4 v = i < vectors && at < v1 ? __ldg(row.body() + at) : Elem<DT>::neg_inf_vec();
      uint32_t in = Elem<DT>::ge_mask(v, bound);
      int total;
      const int before = warp_before(__popc(in), total);
      uint32_t to = 0;
      if (lane == 0 && total > 0) to = add(total);
      to = __shfl_sync(kFull, to, 0) + before;
      for (; in; in &= in - 1) {
        const int e = __ffs(in) - 1;
        place(to++, Elem<DT>::get_dyn(v, e), row.head + static_cast<int64_t>(at) * VEC + e);
      }
    }
    if (scalar && xs >= bound) place(add(1), xs, row.scalar_index(tid));
  }
  if (K > 0) {
    __syncwarp();  // the barrier's halves want whole warps
    if (S > 1) cluster_sync_all();  // no CTA touches another's memory after it
    else __syncthreads();
  }
  if (rank != 0) return;
  const bool ok = valid && !wrong;
  const float nan = __int_as_float(0x7fc00000), ln_s = all.log_sum();
  auto logprob = [&](float x) { return below_max(x, all.m, [&](float d) { return d / T; }) - ln_s; };
  if (tid < p.M) p.logprobs[r * p.M + tid] = !ok ? nan : given ? logprob(xt) : 0.f;
  if (tid == 0) {
    const float H = all.entropy(ln_s);
    p.entropy[r] = ok ? H : nan;
    p.row_status[r] = ok ? SFC_ROW_OK : late ? SFC_ROW_TIMEOUT : SFC_ROW_BADPARAM;
    if (p.stats) p.stats[r] = make_float4(ok ? all.m : nan, all.s, H, 0.f);
  }
  if (K == 0) return;
  auto put = [&](int j, uint64_t key) {  // 0: no alternative in this place
    p.top_ids[r * K + j] = key ? static_cast<int32_t>(ckey_id(key)) : -1;
    p.top_logprobs[r * K + j] = key ? logprob(Keys<DT>::value(ckey_key(key))) : ok ? -INFINITY : nan;
  };
  const int n = ok ? count : 0;
  if (n <= static_cast<int>(kPool)) {
    if (tid < K && tid >= n) put(tid, 0ull);
    for (int i0 = 0; i0 < n; i0 += NT / 4) {  // four lanes count the keys above one
      const int i = i0 + tid / 4;
      const uint64_t key = pool[min(i, n - 1)];
      int above = 0;
      for (int j = tid & 3; j < n; j += 4) above += pool[j] > key;
      above += __shfl_xor_sync(kFull, above, 1);
      above += __shfl_xor_sync(kFull, above, 2);
      if (i < n && above < K && (tid & 3) == 0) put(above, key);
    }
    return;
  }
  auto next = [&](int of, uint64_t limit) {  // the largest key of thread `of` (of the whole row's) below the limit, by its warp
    uint64_t key = best_below<DT>(row, of + lane * NT, 32 * NT, nvec, limit);
    if (scalar && tid == of) {
      const uint64_t k = ckey_of<DT>(xs, row.scalar_index(tid));
      if (k < limit && k > key) key = k;
    }
    return warp_max_key(key);
  };
  uint64_t best = scalar ? ckey_of<DT>(xs, row.scalar_index(tid)) : 0ull;
  float most = -INFINITY;  // in the vectors: ties keep the first
  for (int k = tid; k < nvec; k += NT) {
    const uint4 v = __ldg(row.body() + k);
    if (!(Elem<DT>::vmax(v) > most)) continue;
    most = Elem<DT>::vmax(v);
    float x[VEC];
    Elem<DT>::unpack(v, x);
    int first = 0;
#pragma unroll
    for (int e = VEC - 1; e >= 0; --e)
      if (x[e] == most) first = e;
    best = max(best, ckey_of<DT>(most, row.head + static_cast<int64_t>(k) * VEC + first));
  }
  for (int j = 0; j < K; ++j) {
    const uint64_t w = warp_max_key(best);
    if (lane == 0) winners[wp] = w;
    __syncthreads();
    uint64_t top = winners[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) top = max(top, winners[i]);
    __syncthreads();
    if (tid == 0) put(j, top);
    if (top != 0 && w == top) {  // the winner's warp: uniform
      const int l = __ffs(__ballot_sync(kFull, best == top)) - 1;
      const uint64_t k = next(wp * 32 + l, top);
      if (lane == l) best = k;
    }
  }
}

struct ScoreGradParams {
  const void* logits;
  int64_t row_stride, V;
  const float* temperature;
  const int32_t* tokens;
  int32_t M;
  const float4* stats;
  const float* grad_logprobs;
  const float* grad_entropy;
  unsigned char* grad;
  int64_t grad_stride;
  int32_t per;  // vectors a slice
};

constexpr int kMaxEntries = SFC_MAX_GIVEN + SFC_MAX_TOP;

// Every CTA takes the row's tokens (few) and one slice of its logits. The dense part is written first; after the CTA's
// barrier the first place of each token that lies in the slice overwrites its entry with the whole gradient, rounded once.
template <int DT, int NT, int MINB>
__global__ void __launch_bounds__(NT, MINB) score_backward_kernel(const __grid_constant__ ScoreGradParams p) {
  constexpr int VEC = Elem<DT>::kVec;
  constexpr int U = 4;
  __shared__ int32_t ids[kMaxEntries];
  __shared__ float gs[kMaxEntries];
  const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.y;
  const int64_t r = blockIdx.x;
  const RowSpan<DT> row(p.logits, r * p.row_stride, p.V);
  const int nvec = static_cast<int>(row.nvec), v0 = min(rank * p.per, nvec), v1 = min(v0 + p.per, nvec);
  RowStream<DT, NT, U> stream(row, v0, v1);
  const bool scalar = rank == 0 && tid < row.scalars();
  const float4 st = p.stats[r];
  const float T = p.temperature[r], c = exponent_scale(T), inv_T = fminf(1.f / T, FLT_MAX);
  const bool live = st.x == st.x;  // rows without a log-probability pass no gradient on
  float h = p.grad_entropy ? p.grad_entropy[r] * inv_T : 0.f;
  float own_x = 0.f;
  if (tid < p.M) {  // a masked token's log-probability is the constant -inf
    const int32_t id = p.tokens[r * p.M + tid];
    const bool in = id >= 0 && id < p.V;
    own_x = in ? row.at(id) : -INFINITY;
    ids[tid] = own_x > -INFINITY ? id : -1;
    gs[tid] = own_x > -INFINITY && p.grad_logprobs ? p.grad_logprobs[r * p.M + tid] * inv_T : 0.f;
  }
  __syncthreads();
  float G = 0.f;
  for (int j = lane; j < p.M; j += 32) G += gs[j];
  G = warp_total(G);
  if (large(G, h)) {  // quotients that overflow are held (uniform; upstream gradients that are not finite stay)
    auto hold = [](float q, float up) { return fabsf(up) < INFINITY ? held(q) : q; };
    if (p.grad_entropy) h = hold(h, p.grad_entropy[r]);
    __syncthreads();
    if (tid < p.M && ids[tid] >= 0 && p.grad_logprobs) gs[tid] = hold(gs[tid], p.grad_logprobs[r * p.M + tid]);
    __syncthreads();
    G = 0.f;
    for (int j = lane; j < p.M; j += 32) G += gs[j];
    G = warp_total(G);
  }
  const RowGradient dense(st.x, st.y, logf(st.y), st.z, G, h, c);
  unsigned char* grad = p.grad + r * p.grad_stride * Elem<DT>::kBytes;
  unsigned char* out = grad + static_cast<int64_t>(row.head) * Elem<DT>::kBytes;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 15);
  if (!live) {
    for (int i = v0 + tid; i - lane < v1; i += NT)
      store_vector<DT>(out + static_cast<int64_t>(i) * 16, make_uint4(0u, 0u, 0u, 0u), shift, i < v1);
  } else if (dense.lifted) {
    write_lifted<DT, NT>(dense, row, out, shift, v0, v1);
  } else {
    stream.each([&](const uint4& w, int i) {
      store_vector<DT>(out + static_cast<int64_t>(i) * 16, dense.template vector<DT>(w), shift, i < v1);
    });
  }
  if (scalar) {
    const int64_t i = row.scalar_index(tid);
    Out<DT>::store1(grad, i, live ? dense.at(row.at(i)) : 0.f);
  }
  if (!live) return;
  __syncthreads();  // the dense values are written before the tokens' overwrite theirs
  if (tid >= p.M || ids[tid] < 0) return;
  const int64_t id = ids[tid], lo = row.head + static_cast<int64_t>(v0) * VEC, hi = row.head + static_cast<int64_t>(v1) * VEC;
  if (!(id >= lo && id < hi) && !(rank == 0 && (id < row.head || id >= row.tail()))) return;
  float g = 0.f;
  for (int j = 0; j < p.M; ++j) {
    if (ids[j] != id) continue;
    if (j < tid) return;  // an earlier place of the same token writes it
    g += gs[j];
  }
  Out<DT>::store1(grad, id, dense.at(own_x) + g);
}

int check_rows(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* temperature) {
  if (!logits || !temperature) return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || row_stride < V) return SFC_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SFC_BF16 ? 2 : 4)) return SFC_EINVAL;
  return SFC_OK;
}

int32_t slice_of(int64_t vectors, int64_t slices) {  // in whole 128-byte lines
  return static_cast<int32_t>((vectors + slices - 1) / slices + 7) & ~7;
}

template <int DT, int NT, int MINB>
cudaError_t start(ScoreParams p, int64_t B, cudaStream_t stream) {
  p.per = slice_of(p.V / Elem<DT>::kVec, p.slices);
  cudaLaunchConfig_t cfg = {};
  p.shift = DT == 0 ? 0 : 1;  // cells of 32 elements, larger where a thread has too many
  if (p.K > 0) {
    const int most = std::min(kCells, kCellBytes / 4 / NT), batches = (p.per + 4 * NT - 1) / (4 * NT);
    while ((batches >> p.shift) + 1 > most) ++p.shift;
    cfg.dynamicSmemBytes = static_cast<size_t>((batches >> p.shift) + 1) * NT * sizeof(float);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(B), static_cast<unsigned>(p.slices));
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {1, static_cast<unsigned>(p.slices), 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, score_kernel<DT, NT, MINB>, p);
}

template <int DT>
cudaError_t choose(ScoreParams& p, int64_t B, cudaStream_t stream) {
  const int64_t vectors = p.V / Elem<DT>::kVec;
  // Few rows: slices for every SM (two or four or eight: clusters of other sizes leave SMs out; 24 x 151936 bf16 with six 6.3
  // us, four 5.7), and CTAs as large as keeps some vectors for each thread (1 x 151936: of 256 4.0 us, of 512 4.4; 64 x 151936
  // 10.4 : 7.9). Twice the slices: 64 x 151936 in two of 512 7.6 us, with 5 alternatives 10.3, in four of 256 7.5 and 10.5, in
  // eight of 128 7.7 and 11.2; 128 rows in one of 512 11.1 and 13.5, in two of 256 11.7 and 14.8; 200 rows 17.5 and 21.1, 15.3 and
  // 18.8; 256 rows 17.8 and 21.3, 19.1 and 23.3. Many rows: one CTA each, of a size of which several take turns on a SM. Without
  // alternatives and with 20, 2048 bf16 rows in CTAs of 128 : of 256: x 32000 26.0 and 35.3 : 26.2 and 38.8, x 56000 43.1 and 52.8 :
  // 42.1 and 54.0, x 65000 48.8 and 57.8 : 47.3 and 58.8, x 151936 106.6 and 118.2 : 100.5 and 113.6 (of 512 128 with 20, of 256 cut
  // in two 129: each slice goes through the choice); 1024 f32 rows: x 50000 35.1 and 39.6 : 37.7 and 44.1, x 129280 82.0 and 88.1 :
  // 85.5 and 93.4 (the bound is the one that bf16 wants). Groups of a CTA's threads need vectors to look at: rows below 1024 have
  // CTAs of 128.
  p.slices = 1;
  while (p.slices < kMaxSlices && 2 * p.slices * B <= 152 && vectors >= 4096 * p.slices) p.slices *= 2;
  if (B > 304) return p.V <= 56000 ? start<DT, 128, 8>(p, B, stream) : start<DT, 256, 4>(p, B, stream);
  if (vectors <= 1024) return start<DT, 128, 8>(p, B, stream);
  if (vectors / p.slices <= 3200) return start<DT, 256, 4>(p, B, stream);
  return start<DT, 512, 2>(p, B, stream);
}

template <int DT, int NT, int MINB>
cudaError_t start_backward(ScoreGradParams p, int64_t B, int64_t slices, cudaStream_t stream) {
  p.per = slice_of(p.V / Elem<DT>::kVec, slices);
  score_backward_kernel<DT, NT, MINB><<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(slices)), NT, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t choose_backward(const ScoreGradParams& p, int64_t B, cudaStream_t stream) {
  const int64_t vectors = p.V / Elem<DT>::kVec;
  // many short rows: several small CTAs take turns on a SM
  if (B >= 304 && vectors <= 1656) return start_backward<DT, 128, 8>(p, B, 1, stream);
  if (B >= 304 && vectors <= 3320) return start_backward<DT, 256, 4>(p, B, 1, stream);
  // slices of 320 KB at most; few rows: enough to fill the GPU's 304 CTA slots, of at least two vectors per thread
  const int64_t fill = std::min<int64_t>({8, (vectors + 1023) / 1024, (304 + B - 1) / B});
  return start_backward<DT, 512, 2>(p, B, std::max<int64_t>({1, (vectors + 20479) / 20480, fill}), stream);
}

int result(cudaError_t err) {
  if (err == cudaSuccess) return SFC_OK;
  (void)cudaGetLastError();
  return SFC_ECUDA;
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_token_logprobs(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                  const float* temperature, const int32_t* tokens, int32_t M, int32_t top, float* logprobs,
                                  float* entropy, int32_t* top_ids, float* top_logprobs, float* row_stats, int32_t* row_status,
                                  void* stream) {
  const int rc = sfc::check_rows(logits, dtype, B, V, row_stride, temperature);
  if (rc != SFC_OK) return rc;
  if (M < 0 || M > SFC_MAX_GIVEN || (M > 0 && (!tokens || !logprobs))) return SFC_EINVAL;
  if (top < 0 || top > SFC_MAX_TOP || (top > 0 && (!top_ids || !top_logprobs))) return SFC_EINVAL;
  if (!entropy || !row_status || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  sfc::ScoreParams p{logits, row_stride, V, temperature, tokens, M, top, logprobs, entropy, top_ids, top_logprobs,
                     reinterpret_cast<float4*>(row_stats), row_status, 1, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return sfc::result(dtype == SFC_BF16 ? sfc::choose<0>(p, B, st) : sfc::choose<1>(p, B, st));
}

extern "C" int sfc_token_logprobs_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                           const float* temperature, const int32_t* tokens, int32_t M, const float* row_stats,
                                           const float* grad_logprobs, const float* grad_entropy, void* grad_logits,
                                           int64_t grad_stride, void* stream) {
  const int rc = sfc::check_rows(logits, dtype, B, V, row_stride, temperature);
  if (rc != SFC_OK) return rc;
  if (M < 0 || M > sfc::kMaxEntries || (M > 0 && !tokens) || !row_stats || !grad_logits || grad_stride < V) return SFC_EINVAL;
  const int64_t elt = dtype == SFC_BF16 ? 2 : 4;
  const uintptr_t g = reinterpret_cast<uintptr_t>(grad_logits), l = reinterpret_cast<uintptr_t>(logits);
  if (g % elt || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  if (g < l + ((B - 1) * row_stride + V) * elt && l < g + ((B - 1) * grad_stride + V) * elt) return SFC_EINVAL;
  const sfc::ScoreGradParams p{logits, row_stride, V, temperature, tokens, M, reinterpret_cast<const float4*>(row_stats), grad_logprobs,
                               grad_entropy, static_cast<unsigned char*>(grad_logits), grad_stride, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return sfc::result(dtype == SFC_BF16 ? sfc::choose_backward<0>(p, B, st) : sfc::choose_backward<1>(p, B, st));
}
