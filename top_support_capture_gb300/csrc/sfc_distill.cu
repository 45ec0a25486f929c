// Distillation of a student from a teacher's top logits: the loss of each row against a packed teacher
// distribution (a captured support and its log-probabilities, or raw top logits), and its gradient.
//
//   z = x / T, ln p = z - ln sum_V exp z;  t_i = exp(y_i), or softmax over the row's entries of y_i / T
//   loss = sum_i t_i (ln t_i - ln p_i),   dloss/dx_j = (tau p_j - t_j) / T,   tau = sum_i t_i
//
// A row is cut into slices of 16-byte vectors, one CTA each. In the calls that need the row's statistics the
// slices of a row form a thread-block cluster: each CTA stores its share of the statistics into every CTA of the
// cluster (distributed shared memory), and after the cluster's barrier each merges the shares in slice order, so
// all hold the same bits. The teacher's mass is small work: every CTA sums it for itself.
//
// In the call that gives loss and gradient the slice stays in shared memory between its two uses, so the logits are
// read from HBM once: one thread starts a bulk copy of it before anything else. The wait for the copy is bounded
// (SFC_ROW_TIMEOUT). Rows longer than a cluster's shared memory are read again.
//
// 2048 x 151936 bf16, loss and gradient: 245 us, 0.75 of the measured copy rate (2 x 622 MB). The two CTAs of a SM
// read, compute and write in turns; before the prefetch, which lets HBM work while they compute (258 -> 245 us), the copies
// alone took 126 us, the folds 24, the teacher's entries and merges 44, the gradient's rows 70, added up. Measured
// against that: one CTA per row that streams it twice 313-360 us (the second pass
// finds 8 % in L2); the slice in registers, five CTAs a row 422; the copy in two or four parts that are waited for one by
// one 262 / 274; three or four CTAs a SM in clusters of five or six 282 / 268 (each thread's fixed work grows); clusters that go from row to row
// and start the next copy as the slice is used up 248, at 9.0 instead of 7.4 us for 64 x 32000 and twice the code.
//
// The gradient's dense part tau p_j g / T is written first; after the CTA's barrier the teacher's entries that lie
// in the slice overwrite theirs with the whole gradient, each rounded once, and add their part of the loss.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/sfc.h"
#include "sfc_host.cuh"
#include "sfc_rows.cuh"

namespace sfc {
namespace {

struct DistillParams {
  const void* logits;
  int64_t row_stride, V;
  int32_t W;
  bool normalise;
  const float* temperature;
  const int32_t* ids;
  const float* values;
  const int32_t* lengths;
  const float* grad_loss;
  float* loss;
  float4* stats;  // out (forward) or in (backward)
  int32_t* row_status;
  unsigned char* grad;
  int64_t grad_stride;
  int32_t slices, per;  // CTAs a row, vectors a slice
  bool stall;           // test of the failure path: the copies are never started
};

// What the gradient needs of a row: its softmax (m, s) and its teacher's: t_i = exp((y_i - y0) / T_y) / ty, tau.
// m is NaN on rows that pass no gradient on (no teacher entry, bad parameters).
struct RowTerms {
  float m, s, tau, y0, ty;
};

// Statistics as they are kept between the forward and the backward call: (m, s, tau, 0), or with normalised
// teachers (tau = 1) (m, s, y0, ty).
__device__ __forceinline__ float4 pack_terms(const RowTerms& t, bool normalise) {
  return normalise ? make_float4(t.m, t.s, t.y0, t.ty) : make_float4(t.m, t.s, t.tau, 0.f);
}
__device__ __forceinline__ RowTerms unpack_terms(const float4& v, bool normalise) {
  return normalise ? RowTerms{v.x, v.y, 1.f, v.z, v.w} : RowTerms{v.x, v.y, v.z, 0.f, 1.f};
}

constexpr int kMaxSlices = 8;  // the portable cluster size
constexpr int kKeepBytes = 212992;  // shared memory of one SM that keeps logits: 13 vectors for each of 1024 threads
constexpr uint32_t kStallPolls = 16;
constexpr float kLate = -1.f;  // in place of a mass: a copy did not arrive

__device__ __forceinline__ void prefetch_l2(const void* from, uint32_t bytes) {  // 16-byte aligned, a multiple of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// KEEP: the slice's vectors lie in dynamic shared memory (16 bytes for each).
template <int DT, int NT, int MINB, bool KEEP, bool FWD, bool BWD>
__global__ void __launch_bounds__(NT, MINB) distill_kernel(const __grid_constant__ DistillParams p) {
  constexpr int NW = NT / 32, VEC = Elem<DT>::kVec;
  constexpr int U = 4;  // vectors in flight per thread where they are not kept (and as many again)
  constexpr int kAhead = 76 * MINB;  // CTAs that a prefetch runs ahead: half of what runs at once (a quarter to all: within 2 %)
  constexpr int kBatch = KEEP ? 2 : 4;  // teacher entries that a thread has on their way at once
  extern __shared__ __align__(128) uint4 kept[];
  __shared__ uint64_t full;
  __shared__ float2 red[2 * NW];
  __shared__ float red_mass[NW], red_loss[NW];
  __shared__ float2 table[kMaxSlices];  // (m, s) of the slices
  __shared__ float losses[kMaxSlices];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, S = p.slices, rank = blockIdx.y;
  const int64_t r = blockIdx.x;
  const RowSpan<DT> row(p.logits, r * p.row_stride, p.V);
  const uint4* body = row.body();
  const int nvec = static_cast<int>(row.nvec), v0 = min(rank * p.per, nvec), v1 = min(v0 + p.per, nvec), mine = v1 - v0;
  const bool scalar = rank == 0 && tid < row.scalars();
  if (KEEP) {  // on their way while the row's parameters load
    if (tid == 0) {
      mbar_init(&full, 1);
      mbar_init_fence();
      if (!p.stall) {
        mbar_arrive_expect_tx(&full, mine * 16);
        if (mine > 0) bulk_load(kept, body + v0, mine * 16, &full);
      }
    }
    __syncthreads();  // the barrier exists
  }
  if (FWD && S > 1) cluster_arrive();  // the cluster's CTAs have started: waited for before the first store into another
  const float T = p.temperature[r];
  const int len = p.lengths[r];
  const int n = min(max(len, 0), p.W);
  const int32_t* ids = p.ids + r * p.W;
  const float* values = p.values + r * p.W;
  // the row's entries, a batch at a time (the first is on its way from here): use(ids, values), past the end -1
  struct Entries {
    int32_t id[kBatch];
    float y[kBatch];
  };
  auto load = [&](int j0) {
    Entries b;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int j = j0 + e * NT;
      b.id[e] = j < n ? ids[j] : -1;
      b.y[e] = j < n ? values[j] : 0.f;
    }
    return b;
  };
  const Entries first = load(tid);
  auto entries = [&](auto use) {
    Entries b = first;
    for (int j0 = tid; j0 < n; j0 += kBatch * NT) {
      const Entries next = load(j0 + kBatch * NT);
      use(b, j0);
      b = next;
    }
  };
  const float c = exponent_scale(T), inv_T = fminf(1.f / T, FLT_MAX), inv_Ty = p.normalise ? inv_T : 1.f;
  RowTerms q{__int_as_float(0x7fc00000), 1.f, 0.f, 0.f, 1.f};
  int status = SFC_ROW_OK;
  bool live;  // the row has a teacher and passes its checks: uniform over its CTAs
  if (FWD) {
    if (len > p.W) status = SFC_ROW_OVERFLOW;
    if (!temperature_valid(T) || len < 0) status = SFC_ROW_BADPARAM;
    live = status != SFC_ROW_BADPARAM && n > 0;
    bool late = false;
    if (live) {
      // the teacher: its mass, or its maximum and normaliser; an id outside the row makes it NaN
      SoftmaxAcc a, t;
      float mass = 0.f;
      auto teacher_mass = [&] {
        entries([&](const Entries& b, int j0) {
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            if (j0 + e * NT >= n) break;
            const float v = b.id[e] < 0 || b.id[e] >= p.V ? __int_as_float(0x7fc00000) : b.y[e];
            if (p.normalise) t.add(v, c);
            else mass += expf(v);
          }
        });
      };
      auto fold = [&](const uint4& w) {
        float x[VEC];
        Elem<DT>::unpack(w, x);
        a.add(x, Elem<DT>::vmax(w), c);
      };
      if (KEEP) {
        teacher_mass();
        late = !__all_sync(kFull, mbar_wait(&full, 0, p.stall ? kStallPolls : kWaitPolls));
        if (tid == 0 && r + kAhead / S < gridDim.x) {  // a later CTA's slice on its way to L2 while HBM would idle
          const RowSpan<DT> later(p.logits, (r + kAhead / S) * p.row_stride, p.V);
          const int vecs = static_cast<int>(later.nvec), at = min(rank * p.per, vecs), bytes = (min(at + p.per, vecs) - at) * 16;
          if (bytes > 0) prefetch_l2(later.body() + at, bytes);
        }
        if (!late) {
#pragma unroll 2
          for (int k = tid; k < mine; k += NT) fold(kept[k]);
        }
      } else {
        RowStream<DT, NT, U> stream(row, v0, v1);
        teacher_mass();
        stream.each([&](const uint4& w, int) { fold(w); });
      }
      if (scalar) a.add(row.at(row.scalar_index(tid)), c);
      const SoftmaxStats w = warp_stats(a, c);
      if (lane == 0) red[wp] = make_float2(w.m, w.s);
      if (p.normalise) {
        const SoftmaxStats wt = warp_stats(t, c);
        if (lane == 0) red[NW + wp] = make_float2(wt.m, wt.s);
      } else {
        mass = warp_total(mass);
        if (lane == 0) red_mass[wp] = mass;
      }
      if (KEEP) late = __syncthreads_or(late);
      else __syncthreads();
      SoftmaxStats all = merge_warps<NT>(red, c);
      if (KEEP && late) all = SoftmaxStats{-FLT_MAX, kLate};
      if (S > 1) {
        cluster_wait();
        if (tid < S) dsmem_st64(dsmem_addr(&table[rank], tid), pack_f2(all.m, all.s));
        cluster_sync_all();
        // one lane per slice: its maximum first, then each mass rescaled, summed in a fixed order
        const float2 v = table[lane < S ? lane : 0];
        late = __any_sync(kFull, v.y == kLate);
        all.m = warp_max(v.x);
        all.s = warp_total(lane < S ? v.y * ex2_approx((v.x - all.m) * c) : 0.f);
      }
      q = RowTerms{all.m, all.s, 1.f, 0.f, 1.f};
      live = stats_valid(all.m, all.s);
      if (p.normalise) {
        const SoftmaxStats teacher = merge_warps<NT>(red + NW, c);
        q.y0 = teacher.m;
        q.ty = teacher.s;
        live = live && stats_valid(teacher.m, teacher.s);
      } else {
        q.tau = warp_total(lane < NW ? red_mass[lane] : 0.f);
        live = live && q.tau < INFINITY;
      }
      if (KEEP && late) live = false;
      if (!live) {
        status = KEEP && late ? SFC_ROW_TIMEOUT : SFC_ROW_BADPARAM;
        q.m = __int_as_float(0x7fc00000);
      }
    } else if (S > 1) {
      cluster_wait();
      cluster_sync_all();
    }
    // nothing of the CTA's is still in flight when it ends
    if (KEEP && !live && tid == 0 && !p.stall) mbar_wait(&full, 0);
  } else {
    q = unpack_terms(p.stats[r], p.normalise);
    live = q.m == q.m;
  }
  const float g = BWD && live ? p.grad_loss[r] * inv_T : 0.f;
  const float k = live ? g * q.tau / q.s : 0.f, m = q.m;
  unsigned char* grad = BWD ? p.grad + r * p.grad_stride * Elem<DT>::kBytes : nullptr;
  if (BWD) {
    unsigned char* out = grad + static_cast<int64_t>(row.head) * Elem<DT>::kBytes;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 15);
    const uint64_t minus_m2 = pack_f2(-m, -m), c2 = pack_f2(c, c), k2 = pack_f2(k, k);
    auto gradient = [&](const uint4& w) {
      float x[VEC];
      Elem<DT>::unpack(w, x);
      uint64_t e2[VEC / 2];
      exponentials(x, minus_m2, c2, e2);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) unpack_f2(fmul_f2(e2[e], k2), x[2 * e], x[2 * e + 1]);
      return Out<DT>::pack(x);
    };
    const bool by_warp = DT == 0 && shift != 0;
    auto put = [&](int at, const uint4& w) {
      unsigned char* to = out + static_cast<int64_t>(at) * 16;
      if (by_warp) {
        store_shifted(to, w, shift, at < v1);
      } else if (at < v1) {
        if (shift == 0) {
          *reinterpret_cast<uint4*>(to) = w;
        } else {
          uint32_t* four = reinterpret_cast<uint32_t*>(to);
          four[0] = w.x, four[1] = w.y, four[2] = w.z, four[3] = w.w;
        }
      }
    };
    if (!live) {
      for (int i = v0 + tid; i - lane < v1; i += NT) put(i, make_uint4(0u, 0u, 0u, 0u));
    } else if (KEEP && by_warp) {
      for (int i = tid; i - lane < mine; i += NT) put(v0 + i, gradient(kept[min(i, mine - 1)]));
    } else if (KEEP) {
#pragma unroll 2
      for (int i = tid; i < mine; i += NT) put(v0 + i, gradient(kept[i]));
    } else {
      RowStream<DT, NT, U> stream(row, v0, v1);
      stream.each([&](const uint4& w, int at) { put(at, gradient(w)); });
    }
    if (scalar) {
      const int64_t i = row.scalar_index(tid);
      Out<DT>::store1(grad, i, live ? k * ex2_approx((row.at(i) - m) * c) : 0.f);
    }
    if (live) __syncthreads();  // the dense values are written before the teacher's entries overwrite theirs
  }
  float loss = 0.f;
  if (live) {
    const float ln_ty = p.normalise ? logf(q.ty) : 0.f;
    const int32_t lo = row.head + v0 * VEC, span = (v1 - v0) * VEC, tail = static_cast<int32_t>(row.tail());
    entries([&](const Entries& b, int) {
      float x[kBatch];
      bool here[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {  // an entry of this slice (the first has the elements outside the body); in the
        // gradient's own call the ids may be others than those that the forward call checked
        const int32_t i = b.id[e];
        const bool body_entry = static_cast<uint32_t>(i - lo) < static_cast<uint32_t>(span);
        here[e] = body_entry || (rank == 0 && i >= 0 && (FWD || i < p.V) && (i < row.head || i >= tail));
        x[e] = !here[e] ? 0.f
               : KEEP && body_entry ? Elem<DT>::load1(reinterpret_cast<const unsigned char*>(kept), i - lo)
                                    : row.at(i);
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (!here[e]) continue;
        const float ln_t = (b.y[e] - q.y0) * inv_Ty - ln_ty, w = expf(ln_t);
        if (FWD && w > 0.f) loss += w * (ln_t - (x[e] - m) * inv_T);
        if (BWD) Out<DT>::store1(grad, b.id[e], k * ex2_approx((x[e] - m) * c) - w * g);
      }
    });
  }
  if (!FWD) return;
  loss = warp_total(loss);
  if (lane == 0) red_loss[wp] = loss;
  __syncthreads();
  if (S > 1) {
    if (tid == 0) {
      loss = red_loss[0];
      for (int i = 1; i < NW; ++i) loss += red_loss[i];
      dsmem_st32(dsmem_addr(&losses[rank], 0), __float_as_uint(loss));
    }
    cluster_sync_all();
    if (rank != 0) return;
  }
  if (tid == 0) {
    loss = S > 1 ? losses[0] : red_loss[0];
    for (int i = 1; i < (S > 1 ? S : NW); ++i) loss += S > 1 ? losses[i] : red_loss[i];
    p.loss[r] = live ? loss + q.tau * logf(q.s) : (status < 0 ? __int_as_float(0x7fc00000) : 0.f);
    p.row_status[r] = status;
    if (p.stats) p.stats[r] = pack_terms(q, p.normalise);
  }
}

int check(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* temperature,
          const int32_t* ids, const float* values, const int32_t* lengths, int32_t W, uint32_t flags,
          uint32_t known_flags = SFC_FLAG_NORMALISE_TEACHER) {
  if (!logits || !temperature || !ids || !values || !lengths) return SFC_EINVAL;
  if (dtype != SFC_BF16 && dtype != SFC_F32) return SFC_EINVAL;
  if (B < 1 || B > INT32_MAX || V < 1 || V > INT32_MAX || row_stride < V) return SFC_EINVAL;
  if (W < 1 || W > SFC_MAX_PACKED_WIDTH) return SFC_EINVAL;
  if (flags & ~known_flags) return SFC_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SFC_BF16 ? 2 : 4)) return SFC_EINVAL;
  return SFC_OK;
}

// The gradient's array: element-aligned, rows that do not overlap, and no byte shared with the logits.
int check_grad(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* grad_loss,
               const void* grad, int64_t grad_stride) {
  const int64_t elt = dtype == SFC_BF16 ? 2 : 4;
  if (!grad_loss || !grad || grad_stride < V) return SFC_EINVAL;
  const uintptr_t g = reinterpret_cast<uintptr_t>(grad), l = reinterpret_cast<uintptr_t>(logits);
  if (g % elt) return SFC_EINVAL;
  const uintptr_t g_end = g + ((B - 1) * grad_stride + V) * elt, l_end = l + ((B - 1) * row_stride + V) * elt;
  return g < l_end && l < g_end ? SFC_EINVAL : SFC_OK;
}

template <int DT, int NT, int MINB, bool KEEP, bool FWD, bool BWD>
cudaError_t start(DistillParams p, int64_t B, cudaStream_t stream) {
  auto kern = distill_kernel<DT, NT, MINB, KEEP, FWD, BWD>;
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
  cfg.numAttrs = FWD && p.slices > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT, bool FWD, bool BWD>
cudaError_t choose(DistillParams& p, int64_t B, cudaStream_t stream) {
  const int64_t vectors = p.V / Elem<DT>::kVec;
  auto cut = [&](int64_t per) { return std::max<int64_t>(1, (vectors + per - 1) / per); };
  auto fits = [&](int64_t S) {
    p.slices = static_cast<int32_t>(std::min<int64_t>(S, kMaxSlices));
    return S <= kMaxSlices;
  };
  // few rows: enough slices to fill the GPU's 304 CTA slots, of at least two vectors per thread
  const int64_t fill = std::min<int64_t>({kMaxSlices, cut(1024), (304 + B - 1) / B});
  // Rows that one CTA holds, enough of them to fill the GPU: the smaller the CTA the better, since each thread's fixed
  // work and the CTA's barriers weigh less and more CTAs take turns on a SM (2048 rows, loss and gradient: 5000 bf16 12.6
  // us against 30.9 with two CTAs of 512 a SM, 12000 20.6 : 36.2, 26000 39 : 48, 32000 51 : 57; the gradient alone 16.8 :
  // 32.5, 26.0 : 37.5, 48.5 : 54.2, 54.9 : 59.7; the loss alone 15.1 : 20.0 and 18.4 : 24.7 with CTAs of 128 against 256).
  // The loss alone stays in CTAs of 256, of which four and not three fit a SM (32000: 34.9, with 384 41.5; 608 rows 12.2 : 17.0).
  if (B >= 304) {
    if (vectors <= kKeepBytes / 8 / 16 - 8 && fits(1)) return start<DT, 128, 8, FWD && BWD, FWD, BWD>(p, B, stream);
    if (vectors <= kKeepBytes / 4 / 16 - 8 && fits(1)) return start<DT, 256, 4, FWD && BWD, FWD, BWD>(p, B, stream);
    if constexpr (BWD)
      if (vectors <= kKeepBytes / 3 / 16 - 8 && fits(1)) return start<DT, 384, 3, FWD, FWD, true>(p, B, stream);
  }
  if constexpr (FWD && BWD) {  // a slice, in whole 128-byte lines, within its CTA's shared memory
    if (fits(std::max(fill, cut(kKeepBytes / 2 / 16 - 8)))) return start<DT, 512, 2, true, true, true>(p, B, stream);
    if (fits(cut(kKeepBytes / 16 - 8))) return start<DT, 1024, 1, true, true, true>(p, B, stream);
  }
  // the gradient alone needs no cluster: slices of 320 KB (2048 x 151936 bf16 222 us, of 128 KB 248)
  fits(FWD ? fill : std::max(fill, cut(20480)));
  // the loss alone in CTAs of 256 (64 x 151936 bf16 9.5 us, of 512 13.4) unless each has a SM to itself (8 x 262144 7.4,
  // 6.5), the gradient alone in CTAs of 512 (2048 x 151936 222 us, of 256 238)
  if constexpr (FWD && !BWD)
    if (B * p.slices > 152) return start<DT, 256, 4, false, true, false>(p, B, stream);
  return start<DT, 512, 2, false, FWD, BWD>(p, B, stream);
}

template <bool FWD, bool BWD>
int launch(DistillParams p, int dtype, int64_t B, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == SFC_BF16 ? choose<0, FWD, BWD>(p, B, st) : choose<1, FWD, BWD>(p, B, st);
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}

}  // namespace
}  // namespace sfc

extern "C" int sfc_distill_forward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                   const float* temperature, const int32_t* teacher_ids, const float* teacher_values,
                                   const int32_t* lengths, int32_t packed_width, uint32_t flags, float* loss,
                                   float* row_stats, int32_t* row_status, void* stream) {
  const int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                            packed_width, flags);
  if (rc != SFC_OK) return rc;
  if (!loss || !row_status || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, nullptr, loss,
                             reinterpret_cast<float4*>(row_stats), row_status, nullptr, 0, 1, 0, false};
  return sfc::launch<true, false>(p, dtype, B, stream);
}

extern "C" int sfc_distill_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                    const float* temperature, const int32_t* teacher_ids, const float* teacher_values,
                                    const int32_t* lengths, int32_t packed_width, uint32_t flags,
                                    const float* row_stats, const float* grad_loss, void* grad_logits,
                                    int64_t grad_stride, void* stream) {
  int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                      packed_width, flags);
  if (rc == SFC_OK) rc = sfc::check_grad(logits, dtype, B, V, row_stride, grad_loss, grad_logits, grad_stride);
  if (rc != SFC_OK) return rc;
  if (!row_stats || reinterpret_cast<uintptr_t>(row_stats) % 16) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, grad_loss, nullptr,
                             const_cast<float4*>(reinterpret_cast<const float4*>(row_stats)), nullptr,
                             static_cast<unsigned char*>(grad_logits), grad_stride, 1, 0, false};
  return sfc::launch<false, true>(p, dtype, B, stream);
}

extern "C" int sfc_distill_forward_backward(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                                            const float* temperature, const int32_t* teacher_ids,
                                            const float* teacher_values, const int32_t* lengths,
                                            int32_t packed_width, uint32_t flags, const float* grad_loss, float* loss,
                                            int32_t* row_status, void* grad_logits, int64_t grad_stride,
                                            void* stream) {
  int rc = sfc::check(logits, dtype, B, V, row_stride, temperature, teacher_ids, teacher_values, lengths,
                      packed_width, flags, SFC_FLAG_NORMALISE_TEACHER | SFC_FLAG_TEST_STALL);
  if (rc == SFC_OK) rc = sfc::check_grad(logits, dtype, B, V, row_stride, grad_loss, grad_logits, grad_stride);
  if (rc != SFC_OK) return rc;
  if (!loss || !row_status) return SFC_EINVAL;
  const sfc::DistillParams p{logits, row_stride, V, packed_width, (flags & SFC_FLAG_NORMALISE_TEACHER) != 0,
                             temperature, teacher_ids, teacher_values, lengths, grad_loss, loss, nullptr, row_status,
                             static_cast<unsigned char*>(grad_logits), grad_stride, 1, 0, (flags & SFC_FLAG_TEST_STALL) != 0};
  return sfc::launch<true, true>(p, dtype, B, stream);
}
