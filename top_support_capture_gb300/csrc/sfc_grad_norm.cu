// The global norm of a model's gradients, and their clipping by it:
//
//   norm = sqrt(sum over all tensors of x^2),  scale = min(1, max_norm / (norm + 1e-6)),  out = x scale
//
// The tensors' addresses travel in the launch's parameters (up to kMany of them; longer lists take several launches), so
// nothing is copied to the device and a captured call holds all it needs. Each tensor is cut into chunks of 32 KB; the CTAs
// take equal runs of the list of all chunks.
//
// A batch of 32 or 16 squares is summed in 32 bits, the batches of a thread with a compensated sum in 32 bits (one 64-bit
// addition a batch took more than the memory's time: 534 M bf16 elements 396 us, so 150, 7.1 TB/s), the threads in 64. The
// CTAs' sums lie in the workspace, and whoever needs the norm adds them up in the same fixed order. A batch whose sum lies outside
// [2^-100, 2^100], where squares may overflow or lose bits, is summed in 64 bits by itself: the norm holds over the whole
// range of its elements. Roundings: 8 of a lane's chain, 2 that join the lanes, 2 of the compensated sum, in half steps of the
// sum and so half as many of the norm, and the norm's own: 7 half steps, 2^-21.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"

namespace sfc {
namespace {

constexpr int kThreads = 256, kCtas = 4 * 152, kClipCtas = 3 * 152;  // a wave of CTAs
constexpr int kInFlight = 8;                                        // 16-byte vectors of a thread
constexpr int kChunk = kInFlight * kThreads;                        // vectors
constexpr int kFew = 16, kSome = 250, kMany = 1000;                 // tensors of a launch: parameters of 0.6, 8 and 32 KB

struct Tensor {
  const void* in;
  void* out;
  int64_t count;
  int32_t first;  // the first of its chunks
  int16_t dtype, out_dtype;
};

template <int CAP>
struct Tensors {
  int32_t n, chunks;
  double* partial;      // [all launches' CTAs]
  int32_t slot, slots;  // this launch's first, their number
  float max_norm;
  float* norm;
  Tensor t[CAP];
};
static_assert(sizeof(Tensors<kMany>) <= 32764, "a launch's parameters");

// A launch may start while the one before it in the stream still runs (programmatic dependent launch): until the wait it
// touches nothing that the other writes.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// use(tensor, its chunk) for the chunks [c0, c1) of the list.
template <int CAP, class F>
__device__ __forceinline__ void each_chunk(const Tensors<CAP>& p, int c0, int c1, bool descending, F use) {
  if (c0 >= c1) return;
  int c = descending ? c1 - 1 : c0;
  int lo = 0, hi = p.n - 1;  // the last tensor whose first chunk is not behind c
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.t[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  for (int k = c0; k < c1; ++k) {
    const Tensor t = p.t[lo];
    use(t, c - t.first);
    if (descending) {
      --c;
      if (c < t.first) --lo;
    } else {
      ++c;
      if (lo + 1 < p.n && c >= p.t[lo + 1].first) ++lo;
    }
  }
}

// A batch's squares in 64 bits (out of line: batches of zeros apart, few need it).
template <int DT>
__device__ __noinline__ double exact_squares(uint4 a, uint4 b, uint4 c, uint4 d) {
  constexpr uint32_t kMagnitude = DT == 0 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
  auto bits = [](const uint4& v) { return v.x | v.y | v.z | v.w; };
  double sum = 0.0;
  if (((bits(a) | bits(b) | bits(c) | bits(d)) & kMagnitude) == 0) return sum;
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    float x[Elem<DT>::kVec];
    Elem<DT>::unpack(a, x);
#pragma unroll
    for (int i = 0; i < Elem<DT>::kVec; ++i) sum += static_cast<double>(x[i]) * x[i];
    a = b, b = c, c = d;
  }
  return sum;
}

// The squares that a thread has summed.
struct SquareAcc {
  float sum = 0.f, lost = 0.f;  // of the batches in range, compensated
  double rest = 0.0;            // of the others

  template <int DT>
  __device__ __forceinline__ void add(const uint4 (&v)[4]) {
    constexpr int N = Elem<DT>::kVec;
    uint64_t s2 = 0, t2 = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[N];
      Elem<DT>::unpack(v[u], x);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint64_t a = pack_f2(x[i], x[i + 1]), b = pack_f2(x[i + 2], x[i + 3]);
        s2 = ffma_f2(a, a, s2);
        t2 = ffma_f2(b, b, t2);
      }
    }
    float a, b;
    unpack_f2(fadd_f2(s2, t2), a, b);
    const float s = a + b;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
      const float y = s - lost, t = sum + y;
      lost = (t - sum) - y;
      sum = t;
    } else {
      rest += exact_squares<DT>(v[0], v[1], v[2], v[3]);
    }
  }
  __device__ __forceinline__ double total() const { return rest + (static_cast<double>(sum) - lost); }
};

__device__ __forceinline__ double block_total(double x, double* red) {  // in thread 0
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < kThreads / 32 ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  }
  return x;
}

// ONCE: nothing of the tensor is read or written again by the kernel.
template <int DT, bool ONCE>
__device__ __forceinline__ void square_chunk(const Tensor& t, int chunk, SquareAcc& acc) {
  const RowSpan<DT> x(t.in, 0, t.count);
  const int64_t v0 = static_cast<int64_t>(chunk) * kChunk + threadIdx.x;
  const uint4* body = x.body() + v0;
  static_assert(kInFlight == 8, "two batches");
  uint4 v[2][4];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u)
    v[u / 4][u % 4] = v0 + u * kThreads >= x.nvec ? make_uint4(0u, 0u, 0u, 0u) : ONCE ? ld_stream(body + u * kThreads) : body[u * kThreads];
  if (chunk == 0 && threadIdx.x < x.scalars()) {
    const double s = x.at(x.scalar_index(threadIdx.x));
    acc.rest += s * s;
  }
  acc.template add<DT>(v[0]);
  acc.template add<DT>(v[1]);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) grad_norm_kernel(const __grid_constant__ Tensors<CAP> p) {
  __shared__ double red[kThreads / 32];
  allow_next();
  const int64_t b = blockIdx.x;
  SquareAcc acc;
  each_chunk(p, static_cast<int>(b * p.chunks / gridDim.x), static_cast<int>((b + 1) * p.chunks / gridDim.x), false,
             [&](const Tensor& t, int chunk) {
               if (t.dtype == SFC_BF16) square_chunk<0, true>(t, chunk, acc);
               else square_chunk<1, true>(t, chunk, acc);
             });
  const double sum = block_total(acc.total(), red);
  if (threadIdx.x == 0) p.partial[p.slot + b] = sum;
}

// All CTAs' sums, by a whole CTA: the same order and bits wherever it is called. In thread 0.
__device__ __forceinline__ double total_norm(const double* partial, int slots) {
  __shared__ double red[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < slots; i += kThreads) sum += __ldcg(partial + i);
  return sqrt(block_total(sum, red));
}

__global__ void __launch_bounds__(kThreads) finish_norm_kernel(const double* partial, int slots, float* norm) {
  wait_for_last();
  const double n = total_norm(partial, slots);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

// Eight elements at once: 16 bytes of bf16, 32 of f32 in one access, so that whichever side is wider, a warp's
// instruction covers a run of memory without holes (bf16 to f32 in two stores of 16 bytes: 534 M elements 638 us).
template <class T>
struct Eight;
template <>
struct Eight<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* from) {
    // (not volatile: each address is loaded once, and stored only from what was loaded there)
    asm("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(from));
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ static void store(float* to, const float (&x)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
                 "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* from) { v = *reinterpret_cast<const uint4*>(from); }
  __device__ __forceinline__ void unpack(float (&x)[8]) const { Elem<0>::unpack(v, x); }
  __device__ __forceinline__ static void store(__nv_bfloat16* to, const float (&x)[8]) { *reinterpret_cast<uint4*>(to) = Out<0>::pack(x); }
};

__device__ __forceinline__ void put(float* to, float x) { *to = x; }
__device__ __forceinline__ void put(__nv_bfloat16* to, float x) { *to = __float2bfloat16_rn(x); }
__device__ __forceinline__ float get(const float* from) { return *from; }
__device__ __forceinline__ float get(const __nv_bfloat16* from) { return __bfloat162float(*from); }

template <class InT, class OutT>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int chunk, float scale) {
  constexpr int U = 64 / (8 * sizeof(InT));  // eights of a thread in flight: 64 bytes, half of its share
  const InT* in = static_cast<const InT*>(t.in);
  OutT* out = static_cast<OutT*>(t.out);
  const int per = static_cast<int>(16 / sizeof(InT)) * kChunk;  // elements of a chunk
  const int64_t first = static_cast<int64_t>(chunk) * per;
  // elements before the first eight whose memory is aligned on both sides; where there is none, all go one by one
  const int head = static_cast<int>((-reinterpret_cast<uintptr_t>(in) & (8 * sizeof(InT) - 1)) / sizeof(InT));
  if ((reinterpret_cast<uintptr_t>(out + head) & (8 * sizeof(OutT) - 1)) != 0) {
    const int64_t end = min(first + per, t.count);
#pragma unroll 8
    for (int64_t i = first + threadIdx.x; i < end; i += kThreads) put(out + i, get(in + i) * scale);
    return;
  }
  const int64_t eights = t.count > head ? (t.count - head) / 8 : 0;
  int64_t k0 = first / 8 + threadIdx.x;
  if (chunk == 0) {  // the scalars beside the eights
    const int64_t tail = head + eights * 8, before = min(static_cast<int64_t>(head), t.count);
    const int64_t i = threadIdx.x < before ? threadIdx.x : tail + (threadIdx.x - before);
    if (i < t.count && (threadIdx.x < before || t.count > head)) put(out + i, get(in + i) * scale);
  }
#pragma unroll 1
  for (int half = 0; half < 2; ++half, k0 += U * kThreads) {
    Eight<InT> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * kThreads < eights) v[u].load(in + head + (k0 + u * kThreads) * 8);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * kThreads >= eights) break;
      float x[8];
      v[u].unpack(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= scale;
      Eight<OutT>::store(out + head + (k0 + u * kThreads) * 8, x);
    }
  }
}

// The scale; NaN stays. One below the smallest normal number has too few bits for the ordinary numbers that huge gradients
// become: it is given as the negative of its 2^126-fold.
__device__ __forceinline__ float scale_of(double norm, float max_norm) {
  const double ratio = max_norm / (norm + 1e-6);
  const float scale = max_norm == INFINITY || ratio >= 1.0 ? 1.f : static_cast<float>(ratio);
  return scale < FLT_MIN && ratio > 0.0 ? -static_cast<float>(ratio * 0x1p126) : scale;
}

// A chunk by such a scale, element by element: the second factor is exact. (Out of line: hardly any call needs it.)
__device__ __noinline__ void scale_tiny(const void* in, void* out, int64_t first, int64_t end, bool in_bf16, bool out_bf16, float scale) {
#pragma unroll 1
  for (int64_t i = first + threadIdx.x; i < end; i += kThreads) {
    const float x = in_bf16 ? get(static_cast<const __nv_bfloat16*>(in) + i) : get(static_cast<const float*>(in) + i);
    const float y = x * scale * 0x1p-126f;
    if (out_bf16) put(static_cast<__nv_bfloat16*>(out) + i, y);
    else put(static_cast<float*>(out) + i, y);
  }
}

__device__ __forceinline__ void clip_chunk(const Tensor& t, int chunk, float scale) {
  if (scale == 1.f && t.in == t.out) return;  // in place: nothing to do
  if (scale < 0.f) {
    const int64_t per = kChunk * (t.dtype == SFC_BF16 ? 8 : 4), first = chunk * per;
    scale_tiny(t.in, t.out, first, min(first + per, t.count), t.dtype == SFC_BF16, t.out_dtype == SFC_BF16, -scale);
    return;
  }
  if (t.dtype == SFC_BF16) {
    if (t.out_dtype == SFC_BF16) scale_chunk<__nv_bfloat16, __nv_bfloat16>(t, chunk, scale);
    else scale_chunk<__nv_bfloat16, float>(t, chunk, scale);
  } else {
    if (t.out_dtype == SFC_BF16) scale_chunk<float, __nv_bfloat16>(t, chunk, scale);
    else scale_chunk<float, float>(t, chunk, scale);
  }
}

// The chunks backwards: what the norm's pass read last is still in L2. Three CTAs a SM: with four, the registers spill
// (534 M elements f32 to bf16, both calls: 785 us, with four 1046; f32 to f32 954 : 1013; bf16 to f32 669 : 671).
template <int CAP>
__global__ void __launch_bounds__(kThreads, 3) clip_kernel(const __grid_constant__ Tensors<CAP> p) {
  __shared__ float scale;
  wait_for_last();
  const double norm = total_norm(p.partial, p.slots);
  if (threadIdx.x == 0) {
    scale = scale_of(norm, p.max_norm);
    if (blockIdx.x == 0) *p.norm = static_cast<float>(norm);
  }
  __syncthreads();
  const int64_t b = blockIdx.x;
  each_chunk(p, static_cast<int>(b * p.chunks / gridDim.x), static_cast<int>((b + 1) * p.chunks / gridDim.x), true,
             [&](const Tensor& t, int chunk) { clip_chunk(t, chunk, scale); });
}

// Short lists of a megabyte at most in one launch: a cluster whose CTAs give one another their sums, and then clip the chunks
// that they have read (two tables of 64000 bf16: 5.4 us, in two launches 7.0, and 2.6 us less of the calling thread). The exchange
// is a cluster barrier, behind which every CTA knows the same: sums sent by stores that the receiver's barrier counts would save
// 0.3 us, but wait in software, and a CTA whose wait gave up would leave its chunks as they are while the others clip theirs.
constexpr int kShortCtas = 8, kShortChunks = 32;

template <bool CLIP>
__global__ void __launch_bounds__(kThreads, 2) short_kernel(const __grid_constant__ Tensors<kFew> p) {
  __shared__ double red[kThreads / 32], table[kShortCtas];
  __shared__ float scale;
  const int tid = threadIdx.x, rank = blockIdx.x;
  cluster_arrive_started();
  const int c0 = rank * p.chunks / kShortCtas, c1 = (rank + 1) * p.chunks / kShortCtas;
  SquareAcc acc;
  each_chunk(p, c0, c1, false, [&](const Tensor& t, int chunk) {
    if (t.dtype == SFC_BF16) square_chunk<0, false>(t, chunk, acc);
    else square_chunk<1, false>(t, chunk, acc);
  });
  const double sum = block_total(acc.total(), red);
  cluster_wait();
  if (tid < kShortCtas) dsmem_st64(dsmem_addr(&table[rank], tid), __double_as_longlong(sum));
  cluster_arrive_first_warp();
  cluster_wait();
  if (tid == 0) {
    double total = 0.0;
    for (int i = 0; i < kShortCtas; ++i) total += table[i];
    const double norm = sqrt(total);
    if (CLIP) scale = scale_of(norm, p.max_norm);
    if (rank == 0) *p.norm = static_cast<float>(norm);
  }
  if (!CLIP) return;
  __syncthreads();
  each_chunk(p, c0, c1, true, [&](const Tensor& t, int chunk) { clip_chunk(t, chunk, scale); });
}

struct List {
  const void* const* grads;
  const int64_t* counts;
  const int32_t* dtypes;
  int64_t n;
  void* const* out;
  const int32_t* out_dtypes;
};

int64_t chunks_of(const List& l, int64_t i) {
  const int64_t per = kChunk * (l.dtypes[i] == SFC_BF16 ? 8 : 4);
  return (l.counts[i] + per - 1) / per;
}

// The table of one launch over the tensors from i: as many as fit, those without elements left out. Returns the next.
template <int CAP>
int64_t fill(const List& l, int64_t i, Tensors<CAP>& p) {
  p.n = p.chunks = 0;
  for (; i < l.n && p.n < CAP; ++i) {
    const int64_t chunks = chunks_of(l, i);
    if (chunks == 0) continue;
    p.t[p.n++] = Tensor{l.grads[i], l.out ? l.out[i] : nullptr, l.counts[i], p.chunks, static_cast<int16_t>(l.dtypes[i]),
                        static_cast<int16_t>(l.out ? l.out_dtypes[i] : 0)};
    p.chunks += static_cast<int32_t>(chunks);
  }
  return i;
}

template <int CAP>
unsigned ctas(const Tensors<CAP>& p, int most) {
  return static_cast<unsigned>(std::min(p.chunks, most));
}

// Behind the launch before it, which it may overtake up to its wait.
template <class P, class... Args>
cudaError_t launch_behind(void (*kernel)(P, Args...), unsigned grid, cudaStream_t stream, const P& p, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, args...);
}

cudaError_t launch_short(const Tensors<kFew>& p, bool clip, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kShortCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kShortCtas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return clip ? cudaLaunchKernelEx(&cfg, short_kernel<true>, p) : cudaLaunchKernelEx(&cfg, short_kernel<false>, p);
}

template <int CAP>
cudaError_t run(const List& l, float max_norm, float* norm, double* partial, cudaStream_t stream) {
  Tensors<CAP> p;
  p.partial = partial;
  p.max_norm = max_norm;
  p.norm = norm;
  p.slots = 0;
  for (int64_t i = 0; i < l.n;) {
    i = fill(l, i, p);
    if (p.n == 0) break;
    if constexpr (CAP == kFew)  // (all of the list)
      if (p.chunks <= kShortChunks) return launch_short(p, l.out != nullptr, stream);
    p.slot = p.slots;
    p.slots += static_cast<int32_t>(ctas(p, kCtas));
    grad_norm_kernel<CAP><<<ctas(p, kCtas), kThreads, 0, stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (!l.out || p.slots == 0) return launch_behind(finish_norm_kernel, 1, stream, static_cast<const double*>(partial), p.slots, norm);
  for (int64_t i = 0; i < l.n;) {
    i = fill(l, i, p);
    if (p.n == 0) break;
    const cudaError_t err = launch_behind(clip_kernel<CAP>, ctas(p, kClipCtas), stream, p);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

constexpr int64_t kMaxTensors = 1 << 20, kMaxElements = int64_t{1} << 43;
// (f32 makes the most chunks, and each tensor may end in a partial one)
static_assert(kMaxElements / (kChunk * 4) + kMaxTensors <= INT32_MAX, "chunks are counted in 32 bits");

size_t workspace_bytes_of(int64_t n) { return static_cast<size_t>(n / kMany + 1) * kCtas * sizeof(double); }

int check_list(const List& l) {
  if (l.n < 0 || l.n > kMaxTensors || (l.n > 0 && (!l.grads || !l.counts || !l.dtypes))) return SFC_EINVAL;
  int64_t total = 0;
  for (int64_t i = 0; i < l.n; ++i) {
    const int dt = l.dtypes[i];
    if (dt != SFC_BF16 && dt != SFC_F32) return SFC_EINVAL;
    if (l.counts[i] < 0 || l.counts[i] > kMaxElements || (total += l.counts[i]) > kMaxElements) return SFC_EINVAL;
    if (l.counts[i] > 0 && (!l.grads[i] || reinterpret_cast<uintptr_t>(l.grads[i]) % (dt == SFC_BF16 ? 2 : 4))) return SFC_EINVAL;
  }
  return SFC_OK;
}

struct Range {
  uintptr_t begin, end;
  bool written;
  bool operator<(const Range& o) const { return begin < o.begin; }
};

// What is written: aligned, and no byte of it shared with anything else that is read or written (but a tensor's own place).
int check_out(const List& l) {
  if (!l.out || !l.out_dtypes) return SFC_EINVAL;
  Range* ranges = new (std::nothrow) Range[2 * l.n + 1];
  if (!ranges) return SFC_EINVAL;
  int64_t k = 0;
  int rc = SFC_OK;
  for (int64_t i = 0; i < l.n && rc == SFC_OK; ++i) {
    const int in = l.dtypes[i], to = l.out_dtypes[i];
    const uintptr_t a = reinterpret_cast<uintptr_t>(l.grads[i]), b = reinterpret_cast<uintptr_t>(l.out[i]);
    const int in_bytes = in == SFC_BF16 ? 2 : 4, out_bytes = to == SFC_BF16 ? 2 : 4;
    if (to != SFC_BF16 && to != SFC_F32) rc = SFC_EINVAL;
    if (l.counts[i] == 0) continue;
    if (b == 0 || b % out_bytes) rc = SFC_EINVAL;
    ranges[k++] = Range{b, b + l.counts[i] * out_bytes, true};
    if (a != b || in != to) ranges[k++] = Range{a, a + l.counts[i] * in_bytes, false};
  }
  std::sort(ranges, ranges + k);
  uintptr_t any = 0, written = 0;  // where what began before ends
  for (int64_t i = 0; i < k && rc == SFC_OK; ++i) {
    if (ranges[i].begin < (ranges[i].written ? any : written)) rc = SFC_EINVAL;
    any = std::max(any, ranges[i].end);
    if (ranges[i].written) written = std::max(written, ranges[i].end);
  }
  delete[] ranges;
  return rc;
}

int enqueue(const List& l, float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (!norm || reinterpret_cast<uintptr_t>(workspace) % 8) return SFC_EINVAL;
  if (!workspace || workspace_bytes < workspace_bytes_of(l.n)) return SFC_EWORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const cudaError_t err = l.n <= kFew ? run<kFew>(l, max_norm, norm, partial, st)
                          : l.n <= kSome ? run<kSome>(l, max_norm, norm, partial, st) : run<kMany>(l, max_norm, norm, partial, st);
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return SFC_ECUDA;
  }
  return SFC_OK;
}

}  // namespace
}  // namespace sfc

extern "C" size_t sfc_grad_norm_workspace_size(int64_t n) {
  return n < 0 || n > sfc::kMaxTensors ? 0 : sfc::workspace_bytes_of(n);
}

extern "C" int sfc_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int64_t n, float* norm,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const sfc::List l{grads, counts, dtypes, n, nullptr, nullptr};
  const int rc = sfc::check_list(l);
  return rc != SFC_OK ? rc : sfc::enqueue(l, 0.f, norm, workspace, workspace_bytes, stream);
}

extern "C" int sfc_clip_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int64_t n,
                                  float max_norm, void* const* out, const int32_t* out_dtypes, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const sfc::List l{grads, counts, dtypes, n, out, out_dtypes};
  if (!(max_norm >= 0.f)) return SFC_EINVAL;
  int rc = sfc::check_list(l);
  if (rc == SFC_OK && n > 0) rc = sfc::check_out(l);
  return rc != SFC_OK ? rc : sfc::enqueue(l, max_norm, norm, workspace, workspace_bytes, stream);
}
