// The global norm of a model's gradients, and their clipping by it:
//
//   norm = sqrt(sum over all tensors of x^2),  scale = min(1, max_norm / (norm + 1e-6)),  out = x scale
//
// The tensors' addresses travel in the launch's parameters (up to kMany of them; longer lists take several launches), so
// nothing is copied to the device and a captured call holds all it needs. Each tensor is cut into chunks of kChunk 16-byte
// vectors; the CTAs take equal runs of the list of all chunks.
//
// A batch of 16 to 32 squares is summed in 32 bits and added to a 64-bit sum of its thread; the CTAs' sums lie in the
// workspace, and whoever needs the norm adds them up in the same fixed order. A batch whose 32-bit sum overflowed, or lies
// so low that squares were flushed, is summed again in 64 bits: the norm holds over the whole range of its elements.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>

#include "../../include/sfc.h"
#include "sfc_rows.cuh"

namespace sfc {
namespace {

constexpr int kThreads = 512, kCtas = 4 * 152;  // a wave of CTAs
constexpr int kChunk = 4 * kThreads;            // vectors: four loads in flight per thread
constexpr int kFew = 16, kMany = 1000;          // tensors of a launch: parameters of 0.6 KB, of 32 KB

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

// The part of a chunk in its tensor: vectors [v0, v1) of the tensor's body; the first chunk has the scalars beside it too.
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

// The sum of a batch's squares.
template <int DT, int U>
__device__ __forceinline__ double squares(const uint4 (&v)[U]) {
  constexpr int N = Elem<DT>::kVec;
  uint64_t s2 = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[N];
    Elem<DT>::unpack(v[u], x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t x2 = pack_f2(x[i], x[i + 1]);
      s2 = ffma_f2(x2, x2, s2);
    }
  }
  float a, b;
  unpack_f2(s2, a, b);
  const float s = a + b;
  if (s >= 0x1p-120f && s < INFINITY) return s;
  // overflow, NaN, or nothing but numbers below 2^-60, whose squares lose bits or are 0
  uint32_t any = 0;
  constexpr uint32_t kMagnitude = DT == 0 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
#pragma unroll
  for (int u = 0; u < U; ++u) any |= (v[u].x | v[u].y | v[u].z | v[u].w) & kMagnitude;
  double d = 0.0;
  if (any == 0) return d;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[N];
    Elem<DT>::unpack(v[u], x);
#pragma unroll
    for (int i = 0; i < N; ++i) d += static_cast<double>(x[i]) * x[i];
  }
  return d;
}

__device__ __forceinline__ double block_total(double x, double* red) {  // in thread 0
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  }
  return x;
}

template <int DT>
__device__ __forceinline__ void square_chunk(const Tensor& t, int chunk, double& sum) {
  const RowSpan<DT> x(t.in, 0, t.count);
  const int64_t v0 = static_cast<int64_t>(chunk) * kChunk + threadIdx.x;
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = v0 + u * kThreads < x.nvec ? ld_stream(x.body() + v0 + u * kThreads) : make_uint4(0u, 0u, 0u, 0u);
  if (chunk == 0 && threadIdx.x < x.scalars()) {
    const double s = x.at(x.scalar_index(threadIdx.x));
    sum += s * s;
  }
  sum += squares<DT>(v);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) grad_norm_kernel(const __grid_constant__ Tensors<CAP> p) {
  __shared__ double red[kThreads / 32];
  const int64_t b = blockIdx.x;
  double sum = 0.0;
  each_chunk(p, static_cast<int>(b * p.chunks / gridDim.x), static_cast<int>((b + 1) * p.chunks / gridDim.x), false,
             [&](const Tensor& t, int chunk) {
               if (t.dtype == SFC_BF16) square_chunk<0>(t, chunk, sum);
               else square_chunk<1>(t, chunk, sum);
             });
  sum = block_total(sum, red);
  if (threadIdx.x == 0) p.partial[p.slot + b] = sum;
}

// All CTAs' sums, by a whole CTA: the same order and bits wherever it is called.
__device__ __forceinline__ double total_norm(const double* partial, int slots) {
  __shared__ double red[kThreads / 32];
  __shared__ double norm;
  double sum = 0.0;
  for (int i = threadIdx.x; i < slots; i += kThreads) sum += __ldcg(partial + i);
  sum = block_total(sum, red);
  if (threadIdx.x == 0) norm = sqrt(sum);
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(kThreads) finish_norm_kernel(const double* partial, int slots, float* norm) {
  const double n = total_norm(partial, slots);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

template <int N>
__device__ __forceinline__ void store_elements(float* to, const float (&x)[N]) {
  if (reinterpret_cast<uintptr_t>(to) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) __stcs(reinterpret_cast<float4*>(to + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = x[i];
  }
}
template <int N>
__device__ __forceinline__ void store_elements(__nv_bfloat16* to, const float (&x)[N]) {
  if (reinterpret_cast<uintptr_t>(to) % (2 * N) == 0) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (N == 8) __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
    else __stcs(reinterpret_cast<uint2*>(to), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = __float2bfloat16_rn(x[i]);
  }
}

template <int DT, class OutT>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int chunk, float scale) {
  constexpr int N = Elem<DT>::kVec;
  const RowSpan<DT> x(t.in, 0, t.count);
  OutT* out = static_cast<OutT*>(t.out);
  const int64_t v0 = static_cast<int64_t>(chunk) * kChunk + threadIdx.x;
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (v0 + u * kThreads < x.nvec) v[u] = x.body()[v0 + u * kThreads];
  if (chunk == 0 && threadIdx.x < x.scalars()) {
    const int64_t i = x.scalar_index(threadIdx.x);
    const float y[1] = {x.at(i) * scale};
    if constexpr (sizeof(OutT) == 4) out[i] = y[0];
    else out[i] = __float2bfloat16_rn(y[0]);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t k = v0 + u * kThreads;
    if (k >= x.nvec) break;
    float y[N];
    Elem<DT>::unpack(v[u], y);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] *= scale;
    store_elements<N>(out + x.head + k * N, y);
  }
}

// The same runs of chunks backwards: what the norm's pass read last is still in L2.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 2) clip_kernel(const __grid_constant__ Tensors<CAP> p) {
  const double norm = total_norm(p.partial, p.slots);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = static_cast<float>(norm);
  const double ratio = p.max_norm / (norm + 1e-6);
  const float scale = p.max_norm == INFINITY || ratio >= 1.0 ? 1.f : static_cast<float>(ratio);  // NaN stays
  const int64_t b = blockIdx.x;
  each_chunk(p, static_cast<int>(b * p.chunks / gridDim.x), static_cast<int>((b + 1) * p.chunks / gridDim.x), true,
             [&](const Tensor& t, int chunk) {
               if (scale == 1.f && t.in == t.out) return;  // in place: nothing to do
               if (t.dtype == SFC_BF16) {
                 if (t.out_dtype == SFC_BF16) scale_chunk<0, __nv_bfloat16>(t, chunk, scale);
                 else scale_chunk<0, float>(t, chunk, scale);
               } else {
                 if (t.out_dtype == SFC_BF16) scale_chunk<1, __nv_bfloat16>(t, chunk, scale);
                 else scale_chunk<1, float>(t, chunk, scale);
               }
             });
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
  const int64_t vectors = l.counts[i] / (l.dtypes[i] == SFC_BF16 ? 8 : 4);  // not fewer than its body has
  return l.counts[i] > 0 ? std::max<int64_t>(1, (vectors + kChunk - 1) / kChunk) : 0;
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
unsigned ctas(const Tensors<CAP>& p) {
  return static_cast<unsigned>(std::min(p.chunks, kCtas));
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
    p.slot = p.slots;
    p.slots += static_cast<int32_t>(ctas(p));
    grad_norm_kernel<CAP><<<ctas(p), kThreads, 0, stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (!l.out || p.slots == 0) {
    finish_norm_kernel<<<1, kThreads, 0, stream>>>(partial, p.slots, norm);
    return cudaGetLastError();
  }
  for (int64_t i = 0; i < l.n;) {
    i = fill(l, i, p);
    if (p.n == 0) break;
    clip_kernel<CAP><<<ctas(p), kThreads, 0, stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

constexpr int64_t kMaxTensors = 1 << 20, kMaxElements = int64_t{1} << 44;  // chunks are counted in 32 bits

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
  if ((l.n <= kFew ? run<kFew>(l, max_norm, norm, partial, st) : run<kMany>(l, max_norm, norm, partial, st)) != cudaSuccess) {
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
