// The norm of all gradients of a model, and their clipping:
//   N = sqrt(sum g^2) over every value of every tensor (or max |g|),
//   c = min(1, max_norm / (N + eps)),  out = c g
// A first pass leaves one partial result per workgroup, the second adds these up in every workgroup by
// itself (8 KiB from L2) and scales: two launches, no atomics, and one order of the sums whatever the
// timing. Tensors travel in the kernels' arguments, so that a call needs no table in memory.
//
// Bytes bound both passes, which read the set twice and write it once. 403 MB in bf16, traced in turn with other
// work: 98 us for the norm and 137 for the scaling (4.1 and 5.9 TB/s: some of what the first pass read last is
// still in the card's cache), 235 call after call; 51 MB, which stay in the cache: 12 and 20, 31.9 together. 1024
// workgroups of 8192 values at a time: 2048 and 4096 of them are up to 4% slower. Squares are summed in fp64:
// the result is right for every finite gradient (fp32 squares overflow from 2^64 on and vanish below 2^-75),
// and costs nothing next to the bytes.
#include <type_traits>

#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

namespace {

constexpr int kVecs = kClipChunk / (8 * kThreads);   // loads of eight values a thread and chunk

// max that keeps a NaN
__device__ __forceinline__ double nan_max(double m, double v) { return v > m || v != v ? v : m; }

__device__ __forceinline__ double join(int kind, double a, double b) {
  return kind == 0 ? a + b : nan_max(a, b);
}

// Over the workgroup, in every thread, in a fixed order.
__device__ __forceinline__ double block_join(int kind, double v, double* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = join(kind, v, __shfl_xor(v, off, 64));
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = sh[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s = join(kind, s, sh[w]);
  __syncthreads();
  return s;
}

// The tensor that a chunk belongs to.
__device__ __forceinline__ int find_tensor(const ClipArgs& a, uint32_t chunk) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One chunk through f(row of eight as loaded, first element, values left, what meanwhile() gave); meanwhile()
// runs while the chunk is on its way, and its truth value chooses between two loops.
template <bool BF16, class M, class F>
__device__ __forceinline__ void each8(const ClipTensor& t, int64_t e0, M&& meanwhile, F&& f) {
  RowRaw<BF16> x[kVecs];
  const int64_t end = t.n - e0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int64_t e = 8 * ((int64_t)u * kThreads + threadIdx.x);
    x[u] = {};
    if (e < end) x[u].load(t.g, e0 + e, (int)(end - e < 8 ? end - e : 8));
  }
  auto all = [&](auto way) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t e = 8 * ((int64_t)u * kThreads + threadIdx.x);
      if (e < end) f(x[u], e0 + e, (int)(end - e < 8 ? end - e : 8), way);
    }
  };
  if (meanwhile()) all(std::true_type{});
  else all(std::false_type{});
}

template <class F>
__device__ __forceinline__ void chunk_of(const ClipArgs& a, uint32_t chunk, F&& f) {
  const int i = __builtin_amdgcn_readfirstlane(find_tensor(a, chunk));
  f(a.t[i], (int64_t)(chunk - a.first[i]) * kClipChunk, (a.bf16[i >> 5] >> (i & 31)) & 1);
}

template <bool BF16, int KIND>
__device__ __forceinline__ double chunk_result(const ClipTensor& t, int64_t e0, double acc) {
  each8<BF16>(t, e0, [] { return false; }, [&](const RowRaw<BF16>& x, int64_t, int, auto) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = (double)x.get(i);   // zeros behind the end
      if (KIND == 0)
        acc = __builtin_fma(v, v, acc);
      else
        acc = nan_max(acc, v < 0 ? -v : v);
    }
  });
  return acc;
}

template <int KIND>
__global__ __launch_bounds__(kThreads) void qg_grad_norm(ClipArgs a) {
  __shared__ double sh[kThreads / 64];
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < a.first[a.count]; c += gridDim.x)
    chunk_of(a, c, [&](const ClipTensor& t, int64_t e0, uint32_t bf16) {
      acc = bf16 ? chunk_result<true, KIND>(t, e0, acc) : chunk_result<false, KIND>(t, e0, acc);
    });
  acc = block_join(KIND, acc, sh);
  if (threadIdx.x == 0)
    a.part[blockIdx.x] = (int)blockIdx.x < a.filled ? join(KIND, a.part[blockIdx.x], acc) : acc;
}

// The total of the partial results: the sum of squares, or the maximum.
__device__ __forceinline__ double grad_total(const ClipArgs& a, double* sh) {
  if (a.total != nullptr) return *a.total;
  constexpr int N = kClipSlots / kThreads;
  double v[N], s = 0.0;
#pragma unroll
  for (int k = 0; k < N; ++k) {   // all on their way at once
    const int i = threadIdx.x + k * kThreads;
    v[k] = i < a.slots ? a.part[i] : 0.0;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) s = join(a.kind, s, v[k]);
  return block_join(a.kind, s, sh);
}
__device__ __forceinline__ double norm_of(const ClipArgs& a, double total) {
  return a.kind == 0 ? __builtin_sqrt(total) : total;
}

__global__ __launch_bounds__(kThreads) void qg_grad_total(ClipArgs a) {
  __shared__ double sh[kThreads / 64];
  const double total = grad_total(a, sh);
  if (threadIdx.x != 0) return;
  if (a.norm_out != nullptr) *a.norm_out = (float)norm_of(a, total);
  if (a.total_out != nullptr) *a.total_out = total;
}

// What the gradients are multiplied by: c, or q itself where c would be subnormal or vanish (a norm from 2^126
// max_norm on), whose products may yet be of any size.
struct Factor {
  float c;
  double q;
  bool known, zero, tiny;
};

template <bool BF16, class M>
__device__ __forceinline__ void chunk_scale(const ClipTensor& t, int64_t e0, const Factor& by,
                                            M&& meanwhile) {
  each8<BF16>(t, e0, meanwhile, [&](const RowRaw<BF16>& x, int64_t e, int left, auto tiny) {
    if (by.c == 1.0f && !by.zero && t.out == t.g) return;   // its values stay
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = by.zero ? 0.0f : decltype(tiny)::value ? (float)((double)x.get(i) * by.q) : x.get(i) * by.c;
    row_store<BF16>(t.out, e, left, v);
  });
}

// The factor is formed while the first chunk is on its way. Chunks go from the end on: what the first pass
// read last may still lie in the card's cache.
__global__ __launch_bounds__(kThreads) void qg_grad_scale(ClipArgs a) {
  __shared__ double sh[kThreads / 64];
  Factor by = {0.0f, 0.0, false, false, false};
  auto form = [&] {
    if (by.known) return by.tiny;   // the same for the whole workgroup
    const double norm = norm_of(a, grad_total(a, sh));
    if (a.norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm_out = (float)norm;
    const double q = (double)a.max_norm / (norm + (double)a.eps);
    // a norm of zero leaves zeros as they are, also with max_norm = eps = 0
    by.c = norm == 0.0 || q >= 1.0 ? 1.0f : (float)q;
    by.q = q;
    by.tiny = norm != 0.0 && q < 0x1p-126;
    by.zero = a.zero && !(norm <= 1.7976931348623157e308);
    by.known = true;
    return by.tiny;
  };
  const uint32_t chunks = a.first[a.count];
  if (chunks == 0) form();   // the norm alone
  for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    if (by.known && by.c == 1.0f && !by.zero && a.in_place) return;
    chunk_of(a, chunks - 1 - k, [&](const ClipTensor& t, int64_t e0, uint32_t bf16) {
      if (bf16)
        chunk_scale<true>(t, e0, by, form);
      else
        chunk_scale<false>(t, e0, by, form);
    });
  }
}

}  // namespace

hipError_t launch_grad_norm(const ClipArgs& a, hipStream_t s) {
  if (a.kind == 0)
    hipLaunchKernelGGL(qg_grad_norm<0>, dim3(clip_grid(a.first[a.count])), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(qg_grad_norm<1>, dim3(clip_grid(a.first[a.count])), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_grad_total(const ClipArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(qg_grad_total, dim3(1), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_grad_scale(const ClipArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(qg_grad_scale, dim3(clip_grid(a.first[a.count])), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace qg
