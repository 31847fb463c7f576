// Layer norm over the last dimension of x (T x n), and with center = 0 the norm by the root mean
// square:
//   h = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),  y = gamma h + beta
//   dh = gamma dy,  dx = rstd (dh - mean(dh) - h mean(dh h)),  dgamma = sum_t dy h,
//   dbeta = sum_t dy
// (center = 0: mean = 0 in h and no mean(dh) in dx). The bytes bound both passes.
#include "qg_kernels.hpp"

namespace qg {

constexpr int kNormChunk = 8;   // consecutive elements a thread takes at a time

// Eight elements from e on as fp32; elements at or past `left` are zero.
template <bool BF16>
__device__ __forceinline__ void norm_load(const void* p, int64_t e, int left, bool vec,
                                          float (&v)[8]) {
  if (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + e;
    if (vec && left >= 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(q);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_to_f32(q[i]) : 0.0f;
    }
  } else {
    const float* q = static_cast<const float*>(p) + e;
    if (vec && left >= 8) {
      const float4 a = *reinterpret_cast<const float4*>(q);
      const float4 b = *reinterpret_cast<const float4*>(q + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? q[i] : 0.0f;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void norm_store(void* p, int64_t e, int left, bool vec,
                                           const float (&v)[8]) {
  if (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + e;
    if (vec && left >= 8) {
      *reinterpret_cast<uint4*>(q) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = to_bf16(v[i]);
    }
  } else {
    float* q = static_cast<float*>(p) + e;
    if (vec && left >= 8) {
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = v[i];
    }
  }
}

// Sums of two values over the workgroup's threads.
template <int NW>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
  if (NW == 1) return make_float2(a, b);
  __syncthreads();   // the area's last use
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    s.x += sh[w].x;
    s.y += sh[w].y;
  }
  return s;
}

// A row at a time, held in registers (C chunks a thread, n <= 512 NW C) between its one read and its
// one write: the variance is that of the centred values, so a large mean costs no digits.
template <bool BF16, int NW, int C>
__global__ __launch_bounds__(64 * NW) void qg_norm_fwd(NormArgs a) {
  __shared__ float2 sh[NW];
  const int n = (int)a.n, step = 64 * NW * kNormChunk;
  const bool vec = n % 8 == 0;
  const float rn = 1.0f / (float)n;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t base = row * a.n;
    float v[C][8];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * step + (int)threadIdx.x * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
      if (j < n) norm_load<BF16>(a.x, base + j, n - j, vec, v[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[c][i];
    }
    const float mean = a.center ? group_sum2<NW>(s, 0.0f, sh).x * rn : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * step + (int)threadIdx.x * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] -= mean;
        if (j + i < n) q += v[c][i] * v[c][i];
      }
    }
    const float rstd = 1.0f / sqrt_rn(group_sum2<NW>(q, 0.0f, sh).x * rn + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * step + (int)threadIdx.x * 8;
      if (j >= n) continue;
      float g[8], b[8], y[8];
      norm_load<false>(a.gamma, j, n - j, vec, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[c][i] * rstd * g[i];
      if (a.beta != nullptr) {
        norm_load<false>(a.beta, j, n - j, vec, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += b[i];
      }
      norm_store<BF16>(a.y, base + j, n - j, vec, y);
    }
    if (threadIdx.x == 0) {
      if (a.mean_out != nullptr) a.mean_out[row] = mean;
      a.rstd_out[row] = rstd;
    }
  }
}

// Rows blockIdx.x, + gridDim.x, ...: dx of each, and this workgroup's sums of dy h and dy in
// registers (C chunks a thread), written as one row of partial sums. n <= 64 NW * 8 * C.
template <bool BF16, int NW, int C>
__global__ __launch_bounds__(64 * NW) void qg_norm_bwd(NormArgs a) {
  __shared__ float2 sh[NW];
  const int n = (int)a.n, step = 64 * NW * kNormChunk;
  const bool vec = n % 8 == 0;
  const float rn = 1.0f / (float)n;
  float dg[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[c][i] = db[c][i] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t base = row * a.n;
    const float mean = a.center ? a.mean_in[row] : 0.0f, rstd = a.rstd_in[row];
    float h[C][8], dh[C][8], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * step + (int)threadIdx.x * 8;
      float x[8], d[8], g[8];
      if (j < n) {
        norm_load<BF16>(a.x, base + j, n - j, vec, x);
        norm_load<BF16>(a.dy, base + j, n - j, vec, d);
        norm_load<false>(a.gamma, j, n - j, vec, g);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = j + i < n;
        h[c][i] = in ? (x[i] - mean) * rstd : 0.0f;
        const float di = in ? d[i] : 0.0f;
        dh[c][i] = in ? di * g[i] : 0.0f;
        s1 += dh[c][i];
        s2 += dh[c][i] * h[c][i];
        dg[c][i] += di * h[c][i];
        db[c][i] += di;
      }
    }
    const float2 s = group_sum2<NW>(s1, s2, sh);
    const float m1 = a.center ? s.x * rn : 0.0f, m2 = s.y * rn;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * step + (int)threadIdx.x * 8;
      if (j >= n) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (dh[c][i] - m1 - h[c][i] * m2);
      norm_store<BF16>(a.dx, base + j, n - j, vec, o);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = c * step + (int)threadIdx.x * 8;
    if (j >= n) continue;
    norm_store<false>(a.part, (int64_t)blockIdx.x * a.n + j, n - j, vec, dg[c]);
    if (a.part_b != nullptr)
      norm_store<false>(a.part_b, (int64_t)blockIdx.x * a.n + j, n - j, vec, db[c]);
  }
}

namespace {

// f(NW, C) as integral constants for rows of n <= kNormMaxN: the fewest waves that hold a row in at
// most two chunks a thread, and four chunks for the longest.
template <class F>
void with_row(int64_t n, F&& f) {
  using std::integral_constant;
  if (n <= 512) f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (n <= 1024) f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (n <= 2048) f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (n <= 4096) f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else if (n <= 8192) f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  else if (n <= 16384) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.T < (1 << 20) ? a.T : (1 << 20));
  with_row(a.n, [&](auto nw, auto c) {
    constexpr int NW = decltype(nw)::value, C = decltype(c)::value;
    if (a.bf16)
      hipLaunchKernelGGL((qg_norm_fwd<true, NW, C>), dim3(grid), dim3(64 * NW), 0, s, a);
    else
      hipLaunchKernelGGL((qg_norm_fwd<false, NW, C>), dim3(grid), dim3(64 * NW), 0, s, a);
  });
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  with_row(a.n, [&](auto nw, auto c) {
    constexpr int NW = decltype(nw)::value, C = decltype(c)::value;
    if (a.bf16)
      hipLaunchKernelGGL((qg_norm_bwd<true, NW, C>), dim3((unsigned)a.slabs), dim3(64 * NW), 0, s,
                         a);
    else
      hipLaunchKernelGGL((qg_norm_bwd<false, NW, C>), dim3((unsigned)a.slabs), dim3(64 * NW), 0, s,
                         a);
  });
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_col_sum(a.part, a.slabs, a.n, a.dgamma, s);
  if (e == hipSuccess && a.part_b != nullptr)
    e = launch_col_sum(a.part_b, a.slabs, a.n, a.dbeta, s);
  return e;
}

}  // namespace qg
