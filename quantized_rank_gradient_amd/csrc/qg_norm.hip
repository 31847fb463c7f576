// Layer norm over the last dimension of x (T x n), and with center = 0 the norm by the root mean
// square:
//   h = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),  y = gamma h + beta
//   dh = gamma dy,  dx = rstd (dh - mean(dh) - h mean(dh h)),  dgamma = sum_t dy h,
//   dbeta = sum_t dy
// (center = 0: mean = 0 in h and no mean(dh) in dx). The bytes bound both passes, but for rows of a
// few hundred values (a wave takes one whole: 262144 x 128 in bf16, 62 us forward and 88 backward, 40%
// of the bytes' rate) and the backward pass of rows beyond 16384.
#include <type_traits>

#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

// R rows of the input at a time, W waves to a row, C chunks of eight values a thread
// (n <= 512 W C): a row is read once and held in registers until its one write; the variance is
// that of the centred values, so a large mean costs no digits. 8192 x 4096 in bf16: 29 us, 134 MB at
// 4.6 TB/s.
template <bool BF16, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_norm_fwd(NormArgs a) {
  __shared__ float2 sh[2][W * R];
  const int n = (int)a.n, first = (int)(threadIdx.x / (64 * W)) * W;
  const int tid = (int)threadIdx.x - 64 * first;
  const float rn = 1.0f / (float)n;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + first / W;
    const int cols = row < a.T ? n : 0;
    const int64_t base = row * a.n;
    RowRaw<BF16> x[C];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      if (j < cols) {
        x[c].load(a.x, base + j, cols - j);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[c].get(i);
      }
    }
    const float mean = a.center ? row_sum2<W>(s, 0.0f, sh[0], first).x * rn : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < cols) {
          const float d = x[c].get(i) - mean;
          q += d * d;
        }
    }
    const float rstd = 1.0f / sqrt_rn(row_sum2<W>(q, 0.0f, sh[1], first).x * rn + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      if (j >= cols) continue;
      RowRaw<false> g, b;
      float y[8];
      g.load(a.gamma, j, cols - j);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (x[c].get(i) - mean) * rstd * g.get(i);
      if (a.beta != nullptr) {
        b.load(a.beta, j, cols - j);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += b.get(i);
      }
      row_store<BF16>(a.y, base + j, cols - j, y);
    }
    if (tid == 0 && cols > 0) {
      if (a.mean_out != nullptr) a.mean_out[row] = mean;
      a.rstd_out[row] = rstd;
    }
    if (W > 1 && !a.center) __syncthreads();   // sh[1] is free again before the next row's sum
  }
}

// Rows R blockIdx.x .., + R gridDim.x, ...: dx of each, and the sums of dy h and dy over them in
// registers, joined over the R rows in LDS at the end and written as one row of partial sums. With
// one chunk a thread the next row's values are on their way while a row is summed and written;
// longer rows have no registers for that (1024 threads: 128 each), and rows beyond 16384 spill: 71 of
// them in bf16 and 76 in fp32, 276 and 292 bytes a lane. 8192 x 4096 in bf16: 37 us, 201 MB at 5.4
// TB/s, and 4 us for the sums of the 256 rows; 2048 rows of 16384: 53 us a call, of 32768: 311.
template <bool BF16, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_norm_bwd(NormArgs a) {
  constexpr bool AHEAD = C == 1;
  constexpr int N = 512 * W * C;   // columns held
  __shared__ float2 sh[2][W * R];
  __shared__ float join[R > 1 ? N : 1];
  const int n = (int)a.n, first = (int)(threadIdx.x / (64 * W)) * W;
  const int tid = (int)threadIdx.x - 64 * first;
  const float rn = 1.0f / (float)n;
  float dg[C][8], db[C][8];
  RowRaw<false> gam{};
  if (AHEAD && 8 * tid < n) gam.load(a.gamma, 8 * tid, n - 8 * tid);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[c][i] = db[c][i] = 0.0f;
  RowRaw<BF16> x[C], d[C];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      x[c] = {};
      d[c] = {};
      if (row < a.T && j < n) {
        x[c].load(a.x, row * a.n + j, n - j);
        d[c].load(a.dy, row * a.n + j, n - j);
      }
    }
    mean = a.center && row < a.T ? a.mean_in[row] : 0.0f;
    rstd = row < a.T ? a.rstd_in[row] : 0.0f;
  };
  auto gamma = [&](int c) {
    if (AHEAD) return gam;
    RowRaw<false> g{};
    const int j = 8 * (tid + 64 * W * c);
    if (j < n) g.load(a.gamma, j, n - j);
    return g;
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R + first / W;
  if (AHEAD) fetch(row);
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += step, row += step) {
    if (!AHEAD) fetch(row);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      const RowRaw<false> g = gamma(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // behind the row's end x is 0 and h would be -mean rstd
        const float h = j + i < n ? (x[c].get(i) - mean) * rstd : 0.0f;
        const float di = d[c].get(i), dh = di * g.get(i);
        s1 += dh;
        s2 += dh * h;
        dg[c][i] += di * h;
        db[c][i] += di;
      }
    }
    RowRaw<BF16> xc[C], dc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      xc[c] = x[c];
      dc[c] = d[c];
    }
    const float mc = mean, rc = rstd;
    if (AHEAD) fetch(row + step);
    const float2 s = row_sum2<W>(s1, s2, sh[par], first);
    par ^= 1;
    const float m1 = a.center ? s.x * rn : 0.0f, m2 = s.y * rn;
    if (row < a.T) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = 8 * (tid + 64 * W * c);
        if (j >= n) continue;
        const RowRaw<false> g = gamma(c);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = rc * (dc[c].get(i) * g.get(i) - m1 - (xc[c].get(i) - mc) * rc * m2);
        row_store<BF16>(a.dx, row * a.n + j, n - j, o);
      }
    }
  }
  auto put = [&](float (&v)[C][8], float* part) {
    if (R > 1) {   // one row after another, in order
      for (int r = 0; r < R; ++r) {
        __syncthreads();
        if (first / W == r) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* q = join + 8 * (tid + 64 * W * c) + i;
              if (r > 0) v[c][i] += *q;
              *q = v[c][i];
            }
        }
      }
      if (first / W != R - 1) return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      if (j < n) row_store<false>(part, (int64_t)blockIdx.x * a.n + j, n - j, v[c]);
    }
  };
  put(dg, a.part);
  if (a.part_b != nullptr) put(db, a.part_b);
}

namespace {

// f(W, C, R) as integral constants for rows of n <= kNormMaxN: the fewest waves that hold a row at
// one chunk a thread (the longest: two or four), and as many rows side by side as fill a
// workgroup.
template <class F>
void with_row(int64_t n, F&& f) {
  using std::integral_constant;
  auto go = [&](auto w, auto c) {
    constexpr int W = decltype(w)::value;
    f(w, c, integral_constant<int, (W == 1 ? 8 : 16 / W)>{});
  };
  if (n <= 512) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (n <= 1024) go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  else if (n <= 2048) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (n <= 4096) go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (n <= 8192) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (n <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

}  // namespace

// Rows side by side in a workgroup of the backward pass, for the host's grid.
int norm_rows(int64_t n) {
  int rows = 0;
  with_row(n, [&](auto, auto, auto r) { rows = decltype(r)::value; });
  return rows;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  with_row(a.n, [&](auto w, auto c, auto) {
    // a workgroup for each row of more than a wave; four rows of a wave
    constexpr int W = decltype(w)::value, C = decltype(c)::value, R = W == 1 ? 4 : 1;
    const int64_t groups = (a.T + R - 1) / R;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
    if (a.bf16)
      hipLaunchKernelGGL((qg_norm_fwd<true, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
    else
      hipLaunchKernelGGL((qg_norm_fwd<false, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
  });
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  with_row(a.n, [&](auto w, auto c, auto r) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, R = decltype(r)::value;
    const dim3 grid((unsigned)a.slabs);
    if (a.bf16)
      hipLaunchKernelGGL((qg_norm_bwd<true, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
    else
      hipLaunchKernelGGL((qg_norm_bwd<false, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
  });
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || a.slabs == 1
             ? e
             : launch_col_sum(a.part, a.dgamma, a.part_b, a.dbeta, a.slabs, a.n, s);
}

}  // namespace qg
