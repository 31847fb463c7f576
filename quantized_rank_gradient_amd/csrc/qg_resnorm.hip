// The norms behind a block and before the next one, with the block's gate and scales (T tokens of n):
//   p = gamma1 (u - mean1) rstd1 + beta1,  h = alpha x + rho a(z) p,  y = gamma2 (h - mean2) rstd2 + beta2
// and the gradients of all of it. Each pass reads every tensor once and writes each result once; a token's
// row stays in registers from its loads to its stores, through both norms. Bytes bound both passes.
#include <type_traits>

#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

namespace {

// a(z) and a'(z), each from exp of a number that is not positive: no overflow, and the derivatives keep
// their digits in both tails.
struct Gate {
  float a, d;
};
__device__ __forceinline__ Gate gate_of(int act, float z) {
  if (act == kGateIdentity) return {z, 1.0f};
  const float m = act == kGateTanh ? 2.0f : 1.0f;
  const float e = expf(-m * fabsf(z)), r = 1.0f / (1.0f + e);
  if (act == kGateTanh) return {tanhf(z), 4.0f * (e * r * r)};
  return {z >= 0.0f ? r : z < 0.0f ? e * r : z, e * r * r};
}

template <bool BF16>
__device__ __forceinline__ RowRaw<BF16> row_at(const void* p, int64_t row, int n, int j, bool on) {
  RowRaw<BF16> v{};
  if (on && p != nullptr && j < n) v.load(p, row * n + j, n - j);
  return v;
}

}  // namespace

// R tokens at a time, W waves to a row, C chunks of eight values a thread.
template <bool BF16, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_resnorm_fwd(ResArgs a) {
  __shared__ float2 sh[4][W * R];
  const int n = (int)a.n, first = (int)(threadIdx.x / (64 * W)) * W;
  const int tid = (int)threadIdx.x - 64 * first;
  const float rn = 1.0f / (float)n;
  auto col = [&](int c) { return 8 * (tid + 64 * W * c); };
  // mean and rstd of the row's values v(c, i), by the centred values
  auto stats = [&](auto&& v, float2* s0, float2* s1) {
    float mean = 0.0f;
    if (a.center) {
      float s = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v(c, i);   // zeros behind the row's end
      mean = row_sum2<W>(s, 0.0f, s0, first).x * rn;
    }
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col(c) + i < n) {
          const float d = v(c, i) - mean;
          q += d * d;
        }
    return make_float2(mean, 1.0f / sqrt_rn(row_sum2<W>(q, 0.0f, s1, first).x * rn + a.eps));
  };
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + first / W;
    const bool on = row < a.T;
    RowRaw<BF16> u[C], x[C], z[C];
    const int64_t zrow = a.z != nullptr ? (a.per == 1 ? row : row / a.per) : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      u[c] = row_at<BF16>(a.u, row, n, col(c), on);
      x[c] = row_at<BF16>(a.x, row, n, col(c), on);
      z[c] = row_at<BF16>(a.z, zrow, n, col(c), on);
    }
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    if (a.g1 != nullptr)
      s1 = stats([&](int c, int i) { return u[c].get(i); }, sh[0], sh[1]);
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const RowRaw<false> g1 = row_at<false>(a.g1, 0, n, col(c), on);
      const RowRaw<false> b1 = row_at<false>(a.b1, 0, n, col(c), on);
      const RowRaw<false> rho = row_at<false>(a.rho, 0, n, col(c), on);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float p = u[c].get(i);
        if (a.g1 != nullptr) p = (p - s1.x) * s1.y * g1.get(i) + b1.get(i);
        if (a.z != nullptr) p *= gate_of(a.act, z[c].get(i)).a;
        if (a.rho != nullptr) p *= rho.get(i);
        h[c][i] = col(c) + i < n ? a.alpha * x[c].get(i) + p : 0.0f;
      }
    }
    if (a.g2 != nullptr) s2 = stats([&](int c, int i) { return h[c][i]; }, sh[2], sh[3]);
    if (on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = col(c);
        if (j >= n) continue;
        row_store<BF16>(a.h, row * n + j, n - j, h[c]);
        if (a.g2 == nullptr) continue;
        const RowRaw<false> g2 = row_at<false>(a.g2, 0, n, j, true);
        const RowRaw<false> b2 = row_at<false>(a.b2, 0, n, j, true);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (h[c][i] - s2.x) * s2.y * g2.get(i) + b2.get(i);
        row_store<BF16>(a.y, row * n + j, n - j, y);
      }
      if (tid == 0) {
        a.stats_out[row] = s1.x;
        a.stats_out[a.T + row] = s1.y;
        a.stats_out[2 * a.T + row] = s2.x;
        a.stats_out[3 * a.T + row] = s2.y;
      }
    }
    if (W > 1) __syncthreads();   // the areas of sums are free again before the next row's
  }
}

// Strand by strand, token by token: the gradients that belong to the token are written, those of the
// parameters are summed in registers, and the gate's over a group, too.
template <bool BF16, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_resnorm_bwd(ResArgs a) {
  constexpr int N = 512 * W * C;   // columns held
  __shared__ float2 sh[2][W * R];
  __shared__ float join[R > 1 ? N : 1];
  const int n = (int)a.n, first = (int)(threadIdx.x / (64 * W)) * W;
  const int tid = (int)threadIdx.x - 64 * first;
  const float rn = 1.0f / (float)n;
  auto col = [&](int c) { return 8 * (tid + 64 * W * c); };
  const bool norm1 = a.g1 != nullptr, norm2 = a.g2 != nullptr;
  // this strand's tokens
  const int64_t q = (int64_t)blockIdx.x * R + first / W;
  int64_t lo, hi;
  if (a.split.parts > 1) {
    const int64_t g = q / a.split.parts;
    lo = g * a.per + (q - g * a.split.parts) * a.split.len;
    hi = lo + a.split.len < (g + 1) * a.per ? lo + a.split.len : (g + 1) * a.per;
  } else {
    lo = q * a.split.len;
    hi = lo + a.split.len;
  }
  if (q >= a.split.strands || lo >= a.T) hi = lo = 0;
  if (hi > a.T) hi = a.T;
  int64_t group = a.z != nullptr && hi > lo ? lo / a.per : 0;
  int64_t left = (group + 1) * a.per - lo;   // tokens to the group's end

  float acc[kResSums][C][8], zacc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int k = 0; k < kResSums; ++k) acc[k][c][i] = 0.0f;
      zacc[c][i] = 0.0f;
    }
  for (int64_t it = 0; it < a.split.len; ++it) {
    const int64_t row = lo + it;
    const bool on = row < hi;
    RowRaw<BF16> dh[C], dy[C], h[C], u[C], z[C];
    float m1 = 0.0f, r1 = 0.0f, m2 = 0.0f, r2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      dh[c] = row_at<BF16>(a.dh, row, n, col(c), on);
      u[c] = row_at<BF16>(a.u, row, n, col(c), on);
      dy[c] = row_at<BF16>(norm2 ? a.dy : nullptr, row, n, col(c), on);
      h[c] = row_at<BF16>(norm2 ? a.h_in : nullptr, row, n, col(c), on);
      z[c] = row_at<BF16>(a.z, group, n, col(c), on);
    }
    if (on) {
      m1 = a.center ? a.stats[row] : 0.0f;
      r1 = a.stats[a.T + row];
      m2 = a.center ? a.stats[2 * a.T + row] : 0.0f;
      r2 = a.stats[3 * a.T + row];
    }
    float D[C][8];
    if (norm2) {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const RowRaw<false> g2 = row_at<false>(a.g2, 0, n, col(c), true);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hh = col(c) + i < n ? (h[c].get(i) - m2) * r2 : 0.0f;
          const float d = dy[c].get(i), e = d * g2.get(i);
          s1 += e;
          s2 += e * hh;
          acc[kResG2][c][i] += d * hh;
          acc[kResB2][c][i] += d;
        }
      }
      const float2 s = row_sum2<W>(s1, s2, sh[0], first);
      const float k1 = a.center ? s.x * rn : 0.0f, k2 = s.y * rn;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const RowRaw<false> g2 = row_at<false>(a.g2, 0, n, col(c), true);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          D[c][i] = dh[c].get(i) +
                    r2 * (dy[c].get(i) * g2.get(i) - k1 - (h[c].get(i) - m2) * r2 * k2);
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) D[c][i] = dh[c].get(i);
    }
    const bool ends = left == 1 || row + 1 == hi;   // of the group, in this strand
    float s3 = 0.0f, s4 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = col(c);
      const RowRaw<false> g1 = row_at<false>(a.g1, 0, n, j, true);
      const RowRaw<false> b1 = row_at<false>(a.b1, 0, n, j, norm1);
      const RowRaw<false> rho = row_at<false>(a.rho, 0, n, j, true);
      float o[8], dz[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = j + i < n ? D[c][i] : 0.0f;
        o[i] = a.alpha * d;
        const float uh = norm1 ? (u[c].get(i) - m1) * r1 : u[c].get(i);
        const float p = norm1 ? uh * g1.get(i) + b1.get(i) : uh;
        Gate g = {1.0f, 0.0f};
        if (a.z != nullptr) g = gate_of(a.act, z[c].get(i));
        const float w = a.rho != nullptr ? rho.get(i) : 1.0f, t = d * p;
        acc[kResRho][c][i] += t * g.a;
        zacc[c][i] += t * w;
        dz[i] = zacc[c][i] * g.d;
        const float v = d * w * g.a;   // behind the row's end 0
        acc[kResG1][c][i] += v * uh;
        acc[kResB1][c][i] += v;
        const float f = norm1 ? v * g1.get(i) : v;
        s3 += f;
        s4 += f * uh;
        D[c][i] = f;
      }
      if (!on || j >= n) continue;
      row_store<BF16>(a.dx, row * n + j, n - j, o);
      if (a.z != nullptr && ends) {
        if (a.part_z != nullptr)
          row_store<false>(a.part_z, q * n + j, n - j, zacc[c]);
        else
          row_store<BF16>(a.dz, group * n + j, n - j, dz);
#pragma unroll
        for (int i = 0; i < 8; ++i) zacc[c][i] = 0.0f;
      }
    }
    float k1 = 0.0f, k2 = 0.0f;
    if (norm1) {
      const float2 s = row_sum2<W>(s3, s4, sh[1], first);
      k1 = a.center ? s.x * rn : 0.0f;
      k2 = s.y * rn;
    }
    if (on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = col(c);
        if (j >= n) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = norm1 ? r1 * (D[c][i] - k1 - (u[c].get(i) - m1) * r1 * k2) : D[c][i];
        row_store<BF16>(a.du, row * n + j, n - j, o);
      }
    }
    if (--left == 0) {
      left = a.per;
      ++group;
    }
    // sh[0] and sh[1] are taken in turn with a barrier between them; one alone needs its own
    if (W > 1 && norm1 != norm2) __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kResSums; ++k) {
    if (a.part[k] == nullptr) continue;   // the same for the whole launch
    if (R > 1) {                          // one strand after another, in order
      for (int r = 0; r < R; ++r) {
        __syncthreads();
        if (first / W == r) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* s = join + col(c) + i;
              if (r > 0) acc[k][c][i] += *s;
              *s = acc[k][c][i];
            }
        }
      }
      if (first / W != R - 1) continue;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = col(c);
      if (j < n) row_store<false>(a.part[k], (int64_t)blockIdx.x * n + j, n - j, acc[k][c]);
    }
  }
}

// The parts of the sums, 64 columns a workgroup of 16 rows of threads: blockIdx.y < kResSums the
// parameters' gradients over the slabs, behind them the gate's rows over their strands.
template <bool BF16>
__global__ __launch_bounds__(1024) void qg_resnorm_sums(ResArgs a) {
  __shared__ float sh[16][64];
  const int col = (int)(blockIdx.x * 64 + (threadIdx.x & 63)), slot = (int)(threadIdx.x >> 6);
  const int64_t g = (int64_t)blockIdx.y - kResSums;
  const float* part = g < 0 ? a.part[blockIdx.y] : a.part_z;
  if (part == nullptr) return;
  int64_t rows = a.split.slabs, r0 = 0;
  if (g >= 0) {
    // strands that lie behind the last token have left nothing
    const int64_t tokens = (g + 1) * a.per <= a.T ? a.per : a.T - g * a.per;
    r0 = g * a.split.parts;
    rows = (tokens + a.split.len - 1) / a.split.len;
  }
  float s = 0.0f;
  if (col < a.n)
    for (int64_t r = slot; r < rows; r += 16) s += part[(r0 + r) * a.n + col];
  sh[slot][threadIdx.x & 63] = s;
  __syncthreads();
  if (slot != 0 || col >= a.n) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += sh[k][threadIdx.x];
  if (g < 0) {
    a.sum[blockIdx.y][col] = s;
    return;
  }
  const int64_t e = g * a.n + col;
  if (BF16) {
    const float z = bf16_to_f32(static_cast<const uint16_t*>(a.z)[e]);
    static_cast<uint16_t*>(a.dz)[e] = to_bf16(s * gate_of(a.act, z).d);
  } else {
    static_cast<float*>(a.dz)[e] = s * gate_of(a.act, static_cast<const float*>(a.z)[e]).d;
  }
}

namespace {

// f(W, C, R) for rows of n: the fewest waves that hold a row at one chunk a thread, and as many rows side
// by side as fill eight waves.
template <class F>
void with_res_row(int64_t n, F&& f) {
  using std::integral_constant;
  auto go = [&](auto w, auto c) {
    constexpr int W = decltype(w)::value;
    f(w, c, integral_constant<int, (W < 8 ? 8 / W : 1)>{});
  };
  if (n <= 512) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (n <= 1024) go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  else if (n <= 2048) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (n <= 4096) go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (n <= 8192) go(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  else if (n <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

}  // namespace

ResSplit res_split(int64_t T, int64_t n, int64_t per) {
  int rows = 1;
  with_res_row(n, [&](auto, auto, auto r) { rows = decltype(r)::value; });
  const int64_t want = (int64_t)(n <= 512 ? 512 : 256) * rows, groups = (T + per - 1) / per;
  ResSplit s{};
  if (groups >= want || per == 1) {
    s.whole = (int32_t)((groups + want - 1) / want);
    s.parts = 1;
    s.len = s.whole * per;
    s.strands = (int32_t)((groups + s.whole - 1) / s.whole);
  } else {
    const int64_t most = want / groups < per ? want / groups : per;
    s.len = (per + most - 1) / most;
    s.parts = (int32_t)((per + s.len - 1) / s.len);
    s.whole = 1;
    s.strands = (int32_t)(groups * s.parts);
  }
  s.slabs = (s.strands + rows - 1) / rows;
  return s;
}

hipError_t launch_resnorm_fwd(const ResArgs& a, hipStream_t s) {
  with_res_row(a.n, [&](auto w, auto c, auto) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, R = W == 1 ? 4 : 1;
    const int64_t groups = (a.T + R - 1) / R;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
    if (a.bf16)
      hipLaunchKernelGGL((qg_resnorm_fwd<true, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
    else
      hipLaunchKernelGGL((qg_resnorm_fwd<false, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
  });
  return hipGetLastError();
}

hipError_t launch_resnorm_bwd(const ResArgs& a, hipStream_t s) {
  with_res_row(a.n, [&](auto w, auto c, auto r) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, R = decltype(r)::value;
    const dim3 grid((unsigned)a.split.slabs);
    if (a.bf16)
      hipLaunchKernelGGL((qg_resnorm_bwd<true, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
    else
      hipLaunchKernelGGL((qg_resnorm_bwd<false, W, C, R>), grid, dim3(64 * W * R), 0, s, a);
  });
  const hipError_t e = hipGetLastError();
  bool sums = a.part_z != nullptr;
  for (int k = 0; k < kResSums; ++k) sums |= a.sum[k] != nullptr && a.part[k] != a.sum[k];
  if (e != hipSuccess || !sums) return e;
  const int64_t groups = a.part_z != nullptr ? (a.T + a.per - 1) / a.per : 0;
  const dim3 grid((unsigned)((a.n + 63) / 64), (unsigned)(kResSums + groups));
  if (a.bf16)
    hipLaunchKernelGGL(qg_resnorm_sums<true>, grid, dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL(qg_resnorm_sums<false>, grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace qg
