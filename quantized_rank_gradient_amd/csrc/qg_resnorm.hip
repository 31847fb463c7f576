// The norms behind a block and before the next one, with the block's gate and scales (T tokens of n):
//   p = gamma1 (u - mean1) rstd1 + beta1,  h = alpha x + rho a(z) p,  y = gamma2 (h - mean2) rstd2 + beta2
// and the gradients of all of it. Each pass (but the backward one of rows beyond 8192) reads every tensor once and
// writes each result once; a token's row stays in registers from its loads to its stores, through both norms.
// Bytes bound both passes up to rows of 8192: 8192 x 4096 in bf16 with a gate for every value 74 us forward
// (335 MB at 4.5 TB/s) and 117 backward (537 MB at 4.6); without gate and first norm 53 and 74 (268 and 335 MB).
// The backward pass of longer rows reads some values again (2048 x 16384: 101 and 221 us). Rows that begin at any
// address cost more: 8192 x 4092 (8-byte boundaries) 87 and 141 us, 4095 (2-byte) 106 and 160, of which `fix`
// below has 5 to 6 and 13 to 14.
#include <type_traits>

#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

namespace {

// exp(x) for x <= 0, within 2 ulp: 2^(x log2 e) by the hardware, and what the rounding of x log2 e left out
// by the first term of the series. TAIL: also results below 2^-126 (from x = -87 on).
template <bool TAIL>
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float L = 1.44269502162933349609375f, LO = 1.92596299112661746887e-8f, LN2 = 0.693147180559945f;
  const float t = x * L, r = __builtin_fmaf(x, LO, __builtin_fmaf(x, L, -t));
  float e;
  if constexpr (TAIL) {
    const float k = __builtin_rintf(t);
    e = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(t - k), (int)k);
  } else {
    e = __builtin_amdgcn_exp2f(t);
  }
  return __builtin_fmaf(e, r * LN2, e);
}

// a(z) and a'(z) of eight values, each from exp of a number that is not positive: no overflow, and the
// derivatives keep their digits in both tails. The choices are made once for all of them; TAIL also takes
// values whose exp is subnormal or 0 (beyond 104: the limits).
template <int ACT, bool TAIL>
__device__ __forceinline__ void gates(const float (&z)[8], float (&ga)[8], float (&gd)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float m = (ACT == kGateTanh ? 2.0f : 1.0f) * fabsf(z[i]);
    if (TAIL) m = m > 150.0f ? 150.0f : m;   // NaN stays
    const float e = exp_neg<TAIL>(-m), r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    ga[i] = ACT == kGateTanh ? tanhf(z[i]) : z[i] >= 0.0f ? r : er;
    gd[i] = ACT == kGateTanh ? 4.0f * er * r : er * r;
  }
}
__device__ __forceinline__ void gates_of(int act, const float (&z)[8], float (&ga)[8], float (&gd)[8]) {
  if (act == kGateIdentity) {
#pragma unroll
    for (int i = 0; i < 8; ++i) ga[i] = z[i], gd[i] = 1.0f;
    return;
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(z[i]));
  if (__builtin_amdgcn_ballot_w64(m > 43.0f) != 0) {
    if (act == kGateSigmoid) gates<kGateSigmoid, true>(z, ga, gd);
    else gates<kGateTanh, true>(z, ga, gd);
  } else {
    if (act == kGateSigmoid) gates<kGateSigmoid, false>(z, ga, gd);
    else gates<kGateTanh, false>(z, ga, gd);
  }
}

// How rows are accessed: by n's remainder to eight.
enum { kRowShort = 0, kRowWhole = 1, kRowRest = 2 };

// Eight values from column j on of row `row` (the same for the whole wave) of p, to be read (get, then fix
// where they are used) or written (put); zeros, and nothing written, behind the row's end, without p and
// where it is not `on`. Loads are to go out without a branch, so that the compiler knows how many are on their
// way and waits for the oldest ones alone (8192 x 4096, backward: 164 -> 135 us).
//   kRowWhole  n a multiple of 8: through a resource that ends with the row
//   kRowRest   other n from 8 on: a chunk that the row's end cuts is read as the row's last eight values, and
//              shifted by `fix`; lanes without values read some others (`safe`: eight values that are there)
//   kRowShort  n < 8
template <bool BF16, int MODE>
struct RowIo {
  static constexpr int EACH = BF16 ? 2 : 4;
  static __device__ __forceinline__ rsrc_t at(const void* p, int64_t row, int n, bool on) {
    return make_rsrc(static_cast<const char*>(p) + row * n * EACH, on && p != nullptr ? n * EACH : 0);
  }
  static __device__ __forceinline__ void get(RowRaw<BF16>& v, const void* p, int64_t row, int n, int j,
                                             bool on, const void* safe) {
    if constexpr (MODE == kRowWhole) {
      const rsrc_t r = at(p, row, n, on);
      v.q[0] = bload128(r, j * EACH);
      if constexpr (!BF16) v.q[1] = bload128(r, j * EACH + 16);
    } else if constexpr (MODE == kRowRest) {
      const char* from = on && p != nullptr ? static_cast<const char*>(p) + row * n * EACH
                                            : static_cast<const char*>(safe);
      v.load(from, j < n - 8 ? j : n - 8, 8);
    } else if (on && p != nullptr && j < n) {
      v.load(static_cast<const char*>(p) + row * n * EACH, j, n - j);
    }
  }
  static __device__ __forceinline__ void fix(RowRaw<BF16>& v, const void* p, int n, int j) {
    if constexpr (MODE == kRowRest) {
      constexpr int N = BF16 ? 4 : 8;
      uint32_t w[N];
      __builtin_memcpy(w, v.q, sizeof(w));
      const int by = j <= n - 8 ? 0 : j - (n - 8);   // values too far left; 8 and more: none is the row's
      const bool none = by >= 8 || p == nullptr;
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t up = i + 1 < N ? w[i + 1] : 0;
          w[i] = (by & 1) ? (w[i] >> 16) | (up << 16) : w[i];
        }
      }
#pragma unroll
      for (int step = 1; step < N; step *= 2) {
        const bool on = by & (BF16 ? 2 * step : step);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = on ? (i + step < N ? w[i + step] : 0) : w[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = none ? 0 : w[i];
      __builtin_memcpy(v.q, w, sizeof(w));
    }
  }
  static __device__ __forceinline__ void put(void* p, int64_t row, int n, int j, const float (&v)[8],
                                             bool on) {
    if constexpr (MODE == kRowWhole) {
      const rsrc_t r = at(p, row, n, on);
      uint32_t w[BF16 ? 4 : 8];
#pragma unroll
      for (int i = 0; i < (BF16 ? 4 : 8); ++i)
        w[i] = BF16 ? pack_bf16x2(v[(2 * i) & 7], v[(2 * i + 1) & 7]) : __float_as_uint(v[i]);
#pragma unroll
      for (int k = 0; k < (BF16 ? 1 : 2); ++k)
        bstore128(r, j * EACH + 16 * k, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
    } else if (on && p != nullptr && j < n) {
      row_store<BF16>(static_cast<char*>(p) + row * n * EACH, j, n - j, v);
    }
  }
};
// Eight parameters, or `none` without p.
__device__ __forceinline__ RowRaw<false> vec_at(const float* p, int n, int j, float none) {
  if (p != nullptr) {
    RowRaw<false> v{};
    if (j < n) v.load(p, j, n - j);
    return v;
  }
  const uint32_t u = __float_as_uint(none);
  RowRaw<false> v;
  v.q[0] = v.q[1] = make_uint4(u, u, u, u);
  return v;
}
// First wave of this wave's row of W waves, as a scalar.
template <int W>
__device__ __forceinline__ int first_wave() {
  return __builtin_amdgcn_readfirstlane((int)(threadIdx.x / (64 * W)) * W);
}

}  // namespace

// The tokens lo .. hi - 1 of strand q.
__device__ __forceinline__ void strand_at(const ResArgs& a, int64_t q, int64_t& lo, int64_t& hi) {
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
}

// R tokens at a time, W waves to a row, C chunks of eight values a thread.
template <bool BF16, int MODE, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_resnorm_fwd(ResArgs a) {
  using Io = RowIo<BF16, MODE>;
  constexpr bool WHOLE = MODE == kRowWhole;
  __shared__ float2 sh[4][W * R];
  const int n = (int)a.n, first = first_wave<W>();
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
      for (int i = 0; i < 8; ++i) {
        const float d = v(c, i) - mean;
        if (WHOLE ? col(c) < n : col(c) + i < n) q = __builtin_fmaf(d, d, q);
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
      u[c] = x[c] = z[c] = {};
      Io::get(u[c], a.u, row, n, col(c), on, a.safe);
      Io::get(x[c], a.x, row, n, col(c), on, a.safe);
      Io::get(z[c], a.z, zrow, n, col(c), on, a.safe);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      Io::fix(u[c], a.u, n, col(c));
      Io::fix(x[c], a.x, n, col(c));
      Io::fix(z[c], a.z, n, col(c));
    }
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    if (a.g1 != nullptr)
      s1 = stats([&](int c, int i) { return u[c].get(i); }, sh[0], sh[1]);
    const float r1 = a.g1 != nullptr ? s1.y : 1.0f;
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = col(c);
      const RowRaw<false> g1 = vec_at(a.g1, n, j, 1.0f), b1 = vec_at(a.b1, n, j, 0.0f);
      const RowRaw<false> rho = vec_at(a.rho, n, j, 1.0f);
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p[i] = __builtin_fmaf((u[c].get(i) - s1.x) * r1, g1.get(i), b1.get(i)) * rho.get(i);
      if (a.z != nullptr) {
        float zz[8], ga[8], gd[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) zz[i] = z[c].get(i);
        gates_of(a.act, zz, ga, gd);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] *= ga[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = __builtin_fmaf(a.alpha, x[c].get(i), p[i]);
      if (j + 8 > n) {   // nothing behind the row's end
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (WHOLE || j + i >= n) h[c][i] = 0.0f;
      }
    }
    if (a.g2 != nullptr) s2 = stats([&](int c, int i) { return h[c][i]; }, sh[2], sh[3]);
    if (on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = col(c);
        Io::put(a.h, row, n, j, h[c], true);
        if (a.g2 == nullptr) continue;
        const RowRaw<false> g2 = vec_at(a.g2, n, j, 1.0f), b2 = vec_at(a.b2, n, j, 0.0f);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = __builtin_fmaf((h[c][i] - s2.x) * s2.y, g2.get(i), b2.get(i));
        Io::put(a.y, row, n, j, y, true);
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
// parameters are summed in registers, and the gate's over a group, too. With one chunk a thread the
// parameters stay in registers, and the values of the next token (bf16: the next two) are on their way while
// one is summed and written; longer rows have no registers for that (6144 columns: 202 us without, 252 with one
// token ahead, from spills).
template <bool BF16, int MODE, int W, int C, int R>
__global__ __launch_bounds__(64 * W * R) void qg_resnorm_bwd(ResArgs a) {
  using Io = RowIo<BF16, MODE>;
  constexpr bool WHOLE = MODE == kRowWhole;
  constexpr int DEPTH = C > 1 || W > 8 ? 0 : BF16 ? 2 : 1;   // tokens ahead
  constexpr bool AHEAD = DEPTH > 0;
  constexpr int N = 512 * W * C;   // columns held
  __shared__ float2 sh[2][W * R];
  __shared__ float join[R > 1 ? N : 1];
  const int n = (int)a.n, first = first_wave<W>();
  const int tid = (int)threadIdx.x - 64 * first;
  const float rn = 1.0f / (float)n;
  auto col = [&](int c) { return 8 * (tid + 64 * W * c); };
  const bool norm1 = a.g1 != nullptr, norm2 = a.g2 != nullptr, gated = a.z != nullptr;
  const int64_t q = (int64_t)blockIdx.x * R + first / W;
  int64_t lo, hi;
  strand_at(a, q, lo, hi);
  int64_t group = gated && hi > lo ? lo / a.per : 0;
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
  // without the first norm u is taken as normed already, by ones and zeros in the norm's place
  auto g1_of = [&](int c) { return vec_at(a.g1, n, col(c), 1.0f); };
  auto b1_of = [&](int c) { return vec_at(a.b1, n, col(c), 0.0f); };
  auto g2_of = [&](int c) { return vec_at(a.g2, n, col(c), 1.0f); };
  auto rho_of = [&](int c) { return vec_at(a.rho, n, col(c), 1.0f); };
  RowRaw<false> kg1{}, kb1{}, kg2{}, krho{};
  if (AHEAD) kg1 = g1_of(0), kb1 = b1_of(0), kg2 = g2_of(0), krho = rho_of(0);
  auto g1_at = [&](int c) { return AHEAD ? kg1 : g1_of(c); };
  auto b1_at = [&](int c) { return AHEAD ? kb1 : b1_of(c); };
  auto g2_at = [&](int c) { return AHEAD ? kg2 : g2_of(c); };
  auto rho_at = [&](int c) { return AHEAD ? krho : rho_of(c); };
  struct Token {
    RowRaw<BF16> dh[C], dy[C], h[C], u[C], z[C];   // zeros behind the row's end, and for what is not there
    float m1, r1, m2, r2;
  };
  auto fetch = [&](Token& t, int64_t row, int64_t grp) {
    const bool on = row < hi;   // the same for the whole wave
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = col(c);
      Io::get(t.dh[c], a.dh, row, n, j, on, a.safe);
      Io::get(t.dy[c], a.dy, row, n, j, on, a.safe);
      Io::get(t.h[c], a.h_in, row, n, j, on, a.safe);
      Io::get(t.u[c], a.u, row, n, j, on, a.safe);
      Io::get(t.z[c], a.z, grp, n, j, on, a.safe);
    }
    const float* st = a.stats + (on ? row : 0);
    t.m1 = st[0], t.r1 = st[a.T], t.m2 = st[2 * a.T], t.r2 = st[3 * a.T];
  };
  // The strand's token `it`, from t; those of the one DEPTH further on go to `next`. Strands of a workgroup may
  // differ in length, so every one comes to the sums of all tokens.
  auto token = [&](int64_t it, Token& t, Token& next) {
    const int64_t row = lo + it;
    const bool on = row < hi;   // the same for the whole wave
    const bool ends = left == 1 || row + 1 == hi;   // of the group, in this strand
    if (AHEAD)   // of the group of that token
      fetch(next, row + DEPTH, left > DEPTH ? group : group + (left == 1 && a.per == 1 ? DEPTH : 1));
    else
      fetch(t, row, group);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = col(c);
      Io::fix(t.dh[c], a.dh, n, j), Io::fix(t.dy[c], a.dy, n, j), Io::fix(t.h[c], a.h_in, n, j);
      Io::fix(t.u[c], a.u, n, j), Io::fix(t.z[c], a.z, n, j);
    }
    // hh and uh of an element: (v - mean) rstd
    const float r1 = norm1 ? t.r1 : 1.0f, r2 = t.r2;
    const float c1 = a.center && norm1 ? -t.m1 * r1 : 0.0f, c2 = a.center ? -t.m2 * r2 : 0.0f;
    float D[C][8];
    float2 s = make_float2(0.0f, 0.0f);
    if (on && norm2) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const RowRaw<false> g2 = g2_at(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // dy is 0 behind the row's end
          const float hh = __builtin_fmaf(t.h[c].get(i), r2, c2);
          const float d = t.dy[c].get(i), e = d * g2.get(i);
          s.x += e;
          s.y = __builtin_fmaf(e, hh, s.y);
          acc[kResG2][c][i] = __builtin_fmaf(d, hh, acc[kResG2][c][i]);
          acc[kResB2][c][i] += d;
        }
      }
    }
    if (norm2) s = row_sum2<W>(s.x, s.y, sh[0], first);
    float k1 = a.center ? s.x * rn : 0.0f, k2 = -s.y * rn;
    s = make_float2(0.0f, 0.0f);
    if (on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = col(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) D[c][i] = t.dh[c].get(i);
        if (norm2) {
          const RowRaw<false> g2 = g2_at(c);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float hh = __builtin_fmaf(t.h[c].get(i), r2, c2);
            const float e = __builtin_fmaf(t.dy[c].get(i), g2.get(i), -k1);
            D[c][i] = __builtin_fmaf(r2, __builtin_fmaf(hh, k2, e), D[c][i]);
          }
          if (j + 8 > n) {   // nothing behind the row's end
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (WHOLE || j + i >= n) D[c][i] = 0.0f;
          }
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = a.alpha * D[c][i];
        Io::put(a.dx, row, n, j, o, true);
        const RowRaw<false> g1 = g1_at(c), b1 = b1_at(c), rho = rho_at(c);
        float ga[8], gd[8];
        if (gated) {
          float zz[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) zz[i] = t.z[c].get(i);
          gates_of(a.act, zz, ga, gd);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) ga[i] = 1.0f, gd[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = D[c][i], uh = __builtin_fmaf(t.u[c].get(i), r1, c1);
          const float p = __builtin_fmaf(uh, g1.get(i), b1.get(i)), w = rho.get(i), dp = d * p;
          acc[kResRho][c][i] = __builtin_fmaf(dp, ga[i], acc[kResRho][c][i]);
          zacc[c][i] = __builtin_fmaf(dp, w, zacc[c][i]);
          const float v = d * w * ga[i];
          acc[kResG1][c][i] = __builtin_fmaf(v, uh, acc[kResG1][c][i]);
          acc[kResB1][c][i] += v;
          const float f = v * g1.get(i);
          s.x += f;
          s.y = __builtin_fmaf(f, uh, s.y);
          D[c][i] = f;
        }
        if (gated && ends) {
          RowIo<false, MODE>::put(a.part_z, q, n, j, zacc[c], true);   // once a strand
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = zacc[c][i] * gd[i];
          Io::put(a.dz, group, n, j, o, a.part_z == nullptr);
#pragma unroll
          for (int i = 0; i < 8; ++i) zacc[c][i] = 0.0f;
        }
      }
    }
    if (norm1) s = row_sum2<W>(s.x, s.y, sh[1], first);
    k1 = a.center ? s.x * rn : 0.0f;
    k2 = -s.y * rn;
    if (on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (norm1) {   // without it u has no part in du, not even an infinite one
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float uh = __builtin_fmaf(t.u[c].get(i), r1, c1);
            D[c][i] = r1 * __builtin_fmaf(uh, k2, D[c][i] - k1);
          }
        }
        Io::put(a.du, row, n, col(c), D[c], true);
      }
    }
    if (--left == 0) {
      left = a.per;
      ++group;
    }
    // sh[0] and sh[1] are taken in turn with a barrier between them; one alone needs its own
    if (W > 1 && norm1 != norm2) __syncthreads();
  };
  Token t[DEPTH + 1] = {};
  if (DEPTH > 0) fetch(t[0], lo, group);
  if (DEPTH > 1) fetch(t[1], lo + 1, left == 1 ? group + 1 : group);
  for (int64_t it = 0; it < a.split.len; it += DEPTH + 1) {
#pragma unroll
    for (int d = 0; d <= DEPTH; ++d)
      if (it + d < a.split.len) token(it + d, t[d], t[(d + DEPTH) % (DEPTH + 1)]);
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
    for (int c = 0; c < C; ++c)
      RowIo<false, MODE>::put(a.part[k], blockIdx.x, n, col(c), acc[k][c], true);
  }
}

// Rows beyond kResLong, whose sums of five parameters no workgroup has registers for (2048 x 16384 in bf16 with
// spills 454 us, so 221; 1024 x 32768 867 and 312), in three launches: a token's two means behind the second norm
// (`row_means`), the sums over the tokens by columns, for which a thread needs its own columns alone, and the
// tokens' own gradients. They read 12 values where one pass would read 5, and write as many. The rows come last:
// their results may lie over what the others read.
template <bool BF16, int MODE, int W, int C>
__global__ __launch_bounds__(64 * W) void qg_resnorm_bwd_means(ResArgs a) {
  using Io = RowIo<BF16, MODE>;
  __shared__ float2 sh[2][W];
  const int n = (int)a.n, tid = (int)threadIdx.x;
  const float rn = 1.0f / (float)n;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    RowRaw<BF16> dy[C], h[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      Io::get(dy[c], a.dy, row, n, j, true, a.safe);
      Io::get(h[c], a.h_in, row, n, j, true, a.safe);
    }
    const float r2 = a.stats[3 * a.T + row], c2 = a.center ? -a.stats[2 * a.T + row] * r2 : 0.0f;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      Io::fix(dy[c], a.dy, n, j), Io::fix(h[c], a.h_in, n, j);
      const RowRaw<false> g2 = vec_at(a.g2, n, j, 1.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // dy is 0 behind the row's end
        const float e = dy[c].get(i) * g2.get(i);
        s.x += e;
        s.y = __builtin_fmaf(e, __builtin_fmaf(h[c].get(i), r2, c2), s.y);
      }
    }
    s = row_sum2<W>(s.x, s.y, sh[par], 0);
    if (tid == 0) a.row_means[row] = make_float2(a.center ? s.x * rn : 0.0f, s.y * rn);
  }
}

// Eight columns a thread, a strand a workgroup (blockIdx.y): the sums of drho, dgamma and dbeta, and the gate's
// gradients, for which a group's tokens are summed.
template <bool BF16, int MODE>
__global__ __launch_bounds__(kThreads) void qg_resnorm_bwd_columns(ResArgs a) {
  using Io = RowIo<BF16, MODE>;
  constexpr bool WHOLE = MODE == kRowWhole;
  const int n = (int)a.n, j = 8 * (int)(blockIdx.x * kThreads + threadIdx.x);
  const bool norm1 = a.g1 != nullptr, norm2 = a.g2 != nullptr, gated = a.z != nullptr;
  const int64_t q = blockIdx.y;
  int64_t lo, hi;
  strand_at(a, q, lo, hi);
  int64_t group = gated && hi > lo ? lo / a.per : 0;
  int64_t left = (group + 1) * a.per - lo;   // tokens to the group's end
  const RowRaw<false> g1 = vec_at(a.g1, n, j, 1.0f), b1 = vec_at(a.b1, n, j, 0.0f);
  const RowRaw<false> g2 = vec_at(a.g2, n, j, 1.0f), rho = vec_at(a.rho, n, j, 1.0f);
  float acc[kResSums][8] = {}, zacc[8] = {};
  struct Token {
    RowRaw<BF16> dh, dy, h, u, z;
    float m1, r1, m2, r2;
    float2 k;
  };
  auto fetch = [&](Token& t, int64_t row, int64_t grp) {
    const bool on = row < hi;
    Io::get(t.dh, a.dh, row, n, j, on, a.safe);
    Io::get(t.dy, a.dy, row, n, j, on, a.safe);
    Io::get(t.h, a.h_in, row, n, j, on, a.safe);
    Io::get(t.u, a.u, row, n, j, on, a.safe);
    Io::get(t.z, a.z, grp, n, j, on, a.safe);
    const int64_t at = on ? row : 0;
    const float* st = a.stats + at;
    t.m1 = st[0], t.r1 = st[a.T], t.m2 = st[2 * a.T], t.r2 = st[3 * a.T];
    t.k = norm2 ? a.row_means[at] : make_float2(0.0f, 0.0f);
  };
  auto token = [&](int64_t row, Token& t, Token& next) {
    if (row >= hi) return;
    fetch(next, row + 1, left > 1 ? group : group + 1);
    Io::fix(t.dh, a.dh, n, j), Io::fix(t.dy, a.dy, n, j), Io::fix(t.h, a.h_in, n, j);
    Io::fix(t.u, a.u, n, j), Io::fix(t.z, a.z, n, j);
    const float r1 = norm1 ? t.r1 : 1.0f, r2 = t.r2;
    const float c1 = a.center && norm1 ? -t.m1 * r1 : 0.0f, c2 = a.center ? -t.m2 * r2 : 0.0f;
    float ga[8], gd[8];
    if (gated) {
      float zz[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) zz[i] = t.z.get(i);
      gates_of(a.act, zz, ga, gd);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) ga[i] = 1.0f, gd[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float D = t.dh.get(i);
      if (norm2) {
        const float hh = __builtin_fmaf(t.h.get(i), r2, c2), d = t.dy.get(i);
        acc[kResG2][i] = __builtin_fmaf(d, hh, acc[kResG2][i]);
        acc[kResB2][i] += d;
        const float e = __builtin_fmaf(d, g2.get(i), -t.k.x);
        D = __builtin_fmaf(r2, __builtin_fmaf(hh, -t.k.y, e), D);
      }
      const float uh = __builtin_fmaf(t.u.get(i), r1, c1);
      const float p = __builtin_fmaf(uh, g1.get(i), b1.get(i)), w = rho.get(i), dp = D * p;
      acc[kResRho][i] = __builtin_fmaf(dp, ga[i], acc[kResRho][i]);
      zacc[i] = __builtin_fmaf(dp, w, zacc[i]);
      const float v = D * w * ga[i];
      acc[kResG1][i] = __builtin_fmaf(v, uh, acc[kResG1][i]);
      acc[kResB1][i] += v;
    }
    if (gated && (left == 1 || row + 1 == hi)) {   // the group's last token of this strand
      RowIo<false, MODE>::put(a.part_z, q, n, j, zacc, true);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = zacc[i] * gd[i];
        zacc[i] = 0.0f;
      }
      Io::put(a.dz, group, n, j, o, a.part_z == nullptr);
    }
    if (--left == 0) {
      left = a.per;
      ++group;
    }
  };
  Token t[2] = {};
  fetch(t[0], lo, group);
  for (int64_t row = lo; row < hi; row += 2) {
    token(row, t[0], t[1]);
    token(row + 1, t[1], t[0]);
  }
#pragma unroll
  for (int k = 0; k < kResSums; ++k)
    if (a.part[k] != nullptr) RowIo<false, MODE>::put(a.part[k], q, n, j, acc[k], true);
}

// A token at a time: dx and du. Rows beyond 16384 spill (100 registers in bf16; 114 in fp32); loading them chunk
// by chunk, the next one ahead, spilled as many.
template <bool BF16, int MODE, int W, int C>
__global__ __launch_bounds__(64 * W) void qg_resnorm_bwd_rows(ResArgs a) {
  using Io = RowIo<BF16, MODE>;
  constexpr bool WHOLE = MODE == kRowWhole;
  __shared__ float2 sh[2][W];
  const int n = (int)a.n, tid = (int)threadIdx.x;
  const bool norm1 = a.g1 != nullptr, norm2 = a.g2 != nullptr, gated = a.z != nullptr;
  const float rn = 1.0f / (float)n;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    RowRaw<BF16> dh[C], dy[C], h[C], u[C], z[C];
    const int64_t grp = gated ? row / a.per : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      Io::get(dh[c], a.dh, row, n, j, true, a.safe);
      Io::get(dy[c], a.dy, row, n, j, true, a.safe);
      Io::get(h[c], a.h_in, row, n, j, true, a.safe);
      Io::get(u[c], a.u, row, n, j, true, a.safe);
      Io::get(z[c], a.z, grp, n, j, true, a.safe);
    }
    const float* st = a.stats + row;
    const float r1 = norm1 ? st[a.T] : 1.0f, r2 = st[3 * a.T];
    const float c1 = a.center && norm1 ? -st[0] * r1 : 0.0f, c2 = a.center ? -st[2 * a.T] * r2 : 0.0f;
    const float2 k = norm2 ? a.row_means[row] : make_float2(0.0f, 0.0f);
    float f[C][8];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = 8 * (tid + 64 * W * c);
      Io::fix(dh[c], a.dh, n, j), Io::fix(dy[c], a.dy, n, j), Io::fix(h[c], a.h_in, n, j);
      Io::fix(u[c], a.u, n, j), Io::fix(z[c], a.z, n, j);
      float D[8], o[8], ga[8], gd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) D[i] = dh[c].get(i), ga[i] = 1.0f;
      if (norm2) {
        const RowRaw<false> g2 = vec_at(a.g2, n, j, 1.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hh = __builtin_fmaf(h[c].get(i), r2, c2);
          const float e = __builtin_fmaf(dy[c].get(i), g2.get(i), -k.x);
          D[i] = __builtin_fmaf(r2, __builtin_fmaf(hh, -k.y, e), D[i]);
          if (WHOLE ? j >= n : j + i >= n) D[i] = 0.0f;   // nothing behind the row's end
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.alpha * D[i];
      Io::put(a.dx, row, n, j, o, true);
      if (gated) {
        float zz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) zz[i] = z[c].get(i);
        gates_of(a.act, zz, ga, gd);
      }
      const RowRaw<false> g1 = vec_at(a.g1, n, j, 1.0f), rho = vec_at(a.rho, n, j, 1.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[c][i] = D[i] * rho.get(i) * ga[i] * g1.get(i);
        s.x += f[c][i];
        s.y = __builtin_fmaf(f[c][i], __builtin_fmaf(u[c].get(i), r1, c1), s.y);
      }
    }
    if (norm1) s = row_sum2<W>(s.x, s.y, sh[par], 0);
    const float k1 = a.center ? s.x * rn : 0.0f, k2 = -s.y * rn;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (norm1) {   // as above
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float uh = __builtin_fmaf(u[c].get(i), r1, c1);
          f[c][i] = r1 * __builtin_fmaf(uh, k2, f[c][i] - k1);
        }
      }
      Io::put(a.du, row, n, 8 * (tid + 64 * W * c), f[c], true);
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
  if (col < a.n) {
    const float* at = part + r0 * a.n + col;
    // eight on their way at a time; the order of the sum is the same for any number of them
    for (int64_t r = slot; r < rows; r += 128) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = r + 16 * k < rows ? at[(r + 16 * k) * a.n] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  }
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
  auto slope = [&](float z) {
    const float zz[8] = {z, z, z, z, z, z, z, z};
    float ga[8], gd[8];
    gates_of(a.act, zz, ga, gd);
    return gd[0];
  };
  if (BF16) {
    const float z = bf16_to_f32(static_cast<const uint16_t*>(a.z)[e]);
    static_cast<uint16_t*>(a.dz)[e] = to_bf16(s * slope(z));
  } else {
    static_cast<float*>(a.dz)[e] = s * slope(static_cast<const float*>(a.z)[e]);
  }
}

namespace {

// f(W, C, R) for rows of n: about the fewest waves that hold a row at one chunk a thread, and as many rows
// side by side as fill eight waves. Waves without values cost: 2^25 values in bf16, forward and backward, rows of 1201
// with four waves 126 and 234 us, with three 107 and 218; of 2301 with eight 138 and 250, with five 126 and 231; of
// 5461 with eight of two chunks 141 and 235, with twelve of one 117 and 201.
template <class F>
void with_res_row(int64_t n, F&& f) {
  using std::integral_constant;
  auto go = [&](auto w, auto c) {
    constexpr int W = decltype(w)::value;
    f(w, c, integral_constant<int, (W < 8 ? 8 / W : 1)>{});
  };
  if (n <= 512) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (n <= 1024) go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  else if (n <= 1536) go(integral_constant<int, 3>{}, integral_constant<int, 1>{});
  else if (n <= 2048) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (n <= 2560) go(integral_constant<int, 5>{}, integral_constant<int, 1>{});
  else if (n <= 4096) go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (n <= 6144) go(integral_constant<int, 12>{}, integral_constant<int, 1>{});
  else if (n <= 8192) go(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  else if (n <= 12288) go(integral_constant<int, 12>{}, integral_constant<int, 2>{});
  else if (n <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

}  // namespace

ResSplit res_split(int64_t T, int64_t n, int64_t per) {
  int rows = 1;
  with_res_row(n, [&](auto, auto, auto r) { rows = decltype(r)::value; });
  // long rows: as many that their columns make 512 workgroups
  const int64_t want = n > kResLong ? ((int64_t)1 << 20) / n : (int64_t)(n <= 512 ? 512 : 256) * rows;
  const int64_t groups = (T + per - 1) / per;
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

// f(BF16, MODE, W, C, R) for a call.
template <class F>
void with_res(const ResArgs& a, F&& f) {
  using std::integral_constant;
  auto typed = [&](auto mode, auto w, auto c, auto r) {
    if (a.bf16) f(std::true_type{}, mode, w, c, r);
    else f(std::false_type{}, mode, w, c, r);
  };
  constexpr integral_constant<int, 1> one{};
  if (a.n < 8) return typed(integral_constant<int, kRowShort>{}, one, one, integral_constant<int, 8>{});
  with_res_row(a.n, [&](auto w, auto c, auto r) {
    if (a.n % 8 == 0) typed(integral_constant<int, kRowWhole>{}, w, c, r);
    else typed(integral_constant<int, kRowRest>{}, w, c, r);
  });
}

hipError_t launch_resnorm_fwd(const ResArgs& a, hipStream_t s) {
  with_res(a, [&](auto bf16, auto mode, auto w, auto c, auto) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, R = W == 1 ? 4 : 1;
    const int64_t groups = (a.T + R - 1) / R;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
    hipLaunchKernelGGL((qg_resnorm_fwd<decltype(bf16)::value, decltype(mode)::value, W, C, R>), grid,
                       dim3(64 * W * R), 0, s, a);
  });
  return hipGetLastError();
}

hipError_t launch_resnorm_bwd(const ResArgs& a, hipStream_t s) {
  with_res(a, [&](auto bf16, auto mode, auto w, auto c, auto r) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int MODE = decltype(mode)::value, W = decltype(w)::value, C = decltype(c)::value;
    if constexpr (512 * W * C > kResLong && MODE != kRowShort) {
      const dim3 rows((unsigned)(a.T < (1 << 20) ? a.T : (1 << 20)));
      const dim3 columns((unsigned)((a.n + 8 * kThreads - 1) / (8 * kThreads)), (unsigned)a.split.strands);
      if (a.g2 != nullptr)
        hipLaunchKernelGGL((qg_resnorm_bwd_means<BF16, MODE, W, C>), rows, dim3(64 * W), 0, s, a);
      hipLaunchKernelGGL((qg_resnorm_bwd_columns<BF16, MODE>), columns, dim3(kThreads), 0, s, a);
      hipLaunchKernelGGL((qg_resnorm_bwd_rows<BF16, MODE, W, C>), rows, dim3(64 * W), 0, s, a);
    } else {
      hipLaunchKernelGGL((qg_resnorm_bwd<BF16, MODE, W, C, decltype(r)::value>), dim3((unsigned)a.split.slabs),
                         dim3(64 * W * decltype(r)::value), 0, s, a);
    }
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
