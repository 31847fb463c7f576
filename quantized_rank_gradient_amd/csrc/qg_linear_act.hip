// A linear layer on INT8 weights with its bias, activation and residual in the product's epilogue,
// and its backward pass:
//   Z = X W~^T + bias,  Y = act(Z) + residual                    (W~ = bf16(q s), m x n)
//   dZ = dY act'(Z),  dbias = sum_t dZ,  dX = dZ W~,  G = dZ^T X
// Z is kept in bf16 when the backward pass will ask for it (its rounding moves act' by at most
// |act''| 2^-8 |Z|); the activation itself takes the fp32 Z. dZ is rounded to bf16 for its two
// products, as their MFMAs take it (a pair of bf16 would double them): with the results' own rounding
// dX and G are 2.4e-3 off in the 2-norm, where one rounding gives 1.7e-3. dbias sums the fp32 dZ.
//
// The forward pass has three forms, chosen by lin_fwd_form below. Few tokens (up to 64): the time is
// the weights' bytes; a workgroup takes 16 or 32 weight rows whole, its waves split K, and every
// code goes from memory to registers once, is dequantized there and multiplied by 16 tokens per
// MFMA; the partial sums meet in LDS. Some tokens: a product on tiles that dequantizes the codes
// on their way from LDS to the MFMAs. Many tokens: the products of qg_mm.hpp, on W~ written to the
// workspace by one pass (2 bytes written and read per weight, small against 2 T operations on it).
#include <algorithm>

#include "qg_mm.hpp"
#include "qg_kernels.hpp"

namespace qg {

// ------------------------------------------------------------------- activations ---
// Phi(z), and e = exp(-z^2 / 2): Phi(-x) = e g(x) for x >= 0, with g(x) exp(-x^2/2) exp(x^2/2)
// smooth in t = 1 / (1 + 0.315 x): t times a polynomial of degree 7 in t, fitted here for the
// least relative error over 0 <= x <= 40 (3.8e-7; 1.1e-6 in fp32 down to z = -5), so that the left
// tail keeps its relative accuracy. About 16 instructions; a general complementary error function
// took 30 us of a round of 256 x 256 tiles (of 130).
__device__ __forceinline__ float phi(float z, float& e) {
  const float x = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.315f, x, 1.0f));
  float q = 0.034444138407707214f;
  q = __builtin_fmaf(q, t, -0.12904885411262512f);
  q = __builtin_fmaf(q, t, 0.12526245415210724f);
  q = __builtin_fmaf(q, t, 0.005173159763216972f);
  q = __builtin_fmaf(q, t, 0.10147546231746674f);
  q = __builtin_fmaf(q, t, 0.11121241748332977f);
  q = __builtin_fmaf(q, t, 0.12581878900527954f);
  q = __builtin_fmaf(q, t, 0.12566231191158295f);
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * (x * x));
  q = q * t * e;
  return z < 0.0f ? q : 1.0f - q;
}
constexpr float kTanhK = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;
// 1 / (1 + exp(-z)) by the hardware's exponential and reciprocal (an ulp each)
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;   // a NaN stays one
  if constexpr (ACT == kActGelu) {
    float e;
    return z * phi(z, e);
  }
  // (1 + tanh u) / 2 = sigmoid(2 u)
  if constexpr (ACT == kActGeluTanh) return z * sigmoid(2.0f * kTanhK * (z + kTanhC * z * z * z));
  if constexpr (ACT == kActSilu) return z * sigmoid(z);
  return z;
}
// From some z on every derivative here is 1 or 0 to the last bit, and stopping there keeps z^2, z^3 and
// z times 0 finite: at 40 to the right, to the left at -40 for the GELUs (exp(-800), and less) and
// at -104 for SiLU, whose sigmoid goes down by exp(z) alone (at -40 the derivative is -1.7e-16 still).
template <int ACT>
__device__ __forceinline__ float act_bwd(float z) {
  constexpr float left = ACT == kActSilu ? -104.0f : -40.0f;
  if constexpr (ACT != kActRelu) z = z > 40.0f ? 40.0f : (z < left ? left : z);
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  if constexpr (ACT == kActGelu) {
    float e;
    const float p = phi(z, e);
    return __builtin_fmaf(0.39894228040143268f * z, e, p);
  }
  if constexpr (ACT == kActGeluTanh) {
    const float s = sigmoid(2.0f * kTanhK * (z + kTanhC * z * z * z));
    return s + z * s * (1.0f - s) * 2.0f * kTanhK * (1.0f + 3.0f * kTanhC * z * z);
  }
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 dequant8_w(uint2 w, float s) {
  const float f[8] = {mul_rn(sbyte_to_f32<0>(w.x), s), mul_rn(sbyte_to_f32<1>(w.x), s),
                      mul_rn(sbyte_to_f32<2>(w.x), s), mul_rn(sbyte_to_f32<3>(w.x), s),
                      mul_rn(sbyte_to_f32<0>(w.y), s), mul_rn(sbyte_to_f32<1>(w.y), s),
                      mul_rn(sbyte_to_f32<2>(w.y), s), mul_rn(sbyte_to_f32<3>(w.y), s)};
  return pack_bf16x8(f);
}

// W~ of the whole weight, 16 codes (one scale group) per thread; its sides are multiples of 8, so numel
// is one of 64.
__device__ __forceinline__ void dequant_block(const LinActArgs& a, int block) {
  const int64_t numel = a.m * a.n, e = ((int64_t)block * kThreads + threadIdx.x) * 16;
  if (e >= numel) return;
  const float s = a.Ws[e >> 8];
  const uint4 w = *reinterpret_cast<const uint4*>(a.Wq + e);
  *reinterpret_cast<uint4*>(a.Wt + e) = dequant8_w(make_uint2(w.x, w.y), s);
  *reinterpret_cast<uint4*>(a.Wt + e + 8) = dequant8_w(make_uint2(w.z, w.w), s);
}
__global__ __launch_bounds__(kThreads) void qg_lin_dequant(LinActArgs a) {
  dequant_block(a, blockIdx.x);
}

// ------------------------------------------------------------------ many tokens ---
// Eight outputs (column j on, a multiple of 8) of token i from their sums v.
template <class ACT>
__device__ __forceinline__ void finish8(const LinActArgs& a, int i, int j, const float (&v)[8],
                                        uint4 res, ACT&& act) {
  const int64_t at = (int64_t)i * a.m + j;
  float z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = v[e];
  if (a.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += a.bias[j + e];
  }
  if (a.Z != nullptr) *reinterpret_cast<uint4*>(a.Z + at) = pack_bf16x8(z);
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = act(z[e]);
  if (a.res != nullptr) {
    float q[8];
    unpack_bf16x8(res, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += q[e];
  }
  *reinterpret_cast<uint4*>(a.Y + at) = pack_bf16x8(z);
}
__device__ __forceinline__ uint4 residual8(const LinActArgs& a, int i, int j) {
  return a.res != nullptr && i < (int)a.T && j < (int)a.m
             ? *reinterpret_cast<const uint4*>(a.res + (int64_t)i * a.m + j)
             : make_uint4(0, 0, 0, 0);
}

// One tile of Y (rows: tokens, columns: outputs). 4096 tokens through 11008 x 4096 with gelu, Z kept:
// 352 us (1.05 PFLOP/s; the board's power, and 2.7 rounds of tiles) behind 27 us for W~.
template <class T, int ACT>
__device__ __forceinline__ void fwd_tile(const LinActArgs& a, int i0, int j0, uint16_t* lds) {
  const int rows = (int)a.T, m = (int)a.m, n = (int)a.n;
  f32x16 acc[T::XM][T::XN];
  mm_kloop<T>(MmOperand{a.X, n, rows, n}, MmOperand{a.Wt, n, m, n}, i0, j0, n, lds, acc);
  float* img = reinterpret_cast<float*>(lds);
#pragma unroll 1
  for (int pass = 0; pass < T::PASSES; ++pass) {
    mm_image<T>(img, acc, pass);
    const int ib = i0 + T::IMG_ROWS * pass;
    mm_rows<T, 8>(
        img, [&](int r, int j) { return residual8(a, ib + r, j0 + j); },
        [&](int r, int j, const float(&v)[8], uint4 res) {
          if (ib + r < rows && j0 + j < m)
            finish8(a, ib + r, j0 + j, v, res, [](float z) { return act_fwd<ACT>(z); });
        });
  }
}

// One tile of out (M x N bf16, row-major) = A B^T, for dX (A = dZ by rows, B = W~ by columns) and G
// (A = dZ by columns, B = X by columns).
struct LinProduct {
  MmOperand A, B;
  int M, N, K;
  uint16_t* out;
  int tm, tn, blocks;   // the grid of tiles and the workgroups that it takes
  int split;            // parts of K (64-tiles), and where they meet
  float* parts;
  uint32_t* counts;
};
// `part`: which part of the sum, of tile `t`, where the product is cut.
template <class T>
__device__ __forceinline__ void product_tile(const LinProduct& p, int i0, int j0, int t, int part,
                                             uint16_t* lds) {
  f32x16 acc[T::XM][T::XN];
  if constexpr (T::XM == 1) {
    const int st = (p.K + kMmK - 1) / kMmK, len = (st + p.split - 1) / p.split * kMmK;
    const int k0 = part * len, K = p.K - k0 < len ? p.K - k0 : len;
    mm_kloop<T>(mm_cut<T::AKM>(p.A, k0, K), mm_cut<T::BKM>(p.B, k0, K), i0, j0, K, lds, acc);
    if (p.split > 1 && !mm_join<T>(acc[0][0], p.parts + (size_t)t * p.split * (T::BM * T::BN),
                                   p.counts + t, part, p.split, lds))
      return;
  } else {
    mm_kloop<T>(p.A, p.B, i0, j0, p.K, lds, acc);
  }
  float* img = reinterpret_cast<float*>(lds);
#pragma unroll 1
  for (int pass = 0; pass < T::PASSES; ++pass) {
    mm_image<T>(img, acc, pass);
    const int ib = i0 + T::IMG_ROWS * pass;
    mm_rows<T, 4>(img, MmNone{}, [&](int r, int j, const float(&v)[8], MmNone) {
      const int i = ib + r, jj = j0 + j;
      if (i < p.M && jj < p.N)
        *reinterpret_cast<uint4*>(p.out + (int64_t)i * p.N + jj) = pack_bf16x8(v);
    });
  }
}

// f(tile type, i0, j0, tile, part) for the tile, or quarter of one, or part of its sum, of workgroup b
// of a tm x tn grid of tiles; parts with the same K values run side by side.
template <int X, bool AKM, bool BKM, class F>
__device__ __forceinline__ void lin_tile(int b, int tm, int tn, int split, F&& f) {
  int q = -1, ti, tj, part = 0;
  int t = X > 2 ? mm_pick(b, tm * tn, q) : xcd_remap(b, tm * tn * split);
  if constexpr (X == 1) {
    part = t / (tm * tn);
    t -= part * (tm * tn);
  }
  mm_band(t, tm, tn, ti, tj);
  if constexpr (X > 2) {
    if (q >= 0) {
      using U = MmTile<X / 2, X / 2, AKM, BKM, MmBf16>;
      f(U{}, (2 * ti + (q >> 1)) * U::BM, (2 * tj + (q & 1)) * U::BN, t, 0);
      return;
    }
  }
  using T = MmTile<X, X, AKM, BKM, MmBf16>;
  f(T{}, ti * T::BM, tj * T::BN, t, part);
}

template <int X, int ACT>
__global__ __launch_bounds__(kThreads, X > 2 ? 1 : X > 1 ? 2 : 3) void qg_lin_act_fwd(LinActArgs a,
                                                                                     int tm, int tn) {
  __shared__ __attribute__((
      aligned(16))) uint16_t lds[MmTile<X, X, false, false, MmBf16>::LDS_BYTES / 2];
  lin_tile<X, false, false>(blockIdx.x, tm, tn, 1, [&](auto t, int i0, int j0, int, int) {
    fwd_tile<decltype(t), ACT>(a, i0, j0, lds);
  });
}

// out[c] = sum of part[s][c] over s, always in the same order: 64 columns a workgroup of W waves,
// every W-th row to each.
template <int W>
__device__ __forceinline__ void col_sum_block(const float* part, float* out, int slabs, int64_t cols,
                                              int block, float* sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)block * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int k = wave; k < slabs; k += W) s += part[k * cols + c];
  }
  sh[wave * 64 + lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += sh[w * 64 + lane];
    out[c] = t;
  }
}
__global__ __launch_bounds__(1024) void qg_col_sum(const float* part, float* out,
                                                   const float* part2, float* out2, int slabs,
                                                   int64_t cols) {
  __shared__ float sh[16 * 64];
  col_sum_block<16>(blockIdx.y ? part2 : part, blockIdx.y ? out2 : out, slabs, cols, blockIdx.x, sh);
}

// The backward pass's second half, one launch: the tiles of dX = dZ W~, those of G = dZ^T X, and the
// columns of dbias (any of the three may be missing). 4096 tokens through 11008 x 4096: 578 us,
// 1.28 PFLOP/s, bound by the board's power; 1000 through 1376 x 512: 9 us, the latency of 8 to 22
// stages and an epilogue; 16 through 11008 x 4096: dX 22 us with its sum over 11008 in 6 parts (44
// whole), G 29 us (its 90 MB).
struct LinBackward {
  LinProduct dx, g;
  const float* part;
  float* dbias;
  int slabs;
  int64_t m;
};
template <int X>
__global__ __launch_bounds__(kThreads, X > 2 ? 1 : X > 1 ? 2 : 3) void qg_lin_act_bwd(LinBackward b) {
  __shared__ __attribute__((
      aligned(16))) uint16_t lds[MmTile<X, X, true, true, MmBf16>::LDS_BYTES / 2];
  int k = blockIdx.x;
  if (k < b.dx.blocks) {
    lin_tile<X, false, true>(k, b.dx.tm, b.dx.tn, b.dx.split,
                             [&](auto type, int i0, int j0, int t, int part) {
                               product_tile<decltype(type)>(b.dx, i0, j0, t, part, lds);
                             });
    return;
  }
  k -= b.dx.blocks;
  if (k < b.g.blocks) {
    lin_tile<X, true, true>(k, b.g.tm, b.g.tn, b.g.split,
                            [&](auto type, int i0, int j0, int t, int part) {
                              product_tile<decltype(type)>(b.g, i0, j0, t, part, lds);
                            });
    return;
  }
  col_sum_block<4>(b.part, b.dbias, b.slabs, b.m, k - b.g.blocks, reinterpret_cast<float*>(lds));
}

__device__ __forceinline__ void zero_counts(uint32_t* counts) {
  for (int i = threadIdx.x; i < 2 * kMmParts; i += kThreads) counts[i] = 0;
}
__global__ __launch_bounds__(kThreads) void qg_lin_counts(uint32_t* counts) { zero_counts(counts); }

// And its first half: dZ = bf16(dY act'(Z)) with each workgroup's share of dbias (from the
// unrounded dZ), a wave taking 512 columns of every fourth row of the workgroup's slab; then, in
// further workgroups, W~; and zeros for the counts of the second half's parts. Bound by bytes: 4096
// tokens through 11008 x 4096, 405 MB in 68 us, 6.0 TB/s; with few of them by latency (1000 through
// 1376 x 512: 10 MB in 8 us).
template <int ACT>
__global__ __launch_bounds__(kThreads) void qg_lin_act_dz(LinActArgs a, int64_t slab, int dz_blocks) {
  __shared__ float sh[4][512];
  if (blockIdx.x == 0 && a.counts != nullptr) zero_counts(a.counts);
  if ((int)blockIdx.x >= dz_blocks) {
    dequant_block(a, blockIdx.x - dz_blocks);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t T = a.T, m = a.m;
  const int across = (int)((m + 511) / 512), bx = blockIdx.x % across, by = blockIdx.x / across;
  const int64_t col = (int64_t)bx * 512 + 8 * lane;
  const int64_t t0 = (int64_t)by * slab, t1 = t0 + slab < T ? t0 + slab : T;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (col < m) {
#pragma unroll 4
    for (int64_t t = t0 + wave; t < t1; t += 4) {
      float d[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a.dY + t * m + col), d);
      if constexpr (ACT != kActNone) {
        float z[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(a.Zin + t * m + col), z);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= act_bwd<ACT>(z[e]);
        *reinterpret_cast<uint4*>(a.dZ + t * m + col) = pack_bf16x8(d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[e];
    }
  }
  if (a.dbias == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[wave][8 * lane + e] = sum[e];
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += kThreads) {
    const int64_t cg = (int64_t)bx * 512 + c;
    if (cg < m) a.part[by * m + cg] = (sh[0][c] + sh[1][c]) + (sh[2][c] + sh[3][c]);
  }
}

// -------------------------------------------------------------------- few tokens ---
__device__ __forceinline__ float act_fwd(int act, float z) {
  switch (act) {
    case kActRelu: return act_fwd<kActRelu>(z);
    case kActGelu: return act_fwd<kActGelu>(z);
    case kActGeluTanh: return act_fwd<kActGeluTanh>(z);
    case kActSilu: return act_fwd<kActSilu>(z);
    default: return z;
  }
}

// MR blocks of 16 weight rows x NT blocks of 16 tokens per workgroup of NW waves; the waves take
// runs of kRun chunks of 64 K values in turn. Lane l holds the codes k0 + 16 (l / 16) .. + 15 of
// weight row l % 16 (one 16-byte load) and the same K values of token l % 16, so a chunk is two
// 16 x 16 x 32 MFMAs whose K order is the lanes'. The loads of a run go out while the run before
// it is multiplied.
// One token through 11008 x 4096: 45 MB in 14.4 us of the kernel, 3.1 TB/s. A wave has four runs there
// and one of them ahead, so its first and last loads and the sum over the waves lie open; and 688
// workgroups are two on some CUs and three on others.
// SCALES: how the group scales lie. 2: n % 256 == 0, a run is one group of its row (one scale);
// 1: n % 16 == 0, a lane's 16 codes lie in one group; 0: eight codes do.
constexpr int kRun = 4;
template <int NT, int MR, int NW, int SCALES>
__global__ __launch_bounds__(64 * NW) void qg_lin_few(LinActArgs a) {
  __shared__ __attribute__((aligned(16))) float sh[NW][MR][NT][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t T = (uint32_t)a.T, m = (uint32_t)a.m, n = (uint32_t)a.n;
  const uint32_t o0 = blockIdx.x * (16 * MR);
  const rsrc_t rw = make_rsrc(a.Wq, m * n);
  const rsrc_t rs = make_rsrc(a.Ws, ((m * n + kGroup - 1) / kGroup) * 4);
  const rsrc_t rx = make_rsrc(a.X, T * n * 2);
  const uint32_t g = lane >> 4, r = lane & 15;
  f32x4 acc[MR][NT];
#pragma unroll
  for (int x = 0; x < MR; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
  constexpr int U = NT * MR > 2 ? 2 : kRun;   // chunks of a run fetched together
  constexpr int NS = SCALES == 2 ? 1 : SCALES == 1 ? U : 2 * U;
  struct Fetch {
    uint4 w[U][MR];
    float s[NS][MR];
    uint4 x[U][NT][2];
  };
  // chunks c .. c + U - 1 of this lane's rows and tokens; zeros past K
  auto fetch = [&](Fetch& f, uint32_t c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = (c + u) * 64 + 16 * g;
#pragma unroll
      for (int b = 0; b < MR; ++b) {
        const uint32_t o = o0 + 16 * b + r, e = o * n + k;
        const bool in = o < m && k < n;
        if constexpr (SCALES > 0) {
          f.w[u][b] = bload128(rw, in ? e : kOOB);
          if (SCALES == 1 || u == 0) f.s[SCALES == 1 ? u : 0][b] = bloadf(rs, in ? (e >> 8) * 4 : kOOB);
        } else {
          const bool in1 = o < m && k + 8 < n;
          const uint2 lo = bload64(rw, in ? e : kOOB), hi = bload64(rw, in1 ? e + 8 : kOOB);
          f.w[u][b] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          f.s[2 * u][b] = bloadf(rs, in ? (e >> 8) * 4 : kOOB);
          f.s[2 * u + 1][b] = bloadf(rs, in1 ? ((e + 8) >> 8) * 4 : kOOB);
        }
      }
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        const uint32_t t = 16 * y + r;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          f.x[u][y][h] = bload128(rx, t < T && k + 8 * h < n ? (t * n + k + 8 * h) * 2 : kOOB);
      }
    }
  };
  auto multiply = [&](const Fetch& f) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < MR; ++b) {
          const uint2 q = h ? make_uint2(f.w[u][b].z, f.w[u][b].w) : make_uint2(f.w[u][b].x, f.w[u][b].y);
          const float sc = f.s[SCALES == 2 ? 0 : SCALES == 1 ? u : 2 * u + h][b];
          const bf16x8 wf = __builtin_bit_cast(bf16x8, dequant8_w(q, sc));
#pragma unroll
          for (int y = 0; y < NT; ++y)
            acc[b][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wf, __builtin_bit_cast(bf16x8, f.x[u][y][h]), acc[b][y], 0, 0, 0);
        }
  };
  // fetch number i of this wave: chunk (i / PER) NW kRun + wave kRun + (i % PER) U
  constexpr int PER = kRun / U;
  auto chunk = [&](int i) { return (uint32_t)(((i / PER) * NW + wave) * kRun + (i % PER) * U); };
  const int nk = (int)((n + 63) / 64);
  const int total = (nk + NW * kRun - 1) / (NW * kRun) * PER;
  Fetch f0, f1;
  fetch(f0, chunk(0));
  for (int i = 0; i < total; i += 2) {
    fetch(f1, chunk(i + 1));
    multiply(f0);
    fetch(f0, chunk(i + 2));
    multiply(f1);
  }
#pragma unroll
  for (int b = 0; b < MR; ++b)
#pragma unroll
    for (int y = 0; y < NT; ++y)
      *reinterpret_cast<f32x4*>(&sh[wave][b][y][lane][0]) = acc[b][y];
  __syncthreads();
  // output row 4 (l / 16) + v of block b, token l % 16 of block y: one thread per lane position
  for (int q = threadIdx.x; q < MR * NT * 64; q += 64 * NW) {
    const int l = q & 63, y = (q >> 6) % NT, b = (q >> 6) / NT;
    f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int wv = 0; wv < NW; ++wv) v += *reinterpret_cast<const f32x4*>(&sh[wv][b][y][l][0]);
    const uint32_t t = 16 * y + (l & 15), o = o0 + 16 * b + 4 * (l >> 4);
    if (t >= T || o >= m) continue;
    const int64_t at = (int64_t)t * m + o;   // m is a multiple of 8: four outputs are inside
    float z[4] = {v[0], v[1], v[2], v[3]};
    if (a.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += a.bias[o + e];
    }
    if (a.Z != nullptr)
      *reinterpret_cast<uint2*>(a.Z + at) =
          make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = act_fwd(a.act, z[e]);
    if (a.res != nullptr) {
      const uint2 p = *reinterpret_cast<const uint2*>(a.res + at);
      z[0] += __uint_as_float(p.x << 16);
      z[1] += __uint_as_float(p.x & 0xFFFF0000u);
      z[2] += __uint_as_float(p.y << 16);
      z[3] += __uint_as_float(p.y & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(a.Y + at) =
        make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
  }
}

// ---------------------------------------------------------------- some tokens ---
// A 64 x 64 tile of Y straight from the codes, for token counts at which writing W~ first would
// take longer than the product: 16 waves in four groups of 2 x 2, each group with a ring of three
// stages and every fourth K stage of 64. A stage is 64 rows of X (8 KiB) as in qg_mm.hpp, 64 rows
// of codes (4 KiB; 16-byte chunk c of row r at c ^ ((r / 4) % 4)) and a scale for each of them,
// which every wave loads for itself; a wave dequantizes its fragments on their way from LDS to the
// MFMAs. The groups' sums meet in LDS. n % 64 == 0: a row's 64 codes lie in one scale group.
struct CodeStage {
  static constexpr int X_BYTES = 64 * 64 * 2, C_BYTES = 64 * 64, S_BYTES = 4 * 256;
  static constexpr int BYTES = X_BYTES + C_BYTES + S_BYTES;
  static constexpr int NI = 2 + 1 + 1;   // loads per wave and stage
};
constexpr int kCodeGroups = 4, kCodeStages = 3;

__global__ __launch_bounds__(256 * kCodeGroups) void qg_lin_codes(LinActArgs a, int tm) {
  using S = CodeStage;
  using T = MmTile<1, 1, false, false, MmBf16>;
  constexpr int KG = kCodeGroups, NST = kCodeStages;
  __shared__ __attribute__((aligned(16))) uint8_t lds[KG * NST * S::BYTES];
  static_assert(KG * 64 * 64 * 4 <= (int)sizeof(lds), "the groups' images");
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3, kg = threadIdx.x >> 8;
  const uint32_t rows = (uint32_t)a.T, m = (uint32_t)a.m, n = (uint32_t)a.n;
  const int t = xcd_remap(blockIdx.x, gridDim.x);
  const int i0 = (t % tm) * 64, j0 = (t / tm) * 64;
  const MmStage<64, false> sx(MmOperand{a.X, n, (int32_t)rows, (int32_t)n}, i0);
  // codes: rows 16 wave .. + 15 of the tile; scales: lane l's row l
  const uint32_t crow = 16 * wave + lane / 4, cg = j0 + crow, sg = j0 + lane;
  const uint32_t vc = cg < m ? cg * n + 16 * ((lane & 3) ^ ((crow >> 2) & 3)) : kOOB;
  const v4i32 rs = rsrc_words(a.Ws, ((m * n + kGroup - 1) / kGroup) * 4);
  uint8_t* area = lds + kg * NST * S::BYTES;
  const uint32_t base = lds_addr(reinterpret_cast<const uint16_t*>(area));
  auto issue = [&](int s, int buf) {
    const uint32_t k = (uint32_t)(s * KG + kg) * 64, kb = k < n ? k : n, at = base + buf * S::BYTES;
    sx.issue(k, at);
    const v4i32 rc = rsrc_words(a.Wq + kb, m * n - kb);
    dma16(rc, k < n ? vc : kOOB, at + S::X_BYTES + wave * 1024);
    dma4(rs, sg < m && k < n ? ((sg * n + k) >> 8) * 4 : kOOB,
         at + S::X_BYTES + S::C_BYTES + wave * 256);
  };
  f32x16 acc[1][1];
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[0][0][v] = 0.0f;
  const int am = (wave >> 1) * 32, bn = (wave & 1) * 32;
  const int nk = (int)((n / 64 + KG - 1) / KG);
  static_for<NST - 1>([&](auto s) { issue(decltype(s)::value, decltype(s)::value); });
  for (int k0 = 0; k0 < nk; k0 += NST) {
    static_for<NST>([&](auto bc) {
      constexpr int buf = decltype(bc)::value;
      const int kt = k0 + buf;
      if (kt < nk) {
        wait_vm_lds<(NST - 2) * S::NI>();
        barrier_nofence();
        const uint8_t* st = area + buf * S::BYTES;
        const uint8_t* codes = st + S::X_BYTES;
        const int row = bn + (lane & 31);
        // the stage's fragments and codes on their way at once (the compiler would read two, wait
        // and multiply, four times over)
        v8i16 x[4];
        uint2 q[4];
        const float sc = *reinterpret_cast<const float*>(codes + S::C_BYTES + wave * 256 + 4 * row);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          q[ks] = *reinterpret_cast<const uint2*>(codes + row * 64 + 16 * (ks ^ ((row >> 2) & 3)) +
                                                  8 * (lane >> 5));
          x[ks] = mm_frag<64, false>(reinterpret_cast<const uint16_t*>(st), am, 16 * ks);
        }
        __builtin_amdgcn_sched_barrier(0);
        issue(kt + NST - 1, (buf + NST - 1) % NST);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          acc[0][0] = MmBf16::mfma(__builtin_bit_cast(v8i16, dequant8_w(q[ks], sc)), x[ks], acc[0][0]);
      }
    });
  }
  wait_vm_lds<0>();
  __syncthreads();
  // the four groups' images, then eight outputs of a token per thread
  float* img = reinterpret_cast<float*>(lds);
  mm_put<T>(img + kg * 64 * 64, acc, am, bn);
  __syncthreads();
  const int c = threadIdx.x, r = c / 8, j = 8 * (c % 8);
  if (c >= 64 * 8 || i0 + r >= (int)rows || j0 + j >= (int)m) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < KG; ++k) {
    const float* q = img + k * 64 * 64 + r * 64 + 4 * ((j >> 2) ^ img_swz(r));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += q[e];
  }
  finish8(a, i0 + r, j0 + j, v, residual8(a, i0 + r, j0 + j),
          [&](float z) { return act_fwd(a.act, z); });
}

namespace {

// f(std::integral_constant<int, act>) for the activation of a call.
template <class F>
void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

template <int NT, int MR, int NW>
void launch_few_waves(const LinActArgs& a, int grid, hipStream_t s) {
  if (a.n % 256 == 0)
    hipLaunchKernelGGL((qg_lin_few<NT, MR, NW, 2>), dim3(grid), dim3(64 * NW), 0, s, a);
  else if (a.n % 16 == 0)
    hipLaunchKernelGGL((qg_lin_few<NT, MR, NW, 1>), dim3(grid), dim3(64 * NW), 0, s, a);
  else
    hipLaunchKernelGGL((qg_lin_few<NT, MR, NW, 0>), dim3(grid), dim3(64 * NW), 0, s, a);
}
// Enough waves to cover the memory's latency: K is cut finer where there are few weight rows.
template <int NT, int MR>
void launch_few(const LinActArgs& a, hipStream_t s) {
  const int grid = (int)((a.m + 16 * MR - 1) / (16 * MR));
  if (grid >= 512)
    launch_few_waves<NT, MR, 4>(a, grid, s);
  else
    launch_few_waves<NT, MR, 8>(a, grid, s);
}

int dequant_blocks(const LinActArgs& a) {
  return (int)((a.m * a.n / 16 + kThreads - 1) / kThreads);
}

// f(X) as an integral constant for tiles of 64 X.
template <class F>
void with_x(int x, F&& f) {
  if (x == 4)
    f(std::integral_constant<int, 4>{});
  else if (x == 2)
    f(std::integral_constant<int, 2>{});
  else
    f(std::integral_constant<int, 1>{});
}
int64_t cut(int64_t n, int64_t e) { return (n + e - 1) / e; }
int tile_for(int64_t M, int64_t N, int64_t K, double* ns = nullptr) {
  auto count = [&](int64_t e) { return cut(M, e) * cut(N, e); };
  return mm_choose(count(64), count(128), count(256), K, ns);
}
int tile_blocks(int x, int tiles) { return x == 4 ? mm_grid(tiles) : tiles; }
// The same for a product that may be cut along K.
int split_tile_for(int64_t M, int64_t N, int64_t K, int& split) {
  auto count = [&](int64_t e) { return cut(M, e) * cut(N, e); };
  return mm_choose_split(count(64), count(128), count(256), K, split);
}
int64_t parts_of(int64_t M, int64_t N, int64_t K) {
  int split;
  split_tile_for(M, N, K, split);
  return split > 1 ? cut(M, 64) * cut(N, 64) * split : 0;
}

}  // namespace

// Expected times in us, from measurements with the weights in memory (m x n; T: few, codes, tiles):
//   11008 x 4096   1: 15, 22, -   16: 22, 22, -   32: 31, 23, -   64: 48, 25, -   128: -, 44, 52
//                  256: -, 62, 66   512: -, 123, 76
//   4096 x 11008   16: 21, 48, -   32: 39, 50, -   64: 58, 55, -   128: -, 53, 68   512: -, 108, 97
//   4096 x 4096    16: 9, 21, -    64: 24, 20, -   256: -, 22, 33   512: -, 45, 39
// The formulas below follow them to about a tenth, and where two forms lie closer the slower one may be
// taken (4096 x 11008 at 512: codes, 108 for 97).
int lin_fwd_form(int64_t T, int64_t m, int64_t n) {
  const int64_t tiles = ((T + 63) / 64) * ((m + 63) / 64);
  const double weights = (double)m * (double)n * 1e-6;
  const double codes = (3.0 + 1.15 * (double)((n + 255) / 256)) * (double)((tiles + 255) / 256);
  if (T <= 64) {
    const double few = (2.0 + weights / 3.2) * (1.0 + (double)T / 28.0);
    return n % 64 == 0 && T > 16 && codes < few ? kLinCodes : kLinFew;
  }
  double ns;
  tile_for(T, m, n, &ns);
  return n % 64 == 0 && codes < 2.0 + weights / 1.5 + 1e-3 * ns ? kLinCodes : kLinTiles;
}

int64_t lin_bwd_parts(int64_t T, int64_t m, int64_t n) {
  return parts_of(T, n, m) + parts_of(m, n, T);
}

// Tokens count by blocks of 64 here. While the code tiles stay within one round of 256 their time is
// the same and that of the other form only grows (mm_choose's is monotone in the number of tiles), so
// the first block of each round decides for the round.
bool lin_fwd_tiles_up_to(int64_t T, int64_t m, int64_t n) {
  if (T <= 64) return false;
  if (n % 64 != 0 || lin_fwd_form(T, m, n) == kLinTiles) return true;
  const int64_t blocks = cut(T, 64), tm = cut(m, 64);
  for (int64_t b = 2; b < blocks; b = cut(b * tm, 256) * 256 / tm + 1)
    if (lin_fwd_form(64 * b, m, n) == kLinTiles) return true;
  return false;
}
// dX has more tiles with more tokens, G a longer inner dimension: either bound grows with T.
int64_t lin_bwd_parts_up_to(int64_t T, int64_t m, int64_t n) {
  auto most = [](int64_t M, int64_t N, int64_t K) {
    const int64_t parts = cut(M, 64) * cut(N, 64) * std::min<int64_t>(kMmMaxSplit, cut(K, kMmK));
    return std::min<int64_t>(parts, kMmParts);
  };
  const int64_t dx = 2 * cut(n, 64) <= kMmParts && m > kMmK ? most(T, n, m) : 0;
  const int64_t g = 2 * cut(m, 64) * cut(n, 64) <= kMmParts && T > kMmK ? most(m, n, T) : 0;
  return dx + g;
}

hipError_t launch_linear_act_fwd(const LinActArgs& a, hipStream_t s) {
  const int form = lin_fwd_form(a.T, a.m, a.n);
  if (form == kLinFew && a.T <= 16) {
    launch_few<1, 1>(a, s);
  } else if (form == kLinFew && a.T <= 32) {
    launch_few<2, 2>(a, s);
  } else if (form == kLinFew) {
    launch_few<4, 2>(a, s);
  } else if (form == kLinCodes) {
    const int tm = (int)((a.T + 63) / 64);
    hipLaunchKernelGGL(qg_lin_codes, dim3((unsigned)(tm * ((a.m + 63) / 64))),
                       dim3(256 * kCodeGroups), 0, s, a, tm);
  } else {
    hipLaunchKernelGGL(qg_lin_dequant, dim3((unsigned)dequant_blocks(a)), dim3(kThreads), 0, s, a);
    const int x = tile_for(a.T, a.m, a.n);
    const int tm = (int)cut(a.T, 64 * x), tn = (int)cut(a.m, 64 * x);
    const dim3 grid((unsigned)tile_blocks(x, tm * tn));
    with_act(a.act, [&](auto act) {
      with_x(x, [&](auto xc) {
        hipLaunchKernelGGL((qg_lin_act_fwd<decltype(xc)::value, decltype(act)::value>), grid,
                           dim3(kThreads), 0, s, a, tm, tn);
      });
    });
  }
  return hipGetLastError();
}

hipError_t launch_col_sum(const float* part, float* out, const float* part2, float* out2, int slabs,
                          int64_t cols, hipStream_t s) {
  hipLaunchKernelGGL(qg_col_sum, dim3((unsigned)((cols + 63) / 64), part2 != nullptr ? 2 : 1),
                     dim3(1024), 0, s, part, out, part2, out2, slabs, cols);
  return hipGetLastError();
}

hipError_t launch_linear_act_bwd(const LinActArgs& a, hipStream_t s) {
  const uint16_t* dZ = a.act == kActNone ? a.dY : a.dZ;
  // dZ, the partial sums of dbias and W~, as far as they are needed
  const int across = (int)cut(a.m, 512);
  const int dz = a.act != kActNone || a.dbias != nullptr ? across * a.slabs : 0;
  const int deq = a.dX != nullptr ? dequant_blocks(a) : 0;
  if (dz + deq > 0)
    with_act(a.act, [&](auto act) {
      hipLaunchKernelGGL(qg_lin_act_dz<decltype(act)::value>, dim3((unsigned)(dz + deq)),
                         dim3(kThreads), 0, s, a, cut(a.T, a.slabs), dz);
    });
  LinBackward b{};
  b.dx = {{dZ, a.m, (int32_t)a.T, (int32_t)a.m}, {a.Wt, a.n, (int32_t)a.m, (int32_t)a.n},
          (int)a.T, (int)a.n, (int)a.m, a.dX};
  b.g = {{dZ, a.m, (int32_t)a.T, (int32_t)a.m}, {a.X, a.n, (int32_t)a.T, (int32_t)a.n},
         (int)a.m, (int)a.n, (int)a.T, a.G};
  b.part = a.part;
  b.dbias = a.dbias;
  b.slabs = a.slabs;
  b.m = a.m;
  b.dx.split = b.g.split = 1;
  const int x1 = a.dX != nullptr ? split_tile_for(a.T, a.n, a.m, b.dx.split) : 0;
  const int x2 = a.G != nullptr ? split_tile_for(a.m, a.n, a.T, b.g.split) : 0;
  if (dz + deq == 0 && b.g.split > 1)   // G alone, without an activation
    hipLaunchKernelGGL(qg_lin_counts, dim3(1), dim3(kThreads), 0, s, a.counts);
  b.dx.parts = a.parts;
  b.g.parts = a.parts + parts_of(a.T, a.n, a.m) * (64 * 64);
  b.dx.counts = a.counts;
  b.g.counts = a.counts + kMmParts;
  const int sums = a.dbias != nullptr ? (int)cut(a.m, 64) : 0;
  auto launch = [&](int x, bool dx, bool g, int sum_blocks) {
    auto grid = [&](LinProduct& p, bool on) {
      p.tm = (int)cut(p.M, 64 * x);
      p.tn = (int)cut(p.N, 64 * x);
      p.blocks = on ? tile_blocks(x, p.tm * p.tn) * p.split : 0;
    };
    grid(b.dx, dx);
    grid(b.g, g);
    with_x(x, [&](auto xc) {
      hipLaunchKernelGGL(qg_lin_act_bwd<decltype(xc)::value>,
                         dim3((unsigned)(b.dx.blocks + b.g.blocks + sum_blocks)), dim3(kThreads), 0,
                         s, b);
    });
  };
  if (x1 == 0 && x2 == 0) {
    launch(1, false, false, sums);
  } else if (x1 == x2 || x1 == 0 || x2 == 0) {
    launch(x1 > 0 ? x1 : x2, x1 > 0, x2 > 0, sums);
  } else {   // two shapes of tile: two launches
    launch(x1, true, false, sums);
    launch(x2, false, true, 0);
  }
  return hipGetLastError();
}

}  // namespace qg
