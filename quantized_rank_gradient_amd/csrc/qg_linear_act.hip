// A linear layer on INT8 weights with its bias, activation and residual in the product's epilogue,
// and its backward pass:
//   Z = X W~^T + bias,  Y = act(Z) + residual                    (W~ = bf16(q s), m x n)
//   dZ = dY act'(Z),  dbias = sum_t dZ,  dX = dZ W~,  G = dZ^T X
// Z is kept in bf16 when the backward pass will ask for it (its rounding moves act' by at most
// |act''| 2^-8 |Z|); the activation itself takes the fp32 Z.
//
// Few tokens (T <= kLinFewTokens): the time is the weights' bytes. A workgroup takes 16 or 32
// weight rows whole, its waves split K, and every code goes from memory to registers once, is
// dequantized there and multiplied by 16 tokens per MFMA; the partial sums meet in LDS.
// Many tokens: the products of qg_mm.hpp, on W~ written to the workspace by one pass (2 bytes
// written and read per weight, small against 2 T operations on it).
#include "qg_mm.hpp"
#include "qg_kernels.hpp"

namespace qg {

// ------------------------------------------------------------------- activations ---
// Phi(z), and e = exp(-z^2 / 2): Phi(-x) = e g(x) for x >= 0, with g(x) exp(-x^2/2) exp(x^2/2)
// smooth in t = 1 / (1 + 0.315 x): t times a polynomial of degree 7 in t, fitted here for the
// least relative error over 0 <= x <= 40 (3.8e-7; 1.1e-6 in fp32 down to z = -5), so that the left
// tail keeps its relative accuracy. About 16 instructions; the library's erfcf took 30 us of a
// round of 256 x 256 tiles (of 130).
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
// Past 40 every derivative here is 0 or 1 to the last bit; stopping there keeps z^2 and z^3 finite.
template <int ACT>
__device__ __forceinline__ float act_bwd(float z) {
  if constexpr (ACT != kActRelu) z = z > 40.0f ? 40.0f : (z < -40.0f ? -40.0f : z);
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
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = mul_rn((float)(int8_t)(w.x >> (8 * e)), s);
    f[4 + e] = mul_rn((float)(int8_t)(w.y >> (8 * e)), s);
  }
  return pack_bf16x8(f);
}

// W~ of the whole weight, 16 codes (one scale group) per thread; numel a multiple of 8.
__global__ __launch_bounds__(kThreads) void qg_lin_dequant(const int8_t* Wq, const float* Ws,
                                                          int64_t numel, uint16_t* out) {
  const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16;
  if (e >= numel) return;
  const float s = Ws[e >> 8];
  if (e + 16 <= numel) {
    const uint4 w = *reinterpret_cast<const uint4*>(Wq + e);
    *reinterpret_cast<uint4*>(out + e) = dequant8_w(make_uint2(w.x, w.y), s);
    *reinterpret_cast<uint4*>(out + e + 8) = dequant8_w(make_uint2(w.z, w.w), s);
  } else {
    *reinterpret_cast<uint4*>(out + e) = dequant8_w(*reinterpret_cast<const uint2*>(Wq + e), s);
  }
}

// ------------------------------------------------------------------ many tokens ---
// One tile of Y (rows: tokens, columns: outputs).
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
    auto get = [&](int r, int j) {   // the residual
      const int i = ib + r, jj = j0 + j;
      return a.res != nullptr && i < rows && jj < m
                 ? *reinterpret_cast<const uint4*>(a.res + (int64_t)i * m + jj)
                 : make_uint4(0, 0, 0, 0);
    };
    mm_rows<T, 8>(img, get, [&](int r, int j, const float(&v)[8], uint4 res) {
      const int i = ib + r, jj = j0 + j;
      if (i >= rows || jj >= m) return;
      const int64_t at = (int64_t)i * m + jj;
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = v[e];
      if (a.bias != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += a.bias[jj + e];
      }
      if (a.Z != nullptr) *reinterpret_cast<uint4*>(a.Z + at) = pack_bf16x8(z);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = act_fwd<ACT>(z[e]);
      if (a.res != nullptr) {
        float q[8];
        unpack_bf16x8(res, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += q[e];
      }
      *reinterpret_cast<uint4*>(a.Y + at) = pack_bf16x8(z);
    });
  }
}

// One tile of out (M x N bf16, row-major) = A B^T, for dX (A = dZ by rows, B = W~ by columns) and G
// (A = dZ by columns, B = X by columns).
struct LinProduct {
  MmOperand A, B;
  int M, N, K;
  uint16_t* out;
};
template <class T>
__device__ __forceinline__ void product_tile(const LinProduct& p, int i0, int j0, uint16_t* lds) {
  f32x16 acc[T::XM][T::XN];
  mm_kloop<T>(p.A, p.B, i0, j0, p.K, lds, acc);
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

// f(tile type, i0, j0) for this workgroup's tile, or quarter of one, of a tm x tn grid of tiles.
template <int X, bool AKM, bool BKM, class F>
__device__ __forceinline__ void lin_tile(int tm, int tn, F&& f) {
  int q = -1, ti, tj;
  const int t = X > 2 ? mm_pick(tm * tn, q) : xcd_remap(blockIdx.x, gridDim.x);
  mm_band(t, tm, tn, ti, tj);
  if constexpr (X > 2) {
    if (q >= 0) {
      using U = MmTile<X / 2, X / 2, AKM, BKM, MmBf16>;
      f(U{}, (2 * ti + (q >> 1)) * U::BM, (2 * tj + (q & 1)) * U::BN);
      return;
    }
  }
  using T = MmTile<X, X, AKM, BKM, MmBf16>;
  f(T{}, ti * T::BM, tj * T::BN);
}

template <int X, int ACT>
__global__ __launch_bounds__(kThreads, X > 2 ? 1 : X > 1 ? 2 : 3) void qg_lin_act_fwd(LinActArgs a, int tm,
                                                                         int tn) {
  __shared__ __attribute__((
      aligned(16))) uint16_t lds[MmTile<X, X, false, false, MmBf16>::LDS_BYTES / 2];
  lin_tile<X, false, false>(tm, tn, [&](auto t, int i0, int j0) {
    fwd_tile<decltype(t), ACT>(a, i0, j0, lds);
  });
}
template <int X, bool AKM, bool BKM>
__global__ __launch_bounds__(kThreads, X > 2 ? 1 : X > 1 ? 2 : 3) void qg_lin_act_bwd(LinProduct p, int tm,
                                                                         int tn) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[MmTile<X, X, AKM, BKM, MmBf16>::LDS_BYTES / 2];
  lin_tile<X, AKM, BKM>(tm, tn, [&](auto t, int i0, int j0) {
    product_tile<decltype(t)>(p, i0, j0, lds);
  });
}

// dZ = bf16(dY act'(Z)) and each workgroup's share of dbias (from the unrounded dZ): a wave takes
// 512 columns of every fourth row of the workgroup's slab.
template <int ACT>
__global__ __launch_bounds__(kThreads) void qg_lin_act_dz(const uint16_t* dY, const uint16_t* Z,
                                                         int64_t T, int64_t m, int64_t slab,
                                                         uint16_t* dZ, float* part) {
  __shared__ float sh[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 512 + 8 * lane;
  const int64_t t0 = (int64_t)blockIdx.y * slab, t1 = t0 + slab < T ? t0 + slab : T;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (col < m) {
#pragma unroll 4
    for (int64_t t = t0 + wave; t < t1; t += 4) {
      float d[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(dY + t * m + col), d);
      if constexpr (ACT != kActNone) {
        float z[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(Z + t * m + col), z);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= act_bwd<ACT>(z[e]);
        *reinterpret_cast<uint4*>(dZ + t * m + col) = pack_bf16x8(d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[e];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[wave][8 * lane + e] = sum[e];
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += kThreads) {
    const int64_t cg = (int64_t)blockIdx.x * 512 + c;
    if (cg < m) part[blockIdx.y * m + cg] = (sh[0][c] + sh[1][c]) + (sh[2][c] + sh[3][c]);
  }
}

// out[c] = sum of part[s][c] over s, always in the same order: 64 columns a workgroup, its 16 waves
// every sixteenth row each.
__global__ __launch_bounds__(1024) void qg_col_sum(const float* part, float* out,
                                                   const float* part2, float* out2, int slabs,
                                                   int64_t cols) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const float* p = blockIdx.y ? part2 : part;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int k = wave; k < slabs; k += 16) s += p[k * cols + c];
  }
  sh[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += sh[w][lane];
    (blockIdx.y ? out2 : out)[c] = t;
  }
}

// -------------------------------------------------------------------- few tokens ---
// MR blocks of 16 weight rows x NT blocks of 16 tokens per workgroup of NW waves; the waves take
// the K chunks of 64 in turn. Lane l holds the codes k0 + 16 (l / 16) .. + 15 of weight row l % 16
// (one 16-byte load) and the same K values of token l % 16, so a chunk is two 16 x 16 x 32 MFMAs
// whose K order is the lanes'. RUN16 (n % 16 == 0): a row's 16 codes lie in one scale group.
template <int NT, int MR, int NW, bool RUN16, int ACT>
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
  constexpr int U = NT * MR > 4 ? 2 : 4;   // chunks in flight
  const int nk = (int)((n + 63) / 64);
  for (int c0 = wave; c0 < nk; c0 += NW * U) {
    uint2 w[U][MR][2];
    float s[U][MR][2];
    uint4 x[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = (uint32_t)(c0 + u * NW) * 64 + 16 * g;
#pragma unroll
      for (int b = 0; b < MR; ++b) {
        const uint32_t o = o0 + 16 * b + r, e = o * n + k;
        const bool in = o < m && k < n;
        if constexpr (RUN16) {
          const uint4 q = bload128(rw, in ? e : kOOB);
          w[u][b][0] = make_uint2(q.x, q.y);
          w[u][b][1] = make_uint2(q.z, q.w);
          s[u][b][0] = s[u][b][1] = bloadf(rs, in ? (e >> 8) * 4 : kOOB);
        } else {
          const bool in1 = o < m && k + 8 < n;
          w[u][b][0] = bload64(rw, in ? e : kOOB);
          w[u][b][1] = bload64(rw, in1 ? e + 8 : kOOB);
          s[u][b][0] = bloadf(rs, in ? (e >> 8) * 4 : kOOB);
          s[u][b][1] = bloadf(rs, in1 ? ((e + 8) >> 8) * 4 : kOOB);
        }
      }
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        const uint32_t t = 16 * y + r;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[u][y][h] = bload128(rx, t < T && k + 8 * h < n ? (t * n + k + 8 * h) * 2 : kOOB);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < MR; ++b) {
          const bf16x8 wf = __builtin_bit_cast(bf16x8, dequant8_w(w[u][b][h], s[u][b][h]));
#pragma unroll
          for (int y = 0; y < NT; ++y)
            acc[b][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wf, __builtin_bit_cast(bf16x8, x[u][y][h]), acc[b][y], 0, 0, 0);
        }
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
    for (int e = 0; e < 4; ++e) z[e] = act_fwd<ACT>(z[e]);
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
void launch_few(const LinActArgs& a, hipStream_t s) {
  const int grid = (int)((a.m + 16 * MR - 1) / (16 * MR));
  with_act(a.act, [&](auto act) {
    if (a.n % 16 == 0)
      hipLaunchKernelGGL((qg_lin_few<NT, MR, NW, true, decltype(act)::value>), dim3(grid),
                         dim3(64 * NW), 0, s, a);
    else
      hipLaunchKernelGGL((qg_lin_few<NT, MR, NW, false, decltype(act)::value>), dim3(grid),
                         dim3(64 * NW), 0, s, a);
  });
}

hipError_t launch_dequant_weight(const LinActArgs& a, hipStream_t s) {
  const int64_t threads = (a.m * a.n + 15) / 16;
  hipLaunchKernelGGL(qg_lin_dequant, dim3((unsigned)((threads + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, s, a.Wq, a.Ws, a.m * a.n, a.Wt);
  return hipGetLastError();
}

// f(X, grid, tm, tn) with tiles of 64 X for an M x N output of depth K.
template <class F>
void with_tiles(int64_t M, int64_t N, int64_t K, F&& f) {
  auto cut = [](int64_t n, int e) { return (n + e - 1) / e; };
  auto count = [&](int e) { return cut(M, e) * cut(N, e); };
  const int x = mm_choose(count(64), count(128), count(256), K);
  const int tm = (int)cut(M, 64 * x), tn = (int)cut(N, 64 * x);
  if (x == 4)
    f(std::integral_constant<int, 4>{}, mm_grid(tm * tn), tm, tn);
  else if (x == 2)
    f(std::integral_constant<int, 2>{}, tm * tn, tm, tn);
  else
    f(std::integral_constant<int, 1>{}, tm * tn, tm, tn);
}

template <bool AKM, bool BKM>
void launch_product(const LinProduct& p, hipStream_t s) {
  with_tiles(p.M, p.N, p.K, [&](auto x, int grid, int tm, int tn) {
    hipLaunchKernelGGL((qg_lin_act_bwd<decltype(x)::value, AKM, BKM>), dim3((unsigned)grid),
                       dim3(kThreads), 0, s, p, tm, tn);
  });
}

}  // namespace

hipError_t launch_linear_act_fwd(const LinActArgs& a, hipStream_t s) {
  if (a.T <= 16) {
    launch_few<1, 1, 4>(a, s);
  } else if (a.T <= 32) {
    launch_few<2, 2, 4>(a, s);
  } else if (a.T <= kLinFewTokens) {
    launch_few<4, 2, 4>(a, s);
  } else {
    const hipError_t e = launch_dequant_weight(a, s);
    if (e != hipSuccess) return e;
    with_act(a.act, [&](auto act) {
      with_tiles(a.T, a.m, a.n, [&](auto x, int grid, int tm, int tn) {
        hipLaunchKernelGGL((qg_lin_act_fwd<decltype(x)::value, decltype(act)::value>),
                           dim3((unsigned)grid), dim3(kThreads), 0, s, a, tm, tn);
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
  if (a.act != kActNone || a.dbias != nullptr) {
    const dim3 grid((unsigned)((a.m + 511) / 512), (unsigned)a.slabs);
    const int64_t slab = (a.T + a.slabs - 1) / a.slabs;
    with_act(a.act, [&](auto act) {
      hipLaunchKernelGGL(qg_lin_act_dz<decltype(act)::value>, grid, dim3(kThreads), 0, s, a.dY,
                         a.Zin, a.T, a.m, slab, a.dZ, a.dbias != nullptr ? a.part : nullptr);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.dbias != nullptr && (e = launch_col_sum(a.part, a.dbias, nullptr, nullptr, a.slabs, a.m, s)) != hipSuccess)
      return e;
  }
  if (a.dX != nullptr) {
    const hipError_t e = launch_dequant_weight(a, s);
    if (e != hipSuccess) return e;
    launch_product<false, true>({{dZ, a.m, (int32_t)a.T, (int32_t)a.m},
                                 {a.Wt, a.n, (int32_t)a.m, (int32_t)a.n},
                                 (int)a.T, (int)a.n, (int)a.m, a.dX}, s);
  }
  if (a.G != nullptr)
    launch_product<true, true>({{dZ, a.m, (int32_t)a.T, (int32_t)a.m},
                                {a.X, a.n, (int32_t)a.T, (int32_t)a.n},
                                (int)a.m, (int)a.n, (int)a.T, a.G}, s);
  return hipGetLastError();
}

}  // namespace qg
