// The orthogonalised update (Muon): per layer of weights W (m x n) and gradient G,
//   M <- mu M + G,  N = G + mu M (Nesterov) or M,
//   X_0 = N / (|N|_F + eps),  A = X X^T,  X <- a X + (b A + c A A) X   (ns_steps times),
//   W <- W - lr alpha X - lr weight_decay W, rounded stochastically into the INT8 codes.
// With p = min(m, n): A is p x p, from the rows of X when m <= n and from its columns otherwise
// (X^T X; the update is then X (b A + c A A)). X stays m x n row-major either way; only the
// order in which the products read it changes.
//
// Precision. The products run on fp16 operands with fp32 sums: |entries| of X, A and the
// polynomial B = b A + c A A stay below 2^6 for every accepted polynomial, and fp16 has three
// bits more than bf16 at the same MFMA rate. Each rounding of X puts noise into directions
// where N has next to nothing, and the iteration multiplies small singular values by a (3.44)
// every step, so an error made in X_1 arrives 141 times larger. Only the elementwise term a X
// carries it on (B is small where X is), so X is kept as fp16 hi + fp16 lo (22 bits) up to the last
// two iterates before the result: the products read hi, the epilogue's a X both. Relative error
// against 64 bits, output in bf16 (1.7e-3 from that rounding alone): 2.0e-3 on Gaussian matrices
// and on low rank over noise at 0.1 or 0.01; without lo 2.1e-3, 3.0e-3 and 1.6e-2, with bf16
// operands 1e-2, 2e-2 and 0.13.
// X_0 is N times a power of two (exact for a bf16 N); the rest of 1 / (|N|_F + eps) is applied in
// fp32 by the first products' epilogues. Where eps makes X so small that its values would leave fp16's
// range, the iterates are kept at 2^t X, and the last product takes the 2^t out again.
#include "qg_mm.hpp"

namespace qg {

constexpr float kLoScale = 2048.0f;   // lo = fp16((x - hi) * 2^11): clear of fp16's subnormals

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const f16x2 v = {(_Float16)lo, (_Float16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float f16_lo(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}
__device__ __forceinline__ float f16_hi(uint32_t w) { return f16_lo(w >> 16); }
__device__ __forceinline__ uint4 pack_f16x8(const float (&v)[8]) {
  return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                    pack_f16x2(v[6], v[7]));
}
__device__ __forceinline__ void unpack_f16x8(uint4 w, float (&v)[8]) {
  v[0] = f16_lo(w.x); v[1] = f16_hi(w.x); v[2] = f16_lo(w.y); v[3] = f16_hi(w.y);
  v[4] = f16_lo(w.z); v[5] = f16_hi(w.z); v[6] = f16_lo(w.w); v[7] = f16_hi(w.w);
}

// hi = fp16(v) and lo = fp16((v - hi) 2^11), lo from the very bits of hi: left to itself the
// compiler may round v to fp16 twice in different ways, which are two neighbours at a tie.
__device__ __forceinline__ uint4 split_f16x8(const float (&v)[8], uint4& hi) {
  hi = pack_f16x8(v);
  asm volatile("" : "+v"(hi.x), "+v"(hi.y), "+v"(hi.z), "+v"(hi.w));
  float h[8];
  unpack_f16x8(hi, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (v[i] - h[i]) * kLoScale;
  return pack_f16x8(h);
}

// Layer k's matrices in the workspace: the running X (fp16 hi and lo), the next one, A and B.
struct MuonBufs {
  uint16_t *x, *lo, *y, *ylo, *A, *B;
  float* part;   // small matrices: the slabs of A_0
};
__device__ __forceinline__ MuonBufs muon_bufs(const MuonArgs& a, int k) {
  char* p = a.ws + (size_t)k * a.layer_stride;
  MuonBufs b;
  b.x = reinterpret_cast<uint16_t*>(p + (a.cur ? a.off_x1 : a.off_x0));
  b.lo = reinterpret_cast<uint16_t*>(p + (a.cur ? a.off_lo1 : a.off_lo0));
  b.y = reinterpret_cast<uint16_t*>(p + (a.cur ? a.off_x0 : a.off_x1));
  b.ylo = reinterpret_cast<uint16_t*>(p + (a.cur ? a.off_lo0 : a.off_lo1));
  b.A = reinterpret_cast<uint16_t*>(p + a.off_a);
  b.B = reinterpret_cast<uint16_t*>(p + a.off_b);
  b.part = reinterpret_cast<float*>(p + a.off_part);
  return b;
}

// Sum over the workgroup in a fixed order (every thread gets it).
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  const double s = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  __syncthreads();
  return s;
}

// N of one element from its gradient and (already updated) momentum, one rounding per operation.
__device__ __forceinline__ float muon_n(const MuonArgs& a, float g, float m1) {
  return a.nesterov ? add_rn(g, mul_rn(a.momentum, m1)) : m1;
}

// M <- mu M + G, and the sum of the squares of N (in fp64, so that neither a gradient's smallest
// nor its largest values are lost) for each workgroup. Without a momentum N = G. Bound by its 10
// bytes an element: two matrices of 4096 x 11008 in 151 us, 6.0 TB/s.
__global__ __launch_bounds__(kThreads) void qg_muon_moment(MuonArgs a) {
  __shared__ double sh[4];
  const int k = blockIdx.y;
  const uint16_t* G = a.layer[k].G;
  float* M = a.layer[k].M;
  const int64_t numel = a.m * a.n, step = (int64_t)a.nblk * kThreads * 8;
  double sum = 0.0;
  for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; e < numel; e += step) {
    float g[8], x[8];
    if (e + 8 <= numel) {
      const uint4 w = *reinterpret_cast<const uint4*>(G + e);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[i] = (i & 1) ? __uint_as_float(ws[i >> 1] & 0xFFFF0000u) : bf16_to_f32(ws[i >> 1] & 0xFFFF);
      if (M != nullptr) {
        float4* pm = reinterpret_cast<float4*>(M + e);
        const float4 m0 = pm[0], m1 = pm[1];
        const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = add_rn(mul_rn(a.momentum, mm[i]), g[i]);
        pm[0] = make_float4(x[0], x[1], x[2], x[3]);
        pm[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    } else {
      for (int i = 0; i < 8; ++i) {
        g[i] = e + i < numel ? bf16_to_f32(G[e + i]) : 0.0f;
        x[i] = 0.0f;
        if (M != nullptr && e + i < numel) {
          x[i] = add_rn(mul_rn(a.momentum, M[e + i]), g[i]);
          M[e + i] = x[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = M != nullptr ? muon_n(a, g[i], x[i]) : g[i];
      sum += d * d;
    }
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) a.part[(int64_t)k * a.nblk + blockIdx.x] = sum;
}

// The power of two 2^e that brings a norm into [2^9, 2^10), so that N 2^e fits fp16 with room on
// both sides, and f = 1 / ((norm + eps) 2^e), 0 for a matrix of zeros. With eps >> norm, |X| starts at
// rho = norm / (norm + eps) and grows to rho `grow` at most: below 1, as much of a power of two 2^t as
// keeps 2^t X within 1 to the end, and t = 0 otherwise. (At t = 0 throughout, a norm of 1e-6 eps cost
// 2.4e-2 of the result, and one of 1e-8 eps all of it.)
__device__ __forceinline__ MuonScale muon_scale(double sum, float eps, float grow, int& e) {
  const double norm = sqrt(sum);
  e = 0;
  if (!(norm > 0.0) || isinf(norm)) {
    // zeros stay zeros; with a NaN or an infinity no direction is defined: NaN
    const float f = norm == 0.0 ? 0.0f : __uint_as_float(0x7FC00000u);
    return {f, f, 1.0f};
  }
  e = 9 - ilogb(norm);
  e = e > 126 ? 126 : (e < -126 ? -126 : e);
  const double all = norm + (double)eps, f = 1.0 / ldexp(all, e);
  int t = ilogb(all / (norm * (double)grow));
  t = t < 0 ? 0 : (t > 120 ? 120 : t);
  return {(float)f, (float)ldexp(f, t), ldexpf(1.0f, -t)};
}

// Eight values of row-major G (and M) at element `at`, `left` of them inside the row, as they lie in
// memory: rows of any length start at any element.
struct MuonRaw {
  uint4 g;
  float m[8];
  __device__ __forceinline__ void load(const uint16_t* G, const float* M, int64_t at, int64_t left) {
    if (left >= 8) {
      __builtin_memcpy(&g, G + at, 16);
      if (M != nullptr) __builtin_memcpy(m, M + at, 32);
    } else {
      uint16_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = i < left ? G[at + i] : 0;
        m[i] = M != nullptr && i < left ? M[at + i] : 0.0f;
      }
      __builtin_memcpy(&g, w, 16);
    }
  }
};

// X_0 = fp16 hi (and lo, where N is fp32) of N 2^e with rows ldx apart and zeros behind column n.
// Bound by its 10 bytes an element (two of 4096 x 11008: 180 us, 5.0 TB/s). The first values are on
// their way while the norm is summed: a workgroup of a small matrix has no others (16 of
// 1376 x 512: 22 us, 45 without).
__global__ __launch_bounds__(kThreads) void qg_muon_start(MuonArgs a) {
  __shared__ double sh[4];
  const int k = blockIdx.y;
  const uint16_t* G = a.layer[k].G;
  const float* M = a.layer[k].M;
  const uint32_t cpr = (uint32_t)(a.ldx / 8);
  const int64_t chunks = a.m * cpr, step = (int64_t)gridDim.x * kThreads;
  int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t row = 0;
  int col = 0;
  MuonRaw raw{};
  auto fetch = [&] {
    row = c / cpr;
    col = 8 * (int)(c - row * cpr);
    if (c < chunks) raw.load(G, M, row * a.n + col, a.n - col);
  };
  fetch();
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.nblk; i += kThreads) sum += a.part[(int64_t)k * a.nblk + i];
  sum = block_sum(sum, sh);
  int e;
  const MuonScale scale = muon_scale(sum, a.eps, a.grow, e);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.scal[k] = scale;
  if (blockIdx.x == 0 && k == 0)
    for (int i = threadIdx.x; i < kMmParts; i += kThreads) a.counts[i] = 0;
  const float pw = ldexpf(1.0f, e);
  const MuonBufs b = muon_bufs(a, k);
  while (c < chunks) {
    const uint32_t ws[4] = {raw.g.x, raw.g.y, raw.g.z, raw.g.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float g = (i & 1) ? __uint_as_float(ws[i >> 1] & 0xFFFF0000u) : bf16_to_f32(ws[i >> 1] & 0xFFFF);
      if (M != nullptr) g = muon_n(a, g, raw.m[i]);
      v[i] = mul_rn(g, pw);
    }
    uint4 hi;
    const uint4 lo = split_f16x8(v, hi);
    *reinterpret_cast<uint4*>(b.x + row * a.ldx + col) = hi;
    if (M != nullptr) *reinterpret_cast<uint4*>(b.lo + row * a.ldx + col) = lo;
    c += step;
    fetch();
  }
}

// Which part of the sum over K a workgroup has, of how many, and where they meet.
struct MuonPart {
  int part, split;
  float* parts;
  uint32_t* count;
};

// acc = the tile at (i0, j0) of V V^T (or V^T V, V given K-major) over K; false where another
// workgroup goes on with it.
template <class T>
__device__ __forceinline__ bool sym_product(MmOperand v, int K, int i0, int j0, const MuonPart& part,
                                            uint16_t* lds, f32x16 (&acc)[T::XM][T::XN]) {
  if (T::XM == 1 && part.split > 1) {
    const int st = (K + kMmK - 1) / kMmK, len = (st + part.split - 1) / part.split * kMmK;
    const int k0 = part.part * len;
    K = K - k0 < len ? K - k0 : len;
    v = mm_cut<T::AKM>(v, k0, K);
  }
  mm_kloop<T>(v, v, i0, j0, K, lds, acc);
  if constexpr (T::XM == 1)
    if (part.split > 1)
      return mm_join<T>(acc[0][0], part.parts, part.count, part.part, part.split, lds);
  return true;
}

// A = f^2 X X^T (or X^T X; f = 2^-t after the first step): one tile, and its mirror image where it
// lies above the diagonal.
template <class T>
__device__ __forceinline__ void gram_tile(const MuonArgs& a, int k, int i0, int j0, bool mirror,
                                          const MuonPart& part, uint16_t* lds) {
  const MuonBufs b = muon_bufs(a, k);
  const bool tall = T::AKM;
  const MmOperand x{b.x, a.ldx, (int32_t)a.m, (int32_t)a.ldx};
  f32x16 acc[T::XM][T::XN];
  if (!sym_product<T>(x, (int)(tall ? a.m : a.ldx), i0, j0, part, lds, acc)) return;
  const float f = a.first ? a.scal[k].f : a.scal[k].down;
  const float f2 = f * f;
  float* img = reinterpret_cast<float*>(lds);
  const int p = (int)a.p, ldp = (int)a.ldp;
#pragma unroll 1
  for (int pass = 0; pass < T::PASSES; ++pass) {
    mm_image<T>(img, acc, pass);
    const int ib = i0 + T::IMG_ROWS * pass;
    auto put = [&](int i, int jj, const float(&v)[8]) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = f2 * v[e];
      if (i < p && jj < ldp)
        *reinterpret_cast<uint4*>(b.A + (int64_t)i * ldp + jj) = pack_f16x8(w);
    };
    mm_rows<T, 4>(img, MmNone{},
                  [&](int r, int j, const float(&v)[8], MmNone) { put(ib + r, j0 + j, v); });
    if (mirror)
      mm_columns<T, 4>(img, [&](int r, int j, const float(&v)[8]) { put(j0 + j, ib + r, v); });
  }
}

// B = b A + c A A, likewise.
template <class T>
__device__ __forceinline__ void square_tile(const MuonArgs& a, int k, int i0, int j0, bool mirror,
                                            const MuonPart& part, uint16_t* lds) {
  const MuonBufs b = muon_bufs(a, k);
  const int p = (int)a.p, ldp = (int)a.ldp;
  const MmOperand A{b.A, ldp, p, ldp};
  f32x16 acc[T::XM][T::XN];
  if (!sym_product<T>(A, ldp, i0, j0, part, lds, acc)) return;
  float* img = reinterpret_cast<float*>(lds);
#pragma unroll 1
  for (int pass = 0; pass < T::PASSES; ++pass) {
    mm_image<T>(img, acc, pass);
    const int ib = i0 + T::IMG_ROWS * pass;
    auto put = [&](int i, int jj, const float(&v)[8]) {
      if (i < p && jj < ldp)
        *reinterpret_cast<uint4*>(b.B + (int64_t)i * ldp + jj) = pack_f16x8(v);
    };
    // A is its own mirror image, so B's is in the image once its rows are done
    mm_rows<T, 8, true>(
        img,
        [&](int r, int j) {
          return ib + r < p && j0 + j < ldp
                     ? *reinterpret_cast<const uint4*>(b.A + (int64_t)(ib + r) * ldp + j0 + j)
                     : make_uint4(0, 0, 0, 0);
        },
        [&](int r, int j, float(&v)[8], uint4 q) {
          float w[8];
          unpack_f16x8(q, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = a.b * w[e] + a.c * v[e];
          put(ib + r, j0 + j, v);
        });
    if (mirror) {
      __syncthreads();
      mm_columns<T, 4>(img, [&](int r, int j, const float(&v)[8]) { put(j0 + j, ib + r, v); });
    }
  }
}

// A tile (or a quarter of one, or a part of its sum) of the upper triangle of one layer's A or B;
// `per` tiles a layer. The parts with the same K values run side by side. Four of 4096 x 4096: A in
// 289 us, B in 304 (275 GFLOP each: 0.95 and 0.90 PFLOP/s), bound by the board's power as the
// products are; 16 of 1376 x 512: 16 and 10 us for 576 small tiles, three quarters of a round.
template <int X, bool KM, bool SQUARE>
__global__ __launch_bounds__(kThreads, (MmTile<X, X, KM, KM, MmF16>::OCC)) void qg_muon_sym(
    MuonArgs a, int per, int split) {
  using T = MmTile<X, X, KM, KM, MmF16>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS_BYTES / 2];
  MuonPart part{0, 1, nullptr, nullptr};
  auto tile = [&](auto t, int k, int ti, int tj, bool mirror) {
    using U = decltype(t);
    if constexpr (SQUARE)
      square_tile<U>(a, k, ti * U::BM, tj * U::BN, mirror, part, lds);
    else
      gram_tile<U>(a, k, ti * U::BM, tj * U::BN, mirror, part, lds);
  };
  int q = -1, ti, tj;
  int t = X > 2 ? mm_pick(blockIdx.x, a.count * per, q) : xcd_remap(blockIdx.x, gridDim.x);
  if constexpr (X == 1) {
    const int tiles = a.count * per;
    part.part = t / tiles;
    t -= part.part * tiles;
    part.split = split;
    part.parts = a.parts + (size_t)t * split * (T::BM * T::BN);
    part.count = a.counts + t;
  }
  const int k = t / per;
  mm_triangle(t - k * per, ti, tj);
  if constexpr (X > 2) {
    if (q >= 0) {
      const int si = 2 * ti + (q >> 1), sj = 2 * tj + (q & 1);
      if (si <= sj) tile(MmTile<X / 2, X / 2, KM, KM, MmF16>{}, k, si, sj, si < sj);
      return;
    }
  }
  tile(T{}, k, ti, tj, ti != tj);
}

// Eight weights of row i from column j on (j a multiple of 8) and the scales of the first and the
// last: in rows of any length the eight start at any byte and may lie in two groups. At the end
// of a row that is no multiple of 8 they are fetched and stored one by one.
struct MuonCodes {
  uint2 w;
  float s0, s1;
};
__device__ __forceinline__ MuonCodes muon_codes(const MuonArgs& a, int k, int i, int j) {
  MuonCodes c{};
  const int64_t at = (int64_t)i * a.n + j;
  const int8_t* W = a.layer[k].W + at;
  if (j + 8 <= a.n) {
    __builtin_memcpy(&c.w, W, 8);
  } else {
    for (int e = 0; j + e < a.n; ++e)
      (e < 4 ? c.w.x : c.w.y) |= (uint32_t)(uint8_t)W[e] << (8 * (e & 3));
  }
  const int64_t last = j + 8 <= a.n ? at + 7 : (int64_t)i * a.n + a.n - 1;
  c.s0 = a.layer[k].Ws[at >> 8];
  c.s1 = a.layer[k].Ws[last >> 8];
  return c;
}

// Their update: U = -(lr alpha) X, d = (W + (U / s - (lr weight_decay) W)) + u, and
// W = clamp(floor(d)) where d is finite.
__device__ __forceinline__ void muon_round8(const MuonArgs& a, int k, int i, int j,
                                            const float (&x)[8], const MuonCodes& c) {
  const uint4 h = philox4x32_10(make_uint4((uint32_t)j >> 3, (uint32_t)i, a.step,
                                           a.layer[k].layer_id), a.seed_lo, a.seed_hi);
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, w[2] = {c.w.x, c.w.y};
  const int64_t at = (int64_t)i * a.n + j;
  const int border = kGroup - (int)(at & (kGroup - 1));   // elements before the second group
  const float inv0 = recip_or_zero(c.s0), inv1 = recip_or_zero(c.s1);
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = (int)(int8_t)(w[e >> 2] >> (8 * (e & 3)));
    const float wf = (float)q;
    const float u = (float)((e & 1) ? hw[e >> 1] >> 16 : hw[e >> 1] & 0xFFFF) * 0x1p-16f;
    float t = mul_rn(mul_rn(-a.lr_alpha, x[e]), e < border ? inv0 : inv1);
    if (a.lr_decay != 0.0f) t = t - mul_rn(a.lr_decay, wf);
    const float d = add_rn(add_rn(wf, t), u);
    const int nq = isfinite(d) ? (int)fminf(fmaxf(floorf(d), -127.f), 127.f) : q;
    out[e >> 2] |= (uint32_t)(uint8_t)nq << (8 * (e & 3));
  }
  int8_t* W = a.layer[k].W + at;
  if (j + 8 <= a.n) {
    const uint2 o = make_uint2(out[0], out[1]);
    __builtin_memcpy(W, &o, 8);
  } else {
    for (int e = 0; j + e < a.n; ++e) W[e] = (int8_t)(out[e >> 2] >> (8 * (e & 3)));
  }
}

// Eight results y of row i from column j on (j < n): O in bf16, or the weights (`c`: muon_codes).
template <int OUT>
__device__ __forceinline__ void muon_emit(const MuonArgs& a, int k, int i, int j,
                                          const float (&y)[8], const MuonCodes& c) {
  if constexpr (OUT == kMuonO) {
    uint16_t* O = a.layer[k].O + (int64_t)i * a.n + j;
    const uint4 o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                               pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if (j + 8 <= a.n) {
      __builtin_memcpy(O, &o, 16);
    } else {
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
      for (int e = 0; j + e < a.n; ++e) O[e] = (uint16_t)(ow[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    muon_round8(a, k, i, j, y, c);
  }
}

// One tile of X <- f (a X + B X) (or X B for a tall X; f = 1 between the first and the last step): the
// next X as hi (and lo), or with the last product the result itself in bf16, or the weights. Four of
// 4096 x 4096: 525 us, 1.05 PFLOP/s; a 256 x 256 tile is 102 us of products at full power and 20 us of
// hi and lo read and written (512 KiB a CU at 6.7 TB/s over the chip), which no second workgroup covers:
// there is LDS for one. 16 of 1376 x 512: 30 us, half of it those bytes.
template <class T, int OUT>
__device__ __forceinline__ void update_tile(const MuonArgs& a, int k, int i0, int j0,
                                            uint16_t* lds) {
  const int m = (int)a.m, n = (int)a.n, ldx = (int)a.ldx;
  const MuonBufs b = muon_bufs(a, k);
  const uint16_t *X = b.x, *XL = b.lo;
  const MmOperand x{X, ldx, m, ldx}, B{b.B, a.ldp, (int32_t)a.p, (int32_t)a.ldp};
  f32x16 acc[T::XM][T::XN];
  if (T::BKM)
    mm_kloop<T>(B, x, i0, j0, (int)a.ldp, lds, acc);    // wide: B (m x m) X
  else
    mm_kloop<T>(x, B, i0, j0, (int)a.ldp, lds, acc);    // tall: X B (n x n)
  const float f = (a.first ? a.scal[k].fu : 1.0f) * (a.last ? a.scal[k].down : 1.0f);
  float* img = reinterpret_cast<float*>(lds);
  uint16_t *Y = b.y, *YL = b.ylo;
#pragma unroll 1
  for (int pass = 0; pass < T::PASSES; ++pass) {
    mm_image<T>(img, acc, pass);
    const int ib = i0 + T::IMG_ROWS * pass;
    struct Old {
      uint4 hi, lo;
      MuonCodes w;
    };
    auto get = [&](int r, int j) {
      const int i = ib + r, jj = j0 + j;
      Old o{};
      if (i < m && jj < ldx) {
        o.hi = *reinterpret_cast<const uint4*>(X + (int64_t)i * ldx + jj);
        if (a.lo_in) o.lo = *reinterpret_cast<const uint4*>(XL + (int64_t)i * ldx + jj);
        if (OUT == kMuonW && jj < n) o.w = muon_codes(a, k, i, jj);
      }
      return o;
    };
    mm_rows<T, 8>(img, get, [&](int r, int j, const float(&v)[8], const Old& o) {
      const int i = ib + r, jj = j0 + j;
      if (i >= m || jj >= ldx) return;
      const int64_t at = (int64_t)i * ldx + jj;
      float y[8], l[8];   // without lo its bits are zero
      unpack_f16x8(o.hi, y);
      unpack_f16x8(o.lo, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += l[e] * (1.0f / kLoScale);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f * (a.a * y[e] + v[e]);
      if constexpr (OUT == kMuonX) {
        uint4 hi;
        const uint4 lo = split_f16x8(y, hi);
        *reinterpret_cast<uint4*>(Y + at) = hi;
        if (a.lo_out) *reinterpret_cast<uint4*>(YL + at) = lo;
      } else {
        if (jj < n) muon_emit<OUT>(a, k, i, jj, y, o.w);
      }
    });
  }
}

template <int X, bool TALL, int OUT>
__global__ __launch_bounds__(kThreads, (MmTile<X, X, false, !TALL, MmF16>::OCC)) void qg_muon_update(
    MuonArgs a, int tm, int tn) {
  using T = MmTile<X, X, false, !TALL, MmF16>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS_BYTES / 2];
  const int per = tm * tn;
  int q = -1, ti, tj;
  const int t = X > 2 ? mm_pick(blockIdx.x, a.count * per, q) : xcd_remap(blockIdx.x, gridDim.x);
  const int k = t / per;
  mm_band(t - k * per, tm, tn, ti, tj);
  if constexpr (X > 2) {
    if (q >= 0) {
      using U = MmTile<X / 2, X / 2, false, !TALL, MmF16>;
      update_tile<U, OUT>(a, k, (2 * ti + (q >> 1)) * U::BM, (2 * tj + (q & 1)) * U::BN, lds);
      return;
    }
  }
  update_tile<T, OUT>(a, k, ti * T::BM, tj * T::BN, lds);
}

// ------------------------------------------------- small matrices (p <= kMuonSmall) ---
// The steps commute with each other: X_s = Q X_0 with Q = P_(s-1) ... P_0, P_k = a I + b A_k +
// c A_k A_k and A_(k+1) = P_k A_k P_k, all p x p and symmetric. For p <= 128 that chain fits one
// workgroup's LDS, and the update is five launches in place of 3 s + 2 (a launch costs the host
// 3.6 us: at 64 x 64 the time before). An error in A_k grows by a^2 = 12 with each step here, so
// the chain's operands are pairs of fp16 (hi and lo, 2^-24 of a value) and its sums fp32: as
// accurate as fp32 products, which take five times as long on these matrices.

// Five launches at 64 x 64: 2.4, 3.1, 2.7, 18 and 4 us, 35 in a row; the chain is bound by its
// dependent products (four a step). 128 x 128: the chain 57 us, against 15 launches of 5 us.

// Slab blockIdx.z of A_0 = f^2 X X^T (or X^T X) in fp32.
template <bool KM>
__global__ __launch_bounds__(kThreads, 2) void qg_muon_gram0(MuonArgs a) {
  using T = MmTile<1, 1, KM, KM, MmF16>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS_BYTES / 2];
  const int k = blockIdx.y, t = (int)((a.p + 63) / 64);
  const int i0 = (int)(blockIdx.x / t) * 64, j0 = (int)(blockIdx.x % t) * 64;
  const MuonBufs b = muon_bufs(a, k);
  // K values [k0, k1) of the slab: whole stages
  const int K = (int)(KM ? a.m : a.ldx);
  const int slab = (K + 64 * a.slabs - 1) / (64 * a.slabs) * 64;
  const int k0 = (int)blockIdx.z * slab, k1 = k0 + slab < K ? k0 + slab : K;
  f32x16 acc[1][1] = {}, low[1][1] = {};
  if (k0 < k1) {
    // the slab as a matrix of its own
    auto part = [&](const uint16_t* p) {
      return KM ? MmOperand{p + (int64_t)k0 * a.ldx, a.ldx, k1 - k0, (int32_t)a.ldx}
                : MmOperand{p + k0, a.ldx, (int32_t)a.m, k1 - k0};
    };
    const MmOperand x = part(b.x);
    mm_kloop<T>(x, x, i0, j0, k1 - k0, lds, acc);
    if (a.lo_in) {
      f32x16 two[1][1];
      const MmOperand l = part(b.lo);
      mm_kloop<T>(x, l, i0, j0, k1 - k0, lds, low);
      mm_kloop<T>(l, x, i0, j0, k1 - k0, lds, two);
#pragma unroll
      for (int v = 0; v < 16; ++v) low[0][0][v] += two[0][0][v];
    }
  }
  const float f = a.scal[k].f;
#pragma unroll
  for (int v = 0; v < 16; ++v)
    acc[0][0][v] = f * f * (acc[0][0][v] + low[0][0][v] * (1.0f / kLoScale));
  float* img = reinterpret_cast<float*>(lds);
  mm_image<T>(img, acc, 0);
  float* out = b.part + (int64_t)blockIdx.z * a.p * a.ldp;
  mm_rows<T, 2>(img, MmNone{}, [&](int r, int j, const float(&v)[8], MmNone) {
    if (i0 + r >= a.p || j0 + j >= a.ldp) return;
    float* q = out + (int64_t)(i0 + r) * a.ldp + j0 + j;
    *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
  });
}

// A matrix of edge PP (64 or 128) in LDS as fp16 pairs, rows with permuted 16-byte chunks so that
// the fragments of 16 consecutive rows fall on distinct banks. A workgroup of (PP / 32)^2 waves
// works on it, each on one 32 x 32 block: element v of a wave's f32x16 is row am + lane % 32 and
// column bn + 8 (v / 4) + 4 (lane / 32) + v % 4. (128 x 128 on four waves of 64 x 64 had nothing to
// hide its LDS reads behind: 5.3 us a product against 2.)
template <int PP>
struct ChainMat {
  uint16_t *hi, *lo;
  static __device__ __forceinline__ int at(int row, int col) {
    const int c = PP == 128 ? (col >> 3) ^ (row & 15) : (col >> 3) ^ ((row >> 1) & 7);
    return row * PP + 8 * c + (col & 7);
  }
  __device__ __forceinline__ void put(const f32x16& v, int am, int bn) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = at(am + (lane & 31), bn + 8 * q + 4 * (lane >> 5));
      uint2 h = make_uint2(pack_f16x2(v[4 * q], v[4 * q + 1]),
                           pack_f16x2(v[4 * q + 2], v[4 * q + 3]));
      asm volatile("" : "+v"(h.x), "+v"(h.y));   // lo from these bits, as in split_f16x8
      *reinterpret_cast<uint2*>(hi + o) = h;
      *reinterpret_cast<uint2*>(lo + o) =
          make_uint2(pack_f16x2((v[4 * q] - f16_lo(h.x)) * kLoScale,
                                (v[4 * q + 1] - f16_hi(h.x)) * kLoScale),
                     pack_f16x2((v[4 * q + 2] - f16_lo(h.y)) * kLoScale,
                                (v[4 * q + 3] - f16_hi(h.y)) * kLoScale));
    }
  }
  __device__ __forceinline__ float get(int row, int col) const {
    const int o = at(row, col);
    return f16_lo(hi[o]) + f16_lo(lo[o]) * (1.0f / kLoScale);
  }
  __device__ __forceinline__ v8i16 frag(const uint16_t* m, int row0, int ks) const {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const v8i16*>(m + at(row0 + (lane & 31), ks + 8 * (lane >> 5)));
  }
};
// The wave's block of L R for a symmetric R (its rows serve as its columns).
template <int PP>
__device__ __forceinline__ f32x16 chain_product(const ChainMat<PP>& L, const ChainMat<PP>& R, int am,
                                                int bn) {
  f32x16 out = {}, low = {};
#pragma unroll 4
  for (int ks = 0; ks < PP; ks += 16) {
    const v8i16 ah = L.frag(L.hi, am, ks), al = L.frag(L.lo, am, ks);
    const v8i16 bh = R.frag(R.hi, bn, ks), bl = R.frag(R.lo, bn, ks);
    out = MmF16::mfma(bh, ah, out);
    low = MmF16::mfma(bl, ah, low);
    low = MmF16::mfma(bh, al, low);
  }
#pragma unroll
  for (int v = 0; v < 16; ++v) out[v] += low[v] * (1.0f / kLoScale);
  return out;
}

// Q of one layer, from the slabs of A_0, to the layer's A (hi) and B (lo).
template <int PP>
__global__ __launch_bounds__(PP * PP / 16) void qg_muon_chain(MuonArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * PP * PP];
  const ChainMat<PP> U{lds, lds + PP * PP}, V{lds + 2 * PP * PP, lds + 3 * PP * PP};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int am = wave / (PP / 32) * 32, bn = wave % (PP / 32) * 32;
  const int k = blockIdx.x, p = (int)a.p, ldp = (int)a.ldp;
  const MuonBufs b = muon_bufs(a, k);
  const int i = am + (lane & 31), j0 = bn + 4 * (lane >> 5);   // element v: column j0 + col(v)
  auto col = [](int v) { return 8 * (v >> 2) + (v & 3); };
  f32x16 A = {}, Q = {};
  for (int l = 0; l < a.slabs; ++l)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i < p && j0 + 8 * q < ldp) {
        const float4 t = *reinterpret_cast<const float4*>(b.part + ((int64_t)l * p + i) * ldp + j0 +
                                                          8 * q);
        A[4 * q] += t.x;
        A[4 * q + 1] += t.y;
        A[4 * q + 2] += t.z;
        A[4 * q + 3] += t.w;
      }
  U.put(A, am, bn);
  __syncthreads();
#pragma unroll 1
  for (int it = 0; it < a.ns_steps; ++it) {
    const bool last = it + 1 == a.ns_steps;
    f32x16 P = chain_product<PP>(U, U, am, bn);
#pragma unroll
    for (int v = 0; v < 16; ++v)
      P[v] = (i == j0 + col(v) ? a.a : 0.0f) + (a.b * A[v] + a.c * P[v]);
    V.put(P, am, bn);
    __syncthreads();
    if (!last) A = chain_product<PP>(U, V, am, bn);   // A P
    if (it == 0) {
      Q = P;
    } else {
      __syncthreads();
      U.put(Q, am, bn);
      __syncthreads();
      Q = chain_product<PP>(U, V, am, bn);
    }
    if (last) break;
    __syncthreads();
    U.put(A, am, bn);
    __syncthreads();
    A = chain_product<PP>(U, V, am, bn);   // P A P
    __syncthreads();
    U.put(A, am, bn);
    __syncthreads();
    // rounded, it is no longer symmetric, and the products above would take it for its transpose:
    // what is not symmetric in it grows by 22 with each step (0.3 of the result after five, for
    // one strong direction over noise at 0.01), so it is taken out
#pragma unroll
    for (int v = 0; v < 16; ++v) A[v] = 0.5f * (A[v] + U.get(j0 + col(v), i));
    __syncthreads();
    U.put(A, am, bn);
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = j0 + 8 * q;
    if (i >= p || j >= ldp) continue;
    uint2 h = make_uint2(pack_f16x2(Q[4 * q], Q[4 * q + 1]), pack_f16x2(Q[4 * q + 2], Q[4 * q + 3]));
    asm volatile("" : "+v"(h.x), "+v"(h.y));
    *reinterpret_cast<uint2*>(b.A + (int64_t)i * ldp + j) = h;
    *reinterpret_cast<uint2*>(b.B + (int64_t)i * ldp + j) =
        make_uint2(pack_f16x2((Q[4 * q] - f16_lo(h.x)) * kLoScale,
                              (Q[4 * q + 1] - f16_hi(h.x)) * kLoScale),
                   pack_f16x2((Q[4 * q + 2] - f16_lo(h.y)) * kLoScale,
                              (Q[4 * q + 3] - f16_hi(h.y)) * kLoScale));
  }
}

// One 64 x 64 tile of f Q X (or f X Q), both as pairs.
template <bool TALL, int OUT>
__global__ __launch_bounds__(kThreads, 2) void qg_muon_apply(MuonArgs a, int tn) {
  using T = MmTile<1, 1, false, !TALL, MmF16>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[T::LDS_BYTES / 2];
  const int k = blockIdx.y, i0 = (int)(blockIdx.x / tn) * 64, j0 = (int)(blockIdx.x % tn) * 64;
  const MuonBufs b = muon_bufs(a, k);
  const int m = (int)a.m, n = (int)a.n, ldx = (int)a.ldx, ldp = (int)a.ldp;
  const MmOperand x{b.x, ldx, m, ldx}, xl{b.lo, ldx, m, ldx};
  const MmOperand q{b.A, ldp, (int32_t)a.p, ldp}, ql{b.B, ldp, (int32_t)a.p, ldp};
  f32x16 acc[1][1], low[1][1], two[1][1] = {};
  auto product = [&](const MmOperand& Q, const MmOperand& X, f32x16(&out)[1][1]) {
    if (TALL)
      mm_kloop<T>(X, Q, i0, j0, ldp, lds, out);
    else
      mm_kloop<T>(Q, X, i0, j0, ldp, lds, out);
  };
  product(q, x, acc);
  product(ql, x, low);
  if (a.lo_in) product(q, xl, two);
#pragma unroll
  for (int v = 0; v < 16; ++v)
    acc[0][0][v] += (low[0][0][v] + two[0][0][v]) * (1.0f / kLoScale);
  const float f = a.scal[k].f;
  float* img = reinterpret_cast<float*>(lds);
  mm_image<T>(img, acc, 0);
  mm_rows<T, 2>(
      img,
      [&](int r, int j) {
        MuonCodes c{};
        if (OUT == kMuonW && i0 + r < m && j0 + j < n) c = muon_codes(a, k, i0 + r, j0 + j);
        return c;
      },
      [&](int r, int j, const float(&v)[8], const MuonCodes& c) {
        if (i0 + r >= m || j0 + j >= n) return;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = f * v[e];
        muon_emit<OUT>(a, k, i0 + r, j0 + j, y, c);
      });
}

namespace {

int cut(int64_t n, int e) { return (int)((n + e - 1) / e); }

// f(X) for the tile (64 X) that a launch takes.
template <class F>
void with_tile(int x, F&& f) {
  switch (x) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
}
template <int X>
dim3 blocks(int tiles) { return dim3((unsigned)(X > 2 ? mm_grid(tiles) : tiles)); }

template <bool KM, bool SQUARE>
void launch_sym(const MuonArgs& a, int64_t K, hipStream_t s) {
  auto tiles = [&](int e) {
    const int64_t t = cut(a.p, e);
    return t * (t + 1) / 2;
  };
  const int64_t t1 = a.count * tiles(64), t2 = a.count * tiles(128), t4 = a.count * tiles(256);
  int split = 1;
  const int x = a.parts != nullptr ? mm_choose_split(t1, t2, t4, K, split) : mm_choose(t1, t2, t4, K);
  with_tile(x, [&](auto xc) {
    constexpr int X = decltype(xc)::value;
    const int per = (int)tiles(64 * X);
    hipLaunchKernelGGL((qg_muon_sym<X, KM, SQUARE>), blocks<X>(a.count * per * split),
                       dim3(kThreads), 0, s, a, per, split);
  });
}

template <bool TALL, int OUT>
void launch_update(const MuonArgs& a, hipStream_t s) {
  auto tiles = [&](int e) { return (int64_t)cut(a.m, e) * cut(a.n, e); };
  const int x = mm_choose(a.count * tiles(64), a.count * tiles(128), a.count * tiles(256), a.ldp);
  with_tile(x, [&](auto xc) {
    constexpr int X = decltype(xc)::value;
    const int tm = cut(a.m, 64 * X), tn = cut(a.n, 64 * X);
    hipLaunchKernelGGL((qg_muon_update<X, TALL, OUT>), blocks<X>(a.count * tm * tn),
                       dim3(kThreads), 0, s, a, tm, tn);
  });
}

template <bool TALL>
hipError_t muon_iterations(MuonArgs& a, hipStream_t s) {
  for (int it = 0; it < a.ns_steps; ++it) {
    a.cur = it & 1;
    a.first = it == 0;
    a.last = it + 1 == a.ns_steps;
    a.lo_in = it == 0 ? a.layer[0].M != nullptr : it <= a.ns_steps - kMuonPlain;
    a.lo_out = it + 1 <= a.ns_steps - kMuonPlain;
    launch_sym<TALL, false>(a, TALL ? a.m : a.ldx, s);
    launch_sym<false, true>(a, a.ldp, s);
    if (it + 1 < a.ns_steps)
      launch_update<TALL, kMuonX>(a, s);
    else if (a.layer[0].O != nullptr)
      launch_update<TALL, kMuonO>(a, s);
    else
      launch_update<TALL, kMuonW>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool TALL>
hipError_t muon_small(MuonArgs& a, hipStream_t s) {
  a.lo_in = a.layer[0].M != nullptr;
  const int t = cut(a.p, 64), tm = cut(a.m, 64), tn = cut(a.n, 64);
  hipLaunchKernelGGL(qg_muon_gram0<TALL>, dim3(t * t, a.count, a.slabs), dim3(kThreads), 0, s, a);
  if (t == 1)
    hipLaunchKernelGGL(qg_muon_chain<64>, dim3(a.count), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(qg_muon_chain<128>, dim3(a.count), dim3(1024), 0, s, a);
  if (a.layer[0].O != nullptr)
    hipLaunchKernelGGL((qg_muon_apply<TALL, kMuonO>), dim3(tm * tn, a.count), dim3(kThreads), 0, s, a,
                       tn);
  else
    hipLaunchKernelGGL((qg_muon_apply<TALL, kMuonW>), dim3(tm * tn, a.count), dim3(kThreads), 0, s, a,
                       tn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon(MuonArgs& a, hipStream_t s) {
  a.cur = 0;
  hipLaunchKernelGGL(qg_muon_moment, dim3(a.nblk, a.count), dim3(kThreads), 0, s, a);
  const int64_t chunks = a.m * (a.ldx / 8);
  const int64_t blocks = (chunks + kThreads - 1) / kThreads;
  const int grid = (int)(blocks < 2048 ? blocks : 2048);
  hipLaunchKernelGGL(qg_muon_start, dim3(grid, a.count), dim3(kThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.small) return a.m > a.n ? muon_small<true>(a, s) : muon_small<false>(a, s);
  return a.m > a.n ? muon_iterations<true>(a, s) : muon_iterations<false>(a, s);
}

}  // namespace qg
