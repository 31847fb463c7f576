// FP8 codes of a matrix with one fp32 scale for each run of 128 values along a row (Q), along a column (Qt,
// the transpose) or for each block of 128 x 128 (both), and the way back. One read of the matrix serves both
// orders. Bytes bound it: 2 in and 1 out (or 2) for each bf16 value.
#include <type_traits>

#include "qg_fp8.hpp"
#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

namespace {

// Eight values of row `row` from column c on; zeros behind the row's end and the last row.
template <int SRC>
__device__ __forceinline__ void f8_load(const F8Quant& a, int64_t row, int64_t c, float (&v)[8]) {
  const int left = row < a.rows && c < a.cols ? (int)(a.cols - c < 8 ? a.cols - c : 8) : 0;
  if constexpr (SRC != kF8FromInt8) {
    RowRaw<SRC == kF8FromBf16> x{};
    if (left > 0) x.load(a.src, row * a.cols + c, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x.get(i);
  } else {
    uint64_t w = 0;
    const int64_t e = row * a.cols + c;
    float s0 = 0.0f, s1 = 0.0f;
    if (left > 0) {
      const uint8_t* q = static_cast<const uint8_t*>(a.src) + e;
      if (left >= 8) {
        __builtin_memcpy(&w, q, 8);
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < left) w |= (uint64_t)q[i] << (8 * i);
      }
      s0 = a.src_scale[e >> 8];
      s1 = a.src_scale[(e + left - 1) >> 8];   // eight codes lie in two groups at most
    }
    const int here = kGroup - (int)(e & (kGroup - 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(w >> (8 * i)) * (i < here ? s0 : s1);
  }
}

}  // namespace

// A tile of 128 x 128: thread (rg, cg) has rows 8 rg .. 8 rg + 7 and columns 8 cg .. 8 cg + 7, rg = its row
// of 16 lanes, so that a load takes whole lines and eight codes of a row or of a column leave together.
// The transposed codes go through LDS, to leave as lines too.
template <int FMT, int SRC>
__global__ __launch_bounds__(kThreads) void qg_f8_quantize(F8Quant a, int cb) {
  constexpr int PITCH = kF8Block + 8;   // of a column in LDS
  __shared__ alignas(16) uint8_t tile[kF8Block * PITCH];
  __shared__ float colmax[16][kF8Block];
  __shared__ float colinv[kF8Block];
  const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15;
  const int64_t bj = blockIdx.x % cb, bi = blockIdx.x / cb;
  const int64_t r0 = bi * kF8Block + 8 * rg, c0 = bj * kF8Block + 8 * cg;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f8_load<SRC>(a, r0 + i, c0, x[i]);
  float rmax[8], cmax[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) rmax[k] = cmax[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float m = fabsf(x[i][k]);
      rmax[i] = fmaxf(rmax[i], m);
      cmax[k] = fmaxf(cmax[k], m);
    }
  float sblock = 0.0f;
  if (a.block) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, rmax[i]);
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) colinv[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(colinv[0], colinv[1]), fmaxf(colinv[2], colinv[3]));
    sblock = F8<FMT>::scale(m);
    if (threadIdx.x == 0) {
      if (a.s != nullptr) a.s[bj * f8_blocks(a.rows) + bi] = sblock;
      if (a.st != nullptr) a.st[bi * cb + bj] = sblock;
    }
  }
  if (a.q != nullptr) {
    const int64_t pitch = f8_pitch(a.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = a.block ? sblock : F8<FMT>::scale(row16_max(rmax[i]));
      const float inv = div_rn(1.0f, s);
      const int64_t row = r0 + i;
      if (row >= a.rows) continue;
      if (!a.block && cg == 0) a.s[bj * a.rows + row] = s;
      if (c0 < pitch)
        *reinterpret_cast<uint2*>(a.q + row * pitch + c0) = make_uint2(
            F8<FMT>::pack4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv),
            F8<FMT>::pack4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv));
    }
  }
  if (a.qt == nullptr) return;   // the same for every thread
  if (!a.block) {
#pragma unroll
    for (int k = 0; k < 8; ++k) colmax[rg][8 * cg + k] = cmax[k];
    __syncthreads();
    if (threadIdx.x < kF8Block) {
      float m = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, colmax[r][threadIdx.x]);
      const float s = F8<FMT>::scale(m);
      const int64_t col = bj * kF8Block + threadIdx.x;
      if (col < a.cols) a.st[bi * a.cols + col] = s;
      colinv[threadIdx.x] = div_rn(1.0f, s);
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float inv = a.block ? div_rn(1.0f, sblock) : colinv[8 * cg + k];
    *reinterpret_cast<uint2*>(tile + (8 * cg + k) * PITCH + 8 * rg) = make_uint2(
        F8<FMT>::pack4(x[0][k] * inv, x[1][k] * inv, x[2][k] * inv, x[3][k] * inv),
        F8<FMT>::pack4(x[4][k] * inv, x[5][k] * inv, x[6][k] * inv, x[7][k] * inv));
  }
  __syncthreads();
  const int64_t pitch = f8_pitch(a.rows);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int id = threadIdx.x + u * kThreads, c = id >> 3;
    const int64_t col = bj * kF8Block + c, r = bi * kF8Block + 16 * (id & 7);
    if (col < a.cols && r < pitch) {
      const uint2* t = reinterpret_cast<const uint2*>(tile + c * PITCH + 16 * (id & 7));
      *reinterpret_cast<uint4*>(a.qt + col * pitch + r) =
          make_uint4(t[0].x, t[0].y, t[1].x, t[1].y);
    }
  }
}

// Eight codes a thread.
template <int FMT, bool BF16>
__global__ __launch_bounds__(kThreads) void qg_f8_dequantize(F8Values a) {
  const int64_t pitch = f8_pitch(a.cols), chunks = pitch / 8, all = a.rows * chunks;
  const int64_t per = a.block ? f8_blocks(a.rows) : a.rows;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < all;
       k += (int64_t)gridDim.x * kThreads) {
    const int64_t row = k / chunks, c = 8 * (k - row * chunks);
    if (c >= a.cols) continue;
    const uint2 w = *reinterpret_cast<const uint2*>(a.q + row * pitch + c);
    const float s = a.s[(c / kF8Block) * per + (a.block ? row / kF8Block : row)];
    float lo[4], hi[4];
    F8<FMT>::unpack4(w.x, lo);
    F8<FMT>::unpack4(w.y, hi);
    const float v[8] = {lo[0] * s, lo[1] * s, lo[2] * s, lo[3] * s,
                        hi[0] * s, hi[1] * s, hi[2] * s, hi[3] * s};
    row_store<BF16>(a.out, row * a.cols + c, (int)(a.cols - c < 8 ? a.cols - c : 8), v);
  }
}

hipError_t launch_f8_quantize(const F8Quant& a, hipStream_t s) {
  const int cb = (int)f8_blocks(a.cols);
  const dim3 grid((unsigned)(cb * f8_blocks(a.rows)));
  auto go = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (a.source == kF8FromBf16)
      hipLaunchKernelGGL((qg_f8_quantize<F, kF8FromBf16>), grid, dim3(kThreads), 0, s, a, cb);
    else if (a.source == kF8FromFp32)
      hipLaunchKernelGGL((qg_f8_quantize<F, kF8FromFp32>), grid, dim3(kThreads), 0, s, a, cb);
    else
      hipLaunchKernelGGL((qg_f8_quantize<F, kF8FromInt8>), grid, dim3(kThreads), 0, s, a, cb);
  };
  if (a.format == kF8E4M3) go(std::integral_constant<int, 0>{});
  else go(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const F8Values& a, hipStream_t s) {
  const int64_t wgs = (a.rows * (f8_pitch(a.cols) / 8) + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(wgs < 16384 ? wgs : 16384));
  auto go = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (a.bf16)
      hipLaunchKernelGGL((qg_f8_dequantize<F, true>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((qg_f8_dequantize<F, false>), grid, dim3(kThreads), 0, s, a);
  };
  if (a.format == kF8E4M3) go(std::integral_constant<int, 0>{});
  else go(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

}  // namespace qg
