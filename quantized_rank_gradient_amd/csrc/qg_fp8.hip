// FP8 codes of a matrix with one fp32 scale for each run of 128 values along a row (Q), along a column (Qt,
// the transpose) or for each block of 128 x 128 (both), and the way back. One read of the matrix serves both
// orders. Bytes bound it: 2 in and 1 out (or 2) for each bf16 value. 4096 x 11008 in both orders 42 us (180 MB
// at 4.3 TB/s; from fp32 52, 270 MB at 5.2), 4096 x 4096 along rows 12, the values of 4096 x 11008 codes 23
// (135 MB at 5.9); INT8 weights of 11008 x 4096 in both orders 38 to 41 us for 135 MB: there the two writes of
// 128 bytes a row take as long.
#include <type_traits>

#include "qg_fp8.hpp"
#include "qg_gemm.hpp"
#include "qg_kernels.hpp"
#include "qg_rows.hpp"

namespace qg {

namespace {

// Eight values of a row from column c on, for matrices of eight columns or more: read without a branch, as
// the row's last eight where c lies further right, and from the last row below it (get), and shifted into
// their places, zeros behind the ends, where a tile lies over one (fix).
template <int SRC>
struct F8Row {
  RowRaw<SRC == kF8FromBf16> x;
  uint32_t w[2];
  float s0, s1;
  int here;   // values of the first scale
  __device__ __forceinline__ void get(const F8Quant& a, int64_t row, int64_t c) {
    const int64_t e = (row < a.rows ? row : a.rows - 1) * a.cols + (c < a.cols - 8 ? c : a.cols - 8);
    if constexpr (SRC != kF8FromInt8) {
      x.load(a.src, e, 8);
    } else {
      __builtin_memcpy(w, static_cast<const uint8_t*>(a.src) + e, 8);
      // eight codes lie in two groups at most, and in one where every row begins at a multiple of eight
      s0 = s1 = a.src_scale[e >> 8];
      if (a.cols & 7) s1 = a.src_scale[(e + 7) >> 8];
      here = kGroup - (int)(e & (kGroup - 1));
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (SRC != kF8FromInt8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x.get(i);
    } else {
      static_for<8>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        v[i] = sbyte_to_f32<i & 3>(w[i >> 2]) * (i < here ? s0 : s1);
      });
    }
  }
  static __device__ __forceinline__ void fix(const F8Quant& a, int64_t row, int64_t c, float (&v)[8]) {
    const int64_t by = row >= a.rows ? 8 : c - (a.cols - 8);
#pragma unroll
    for (int step = 1; step < 8; step *= 2) {
      const bool on = by > 0 && (by & step);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = on ? (i + step < 8 ? v[i + step] : 0.0f) : v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = by >= 8 ? 0.0f : v[i];
  }
};
// The same of matrices of fewer columns.
template <int SRC>
__device__ __forceinline__ void f8_narrow(const F8Quant& a, int64_t row, int64_t c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t e = row * a.cols + c + i;
    v[i] = 0.0f;
    if (row >= a.rows || c + i >= a.cols) continue;
    if (SRC == kF8FromBf16) v[i] = bf16_to_f32(static_cast<const uint16_t*>(a.src)[e]);
    if (SRC == kF8FromFp32) v[i] = static_cast<const float*>(a.src)[e];
    if (SRC == kF8FromInt8) v[i] = (float)static_cast<const int8_t*>(a.src)[e] * a.src_scale[e >> 8];
  }
}

}  // namespace

// A tile of 128 x 128: thread (rg, cg) has rows 8 rg .. 8 rg + 7 and columns 8 cg .. 8 cg + 7, rg = its row
// of 16 lanes, so that a load takes whole lines and eight codes of a row or of a column leave together.
// The transposed codes go through LDS, to leave as lines too.
template <int FMT, int SRC>
__global__ __launch_bounds__(kThreads) void qg_f8_quantize(F8Quant a, int cb) {
  // The transposed codes: column c in row c ^ (c / 8 & 1), eight rows' codes rg in its 8-byte slot
  // rg ^ (c / 8), so that neither writes (16 columns that lie 8 apart, four slots) nor reads meet a bank
  // more often than they have to.
  __shared__ alignas(16) uint8_t tile[kF8Block * kF8Block];
  __shared__ float colmax[16][kF8Block];
  __shared__ float colinv[kF8Block];
  const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15;
  const int64_t bj = blockIdx.x % cb, bi = blockIdx.x / cb;
  const int64_t r0 = bi * kF8Block + 8 * rg, c0 = bj * kF8Block + 8 * cg;
  float x[8][8];
  if (a.cols >= 8) {
    F8Row<SRC> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i].get(a, r0 + i, c0);
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i].values(x[i]);
    if ((bi + 1) * kF8Block > a.rows || (bj + 1) * kF8Block > a.cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) F8Row<SRC>::fix(a, r0 + i, c0, x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f8_narrow<SRC>(a, r0 + i, c0, x[i]);
  }
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
  float sblock = 0.0f, iblock = 0.0f;
  if (a.block) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, rmax[i]);
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) colinv[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(colinv[0], colinv[1]), fmaxf(colinv[2], colinv[3]));
    sblock = F8<FMT>::scale(m);
    iblock = div_rn(1.0f, sblock);
    if (threadIdx.x == 0) {
      if (a.s != nullptr) a.s[bj * f8_blocks(a.rows) + bi] = sblock;
      if (a.st != nullptr) a.st[bi * cb + bj] = sblock;
    }
  }
  if (a.q != nullptr) {
    const int64_t pitch = f8_pitch(a.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = sblock, inv = iblock;
      if (!a.block) {
        s = F8<FMT>::scale(row16_max(rmax[i]));
        inv = div_rn(1.0f, s);
      }
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
    const float inv = a.block ? iblock : colinv[8 * cg + k];
    *reinterpret_cast<uint2*>(tile + (8 * cg + (k ^ (cg & 1))) * kF8Block + 8 * (rg ^ cg)) = make_uint2(
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
      const int g = c >> 3, odd = g & 1;
      const uint4 t = *reinterpret_cast<const uint4*>(tile + (c ^ odd) * kF8Block +
                                                      16 * ((id & 7) ^ (g >> 1)));
      *reinterpret_cast<uint4*>(a.qt + col * pitch + r) =
          odd ? make_uint4(t.z, t.w, t.x, t.y) : t;
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
