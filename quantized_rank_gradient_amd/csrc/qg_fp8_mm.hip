// Product of FP8 operands with a scale for each run of 128 values along K (A, and B by rows) or for each
// block of 128 x 128 (B):
//   out(i, j) = sum over blocks k of sa(k, i) sb(k, j) sum over the block of A(i, .) B(j, .)
// One v_mfma_f32_16x16x128_f8f6f4 takes a whole block of K: it starts from zero, and its four results per
// lane are scaled into the fp32 accumulators by the vector unit while the matrix unit works on the next
// ones. B enters as the MFMA's rows, so that a lane holds results of one row i of A (one scale sa) and
// four rows j of B.
//
// The order of K within a block is free as long as both operands agree: lane group g (lane / 16) takes the
// 16-byte chunks g and g + 4 of a row's 128 bytes.
#include "qg_fp8.hpp"
#include "qg_gemm.hpp"
#include "qg_kernels.hpp"
#include "qg_mm.hpp"
#include "qg_rows.hpp"

namespace qg {

typedef int v8i32 __attribute__((ext_vector_type(8)));

namespace {

// rows x cols of `first` (e4m3) and `second` (AF): zero scales stand for none.
template <int AF>
__device__ __forceinline__ f32x4 f8_mfma(v8i32 first, v8i32 second) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first, second, zero, 0, AF, 0, 0, 0, 0);
}

__device__ __forceinline__ v8i32 join8(uint4 lo, uint4 hi) {
  return v8i32{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// N consecutive results of one row (N a multiple of 4), those behind the last column left out.
template <int N>
__device__ __forceinline__ void f8_store(const F8Mm& a, int64_t i, int64_t j, const float* v) {
  const int64_t left = a.N - j;
  if (a.bf16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + i * a.N + j;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      if (left >= k + 4) {
        const uint2 w = make_uint2(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]));
        __builtin_memcpy(o + k, &w, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (left > k + e) o[k + e] = to_bf16(v[k + e]);
      }
    }
  } else {
    float* o = static_cast<float*>(a.out) + i * a.N + j;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      if (left >= k + 4) {
        __builtin_memcpy(o + k, v + k, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (left > k + e) o[k + e] = v[k + e];
      }
    }
  }
}

}  // namespace

// WI x WJ waves, each NI x NJ blocks of 16 x 16: a tile of BI rows of A and BJ rows of B. Lane group g's
// four rows of block jt are the wave's rows 4 NJ g + 4 jt + v, so that a lane's results of a row are 4 NJ
// consecutive columns.
template <int WI_, int WJ_, int NI_, int NJ_>
struct F8Tile {
  static constexpr int WI = WI_, WJ = WJ_, NI = NI_, NJ = NJ_;
  static constexpr int WAVES = WI * WJ, THREADS = 64 * WAVES;
  static constexpr int BI = 16 * WI * NI, BJ = 16 * WJ * NJ;
  static constexpr int A_BYTES = BI * kF8Block, B_BYTES = BJ * kF8Block;
  static constexpr int SA = A_BYTES + B_BYTES, SB = SA + 4 * BI;   // the scales' areas in a stage
  static constexpr int STAGE = SB + 4 * BJ;
  static constexpr int LDS = 2 * STAGE;
};

// 16-byte chunk c of a row lies in slot c ^ swz(row): the 16 rows that a group of lanes reads at a time
// fall on all banks. Rows of A are read 16 in a row, rows of B four in a row from each of four groups.
__device__ __forceinline__ int swz_a(int row) { return (row >> 1) & 7; }
template <int NJ>
__device__ __forceinline__ int swz_b(int row) {
  return ((row >> 1) & 1) | (((row / (4 * NJ)) & 3) << 1);
}

template <class T, int AF, bool BBLOCK>
__global__ __launch_bounds__(T::THREADS, T::THREADS == 512 ? 2 : 1) void qg_f8_mm(F8Mm a, int tm, int tn) {
  __shared__ alignas(1024) uint16_t lds16[T::LDS / 2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / T::WJ, wj = wave % T::WJ, g = lane >> 4, l16 = lane & 15;
  int ti, tj;
  mm_band(xcd_remap(blockIdx.x, tm * tn), tm, tn, ti, tj);
  const int64_t i0 = (int64_t)ti * T::BI, j0 = (int64_t)tj * T::BJ;
  const int64_t pitch = f8_pitch(a.K);
  const int nk = (int)f8_blocks(a.K);
  const uint32_t base = lds_addr(lds16);
  const char* lds = reinterpret_cast<const char*>(lds16);

  // this lane's chunks of a stage, as offsets from the tile's first row
  constexpr int PA = T::BI / (8 * T::WAVES), PB = T::BJ / (8 * T::WAVES);
  const int64_t rows_a = a.M - i0 < T::BI ? a.M - i0 : T::BI;
  const int64_t rows_b = a.N - j0 < T::BJ ? a.N - j0 : T::BJ;
  const uint8_t* pa = a.A + i0 * pitch;
  const uint8_t* pb = a.B + j0 * pitch;
  uint32_t va[PA], vb[PB], ka[PA], kb[PB];
#pragma unroll
  for (int u = 0; u < PA; ++u) {
    const int row = 8 * (wave * PA + u) + (lane >> 3);
    ka[u] = 16 * ((lane & 7) ^ swz_a(row));
    va[u] = row < rows_a ? (uint32_t)(row * pitch) + ka[u] : kOOB;
  }
#pragma unroll
  for (int u = 0; u < PB; ++u) {
    const int row = 8 * (wave * PB + u) + (lane >> 3);
    kb[u] = 16 * ((lane & 7) ^ swz_b<T::NJ>(row));
    vb[u] = row < rows_b ? (uint32_t)(row * pitch) + kb[u] : kOOB;
  }
  const int64_t nb = f8_blocks(a.N);
  auto issue = [&](int kt, int buf) {
    const uint32_t k0 = kt * kF8Block, left = (uint32_t)(pitch - k0), to = base + buf * T::STAGE;
    const v4i32 ra = rsrc_words(pa + k0, (uint32_t)(rows_a * pitch - k0));
    const v4i32 rb = rsrc_words(pb + k0, (uint32_t)(rows_b * pitch - k0));
#pragma unroll
    for (int u = 0; u < PA; ++u)
      dma16(ra, ka[u] < left ? va[u] : kOOB, to + 1024 * (wave * PA + u));
#pragma unroll
    for (int u = 0; u < PB; ++u)
      dma16(rb, kb[u] < left ? vb[u] : kOOB, to + T::A_BYTES + 1024 * (wave * PB + u));
    // scales, 64 a load; rows behind the last one read zeros
    constexpr int LA = T::BI / 64, LB = BBLOCK ? 1 : T::BJ / 64;
    if (wave < LA) {
      const v4i32 rs = rsrc_words(a.sa + (int64_t)kt * a.M + i0, (uint32_t)(rows_a * 4));
      dma4(rs, 4 * (64 * wave + lane), to + T::SA + 256 * wave);
    } else if (wave < LA + LB) {
      if constexpr (BBLOCK) {
        constexpr int NBT = (T::BJ + kF8Block - 1) / kF8Block;   // blocks that the tile touches
        const int64_t b0 = j0 / kF8Block;
        const v4i32 rs = rsrc_words(a.sb + kt * nb + b0, (uint32_t)((nb - b0) * 4));
        if (lane < NBT) dma4(rs, 4 * lane, to + T::SB);
      } else {
        const int w = wave - LA;
        const v4i32 rs = rsrc_words(a.sb + (int64_t)kt * a.N + j0, (uint32_t)(rows_b * 4));
        dma4(rs, 4 * (64 * w + lane), to + T::SB + 256 * w);
      }
    }
  };
  static_assert(T::WAVES >= T::BI / 64 + T::BJ / 64, "a wave for each load of scales");

  f32x4 acc[T::NJ][T::NI];
#pragma unroll
  for (int y = 0; y < T::NJ; ++y)
#pragma unroll
    for (int x = 0; x < T::NI; ++x) acc[y][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  issue(0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vm_lds<0>();      // this wave's part of the stage has come,
    barrier_nofence();     // and every wave's, and none still reads the other buffer
    if (kt + 1 < nk) issue(kt + 1, (kt + 1) & 1);
    const char* st = lds + (kt & 1) * T::STAGE;
    auto frag_a = [&](int x) {
      const int row = 16 * (wi * T::NI + x) + l16;
      const char* p = st + row * kF8Block;
      return join8(*reinterpret_cast<const uint4*>(p + 16 * (g ^ swz_a(row))),
                   *reinterpret_cast<const uint4*>(p + 16 * ((g + 4) ^ swz_a(row))));
    };
    auto frag_b = [&](int y) {
      const int row = 16 * wj * T::NJ + 4 * T::NJ * (l16 >> 2) + 4 * y + (l16 & 3);
      const char* p = st + T::A_BYTES + row * kF8Block;
      return join8(*reinterpret_cast<const uint4*>(p + 16 * (g ^ swz_b<T::NJ>(row))),
                   *reinterpret_cast<const uint4*>(p + 16 * ((g + 4) ^ swz_b<T::NJ>(row))));
    };
    v8i32 fa[T::NI];
    float sc[T::NI];
    float sblock = 1.0f;
    if constexpr (BBLOCK)
      sblock = *reinterpret_cast<const float*>(st + T::SB + 4 * (16 * wj * T::NJ / kF8Block));
#pragma unroll
    for (int x = 0; x < T::NI; ++x) {
      fa[x] = frag_a(x);
      sc[x] = *reinterpret_cast<const float*>(st + T::SA + 4 * (16 * (wi * T::NI + x) + l16));
      if constexpr (BBLOCK) sc[x] *= sblock;
    }
    static_for<T::NJ>([&](auto yc) {
      constexpr int y = decltype(yc)::value;
      const v8i32 fb = frag_b(y);
      float4 sb;
      if constexpr (!BBLOCK)
        sb = *reinterpret_cast<const float4*>(
            st + T::SB + 4 * (16 * wj * T::NJ + 4 * T::NJ * g + 4 * y));
#pragma unroll
      for (int x = 0; x < T::NI; ++x) {
        const f32x4 p = f8_mfma<AF>(fb, fa[x]);
        if constexpr (BBLOCK) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[y][x][v] = __builtin_fmaf(p[v], sc[x], acc[y][x][v]);
        } else {
          const float s[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[y][x][v] = __builtin_fmaf(p[v], sc[x] * s[v], acc[y][x][v]);
        }
      }
    });
  }
#pragma unroll
  for (int x = 0; x < T::NI; ++x) {
    const int64_t i = i0 + 16 * (wi * T::NI + x) + l16;
    const int64_t j = j0 + 16 * wj * T::NJ + 4 * T::NJ * g;
    if (i >= a.M) continue;
    float v[4 * T::NJ];
#pragma unroll
    for (int y = 0; y < T::NJ; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * y + e] = acc[y][x][e];
    f8_store<4 * T::NJ>(a, i, j, v);
  }
}

// Few rows of A (up to 16): a workgroup takes 16 rows of B, its KW waves the blocks of K in turn, each from
// memory straight into the MFMA's registers, U blocks on their way at a time. B's bytes bound it. With
// a.X the rows of A are quantized on the way: the four lanes of a row hold its run of 128 values.
template <int KW, int U, int AF, bool BBLOCK, bool QUANT>
__global__ __launch_bounds__(64 * KW) void qg_f8_few(F8Mm a) {
  __shared__ f32x4 sum[KW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t j0 = (int64_t)blockIdx.x * 16, pitch = f8_pitch(a.K), nb = f8_blocks(a.N);
  const int nk = (int)f8_blocks(a.K);
  const bool on_a = l16 < a.M, on_b = j0 + l16 < a.N;
  const uint8_t* pb = a.B + (j0 + l16) * pitch;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto chunk = [&](const uint8_t* p, bool on, int64_t k) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (on && k < pitch) w = *reinterpret_cast<const uint4*>(p + k);
    return w;
  };
  for (int kt0 = wave; kt0 < nk; kt0 += KW * U) {
    v8i32 fb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (int64_t)(kt0 + KW * u) * kF8Block + 16 * g;
      fb[u] = join8(chunk(pb, on_b, k), chunk(pb, on_b, k + 64));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = kt0 + KW * u;
      if (kt >= nk) continue;   // the same for the whole wave
      const int64_t k = (int64_t)kt * kF8Block + 16 * g;
      v8i32 fa;
      float s;
      if constexpr (QUANT) {
        float v[32];
        float m = 0.0f;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int64_t c = k + 64 * (h >> 1) + 8 * (h & 1);
          const int left = on_a && c < a.K ? (int)(a.K - c < 8 ? a.K - c : 8) : 0;
          RowRaw<true> x{};
          if (left > 0) x.load(a.X, l16 * a.K + c, left);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[8 * h + e] = x.get(e);
            m = fmaxf(m, fabsf(v[8 * h + e]));
          }
        }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        s = F8<AF>::scale(m);
        const float inv = div_rn(1.0f, s);
#pragma unroll
        for (int h = 0; h < 8; ++h)
          fa[h] = (int)F8<AF>::pack4(v[4 * h] * inv, v[4 * h + 1] * inv, v[4 * h + 2] * inv,
                                     v[4 * h + 3] * inv);
      } else {
        const uint8_t* pa = a.A + l16 * pitch;
        fa = join8(chunk(pa, on_a, k), chunk(pa, on_a, k + 64));
        s = on_a ? a.sa[(int64_t)kt * a.M + l16] : 0.0f;
      }
      const f32x4 p = f8_mfma<AF>(fb[u], fa);
      if constexpr (BBLOCK) {
        s *= a.sb[kt * nb + j0 / kF8Block];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(p[v], s, acc[v]);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t j = j0 + 4 * g + v;
          const float sb = j < a.N ? a.sb[(int64_t)kt * a.N + j] : 0.0f;
          acc[v] = __builtin_fmaf(p[v], s * sb, acc[v]);
        }
      }
    }
  }
  sum[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < KW; ++w) {
    const f32x4 o = sum[w][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += o[v];
  }
  if (!on_a || j0 + 4 * g >= a.N) return;
  const float v[4] = {acc[0], acc[1], acc[2], acc[3]};
  f8_store<4>(a, l16, j0 + 4 * g, v);
}

namespace {

template <class T, int AF, bool BBLOCK>
hipError_t f8_tiles(const F8Mm& a, hipStream_t s) {
  const int tm = (int)((a.M + T::BI - 1) / T::BI), tn = (int)((a.N + T::BJ - 1) / T::BJ);
  hipLaunchKernelGGL((qg_f8_mm<T, AF, BBLOCK>), dim3((unsigned)(tm * tn)), dim3(T::THREADS), 0, s, a,
                     tm, tn);
  return hipGetLastError();
}

template <int AF, bool BBLOCK>
hipError_t f8_mm(const F8Mm& a, hipStream_t s) {
  if (a.M <= kF8Few) {
    const dim3 grid((unsigned)((a.N + 15) / 16));
    if (a.X != nullptr)
      hipLaunchKernelGGL((qg_f8_few<4, 4, AF, BBLOCK, true>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((qg_f8_few<4, 4, AF, BBLOCK, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const int64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (big >= 192) return f8_tiles<F8Tile<4, 2, 4, 8>, AF, BBLOCK>(a, s);
  return f8_tiles<F8Tile<2, 2, 4, 4>, AF, BBLOCK>(a, s);
}

}  // namespace

hipError_t launch_f8_mm(const F8Mm& a, hipStream_t s) {
  if (a.a_format == kF8E4M3) return a.b_block ? f8_mm<0, true>(a, s) : f8_mm<0, false>(a, s);
  return a.b_block ? f8_mm<1, true>(a, s) : f8_mm<1, false>(a, s);
}

}  // namespace qg
