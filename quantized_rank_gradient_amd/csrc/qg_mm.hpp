// Matrix products of 16-bit operands (fp16 or bf16) with fp32 accumulation for the operators
// whose time is one dense product: out(i, j) = sum_k A(i, k) B(j, k).
//
// A workgroup of four waves (2 x 2) computes a (64 XM) x (64 XN) tile, each wave XM x XN blocks
// of v_mfma_f32_32x32x16. K runs in stages of 64 through two LDS buffers that are filled by
// direct-to-LDS loads, so no register holds a value on its way. An operand is stored either
//   K-contiguous   element (c, k) at base + c * ld + k   (a row-major matrix times a transpose)
//   K-major        element (c, k) at base + k * ld + c
// and stays in that order in LDS: K-contiguous tiles are rows of 64 (128 bytes, whole cache
// lines), read with one ds_read_b128 per fragment; K-major tiles are 64 rows of the tile's edge,
// read with two transposing ds_read_b64_tr_b16. The 16-byte chunks of a row are permuted so that
// the lanes of a read fall on distinct banks.
//
// The fragments enter the MFMA as (B, A), so that a lane's accumulators hold four consecutive
// columns j of one row i: the tile goes to LDS as fp32 in 16-byte pieces (mm_image), and every
// epilogue then works on eight consecutive columns of a row with wide loads and stores.
#pragma once

#include "qg_gemm.hpp"

namespace qg {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short v8i16 __attribute__((ext_vector_type(8)));

// The operands' element type.
struct MmF16 {
  static __device__ __forceinline__ f32x16 mfma(v8i16 a, v8i16 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
struct MmBf16 {
  static __device__ __forceinline__ f32x16 mfma(v8i16 a, v8i16 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

constexpr int kMmK = 64;   // K values per stage

// An operand in memory: `rows` rows of ld elements, ld a multiple of 8 and the base 16-byte
// aligned. K-contiguous: rows run along the output, K <= ld. K-major: rows run along K, and
// columns at or past c_end (a multiple of 8 from it on) read as zero.
struct MmOperand {
  const uint16_t* p;
  int64_t ld;
  int32_t rows;    // rows of the matrix: reads past them give zeros
  int32_t c_end;   // columns that are read: K (K-contiguous) or the output extent (K-major)
};

template <int XM_, int XN_, bool AKM_, bool BKM_, class E_>
struct MmTile {
  static constexpr int XM = XM_, XN = XN_, BM = 64 * XM_, BN = 64 * XN_;
  static constexpr bool AKM = AKM_, BKM = BKM_;
  using E = E_;
  static constexpr int A_ELEMS = BM * kMmK, B_ELEMS = BN * kMmK, STAGE = A_ELEMS + B_ELEMS;
  // rows of the fp32 image that the epilogue holds at a time
  static constexpr int IMG_ROWS = 128, PASSES = BM / IMG_ROWS;
  static_assert(BM % IMG_ROWS == 0 && BN >= 128, "tile edges");
  static constexpr int LDS_BYTES =
      2 * STAGE * 2 > IMG_ROWS * BN * 4 ? 2 * STAGE * 2 : IMG_ROWS * BN * 4;
  // workgroups per CU that the LDS and the accumulators leave room for
  static constexpr int OCC = XM * XN > 8 ? 1 : 2;
};

// Fills one operand tile of W rows (or columns) from output index c0.
template <int W, bool KM>
struct MmStage {
  static constexpr int NI = W / 32;                    // 1 KiB loads per wave and stage
  static constexpr int CPR = KM ? W / 8 : kMmK / 8;    // chunks per tile row
  static constexpr int RPI = 64 / CPR;                 // tile rows per load
  MmOperand o;
  uint32_t vo[NI];   // byte offset of this lane's chunk from the stage's origin

  __device__ MmStage(const MmOperand& o_, int c0) : o(o_) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = (wave * NI + i) * RPI + lane / CPR;
      if constexpr (KM) {
        const uint32_t c = c0 + 8 * kmaj_slot<W>(row, lane % CPR);
        vo[i] = c < (uint32_t)o.c_end ? (row * (uint32_t)o.ld + c) * 2 : kOOB;
      } else {
        const uint32_t rg = c0 + row;
        vo[i] = rg < (uint32_t)o.rows ? (rg * (uint32_t)o.ld + 8 * kcol(row, lane)) * 2 : kOOB;
      }
    }
  }
  // K-contiguous: the chunk that this lane loads into slot lane % 8 of a row
  static __device__ __forceinline__ int kcol(int row, int lane) {
    return (lane % 8) ^ ((row >> 1) & 7);
  }

  // tile: LDS byte address of the stage's tile
  __device__ __forceinline__ void issue(uint32_t k0, uint32_t tile) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if constexpr (KM) {
      const uint32_t kb = k0 < (uint32_t)o.rows ? k0 : (uint32_t)o.rows;
      const v4i32 st = rsrc_words(o.p + (size_t)kb * o.ld,
                                  ((uint32_t)o.rows - kb) * (uint32_t)o.ld * 2);
#pragma unroll
      for (int i = 0; i < NI; ++i) dma16(st, vo[i], tile + (wave * NI + i) * 1024);
    } else {
      const uint32_t kb = k0 < (uint32_t)o.c_end ? k0 : (uint32_t)o.c_end;
      const v4i32 st = rsrc_words(o.p + kb, ((uint32_t)o.rows * (uint32_t)o.ld - kb) * 2);
      const uint32_t left = (uint32_t)o.c_end - kb;   // K values left in the rows
      if (left >= (uint32_t)kMmK) {
#pragma unroll
        for (int i = 0; i < NI; ++i) dma16(st, vo[i], tile + (wave * NI + i) * 1024);
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int row = (wave * NI + i) * RPI + lane / CPR;
          dma16(st, 8u * kcol(row, lane) < left ? vo[i] : kOOB, tile + (wave * NI + i) * 1024);
        }
      }
    }
  }
};

// The fragment of rows (columns) c .. c + 31 and K values ks .. ks + 15 of a tile in LDS.
template <int W, bool KM>
__device__ __forceinline__ v8i16 mm_frag(const uint16_t* tile, int c, int ks) {
  const int lane = threadIdx.x & 63;
  if constexpr (!KM) {
    const int row = c + (lane & 31);
    return *reinterpret_cast<const v8i16*>(
        tile + row * kMmK + 8 * (((ks >> 3) + (lane >> 5)) ^ ((row >> 1) & 7)));
  } else {
    typedef __attribute__((address_space(3))) v4i16* lptr;
    const int row = ks + 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int col = c + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const uint16_t* p0 = tile + row * W + 8 * kmaj_slot<W>(row, col >> 3) + (col & 7);
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr)(__attribute__((address_space(3))) void*)(p0));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr)(__attribute__((address_space(3))) void*)(p0 + 4 * W));
    return v8i16{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
}

// acc = A(tile rows i0 ..) B(tile columns j0 ..)^T over K. Element v of acc[x][y] is row
// 32 x + lane % 32 and column 32 y + 8 (v / 4) + 4 (lane / 32) + v % 4 of the wave's sub-tile.
template <class T>
__device__ __forceinline__ void mm_kloop(const MmOperand& oa, const MmOperand& ob, int i0, int j0,
                                         int K, uint16_t* lds, f32x16 (&acc)[T::XM][T::XN]) {
  const int wave = threadIdx.x >> 6;
  const int am = (wave >> 1) * 32 * T::XM, bn = (wave & 1) * 32 * T::XN;
  const MmStage<T::BM, T::AKM> sa(oa, i0);
  const MmStage<T::BN, T::BKM> sb(ob, j0);
#pragma unroll
  for (int x = 0; x < T::XM; ++x)
#pragma unroll
    for (int y = 0; y < T::XN; ++y)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[x][y][v] = 0.0f;
  const int nk = (K + kMmK - 1) / kMmK;
  const uint32_t base = lds_addr(lds);
  sa.issue(0, base);
  sb.issue(0, base + 2 * T::A_ELEMS);
  for (int k0 = 0; k0 < nk; k0 += 2) {
    static_for<2>([&](auto bc) {
      constexpr int buf = decltype(bc)::value;
      const int kt = k0 + buf;
      if (kt < nk) {
        wait_vm_lds<0>();
        barrier_nofence();
        if (kt + 1 < nk) {
          const uint32_t nxt = base + (buf ^ 1) * 2 * T::STAGE;
          sa.issue((kt + 1) * kMmK, nxt);
          sb.issue((kt + 1) * kMmK, nxt + 2 * T::A_ELEMS);
        }
        const uint16_t* As = lds + buf * T::STAGE;
        const uint16_t* Bs = As + T::A_ELEMS;
#pragma unroll
        for (int ks = 0; ks < kMmK; ks += 16) {
          v8i16 a[T::XM], b[T::XN];
#pragma unroll
          for (int x = 0; x < T::XM; ++x) a[x] = mm_frag<T::BM, T::AKM>(As, am + 32 * x, ks);
#pragma unroll
          for (int y = 0; y < T::XN; ++y) b[y] = mm_frag<T::BN, T::BKM>(Bs, bn + 32 * y, ks);
#pragma unroll
          for (int x = 0; x < T::XM; ++x)
#pragma unroll
            for (int y = 0; y < T::XN; ++y) acc[x][y] = T::E::mfma(b[y], a[x], acc[x][y]);
        }
      }
    });
  }
  __syncthreads();   // the epilogue reuses the LDS area
}

// The fp32 image of IMG_ROWS rows of the tile: row r's columns j .. j + 3 at 16-byte chunk
// (j / 4) ^ img_swz(r). The permutation keeps pairs of chunks together, and puts on distinct
// banks both the 32 rows of a column that the accumulators are written by and the 8 groups of
// 8 rows that mm_column8 reads.
__device__ __forceinline__ int img_swz(int r) { return 2 * (((r >> 3) ^ r) & 7); }

// Writes rows IMG_ROWS * pass .. of the accumulated tile into the image; barriers around it.
template <class T>
__device__ __forceinline__ void mm_image(float* img, const f32x16 (&acc)[T::XM][T::XN],
                                         int pass) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int am = (wave >> 1) * 32 * T::XM, bn = (wave & 1) * 32 * T::XN;
  if (pass > 0) __syncthreads();
  if (am / T::IMG_ROWS == pass) {
#pragma unroll
    for (int x = 0; x < T::XM; ++x) {
      const int r = am % T::IMG_ROWS + 32 * x + (lane & 31);
#pragma unroll
      for (int y = 0; y < T::XN; ++y)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = bn + 32 * y + 8 * q + 4 * (lane >> 5);
          *reinterpret_cast<float4*>(img + r * T::BN + 4 * ((j >> 2) ^ img_swz(r))) =
              make_float4(acc[x][y][4 * q], acc[x][y][4 * q + 1], acc[x][y][4 * q + 2],
                          acc[x][y][4 * q + 3]);
        }
    }
  }
  __syncthreads();
}

// f(row, column, v): eight consecutive columns of an image row; every chunk once over the
// workgroup, consecutive threads on consecutive chunks.
template <class T, class F>
__device__ __forceinline__ void mm_rows(const float* img, F&& f) {
  constexpr int CPR = T::BN / 8;
#pragma unroll 2
  for (int c = threadIdx.x; c < T::IMG_ROWS * CPR; c += kThreads) {
    const int r = c / CPR, j = 8 * (c % CPR);
    const float* p = img + r * T::BN + 4 * ((j >> 2) ^ img_swz(r));
    const float4 lo = *reinterpret_cast<const float4*>(p);
    const float4 hi = *reinterpret_cast<const float4*>(p + 4);
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    f(r, j, v);
  }
}

// f(row, column, v): eight consecutive rows of an image column (the transpose's rows); eight
// lanes on consecutive row groups, so that a store of the transpose covers 128 bytes of a row.
template <class T, class F>
__device__ __forceinline__ void mm_columns(const float* img, F&& f) {
  constexpr int GR = T::IMG_ROWS / 8;   // row groups
#pragma unroll 2
  for (int c = threadIdx.x; c < GR * T::BN; c += kThreads) {
    const int g = c % 8 + 8 * (c / (8 * T::BN)), j = (c / 8) % T::BN;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = 8 * g + e;
      v[e] = img[r * T::BN + 4 * ((j >> 2) ^ img_swz(r)) + (j & 3)];
    }
    f(8 * g, j, v);
  }
}

// Tile of workgroup `t` out of tm x tn: bands of eight tile rows, columns of tiles within a
// band, so that neighbours (on one XCD after xcd_remap) share operand rows and columns in L2.
__device__ __forceinline__ void mm_band(int t, int tm, int tn, int& ti, int& tj) {
  constexpr int BAND = 8;
  const int b = t / (BAND * tn);
  const int h = tm - b * BAND < BAND ? tm - b * BAND : BAND;
  const int r = t - b * BAND * tn;
  ti = b * BAND + r % h;
  tj = r / h;
}

// Tile t of the upper triangle (ti <= tj) of a symmetric output, column by column.
__device__ __forceinline__ void mm_triangle(int t, int& ti, int& tj) {
  int j = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
  while (j * (j + 1) / 2 > t) --j;
  while ((j + 1) * (j + 2) / 2 <= t) ++j;
  tj = j;
  ti = t - j * (j + 1) / 2;
}

}  // namespace qg
