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
#include "qg_kernels.hpp"

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

// The operand's K values from k0 on, K of them.
template <bool KM>
__device__ __forceinline__ MmOperand mm_cut(MmOperand o, int k0, int K) {
  if constexpr (KM) {
    o.p += (int64_t)k0 * o.ld;
    o.rows = K;
  } else {
    o.p += k0;
    o.c_end = K;
  }
  return o;
}

// XM = XN = 4 (256 x 256, one workgroup per CU) for outputs that fill the chip with them, 2
// (128 x 128, two per CU), and 1 (64 x 64, three per CU) where the time is the latency of a
// stage: its ring of stages keeps more loads in flight.
template <int XM_, int XN_, bool AKM_, bool BKM_, class E_>
struct MmTile {
  static constexpr int XM = XM_, XN = XN_, BM = 64 * XM_, BN = 64 * XN_;
  static constexpr bool AKM = AKM_, BKM = BKM_;
  using E = E_;
  static constexpr int A_ELEMS = BM * kMmK, B_ELEMS = BN * kMmK, STAGE = A_ELEMS + B_ELEMS;
  static constexpr int NST = XM * XN == 1 ? 3 : 2;   // stages in LDS
  // rows of the fp32 image that the epilogue holds at a time
  static constexpr int IMG_ROWS = BM < 128 ? BM : 128, PASSES = BM / IMG_ROWS;
  static constexpr int LDS_BYTES =
      NST * STAGE * 2 > IMG_ROWS * BN * 4 ? NST * STAGE * 2 : IMG_ROWS * BN * 4;
  // workgroups per CU that the LDS and the accumulators leave room for
  static constexpr int OCC = XM * XN > 8 ? 1 : XM * XN > 1 ? 2 : 3;
};

// Position of 16-byte chunk j of row k in a K-major tile of W columns: for rows of 256 or 512
// bytes as kmaj_slot; rows of 128 bytes alternate between the halves of the 64 banks by
// themselves, and every second pair of rows swaps its 64-byte blocks.
template <int W>
__device__ __forceinline__ int mm_slot(int k, int j) {
  if constexpr (W >= 128)
    return kmaj_slot<W>(k, j);
  else
    return j ^ (4 * ((k >> 1) & 1));
}

// Fills one operand tile of W rows (or columns) from output index c0.
template <int W, bool KM>
struct MmStage {
  static constexpr int NI = W / 32;                    // 1 KiB loads per wave and stage
  static constexpr int CPR = KM ? W / 8 : kMmK / 8;    // chunks per tile row
  static constexpr int RPI = 64 / CPR;                 // tile rows per load
  MmOperand o;
  uint32_t wofs;     // byte offset of this wave's loads in a tile
  uint32_t vo[NI];   // byte offset of this lane's chunk from the stage's origin

  __device__ MmStage(const MmOperand& o_, int c0) : o(o_) {
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3;
    wofs = __builtin_amdgcn_readfirstlane(wave * NI * 1024);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = (wave * NI + i) * RPI + lane / CPR;
      if constexpr (KM) {
        // no operand has kOOB bytes; rows behind the last one may lie further than 32 bits reach
        const uint32_t c = c0 + 8 * mm_slot<W>(row, lane % CPR);
        const uint64_t at = ((uint64_t)row * (uint64_t)o.ld + c) * 2;
        vo[i] = c < (uint32_t)o.c_end && at < kOOB ? (uint32_t)at : kOOB;
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

  // What the loads of one stage share: the resource from the stage's origin on, and for a
  // K-contiguous operand the K values left in its rows. Chunks at or past K go out of range; a
  // stage may lie behind the last one.
  struct At {
    v4i32 rs;
    uint32_t left, tile;
  };
  // tile: LDS byte address of the stage's tile
  __device__ __forceinline__ At at(uint32_t k0, uint32_t tile) const {
    const uint32_t end = (uint32_t)(KM ? o.rows : o.c_end);
    const uint32_t kb = k0 < end ? k0 : end;
    At s;
    s.left = end - kb;
    s.tile = tile + wofs;
    if constexpr (KM)
      s.rs = rsrc_words(o.p + (size_t)kb * o.ld, s.left * (uint32_t)o.ld * 2);
    else
      s.rs = rsrc_words(o.p + kb, ((uint32_t)o.rows * (uint32_t)o.ld - kb) * 2);
    return s;
  }
  // load i of this wave
  __device__ __forceinline__ void one(const At& s, int i) const {
    if constexpr (KM) {
      dma16(s.rs, vo[i], s.tile + i * 1024);
    } else {
      const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3;
      const int row = (wave * NI + i) * RPI + lane / CPR;
      dma16(s.rs, 8u * kcol(row, lane) < s.left ? vo[i] : kOOB, s.tile + i * 1024);
    }
  }
  __device__ __forceinline__ void issue(uint32_t k0, uint32_t tile) const {
    const At s = at(k0, tile);
#pragma unroll
    for (int i = 0; i < NI; ++i) one(s, i);
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
    const uint16_t* p0 = tile + row * W + 8 * mm_slot<W>(row, col >> 3) + (col & 7);
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr)(__attribute__((address_space(3))) void*)(p0));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr)(__attribute__((address_space(3))) void*)(p0 + 4 * W));
    return v8i16{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
}

// The fragments of one K step of a stage (16 K values) for this wave.
template <class T>
struct MmFrags {
  static constexpr int N = T::XM + T::XN;
  v8i16 a[T::XM], b[T::XN];
  template <int I>
  __device__ __forceinline__ void one(const uint16_t* stage, int ks) {
    const int wave = (threadIdx.x >> 6) & 3;
    if constexpr (I < T::XM)
      a[I] = mm_frag<T::BM, T::AKM>(stage, (wave >> 1) * 32 * T::XM + 32 * I, ks);
    else
      b[I - T::XM] = mm_frag<T::BN, T::BKM>(stage + T::A_ELEMS,
                                            (wave & 1) * 32 * T::XN + 32 * (I - T::XM), ks);
  }
  __device__ __forceinline__ void load(const uint16_t* stage, int ks) {
    static_for<N>([&](auto i) { this->template one<decltype(i)::value>(stage, ks); });
  }
};

template <class T>
__device__ __forceinline__ void mm_kloop_ring(const MmOperand& oa, const MmOperand& ob, int i0,
                                              int j0, int K, uint16_t* lds,
                                              f32x16 (&acc)[T::XM][T::XN]);

// One K step: the MFMAs of `cur`, and spread evenly between them the reads of the next step's
// fragments and loads L0 .. L1 - 1 of a later stage (load(l) issues one). The order is fixed: with
// one wave per SIMD nothing else covers a burst of reads or of loads.
template <class T, int L0, int L1, class F>
__device__ __forceinline__ void mm_step(const MmFrags<T>& cur, MmFrags<T>& next,
                                        const uint16_t* stage, int ks,
                                        f32x16 (&acc)[T::XM][T::XN], F&& load) {
  constexpr int MF = T::XM * T::XN, FR = MmFrags<T>::N;
  static_for<MF>([&](auto ic) {
    constexpr int i = decltype(ic)::value, x = i / T::XN, y = i % T::XN;
    acc[x][y] = T::E::mfma(cur.b[y], cur.a[x], acc[x][y]);
    constexpr int r0 = i * FR / MF, r1 = (i + 1) * FR / MF;
    static_for<r1 - r0>([&](auto rc) {
      next.template one<r0 + decltype(rc)::value>(stage, ks);
    });
    constexpr int l0 = L0 + i * (L1 - L0) / MF, l1 = L0 + (i + 1) * (L1 - L0) / MF;
    static_for<l1 - l0>([&](auto lc) { load(l0 + decltype(lc)::value); });
    __builtin_amdgcn_sched_barrier(0);
  });
}

// acc = A(tile rows i0 ..) B(tile columns j0 ..)^T over K. Element v of acc[x][y] is row
// 32 x + lane % 32 and column 32 y + 8 (v / 4) + 4 (lane / 32) + v % 4 of the wave's sub-tile.
//
// Each K step's fragments are read while the step before is multiplied, across stages too: the
// last step's fragments are in registers when the workgroup meets at the stage's one barrier, so
// after it the stage's buffer is free for the stage after next.
template <class T>
__device__ __forceinline__ void mm_kloop(const MmOperand& oa, const MmOperand& ob, int i0, int j0,
                                         int K, uint16_t* lds, f32x16 (&acc)[T::XM][T::XN]) {
  if constexpr (T::NST > 2) {
    mm_kloop_ring<T>(oa, ob, i0, j0, K, lds, acc);
    return;
  }
  using SA = MmStage<T::BM, T::AKM>;
  using SB = MmStage<T::BN, T::BKM>;
  const SA sa(oa, i0);
  const SB sb(ob, j0);
#pragma unroll
  for (int x = 0; x < T::XM; ++x)
#pragma unroll
    for (int y = 0; y < T::XN; ++y)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[x][y][v] = 0.0f;
  // Stages come in pairs, without a branch in the loop: one behind the last multiplies zeros, and
  // the two whose loads are issued past the end read nothing.
  const int nk = (K + 2 * kMmK - 1) / (2 * kMmK) * 2;
  const uint32_t base = lds_addr(lds);
  constexpr int NI = SA::NI + SB::NI;
  MmFrags<T> f0, f1;
  typename SA::At ta;
  typename SB::At tb;
  auto load = [&](int l) {
    if (l < SA::NI)
      sa.one(ta, l);
    else
      sb.one(tb, l - SA::NI);
  };
  auto open = [&](int kt, int buf) {
    ta = sa.at(kt * kMmK, base + buf * 2 * T::STAGE);
    tb = sb.at(kt * kMmK, base + buf * 2 * T::STAGE + 2 * T::A_ELEMS);
  };
  // A stage's loads go out over the two K steps behind the barrier that frees its buffer, one
  // beside each MFMA: all of them in one step are more than the vector memory path takes in its
  // time (64 KiB in 512 MFMA cycles), and the waves stall at issue. 4096 x 4096 x 8192: one step
  // 1300 TFLOP/s, two 1354, three 1358 with less time for the last ones to arrive.
  constexpr int S1 = NI / 2;
  sa.issue(0, base);
  sb.issue(0, base + 2 * T::A_ELEMS);
  open(1, 1);
  static_for<S1>([&](auto l) { load(decltype(l)::value); });
  wait_vm_lds<S1>();
  barrier_nofence();
  f0.load(lds, 0);
  for (int kt = 0; kt < nk; kt += 2) {
    static_for<2>([&](auto bc) {
      constexpr int buf = decltype(bc)::value;
      const uint16_t* cur = lds + buf * T::STAGE;
      mm_step<T, S1, NI>(f0, f1, cur, 16, acc, load);
      mm_step<T, 0, 0>(f1, f0, cur, 32, acc, load);
      mm_step<T, 0, 0>(f0, f1, cur, 48, acc, load);
      wait_vm_lds<0>();
      barrier_nofence();
      open(kt + buf + 2, buf);
      mm_step<T, 0, S1>(f1, f0, lds + (buf ^ 1) * T::STAGE, 0, acc, load);
    });
  }
  // the epilogue reuses the LDS area: no load may still be on its way there
  wait_vm_lds<0>();
  __syncthreads();
}

// The same for small tiles: a ring of NST stages, NST - 1 of them loading while one is multiplied.
// Stages past K read nothing, so that every stage has as many loads to wait for.
template <class T>
__device__ __forceinline__ void mm_kloop_ring(const MmOperand& oa, const MmOperand& ob, int i0,
                                              int j0, int K, uint16_t* lds,
                                              f32x16 (&acc)[T::XM][T::XN]) {
  using SA = MmStage<T::BM, T::AKM>;
  using SB = MmStage<T::BN, T::BKM>;
  constexpr int NI = SA::NI + SB::NI, NST = T::NST;
  const SA sa(oa, i0);
  const SB sb(ob, j0);
#pragma unroll
  for (int x = 0; x < T::XM; ++x)
#pragma unroll
    for (int y = 0; y < T::XN; ++y)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[x][y][v] = 0.0f;
  const int nk = (K + kMmK - 1) / kMmK;
  const uint32_t base = lds_addr(lds);
  static_for<NST - 1>([&](auto sc) {
    constexpr int s = decltype(sc)::value;
    sa.issue(s * kMmK, base + s * 2 * T::STAGE);
    sb.issue(s * kMmK, base + s * 2 * T::STAGE + 2 * T::A_ELEMS);
  });
  for (int k0 = 0; k0 < nk; k0 += NST) {
    static_for<NST>([&](auto bc) {
      constexpr int buf = decltype(bc)::value, nb = (buf + NST - 1) % NST;
      const int kt = k0 + buf;
      if (kt < nk) {
        // this stage has arrived for every wave, and none still reads the one before it
        wait_vm_lds<(NST - 2) * NI>();
        barrier_nofence();
        // all of the stage's fragments on their way at once, and the loads issued meanwhile; left
        // to itself the compiler reads two, waits and multiplies, four times over
        MmFrags<T> f[kMmK / 16];
        static_for<kMmK / 16>([&](auto kc) {
          f[decltype(kc)::value].load(lds + buf * T::STAGE, 16 * decltype(kc)::value);
        });
        __builtin_amdgcn_sched_barrier(0);
        sa.issue((kt + NST - 1) * kMmK, base + nb * 2 * T::STAGE);
        sb.issue((kt + NST - 1) * kMmK, base + nb * 2 * T::STAGE + 2 * T::A_ELEMS);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < kMmK / 16; ++ks)
#pragma unroll
          for (int x = 0; x < T::XM; ++x)
#pragma unroll
            for (int y = 0; y < T::XN; ++y)
              acc[x][y] = T::E::mfma(f[ks].b[y], f[ks].a[x], acc[x][y]);
      }
    });
  }
  wait_vm_lds<0>();
  __syncthreads();
}

// Part `part` of `split` of one tile's sum over K: true for the workgroup that comes last, whose acc
// then holds the whole sum, added in the order of the parts whatever order they came in. `parts`:
// the tile's split x BM x BN floats; `count`: its counter, 0 before and after.
//
// The parts go through atomic stores and loads of the whole device's scope: these pass the XCDs'
// own L2 caches by. A fence of that scope instead empties the cache for each workgroup, one after
// another: 264 of them took 40 us.
template <class T>
__device__ __forceinline__ bool mm_join(f32x16& acc, float* parts, uint32_t* count, int part,
                                        int split, uint16_t* lds) {
  static_assert(T::XM == 1 && T::XN == 1, "one block per wave");
  constexpr auto relaxed = __ATOMIC_RELAXED;
  auto at = [&](int s, int v) {
    return reinterpret_cast<uint64_t*>(parts + (size_t)s * (T::BM * T::BN)) + v * kThreads +
           threadIdx.x;
  };
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const uint64_t lo = __float_as_uint(acc[2 * v]), hi = __float_as_uint(acc[2 * v + 1]);
    __hip_atomic_store(at(part, v), lo | hi << 32, relaxed, __HIP_MEMORY_SCOPE_AGENT);
  }
  wait_vm_lds<0>();   // each wave's part is in memory
  __syncthreads();    // and every wave's, before it is counted
  volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(lds);
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(count, 1u, relaxed, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = *flag == (uint32_t)split - 1;
  __syncthreads();
  if (!last) return false;
  if (threadIdx.x == 0) __hip_atomic_store(count, 0u, relaxed, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  for (int s = 0; s < split; ++s) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const uint64_t w = __hip_atomic_load(at(s, v), relaxed, __HIP_MEMORY_SCOPE_AGENT);
      acc[2 * v] += __uint_as_float((uint32_t)w);
      acc[2 * v + 1] += __uint_as_float((uint32_t)(w >> 32));
    }
  }
  return true;
}

// The fp32 image of IMG_ROWS rows of the tile: row r's columns j .. j + 3 at 16-byte chunk
// (j / 4) ^ img_swz(r). The permutation keeps pairs of chunks together, and puts on distinct
// banks both the 32 rows of a column that the accumulators are written by and the 8 groups of
// 8 rows that mm_column8 reads.
__device__ __forceinline__ int img_swz(int r) { return 2 * (((r >> 3) ^ r) & 7); }

// The wave's accumulators into an image, from row r0 and column bn on.
template <class T>
__device__ __forceinline__ void mm_put(float* img, const f32x16 (&acc)[T::XM][T::XN], int r0,
                                       int bn) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int x = 0; x < T::XM; ++x) {
    const int r = r0 + 32 * x + (lane & 31);
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

// Writes rows IMG_ROWS * pass .. of the accumulated tile into the image; barriers around it.
template <class T>
__device__ __forceinline__ void mm_image(float* img, const f32x16 (&acc)[T::XM][T::XN],
                                         int pass) {
  const int wave = threadIdx.x >> 6;
  const int am = (wave >> 1) * 32 * T::XM, bn = (wave & 1) * 32 * T::XN;
  if (pass > 0) __syncthreads();
  if (am / T::IMG_ROWS == pass) mm_put<T>(img, acc, am % T::IMG_ROWS, bn);
  __syncthreads();
}

// Eight consecutive columns of an image row at a time, every chunk once over the workgroup,
// consecutive threads on consecutive chunks: pre(row, column) fetches what the chunk needs from
// memory, f(row, column, v, fetched) finishes it. Fetches go out U at a time ahead of their use: a
// workgroup alone on its CU has nothing else to cover their latency. With KEEP, what f makes of v
// goes back into the image.
template <class T, int U_, bool KEEP = false, class P, class F>
__device__ __forceinline__ void mm_rows(float* img, P&& pre, F&& f) {
  constexpr int CPR = T::BN / 8, PER = T::IMG_ROWS * CPR / kThreads, U = U_ < PER ? U_ : PER;
  static_assert(PER % U == 0, "whole batches");
  using Pre = decltype(pre(0, 0));
#pragma unroll 1
  for (int c0 = threadIdx.x; c0 < T::IMG_ROWS * CPR; c0 += U * kThreads) {
    Pre p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kThreads;
      p[u] = pre(c / CPR, 8 * (c % CPR));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kThreads;
      const int r = c / CPR, j = 8 * (c % CPR);
      float4* q = reinterpret_cast<float4*>(img + r * T::BN + 4 * ((j >> 2) ^ img_swz(r)));
      const float4 lo = q[0], hi = q[1];
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      f(r, j, v, p[u]);
      if constexpr (KEEP) {
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}
// Nothing to fetch.
struct MmNone {
  __device__ MmNone operator()(int, int) const { return {}; }
};

// The same for eight consecutive rows of an image column (the transpose's rows); eight lanes on
// consecutive row groups, so that a store of the transpose covers 128 bytes of a row.
template <class T, int U_, class F>
__device__ __forceinline__ void mm_columns(const float* img, F&& f) {
  constexpr int N = T::IMG_ROWS / 8 * T::BN, PER = N / kThreads, U = U_ < PER ? U_ : PER;
  static_assert(PER % U == 0, "whole batches");
#pragma unroll 1
  for (int c0 = threadIdx.x; c0 < N; c0 += U * kThreads) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kThreads;
      const int r = 8 * (c % 8 + 8 * (c / (8 * T::BN))), j = (c / 8) % T::BN;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = img[(r + e) * T::BN + 4 * ((j >> 2) ^ img_swz(r + e)) + (j & 3)];
      f(r, j, v);
    }
  }
}

// A launch of `tiles` large tiles on a chip that takes kMmSlots at a time: where a last, mostly
// empty round would be left, its `sub` tiles go out as four quarters each (tiles of half the edge),
// first, so that later rounds start at different times on different CUs and the memory-bound
// epilogues of some run under the products of others.
constexpr int kMmSlots = 256;
constexpr int mm_sub(int tiles) {
  return tiles >= kMmSlots && tiles % kMmSlots <= kMmSlots / 4 ? tiles % kMmSlots : 0;
}
constexpr int mm_grid(int tiles) { return tiles + 3 * mm_sub(tiles); }
// Which tile a launch takes (1, 2 or 4: edges of 64, 128 or 256), by the time that each is expected
// to need for its number of tiles t and its K stages, in ns from measurements: a round of 768, 512
// or 256 workgroups (3, 2 or 1 on a CU) takes 640, 1000 or 1650 a stage; a last round takes less
// with fewer on a CU, down to 290 (one small tile on each), 620 and 1070 (few CUs busy draw less
// power); quarters take the time of middle tiles. Each round's epilogue takes about 2, 4 or 9 us. The
// time never falls as tiles are added.
// Examples (small, middle, large; us): 512^3 4.6, 6.5, 15.9; 1376 x 512 x 1000 6.9, 9.8, 23.5;
// 2048^3 29, 26, 41; 2048 x 1024 x 4096 27, 41, 70; 4096^3 -, 132, 113.
inline int mm_choose(int64_t t1, int64_t t2, int64_t t4, int64_t K, double* ns = nullptr) {
  const double st = (double)((K + kMmK - 1) / kMmK);
  auto part = [](int64_t t, int64_t cu) { return (t + cu - 1) / cu; };
  const int64_t r1 = t1 % 768, r2 = t2 % 512, r4 = t4 % kMmSlots;
  // a last round of r workgroups: one, then two, then three on a CU
  auto last = [](int64_t r, double one, double two, double three) {
    if (r == 0) return 0.0;
    if (r <= 256) return one;
    const double f = (double)(r <= 512 ? r - 256 : r - 512) / 256;
    return r <= 512 ? one + (two - one) * f : two + (three - two) * f;
  };
  const double c1 = st * (640 * (t1 / 768) + last(r1, 290, 430, 640)) + 2e3 * part(t1, 768);
  const double c2 = st * (1000 * (t2 / 512) + last(r2, 620, 1000, 1000)) + 4e3 * part(t2, 512);
  const bool quarters = t4 <= (1 << 30) && mm_sub((int)t4) > 0;
  const double c4 =
      st * (1650 * (t4 / kMmSlots) +
            (r4 == 0 ? 0 : quarters ? 620 : r4 > 252 ? 1650 : 1070 + 2.3 * r4)) +
      9e3 * part(t4, kMmSlots);
  if (ns != nullptr) *ns = c1 <= c2 && c1 <= c4 ? c1 : c2 <= c4 ? c2 : c4;
  return c1 <= c2 && c1 <= c4 ? 1 : c2 <= c4 ? 2 : 4;
}
// The same with K cut into `split` parts of whole stages where few small tiles leave CUs idle: a
// stage takes a workgroup 250 ns however few others run (fragment reads, loads and MFMAs of one wave
// per SIMD follow one another; a ring of five stages gains 15% there and costs launches of three
// workgroups on a CU 10%). mm_join then takes about 4 us and 0.5 us a part (a launch's 5
// products of 213 x 213 x 3490: 15 us each whole, 9.5 in five parts; 400 x 400 x 4000, two layers:
// 17 and 12). With the join of 128 x 128 sums, 15 us, no shape was faster cut.
inline int mm_choose_split(int64_t t1, int64_t t2, int64_t t4, int64_t K, int& split) {
  double best;
  int x = mm_choose(t1, t2, t4, K, &best);
  split = 1;
  const int64_t st = (K + kMmK - 1) / kMmK, none = int64_t(1) << 40;
  for (int s = 2; s <= kMmMaxSplit && t1 * s <= kMmParts; ++s) {
    const int64_t len = (st + s - 1) / s;
    if ((s - 1) * len >= st) continue;   // a part would be empty
    double ns;
    mm_choose(t1 * s, none, none, len * kMmK, &ns);
    ns += 4000 + 500 * s;
    if (ns < best) best = ns, x = 1, split = s;
  }
  return x;
}
// The tile of workgroup b of such a launch, and its quarter (-1: the whole tile).
__device__ __forceinline__ int mm_pick(int b, int tiles, int& quarter) {
  const int sub = mm_sub(tiles);
  if (b < 4 * sub) {
    quarter = b & 3;
    return tiles - sub + (b >> 2);
  }
  quarter = -1;
  return xcd_remap(b - 4 * sub, tiles - sub);
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
