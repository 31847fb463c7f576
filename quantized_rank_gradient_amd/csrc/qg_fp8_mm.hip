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
//
// Precision: the accumulators are fp32. Inside the instruction, products of eight neighbouring values are
// added in fewer digits: each is cut off at 2^-13 of the largest one's power of two (measured, and so in
// the other FP8 instructions); the sums of eight are joined in fp32. That is 1e-5 of the result in the 2-norm
// for normally distributed values, 4e-5 where their sizes spread over e^3, beside the operands' own rounding of
// some 4e-2; the alternative is products in bf16 at half the rate.
//
// What bounds the large tiles: 64 KiB of operands a stage come through L2 and are written to LDS, 192 KiB read
// from there, beside 2048 cycles of MFMA a SIMD. Diagnostic copies of the loop (4096 x 4096 x 11008 with blocks,
// 207 us at the time): without the scaling 188, without loads 162, without LDS reads 130, without both 95. So the
// time is in the data's way into the registers, then in the scaling (with runs on both sides twice as many
// operations: 11008 x 4096 x 4096, median of rounds of 60 calls, 169 us with blocks, 197 with runs).
#include <algorithm>

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

// Four or eight consecutive results of one row, those behind the last column left out.
template <int N>
__device__ __forceinline__ void f8_store(const F8Mm& a, int64_t i, int64_t j, const float* v) {
  const int64_t left = a.N - j, at = i * a.N + j;
  if (a.bf16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
    if (left >= N) {
      uint32_t w[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      __builtin_memcpy(o, w, 2 * N);
    } else {
#pragma unroll
      for (int k = 0; k < N - 1; ++k)
        if (left > k) o[k] = to_bf16(v[k]);
    }
  } else {
    float* o = static_cast<float*>(a.out) + at;
    if (left >= N) {
      __builtin_memcpy(o, v, 4 * N);
    } else {
#pragma unroll
      for (int k = 0; k < N - 1; ++k)
        if (left > k) o[k] = v[k];
    }
  }
}

// A wave's 16 rows of 16 NJ results, a lane with 4 NJ consecutive ones of a row (`v`), leave as whole rows by
// way of LDS: 16-byte chunk c of row r in slot c ^ r (over the chunks of 256 bytes), so that neither side
// meets a bank twice. Written from the lanes that hold them, a store would touch 64 lines for 16 bytes each
// (4096 x 4096 x 4096: 94 us instead of 60).
template <int NJ, class Out>
__device__ __forceinline__ void f8_rows(const F8Mm& a, char* lds, int64_t i0, int64_t j0,
                                        const float (&v)[4 * NJ]) {
  constexpr int EACH = sizeof(Out), ROW = 16 * NJ * EACH, CH = ROW / 16, PER = 16 / EACH;
  constexpr int MINE = 4 * NJ / PER;   // chunks of this lane
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  auto slot = [](int r, int c) { return c ^ (r & (CH < 16 ? CH - 1 : 15)); };
#pragma unroll
  for (int q = 0; q < MINE; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = EACH == 2 ? pack_bf16x2(v[q * PER + (2 * k) % PER], v[q * PER + (2 * k + 1) % PER])
                       : __float_as_uint(v[q * PER + k % PER]);
    *reinterpret_cast<uint4*>(lds + l16 * ROW + 16 * slot(l16, g * MINE + q)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  Out* out = static_cast<Out*>(a.out);
#pragma unroll
  for (int q = 0; q < 16 * CH / 64; ++q) {
    const int r = (64 * q + lane) / CH, c = (64 * q + lane) % CH;
    const uint4 w = *reinterpret_cast<const uint4*>(lds + r * ROW + 16 * slot(r, c));
    const int64_t i = i0 + r, j = j0 + PER * c, left = a.N - j;
    if (i >= a.M) continue;
    Out* o = out + i * a.N + j;
    if (left >= PER) {
      __builtin_memcpy(o, &w, 16);
    } else {
      Out e[PER];
      __builtin_memcpy(e, &w, 16);
#pragma unroll
      for (int k = 0; k < PER - 1; ++k)
        if (left > k) o[k] = e[k];
    }
  }
}

}  // namespace

// WI x WJ waves, each NI x NJ blocks of 16 x 16: a tile of BI rows of A and BJ rows of B, in LDS NST stages
// (blocks of K) at a time. Lane group g's four rows of block jt are the wave's rows 4 NJ g + 4 jt + v, so
// that a lane's results of a row are 4 NJ consecutive columns.
// STEPS: the loop over K that goes by steps, or the ring of small tiles.
template <int WI_, int WJ_, int NI_, int NJ_, int NST_, bool STEPS_>
struct F8Tile {
  static constexpr bool STEPS = STEPS_;
  static constexpr int WI = WI_, WJ = WJ_, NI = NI_, NJ = NJ_, NST = NST_;
  static constexpr int WAVES = WI * WJ, THREADS = 64 * WAVES;
  static constexpr int BI = 16 * WI * NI, BJ = 16 * WJ * NJ;
  static constexpr int A_BYTES = BI * kF8Block, B_BYTES = BJ * kF8Block;
  // the scales' areas in a stage, and one for the loads of waves that have none to load
  static constexpr int SA = A_BYTES + B_BYTES, SB = SA + 4 * BI, NONE = SB + 4 * BJ;
  static constexpr int STAGE = NONE + 256;
  static constexpr int LDS = NST * STAGE;
  // workgroups on a CU that LDS leaves room for, as waves on a SIMD
  static constexpr int OCC = (160 * 1024 / LDS) * WAVES / 4;
};

// 16-byte chunk c of a row lies in slot c ^ swz(row): the 16 rows that a group of lanes reads at a time
// fall on all banks. Rows of A are read 16 in a row, rows of B four in a row from each of four groups.
__device__ __forceinline__ int swz_a(int row) { return (row >> 1) & 7; }
template <int NJ>
__device__ __forceinline__ int swz_b(int row) {
  return ((row >> 1) & 1) | (((row / (4 * NJ)) & 3) << 1);
}

// One stage's fragments, read from LDS.
template <class T, bool BBLOCK>
struct F8Reader {
  const char *a0, *a1, *b0, *b1;   // this lane's chunks g and g + 4 of the first fragment
  const char *sa, *sb;
  __device__ F8Reader(const char* lds, int wi, int wj) {
    const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
    const int ra = 16 * wi * T::NI + l16;
    const int rb = 16 * wj * T::NJ + 4 * T::NJ * (l16 >> 2) + (l16 & 3);
    // the swizzles of a fragment's rows are those of the first one's: 16 rows, and 4 rows, further on
    const char* pa = lds + ra * kF8Block;
    const char* pb = lds + T::A_BYTES + rb * kF8Block;
    a0 = pa + 16 * (g ^ swz_a(ra));
    a1 = pa + 16 * ((g + 4) ^ swz_a(ra));
    b0 = pb + 16 * (g ^ swz_b<T::NJ>(rb));
    b1 = pb + 16 * ((g + 4) ^ swz_b<T::NJ>(rb));
    sa = lds + T::SA + 4 * ra;
    sb = lds + T::SB + 4 * (BBLOCK ? 16 * wj * T::NJ / kF8Block : 16 * wj * T::NJ + 4 * T::NJ * g);
  }
  __device__ __forceinline__ v8i32 a(int st, int x) const {
    return join8(*reinterpret_cast<const uint4*>(a0 + st + 16 * kF8Block * x),
                 *reinterpret_cast<const uint4*>(a1 + st + 16 * kF8Block * x));
  }
  __device__ __forceinline__ v8i32 b(int st, int y) const {
    return join8(*reinterpret_cast<const uint4*>(b0 + st + 4 * kF8Block * y),
                 *reinterpret_cast<const uint4*>(b1 + st + 4 * kF8Block * y));
  }
  __device__ __forceinline__ float scale_a(int st, int x) const {
    return *reinterpret_cast<const float*>(sa + st + 64 * x);
  }
  __device__ __forceinline__ float scale_block(int st) const {
    return *reinterpret_cast<const float*>(sb + st);
  }
  __device__ __forceinline__ f32x4 scale_b(int st, int y) const {
    return *reinterpret_cast<const f32x4*>(sb + st + 16 * y);
  }
};

// The loads of a workgroup's stages: LOADS for each wave and stage.
template <class T, bool BBLOCK>
struct F8Loader {
  // The loads of codes take 8 rows each: this lane's chunk and offset in the wave's first one and wherever
  // the swizzle changes (A: with every second load; B: every NJ / 2); the others lie a multiple of 8 rows
  // further on. Rows behind the last one are behind the resource's end.
  static constexpr int PA = T::BI / (8 * T::WAVES), PB = T::BJ / (8 * T::WAVES);
  static constexpr int LOADS = PA + PB + 1;
  static constexpr int CA = PA < 2 ? PA : 2, H = T::NJ < 2 ? 1 : T::NJ / 2, CB = PB / H;
  static_assert(PA % CA == 0 && CB * H == PB && PA > 0 && PB > 0, "whole periods of the swizzles");
  const uint8_t *pa, *pb;
  const float* ps;        // the wave's scales of a stage, 64 in one load; those behind the last are zeros
  int64_t each;           // how far the next stage's lie
  uint32_t pitch, bytes_a, bytes_b, bytes_s, ts;
  int first, nk, wave;    // the first block of K, and how many
  uint32_t ka[CA], kb[CB], va[CA], vb[CB];
  // of the stage that is being loaded
  uint32_t left, to;
  v4i32 ra, rb, rs;

  __device__ F8Loader(const F8Mm& a, int64_t i0, int64_t j0, int first_, int nk_, int wave_)
      : first(first_), nk(nk_), wave(wave_) {
    const int lane = threadIdx.x & 63;
    const int64_t rows_a = a.M - i0 < T::BI ? a.M - i0 : T::BI;
    const int64_t rows_b = a.N - j0 < T::BJ ? a.N - j0 : T::BJ;
    pitch = (uint32_t)f8_pitch(a.K);   // at most 2^20, so that a tile's offsets stay below 2^28
    pa = a.A + i0 * pitch;
    pb = a.B + j0 * pitch;
    bytes_a = (uint32_t)rows_a * pitch;
    bytes_b = (uint32_t)rows_b * pitch;
#pragma unroll
    for (int u = 0; u < CA; ++u) {
      const uint32_t row = 8 * (wave * PA + u) + (lane >> 3);
      ka[u] = 16 * ((lane & 7) ^ swz_a(row));
      va[u] = row * pitch + ka[u];
    }
#pragma unroll
    for (int u = 0; u < CB; ++u) {
      const uint32_t row = 8 * (wave * PB + u * H) + (lane >> 3);
      kb[u] = 16 * ((lane & 7) ^ swz_b<T::NJ>(row));
      vb[u] = row * pitch + kb[u];
    }
    constexpr int LA = (T::BI + 63) / 64, LB = BBLOCK ? 1 : (T::BJ + 63) / 64;
    static_assert(T::WAVES >= LA + LB, "a wave for each load of scales");
    int64_t ns = 0;
    ps = a.sa;
    each = 0;
    ts = T::NONE;
    if (wave < LA) {
      ps = a.sa + i0 + 64 * wave, ns = rows_a - 64 * wave, each = a.M, ts = T::SA + 256 * wave;
    } else if (wave < LA + LB) {
      const int w = wave - LA;
      if constexpr (BBLOCK)
        ps = a.sb + j0 / kF8Block, each = f8_blocks(a.N), ns = each - j0 / kF8Block, ts = T::SB;
      else
        ps = a.sb + j0 + 64 * w, ns = rows_b - 64 * w, each = a.N, ts = T::SB + 256 * w;
    }
    bytes_s = (uint32_t)(ns > 64 ? 64 : ns > 0 ? ns : 0) * 4;
  }
  // Turns to stage kt, which goes to LDS byte address to_. One behind the last reads nothing, without a
  // branch, so that a loop around it is one block.
  __device__ __forceinline__ void open(int kt, uint32_t to_) {
    const bool on = kt < nk;
    const uint32_t k0 = on ? (uint32_t)(first + kt) * kF8Block : pitch;
    left = pitch - k0;
    to = to_;
    ra = rsrc_words(pa + k0, bytes_a - k0);
    rb = rsrc_words(pb + k0, bytes_b - k0);
    rs = rsrc_words(ps + (on ? first + kt : 0) * each, on ? bytes_s : 0);
  }
  template <int L>
  __device__ __forceinline__ void load() const {
    if constexpr (L < PA) {
      const uint32_t off = va[L % CA] + (L / CA * CA) * 8 * pitch;
      dma16(ra, ka[L % CA] < left ? off : kOOB, to + 1024 * (wave * PA + L));
    } else if constexpr (L < PA + PB) {
      constexpr int u = L - PA;
      const uint32_t off = vb[u / H] + (u % H) * 8 * pitch;
      dma16(rb, kb[u / H] < left ? off : kOOB, to + T::A_BYTES + 1024 * (wave * PB + u));
    } else {
      dma4(rs, 4 * (threadIdx.x & 63), to + ts);
    }
  }
  __device__ __forceinline__ void issue(int kt, uint32_t to_) {
    open(kt, to_);
    static_for<LOADS>([&](auto l) { load<decltype(l)::value>(); });
  }
};

// to += p, scaled by s (BBLOCK) or by s and the four rows' own scales.
template <bool BBLOCK>
__device__ __forceinline__ void f8_add(f32x4& to, const f32x4& p, float s, const f32x4& rows) {
#pragma unroll
  for (int v = 0; v < 4; ++v) to[v] = __builtin_fmaf(p[v], BBLOCK ? s : s * rows[v], to[v]);
}

// A step is one fragment of B against the wave's NI fragments of A. Its MFMAs go out one by one, beside each
// the scaling of a result of the step before, and the reads of the next step's fragment; the last step of a
// stage reads the next stage's fragments, each of A where its last MFMA has taken it. So the workgroup meets
// in front of that step: all it still needs of the stage is in registers, and the stage's buffer is free for
// the loads of the stage after the next, which go out beside the MFMAs of two steps (4096 x 4096 x 11008:
// 203 us with one step, 184 with two, 192 with three or more: the last ones come too late). The order is
// fixed: left to itself the compiler puts each scaling right behind its MFMA and waits for it. Alone on a CU,
// a workgroup has nothing else to do while its loads are on their way, so that three stages pay there
// (1024 x 4096 x 4096 in tiles of 128 with 8 waves: 27.8 us with two stages, 22.5 with three, 22.7 with four).
template <class T, int AF, bool BBLOCK>
__device__ __forceinline__ void f8_kloop_steps(F8Loader<T, BBLOCK>& ld, const F8Reader<T, BBLOCK>& rd,
                                               uint32_t base, f32x4 (&acc)[T::NJ][T::NI]) {
  constexpr int NI = T::NI, NJ = T::NJ, NST = T::NST;
  static_assert(NJ % 2 == 0, "fragments of B and results alternate between two sets");
  f32x4 part[2][NI], sb[2];
  v8i32 fa[NI], fb[2];
  float sc[NI], sp[NI];   // the stage's scales of A (with the block's), and those of the stage before
#pragma unroll
  for (int x = 0; x < NI; ++x) {
    part[1][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    sp[x] = 0.0f;
  }
  sb[0] = sb[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto fetch_scales = [&](int st) {
    float block = 1.0f;
    if constexpr (BBLOCK) block = rd.scale_block(st);
#pragma unroll
    for (int x = 0; x < NI; ++x) sc[x] = BBLOCK ? rd.scale_a(st, x) * block : rd.scale_a(st, x);
  };
  constexpr int SPREAD = 2, GROUPS = SPREAD * NI, LOADS = F8Loader<T, BBLOCK>::LOADS;
  auto loads_of = [&](auto gc) {   // beside MFMA gc of those steps
    constexpr int lo = decltype(gc)::value * LOADS / GROUPS;
    constexpr int hi = (decltype(gc)::value + 1) * LOADS / GROUPS;
    static_for<hi - lo>([&](auto l) { ld.template load<lo + decltype(l)::value>(); });
  };
  for (int s = 0; s < NST - 1; ++s) ld.issue(s, base + s * T::STAGE);
  wait_vm_lds<(NST - 2) * LOADS>();
  barrier_nofence();
  ld.open(NST - 1, base + (NST - 1) * T::STAGE);
  static_for<NI>([&](auto x) { loads_of(x); });
#pragma unroll
  for (int x = 0; x < NI; ++x) fa[x] = rd.a(0, x);
  fb[0] = rd.b(0, 0);
  if constexpr (!BBLOCK) sb[0] = rd.scale_b(0, 0);
  fetch_scales(0);
  int st = 0;
  for (int kt = 0; kt < ld.nk; ++kt) {
    const int next = st == (NST - 1) * T::STAGE ? 0 : st + T::STAGE;
    static_for<NJ>([&](auto yc) {
      constexpr int y = decltype(yc)::value, cur = y & 1, old = cur ^ 1, yo = (y + NJ - 1) % NJ;
      constexpr int step = (y + 1) % NJ;   // from the one on that frees the stage's buffer
      if constexpr (y == NJ - 1) {
        wait_vm_lds<(NST - 2) * LOADS>();   // this wave's part of the next stage has come,
        barrier_nofence();                  // and every wave's, and none still reads this stage
        ld.open(kt + NST, base + st);
      }
      static_for<NI>([&](auto xc) {
        constexpr int x = decltype(xc)::value;
        part[cur][x] = f8_mfma<AF>(fb[cur], fa[x]);
        // behind the last stage this reads what is not used
        if constexpr (x == 0) fb[old] = y < NJ - 1 ? rd.b(st, y + 1) : rd.b(next, 0);
        if constexpr (y == NJ - 1) fa[x] = rd.a(next, x);
        if constexpr (step < SPREAD) loads_of(std::integral_constant<int, step * NI + x>{});
        f8_add<BBLOCK>(acc[yo][x], part[old][x], y == 0 ? sp[x] : sc[x], sb[old]);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (!BBLOCK) sb[old] = y < NJ - 1 ? rd.scale_b(st, y + 1) : rd.scale_b(next, 0);
      if constexpr (y == NJ - 1) {
#pragma unroll
        for (int x = 0; x < NI; ++x) sp[x] = sc[x];
        fetch_scales(next);
      }
    });
    st = next;
  }
#pragma unroll
  for (int x = 0; x < NI; ++x) f8_add<BBLOCK>(acc[NJ - 1][x], part[1][x], sp[x], sb[1]);
}

// Small tiles: a ring of NST stages, NST - 1 of them loading while one is multiplied. Stages behind the last
// one read nothing, so that every stage has as many loads to wait for.
template <class T, int AF, bool BBLOCK>
__device__ __forceinline__ void f8_kloop_ring(F8Loader<T, BBLOCK>& ld, const F8Reader<T, BBLOCK>& rd,
                                              uint32_t base, f32x4 (&acc)[T::NJ][T::NI]) {
  constexpr int NI = T::NI, NJ = T::NJ, NST = T::NST, LOADS = F8Loader<T, BBLOCK>::LOADS;
  for (int s = 0; s < NST - 1; ++s) ld.issue(s, base + s * T::STAGE);
  int st = 0, free = (NST - 1) * T::STAGE;
  for (int kt = 0; kt < ld.nk; ++kt) {
    wait_vm_lds<(NST - 2) * LOADS>();   // this wave's part of the stage has come,
    barrier_nofence();                  // and every wave's, and none still reads the one before it
    v8i32 fa[NI], fb[NJ];
    f32x4 sb[NJ];
    float sc[NI], block = 1.0f;
    if constexpr (BBLOCK) block = rd.scale_block(st);
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      fa[x] = rd.a(st, x);
      sc[x] = rd.scale_a(st, x) * block;
    }
#pragma unroll
    for (int y = 0; y < NJ; ++y) {
      fb[y] = rd.b(st, y);
      sb[y] = BBLOCK ? f32x4{1.0f, 1.0f, 1.0f, 1.0f} : rd.scale_b(st, y);
    }
    ld.issue(kt + NST - 1, base + free);
    f32x4 part[NJ][NI];
#pragma unroll
    for (int y = 0; y < NJ; ++y)
#pragma unroll
      for (int x = 0; x < NI; ++x) part[y][x] = f8_mfma<AF>(fb[y], fa[x]);
#pragma unroll
    for (int y = 0; y < NJ; ++y)
#pragma unroll
      for (int x = 0; x < NI; ++x) f8_add<BBLOCK>(acc[y][x], part[y][x], sc[x], sb[y]);
    free = st;
    st = st == (NST - 1) * T::STAGE ? 0 : st + T::STAGE;
  }
}

// Tile `at` of tm x tn of a product, or of a part of `per` blocks of K: the parts' tiles one part behind another.
template <class T, int AF, bool BBLOCK>
__device__ __forceinline__ void f8_tile(const F8Mm& a, int at, int tm, int tn, int per, uint16_t* lds) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / T::WJ, wj = wave % T::WJ;
  const int blocks = (int)f8_blocks(a.K), part = at / (tm * tn), first = part * per;
  int ti, tj;
  mm_band(xcd_remap(at - part * (tm * tn), tm * tn), tm, tn, ti, tj);
  const int64_t i0 = (int64_t)ti * T::BI, j0 = (int64_t)tj * T::BJ;
  F8Mm o = a;   // where the results go
  if (per < blocks) {
    o.out = a.part + part * f8_part_stride(a.M, a.N);
    o.bf16 = 0;
  }
  F8Loader<T, BBLOCK> ld(a, i0, j0, first, blocks - first < per ? blocks - first : per, wave);
  const F8Reader<T, BBLOCK> rd(reinterpret_cast<const char*>(lds), wi, wj);
  f32x4 acc[T::NJ][T::NI];
#pragma unroll
  for (int y = 0; y < T::NJ; ++y)
#pragma unroll
    for (int x = 0; x < T::NI; ++x) acc[y][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (T::STEPS)
    f8_kloop_steps<T, AF, BBLOCK>(ld, rd, lds_addr(lds), acc);
  else
    f8_kloop_ring<T, AF, BBLOCK>(ld, rd, lds_addr(lds), acc);
  // the last stages' loads have ended, and no wave still reads, before the LDS is used again
  wait_vm_lds<0>();
  __syncthreads();
  const int g = (threadIdx.x & 63) >> 4, l16 = threadIdx.x & 15;
#pragma unroll
  for (int x = 0; x < T::NI; ++x) {
    const int64_t i = i0 + 16 * (wi * T::NI + x), j = j0 + 16 * wj * T::NJ;
    float v[4 * T::NJ];
#pragma unroll
    for (int y = 0; y < T::NJ; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * y + e] = acc[y][x][e];
    if constexpr (T::NJ >= 4) {
      char* mine = reinterpret_cast<char*>(lds) + wave * (16 * 16 * T::NJ * 4);
      if (o.bf16)
        f8_rows<T::NJ, uint16_t>(o, mine, i, j, v);
      else
        f8_rows<T::NJ, float>(o, mine, i, j, v);
    } else if (i + l16 < a.M) {
      f8_store<4 * T::NJ>(o, i + l16, j + 4 * T::NJ * g, v);
    }
  }
}

template <class T, int AF, bool BBLOCK>
__global__ __launch_bounds__(T::THREADS, T::OCC) void qg_f8_mm(F8Mm a, int tm, int tn, int per) {
  __shared__ alignas(1024) uint16_t lds[T::LDS / 2];
  f8_tile<T, AF, BBLOCK>(a, blockIdx.x, tm, tn, per, lds);
}
// out = the parts' sums, added from the first on.
__global__ __launch_bounds__(256) void qg_f8_join(F8Mm a, int parts) {
  const int64_t numel = a.M * a.N, stride = f8_part_stride(a.M, a.N);
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= numel) return;
  f32x4 q[kF8Parts];
#pragma unroll
  for (int p = 0; p < kF8Parts; ++p)   // up to the stride there is memory behind the last value
    if (p < parts) q[p] = *reinterpret_cast<const f32x4*>(a.part + p * stride + at);
#pragma unroll
  for (int p = 1; p < kF8Parts; ++p)
    if (p < parts) {
#pragma unroll
      for (int v = 0; v < 4; ++v) q[0][v] += q[p][v];
    }
  if (a.bf16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
    if (numel - at >= 4) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(q[0][0], q[0][1]), pack_bf16x2(q[0][2], q[0][3]));
    } else {
#pragma unroll
      for (int v = 0; v < 3; ++v)
        if (numel - at > v) o[v] = to_bf16(q[0][v]);
    }
  } else {
    float* o = static_cast<float*>(a.out) + at;
    if (numel - at >= 4) {
      *reinterpret_cast<f32x4*>(o) = q[0];
    } else {
#pragma unroll
      for (int v = 0; v < 3; ++v)
        if (numel - at > v) o[v] = q[0][v];
    }
  }
}
// Two products of one launch, the first with blocks, the second with runs on its right side: both are small,
// and a launch would take as long as one of them.
template <class T, int AF>
__global__ __launch_bounds__(T::THREADS, T::OCC) void qg_f8_mm_pair(F8Mm a, F8Mm b, int tma, int tna, int tmb,
                                                                   int tnb) {
  __shared__ alignas(1024) uint16_t lds[T::LDS / 2];
  const int n = tma * tna;
  if ((int)blockIdx.x < n)
    f8_tile<T, AF, true>(a, blockIdx.x, tma, tna, (int)f8_blocks(a.K), lds);
  else
    f8_tile<T, AF, false>(b, blockIdx.x - n, tmb, tnb, (int)f8_blocks(b.K), lds);
}

// Few rows of A (up to 16 NT): a workgroup takes 16 rows of B, its KW waves the blocks of K in turn, each from
// memory straight into the MFMA's registers, U blocks on their way at a time. B's bytes bound it, and with
// more than 16 rows those of A, which every workgroup reads. With QUANT the rows of A come as bf16 values
// (a.X) and are quantized into LDS first, by the whole workgroup (a row of 16 lanes for a run), while the
// first blocks of B are on their way: a launch less, and every value once for a workgroup instead of once
// for each of its waves. One token through 11008 x 4096 (45 MB): 11.8 us with 16 waves, 13.3 with 8; with
// 32 rows of B for a workgroup 14.2 (16 waves, 344 workgroups). K = 4096 is one batch of KW U blocks; a longer K
// waits for memory anew with each further one, and its weight has fewer rows for the CUs: 4096 x 11008 (45 MB,
// three batches, 256 workgroups) 14.9.
template <int NT, int KW, int U, int AF, bool BBLOCK, bool QUANT>
__global__ __launch_bounds__(64 * KW) void qg_f8_few(F8Mm a) {
  extern __shared__ uint4 few_codes[];
  uint8_t* codes = reinterpret_cast<uint8_t*>(few_codes);
  __shared__ f32x4 sum[KW][NT][64];
  static_assert(NT == 1 || !QUANT, "rows that are quantized here are one tile");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t j0 = (int64_t)blockIdx.x * 16, nb = f8_blocks(a.N);
  const int pitch = (int)f8_pitch(a.K), nk = (int)f8_blocks(a.K), M = (int)a.M;
  // QUANT: M rows of whole blocks (16 bytes apart on the banks), and behind them the scales
  const int row_bytes = nk * kF8Block + 16;
  float* scales = reinterpret_cast<float*>(codes + (QUANT ? M * row_bytes : 0));
  auto chunk = [&](const uint8_t* p, bool on, int k) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (on && k < pitch) w = *reinterpret_cast<const uint4*>(p + k);
    return w;
  };
  const uint8_t* pb = a.B + (j0 + l16) * pitch;
  const bool on_b = j0 + l16 < a.N;
  v8i32 fb[U];
  auto fetch = [&](int kt0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (kt0 + KW * u) * kF8Block + 16 * g;
      fb[u] = join8(chunk(pb, on_b, k), chunk(pb, on_b, k + 64));
    }
  };
  fetch(wave);
  if constexpr (QUANT) {
    constexpr int AT = 4;   // runs of a row of lanes on their way at a time
    const int runs = M * nk;
    for (int run0 = threadIdx.x >> 4; run0 < runs; run0 += 4 * KW * AT) {
      RowRaw<true> x[AT];
#pragma unroll
      for (int q = 0; q < AT; ++q) {
        const int run = run0 + 4 * KW * q, t = run / nk, c = (run - t * nk) * kF8Block + 8 * l16;
        x[q] = {};
        if (run < runs && c < a.K) x[q].load(a.X, t * a.K + c, (int)a.K - c);
      }
#pragma unroll
      for (int q = 0; q < AT; ++q) {
        const int run = run0 + 4 * KW * q, t = run / nk, kt = run - t * nk;
        if (run >= runs) continue;   // the same for 16 lanes
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[q].get(i)));
        const float s = F8<AF>::scale(row16_max(m)), inv = div_rn(1.0f, s);
        *reinterpret_cast<uint2*>(codes + t * row_bytes + kt * kF8Block + 8 * l16) = make_uint2(
            F8<AF>::pack4(x[q].get(0) * inv, x[q].get(1) * inv, x[q].get(2) * inv, x[q].get(3) * inv),
            F8<AF>::pack4(x[q].get(4) * inv, x[q].get(5) * inv, x[q].get(6) * inv, x[q].get(7) * inv));
        if (l16 == 0) scales[t * nk + kt] = s;
      }
    }
    __syncthreads();
  }
  f32x4 acc[NT];
#pragma unroll
  for (int x = 0; x < NT; ++x) acc[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kt0 = wave; kt0 < nk; kt0 += KW * U) {
    if (kt0 != wave) fetch(kt0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = kt0 + KW * u;
      if (kt >= nk) continue;   // the same for the whole wave
      const int k = kt * kF8Block + 16 * g;
      f32x4 rows;
      if constexpr (BBLOCK) {
        const float sb = a.sb[kt * nb + j0 / kF8Block];
        rows = f32x4{sb, sb, sb, sb};
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t j = j0 + 4 * g + v;
          rows[v] = j < a.N ? a.sb[(int64_t)kt * a.N + j] : 0.0f;
        }
      }
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int i = 16 * x + l16;
        const bool on = i < M;
        v8i32 fa;
        float s = 0.0f;
        if constexpr (QUANT) {
          uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
          if (on) {
            lo = *reinterpret_cast<const uint4*>(codes + i * row_bytes + k);
            hi = *reinterpret_cast<const uint4*>(codes + i * row_bytes + k + 64);
            s = scales[i * nk + kt];
          }
          fa = join8(lo, hi);
        } else {
          const uint8_t* p = a.A + (int64_t)i * pitch;
          fa = join8(chunk(p, on, k), chunk(p, on, k + 64));
          if (on) s = a.sa[(int64_t)kt * M + i];
        }
        f8_add<false>(acc[x], f8_mfma<AF>(fb[u], fa), s, rows);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x) sum[wave][x][lane] = acc[x];
  __syncthreads();
  static_assert(NT <= KW, "a wave for each of the tiles");
  if (wave >= NT) return;
  f32x4 o = sum[0][wave][lane];
#pragma unroll
  for (int w = 1; w < KW; ++w) {
    const f32x4 q = sum[w][wave][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] += q[v];
  }
  const int64_t i = 16 * wave + l16, j = j0 + 4 * g;
  if (i >= a.M || j >= a.N) return;
  const float v[4] = {o[0], o[1], o[2], o[3]};
  f8_store<4>(a, i, j, v);
}

namespace {

template <class T, int AF, bool BBLOCK>
hipError_t f8_tiles(const F8Mm& a, int per, hipStream_t s) {
  const int tm = (int)((a.M + T::BI - 1) / T::BI), tn = (int)((a.N + T::BJ - 1) / T::BJ);
  const int parts = ((int)f8_blocks(a.K) + per - 1) / per;
  hipLaunchKernelGGL((qg_f8_mm<T, AF, BBLOCK>), dim3((unsigned)(tm * tn * parts)), dim3(T::THREADS), 0, s, a,
                     tm, tn, per);
  if (parts > 1)
    hipLaunchKernelGGL(qg_f8_join, dim3((unsigned)((a.M * a.N + 1023) / 1024)), dim3(256), 0, s, a, parts);
  return hipGetLastError();
}

// Which tile (1, 2, 3 or 4: edges of 64, 128, 128 with a CU of its own, or 256) a product takes, by the time
// that each is expected to need for its number of tiles t and its blocks of K, in us from measurements: a
// round of 512, 512, 256 or 256 workgroups (2, 2, 1 or 1 on a CU) takes 0.45, 1.12, 0.6 or 1.85 a block; a last
// round takes less with fewer on a CU, down to 0.26, 0.75, 0.5 and 1.2.
// Examples (1, 2, 3, 4; us): 64 x 11008 x 4096 12.5, 27, 20, 43; 256 x 11008 x 4096 27, 28, 21, 44;
// 512 x 4096 x 4096 18, 27, 20, 44; 1024 x 4096 x 4096 32, 28, 22.5, 45; 512 x 11008 x 4096 47, 35, 39, 47;
// 4096 x 4096 x 11008 312, 189, 219, 163.
// With fewer tiles than places on the card, K may be cut into parts of `per` blocks, whose sums a launch of its
// own adds (3 us and their bytes, at 4 TB/s there and back). Without and with parts, us: 64 x 4096 x 11008 27.0
// and 14.7, 128 of them 27.8 and 20.5; runs on both sides, 512 x 512 x 32768 87 and 31, 512 x 1376 x 32768 88
// and 44, 512 x 512 x 4096 13.6 and 10.3; 256 x 4096 x 11008 28.6 and no less.
struct F8Choice {
  int edge;
  int64_t per;
  double us;
};
F8Choice f8_choose(const F8Mm& a) {
  const int64_t M = a.M, N = a.N, st = f8_blocks(a.K);
  auto tiles = [&](int64_t e) { return ((M + e - 1) / e) * ((N + e - 1) / e); };
  auto cost = [&](int64_t t, int64_t blocks, int64_t slots, double one, double full, double each) {
    const int64_t r = t % slots;
    const double part = (double)(r > 256 ? r - 256 : 0) / 256;
    const double last = r == 0 ? 0.0 : slots == 256 ? one + (full - one) * (double)r / 256
                                                    : one + (full - one) * part;
    return (double)blocks * (full * (double)(t / slots) + last) + each * (double)((t + slots - 1) / slots);
  };
  F8Choice best{1, st, cost(tiles(64), st, 512, 0.26, 0.45, 3)};
  auto take = [&](int edge, int64_t per, double us) {
    if (us < best.us) best = {edge, per, us};
  };
  take(3, st, cost(tiles(128), st, 256, 0.5, 0.6, 3));
  take(2, st, cost(tiles(128), st, 512, 0.75, 1.12, 3));
  take(4, st, cost(tiles(256), st, 256, 1.2, 1.85, 4));
  if (a.part == nullptr || f8_part_bytes(M, N, a.K) == 0) return best;
  for (int64_t parts = 2; parts <= kF8Parts && st / parts >= kF8PartBlocks; ++parts) {
    const int64_t per = (st + parts - 1) / parts, p = (st + per - 1) / per;
    const double join = 3 + (double)(8 * p * M * N) / 4e6;
    if (tiles(64) * p <= 512) take(1, per, join + cost(tiles(64) * p, per, 512, 0.26, 0.45, 3));
    if (tiles(128) * p <= 256) take(3, per, join + cost(tiles(128) * p, per, 256, 0.5, 0.6, 3));
  }
  return best;
}
// Whether up to 64 rows go by rows of B: its bytes once, and those of A for every 16 rows of B, or where these
// are few what one CU streams (37 to 51 bytes a ns), against the time of the tiles. By rows and by tiles (with
// parts of K), us: 24 rows x 4096 x 11008 16.8 and 15.7, 17 x 4096 x 4096 with the quantization in front 11.7
// and 15.2, 64 x 512 x 11008 26.3 and 9.5, 40 x 300 x 60000 74 and 22. Up to 16 rows are not compared: with the
// quantization in front 16 tokens x 11008 x 4096 take 20.8 us by rows, where 17, by tiles, take 18.6.
bool f8_few_wins(int64_t M, int64_t N, int64_t K, double tiles_us) {
  if (M <= 16) return true;
  const double b = (double)(N * K), a = (double)(N * K) / 16 * (double)M;
  const double all = b / 4.93e6 + a / 8.3e6, one = (double)K * (double)(M + 16) / 45e3;
  return M <= 64 && 2.7 + std::max(all, one) < tiles_us;
}

// The small tiles, and what they cover.
using F8Small = F8Tile<2, 2, 2, 2, 4, false>;
int small_tiles(int64_t n) { return (int)((n + F8Small::BI - 1) / F8Small::BI); }
bool f8_small(const F8Mm& a) {
  const F8Choice c = f8_choose(a);
  return c.edge == 1 && c.per == f8_blocks(a.K) && !f8_few_wins(a.M, a.N, a.K, c.us);
}

template <int AF>
hipError_t f8_pair(const F8Mm& a, const F8Mm& b, hipStream_t s) {
  const int tma = small_tiles(a.M), tna = small_tiles(a.N), tmb = small_tiles(b.M), tnb = small_tiles(b.N);
  hipLaunchKernelGGL((qg_f8_mm_pair<F8Small, AF>), dim3((unsigned)(tma * tna + tmb * tnb)),
                     dim3(F8Small::THREADS), 0, s, a, b, tma, tna, tmb, tnb);
  return hipGetLastError();
}

template <int AF, bool BBLOCK>
hipError_t f8_mm(const F8Mm& a, hipStream_t s) {
  auto few = [&](auto nt, auto quant) {
    constexpr int NT = decltype(nt)::value, KW = 16, U = 2;
    constexpr bool QUANT = decltype(quant)::value;
    hipLaunchKernelGGL((qg_f8_few<NT, KW, U, AF, BBLOCK, QUANT>), dim3((unsigned)((a.N + 15) / 16)),
                       dim3(64 * KW), QUANT ? (unsigned)f8_few_lds(a.M, a.K) : 0, s, a);
    return hipGetLastError();
  };
  using std::integral_constant;
  if (a.X != nullptr) return few(integral_constant<int, 1>{}, std::true_type{});
  const F8Choice c = f8_choose(a);
  if (f8_few_wins(a.M, a.N, a.K, c.us)) {
    if (a.M <= 16) return few(integral_constant<int, 1>{}, std::false_type{});
    if (a.M <= 32) return few(integral_constant<int, 2>{}, std::false_type{});
    return few(integral_constant<int, 4>{}, std::false_type{});
  }
  const int per = (int)c.per;
  if (c.edge == 4) return f8_tiles<F8Tile<4, 2, 4, 8, 2, true>, AF, BBLOCK>(a, per, s);
  if (c.edge == 3) return f8_tiles<F8Tile<4, 2, 2, 4, 3, true>, AF, BBLOCK>(a, per, s);
  if (c.edge == 2) return f8_tiles<F8Tile<2, 2, 4, 4, 2, true>, AF, BBLOCK>(a, per, s);
  return f8_tiles<F8Small, AF, BBLOCK>(a, per, s);
}

}  // namespace

hipError_t launch_f8_mm_pair(const F8Mm& a, const F8Mm& b, hipStream_t s) {
  if (f8_small(a) && f8_small(b) && a.a_format == b.a_format && a.b_block && !b.b_block)
    return a.a_format == kF8E4M3 ? f8_pair<0>(a, b, s) : f8_pair<1>(a, b, s);
  const hipError_t e = launch_f8_mm(a, s);
  return e == hipSuccess ? launch_f8_mm(b, s) : e;
}

hipError_t launch_f8_mm(const F8Mm& a, hipStream_t s) {
  if (a.a_format == kF8E4M3) return a.b_block ? f8_mm<0, true>(a, s) : f8_mm<0, false>(a, s);
  return a.b_block ? f8_mm<1, true>(a, s) : f8_mm<1, false>(a, s);
}

}  // namespace qg
