// Rows of bf16 or fp32 values taken eight at a time, at any element's address, and sums over a wave: what
// the kernels that work along rows share.
#pragma once

#include "qg_device.hpp"

namespace qg {

// Eight elements from e on as fp32, at any element's address; elements at or past `left` are zero.
template <bool BF16>
struct RowRaw {
  uint4 q[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t e, int left) {
    if (left >= 8) {
      __builtin_memcpy(q, static_cast<const char*>(p) + e * (BF16 ? 2 : 4), sizeof(q));
      return;
    }
    uint32_t w[BF16 ? 4 : 8] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) {
        if constexpr (BF16)
          w[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(p)[e + i] << (16 * (i & 1));
        else
          w[i] = static_cast<const uint32_t*>(p)[e + i];
      }
    __builtin_memcpy(q, w, sizeof(q));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) {
      const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
      return __uint_as_float((i & 1) ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
    } else {
      const uint32_t u[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
      return __uint_as_float(u[i]);
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void row_store(void* p, int64_t e, int left, const float (&v)[8]) {
  if (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + e;
    if (left >= 8) {
      const uint4 w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      __builtin_memcpy(q, &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < left) q[i] = to_bf16(v[i]);
    }
  } else {
    float* q = static_cast<float*>(p) + e;
    if (left >= 8) {
      __builtin_memcpy(q, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < left) q[i] = v[i];
    }
  }
}

// Sum over the wave, in every lane: four steps within rows of 16 lanes, two across rows, by
// lane-shifted adds (no LDS round trips).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8: lane 15 of a row holds its sum
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3: lane 63 holds the wave's
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums over the W waves of one row (`first`: the row's first wave in the workgroup). Every wave of
// the workgroup calls it; `sh` is a different area from one call to the next but one.
template <int W>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* sh, int first) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (W == 1) return make_float2(a, b);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    s.x += sh[first + w].x;
    s.y += sh[first + w].y;
  }
  return s;
}

}  // namespace qg
