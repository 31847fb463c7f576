// FP8 quantization, value by value (OCP e4m3 and e5m2), as the quantizing kernels and the product of few
// rows share it:  s = max(amax / qmax, 2^-126),  q = rne(x (1 / s)).
#pragma once

#include "qg_device.hpp"

namespace qg {

template <int FMT>
struct F8 {
  // the largest finite value: 448 in e4m3, 57344 in e5m2
  static constexpr float kMax = FMT == 0 ? 448.0f : 57344.0f;
  // Four values as four codes. The converter rounds half to even; |v| passes kMax by at most 2^-22 of
  // itself, which rounds down to it. NaN keeps its code.
  static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    int w = 0;
    if constexpr (FMT == 0) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return (uint32_t)w;
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float (&v)[4]) {
    if constexpr (FMT == 0) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
      v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
    } else {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
      v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
    }
  }
  static __device__ __forceinline__ float scale(float amax) {
    return fmaxf(div_rn(amax, kMax), 0x1p-126f);
  }
};

// Maximum over each row of 16 lanes, in every lane, by lane rotations within the row.
__device__ __forceinline__ float row16_max(float v) {
  auto step = [&](auto ctrl) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(
                     0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  step(std::integral_constant<int, 0x128>{});
  step(std::integral_constant<int, 0x124>{});
  step(std::integral_constant<int, 0x122>{});
  step(std::integral_constant<int, 0x121>{});
  return v;
}

}  // namespace qg
