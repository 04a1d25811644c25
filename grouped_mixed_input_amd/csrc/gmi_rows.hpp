// gmi_rows.hpp -- what the row-wise kernels share: reductions over lanes,
// eight 16-bit columns at a time, fp8 codes with a scale per block of 128
// columns (16 neighbouring lanes), and an exponential to the last bits.
#pragma once

#include "gmi_device.hpp"

namespace gmi {

// max / sum over aligned groups of 16 lanes, result in every lane (quad swaps
// then half-row and row mirrors: four DPP moves, no LDS)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  return fmaxf(v, dpp<0x140>(v));
}
__device__ __forceinline__ float sum64(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = from_bits<DT>(v[i] & 0xffffu);
    f[2 * i + 1] = from_bits<DT>(v[i] >> 16);
  }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7])};
}

constexpr float kF8Max = 448.0f;

// One 16-byte access, or past the caches (NT).
template <bool NT>
__device__ __forceinline__ u32x4 load16(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load((const u32x4*)p);
  return *(const u32x4*)p;
}
template <bool NT, class V>
__device__ __forceinline__ void store(void* p, V v) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, (V*)p);
  else
    *(V*)p = v;
}

// fp8 codes of the quotients v / s, by the product with 1 / s and one
// correction from the remainder.  The product alone carries the reciprocal's
// rounding, which puts values on a border of two codes on either side of it.
// (0.3 us of 78 in the norm of 16384 x 4096; the full division takes 2.3.)
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], float s) {
  const bool finite = s < __builtin_inff();
  const float inv = 1.0f / s, den = finite ? s : 0.0f;  // v / inf: 0, without a remainder
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = v[e] * inv;
    t[e] = __builtin_fmaf(__builtin_fmaf(-t[e], den, v[e]), inv, t[e]);
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// Scale of a block from the largest magnitude of its 128 columns; the bound
// keeps that of an all-zero block a normal number.
__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax, kF8Max * 0x1p-126f) / kF8Max; }

// e^d for d <= 0 (0 for -infinity, NaN for NaN) as 2^t with t = d log2 e rounded,
// times e^(d - t ln 2), which is 1 + (d - t ln 2) to fp32.  2^t alone would carry
// t's rounding, d 2^-24 of the result (3e-6 at d = -40).  (16384 tokens x 128:
// routing 16.85 us, 16.65 without the factor and 17.2 with the library's expf;
// backward 5.65, 5.4 and 5.8.)
__device__ __forceinline__ float exp_le0(float d) {
  constexpr float LOG2E = 1.44269504f, LN2 = 0.693147182f, LN2_REST = -1.90465434e-9f;
  d = __builtin_elementwise_maximum(d, -104.0f);  // 2^-150, which is 0; an infinity would leave NaN below
  const float t = d * LOG2E;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, __builtin_fmaf(-LN2_REST, t, __builtin_fmaf(-LN2, t, d)), e);
}

}  // namespace gmi
