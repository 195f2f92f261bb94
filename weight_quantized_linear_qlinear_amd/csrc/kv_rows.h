// Rows of K and V on their way into a cache: what the kernels that write and read entries share.
//
// The 4-bit form.  A row of D channels (D a multiple of 32) is e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6
// and a sign) with an fp16 scale per group of 32 channels:
//   s = fp16(fp32(absmax / 6)), 1 for an all-zero group, 2^-24 where a positive absmax would round to 0,
//       65504 where it would pass that, NaN where the group holds a NaN or an infinity
//   code = e2m1(x / s), round to nearest, ties to even, saturating at 6
// Its D / 2 bytes lie as the attention kernels want them: the groups in runs of P = 8, 4, 2 or 1, the
// largest that fits each time (D = 96: 2, 1); byte c P + g of a run (c < 16) is channels 2 c (low nibble)
// and 2 c + 1 of the run's group g.  So the four bytes per group that a lane needs of K, and the byte
// per group that it needs of V, lie side by side.
#pragma once

#include "qlq_device.h"

namespace qlq {

__device__ __forceinline__ uint32_t kv_f16_scale(float absmax, float qmax) {   // the 8-bit codec's rule
  if (absmax == 0.0f) return 0x3C00u;
  const float c = __builtin_amdgcn_fmed3f(absmax / qmax, 65504.0f, -65504.0f);
  const uint32_t s = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)c);
  return s == 0u ? 1u : s;
}

__device__ __forceinline__ float f16_value(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

__device__ __forceinline__ int64_t load_index(const void* p, int is64, int64_t i) {
  return is64 ? static_cast<const int64_t*>(p)[i] : (int64_t)static_cast<const int32_t*>(p)[i];
}

// Eight bf16 at p (any alignment unless vec).
__device__ __forceinline__ u32x4 load8(const uint16_t* p, bool vec) {
  if (vec) return ld16(p);
  u32x4 r;
  r.x = p[0] | ((uint32_t)p[1] << 16);
  r.y = p[2] | ((uint32_t)p[3] << 16);
  r.z = p[4] | ((uint32_t)p[5] << 16);
  r.w = p[6] | ((uint32_t)p[7] << 16);
  return r;
}

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf16_bits_to_f32(d[e] & 0xFFFF);
    f[2 * e + 1] = bf16_bits_to_f32(d[e] >> 16);
  }
}

// Scale of a 4-bit group from its largest magnitude / 6 (zero: all of it; bad: a NaN or an infinity in it).
__device__ __forceinline__ uint32_t kv4_f16_scale(float am6, bool zero, bool bad) {
  if (bad) return 0x7E00u;
  if (zero) return 0x3C00u;
  const uint32_t s = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)__builtin_amdgcn_fmed3f(am6, 65504.0f, -65504.0f));
  return s == 0u ? 1u : s;
}

// Two quotients -> the codes of a byte (low nibble first), saturating.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2_sat(float a, float b) {
  a = __builtin_amdgcn_fmed3f(a, 6.0f, -6.0f);
  b = __builtin_amdgcn_fmed3f(b, 6.0f, -6.0f);
  return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, 1.0f, 0) & 0xFFu;
}

// Where a group's bytes lie in a 4-bit row of NG groups: byte first + c * step, c < 16.
struct Kv4Run {
  int first, step;
};
__device__ __forceinline__ Kv4Run kv4_run(int NG, int g) {
  int at = 0, P = 8;
  while (NG - at < P || g >= at + P) {
    if (NG - at < P) P /= 2;
    else at += P;
  }
  return {16 * at + (g - at), P};
}

}  // namespace qlq
