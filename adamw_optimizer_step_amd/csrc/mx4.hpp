// The 4-bit format: per row and block of 32 columns, one power of two 2^e and e2m1
// values q = RNE(x / 2^e). e is the least exponent for which the block's amax / 2^e
// rounds to at most 6 (amax < 7 * 2^e), kept in [kMx4Emin, kMx4Emax]; the scale byte
// is e + 127 (E8M0). So the largest value is rounded like every other, by half a step
// at most, but at e = 125, where what exceeds 6 * 2^125 becomes that: 8 * 2^125 is
// no finite number. A block with a NaN or an infinity has the scale byte 255, which
// stands for NaN, and zeros: e2m1 has neither. A block of zeros has e = kMx4Emin.
//
// Two values share a byte, the even column in its lower half. Rows are padded with
// zeros to whole k-tiles of 128 columns (64 bytes). The 4 scale bytes of a row's
// k-tile are one word, and the words of all rows lie together for each k-tile,
// scale[k-tile][row]: what a product's block reads of them is then contiguous.
#pragma once
#include "rows.hpp"

namespace ma {

constexpr int kMx4Tile = 128, kMx4Block = 32;
constexpr int kMx4Emin = -126, kMx4Emax = 125;
constexpr uint32_t kMx4Nan = 255;

__host__ __device__ constexpr int64_t mx4_tiles(int64_t cols) { return (cols + kMx4Tile - 1) / kMx4Tile; }

// A block's scale byte from the bits of its largest magnitude. 7 = 1.75 * 2^2.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return kMx4Nan;
  const int e = (int)(amax >> 23) - 127 - 2 + ((amax & 0x7FFFFFu) >= 0x600000u ? 1 : 0);   // (subnormal: e clamps)
  return (uint32_t)((e < kMx4Emin ? kMx4Emin : (e > kMx4Emax ? kMx4Emax : e)) + 127);
}

// 8 values over 2^(byte - 127) as e2m1, the first in the lowest 4 bits; zeros for a NaN block.
// The conversion rounds to nearest even and stops at 6.
__device__ __forceinline__ uint32_t mx4_encode(const float (&v)[8], uint32_t byte) {
  if (byte == kMx4Nan) return 0;
  const float s = __uint_as_float(byte << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
}

// The power of two a scale byte stands for.
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : (byte == kMx4Nan ? 0x7FC00000u : byte << 23));
}

// 8 e2m1 values times s
__device__ __forceinline__ void mx4_decode(uint32_t q, float s, float (&v)[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
  const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  v[4] = c[0] * s; v[5] = c[1] * s; v[6] = d[0] * s; v[7] = d[1] * s;
}

}  // namespace ma
