// Row access shared by the kernels around the optimizer step (embedding, layer
// norm, 8-bit checkpoints): 8 consecutive elements of a row per lane, at the
// element type's own alignment, and the checkpoint format.
#pragma once
#include "common.hpp"

namespace ma {

// A 16-byte access at 2- or 4-byte alignment: gfx950 serves it as one
// global_load_dwordx4 / global_store_dwordx4 whatever the address, so a row
// that starts anywhere (odd column counts, views) takes the same path as an
// aligned one; a wave's accesses stay contiguous and touch one more cache line.
template <int DT> struct U16;
template <> struct U16<DT_BF16> { typedef u32x4_t T __attribute__((aligned(2))); };
template <> struct U16<DT_F32> { typedef u32x4_t T __attribute__((aligned(4))); };

template <int DT>
__device__ __forceinline__ const unsigned char* elem_ptr(const void* base, int64_t i) {
  return reinterpret_cast<const unsigned char*>(base) + i * elem_bytes<DT>();
}
template <int DT>
__device__ __forceinline__ unsigned char* elem_ptr(void* base, int64_t i) {
  return reinterpret_cast<unsigned char*>(base) + i * elem_bytes<DT>();
}

// The raw 8 elements at p (16 bytes of bf16, 32 of fp32), converted later, so
// that several loads can be in flight at a low register cost.
template <int DT> struct Raw8 { u32x4_t u[DT == DT_BF16 ? 1 : 2]; };

template <int DT>
__device__ __forceinline__ Raw8<DT> raw_zero() {
  Raw8<DT> r;
#pragma unroll
  for (auto& u : r.u) u = u32x4_t{0u, 0u, 0u, 0u};
  return r;
}

template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> raw_load(const unsigned char* p) {
  typedef typename U16<DT>::T V;
  Raw8<DT> r;
  constexpr int N = DT == DT_BF16 ? 1 : 2;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const V* q = reinterpret_cast<const V*>(p) + i;
    if constexpr (NT) r.u[i] = __builtin_nontemporal_load(q);
    else r.u[i] = *q;
  }
  return r;
}

// Elements col .. col+7 of a row of `cols` elements at `row`; zeros past its end.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> raw_load_row(const unsigned char* row, int col, int cols) {
  const unsigned char* p = row + (int64_t)col * elem_bytes<DT>();
  if (col + 8 <= cols) return raw_load<DT, NT>(p);
  Raw8<DT> r = raw_zero<DT>();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (col + i < cols) {
      if constexpr (DT == DT_BF16) r.u[0][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      else r.u[i / 4][i % 4] = reinterpret_cast<const uint32_t*>(p)[i];
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void raw_f32(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == DT_BF16) v[i] = __uint_as_float(i & 1 ? r.u[0][i / 2] & 0xFFFF0000u : r.u[0][i / 2] << 16);
    else v[i] = __uint_as_float(r.u[i / 4][i % 4]);
  }
}

// v to elements col .. col+7 of the row (those inside it), rounded once.
template <int DT, bool NT = false>
__device__ __forceinline__ void store_row(unsigned char* row, int col, int cols, const float (&v)[8]) {
  typedef typename U16<DT>::T V;
  unsigned char* p = row + (int64_t)col * elem_bytes<DT>();
  if (col + 8 <= cols) {
    u32x4_t u[2];
    if constexpr (DT == DT_BF16) {
      u[0] = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i / 4][i % 4] = __float_as_uint(v[i]);
    }
    constexpr int N = DT == DT_BF16 ? 1 : 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (NT) __builtin_nontemporal_store((V)u[i], reinterpret_cast<V*>(p) + i);
      else reinterpret_cast<V*>(p)[i] = u[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) store1<DT>(p, i, v[i]);
}

// ----------------------------------------------------------------------------
// The 8-bit checkpoint: per row and block of 128 columns, one power of two
// 2^e and e4m3 values q = RNE(x / 2^e). e is the least exponent with
// amax <= 448 * 2^e, kept in [kActEmin, kActEmax]; the stored byte is e + 127.
// A power of two makes the division exact (one rounding in all) and makes
// q * 2^e exact in bf16: 4 significant bits, and with e >= -117 the smallest
// value, 2^-9 * 2^-117, is a normal number. At e = 120 the values stop at
// 240 * 2^120, the largest that stays finite. NaN and infinities are stored as
// NaN and take no part in amax; a block with no finite nonzero value has
// e = kActEmin.
// ----------------------------------------------------------------------------
constexpr int kActBlock = 128;
constexpr int kActEmin = -117, kActEmax = 120;

__host__ __device__ constexpr int64_t act_pitch(int64_t cols) { return round_up(cols, kActBlock); }

// The block's exponent from its amax (finite, >= 0). 448 = 0.875 * 2^9.
__device__ __forceinline__ int act_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int ex = (int)(b >> 23) - 126;               // amax = m * 2^ex, m in [0.5, 1) (subnormal: e clamps)
  const int e = ex - 9 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // m > 0.875
  return e < kActEmin ? kActEmin : (e > kActEmax ? kActEmax : e);
}

__device__ __forceinline__ float act_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// |x| where it counts towards amax
__device__ __forceinline__ float act_mag(float x) {
  const float a = __builtin_fabsf(x);
  return a < __builtin_inff() ? a : 0.0f;
}

// 8 values over 2^e as e4m3 bytes
__device__ __forceinline__ uint2 act_encode(const float (&v)[8], int e) {
  const float inv = act_pow2(-e);
  const float most = e == kActEmax ? 240.0f : 448.0f;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = v[i] * inv;
    // finite values are within `most`, but for those of the largest exponent
    t[i] = act_mag(v[i]) == __builtin_fabsf(v[i]) ? __builtin_fminf(__builtin_fmaxf(x, -most), most) : __builtin_nanf("");
  }
  uint32_t lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
  return make_uint2(lo, hi);
}

// 8 e4m3 bytes times s (a power of two)
__device__ __forceinline__ void act_decode(uint2 q, float s, float (&v)[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, true);
  const f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, true);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  v[4] = c[0] * s; v[5] = c[1] * s; v[6] = d[0] * s; v[7] = d[1] * s;
}

__device__ __forceinline__ float act_scale(uint8_t b) { return __uint_as_float((uint32_t)b << 23); }

// amax over the 16 lanes that hold one block (lanes 16j .. 16j+15, 8 columns each)
__device__ __forceinline__ float act_block_amax(const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = __builtin_fmaxf(a, act_mag(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = __builtin_fmaxf(a, __shfl_xor(a, o, kWave));
  return a;
}

}  // namespace ma
