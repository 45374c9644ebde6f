// Row access shared by the kernels around the optimizer step (embedding, layer
// norm, 8-bit checkpoints): 8 consecutive elements of a row per lane, at the
// element type's own alignment, and the checkpoint format.
#pragma once
#include "common.hpp"

namespace ma {

// Calls whose operands together exceed this do not fit the 256 MB memory-side
// cache beside anything else: they mark the larger of what they pass through as
// non-temporal, so that it does not push out what the rest of the call, or the
// next one, can still find there. Below it they leave the cache to the next
// call. (Packing 24576 x 4096 bf16, 302 MB: 49 us with x loaded non-temporally, 56
// without; layer norm of 24576 x 2048 bf16 with its checkpoint, 252 MB: 50 with y
// stored so, 53 without; of 32768 x 1024, 134 MB, 23.5 against 25, but 53.5 against
// 46 together with a pass over y after it.)
// Three operands are loaded non-temporally whatever the size, as what the call reads
// for the last time: a checkpoint's q in unpacking and in norm's backward pass, x in
// that pass, and the embedding gradient's dout. Measured on large calls only.
constexpr int64_t kStreamBytes = (int64_t)192 << 20;

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
// that several loads can be in flight at a low register cost. NT (non-temporal)
// holds for bf16, where a wave's access covers whole cache lines; the two halves
// of an fp32 access meet in the cache (zeros written through it 5.9 TB/s, past
// it 2.2 TB/s).
template <int DT> struct Raw8 { u32x4_t u[DT == DT_BF16 ? 1 : 2]; };

// 8 bytes, optionally non-temporal (see kStreamBytes)
typedef uint32_t u32x2_nt_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint2 ld8_nt(const void* p) {
  const u32x2_nt_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x2_nt_t*>(p));
  return make_uint2(x[0], x[1]);
}

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
    if constexpr (NT && DT == DT_BF16) r.u[i] = __builtin_nontemporal_load(q);
    else r.u[i] = *q;
  }
  return r;
}

// Elements col .. col+7 (col < cols) of a row of `cols` elements at `row`. The
// row's last, partial group loads the row's last 8 elements instead, whole and
// inside the row; raw_f32_row (or raw_fix) moves them to their places. Rows of
// fewer than 8 elements are put together one by one.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> raw_load_row(const unsigned char* row, int col, int cols) {
  if (cols >= 8) return raw_load<DT, NT>(row + (int64_t)(col + 8 <= cols ? col : cols - 8) * elem_bytes<DT>());
  Raw8<DT> r = raw_zero<DT>();
#pragma unroll 1
  for (int k = cols - 1; k >= 0; --k) {
    if constexpr (DT == DT_BF16) {
#pragma unroll
      for (int i = 3; i > 0; --i) r.u[0][i] = r.u[0][i] << 16 | r.u[0][i - 1] >> 16;
      r.u[0][0] = r.u[0][0] << 16 | reinterpret_cast<const uint16_t*>(row)[k];
    } else {
#pragma unroll
      for (int i = 7; i > 0; --i) r.u[i / 4][i % 4] = r.u[(i - 1) / 4][(i - 1) % 4];
      r.u[0][0] = reinterpret_cast<const uint32_t*>(row)[k];
    }
  }
  return r;
}

// What raw_load_row(row, col, cols) loaded, with every element in its place and
// zeros past the row's end.
template <int DT>
__device__ __forceinline__ void raw_fix(Raw8<DT>& r, int col, int cols) {
  if ((cols & 7) == 0) return;     // (the same for every lane: no row has a partial group)
  const int by = col + 8 - cols;   // elements too far up
  if (by <= 0 || cols < 8) return;
  constexpr int W = DT == DT_BF16 ? 4 : 8;   // 32-bit words, 2 or 1 elements each
  uint32_t w[W + 4] = {};
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = r.u[i / 4][i % 4];
  constexpr int E = DT == DT_BF16 ? 2 : 1;
#pragma unroll
  for (int step = 4; step >= E; step /= 2) {
    if (by & step) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = w[i + step / E];
    }
  }
  if constexpr (DT == DT_BF16) {
    if (by & 1) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = w[i] >> 16 | w[i + 1] << 16;
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) r.u[i / 4][i % 4] = w[i];
}

// ----------------------------------------------------------------------------
// Reductions across lanes by DPP moves: no LDS round trips. Lane exchanges
// within 16 lanes: neighbours, pairs, halves mirrored, the row mirrored.
// ----------------------------------------------------------------------------
template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
constexpr int kDppNeighbour = 0xB1, kDppPair = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <typename T, typename F>
__device__ __forceinline__ T reduce16(T x, F&& f) {
  x = f(x, dpp<kDppNeighbour>(x));
  x = f(x, dpp<kDppPair>(x));
  x = f(x, dpp<kDppHalfMirror>(x));
  return f(x, dpp<kDppMirror>(x));
}

// The wave's sum, the same in every lane.
__device__ __forceinline__ float wave_sum_dpp(float x) {
  x = reduce16(x, [](float a, float b) { return a + b; });
  const float a = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 0)), b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 16));
  const float c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 32)), d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 48));
  return (a + b) + (c + d);
}

template <int DT>
__device__ __forceinline__ void raw_f32(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == DT_BF16) v[i] = __uint_as_float(i & 1 ? r.u[0][i / 2] & 0xFFFF0000u : r.u[0][i / 2] << 16);
    else v[i] = __uint_as_float(r.u[i / 4][i % 4]);
  }
}

template <int DT>
__device__ __forceinline__ void raw_f32_row(Raw8<DT> r, int col, int cols, float (&v)[8]) {
  raw_fix<DT>(r, col, cols);
  raw_f32<DT>(r, v);
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
      if constexpr (NT && DT == DT_BF16) __builtin_nontemporal_store((V)u[i], reinterpret_cast<V*>(p) + i);
      else reinterpret_cast<V*>(p)[i] = u[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) store1<DT>(p, i, v[i]);
}

// ----------------------------------------------------------------------------
// The same with 4 consecutive elements per lane, for fp32 streams: a wave's 16-byte
// accesses are then one contiguous stretch, where those of 8 elements leave every
// other 16 bytes to the next access (49152 rows of 1024 fp32 copied by index: 47 us
// against 74, non-temporal stores included, which need whole lines).
// ----------------------------------------------------------------------------
template <int DT> struct Quad;
template <> struct Quad<DT_BF16> { typedef u32x2_nt_t R; typedef u32x2_nt_t T __attribute__((aligned(2))); };
template <> struct Quad<DT_F32> { typedef u32x4_t R; typedef u32x4_t T __attribute__((aligned(4))); };
template <int DT> struct Raw4 { typename Quad<DT>::R u; };

template <int DT>
__device__ __forceinline__ Raw4<DT> quad_zero() {
  Raw4<DT> r;
  r.u = (typename Quad<DT>::R)(0u);
  return r;
}

// Elements col .. col+3 (col < cols) of the row; its last, partial group loads the
// row's last 4 elements, and quad_f32 moves them to their places. Rows of fewer
// than 4 elements are put together one by one.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw4<DT> quad_load_row(const unsigned char* row, int col, int cols) {
  typedef typename Quad<DT>::T V;
  Raw4<DT> r;
  if (cols >= 4) {
    const V* p = reinterpret_cast<const V*>(row + (int64_t)(col + 4 <= cols ? col : cols - 4) * elem_bytes<DT>());
    if constexpr (NT) r.u = __builtin_nontemporal_load(p);
    else r.u = *p;
    return r;
  }
  r = quad_zero<DT>();
#pragma unroll 1
  for (int k = cols - 1; k >= 0; --k) {
    if constexpr (DT == DT_BF16) {
      r.u[1] = r.u[1] << 16 | r.u[0] >> 16;
      r.u[0] = r.u[0] << 16 | reinterpret_cast<const uint16_t*>(row)[k];
    } else {
      r.u[3] = r.u[2];
      r.u[2] = r.u[1];
      r.u[1] = r.u[0];
      r.u[0] = reinterpret_cast<const uint32_t*>(row)[k];
    }
  }
  return r;
}

// The values that quad_load_row(row, col, cols) read, with every one in its place
// and zeros past the row's end.
__device__ __forceinline__ void quad_fix(int col, int cols, float (&v)[4]) {
  const int by = col + 4 - cols;   // elements too far up
  if (by <= 0 || cols < 4) return;
  if (by & 2) { v[0] = v[2]; v[1] = v[3]; v[2] = v[3] = 0.0f; }
  if (by & 1) { v[0] = v[1]; v[1] = v[2]; v[2] = v[3]; v[3] = 0.0f; }
}

template <int DT>
__device__ __forceinline__ void quad_f32(const Raw4<DT>& r, int col, int cols, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_BF16) v[i] = __uint_as_float(i & 1 ? r.u[i / 2] & 0xFFFF0000u : r.u[i / 2] << 16);
    else v[i] = __uint_as_float(r.u[i]);
  }
  if (cols & 3) quad_fix(col, cols, v);
}

// v to elements col .. col+3 of the row (those inside it), rounded once.
template <int DT, bool NT = false>
__device__ __forceinline__ void quad_store_row(unsigned char* row, int col, int cols, const float (&v)[4]) {
  typedef typename Quad<DT>::T V;
  unsigned char* p = row + (int64_t)col * elem_bytes<DT>();
  if (col + 4 <= cols) {
    V u;
    if constexpr (DT == DT_BF16) u = V{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else u = V{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    if constexpr (NT) __builtin_nontemporal_store(u, reinterpret_cast<V*>(p));
    else *reinterpret_cast<V*>(p) = u;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
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

// The exponent of the block that the 16 lanes 16j .. 16j+15 hold, E = 8 columns
// each, or the 32 lanes 32j .. 32j+31 with E = 4. Magnitudes are compared as their bits, where infinities and NaN stand
// above every finite value: a block without any is done in one pass, another
// goes over its values again without them.
template <int E>
__device__ __forceinline__ int act_block_exponent(const float (&v)[E]) {
  constexpr uint32_t kInf = 0x7F800000u;
  auto over = [](uint32_t a) __attribute__((always_inline)) {
    a = reduce16(a, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
    if constexpr (E == 4) {
      const uint32_t b = (uint32_t)__shfl_xor((int)a, 16, 64);
      a = a > b ? a : b;
    }
    return a;
  };
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    a = a > m ? a : m;
  }
  a = over(a);
  if (__any(a >= kInf)) {
    a = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      a = m < kInf && m > a ? m : a;
    }
    a = over(a);
  }
  return act_exponent(__uint_as_float(a));
}

// 8 (or 4) values over 2^e as e4m3 bytes. Every finite value is within 448 * 2^e but
// for those of the largest exponent; NaN and what exceeds the range, here the
// infinities, become NaN.
template <int E>
__device__ __forceinline__ void act_encode(const float (&v)[E], int e, uint32_t (&q)[E / 4]) {
  const float inv = act_pow2(-e);
  float t[E];
#pragma unroll
  for (int i = 0; i < E; ++i) t[i] = v[i] * inv;
  if (e == kActEmax) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (__builtin_fabsf(t[i]) < __builtin_inff()) t[i] = __builtin_fminf(__builtin_fmaxf(t[i], -240.0f), 240.0f);
  }
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    uint32_t b = 0;
    b = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i], t[4 * i + 1], b, false);
    q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i + 2], t[4 * i + 3], b, true);
  }
}

__device__ __forceinline__ float act_scale(uint32_t b) { return __uint_as_float(b << 23); }

// 4 or 8 e4m3 bytes times s (a power of two)
__device__ __forceinline__ void act_decode(uint32_t q, float s, float (&v)[4]) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, true);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
}
__device__ __forceinline__ void act_decode(uint2 q, float s, float (&v)[8]) {
  float a[4], b[4];
  act_decode(q.x, s, a);
  act_decode(q.y, s, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}

// 4 e4m3 bytes times s as packed bf16, exact
__device__ __forceinline__ uint2 act_decode_bf16(uint32_t q, float s) {
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, true)));
}

}  // namespace ma
