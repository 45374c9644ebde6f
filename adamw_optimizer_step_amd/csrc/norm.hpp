// What the kernels of the two norms (layer norm, root-mean-square norm) share: a row
// held in the registers of a group of lanes, sums over the group, and lanes and
// chunks per row by its length.
#pragma once
#include <type_traits>

#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

// threads of a block: a wave per row takes 4 rows, more lanes per row one row
constexpr int norm_threads(int G) { return G == 64 ? 256 : G; }

// Sums over the G lanes of a row's group, the same in every lane: within the
// wave, then over the group's waves through `part` (the group's own; each
// reduction of a row its own array, and two sets alternating between rows, so
// one barrier per reduction is enough).
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*part)[16]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum_dpp(v[n]);
  if constexpr (G > 64) {
    const int wave = threadIdx.x % G >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) part[n][wave] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) v[n] += part[n][w];
    }
  }
}

// x, the same in every lane of a wave, in a scalar register where the others are all taken.
template <int WIDTH>
__device__ __forceinline__ float uniform(float x) {
  if constexpr (WIDTH < 2048) return x;
  else return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// Chunk c of a row: the G lanes' 8 values each of G * 8 columns, 8 consecutive ones
// per lane, or two times 4 where an operand is fp32 (rows.hpp, quad_load_row).
template <int DT, int G, bool QUADS> struct Chunk {
  Raw8<DT> r = raw_zero<DT>();
  static constexpr int H = 1, E = 8;   // parts of E values
  static __device__ __forceinline__ int col(int c, int, int t) { return (c * G + t) * 8; }
  template <bool NT = false> __device__ __forceinline__ void load(const unsigned char* row, int c, int t, int cols) {
    if (col(c, 0, t) < cols) r = raw_load_row<DT, NT>(row, col(c, 0, t), cols);
  }
  __device__ __forceinline__ void f32(int c, int, int t, int cols, float (&v)[8]) const { raw_f32_row<DT>(r, col(c, 0, t), cols, v); }
  template <bool NT> static __device__ __forceinline__ void store(unsigned char* row, int col, int cols, const float (&v)[8]) { store_row<DT, NT>(row, col, cols, v); }
};
template <int DT, int G> struct Chunk<DT, G, true> {
  Raw4<DT> r[2] = {quad_zero<DT>(), quad_zero<DT>()};
  static constexpr int H = 2, E = 4;
  static __device__ __forceinline__ int col(int c, int h, int t) { return (c * 2 + h) * G * 4 + t * 4; }
  template <bool NT = false> __device__ __forceinline__ void load(const unsigned char* row, int c, int t, int cols) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (col(c, h, t) < cols) r[h] = quad_load_row<DT, NT>(row, col(c, h, t), cols);
  }
  __device__ __forceinline__ void f32(int c, int h, int t, int cols, float (&v)[4]) const { quad_f32<DT>(r[h], col(c, h, t), cols, v); }
  template <bool NT> static __device__ __forceinline__ void store(unsigned char* row, int col, int cols, const float (&v)[4]) { quad_store_row<DT, NT>(row, col, cols, v); }
};

constexpr int norm_bwd_threads(int G) { return G < 512 ? 512 : G; }
template <int XD> constexpr int raw_dt() { return XD == DT_ACT8 ? DT_BF16 : XD; }

// The forward pass's waves per CU: each goes through its rows with the next one's
// loads ahead, and gain and bias in registers. Fewer wait for memory less well,
// more spread the writes over more of it (24576 x 2048 bf16 with its checkpoint, us:
// 49 with 16, 52 with 24, 57 with 20 or with a block per row; 4096 x 16384: 49, 58,
// 65, 75; without the row ahead 57 and 75).
constexpr int kNormWaves = 16;

// Lanes and chunks per row by its length: f(NormShape<G, CH>).
//
// Forward: two chunks per lane keep twice the bytes in flight per wave and halve
// the steps of the reductions (bf16 with a checkpoint, us: 49152 x 1024 50 against 51
// with one; 24576 x 2048 49 and 52; 8192 x 8192 62 and 77). Few rows leave the chip empty, and one chunk is the shorter
// chain (100 rows of 1024 3.3 us against 4.0, of 4096 3.6 against 4.2, of 8192 4.3
// against 4.6).
//
// Backward: one chunk per lane, where the row ahead, the row's xh and g and the
// sums for dgain and dbias fit the registers of 16 waves per CU (49152 x 1024 53 us
// against 60 with two; 16384 x 4096 72 against 112; 8192 x 8192 73 against 88).
constexpr int64_t kNormFewRows = 512;
template <int G_, int CH_> struct NormShape { static constexpr int G = G_, CH = CH_; };
template <typename F>
static hipError_t norm_one_chunk(int64_t cols, F&& f) {
  if (cols <= 512) return f(NormShape<64, 1>());
  if (cols <= 1024) return f(NormShape<128, 1>());
  if (cols <= 2048) return f(NormShape<256, 1>());
  if (cols <= 4096) return f(NormShape<512, 1>());
  if (cols <= 8192) return f(NormShape<1024, 1>());
  return f(NormShape<1024, 2>());   // kMaxNormCols
}
template <typename F>
static hipError_t norm_fwd_shape(int64_t rows, int64_t cols, F&& f) {
  if (cols <= 512 || rows <= kNormFewRows) return norm_one_chunk(cols, f);
  if (cols <= 1024) return f(NormShape<64, 2>());
  if (cols <= 2048) return f(NormShape<128, 2>());
  if (cols <= 4096) return f(NormShape<256, 2>());
  if (cols <= 8192) return f(NormShape<512, 2>());
  return f(NormShape<1024, 2>());
}
template <typename F>
static hipError_t norm_bwd_shape(int64_t cols, F&& f) {
  return norm_one_chunk(cols, f);
}

}  // namespace ma
