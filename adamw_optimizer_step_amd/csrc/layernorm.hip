// Layer norm forward and backward (gfx950). Per row of `cols` values:
//   mean = sum x / cols;  var = sum (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) * rstd;  y = xh * gain + bias
//   g = dy * gain;  dx = rstd * (g - mean(g) - xh * mean(g xh))
//   dgain = sum over rows of dy * xh;  dbias = sum over rows of dy
//
// One read of every operand: a group of G lanes holds a row in registers, CH
// chunks of 8 consecutive values per lane (lane t: columns (c G + t) 8 .. +7),
// so the variance is the sum of squared differences from the mean, not a
// difference of two large sums. All sums are fp32, in a fixed order.
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

constexpr int norm_threads(int G) { return G < 256 ? 256 : G; }

// Sums over the G lanes of a row's group, the same in every lane: within the
// wave, then over the group's waves through `part` (the group's own; each
// reduction of a row its own array, and two sets alternating between rows, so
// one barrier per reduction is enough).
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*part)[16]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if constexpr (G > 64) {
    const int wave = threadIdx.x >> 6;
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

template <int XD, int YD, int G, int CH>
__global__ void __launch_bounds__(norm_threads(G)) k_norm_fwd(const NormFwdArgs a) {
  constexpr int ROWS = norm_threads(G) / G;
  __shared__ float part[2][2][1][16];
  const int t = threadIdx.x % G;
  const float n = (float)a.cols;
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / G; row < a.rows; row += (int64_t)gridDim.x * ROWS, flip ^= 1) {
    const unsigned char* src = elem_ptr<XD>(a.x, row * a.cols);
    float x[CH][8];
    {
      Raw8<XD> raw[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * G + t) * 8;
        raw[c] = col < a.cols ? raw_load_row<XD>(src, col, a.cols) : raw_zero<XD>();
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) raw_f32<XD>(raw[c], x[c]);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[c][e];
    group_sum<G>(s, part[flip][0]);
    const float mean = s[0] / n;
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = (c * G + t) * 8 + e < a.cols ? x[c][e] - mean : 0.0f;
        q[0] = __builtin_fmaf(d, d, q[0]);
      }
    group_sum<G>(q, part[flip][1]);
    const float rstd = 1.0f / __fsqrt_rn(q[0] / n + a.eps);
    if (t == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
    unsigned char* dst = elem_ptr<YD>(a.y, row * a.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (col >= a.cols) continue;
      float y[8], w[8], b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (x[c][e] - mean) * rstd;
      if (a.gain) {
        raw_f32<DT_F32>(raw_load_row<DT_F32>(elem_ptr<DT_F32>(a.gain, 0), col, a.cols), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= w[e];
      }
      if (a.bias) {
        raw_f32<DT_F32>(raw_load_row<DT_F32>(elem_ptr<DT_F32>(a.bias, 0), col, a.cols), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += b[e];
      }
      store_row<YD>(dst, col, a.cols, y);
    }
    if (a.q) {
      const int64_t pitch = act_pitch(a.cols);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * G + t) * 8;
        const int e = act_exponent(act_block_amax(x[c]));
        if (col >= pitch) continue;
        *reinterpret_cast<uint2*>(a.q + row * pitch + col) = act_encode(x[c], e);
        if (t % 16 == 0) a.qscale[row * (pitch / kActBlock) + col / kActBlock] = (uint8_t)(e + 127);
      }
    }
  }
}

// The backward pass: a fixed number of blocks, each with a contiguous share of
// the rows, keeps the sums for dgain and dbias of its columns in registers and
// writes them once; k_norm_cols adds the blocks' sums in order.
template <int XD> constexpr int raw_dt() { return XD == DT_ACT8 ? DT_BF16 : XD; }

template <int XD, int DYD, int DXD, int G, int CH>
__global__ void __launch_bounds__(norm_threads(G)) k_norm_bwd(const NormBwdArgs a) {
  constexpr int ROWS = norm_threads(G) / G;
  __shared__ float part[2][2][16];
  __shared__ float join[G == 64 ? 512 * CH : 1];
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const float n = (float)a.cols;
  const int64_t pitch = act_pitch(a.cols);
  const int64_t units = (a.rows + ROWS - 1) / ROWS, share = (units + a.blocks - 1) / a.blocks;
  const int64_t u0 = blockIdx.x * share, u1 = u0 + share < units ? u0 + share : units;
  float dg[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[c][e] = db[c][e] = 0.0f;
  int flip = 0;
  for (int64_t u = u0; u < u1; ++u, flip ^= 1) {
    const int64_t row = u * ROWS + group;
    if (G == 64 && row >= a.rows) break;
    float xh[CH][8], g[CH][8];
    float s[2] = {0.0f, 0.0f};
    const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * row);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[c][e] = g[c][e] = 0.0f;
      if (col >= a.cols) continue;
      if constexpr (XD == DT_ACT8) {
        const float sc = act_scale(a.qscale[row * (pitch / kActBlock) + col / kActBlock]);
        act_decode(*reinterpret_cast<const uint2*>(a.q + row * pitch + col), sc, xh[c]);
      } else {
        raw_f32<raw_dt<XD>()>(raw_load_row<raw_dt<XD>()>(elem_ptr<raw_dt<XD>()>(a.x, row * a.cols), col, a.cols), xh[c]);
      }
      raw_f32<DYD>(raw_load_row<DYD>(elem_ptr<DYD>(a.dy, row * a.cols), col, a.cols), g[c]);
      float w[8];
      if (a.gain) raw_f32<DT_F32>(raw_load_row<DT_F32>(elem_ptr<DT_F32>(a.gain, 0), col, a.cols), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[c][e] = (xh[c][e] - st.x) * st.y;
        if (col + e >= a.cols) xh[c][e] = 0.0f;   // its dy is zero, but a NaN or infinite factor would not be
        dg[c][e] = __builtin_fmaf(g[c][e], xh[c][e], dg[c][e]);
        db[c][e] += g[c][e];
        if (a.gain) g[c][e] *= w[e];
        s[0] += g[c][e];
        s[1] = __builtin_fmaf(g[c][e], xh[c][e], s[1]);
      }
    }
    group_sum<G>(s, part[flip]);
    const float m0 = s[0] / n, m1 = s[1] / n;
    unsigned char* dst = elem_ptr<DXD>(a.dx, row * a.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (col >= a.cols) continue;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = st.y * (g[c][e] - m0 - xh[c][e] * m1);
      store_row<DXD>(dst, col, a.cols, d);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = a.partial + ((int64_t)blockIdx.x * 2 + which) * a.cols;
    float(&v)[CH][8] = which ? db : dg;
    if constexpr (G == 64) {
      // the block's rows in order of their wave
      for (int w = 0; w < ROWS; ++w) {
        __syncthreads();
        if (group != w) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* p = &join[(c * 8 + e) * 64 + t];
            v[c][e] = w ? *p + v[c][e] : v[c][e];
            if (w + 1 < ROWS) *p = v[c][e];
          }
      }
      if (group != ROWS - 1) continue;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (col < a.cols) store_row<DT_F32>(reinterpret_cast<unsigned char*>(out), col, a.cols, v[c]);
    }
  }
}

// dgain (y = 0) and dbias (y = 1): 64 columns per block, its 16 waves summing
// 16 contiguous shares of the blocks' sums, then those in order.
__global__ void __launch_bounds__(1024) k_norm_cols(const NormBwdArgs a) {
  __shared__ float part[16][64];
  float* out = blockIdx.y ? a.dbias : a.dgain;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const int share = (a.blocks + 15) / 16, b0 = wave * share, b1 = b0 + share < a.blocks ? b0 + share : a.blocks;
  float v = 0.0f;
  if (col < a.cols) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) v += a.partial[((int64_t)b * 2 + blockIdx.y) * a.cols + col];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < a.cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += part[w][lane];
    out[col] = a.accumulate ? __fadd_rn(out[col], t) : t;
  }
}

// Lanes and chunks per row by its length: f(G, CH) as integral constants.
template <int G_, int CH_> struct NormShape { static constexpr int G = G_, CH = CH_; };
template <typename F>
static hipError_t norm_shape(int64_t cols, F&& f) {
  if (cols <= 512) return f(NormShape<64, 1>());
  if (cols <= 1024) return f(NormShape<64, 2>());
  if (cols <= 2048) return f(NormShape<256, 1>());
  if (cols <= 4096) return f(NormShape<256, 2>());
  if (cols <= 8192) return f(NormShape<1024, 1>());
  return f(NormShape<1024, 2>());   // kMaxNormCols
}
static int norm_rows_per_block(int64_t cols) { return cols <= 1024 ? 4 : 1; }

template <int XD, int YD>
static hipError_t norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  return norm_shape(a.cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    const int64_t per = norm_threads(G) / G, want = (a.rows + per - 1) / per, most = (int64_t)1 << 21;
    hipLaunchKernelGGL((k_norm_fwd<XD, YD, G, CH>), dim3((unsigned)(want < most ? want : most)), dim3(norm_threads(G)), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int x_dt, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_dt == DT_F32) return y_dt == DT_F32 ? norm_fwd<DT_F32, DT_F32>(a, s) : norm_fwd<DT_F32, DT_BF16>(a, s);
  return y_dt == DT_F32 ? norm_fwd<DT_BF16, DT_F32>(a, s) : norm_fwd<DT_BF16, DT_BF16>(a, s);
}

int norm_bwd_blocks(int64_t rows, int64_t cols) {
  const int64_t per = norm_rows_per_block(cols), units = (rows + per - 1) / per;
  const int64_t most = cols <= 4096 ? 1024 : 512;
  return (int)(units < most ? units : most);
}

template <int XD, int DYD, int DXD>
static hipError_t norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  return norm_shape(a.cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    hipLaunchKernelGGL((k_norm_bwd<XD, DYD, DXD, G, CH>), dim3((unsigned)a.blocks), dim3(norm_threads(G)), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int x_dt, int dy_dt, int dx_dt, hipStream_t s) {
  hipError_t err = hipSuccess;
  if (a.blocks > 0) {
    // dx has x's type, or dy's where x is a checkpoint
    if (x_dt == DT_ACT8) err = dy_dt == DT_F32 ? norm_bwd<DT_ACT8, DT_F32, DT_F32>(a, s) : norm_bwd<DT_ACT8, DT_BF16, DT_BF16>(a, s);
    else if (x_dt == DT_F32) err = dy_dt == DT_F32 ? norm_bwd<DT_F32, DT_F32, DT_F32>(a, s) : norm_bwd<DT_F32, DT_BF16, DT_F32>(a, s);
    else err = dy_dt == DT_F32 ? norm_bwd<DT_BF16, DT_F32, DT_BF16>(a, s) : norm_bwd<DT_BF16, DT_BF16, DT_BF16>(a, s);
  }
  if (err != hipSuccess || (!a.dgain && !a.dbias)) return err;
  hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace ma
