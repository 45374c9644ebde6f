// Layer norm forward and backward (gfx950). Per row of `cols` values:
//   mean = sum x / cols;  var = sum (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) * rstd;  y = xh * gain + bias
//   g = dy * gain;  dx = rstd * (g - mean(g) - xh * mean(g xh))
//   dgain = sum over rows of dy * xh;  dbias = sum over rows of dy
//
// One read of every operand: a group of G lanes holds a row in registers, CH
// chunks of 8 consecutive values per lane (lane t: columns (c G + t) 8 .. +7),
// so the variance is the sum of squared differences from the mean, not a
// difference of two large sums. All sums are fp32, in a fixed order. y and dx are
// rounded once; xh is held and recomputed in fp32.
//
// Bound by memory: forward of 24576 x 2048 bf16 with its checkpoint, 252 MB in 43
// us (5.9 TB/s), 49 where its operands are cold; backward of 49152 x 1024 bf16, 302 MB in 52 us (5.8 TB/s) and
// 4.7 for k_norm_cols; backward out of a checkpoint of 31948 x 962 with fp32 dy,
// 278 MB in 49 us.
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
  __device__ __forceinline__ void load(const unsigned char* row, int c, int t, int cols) {
    if (col(c, 0, t) < cols) r = raw_load_row<DT>(row, col(c, 0, t), cols);
  }
  __device__ __forceinline__ void f32(int c, int, int t, int cols, float (&v)[8]) const { raw_f32_row<DT>(r, col(c, 0, t), cols, v); }
  template <bool NT> static __device__ __forceinline__ void store(unsigned char* row, int col, int cols, const float (&v)[8]) { store_row<DT, NT>(row, col, cols, v); }
};
template <int DT, int G> struct Chunk<DT, G, true> {
  Raw4<DT> r[2] = {quad_zero<DT>(), quad_zero<DT>()};
  static constexpr int H = 2, E = 4;
  static __device__ __forceinline__ int col(int c, int h, int t) { return (c * 2 + h) * G * 4 + t * 4; }
  __device__ __forceinline__ void load(const unsigned char* row, int c, int t, int cols) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (col(c, h, t) < cols) r[h] = quad_load_row<DT>(row, col(c, h, t), cols);
  }
  __device__ __forceinline__ void f32(int c, int h, int t, int cols, float (&v)[4]) const { quad_f32<DT>(r[h], col(c, h, t), cols, v); }
  template <bool NT> static __device__ __forceinline__ void store(unsigned char* row, int col, int cols, const float (&v)[4]) { quad_store_row<DT, NT>(row, col, cols, v); }
};

template <int XD, int YD, int G, int CH, bool NT>
__global__ void __launch_bounds__(norm_threads(G)) k_norm_fwd(const NormFwdArgs a) {
  constexpr int ROWS = norm_threads(G) / G;
  constexpr bool QUADS = XD == DT_F32 || YD == DT_F32;
  typedef Chunk<XD, G, QUADS> XC;
  typedef Chunk<DT_F32, G, QUADS> PC;
  constexpr int H = XC::H, E = XC::E;
  __shared__ float part[2][3][1][16];
  const int t = threadIdx.x % G;
  const float per = 1.0f / (float)a.cols;
  const float per16 = 16.0f * per;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
  XC next[CH];
  auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      next[c] = XC();
      if (r < a.rows) next[c].load(elem_ptr<XD>(a.x, r * a.cols), c, t, a.cols);
    }
  };
  load(row);
  PC gain[CH], bias[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (a.gain) gain[c].load(elem_ptr<DT_F32>(a.gain, 0), c, t, a.cols);
    if (a.bias) bias[c].load(elem_ptr<DT_F32>(a.bias, 0), c, t, a.cols);
  }
  for (int flip = 0; row < a.rows; row += step, flip ^= 1) {
    float x[CH][H][E];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int h = 0; h < H; ++h) next[c].f32(c, h, t, a.cols, x[c][h]);
    if (step < a.rows) load(row + step);
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] += x[c][h][e];
    group_sum<G>(s, part[flip][0]);
    float mean = uniform<G * CH>(s[0] * per);
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int in = a.cols - XC::col(c, h, t);
        if (in >= E) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float d = x[c][h][e] - mean;
            q[0] = __builtin_fmaf(d, d, q[0]);
          }
        } else if (in > 0) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float d = e < in ? x[c][h][e] - mean : 0.0f;
            q[0] = __builtin_fmaf(d, d, q[0]);
          }
        }
      }
    }
    group_sum<G>(q, part[flip][1]);
    // The mean so far is off by the roundings of the sum and of 1 / cols, some steps of |mean|. That shows where the
    // mean is large beside the deviation: a row of equal values would have a variance, and with a small eps |y| of 1.
    // So where it is more than 4 of them (NaN and infinities fail the test) the mean is corrected: the differences
    // from it are small, and their sum, nearly exact, over cols is what it is off by. On every row this costs up to
    // a fifth (60000 x 256 bf16 21.2 us against 17.5), so at most 2 % where no row needs it, and that where all do.
    if (q[0] * per16 < mean * mean) {
      float r[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int in = a.cols - XC::col(c, h, t);
          if (in >= E) {
#pragma unroll
            for (int e = 0; e < E; ++e) r[0] += x[c][h][e] - mean;
          } else if (in > 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) r[0] += e < in ? x[c][h][e] - mean : 0.0f;
          }
        }
      }
      group_sum<G>(r, part[flip][2]);
      float off = r[0] * per;
      off = __builtin_fmaf(__builtin_fmaf(-off, (float)a.cols, r[0]), per, off);   // r / cols: the quotient and the rest's
      mean = uniform<G * CH>(mean + off);
      q[0] = __builtin_fmaf(-r[0], off, q[0]);
      if (q[0] < 0.0f) q[0] = 0.0f;
    }
    const float rstd = uniform<G * CH>(rsqrtf(__builtin_fmaf(q[0], per, a.eps)));
    if (t == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
    unsigned char* dst = elem_ptr<YD>(a.y, row * a.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int col = XC::col(c, h, t);
        if (col >= a.cols) continue;
        float y[E], w[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (x[c][h][e] - mean) * rstd;
        if (a.gain) {
          gain[c].f32(c, h, t, a.cols, w);
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] *= w[e];
        }
        if (a.bias) {
          bias[c].f32(c, h, t, a.cols, w);
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] += w[e];
        }
        Chunk<YD, G, QUADS>::template store<NT>(dst, col, a.cols, y);
      }
    }
    if (a.q) {
      const int64_t pitch = act_pitch(a.cols);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int col = XC::col(c, h, t);
          const int e = act_block_exponent(x[c][h]);
          if (col >= pitch) continue;
          uint32_t b[E / 4];
          act_encode<E>(x[c][h], e, b);
          uint8_t* to = a.q + row * pitch + col;
          if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(b[0], b[1]);
          else *reinterpret_cast<uint32_t*>(to) = b[0];
          if (t % (kActBlock / E) == 0) a.qscale[row * (pitch / kActBlock) + col / kActBlock] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

// The backward pass: as many blocks as are resident at once, each with a
// contiguous share of the rows, its groups taking a row each at a time, keep the
// sums for dgain and dbias of their columns in registers; the groups' sums are
// added in LDS, pairs of halves, and written once per block. k_norm_cols adds the
// blocks' sums in order.
constexpr int norm_bwd_threads(int G) { return G < 512 ? 512 : G; }
template <int XD> constexpr int raw_dt() { return XD == DT_ACT8 ? DT_BF16 : XD; }

// The sums for dgain and dbias of 64 columns over all of few rows (at most
// kNormDirectRows), by the blocks of the same launch that take no rows: a lane per
// column, the block's waves every W-th row, then the waves in order. Reads x and
// dy once more, from the caches, and saves the partial sums and a launch.
template <int XD, int DYD, int W>
__device__ __forceinline__ void norm_cols_direct(const NormBwdArgs& a, int tile, float (*part)[2][64]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = tile * 64 + lane;
  const int64_t pitch = act_pitch(a.cols);
  float dg = 0.0f, db = 0.0f;
  if (col < a.cols) {
    // U rows in flight as long as so many are left
    int row = wave;
    auto rows_by = [&](auto n) __attribute__((always_inline)) {
      constexpr int U = decltype(n)::value;
      for (; row + (U - 1) * W < (int)a.rows; row += U * W) {
        float x[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = row + u * W;
          if constexpr (XD == DT_ACT8)
            x[u] = __builtin_amdgcn_cvt_f32_fp8(a.q[r * pitch + col], 0) * act_scale(a.qscale[r * (pitch / kActBlock) + col / kActBlock]);
          else
            x[u] = load1<raw_dt<XD>()>(a.x, (int64_t)r * a.cols + col);
          d[u] = load1<DYD>(a.dy, (int64_t)r * a.cols + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = row + u * W;
          dg = __builtin_fmaf(d[u], (x[u] - a.stats[2 * r]) * a.stats[2 * r + 1], dg);
          db += d[u];
        }
      }
    };
    rows_by(std::integral_constant<int, 16>());
    rows_by(std::integral_constant<int, 4>());
    rows_by(std::integral_constant<int, 1>());
  }
  part[wave][0][lane] = dg;
  part[wave][1][lane] = db;
  __syncthreads();
  float* out = wave == 0 ? a.dgain : (wave == 1 ? a.dbias : nullptr);
  if (!out || col >= a.cols) return;
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) t += part[w][wave][lane];
  out[col] = a.accumulate ? __fadd_rn(out[col], t) : t;
}

template <int XD, int DYD, int DXD, int G, int CH, bool DIRECT>
__global__ void __launch_bounds__(norm_bwd_threads(G)) k_norm_bwd(const NormBwdArgs a) {
  constexpr int ROWS = norm_bwd_threads(G) / G, W = norm_bwd_threads(G) / 64;
  __shared__ float part[2][ROWS][2][16];
  __shared__ float join[ROWS > 1 ? ROWS / 2 : 1][ROWS > 1 ? G * CH * 8 : 1];
  if constexpr (DIRECT) {
    __shared__ float cols[W][2][64];
    // (the last blocks: first, they would read columns past cold caches; 512 x 1024 bf16 8.2 us against 4.9)
    if ((int)blockIdx.x >= a.blocks) {
      norm_cols_direct<XD, DYD, W>(a, (int)blockIdx.x - a.blocks, cols);
      return;
    }
  }
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const float per = 1.0f / (float)a.cols;
  const int64_t pitch = act_pitch(a.cols);
  const int64_t units = (a.rows + ROWS - 1) / ROWS, share = (units + a.blocks - 1) / a.blocks;
  const int64_t u0 = blockIdx.x * share, u1 = u0 + share < units ? u0 + share : units;
  float dg[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[c][e] = db[c][e] = 0.0f;
  // a row's operands, loaded while the row before it is computed; x comes from a
  // forward pass long ago and is not read again soon (non-temporal), dy is fresh
  constexpr int XR = raw_dt<XD>();
  struct Row {
    Raw8<XR> x[CH];
    uint2 q[CH];
    uint32_t sc[CH];
    Raw8<DYD> dy[CH];
    float2 st;
  };
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    Row r;
    if (row >= a.rows) return r;
    r.st = *reinterpret_cast<const float2*>(a.stats + 2 * row);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (col >= a.cols) continue;
      if constexpr (XD == DT_ACT8) {
        r.q[c] = ld8_nt(a.q + row * pitch + col);
        r.sc[c] = a.qscale[row * (pitch / kActBlock) + col / kActBlock];
      } else {
        r.x[c] = raw_load_row<XR, true>(elem_ptr<XR>(a.x, row * a.cols), col, a.cols);
      }
      r.dy[c] = raw_load_row<DYD>(elem_ptr<DYD>(a.dy, row * a.cols), col, a.cols);
    }
    return r;
  };
  // where the registers are there: the row ahead, and xh and g kept over the reduction (else they are read again, from L2)
  constexpr bool AHEAD = G * CH < 2048, HOLD = G * CH < 2048;
  float w0[8];   // the gain, kept where a lane has one chunk only
  if (CH == 1 && a.gain && t * 8 < a.cols)
    raw_f32_row<DT_F32>(raw_load_row<DT_F32>(elem_ptr<DT_F32>(a.gain, 0), t * 8, a.cols), t * 8, a.cols, w0);
  Row next = load(AHEAD && u0 < u1 ? u0 * ROWS + group : a.rows);
  int flip = 0;
  for (int64_t u = u0; u < u1; ++u, flip ^= 1) {
    const int64_t row = u * ROWS + group;
    const bool valid = row < a.rows;
    if (G == 64 && !valid) break;   // (wider groups meet at barriers)
    const Row now = AHEAD ? next : load(row);
    if constexpr (AHEAD) next = load(u + 1 < u1 ? row + ROWS : a.rows);
    float s[2] = {0.0f, 0.0f};
    const float2 st = now.st;
    // xh and dy of chunk c (zeros past the row's end, whatever the row's factors are), and the gain
    auto chunk = [&](const Row& r, int c, float (&xh)[8], float (&d)[8], float (&w)[8]) __attribute__((always_inline)) {
      const int col = (c * G + t) * 8;
      if constexpr (XD == DT_ACT8) act_decode(r.q[c], act_scale(r.sc[c]), xh);
      else raw_f32_row<XR>(r.x[c], col, a.cols, xh);
      raw_f32_row<DYD>(r.dy[c], col, a.cols, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[e] = (xh[e] - st.x) * st.y;
      if ((a.cols & 7) && col + 8 > a.cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e >= a.cols) xh[e] = 0.0f;
      }
      if (a.gain) {
        if constexpr (CH == 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = w0[e];
        } else {
          raw_f32_row<DT_F32>(raw_load_row<DT_F32>(elem_ptr<DT_F32>(a.gain, 0), col, a.cols), col, a.cols, w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
    };
    float xh[HOLD ? CH : 1][8], g[HOLD ? CH : 1][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float(&x)[8] = xh[HOLD ? c : 0], (&d)[8] = g[HOLD ? c : 0], w[8];
      if (!valid || (c * G + t) * 8 >= a.cols) continue;
      chunk(now, c, x, d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[c][e] = __builtin_fmaf(d[e], x[e], dg[c][e]);
        db[c][e] += d[e];
        d[e] *= w[e];
        s[0] += d[e];
        s[1] = __builtin_fmaf(d[e], x[e], s[1]);
      }
    }
    group_sum<G>(s, part[flip][group]);
    const float m0 = s[0] * per, m1 = s[1] * per;
    const Row again = HOLD ? Row() : load(row);
    unsigned char* dst = elem_ptr<DXD>(a.dx, row * a.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (!valid || col >= a.cols) continue;
      float(&x)[8] = xh[HOLD ? c : 0], (&d)[8] = g[HOLD ? c : 0], w[8], out[8];
      if constexpr (!HOLD) {
        chunk(again, c, x, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = st.y * (d[e] - m0 - x[e] * m1);
      store_row<DXD>(dst, col, a.cols, out);
    }
  }
  if (DIRECT || !a.partial) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    // by 32 columns, so that k_norm_cols reads one contiguous stretch
    float* const out = a.partial + (int64_t)which * round_up(a.cols, 32) * a.blocks;
    float(&v)[CH][8] = which ? db : dg;
#pragma unroll
    for (int half = ROWS / 2; half > 0; half /= 2) {
      __syncthreads();
      if (group >= half && group < 2 * half) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) join[group - half][(c * 8 + e) * G + t] = v[c][e];
      }
      __syncthreads();
      if (group < half) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] += join[group][(c * 8 + e) * G + t];
      }
    }
    if (group) continue;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * G + t) * 8;
      if (col < a.cols) {
        float4* p = reinterpret_cast<float4*>(out + ((int64_t)(col / 32) * a.blocks + blockIdx.x) * 32 + col % 32);
        p[0] = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
        p[1] = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
      }
    }
  }
}

// dgain (y = 0) and dbias (y = 1): 32 columns per block, 32 groups of lanes
// summing as many contiguous shares of the blocks' sums, then those in order.
__global__ void __launch_bounds__(1024) k_norm_cols(const NormBwdArgs a) {
  __shared__ float part[32][32];
  float* out = blockIdx.y ? a.dbias : a.dgain;
  if (!out) return;
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int share = (a.blocks + 31) / 32, b0 = group * share, b1 = b0 + share < a.blocks ? b0 + share : a.blocks;
  float v = 0.0f;
  const float* src = a.partial + (int64_t)blockIdx.y * round_up(a.cols, 32) * a.blocks + (int64_t)blockIdx.x * a.blocks * 32 + lane;
  constexpr int U = 16;   // a share is no longer (norm_bwd_blocks)
  float x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = b0 + u < b1 ? src[(b0 + u) * 32] : 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) v += x[u];
  part[group][lane] = v;
  __syncthreads();
  if (group == 0 && col < a.cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += part[w][lane];
    out[col] = a.accumulate ? __fadd_rn(out[col], t) : t;
  }
}

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
static hipError_t norm_fwd_shape(int64_t rows, int64_t cols, F&& f) {
  if (cols <= 512) return f(NormShape<64, 1>());
  if (rows <= kNormFewRows) {
    if (cols <= 1024) return f(NormShape<128, 1>());
    if (cols <= 2048) return f(NormShape<256, 1>());
    if (cols <= 4096) return f(NormShape<512, 1>());
    if (cols <= 8192) return f(NormShape<1024, 1>());
  }
  if (cols <= 1024) return f(NormShape<64, 2>());
  if (cols <= 2048) return f(NormShape<128, 2>());
  if (cols <= 4096) return f(NormShape<256, 2>());
  if (cols <= 8192) return f(NormShape<512, 2>());
  return f(NormShape<1024, 2>());   // kMaxNormCols
}
template <typename F>
static hipError_t norm_bwd_shape(int64_t cols, F&& f) {
  if (cols <= 512) return f(NormShape<64, 1>());
  if (cols <= 1024) return f(NormShape<128, 1>());
  if (cols <= 2048) return f(NormShape<256, 1>());
  if (cols <= 4096) return f(NormShape<512, 1>());
  if (cols <= 8192) return f(NormShape<1024, 1>());
  return f(NormShape<1024, 2>());
}

template <int XD, int YD>
static hipError_t norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  return norm_fwd_shape(a.rows, a.cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    const int64_t per = norm_threads(G) / G, want = (a.rows + per - 1) / per, most = (int64_t)256 * kNormWaves * 64 / norm_threads(G);
    const dim3 grid((unsigned)(want < most ? want : most)), block(norm_threads(G));
    const int64_t bytes = a.rows * a.cols * (elem_bytes<XD>() + elem_bytes<YD>() + (a.q ? 1 : 0));
    if (bytes > kStreamBytes) hipLaunchKernelGGL((k_norm_fwd<XD, YD, G, CH, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<XD, YD, G, CH, false>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int x_dt, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_dt == DT_F32) return y_dt == DT_F32 ? norm_fwd<DT_F32, DT_F32>(a, s) : norm_fwd<DT_F32, DT_BF16>(a, s);
  return y_dt == DT_F32 ? norm_fwd<DT_BF16, DT_F32>(a, s) : norm_fwd<DT_BF16, DT_BF16>(a, s);
}

// Whether the rows are so few that no partial sums are kept: reading x and dy
// again costs less than a launch more (bf16 of 1024 columns: 513 rows 4.9 us in one
// launch, 4.9 + 3 in two; 1000 rows 8.1 and 5.2 + 3.3; 2000 rows 17 and 6.9 + 3.5).
constexpr int64_t kNormDirectRows = 1024;
bool norm_bwd_direct(int64_t rows) { return rows <= kNormDirectRows; }

// As many as are resident at once (16 waves per CU); where a row takes 256 lanes
// or more at least 4 steps each, down to 128 blocks: every block writes, and
// k_norm_cols reads, two rows of sums (1537 x 2047, fp32 dy: 11 + 4.3 us with 193
// blocks, 12.4 + 3.9 with 385).
int norm_bwd_blocks(int64_t rows, int64_t cols) {
  int64_t units = rows, most = 0;
  bool wide = false;
  (void)norm_bwd_shape(cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, T = norm_bwd_threads(G);
    units = (rows + T / G - 1) / (T / G);
    most = 256 * 16 * 64 / T;
    static_assert(256 * 16 * 64 / T <= 32 * 16, "k_norm_cols' shares");
    wide = G >= 256;
    return hipSuccess;
  });
  if (wide && !norm_bwd_direct(rows)) {
    const int64_t want = (units + 3) / 4, least = units < 128 ? units : 128;
    units = want > least ? want : least;
  }
  return (int)(units < most ? units : most);
}

template <int XD, int DYD, int DXD>
static hipError_t norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  return norm_bwd_shape(a.cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    const int tiles = a.dgain || a.dbias ? (a.cols + 63) / 64 : 0;
    if (norm_bwd_direct(a.rows))
      hipLaunchKernelGGL((k_norm_bwd<XD, DYD, DXD, G, CH, true>), dim3((unsigned)(a.blocks + tiles)), dim3(norm_bwd_threads(G)), 0, s, a);
    else
      hipLaunchKernelGGL((k_norm_bwd<XD, DYD, DXD, G, CH, false>), dim3((unsigned)a.blocks), dim3(norm_bwd_threads(G)), 0, s, a);
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
  if (err != hipSuccess || (!a.dgain && !a.dbias) || (a.rows > 0 && norm_bwd_direct(a.rows))) return err;
  hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((a.cols + 31) / 32), 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace ma
