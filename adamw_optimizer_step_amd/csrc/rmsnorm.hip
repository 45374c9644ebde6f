// Root-mean-square norm with the residual's addition, forward and backward (gfx950).
// Per row of `cols` values:
//   t = x + residual, rounded to the residual's type (t = x without one)
//   rstd = 1 / sqrt(sum t^2 / cols + eps);  y = t * rstd * gain
//   backward: xh = t * rstd, g = dy * gain
//   dx = dtotal + rstd * (g - xh * mean(g xh));  dgain = sum over rows of dy * xh
// The norm reads t as it is stored, so the backward pass, which has the stored t,
// differentiates the function that was computed. y goes out in bf16 or fp32, or as
// the 8-bit rows of rows.hpp, rounded from fp32 once, or both.
//
// One read of every operand: a group of G lanes holds a row in registers (norm.hpp).
// Sums are fp32, in a fixed order; each output is rounded once.
//
// Bound by memory. With a bf16 residual to 8 bits, 24576 x 2048: 58.8 us, 6.0 TB/s; onto a
// fp32 stream, 1537 x 2047: 8.6 (4.4; 513 of 1024 blocks take two rows); backward with dtotal, 49152 x 1024
// bf16: 71 (5.7) and 4.6 for the column sums; 1 x 1024: 2.2, a chain of a load, a reduction
// and a store.
#include "norm.hpp"

namespace ma {

// v rounded to type DT
template <int DT, int E>
__device__ __forceinline__ void round_to(float (&v)[E]) {
  if constexpr (DT == DT_BF16) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const uint32_t u = pack_bf16x2(v[e], v[e + 1]);
      v[e] = __uint_as_float(u << 16);
      v[e + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
}

// NT: more bytes than the caches keep, none of which is read or written twice: loads and stores
// non-temporal (24576 x 2048 to 8 bits 59 us; loads through the caches 66, stores 68; 16384 x 4096 onto
// a fp32 stream 115, 133, 136).
template <int XD, int TD, int YD, int G, int CH, bool NT>
__global__ void __launch_bounds__(norm_threads(G), 4) k_rms_fwd(const RmsFwdArgs a) {
  constexpr int ROWS = norm_threads(G) / G;
  constexpr bool QUADS = XD == DT_F32 || TD == DT_F32 || YD == DT_F32;
  typedef Chunk<XD, G, QUADS> XC;
  typedef Chunk<TD, G, QUADS> RC;
  typedef Chunk<DT_F32, G, QUADS> PC;
  constexpr int H = XC::H, E = XC::E;
  __shared__ float part[2][1][16];
  const int t = threadIdx.x % G;
  const float per = 1.0f / (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
  // (the widest rows of a fp32 stream leave no registers for the row ahead)
  constexpr bool AHEAD = !QUADS || G * CH < 2048;
  XC next[CH];
  RC beside[CH];
  auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      next[c] = XC();
      beside[c] = RC();
      if (r >= a.rows) continue;
      next[c].template load<NT>(elem_ptr<XD>(a.x, r * a.cols), c, t, a.cols);
      if (a.residual) beside[c].template load<NT>(elem_ptr<TD>(a.residual, r * a.cols), c, t, a.cols);
    }
  };
  if constexpr (AHEAD) load(row);
  PC gain[CH];
  if (a.gain) {
#pragma unroll
    for (int c = 0; c < CH; ++c) gain[c].load(elem_ptr<DT_F32>(a.gain, 0), c, t, a.cols);
  }
  for (int flip = 0; row < a.rows; row += step, flip ^= 1) {
    if constexpr (!AHEAD) load(row);
    float v[CH][H][E];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        next[c].f32(c, h, t, a.cols, v[c][h]);
        if (a.residual) {
          float r[E];
          beside[c].f32(c, h, t, a.cols, r);
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][h][e] += r[e];
          round_to<TD, E>(v[c][h]);
        }
      }
    }
    if (AHEAD && step < a.rows) load(row + step);
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] = __builtin_fmaf(v[c][h][e], v[c][h][e], s[0]);
    group_sum<G>(s, part[flip]);
    const float rstd = uniform<G * CH>(rsqrtf(__builtin_fmaf(s[0], per, a.eps)));
    if (t == 0) a.rstd[row] = rstd;
    const int64_t pitch = act_pitch(a.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int col = XC::col(c, h, t);
        if (a.residual && col < a.cols) RC::template store<NT>(elem_ptr<TD>(a.total, row * a.cols), col, a.cols, v[c][h]);
        float w[E];
        if (a.gain) gain[c].f32(c, h, t, a.cols, w);
        float(&y)[E] = v[c][h];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          y[e] *= rstd;
          if (a.gain) y[e] *= w[e];
        }
        if (a.y && col < a.cols) Chunk<YD, G, QUADS>::template store<NT>(elem_ptr<YD>(a.y, row * a.cols), col, a.cols, y);
        if (a.q) {
          // (past the row's end rstd may have made a NaN of zero)
          if (col + E > a.cols) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (col + e >= a.cols) y[e] = 0.0f;
          }
          const int ex = act_block_exponent(y);
          if (col >= pitch) continue;
          uint32_t b[E / 4];
          act_encode<E>(y, ex, b);
          uint8_t* to = a.q + row * pitch + col;
          if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(b[0], b[1]);
          else *reinterpret_cast<uint32_t*>(to) = b[0];
          if (t % (kActBlock / E) == 0) a.qscale[row * (pitch / kActBlock) + col / kActBlock] = (uint8_t)(ex + 127);
        }
      }
    }
  }
}

// The sums for dgain of 64 columns over all of few rows, by the blocks of the same
// launch that take no rows: a lane per column, the block's waves every W-th row, then
// the waves in order.
template <int XD, int DYD, int W>
__device__ __forceinline__ void rms_cols_direct(const RmsBwdArgs& a, int tile, float (*part)[64]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = tile * 64 + lane;
  const int64_t pitch = act_pitch(a.cols);
  float dg = 0.0f;
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
        for (int u = 0; u < U; ++u) dg = __builtin_fmaf(d[u], x[u] * a.rstd[row + u * W], dg);
      }
    };
    rows_by(std::integral_constant<int, 16>());
    rows_by(std::integral_constant<int, 4>());
    rows_by(std::integral_constant<int, 1>());
  }
  part[wave][lane] = dg;
  __syncthreads();
  if (wave || col >= a.cols) return;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += part[w][lane];
  a.dgain[col] = a.accumulate ? __fadd_rn(a.dgain[col], s) : s;
}

// The backward pass: as many blocks as are resident at once, each with a contiguous
// share of the rows, its groups taking a row each at a time, keep the sums for dgain
// of their columns in registers; the groups' sums are added in LDS, pairs of halves,
// and written once per block. launch_norm_cols adds the blocks' sums in order.
template <int XD, int DYD, int DXD, int G, int CH, bool DIRECT>
__global__ void __launch_bounds__(norm_bwd_threads(G)) k_rms_bwd(const RmsBwdArgs a) {
  constexpr int ROWS = norm_bwd_threads(G) / G, W = norm_bwd_threads(G) / 64;
  __shared__ float part[2][ROWS][1][16];
  __shared__ float join[ROWS > 1 ? ROWS / 2 : 1][ROWS > 1 ? G * CH * 8 : 1];
  if constexpr (DIRECT) {
    __shared__ float cols[W][64];
    if ((int)blockIdx.x >= a.blocks) {
      rms_cols_direct<XD, DYD, W>(a, (int)blockIdx.x - a.blocks, cols);
      return;
    }
  }
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const float per = 1.0f / (float)a.cols;
  const int64_t pitch = act_pitch(a.cols);
  const int64_t units = (a.rows + ROWS - 1) / ROWS, share = (units + a.blocks - 1) / a.blocks;
  const int64_t u0 = blockIdx.x * share, u1 = u0 + share < units ? u0 + share : units;
  float dg[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[c][e] = 0.0f;
  // a row's operands, loaded while the row before it is computed; x and dtotal are read here
  // for the last time, non-temporal where they are bf16 (x 85.9 -> 77.8 us for 49152 x 1024, dtotal 28.3 -> 26.2
  // for 16384 x 1024). dy not: wide rows read it twice (2000 x 16384 76 us, else 84)
  constexpr int XR = raw_dt<XD>();
  struct Row {
    Raw8<XR> x[CH];
    uint2 q[CH];
    uint32_t sc[CH];
    Raw8<DYD> dy[CH];
    Raw8<DXD> dt[CH];
    float rstd;
  };
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    Row r;
    if (row >= a.rows) return r;
    r.rstd = a.rstd[row];
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
      if (a.dtotal) r.dt[c] = raw_load_row<DXD, true>(elem_ptr<DXD>(a.dtotal, row * a.cols), col, a.cols);
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
    float s[1] = {0.0f};
    // xh and dy of chunk c (zeros past the row's end, whatever rstd is), and the gain
    auto chunk = [&](const Row& r, int c, float (&xh)[8], float (&d)[8], float (&w)[8]) __attribute__((always_inline)) {
      const int col = (c * G + t) * 8;
      if constexpr (XD == DT_ACT8) act_decode(r.q[c], act_scale(r.sc[c]), xh);
      else raw_f32_row<XR>(r.x[c], col, a.cols, xh);
      raw_f32_row<DYD>(r.dy[c], col, a.cols, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[e] *= r.rstd;
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
        d[e] *= w[e];
        s[0] = __builtin_fmaf(d[e], x[e], s[0]);
      }
    }
    group_sum<G>(s, part[flip][group]);
    const float m = s[0] * per;
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
      for (int e = 0; e < 8; ++e) out[e] = now.rstd * (d[e] - x[e] * m);
      if (a.dtotal) {
        float dt[8];
        raw_f32_row<DXD>(HOLD ? now.dt[c] : again.dt[c], col, a.cols, dt);
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] += dt[e];
      }
      store_row<DXD>(dst, col, a.cols, out);
    }
  }
  if (DIRECT || !a.partial) return;
#pragma unroll
  for (int half = ROWS / 2; half > 0; half /= 2) {
    __syncthreads();
    if (group >= half && group < 2 * half) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[group - half][(c * 8 + e) * G + t] = dg[c][e];
    }
    __syncthreads();
    if (group < half) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[c][e] += join[group][(c * 8 + e) * G + t];
    }
  }
  if (group) return;
  // by 32 columns, so that the sum over the blocks reads one contiguous stretch
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * G + t) * 8;
    if (col < a.cols) {
      float4* p = reinterpret_cast<float4*>(a.partial + ((int64_t)(col / 32) * a.blocks + blockIdx.x) * 32 + col % 32);
      p[0] = make_float4(dg[c][0], dg[c][1], dg[c][2], dg[c][3]);
      p[1] = make_float4(dg[c][4], dg[c][5], dg[c][6], dg[c][7]);
    }
  }
}

// One chunk per lane where an operand is fp32: two of them and the row ahead of two
// streams pass the registers of 16 waves per CU.
template <int XD, int TD, int YD>
static hipError_t rms_fwd(const RmsFwdArgs& a, hipStream_t s) {
  auto go = [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    const int64_t per = norm_threads(G) / G, want = (a.rows + per - 1) / per, most = (int64_t)256 * kNormWaves * 64 / norm_threads(G);
    const dim3 grid((unsigned)(want < most ? want : most)), block(norm_threads(G));
    const int64_t bytes = a.rows * a.cols * (elem_bytes<XD>() + (a.residual ? 2 * elem_bytes<TD>() : 0) + (a.y ? elem_bytes<YD>() : 0) + (a.q ? 1 : 0));
    // (half: 8192 x 2048 to 8 bits, 117 MB, 22 us against 25, and 40 against 43 with its neighbours;
    // 4096 x 2048 with what reads its results 32 against 30)
    if (bytes > kStreamBytes / 2) hipLaunchKernelGGL((k_rms_fwd<XD, TD, YD, G, CH, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_rms_fwd<XD, TD, YD, G, CH, false>), grid, block, 0, s, a);
    return hipGetLastError();
  };
  if constexpr (XD == DT_F32 || TD == DT_F32 || YD == DT_F32) return norm_one_chunk(a.cols, go);
  else return norm_fwd_shape(a.rows, a.cols, go);
}

hipError_t launch_rms_fwd(const RmsFwdArgs& a, int x_dt, int total_dt, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  auto go = [&](auto x, auto t) {
    constexpr int XD = decltype(x)::value, TD = decltype(t)::value;
    return y_dt == DT_F32 ? rms_fwd<XD, TD, DT_F32>(a, s) : rms_fwd<XD, TD, DT_BF16>(a, s);
  };
  typedef std::integral_constant<int, DT_F32> F;
  typedef std::integral_constant<int, DT_BF16> B;
  if (x_dt == DT_F32) return total_dt == DT_F32 ? go(F(), F()) : go(F(), B());
  return total_dt == DT_F32 ? go(B(), F()) : go(B(), B());
}

template <int XD, int DYD, int DXD>
static hipError_t rms_bwd(const RmsBwdArgs& a, hipStream_t s) {
  return norm_bwd_shape(a.cols, [&](auto sh) {
    constexpr int G = decltype(sh)::G, CH = decltype(sh)::CH;
    const int tiles = a.dgain ? (a.cols + 63) / 64 : 0;
    if (norm_bwd_direct(a.rows))
      hipLaunchKernelGGL((k_rms_bwd<XD, DYD, DXD, G, CH, true>), dim3((unsigned)(a.blocks + tiles)), dim3(norm_bwd_threads(G)), 0, s, a);
    else
      hipLaunchKernelGGL((k_rms_bwd<XD, DYD, DXD, G, CH, false>), dim3((unsigned)a.blocks), dim3(norm_bwd_threads(G)), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_rms_bwd(const RmsBwdArgs& a, int x_dt, int dy_dt, int dx_dt, hipStream_t s) {
  hipError_t err = hipSuccess;
  if (a.blocks > 0) {
    // dx has x's type, or dy's where x is held in 8 bits
    if (x_dt == DT_ACT8) err = dy_dt == DT_F32 ? rms_bwd<DT_ACT8, DT_F32, DT_F32>(a, s) : rms_bwd<DT_ACT8, DT_BF16, DT_BF16>(a, s);
    else if (x_dt == DT_F32) err = dy_dt == DT_F32 ? rms_bwd<DT_F32, DT_F32, DT_F32>(a, s) : rms_bwd<DT_F32, DT_BF16, DT_F32>(a, s);
    else err = dy_dt == DT_F32 ? rms_bwd<DT_BF16, DT_F32, DT_BF16>(a, s) : rms_bwd<DT_BF16, DT_BF16, DT_BF16>(a, s);
  }
  if (err != hipSuccess || !a.dgain || (a.rows > 0 && norm_bwd_direct(a.rows))) return err;
  return launch_norm_cols(a.partial, a.blocks, a.cols, a.accumulate, a.dgain, s);
}

}  // namespace ma
