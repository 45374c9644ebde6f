// The product of a 4-bit weight matrix (mx4.hpp) with rows held in 4 bits or in 8
// (rows.hpp):
//   y[m,n] (+)= sum over k of x[m,k] * w[n,k]
// on the scaled matrix instructions of gfx950: 16 x 16 outputs and 128 k each, whose
// operands are e2m1 or e4m3 values with a power of two for every 32 k, and whose
// sums are fp32. Nothing is unpacked; products of held values are exact.
#include "mx4.hpp"
#include "train_ops.hpp"

namespace ma {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
constexpr int kFmt8 = 0, kFmt4 = 4;   // the instructions' codes for e4m3 and e2m1

// w first: a lane's results are 4 consecutive outputs n of one row m.
template <int XB>
__device__ __forceinline__ f32x4_t mx_mfma16(const i32x8_t& w, const i32x8_t& x, const f32x4_t& c, int ws, int xs) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, kFmt4, XB == 8 ? kFmt8 : kFmt4, 0, ws, 0, xs);
}

// Few rows: a block of WAVES waves takes 16 outputs n of MB * 16 rows m, each wave a
// contiguous share of the k-tiles; the waves' sums are added in order in LDS. The
// operands go from memory to registers: lane l holds row l % 16 and, of every k-tile,
// 32 values from 32 * (l / 16) (of 8-bit rows two times 16, from 16 * (l / 16) and 64
// further: so the instruction pairs them with 4-bit ones). Rows past the end are read
// from inside the matrix; their results are not stored.
template <int XB, int YD, int MB>
__global__ void __launch_bounds__(1024) k_mx4_rows(const Mx4MatmulArgs a) {
  extern __shared__ float join[];   // [waves][MB][64][4]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t nt = (a.outs + 15) / 16;
  const int64_t n0 = (int64_t)blockIdx.x % nt * 16, m0 = (int64_t)blockIdx.x / nt * (16 * MB);
  const int kt = (int)mx4_tiles(a.ins), k0 = (int)((int64_t)kt * wave / waves), k1 = (int)((int64_t)kt * (wave + 1) / waves);
  const int64_t n = n0 + r < a.outs ? n0 + r : a.outs - 1;
  const uint8_t* const wq = a.wq + n * kt * 64 + g * 16;
  const uint8_t* const ws = a.wscale + n * 4 + g;
  const uint8_t *xq[MB], *xs[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t m = m0 + b * 16 + r < a.rows ? m0 + b * 16 + r : a.rows - 1;
    xq[b] = a.xq + m * kt * (XB == 8 ? 128 : 64) + g * 16;
    xs[b] = a.xscale + (XB == 8 ? m * kt : m * 4 + g);
  }
  f32x4_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int t = k0; t < k1; ++t) {
    const u32x4_t u = *reinterpret_cast<const u32x4_t*>(wq + (int64_t)t * 64);
    const i32x8_t w = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], 0, 0, 0, 0};
    const int sw = ws[(int64_t)t * a.outs * 4];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      i32x8_t x;
      int sx;
      if constexpr (XB == 8) {
        const u32x4_t p = *reinterpret_cast<const u32x4_t*>(xq[b] + (int64_t)t * 128), q = *reinterpret_cast<const u32x4_t*>(xq[b] + (int64_t)t * 128 + 64);
        x = i32x8_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)q[0], (int)q[1], (int)q[2], (int)q[3]};
        sx = xs[b][t];
      } else {
        const u32x4_t p = *reinterpret_cast<const u32x4_t*>(xq[b] + (int64_t)t * 64);
        x = i32x8_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
        sx = xs[b][(int64_t)t * a.rows * 4];
      }
      acc[b] = mx_mfma16<XB>(w, x, acc[b], sw, sx);
    }
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) *reinterpret_cast<float4*>(join + ((wave * MB + b) * 64 + lane) * 4) = make_float4(acc[b][0], acc[b][1], acc[b][2], acc[b][3]);
  __syncthreads();
  for (int b = wave; b < MB; b += waves) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < waves; ++w) {
      const float4 p = *reinterpret_cast<const float4*>(join + ((w * MB + b) * 64 + lane) * 4);
      v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
    }
    const int64_t m = m0 + b * 16 + r, at = n0 + g * 4;
    if (m >= a.rows || at >= a.outs) continue;
    unsigned char* out = elem_ptr<YD>(a.y, m * a.outs);
    if (a.accumulate) {
      float old[4];
      quad_f32<YD>(quad_load_row<YD>(out, (int)at, (int)a.outs), (int)at, (int)a.outs, old);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __fadd_rn(old[e], v[e]);
    }
    quad_store_row<YD>(out, (int)at, (int)a.outs, v);
  }
}

template <int XB, int YD, int MB>
static hipError_t mx4_rows(const Mx4MatmulArgs& a, int waves, hipStream_t s) {
  const int64_t blocks = (a.outs + 15) / 16 * ((a.rows + 16 * MB - 1) / (16 * MB));
  hipLaunchKernelGGL((k_mx4_rows<XB, YD, MB>), dim3((unsigned)blocks), dim3(64 * waves), (size_t)waves * MB * 1024, s, a);
  return hipGetLastError();
}

template <int XB, int YD>
static hipError_t mx4_product(const Mx4MatmulArgs& a, hipStream_t s) {
  return a.rows <= 16 ? mx4_rows<XB, YD, 1>(a, 4, s) : mx4_rows<XB, YD, 4>(a, 4, s);
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int x_bits, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_bits == 8) return y_dt == DT_F32 ? mx4_product<8, DT_F32>(a, s) : mx4_product<8, DT_BF16>(a, s);
  return y_dt == DT_F32 ? mx4_product<4, DT_F32>(a, s) : mx4_product<4, DT_BF16>(a, s);
}

}  // namespace ma
