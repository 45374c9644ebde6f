// Weight gradient of a linear layer out of its input's 8-bit checkpoint:
//   grad[n,k] (+)= sum over tokens t of dy[t,n] * x[t,k],  x[t,k] = q[t,k] * 2^e
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

// 64 x 64 outputs per block, 4 x 4 per thread, 16 tokens at a time through LDS.
template <int DYD, int GD>
__global__ void __launch_bounds__(256) k_wgrad(const WgradArgs a) {
  __shared__ float p[16][64], q[16][64];
  const int tid = threadIdx.x, tn = tid / 16, tk = tid % 16;
  const int n0 = blockIdx.y * 64, k0 = blockIdx.x * 64;
  const int64_t pitch = act_pitch(a.ins), kb = pitch / kActBlock;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < a.tokens; t0 += 16) {
    __syncthreads();
    for (int i = tid; i < 1024; i += 256) {
      const int64_t t = t0 + i / 64;
      const int n = n0 + i % 64, k = k0 + i % 64;
      p[i / 64][i % 64] = t < a.tokens && n < a.outs ? load1<DYD>(a.dy, t * a.outs + n) : 0.0f;
      q[i / 64][i % 64] = t < a.tokens && k < a.ins
          ? __builtin_amdgcn_cvt_f32_fp8(a.q[t * pitch + k], 0) * act_scale(a.qscale[t * kb + k / kActBlock]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = __builtin_fmaf(p[j][tn * 4 + x], q[j][tk * 4 + y], acc[x][y]);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int n = n0 + tn * 4 + x, k = k0 + tk * 4 + y;
      if (n >= a.outs || k >= a.ins) continue;
      const int64_t i = (int64_t)n * a.ins + k;
      store1<GD>(a.grad, i, a.accumulate ? load1<GD>(a.grad, i) + acc[x][y] : acc[x][y]);
    }
}

int wgrad_splits(int64_t, int64_t, int64_t, int) { return 1; }

hipError_t launch_wgrad(const WgradArgs& a, int dy_dt, int grad_dt, hipStream_t s) {
  const dim3 grid((unsigned)((a.ins + 63) / 64), (unsigned)((a.outs + 63) / 64));
  auto go = [&](auto dyd, auto gd) {
    hipLaunchKernelGGL((k_wgrad<decltype(dyd)::value, decltype(gd)::value>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, DT_F32> F;
  typedef std::integral_constant<int, DT_BF16> B;
  if (dy_dt == DT_F32) return grad_dt == DT_F32 ? go(F(), F()) : go(F(), B());
  return grad_dt == DT_F32 ? go(B(), F()) : go(B(), B());
}

}  // namespace ma
