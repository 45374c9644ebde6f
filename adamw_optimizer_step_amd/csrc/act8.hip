// 8-bit activation checkpoints (format: rows.hpp): pack and unpack (gfx950).
// A group of 16 lanes holds one block of 128 columns of one row, 8 values per
// lane: its amax takes four shuffles, and a wave reads 4 blocks at a time.
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

constexpr int kActUnroll = 4;    // blocks of 128 per 16-lane group and pass

template <int XD>
__global__ void __launch_bounds__(256) k_act_pack(const ActArgs a) {
  const int lane16 = threadIdx.x & 15;
  const int64_t pitch = act_pitch(a.cols), kb = pitch / kActBlock, total = a.rows * kb;
  const int64_t b0 = (int64_t)blockIdx.x * (16 * kActUnroll) + (threadIdx.x >> 4);
  Raw8<XD> raw[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    raw[u] = raw_zero<XD>();
    if (b < total) {
      const int64_t row = b / kb;
      const int col = (int)(b - row * kb) * kActBlock + lane16 * 8;
      if (col < a.cols) raw[u] = raw_load_row<XD>(elem_ptr<XD>(a.x, row * a.cols), col, a.cols);
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    float v[8];
    raw_f32<XD>(raw[u], v);
    const int e = act_exponent(act_block_amax(v));
    if (b >= total) continue;
    *reinterpret_cast<uint2*>(a.q + b * kActBlock + lane16 * 8) = act_encode(v, e);
    if (lane16 == 0) a.qscale[b] = (uint8_t)(e + 127);
  }
}

template <int OD>
__global__ void __launch_bounds__(256) k_act_unpack(const ActArgs a) {
  const int lane16 = threadIdx.x & 15;
  const int64_t pitch = act_pitch(a.cols), kb = pitch / kActBlock, total = a.rows * kb;
  const int64_t b0 = (int64_t)blockIdx.x * (16 * kActUnroll) + (threadIdx.x >> 4);
  uint2 q[kActUnroll];
  float s[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    q[u] = make_uint2(0, 0);
    s[u] = 0.0f;
    if (b < total) {
      q[u] = *reinterpret_cast<const uint2*>(a.q + b * kActBlock + lane16 * 8);
      s[u] = act_scale(a.qscale[b]);
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    if (b >= total) continue;
    const int64_t row = b / kb;
    const int col = (int)(b - row * kb) * kActBlock + lane16 * 8;
    float v[8];
    act_decode(q[u], s[u], v);
    if (col < a.cols) store_row<OD>(elem_ptr<OD>(a.out, row * a.cols), col, a.cols, v);
  }
}

static dim3 act_grid(const ActArgs& a) {
  const int64_t total = a.rows * (act_pitch(a.cols) / kActBlock);
  return dim3((unsigned)((total + 16 * kActUnroll - 1) / (16 * kActUnroll)));
}

hipError_t launch_act_pack(const ActArgs& a, int x_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_dt == DT_F32) hipLaunchKernelGGL((k_act_pack<DT_F32>), act_grid(a), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_act_pack<DT_BF16>), act_grid(a), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_act_unpack(const ActArgs& a, int out_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (out_dt == DT_F32) hipLaunchKernelGGL((k_act_unpack<DT_F32>), act_grid(a), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_act_unpack<DT_BF16>), act_grid(a), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ma
