// 8-bit activation checkpoints (format: rows.hpp): pack and unpack (gfx950).
// A group of 16 lanes holds one block of 128 columns of one row, 8 values per
// lane, so that its amax takes four lane exchanges; 4 blocks per group in flight.
// HBM-bound: 24576 x 4096 bf16 (302 MB each way) packs in 48 us (6.3 TB/s) and
// unpacks in 47 us. Packing reads x non-temporally where kStreamBytes says so (63
// us without); unpacking always does for q, which is read once (60 us without).
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

constexpr int kActUnroll = 4;    // blocks of 128 per 16-lane group and pass

template <int XD, bool NT>
__global__ void __launch_bounds__(256) k_act_pack(const ActArgs a) {
  const int lane16 = threadIdx.x & 15;
  const int64_t pitch = act_pitch(a.cols), kb = pitch / kActBlock, total = a.rows * kb;
  const int64_t b0 = (int64_t)blockIdx.x * (16 * kActUnroll) + (threadIdx.x >> 4);
  Raw8<XD> raw[kActUnroll];
  int col[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    raw[u] = raw_zero<XD>();
    col[u] = 0;
    if (b < total) {
      const uint32_t row = (uint32_t)b / (uint32_t)kb;   // rows * pitch <= 2^36: at most 2^29 blocks
      const int at = (int)((uint32_t)b - row * (uint32_t)kb) * kActBlock + lane16 * 8;
      if (at < a.cols) {
        raw[u] = raw_load_row<XD, NT>(elem_ptr<XD>(a.x, (int64_t)row * a.cols), at, a.cols);
        col[u] = at;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    float v[8];
    raw_f32_row<XD>(raw[u], col[u], a.cols, v);
    const int e = act_block_exponent(v);
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
      q[u] = ld8_nt(a.q + b * kActBlock + lane16 * 8);
      s[u] = act_scale(a.qscale[b]);
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * 16;
    if (b >= total) continue;
    const uint32_t row = (uint32_t)b / (uint32_t)kb;
    const int col = (int)((uint32_t)b - row * (uint32_t)kb) * kActBlock + lane16 * 8;
    if (col >= a.cols) continue;
    unsigned char* out = elem_ptr<OD>(a.out, (int64_t)row * a.cols);
    if constexpr (OD == DT_BF16) {
      if (col + 8 <= a.cols) {   // converted straight to packed bf16
        const uint2 lo = act_decode_bf16(q[u].x, s[u]), hi = act_decode_bf16(q[u].y, s[u]);
        *reinterpret_cast<U16<DT_BF16>::T*>(out + (int64_t)col * 2) = u32x4_t{lo.x, lo.y, hi.x, hi.y};
        continue;
      }
    }
    float v[8];
    act_decode(q[u], s[u], v);
    store_row<OD>(out, col, a.cols, v);
  }
}

static dim3 act_grid(const ActArgs& a) {
  const int64_t total = a.rows * (act_pitch(a.cols) / kActBlock);
  return dim3((unsigned)((total + 16 * kActUnroll - 1) / (16 * kActUnroll)));
}

hipError_t launch_act_pack(const ActArgs& a, int x_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool stream = a.rows * a.cols * (1 + (x_dt == DT_F32 ? 4 : 2)) > kStreamBytes;
  auto go = [&](auto k) { hipLaunchKernelGGL(k, act_grid(a), dim3(256), 0, s, a); };
  if (x_dt == DT_F32) stream ? go(k_act_pack<DT_F32, true>) : go(k_act_pack<DT_F32, false>);
  else stream ? go(k_act_pack<DT_BF16, true>) : go(k_act_pack<DT_BF16, false>);
  return hipGetLastError();
}

hipError_t launch_act_unpack(const ActArgs& a, int out_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (out_dt == DT_F32) hipLaunchKernelGGL((k_act_unpack<DT_F32>), act_grid(a), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_act_unpack<DT_BF16>), act_grid(a), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ma
