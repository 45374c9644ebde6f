// 8-bit activation checkpoints (format: rows.hpp): pack and unpack (gfx950).
// A group of 16 lanes holds one block of 128 columns of one row, 8 values per
// lane, so that its amax takes four lane exchanges; 4 blocks per group in flight.
// fp32 goes by 4 values per lane and 32 lanes per block (rows.hpp, quad_load_row).
// HBM-bound: 24576 x 4096 bf16 (302 MB each way) packs in 49 us (6.2 TB/s) and
// unpacks in 47 us in turn with packing, 55 behind one another. Packing reads x
// non-temporally where kStreamBytes says so (56 to 63 us without); unpacking always
// does for q, which is read once (60 us without, where it takes 47).
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

constexpr int kActUnroll = 4;    // blocks of 128 per group of lanes and pass
template <int DT> constexpr int act_lanes() { return DT == DT_F32 ? 32 : 16; }
template <int DT> constexpr int act_per_group() { return 256 / act_lanes<DT>(); }   // groups of a thread block

template <int XD, bool NT>
__global__ void __launch_bounds__(256) k_act_pack(const ActArgs a) {
  constexpr int L = act_lanes<XD>(), E = kActBlock / L, GROUPS = act_per_group<XD>();
  const int lane = threadIdx.x % L;
  const int64_t pitch = act_pitch(a.cols), kb = pitch / kActBlock, total = a.rows * kb;
  const int64_t b0 = (int64_t)blockIdx.x * (GROUPS * kActUnroll) + threadIdx.x / L;
  typedef std::conditional_t<E == 8, Raw8<XD>, Raw4<XD>> Raw;
  Raw raw[kActUnroll];
  int col[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * GROUPS;
    if constexpr (E == 8) raw[u] = raw_zero<XD>();
    else raw[u] = quad_zero<XD>();
    col[u] = 0;
    if (b < total) {
      const uint32_t row = (uint32_t)b / (uint32_t)kb;   // rows * pitch <= 2^36: at most 2^29 blocks
      const int at = (int)((uint32_t)b - row * (uint32_t)kb) * kActBlock + lane * E;
      if (at < a.cols) {
        const unsigned char* x = elem_ptr<XD>(a.x, (int64_t)row * a.cols);
        if constexpr (E == 8) raw[u] = raw_load_row<XD, NT>(x, at, a.cols);
        else raw[u] = quad_load_row<XD, NT>(x, at, a.cols);
        col[u] = at;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * GROUPS;
    float v[E];
    if constexpr (E == 8) raw_f32_row<XD>(raw[u], col[u], a.cols, v);
    else quad_f32<XD>(raw[u], col[u], a.cols, v);
    const int e = act_block_exponent(v);
    if (b >= total) continue;
    uint32_t q[E / 4];
    act_encode<E>(v, e, q);
    uint8_t* out = a.q + b * kActBlock + lane * E;
    if constexpr (E == 8) *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(out) = q[0];
    if (lane == 0) a.qscale[b] = (uint8_t)(e + 127);
  }
}

template <int OD, bool NT>
__global__ void __launch_bounds__(256) k_act_unpack(const ActArgs a) {
  constexpr int L = act_lanes<OD>(), E = kActBlock / L, GROUPS = act_per_group<OD>();
  const int lane = threadIdx.x % L;
  const int64_t pitch = act_pitch(a.cols), kb = pitch / kActBlock, total = a.rows * kb;
  const int64_t b0 = (int64_t)blockIdx.x * (GROUPS * kActUnroll) + threadIdx.x / L;
  uint2 q[kActUnroll];
  float s[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * GROUPS;
    q[u] = make_uint2(0, 0);
    s[u] = 0.0f;
    if (b < total) {
      const uint8_t* p = a.q + b * kActBlock + lane * E;
      if constexpr (E == 8) q[u] = ld8_nt(p);
      else q[u].x = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
      s[u] = act_scale(a.qscale[b]);
    }
  }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t b = b0 + u * GROUPS;
    if (b >= total) continue;
    const uint32_t row = (uint32_t)b / (uint32_t)kb;
    const int col = (int)((uint32_t)b - row * (uint32_t)kb) * kActBlock + lane * E;
    if (col >= a.cols) continue;
    unsigned char* out = elem_ptr<OD>(a.out, (int64_t)row * a.cols);
    if constexpr (E == 4) {
      float v[4];
      act_decode(q[u].x, s[u], v);
      quad_store_row<OD, NT>(out, col, a.cols, v);
    } else {
      if (col + 8 <= a.cols) {   // converted straight to packed bf16
        const uint2 lo = act_decode_bf16(q[u].x, s[u]), hi = act_decode_bf16(q[u].y, s[u]);
        *reinterpret_cast<U16<DT_BF16>::T*>(out + (int64_t)col * 2) = u32x4_t{lo.x, lo.y, hi.x, hi.y};
        continue;
      }
      float v[8];
      act_decode(q[u], s[u], v);
      store_row<OD>(out, col, a.cols, v);
    }
  }
}

template <int DT>
static dim3 act_grid(const ActArgs& a) {
  const int64_t total = a.rows * (act_pitch(a.cols) / kActBlock), per = act_per_group<DT>() * kActUnroll;
  return dim3((unsigned)((total + per - 1) / per));
}

hipError_t launch_act_pack(const ActArgs& a, int x_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool stream = a.rows * a.cols * (1 + (x_dt == DT_F32 ? 4 : 2)) > kStreamBytes;
  auto go = [&](auto k, dim3 grid) { hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a); };
  if (x_dt == DT_F32) stream ? go(k_act_pack<DT_F32, true>, act_grid<DT_F32>(a)) : go(k_act_pack<DT_F32, false>, act_grid<DT_F32>(a));
  else stream ? go(k_act_pack<DT_BF16, true>, act_grid<DT_BF16>(a)) : go(k_act_pack<DT_BF16, false>, act_grid<DT_BF16>(a));
  return hipGetLastError();
}

hipError_t launch_act_unpack(const ActArgs& a, int out_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool stream = a.rows * a.cols * 5 > kStreamBytes;
  auto go = [&](auto k, dim3 grid) { hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a); };
  if (out_dt == DT_F32) stream ? go(k_act_unpack<DT_F32, true>, act_grid<DT_F32>(a)) : go(k_act_unpack<DT_F32, false>, act_grid<DT_F32>(a));
  else go(k_act_unpack<DT_BF16, false>, act_grid<DT_BF16>(a));
  return hipGetLastError();
}

}  // namespace ma
