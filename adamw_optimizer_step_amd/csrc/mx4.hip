// 4-bit matrices (format: mx4.hpp): pack, of a matrix or of its transpose, and unpack
// (gfx950). Bound by memory: 16384 x 4096 bf16 packed in 31 us and unpacked in 29,
// 5.4 and 5.9 TB/s.
#include "mx4.hpp"
#include "train_ops.hpp"

namespace ma {

// Packing along the rows: 16 lanes hold a k-tile of 128 columns of one row, 8
// values per lane, 4 lanes a block of 32. A block of threads takes 16 rows and up to 4 k-tiles of
// each, all in flight: 1 KB of a row of bf16 and, for each k-tile, 64 bytes of scales at once
// (of narrower matrices, more rows). Along the rows, one k-tile after the other, with scales stored as
// bytes: 35 us for 16384 x 4096 bf16, so 33 (both with loads through the caches).
constexpr int kMx4Unroll = 4;

struct Mx4Place {
  int64_t row;
  int t;
  bool in;
};
// the place of part u of this thread block's 16 groups of lanes; log2t: 4 >> log2t rows apart
__device__ __forceinline__ Mx4Place mx4_place(const Mx4Args& a, int u, int kt, int log2t) {
  const int per = (kt + (1 << log2t) - 1) >> log2t;   // thread blocks along a row
  const uint32_t block = blockIdx.x / (uint32_t)per, at = blockIdx.x - block * per;
  Mx4Place p;
  p.row = (int64_t)block * (16 * kMx4Unroll >> log2t) + (u >> log2t) * 16 + threadIdx.x / 16;
  p.t = (int)(at << log2t) + (u & ((1 << log2t) - 1));
  p.in = p.row < a.rows && p.t < kt;
  return p;
}
static int mx4_log2t(int64_t kt) { return kt >= 3 ? 2 : (kt == 2 ? 1 : 0); }

template <int XD, bool NT>
__global__ void __launch_bounds__(256) k_mx4_pack(const Mx4Args a, int log2t) {
  const int lane = threadIdx.x & 15, kt = (int)mx4_tiles(a.cols);
  Raw8<XD> raw[kMx4Unroll];
#pragma unroll
  for (int u = 0; u < kMx4Unroll; ++u) {
    const Mx4Place p = mx4_place(a, u, kt, log2t);
    const int col = p.t * kMx4Tile + lane * 8;
    raw[u] = raw_zero<XD>();
    if (p.in && col < a.cols) raw[u] = raw_load_row<XD, NT>(elem_ptr<XD>(a.x, p.row * a.cols), col, a.cols);
  }
#pragma unroll
  for (int u = 0; u < kMx4Unroll; ++u) {
    const Mx4Place p = mx4_place(a, u, kt, log2t);
    const int col = p.t * kMx4Tile + lane * 8;
    float v[8];
    raw_f32_row<XD>(raw[u], col < a.cols ? col : 0, a.cols, v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      m = m > w ? m : w;
    }
    uint32_t o = dpp<kDppNeighbour>(m);
    m = m > o ? m : o;
    o = dpp<kDppPair>(m);
    m = m > o ? m : o;
    const uint32_t byte = mx4_scale_byte(m);
    // the k-tile's 4 bytes as one word, in every lane of its 16
    uint32_t word = byte << (8 * (lane / 4));
    word |= dpp<kDppHalfMirror>(word);
    word |= dpp<kDppMirror>(word);
    if (!p.in) continue;
    reinterpret_cast<uint32_t*>(a.q)[(p.row * kt + p.t) * 16 + lane] = mx4_encode(v, byte);
    if (lane == 0) reinterpret_cast<uint32_t*>(a.scale)[(int64_t)p.t * a.rows + p.row] = word;
  }
}

// Packing the transpose: a lane holds 32 rows of E columns (16 bytes of each row), so
// that every block of 32 is in one lane; 8 lanes take a line of each row, and the
// wave's 8 groups of them 8 blocks of rows: 256 rows become 128 bytes of each packed
// row, loaded and stored in whole lines without LDS. A block is one wave, as small matrices
// are a few of them (1003 x 333 fp32 in 5.1 us: 44 blocks, a chain of one load and one store).
template <int XD>
__global__ void __launch_bounds__(64) k_mx4_pack_t(const Mx4Args a) {
  typedef typename U16<XD>::T V;
  constexpr int E = 16 / elem_bytes<XD>();
  const int lane = threadIdx.x;
  const int64_t strips = (a.cols + 8 * E - 1) / (8 * E);
  const int64_t job = blockIdx.x, r0 = job / strips * 256 + (lane >> 3) * 32;
  const int64_t at = (job % strips) * (8 * E) + (lane & 7) * E;
  const int64_t kt = mx4_tiles(a.rows), padded = kt * kMx4Tile;
  if (at >= a.cols || r0 >= padded) return;
  // a row's last, partial group takes the row's last E columns: those it shares with
  // the lane before are packed by both, alike
  const bool narrow = a.cols < E;
  const int64_t col = narrow ? 0 : (at + E <= a.cols ? at : a.cols - E);
  u32x4_t raw[32];
#pragma unroll
  for (int r = 0; r < 32; ++r) raw[r] = u32x4_t{0u, 0u, 0u, 0u};
  if (narrow) {
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      if (r0 + r >= a.rows) continue;
      const unsigned char* p = elem_ptr<XD>(a.x, (r0 + r) * a.cols);
      if constexpr (XD == DT_F32) raw[r] = quad_load_row<XD>(p, 0, a.cols).u;
      else raw[r] = raw_load_row<XD>(p, 0, a.cols).u[0];
    }
  } else {
#pragma unroll
    for (int r = 0; r < 32; ++r)
      if (r0 + r < a.rows) raw[r] = *reinterpret_cast<const V*>(elem_ptr<XD>(a.x, (r0 + r) * a.cols + col));
  }
#pragma unroll
  for (int c = 0; c < E; ++c) {
    if (col + c >= a.cols) continue;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      uint32_t w;
      if constexpr (XD == DT_F32) w = raw[r][c];
      else w = c & 1 ? raw[r][c / 2] & 0xFFFF0000u : raw[r][c / 2] << 16;
      v[r] = __uint_as_float(w);
      w &= 0x7FFFFFFFu;
      m = m > w ? m : w;
    }
    const uint32_t byte = mx4_scale_byte(m);
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float part[8] = {v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3], v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]};
      q[i] = mx4_encode(part, byte);
    }
    *reinterpret_cast<u32x4_t*>(a.q + (col + c) * (padded / 2) + r0 / 2) = q;
    a.scale[((r0 / kMx4Tile) * a.cols + col + c) * 4 + (r0 / kMx4Block) % 4] = (uint8_t)byte;
  }
}

// Unpacking: the same lanes, k-tiles one after the other along the rows, as what it writes is the most
// (16384 x 4096 to bf16 29 us; in the packing's order 33).
template <int OD, bool NT>
__global__ void __launch_bounds__(256) k_mx4_unpack(const Mx4Args a) {
  const int lane = threadIdx.x & 15;
  const int64_t kt = mx4_tiles(a.cols), total = a.rows * kt;
  const int64_t b0 = (int64_t)blockIdx.x * (16 * kMx4Unroll) + threadIdx.x / 16;
  uint32_t q[kMx4Unroll], s[kMx4Unroll];
#pragma unroll
  for (int u = 0; u < kMx4Unroll; ++u) {
    const int64_t b = b0 + u * 16;
    q[u] = s[u] = 0;
    if (b < total) {
      const uint32_t row = (uint32_t)b / (uint32_t)kt, t = (uint32_t)b - row * (uint32_t)kt;   // at most 2^29 k-tiles
      q[u] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(a.q) + b * 16 + lane);
      s[u] = a.scale[((int64_t)t * a.rows + row) * 4 + lane / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < kMx4Unroll; ++u) {
    const int64_t b = b0 + u * 16;
    if (b >= total) continue;
    const uint32_t row = (uint32_t)b / (uint32_t)kt;
    const int col = (int)((uint32_t)b - row * (uint32_t)kt) * kMx4Tile + lane * 8;
    if (col >= a.cols) continue;
    float v[8];
    mx4_decode(q[u], mx4_scale(s[u]), v);
    store_row<OD, NT>(elem_ptr<OD>(a.out, (int64_t)row * a.cols), col, a.cols, v);
  }
}

static dim3 mx4_grid(const Mx4Args& a) {
  const int64_t kt = mx4_tiles(a.cols), log2t = mx4_log2t(kt), rows = 16 * kMx4Unroll >> log2t;
  return dim3((unsigned)((a.rows + rows - 1) / rows * ((kt + (1 << log2t) - 1) >> log2t)));
}

hipError_t launch_mx4_pack(const Mx4Args& a, int x_dt, bool transpose, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool f32 = x_dt == DT_F32;
  if (transpose) {
    const int64_t strip = f32 ? 32 : 64;
    const dim3 grid((unsigned)((a.rows + 255) / 256 * ((a.cols + strip - 1) / strip)));
    if (f32) hipLaunchKernelGGL(k_mx4_pack_t<DT_F32>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(k_mx4_pack_t<DT_BF16>, grid, dim3(64), 0, s, a);
    return hipGetLastError();
  }
  // bf16 x past the caches from half of what they keep (16384 x 4096 30 us against 33; 8192 x 2048,
  // written just before, 21.6 with its writer against 20.6); fp32 by 8 columns always through them (rows.hpp)
  const bool stream = a.rows * a.cols * 2 > kStreamBytes / 2;
  auto go = [&](auto k) { hipLaunchKernelGGL(k, mx4_grid(a), dim3(256), 0, s, a, mx4_log2t(mx4_tiles(a.cols))); };
  if (f32) go(k_mx4_pack<DT_F32, false>);
  else stream ? go(k_mx4_pack<DT_BF16, true>) : go(k_mx4_pack<DT_BF16, false>);
  return hipGetLastError();
}

hipError_t launch_mx4_unpack(const Mx4Args& a, int out_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool stream = a.rows * a.cols * 2 > kStreamBytes;   // (bf16 only, as in packing)
  const int64_t per = 16 * kMx4Unroll;
  const dim3 grid((unsigned)((a.rows * mx4_tiles(a.cols) + per - 1) / per));
  auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a); };
  if (out_dt == DT_F32) go(k_mx4_unpack<DT_F32, false>);
  else stream ? go(k_mx4_unpack<DT_BF16, true>) : go(k_mx4_unpack<DT_BF16, false>);
  return hipGetLastError();
}

}  // namespace ma
