// The product of a 4-bit weight matrix (mx4.hpp) with rows held in 4 bits or in 8
// (rows.hpp):
//   y[m,n] (+)= sum over k of x[m,k] * w[n,k]
// on the scaled matrix instructions of gfx950: 16 x 16 outputs and 128 k each, whose
// operands are e2m1 or e4m3 values with a power of two for every 32 k, and whose
// sums are fp32. Nothing is unpacked; products of held values are exact.
#include <type_traits>

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

// ---------------------------------------------------------------------------
// Many rows: output tiles of BM rows m and BN outputs n, by WGM x WGN waves of FM x FN
// blocks of 32 x 32.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) unsigned char lds_u8_t;

// BYTES per lane from memory into LDS, the lanes' side by side from `to` (the same for
// every lane); a single byte as a word.
template <int BYTES>
__device__ __forceinline__ void copy_lds(const uint8_t* from, lds_u8_t* to) {
  static_assert(BYTES == 16 || BYTES == 4 || BYTES == 1, "a chunk, a word or a byte");
  if constexpr (BYTES == 16) __builtin_amdgcn_global_load_lds(from, (lds_void_t*)to, 16, 0, 0);
  else if constexpr (BYTES == 4) __builtin_amdgcn_global_load_lds(from, (lds_void_t*)to, 4, 0, 0);
  else __builtin_amdgcn_global_load_lds(from, (lds_void_t*)to, 1, 0, 0);
}

template <int XB_, int WGM_, int WGN_, int FM_, int FN_, int STAGES_>
struct Mx4Tile {
  static constexpr int XB = XB_, WGM = WGM_, WGN = WGN_, FM = FM_, FN = FN_, STAGES = STAGES_;
  static constexpr int WTM = FM * 32, WTN = FN * 32, BM = WGM * WTM, BN = WGN * WTN, NW = WGM * WGN, NT = NW * 64;
  static constexpr int XR = XB == 8 ? 128 : 64, WR = 64;   // bytes of a row's k-tile
  // a stage: x's rows, w's rows, and a word of scales for each of them
  static constexpr int W_AT = BM * XR, S_AT = W_AT + BN * WR, STAGE = S_AT + (BM + BN) * 4;
  // copies of 1024 bytes (64 words of scales) per wave and k-tile
  static constexpr int NX = BM * XR / 1024 / NW, NWT = BN * WR / 1024 / NW, NS = (BM + BN) / 64 / NW, COPIES = NX + NWT + NS;
  static constexpr int LDE = WTN + 4;   // epilogue staging pitch (floats)
  static_assert(NX * NW * 1024 == BM * XR && NWT * NW * 1024 == BN * WR && NS * NW * 64 == BM + BN, "whole copies");
  static_assert((STAGES - 1) * COPIES <= 63, "vmcnt's range");
  static_assert(NW * 32 * LDE * 4 <= STAGES * STAGE && STAGES * STAGE <= 160 * 1024, "LDS");
};

// Until at most N of this wave's memory accesses are outstanding (they end in order).
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// One block per output tile and split of the k-tiles.
//
// LDS holds a ring of STAGES k-tiles of both operands as they are in memory, with
// their scales, copied there directly. Rows are 4 (8 bits: 8) chunks of 16 bytes, and
// 16 lanes of a read take 16 rows at one chunk: chunk c of row r lies at c ^ (r / 4)
// (c ^ (r / 2)), which spreads them over all banks. While the first half of k-tile t
// is multiplied, the second half's fragments are read; before the second half, k-tile
// t + 1 has landed and one barrier says so to every wave, after which its first
// fragments are read and k-tile t + STAGES is sent for into the stage just read.
template <typename TL, int YD>
__global__ void __launch_bounds__(TL::NT, TL::STAGES * TL::STAGE > 80 * 1024 ? TL::NW / 4 : TL::NW / 2) k_mx4_tile(const Mx4MatmulArgs a) {
  constexpr int XB = TL::XB, FM = TL::FM, FN = TL::FN, S = TL::STAGES;
  constexpr int XC = TL::XR / 16, XV = XB == 8 ? 2 : 1;   // chunks of a row, chunks per fragment
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S * TL::STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WGN, wn = wave % TL::WGN, l32 = lane & 31, g = lane >> 5;

  // job: split-major, then bands of 4 tile rows walked column by column; XCD b % 8
  // takes a contiguous eighth, so that its 32 CUs work on 4 x 8 tiles that share 4
  // panels of x and 8 of w in its L2
  const int64_t tm = (a.rows + TL::BM - 1) / TL::BM, tn = (a.outs + TL::BN - 1) / TL::BN, tiles = tm * tn;
  const int64_t jobs = tiles * a.splits, per = (jobs + 7) / 8;
  const int64_t job = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
  if (job >= jobs) return;
  const int split = (int)(job / tiles);
  const int64_t t = job - split * tiles, band = t / (4 * tn), rem = tm - band * 4, bh = rem < 4 ? rem : 4, idx = t - band * 4 * tn;
  const int64_t m0 = (band * 4 + idx % bh) * TL::BM, n0 = idx / bh * TL::BN;
  const int kt = (int)mx4_tiles(a.ins), v0 = (int)((int64_t)kt * split / a.splits), v1 = (int)((int64_t)kt * (split + 1) / a.splits);

  // this lane's place in each of its wave's copies: a 32-bit offset from the tile's first
  // row (rows past the end are read from the last one; their results are not stored)
  const int mlast = (int)(a.rows - m0 < TL::BM ? a.rows - m0 : TL::BM) - 1, nlast = (int)(a.outs - n0 < TL::BN ? a.outs - n0 : TL::BN) - 1;
  uint32_t xoff[TL::NX], woff[TL::NWT], soff[TL::NS];
#pragma unroll
  for (int q = 0; q < TL::NX; ++q) {
    const int r = (wave * TL::NX + q) * (64 / XC) + lane / XC, c = (lane % XC) ^ (XB == 8 ? (r >> 1) & 7 : (r >> 2) & 3);
    xoff[q] = (uint32_t)(r < mlast ? r : mlast) * (uint32_t)(kt * TL::XR) + (uint32_t)c * 16;
  }
#pragma unroll
  for (int q = 0; q < TL::NWT; ++q) {
    const int r = (wave * TL::NWT + q) * 16 + lane / 4, c = (lane % 4) ^ ((r >> 2) & 3);
    woff[q] = (uint32_t)(r < nlast ? r : nlast) * (uint32_t)(kt * TL::WR) + (uint32_t)c * 16;
  }
#pragma unroll
  for (int q = 0; q < TL::NS; ++q) {
    const int r = (wave * TL::NS + q) * 64 + lane, rx = r < mlast ? r : mlast, rw = r - TL::BM < nlast ? r - TL::BM : nlast;
    soff[q] = r < TL::BM ? (uint32_t)rx * (XB == 8 ? (uint32_t)kt : 4u) : (uint32_t)rw * 4;
  }
  const uint8_t* const xq = a.xq + m0 * kt * TL::XR;
  const uint8_t* const wq = a.wq + n0 * kt * TL::WR;
  const uint8_t* const xs = a.xscale + m0 * (XB == 8 ? kt : 4);
  const uint8_t* const ws = a.wscale + n0 * 4;
  const int64_t xs_step = XB == 8 ? 1 : a.rows * 4, ws_step = (int64_t)a.outs * 4;
  lds_u8_t* const lds = (lds_u8_t*)smem;
  // copy i of this wave's share of k-tile v
  auto copy = [&](int v, lds_u8_t* st, int i) __attribute__((always_inline)) {
    if (i < TL::NX) {
      copy_lds<16>(xq + (int64_t)v * TL::XR + xoff[i], st + (wave * TL::NX + i) * 1024);
    } else if (i < TL::NX + TL::NWT) {
      const int q = i - TL::NX;
      copy_lds<16>(wq + (int64_t)v * TL::WR + woff[q], st + TL::W_AT + (wave * TL::NWT + q) * 1024);
    } else {
      const int q = i - TL::NX - TL::NWT, r = (wave * TL::NS + q) * 64;
      lds_u8_t* const to = st + TL::S_AT + r * 4;
      if (r >= TL::BM) copy_lds<4>(ws + v * ws_step + soff[q], to);
      else copy_lds<XB == 8 ? 1 : 4>(xs + v * xs_step + soff[q], to);
    }
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // fragments of half h of a k-tile: lane (l32, g) holds row l32 of each block and 32 values
  // from 64 h + 32 g (8 bits: two times 16, from 64 h + 16 g and 32 further)
  u32x4_t fx[2][FM][XV], fw[2][FN];
  int sx[FM], sw[FN], nx[FM], nw[FN];   // this k-tile's scales, and the next one's as they are in LDS
  int xat[FM], wat[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) xat[i] = (wm * TL::WTM + i * 32 + l32) * TL::XR;
#pragma unroll
  for (int j = 0; j < FN; ++j) wat[j] = TL::W_AT + (wn * TL::WTN + j * 32 + l32) * TL::WR;
  const int swx = XB == 8 ? (l32 >> 1) & 7 : (l32 >> 2) & 3, sww = (l32 >> 2) & 3;
  constexpr int READS = FM * XV + FN;
  auto read = [&](lds_u8_t* st, int h, int i) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
    if (i < FM * XV) {
      const int c = XB == 8 ? 4 * h + 2 * (i % XV) + g : 2 * h + g;
      fx[h][i / XV][i % XV] = *(lds_u32x4_t*)(st + xat[i / XV] + ((c ^ swx) << 4));
    } else {
      fw[h][i - FM * XV] = *(lds_u32x4_t*)(st + wat[i - FM * XV] + (((2 * h + g) ^ sww) << 4));
    }
  };
  auto scales = [&](lds_u8_t* st, int i) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) int lds_int_t;
    if (i < FM) nx[i] = *(lds_int_t*)(st + TL::S_AT + (wm * TL::WTM + i * 32 + l32) * 4);
    else nw[i - FM] = *(lds_int_t*)(st + TL::S_AT + (TL::BM + wn * TL::WTN + (i - FM) * 32 + l32) * 4);
  };
  // byte 2 h of a word moved down by g bytes is the lane's
  auto take = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = XB == 4 ? (int)((unsigned)nx[i] >> (8 * g)) : nx[i];
#pragma unroll
    for (int j = 0; j < FN; ++j) sw[j] = (int)((unsigned)nw[j] >> (8 * g));
  };
  auto multiply = [&](auto half, int i, int j) __attribute__((always_inline)) {
    constexpr int h = decltype(half)::value;
    const u32x4_t &u = fw[h][j], &x0 = fx[h][i][0], &x1 = fx[h][i][XV - 1];
    const i32x8_t w = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], 0, 0, 0, 0};
    const i32x8_t x = XB == 8 ? i32x8_t{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]}
                              : i32x8_t{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], 0, 0, 0, 0};
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc[i][j], kFmt4, XB == 8 ? kFmt8 : kFmt4, 2 * h, sw[j], XB == 8 ? 0 : 2 * h, sx[i]);
  };
  typedef std::integral_constant<int, 0> First;
  typedef std::integral_constant<int, 1> Second;
  // reads per MFMA: the last one is sent for well before its half ends
  constexpr int MM = FM * FN, PACE = (READS + MM / 2 - 1) / (MM / 2);

  // k-tile v, its first fragments and scales in registers. FILL: k-tile v + S exists.
  lds_u8_t* cur = lds;
  auto tile = [&](int v, auto fill) __attribute__((always_inline)) {
    constexpr bool FILL = decltype(fill)::value;
    lds_u8_t* const nxt = cur == lds + (S - 1) * TL::STAGE ? lds : cur + TL::STAGE;
#pragma unroll
    for (int k = 0; k < MM; ++k) {
      multiply(First(), k / FN, k % FN);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = k * PACE; i < (k + 1) * PACE && i < READS; ++i) read(cur, 1, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave has read all of k-tile v
    const bool more = FILL || v + 1 < v1;
    if (more) {
      if (FILL) {
        wait_vm<(S - 2) * TL::COPIES>();
      } else {
        const int later = v1 - 2 - v;   // k-tiles sent for after v + 1
        if (later >= 2 && S > 3) wait_vm<(S > 3 ? 2 : 0) * TL::COPIES>();
        else if (later >= 1 && S > 2) wait_vm<(S > 2 ? 1 : 0) * TL::COPIES>();
        else wait_vm<0>();
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < MM; ++k) {
      multiply(Second(), k / FN, k % FN);
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        constexpr int ALL = FM + FN + READS;
#pragma unroll
        for (int i = k * 2 * PACE; i < (k + 1) * 2 * PACE && i < ALL; ++i) {
          if (i < FM + FN) scales(nxt, i);
          else read(nxt, 0, i - FM - FN);
        }
      }
      if (FILL) {
#pragma unroll
        for (int i = k * TL::COPIES / MM; i < (k + 1) * TL::COPIES / MM; ++i) copy(v + S, cur, i);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    take();
    cur = nxt;
  };
  typedef std::integral_constant<bool, true> Fill;
  typedef std::integral_constant<bool, false> Last;
#pragma unroll
  for (int v = 0; v < S; ++v) {
    if (v0 + v < v1) {
#pragma unroll
      for (int i = 0; i < TL::COPIES; ++i) copy(v0 + v, lds + v * TL::STAGE, i);
    }
  }
  if (v1 - v0 >= S) wait_vm<(S - 1) * TL::COPIES>();
  else wait_vm<0>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM + FN; ++i) scales(lds, i);
#pragma unroll
  for (int i = 0; i < READS; ++i) read(lds, 0, i);
  take();
  int v = v0;
  for (; v < v1 - S; ++v) tile(v, Fill());
  for (; v < v1; ++v) tile(v, Last());

  // 32 rows of the wave's block at a time through its own part of LDS, so that stores are
  // 8 consecutive values per lane
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  float* const mine = reinterpret_cast<float*>(smem) + wave * 32 * TL::LDE;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<float4*>(mine + l32 * TL::LDE + j * 32 + b * 8 + g * 4) =
            make_float4(acc[i][j][4 * b], acc[i][j][4 * b + 1], acc[i][j][4 * b + 2], acc[i][j][4 * b + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < 32 * TL::WTN / 512; ++u) {
      constexpr int LPR = TL::WTN / 8;
      const int row = u * (64 / LPR) + lane / LPR, c = lane % LPR * 8;
      const float4 x = *reinterpret_cast<const float4*>(mine + row * TL::LDE + c), y = *reinterpret_cast<const float4*>(mine + row * TL::LDE + c + 4);
      float o[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const int64_t m = m0 + wm * TL::WTM + i * 32 + row;
      const int n = (int)n0 + wn * TL::WTN + c;
      if (m >= a.rows || n >= a.outs) continue;
      if (a.splits > 1) {
        store_row<DT_F32>(elem_ptr<DT_F32>(a.partial, split * mx4_partial(a.rows, a.outs) + m * a.outs), n, a.outs, o);
        continue;
      }
      unsigned char* out = elem_ptr<YD>(a.y, m * a.outs);
      if (a.accumulate) {
        float old[8];
        raw_f32_row<YD>(raw_load_row<YD>(out, n, a.outs), n, a.outs, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __fadd_rn(old[e], o[e]);
      }
      store_row<YD>(out, n, a.outs, o);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The splits' partial products, added in order: 4 consecutive values per thread, 8
// splits in flight.
template <int YD>
__global__ void __launch_bounds__(256) k_mx4_join(const Mx4MatmulArgs a) {
  const int64_t total = a.rows * a.outs, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  float v[4] = {};
  const int n = total - i < 4 ? (int)(total - i) : 4;
  const int64_t stride = mx4_partial(a.rows, a.outs);   // past the end there is room, not read further
  constexpr int U = 8;
  for (int s = 0; s < a.splits; s += U) {
    u32x4_t x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = u32x4_t{0u, 0u, 0u, 0u};
      if (s + u < a.splits) x[u] = *reinterpret_cast<const u32x4_t*>(a.partial + (s + u) * stride + i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __uint_as_float(x[u][e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= n) continue;
    if (a.accumulate) v[e] = __fadd_rn(load1<YD>(a.y, i + e), v[e]);
    store1<YD>(a.y, i + e, v[e]);
  }
}

Mx4Plan mx4_plan(int64_t rows, int64_t outs, int64_t ins, int x_bits) {
  (void)ins;
  (void)x_bits;
  if (rows <= 64) return {0, 1};
  return {rows > 128 && outs > 128 ? 256 : 128, 1};
}

template <typename TL, int YD>
static hipError_t mx4_tile(const Mx4MatmulArgs& a, hipStream_t s) {
  const int64_t jobs = ((a.rows + TL::BM - 1) / TL::BM) * ((a.outs + TL::BN - 1) / TL::BN) * a.splits;
  hipLaunchKernelGGL((k_mx4_tile<TL, YD>), dim3((unsigned)((jobs + 7) / 8 * 8)), dim3(TL::NT), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  hipLaunchKernelGGL((k_mx4_join<YD>), dim3((unsigned)((a.rows * a.outs + 1023) / 1024)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int XB, int YD>
static hipError_t mx4_product(const Mx4MatmulArgs& a, hipStream_t s) {
  if (a.edge == 256) return mx4_tile<Mx4Tile<XB, 2, 2, 4, 4, XB == 8 ? 3 : 4>, YD>(a, s);
  if (a.edge == 128) return mx4_tile<Mx4Tile<XB, 2, 2, 2, 2, XB == 8 ? 3 : 4>, YD>(a, s);
  return a.rows <= 16 ? mx4_rows<XB, YD, 1>(a, 4, s) : mx4_rows<XB, YD, 4>(a, 4, s);
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int x_bits, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_bits == 8) return y_dt == DT_F32 ? mx4_product<8, DT_F32>(a, s) : mx4_product<8, DT_BF16>(a, s);
  return y_dt == DT_F32 ? mx4_product<4, DT_F32>(a, s) : mx4_product<4, DT_BF16>(a, s);
}

}  // namespace ma
