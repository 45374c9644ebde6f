// The product of a 4-bit weight matrix (mx4.hpp) with rows held in 4 bits or in 8
// (rows.hpp):
//   y[m,n] (+)= sum over k of x[m,k] * w[n,k]
// on the scaled matrix instructions of gfx950: 16 x 16 outputs and 128 k each, whose
// operands are e2m1 or e4m3 values with a power of two for every 32 k, and whose
// sums are fp32. Nothing is unpacked; products of held values are exact, and their sums cut nothing off
// (8-bit rows take two instructions for that, see mx_exact).
//
// Two kernels: few rows are bound by reading w (k_mx4_rows), many by the matrix instructions
// (k_mx4_tile). On random data the chip's power holds those alone to 7.28 PFLOP/s for 4-bit
// rows and 4.66 for 8-bit ones (9.6 and 5.0 on zeros); of 32 x 32 x 64 to 6.4 and 4.2.
#include <algorithm>
#include <type_traits>
#include <utility>

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

// The instructions add 8 consecutive k at a time, their products cut off towards zero at 2^-13 of the largest
// one's power of two (the product of its factors'), and these sums in fp32. Products of two 4-bit values are
// whole all the same. Those with 8-bit values lose bits beside a large one, up to 7 * 2^-13 of it and always towards
// zero: 2e-5 of a result on even data, but all of it where large products cancel. So the 8-bit operand
// goes in two parts, and nothing is cut off: values of 2 .. 448, whose products are multiples of 2^-3, the
// largest's power of two at most 2^10; and those below, multiples of 2^-10, at most 2^2. That takes twice the
// instructions: 12288 x (4096 x 16384) to bf16 takes 1150 us, in one part 573.
template <int XB> constexpr bool mx_exact = XB == 8;
// The values of 2 and more (and NaN), bit 6 of each byte; the others 0.
__device__ __forceinline__ i32x8_t mx_large(const i32x8_t& x) {
  i32x8_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // selectors 12 and 13 are the bytes 0x00 and 0xFF
    const uint32_t pick = ((uint32_t)x[i] >> 6 & 0x01010101u) | 0x0C0C0C0Cu;
    r[i] = x[i] & (int)__builtin_amdgcn_perm(0u, 0u, pick);
  }
  return r;
}

// Few rows: a block takes 16 outputs n of MB * 16 rows m, each wave a contiguous share of the
// k-tiles; the waves' sums are added in order in LDS. The operands go from memory to
// registers, several k-tiles at once: lane l holds row l % 16 and, of every k-tile,
// 32 values from 32 * (l / 16) (of 8-bit rows two times 16, from 16 * (l / 16) and 64
// further: so the instruction pairs them with 4-bit ones). Rows past the end are read
// from inside the matrix; their results are not stored.
//   1 x (16384 x 4096) of 8 bits 10.9 us, 3.3 TB/s (4 k-tiles in flight; 8: no faster), of 4 bits 8.8;
//   129 x (1003 x 333) of 4 bits 6.2, a chain of two loads, the join and a store
template <int XB, int YD, int MB>
__global__ void __launch_bounds__(512) k_mx4_rows(const Mx4MatmulArgs a) {
  extern __shared__ float join[];   // [waves][MB][64][4]
  constexpr int U = MB == 1 ? 4 : 2, XV = XB == 8 ? 2 : 1;   // k-tiles in flight
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
  auto tiles = [&](int t, auto count) __attribute__((always_inline)) {
    constexpr int N = decltype(count)::value;
    u32x4_t w[N], x[N][MB][XV];
    int sw[N], sx[N][MB];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int64_t at = t + u;
      w[u] = *reinterpret_cast<const u32x4_t*>(wq + at * 64);
      sw[u] = ws[at * a.outs * 4];
#pragma unroll
      for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int v = 0; v < XV; ++v) x[u][b][v] = *reinterpret_cast<const u32x4_t*>(xq[b] + at * (64 * XV) + v * 64);
        sx[u][b] = XB == 8 ? xs[b][at] : xs[b][at * a.rows * 4];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const i32x8_t w8 = {(int)w[u][0], (int)w[u][1], (int)w[u][2], (int)w[u][3], 0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const u32x4_t &p = x[u][b][0], &q = x[u][b][XV - 1];
        const i32x8_t x8 = XB == 8 ? i32x8_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)q[0], (int)q[1], (int)q[2], (int)q[3]}
                                   : i32x8_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
        if constexpr (mx_exact<XB>) {
          const i32x8_t large = mx_large(x8);
          acc[b] = mx_mfma16<XB>(w8, large, acc[b], sw[u], sx[u][b]);
          acc[b] = mx_mfma16<XB>(w8, x8 ^ large, acc[b], sw[u], sx[u][b]);
        } else {
          acc[b] = mx_mfma16<XB>(w8, x8, acc[b], sw[u], sx[u][b]);
        }
      }
    }
  };
  int t = k0;
  for (; t + U <= k1; t += U) tiles(t, std::integral_constant<int, U>());
  for (; t < k1; ++t) tiles(t, std::integral_constant<int, 1>());
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

// ---------------------------------------------------------------------------
// Many rows: output tiles of BM rows m and BN outputs n, by WGM x WGN waves of FM x FN
// blocks of 16 x 16.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) unsigned char lds_u8_t;

// 16 bytes per lane from memory, at base + off, into LDS, the lanes' side by side from `to` (base
// and `to` the same for every lane). In assembler, as the compiler waits for all LDS reads at
// each one's use where it knows of such a copy under way. Nothing is loaded into a register. A copy
// comes one wait state after m0 was written (wait_states.py checks that, and the others below). m0 is
// reserved: the compiler keeps nothing in it, and cannot be told of it.
__device__ __forceinline__ void copy_chunks(const uint8_t* base, uint32_t off, lds_u8_t* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(at), "v"(off), "s"(base) : "memory");
}
// A word, or a byte as a word, of the first 32 lanes.
template <int BYTES>
__device__ __forceinline__ void copy_words(const uint8_t* base, uint32_t off, lds_u8_t* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to);
  uint64_t all;
#define MA_COPY(op) \
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, exec\n\ts_mov_b32 exec_hi, 0\n\t" op " %2, %3\n\ts_mov_b64 exec, %0" : "=&s"(all) : "s"(at), "v"(off), "s"(base) : "memory")
  if constexpr (BYTES == 4) MA_COPY("global_load_lds_dword");
  else MA_COPY("global_load_lds_ubyte");
#undef MA_COPY
}

template <int XB_, int WGM_, int WGN_, int FM_, int FN_, int STAGES_>
struct Mx4Tile {
  static constexpr int XB = XB_, WGM = WGM_, WGN = WGN_, FM = FM_, FN = FN_, STAGES = STAGES_;
  static constexpr int WTM = FM * 16, WTN = FN * 16, BM = WGM * WTM, BN = WGN * WTN, NW = WGM * WGN, NT = NW * 64;
  static constexpr int XR = XB == 8 ? 128 : 64, WR = 64;   // bytes of a row's k-tile
  // a stage: x's rows, w's rows, and a word of scales for each of them
  static constexpr int W_AT = BM * XR, S_AT = W_AT + BN * WR, STAGE = S_AT + (BM + BN) * 4;
  // copies of 1024 bytes, and of 32 rows' scales of each operand, per wave and k-tile
  static constexpr int NX = BM * XR / 1024 / NW, NWT = BN * WR / 1024 / NW, COPIES = NX + NWT + 2;
  static constexpr int BLOCKS = STAGES * STAGE > 80 * 1024 ? 1 : 2;   // per CU
  static_assert(NX * NW * 1024 == BM * XR && NWT * NW * 1024 == BN * WR && BM == 32 * NW && BN == 32 * NW, "whole copies");
  static_assert((STAGES - 1) * COPIES <= 63 && STAGES >= 3 && STAGES <= 4, "vmcnt's range, the waits");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

// Until at most N of this wave's memory accesses are outstanding (they end in order).
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// This wave's LDS reads are done, then the block's barrier.
__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// acc += w x, 16 x 16 outputs and 128 k, in place: from the builtin the compiler makes a new
// accumulator each time, and moves them all. What a vector instruction wrote is read two wait states
// later at the earliest, which the compiler does not see to here. FRESH: w, x or a scale may
// have been computed by the instruction before. acc: cleared() has the wait. Whoever reads acc
// otherwise calls settled() first.
template <int XB> struct MxRow { typedef u32x4_t T; };   // a lane's 32 values of x
template <> struct MxRow<8> { typedef i32x8_t T; };
template <int XB, bool FRESH>
__device__ __forceinline__ void mx_mfma16_into(f32x4_t& acc, u32x4_t w, typename MxRow<XB>::T x, int ws, int xs) {
#if defined(__HIP_DEVICE_COMPILE__)   // (the host's pass knows other registers)
#define MA_MFMA(wait, fmt)                                                                                                   \
  asm volatile(wait "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:" fmt : "+v"(acc) : "v"(w), "v"(x), "v"(ws), "v"(xs))
  if constexpr (XB == 8) {
    if constexpr (FRESH) MA_MFMA("s_nop 1\n\t", "0"); else MA_MFMA("", "0");
  } else {
    if constexpr (FRESH) MA_MFMA("s_nop 1\n\t", "4"); else MA_MFMA("", "4");
  }
#undef MA_MFMA
#endif
}

// The MFMAs into these 4 accumulators are done: 16 passes and more have gone by.
__device__ __forceinline__ void settled(f32x4_t& a, f32x4_t& b, f32x4_t& c, f32x4_t& d) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 15\n\ts_nop 7" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
#endif
}

// Zeros in these 4 accumulators, and two wait states. They are written here: plain zeros the compiler
// writes again right in front of the MFMA that reads them first.
__device__ __forceinline__ void cleared(f32x4_t& a, f32x4_t& b, f32x4_t& c, f32x4_t& d) {
  a = b = c = d = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 1" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
#endif
}

// What a row's chunks of 16 bytes are exchanged by. A read of a fragment takes 16 rows at 4
// chunks g, lane 16 g + r; LDS serves lanes 0-3, 12-15 and 20-27 together, then 4-11, 16-19
// and 28-31, the others alike: rows 0-3 and 12-15 at one chunk beside rows 4-11 at the next.
// With these values each time all 64 banks are met once.
template <int CHUNKS>
__device__ __forceinline__ int spread(int r) {
  return CHUNKS == 8 ? ((r >> 1) + 2) & 7 : -(r >> 2) & 3;
}

// f(0), f(1), .. f(N - 1), each with its number as a constant.
template <typename F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each(f, std::make_integer_sequence<int, N>());
}

// 8 consecutive outputs per lane of 16 x 32: from two blocks' accumulators, where lane (l16, g)
// has outputs 4 g .. 4 g + 3 of its row, those of 8 g .. 8 g + 7 as packed bf16.
__device__ __forceinline__ u32x4_t pack_pair(const f32x4_t& a, const f32x4_t& b) {
  typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = pack_bf16x2(a[2 * i], a[2 * i + 1]), y = pack_bf16x2(b[2 * i], b[2 * i + 1]);
    const u32x2_t u = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(x, y, false, false));
    const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(u.x, u.y, false, false));
    lo[i] = v.x;
    hi[i] = v.y;
  }
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// Of two parts of 16 rows, in which lane (l16, g) has chunk g of row l16: the first 8 rows of both
// side by side, lanes 8 .. 15 of each 16 having p's last rows' place taken by q's first, and the last 8.
__device__ __forceinline__ void rows_side_by_side(u32x4_t& p, u32x4_t& q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = (int)p[i], b = (int)q[i];
    p[i] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false);   // lanes 8..15 from 8 lanes below, of q
    q[i] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false);   // lanes 0..7 from 8 above, of p
  }
}

// An output tile and split of the k-tiles.
struct Mx4Job {
  int m0, n0, split, v0, v1;
};

// Persistent blocks, each of which works on a list of output tiles.
//
// LDS holds a ring of STAGES k-tiles of both operands as they are in memory, with
// their scales, copied there directly. Rows are 4 (8 bits: 8) chunks of 16 bytes; chunk c
// of row r lies at c ^ spread(r), see there.
//
// A k-tile's MFMAs go by pairs of x's blocks and, within a pair, w's blocks. In the first
// half of them x of the later pairs is read; then the next k-tile has landed and one barrier
// says so to every wave, and that every wave has read all of this one. In the second half the
// first pair of x of the next k-tile is read, and w's blocks take the place of the present ones
// as the last pair is done with them. Copies of the k-tile STAGES further into the stage just
// read are spread over the k-tile's length from there. The loop turns at the barrier, where
// nothing is under way from LDS: at a turn the compiler waits for all that is.
//
// The k-tiles of one output tile follow on those of the one before: its first ones are copied,
// and its first fragments read, before the results are stored, and the stores end while it is
// worked on. Results go from the registers to memory, without LDS or a barrier.
//
// Measured, call after call: 12288 x (16384 x 4096) of 4 bits 423 to 437 us, 3.8 PFLOP/s, the matrix units busy for 44 %
// of the cycles at 1.9 GHz; 12288 x (4096 x 16384) of 8 bits 1150, 1.4, 59 % at 1.9 GHz. A k-tile of 256 x 256 takes 0.9 us
// (4 bits; 2.9 of 8), of which the MFMAs alone are 0.61, the LDS reads alone 0.78, the copies alone 0.77; the
// stores at a tile's end 5 us (bf16) to 15 (fp32), with all blocks' at the same time. Tried, and no faster: blocks
// started at different times (+1 to +8 %), 4 waves of 128 x 128 (spills), 32 x 32 x 64 instructions,
// copies in the k-tile's first part, branches between the MFMAs that spread the waves' copies.
// ADDS: results are added to y (whole sums only), in kernels of their own: in one with the others,
// 12288 x (16384 x 4096) of 4 bits takes 569 us, else 523 on the same card.
template <typename TL, int YD, bool ADDS>
__global__ void __launch_bounds__(TL::NT, TL::NW * TL::BLOCKS / 4) k_mx4_tile(const Mx4MatmulArgs a) {
  constexpr int XB = TL::XB, FM = TL::FM, FN = TL::FN, S = TL::STAGES;
  constexpr int XC = TL::XR / 16;   // chunks of a row
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S * TL::STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WGN, wn = wave % TL::WGN, l16 = lane & 15, g = lane >> 4;
  const int kt = (int)mx4_tiles(a.ins);

  // jobs: split-major, then bands of 4 tile rows walked column by column; XCD b % 8
  // takes a contiguous eighth, and its blocks every 32nd (64th) of it: at a time they work
  // on 4 x 8 tiles that share 4 panels of x and 8 of w in its L2
  // (fewer than 2^29 jobs)
  const int tm = (int)((a.rows + TL::BM - 1) / TL::BM), tn = (a.outs + TL::BN - 1) / TL::BN, tiles = tm * tn;
  const int jobs = tiles * a.splits, per = (jobs + 7) / 8, first_job = (int)(blockIdx.x % 8) * per;
  const int end_job = first_job + per < jobs ? first_job + per : jobs, stride = (int)(gridDim.x / 8);
  // (divisions leave the scalar registers)
  auto scalar = [](int x) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(x); };
  auto job_at = [&](int job) __attribute__((always_inline)) {
    Mx4Job j;
    j.split = scalar(job / tiles);
    const int t = job - j.split * tiles, band = scalar(t / (4 * tn)), rem = tm - band * 4, bh = rem < 4 ? rem : 4, idx = t - band * 4 * tn;
    const int column = scalar(idx / bh);
    j.m0 = (band * 4 + idx - column * bh) * TL::BM;
    j.n0 = column * TL::BN;
    j.v0 = scalar((int)((int64_t)kt * j.split / a.splits));
    j.v1 = scalar((int)((int64_t)kt * (j.split + 1) / a.splits));
    return j;
  };
  int job = first_job + (int)(blockIdx.x / 8);
  if (job >= end_job) return;

  // where the copies are: the next k-tile's rows and scales, how many k-tiles of the job are left,
  // and this lane's place in each of its wave's copies, a 32-bit offset from the tile's first row
  // (rows past the end are read from the last one; their results are not stored)
  const uint8_t *xq, *wq, *xs, *ws;
  int left;
  uint32_t xoff[TL::NX], woff[TL::NWT], sxoff, swoff;
  const int64_t xs_step = XB == 8 ? 1 : a.rows * 4, ws_step = (int64_t)a.outs * 4;
  auto copies_of = [&](const Mx4Job& j) __attribute__((always_inline)) {
    const int mlast = (int)(a.rows - j.m0 < TL::BM ? a.rows - j.m0 : TL::BM) - 1, nlast = (int)(a.outs - j.n0 < TL::BN ? a.outs - j.n0 : TL::BN) - 1;
#pragma unroll
    for (int q = 0; q < TL::NX; ++q) {
      const int r = (wave * TL::NX + q) * (64 / XC) + lane / XC, c = (lane % XC) ^ spread<XC>(r);
      xoff[q] = (uint32_t)(r < mlast ? r : mlast) * (uint32_t)(kt * TL::XR) + (uint32_t)c * 16;
    }
#pragma unroll
    for (int q = 0; q < TL::NWT; ++q) {
      const int r = (wave * TL::NWT + q) * 16 + lane / 4, c = (lane % 4) ^ spread<4>(r);
      woff[q] = (uint32_t)(r < nlast ? r : nlast) * (uint32_t)(kt * TL::WR) + (uint32_t)c * 16;
    }
    // scales: those of rows r, r + 16, r + 32 and r + 48 lie side by side
    const int r = wave / 2 * 64 + lane % 4 * 16 + wave % 2 * 8 + (lane & 31) / 4;
    sxoff = (uint32_t)(r < mlast ? r : mlast) * (XB == 8 ? (uint32_t)kt : 4u);
    swoff = (uint32_t)(r < nlast ? r : nlast) * 4u;
    xq = a.xq + ((int64_t)j.m0 * kt + j.v0) * TL::XR;
    wq = a.wq + ((int64_t)j.n0 * kt + j.v0) * TL::WR;
    xs = a.xscale + (XB == 8 ? (int64_t)j.m0 * kt + j.v0 : (j.v0 * a.rows + j.m0) * 4);
    ws = a.wscale + ((int64_t)j.v0 * a.outs + j.n0) * 4;
    left = j.v1 - j.v0;
  };
  lds_u8_t* const lds = (lds_u8_t*)smem;
  // copy i of this wave's share of the next k-tile
  auto copy = [&](lds_u8_t* st, int i) __attribute__((always_inline)) {
    if (i < TL::NX) copy_chunks(xq, xoff[i], st + (wave * TL::NX + i) * 1024);
    else if (i < TL::NX + TL::NWT) copy_chunks(wq, woff[i - TL::NX], st + TL::W_AT + (wave * TL::NWT + i - TL::NX) * 1024);
    else if (i == TL::NX + TL::NWT) copy_words<XB == 8 ? 1 : 4>(xs, sxoff, st + TL::S_AT + wave * 128);
    else copy_words<4>(ws, swoff, st + TL::S_AT + TL::BM * 4 + wave * 128);
  };
  int copy_job = job;
  // on to the next k-tile, of the next job after the last; behind the last job the last k-tile
  // is copied again, to no use
  auto copied = [&]() __attribute__((always_inline)) {
    if (--left > 0) {
      xq += TL::XR;
      wq += TL::WR;
      xs += xs_step;
      ws += ws_step;
    } else if (copy_job + stride < end_job) {
      copy_job += stride;
      copies_of(job_at(copy_job));
    }
  };

  f32x4_t acc[FM][FN];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int b = 0; b < FN; b += 4) cleared(acc[i][b], acc[i][b + 1], acc[i][b + 2], acc[i][b + 3]);
  };
  clear();

  // fragments: lane (l16, g) holds row l16 of each block and 32 values from 32 g (8 bits: two
  // times 16, from 16 g and 64 further), and their scale
  typename MxRow<XB>::T fx[FM];
  u32x4_t fw[FN];
  int rx[FM], rw[FN], sx[2], sw[FN];   // words of scales as they are in LDS; a pair's and w's, moved down to the lane's byte
  const int swx = spread<XC>(l16), sww = spread<4>(l16);
  const int xat = (wm * TL::WTM + l16) * TL::XR, wat = TL::W_AT + (wn * TL::WTN + l16) * TL::WR + ((g ^ sww) << 4);
  const int xat0 = xat + ((g ^ swx) << 4), xat1 = xat + (((4 + g) ^ swx) << 4);
  const int sxat = TL::S_AT + wm * TL::WTM * 4 + l16 * 16, swat = TL::S_AT + (TL::BM + wn * TL::WTN) * 4 + l16 * 16;
  typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
  auto read_x = [&](lds_u8_t* st, int i) __attribute__((always_inline)) {
    const u32x4_t lo = *(lds_u32x4_t*)(st + xat0 + i * 16 * TL::XR);
    if constexpr (XB == 8) {
      const u32x4_t hi = *(lds_u32x4_t*)(st + xat1 + i * 16 * TL::XR);
      fx[i] = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    } else {
      fx[i] = lo;
    }
  };
  auto read_w = [&](lds_u8_t* st, int j) __attribute__((always_inline)) { fw[j] = *(lds_u32x4_t*)(st + wat + j * 16 * TL::WR); };
  // the scales of 4 blocks at once: a quarter of the reads (12288 x (4096 x 16384) of 8 bits onto fp32 1144 -> 1119 us)
  auto read_sx = [&](lds_u8_t* st, int four) __attribute__((always_inline)) {
    const u32x4_t v = *(lds_u32x4_t*)(st + sxat + four * 256);
#pragma unroll
    for (int i = 0; i < 4; ++i) rx[four * 4 + i] = (int)v[i];
  };
  auto read_sw = [&](lds_u8_t* st) __attribute__((always_inline)) {
    const u32x4_t v = *(lds_u32x4_t*)(st + swat);
#pragma unroll
    for (int j = 0; j < 4; ++j) rw[j] = (int)v[j];
  };
  constexpr int MM = FM * FN, HALF = MM / 2, LATER = FM - 2;   // LATER: reads of x in the first half
  // copies after every SPACE-th MFMA from the barrier on
  constexpr int SPACE = MM / TL::COPIES;
  static_assert(SPACE >= 1 && (FM == 4 || FM == 8) && FN == 4 && LATER <= HALF * 3 / 4, "copies and reads fit between the MFMAs");

  // MFMA k of a k-tile, from the scales' words on; EXACT: two of them, x block by x block, the large
  // parts of x for all of w's blocks and then the others
  constexpr bool EXACT = mx_exact<XB>;
  typename MxRow<XB>::T large;
  auto step = [&](auto number) __attribute__((always_inline)) {
    constexpr int k = decltype(number)::value;
    if constexpr (EXACT) {
      constexpr int i = k / FN, part = k % FN / (FN / 2), j0 = k % (FN / 2) * 2;
      if constexpr (j0 == 0 && part == 0) {
        sx[0] = rx[i];
        large = mx_large(fx[i]);
        fx[i] = fx[i] ^ large;
      }
      each<2>([&](auto other) __attribute__((always_inline)) {
        constexpr int j = j0 + decltype(other)::value;
        if constexpr (i == 0 && part == 0) sw[j] = (int)((unsigned)rw[j] >> (8 * g));
        mx_mfma16_into<XB, (i == 0 && part == 0) || j == 0>(acc[i][j], fw[j], part == 0 ? large : fx[i], sw[j], sx[0]);
      });
    } else {
      constexpr int i = k / (2 * FN) * 2 + k % 2, j = k % (2 * FN) / 2;
      if constexpr (i == 0) sw[j] = (int)((unsigned)rw[j] >> (8 * g));
      if constexpr (j == 0) sx[i % 2] = XB == 8 ? rx[i] : (int)((unsigned)rx[i] >> (8 * g));
      mx_mfma16_into<XB, i == 0 || j == 0>(acc[i][j], fw[j], fx[i], sw[j], sx[i % 2]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // the first half of the k-tile in stage `cur`, its w and first x in registers; copies to `to` go on
  auto first = [&](lds_u8_t* cur, lds_u8_t* to, auto copies) __attribute__((always_inline)) {
    each<HALF>([&](auto number) __attribute__((always_inline)) {
      constexpr int k = decltype(number)::value, q = k + HALF;
      step(number);
      each<LATER>([&](auto n) __attribute__((always_inline)) {
        constexpr int b = decltype(n)::value;
        if constexpr (b * (HALF * 3 / 4) / LATER == k) read_x(cur, 2 + b);
      });
      if constexpr (FM == 8 && k == 1) read_sx(cur, 1);
      if constexpr (decltype(copies)::value && q % SPACE == 0 && q / SPACE < TL::COPIES) copy(to, q / SPACE);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // the second half, and the first reads of the next k-tile, in `nxt`
  auto second = [&](lds_u8_t* cur, lds_u8_t* nxt) __attribute__((always_inline)) {
    each<HALF>([&](auto number) __attribute__((always_inline)) {
      constexpr int q = decltype(number)::value, k = q + HALF;
      step(std::integral_constant<int, k>());
      if constexpr (q < 2) read_x(nxt, q);
      if constexpr (q == HALF - (EXACT ? 3 : 6)) read_sx(nxt, 0);   // the last blocks' are taken

      if constexpr (q == HALF - 4) read_sw(nxt);
      if constexpr (EXACT && k >= MM - FN / 2) {
        read_w(nxt, k % (FN / 2) * 2);
        read_w(nxt, k % (FN / 2) * 2 + 1);
      }
      if constexpr (!EXACT && k >= MM - 2 * FN && k % 2 == 1) read_w(nxt, k % (2 * FN) / 2);
      if constexpr (q % SPACE == 0 && q / SPACE < TL::COPIES) copy(cur, q / SPACE);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Results of a job, and zeros in their place: 16 bytes per lane (8 where bf16 is added to) and
  // whole lines, of 8 rows at a time.
  auto store = [&](const Mx4Job& j) __attribute__((always_inline)) {
    const int at_m = j.m0 + wm * TL::WTM + (l16 & 7), at_n = j.n0 + wn * TL::WTN;
    auto put = [&](auto type, auto adds, auto past) __attribute__((always_inline)) {
      constexpr int OD = decltype(type)::value;
      constexpr bool ADD = decltype(adds)::value, PAIRS = OD == DT_BF16 && !ADD, NT = decltype(past)::value;
      constexpr int E = PAIRS ? 8 : 4, W = PAIRS ? 4 : 2;   // outputs per lane; blocks that are side by side
      unsigned char* const base = a.splits > 1 ? elem_ptr<OD>(a.partial, j.split * mx4_partial(a.rows, a.outs)) : reinterpret_cast<unsigned char*>(a.y);
      // what is added to, 16 rows ahead in place of those that are done: loaded where it is needed,
      // each is a memory's latency (24576 x (2048 x 8192) of 4 bits onto fp32 314 us, so 283)
      Raw4<OD> old[ADD ? FN : 1];
      auto load = [&](int i, int b) __attribute__((always_inline)) {
        if constexpr (ADD) {
          const int n = at_n + b * 16 + (l16 >> 3) * 16 + g * 4;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t m = (int64_t)at_m + i * 16 + h * 8;
            Raw4<OD>& r = old[b + h];
            r = quad_zero<OD>();
            if (m >= a.rows || n >= a.outs) continue;
            const unsigned char* const row = base + m * a.outs * elem_bytes<OD>();
            if (n + 4 <= a.outs) {
              r.u = *reinterpret_cast<const typename Quad<OD>::T*>(row + (int64_t)n * elem_bytes<OD>());
            } else {
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                if (n + e >= a.outs) continue;
                if constexpr (OD == DT_BF16) r.u[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[n + e] << (16 * (e % 2));
                else r.u[e] = reinterpret_cast<const uint32_t*>(row)[n + e];
              }
            }
          }
        }
      };
#pragma unroll
      for (int b = 0; ADD && b < FN; b += 2) load(0, b);
      each<FM>([&](auto number) __attribute__((always_inline)) {
        constexpr int i = decltype(number)::value;
#pragma unroll
        for (int b = 0; b < FN; b += 4) settled(acc[i][b], acc[i][b + 1], acc[i][b + 2], acc[i][b + 3]);
#pragma unroll
        for (int b = 0; b < FN; b += W) {
          u32x4_t part[2];
          if constexpr (PAIRS) {
            part[0] = pack_pair(acc[i][b], acc[i][b + 1]);
            part[1] = pack_pair(acc[i][b + 2], acc[i][b + 3]);
          } else {
            part[0] = __builtin_bit_cast(u32x4_t, acc[i][b]);
            part[1] = __builtin_bit_cast(u32x4_t, acc[i][b + 1]);
          }
          rows_side_by_side(part[0], part[1]);
          const int n = at_n + b * 16 + (l16 >> 3) * (W * 8) + g * E;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t m = (int64_t)at_m + i * 16 + h * 8;
            if (m >= a.rows || n >= a.outs) continue;
            unsigned char* const row = base + m * a.outs * elem_bytes<OD>();
            if constexpr (PAIRS) {
              if (n + 8 <= a.outs) {
                typedef U16<DT_BF16>::T V;
                V* const to = reinterpret_cast<V*>(row + (int64_t)n * 2);
                if constexpr (NT) __builtin_nontemporal_store((V)part[h], to);
                else *to = part[h];
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (n + e < a.outs) reinterpret_cast<uint16_t*>(row)[n + e] = (uint16_t)(part[h][e / 2] >> (16 * (e % 2)));
              }
            } else {
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(part[h][e]);
              if constexpr (ADD) {
                float o[4];
                quad_f32<OD>(old[b + h], 0, 4, o);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __fadd_rn(o[e], v[e]);
              }
              quad_store_row<OD, NT>(row, n, a.outs, v);
            }
          }
          if constexpr (ADD && i + 1 < FM) load(i + 1, b);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    typedef std::integral_constant<int, DT_F32> F;
    typedef std::integral_constant<int, YD> Y;
    typedef std::integral_constant<bool, true> Yes;
    typedef std::integral_constant<bool, false> No;
    if constexpr (ADDS) {
      put(Y(), Yes(), No());
    } else {
      if (a.splits > 1) put(F(), No(), No());
      else if (a.stream) put(Y(), No(), Yes());
      else put(Y(), No(), No());
    }
    clear();
  };

  copies_of(job_at(job));
#pragma unroll
  for (int v = 0; v < S; ++v) {
#pragma unroll
    for (int i = 0; i < TL::COPIES; ++i) copy(lds + v * TL::STAGE, i);
    copied();
  }
  wait_vm<(S - 1) * TL::COPIES>();
  block_barrier();
#pragma unroll
  for (int i = 0; i < 2; ++i) read_x(lds, i);
  read_sx(lds, 0);
  read_sw(lds);
#pragma unroll
  for (int j = 0; j < FN; ++j) read_w(lds, j);
  first(lds, lds, std::integral_constant<bool, false>());
  Mx4Job now = job_at(job);
  int more = now.v1 - now.v0;   // k-tiles of the job that are not done
  lds_u8_t* cur = lds;
  // After the stores of a whole tile (STORES of them at least, behind the copies that are waited for)
  // the first turns do not wait for them; the counter does not go beyond 63.
  constexpr int KEEP = (S - 2) * TL::COPIES, STORES = YD == DT_BF16 ? MM / 2 : MM, RELAXED = KEEP + STORES < 63 ? KEEP + STORES : 63;
  int relaxed = 0;
  for (;;) {
    // the next k-tile has landed: what was sent for after it may still be under way
    if (relaxed > 0) wait_vm<RELAXED>();
    else wait_vm<KEEP>();
    --relaxed;
    block_barrier();
    lds_u8_t *const to = cur, *const nxt = cur == lds + (S - 1) * TL::STAGE ? lds : cur + TL::STAGE;
    second(cur, nxt);
    if (--more == 0) {
      store(now);
      relaxed = now.m0 + TL::BM <= a.rows && now.n0 + TL::BN <= a.outs ? S - 2 : 0;
      job += stride;
      if (job >= end_job) break;
      now = job_at(job);
      more = now.v1 - now.v0;
    }
    first(nxt, to, std::integral_constant<bool, true>());
    copied();
    cur = nxt;
  }
  wait_vm<0>();   // no copy into LDS outlives the block
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

// Few rows: blocks of 16, 32 or 64 rows, and waves per block: 8 of them, fewer where blocks * waves would be
// beyond 32 per CU or a wave would have less than 2 k-tiles. (All of 4 bits: 1 x (4096 x 4096) 4.5 us with 8 waves,
// 4.8 with 16; 1 x (4096 x 16384) 8.8 and 9.6; 1 x (16384 x 4096) 8.7 with 8 and 9.0 with 4.)
static int mx4_rows_mb(int64_t rows) { return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4); }
static int64_t mx4_rows_blocks(int64_t rows, int64_t outs) {
  const int64_t m = 16 * mx4_rows_mb(rows);
  return (outs + 15) / 16 * ((rows + m - 1) / m);
}
static int mx4_rows_waves(int64_t rows, int64_t outs, int64_t ins) {
  const int64_t blocks = mx4_rows_blocks(rows, outs), kt = mx4_tiles(ins);
  int waves = 1;
  while (waves < 8 && blocks * waves < 8192 && kt >= 4 * waves) waves *= 2;
  return waves;
}

// The form, and the splits of the k-tiles, by the time they should take (us), fitted to what 78 sizes took in
// every form and with up to 11 splits, 4 bits and 8 (profiles/mx4_forms.md; the choice for 8 bits is 2 % off the
// best on average, 22 % at most). Few rows' blocks each read their rows of both operands, at 7 TB/s from the
// caches, and 35 GB/s a block. Tiles have a fixed part, what the jobs take that share a CU (two small ones at a
// time, a big one) and the partial results' way to memory and back.
//   k-tile of 128 x 128, 4 bits 0.47 alone, 0.79 for a pair; 8 bits 1.1, 1.8
//   k-tile of 256 x 256, 4 bits 0.93; 8 bits 2.8
Mx4Plan mx4_plan(int64_t rows, int64_t outs, int64_t ins, int x_bits) {
  const bool x8 = x_bits == 8;
  const int64_t kt = mx4_tiles(ins), blocks = mx4_rows_blocks(rows, outs);
  const int waves = mx4_rows_waves(rows, outs, ins);
  const double mb = (double)rows * (double)outs * 4e-6;   // of one fp32 result
  Mx4Plan best{0, 1};
  const int64_t in_block = rows < 16 * mx4_rows_mb(rows) ? rows : 16 * mx4_rows_mb(rows);
  const double block = (double)kt * (1024 + (double)in_block * (x8 ? 128 : 64));   // bytes
  double best_us = 2.7 + 0.12 * waves + (double)blocks / 730 + std::max((double)blocks * block / 7e6, (double)((blocks + 255) / 256) * block / 35e3);
  if (blocks > ((int64_t)1 << 31) / (64 * waves)) best_us = 1e30;   // beyond a launch's threads
  for (int edge = 128; edge <= 256; edge *= 2) {
    const int64_t tiles = ((rows + edge - 1) / edge) * ((outs + edge - 1) / edge);
    for (int64_t s = 1; s <= 64 && s <= kt; ++s) {
      const int64_t jobs = tiles * s, rounds = (jobs + 255) / 256, share = (kt + s - 1) / s;
      const double full = jobs < 256 ? (double)jobs / 256 : 1.0;
      double us;
      if (edge == 128) us = 3.5 + (double)(rounds / 2) * ((double)share * (x8 ? 1.8 : 0.79) + 2.2) + (double)(rounds % 2) * ((double)share * (x8 ? 1.1 : 0.47) + 1.5);
      else us = 7.0 + (double)rounds * ((double)share * (x8 ? 2.8 : 0.93) + 5.0 * full);
      if (s > 1) us += 4.0 + (double)s * mb * (1 / 6.0 + 1 / 9.0);
      if (us < best_us * 0.999) { best_us = us; best = {edge, (int)s}; }
    }
  }
  return best;
}

template <int XB, int YD, int MB>
static hipError_t mx4_rows(const Mx4MatmulArgs& a, int waves, hipStream_t s) {
  hipLaunchKernelGGL((k_mx4_rows<XB, YD, MB>), dim3((unsigned)mx4_rows_blocks(a.rows, a.outs)), dim3(64 * waves), (size_t)waves * MB * 1024, s, a);
  return hipGetLastError();
}

template <typename TL, int YD>
static hipError_t mx4_tile(const Mx4MatmulArgs& a, hipStream_t s) {
  const int64_t jobs = ((a.rows + TL::BM - 1) / TL::BM) * ((a.outs + TL::BN - 1) / TL::BN) * a.splits;
  const int64_t want = (jobs + 7) / 8 * 8, most = 256 * TL::BLOCKS;   // resident blocks
  const dim3 grid((unsigned)(want < most ? want : most));
  if (a.accumulate && a.splits == 1) hipLaunchKernelGGL((k_mx4_tile<TL, YD, true>), grid, dim3(TL::NT), 0, s, a);
  else hipLaunchKernelGGL((k_mx4_tile<TL, YD, false>), grid, dim3(TL::NT), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  hipLaunchKernelGGL((k_mx4_join<YD>), dim3((unsigned)((a.rows * a.outs + 1023) / 1024)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int XB, int YD>
static hipError_t mx4_product(const Mx4MatmulArgs& a, hipStream_t s) {
  if (a.edge == 256) return mx4_tile<Mx4Tile<XB, 2, 4, 8, 4, XB == 8 ? 3 : 4>, YD>(a, s);
  if (a.edge == 128) return mx4_tile<Mx4Tile<XB, 2, 2, 4, 4, XB == 8 ? 3 : 4>, YD>(a, s);
  const int waves = mx4_rows_waves(a.rows, a.outs, a.ins), mb = mx4_rows_mb(a.rows);
  return mb == 1 ? mx4_rows<XB, YD, 1>(a, waves, s) : (mb == 2 ? mx4_rows<XB, YD, 2>(a, waves, s) : mx4_rows<XB, YD, 4>(a, waves, s));
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int x_bits, int y_dt, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (x_bits == 8) return y_dt == DT_F32 ? mx4_product<8, DT_F32>(a, s) : mx4_product<8, DT_BF16>(a, s);
  return y_dt == DT_F32 ? mx4_product<4, DT_F32>(a, s) : mx4_product<4, DT_BF16>(a, s);
}

}  // namespace ma
