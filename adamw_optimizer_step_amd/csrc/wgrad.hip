// Weight gradient of a linear layer out of its input's 8-bit checkpoint:
//   grad[n,k] (+)= sum over tokens t of dy[t,n] * x[t,k],  x[t,k] = q[t,k] * 2^e
// on bf16 MFMA with fp32 accumulators. x is exact in bf16 (rows.hpp), so the
// products are too. fp32 dy is taken as three bf16 terms, dy = hi + mid + lo
// exactly from 2^-110 up, and to 2^-133, bf16's least number, below (8 significant
// bits each, cut off, not rounded, so that no term overflows), whose products are
// summed in the same accumulators.
//
// Bound by the matrix instructions where tokens and outputs are many: 12288 x
// (16384 x 4096) bf16 in 1.23 to 1.34 ms (medians of several runs and cards), 1.23 to
// 1.34 PFLOP/s at the 1.75 GHz that the card holds under this load, the matrix units
// busy 71 % of it. A plain library product of the unpacked operands in this layout
// reaches 1.24 PFLOP/s, of contiguous ones 1.43. fp32 dy, three products: 8192 x (2048 x 2048) 166 us + 14
// for the join (1.2 PFLOP/s of bf16 products).
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

namespace wg {

// Block tile of WGM x WGN waves, each FM x FN accumulator blocks of 32 x 32; a
// k-tile is 64 tokens of bf16 dy or 32 of fp32 dy's PL = 3 terms.
template <int DYD, int WGM_, int WGN_, int FM_, int FN_>
struct Tile {
  static constexpr int PL = DYD == DT_F32 ? 3 : 1, BK = DYD == DT_F32 ? 32 : 64;
  static constexpr int WGM = WGM_, WGN = WGN_, FM = FM_, FN = FN_;
  static constexpr int WTM = FM * 32, WTN = FN * 32, BM = WGM * WTM, BN = WGN * WTN, NT = WGM * WGN * 64;
  static constexpr int P_ROW = BM * 2, Q_ROW = BN * 2, P_PLANE = BK * P_ROW, P_BYTES = PL * P_PLANE, STAGE = P_BYTES + BK * Q_ROW;
  // loads per thread and k-tile: 8 values of dy, 16 of the checkpoint
  static constexpr int PC = BM / 8, NP = BK * PC / NT, P_STEP = NT / PC;
  static constexpr int QC = BN / 16, NQ = BK * QC / NT, Q_STEP = NT / QC;
  static constexpr int KS = BK / 16 * PL;   // MFMA steps per k-tile; even, so that the fragment sets alternate over tiles
  static constexpr int LDE = WTN + 4;       // epilogue staging pitch (floats)
  static_assert(P_STEP % 4 == 0 && Q_STEP % 4 == 0 && NQ >= 1 && KS % 2 == 0 && WGM * WGN * 32 * LDE * 4 <= 2 * STAGE, "tile");
};
// The big tile reads each operand from LDS half as often per product: 64 tokens
// of 128 x 128 outputs take it 0.30 to 0.40 us, the small one 0.54 to 0.66; the
// small one spreads few outputs over more CUs (wgrad_plan).
template <int DYD> using Big = Tile<DYD, 2, 4, 4, 2>;     // 256 x 256, 8 waves of 128 x 64
template <int DYD> using Small = Tile<DYD, 2, 2, 2, 2>;   // 128 x 128, 4 waves of 64 x 64

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
typedef __attribute__((address_space(3))) unsigned char lds_u8_t;

// A fragment of 32 rows (n or k) x 16 tokens: two transposing reads of 4
// tokens each. A group of 16 lanes reads 4 tokens x 16 values, lane 4a + b the
// values 4b .. 4b+3 of token a, and receives 4 tokens of its own value; lane
// (l32, lh) so holds tokens 8 lh .. 8 lh + 7 of value l32.
__device__ __forceinline__ u32x4_t frag(lds_u8_t* p, int row4) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + row4));
  typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
  const u32x2_t x = __builtin_bit_cast(u32x2_t, a), y = __builtin_bit_cast(u32x2_t, b);
  return u32x4_t{x.x, x.y, y.x, y.y};
}

// The three terms of 8 fp32 values: the leading 8 significant bits, the next 8,
// the last 8, cut off each time. Infinities and NaN are all in the first term.
__device__ __forceinline__ void split_terms(const Raw8<DT_F32>& r, u32x4_t (&out)[3]) {
  auto upper = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302); };   // the upper halves, packed
  uint32_t most = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t t[3][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b = r.u[(2 * w + i) / 4][(2 * w + i) % 4], mag = b & 0x7FFFFFFFu;
      most = most > mag ? most : mag;
      const float rest = __uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u);
      t[0][i] = b;
      t[1][i] = __float_as_uint(rest);
      t[2][i] = __float_as_uint(rest - __uint_as_float(t[1][i] & 0xFFFF0000u));
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) out[p][w] = upper(t[p][0], t[p][1]);
  }
  if (__builtin_expect(most >= 0x7F800000u, 0)) {
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t b = r.u[(2 * w + i) / 4][(2 * w + i) % 4], mag = b & 0x7FFFFFFFu;
        if (mag < 0x7F800000u) continue;
        const uint32_t keep = i ? 0x0000FFFFu : 0xFFFF0000u;
        if (mag > 0x7F800000u) out[0][w] |= i ? 0x00400000u : 0x40u;   // a NaN stays one
        out[1][w] &= keep;
        out[2][w] &= keep;
      }
  }
}

}  // namespace wg

// One block per output tile and split of the tokens.
//
// LDS holds two k-tiles of both operands as bf16, rows of tokens: dy as it is
// in memory (or its three terms), x converted on the way (the scale of a row's
// 16 values is one byte). A thread's loads of k-tile v + 2 are issued while v is
// multiplied and written to LDS while v + 1 is, so they have one k-tile's time
// to arrive, and one barrier per k-tile is enough. 16-byte chunks are placed so
// that the transposing reads (4 rows x 32 bytes per 16 lanes) and the writes
// touch different banks: dy's chunk c of row r at c ^ 4 (r % 4); x's even chunks
// in the row's first half, odd ones in the second (a lane writes two neighbours,
// one after the other), index ^ 4 (r % 4) ^ 2 (c % 2).
template <int DYD, int GD, typename TL>
__global__ void __launch_bounds__(TL::NT, 2) k_wgrad(const WgradArgs a) {
  using namespace wg;
  constexpr int PL = TL::PL, BK = TL::BK, KS = TL::KS;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * TL::STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;

  // job: split-major, then bands of 4 tile rows walked column by column; XCD
  // b % 8 takes a contiguous eighth, so that its 32 CUs work on 4 x 8 tiles
  // that share 4 panels of dy and 8 of x in its L2
  const int tm = (a.outs + TL::BM - 1) / TL::BM, tn = (a.ins + TL::BN - 1) / TL::BN, tiles = tm * tn;
  const int jobs = tiles * a.splits, per = (jobs + 7) / 8;
  const int job = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (job >= jobs) return;
  const int split = job / tiles, t = job - split * tiles;
  const int band = t / (4 * tn), rem = tm - band * 4, bh = rem < 4 ? rem : 4, idx = t - band * 4 * tn;
  const int n0 = (band * 4 + idx % bh) * TL::BM, k0 = idx / bh * TL::BN;

  const int64_t pitch = act_pitch(a.ins), kb = pitch / kActBlock;
  const int vtiles = (int)((a.tokens + BK - 1) / BK);
  const int v0 = (int)((int64_t)vtiles * split / a.splits), v1 = (int)((int64_t)vtiles * (split + 1) / a.splits);

  // this thread's share of a k-tile
  const int pc = tid % TL::PC, pr = tid / TL::PC, qc = tid % TL::QC, qr = tid / TL::QC;
  // columns beyond the matrix are read from inside it; their outputs are not stored
  const int pcol = n0 + pc * 8 < a.outs ? n0 + pc * 8 : 0;
  const int qcol = k0 + qc * 16 < pitch ? k0 + qc * 16 : 0;
  const int pw = pr * TL::P_ROW + ((pc ^ (4 * (pr % 4))) << 4);
  const int qs = 4 * (qr % 4);
  const int qw0 = TL::P_BYTES + qr * TL::Q_ROW + ((qc ^ qs) << 4);
  const int qw1 = TL::P_BYTES + qr * TL::Q_ROW + (((qc + TL::QC) ^ qs ^ 2) << 4);

  // a k-tile's rows from a scalar address, the lane's place in them as a 32-bit offset
  const uint32_t poff = (uint32_t)pr * (uint32_t)(a.outs * elem_bytes<DYD>()) + (uint32_t)(pcol * elem_bytes<DYD>());
  const uint32_t qoff = (uint32_t)qr * (uint32_t)pitch + (uint32_t)qcol;
  const uint32_t soff = (uint32_t)qr * (uint32_t)kb + (uint32_t)(qcol / kActBlock);
  const int64_t prow = (int64_t)a.outs * elem_bytes<DYD>();

  Raw8<DYD> p[TL::NP];
  u32x4_t q[TL::NQ];
  uint32_t sc[TL::NQ];
  // A k-tile is whole if its rows are there and, where a row's last chunk of dy
  // is partial, 8 more rows, into which that chunk is read on.
  const int64_t slack = a.outs & 7 ? 8 : 0;
  const int whole_tiles = a.tokens > slack ? (int)((a.tokens - slack) / BK) : 0;
  auto load_p = [&](int v, auto fast) __attribute__((always_inline)) {
    const int64_t t0 = (int64_t)v * BK;
    const unsigned char* base = reinterpret_cast<const unsigned char*>(a.dy) + t0 * prow;
    if (decltype(fast)::value || v < whole_tiles) {
#pragma unroll
      for (int j = 0; j < TL::NP; ++j) p[j] = raw_load<DYD>(base + j * TL::P_STEP * prow + poff);
    } else if constexpr (PL == 1) {
#pragma unroll
      for (int j = 0; j < TL::NP; ++j) {
        const int64_t r = t0 + pr + j * TL::P_STEP;
        p[j] = r < a.tokens ? raw_load_row<DYD>(elem_ptr<DYD>(a.dy, r * a.outs), pcol, a.outs) : raw_zero<DYD>();
      }
#pragma unroll
      for (int j = 0; j < TL::NP; ++j) raw_fix<DYD>(p[j], pcol, a.outs);
    }
  };
  auto load_q = [&](int v, auto fast) __attribute__((always_inline)) {
    const int64_t t0 = (int64_t)v * BK;
    const uint8_t *base = a.q + t0 * pitch, *sbase = a.qscale + t0 * kb;
    if (decltype(fast)::value || t0 + BK <= a.tokens) {
#pragma unroll
      for (int j = 0; j < TL::NQ; ++j) {
        q[j] = *reinterpret_cast<const u32x4_t*>(base + j * TL::Q_STEP * pitch + qoff);
        sc[j] = (sbase + j * TL::Q_STEP * kb)[soff];
      }
    } else {
#pragma unroll
      for (int j = 0; j < TL::NQ; ++j) {
        const int64_t r = t0 + qr + j * TL::Q_STEP;
        q[j] = u32x4_t{0u, 0u, 0u, 0u};
        sc[j] = 127;
        if (r < a.tokens) {
          q[j] = *reinterpret_cast<const u32x4_t*>(a.q + r * pitch + qcol);
          sc[j] = a.qscale[r * kb + qcol / kActBlock];
        }
      }
    }
  };
  auto put_p = [&](lds_u8_t* st, const Raw8<DYD>& x) __attribute__((always_inline)) {
    u32x4_t w[PL];
    if constexpr (PL == 1) w[0] = x.u[0];
    else split_terms(x, w);
#pragma unroll
    for (int i = 0; i < PL; ++i) *(lds_u32x4_t*)(st + i * TL::P_PLANE) = w[i];
  };
  auto stage_p = [&](int v, lds_u8_t* st, auto fast) __attribute__((always_inline)) {
    if (PL == 1 || decltype(fast)::value || v < whole_tiles) {
#pragma unroll
      for (int j = 0; j < TL::NP; ++j) put_p(st + pw + j * TL::P_STEP * TL::P_ROW, p[j]);
    } else {
      // the last k-tile of fp32 dy is read here, row by row (there are no registers for more)
#pragma unroll 1
      for (int j = 0; j < TL::NP; ++j) {
        const int64_t r = (int64_t)v * BK + pr + j * TL::P_STEP;
        Raw8<DYD> x = r < a.tokens ? raw_load_row<DYD>(elem_ptr<DYD>(a.dy, r * a.outs), pcol, a.outs) : raw_zero<DYD>();
        raw_fix<DYD>(x, pcol, a.outs);
        put_p(st + pw + j * TL::P_STEP * TL::P_ROW, x);
      }
    }
  };
  auto stage_q = [&](lds_u8_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TL::NQ; ++j) {
      const float s = act_scale(sc[j]);
      u32x4_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint2 b = act_decode_bf16(q[j][2 * h + i], s);
          w[h][2 * i] = b.x;
          w[h][2 * i + 1] = b.y;
        }
      *(lds_u32x4_t*)(st + qw0 + j * TL::Q_STEP * TL::Q_ROW) = w[0];
      *(lds_u32x4_t*)(st + qw1 + j * TL::Q_STEP * TL::Q_ROW) = w[1];
    }
  };

  f32x16_t acc[TL::FM][TL::FN];
#pragma unroll
  for (int i = 0; i < TL::FM; ++i)
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // fragment addresses (step and second half are immediate offsets)
  const int g = lane >> 4, a4 = (lane >> 2) & 3, b4 = lane & 3;
  int po[TL::FM], qo[TL::FN];
#pragma unroll
  for (int i = 0; i < TL::FM; ++i) {
    const int c = (wm * TL::WTM + i * 32) / 8 + 2 * (g & 1) + (b4 >> 1);
    po[i] = (8 * (g >> 1) + a4) * TL::P_ROW + ((c ^ (4 * a4)) << 4) + (b4 & 1) * 8;
  }
#pragma unroll
  for (int j = 0; j < TL::FN; ++j) {
    const int c = (wn * TL::WTN + j * 32) / 8 + 2 * (g & 1) + (b4 >> 1);
    qo[j] = TL::P_BYTES + (8 * (g >> 1) + a4) * TL::Q_ROW + ((((c >> 1) + TL::QC * (c & 1)) ^ (4 * a4) ^ (2 * (c & 1))) << 4) + (b4 & 1) * 8;
  }
  lds_u8_t* const lds = (lds_u8_t*)smem;
  u32x4_t fp[2][TL::FM], fq[2][TL::FN];
  // step ks: 16 tokens ks / PL of term ks % PL; the terms share x's fragments
  auto read = [&](lds_u8_t* st, int ks) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) fp[ks & 1][i] = frag(st + po[i] + (ks % PL) * TL::P_PLANE + ks / PL * 16 * TL::P_ROW, 4 * TL::P_ROW);
    if (ks % PL == 0) {
#pragma unroll
      for (int j = 0; j < TL::FN; ++j) fq[ks / PL & 1][j] = frag(st + qo[j] + ks / PL * 16 * TL::Q_ROW, 4 * TL::Q_ROW);
    }
  };
  // x first: each lane's accumulators are 4 consecutive k of one row n
  auto multiply = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
      for (int j = 0; j < TL::FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fq[ks / PL & 1][j]),
                                                            __builtin_bit_cast(bf16x8_t, fp[ks & 1][i]), acc[i][j], 0, 0, 0);
  };
  // every wave's LDS accesses so far are done before any wave goes on; loads from memory stay in flight
  auto barrier = [&]() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  typedef std::integral_constant<bool, true> Fast;
  typedef std::integral_constant<bool, false> Any;
  if (v0 < v1) {
    load_p(v0, Any());
    load_q(v0, Any());
    stage_p(v0, lds, Any());
    stage_q(lds);
    if (v0 + 1 < v1) {
      load_p(v0 + 1, Any());
      load_q(v0 + 1, Any());
    }
    barrier();
    read(lds, 0);
  }
  // k-tile v: the staging of v + 1 and the loads of v + 2 go between its MFMAs.
  // FAST: both exist and are whole, so that all of it is one block of
  // instructions without branches, interleaved as the groups say (12288 x (16384 x
  // 4096) bf16: 1600 us -> 1350 by that).
  auto tile = [&](int v, auto fast) __attribute__((always_inline)) {
    constexpr bool F = decltype(fast)::value;
    lds_u8_t* const cur = lds + ((v - v0) & 1) * TL::STAGE;
    lds_u8_t* const nxt = lds + ((v - v0 + 1) & 1) * TL::STAGE;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) {
        read(cur, ks + 1);
      } else if (F || v + 1 < v1) {
        barrier();
        read(nxt, 0);
      }
      // (not FAST: after the MFMAs, whose fragments then leave their registers)
      if constexpr (!F) {
        multiply(ks);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (ks == KS / 2 - 1) {
        if (F || v + 1 < v1) stage_p(v + 1, nxt, fast);
        if (F || v + 2 < v1) load_p(v + 2, fast);
      }
      if (ks == KS - 2) {
        if (F || v + 1 < v1) stage_q(nxt);
        if (F || v + 2 < v1) load_q(v + 2, fast);
      }
      if constexpr (F) {
        multiply(ks);
        // per MFMA up to 3 LDS reads, 3 conversions, a write and a load
#pragma unroll
        for (int i = 0; i < TL::FM * TL::FN; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int fast_end = (v1 < whole_tiles ? v1 : whole_tiles) - 2;
  int v = v0;
  for (; v < fast_end; ++v) tile(v, Fast());
  for (; v < v1; ++v) tile(v, Any());

  // 32 rows of the wave's block at a time through its own part of LDS, so that
  // stores are 8 consecutive values per lane and whole rows per 8 lanes
  barrier();
  float* const mine = reinterpret_cast<float*>(smem) + wave * 32 * TL::LDE;
  const int l32 = lane & 31, lh = lane >> 5;
  const bool whole = a.splits == 1;
#pragma unroll
  for (int i = 0; i < TL::FM; ++i) {
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<float4*>(mine + l32 * TL::LDE + j * 32 + b * 8 + lh * 4) =
            make_float4(acc[i][j][4 * b], acc[i][j][4 * b + 1], acc[i][j][4 * b + 2], acc[i][j][4 * b + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < 32 * TL::WTN / 512; ++u) {
      constexpr int LPR = TL::WTN / 8;
      const int row = u * (64 / LPR) + lane / LPR, c = lane % LPR * 8;
      const float4 x = *reinterpret_cast<const float4*>(mine + row * TL::LDE + c), y = *reinterpret_cast<const float4*>(mine + row * TL::LDE + c + 4);
      float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const int n = n0 + wm * TL::WTM + i * 32 + row, k = k0 + wn * TL::WTN + c;
      if (n >= a.outs || k >= a.ins) continue;
      if (!whole) {
        store_row<DT_F32>(elem_ptr<DT_F32>(a.partial, split * wgrad_partial(a.outs, a.ins) + (int64_t)n * a.ins), k, a.ins, v);
        continue;
      }
      unsigned char* out = elem_ptr<GD>(a.grad, (int64_t)n * a.ins);
      if (a.accumulate) {
        float old[8];
        raw_f32_row<GD>(raw_load_row<GD>(out, k, a.ins), k, a.ins, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(old[e], v[e]);
      }
      store_row<GD>(out, k, a.ins, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The splits' partial products, added in order: 4 consecutive values per thread
// (few outputs have many splits, and want many threads), 8 splits in flight.
template <int GD>
__global__ void __launch_bounds__(256) k_wgrad_join(const WgradArgs a) {
  const int64_t total = (int64_t)a.outs * a.ins, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  float v[4] = {};
  const int n = total - i < 4 ? (int)(total - i) : 4;
  const int64_t stride = wgrad_partial(a.outs, a.ins);   // past the end there is room, not read further
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
    if (a.accumulate) v[e] = __fadd_rn(load1<GD>(a.grad, i + e), v[e]);
    store1<GD>(a.grad, i + e, v[e]);
  }
}

// Tile and number of splits by the time they should take (us), from what single
// launches of 64 .. 4096 tokens took: a fixed part, the k-tiles of the blocks
// that share a CU (one or two small tiles, one big one, slower as more CUs draw
// on memory and power), the outputs or partial products written, and the join.
//   k-tile of 64 tokens, bf16 dy: 128 x 128 0.66 alone, 1.08 for a pair; 256 x 256 1.2 (64 blocks) to 1.6 (256)
//   k-tile of 32 tokens, fp32 dy: 0.92, 1.5; 1.75 to 2.3
WgradPlan wgrad_plan(int64_t tokens, int64_t outs, int64_t ins, int dy_dt) {
  const bool f32 = dy_dt == DT_F32;
  const int64_t bk = f32 ? 32 : 64, vt = (tokens + bk - 1) / bk;
  const double mb = (double)outs * (double)ins * 4e-6;   // of one fp32 result
  WgradPlan best{false, 1};
  double best_us = 1e30;
  for (int big = 0; big < 2; ++big) {
    const int64_t edge = big ? 256 : 128, tiles = ((outs + edge - 1) / edge) * ((ins + edge - 1) / edge);
    for (int64_t s = 1; s <= 64 && s <= (vt > 1 ? vt : 1); ++s) {
      const int64_t jobs = tiles * s, rounds = (jobs + 255) / 256;   // blocks per CU
      const double full = jobs < 256 ? (double)jobs / 256 : 1.0;
      const double small_us = (double)(rounds / 2) * (f32 ? 1.5 : 1.08) + (double)(rounds % 2) * (f32 ? 0.92 : 0.66);
      const double big_us = (double)rounds * (f32 ? 1.75 + 0.55 * full : 1.2 + 0.4 * full);
      double us = 5.5 + (double)((vt + s - 1) / s) * (big ? big_us : small_us) + (double)s * mb / 5.5;
      if (s > 1) us += 2.5 + (double)(s + 1) * mb / 6.5;
      if (us < best_us * 0.999) { best_us = us; best = {big != 0, (int)s}; }
    }
  }
  return best;
}

template <int DYD, int GD, typename TL>
static hipError_t wgrad_tile(const WgradArgs& a, hipStream_t s) {
  const int64_t jobs = (int64_t)((a.outs + TL::BM - 1) / TL::BM) * ((a.ins + TL::BN - 1) / TL::BN) * a.splits;
  hipLaunchKernelGGL((k_wgrad<DYD, GD, TL>), dim3((unsigned)((jobs + 7) / 8 * 8)), dim3(TL::NT), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  const int64_t total = (int64_t)a.outs * a.ins;
  hipLaunchKernelGGL((k_wgrad_join<GD>), dim3((unsigned)((total + 1023) / 1024)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DYD, int GD>
static hipError_t wgrad(const WgradArgs& a, hipStream_t s) {
  return a.big ? wgrad_tile<DYD, GD, wg::Big<DYD>>(a, s) : wgrad_tile<DYD, GD, wg::Small<DYD>>(a, s);
}

hipError_t launch_wgrad(const WgradArgs& a, int dy_dt, int grad_dt, hipStream_t s) {
  if (dy_dt == DT_F32) return grad_dt == DT_F32 ? wgrad<DT_F32, DT_F32>(a, s) : wgrad<DT_F32, DT_BF16>(a, s);
  return grad_dt == DT_F32 ? wgrad<DT_BF16, DT_F32>(a, s) : wgrad<DT_BF16, DT_BF16>(a, s);
}

}  // namespace ma
