// Embedding lookup with scaling, and its gradient by sorted tokens (gfx950).
//
//   forward   out[i,:]  = RNE(scale * table[t_i,:])
//   backward  grad[v,:] (+)= scale * sum over { i : t_i = v } of dout[i,:]
//
// Few positions are summed in ascending i, more in contiguous parts that are added
// in order: the same tokens give the same bits.
//
// A token outside [0, rows) is ignored: its output row is zero and no gradient
// comes of it (a row of another shard, a masked position).
#include "rows.hpp"
#include "train_ops.hpp"

namespace ma {

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t i) {
  return wide ? reinterpret_cast<const int64_t*>(tokens)[i] : (int64_t) reinterpret_cast<const int32_t*>(tokens)[i];
}

// ---------------------------------------------------------------------------
// forward: LPR lanes per output row, two rows per lane group, whose reads are in
// flight together behind their tokens. Bound by memory: 49152 tokens x 1024 from
// fp32 to bf16, 155 MB moved, take 31 us (25 at a large copy's rate); one row per
// group 30.5 but 10.5 against 9.5 for 256 columns, four 5.9 against 4.4 for 400
// tokens x 2048. Rows of at most 128 or 256 columns take 16 or 32 lanes, not a
// whole wave (128 columns: 5.9 us against 9.5; 256: 9.6 against 10.7).
// ---------------------------------------------------------------------------
constexpr int kLookupRows = 2;
// fp32 results by 4 columns per lane (fp32 to fp32 of the case above 76 -> 48 us, bf16
// to fp32 69 -> 40; fp32 to bf16 31 by 8, 33 by 4)
template <int TD, int OD> constexpr bool lookup_quads() { return OD == DT_F32; }
template <int TD, int OD, int LPR, bool NT>
__global__ void __launch_bounds__(256) k_embed_fwd(const EmbedFwdArgs a) {
  constexpr int R = kLookupRows, GROUPS = 256 / LPR;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int64_t r0 = ((int64_t)blockIdx.x * GROUPS + group) * R;
  int64_t tok[R];
  bool in[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    tok[r] = r0 + r < a.n_tokens ? token_at(a.tokens, a.wide, r0 + r) : -1;
    in[r] = tok[r] >= 0 && tok[r] < a.rows;
  }
  if constexpr (lookup_quads<TD, OD>()) {
    for (int col = lane * 4; col < a.cols; col += LPR * 4) {
      Raw4<TD> x[R];
#pragma unroll
      for (int r = 0; r < R; ++r)
        x[r] = in[r] ? quad_load_row<TD>(elem_ptr<TD>(a.table, tok[r] * a.cols), col, a.cols) : quad_zero<TD>();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r0 + r >= a.n_tokens) break;
        float v[4];
        quad_f32<TD>(x[r], col, a.cols, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = in[r] ? v[e] * a.scale : 0.0f;
        quad_store_row<OD, NT>(elem_ptr<OD>(a.out, (r0 + r) * a.cols), col, a.cols, v);
      }
    }
    return;
  }
  for (int col = lane * 8; col < a.cols; col += LPR * 8) {
    Raw8<TD> x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = raw_zero<TD>();
      if (in[r]) x[r] = raw_load_row<TD>(elem_ptr<TD>(a.table, tok[r] * a.cols), col, a.cols);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r0 + r >= a.n_tokens) break;
      float v[8];
      raw_f32_row<TD>(x[r], col, a.cols, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in[r] ? v[e] * a.scale : 0.0f;
      store_row<OD, NT>(elem_ptr<OD>(a.out, (r0 + r) * a.cols), col, a.cols, v);
    }
  }
}

template <int TD, int OD, bool NT>
static hipError_t embed_fwd(const EmbedFwdArgs& a, hipStream_t s) {
  constexpr int per_lane = lookup_quads<TD, OD>() ? 4 : 8;
  const int chunks = (a.cols + per_lane - 1) / per_lane;
  auto grid = [&](int lpr) { const int64_t per = 256 / lpr * kLookupRows; return dim3((unsigned)((a.n_tokens + per - 1) / per)); };
  if (chunks <= 16) hipLaunchKernelGGL((k_embed_fwd<TD, OD, 16, NT>), grid(16), dim3(256), 0, s, a);
  else if (chunks <= 32) hipLaunchKernelGGL((k_embed_fwd<TD, OD, 32, NT>), grid(32), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_embed_fwd<TD, OD, 64, NT>), grid(64), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int TD, int OD>
static hipError_t embed_fwd(const EmbedFwdArgs& a, hipStream_t s) {
  const bool stream = a.n_tokens * a.cols * (elem_bytes<TD>() + elem_bytes<OD>()) > kStreamBytes;
  return stream ? embed_fwd<TD, OD, true>(a, s) : embed_fwd<TD, OD, false>(a, s);
}

hipError_t launch_embed_fwd(const EmbedFwdArgs& a, int table_dt, int out_dt, hipStream_t s) {
  if (a.n_tokens == 0) return hipSuccess;
  if (table_dt == DT_F32) return out_dt == DT_F32 ? embed_fwd<DT_F32, DT_F32>(a, s) : embed_fwd<DT_F32, DT_BF16>(a, s);
  return out_dt == DT_F32 ? embed_fwd<DT_BF16, DT_F32>(a, s) : embed_fwd<DT_BF16, DT_BF16>(a, s);
}

// ---------------------------------------------------------------------------
// backward, 1: the tokens' positions sorted by slot, stable, in one launch. Row
// v has slot (v mod NB) * M + v / NB with M = ceil(rows / NB): block b of NB (a
// power of two) owns the M slots b M .., the rows b mod NB (interleaved, so that
// frequent rows with neighbouring ids go to different blocks). It reads all
// tokens, each of its 16 waves a contiguous sixteenth: it counts how many valid
// tokens belong to earlier blocks (where its own part of the sorted order
// begins) and keeps its own tokens in LDS, a list per wave. Each wave numbers its
// list's tokens within their rows, 64 at a time; the rows' counts are added up
// over the waves, and every token's position goes to its place. A wave whose
// list overflows (a few rows have most of the tokens) reads its share again.
// No global atomics, and the order is ascending position.
//
// Every block reads every token, from its XCD's L2: what a block does per 64
// tokens (a load, a compare, two ballots) bounds it, not memory. 49152 tokens of
// 50304 rows: 15 us; 5003: 6.6, mostly its chain of waits; all in one row: 81; 2^20
// evenly spread: 146; with Zipf's frequencies, where lists overflow: 1716.
// ---------------------------------------------------------------------------
constexpr int kBinThreads = 1024, kBinWaves = kBinThreads / 64, kBinRows = 512, kBinBits = 9, kBinList = 1024;

// The next numbers of the lanes' rows: a lane with own = true gets next[bin] plus
// the number of lower lanes with the same row, and next[bin] moves on by all of them.
__device__ __forceinline__ uint32_t embed_next(volatile uint32_t* next, bool own, int bin) {
  // the lanes with the same row as this one, by the bits of its index
  uint64_t same = __ballot(own);
#pragma unroll
  for (int i = 0; i < kBinBits; ++i) {
    const uint64_t m = __ballot(bin >> i & 1);
    same &= bin >> i & 1 ? m : ~m;
  }
  const int rank = __builtin_popcountll(same & (((uint64_t)1 << (threadIdx.x & 63)) - 1));
  const uint32_t at = next[bin];
  if (own && rank == 0) next[bin] = at + (uint32_t)__builtin_popcountll(same);
  return at + rank;
}

// The 64 * U tokens from `first` of a share that ends at n, token u * 64 + lane in v[u], as
// 32 bits: 0xFFFFFFFF (no row) for one outside them or past the end.
template <bool WIDE, int U>
__device__ __forceinline__ void tokens32(const void* share, int first, int n, int lane, uint32_t (&v)[U]) {
  if (first + 64 * U <= n) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (WIDE) {
        const uint2 t = reinterpret_cast<const uint2*>(share)[first + u * 64 + lane];
        v[u] = t.y ? 0xFFFFFFFFu : t.x;
      } else {
        v[u] = reinterpret_cast<const uint32_t*>(share)[first + u * 64 + lane];
      }
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + u * 64 + lane;
    v[u] = 0xFFFFFFFFu;
    if (i < n) {
      if constexpr (WIDE) {
        const uint2 t = reinterpret_cast<const uint2*>(share)[i];
        v[u] = t.y ? 0xFFFFFFFFu : t.x;
      } else {
        v[u] = reinterpret_cast<const uint32_t*>(share)[i];
      }
    }
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kBinThreads) k_embed_bin(const EmbedBwdArgs a) {
  __shared__ uint32_t hist[kBinWaves][kBinRows];
  __shared__ uint32_t list[kBinWaves][kBinList];   // (offset in the wave's share) * kBinRows + owned row
  __shared__ uint16_t nth[kBinWaves][kBinList];    // which of its row's tokens in the share it is
  __shared__ uint32_t wsum[kBinWaves], scan[kBinWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t mask = ((uint32_t)1 << a.log2nb) - 1, me = blockIdx.x, rows = (uint32_t)a.rows;
  for (int i = lane; i < kBinRows; i += 64) hist[wave][i] = 0;
  const int seg = (int)round_up((a.n_tokens + kBinWaves - 1) / kBinWaves, 64);   // <= 2^21: an offset and a row fit 32 bits
  const int64_t i0 = (int64_t)wave * seg;
  const int n = (int)(i0 + seg < a.n_tokens ? seg : (i0 < a.n_tokens ? a.n_tokens - i0 : 0));
  const void* share = reinterpret_cast<const unsigned char*>(a.tokens) + i0 * (WIDE ? 8 : 4);
  uint32_t less = 0;
  int kept = 0;
  constexpr int U = 8;
  for (int i = 0; i < n; i += 64 * U) {
    uint32_t v[U];
    tokens32<WIDE, U>(share, i, n, lane, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t b = v[u] < rows ? v[u] & mask : 0xFFFFFFFFu;
      less += (uint32_t)__builtin_popcountll(__ballot(b < me));
      const uint64_t owns = __ballot(b == me);
      if (!owns) continue;
      const int k = kept + __builtin_popcountll(owns & (((uint64_t)1 << lane) - 1));
      if (b == me && k < kBinList) list[wave][k] = (uint32_t)(i + u * 64 + lane) * kBinRows + (v[u] >> a.log2nb);
      kept += __builtin_popcountll(owns);
    }
  }
  // each of them counted at its row: f(lane's token is one, its row, its place in the list or its offset)
  const bool listed = kept <= kBinList;
  auto own_tokens = [&](auto&& f) __attribute__((always_inline)) {
    if (listed) {
      for (int k = 0; k < kept; k += 64) {
        const uint32_t x = k + lane < kept ? list[wave][k + lane] : 0u;
        f(k + lane < kept, (int)(x % kBinRows), (int)(x / kBinRows), k + lane);
      }
    } else {
      constexpr int V = 4;
      for (int i = 0; i < n; i += 64 * V) {
        uint32_t v[V];
        tokens32<WIDE, V>(share, i, n, lane, v);
#pragma unroll
        for (int u = 0; u < V; ++u) f(v[u] < rows && (v[u] & mask) == me, (int)(v[u] >> a.log2nb) & (kBinRows - 1), i + u * 64 + lane, 0);
      }
    }
  };
  own_tokens([&](bool own, int bin, int, int k) {
    const uint32_t at = embed_next(hist[wave], own, bin);
    if (own && listed) nth[wave][k] = (uint16_t)at;
  });
  if (lane == 0) wsum[wave] = less;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < kBinWaves; ++w) base += wsum[w];
  // per row (thread): exclusive counts over the waves, the total, and the totals' scan over the owned rows
  uint32_t total = 0, upto = 0;
  if (tid < kBinRows) {
#pragma unroll
    for (int w = 0; w < kBinWaves; ++w) {
      const uint32_t h = hist[w][tid];
      hist[w][tid] = total;
      total += h;
    }
  }
  upto = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t x = __shfl_up(upto, o, 64);
    upto += lane >= o ? x : 0u;
  }
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBinRows / 64; ++w) upto += w < wave ? scan[w] : 0u;
  const uint32_t at = base + upto - total;
  const int32_t slot0 = (int32_t)me * a.per_block;
  if (tid < a.per_block) {
    a.start[slot0 + tid] = (int32_t)at;
    a.count[slot0 + tid] = (int32_t)total;
  }
  if (tid < kBinRows) {
    if (me == mask && tid == kBinRows - 1) *a.n_valid = (int32_t)(base + upto);
#pragma unroll
    for (int w = 0; w < kBinWaves; ++w) hist[w][tid] += at;
  }
  __syncthreads();
  own_tokens([&](bool own, int bin, int offset, int k) {
    uint32_t to;
    if (listed) to = own ? hist[wave][bin] + nth[wave][k] : 0u;
    else to = embed_next(hist[wave], own, bin);
    if (own) {
      a.order[to] = (int32_t)(i0 + offset);
      a.keys[to] = slot0 + bin;
    }
  });
}

// ---------------------------------------------------------------------------
// backward, 2: the sums, a slice of 512 * CH columns per wave. A wave takes a
// row: it sums its run of the sorted positions (at most a.piece tokens) and
// writes it, zeros for an empty one, or adds it to a row that occurs. (One row
// per wave, not more: most rows are empty or short, and what a wave waits for is
// one chain of count, position, row.) Longer runs are summed by the piece waves (the launch's
// first blocks), one per a.piece sorted positions: the part of a long run
// that its first position belongs to goes to partial row 2p, that of another
// long run that its last position belongs to to 2p + 1 (no third one fits), and
// k_embed_join adds a run's parts in order.
// 49152 tokens x 1024 bf16 into 50304 rows: 55 us (100 MB read, 206 written, 49 at
// the rate of a large copy); 65 with 8 columns per lane, their place checked at each
// load and cached stores; two rows per wave 70, four 79.
// ---------------------------------------------------------------------------
// A lane's columns of a slice: 4 from col + 256 k, k < 2 CH (see quad_load_row). Every
// lane loads 4 columns inside the row, so that the loads are free of branches: the
// row's last, partial group its last 4, moved to their places once the sum is
// whole; lanes past the row's end anything, which is not stored.
template <int DD, int CH>
__device__ __forceinline__ void embed_sum(const EmbedBwdArgs& a, int32_t pos, int from, int to, int col, float (&acc)[2 * CH][4]) {
  constexpr int Q = 2 * CH;
#pragma unroll
  for (int k = 0; k < Q; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = 0.0f;
  if (__builtin_expect(a.cols < 4, 0)) {
#pragma unroll 1
    for (int j = from; j < to; ++j) {
      float v[4];
      quad_f32<DD>(quad_load_row<DD>(elem_ptr<DD>(a.dout, (int64_t)__builtin_amdgcn_readlane(pos, j) * a.cols), 0, a.cols), 0, a.cols, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][e] += v[e];
    }
    return;
  }
  int at[Q];
#pragma unroll
  for (int k = 0; k < Q; ++k) at[k] = (col + k * 256 + 4 <= a.cols ? col + k * 256 : a.cols - 4) * elem_bytes<DD>();
  typedef typename Quad<DD>::T V;
  constexpr int U = (DD == DT_BF16 ? 16 : 8) / CH;   // 64 registers of rows in flight; each row is read once (non-temporal)
  for (int j = from; j < to; j += U) {
    Raw4<DD> x[U][Q];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < to) {
        const unsigned char* row = elem_ptr<DD>(a.dout, (int64_t)__builtin_amdgcn_readlane(pos, j + u) * a.cols);
#pragma unroll
        for (int k = 0; k < Q; ++k) x[u][k].u = __builtin_nontemporal_load(reinterpret_cast<const V*>(row + at[k]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < to) {
#pragma unroll
        for (int k = 0; k < Q; ++k) {
          float v[4];
          quad_f32<DD>(x[u][k], 0, 0, v);   // (as they are)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][e] += v[e];
        }
      }
    }
  }
  if (a.cols & 3) {
#pragma unroll
    for (int k = 0; k < Q; ++k) quad_fix(col + k * 256, a.cols, acc[k]);
  }
}

// A row's sum, scaled, to the gradient, or added to what is there.
template <int CH, bool ACC, bool NT = false>
__device__ __forceinline__ void embed_store(const EmbedBwdArgs& a, int64_t v, int col, float (&acc)[2 * CH][4]) {
  unsigned char* out = reinterpret_cast<unsigned char*>(a.grad + v * a.cols);
#pragma unroll
  for (int k = 0; k < 2 * CH; ++k) {
    const int cc = col + k * 256;
    if (cc >= a.cols) continue;
    float old[4] = {};
    if constexpr (ACC) quad_f32<DT_F32>(quad_load_row<DT_F32>(out, cc, a.cols), cc, a.cols, old);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = ACC ? __fadd_rn(old[e], __fmul_rn(acc[k][e], a.scale)) : acc[k][e] * a.scale;
    quad_store_row<DT_F32, NT>(out, cc, a.cols, acc[k]);
  }
}

template <int DD, int CH, bool ACC, bool NT>
__global__ void __launch_bounds__(256) k_embed_sum(const EmbedBwdArgs a, int piece_blocks) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = blockIdx.y * 512 * CH + lane * 4;
  float acc[2 * CH][4];
  if ((int)blockIdx.x < piece_blocks) {
    const int64_t p = (int64_t)blockIdx.x * 4 + wave;
    const int64_t first = p * a.piece;
    const int64_t left = *a.n_valid - first;
    if (left <= 0) return;
    const int n = left < a.piece ? (int)left : a.piece;
    const int32_t key = lane < n ? a.keys[first + lane] : 0, pos = lane < n ? a.order[first + lane] : 0;
    const int32_t va = __builtin_amdgcn_readlane(key, 0), vb = __builtin_amdgcn_readlane(key, n - 1);
    for (int side = 0; side < 2; ++side) {
      const int32_t v = side ? vb : va;
      if (side && vb == va) break;
      const int64_t s = a.start[v], c = a.count[v];
      if (c <= a.piece) continue;
      const int from = s > first ? (int)(s - first) : 0;
      const int to = s + c - first < n ? (int)(s + c - first) : n;
      embed_sum<DD, CH>(a, pos, from, to, col, acc);
      unsigned char* out = reinterpret_cast<unsigned char*>(a.partial + (2 * p + side) * a.cols);
#pragma unroll
      for (int k = 0; k < 2 * CH; ++k)
        if (col + k * 256 < a.cols) quad_store_row<DT_F32>(out, col + k * 256, a.cols, acc[k]);
    }
    return;
  }
  // the wave's row: waves that run together write neighbouring rows
  const int64_t v = (int64_t)((int)blockIdx.x - piece_blocks) * 4 + wave;
  if (v >= a.rows) return;
  const int32_t slot = (int32_t)(v & (((int64_t)1 << a.log2nb) - 1)) * a.per_block + (int32_t)(v >> a.log2nb);
  const int c = a.count[slot];
  if (c > a.piece || (ACC && c == 0)) return;
  const int64_t s = a.start[slot];
  const int32_t pos = lane < c ? a.order[s + lane] : 0;
  embed_sum<DD, CH>(a, pos, 0, c, col, acc);
  embed_store<CH, ACC, NT>(a, v, col, acc);
}

// The long runs that start in one of the block's kJoinPieces pieces (at most one
// in each): the block's waves sum a run's parts in as many contiguous shares,
// 256 columns per block, and the shares are added in order. 4 to 5 us for the
// lookups behind one another (count, slot, run, parts), 7 for 49152 Zipf tokens.
constexpr int kJoinWaves = 8, kJoinPieces = 4;
__global__ void __launch_bounds__(kJoinWaves * 64) k_embed_join(const EmbedBwdArgs a) {
  __shared__ float4 part[kJoinWaves][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t n_valid = *a.n_valid;
  // lane i: does a long run start in piece i? (the last piece's last run goes on nowhere)
  const int64_t mine = (int64_t)blockIdx.x * kJoinPieces + lane;
  bool starts = false;
  int32_t slot = 0, s = 0, c = 0;
  if (lane < kJoinPieces && n_valid - mine * a.piece > a.piece) {
    slot = a.keys[(mine + 1) * a.piece - 1];
    s = a.start[slot];
    c = a.count[slot];
    starts = c > a.piece && s >= mine * a.piece;
  }
  const int col = blockIdx.y * 256 + lane * 4;
  const bool whole = col + 4 <= a.cols;
  for (uint64_t todo = __ballot(starts); todo; todo &= todo - 1) {
    const int i = __builtin_ctzll(todo);
    const int64_t p = (int64_t)blockIdx.x * kJoinPieces + i;
    const int64_t rs = __builtin_amdgcn_readlane(s, i), rc = __builtin_amdgcn_readlane(c, i);
    const int64_t last = (rs + rc - 1) / a.piece;
    const int64_t n = last - p + 1, share = (n + kJoinWaves - 1) / kJoinWaves;
    const int64_t q0 = p + wave * share, q1 = q0 + share < last + 1 ? q0 + share : last + 1;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    typedef typename U16<DT_F32>::T V;
    if (whole) {
      constexpr int U = 8;   // parts in flight
      for (int64_t q = q0; q < q1; q += U) {
        u32x4_t x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u] = u32x4_t{0u, 0u, 0u, 0u};
          if (q + u < q1) x[u] = *reinterpret_cast<const V*>(a.partial + (2 * (q + u) + (q + u == p && rs > p * a.piece)) * a.cols + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          acc.x += __uint_as_float(x[u][0]); acc.y += __uint_as_float(x[u][1]); acc.z += __uint_as_float(x[u][2]); acc.w += __uint_as_float(x[u][3]);
        }
      }
    } else if (col < a.cols) {
#pragma unroll 8
      for (int64_t q = q0; q < q1; ++q) {
        const float* src = a.partial + (2 * q + (q == p && rs > p * a.piece)) * a.cols;
        // the row's end: columns past it repeat the last one, and are not stored
        acc.x += src[col]; acc.y += src[col + 1 < a.cols ? col + 1 : col]; acc.z += src[col + 2 < a.cols ? col + 2 : col];
      }
    }
    __syncthreads();   // the run before is stored
    part[wave][lane] = acc;
    __syncthreads();
    const int cc = blockIdx.y * 256 + threadIdx.x;
    if (threadIdx.x < 256 && cc < a.cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWaves; ++w) t += reinterpret_cast<const float*>(part[w])[threadIdx.x];
      const int32_t sl = __builtin_amdgcn_readlane(slot, i);
      const int64_t v = ((int64_t)(sl % a.per_block) << a.log2nb) + sl / a.per_block;
      float* g = a.grad + v * a.cols + cc;
      *g = a.accumulate ? __fadd_rn(*g, __fmul_rn(t, a.scale)) : t * a.scale;
    }
  }
}

// ---------------------------------------------------------------------------
// backward of few tokens (at most kEmbedDirect), in one launch and without a
// sort. The first blocks take a token per wave: the wave has all tokens in
// registers, and if its token is the first of its row it finds the others by
// comparison and sums them in ascending position; more than kDirectAlone are
// shared out among the block's waves and joined in order (500 tokens into 1000 x
// 1024, the most frequent 67 times: 16 -> 10.5 us; 500 equal ones: 164 -> 50). When the gradient is
// written whole, the other blocks write zeros to the rows that no token names,
// flagged in LDS, 16 rows a block or up to kDirectRows short ones: few, as a short
// front of writes moves over memory fastest (zeros of 206 MB in order: 6.5 TB/s by
// blocks of 4 KB, 5.5 of 64 KB), but each block reads all tokens (500 into 50304 x
// 1024: 38.5 us with 16 rows, 40.4 with 64; into 60000 x 64 11.8 and 9.9).
// ---------------------------------------------------------------------------
constexpr int kDirectWaves = 8, kDirectAlone = 16, kDirectRows = 64, kDirectWords = kEmbedDirect / 64;

template <int DD, int CH, bool ACC, bool WIDE>
__global__ void __launch_bounds__(kDirectWaves * 64) k_embed_direct(const EmbedBwdArgs a, int token_blocks, int fill_rows) {
  __shared__ uint16_t found[kDirectWaves][kEmbedDirect];
  __shared__ float part[kDirectWaves][CH * 8][64];
  __shared__ uint32_t counts[kDirectWaves];
  __shared__ uint32_t named[kDirectRows];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = blockIdx.y * 512 * CH + lane * 4;
  const int n = (int)a.n_tokens;
  if ((int)blockIdx.x < token_blocks) {
    uint32_t t[kDirectWords];
    tokens32<WIDE, kDirectWords>(a.tokens, 0, n, lane, t);
    const int item = (int)blockIdx.x * kDirectWaves + wave;   // (past the last token: none, as outside the table)
    uint32_t mine = 0xFFFFFFFFu;
#pragma unroll
    for (int w = 0; w < kDirectWords; ++w)
      if (item / 64 == w) mine = t[w];
    const uint32_t v = __builtin_amdgcn_readlane(mine, item % 64);
    int count = 0;
    if (v < (uint32_t)a.rows) {
#pragma unroll
      for (int w = 0; w < kDirectWords; ++w) {
        const uint64_t m = __ballot(t[w] == v);
        if (!m || count < 0) continue;
        if (!count && w * 64 + __builtin_ctzll(m) != item) {   // an earlier token's wave has the row
          count = -1;
          continue;
        }
        if (t[w] == v) found[wave][count + __builtin_popcountll(m & (((uint64_t)1 << lane) - 1))] = (uint16_t)(w * 64 + lane);
        count += __builtin_popcountll(m);
      }
    }
    if (lane == 0) counts[wave] = count > kDirectAlone ? count : 0;
    float acc[2 * CH][4];
    if (count > 0 && count <= kDirectAlone) {
      embed_sum<DD, CH>(a, lane < count ? found[wave][lane] : 0, 0, count, col, acc);
      embed_store<CH, ACC>(a, v, col, acc);
    }
    __syncthreads();
    for (int owner = 0; owner < kDirectWaves; ++owner) {
      const int c = __builtin_amdgcn_readfirstlane(counts[owner]);
      if (!c) continue;
      const int share = (c + kDirectWaves - 1) / kDirectWaves, from = wave * share, left = c - from < share ? c - from : share;
#pragma unroll 1
      for (int i = 0; i == 0 || i < left; i += 64) {
        const int some = left - i < 64 ? left - i : 64;
        embed_sum<DD, CH>(a, lane < some ? found[owner][from + i + lane] : 0, 0, some, col, acc);
#pragma unroll
        for (int k = 0; k < 2 * CH; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* const p = &part[wave][k * 4 + e][lane];
            *p = i ? *p + acc[k][e] : acc[k][e];
          }
      }
      __syncthreads();
      if (wave == owner) {
#pragma unroll 1
        for (int w = 0; w < kDirectWaves; ++w) {
#pragma unroll
          for (int k = 0; k < 2 * CH; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = part[w][k * 4 + e][lane];
              acc[k][e] = w ? acc[k][e] + x : x;
            }
        }
        embed_store<CH, ACC>(a, v, col, acc);
      }
      __syncthreads();
    }
    return;
  }
  const int64_t first = (int64_t)((int)blockIdx.x - token_blocks) * fill_rows;
  if ((int)threadIdx.x < fill_rows) named[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEmbedDirect; i += kDirectWaves * 64) {
    if (i + (int)threadIdx.x < n) {
      const int64_t v = token_at(a.tokens, WIDE, i + threadIdx.x) - first;
      if (v >= 0 && v < fill_rows) named[v] = 1;   // (every writer writes the same)
    }
  }
  __syncthreads();
  typedef typename U16<DT_F32>::T V;
  const int c0 = blockIdx.y * 512 * CH, c1 = a.cols < c0 + 512 * CH ? a.cols : c0 + 512 * CH;
  for (int r = wave; r < fill_rows && first + r < a.rows; r += kDirectWaves) {
    if (named[r]) continue;
    float* out = a.grad + (first + r) * a.cols;
    for (int c = c0 + lane * 4; c < c1; c += 256) {
      if (c + 4 <= c1) {
        *reinterpret_cast<V*>(out + c) = u32x4_t{0u, 0u, 0u, 0u};
      } else {
        for (int e = c; e < c1; ++e) out[e] = 0.0f;
      }
    }
  }
}

// blocks of the sort: one per CU; more where a block would own more rows than its counters hold
static int embed_log2nb(int64_t rows) {
  int log2nb = 8;
  while (((rows + ((int64_t)1 << log2nb) - 1) >> log2nb) > kBinRows) ++log2nb;
  return log2nb;
}
static int64_t embed_per_block(int64_t rows) { return (rows + ((int64_t)1 << embed_log2nb(rows)) - 1) >> embed_log2nb(rows); }
static int64_t embed_pieces(int64_t n_tokens) { return (n_tokens + embed_piece(n_tokens) - 1) / embed_piece(n_tokens); }

size_t embed_bwd_workspace(int64_t rows, int64_t cols, int64_t n_tokens) {
  if (n_tokens <= kEmbedDirect) return 256;   // (not used; 0 would be an error)
  const int64_t partial = 2 * embed_pieces(n_tokens) * cols * 4;
  const int64_t slots = embed_per_block(rows) << embed_log2nb(rows);
  return (size_t)(256 + 2 * round_up(slots * 4, 256) + 2 * round_up(n_tokens * 4, 256) + round_up(partial, 256));
}

void embed_bwd_carve(EmbedBwdArgs& a, unsigned char* ws) {
  a.log2nb = embed_log2nb(a.rows);
  a.piece = embed_piece(a.n_tokens);
  a.per_block = (int32_t)embed_per_block(a.rows);
  const int64_t slots = (int64_t)a.per_block << a.log2nb;
  auto take = [&](int64_t bytes) { unsigned char* p = ws; ws += round_up(bytes, 256); return p; };
  a.n_valid = reinterpret_cast<int32_t*>(take(256));
  a.start = reinterpret_cast<int32_t*>(take(slots * 4));
  a.count = reinterpret_cast<int32_t*>(take(slots * 4));
  a.order = reinterpret_cast<int32_t*>(take(a.n_tokens * 4));
  a.keys = reinterpret_cast<int32_t*>(take(a.n_tokens * 4));
  a.partial = reinterpret_cast<float*>(ws);
}

template <int DD, int CH>
static void embed_sum_launch(const EmbedBwdArgs& a, hipStream_t s) {
  if (a.n_tokens <= kEmbedDirect) {
    const int tb = (int)((a.n_tokens + kDirectWaves - 1) / kDirectWaves);
    const int fr = a.cols <= 256 ? kDirectRows : (a.cols <= 512 ? kDirectRows / 2 : kDirectRows / 4);
    const int64_t fill = a.accumulate ? 0 : (a.rows + fr - 1) / fr;
    const dim3 grid((unsigned)(tb + fill), (unsigned)((a.cols + 512 * CH - 1) / (512 * CH)));
    auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(kDirectWaves * 64), 0, s, a, tb, fr); };
    if (a.accumulate) a.wide ? go(k_embed_direct<DD, CH, true, true>) : go(k_embed_direct<DD, CH, true, false>);
    else a.wide ? go(k_embed_direct<DD, CH, false, true>) : go(k_embed_direct<DD, CH, false, false>);
    return;
  }
  const int64_t pieces = embed_pieces(a.n_tokens);
  const int pb = (int)((pieces + 3) / 4);
  const dim3 grid((unsigned)(pb + (a.rows + 3) / 4), (unsigned)((a.cols + 512 * CH - 1) / (512 * CH)));
  if (a.accumulate) hipLaunchKernelGGL((k_embed_sum<DD, CH, true, false>), grid, dim3(256), 0, s, a, pb);
  else if (a.rows * a.cols * 4 > kStreamBytes) hipLaunchKernelGGL((k_embed_sum<DD, CH, false, true>), grid, dim3(256), 0, s, a, pb);
  else hipLaunchKernelGGL((k_embed_sum<DD, CH, false, false>), grid, dim3(256), 0, s, a, pb);
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, int dout_dt, hipStream_t s) {
  if (a.n_tokens == 0 && a.accumulate) return hipSuccess;
  const bool direct = a.n_tokens <= kEmbedDirect;
  hipError_t err = hipSuccess;
  if (!direct) {
    if (a.wide) hipLaunchKernelGGL((k_embed_bin<true>), dim3(1u << a.log2nb), dim3(kBinThreads), 0, s, a);
    else hipLaunchKernelGGL((k_embed_bin<false>), dim3(1u << a.log2nb), dim3(kBinThreads), 0, s, a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  if (dout_dt == DT_F32) {
    if (a.cols <= 512) embed_sum_launch<DT_F32, 1>(a, s);
    else embed_sum_launch<DT_F32, 2>(a, s);
  } else {
    if (a.cols <= 512) embed_sum_launch<DT_BF16, 1>(a, s);
    else embed_sum_launch<DT_BF16, 2>(a, s);
  }
  if ((err = hipGetLastError()) != hipSuccess) return err;
  if (!direct) {
    hipLaunchKernelGGL(k_embed_join, dim3((unsigned)((embed_pieces(a.n_tokens) + kJoinPieces - 1) / kJoinPieces), (unsigned)((a.cols + 255) / 256)),
                       dim3(kJoinWaves * 64), 0, s, a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace ma
