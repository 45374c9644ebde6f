// Embedding lookup with scaling, and its gradient by sorted tokens (gfx950).
//
//   forward   out[i,:]  = RNE(scale * table[t_i,:])
//   backward  grad[v,:] (+)= scale * sum over { i : t_i = v }, i ascending, of dout[i,:]
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
// forward: LPR lanes per output row, R rows per lane group at a time, so that
// R independent row reads are in flight behind their R token reads.
// ---------------------------------------------------------------------------
template <int TD, int OD, int LPR>
__global__ void __launch_bounds__(256) k_embed_fwd(const EmbedFwdArgs a) {
  constexpr int R = 4, GROUPS = 256 / LPR;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int64_t r0 = ((int64_t)blockIdx.x * GROUPS + group) * R;
  int64_t tok[R];
  bool in[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    tok[r] = r0 + r < a.n_tokens ? token_at(a.tokens, a.wide, r0 + r) : -1;
    in[r] = tok[r] >= 0 && tok[r] < a.rows;
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
      raw_f32<TD>(x[r], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in[r] ? v[e] * a.scale : 0.0f;
      store_row<OD>(elem_ptr<OD>(a.out, (r0 + r) * a.cols), col, a.cols, v);
    }
  }
}

template <int TD, int OD>
static hipError_t embed_fwd(const EmbedFwdArgs& a, hipStream_t s) {
  const int chunks = (a.cols + 7) / 8;
  auto grid = [&](int lpr) { const int64_t per = 256 / lpr * 4; return dim3((unsigned)((a.n_tokens + per - 1) / per)); };
  if (chunks <= 16) hipLaunchKernelGGL((k_embed_fwd<TD, OD, 16>), grid(16), dim3(256), 0, s, a);
  else if (chunks <= 32) hipLaunchKernelGGL((k_embed_fwd<TD, OD, 32>), grid(32), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_embed_fwd<TD, OD, 64>), grid(64), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_embed_fwd(const EmbedFwdArgs& a, int table_dt, int out_dt, hipStream_t s) {
  if (a.n_tokens == 0) return hipSuccess;
  if (table_dt == DT_F32) return out_dt == DT_F32 ? embed_fwd<DT_F32, DT_F32>(a, s) : embed_fwd<DT_F32, DT_BF16>(a, s);
  return out_dt == DT_F32 ? embed_fwd<DT_BF16, DT_F32>(a, s) : embed_fwd<DT_BF16, DT_BF16>(a, s);
}

// ---------------------------------------------------------------------------
// backward, 1: the tokens' positions sorted by (row mod NB, row / NB), stable,
// in one launch. Block b of NB (a power of two) owns the rows v = b mod NB
// (interleaved: frequent rows with neighbouring ids go to different blocks).
// It reads all tokens twice. First pass: how many valid tokens belong to
// earlier blocks (where its own part of the sorted order begins), and how
// often each of its rows occurs in each wave's sixteenth of the tokens.
// Second pass: every wave writes its tokens' positions behind those of the
// waves before it. No global atomics, and the order is ascending position.
// ---------------------------------------------------------------------------
constexpr int kBinThreads = 1024, kBinWaves = kBinThreads / 64, kBinRows = 512;

__global__ void __launch_bounds__(kBinThreads) k_embed_bin(const EmbedBwdArgs a, int log2nb) {
  __shared__ uint32_t hist[kBinWaves][kBinRows];
  __shared__ uint32_t scan[kBinRows];
  __shared__ uint32_t wsum[kBinWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t nb = (int64_t)1 << log2nb, me = blockIdx.x;
  const int mine = (int)((a.rows - me + nb - 1) >> log2nb);   // rows owned, <= kBinRows; 0 if me >= rows
  for (int i = tid; i < kBinWaves * kBinRows; i += kBinThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t seg = round_up((a.n_tokens + kBinWaves - 1) / kBinWaves, 64);
  const int64_t i0 = wave * seg, i1 = i0 + seg < a.n_tokens ? i0 + seg : a.n_tokens;
  uint32_t less = 0;
  constexpr int U = 8;
  for (int64_t i = i0; i < i1; i += 64 * U) {
    int64_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = i + u * 64 + lane < i1 ? token_at(a.tokens, a.wide, i + u * 64 + lane) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = v[u] >= 0 && v[u] < a.rows;
      const int64_t b = v[u] & (nb - 1);
      less += in && b < me;
      if (in && b == me) atomicAdd(&hist[wave][v[u] >> log2nb], 1u);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) less += __shfl_xor(less, o, 64);
  if (lane == 0) wsum[wave] = less;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < kBinWaves; ++w) base += wsum[w];
  // per row: exclusive counts over the waves, and the row's total
  uint32_t total = 0;
  if (tid < kBinRows) {
#pragma unroll
    for (int w = 0; w < kBinWaves; ++w) {
      const uint32_t h = hist[w][tid];
      hist[w][tid] = total;
      total += h;
    }
    scan[tid] = total;
  }
  // inclusive scan of the totals over the owned rows
#pragma unroll
  for (int o = 1; o < kBinRows; o <<= 1) {
    __syncthreads();
    const uint32_t x = tid < kBinRows && tid >= o ? scan[tid - o] : 0u;
    __syncthreads();
    if (tid < kBinRows) scan[tid] += x;
  }
  __syncthreads();
  if (tid < mine) {
    const int64_t v = ((int64_t)tid << log2nb) + me;
    a.start[v] = (int32_t)(base + scan[tid] - total);
    a.count[v] = (int32_t)total;
  }
  if (me == nb - 1 && tid == 0) *a.n_valid = (int32_t)(base + scan[kBinRows - 1]);
  if (tid < kBinRows) {
    const uint32_t at = base + scan[tid] - total;
#pragma unroll
    for (int w = 0; w < kBinWaves; ++w) hist[w][tid] += at;
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 64 * U) {
    int64_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = i + u * 64 + lane < i1 ? token_at(a.tokens, a.wide, i + u * 64 + lane) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool own = v[u] >= 0 && v[u] < a.rows && (v[u] & (nb - 1)) == me;
      const int bin = (int)(v[u] >> log2nb);
      uint64_t left = __ballot(own);
      // one step per different row among the 64 tokens
      while (left) {
        const int first = __builtin_ctzll(left);
        const int bin0 = __builtin_amdgcn_readlane(bin, first);
        const uint64_t same = __ballot(own && bin == bin0);
        volatile uint32_t& next = hist[wave][bin0];
        const uint32_t at = next;
        if (own && bin == bin0) {
          const uint32_t k = at + __builtin_popcountll(same & (((uint64_t)1 << lane) - 1));
          a.order[k] = (int32_t)(i + u * 64 + lane);
          a.keys[k] = (int32_t)v[u];
        }
        if (lane == first) next = at + (uint32_t)__builtin_popcountll(same);
        left &= ~same;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward, 2: the sums. One wave per row of the table and slice of 512 * CH
// columns sums the row's run (at most kEmbedPiece tokens) and writes it, zeros
// for an empty one; when accumulating, one wave per sorted position, of which
// those at the start of a run work. Longer runs are summed by the piece waves
// (the launch's first blocks), one per kEmbedPiece sorted positions: the part
// of a long run that its first position belongs to goes to partial row 2p, that
// of another long run that its last position belongs to to 2p + 1 (no third
// one fits), and k_embed_join adds a run's parts in order.
// ---------------------------------------------------------------------------
template <int DD, int CH>
__device__ __forceinline__ void embed_sum(const EmbedBwdArgs& a, int32_t pos, int from, int to, int col, float (&acc)[CH][8]) {
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[c][e] = 0.0f;
  constexpr int U = 4;
  for (int j = from; j < to; j += U) {
    Raw8<DD> x[U][CH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < to) {
        const int64_t p = __builtin_amdgcn_readlane(pos, j + u);
        const unsigned char* row = elem_ptr<DD>(a.dout, p * a.cols);
#pragma unroll
        for (int c = 0; c < CH; ++c)
          x[u][c] = col + c * 512 < a.cols ? raw_load_row<DD>(row, col + c * 512, a.cols) : raw_zero<DD>();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < to) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float v[8];
          raw_f32<DD>(x[u][c], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c][e] += v[e];
        }
      }
    }
  }
}

template <int DD, int CH, bool ACC>
__global__ void __launch_bounds__(256) k_embed_sum(const EmbedBwdArgs a, int piece_blocks) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = blockIdx.y * 512 * CH + lane * 8;
  float acc[CH][8];
  if ((int)blockIdx.x < piece_blocks) {
    const int64_t p = (int64_t)blockIdx.x * 4 + wave;
    const int64_t first = p * kEmbedPiece;
    const int64_t left = *a.n_valid - first;
    if (left <= 0) return;
    const int n = left < kEmbedPiece ? (int)left : kEmbedPiece;
    const int32_t key = lane < n ? a.keys[first + lane] : 0, pos = lane < n ? a.order[first + lane] : 0;
    const int32_t va = __builtin_amdgcn_readlane(key, 0), vb = __builtin_amdgcn_readlane(key, n - 1);
    for (int side = 0; side < 2; ++side) {
      const int32_t v = side ? vb : va;
      if (side && vb == va) break;
      const int64_t s = a.start[v], c = a.count[v];
      if (c <= kEmbedPiece) continue;
      const int from = s > first ? (int)(s - first) : 0;
      const int to = s + c - first < n ? (int)(s + c - first) : n;
      embed_sum<DD, CH>(a, pos, from, to, col, acc);
      unsigned char* out = reinterpret_cast<unsigned char*>(a.partial + (2 * p + side) * a.cols);
#pragma unroll
      for (int k = 0; k < CH; ++k)
        if (col + k * 512 < a.cols) store_row<DT_F32>(out, col + k * 512, a.cols, acc[k]);
    }
    return;
  }
  const int64_t item = (int64_t)(blockIdx.x - piece_blocks) * 4 + wave;
  int64_t v = item;
  if constexpr (ACC) {
    if (item >= *a.n_valid) return;
    v = a.keys[item];
  } else {
    if (item >= a.rows) return;
  }
  const int64_t s = a.start[v];
  const int c = a.count[v];
  if (c > kEmbedPiece || (ACC && s != item)) return;
  const int32_t pos = lane < c ? a.order[s + lane] : 0;
  embed_sum<DD, CH>(a, pos, 0, c, col, acc);
  unsigned char* out = reinterpret_cast<unsigned char*>(a.grad + v * a.cols);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int cc = col + k * 512;
    if (cc >= a.cols) continue;
    float old[8] = {};
    if constexpr (ACC) raw_f32<DT_F32>(raw_load_row<DT_F32>(out, cc, a.cols), old);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = ACC ? __fadd_rn(old[e], __fmul_rn(acc[k][e], a.scale)) : acc[k][e] * a.scale;
    store_row<DT_F32, !ACC>(out, cc, a.cols, acc[k]);
  }
}

// The long run that starts in piece p, if one does: 16 waves sum its parts in
// 16 contiguous shares, 256 columns each, and the shares are added in order.
__global__ void __launch_bounds__(1024) k_embed_join(const EmbedBwdArgs a) {
  __shared__ float part[16][256];
  const int64_t p = blockIdx.x, first = p * kEmbedPiece;
  const int64_t left = *a.n_valid - first;
  if (left <= kEmbedPiece) return;   // no run of this piece goes on in another
  const int32_t v = a.keys[first + kEmbedPiece - 1];
  const int64_t s = a.start[v], c = a.count[v];
  if (c <= kEmbedPiece || s < first) return;
  const int64_t last = (s + c - 1) / kEmbedPiece;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t n = last - p + 1, share = (n + 15) / 16;
  const int64_t q0 = p + wave * share, q1 = q0 + share < last + 1 ? q0 + share : last + 1;
  const int col = blockIdx.y * 256 + lane;
  float acc[4] = {};
#pragma unroll 4
  for (int64_t q = q0; q < q1; ++q) {
    const float* src = a.partial + (2 * q + (q == p && s > first)) * a.cols;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + 64 * k < a.cols) acc[k] += src[col + 64 * k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) part[wave][lane + 64 * k] = acc[k];
  __syncthreads();
  if (threadIdx.x < 256) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += part[w][threadIdx.x];
    const int cc = blockIdx.y * 256 + threadIdx.x;
    if (cc < a.cols) {
      float* g = a.grad + (int64_t)v * a.cols + cc;
      *g = a.accumulate ? __fadd_rn(*g, __fmul_rn(t, a.scale)) : t * a.scale;
    }
  }
}

static int64_t embed_pieces(int64_t n_tokens) { return (n_tokens + kEmbedPiece - 1) / kEmbedPiece; }

size_t embed_bwd_workspace(int64_t rows, int64_t cols, int64_t n_tokens) {
  const int64_t partial = n_tokens > kEmbedPiece ? 2 * embed_pieces(n_tokens) * cols * 4 : 0;
  return (size_t)(256 + 2 * round_up(rows * 4, 256) + 2 * round_up(n_tokens * 4, 256) + round_up(partial, 256));
}

void embed_bwd_carve(EmbedBwdArgs& a, unsigned char* ws) {
  auto take = [&](int64_t bytes) { unsigned char* p = ws; ws += round_up(bytes, 256); return p; };
  a.n_valid = reinterpret_cast<int32_t*>(take(256));
  a.start = reinterpret_cast<int32_t*>(take(a.rows * 4));
  a.count = reinterpret_cast<int32_t*>(take(a.rows * 4));
  a.order = reinterpret_cast<int32_t*>(take(a.n_tokens * 4));
  a.keys = reinterpret_cast<int32_t*>(take(a.n_tokens * 4));
  a.partial = reinterpret_cast<float*>(ws);
}

template <int DD, int CH>
static void embed_sum_launch(const EmbedBwdArgs& a, hipStream_t s) {
  const int64_t pieces = a.n_tokens > kEmbedPiece ? embed_pieces(a.n_tokens) : 0;
  const int pb = (int)((pieces + 3) / 4);
  const int64_t items = a.accumulate ? a.n_tokens : a.rows;
  const dim3 grid((unsigned)(pb + (items + 3) / 4), (unsigned)((a.cols + 512 * CH - 1) / (512 * CH)));
  if (a.accumulate) hipLaunchKernelGGL((k_embed_sum<DD, CH, true>), grid, dim3(256), 0, s, a, pb);
  else hipLaunchKernelGGL((k_embed_sum<DD, CH, false>), grid, dim3(256), 0, s, a, pb);
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, int dout_dt, hipStream_t s) {
  if (a.n_tokens == 0 && a.accumulate) return hipSuccess;
  int log2nb = 8;   // a block per CU; more where a block would own more rows than its counters hold
  while (((a.rows + ((int64_t)1 << log2nb) - 1) >> log2nb) > kBinRows) ++log2nb;
  hipLaunchKernelGGL(k_embed_bin, dim3(1u << log2nb), dim3(kBinThreads), 0, s, a, log2nb);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (dout_dt == DT_F32) {
    if (a.cols <= 512) embed_sum_launch<DT_F32, 1>(a, s);
    else embed_sum_launch<DT_F32, 2>(a, s);
  } else {
    if (a.cols <= 512) embed_sum_launch<DT_BF16, 1>(a, s);
    else embed_sum_launch<DT_BF16, 2>(a, s);
  }
  if ((err = hipGetLastError()) != hipSuccess) return err;
  if (a.n_tokens > kEmbedPiece) {
    hipLaunchKernelGGL(k_embed_join, dim3((unsigned)embed_pieces(a.n_tokens), (unsigned)((a.cols + 255) / 256)), dim3(1024), 0, s, a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace ma
