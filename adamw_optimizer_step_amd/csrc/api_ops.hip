// C ABI of the operators around the optimizer step (embedding, norms, 8-bit
// activation checkpoints, weight gradient, 4-bit matrices and their product):
// argument validation and the launches. See include/muon_adamw.h for the contract of every entry point.
#include <algorithm>
#include <cmath>

#include "../../include/muon_adamw.h"
#include "host.hpp"
#include "mx4.hpp"
#include "rows.hpp"
#include "train_ops.hpp"

using namespace ma;

namespace {

// size limits: keep every launch within 2^32 threads and every index within its type
constexpr int64_t kMaxRows = (int64_t)1 << 24, kMaxCols = (int64_t)1 << 24, kMaxTokens = (int64_t)1 << 25;
constexpr int64_t kMaxEmbedCols = (int64_t)1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 36, kMaxTable = (int64_t)1 << 35;   // (a wave per row and 1024 columns of the table)

bool dt_ok(int dt) { return dt == MA_F32 || dt == MA_BF16; }
int64_t dt_size(int dt) { return dt == MA_BF16 ? 2 : 4; }

// A device buffer of a call. Null with zero bytes, or where optional.
struct Buf {
  const void* p;
  int64_t bytes;
  int align;
  bool out, optional;
  const char* name;
};

// Every buffer present and aligned, and no output overlapping another buffer.
template <int N>
int check_buffers(const char* fn, const Buf (&b)[N]) {
  for (const Buf& x : b) {
    if (!x.p) {
      if (x.bytes > 0 && !x.optional) return fail(MA_ERR_INVALID_ARG, "%s: %s is null", fn, x.name);
      continue;
    }
    if ((uintptr_t)x.p % x.align) return fail(MA_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, x.name, x.align);
  }
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j) {
      if (i == j || !b[i].out || !b[i].p || !b[j].p || b[i].bytes <= 0 || b[j].bytes <= 0) continue;
      const uintptr_t x = (uintptr_t)b[i].p, y = (uintptr_t)b[j].p;
      if (x < y + (uintptr_t)b[j].bytes && y < x + (uintptr_t)b[i].bytes)
        return fail(MA_ERR_INVALID_ARG, "%s: device buffers overlap (%s and %s)", fn, b[i].name, b[j].name);
    }
  return MA_OK;
}

int check_size(const char* fn, const char* what, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi) return fail(MA_ERR_INVALID_ARG, "%s: %s %lld outside %lld..%lld", fn, what, (long long)v, (long long)lo, (long long)hi);
  return MA_OK;
}

int check_matrix(const char* fn, int64_t rows, int64_t row_lo, int64_t row_hi, int64_t cols, int64_t col_hi) {
  int rc;
  if ((rc = check_size(fn, "rows", rows, row_lo, row_hi)) || (rc = check_size(fn, "cols", cols, 1, col_hi))) return rc;
  if (rows * cols > kMaxElems) return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements", fn);
  return MA_OK;
}

int check_dtype(const char* fn, const char* what, int dt) {
  if (!dt_ok(dt)) return fail(MA_ERR_UNSUPPORTED, "%s: %s dtype %d is neither MA_F32 nor MA_BF16", fn, what, dt);
  return MA_OK;
}

int check_flag(const char* fn, int v) {
  if (v != 0 && v != 1) return fail(MA_ERR_INVALID_ARG, "%s: accumulate %d is not 0 or 1", fn, v);
  return MA_OK;
}

int check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need == 0) return MA_OK;
  if (!ws) return fail(MA_ERR_WORKSPACE, "%s: workspace is null (%zu bytes needed)", fn, need);
  if (have < need) return fail(MA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, have, need);
  if ((uintptr_t)ws % MA_WORKSPACE_ALIGN) return fail(MA_ERR_WORKSPACE, "%s: workspace is not %d-byte aligned", fn, MA_WORKSPACE_ALIGN);
  return MA_OK;
}

int done(hipError_t err, const char* fn) { return err == hipSuccess ? MA_OK : hip_fail(err, fn); }

int embedding_sizes(const char* fn, int64_t rows, int64_t cols, int64_t n_tokens) {
  int rc;
  if ((rc = check_matrix(fn, rows, 1, kMaxRows, cols, kMaxEmbedCols)) || (rc = check_size(fn, "n_tokens", n_tokens, 0, kMaxTokens))) return rc;
  if (rows * cols > kMaxTable) return fail(MA_ERR_INVALID_ARG, "%s: a table of more than 2^35 elements", fn);
  if (n_tokens * cols > kMaxElems) return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements", fn);
  return MA_OK;
}

}  // namespace

int ma_embedding_forward(const void* table, int32_t table_dtype, int64_t rows, int64_t cols, const void* tokens, int32_t token_bytes,
                         int64_t n_tokens, float scale, void* out, int32_t out_dtype, void* stream) {
  const char* fn = "ma_embedding_forward";
  EntryMark mark(fn);
  int rc;
  if ((rc = embedding_sizes(fn, rows, cols, n_tokens)) || (rc = check_dtype(fn, "table", table_dtype)) || (rc = check_dtype(fn, "out", out_dtype)))
    return rc;
  if (token_bytes != 4 && token_bytes != 8) return fail(MA_ERR_UNSUPPORTED, "%s: token_bytes %d is neither 4 nor 8", fn, token_bytes);
  if (!std::isfinite(scale)) return fail(MA_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  const Buf bufs[] = {{table, rows * cols * dt_size(table_dtype), (int)dt_size(table_dtype), false, false, "table"},
                      {tokens, n_tokens * token_bytes, token_bytes, false, false, "tokens"},
                      {out, n_tokens * cols * dt_size(out_dtype), (int)dt_size(out_dtype), true, false, "out"}};
  if ((rc = check_buffers(fn, bufs))) return rc;
  if (n_tokens == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const EmbedFwdArgs a{table, tokens, out, rows, n_tokens, (int32_t)cols, token_bytes == 8, scale};
  ProfScope ps(MA_K_EMBEDDING, s);
  return done(launch_embed_fwd(a, table_dtype, out_dtype, s), fn);
}

size_t ma_embedding_workspace_size(int64_t rows, int64_t cols, int64_t n_tokens) {
  if (embedding_sizes("ma_embedding_workspace_size", rows, cols, n_tokens)) return 0;
  // short pieces take more room than long ones of somewhat more tokens
  const size_t need = embed_bwd_workspace(rows, cols, n_tokens);
  return n_tokens > kEmbedShortPieces ? std::max(need, embed_bwd_workspace(rows, cols, kEmbedShortPieces)) : need;
}

int ma_embedding_backward(const void* dout, int32_t dout_dtype, const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t rows,
                          int64_t cols, float scale, int32_t accumulate, float* grad, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ma_embedding_backward";
  EntryMark mark(fn);
  int rc;
  if ((rc = embedding_sizes(fn, rows, cols, n_tokens)) || (rc = check_dtype(fn, "dout", dout_dtype)) || (rc = check_flag(fn, accumulate))) return rc;
  if (token_bytes != 4 && token_bytes != 8) return fail(MA_ERR_UNSUPPORTED, "%s: token_bytes %d is neither 4 nor 8", fn, token_bytes);
  if (!std::isfinite(scale)) return fail(MA_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  const size_t need = embed_bwd_workspace(rows, cols, n_tokens);
  const Buf bufs[] = {{dout, n_tokens * cols * dt_size(dout_dtype), (int)dt_size(dout_dtype), false, false, "dout"},
                      {tokens, n_tokens * token_bytes, token_bytes, false, false, "tokens"},
                      {grad, rows * cols * 4, 4, true, false, "grad"},
                      {workspace, (int64_t)need, 1, true, true, "the workspace"}};
  if ((rc = check_workspace(fn, workspace, workspace_bytes, need)) || (rc = check_buffers(fn, bufs))) return rc;
  if (n_tokens == 0 && accumulate) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  EmbedBwdArgs a{};
  a.dout = dout;
  a.tokens = tokens;
  a.grad = grad;
  a.rows = rows;
  a.n_tokens = n_tokens;
  a.cols = (int32_t)cols;
  a.wide = token_bytes == 8;
  a.accumulate = accumulate;
  a.scale = scale;
  embed_bwd_carve(a, reinterpret_cast<unsigned char*>(workspace));
  ProfScope ps(MA_K_EMBEDDING, s);
  return done(launch_embed_bwd(a, dout_dtype, s), fn);
}

int ma_layernorm_forward(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, const float* gain, const float* bias, float eps, void* y,
                         int32_t y_dtype, float* stats, uint8_t* ckpt_q, uint8_t* ckpt_scale, void* stream) {
  const char* fn = "ma_layernorm_forward";
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxNormCols)) || (rc = check_dtype(fn, "x", x_dtype)) || (rc = check_dtype(fn, "y", y_dtype)))
    return rc;
  if (!std::isfinite(eps) || eps < 0.0f) return fail(MA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!ckpt_q != !ckpt_scale) return fail(MA_ERR_INVALID_ARG, "%s: a checkpoint needs both q and scale", fn);
  const int64_t pitch = act_pitch(cols);
  const Buf bufs[] = {{x, rows * cols * dt_size(x_dtype), (int)dt_size(x_dtype), false, false, "x"},
                      {gain, cols * 4, 4, false, true, "gain"},
                      {bias, cols * 4, 4, false, true, "bias"},
                      {y, rows * cols * dt_size(y_dtype), (int)dt_size(y_dtype), true, false, "y"},
                      {stats, rows * 8, 8, true, false, "stats"},
                      {ckpt_q, rows * pitch, 16, true, true, "the checkpoint's q"},
                      {ckpt_scale, rows * (pitch / kActBlock), 1, true, true, "the checkpoint's scale"}};
  if ((rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const NormFwdArgs a{x, gain, bias, y, stats, ckpt_q, ckpt_scale, rows, (int32_t)cols, eps};
  ProfScope ps(MA_K_LAYERNORM, s);
  return done(launch_norm_fwd(a, x_dtype, y_dtype, s), fn);
}

static size_t norm_workspace(int64_t rows, int64_t cols) {
  return norm_bwd_direct(rows) ? 0 : (size_t)round_up(norm_bwd_blocks(rows, cols) * 2 * round_up(cols, 32) * 4, MA_WORKSPACE_ALIGN);
}

size_t ma_layernorm_workspace_size(int64_t rows, int64_t cols) {
  if (check_matrix("ma_layernorm_workspace_size", rows, 0, kMaxRows, cols, kMaxNormCols)) return 0;
  return norm_workspace(rows, cols);
}

int ma_layernorm_backward(const void* dy, int32_t dy_dtype, const void* x, int32_t x_dtype, const uint8_t* ckpt_q, const uint8_t* ckpt_scale,
                          int64_t rows, int64_t cols, const float* stats, const float* gain, void* dx, int32_t dx_dtype, float* dgain,
                          float* dbias, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ma_layernorm_backward";
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxNormCols)) || (rc = check_dtype(fn, "dy", dy_dtype)) ||
      (rc = check_dtype(fn, "dx", dx_dtype)) || (rc = check_flag(fn, accumulate)))
    return rc;
  if (!ckpt_q != !ckpt_scale) return fail(MA_ERR_INVALID_ARG, "%s: a checkpoint needs both q and scale", fn);
  if (x && ckpt_q) return fail(MA_ERR_INVALID_ARG, "%s: give x or its checkpoint, not both", fn);
  const bool held = !x;   // (an empty x may be null too)
  if (!held && (rc = check_dtype(fn, "x", x_dtype))) return rc;
  if (rows > 0 && dx_dtype != (held ? dy_dtype : x_dtype))
    return fail(MA_ERR_UNSUPPORTED, "%s: dx has the type of x, or of dy where x is a checkpoint", fn);
  const int64_t pitch = act_pitch(cols);
  const bool sums = dgain || dbias;
  const size_t need = sums ? norm_workspace(rows, cols) : 0;
  const Buf bufs[] = {{dy, rows * cols * dt_size(dy_dtype), (int)dt_size(dy_dtype), false, false, "dy"},
                      {x, held ? 0 : rows * cols * dt_size(x_dtype), held ? 1 : (int)dt_size(x_dtype), false, false, "x"},
                      {ckpt_q, rows * pitch, 16, false, !held, "x and the checkpoint's q"},
                      {ckpt_scale, rows * (pitch / kActBlock), 1, false, !held, "the checkpoint's scale"},
                      {stats, rows * 8, 8, false, false, "stats"},
                      {gain, cols * 4, 4, false, true, "gain"},
                      {dx, rows * cols * dt_size(dx_dtype), (int)dt_size(dx_dtype), true, false, "dx"},
                      {dgain, cols * 4, 4, true, true, "dgain"},
                      {dbias, cols * 4, 4, true, true, "dbias"},
                      {workspace, (int64_t)need, 1, true, true, "the workspace"}};
  if ((rc = check_workspace(fn, workspace, workspace_bytes, need)) || (rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0 && (!sums || accumulate)) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const NormBwdArgs a{dy, x, ckpt_q, ckpt_scale, stats, gain, dx, dgain, dbias, need ? reinterpret_cast<float*>(workspace) : nullptr,
                      rows, (int32_t)cols, accumulate, norm_bwd_blocks(rows, cols)};
  ProfScope ps(MA_K_LAYERNORM, s);
  return done(launch_norm_bwd(a, held ? DT_ACT8 : x_dtype, dy_dtype, dx_dtype, s), fn);
}

int ma_rmsnorm_forward(const void* x, int32_t x_dtype, const void* residual, int32_t residual_dtype, int64_t rows, int64_t cols,
                       const float* gain, float eps, void* total, void* y, int32_t y_dtype, float* rstd, uint8_t* held_q,
                       uint8_t* held_scale, void* stream) {
  const char* fn = "ma_rmsnorm_forward";
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxNormCols)) || (rc = check_dtype(fn, "x", x_dtype))) return rc;
  if (residual && (rc = check_dtype(fn, "residual", residual_dtype))) return rc;
  if (!std::isfinite(eps) || eps < 0.0f) return fail(MA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!held_q != !held_scale) return fail(MA_ERR_INVALID_ARG, "%s: a checkpoint needs both q and scale", fn);
  if (rows > 0 && !residual != !total) return fail(MA_ERR_INVALID_ARG, "%s: total and residual are given together", fn);
  if ((y || !held_q) && (rc = check_dtype(fn, "y", y_dtype))) return rc;
  const int t_dtype = residual ? residual_dtype : x_dtype;
  const int64_t pitch = act_pitch(cols), t_bytes = rows * cols * dt_size(t_dtype);
  const Buf bufs[] = {{x, rows * cols * dt_size(x_dtype), (int)dt_size(x_dtype), false, false, "x"},
                      {residual, t_bytes, (int)dt_size(t_dtype), false, true, "residual"},
                      {gain, cols * 4, 4, false, true, "gain"},
                      {total, t_bytes, (int)dt_size(t_dtype), true, true, "total"},
                      {y, y ? rows * cols * dt_size(y_dtype) : rows, y ? (int)dt_size(y_dtype) : 1, true, held_q != nullptr, "y"},
                      {rstd, rows * 4, 4, true, false, "rstd"},
                      {held_q, rows * pitch, 16, true, true, "the checkpoint's q"},
                      {held_scale, rows * (pitch / kActBlock), 1, true, true, "the checkpoint's scale"}};
  if ((rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const RmsFwdArgs a{x, residual, gain, total, y, rstd, held_q, held_scale, rows, (int32_t)cols, eps};
  ProfScope ps(MA_K_RMSNORM, s);
  return done(launch_rms_fwd(a, x_dtype, t_dtype, y ? y_dtype : MA_BF16, s), fn);
}

static size_t rms_workspace(int64_t rows, int64_t cols) {
  return norm_bwd_direct(rows) ? 0 : (size_t)round_up(norm_bwd_blocks(rows, cols) * round_up(cols, 32) * 4, MA_WORKSPACE_ALIGN);
}

size_t ma_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
  if (check_matrix("ma_rmsnorm_workspace_size", rows, 0, kMaxRows, cols, kMaxNormCols)) return 0;
  return rms_workspace(rows, cols);
}

int ma_rmsnorm_backward(const void* dy, int32_t dy_dtype, const void* t, int32_t t_dtype, const uint8_t* held_q, const uint8_t* held_scale,
                        int64_t rows, int64_t cols, const float* rstd, const float* gain, const void* dtotal, void* dx, int32_t dx_dtype,
                        float* dgain, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ma_rmsnorm_backward";
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxNormCols)) || (rc = check_dtype(fn, "dy", dy_dtype)) ||
      (rc = check_dtype(fn, "dx", dx_dtype)) || (rc = check_flag(fn, accumulate)))
    return rc;
  if (!held_q != !held_scale) return fail(MA_ERR_INVALID_ARG, "%s: a checkpoint needs both q and scale", fn);
  if (t && held_q) return fail(MA_ERR_INVALID_ARG, "%s: give t or its checkpoint, not both", fn);
  const bool held = !t;   // (an empty t may be null too)
  if (!held && (rc = check_dtype(fn, "t", t_dtype))) return rc;
  if (rows > 0 && dx_dtype != (held ? dy_dtype : t_dtype))
    return fail(MA_ERR_UNSUPPORTED, "%s: dx has the type of t, or of dy where t is a checkpoint", fn);
  const int64_t pitch = act_pitch(cols), dx_bytes = rows * cols * dt_size(dx_dtype);
  const size_t need = dgain ? rms_workspace(rows, cols) : 0;
  const Buf bufs[] = {{dy, rows * cols * dt_size(dy_dtype), (int)dt_size(dy_dtype), false, false, "dy"},
                      {t, held ? 0 : rows * cols * dt_size(t_dtype), held ? 1 : (int)dt_size(t_dtype), false, false, "t"},
                      {held_q, rows * pitch, 16, false, !held, "t and the checkpoint's q"},
                      {held_scale, rows * (pitch / kActBlock), 1, false, !held, "the checkpoint's scale"},
                      {rstd, rows * 4, 4, false, false, "rstd"},
                      {gain, cols * 4, 4, false, true, "gain"},
                      {dtotal, dx_bytes, (int)dt_size(dx_dtype), false, true, "dtotal"},
                      {dx, dx_bytes, (int)dt_size(dx_dtype), true, false, "dx"},
                      {dgain, cols * 4, 4, true, true, "dgain"},
                      {workspace, (int64_t)need, 1, true, true, "the workspace"}};
  if ((rc = check_workspace(fn, workspace, workspace_bytes, need)) || (rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0 && (!dgain || accumulate)) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const RmsBwdArgs a{dy, t, held_q, held_scale, rstd, gain, dtotal, dx, dgain, need ? reinterpret_cast<float*>(workspace) : nullptr,
                     rows, (int32_t)cols, accumulate, norm_bwd_blocks(rows, cols)};
  ProfScope ps(MA_K_RMSNORM, s);
  return done(launch_rms_bwd(a, held ? DT_ACT8 : t_dtype, dy_dtype, dx_dtype, s), fn);
}

static int act_call(const char* fn, const void* x, int32_t dtype, bool pack, int64_t rows, int64_t cols, const uint8_t* q, const uint8_t* scale,
                    void* stream) {
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxCols)) || (rc = check_dtype(fn, pack ? "x" : "out", dtype))) return rc;
  const int64_t pitch = act_pitch(cols);
  if (rows * pitch > (dtype == MA_F32 ? kMaxElems / 2 : kMaxElems)) return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements (2^35 fp32 ones)", fn);
  const Buf bufs[] = {{x, rows * cols * dt_size(dtype), (int)dt_size(dtype), !pack, false, pack ? "x" : "out"},
                      {q, rows * pitch, 16, pack, false, "q"},
                      {scale, rows * (pitch / kActBlock), 1, pack, false, "scale"}};
  if ((rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const ActArgs a{pack ? x : nullptr, pack ? nullptr : const_cast<void*>(x), const_cast<uint8_t*>(q), const_cast<uint8_t*>(scale), rows, (int32_t)cols};
  ProfScope ps(MA_K_ACT, s);
  return done(pack ? launch_act_pack(a, dtype, s) : launch_act_unpack(a, dtype, s), fn);
}

int ma_act_pack(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, uint8_t* q, uint8_t* scale, void* stream) {
  return act_call("ma_act_pack", x, x_dtype, true, rows, cols, q, scale, stream);
}

int ma_act_unpack(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, void* out, int32_t out_dtype, void* stream) {
  return act_call("ma_act_unpack", out, out_dtype, false, rows, cols, q, scale, stream);
}

// bytes of q and of scale of a 4-bit rows x cols matrix
static int64_t mx4_q_bytes(int64_t rows, int64_t cols) { return rows * mx4_tiles(cols) * (kMx4Tile / 2); }
static int64_t mx4_scale_bytes(int64_t rows, int64_t cols) { return rows * mx4_tiles(cols) * 4; }

static int mx4_call(const char* fn, const void* x, int32_t dtype, bool pack, int64_t rows, int64_t cols, int32_t transpose, const uint8_t* q,
                    const uint8_t* scale, void* stream) {
  EntryMark mark(fn);
  int rc;
  if ((rc = check_matrix(fn, rows, 0, kMaxRows, cols, kMaxCols)) || (rc = check_dtype(fn, pack ? "x" : "out", dtype))) return rc;
  if (transpose != 0 && transpose != 1) return fail(MA_ERR_INVALID_ARG, "%s: transpose %d is not 0 or 1", fn, transpose);
  // the packed matrix's sizes
  const int64_t pr = transpose ? cols : rows, pc = transpose ? rows : cols;
  if (pr * mx4_tiles(pc) * kMx4Tile > (dtype == MA_F32 ? kMaxElems / 2 : kMaxElems))
    return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements (2^35 fp32 ones)", fn);
  const Buf bufs[] = {{x, rows * cols * dt_size(dtype), (int)dt_size(dtype), !pack, false, pack ? "x" : "out"},
                      {q, mx4_q_bytes(pr, pc), 16, pack, false, "q"},
                      {scale, mx4_scale_bytes(pr, pc), 4, pack, false, "scale"}};
  if ((rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const Mx4Args a{pack ? x : nullptr, pack ? nullptr : const_cast<void*>(x), const_cast<uint8_t*>(q), const_cast<uint8_t*>(scale), rows, (int32_t)cols};
  ProfScope ps(MA_K_MX4, s);
  return done(pack ? launch_mx4_pack(a, dtype, transpose != 0, s) : launch_mx4_unpack(a, dtype, s), fn);
}

int ma_mx4_pack(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int32_t transpose, uint8_t* q, uint8_t* scale, void* stream) {
  return mx4_call("ma_mx4_pack", x, x_dtype, true, rows, cols, transpose, q, scale, stream);
}

int ma_mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, void* out, int32_t out_dtype, void* stream) {
  return mx4_call("ma_mx4_unpack", out, out_dtype, false, rows, cols, 0, q, scale, stream);
}

static int mx4_matmul_sizes(const char* fn, int64_t rows, int64_t outs, int64_t ins, int32_t x_bits) {
  int rc;
  if ((rc = check_size(fn, "rows", rows, 0, kMaxRows)) || (rc = check_size(fn, "outs", outs, 1, kMaxCols / 2)) ||
      (rc = check_size(fn, "ins", ins, 1, kMaxCols / 2)))
    return rc;
  if (x_bits != 4 && x_bits != 8) return fail(MA_ERR_UNSUPPORTED, "%s: x_bits %d is neither 4 nor 8", fn, x_bits);
  const int64_t pitch = mx4_tiles(ins) * kMx4Tile;
  if (rows * outs > kMaxElems || rows * pitch > kMaxElems || outs * pitch > kMaxElems)
    return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements", fn);
  return MA_OK;
}

static size_t mx4_workspace(int splits, int64_t rows, int64_t outs) {
  return splits > 1 ? (size_t)(splits * mx4_partial(rows, outs) * 4) : 0;
}

size_t ma_mx4_matmul_workspace_size(int64_t rows, int64_t outs, int64_t ins, int32_t x_bits) {
  if (mx4_matmul_sizes("ma_mx4_matmul_workspace_size", rows, outs, ins, x_bits)) return 0;
  return mx4_workspace(mx4_plan(rows, outs, ins, x_bits).splits, rows, outs);
}

int ma_test_mx4_matmul_plan(int64_t rows, int64_t outs, int64_t ins, int32_t x_bits, int32_t* edge, int32_t* splits) {
  const char* fn = "ma_test_mx4_matmul_plan";
  int rc;
  if ((rc = mx4_matmul_sizes(fn, rows, outs, ins, x_bits))) return rc;
  if (!edge || !splits) return fail(MA_ERR_INVALID_ARG, "%s: edge or splits is null", fn);
  const Mx4Plan plan = mx4_plan(rows, outs, ins, x_bits);
  *edge = plan.edge;
  *splits = plan.splits;
  return MA_OK;
}

int ma_mx4_matmul(const uint8_t* xq, const uint8_t* xscale, int32_t x_bits, int64_t rows, const uint8_t* wq, const uint8_t* wscale,
                  int64_t outs, int64_t ins, void* y, int32_t y_dtype, int32_t accumulate, void* workspace, size_t workspace_bytes,
                  void* stream) {
  const char* fn = "ma_mx4_matmul";
  EntryMark mark(fn);
  int rc;
  if ((rc = mx4_matmul_sizes(fn, rows, outs, ins, x_bits)) || (rc = check_dtype(fn, "y", y_dtype)) || (rc = check_flag(fn, accumulate))) return rc;
  const Mx4Plan plan = mx4_plan(rows, outs, ins, x_bits);
  const size_t need = mx4_workspace(plan.splits, rows, outs);
  const int64_t tiles = mx4_tiles(ins);
  const Buf bufs[] = {{xq, rows * tiles * (x_bits == 8 ? 128 : 64), 16, false, false, "xq"},
                      {xscale, rows * tiles * (x_bits == 8 ? 1 : 4), x_bits == 8 ? 1 : 4, false, false, "xscale"},
                      {wq, mx4_q_bytes(outs, ins), 16, false, false, "wq"},
                      {wscale, mx4_scale_bytes(outs, ins), 4, false, false, "wscale"},
                      {y, rows * outs * dt_size(y_dtype), (int)dt_size(y_dtype), true, false, "y"},
                      {workspace, (int64_t)need, 1, true, true, "the workspace"}};
  if ((rc = check_workspace(fn, workspace, workspace_bytes, need)) || (rc = check_buffers(fn, bufs))) return rc;
  if (rows == 0) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const Mx4MatmulArgs a{xq, xscale, wq, wscale, y, reinterpret_cast<float*>(workspace), rows, (int32_t)outs, (int32_t)ins, accumulate,
                        plan.edge, plan.splits, rows * outs * dt_size(y_dtype) > kStreamBytes};
  ProfScope ps(MA_K_MX4_MATMUL, s);
  return done(launch_mx4_matmul(a, x_bits, y_dtype, s), fn);
}

static int wgrad_sizes(const char* fn, int64_t tokens, int64_t outs, int64_t ins, int32_t dy_dtype) {
  int rc;
  if ((rc = check_size(fn, "tokens", tokens, 0, kMaxTokens)) || (rc = check_size(fn, "outs", outs, 1, kMaxCols / 2)) ||
      (rc = check_size(fn, "ins", ins, 1, kMaxCols / 2)) || (rc = check_dtype(fn, "dy", dy_dtype)))
    return rc;
  if (outs * ins > ((int64_t)1 << 31)) return fail(MA_ERR_INVALID_ARG, "%s: outs * ins beyond 2^31", fn);
  if (tokens * outs > kMaxElems || tokens * act_pitch(ins) > kMaxElems) return fail(MA_ERR_INVALID_ARG, "%s: more than 2^36 elements", fn);
  return MA_OK;
}

static size_t wgrad_workspace(int splits, int64_t outs, int64_t ins) {
  return splits > 1 ? (size_t)(splits * wgrad_partial(outs, ins) * 4) : 0;
}

size_t ma_act_weight_grad_workspace_size(int64_t tokens, int64_t outs, int64_t ins, int32_t dy_dtype) {
  if (wgrad_sizes("ma_act_weight_grad_workspace_size", tokens, outs, ins, dy_dtype)) return 0;
  return wgrad_workspace(wgrad_plan(tokens, outs, ins, dy_dtype).splits, outs, ins);
}

int ma_test_act_weight_grad_plan(int64_t tokens, int64_t outs, int64_t ins, int32_t dy_dtype, int32_t* edge, int32_t* splits) {
  const char* fn = "ma_test_act_weight_grad_plan";
  int rc;
  if ((rc = wgrad_sizes(fn, tokens, outs, ins, dy_dtype))) return rc;
  if (!edge || !splits) return fail(MA_ERR_INVALID_ARG, "%s: edge or splits is null", fn);
  const WgradPlan plan = wgrad_plan(tokens, outs, ins, dy_dtype);
  *edge = plan.big ? 256 : 128;
  *splits = plan.splits;
  return MA_OK;
}

int ma_act_weight_grad(const void* dy, int32_t dy_dtype, const uint8_t* q, const uint8_t* scale, int64_t tokens, int64_t outs, int64_t ins,
                       void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ma_act_weight_grad";
  EntryMark mark(fn);
  int rc;
  if ((rc = wgrad_sizes(fn, tokens, outs, ins, dy_dtype)) || (rc = check_dtype(fn, "grad", grad_dtype)) || (rc = check_flag(fn, accumulate))) return rc;
  const int64_t pitch = act_pitch(ins);
  const WgradPlan plan = wgrad_plan(tokens, outs, ins, dy_dtype);
  const size_t need = wgrad_workspace(plan.splits, outs, ins);
  const Buf bufs[] = {{dy, tokens * outs * dt_size(dy_dtype), (int)dt_size(dy_dtype), false, false, "dy"},
                      {q, tokens * pitch, 16, false, false, "q"},
                      {scale, tokens * (pitch / kActBlock), 1, false, false, "scale"},
                      {grad, outs * ins * dt_size(grad_dtype), (int)dt_size(grad_dtype), true, false, "grad"},
                      {workspace, (int64_t)need, 1, true, true, "the workspace"}};
  if ((rc = check_workspace(fn, workspace, workspace_bytes, need)) || (rc = check_buffers(fn, bufs))) return rc;
  if (tokens == 0 && accumulate) return MA_OK;
  if ((rc = check_stream_device(stream, "the stream"))) return rc;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const WgradArgs a{dy, q, scale, grad, reinterpret_cast<float*>(workspace), tokens, (int32_t)outs, (int32_t)ins, accumulate,
                    plan.splits, plan.big};
  ProfScope ps(MA_K_WEIGHT_GRAD, s);
  return done(launch_wgrad(a, dy_dtype, grad_dtype, s), fn);
}
