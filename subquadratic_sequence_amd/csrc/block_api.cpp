// C ABI of the operators around the long convolution: argument validation,
// workspace layout and launch sequences. Every check runs on the host before
// the first HIP call.
#include "../../include/hyena.h"

#include <math.h>
#include <stdint.h>

#include "common.h"
#include "kernels_block.h"

using hy::align_up;

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool aligned16(const void* p) { return p != nullptr && aligned(p, 16); }
bool aligned16_or_null(const void* p) { return aligned(p, 16); }
bool dtype_ok(int dtype) { return dtype == HYENA_F32 || dtype == HYENA_BF16; }
size_t esize(int dtype) { return dtype == HYENA_BF16 ? 2 : 4; }
// elements per 16 bytes: row strides are multiples of it
int vec_of(int dtype) { return dtype == HYENA_BF16 ? 8 : 4; }

int device_ok() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) return HYENA_ERR_HIP;
  return HYENA_OK;
}

// ------------------------------------------------ gated linear recurrence
constexpr long long kMaxElems = 1LL << 40;

bool glr_shape_ok(int B, int L, int D) {
  if (B < 1 || B > (1 << 20) || L < 1 || L > (1 << 24) || D < 8 || D > (1 << 16) || D % 8) return false;
  if ((long long)B * D >= (1LL << 31)) return false;
  return (long long)B * D <= (kMaxElems - 1) / L;
}

// strides of an input: not negative, whole 16-byte steps; bounded so that every
// offset fits 63 bits
bool in_strides_ok(long long batch, long long row, int dtype) {
  const int v = vec_of(dtype);
  const long long cap = 1LL << 38;
  return batch >= 0 && row >= 0 && batch < cap && row < cap && batch % v == 0 && row % v == 0;
}
// strides of an output: rows and samples apart
bool out_strides_ok(long long batch, long long row, int B, int L, int D, int dtype) {
  if (!in_strides_ok(batch, row, dtype)) return false;
  if (L > 1 && row < D) return false;
  return B == 1 || batch >= (long long)(L - 1) * row + D;
}

struct GlrWs {
  size_t agg, agg_r, sub, part, total;
};
GlrWs glr_ws(int B, int L, int D, int dtype, bool bwd) {
  const hy::GlrPlan p = hy::glr_plan(B, L, D, dtype == HYENA_BF16, bwd);
  GlrWs w{};
  size_t off = 0;
  const size_t chunks = (size_t)B * p.C * D;
  w.agg = off;
  if (p.C > 1 || bwd) off = align_up(off + chunks * 8, kAlign);
  if (bwd) {
    w.agg_r = off;
    off = align_up(off + chunks * 4, kAlign);
    w.sub = off;
    off = align_up(off + (size_t)B * p.nsb_total * D * 8, kAlign);
    w.part = off;
    off = align_up(off + chunks * 4, kAlign);
  }
  w.total = off ? off : kAlign;
  return w;
}

// the checks of the inputs that both directions share
int glr_inputs_check(const hyena_glr_inputs* in) {
  if (in == nullptr || !dtype_ok(in->dtype)) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(in->v) || !aligned16(in->f)) return HYENA_ERR_INVALID_ARG;
  if (!aligned16_or_null(in->g) || !aligned16_or_null(in->bias) || !aligned16_or_null(in->h0) || !aligned(in->lens, 4))
    return HYENA_ERR_INVALID_ARG;
  if (in->B < 1) return HYENA_ERR_INVALID_ARG;
  if (!glr_shape_ok(in->B, in->L, in->D)) return HYENA_ERR_UNSUPPORTED;
  if (!in_strides_ok(in->v_batch, in->v_row, in->dtype) || !in_strides_ok(in->f_batch, in->f_row, in->dtype))
    return HYENA_ERR_INVALID_ARG;
  if (in->g && !in_strides_ok(in->g_batch, in->g_row, in->dtype)) return HYENA_ERR_INVALID_ARG;
  return HYENA_OK;
}

hy::GlrArgs glr_args(const hyena_glr_inputs* in) {
  hy::GlrArgs a{};
  a.B = in->B;
  a.L = in->L;
  a.D = in->D;
  a.v = in->v;
  a.f = in->f;
  a.g = in->g;
  a.vb = in->v_batch;
  a.vr = in->v_row;
  a.fb = in->f_batch;
  a.fr = in->f_row;
  a.gb = in->g_batch;
  a.gr = in->g_row;
  a.bias = in->bias;
  a.h0 = in->h0;
  a.reset = in->reset;
  a.lens = in->lens;
  a.pad_zero = in->pad_zero != 0;
  return a;
}

// ------------------------------------------------ group norm, channels last
bool act_ok(int act) { return act == HYENA_ACT_NONE || act == HYENA_ACT_SILU || act == HYENA_ACT_GELU; }

bool gn_shape_ok(int B, int S, int C, int G) {
  if (B < 1 || B > (1 << 24) || S < 1 || S > (1 << 24) || C < 8 || C > 8192 || C % 8) return false;
  if (G < 1 || G > C || C % G) return false;
  if ((long long)B * C >= (1LL << 31)) return false;
  return (long long)B * C <= (kMaxElems - 1) / S;
}

struct GnWs {
  size_t part, chan, total;
};
GnWs gn_ws(int B, int S, int C, int G, int dtype, bool bwd) {
  const hy::GnPlan p = hy::gn_plan(B, S, C, G, dtype == HYENA_BF16, bwd);
  GnWs w{};
  size_t off = 0;
  w.part = off;
  if (p.chunks > 1) off = align_up(off + (size_t)B * p.chunks * G * 8, kAlign);
  w.chan = off;
  if (bwd) off = align_up(off + (size_t)p.chan_rows * 2 * C * 4, kAlign);
  w.total = off ? off : kAlign;
  return w;
}

// ---------------------------------------------- gated feed-forward block
bool ffn_shape_ok(int M, int D, int F) {
  if (M < 1 || M > (1 << 24)) return false;
  return D >= 8 && D <= (1 << 16) && D % 8 == 0 && F >= 8 && F <= (1 << 16) && F % 8 == 0;
}

struct FfnWs {
  size_t z, dpq, part, total;
};
FfnWs ffn_ws(int M, int D, int F, int dtype, bool bwd) {
  const hy::FfnPlan p = hy::ffn_plan(M, D, F, dtype == HYENA_BF16, bwd);
  const size_t e = esize(dtype);
  FfnWs w{};
  size_t off = align_up((size_t)M * F * e, kAlign);
  w.dpq = off;
  if (bwd) off = align_up(off + (size_t)M * 2 * F * e, kAlign);
  w.part = off;
  off = align_up(off + p.part_floats * 4, kAlign);
  w.total = off;
  return w;
}

}  // namespace

extern "C" {

size_t hyena_glr_workspace_bytes(int B, int L, int D, int dtype) {
  if (!glr_shape_ok(B, L, D) || !dtype_ok(dtype)) return 0;
  return glr_ws(B, L, D, dtype, false).total;
}

size_t hyena_glr_bwd_workspace_bytes(int B, int L, int D, int dtype) {
  if (!glr_shape_ok(B, L, D) || !dtype_ok(dtype)) return 0;
  return glr_ws(B, L, D, dtype, true).total;
}

int hyena_glr_fwd(const hyena_glr_inputs* in, void* y, long long y_batch, long long y_row, float* h_last, void* ws,
                  size_t ws_bytes, hipStream_t stream) {
  const int st = glr_inputs_check(in);
  if (st != HYENA_OK) return st;
  if (!aligned16(y) || !aligned16_or_null(h_last) || !aligned16(ws)) return HYENA_ERR_INVALID_ARG;
  if (!out_strides_ok(y_batch, y_row, in->B, in->L, in->D, in->dtype)) return HYENA_ERR_INVALID_ARG;
  const GlrWs w = glr_ws(in->B, in->L, in->D, in->dtype, false);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  const bool bf = in->dtype == HYENA_BF16;
  hy::GlrArgs a = glr_args(in);
  a.y = y;
  a.yb = y_batch;
  a.yr = y_row;
  a.h_last = h_last;
  a.agg = reinterpret_cast<float2*>(static_cast<char*>(ws) + w.agg);
  HY_CHECK_HIP(hy::glr_fwd(a, hy::glr_plan(in->B, in->L, in->D, bf, false), bf, stream));
  return HYENA_OK;
}

int hyena_glr_bwd(const hyena_glr_inputs* in, const void* dy, long long dy_batch, long long dy_row,
                  const float* dh_last, void* dv, void* df, void* dg, long long d_batch, long long d_row,
                  float* dbias, float* dh0, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = glr_inputs_check(in);
  if (st != HYENA_OK) return st;
  if (!aligned16(dy) || !aligned16(dv) || !aligned16(df) || !aligned16(ws)) return HYENA_ERR_INVALID_ARG;
  if ((in->g == nullptr) != (dg == nullptr) || !aligned16_or_null(dg)) return HYENA_ERR_INVALID_ARG;
  if (!aligned16_or_null(dh_last) || !aligned16_or_null(dbias) || !aligned16_or_null(dh0)) return HYENA_ERR_INVALID_ARG;
  if (!in_strides_ok(dy_batch, dy_row, in->dtype)) return HYENA_ERR_INVALID_ARG;
  if (!out_strides_ok(d_batch, d_row, in->B, in->L, in->D, in->dtype)) return HYENA_ERR_INVALID_ARG;
  const GlrWs w = glr_ws(in->B, in->L, in->D, in->dtype, true);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  const bool bf = in->dtype == HYENA_BF16;
  char* wb = static_cast<char*>(ws);
  hy::GlrArgs a = glr_args(in);
  a.dy = dy;
  a.dyb = dy_batch;
  a.dyr = dy_row;
  a.dh_last = dh_last;
  a.dv = dv;
  a.df = df;
  a.dg = dg;
  a.db = d_batch;
  a.dr = d_row;
  a.dbias = dbias;
  a.dh0 = dh0;
  a.agg = reinterpret_cast<float2*>(wb + w.agg);
  a.agg_r = reinterpret_cast<float*>(wb + w.agg_r);
  a.sub = reinterpret_cast<float2*>(wb + w.sub);
  a.part = reinterpret_cast<float*>(wb + w.part);
  HY_CHECK_HIP(hy::glr_bwd(a, hy::glr_plan(in->B, in->L, in->D, bf, true), bf, stream));
  return HYENA_OK;
}

int hyena_glr_step(int B, int D, int S, int dtype, const void* v, long long v_row, const void* f, long long f_row,
                   const void* g, long long g_row, const float* bias, const int* slots, const float* state,
                   float* state_out, void* y, long long y_row, int pad_zero, hipStream_t stream) {
  if (!dtype_ok(dtype) || B < 1 || S < 1) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(v) || !aligned16(f) || !aligned16(state) || !aligned16(state_out) || !aligned16(y))
    return HYENA_ERR_INVALID_ARG;
  if (!aligned16_or_null(g) || !aligned16_or_null(bias) || !aligned(slots, 4)) return HYENA_ERR_INVALID_ARG;
  if (B > 8192 || S > (1 << 24) || D < 8 || D > (1 << 16) || D % 8) return HYENA_ERR_UNSUPPORTED;
  if (slots == nullptr && S < B) return HYENA_ERR_INVALID_ARG;
  if (!in_strides_ok(0, v_row, dtype) || !in_strides_ok(0, f_row, dtype) || (g && !in_strides_ok(0, g_row, dtype)))
    return HYENA_ERR_INVALID_ARG;
  if (!out_strides_ok(0, y_row, 1, B, D, dtype)) return HYENA_ERR_INVALID_ARG;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  hy::GlrStepArgs a{B, D, S, v, f, g, v_row, f_row, g_row, bias, slots, state, state_out, y, y_row, pad_zero != 0};
  HY_CHECK_HIP(hy::glr_step(a, dtype == HYENA_BF16, stream));
  return HYENA_OK;
}

size_t hyena_group_norm_workspace_bytes(int B, int S, int C, int G, int dtype) {
  if (!gn_shape_ok(B, S, C, G) || !dtype_ok(dtype)) return 0;
  return gn_ws(B, S, C, G, dtype, false).total;
}

size_t hyena_group_norm_bwd_workspace_bytes(int B, int S, int C, int G, int dtype) {
  if (!gn_shape_ok(B, S, C, G) || !dtype_ok(dtype)) return 0;
  return gn_ws(B, S, C, G, dtype, true).total;
}

int hyena_group_norm_fwd(int B, int S, int C, int G, int dtype, int act, float eps, const void* x, const float* gamma,
                         const float* beta, const int* lens, int pad_zero, void* y, float* mean, float* rstd,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || B < 1) return HYENA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !isfinite(eps)) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(ws)) return HYENA_ERR_INVALID_ARG;
  if (!aligned16_or_null(gamma) || !aligned16_or_null(beta) || !aligned16_or_null(mean) || !aligned16_or_null(rstd) ||
      !aligned(lens, 4))
    return HYENA_ERR_INVALID_ARG;
  if (!gn_shape_ok(B, S, C, G)) return HYENA_ERR_UNSUPPORTED;
  const GnWs w = gn_ws(B, S, C, G, dtype, false);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  hy::GnArgs a{};
  a.B = B;
  a.S = S;
  a.C = C;
  a.G = G;
  a.act = act;
  a.eps = eps;
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.lens = lens;
  a.pad_zero = pad_zero != 0;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.part = reinterpret_cast<float2*>(static_cast<char*>(ws) + w.part);
  HY_CHECK_HIP(hy::gn_fwd(a, hy::gn_plan(B, S, C, G, dtype == HYENA_BF16, false), dtype == HYENA_BF16, stream));
  return HYENA_OK;
}

int hyena_group_norm_bwd(int B, int S, int C, int G, int dtype, int act, const void* x, const void* dy,
                         const float* gamma, const float* beta, const int* lens, const float* mean, const float* rstd,
                         void* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || B < 1) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(mean) || !aligned16(rstd) || !aligned16(ws))
    return HYENA_ERR_INVALID_ARG;
  if (!aligned16_or_null(gamma) || !aligned16_or_null(beta) || !aligned16_or_null(dgamma) ||
      !aligned16_or_null(dbeta) || !aligned(lens, 4))
    return HYENA_ERR_INVALID_ARG;
  if (!gn_shape_ok(B, S, C, G)) return HYENA_ERR_UNSUPPORTED;
  const GnWs w = gn_ws(B, S, C, G, dtype, true);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  char* wb = static_cast<char*>(ws);
  hy::GnArgs a{};
  a.B = B;
  a.S = S;
  a.C = C;
  a.G = G;
  a.act = act;
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.lens = lens;
  a.dx = dx;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = reinterpret_cast<float2*>(wb + w.part);
  a.chan = reinterpret_cast<float*>(wb + w.chan);
  HY_CHECK_HIP(hy::gn_bwd(a, hy::gn_plan(B, S, C, G, dtype == HYENA_BF16, true), dtype == HYENA_BF16, stream));
  return HYENA_OK;
}

size_t hyena_ffn_workspace_bytes(int M, int D, int F, int dtype) {
  if (!ffn_shape_ok(M, D, F) || !dtype_ok(dtype)) return 0;
  return ffn_ws(M, D, F, dtype, false).total;
}

size_t hyena_ffn_bwd_workspace_bytes(int M, int D, int F, int dtype) {
  if (!ffn_shape_ok(M, D, F) || !dtype_ok(dtype)) return 0;
  return ffn_ws(M, D, F, dtype, true).total;
}

int hyena_ffn_fwd(int M, int D, int F, int dtype, int act, const void* x, const void* w_in, const void* w_out, void* y,
                  void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || M < 1) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_in) || !aligned16(w_out) || !aligned16(y) || !aligned16(ws))
    return HYENA_ERR_INVALID_ARG;
  if (!ffn_shape_ok(M, D, F)) return HYENA_ERR_UNSUPPORTED;
  const FfnWs w = ffn_ws(M, D, F, dtype, false);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  const bool bf = dtype == HYENA_BF16;
  char* wb = static_cast<char*>(ws);
  hy::FfnArgs a{};
  a.M = M;
  a.D = D;
  a.F = F;
  a.act = act;
  a.x = x;
  a.w_in = w_in;
  a.w_out = w_out;
  a.y = y;
  a.z = wb + w.z;
  a.part = reinterpret_cast<float*>(wb + w.part);
  HY_CHECK_HIP(hy::ffn_fwd(a, hy::ffn_plan(M, D, F, bf, false), bf, stream));
  return HYENA_OK;
}

int hyena_ffn_bwd(int M, int D, int F, int dtype, int act, const void* x, const void* w_in, const void* w_out,
                  const void* dy, void* dx, void* dw_in, void* dw_out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || M < 1) return HYENA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_in) || !aligned16(w_out) || !aligned16(dy) || !aligned16(dx) ||
      !aligned16(dw_in) || !aligned16(dw_out) || !aligned16(ws))
    return HYENA_ERR_INVALID_ARG;
  if (!ffn_shape_ok(M, D, F)) return HYENA_ERR_UNSUPPORTED;
  const FfnWs w = ffn_ws(M, D, F, dtype, true);
  if (ws_bytes < w.total) return HYENA_ERR_WORKSPACE;
  if (device_ok() != HYENA_OK) return HYENA_ERR_HIP;
  const bool bf = dtype == HYENA_BF16;
  char* wb = static_cast<char*>(ws);
  hy::FfnArgs a{};
  a.M = M;
  a.D = D;
  a.F = F;
  a.act = act;
  a.x = x;
  a.w_in = w_in;
  a.w_out = w_out;
  a.dy = dy;
  a.dx = dx;
  a.dw_in = dw_in;
  a.dw_out = dw_out;
  a.z = wb + w.z;
  a.dpq = wb + w.dpq;
  a.part = reinterpret_cast<float*>(wb + w.part);
  HY_CHECK_HIP(hy::ffn_bwd(a, hy::ffn_plan(M, D, F, bf, true), bf, stream));
  return HYENA_OK;
}

}  // extern "C"
