// Gated linear recurrence over [B][L][D]: forward, backward and single positions.
//
//   a_t = sigmoid(f_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) v_t,  y_t = h_t silu(g_t)
//
// A run of positions acts on the state as h -> A h + X, and two runs compose to
// (A2 A1, A2 X1 + X2): a scan. The same run acts on the gradient that flows
// towards the past, mu_t = a_t lam_t = a_t (r_t + mu_{t+1}) with r = dy silu(g), as
// mu -> A mu + R with the same A. All of it is memory bound: per element the
// forward reads v, f, g and writes y, the backward reads four and writes three.
//
// A workgroup owns 64 channels (16 lanes of 4: 128-byte row segments in bf16)
// and walks a chunk of the sequence in sub-blocks of 16 runs of R positions. A
// run is one thread's, held in registers; the 16 runs of a sub-block are joined
// through LDS by 64 threads, one per channel, which also carry the state.
// With enough samples and channels to fill the card one chunk is the whole
// sequence, and everything is read once. Otherwise a first launch leaves the
// (A, X[, R]) of each chunk, and every workgroup of the second folds those of
// the chunks before it (behind it for mu) in order: no waiting between
// workgroups and no order that varies.
//
// Measured, bf16 with a gate: 8 x 2048 x 768 forward 16 + 23 us (its four tensors once,
// 101 MB, take 19 us at the 5.3 TB/s of a large copy), backward 25 + 50 us and 5 for
// dbias; 1M x 256 backward 493 + 874 + 5 us, 4.3 TB/s of the 11 passes it makes. A
// single position of 16 x 768 states takes 3.7 us on the GPU.
#include "act.h"
#include "kernels_block.h"

namespace hy {

namespace {

typedef __bf16 bf16v4 __attribute__((ext_vector_type(4)));

// four channels of a row, as stored
template <typename T> struct Raw4;
template <> struct Raw4<float> { typedef float4 type; };
template <> struct Raw4<bf16> { typedef bf16v4 type; };

__device__ __forceinline__ void unpack(const float4& r, float (&v)[4]) {
  v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
}
__device__ __forceinline__ void unpack(const bf16v4& r, float (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = (float)r[k];
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
  bf16v4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = (bf16)v[k];
  *reinterpret_cast<bf16v4*>(p) = r;
}
__device__ __forceinline__ void load4f(const float* p, float (&v)[4]) { unpack(*reinterpret_cast<const float4*>(p), v); }

// A h + X for a run; A = 0 (a reset inside the run) cuts off whatever h holds
__device__ __forceinline__ float act_on(float A, float h, float X) { return A == 0.f ? X : fmaf(A, h, X); }

// The product of two runs' A: a reset in either cuts the joined run, whatever the other holds
__device__ __forceinline__ float join(float A, float B) { return A == 0.f || B == 0.f ? 0.f : A * B; }

// Rows of one thread: its run of R positions of sub-block sb
template <typename T, int R> struct Run {
  typename Raw4<T>::type x[R];
  __device__ __forceinline__ void load(const T* p, long long row, int t0, int tmax) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // rows behind the sequence repeat its last one; their values go unused
      const int t = t0 + i < tmax ? t0 + i : tmax;
      x[i] = *reinterpret_cast<const typename Raw4<T>::type*>(p + (long long)t * row);
    }
  }
};

// Per-workgroup position: channel tile, chunk, sample; the lane's channels
struct Where {
  int b, chunk, ch, sub, len;
  bool on;
};
__device__ __forceinline__ Where where(const GlrArgs& a, const GlrPlan& p) {
  Where w;
  long long id = blockIdx.x;
  const int ct = (int)(id % p.ctiles);
  id /= p.ctiles;
  w.chunk = (int)(id % p.C);
  w.b = (int)(id / p.C);
  w.sub = threadIdx.x >> 4;
  w.ch = ct * kGlrTile + (threadIdx.x & 15) * 4;
  w.on = w.ch < a.D;
  if (!w.on) w.ch = 0;  // idle lanes read channel 0 and write nothing
  w.len = a.L;
  if (a.lens) {
    const int n = a.lens[w.b];
    w.len = n < 0 ? 0 : (n < a.L ? n : a.L);
  }
  return w;
}

constexpr int kThreads = kGlrTile / 4 * kGlrSubs;  // 256
static_assert(kThreads == 256, "16 lanes of 4 channels, 16 runs");

// LDS rows of 64 channels plus 4: the 16 runs' rows start on different banks
constexpr int kLd = kGlrTile + 4;

// gates of one element: a, the input x = (1 - a) v; MASK: a = 1, x = 0 behind
// the length, a = 0 at a reset
template <bool MASK>
__device__ __forceinline__ void gate(float v, float f, float bias, bool live, bool rst, float& a, float& x) {
  float s, c;
  sigmoids(f + bias, s, c);
  a = s;
  x = c * v;
  if (MASK) {
    a = rst ? 0.f : a;
    a = live ? a : 1.f;
    x = live ? x : 0.f;
  }
}

template <bool MASK> __device__ __forceinline__ float step(float a, float h, float x) {
  return MASK ? act_on(a, h, x) : fmaf(a, h, x);
}

// State at the start of the workgroup's chunk for channel c = ct * 64 + tid of
// the 64 threads that carry it: h0 and the chunks before, in order. All 256
// threads fold a quarter of the chunks each; sm holds 3 x 64 float2.
__device__ __forceinline__ float chunk_carry(const float2* agg, int first, int last, int D, int ch, bool on,
                                             float start, float2* sm) {
  // quarter q of [first, last) (ascending: the fold runs first -> last)
  const int q = threadIdx.x >> 6, c = threadIdx.x & 63;
  const int n = last - first, per = (n + 3) >> 2;
  const int k0 = first + q * per, k1 = k0 + per < last ? k0 + per : last;
  float A = 1.f, X = 0.f;
  if (on) {
#pragma unroll 8
    for (int k = k0; k < k1; ++k) {
      const float2 e = agg[(size_t)k * D + ch];
      X = act_on(e.x, X, e.y);
      A = join(A, e.x);
    }
  }
  if (q) sm[(q - 1) * 64 + c] = make_float2(A, X);
  __syncthreads();
  float h = start;
  if (q == 0) {
    h = act_on(A, h, X);
    for (int i = 0; i < 3; ++i) h = act_on(sm[i * 64 + c].x, h, sm[i * 64 + c].y);
  }
  return h;
}

// ------------------------------------------------------------ first launch
// (A, X) of every chunk (and R, and of every sub-block, for the backward)
template <typename T, int R, bool BWD, bool GATE, bool MASK>
__global__ __launch_bounds__(256) void glr_agg_kernel(GlrArgs a, GlrPlan p) {
  __shared__ float sA[kGlrSubs][kLd], sX[kGlrSubs][kLd], sR[BWD ? kGlrSubs : 1][kLd];
  const Where w = where(a, p);
  const T* v = static_cast<const T*>(a.v) + w.b * a.vb + w.ch;
  const T* f = static_cast<const T*>(a.f) + w.b * a.fb + w.ch;
  const T* g = GATE ? static_cast<const T*>(a.g) + w.b * a.gb + w.ch : nullptr;
  const T* dy = BWD ? static_cast<const T*>(a.dy) + w.b * a.dyb + w.ch : nullptr;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.bias) load4f(a.bias + w.ch, bias);
  const int sb0 = w.chunk * p.nsb, sb1 = sb0 + p.nsb < p.nsb_total ? sb0 + p.nsb : p.nsb_total;
  const int tmax = a.L - 1;
  const int cch = (int)(blockIdx.x % p.ctiles) * kGlrTile + threadIdx.x;  // channel of a carrying thread
  const bool carries = threadIdx.x < kGlrTile && cch < a.D;
  float cA = 1.f, cX = 0.f, cR = 0.f;
  for (int sb = sb0; sb < sb1; ++sb) {
    const int t0 = sb * p.SB + w.sub * R;
    Run<T, R> rv, rf, rg, rd;
    rv.load(v, a.vr, t0, tmax);
    rf.load(f, a.fr, t0, tmax);
    if (BWD) {
      if (GATE) rg.load(g, a.gr, t0, tmax);
      rd.load(dy, a.dyr, t0, tmax);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads on their way before the first is used
    float A[4] = {1.f, 1.f, 1.f, 1.f}, X[4] = {0.f, 0.f, 0.f, 0.f}, Rr[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = t0 + i;
      const bool live = t < w.len;
      const bool rst = MASK && live && a.reset && a.reset[(long long)w.b * a.L + t];
      float vv[4], ff[4], gg[4], dd[4];
      unpack(rv.x[i], vv);
      unpack(rf.x[i], ff);
      if (BWD) {
        if (GATE) unpack(rg.x[i], gg);
        unpack(rd.x[i], dd);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float al, x;
        // without masks the rows behind L only exist in the last sub-block
        gate<true>(vv[k], ff[k], bias[k], live, rst, al, x);
        X[k] = step<MASK>(al, X[k], x);
        A[k] = MASK ? join(A[k], al) : A[k] * al;
        if (BWD) {
          const float r = live ? dd[k] * (GATE ? act_f<HYENA_ACT_SILU, T>(gg[k]) : 1.f) : 0.f;
          // prefix product times r_t; a reset at or before t keeps r from reaching the left end
          Rr[k] += MASK ? (A[k] == 0.f ? 0.f : A[k] * r) : A[k] * r;
        }
      }
    }
    const int col = (threadIdx.x & 15) * 4;
    *reinterpret_cast<float4*>(&sA[w.sub][col]) = make_float4(A[0], A[1], A[2], A[3]);
    *reinterpret_cast<float4*>(&sX[w.sub][col]) = make_float4(X[0], X[1], X[2], X[3]);
    if (BWD) *reinterpret_cast<float4*>(&sR[w.sub][col]) = make_float4(Rr[0], Rr[1], Rr[2], Rr[3]);
    __syncthreads();
    if (carries) {
      float bA = 1.f, bX = 0.f;
#pragma unroll
      for (int s = 0; s < kGlrSubs; ++s) {
        const float sa = sA[s][threadIdx.x], sx = sX[s][threadIdx.x];
        if (BWD) cR = act_on(cA, sR[s][threadIdx.x], cR);
        cX = act_on(sa, cX, sx);
        cA = join(cA, sa);
        bX = act_on(sa, bX, sx);
        bA = join(bA, sa);
      }
      if (BWD) a.sub[((size_t)w.b * p.nsb_total + sb) * a.D + cch] = make_float2(bA, bX);
    }
    __syncthreads();
  }
  if (carries) {
    const size_t at = ((size_t)w.b * p.C + w.chunk) * a.D + cch;
    a.agg[at] = make_float2(cA, cX);
    if (BWD) a.agg_r[at] = cR;
  }
}

// ----------------------------------------------------------------- forward
template <typename T, int R, bool GATE, bool MASK>
__global__ __launch_bounds__(256) void glr_fwd_kernel(GlrArgs a, GlrPlan p) {
  __shared__ float sA[kGlrSubs][kLd], sX[kGlrSubs][kLd], sH[kGlrSubs][kLd];
  __shared__ float2 sC[3 * 64];
  const Where w = where(a, p);
  const T* v = static_cast<const T*>(a.v) + w.b * a.vb + w.ch;
  const T* f = static_cast<const T*>(a.f) + w.b * a.fb + w.ch;
  const T* g = GATE ? static_cast<const T*>(a.g) + w.b * a.gb + w.ch : nullptr;
  T* y = static_cast<T*>(a.y) + w.b * a.yb + w.ch;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.bias) load4f(a.bias + w.ch, bias);
  const int sb0 = w.chunk * p.nsb, sb1 = sb0 + p.nsb < p.nsb_total ? sb0 + p.nsb : p.nsb_total;
  const int tmax = a.L - 1;
  const int cch = (int)(blockIdx.x % p.ctiles) * kGlrTile + (threadIdx.x & 63);
  const bool con = cch < a.D;
  const bool carries = threadIdx.x < kGlrTile && con;
  const int ylen = MASK && a.pad_zero ? a.L : w.len;  // rows of y to write
  float h = con && a.h0 ? a.h0[(size_t)w.b * a.D + cch] : 0.f;
  if (p.C > 1) h = chunk_carry(a.agg + (size_t)w.b * p.C * a.D, 0, w.chunk, a.D, cch, con, h, sC);
  for (int sb = sb0; sb < sb1; ++sb) {
    const int t0 = sb * p.SB + w.sub * R;
    Run<T, R> rv, rf, rg;
    rv.load(v, a.vr, t0, tmax);
    rf.load(f, a.fr, t0, tmax);
    if (GATE) rg.load(g, a.gr, t0, tmax);
    __builtin_amdgcn_sched_barrier(0);
    float al[R][4], x[R][4], A[4] = {1.f, 1.f, 1.f, 1.f}, X[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = t0 + i;
      const bool live = t < w.len;
      const bool rst = MASK && live && a.reset && a.reset[(long long)w.b * a.L + t];
      float vv[4], ff[4];
      unpack(rv.x[i], vv);
      unpack(rf.x[i], ff);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        gate<true>(vv[k], ff[k], bias[k], live, rst, al[i][k], x[i][k]);
        X[k] = step<MASK>(al[i][k], X[k], x[i][k]);
        A[k] = MASK ? join(A[k], al[i][k]) : A[k] * al[i][k];
      }
    }
    const int col = (threadIdx.x & 15) * 4;
    *reinterpret_cast<float4*>(&sA[w.sub][col]) = make_float4(A[0], A[1], A[2], A[3]);
    *reinterpret_cast<float4*>(&sX[w.sub][col]) = make_float4(X[0], X[1], X[2], X[3]);
    __syncthreads();
    if (threadIdx.x < kGlrTile) {
#pragma unroll
      for (int s = 0; s < kGlrSubs; ++s) {
        sH[s][threadIdx.x] = h;
        h = act_on(sA[s][threadIdx.x], h, sX[s][threadIdx.x]);
      }
    }
    __syncthreads();
    float hh[4];
    load4f(&sH[w.sub][col], hh);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = t0 + i;
      float gg[4], yy[4];
      if (GATE) unpack(rg.x[i], gg);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        hh[k] = step<MASK>(al[i][k], hh[k], x[i][k]);
        yy[k] = GATE ? hh[k] * act_f<HYENA_ACT_SILU, T>(gg[k]) : hh[k];
      }
      if (MASK && t >= w.len) yy[0] = yy[1] = yy[2] = yy[3] = 0.f;
      if (w.on && t < ylen) store4(y + (long long)t * a.yr, yy);
    }
  }
  if (carries && a.h_last && w.chunk == p.C - 1) a.h_last[(size_t)w.b * a.D + cch] = h;
}

// ---------------------------------------------------------------- backward
// Sub-blocks in reverse order; each needs the state before it, folded from the
// sub-block aggregates of the chunk on entry (kept in their X slots).
template <typename T, int R, bool GATE, bool MASK>
__global__ __launch_bounds__(256) void glr_bwd_kernel(GlrArgs a, GlrPlan p) {
  __shared__ float sA[kGlrSubs][kLd], sX[kGlrSubs][kLd], sR[kGlrSubs][kLd], sH[kGlrSubs][kLd], sM[kGlrSubs][kLd];
  __shared__ float2 sC[3 * 64];
  const Where w = where(a, p);
  const T* v = static_cast<const T*>(a.v) + w.b * a.vb + w.ch;
  const T* f = static_cast<const T*>(a.f) + w.b * a.fb + w.ch;
  const T* g = GATE ? static_cast<const T*>(a.g) + w.b * a.gb + w.ch : nullptr;
  const T* dy = static_cast<const T*>(a.dy) + w.b * a.dyb + w.ch;
  T* dv = static_cast<T*>(a.dv) + w.b * a.db + w.ch;
  T* df = static_cast<T*>(a.df) + w.b * a.db + w.ch;
  T* dg = GATE ? static_cast<T*>(a.dg) + w.b * a.db + w.ch : nullptr;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.bias) load4f(a.bias + w.ch, bias);
  const int sb0 = w.chunk * p.nsb, sb1 = sb0 + p.nsb < p.nsb_total ? sb0 + p.nsb : p.nsb_total;
  const int tmax = a.L - 1;
  const int cch = (int)(blockIdx.x % p.ctiles) * kGlrTile + (threadIdx.x & 63);
  const bool con = cch < a.D;
  const bool carries = threadIdx.x < kGlrTile && con;
  const size_t bd = (size_t)w.b * a.D + cch;
  // h before the chunk, mu behind it
  float h = con && a.h0 ? a.h0[bd] : 0.f;
  float mu = con && a.dh_last ? a.dh_last[bd] : 0.f;
  float2* subs = a.sub + (size_t)w.b * p.nsb_total * a.D;
  if (p.C > 1) {
    h = chunk_carry(a.agg + (size_t)w.b * p.C * a.D, 0, w.chunk, a.D, cch, con, h, sC);
    // mu -> A mu + R, chunks from the last down to the next: quarters of [chunk + 1, C)
    const int q = threadIdx.x >> 6, c = threadIdx.x & 63;
    const int first = w.chunk + 1, n = p.C - first, per = (n + 3) >> 2;
    const int k0 = first + q * per, k1 = k0 + per < p.C ? k0 + per : p.C;
    float A = 1.f, X = 0.f;
    const float2* ag = a.agg + (size_t)w.b * p.C * a.D;
    const float* ar = a.agg_r + (size_t)w.b * p.C * a.D;
    if (con) {
#pragma unroll 8
      for (int k = k1 - 1; k >= k0; --k) {
        const float e = ag[(size_t)k * a.D + cch].x;
        X = act_on(e, X, ar[(size_t)k * a.D + cch]);
        A = join(A, e);
      }
    }
    __syncthreads();  // the forward fold has read sC
    if (q) sC[(q - 1) * 64 + c] = make_float2(A, X);
    __syncthreads();
    if (q == 0) {
      for (int i = 2; i >= 0; --i) mu = act_on(sC[i * 64 + c].x, mu, sC[i * 64 + c].y);
      mu = act_on(A, mu, X);
    }
  }
  if (carries && p.nsb_total > 1) {
#pragma unroll 4
    for (int sb = sb0; sb < sb1; ++sb) {
      const float2 e = subs[(size_t)sb * a.D + cch];
      subs[(size_t)sb * a.D + cch].y = h;
      h = act_on(e.x, h, e.y);
    }
  }
  float db[4] = {0.f, 0.f, 0.f, 0.f};
  for (int sb = sb1 - 1; sb >= sb0; --sb) {
    const int t0 = sb * p.SB + w.sub * R;
    Run<T, R> rv, rf, rg, rd;
    rv.load(v, a.vr, t0, tmax);
    rf.load(f, a.fr, t0, tmax);
    if (GATE) rg.load(g, a.gr, t0, tmax);
    rd.load(dy, a.dyr, t0, tmax);
    if (carries && p.nsb_total > 1) h = subs[(size_t)sb * a.D + cch].y;
    __builtin_amdgcn_sched_barrier(0);
    // the run's (A, X, R); c = 1 - a, r = dy silu(g), q = dy silu'(g) for the second pass
    float al[R][4], cc[R][4], rr[R][4], qq[R][4];
    float A[4] = {1.f, 1.f, 1.f, 1.f}, X[4] = {0.f, 0.f, 0.f, 0.f}, Rr[4] = {0.f, 0.f, 0.f, 0.f};
    bool rst[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = t0 + i;
      const bool live = t < w.len;
      rst[i] = MASK && live && a.reset && a.reset[(long long)w.b * a.L + t];
      float vv[4], ff[4], gg[4], dd[4];
      unpack(rv.x[i], vv);
      unpack(rf.x[i], ff);
      if (GATE) unpack(rg.x[i], gg);
      unpack(rd.x[i], dd);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float s, c;
        sigmoids(ff[k] + bias[k], s, c);
        al[i][k] = live ? s : 1.f;
        cc[i][k] = live ? c : 0.f;
        const float x = live ? c * vv[k] : 0.f;
        float sg = 1.f, ds = 0.f;
        if (GATE) act_d<HYENA_ACT_SILU, T>(gg[k], sg, ds);
        rr[i][k] = live ? dd[k] * sg : 0.f;
        qq[i][k] = live ? dd[k] * ds : 0.f;
        const float ae = MASK && rst[i] ? 0.f : al[i][k];
        X[k] = step<MASK>(ae, X[k], x);
        A[k] = MASK ? join(A[k], ae) : A[k] * ae;
        Rr[k] += MASK ? (A[k] == 0.f ? 0.f : A[k] * rr[i][k]) : A[k] * rr[i][k];
      }
    }
    const int col = (threadIdx.x & 15) * 4;
    *reinterpret_cast<float4*>(&sA[w.sub][col]) = make_float4(A[0], A[1], A[2], A[3]);
    *reinterpret_cast<float4*>(&sX[w.sub][col]) = make_float4(X[0], X[1], X[2], X[3]);
    *reinterpret_cast<float4*>(&sR[w.sub][col]) = make_float4(Rr[0], Rr[1], Rr[2], Rr[3]);
    __syncthreads();
    if (threadIdx.x < kGlrTile) {
#pragma unroll
      for (int s = 0; s < kGlrSubs; ++s) {
        sH[s][threadIdx.x] = h;
        h = act_on(sA[s][threadIdx.x], h, sX[s][threadIdx.x]);
      }
#pragma unroll
      for (int s = kGlrSubs - 1; s >= 0; --s) {
        sM[s][threadIdx.x] = mu;
        mu = act_on(sA[s][threadIdx.x], mu, sR[s][threadIdx.x]);
      }
    }
    __syncthreads();
    float hp[R][4], mm[4];  // h_{t-1} (0 at a reset) of the run's positions
    {
      float hh[4];
      load4f(&sH[w.sub][col], hh);
      load4f(&sM[w.sub][col], mm);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float vv[4], o[4];
        unpack(rv.x[i], vv);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hp[i][k] = MASK && rst[i] ? 0.f : hh[k];
          // behind the length v may hold anything
          hh[k] = fmaf(al[i][k], hp[i][k], t0 + i < w.len ? cc[i][k] * vv[k] : 0.f);
          o[k] = qq[i][k] * hh[k];
        }
        const int t = t0 + i;
        if (GATE && w.on && t < a.L) {
          if (t >= w.len) o[0] = o[1] = o[2] = o[3] = 0.f;
          store4(dg + (long long)t * a.dr, o);
        }
      }
    }
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const int t = t0 + i;
      const bool live = t < w.len;
      float vv[4], ov[4], of[4];
      unpack(rv.x[i], vv);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lam = live ? rr[i][k] + mm[k] : 0.f;
        ov[k] = live ? cc[i][k] * lam : 0.f;
        of[k] = live ? al[i][k] * ov[k] * (hp[i][k] - vv[k]) : 0.f;
        db[k] += of[k];
        if (live) mm[k] = MASK && rst[i] ? 0.f : al[i][k] * lam;
      }
      if (w.on && t < a.L) {
        store4(dv + (long long)t * a.dr, ov);
        store4(df + (long long)t * a.dr, of);
      }
    }
  }
  if (carries && a.dh0 && w.chunk == 0) a.dh0[bd] = mu;
  if (a.dbias) {
    // the 16 runs' sums of the workgroup, in order
    __syncthreads();
    const int col = (threadIdx.x & 15) * 4;
    *reinterpret_cast<float4*>(&sA[w.sub][col]) = make_float4(db[0], db[1], db[2], db[3]);
    __syncthreads();
    if (carries) {
      float t = 0.f;
#pragma unroll
      for (int s = 0; s < kGlrSubs; ++s) t += sA[s][threadIdx.x];
      a.part[((size_t)w.b * p.C + w.chunk) * a.D + cch] = t;
    }
  }
}

// ------------------------------------------------------------ one position
// Rows that share a slot are consecutive positions of one sequence: the
// workgroup of the first such row walks the later ones in row order (the
// others leave at once), so no two workgroups touch one slot.
template <typename T>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStepArgs a) {
  const int r = blockIdx.y;
  const int ch = (blockIdx.x * 256 + threadIdx.x) * 4;
  int slot = r;
  bool later = false;  // a later row has the same slot
  if (a.slots) {
    slot = a.slots[r];
    if (slot < 0 || slot >= a.S) {
      const float none[4] = {0.f, 0.f, 0.f, 0.f};
      if (a.pad_zero && ch < a.D) store4(static_cast<T*>(a.y) + r * a.yr + ch, none);
      return;
    }
    // the whole workgroup reads the slots, 256 at a time
    bool before = false;
    for (int i = threadIdx.x; i < a.B; i += 256) {
      const bool same = a.slots[i] == slot;
      before |= same && i < r;
      later |= same && i > r;
    }
    if (__syncthreads_or(before)) return;
    later = __syncthreads_or(later);
  }
  if (ch >= a.D) return;
  const T* v = static_cast<const T*>(a.v) + ch;
  const T* f = static_cast<const T*>(a.f) + ch;
  const T* g = a.g ? static_cast<const T*>(a.g) + ch : nullptr;
  T* y = static_cast<T*>(a.y) + ch;
  float bias[4] = {0.f, 0.f, 0.f, 0.f}, h[4];
  if (a.bias) load4f(a.bias + ch, bias);
  load4f(a.state + (size_t)slot * a.D + ch, h);
  for (int i = r; i < a.B; ++i) {
    if (i > r && a.slots[i] != slot) continue;
    float vv[4], ff[4], yy[4];
    unpack(*reinterpret_cast<const typename Raw4<T>::type*>(v + i * a.vr), vv);
    unpack(*reinterpret_cast<const typename Raw4<T>::type*>(f + i * a.fr), ff);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float s, c;
      sigmoids(ff[k] + bias[k], s, c);
      h[k] = fmaf(s, h[k], c * vv[k]);
      yy[k] = h[k];
    }
    if (g) {
      float gg[4];
      unpack(*reinterpret_cast<const typename Raw4<T>::type*>(g + i * a.gr), gg);
#pragma unroll
      for (int k = 0; k < 4; ++k) yy[k] *= act_f<HYENA_ACT_SILU, T>(gg[k]);
    }
    store4(y + i * a.yr, yy);
    if (!later) break;
  }
  store4(a.state_out + (size_t)slot * a.D + ch, h);
}

template <typename T, int R, bool GATE, bool MASK>
hipError_t fwd_go(const GlrArgs& a, const GlrPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)p.ctiles * p.C * a.B);
  if (p.C > 1) glr_agg_kernel<T, R, false, GATE, MASK><<<grid, 256, 0, s>>>(a, p);
  glr_fwd_kernel<T, R, GATE, MASK><<<grid, 256, 0, s>>>(a, p);
  return hipGetLastError();
}

template <typename T, int R, bool GATE, bool MASK>
hipError_t bwd_go(const GlrArgs& a, const GlrPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)p.ctiles * p.C * a.B);
  if (p.nsb_total > 1) glr_agg_kernel<T, R, true, GATE, MASK><<<grid, 256, 0, s>>>(a, p);
  glr_bwd_kernel<T, R, GATE, MASK><<<grid, 256, 0, s>>>(a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dbias) return e;
  return colsum(a.part, a.dbias, (long long)a.B * p.C, a.D, a.D, s);
}

}  // namespace

constexpr int kRunFwdBf16 = 8, kRunFwdF32 = 4, kRunBwd = 4;

GlrPlan glr_plan(int B, int L, int D, bool bf16, bool bwd) {
  GlrPlan p{};
  p.R = bwd ? kRunBwd : (bf16 ? kRunFwdBf16 : kRunFwdF32);
  p.SB = p.R * kGlrSubs;
  p.nsb_total = (L + p.SB - 1) / p.SB;
  p.ctiles = (D + kGlrTile - 1) / kGlrTile;
  // About 1024 workgroups (four per CU); at most 256 chunks, whose aggregates every
  // workgroup folds. bf16 with a gate, us, with 512, 1024 and 2048 workgroups:
  // 8 x 2048 x 768 forward 51, 39, 39, backward 88, 81, 75; 65536 x 768 backward 325, 280, 299.
  // With at most 64, 128 and 256 chunks: 1M x 256 forward 990, 742, 683.
  const long long tiles = (long long)B * p.ctiles;
  long long C = (1024 + tiles - 1) / tiles;
  if (C > 256) C = 256;
  if (C > p.nsb_total) C = p.nsb_total;
  p.nsb = (int)((p.nsb_total + C - 1) / C);
  p.C = (p.nsb_total + p.nsb - 1) / p.nsb;
  return p;
}

hipError_t glr_fwd(const GlrArgs& a, const GlrPlan& p, bool bf, hipStream_t s) {
  const bool mask = a.reset || a.lens;
  const int sel = (bf ? 4 : 0) + (a.g ? 2 : 0) + (mask ? 1 : 0);
  switch (sel) {
    case 0: return fwd_go<float, kRunFwdF32, false, false>(a, p, s);
    case 1: return fwd_go<float, kRunFwdF32, false, true>(a, p, s);
    case 2: return fwd_go<float, kRunFwdF32, true, false>(a, p, s);
    case 3: return fwd_go<float, kRunFwdF32, true, true>(a, p, s);
    case 4: return fwd_go<bf16, kRunFwdBf16, false, false>(a, p, s);
    case 5: return fwd_go<bf16, kRunFwdBf16, false, true>(a, p, s);
    case 6: return fwd_go<bf16, kRunFwdBf16, true, false>(a, p, s);
    default: return fwd_go<bf16, kRunFwdBf16, true, true>(a, p, s);
  }
}

hipError_t glr_bwd(const GlrArgs& a, const GlrPlan& p, bool bf, hipStream_t s) {
  const bool mask = a.reset || a.lens;
  const int sel = (bf ? 4 : 0) + (a.g ? 2 : 0) + (mask ? 1 : 0);
  switch (sel) {
    case 0: return bwd_go<float, kRunBwd, false, false>(a, p, s);
    case 1: return bwd_go<float, kRunBwd, false, true>(a, p, s);
    case 2: return bwd_go<float, kRunBwd, true, false>(a, p, s);
    case 3: return bwd_go<float, kRunBwd, true, true>(a, p, s);
    case 4: return bwd_go<bf16, kRunBwd, false, false>(a, p, s);
    case 5: return bwd_go<bf16, kRunBwd, false, true>(a, p, s);
    case 6: return bwd_go<bf16, kRunBwd, true, false>(a, p, s);
    default: return bwd_go<bf16, kRunBwd, true, true>(a, p, s);
  }
}

hipError_t glr_step(const GlrStepArgs& a, bool bf, hipStream_t s) {
  const dim3 grid((a.D / 4 + 255) / 256, a.B);
  if (bf) glr_step_kernel<bf16><<<grid, 256, 0, s>>>(a);
  else glr_step_kernel<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace hy
