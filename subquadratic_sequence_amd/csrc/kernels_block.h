// Internal launcher interface between the C ABI (block_api.cpp) and the kernels
// of the operators around the long convolution.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace hy {

// ------------------------------------------------ gated linear recurrence
constexpr int kGlrTile = 64;  // channels per workgroup
constexpr int kGlrSubs = 16;  // time runs per sub-block (one per 16 lanes of a 256-thread workgroup)

// Split of the sequence: sub-blocks of SB positions, NSB sub-blocks per chunk,
// C chunks, one workgroup per (channel tile, chunk, sample).
struct GlrPlan {
  int R, SB, nsb_total, nsb, C, ctiles;
};
GlrPlan glr_plan(int B, int L, int D, bool bf16, bool bwd);

struct GlrArgs {
  int B, L, D;
  const void *v, *f, *g;
  long long vb, vr, fb, fr, gb, gr;
  const float *bias, *h0;
  const unsigned char* reset;
  const int* lens;
  bool pad_zero;  // write 0 to y at padding
  // forward
  void* y;
  long long yb, yr;
  float* h_last;
  // backward
  const void* dy;
  long long dyb, dyr;
  const float* dh_last;
  void *dv, *df, *dg;
  long long db, dr;
  float *dbias, *dh0;
  // workspace: chunk aggregates [B][C][D] (float2 (A, X); backward also R), sub-block
  // aggregates [B][nsb_total][D] float2 and bias partials [B][C][D] (backward)
  float2* agg;
  float* agg_r;
  float2* sub;
  float* part;
};
hipError_t glr_fwd(const GlrArgs& a, const GlrPlan& p, bool bf16, hipStream_t s);
hipError_t glr_bwd(const GlrArgs& a, const GlrPlan& p, bool bf16, hipStream_t s);

struct GlrStepArgs {
  int B, D, S;
  const void *v, *f, *g;
  long long vr, fr, gr;
  const float* bias;
  const int* slots;
  const float* state;
  float* state_out;
  void* y;
  long long yr;
  bool pad_zero;
};
hipError_t glr_step(const GlrStepArgs& a, bool bf16, hipStream_t s);

// ------------------------------------------------ group norm, channels last
struct GnArgs {
  int B, S, C, G, act;
  float eps;
  const void *x, *dy;
  const float *gamma, *beta;
  const int* lens;
  bool pad_zero;  // write 0 to y at padding
  void *y, *dx;
  float *mean, *rstd;           // forward outputs (may be null)
  const float *mean_in, *rstd_in;  // backward inputs
  float *dgamma, *dbeta;        // may be null
  float2* part;                 // [B][chunks][G]: (mean, M2) or the two group sums
  float* chan;                  // [rows][2][C] channel sums (backward; both gradients wanted or not)
};
// How the rows of a sample are dealt out.
//   rows form (S = 1, C / G a multiple of 8): `lanes` lanes of `nv` vectors of 8
//   channels per group, `slots` samples side by side, `per` samples per workgroup;
//   otherwise `slots` rows of C / vec threads, blocks of rows dealt to `chunks`
struct GnPlan {
  bool rows_form;
  int vec;               // channels of a thread (general form)
  int threads, slots, per, chunks;
  int lanes, nv;         // rows form
  int group_lanes;       // lanes that reduce one group (general form)
  int samples;           // samples a workgroup of the one-chunk backward takes
  long long chan_rows;   // rows of the channel sums
};
GnPlan gn_plan(int B, int S, int C, int G, bool bf16, bool bwd);
hipError_t gn_fwd(const GnArgs& a, const GnPlan& p, bool bf16, hipStream_t s);
hipError_t gn_bwd(const GnArgs& a, const GnPlan& p, bool bf16, hipStream_t s);

// out[d] = sum over rows of part [rows][ld], columns [0, D), in a fixed order
hipError_t colsum(const float* part, float* out, long long rows, int ld, int D, hipStream_t s);

// ---------------------------------------------- gated feed-forward block
struct FfnArgs {
  int M, D, F, act;
  const void *x, *w_in, *w_out, *dy;
  void *y, *dx, *dw_in, *dw_out;
  void *z, *dpq;  // workspace [M][F], [M][2F] (storage type)
  float* part;    // partial sums of split products
};
struct FfnProduct {
  int tile, splits;  // block tile (index), K splits
};
struct FfnPlan {
  FfnProduct gate, y, dz, dx, dw_in, dw_out;
  size_t part_floats;
};
FfnPlan ffn_plan(int M, int D, int F, bool bf16, bool bwd);
hipError_t ffn_fwd(const FfnArgs& a, const FfnPlan& p, bool bf16, hipStream_t s);
hipError_t ffn_bwd(const FfnArgs& a, const FfnPlan& p, bool bf16, hipStream_t s);

}  // namespace hy
