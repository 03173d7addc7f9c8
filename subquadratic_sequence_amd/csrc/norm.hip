// Group norm with an activation, channels last: x [B][S][C], statistics over the
// S positions of a sample and the C / G channels of a group.
//
//   n = gamma xh + beta, xh = (x - mean) rstd, y = act(n)
//   dn = dy act'(n), dx = rstd (gamma dn - m1 - xh m2), m1 = avg(gamma dn), m2 = avg(gamma dn xh)
//
// Memory bound: the forward must read x and write y, the backward read x and dy
// and write dx. A thread owns 8 neighbouring channels and walks rows, whatever
// the groups are; groups only meet where the threads' sums do, in LDS. Variances
// come from deviations: a block of rows in registers gives its own mean and
// M2 = sum (x - mean)^2, and (n, mean, M2) triples join exactly as
//   mean = m_a + d n_b / n,  M2 = M2_a + M2_b + d^2 n_a n_b / n,  d = m_b - m_a.
//
//  * Samples of one row (S = 1: a norm per token) whose groups are whole
//    vectors: a group is a few lanes of one wave, everything stays in
//    registers and moves once.
//  * Many samples: one workgroup per sample reads it twice, the second time
//    from cache.
//  * Few large samples: chunks of rows, one launch for the sums of every chunk,
//    a second in which each workgroup joins the chunks' sums of its sample
//    (a few kB from L2) and writes its rows.
#include "act.h"
#include "kernels_block.h"
#include "vec8.h"

namespace hy {

namespace {

struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(Moments a, Moments b) {
  const float n = a.n + b.n;
  const float w = n > 0.f ? b.n / n : 0.f, d = b.mean - a.mean;
  return Moments{n, fmaf(d, w, a.mean), fmaf(d * d, a.n * w, a.m2 + b.m2)};
}
__device__ __forceinline__ Moments shfl_down(Moments m, int o, int w) {
  return Moments{__shfl_down(m.n, o, w), __shfl_down(m.mean, o, w), __shfl_down(m.m2, o, w)};
}

__device__ __forceinline__ int live_rows(const int* lens, int b, int S) {
  if (!lens) return S;
  const int n = lens[b];
  return n < 0 ? 0 : (n < S ? n : S);
}

// Rows of a chunk that thread row-slot `slot` of `slots` walks: slot, slot + slots, ...
__device__ __forceinline__ int slot_rows(int rows, int slot, int slots) {
  return rows > slot ? (rows - slot + slots - 1) / slots : 0;
}

constexpr int kU = 4;  // rows of a thread in flight

// gamma and beta of 8 channels (1 and 0 without them)
__device__ __forceinline__ void affine(const float* gamma, const float* beta, int c, float (&ga)[8], float (&be)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    ga[k] = 1.f;
    be[k] = 0.f;
  }
  if (gamma) ld8(gamma + c, ga);
  if (beta) ld8(beta + c, be);
}

// A workgroup's place in the general form
struct Place {
  int b, chunk, slot, c, r0, rows;  // rows: live rows of the chunk
  bool on;
};
__device__ __forceinline__ Place place(const GnArgs& a, const GnPlan& p, int b, int chunk) {
  Place w;
  w.chunk = chunk;
  w.b = b;
  const int nv = a.C >> 3;
  w.slot = threadIdx.x / nv;
  w.c = (threadIdx.x - w.slot * nv) * 8;
  w.on = w.slot < p.slots;
  w.r0 = w.chunk * p.per;
  const int left = live_rows(a.lens, w.b, a.S) - w.r0;
  w.rows = left < 0 ? 0 : (left < p.per ? left : p.per);
  return w;
}

// Joins entries [0, n) of every group, `lanes` lanes to a group; emit(g, m) runs
// in one lane of each.
template <typename Entry, typename Emit>
__device__ __forceinline__ void join_groups(int G, int n, int lanes, Entry entry, Emit emit) {
  const int l = threadIdx.x & (lanes - 1);
  for (int g = threadIdx.x / lanes; g < G; g += blockDim.x / lanes) {
    Moments m{0.f, 0.f, 0.f};
    for (int i = l; i < n; i += lanes) m = join(m, entry(g, i));
    for (int o = lanes >> 1; o; o >>= 1) m = join(m, shfl_down(m, o, lanes));
    if (l == 0) emit(g, m);
  }
}
template <typename Entry, typename Emit>
__device__ __forceinline__ void sum_groups(int G, int n, int lanes, Entry entry, Emit emit) {
  const int l = threadIdx.x & (lanes - 1);
  for (int g = threadIdx.x / lanes; g < G; g += blockDim.x / lanes) {
    float2 m = make_float2(0.f, 0.f);
    for (int i = l; i < n; i += lanes) {
      const float2 e = entry(g, i);
      m.x += e.x;
      m.y += e.y;
    }
    for (int o = lanes >> 1; o; o >>= 1) {
      m.x += __shfl_down(m.x, o, lanes);
      m.y += __shfl_down(m.y, o, lanes);
    }
    if (l == 0) emit(g, m);
  }
}

// ------------------------------------------------------------- general form
// Moments of a chunk's groups: out(g, (mean, M2)) for every group.
// sm: [slots][C] float2
template <typename T, typename Emit>
__device__ __forceinline__ void chunk_moments(const GnArgs& a, const GnPlan& p, const Place& w, float2* sm, Emit emit) {
  if (w.on) {
    float n = 0.f, mean[8], m2[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) mean[k] = m2[k] = 0.f;
    const T* x = static_cast<const T*>(a.x) + ((size_t)w.b * a.S + w.r0) * a.C + w.c;
    for (int r = w.slot; r < w.rows; r += kU * p.slots) {
      float v[kU][8];
      bool ok[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ru = r + u * p.slots;
        ok[u] = ru < w.rows;
        ld8(x + (size_t)(ok[u] ? ru : r) * a.C, v[u]);
      }
      float m = 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u) m += ok[u] ? 1.f : 0.f;
      const float im = 1.f / m, wn = m / (n + m), wd = n * wn;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int u = 0; u < kU; ++u) s += ok[u] ? v[u][k] : 0.f;
        const float bm = s * im;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float d = ok[u] ? v[u][k] - bm : 0.f;
          q = fmaf(d, d, q);
        }
        const float d = bm - mean[k];
        mean[k] = fmaf(d, wn, mean[k]);
        m2[k] += fmaf(d * d, wd, q);
      }
      n += m;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sm[(size_t)w.slot * a.C + w.c + k] = make_float2(mean[k], m2[k]);
  }
  __syncthreads();
  const int cg = a.C / a.G;
  join_groups(
      a.G, cg * p.slots, p.group_lanes,
      [&](int g, int i) {
        const int s = i / cg, c = i - s * cg;
        const float2 e = sm[(size_t)s * a.C + g * cg + c];
        return Moments{(float)slot_rows(w.rows, s, p.slots), e.x, e.y};
      },
      emit);
}

// y of the chunk's rows with stat(g) = (mean, rstd)
template <typename T, int ACT>
__device__ __forceinline__ void chunk_apply(const GnArgs& a, const GnPlan& p, const Place& w, const float2* stat) {
  if (!w.on) return;
  const int cg = a.C / a.G;
  float ga[8], be[8], mean[8];
  affine(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 st = stat[(w.c + k) / cg];
    mean[k] = st.x;
    ga[k] *= st.y;
  }
  const size_t at = ((size_t)w.b * a.S + w.r0) * a.C + w.c;
  const T* x = static_cast<const T*>(a.x) + at;
  T* y = static_cast<T*>(a.y) + at;
  const int left = a.S - w.r0, all = !a.pad_zero ? w.rows : (left < p.per ? left : p.per);  // rows of y to write
  for (int r = w.slot; r < all; r += kU * p.slots) {
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ru = r + u * p.slots;
      ld8(x + (size_t)(ru < all ? ru : r) * a.C, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ru = r + u * p.slots;
      if (ru < all) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[u][k] = ru < w.rows ? act_f<ACT>(fmaf(v[u][k] - mean[k], ga[k], be[k])) : 0.f;
        st8(y + (size_t)ru * a.C, v[u]);
      }
    }
  }
}

__device__ __forceinline__ float2 stat_of(const GnArgs& a, int b, int g, Moments m) {
  const float var = m.n > 0.f ? m.m2 / m.n : 0.f;
  const float2 st = make_float2(m.mean, 1.f / sqrtf(var + a.eps));
  if (a.mean) a.mean[(size_t)b * a.G + g] = st.x;
  if (a.rstd) a.rstd[(size_t)b * a.G + g] = st.y;
  return st;
}

extern __shared__ float2 gn_smem[];

template <typename T> __global__ __launch_bounds__(1024) void gn_moments_kernel(GnArgs a, GnPlan p) {
  const Place w = place(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  float2* out = a.part + ((size_t)w.b * p.chunks + w.chunk) * a.G;
  chunk_moments<T>(a, p, w, gn_smem, [&](int g, Moments m) { out[g] = make_float2(m.mean, m.m2); });
}

// second launch (chunks > 1) or the whole of it (FUSED: one chunk per sample)
template <typename T, int ACT, bool FUSED> __global__ __launch_bounds__(1024) void gn_apply_kernel(GnArgs a, GnPlan p) {
  const Place w = place(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  const int cg = a.C / a.G;
  float2* stat = gn_smem;
  if (FUSED) {
    stat = gn_smem + (size_t)p.slots * a.C;
    chunk_moments<T>(a, p, w, gn_smem, [&](int g, Moments m) { stat[g] = stat_of(a, w.b, g, m); });
  } else {
    const float2* part = a.part + (size_t)w.b * p.chunks * a.G;
    const int live = live_rows(a.lens, w.b, a.S);
    GnArgs first = a;
    if (w.chunk) first.mean = first.rstd = nullptr;  // one workgroup per sample writes the statistics
    join_groups(
        a.G, p.chunks, p.group_lanes,
        [&](int g, int i) {
          const int left = live - i * p.per;
          const int rows = left < 0 ? 0 : (left < p.per ? left : p.per);
          const float2 e = part[(size_t)i * a.G + g];
          return Moments{(float)rows * cg, e.x, e.y};
        },
        [&](int g, Moments m) { stat[g] = stat_of(first, w.b, g, m); });
  }
  __syncthreads();
  chunk_apply<T, ACT>(a, p, w, stat);
}

// Sums of a chunk: per channel (sum dn xh, sum dn) to `chan`, per group of the
// gamma-weighted (sum gamma dn, sum gamma dn xh) to emit. `add`: on top of what chan holds.
template <typename T, int ACT, typename Emit>
__device__ __forceinline__ void chunk_sums(const GnArgs& a, const GnPlan& p, const Place& w, float2* sm, float* chan,
                                           bool add, Emit emit) {
  const int cg = a.C / a.G;
  if (w.on) {
    float ga[8], be[8], mean[8], rs[8], s1[8], s2[8];
    affine(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const size_t g = (size_t)w.b * a.G + (w.c + k) / cg;
      mean[k] = a.mean_in[g];
      rs[k] = a.rstd_in[g];
      s1[k] = s2[k] = 0.f;
    }
    const size_t at = ((size_t)w.b * a.S + w.r0) * a.C + w.c;
    const T* x = static_cast<const T*>(a.x) + at;
    const T* dy = static_cast<const T*>(a.dy) + at;
    for (int r = w.slot; r < w.rows; r += kU * p.slots) {
      float v[kU][8], d[kU][8];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ru = r + u * p.slots;
        ld8(x + (size_t)(ru < w.rows ? ru : r) * a.C, v[u]);
        ld8(dy + (size_t)(ru < w.rows ? ru : r) * a.C, d[u]);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (r + u * p.slots < w.rows) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = (v[u][k] - mean[k]) * rs[k];
            float y, da;
            act_d<ACT>(fmaf(xh, ga[k], be[k]), y, da);
            const float dn = d[u][k] * da;
            s1[k] += dn;
            s2[k] = fmaf(dn, xh, s2[k]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sm[(size_t)w.slot * a.C + w.c + k] = make_float2(s1[k], s2[k]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
    float2 t = sm[c];
    for (int s = 1; s < p.slots; ++s) {
      const float2 e = sm[(size_t)s * a.C + c];
      t.x += e.x;
      t.y += e.y;
    }
    if (a.dgamma || a.dbeta) {
      // (a thread meets the same channels for every sample of its workgroup)
      chan[c] = add ? chan[c] + t.y : t.y;
      chan[a.C + c] = add ? chan[a.C + c] + t.x : t.x;
    }
    const float ga = a.gamma ? a.gamma[c] : 1.f;
    sm[c] = make_float2(t.x * ga, t.y * ga);
  }
  __syncthreads();
  sum_groups(a.G, cg, p.group_lanes, [&](int g, int i) { return sm[g * cg + i]; }, emit);
}

// dx of the chunk's rows; avg[g] = (m1, m2)
template <typename T, int ACT>
__device__ __forceinline__ void chunk_dx(const GnArgs& a, const GnPlan& p, const Place& w, const float2* avg) {
  if (!w.on) return;
  const int cg = a.C / a.G;
  float ga[8], be[8], mean[8], rs[8], m1[8], m2[8];
  affine(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int g = (w.c + k) / cg;
    mean[k] = a.mean_in[(size_t)w.b * a.G + g];
    rs[k] = a.rstd_in[(size_t)w.b * a.G + g];
    m1[k] = avg[g].x;
    m2[k] = avg[g].y;
  }
  const size_t at = ((size_t)w.b * a.S + w.r0) * a.C + w.c;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* dy = static_cast<const T*>(a.dy) + at;
  T* dx = static_cast<T*>(a.dx) + at;
  const int all = a.S - w.r0 < p.per ? a.S - w.r0 : p.per;  // padded rows of the chunk get zeros
  for (int r = w.slot; r < all; r += kU * p.slots) {
    float v[kU][8], d[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ru = r + u * p.slots;
      ld8(x + (size_t)(ru < all ? ru : r) * a.C, v[u]);
      ld8(dy + (size_t)(ru < all ? ru : r) * a.C, d[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int ru = r + u * p.slots;
      if (ru < all) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = (v[u][k] - mean[k]) * rs[k];
          float y, da;
          act_d<ACT>(fmaf(xh, ga[k], be[k]), y, da);
          const float t = fmaf(d[u][k] * da, ga[k], -m1[k]);
          v[u][k] = ru < w.rows ? rs[k] * fmaf(-xh, m2[k], t) : 0.f;
        }
        st8(dx + (size_t)ru * a.C, v[u]);
      }
    }
  }
}

template <typename T, int ACT> __global__ __launch_bounds__(1024) void gn_sums_kernel(GnArgs a, GnPlan p) {
  const Place w = place(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  float2* out = a.part + ((size_t)w.b * p.chunks + w.chunk) * a.G;
  float* chan = a.chan + (size_t)blockIdx.x * 2 * a.C;
  chunk_sums<T, ACT>(a, p, w, gn_smem, chan, false, [&](int g, float2 m) { out[g] = m; });
}

// second launch (chunks > 1): dx of one chunk
template <typename T, int ACT> __global__ __launch_bounds__(1024) void gn_dx_kernel(GnArgs a, GnPlan p) {
  const Place w = place(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  const int live = live_rows(a.lens, w.b, a.S);
  const float inv = live ? 1.f / ((float)live * (float)(a.C / a.G)) : 0.f;
  float2* avg = gn_smem;
  const float2* part = a.part + (size_t)w.b * p.chunks * a.G;
  sum_groups(a.G, p.chunks, p.group_lanes, [&](int g, int i) { return part[(size_t)i * a.G + g]; },
             [&](int g, float2 m) { avg[g] = make_float2(m.x * inv, m.y * inv); });
  __syncthreads();
  chunk_dx<T, ACT>(a, p, w, avg);
}

// one chunk per sample: a workgroup takes `samples` of them one after the other
template <typename T, int ACT> __global__ __launch_bounds__(1024) void gn_bwd_kernel(GnArgs a, GnPlan p) {
  float2* avg = gn_smem + (size_t)p.slots * a.C;
  float* chan = a.chan + (size_t)blockIdx.x * 2 * a.C;
  const int b0 = blockIdx.x * p.samples, b1 = b0 + p.samples < a.B ? b0 + p.samples : a.B;
  for (int b = b0; b < b1; ++b) {
    const Place w = place(a, p, b, 0);
    const int live = live_rows(a.lens, b, a.S);
    const float inv = live ? 1.f / ((float)live * (float)(a.C / a.G)) : 0.f;
    chunk_sums<T, ACT>(a, p, w, gn_smem, chan, b > b0,
                       [&](int g, float2 m) { avg[g] = make_float2(m.x * inv, m.y * inv); });
    __syncthreads();
    chunk_dx<T, ACT>(a, p, w, avg);
  }
}

// ---------------------------------------------------------------- rows form
// One row per sample: lanes [0, LANES) of a group hold NV vectors each.
template <int NV> struct RowPlace {
  int slot, g, c0, nvec;  // first channel of the lane's first vector; vectors of the group
  int step;               // channels between its vectors
  bool on, has[NV];
};
template <int NV> __device__ __forceinline__ RowPlace<NV> row_place(const GnArgs& a, const GnPlan& p) {
  RowPlace<NV> w;
  const int tps = a.G * p.lanes;
  w.slot = threadIdx.x / tps;
  const int t = threadIdx.x - w.slot * tps;
  w.on = w.slot < p.slots;
  w.g = t / p.lanes;
  const int l = t & (p.lanes - 1);
  const int cg = a.C / a.G;
  w.nvec = cg >> 3;
  w.c0 = w.g * cg + l * 8;
  w.step = p.lanes * 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) w.has[i] = l + i * p.lanes < w.nvec;
  return w;
}
__device__ __forceinline__ float lane_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <typename T, int ACT, int NV> __global__ __launch_bounds__(1024) void gn_rows_kernel(GnArgs a, GnPlan p) {
  const RowPlace<NV> w = row_place<NV>(a, p);
  if (!w.on) return;
  const float inv = 1.f / (float)(a.C / a.G);
  const long long b0 = (long long)blockIdx.x * p.per, b1 = b0 + p.per < a.B ? b0 + p.per : a.B;
  for (long long b = b0 + w.slot; b < b1; b += p.slots) {
    float v[NV][8];
    const T* x = static_cast<const T*>(a.x) + b * a.C + w.c0;
    const bool live = live_rows(a.lens, (int)b, 1) == 1;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i]) ld8(x + i * w.step, v[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i])
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[i][k];
    const float mean = lane_sum(s, p.lanes) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i])
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[i][k] -= mean;
          q = fmaf(v[i][k], v[i][k], q);
        }
    const float var = lane_sum(q, p.lanes) * inv;
    const float rstd = 1.f / sqrtf((live ? var : 0.f) + a.eps);
    if ((w.c0 - w.g * (a.C / a.G)) == 0) {
      if (a.mean) a.mean[b * a.G + w.g] = live ? mean : 0.f;
      if (a.rstd) a.rstd[b * a.G + w.g] = rstd;
    }
    if (!live && !a.pad_zero) continue;
    T* y = static_cast<T*>(a.y) + b * a.C + w.c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i]) {
        float ga[8], be[8];
        affine(a.gamma, a.beta, w.c0 + i * w.step, ga, be);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = live ? act_f<ACT>(fmaf(v[i][k] * rstd, ga[k], be[k])) : 0.f;
        st8(y + i * w.step, v[i]);
      }
  }
}

template <typename T, int ACT, int NV> __global__ __launch_bounds__(1024) void gn_rows_dx_kernel(GnArgs a, GnPlan p) {
  const RowPlace<NV> w = row_place<NV>(a, p);
  const float inv = 1.f / (float)(a.C / a.G);
  const long long b0 = (long long)blockIdx.x * p.per, b1 = b0 + p.per < a.B ? b0 + p.per : a.B;
  float s1[NV][8], s2[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s1[i][k] = s2[i][k] = 0.f;
  if (w.on) {
    for (long long b = b0 + w.slot; b < b1; b += p.slots) {
      const bool live = live_rows(a.lens, (int)b, 1) == 1;
      const T* x = static_cast<const T*>(a.x) + b * a.C + w.c0;
      const T* dy = static_cast<const T*>(a.dy) + b * a.C + w.c0;
      T* dx = static_cast<T*>(a.dx) + b * a.C + w.c0;
      const float mean = a.mean_in[b * a.G + w.g], rstd = a.rstd_in[b * a.G + w.g];
      float v[NV][8], d[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (w.has[i]) {
          ld8(x + i * w.step, v[i]);
          ld8(dy + i * w.step, d[i]);
        }
      float t1 = 0.f, t2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (w.has[i]) {
          float ga[8], be[8];
          affine(a.gamma, a.beta, w.c0 + i * w.step, ga, be);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = (v[i][k] - mean) * rstd;
            float y, da;
            act_d<ACT>(fmaf(xh, ga[k], be[k]), y, da);
            const float dn = live ? d[i][k] * da : 0.f;
            s1[i][k] += dn;
            if (live) s2[i][k] = fmaf(dn, xh, s2[i][k]);
            v[i][k] = xh;
            d[i][k] = dn * ga[k];
            t1 += d[i][k];
            t2 = fmaf(d[i][k], xh, t2);
          }
        }
      const float m1 = lane_sum(t1, p.lanes) * inv, m2 = lane_sum(t2, p.lanes) * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (w.has[i]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = live ? rstd * fmaf(-v[i][k], m2, d[i][k] - m1) : 0.f;
          st8(dx + i * w.step, v[i]);
        }
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  // the slots' channel sums, in order
  if (w.on)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i])
#pragma unroll
        for (int k = 0; k < 8; ++k)
          gn_smem[(size_t)w.slot * a.C + w.c0 + i * w.step + k] = make_float2(s1[i][k], s2[i][k]);
  __syncthreads();
  float* chan = a.chan + (size_t)blockIdx.x * 2 * a.C;
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
    float2 t = gn_smem[c];
    for (int s = 1; s < p.slots; ++s) {
      const float2 e = gn_smem[(size_t)s * a.C + c];
      t.x += e.x;
      t.y += e.y;
    }
    chan[c] = t.y;
    chan[a.C + c] = t.x;
  }
}

// out[d] = sum over rows of part [rows][ld]: 64 columns per workgroup, the rows
// dealt to 16 threads per column, their sums joined in order
__global__ __launch_bounds__(1024) void colsum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                      long long rows, int ld, int D) {
  __shared__ float sm[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  float t = 0.f;
  if (c < D) {
#pragma unroll 8
    for (long long r = q; r < rows; r += 16) t += part[r * ld + c];
  }
  sm[q][threadIdx.x & 63] = t;
  __syncthreads();
  if (q == 0 && c < D) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sm[i][threadIdx.x];
    out[c] = t;
  }
}

template <typename F> hipError_t launch(F kernel, unsigned grid, int threads, size_t smem, const GnArgs& a,
                                        const GnPlan& p, hipStream_t s) {
  if (smem > (64u << 10)) {  // rare: C or G in the thousands
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != hipSuccess) return e;
  }
  kernel<<<grid, threads, smem, s>>>(a, p);
  return hipGetLastError();
}

size_t slots_bytes(const GnArgs& a, const GnPlan& p) { return (size_t)p.slots * a.C * sizeof(float2); }

template <typename T, int ACT> hipError_t rows_go(const GnArgs& a, const GnPlan& p, bool bwd, hipStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.B + p.per - 1) / p.per);
  const size_t sm = bwd && (a.dgamma || a.dbeta) ? slots_bytes(a, p) : 0;
#define HY_GN_ROWS(NV)                                                                    \
  if (p.nv <= NV)                                                                         \
    return bwd ? launch(gn_rows_dx_kernel<T, ACT, NV>, grid, p.threads, sm, a, p, s)      \
               : launch(gn_rows_kernel<T, ACT, NV>, grid, p.threads, sm, a, p, s);
  HY_GN_ROWS(1)
  HY_GN_ROWS(2)
  HY_GN_ROWS(3)
  HY_GN_ROWS(4)
  HY_GN_ROWS(8)
  HY_GN_ROWS(16)
#undef HY_GN_ROWS
  return hipErrorInvalidValue;
}

template <typename T, int ACT> hipError_t fwd_go(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  if (p.rows_form) return rows_go<T, ACT>(a, p, false, s);
  const unsigned grid = (unsigned)((long long)a.B * p.chunks);
  const size_t sums = slots_bytes(a, p), stat = (size_t)a.G * sizeof(float2);
  if (p.chunks == 1) return launch(gn_apply_kernel<T, ACT, true>, grid, p.threads, sums + stat, a, p, s);
  const hipError_t e = launch(gn_moments_kernel<T>, grid, p.threads, sums, a, p, s);
  if (e != hipSuccess) return e;
  return launch(gn_apply_kernel<T, ACT, false>, grid, p.threads, stat, a, p, s);
}

template <typename T, int ACT> hipError_t bwd_go(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * p.chunks);
  const size_t sums = slots_bytes(a, p), avg = (size_t)a.G * sizeof(float2);
  hipError_t e;
  if (p.rows_form) {
    e = rows_go<T, ACT>(a, p, true, s);
  } else if (p.chunks == 1) {
    e = launch(gn_bwd_kernel<T, ACT>, (unsigned)p.chan_rows, p.threads, sums + avg, a, p, s);
  } else {
    e = launch(gn_sums_kernel<T, ACT>, grid, p.threads, sums, a, p, s);
    if (e == hipSuccess) e = launch(gn_dx_kernel<T, ACT>, grid, p.threads, avg, a, p, s);
  }
  if (e == hipSuccess && a.dgamma) e = colsum(a.chan, a.dgamma, p.chan_rows, 2 * a.C, a.C, s);
  if (e == hipSuccess && a.dbeta) e = colsum(a.chan + a.C, a.dbeta, p.chan_rows, 2 * a.C, a.C, s);
  return e;
}

}  // namespace

hipError_t colsum(const float* part, float* out, long long rows, int ld, int D, hipStream_t s) {
  colsum_kernel<<<(D + 63) / 64, 1024, 0, s>>>(part, out, rows, ld, D);
  return hipGetLastError();
}

GnPlan gn_plan(int B, int S, int C, int G) {
  GnPlan p{};
  const int cg = C / G, nv = C / 8;
  if (S == 1 && cg % 8 == 0) {
    // lanes per group: the power of two (at most a wave) with the fewest idle
    // lane-vectors, at most 16 vectors a lane; the widest among equals
    p.rows_form = true;
    const int q = cg / 8;
    int best = -1;
    for (int l = 64; l >= 1; l >>= 1) {
      if (l > q && l > 1) continue;
      const int n = (q + l - 1) / l;
      if (n > 16) continue;
      const int waste = n * l - q;
      if (best < 0 || waste < best) {
        best = waste;
        p.lanes = l;
        p.nv = n;
      }
    }
    const int tps = G * p.lanes;
    p.slots = tps >= 256 ? 1 : 256 / tps;
    if ((long long)p.slots * C > 8192) p.slots = 8192 / C;  // the backward's channel sums take 64 KB of LDS at most
    p.threads = (tps * p.slots + 63) / 64 * 64;
    // about 2048 workgroups
    long long per = (B + 2047LL) / 2048;
    per = (per + p.slots - 1) / p.slots * p.slots;
    p.per = (int)per;
    p.chunks = 1;
    p.chan_rows = (B + per - 1) / per;
    return p;
  }
  p.slots = nv >= 256 ? 1 : 256 / nv;
  p.threads = (nv * p.slots + 63) / 64 * 64;
  // about 1024 workgroups, chunks of whole register blocks of rows
  long long chunks = B >= 512 ? 1 : (1024 + B - 1) / B;
  const int unit = p.slots * kU;
  long long per = (S + chunks - 1) / chunks;
  per = (per + unit - 1) / unit * unit;
  p.per = (int)(per < S ? per : S);
  p.chunks = (S + p.per - 1) / p.per;
  const int n = p.chunks > 1 ? p.chunks : cg * p.slots;
  p.group_lanes = 1;
  while (p.group_lanes < 64 && p.group_lanes * 2 <= n) p.group_lanes *= 2;
  // the backward's channel sums: one row per workgroup, at most 2048 of them
  p.samples = p.chunks == 1 ? (B + 2047) / 2048 : 1;
  p.chan_rows = p.chunks == 1 ? (B + p.samples - 1) / p.samples : (long long)B * p.chunks;
  return p;
}

#define HY_GN_DISPATCH(fn)                                                     \
  switch ((bf ? 3 : 0) + a.act) {                                              \
    case 0: return fn<float, HYENA_ACT_NONE>(a, p, s);                         \
    case 1: return fn<float, HYENA_ACT_SILU>(a, p, s);                         \
    case 2: return fn<float, HYENA_ACT_GELU>(a, p, s);                         \
    case 3: return fn<bf16, HYENA_ACT_NONE>(a, p, s);                          \
    case 4: return fn<bf16, HYENA_ACT_SILU>(a, p, s);                          \
    default: return fn<bf16, HYENA_ACT_GELU>(a, p, s);                         \
  }
hipError_t gn_fwd(const GnArgs& a, const GnPlan& p, bool bf, hipStream_t s) { HY_GN_DISPATCH(fwd_go) }
hipError_t gn_bwd(const GnArgs& a, const GnPlan& p, bool bf, hipStream_t s) { HY_GN_DISPATCH(bwd_go) }
#undef HY_GN_DISPATCH

}  // namespace hy
