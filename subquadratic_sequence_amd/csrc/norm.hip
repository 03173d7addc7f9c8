// Group norm with an activation, channels last: x [B][S][C], statistics over the
// S positions of a sample and the C / G channels of a group.
//
//   n = gamma xh + beta, xh = (x - mean) rstd, y = act(n)
//   dn = dy act'(n), dx = rstd (gamma dn - m1 - xh m2), m1 = avg(gamma dn), m2 = avg(gamma dn xh)
//
// Memory bound: the forward must read x and write y, the backward read x and dy
// and write dx. A thread owns 16 bytes of neighbouring channels (fp32 rows of more
// than 4096 channels: 32) and walks rows, whatever the groups are; groups only meet
// where the threads' sums do, in LDS. Variances come from deviations: a block of rows
// in registers gives its own mean and M2 = sum (x - mean)^2, two of them join as mean =
// m_a + d n_b / n, M2 = M2_a + M2_b + d^2 n_a n_b / n with d = m_b - m_a, and many as
// mean = sum n_i m_i / n, then M2 = sum M2_i + n_i (m_i - mean)^2 (two short sums
// instead of a chain of divisions).
//
//  * Samples of one row (S = 1: a norm per token) whose groups are whole
//    vectors: a group is a few lanes of one wave, everything stays in
//    registers and moves once.
//  * Many samples: one workgroup per sample reads it twice, the second time
//    from cache.
//  * Few large samples: chunks of rows, one launch for the sums of every chunk,
//    a second in which each workgroup joins the chunks' sums of its sample
//    (a few kB from L2) and writes its rows.
//
// Measured: fp32, 8 x 64^2 x 384 forward 11 + 21 us (x and y once, 101 MB, take 19 us at the
// 5.3 TB/s of a large copy); 2 x 64^3 x 128 backward 103 + 128 + 5 us, 5.8 TB/s of its five
// passes (three are the floor: 152 us). bf16, 16384 single rows of 768: 12 us (floor 9.5).
#include "act.h"
#include "kernels_block.h"
#include "vec8.h"

namespace hy {

namespace {

struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ int live_rows(const int* lens, int b, int S) {
  if (!lens) return S;
  const int n = lens[b];
  return n < 0 ? 0 : (n < S ? n : S);
}

// The rows of a sample are dealt to its chunks in blocks of `unit` (slots rows side by
// side, N of them one after the other per thread): block i goes to chunk i mod
// chunks, so that the workgroups of a launch read neighbouring memory at any time
// (each with a long stretch of its own, they would meet on the same HBM channels).
// Rows of a slot (of all slots, for slot < 0) in a chunk, of `rows` in the sample:
__device__ __forceinline__ int dealt(int rows, int chunk, int chunks, int unit, int slot, int slots) {
  const int full = rows / unit, rest = rows - full * unit;
  const int mine = full > chunk ? (full - chunk + chunks - 1) / chunks : 0;
  int n = mine * (slot < 0 ? unit : unit / slots);
  if (full % chunks == chunk) n += slot < 0 ? rest : (rest > slot ? (rest - slot + slots - 1) / slots : 0);
  return n;
}

// V channels of a row
template <typename T, int V> struct Raw;
template <> struct Raw<float, 4> { float4 a; };
template <> struct Raw<float, 8> { float4 a, b; };
template <> struct Raw<bf16, 8> { bf16v8 a; };
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float (&v)[4]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
}
__device__ __forceinline__ void unpack(const Raw<float, 8>& r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void unpack(const Raw<bf16, 8>& r, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = (float)r.a[k];
}
__device__ __forceinline__ void put(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T> __device__ __forceinline__ void put(T* p, const float (&v)[8]) { st8(p, v); }

// Rows of a thread in flight (64 to 128 bytes of each tensor)
constexpr int rows_ahead(int v) { return v == 4 ? 8 : 4; }

// gamma and beta of V channels (1 and 0 without them)
template <int V>
__device__ __forceinline__ void affine(const float* gamma, const float* beta, int c, float (&ga)[V], float (&be)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    ga[k] = 1.f;
    be[k] = 0.f;
  }
  if (gamma) unpack(*reinterpret_cast<const Raw<float, V>*>(gamma + c), ga);
  if (beta) unpack(*reinterpret_cast<const Raw<float, V>*>(beta + c), be);
}

// A workgroup's place in the general form
struct Place {
  int b, chunk, slot, c, rows;  // rows: live rows of the sample
  unsigned off;                 // elements from a block's first row to the thread's first
  size_t at, step;              // elements to the sample, between a thread's rows
  bool on;
};
template <int V>
__device__ __forceinline__ Place place(const GnArgs& a, const GnPlan& p, int b, int chunk) {
  Place w;
  w.chunk = chunk;
  w.b = b;
  const int nv = a.C / V;
  w.slot = threadIdx.x / nv;
  w.c = (threadIdx.x - w.slot * nv) * V;
  w.on = w.slot < p.slots;
  w.rows = live_rows(a.lens, w.b, a.S);
  w.off = (unsigned)(w.slot * a.C + w.c);
  w.at = (size_t)w.b * a.S * a.C;
  w.step = (size_t)p.slots * a.C;
  return w;
}
// Walks a thread's rows below `rows`, a block at a time: load(raw, at, n) and
// use(raw, at, n), at the elements from the sample to the block, n how many of the
// block's N rows per thread there are. The next block is on its way while one is
// used. A block's address is uniform: a load costs no vector address of its own.
// LAST_FIRST: from the last block to the first, for a second pass over what a first
// launch has read: its end is still in the last-level cache.
template <int N, bool LAST_FIRST, typename R, typename Load, typename Use>
__device__ __forceinline__ void walk(const GnPlan& p, const Place& w, int rows, int C, Load load, Use use) {
  const int unit = p.slots * N, full = rows / unit, rest = rows - full * unit;
  const int mine = full > w.chunk ? (full - w.chunk + p.chunks - 1) / p.chunks : 0;
  auto at = [&](int i) {
    const int k = LAST_FIRST ? mine - 1 - i : i;
    return (size_t)(w.chunk + (long long)k * p.chunks) * unit * C;
  };
  R a, b;
  int i = 0;
  if (mine > 0) {
    // behind the last block the loads repeat it: without branches around them the
    // compiler's count of loads in flight stays exact
    load(a, at(0), N);
    for (;;) {
      const int j = i + 1;
      load(b, at(j < mine ? j : i), N);
      __builtin_amdgcn_sched_barrier(0);  // (the compiler would move the loads down to their use)
      use(a, at(i), N);
      if (j >= mine) break;
      i = j + 1;
      load(a, at(i < mine ? i : j), N);
      __builtin_amdgcn_sched_barrier(0);
      use(b, at(j), N);
      if (i >= mine) break;
    }
  }
  if (full % p.chunks == w.chunk && w.slot < rest) {
    const int n = (rest - w.slot + p.slots - 1) / p.slots;
    const size_t end = (size_t)full * unit * C;
    load(a, end, n);
    use(a, end, n);
  }
}
template <typename T, int V, int N> struct Block {
  Raw<T, V> r[N];
};
template <typename T, int V, int N> struct Block2 {
  Raw<T, V> x[N], d[N];
};
// row u of a walk's body: rows that are not there repeat the first
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> fetch(const T* sample, const Place& w, size_t at, int u, int n) {
  return *reinterpret_cast<const Raw<T, V>*>(sample + at + (u < n ? u : 0) * w.step + w.off);
}
// zeros to the thread's rows in [rows, S)
template <int N, int V, typename T>
__device__ __forceinline__ void pad(const GnArgs& a, const GnPlan& p, const Place& w, T* out) {
  float zero[V];
#pragma unroll
  for (int k = 0; k < V; ++k) zero[k] = 0.f;
  if (w.rows == a.S) return;
  const int unit = p.slots * N;
  for (int i = w.chunk; (long long)i * unit < a.S; i += p.chunks)
    for (int u = 0; u < N; ++u) {
      const int r = i * unit + u * p.slots + w.slot;
      if (r >= w.rows && r < a.S) put(out + (size_t)r * a.C + w.c, zero);
    }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
// Joins entries [0, n) of every group, `lanes` lanes to a group; emit(g, m) runs
// in one lane of each.
template <typename Entry, typename Emit>
__device__ __forceinline__ void join_groups(int G, int n, int lanes, Entry entry, Emit emit) {
  const int l = threadIdx.x & (lanes - 1);
  for (int g = threadIdx.x / lanes; g < G; g += blockDim.x / lanes) {
    float cnt = 0.f, sum = 0.f, m2 = 0.f;
#pragma unroll 4
    for (int i = l; i < n; i += lanes) {
      const Moments e = entry(g, i);
      cnt += e.n;
      sum = fmaf(e.n, e.mean, sum);
    }
    cnt = lanes_sum(cnt, lanes);
    sum = lanes_sum(sum, lanes);
    const float mean = cnt > 0.f ? sum / cnt : 0.f;
#pragma unroll 4
    for (int i = l; i < n; i += lanes) {
      const Moments e = entry(g, i);
      const float d = e.n > 0.f ? e.mean - mean : 0.f;
      m2 += fmaf(e.n * d, d, e.m2);
    }
    m2 = lanes_sum(m2, lanes);
    if (l == 0) emit(g, Moments{cnt, mean, m2});
  }
}
template <typename Entry, typename Emit>
__device__ __forceinline__ void sum_groups(int G, int n, int lanes, Entry entry, Emit emit) {
  const int l = threadIdx.x & (lanes - 1);
  for (int g = threadIdx.x / lanes; g < G; g += blockDim.x / lanes) {
    float2 m = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = l; i < n; i += lanes) {
      const float2 e = entry(g, i);
      m.x += e.x;
      m.y += e.y;
    }
    m.x = lanes_sum(m.x, lanes);
    m.y = lanes_sum(m.y, lanes);
    if (l == 0) emit(g, m);
  }
}

// ------------------------------------------------------------- general form
// Moments of a chunk's groups: emit(g, moments) for every group.
// sm: [slots][C] float2
template <typename T, int V, typename Emit>
__device__ __forceinline__ void chunk_moments(const GnArgs& a, const GnPlan& p, const Place& w, float2* sm, Emit emit) {
  constexpr int N = rows_ahead(V);
  if (w.on) {
    float n = 0.f, mean[V], m2[V];
#pragma unroll
    for (int k = 0; k < V; ++k) mean[k] = m2[k] = 0.f;
    const T* x = static_cast<const T*>(a.x) + w.at;
    auto load = [&](Block<T, V, N>& k, size_t at, int cnt) {
#pragma unroll
      for (int u = 0; u < N; ++u) k.r[u] = fetch<T, V>(x, w, at, u, cnt);
    };
    walk<N, false, Block<T, V, N>>(p, w, w.rows, a.C, load, [&](const Block<T, V, N>& blk, size_t, int cnt) {
      float v[N][V];
#pragma unroll
      for (int u = 0; u < N; ++u) unpack(blk.r[u], v[u]);
      const float m = (float)cnt, im = 1.f / m, wn = m / (n + m), wd = n * wn;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int u = 0; u < N; ++u) s += u < cnt ? v[u][k] : 0.f;
        const float bm = s * im;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const float d = u < cnt ? v[u][k] - bm : 0.f;
          q = fmaf(d, d, q);
        }
        const float d = bm - mean[k];
        mean[k] = fmaf(d, wn, mean[k]);
        m2[k] += fmaf(d * d, wd, q);
      }
      n += m;
    });
#pragma unroll
    for (int k = 0; k < V; ++k) sm[(size_t)w.slot * a.C + w.c + k] = make_float2(mean[k], m2[k]);
  }
  __syncthreads();
  const int cg = a.C / a.G;
  join_groups(
      a.G, cg * p.slots, p.group_lanes,
      [&](int g, int i) {
        const int s = i / cg, c = i - s * cg;
        const float2 e = sm[(size_t)s * a.C + g * cg + c];
        return Moments{(float)dealt(w.rows, w.chunk, p.chunks, p.slots * N, s, p.slots), e.x, e.y};
      },
      emit);
}

// y of the chunk's rows with stat(g) = (mean, rstd)
template <typename T, int V, int ACT>
__device__ __forceinline__ void chunk_apply(const GnArgs& a, const GnPlan& p, const Place& w, const float2* stat) {
  constexpr int N = rows_ahead(V);
  if (!w.on) return;
  const int cg = a.C / a.G;
  float ga[V], be[V], mean[V];
  affine<V>(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float2 st = stat[(w.c + k) / cg];
    mean[k] = st.x;
    ga[k] *= st.y;
  }
  const T* x = static_cast<const T*>(a.x) + w.at;
  T* y = static_cast<T*>(a.y) + w.at;
  auto load = [&](Block<T, V, N>& k, size_t at, int cnt) {
#pragma unroll
    for (int u = 0; u < N; ++u) k.r[u] = fetch<T, V>(x, w, at, u, cnt);
  };
  walk<N, true, Block<T, V, N>>(p, w, w.rows, a.C, load, [&](const Block<T, V, N>& blk, size_t at, int cnt) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float v[V];
      unpack(blk.r[u], v);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = act_f<ACT, T>(fmaf(v[k] - mean[k], ga[k], be[k]));
      if (u < cnt) put(y + at + u * w.step + w.off, v);
    }
  });
  if (a.pad_zero) pad<N, V>(a, p, w, y);
}

__device__ __forceinline__ float2 stat_of(const GnArgs& a, int b, int g, Moments m) {
  const float var = m.n > 0.f ? m.m2 / m.n : 0.f;
  const float2 st = make_float2(m.mean, 1.f / sqrtf(var + a.eps));
  if (a.mean) a.mean[(size_t)b * a.G + g] = st.x;
  if (a.rstd) a.rstd[(size_t)b * a.G + g] = st.y;
  return st;
}

extern __shared__ float2 gn_smem[];

template <typename T, int V, int TPB> __global__ __launch_bounds__(TPB) void gn_moments_kernel(GnArgs a, GnPlan p) {
  const Place w = place<V>(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  float2* out = a.part + ((size_t)w.b * p.chunks + w.chunk) * a.G;
  chunk_moments<T, V>(a, p, w, gn_smem, [&](int g, Moments m) { out[g] = make_float2(m.mean, m.m2); });
}

// second launch (chunks > 1) or the whole of it (FUSED: one chunk per sample)
template <typename T, int V, int ACT, bool FUSED, int TPB>
__global__ __launch_bounds__(TPB) void gn_apply_kernel(GnArgs a, GnPlan p) {
  const Place w = place<V>(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  const int cg = a.C / a.G;
  float2* stat = gn_smem;
  if (FUSED) {
    stat = gn_smem + (size_t)p.slots * a.C;
    chunk_moments<T, V>(a, p, w, gn_smem, [&](int g, Moments m) { stat[g] = stat_of(a, w.b, g, m); });
  } else {
    const float2* part = a.part + (size_t)w.b * p.chunks * a.G;
    const int live = live_rows(a.lens, w.b, a.S);
    GnArgs first = a;
    if (w.chunk) first.mean = first.rstd = nullptr;  // one workgroup per sample writes the statistics
    join_groups(
        a.G, p.chunks, p.group_lanes,
        [&](int g, int i) {
          const int rows = dealt(live, i, p.chunks, p.slots * rows_ahead(V), -1, p.slots);
          const float2 e = part[(size_t)i * a.G + g];
          return Moments{(float)rows * cg, e.x, e.y};
        },
        [&](int g, Moments m) { stat[g] = stat_of(first, w.b, g, m); });
  }
  __syncthreads();
  chunk_apply<T, V, ACT>(a, p, w, stat);
}

// Sums of a chunk: per channel (sum dn xh, sum dn) to `chan`, per group of the
// gamma-weighted (sum gamma dn, sum gamma dn xh) to emit. `add`: on top of what chan holds.
template <typename T, int V, int ACT, int TPB, typename Emit>
__device__ __forceinline__ void chunk_sums(const GnArgs& a, const GnPlan& p, const Place& w, float2* sm, float* chan,
                                           bool add, Emit emit) {
  constexpr int N = TPB > 256 ? 1 : 4;  // (wide rows: large workgroups, few registers a thread)
  const int cg = a.C / a.G;
  if (w.on) {
    float ga[V], be[V], mean[V], rs[V], s1[V], s2[V];
    affine<V>(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const size_t g = (size_t)w.b * a.G + (w.c + k) / cg;
      mean[k] = a.mean_in[g];
      rs[k] = a.rstd_in[g];
      s1[k] = s2[k] = 0.f;
    }
    const T* x = static_cast<const T*>(a.x) + w.at;
    const T* dy = static_cast<const T*>(a.dy) + w.at;
    auto load = [&](Block2<T, V, N>& k, size_t at, int cnt) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        k.x[u] = fetch<T, V>(x, w, at, u, cnt);
        k.d[u] = fetch<T, V>(dy, w, at, u, cnt);
      }
    };
    walk<N, false, Block2<T, V, N>>(p, w, w.rows, a.C, load, [&](const Block2<T, V, N>& blk, size_t at, int cnt) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        float v[V], d[V];
        unpack(blk.x[u], v);
        unpack(blk.d[u], d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float xh = (v[k] - mean[k]) * rs[k];
          float y, da;
          act_d<ACT, T>(fmaf(xh, ga[k], be[k]), y, da);
          const float dn = u < cnt ? d[k] * da : 0.f;
          s1[k] += dn;
          s2[k] = fmaf(dn, xh, s2[k]);
        }
      }
    });
#pragma unroll
    for (int k = 0; k < V; ++k) sm[(size_t)w.slot * a.C + w.c + k] = make_float2(s1[k], s2[k]);
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
template <typename T, int V, int ACT, int TPB>
__device__ __forceinline__ void chunk_dx(const GnArgs& a, const GnPlan& p, const Place& w, const float2* avg) {
  constexpr int N = TPB > 256 ? 1 : 4;  // (wide rows: large workgroups, few registers a thread)
  if (!w.on) return;
  const int cg = a.C / a.G;
  float ga[V], be[V], mean[V], rs[V], m1[V], m2[V];
  affine<V>(a.gamma, a.beta, w.c, ga, be);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int g = (w.c + k) / cg;
    mean[k] = a.mean_in[(size_t)w.b * a.G + g];
    rs[k] = a.rstd_in[(size_t)w.b * a.G + g];
    m1[k] = avg[g].x;
    m2[k] = avg[g].y;
  }
  const T* x = static_cast<const T*>(a.x) + w.at;
  const T* dy = static_cast<const T*>(a.dy) + w.at;
  T* dx = static_cast<T*>(a.dx) + w.at;
  auto load = [&](Block2<T, V, N>& k, size_t at, int cnt) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      k.x[u] = fetch<T, V>(x, w, at, u, cnt);
      k.d[u] = fetch<T, V>(dy, w, at, u, cnt);
    }
  };
  walk<N, true, Block2<T, V, N>>(p, w, w.rows, a.C, load, [&](const Block2<T, V, N>& blk, size_t at, int cnt) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float v[V], d[V];
      unpack(blk.x[u], v);
      unpack(blk.d[u], d);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float xh = (v[k] - mean[k]) * rs[k];
        float y, da;
        act_d<ACT, T>(fmaf(xh, ga[k], be[k]), y, da);
        v[k] = rs[k] * fmaf(-xh, m2[k], fmaf(d[k] * da, ga[k], -m1[k]));
      }
      if (u < cnt) put(dx + at + u * w.step + w.off, v);
    }
  });
  pad<N, V>(a, p, w, dx);
}

template <typename T, int V, int ACT, int TPB> __global__ __launch_bounds__(TPB) void gn_sums_kernel(GnArgs a, GnPlan p) {
  const Place w = place<V>(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  float2* out = a.part + ((size_t)w.b * p.chunks + w.chunk) * a.G;
  float* chan = a.chan + (size_t)blockIdx.x * 2 * a.C;
  chunk_sums<T, V, ACT, TPB>(a, p, w, gn_smem, chan, false, [&](int g, float2 m) { out[g] = m; });
}

// second launch (chunks > 1): dx of one chunk
template <typename T, int V, int ACT, int TPB> __global__ __launch_bounds__(TPB) void gn_dx_kernel(GnArgs a, GnPlan p) {
  const Place w = place<V>(a, p, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
  const int live = live_rows(a.lens, w.b, a.S);
  const float inv = live ? 1.f / ((float)live * (float)(a.C / a.G)) : 0.f;
  float2* avg = gn_smem;
  const float2* part = a.part + (size_t)w.b * p.chunks * a.G;
  sum_groups(a.G, p.chunks, p.group_lanes, [&](int g, int i) { return part[(size_t)i * a.G + g]; },
             [&](int g, float2 m) { avg[g] = make_float2(m.x * inv, m.y * inv); });
  __syncthreads();
  chunk_dx<T, V, ACT, TPB>(a, p, w, avg);
}

// one chunk per sample: a workgroup takes `samples` of them one after the other
template <typename T, int V, int ACT, int TPB> __global__ __launch_bounds__(TPB) void gn_bwd_kernel(GnArgs a, GnPlan p) {
  float2* avg = gn_smem + (size_t)p.slots * a.C;
  float* chan = a.chan + (size_t)blockIdx.x * 2 * a.C;
  const int b0 = blockIdx.x * p.samples, b1 = b0 + p.samples < a.B ? b0 + p.samples : a.B;
  for (int b = b0; b < b1; ++b) {
    const Place w = place<V>(a, p, b, 0);
    const int live = live_rows(a.lens, b, a.S);
    const float inv = live ? 1.f / ((float)live * (float)(a.C / a.G)) : 0.f;
    chunk_sums<T, V, ACT, TPB>(a, p, w, gn_smem, chan, b > b0,
                       [&](int g, float2 m) { avg[g] = make_float2(m.x * inv, m.y * inv); });
    __syncthreads();
    chunk_dx<T, V, ACT, TPB>(a, p, w, avg);
  }
}

// ---------------------------------------------------------------- rows form
// One row per sample: lanes [0, LANES) of a group hold NV vectors each.
// Threads of a workgroup, by the registers that NV vectors take
constexpr int row_threads(int nv) { return nv == 1 ? 1024 : (nv <= 3 ? 512 : 256); }

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
template <typename T, int ACT, int NV> __global__ __launch_bounds__(row_threads(NV)) void gn_rows_kernel(GnArgs a, GnPlan p) {
  const RowPlace<NV> w = row_place<NV>(a, p);
  if (!w.on) return;
  const float inv = 1.f / (float)(a.C / a.G);
  const long long b0 = (long long)blockIdx.x * p.per, b1 = b0 + p.per < a.B ? b0 + p.per : a.B;
  for (long long b = b0 + w.slot; b < b1; b += p.slots) {
    float v[NV][8];
    const bool live = live_rows(a.lens, (int)b, 1) == 1;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i]) ld8(static_cast<const T*>(a.x) + b * a.C + w.c0 + i * w.step, v[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i])
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[i][k];
    const float mean = lanes_sum(s, p.lanes) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w.has[i])
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[i][k] -= mean;
          q = fmaf(v[i][k], v[i][k], q);
        }
    const float var = lanes_sum(q, p.lanes) * inv;
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
        affine<8>(a.gamma, a.beta, w.c0 + i * w.step, ga, be);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = live ? act_f<ACT, T>(fmaf(v[i][k] * rstd, ga[k], be[k])) : 0.f;
        st8(y + i * w.step, v[i]);
      }
  }
}

template <typename T, int ACT, int NV> __global__ __launch_bounds__(row_threads(NV)) void gn_rows_dx_kernel(GnArgs a, GnPlan p) {
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
          affine<8>(a.gamma, a.beta, w.c0 + i * w.step, ga, be);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = (v[i][k] - mean) * rstd;
            float y, da;
            act_d<ACT, T>(fmaf(xh, ga[k], be[k]), y, da);
            const float dn = live ? d[i][k] * da : 0.f;
            s1[i][k] += dn;
            if (live) s2[i][k] = fmaf(dn, xh, s2[i][k]);
            v[i][k] = xh;
            d[i][k] = dn * ga[k];
            t1 += d[i][k];
            t2 = fmaf(d[i][k], xh, t2);
          }
        }
      const float m1 = lanes_sum(t1, p.lanes) * inv, m2 = lanes_sum(t2, p.lanes) * inv;
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

template <typename T, int V, int ACT, int TPB> hipError_t fwd_general(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * p.chunks);
  const size_t sums = slots_bytes(a, p), stat = (size_t)a.G * sizeof(float2);
  if (p.chunks == 1) return launch(gn_apply_kernel<T, V, ACT, true, TPB>, grid, p.threads, sums + stat, a, p, s);
  const hipError_t e = launch(gn_moments_kernel<T, V, TPB>, grid, p.threads, sums, a, p, s);
  if (e != hipSuccess) return e;
  return launch(gn_apply_kernel<T, V, ACT, false, TPB>, grid, p.threads, stat, a, p, s);
}

template <typename T, int V, int ACT, int TPB> hipError_t bwd_general(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * p.chunks);
  const size_t sums = slots_bytes(a, p), avg = (size_t)a.G * sizeof(float2);
  if (p.chunks == 1) return launch(gn_bwd_kernel<T, V, ACT, TPB>, (unsigned)p.chan_rows, p.threads, sums + avg, a, p, s);
  const hipError_t e = launch(gn_sums_kernel<T, V, ACT, TPB>, grid, p.threads, sums, a, p, s);
  if (e != hipSuccess) return e;
  return launch(gn_dx_kernel<T, V, ACT, TPB>, grid, p.threads, avg, a, p, s);
}

template <typename T, int V, int ACT> hipError_t general(const GnArgs& a, const GnPlan& p, bool bwd, hipStream_t s) {
  if (p.threads <= 256) return bwd ? bwd_general<T, V, ACT, 256>(a, p, s) : fwd_general<T, V, ACT, 256>(a, p, s);
  return bwd ? bwd_general<T, V, ACT, 1024>(a, p, s) : fwd_general<T, V, ACT, 1024>(a, p, s);
}

template <typename T, int ACT> hipError_t fwd_go(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  if (p.rows_form) return rows_go<T, ACT>(a, p, false, s);
  if constexpr (sizeof(T) == 4)
    if (p.vec == 4) return general<T, 4, ACT>(a, p, false, s);
  return general<T, 8, ACT>(a, p, false, s);
}

template <typename T, int ACT> hipError_t bwd_go(const GnArgs& a, const GnPlan& p, hipStream_t s) {
  hipError_t e;
  if (p.rows_form) {
    e = rows_go<T, ACT>(a, p, true, s);
  } else {
    e = hipSuccess;
    if constexpr (sizeof(T) == 4) {
      if (p.vec == 4) e = general<T, 4, ACT>(a, p, true, s);
      else e = general<T, 8, ACT>(a, p, true, s);
    } else {
      e = general<T, 8, ACT>(a, p, true, s);
    }
  }
  // the channel sums are [rows][dgamma C, dbeta C]: one launch when they go to neighbouring outputs
  if (e == hipSuccess && a.dgamma && a.dbeta == a.dgamma + a.C) return colsum(a.chan, a.dgamma, p.chan_rows, 2 * a.C, 2 * a.C, s);
  if (e == hipSuccess && a.dgamma) e = colsum(a.chan, a.dgamma, p.chan_rows, 2 * a.C, a.C, s);
  if (e == hipSuccess && a.dbeta) e = colsum(a.chan + a.C, a.dbeta, p.chan_rows, 2 * a.C, a.C, s);
  return e;
}

}  // namespace

hipError_t colsum(const float* part, float* out, long long rows, int ld, int D, hipStream_t s) {
  colsum_kernel<<<(D + 63) / 64, 1024, 0, s>>>(part, out, rows, ld, D);
  return hipGetLastError();
}

GnPlan gn_plan(int B, int S, int C, int G, bool bf, bool bwd) {
  GnPlan p{};
  p.vec = bf || C > 4096 ? 8 : 4;
  const int cg = C / G, nv = C / p.vec;
  if (S == 1 && cg % 8 == 0) {
    // lanes per group, a power of two up to a wave, with `n` vectors each: few idle
    // places and few vectors (a lane's vectors follow one another in time)
    const int q = cg / 8;
    double best = 1e30;
    for (int l = 64; l >= 1; l >>= 1) {
      const int n = (q + l - 1) / l;
      if (n > 16 || (long long)G * l > row_threads(n)) continue;
      const double cost = (double)l * n * (1 + n / 8.0);
      if (cost < best) {
        best = cost;
        p.lanes = l;
        p.nv = n;
        p.rows_form = true;
      }
    }
  }
  if (p.rows_form) {
    const int tps = G * p.lanes;
    p.slots = tps >= 256 ? 1 : 256 / tps;
    if ((long long)p.slots * C > 8192) p.slots = 8192 / C;  // the backward's channel sums take 64 KB of LDS at most
    p.threads = (tps * p.slots + 63) / 64 * 64;
    // Forward: about 2048 workgroups (bf16 rows, us, with 1024 and 2048: 100k x 256 27.0 and 21.0).
    // Backward: about 512, each of which leaves a row of channel sums to be added up (with 512
    // and 2048: 16k x 768 27.8 and 42.2, 8192 x 2048 37.8 and 61; 100k x 256 51.6 and 40.0)
    const int groups = bwd ? 512 : 2048;
    long long per = ((long long)B + groups - 1) / groups;
    per = (per + p.slots - 1) / p.slots * p.slots;
    p.per = (int)per;
    p.chunks = 1;
    p.chan_rows = (B + per - 1) / per;
    return p;
  }
  p.slots = nv >= 256 ? 1 : 256 / nv;
  p.threads = (nv * p.slots + 63) / 64 * 64;
  // One launch as soon as the samples give every CU a workgroup, and from half of that on if a
  // sample is at most 512 KB (bf16 forward, us, one launch and two: 256 x 256 x 128 10.8 and 12.5,
  // 200 x 1024 x 128 27 and 32, 64 x 256 x 512 20.3 and 15.9, 100 x 4096 x 256 154 and 112).
  // Otherwise about 256 workgroups: each of the second launch joins its sample's chunks, so a
  // sample cut finer costs more (256 and 1024 workgroups: 8 x 4096 x 384 21.8 and 36.2,
  // 1 x 65536 x 512 44 and 119); but up to 8 chunks a sample while they are under about 1024, whose
  // join is short, to even out the CUs' loads (100 x 4096 x 256, 300 and 800: 133 and 119).
  const bool one = B >= 256 || (B >= 128 && (long long)S * C * (bf ? 2 : 4) <= (512 << 10));
  long long chunks = 1;
  if (!one) {
    const long long even = (1024 + B - 1) / B < 8 ? (1024 + B - 1) / B : 8;
    chunks = (256 + B - 1) / B > even ? (256 + B - 1) / B : even;
  }
  // no chunk without a block of rows
  const int unit = p.slots * rows_ahead(p.vec);
  if (chunks > (S + unit - 1) / unit) chunks = (S + unit - 1) / unit;
  p.chunks = (int)chunks;
  // lanes that join a group's sums: all groups in one go
  p.group_lanes = 1;
  while (p.group_lanes < 64 && p.group_lanes * 2 * G <= p.threads) p.group_lanes *= 2;
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
