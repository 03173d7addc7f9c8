// Gated feed-forward block: (p, q) = x W_in, z = p act(q), y = z W_out, and its
// backward pass, on the MFMA units of gfx950.
//
// Every product is C [M][N] = A [M][K] B [K][N] in fp32 accumulators, with the
// operands read as they are stored: K contiguous (rows of x, dy, z; W_in and
// W_out where their transposes are needed) or K strided (W_in and W_out as they
// are; both operands of the weight gradients, whose K runs over the rows of x).
//  * Global to LDS: 16-byte loads that write LDS directly, tiles of 128 bytes of K (two
//    MFMA slices in bf16) in two stages. The one barrier per tile stands between its
//    two slices: the fragments of the second are in registers by then, so the
//    tile's stage can be written again and the next tile's first fragments are read
//    under the second slice's products. A tile is on its way for a whole tile's time.
//    Reads and loads are spread between the MFMA instructions.
//  * LDS: a tile is R rows (or columns) by 128 bytes of K. K contiguous: rows of
//    128 bytes, 16-byte chunk c of row r at slot c ^ (r & 7), so that the 16 rows
//    of a fragment read spread over the banks. K strided: rows of k, R elements
//    each; blocks of 16 columns are exchanged by a function of k so that the rows
//    of one transposing read (ds_read_b64_tr_b16; for fp32 four 4-byte reads) lie
//    in different banks. (No bank conflicts by the counters.)
//  * MFMA: 16x16x32 bf16. The operands go in swapped, so that a lane ends with four
//    neighbouring columns of one row of C. (fp32 with few products per operand: 4 x
//    16x16x4.)
//  * In the larger tiles fp32 operands are split in registers into three bf16 words,
//    x = h + m + l: h and m round to nearest, so |m| <= 2^-9 |x|, |l| <= 2^-18 |x| and the
//    rest is below 2^-27 |x|. The products h h', h m', m h', h l', l h', m m' leave out less
//    than 2^-25 of |x x'|, under the 2^-24 of an fp32 rounding; sums stay in fp32. Six bf16
//    MFMAs take 96 cycles where the fp32 ones take 256. An infinity gives NaN (inf - inf).
//  * The gated product reads the p and the q columns of W_in as one tile and
//    multiplies p by act(q) in registers. The backward computes them again, reads
//    dz = dy W_out^T where the epilogue needs it, and writes dp and dq in its place.
//    In bf16 dz waits there as two words (dz to 2^-17), so that dp and dq are rounded
//    once; one word, rounded, made the gradients' error 1.7 times one rounding's
//    instead of 1.4 and the backward of 16384 x 768 x 2048 33 of 531 us faster.
//    Other homes for dz (backward, us, against the kept form): a third accumulator with
//    half the tile, 2048 x 768 x 2048 107 and 116, 16384 x 768 x 2048 535 and 530,
//    16384 x 2048 x 5632 3173 and 2940; the workgroup's own product, left in memory and
//    taken back from cache, 326 us for what takes 88 + 206 at 16384 x 768 x 2048.
//
// Measured at 16384 x 768 x 2048, bf16: gate 98 us (1050 TFLOP/s), y 48 us; backward dz 88,
// gates 206 (103 GFLOP, and 336 MB in the epilogue while the matrix units wait), dx 89
// (1160 TFLOP/s), dw_in 99 + 12 and dw_out 77 + 6 us with the sums of their K splits. fp32,
// 4099 x 384 x 1032: 72 + 42 us. 8 rows of 768 x 2048: 5.6 + 6.0 us.
#include <type_traits>

#include "act.h"
#include "kernels_block.h"

namespace hy {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kThreads = 512;         // 8 waves
constexpr int kWm = 2, kWn = 4;       // wave rows and columns of a block tile
constexpr unsigned kOut = 0x80000000u, kRange = 0x7fffffffu;  // an offset outside the loads' range reads zero

template <typename T> struct Elem {
  static constexpr int E = sizeof(T);
  static constexpr int V = 16 / E;    // elements per 16 bytes
  static constexpr int BK = 128 / E;  // K per tile
};

// Where 16-column block c of LDS row k starts in a K-strided tile, in blocks: k
// enters through the bits that differ between the rows of one fragment read
template <typename T, int R> __device__ __forceinline__ int mix(int k) {
  constexpr int mask = (R & (R - 1)) == 0 ? R / 16 - 1 : 3;  // R = 192: within groups of four blocks
  if (sizeof(T) == 2) return ((k & 3) | (((k >> 3) & 3) << 2)) & mask;
  return ((k >> 2) & 3) & mask;
}

// 16 bytes a lane from base + off (zeros where off is out of range) to the wave's 1 KB
// of LDS at `dst`. Written out because the compiler, which cannot tell the stages
// apart, waits for every such load it knows of before each transposing LDS read;
// the waits that are needed stand in tile_barrier. The instruction has no
// destination register, its operands are read when it issues.
__device__ __forceinline__ void load_lds(const char* base, unsigned off, char* dst) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  const unsigned long long b = reinterpret_cast<unsigned long long>(base);
  const u32x4 rs = {(unsigned)b, (unsigned)(b >> 32) & 0xffffu, kRange, 0x00020000u};
  const unsigned at = (unsigned)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rs)
               : "memory", "m0");
}

// Loads of one operand's tiles: R rows of K-contiguous data, or R columns of
// K-strided data (PAIR: the second half of the columns lies `second` elements on).
template <typename T, bool KS, int R, bool PAIR = false> struct Loader {
  static constexpr int E = Elem<T>::E, V = Elem<T>::V, BK = Elem<T>::BK;
  static constexpr int NL = R * 128 / (kThreads * 16);
  const char* base;   // first element of the next tile
  size_t step;        // bytes between tiles
  unsigned off[NL];
  int kk[NL];         // K of the load within its tile
  // origin: element (row or column r0, k0) of the operand; n: valid rows or columns from r0 on
  __device__ __forceinline__ void init(const T* origin, long long ld, int n, long long second = 0) {
    base = reinterpret_cast<const char*>(origin);
    step = KS ? (size_t)BK * ld * E : (size_t)128;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if (!KS) {
        const int r = (i * (kThreads / 64) + wave) * 8 + (lane >> 3), c = (lane & 7) ^ (lane >> 3);
        // rows behind the last one repeat the first: they only feed rows of C that are not stored
        off[i] = (unsigned)((r < n ? (long long)r * ld * E : 0) + c * 16);
        kk[i] = c * V;
      } else {
        constexpr int RB = R * E;
        const int flat = (i * (kThreads / 64) + wave) * 1024 + lane * 16;
        const int k = flat / RB, el = flat % RB / E;
        int col = ((el >> 4) ^ mix<T, R>(k)) * 16 + (el & 15);
        long long at;
        if (PAIR) {
          const int h = col >= R / 2;
          if (h) col -= R / 2;
          at = (col < n ? col : 0) + (h ? second : 0);
        } else {
          at = col < n ? col : 0;
        }
        off[i] = (unsigned)(((long long)k * ld + at) * E);
        kk[i] = k;
      }
    }
  }
  // load i of the next tile into LDS at `dst`; left: K elements from the tile's start on
  __device__ __forceinline__ void issue(int i, char* dst, int left) const {
    const unsigned o = left >= BK || kk[i] < left ? off[i] : kOut;
    load_lds(base, o, dst + (i * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 1024);
  }
  __device__ __forceinline__ void issue(char* dst, int left) {
#pragma unroll
    for (int i = 0; i < NL; ++i) issue(i, dst, left);
    base += step;
  }
};

// Fragments of a tile: 16 rows (columns) by one K slice (32 bf16 or 16 fp32)
template <typename T> struct Frag;
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { f32x4 v; };

template <typename T, bool KS, int R> struct Reader {
  int lane_off, flip;
  __device__ __forceinline__ void init() {
    const int l = threadIdx.x & 63;
    flip = 0;
    if (!KS) {
      lane_off = (l & 15) * 128 + (((l >> 4) ^ (l & 7)) * 16);
    } else if (sizeof(T) == 2) {
      const int k = (l >> 4) * 8 + ((l & 15) >> 2);
      lane_off = k * (R * 2) + (l & 3) * 8;
      flip = mix<T, R>(k);
    } else {
      lane_off = (l >> 4) * 4 * (R * 4) + (l & 15) * 4;
      flip = mix<T, R>((l >> 4) * 4);
    }
  }
  __device__ __forceinline__ Frag<T> read(const char* tile, int block, int slice) const {
    Frag<T> f;
    if constexpr (!KS) {
      // the second slice's chunks are 4 to 7: bit 2 of the slot
      f.v = *reinterpret_cast<const decltype(f.v)*>(tile + block * 2048 + (lane_off ^ (slice * 64)));
    } else if constexpr (sizeof(T) == 2) {
      const char* p = tile + lane_off + (block ^ flip) * 32 + slice * (32 * R * 2);
      typedef __attribute__((address_space(3))) s16x4* tp;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(p));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(p + 4 * R * 2));
      f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const char* p = tile + lane_off + (block ^ flip) * 64 + slice * (16 * R * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = *reinterpret_cast<const float*>(p + j * (R * 4));
    }
    return f;
  }
};

// acc[x][y] (16 columns of block y by 16 rows of block x) += B^T A^T over one K slice
template <int MI, int NJ>
__device__ __forceinline__ void mma_all(const Frag<bf16> (&n)[NJ], const Frag<bf16> (&m)[MI], f32x4 (&acc)[MI][NJ]) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n[j].v, m[i].v, acc[i][j], 0, 0, 0);
}
template <int MI, int NJ>
__device__ __forceinline__ void mma_all(const Frag<float> (&n)[NJ], const Frag<float> (&m)[MI], f32x4 (&acc)[MI][NJ]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(n[j].v[k], m[i].v[k], acc[i][j], 0, 0, 0);
}

// Eight fp32 values as three bf16 words each, two values at a time: one packed
// conversion, and the parts taken back as fp32 by a shift and a mask
struct Words {
  bf16x8 h, m, l;
};
__device__ __forceinline__ unsigned pack(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  return __builtin_bit_cast(unsigned, bf16x2{(bf16)a, (bf16)b});
}
__device__ __forceinline__ Words split(const Frag<float>& a, const Frag<float>& b) {
  typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
  u32x4 h, m, l;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x = k < 2 ? a.v[2 * k] : b.v[2 * k - 4], y = k < 2 ? a.v[2 * k + 1] : b.v[2 * k - 3];
    h[k] = pack(x, y);
    x -= __uint_as_float(h[k] << 16);
    y -= __uint_as_float(h[k] & 0xffff0000u);
    m[k] = pack(x, y);
    x -= __uint_as_float(m[k] << 16);
    y -= __uint_as_float(m[k] & 0xffff0000u);
    l[k] = pack(x, y);
  }
  return Words{__builtin_bit_cast(bf16x8, h), __builtin_bit_cast(bf16x8, m), __builtin_bit_cast(bf16x8, l)};
}
// acc[j] += B_j^T A^T, smallest terms first; neighbouring MFMAs go to different accumulators
template <int NJ> __device__ __forceinline__ void mma_row(const Words (&n)[NJ], const Words& m, f32x4 (&acc)[NJ]) {
#pragma unroll
  for (int t = 0; t < 6; ++t)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const bf16x8 x = t == 0 ? n[j].l : (t == 2 || t == 3 ? n[j].m : n[j].h);
      const bf16x8 y = t == 1 ? m.l : (t == 2 || t == 4 ? m.m : m.h);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc[j], 0, 0, 0);
    }
}
// fp32 tiles of a wave large enough for their splits to hide behind their products, in
// us per K tile: 256 x 256 4.4 (the fp32 MFMA's peak rate is 6.8), 128 x 128 1.5 (1.7)
template <typename T, int MI, int NJ> constexpr bool kSplit = sizeof(T) == 4 && MI * NJ >= 8;

// At most N of this wave's loads still on their way, its LDS reads done; then the workgroup meets
template <int N> __device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr size_t lds_bytes(int ra, int rb) { return (size_t)2 * (ra + rb) * 128; }

// One product into acc[MI][NJ]: blocks of 16 rows from block row `ma`, column blocks nb[j].
template <typename T, bool AKS, bool BKS, int RA, int RB, bool PAIR, int MI, int NJ>
__device__ __forceinline__ void product(Loader<T, AKS, RA>& la, Loader<T, BKS, RB, PAIR>& lb, int K, char* smem, int ma,
                                        const int (&nb)[NJ], f32x4 (&acc)[MI][NJ]) {
  constexpr int BK = Elem<T>::BK, ABYTES = RA * 128, STAGE = (RA + RB) * 128;
  constexpr int NL = Loader<T, AKS, RA>::NL + Loader<T, BKS, RB, PAIR>::NL;  // loads of a thread per tile
  struct Frags {
    Frag<T> a[MI], b[NJ];
  };
  Reader<T, AKS, RA> ra;
  Reader<T, BKS, RB> rb;
  ra.init();
  rb.init();
  constexpr int NA = Loader<T, AKS, RA>::NL, NB = Loader<T, BKS, RB, PAIR>::NL;
  // part i of MI: that part's fragment reads and loads, and one row of products
  auto read_part = [&](Frags& f, const char* tile, int slice, int i) {
    f.a[i] = ra.read(tile, ma + i, slice);
#pragma unroll
    for (int j = i * NJ / MI; j < (i + 1) * NJ / MI; ++j) f.b[j] = rb.read(tile + ABYTES, nb[j], slice);
  };
  auto load_part = [&](char* tile, int left, int i) {
#pragma unroll
    for (int l = i * NA / MI; l < (i + 1) * NA / MI; ++l) la.issue(l, tile, left);
#pragma unroll
    for (int l = i * NB / MI; l < (i + 1) * NB / MI; ++l) lb.issue(l, tile + ABYTES, left);
  };
  auto multiply_part = [&](const Frags& f, int i) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if constexpr (sizeof(T) == 2)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j].v, f.a[i].v, acc[i][j], 0, 0, 0);
    if constexpr (sizeof(T) == 4)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(f.b[j].v[k], f.a[i].v[k], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Tiles behind the last are asked for like any other; their offsets lie outside
  // the range, so they read nothing and the loop needs no branches.
  la.issue(smem, K);
  lb.issue(smem + ABYTES, K);
  la.issue(smem + STAGE, K - BK);
  lb.issue(smem + STAGE + ABYTES, K - BK);
  tile_barrier<NL>();
  if constexpr (kSplit<T, MI, NJ>) {
    // fp32: both slices of a tile make one MFMA depth of split words. Row block i + 1
    // is split while block i is multiplied, block i + 2 on its way from LDS.
    char *cur = smem, *nxt = smem + STAGE;
    for (int left = K; left > 0; left -= BK) {
      Frag<T> raw[2][2];
      raw[0][0] = ra.read(cur, ma, 0);
      raw[0][1] = ra.read(cur, ma, 1);
      Words b[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        b[j] = split(rb.read(cur + ABYTES, nb[j], 0), rb.read(cur + ABYTES, nb[j], 1));
      Words a = split(raw[0][0], raw[0][1]);
      raw[1][0] = ra.read(cur, ma + 1, 0);
      raw[1][1] = ra.read(cur, ma + 1, 1);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        Words next = a;
        if (i + 2 < MI) {
          raw[i & 1][0] = ra.read(cur, ma + i + 2, 0);
          raw[i & 1][1] = ra.read(cur, ma + i + 2, 1);
        }
        if (i + 1 < MI) next = split(raw[(i + 1) & 1][0], raw[(i + 1) & 1][1]);
        mma_row<NJ>(b, a, acc[i]);
#pragma unroll
        for (int k = 0; k < 6 * NJ; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                             // one MFMA,
          __builtin_amdgcn_sched_group_barrier(0x002, (44 + 6 * NJ - 1) / (6 * NJ), 0);  // its share of the split
        }
        a = next;
      }
      tile_barrier<0>();  // the next tile is in LDS; every wave has read all of this one
      la.issue(cur, left - 2 * BK);
      lb.issue(cur + ABYTES, left - 2 * BK);
      char* t = cur;
      cur = nxt;
      nxt = t;
    }
    tile_barrier<0>();
    return;
  }
  Frags f0, f1;
#pragma unroll
  for (int i = 0; i < MI; ++i) read_part(f0, smem, 0, i);
  char *cur = smem, *nxt = smem + STAGE;
  for (int left = K; left > 0; left -= BK) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      read_part(f1, cur, 1, i);
      multiply_part(f0, i);
    }
    tile_barrier<0>();  // the next tile is in LDS; every wave has read all of this one
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      read_part(f0, nxt, 0, i);
      load_part(cur, left - 2 * BK, i);
      multiply_part(f1, i);
    }
    la.base += la.step;
    lb.base += lb.step;
    char* t = cur;
    cur = nxt;
    nxt = t;
  }
  tile_barrier<0>();  // the stages may be written again
}

template <int MI, int NJ> __device__ __forceinline__ void zero(f32x4 (&acc)[MI][NJ]) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
}

__device__ __forceinline__ void store(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store(bf16* p, f32x4 v) {
  bf16x4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = (bf16)v[k];
  *reinterpret_cast<bf16x4*>(p) = r;
}

// With lo != 0 what the rounding leaves goes lo elements further on, as a second bf16 word
__device__ __forceinline__ void store_words(float* p, long long, f32x4 v) { store(p, v); }
__device__ __forceinline__ void store_words(bf16* p, long long lo, f32x4 v) {
  store(p, v);
  if (lo) {
    f32x4 l;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float h = (float)(bf16)v[k];
      l[k] = fabsf(h) == INFINITY ? 0.f : v[k] - h;
    }
    store(p + lo, l);
  }
}

template <typename T> using Raw4 = std::conditional_t<sizeof(T) == 2, bf16x4, f32x4>;  // four elements as stored
__device__ __forceinline__ f32x4 load(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load(const bf16* p) {
  const bf16x4 r = *reinterpret_cast<const bf16x4*>(p);
  return f32x4{(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
}

constexpr int kXcds = 8;
// Tile of workgroup `bid` when consecutive workgroups go round robin to the XCDs:
// each XCD gets a contiguous range of tiles, whose operands meet in its L2
__device__ __forceinline__ int xcd_tile(int bid, int total) {
  const int q = total / kXcds, r = total % kXcds, x = bid % kXcds, k = bid / kXcds;
  return x < r ? x * (q + 1) + k : r * (q + 1) + (x - r) * q + k;
}

// Block row and column of a tile number: groups of 8 block rows, columns of a
// group one after the other, so that the 32 tiles an XCD works on at a time span
// about 8 x 4 blocks and share their operands in its L2
__device__ __forceinline__ void tile_place(int tile, int ntm, int ntn, int& tm, int& tn) {
  const int per = 8 * ntn, g = tile / per, r = tile - g * per;
  const int rows = ntm - g * 8 < 8 ? ntm - g * 8 : 8;
  tm = g * 8 + r % rows;
  tn = r / rows;
}

extern __shared__ char ffn_smem[];

// ------------------------------------------------------------ plain product
// C [M][N] = A B; with splits > 1 (grid.y), split s sums K tiles [s per, (s + 1) per)
// into out + s M N in fp32
template <typename T, typename O, bool AKS, bool BKS, int TM, int TN>
__global__ __launch_bounds__(kThreads, 1) void ffn_gemm_kernel(const T* A, const T* B, O* C, int M, int N, int K,
                                                            long long lda, long long ldb, long long ldc,
                                                            long long lo, int ntn, int per) {
  constexpr int MI = TM / kWm / 16, NJ = TN / kWn / 16, BK = Elem<T>::BK;
  const int tile = xcd_tile(blockIdx.x, gridDim.x);
  int tm, tn;
  tile_place(tile, (M + TM - 1) / TM, ntn, tm, tn);
  const int m0 = tm * TM, n0 = tn * TN;
  const long long k0 = (long long)blockIdx.y * per * BK;
  const int kn = K - k0 < (long long)per * BK ? (int)(K - k0) : per * BK;
  C += (size_t)blockIdx.y * M * N;
  Loader<T, AKS, TM> la;
  Loader<T, BKS, TN> lb;
  la.init(AKS ? A + k0 * lda + m0 : A + (long long)m0 * lda + k0, lda, M - m0);
  lb.init(BKS ? B + k0 * ldb + n0 : B + (long long)n0 * ldb + k0, ldb, N - n0);
  const int wave = threadIdx.x >> 6, wm = wave % kWm, wn = wave / kWm, lane = threadIdx.x & 63;
  int nb[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) nb[j] = wn * NJ + j;
  f32x4 acc[MI][NJ];
  zero(acc);
  product<T, AKS, BKS, TM, TN, false, MI, NJ>(la, lb, kn, ffn_smem, wm * MI, nb, acc);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = m0 + (wm * MI + i) * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + nb[j] * 16 + (lane >> 4) * 4;
      if (m < M && n < N) store_words(C + m * ldc + n, lo, acc[i][j]);
    }
  }
}

// ------------------------------------------------------------ gated product
// Block of the gated product: TM rows by TF columns of p and of q, in acc[.][j] and
// acc[.][NH + j]
template <int TM, int TF> struct GatePlace {
  static constexpr int MI = TM / kWm / 16, NH = TF / kWn / 16, NJ = 2 * NH;
  int m0, f0, wm, wn, lane;
  __device__ __forceinline__ GatePlace(int M, int F, int ntn) {
    int tm, tn;
    tile_place(xcd_tile(blockIdx.x, gridDim.x), (M + TM - 1) / TM, ntn, tm, tn);
    m0 = tm * TM;
    f0 = tn * TF;
    const int wave = threadIdx.x >> 6;
    wm = wave % kWm;
    wn = wave / kWm;
    lane = threadIdx.x & 63;
  }
  __device__ __forceinline__ int row(int i) const { return m0 + (wm * MI + i) * 16 + (lane & 15); }
  __device__ __forceinline__ int col(int j) const { return f0 + (wn * NH + j) * 16 + (lane >> 4) * 4; }
  template <typename T>
  __device__ __forceinline__ void run(const T* x, const T* w_in, int M, int D, int F, f32x4 (&acc)[MI][NJ]) const {
    Loader<T, false, TM> la;
    Loader<T, true, 2 * TF, true> lb;
    la.init(x + (long long)m0 * D, D, M - m0);
    lb.init(w_in + f0, 2LL * F, F - f0, F);
    int nb[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) nb[j] = (j < NH ? 0 : TF / 16) + wn * NH + j % NH;
    zero(acc);
    product<T, false, true, TM, 2 * TF, true, MI, NJ>(la, lb, D, ffn_smem, wm * MI, nb, acc);
  }
};

// z [M][F] = p act(q), (p, q) = x W_in
template <typename T, int ACT, int TM, int TF>
__global__ __launch_bounds__(kThreads, 1) void ffn_gate_kernel(const T* x, const T* w_in, T* z, int M, int D, int F,
                                                               int ntn) {
  constexpr int MI = TM / kWm / 16, NH = TF / kWn / 16, NJ = 2 * NH;
  GatePlace<TM, TF> w(M, F, ntn);
  f32x4 acc[MI][NJ];
  w.template run<T>(x, w_in, M, D, F, acc);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = w.row(i);
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      const int f = w.col(j);
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[i][j][k] * act_f<ACT, T>(acc[i][NH + j][k]);
      if (m < M && f < F) store(z + (size_t)m * F + f, v);
    }
  }
}

// The backward's gates: p and q again, dz = dy W_out^T from the p half of dpq [M][2F];
// dp = dz act(q) (in dz's place), dq = dz p act'(q), z = p act(q) to z [M][F]
template <typename T, int ACT, int TM, int TF>
__global__ __launch_bounds__(kThreads, 1) void ffn_dgate_kernel(const T* x, const T* w_in, T* dpq, T* z, int M, int D,
                                                                int F, int ntn) {
  constexpr int MI = TM / kWm / 16, NH = TF / kWn / 16, NJ = 2 * NH;
  GatePlace<TM, TF> w(M, F, ntn);
  f32x4 acc[MI][NJ];
  w.template run<T>(x, w_in, M, D, F, acc);
  // all of dz first (the loads overlap); places outside the matrix read their last neighbour
  constexpr int W = sizeof(T) == 2 ? 2 : 1;  // words of dz
  Raw4<T> g4[MI][NH][W];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      const int m = w.row(i) < M ? w.row(i) : M - 1, f = w.col(j) < F ? w.col(j) : F - 4;
#pragma unroll
      for (int k = 0; k < W; ++k)
        g4[i][j][k] = *reinterpret_cast<const Raw4<T>*>(dpq + (size_t)m * 2 * F + k * F + f);
    }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = w.row(i);
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      const int f = w.col(j);
      if (m >= M || f >= F) continue;
      T* d = dpq + (size_t)m * 2 * F + f;
      f32x4 g;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[k] = (float)g4[i][j][0][k];
        if constexpr (W == 2) g[k] += (float)g4[i][j][1][k];
      }
      f32x4 vz, vp, vq;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float p = acc[i][j][k];
        float s, ds;
        act_d<ACT, T>(acc[i][NH + j][k], s, ds);
        vz[k] = p * s;
        vp[k] = g[k] * s;
        vq[k] = g[k] * p * ds;
      }
      store(z + (size_t)m * F + f, vz);
      store(d, vp);
      store(d + F, vq);
    }
  }
}

// ---------------------------------------------------------------- few rows
// Up to 64 rows (decoding): the products stream the weights once. A workgroup owns
// NBT blocks of 16 columns (PAIR: NBT / 2 of p and of q), its eight waves a range of
// K each, with LDS of their own: no barrier until their sums are joined, in wave
// order. RING slices of x and W are on their way to LDS per wave.
enum { kStore = 0, kGate = 1, kDgate = 2 };

// Loads of one wave's slices of an operand: KC, NB blocks of 16 rows; KS, NB blocks of
// 16 columns (PAIR: the second half `second` elements on); 1 KB a block
template <typename T, bool KS, int NB, bool PAIR = false> struct WaveLoader {
  static constexpr int E = Elem<T>::E, V = Elem<T>::V, BK = Elem<T>::BK / 2;
  const char* base;
  size_t step;
  unsigned off[NB];
  int kk[NB];
  __device__ __forceinline__ void init(const T* origin, long long ld, int n, long long second = 0) {
    base = reinterpret_cast<const char*>(origin);
    step = KS ? (size_t)BK * ld * E : (size_t)64;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (!KS) {
        const int r = i * 16 + (lane >> 2), c = (lane & 3) ^ ((lane >> 4) & 3);
        off[i] = (unsigned)((r < n ? (long long)r * ld * E : 0) + c * 16);
        kk[i] = c * V;
      } else {
        constexpr int R = NB * 16, RB = R * E;
        const int flat = i * 1024 + lane * 16, k = flat / RB, el = flat % RB / E;
        int col = ((el >> 4) ^ mix<T, R>(k)) * 16 + (el & 15);
        long long at;
        if (PAIR) {
          const int h = col >= R / 2;
          if (h) col -= R / 2;
          at = (col < n ? col : 0) + (h ? second : 0);
        } else {
          at = col < n ? col : 0;
        }
        off[i] = (unsigned)(((long long)k * ld + at) * E);
        kk[i] = k;
      }
    }
  }
  __device__ __forceinline__ void issue(char* dst, int left) {
#pragma unroll
    for (int i = 0; i < NB; ++i) load_lds(base, left >= BK || kk[i] < left ? off[i] : kOut, dst + i * 1024);
    base += step;
  }
};

// fragment of block b of a KC slice (rows of 64 bytes, chunk c of row r at slot c ^ ((r >> 2) & 3))
template <typename T> __device__ __forceinline__ Frag<T> wave_rows(const char* slice, int b) {
  const int l = threadIdx.x & 63;
  Frag<T> f;
  f.v = *reinterpret_cast<const decltype(f.v)*>(slice + b * 1024 + (l & 15) * 64 + (((l >> 4) ^ ((l >> 2) & 3)) * 16));
  return f;
}

constexpr int kFewWaves = 8;
constexpr int few_ring(int mb, int nbt) { return 20 / (mb + nbt) < 8 ? 20 / (mb + nbt) : 8; }
constexpr size_t few_lds(int mb, int nbt) {
  const size_t ring = (size_t)kFewWaves * few_ring(mb, nbt) * (mb + nbt) * 1024, sums = (size_t)kFewWaves * mb * nbt * 1024;
  return ring > sums ? ring : sums;
}

// B: W [K][ldb] (KS) or [N][ldb] (K contiguous). kStore: C [M][ldc]; kGate: z = C [M][N];
// kDgate: C = z [M][N], dpq [M][2N]
template <typename T, bool BKS, int MODE, int ACT, int MB, int NBT>
__global__ __launch_bounds__(512, 1) void ffn_few_kernel(const T* A, const T* B, T* C, T* dpq, int M, int N, int K,
                                                         long long lda, long long ldb, long long ldc,
                                                         long long lo) {
  constexpr bool PAIR = MODE != kStore;
  constexpr int BK = Elem<T>::BK / 2, RING = few_ring(MB, NBT), SLICE = (MB + NBT) * 1024;
  constexpr int NO = PAIR ? NBT / 2 : NBT;  // column blocks of the output
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring strips, which share the 128-byte lines of a row of W, on one XCD
  const int n0 = xcd_tile(blockIdx.x, gridDim.x) * NO * 16;
  const int slices = (K + BK - 1) / BK, per = (slices + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * per < slices ? wave * per : slices, s1 = s0 + per < slices ? s0 + per : slices;
  const long long k0 = (long long)s0 * BK;
  WaveLoader<T, false, MB> la;
  WaveLoader<T, BKS, NBT, PAIR && BKS> lb;
  la.init(A + k0, lda, M);
  lb.init(BKS ? B + k0 * ldb + n0 : B + (long long)n0 * ldb + k0, ldb, N - n0, N);
  Reader<T, true, NBT * 16> rb;
  rb.init();
  char* ring = ffn_smem + wave * (RING * SLICE);
  // K elements of this wave's range behind slice i (loads beyond it read nothing)
  const int range = s1 < slices ? (s1 - s0) * BK : (int)(K - k0);
  f32x4 acc[MB][NBT];
  zero(acc);
#pragma unroll
  for (int i = 0; i < RING; ++i) {
    la.issue(ring + i * SLICE, range - i * BK);
    lb.issue(ring + i * SLICE + MB * 1024, range - i * BK);
  }
  char* cur = ring;
  for (int i = 0; i < s1 - s0; ++i) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RING - 1) * (MB + NBT)) : "memory");
    Frag<T> a[MB], b[NBT];
#pragma unroll
    for (int x = 0; x < MB; ++x) a[x] = wave_rows<T>(cur, x);
#pragma unroll
    for (int x = 0; x < NBT; ++x) {
      if constexpr (BKS) b[x] = rb.read(cur + MB * 1024, x, 0);
      else b[x] = wave_rows<T>(cur + MB * 1024, x);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next loads write there
    la.issue(cur, range - (i + RING) * BK);
    lb.issue(cur + MB * 1024, range - (i + RING) * BK);
    mma_all<MB, NBT>(b, a, acc);
    cur = cur + SLICE == ring + RING * SLICE ? ring : cur + SLICE;
  }
  tile_barrier<0>();
  // [wave][row][column]
  float* sums = reinterpret_cast<float*>(ffn_smem);
#pragma unroll
  for (int x = 0; x < MB; ++x)
#pragma unroll
    for (int y = 0; y < NBT; ++y)
      store(sums + (((size_t)wave * MB + x) * 16 + (lane & 15)) * (NBT * 16) + y * 16 + (lane >> 4) * 4, acc[x][y]);
  __syncthreads();
  auto joined = [&](int m, int c) {
    const float* p = sums + m * (NBT * 16) + c;
    f32x4 t = load(p);
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) t += load(p + (size_t)w * (MB * 16 * NBT * 16));
    return t;
  };
  for (int e = threadIdx.x; e < MB * 16 * NO * 4; e += 512) {
    const int m = e / (NO * 4), c = e % (NO * 4) * 4, n = n0 + c;
    if (m >= M || n >= N) continue;
    const f32x4 p = joined(m, c);
    if constexpr (MODE == kStore) {
      store_words(C + m * ldc + n, lo, p);
    } else {
      const f32x4 q = joined(m, NO * 16 + c);
      f32x4 z;
      if constexpr (MODE == kGate) {
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = p[k] * act_f<ACT, T>(q[k]);
      } else {
        T* d = dpq + (size_t)m * 2 * N + n;
        f32x4 g = load(d);
        if constexpr (sizeof(T) == 2) g += load(d + N);
        f32x4 vp, vq;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v, dv;
          act_d<ACT, T>(q[k], v, dv);
          z[k] = p[k] * v;
          vp[k] = g[k] * v;
          vq[k] = g[k] * p[k] * dv;
        }
        store(d, vp);
        store(d + N, vq);
      }
      store(C + (size_t)m * N + n, z);
    }
  }
}

// out = sum of the splits' partial results, in order
template <typename T> __global__ __launch_bounds__(256) void ffn_join_kernel(const float* part, T* out, long long n4, int splits) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const f32x4* p = reinterpret_cast<const f32x4*>(part) + i;
  f32x4 t = p[0];
  for (int s = 1; s < splits; ++s) t += p[s * n4];
  store(out + i * 4, t);
}

// Lets a kernel take more than 64 KB of LDS, once per kernel (K) and device
template <auto K> hipError_t allow_lds(size_t bytes) {
  static DeviceCache done;
  hipError_t e = hipSuccess;
  done.get([&] {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(K), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return e == hipSuccess ? 1 : 0;
  });
  return e;
}

// The tile index that stands for the few-rows kernel, and its largest M (bf16 forward, us, few
// rows and tiles: 16 x 768 x 2048 14.4 and 16.5, 64 x 768 x 2048 16.5 and 18.0, 16 x 2048 x 5632
// 29.6 and 36.8, 64 x 2048 x 5632 40.4 and 39.9)
constexpr int kFew = 4, kFewRows = 64;
constexpr int kTm[] = {256, 256, 128, 64}, kTn[] = {256, 192, 128, 128};  // block tiles of the plain product

template <typename T, bool AKS, bool BKS, int TM, int TN>
hipError_t gemm_tiles(const T* A, const T* B, T* C, int M, int N, int K, long long lda, long long ldb, long long ldc,
                      long long lo, int splits, float* part, hipStream_t s) {
  constexpr size_t lds = lds_bytes(TM, TN);
  const int ntn = (N + TN - 1) / TN, ntm = (M + TM - 1) / TM, tiles = (K + Elem<T>::BK - 1) / Elem<T>::BK;
  const int per = (tiles + splits - 1) / splits;
  hipError_t e;
  if (splits == 1) {
    constexpr auto k = ffn_gemm_kernel<T, T, AKS, BKS, TM, TN>;
    if ((e = allow_lds<k>(lds)) != hipSuccess) return e;
    k<<<dim3(ntm * ntn), kThreads, lds, s>>>(A, B, C, M, N, K, lda, ldb, ldc, lo, ntn, per);
    return hipGetLastError();
  }
  constexpr auto k = ffn_gemm_kernel<T, float, AKS, BKS, TM, TN>;
  if ((e = allow_lds<k>(lds)) != hipSuccess) return e;
  const int used = (tiles + per - 1) / per;
  k<<<dim3(ntm * ntn, used), kThreads, lds, s>>>(A, B, part, M, N, K, lda, ldb, N, 0, ntn, per);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const long long n4 = (long long)M * N / 4;
  ffn_join_kernel<T><<<(unsigned)((n4 + 255) / 256), 256, 0, s>>>(part, C, n4, used);
  return hipGetLastError();
}

template <typename T, bool BKS, int MODE, int ACT, int MB, int NBT>
hipError_t few_launch(const T* A, const T* B, T* C, T* dpq, int M, int N, int K, long long lda, long long ldb,
                      long long ldc, long long lo, hipStream_t s) {
  constexpr size_t lds = few_lds(MB, NBT);
  constexpr auto k = ffn_few_kernel<T, BKS, MODE, ACT, MB, NBT>;
  const hipError_t e = allow_lds<k>(lds);
  if (e != hipSuccess) return e;
  const int cols = (MODE == kStore ? NBT : NBT / 2) * 16;
  k<<<(N + cols - 1) / cols, 512, lds, s>>>(A, B, C, dpq, M, N, K, lda, ldb, ldc, lo);
  return hipGetLastError();
}
// Narrow columns while they make at most one workgroup per CU, twice the width beyond
template <typename T, bool BKS, int MODE, int ACT>
hipError_t few_go(const T* A, const T* B, T* C, T* dpq, int M, int N, int K, long long lda, long long ldb,
                  long long ldc, long long lo, hipStream_t s) {
  constexpr int W = MODE == kStore ? 1 : 2;
  const bool wide = N > 256 * 16;
#define HY_FFN_FEW(MB)                                                                                     \
  return wide ? few_launch<T, BKS, MODE, ACT, MB, 2 * W>(A, B, C, dpq, M, N, K, lda, ldb, ldc, lo, s)          \
              : few_launch<T, BKS, MODE, ACT, MB, W>(A, B, C, dpq, M, N, K, lda, ldb, ldc, lo, s);
  if (M <= 16) HY_FFN_FEW(1)
  if (M <= 32) HY_FFN_FEW(2)
  HY_FFN_FEW(4)
#undef HY_FFN_FEW
}

template <typename T, bool AKS, bool BKS>
hipError_t gemm_go(const FfnProduct& p, const T* A, const T* B, T* C, int M, int N, int K, long long lda, long long ldb,
                   long long ldc, float* part, hipStream_t s, long long lo = 0) {
  if constexpr (!AKS)
    if (p.tile == kFew) return few_go<T, BKS, kStore, HYENA_ACT_NONE>(A, B, C, nullptr, M, N, K, lda, ldb, ldc, lo, s);
  switch (p.tile) {
    case 0: return gemm_tiles<T, AKS, BKS, 256, 256>(A, B, C, M, N, K, lda, ldb, ldc, lo, p.splits, part, s);
    case 1: return gemm_tiles<T, AKS, BKS, 256, 192>(A, B, C, M, N, K, lda, ldb, ldc, lo, p.splits, part, s);
    case 2: return gemm_tiles<T, AKS, BKS, 128, 128>(A, B, C, M, N, K, lda, ldb, ldc, lo, p.splits, part, s);
    default: return gemm_tiles<T, AKS, BKS, 64, 128>(A, B, C, M, N, K, lda, ldb, ldc, lo, p.splits, part, s);
  }
}

template <typename T, int ACT, int TM, int TF> hipError_t gate_tiles(const FfnArgs& a, bool bwd, hipStream_t s) {
  constexpr size_t lds = lds_bytes(TM, 2 * TF);
  const T *x = static_cast<const T*>(a.x), *w_in = static_cast<const T*>(a.w_in);
  const int ntn = (a.F + TF - 1) / TF, grid = (a.M + TM - 1) / TM * ntn;
  hipError_t e;
  if (!bwd) {
    constexpr auto k = ffn_gate_kernel<T, ACT, TM, TF>;
    if ((e = allow_lds<k>(lds)) != hipSuccess) return e;
    k<<<grid, kThreads, lds, s>>>(x, w_in, static_cast<T*>(a.z), a.M, a.D, a.F, ntn);
  } else {
    constexpr auto k = ffn_dgate_kernel<T, ACT, TM, TF>;
    if ((e = allow_lds<k>(lds)) != hipSuccess) return e;
    k<<<grid, kThreads, lds, s>>>(x, w_in, static_cast<T*>(a.dpq), static_cast<T*>(a.z), a.M, a.D, a.F, ntn);
  }
  return hipGetLastError();
}

template <typename T, int ACT> hipError_t gate_go(const FfnArgs& a, int tile, bool bwd, hipStream_t s) {
  if (tile == kFew) {
    const T *x = static_cast<const T*>(a.x), *w_in = static_cast<const T*>(a.w_in);
    T *z = static_cast<T*>(a.z), *dpq = static_cast<T*>(a.dpq);
    return bwd ? few_go<T, true, kDgate, ACT>(x, w_in, z, dpq, a.M, a.F, a.D, a.D, 2LL * a.F, 0, 0, s)
               : few_go<T, true, kGate, ACT>(x, w_in, z, dpq, a.M, a.F, a.D, a.D, 2LL * a.F, 0, 0, s);
  }
  switch (tile) {
    case 0: return gate_tiles<T, ACT, 256, 128>(a, bwd, s);
    case 2: return gate_tiles<T, ACT, 128, 64>(a, bwd, s);
    default: return gate_tiles<T, ACT, 64, 64>(a, bwd, s);
  }
}

template <typename T, int ACT> hipError_t fwd_go(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  hipError_t e = gate_go<T, ACT>(a, p.gate.tile, false, s);
  if (e != hipSuccess) return e;
  return gemm_go<T, false, true>(p.y, static_cast<T*>(a.z), static_cast<const T*>(a.w_out), static_cast<T*>(a.y), a.M,
                                 a.D, a.F, a.F, a.D, a.D, a.part, s);
}

template <typename T, int ACT> hipError_t bwd_go(const FfnArgs& a, const FfnPlan& p, hipStream_t s) {
  const T *x = static_cast<const T*>(a.x), *w_in = static_cast<const T*>(a.w_in),
          *w_out = static_cast<const T*>(a.w_out), *dy = static_cast<const T*>(a.dy);
  T *z = static_cast<T*>(a.z), *dpq = static_cast<T*>(a.dpq);
  const long long F2 = 2LL * a.F;
  // dz = dy W_out^T into the place of dpq (W_out as stored is K contiguous for it): in bf16 as two
  // words, so that the second product with it rounds once
  hipError_t e = gemm_go<T, false, false>(p.dz, dy, w_out, dpq, a.M, a.F, a.D, a.D, a.D, F2, a.part, s, a.F);
  if (e != hipSuccess) return e;
  if ((e = gate_go<T, ACT>(a, p.gate.tile, true, s)) != hipSuccess) return e;
  // dx = dpq W_in^T: W_in as stored is K contiguous for it
  e = gemm_go<T, false, false>(p.dx, dpq, w_in, static_cast<T*>(a.dx), a.M, a.D, 2 * a.F, F2, F2, a.D, a.part, s);
  if (e != hipSuccess) return e;
  e = gemm_go<T, true, true>(p.dw_in, x, dpq, static_cast<T*>(a.dw_in), a.D, 2 * a.F, a.M, a.D, F2, F2, a.part, s);
  if (e != hipSuccess) return e;
  return gemm_go<T, true, true>(p.dw_out, z, dy, static_cast<T*>(a.dw_out), a.F, a.D, a.M, a.F, a.D, a.D, a.part, s);
}

// Tile and K splits of a product by an estimate of its time. Measured at 4096-deep
// products: a workgroup alone on a CU takes `alone` us per K tile of 128 bytes, several
// share the CU at `pace` each; every round of workgroups adds `round` us of first loads
// and stores (in proportion to the area: the stores of all CUs share HBM); splits write
// and read their partial sums at about 4 TB/s and add a launch.
FfnProduct choose(long long M, long long N, long long K, bool bf, bool may_split, bool gate) {
  static const double pace_bf[] = {1.15, 0.92, 0.35, 0.27}, alone_bf[] = {1.15, 0.92, 0.64, 0.53};
  static const double pace_f32[] = {4.4, 3.5, 1.5, 1.05}, alone_f32[] = {4.4, 3.5, 1.7, 1.2};
  static const double round[] = {9, 7, 2.5, 1.5};
  const long long kt = (K + (bf ? 63 : 31)) / (bf ? 64 : 32);
  FfnProduct best{0, 1};
  double best_us = 1e30;
  for (int c = 0; c < 4; ++c) {
    if (gate && c == 1) continue;
    const double pace = bf ? pace_bf[c] : pace_f32[c], alone = bf ? alone_bf[c] : alone_f32[c];
    const long long tiles = ((M + kTm[c] - 1) / kTm[c]) * ((N + kTn[c] - 1) / kTn[c]);
    for (int s = 1; s <= 32; ++s) {
      if (s > 1 && (!may_split || kt / s < 4 || tiles * s > 512)) break;
      const long long rounds = (tiles * s + 255) / 256;
      const double per = rounds * pace > alone ? rounds * pace : alone;
      double us = (kt + s - 1) / s * per + rounds * round[c] + 2;
      if (s > 1) us += 4 + (double)M * N * s * 8e-6 / 4;
      if (us < best_us) {
        best_us = us;
        best = FfnProduct{c, s};
      }
    }
  }
  return best;
}

}  // namespace

FfnPlan ffn_plan(int M, int D, int F, bool bf, bool bwd) {
  FfnPlan p{};
  const FfnProduct few{kFew, 1};
  const bool is_few = M <= kFewRows;
  auto need = [&](const FfnProduct& q, long long m, long long n) {
    const size_t f = q.splits > 1 ? (size_t)q.splits * m * n : 0;
    if (f > p.part_floats) p.part_floats = f;
  };
  p.gate = is_few ? few : choose(M, 2LL * F, D, bf, false, true);
  if (!bwd) {
    p.y = is_few ? few : choose(M, D, F, bf, true, false);
    need(p.y, M, D);
  } else {
    p.dz = is_few ? few : choose(M, F, D, bf, false, false);  // written into a wider matrix: not split
    p.dx = is_few ? few : choose(M, D, 2LL * F, bf, true, false);
    p.dw_in = choose(D, 2LL * F, M, bf, true, false);
    p.dw_out = choose(F, D, M, bf, true, false);
    need(p.dx, M, D);
    need(p.dw_in, D, 2LL * F);
    need(p.dw_out, F, D);
  }
  return p;
}

#define HY_FFN_DISPATCH(fn)                                                    \
  switch ((bf ? 3 : 0) + a.act) {                                              \
    case 0: return fn<float, HYENA_ACT_NONE>(a, p, s);                         \
    case 1: return fn<float, HYENA_ACT_SILU>(a, p, s);                         \
    case 2: return fn<float, HYENA_ACT_GELU>(a, p, s);                         \
    case 3: return fn<bf16, HYENA_ACT_NONE>(a, p, s);                          \
    case 4: return fn<bf16, HYENA_ACT_SILU>(a, p, s);                          \
    default: return fn<bf16, HYENA_ACT_GELU>(a, p, s);                         \
  }
hipError_t ffn_fwd(const FfnArgs& a, const FfnPlan& p, bool bf, hipStream_t s) { HY_FFN_DISPATCH(fwd_go) }
hipError_t ffn_bwd(const FfnArgs& a, const FfnPlan& p, bool bf, hipStream_t s) { HY_FFN_DISPATCH(bwd_go) }
#undef HY_FFN_DISPATCH

}  // namespace hy
