// ar_products.hip -- the experts' matrix products between dispatch and combine, and their gradients. Expert e owns the
// rows [offsets[e], offsets[e] + counts[e]) of the sorted buffers and the matrices w[e] ([out][in], as a linear layer
// keeps them):
//   gated     g = x w_gate^T, u = x w_up^T, h = act(g) u            (both products in one pass over x)
//   linear    y = x w^T
//   input     dx = dy w, or dx = dg w_gate + du w_up in one sum      (gradients towards the rows)
//   weight    dw[e] = dy^T x over the expert's rows, zero without rows
//   slopes    dg = dh u act'(g), du = dh act(g)
//
// One tile kernel serves all of them. A workgroup computes a BM x BN tile of the result with matrix instructions
// (16 x 16 results from 16 bytes of either operand per lane, fp32 sums); operands pass through LDS in steps of 128 bytes
// along the sum, two buffers in turn. An operand lies in memory either along the sum (rows of x, dy, and of w in the
// forward products: "KC") or across it (w for the rows' gradients, x and dy for the weights': "KS"); the second kind is
// kept in LDS as it lies and transposed on the way to registers (ds_read_tr for 16-bit types), so no operand is
// ever transposed in memory.
//
// The host does not know the segments, so a tile's expert and rows are found on the device: a wave sums the experts'
// tile counts (64 experts a step) and the grid is as large as any segments of so many rows need.
#include "ar_block.h"
#include "ar_internal.h"
#include "ar_products.h"

namespace ar {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define AR_LDS __attribute__((address_space(3)))

constexpr int kStep = 128;            // bytes of the sum per step and row
constexpr int kChunks = kStep / 16;   // 16-byte chunks of a step

enum Kind { kGated = 0, kLinear = 1, kInput = 2, kWeight = 3 };

// ------------------------------------------------------------------------------------------ segments
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// First row and row count of expert e's segment, whatever the tables hold: never outside [0, rows).
__device__ __forceinline__ void segment(const ProductArgs& a, int e, int* first, int* n) {
  if (!a.offsets) {
    *first = 0;
    *n = a.rows;
    return;
  }
  const int lo = gptr<int32_t>(a.offsets)[e];
  int m = a.counts ? gptr<int32_t>(a.counts)[e] : static_cast<int>(static_cast<uint32_t>(gptr<int32_t>(a.offsets)[e + 1]) -
                                                                   static_cast<uint32_t>(lo));
  if (lo < 0 || lo >= a.rows || m < 0) m = 0;
  *first = m > 0 ? lo : 0;
  *n = m < a.rows - *first ? m : a.rows - *first;
}

// Tiles of expert e: its elements (rows * width) over `unit`.
__device__ __forceinline__ int tiles_of(const ProductArgs& a, int e, int64_t width, int unit) {
  int first, n;
  segment(a, e, &first, &n);
  return static_cast<int>((n * width + unit - 1) / unit);
}

// Tiles of all experts. All lanes of a wave take part; the result is the same in each.
__device__ __forceinline__ int all_tiles(const ProductArgs& a, int64_t width, int unit) {
  if (!a.offsets) return tiles_of(a, 0, width, unit);
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int e = lane; e < a.experts; e += 64) sum += tiles_of(a, e, width, unit);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
  return uniform(sum);
}

// The expert that tile t (below all_tiles) belongs to, and the tile's number among the expert's.
__device__ __forceinline__ void find_tile(const ProductArgs& a, int t, int64_t width, int unit, int* expert, int* index) {
  *expert = 0;
  *index = t;
  if (!a.offsets) return;
  const int lane = threadIdx.x & 63;
  for (int e0 = 0, before = 0; e0 < a.experts; e0 += 64) {
    const int own = e0 + lane < a.experts ? tiles_of(a, e0 + lane, width, unit) : 0;
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(upto, d, 64);
      if (lane >= d) upto += y;
    }
    upto += before;
    const uint64_t mine = __ballot(t >= upto - own && t < upto);
    if (mine) {
      const int l = __builtin_ctzll(mine);
      *expert = uniform(e0 + l);
      *index = uniform(t - __shfl(upto - own, l, 64));
      return;
    }
    before = __shfl(upto, 63, 64);
  }
}

// ------------------------------------------------------------------------------------------ operands
// Products of 16-byte fragments: lane l holds row l % 16 and the (l / 16)-th chunk along the sum. fp32 takes four
// instructions of four sums each; which sums meet in one instruction does not matter as long as both operands agree.
template <int DT> __device__ __forceinline__ f32x4 mma(const u32x4& x, const u32x4& y, f32x4 c) {
  if constexpr (DT == AR_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  } else if constexpr (DT == AR_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[i]), __uint_as_float(y[i]), c, 0, 0, 0);
    return c;
  }
}

// How an operand's tile lies in LDS, in 16-byte chunks. KC: [row][8 chunks along the sum]; KS: [sum][row chunks]. Chunks
// are exchanged within an LDS row by an exclusive or, so that the 64 lanes of a fragment read spread over all banks.
//   KC, rows in order:  16 rows a read, one chunk each: bits 1 to 3 of the row (bit 0 is the half of the 256-byte bank
//                       row that it lies in).
//   KC, PAIRED:         the read takes rows 0-3, 8-11, 16-19, 24-27 (see n_of): bits 1, 3 and 4.
//   KS, 16-bit:         4 rows of the sum of 32 bytes each for 16 lanes, the next 16 lanes 8 rows on.
//   KS, fp32:           one row of the sum of 64 bytes for 16 lanes, the next 16 lanes 4 rows on.
template <bool PAIRED> __device__ __forceinline__ int mix_kc(int row) {
  return PAIRED ? ((row >> 1) & 1) | ((row >> 2) & 6) : (row >> 1) & 7;
}
template <int DT> __device__ __forceinline__ int mix_ks(int k) {
  if constexpr (Traits<DT>::kSize == 2) return ((k & 3) << 1) | (k & 8);
  else return k & 12;
}

// The column (0 to 63 of a wave's 64) of result element i of lane group q in subtile j. KS operands: in order. KC operands:
// PAIRED, two subtiles give a lane 8 neighbours, which it stores together.
template <bool PAIRED> __device__ __forceinline__ int n_of(int j, int q, int i) {
  return PAIRED ? (j / 2) * 32 + q * 8 + (j % 2) * 4 + i : j * 16 + q * 4 + i;
}

// One operand's tile of R rows, for NT threads: from memory through registers into LDS.
template <int DT, bool KS, bool PAIRED, int R, int NT> struct Tile {
  static constexpr int V = Traits<DT>::kVec, ES = Traits<DT>::kSize;
  static constexpr int kRowChunks = KS ? R / V : kChunks;      // chunks of an LDS row
  static constexpr int kLoads = R * kChunks / NT;               // chunks a thread moves
  static constexpr int kStride = NT / kRowChunks;               // LDS rows between a thread's chunks
  static_assert(R * kChunks % NT == 0 && NT % kRowChunks == 0, "whole loads");
  static_assert(KS ? (kStride % 4 == 0) : (kStride % 32 == 0), "a thread's chunks are mixed alike");

  uint32_t at[kLoads];  // KC: byte offset of the row (clamped to the last one)
  int lds_row, chunk;   // of the first chunk: where it lies in LDS, and the chunk of the row in memory
  int limit;            // KS: rows (columns in memory) left in the matrix from the tile's first

  // `map` turns an LDS row into a row of the tile; rows past `nrows` repeat the last one, and their results go nowhere.
  template <class Map> __device__ __forceinline__ void init(int nrows, uint32_t stride, Map map) {
    const int tid = threadIdx.x;
    lds_row = tid / kRowChunks;
    limit = nrows;
    if constexpr (!KS) {
      chunk = (tid % kRowChunks) ^ mix_kc<PAIRED>(lds_row);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = map(lds_row + i * kStride);
        at[i] = static_cast<uint32_t>(r < nrows ? r : nrows - 1) * stride;
      }
    }
  }

  // Reads the step of the sum that starts `k0` elements in: `base` is the matrix at the tile's first row and sum element
  // 0; what lies past `K` is zero.
  __device__ __forceinline__ void fetch(u32x4 (&v)[kLoads], const char* base, uint32_t stride, int k0, int K) const {
    if constexpr (!KS) {
      const int k = k0 + chunk * V;
      const char* p = base + static_cast<int64_t>(k) * ES;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (k + V <= K) v[i] = ldu16(p + at[i]);
        else v[i] = part(p + at[i], K - k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int row = lds_row + i * kStride, k = k0 + row;
        const int c = ((static_cast<int>(threadIdx.x) % kRowChunks) ^ mix_ks<DT>(row)) * V;
        const char* p = base + static_cast<int64_t>(k) * stride + c * ES;
        if (k < K && c + V <= limit) v[i] = ldu16(p);
        else v[i] = part(p, k < K ? limit - c : 0);
      }
    }
  }
  // The first n elements of a chunk, zeros behind them.
  __device__ static __forceinline__ u32x4 part(const char* p, int n) {
    u32x4 w = {0, 0, 0, 0};
    if (n <= 0) return w;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t bits = i < n ? load_elem<DT>(p, i) : 0;
      if constexpr (ES == 2) w[i >> 1] |= bits << (16 * (i & 1));
      else w[i] = bits;
    }
    return w;
  }
  __device__ __forceinline__ void put(const u32x4 (&v)[kLoads], AR_LDS char* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *(AR_LDS u32x4*)(lds + (threadIdx.x + i * NT) * 16) = v[i];
  }

  // Fragment of rows r0 to r0 + 15 (KC, PAIRED: the 16 rows of subtile `r0 / 16`), chunks 4 kk to 4 kk + 3 of the step.
  __device__ static __forceinline__ u32x4 read(const AR_LDS char* lds, int r0, int kk) {
    const int l = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    if constexpr (!KS) {
      const int j = (r0 / 16) & 3;
      const int row = PAIRED ? (r0 & ~63) + n_of<true>(j, l >> 2, l & 3) : r0 + l;
      return *(const AR_LDS u32x4*)(lds + row * kStep + (((kk * 4 + q) ^ mix_kc<PAIRED>(row)) * 16));
    } else if constexpr (ES == 2) {
      const int k = kk * 32 + q * 8 + (l >> 2), c = r0 + (l & 3) * 4;
      const AR_LDS char* p = lds + k * (R * ES) + (((c / V) ^ mix_ks<DT>(k)) * 16) + (c % V) * ES;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS i16x4*)(p));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS i16x4*)(p + 4 * R * ES));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kk * 16 + q * 4 + i, c = r0 + l;
        w[i] = *(const AR_LDS uint32_t*)(lds + k * (R * ES) + (((c / V) ^ mix_ks<DT>(k)) * 16) + (c % V) * ES);
      }
      return w;
    }
  }
};

// ------------------------------------------------------------------------------------------ activations
// value: act(x); slope: act'(x). fp32 results take the accurate exponential, 16-bit ones the instruction (its error grows
// with the exponent, |x| 2^-24, far below their rounding). The normal distribution comes from erfc, which keeps its
// digits where 1 + erf cancels.
template <int DT> __device__ __forceinline__ float exp_of(float x) { return DT == AR_F32 ? expf(x) : __expf(x); }
template <int DT, bool SLOPE> __device__ __forceinline__ void activate(int act, float x, float* value, float* slope) {
  if (act == AR_ACT_SILU) {
    const float p = 1.0f / (1.0f + exp_of<DT>(-x));
    *value = x * p;
    if constexpr (SLOPE) *slope = p * (1.0f + x * (1.0f - p));
  } else if (act == AR_ACT_GELU) {
    const float p = 0.5f * erfcf(x * -0.70710678118654752f);
    *value = x * p;
    if constexpr (SLOPE) *slope = p + x * (0.39894228040143268f * exp_of<DT>(-0.5f * x * x));
  } else {
    // 1 + tanh(z) = 2 s and 1 - tanh(z)^2 = 4 s (1 - s), with s the logistic function of 2 z
    constexpr float a = 0.79788456080286536f, b = 0.044715f;
    const float s = 1.0f / (1.0f + exp_of<DT>(-2.0f * a * (x + b * x * x * x)));
    *value = x * s;
    // the second term is 0 far out, where its last factor leaves the range
    if constexpr (SLOPE)
      *slope = s + (fabsf(x) < 64.0f ? 2.0f * a * x * s * (1.0f - s) * (1.0f + 3.0f * b * x * x) : 0.0f);
  }
}

// ------------------------------------------------------------------------------------------ results
// N neighbouring elements of a row to p, of which `left` lie in the row.
template <int DT, int N> __device__ __forceinline__ void store_run(char* p, const float* v, int left) {
  if constexpr (Traits<DT>::kSize == 4) {
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(v[i + k]);
        stu16(p + 4 * i, w);
      }
      return;
    }
  } else {
    if (left >= N) {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = narrow<DT>(v[2 * i]) | narrow<DT>(v[2 * i + 1]) << 16;
      if constexpr (N == 8) stu16(p, u32x4{w[0], w[1], w[2], w[3]});
      else *gptr<u32x2_a1>(p) = u32x2{w[0], w[1]};
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < left) store_elem<DT>(p, i, narrow<DT>(v[i]));
}

// ------------------------------------------------------------------------------------------ the tile kernel
template <int KIND> constexpr bool kRowsKS = KIND == kWeight;                        // operand of the tile's rows
template <int KIND> constexpr bool kColsKS = KIND == kWeight || KIND == kInput;      // operand of its columns

template <int DT, int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(const ProductArgs a) {
  constexpr int NT = WM * WN * 64, ES = Traits<DT>::kSize, K_STEP = kStep / ES;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool PAIRED = !kColsKS<KIND>;
  static_assert(BN / WN == 64, "a wave has 64 columns");
  constexpr int COLS = KIND == kGated ? BN / 2 : BN;  // columns of the result
  using A = Tile<DT, kRowsKS<KIND>, false, BM, NT>;
  using B = Tile<DT, kColsKS<KIND>, PAIRED, BN, NT>;
  __shared__ __align__(128) char smem[2][(BM + BN) * kStep];
  const int wave = uniform(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int l = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;

  // Tiles of the result: rows of it per expert (weight: of every matrix) and columns.
  const int across = (a.n + COLS - 1) / COLS;
  int down, total;
  if constexpr (KIND == kWeight) {
    down = (a.m + BM - 1) / BM;
    total = a.experts * (a.a1 ? 2 : 1) * down * across;
  } else {
    down = min(all_tiles(a, 1, BM), a.most);
    total = down * across;
  }
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    // which tile
    int e, mt, nt, which = 0, first, n, K;
    if constexpr (KIND == kWeight) {
      nt = id % across;
      mt = id / across % down;
      const int z = id / (across * down);
      e = a.a1 ? z >> 1 : z;
      which = a.a1 ? z & 1 : 0;
    } else {
      nt = id % across;
      find_tile(a, id / across, 1, BM, &e, &mt);
    }
    segment(a, e, &first, &n);
    first = uniform(first);
    n = uniform(n);
    const int m0 = mt * BM, n0 = nt * COLS;
    if (KIND != kWeight && m0 >= n) continue;  // tables that describe no segments
    // the operands at the tile's first row or column and sum element 0
    const char *pa, *pb, *pa1 = nullptr, *pb1 = nullptr;
    uint32_t sa, sb;
    int rows_left, cols_left = a.n - n0;
    A ta;
    B tb;
    const int64_t wofs = static_cast<int64_t>(e) * a.w_stride * ES;
    if constexpr (KIND == kWeight) {
      sa = static_cast<uint32_t>(a.m) * ES;
      sb = static_cast<uint32_t>(a.n) * ES;
      rows_left = a.m - m0;
      K = n;
      pa = static_cast<const char*>(which ? a.a1 : a.a0) + static_cast<int64_t>(first) * sa + static_cast<int64_t>(m0) * ES;
      pb = static_cast<const char*>(a.b0) + static_cast<int64_t>(first) * sb + static_cast<int64_t>(n0) * ES;
    } else {
      sa = static_cast<uint32_t>(a.k) * ES;
      rows_left = n - m0;
      K = a.k;
      const int64_t ofs = static_cast<int64_t>(first + m0) * sa;
      pa = static_cast<const char*>(a.a0) + ofs;
      if (a.a1) pa1 = static_cast<const char*>(a.a1) + ofs;
      sb = static_cast<uint32_t>(KIND == kInput ? a.n : a.k) * ES;
      const int64_t col = wofs + static_cast<int64_t>(n0) * (KIND == kInput ? ES : sb);
      pb = static_cast<const char*>(a.b0) + col;
      if (a.b1) pb1 = static_cast<const char*>(a.b1) + col;
    }
    ta.init(rows_left, sa, [](int r) { return r; });
    if constexpr (KIND == kGated) {
      // a wave's 64 columns are 32 of w_gate and the same 32 of w_up
      tb.init(cols_left, sb, [](int r) { return (r / 64) * 32 + r % 32; });
    } else {
      tb.init(cols_left, sb, [](int r) { return r; });
    }
    const int steps1 = (K + K_STEP - 1) / K_STEP, steps = KIND == kInput && a.b1 ? 2 * steps1 : steps1;

    f32x4 acc[NI][MI];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0, 0, 0, 0};

    u32x4 va[A::kLoads], vb[B::kLoads];
    auto fetch = [&](int s) {
      const bool second = s >= steps1;
      const int k0 = (second ? s - steps1 : s) * K_STEP;
      ta.fetch(va, second ? pa1 : pa, sa, k0, K);
      if constexpr (KIND == kGated) {
        // rows 32 to 63 of every 64 in LDS are of w_up; whole waves read one matrix
#pragma unroll
        for (int i = 0; i < B::kLoads; ++i) {
          const int r = tb.lds_row + i * B::kStride, k = k0 + tb.chunk * B::V;
          const char* p = ((r & 32) ? pb1 : pb) + static_cast<int64_t>(k) * ES + tb.at[i];
          vb[i] = k + B::V <= K ? ldu16(p) : B::part(p, K - k);
        }
      } else {
        tb.fetch(vb, second ? pb1 : pb, sb, k0, K);
      }
    };
    auto put = [&](int s) {
      AR_LDS char* at = (AR_LDS char*)(smem[s & 1]);
      ta.put(va, at);
      tb.put(vb, at + BM * kStep);
    };
    if (steps > 0) {
      fetch(0);
      put(0);
    }
    for (int s = 0; s < steps; ++s) {
      __syncthreads();  // the buffer of this step is filled, and nobody reads the other one any more
      if (s + 1 < steps) fetch(s + 1);
      const AR_LDS char* at = (const AR_LDS char*)(smem[s & 1]);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        u32x4 fb[NI], fa[MI];
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[j] = B::read(at + BM * kStep, wn * 64 + j * 16, kk);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = A::read(at, wm * (BM / WM) + i * 16, kk);
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int i = 0; i < MI; ++i) acc[j][i] = mma<DT>(fb[j], fa[i], acc[j][i]);
      }
      if (s + 1 < steps) put(s + 1);
    }
    __syncthreads();  // the next tile's first step goes to the buffer that slower waves may still read

    // results: lane l of group q has row l of every 16 and four neighbouring columns of every subtile
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = wm * (BM / WM) + i * 16 + l;
      if (r >= rows_left) continue;
      if constexpr (KIND == kGated) {
        const int c = wn * 32 + q * 8, left = a.n - n0 - c;
        if (left <= 0) continue;
        const int64_t ofs = (static_cast<int64_t>(first + m0 + r) * a.n + n0 + c) * ES;
        float g[8], u[8], h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          g[k] = acc[k / 4][i][k % 4];
          u[k] = acc[2 + k / 4][i][k % 4];
          activate<DT, false>(a.act, g[k], &h[k], nullptr);
          h[k] *= u[k];
        }
        store_run<DT, 8>(static_cast<char*>(a.c0) + ofs, h, left);
        if (a.c1) {
          store_run<DT, 8>(static_cast<char*>(a.c1) + ofs, g, left);
          store_run<DT, 8>(static_cast<char*>(a.c2) + ofs, u, left);
        }
      } else {
        char* out;
        if constexpr (KIND == kWeight)
          out = static_cast<char*>(which ? a.c1 : a.c0) +
                (static_cast<int64_t>(e) * a.c_stride + static_cast<int64_t>(m0 + r) * a.n + n0) * ES;
        else out = static_cast<char*>(a.c0) + (static_cast<int64_t>(first + m0 + r) * a.n + n0) * ES;
        constexpr int RUN = PAIRED ? 8 : 4;
#pragma unroll
        for (int j = 0; j < NI; j += RUN / 4) {
          const int c = wn * 64 + n_of<PAIRED>(j, q, 0), left = a.n - n0 - c;
          float v[RUN];
#pragma unroll
          for (int k = 0; k < RUN; ++k) v[k] = acc[j + k / 4][i][k % 4];
          if (left > 0) store_run<DT, RUN>(out + c * ES, v, left);
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ slopes
// dg and du of an expert's rows; a segment's rows lie one behind the other, so its elements are walked in a row.
constexpr int kSlopeUnit = 8192, kSlopeThreads = 256;

template <int DT> __global__ __launch_bounds__(kSlopeThreads) void slopes_kernel(const ProductArgs a) {
  constexpr int V = Traits<DT>::kVec, ES = Traits<DT>::kSize;
  const int total = min(all_tiles(a, a.n, kSlopeUnit), a.most);
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    int e, t, first, n;
    find_tile(a, id, a.n, kSlopeUnit, &e, &t);
    segment(a, e, &first, &n);
    const int64_t base = static_cast<int64_t>(uniform(first)) * a.n + static_cast<int64_t>(t) * kSlopeUnit;
    const int64_t rest = static_cast<int64_t>(uniform(n)) * a.n - static_cast<int64_t>(t) * kSlopeUnit;
    if (rest <= 0) continue;  // tables that describe no segments
    const int len = rest < kSlopeUnit ? static_cast<int>(rest) : kSlopeUnit;
    for (int i = threadIdx.x * V; i < len; i += kSlopeThreads * V) {
      const int64_t ofs = (base + i) * ES;
      const char *pd = static_cast<const char*>(a.a0) + ofs, *pg = static_cast<const char*>(a.b0) + ofs,
                 *pu = static_cast<const char*>(a.b1) + ofs;
      char *og = static_cast<char*>(a.c0) + ofs, *ou = static_cast<char*>(a.c1) + ofs;
      float d[V], g[V], u[V];
      const int left = len - i;
      if (left >= V) {
        Slot<DT>::unpack(ldu16(pd), d);
        Slot<DT>::unpack(ldu16(pg), g);
        Slot<DT>::unpack(ldu16(pu), u);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const bool in = k < left;
          d[k] = in ? widen<DT>(load_elem<DT>(pd, k)) : 0.0f;
          g[k] = in ? widen<DT>(load_elem<DT>(pg, k)) : 0.0f;
          u[k] = in ? widen<DT>(load_elem<DT>(pu, k)) : 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float value, slope;
        activate<DT, true>(a.act, g[k], &value, &slope);
        g[k] = d[k] * u[k] * slope;
        u[k] = d[k] * value;
      }
      store_run<DT, V>(og, g, left);
      store_run<DT, V>(ou, u, left);
    }
  }
}

// ------------------------------------------------------------------------------------------ launches
int grid_of(int64_t most, int per_cu) {
  const int64_t cap = static_cast<int64_t>(cu_count()) * per_cu;
  return static_cast<int>(most < cap ? most : cap);
}

template <int DT, int KIND> hipError_t launch_tiles(ProductArgs a, hipStream_t s) {
  constexpr int BM = 128, BN = 128, COLS = KIND == kGated ? BN / 2 : BN;
  const int64_t across = tiles_up(a.n, COLS);
  const int64_t down = KIND == kWeight ? matrices(a) * tiles_up(a.m, BM) : row_tiles(a, 1, BM);
  a.most = static_cast<int>(down);
  if (down == 0) return hipSuccess;
  tile_kernel<DT, KIND, BM, BN, 2, 2><<<grid_of(down * across, 2), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int KIND> hipError_t launch_kind(const ProductArgs& a, int dtype, hipStream_t s) {
  if (dtype == AR_BF16) return launch_tiles<AR_BF16, KIND>(a, s);
  if (dtype == AR_F16) return launch_tiles<AR_F16, KIND>(a, s);
  return launch_tiles<AR_F32, KIND>(a, s);
}

}  // namespace

hipError_t launch_gated(const ProductArgs& a, int dtype, hipStream_t s) { return launch_kind<kGated>(a, dtype, s); }
hipError_t launch_linear(const ProductArgs& a, int dtype, hipStream_t s) { return launch_kind<kLinear>(a, dtype, s); }
hipError_t launch_input_grad(const ProductArgs& a, int dtype, hipStream_t s) { return launch_kind<kInput>(a, dtype, s); }
hipError_t launch_weight_grad(const ProductArgs& a, int dtype, hipStream_t s) { return launch_kind<kWeight>(a, dtype, s); }

hipError_t launch_slopes(ProductArgs a, int dtype, hipStream_t s) {
  a.most = static_cast<int>(row_tiles(a, a.n, kSlopeUnit));
  if (a.most == 0) return hipSuccess;
  const int grid = grid_of(a.most, 8);
  if (dtype == AR_BF16) slopes_kernel<AR_BF16><<<grid, kSlopeThreads, 0, s>>>(a);
  else if (dtype == AR_F16) slopes_kernel<AR_F16><<<grid, kSlopeThreads, 0, s>>>(a);
  else slopes_kernel<AR_F32><<<grid, kSlopeThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ar
