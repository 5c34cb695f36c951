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
// along the sum. An operand lies in memory either along the sum (rows of x, dy, and of w in the forward products: "KC")
// or across it (w for the rows' gradients, x and dy for the weights': "KS"); the second kind is kept in LDS as it lies and
// transposed on the way to registers (ds_read_tr for 16-bit types), so no operand is ever transposed in memory.
//
// The host does not know the segments, so a tile's expert and rows are found on the device: a wave sums the experts'
// tile counts (64 experts a step) and the grid is as large as any segments of so many rows need.
//
// Sums are fp32 and rounded once, to the results' type. The gated gradient rounds dg and du to it before the two products
// that read them, which take 16-bit operands anyway: the gradients' error is sqrt(2) of one rounding's (bf16 0.0023 of the norm
// for 0.0017, fp16 0.00029 for 0.00021).
//
// What bounds it: with many rows, the matrix instructions and the power they draw, and whole rounds of tiles. Rates of calls in a
// row, bf16, next to one library product of the same size: 32,768 rows of one matrix, gated 2 x 2048 x 4096 with both products
// kept 1,230 TF (library 1,530), linear 4096 x 4096 1,340 (1,530), dx 1,330 (1,330), dw 1,380 (1,200). The same gated rows at 32
// experts, spread evenly 1,160 TF; as a router leaves them 990 (1.10 ms): tiles that are not full make 2,368 of 2,048, 10 rounds
// of 256 in the place of 8. A dense 16,384 x 4160 x 4096: matrix units busy 74% of the time, 1,300 TF, and 1,430 on
// zeros, which draw less power.
// With few rows, reading the weights: 4.9 TB/s (a copy reaches 4.8). Weights' gradients of few rows, writing them: 268 MB in
// 80 us, and 0.19 us more for every row of 16 experts of 4096 x 2048. Rows of odd numbers of 16-bit elements (or odd
// addresses) cannot be loaded straight into LDS, and take twice to four and a half times as long: 16 experts of 2049 x 2049
// (of 2048 x 2048), 2,048 rows: forward 129 us (42), dx 126 (38), dw 164 (54); 16,384 rows 544 (121), 535 (121), 562 (139). Rows of
// 2050, whose last chunk is mended: 80, 54, 74; 292, 220, 175.
// A sum is never split over workgroups: dw of few tiles over many rows leaves most of the GPU idle (64 x 64 to 256 x 256 over 8,192
// rows 42 to 48 us in bf16, 210 in fp32; 16 of 2048 x 2048 with 16,384 rows at one expert 326 us, spread evenly 138).
#include "ar_block.h"
#include "ar_internal.h"
#include "ar_products.h"

#include <type_traits>

namespace ar {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define AR_LDS __attribute__((address_space(3)))

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

// The segments of the first 64 experts, one a lane, held from the count of all tiles to the search for one.
struct Lane {
  int first, n;
};
__device__ __forceinline__ Lane lane_segment(const ProductArgs& a, int e) {
  Lane s{0, 0};
  if (e < a.experts) segment(a, e, &s.first, &s.n);
  return s;
}
// Tiles of n rows: their elements (n * width) over `unit`.
__device__ __forceinline__ int tiles_of(int n, int64_t width, int unit) { return static_cast<int>((n * width + unit - 1) / unit); }

// Tiles of all experts. All lanes of a wave take part; the result is the same in each.
__device__ __forceinline__ int all_tiles(const ProductArgs& a, const Lane& own, int64_t width, int unit) {
  if (!a.offsets) return tiles_of(a.rows, width, unit);
  int sum = tiles_of(own.n, width, unit);
  for (int e = (threadIdx.x & 63) + 64; e < a.experts; e += 64) sum += tiles_of(lane_segment(a, e).n, width, unit);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
  return uniform(sum);
}

// Tile t of all: its expert, its number among the expert's tiles, and the expert's rows. False if no expert has it.
struct Place {
  int expert, index, first, n;
};
__device__ __forceinline__ bool find_tile(const ProductArgs& a, const Lane& mine, int t, int64_t width, int unit, Place* at) {
  if (!a.offsets) {
    *at = Place{0, t, 0, a.rows};
    return true;
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0, before = 0; e0 < a.experts; e0 += 64) {
    const Lane s = e0 == 0 ? mine : lane_segment(a, e0 + lane);
    const int own = tiles_of(s.n, width, unit);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(upto, d, 64);
      if (lane >= d) upto += y;
    }
    upto += before;
    const uint64_t has = __ballot(t >= upto - own && t < upto);
    if (has) {
      const int l = __builtin_ctzll(has);
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      *at = Place{uniform(e0 + l), t - of(upto - own), of(s.first), of(s.n)};
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
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

// How an operand's tile lies in LDS, in 16-byte chunks. KC: [row][CH chunks along the sum]; KS: [sum][row chunks]. Chunks
// are exchanged within an LDS row by an exclusive or, so that the 64 lanes of a fragment read spread over all banks (no
// conflicts were counted).
//   KC: 16 rows a read, one chunk each, and the next chunk for the next 16 lanes. With 8 chunks in an LDS row, bits 1 to 3
//       of the row (bit 0 is the half of the 256-byte bank row that it lies in); with 4, bits 2 and 3 in Gray order.
//       PAIRED reads take rows 0-3, 8-11, 16-19, 24-27 (see n_of): bits 3 and 4 in the place of 2 and 3.
//   KS, 16-bit: 4 rows of the sum of 32 bytes each for 16 lanes, the next 16 lanes 8 rows on.
//   KS, fp32: one row of the sum of 64 bytes for 16 lanes, the next 16 lanes 4 rows on.
template <int CH, bool PAIRED> __device__ __forceinline__ int mix_kc(int row) {
  if constexpr (CH == 8) return PAIRED ? ((row >> 1) & 1) | ((row >> 2) & 6) : (row >> 1) & 7;
  const int t = PAIRED ? row >> 3 : row >> 2;
  return ((t >> 1) & 1) | ((t ^ (t >> 1)) & 1) << 1;
}
//   KS with 128-byte LDS rows: two of them share a bank row, and 8 chunks are there to exchange.
template <int DT, int R> __device__ __forceinline__ int mix_ks(int k) {
  if constexpr (Traits<DT>::kSize == 4) return k & 12;
  else if constexpr (R * 2 >= 256) return ((k & 3) << 1) | (k & 8);
  else return (k & 2) | ((k & 8) >> 1);
}

// The column (0 to 63 of a wave's 64) of result element i of lane group q in subtile j. KS operands: in order. KC operands:
// PAIRED, two subtiles give a lane 8 neighbours, which it stores together.
template <bool PAIRED> __device__ __forceinline__ int n_of(int j, int q, int i) {
  return PAIRED ? (j / 2) * 32 + q * 8 + (j % 2) * 4 + i : j * 16 + q * 4 + i;
}

// 16 bytes per lane from memory straight into LDS: lane l's go to `lds` (uniform, an LDS byte address) + 16 l. `base` and
// `bytes` are uniform too; a lane whose offset reaches `bytes` gets zeros. Nothing waits here (see ready).
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ void load_lds(const char* base, uint32_t bytes, uint32_t at, uint32_t lds) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  auto scalar = [](uint32_t v) { return static_cast<uint32_t>(uniform(static_cast<int>(v))); };
  const u32x4 rsrc = {scalar(static_cast<uint32_t>(b)), scalar(static_cast<uint32_t>(b >> 32) & 0xFFFFu), scalar(bytes), 0x00020000u};
  // m0 is named as overwritten, so that nothing the compiler put there is taken to outlive the statement (it warns that m0 is
  // a register it does not allocate; the build leaves that warning out)
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(at), "s"(rsrc), "s"(scalar(lds))
               : "memory", "m0");
}
// All but the last N of a wave's loads have landed and its reads of LDS are done, for all waves of the workgroup.
template <int N> __device__ __forceinline__ void ready() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The first n elements of a 16-byte chunk, zeros behind them.
template <int DT> __device__ __forceinline__ u32x4 first_elements(const char* p, int n) {
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Traits<DT>::kVec; ++i) {
    const uint32_t bits = i < n ? load_elem<DT>(p, i) : 0;
    if constexpr (Traits<DT>::kSize == 2) w[i >> 1] |= bits << (16 * (i & 1));
    else w[i] = bits;
  }
  return w;
}

// One operand's tile of R rows and CH chunks of the sum, for NT threads: from memory through registers into LDS, or (DIRECT)
// straight into it, for rows and addresses that are multiples of 4 bytes.
template <int DT, bool KS, bool PAIRED, bool DIRECT, int CH, int R, int NT> struct Tile {
  static constexpr int V = Traits<DT>::kVec, ES = Traits<DT>::kSize;
  static constexpr int kRowChunks = KS ? R / V : CH;           // chunks of an LDS row
  static constexpr int kLoads = R * CH / NT;                    // chunks a thread moves
  static constexpr int kStride = NT / kRowChunks;               // LDS rows between a thread's chunks
  static_assert(R * CH % NT == 0 && NT % kRowChunks == 0, "whole loads");
  static_assert(KS ? (kStride % 4 == 0) : (kStride % 32 == 0), "a thread's chunks are mixed alike");

  uint32_t at[kLoads];  // KC: byte offset of the row (clamped to the last one). DIRECT: of the chunk in the step
  int lds_row, chunk;   // of the first chunk: where it lies in LDS, and the chunk of the row in memory
  int limit;            // KS: rows (columns in memory) left in the matrix from the tile's first

  // `map` turns an LDS row into a row of the tile; rows past `nrows` repeat the last one, and their results go nowhere.
  template <class Map> __device__ __forceinline__ void init(int nrows, uint32_t stride, Map map) {
    const int tid = threadIdx.x;
    lds_row = tid / kRowChunks;
    limit = nrows;
    if constexpr (!KS) {
      chunk = (tid % kRowChunks) ^ mix_kc<CH, PAIRED>(lds_row);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = map(lds_row + i * kStride);
        at[i] = static_cast<uint32_t>(r < nrows ? r : nrows - 1) * stride + (DIRECT ? chunk * 16 : 0);
      }
    } else if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = lds_row + i * kStride;
        at[i] = static_cast<uint32_t>(k) * stride + (static_cast<uint32_t>(tid % kRowChunks) ^ mix_ks<DT, R>(k)) * 16;
      }
    }
  }

  // Load i of a step of the sum straight into LDS. `base` is the matrix at the tile's first row and the step's first element;
  // what lies `bytes` or more behind it, and (KC) chunks that are not `in` the sum, leave zeros. (KS: a chunk past a row's
  // end reads the start of the next ones, whose results go nowhere.)
  __device__ __forceinline__ void load(int i, const char* base, uint32_t bytes, bool in, uint32_t to) const {
    load_lds(base, bytes, KS || in ? at[i] : kNowhere, to + i * NT * 16);
  }

  // KC: zeros for the elements of the chunk that the end of the sum cuts, `n` elements into the step: their loads brought the
  // next row's first ones.
  __device__ __forceinline__ static void cut(AR_LDS char* lds, int n) {
    static_assert(!KS, "across the sum, whole rows are left out");
#pragma unroll
    for (int row = threadIdx.x; row < R; row += NT) {
      AR_LDS char* p = lds + row * (CH * 16) + ((n / V) ^ mix_kc<CH, PAIRED>(row)) * 16;
      for (int e = n % V; e < V; ++e) {
        if constexpr (ES == 2) ((AR_LDS uint16_t*)p)[e] = 0;
        else ((AR_LDS uint32_t*)p)[e] = 0;
      }
    }
  }

  // Chunk i of the step of the sum that starts at element k0, through a register. `base` is the matrix at the tile's first row
  // and that element, `left` the bytes from there to its end (KC: to the end of the tile's last row); elements past K are
  // zero. A chunk that a row's end cuts is read on into the next row where there is one.
  __device__ __forceinline__ u32x4 fetch(int i, const char* base, uint32_t stride, uint32_t left, int k0, int K) const {
    if constexpr (!KS) {
      const int n = K - k0 - chunk * V;
      const uint32_t at_byte = at[i] + chunk * 16;
      if (n <= 0) return u32x4{0, 0, 0, 0};
      if (!chunk_inside(at_byte, left)) return first_elements<DT>(base + at_byte, n);
      u32x4 w = ldu16(base + at_byte);
      if (k0 + CH * V > K) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (ES == 2) w[j] &= 2 * j + 1 < n ? ~0u : 2 * j < n ? 0xFFFFu : 0u;
          else w[j] &= j < n ? ~0u : 0u;
        }
      }
      return w;
    } else {
      const int row = lds_row + i * kStride;
      const int c = ((static_cast<int>(threadIdx.x) % kRowChunks) ^ mix_ks<DT, R>(row)) * V;
      const uint32_t at_byte = static_cast<uint32_t>(row) * stride + c * ES;
      if (k0 + row >= K) return u32x4{0, 0, 0, 0};
      if (!chunk_inside(at_byte, left)) return first_elements<DT>(base + at_byte, limit - c);
      return ldu16(base + at_byte);
    }
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
      return *(const AR_LDS u32x4*)(lds + row * (CH * 16) + (((kk * 4 + q) ^ mix_kc<CH, PAIRED>(row)) * 16));
    } else if constexpr (ES == 2) {
      const int k = kk * 32 + q * 8 + (l >> 2), c = r0 + (l & 3) * 4;
      const AR_LDS char* p = lds + k * (R * ES) + (((c / V) ^ mix_ks<DT, R>(k)) * 16) + (c % V) * ES;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS i16x4*)(p));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS i16x4*)(p + 4 * R * ES));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kk * 16 + q * 4 + i, c = r0 + l;
        w[i] = *(const AR_LDS uint32_t*)(lds + k * (R * ES) + (((c / V) ^ mix_ks<DT, R>(k)) * 16) + (c % V) * ES);
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

// Columns across the sum lie in a lane's subtiles as four neighbours each. Lane groups 0 and 1, and 2 and 3, exchange halves of
// two subtiles, x and y: the even group is left with 8 neighbours of x, the odd one with 8 of y. Stores
// of 16 bytes in the place of 8: gated gradient of 16,384 rows, 32 experts of 2 x 2048 x 4096 bf16, 1470 -> 1373 us.
template <int DT> __device__ __forceinline__ u32x4 neighbours(const f32x4& x, const f32x4& y) {
  auto pack = [](float lo, float hi) { return narrow<DT>(lo) | narrow<DT>(hi) << 16; };
  const auto a = __builtin_amdgcn_permlane16_swap(pack(x[0], x[1]), pack(y[0], y[1]), false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(pack(x[2], x[3]), pack(y[2], y[3]), false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}
// 8 elements of 16 bits to p, of which `left` lie in the row.
__device__ __forceinline__ void store_words(char* p, const u32x4& w, int left) {
  if (left >= 8) {
    stu16(p, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) store_elem<AR_BF16>(p, i, w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
}

// ------------------------------------------------------------------------------------------ the tile kernel
template <int KIND> constexpr bool kRowsKS = KIND == kWeight;                        // operand of the tile's rows
template <int KIND> constexpr bool kColsKS = KIND == kWeight || KIND == kInput;      // operand of its columns

// Tiles follow each other so that the workgroups of one XCD (every eighth one) work on neighbouring tiles, kRaster tiles
// down before the next column, and share the operands in its L2.
constexpr int kRaster = 4;
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int x = id & 7, q = total >> 3, r = total & 7;
  return x * q + (x < r ? x : r) + (id >> 3);
}
__device__ __forceinline__ void raster(int t, int down, int across, int* row, int* col) {
  const int group = t / (kRaster * across), in = t - group * (kRaster * across);
  const int high = min(kRaster, down - group * kRaster);
  *col = in / high;
  *row = group * kRaster + in - *col * high;
}

// How operands come into LDS: through registers; straight, in whole 16-byte chunks of the sum; or straight, with the chunk
// that the end of the sum cuts mended in LDS (which costs the large tiles registers that they do not have).
enum Loads { kRegisters = 0, kWhole = 1, kCut = 2 };

// WM x WN waves, each with a part of BM / WM rows and BN / WN columns (gated: of half as many, and both products of them) in
// registers. Sizes of a part: 128 x 64 in the 256 x 256 tile, whose 128 registers of sums leave room for the fragments of a
// step; 64 x 64 in the 128 x 128 one; 16 x 64 in the 64 x 64 one. 128 x 128 for each of four waves spills. LDS: five operand tiles
// of 128 bytes along the sum, 160 / 80 / 40 KB, room for 1 / 2 / 4 workgroups on a compute unit. Registers allow as many with
// loads straight into LDS (but one of the 128 x 128 linear kernel that mends chunks), and fewer through registers: one of 128 x 128,
// three of 64 x 64 (linear, dx). The compiler keeps sums of the 128 x 128 tiles, and of some 64 x 64 ones, in accumulation
// registers and moves them there and back in every step (96 moves beside 32 matrix instructions of 16-bit types, 84 beside 128 of
// fp32); the 256 x 256 tiles have no moves, but keep some scalars in vector registers (5 to 14 reads of them a step).
// Steps of half the length took 11% longer (131,072 rows, 64 experts of 2048 x 1024), having twice the barriers.
// Level or worse at 32 experts of 2 x 2048 x 4096 bf16: 32 x 32 instructions (3%), a raised wave priority (0), workgroups that
// start their next tile's loads before they write results (0 to 70%: the tiles of uneven segments spread less evenly).
template <int DT, int KIND, int LOADS, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(const ProductArgs a) {
  constexpr bool DIRECT = LOADS != kRegisters;
  constexpr int CH = 8, PLACES = DIRECT ? 5 : 4;  // chunks of the sum per step; operand tiles that LDS holds
  constexpr int NT = WM * WN * 64, ES = Traits<DT>::kSize, V = 16 / ES, K_STEP = CH * V;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool PAIRED = !kColsKS<KIND>;
  constexpr int WCOLS = BN / WN;  // a wave's columns, in blocks of 64
  static_assert(WCOLS % 64 == 0 && MI * 16 * WM == BM, "whole blocks");
  constexpr int COLS = KIND == kGated ? BN / 2 : BN;  // columns of the result
  using A = Tile<DT, kRowsKS<KIND>, false, DIRECT, CH, BM, NT>;
  using B = Tile<DT, kColsKS<KIND>, PAIRED, DIRECT, CH, BN, NT>;
  static_assert(BM == BN, "operand tiles take each other's places");
  __shared__ __align__(1024) char smem[PLACES][BM * CH * 16];
  const int wave = uniform(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int l = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;

  // Tiles of the result: rows of it per expert (weight: of every matrix) and columns.
  const int across = (a.n + COLS - 1) / COLS;
  int down, total;
  Lane mine{0, 0};
  if constexpr (KIND == kWeight) {
    down = (a.m + BM - 1) / BM;
    total = a.experts * (a.a1 ? 2 : 1) * down * across;
  } else {
    if (a.offsets) mine = lane_segment(a, threadIdx.x & 63);
    down = min(all_tiles(a, mine, 1, BM), a.most);
    total = down * across;
  }
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    // which tile
    int e, mt, nt, which = 0, first, n, K;
    if constexpr (KIND == kWeight) {
      // every matrix's tiles go to all XCDs: experts differ in rows, and so in work
      const int z = id / (across * down);
      raster(xcd_order(id - z * (across * down), across * down), down, across, &mt, &nt);
      e = a.a1 ? z >> 1 : z;
      which = a.a1 ? z & 1 : 0;
    } else {
      int row;
      raster(xcd_order(id, total), down, across, &row, &nt);
      Place at{};
      if (!find_tile(a, mine, row, 1, BM, &at)) continue;  // tables that changed meanwhile
      e = at.expert;
      mt = at.index;
      first = at.first;
      n = at.n;
    }
    e = uniform(e);
    if constexpr (KIND == kWeight) segment(a, e, &first, &n);
    first = uniform(first);
    n = uniform(n);
    const int m0 = uniform(mt) * BM, n0 = uniform(nt) * COLS;
    // the operands at the tile's first row or column and sum element 0, and the bytes of them per row and per step
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

    // A wave's part of the tile may lie wholly or in its second half past the result: it is not computed there.
    const int rows_wave = rows_left - wm * (BM / WM);
    const bool none = rows_wave <= 0 || cols_left <= wn * (KIND == kGated ? WCOLS / 2 : WCOLS), half = MI > 1 && rows_wave <= BM / WM / 2;
    auto read_a = [&](const AR_LDS char* at, int i, int kk) { return A::read(at, wm * (BM / WM) + i * 16, kk); };
    auto read_b = [&](const AR_LDS char* at, int j, int kk) { return B::read(at, wn * WCOLS + j * 16, kk); };
    // the products of one step, for the first `count` of the wave's MI times 16 rows
    auto simple = [&](const AR_LDS char* at_a, const AR_LDS char* at_b, auto count) {
      constexpr int N = decltype(count)::value;
#pragma unroll
      for (int kk = 0; kk < (N > 0 ? CH / 4 : 0); ++kk) {
        u32x4 fb[NI], fa[N > 0 ? N : 1];
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[j] = read_b(at_b, j, kk);
#pragma unroll
        for (int i = 0; i < N; ++i) fa[i] = read_a(at_a, i, kk);
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) acc[j][i] = mma<DT>(fb[j], fa[i], acc[j][i]);
      }
    };
    constexpr std::integral_constant<int, MI> kAll{};
    constexpr std::integral_constant<int, MI / 2> kHalf{};
    constexpr std::integral_constant<int, 0> kNone{};
    if constexpr (DIRECT) {
      // A step's products go in groups of NI, 16 rows and 4 chunks each. Fragments of rows are read four groups ahead, so
      // that the last four groups of a step need nothing more from LDS: before them all waves meet, the next step has
      // arrived and this one's places are free, and while they run the next step's first fragments are read. LDS has five
      // places for the two operands' tiles in turn: the columns' loads start one step ahead, the rows' two, a few in every
      // group, so that no wave's products wait for its loads to be issued.
      const int64_t step_a = kRowsKS<KIND> ? static_cast<int64_t>(sa) * K_STEP : CH * 16;
      const int64_t step_b = kColsKS<KIND> ? static_cast<int64_t>(sb) * K_STEP : CH * 16;
      constexpr int kPlace = BM * CH * 16, kGroups = 2 * MI;
      AR_LDS char* const places = (AR_LDS char*)(smem[0]);
      const uint32_t to_wave = uniform(static_cast<int>(reinterpret_cast<uintptr_t>(places))) + wave * 1024;
      auto advance = [](int& place) { place = place >= PLACES - 2 ? place - (PLACES - 2) : place + 2; };
      int next_a = 0, next_b = 0, ka = 0, kb = 0, to_a = 0, to_b = 1;  // the steps to load, their first elements, places
      // What the loads of a step may read from its base on; nothing behind the last step, where loads are issued too, so
      // that their number in flight stays the same.
      const int high = rows_left < BM ? rows_left : BM, wide = cols_left < COLS ? cols_left : COLS;
      int64_t left_a = kRowsKS<KIND> ? across_left(K, 0, sa, m0, ES) : along_left(high, sa, K, 0, ES);
      int64_t left_b = kColsKS<KIND> ? across_left(K, 0, sb, n0, ES) : along_left(wide, sb, K, 0, ES);
      const int64_t again_a = left_a, again_b = left_b;
      uint32_t bytes_a = 0, bytes_b = 0;
      auto allowed = [&](int64_t left, int step) {
        // the upper half apart: a comparison of 64 bits is none for scalar registers
        const uint32_t b = load_bytes(uniform(static_cast<int>(left >> 32)), static_cast<uint32_t>(left));
        return step < steps ? b : 0;
      };
      auto load_a = [&](int i) {
        if (i == 0) bytes_a = allowed(left_a, next_a);
        ta.load(i, pa, bytes_a, ka + ta.chunk * V < K, to_wave + to_a * kPlace);
        if (i + 1 < A::kLoads) return;
        pa += step_a;
        left_a -= step_a;
        ka += K_STEP;
        if (KIND == kInput && ++next_a == steps1) {  // on to the second product of the sum
          pa = pa1;
          left_a = again_a;
          ka = 0;
        }
        if (KIND != kInput) ++next_a;
        advance(to_a);
      };
      auto load_b = [&](int i) {
        if (i == 0) bytes_b = allowed(left_b, next_b);
        // gated: LDS rows 32 to 63 of every 64 are of w_up; whole waves read one matrix
        const bool of_up = KIND == kGated && ((wave * (64 / CH) + i * B::kStride) & 32) != 0;
        tb.load(i, of_up ? pb1 : pb, bytes_b, kb + tb.chunk * V < K, to_wave + to_b * kPlace);
        if (i + 1 < B::kLoads) return;
        pb += step_b;
        if (KIND == kGated) pb1 += step_b;
        left_b -= step_b;
        kb += K_STEP;
        if (KIND == kInput && ++next_b == steps1) {
          pb = pb1;
          left_b = again_b;
          kb = 0;
        }
        if (KIND != kInput) ++next_b;
        advance(to_b);
      };
      auto all_a = [&] {
#pragma unroll
        for (int i = 0; i < A::kLoads; ++i) load_a(i);
      };
      auto all_b = [&] {
#pragma unroll
        for (int i = 0; i < B::kLoads; ++i) load_b(i);
      };
      int at_a = 0, at_b = 1;
      // The chunk that a product's end cuts, once its last step has arrived.
      const int cut_at = K - (steps1 - 1) * K_STEP;
      auto cut_last = [&](int step) {
        if (KIND == kWeight || LOADS != kCut || cut_at % V == 0 || (step + 1 != steps1 && step + 1 != steps)) return;
        if constexpr (!kRowsKS<KIND>) A::cut(places + at_a * kPlace, cut_at);
        if constexpr (!kColsKS<KIND>) B::cut(places + at_b * kPlace, cut_at);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      };
      if (steps > 0) {
        all_a();
        all_b();
        all_a();
        ready<A::kLoads>();
        all_b();
        cut_last(0);
      }
      // Steps in which a wave multiplies `count` times 16 rows, one fragment after the other.
      auto plain_steps = [&](auto count) {
        for (int s = 0; s < steps; ++s) {
          all_a();
          simple(places + at_a * kPlace, places + at_b * kPlace, count);
          advance(at_a);
          advance(at_b);
          ready<A::kLoads>();
          cut_last(s + 1);
          all_b();
        }
      };
      if (none) {
        plain_steps(kNone);
      } else if (half) {
        plain_steps(kHalf);
      } else if constexpr (kGroups < 8) {
        plain_steps(kAll);
      } else if (steps > 0) {
        u32x4 b0[NI], b1[NI], rows[4];
#pragma unroll
        for (int j = 0; j < NI; ++j) b0[j] = read_b(places + at_b * kPlace, j, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = read_a(places + at_a * kPlace, i % MI, i / MI);
        // Scalar loads are done here too: with some possibly on their way, every wait for a fragment in the loop would be one
        // for all of them.
        __builtin_amdgcn_s_waitcnt(0xC07F);
        auto group = [&](int g, const u32x4(&b)[NI]) {
#pragma unroll
          for (int j = 0; j < NI; ++j) acc[j][g % MI] = mma<DT>(b[j], rows[g % 4], acc[j][g % MI]);
        };
        constexpr int kReads = NI / 4;
        static_assert(A::kLoads % 4 == 0 && B::kLoads % 4 == 0 && kGroups >= 8, "loads in groups");
        for (int s = 0; s < steps; ++s) {
          const AR_LDS char *now_a = places + at_a * kPlace, *now_b = places + at_b * kPlace;
          advance(at_a);
          advance(at_b);
          const AR_LDS char *then_a = places + at_a * kPlace, *then_b = places + at_b * kPlace;
#pragma unroll
          for (int g = 0; g < kGroups - 4; ++g) {
            group(g, g < MI ? b0 : b1);
            if (g < 4) {
#pragma unroll
              for (int j = g * kReads; j < (g + 1) * kReads; ++j) b1[j] = read_b(now_b, j, 1);
            }
            rows[g % 4] = read_a(now_a, (g + 4) % MI, (g + 4) / MI);
            if (g < 4) {
#pragma unroll
              for (int i = g * (A::kLoads / 4); i < (g + 1) * (A::kLoads / 4); ++i) load_a(i);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          ready<A::kLoads>();
          cut_last(s + 1);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            group(kGroups - 4 + h, b1);
#pragma unroll
            for (int j = h * kReads; j < (h + 1) * kReads; ++j) b0[j] = read_b(then_b, j, 0);
            rows[h] = read_a(then_a, h % MI, h / MI);
#pragma unroll
            for (int i = h * (B::kLoads / 4); i < (h + 1) * (B::kLoads / 4); ++i) load_b(i);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      ready<0>();  // nothing is in flight when the workgroup goes on or ends
    } else {
      u32x4 va[A::kLoads], vb[B::kLoads];
      const int high = rows_left < BM ? rows_left : BM, wide = cols_left < COLS ? cols_left : COLS;
      auto fetch = [&](int s) {
        const bool second = s >= steps1;
        const int k0 = (second ? s - steps1 : s) * K_STEP;
        auto from = [&](const char* p, bool ks, uint32_t stride) { return p + static_cast<int64_t>(k0) * (ks ? stride : ES); };
        auto left = [&](int64_t bytes) { return load_bytes(static_cast<uint32_t>(bytes >> 32), static_cast<uint32_t>(bytes)); };
        const uint32_t left_a = left(kRowsKS<KIND> ? across_left(K, k0, sa, m0, ES) : along_left(high, sa, K, k0, ES));
        const uint32_t left_b = left(kColsKS<KIND> ? across_left(K, k0, sb, n0, ES) : along_left(wide, sb, K, k0, ES));
        const char *at_a = from(second ? pa1 : pa, kRowsKS<KIND>, sa), *at_b = from(second ? pb1 : pb, kColsKS<KIND>, sb);
        const char* at_up = KIND == kGated ? from(pb1, false, sb) : nullptr;
#pragma unroll
        for (int i = 0; i < A::kLoads; ++i) va[i] = ta.fetch(i, at_a, sa, left_a, k0, K);
#pragma unroll
        for (int i = 0; i < B::kLoads; ++i) {
          // gated: LDS rows 32 to 63 of every 64 are of w_up; whole waves read one matrix
          const bool of_up = KIND == kGated && ((wave * (64 / CH) + i * B::kStride) & 32) != 0;
          vb[i] = tb.fetch(i, of_up ? at_up : at_b, sb, left_b, k0, K);
        }
      };
      auto put = [&](int s) {
        ta.put(va, (AR_LDS char*)(smem[2 * (s & 1)]));
        tb.put(vb, (AR_LDS char*)(smem[2 * (s & 1) + 1]));
      };
      if (steps > 0) {
        fetch(0);
        put(0);
      }
      for (int s = 0; s < steps; ++s) {
        __syncthreads();  // the buffer of this step is filled, and nobody reads the other one any more
        if (s + 1 < steps) fetch(s + 1);
        const AR_LDS char *now_a = (const AR_LDS char*)(smem[2 * (s & 1)]), *now_b = (const AR_LDS char*)(smem[2 * (s & 1) + 1]);
        if (!none && half) simple(now_a, now_b, kHalf);
        else if (!none) simple(now_a, now_b, kAll);
        if (s + 1 < steps) put(s + 1);
      }
      __syncthreads();  // the next tile's first step goes to a buffer that slower waves may still read
    }

    // results: lane l of group q has row l of every 16 and four neighbouring columns of every subtile
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = wm * (BM / WM) + i * 16 + l;
      if (r >= rows_left) continue;
      if constexpr (KIND == kGated) {
#pragma unroll
        for (int j = 0; j < NI; j += 4) {
          const int c = wn * (WCOLS / 2) + j * 8 + q * 8, left = a.n - n0 - c;
          if (left <= 0) continue;
          const int64_t ofs = (static_cast<int64_t>(first + m0 + r) * a.n + n0 + c) * ES;
          float g[8], u[8], h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            g[k] = acc[j + k / 4][i][k % 4];
            u[k] = acc[j + 2 + k / 4][i][k % 4];
            activate<DT, false>(a.act, g[k], &h[k], nullptr);
            h[k] *= u[k];
          }
          store_run<DT, 8>(static_cast<char*>(a.c0) + ofs, h, left);
          if (a.c1) {
            store_run<DT, 8>(static_cast<char*>(a.c1) + ofs, g, left);
            store_run<DT, 8>(static_cast<char*>(a.c2) + ofs, u, left);
          }
        }
      } else {
        char* out;
        if constexpr (KIND == kWeight)
          out = static_cast<char*>(which ? a.c1 : a.c0) +
                (static_cast<int64_t>(e) * a.c_stride + static_cast<int64_t>(m0 + r) * a.n + n0) * ES;
        else out = static_cast<char*>(a.c0) + (static_cast<int64_t>(first + m0 + r) * a.n + n0) * ES;
        if constexpr (PAIRED || ES == 4) {
          constexpr int RUN = PAIRED ? 8 : 4;
#pragma unroll
          for (int j = 0; j < NI; j += RUN / 4) {
            const int c = wn * WCOLS + n_of<PAIRED>(j, q, 0), left = a.n - n0 - c;
            float v[RUN];
#pragma unroll
            for (int k = 0; k < RUN; ++k) v[k] = acc[j + k / 4][i][k % 4];
            if (left > 0) store_run<DT, RUN>(out + c * ES, v, left);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NI; j += 2) {
            const int c = wn * WCOLS + (j + (q & 1)) * 16 + (q & 2) * 4, left = a.n - n0 - c;
            const u32x4 w = neighbours<DT>(acc[j][i], acc[j + 1][i]);
            if (left > 0) store_words(out + c * ES, w, left);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ few rows
// The forward products where an expert has a few rows only: bound by reading the weights once. A workgroup takes 32 rows of
// weights (gated: 16 of either) and 16 of the expert's rows; where one has more, its weights come from the caches again
// (64 experts of 1024 x 2048, 32 rows for one of them 9 us, 512 rows 26; all rows in one workgroup: 15 and 185). Its four waves split the sum in blocks of a
// cache line (128 bytes of every row), in turn, straight into the registers that the matrix instruction takes, the next
// block ahead of the products of this one; their sums meet in LDS. Many short workgroups keep more loads in flight than
// 128-row tiles do where those are few. Workgroups of neighbouring columns start at different blocks: rows of a power of
// two of bytes would have all of them read the same few memory channels at a time (8 of 64 experts, 2 x 1024 x 2048 bf16:
// 18.2 -> 14.6 us; 8 experts, 8192 x 4096: 114 -> 95).
constexpr int kFewRows = 16, kFewThreads = 256, kFewWaves = kFewThreads / 64;
constexpr int kUnits = kFewUnits;  // loads of a row's 64 bytes per block (4: 10% slower at 64 experts of 1024 x 1024)
constexpr int kFirstStep = 9;  // blocks between the first ones of neighbouring workgroups

template <int DT, int KIND> __global__ __launch_bounds__(kFewThreads) void few_kernel(const ProductArgs a) {
  constexpr int ES = Traits<DT>::kSize, V = Traits<DT>::kVec, BLOCK = few_block(V);  // elements of a block
  constexpr int COLS = KIND == kGated ? 16 : 32;
  __shared__ f32x4 sums[kFewWaves][2][64];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int across = (a.n + COLS - 1) / COLS;
  const int total = a.most * across;  // there may be fewer
  const uint32_t row_bytes = static_cast<uint32_t>(a.k) * ES;
  const int blocks = a.k / BLOCK;
  const Lane mine = a.offsets ? lane_segment(a, lane) : Lane{0, 0};
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    Place at{};
    if (!find_tile(a, mine, id / across, 1, kFewRows, &at)) return;
    const int n0 = id % across * COLS, cols_left = a.n - n0;
    const char* w[2];
    uint32_t wofs[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = KIND == kGated ? l : j * 16 + l;
      w[j] = static_cast<const char*>(KIND == kGated && j ? a.b1 : a.b0) +
             (static_cast<int64_t>(at.expert) * a.w_stride + static_cast<int64_t>(n0) * a.k) * ES;
      wofs[j] = static_cast<uint32_t>(row < cols_left ? row : cols_left - 1) * row_bytes + q * 16;
    }
    const int turn = blocks > 0 ? id % across * kFirstStep % blocks : 0;
    const int m0 = at.index * kFewRows, last = at.n - m0 - 1;
    const char* x = static_cast<const char*>(a.a0) + static_cast<int64_t>(at.first + m0) * row_bytes;
    const uint32_t xofs = static_cast<uint32_t>(l < last ? l : last) * row_bytes + q * 16;
    f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    struct Block {
      u32x4 w[2][kUnits], x[kUnits];
    };
    auto load = [&](Block& f, int block) {
      block += turn;
      const int64_t from = static_cast<int64_t>(block >= blocks ? block - blocks : block) * (BLOCK * ES);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j) f.w[j][u] = ldu16(w[j] + from + wofs[j] + u * 64);
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) f.x[u] = ldu16(x + from + xofs + u * 64);
    };
    auto multiply = [&](const Block& f) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = mma<DT>(f.w[j][u], f.x[u], acc[j]);
    };
    Block f0, f1;
    int b = wave;
    if (b < blocks) load(f0, b);
    for (; b < blocks; b += 2 * kFewWaves) {
      if (b + kFewWaves < blocks) load(f1, b + kFewWaves);
      multiply(f0);
      if (b + 2 * kFewWaves < blocks) load(f0, b + 2 * kFewWaves);
      if (b + kFewWaves < blocks) multiply(f1);
    }
    // what is left behind the last whole block, 64 bytes of every row or less for a wave
    static_assert(kUnits <= kFewWaves, "a wave takes one load's worth of the rest");
    const int rest = blocks * BLOCK + wave * 4 * V, k = rest + q * V;
    if (rest < a.k) {
      const int64_t from = static_cast<int64_t>(rest) * ES;
      auto end = [&](const char* p) {
        u32x4 v = {0, 0, 0, 0};
        if (few_whole(k, a.k, V)) v = ldu16(p);
        else if (k < a.k) v = first_elements<DT>(p, a.k - k);
        return v;
      };
      const u32x4 xt = end(x + from + xofs);
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[j] = mma<DT>(end(w[j] + from + wofs[j]), xt, acc[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) sums[wave][j][lane] = acc[j];
    __syncthreads();
    // results: lane l of group q has row l and four neighbouring columns of either half
    if (wave == 0 && l <= last) {
      f32x4 sum[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sum[j] = sums[0][j][lane];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) sum[j] += sums[v][j][lane];
      }
      const int64_t ofs = (static_cast<int64_t>(at.first + m0 + l) * a.n + n0) * ES;
      if constexpr (KIND == kGated) {
        const int c = q * 4, left = cols_left - c;
        float g[4], u[4], h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = sum[0][i];
          u[i] = sum[1][i];
          activate<DT, false>(a.act, g[i], &h[i], nullptr);
          h[i] *= u[i];
        }
        if (left > 0) {
          store_run<DT, 4>(static_cast<char*>(a.c0) + ofs + c * ES, h, left);
          if (a.c1) {
            store_run<DT, 4>(static_cast<char*>(a.c1) + ofs + c * ES, g, left);
            store_run<DT, 4>(static_cast<char*>(a.c2) + ofs + c * ES, u, left);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = j * 16 + q * 4, left = cols_left - c;
          const float v[4] = {sum[j][0], sum[j][1], sum[j][2], sum[j][3]};
          if (left > 0) store_run<DT, 4>(static_cast<char*>(a.c0) + ofs + c * ES, v, left);
        }
      }
    }
    __syncthreads();  // the sums are read before the next ones come
  }
}

// ------------------------------------------------------------------------------------------ slopes
// dg and du of an expert's rows; a segment's rows lie one behind the other, so its elements are walked in a row.
// UNIT: elements a workgroup takes at a time. Few are spread over more workgroups: 402 x 530 fp16, 12.6 us with the large unit.
constexpr int kSlopeThreads = 256, kSlopeUnit = 8192, kSlopeLeast = 1024;

template <int DT, int UNIT> __global__ __launch_bounds__(kSlopeThreads) void slopes_kernel(const ProductArgs a) {
  constexpr int V = Traits<DT>::kVec, ES = Traits<DT>::kSize;
  const Lane mine = a.offsets ? lane_segment(a, threadIdx.x & 63) : Lane{0, 0};
  const int total = min(all_tiles(a, mine, a.n, UNIT), a.most);
  for (int id = blockIdx.x; id < total; id += gridDim.x) {
    Place at;
    if (!find_tile(a, mine, id, a.n, UNIT, &at)) continue;  // tables that changed meanwhile
    const int64_t base = static_cast<int64_t>(at.first) * a.n + static_cast<int64_t>(at.index) * UNIT;
    const int64_t rest = static_cast<int64_t>(at.n) * a.n - static_cast<int64_t>(at.index) * UNIT;
    const int len = rest < UNIT ? static_cast<int>(rest) : UNIT;
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
constexpr int kMostGroups = 1024;  // workgroups per compute unit and launch; what is left is taken in turn
int64_t most_experts(const ProductArgs& a) { return !a.offsets ? 1 : a.experts < a.rows ? a.experts : a.rows; }
int grid_of(int64_t most, int per_cu) {
  const int64_t cap = static_cast<int64_t>(cu_count()) * per_cu;
  return static_cast<int>(most < cap ? most : cap);
}

template <int DT, int KIND, int LOADS, int BM, int BN, int WM, int WN>
hipError_t launch_tile(ProductArgs a, hipStream_t s) {
  constexpr int COLS = KIND == kGated ? BN / 2 : BN;
  const int64_t across = tiles_up(a.n, COLS);
  const int64_t down = KIND == kWeight ? matrices(a) * tiles_up(a.m, BM) : row_tiles(a, 1, BM);
  a.most = static_cast<int>(down);
  if (down == 0) return hipSuccess;
  tile_kernel<DT, KIND, LOADS, BM, BN, WM, WN><<<grid_of(down * across, kMostGroups), WM * WN * 64, 0, s>>>(a);
  return hipGetLastError();
}

// Whether all rows and addresses are multiples of 4 bytes, which loads straight into LDS take.
bool in_words(const ProductArgs& a, int kind, int esize) {
  const int64_t v = 4 / esize;
  uintptr_t p = 0;
  for (const void* x : {a.a0, a.a1, a.b0, a.b1}) p |= reinterpret_cast<uintptr_t>(x);
  const int64_t in = kind == kWeight ? a.m : a.k, cols = kind == kInput || kind == kWeight ? a.n : 0;
  const int64_t apart = kind == kWeight || a.experts == 1 ? 0 : a.w_stride;
  return p % 4 == 0 && in % v == 0 && cols % v == 0 && apart % v == 0;
}

template <int DT, int KIND> hipError_t launch_few(ProductArgs a, hipStream_t s) {
  a.most = static_cast<int>(row_tiles(a, 1, kFewRows));
  const int64_t across = tiles_up(a.n, KIND == kGated ? 16 : 32);
  few_kernel<DT, KIND><<<grid_of(a.most * across, kMostGroups), kFewThreads, 0, s>>>(a);
  return hipGetLastError();
}

// Which kernel. The host knows rows and experts, not how the rows are spread. (bf16, one MI355X, rows for each expert.)
//   Few rows (forward products) where 128-wide tiles would leave the GPU short of workgroups: few_kernel. One matrix, up to
//     16 rows: 4096 x 4096 12-15 us against 27 with 64 x 64 tiles and 33 with 128 x 128, the matrix in the last-level cache. Read
//     from memory, 16 rows 13.8 us; from 17 to 512 rows 64 x 64 tiles take 42-43 (a library product 18-29): too few of them
//     to keep memory busy. Experts: up to 4 rows each on
//     average, in fp32 16; rows are spread unevenly, so some experts have many times that, which tiles serve better. 8
//     experts, one row each, gated 2 x 1024 x 2048: 14.3 / 24 / 27. Segments of a router, few_kernel against tiles, bf16,
//     gated (up to 8 tiles for each CU): 16 of 2 x 8192 x 4096, 2 rows on average 200 / 248, 8 rows 265 / 252; 64 of 2 x 2048
//     x 2048, 2 rows 97 / 120, 8 rows 147 / 135; but 128 of 2 x 4096 x 1024 (32 for each CU), 2 rows 180 / 165; linear (one
//     for each CU): 16 of 2048 x 1024, 4 rows 9.1 / 10.8, 8 rows 13.9 / 10.9; but 64 of 2048 x 2048 (4 for each CU), 4 rows
//     52 / 46. Over 60 such shapes and 1 to 16 rows either choice is within 2% of the better one on average. fp32, 4 experts of
//     2048 x 4096, 16 rows: 31 / 99, 64 rows 97 / 107.
//     The rows are those of the buffers: segments that a sort padded count with their pads. 8 slots at 64 experts of 2 x 1024 x
//     2048 bf16, padded to 1, 16, 128 rows (8, 128, 1,024 rows): 13.2, 15.7 us, and 24.8 with tiles.
//   256 x 256 tiles (16-bit types, whole chunks): half the reads of the operands, but one workgroup a CU. From 192 rows an
//     expert and three tiles for four CUs on. 16 of 2048 x 2048: 128 rows, gated 75 us with 128 x 128 tiles / 81 with
//     256 x 256; 256 rows 112 / 86, linear (128 large tiles) 53 / 58; 1024 rows 329 / 249. Gradients of weights write more
//     than they multiply when rows are few, and take large tiles whenever there are enough: 16 of 2048 x 2048, 1 row
//     56 / 50, 1024 rows 191 / 142; one of 4096 x 4096, 1024 rows 47 / 36.
//   64 x 64 tiles where there is not one of 128 x 128 for each CU: one of 4096 x 4096, 128 rows 28 / 48, 1024 rows (256
//     tiles) 57 / 55; 32 of 512 x 512, 128 rows 9.3 / 12.5; 16 of 2048 x 2048, 128 rows (256 tiles) 54 / 44. fp32, which the
//     matrix instructions bound in either: always (4 of 2048 x 4096, gated, 64 rows 107 / 296, 512 rows 534 / 535, 2048 rows
//     2081 / 2099); weights' gradients where the busiest CU has at least a tenth less to do with them (6 of 1190 x 530, 300
//     tiles, 100 rows 18.6 / 23.8, 1000 rows 97 / 135; 10 of 1003 x 770, 560 tiles, 33 / 40; but 10 of 1000 x 768, 480 tiles,
//     100 rows 29.8 / 28.3, 1000 rows 150 / 144).
template <int DT, int KIND, int LOADS> hipError_t launch_small(const ProductArgs& a, bool least, hipStream_t s) {
  if (least) return launch_tile<DT, KIND, LOADS, 64, 64, 4, 1>(a, s);
  return launch_tile<DT, KIND, LOADS, 128, 128, 2, 2>(a, s);
}

template <int DT, int KIND> hipError_t launch_tiles(const ProductArgs& a, hipStream_t s) {
  constexpr int COLS = KIND == kGated ? 64 : 128, V = Traits<DT>::kVec;
  const int64_t cus = cu_count(), across = tiles_up(a.n, COLS);
  if constexpr (KIND == kGated || KIND == kLinear) {
    const bool spread = a.offsets && Traits<DT>::kSize == 2;
    const int64_t rows = spread ? 4 : 16, tiles = !spread ? 4 : KIND == kGated ? 8 : 1;
    if (a.rows <= rows * a.experts && most_experts(a) * across <= tiles * cus) return launch_few<DT, KIND>(a, s);
  }
  const int64_t down = KIND == kWeight ? matrices(a) * tiles_up(a.m, 128) : tiles_up(a.rows, 128);
  bool least = down * across < cus;
  if constexpr (KIND == kWeight && Traits<DT>::kSize == 4) {
    const int64_t small = matrices(a) * tiles_up(a.m, 64) * tiles_up(a.n, 64);
    least = least || 10 * tiles_up(small, cus) < 9 * 4 * tiles_up(down * across, cus);
  }
  const bool whole = KIND == kWeight || a.k % V == 0;
  if constexpr (Traits<DT>::kSize == 2) {
    if (!in_words(a, KIND, 2)) return launch_small<DT, KIND, kRegisters>(a, least, s);
    const int64_t large = KIND == kWeight ? matrices(a) * tiles_up(a.m, 256) : a.rows / 256;
    if (whole && (KIND == kWeight || a.rows >= 192 * static_cast<int64_t>(a.experts)) &&
        large * tiles_up(a.n, 2 * COLS) * 4 >= 3 * cus)
      return launch_tile<DT, KIND, kWhole, 256, 256, 2, 4>(a, s);
  }
  if constexpr (KIND != kWeight) {
    if constexpr (Traits<DT>::kSize == 4) return launch_tile<DT, KIND, kCut, 64, 64, 4, 1>(a, s);
    else if (!whole) return launch_small<DT, KIND, kCut>(a, least, s);
  }
  if constexpr (KIND == kWeight || Traits<DT>::kSize == 2) return launch_small<DT, KIND, kWhole>(a, least, s);
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

template <int DT, int UNIT> static hipError_t slopes_of(ProductArgs a, hipStream_t s) {
  a.most = static_cast<int>(row_tiles(a, a.n, UNIT));
  if (a.most == 0) return hipSuccess;
  slopes_kernel<DT, UNIT><<<grid_of(a.most, 8), kSlopeThreads, 0, s>>>(a);
  return hipGetLastError();
}
template <int DT> static hipError_t slopes_of(const ProductArgs& a, hipStream_t s) {
  if (static_cast<int64_t>(a.rows) * a.n < 4 * static_cast<int64_t>(kSlopeUnit) * cu_count()) return slopes_of<DT, kSlopeLeast>(a, s);
  return slopes_of<DT, kSlopeUnit>(a, s);
}
hipError_t launch_slopes(ProductArgs a, int dtype, hipStream_t s) {
  if (dtype == AR_BF16) return slopes_of<AR_BF16>(a, s);
  if (dtype == AR_F16) return slopes_of<AR_F16>(a, s);
  return slopes_of<AR_F32>(a, s);
}

}  // namespace ar
