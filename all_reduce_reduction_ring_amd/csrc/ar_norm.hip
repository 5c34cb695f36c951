// ar_norm.hip -- the reduction of N ranks' partial products with what follows it in a transformer layer, in one pass:
//   h = sum_r x_r + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gamma
// and its gradient, with dy the sum of N ranks' partial gradients:
//   xhat = h rstd;  g = dy gamma;  dx = rstd (g - xhat mean(g xhat)) + residual's gradient;  dgamma = sum_rows dy xhat
// y may leave as E4M3 codes with one scale per 128 elements of a row; h may leave a second time in that form, as the
// checkpoint the gradient is computed from.
//
// Both are bound by HBM: a row is read once, held in registers while its sums are formed, and written once. A workgroup
// takes a row (short rows: several to a wave; backward: several rows to a workgroup); a lane holds one slot of 8 elements,
// laid out so that 16 or 32 neighbouring lanes hold one 128-element block, and a block's scale is a maximum over them. Sums,
// statistics and the values that are quantised stay in fp32; h, y and dx are rounded once, when they are stored. The norm
// is taken of the unrounded h. Times below are one MI355X's, a kernel or call among others.
#include "ar_block.h"
#include "ar_e4m3.h"
#include "ar_internal.h"

namespace ar {
namespace {

// A lane's slot of 8 elements is kVecs vectors: 2-byte types, elements [8 i, 8 i + 8) for slot index i. fp32, whole waves:
// elements [512 u + 4 l, + 4) and the same + 256 for i = 64 u + l, so that every access of a wave is 1 KiB in one piece
// (rows that share cache lines, 6 x 4993 x 3545: 201 us; in pieces of 256 bytes 224; few rows with 8-bit results lose by the
// longer way to a block's maximum, 8 x 16 x 4096 5.0 -> 5.7); a 128-element block lies in 32 lanes' vectors. fp32, rows of 16 or 32 lanes (MODE without kWide): [128 b + 4 l, + 4) and the same + 64 for i = 16 b + l.
constexpr int kWide = 4;
constexpr int policy(int mode) { return mode & 3; }
template <int DT> constexpr int kVecs = Traits<DT>::kSize == 2 ? 1 : 2;
template <int DT, int MODE> constexpr bool kTwoBlocks = kVecs<DT> == 2 && (MODE & kWide) != 0;
template <int DT, int MODE> __device__ __forceinline__ int first_of(int i) {
  if constexpr (Traits<DT>::kSize == 2) return i * 8;
  else if constexpr ((MODE & kWide) != 0) return (i >> 6) * 4 * kBlock + (i & 63) * 4;
  else return (i >> 4) * kBlock + (i & 15) * 4;
}
// The first element of vector v of the slot that starts at e0.
template <int MODE> __device__ __forceinline__ int vec_at(int e0, int v) {
  return e0 + v * ((MODE & kWide) != 0 ? 2 * kBlock : kBlock / 2);
}

template <int DT> struct Raw {
  u32x4 w[kVecs<DT>];
};

// A slot of a row as stored, from the clamped places.
template <int DT, int MODE> __device__ __forceinline__ Raw<DT> load_raw(const void* row, int e0, int hidden) {
  Raw<DT> r;
#pragma unroll
  for (int v = 0; v < kVecs<DT>; ++v) r.w[v] = load_vec<DT, policy(MODE)>(row, vec_at<MODE>(e0, v), hidden);
  return r;
}
template <int DT> __device__ __forceinline__ void unpack_raw(const Raw<DT>& r, float (&v)[kPerLane]) {
  if constexpr (kVecs<DT> == 1) {
    Slot<DT>::unpack(r.w[0], v);
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) v[k] = __uint_as_float(r.w[k / 4][k % 4]);
  }
}
// Values read from clamped places, moved where they belong.
template <int DT, int MODE> __device__ __forceinline__ void settle(float (&v)[kPerLane], int e0, int hidden) {
#pragma unroll
  for (int i = 0; i < kVecs<DT>; ++i) settle_vec<DT, policy(MODE)>(v + i * Traits<DT>::kVec, vec_at<MODE>(e0, i), hidden);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int NR, typename F> __device__ __forceinline__ void each_rank(int n, F f) {
  if constexpr (NR > 0) {
#pragma unroll
    for (int r = 0; r < NR; ++r) f(r);
  } else {
    for (int r = 0; r < n; ++r) f(r);
  }
}

// A slot rounded into the type and stored to the row `to(r)` of every rank.
template <int DT, int NR, int MODE, typename F>
__device__ __forceinline__ void store_slot(const float (&v)[kPerLane], int e0, int hidden, int n, F to) {
  constexpr int V = Traits<DT>::kVec, kSize = Traits<DT>::kSize;
#pragma unroll
  for (int i = 0; i < kVecs<DT>; ++i) {
    float x[V];
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = v[i * V + k];
    const u32x4 w = Slot<DT>::pack(x);
    const int e = vec_at<MODE>(e0, i);
    const uint32_t at = static_cast<uint32_t>(e) * kSize;
    if (e + V <= hidden) each_rank<NR>(n, [&](int r) { st_row<policy(MODE)>(to(r), at, w); });
    else if (e < hidden) {
#pragma unroll 1
      for (int r = 0; r < n; ++r) st_row_part<kSize>(to(r), at, w, (hidden - e) * kSize);
    }
  }
}

// A slot's 8 codes, as two words (elements 0-3 and 4-7), to the row `to(r)` of every rank.
template <int DT, int NR, int MODE, typename F>
__device__ __forceinline__ void store_codes(const uint32_t (&w)[2], int e0, int hidden, int n, F to) {
  constexpr int V = Traits<DT>::kVec;
#pragma unroll
  for (int i = 0; i < kVecs<DT>; ++i) {
    const int e = vec_at<MODE>(e0, i);
    if (e + V <= hidden) {
      each_rank<NR>(n, [&](int r) {
        uint8_t* p = to(r) + opaque(e);
        if constexpr (V == 8 && policy(MODE) == kStream) __builtin_nontemporal_store(u32x2{w[0], w[1]}, gptr<u32x2_a1>(p));
        else if constexpr (V == 8) *gptr<u32x2_a1>(p) = u32x2{w[0], w[1]};
        else if constexpr (policy(MODE) == kStream) __builtin_nontemporal_store(w[i], gptr<u32_a1>(p));
        else *gptr<u32_a1>(p) = w[i];
      });
    } else if (e < hidden) {
#pragma unroll 1
      for (int r = 0; r < n; ++r) st_row_part<1>(to(r), e, u32x4{V == 8 ? w[0] : w[i], w[1], 0, 0}, hidden - e);
    }
  }
}

struct RawCodes {
  uint32_t w[2];
  float scale[2];  // of the two halves
};
template <int DT, int MODE>
__device__ __forceinline__ RawCodes load_codes(const uint8_t* row, const float* scales, int e0, int hidden) {
  constexpr int V = Traits<DT>::kVec;
  RawCodes r{{0, 0}, {0.0f, 0.0f}};
  if constexpr (policy(MODE) == kExact) {
    for (int k = 0; k < V; ++k)
      if (e0 + k < hidden) r.w[k >> 2] |= static_cast<uint32_t>(gptr<uint8_t>(row)[e0 + k]) << (8 * (k & 3));
  } else if constexpr (V == 8) {
    const u32x2 p = *gptr<u32x2_a1>(row + opaque(clamped<8>(e0, hidden)));
    r.w[0] = p[0];
    r.w[1] = p[1];
  } else {
    r.w[0] = *gptr<u32_a1>(row + opaque(clamped<4>(vec_at<MODE>(e0, 0), hidden)));
    r.w[1] = *gptr<u32_a1>(row + opaque(clamped<4>(vec_at<MODE>(e0, 1), hidden)));
  }
  auto scale_of = [&](int e) { return *gptr<float>(scales + opaque((e < hidden ? e : hidden - 1) / kBlock)); };
  r.scale[0] = scale_of(e0);
  r.scale[1] = kTwoBlocks<DT, MODE> ? scale_of(vec_at<MODE>(e0, 1)) : r.scale[0];
  return r;
}
__device__ __forceinline__ void unpack_codes(const RawCodes& r, float (&v)[kPerLane]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(r.w[i]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(r.w[i]), true);
    v[4 * i] = lo[0] * r.scale[i];
    v[4 * i + 1] = lo[1] * r.scale[i];
    v[4 * i + 2] = hi[0] * r.scale[i];
    v[4 * i + 3] = hi[1] * r.scale[i];
  }
}

// A slot of gamma as stored (fp32 whatever the type, where gamma_f32 says so), and its values, zeros past the row's end.
struct RawGamma {
  u32x4 w[2];
};
template <int DT, int MODE> __device__ __forceinline__ RawGamma load_gamma(const NormCommon& a, int e0) {
  RawGamma r;
  if (Traits<DT>::kSize == 2 && a.gamma_f32) {
    const uint32_t at = clamped<kPerLane>(e0, a.hidden) * 4;
    if constexpr (policy(MODE) == kExact) {
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) r.w[k >> 2][k & 3] = e0 + k < a.hidden ? gptr<uint32_t>(a.gamma)[e0 + k] : 0;
    } else {
      r.w[0] = ld_row<kCached>(a.gamma, at);
      r.w[1] = ld_row<kCached>(a.gamma, at + 16);
    }
  } else {
    const Raw<DT> x = load_raw<DT, (policy(MODE) == kExact ? kExact : kCached) | (MODE & kWide)>(a.gamma, e0, a.hidden);
#pragma unroll
    for (int v = 0; v < kVecs<DT>; ++v) r.w[v] = x.w[v];
  }
  return r;
}
template <int DT, int MODE>
__device__ __forceinline__ void unpack_gamma(const NormCommon& a, const RawGamma& r, int e0, float (&v)[kPerLane]) {
  if (Traits<DT>::kSize == 2 && !a.gamma_f32) {
    Slot<Traits<DT>::kSize == 2 ? DT : AR_BF16>::unpack(r.w[0], v);
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) v[k] = __uint_as_float(r.w[k / 4][k % 4]);
  }
  settle<DT, MODE>(v, e0, a.hidden);
}

// Sum over the workgroup, in every thread; `lds` holds one float per wave, for one call of a workgroup.
__device__ __forceinline__ float group_sum(float v, float* lds) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < waves; ++w) t += lds[w];
  return t;
}

constexpr int kMaxThreads = 1024;
constexpr int kShortThreads = 256;  // a forward workgroup of several rows
constexpr int kFewRanks = 8;
// The arguments that the kernels for NR ranks take (NR 0: any number).
template <int NR> using ArgsFor = NormArgsOf<NR == 0 ? AR_MAX_RANKS : kFewRanks>;
template <int NR> ArgsFor<NR> args_for(const NormArgs& a) {
  ArgsFor<NR> b;
  static_cast<NormCommon&>(b) = a;
  for (int r = 0; r < (NR == 0 ? AR_MAX_RANKS : NR); ++r) {
    b.in[r] = a.in[r];
    b.out[r] = a.out[r];
    b.out_scales[r] = a.out_scales[r];
  }
  return b;
}
constexpr int kRankBatch = 4;
constexpr int kTeamThreads = 512;  // a backward workgroup of several teams

// The ranks' slots of a row (NR: their number if known; otherwise `batch` of them from rank r0 on), and their sum in
// rank order onto h.
template <int DT, int NR, int MODE> struct RankSlots {
  static constexpr int kBatch = NR > 0 ? NR : kRankBatch;
  Raw<DT> raw[kBatch];
  __device__ __forceinline__ void load(const ArgsFor<NR>& a, int64_t off, int e0, int r0) {
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (NR > 0 || r0 + r < a.n)
        raw[r] = load_raw<DT, MODE>(static_cast<const char*>(a.in[r0 + r]) + off, e0, a.hidden);
  }
  __device__ __forceinline__ void add(const ArgsFor<NR>& a, int r0, float (&h)[kPerLane]) const {
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      if (NR > 0 || r0 + r < a.n) {
        float v[kPerLane];
        unpack_raw<DT>(raw[r], v);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) h[k] = r0 + r == 0 ? v[k] : h[k] + v[k];
      }
    }
  }
};

// h = the sum of the ranks' slots, the first ones already on their way.
template <int DT, int NR, int MODE>
__device__ __forceinline__ void sum_ranks(const ArgsFor<NR>& a, const RankSlots<DT, NR, MODE>& first, int64_t off, int e0,
                                          float (&h)[kPerLane]) {
  first.add(a, 0, h);
  if constexpr (NR == 0) {
    for (int r0 = kRankBatch; r0 < a.n; r0 += kRankBatch) {
      RankSlots<DT, NR, MODE> more;
      more.load(a, off, e0, r0);
      more.add(a, r0, h);
    }
  }
}

// One row's slot as codes: the scale per block by the codec's rule. All lanes of the row take part.
template <int DT, int MODE>
__device__ __forceinline__ void quant8(const float (&v)[kPerLane], float (&scale)[2], uint32_t (&w)[2]) {
  float inv[2];
  if constexpr (kTwoBlocks<DT, MODE>) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float m = row16_max(lane_amax<4>(v + 4 * i)), other = __shfl_xor(m, 16, 64);
      const BlockScale s = scale_for(m > other ? m : other);
      inv[i] = s.inv;
      scale[i] = s.scale;
    }
  } else {
    const BlockScale s = block_scale(v);
    inv[0] = inv[1] = s.inv;
    scale[0] = scale[1] = s.scale;
  }
  float q[kPerLane], r[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) q[k] = v[k] * inv[k >> 2];
  e4m3_round4(q, r, &w[0]);
  e4m3_round4(q + 4, r + 4, &w[1]);
  w[0] = canonical_nan_codes(w[0]);
  w[1] = canonical_nan_codes(w[1]);
}

// The scales of slot i to the row of scales `to(r)` of every rank, by the first lane of each block.
template <int DT, int NR, int MODE, typename F>
__device__ __forceinline__ void store_scales(const float (&scale)[2], int i, int hidden, int n, F to) {
  const int e0 = first_of<DT, MODE>(i);
  if constexpr (kTwoBlocks<DT, MODE>) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int e = vec_at<MODE>(e0, v);
      if ((i & 31) == 0 && e < hidden) each_rank<NR>(n, [&](int r) { *gptr<float>(to(r) + opaque(e / kBlock)) = scale[v]; });
    }
  } else {
    if ((i & 15) == 0 && e0 < hidden) each_rank<NR>(n, [&](int r) { *gptr<float>(to(r) + opaque(i >> 4)) = scale[0]; });
  }
}

// One workgroup, one row; LANES > 0: LANES lanes to a row (rows of at most LANES slots). One slot a lane wherever 1024
// threads cover the row: with 55 registers at 8 ranks, 8 waves a SIMD hide the loads of all ranks, which are issued
// together (8 x 8192 x 8192 bf16 with 8-bit results: 365 us with one slot, 373 with two, 370 with four; streaming, 348 us,
// 5.6 TB/s; one row of 4096, 8 ranks: 3.4 / 4.2 / 5.8 us).
template <int DT, int S, int NR, int MODE, int LANES>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_kernel(ArgsFor<NR> a, int64_t row0) {
  __shared__ float lds[kMaxThreads / 64];
  constexpr int kSize = Traits<DT>::kSize;
  const int nb = (a.hidden + kBlock - 1) / kBlock, threads = static_cast<int>(blockDim.x);
  const int tid = static_cast<int>(LANES > 0 ? threadIdx.x % LANES : threadIdx.x);
  int64_t row = row0 + blockIdx.x;
  if constexpr (LANES > 0) {
    row = row0 + static_cast<int64_t>(blockIdx.x) * (kShortThreads / LANES) + threadIdx.x / LANES;
    if (row >= a.rows) return;
  }
  const int64_t at = row * a.hidden;
  float h[S][kPerLane];
  RawGamma gam[S];
  float ss = 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) gam[s] = load_gamma<DT, MODE>(a, first_of<DT, MODE>(s * threads + tid));
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e0 = first_of<DT, MODE>(s * threads + tid);
    RankSlots<DT, NR, MODE> first;
    Raw<DT> res;
    first.load(a, at * kSize, e0, 0);
    if (a.residual) res = load_raw<DT, MODE>(static_cast<const char*>(a.residual) + at * kSize, e0, a.hidden);
    sum_ranks<DT, NR, MODE>(a, first, at * kSize, e0, h[s]);
    if (a.residual) {
      float v[kPerLane];
      unpack_raw<DT>(res, v);
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) h[s][k] += v[k];
    }
    settle<DT, MODE>(h[s], e0, a.hidden);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) ss += h[s][k] * h[s][k];
  }
  if constexpr (LANES > 0) ss = lanes_sum<LANES>(ss);
  else ss = group_sum(ss, lds);
  const float mean = ss / static_cast<float>(a.hidden);
  const float rstd = 1.0f / sqrtf(mean + a.eps);
  if (a.rstd && tid == 0) gptr<float>(a.rstd)[row] = rstd;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int i = s * threads + tid;
    const int e0 = first_of<DT, MODE>(i);
    if (a.residual_out)
      store_slot<DT, 1, MODE>(h[s], e0, a.hidden, 1, [&](int) { return static_cast<char*>(a.residual_out) + at * kSize; });
    if (a.codes) {
      float sc[2];
      uint32_t w[2];
      quant8<DT, MODE>(h[s], sc, w);
      store_codes<DT, 1, MODE>(w, e0, a.hidden, 1, [&](int) { return a.codes + at; });
      store_scales<DT, 1, MODE>(sc, i, a.hidden, 1, [&](int) { return a.scales + row * nb; });
    }
    float y[kPerLane];
    unpack_gamma<DT, MODE>(a, gam[s], e0, y);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) y[k] = h[s][k] * rstd * y[k];
    if (a.out8) {
      float sc[2];
      uint32_t w[2];
      quant8<DT, MODE>(y, sc, w);
      store_codes<DT, NR, MODE>(w, e0, a.hidden, a.n, [&](int r) { return static_cast<uint8_t*>(a.out[r]) + at; });
      store_scales<DT, NR, MODE>(sc, i, a.hidden, a.n, [&](int r) { return a.out_scales[r] + row * nb; });
    } else {
      store_slot<DT, NR, MODE>(y, e0, a.hidden, a.n, [&](int r) { return static_cast<char*>(a.out[r]) + at * kSize; });
    }
  }
}

// What a lane reads of one slot of a row in the backward pass.
template <int DT, int NR, int MODE> struct BwdSlot {
  RankSlots<DT, NR, MODE> first;
  Raw<DT> saved, res;
  RawCodes codes;
  __device__ __forceinline__ void load(const ArgsFor<NR>& a, int64_t row, int e0, bool residual) {
    constexpr int kSize = Traits<DT>::kSize;
    const int64_t at = row * a.hidden;
    first.load(a, at * kSize, e0, 0);
    if (a.saved_scales)
      codes = load_codes<DT, MODE>(static_cast<const uint8_t*>(a.saved) + at,
                                    a.saved_scales + row * ((a.hidden + kBlock - 1) / kBlock), e0, a.hidden);
    else
      saved = load_raw<DT, MODE>(static_cast<const char*>(a.saved) + at * kSize, e0, a.hidden);
    if (residual) res = load_raw<DT, MODE>(static_cast<const char*>(a.residual) + at * kSize, e0, a.hidden);
  }
};

// dgamma of one 128-element block of columns by a whole workgroup: 16 lanes to a row, every row once.
template <int DT, int NR, int WIDE_MODE>
__device__ __forceinline__ void columns_dgamma(const ArgsFor<NR>& a, int block, float* lds, float* dgamma) {
  constexpr int V = Traits<DT>::kVec, MODE = policy(WIDE_MODE);
  const int lane = threadIdx.x & 15, at_once = static_cast<int>(blockDim.x) >> 4;
  const int e0 = first_of<DT, MODE>(block * 16 + lane);
  float dg[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) dg[k] = 0.0f;
  for (int64_t row = threadIdx.x >> 4; row < a.rows; row += at_once) {
    BwdSlot<DT, NR, MODE> x;
    x.load(a, row, e0, false);
    const float rstd = gptr<float>(a.rstd_in)[row];
    float g[kPerLane], xh[kPerLane];
    sum_ranks<DT, NR, MODE>(a, x.first, row * a.hidden * Traits<DT>::kSize, e0, g);
    if (a.saved_scales) unpack_codes(x.codes, xh);
    else unpack_raw<DT>(x.saved, xh);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) dg[k] += g[k] * (xh[k] * rstd);
  }
  settle<DT, MODE>(dg, e0, a.hidden);
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    dg[k] += __shfl_xor(dg[k], 16, 64);
    dg[k] += __shfl_xor(dg[k], 32, 64);
    if ((threadIdx.x & 63) < 16) lds[(threadIdx.x >> 6) * kBlock + lane * kPerLane + k] = dg[k];
  }
  __syncthreads();
  if (threadIdx.x < kBlock) {
    float sum = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x) >> 6; ++w) sum += lds[w * kBlock + threadIdx.x];
    const int k = threadIdx.x % kPerLane;
    const int e = vec_at<MODE>(first_of<DT, MODE>(block * 16 + static_cast<int>(threadIdx.x) / kPerLane), k / V) + k % V;
    if (e < a.hidden) gptr<float>(dgamma)[e] = sum;
  }
}

// A workgroup holds R teams of threads, each of which takes a row at a time: team i of workgroup b the rows
// b R + i, + groups R, + 2 groups R, ... Every thread keeps its columns' sums of dy xhat in registers over all its rows;
// the teams' sums are joined in LDS and leave as one row of partial sums per workgroup, which dgamma_kernel adds up in
// order. One slot a lane (S = 1): the next row is read while this one's dot product is joined and its results are
// stored; not so fp32 rows of 6 and 8 ranks, whose next row does not fit the registers beside this one (6 ranks, ahead
// against not: 5461 x 4096 252 / 235 us, 4096 x 4096 from 8 bits 182 / 166, 16,384 x 200 64 / 44, 600 x 2048 24.5 / 19.4;
// rank counts without a kernel of their own read a batch's slots ahead). Wider rows (S > 1) have one team and read their row
// when its turn comes.
// LANES > 0: a team is LANES lanes of a wave (rows of at most LANES slots).
// 8 x 8192 x 4096 bf16 from 8 bits 213 us (5.5 TB/s), one rank, 16,384 x 2048 48 us (5.6 TB/s); a workgroup per row without
// reading ahead ran 231 and 55 us.
// SMALL: no second launch; the workgroups from `groups` on each sum a block of columns instead, reading those again.
template <int DT, int S, int NR, int MODE, bool SMALL, int LANES>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_bwd_kernel(ArgsFor<NR> a, int team_threads, int groups,
                                                                  float* dgamma) {
  constexpr bool kAhead = S == 1 && (Traits<DT>::kSize == 2 || NR < 6);
  __shared__ float lds[2][kMaxThreads / 64];
  __shared__ float join[S == 1 ? kTeamThreads * kPerLane : 1];
  // Wide rows: dgamma's sums lie in LDS (each thread its own), so that the row's values keep the registers.
  __shared__ f32x4 wide_dg[S == 1 ? 1 : 2 * S * kMaxThreads];
  constexpr int kSize = Traits<DT>::kSize;
  if constexpr (SMALL) {
    if (static_cast<int>(blockIdx.x) >= groups) {
      columns_dgamma<DT, NR, MODE>(a, static_cast<int>(blockIdx.x) - groups, join, dgamma);
      return;
    }
  }
  const int teams = S == 1 ? static_cast<int>(blockDim.x) / team_threads : 1;
  const int team = LANES > 0 ? static_cast<int>(threadIdx.x) / LANES
                   : S == 1  ? __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / team_threads)
                             : 0;
  const int tid = static_cast<int>(threadIdx.x) - team * team_threads;
  const int64_t step = static_cast<int64_t>(groups) * teams;
  float dg[1][kPerLane];
  RawGamma gam;
  if constexpr (S == 1) gam = load_gamma<DT, MODE>(a, first_of<DT, MODE>(tid));
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) dg[0][k] = 0.0f;
  if constexpr (S > 1) {
    for (int i = 0; i < 2 * S; ++i) wide_dg[i * kMaxThreads + tid] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  int flip = 0;
  BwdSlot<DT, NR, MODE> next;
  float rstd_next = 0.0f;
  int64_t base = static_cast<int64_t>(blockIdx.x) * teams;
  if (kAhead && base + team < a.rows) {
    next.load(a, base + team, first_of<DT, MODE>(tid), a.residual);
    rstd_next = gptr<float>(a.rstd_in)[base + team];
  }
  for (; base < a.rows; base += step, flip ^= 1) {  // all teams stay in the loop for the barriers in it
    const int64_t row = base + team, at = row * a.hidden;
    const bool active = S > 1 || row < a.rows;
    float g[S][kPerLane], xh[S][kPerLane];
    Raw<DT> res[S];
    float dot = 0.0f, rstd = 0.0f;
    if (active) {
      rstd = kAhead ? rstd_next : gptr<float>(a.rstd_in)[row];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int e0 = first_of<DT, MODE>(s * team_threads + tid);
        BwdSlot<DT, NR, MODE> x;
        if (kAhead) x = next;
        else x.load(a, row, e0, a.residual);
        sum_ranks<DT, NR, MODE>(a, x.first, at * kSize, e0, g[s]);
        settle<DT, MODE>(g[s], e0, a.hidden);
        if (a.saved_scales) unpack_codes(x.codes, xh[s]);
        else unpack_raw<DT>(x.saved, xh[s]);
        settle<DT, MODE>(xh[s], e0, a.hidden);
        res[s] = x.res;
        float y[kPerLane];
        unpack_gamma<DT, MODE>(a, S == 1 ? gam : load_gamma<DT, MODE>(a, e0), e0, y);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) xh[s][k] *= rstd;
        if constexpr (S > 1) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f32x4 sum = wide_dg[(2 * s + i) * kMaxThreads + tid];
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[k] += g[s][4 * i + k] * xh[s][4 * i + k];
            wide_dg[(2 * s + i) * kMaxThreads + tid] = sum;
          }
        }
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          if constexpr (S == 1) dg[0][k] += g[s][k] * xh[s][k];
          g[s][k] *= y[k];
          dot += g[s][k] * xh[s][k];
        }
      }
      // The clamped vectors reach into other lanes' elements, which are overwritten behind the barrier where a result
      // goes in place. All else has been used by then; the residual's gradient has to have arrived.
      if (a.residual) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int v = 0; v < kVecs<DT>; ++v) arrived(res[s].w[v]);
      }
      if (kAhead && row + step < a.rows) {
        next.load(a, row + step, first_of<DT, MODE>(tid), a.residual);
        rstd_next = gptr<float>(a.rstd_in)[row + step];
      }
    }
    if constexpr (LANES > 0) dot = lanes_sum<LANES>(dot);
    else dot = wave_sum(dot);
    if (LANES == 0 && team_threads > 64) {
      if ((threadIdx.x & 63) == 0) lds[flip][threadIdx.x >> 6] = dot;
      __syncthreads();
      dot = 0.0f;
      const int w0 = team * (team_threads >> 6);
      for (int w = 0; w < team_threads >> 6; ++w) dot += lds[flip][w0 + w];
    }
    if (!active) continue;
    const float mean = dot / static_cast<float>(a.hidden);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e0 = first_of<DT, MODE>(s * team_threads + tid);
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) g[s][k] = rstd * (g[s][k] - xh[s][k] * mean);
      if (a.residual) {
        float v[kPerLane];
        unpack_raw<DT>(res[s], v);
        settle<DT, MODE>(v, e0, a.hidden);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) g[s][k] += v[k];
      }
      store_slot<DT, NR, MODE>(g[s], e0, a.hidden, a.n, [&](int r) { return static_cast<char*>(a.out[r]) + at * kSize; });
    }
  }
  if constexpr (SMALL) return;
  // The teams' sums: those inside a wave first, then, in order, one part of `width` threads after another.
  int parts = teams, part = team, width = team_threads;
  bool holds = true;
  if constexpr (LANES > 0) {
#pragma unroll
    for (int d = LANES; d < 64; d *= 2)
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) dg[0][k] += __shfl_xor(dg[0][k], d, 64);
    parts = static_cast<int>(blockDim.x) >> 6;
    part = static_cast<int>(threadIdx.x) >> 6;
    width = LANES;
    holds = (threadIdx.x & 63) < LANES;
  }
  if (parts > 1) {
    const int others = width * (parts - 1);
    if (part > 0 && holds) {
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) join[k * others + (part - 1) * width + tid] = dg[0][k];
    }
    __syncthreads();
    if (part > 0) return;
    for (int t = 0; t < parts - 1; ++t) {
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) dg[0][k] += join[k * others + t * width + tid];
    }
  }
  if (!holds) return;
  float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.hidden;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e0 = first_of<DT, MODE>(s * team_threads + tid);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = vec_at<MODE>(e0, k / Traits<DT>::kVec) + k % Traits<DT>::kVec;
      float sum = dg[0][k];
      if constexpr (S > 1) sum = wide_dg[(2 * s + k / 4) * kMaxThreads + tid][k % 4];
      if (e < a.hidden) gptr<float>(to)[e] = sum;
    }
  }
}

// dgamma[c] = the sum over the groups' partial sums of column c: 16 columns a workgroup, 64 threads to a column, eight
// loads of a thread on their way (512 rows of 2048: 4.6 us; 32 threads to a column, one load after another: 11 us).
constexpr int kSumColumns = 16, kSumParts = 1024 / kSumColumns, kSumBatch = 8;
__global__ __launch_bounds__(1024) void dgamma_kernel(const float* partial, int64_t groups, int hidden, float* dgamma) {
  __shared__ float lds[kSumParts][kSumColumns + 1];
  const int c = threadIdx.x % kSumColumns, part = threadIdx.x / kSumColumns;
  const int col = blockIdx.x * kSumColumns + c;
  float t = 0.0f;
  if (col < hidden) {
    for (int64_t g0 = part; g0 < groups; g0 += kSumBatch * kSumParts) {
      float x[kSumBatch];
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        const int64_t g = g0 + u * kSumParts;
        x[u] = g < groups ? gptr<float>(partial)[g * hidden + col] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) t += x[u];
    }
  }
  lds[part][c] = t;
  __syncthreads();
  if (part == 0 && col < hidden) {
    float sum = 0.0f;
#pragma unroll 8
    for (int p = 0; p < kSumParts; ++p) sum += lds[p][c];
    gptr<float>(dgamma)[col] = sum;
  }
}

// Threads and slots per thread for a row of `hidden` elements: one slot of 8 a lane, two or four only where 1024
// threads do not cover the row. Whole waves, but for rows of up to 128 or 256 elements, which 16 or 32 lanes take
// (against a wave per row, bf16: 16,384 rows of 64, 2 ranks, forward 11.3 -> 5.0 us, backward 15.9 -> 9.2; of 256, 12.6 ->
// 9.5 and 18.7 -> 15.1; 131,072 rows of 128, one rank, 54 -> 21 and 71 -> 28).
struct Shape {
  int threads, slots;
};
Shape wave_shape(int hidden) {
  const int slots = (hidden + kBlock - 1) / kBlock * 16;  // whole blocks: 16 lanes each
  const int per = slots <= kMaxThreads ? 1 : slots <= 2 * kMaxThreads ? 2 : 4;
  return Shape{((slots + per - 1) / per + 63) / 64 * 64, per};
}
Shape shape_of(int hidden) {
  if (hidden <= 2 * kBlock) return Shape{hidden <= kBlock ? 16 : 32, 1};
  return wave_shape(hidden);
}

// Backward: teams per workgroup, as many as make 512 threads while there are rows for 256 workgroups (16,384 rows of 256
// bf16 with a wave each: 28.5 us with one team, 17.9 us with eight); whole waves.
int teams_of(int64_t rows, const Shape& sh) {
  const int unit = sh.threads < 64 ? 64 / sh.threads : 1;
  int64_t teams = kTeamThreads / sh.threads;
  if (teams > rows / 256) teams = rows / 256 / unit * unit;
  return sh.slots > 1 || teams < unit ? unit : static_cast<int>(teams);
}
// Workgroups: for 16 waves on each of the 256 compute units, or for 8 where a wave's own loads are many (6 ranks and
// more: 8 x 8192 x 4096 bf16 232 us, against 244 us with 16 waves; one rank, 16,384 x 2048: 83 us against 59 us); one
// for every CU at least, no more than there are rows for. Each leaves a row of partial sums.
int64_t groups_of(int64_t rows, const Shape& sh, int n) {
  const int teams = teams_of(rows, sh);
  int64_t most = (n >= 6 ? 2048 : 4096) / (teams * sh.threads / 64) / 256 * 256;
  if (most < 256) most = 256;
  if (most > 1024) most = 1024;
  const int64_t all = rows / teams + (rows % teams != 0);  // rows may be as many as the type holds
  return all < most ? all : most;
}

constexpr int64_t kMaxGrid = 1 << 21;  // a launch has fewer than 2^32 threads

// Backward without partial sums, in one launch: dgamma's columns read the ranks' rows and the saved ones a second time, each
// block of columns by one workgroup, 64 rows at once. Up to 256 rows, 24 MiB read twice and kOnceReads vectors of the ranks
// and the saved row under one another in a column. Two launches against one: 1 row of 4096 bf16, 8 ranks 8.2 / 4.0 us, 128 of
// 1000, 2 ranks 6.7 / 4.6; 200 of 4096, 8 ranks 14.1 / 12.1; 128 of 4096 fp32, 4 ranks 11.3 / 8.5. Beyond: 512 of 1000 bf16,
// 2 ranks 7.8 / 9.4, 256 of 200, 8 ranks 6.4 / 8.1, 200 of 1024, 16 ranks 11.4 / 14.2; fp32, 200 of 1024, 8 ranks 9.0 / 13.2,
// 16 ranks 12.9 / 23.6, 256 of 4096, 4 ranks 15.0 / 14.1.
constexpr int64_t kOnceReads = 2200;
bool reads_twice(const NormArgs& a, int size) {
  const int64_t reads = a.rows * (a.n + 1) * (size == 2 ? 1 : 2);
  return a.hidden <= kMaxThreads * kPerLane && a.rows <= 256 && reads <= kOnceReads &&
         a.rows * a.hidden * size * (a.n + 1) <= (24 << 20);
}
bool over_inputs(const NormArgs& a) {
  for (int r = 0; r < a.n; ++r)
    for (int i = 0; i < a.n; ++i)
      if (a.out[r] == a.in[i]) return true;
  return false;
}

template <int DT, int NR, int MODE> hipError_t run_bwd_once(const NormArgs& a, float* dgamma, hipStream_t s) {
  const Shape sh = wave_shape(a.hidden);
  const int teams = kMaxThreads / sh.threads, blocks = (a.hidden + kBlock - 1) / kBlock;
  const int groups = static_cast<int>((a.rows + teams - 1) / teams);
  const dim3 block(teams * sh.threads);
  const auto b = args_for<NR>(a);
  if (groups > 0 && over_inputs(a)) {  // all columns first, then the rows that overwrite what those read
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 1, NR, MODE, true, 0>), dim3(blocks), block, 0, s, b, sh.threads, 0, dgamma);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 1, NR, MODE, true, 0>), dim3(groups), block, 0, s, b, sh.threads, groups,
                       dgamma);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 1, NR, MODE, true, 0>), dim3(groups + blocks), block, 0, s, b, sh.threads,
                     groups, dgamma);
  return hipGetLastError();
}

template <int DT, int S, int NR, int MODE, int LANES>
hipError_t run_bwd(const NormArgs& a, const Shape& sh, float* dgamma, hipStream_t s) {
  const int teams = teams_of(a.rows, sh), groups = static_cast<int>(groups_of(a.rows, sh, a.n));
  if (groups > 0) {
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, S, NR, MODE, false, LANES>), dim3(groups), dim3(teams * sh.threads), 0, s,
                       args_for<NR>(a), sh.threads, groups, nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(dgamma_kernel, dim3((a.hidden + kSumColumns - 1) / kSumColumns), dim3(1024), 0, s, a.partial,
                     static_cast<int64_t>(groups), a.hidden, dgamma);
  return hipGetLastError();
}

template <int DT, int S, int NR, int MODE, int LANES>
hipError_t run_fwd(const NormArgs& a, const Shape& sh, hipStream_t s) {
  constexpr int kRows = LANES > 0 ? kShortThreads / LANES : 1;  // of a workgroup
  const int threads = LANES > 0 ? kShortThreads : sh.threads;
  for (int64_t row = 0; row < a.rows; row += kMaxGrid * kRows) {
    const int64_t left = (a.rows - row + kRows - 1) / kRows, groups = left < kMaxGrid ? left : kMaxGrid;
    hipLaunchKernelGGL((rmsnorm_kernel<DT, S, NR, MODE, LANES>), dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s,
                       args_for<NR>(a), row);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// dgamma: of the backward pass; null for the forward
template <int DT, int S, int NR, int MODE, int LANES>
hipError_t run(const NormArgs& a, float* dgamma, const Shape& sh, hipStream_t s) {
  if (!dgamma) return run_fwd<DT, S, NR, MODE, LANES>(a, sh, s);
  if constexpr (S == 1 && policy(MODE) != kStream) {
    if (reads_twice(a, Traits<DT>::kSize)) return run_bwd_once<DT, NR, MODE | kWide>(a, dgamma, s);
  }
  return run_bwd<DT, S, NR, MODE, LANES>(a, sh, dgamma, s);
}
// Rank counts that a layer's heads and widths divide by have kernels of their own, 0.5 MB of code each; 5, 7 and more than 8
// loop over batches of kRankBatch ranks. Against kernels of their own, 5 and 7 ranks lose in small calls (16 x 4096 bf16 3.6
// against 3.2 us and 3.9 against 3.5, gradient of 64 x 2048 5.4 / 5.0 and 5.9 / 5.4) and are level in large ones (536 MB of
// bf16 inputs, 4096 wide: 229 / 232 us and 219 / 221, gradient 251 / 256 and 228 / 229, of as many bytes of fp32 248 / 247
// and 232 / 230). 9 ranks run at 5.5 TB/s and 5.3, 16 at 4.9 and 4.9.
template <int DT, int S, int MODE, int LANES>
hipError_t run_n(const NormArgs& a, float* dgamma, const Shape& sh, hipStream_t s) {
  switch (a.n) {
    case 1: return run<DT, S, 1, MODE, LANES>(a, dgamma, sh, s);
    case 2: return run<DT, S, 2, MODE, LANES>(a, dgamma, sh, s);
    case 3: return run<DT, S, 3, MODE, LANES>(a, dgamma, sh, s);
    case 4: return run<DT, S, 4, MODE, LANES>(a, dgamma, sh, s);
    case 6: return run<DT, S, 6, MODE, LANES>(a, dgamma, sh, s);
    case 8: return run<DT, S, 8, MODE, LANES>(a, dgamma, sh, s);
    default: return run<DT, S, 0, MODE, LANES>(a, dgamma, sh, s);
  }
}

template <int DT> hipError_t launch(const NormArgs& a, float* dgamma, hipStream_t s) {
  const Shape sh = shape_of(a.hidden);
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  if (a.hidden < Traits<DT>::kVec) return run<DT, 1, 0, kExact, 16>(a, dgamma, sh, s);
  if (sh.threads == 16) return run_n<DT, 1, kCached, 16>(a, dgamma, sh, s);
  if (sh.threads == 32) return run_n<DT, 1, kCached, 32>(a, dgamma, sh, s);
  const bool stream = streams(a.rows * row * (2 * a.n + 2), row);
  switch (sh.slots) {
    case 1: return stream ? run_n<DT, 1, kStream | kWide, 0>(a, dgamma, sh, s) : run_n<DT, 1, kCached | kWide, 0>(a, dgamma, sh, s);
    case 2: return stream ? run_n<DT, 2, kStream | kWide, 0>(a, dgamma, sh, s) : run_n<DT, 2, kCached | kWide, 0>(a, dgamma, sh, s);
    default: return stream ? run_n<DT, 4, kStream | kWide, 0>(a, dgamma, sh, s) : run_n<DT, 4, kCached | kWide, 0>(a, dgamma, sh, s);
  }
}

}  // namespace

int64_t rmsnorm_bwd_groups(int64_t rows, int64_t hidden, int n) {
  return groups_of(rows, shape_of(static_cast<int>(hidden)), n);
}

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, hipStream_t s) {
  return launch_rmsnorm_bwd(a, dtype, nullptr, s);
}

hipError_t launch_rmsnorm_bwd(const NormArgs& a, int dtype, float* dgamma, hipStream_t s) {
  switch (dtype) {
    case AR_F32: return launch<AR_F32>(a, dgamma, s);
    case AR_BF16: return launch<AR_BF16>(a, dgamma, s);
    case AR_F16: return launch<AR_F16>(a, dgamma, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ar
