// ar_norm.hip -- the reduction of N ranks' partial products with what follows it in a transformer layer, in one pass:
//   h = sum_r x_r + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gamma
// and its gradient, with dy the sum of N ranks' partial gradients:
//   xhat = h rstd;  g = dy gamma;  dx = rstd (g - xhat mean(g xhat)) + residual's gradient;  dgamma = sum_rows dy xhat
// y may leave as E4M3 codes with one scale per 128 elements of a row; h may leave a second time in that form, as the
// checkpoint the gradient is computed from.
//
// Both are bound by HBM: a row is read once, held in registers while its sum of squares is formed, and written once.
// A workgroup takes a row; a lane holds its elements in slots of 8 laid out so that the 16 lanes of a DPP row hold one
// 128-element block (see load8). Sums, statistics and the values that are quantised stay in fp32; h, y and dx are
// rounded once, when they are stored. The norm is taken of the unrounded h.
#include "ar_block.h"
#include "ar_e4m3.h"
#include "ar_internal.h"

namespace ar {
namespace {

// A lane's slot: 2-byte types, elements [8 i, 8 i + 8) for slot index i (one 16-byte access); fp32, elements
// [128 b + 4 l, + 4) and the same + 64 for i = 16 b + l (two 16-byte accesses, each covering whole lines per wave).
template <int DT> __device__ __forceinline__ int first_of(int i) {
  if constexpr (Traits<DT>::kSize == 2) return i * 8;
  else return (i >> 4) * kBlock + (i & 15) * 4;
}
// Element k of the slot that starts at e0.
template <int DT> __device__ __forceinline__ int elem_of(int e0, int k) {
  if constexpr (Traits<DT>::kSize == 2) return e0 + k;
  else return e0 + k + (k < 4 ? 0 : kBlock / 2 - 4);
}
template <int DT> __device__ __forceinline__ bool whole_slot(int e0, int hidden) {
  return elem_of<DT>(e0, kPerLane - 1) < hidden;
}

// The slot's 8 values of a row (zeros past its end).
template <int DT>
__device__ __forceinline__ void load8(const void* row, int e0, int hidden, float (&v)[kPerLane]) {
  if (whole_slot<DT>(e0, hidden)) {
    if constexpr (Traits<DT>::kSize == 2) {
      Slot<DT>::unpack(ldu16(static_cast<const uint16_t*>(row) + e0), v);
    } else {
      const u32x4 a = ldu16(static_cast<const float*>(row) + e0);
      const u32x4 b = ldu16(static_cast<const float*>(row) + e0 + kBlock / 2);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = __uint_as_float(a[k]);
        v[k + 4] = __uint_as_float(b[k]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = elem_of<DT>(e0, k);
      v[k] = e < hidden ? widen<DT>(load_elem<DT>(row, e)) : 0.0f;
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* row, int e0, int hidden, const float (&v)[kPerLane]) {
  if (whole_slot<DT>(e0, hidden)) {
    if constexpr (Traits<DT>::kSize == 2) {
      stu16_nt(static_cast<uint16_t*>(row) + e0, Slot<DT>::pack(v));
    } else {
      u32x4 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = __float_as_uint(v[k]);
        b[k] = __float_as_uint(v[k + 4]);
      }
      stu16_nt(static_cast<float*>(row) + e0, a);
      stu16_nt(static_cast<float*>(row) + e0 + kBlock / 2, b);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = elem_of<DT>(e0, k);
      if (e < hidden) store_elem<DT>(row, e, narrow<DT>(v[k]));
    }
  }
}

// The slot's 8 codes, as two words (elements 0-3 and 4-7).
template <int DT>
__device__ __forceinline__ void store_codes(uint8_t* row, int e0, int hidden, uint32_t w0, uint32_t w1) {
  if (whole_slot<DT>(e0, hidden)) {
    if constexpr (Traits<DT>::kSize == 2) {
      __builtin_nontemporal_store(u32x2{w0, w1}, gptr<u32x2_a1>(row + e0));
    } else {
      __builtin_nontemporal_store(w0, gptr<u32_a1>(row + e0));
      __builtin_nontemporal_store(w1, gptr<u32_a1>(row + e0 + kBlock / 2));
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = elem_of<DT>(e0, k);
      if (e < hidden) gptr<uint8_t>(row)[e] = static_cast<uint8_t>((k < 4 ? w0 : w1) >> (8 * (k & 3)));
    }
  }
}

template <int DT>
__device__ __forceinline__ void load_codes(const uint8_t* row, const float* scales, int e0, int hidden,
                                           float (&v)[kPerLane]) {
  uint32_t w[2] = {0, 0};
  if (whole_slot<DT>(e0, hidden)) {
    if constexpr (Traits<DT>::kSize == 2) {
      const u32x2 p = *gptr<u32x2_a1>(row + e0);
      w[0] = p[0];
      w[1] = p[1];
    } else {
      w[0] = *gptr<u32_a1>(row + e0);
      w[1] = *gptr<u32_a1>(row + e0 + kBlock / 2);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = elem_of<DT>(e0, k);
      if (e < hidden) w[k >> 2] |= static_cast<uint32_t>(gptr<uint8_t>(row)[e]) << (8 * (k & 3));
    }
  }
  const float sc = e0 < hidden ? gptr<float>(scales)[e0 / kBlock] : 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
    v[4 * i] = lo[0] * sc;
    v[4 * i + 1] = lo[1] * sc;
    v[4 * i + 2] = hi[0] * sc;
    v[4 * i + 3] = hi[1] * sc;
  }
}

template <int DT>
__device__ __forceinline__ void load_gamma(const void* gamma, int f32, int e0, int hidden, float (&v)[kPerLane]) {
  if (Traits<DT>::kSize == 2 && f32) {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) v[k] = e0 + k < hidden ? gptr<float>(gamma)[e0 + k] : 0.0f;
  } else {
    load8<DT>(gamma, e0, hidden, v);
  }
}

// Sum over the workgroup, in every thread; `lds` holds one float per wave and is free again two barriers later, so
// callers alternate between two of them.
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

// The sum of the ranks' slot in rank order.
template <int DT>
__device__ __forceinline__ void sum_ranks(const NormArgs& a, int64_t at, int e0, float (&h)[kPerLane]) {
  const int64_t off = at * Traits<DT>::kSize;
  load8<DT>(static_cast<const char*>(a.in[0]) + off, e0, a.hidden, h);
  for (int r = 1; r < a.n; ++r) {
    float v[kPerLane];
    load8<DT>(static_cast<const char*>(a.in[r]) + off, e0, a.hidden, v);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) h[k] += v[k];
  }
}

// One row's slot as codes: the scale per block by the codec's rule. All 64 lanes take part.
template <int DT>
__device__ __forceinline__ void quant8(const float (&v)[kPerLane], float* scale, uint32_t* w0, uint32_t* w1) {
  const BlockScale s = block_scale(v);
  float q[kPerLane], r[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) q[k] = v[k] * s.inv;
  e4m3_round4(q, r, w0);
  e4m3_round4(q + 4, r + 4, w1);
  *w0 = canonical_nan_codes(*w0);
  *w1 = canonical_nan_codes(*w1);
  *scale = s.scale;
}

template <int DT, int S>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_kernel(NormArgs a) {
  __shared__ float lds[2][kMaxThreads / 64];
  constexpr int kSize = Traits<DT>::kSize;
  const int nb = (a.hidden + kBlock - 1) / kBlock;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const int64_t at = row * a.hidden;
    float h[S][kPerLane];
    float ss = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e0 = first_of<DT>(s * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
      sum_ranks<DT>(a, at, e0, h[s]);
      if (a.residual) {
        float v[kPerLane];
        load8<DT>(static_cast<const char*>(a.residual) + at * kSize, e0, a.hidden, v);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) h[s][k] += v[k];
      }
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) ss += h[s][k] * h[s][k];
    }
    const float mean = group_sum(ss, lds[flip]) / static_cast<float>(a.hidden);
    const float rstd = 1.0f / sqrtf(mean + a.eps);
    if (a.rstd && threadIdx.x == 0) gptr<float>(a.rstd)[row] = rstd;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int i = s * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
      const int e0 = first_of<DT>(i);
      const bool block_lane = (i & 15) == 0 && e0 < a.hidden;
      if (a.residual_out) store8<DT>(static_cast<char*>(a.residual_out) + at * kSize, e0, a.hidden, h[s]);
      if (a.codes) {
        float sc;
        uint32_t w0, w1;
        quant8<DT>(h[s], &sc, &w0, &w1);
        store_codes<DT>(a.codes + at, e0, a.hidden, w0, w1);
        if (block_lane) gptr<float>(a.scales)[row * nb + (i >> 4)] = sc;
      }
      float y[kPerLane];
      load_gamma<DT>(a.gamma, a.gamma_f32, e0, a.hidden, y);
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) y[k] = h[s][k] * rstd * y[k];
      if (a.out8) {
        float sc;
        uint32_t w0, w1;
        quant8<DT>(y, &sc, &w0, &w1);
        for (int r = 0; r < a.n; ++r) {
          store_codes<DT>(static_cast<uint8_t*>(a.out[r]) + at, e0, a.hidden, w0, w1);
          if (block_lane) gptr<float>(a.out_scales[r])[row * nb + (i >> 4)] = sc;
        }
      } else {
        for (int r = 0; r < a.n; ++r) store8<DT>(static_cast<char*>(a.out[r]) + at * kSize, e0, a.hidden, y);
      }
    }
  }
}

// A workgroup takes rows blockIdx, blockIdx + groups, ...; its threads keep their columns' sums of dy xhat in
// registers over all of them and leave one row of partial sums behind, which dgamma_kernel adds up in order.
template <int DT, int S>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_bwd_kernel(NormArgs a) {
  __shared__ float lds[2][kMaxThreads / 64];
  constexpr int kSize = Traits<DT>::kSize;
  const int nb = (a.hidden + kBlock - 1) / kBlock;
  float dg[S][kPerLane];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) dg[s][k] = 0.0f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const int64_t at = row * a.hidden;
    const float rstd = gptr<float>(a.rstd_in)[row];
    float g[S][kPerLane], xh[S][kPerLane];
    float dot = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e0 = first_of<DT>(s * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
      sum_ranks<DT>(a, at, e0, g[s]);
      if (a.saved_scales) load_codes<DT>(static_cast<const uint8_t*>(a.saved) + at, a.saved_scales + row * nb, e0, a.hidden, xh[s]);
      else load8<DT>(static_cast<const char*>(a.saved) + at * kSize, e0, a.hidden, xh[s]);
      float gam[kPerLane];
      load_gamma<DT>(a.gamma, a.gamma_f32, e0, a.hidden, gam);
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        xh[s][k] *= rstd;
        dg[s][k] += g[s][k] * xh[s][k];
        g[s][k] *= gam[k];
        dot += g[s][k] * xh[s][k];
      }
    }
    const float mean = group_sum(dot, lds[flip]) / static_cast<float>(a.hidden);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e0 = first_of<DT>(s * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) g[s][k] = rstd * (g[s][k] - xh[s][k] * mean);
      if (a.residual) {
        float v[kPerLane];
        load8<DT>(static_cast<const char*>(a.residual) + at * kSize, e0, a.hidden, v);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) g[s][k] += v[k];
      }
      for (int r = 0; r < a.n; ++r) store8<DT>(static_cast<char*>(a.out[r]) + at * kSize, e0, a.hidden, g[s]);
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e0 = first_of<DT>(s * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int e = elem_of<DT>(e0, k);
      if (e < a.hidden) gptr<float>(a.partial)[static_cast<int64_t>(blockIdx.x) * a.hidden + e] = dg[s][k];
    }
  }
}

// dgamma[c] = the sum over the groups' partial sums of column c: 32 columns a workgroup, 32 threads to a column.
__global__ __launch_bounds__(1024) void dgamma_kernel(const float* partial, int64_t groups, int hidden, float* dgamma) {
  __shared__ float lds[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float t = 0.0f;
  if (col < hidden)
    for (int64_t g = part; g < groups; g += 32) t += gptr<float>(partial)[g * hidden + col];
  lds[part][threadIdx.x & 31] = t;
  __syncthreads();
  if (part == 0 && col < hidden) {
    float sum = 0.0f;
    for (int p = 0; p < 32; ++p) sum += lds[p][threadIdx.x];
    gptr<float>(dgamma)[col] = sum;
  }
}

// Threads and slots per thread for a row of `hidden` elements: one slot of 8 while 256 threads cover the row, then
// 2 and 4 slots, then more threads.
struct Shape {
  int threads, slots;
};
Shape shape_of(int hidden) {
  const int slots = (hidden + kBlock - 1) / kBlock * 16;  // whole blocks: 16 lanes each
  int per = slots > 512 ? 4 : slots > 256 ? 2 : 1;
  int threads = (slots + per - 1) / per;
  threads = (threads + 63) / 64 * 64;
  return Shape{threads, per};
}

constexpr int64_t kMaxGroups = 1024;

template <int DT> hipError_t launch_fwd(const NormArgs& a, hipStream_t s) {
  const Shape sh = shape_of(a.hidden);
  const dim3 grid(static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20))), block(sh.threads);
  switch (sh.slots) {
    case 1: hipLaunchKernelGGL((rmsnorm_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((rmsnorm_kernel<DT, 2>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((rmsnorm_kernel<DT, 4>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <int DT> hipError_t launch_bwd(const NormArgs& a, int64_t groups, hipStream_t s) {
  const Shape sh = shape_of(a.hidden);
  const dim3 grid(static_cast<unsigned>(groups)), block(sh.threads);
  switch (sh.slots) {
    case 1: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 2>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, 4>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

int64_t rmsnorm_bwd_groups(int64_t rows, int64_t) { return rows < kMaxGroups ? rows : kMaxGroups; }

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case AR_F32: return launch_fwd<AR_F32>(a, s);
    case AR_BF16: return launch_fwd<AR_BF16>(a, s);
    case AR_F16: return launch_fwd<AR_F16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_rmsnorm_bwd(const NormArgs& a, int dtype, float* dgamma, hipStream_t s) {
  const int64_t groups = rmsnorm_bwd_groups(a.rows, a.hidden);
  hipError_t e = hipSuccess;
  if (groups > 0) {
    switch (dtype) {
      case AR_F32: e = launch_bwd<AR_F32>(a, groups, s); break;
      case AR_BF16: e = launch_bwd<AR_BF16>(a, groups, s); break;
      case AR_F16: e = launch_bwd<AR_F16>(a, groups, s); break;
      default: return hipErrorInvalidValue;
    }
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(dgamma_kernel, dim3((a.hidden + 31) / 32), dim3(1024), 0, s, a.partial, groups, a.hidden, dgamma);
  return hipGetLastError();
}

}  // namespace ar
