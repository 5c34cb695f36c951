// ar_block.h -- launchers of the block-boundary operators (norm, experts), shared by the host layer and their kernel
// files, and the loads and reductions that these kernels have in common.
#pragma once

#include "ar_device.h"
#include "ar_steps.h"

namespace ar {

// ------------------------------------------------------------------------------------------ norm
struct NormCommon {
  const void* residual;   // forward: the residual read; backward: its gradient. May be null
  void* residual_out;     // forward only, may be null
  const void* gamma;
  const void* saved;      // backward: the stored residual (dtype, or codes when saved_scales is set)
  uint8_t* codes;         // forward: the 8-bit checkpoint, may be null
  float* scales;          // forward: its scales
  const float* saved_scales;
  float* rstd;            // forward: written, may be null
  const float* rstd_in;   // backward
  float* partial;         // backward: [groups][hidden] partial sums of dgamma
  int64_t rows;
  int hidden;
  int n;
  int gamma_f32;          // gamma is fp32 whatever the dtype
  int out8;               // forward: out holds E4M3 codes, out_scales their scales
  float eps;
};
// M: the most ranks. Kernels for up to 8 take the small form: a launch with 64 ranks' pointers (1.7 KB of arguments)
// costs the host about a microsecond more.
template <int M> struct NormArgsOf : NormCommon {
  const void* in[M];
  void* out[M];
  float* out_scales[M];
};
using NormArgs = NormArgsOf<AR_MAX_RANKS>;

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_rmsnorm_bwd(const NormArgs& a, int dtype, float* dgamma, hipStream_t s);
// Workgroups (and so partial sums of dgamma) of the backward kernel for n ranks; a function of the sizes alone. Most with
// one rank.
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t hidden, int n);

// ------------------------------------------------------------------------------------------ experts
struct SortArgs {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* counts;
  int32_t* pos;
  int32_t* src;
  int32_t* hist;  // tiled form: [tiles][experts]
  int64_t slots;
  int64_t rows;   // entries of src
  int experts;
  int align;
};
int64_t sort_workspace(int64_t slots, int experts);
hipError_t launch_expert_sort(const SortArgs& a, hipStream_t s);

struct MoveArgs {
  const void* x;           // dispatch: the tokens' rows. combine, its gradient: the experts' rows
  void* y;                 // dispatch: the sorted rows. combine: the tokens' rows. Gradient: the rows' gradients
  const void* x_scales;    // dispatch of 8-bit rows
  void* y_scales;
  const int32_t* pos;      // [tokens][k]
  const float* weights;    // [tokens][k], may be null
  const void* extra;       // combine: the addend, may be null. Gradient: the output's gradient
  float* dweights;         // gradient
  const int32_t* offsets;  // with counts: the pad rows to zero, may be null
  const int32_t* counts;
  int64_t tokens;
  int64_t rows;
  int hidden;              // rows are below 2^31 bytes
  int k;
  int experts;
};
hipError_t launch_expert_dispatch(const MoveArgs& a, int esize, hipStream_t s);
hipError_t launch_expert_combine(const MoveArgs& a, int dtype, hipStream_t s);
hipError_t launch_expert_combine_bwd(const MoveArgs& a, int dtype, hipStream_t s);

// Whether a call over `bytes` bytes in rows of `row_bytes` streams past the caches: from 128 MiB up, half of the 256 MiB
// last-level cache, in rows of whole lines. Default policy against streaming, three calls' data in turn, 4096 bf16 wide:
// norm of 8 ranks, 75 MB 13.1 against 14.0 us, 151 MB 34.7 against 29.4, 8 x 8192 x 8192 with 8-bit results 370 against
// 348; its gradient 20.3 / 19.7, 42.5 / 36.8 and (8 x 8192 x 4096) 238 / 214 us; combine 38 MB 8.9 / 7.9, 151 MB
// 31.4 / 26.3, 1.3 GB 257 / 229 us; its gradient 71 MB 16.4 / 19.0, 143 MB 36.8 / 32.0, 600 MB 122 / 113 us. Norm of 300 x
// 32,768 bf16, 4 and 8 ranks 51.9 / 40.7 and 83.6 / 72.0, of 1024 x 16,384 fp32, 2 ranks 79.9 / 75.9, its gradient 97.0 /
// 87.7, of 4096 x 16,384 bf16, 8 ranks 473 / 462, its gradient 487 / 478. Rows that share lines lose by non-temporal
// stores (8 x 4096 x 2050 fp32: 185 us streaming, 131 us cached).
inline bool streams(int64_t bytes, int64_t row_bytes) { return bytes >= (int64_t(128) << 20) && row_bytes % 128 == 0; }

// ------------------------------------------------------------------------------------------ device helpers
// How a kernel reads and writes rows. kStream: non-temporal loads and stores, for the calls that streams() names. kCached:
// default policy. kExact: default policy, and the vector that a row's end cuts is read element by element in its own place.
constexpr int kCached = 0, kStream = 1, kExact = 2;

// 16-, 8- and 4-byte accesses at any byte address: rows of odd widths start anywhere. The unaligned type leaves one
// instruction (global memory takes unaligned vectors on HSA); aligned addresses lose nothing by it.
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

__device__ __forceinline__ u32x4 ldu16(const void* p) { return *gptr<u32x4_a1>(p); }
__device__ __forceinline__ u32x4 ldu16_nt(const void* p) { return __builtin_nontemporal_load(gptr<u32x4_a1>(p)); }
__device__ __forceinline__ void stu16(void* p, const u32x4& v) { *gptr<u32x4_a1>(p) = v; }
__device__ __forceinline__ void stu16_nt(void* p, const u32x4& v) { __builtin_nontemporal_store(v, gptr<u32x4_a1>(p)); }

// Rows are handled in vectors of V elements. The vector that would run past a row's end is read from the place of the
// last whole one instead, so loads need no branch and stay together, and the values are moved down once they are fp32
// (sums of such vectors too), with zeros behind them. For rows of at least V elements.
template <int V> __device__ __forceinline__ uint32_t clamped(int e, int hidden) {
  return static_cast<uint32_t>(e + V <= hidden ? e : hidden - V);
}
template <int V> __device__ __forceinline__ void drop_past_end(float* v, int e, int hidden) {
  const int m = e + V - hidden;  // values that belong to elements before e
  if (m <= 0) return;
#pragma unroll
  for (int d = V / 2; d > 0; d >>= 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (m & d) ? (i + d < V ? v[i + d] : 0.0f) : v[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = m < V ? v[i] : 0.0f;
}

// 16 bytes at byte offset `at` of a row. The offset is hidden from the optimiser so that it stays a 32-bit register
// next to the row's scalar address in every access (global addresses of the form base + 32-bit offset): worked out as
// 64-bit addresses once for each of the many streams of a kernel, they took most of its registers.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
// The loads of v have returned when this is passed.
__device__ __forceinline__ void arrived(u32x4& v) { asm volatile("" : "+v"(v)); }
template <int MODE> __device__ __forceinline__ u32x4 ld_row(const void* row, uint32_t at) {
  if constexpr (MODE == kStream) return ldu16_nt(static_cast<const char*>(row) + opaque(at));
  else return ldu16(static_cast<const char*>(row) + opaque(at));
}
template <int MODE> __device__ __forceinline__ void st_row(void* row, uint32_t at, const u32x4& w) {
  if constexpr (MODE == kStream) stu16_nt(static_cast<char*>(row) + opaque(at), w);
  else stu16(static_cast<char*>(row) + opaque(at), w);
}
// The first n < 16 bytes of a vector, n a multiple of SIZE.
template <int SIZE> __device__ __forceinline__ void st_row_part(void* row, uint32_t at, u32x4 w, int n) {
  char* p = static_cast<char*>(row) + at;
#pragma unroll 1
  for (int i = 0; i < n; i += SIZE) {
    if constexpr (SIZE == 4) {
      *gptr<uint32_t>(p + i) = w[0];
      w = u32x4{w[1], w[2], w[3], 0};
    } else if constexpr (SIZE == 2) {
      *gptr<uint16_t>(p + i) = static_cast<uint16_t>(w[0]);
      w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, 0};
    } else {
      *gptr<uint8_t>(p + i) = static_cast<uint8_t>(w[0]);
      w = u32x4{w[0] >> 8 | w[1] << 24, w[1] >> 8 | w[2] << 24, w[2] >> 8 | w[3] << 24, 0};
    }
  }
}

// Elements [e, e + kVec) of a row as stored, from the clamped place. kExact: the vector that the row's end cuts element by
// element, in its own place; for rows shorter than a vector, and where another lane may by then have written the
// elements before e (results in place of what is read).
template <int DT, int MODE> __device__ __forceinline__ u32x4 load_vec(const void* row, int e, int hidden) {
  constexpr int V = Traits<DT>::kVec;
  if constexpr (MODE != kExact) return ld_row<MODE>(row, clamped<V>(e, hidden) * Traits<DT>::kSize);
  if (e + V <= hidden) return ld_row<MODE>(row, static_cast<uint32_t>(e) * Traits<DT>::kSize);
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t bits = e + i < hidden ? load_elem<DT>(row, e + i) : 0;
    if constexpr (Traits<DT>::kSize == 2) w[i >> 1] |= bits << (16 * (i & 1));
    else w[i % 4] = bits;
  }
  return w;
}
// Such a vector's values once they are fp32, moved where they belong.
template <int DT, int MODE> __device__ __forceinline__ void settle_vec(float* v, int e, int hidden) {
  if constexpr (MODE != kExact) drop_past_end<Traits<DT>::kVec>(v, e, hidden);
}
// Elements [e, e + kVec) to a row, as far as it goes.
template <int DT, int MODE> __device__ __forceinline__ void store_vec(void* row, int e, int hidden, const u32x4& w) {
  constexpr int kSize = Traits<DT>::kSize;
  if (e + Traits<DT>::kVec <= hidden) st_row<MODE>(row, static_cast<uint32_t>(e) * kSize, w);
  else if (e < hidden) st_row_part<kSize>(row, static_cast<uint32_t>(e) * kSize, w, (hidden - e) * kSize);
}

// Sum over the 64 lanes of a wave, the same in every lane; all lanes must be active. Four steps inside the 16-lane
// rows, then the four rows through scalar registers: no LDS round trip.
__device__ __forceinline__ float wave_sum(float v) {
  auto step = [](float x, int y) { return x + __int_as_float(y); };
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));  // row_half_mirror
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));  // row_mirror
  auto row = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Sum over the LANES lanes (8, 16 or 32) that share a row, in each of them; they are active or not together.
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
  auto step = [](float x, int y) { return x + __int_as_float(y); };
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));  // row_half_mirror
  if constexpr (LANES >= 16)
    v = step(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));  // row_mirror
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

}  // namespace ar
