// ar_block.h -- launchers of the block-boundary operators (norm, experts), shared by the host layer and their kernel
// files, and the loads and reductions that these kernels have in common.
#pragma once

#include "ar_device.h"

namespace ar {

// ------------------------------------------------------------------------------------------ norm
struct NormArgs {
  const void* in[AR_MAX_RANKS];
  void* out[AR_MAX_RANKS];
  float* out_scales[AR_MAX_RANKS];
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

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_rmsnorm_bwd(const NormArgs& a, int dtype, float* dgamma, hipStream_t s);
// Workgroups (and so partial sums of dgamma) of the backward kernel; a function of the sizes alone.
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t hidden);

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
  int64_t hidden;
  int k;
  int experts;
};
hipError_t launch_expert_dispatch(const MoveArgs& a, int esize, hipStream_t s);
hipError_t launch_expert_combine(const MoveArgs& a, int dtype, hipStream_t s);
hipError_t launch_expert_combine_bwd(const MoveArgs& a, int dtype, hipStream_t s);

// ------------------------------------------------------------------------------------------ device helpers
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

// Sum over the 64 lanes of a wave, in every lane. All lanes must be active.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace ar
