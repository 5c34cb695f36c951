// ar_experts.hip -- tokens sorted by expert and back.
//   sort      slot q = t k + j (token t, choice j) goes to expert ids[q]; the slots of an expert take consecutive rows
//             in slot order, each expert's segment starts on a multiple of `align`; pos[q] is the slot's row (-1: the
//             id is no expert), src[row] the slot (-1: no slot there).
//   dispatch  xs[pos[t, j]] = x[t], pad rows zero
//   combine   out[t] = addend[t] + sum_j w[t, j] ys[pos[t, j]]; without weights it is dispatch's gradient
//   gradient  dys[pos[t, j]] = w[t, j] dout[t], pad rows zero; dw[t, j] = <dout[t], ys[pos[t, j]]>
//
// Everything is laid out by token, not by sorted row: a token's own row is then read (or written) once, and its k
// sorted rows, which are whole rows wherever they lie, once each. Rows out of [0, rows) are taken as absent.
#include "ar_block.h"
#include "ar_internal.h"

namespace ar {
namespace {

// ------------------------------------------------------------------------------------------ sort
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = AR_MAX_EXPERTS;
constexpr int64_t kOneGroupSlots = 8192;  // up to here one workgroup sorts everything in one launch

// The lanes of the wave that hold the same expert as this one (0 for a lane whose slot goes nowhere). All lanes take
// part; `bits` covers every expert number.
__device__ __forceinline__ uint64_t same_expert(int e, bool in, int bits) {
  uint64_t m = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? set : ~set;
  }
  return in ? m : 0;
}

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t q, int64_t slots, int experts, bool* in) {
  const int e = q < slots ? gptr<int32_t>(ids)[q] : -1;
  *in = e >= 0 && e < experts;
  return *in ? e : 0;
}

// Exclusive sum over the workgroup's threads; `lds` holds one value per wave. Returns the total in *total.
__device__ __forceinline__ int group_exclusive(int v, int* lds, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) before += lds[w];
    all += lds[w];
  }
  *total = all;
  __syncthreads();
  return before + x - v;
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortArgs a, int64_t tile) {
  __shared__ int hist[kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * tile;
  for (int64_t q = lo + threadIdx.x; q < lo + tile && q < a.slots; q += kSortThreads) {
    bool in;
    const int e = expert_of(a.ids, q, a.slots, a.experts, &in);
    if (in) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
    gptr<int32_t>(a.hist)[static_cast<int64_t>(blockIdx.x) * a.experts + e] = hist[e];
}

// One workgroup per tile of slots (one tile: no histogram launch before it). Every workgroup adds up the tiles'
// histograms for itself, so the tiles need no order among each other.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(SortArgs a, int64_t tile) {
  __shared__ int next[kSortWaves][kMaxExperts];  // first the waves' counts, then the next row of (wave, expert)
  __shared__ int scan[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
    for (int w = 0; w < kSortWaves; ++w) next[w][e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * tile;
  const int64_t hi = lo + tile < a.slots ? lo + tile : a.slots;
  const int64_t per_wave = (tile + kSortThreads - 1) / kSortThreads * 64;
  const int64_t w_lo = lo + wave * per_wave, w_hi = w_lo + per_wave < hi ? w_lo + per_wave : hi;
  for (int64_t q0 = w_lo; q0 < w_hi; q0 += 64) {
    bool in;
    const int e = expert_of(a.ids, q0 + lane, w_hi, a.experts, &in);
    if (in) atomicAdd(&next[wave][e], 1);
  }
  __syncthreads();
  // thread e: its expert's slots in all tiles, in the tiles before this one, and the segment's start
  const int e = threadIdx.x;
  int total = 0, before = 0;
  if (e < a.experts) {
    if (a.hist) {
      for (int64_t t = 0; t < gridDim.x; ++t) {
        const int c = gptr<int32_t>(a.hist)[t * a.experts + e];
        total += c;
        if (t < blockIdx.x) before += c;
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += next[w][e];
    }
  }
  const int padded = (total + a.align - 1) / a.align * a.align;
  int rows = 0;
  const int first = group_exclusive(padded, scan, &rows);
  if (e < a.experts) {
    int at = first + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = next[w][e];
      next[w][e] = at;
      at += c;
    }
    if (blockIdx.x == 0) {
      gptr<int32_t>(a.offsets)[e] = first;
      gptr<int32_t>(a.counts)[e] = total;
      if (e == 0) gptr<int32_t>(a.offsets)[a.experts] = rows;
    }
    // rows of this segment that no slot takes
    if (e % gridDim.x == blockIdx.x)
      for (int p = first + total; p < first + padded; ++p) gptr<int32_t>(a.src)[p] = -1;
  }
  for (int64_t p = rows + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; p < a.rows;
       p += static_cast<int64_t>(gridDim.x) * kSortThreads)
    gptr<int32_t>(a.src)[p] = -1;
  __syncthreads();
  for (int64_t q0 = w_lo; q0 < w_hi; q0 += 64) {
    const int64_t q = q0 + lane;
    bool in;
    const int x = expert_of(a.ids, q, w_hi, a.experts, &in);
    const uint64_t same = same_expert(x, in, bits);
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    int p = 0;
    if (in && rank == 0) p = atomicAdd(&next[wave][x], __popcll(same));  // the lowest lane takes rows for all of them
    p = __shfl(p, in ? __ffsll(static_cast<unsigned long long>(same)) - 1 : lane, 64) + rank;
    if (q < w_hi) gptr<int32_t>(a.pos)[q] = in ? p : -1;
    if (in) gptr<int32_t>(a.src)[p] = static_cast<int32_t>(q);
  }
}

// ------------------------------------------------------------------------------------------ rows
constexpr int kThreads = 256;
constexpr int kChoices = 8;  // choices of a token handled together

// The rows of choices j0 .. j0 + 7 (-1: none).
__device__ __forceinline__ void load_rows(const MoveArgs& a, int64_t t, int j0, int (&p)[kChoices]) {
#pragma unroll
  for (int j = 0; j < kChoices; ++j) {
    const int v = j0 + j < a.k ? gptr<int32_t>(a.pos)[t * a.k + j0 + j] : -1;
    p[j] = v >= 0 && v < a.rows ? v : -1;
  }
}

// Copy a row of `bytes` bytes (a multiple of the element size) to the rows p of `to`, by `lanes` lanes.
__device__ __forceinline__ void spread_row(const char* from, char* to, int64_t bytes, const int (&p)[kChoices],
                                           int lane, int lanes) {
  for (int64_t b = lane * 16; b < bytes; b += lanes * 16) {
    if (b + 16 <= bytes) {
      const u32x4 v = ldu16(from + b);
#pragma unroll
      for (int j = 0; j < kChoices; ++j)
        if (p[j] >= 0) stu16_nt(to + p[j] * bytes + b, v);
    } else {
      for (int64_t c = b; c < bytes; ++c) {
        const uint8_t v = gptr<uint8_t>(from)[c];
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (p[j] >= 0) gptr<uint8_t>(to)[p[j] * bytes + c] = v;
      }
    }
  }
}

__device__ __forceinline__ void zero_bytes(char* to, int64_t bytes) {
  for (int64_t b = threadIdx.x * 16; b < bytes; b += kThreads * 16) {
    if (b + 16 <= bytes) stu16_nt(to + b, u32x4{0, 0, 0, 0});
    else
      for (int64_t c = b; c < bytes; ++c) gptr<uint8_t>(to)[c] = 0;
  }
}

// The pad rows of expert e's segment, zeroed by one workgroup.
__device__ __forceinline__ void zero_pads(const MoveArgs& a, int e, int64_t row_bytes, int64_t scale_bytes) {
  int64_t lo = static_cast<int64_t>(gptr<int32_t>(a.offsets)[e]) + gptr<int32_t>(a.counts)[e];
  int64_t hi = gptr<int32_t>(a.offsets)[e + 1];
  if (lo < 0) lo = 0;
  if (hi > a.rows) hi = a.rows;
  if (lo >= hi) return;
  zero_bytes(static_cast<char*>(a.y) + lo * row_bytes, (hi - lo) * row_bytes);
  if (scale_bytes) zero_bytes(static_cast<char*>(a.y_scales) + lo * scale_bytes, (hi - lo) * scale_bytes);
}

// LANES lanes take a token, tokens in steps of the token workgroups' number.
template <int LANES> __device__ __forceinline__ int64_t first_token() {
  return static_cast<int64_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
}

// Workgroups past the tokens' zero the experts' pad rows.
template <int LANES>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(MoveArgs a, int64_t row_bytes, int64_t scale_bytes,
                                                            int64_t token_groups) {
  if (static_cast<int64_t>(blockIdx.x) >= token_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x - token_groups), row_bytes, scale_bytes);
    return;
  }
  const int lane = threadIdx.x % LANES;
  for (int64_t t = first_token<LANES>(); t < a.tokens; t += token_groups * (kThreads / LANES)) {
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
      int p[kChoices];
      load_rows(a, t, j0, p);
      spread_row(static_cast<const char*>(a.x) + t * row_bytes, static_cast<char*>(a.y), row_bytes, p, lane, LANES);
      if (scale_bytes)
        spread_row(static_cast<const char*>(a.x_scales) + t * scale_bytes, static_cast<char*>(a.y_scales), scale_bytes,
                   p, lane, LANES);
    }
  }
}

// A 16-byte vector of a row from element e on (zeros past its end), and its store.
template <int DT>
__device__ __forceinline__ void load_vec(const void* row, int64_t e, int64_t hidden, float (&v)[Traits<DT>::kVec]) {
  if (e + Traits<DT>::kVec <= hidden) {
    Slot<DT>::unpack(ldu16(static_cast<const char*>(row) + e * Traits<DT>::kSize), v);
  } else {
#pragma unroll
    for (int i = 0; i < Traits<DT>::kVec; ++i) v[i] = e + i < hidden ? widen<DT>(load_elem<DT>(row, e + i)) : 0.0f;
  }
}
template <int DT>
__device__ __forceinline__ void store_vec(void* row, int64_t e, int64_t hidden, const float (&v)[Traits<DT>::kVec]) {
  if (e + Traits<DT>::kVec <= hidden) {
    stu16_nt(static_cast<char*>(row) + e * Traits<DT>::kSize, Slot<DT>::pack(v));
  } else {
#pragma unroll
    for (int i = 0; i < Traits<DT>::kVec; ++i)
      if (e + i < hidden) store_elem<DT>(row, e + i, narrow<DT>(v[i]));
  }
}

// The sum runs in fp32 over the choices in order, the addend last, and is rounded once.
template <int DT, int LANES>
__global__ __launch_bounds__(kThreads) void combine_kernel(MoveArgs a) {
  constexpr int V = Traits<DT>::kVec;
  const int64_t row = a.hidden * Traits<DT>::kSize;
  for (int64_t t = first_token<LANES>(); t < a.tokens; t += static_cast<int64_t>(gridDim.x) * (kThreads / LANES)) {
    for (int64_t e = threadIdx.x % LANES * V; e < a.hidden; e += LANES * V) {
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.0f;
      for (int j0 = 0; j0 < a.k; j0 += kChoices) {
        int p[kChoices];
        load_rows(a, t, j0, p);
        float v[kChoices][V];
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (p[j] >= 0) load_vec<DT>(static_cast<const char*>(a.x) + p[j] * row, e, a.hidden, v[j]);
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
          if (p[j] < 0) continue;
          const float w = a.weights ? gptr<float>(a.weights)[t * a.k + j0 + j] : 1.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(w, v[j][i], acc[i]);
        }
      }
      if (a.extra) {
        float v[V];
        load_vec<DT>(static_cast<const char*>(a.extra) + t * row, e, a.hidden, v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += v[i];
      }
      store_vec<DT>(static_cast<char*>(a.y) + t * row, e, a.hidden, acc);
    }
  }
}

// LANES is 64 (a wave per token) or 256 (a workgroup per token, the waves' dot products joined in LDS).
template <int DT, int LANES>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(MoveArgs a, int64_t token_groups) {
  constexpr int V = Traits<DT>::kVec;
  __shared__ float lds[kThreads / 64][kChoices];
  const int64_t row = a.hidden * Traits<DT>::kSize;
  if (static_cast<int64_t>(blockIdx.x) >= token_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x - token_groups), row, 0);
    return;
  }
  const int lane = threadIdx.x % LANES;
  // whole waves take the loop together; with 256 lanes the whole workgroup
  for (int64_t t = first_token<LANES>(); t < a.tokens; t += token_groups * (kThreads / LANES)) {
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
      int p[kChoices];
      load_rows(a, t, j0, p);
      float w[kChoices], dot[kChoices];
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        w[j] = p[j] >= 0 ? gptr<float>(a.weights)[t * a.k + j0 + j] : 0.0f;
        dot[j] = 0.0f;
      }
      for (int64_t e = lane * V; e < a.hidden; e += LANES * V) {
        float g[V];
        load_vec<DT>(static_cast<const char*>(a.extra) + t * row, e, a.hidden, g);
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
          if (p[j] < 0) continue;
          float v[V], d[V];
          load_vec<DT>(static_cast<const char*>(a.x) + p[j] * row, e, a.hidden, v);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[j] = fmaf(g[i], v[i], dot[j]);
            d[i] = w[j] * g[i];
          }
          store_vec<DT>(static_cast<char*>(a.y) + p[j] * row, e, a.hidden, d);
        }
      }
#pragma unroll
      for (int j = 0; j < kChoices; ++j) dot[j] = wave_sum(dot[j]);
      if constexpr (LANES == kThreads) {
        __syncthreads();  // the sums of the step before are read
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < kChoices; ++j) lds[threadIdx.x >> 6][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kChoices && j0 + static_cast<int>(threadIdx.x) < a.k) {
          float sum = 0.0f;
          for (int u = 0; u < kThreads / 64; ++u) sum += lds[u][threadIdx.x];
          gptr<float>(a.dweights)[t * a.k + j0 + threadIdx.x] = sum;
        }
      } else if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (j0 + j < a.k) gptr<float>(a.dweights)[t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

// Slots per workgroup of the tiled sort: 2048, more where that would make over 512 tiles (every workgroup reads all
// tiles' histograms).
int64_t sort_tile(int64_t slots) {
  const int64_t even = (slots + 511) / 512;
  return even <= 2048 ? 2048 : (even + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// Lanes per token: a workgroup for rows of 128 vectors and more, a wave below, 16 lanes up to 16 vectors.
int lanes_for(int64_t vectors) { return vectors >= 128 ? 256 : vectors > 16 ? 64 : 16; }
int64_t groups_for(int64_t tokens, int lanes) {
  const int64_t groups = (tokens + kThreads / lanes - 1) / (kThreads / lanes);
  return groups < (1 << 22) ? groups : (1 << 22);  // a launch has fewer than 2^32 threads
}

template <int DT> hipError_t combine_dt(const MoveArgs& a, hipStream_t s) {
  const int lanes = lanes_for((a.hidden + Traits<DT>::kVec - 1) / Traits<DT>::kVec);
  const dim3 grid(static_cast<unsigned>(groups_for(a.tokens, lanes))), block(kThreads);
  if (lanes == 256) hipLaunchKernelGGL((combine_kernel<DT, 256>), grid, block, 0, s, a);
  else if (lanes == 64) hipLaunchKernelGGL((combine_kernel<DT, 64>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_kernel<DT, 16>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int DT> hipError_t combine_bwd_dt(const MoveArgs& a, hipStream_t s) {
  int lanes = lanes_for((a.hidden + Traits<DT>::kVec - 1) / Traits<DT>::kVec);
  if (lanes < 64) lanes = 64;
  const int64_t groups = groups_for(a.tokens, lanes);
  const dim3 grid(static_cast<unsigned>(groups + (a.offsets ? a.experts : 0))), block(kThreads);
  if (lanes == 256) hipLaunchKernelGGL((combine_bwd_kernel<DT, 256>), grid, block, 0, s, a, groups);
  else hipLaunchKernelGGL((combine_bwd_kernel<DT, 64>), grid, block, 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace

int64_t sort_workspace(int64_t slots, int experts) {
  if (slots <= kOneGroupSlots) return 0;
  const int64_t tile = sort_tile(slots);
  return (slots + tile - 1) / tile * experts * 4;
}

hipError_t launch_expert_sort(const SortArgs& a, hipStream_t s) {
  const dim3 block(kSortThreads);
  if (a.slots <= kOneGroupSlots) {
    SortArgs b = a;
    b.hist = nullptr;
    hipLaunchKernelGGL(sort_kernel, dim3(1), block, 0, s, b, a.slots > 0 ? a.slots : 1);
    return hipGetLastError();
  }
  const int64_t tile = sort_tile(a.slots);
  const dim3 grid(static_cast<unsigned>((a.slots + tile - 1) / tile));
  hipLaunchKernelGGL(sort_hist_kernel, grid, block, 0, s, a, tile);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sort_kernel, grid, block, 0, s, a, tile);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const MoveArgs& a, int esize, hipStream_t s) {
  const int64_t row = a.hidden * esize, scale = a.x_scales ? (a.hidden + AR_FP8_BLOCK - 1) / AR_FP8_BLOCK * 4 : 0;
  const int lanes = lanes_for((row + 15) / 16);
  const int64_t groups = groups_for(a.tokens, lanes);
  const dim3 grid(static_cast<unsigned>(groups + (a.offsets ? a.experts : 0))), block(kThreads);
  if (grid.x == 0) return hipSuccess;
  if (lanes == 256) hipLaunchKernelGGL(dispatch_kernel<256>, grid, block, 0, s, a, row, scale, groups);
  else if (lanes == 64) hipLaunchKernelGGL(dispatch_kernel<64>, grid, block, 0, s, a, row, scale, groups);
  else hipLaunchKernelGGL(dispatch_kernel<16>, grid, block, 0, s, a, row, scale, groups);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const MoveArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case AR_F32: return combine_dt<AR_F32>(a, s);
    case AR_BF16: return combine_dt<AR_BF16>(a, s);
    case AR_F16: return combine_dt<AR_F16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_expert_combine_bwd(const MoveArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case AR_F32: return combine_bwd_dt<AR_F32>(a, s);
    case AR_BF16: return combine_bwd_dt<AR_BF16>(a, s);
    case AR_F16: return combine_bwd_dt<AR_F16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ar
