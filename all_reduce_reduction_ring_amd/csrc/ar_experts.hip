// ar_experts.hip -- tokens sorted by expert and back.
//   sort      slot q = t k + j (token t, choice j) goes to expert ids[q]; the slots of an expert take consecutive rows
//             in slot order, each expert's segment starts on a multiple of `align`; pos[q] is the slot's row (-1: the
//             id is no expert), src[row] the slot (-1: no slot there).
//   dispatch  xs[pos[t, j]] = x[t], pad rows zero
//   combine   out[t] = addend[t] + sum_j w[t, j] ys[pos[t, j]]; without weights it is dispatch's gradient
//   gradient  dys[pos[t, j]] = w[t, j] dout[t], pad rows zero; dw[t, j] = <dout[t], ys[pos[t, j]]>
//
// All of it is bound by HBM, or, in small calls, by one chain of dependent loads (positions, then rows). Everything is laid
// out by token, not by sorted row: a token's own row is then read (or written) once, and its k
// sorted rows, which are whole rows wherever they lie, once each. Rows out of [0, rows) are taken as absent.
#include "ar_block.h"
#include "ar_internal.h"

namespace ar {
namespace {

// ------------------------------------------------------------------------------------------ sort
constexpr int kSortThreads = 1024;
// Few slots go to a workgroup of a quarter of the size, which has a thread for each of 256 experts. With a dispatch of short
// rows behind it, large workgroup against small: 64 slots 5.3 / 4.5 us (8 experts), 5.6 / 4.8 (64), 6.0 / 4.9 (128), 6.0 /
// 5.0 (256); 512 slots 6.0 / 5.3, 6.0 / 5.5, 6.3 / 5.7, 6.3 / 5.9; 1024 slots 6.1 / 5.9, 6.4 / 6.5, 6.5 / 6.7, 6.6 / 7.0.
constexpr int kFewThreads = 256, kFewSlots = 512;
constexpr int kMaxExperts = AR_MAX_EXPERTS;
constexpr int kTileBatch = 8;             // histograms read together
constexpr int kHeld = 4;  // slots a thread reads at a time; a thread's first ones stay in registers between the passes
// Up to here one workgroup sorts everything in one launch (4096 slots, 64 experts: 7.7 us against 7.9 us in two; 8192:
// 11.4 against 8.1 us).
constexpr int64_t kOneGroupSlots = kSortThreads * kHeld;

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

// The experts of slots q0 + lane, q0 + 64 + lane, ... (-1: none, or past `end`).
__device__ __forceinline__ void load_experts(const SortArgs& a, int64_t q0, int64_t end, int (&e)[kHeld]) {
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int64_t q = q0 + u * 64 + (threadIdx.x & 63);
    e[u] = q < end ? gptr<int32_t>(a.ids)[q] : -1;
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) e[u] = e[u] < a.experts ? (e[u] < 0 ? -1 : e[u]) : -1;
}

// Exclusive sum over the workgroup's threads; `lds` holds one value per wave. Returns the total in *total.
template <int WAVES> __device__ __forceinline__ int group_exclusive(int v, int* lds, int* total) {
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
  for (int w = 0; w < WAVES; ++w) {
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
    const int e = gptr<int32_t>(a.ids)[q];
    if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
    gptr<int32_t>(a.hist)[static_cast<int64_t>(blockIdx.x) * a.experts + e] = hist[e];
}

// 131,072 slots to 64 experts: 8.5 us in two launches; with one thread per expert walking the tiles' histograms it was 20.
// One workgroup per tile of slots (one tile: no histogram launch before it). Every workgroup adds up the tiles'
// histograms for itself, so the tiles need no order among each other.
template <int T, int EXPERTS>
__global__ __launch_bounds__(T) void sort_kernel(SortArgs a, int64_t tile) {
  constexpr int kWaves = T / 64;
  __shared__ int next[kWaves][EXPERTS];  // first the waves' counts, then the next row of (wave, expert)
  __shared__ int part[2][T];
  __shared__ int scan[kWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  for (int e = threadIdx.x; e < a.experts; e += T)
    for (int w = 0; w < kWaves; ++w) next[w][e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * tile;
  const int64_t hi = lo + tile < a.slots ? lo + tile : a.slots;
  const int64_t per_wave = (tile + T - 1) / T * 64;
  const int64_t w_lo = lo + wave * per_wave, w_hi = w_lo + per_wave < hi ? w_lo + per_wave : hi;
  int held[kHeld];
  load_experts(a, w_lo, w_hi, held);
  for (int64_t q0 = w_lo; q0 < w_hi; q0 += kHeld * 64) {
    int x[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) x[u] = held[u];
    if (q0 != w_lo) load_experts(a, q0, w_hi, x);
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (x[u] >= 0) atomicAdd(&next[wave][x[u]], 1);
  }
  __syncthreads();
  // thread e: its expert's slots in all tiles, in the tiles before this one, and the segment's start
  const int e = threadIdx.x;
  int total = 0, before = 0;
  if (a.hist) {
    // the tiles' histograms, an equal part of the tiles for each of the 1024 >> bits threads of an expert
    const int x = threadIdx.x & ((1 << bits) - 1), tiles = static_cast<int>(gridDim.x);
    if (x < a.experts) {
      for (int t0 = threadIdx.x >> bits; t0 < tiles; t0 += kTileBatch * (T >> bits)) {
        int c[kTileBatch];
#pragma unroll
        for (int u = 0; u < kTileBatch; ++u) {
          const int t = t0 + u * (T >> bits);
          c[u] = t < tiles ? gptr<int32_t>(a.hist)[static_cast<int64_t>(t) * a.experts + x] : 0;
        }
#pragma unroll
        for (int u = 0; u < kTileBatch; ++u) {
          total += c[u];
          if (t0 + u * (T >> bits) < static_cast<int>(blockIdx.x)) before += c[u];
        }
      }
    }
    part[0][threadIdx.x] = total;
    part[1][threadIdx.x] = before;
    __syncthreads();
    total = before = 0;
    if (e < a.experts) {
      for (int i = e; i < T; i += 1 << bits) {
        total += part[0][i];
        before += part[1][i];
      }
    }
  } else if (e < a.experts) {
    for (int w = 0; w < kWaves; ++w) total += next[w][e];
  }
  const int padded = (total + a.align - 1) / a.align * a.align;
  int rows = 0;
  const int first = group_exclusive<kWaves>(padded, scan, &rows);
  if (e < a.experts) {
    int at = first + before;
    for (int w = 0; w < kWaves; ++w) {
      const int c = next[w][e];
      next[w][e] = at;
      at += c;
    }
    if (blockIdx.x == 0) {
      gptr<int32_t>(a.offsets)[e] = first;
      gptr<int32_t>(a.counts)[e] = total;
      if (e == 0) gptr<int32_t>(a.offsets)[a.experts] = rows;
    }
    part[0][e] = first + total;
    part[1][e] = first + padded;
  }
  for (int64_t p = rows + static_cast<int64_t>(blockIdx.x) * T + threadIdx.x; p < a.rows;
       p += static_cast<int64_t>(gridDim.x) * T)
    gptr<int32_t>(a.src)[p] = -1;
  __syncthreads();
  if (a.align > 1) {  // rows of the segments that no slot takes, 16 lanes to a segment
    constexpr int kAtOnce = T / kPadLanes;
    for (int x = static_cast<int>(blockIdx.x) * kAtOnce + static_cast<int>(threadIdx.x) / kPadLanes; x < a.experts;
         x += static_cast<int>(gridDim.x) * kAtOnce) {
      const sorted_row_t end = part[1][x];
      for (sorted_row_t p = part[0][x] + lane % kPadLanes; p < end; p += kPadLanes) gptr<int32_t>(a.src)[p] = -1;
    }
  }
  for (int64_t q0 = w_lo; q0 < w_hi; q0 += kHeld * 64) {
    int x[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) x[u] = held[u];
    if (q0 != w_lo) load_experts(a, q0, w_hi, x);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int64_t q = q0 + u * 64 + lane;
      if (q - lane >= w_hi) break;
      const bool in = x[u] >= 0;
      const uint64_t same = same_expert(x[u], in, bits);
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      int p = 0;
      if (in && rank == 0) p = atomicAdd(&next[wave][x[u]], __popcll(same));  // the lowest lane takes rows for all of them
      p = __shfl(p, in ? __ffsll(static_cast<unsigned long long>(same)) - 1 : lane, 64) + rank;
      if (q < w_hi) gptr<int32_t>(a.pos)[q] = in ? p : -1;
      if (in) gptr<int32_t>(a.src)[p] = static_cast<int32_t>(q);
    }
  }
}

// ------------------------------------------------------------------------------------------ rows
// A workgroup of LANES threads (64, 128 or 256) takes a token. What it knows about the token's rows is kept in scalar
// registers: the rows' addresses and the tests whether they are there.
// The rows of choices j0 .. j0 + 7 of token t (-1: none); in scalar registers. One load for all of them.
__device__ __forceinline__ void load_rows(const MoveArgs& a, int64_t t, int j0, int (&p)[kChoices]) {
  const int lane = threadIdx.x & 63;
  int v = -1;
  if (lane < kChoices && j0 + lane < a.k) v = gptr<int32_t>(a.pos + t * a.k)[j0 + lane];
  v = v >= 0 && v < a.rows ? v : -1;
#pragma unroll
  for (int j = 0; j < kChoices; ++j) p[j] = __builtin_amdgcn_readlane(v, j);
}
// Their weights, 0 where there is no row.
__device__ __forceinline__ void load_weights(const MoveArgs& a, int64_t t, int j0, const int (&p)[kChoices],
                                             float (&w)[kChoices]) {
  const int lane = threadIdx.x & 63;
  float v = 1.0f;
  if (a.weights && lane < kChoices && j0 + lane < a.k) v = gptr<float>(a.weights + t * a.k)[j0 + lane];
#pragma unroll
  for (int j = 0; j < kChoices; ++j)
    w[j] = p[j] >= 0 ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j)) : 0.0f;
}

__device__ __forceinline__ void zero_bytes(char* to, int64_t bytes, int64_t part, int64_t parts) {
  const int64_t threads = blockDim.x;
  for (int64_t b = (part * threads + threadIdx.x) * 16; b < bytes; b += parts * threads * 16) {
    if (b + 16 <= bytes) stu16_nt(to + b, u32x4{0, 0, 0, 0});
    else
      for (int64_t c = b; c < bytes; ++c) gptr<uint8_t>(to)[c] = 0;
  }
}

// The pad rows of one expert's segment, zeroed by `parts` workgroups.
__device__ __forceinline__ void zero_pads(const MoveArgs& a, int group, int parts, int64_t row_bytes,
                                          int64_t scale_bytes) {
  const int e = group / parts, part = group % parts;
  int64_t lo = static_cast<int64_t>(gptr<int32_t>(a.offsets)[e]) + gptr<int32_t>(a.counts)[e];
  int64_t hi = gptr<int32_t>(a.offsets)[e + 1];
  if (lo < 0) lo = 0;
  if (hi > a.rows) hi = a.rows;
  if (lo >= hi) return;
  zero_bytes(static_cast<char*>(a.y) + lo * row_bytes, (hi - lo) * row_bytes, part, parts);
  if (scale_bytes)
    zero_bytes(static_cast<char*>(a.y_scales) + lo * scale_bytes, (hi - lo) * scale_bytes, part, parts);
}

// The first pad_groups workgroups zero the experts' pad rows (first, so that none of them is left running alone at the
// end), the others copy their tokens' rows. U 16-byte vectors a lane at a time. The last vector of a row is moved up to
// end with it (its first bytes are then written twice, with the same values); rows below 16 bytes go byte by byte.
// 128 lanes of 4 vectors, 16,384 x 8 rows of 8 KiB with the sort: 235 us (the kernel 222, 5.4 TB/s, mostly writes); 256
// lanes of 2 252 us, 128 of 2 243, 64 of 2, 4 or 8 249 to 251, a wave per choice 248. Rows of 512 bytes to 16 KiB agree.
constexpr int kCopyLanes = 128, kCopyUnroll = 4;
template <int MODE>
__global__ __launch_bounds__(kCopyLanes) void dispatch_kernel(MoveArgs a, row_bytes_t row_bytes, row_bytes_t scale_bytes,
                                                              int pad_groups, int pad_parts) {
  constexpr int LANES = kCopyLanes, U = kCopyUnroll;
  if (static_cast<int>(blockIdx.x) < pad_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x), pad_parts, row_bytes, scale_bytes);
    return;
  }
  const row_bytes_t lane = threadIdx.x;
  for (int64_t t = blockIdx.x - pad_groups; t < a.tokens; t += gridDim.x - pad_groups) {
    const char* from = static_cast<const char*>(a.x) + t * row_bytes;
    int p[kChoices];
    // Calls that stream read the positions before the row, all others the row first, while the positions are on their way.
    // With the sort, row first against positions first: 48 tokens, 4 choices of 4 KiB 6.1 / 6.2 us; 1536 x 8 of 8 KiB 30.2 /
    // 31.4; 16,384 x 8 of 8194 bytes 301 / 314; streaming, 16,384 x 8 of 8 KiB, 251 / 237. Few tokens of wide rows lose by
    // it: 48 tokens, 4 choices of 8 KiB 7.0 / 6.6; 10 choices of 16 KiB, whose positions are read in every step, 13.1 / 11.2.
    auto put = [&](const u32x4 (&v)[U], const uint32_t (&at)[U], row_bytes_t b0) {
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (p[j] < 0) continue;
        char* to = static_cast<char*>(a.y) + p[j] * static_cast<int64_t>(row_bytes);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b0 + u * LANES * 16 < row_bytes) st_row<MODE>(to, at[u], v[u]);
      }
    };
    auto get = [&](u32x4 (&v)[U], uint32_t (&at)[U], row_bytes_t b0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at[u] = vector_place(b0 + u * LANES * 16, row_bytes);
        v[u] = ld_row<kCached>(from, at[u]);
      }
    };
    u32x4 v[U];
    uint32_t at[U];
    if (row_bytes >= kVectorBytes) {
      if constexpr (MODE == kStream) {
        for (int left = a.k; left > 0; left -= kChoices) {
          const int j0 = a.k - left;
          load_rows(a, t, j0, p);
          for (row_bytes_t b0 = lane * 16; b0 < row_bytes; b0 += LANES * U * 16) {
            get(v, at, b0);
            put(v, at, b0);
          }
        }
      } else {
        for (row_bytes_t b0 = 0; b0 < row_bytes; b0 += LANES * U * 16) {
          get(v, at, b0 + lane * 16);
          for (int left = a.k; left > 0; left -= kChoices) {
            const int j0 = a.k - left;
            if (b0 == 0 || a.k > kChoices) load_rows(a, t, j0, p);
            put(v, at, b0 + lane * 16);
          }
        }
      }
    }
    for (int left = a.k; left > 0; left -= kChoices) {
      const int j0 = a.k - left;
      if (row_bytes < kVectorBytes || a.k > kChoices) load_rows(a, t, j0, p);
      if (row_bytes < kVectorBytes && lane < row_bytes) {
        const uint8_t v = gptr<uint8_t>(from)[lane];
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (p[j] >= 0) gptr<uint8_t>(static_cast<char*>(a.y) + p[j] * static_cast<int64_t>(row_bytes))[lane] = v;
      }
      for (row_bytes_t b = lane * 4; b < scale_bytes; b += LANES * 4) {
        const uint32_t v = *gptr<uint32_t>(static_cast<const char*>(a.x_scales) + t * scale_bytes + opaque(b));
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (p[j] >= 0)
            *gptr<uint32_t>(static_cast<char*>(a.y_scales) + p[j] * static_cast<int64_t>(scale_bytes) + opaque(b)) = v;
      }
    }
  }
}

// First element of the wave's part of a row, and this lane's offset from it. The loops over a row run on the wave's
// first element, so that all lanes stay in them (load_rows reads lanes 0 to 7); lanes past the end read clamped places.
template <int DT> __device__ __forceinline__ int wave_first() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x / 64) * 64 * Traits<DT>::kVec;
}
template <int DT> __device__ __forceinline__ int lane_elem() { return static_cast<int>(threadIdx.x & 63) * Traits<DT>::kVec; }

// The sum runs in fp32 over the choices in order, the addend last, and is rounded once. A slot without a row adds
// nothing: its row is not read. The rows of up to eight choices, U vectors of each, are on their way together (16,384 x 8
// rows of 8 KiB onto the residual: 222 us, 6.0 TB/s; with a wait after every row 342).
template <int DT, int LANES, int U, int MODE>
__global__ __launch_bounds__(LANES) void combine_kernel(MoveArgs a) {
  constexpr int V = Traits<DT>::kVec;
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    int p[kChoices];
    float w[kChoices];
    load_rows(a, t, 0, p);
    load_weights(a, t, 0, p, w);
    for (int b0 = wave_first<DT>(); b0 < a.hidden; b0 += LANES * V * U) {
      float acc[U][V];
      u32x4 add[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
        if (a.extra && b0 + u * LANES * V < a.hidden)
          add[u] = load_vec<DT, MODE>(static_cast<const char*>(a.extra) + t * row, b0 + u * LANES * V + lane_elem<DT>(),
                                       a.hidden);
      }
      for (int left = a.k; left > 0; left -= kChoices) {
        const int j0 = a.k - left;
        if (a.k > kChoices) {
          load_rows(a, t, j0, p);
          load_weights(a, t, j0, p, w);
        }
        u32x4 x[kChoices][U];
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
          if (p[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (b0 + u * LANES * V < a.hidden)
              x[j][u] = load_vec<DT, MODE>(static_cast<const char*>(a.x) + p[j] * row,
                                            b0 + u * LANES * V + lane_elem<DT>(), a.hidden);
        }
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
          if (p[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (b0 + u * LANES * V >= a.hidden) continue;
            float v[V];
            Slot<DT>::unpack(x[j][u], v);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w[j], v[i], acc[u][i]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b0 + u * LANES * V >= a.hidden) continue;
        const int e = b0 + u * LANES * V + lane_elem<DT>();
        if (a.extra) {
          float v[V];
          Slot<DT>::unpack(add[u], v);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] += v[i];
        }
        settle_vec<DT, MODE>(acc[u], e, a.hidden);
        store_vec<DT, MODE>(static_cast<char*>(a.y) + t * row, e, a.hidden, Slot<DT>::pack(acc[u]));
      }
    }
  }
}

// The waves' dot products are joined in LDS. The first pad_groups workgroups zero the pad rows. 8192 x 4 rows of 8 KiB:
// 111 us, 5.5 TB/s. The token's gradient is read with the rows, behind the positions: ahead of them it was level in 2-byte
// types and slower in fp32, by a wait in every step (16 x 4 rows of 8192 8.7 -> 11.7 us, 8192 x 8 of 1024 108 -> 122).
template <int DT, int LANES, int U, int MODE>
__global__ __launch_bounds__(LANES) void combine_bwd_kernel(MoveArgs a, int pad_groups, int pad_parts) {
  constexpr int V = Traits<DT>::kVec;
  constexpr int kWaves = LANES / 64;
  __shared__ float lds[2][kWaves][kChoices];
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  if (static_cast<int>(blockIdx.x) < pad_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x), pad_parts, row, 0);
    return;
  }
  int flip = 0;
  for (int64_t t = blockIdx.x - pad_groups; t < a.tokens; t += gridDim.x - pad_groups) {
    for (int left = a.k; left > 0; left -= kChoices, flip ^= 1) {
      const int j0 = a.k - left;
      int p[kChoices];
      float w[kChoices], dot[kChoices];
      load_rows(a, t, j0, p);
      load_weights(a, t, j0, p, w);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) dot[j] = 0.0f;
      for (int b0 = wave_first<DT>(); b0 < a.hidden; b0 += LANES * V * U) {
        u32x4 d[U], x[kChoices][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b0 + u * LANES * V < a.hidden)
            d[u] = load_vec<DT, MODE>(static_cast<const char*>(a.extra) + t * row, b0 + u * LANES * V + lane_elem<DT>(),
                                      a.hidden);
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
          if (p[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (b0 + u * LANES * V < a.hidden)
              x[j][u] = load_vec<DT, MODE>(static_cast<const char*>(a.x) + p[j] * row,
                                            b0 + u * LANES * V + lane_elem<DT>(), a.hidden);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (b0 + u * LANES * V >= a.hidden) continue;
          const int e = b0 + u * LANES * V + lane_elem<DT>();
          float dv[V];
          Slot<DT>::unpack(d[u], dv);
          settle_vec<DT, MODE>(dv, e, a.hidden);
#pragma unroll
          for (int j = 0; j < kChoices; ++j) {
            if (p[j] < 0) continue;
            float v[V], y[V];
            Slot<DT>::unpack(x[j][u], v);
            settle_vec<DT, MODE>(v, e, a.hidden);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              dot[j] = fmaf(dv[i], v[i], dot[j]);
              y[i] = w[j] * dv[i];
            }
            store_vec<DT, MODE>(static_cast<char*>(a.y) + p[j] * row, e, a.hidden, Slot<DT>::pack(y));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kChoices; ++j)
        if (p[j] >= 0) dot[j] = wave_sum(dot[j]);
      if constexpr (kWaves > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < kChoices; ++j) lds[flip][threadIdx.x >> 6][j] = dot[j];
        }
        __syncthreads();  // one buffer is read while the next step fills the other
        if (threadIdx.x < kChoices && j0 + static_cast<int>(threadIdx.x) < a.k) {
          float sum = 0.0f;
#pragma unroll
          for (int u = 0; u < kWaves; ++u) sum += lds[flip][u][threadIdx.x];
          gptr<float>(a.dweights + t * a.k)[j0 + threadIdx.x] = sum;
        }
      } else if (threadIdx.x == 0) {
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (j0 + j < a.k) gptr<float>(a.dweights + t * a.k)[j0 + j] = dot[j];
      }
    }
  }
}

// Slots per workgroup of the tiled sort: 1024, more where that would make over 512 tiles (every workgroup reads all
// tiles' histograms).
int64_t sort_tile(int64_t slots) {
  const int64_t even = (slots + 511) / 512;
  return (even + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// ------------------------------------------------------------------------------------------ short rows
// Rows of up to 32 vectors: LANES lanes (8, 16 or 32) take a token, one vector a lane, several tokens a wave. A wave per
// token leaves most lanes idle there, and the kernels wait for one chain of loads after another: positions, rows. 16,384
// tokens of 4 choices, bf16, against a wave per token: 64 wide, combine 13.3 -> 3.7 us, its gradient 25.5 -> 6.1, sort
// and dispatch 19.3 -> 11.7; 256 wide, 14.1 -> 9.4, 26.1 -> 15.1, 21.2 -> 17.1.
constexpr int kShortThreads = 256;

// The rows of choices j0 .. j0 + 7 of token t (-1: none), one register each.
__device__ __forceinline__ void load_rows_each(const MoveArgs& a, int64_t t, int j0, int (&p)[kChoices]) {
#pragma unroll
  for (int j = 0; j < kChoices; ++j) p[j] = j0 + j < a.k ? gptr<int32_t>(a.pos + t * a.k)[j0 + j] : -1;
#pragma unroll
  for (int j = 0; j < kChoices; ++j) p[j] = p[j] >= 0 && p[j] < a.rows ? p[j] : -1;
}

template <int LANES>
__global__ __launch_bounds__(kShortThreads) void dispatch_short_kernel(MoveArgs a, row_bytes_t row_bytes,
                                                                       row_bytes_t scale_bytes, int pad_groups,
                                                                       int pad_parts) {
  if (static_cast<int>(blockIdx.x) < pad_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x), pad_parts, row_bytes, scale_bytes);
    return;
  }
  constexpr int kTokens = kShortThreads / LANES;
  const row_bytes_t lane = threadIdx.x % LANES;
  for (int64_t t = static_cast<int64_t>(blockIdx.x - pad_groups) * kTokens + threadIdx.x / LANES; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x - pad_groups) * kTokens) {
    const int64_t at = vector_place(lane * 16, row_bytes);
    const u32x4 v = ldu16(static_cast<const char*>(a.x) + t * row_bytes + at);
    uint32_t sc = 0;
    if (lane * 4 < scale_bytes) sc = *gptr<uint32_t>(static_cast<const char*>(a.x_scales) + t * scale_bytes + lane * 4);
    for (int left = a.k; left > 0; left -= kChoices) {
      const int j0 = a.k - left;
      int p[kChoices];
      load_rows_each(a, t, j0, p);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (p[j] < 0) continue;
        if (lane * 16 < row_bytes) stu16(static_cast<char*>(a.y) + p[j] * static_cast<int64_t>(row_bytes) + at, v);
        if (lane * 4 < scale_bytes)
          *gptr<uint32_t>(static_cast<char*>(a.y_scales) + p[j] * static_cast<int64_t>(scale_bytes) + lane * 4) = sc;
      }
    }
  }
}

template <int DT, int LANES, int MODE>
__global__ __launch_bounds__(kShortThreads) void combine_short_kernel(MoveArgs a) {
  constexpr int V = Traits<DT>::kVec, kTokens = kShortThreads / LANES;
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  const int e = static_cast<int>(threadIdx.x) % LANES * V;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / LANES; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * kTokens) {
    float acc[V];
    u32x4 add = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (a.extra) add = load_vec<DT, MODE>(static_cast<const char*>(a.extra) + t * row, e, a.hidden);
    for (int left = a.k; left > 0; left -= kChoices) {
      const int j0 = a.k - left;
      int p[kChoices];
      float w[kChoices];
      load_rows_each(a, t, j0, p);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) w[j] = a.weights && j0 + j < a.k ? gptr<float>(a.weights + t * a.k)[j0 + j] : 1.0f;
      u32x4 x[kChoices];
#pragma unroll
      for (int j = 0; j < kChoices; ++j)
        if (p[j] >= 0) x[j] = load_vec<DT, MODE>(static_cast<const char*>(a.x) + p[j] * row, e, a.hidden);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (p[j] < 0) continue;
        float v[V];
        Slot<DT>::unpack(x[j], v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(w[j], v[i], acc[i]);
      }
    }
    if (a.extra) {
      float v[V];
      Slot<DT>::unpack(add, v);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += v[i];
    }
    settle_vec<DT, MODE>(acc, e, a.hidden);
    store_vec<DT, MODE>(static_cast<char*>(a.y) + t * row, e, a.hidden, Slot<DT>::pack(acc));
  }
}

template <int DT, int LANES, int MODE>
__global__ __launch_bounds__(kShortThreads) void combine_bwd_short_kernel(MoveArgs a, int pad_groups, int pad_parts) {
  constexpr int V = Traits<DT>::kVec, kTokens = kShortThreads / LANES;
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  if (static_cast<int>(blockIdx.x) < pad_groups) {
    zero_pads(a, static_cast<int>(blockIdx.x), pad_parts, row, 0);
    return;
  }
  const int e = static_cast<int>(threadIdx.x) % LANES * V;
  for (int64_t t = static_cast<int64_t>(blockIdx.x - pad_groups) * kTokens + threadIdx.x / LANES; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x - pad_groups) * kTokens) {
    const u32x4 d = load_vec<DT, MODE>(static_cast<const char*>(a.extra) + t * row, e, a.hidden);
    for (int left = a.k; left > 0; left -= kChoices) {
      const int j0 = a.k - left;
      int p[kChoices];
      float w[kChoices];
      load_rows_each(a, t, j0, p);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) w[j] = j0 + j < a.k ? gptr<float>(a.weights + t * a.k)[j0 + j] : 0.0f;
      u32x4 x[kChoices];
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        x[j] = u32x4{0, 0, 0, 0};
        if (p[j] >= 0) x[j] = load_vec<DT, MODE>(static_cast<const char*>(a.x) + p[j] * row, e, a.hidden);
      }
      float dv[V];
      Slot<DT>::unpack(d, dv);
      settle_vec<DT, MODE>(dv, e, a.hidden);
      float dot[kChoices];
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        dot[j] = 0.0f;
        if (j0 + j >= a.k) continue;
        float v[V], y[V];
        Slot<DT>::unpack(x[j], v);
        settle_vec<DT, MODE>(v, e, a.hidden);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot[j] = fmaf(dv[i], v[i], dot[j]);
          y[i] = w[j] * dv[i];
        }
        dot[j] = lanes_sum<LANES>(dot[j]);
        if (p[j] < 0) dot[j] = 0.0f;  // rather than the gradient's infinities and NaN times zero
        else store_vec<DT, MODE>(static_cast<char*>(a.y) + p[j] * row, e, a.hidden, Slot<DT>::pack(y));
      }
      if (e == 0) {
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
          if (j0 + j < a.k) gptr<float>(a.dweights + t * a.k)[j0 + j] = dot[j];
      }
    }
  }
}

constexpr int kUnroll = 2;  // vectors of a row a lane takes at a time

// Lanes per token: as many as have two vectors each, up to 256 (65,536 x 4 rows of 2 KiB, combine: 64 lanes 114 us, 128
// 127, 256 185); with few tokens, where waves are short, twice as many (777 x 3 rows of 1025 fp32: 64 lanes 5.2 us, 256
// 4.1). The gradient's dot products are added lane by lane, so their bits go by this too.
int lanes_for(int64_t vectors, int64_t tokens) {
  if (tokens < 2048) vectors *= 2;
  return vectors > 256 ? 256 : vectors > 128 ? 128 : 64;
}
// A launch has fewer than 2^32 threads.
int64_t groups_for(int64_t tokens) { return tokens < (1 << 23) ? tokens : (1 << 23); }

// Lanes per token of the kernels for short rows (0: the row is not short).
int short_lanes(int64_t vectors) { return vectors > 32 ? 0 : vectors > 16 ? 32 : vectors > 8 ? 16 : 8; }
unsigned short_groups(int64_t tokens, int lanes) {
  const int64_t per = kShortThreads / lanes;
  return static_cast<unsigned>(groups_for((tokens + per - 1) / per));
}

// Workgroups per expert that zero its pad rows: one for every 64 KiB that an expert's pads can have on average.
int pad_parts(const MoveArgs& a, int64_t row_bytes) {
  const int64_t spare = (a.rows - a.tokens * a.k) * row_bytes / a.experts >> 16;
  return spare < 1 ? 1 : spare > 16 ? 16 : static_cast<int>(spare);
}

template <int DT, int LANES, int U, int MODE> hipError_t combine_run(const MoveArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((combine_kernel<DT, LANES, U, MODE>), dim3(static_cast<unsigned>(groups_for(a.tokens))),
                     dim3(LANES), 0, s, a);
  return hipGetLastError();
}
template <int DT, int MODE> hipError_t combine_lanes(const MoveArgs& a, int lanes, hipStream_t s) {
  if (lanes == 256) return combine_run<DT, 256, kUnroll, MODE>(a, s);
  if (lanes == 128) return combine_run<DT, 128, kUnroll, MODE>(a, s);
  return combine_run<DT, 64, kUnroll, MODE>(a, s);
}
template <int DT, int LANES> hipError_t combine_short(const MoveArgs& a, bool exact, hipStream_t s) {
  const dim3 grid(short_groups(a.tokens, LANES)), block(kShortThreads);
  if (exact) hipLaunchKernelGGL((combine_short_kernel<DT, LANES, kExact>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_short_kernel<DT, LANES, kCached>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <int DT> hipError_t combine_dt(const MoveArgs& a, hipStream_t s) {
  constexpr int V = Traits<DT>::kVec;
  const bool exact = a.hidden < V || (a.extra == a.y && a.hidden % V != 0);
  switch (short_lanes((a.hidden + V - 1) / V)) {
    case 8: return combine_short<DT, 8>(a, exact, s);
    case 16: return combine_short<DT, 16>(a, exact, s);
    case 32: return combine_short<DT, 32>(a, exact, s);
  }
  // In place at widths that a vector does not divide, one wave a token, against apart from the addend: 16,384 x 8 rows of
  // 4097 bf16 291 / 270 us, 16,384 x 4 of 1001 fp32 90 / 79, 1000 x 4 of 4097 bf16 21.8 / 12.3, 48 x 4 of 1025 bf16 6.1 / 3.2.
  if (exact) return combine_run<DT, 64, 1, kExact>(a, s);
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  const int lanes = lanes_for((a.hidden + V - 1) / V, a.tokens);
  return streams(a.tokens * row * (int64_t(a.k) + 2), row) ? combine_lanes<DT, kStream>(a, lanes, s)
                                                  : combine_lanes<DT, kCached>(a, lanes, s);
}

template <int DT, int LANES, int U, int MODE> hipError_t combine_bwd_run(const MoveArgs& a, hipStream_t s) {
  const int parts = pad_parts(a, static_cast<int64_t>(a.hidden) * Traits<DT>::kSize);
  const int pads = a.offsets ? a.experts * parts : 0;
  hipLaunchKernelGGL((combine_bwd_kernel<DT, LANES, U, MODE>),
                     dim3(static_cast<unsigned>(groups_for(a.tokens) + pads)), dim3(LANES), 0, s, a, pads, parts);
  return hipGetLastError();
}
template <int DT, int U, int MODE> hipError_t combine_bwd_lanes(const MoveArgs& a, int lanes, hipStream_t s) {
  if (lanes == 256) return combine_bwd_run<DT, 256, U, MODE>(a, s);
  if (lanes == 128) return combine_bwd_run<DT, 128, U, MODE>(a, s);
  return combine_bwd_run<DT, 64, U, MODE>(a, s);
}
template <int DT, int LANES> hipError_t combine_bwd_short(const MoveArgs& a, bool exact, hipStream_t s) {
  const int parts = pad_parts(a, static_cast<int64_t>(a.hidden) * Traits<DT>::kSize);
  const int pads = a.offsets ? a.experts * parts : 0;
  const dim3 grid(short_groups(a.tokens, LANES) + pads), block(kShortThreads);
  if (exact) hipLaunchKernelGGL((combine_bwd_short_kernel<DT, LANES, kExact>), grid, block, 0, s, a, pads, parts);
  else hipLaunchKernelGGL((combine_bwd_short_kernel<DT, LANES, kCached>), grid, block, 0, s, a, pads, parts);
  return hipGetLastError();
}
template <int DT> hipError_t combine_bwd_dt(const MoveArgs& a, hipStream_t s) {
  constexpr int V = Traits<DT>::kVec;
  const bool exact = a.hidden < V || (a.x == a.y && a.hidden % V != 0);
  switch (short_lanes((a.hidden + V - 1) / V)) {
    case 8: return combine_bwd_short<DT, 8>(a, exact, s);
    case 16: return combine_bwd_short<DT, 16>(a, exact, s);
    case 32: return combine_bwd_short<DT, 32>(a, exact, s);
  }
  const int64_t row = static_cast<int64_t>(a.hidden) * Traits<DT>::kSize;
  const int lanes = lanes_for((a.hidden + V - 1) / V, a.tokens);
  // in place with the same lanes, so that dweights has the same bits
  if (exact) return combine_bwd_lanes<DT, 1, kExact>(a, lanes, s);
  return streams(a.tokens * row * (2 * int64_t(a.k) + 1), row) ? combine_bwd_lanes<DT, kUnroll, kStream>(a, lanes, s)
                                                      : combine_bwd_lanes<DT, kUnroll, kCached>(a, lanes, s);
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
    const int64_t tile = a.slots > 0 ? a.slots : 1;
    if (a.slots <= kFewSlots && a.experts <= kFewThreads)
      hipLaunchKernelGGL((sort_kernel<kFewThreads, kFewThreads>), dim3(1), dim3(kFewThreads), 0, s, b, tile);
    else
      hipLaunchKernelGGL((sort_kernel<kSortThreads, kMaxExperts>), dim3(1), block, 0, s, b, tile);
    return hipGetLastError();
  }
  const int64_t tile = sort_tile(a.slots);
  const dim3 grid(static_cast<unsigned>((a.slots + tile - 1) / tile));
  hipLaunchKernelGGL(sort_hist_kernel, grid, block, 0, s, a, tile);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sort_kernel<kSortThreads, kMaxExperts>), grid, block, 0, s, a, tile);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const MoveArgs& a, int esize, hipStream_t s) {
  const row_bytes_t row = static_cast<row_bytes_t>(a.hidden) * static_cast<row_bytes_t>(esize);
  const row_bytes_t scale = a.x_scales ? row_scale_bytes(static_cast<row_bytes_t>(a.hidden), AR_FP8_BLOCK) : 0;
  if (a.tokens == 0) return hipSuccess;
  const int parts = pad_parts(a, row);
  const int pads = a.offsets ? a.experts * parts : 0;
  const int lanes = row < kVectorBytes ? 0 : short_lanes(row_vectors(row));
  if (lanes) {
    const dim3 grid(short_groups(a.tokens, lanes) + pads), block(kShortThreads);
    if (lanes == 8) hipLaunchKernelGGL(dispatch_short_kernel<8>, grid, block, 0, s, a, row, scale, pads, parts);
    else if (lanes == 16) hipLaunchKernelGGL(dispatch_short_kernel<16>, grid, block, 0, s, a, row, scale, pads, parts);
    else hipLaunchKernelGGL(dispatch_short_kernel<32>, grid, block, 0, s, a, row, scale, pads, parts);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(groups_for(a.tokens) + pads)), block(kCopyLanes);
  if (streams(a.tokens * row * (int64_t(a.k) + 1), row))
    hipLaunchKernelGGL(dispatch_kernel<kStream>, grid, block, 0, s, a, row, scale, pads, parts);
  else
    hipLaunchKernelGGL(dispatch_kernel<kCached>, grid, block, 0, s, a, row, scale, pads, parts);
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
