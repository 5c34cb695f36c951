// ar_grads.hip -- the norm over all gradients of a model, and the gradients scaled down to a norm. The step between the
// gradients' all-reduce and the optimizer.
//   norm = sqrt(sum of x^2) or max |x| over every element of every tensor
//   out  = x min(1, max_norm / (norm + eps))
//
// Both are bound by HBM: the norm reads every element once, clipping reads it a second time and writes it. A table of
// pieces of a few KiB (planned on the host, kept on the device) spreads tensors of any sizes evenly over the workgroups,
// without a search for a workgroup's elements. Squares are summed in 64 bits: an fp32 gradient's square leaves fp32
// from 1.8e19 up and below 1e-19, and sums over a billion elements would lose digits; the conversions and sums cost
// less than the loads. Partial sums of the workgroups go through the workspace, and every workgroup of the second launch
// adds all of them up in the same order, so nothing is left to atomics and the result depends on the table alone.
// Measured: 1.34 G elements, bf16 but for the norms' fp32 weights: the norm 450 us, 6.0 TB/s; clipping behind it 1025 us, 5.2
// TB/s read and written (a copy of 4 GiB: 4.8). 61 M fp32 elements in tensors of odd sizes: 35 us, 44 with both launches of a call.
// 0.7 M elements: 2.7 + 4.0 us, the launches' own time.
#include "ar_block.h"
#include "ar_grads.h"
#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kThreads = 256;

// Magnitudes as integers order like the numbers, infinities and NaN above them, so that one maximum carries a NaN along.
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// The value of all threads, in every thread, in an order that the number of threads fixes.
template <bool MAX> __device__ __forceinline__ double group_total(double v) {
  __shared__ double lds[kThreads / 64];
  auto join = [](double x, double y) { return MAX ? (x > y ? x : y) : x + y; };  // maxima are whole numbers here
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = join(v, __shfl_xor(v, d, 64));
  __syncthreads();  // a second total in one kernel
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double all = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) all = join(all, lds[w]);
  return all;
}

// One piece's contribution to this thread's sum of squares, or its largest magnitude.
template <int DT, bool MAX> __device__ __forceinline__ void take(const ar_grad_piece& p, double& sum, uint32_t& top) {
  constexpr int V = Traits<DT>::kVec, kAhead = 4;
  const char* in = static_cast<const char*>(p.in);
  auto add = [&](const float* v) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (MAX) top = max(top, magnitude(v[k]));
      else sum = __builtin_fma(static_cast<double>(v[k]), static_cast<double>(v[k]), sum);
    }
  };
  const int64_t vecs = p.numel / V;
  int64_t i = threadIdx.x;
  for (; i + (kAhead - 1) * kThreads < vecs; i += kAhead * kThreads) {
    u32x4 w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) w[u] = ldu16(in + (i + u * kThreads) * 16);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float v[V];
      Slot<DT>::unpack(w[u], v);
      add(v);
    }
  }
  for (; i < vecs; i += kThreads) {
    float v[V];
    Slot<DT>::unpack(ldu16(in + i * 16), v);
    add(v);
  }
  const int64_t e = vecs * V + threadIdx.x;
  if (e < p.numel) {
    float v[V] = {widen<DT>(load_elem<DT>(in, e))};
    add(v);
  }
}

template <bool MAX> __global__ __launch_bounds__(kThreads) void norm_kernel(const GradArgs a) {
  double sum = 0.0;
  uint32_t top = 0;
  for (int64_t i = blockIdx.x; i < a.npieces; i += gridDim.x) {
    const ar_grad_piece p = a.pieces[i];
    if (p.dtype == AR_F32) take<AR_F32, MAX>(p, sum, top);
    else if (p.dtype == AR_BF16) take<AR_BF16, MAX>(p, sum, top);
    else if (p.dtype == AR_F16) take<AR_F16, MAX>(p, sum, top);
  }
  const double all = group_total<MAX>(MAX ? static_cast<double>(top) : sum);
  if (threadIdx.x == 0) gptr<double>(a.partial)[blockIdx.x] = all;
}

// The norm, from the workgroups' partial results.
template <bool MAX> __device__ __forceinline__ float total_norm(const GradArgs& a) {
  double v = 0.0;
  for (int i = threadIdx.x; i < a.groups; i += kThreads) {
    const double x = gptr<double>(a.partial)[i];
    v = MAX ? (x > v ? x : v) : v + x;
  }
  v = group_total<MAX>(v);
  const float norm = MAX ? __uint_as_float(static_cast<uint32_t>(v)) : static_cast<float>(sqrt(v));
  return is_nan(norm) ? __uint_as_float(kNaN32) : norm;
}

template <bool MAX> __global__ __launch_bounds__(kThreads) void finish_kernel(const GradArgs a) {
  const float norm = total_norm<MAX>(a);
  if (threadIdx.x == 0) *gptr<float>(a.norm) = norm;
}

template <int DT> __device__ __forceinline__ void scale(const ar_grad_piece& p, float c) {
  constexpr int V = Traits<DT>::kVec, kAhead = 4;
  const char* in = static_cast<const char*>(p.in);
  char* out = static_cast<char*>(p.out ? p.out : const_cast<void*>(p.in));
  auto one = [&](const u32x4& w) {
    float v[V];
    Slot<DT>::unpack(w, v);
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] *= c;
    return Slot<DT>::pack(v);
  };
  const int64_t vecs = p.numel / V;
  int64_t i = threadIdx.x;
  for (; i + (kAhead - 1) * kThreads < vecs; i += kAhead * kThreads) {
    u32x4 w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) w[u] = ldu16(in + (i + u * kThreads) * 16);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) stu16(out + (i + u * kThreads) * 16, one(w[u]));
  }
  for (; i < vecs; i += kThreads) stu16(out + i * 16, one(ldu16(in + i * 16)));
  const int64_t e = vecs * V + threadIdx.x;
  if (e < p.numel) store_elem<DT>(out, e, narrow<DT>(widen<DT>(load_elem<DT>(in, e)) * c));
}

// Pieces from the last to the first: what the norm read last is still in the last-level cache.
template <bool MAX> __global__ __launch_bounds__(kThreads) void clip_kernel(const GradArgs a) {
  const float norm = total_norm<MAX>(a);
  if (blockIdx.x == 0 && threadIdx.x == 0) *gptr<float>(a.norm) = norm;
  // 1 also where both sides are 0 or infinite; a NaN goes on into the quotient
  const float c = norm + a.eps <= a.max_norm ? 1.0f : a.max_norm / (norm + a.eps);
  for (int64_t i = a.npieces - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const ar_grad_piece p = a.pieces[i];
    if (c == 1.0f && (!p.out || p.out == p.in)) continue;  // x * 1 in place
    if (p.dtype == AR_F32) scale<AR_F32>(p, c);
    else if (p.dtype == AR_BF16) scale<AR_BF16>(p, c);
    else if (p.dtype == AR_F16) scale<AR_F16>(p, c);
  }
}

}  // namespace

hipError_t launch_grad_norm(GradArgs a, bool max_kind, bool clip, hipStream_t s) {
  a.groups = grad_groups(a.npieces);
  if (a.groups > 0) {
    if (max_kind) norm_kernel<true><<<a.groups, kThreads, 0, s>>>(a);
    else norm_kernel<false><<<a.groups, kThreads, 0, s>>>(a);
  }
  if (clip && a.groups > 0) {
    if (max_kind) clip_kernel<true><<<a.groups, kThreads, 0, s>>>(a);
    else clip_kernel<false><<<a.groups, kThreads, 0, s>>>(a);
  } else {
    if (max_kind) finish_kernel<true><<<1, kThreads, 0, s>>>(a);
    else finish_kernel<false><<<1, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace ar
