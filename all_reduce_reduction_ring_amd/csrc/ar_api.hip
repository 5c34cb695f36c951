// ar_api.hip -- the C ABI of libar: argument validation, dispatch to the kernels, the per-thread last-call
// record. Nothing here allocates device memory or synchronises the stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "ar.h"
#include "ar_block.h"
#include "ar_grads.h"
#include "ar_internal.h"
#include "ar_products.h"

namespace ar {

int cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 0;
  const int slot = dev < 64 ? dev : 63;
  int v = cache[slot].load(std::memory_order_relaxed);
  if (v <= 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cache[slot].store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace ar

namespace ar {

template <int DT>
hipError_t collapsed_for(const RankPtrs& p, int n, int64_t count, int op, int algo, int64_t head, hipStream_t s) {
  if (large_launch(n, count, kElemSize<DT>, algo)) return launch_collapsed_dt<DT, 1>(p, n, count, op, algo, head, s);
  return launch_collapsed_dt<DT, 0>(p, n, count, op, algo, head, s);
}

hipError_t launch_collapsed(const RankPtrs& p, int n, int64_t count, int dtype, int op, int algo, int64_t head,
                            hipStream_t s) {
  switch (dtype) {
    case AR_F32: return collapsed_for<AR_F32>(p, n, count, op, algo, head, s);
    case AR_BF16: return collapsed_for<AR_BF16>(p, n, count, op, algo, head, s);
    case AR_F16: return collapsed_for<AR_F16>(p, n, count, op, algo, head, s);
    case AR_I32: return collapsed_for<AR_I32>(p, n, count, op, algo, head, s);
    default: return hipErrorInvalidValue;
  }
}

// Measured on MI355X (N = 8, 256 MiB bf16 per rank, in place): slots starting 16 bytes past a 256-byte boundary
// ran 24% slower than aligned ones, 64 bytes past 10%, 128 bytes past 2.5%; a multiple of 256 bytes matched.
// Buffers whose addresses differ modulo 16 but are all multiples of 4 take slots from element 0.
int64_t vector_head(const RankPtrs& p, int n, int64_t count, int esize) {
  constexpr uintptr_t kWide = 256, kNarrow = 16;
  constexpr int64_t kWideMinBytes = 1 << 20;
  const uintptr_t aligns[2] = {count * esize >= kWideMinBytes ? kWide : kNarrow, kNarrow};
  for (uintptr_t al : aligns) {
    const uintptr_t res = reinterpret_cast<uintptr_t>(p.in[0]) % al;
    bool same = true;
    for (int r = 0; r < n && same; ++r)
      same = reinterpret_cast<uintptr_t>(p.in[r]) % al == res && reinterpret_cast<uintptr_t>(p.out[r]) % al == res;
    if (!same) continue;
    if (res % static_cast<uintptr_t>(esize) != 0) return -1;
    const int64_t head = static_cast<int64_t>(((al - res) % al) / static_cast<uintptr_t>(esize));
    return head < count ? head : count;
  }
  // Addresses that differ modulo 16: the 16-byte accesses need only 4-byte alignment, so slots from element 0
  // still work when every address is a multiple of 4 (some vectors then straddle two cache lines).
  for (int r = 0; r < n; ++r)
    if ((reinterpret_cast<uintptr_t>(p.in[r]) | reinterpret_cast<uintptr_t>(p.out[r])) % 4 != 0) return -1;
  return 0;
}

template <int DT>
hipError_t segments_for(const RankPtrs& p, int n, const int64_t* counts, int nseg, int op, int algo, hipStream_t s) {
  int64_t total = 0;
  for (int i = 0; i < nseg; ++i) total += counts[i];
  if (large_launch(n, total, kElemSize<DT>, algo)) return launch_segments_dt<DT, 1>(p, n, counts, nseg, op, algo, s);
  return launch_segments_dt<DT, 0>(p, n, counts, nseg, op, algo, s);
}

hipError_t launch_segments(const RankPtrs& p, int n, const int64_t* counts, int nseg, int dtype, int op, int algo,
                           hipStream_t s) {
  switch (dtype) {
    case AR_F32: return segments_for<AR_F32>(p, n, counts, nseg, op, algo, s);
    case AR_BF16: return segments_for<AR_BF16>(p, n, counts, nseg, op, algo, s);
    case AR_F16: return segments_for<AR_F16>(p, n, counts, nseg, op, algo, s);
    case AR_I32: return segments_for<AR_I32>(p, n, counts, nseg, op, algo, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ar

namespace {

thread_local ar_call_record g_last;
thread_local bool g_has_last = false;
thread_local uint64_t g_seq = 0;

// AR_LOG set to anything but "" or "0" in the environment (read once, at the first call): one line per call on
// stderr, written when the call returns (its work may still be queued).
bool log_calls() {
  static const bool on = [] {
    const char* v = std::getenv("AR_LOG");
    return v != nullptr && v[0] != '\0' && std::strcmp(v, "0") != 0;
  }();
  return on;
}

int finish(const char* entry, int nranks, size_t count, int dtype, int op, int algo, int status) {
  g_last.seq = ++g_seq;
  g_last.entry = entry;
  g_last.nranks = nranks;
  g_last.count = count;
  g_last.dtype = dtype;
  g_last.op = op;
  g_last.algo = algo;
  g_last.status = status;
  g_has_last = true;
  if (log_calls())
    std::fprintf(stderr, "ar: seq=%llu %s nranks=%d count=%zu dtype=%d op=%d algo=%d status=%d\n",
                 static_cast<unsigned long long>(g_last.seq), entry, nranks, count, dtype, op, algo, status);
  return status;
}

int esize_of(int dtype) { return (dtype == AR_BF16 || dtype == AR_F16) ? 2 : 4; }
bool valid_dtype(int d) { return d >= AR_F32 && d <= AR_I32; }
bool valid_op(int o) { return o >= AR_SUM && o <= AR_MAX; }
bool valid_algo(int a) { return a >= AR_ALGO_RING && a <= AR_ALGO_AUTO; }
bool is_pow2(int n) { return n > 0 && (n & (n - 1)) == 0; }

// Cost table of the tree and the ring (time = steps * alpha + bytes per rank / bandwidth): the tree wins iff
// bytes < N (N - 1 - L) alpha B, L = ceil(log2 N). alpha [ns] * B [GB/s] is bytes.
int auto_algo(int nranks, size_t count, int dtype) {
  int levels = 0;
  while ((1 << levels) < nranks) ++levels;
  const int64_t spare_steps = static_cast<int64_t>(nranks) - 1 - levels;
  if (spare_steps <= 0) return AR_ALGO_RING;
  const uint64_t threshold = static_cast<uint64_t>(nranks) * static_cast<uint64_t>(spare_steps) *
                             static_cast<uint64_t>(AR_AUTO_STEP_NS) * static_cast<uint64_t>(AR_AUTO_LINK_GBPS);
  const uint64_t es = static_cast<uint64_t>(esize_of(dtype));
  // count * es < threshold, without overflow: count < ceil(threshold / es)
  return static_cast<uint64_t>(count) < (threshold + es - 1) / es ? AR_ALGO_TREE : AR_ALGO_RING;
}

size_t workspace_bytes(int nranks, size_t count, int dtype, int algo) {
  if (algo == AR_ALGO_AUTO) algo = auto_algo(nranks, count, dtype);
  const bool stepwise =
      algo == AR_ALGO_RING_STEPWISE || algo == AR_ALGO_RHD_STEPWISE || algo == AR_ALGO_TREE_STEPWISE;
  if (!stepwise || esize_of(dtype) == 4 || nranks < 2) return 0;
  return static_cast<size_t>(nranks) * static_cast<size_t>(ar::stepwise_ws_stride(static_cast<int64_t>(count))) * 4;
}

struct Range {
  uintptr_t lo, hi;
};

// Overlap among [p, p + bytes) ranges; sorted by start, any overlap shows up between neighbours.
bool any_overlap(Range* r, int m) {
  std::sort(r, r + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  for (int k = 1; k < m; ++k)
    if (r[k].lo < r[k - 1].hi) return true;
  return false;
}

int allreduce_impl(const char* entry, const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count,
                   int dtype, int op, int algo, void* workspace, size_t ws_bytes, void* stream,
                   bool library_scratch = false) {
  auto done = [&](int st) { return finish(entry, nranks, count, dtype, op, algo, st); };
  if (!valid_dtype(dtype) || !valid_op(op) || !valid_algo(algo)) return done(AR_ERR_INVALID);
  if (nranks < 1 || nranks > AR_MAX_RANKS) return done(AR_ERR_INVALID);
  if (algo == AR_ALGO_AUTO) algo = auto_algo(nranks, count, dtype);  // recorded as the algorithm that ran
  if (algo == AR_ALGO_RHD || algo == AR_ALGO_RHD_STEPWISE) {
    if (!is_pow2(nranks)) return done(AR_ERR_UNSUPPORTED);
  }
  if (algo == AR_ALGO_RING_FP8) {
    if ((dtype != AR_F32 && dtype != AR_BF16) || (op != AR_SUM && op != AR_AVG)) return done(AR_ERR_UNSUPPORTED);
  }
  if (count == 0) return done(AR_OK);
  if (!in_bufs || !out_bufs) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  if (count > (SIZE_MAX / 2) / es) return done(AR_ERR_INVALID);
  const size_t bytes = count * es;
  Range ranges[2 * AR_MAX_RANKS + 1];
  int m = 0;
  bool vec = true;
  for (int r = 0; r < nranks; ++r) {
    if (!in_bufs[r] || !out_bufs[r]) return done(AR_ERR_INVALID);
    const uintptr_t i = reinterpret_cast<uintptr_t>(in_bufs[r]), o = reinterpret_cast<uintptr_t>(out_bufs[r]);
    if (i > UINTPTR_MAX - bytes || o > UINTPTR_MAX - bytes) return done(AR_ERR_INVALID);
    ranges[m++] = Range{i, i + bytes};
    if (o != i) ranges[m++] = Range{o, o + bytes};
    if ((i | o) & 15u) vec = false;  // the round-per-launch and fp8 kernels take 16-byte slots from offset 0
  }
  const size_t need = workspace_bytes(nranks, count, dtype, algo);
  if (need > 0 && library_scratch) {
    if (need > AR_NOALLOC_WS_BYTES) return done(AR_ERR_WORKSPACE);
    if (ar::noalloc_scratch(&workspace) != hipSuccess) return done(AR_ERR_HIP);
    ws_bytes = AR_NOALLOC_WS_BYTES;
  }
  if (need > 0) {
    if (!workspace || ws_bytes < need) return done(AR_ERR_WORKSPACE);
    const uintptr_t w = reinterpret_cast<uintptr_t>(workspace);
    if (w & 255u) return done(AR_ERR_INVALID);
    ranges[m++] = Range{w, w + need};
  }
  if (any_overlap(ranges, m)) return done(AR_ERR_ALIAS);

  ar::RankPtrs p;
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < nranks; ++r) {
    p.in[r] = in_bufs[r];
    p.out[r] = out_bufs[r];
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n64 = static_cast<int64_t>(count);
  hipError_t e = hipSuccess;
  const int64_t head = ar::vector_head(p, nranks, n64, static_cast<int>(es));
  if (nranks == 1 && algo != AR_ALGO_RING_FP8) {
    e = ar::launch_collapsed(p, 1, n64, dtype, op, AR_ALGO_RING, head, s);
  } else {
    switch (algo) {
      case AR_ALGO_RING:
      case AR_ALGO_FUSED:
      case AR_ALGO_RHD:
      case AR_ALGO_TREE: e = ar::launch_collapsed(p, nranks, n64, dtype, op, algo, head, s); break;
      case AR_ALGO_RING_STEPWISE:
        e = ar::launch_ring_stepwise(p, nranks, n64, dtype, op, static_cast<float*>(workspace), vec, s);
        break;
      case AR_ALGO_RHD_STEPWISE:
        e = ar::launch_rhd_stepwise(p, nranks, n64, dtype, op, static_cast<float*>(workspace), vec, s);
        break;
      case AR_ALGO_TREE_STEPWISE:
        e = ar::launch_tree_stepwise(p, nranks, n64, dtype, op, static_cast<float*>(workspace), vec, s);
        break;
      case AR_ALGO_RING_FP8: e = ar::launch_fp8_ring(p, nranks, n64, dtype, op, vec, s); break;
      default: return done(AR_ERR_INVALID);
    }
  }
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

// Shared validation of reduce-scatter / all-gather: `full` are the N buffers of `count` elements, `part` the N
// chunk buffers; a chunk buffer placed at its own chunk inside its rank's full buffer is the in-place form.
int rsag_impl(const char* entry, const void* const* full, const void* const* part, int nranks, size_t count,
              int dtype, int op, bool is_rs, void* const* writable_full, void* const* writable_part, void* stream) {
  auto done = [&](int st) { return finish(entry, nranks, count, dtype, op, -1, st); };
  if (!valid_dtype(dtype) || (is_rs && !valid_op(op))) return done(AR_ERR_INVALID);
  if (nranks < 1 || nranks > AR_MAX_RANKS) return done(AR_ERR_INVALID);
  if (count == 0) return done(AR_OK);
  if (!full || !part) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  if (count > (SIZE_MAX / 2) / es) return done(AR_ERR_INVALID);
  const size_t bytes = count * es;
  const size_t q = count / nranks, rr = count % nranks;
  Range ranges[2 * AR_MAX_RANKS];
  int m = 0;
  for (int r = 0; r < nranks; ++r) {
    const size_t lo = r * q + (static_cast<size_t>(r) < rr ? r : rr), len = q + (static_cast<size_t>(r) < rr ? 1 : 0);
    const uintptr_t f = reinterpret_cast<uintptr_t>(full[r]), c = reinterpret_cast<uintptr_t>(part[r]);
    if (!f) return done(AR_ERR_INVALID);
    if (len > 0 && !c) return done(AR_ERR_INVALID);
    if (f > UINTPTR_MAX - bytes || (c && c > UINTPTR_MAX - len * es)) return done(AR_ERR_INVALID);
    ranges[m++] = Range{f, f + bytes};
    if (len > 0 && c != f + lo * es) ranges[m++] = Range{c, c + len * es};
  }
  if (any_overlap(ranges, m)) return done(AR_ERR_ALIAS);
  ar::RankPtrs p;
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < nranks; ++r) {
    p.in[r] = is_rs ? full[r] : part[r];
    p.out[r] = is_rs ? writable_part[r] : writable_full[r];
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = is_rs ? ar::launch_reduce_scatter(p, nranks, static_cast<int64_t>(count), dtype, op, s)
                       : ar::launch_all_gather(p, nranks, static_cast<int64_t>(count), static_cast<int>(es), s);
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

}  // namespace

extern "C" {

int ar_reduce_scatter(const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count, int dtype, int op,
                      void* stream) {
  return rsag_impl("ar_reduce_scatter", in_bufs, const_cast<const void* const*>(out_bufs), nranks, count, dtype, op,
                   true, nullptr, out_bufs, stream);
}

int ar_all_gather(const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count, int dtype,
                  void* stream) {
  return rsag_impl("ar_all_gather", const_cast<const void* const*>(out_bufs), in_bufs, nranks, count, dtype, AR_SUM,
                   false, out_bufs, nullptr, stream);
}

int ar_epilogue(const void* acc, void* out, size_t count, int dtype, int op, int nranks, void* stream) {
  auto done = [&](int st) { return finish("ar_epilogue", nranks, count, dtype, op, -1, st); };
  if (!valid_dtype(dtype) || !valid_op(op) || nranks < 1 || nranks > AR_MAX_RANKS) return done(AR_ERR_INVALID);
  if (count == 0) return done(AR_OK);
  if (!acc || !out || count > (SIZE_MAX / 2) / 4) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  const uintptr_t a = reinterpret_cast<uintptr_t>(acc), o = reinterpret_cast<uintptr_t>(out);
  if (a % 4 != 0 || o % es != 0) return done(AR_ERR_INVALID);
  if (a > UINTPTR_MAX - 4 * count || o > UINTPTR_MAX - es * count) return done(AR_ERR_INVALID);
  // in place only element for element (4-byte types); a 2-byte output over its own partials would overwrite
  // partials other threads have not read yet
  const bool in_place = a == o && es == 4;
  if (!in_place && a < o + es * count && o < a + 4 * count) return done(AR_ERR_ALIAS);
  const hipError_t e = ar::launch_epilogue(acc, out, static_cast<int64_t>(count), dtype, op, nranks,
                                           static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_version(void) { return AR_VERSION; }

int ar_chunk_bounds(int nranks, size_t count, int64_t* lo) {
  if (!lo || nranks < 1 || nranks > AR_MAX_RANKS || count > static_cast<size_t>(INT64_MAX)) return AR_ERR_INVALID;
  const int64_t c64 = static_cast<int64_t>(count), q = c64 / nranks, r = c64 % nranks;
  for (int c = 0; c <= nranks; ++c) lo[c] = c * q + (c < r ? c : r);
  return AR_OK;
}

const char* ar_status_string(int status) {
  switch (status) {
    case AR_OK: return "AR_OK: success";
    case AR_ERR_INVALID: return "AR_ERR_INVALID: invalid argument";
    case AR_ERR_UNSUPPORTED: return "AR_ERR_UNSUPPORTED: unsupported combination of algorithm, dtype, op or rank count";
    case AR_ERR_ALIAS: return "AR_ERR_ALIAS: rank buffers overlap (only exact in-place is allowed)";
    case AR_ERR_WORKSPACE: return "AR_ERR_WORKSPACE: workspace missing or too small";
    case AR_ERR_HIP: return "AR_ERR_HIP: HIP runtime error at launch";
    default: return "unknown ar_status";
  }
}

int ar_last_call(ar_call_record* rec) {
  if (!rec || !g_has_last) return AR_ERR_INVALID;
  *rec = g_last;
  return AR_OK;
}

int ar_auto_algo(int nranks, size_t count, int dtype) {
  if (!valid_dtype(dtype) || nranks < 1 || nranks > AR_MAX_RANKS) return -AR_ERR_INVALID;
  return auto_algo(nranks, count, dtype);
}

int ar_allreduce_workspace_size(int nranks, size_t count, int dtype, int op, int algo, size_t* bytes) {
  if (!bytes || !valid_dtype(dtype) || !valid_op(op) || !valid_algo(algo) || nranks < 1 || nranks > AR_MAX_RANKS)
    return AR_ERR_INVALID;
  *bytes = workspace_bytes(nranks, count, dtype, algo);
  return AR_OK;
}

int ar_allreduce(const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count, int dtype, int op,
                 int algo, void* stream) {
  return allreduce_impl("ar_allreduce", in_bufs, out_bufs, nranks, count, dtype, op, algo, nullptr, 0, stream);
}

int ar_allreduce_ws(const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count, int dtype, int op,
                    int algo, void* workspace, size_t ws_bytes, void* stream) {
  return allreduce_impl("ar_allreduce_ws", in_bufs, out_bufs, nranks, count, dtype, op, algo, workspace, ws_bytes,
                        stream);
}

int ar_allreduce_noalloc(const void* const* in_bufs, void* const* out_bufs, int nranks, size_t count, int dtype,
                         int op, int algo, void* stream) {
  return allreduce_impl("ar_allreduce_noalloc", in_bufs, out_bufs, nranks, count, dtype, op, algo, nullptr, 0, stream,
                        true);
}

int ar_bucket_plan(const int64_t* numels, int ntensors, int dtype, int nranks, size_t cap_bytes, int32_t* bucket_of,
                   int64_t* offset_of, int64_t* bucket_count, int* nbuckets) {
  auto done = [&](int st) { return finish("ar_bucket_plan", nranks, static_cast<size_t>(ntensors), dtype, -1, -1, st); };
  if (ntensors < 0 || !valid_dtype(dtype) || nranks < 1 || nranks > AR_MAX_RANKS || cap_bytes == 0 || !nbuckets)
    return done(AR_ERR_INVALID);
  if (ntensors > 0 && (!numels || !bucket_of || !offset_of || !bucket_count)) return done(AR_ERR_INVALID);
  const int64_t es = esize_of(dtype);
  const int64_t g = 16 / es;                 // elements per 16-byte group
  const int64_t unit = g * nranks;           // bucket length granularity: N chunks of whole groups
  // Bounds keep every product below INT64_MAX: numel * es <= INT64_MAX/4 and cap <= INT64_MAX/4.
  const int64_t cap = cap_bytes > static_cast<size_t>(INT64_MAX / 4) ? INT64_MAX / 4 : static_cast<int64_t>(cap_bytes);
  for (int t = 0; t < ntensors; ++t)
    if (numels[t] < 0 || numels[t] > (INT64_MAX / 4) / es) return done(AR_ERR_INVALID);
  int b = -1;
  int64_t fill = 0;
  for (int t = 0; t < ntensors; ++t) {
    const int64_t len = (numels[t] + g - 1) / g * g;
    const bool over = fill > 0 && (fill + len) * es > cap;
    if (b < 0 || over) {
      if (b >= 0) bucket_count[b] = (fill + unit - 1) / unit * unit;
      ++b;
      fill = 0;
    }
    bucket_of[t] = b;
    offset_of[t] = fill;
    fill += len;
  }
  if (b >= 0) bucket_count[b] = (fill + unit - 1) / unit * unit;
  *nbuckets = b + 1;
  return done(AR_OK);
}

int ar_allreduce_buckets(const void* const* flat_in, void* const* flat_out, int nranks, const int64_t* bucket_count,
                         int nbuckets, int dtype, int op, int algo, void* stream) {
  size_t total = 0;
  auto done = [&](int st) { return finish("ar_allreduce_buckets", nranks, total, dtype, op, algo, st); };
  if (!valid_dtype(dtype) || !valid_op(op) || !valid_algo(algo)) return done(AR_ERR_INVALID);
  if (nranks < 1 || nranks > AR_MAX_RANKS || nbuckets < 0) return done(AR_ERR_INVALID);
  if (algo != AR_ALGO_RING && algo != AR_ALGO_FUSED && algo != AR_ALGO_RHD && algo != AR_ALGO_TREE)
    return done(AR_ERR_UNSUPPORTED);
  if (algo == AR_ALGO_RHD && !is_pow2(nranks)) return done(AR_ERR_UNSUPPORTED);
  if (nbuckets == 0) return done(AR_OK);
  if (!bucket_count || !flat_in || !flat_out) return done(AR_ERR_INVALID);
  const int64_t es = esize_of(dtype);
  const int64_t unit = static_cast<int64_t>(nranks) * (16 / es);
  for (int b = 0; b < nbuckets; ++b) {
    const int64_t c = bucket_count[b];
    if (c < 0 || c % unit != 0 || c > (INT64_MAX / 4) / es) return done(AR_ERR_INVALID);
    if (static_cast<size_t>(c) > (SIZE_MAX / 4) / static_cast<size_t>(es) - total) return done(AR_ERR_INVALID);
    total += static_cast<size_t>(c);
  }
  if (total == 0) return done(AR_OK);
  const size_t bytes = total * static_cast<size_t>(es);
  Range ranges[2 * AR_MAX_RANKS];
  int m = 0;
  for (int r = 0; r < nranks; ++r) {
    if (!flat_in[r] || !flat_out[r]) return done(AR_ERR_INVALID);
    const uintptr_t i = reinterpret_cast<uintptr_t>(flat_in[r]), o = reinterpret_cast<uintptr_t>(flat_out[r]);
    if ((i | o) & 15u) return done(AR_ERR_INVALID);
    if (i > UINTPTR_MAX - bytes || o > UINTPTR_MAX - bytes) return done(AR_ERR_INVALID);
    ranges[m++] = Range{i, i + bytes};
    if (o != i) ranges[m++] = Range{o, o + bytes};
  }
  if (any_overlap(ranges, m)) return done(AR_ERR_ALIAS);
  ar::RankPtrs p;
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < nranks; ++r) {
    p.in[r] = flat_in[r];
    p.out[r] = flat_out[r];
  }
  const int a = nranks == 1 ? AR_ALGO_RING : algo;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // A bucket of at least kOwnLaunchBytes per rank runs as one all-reduce launch of its own (each launch's
  // workgroups start together at the bucket's front; on MI355X that measured 18% faster than dealing the same
  // buckets out in one segment launch); runs of smaller buckets share segment launches, where a launch per bucket
  // would cost more than its work.
  constexpr int64_t kOwnLaunchBytes = 16 << 20;
  auto at = [&](int64_t elem) {
    ar::RankPtrs q = p;
    for (int r = 0; r < nranks; ++r) {
      q.in[r] = static_cast<const char*>(p.in[r]) + elem * es;
      q.out[r] = static_cast<char*>(p.out[r]) + elem * es;
    }
    return q;
  };
  hipError_t e = hipSuccess;
  int64_t start = 0;
  for (int b = 0; b < nbuckets && e == hipSuccess;) {
    if (bucket_count[b] * es >= kOwnLaunchBytes) {
      const ar::RankPtrs q = at(start);
      e = ar::launch_collapsed(q, nranks, bucket_count[b], dtype, op, a,
                               ar::vector_head(q, nranks, bucket_count[b], static_cast<int>(es)), s);
      start += bucket_count[b++];
      continue;
    }
    int b1 = b;
    int64_t run = 0;
    while (b1 < nbuckets && bucket_count[b1] * es < kOwnLaunchBytes) run += bucket_count[b1++];
    if (run > 0) e = ar::launch_segments(at(start), nranks, bucket_count + b, b1 - b, dtype, op, a, s);
    start += run;
    b = b1;
  }
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_allreduce_tensors(const ar_tensor_desc* d_descs, const void* const* d_in, void* const* d_out, int ntensors,
                         int nranks, int dtype, int op, int algo, void* stream) {
  auto done = [&](int st) {
    return finish("ar_allreduce_tensors", nranks, static_cast<size_t>(ntensors < 0 ? 0 : ntensors), dtype, op, algo, st);
  };
  if (!valid_dtype(dtype) || !valid_op(op) || !valid_algo(algo)) return done(AR_ERR_INVALID);
  if (nranks < 1 || nranks > AR_MAX_RANKS || ntensors < 0) return done(AR_ERR_INVALID);
  if (algo != AR_ALGO_RING && algo != AR_ALGO_FUSED && algo != AR_ALGO_RHD && algo != AR_ALGO_TREE)
    return done(AR_ERR_UNSUPPORTED);
  if (algo == AR_ALGO_RHD && !is_pow2(nranks)) return done(AR_ERR_UNSUPPORTED);
  if (ntensors == 0) return done(AR_OK);
  if (!d_descs || !d_in || !d_out) return done(AR_ERR_INVALID);
  const int a = nranks == 1 ? AR_ALGO_RING : algo;
  hipError_t e = ar::launch_tensors(d_descs, d_in, d_out, ntensors, nranks, dtype, op, a,
                                    static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

static int batched_copy(const char* entry, const ar_copy_desc* d_descs, int ndescs, int dtype, void* stream) {
  auto done = [&](int st) { return finish(entry, 0, static_cast<size_t>(ndescs), dtype, -1, -1, st); };
  if (ndescs < 0 || !valid_dtype(dtype)) return done(AR_ERR_INVALID);
  if (ndescs == 0) return done(AR_OK);
  if (!d_descs) return done(AR_ERR_INVALID);
  hipError_t e = ar::launch_batched_copy(d_descs, ndescs, esize_of(dtype), static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_bucket_pack(const ar_copy_desc* d_descs, int ndescs, int dtype, void* stream) {
  return batched_copy("ar_bucket_pack", d_descs, ndescs, dtype, stream);
}

int ar_bucket_unpack(const ar_copy_desc* d_descs, int ndescs, int dtype, void* stream) {
  return batched_copy("ar_bucket_unpack", d_descs, ndescs, dtype, stream);
}

int ar_fp8_quant(const void* in, int in_dtype, size_t count, uint8_t* codes, float* scales, void* stream) {
  auto done = [&](int st) { return finish("ar_fp8_quant", 1, count, in_dtype, -1, -1, st); };
  if (in_dtype != AR_F32 && in_dtype != AR_BF16) return done(AR_ERR_INVALID);
  if (count == 0) return done(AR_OK);
  if (!in || !codes || !scales || count > static_cast<size_t>(INT64_MAX / 8)) return done(AR_ERR_INVALID);
  hipError_t e = ar::launch_fp8_quant(in, in_dtype, static_cast<int64_t>(count), codes, scales,
                                      static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_fp8_dequant(const uint8_t* codes, const float* scales, size_t count, void* out, int out_dtype, void* stream) {
  auto done = [&](int st) { return finish("ar_fp8_dequant", 1, count, out_dtype, -1, -1, st); };
  if (out_dtype != AR_F32 && out_dtype != AR_BF16) return done(AR_ERR_INVALID);
  if (count == 0) return done(AR_OK);
  if (!codes || !scales || !out || count > static_cast<size_t>(INT64_MAX / 8)) return done(AR_ERR_INVALID);
  hipError_t e = ar::launch_fp8_dequant(codes, scales, static_cast<int64_t>(count), out, out_dtype,
                                        static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------ block boundary
namespace {

// The address ranges of one call, collected and then checked together. A range given twice as the same in-place pair
// is added once by its caller.
struct Ranges {
  Range r[3 * AR_MAX_RANKS + 16];
  int m = 0;
  bool bad = false;  // a required pointer is NULL, misaligned, or its range wraps
  void add(const void* p, size_t bytes, size_t align, bool required = true) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!a) {
      bad = bad || required;
      return;
    }
    if (a % align != 0 || a > UINTPTR_MAX - bytes) bad = true;
    else if (bytes > 0) r[m++] = Range{a, a + bytes};
  }
};

bool mul(size_t a, size_t b, size_t* out) { return !__builtin_mul_overflow(a, b, out) && *out <= (size_t(1) << 62); }

size_t blocks_of(size_t hidden) { return (hidden + AR_FP8_BLOCK - 1) / AR_FP8_BLOCK; }

// What both norm entry points check of their common arguments; AR_OK goes on.
int norm_common(int nranks, size_t rows, size_t hidden, int dtype, int gamma_dtype, size_t* bytes) {
  if (!valid_dtype(dtype) || !valid_dtype(gamma_dtype) || nranks < 1 || nranks > AR_MAX_RANKS || hidden == 0)
    return AR_ERR_INVALID;
  if (gamma_dtype != dtype && gamma_dtype != AR_F32) return AR_ERR_INVALID;
  if (dtype == AR_I32 || hidden > AR_NORM_MAX_HIDDEN) return AR_ERR_UNSUPPORTED;
  size_t e;
  if (!mul(rows, hidden, &e) || !mul(e, static_cast<size_t>(esize_of(dtype)), bytes)) return AR_ERR_INVALID;
  return AR_OK;
}

bool rows_fit(size_t tokens, int k, int nexperts, int align, size_t* rows) {
  if (k < 1 || nexperts < 1 || nexperts > AR_MAX_EXPERTS || align < 1) return false;
  size_t slots;
  if (!mul(tokens, static_cast<size_t>(k), &slots) || slots > INT32_MAX) return false;
  const size_t used = slots < static_cast<size_t>(nexperts) ? slots : static_cast<size_t>(nexperts);
  *rows = slots + used * static_cast<size_t>(align - 1);
  return *rows <= INT32_MAX;
}

}  // namespace

extern "C" {

int ar_allreduce_rmsnorm(const void* const* in_bufs, int nranks, size_t rows, size_t hidden, int dtype,
                         const void* residual, const void* gamma, int gamma_dtype, float eps, void* const* out_bufs,
                         float* const* out_scales, void* residual_out, float* rstd, uint8_t* saved,
                         float* saved_scales, void* stream) {
  size_t bytes = 0;
  auto done = [&](int st) { return finish("ar_allreduce_rmsnorm", nranks, rows * hidden, dtype, AR_SUM, -1, st); };
  const int st = norm_common(nranks, rows, hidden, dtype, gamma_dtype, &bytes);
  if (st != AR_OK) return done(st);
  if (!(eps >= 0.0f) || !(eps <= 3.402823466e38f)) return done(AR_ERR_INVALID);
  if (rows == 0) return done(AR_OK);
  if (!in_bufs || !out_bufs || (saved == nullptr) != (saved_scales == nullptr)) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype)), codes = rows * hidden, scales = rows * blocks_of(hidden) * 4;
  Ranges g;
  ar::NormArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int r = 0; r < nranks; ++r) {
    g.add(in_bufs[r], bytes, es);
    if (out_scales) {
      g.add(out_bufs[r], codes, 1);
      g.add(out_scales[r], scales, 4);
      a.out_scales[r] = out_scales[r];
    } else if (out_bufs[r] != in_bufs[r]) {
      g.add(out_bufs[r], bytes, es);
    }
    a.in[r] = in_bufs[r];
    a.out[r] = out_bufs[r];
  }
  g.add(residual, bytes, es, false);
  if (residual_out != residual) g.add(residual_out, bytes, es, false);
  g.add(gamma, hidden * static_cast<size_t>(esize_of(gamma_dtype)), static_cast<size_t>(esize_of(gamma_dtype)));
  g.add(rstd, rows * 4, 4, false);
  g.add(saved, codes, 1, false);
  g.add(saved_scales, scales, 4, false);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  a.residual = residual;
  a.residual_out = residual_out;
  a.gamma = gamma;
  a.codes = saved;
  a.scales = saved_scales;
  a.rstd = rstd;
  a.rows = static_cast<int64_t>(rows);
  a.hidden = static_cast<int>(hidden);
  a.n = nranks;
  a.gamma_f32 = gamma_dtype == AR_F32;
  a.out8 = out_scales != nullptr;
  a.eps = eps;
  return done(ar::launch_rmsnorm(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_allreduce_rmsnorm_bwd_workspace_size(size_t rows, size_t hidden, size_t* bytes) {
  auto done = [&](int st) {
    return finish("ar_allreduce_rmsnorm_bwd_workspace_size", 0, rows * hidden, AR_F32, -1, -1, st);
  };
  if (!bytes || hidden == 0 || rows > static_cast<size_t>(INT64_MAX)) return done(AR_ERR_INVALID);
  if (hidden > AR_NORM_MAX_HIDDEN) return done(AR_ERR_UNSUPPORTED);
  *bytes = static_cast<size_t>(ar::rmsnorm_bwd_groups(static_cast<int64_t>(rows), static_cast<int64_t>(hidden), 1)) *
           hidden * 4;
  return done(AR_OK);
}

int ar_allreduce_rmsnorm_bwd(const void* const* in_bufs, int nranks, size_t rows, size_t hidden, int dtype,
                             const void* saved, const float* saved_scales, const void* gamma, int gamma_dtype,
                             const float* rstd, const void* residual_grad, void* const* out_bufs, float* dgamma,
                             void* workspace, size_t ws_bytes, void* stream) {
  size_t bytes = 0;
  auto done = [&](int st) { return finish("ar_allreduce_rmsnorm_bwd", nranks, rows * hidden, dtype, AR_SUM, -1, st); };
  const int st = norm_common(nranks, rows, hidden, dtype, gamma_dtype, &bytes);
  if (st != AR_OK) return done(st);
  if (!dgamma || (rows > 0 && (!in_bufs || !out_bufs))) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  const size_t need = static_cast<size_t>(ar::rmsnorm_bwd_groups(static_cast<int64_t>(rows),
                                                                 static_cast<int64_t>(hidden), 1)) * hidden * 4;
  Ranges g;
  ar::NormArgs a;
  std::memset(&a, 0, sizeof(a));
  g.add(dgamma, hidden * 4, 4);
  if (rows > 0) {
    bool in_place = false;
    for (int r = 0; r < nranks; ++r) {
      g.add(in_bufs[r], bytes, es);
      if (out_bufs[r] == residual_grad && residual_grad && !in_place) in_place = true;  // one of them at most
      else if (out_bufs[r] != in_bufs[r]) g.add(out_bufs[r], bytes, es);
      a.in[r] = in_bufs[r];
      a.out[r] = out_bufs[r];
    }
    if (saved_scales) {
      g.add(saved, rows * hidden, 1);
      g.add(saved_scales, rows * blocks_of(hidden) * 4, 4);
    } else {
      g.add(saved, bytes, es);
    }
    g.add(gamma, hidden * static_cast<size_t>(esize_of(gamma_dtype)), static_cast<size_t>(esize_of(gamma_dtype)));
    g.add(rstd, rows * 4, 4);
    g.add(residual_grad, bytes, es, false);
    if (g.bad) return done(AR_ERR_INVALID);
    if (!workspace || ws_bytes < need) return done(AR_ERR_WORKSPACE);
    g.add(workspace, need, 256);
  }
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  a.residual = residual_grad;
  a.gamma = gamma;
  a.saved = saved;
  a.saved_scales = saved_scales;
  a.rstd_in = rstd;
  a.partial = static_cast<float*>(workspace);
  a.rows = static_cast<int64_t>(rows);
  a.hidden = static_cast<int>(hidden);
  a.n = nranks;
  a.gamma_f32 = gamma_dtype == AR_F32;
  const hipError_t e = ar::launch_rmsnorm_bwd(a, dtype, dgamma, static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_rows(size_t tokens, int k, int nexperts, int align, size_t* rows) {
  auto done = [&](int st) { return finish("ar_expert_rows", 0, tokens, AR_I32, -1, -1, st); };
  size_t r = 0;
  if (!rows || !rows_fit(tokens, k, nexperts, align, &r)) return done(AR_ERR_INVALID);
  *rows = r;
  return done(AR_OK);
}

int ar_expert_sort_workspace_size(size_t tokens, int k, int nexperts, size_t* bytes) {
  auto done = [&](int st) { return finish("ar_expert_sort_workspace_size", 0, tokens, AR_I32, -1, -1, st); };
  size_t r = 0;
  if (!bytes || !rows_fit(tokens, k, nexperts, 1, &r)) return done(AR_ERR_INVALID);
  *bytes = static_cast<size_t>(ar::sort_workspace(static_cast<int64_t>(r), nexperts));
  return done(AR_OK);
}

int ar_expert_sort(const int32_t* ids, size_t tokens, int k, int nexperts, int align, int32_t* offsets,
                   int32_t* counts, int32_t* pos, int32_t* src, size_t rows, void* workspace, size_t ws_bytes,
                   void* stream) {
  auto done = [&](int st) { return finish("ar_expert_sort", 0, tokens, AR_I32, -1, -1, st); };
  size_t most = 0;
  if (!rows_fit(tokens, k, nexperts, align, &most) || rows < most || rows > INT32_MAX) return done(AR_ERR_INVALID);
  const size_t slots = tokens * static_cast<size_t>(k);
  const size_t need = static_cast<size_t>(ar::sort_workspace(static_cast<int64_t>(slots), nexperts));
  Ranges g;
  g.add(ids, slots * 4, 4, slots > 0);
  g.add(offsets, (static_cast<size_t>(nexperts) + 1) * 4, 4);
  g.add(counts, static_cast<size_t>(nexperts) * 4, 4);
  g.add(pos, slots * 4, 4, slots > 0);
  g.add(src, rows * 4, 4, rows > 0);
  if (g.bad) return done(AR_ERR_INVALID);
  if (need > 0) {
    if (!workspace || ws_bytes < need) return done(AR_ERR_WORKSPACE);
    g.add(workspace, need, 256);
    if (g.bad) return done(AR_ERR_INVALID);
  }
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  const ar::SortArgs a{ids, offsets, counts, pos, src, static_cast<int32_t*>(workspace), static_cast<int64_t>(slots),
                       static_cast<int64_t>(rows), nexperts, align};
  return done(ar::launch_expert_sort(a, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_dispatch(const void* x, const float* x_scales, const int32_t* pos, const int32_t* offsets,
                       const int32_t* counts, size_t tokens, int k, int nexperts, size_t hidden, int elem_size,
                       void* xs, float* xs_scales, size_t rows, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_dispatch", 0, tokens, elem_size, -1, -1, st); };
  size_t most = 0, xe = 0, xb = 0, ye = 0, yb = 0;
  if (!rows_fit(tokens, k, nexperts, 1, &most) || hidden == 0 || rows > INT32_MAX) return done(AR_ERR_INVALID);
  if (elem_size != 1 && elem_size != 2 && elem_size != 4) return done(AR_ERR_INVALID);
  // without tokens, or without rows, one of the two is empty and has no address
  if (tokens > 0 && rows > 0 && (x_scales == nullptr) != (xs_scales == nullptr)) return done(AR_ERR_INVALID);
  if ((x_scales || xs_scales) && elem_size != 1) return done(AR_ERR_INVALID);
  if ((offsets == nullptr) != (counts == nullptr)) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(elem_size), nb = blocks_of(hidden) * 4;
  if (!mul(tokens, hidden, &xe) || !mul(xe, es, &xb) || !mul(rows, hidden, &ye) || !mul(ye, es, &yb))
    return done(AR_ERR_INVALID);
  if (hidden > INT32_MAX / es) return done(AR_ERR_UNSUPPORTED);
  if (tokens == 0) return done(AR_OK);
  Ranges g;
  g.add(x, xb, es);
  g.add(x_scales, tokens * nb, 4, false);
  g.add(pos, tokens * static_cast<size_t>(k) * 4, 4);
  g.add(offsets, (static_cast<size_t>(nexperts) + 1) * 4, 4, false);
  g.add(counts, static_cast<size_t>(nexperts) * 4, 4, false);
  g.add(xs, yb, es, rows > 0);
  g.add(xs_scales, rows * nb, 4, false);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::MoveArgs a{};
  a.x = x;
  a.y = xs;
  a.x_scales = x_scales;
  a.y_scales = xs_scales;
  a.pos = pos;
  a.offsets = offsets;
  a.counts = counts;
  a.tokens = static_cast<int64_t>(tokens);
  a.rows = static_cast<int64_t>(rows);
  a.hidden = static_cast<int>(hidden);
  a.k = k;
  a.experts = nexperts;
  const hipError_t e = ar::launch_expert_dispatch(a, elem_size, static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_combine(const void* ys, const int32_t* pos, const float* weights, const void* addend, size_t tokens,
                      int k, size_t hidden, int dtype, size_t rows, void* out, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_combine", 0, tokens, dtype, AR_SUM, -1, st); };
  size_t most = 0, oe = 0, ob = 0, ye = 0, yb = 0;
  if (!valid_dtype(dtype) || !rows_fit(tokens, k, 1, 1, &most) || hidden == 0 || rows > INT32_MAX)
    return done(AR_ERR_INVALID);
  if (dtype == AR_I32) return done(AR_ERR_UNSUPPORTED);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  if (!mul(tokens, hidden, &oe) || !mul(oe, es, &ob) || !mul(rows, hidden, &ye) || !mul(ye, es, &yb))
    return done(AR_ERR_INVALID);
  if (hidden > INT32_MAX / es) return done(AR_ERR_UNSUPPORTED);
  if (tokens == 0) return done(AR_OK);
  Ranges g;
  g.add(ys, yb, es, rows > 0);
  g.add(pos, tokens * static_cast<size_t>(k) * 4, 4);
  g.add(weights, tokens * static_cast<size_t>(k) * 4, 4, false);
  g.add(addend, ob, es, false);
  if (!out) return done(AR_ERR_INVALID);
  if (out != addend) g.add(out, ob, es);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::MoveArgs a{};
  a.x = ys;
  a.y = out;
  a.pos = pos;
  a.weights = weights;
  a.extra = addend;
  a.tokens = static_cast<int64_t>(tokens);
  a.rows = static_cast<int64_t>(rows);
  a.hidden = static_cast<int>(hidden);
  a.k = k;
  const hipError_t e = ar::launch_expert_combine(a, dtype, static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_combine_bwd(const void* dout, const void* ys, const int32_t* pos, const float* weights,
                          const int32_t* offsets, const int32_t* counts, size_t tokens, int k, int nexperts,
                          size_t hidden, int dtype, size_t rows, void* dys, float* dweights, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_combine_bwd", 0, tokens, dtype, AR_SUM, -1, st); };
  size_t most = 0, oe = 0, ob = 0, ye = 0, yb = 0;
  if (!valid_dtype(dtype) || !rows_fit(tokens, k, nexperts, 1, &most) || hidden == 0 || rows > INT32_MAX)
    return done(AR_ERR_INVALID);
  if (dtype == AR_I32) return done(AR_ERR_UNSUPPORTED);
  if ((offsets == nullptr) != (counts == nullptr)) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  if (!mul(tokens, hidden, &oe) || !mul(oe, es, &ob) || !mul(rows, hidden, &ye) || !mul(ye, es, &yb))
    return done(AR_ERR_INVALID);
  if (hidden > INT32_MAX / es) return done(AR_ERR_UNSUPPORTED);
  if (tokens == 0) return done(AR_OK);
  Ranges g;
  g.add(dout, ob, es);
  g.add(ys, yb, es, rows > 0);
  g.add(pos, tokens * static_cast<size_t>(k) * 4, 4);
  g.add(weights, tokens * static_cast<size_t>(k) * 4, 4);
  g.add(offsets, (static_cast<size_t>(nexperts) + 1) * 4, 4, false);
  g.add(counts, static_cast<size_t>(nexperts) * 4, 4, false);
  if (dys != ys) g.add(dys, yb, es, rows > 0);
  g.add(dweights, tokens * static_cast<size_t>(k) * 4, 4);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::MoveArgs a{};
  a.x = ys;
  a.y = dys;
  a.pos = pos;
  a.weights = weights;
  a.extra = dout;
  a.dweights = dweights;
  a.offsets = offsets;
  a.counts = counts;
  a.tokens = static_cast<int64_t>(tokens);
  a.rows = static_cast<int64_t>(rows);
  a.hidden = static_cast<int>(hidden);
  a.k = k;
  a.experts = nexperts;
  const hipError_t e = ar::launch_expert_combine_bwd(a, dtype, static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------ experts' products
namespace {

// The sizes of one call of the products: what all of them check of their common arguments. AR_OK goes on.
struct ProductSizes {
  size_t in_bytes, out_bytes;  // the buffers of rows of `in` and of `out` elements
  size_t matrix;               // elements of a matrix
};
int product_common(size_t rows, size_t in, size_t out, int dtype, const int32_t* offsets, const int32_t* counts,
                   int nexperts, ProductSizes* z) {
  if (!valid_dtype(dtype) || in == 0 || out == 0 || rows > INT32_MAX) return AR_ERR_INVALID;
  if (nexperts < 1 || nexperts > AR_MAX_EXPERTS || (!offsets && (counts || nexperts != 1))) return AR_ERR_INVALID;
  if (dtype == AR_I32 || in > AR_PRODUCT_MAX_WIDTH || out > AR_PRODUCT_MAX_WIDTH) return AR_ERR_UNSUPPORTED;
  const size_t es = static_cast<size_t>(esize_of(dtype));
  z->in_bytes = rows * in * es;  // below 2^53
  z->out_bytes = rows * out * es;
  z->matrix = in * out;
  return AR_OK;
}

// Adds one matrix per expert, `stride` elements apart (none but the size of a matrix matters for a single expert), and a
// second set of the same layout (or NULL) that may lie in the gaps of the first, as the halves of one tensor do. Where both
// are NULL there is nothing to check: a caller who leaves a weight out has no stride for it.
bool add_matrices(Ranges& g, const void* p0, const void* p1, size_t matrix, size_t stride, int nexperts, size_t es) {
  if (!p0 && !p1) return true;
  size_t span = 0;
  if (nexperts == 1) stride = matrix;
  if (stride < matrix || !mul(stride, static_cast<size_t>(nexperts - 1), &span) || !mul(span + matrix, es, &span))
    return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p0), b = reinterpret_cast<uintptr_t>(p1);
  const uintptr_t lo = a < b ? a : b, d = a < b ? b - a : a - b;
  if (p0 && p1 && d < span && nexperts > 1 && a % es == 0 && b % es == 0) {
    const size_t off = d % (stride * es), size = matrix * es;
    if (off >= size && stride * es - off >= size) {
      g.add(reinterpret_cast<const void*>(lo), d + span, es);
      return true;
    }
  }
  g.add(p0, span, es, false);
  g.add(p1, span, es, false);
  return true;
}

bool too_many_tiles(const ar::ProductArgs& a, int64_t in, int64_t out) {
  const int64_t wide = in > out ? in : out;
  return ar::row_tiles(a, 1, 16) * ar::tiles_up(wide, 16) > ar::kMostTiles ||
         2 * static_cast<int64_t>(a.experts) * ar::tiles_up(in, 64) * ar::tiles_up(out, 64) > ar::kMostTiles;
}

void add_segments(Ranges& g, const int32_t* offsets, const int32_t* counts, int nexperts) {
  g.add(offsets, (static_cast<size_t>(nexperts) + 1) * 4, 4, false);
  g.add(counts, static_cast<size_t>(nexperts) * 4, 4, false);
}

ar::ProductArgs product_args(size_t rows, const int32_t* offsets, const int32_t* counts, int nexperts) {
  ar::ProductArgs a{};
  a.offsets = offsets;
  a.counts = counts;
  a.rows = static_cast<int>(rows);
  a.experts = nexperts;
  return a;
}

bool valid_act(int act) { return act >= AR_ACT_SILU && act <= AR_ACT_GELU_TANH; }

}  // namespace

extern "C" {

int ar_expert_gated(const void* xs, const void* w_gate, const void* w_up, size_t w_stride, const int32_t* offsets,
                    const int32_t* counts, int nexperts, size_t rows, size_t hidden, size_t inner, int dtype, int act,
                    void* out, void* gate, void* up, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_gated", 0, rows, dtype, -1, -1, st); };
  ProductSizes z;
  const int st = product_common(rows, hidden, inner, dtype, offsets, counts, nexperts, &z);
  if (st != AR_OK) return done(st);
  if (!valid_act(act) || (gate == nullptr) != (up == nullptr)) return done(AR_ERR_INVALID);
  if (rows == 0) return done(AR_OK);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  Ranges g;
  g.add(xs, z.in_bytes, es);
  if (!w_gate || !w_up || !add_matrices(g, w_gate, w_up, z.matrix, w_stride, nexperts, es)) return done(AR_ERR_INVALID);
  add_segments(g, offsets, counts, nexperts);
  g.add(out, z.out_bytes, es);
  g.add(gate, z.out_bytes, es, false);
  g.add(up, z.out_bytes, es, false);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::ProductArgs a = product_args(rows, offsets, counts, nexperts);
  a.a0 = xs;
  a.b0 = w_gate;
  a.b1 = w_up;
  a.c0 = out;
  a.c1 = gate;
  a.c2 = up;
  a.w_stride = static_cast<int64_t>(w_stride);
  a.n = static_cast<int>(inner);
  a.k = static_cast<int>(hidden);
  a.act = act;
  if (too_many_tiles(a, a.k, a.n)) return done(AR_ERR_UNSUPPORTED);
  return done(ar::launch_gated(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_gated_bwd(const void* dout, const void* gate, const void* up, const void* xs, const void* w_gate,
                        const void* w_up, size_t w_stride, const int32_t* offsets, const int32_t* counts, int nexperts,
                        size_t rows, size_t hidden, size_t inner, int dtype, int act, void* dgate, void* dup, void* dxs,
                        void* dw_gate, void* dw_up, size_t dw_stride, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_gated_bwd", 0, rows, dtype, -1, -1, st); };
  ProductSizes z;
  const int st = product_common(rows, hidden, inner, dtype, offsets, counts, nexperts, &z);
  if (st != AR_OK) return done(st);
  if (!valid_act(act) || (dw_gate == nullptr) != (dw_up == nullptr)) return done(AR_ERR_INVALID);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  const bool some = rows > 0;
  Ranges g;
  g.add(dout, z.out_bytes, es, some);
  g.add(gate, z.out_bytes, es, some);
  g.add(up, z.out_bytes, es, some);
  auto in_place = [&](const void* p) { return p == dout || p == gate || p == up; };
  if (some && (!dgate || !dup)) return done(AR_ERR_INVALID);
  if (!in_place(dgate)) g.add(dgate, z.out_bytes, es, some);
  if (!in_place(dup)) g.add(dup, z.out_bytes, es, some);
  // the rows' gradient needs the weights, and the weights' the rows
  g.add(xs, z.in_bytes, es, some && dw_gate);
  if (some && dxs && (!w_gate || !w_up)) return done(AR_ERR_INVALID);
  if (!add_matrices(g, w_gate, w_up, z.matrix, w_stride, nexperts, es) ||
      !add_matrices(g, dw_gate, dw_up, z.matrix, dw_stride, nexperts, es))
    return done(AR_ERR_INVALID);
  add_segments(g, offsets, counts, nexperts);
  g.add(dxs, z.in_bytes, es, false);
  if (g.bad) return done(AR_ERR_INVALID);
  if ((some && dgate == dup) || any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::ProductArgs a = product_args(rows, offsets, counts, nexperts);
  a.act = act;
  const int in = static_cast<int>(hidden), wide = static_cast<int>(inner);
  if (too_many_tiles(a, in, wide)) return done(AR_ERR_UNSUPPORTED);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (some) {
    ar::ProductArgs b = a;
    b.a0 = dout;
    b.b0 = gate;
    b.b1 = up;
    b.c0 = dgate;
    b.c1 = dup;
    b.n = wide;
    e = ar::launch_slopes(b, dtype, s);
  }
  if (e == hipSuccess && some && dxs) {
    ar::ProductArgs b = a;
    b.a0 = dgate;
    b.a1 = dup;
    b.b0 = w_gate;
    b.b1 = w_up;
    b.w_stride = static_cast<int64_t>(w_stride);
    b.c0 = dxs;
    b.n = in;
    b.k = wide;
    e = ar::launch_input_grad(b, dtype, s);
  }
  if (e == hipSuccess && dw_gate) {
    ar::ProductArgs b = a;
    b.a0 = dgate;
    b.a1 = dup;
    b.b0 = xs;
    b.c0 = dw_gate;
    b.c1 = dw_up;
    b.c_stride = static_cast<int64_t>(dw_stride);
    b.m = wide;
    b.n = in;
    if (b.a1 == nullptr) b.a1 = dw_up;  // without rows nothing is read, and both gradients are still set to zero
    e = ar::launch_weight_grad(b, dtype, s);
  }
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_linear(const void* xs, const void* w, size_t w_stride, const int32_t* offsets, const int32_t* counts,
                     int nexperts, size_t rows, size_t in, size_t out, int dtype, void* ys, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_linear", 0, rows, dtype, -1, -1, st); };
  ProductSizes z;
  const int st = product_common(rows, in, out, dtype, offsets, counts, nexperts, &z);
  if (st != AR_OK) return done(st);
  if (rows == 0) return done(AR_OK);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  Ranges g;
  g.add(xs, z.in_bytes, es);
  if (!w || !add_matrices(g, w, nullptr, z.matrix, w_stride, nexperts, es)) return done(AR_ERR_INVALID);
  add_segments(g, offsets, counts, nexperts);
  g.add(ys, z.out_bytes, es);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::ProductArgs a = product_args(rows, offsets, counts, nexperts);
  a.a0 = xs;
  a.b0 = w;
  a.c0 = ys;
  a.w_stride = static_cast<int64_t>(w_stride);
  a.n = static_cast<int>(out);
  a.k = static_cast<int>(in);
  if (too_many_tiles(a, a.k, a.n)) return done(AR_ERR_UNSUPPORTED);
  return done(ar::launch_linear(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? AR_OK : AR_ERR_HIP);
}

int ar_expert_linear_bwd(const void* dys, const void* xs, const void* w, size_t w_stride, const int32_t* offsets,
                         const int32_t* counts, int nexperts, size_t rows, size_t in, size_t out, int dtype, void* dxs,
                         void* dw, size_t dw_stride, void* stream) {
  auto done = [&](int st) { return finish("ar_expert_linear_bwd", 0, rows, dtype, -1, -1, st); };
  ProductSizes z;
  const int st = product_common(rows, in, out, dtype, offsets, counts, nexperts, &z);
  if (st != AR_OK) return done(st);
  const size_t es = static_cast<size_t>(esize_of(dtype));
  const bool some = rows > 0;
  Ranges g;
  g.add(dys, z.out_bytes, es, some);
  g.add(xs, z.in_bytes, es, some && dw);
  if (some && dxs && !w) return done(AR_ERR_INVALID);
  if (!add_matrices(g, w, nullptr, z.matrix, w_stride, nexperts, es) ||
      !add_matrices(g, dw, nullptr, z.matrix, dw_stride, nexperts, es))
    return done(AR_ERR_INVALID);
  add_segments(g, offsets, counts, nexperts);
  g.add(dxs, z.in_bytes, es, false);
  if (g.bad) return done(AR_ERR_INVALID);
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  ar::ProductArgs a = product_args(rows, offsets, counts, nexperts);
  if (too_many_tiles(a, static_cast<int64_t>(in), static_cast<int64_t>(out))) return done(AR_ERR_UNSUPPORTED);
  a.a0 = dys;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (some && dxs) {
    ar::ProductArgs b = a;
    b.b0 = w;
    b.w_stride = static_cast<int64_t>(w_stride);
    b.c0 = dxs;
    b.n = static_cast<int>(in);
    b.k = static_cast<int>(out);
    e = ar::launch_input_grad(b, dtype, s);
  }
  if (e == hipSuccess && dw) {
    a.b0 = xs;
    a.c0 = dw;
    a.c_stride = static_cast<int64_t>(dw_stride);
    a.m = static_cast<int>(out);
    a.n = static_cast<int>(in);
    e = ar::launch_weight_grad(a, dtype, s);
  }
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------ gradients' norm
namespace {

bool float_dtype(int dtype) { return dtype == AR_F32 || dtype == AR_BF16 || dtype == AR_F16; }

int grad_norm_impl(const char* entry, const ar_grad_piece* d_pieces, size_t npieces, int kind, bool clip, float max_norm,
                   float eps, float* norm, void* workspace, size_t ws_bytes, void* stream) {
  auto done = [&](int st) { return finish(entry, 0, npieces, AR_F32, -1, -1, st); };
  if ((kind != AR_NORM_L2 && kind != AR_NORM_MAX) || npieces > INT32_MAX) return done(AR_ERR_INVALID);
  if (clip && (!(max_norm >= 0.0f) || !(eps >= 0.0f) || !(eps <= 3.402823466e38f))) return done(AR_ERR_INVALID);
  const size_t need = static_cast<size_t>(ar::grad_groups(static_cast<int64_t>(npieces))) * sizeof(double);
  Ranges g;
  g.add(d_pieces, npieces * sizeof(ar_grad_piece), 8, npieces > 0);
  g.add(norm, 4, 4);
  if (g.bad) return done(AR_ERR_INVALID);
  if (need > 0) {
    if (!workspace || ws_bytes < need) return done(AR_ERR_WORKSPACE);
    g.add(workspace, need, 256);
    if (g.bad) return done(AR_ERR_INVALID);
  }
  if (any_overlap(g.r, g.m)) return done(AR_ERR_ALIAS);
  const ar::GradArgs a{d_pieces, static_cast<int64_t>(npieces), static_cast<double*>(workspace), norm, max_norm, eps, 0};
  const hipError_t e = ar::launch_grad_norm(a, kind == AR_NORM_MAX, clip, static_cast<hipStream_t>(stream));
  return done(e == hipSuccess ? AR_OK : AR_ERR_HIP);
}

// The tensors' ranges, and whether any two of them overlap. `room` holds two for each tensor.
int check_tensors(const ar_grad_piece* t, int n, Range* room, int64_t* total) {
  int m = 0;
  *total = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel < 0 || !valid_dtype(t[i].dtype)) return AR_ERR_INVALID;
    if (!float_dtype(t[i].dtype)) return AR_ERR_UNSUPPORTED;
    if (t[i].numel == 0) continue;
    const size_t es = static_cast<size_t>(esize_of(t[i].dtype));
    const uintptr_t in = reinterpret_cast<uintptr_t>(t[i].in), out = reinterpret_cast<uintptr_t>(t[i].out);
    if (t[i].numel > (int64_t(1) << 60)) return AR_ERR_INVALID;
    const size_t bytes = static_cast<size_t>(t[i].numel) * es;
    if (!in || in % es || out % es || in > UINTPTR_MAX - bytes || out > UINTPTR_MAX - bytes) return AR_ERR_INVALID;
    room[m++] = Range{in, in + bytes};
    if (out && out != in) room[m++] = Range{out, out + bytes};
    *total += static_cast<int64_t>(bytes);
    if (*total > (int64_t(1) << 62)) return AR_ERR_INVALID;
  }
  return any_overlap(room, m) ? AR_ERR_ALIAS : AR_OK;
}

}  // namespace

extern "C" {

int ar_grad_plan(const ar_grad_piece* tensors, int ntensors, ar_grad_piece* pieces, size_t* npieces) {
  auto done = [&](int st) {
    return finish("ar_grad_plan", 0, static_cast<size_t>(ntensors < 0 ? 0 : ntensors), AR_F32, -1, -1, st);
  };
  if (!npieces || ntensors < 0 || (ntensors > 0 && !tensors)) return done(AR_ERR_INVALID);
  const size_t room = pieces ? *npieces : 0;
  *npieces = 0;
  if (ntensors == 0) return done(AR_OK);
  Range* ranges = static_cast<Range*>(std::malloc(2 * sizeof(Range) * static_cast<size_t>(ntensors)));
  if (!ranges) return done(AR_ERR_INVALID);
  int64_t total = 0;
  const int st = check_tensors(tensors, ntensors, ranges, &total);
  std::free(ranges);
  if (st != AR_OK) return done(st);
  const uint64_t piece = static_cast<uint64_t>(ar::piece_bytes(total));
  size_t n = 0;
  for (int i = 0; i < ntensors; ++i) {
    const uint64_t es = static_cast<uint64_t>(esize_of(tensors[i].dtype));
    const uint64_t bytes = static_cast<uint64_t>(tensors[i].numel) * es;
    const uintptr_t in = reinterpret_cast<uintptr_t>(tensors[i].in), out = reinterpret_cast<uintptr_t>(tensors[i].out);
    // cuts at multiples of the piece's size from the 256 bytes that the tensor starts in
    uint64_t next = piece - in % 256;
    for (uint64_t at = 0; at < bytes; at = next, next += piece, ++n) {
      if (!pieces) {  // the rest of the count at once
        n += next >= bytes ? 1 : 1 + (bytes - next + piece - 1) / piece;
        break;
      }
      if (n >= room) return done(AR_ERR_INVALID);
      const uint64_t end = next < bytes ? next : bytes;
      pieces[n] = ar_grad_piece{reinterpret_cast<const void*>(in + at), out ? reinterpret_cast<void*>(out + at) : nullptr,
                                static_cast<int64_t>((end - at) / es), tensors[i].dtype, 0};
    }
  }
  *npieces = n;
  return done(AR_OK);
}

int ar_grad_norm_workspace_size(size_t npieces, size_t* bytes) {
  auto done = [&](int st) { return finish("ar_grad_norm_workspace_size", 0, npieces, AR_F32, -1, -1, st); };
  if (!bytes || npieces > INT32_MAX) return done(AR_ERR_INVALID);
  *bytes = static_cast<size_t>(ar::grad_groups(static_cast<int64_t>(npieces))) * sizeof(double);
  return done(AR_OK);
}

int ar_grad_norm(const ar_grad_piece* d_pieces, size_t npieces, int kind, float* norm, void* workspace, size_t ws_bytes,
                 void* stream) {
  return grad_norm_impl("ar_grad_norm", d_pieces, npieces, kind, false, 0.0f, 0.0f, norm, workspace, ws_bytes, stream);
}

int ar_grad_clip(const ar_grad_piece* d_pieces, size_t npieces, int kind, float max_norm, float eps, float* norm,
                 void* workspace, size_t ws_bytes, void* stream) {
  return grad_norm_impl("ar_grad_clip", d_pieces, npieces, kind, true, max_norm, eps, norm, workspace, ws_bytes, stream);
}

}  // extern "C"
