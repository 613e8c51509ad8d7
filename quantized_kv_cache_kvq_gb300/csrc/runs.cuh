// runs.cuh -- what kvq_map_runs, kvq_append_runs and kvq_attn_runs share: a *run* is the new tokens one request
// brings to a step, rows run_starts[s] .. run_starts[s + 1] - 1 of the step's tensors (one row per request
// when there is no run_starts), the last of them at position seq_lens[s] - 1 of its request.
#pragma once

#include "kvq_common.cuh"

namespace kvq {
namespace runs {

constexpr int kMaxBatch = KVQ_MAX_BATCH;
constexpr int kMaxContext = KVQ_MAX_CONTEXT;  // positions and their sums with a tile stay below 2^31
// Exponents of the page scales 2^e: the powers of two that fp16 holds (2^-24 is its smallest subnormal).
constexpr int kMinExp = -24, kMaxExp = 15;

// Row r0, length n and context length of request s; n = 0 and r0 = -1 for a run that cannot be (the caller reports it).
struct Run {
  int row0, n, len;
};
__device__ __forceinline__ Run load_run(const int32_t* run_starts, const int32_t* seq_lens, int s, int num_rows, int max_run,
                                        int max_pages) {
  const int a = run_starts ? run_starts[s] : s, b = run_starts ? run_starts[s + 1] : s + 1;
  const int len = seq_lens[s];
  if (a < 0 || b < a || b > num_rows || b - a > max_run || len < 0 || len > kMaxContext ||
      len > static_cast<long long>(max_pages) * kPage)
    return Run{-1, 0, 0};
  return Run{a, b - a, len};
}

// Page nth of those that a run of positions first .. len - 1 touches: the run's first position, the page's, its new tokens [from, to),
// its index.  Nothing (to = from) for one that the run does not have, whatever the numbers: where runs overlap, against the
// rules, the sums over them may wrap, and a page may be looked up in a run that has none.
struct RunPage {
  int first, p0, from, to, page;
};
__host__ __device__ __forceinline__ RunPage page_of_run(int first, int len, int nth) {
  const int page = first / kPage + nth;
  if (nth < 0 || first < 0 || len <= 0 || nth > (len - 1) / kPage - first / kPage) return RunPage{0, 0, 0, 0, 0};
  const int p0 = page * kPage;
  return RunPage{first, p0, first > p0 ? first - p0 : 0, len - p0 < kPage ? len - p0 : kPage, page};
}

// 2^e as fp16 bits, kMinExp <= e <= kMaxExp: subnormal below 2^-14.
__device__ __forceinline__ uint16_t exp_to_f16(int e) {
  return static_cast<uint16_t>(e >= -14 ? (e + 15) << 10 : 1 << (e + 24));
}
// 2^e as binary32, for normal exponents.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The exponent of a stored page scale (fp16 bits of a power of two; anything else, a page that was never written
// included, is read as the smallest exponent >= log2 of it that is in range, so that no caller meets an odd scale).
__device__ __forceinline__ int f16_to_exp(uint16_t b) {
  const uint32_t u = b & 0x7FFFu;
  if (u >= 0x400u) {
    const int e = static_cast<int>(u >> 10) - 15 + ((u & 0x3FFu) != 0);
    return e > kMaxExp ? kMaxExp : e;
  }
  return u <= 1 ? kMinExp : 32 - __clz(u - 1) - 24;
}

// Host checks of a page-scaled cache descriptor (append_runs.cu).
kvq_status check_page_scaled_cache(const kvq_cache* c);

}  // namespace runs
}  // namespace kvq
