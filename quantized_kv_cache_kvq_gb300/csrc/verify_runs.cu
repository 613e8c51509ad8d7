// verify_runs.cu -- kvq_verify_runs: which path of a tree of drafted tokens the target's probabilities accept, from given random numbers.
//
// Recursive rejection at a row with probabilities p and draft probabilities q: child x is accepted with probability
// min(1, p_k(x) / q(x)), p_0 = p / sum p, and a refusal goes on with p_{k+1} = max(p_k - q, 0) / sum of it.  All of these are one family:
//     p_k = max(p - c_k q, 0) / Z_k,   Z_k = sum max(p - c_k q, 0),   c_0 = 0,  c_{k+1} = c_k + Z_k
// (p_k - q = (max(p - c_k q, 0) - Z_k q) / Z_k, positive where p > (c_k + Z_k) q), so a refusal costs one sum over the vocabulary and no
// vector is kept.  Without draft probabilities the token is drawn from p and followed to the child that holds it; greedy, it is the largest score's.
//
// Sums are whole numbers, floor(2^44 w) in 64 bits: they do not depend on the order, the split or the batch, and the cumulative
// distribution that a token is drawn from is exact (with binary32 sums of a flat distribution of 10^5 tokens, a random number in a
// hundred would find another token).
//
// A cluster of eight blocks has a request and walks its tree: only the rows of the path are read.  A row is cut into one piece for each warp;
// after every pass the warps send their sums to all blocks, whose mbarriers count the bytes, and all blocks take the same decision.  What decides is
// read by the first block alone and handed to the others (the tree at the start, a child's numbers beside the sums), so that blocks take
// the same number of exchanges whatever another stream does to the inputs.
// Bound by the latency of the passes, which follow each other, each with its loads, an exchange and a decision: 32 trees of 25..64 over 131072
// tokens, fp32, 48 us in a graph (62 with the L2 flushed; 14 for the paths' rows at the copy rate), the slowest tree's time, so 49 to 60 with other
// draws; 16 greedy ones of 9..16 rows over 32000, bf16, 14 to 19 us.  A cluster barrier for each exchange took 54, sums by shifted significands and
// two loads in flight 87.  Greedy trees read whole, all rows before one exchange: 26 us for 16 trees of 12 rows over 32000, bf16, that take 16.5
// row by row.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "decode_kernel.cuh"
#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
// Warps of a block.  64 registers a thread: two blocks on an SM, so that 38 requests run at once.  That costs spills (88 bytes with fp32, 164 with
// BF16).  With 102 registers, no spills and one block on an SM the 32 trees above take 64 us, not 48, 64 greedy ones 39, not 29; up to 16 trees take
// the same to 1 or 2 us either way.
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kPieces = kCluster * kWarps;
constexpr int kMaxVocab = 1 << 19;  // sums of 2^19 times 2^44 fit 64 bits
constexpr uint32_t kAll = 0xffffffffu;

struct VerifyArgs {
  const void* target;
  const void* draft;
  long long target_stride, draft_stride;
  int vocab;
  const int32_t* tokens;
  const int32_t* parents;
  const float* uniform;
  const int32_t* run_starts;
  int batch, num_rows;
  int32_t* keep;
  int32_t* kept;
  int32_t* next;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  int32_t* err;
};

// What the first block reads for the decision after a pass.
struct Ask {
  float u, p, q;  // of the child that is tried next
  float draw;     // the row's own random number
};
struct Shared {
  int32_t parent[KVQ_MAX_TREE], token[KVQ_MAX_TREE];
  // Sums of a pass, its largest keys, or the token drawn + 1, of all warps: two in turn, and two for the passes over p itself, of rows in turn.
  unsigned long long part[4][kPieces];
  unsigned long long ask[2][2];  // an Ask
  uint64_t bar[2];               // of the exchanges in turn
  int run[4];   // row0, n, len, whether there is a run
};

template <bool BF16>
__device__ __forceinline__ float value_at(const void* p, long long i) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16) : static_cast<const float*>(p)[i];
}
template <bool BF16>
constexpr int kVecOf = BF16 ? 8 : 4;  // elements of 16 bytes

// 16 bytes of a row of n elements from element i on, zeros outside.  One load where they are aligned and all inside.
template <bool BF16>
__device__ __forceinline__ uint4 load_vec(const uint8_t* row, int i, int n) {
  constexpr int kSize = BF16 ? 2 : 4, kVec = kVecOf<BF16>;
  const uint8_t* p = row + static_cast<long long>(i) * kSize;
  if (i >= 0 && i + kVec <= n && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) return *reinterpret_cast<const uint4*>(p);
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    auto bits = [&](int j) -> uint32_t {
      if (j < 0 || j >= n) return 0u;
      return BF16 ? reinterpret_cast<const uint16_t*>(row)[j] : reinterpret_cast<const uint32_t*>(row)[j];
    };
    u[e] = BF16 ? bits(i + 2 * e) | bits(i + 2 * e + 1) << 16 : bits(i + e);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
template <bool BF16>
__device__ __forceinline__ void unpack(uint4 w, float (&x)[kVecOf<BF16>]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (BF16) {
      x[(2 * e) % kVecOf<BF16>] = __uint_as_float(u[e] << 16);
      x[(2 * e + 1) % kVecOf<BF16>] = __uint_as_float(u[e] & 0xFFFF0000u);
    } else {
      x[e] = __uint_as_float(u[e]);
    }
  }
}
// Elements by which a row begins behind a 16-byte boundary.
template <bool BF16>
__device__ __forceinline__ int phase_of(const uint8_t* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / (BF16 ? 2 : 4);
}

// A probability as it is taken: 0 for what is none.  bad: 1 outside [0, 1], 2 not finite.
__device__ __forceinline__ float probability(float x, int& bad) {
  if (x >= 0.f && x <= 1.f) return x;
  bad |= isfinite(x) ? 1 : 2;
  return 0.f;
}
// floor(2^44 x), 0 <= x <= 1: the significand (x = m 2^(e - 150)) shifted.
__device__ __forceinline__ unsigned long long whole(float x) {
  const uint32_t b = __float_as_uint(x), e = b >> 23;
  const unsigned long long m = static_cast<unsigned long long>(b & 0x7FFFFFu | 0x800000u) << 21;
  return e == 0 ? 0 : m >> min(127u - e, 63u);
}
// The same of many values at once, in 32-bit sums of two parts.  x + 2 is x rounded to a multiple of 2^-22 (values in [2, 4) have that step), what
// it leaves is exact, and times 2^44 it is below 2^22 in magnitude, so that adding 1.5 2^23, rounded down, is its floor.  Up to 2^9 values.
struct Whole {
  uint32_t high = 0, low = 0, n = 0;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(x, 2.f), left = __fsub_rn(x, __fsub_rn(t, 2.f));
    high += __float_as_uint(t);
    low += __float_as_uint(__fmaf_rd(left, 0x1p44f, 12582912.f));
    ++n;
  }
  __device__ __forceinline__ unsigned long long sum() const {
    const uint32_t h = high - n * 0x40000000u;
    const int32_t l = static_cast<int32_t>(low - n * 0x4B400000u);
    return (static_cast<unsigned long long>(h) << 22) + static_cast<long long>(l);
  }
};
__device__ __forceinline__ float rest(float p, float q, float c) { return fmaxf(__fsub_rn(p, __fmul_rn(c, q)), 0.f); }

// Scores in the order of their values as unsigned numbers: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x, int& bad) {
  if (x != x) {
    bad |= 2;
    x = -INFINITY;
  }
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Of values below 2^63: three parts of 22 bits, whose sums fit 32.
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const uint32_t a = __reduce_add_sync(kAll, static_cast<uint32_t>(v) & 0x3FFFFFu);
  const uint32_t b = __reduce_add_sync(kAll, static_cast<uint32_t>(v >> 22) & 0x3FFFFFu);
  const uint32_t c = __reduce_add_sync(kAll, static_cast<uint32_t>(v >> 44));
  return a + (static_cast<unsigned long long>(b) << 22) + (static_cast<unsigned long long>(c) << 44);
}

// What a block tells the others goes straight into their shared memory and counts there as bytes of an mbarrier's phase.
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(dec::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void send(uint32_t to, unsigned long long v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(to), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(dec::smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
constexpr long long kWaitClocks = 4000000000ll;  // some seconds: a wait that lasts longer gives up

// A hint to the L2 to bring a warp's piece of a row that a refusal would need.
template <bool BF16>
__device__ __forceinline__ void bring(const uint8_t* row, int vocab, int piece) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row), bytes = static_cast<uintptr_t>(vocab) * (BF16 ? 2 : 4);
  const uintptr_t from = (at + bytes * piece / kPieces + 15) & ~static_cast<uintptr_t>(15), to = (at + bytes * (piece + 1) / kPieces) & ~static_cast<uintptr_t>(15);
  if (from < to) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(static_cast<uint32_t>(to - from)) : "memory");
}

enum class Pass { kGreedy, kTarget, kRest };

// A warp's piece of a row: the sum of whole(p), of whole(rest(p, q, c)), or the largest (score, ~index).  kAtOnce loads of a row are on their way
// together.
constexpr int kAtOnce = 4;
template <bool BF16, Pass PASS>
__device__ __forceinline__ unsigned long long pass_over(const uint8_t* p, const uint8_t* q, float c, int vocab, int piece, int& bad) {
  constexpr int kVec = kVecOf<BF16>;
  const int lane = threadIdx.x & 31, off = phase_of<BF16>(p);
  const int n = (vocab + off + kVec - 1) / kVec;
  const int v0 = n * piece / kPieces, v1 = n * (piece + 1) / kPieces;
  unsigned long long best = 0;
  Whole sum;
  uint32_t top = 0;  // largest value as bits: above 1.0's, one of them is no probability
#pragma unroll 1
  for (int v = v0 + lane; v - lane < v1; v += 32 * kAtOnce) {
    uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = v + 32 * k < v1 ? (v + 32 * k) * kVec - off : vocab;
      x[k] = load_vec<BF16>(p, i, vocab);
      if (PASS == Pass::kRest) y[k] = load_vec<BF16>(q, i, vocab);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (v - lane + 32 * k >= v1) break;  // no lane has one
      const int i = v + 32 * k < v1 ? (v + 32 * k) * kVec - off : vocab;
      float a[kVec], b[kVec];
      unpack<BF16>(x[k], a);
      if (PASS == Pass::kRest) unpack<BF16>(y[k], b);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (PASS == Pass::kGreedy) {
          const bool in = i + e >= 0 && i + e < vocab;
          const unsigned long long key = static_cast<unsigned long long>(ordered(a[e], bad)) << 32 | static_cast<uint32_t>(~(i + e));
          if (in && key > best) best = key;
        } else {
          top = max(top, __float_as_uint(a[e]));
          if (PASS == Pass::kRest) top = max(top, __float_as_uint(b[e]));
          sum.add(PASS == Pass::kRest ? rest(a[e], b[e], c) : a[e]);
        }
      }
    }
  }
  if (PASS == Pass::kGreedy) {
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(kAll, best, o));
    return best;
  }
  unsigned long long total = sum.sum();
  if (top > 0x3F800000u) {  // value by value
    total = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
      float a[kVec], b[kVec] = {};
      unpack<BF16>(load_vec<BF16>(p, v * kVec - off, vocab), a);
      if (PASS == Pass::kRest) unpack<BF16>(load_vec<BF16>(q, v * kVec - off, vocab), b);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float pe = probability(a[e], bad);
        total += whole(PASS == Pass::kRest ? rest(pe, probability(b[e], bad), c) : pe);
      }
    }
  }
  return warp_sum(total);
}

// The token of a piece at which the sum over the piece first exceeds t (t is less than the piece's sum).
template <bool BF16, bool REST>
__device__ __forceinline__ int token_at(const uint8_t* p, const uint8_t* q, float c, int vocab, int piece, unsigned long long t) {
  constexpr int kVec = kVecOf<BF16>, kSteps = 4;  // steps of 32 vectors whose loads are on their way together
  const int lane = threadIdx.x & 31, off = phase_of<BF16>(p);
  const int n = (vocab + off + kVec - 1) / kVec;
  const int v0 = n * piece / kPieces, v1 = n * (piece + 1) / kPieces;
  int bad = 0;
  auto weight = [&](float x, float y) {
    const float pe = probability(x, bad);
    return whole(REST ? rest(pe, probability(y, bad), c) : pe);
  };
#pragma unroll 1
  for (int b = v0; b < v1; b += 32 * kSteps) {
    uint4 x[kSteps], y[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int v = b + 32 * k + lane, i = v < v1 ? v * kVec - off : vocab;
      x[k] = load_vec<BF16>(p, i, vocab);
      y[k] = REST ? load_vec<BF16>(q, i, vocab) : make_uint4(0, 0, 0, 0);
    }
    unsigned long long mine[kSteps], all[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float u[kVec], w[kVec];
      unpack<BF16>(x[k], u);
      unpack<BF16>(y[k], w);
      mine[k] = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) mine[k] += weight(u[e], w[e]);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) all[k] = warp_sum(mine[k]);
    int step = -1;
    uint4 px = make_uint4(0, 0, 0, 0), py = px;
    unsigned long long sum = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (step >= 0) continue;
      if (t < all[k]) {
        step = k;
        px = x[k];
        py = y[k];
        sum = mine[k];
      } else {
        t -= all[k];
      }
    }
    if (step < 0) continue;
    unsigned long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(kAll, inc, o);
      if (lane >= o) inc += up;
    }
    const int l = __ffs(__ballot_sync(kAll, inc > t)) - 1;
    float u[kVec], w[kVec];
    unpack<BF16>(px, u);
    unpack<BF16>(py, w);
    unsigned long long cum = inc - sum;
    int tok = -1;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {  // the first e at which the sum exceeds t
      cum += weight(u[e], w[e]);
      if (tok < 0 && cum > t) tok = (b + 32 * step + lane) * kVec - off + e;
    }
    return __shfl_sync(kAll, tok, l);
  }
  return 0;  // cannot be, unless the row changed under the call
}

template <bool BF16>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / kCluster, piece = rank * kWarps + warp;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) dec::mbar_init(&sh.bar[i], 1);
    dec::fence_mbar_init();
  }
  cluster.sync();  // every block runs, and has its barriers, before another one writes to it
  if (rank == 0) {  // the run and its tree, to all blocks
    __shared__ int run[4];
    if (tid == 0) {
      const int r0 = a.run_starts ? a.run_starts[s] : s, r1 = a.run_starts ? a.run_starts[s + 1] : s + 1;
      const int len = a.seq_lens ? a.seq_lens[s] : 0;
      const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.num_rows && r1 - r0 <= KVQ_MAX_TREE && (!a.seq_lens || (len >= r1 - r0 && len <= kMaxContext));
      if (!ok) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      run[0] = r0;
      run[1] = ok ? r1 - r0 : 0;
      run[2] = len;
      run[3] = ok;
    }
    __syncthreads();
    for (int r = 0; r < kCluster; ++r) {
      Shared* to = cluster.map_shared_rank(&sh, r);
      if (tid < 4) to->run[tid] = run[tid];
    }
    for (int i = tid; i < run[1]; i += kThreads) {
      const int up = a.parents[run[0] + i], tok = a.tokens[run[0] + i];
      if (up < -1 || up >= i) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      if (i > 0 && (tok < 0 || tok >= a.vocab)) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      for (int r = 0; r < kCluster; ++r) {
        Shared* to = cluster.map_shared_rank(&sh, r);
        to->parent[i] = i == 0 || up >= i ? -1 : up;
        to->token[i] = tok;
      }
    }
  }
  cluster.sync();
  const int row0 = sh.run[0], n = sh.run[1];
  const bool writer = rank == 0 && tid == 0, asks = rank == 0 && warp == 0;
  if (n == 0) {
    if (writer) {
      a.kept[s] = 0;
      a.next[s] = -1;
      if (a.seq_lens_out) a.seq_lens_out[s] = sh.run[2];
    }
    return;
  }
  const bool greedy = a.uniform == nullptr, drafts = a.draft != nullptr;
  int bad = 0;
  constexpr int kSize = BF16 ? 2 : 4;
  // the first child of `cur` behind row `j`, n for none
  auto next_child = [&](int cur, int j) {
    for (int b = (j + 1) & ~31; b < n; b += 32) {
      const int i = b + lane;
      const unsigned hit = __ballot_sync(kAll, i > j && i < n && sh.parent[i] == cur);
      if (hit) return b + __ffs(hit) - 1;
    }
    return n;
  };
  // The numbers that decide about a child, and the row's own: loaded before a pass, looked at (`taken`) behind it, so that nothing waits for them.
  auto ask = [&](int cur, int child) {
    Ask k{0.f, 0.f, 0.f, 0.f};
    k.draw = a.uniform[2 * (static_cast<long long>(row0) + cur) + 1];
    if (child < n) {
      const int tok = sh.token[child];
      k.u = a.uniform[2 * (static_cast<long long>(row0) + child)];
      if (tok >= 0 && tok < a.vocab) {
        const long long row = row0 + cur;
        k.p = value_at<BF16>(a.target, row * a.target_stride + tok);
        k.q = value_at<BF16>(a.draft, row * a.draft_stride + tok);
      }
    }
    return k;
  };
  auto taken = [&](Ask k) {
    if (asks) {
      if (!(k.u >= 0.f && k.u < 1.f)) report(a.err, KVQ_ERR_RANGE);
      k.p = probability(k.p, bad);
      k.q = probability(k.q, bad);
    }
    return k;
  };
  // A warp's number, and beside it what is asked, to all blocks; those of all warps are in sh.part[buf] afterwards.  A block sends for an exchange when
  // it has all of the last one's, so the barriers and buffers of two exchanges in turn are never written while they are still in use.
  uint32_t turn = 0;
  bool alive = true;
  Ask asked{};
  auto exchange = [&](unsigned long long v, int buf, const Ask& raw) {
    uint64_t* bar = &sh.bar[turn & 1];
    if (tid == 0) {  // 8 bytes of every warp, 16 that are asked
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(dec::smem_u32(bar)), "r"(kPieces * 8 + 16) : "memory");
    }
    const Ask k = taken(raw);
    if (lane < kCluster) {
      const uint32_t there = at_rank(bar, lane);
      send(at_rank(&sh.part[buf][piece], lane), v, there);
      if (asks) {
        auto pair = [](float a, float b) { return static_cast<unsigned long long>(__float_as_uint(b)) << 32 | __float_as_uint(a); };
        send(at_rank(&sh.ask[turn & 1][0], lane), pair(k.u, k.p), there);
        send(at_rank(&sh.ask[turn & 1][1], lane), pair(k.q, k.draw), there);
      }
    }
    if (alive && !try_wait_cluster(bar, (turn >> 1) & 1u)) {
      const long long t0 = clock64();
      while (alive && !try_wait_cluster(bar, (turn >> 1) & 1u)) alive = clock64() - t0 <= kWaitClocks;
    }
    alive = __all_sync(kAll, alive);
    const unsigned long long a0 = sh.ask[turn & 1][0], a1 = sh.ask[turn & 1][1];
    asked = Ask{__uint_as_float(static_cast<uint32_t>(a0)), __uint_as_float(static_cast<uint32_t>(a0 >> 32)), __uint_as_float(static_cast<uint32_t>(a1)),
                __uint_as_float(static_cast<uint32_t>(a1 >> 32))};
    ++turn;
  };
  auto total = [&](const unsigned long long* part) {
    unsigned long long v = 0;
#pragma unroll
    for (int i = 0; i < kPieces / 32; ++i) v += part[32 * i + lane];
    return warp_sum(v);
  };
  int cur = 0, kept = 1, last = -1;
  if (writer) a.keep[row0] = 0;
  for (int step = 0; step < n && alive; ++step) {  // a path has at most n rows
    const long long row = row0 + cur;
    const uint8_t* p = static_cast<const uint8_t*>(a.target) + row * a.target_stride * kSize;
    const uint8_t* q = drafts ? static_cast<const uint8_t*>(a.draft) + row * a.draft_stride * kSize : nullptr;
    int go = n, drawn = -1;
    if (greedy) {
      const int buf = 2 + (step & 1);
      exchange(pass_over<BF16, Pass::kGreedy>(p, q, 0.f, a.vocab, piece, bad), buf, Ask{});
      unsigned long long best = 0;
#pragma unroll
      for (int i = 0; i < kPieces / 32; ++i) best = max(best, sh.part[buf][32 * i + lane]);
#pragma unroll
      for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(kAll, best, o));
      drawn = static_cast<int>(~static_cast<uint32_t>(best));
    } else {
      int child = drafts ? next_child(cur, 0) : n;
      Ask k{};
      if (asks) k = ask(cur, child);
      if (child < n && lane == 0) bring<BF16>(q, a.vocab, piece);
      const unsigned long long* const first = sh.part[2 + (step & 1)];
      exchange(pass_over<BF16, Pass::kTarget>(p, q, 0.f, a.vocab, piece, bad), 2 + (step & 1), k);
      const unsigned long long* part = first;
      unsigned long long z = total(part);
      const unsigned long long z0 = z;
      float c = 0.f;
      if (child < n) {
        while (child < n && alive) {
          k = asked;
          const double zd = static_cast<double>(z) * 0x1p-44, cq = static_cast<double>(c) * static_cast<double>(k.q);
          if (__dmul_rn(static_cast<double>(k.u) * static_cast<double>(k.q), zd) < __dsub_rn(static_cast<double>(k.p), cq)) {
            go = child;
            break;
          }
          c = static_cast<float>(__dadd_rn(static_cast<double>(c), zd));
          child = next_child(cur, child);
          if (asks) k = ask(cur, child);
          const int buf = turn & 1;
          exchange(pass_over<BF16, Pass::kRest>(p, q, c, a.vocab, piece, bad), buf, k);
          part = sh.part[buf];
          z = total(part);
        }
      }
      if (go == n) {  // draw
        const float u = asked.draw;
        if (writer && !(u >= 0.f && u < 1.f)) report(a.err, KVQ_ERR_RANGE);
        if (z == 0 && c != 0.f) {
          part = first;
          z = z0;
          c = 0.f;
        }
        if (z == 0) {
          if (writer) report(a.err, KVQ_ERR_RANGE);
        } else {
          const double td = floor(__dmul_rn(static_cast<double>(u), static_cast<double>(z)));
          const unsigned long long t = td > 0. ? (td < static_cast<double>(z) ? static_cast<unsigned long long>(td) : z - 1) : 0;
          // the piece that holds t, and what is before it
          unsigned long long before = 0, mine = 0;
          int which = -1;
          for (int i = 0; i < kPieces / 32 && which < 0; ++i) {
            const unsigned long long v = part[32 * i + lane];
            unsigned long long inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned long long up = __shfl_up_sync(kAll, inc, o);
              if (lane >= o) inc += up;
            }
            const unsigned hit = __ballot_sync(kAll, before + inc > min(t, z - 1));
            if (hit) {
              const int l = __ffs(hit) - 1;
              which = 32 * i + l;
              mine = before + __shfl_sync(kAll, inc - v, l);
            }
            before += __shfl_sync(kAll, inc, 31);
          }
          unsigned long long tok = 0;
          if (which == piece)
            tok = 1 + (c != 0.f ? token_at<BF16, true>(p, q, c, a.vocab, piece, min(t, z - 1) - mine)
                                : token_at<BF16, false>(p, q, c, a.vocab, piece, min(t, z - 1) - mine));
          const int buf = turn & 1;
          exchange(tok, buf, Ask{});
          drawn = static_cast<int>(total(sh.part[buf])) - 1;
        }
      }
    }
    if (!drafts && drawn >= 0) {
      go = cur;
      do go = next_child(cur, go); while (go < n && sh.token[go] != drawn);
    }
    if (!alive) break;
    if (go >= n) {
      last = drawn;
      break;
    }
    if (writer) a.keep[row0 + kept] = go;
    ++kept;
    cur = go;
  }
  if (!alive) report(a.err, KVQ_ERR_TIMEOUT);
  if (bad) report(a.err, bad & 2 ? KVQ_ERR_NONFINITE_INPUT : KVQ_ERR_RANGE);
  if (rank == 0) {
    __syncthreads();
    for (int i = kept + tid; i < n; i += kThreads) a.keep[row0 + i] = -1;
    if (tid == 0) {
      a.kept[s] = kept;
      a.next[s] = last;
      if (a.seq_lens_out) a.seq_lens_out[s] = sh.run[2] - n + kept;
    }
  }
  cluster.sync();  // no block ends while another may still write to it
}

}  // namespace
}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_verify_runs(const void* target, int64_t target_row_stride, const void* draft, int64_t draft_row_stride,
                                      int32_t dtype, int32_t vocab, const int32_t* tokens, const int32_t* parents, const float* uniform,
                                      const int32_t* run_starts, int32_t batch, int32_t num_rows, int32_t* keep, int32_t* kept_lens,
                                      int32_t* next_tokens, const int32_t* seq_lens, int32_t* seq_lens_out, int32_t* err_word,
                                      kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::runs;
  if (dtype != KVQ_DTYPE_F32 && dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > kMaxVocab || batch < 0 || batch > kMaxBatch || num_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (!run_starts && num_rows != batch) return KVQ_ERR_INVALID_ARG;
  if ((seq_lens != nullptr) != (seq_lens_out != nullptr) || (draft && !uniform)) return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  if (!kept_lens || !next_tokens) return KVQ_ERR_INVALID_ARG;
  const uintptr_t mask = dtype == KVQ_DTYPE_BF16 ? 1u : 3u;
  if (num_rows > 0) {
    if (!target || !tokens || !parents || !keep) return KVQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(target) & mask) || (reinterpret_cast<uintptr_t>(draft) & mask)) return KVQ_ERR_INVALID_ARG;
    if (target_row_stride < vocab || (draft && draft_row_stride < vocab)) return KVQ_ERR_INVALID_ARG;
  }
  const VerifyArgs a{target, draft, target_row_stride, draft_row_stride, vocab, tokens, parents, uniform, run_starts, batch, num_rows, keep, kept_lens,
                     next_tokens, seq_lens, seq_lens_out, err_word};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_DTYPE_BF16) verify_kernel<true><<<batch * kCluster, kThreads, 0, st>>>(a);
  else verify_kernel<false><<<batch * kCluster, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
