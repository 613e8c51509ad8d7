// append_runs.cu -- kvq_append_runs: quantize the runs' keys and values into page-scaled tiles.
//
// A page of one kv head has one scale 2^e per plane, e the smallest exponent with amax <= qmax 2^e (qmax 448 for E4M3,
// 127 for INT8).  A power of two because a page fills over many steps: when a later token needs a larger scale, the
// codes already there are multiplied by 2^-d, which is exact for E4M3 down to its subnormals and rounds INT8 codes
// once, and the errors of repeated growth sum to less than one step of the final scale (1/2 + 1/4 + ...); with a free
// scale every token could move the scale and each move would add half a step.  It also makes the division exact, so
// the codes are a function of the inputs alone: code = rne(x 2^-e).
//
// One block per (page, kv head) item: all tokens that a run brings to a page are reduced together, so there are no atomics
// and the result does not depend on any order.
//
// Bound by memory: 512 (bf16) or 1024 (fp32) bytes read and 256 written for every token and kv head.  A value tile's 16-byte
// words hold four tokens of four channels, which lie in eight threads: they are put together by shuffles (byte stores into
// the staged tile, with their bank conflicts, took 27 us on 11996 tokens of 8 heads).  A block fetches its next item while it
// quantizes one: 20.6 us there with inputs that are not in the L2, against 10.9 for the bytes at the copy rate; about 10 us
// are issue slots (2,200 instructions of a warp for an item).
#include <algorithm>

#include "codes.cuh"
#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 2048;
constexpr int kSmemStatic = 2 * kTile + 128;  // of the kernel, at most

struct AppendArgs {
  uint8_t* k;
  uint8_t* v;
  uint16_t* ks;
  uint16_t* vs;
  int H, num_pages;
  const void* kin;
  const void* vin;
  long long k_stride, v_stride;  // elements between rows
  const int32_t* run_starts;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int max_pages, batch, num_rows;
  int32_t* err;
};

template <bool INT8>
__device__ __forceinline__ int exponent_for(float amax) {
  // amax = (1 + f) 2^k; qmax = (1 + lead) 2^k0
  constexpr int k0 = INT8 ? 6 : 8;
  constexpr uint32_t lead = INT8 ? 0x7E0000u : 0x600000u;
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - k0 + ((b & 0x7FFFFFu) > lead ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// eight channels of one row, as loaded and as values
template <bool BF16>
struct Raw {
  static constexpr int kWords = BF16 ? 1 : 2;
  uint4 w[kWords];
  // from this thread's words of a stage, kThreads words apart
  __device__ __forceinline__ void load(const uint4* stage) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = stage[i * kThreads];
  }
  // Largest magnitude, as binary32 bits: as integers, a NaN is above infinity and that above what is finite.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (BF16) asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(u[e] & 0x7FFF7FFFu));
        else m = max(m, u[e] & 0x7FFFFFFFu);
      }
    }
    return BF16 ? max(m & 0xFFFF0000u, m << 16) : m;
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (BF16) {
          x[2 * e] = __uint_as_float(u[e] << 16);
          x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        } else {
          x[4 * i + e] = __uint_as_float(u[e]);
        }
      }
    }
  }
};

// the largest finite magnitude of 8 values; a NaN becomes 0, an infinity stays (it saturates) and is not counted
__device__ __forceinline__ float amax8(float (&x)[8], bool& odd) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    if (!(a < INFINITY)) {
      odd = true;
      if (x[i] != x[i]) x[i] = 0.f;
    } else {
      m = fmaxf(m, a);
    }
  }
  return m;
}

// Asynchronous copies to the issuing thread's own words of shared memory (nothing but their wait is needed to read them back).
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool there) {  // zeros where there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(int* dst, const int* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kStages = 2;  // an item on its way while one is quantized
// Blocks on an SM, where its shared memory holds as many.  11996 tokens of 8 heads, bf16, inputs not in the L2: 20.6 us with 6 blocks and 2 stages, 22.4 with 7 and
// 2, 22.3 with 6 and 3, 21.5 with 5 and 3, 28.6 with 8 and 3 (64 registers do not hold the loop).
constexpr int kBlocksBf16 = 6, kBlocksF32 = 4;
template <bool BF16>
__host__ __device__ constexpr int stage_bytes() {
  return kThreads * (4 * Raw<BF16>::kWords * 16 + 4);  // [plane][token][word][thread] and the page's table entry
}

template <bool INT8, bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? kBlocksBf16 : kBlocksF32) append_runs_kernel(const AppendArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* stages = smem;
  int* s_cum = reinterpret_cast<int*>(smem + kStages * stage_bytes<BF16>());  // [batch + 1] pages of the runs before
  int* s_first = s_cum + a.batch + 1;                                         // the run's first position,
  int* s_len = s_first + a.batch;                                             // its context,
  int* s_row = s_len + a.batch;                                               // its first row
  __shared__ int s_warp[kThreads / 32];
  __shared__ uint32_t s_max[2][kThreads / 32];
  __shared__ __align__(16) uint8_t s_tile[2][kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // pages that each run touches, summed over the batch
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    int loc = 0;
    auto pages = [&](int s) {
      const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.num_rows, a.max_pages);
      s_first[s] = r.len - r.n;
      s_len[s] = r.len;
      s_row[s] = r.row0;
      if (!a.run_starts && r.n && r.len == 0) return 0;  // nothing to append
      if (r.row0 < 0 || r.n > r.len) {
        if (blockIdx.x == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
        return 0;
      }
      return r.n ? (r.len - 1) / kPage - (r.len - r.n) / kPage + 1 : 0;
    };
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s < a.batch) loc += s_cum[s + 1] = pages(s);
    }
    int inc = loc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int run = inc - loc;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s < a.batch) s_cum[s + 1] = run += s_cum[s + 1];
    }
    if (tid == 0) s_cum[0] = 0;
    __syncthreads();
  }

  const long long items = static_cast<long long>(s_cum[a.batch]) * a.H;
  const int t8 = tid >> 4, ch = (tid & 15) * 8;
  // Where an item lies; blocks go through the items in steps of the grid.
  struct Walk {
    int pi, h, run;  // page (of all runs'), kv head, run
  };
  const int step_pi = gridDim.x / a.H, step_h = gridDim.x % a.H;
  auto advance = [&](Walk& w) {
    w.pi += step_pi;
    w.h += step_h;
    if (w.h >= a.H) {
      w.h -= a.H;
      ++w.pi;
    }
    while (w.run + 1 < a.batch && s_cum[w.run + 1] <= w.pi) ++w.run;
  };
  auto page_at = [&](const Walk& w) { return page_of_run(s_first[w.run], s_len[w.run], w.pi - s_cum[w.run]); };
  Walk ahead{static_cast<int>(blockIdx.x / a.H), static_cast<int>(blockIdx.x % a.H), 0};
  {
    int hi = a.batch - 1;  // last run with cum <= pi
    while (ahead.run < hi) {
      const int mid = (ahead.run + hi + 1) >> 1;
      if (s_cum[mid] <= ahead.pi) ahead.run = mid; else hi = mid - 1;
    }
  }
  Walk here = ahead;
  constexpr int kWords = Raw<BF16>::kWords;
  auto words_of = [&](int stage) { return reinterpret_cast<uint4*>(stages + stage * stage_bytes<BF16>()) + tid; };
  auto entry_of = [&](int stage) { return reinterpret_cast<int*>(stages + stage * stage_bytes<BF16>() + kThreads * 4 * kWords * 16) + tid; };
  auto fetch = [&](long long item, int stage) {
    if (item < items) {
      const RunPage p = page_at(ahead);
      uint4* dst = words_of(stage);
      copy4(entry_of(stage), a.block_table + static_cast<size_t>(ahead.run) * a.max_pages + p.page);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = t8 + 8 * i;
        const bool there = t >= p.from && t < p.to;
        const long long row = there ? s_row[ahead.run] + (p.p0 + t - p.first) : 0;
        const int col = ahead.h * kHeadDim + ch;
        constexpr int kSize = BF16 ? 2 : 4;
        const uint8_t* ks = static_cast<const uint8_t*>(a.kin) + (row * a.k_stride + col) * kSize;
        const uint8_t* vs = static_cast<const uint8_t*>(a.vin) + (row * a.v_stride + col) * kSize;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          copy16(dst + (i * kWords + w) * kThreads, ks + 16 * w, there);
          copy16(dst + ((2 + i) * kWords + w) * kThreads, vs + 16 * w, there);
        }
      }
      advance(ahead);
    }
    copies_commit();
  };
  for (int i = 0; i < kStages - 1; ++i) fetch(blockIdx.x + static_cast<long long>(i) * gridDim.x, i);
  int stage = 0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    fetch(item + static_cast<long long>(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
    copies_wait<kStages - 1>();
    const RunPage page = page_at(here);
    const int h = here.h, from = page.from, phys = *entry_of(stage);
    advance(here);
    float x[2][2][8];  // [plane][token t8, t8 + 8][channel]
    uint32_t top_k = 0, top_v = 0;
    {
      const uint4* src = words_of(stage);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Raw<BF16> k, v;
        k.load(src + i * kWords * kThreads);
        v.load(src + (2 + i) * kWords * kThreads);
        k.values(x[0][i]);
        v.values(x[1][i]);
        top_k = max(top_k, k.top());
        top_v = max(top_v, v.top());
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (page.to <= from) continue;
    if (phys < 0 || phys >= a.num_pages) {
      if (tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      continue;
    }
    const size_t tile = (static_cast<size_t>(phys) * a.H + h) * kTile;
    const size_t si = static_cast<size_t>(h) * a.num_pages + phys;

    int ek0 = kMinExp, ev0 = kMinExp;
    constexpr uint32_t kZero = INT8 ? 0x80808080u : 0u;
    uint4 wk = make_uint4(kZero, kZero, kZero, kZero), wv = wk;
    if (from > 0) {  // the page holds earlier tokens of its request
      ek0 = f16_to_exp(a.ks[si]);
      ev0 = f16_to_exp(a.vs[si]);
      wk = *reinterpret_cast<const uint4*>(a.k + tile + 16 * tid);
      wv = *reinterpret_cast<const uint4*>(a.v + tile + 16 * tid);
    }
    bool odd = false;
    if (max(top_k, top_v) >= 0x7F800000u) {  // something is not finite here
      float mk = 0.f, mv = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mk = fmaxf(mk, amax8(x[0][i], odd));
        mv = fmaxf(mv, amax8(x[1][i], odd));
      }
      top_k = __float_as_uint(mk);
      top_v = __float_as_uint(mv);
      report(a.err, KVQ_ERR_NONFINITE_INPUT);
    }
    top_k = __reduce_max_sync(0xffffffffu, top_k);
    top_v = __reduce_max_sync(0xffffffffu, top_v);
    if (lane == 0) {
      s_max[0][warp] = top_k;
      s_max[1][warp] = top_v;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      top_k = max(top_k, s_max[0][w]);
      top_v = max(top_v, s_max[1][w]);
    }
    const float mk = __uint_as_float(top_k), mv = __uint_as_float(top_v);
    constexpr float kTop = (INT8 ? 127.f : 448.f) * 32768.f;
    if (tid == 0 && (mk > kTop || mv > kTop)) report(a.err, KVQ_ERR_RANGE);
    const int ek = max(exponent_for<INT8>(mk), ek0), ev = max(exponent_for<INT8>(mv), ev0);
    if (from > 0) {
      if (ek > ek0) wk = rescale<INT8>(wk, exp2_int(ek0 - ek));
      if (ev > ev0) wv = rescale<INT8>(wv, exp2_int(ev0 - ev));
    }
    // The staged tiles, as 16-byte words in an order that spreads the stores over the banks.
    auto k_word = [](int w) { return w ^ ((w >> 5 & 1) << 2); };
    auto v_word = [](int w) { return w ^ ((w >> 3 & 1) | (w >> 5 & 1) << 1); };
    uint4* tk = reinterpret_cast<uint4*>(s_tile[0]);
    uint4* tv = reinterpret_cast<uint4*>(s_tile[1]);
    if (from > 0) {
      tk[k_word(tid)] = wk;
      tv[v_word(tid)] = wv;
      __syncthreads();
    }
    const float fk = exp2_int(-ek), fv = exp2_int(-ev);
    if (INT8 && (odd || mk > kTop || mv > kTop)) {  // beyond the largest code
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[0][i][e] = fminf(fmaxf(x[0][i][e], -127.f / fk), 127.f / fk);
          x[1][i][e] = fminf(fmaxf(x[1][i][e], -127.f / fv), 127.f / fv);
        }
    }
    // Keys: eight channels of a token are half a word.  Tokens behind the last get code 0.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t8 + 8 * i;
      const float(&y)[8] = x[0][i];
      if (t >= from)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(tk + k_word(k8_offset(t, ch) >> 4)) + (ch & 8)) =
            make_uint2(encode4<INT8>(y[0], y[1], y[2], y[3], fk), encode4<INT8>(y[4], y[5], y[6], y[7], fk));
    }
    // Values: the word of channels 32 b + g + {0, 8, 16, 24} (b = lane >> 2 & 3) and tokens t8 & ~1, + 1, + 8, + 9.
    {
      const int p = lane >> 4, u = lane & 3;
      uint32_t v[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[i][h] = encode4<INT8>(x[1][i][4 * h], x[1][i][4 * h + 1], x[1][i][4 * h + 2], x[1][i][4 * h + 3], fv);
      // channels 4 p .. 4 p + 3 of both tokens of the pair
      const uint32_t m0 = p ? v[0][1] : v[0][0], m1 = p ? v[1][1] : v[1][0];
      const uint32_t o0 = __shfl_xor_sync(0xffffffffu, p ? v[0][0] : v[0][1], 16), o1 = __shfl_xor_sync(0xffffffffu, p ? v[1][0] : v[1][1], 16);
      const uint32_t e0 = p ? o0 : m0, d0 = p ? m0 : o0, e1 = p ? o1 : m1, d1 = p ? m1 : o1;  // even, odd token
      // w[i]: channel 4 p + i of this lane's eight: tokens t, t + 1, t + 8, t + 9
      uint32_t w[4];
      const uint32_t l01 = __byte_perm(e0, d0, 0x5140), l23 = __byte_perm(e0, d0, 0x7362);
      const uint32_t h01 = __byte_perm(e1, d1, 0x5140), h23 = __byte_perm(e1, d1, 0x7362);
      w[0] = __byte_perm(l01, h01, 0x5410);
      w[1] = __byte_perm(l01, h01, 0x7632);
      w[2] = __byte_perm(l23, h23, 0x5410);
      w[3] = __byte_perm(l23, h23, 0x7632);
      // 4 x 4 transpose over the lanes u: afterwards w[i] is channel 4 p + u of lane i's eight
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bool up = u & 1;
        const uint32_t r = __shfl_xor_sync(0xffffffffu, up ? w[2 * b] : w[2 * b + 1], 1);
        if (up) w[2 * b] = r; else w[2 * b + 1] = r;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bool up = u & 2;
        const uint32_t r = __shfl_xor_sync(0xffffffffu, up ? w[b] : w[b + 2], 2);
        if (up) w[b] = r; else w[b + 2] = r;
      }
      const uint4 word = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x5410),
                                    __byte_perm(w[2], w[3], 0x7632));
      const int at = v_word(32 * (lane >> 2 & 3) + 4 * (4 * p + u) + warp);
      const int t0 = 2 * warp;  // the pair's tokens t0, t0 + 1 (bytes 0, 1 of a half word), t0 + 8, t0 + 9
      if (from == 0) {
        tv[at] = word;
      } else {  // keep the earlier tokens' bytes
        const uint32_t lo = (t0 >= from ? 0x00FF00FFu : 0u) | (t0 + 1 >= from ? 0xFF00FF00u : 0u);
        const uint32_t hi = (t0 + 8 >= from ? 0x00FF00FFu : 0u) | (t0 + 9 >= from ? 0xFF00FF00u : 0u);
        const uint4 was = tv[at];
        tv[at] = make_uint4((word.x & lo) | (was.x & ~lo), (word.y & hi) | (was.y & ~hi), (word.z & lo) | (was.z & ~lo),
                            (word.w & hi) | (was.w & ~hi));
      }
    }
    __syncthreads();
    *reinterpret_cast<uint4*>(a.k + tile + 16 * tid) = tk[k_word(tid)];
    *reinterpret_cast<uint4*>(a.v + tile + 16 * tid) = tv[v_word(tid)];
    if (tid == 0) {
      a.ks[si] = exp_to_f16(ek);
      a.vs[si] = exp_to_f16(ev);
    }
    // the next item writes s_max before its first barrier and s_tile only behind it
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool INT8, bool BF16>
cudaError_t launch(const AppendArgs& a, long long items, cudaStream_t s) {
  auto kern = append_runs_kernel<INT8, BF16>;
  auto smem_of = [](size_t batch) { return kStages * stage_bytes<BF16>() + (4 * batch + 1) * sizeof(int); };
  const size_t smem = smem_of(a.batch);
  static SmemLimit limit;
  const cudaError_t e = limit.raise(kern, smem_of(kMaxBatch));
  if (e != cudaSuccess) return e;
  // As many blocks as the SMs hold at once, each going through its share of the items: a large batch's tables leave room for
  // fewer (bf16, 1024 requests: five; of 64 tokens and 8 heads each 265 us with six, the sixth a second wave, 175 with five).
  const int sms = device_sm_count(), sm_smem = device_attr<cudaDevAttrMaxSharedMemoryPerMultiprocessor>();
  const int reserved = device_attr<cudaDevAttrReservedSharedMemoryPerBlock>();
  if (sms <= 0 || sm_smem <= 0) return cudaErrorInvalidDevice;
  const int fit = std::max(1, sm_smem / static_cast<int>(smem + kSmemStatic + reserved));
  const long long blocks = static_cast<long long>(sms) * std::min(BF16 ? kBlocksBf16 : kBlocksF32, fit);
  kern<<<static_cast<unsigned>(std::min(items, blocks)), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

kvq_status check_page_scaled_cache(const kvq_cache* c) {
  if (!c) return KVQ_ERR_INVALID_ARG;
  if (!fmt_page_scaled(c->k_fmt) || c->v_fmt != c->k_fmt || c->n_outlier_pairs != 0) return KVQ_ERR_UNSUPPORTED_LAYOUT;
  if (c->num_kv_heads <= 0 || c->num_kv_heads > KVQ_MAX_KV_HEADS || c->num_pages < 0 || c->reserved != 0 || c->reserved2 != 0)
    return KVQ_ERR_INVALID_ARG;
  if (!c->k_data || !c->v_data || !c->k_scale || !c->v_scale) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(c->k_data) || !aligned16(c->v_data) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_append_runs(const kvq_cache* cache, const void* k, int64_t k_row_stride, const void* v,
                                      int64_t v_row_stride, int32_t in_dtype, const int32_t* run_starts, int32_t batch,
                                      int32_t num_rows, const int32_t* block_table, int32_t max_pages_per_seq,
                                      const int32_t* seq_lens, int32_t* err_word, kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::runs;
  const kvq_status st = check_page_scaled_cache(cache);
  if (st != KVQ_OK) return st;
  if (in_dtype != KVQ_DTYPE_F32 && in_dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARG;
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_pages_per_seq < 0) return KVQ_ERR_INVALID_ARG;
  if (!run_starts && num_rows != batch) return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || num_rows == 0) return KVQ_OK;
  const int64_t width = static_cast<int64_t>(cache->num_kv_heads) * kHeadDim;
  const int64_t unit = in_dtype == KVQ_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
  if (k_row_stride < width || v_row_stride < width || k_row_stride % unit || v_row_stride % unit) return KVQ_ERR_INVALID_ARG;
  if (!k || !v || !seq_lens || !block_table || !aligned16(k) || !aligned16(v)) return KVQ_ERR_INVALID_ARG;
  if (max_pages_per_seq == 0) return KVQ_ERR_INVALID_ARG;
  AppendArgs a{static_cast<uint8_t*>(cache->k_data), static_cast<uint8_t*>(cache->v_data), cache->k_scale, cache->v_scale,
               cache->num_kv_heads, cache->num_pages, k, v, k_row_stride, v_row_stride, run_starts, seq_lens, block_table,
               max_pages_per_seq, batch, num_rows, err_word};
  // pages touched: at most one per row, and a run of n tokens touches at most (n + 14) / 16 + 1
  const long long pages = std::min<long long>(num_rows, num_rows / kPage + 2ll * batch);
  const long long items = pages * cache->num_kv_heads;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = in_dtype == KVQ_DTYPE_BF16;
  const cudaError_t e = cache->k_fmt == KVQ_FMT_INT8_PAGE ? (bf16 ? launch<true, true>(a, items, s) : launch<true, false>(a, items, s))
                                                          : (bf16 ? launch<false, true>(a, items, s) : launch<false, false>(a, items, s));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
