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
#include <algorithm>

#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 2048;

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

template <bool INT8>
__device__ __forceinline__ uint8_t encode(float x) {  // x = value 2^-e
  if (INT8) {
    const int c = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
    return static_cast<uint8_t>(c + 128);
  }
  return f32_to_e4m3_bits(x);
}
template <bool INT8>
__device__ __forceinline__ float decode(uint8_t b) {
  return INT8 ? static_cast<float>(static_cast<int>(b) - 128) : e4m3_bits_to_f32(b);
}

template <bool INT8>
__device__ __forceinline__ uint4 rescale(uint4 w, float f) {  // 16 codes times f = 2^-d
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r |= static_cast<uint32_t>(encode<INT8>(decode<INT8>(x[i] >> (8 * j)) * f)) << (8 * j);
    x[i] = r;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// eight channels of one row
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, long long at, float (&x)[8]) {
  if (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

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

template <bool INT8, bool BF16>
__global__ void __launch_bounds__(kThreads) append_runs_kernel(const AppendArgs a) {
  __shared__ int s_cum[kMaxBatch + 1];
  __shared__ int s_warp[kThreads / 32];
  __shared__ float s_max[2][kThreads / 32];
  __shared__ __align__(16) uint8_t s_tile[2][kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // pages that each run touches, summed over the batch
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    int loc = 0;
    auto pages = [&](int s) {
      const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.num_rows, a.max_pages);
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
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int pi = static_cast<int>(item / a.H), h = static_cast<int>(item % a.H);
    int lo = 0, hi = a.batch - 1;  // last s with cum[s] <= pi
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cum[mid] <= pi) lo = mid; else hi = mid - 1;
    }
    const int s = lo;
    const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.num_rows, a.max_pages);
    const int first = r.len - r.n;                       // position of the run's first token
    const int page = first / kPage + (pi - s_cum[s]);
    const int p0 = page * kPage;
    if (page < first / kPage || p0 >= r.len) continue;  // runs that overlap (reported where they are read)
    const int from = max(first - p0, 0), to = min(r.len - p0, kPage);  // the page's tokens that are new
    const int phys = a.block_table[static_cast<size_t>(s) * a.max_pages + page];
    if (phys < 0 || phys >= a.num_pages) {
      if (tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      continue;
    }
    const size_t tile = (static_cast<size_t>(phys) * a.H + h) * kTile;
    const size_t si = static_cast<size_t>(h) * a.num_pages + phys;

    float x[2][2][8];  // [plane][token t8, t8 + 8][channel]
    bool odd = false;
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t8 + 8 * i;
      if (t >= from && t < to) {
        const long long row = r.row0 + (p0 + t - first);
        load8<BF16>(a.kin, row * a.k_stride + h * kHeadDim + ch, x[0][i]);
        load8<BF16>(a.vin, row * a.v_stride + h * kHeadDim + ch, x[1][i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[0][i][e] = x[1][i][e] = 0.f;
      }
    }
    int ek0 = kMinExp, ev0 = kMinExp;
    constexpr uint32_t kZero = INT8 ? 0x80808080u : 0u;
    uint4 wk = make_uint4(kZero, kZero, kZero, kZero), wv = wk;
    if (from > 0) {  // the page holds earlier tokens of its request
      ek0 = f16_to_exp(a.ks[si]);
      ev0 = f16_to_exp(a.vs[si]);
      wk = *reinterpret_cast<const uint4*>(a.k + tile + 16 * tid);
      wv = *reinterpret_cast<const uint4*>(a.v + tile + 16 * tid);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mk = fmaxf(mk, amax8(x[0][i], odd));
      mv = fmaxf(mv, amax8(x[1][i], odd));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (lane == 0) {
      s_max[0][warp] = mk;
      s_max[1][warp] = mv;
    }
    if (odd) report(a.err, KVQ_ERR_NONFINITE_INPUT);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      mk = fmaxf(mk, s_max[0][w]);
      mv = fmaxf(mv, s_max[1][w]);
    }
    constexpr float kTop = (INT8 ? 127.f : 448.f) * 32768.f;
    if (tid == 0 && (mk > kTop || mv > kTop)) report(a.err, KVQ_ERR_RANGE);
    const int ek = max(exponent_for<INT8>(mk), ek0), ev = max(exponent_for<INT8>(mv), ev0);
    if (from > 0) {
      if (ek > ek0) wk = rescale<INT8>(wk, exp2_int(ek0 - ek));
      if (ev > ev0) wv = rescale<INT8>(wv, exp2_int(ev0 - ev));
    }
    *reinterpret_cast<uint4*>(&s_tile[0][16 * tid]) = wk;
    *reinterpret_cast<uint4*>(&s_tile[1][16 * tid]) = wv;
    __syncthreads();
    const float fk = exp2_int(-ek), fv = exp2_int(-ev);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t8 + 8 * i;
      if (t >= from) {  // new tokens; behind the last one, code 0
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= static_cast<uint32_t>(encode<INT8>(x[0][i][e] * fk)) << (8 * (e & 3));
        *reinterpret_cast<uint2*>(&s_tile[0][k8_offset(t, ch)]) = make_uint2(w[0], w[1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s_tile[1][v8_offset(t, ch + e)] = encode<INT8>(x[1][i][e] * fv);
      }
    }
    __syncthreads();
    *reinterpret_cast<uint4*>(a.k + tile + 16 * tid) = *reinterpret_cast<const uint4*>(&s_tile[0][16 * tid]);
    *reinterpret_cast<uint4*>(a.v + tile + 16 * tid) = *reinterpret_cast<const uint4*>(&s_tile[1][16 * tid]);
    if (tid == 0) {
      a.ks[si] = exp_to_f16(ek);
      a.vs[si] = exp_to_f16(ev);
    }
    // the next item writes s_max before its first barrier and s_tile only behind it
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool INT8>
cudaError_t launch(const AppendArgs& a, bool bf16, unsigned grid, cudaStream_t s) {
  if (bf16) append_runs_kernel<INT8, true><<<grid, kThreads, 0, s>>>(a);
  else append_runs_kernel<INT8, false><<<grid, kThreads, 0, s>>>(a);
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
  const unsigned grid = static_cast<unsigned>(std::min<long long>(items, 152 * 12));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = in_dtype == KVQ_DTYPE_BF16;
  const cudaError_t e = cache->k_fmt == KVQ_FMT_INT8_PAGE ? launch<true>(a, bf16, grid, s) : launch<false>(a, bf16, grid, s);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
