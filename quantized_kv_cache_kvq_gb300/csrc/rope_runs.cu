// rope_runs.cu -- kvq_rope_runs: RMS norm of every head of queries and keys, and the rotation to the row's position, in one pass.
//
//     y = x / sqrt(mean x^2 + eps) w,   (y_j, y_{j + 64}) -> (y_j c_j - y_{j + 64} s_j, y_{j + 64} c_j + y_j s_j)
//
// Eight lanes have a head: channels 8 l .. 8 l + 7 and the 64 further ones, so that a pair lies in one thread, loads are 16 bytes
// and the sum of squares takes three shuffles.  A warp takes kHeads heads of one row, four at a time, with the row's cosines and sines in
// registers; all its loads are issued before the first is used.  Everything is binary32 and rounded once.
// Bound by memory: 11996 rows of 32 heads, fp32, 64.4 us, 6,210 GB/s (91 % of the copy rate); 694 rows of 40 heads, bf16, 9 us in a graph (13 MB).
#include <cmath>

#include "decode_kernel.cuh"
#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 256;
constexpr int kRounds = 2;           // heads that a group of eight lanes takes
constexpr int kHeads = 4 * kRounds;  // of a warp's item

struct RopeArgs {
  const void* x[2];  // queries, keys
  void* y[2];
  long long x_stride[2], y_stride[2];
  int heads[2], items[2];  // heads, and items of a row
  const float* weight[2];
  float eps;
  const int32_t* positions;
  const float* cos_sin;
  int max_position;
  const int32_t* run_starts;
  int batch, num_rows;
  int32_t* err;
};

// Eight channels as loaded.
template <bool BF16>
struct Raw {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = *reinterpret_cast<const uint4*>(p + 16 * i);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if (BF16) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = w[BF16 ? 0 : i];
        x[4 * i] = __uint_as_float(v.x); x[4 * i + 1] = __uint_as_float(v.y);
        x[4 * i + 2] = __uint_as_float(v.z); x[4 * i + 3] = __uint_as_float(v.w);
      }
    }
  }
};
template <bool BF16>
__device__ __forceinline__ void store8(uint8_t* p, const float (&x)[8]) {
  if (BF16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(dec::pack_bf16(x[0], x[1]), dec::pack_bf16(x[2], x[3]), dec::pack_bf16(x[4], x[5]), dec::pack_bf16(x[6], x[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// Sum over the eight lanes of a head of the squares times f^2.
__device__ __forceinline__ float squares(const float (&a)[8], const float (&b)[8], float f) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(a[e] * f, a[e] * f, fmaf(b[e] * f, b[e] * f, s));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int per_row = a.items[0] + a.items[1];
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long row = item / per_row;
  if (row >= a.num_rows) return;
  int used = a.num_rows;
  const int pos = a.positions[row];
  if (a.run_starts) used = a.run_starts[a.batch];
  int part = static_cast<int>(item - row * per_row);
  if (used < 0 || used > a.num_rows) {
    if (item == 0 && lane == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  if (row >= used) return;
  if (pos < 0 || pos >= a.max_position) {
    if (part == 0 && lane == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  const int which = part >= a.items[0];
  if (which) part -= a.items[0];
  constexpr int kSize = BF16 ? 2 : 4;
  const int h0 = part * kHeads + (lane >> 3);
  const uint8_t* x = static_cast<const uint8_t*>(a.x[which]) + row * a.x_stride[which] * kSize;
  Raw<BF16> lo[kRounds], hi[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    if (h0 + 4 * i < a.heads[which]) {
      const uint8_t* p = x + ((h0 + 4 * i) * kHeadDim + 8 * l) * kSize;
      lo[i].load(p);
      hi[i].load(p + 64 * kSize);
    }
  float c[8], s[8];
  const float* cs = a.cos_sin + static_cast<long long>(pos) * kHeadDim + 8 * l;
  load8(cs, c);
  load8(cs + 64, s);
  const float* weight = a.weight[which];
  uint8_t* y = static_cast<uint8_t*>(a.y[which]) + row * a.y_stride[which] * kSize;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const bool real = h0 + 4 * i < a.heads[which];
    float u[8] = {}, v[8] = {};
    if (real) {
      lo[i].values(u);
      hi[i].values(v);
    }
    if (weight) {
      float f = 1.f, mean = squares(u, v, 1.f) * (1.f / kHeadDim) + a.eps;
      // squares that leave binary32: once more, of the values times a power of two
      const bool large = !(mean < 1e37f), small = mean < 1e-30f;
      if (__any_sync(0xffffffffu, large || small)) {
        f = large ? 0x1p-70f : small ? 0x1p100f : 1.f;
        mean = squares(u, v, f) * (1.f / kHeadDim) + a.eps * f * f;
      }
      const float inv = rsqrtf(mean);
      float wl[8], wh[8];
      load8(weight + 8 * l, wl);
      load8(weight + 64 + 8 * l, wh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] = u[e] * f * inv * wl[e];
        v[e] = v[e] * f * inv * wh[e];
      }
    }
    if (!real) continue;
    float p[8], q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = fmaf(u[e], c[e], -(v[e] * s[e]));
      q[e] = fmaf(v[e], c[e], u[e] * s[e]);
    }
    uint8_t* dst = y + ((h0 + 4 * i) * kHeadDim + 8 * l) * kSize;
    store8<BF16>(dst, p);
    store8<BF16>(dst + 64 * kSize, q);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_rope_runs(const void* q, int64_t q_row_stride, int32_t num_q_heads, const void* k, int64_t k_row_stride,
                                    int32_t num_kv_heads, int32_t dtype, const float* q_weight, const float* k_weight, float eps,
                                    const int32_t* positions, const float* cos_sin, int32_t max_position, void* q_out,
                                    int64_t q_out_row_stride, void* k_out, int64_t k_out_row_stride, const int32_t* run_starts,
                                    int32_t batch, int32_t num_rows, int32_t* err_word, kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::runs;
  if (dtype != KVQ_DTYPE_F32 && dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads < 0 || num_kv_heads < 0 || num_q_heads > KVQ_MAX_KV_HEADS * KVQ_MAX_GROUP || num_kv_heads > KVQ_MAX_KV_HEADS)
    return KVQ_ERR_INVALID_ARG;
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_position < 0 || !std::isfinite(eps) || eps < 0.f) return KVQ_ERR_INVALID_ARG;
  if ((q != nullptr) != (num_q_heads > 0) || (k != nullptr) != (num_kv_heads > 0)) {
    if (num_rows > 0) return KVQ_ERR_INVALID_ARG;
  }
  if (num_rows == 0 || num_q_heads + num_kv_heads == 0) return KVQ_OK;
  if (!positions || !cos_sin || !aligned16(cos_sin)) return KVQ_ERR_INVALID_ARG;
  RopeArgs a{{q, k}, {q_out, k_out}, {q_row_stride, k_row_stride}, {q_out_row_stride, k_out_row_stride}, {num_q_heads, num_kv_heads}, {0, 0},
             {q_weight, k_weight}, eps, positions, cos_sin, max_position, run_starts, batch, num_rows, err_word};
  const int64_t unit = dtype == KVQ_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
  for (int i = 0; i < 2; ++i) {
    if (a.heads[i] == 0) continue;
    const int64_t width = static_cast<int64_t>(a.heads[i]) * kHeadDim;
    if (!a.y[i] || !aligned16(a.x[i]) || !aligned16(a.y[i]) || !aligned16(a.weight[i])) return KVQ_ERR_INVALID_ARG;
    if (a.x_stride[i] < width || a.x_stride[i] % unit || a.y_stride[i] < width || a.y_stride[i] % unit) return KVQ_ERR_INVALID_ARG;
    if (a.x[i] == a.y[i] && a.x_stride[i] != a.y_stride[i] && num_rows > 1) return KVQ_ERR_INVALID_ARG;
    a.items[i] = (a.heads[i] + kHeads - 1) / kHeads;
  }
  const long long items = static_cast<long long>(num_rows) * (a.items[0] + a.items[1]);
  const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFF) return KVQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_DTYPE_BF16) rope_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  else rope_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
