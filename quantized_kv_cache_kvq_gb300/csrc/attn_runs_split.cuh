// attn_runs_split.cuh -- the split kernel of kvq_attn_runs (short runs: single-token decode, drafts) and of kvq_attn_tree, its
// merge and their launch.
//
// Split kernel.  A unit is one (request, kv head, tile of up to 8 NT rows), a row being a (query token, query head of the
// group) pair; its pages are those of the request.  All units' pages are laid end to end and cut into equal contiguous
// ranges, one per warp of a persistent grid, as in the single-token decode of the other layouts: pages stream through a
// ring of bulk copies per warp, the page's 16 tokens are the M dimension of every tensor-core product (mma.sync: a page gives
// each row 2 x 2048 multiply-adds for 4096 bytes, far below where the tensor rate matters), and the pieces are merged
// with log-sum-exp weights.  Bound by HBM: 4,100 bytes a page and kv head.  64 requests of 32768 tokens, 4 kv and 28 query heads,
// INT8: 345 us, 6,240 GB/s (92 % of the copy rate); 128 of 1024..16384, 8 and 32 heads, E4M3: 262 us, 6,010 GB/s; 16 drafts of
// 2..4 tokens over 11000..11996, two row blocks a page: 79 us, 4,790 GB/s (dependent products that 12 warps do not hide).
#pragma once

#include <algorithm>

#include "attn_runs.cuh"

namespace kvq {
namespace runs {

using dec::bulk_g2s_hint;
using dec::col_max8;
using dec::col_sum8;
using dec::ex2;
using dec::kFull;
using dec::lds128;
using dec::mbar_arrive;
using dec::mbar_arrive_expect_tx;
using dec::mbar_wait;
using dec::mma_f16_4;
using dec::movmatrix_trans;
using dec::pack_f16;
using dec::unpack_f16;

namespace {

constexpr int kStageBytes = 4096;
constexpr int kMaxStages = 8;
constexpr int kMergeWarps = 16;  // of a block; with 8 the three calls at the merge kernel take 19, 35 and 55 us
constexpr int kSmemStatic = 2048;  // of shared memory, left for what the kernel declares statically
constexpr int kMinPages = 2;  // pages a warp, so that short contexts leave the merge fewer pieces

// Page descriptors, one per lane for 32 pages ahead.
struct Desc {
  int32_t phys;    // -1: nothing to read (past the tile's last visible token, or reported as out of range)
  int32_t page;    // page index in the request
  int32_t unit;    // global unit index
  uint16_t ks, vs;  // the page's scales as stored
};

struct Unit {
  int seq, kvh, tile;
};

// q as B fragments: b0, b1 of k-step kb hold channels 64 (kb >> 2) + 16 c + 4 (kb & 3) + {0, 1} and {2, 3} of row g.
template <int NT>
struct Query {
  uint32_t hi[NT][8][2];
  float scale[NT][2];  // rows 2c, 2c + 1: sm_scale log2 e 2^er (the row was multiplied by 2^-er)
  int limit[NT][2];    // tokens t < limit are visible to rows 2c, 2c + 1; a tree's: the rows of the mask, -1 for none
  int min_limit;       // over the tile's rows: tokens before it are visible to all
  int end;             // a tree's: the context's length
};

template <int NT>
struct State {
  float o[NT][8][4];
  float m[NT][2], l[NT][2];
};

template <int NT>
__device__ __forceinline__ void reset(State<NT>& s) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s.o[n][i][0] = s.o[n][i][1] = s.o[n][i][2] = s.o[n][i][3] = 0.f;
    s.m[n][0] = s.m[n][1] = -INFINITY;
    s.l[n][0] = s.l[n][1] = 0.f;
  }
}

// Rows of a run that this kernel takes, as tiles of 8 NT rows.
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Run& r, int rows_per_tile) {
  const long long rows = static_cast<long long>(r.n) * a.G;
  return rows > a.few_rows ? 0 : static_cast<int>((rows + rows_per_tile - 1) / rows_per_tile);
}

template <int NT, bool F32, bool TREE>
__device__ void load_q(const AttnArgs& a, const Unit& u, Query<NT>& f, uint32_t* lo) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const Run run = load_run(a.run_starts, a.seq_lens, u.seq, a.num_rows, a.max_run, a.max_pages);
  const int rows = run.n * a.G;
  int min_limit = 0x7FFFFFFF;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = (u.tile * NT + n) * 8 + g;
    const bool real = r < rows;
    const int tok = real ? r / a.G : 0, head = real ? r % a.G : 0;
    const int limit = TREE ? (real ? run.row0 + tok : -1) : real ? run.len - run.n + tok + 1 : 0;
    if (real) min_limit = min(min_limit, TREE ? run.len - run.n : limit);
    float x[32];  // channels 64 jj + 16 c + i
    float amax = 0.f;
    const long long at = static_cast<long long>(run.row0 + tok) * a.q_stride + (u.kvh * a.G + head) * kHeadDim + 16 * c;
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
      for (int e = 0; e < 16; e += F32 ? 4 : 8) {
        if (!real) {
#pragma unroll
          for (int i = 0; i < (F32 ? 4 : 8); ++i) x[16 * jj + e + i] = 0.f;
        } else if (F32) {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + 64 * jj + e);
          x[16 * jj + e] = w.x; x[16 * jj + e + 1] = w.y; x[16 * jj + e + 2] = w.z; x[16 * jj + e + 3] = w.w;
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + 64 * jj + e);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[16 * jj + e + 2 * i] = __uint_as_float(ws[i] << 16);
            x[16 * jj + e + 2 * i + 1] = __uint_as_float(ws[i] & 0xFFFF0000u);
          }
        }
      }
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // the row times 2^-er, largest element in [2^8, 2^9): bf16 elements are then exact in fp16 down to 2^-22 of it
    int er = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 8;
    er = min(max(er, -100), 120);
    const float f0 = exp2_int(-er);
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 16 * (kb >> 2) + 4 * (kb & 3) + 2 * h;
        const float x0 = x[i] * f0, x1 = x[i + 1] * f0;
        const uint32_t hi = pack_f16(x0, x1);
        f.hi[n][kb][h] = hi;
        if (F32) {  // what fp16 leaves out, in a second product: 22 bits of the query
          const float2 r2 = unpack_f16(hi);
          lo[((n * 8 + kb) * 2 + h) * 32 + lane] = pack_f16(x0 - r2.x, x1 - r2.y);
        }
      }
    const float sc = a.sm_scale * dec::kLog2e * exp2_int(er);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f.scale[n][h] = __shfl_sync(kFull, sc, 4 * (2 * c + h));
      f.limit[n][h] = __shfl_sync(kFull, limit, 4 * (2 * c + h));
    }
  }
  f.min_limit = __reduce_min_sync(kFull, min_limit);
  if (TREE) f.end = run.len;
  if (F32) __syncwarp();
}

// Weights are multiplied by 2^kShift before they are rounded to fp16, whose normal range then reaches down to 2^-(14 + kShift)
// of the largest; numerator and denominator carry the same factor.  The running maximum moves only when a logit exceeds it by
// kSlack, so that most pages need no rescaling; the largest weight is then 2^(kShift + kSlack) < 65504.
template <bool F32>
struct Weight {
  static constexpr float kShift = F32 ? 12.f : 8.f, kSlack = F32 ? 3.f : 7.f;
};

// What a mask row of a tree says about the page at p0, whose run begins at `ctx`: bit t for its token t.  Tokens before the run are
// seen, tokens behind the context are not.
__device__ __forceinline__ uint32_t page_bits(const AttnArgs& a, int row, int p0, int ctx, int end) {
  if (row < 0) return 0;
  const int32_t* words = a.mask + static_cast<long long>(row) * a.mask_words;
  const int j = p0 - ctx, w = j >> 5;  // -1: before the run
  const uint32_t lo = w < 0 ? 0xFFFFFFFFu : w < a.mask_words ? static_cast<uint32_t>(words[w]) : 0u;
  const uint32_t hi = w + 1 < a.mask_words ? static_cast<uint32_t>(words[w + 1]) : 0u;
  return __funnelshift_r(lo, hi, j & 31) & ((1u << min(end - p0, kPage)) - 1);
}

// One page: st holds its key tile and its value tile.
template <bool INT8, int NT, bool F32, bool TREE>
__device__ __forceinline__ void process(const AttnArgs& a, const uint8_t* st, const Query<NT>& f, const uint32_t* lo, State<NT>& s,
                                        int p0, uint32_t scale) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  float S[NT][4] = {};
#pragma unroll
  for (int jj = 0; jj < 2; ++jj) {
    const uint4 k0 = lds128(st + (jj * 32 + lane) * 16), k1 = lds128(st + ((2 + jj) * 32 + lane) * 16);
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = codes_lo<INT8>(w0[i]), a1 = codes_lo<INT8>(w1[i]);
      const uint32_t a2 = codes_hi<INT8>(w0[i]), a3 = codes_hi<INT8>(w1[i]);
      const int kb = 4 * jj + i;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16_4(S[n], a0, a1, a2, a3, f.hi[n][kb][0], f.hi[n][kb][1]);
        if (F32) mma_f16_4(S[n], a0, a1, a2, a3, lo[((n * 8 + kb) * 2) * 32 + lane], lo[((n * 8 + kb) * 2 + 1) * 32 + lane]);
      }
    }
  }
  const float ks = exp2_int(static_cast<int>(scale & 0xFFu) - 32);
  const int evi = static_cast<int>((scale >> 8) & 0xFFu) - 32;
  const float ev = static_cast<float>(evi), unscale = exp2_int(-evi);
  const bool masked = p0 + kPage > f.min_limit;
  uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float y[4];  // tokens g (0, 1) and g + 8 (2, 3), rows 2c, 2c + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fmaf(S[n][i], f.scale[n][i & 1] * ks, ev);
    if (masked) {
      uint32_t bits[2];
      if (TREE) {
#pragma unroll
        for (int h = 0; h < 2; ++h) bits[h] = page_bits(a, f.limit[n][h], p0, f.min_limit, f.end);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (TREE ? !(bits[i & 1] >> (g + 8 * (i >> 1)) & 1u) : p0 + g + 8 * (i >> 1) >= f.limit[n][i & 1]) y[i] = -INFINITY;
    }
    if (__any_sync(kFull, fmaxf(y[0], y[2]) > s.m[n][0] + Weight<F32>::kSlack || fmaxf(y[1], y[3]) > s.m[n][1] + Weight<F32>::kSlack)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = fmaxf(s.m[n][h], col_max8(fmaxf(y[h], y[2 + h])));
        const float alpha = s.m[n][h] == -INFINITY ? 0.f : ex2(s.m[n][h] - mn);
        s.m[n][h] = mn;
        s.l[n][h] *= alpha;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          s.o[n][mt][h] *= alpha;
          s.o[n][mt][2 + h] *= alpha;
        }
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = s.m[n][i & 1];
      p[i] = ex2(y[i] - (m == -INFINITY ? 0.f : m) + Weight<F32>::kShift);
    }
    s.l[n][0] = fmaf(p[0] + p[2], unscale, s.l[n][0]);
    s.l[n][1] = fmaf(p[1] + p[3], unscale, s.l[n][1]);
    const uint32_t h01 = pack_f16(p[0], p[1]), h23 = pack_f16(p[2], p[3]);
    bh[n][0] = movmatrix_trans(h01);
    bh[n][1] = movmatrix_trans(h23);
    if (F32) {
      const float2 r01 = unpack_f16(h01), r23 = unpack_f16(h23);
      bl[n][0] = movmatrix_trans(pack_f16(p[0] - r01.x, p[1] - r01.y));
      bl[n][1] = movmatrix_trans(pack_f16(p[2] - r23.x, p[3] - r23.y));
    }
  }
#pragma unroll
  for (int mm = 0; mm < 4; ++mm) {
    const uint4 vb = lds128(st + 2048 + (mm * 32 + lane) * 16);
    const uint32_t w[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t a0 = codes_lo<INT8>(w[2 * half]), a1 = codes_hi<INT8>(w[2 * half]);
      const uint32_t a2 = codes_lo<INT8>(w[2 * half + 1]), a3 = codes_hi<INT8>(w[2 * half + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16_4(s.o[n][2 * mm + half], a0, a1, a2, a3, bh[n][0], bh[n][1]);
        if (F32) mma_f16_4(s.o[n][2 * mm + half], a0, a1, a2, a3, bl[n][0], bl[n][1]);
      }
    }
  }
}

// E4M3 only: the value codes of tokens that no row sees become 0, since a NaN byte there would survive a zero weight.
__device__ __forceinline__ void zero_value_tail(uint8_t* v, int nvalid) {
  const int lane = threadIdx.x & 31;
  for (int e = lane; e < (kPage - nvalid) * kHeadDim; e += 32) v[v8_offset(nvalid + e / kHeadDim, e % kHeadDim)] = 0;
  __syncwarp();
}

template <int NT>
__device__ __forceinline__ void write_piece(const AttnArgs& a, long long slot, const State<NT>& s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long row = slot * (8 * NT) + 8 * n + 2 * c + h;
      const float l = col_sum8(s.l[n][h]);
      float* acc = a.ws_acc + row * kHeadDim;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        acc[16 * mt + g] = s.o[n][mt][h];
        acc[16 * mt + g + 8] = s.o[n][mt][2 + h];
      }
      if (g == 0) *reinterpret_cast<float2*>(a.ws_stats + row * 2) = make_float2(s.m[n][h], l);
    }
}

template <bool INT8, int NT, bool F32, int NW, bool TREE>
__global__ void __launch_bounds__(NW * 32, 1) split_kernel(const AttnArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long* cum = reinterpret_cast<long long*>(smem);  // pages of all tiles (one kv head) of the requests before
  const int cum_bytes = ((a.batch + 1) * 12 + 127) & ~127;
  int* cumt = reinterpret_cast<int*>(smem + (a.batch + 1) * 8);  // row tiles of the requests before
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long all_tiles = 0;  // runs that overlap, against the rules, may have more than 32 bits count
  {
    __shared__ long long w_pages[NW], w_tiles[NW];
    const int per = (a.batch + blockDim.x - 1) / blockDim.x;
    const int s0 = threadIdx.x * per;
    long long lp = 0, lt = 0;
    for (int i = 0; i < per; ++i) {
      const int s = s0 + i;
      if (s < a.batch) {
        const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.max_run, a.max_pages);
        if (r.row0 < 0 && blockIdx.x == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
        const int t = tiles_of(a, r, 8 * NT);
        const long long p = static_cast<long long>(t) * ((r.len + kPage - 1) / kPage);
        cum[s + 1] = p;
        cumt[s + 1] = t;
        lp += p;
        lt += t;
      }
    }
    long long ip = lp, it = lt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long tp = __shfl_up_sync(kFull, ip, o);
      const long long tt = __shfl_up_sync(kFull, it, o);
      if (lane >= o) { ip += tp; it += tt; }
    }
    if (lane == 31) { w_pages[warp] = ip; w_tiles[warp] = it; }
    __syncthreads();
    long long rp = ip - lp, rt = it - lt;
    for (int w = 0; w < warp; ++w) { rp += w_pages[w]; rt += w_tiles[w]; }
    for (int w = 0; w < NW; ++w) all_tiles += w_tiles[w];
    for (int i = 0; i < per; ++i) {
      const int s = s0 + i;
      if (s < a.batch) {
        cum[s + 1] = rp += cum[s + 1];
        rt += cumt[s + 1];
        cumt[s + 1] = static_cast<int>(rt);
      }
    }
    if (threadIdx.x == 0) {
      cum[0] = 0;
      cumt[0] = 0;
    }
    __syncthreads();
  }
  if (all_tiles > a.max_tiles) {  // runs that overlap: more tiles than the rows can make
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      *a.ws_units = 0;  // nothing for the merge
    }
    return;
  }
  const long long T = a.Hkv * cum[a.batch];
  const long long W = min(static_cast<long long>(a.w_max), (T + kMinPages - 1) / kMinPages);
  // What the merge needs to know of each unit: it then starts with one load.
  const int n_units = a.Hkv * cumt[a.batch];
  auto write_records = [&]() {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ws_units = n_units;
    for (int u = blockIdx.x * blockDim.x + threadIdx.x; u < n_units; u += gridDim.x * blockDim.x) {
      int lo_s = 0, hi_s = a.batch - 1;  // first s with Hkv cumt[s + 1] > u
      while (lo_s < hi_s) {
        const int mid = (lo_s + hi_s) >> 1;
        if (a.Hkv * cumt[mid + 1] > u) hi_s = mid; else lo_s = mid + 1;
      }
      const Run r = load_run(a.run_starts, a.seq_lens, lo_s, a.num_rows, a.max_run, a.max_pages);
      const int tiles = cumt[lo_s + 1] - cumt[lo_s], local = u - a.Hkv * cumt[lo_s], kvh = local / tiles, tile = local - kvh * tiles;
      const int P = (r.len + kPage - 1) / kPage;
      UnitRecord rec{r.row0, r.n * a.G - tile * 8 * NT, tile * 8 * NT, kvh, 0, 0};
      if (P > 0) {
        const long long b = a.Hkv * cum[lo_s] + static_cast<long long>(local) * P;
        // warp w covers pages [T w / W, T (w + 1) / W): the warp that holds page x
        auto warp_of = [&](long long x) {
          long long w = x * W / T;
          while (w + 1 < W && T * (w + 1) / W <= x) ++w;
          while (w > 0 && T * w / W > x) --w;
          return static_cast<int>(w);
        };
        rec.w0 = warp_of(b);
        rec.pieces = warp_of(b + P - 1) - rec.w0 + 1;
      }
      a.ws_rec[u] = rec;
    }
  };
  const long long wid = static_cast<long long>(blockIdx.x) * a.nwa + warp;
  if (warp >= a.nwa || wid >= W) return write_records();
  const long long x_begin = T * wid / W, x_end = T * (wid + 1) / W;
  const long long n = x_end - x_begin;

  constexpr int kLoBytes = F32 ? NT * 8 * 2 * 32 * 4 : 0;
  uint8_t* wbase = smem + cum_bytes + warp * (a.stages * kStageBytes + kLoBytes + kMaxStages * 8);
  uint32_t* lo = reinterpret_cast<uint32_t*>(wbase + a.stages * kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(wbase + a.stages * kStageBytes + kLoBytes);
  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) dec::mbar_init(&bars[i], 1);
    dec::fence_mbar_init();
  }
  __syncwarp();

  auto make_desc = [&](long long x) {
    Desc d{-1, 0, 0, 0, 0};
    if (x >= x_end) return d;
    int lo_s = 0, hi_s = a.batch - 1;  // first s with Hkv cum[s + 1] > x
    while (lo_s < hi_s) {
      const int mid = (lo_s + hi_s) >> 1;
      if (a.Hkv * cum[mid + 1] > x) hi_s = mid; else lo_s = mid + 1;
    }
    const int s = lo_s;
    const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.max_run, a.max_pages);
    const int P = (r.len + kPage - 1) / kPage, tiles = cumt[s + 1] - cumt[s];
    const long long rem = x - a.Hkv * cum[s];
    const int local = static_cast<int>(rem / P);  // kvh * tiles + tile
    d.page = static_cast<int>(rem - static_cast<long long>(local) * P);
    d.unit = a.Hkv * cumt[s] + local;
    const int kvh = local / tiles, tile = local - kvh * tiles;
    const int last_row = min((tile + 1) * 8 * NT, r.n * a.G) - 1;
    const int limit = TREE ? r.len : r.len - r.n + last_row / a.G + 1;
    if (d.page * kPage >= limit) return d;  // no row of the tile sees this page
    const int phys = a.block_table[static_cast<size_t>(s) * a.max_pages + d.page];
    if (phys < 0 || phys >= a.num_pages) {
      report(a.err, KVQ_ERR_DEVICE_BOUNDS);
      return d;
    }
    d.phys = phys;
    const size_t si = static_cast<size_t>(kvh) * a.num_pages + phys;
    d.ks = a.ks[si];
    d.vs = a.vs[si];
    return d;
  };
  auto unit_of = [&](int unit) {
    int lo_s = 0, hi_s = a.batch - 1;  // first s with Hkv cumt[s + 1] > unit
    while (lo_s < hi_s) {
      const int mid = (lo_s + hi_s) >> 1;
      if (a.Hkv * cumt[mid + 1] > unit) hi_s = mid; else lo_s = mid + 1;
    }
    const int tiles = cumt[lo_s + 1] - cumt[lo_s], local = unit - a.Hkv * cumt[lo_s];
    return Unit{lo_s, local / tiles, local % tiles};
  };
  const uint64_t pol = dec::stream_policy(false);
  auto issue = [&](int st, int phys, int kvh, uint32_t leader) {
    if (phys < 0) {
      mbar_arrive(&bars[st], leader);
      return;
    }
    const size_t tile = (static_cast<size_t>(phys) * a.Hkv + kvh) * 2048;
    uint8_t* dst = wbase + st * kStageBytes;
    mbar_arrive_expect_tx(&bars[st], kStageBytes, leader);
    bulk_g2s_hint(dst, a.k + tile, 2048, &bars[st], pol, leader);
    bulk_g2s_hint(dst + 2048, a.v + tile, 2048, &bars[st], pol, leader);
  };
  auto kvh_of = [&](int unit) { return unit_of(unit).kvh; };
  // exponents + 32 of a descriptor's scales (bits 0..7 key, 8..15 value); apart from the descriptor, so that nothing waits
  // for the loads before they are needed
  auto exponents = [](const Desc& d) {
    return static_cast<uint32_t>(f16_to_exp(d.ks) + 32) | static_cast<uint32_t>(f16_to_exp(d.vs) + 32) << 8;
  };

  Desc cur = make_desc(x_begin + lane);
  int cur_kvh = cur.phys >= 0 ? kvh_of(cur.unit) : 0;
  for (int j = 0; j < a.stages && j < n; ++j)
    issue(j, __shfl_sync(kFull, cur.phys, j), __shfl_sync(kFull, cur_kvh, j), dec::elect_one());
  write_records();
  Desc nxt = make_desc(x_begin + 32 + lane);
  int nxt_kvh = nxt.phys >= 0 ? kvh_of(nxt.unit) : 0;
  uint32_t cur_scale = exponents(cur);

  Query<NT> f;
  State<NT> s;
  reset(s);
  int unit = -1;
  int limit_max = 0;
  int stage = 0;
  uint32_t parity = 0;
  bool ok = true;
  long long stopped = 0;
  for (long long j = 0; j < n; ++j) {
    const int jl = static_cast<int>(j & 31);
    if (j > 0 && jl == 0) {
      cur = nxt;
      cur_kvh = nxt_kvh;
      cur_scale = exponents(cur);
      nxt = make_desc(x_begin + j + 32 + lane);
      nxt_kvh = nxt.phys >= 0 ? kvh_of(nxt.unit) : 0;
    }
    const int phys = __shfl_sync(kFull, cur.phys, jl), page = __shfl_sync(kFull, cur.page, jl);
    const int u = __shfl_sync(kFull, cur.unit, jl);
    const uint32_t scale = __shfl_sync(kFull, cur_scale, jl);
    if (u != unit) {
      if (unit >= 0) { write_piece(a, wid + unit, s); reset(s); }
      unit = u;
      const Unit uu = unit_of(u);
      load_q<NT, F32, TREE>(a, uu, f, lo);
      int lm = TREE ? f.end : 0;
      if (!TREE) {
#pragma unroll
        for (int t = 0; t < NT; ++t) lm = max(lm, max(f.limit[t][0], f.limit[t][1]));
        lm = __reduce_max_sync(kFull, lm);
      }
      limit_max = lm;
    }
    if (!__all_sync(kFull, mbar_wait(&bars[stage], parity))) { ok = false; stopped = j; break; }
    uint8_t* st = wbase + stage * kStageBytes;
    if (phys >= 0) {
      if (!INT8 && (page + 1) * kPage > limit_max) zero_value_tail(st + 2048, limit_max - page * kPage);
      process<INT8, NT, F32, TREE>(a, st, f, lo, s, page * kPage, scale);
    }
    __syncwarp();
    const long long jn = j + a.stages;
    if (jn < n) {
      const bool in_cur = (jn >> 5) == (j >> 5);
      const int l = static_cast<int>(jn & 31);
      const int pc = __shfl_sync(kFull, cur.phys, l), pn = __shfl_sync(kFull, nxt.phys, l);
      const int kc = __shfl_sync(kFull, cur_kvh, l), kn = __shfl_sync(kFull, nxt_kvh, l);
      dec::fence_proxy_async();
      issue(stage, in_cur ? pc : pn, in_cur ? kc : kn, dec::elect_one());
    }
    if (++stage == a.stages) { stage = 0; parity ^= 1u; }
  }
  if (!ok) {
    if (lane == 0) report(a.err, KVQ_ERR_TIMEOUT);
    // no copy may land after the warp has gone: wait (bounded) for those in flight
    for (long long k = stopped; k < n && k < stopped + a.stages; ++k)
      (void)mbar_wait(&bars[k % a.stages], static_cast<uint32_t>((k / a.stages) & 1));
    return;
  }
  if (unit >= 0) write_piece(a, wid + unit, s);
}

// The pieces of a row under log-sum-exp weights.  The unit's record, then everything it points to in one round of loads; what
// it costs is the latency of those two (a first version looked the row up from the lengths: 8.5 us alone on 64 requests of 28
// heads).  One warp to a row, or, where the grid has a block for every row (few requests, whose contexts are then cut into
// hundreds of pieces), a block: its warps take the pieces in turn.  The whole call for 2 requests of up to 16723 tokens, 2 kv and 6
// query heads: 146 us with a warp to a row, 17 with a block; one of 120000, one head: 622 and 31; 8 and 32 heads: 135 and 54.
template <int NT, bool F32>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const AttnArgs a) {
  constexpr int kU = 16, kRows = 8 * NT;
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ __align__(16) float s_acc[kMergeWarps][kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_units = *a.ws_units;
  long long gw = static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
  UnitRecord rec = a.ws_rec[min(gw / kRows, static_cast<long long>(a.max_tiles) * a.Hkv - 1)];
  const bool wide = static_cast<long long>(n_units) * kRows <= gridDim.x;
  if (wide) gw = blockIdx.x;
  const long long unit = gw / kRows;
  const int r = static_cast<int>(gw % kRows);
  if (unit >= n_units) return;
  if (wide) rec = a.ws_rec[unit];
  if (r >= rec.rows) return;
  const bool split = wide && rec.pieces > kU;  // the same in all warps of a block
  if (wide && !split && warp > 0) return;
  // this warp's pieces: 8 NT rows of the workspace apart, or kMergeWarps times that
  const long long first = (rec.w0 + unit) * kRows + r + (split ? warp * kRows : 0);
  const long long step = split ? kMergeWarps * kRows : kRows;
  const int pieces = split ? (rec.pieces - warp + kMergeWarps - 1) / kMergeWarps : rec.pieces;
  const float* stats = a.ws_stats + first * 2;
  const float* accs = a.ws_acc + first * kHeadDim + 4 * lane;
  auto acc_of = [&](int k) { return *reinterpret_cast<const float4*>(accs + k * step * kHeadDim); };
  auto stats_of = [&](int k) { return *reinterpret_cast<const float2*>(stats + k * step * 2); };
  float4 v[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k)
    if (k < pieces) v[k] = acc_of(k);
  float m = -INFINITY, l = 0.f, m_mine = -INFINITY;  // m_mine: of piece `lane`
  bool nan = false;  // of a query that is not finite
  for (int i = lane; i < pieces; i += 32) {
    const float2 st = stats_of(i);
    if (i < 32) m_mine = st.x;
    const float mm = fmaxf(m, st.x);
    nan |= st.y != st.y;
    if (mm != -INFINITY) {
      l = (m == -INFINITY ? 0.f : l * ex2(m - mm)) + (st.x == -INFINITY ? 0.f : st.y * ex2(st.x - mm));
      m = mm;
    }
  }
  float gm = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(kFull, gm, o));
  l = m == -INFINITY ? 0.f : l * ex2(m - gm);
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
  m = gm;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wt_mine = m_mine == -INFINITY ? 0.f : ex2(m_mine - m);  // of piece k0 + lane, k0 a multiple of 32
#pragma unroll 1
  for (int k0 = 0; k0 < pieces; k0 += kU) {
    if (k0 > 0) {
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (k0 + k < pieces) v[k] = acc_of(k0 + k);
      if (k0 % 32 == 0) {
        const float mi = k0 + lane < pieces ? stats_of(k0 + lane).x : -INFINITY;
        wt_mine = mi == -INFINITY ? 0.f : ex2(mi - m);
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const float wt = __shfl_sync(kFull, wt_mine, (k0 & 16) + k);
      if (k0 + k < pieces && wt != 0.f) {
        acc.x += v[k].x * wt; acc.y += v[k].y * wt; acc.z += v[k].z * wt; acc.w += v[k].w * wt;
      }
    }
  }
  if (__any_sync(kFull, nan)) l = NAN;
  if (split) {
    *reinterpret_cast<float4*>(&s_acc[warp][4 * lane]) = acc;
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    __syncthreads();
    if (warp > 0) return;
    const float mk = lane < kMergeWarps ? s_m[lane] : -INFINITY, lk = lane < kMergeWarps ? s_l[lane] : 0.f;
    m = mk;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float wk = mk == -INFINITY ? 0.f : ex2(mk - m);
    l = wk == 0.f ? 0.f : lk * wk;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    if (__any_sync(kFull, lk != lk)) l = NAN;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) {
      const float wt = __shfl_sync(kFull, wk, k);
      const float4 x = *reinterpret_cast<const float4*>(&s_acc[k][4 * lane]);
      if (wt != 0.f) { acc.x += x.x * wt; acc.y += x.y * wt; acc.z += x.z * wt; acc.w += x.w * wt; }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is 0
  const int in_run = rec.row_in_run + r;
  const long long row = static_cast<long long>(rec.row0 + in_run / a.G) * a.Hq + rec.kvh * a.G + in_run % a.G;
  const long long at = row * kHeadDim + 4 * lane;
  if (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(dec::pack_bf16(acc.x * inv, acc.y * inv), dec::pack_bf16(acc.z * inv, acc.w * inv));
  }
  if (a.lse && lane == 0)
    a.lse[row] = l == 0.f ? -INFINITY : (m + (log2f(l) - Weight<F32>::kShift)) * dec::kLn2;
}

// ------------------------------------------------------------------------------------------------ launch
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kSplitWarps = 16;  // the most that any variant uses (sizes the workspace)

// Row tiles of 8 when no run has more rows, of 16 otherwise.
int row_blocks(long long max_rows) { return max_rows <= 8 ? 1 : 2; }

// The split kernel's part of a workspace, for at most `tiles` row tiles of 8 nt rows.
struct SplitWorkspace {
  size_t units, rec, stats, acc, total;
  long long tiles;
  void put(AttnArgs& a, uint8_t* ws) const {
    a.max_tiles = static_cast<int>(std::min<long long>(tiles, 0x7FFFFFFF));
    a.ws_units = reinterpret_cast<int*>(ws + units);
    a.ws_rec = reinterpret_cast<UnitRecord*>(ws + rec);
    a.ws_stats = reinterpret_cast<float*>(ws + stats);
    a.ws_acc = reinterpret_cast<float*>(ws + acc);
  }
};
inline SplitWorkspace split_workspace(size_t tiles, int nt, int hkv, int sms) {
  SplitWorkspace w{};
  w.tiles = static_cast<long long>(tiles);
  const size_t slots = static_cast<size_t>(sms) * kSplitWarps + tiles * hkv;
  w.units = 0;
  w.rec = 256;
  w.stats = w.rec + align256(tiles * hkv * sizeof(UnitRecord));
  w.acc = w.stats + align256(slots * 8 * nt * 2 * sizeof(float));
  w.total = w.acc + align256(slots * 8 * nt * kHeadDim * sizeof(float));
  return w;
}

template <bool INT8, int NT, bool F32, int NW, bool TREE>
cudaError_t launch_split(AttnArgs& a, int sms, int smem_max, cudaStream_t s) {
  constexpr int lo_bytes = F32 ? NT * 8 * 2 * 32 * 4 : 0;
  const int cum_bytes = ((a.batch + 1) * 12 + 127) & ~127;
  a.nwa = NW;
  a.stages = std::min(kMaxStages, (smem_max - kSmemStatic - cum_bytes - NW * (lo_bytes + kMaxStages * 8)) / (NW * kStageBytes));
  a.w_max = sms * NW;
  const size_t smem = cum_bytes + static_cast<size_t>(NW) * (a.stages * kStageBytes + lo_bytes + kMaxStages * 8);
  auto kern = split_kernel<INT8, NT, F32, NW, TREE>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(kern, smem_max - kSmemStatic);
  if (e != cudaSuccess) return e;
  kern<<<sms, NW * 32, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.max_tiles) * a.Hkv * (8 * NT);
  cudaLaunchConfig_t cfg = {};
  // a warp to a row; blocks for as many rows as the SMs hold two of, so that few rows have a block each
  cfg.gridDim = dim3(static_cast<unsigned>(std::max((rows + kMergeWarps - 1) / kMergeWarps, std::min<long long>(rows, 2 * sms))));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<NT, F32>, a);
}

template <bool INT8, bool TREE = false>
cudaError_t launch(AttnArgs& a, bool f32, int nt, int sms, int smem_max, cudaStream_t s) {
  if (nt == 1) return f32 ? launch_split<INT8, 1, true, 12, TREE>(a, sms, smem_max, s) : launch_split<INT8, 1, false, 16, TREE>(a, sms, smem_max, s);
  return f32 ? launch_split<INT8, 2, true, 8, TREE>(a, sms, smem_max, s) : launch_split<INT8, 2, false, 12, TREE>(a, sms, smem_max, s);
}

}  // namespace
}  // namespace runs
}  // namespace kvq
