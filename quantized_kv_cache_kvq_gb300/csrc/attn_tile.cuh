// attn_tile.cuh -- what the tcgen05 kernels of kvq_attn_runs and kvq_attn_tree share: PTX, and the work of a CTA.
//
// A unit is one (request, kv head, S::kRows consecutive (token, head) rows of the run); its key tiles are the 128-token tiles that its
// rows see.  All units' tiles are laid end to end and cut into equal contiguous ranges, one for each CTA.  S: a kernel's rows of a unit, threads, shared
// state (`Tail`: `unit` for each warp, `start`, `n`), and whether runs are trees.
#pragma once

#include "attn_runs.cuh"

namespace kvq {
namespace runs {
namespace {

using dec::ex2;
using dec::smem_u32;

constexpr int kKeys = 128;      // keys of a tile
constexpr int kPagesPerTile = kKeys / kPage;
constexpr float kTileShift = 7.f;  // weights are held times 2^7 ..
constexpr float kSlack = 8.f;      // .. and may grow to 2^15 before the running maximum (and O) is moved
constexpr uint32_t kIdesc = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);  // fp16 x fp16 -> fp32, M = N = 128

struct RunInfo {
  int len, n, row0;
};
struct UnitInfo {
  int s, kvh, u;
  RunInfo run;
};

// A tile is the first, the last of its piece; both halves have rows.
constexpr int kFirst = 1, kLast = 2, kBoth = 4;

// ------------------------------------------------------------------------------------------------ PTX
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  // K-major, 128-byte swizzle: 1024 bytes between groups of 8 rows
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Issued by the whole converged warp with the same operands, predicated on the one lane that elect.sync picked: the operands
// then stay in uniform registers (issued from one lane's branch, every product cost ~97 clocks to set up, 64 to run).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(kIdesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(kIdesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps the uses of loaded values behind the wait: arithmetic is otherwise free to move over a volatile statement.
template <int N>
__device__ __forceinline__ void loaded(float* r) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]), "+f"(r[i + 6]),
                 "+f"(r[i + 7]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]),
        "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(u[0]),
      "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
      "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
      : "memory");
}

// Bounded wait (some seconds of clocks): false when the phase did not complete or another role has given up.
constexpr long long kWaitClocks = 4000000000ll;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort) {
  if (dec::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!dec::mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(abort)) return false;
    if (clock64() - t0 > kWaitClocks) {
      *reinterpret_cast<volatile int*>(abort) = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {  // one verdict for the whole warp
  return __all_sync(dec::kFull, wait(bar, parity, abort));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ------------------------------------------------------------------------------------------------ work
__device__ __forceinline__ RunInfo run_info(const AttnArgs& a, int s) {
  const Run r = load_run(a.run_starts, a.seq_lens, s, a.num_rows, a.max_run, a.max_pages);
  return RunInfo{r.len, r.n, r.row0};
}
template <class S>
__device__ __forceinline__ int units_of(const AttnArgs& a, const RunInfo& r) {
  const int rows = r.n * a.G;
  return rows > a.few_rows ? (rows + S::kRows - 1) / S::kRows : 0;
}
// Key tiles of unit u: up to the last token that its last row sees (a tree's: to the end of the context), one at least (whose columns
// may all be hidden).
template <class S>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const RunInfo& r, int u) {
  const int last = min(r.n - 1, (S::kRows * (u + 1) - 1) / a.G);
  const int limit = S::kTree ? r.len : r.len - r.n + last + 1;
  return max(1, (limit + kKeys - 1) / kKeys);
}

// Halves of 128 rows that a unit has rows in.
template <class S>
__device__ __forceinline__ int halves_of(const AttnArgs& a, const RunInfo& r, int u) {
  return S::kRows > 128 && r.n * a.G - u * S::kRows > 128 ? 2 : 1;
}

// Where a warp is in its CTA's range of tiles.  The unit lives in shared memory: in registers it would be spilled, and
// with 227 KB of shared memory the L1 that is left loses what is spilled to the L2 (~500 clocks a use).
template <class S>
__device__ __forceinline__ int set_unit(const AttnArgs& a, UnitInfo* at, int s, int kvh, int u) {
  const RunInfo r = run_info(a, s);
  const UnitInfo i{s, kvh, u, r};
  __syncwarp();
  *at = i;  // every lane the same
  __syncwarp();
  return tiles_of<S>(a, r, u) << 1 | (halves_of<S>(a, r, u) - 1);
}
template <class S>
__device__ __forceinline__ int next_unit(const AttnArgs& a, UnitInfo* at) {
  UnitInfo i = *at;
  if (++i.u == units_of<S>(a, i.run)) {
    i.u = 0;
    if (++i.kvh == a.Hkv) {
      i.kvh = 0;
      do i.run = run_info(a, ++i.s); while (units_of<S>(a, i.run) == 0);  // called only where a later unit exists
    }
  }
  __syncwarp();
  *at = i;
  __syncwarp();
  return tiles_of<S>(a, i.run, i.u) << 1 | (halves_of<S>(a, i.run, i.u) - 1);
}
template <class S>
struct Cursor {
  UnitInfo* at;
  int j, left;
  int shape;   // tiles of the unit << 1 | both halves have rows
  bool first;  // the tile is the first of its piece
  __device__ __forceinline__ void begin(const AttnArgs& a, typename S::Tail* t) {
    at = &t->unit[threadIdx.x >> 5];
    shape = set_unit<S>(a, at, t->start[0], t->start[1], t->start[2]);
    j = t->start[3];
    left = t->n;
    first = true;
  }
  __device__ __forceinline__ int tiles() const { return shape >> 1; }
  __device__ __forceinline__ int halves() const { return 1 + (shape & 1); }
  __device__ __forceinline__ bool last() const { return left == 1 || j + 1 == tiles(); }
  __device__ __forceinline__ void advance(const AttnArgs& a) {
    first = false;
    if (--left == 0 || ++j < tiles()) return;
    j = 0;
    first = true;
    shape = next_unit<S>(a, at);
  }
};

// The CTA's range.  A unit costs its tiles and unit_cost more (its query, the first S that nothing overlaps, its output), so
// ranges are equal in that; a cut inside a unit's extra cost is a cut before its first tile.
struct Place {
  int s, kvh, u, j;
  long long tile;  // tiles before it
};
// Where x lies; all lanes of a warp.  cum[s], units[s]: cost and units of one kv head of the runs before s.
template <class S>
__device__ Place find_place(const AttnArgs& a, const long long* cum, const int* units, long long x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.batch - 1;  // first s with Hkv cum[s + 1] > x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.Hkv * cum[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  const RunInfo r = run_info(a, lo);
  const int r_units = units_of<S>(a, r);
  const long long per_head = cum[lo + 1] - cum[lo], rem = x - a.Hkv * cum[lo];
  Place p{lo, static_cast<int>(rem / per_head), 0, 0, 0};
  long long at = rem - p.kvh * per_head;
  for (int u0 = 0; u0 < r_units; u0 += 32) {  // the unit of the head
    const int n = u0 + lane < r_units ? tiles_of<S>(a, r, u0 + lane) + a.unit_cost : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(dec::kFull, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(dec::kFull, inc > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      p.u = u0 + l;
      p.j = max(0, static_cast<int>(at - __shfl_sync(dec::kFull, inc - n, l)) - a.unit_cost);
      const long long before = rem - at + __shfl_sync(dec::kFull, inc - n, l);  // cost of the run's units before
      p.tile = a.Hkv * cum[lo] + before - a.unit_cost * (static_cast<long long>(a.Hkv) * units[lo] + static_cast<long long>(p.kvh) * r_units + p.u) + p.j;
      return p;
    }
    at -= __shfl_sync(dec::kFull, inc, 31);
  }
  return p;  // cannot be: x < the total
}
// cum and units: shared memory that the ring takes over later.
template <class S>
__device__ void plan(const AttnArgs& a, typename S::Tail* t, long long* cum, int* units) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < a.batch; s += S::kThreads / 32) {
    const RunInfo r = run_info(a, s);
    if (r.row0 < 0 && blockIdx.x == 0 && lane == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    const int r_units = units_of<S>(a, r);
    long long n = 0;
    for (int u = lane; u < r_units; u += 32) n += tiles_of<S>(a, r, u) + a.unit_cost;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(dec::kFull, n, o);
    if (lane == 0) {
      cum[s + 1] = n;
      units[s + 1] = r_units;
    }
  }
  __syncthreads();
  if (warp == 0) {
    long long base = 0;
    int ubase = 0;
    if (lane == 0) cum[0] = units[0] = 0;
    for (int s0 = 0; s0 < a.batch; s0 += 32) {
      const int s = s0 + lane;
      long long v = s < a.batch ? cum[s + 1] : 0;
      int w = s < a.batch ? units[s + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(dec::kFull, v, o);
        const int y = __shfl_up_sync(dec::kFull, w, o);
        if (lane >= o) { v += x; w += y; }
      }
      if (s < a.batch) { cum[s + 1] = base + v; units[s + 1] = ubase + w; }
      base += __shfl_sync(dec::kFull, v, 31);
      ubase += __shfl_sync(dec::kFull, w, 31);
    }
    __syncwarp();
    const long long T = base * a.Hkv;
    const long long W = min(static_cast<long long>(gridDim.x), T);
    int n = 0;
    if (blockIdx.x < W) {
      const long long x1 = T * (blockIdx.x + 1) / W;
      const Place p = find_place<S>(a, cum, units, T * blockIdx.x / W);
      const long long end = x1 < T ? find_place<S>(a, cum, units, x1).tile : T - a.unit_cost * (static_cast<long long>(a.Hkv) * ubase);
      n = static_cast<int>(end - p.tile);
      if (lane == 0) {
        t->start[0] = p.s;
        t->start[1] = p.kvh;
        t->start[2] = p.u;
        t->start[3] = p.j;
      }
    }
    if (lane == 0) t->n = n;
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------------------------ shared by the roles
__device__ __forceinline__ uint4 ldg_codes(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Column k of a 32-column chunk: page parity (k >> 2) & 1, token of the page.
__device__ __forceinline__ constexpr int col_token(int k) { return 2 * (k >> 3) + (k & 1) + 8 * ((k >> 1) & 1); }

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
// This thread's channels of O times alpha.
template <int CHANNELS>
__device__ __noinline__ void rescale_o(uint32_t to, float alpha) {
#pragma unroll 1
  for (int i = 0; i < CHANNELS / 16; ++i) {
    float o[16];
    uint32_t* u = reinterpret_cast<uint32_t*>(o);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(to + 16 * i));
    wait_ld();
    loaded<16>(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] *= alpha;
    tmem_st16(to + 16 * i, u);
  }
}
// This thread's channels of O, divided and rounded, to the output.
template <int CHANNELS>
__device__ __noinline__ void store_out(uint32_t to, float inv, uint16_t* dst_row, bool valid) {
  uint4* dst = reinterpret_cast<uint4*>(dst_row);
#pragma unroll 1
  for (int i = 0; i < CHANNELS / 32; ++i) {
    float o[32];
    tmem_ld32(to + 32 * i, o);
    wait_ld();
    loaded<32>(o);
    if (valid) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[4 * i + e] = make_uint4(dec::pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv), dec::pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                    dec::pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv), dec::pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
    }
  }
}
// The same as they are, for the merge.
template <int CHANNELS>
__device__ __noinline__ void store_piece(uint32_t to, float* dst_row) {
  float4* dst = reinterpret_cast<float4*>(dst_row);
#pragma unroll 1
  for (int i = 0; i < CHANNELS / 32; ++i) {
    float o[32];
    tmem_ld32(to + 32 * i, o);
    wait_ld();
    loaded<32>(o);
#pragma unroll
    for (int e = 0; e < 8; ++e) dst[8 * i + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
}

// ------------------------------------------------------------------------------------------------ merge
// The units that more than one CTA worked on: warp i of block (c, .) merges row i of the unit that began in CTA c.
template <int kRows, int kAtOnce>
__global__ void __launch_bounds__(256) tile_merge_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int in_unit = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int32_t* rec = a.tw_rec + 8 * c;
  // loads that do not wait for each other: the record, the next CTAs' ends, the first two pieces
  const int4 unit = *reinterpret_cast<const int4*>(rec);
  const bool ends = c + 1 + lane < a.tile_ctas && a.tw_rec[8 * (c + 1 + lane) + 4];
  auto stats_of = [&](int k) { return *reinterpret_cast<const float2*>(a.tw_stats + (static_cast<size_t>(k == c ? 2 * c + 1 : 2 * k) * kRows + in_unit) * 2); };
  auto acc_of = [&](int k) { return *reinterpret_cast<const float4*>(a.tw_acc + (static_cast<size_t>(k == c ? 2 * c + 1 : 2 * k) * kRows + in_unit) * kHeadDim + 4 * lane); };
  if (!unit.x) return;
  const RunInfo run = run_info(a, unit.y);
  const int r = unit.w * kRows + in_unit;
  if (r >= run.n * a.G) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const unsigned hit = __ballot_sync(dec::kFull, ends);
  int end = c + __ffs(hit);  // the last CTA with a piece
  if (!hit) {
    end = c + 33;
    while (end + 1 < a.tile_ctas && !a.tw_rec[8 * end + 4]) ++end;
  }
  // Loads of kAtOnce pieces are on their way together.
  for (int k0 = c; k0 <= end; k0 += kAtOnce) {
    float2 st[kAtOnce];
    float4 v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (k0 + i <= end) {
        st[i] = stats_of(k0 + i);
        v[i] = acc_of(k0 + i);
      }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (k0 + i > end) break;
      const float mn = fmaxf(m, st[i].x);
      const float f0 = m == -INFINITY ? 0.f : ex2(m - mn), f1 = st[i].x == -INFINITY ? (st[i].y == 0.f ? 0.f : 1.f) : ex2(st[i].x - mn);
      m = mn;
      l = l * f0 + st[i].y * f1;
      acc.x = acc.x * f0 + v[i].x * f1;
      acc.y = acc.y * f0 + v[i].y * f1;
      acc.z = acc.z * f0 + v[i].z * f1;
      acc.w = acc.w * f0 + v[i].w * f1;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int head = unit.z * a.G + r % a.G;
  const long long at = static_cast<long long>(run.row0 + r / a.G) * a.Hq + head;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * kHeadDim + 4 * lane) =
      make_uint2(dec::pack_bf16(acc.x * inv, acc.y * inv), dec::pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + (log2f(l) - kTileShift)) * dec::kLn2;
}

// A workspace of pieces, two for each CTA, with the offsets of its three arrays.
inline size_t pieces_workspace(int rows, int sms, size_t* acc, size_t* stats, size_t* rec) {
  *rec = 0;
  *stats = 8 * sizeof(int32_t) * static_cast<size_t>(sms);
  *stats = (*stats + 255) & ~static_cast<size_t>(255);
  *acc = *stats + static_cast<size_t>(sms) * 2 * rows * 2 * sizeof(float);
  return *acc + static_cast<size_t>(sms) * 2 * rows * kHeadDim * sizeof(float);
}

}  // namespace
}  // namespace runs
}  // namespace kvq
