// attn_runs_tile.cu -- kvq_attn_runs for long runs (prompts and chunks of them), BF16 queries: tcgen05 products.
//
// A unit is one (request, kv head, 256 consecutive (token, head) rows of the run); its key tiles are the 128-token tiles
// up to its last visible token.  All units' tiles are laid end to end and cut into equal contiguous ranges, one per CTA
// of a grid of one CTA per SM, so that one long prompt, many short ones and a short chunk behind a long context load the
// machine alike.  A range may begin or end inside a unit: such pieces leave (m, l, O) in the workspace for the merge.
//
// Per key tile and 128-row half of the unit:  S = Q K^T (both from shared memory, S in TMEM), the softmax of a row by two
// threads, P (fp16) over S's columns in TMEM,  O += P V (V from shared memory, O in TMEM).  fp16 operands: codes of either
// format are exact in it, a bf16 query is exact after a power of two is taken from its row.  With
// S = 128 x 128 x 128 at 8192 flop a clock the two halves cost 2048 clocks a tile on the tensor core.  The codes go from global
// memory through registers to shared memory once for all 256 rows (eight converting warps), and eight warps do the softmax of
// one half while the tensor core works on the other.
// Bound by a half's chain of S, maximum, weights, products and the next S, ~4,000 clocks a tile (reads of TMEM take ~250 clocks
// and 80 registers do not hold a half row, so S is read twice; there are no TMEM columns for a second S).  A causal prompt of
// 11996 tokens, 32 query and 8 kv heads, E4M3: 1,030 us, 1,144 TFLOP/s.
//
// Warps: 0-15 softmax (0-3 rows 0..127 and keys 0..63 of a tile, 4-7 rows 128..255, 8-15 the same rows and keys 64..127),
// 16-23 convert, 24 issues the products.
// The loops are kept rolled and what happens once a unit is called: all roles' code is live at once, and unrolled
// (100 KB) it spent most of the time on instruction fetches (2.9 ms on a prompt of 11996 tokens).
// Shared memory: Q 2 x 32 KB, then a ring of 32 KB slots taking K and V tiles in turn, every operand as 64-element
// columns of 128-byte rows, 128-byte swizzle (16-byte chunk index ^ row & 7).
// Key order inside a tile.  The value tiles hold tokens 2q, 2q+1, 2q+8, 2q+9 of a channel in one lane's word.  Two pages'
// such words make one 16-byte chunk of the V operand, so key column 32 (p >> 1) + 8 q + 4 (p & 1) + i stands for token
// 2 q + (i & 1) + 8 (i >> 1) of page p: K rows are placed accordingly and P's columns follow.
#include "attn_runs.cuh"

namespace kvq {
namespace runs {
namespace {

using dec::ex2;
using dec::smem_u32;

constexpr int kRows = 256;      // rows of a unit
constexpr int kKeys = 128;      // keys of a tile
constexpr int kPagesPerTile = kKeys / kPage;
constexpr int kSlots = 5;       // ring of operand tiles
constexpr int kOperand = 32768;  // 128 x 128 fp16
constexpr int kSoftmaxWarps = 16, kConvertWarp = 16, kMmaWarp = 24;  // first warps of the roles
constexpr int kThreads = 28 * 32;
// Registers: 72 a thread at launch; the softmax warps take what the last warpgroup, of which only one warp works, gives back.  None of the loops may spill: with 227 KB of shared memory the L1 keeps nothing, and a
// spilled value costs ~500 clocks a use.
constexpr int kRegsSoftmax = 80, kRegsConvert = 72, kRegsMma = 40;
static_assert(16 * kRegsSoftmax + 8 * kRegsConvert + 4 * kRegsMma <= 28 * 72, "no more than the block was launched with");
// Key tiles that the L2 is ahead.  A prompt of 11996 tokens 1092 -> 1030 us, 24 chunks of 64 tokens behind 9001 253 -> 232 us; 2, 3,
// 4 and 6 tiles are within 1 % of each other.
constexpr int kAhead = 3;
constexpr int kScaleSlots = 3;  // a tile's scales are read until its V slot is free, which the K of the third next tile waits for
constexpr float kTileShift = 7.f;  // weights are held times 2^7 ..
constexpr float kSlack = 8.f;      // .. and may grow to 2^15 before the running maximum (and O) is moved
constexpr int kOffQ = 0, kOffRing = 2 * kOperand, kOffTail = kOffRing + kSlots * kOperand;
constexpr int kTailBytes = 3 * 1024;
constexpr int kSmemBytes = kOffTail + kTailBytes;
constexpr uint32_t kIdesc = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);  // fp16 x fp16 -> fp32, M = N = 128
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // columns: S (and P) of the two halves, then O

struct RunInfo {
  int len, n, row0;
};
struct UnitInfo {
  int s, kvh, u;
  RunInfo run;
};

// A tile is the first, the last of its piece; both halves have rows.
constexpr int kFirst = 1, kLast = 2, kBoth = 4;
struct Tail {  // shared memory behind the operands
  float2 scale[kScaleSlots][kPagesPerTile];  // 2^ek sm_scale log2 e, ev (0, -inf for an absent page)
  int flags[kScaleSlots];  // of a tile, with its K: kFirst, kLast, kBoth
  float peer[kSoftmaxWarps][32];  // what the two warps of a row tell each other
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2];
  uint64_t drained;  // every product of the CTA
  uint32_t tmem;
  int abort;
  UnitInfo unit[kMmaWarp];  // where each warp is
  int start[4];  // request, kv head, unit, first tile of the CTA's range
  int n;         // its tiles
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");

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
__device__ __forceinline__ int units_of(const AttnArgs& a, const RunInfo& r) {
  const int rows = r.n * a.G;
  return rows > a.few_rows ? (rows + kRows - 1) / kRows : 0;
}
// Key tiles of unit u: up to the last token that its last row sees, one at least (whose columns may all be hidden).
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const RunInfo& r, int u) {
  const int last = min(r.n - 1, (kRows * (u + 1) - 1) / a.G);
  const int limit = r.len - r.n + last + 1;
  return max(1, (limit + kKeys - 1) / kKeys);
}

__device__ __forceinline__ int halves_of(const AttnArgs& a, const RunInfo& r, int u) { return r.n * a.G - u * kRows > 128 ? 2 : 1; }

// Where a warp is in its CTA's range of tiles.  The unit lives in shared memory: in registers it would be spilled, and
// with 227 KB of shared memory the L1 that is left loses what is spilled to the L2 (~500 clocks a use).
__device__ __forceinline__ int set_unit(const AttnArgs& a, UnitInfo* at, int s, int kvh, int u) {
  const RunInfo r = run_info(a, s);
  const UnitInfo i{s, kvh, u, r};
  __syncwarp();
  *at = i;  // every lane the same
  __syncwarp();
  return tiles_of(a, r, u) << 1 | (halves_of(a, r, u) - 1);
}
__device__ __forceinline__ int next_unit(const AttnArgs& a, UnitInfo* at) {
  UnitInfo i = *at;
  if (++i.u == units_of(a, i.run)) {
    i.u = 0;
    if (++i.kvh == a.Hkv) {
      i.kvh = 0;
      do i.run = run_info(a, ++i.s); while (units_of(a, i.run) == 0);  // called only where a later unit exists
    }
  }
  __syncwarp();
  *at = i;
  __syncwarp();
  return tiles_of(a, i.run, i.u) << 1 | (halves_of(a, i.run, i.u) - 1);
}
struct Cursor {
  UnitInfo* at;
  int j, left;
  int shape;   // tiles of the unit << 1 | both halves have rows
  bool first;  // the tile is the first of its piece
  __device__ __forceinline__ void begin(const AttnArgs& a, Tail* t) {
    at = &t->unit[threadIdx.x >> 5];
    shape = set_unit(a, at, t->start[0], t->start[1], t->start[2]);
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
    shape = next_unit(a, at);
  }
};

// The CTA's range.  A unit costs its tiles and unit_cost more (its query, the first S that nothing overlaps, its output), so
// ranges are equal in that; a cut inside a unit's extra cost is a cut before its first tile.
struct Place {
  int s, kvh, u, j;
  long long tile;  // tiles before it
};
// Where x lies; all lanes of a warp.  cum[s], units[s]: cost and units of one kv head of the runs before s.
__device__ Place find_place(const AttnArgs& a, const long long* cum, const int* units, long long x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.batch - 1;  // first s with Hkv cum[s + 1] > x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.Hkv * cum[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  const RunInfo r = run_info(a, lo);
  const int r_units = units_of(a, r);
  const long long per_head = cum[lo + 1] - cum[lo], rem = x - a.Hkv * cum[lo];
  Place p{lo, static_cast<int>(rem / per_head), 0, 0, 0};
  long long at = rem - p.kvh * per_head;
  for (int u0 = 0; u0 < r_units; u0 += 32) {  // the unit of the head
    const int n = u0 + lane < r_units ? tiles_of(a, r, u0 + lane) + a.unit_cost : 0;
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
__device__ void plan(const AttnArgs& a, Tail* t, long long* cum, int* units) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < a.batch; s += kThreads / 32) {
    const RunInfo r = run_info(a, s);
    if (r.row0 < 0 && blockIdx.x == 0 && lane == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    const int r_units = units_of(a, r);
    long long n = 0;
    for (int u = lane; u < r_units; u += 32) n += tiles_of(a, r, u) + a.unit_cost;
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
      const Place p = find_place(a, cum, units, T * blockIdx.x / W);
      const long long end = x1 < T ? find_place(a, cum, units, x1).tile : T - a.unit_cost * (static_cast<long long>(a.Hkv) * ubase);
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

// ------------------------------------------------------------------------------------------------ converting warps
__device__ __forceinline__ uint4 ldg_codes(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

template <bool INT8>
__device__ void convert_role(const AttnArgs& a, Tail* t, uint8_t* ring) {
  const int cw = (threadIdx.x >> 5) - kConvertWarp, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  constexpr uint32_t kZero = INT8 ? 0x80808080u : 0u;
  // Everything is loaded one step before its use and left untouched until then, so that no load is waited for where it is
  // issued: block-table entries a tile ahead, a word of V where the word of K before it leaves its register, the next
  // tile's K where V does.  An absent page (behind the context, or an entry outside the cache) is read as page 0 and
  // cleared when it is converted.
  Cursor c;
  c.begin(a, t);
  // Entry of page (lane & 7) of a tile; 0 behind the context.
  auto load_entry = [&](int s, int j, int len) {
    const int page = j * kPagesPerTile + (lane & 7);
    return page * kPage < len ? a.block_table[static_cast<size_t>(s) * a.max_pages + page] : 0;
  };
  auto absent = [&](int entry) { return entry < 0 || entry >= a.num_pages; };
  auto present = [&](int entry) { return absent(entry) ? 0 : entry; };
  const uint32_t page_bytes = a.Hkv * 2048;  // of one plane
  uint4 buf[4];
  uint16_t ks = 0, vs = 0;  // scales of the warp's key page
  auto tile_at = [&](const uint8_t* plane, int phys, int from) {  // this head's tile of lane from's page
    return plane + static_cast<uint64_t>(static_cast<uint32_t>(__shfl_sync(dec::kFull, phys, from))) * page_bytes;
  };
  // K: page cw, four words of 512 bytes.  V: channels 32 mm .. of the pages 4 quad .., odd rows taking the pairs of pages
  // crosswise.
  const int mm = cw & 3, quad = cw >> 2;
  auto load_k = [&](const uint8_t* plane, int phys, int i) { buf[i] = ldg_codes(tile_at(plane, phys, cw) + i * 512); };
  auto load_v = [&](const uint8_t* plane, int phys, int i) { buf[i] = ldg_codes(tile_at(plane, phys, 4 * quad + (i ^ (2 * (g & 1))))); };
  auto k_plane = [&]() { return a.k + c.at->kvh * 2048 + lane * 16; };
  auto load_scales = [&](int phys) {
    const int p = __shfl_sync(dec::kFull, phys, cw);
    if (a.num_pages > 0) {
      const size_t si = static_cast<size_t>(c.at->kvh) * a.num_pages + p;
      ks = a.ks[si];
      vs = a.vs[si];
    }
  };
  int slot = 0;
  uint32_t phase = 0;
  auto publish = [&]() {
    dec::fence_proxy_async();
    __syncwarp();
    if (lane == 0) arrive(&t->full[slot]);
    if (++slot == kSlots) { slot = 0; phase ^= 1u; }
  };
  // this lane's rows: token 8 h + g of page p goes to row 32 (p >> 1) + 8 (g >> 1) + 4 (p & 1) + 2 h + (g & 1)
  const int k_low = 4 * (cw & 1) + (g & 1);  // row & 7 for h = 0
  const int k_row = 32 * (cw >> 1) + 8 * (g >> 1) + k_low;
  const int v_row = 32 * mm + g;
  int entry = load_entry(c.at->s, c.j, c.at->run.len), entry_next = 0;
  // Registers hold 16 KB on their way to an SM, enough for what the L2 has and a quarter of what HBM needs: lines of the tile
  // kAhead on in the unit are brought to the L2, one a lane (K of page cw the first 16, V the others), by an entry that was
  // loaded a tile before.
  auto entry_ahead = [&]() {
    const int page = (c.j + kAhead) * kPagesPerTile + cw;
    return page * kPage < c.at->run.len ? a.block_table[static_cast<size_t>(c.at->s) * a.max_pages + page] : -1;
  };
  int far = entry_ahead();
  {
    const int phys = present(entry);
    const uint8_t* plane = k_plane();
#pragma unroll
    for (int i = 0; i < 4; ++i) load_k(plane, phys, i);
    load_scales(phys);
  }
#pragma unroll 1
  for (int at = 0; c.left > 0;) {
    const int in_context = c.at->run.len - c.j * kKeys;  // tokens of the tile that the context has
    if (!absent(far)) {
      const uint8_t* plane = lane < 16 ? a.k : a.v;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(plane + static_cast<uint64_t>(far) * page_bytes + c.at->kvh * 2048 + (lane & 15) * 128));
    }
    const bool here = (lane & 7) * kPage < in_context;
    // bits 0..7: absent pages; 8..: the tile's flags
    const unsigned lost = (__ballot_sync(dec::kFull, !here || absent(entry)) & 0xFFu) |
                          ((c.first ? kFirst : 0) | (c.last() ? kLast : 0) | (c.halves() == 2 ? kBoth : 0)) << 8;
    if (here && absent(entry) && cw == 0 && lane < 8) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    if (!wait_warp(&t->empty[slot], phase ^ 1u, &t->abort)) return;
    if ((lost >> cw) & 1u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) buf[i] = make_uint4(kZero, kZero, kZero, kZero);
    }
    {
      const int phys = present(entry);
      const uint8_t* plane = a.v + c.at->kvh * 2048 + (mm * 32 + lane) * 16;
      uint8_t* dst = ring + slot * kOperand + k_row * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // word i = (token half, channel half)
        const uint4 x = buf[i];
        const int low = k_low + 2 * (i >> 1);
        uint8_t* base = dst + (i & 1) * 16384 + 2 * (i >> 1) * 128;
        *reinterpret_cast<uint4*>(base + (((2 * q) ^ low) << 4)) =
            make_uint4(codes_lo<INT8>(x.x), codes_hi<INT8>(x.x), codes_lo<INT8>(x.y), codes_hi<INT8>(x.y));
        *reinterpret_cast<uint4*>(base + (((2 * q + 1) ^ low) << 4)) =
            make_uint4(codes_lo<INT8>(x.z), codes_hi<INT8>(x.z), codes_lo<INT8>(x.w), codes_hi<INT8>(x.w));
        load_v(plane, phys, i);
      }
    }
    if (lane == 0) {
      if (cw == 0) t->flags[at] = lost >> 8;
      const int ek = f16_to_exp(ks), ev = f16_to_exp(vs);
      t->scale[at][cw] = (lost >> cw) & 1u ? make_float2(0.f, -INFINITY)
                                           : make_float2(fabsf(a.sm_scale) * dec::kLog2e * exp2_int(ek), static_cast<float>(ev));
    }
    publish();
    if (++at == kScaleSlots) at = 0;
    c.advance(a);
    const bool more = c.left > 0;
    if (more) {
      entry_next = load_entry(c.at->s, c.j, c.at->run.len);
      far = entry_ahead();
    }
    if (!wait_warp(&t->empty[slot], phase ^ 1u, &t->abort)) return;
    if (in_context < kKeys || (lost & 0xFFu)) {  // what lies behind the context may be anything, a NaN too
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int page = 4 * quad + (i ^ (2 * (g & 1)));
        const int nvalid = (lost >> page) & 1u ? 0 : in_context - page * kPage;
        auto mask = [&](int tok) { return (tok < nvalid ? 0x00FF00FFu : 0u) | (tok + 1 < nvalid ? 0xFF00FF00u : 0u); };
        const uint32_t m0 = mask(2 * q), m1 = mask(2 * q + 8);
        uint4& w = buf[i];
        w.x = (w.x & m0) | (kZero & ~m0);
        w.z = (w.z & m0) | (kZero & ~m0);
        w.y = (w.y & m1) | (kZero & ~m1);
        w.w = (w.w & m1) | (kZero & ~m1);
      }
    }
    entry = entry_next;
    {
      const int phys = present(entry);
      const uint8_t* plane = k_plane();
      uint8_t* dst = ring + slot * kOperand + v_row * 128 + quad * 16384;
#pragma unroll
      for (int pp = 0; pp < 2; ++pp) {
        const uint4 x = buf[2 * pp], y = buf[2 * pp + 1];
        // pair of pages 2 quad + (pp ^ (g & 1)): column 32 pair + 8 q + {its first page: 0..3, its second: 4..7}
        uint8_t* base = dst + (((4 * ((pp ^ g) & 1) + q) ^ g) << 4);
        *reinterpret_cast<uint4*>(base) = make_uint4(codes_lo<INT8>(x.x), codes_lo<INT8>(x.y), codes_lo<INT8>(y.x), codes_lo<INT8>(y.y));
        *reinterpret_cast<uint4*>(base + 8 * 128) = make_uint4(codes_hi<INT8>(x.x), codes_hi<INT8>(x.y), codes_hi<INT8>(y.x), codes_hi<INT8>(y.y));
        *reinterpret_cast<uint4*>(base + 16 * 128) = make_uint4(codes_lo<INT8>(x.z), codes_lo<INT8>(x.w), codes_lo<INT8>(y.z), codes_lo<INT8>(y.w));
        *reinterpret_cast<uint4*>(base + 24 * 128) = make_uint4(codes_hi<INT8>(x.z), codes_hi<INT8>(x.w), codes_hi<INT8>(y.z), codes_hi<INT8>(y.w));
        load_k(plane, phys, 2 * pp);  // behind the last tile: read again and thrown away
        load_k(plane, phys, 2 * pp + 1);
      }
      load_scales(phys);
    }
    publish();
  }
  // the products' last arrivals on the ring land before the CTA may end
  for (int i = 0; i < kSlots && i < 2 * t->n; ++i) {
    if (--slot < 0) { slot = kSlots - 1; phase ^= 1u; }
    if (!wait_warp(&t->empty[slot], phase, &t->abort)) return;
  }
}

// ------------------------------------------------------------------------------------------------ products
__device__ void mma_role(Tail* t, uint32_t smem_base, uint32_t tmem, uint32_t leader) {
  tmem = dec::uniform_u32(tmem);
  const uint64_t ring = smem_desc(smem_base + kOffRing);
  const uint64_t qd = smem_desc(smem_base + kOffQ);
  // Eight steps of 16: 32 bytes apart inside a 64-element column of rows, the second column 16 KB on; the weights of keys
  // 64.. lie in those columns of S.  Unrolled: in a loop a product took ~90 clocks to issue, more than to run.
  auto k_step = [](int ks) { return static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4); };
  auto qk = [&](int i, int slot) {
    const uint64_t x = qd + static_cast<uint64_t>(i * (kOperand >> 4)), y = ring + static_cast<uint64_t>(slot * (kOperand >> 4));
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_ss(tmem + kTmemS + 128 * i, x + k_step(ks), y + k_step(ks), ks > 0, leader);
  };
  auto pv = [&](int i, int slot, bool acc) {
    const uint64_t y = ring + static_cast<uint64_t>(slot * (kOperand >> 4));
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      mma_ts(tmem + kTmemO + 128 * i, tmem + kTmemS + 128 * i + (ks >> 2) * 64 + (ks & 3) * 8, y + k_step(ks), acc || ks > 0, leader);
  };
  int slot = 0;  // of the operand tile taken next
  uint32_t phase = 0, q_phase = 0, p_phase = 0;  // the latter: bit i for half i
  auto next_slot = [&]() {
    if (++slot == kSlots) { slot = 0; phase ^= 1u; }
  };
  const int total = dec::uniform_u32(t->n);
  int flags = kLast;  // of the tile before; its last: the next one's S is not issued yet
#pragma unroll 1
  for (int jj = 0, at = 0; jj < total; ++jj) {
    if (flags & kLast) {  // first tile of a piece
      if (!wait_warp(&t->full[slot], phase, &t->abort)) return;
      flags = dec::uniform_u32(*reinterpret_cast<volatile int*>(&t->flags[at]));
      for (int i = 0; i < (flags & kBoth ? 2 : 1); ++i) {
        if (!wait_warp(&t->q_full[i], (q_phase >> i) & 1u, &t->abort)) return;
        q_phase ^= 1u << i;
        fence_after();
        qk(i, slot);
        commit(&t->s_full[i], leader);
      }
      commit(&t->empty[slot], leader);
      next_slot();
    } else {  // its K has come with its flags
      flags = dec::uniform_u32(*reinterpret_cast<volatile int*>(&t->flags[at]));
    }
    const bool more = !(flags & kLast), two = (flags & kBoth) != 0;
    const int v_slot = slot;
    const uint32_t v_phase = phase;
    next_slot();
#pragma unroll 1
    for (int i = 0; i < 1 + two; ++i) {
      if (!wait_warp(&t->p_full[i], (p_phase >> i) & 1u, &t->abort)) return;
      p_phase ^= 1u << i;
      if (i == 0 && !wait_warp(&t->full[v_slot], v_phase, &t->abort)) return;
      fence_after();
      pv(i, v_slot, !(flags & kFirst));
      commit(&t->pv_done[i], leader);
      if (i == two) commit(&t->empty[v_slot], leader);
      if (more) {
        if (i == 0 && !wait_warp(&t->full[slot], phase, &t->abort)) return;
        fence_after();
        qk(i, slot);
        commit(&t->s_full[i], leader);
        if (i == two) commit(&t->empty[slot], leader);
      }
    }
    if (more) next_slot();
    if (++at == kScaleSlots) at = 0;
  }
}

// ------------------------------------------------------------------------------------------------ softmax
// Column k of a 32-column chunk: page parity (k >> 2) & 1, token of the page.
__device__ __forceinline__ constexpr int col_token(int k) { return 2 * (k >> 3) + (k & 1) + 8 * ((k >> 1) & 1); }

// Two threads have a row: one the keys 0..63 of a tile and the output's channels 0..63, its peer (8 warps on) the others.
// Each goes over its columns of S in TMEM twice, the maximum, then the weights, 32 columns (pages 2 i and 2 i + 1, in groups
// of four columns) at a time.  y = x log2 e + ev = S k + ev; since k >= 0 a page's largest S gives its largest y.  Keys that
// the row does not see (token >= seen of the tile) have -inf, whatever S holds there.
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float row_max(uint32_t ts, const float2* scale, float rk) {
  float tm = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    float s[32];
    tmem_ld32(ts + 32 * i, s);
    const float4 sc = *reinterpret_cast<const float4*>(scale + 2 * i);
    wait_ld();
    loaded<32>(s);
    float pm[2];
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const float* x = s + 4 * par;  // columns 0..3, 8..11, 16..19, 24..27 from here
      const float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[8], x[9]), m2 = max3(x[10], x[11], x[16]);
      const float m3 = max3(x[17], x[18], x[19]), m4 = max3(x[24], x[25], x[26]);
      pm[par] = fmaxf(max3(m0, m1, m2), max3(m3, m4, x[27]));
    }
    tm = max3(tm, fmaf(pm[0], sc.x * rk, sc.y), fmaf(pm[1], sc.z * rk, sc.w));
  }
  return tm;
}
__device__ __forceinline__ float row_max_masked(uint32_t ts, const float2* scale, float rk, int seen) {
  float tm = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    float s[32];
    tmem_ld32(ts + 32 * i, s);
    const float4 sc = *reinterpret_cast<const float4*>(scale + 2 * i);
    const float k0 = sc.x * rk, k1 = sc.z * rk;
    wait_ld();
    loaded<32>(s);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float y = (e >> 2) & 1 ? fmaf(s[e], k1, sc.w) : fmaf(s[e], k0, sc.y);
      tm = fmaxf(tm, kPage * (2 * i + ((e >> 2) & 1)) + col_token(e) < seen ? y : -INFINITY);
    }
  }
  return tm;
}
// Weights 2^{y + base} as fp16 pairs over the columns of S, and their sum without the value scales.
template <bool MASKED>
__device__ __forceinline__ float weights(uint32_t ts, const float2* scale, float rk, float base, int seen) {
  float l = 0.f;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    float s[32];
    uint32_t pk[16];
    tmem_ld32(ts + 32 * i, s);
    const float4 sc = *reinterpret_cast<const float4*>(scale + 2 * i);
    const dec::f2x k2[2] = {dec::f2_splat(sc.x * rk), dec::f2_splat(sc.z * rk)};
    const dec::f2x b2[2] = {dec::f2_splat(sc.y + base), dec::f2_splat(sc.w + base)};
    const float un[2] = {sc.y == -INFINITY ? 0.f : ex2(-sc.y), sc.w == -INFINITY ? 0.f : ex2(-sc.w)};
    wait_ld();
    loaded<32>(s);
    dec::f2x sum[2];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const int par = (e >> 2) & 1;
      float y0, y1;
      dec::f2_unpack(dec::f2_fma(dec::f2_pack(s[e], s[e + 1]), k2[par], b2[par]), y0, y1);
      if (MASKED) {
        y0 = kPage * (2 * i + par) + col_token(e) < seen ? y0 : -INFINITY;
        y1 = kPage * (2 * i + par) + col_token(e + 1) < seen ? y1 : -INFINITY;
      }
      const float p0 = ex2(y0), p1 = ex2(y1);
      const dec::f2x p2 = dec::f2_pack(p0, p1);
      sum[par] = (e & ~4) == 0 ? p2 : dec::f2_add(sum[par], p2);
      pk[e >> 1] = dec::pack_f16(p0, p1);
    }
    tmem_st16(ts + 16 * i, pk);
    float l0, l1, l2, l3;
    dec::f2_unpack(sum[0], l0, l1);
    dec::f2_unpack(sum[1], l2, l3);
    l = fmaf(l0 + l1, un[0], fmaf(l2 + l3, un[1], l));
  }
  return l;
}
// This thread's channels of O times alpha.
__device__ __noinline__ void rescale_o(uint32_t to, float alpha) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
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
// Rows 16 part .. of the warp pair's 32 (at: element of this lane's row in q, negative for none) times a power of two each, to
// shared memory (qs: the half's operand); the factors go to scale[row].  Sixteen lanes read a row: with a row to a thread,
// every load touched 32 lines and the L1 took 17,000 clocks for a unit's queries.
__device__ __noinline__ void stage_query(const uint16_t* q, long long at, float sm_scale, uint8_t* qs, int row0, int part, float* scale) {
  const int lane = threadIdx.x & 31, chunk = lane & 15;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long src = __shfl_sync(dec::kFull, at, 16 * part + 2 * i + (lane >> 4));
    w[i] = src >= 0 ? *reinterpret_cast<const uint4*>(q + src + 8 * chunk) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t top = 0;  // largest exponent field
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max((u[e] >> 7) & 0xFFu, (u[e] >> 23) & 0xFFu));
#pragma unroll
    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(dec::kFull, top, o));
    // largest element in [2^8, 2^9): bf16 elements are then exact in fp16 down to 2^-22 of it
    const int er = min(max(static_cast<int>(top) - 127 - 8, -100), 120);
    const float f = copysignf(exp2_int(-er), sm_scale);  // a negative scale goes into the query
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      h[e] = dec::pack_f16(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f);
    const int in32 = 16 * part + 2 * i + (lane >> 4), row = row0 + in32;
    *reinterpret_cast<uint4*>(qs + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    if (chunk == 0) scale[in32] = exp2_int(er);
  }
  dec::fence_proxy_async();
}
// This thread's channels of O, divided and rounded, to the output.
__device__ __noinline__ void store_out(uint32_t to, float inv, uint16_t* dst_row, bool valid) {
  uint4* dst = reinterpret_cast<uint4*>(dst_row);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
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
__device__ __noinline__ void store_piece(uint32_t to, float* dst_row) {
  float4* dst = reinterpret_cast<float4*>(dst_row);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    float o[32];
    tmem_ld32(to + 32 * i, o);
    wait_ld();
    loaded<32>(o);
#pragma unroll
    for (int e = 0; e < 8; ++e) dst[8 * i + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
}

// At the end of a unit the next one's query is staged, so that its first S is issued, before O is stored.
__device__ void softmax_role(const AttnArgs& a, Tail* t, uint8_t* smem, uint32_t tmem, int32_t* rec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = (warp >> 2) & 1, part = warp >> 3;  // rows, columns
  const int row = (warp & 3) * 32 + lane;              // of the half
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp & 3)
  const uint32_t ts = tmem + kTmemS + 128 * half + 64 * part + lanes, to = tmem + kTmemO + 128 * half + 64 * part + lanes;
  // A value for the peer and the peer's for this thread.  The meetings have no limit of their own, so a warp whose wait has given
  // up goes on to the end of its range all the same, without waiting or handing anything on: the two take every meeting that
  // the range has, wherever either of them gave up (one that left the loop would keep its peer waiting: the peer's own waits may
  // have been over before).  What it computes from then on is thrown away with the call's error.
  const int bar = 1 + (warp & 7);
  auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory"); };
  bool alive = true;
  auto wait_for = [&](uint64_t* b, uint32_t parity) {
    if (alive) alive = wait_warp(b, parity, &t->abort);
  };
  auto exchange = [&](float x) {
    t->peer[warp][lane] = x;
    meet();
    return t->peer[warp ^ 8][lane];
  };
  Cursor c;
  c.begin(a, t);
  const int total = c.left;
  uint32_t s_phase = 0, pv_phase = 0;  // parities of the next completion of s_full and of pv_done
  float m = -INFINITY, l = 0.f, rk = 1.f;
  int limit = 0;  // tokens that the row sees; 0 for a row past the run's last
  bool begins = false, staged = false;
  auto locate = [&](bool& valid, int& tok, long long& out_at) {  // this thread's row of the unit
    const UnitInfo u = *c.at;
    const int r = u.u * kRows + half * 128 + row;
    valid = r < u.run.n * a.G;
    tok = valid ? r / a.G : 0;
    out_at = static_cast<long long>(u.run.row0 + tok) * a.Hq + u.kvh * a.G + (valid ? r - tok * a.G : 0);
  };
  auto begin_unit = [&]() {
    bool valid;
    int tok;
    long long out_at;
    locate(valid, tok, out_at);
    const RunInfo run = c.at->run;
    limit = valid ? max(run.len - run.n + tok + 1, 0) : 0;
    begins = c.j == 0;
    m = -INFINITY;
    l = 0.f;
    const long long row_at = static_cast<long long>(run.row0 + tok);
    meet();  // the peer has read what the last exchange left
    stage_query(static_cast<const uint16_t*>(a.q), valid ? row_at * a.q_stride + (out_at - row_at * a.Hq) * kHeadDim : -1, a.sm_scale,
                smem + kOffQ + half * kOperand, (warp & 3) * 32, part, t->peer[warp & 7]);
    meet();
    rk = t->peer[warp & 7][lane];
    __syncwarp();
    if (alive && lane == 0) arrive(&t->q_full[half]);
    staged = true;
  };
#pragma unroll 1
  for (int jj = 0; jj < total; ++jj) {
    if (half >= c.halves()) {  // 128 rows or fewer: the other half's alone
      c.advance(a);
      continue;
    }
    if (!staged) begin_unit();
    wait_for(&t->s_full[half], s_phase);
    s_phase ^= 1u;
    fence_after();
    const float2* scale = t->scale[jj % kScaleSlots] + 4 * part;
    const int seen = limit - c.j * kKeys - 64 * part;  // of this thread's 64 keys
    const bool masked = __any_sync(dec::kFull, seen < 64);
    float tm = masked ? row_max_masked(ts, scale, rk, seen) : row_max(ts, scale, rk);
    tm = fmaxf(tm, exchange(tm));
    if (c.first) {
      m = tm;
    } else {  // the running maximum moves only when a row outgrows it by 2^kSlack
      const bool move = tm > m + kSlack || (m == -INFINITY && tm > m);
      if (__any_sync(dec::kFull, move)) {
        wait_for(&t->pv_done[half], pv_phase ^ 1u);  // O is the previous tiles' sum
        fence_after();
        const float alpha = !move ? 1.f : m == -INFINITY ? 0.f : ex2(m - tm);
        m = move ? tm : m;
        l *= alpha;
        rescale_o(to, alpha);
      }
    }
    const float base = kTileShift - (m == -INFINITY ? 0.f : m);
    l += masked ? weights<true>(ts, scale, rk, base, seen) : weights<false>(ts, scale, rk, base, 0);
    wait_st();
    fence_before();
    __syncwarp();
    if (alive && lane == 0) arrive(&t->p_full[half]);
    const uint32_t parity = pv_phase;  // of this tile's PV
    pv_phase ^= 1u;
    if (!c.last()) {
      c.advance(a);
      continue;
    }
    const bool whole = begins && c.j + 1 == c.tiles();
    if (threadIdx.x == 0 && begins && !whole) {  // the unit began here and goes on in the next CTA
      rec[1] = c.at->s;
      rec[2] = c.at->kvh;
      rec[3] = c.at->u;
      rec[0] = 1;
    }
    const float m0 = m;
    meet();  // the peer has read the tile's maximum
    const float l0 = l + exchange(l);
    const size_t piece = static_cast<size_t>(2 * blockIdx.x + (begins ? 1 : 0)) * kRows + half * 128 + row;
    bool valid;
    int tok;
    long long out_at;
    locate(valid, tok, out_at);
    c.advance(a);
    staged = false;
    if (jj + 1 < total && half < c.halves()) begin_unit();
    wait_for(&t->pv_done[half], parity);
    fence_after();
    valid = valid && alive;
    if (whole) {
      store_out(to, l0 == 0.f ? 0.f : 1.f / l0, static_cast<uint16_t*>(a.out) + out_at * kHeadDim + 64 * part, valid);
      if (a.lse && valid && part == 0) a.lse[out_at] = l0 == 0.f ? -INFINITY : (m0 + (log2f(l0) - kTileShift)) * dec::kLn2;
    } else {
      store_piece(to, a.tw_acc + piece * kHeadDim + 64 * part);
      if (part == 0) *reinterpret_cast<float2*>(a.tw_stats + piece * 2) = make_float2(m0, l0);
    }
    fence_before();
  }
}

// tw_rec of a CTA: [0] a unit begins here and goes on in the next CTA, [1..3] that unit, [4] the unit that began in an
// earlier CTA ends here.
template <bool INT8>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint8_t* smem = smem_raw;
  Tail* t = reinterpret_cast<Tail*>(smem + kOffTail);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) t->abort = 0;
  plan(a, t, reinterpret_cast<long long*>(smem + kOffRing), reinterpret_cast<int*>(smem + kOffRing + 8 * (kMaxBatch + 1)));
  int32_t* rec = a.tw_rec + 8 * blockIdx.x;
  if (t->n == 0) {  // fewer tiles than CTAs
    if (threadIdx.x == 0) {
      rec[0] = rec[4] = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      dec::mbar_init(&t->full[i], 8);
      dec::mbar_init(&t->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      dec::mbar_init(&t->q_full[i], 8);
      dec::mbar_init(&t->s_full[i], 1);
      dec::mbar_init(&t->p_full[i], 8);
      dec::mbar_init(&t->pv_done[i], 1);
    }
    dec::mbar_init(&t->drained, 1);
    dec::fence_mbar_init();
    // which pieces of this CTA the merge has to look at
    const int first_tiles = tiles_of(a, run_info(a, t->start[0]), t->start[2]);
    rec[4] = t->start[3] > 0 && t->start[3] + t->n >= first_tiles;
    rec[0] = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&t->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = t->tmem;
  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_role(a, t, smem, tmem, rec);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    convert_role<INT8>(a, t, smem + kOffRing);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kMmaWarp) {
      const uint32_t leader = dec::elect_one();
      mma_role(t, smem_u32(smem), tmem, leader);
      // However the role ended: TMEM and shared memory are given back when the last product that it issued is through with
      // them (products wait for nothing; the limit is there all the same).
      commit(&t->drained, leader);
      const long long t0 = clock64();
      while (!__all_sync(dec::kFull, dec::mbar_try_wait(&t->drained, 0)))
        if (__any_sync(dec::kFull, clock64() - t0 > kWaitClocks)) {
          *reinterpret_cast<volatile int*>(&t->abort) = 1;
          break;
        }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (threadIdx.x == 0) {
    if (t->abort) report(a.err, KVQ_ERR_TIMEOUT);
    // This grid may have run beside the short runs' kernels; it does not end before they do, so that whatever waits for it
    // waits for them.
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// The units that more than one CTA worked on: warp i of block (c, .) merges row i of the unit that began in CTA c.
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
#pragma unroll 4
  for (int k = c; k <= end; ++k) {
    const float2 st = stats_of(k);
    const float4 v = acc_of(k);
    const float mn = fmaxf(m, st.x);
    const float f0 = m == -INFINITY ? 0.f : ex2(m - mn), f1 = st.x == -INFINITY ? (st.y == 0.f ? 0.f : 1.f) : ex2(st.x - mn);
    m = mn;
    l = l * f0 + st.y * f1;
    acc.x = acc.x * f0 + v.x * f1;
    acc.y = acc.y * f0 + v.y * f1;
    acc.z = acc.z * f0 + v.z * f1;
    acc.w = acc.w * f0 + v.w * f1;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int head = unit.z * a.G + r % a.G;
  const long long at = static_cast<long long>(run.row0 + r / a.G) * a.Hq + head;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * kHeadDim + 4 * lane) =
      make_uint2(dec::pack_bf16(acc.x * inv, acc.y * inv), dec::pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + (log2f(l) - kTileShift)) * dec::kLn2;
}

}  // namespace

size_t tile_workspace(int sms, size_t* acc, size_t* stats, size_t* rec) {
  *rec = 0;
  *stats = 8 * sizeof(int32_t) * static_cast<size_t>(sms);
  *stats = (*stats + 255) & ~static_cast<size_t>(255);
  *acc = *stats + static_cast<size_t>(sms) * 2 * kRows * 2 * sizeof(float);
  return *acc + static_cast<size_t>(sms) * 2 * kRows * kHeadDim * sizeof(float);
}

cudaError_t launch_tile(AttnArgs& a, bool int8, int sms, cudaStream_t s) {
  auto kern = int8 ? tile_kernel<true> : tile_kernel<false>;
  static bool configured[2][kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !configured[int8][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) configured[int8][dev] = true;
  }
  a.tile_ctas = sms;
  // A unit's own cost in tiles, by ranges ending together on a prompt of 2000 tokens (85.3, 83.9, 82.9 us with 2, 3, 4) and of
  // 11996 (1192, 1188, 1186 us); with a unit counted as nothing the ranges of short units ended 40 % behind the others.
  a.unit_cost = 4;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(static_cast<unsigned>(sms), kRows / 8);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, tile_merge_kernel, a);
}

}  // namespace runs
}  // namespace kvq
