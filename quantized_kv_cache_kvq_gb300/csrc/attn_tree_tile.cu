// attn_tree_tile.cu -- kvq_attn_tree for BF16 queries of more than a few rows: tcgen05 products.
//
// A unit is one (request, kv head, 128 consecutive (token, head) rows); its key tiles are the 128-token tiles of the whole context.  A tree's rows are
// few beside its context, so the tiles are what the cache costs to bring: 32.8 KB from HBM, 1,520 clocks of an SM's share of the copy
// rate.  Everything else is laid out to stay below that:
//   * the query lies in TMEM (the first operand of S = Q K^T), so all shared memory is a ring of six operand tiles;
//   * the softmax takes half tiles of 64 keys: four teams of four warps (a thread has a row) take them in turn and S has five buffers, so that
//     the exponentials never wait for a product or a barrier;
//   * O is one accumulator for all teams.  Its reference, a row's running maximum, goes from a half tile to the next through shared memory; it moves
//     only where a row outgrows it by 2^8, and only then is O rescaled, when all P V so far are through;
//   * one warp issues S, another P V, each as soon as its operands are there;
//   * codes of K and V are loaded a whole tile ahead (eight words of 16 bytes a thread), and a warp of its own looks several tiles ahead and has
//     the L2 bring them;
//   * of the masks only those words are read that say something of the tile: tokens before the run are seen by all.
//
// TMEM columns: S (and P, over the first half of each) five times 64, Q 64, O 128.
// Warps: 0-15 softmax (team w >> 2, rows 32 (w & 3) ..), 16-23 convert, 24 issues S, 25 looks ahead, 26 issues P V.
// Operand layouts, key order inside a tile, scales in the exponent: as in attn_runs_tile.cu.
#include "attn_tile.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kRows = 128;      // rows of a unit
constexpr int kSlots = 6;       // ring of operand tiles
constexpr int kOperand = 32768;  // 128 x 128 fp16
constexpr int kSoftmaxWarps = 16, kConvertWarp = 16, kMmaWarp = 24, kScoutWarp = 25, kPvWarp = 26;  // first warps of the roles
constexpr int kThreads = 28 * 32;
// Registers: 72 a thread at launch; the softmax warps take what the last warpgroup, of which only one warp works, gives back.  None of the loops
// may spill (with 72 the softmax does).
constexpr int kRegsSoftmax = 80, kRegsConvert = 72, kRegsMma = 40;
static_assert(16 * kRegsSoftmax + 8 * kRegsConvert + 4 * kRegsMma <= 28 * 72, "no more than the block was launched with");
// Descriptions of key tiles, written by the scout four (a group) at a time.  A tile's is read last by its softmax, which is over when the third tile
// after it has been converted (V of that one waits for its V slot): with four groups, one is written again when the group after it is done.
constexpr int kGroup = 4, kGroups = 4, kDescs = kGroup * kGroups;
constexpr int kOffTail = kSlots * kOperand, kTailBytes = 10 * 1024;
constexpr int kSmemBytes = kOffTail + kTailBytes;
constexpr int kBufs = 5;  // of S
constexpr uint32_t kTmemS = 0, kTmemQ = 320, kTmemO = 384;

struct Desc {  // of a key tile
  float2 scale[kPagesPerTile];   // 2^ek |sm_scale| log2 e, ev (0, -inf for an absent page)
  uint32_t tile[kPagesPerTile];  // page Hkv + kv head; an absent page's (behind the context, or outside the cache) is read as page 0 and cleared
  int lost, in_context;          // absent pages; tokens that the context has from the tile's first on
  int flags, pad;                // kFirst, kLast
};
struct Tail {  // shared memory behind the operands
  Desc desc[kDescs];
  uint64_t full[kSlots], empty[kSlots];
  // Of the half tiles in turn: S there, weights there, P V done; and of the teams' half tiles, for each 32 rows: the running maximum there.
  // (A parity tells apart only a phase and the one before it: tests/test_tree_tile_waits.py goes through the waits.)
  uint64_t s_full[kBufs], p_full[kBufs], pv_done[kBufs], m_ready[4][4];
  uint64_t q_full;
  uint64_t desc_full[kGroups], desc_done[kGroups];
  uint64_t drained;  // every product of the CTA
  uint32_t tmem;
  int abort;
  UnitInfo unit[kScoutWarp + 1];  // where each warp is
  int start[4];             // request, kv head, unit, first tile of the CTA's range
  int n;                    // its tiles
  float m[kRows];         // a row's running maximum, O's reference
  float peer[4][kRows];   // what the four threads of a row tell each other about its query
  float2 ends[4][kRows];  // references and sums of a row's four threads at the end of a piece
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");
struct Tree {
  static constexpr int kRows = runs::kRows, kThreads = runs::kThreads;
  static constexpr bool kTree = true;
  using Tail = runs::Tail;
};

// ------------------------------------------------------------------------------------------------ scout
// One warp looks ahead of the converting warps: block-table entries, scales and flags of four tiles at a time (a page a lane), and a hint to
// the L2 to bring their codes.  (With the lookups in every converting warp, a loop's moves waited for loads that were only to be needed
// two tiles on: 1,700 of a tile's 4,400 clocks.)
__device__ void scout_role(const AttnArgs& a, Tail* t) {
  const int lane = threadIdx.x & 31, mine = lane >> 3, page = lane & 7;
  Cursor<Tree> c;
  c.begin(a, t);
  const int total = c.left;
  for (int g = 0; g * kGroup < total; ++g) {
    int entry = 0, kvh = 0, in_context = 0, flags = 0;
    bool there = false;  // the lane has a tile
#pragma unroll 1
    for (int i = 0; i < kGroup && g * kGroup + i < total; ++i) {
      if (i == mine) {
        const int p = c.j * kPagesPerTile + page;
        there = true;
        in_context = c.at->run.len - c.j * kKeys;
        kvh = c.at->kvh;
        flags = (c.first ? kFirst : 0) | (c.last() ? kLast : 0);
        if (page * kPage < in_context) entry = a.block_table[static_cast<size_t>(c.at->s) * a.max_pages + p];
      }
      c.advance(a);
    }
    const bool here = there && page * kPage < in_context, known = entry >= 0 && entry < a.num_pages;
    if (here && !known) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    const uint32_t tile = known ? static_cast<uint32_t>(entry) * a.Hkv + kvh : kvh;
    uint16_t ks = 0, vs = 0;
    if (here && known) {
      const size_t si = static_cast<size_t>(kvh) * a.num_pages + entry;
      ks = a.ks[si];
      vs = a.vs[si];
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.k + static_cast<uint64_t>(tile) * 2048), "r"(2048) : "memory");
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.v + static_cast<uint64_t>(tile) * 2048), "r"(2048) : "memory");
    }
    if (g >= kGroups - 1 && !wait_warp(&t->desc_done[(g - (kGroups - 1)) % kGroups], ((g - (kGroups - 1)) / kGroups) & 1u, &t->abort)) return;
    const unsigned lost = __ballot_sync(dec::kFull, !here || !known) >> (8 * mine) & 0xFFu;
    if (there) {
      Desc& d = t->desc[(g * kGroup + mine) % kDescs];
      d.scale[page] = here && known ? make_float2(fabsf(a.sm_scale) * dec::kLog2e * exp2_int(f16_to_exp(ks)), static_cast<float>(f16_to_exp(vs)))
                                    : make_float2(0.f, -INFINITY);
      d.tile[page] = tile;
      if (page == 0) {
        d.lost = lost;
        d.in_context = in_context;
        d.flags = flags;
      }
    }
    __syncwarp();
    if (lane == 0) arrive(&t->desc_full[g % kGroups]);
  }
}

// ------------------------------------------------------------------------------------------------ converting warps
template <bool INT8>
__device__ void convert_role(const AttnArgs& a, Tail* t, uint8_t* ring) {
  const int cw = (threadIdx.x >> 5) - kConvertWarp, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  constexpr uint32_t kZero = INT8 ? 0x80808080u : 0u;
  // Codes are loaded one tile ahead: where a word has been converted, its register takes the next tile's.
  uint4 kb[4], vb[4];
  // K: page cw, four words of 512 bytes.  V: channels 32 mm .. of the pages 4 quad .., odd rows taking the pairs of pages crosswise.
  const int mm = cw & 3, quad = cw >> 2;
  const uint8_t* k_base = a.k + lane * 16;
  const uint8_t* v_base = a.v + (mm * 32 + lane) * 16;
  auto load_k = [&](const Desc& d) { return k_base + static_cast<uint64_t>(d.tile[cw]) * 2048; };
  auto load_v = [&](const Desc& d, int i) { return ldg_codes(v_base + static_cast<uint64_t>(d.tile[4 * quad + (i ^ (2 * (g & 1)))]) * 2048); };
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
  const int total = t->n;
  if (!wait_warp(&t->desc_full[0], 0, &t->abort)) return;
  {
    const Desc& d = t->desc[0];
    const uint8_t* src = load_k(d);
#pragma unroll
    for (int i = 0; i < 4; ++i) kb[i] = ldg_codes(src + i * 512);
#pragma unroll
    for (int i = 0; i < 4; ++i) vb[i] = load_v(d, i);
  }
#pragma unroll 1
  for (int jj = 0; jj < total; ++jj) {
    const int lost = t->desc[jj % kDescs].lost, in_context = t->desc[jj % kDescs].in_context;
    const int ahead = jj + 1 < total ? jj + 1 : jj;  // behind the last tile: read again and thrown away
    if (ahead % kGroup == 0 && ahead > jj && !wait_warp(&t->desc_full[ahead / kGroup % kGroups], (ahead / kDescs) & 1u, &t->abort)) return;
    const Desc& next = t->desc[ahead % kDescs];
    if (!wait_warp(&t->empty[slot], phase ^ 1u, &t->abort)) return;
    if ((lost >> cw) & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) kb[i] = make_uint4(kZero, kZero, kZero, kZero);
    }
    {
      const uint8_t* src = load_k(next);
      uint8_t* dst = ring + slot * kOperand + k_row * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // word i = (token half, channel half)
        const uint4 x = kb[i];
        const int low = k_low + 2 * (i >> 1);
        uint8_t* base = dst + (i & 1) * 16384 + 2 * (i >> 1) * 128;
        *reinterpret_cast<uint4*>(base + (((2 * q) ^ low) << 4)) =
            make_uint4(codes_lo<INT8>(x.x), codes_hi<INT8>(x.x), codes_lo<INT8>(x.y), codes_hi<INT8>(x.y));
        *reinterpret_cast<uint4*>(base + (((2 * q + 1) ^ low) << 4)) =
            make_uint4(codes_lo<INT8>(x.z), codes_hi<INT8>(x.z), codes_lo<INT8>(x.w), codes_hi<INT8>(x.w));
        kb[i] = ldg_codes(src + i * 512);
      }
    }
    publish();
    if (!wait_warp(&t->empty[slot], phase ^ 1u, &t->abort)) return;
    if (in_context < kKeys || lost) {  // what lies behind the context may be anything, a NaN too
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int page = 4 * quad + (i ^ (2 * (g & 1)));
        const int nvalid = (lost >> page) & 1 ? 0 : in_context - page * kPage;
        auto mask = [&](int tok) { return (tok < nvalid ? 0x00FF00FFu : 0u) | (tok + 1 < nvalid ? 0xFF00FF00u : 0u); };
        const uint32_t m0 = mask(2 * q), m1 = mask(2 * q + 8);
        uint4& w = vb[i];
        w.x = (w.x & m0) | (kZero & ~m0);
        w.z = (w.z & m0) | (kZero & ~m0);
        w.y = (w.y & m1) | (kZero & ~m1);
        w.w = (w.w & m1) | (kZero & ~m1);
      }
    }
    {
      uint8_t* dst = ring + slot * kOperand + v_row * 128 + quad * 16384;
#pragma unroll
      for (int pp = 0; pp < 2; ++pp) {
        const uint4 x = vb[2 * pp], y = vb[2 * pp + 1];
        // pair of pages 2 quad + (pp ^ (g & 1)): column 32 pair + 8 q + {its first page: 0..3, its second: 4..7}
        uint8_t* base = dst + (((4 * ((pp ^ g) & 1) + q) ^ g) << 4);
        *reinterpret_cast<uint4*>(base) = make_uint4(codes_lo<INT8>(x.x), codes_lo<INT8>(x.y), codes_lo<INT8>(y.x), codes_lo<INT8>(y.y));
        *reinterpret_cast<uint4*>(base + 8 * 128) = make_uint4(codes_hi<INT8>(x.x), codes_hi<INT8>(x.y), codes_hi<INT8>(y.x), codes_hi<INT8>(y.y));
        *reinterpret_cast<uint4*>(base + 16 * 128) = make_uint4(codes_lo<INT8>(x.z), codes_lo<INT8>(x.w), codes_lo<INT8>(y.z), codes_lo<INT8>(y.w));
        *reinterpret_cast<uint4*>(base + 24 * 128) = make_uint4(codes_hi<INT8>(x.z), codes_hi<INT8>(x.w), codes_hi<INT8>(y.z), codes_hi<INT8>(y.w));
        vb[2 * pp] = load_v(next, 2 * pp);
        vb[2 * pp + 1] = load_v(next, 2 * pp + 1);
      }
    }
    publish();
    if ((jj % kGroup == kGroup - 1 || jj + 1 == total) && lane == 0) arrive(&t->desc_done[jj / kGroup % kGroups]);
  }
  // the products' last arrivals on the ring land before the CTA may end
  for (int i = 0; i < kSlots && i < 2 * total; ++i) {
    if (--slot < 0) { slot = kSlots - 1; phase ^= 1u; }
    if (!wait_warp(&t->empty[slot], phase, &t->abort)) return;
  }
}

// ------------------------------------------------------------------------------------------------ products
// Steps of 16 channels or keys: 32 bytes apart inside a 64-element column of rows, the second column 16 KB on.
__device__ __forceinline__ uint64_t k_step(int ks) { return static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4); }
// Half tile u: keys 64 (u & 1) .. of tile u >> 1.  S of one is issued when its buffer's last weights have been used.
__device__ void score_role(Tail* t, uint32_t smem_base, uint32_t tmem, uint32_t leader) {
  tmem = dec::uniform_u32(tmem);
  const uint64_t ring = smem_desc(smem_base);
  const int total = dec::uniform_u32(t->n);
  int slot = 0, buf = 0;
  uint32_t phase = 0, q_phase = 0, used = 0;  // used: times that the buffer has been used, mod 2
#pragma unroll 1
  for (int tile = 0; tile < total; ++tile) {
    if (!wait_warp(&t->full[slot], phase, &t->abort)) return;
    const int flags = dec::uniform_u32(*reinterpret_cast<volatile int*>(&t->desc[tile % kDescs].flags));
    if (flags & kFirst) {
      if (!wait_warp(&t->q_full, q_phase, &t->abort)) return;
      q_phase ^= 1u;
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if (2 * tile + half >= kBufs && !wait_warp(&t->pv_done[buf], used ^ 1u, &t->abort)) return;
      fence_after();
      // rows 64 half .. of the K tile: 8 KB on
      const uint64_t y = ring + static_cast<uint64_t>((slot * kOperand + half * 8192) >> 4);
      const uint32_t s = tmem + kTmemS + 64 * buf;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ts<64>(s, tmem + kTmemQ + 8 * ks, y + k_step(ks), ks > 0, leader);
      commit(&t->s_full[buf], leader);
      if (++buf == kBufs) { buf = 0; used ^= 1u; }
    }
    commit(&t->empty[slot], leader);
    slot += 2;
    if (slot >= kSlots) { slot -= kSlots; phase ^= 1u; }
  }
}
__device__ void pv_role(Tail* t, uint32_t smem_base, uint32_t tmem, uint32_t leader) {
  tmem = dec::uniform_u32(tmem);
  const uint64_t ring = smem_desc(smem_base);
  const int total = dec::uniform_u32(t->n);
  int slot = 1, buf = 0;
  uint32_t phase = 0, used = 0;
#pragma unroll 1
  for (int tile = 0; tile < total; ++tile) {
    if (!wait_warp(&t->full[slot], phase, &t->abort)) return;
    const int flags = dec::uniform_u32(*reinterpret_cast<volatile int*>(&t->desc[tile % kDescs].flags));
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if (!wait_warp(&t->p_full[buf], used, &t->abort)) return;
      fence_after();
      // keys 64 half .. of the V tile: its second column of rows
      const uint64_t y = ring + static_cast<uint64_t>((slot * kOperand + half * 16384) >> 4);
      const uint32_t p = tmem + kTmemS + 64 * buf;
      const bool fresh = (flags & kFirst) && half == 0;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma_ts(tmem + kTmemO, p + 8 * ks, y + k_step(ks), !fresh || ks > 0, leader);
      commit(&t->pv_done[buf], leader);
      if (++buf == kBufs) { buf = 0; used ^= 1u; }
    }
    commit(&t->empty[slot], leader);
    slot += 2;
    if (slot >= kSlots) { slot -= kSlots; phase ^= 1u; }
  }
}

// ------------------------------------------------------------------------------------------------ softmax
// What a mask row says about the page at p0 of a context whose run begins at `ctx`: bit t for its token t.
__device__ __forceinline__ uint32_t page_bits(const AttnArgs& a, long long row, int p0, int ctx, int end) {
  const int j = p0 - ctx, w = j >> 5;
  const int32_t* words = a.mask + row * a.mask_words;
  auto word = [&](int i) { return i < 0 ? 0xFFFFFFFFu : i < a.mask_words ? static_cast<uint32_t>(words[i]) : 0u; };
  return __funnelshift_r(word(w), word(w + 1), j & 31) & ((1u << min(max(end - p0, 0), kPage)) - 1);
}

// At the end of a piece the next one's query is staged, so that its first S is issued, before O is stored.  A warp whose wait has given up
// goes on to the end of its range all the same, without waiting or handing anything on: the four warps of 32 rows take every meeting that the range
// has.  What it computes from then on is thrown away with the call's error.
__device__ void softmax_role(const AttnArgs& a, Tail* t, uint32_t tmem, int32_t* rec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp >> 2, quarter = warp & 3;
  const int row = quarter * 32 + lane;  // of the unit
  const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;  // TMEM lane 32 (warp & 3)
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory"); };  // the four warps of 32 rows
  bool alive = true;
  auto wait_for = [&](uint64_t* b, uint32_t parity) {
    if (alive) alive = wait_warp(b, parity, &t->abort);
  };
  auto wait_turn = [&](uint64_t* bars, int u) { wait_for(&bars[u % kBufs], (u / kBufs) & 1u); };  // a half tile's of kBufs in turn
  Cursor<Tree> c;
  c.begin(a, t);
  const int total = c.left;
  float m = -INFINITY, l = 0.f, rk = 1.f;  // the reference of this thread's sum, and that
  int ctx = 0, end = 0;    // the unit's run begins there, its context ends there
  int mask_row = -1;       // this thread's row of the mask, -1 past the run's last
  bool begins = false, active = false;  // the piece has its unit's first tile; the warp has rows
  auto locate = [&](bool& valid, int& tok, long long& out_at) {  // this thread's row of the unit
    const UnitInfo u = *c.at;
    const int r = u.u * kRows + row;
    valid = r < u.run.n * a.G;
    tok = valid ? r / a.G : 0;
    out_at = static_cast<long long>(u.run.row0 + tok) * a.Hq + u.kvh * a.G + (valid ? r - tok * a.G : 0);
  };
  // The row (channels 32 team .. of it) times a power of two, its largest element in [2^8, 2^9) (bf16 elements are then exact in fp16 down to 2^-22
  // of it), to TMEM.
  auto begin_unit = [&]() {
    bool valid;
    int tok;
    long long out_at;
    locate(valid, tok, out_at);
    const RunInfo run = c.at->run;
    ctx = run.len - run.n;
    end = run.len;
    mask_row = valid ? run.row0 + tok : -1;
    begins = c.j == 0;
    active = c.at->u * kRows + quarter * 32 < run.n * a.G;
    m = -INFINITY;
    l = 0.f;
    if (active) {
      uint32_t u[16];
      const long long row_at = static_cast<long long>(run.row0 + tok);
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + row_at * a.q_stride + (out_at - row_at * a.Hq) * kHeadDim + 32 * team;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = valid ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        u[4 * i] = w.x; u[4 * i + 1] = w.y; u[4 * i + 2] = w.z; u[4 * i + 3] = w.w;
      }
      uint32_t top = 0;  // largest exponent field
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max(top, max((u[e] >> 7) & 0xFFu, (u[e] >> 23) & 0xFFu));
      meet();  // the others have read what the last meetings left
      t->peer[team][row] = static_cast<float>(top);
      meet();
      const float all = fmaxf(fmaxf(t->peer[0][row], t->peer[1][row]), fmaxf(t->peer[2][row], t->peer[3][row]));
      const int er = min(max(static_cast<int>(all) - 127 - 8, -100), 120);
      const float f = copysignf(exp2_int(-er), a.sm_scale);  // a negative scale goes into the query
#pragma unroll
      for (int e = 0; e < 16; ++e) u[e] = dec::pack_f16(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f);
      rk = exp2_int(er);
      tmem_st16(tmem + kTmemQ + 16 * team + lanes, u);
      wait_st();
    }
    fence_before();
    __syncwarp();
    if (alive && lane == 0) arrive(&t->q_full);
  };
  begin_unit();
#pragma unroll 1
  for (int jj = 0; jj < total; ++jj) {
    if ((jj & 1) == team >> 1) {
      const int half = team & 1, u = 2 * jj + half;  // u & 3 is the team
      const uint32_t ts = tmem + kTmemS + 64 * (u % kBufs) + lanes;
      const float2* scale = t->desc[jj % kDescs].scale + 4 * half;
      const int p0 = c.j * kKeys + 64 * half;  // position of the half tile's first token
      const bool masked = p0 + 64 > ctx;       // the same in all lanes
      Masked seen{0, 0};
      if (masked && mask_row >= 0) {
        seen.b01 = page_bits(a, mask_row, p0, ctx, end) | page_bits(a, mask_row, p0 + kPage, ctx, end) << 16;
        seen.b23 = page_bits(a, mask_row, p0 + 2 * kPage, ctx, end) | page_bits(a, mask_row, p0 + 3 * kPage, ctx, end) << 16;
      }
      wait_turn(t->s_full, u);
      fence_after();
      float tm = -INFINITY;
      if (active) tm = masked ? row_max_masked(ts, scale, rk, seen) : row_max(ts, scale, rk);
      const bool first = c.first && half == 0;  // of the piece
      if (u > 0) wait_for(&t->m_ready[(u - 1) & 3][quarter], ((u - 1) >> 2) & 1u);
      const float was = first ? -INFINITY : t->m[row];
      const bool move = tm > was + kSlack;
      const float now = move ? tm : was;
      if (active && (first || move)) t->m[row] = now;
      __syncwarp();
      if (alive && lane == 0) arrive(&t->m_ready[team][quarter]);
      if (active) {
        if (!first && __any_sync(dec::kFull, move)) {
          wait_turn(t->pv_done, u - 1);  // O is the sum of the half tiles before
          fence_after();
          rescale_o<128>(tmem + kTmemO + lanes, !move ? 1.f : was == -INFINITY ? 0.f : ex2(was - now));
        }
        if (m != now) {
          l *= m == -INFINITY ? 0.f : ex2(m - now);
          m = now;
        }
        const float base = kTileShift - (m == -INFINITY ? 0.f : m);
        l += masked ? weights<true>(ts, scale, rk, base, seen) : weights<false>(ts, scale, rk, base, seen);
        wait_st();
      }
      fence_before();
      __syncwarp();
      if (alive && lane == 0) arrive(&t->p_full[u % kBufs]);
    }
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
    const bool had = active;
    float top = -INFINITY, sum = 0.f;
    if (had) {
      t->ends[team][row] = make_float2(m, l);
      meet();
      top = t->m[row];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = t->ends[i][row];
        // a sum without a maximum is 0, or no number (of a query that is none), and stays
        sum += x.y * (x.x == -INFINITY ? 1.f : ex2(x.x - top));
      }
    }
    const size_t piece = static_cast<size_t>(2 * blockIdx.x + (begins ? 1 : 0)) * kRows + row;
    bool valid;
    int tok;
    long long out_at;
    locate(valid, tok, out_at);
    c.advance(a);
    wait_turn(t->s_full, 2 * jj + 1);  // the last S: the query in TMEM is free
    if (jj + 1 < total) begin_unit();
    if (had) {  // (warps without rows do not wait: the meeting below is what keeps the barriers from going on to a later phase meanwhile)
      wait_turn(t->pv_done, 2 * jj + 1);
      fence_after();
      valid = valid && alive;
      if (whole) {
        store_out<32>(tmem + kTmemO + 32 * team + lanes, sum == 0.f ? 0.f : 1.f / sum, static_cast<uint16_t*>(a.out) + out_at * kHeadDim + 32 * team, valid);
        if (a.lse && valid && team == 0) a.lse[out_at] = sum == 0.f ? -INFINITY : (top + (log2f(sum) - kTileShift)) * dec::kLn2;
      } else {
        store_piece<32>(tmem + kTmemO + 32 * team + lanes, a.tw_acc + piece * kHeadDim + 32 * team);
        if (team == 0) *reinterpret_cast<float2*>(a.tw_stats + piece * 2) = make_float2(top, sum);
      }
      fence_before();
      meet();  // no team goes on to its next weights before the other three warps have read this O
    }
  }
}

// tw_rec of a CTA: [0] a unit begins here and goes on in the next CTA, [1..3] that unit, [4] the unit that began in an
// earlier CTA ends here.
template <bool INT8>
__global__ void __launch_bounds__(kThreads, 1) tree_tile_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Tail* t = reinterpret_cast<Tail*>(smem + kOffTail);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) t->abort = 0;
  plan<Tree>(a, t, reinterpret_cast<long long*>(smem), reinterpret_cast<int*>(smem + 8 * (kMaxBatch + 1)));
  int32_t* rec = a.tw_rec + 8 * blockIdx.x;
  if (t->n == 0) {  // fewer tiles than CTAs
    if (threadIdx.x == 0) rec[0] = rec[4] = 0;
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      dec::mbar_init(&t->full[i], 8);
      dec::mbar_init(&t->empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      dec::mbar_init(&t->s_full[i], 1);
      dec::mbar_init(&t->p_full[i], 4);
      dec::mbar_init(&t->pv_done[i], 1);
    }
    for (int i = 0; i < 16; ++i) dec::mbar_init(&t->m_ready[i >> 2][i & 3], 1);
    for (int i = 0; i < kGroups; ++i) {
      dec::mbar_init(&t->desc_full[i], 1);
      dec::mbar_init(&t->desc_done[i], 8);
    }
    dec::mbar_init(&t->q_full, kSoftmaxWarps);
    dec::mbar_init(&t->drained, 2);
    dec::fence_mbar_init();
    // which pieces of this CTA the merge has to look at
    const int first_tiles = tiles_of<Tree>(a, run_info(a, t->start[0]), t->start[2]);
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
    softmax_role(a, t, tmem, rec);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    convert_role<INT8>(a, t, smem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kMmaWarp || warp == kPvWarp) {
      const uint32_t leader = dec::elect_one();
      if (warp == kMmaWarp) score_role(t, smem_u32(smem), tmem, leader);
      else pv_role(t, smem_u32(smem), tmem, leader);
      // However the roles ended: TMEM and shared memory are given back when the last products that they issued are through with
      // them (products wait for nothing; the limit is there all the same).
      commit(&t->drained, leader);
      const long long t0 = clock64();
      while (!__all_sync(dec::kFull, dec::mbar_try_wait(&t->drained, 0)))
        if (__any_sync(dec::kFull, clock64() - t0 > 2 * kWaitClocks)) {
          *reinterpret_cast<volatile int*>(&t->abort) = 1;
          break;
        }
    } else if (warp == kScoutWarp) {
      scout_role(a, t);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (threadIdx.x == 0 && t->abort) report(a.err, KVQ_ERR_TIMEOUT);
}

}  // namespace

size_t tree_tile_workspace(int sms, size_t* acc, size_t* stats, size_t* rec) { return pieces_workspace(kRows, sms, acc, stats, rec); }

cudaError_t launch_tree_tile(AttnArgs& a, bool int8, int sms, cudaStream_t s) {
  auto kern = int8 ? tree_tile_kernel<true> : tree_tile_kernel<false>;
  static SmemLimit limit[2];
  cudaError_t e = limit[int8].raise(kern, kSmemBytes);
  if (e != cudaSuccess) return e;
  a.tile_ctas = sms;
  a.unit_cost = 3;
  kern<<<sms, kThreads, kSmemBytes, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(sms), kRows / 8);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, tile_merge_kernel<kRows>, a);
}

}  // namespace runs
}  // namespace kvq
