// attn_tree_tile.cu -- kvq_attn_tree for BF16 queries of more than a few rows: tcgen05 products.
//
// A unit is one (request, kv head, 128 consecutive (token, head) rows); its key tiles are the 128-token tiles of the whole context.  A tree's rows are
// few beside its context, so the tiles are what the cache costs to bring: 32.8 KB from HBM, 1,520 clocks of an SM's share of the copy
// rate.  The layout aims at that and comes to about 2,400:
//   * the query lies in TMEM (the first operand of S = Q K^T), so all shared memory is a ring of six operand tiles;
//   * S has two buffers in TMEM and O one: while the softmax works on a tile, the next one's S and the last one's P V run (512 clocks each);
//   * four threads have a row, 32 keys each, and keep their S in registers: one read of TMEM a tile;
//   * the running maximum moves only where a row outgrows it by 2^8; whether any row does is one barrier with a vote among the four warps of
//     32 rows, so the maximum itself is exchanged, and O rescaled, only then;
//   * codes of K and V are loaded a whole tile ahead (eight words of 16 bytes a thread), and a warp of its own looks several tiles ahead and has
//     the L2 bring them;
//   * of the masks only those words are read that say something of the tile: tokens before the run are seen by all.
//
// Bound by the warps' work together: converting 16 K codes of K and V and handing them on is about 1,750 clocks a tile with nothing beside it, the
// softmax's chain (maximum 600, weights 1,200, waits) about 2,300.  16 trees of 9..16 tokens over 11500, 8 and 32 heads, E4M3: 114 us, 3,340 GB/s; 64 trees
// of 25..64 over 2000..8192, 4 and 28 heads, INT8: 246 us.  A call's start (10 us to the first weights) and end (9 us from the last tile through the
// merge) are about what a single request over 300 tokens takes, 15 to 17 us.  Slower, where this form took 117 for the first of the two and 250
// for the second: two teams of softmax warps with an O each 122 and 269; half tiles for two, three or four teams with one O, S and P V issued by
// two warps, 153, 143, 128 and 297, 292, 263; K and V converted by warps of their own 121 and 261; lookups by the converting warps themselves
// 150 and 335.
//
// TMEM columns: S (and P, over the first half of each 32 columns) twice 128, O 128, Q 64.
// Warps: 0-15 softmax (rows 32 (w & 3) .., keys 32 (w >> 2) .. of a tile), 16-23 convert, 24 issues the products, 25 looks ahead.
// Operand layouts, key order inside a tile, scales in the exponent: as in attn_runs_tile.cu.
#include "attn_tile.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kRows = 128;      // rows of a unit
constexpr int kSlots = 6;       // ring of operand tiles
constexpr int kOperand = 32768;  // 128 x 128 fp16
constexpr int kSoftmaxWarps = 16, kConvertWarp = 16, kMmaWarp = 24, kScoutWarp = 25;  // first warps of the roles
constexpr int kThreads = 28 * 32;
// Registers: 72 a thread at launch; the softmax warps take what the last warpgroup, of which only two warps work, gives back.  None of the loops
// may spill (with 72 the softmax does).
constexpr int kRegsSoftmax = 80, kRegsConvert = 72, kRegsMma = 40;
static_assert(16 * kRegsSoftmax + 8 * kRegsConvert + 4 * kRegsMma <= 28 * 72, "no more than the block was launched with");
// Descriptions of key tiles, written by the scout four (a group) at a time.  A tile's is read last by its softmax, which is over when the third tile
// after it has been converted (V of that one waits for its V slot): with four groups, one is written again when the group after it is done.
constexpr int kGroup = 4, kGroups = 4, kDescs = kGroup * kGroups;
constexpr int kOffTail = kSlots * kOperand, kTailBytes = 10 * 1024;
constexpr int kSmemBytes = kOffTail + kTailBytes;
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemQ = 384;

struct Desc {  // of a key tile
  float2 scale[kPagesPerTile];   // 2^ek |sm_scale| log2 e, ev (0, -inf for an absent page)
  uint32_t tile[kPagesPerTile];  // page Hkv + kv head; an absent page's (behind the context, or outside the cache) is read as page 0 and cleared
  int lost, in_context;          // absent pages; tokens that the context has from the tile's first on
  int flags, pad;                // kFirst, kLast
};
struct Tail {  // shared memory behind the operands
  Desc desc[kDescs];
  uint64_t full[kSlots], empty[kSlots];
  // Of the tiles in turn.  A parity tells apart only a phase and the one before it: when a warp is at a tile, the P V of the tile before
  // may be running still (this tile's S went ahead of it) or this tile's be over, so one barrier would not do.
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full;
  uint64_t desc_full[kGroups], desc_done[kGroups];
  uint64_t drained;  // every product of the CTA
  uint32_t tmem;
  int abort;
  UnitInfo unit[kScoutWarp + 1];  // where each warp is
  int start[4];             // request, kv head, unit, first tile of the CTA's range
  int n;                    // its tiles
  // What the four threads of a row tell each other: maxima of a tile (two in turn), then sums or exponents.
  float peer_m[2][4][kRows], peer[4][kRows];
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
__device__ void mma_role(Tail* t, uint32_t smem_base, uint32_t tmem, uint32_t leader) {
  tmem = dec::uniform_u32(tmem);
  const uint64_t ring = smem_desc(smem_base);
  // Eight steps of 16: 32 bytes apart inside a 64-element column of rows, the second column 16 KB on; the weights of 32 keys lie in the first
  // half of those 32 columns of S.
  auto k_step = [](int ks) { return static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4); };
  const int total = dec::uniform_u32(t->n);
  int slot = 0;  // of the operand tile taken next
  uint32_t phase = 0, q_phase = 0;
  auto next_slot = [&]() {
    if (++slot == kSlots) { slot = 0; phase ^= 1u; }
  };
  // S of tile `tile`, whose K is in `slot`; its flags, or -1 where a wait gave up.
  auto score = [&](int tile, int k_slot, uint32_t k_phase) {
    if (!wait_warp(&t->full[k_slot], k_phase, &t->abort)) return -1;
    const int flags = dec::uniform_u32(*reinterpret_cast<volatile int*>(&t->desc[tile % kDescs].flags));
    if (flags & kFirst) {
      if (!wait_warp(&t->q_full, q_phase, &t->abort)) return -1;
      q_phase ^= 1u;
    }
    fence_after();
    const uint64_t y = ring + static_cast<uint64_t>(k_slot * (kOperand >> 4));
    const uint32_t s = tmem + kTmemS + 128 * (tile & 1);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) mma_ts(s, tmem + kTmemQ + 8 * ks, y + k_step(ks), ks > 0, leader);
    commit(&t->s_full[tile & 1], leader);
    commit(&t->empty[k_slot], leader);
    return flags;
  };
  int flags = score(0, 0, 0);
  if (flags < 0) return;
  next_slot();
#pragma unroll 1
  for (int tile = 0; tile < total; ++tile) {
    const int v_slot = slot;
    const uint32_t v_phase = phase;
    next_slot();
    // The next tile's S goes before this one's P V while it belongs to the same piece (the next piece's query comes with this tile's end).
    int next_flags = 0;
    const bool last = (flags & kLast) != 0, more = tile + 1 < total;
    if (more && !last) {
      next_flags = score(tile + 1, slot, phase);
      if (next_flags < 0) return;
    }
    if (!wait_warp(&t->p_full[tile & 1], (tile >> 1) & 1u, &t->abort)) return;
    if (!wait_warp(&t->full[v_slot], v_phase, &t->abort)) return;
    fence_after();
    const uint64_t y = ring + static_cast<uint64_t>(v_slot * (kOperand >> 4));
    const uint32_t p = tmem + kTmemS + 128 * (tile & 1);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      mma_ts(tmem + kTmemO, p + 32 * (ks >> 1) + 8 * (ks & 1), y + k_step(ks), !(flags & kFirst) || ks > 0, leader);
    commit(&t->pv_done[tile & 1], leader);
    commit(&t->empty[v_slot], leader);
    if (more && last) {
      next_flags = score(tile + 1, slot, phase);
      if (next_flags < 0) return;
    }
    if (more) next_slot();
    flags = next_flags;
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
// goes on to the end of its range all the same, without waiting or handing anything on: the four warps of a row take every meeting that the range
// has.  What it computes from then on is thrown away with the call's error.
__device__ void softmax_role(const AttnArgs& a, Tail* t, uint32_t tmem, int32_t* rec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp >> 2;                  // keys 32 part .. of a tile, channels 32 part ..
  const int row = (warp & 3) * 32 + lane;      // of the unit
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp & 3)
  const uint32_t ts = tmem + kTmemS + 32 * part + lanes, to = tmem + kTmemO + 32 * part + lanes;
  const int bar = 1 + (warp & 3);
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); };
  auto meet_any = [&](bool x) {  // whether any thread of the four warps says so
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)), "r"(bar) : "memory");
    return r != 0;
  };
  bool alive = true;
  auto wait_for = [&](uint64_t* b, uint32_t parity) {
    if (alive) alive = wait_warp(b, parity, &t->abort);
  };
  Cursor<Tree> c;
  c.begin(a, t);
  const int total = c.left;
  float m = -INFINITY, l = 0.f, rk = 1.f;
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
  // The row times a power of two, its largest element in [2^8, 2^9) (bf16 elements are then exact in fp16 down to 2^-22 of it), to TMEM.
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
    active = c.at->u * kRows + (warp & 3) * 32 < run.n * a.G;
    m = -INFINITY;
    l = 0.f;
    if (active) {
      uint32_t u[16];
      const long long row_at = static_cast<long long>(run.row0 + tok);
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + row_at * a.q_stride + (out_at - row_at * a.Hq) * kHeadDim + 32 * part;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = valid ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        u[4 * i] = w.x; u[4 * i + 1] = w.y; u[4 * i + 2] = w.z; u[4 * i + 3] = w.w;
      }
      uint32_t top = 0;  // largest exponent field
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max(top, max((u[e] >> 7) & 0xFFu, (u[e] >> 23) & 0xFFu));
      meet();  // the others have read what the last meeting left
      t->peer[part][row] = static_cast<float>(top);
      meet();
      const float all = fmaxf(fmaxf(t->peer[0][row], t->peer[1][row]), fmaxf(t->peer[2][row], t->peer[3][row]));
      const int er = min(max(static_cast<int>(all) - 127 - 8, -100), 120);
      const float f = copysignf(exp2_int(-er), a.sm_scale);  // a negative scale goes into the query
#pragma unroll
      for (int e = 0; e < 16; ++e) u[e] = dec::pack_f16(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f);
      rk = exp2_int(er);
      tmem_st16(tmem + kTmemQ + 16 * part + lanes, u);
      wait_st();
    }
    fence_before();
    __syncwarp();
    if (alive && lane == 0) arrive(&t->q_full);
  };
  begin_unit();
#pragma unroll 1
  for (int jj = 0; jj < total; ++jj) {
    const int buf = jj & 1;
    wait_for(&t->s_full[buf], (jj >> 1) & 1u);
    fence_after();
    if (active) {
      float s[32];
      tmem_ld32(ts + 128 * buf, s);
      const float4 sc = *reinterpret_cast<const float4*>(t->desc[jj % kDescs].scale + 2 * part);
      // y = S k + e of the two pages; k >= 0, so a page's largest S gives its largest y
      float k0 = sc.x * rk, k1 = sc.z * rk, e0 = sc.y, e1 = sc.w;
      wait_ld();
      loaded<32>(s);
      const int p0 = c.j * kKeys + 32 * part;  // position of the thread's first page
      if (p0 + 2 * kPage > ctx) {  // the same in all lanes of the warp
        const uint32_t b0 = mask_row < 0 ? 0 : page_bits(a, mask_row, p0, ctx, end), b1 = mask_row < 0 ? 0 : page_bits(a, mask_row, p0 + kPage, ctx, end);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float y = (e >> 2) & 1 ? fmaf(s[e], k1, e1) : fmaf(s[e], k0, e0);
          s[e] = ((e >> 2) & 1 ? b1 : b0) >> col_token(e) & 1u ? y : -INFINITY;
        }
        k0 = k1 = 1.f;
        e0 = e1 = 0.f;
      }
      float pm[2];
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const float* x = s + 4 * par;  // columns 0..3, 8..11, 16..19, 24..27 from here
        const float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[8], x[9]), m2 = max3(x[10], x[11], x[16]);
        const float m3 = max3(x[17], x[18], x[19]), m4 = max3(x[24], x[25], x[26]);
        pm[par] = fmaxf(max3(m0, m1, m2), max3(m3, m4, x[27]));
      }
      const float tm = fmaxf(fmaf(pm[0], k0, e0), fmaf(pm[1], k1, e1));
      t->peer_m[buf][part][row] = tm;
      if (meet_any(tm > m + kSlack)) {
        const float all = fmaxf(fmaxf(t->peer_m[buf][0][row], t->peer_m[buf][1][row]), fmaxf(t->peer_m[buf][2][row], t->peer_m[buf][3][row]));
        const bool move = all > m + kSlack;
        if (!c.first && __any_sync(dec::kFull, move)) {
          wait_for(&t->pv_done[buf ^ 1], ((jj - 1) >> 1) & 1u);  // O is the previous tiles' sum
          fence_after();
          const float alpha = !move ? 1.f : m == -INFINITY ? 0.f : ex2(m - all);
          l *= alpha;
          rescale_o<32>(to, alpha);
        }
        m = move ? all : m;
      }
      const float base = kTileShift - (m == -INFINITY ? 0.f : m);
      const dec::f2x k2[2] = {dec::f2_splat(k0), dec::f2_splat(k1)};
      const dec::f2x b2[2] = {dec::f2_splat(e0 + base), dec::f2_splat(e1 + base)};
      const float un[2] = {sc.y == -INFINITY ? 0.f : ex2(-sc.y), sc.w == -INFINITY ? 0.f : ex2(-sc.w)};
      dec::f2x sum[2];
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const int par = (e >> 2) & 1;
        float y0, y1;
        dec::f2_unpack(dec::f2_fma(dec::f2_pack(s[e], s[e + 1]), k2[par], b2[par]), y0, y1);
        const float w0 = ex2(y0), w1 = ex2(y1);
        const dec::f2x w2 = dec::f2_pack(w0, w1);
        sum[par] = (e & ~4) == 0 ? w2 : dec::f2_add(sum[par], w2);
        pk[e >> 1] = dec::pack_f16(w0, w1);
      }
      tmem_st16(ts + 128 * buf, pk);
      float l0, l1, l2, l3;
      dec::f2_unpack(sum[0], l0, l1);
      dec::f2_unpack(sum[1], l2, l3);
      l = fmaf(l0 + l1, un[0], fmaf(l2 + l3, un[1], l));
      wait_st();
    }
    fence_before();
    __syncwarp();
    if (alive && lane == 0) arrive(&t->p_full[buf]);
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
    const float m0 = m;
    float l0 = 0.f;
    if (had) {
      meet();  // the others have read what the last meeting left
      t->peer[part][row] = l;
      meet();
      l0 = (t->peer[0][row] + t->peer[1][row]) + (t->peer[2][row] + t->peer[3][row]);
    }
    const size_t piece = static_cast<size_t>(2 * blockIdx.x + (begins ? 1 : 0)) * kRows + row;
    bool valid;
    int tok;
    long long out_at;
    locate(valid, tok, out_at);
    c.advance(a);
    if (jj + 1 < total) begin_unit();
    wait_for(&t->pv_done[buf], (jj >> 1) & 1u);
    fence_after();
    valid = valid && alive;
    if (had) {
      if (whole) {
        store_out<32>(to, l0 == 0.f ? 0.f : 1.f / l0, static_cast<uint16_t*>(a.out) + out_at * kHeadDim + 32 * part, valid);
        if (a.lse && valid && part == 0) a.lse[out_at] = l0 == 0.f ? -INFINITY : (m0 + (log2f(l0) - kTileShift)) * dec::kLn2;
      } else {
        store_piece<32>(to, a.tw_acc + piece * kHeadDim + 32 * part);
        if (part == 0) *reinterpret_cast<float2*>(a.tw_stats + piece * 2) = make_float2(m0, l0);
      }
    }
    fence_before();
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
    for (int i = 0; i < 2; ++i) {
      dec::mbar_init(&t->s_full[i], 1);
      dec::mbar_init(&t->p_full[i], kSoftmaxWarps);
      dec::mbar_init(&t->pv_done[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      dec::mbar_init(&t->desc_full[i], 1);
      dec::mbar_init(&t->desc_done[i], 8);
    }
    dec::mbar_init(&t->q_full, kSoftmaxWarps);
    dec::mbar_init(&t->drained, 1);
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
  // A unit's own cost in tiles.  16 trees of up to 64 rows over 11000..11996 tokens and 64 trees of up to 448 over up to 8192, in a graph: 117 and 272 us
  // with 0, 117 and 262 with 1, 117 and 257 with 2, 116 and 248 with 3, 115 and 247 with 4, 115 and 249 with 6, 121 and 253 with 8.
  a.unit_cost = 4;
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
  return cudaLaunchKernelEx(&cfg, tile_merge_kernel<kRows, 4>, a);
}

}  // namespace runs
}  // namespace kvq
