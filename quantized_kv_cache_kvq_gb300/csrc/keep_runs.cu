// keep_runs.cu -- kvq_keep_runs: the accepted path of every request's tree moved to the front of its run, in the caches of all layers.
//
// The j-th kept token comes from position p0 + keep[j] and goes to p0 + j (p0: where the run began); lists rise, so keep[j] >= j and a page
// takes tokens only from itself and from later ones: a request's pages are rewritten from the first on, each read whole before it is written.
// A page's scale becomes the largest, 2^e, that its tokens had; codes of a token under 2^(e - d) become rne(code 2^-d), as in an append.
//
// One launch for all layers.  A block has one request and a few (layer, kv head) pairs: where every slot's token comes from is looked up once for
// all of them.  A key token is eight 16-byte words of its tile, so a thread moves one word of the new tile; a value word holds four tokens of four
// channels, so a thread puts one together from the words of its four tokens.  Words that stay as they are are read, since a scale that grows
// would change them, but not written.
// A value tile's tokens lie in all of its lines, so moving one token reads and writes 2 KB: 32 requests that keep a path of trees of 25..64 in 36
// layers of 8 heads read 44 MB where the tokens, read and written, are 19 (26.8 us; 2.8 for the tokens at the copy rate), a layer of 4 requests
// takes 8 us.  With one block for each (request, layer, head) and the lookups in each it was 69 us.  The next pair's loads issued a pair
// ahead: 34.  Keys and values by blocks of their own: 33.  Ten blocks on an SM with 48 registers: no change.
#include <algorithm>

#include "codes.cuh"
#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 128;  // a 16-byte word of a tile each
constexpr int kTile = 2048;
constexpr int kMaxLayers = 128;  // of a launch
constexpr int kResident = 8;     // blocks on an SM

struct Planes {
  uint8_t* k;
  uint8_t* v;
  uint16_t* ks;
  uint16_t* vs;
};
struct KeepArgs {
  int H, num_pages, layers;
  const int32_t* run_starts;
  const int32_t* seq_lens;
  const int32_t* block_table;
  const int32_t* keep;
  const int32_t* kept;
  int max_pages, batch, num_rows;
  int32_t* err;
  Planes layer[kMaxLayers];
};

template <bool INT8>
__global__ void __launch_bounds__(kThreads, kResident) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int s_list[KVQ_MAX_TREE];
  __shared__ int s_phys[KVQ_MAX_TREE / kPage + 2];  // pages of the run, from its first token's on
  const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int m = a.kept[s];
  const int r0 = a.run_starts ? a.run_starts[s] : s, r1 = a.run_starts ? a.run_starts[s + 1] : s + 1, len = a.seq_lens[s];
  const int n = r1 - r0, p0 = len - m;
  const bool first = blockIdx.x == 0;
  if (r0 < 0 || r1 < r0 || r1 > a.num_rows || n > KVQ_MAX_TREE || m < 0 || m > n || len < m || len > kMaxContext ||
      static_cast<long long>(p0) + n > static_cast<long long>(a.max_pages) * kPage) {
    if (first && tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  // the list rises and stays in the run; nothing to do where no token moves
  bool bad = false, moves = false;
  for (int j = tid; j < m; j += kThreads) {
    const int i = a.keep[r0 + j], before = j ? a.keep[r0 + j - 1] : -1;
    bad |= i <= before || i >= n;
    moves |= i != j;
    s_list[j] = i;
  }
  bad = __syncthreads_or(bad);
  moves = __syncthreads_or(moves);
  if (bad) {
    if (first && tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  if (!moves) return;
  // pages up to the last kept token's
  const int page0 = p0 / kPage, pages = (p0 + s_list[m - 1]) / kPage - page0 + 1;
  for (int i = tid; i < pages; i += kThreads) {
    const int phys = a.block_table[static_cast<size_t>(s) * a.max_pages + page0 + i];
    bad |= phys < 0 || phys >= a.num_pages;
    s_phys[i] = phys;
  }
  if (__syncthreads_or(bad)) {
    if (first && tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  const int dst_pages = (len - 1) / kPage - page0 + 1;
  const int tk = ((tid >> 6) << 3) | ((tid >> 2) & 7), q = tid & 3;  // the key word's token; the value word's are 2 q, 2 q + 1, 2 q + 8, 2 q + 9
  const int pairs = a.H * a.layers;
  for (int d = 0; d < dst_pages; ++d) {
    const int at = (page0 + d) * kPage;        // position of the page's first token
    const int from = max(0, p0 - at), to = min(kPage, len - at);  // kept tokens of the run
    if (s_list[at + to - 1 - p0] == at + to - 1 - p0) continue;  // the list rises: nothing moves before it either
    // Where slot t's token is, counted from the run's first page on; -1: behind the last token.
    auto source = [&](int t) { return t >= to ? -1 : t < from ? at + t - page0 * kPage : p0 + s_list[at + t - p0] - page0 * kPage; };
    const int self = d * kPage;  // slot 0 of the page in that count
    const int sk = source(tk);
    int sv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = source(2 * q + (i & 1) + 8 * (i >> 1));
    const bool v_stays = sv[0] == self + 2 * q && sv[1] == self + 2 * q + 1 && sv[2] == self + 2 * q + 8 && sv[3] == self + 2 * q + 9;
    const int mine = source(lane & 15);  // lanes 0..15 look up the keys' scales, the others the values'
    auto phys_of = [&](int src) { return s_phys[src >> 4]; };
    constexpr uint32_t kZero = INT8 ? 0x80808080u : 0u;
#pragma unroll 1
    for (int pair = blockIdx.x; pair < pairs; pair += gridDim.x) {
      const int layer = pair / a.H, h = pair - layer * a.H;
      const Planes& P = a.layer[layer];
      auto tile_of = [&](int src) { return (static_cast<size_t>(phys_of(src)) * a.H + h) * kTile; };
      const size_t si = static_cast<size_t>(h) * a.num_pages;
      int e_mine = kMinExp;
      if (mine >= 0) e_mine = f16_to_exp((lane < 16 ? P.ks : P.vs)[si + phys_of(mine)]);
      uint4 wk = make_uint4(kZero, kZero, kZero, kZero), v[4];
      if (sk >= 0) {
        const int slot = sk & 15;
        wk = *reinterpret_cast<const uint4*>(P.k + tile_of(sk) + 16 * (((((slot >> 3) << 1) | ((tid >> 5) & 1)) << 5) | ((slot & 7) << 2) | q));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sv[i] >= 0) v[i] = *reinterpret_cast<const uint4*>(P.v + tile_of(sv[i]) + 16 * ((tid & ~3) | ((sv[i] & 7) >> 1)));
      int top = e_mine;
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int ek = __shfl_sync(0xffffffffu, top, 0), ev = __shfl_sync(0xffffffffu, top, 16);
      const bool grows = __any_sync(0xffffffffu, mine >= 0 && e_mine < top);  // some code is rescaled
      const int e_k = __shfl_sync(0xffffffffu, e_mine, tk & 15);
      if (sk >= 0 && e_k < ek) wk = rescale<INT8>(wk, exp2_int(e_k - ek));
      uint32_t out[2] = {kZero, kZero};   // per channel half (bit 4): of channels + 0, + 8 tokens t, t + 1 ..
      uint32_t out2[2] = {kZero, kZero};  // .. and t + 8, t + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e_v = __shfl_sync(0xffffffffu, e_mine, 16 + 2 * q + (i & 1) + 8 * (i >> 1));
        if (sv[i] < 0) continue;
        const int slot = sv[i] & 15;
        // the token's bytes: words 2 h + (slot >> 3), bytes (slot & 1) and 2 + (slot & 1)
        const uint32_t a0 = slot >> 3 ? v[i].y : v[i].x, a1 = slot >> 3 ? v[i].w : v[i].z;
        uint32_t four = __byte_perm(a0, a1, slot & 1 ? 0x7531 : 0x6420);  // its codes of channels + 0, + 8, + 16, + 24
        if (e_v < ev) four = rescale4<INT8>(four, exp2_int(e_v - ev));
        const uint32_t keep = i & 1 ? 0x00FF00FFu : 0xFF00FF00u;  // bytes of the other token of the pair
        const uint32_t c0 = __byte_perm(four, 0, i & 1 ? 0x1404 : 0x4140);  // channels + 0 and + 8
        const uint32_t c1 = __byte_perm(four, 0, i & 1 ? 0x3424 : 0x4342);
        uint32_t* o = i >> 1 ? out2 : out;
        o[0] = (o[0] & keep) | c0;
        o[1] = (o[1] & keep) | c1;
      }
      const size_t tile = (static_cast<size_t>(s_phys[d]) * a.H + h) * kTile;
      __syncthreads();  // everything that goes into the page has been read
      if (grows || sk != self + tk) *reinterpret_cast<uint4*>(P.k + tile + 16 * tid) = wk;
      if (grows || !v_stays) *reinterpret_cast<uint4*>(P.v + tile + 16 * tid) = make_uint4(out[0], out2[0], out[1], out2[1]);
      if (tid == 0) {
        P.ks[si + s_phys[d]] = exp_to_f16(ek);
        P.vs[si + s_phys[d]] = exp_to_f16(ev);
      }
    }
    __syncthreads();  // later pages do not look at this one again, but a table with the same page twice would
  }
}

}  // namespace
}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_keep_runs(const kvq_cache* caches, int32_t n_caches, const int32_t* run_starts, int32_t batch, int32_t num_rows,
                                    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* keep,
                                    const int32_t* kept_lens, int32_t* err_word, kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::runs;
  if (n_caches < 0 || (n_caches > 0 && !caches)) return KVQ_ERR_INVALID_ARG;
  for (int i = 0; i < n_caches; ++i) {
    const kvq_status st = check_page_scaled_cache(caches + i);
    if (st != KVQ_OK) return st;
    if (caches[i].k_fmt != caches[0].k_fmt) return KVQ_ERR_UNSUPPORTED_LAYOUT;
    if (caches[i].num_kv_heads != caches[0].num_kv_heads || caches[i].num_pages != caches[0].num_pages) return KVQ_ERR_INVALID_ARG;
  }
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_pages_per_seq < 0) return KVQ_ERR_INVALID_ARG;
  if (!run_starts && num_rows != batch) return KVQ_ERR_INVALID_ARG;
  if (n_caches == 0 || batch == 0 || num_rows == 0) return KVQ_OK;
  if (!seq_lens || !keep || !kept_lens || !block_table || max_pages_per_seq == 0) return KVQ_ERR_INVALID_ARG;
  KeepArgs a{};
  a.H = caches[0].num_kv_heads;
  a.num_pages = caches[0].num_pages;
  a.run_starts = run_starts;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.keep = keep;
  a.kept = kept_lens;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.num_rows = num_rows;
  a.err = err_word;
  for (int i0 = 0; i0 < n_caches; i0 += kMaxLayers) {
    const int n = std::min(kMaxLayers, n_caches - i0);
    for (int i = 0; i < n; ++i) {
      const kvq_cache& c = caches[i0 + i];
      a.layer[i] = Planes{static_cast<uint8_t*>(c.k_data), static_cast<uint8_t*>(c.v_data), c.k_scale, c.v_scale};
    }
    a.layers = n;
    // Three times the blocks that the SMs hold at once, so that requests of more pages, or of none that change, even out: 32 requests of 36 layers
    // and 8 heads take 26.8 us, with as many blocks as are held 30.8, with six times 28.8 (in a graph; 33, 37 and 35 with the L2 flushed).
    const int want = std::max(1, 3 * device_sm_count() * kResident / batch);
    const dim3 grid(std::min(a.H * n, want), batch);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (caches[0].k_fmt == KVQ_FMT_INT8_PAGE) keep_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else keep_kernel<false><<<grid, kThreads, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  }
  return KVQ_OK;
}
