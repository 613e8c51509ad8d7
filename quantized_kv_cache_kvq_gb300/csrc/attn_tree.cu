// attn_tree.cu -- kvq_attn_tree: attention of trees of drafted tokens over a page-scaled cache; the host side.
//
// Every row sees the tokens before its run, and of its run what its mask says.  Calls of few rows (and of fp32 queries) have the split
// kernel (attn_runs_split.cuh), which looks at the masks in the pages that the run touches; the others the tile kernel (attn_tree_tile.cu),
// for all their runs.
#include <algorithm>

#include "attn_runs_split.cuh"

namespace kvq {
namespace runs {
namespace {

// Calls whose longest run has more (token, head) rows are the tile kernel's.  The split kernel makes one pass over the context for every 16 rows.  Both
// kernels at 16, 20, 64 and 256 rows a request, 8 and 32 heads, E4M3, in a graph (us, split / tile):
//     1 request of 300 tokens     20/17   21/15    20/17     21/21       1 of 12000     21/27    26/27    35/29     76/39
//     4 of 12000                  40/41   50/42    80/48    263/80      16 of 2000      29/37    40/37    65/39    215/68
//     16 of 12000                 86/113 143/114  271/123  1006/233     64 of 2000      76/92   120/94   224/100   822/193
// Above 16 rows the tile kernel is no slower in any but one of them (26/27); at 16 it is the faster one where the context is short, by up to 3 us.
constexpr int kFewRows = 16;

struct Workspace {
  SplitWorkspace split;
  size_t tw_acc, tw_stats, tw_rec, total;
  int nt;     // split kernel: row tiles of 8 nt rows
  bool tile;  // the tile kernel's
};
Workspace workspace(int batch, int num_rows, int max_run, int hkv, int hq, int q_dtype, int sms) {
  const int G = hq / hkv;
  const long long max_rows = static_cast<long long>(max_run) * G;
  Workspace w{};
  w.tile = q_dtype == KVQ_DTYPE_BF16 && max_rows > kFewRows;
  w.nt = row_blocks(max_rows);
  if (w.tile) {
    w.total = tree_tile_workspace(sms, &w.tw_acc, &w.tw_stats, &w.tw_rec);
  } else {
    // Row tiles: no run has more than max_run tokens, and all of them no more than num_rows.
    const long long of_run = std::max(1ll, (max_rows + 8 * w.nt - 1) / (8 * w.nt));
    const long long tiles = std::min(static_cast<long long>(num_rows) * G / (8 * w.nt) + batch, of_run * batch);
    w.split = split_workspace(static_cast<size_t>(tiles), w.nt, hkv, sms);
    w.total = w.split.total;
  }
  return w;
}
// What a caller is told: enough for every call of no more requests, rows and max_run too.  The split kernel's part grows with each of them;
// the tile kernel's is the same for all its calls, so beside it stands the largest that a call of few rows takes.
size_t workspace_size(int batch, int num_rows, int max_run, int hkv, int hq, int q_dtype, int sms) {
  const Workspace w = workspace(batch, num_rows, max_run, hkv, hq, q_dtype, sms);
  return w.tile ? std::max(w.total, split_workspace(batch, row_blocks(kFewRows), hkv, sms).total) : w.total;
}

}  // namespace
}  // namespace runs
}  // namespace kvq

using namespace kvq;
using namespace kvq::runs;

extern "C" size_t kvq_attn_tree_workspace_size(int32_t batch, int32_t num_rows, int32_t max_run, int32_t num_kv_heads,
                                               int32_t num_q_heads, int32_t q_dtype) {
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_run < 0 || max_run > KVQ_MAX_TREE || num_kv_heads <= 0 || num_q_heads <= 0 ||
      num_q_heads % num_kv_heads || (q_dtype != KVQ_DTYPE_F32 && q_dtype != KVQ_DTYPE_BF16))
    return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return 0;
  return workspace_size(batch, num_rows, std::min(max_run, num_rows), num_kv_heads, num_q_heads, q_dtype, sms);
}

extern "C" kvq_status kvq_attn_tree(const kvq_cache* cache, const void* q, int64_t q_row_stride, int32_t q_dtype, int32_t num_q_heads,
                                    const int32_t* run_starts, int32_t batch, int32_t num_rows, int32_t max_run,
                                    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* mask,
                                    int32_t mask_words, float sm_scale, void* out, float* lse, void* workspace_dev, size_t ws_bytes,
                                    int32_t* err_word, kvq_stream_t stream) {
  AttnArgs a{};
  const kvq_status st = attn_args(&a, cache, q, q_row_stride, q_dtype, num_q_heads, run_starts, batch, num_rows, max_run, block_table,
                                  max_pages_per_seq, seq_lens, sm_scale, out, lse, workspace_dev, err_word);
  if (st != KVQ_OK) return st;
  if (max_run > KVQ_MAX_TREE || mask_words < (max_run + 31) / 32) return KVQ_ERR_INVALID_ARG;
  if (a.batch == 0) return KVQ_OK;
  if (!mask) return KVQ_ERR_INVALID_ARG;
  a.mask = mask;
  a.mask_words = mask_words;
  const int sms = device_sm_count(), smem_max = device_smem_optin();
  if (sms <= 0 || smem_max <= 0) return KVQ_ERR_CUDA;
  const Workspace w = workspace(batch, num_rows, a.max_run, a.Hkv, a.Hq, q_dtype, sms);
  if (ws_bytes < w.total) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool int8 = cache->k_fmt == KVQ_FMT_INT8_PAGE, f32 = q_dtype == KVQ_DTYPE_F32;
  cudaError_t e;
  if (w.tile) {
    a.few_rows = 0;
    a.tw_acc = reinterpret_cast<float*>(ws + w.tw_acc);
    a.tw_stats = reinterpret_cast<float*>(ws + w.tw_stats);
    a.tw_rec = reinterpret_cast<int32_t*>(ws + w.tw_rec);
    if (a.num_pages == 0) a.k = a.v = ws;  // absent pages are read as page 0 and thrown away
    e = launch_tree_tile(a, int8, sms, s);
  } else {
    a.few_rows = 0x7FFFFFFF;
    w.split.put(a, ws);
    e = int8 ? launch<true, true>(a, f32, w.nt, sms, smem_max, s) : launch<false, true>(a, f32, w.nt, sms, smem_max, s);
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
