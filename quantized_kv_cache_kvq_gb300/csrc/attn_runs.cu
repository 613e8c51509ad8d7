// attn_runs.cu -- kvq_attn_runs: causal attention of runs of query tokens over a page-scaled cache; the host side.  Short runs
// (single-token decode, drafts) have the split kernel (attn_runs_split.cuh), long BF16 ones the tile kernel (attn_runs_tile.cu).
#include <algorithm>
#include <cmath>

#include "attn_runs_split.cuh"

namespace kvq {
namespace runs {

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Workspace {
  SplitWorkspace split;
  size_t tw_acc, tw_stats, tw_rec, total;
  int nt;        // row tiles of 8 nt rows
  int few_rows;  // runs with more rows go to the tile kernel
  bool tile;     // there may be such runs
};

// BF16 runs of more than 16 (token, head) rows, where a unit's two row blocks end, are the tile kernel's; fp32 queries have the split
// kernel for every length.  16 drafts over 11500 tokens, 8 and 32 heads, E4M3 (INT8): the split kernel, one pass over the context for
// every 16 rows, 96 us (95) at 16 rows, 141-143 (152) at 20 to 32, 213 (217) at 48; the tile kernel 200 (208) at 20 to 48.
constexpr int kFewRows = 16;

Workspace workspace(int batch, int num_rows, int max_run, int hkv, int hq, int q_dtype, int sms) {
  const int G = hq / hkv;
  const long long max_rows = static_cast<long long>(max_run) * G;
  const int nt = row_blocks(max_rows);
  Workspace w{};
  w.nt = nt;
  w.tile = q_dtype == KVQ_DTYPE_BF16 && max_rows > kFewRows;
  w.few_rows = w.tile ? kFewRows : 0x7FFFFFFF;
  const size_t tiles = w.tile ? batch : (static_cast<size_t>(num_rows) * G) / (8 * nt) + batch;
  w.split = split_workspace(tiles, nt, hkv, sms);
  w.total = w.split.total;
  if (w.tile) {
    const size_t base = w.total;
    w.total += tile_workspace(sms, &w.tw_acc, &w.tw_stats, &w.tw_rec);
    w.tw_acc += base;
    w.tw_stats += base;
    w.tw_rec += base;
  }
  return w;
}

}  // namespace
}  // namespace runs
}  // namespace kvq

using namespace kvq;
using namespace kvq::runs;

extern "C" size_t kvq_attn_runs_workspace_size(int32_t batch, int32_t num_rows, int32_t max_run, int32_t num_kv_heads,
                                               int32_t num_q_heads, int32_t q_dtype) {
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_run < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
      num_q_heads % num_kv_heads || (q_dtype != KVQ_DTYPE_F32 && q_dtype != KVQ_DTYPE_BF16))
    return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return 0;
  return workspace(batch, num_rows, max_run, num_kv_heads, num_q_heads, q_dtype, sms).total;
}

// The checks and arguments that kvq_attn_runs and kvq_attn_tree share.
kvq_status kvq::runs::attn_args(AttnArgs* args, const kvq_cache* cache, const void* q, int64_t q_row_stride, int32_t q_dtype,
                                int32_t num_q_heads, const int32_t* run_starts, int32_t batch, int32_t num_rows, int32_t max_run,
                                const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* seq_lens, float sm_scale,
                                void* out, float* lse, void* workspace_dev, int32_t* err_word) {
  AttnArgs& a = *args;
  const kvq_status st = check_page_scaled_cache(cache);
  if (st != KVQ_OK) return st;
  const int hkv = cache->num_kv_heads;
  if (q_dtype != KVQ_DTYPE_F32 && q_dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_q_heads % hkv) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads / hkv > kMaxGroup) return KVQ_ERR_UNSUPPORTED_LAYOUT;
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || max_run < 0 || max_pages_per_seq < 0 || !std::isfinite(sm_scale))
    return KVQ_ERR_INVALID_ARG;
  if (!run_starts && num_rows != batch) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(num_rows) * num_q_heads > 0x7FFFFFFF) return KVQ_ERR_INVALID_ARG;
  a.batch = 0;  // nothing to do
  if (batch == 0 || num_rows == 0) return KVQ_OK;
  if (!run_starts && max_run < 1) return KVQ_ERR_INVALID_ARG;
  const int64_t unit = q_dtype == KVQ_DTYPE_BF16 ? 8 : 4;  // elements of 16 bytes
  if (q_row_stride < static_cast<int64_t>(num_q_heads) * kHeadDim || q_row_stride % unit) return KVQ_ERR_INVALID_ARG;
  if (!q || !seq_lens || !out || !workspace_dev || (max_pages_per_seq > 0 && !block_table)) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace_dev)) return KVQ_ERR_INVALID_ARG;
  a.k = static_cast<const uint8_t*>(cache->k_data);
  a.v = static_cast<const uint8_t*>(cache->v_data);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.num_pages = cache->num_pages;
  a.Hkv = hkv;
  a.Hq = num_q_heads;
  a.G = num_q_heads / hkv;
  a.q = q;
  a.q_stride = q_row_stride;
  a.run_starts = run_starts;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.num_rows = num_rows;
  a.max_run = std::min(max_run, num_rows);
  a.sm_scale = sm_scale;
  a.out = out;
  a.lse = lse;
  a.err = err_word;
  return KVQ_OK;
}

extern "C" kvq_status kvq_attn_runs(const kvq_cache* cache, const void* q, int64_t q_row_stride, int32_t q_dtype,
                                    int32_t num_q_heads, const int32_t* run_starts, int32_t batch, int32_t num_rows,
                                    int32_t max_run, const int32_t* block_table, int32_t max_pages_per_seq,
                                    const int32_t* seq_lens, float sm_scale, void* out, float* lse, void* workspace_dev,
                                    size_t ws_bytes, int32_t* err_word, kvq_stream_t stream) {
  AttnArgs a{};
  const kvq_status st = attn_args(&a, cache, q, q_row_stride, q_dtype, num_q_heads, run_starts, batch, num_rows, max_run, block_table,
                                  max_pages_per_seq, seq_lens, sm_scale, out, lse, workspace_dev, err_word);
  if (st != KVQ_OK || a.batch == 0) return st;
  const int sms = device_sm_count(), smem_max = device_smem_optin();
  if (sms <= 0 || smem_max <= 0) return KVQ_ERR_CUDA;
  const Workspace w = workspace(batch, num_rows, a.max_run, a.Hkv, a.Hq, q_dtype, sms);
  if (ws_bytes < w.total) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
  a.few_rows = w.few_rows;
  w.split.put(a, ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = q_dtype == KVQ_DTYPE_F32;
  const bool int8 = cache->k_fmt == KVQ_FMT_INT8_PAGE;
  cudaError_t e = int8 ? launch<true>(a, f32, w.nt, sms, smem_max, s) : launch<false>(a, f32, w.nt, sms, smem_max, s);
  if (e == cudaSuccess && w.tile) {
    a.tw_acc = reinterpret_cast<float*>(ws + w.tw_acc);
    a.tw_stats = reinterpret_cast<float*>(ws + w.tw_stats);
    a.tw_rec = reinterpret_cast<int32_t*>(ws + w.tw_rec);
    if (a.num_pages == 0) a.k = a.v = ws;  // absent pages are read as page 0 and thrown away
    e = launch_tile(a, int8, sms, s);
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
