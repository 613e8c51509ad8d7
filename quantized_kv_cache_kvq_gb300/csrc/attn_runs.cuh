// attn_runs.cuh -- arguments shared by the kernels of kvq_attn_runs and kvq_attn_tree.
//
// For row r of a run (query token i = r / G of query head kvh G + r % G, at position p = len - n + i):
//     x_t = sm_scale 2^{ek} (q . kc_t)   for t <= p,       out = sum_t e^{x_t} 2^{ev} vc_t / sum_t e^{x_t}
// with kc, vc the codes and ek, ev the exponents of the page that holds t.  The value scale goes into the exponent:
// with y_t = x_t log2 e + ev and m = max_t y_t,  out = sum_t 2^{y_t - m} vc_t / sum_t 2^{y_t - m} 2^{-ev}.  So the
// products take the codes as they are, the weights never exceed 1, and both scales are exact.
#pragma once

#include "decode_kernel.cuh"
#include "runs.cuh"

namespace kvq {
namespace runs {

// Two codes as fp16: bytes 0, 1 (lo) or 2, 3 (hi) of a word, exact in either format.
template <bool INT8>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  if (INT8) return dec::u8x2_to_f16x2(w, 0);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
template <bool INT8>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  if (INT8) return dec::u8x2_to_f16x2(w, 1);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// A unit of the split kernel: its rows are rows row_in_run .. of a run (row0: the run's first row in the step), at most
// `rows` of them; its pieces are those of warps w0 .. w0 + pieces - 1.
struct UnitRecord {
  int row0, rows, row_in_run, kvh, w0, pieces;
};

struct AttnArgs {
  const uint8_t* k;
  const uint8_t* v;
  const uint16_t* ks;
  const uint16_t* vs;
  int num_pages;
  int Hkv, G, Hq;
  const void* q;
  long long q_stride;  // elements between rows
  const int32_t* run_starts;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int max_pages, batch, num_rows, max_run;
  const int32_t* mask;  // trees only: [num_rows][mask_words]
  int mask_words;
  float sm_scale;
  void* out;   // [num_rows][Hq][128], the queries' type
  float* lse;  // [num_rows][Hq] or nullptr
  int few_rows;  // runs of at most this many (token, head) rows are the split kernel's, the others the tile kernel's
  // split kernel
  int* ws_units;            // number of units
  UnitRecord* ws_rec;       // [units]
  float* ws_stats;          // [slots][rows][2]: m, l
  float* ws_acc;            // [slots][rows][128]
  int max_tiles;            // row tiles that the workspace has room for
  int w_max, nwa, stages;
  // tile kernel
  float* tw_acc;    // [2 w][rows of a unit][128]: 256, of trees 128
  float* tw_stats;  // [2 w][rows of a unit][2]
  int32_t* tw_rec;  // [w][8]
  int tile_ctas;            // CTAs
  int unit_cost;            // what a unit costs beside its tiles, in tiles
  int32_t* err;
};

// Checks the arguments and fills `args`, all but the workspace's; batch 0: there is nothing to do (attn_runs.cu).
kvq_status attn_args(AttnArgs* args, const kvq_cache* cache, const void* q, int64_t q_row_stride, int32_t q_dtype, int32_t num_q_heads,
                     const int32_t* run_starts, int32_t batch, int32_t num_rows, int32_t max_run, const int32_t* block_table,
                     int32_t max_pages_per_seq, const int32_t* seq_lens, float sm_scale, void* out, float* lse, void* workspace_dev,
                     int32_t* err_word);

// Tile kernel and its merge (attn_runs_tile.cu); its part of the workspace, with the offsets of the three arrays.
cudaError_t launch_tile(AttnArgs& a, bool int8, int sms, cudaStream_t s);
size_t tile_workspace(int sms, size_t* acc, size_t* stats, size_t* rec);
// The same for trees (attn_tree_tile.cu).
cudaError_t launch_tree_tile(AttnArgs& a, bool int8, int sms, cudaStream_t s);
size_t tree_tile_workspace(int sms, size_t* acc, size_t* stats, size_t* rec);

}  // namespace runs
}  // namespace kvq
