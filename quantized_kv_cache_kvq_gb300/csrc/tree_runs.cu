// tree_runs.cu -- kvq_tree_runs: what every row of a tree of drafted tokens sees of its run, and its position.
//
// mask(i) = mask(parent(i)) | bit i, depth(i) = depth(parent(i)) + 1.  One block a request.  Rows are taken 32 at a time (a chunk, whose
// bits are one word): inside a chunk a warp finds every row's ancestors by pointer doubling in registers, five rounds whatever the shape, and
// the row's first ancestor before the chunk; the words of that ancestor, complete when the chunk's turn comes, are the row's other words.  So
// a chain of 1024 tokens is 32 dependent steps, not 1024.  Only words below the diagonal are kept in shared memory (62 KB for 1024 rows).
#include <algorithm>

#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32;

struct TreeArgs {
  const int32_t* parents;
  const int32_t* run_starts;
  const int32_t* seq_lens;
  int batch, num_rows, words;
  int32_t* mask;
  int32_t* positions;
  int32_t* err;
};

// First word of a chunk's rows in shared memory: 32 rows of as many words as there are chunks before.
__host__ __device__ constexpr int chunk_at(int c) { return kChunk * (c * (c - 1) / 2); }
// Rows of a run, rounded up to whole chunks; their own words, exits and depths, and the words below the diagonal.
__host__ __device__ constexpr size_t tree_smem(int chunks) { return (3 * kChunk * chunks + chunk_at(chunks)) * sizeof(int32_t); }

__global__ void __launch_bounds__(kThreads) tree_kernel(const TreeArgs a, int most) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Run run = load_run(a.run_starts, a.seq_lens, s, a.num_rows, most, kMaxContext / kPage);
  if (run.row0 < 0 || run.n > run.len) {
    if (tid == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  const int n = run.n, chunks = (n + kChunk - 1) / kChunk;
  uint32_t* own = reinterpret_cast<uint32_t*>(smem);              // [rows] ancestors inside the chunk, and the row itself
  int* exits = reinterpret_cast<int*>(own + kChunk * chunks);     // [rows] first ancestor before the chunk, -1 for none
  int* depth = exits + kChunk * chunks;                           // [rows]
  uint32_t* below = reinterpret_cast<uint32_t*>(depth + kChunk * chunks);
  for (int c = warp; c < chunks; c += kThreads / 32) {
    const int i = kChunk * c + lane;
    int up = -1;
    if (i < n) {
      up = a.parents[run.row0 + i];
      if (up < -1 || up >= i) {
        report(a.err, KVQ_ERR_DEVICE_BOUNDS);
        up = -1;
      }
    }
    uint32_t m = 1u << lane;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
      const bool inside = up >= kChunk * c;
      const int src = inside ? up - kChunk * c : lane;
      const uint32_t m2 = __shfl_sync(0xffffffffu, m, src);
      const int up2 = __shfl_sync(0xffffffffu, up, src);
      if (inside) {
        m |= m2;
        up = up2;
      }
    }
    own[i] = m;
    exits[i] = up;
  }
  __syncthreads();
  // 1 << shift lanes to a row, a word each: a chunk's 32 rows are four rounds of the block at most
  const int shift = a.words > 16 ? 5 : a.words > 1 ? 32 - __clz(a.words - 1) : 0;
  for (int c = 0; c < chunks; ++c) {
    const int rows = min(kChunk, n - kChunk * c);
    uint32_t* mine = below + chunk_at(c);
    if (tid < rows) {
      const int i = kChunk * c + tid, e = exits[i];
      depth[i] = __popc(own[i]) + (e >= 0 ? depth[e] : 0);
      if (a.positions) a.positions[run.row0 + i] = run.len - n + depth[i] - 1;
    }
    int32_t* out = a.mask + static_cast<long long>(run.row0 + kChunk * c) * a.words;
    const int step = kThreads >> shift, word = lane & ((1 << shift) - 1);
    // at most four rows a lane, all of whose loads are issued before the first is used
    int e[4];
    uint32_t here[4], x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (tid >> shift) + k * step;
      e[k] = r < rows ? exits[kChunk * c + r] : -1;
      here[k] = r < rows ? own[kChunk * c + r] : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ec = e[k] >> 5;  // -1 for none
      x[k] = e[k] < 0 || word > ec ? 0u : word == ec ? own[e[k]] : below[chunk_at(ec) + (e[k] & 31) * ec + word];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (tid >> shift) + k * step;
      if (r >= rows || word >= a.words) continue;
      if (word < c) mine[r * c + word] = x[k];
      int32_t* to = out + static_cast<long long>(r) * a.words;
      to[word] = static_cast<int32_t>(word == c ? here[k] : x[k]);
      for (int w = word + 32; w < a.words; w += 32) to[w] = 0;  // words that no run has
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_tree_runs(const int32_t* parents, const int32_t* run_starts, int32_t batch, int32_t num_rows,
                                    const int32_t* seq_lens, int32_t* mask, int32_t mask_words, int32_t* positions, int32_t* err_word,
                                    kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::runs;
  if (batch < 0 || batch > kMaxBatch || num_rows < 0 || mask_words < 1) return KVQ_ERR_INVALID_ARG;
  if (!run_starts && num_rows != batch) return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || num_rows == 0) return KVQ_OK;
  if (!parents || !seq_lens || !mask) return KVQ_ERR_INVALID_ARG;
  static SmemLimit limit;
  if (limit.raise(tree_kernel, tree_smem(KVQ_MAX_TREE / kChunk)) != cudaSuccess) return KVQ_ERR_CUDA;
  const int most = std::min({KVQ_MAX_TREE, num_rows, mask_words > KVQ_MAX_TREE / kChunk ? KVQ_MAX_TREE : mask_words * kChunk});
  const TreeArgs a{parents, run_starts, seq_lens, batch, num_rows, mask_words, mask, positions, err_word};
  tree_kernel<<<batch, kThreads, tree_smem((most + kChunk - 1) / kChunk), reinterpret_cast<cudaStream_t>(stream)>>>(a, most);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
