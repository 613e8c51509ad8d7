// tree_runs.cu -- kvq_tree_runs: what every row of a tree of drafted tokens sees of its run, and its position.
//
// mask(i) = mask(parent(i)) | bit i, depth(i) = depth(parent(i)) + 1.  One block a request.  Rows are taken 32 at a time (a chunk, whose
// bits are one word): inside a chunk a warp finds every row's ancestors by pointer doubling in registers, five rounds whatever the shape, and
// the row's first ancestor before the chunk; the words of that ancestor, complete when the chunk's turn comes, are the row's other words.  So
// a chain of 1024 tokens is 32 dependent steps, not 1024.  Shared memory keeps the rows' words up to their own, in 16-byte pieces (74 KB for 1024
// rows); a thread takes such a piece of a row.  Bound by the bytes written where rows are long, by the latency of its steps where they are few.
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

// Pieces of four words that a row of chunk c keeps, and the first of the chunk's 32 rows: the chunks 4 i .. 4 i + 3 before have i + 1 each.
__host__ __device__ constexpr int row_pieces(int c) { return (c >> 2) + 1; }
__host__ __device__ constexpr int chunk_at(int c) { return kChunk * (2 * (c >> 2) * ((c >> 2) + 1) + (c & 3) * row_pieces(c)); }
// Rows of a run, rounded up to whole chunks: their own words, exits and depths, and their pieces.
__host__ __device__ constexpr size_t tree_smem(int chunks) { return 3 * kChunk * chunks * sizeof(int32_t) + chunk_at(chunks) * sizeof(uint4); }

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
  uint4* kept = reinterpret_cast<uint4*>(depth + kChunk * chunks);
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
  // 1 << shift threads to a row, four words each: a chunk's rows are one round of the block
  const int quads = (min(a.words, kChunk) + 3) >> 2, shift = quads > 1 ? 32 - __clz(quads - 1) : 0;
  const int r = tid >> shift, quad = tid & ((1 << shift) - 1);
  const bool whole = (a.words & 3) == 0 && (reinterpret_cast<uintptr_t>(a.mask) & 15u) == 0;  // pieces of the mask are 16-byte words
  for (int c = 0; c < chunks; ++c) {
    const int rows = min(kChunk, n - kChunk * c);
    if (tid < rows) {
      const int i = kChunk * c + tid, e = exits[i];
      depth[i] = __popc(own[i]) + (e >= 0 ? depth[e] : 0);
      if (a.positions) a.positions[run.row0 + i] = run.len - n + depth[i] - 1;
    }
    if (r < rows && quad < quads) {
      const int e = exits[kChunk * c + r], ec = e >> 5;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (e >= 0 && quad < row_pieces(ec)) x = kept[chunk_at(ec) + (e & 31) * row_pieces(ec) + quad];
      if (quad == c >> 2) {
        const uint32_t here = own[kChunk * c + r];
        if ((c & 3) == 0) x.x = here;
        if ((c & 3) == 1) x.y = here;
        if ((c & 3) == 2) x.z = here;
        if ((c & 3) == 3) x.w = here;
      }
      if (quad < row_pieces(c)) kept[chunk_at(c) + r * row_pieces(c) + quad] = x;
      int32_t* out = a.mask + static_cast<long long>(run.row0 + kChunk * c + r) * a.words;
      if (whole) {
        *reinterpret_cast<uint4*>(out + 4 * quad) = x;
      } else {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * quad + i < a.words) out[4 * quad + i] = static_cast<int32_t>(w[i]);
      }
      for (int w = kChunk + quad; w < a.words; w += quads) out[w] = 0;  // words that no run has
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
