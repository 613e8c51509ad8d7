// tree_runs.cu -- kvq_tree_runs: what every row of a tree of drafted tokens sees of its run, and its position.
//
// mask(i) = mask(parent(i)) | bit i, depth(i) = depth(parent(i)) + 1.  One block a request.  Rows are taken 32 at a time (a chunk, whose
// bits are one word of a mask) by a warp.  Inside a chunk it finds every row's ancestors by pointer doubling in registers, five rounds
// whatever the shape, and the row's first ancestor before the chunk (its exit); both are kept in shared memory.  Then a thread to a row goes from
// exit to exit, which is at most one step for each chunk before: the ancestors in an exit's chunk are the exit's own word.  A chain of 1024
// tokens is 32 steps, not 1024.  The words are put together in shared memory and leave in whole rows.
// Bound by the bytes written where masks are long (1024 runs of 200..1000 tokens, 32 words a row, 68 MB: 22.6 us, 10 at the copy rate), by latency where
// they are short (16 runs of up to 64 tokens: 6 us).  Rows built one chunk after the other, with a barrier of the block for each, took 37 to 65 us there.
#include <algorithm>

#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kChunk = 32;
constexpr int kMaxWords = KVQ_MAX_TREE / kChunk;

struct TreeArgs {
  const int32_t* parents;
  const int32_t* run_starts;
  const int32_t* seq_lens;
  int batch, num_rows, words;
  int32_t* mask;
  int32_t* positions;
  int32_t* err;
};

struct Link {
  uint32_t own;  // ancestors inside the chunk, and the row itself
  int exit;      // first ancestor before the chunk, -1 for none
};
// Words from one row to the next where a chunk's rows are put together: whole 16-byte words, and not all rows in the same banks.
__host__ __device__ constexpr int row_stride(int words) { return (words + 3) / 4 * 4 + 4; }
__host__ __device__ constexpr size_t tree_smem(int chunks, int words, int threads) {
  return chunks * kChunk * sizeof(Link) + static_cast<size_t>(threads) * row_stride(words) * sizeof(uint32_t);
}

__global__ void __launch_bounds__(kMaxThreads) tree_kernel(const TreeArgs a, int most) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Run run = load_run(a.run_starts, a.seq_lens, s, a.num_rows, most, kMaxContext / kPage);
  if (run.row0 < 0 || run.n > run.len) {
    if (threadIdx.x == 0) report(a.err, KVQ_ERR_DEVICE_BOUNDS);
    return;
  }
  const int n = run.n, chunks = (n + kChunk - 1) / kChunk, words = min(a.words, kMaxWords);
  Link* links = reinterpret_cast<Link*>(smem);
  for (int c = warp; c < chunks; c += warps) {
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
    links[i] = Link{m, up};
  }
  __syncthreads();
  const int stride = row_stride(words), quads = (words + 3) >> 2;
  uint32_t* rows = reinterpret_cast<uint32_t*>(links + kChunk * ((most + kChunk - 1) / kChunk)) + warp * kChunk * stride;  // this warp's
  // quads threads to a row on the way out, 1 << shift of them where that is a power of two
  const int shift = quads > 1 ? 32 - __clz(quads - 1) : 0, quad = lane & ((1 << shift) - 1);
  const bool whole = (a.words & 3) == 0 && (reinterpret_cast<uintptr_t>(a.mask) & 15u) == 0;  // the mask's rows are 16-byte words
  for (int c = warp; c < chunks; c += warps) {
    const int there = min(kChunk, n - kChunk * c);
    for (int i = lane; i < kChunk * (stride >> 2); i += 32) reinterpret_cast<uint4*>(rows)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
    if (lane < there) {
      int depth = -1;
      for (int e = kChunk * c + lane; e >= 0;) {
        const Link k = links[e];
        rows[lane * stride + (e >> 5)] = k.own;
        depth += __popc(k.own);
        e = k.exit;
      }
      if (a.positions) a.positions[run.row0 + kChunk * c + lane] = run.len - n + depth;
    }
    __syncwarp();
    int32_t* out = a.mask + static_cast<long long>(run.row0 + kChunk * c) * a.words;
    for (int r = lane >> shift; r < there; r += 32 >> shift) {
      int32_t* to = out + static_cast<long long>(r) * a.words;
      if (quad < quads) {
        const uint4 x = *reinterpret_cast<const uint4*>(rows + r * stride + 4 * quad);
        if (whole) {
          *reinterpret_cast<uint4*>(to + 4 * quad) = x;
        } else {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * quad + i < words) to[4 * quad + i] = static_cast<int32_t>(w[i]);
        }
      }
      for (int w = kMaxWords + quad; w < a.words; w += 1 << shift) to[w] = 0;  // words that no run has
    }
    __syncwarp();
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
  if (limit.raise(tree_kernel, tree_smem(kMaxWords, kMaxWords, kMaxThreads)) != cudaSuccess) return KVQ_ERR_CUDA;
  const int words = std::min(mask_words, kMaxWords);
  const int most = std::min({KVQ_MAX_TREE, num_rows, words * kChunk}), chunks = (most + kChunk - 1) / kChunk;
  const int threads = std::min(kMaxThreads, kChunk * chunks);  // a warp to a chunk, eight at most
  const TreeArgs a{parents, run_starts, seq_lens, batch, num_rows, mask_words, mask, positions, err_word};
  tree_kernel<<<batch, threads, tree_smem(chunks, words, threads), reinterpret_cast<cudaStream_t>(stream)>>>(a, most);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
