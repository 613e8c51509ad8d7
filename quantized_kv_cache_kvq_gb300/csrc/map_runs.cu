// map_runs.cu -- kvq_map_runs: block tables, slot map, positions and the free-page stack from request lengths.
//
// The mathematics are three exclusive sums over the batch (tokens, pages wanted, pages handed back) and
// index arithmetic.  With fc pages on the stack, R handed back and A wanted, the i-th page handed out is entry F - 1 - i
// of the stack with the handed-back pages on top (F = fc + R).  Since pages are only ever pushed at fc and above, and
// only ever taken from below fc once the handed-back ones are used up, no entry is both read and written: every
// output follows from the inputs alone, and the blocks share nothing but the inputs and whether one of them met a page number that
// cannot be.  Everything is written behind a cluster barrier that all blocks reach after their reads of the states that may be
// updated in place (lengths, stack height) and their look at the page numbers: a step is taken whole or not at all.
// A request's pages are those of its length, or the caller keeps their number beside it: a draft's rejected tokens then leave
// their pages with the request, which uses them before it takes new ones.
// Bound by latency: one launch, two dependent rounds of loads.  64 requests of one token 5.8 us in a graph (8.4 a call from Python),
// 256 requests with prompts and finished ones among them 10.8 (12.3), 1024 prompts of 83,360 tokens 13.4 (15.0), 1.2 of which the
// look at the page numbers and the barrier behind it cost.  Rows written ahead of the look, or between the halves of the barrier,
// come to the same or more (13.9, 13.5).
#include "runs.cuh"

namespace kvq {
namespace runs {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxPage = 0x7FFFFFFF / kPage;  // the last page whose slots fit 31 bits

struct MapArgs {
  const int32_t* new_lens;
  const int32_t* seq_lens;
  int batch;
  int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int32_t* block_table;
  int max_pages;
  int32_t* run_starts;
  int32_t* seq_lens_out;
  int32_t* free_count_out;
  int32_t* slots;
  int32_t* positions;
  int max_rows;
  const int32_t* kept;  // pages that a finished request leaves to others, or nullptr
  int32_t* held;        // pages that a request has, in and out, or nullptr: those of its length
  int32_t* err;
};

// Last index i in [0, n) with a[i] <= x; a is non-decreasing with a[0] = 0 and x < a[n].
__device__ __forceinline__ int find_segment(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1) map_runs_kernel(const MapArgs a) {
  __shared__ int s_start[kMaxBatch + 1], s_want[kMaxBatch + 1], s_back[kMaxBatch + 1];
  __shared__ int s_old[kMaxBatch], s_held[kMaxBatch], s_kept[kMaxBatch];
  __shared__ long long s_tot[3][kThreads / 32];
  __shared__ int s_bad, s_odd_page;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = s_odd_page = 0;
  const int fc = *a.free_count;
  int old = 0, add = 0;
  bool gone = false, bad = false;
  if (tid < a.batch) {
    old = a.seq_lens[tid];
    add = a.new_lens[tid];
    gone = add < 0;
    if (gone) add = 0;
    const long long cap = min(static_cast<long long>(a.max_pages) * kPage, static_cast<long long>(kMaxContext));
    bad = old < 0 || old > cap || static_cast<long long>(old) + add > cap;
  }
  const int needed = bad ? 0 : (old + kPage - 1) / kPage;
  const int had = a.held && tid < a.batch ? a.held[tid] : needed;
  bad |= had < needed || had > a.max_pages;
  int held = bad ? 0 : had, kept = 0;
  if (gone && a.kept) {
    kept = a.kept[tid];
    if (kept < 0 || kept > held) {
      bad = true;
      kept = held = 0;
    }
  }
  // (tokens, pages wanted, pages handed back), summed in 64 bits: the totals are checked before anything is written
  long long v[3] = {bad ? 0 : add, bad || gone ? 0 : max(0ll, (static_cast<long long>(old) + add + kPage - 1) / kPage - held),
                    gone ? held - kept : 0};
  long long inc[3] = {v[0], v[1], v[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const long long t = __shfl_up_sync(0xffffffffu, inc[q], o);
      if (lane >= o) inc[q] += t;
    }
  if (lane == 31)
    for (int q = 0; q < 3; ++q) s_tot[q][warp] = inc[q];
  __syncthreads();
  const bool alone = gridDim.x == 1;
  if (!alone) asm volatile("barrier.cluster.arrive;" ::: "memory");  // this block's s_odd_page may be written by the others
  if (bad) s_bad = 1;
  long long total[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    long long t = s_tot[q][lane], before = lane < warp ? t : 0;  // kThreads / 32 == 32 warps, one per lane
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      t += __shfl_xor_sync(0xffffffffu, t, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    total[q] = t;
    inc[q] += before;
  }
  __syncthreads();
  int status = KVQ_OK;
  if (s_bad || total[0] > a.max_rows || fc < 0 || fc > a.free_capacity || fc + total[2] - total[1] > a.free_capacity)
    status = KVQ_ERR_DEVICE_BOUNDS;
  else if (total[1] > fc + total[2])
    status = KVQ_ERR_NO_PAGES;
  if (tid < a.batch) {
    s_start[tid] = static_cast<int>(inc[0] - v[0]);
    s_want[tid] = static_cast<int>(inc[1] - v[1]);
    s_back[tid] = static_cast<int>(inc[2] - v[2]);
    s_old[tid] = old;
    s_held[tid] = held;
    s_kept[tid] = kept;
  }
  bool ok = status == KVQ_OK;
  const int R = ok ? static_cast<int>(total[2]) : 0, F = fc + R;
  int n_rows = ok ? static_cast<int>(total[0]) : 0, A = ok ? static_cast<int>(total[1]) : 0;
  if (tid == 0) {
    s_start[a.batch] = n_rows;
    s_want[a.batch] = A;
    s_back[a.batch] = R;
  }
  __syncthreads();

  const int stride = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
  auto handed_back = [&](int i) {  // i-th page of the finished requests
    const int s = find_segment(s_back, a.batch, i);
    return a.block_table[static_cast<size_t>(s) * a.max_pages + s_kept[s] + (i - s_back[s])];
  };
  auto page_of = [&](int i) {  // i-th page handed out
    const int e = F - 1 - i;
    return e >= fc ? handed_back(e - fc) : a.free_pages[e];
  };
  // Every page number that the step moves or goes on in is looked at before anything is written: one that cannot be, found by
  // any block, stops all of them.
  bool odd_page = false;
  auto look = [&](int page) {
    odd_page |= page < 0 || page > kMaxPage;
    return page;
  };
  int out0 = 0, out1 = 0, back0 = 0, back1 = 0;  // this thread's first pages, kept until they are written
  if (ok) {
    if (tid < a.batch && add > 0)
      for (int j = old / kPage, end = min(held, (old + add + kPage - 1) / kPage); j < end; ++j)
        look(a.block_table[static_cast<size_t>(tid) * a.max_pages + j]);
#pragma unroll 1
    for (int i = first; i < A; i += stride) {
      const int page = look(page_of(i));
      if (i == first) out0 = page;
      if (i == first + stride) out1 = page;
    }
#pragma unroll 1
    for (int i = first; i < R - A; i += stride) {
      const int page = look(handed_back(i));
      if (i == first) back0 = page;
      if (i == first + stride) back1 = page;
    }
  }
  if (!alone) asm volatile("barrier.cluster.wait;" ::: "memory");
  odd_page = __syncthreads_or(odd_page);
  if (!alone) {
    if (odd_page && tid < gridDim.x)
      asm volatile(
          "{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %0, %1;\n\tst.shared::cluster.u32 [there], %2;\n\t}" ::"r"(
              static_cast<uint32_t>(__cvta_generic_to_shared(&s_odd_page))),
          "r"(tid), "r"(1)
          : "memory");
    asm volatile("barrier.cluster.arrive;" ::: "memory");
    asm volatile("barrier.cluster.wait;" ::: "memory");
    odd_page = s_odd_page;
  }
  // from here on every block has read the lengths and the stack height, which may be overwritten, and knows of odd pages
  if (odd_page) {
    status = KVQ_ERR_DEVICE_BOUNDS;
    ok = false;
    n_rows = A = 0;
  }
  if (ok) {
#pragma unroll 1
    for (int i = first; i < A; i += stride) {
      const int s = find_segment(s_want, a.batch, i);
      a.block_table[static_cast<size_t>(s) * a.max_pages + s_held[s] + (i - s_want[s])] =
          i == first ? out0 : i == first + stride ? out1 : page_of(i);
    }
#pragma unroll 1
    for (int i = first; i < R - A; i += stride)
      a.free_pages[fc + i] = i == first ? back0 : i == first + stride ? back1 : handed_back(i);
  }
  if (a.slots || a.positions) {
    // four rows in a row to a thread: one search, and mostly one page, for them
    for (int r0 = 4 * first; r0 < a.max_rows; r0 += 4 * stride) {
      int s = r0 < n_rows ? find_segment(s_start, a.batch, r0) : 0, j = -1, page = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        if (r >= a.max_rows) break;
        int slot = -1, pos = 0;
        if (r < n_rows) {
          while (r >= s_start[s + 1]) {
            ++s;
            j = -1;
          }
          const int o = s_old[s], h = s_held[s];
          pos = o + (r - s_start[s]);
          if (pos / kPage != j) {
            j = pos / kPage;
            page = j < h ? a.block_table[static_cast<size_t>(s) * a.max_pages + j] : page_of(s_want[s] + j - h);
          }
          slot = page * kPage + pos % kPage;
        }
        if (a.slots) a.slots[r] = slot;
        if (a.positions) a.positions[r] = pos;
      }
    }
  }
  if (blockIdx.x == 0) {
    if (tid < a.batch) {
      a.run_starts[tid] = ok ? s_start[tid] : 0;
      a.seq_lens_out[tid] = !ok ? old : gone ? 0 : old + add;
      if (a.held && ok) a.held[tid] = gone ? 0 : held + static_cast<int>(v[1]);
    }
    if (tid == 0) {
      a.run_starts[a.batch] = n_rows;
      *a.free_count_out = ok ? F - A : fc;
      if (!ok) report(a.err, status);
    }
  }
}

}  // namespace
}  // namespace runs
}  // namespace kvq

extern "C" kvq_status kvq_map_runs(const int32_t* new_lens, const int32_t* seq_lens, int32_t batch, int32_t* free_pages,
                                   int32_t free_capacity, const int32_t* free_count, int32_t* block_table,
                                   int32_t max_pages_per_seq, int32_t* run_starts, int32_t* seq_lens_out,
                                   int32_t* free_count_out, int32_t* slot_mapping, int32_t* positions, int32_t max_rows,
                                   int32_t* err_word, kvq_stream_t stream) {
  return kvq_map_runs_ex(new_lens, seq_lens, batch, free_pages, free_capacity, free_count, block_table, max_pages_per_seq, run_starts,
                         seq_lens_out, free_count_out, slot_mapping, positions, max_rows, nullptr, nullptr, err_word, stream);
}

extern "C" kvq_status kvq_map_runs_ex(const int32_t* new_lens, const int32_t* seq_lens, int32_t batch, int32_t* free_pages,
                                      int32_t free_capacity, const int32_t* free_count, int32_t* block_table,
                                      int32_t max_pages_per_seq, int32_t* run_starts, int32_t* seq_lens_out,
                                      int32_t* free_count_out, int32_t* slot_mapping, int32_t* positions, int32_t max_rows,
                                      const int32_t* kept_pages, int32_t* held_pages, int32_t* err_word, kvq_stream_t stream) {
  using namespace kvq::runs;
  if (batch < 0 || batch > kMaxBatch || free_capacity < 0 || max_pages_per_seq < 0 || max_rows < 0) return KVQ_ERR_INVALID_ARG;
  if ((slot_mapping || positions) && max_rows > 1 << 30) return KVQ_ERR_INVALID_ARG;  // rows are indexed with 32-bit integers
  if (!free_count || !run_starts || !free_count_out || (free_capacity > 0 && !free_pages)) return KVQ_ERR_INVALID_ARG;
  if (batch > 0 && (!new_lens || !seq_lens || !seq_lens_out || (max_pages_per_seq > 0 && !block_table)))
    return KVQ_ERR_INVALID_ARG;
  MapArgs a{new_lens,   seq_lens,     batch,          free_pages,   free_capacity, free_count, block_table, max_pages_per_seq,
            run_starts, seq_lens_out, free_count_out, slot_mapping, positions,     max_rows,   kept_pages,
            held_pages, err_word};
  cudaLaunchConfig_t cfg = {};
  // one block while its threads have a few rows each: a cluster of eight starts later (64 requests: 8.1 instead of 11 us a call)
  const long long work = batch + (slot_mapping || positions ? max_rows : 0ll);
  const unsigned blocks = work <= 2 * kThreads ? 1 : 8;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, map_runs_kernel, a) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
