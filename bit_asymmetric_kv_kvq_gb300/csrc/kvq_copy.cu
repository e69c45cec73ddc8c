// Copies of whole sequences between caches or within one (kvq_copy_sequences in include/kvq.h).
//
// A sequence's cache is, per kv head, one contiguous run of pages and one run of fp16 rows for keys
// and one for values, so the work is three runs of 16-byte columns per (sequence, head).  Nothing is
// computed: HBM bounds it.
//
// One thread owns one column of one kv head for EVERY sequence of the batch.  Within one cache it fetches the
// column's source for each destination sequence into its own slots of shared memory (asynchronous
// copies, all in flight together), waits for its own copies, and only then writes.  No other thread
// touches the column, so the copy may run in place under any map -- permutations with cycles, one
// source for many -- without a barrier for the data and without a second buffer.  Between caches the
// column passes through registers.
//
// Measured (GB300): half of 32 sequences of 32768 tokens x 8 heads replaced in place, 819 MB read and
// written, 129 us (6.35 TB/s); with the index looked up per sequence and thread instead of a list of the
// sequences that move, 171 us.  One sequence of 4096 tokens x 32 heads into eight, 129 MB, 23.9 us (5.38 TB/s); with one
// column's loads in flight at a time, 26.6 us; 32 sequences of 8192 tokens x 8 heads in another order, 715 MB, 113 us
// (6.35 TB/s; 182 us).
#include "kvq_chunk.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

// Columns of a CTA (threads) for a batch: one 16-byte slot per sequence and thread, at most
// kSlotBytes a CTA so that two or three CTAs share an SM and one loads while another stores.
constexpr int kSlotBytes = 72 * 1024;
constexpr int kMoves = 128;
constexpr int kMaxSlotBytes = 224 * 1024;  // in place with very large batches: one CTA of a few columns

// The column of this thread: its place in the first sequence of each cache, and the strides between sequences.
struct Column {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_seq, dst_seq;
  bool live;
  __device__ __forceinline__ Column(const CopySequencesParams& p, int64_t col0) {
    const int64_t per_head = p.run[0].columns + p.run[1].columns + p.run[2].columns;
    live = col0 < per_head * p.Hkv;
    const int64_t h = per_head * p.Hkv < ((int64_t)1 << 31) ? (int64_t)((uint32_t)col0 / (uint32_t)per_head) : col0 / per_head;
    int64_t col = col0 - h * per_head;
    int r = 0;
    if (col >= p.run[0].columns) {
      col -= p.run[0].columns;
      r = 1;
      if (col >= p.run[1].columns) {
        col -= p.run[1].columns;
        r = 2;
      }
    }
    const CopyRun& run = p.run[r];
    src = run.src + h * run.src_stride + col * 16;
    dst = run.dst + h * run.dst_stride + col * 16;
    src_seq = run.src_stride * p.Hkv;
    dst_seq = run.dst_stride * p.Hkv;
  }
};

// The sequences [b0, b1), at most kMoves, that have to move: (destination, source) in order.  An index out of
// range is reported and its sequence left as it was.  Every thread of the CTA calls this.
__device__ __forceinline__ int list_moves(const CopySequencesParams& p, int b0, int b1, int2* moves, int* n_moves) {
  __syncthreads();  // the last list is done with
  if (threadIdx.x == 0) *n_moves = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int width = min((int)blockDim.x, 32);
    const unsigned all = width == 32 ? 0xffffffffu : (1u << width) - 1u;
    for (int i0 = b0; i0 < b1; i0 += width) {
      const int i = i0 + threadIdx.x;
      const bool in = i < b1;
      const int from = in ? p.index[i] : 0;
      const bool good = in && from >= 0 && from < p.n_src;
      if (in && !good && blockIdx.x == 0) report_error(p.err, kDevBadArgument);
      const bool move = good && !(p.in_place && from == i);
      const unsigned who = __ballot_sync(all, move);
      if (move) moves[*n_moves + __popc(who & ((1u << threadIdx.x) - 1u))] = make_int2(i, from);
      __syncwarp(all);
      if (threadIdx.x == 0) *n_moves += __popc(who);
      __syncwarp(all);
    }
  }
  __syncthreads();
  return *n_moves;
}

// Within one cache: all sequences of a column are fetched before the first is written.
__global__ void __launch_bounds__(128) reorder_sequences_kernel(const CopySequencesParams p) {
  extern __shared__ __align__(16) uint4 slots[];
  __shared__ int2 moves[kMoves];
  __shared__ int n_moves;
  const int lanes = blockDim.x;
  const Column c(p, (int64_t)blockIdx.x * lanes + threadIdx.x);
  uint4* mine = slots + threadIdx.x;
  auto write = [&](int at, int n) {
    if (!c.live) return;
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      *reinterpret_cast<uint4*>(c.dst + moves[i].x * c.dst_seq) = mine[(size_t)(at + i) * lanes];
  };
  int done = 0, n = 0;
  for (int b = 0; b < p.n_dst; b += kMoves) {
    n = list_moves(p, b, min(b + kMoves, p.n_dst), moves, &n_moves);
    if (c.live) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) cp_async16(mine + (size_t)(done + i) * lanes, c.src + moves[i].y * c.src_seq);
    }
    done += n;
  }
  cp_async_commit();
  cp_async_wait_all();
  if (p.n_dst <= kMoves) {  // the list is still there
    write(0, n);
    return;
  }
  done = 0;
  for (int b = 0; b < p.n_dst; b += kMoves) {
    n = list_moves(p, b, min(b + kMoves, p.n_dst), moves, &n_moves);
    write(done, n);
    done += n;
  }
}

// Into another cache.  A thread takes kColumns columns: their loads are in flight together, the list of moves is made for
// more bytes, and a source that follows itself is read once.
constexpr int kColumns = 4;

__global__ void __launch_bounds__(256) copy_sequences_kernel(const CopySequencesParams p) {
  __shared__ int2 moves[kMoves];
  __shared__ int n_moves;
  const int64_t col0 = (int64_t)blockIdx.x * kColumns * blockDim.x + threadIdx.x;
  const Column c[kColumns] = {{p, col0}, {p, col0 + blockDim.x}, {p, col0 + 2 * blockDim.x}, {p, col0 + 3 * blockDim.x}};
  uint4 v[kColumns] = {};
  int held = -1;
  for (int b = 0; b < p.n_dst; b += kMoves) {
    const int n = list_moves(p, b, min(b + kMoves, p.n_dst), moves, &n_moves);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const int2 m = moves[i];
      if (m.y != held) {
        held = m.y;
#pragma unroll
        for (int k = 0; k < kColumns; ++k)
          if (c[k].live) v[k] = __ldg(reinterpret_cast<const uint4*>(c[k].src + m.y * c[k].src_seq));
      }
#pragma unroll
      for (int k = 0; k < kColumns; ++k)
        if (c[k].live) *reinterpret_cast<uint4*>(c[k].dst + m.x * c[k].dst_seq) = v[k];
    }
  }
}

}  // namespace

// In place, all sequences of a column have to be in shared memory before the first is written.
int copy_sequences_max_in_place() { return kMaxSlotBytes / 16; }

cudaError_t launch_copy_sequences(const CopySequencesParams& p, cudaStream_t s) {
  const int64_t total = (p.run[0].columns + p.run[1].columns + p.run[2].columns) * p.Hkv;
  if (total <= 0 || p.n_dst <= 0) return cudaSuccess;
  int threads = p.in_place ? 128 : 256;
  if (p.in_place) {
    while (threads > 32 && (int64_t)threads * 16 * p.n_dst > kSlotBytes) threads >>= 1;
    while (threads > 1 && (int64_t)threads * 16 * p.n_dst > kMaxSlotBytes) threads >>= 1;
  }
  const int64_t per_cta = (int64_t)threads * (p.in_place ? 1 : kColumns);
  const int64_t grid = (total + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (!p.in_place) {
    copy_sequences_kernel<<<(unsigned)grid, threads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const cudaError_t e = cudaFuncSetAttribute(reorder_sequences_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxSlotBytes);
  if (e != cudaSuccess) return e;
  reorder_sequences_kernel<<<(unsigned)grid, threads, (size_t)threads * 16 * p.n_dst, s>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
