// Copies of whole sequences between caches or within one (kvq_copy_sequences in include/kvq.h).
//
// A sequence's cache is, per kv head, one contiguous run of pages and one run of fp16 rows for keys
// and one for values, so the work is three runs of 16-byte columns per (sequence, head).  Nothing is
// computed: HBM bounds it.
//
// One thread owns one column of one kv head for EVERY sequence of the batch: it fetches the column's
// source for each destination sequence into its own slots of shared memory (asynchronous copies, all
// in flight together), waits for its own copies, and only then writes.  No other thread touches the
// column, so the copy may run in place under any map -- permutations with cycles, one source for
// many -- without a barrier and without a second buffer.
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

// Columns of a CTA (threads) for a batch: one 16-byte slot per sequence and thread, at most
// kSlotBytes a CTA so that two or three CTAs share an SM and one loads while another stores.
constexpr int kSlotBytes = 72 * 1024;
constexpr int kMaxSlotBytes = 227 * 1024;  // in place with very large batches: one CTA of a few columns

__global__ void __launch_bounds__(128) copy_sequences_kernel(const CopySequencesParams p) {
  extern __shared__ __align__(16) uint4 slots[];
  const int64_t per_head = p.run[0].columns + p.run[1].columns + p.run[2].columns;
  const int64_t total = per_head * p.Hkv;
  const int lanes = blockDim.x;
  const int64_t col0 = (int64_t)blockIdx.x * lanes + threadIdx.x;
  if (col0 >= total) return;
  const int64_t h = col0 / per_head;
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
  const uint8_t* src = run.src + h * run.src_stride + col * 16;
  uint8_t* dst = run.dst + h * run.dst_stride + col * 16;
  const int64_t src_seq = run.src_stride * p.Hkv, dst_seq = run.dst_stride * p.Hkv;
  uint4* mine = slots + threadIdx.x;
  for (int b0 = 0; b0 < p.n_dst; b0 += p.slots) {
    const int nb = min(p.slots, p.n_dst - b0);
    for (int i = 0; i < nb; ++i) {
      const int from = p.index[b0 + i];
      if (from < 0 || from >= p.n_src) {  // reported, and the sequence is left as it was
        if (col0 == 0) report_error(p.err, kDevBadArgument);
        continue;
      }
      if (p.in_place && from == b0 + i) continue;
      cp_async16(mine + (size_t)i * lanes, src + from * src_seq);
    }
    cp_async_commit();
    cp_async_wait_all();
    for (int i = 0; i < nb; ++i) {
      const int from = p.index[b0 + i];
      if (from < 0 || from >= p.n_src || (p.in_place && from == b0 + i)) continue;
      *reinterpret_cast<uint4*>(dst + (b0 + i) * dst_seq) = mine[(size_t)i * lanes];
    }
  }
}

}  // namespace

// In place, all sequences of a column have to be in shared memory before the first is written.
int copy_sequences_max_in_place() { return kMaxSlotBytes / 16; }

cudaError_t launch_copy_sequences(CopySequencesParams p, cudaStream_t s) {
  const int64_t total = (p.run[0].columns + p.run[1].columns + p.run[2].columns) * p.Hkv;
  if (total <= 0 || p.n_dst <= 0) return cudaSuccess;
  int threads = 128;
  if (p.in_place) {
    while (threads > 32 && (int64_t)threads * 16 * p.n_dst > kSlotBytes) threads >>= 1;
    while (threads > 1 && (int64_t)threads * 16 * p.n_dst > kMaxSlotBytes) threads >>= 1;
    p.slots = p.n_dst;
  } else {
    p.slots = p.n_dst < 16 ? p.n_dst : 16;
  }
  const size_t smem = (size_t)threads * 16 * p.slots;
  cudaError_t e = cudaFuncSetAttribute(copy_sequences_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxSlotBytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = (total + threads - 1) / threads;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  copy_sequences_kernel<<<(unsigned)grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
