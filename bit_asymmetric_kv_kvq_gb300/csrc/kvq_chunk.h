// Chunk attention and copies of sequences: what the C boundary hands to their kernels.
#pragma once

#include "kvq_internal.h"

namespace kvq {

// One run of 16-byte columns of every (sequence, kv head): the pages, or the fp16 key or value rows.
struct CopyRun {
  const uint8_t* src;   // unit (b, h) at src + (b * Hkv + h) * src_stride
  uint8_t* dst;
  int64_t src_stride, dst_stride;  // bytes
  int64_t columns;      // 16-byte columns of a unit
};

struct CopySequencesParams {
  CopyRun run[3];
  const int32_t* index; // [n_dst] source sequence of every destination sequence (device)
  int32_t n_src, n_dst, Hkv, in_place;
  int* err;
};

// Attention of a chunk of new tokens (kvq_chunk.cu).  The work list is cut into jobs -- up to 256 query
// rows (token-major, the heads of a kv head beside each other) of one unit -- and a job into tiles
// of up to 128 keys: the page tiles, then tiles over the unit's fp16 rows followed by the new tokens.
struct ChunkParams {
  const uint16_t* q;        // [B][Hq][n][D] fp16 bits
  const uint16_t* k_new;    // [B*Hkv][n][D]
  const uint16_t* v_new;
  uint16_t* out;            // [B][Hq][n][D]
  const uint8_t* pages;
  int64_t unit_page_stride;
  const uint16_t* wk;       // fp16 rows [units][S + R][D], rows 0 .. n_w in use
  const uint16_t* wv;
  int64_t win_unit_stride;  // elements
  int64_t n_units, n_pages, n, Tq;
  int32_t n_s, n_w, Hkv, Hq, log2hg, G, R, nsp, bk, bv;
  PageLayout lay;
  float scale_log2;         // softmax_scale * log2(e)
  const unsigned long long* rope_turns;
  int* err;
  int32_t lut;
  float k_lev[16], v_lev[16];
  unsigned long long wait_ns;  // test hooks, as in DecodeParams: withhold tile k of every CTA's piece of the list
  int32_t test_withhold;
  int32_t pages_per_tile;   // the rest is set by the launcher
  int64_t page_tiles;       // page tiles of a unit
  int64_t jobs_per_unit, tiles_per_unit, unit_cost, total_cost, per_cta;  // costs in tiles
  int32_t log2_job_tokens;  // tokens of a job
  int32_t rows_max;         // rows a partial slot holds
  void* part_first;         // [grid] where every CTA's part of the list begins
  float* part_acc;          // [2 * grid][rows_max][D] partial sums of jobs that CTAs share
  float* part_ml;           // [2 * grid][rows_max][2]
};

// Launchers (return cudaGetLastError() after the launch; launch_chunk cudaErrorNotSupported, before any, when one SM's
// share is too large to count).
cudaError_t launch_copy_sequences(const CopySequencesParams& p, cudaStream_t s);
int copy_sequences_max_in_place();
cudaError_t launch_chunk(ChunkParams p, bool rope, int sm_count, void* workspace, int* launches, cudaStream_t s);
int64_t chunk_workspace_bytes(int64_t n, int hg, int sm_count);

}  // namespace kvq
