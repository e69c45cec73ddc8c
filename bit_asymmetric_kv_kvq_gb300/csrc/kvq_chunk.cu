// Attention of a chunk of new tokens over the quantized pages, the fp16 rows and the chunk itself
// (kvq_chunk_attention in include/kvq.h), on the fifth-generation tensor cores.
//
// Mathematics.  out_i = sum_j p_ij v_j with p = softmax_j(scale q_i . k_j) over the cached tokens and the
// chunk's tokens up to i.  One pass over the keys with a running maximum m and sum l per query row
// (base 2; the maximum is renewed, and the accumulator rescaled, only when it rises by more than 2^8).
//
// Work list.  A job is up to 256 query rows of one (sequence, kv head) unit -- the chunk's tokens with the
// heads that share the kv head beside each other, so grouped heads fill the tiles -- and a tile is up
// to 128 keys: whole pages first, then the unit's fp16 rows (sink, window) followed by the new tokens as
// far as the job's last token sees.  The flat list of all jobs' tiles (and start-ups, kJobCost) is cut into
// contiguous pieces of equal cost, one per SM, so few rows over a long cache are spread over the whole GPU
// and many rows leave no partly filled last wave.  A job that a cut divides leaves unnormalised partials (m, l, acc) in the
// workspace, at most two per CTA, and merge_chunk_kernel joins them in CTA order.
//
// A CTA.  Producer warps expand codes into fp16 operand tiles in shared memory (four for keys -- two sets of
// four, taking turns, where keys are rotated -- and four for values; new tokens are copied as they are), one
// thread issues the products, and two groups of four warps, a thread per query row, turn S = Q K^T into P
// (fp16, back into tensor memory over S).  The two groups are two streams whose products
// alternate, PV of one after QK of the other, so the tensor cores work on one stream while the other is in
// its softmax.  With more than 128 rows the streams are the two halves of the rows over the same key
// tiles; with up to 128 they are the even and the odd key tiles of the same rows, joined at the end
// through shared memory.
//
// Operand precision.  Every product is fp16 x fp16 with fp32 accumulation.  A dequantized key z + s c has up
// to 15 significant bits and, in outlier channels, a magnitude of tens, whose fp16 rounding would cost
// 1e-3 of a weight.  A constant added to a channel of ALL keys shifts every score of a row alike and
// cancels in the softmax, so keys enter as k - mu_c with mu_c the centre of the channel's range in one page
// where that centre lies outside the range's own width (else 0): the large common part is gone before
// rounding.  Rotated keys have no such constant: they are rounded to fp16, and what that leaves over of the
// eight pairs of channels that hold the outliers enters through a 16-column product of its own (22 bits there;
// a low half of all channels made the product and the tile half as expensive again).  Weights are rounded to
// fp16 scaled by 2^7, so a weight down to 2^-31 of the maximum still counts; values z + s c are rounded once.
//
// What bounds it (GB300; 1863 TFLOP/s bf16 and 6801 GB/s measured, 4 D flops per visible pair of query and key):
//   A  512 tokens, batch 4 x 40 heads over 8192 tokens, K4V2      372 us   354 GFLOP: 950 TFLOP/s, 0.51
//   B  a whole prompt of 4099 tokens, batch 2 x 32 heads on 8     329 us   275 GFLOP: 836 TFLOP/s, 0.45 (kvq_chunk_step)
//   C  8 tokens, batch 32 x 32 heads on 8 over 32768, K2V2        566 us   824 MB of pages: 1.46 TB/s, 0.21
//   D  33 tokens, 32 heads on 8 over 1,048,576, K3V3, rotated     2.08 ms  567 GFLOP, 990 MB of pages
// Long chunks (A, B): a tile of 256 rows x 128 keys takes 4,050 cycles, its products 2,740 at the matrix rate; the
// softmax of either stream (every score through tensor memory twice, an exponential, the rounding) is about as long as
// both streams' products, which hide it only in part, and a job's start and end cost another 13,000 cycles.  Few rows
// (C, D): the producers.  Every code becomes 16 bits of an operand tile once per job, 32,768 elements a tile (2,700
// cycles in C; 10,000 in D, where each pair of channels of a key takes a sine and a cosine besides), and the products'
// 128 rows cost the same whether they are used or not.
//
// Steps that paid, in us of the workloads above: roles for warps instead of one block that does everything in turn,
// A 980 -> 461, B 1255 -> 660, C 1366 -> 723; an issuing warp that waits once a step, A 461 -> 391, C 723 -> 616; a row
// of codes in registers, a low tile of 16 columns and two producer sets for rotated keys, D 4531 -> 2365; S read once,
// A 399 -> 384; zero points prepared once per block, C 655 -> 576; new tokens copied straight into place, B 528 -> 451;
// start-up costs in the cuts, B 451 -> 329; sparse entries written over the dense keys and loops compiled per code
// width, D 2252 -> 2077.  Tried and slower: unrolled producer loops (instruction-cache misses), a 16-column
// double-buffered softmax, 64 columns a pass with registers moved between warpgroups (spills), sixteen softmax warps,
// both streams on both halves of the rows, two sets of key producers where keys are not rotated, bitstream zero points
// and steps converted once per block (D 2108), value codes fetched an octet ahead (D 2080).
#include <atomic>
#include <cstddef>

#include <cuda_fp16.h>

#include "kvq_chunk.h"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kD = kHeadDim;
constexpr int kRows = 128;   // query rows of a stream
constexpr int kTile = 128;   // keys of a tile
constexpr int kProducers = 4;  // warps that make a key tile, and as many that make a value tile: a 32-token block each
template <bool ROPE>
constexpr int kKeySets = ROPE ? 2 : 1;  // sets of key producers, taking turns at the tiles
template <bool ROPE>
constexpr int kThreads = (8 + (kKeySets<ROPE> + 1) * kProducers + 1) * 32;
constexpr float kLazy = 8.0f;      // log2 units the running maximum may lag behind
constexpr float kWeightExp = 7.0f; // weights are at most 2^(8 + 7): below fp16's 65504
// A job costs more than its tiles: its queries are fetched, the pipeline fills, its rows are written.  The cuts between
// CTAs count that as four tiles (13,000 cycles a job, 3,000 to 4,000 a tile).  A prompt of 4099 tokens, whose first jobs
// are short, takes 451 us without it, and 367, 344, 329, 336, 347, 363 with 2, 3, 4, 5, 7, 10; other workloads hardly move.
constexpr int kJobCost = 4;
constexpr int kTmemColumns = 512;  // S / P of the two streams at 0 and 128, O at 256 and 384
constexpr int kValueStages = 2;
constexpr int kBadSlots = 4;       // marks of non-finite values: producers run at most three jobs ahead

// A place in the work list: a job of a unit, and a tile of the job; `lead` is what is left there of the job's
// start-up cost (see kJobCost).  (Counts of one CTA and one unit fit 32 bits.)
struct Piece {
  int32_t unit, job, tile, lead;
};

struct __align__(16) Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_ready[2], o_done[2], q_full[2], x_written, x_read, k_sync, v_sync;
  Piece first;                 // where this CTA's part of the work list begins
  uint32_t tmem;
  uint32_t bad[kBadSlots][8];  // tokens of the job with a non-finite value that some of its rows must not see
  __half2 mu[kD / 2];          // per channel pair
  alignas(16) uint32_t k_meta[2][2][kProducers][128], v_meta[kProducers][2][128];  // zero points and steps of two tiles' blocks
  alignas(8) uint8_t lo_slot[2][kProducers][64];  // rotated keys: a pair's place in the low tile, or 255
  alignas(16) unsigned long long turns[kD / 2];  // rotated keys: the turn per token of every pair
  float k_lev[16], v_lev[16];
  float xm[kRows], xl[kRows];  // the second stream's m and l
};

static_assert(offsetof(Shared, k_meta) % 16 == 0 && offsetof(Shared, v_meta) % 16 == 0, "16-byte asynchronous copies");

// Row of the value tile (and column of O) that holds channel d: the low bit of d moves to bit 2 within
// groups of eight, which spreads the page producer's 16-byte stores over all banks.
__device__ __forceinline__ int value_row(int d) { return (d & ~7) | ((d & 1) << 2) | ((d & 7) >> 1); }

// ------------------------------------------------------------ work list

// fp16 tiles of the first `jobs` jobs of a unit: sum over k = 1..jobs of ceil((n_w + k * job_tokens) / 128).
// Job sizes are powers of two, so the terms repeat with a fixed step after max(1, 128 / job_tokens) jobs.
__host__ __device__ inline int64_t f16_tiles_before(int64_t n_w, int log2_job_tokens, int64_t jobs) {
  const int lp = log2_job_tokens < 7 ? 7 - log2_job_tokens : 0;            // log2 of the jobs in a period
  const int64_t step = log2_job_tokens > 7 ? 1 << (log2_job_tokens - 7) : 1;  // tiles a period adds
  const int64_t m = jobs >> lp, rem = jobs - (m << lp);
  int64_t sum = 0;
  for (int i = 1; i <= (1 << lp); ++i) {
    const int64_t c = (n_w + ((int64_t)i << log2_job_tokens) + 127) >> 7;
    sum += m * c + step * (m * (m - 1) / 2) + (i <= rem ? c + step * m : 0);
  }
  return sum;
}

__device__ __noinline__ Piece find_piece(const ChunkParams& p, int64_t g) {
  const int64_t unit = g / p.unit_cost, r = g - unit * p.unit_cost;
  const int64_t per_job = p.page_tiles + kJobCost;
  int64_t lo = 0, hi = p.jobs_per_unit - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (mid * per_job + f16_tiles_before(p.n_w, p.log2_job_tokens, mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  const int64_t in_job = r - (lo * per_job + f16_tiles_before(p.n_w, p.log2_job_tokens, lo));
  return Piece{(int32_t)unit, (int32_t)lo, (int32_t)(in_job > kJobCost ? in_job - kJobCost : 0),
               (int32_t)(in_job < kJobCost ? kJobCost - in_job : 0)};
}

// A job's first chunk token, its tokens and its tiles.
__device__ __forceinline__ int64_t job_tok0(const ChunkParams& p, int job) { return (int64_t)job << p.log2_job_tokens; }
__device__ __forceinline__ int job_tokens(const ChunkParams& p, int job) {
  const int64_t left = p.n - job_tok0(p, job), full = (int64_t)1 << p.log2_job_tokens;
  return (int)(left < full ? left : full);
}
__device__ __forceinline__ int job_tiles(const ChunkParams& p, int job) {
  return (int)(p.page_tiles + ((p.n_w + job_tok0(p, job) + job_tokens(p, job) + 127) >> 7));
}

// ------------------------------------------------------------ operand tiles

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts4(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}
__device__ __forceinline__ void sts2(uint32_t addr, uint16_t a) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(a) : "memory");
}
// 16 bytes into shared memory asynchronously, or zeros (src is then not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst_smem, const void* src_gmem, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src_gmem), "r"(copy ? 16 : 0)
               : "memory");
}
template <int N>  // all but the newest N groups
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Pair j of a fragment-order word as two exact fp16 integers: the codes are masked into the mantissas
// of two numbers 1024 * 2^.., and one fused multiply-add takes the offset away and the shift back.
template <int B>
__device__ __forceinline__ __half2 code_pair(uint32_t word, int j) {
  constexpr int kFit = 10 / B;  // pairs whose bits lie in the 10-bit mantissa
  constexpr uint32_t m = (1u << B) - 1u;
  const uint32_t w = j < kFit ? word : word >> (B * kFit);
  const int sh = B * (j < kFit ? j : j - kFit);
  const float inv = 1.0f / (float)(1 << sh);
  const uint32_t x = (w & ((m | (m << 16)) << sh)) | 0x64006400u;
  return __hfma2(h2(x), __float2half2_rn(inv), __float2half2_rn(-1024.0f * inv));
}

// Codes of a 32-token block of a fragment-order page: two 16-token tiles of 2B words per lane.
template <int B>
__device__ __forceinline__ void load_codes(const uint8_t* codes, int block, int lane, uint32_t (&w)[4 * B]) {
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const uint4* src = reinterpret_cast<const uint4*>(codes) + ((2 * block + a) * 32 + lane) * (B / 2);
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint4 v = __ldg(src + i);
      w[2 * B * a + 4 * i] = v.x;
      w[2 * B * a + 4 * i + 1] = v.y;
      w[2 * B * a + 4 * i + 2] = v.z;
      w[2 * B * a + 4 * i + 3] = v.w;
    }
  }
}

// Keys of a 32-token block of a fragment-order page, for one warp.  Lane l = 4g + t holds, per token
// row, the 32 channels 8i + 2t + {0, 1}; the key tile's column order puts them side by side
// (column 64 (i/8) + 16 t + 8 ((i/4) % 2) + 2 (i % 4) + {0, 1}; the queries are stored in the same order), so every
// store is 16 bytes and eight neighbouring lanes hit all banks.  Key rows take the token order
// 16a + 8b + 2t' + e -> 8t' + 4a + 2b + e that the value block's words come in.  meta: the group's 128
// zero point / step words in shared memory (rewritten).
//
// The loop over the channels is kept a loop (the words are shifted along as it goes): the five roles of a
// CTA run different code side by side, and unrolled bodies miss the instruction caches -- the unrolled
// form of this kernel spent 4.6 of 13.6 cycles per issued instruction waiting for instructions.
template <int B>
__device__ __forceinline__ void key_block(uint32_t (&w)[4 * B], uint2* meta, const __half2* mu, int slot, uint32_t tile,
                                          int lane) {
  const int g = lane >> 2, t = lane & 3;
  // once per block: (z - mu, s) of the 64 channel pairs, in the order the lanes want them
  {
    uint2 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) m[h] = meta[lane + 32 * h];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pair = lane + 32 * h;  // 4 (4q + k) + t -> 4 (4q + t) + k
      const __half2 z = __hsub2(h2(__byte_perm(m[h].x, m[h].y, 0x5410)), mu[pair]);
      meta[(pair & ~15) | ((pair & 3) << 2) | ((pair >> 2) & 3)] = make_uint2(u32(z), __byte_perm(m[h].x, m[h].y, 0x7632));
    }
    __syncwarp();
  }
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {  // 32 channels: i = 4q .. 4q + 3
    const uint4 za = *reinterpret_cast<const uint4*>(meta + 4 * (4 * q + t)), zb = *reinterpret_cast<const uint4*>(meta + 4 * (4 * q + t) + 2);
    const __half2 z[4] = {h2(za.x), h2(za.z), h2(zb.x), h2(zb.z)}, s[4] = {h2(za.y), h2(za.w), h2(zb.y), h2(zb.w)};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = u32(__hfma2(code_pair<B>(w[2 * B * a + b * B], k), s[k], z[k]));
        const int row = 32 * slot + 8 * (g >> 1) + 4 * a + 2 * b + (g & 1);
        sts16(tile + tc::chunk_offset(q >> 1, row, 2 * t + (q & 1)), o[0], o[1], o[2], o[3]);
      }
    // the next 32 channels' codes: the upper half of a 2-bit word's pairs, or the next word
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int u = 0; u < B; ++u) {
        uint32_t& v = w[x * B + u];
        if (B == 2) v = u == 0 ? ((q & 1) ? w[x * B + 1] : v >> 8) : v;
        else v = u + 1 < B ? w[x * B + u + 1] : v;
      }
  }
}

// Values of a 32-token block of a fragment-order page, for one warp: the tile is [channel][token], and
// a lane's words hold the token pairs that make 16 bytes of a channel's row.  meta: the block's
// [32 tokens][D/G] zero point / step words in 512 bytes of shared memory (rewritten); half = 1 when G = 64.
template <int B>
__device__ __forceinline__ void value_block(uint32_t (&w)[4 * B], uint32_t* meta, int half, int slot, uint32_t tile,
                                            int lane) {
  const int g = lane >> 2, t = lane & 3;
  // once per block: (z, s) of the 16 token pairs for each 32 channels, in the order the lanes want them
  uint2* prep = reinterpret_cast<uint2*>(meta);
  {
    uint2 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h, q = i >> 4, tt = (i >> 2) & 3, tok = 16 * ((i >> 1) & 1) + 8 * (i & 1) + 2 * tt;
      const uint32_t* at = meta + tok * (4 >> half) + (q >> half);
      const uint32_t m0 = at[0], m1 = at[4 >> half];
      m[h] = make_uint2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) prep[lane + 32 * h] = m[h];  // [q][t][a][b]
    __syncwarp();
  }
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {  // channels 32q .. 32q + 31
    const uint4 za = *reinterpret_cast<const uint4*>(prep + 4 * (4 * q + t)), zb = *reinterpret_cast<const uint4*>(prep + 4 * (4 * q + t) + 2);
    const __half2 z[2][2] = {{h2(za.x), h2(za.z)}, {h2(zb.x), h2(zb.z)}}, s[2][2] = {{h2(za.y), h2(za.w)}, {h2(zb.y), h2(zb.w)}};
#pragma unroll
    for (int x = 0; x < 2; ++x)  // channels 16 (2q + x) + 8r + g: pair 2q + x of word r
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t o[4];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            o[2 * a + b] = u32(__hfma2(code_pair<B>(w[2 * B * a + (2 * b + r) * (B / 2)], x), s[a][b], z[a][b]));
        const int row = value_row(32 * q + 16 * x + 8 * r + g);
        sts16(tile + tc::chunk_offset(slot >> 1, row, 4 * (slot & 1) + t), o[0], o[1], o[2], o[3]);
      }
    // the next 32 channels' pairs: two pairs down, and for 4-bit codes the second word after two steps
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      uint32_t& v = w[x * (B / 2)];
      v = B == 4 && (q & 1) ? w[x * (B / 2) + B / 2 - 1] : v >> (2 * B);
    }
  }
}

// Column of channel c in a key or query tile of fragment-order caches (see key_block), as a byte offset.
__device__ __forceinline__ uint32_t frag_column(int row, int c) {
  const int i = c >> 3, t = (c & 7) >> 1;
  return tc::chunk_offset(i >> 3, row, 2 * t + ((i >> 2) & 1)) + (uint32_t)(4 * (i & 3) + 2 * (c & 1));
}

// Thirty-two contiguous channels of an fp16 row into a tile in that order: the 16 words are a 4 x 4
// transpose of the 16-byte chunks.
__device__ __forceinline__ void store_frag_row(uint32_t tile, int row, int q, const uint4 (&v)[4]) {
  const uint32_t* x = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
  for (int t = 0; t < 4; ++t)
    sts16(tile + tc::chunk_offset(q / 2, row, 2 * t + (q & 1)), x[t], x[4 + t], x[8 + t], x[12 + t]);
}

// Cosine and sine of frequency i at a position: the turn's fraction in 0.32 fixed point (position times the 0.64
// fraction of a turn per token, whole turns dropped), then the approximations, which are off by 2^-20.5 at most.
__device__ __forceinline__ float2 key_turn(uint32_t pos, uint2 t) {
  const float a = (float)(int32_t)(pos * t.y + __umulhi(pos, t.x)) * (6.28318530718f / 4294967296.0f);
  return make_float2(__cosf(a), __sinf(a));
}

// Rotated keys: the eight pairs whose channels are largest in a sample of the unit's keys -- one page's ranges, or
// the first fp16 rows when there is no page -- have their fp16 rounding made up for by a second, 16-channel tile
// that holds what it left over.  Every lane returns pairs 2 lane, 2 lane + 1's places in it (255: none).
__device__ __forceinline__ uint2 low_places(const ChunkParams& p, const uint8_t* unit_pages, const uint16_t* rows,
                                            const uint16_t* fresh, int lane) {
  float size[2] = {0.0f, 0.0f};
  if (p.n_pages > 0) {
    const uint32_t* m =
        reinterpret_cast<const uint32_t*>(unit_pages + (p.n_pages / 2) * p.lay.bytes + p.lay.off_km);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const __half2 v = h2(__ldg(m + 2 * lane + (c & 1) + 64 * (c >> 1)));
      const float z = __low2float(v), top = z + __high2float(v) * (float)((1 << p.bk) - 1);
      size[c & 1] = fmaxf(size[c & 1], fmaxf(fabsf(z), fabsf(top)));
    }
    // sparse entries are outside those ranges: those of 32 tokens
    const uint8_t* pg = unit_pages + (p.n_pages / 2) * p.lay.bytes;
#pragma unroll 1
    for (int e = 0; e < p.nsp; ++e) {
      const uint32_t mine = ((uint32_t)(pg[p.lay.off_si + lane * p.nsp + e] & 63) << 16) |
                            (reinterpret_cast<const uint16_t*>(pg + p.lay.off_sv)[lane * p.nsp + e] & 0x7FFFu);
#pragma unroll 4
      for (int i = 0; i < 32; ++i) {
        const uint32_t x = __shfl_sync(0xffffffffu, mine, i);
        const float v = __half2float(__ushort_as_half((uint16_t)x));
        if ((int)(x >> 17) == lane) {
          if ((x >> 16) & 1u) size[1] = fmaxf(size[1], v);
          else size[0] = fmaxf(size[0], v);
        }
      }
    }
  } else {
    const int64_t total = p.n_w + p.n;
    for (int64_t j = 0; j < 16 && j < total; ++j) {
      const uint32_t* r = reinterpret_cast<const uint32_t*>(j < p.n_w ? rows + j * kD : fresh + (j - p.n_w) * kD);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float2 v = __half22float2(h2(__ldg(r + lane + 32 * c)));
        size[0] = fmaxf(size[0], fabsf(v.x));
        size[1] = fmaxf(size[1], fabsf(v.y));
      }
    }
  }
  uint2 place = make_uint2(255, 255);
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    // the largest left over; sizes are >= 0, so their bits order them, and the low bits break ties
    const uint32_t a = place.x == 255 ? (__float_as_uint(size[0]) & ~127u) | (127 - 2 * lane) : 0;
    const uint32_t b = place.y == 255 ? (__float_as_uint(size[1]) & ~127u) | (126 - 2 * lane) : 0;
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(a, b));
    if (a == top) place.x = k;
    else if (b == top) place.y = k;
  }
  return place;
}

// Eight channels 8q + k and their rotation partners 64 + 8q + k of a key row, fp32, into the key tile
// (channel order as it is): rotated, with what fp16 leaves over of eight chosen pairs in the low tile, or shifted
// by mu.
template <bool ROPE>
__device__ __forceinline__ void store_key_octets(const ChunkParams& p, const Shared& sh, uint32_t tile, int row, int q,
                                                 uint32_t pos, const uint8_t* lo_slot, float (&x)[8], float (&y)[8]) {
  uint32_t hx[4], hy[4];
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    if constexpr (ROPE) {
      const uint4 tt = reinterpret_cast<const uint4*>(sh.turns)[4 * q + k / 2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 cs = key_turn(pos, e ? make_uint2(tt.z, tt.w) : make_uint2(tt.x, tt.y));
        const float a = x[k + e] * cs.x - y[k + e] * cs.y, b = x[k + e] * cs.y + y[k + e] * cs.x;
        x[k + e] = a;
        y[k + e] = b;
      }
    } else {
      const float2 mx = __half22float2(sh.mu[4 * q + k / 2]), my = __half22float2(sh.mu[32 + 4 * q + k / 2]);
      x[k] -= mx.x;
      x[k + 1] -= mx.y;
      y[k] -= my.x;
      y[k + 1] -= my.y;
    }
    const __half2 a = __floats2half2_rn(x[k], x[k + 1]), b = __floats2half2_rn(y[k], y[k + 1]);
    hx[k / 2] = u32(a);
    hy[k / 2] = u32(b);
  }
  sts16(tile + tc::chunk_offset(0, row, q), hx[0], hx[1], hx[2], hx[3]);
  sts16(tile + tc::chunk_offset(1, row, q), hy[0], hy[1], hy[2], hy[3]);
  if constexpr (ROPE) {
    const uint2 slots = *reinterpret_cast<const uint2*>(lo_slot + 8 * q);
    if ((slots.x & slots.y) != 0xFFFFFFFFu) {  // the octet holds one of the eight pairs
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t j = ((k < 4 ? slots.x : slots.y) >> (8 * (k & 3))) & 255u;
        if (j != 255u) {
          const float2 fa = __half22float2(h2(hx[k / 2])), fb = __half22float2(h2(hy[k / 2]));
          const uint32_t lo = tile + tc::kTileBytes;
          sts2(lo + tc::offset16(row, j), __half_as_ushort(__float2half_rn(x[k] - (k & 1 ? fa.y : fa.x))));
          sts2(lo + tc::offset16(row, 8 + j), __half_as_ushort(__float2half_rn(y[k] - (k & 1 ? fb.y : fb.x))));
        }
      }
    }
  }
}

// A code as a float: its bits in the mantissa of 2^23, less 2^23.
__device__ __forceinline__ float code_float(uint32_t codes, int shift, uint32_t mask) {
  return __uint_as_float(((codes >> shift) & mask) | 0x4B000000u) - 8388608.0f;
}

// Sparse entries of a lane's token of a bitstream page, over the dense key the lane has written: an entry's channel and
// its rotation partner are made again and stored.  (Within the loop over the octets an entry costs all lanes a select
// over eight channels in every octet that any lane has one in.)
template <bool ROPE, bool LUT>
__device__ __forceinline__ void sparse_pairs(const ChunkParams& p, const Shared& sh, const uint8_t* page, int tk, int row,
                                             const uint32_t* meta, uint32_t pos, const uint8_t* lo_slot, uint32_t tile) {
  uint32_t sp[4];  // channel << 16 | fp16 bits
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sp[e] = 0xFFFFFFFFu;
    if (e < p.nsp)
      sp[e] = (uint32_t)page[p.lay.off_si + tk * p.nsp + e] << 16 |
              reinterpret_cast<const uint16_t*>(page + p.lay.off_sv)[tk * p.nsp + e];
  }
  const int bits = p.bk;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(page + p.lay.off_kc) + tk * 4 * bits;
#pragma unroll 1
  for (int e = 0; e < p.nsp; ++e) {
    const uint32_t s = sp[0];
    const int c = (int)(s >> 16) & 127, partner = c ^ 64, pair = c & 63;
    const int at = partner * bits, word = at >> 5;
    const uint32_t code = __funnelshift_r(__ldg(codes + word), __ldg(codes + min(word + 1, 4 * bits - 1)), at & 31);
    const float2 zs = __half22float2(h2(meta[partner]));
    const uint32_t mask = (1u << bits) - 1u;
    float u = fmaf(zs.y, LUT ? sh.k_lev[code & mask] : code_float(code, 0, mask), zs.x);
#pragma unroll
    for (int i = 1; i < 4; ++i)  // unless the partner is an entry too
      if ((int)(sp[i] >> 16) == partner) u = __half2float(__ushort_as_half((uint16_t)sp[i]));
    const float v = __half2float(__ushort_as_half((uint16_t)s));
    float x = c < 64 ? v : u, y = c < 64 ? u : v;
    if constexpr (ROPE) {
      const unsigned long long t = sh.turns[pair];
      const float2 cs = key_turn(pos, make_uint2((uint32_t)t, (uint32_t)(t >> 32)));
      const float a = x * cs.x - y * cs.y, b = x * cs.y + y * cs.x;
      x = a;
      y = b;
    } else {
      x -= __half2float(reinterpret_cast<const __half*>(sh.mu)[pair]);
      y -= __half2float(reinterpret_cast<const __half*>(sh.mu)[64 + pair]);
    }
    const __half hx = __float2half_rn(x), hy = __float2half_rn(y);
    sts2(tile + tc::chunk_offset(0, row, pair >> 3) + 2 * (pair & 7), __half_as_ushort(hx));
    sts2(tile + tc::chunk_offset(1, row, pair >> 3) + 2 * (pair & 7), __half_as_ushort(hy));
    if constexpr (ROPE) {
      const uint32_t j = lo_slot[pair];
      if (j != 255u) {
        const uint32_t lo = tile + tc::kTileBytes;
        sts2(lo + tc::offset16(row, j), __half_as_ushort(__float2half_rn(x - __half2float(hx))));
        sts2(lo + tc::offset16(row, 8 + j), __half_as_ushort(__float2half_rn(y - __half2float(hy))));
      }
    }
    // the next entry to the front; the others stay in sight
    sp[0] = sp[1];
    sp[1] = sp[2];
    sp[2] = sp[3];
    sp[3] = s;
  }
}

// Keys of a 32-token block of a bitstream page, for one warp: lane = token, its row of codes in registers, an
// octet of channels and their rotation partners at a time.  meta: the group's 128 zero point / step words in
// shared memory.
template <int BITS, bool ROPE, bool LUT>
__device__ __forceinline__ void key_block_dense(const ChunkParams& p, const Shared& sh, const uint8_t* page, int block,
                                               int slot, const uint4* meta, uint32_t pos, const uint8_t* lo_slot,
                                               uint32_t tile, int lane) {
  const int tk = 32 * block + lane, row = 32 * slot + lane;
  constexpr uint32_t mask = (1u << BITS) - 1u;
  uint32_t w[2][2 * BITS];  // codes of channels 0..63 and 64..127
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < BITS; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(page + p.lay.off_kc) + (tk * 2 + h) * BITS + i);
      w[h][2 * i] = v.x;
      w[h][2 * i + 1] = v.y;
    }
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    float x[8], y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float(&o)[8] = h ? y : x;
      const uint4 ma = meta[16 * h + 2 * q], mb = meta[16 * h + 2 * q + 1];
      const uint32_t m[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 zs = __half22float2(h2(m[k]));
        const float c = LUT ? sh.k_lev[(w[h][0] >> (BITS * k)) & mask] : code_float(w[h][0], BITS * k, mask);
        o[k] = fmaf(zs.y, c, zs.x);
      }
      // the next octet's codes to the front
#pragma unroll
      for (int i = 0; i < 2 * BITS; ++i) w[h][i] = __funnelshift_rc(w[h][i], i + 1 < 2 * BITS ? w[h][i + 1] : 0u, 8 * BITS);
    }
    store_key_octets<ROPE>(p, sh, tile, row, q, pos, lo_slot, x, y);
  }
}

template <bool ROPE, bool LUT>
__device__ __forceinline__ void key_block_bits(const ChunkParams& p, const Shared& sh, const uint8_t* page, int block,
                                               int slot, const uint4* meta, uint32_t pos, const uint8_t* lo_slot,
                                               uint32_t tile, int lane) {
  if (p.bk == 2) key_block_dense<2, ROPE, LUT>(p, sh, page, block, slot, meta, pos, lo_slot, tile, lane);
  else if (p.bk == 3) key_block_dense<3, ROPE, LUT>(p, sh, page, block, slot, meta, pos, lo_slot, tile, lane);
  else key_block_dense<4, ROPE, LUT>(p, sh, page, block, slot, meta, pos, lo_slot, tile, lane);
  if (p.nsp)
    sparse_pairs<ROPE, LUT>(p, sh, page, 32 * block + lane, 32 * slot + lane, reinterpret_cast<const uint32_t*>(meta), pos,
                            lo_slot, tile);
}

// Codes of channels 8 oct .. 8 oct + 7 of a bitstream row (4 * bits words).
__device__ __forceinline__ uint32_t octet(const uint32_t* row, int bits, int oct) {
  const int off = 8 * oct * bits, w = off >> 5;
  const uint32_t lo = __ldg(row + w), hi = __ldg(row + min(w + 1, 4 * bits - 1));
  return __funnelshift_r(lo, hi, off & 31);
}

// Values of a 32-token block of a bitstream page, for one warp: lane = two neighbouring tokens of every second octet
// of channels.  meta: the block's [32 tokens][D/G] zero point / step words in shared memory; page null: zeros.
template <bool LUT>
__device__ __forceinline__ void value_block_bits(const ChunkParams& p, const Shared& sh, const uint8_t* page, int block,
                                                 int slot, const uint32_t* meta, uint32_t tile, int lane) {
  const int bits = p.bv, tp = lane & 15, per_token = kD / p.G;
  const uint32_t mask = (1u << bits) - 1u;
  const uint32_t* row =
      page ? reinterpret_cast<const uint32_t*>(page + p.lay.off_vc) + (32 * block + 2 * tp) * 4 * bits : nullptr;
#pragma unroll 1
  for (int it = 0; it < 8; ++it) {
    const int q = 2 * it + (lane >> 4);
    uint32_t o[8] = {};
    if (page) {
      const uint32_t c0 = octet(row, bits, q), c1 = octet(row + 4 * bits, bits, q);
      const uint32_t* m = meta + 2 * tp * per_token + 8 * q / p.G;
      const float2 a = __half22float2(h2(m[0])), b = __half22float2(h2(m[per_token]));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f0 = LUT ? sh.v_lev[(c0 >> (bits * k)) & mask] : code_float(c0, bits * k, mask);
        const float f1 = LUT ? sh.v_lev[(c1 >> (bits * k)) & mask] : code_float(c1, bits * k, mask);
        o[k] = u32(__floats2half2_rn(fmaf(a.y, f0, a.x), fmaf(b.y, f1, b.x)));
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      sts4(tile + tc::chunk_offset(slot >> 1, value_row(8 * q + k), 4 * (slot & 1) + (tp >> 2)) + 4 * (tp & 3), o[k]);
  }
}

// Sparse entries of a 32-token block of a fragment-order page, over the dense keys the warp has written.
__device__ __forceinline__ void sparse_block(const ChunkParams& p, const Shared& sh, const uint8_t* pg, int block,
                                             int slot, uint32_t tile, int lane) {
  const int tk = 32 * block + lane;
  const int row = 32 * slot + 8 * ((lane & 7) >> 1) + 4 * (lane >> 4) + 2 * ((lane >> 3) & 1) + (lane & 1);
  for (int e = 0; e < p.nsp; ++e) {
    const int c = pg[p.lay.off_si + tk * p.nsp + e];
    const float v = __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(pg + p.lay.off_sv)[tk * p.nsp + e]));
    const float m = __half2float(reinterpret_cast<const __half*>(sh.mu)[c]);
    sts2(tile + frag_column(row, c), __half_as_ushort(__float2half_rn(v - m)));
  }
}

// The fp16 rows of a tile: rows j0 .. j0 + 127 of the list that is the cache's rows followed by the new tokens, as far
// as the job's last token sees.
struct F16Rows {
  const uint16_t *a, *b;  // row r of the tile is at a + r * D for r < split, at b + r * D from there on
  int split, end;         // rows from `end` on are not there
  __device__ __forceinline__ F16Rows(const uint16_t* rows, const uint16_t* fresh, int n_w, int64_t j0, int64_t last)
      : a(rows + j0 * kD), b(fresh + (j0 - n_w) * kD) {
    const int64_t left = n_w - j0, n = last - j0;
    split = (int)(left < 0 ? 0 : left < kTile ? left : kTile);
    end = (int)(n < kTile ? n : kTile);
  }
  __device__ __forceinline__ const uint16_t* row(int r) const { return (r < split ? a : b) + r * kD; }
};

// This lane's 16-byte chunks of a warp's 32 rows of an fp16 tile, straight into the tile: row 32 warp + 2 i + lane / 16,
// chunk lane % 16.  All sixteen are in flight at once and hold no registers (a load takes 1,700 cycles while the kernel
// runs; with 4 KB a warp on its way a tile took 5,000).
__device__ __forceinline__ uint32_t raw_chunk(int warp, int lane, int i) {
  return tc::chunk_offset((lane & 15) >> 3, 32 * warp + 2 * i + (lane >> 4), lane & 7);
}
__device__ __forceinline__ void raw_rows(const F16Rows& f, uint32_t tile, int warp, int lane) {
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = 32 * warp + 2 * i + (lane >> 4);
    cp_async16_or_zero(tile + raw_chunk(warp, lane, i), f.row(r) + 8 * (lane & 15), r < f.end);
  }
  cp_async_commit();
  cp_async_wait_all();
}

// Keys of an fp16 tile, zeros from the end of its rows on.
template <bool FRAG, bool ROPE>
__device__ __forceinline__ void key_tile_f16(const ChunkParams& p, const Shared& sh, const F16Rows& f, int64_t j0,
                                             const uint8_t* lo_slot, uint32_t tile, int warp, int lane) {
  if (!ROPE && p.page_tiles == 0) {  // no pages: mu is 0 and the columns keep their order
    raw_rows(f, tile, warp, lane);
  } else if constexpr (FRAG) {
    const int q = lane >> 3;  // 32 channels of eight rows: all banks of a store
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {  // two rows' loads in flight per lane
      uint4 v[2][4] = {};
      const int row0 = 8 * (warp + 2 * kProducers * half) + (lane & 7);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + 8 * kProducers * h;
        const uint4* src = reinterpret_cast<const uint4*>(f.row(row)) + 4 * q;
        if (row < f.end) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[h][i] = __ldg(src + i);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t* x = reinterpret_cast<uint32_t*>(v[h]);
        if (row0 + 8 * kProducers * h < f.end) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = u32(__hsub2(h2(x[i]), sh.mu[16 * q + i]));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) store_frag_row(tile, row0 + 8 * kProducers * h, q, v[h]);
    }
  } else {
    const int row = 32 * warp + lane;
    // positions: the sink's rows first, the window behind the quantized tokens, then the new tokens
    const int64_t j = j0 + row;
    const uint32_t pos = (uint32_t)(j < p.n_s ? j : j + p.Tq);
    const uint4* src = reinterpret_cast<const uint4*>(f.row(row));
#pragma unroll 2
    for (int q = 0; q < 8; ++q) {
      float x[8] = {}, y[8] = {};
      if (row < f.end) {
        const uint4 vx = __ldg(src + q), vy = __ldg(src + 8 + q);
        const __half2 *hx = reinterpret_cast<const __half2*>(&vx), *hy = reinterpret_cast<const __half2*>(&vy);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 a = __half22float2(hx[k]), b = __half22float2(hy[k]);
          x[2 * k] = a.x;
          x[2 * k + 1] = a.y;
          y[2 * k] = b.x;
          y[2 * k + 1] = b.y;
        }
      }
      store_key_octets<ROPE>(p, sh, tile, row, q, pos, lo_slot, x, y);
    }
  }
}

// Values of an fp16 tile: token rows as they are (the product takes them MN-major); next to page tiles the channels of
// every eight go into value_row order.  Tokens behind the job's first (row job0 of the tile) are hidden from some of its
// rows, and 0 * inf or 0 * NaN would carry what they hold into those rows: non-finite values there enter the product as
// 0 and their tokens are marked, for patch_values to add them to the rows that do see them.
__device__ __forceinline__ void value_tile_f16(uint32_t* bad, const F16Rows& f, int job0, bool reorder, uint32_t tile,
                                               int warp, int lane) {
  raw_rows(f, tile, warp, lane);
  const bool check = 32 * warp + 31 > job0;
  if (!reorder && !check) return;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {  // each lane the chunks it copied itself
    const uint32_t at = tile + raw_chunk(warp, lane, i);
    const int r = 32 * warp + 2 * i + (lane >> 4);
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    if (check && r > job0) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool lo = (w[k] & 0x7C00u) == 0x7C00u, hi = (w[k] & 0x7C000000u) == 0x7C000000u;
        any |= lo || hi;
        w[k] &= (lo ? 0u : 0x0000FFFFu) | (hi ? 0u : 0xFFFF0000u);
      }
      if (any) atomicOr(&bad[(r - job0) >> 5], 1u << ((r - job0) & 31));
    }
    if (reorder)
      sts16(at, __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[0], w[1], 0x7632),
            __byte_perm(w[2], w[3], 0x7632));
    else
      sts16(at, w[0], w[1], w[2], w[3]);
  }
}

// What the marked tokens up to the row's own add to its channels 32y .. 32y + 31: their non-finite values
// (every visible token has a positive weight, so inf or NaN is the sum's).  `o` is in value_row order if reordered.
__device__ __forceinline__ void patch_values(const uint32_t* bad, const uint16_t* job_v, int token, int y, bool reordered,
                                             uint32_t* o) {
#pragma unroll 1
  for (int i = 1; i <= token; ++i) {
    if (!((bad[i >> 5] >> (i & 31)) & 1u)) continue;
#pragma unroll 1
    for (int c = 0; c < 32; ++c) {
      const float f = __half2float(__ushort_as_half(job_v[(int64_t)i * kD + 32 * y + c]));
      const int at = reordered ? value_row(c) : c;
      if (!isfinite(f)) o[at] = __float_as_uint(__uint_as_float(o[at]) + f);
    }
  }
}

// Two fp32 numbers in a 64-bit register, and the packed forms of multiply-add and add.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ the kernel

constexpr int kKeyStages = 2;
template <bool ROPE>  // a rotated key tile has a low tile behind it, and so have the queries' tiles, behind all others
constexpr int kKeyBytes = tc::kTileBytes + (ROPE ? tc::kTile16Bytes : 0);
template <bool ROPE>
constexpr int kSmemBytes = 2 * kKeyBytes<ROPE> + kKeyStages * kKeyBytes<ROPE> + kValueStages * tc::kTileBytes + 1024;
static_assert(kSmemBytes<true> + sizeof(Shared) <= 227 * 1024 && kSmemBytes<false> + sizeof(Shared) <= 227 * 1024, "shared memory");
static_assert(kKeyBytes<true> % 1024 == 0 && kKeySets<true> == kKeyStages, "a set of key producers per stage");

// A CTA's walk over its pieces of the work list: `count` tiles from tile t_begin of one job of one unit.
struct Walk {
  int32_t unit, job, t_begin, count;
  int32_t left;          // cost left to the CTA from this piece on, without what is left of the job's start-up cost
  int32_t tokens, rows;  // chunk tokens and query rows of the job
  bool dual;             // streams: even and odd tiles of up to 128 rows (else two halves of the rows)
  __device__ __forceinline__ Walk(const ChunkParams& p, const Piece& first, int32_t cost)
      : unit(first.unit), job(first.job), t_begin(first.tile), left(cost - first.lead) {
    at(p);
  }
  __device__ __forceinline__ void at(const ChunkParams& p) {
    tokens = job_tokens(p, job);
    const int whole = job_tiles(p, job) - t_begin;
    count = whole < left ? whole : left;  // <= 0: the end of the CTA's part
    rows = tokens << p.log2hg;
    dual = rows <= kRows;
  }
  __device__ __forceinline__ int64_t tok0(const ChunkParams& p) const { return job_tok0(p, job); }
  // Whether the piece is all of its job.
  __device__ __forceinline__ bool whole(const ChunkParams& p) const { return t_begin == 0 && count == job_tiles(p, job); }
  __device__ __forceinline__ void next(const ChunkParams& p) {
    left -= count + kJobCost;
    t_begin = 0;
    if (++job == p.jobs_per_unit) {
      job = 0;
      ++unit;
    }
    at(p);
  }
};

// Waits poll with the barrier's own short suspension and look at the clock every 256 polls.
__device__ __forceinline__ bool wait(const ChunkParams& p, uint64_t* bar, uint32_t parity) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 255u) == 0) {
      const unsigned long long now = global_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > (p.wait_ns ? p.wait_ns : kWaitLimitNs)) return false;
    }
  }
  return true;
}

// Barrier among warps of one role, with the time limit of every wait (a hardware barrier has none).
__device__ __forceinline__ bool meet(const ChunkParams& p, uint64_t* bar, uint32_t* count) {
  mbar_arrive(bar);
  return wait(p, bar, (*count)++ & 1);
}

// The value of lane 0, known to be the same in every lane.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// One product of a stream with a tile: S = Q K^T (rotated keys with their low tile), or O (+)= P V.  A
// descriptor's high word is the same for every tile; the low word moves by 2 (32 bytes) with every 16
// columns and by a block's size after 64.
template <bool ROPE>
__device__ __forceinline__ void issue_qk(uint32_t d, uint64_t q, uint64_t k, uint64_t q_lo, uint64_t k_lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t off = ((i >> 2) * tc::kBlockBytes + (i & 3) * 32) >> 4;
    tc::mma_ss(d, q + off, k + off, tc::instruction(kTile), i > 0);
  }
  if constexpr (ROPE) tc::mma_ss(d, q_lo, k_lo, tc::instruction(kTile), true);
}
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t pcol, uint64_t v, bool accumulate) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t off = ((i >> 2) * tc::kBlockBytes + (i & 3) * 32) >> 4;
    tc::mma_ts(d, pcol + 8 * i, v + off, tc::instruction(kD), accumulate || i > 0);
  }
}
// The same with token rows (fp16 tiles): 16 tokens are 16 rows of 128 bytes.
__device__ __forceinline__ void issue_pv_rows(uint32_t d, uint32_t pcol, uint64_t v, bool accumulate) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    tc::mma_ts(d, pcol + 8 * i, v + i * (2048 >> 4), tc::instruction(kD) | tc::kTransposeB, accumulate || i > 0);
}

// The issuing warp.  Step s of a piece is one stream's turn at one tile; QK runs two steps ahead of PV, so
// between a stream's QK and its PV the tensor cores have the other stream's products.  P overlies S: QK of
// step s + 2 comes behind PV of step s, which reads P, in issue order.  The warp walks along as a whole
// with everything uniform, so addresses and descriptors stay in uniform registers, and waits for one
// barrier a step: the tensor cores hold only a few products in advance, so what lies between two steps'
// products is their idle time.  The softmax streams watch the operand tiles for it (see operands_ready).
template <bool ROPE>
__device__ __forceinline__ bool issue_role(const ChunkParams& p, Shared& sh, uint32_t sq, uint32_t sk, uint32_t sv,
                                           uint32_t tmem_, int32_t cost_of_cta) {
  constexpr int KS = kKeyStages;
  const bool leader = tc::elect();
  const uint32_t tmem = uniform(tmem_);
  const uint64_t dq = tc::descriptor(sq), dk = tc::descriptor(sk), dv = tc::descriptor(sv), dv_rows = tc::descriptor_mn(sv);
  const uint64_t dq_lo = tc::descriptor16(sv + kValueStages * tc::kTileBytes), dk_lo = tc::descriptor16(sk + tc::kTileBytes);
  uint32_t kt = 0, vt = 0, jobs = 0, used0 = 0, used1 = 0;  // key and value tiles, pieces, steps of the streams so far
  for (Walk w(p, sh.first, cost_of_cta); (int)uniform(w.count) > 0; w.next(p)) {
    const bool dual = uniform(w.dual);
    const int tiles = (int)uniform(w.count), steps = dual ? tiles : 2 * tiles;
    if (!wait(p, &sh.q_full[0], jobs & 1) || !wait(p, &sh.q_full[1], jobs & 1)) return false;
    ++jobs;
#pragma unroll 1
    for (int s = -2; s < steps; ++s) {
      const uint32_t q = s & 1, at = 128 * q;
      const bool last = dual || q == 1;  // the tile's last step
      const uint32_t vs = vt % kValueStages, ks = kt % KS;
      const bool paged = uniform(w.t_begin) + (dual ? s : s >> 1) < (int)p.page_tiles;  // of step s
      if (s >= 0) {  // the stream's weights, its value tile and the key tile of its next step are there
        if (!wait(p, &sh.p_ready[q], (q ? used1 : used0) & 1)) return false;
        if (q) ++used1;
        else ++used0;
      } else if (s + 2 < steps) {
        if (!wait(p, &sh.k_full[ks], (kt / KS) & 1)) return false;
      }
      tc::fence_after();
      if (leader) {
        if (s >= 0) {
          const uint32_t stage = vs * (tc::kTileBytes >> 4);
          if (paged) issue_pv(tmem + 256 + at, tmem + at, dv + stage, s >= 2);
          else issue_pv_rows(tmem + 256 + at, tmem + at, dv_rows + stage, s >= 2);
          if (last) tc::commit(&sh.v_empty[vs]);
        }
        if (s + 2 < steps) {
          issue_qk<ROPE>(tmem + at, dq + (dual ? 0 : q * (tc::kTileBytes >> 4)), dk + ks * (kKeyBytes<ROPE> >> 4),
                         dq_lo + (dual ? 0 : q * (tc::kTile16Bytes >> 4)), dk_lo + ks * (kKeyBytes<ROPE> >> 4));
          tc::commit(&sh.s_full[q]);
        } else if (s >= 0) {
          tc::commit(&sh.o_done[q]);
        }
      }
      __syncwarp();
      if (last) {
        vt += s >= 0 ? 1 : 0;
        kt += s + 2 < steps ? 1 : 0;
      }
    }
  }
  return true;
}

// Of a piece's tiles, how many hold page `in_tile` of a tile: they are the first ones.
__device__ __forceinline__ int pages_of_warp(const ChunkParams& p, int64_t t_begin, int count, int in_tile) {
  if (in_tile >= p.pages_per_tile) return 0;
  const int64_t n = (p.n_pages - in_tile + p.pages_per_tile - 1) / p.pages_per_tile - t_begin;
  return (int)(n < 0 ? 0 : n < count ? n : count);
}

// Key producers: warp 0..3 of a set.
template <int BK, bool ROPE, bool LUT>
__device__ __forceinline__ bool key_role(const ChunkParams& p, Shared& sh, uint32_t sk, int32_t cost_of_cta,
                                         int set, int warp, int lane) {
  constexpr bool FRAG = BK != 0;
  constexpr int KS = kKeyStages, SETS = kKeySets<ROPE>;
  const int tid = 32 * (kProducers * set + warp) + lane;
  uint32_t kt0 = 0, syncs = 0;
  // the warp's 32-token block: its page of a tile and its place in the page
  const int in_tile = 32 * warp / p.R, block = (32 * warp - in_tile * p.R) / 32;
  for (Walk w(p, sh.first, cost_of_cta); w.count > 0; w.next(p)) {
    const uint8_t* unit_pages = p.pages + w.unit * p.unit_page_stride;
    const uint16_t* rows = p.wk + w.unit * p.win_unit_stride;
    const uint16_t* fresh = p.k_new + w.unit * p.n * kD;
    uint8_t* lo_slot = sh.lo_slot[set][warp];
    if constexpr (ROPE) {
      const uint2 place = low_places(p, unit_pages, rows, fresh, lane);
      __syncwarp();
      lo_slot[2 * lane] = (uint8_t)place.x;
      lo_slot[2 * lane + 1] = (uint8_t)place.y;
      __syncwarp();
    } else {  // mu: the centre of each channel's range in one page of the unit
      if (!meet(p, &sh.k_sync, &syncs)) return false;  // the last piece's tiles no longer need the old one
      float mu = 0.0f;
      if (p.n_pages > 0 && tid < kD) {
        const uint8_t* pg = unit_pages + (p.n_pages / 2) * p.lay.bytes;
        const __half2 m = h2(reinterpret_cast<const uint32_t*>(pg + p.lay.off_km)[tid]);
        const float range = __high2float(m) * (float)((1 << p.bk) - 1);
        const float centre = __low2float(m) + 0.5f * range;
        if (fabsf(centre) > range && fabsf(centre) <= 4096.0f) mu = centre;
      }
      if (tid < kD) reinterpret_cast<__half*>(sh.mu)[tid] = __float2half_rn(mu);
      if (!meet(p, &sh.k_sync, &syncs)) return false;
    }
    // the next tile's meta words are on their way to shared memory, and its codes to registers (fragment order) or L2
    constexpr int NW = FRAG ? 4 * BK : 1;
    uint32_t next[NW];
    const int count = w.count, first = SETS == 1 ? 0 : (int)((kt0 ^ (uint32_t)set) & 1);  // this set's first tile
    // tiles of the piece whose page of this warp exists, and that page in tile `first`
    const int paged = pages_of_warp(p, w.t_begin, count, in_tile);
    const uint8_t* pg = unit_pages + (int64_t)((w.t_begin + first) * p.pages_per_tile + in_tile) * p.lay.bytes;
    const int64_t stride = (int64_t)SETS * p.pages_per_tile * p.lay.bytes;
    const int meta_at = p.lay.off_km + (32 * block / p.G) * (kD * 4) + 16 * lane;
    auto fetch = [&](int i, const uint8_t* page) {
      if (i < paged) {
        if constexpr (FRAG) {
          load_codes<BK>(page + p.lay.off_kc, block, lane, next);
        } else if (128 * lane < 512 * p.bk) {  // the block's 512 * bits bytes
          prefetch_l2(page + p.lay.off_kc + block * 512 * p.bk + 128 * lane);
        }
        cp_async16(&sh.k_meta[set][(i / SETS) & 1][warp][4 * lane], page + meta_at);
      }
      cp_async_commit();
    };
    fetch(first, pg);
#pragma unroll 1
    for (int i = first; i < count; i += SETS, pg += stride) {
      const int t = w.t_begin + i;
      const uint32_t kt = kt0 + i, st = kt % KS, tile = sk + st * kKeyBytes<ROPE>;
      uint32_t codes[NW];
#pragma unroll
      for (int k = 0; k < NW; ++k) codes[k] = next[k];
      fetch(i + SETS, pg + stride);
      if (!wait(p, &sh.k_empty[st], ((kt / KS) & 1) ^ 1)) return false;
      if (t < p.page_tiles) {
        uint32_t* meta = sh.k_meta[set][(i / SETS) & 1][warp];
        cp_async_wait<1>();
        __syncwarp();
        if constexpr (FRAG) {
          if (i < paged) {
            key_block<BK>(codes, reinterpret_cast<uint2*>(meta), sh.mu, warp, tile, lane);
            if (p.nsp > 0) {
              __syncwarp();
              sparse_block(p, sh, pg, block, warp, tile, lane);
            }
          } else {
            for (int x = lane; x < 32 * 16; x += 32)
              sts16(tile + tc::chunk_offset(x >> 8, 32 * warp + ((x & 255) >> 3), x & 7), 0, 0, 0, 0);
          }
        } else {
          if (i < paged) {
            const int page = t * p.pages_per_tile + in_tile;
            key_block_bits<ROPE, LUT>(p, sh, pg, block, warp, reinterpret_cast<const uint4*>(meta),
                                      (uint32_t)(p.n_s + page * p.R + 32 * block + lane), lo_slot, tile, lane);
          } else {
            for (int x = lane; x < 32 * 16; x += 32)
              sts16(tile + tc::chunk_offset(x >> 8, 32 * warp + ((x & 255) >> 3), x & 7), 0, 0, 0, 0);
            if constexpr (ROPE) {
              for (int x = lane; x < 32 * 2; x += 32)
                sts16(tile + tc::kTileBytes + 32 * 32 * warp + 16 * x, 0, 0, 0, 0);
            }
          }
        }
      } else {
        const int64_t j0 = (int64_t)(t - (int)p.page_tiles) * kTile;
        const F16Rows f(rows, fresh, p.n_w, j0, p.n_w + w.tok0(p) + w.tokens);
        key_tile_f16<FRAG, ROPE>(p, sh, f, j0, lo_slot, tile, warp, lane);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && (int64_t)kt != (int64_t)p.test_withhold - 1) mbar_arrive(&sh.k_full[st]);
    }
    kt0 += (uint32_t)w.count;
  }
  return true;
}

// Value producers: warp 0..3.
template <int BV, bool ROPE, bool LUT>
__device__ __forceinline__ bool value_role(const ChunkParams& p, Shared& sh, uint32_t sv, int32_t cost_of_cta,
                                           int warp, int lane) {
  constexpr bool FRAG = BV != 0;
  uint32_t kt = 0, jobs = 0, syncs = 0;
  const int in_tile = 32 * warp / p.R, block = (32 * warp - in_tile * p.R) / 32, half = p.G == 64 ? 1 : 0;
  for (Walk w(p, sh.first, cost_of_cta); w.count > 0; ++jobs, w.next(p)) {
    const uint8_t* unit_pages = p.pages + w.unit * p.unit_page_stride;
    const uint16_t* rows = p.wv + w.unit * p.win_unit_stride;
    const uint16_t* fresh = p.v_new + w.unit * p.n * kD;
    uint32_t* bad = sh.bad[jobs % kBadSlots];
    if (warp == 0 && lane < 8) bad[lane] = 0;
    if (!meet(p, &sh.v_sync, &syncs)) return false;
    constexpr int NW = FRAG ? 4 * BV : 1;
    uint32_t next[NW];
    const int count = w.count, paged = pages_of_warp(p, w.t_begin, count, in_tile);
    const uint8_t* pg = unit_pages + (int64_t)(w.t_begin * p.pages_per_tile + in_tile) * p.lay.bytes;
    const int64_t stride = (int64_t)p.pages_per_tile * p.lay.bytes;
    const int meta_at = p.lay.off_vm + 32 * block * (16 >> half) + 16 * lane;
    auto fetch = [&](int i, const uint8_t* page) {
      if (i < paged) {
        if constexpr (FRAG) {
          load_codes<BV>(page + p.lay.off_vc, block, lane, next);
        } else if (128 * lane < 512 * p.bv) {
          prefetch_l2(page + p.lay.off_vc + block * 512 * p.bv + 128 * lane);
        }
        if (lane < (32 >> half)) cp_async16(&sh.v_meta[warp][i & 1][4 * lane], page + meta_at);
      }
      cp_async_commit();
    };
    auto ready = [&] { return wait(p, &sh.v_empty[kt % kValueStages], ((kt / kValueStages) & 1) ^ 1); };
    auto done = [&] {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.v_full[kt % kValueStages]);
      ++kt;
    };
    int i = 0;
    fetch(0, pg);
#pragma unroll 1
    for (; i < count && w.t_begin + i < (int)p.page_tiles; ++i, pg += stride) {
      const uint32_t tile = sv + (kt % kValueStages) * tc::kTileBytes;
      uint32_t codes[NW];
#pragma unroll
      for (int k = 0; k < NW; ++k) codes[k] = next[k];
      fetch(i + 1, pg + stride);
      if (!ready()) return false;
      cp_async_wait<1>();
      __syncwarp();
      if constexpr (FRAG) {
        if (i < paged) {
          value_block<BV>(codes, sh.v_meta[warp][i & 1], half, warp, tile, lane);
        } else {
          for (int x = lane; x < 128 * 4; x += 32)
            sts16(tile + tc::chunk_offset(warp >> 1, x >> 2, 4 * (warp & 1) + (x & 3)), 0, 0, 0, 0);
        }
      } else {
        value_block_bits<LUT>(p, sh, i < paged ? pg : nullptr, block, warp, sh.v_meta[warp][i & 1], tile, lane);
      }
      done();
    }
#pragma unroll 1
    for (; i < count; ++i) {  // fp16 rows
      const int64_t j0 = (int64_t)(w.t_begin + i - (int)p.page_tiles) * kTile, job0 = p.n_w + w.tok0(p);
      const F16Rows f(rows, fresh, p.n_w, j0, job0 + w.tokens);
      if (!ready()) return false;
      value_tile_f16(bad, f, (int)(job0 - j0 < kTile ? job0 - j0 : kTile), p.page_tiles > 0,
                     sv + (kt % kValueStages) * tc::kTileBytes, warp, lane);
      done();
    }
  }
  return true;
}

// What a step's products need besides the weights: its value tile, and the key tile of the stream's next step
// (`ahead` tiles on, if the piece has it).  One thread of the stream waits before it reports its weights.
template <int KS>
__device__ __forceinline__ bool operands_ready(const ChunkParams& p, Shared& sh, uint32_t tile, uint32_t ahead,
                                               uint32_t end) {
  if (!wait(p, &sh.v_full[tile % kValueStages], (tile / kValueStages) & 1)) return false;
  const uint32_t next = tile + ahead;
  return next >= end || wait(p, &sh.k_full[next % KS], (next / KS) & 1);
}

template <bool FRAG, bool ROPE>
__device__ __forceinline__ bool softmax_role(const ChunkParams& p, Shared& sh, uint32_t sq, uint32_t sq_lo,
                                             uint8_t* exchange, uint32_t tmem, int32_t cost_of_cta, int q, int warp, int lane) {
  constexpr int KS = kKeyStages;
  const int r = 32 * warp + lane;
  const uint32_t my_s = tmem + 128 * q + ((uint32_t)(32 * warp) << 16), my_o = my_s + 256;
  const int hg = 1 << p.log2hg;
  uint32_t tiles0 = 0, done = 0, jobs = 0, finals = 0, halves = 0;  // tiles, steps, pieces, pieces with steps of this stream, exchanges so far
  for (Walk w(p, sh.first, cost_of_cta); w.count > 0; ++jobs, w.next(p)) {
    const int tiles = w.count;
    const int b = w.unit / p.Hkv, kvh = w.unit - b * p.Hkv;
    const int64_t head_row = (int64_t)b * p.Hq + kvh * hg, tok0 = w.tok0(p);  // query row (token i, head h): (head_row + h) * n + tok0 + i
    // queries: job row = token * hg + head; channels in the key tiles' column order.  This stream's last
    // product of the piece before has finished, and with it every earlier one that read the tile.
    {
      const int first = w.dual ? 64 * q : 128 * q, count = w.dual ? 64 : 128;
      // two eights of rows in flight per warp
#pragma unroll 1
      for (int task = warp; task < count / 8; task += 8) {
        uint4 v[2][4] = {};
        const int c = lane >> 3;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = first + 8 * (task + 4 * h) + (lane & 7);
          if (row < w.rows) {
            const int64_t src_row = (head_row + (row & (hg - 1))) * p.n + tok0 + (row >> p.log2hg);
            const uint4* src = reinterpret_cast<const uint4*>(p.q + src_row * kD) + 4 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = __ldg(src + i);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = first + 8 * (task + 4 * h) + (lane & 7);
          const uint32_t tile = sq + (row >> 7) * tc::kTileBytes;
          if (FRAG && p.page_tiles > 0) {
            store_frag_row(tile, row & 127, c, v[h]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts16(tile + tc::chunk_offset(c >> 1, row & 127, 4 * (c & 1) + i), v[h][i].x, v[h][i].y, v[h][i].z, v[h][i].w);
          }
        }
      }
      // the next job's rows are on their way to L2 meanwhile
      if (w.job + 1 < p.jobs_per_unit) {
        const int row = (w.dual ? r : 128 * q + r);
        const int64_t i = tok0 + w.tokens + (row >> p.log2hg);
        if (i < p.n) {
          const uint16_t* next = p.q + ((head_row + (row & (hg - 1))) * p.n + i) * kD;
          prefetch_l2(next);
          prefetch_l2(next + 64);
        }
      }
    }
    if constexpr (ROPE) {  // the low tile's queries: columns j and 8 + j are the channels of the pair at place j
      const uint2 place = low_places(p, p.pages + w.unit * p.unit_page_stride, p.wk + w.unit * p.win_unit_stride,
                                     p.k_new + w.unit * p.n * kD, lane);
      const int row = w.dual ? r : 128 * q + r;
      const bool mine = !w.dual || (r >> 6) == q;
      const int64_t src_row = (head_row + (row & (hg - 1))) * p.n + tok0 + (row >> p.log2hg);
#pragma unroll 1
      for (int i = 0; i < 64; ++i) {
        const uint32_t j = __shfl_sync(0xffffffffu, i & 1 ? place.y : place.x, i >> 1);
        if (j == 255u || !mine) continue;
        const uint32_t tile = sq_lo + (row >> 7) * tc::kTile16Bytes;
        sts2(tile + tc::offset16(row & 127, j), row < w.rows ? p.q[src_row * kD + i] : (uint16_t)0);
        sts2(tile + tc::offset16(row & 127, 8 + j), row < w.rows ? p.q[src_row * kD + 64 + i] : (uint16_t)0);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&sh.q_full[q]);

    const int job_row = w.dual ? r : 128 * q + r;
    const int64_t seen0 = p.n_w + tok0 + (job_row >> p.log2hg) + 1;  // fp16 rows this row sees
    const bool live = job_row - lane < w.rows;
    float m_run = -INFINITY;
    uint64_t sum2 = 0;  // l in two halves
    const int steps = w.dual ? (tiles - q + 1) / 2 : tiles;
    for (int i = 0; i < steps; ++i, ++done) {
      const int t = w.t_begin + (w.dual ? 2 * i + q : i);
      int limit;  // columns this row sees
      if (t < p.page_tiles) {
        const int64_t left = p.n_pages - t * p.pages_per_tile;
        limit = (int)(left < p.pages_per_tile ? left : p.pages_per_tile) * p.R;
      } else {
        const int64_t seen = seen0 - (int64_t)(t - (int)p.page_tiles) * kTile;
        limit = (int)(seen < 0 ? 0 : seen > kTile ? kTile : seen);
      }
      if (!wait(p, &sh.s_full[q], done & 1)) return false;
      tc::fence_after();
      const uint32_t tile = tiles0 + (w.dual ? 2 * i + q : i);  // of all tiles of this CTA
      if (r == kRows - 32 && (w.dual || q == 1)) mbar_arrive(&sh.k_empty[tile % KS]);  // its last product is done
      if (!live) {  // no query row in this warp: its rows of S, P and O are never looked at
        tc::fence_before();
        if (r == kRows - 32 && !operands_ready<KS>(p, sh, tile, w.dual ? 2 : 1, tiles0 + tiles)) return false;
        mbar_arrive(&sh.p_ready[q]);
        continue;
      }
      const bool masked = __any_sync(0xffffffffu, limit < kTile);
      const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
#pragma unroll 1
      for (int col = 0; col < kTile; col += 32) {  // one pass: S is read once
        uint32_t v[32], wt[16];
        tc::ld32(my_s + col, v);
        tc::wait_ld();
        tc::tie32(v);
        if (masked) {  // hidden columns to -inf, whatever they hold
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = col + k < limit ? v[k] : 0xFF800000u;
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          m0 = max3(m0, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
          m1 = max3(m1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
        }
        const float ms = fmaxf(m0, m1) * p.scale_log2;
        const bool renew = ms > m_run + kLazy;  // also from -inf
        if (__any_sync(0xffffffffu, renew)) {
          // rare: a higher maximum.  It is a whole number, so what was summed and stored moves by a power of two:
          // l, the tile's weights so far, and O, whose last product finished with this S (they were committed
          // together).
          const float m_new = renew ? ceilf(ms) : m_run;
          const float factor = renew ? ex2(m_run - m_new) : 1.0f;
          m_run = m_new;
          unpack2(sum2, m0, m1);
          sum2 = pack2(m0 * factor, m1 * factor);
          const __half2 f2 = __float2half2_rn(factor);
#pragma unroll 1
          for (int c = 0; c < col / 2; c += 16) {
            tc::ld16(my_s + c, wt);
            tc::wait_ld16(wt);
#pragma unroll
            for (int k = 0; k < 16; ++k) wt[k] = u32(__hmul2(h2(wt[k]), f2));
            tc::st16(my_s + c, wt);
          }
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {
              tc::ld16(my_o + c, wt);
              tc::wait_ld16(wt);
#pragma unroll
              for (int k = 0; k < 16; ++k) wt[k] = __float_as_uint(__uint_as_float(wt[k]) * factor);
              tc::st16(my_o + c, wt);
            }
          }
        }
        const float shift = kWeightExp - (m_run == -INFINITY ? 0.0f : m_run);
        const uint64_t shift2 = pack2(shift, shift);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float a, c;
          unpack2(fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), scale2, shift2), a, c);
          a = ex2(a);
          c = ex2(c);
          sum2 = add2(sum2, pack2(a, c));
          wt[k / 2] = u32(__floats2half2_rn(a, c));
        }
        tc::st16(my_s + col / 2, wt);
      }
      tc::wait_st();
      tc::fence_before();
      if (r == kRows - 32 && !operands_ready<KS>(p, sh, tile, w.dual ? 2 : 1, tiles0 + tiles)) return false;
      mbar_arrive(&sh.p_ready[q]);
    }
    if (steps > 0) {
      if (!wait(p, &sh.o_done[q], finals & 1)) return false;
      ++finals;
      tc::fence_after();
    } else if (!wait(p, &sh.o_done[0], jobs & 1)) {  // a stream without steps must not run ahead into the next queries
      return false;
    }

    float l_run, l_half;
    unpack2(sum2, l_run, l_half);
    l_run += l_half;
    // the row's result, or its partial when the job is cut; two streams of the same rows are joined first
    const bool whole = w.whole(p);
    const bool join = w.dual && tiles > 1;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (w.t_begin == 0 ? 1 : 0);
    float* xo = reinterpret_cast<float*>(exchange);  // [64 columns][128 rows]
    float f0 = 1.0f, f1 = 0.0f;
    const uint32_t* bad = sh.bad[jobs % kBadSlots];
    const bool patch = w.t_begin + w.count > p.page_tiles
                           ? (bad[0] | bad[1] | bad[2] | bad[3] | bad[4] | bad[5] | bad[6] | bad[7]) != 0
                           : false;
#pragma unroll 1
    for (int y = 0; y < 4; ++y) {
      if (join && q == 1) {
        uint32_t o[32];
        tc::ld32(my_o + 32 * y, o);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) xo[(32 * (y & 1) + k) * kRows + r] = __uint_as_float(o[k]);
        if (y == 0) {
          sh.xm[r] = m_run;
          sh.xl[r] = l_run;
        }
        if (y & 1) {
          mbar_arrive(&sh.x_written);
          if (!wait(p, &sh.x_read, halves++ & 1)) return false;
        }
        continue;
      }
      if (w.dual && q == 1) break;
      if (join && !(y & 1)) {
        if (y) mbar_arrive(&sh.x_read);
        if (!wait(p, &sh.x_written, halves++ & 1)) return false;
        if (y == 0) {
          const float m1 = sh.xm[r], m = fmaxf(m_run, m1);
          f0 = m_run == -INFINITY ? 0.0f : ex2(m_run - m);
          f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - m);
          l_run = l_run * f0 + sh.xl[r] * f1;
          m_run = m;
        }
      }
      uint32_t o[32];
      tc::ld32(my_o + 32 * y, o);
      tc::wait_ld();
      if (join) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + xo[(32 * (y & 1) + k) * kRows + r] * f1);
      }
      if (patch) {
        uint32_t fixed[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) fixed[k] = o[k];
        patch_values(bad, p.v_new + (w.unit * p.n + tok0) * kD, min(job_row >> p.log2hg, w.tokens - 1), y, p.page_tiles > 0,
                     fixed);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = fixed[k];
      }
      if (job_row < w.rows) {
        // channel c of the 32: column value_row(c), or column c without pages
        const bool plain = p.page_tiles == 0;
        auto at = [&](int c) { return __uint_as_float(plain ? o[c] : o[(c & ~7) | ((c & 1) << 2) | ((c & 7) >> 1)]); };
        if (whole) {
          const float inv = l_run > 0.0f ? 1.0f / l_run : l_run == 0.0f ? 0.0f : l_run;
          const int64_t row = (head_row + (job_row & (hg - 1))) * p.n + tok0 + (job_row >> p.log2hg);
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * kD) + 4 * y;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = u32(__floats2half2_rn(at(8 * c + 2 * k) * inv, at(8 * c + 2 * k + 1) * inv));
            dst[c] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_acc + (slot * p.rows_max + job_row) * kD) + 8 * y;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            dst[c] = make_float4(at(4 * c), at(4 * c + 1), at(4 * c + 2), at(4 * c + 3));
          if (y == 0)
            *reinterpret_cast<float2*>(p.part_ml + (slot * p.rows_max + job_row) * 2) = make_float2(m_run, l_run);
        }
      }
    }
    if (join && q == 0) mbar_arrive(&sh.x_read);
    tc::fence_before();  // O is read before the next piece's first product, which waits for its queries
    tiles0 += tiles;
  }
  return true;
}

// BK, BV: code widths of fragment-order pages, or 0 for bitstream pages (widths at run time; LUT: codebook levels).
template <int BK, int BV, bool ROPE, bool LUT>
__global__ void __launch_bounds__(kThreads<ROPE>, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  uint8_t* const base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t sq = smem_u32(base), sk = sq + 2 * tc::kTileBytes;
  const uint32_t sv = sk + kKeyStages * kKeyBytes<ROPE>;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be
  constexpr int kIssuer = kThreads<ROPE> / 32 - 1;
  const int64_t g_begin = (int64_t)blockIdx.x * p.per_cta;
  const int32_t cost_of_cta = (int32_t)min(p.per_cta, p.total_cost - g_begin);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], kProducers);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], kProducers);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], kRows);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.q_full[i], kRows);
    }
    mbar_init(&sh.x_written, kRows);
    mbar_init(&sh.x_read, kRows);
    mbar_init(&sh.k_sync, kKeySets<ROPE> * kProducers * 32);
    mbar_init(&sh.v_sync, kProducers * 32);
    fence_mbar_init();
  }
  if (ROPE && tid < kD / 2) sh.turns[tid] = p.rope_turns[tid];
  if (tid < 16) {
    sh.k_lev[tid] = p.k_lev[tid];
    sh.v_lev[tid] = p.v_lev[tid];
  }
  if (tid == 32) {
    sh.first = find_piece(p, g_begin);
    reinterpret_cast<Piece*>(p.part_first)[blockIdx.x] = sh.first;
  }
  if (warp == kIssuer) tc::alloc(&sh.tmem, kTmemColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_allow_next();

  bool ok = true;
  if (warp < 8) {
    ok = softmax_role<BK != 0, ROPE>(p, sh, sq, sv + kValueStages * tc::kTileBytes, base + tc::kTileBytes, tmem, cost_of_cta, warp >> 2, warp & 3, lane);
  } else if (warp < kIssuer) {
    const int i = warp - 8;
    if constexpr (BK != 0) {
      // expanding fragment-order pages, keys on warp schedulers 0 and 1 and values on 2 and 3: fewer different
      // loops per instruction cache
      const int block = (i >> 2) * 2 + (i & 1);
      if (i & 2) ok = value_role<BV, ROPE, LUT>(p, sh, sv, cost_of_cta, block, lane);
      else ok = key_role<BK, ROPE, LUT>(p, sh, sk, cost_of_cta, 0, block, lane);
    } else if (i < kProducers) {
      ok = value_role<BV, ROPE, LUT>(p, sh, sv, cost_of_cta, i, lane);
    } else {
      ok = key_role<BK, ROPE, LUT>(p, sh, sk, cost_of_cta, i / kProducers - 1, i % kProducers, lane);
    }
  } else {
    ok = issue_role<ROPE>(p, sh, sq, sk, sv, tmem, cost_of_cta);
  }
  if (!ok) report_error(p.err, kDevWaitTimeout);
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kIssuer) tc::dealloc(tmem, kTmemColumns);
}

// Join the partials of the jobs that the cuts between CTAs divide: CTA x of the grid handles the job that
// the cut before piece x + 1 divides, if no earlier cut divides it too; a warp per query row.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) merge_chunk_kernel(const __grid_constant__ ChunkParams p) {
  pdl_wait();
  const int64_t cut = ((int64_t)blockIdx.x + 1) * p.per_cta;
  const Piece x = reinterpret_cast<const Piece*>(p.part_first)[blockIdx.x + 1];
  if (x.tile == 0) return;           // the cut falls between two jobs
  if (p.per_cta < x.tile) return;    // an earlier cut divides the same job
  const int64_t c0 = blockIdx.x, c1 = (cut - x.tile + job_tiles(p, x.job) - 1) / p.per_cta;
  const int64_t tok0 = job_tok0(p, x.job);
  const int hg = 1 << p.log2hg, rows = job_tokens(p, x.job) << p.log2hg;
  const int lane = threadIdx.x & 31;
  const int64_t b = x.unit / p.Hkv, kvh = x.unit - b * p.Hkv;
  for (int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); r < rows; r += gridDim.y * (kMergeThreads / 32)) {
    float M = -INFINITY, L = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t c = c0; c <= c1; ++c) {
      const int64_t slot = 2 * c + (c == c0 ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * p.rows_max + r) * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_acc + (slot * p.rows_max + r) * kD + 4 * lane);
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // no key of that piece is visible to the row
      const float m = fmaxf(M, ml.x);
      const float fo = M == -INFINITY ? 0.0f : exp2f(M - m), fn = ml.x == -INFINITY ? 1.0f : exp2f(ml.x - m);
      L = L * fo + ml.y * fn;
      a.x = a.x * fo + v.x * fn;
      a.y = a.y * fo + v.y * fn;
      a.z = a.z * fo + v.z * fn;
      a.w = a.w * fo + v.w * fn;
      M = m;
    }
    const float inv = L > 0.0f ? 1.0f / L : L == 0.0f ? 0.0f : L;
    const int64_t row = (b * p.Hq + kvh * hg + (r & (hg - 1))) * p.n + tok0 + (r >> p.log2hg);
    const __half2 lo = __floats2half2_rn(a.x * inv, a.y * inv), hi = __floats2half2_rn(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * kD + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

constexpr int64_t kFirstBytes = 16;
static_assert(sizeof(Piece) <= kFirstBytes, "a CTA's place in the work list");

// Rows of a partial slot: a job's.
int64_t slot_rows(int64_t n, int hg) { return n >= 2 * kRows / hg ? 2 * kRows : n * hg; }

template <int BK, int BV, bool ROPE, bool LUT>
cudaError_t launch_t(const ChunkParams& p, int64_t grid, int* launches, cudaStream_t s) {
  constexpr size_t smem = kSmemBytes<ROPE>;
  // the attribute is the device's for good: set once per device of the first 64, every time on others
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(chunk_kernel<BK, BV, ROPE, LUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  chunk_kernel<BK, BV, ROPE, LUT><<<(unsigned)grid, kThreads<ROPE>, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  if (grid == 1 || p.per_cta % p.unit_cost == 0) return cudaSuccess;  // no cut inside a job
  cudaLaunchConfig_t cfg{};
  const int64_t by = (p.rows_max + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)by);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, merge_chunk_kernel, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

// Every CTA's place in the work list, then two partial slots per CTA, each with the rows a job can have,
// of D + 2 floats a row.
int64_t chunk_workspace_bytes(int64_t n, int hg, int sm_count) {
  return (int64_t)sm_count * (kFirstBytes + 2 * slot_rows(n, hg) * (kD + 2) * (int64_t)sizeof(float));
}

cudaError_t launch_chunk(ChunkParams p, bool rope, int sm_count, void* workspace, int* launches, cudaStream_t s) {
  const int hg = 1 << p.log2hg;
  p.log2_job_tokens = (p.n * hg > kRows ? 8 : 7) - p.log2hg;
  p.pages_per_tile = kTile / p.R;
  p.page_tiles = (p.n_pages + p.pages_per_tile - 1) / p.pages_per_tile;
  const int64_t job_tokens = (int64_t)1 << p.log2_job_tokens;
  p.jobs_per_unit = (p.n + job_tokens - 1) / job_tokens;
  p.tiles_per_unit = p.jobs_per_unit * p.page_tiles + f16_tiles_before(p.n_w, p.log2_job_tokens, p.jobs_per_unit - 1) +
                     ((p.n_w + p.n + 127) >> 7);
  p.unit_cost = p.tiles_per_unit + kJobCost * p.jobs_per_unit;
  p.total_cost = p.n_units * p.unit_cost;
  int64_t grid = p.total_cost < sm_count ? p.total_cost : sm_count;
  p.per_cta = (p.total_cost + grid - 1) / grid;
  grid = (p.total_cost + p.per_cta - 1) / p.per_cta;
  if (p.per_cta >= ((int64_t)1 << 31)) return cudaErrorNotSupported;  // days of work: refused before any
  p.rows_max = (int32_t)slot_rows(p.n, hg);
  p.part_first = workspace;
  p.part_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) + sm_count * kFirstBytes);
  p.part_ml = p.part_acc + 2 * (int64_t)sm_count * p.rows_max * kD;
  if (p.lay.frag) {
    if (p.bk == 2 && p.bv == 2) return launch_t<2, 2, false, false>(p, grid, launches, s);
    if (p.bk == 4 && p.bv == 2) return launch_t<4, 2, false, false>(p, grid, launches, s);
    if (p.bk == 4 && p.bv == 4) return launch_t<4, 4, false, false>(p, grid, launches, s);
    return cudaErrorInvalidValue;
  }
  if (p.lut)
    return rope ? launch_t<0, 0, true, true>(p, grid, launches, s) : launch_t<0, 0, false, true>(p, grid, launches, s);
  return rope ? launch_t<0, 0, true, false>(p, grid, launches, s) : launch_t<0, 0, false, false>(p, grid, launches, s);
}

}  // namespace kvq
