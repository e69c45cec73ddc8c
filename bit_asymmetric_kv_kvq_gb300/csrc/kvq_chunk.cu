// Attention of a chunk of new tokens over the quantized pages, the fp16 rows and the chunk itself
// (kvq_chunk_attention in include/kvq.h), on the fifth-generation tensor cores.
//
// Mathematics.  out_i = sum_j p_ij v_j with p = softmax_j(scale q_i . k_j) over the cached tokens and the
// chunk's tokens up to i.  One pass over the keys with a running maximum m and sum l per query row
// (base 2; the maximum is renewed, and the accumulator rescaled, only when it rises by more than 2^8).
//
// Work list.  A job is 128 query rows of one (sequence, kv head) unit -- the chunk's tokens with the heads
// that share the kv head beside each other, so grouped heads fill the tile -- and a tile is up to 128
// keys: whole pages first, then the unit's fp16 rows (sink, window) followed by the new tokens as far
// as the job's last token sees.  The flat list of all jobs' tiles is cut into equal contiguous pieces,
// one per CTA, so few rows over a long cache are spread over the whole GPU and many rows leave no
// partly filled last wave.  A job that a cut divides leaves unnormalised partials (m, l, acc) in the
// workspace, at most two per CTA, and merge_chunk_kernel joins them in CTA order.
//
// A tile.  All warps expand codes into fp16 operand tiles in shared memory; one thread issues
// S = Q K^T (128 x 128 x 128) into tensor memory; four warps, a thread per query row, turn S into P (fp16,
// back into tensor memory over S); one thread issues O += P V.  Two CTAs per SM overlap one's
// expansion with the other's products.
//
// Operand precision.  Every product is fp16 x fp16 with fp32 accumulation.  A dequantized key z + s c has up
// to 15 significant bits and, in outlier channels, a magnitude of tens, whose fp16 rounding would cost
// 1e-3 of a weight.  A constant added to a channel of ALL keys shifts every score of a row alike and
// cancels in the softmax, so keys enter as k - mu_c with mu_c the centre of the channel's range in one page
// where that centre lies outside the range's own width (else 0): the large common part is gone before
// rounding.  Rotated keys have no such constant: they enter as hi + lo, two fp16 halves and two
// products (22 bits).  Weights are rounded to fp16 scaled by 2^7, so a weight down to 2^-31 of the
// maximum still counts; values z + s c are rounded once.
#include <cuda_fp16.h>

#include "kvq_internal.h"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kD = kHeadDim;
constexpr int kRows = 128;   // query rows of a job
constexpr int kTile = 128;   // keys of a tile
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLazy = 8.0f;      // log2 units the running maximum may lag behind
constexpr float kWeightExp = 7.0f; // weights are at most 2^(8 + 7): below fp16's 65504
constexpr int kTmemColumns = 256;  // S / P: 0..127, O: 128..255

struct Shared {
  uint64_t bar;
  uint32_t tmem;
  int bad;                    // some token of the tile has a non-finite value (see patch_values)
  uint32_t bad_tokens[4];
  __half2 mu[kD / 2];         // per channel pair
  float k_lev[16], v_lev[16];
};

// Row of the value tile (and column of O) that holds channel d: the low bit of d moves to bit 2 within
// groups of eight, which spreads the page producer's 16-byte stores over all banks.
__device__ __forceinline__ int value_row(int d) { return (d & ~7) | ((d & 1) << 2) | ((d & 7) >> 1); }

// ------------------------------------------------------------ work list

// fp16 tiles of the first `jobs` jobs of a unit: sum over k = 1..jobs of ceil((n_w + k * job_tokens) / 128).
__host__ __device__ inline int64_t f16_tiles_before(int64_t n_w, int log2_job_tokens, int64_t jobs) {
  const int period = 1 << (7 - log2_job_tokens);  // jobs per 128 tokens
  const int64_t m = jobs / period, rem = jobs - m * period;
  int64_t sum = 0;
  for (int i = 1; i <= period; ++i) {
    const int64_t c = (n_w + ((int64_t)i << log2_job_tokens) + 127) >> 7;
    sum += m * c + m * (m - 1) / 2 + (i <= rem ? c + m : 0);
  }
  return sum;
}

struct Piece {
  int64_t unit, job;         // job of the unit
  int64_t job_start;         // its first tile in the flat list
  int64_t tiles;             // its tiles
  int64_t tok0;              // first chunk token of the job
  int tokens;                // chunk tokens of the job
};

__host__ __device__ inline Piece find_piece(const ChunkParams& p, int64_t g) {
  Piece x;
  x.unit = g / p.tiles_per_unit;
  const int64_t r = g - x.unit * p.tiles_per_unit;
  int64_t lo = 0, hi = p.jobs_per_unit - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (mid * p.page_tiles + f16_tiles_before(p.n_w, p.log2_job_tokens, mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  x.job = lo;
  x.job_start = x.unit * p.tiles_per_unit + lo * p.page_tiles + f16_tiles_before(p.n_w, p.log2_job_tokens, lo);
  x.tok0 = lo << p.log2_job_tokens;
  const int64_t left = p.n - x.tok0, full = (int64_t)1 << p.log2_job_tokens;
  x.tokens = (int)(left < full ? left : full);
  x.tiles = p.page_tiles + ((p.n_w + x.tok0 + x.tokens + 127) >> 7);
  return x;
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

// Keys of a 32-token block of a fragment-order page, for one warp.  Lane l = 4g + t holds, per token
// row, the 32 channels 8i + 2t + {0, 1}; the key tile's column order puts them side by side
// (column 64 (i/8) + 16 t + 8 ((i/4) % 2) + 2 (i % 4) + {0, 1}; the queries are stored in the same order), so every
// store is 16 bytes and eight neighbouring lanes hit all banks.  Key rows take the token order
// 16a + 8b + 2t' + e -> 8t' + 4a + 2b + e that the value block's words come in.
template <int B>
__device__ __forceinline__ void key_block(const ChunkParams& p, const Shared& sh, const uint8_t* page, int block,
                                          int slot, uint32_t tile, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t w[2][2 * B];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const uint4* src = reinterpret_cast<const uint4*>(page + p.lay.off_kc) + ((2 * block + a) * 32 + lane) * (B / 2);
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint4 v = __ldg(src + i);
      w[a][4 * i] = v.x;
      w[a][4 * i + 1] = v.y;
      w[a][4 * i + 2] = v.z;
      w[a][4 * i + 3] = v.w;
    }
  }
  const uint2* meta = reinterpret_cast<const uint2*>(page + p.lay.off_km) + (32 * block / p.G) * (kD / 2);
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // 32 channels: i = 4q .. 4q + 3
    __half2 z[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pair = 4 * (4 * q + k) + t;
      const uint2 m = __ldg(meta + pair);
      z[k] = __hsub2(h2(__byte_perm(m.x, m.y, 0x5410)), sh.mu[pair]);
      s[k] = h2(__byte_perm(m.x, m.y, 0x7632));
    }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = B == 2 ? q / 2 : q, j = B == 2 ? 4 * (q % 2) + k : k;
          o[k] = u32(__hfma2(code_pair<B>(w[a][b * B + u], j), s[k], z[k]));
        }
        const int row = 32 * slot + 8 * (g >> 1) + 4 * a + 2 * b + (g & 1);
        sts16(tile + tc::chunk_offset(q / 2, row, 2 * t + (q & 1)), o[0], o[1], o[2], o[3]);
      }
  }
}

// Values of a 32-token block of a fragment-order page, for one warp: the tile is [channel][token], and
// a lane's words hold the token pairs that make 16 bytes of a channel's row.
template <int B>
__device__ __forceinline__ void value_block(const ChunkParams& p, const uint8_t* page, int block, int slot,
                                            uint32_t tile, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t w[2][2 * B];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const uint4* src = reinterpret_cast<const uint4*>(page + p.lay.off_vc) + ((2 * block + a) * 32 + lane) * (B / 2);
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint4 v = __ldg(src + i);
      w[a][4 * i] = v.x;
      w[a][4 * i + 1] = v.y;
      w[a][4 * i + 2] = v.z;
      w[a][4 * i + 3] = v.w;
    }
  }
  const uint32_t* meta = reinterpret_cast<const uint32_t*>(page + p.lay.off_vm);
  const int per_token = kD / p.G, half = p.G == 64 ? 1 : 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // channels 32q .. 32q + 31
    __half2 z[2][2], s[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int tok = 32 * block + 16 * a + 8 * b + 2 * t;
        const uint32_t m0 = __ldg(meta + tok * per_token + (q >> half));
        const uint32_t m1 = __ldg(meta + (tok + 1) * per_token + (q >> half));
        z[a][b] = h2(__byte_perm(m0, m1, 0x5410));
        s[a][b] = h2(__byte_perm(m0, m1, 0x7632));
      }
#pragma unroll
    for (int x = 2 * q; x < 2 * q + 2; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t o[4];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int u = x / (16 / B), j = x % (16 / B);
            o[2 * a + b] = u32(__hfma2(code_pair<B>(w[a][(2 * b + r) * (B / 2) + u], j), s[a][b], z[a][b]));
          }
        const int row = value_row(16 * x + 8 * r + g);
        sts16(tile + tc::chunk_offset(slot / 2, row, 4 * (slot & 1) + t), o[0], o[1], o[2], o[3]);
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

__device__ __forceinline__ float2 key_turn(const ChunkParams& p, int64_t pos, int i) {
  const unsigned long long t = (unsigned long long)pos * p.rope_turns[i];
  float s, c;
  sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// Eight channels 8q + k and their rotation partners 64 + 8q + k of a key row, fp32, into the key tile
// (channel order as it is): rotated and split into hi + lo, or shifted by mu.
template <bool ROPE>
__device__ __forceinline__ void store_key_octets(const ChunkParams& p, const Shared& sh, uint32_t tile, int row, int q,
                                                 int64_t pos, float (&x)[8], float (&y)[8]) {
  uint32_t hx[4], hy[4], lx[4], ly[4];
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    if constexpr (ROPE) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 cs = key_turn(p, pos, 8 * q + k + e);
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
    if constexpr (ROPE) {
      const float2 fa = __half22float2(a), fb = __half22float2(b);
      lx[k / 2] = u32(__floats2half2_rn(x[k] - fa.x, x[k + 1] - fa.y));
      ly[k / 2] = u32(__floats2half2_rn(y[k] - fb.x, y[k + 1] - fb.y));
    }
  }
  sts16(tile + tc::chunk_offset(0, row, q), hx[0], hx[1], hx[2], hx[3]);
  sts16(tile + tc::chunk_offset(1, row, q), hy[0], hy[1], hy[2], hy[3]);
  if constexpr (ROPE) {
    sts16(tile + tc::kTileBytes + tc::chunk_offset(0, row, q), lx[0], lx[1], lx[2], lx[3]);
    sts16(tile + tc::kTileBytes + tc::chunk_offset(1, row, q), ly[0], ly[1], ly[2], ly[3]);
  }
}

// Codes of channels 8 oct .. 8 oct + 7 of a bitstream row (4 * bits words).
__device__ __forceinline__ uint32_t octet(const uint32_t* row, int bits, int oct) {
  const int off = 8 * oct * bits, w = off >> 5;
  const uint32_t lo = __ldg(row + w), hi = __ldg(row + min(w + 1, 4 * bits - 1));
  return __funnelshift_r(lo, hi, off & 31);
}

// Key tile of bitstream pages: lane = token, one octet pair of channels at a time.
template <bool ROPE>
__device__ __forceinline__ void key_tile_bits(const ChunkParams& p, const Shared& sh, const uint8_t* unit_pages,
                                              int64_t page0, uint32_t tile, int warp, int lane) {
  const int bits = p.bk, mask = (1 << bits) - 1;
  for (int task = warp; task < 32; task += kWarps) {
    const int q = task >> 2, tok = 32 * (task & 3) + lane;
    const int in_tile = tok / p.R;
    const int64_t page = page0 + in_tile;
    float x[8], y[8];
    int64_t pos = 0;
    if (in_tile < p.pages_per_tile && page < p.n_pages) {
      const int tk = tok - in_tile * p.R;
      const uint8_t* pg = unit_pages + page * p.lay.bytes;
      pos = p.n_s + page * p.R + tk;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(pg + p.lay.off_kc) + tk * 4 * bits;
      const uint32_t cx = octet(row, bits, q), cy = octet(row, bits, q + 8);
      const uint4* mp = reinterpret_cast<const uint4*>(pg + p.lay.off_km) + (tk / p.G) * (kD / 4);
      uint4 mv[4] = {__ldg(mp + 2 * q), __ldg(mp + 2 * q + 1), __ldg(mp + 16 + 2 * q), __ldg(mp + 17 + 2 * q)};
      const uint32_t* m = reinterpret_cast<const uint32_t*>(mv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __half2 a = h2(m[k]), b = h2(m[8 + k]);
        const int ca = (cx >> (bits * k)) & mask, cb = (cy >> (bits * k)) & mask;
        const float fa = p.lut ? sh.k_lev[ca] : (float)ca, fb = p.lut ? sh.k_lev[cb] : (float)cb;
        x[k] = fmaf(__high2float(a), fa, __low2float(a));
        y[k] = fmaf(__high2float(b), fb, __low2float(b));
      }
      for (int e = 0; e < p.nsp; ++e) {
        const int c = pg[p.lay.off_si + tk * p.nsp + e];
        const float v = __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(pg + p.lay.off_sv)[tk * p.nsp + e]));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (c == 8 * q + k) x[k] = v;
          if (c == 64 + 8 * q + k) y[k] = v;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = y[k] = 0.0f;
    }
    store_key_octets<ROPE>(p, sh, tile, tok, q, pos, x, y);
  }
}

// Value tile of bitstream pages: lane = two neighbouring tokens, one octet of channels at a time.
__device__ __forceinline__ void value_tile_bits(const ChunkParams& p, const Shared& sh, const uint8_t* unit_pages,
                                                int64_t page0, uint32_t tile, int warp, int lane) {
  const int bits = p.bv, mask = (1 << bits) - 1;
  for (int task = warp; task < 32; task += kWarps) {
    const int q = task >> 1, tp = 32 * (task & 1) + lane, tok = 2 * tp;
    const int in_tile = tok / p.R;
    const int64_t page = page0 + in_tile;
    uint32_t o[8] = {};
    if (in_tile < p.pages_per_tile && page < p.n_pages) {
      const int tk = tok - in_tile * p.R;
      const uint8_t* pg = unit_pages + page * p.lay.bytes;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(pg + p.lay.off_vc) + tk * 4 * bits;
      const uint32_t c0 = octet(row, bits, q), c1 = octet(row + 4 * bits, bits, q);
      const uint32_t* m = reinterpret_cast<const uint32_t*>(pg + p.lay.off_vm) + tk * (kD / p.G) + 8 * q / p.G;
      const __half2 a = h2(__ldg(m)), b = h2(__ldg(m + kD / p.G));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i0 = (c0 >> (bits * k)) & mask, i1 = (c1 >> (bits * k)) & mask;
        const float f0 = p.lut ? sh.v_lev[i0] : (float)i0, f1 = p.lut ? sh.v_lev[i1] : (float)i1;
        o[k] = u32(__floats2half2_rn(fmaf(__high2float(a), f0, __low2float(a)), fmaf(__high2float(b), f1, __low2float(b))));
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      sts4(tile + tc::chunk_offset(tp >> 5, value_row(8 * q + k), (tp & 31) >> 2) + 4 * (tp & 3), o[k]);
  }
}

// Sparse entries of fragment-order pages, over the dense keys already in the tile.
__device__ __forceinline__ void sparse_keys(const ChunkParams& p, const Shared& sh, const uint8_t* unit_pages,
                                            int64_t page0, uint32_t tile, int tid) {
  for (int i = tid; i < kTile * p.nsp; i += kThreads) {
    const int tok = i / p.nsp, e = i - tok * p.nsp;
    const int in_tile = tok / p.R;
    const int64_t page = page0 + in_tile;
    if (in_tile >= p.pages_per_tile || page >= p.n_pages) continue;
    const int tk = tok - in_tile * p.R;
    const uint8_t* pg = unit_pages + page * p.lay.bytes;
    const int c = pg[p.lay.off_si + tk * p.nsp + e];
    const float v = __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(pg + p.lay.off_sv)[tk * p.nsp + e]));
    const float m = __half2float(reinterpret_cast<const __half*>(sh.mu)[c]);
    const int x = tok & 31;  // 16a + 8b + 2t' + e'
    const int row = (tok & ~31) + 8 * ((x & 7) >> 1) + 4 * (x >> 4) + 2 * ((x >> 3) & 1) + (x & 1);
    sts2(tile + frag_column(row, c), __half_as_ushort(__float2half_rn(v - m)));
  }
}

// Source row of concatenated fp16 row j of a unit: the cache's rows, then the new tokens.
__device__ __forceinline__ const uint16_t* f16_row(const uint16_t* rows, const uint16_t* fresh, int n_w, int64_t j) {
  return j < n_w ? rows + j * kD : fresh + (j - n_w) * kD;
}

// Keys of an fp16 tile: rows j0 .. j0 + 127 of the list, zeros from `end` on.
template <bool FRAG, bool ROPE>
__device__ __forceinline__ void key_tile_f16(const ChunkParams& p, const Shared& sh, const uint16_t* rows,
                                             const uint16_t* fresh, int64_t j0, int64_t end, uint32_t tile, int warp,
                                             int lane) {
  if constexpr (FRAG) {
    for (int task = warp; task < 16; task += kWarps) {
      const int row = 8 * task + (lane >> 2), q = lane & 3;
      uint4 v[4] = {};
      if (j0 + row < end) {
        const uint4* src = reinterpret_cast<const uint4*>(f16_row(rows, fresh, p.n_w, j0 + row)) + 4 * q;
        uint32_t* x = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(src + i);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = u32(__hsub2(h2(x[i]), sh.mu[16 * q + i]));
      }
      store_frag_row(tile, row, q, v);
    }
  } else {
    for (int task = warp; task < 32; task += kWarps) {
      const int q = task >> 2, row = 32 * (task & 3) + lane;
      const int64_t j = j0 + row;
      float x[8] = {}, y[8] = {};
      if (j < end) {
        const uint4* src = reinterpret_cast<const uint4*>(f16_row(rows, fresh, p.n_w, j));
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
      // positions: the sink's rows first, the window behind the quantized tokens, then the new tokens
      store_key_octets<ROPE>(p, sh, tile, row, q, j < p.n_s ? j : j + p.Tq, x, y);
    }
  }
}

// Values of an fp16 tile.  Tokens from `cut` on are hidden from some of the job's rows, and 0 * inf or
// 0 * NaN would carry what they hold into those rows: non-finite values there enter the product as 0
// and are marked, for patch_values to add to the rows that do see them.
__device__ __forceinline__ void value_tile_f16(const ChunkParams& p, Shared& sh, const uint16_t* rows,
                                               const uint16_t* fresh, int64_t j0, int64_t end, int64_t cut,
                                               uint32_t tile, int warp, int lane) {
  for (int task = warp; task < 32; task += kWarps) {
    const int cp = 32 * (task & 1) + lane, o = task >> 1;  // channel pair, octet of tokens
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t j = j0 + 8 * o + i;
      x[i] = j < end ? __ldg(reinterpret_cast<const uint32_t*>(f16_row(rows, fresh, p.n_w, j)) + cp) : 0u;
    }
    if (j0 + 8 * o + 7 >= cut) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool lo = (x[i] & 0x7C00u) == 0x7C00u, hi = (x[i] & 0x7C000000u) == 0x7C000000u;
        if ((lo || hi) && j0 + 8 * o + i >= cut) {
          x[i] &= lo ? 0xFFFF0000u : 0xFFFFFFFFu;
          x[i] &= hi ? 0x0000FFFFu : 0xFFFFFFFFu;
          sh.bad = 1;
          atomicOr(&sh.bad_tokens[o >> 2], 1u << ((8 * o + i) & 31));
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t sel = e ? 0x7632 : 0x5410;
      sts16(tile + tc::chunk_offset(o >> 3, value_row(2 * cp + e), o & 7), __byte_perm(x[0], x[1], sel),
            __byte_perm(x[2], x[3], sel), __byte_perm(x[4], x[5], sel), __byte_perm(x[6], x[7], sel));
    }
  }
}

// Add p_j v_j for the marked non-finite values of a tile to the rows that see token j (rare and slow).
__device__ __noinline__ void patch_values(const ChunkParams& p, const Shared& sh, const uint16_t* rows,
                                          const uint16_t* fresh, int64_t j0, int limit, uint32_t tmem) {
  for (int j = 0; j < kTile; ++j) {
    if (!((sh.bad_tokens[j >> 5] >> (j & 31)) & 1u)) continue;
    const uint32_t pair = tc::ld1(tmem + j / 2);
    tc::wait_ld();
    const float w = __half2float(j & 1 ? __high2half(h2(pair)) : __low2half(h2(pair)));
    const uint16_t* v = f16_row(rows, fresh, p.n_w, j0 + j);
    for (int c = 0; c < kD; ++c) {
      const float f = __half2float(__ushort_as_half(v[c]));
      if (isfinite(f)) continue;
      const uint32_t at = tmem + kTile + value_row(c);
      const uint32_t acc = tc::ld1(at);
      tc::wait_ld();
      const float sum = __uint_as_float(acc) + w * f;
      tc::st1(at, j < limit ? __float_as_uint(sum) : acc);
      tc::wait_st();
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ the kernel

// BK, BV: code widths of fragment-order pages, or 0 for bitstream pages (widths at run time).
template <int BK, int BV, bool ROPE>
__global__ void __launch_bounds__(kThreads, ROPE ? 1 : 2) chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr bool FRAG = BK != 0;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + tc::kTileBytes, sv = sk + (ROPE ? 2 : 1) * tc::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    fence_mbar_init();
  }
  if (tid < 16) {
    sh.k_lev[tid] = p.k_lev[tid];
    sh.v_lev[tid] = p.v_lev[tid];
  }
  if (warp == 0) tc::alloc(&sh.tmem, kTmemColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t my_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  pdl_allow_next();

  uint32_t phase = 0;
  bool failed = false;
  const int64_t g_begin = (int64_t)blockIdx.x * p.per_cta;
  const int64_t g_end = min(g_begin + p.per_cta, p.total_tiles);
  const int hg = 1 << p.log2hg;
  for (int64_t g = g_begin; g < g_end && !failed;) {
    const Piece x = find_piece(p, g);
    const int64_t t_begin = g - x.job_start;
    const int64_t t_end = min(x.tiles, t_begin + (g_end - g));
    const int64_t b = x.unit / p.Hkv, kvh = x.unit - b * p.Hkv;
    const uint8_t* unit_pages = p.pages + x.unit * p.unit_page_stride;
    const uint16_t* rows_k = p.wk + x.unit * p.win_unit_stride;
    const uint16_t* rows_v = p.wv + x.unit * p.win_unit_stride;
    const uint16_t* new_k = p.k_new + x.unit * p.n * kD;
    const uint16_t* new_v = p.v_new + x.unit * p.n * kD;
    const int rows = x.tokens << p.log2hg;

    // queries: row r = token r / hg, head r % hg of the group; channels in the key tile's column order
    for (int task = warp; task < 16; task += kWarps) {
      const int r = 8 * task + (lane >> 2), q = lane & 3;
      uint4 v[4] = {};
      if (r < rows) {
        const int64_t row = (b * p.Hq + kvh * hg + (r & (hg - 1))) * p.n + x.tok0 + (r >> p.log2hg);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + row * kD) + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(src + i);
      }
      if constexpr (FRAG) {
        store_frag_row(sq, r, q, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sts16(sq + tc::chunk_offset(q >> 1, r, 4 * (q & 1) + i), v[i].x, v[i].y, v[i].z, v[i].w);
      }
    }
    // mu: the centre of each channel's range in one page of the unit
    if (tid < kD) {
      float mu = 0.0f;
      if (!ROPE && p.n_pages > 0) {
        const uint8_t* pg = unit_pages + (p.n_pages / 2) * p.lay.bytes;
        const __half2 m = h2(reinterpret_cast<const uint32_t*>(pg + p.lay.off_km)[tid]);
        const float range = __high2float(m) * (float)((1 << p.bk) - 1);
        const float centre = __low2float(m) + 0.5f * range;
        if (fabsf(centre) > range && fabsf(centre) <= 4096.0f) mu = centre;
      }
      reinterpret_cast<__half*>(sh.mu)[tid] = __float2half_rn(mu);
    }
    __syncthreads();

    float m_run = -INFINITY, l_run = 0.0f;
    for (int64_t t = t_begin; t < t_end; ++t) {
      const bool first = t == t_begin, paged = t < p.page_tiles;
      const int64_t j0 = (t - p.page_tiles) * kTile;  // first concatenated fp16 row of an fp16 tile
      if (tid < 5) {
        if (tid == 4) sh.bad = 0;
        else sh.bad_tokens[tid] = 0;
      }
      int valid = kTile;  // columns of a page tile that hold tokens
      if (paged) {
        const int64_t page0 = t * p.pages_per_tile;
        const int64_t left = p.n_pages - page0;
        valid = (int)(left < p.pages_per_tile ? left : p.pages_per_tile) * p.R;
        if constexpr (FRAG) {
          // warps 0..3: keys of 32-token block `warp`, warps 4..7: values
          const int slot = warp & 3, tok = 32 * slot;
          if (tok < valid) {
            const int in_tile = tok / p.R;
            const uint8_t* pg = unit_pages + (page0 + in_tile) * p.lay.bytes;
            const int block = (tok - in_tile * p.R) / 32;
            if (warp < 4) key_block<BK>(p, sh, pg, block, slot, sk, lane);
            else value_block<BV>(p, pg, block, slot, sv, lane);
          } else if (warp < 4) {
            for (int i = lane; i < 32 * 16; i += 32)
              sts16(sk + tc::chunk_offset(i >> 8, tok + ((i & 255) >> 3), i & 7), 0, 0, 0, 0);
          } else {
            for (int i = lane; i < 128 * 4; i += 32)
              sts16(sv + tc::chunk_offset(slot >> 1, i >> 2, 4 * (slot & 1) + (i & 3)), 0, 0, 0, 0);
          }
          if (p.nsp > 0) {
            __syncthreads();
            sparse_keys(p, sh, unit_pages, page0, sk, tid);
          }
        } else {
          key_tile_bits<ROPE>(p, sh, unit_pages, page0, sk, warp, lane);
          value_tile_bits(p, sh, unit_pages, page0, sv, warp, lane);
        }
      } else {
        const int64_t end = p.n_w + x.tok0 + x.tokens;  // rows the job's last token sees
        __syncthreads();                                // the marks are cleared
        key_tile_f16<FRAG, ROPE>(p, sh, rows_k, new_k, j0, end, sk, warp, lane);
        value_tile_f16(p, sh, rows_v, new_v, j0, end, p.n_w + x.tok0 + 1, sv, warp, lane);
      }
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * tc::kBlockBytes + (k & 3) * 32;
          tc::mma_ss(tmem, tc::descriptor(sq + off), tc::descriptor(sk + off), tc::instruction(kTile), k > 0);
        }
        if constexpr (ROPE) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t off = (k >> 2) * tc::kBlockBytes + (k & 3) * 32;
            tc::mma_ss(tmem, tc::descriptor(sq + off), tc::descriptor(sk + tc::kTileBytes + off),
                       tc::instruction(kTile), true);
          }
        }
        tc::commit(&sh.bar);
      }
      failed |= !mbar_wait(&sh.bar, phase);
      phase ^= 1;
      tc::fence_after();
      int limit = valid;  // columns this thread's row sees
      if (warp < 4) {
        const int r = tid;
        if (!paged) {
          const int64_t seen = p.n_w + x.tok0 + (r >> p.log2hg) + 1 - j0;
          limit = (int)(seen < 0 ? 0 : seen > kTile ? kTile : seen);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t s[32];
          tc::ld32(my_tmem + 32 * y, s);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * y + i < limit) mx = fmaxf(mx, __uint_as_float(s[i]));
        }
        const float ms = mx * p.scale_log2;
        const bool renew = ms > m_run + kLazy;  // also from -inf
        const float factor = renew ? ex2(m_run - ms) : 1.0f;
        if (renew) m_run = ms;
        l_run *= factor;
        if (!first && __any_sync(0xffffffffu, renew)) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t o[32];
            tc::ld32(my_tmem + kTile + 32 * y, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
            tc::st32(my_tmem + kTile + 32 * y, o);
          }
        }
        const float shift = kWeightExp - (m_run == -INFINITY ? 0.0f : m_run);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t s[32], w[16];
          tc::ld32(my_tmem + 32 * y, s);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a = ex2(fmaf(__uint_as_float(s[i]), p.scale_log2, shift));
            float c = ex2(fmaf(__uint_as_float(s[i + 1]), p.scale_log2, shift));
            a = 32 * y + i < limit ? a : 0.0f;
            c = 32 * y + i + 1 < limit ? c : 0.0f;
            l_run += a + c;
            w[i / 2] = u32(__floats2half2_rn(a, c));
          }
          tc::st16(my_tmem + 16 * y, w);
        }
        tc::wait_st();
      }
      tc::fence_before();
      __syncthreads();
      if (tid == 0) {
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * tc::kBlockBytes + (k & 3) * 32;
          tc::mma_ts(tmem + kTile, tmem + 8 * k, tc::descriptor(sv + off), tc::instruction(kD), !(first && k == 0));
        }
        tc::commit(&sh.bar);
      }
      failed |= !mbar_wait(&sh.bar, phase);
      phase ^= 1;
      tc::fence_after();
      if (warp < 4 && sh.bad) patch_values(p, sh, rows_v, new_v, j0, limit, my_tmem);
      failed = __syncthreads_or(failed);
      if (failed) break;
    }

    // the row's result, or its partial when the job is cut
    if (warp < 4 && !failed) {
      const bool whole = t_begin == 0 && t_end == x.tiles;
      const int r = tid;
      const float inv = l_run > 0.0f ? 1.0f / l_run : l_run == 0.0f ? 0.0f : l_run;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (t_begin == 0 ? 1 : 0);
      const int64_t row = (b * p.Hq + kvh * hg + (r & (hg - 1))) * p.n + x.tok0 + (r >> p.log2hg);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t o[32];
        tc::ld32(my_tmem + kTile + 32 * y, o);
        tc::wait_ld();
        if (r < rows) {
          // column 8c + (e << 2 | i) holds channel 8c + 2i + e
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + row * kD) + 4 * y;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = u32(__floats2half2_rn(__uint_as_float(o[8 * c + i]) * inv, __uint_as_float(o[8 * c + 4 + i]) * inv));
              dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_acc + (slot * p.rows_max + r) * kD) + 8 * y;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 4; i += 2)
                dst[2 * c + i / 2] = make_float4(__uint_as_float(o[8 * c + i]), __uint_as_float(o[8 * c + 4 + i]),
                                                 __uint_as_float(o[8 * c + i + 1]), __uint_as_float(o[8 * c + 5 + i]));
          }
        }
      }
      if (!whole && r < rows)
        *reinterpret_cast<float2*>(p.part_ml + (slot * p.rows_max + r) * 2) = make_float2(m_run, l_run);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    g += t_end - t_begin;
  }
  if (failed && tid == 0) report_error(p.err, kDevWaitTimeout);
  __syncthreads();
  if (warp == 0) tc::dealloc(tmem, kTmemColumns);
}

// Join the partials of the jobs that the cuts between CTAs divide: CTA x of the grid handles the job that
// the cut before piece x + 1 divides, if no earlier cut divides it too; a warp per query row.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) merge_chunk_kernel(const __grid_constant__ ChunkParams p) {
  pdl_wait();
  const int64_t cut = ((int64_t)blockIdx.x + 1) * p.per_cta;
  const Piece x = find_piece(p, cut);
  if (x.job_start >= cut) return;              // the cut falls between two jobs
  if (cut - p.per_cta > x.job_start) return;   // an earlier cut divides the same job
  const int64_t c0 = blockIdx.x, c1 = (x.job_start + x.tiles - 1) / p.per_cta;
  const int hg = 1 << p.log2hg, rows = x.tokens << p.log2hg;
  const int lane = threadIdx.x & 31;
  const int64_t b = x.unit / p.Hkv, kvh = x.unit - b * p.Hkv;
  for (int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); r < rows; r += gridDim.y * (kMergeThreads / 32)) {
    float M = -INFINITY, L = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t c = c0; c <= c1; ++c) {
      const int64_t slot = 2 * c + (c == c0 ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * p.rows_max + r) * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_acc + (slot * p.rows_max + r) * kD + 4 * lane);
      const float m = fmaxf(M, ml.x);
      const float fo = M == -INFINITY ? 0.0f : exp2f(M - m), fn = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x - m);
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // no key of that piece is visible to the row
      L = L * fo + ml.y * fn;
      a.x = a.x * fo + v.x * fn;
      a.y = a.y * fo + v.y * fn;
      a.z = a.z * fo + v.z * fn;
      a.w = a.w * fo + v.w * fn;
      M = m;
    }
    const float inv = L > 0.0f ? 1.0f / L : L == 0.0f ? 0.0f : L;
    const int64_t row = (b * p.Hq + kvh * hg + (r & (hg - 1))) * p.n + x.tok0 + (r >> p.log2hg);
    const __half2 lo = __floats2half2_rn(a.x * inv, a.y * inv), hi = __floats2half2_rn(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * kD + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

constexpr int kCtasPerSm = 2;

int64_t slot_rows(int64_t n, int hg) { return n * hg < kRows ? n * hg : kRows; }

template <int BK, int BV, bool ROPE>
cudaError_t launch_t(const ChunkParams& p, int64_t grid, int* launches, cudaStream_t s) {
  constexpr size_t smem = (ROPE ? 4 : 3) * tc::kTileBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel<BK, BV, ROPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  chunk_kernel<BK, BV, ROPE><<<(unsigned)grid, kThreads, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  if (grid == 1) return cudaSuccess;
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

// Two partial slots per CTA, each with the rows a job can have, of D + 2 floats a row.
int64_t chunk_workspace_bytes(int64_t n, int hg, int sm_count) {
  return 2 * (int64_t)kCtasPerSm * sm_count * slot_rows(n, hg) * (kD + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_chunk(ChunkParams p, bool rope, int sm_count, void* workspace, int* launches, cudaStream_t s) {
  const int hg = 1 << p.log2hg;
  p.log2_job_tokens = 7 - p.log2hg;
  p.pages_per_tile = kTile / p.R;
  p.page_tiles = (p.n_pages + p.pages_per_tile - 1) / p.pages_per_tile;
  const int64_t job_tokens = (int64_t)1 << p.log2_job_tokens;
  p.jobs_per_unit = (p.n + job_tokens - 1) / job_tokens;
  p.tiles_per_unit = p.jobs_per_unit * p.page_tiles + f16_tiles_before(p.n_w, p.log2_job_tokens, p.jobs_per_unit - 1) +
                     ((p.n_w + p.n + 127) >> 7);
  p.total_tiles = p.n_units * p.tiles_per_unit;
  const int64_t resident = (int64_t)(rope ? 1 : kCtasPerSm) * sm_count;
  int64_t grid = p.total_tiles < resident ? p.total_tiles : resident;
  p.per_cta = (p.total_tiles + grid - 1) / grid;
  grid = (p.total_tiles + p.per_cta - 1) / p.per_cta;
  p.rows_max = (int32_t)slot_rows(p.n, hg);
  p.part_acc = static_cast<float*>(workspace);
  p.part_ml = p.part_acc + 2 * resident * p.rows_max * kD;
  if (p.lay.frag) {
    if (p.bk == 2 && p.bv == 2) return launch_t<2, 2, false>(p, grid, launches, s);
    if (p.bk == 4 && p.bv == 2) return launch_t<4, 2, false>(p, grid, launches, s);
    if (p.bk == 4 && p.bv == 4) return launch_t<4, 4, false>(p, grid, launches, s);
    return cudaErrorInvalidValue;
  }
  return rope ? launch_t<0, 0, true>(p, grid, launches, s) : launch_t<0, 0, false>(p, grid, launches, s);
}

}  // namespace kvq
