// Rotary positions of new queries and keys, from the projections' layout into the cache's
// (kvq_rope in include/kvq.h).
//
// Pair i of a head is turned by the angle t = pos * w_i and scaled by the gain m of the long-context
// scaling:  x'_a = m (x_a cos t - x_b sin t),  x'_b = m (x_a sin t + x_b cos t).
//
// Angles: w_i / (2 pi) is kept as a 0.64 fixed-point fraction of a turn (the form the decode kernels
// use for keys rotated at decode), so pos * w_i modulo one turn is one 64-bit product whose overflow
// drops the whole turns: exact to 2^-64 * pos turns whatever the position, where an fp32 angle would
// lose the sine of far positions altogether.  Its top 32 bits, as a signed fraction in [-1/2, 1/2),
// go through sincospif in fp32.
//
// Every element is read once and written once, so HBM bounds it; the trigonometry is shared by all
// heads of a token: a CTA takes a few tokens, computes their cosines and sines once into shared
// memory and then streams 16-byte chunks of every head of them.
//
// Measured (GB300): 32768 tokens x 48 heads of bf16 to fp16, 805 MB, 137 us (5.9 TB/s, 0.86 of the copy rate); the
// few rows of a decode step are bound by the launch and the host's call.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvq.h"
#include "kvq_internal.h"

namespace {

constexpr int kMaxPairs = 128;  // head_dim up to 256
constexpr int kMaxParts = 4;
constexpr int kThreads = 256;
constexpr int kMaxTileTokens = 16;

struct RopePart {
  const void* x;
  void* out;
  int64_t xb, xt, xh, ob, ot, oh;  // strides in elements
  int32_t rotate;
  int32_t head0;  // first of the part's heads in the list of all parts' heads
};

struct RopeParams {
  unsigned long long turns[kMaxPairs];
  RopePart part[kMaxParts];
  int32_t n_parts, heads;  // heads of all parts
  int32_t D, rot, interleaved;
  float gain;
  int64_t batch, n_tokens;
  const int64_t* positions;  // [batch][n_tokens] or null: position0 + token
  int64_t position0;
  int32_t log2_tile;    // tokens of a CTA's tile
  int32_t head_splits;  // CTAs that share a tile, each with heads_per_cta heads
  int32_t heads_per_cta;
  int64_t tiles;        // ceil(batch * n_tokens / tile)
};

__device__ __forceinline__ float2 turn_of(const RopeParams& p, int64_t pos, int pair) {
  const unsigned long long t = (unsigned long long)pos * p.turns[pair];  // modulo 2^64: modulo one turn
  float s, c;
  sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c * p.gain, s * p.gain);
}

__device__ __forceinline__ int64_t position_of(const RopeParams& p, int64_t bt) {
  return p.positions ? p.positions[bt] : p.position0 + bt % p.n_tokens;
}

// fp32 values of elements, and their rounding to nearest
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements through 16-byte accesses.
template <typename T>
struct Chunk {
  static constexpr int kWords = (int)sizeof(T) / 2;  // 16-byte words
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* at) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(at) + i);
  }
  __device__ __forceinline__ void store(T* at) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(at)[i] = w[i];
  }
  __device__ __forceinline__ float get(int i) const {
    T v;
    memcpy(&v, reinterpret_cast<const char*>(w) + i * sizeof(T), sizeof(T));
    return widen(v);
  }
  __device__ __forceinline__ void set(int i, float f) {
    const T v = narrow<T>(f);
    memcpy(reinterpret_cast<char*>(w) + i * sizeof(T), &v, sizeof(T));
  }
};

// Vector form: 16-byte aligned rows, head_dim and the rotated part multiples of 16.  A task is two
// 8-channel chunks of a head: the two halves of eight pairs (half layout), or sixteen consecutive
// channels (interleaved pairs, or channels that are only moved); both use the turns of pairs 8j..8j+7.
// A thread keeps its token and its chunks and walks over the heads, so its eight turns stay in registers and an
// address moves by a stride: with a division per task to find its place the prompt above took 193 us.
template <typename TX, typename TO, bool HALVES>
__global__ void __launch_bounds__(kThreads) rope_vector_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 turn[kMaxTileTokens * kMaxPairs];
  const int64_t tile = blockIdx.x / p.head_splits;
  const int head0 = (int)(blockIdx.x % p.head_splits) * p.heads_per_cta;
  const int head1 = min(head0 + p.heads_per_cta, p.heads);
  const int64_t bt0 = tile << p.log2_tile;
  const int64_t total = p.batch * p.n_tokens;
  const int tokens = (int)min((int64_t)1 << p.log2_tile, total - bt0);
  const int pairs = p.rot / 2, chunks = p.D / 16, rot_chunks = p.rot / 16;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tok = i / pairs;
    turn[i] = turn_of(p, position_of(p, bt0 + tok), i - tok * pairs);
  }
  __syncthreads();
  // thread -> (head of a group, token, chunk), the chunk fastest: a warp writes neighbouring tokens' rows of a head
  const int row = threadIdx.x / chunks, j = threadIdx.x - row * chunks;
  const int tok = row & ((1 << p.log2_tile) - 1), hp = row >> p.log2_tile;
  const int step = kThreads / (chunks << p.log2_tile);
  if (hp >= step || tok >= tokens) return;
  const int64_t b = (bt0 + tok) / p.n_tokens, t = (bt0 + tok) - b * p.n_tokens;
  const bool in_rot = j < rot_chunks;
  float2 cs[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) cs[k] = in_rot ? turn[tok * pairs + 8 * j + k] : make_float2(1.0f, 0.0f);
#pragma unroll 1
  for (int pi = 0; pi < p.n_parts; ++pi) {
    const RopePart& part = p.part[pi];
    const int first = max(head0, part.head0);
    const int last = min(head1, pi + 1 < p.n_parts ? p.part[pi + 1].head0 : p.heads);
    const bool turned = part.rotate && in_rot, halves = HALVES && turned;
    const int ca = halves ? 8 * j : 16 * j, cb = halves ? p.rot / 2 + 8 * j : 16 * j + 8;
    const TX* x = static_cast<const TX*>(part.x) + b * part.xb + t * part.xt + (first + hp - part.head0) * part.xh;
    TO* o = static_cast<TO*>(part.out) + b * part.ob + t * part.ot + (first + hp - part.head0) * part.oh;
    const int64_t xs = step * part.xh, os = step * part.oh;
    // a few heads' loads together, then their stores (an output may be its input's own memory, so the compiler
    // cannot move loads over stores by itself)
    constexpr int kTogether = sizeof(TX) == 2 ? 4 : 2;
#pragma unroll 1
    for (int h = first + hp; h < last; h += kTogether * step, x += kTogether * xs, o += kTogether * os) {
      Chunk<TX> a[kTogether], c[kTogether];
#pragma unroll
      for (int e = 0; e < kTogether; ++e) {
        if (h + e * step < last) {
          a[e].load(x + e * xs + ca);
          c[e].load(x + e * xs + cb);
        }
      }
#pragma unroll
      for (int e = 0; e < kTogether; ++e) {
        if (h + e * step >= last) break;
        float u[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          u[k] = a[e].get(k);
          u[8 + k] = c[e].get(k);
        }
        if (turned) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // first and second of pair k: (k, 8 + k) of the two halves, or (2k, 2k + 1)
            float &x0 = u[HALVES ? k : 2 * k], &x1 = u[HALVES ? 8 + k : 2 * k + 1];
            const float y0 = x0 * cs[k].x - x1 * cs[k].y, y1 = x0 * cs[k].y + x1 * cs[k].x;
            x0 = y0;
            x1 = y1;
          }
        }
        Chunk<TO> oa, oc;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          oa.set(k, u[k]);
          oc.set(k, u[8 + k]);
        }
        oa.store(o + e * os + ca);
        oc.store(o + e * os + cb);
      }
    }
  }
}

// Any alignment, strides and even rotated part: one pair of channels at a time.
template <typename TX, typename TO>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 turn[kMaxTileTokens * kMaxPairs];
  const int64_t tile = blockIdx.x / p.head_splits;
  const int head0 = (int)(blockIdx.x % p.head_splits) * p.heads_per_cta;
  const int heads = min(p.heads_per_cta, p.heads - head0);
  const int64_t bt0 = tile << p.log2_tile;
  const int64_t total = p.batch * p.n_tokens;
  const int tokens = (int)min((int64_t)1 << p.log2_tile, total - bt0);
  const int pairs = p.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tok = i / pairs;
    turn[i] = turn_of(p, position_of(p, bt0 + tok), i - tok * pairs);
  }
  __syncthreads();
  const int units = p.D / 2;  // pairs, then the channels behind the rotated part two at a time
  const int tasks = heads * tokens * units;
  for (int i = threadIdx.x; i < tasks; i += kThreads) {
    const int row = i / units, j = i - row * units;
    const int h_rel = row / tokens, tok = row - h_rel * tokens;
    const int hall = head0 + h_rel;
    int pi = 0;
    for (int k = 1; k < p.n_parts; ++k) pi += hall >= p.part[k].head0 ? 1 : 0;
    const RopePart& part = p.part[pi];
    const int64_t b = (bt0 + tok) / p.n_tokens, t = (bt0 + tok) - b * p.n_tokens;
    const int h = hall - part.head0;
    const bool turned = part.rotate && j < pairs;
    const int ca = turned && !p.interleaved ? j : 2 * j, cb = turned && !p.interleaved ? j + pairs : 2 * j + 1;
    const TX* x = static_cast<const TX*>(part.x) + b * part.xb + t * part.xt + h * part.xh;
    TO* o = static_cast<TO*>(part.out) + b * part.ob + t * part.ot + h * part.oh;
    float x0 = widen(x[ca]), x1 = widen(x[cb]);
    if (turned) {
      const float2 cs = turn[tok * pairs + j];
      const float y0 = x0 * cs.x - x1 * cs.y, y1 = x0 * cs.y + x1 * cs.x;
      x0 = y0;
      x1 = y1;
    }
    o[ca] = narrow<TO>(x0);
    o[cb] = narrow<TO>(x1);
  }
}

template <typename TX, typename TO>
void launch_typed(const RopeParams& p, bool vector, unsigned grid, cudaStream_t s) {
  if (vector && !p.interleaved) rope_vector_kernel<TX, TO, true><<<grid, kThreads, 0, s>>>(p);
  else if (vector) rope_vector_kernel<TX, TO, false><<<grid, kThreads, 0, s>>>(p);
  else rope_scalar_kernel<TX, TO><<<grid, kThreads, 0, s>>>(p);
}

template <typename TX>
void launch_out(const RopeParams& p, int out_type, bool vector, unsigned grid, cudaStream_t s) {
  switch (out_type) {
    case KVQ_TYPE_F16: launch_typed<TX, __half>(p, vector, grid, s); break;
    case KVQ_TYPE_BF16: launch_typed<TX, __nv_bfloat16>(p, vector, grid, s); break;
    default: launch_typed<TX, float>(p, vector, grid, s); break;
  }
}

constexpr double kPi = 3.14159265358979323846264338327950288;

// Angle per position of pair i.
double frequency(const kvq_rope_config& c, int i) {
  double w = std::pow(c.base, -2.0 * i / (double)c.rot_dim);
  switch (c.scaling) {
    case KVQ_ROPE_LINEAR: return w / c.factor;
    case KVQ_ROPE_WAVELENGTH: {  // turns within the original context decide: few -> divided, many -> kept
      const double turns = (double)c.original_context * w / (2.0 * kPi);
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - c.low) / (c.high - c.low)));
      return w / c.factor * (1.0 - keep) + w * keep;
    }
    case KVQ_ROPE_YARN: {  // the same decision, blended linearly in the pair's index
      auto index = [&](double turns) {
        return c.rot_dim * std::log((double)c.original_context / (turns * 2.0 * kPi)) / (2.0 * std::log(c.base));
      };
      const double lo = std::fmax(std::floor(index(c.high)), 0.0);
      const double hi = std::fmin(std::ceil(index(c.low)), (double)c.rot_dim - 1.0);
      const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      return w / c.factor * ramp + w * (1.0 - ramp);
    }
    default: return w;
  }
}

// w / (2 pi) modulo one turn as a 0.64 fixed-point fraction.
unsigned long long turn_fraction(double w) {
  double x = w / (2.0 * kPi);
  x -= std::floor(x);
  const double hi = std::floor(x * 4294967296.0);
  const double lo = std::floor((x * 4294967296.0 - hi) * 4294967296.0);
  return ((unsigned long long)hi << 32) | (unsigned long long)lo;
}

bool finite_positive(double x) { return x > 0.0 && std::isfinite(x); }

int type_bytes(int t) { return t == KVQ_TYPE_F32 ? 4 : 2; }

}  // namespace

extern "C" kvq_status kvq_rope(const kvq_rope_config* cfg, const kvq_rope_part* parts, int32_t n_parts, int32_t x_type,
                               int32_t out_type, int32_t batch, int64_t n_tokens, const int64_t* positions,
                               int64_t position0, void* stream) {
  if (!cfg || !parts) return KVQ_ERR_INVALID_ARG;
  const kvq_rope_config& c = *cfg;
  if (c.head_dim < 2 || c.rot_dim < 2 || c.rot_dim > c.head_dim || c.rot_dim % 2 || c.head_dim % 2)
    return KVQ_ERR_INVALID_ARG;
  if (c.interleaved != 0 && c.interleaved != 1) return KVQ_ERR_INVALID_ARG;
  if (!(c.base > 1.0) || !std::isfinite(c.base) || !finite_positive(c.attention_factor)) return KVQ_ERR_INVALID_ARG;
  if (c.scaling < KVQ_ROPE_NONE || c.scaling > KVQ_ROPE_YARN) return KVQ_ERR_INVALID_ARG;
  if (c.scaling != KVQ_ROPE_NONE && !finite_positive(c.factor)) return KVQ_ERR_INVALID_ARG;
  if ((c.scaling == KVQ_ROPE_WAVELENGTH || c.scaling == KVQ_ROPE_YARN) &&
      (c.original_context < 1 || !finite_positive(c.low) || !finite_positive(c.high) || !(c.high > c.low)))
    return KVQ_ERR_INVALID_ARG;
  if (x_type < KVQ_TYPE_F16 || x_type > KVQ_TYPE_F32 || out_type < KVQ_TYPE_F16 || out_type > KVQ_TYPE_F32)
    return KVQ_ERR_INVALID_ARG;
  if (n_parts < 1 || batch < 1 || n_tokens < 1) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(positions) % 8) return KVQ_ERR_INVALID_ARG;
  if (n_parts > kMaxParts || c.head_dim > 2 * kMaxPairs) return KVQ_ERR_UNSUPPORTED;
  const int xs = type_bytes(x_type), os = type_bytes(out_type);
  RopeParams p{};
  bool vector = c.head_dim % 16 == 0 && c.rot_dim % 16 == 0;
  int64_t heads = 0;
  for (int i = 0; i < n_parts; ++i) {
    const kvq_rope_part& q = parts[i];
    if (!q.x || !q.out || q.num_heads < 1 || (q.rotate != 0 && q.rotate != 1)) return KVQ_ERR_INVALID_ARG;
    if (q.x == q.out && (x_type != out_type || (batch > 1 && q.x_batch_stride != q.out_batch_stride) ||
                         (n_tokens > 1 && q.x_token_stride != q.out_token_stride) ||
                         (q.num_heads > 1 && q.x_head_stride != q.out_head_stride)))
      return KVQ_ERR_INVALID_ARG;  // in place, every element is written where it was read
    if (reinterpret_cast<uintptr_t>(q.x) % xs || reinterpret_cast<uintptr_t>(q.out) % os) return KVQ_ERR_INVALID_ARG;
    auto vec = [](const void* ptr, int64_t a, int64_t b, int64_t h, int size) {
      return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (a * size) % 16 == 0 && (b * size) % 16 == 0 &&
             (h * size) % 16 == 0;
    };
    vector = vector && vec(q.x, q.x_batch_stride, q.x_token_stride, q.x_head_stride, xs) &&
             vec(q.out, q.out_batch_stride, q.out_token_stride, q.out_head_stride, os);
    p.part[i] = RopePart{q.x, q.out, q.x_batch_stride, q.x_token_stride, q.x_head_stride,
                         q.out_batch_stride, q.out_token_stride, q.out_head_stride, q.rotate, (int32_t)heads};
    heads += q.num_heads;
  }
  if (heads > 65536 || n_tokens > ((int64_t)1 << 40) / batch) return KVQ_ERR_UNSUPPORTED;
  for (int i = 0; i < c.rot_dim / 2; ++i) p.turns[i] = turn_fraction(frequency(c, i));
  p.n_parts = n_parts;
  p.heads = (int32_t)heads;
  p.D = c.head_dim;
  p.rot = c.rot_dim;
  p.interleaved = c.interleaved;
  p.gain = (float)c.attention_factor;
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.positions = positions;
  p.position0 = position0;
  // Tokens of a tile: as many as still leave a few CTAs per SM (their sines are shared by all heads
  // only within a CTA, so heads are split over CTAs only when there are too few tokens).
  const int64_t total = batch * n_tokens;
  const int64_t enough = 4 * 152;
  while (p.log2_tile < 4 && (total >> (p.log2_tile + 1)) >= enough) p.log2_tile++;
  p.tiles = (total + ((int64_t)1 << p.log2_tile) - 1) >> p.log2_tile;
  p.head_splits = 1;
  if (p.tiles < enough) {
    const int64_t want = (enough + p.tiles - 1) / p.tiles;
    p.head_splits = (int32_t)(want < heads ? want : heads);
  }
  p.heads_per_cta = (int32_t)((heads + p.head_splits - 1) / p.head_splits);
  p.head_splits = (int32_t)((heads + p.heads_per_cta - 1) / p.heads_per_cta);
  const int64_t grid = p.tiles * p.head_splits;
  if (grid > 0x7fffffffll) return KVQ_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (x_type) {
    case KVQ_TYPE_F16: launch_out<__half>(p, out_type, vector, (unsigned)grid, s); break;
    case KVQ_TYPE_BF16: launch_out<__nv_bfloat16>(p, out_type, vector, (unsigned)grid, s); break;
    default: launch_out<float>(p, out_type, vector, (unsigned)grid, s); break;
  }
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
