// Key/value cache in 4 bits: its layout, and the kernels that store into it,
// read it back, pool its keys and evict from it. (Attention over it is in
// kv4_attn.cuh.)
//
// A value x is held as x^ = s * (c - z) with, per token, kv head and group of
// 32 channels, a scale s of four significant bits (5 exponent bits, 3 of
// mantissa: the upper bits of an fp16 number, 2^-17 .. 3840) and a 4-bit zero
// point z, and a 4-bit code c per channel: 72 bytes a row against bf16's 256.
// |c - z| <= 15 takes four bits, so x^ has at most eight significant bits and
// is a multiple of 2^-17: every x^ is exactly a bf16 and exactly an fp16
// number (at most 57600), whichever the products want, and no rounding comes
// after the one into the cache.
//
// The cache of one kv head of one sequence is a run of 64-token tiles of
// 9,216 bytes: [key codes 4096][key parameters 512][value codes 4096][value
// parameters 512], so that a tile is one aligned bulk copy.
//   codes       64 bytes a token; 32-bit word w holds channels 8w .. 8w+7,
//               channel 8w + 2j in nibble j, channel 8w + 2j + 1 in nibble
//               j + 4: one mask yields a pair of neighbours 16 bits apart.
//   values      as the keys, but tokens with bit 2 of their index set hold
//               their two 32-byte halves swapped (the attention kernel reads
//               8-byte pieces of four tokens at a time: two of even and two
//               of odd index, which then fall on all 32 banks).
//   parameters  four uint16 a token: scale code << 7 | z, that is the scale's
//               fp16 bits with the zero point in its free low bits.
#pragma once

#include "common.cuh"

namespace moba {

constexpr int kKv4Tile = 64;                              // tokens in a tile
constexpr int kKv4Row = kHeadDim / 2;                     // code bytes of a token
constexpr int kKv4Params = kKv4Tile * kKv4Row;            // offset of a half's parameters
constexpr int kKv4Half = kKv4Params + kKv4Tile * 8;       // bytes of a tile's keys (and of its values)
constexpr int kKv4TileBytes = 2 * kKv4Half;
constexpr float kKv4Top = 28800.f;  // inputs saturate here: a group's span then stays below 15 * 3840
constexpr uint32_t kKv4ScaleMin = 1, kKv4ScaleMax = 0xD7;  // 2^-17 .. 3840

// Bytes before tile `tile` of head `h` of sequence `b`.
__host__ __device__ __forceinline__ int64_t kv4_tile_off(int64_t tiles, int heads, int b, int h, int64_t tile) {
  return (((int64_t)b * heads + h) * tiles + tile) * kKv4TileBytes;
}

// Byte offset, within a half, of word w of a token's codes.
__device__ __forceinline__ int kv4_word_off(int tok, int w, bool is_v) {
  const int x = is_v ? (w ^ ((tok & 4) << 1)) : w;
  return tok * kKv4Row + x * 4;
}

// Scale of a parameter: its fp16 bits.
__device__ __forceinline__ float kv4_scale(uint32_t par) {
  return __half2float(__ushort_as_half((unsigned short)(par & 0x7F80u)));
}

// The eight channels of a code word, in fp32.
__device__ __forceinline__ void kv4_decode(uint32_t word, uint32_t par, float (&x)[8]) {
  const float s = kv4_scale(par);
  const float z = (float)(par & 15u);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = s * ((float)((word >> (4 * j)) & 15u) - z);
    x[2 * j + 1] = s * ((float)((word >> (4 * j + 16)) & 15u) - z);
  }
}

// A length the caller left on the device: outside [0, capacity] it is a
// caller's error, recorded and cut to the range.
__device__ __forceinline__ int kv4_length(const int32_t* lengths, int b, int64_t capacity) {
  const int n = lengths[b];
  if (n < 0 || n > capacity) {
    record_status(MOBA_ERR_DEVICE_CHECK);
    return n < 0 ? 0 : (int)capacity;
  }
  return n;
}

// Sequence of packed token t: the last b with cu[b] <= t. -1 behind the last
// sequence (or before the first).
__device__ __forceinline__ int kv4_sequence(const int32_t* cu, int batch, int64_t t) {
  if (t < cu[0] || t >= cu[batch]) return -1;
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ append

// Scale code of a step: the nearest value of four significant bits, ties to
// even (below 2^-14, the nearest multiple of 2^-17).
__device__ __forceinline__ uint32_t kv4_scale_code(float step) {
  const uint32_t bits = __float_as_uint(step);
  const uint32_t normal = ((bits + 0x7FFFFu + ((bits >> 20) & 1u)) >> 20) - (112u << 3);
  const uint32_t small = (uint32_t)__float2int_rn(step * 131072.f);
  const uint32_t code = step >= 6.103515625e-05f ? normal : small;
  return min(max(code, kKv4ScaleMin), kKv4ScaleMax);
}

// floor(x / s + 1/2) for |x| <= 28800 and a scale s: the rounded product with
// 1/s is off by one at most, and the remainder x - r s is exact in fp32 (x and
// s r have few bits), so comparing it with s/2 settles it.
__device__ __forceinline__ float kv4_round_quotient(float x, float s, float inv) {
  float r = rintf(x * inv);
  const float d = fmaf(-r, s, x);
  if (d >= 0.5f * s) r += 1.f;
  if (d < -0.5f * s) r -= 1.f;
  return r;
}

// One lane's eight channels of a row; four neighbouring lanes hold a group.
// Returns the code word, and the group's parameter.
__device__ __forceinline__ uint32_t kv4_quantise(uint4 raw, uint32_t* par) {
  float x[8];
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = x[j] == x[j] ? fminf(fmaxf(x[j], -kKv4Top), kKv4Top) : 0.f;  // a NaN is stored as zero
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
  }
  const uint32_t code = kv4_scale_code(__fdiv_rn(hi - lo, 15.f));
  const float s = kv4_scale(code << 7);
  const float inv = __fdiv_rn(1.f, s);
  const float z = fminf(kv4_round_quotient(-lo, s, inv), 15.f);
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float c0 = fminf(fmaxf(kv4_round_quotient(x[2 * j], s, inv) + z, 0.f), 15.f);
    const float c1 = fminf(fmaxf(kv4_round_quotient(x[2 * j + 1], s, inv) + z, 0.f), 15.f);
    word |= (uint32_t)c0 << (4 * j) | (uint32_t)c1 << (4 * j + 16);
  }
  *par = code << 7 | (uint32_t)z;
  return word;
}

struct Kv4AppendParams {
  const __nv_bfloat16 *k, *v;   // [total][heads][128]
  const int32_t *cu, *start;    // [batch + 1] (null: total / batch tokens each), [batch]
  int64_t total, tiles;
  int batch, heads;
  uint8_t* kv4;
  float* acc;                   // [batch][heads][tiles * 64], or null
};

constexpr int kKv4AppendThreads = 256;

// Half a warp per row (token, kv head): 16 lanes of 8 channels, keys and
// values together. HBM-bound: 512 bytes read and 144 written a row.
__global__ void __launch_bounds__(kKv4AppendThreads) kv4_append_kernel(Kv4AppendParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.x * kKv4AppendThreads + threadIdx.x) >> 4;
  const int64_t t = row / p.heads;
  const int h = (int)(row - t * p.heads);
  int b = -1;
  int64_t at = 0;
  if (t < p.total) {
    if (p.cu) {
      b = kv4_sequence(p.cu, p.batch, t);
      if (b >= 0) at = (int64_t)p.start[b] + (t - p.cu[b]);
    } else {
      const int64_t n = p.total / p.batch;
      b = (int)(t / n);
      at = (int64_t)p.start[b] + (t - b * n);
    }
    if (b >= 0 && (at < 0 || at >= p.tiles * kKv4Tile)) {  // no room: skipped and reported
      record_status(MOBA_ERR_DEVICE_CHECK);
      b = -1;
    }
  }
  uint4 rk = make_uint4(0, 0, 0, 0), rv = rk;
  if (b >= 0) {
    rk = __ldg(reinterpret_cast<const uint4*>(p.k + row * kHeadDim) + lane);
    rv = __ldg(reinterpret_cast<const uint4*>(p.v + row * kHeadDim) + lane);
  }
  uint32_t pk, pv;
  const uint32_t wk = kv4_quantise(rk, &pk);
  const uint32_t wv = kv4_quantise(rv, &pv);
  if (b < 0) return;
  const int tok = (int)(at % kKv4Tile);
  uint8_t* tile = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, at / kKv4Tile);
  *reinterpret_cast<uint32_t*>(tile + kv4_word_off(tok, lane, false)) = wk;
  *reinterpret_cast<uint32_t*>(tile + kKv4Half + kv4_word_off(tok, lane, true)) = wv;
  if ((lane & 3) == 0) {
    *reinterpret_cast<uint16_t*>(tile + kKv4Params + tok * 8 + (lane >> 2) * 2) = (uint16_t)pk;
    *reinterpret_cast<uint16_t*>(tile + kKv4Half + kKv4Params + tok * 8 + (lane >> 2) * 2) = (uint16_t)pv;
  }
  if (p.acc && lane == 0) p.acc[((int64_t)b * p.heads + h) * p.tiles * kKv4Tile + at] = 0.f;
}

// ------------------------------------------------------------------ load

struct Kv4LoadParams {
  const uint8_t* kv4;
  const int32_t *lengths, *first;  // first may be null (token 0)
  int64_t tiles, n;
  int batch, heads;
  __nv_bfloat16 *k, *v;  // [batch][n][heads][128]
};

constexpr int kKv4LoadThreads = 256;

// Half a warp per row, 8 channels a lane: 144 bytes read, 512 written.
__global__ void __launch_bounds__(kKv4LoadThreads) kv4_load_kernel(Kv4LoadParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.x * kKv4LoadThreads + threadIdx.x) >> 4;
  if (row >= (int64_t)p.batch * p.n * p.heads) return;
  const int64_t t = row / p.heads;
  const int h = (int)(row - t * p.heads);
  const int b = (int)(t / p.n);
  const int64_t at = (p.first ? (int64_t)p.first[b] : 0) + (t - b * p.n);
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  uint4 o[2] = {};
  if (at >= 0 && at < len) {
    const int tok = (int)(at % kKv4Tile);
    const uint8_t* tile = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, at / kKv4Tile);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint8_t* half = tile + s * kKv4Half;
      const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(half + kv4_word_off(tok, lane, s == 1)));
      const uint32_t par = __ldg(reinterpret_cast<const uint16_t*>(half + kKv4Params + tok * 8 + (lane >> 2) * 2));
      float x[8];
      kv4_decode(word, par, x);
      o[s] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                        pack_bf16x2(x[6], x[7]));
    }
  }
  reinterpret_cast<uint4*>(p.k + row * kHeadDim)[lane] = o[0];
  reinterpret_cast<uint4*>(p.v + row * kHeadDim)[lane] = o[1];
}

// ------------------------------------------------------------------ pool

struct Kv4PoolParams {
  const uint8_t* kv4;
  const int32_t* lengths;
  int64_t tiles;
  int heads, B, blocks;  // blocks = capacity / B
  float* kmean;          // [batch][heads][blocks][128]
};

constexpr int kKv4PoolThreads = 256;

// One CTA per (block, head, sequence): thread = (code word, every 16th token),
// fp32 sums in a fixed order. Blocks that the sequence has not completed are
// written as zero.
__global__ void __launch_bounds__(kKv4PoolThreads) kv4_pool_kernel(Kv4PoolParams p) {
  grid_dependency_sync();
  __shared__ float part[16][kHeadDim];
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int w = threadIdx.x & 15, lane = threadIdx.x >> 4;
  float sum[8] = {};
  const bool complete = (int64_t)(j + 1) * p.B <= len;
  if (complete) {
    const int64_t t0 = (int64_t)j * p.B;
    for (int i = lane; i < p.B; i += 16) {
      const int64_t t = t0 + i;
      const int tok = (int)(t % kKv4Tile);
      const uint8_t* tile = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, t / kKv4Tile);
      const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(tile + kv4_word_off(tok, w, false)));
      const uint32_t par = __ldg(reinterpret_cast<const uint16_t*>(tile + kKv4Params + tok * 8 + (w >> 2) * 2));
      float x[8];
      kv4_decode(word, par, x);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += x[c];
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) part[lane][w * 8 + c] = sum[c];
  __syncthreads();
  if (threadIdx.x < kHeadDim) {
    float s = 0.f;
    for (int i = 0; i < 16; ++i) s += part[i][threadIdx.x];
    p.kmean[(((int64_t)b * p.heads + h) * p.blocks + j) * kHeadDim + threadIdx.x] = complete ? s / (float)p.B : 0.f;
  }
}

// ------------------------------------------------------------------ evict

struct Kv4EvictParams {
  const uint8_t* kv4;
  const float* acc;        // [batch][heads][tiles * 64]
  const int32_t* lengths;
  int64_t tiles, dst_tiles;
  int batch, heads, budget, recent;
  uint8_t* dst;
  float* dst_acc;          // [batch][heads][dst_tiles * 64]
  int32_t* kept;           // [batch][heads][budget], ascending, padded with -1
  int32_t* new_lengths;    // [batch]
};

constexpr int kKv4SelectThreads = 1024;

// Weights as integers of the same order; a NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t kv4_weight_key(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum of x over the block's threads, and the total.
__device__ __forceinline__ uint32_t kv4_block_scan(uint32_t x, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
    if (i < warp) before += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  return before + s - x;
}

// The tokens that stay, for one (head, sequence) a CTA: the last `recent`, and
// of the others the `budget - recent` of the largest weight, equal weights to
// the lower index. A radix selection finds the smallest kept weight in four
// passes of eight bits, then one pass writes the kept indexes in order.
__global__ void __launch_bounds__(kKv4SelectThreads) kv4_select_kernel(Kv4EvictParams p) {
  grid_dependency_sync();
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_prefix, s_need;
  const int h = blockIdx.x, b = blockIdx.y;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int tid = threadIdx.x;
  if (h == 0 && tid == 0) p.new_lengths[b] = min(len, p.budget);
  int32_t* kept = p.kept + ((int64_t)b * p.heads + h) * p.budget;
  if (len <= p.budget) {
    for (int i = tid; i < p.budget; i += kKv4SelectThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const float* acc = p.acc + ((int64_t)b * p.heads + h) * p.tiles * kKv4Tile;
  const int older = len - p.recent;        // > budget - recent >= 0
  const uint32_t want = p.budget - p.recent;
  uint32_t prefix = 0, need = want;        // of the keys that share `prefix`, `need` stay
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kKv4SelectThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < older; i += kKv4SelectThreads) {
        const uint32_t key = kv4_weight_key(acc[i]);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t left = need;
        int d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_prefix = prefix | (uint32_t)d << shift;
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // keys above `prefix` stay, and the first `need` equal to it
  uint32_t kept_before = 0, equal_before = 0;
  for (int i0 = 0; i0 < older; i0 += kKv4SelectThreads) {
    const int i = i0 + tid;
    const uint32_t key = i < older && want > 0 ? kv4_weight_key(acc[i]) : 0;
    const bool in = i < older && want > 0;
    const uint32_t eq = in && key == prefix;
    uint32_t n_eq, n_kept;
    const uint32_t my_eq = kv4_block_scan(eq, warp_sums, &n_eq);
    const uint32_t stay = in && (key > prefix || (eq && equal_before + my_eq < need));
    const uint32_t my = kv4_block_scan(stay, warp_sums, &n_kept);
    if (stay) kept[kept_before + my] = i;
    kept_before += n_kept;
    equal_before += n_eq;
  }
  for (int i = tid; i < p.recent; i += kKv4SelectThreads) kept[want + i] = older + i;
}

constexpr int kKv4MoveThreads = 256;

// Half a warp per kept token: its codes, parameters and weight.
__global__ void __launch_bounds__(kKv4MoveThreads) kv4_move_kernel(Kv4EvictParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 15;
  const int to = (int)(((int64_t)blockIdx.x * kKv4MoveThreads + threadIdx.x) >> 4);
  if (to >= p.budget) return;
  const int64_t pair = blockIdx.y;  // sequence * heads + head
  const int from = p.kept[pair * p.budget + to];
  if (from < 0) return;
  const uint8_t* src = p.kv4 + (pair * p.tiles + from / kKv4Tile) * kKv4TileBytes;
  uint8_t* dst = p.dst + (pair * p.dst_tiles + to / kKv4Tile) * kKv4TileBytes;
  const int ft = from % kKv4Tile, tt = to % kKv4Tile;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    *reinterpret_cast<uint32_t*>(dst + s * kKv4Half + kv4_word_off(tt, lane, s == 1)) =
        *reinterpret_cast<const uint32_t*>(src + s * kKv4Half + kv4_word_off(ft, lane, s == 1));
    if (lane < 2)
      *reinterpret_cast<uint32_t*>(dst + s * kKv4Half + kKv4Params + tt * 8 + lane * 4) =
          *reinterpret_cast<const uint32_t*>(src + s * kKv4Half + kKv4Params + ft * 8 + lane * 4);
  }
  if (lane == 0) p.dst_acc[pair * p.dst_tiles * kKv4Tile + to] = p.acc[pair * p.tiles * kKv4Tile + from];
}

}  // namespace moba
