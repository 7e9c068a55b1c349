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

// The eight channels of a code word as bf16. 128 + c has bf16's eight bits (a
// nibble under 0x4300), so has its difference from 128 + z, and times a scale of
// four it is a value that bf16 holds: all exact.
__device__ __forceinline__ uint4 kv4_decode(uint32_t word, uint32_t par) {
  const __nv_bfloat162 s = __float2bfloat162_rn(kv4_scale(par));
  const uint32_t zz = 0x43004300u | (par & 15u) * 0x10001u;
  const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162*>(&zz);
  uint32_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = (word >> (4 * j) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), z), s);
    x[j] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
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

// hi - lo, rounded to odd: a span that fp32 does not hold (hi has 8 bits, lo may lie far below) stays on its side of
// the ties between two scales, which are spans of few bits, and so does its 15th.
__device__ __forceinline__ float kv4_span(float lo, float hi) {
  const float d = __fsub_rz(hi, lo);
  return __uint_as_float(__float_as_uint(d) | (__fsub_ru(hi, lo) != d ? 1u : 0u));
}

// A nudge for floor(x / s + 1/2): x has 8 significant bits and s four, so a
// quotient between 1/2 and 16 that is not k + 1/2 is at least 2^-10 away from
// it, while x * fl(1/s) is off by less than 2^-18: with the nudge added, halves
// go up and nothing else moves.
constexpr float kKv4Nudge = 1.f / 4096;

// A group of 32 channels (bf16, four uint4) of a row: its four code words, and
// its parameter. One thread holds a whole group: no exchange, and scale and
// zero point are found once for 32 codes, which then take two fused
// multiply-adds each: floor(x / s + z + 1/2) / 16 saturated to [0, 1], and
// that by just under 16 onto 2^23, rounded down.
__device__ __forceinline__ uint4 kv4_quantise(const uint4 (&raw)[4], uint32_t* par) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
  float lo = 0.f, hi = 0.f;
  __nv_bfloat162 lo2 = __float2bfloat162_rn(0.f), hi2 = lo2;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    lo2 = __hmin2_nan(lo2, x);
    hi2 = __hmax2_nan(hi2, x);
  }
  lo = fminf(__low2float(lo2), __high2float(lo2));
  hi = fmaxf(__low2float(hi2), __high2float(hi2));
  // a NaN stays in lo2 and hi2; with magnitudes over 28800 it takes the way through fp32
  const float sum = (__low2float(lo2) + __high2float(lo2)) + (__low2float(hi2) + __high2float(hi2));
  const bool odd = !(sum == sum) || lo < -kKv4Top || hi > kKv4Top;
  auto clean = [](float x) { return x == x ? fminf(fmaxf(x, -kKv4Top), kKv4Top) : 0.f; };
  if (odd) {
    lo = hi = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = clean(__uint_as_float(w[i] << 16)), y = clean(__uint_as_float(w[i] & 0xFFFF0000u));
      lo = fminf(lo, fminf(x, y));
      hi = fmaxf(hi, fmaxf(x, y));
    }
  }
  const uint32_t code = kv4_scale_code(__fdiv_rn(kv4_span(lo, hi), 15.f));
  const float inv = __frcp_rn(kv4_scale(code << 7));
  const float z = fminf(__fadd_rd(fmaf(-lo, inv, 0.5f + kKv4Nudge), 8388608.f) - 8388608.f, 15.f);
  const float k = inv * 0.0625f, c0 = (z + (0.5f + kKv4Nudge)) * 0.0625f;
  *par = code << 7 | (uint32_t)z;
  auto one = [&](float x) {
    if (odd) x = clean(x);
    return __float_as_uint(__fmaf_rd(__saturatef(fmaf(x, k, c0)), 16.f - 1.f / 16384, 8388608.f));
  };
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t pair[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      pair[j] = __byte_perm(one(__uint_as_float(w[4 * i + j] << 16)), one(__uint_as_float(w[4 * i + j] & 0xFFFF0000u)),
                            0x5410);
    out[i] = (pair[0] + pair[1] * 16u) + (pair[2] * 256u + pair[3] * 4096u);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
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

// Four threads per row (token, kv head), a group of keys and the group of
// values each; a CTA takes 64 tokens of one head, whose places in the cache
// lie side by side, so that its stores fill whole lines. HBM-bound: 512 bytes
// read and 144 written a row. 128K tokens of 8 heads: 131 us, 5.3 TB/s (a copy
// reaches 6.5; three quarters of the issue slots are taken, by the rounding).
__global__ void __launch_bounds__(kKv4AppendThreads) kv4_append_kernel(Kv4AppendParams p) {
  grid_dependency_sync();
  const int g = threadIdx.x & 3, h = blockIdx.y;
  const int64_t t = (int64_t)blockIdx.x * (kKv4AppendThreads / 4) + (threadIdx.x >> 2);
  if (t >= p.total) return;
  const int64_t row = t * p.heads + h;
  uint4 rk[4], rv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rk[i] = __ldg(reinterpret_cast<const uint4*>(p.k + row * kHeadDim + g * 32) + i);
#pragma unroll
  for (int i = 0; i < 4; ++i) rv[i] = __ldg(reinterpret_cast<const uint4*>(p.v + row * kHeadDim + g * 32) + i);
  int b;
  int64_t at;
  if (p.cu) {
    b = kv4_sequence(p.cu, p.batch, t);
    if (b < 0) return;
    at = (int64_t)p.start[b] + (t - p.cu[b]);
  } else {
    const int64_t n = p.total / p.batch;
    b = (int)(t / n);
    at = (int64_t)p.start[b] + (t - b * n);
  }
  if (at < 0 || at >= p.tiles * kKv4Tile) {  // no room: skipped and reported
    record_status(MOBA_ERR_DEVICE_CHECK);
    return;
  }
  const int tok = (int)(at % kKv4Tile);
  uint8_t* tile = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, at / kKv4Tile);
  uint32_t par;
  *reinterpret_cast<uint4*>(tile + kv4_word_off(tok, 4 * g, false)) = kv4_quantise(rk, &par);
  *reinterpret_cast<uint16_t*>(tile + kKv4Params + tok * 8 + g * 2) = (uint16_t)par;
  *reinterpret_cast<uint4*>(tile + kKv4Half + kv4_word_off(tok, 4 * g, true)) = kv4_quantise(rv, &par);
  *reinterpret_cast<uint16_t*>(tile + kKv4Half + kKv4Params + tok * 8 + g * 2) = (uint16_t)par;
  if (p.acc && g == 0) p.acc[((int64_t)b * p.heads + h) * p.tiles * kKv4Tile + at] = 0.f;
}

// ------------------------------------------------------------------ load

struct Kv4LoadParams {
  const uint8_t* kv4;
  const int32_t *lengths, *first;  // first may be null (token 0)
  int64_t tiles, n;
  int batch, heads;
  __nv_bfloat16 *k, *v;  // [batch][n][heads][128]
};

constexpr int kKv4LoadThreads = 256, kKv4LoadRows = 4;

// A CTA per 64 tokens of a kv head, half a warp per row, 8 channels a lane,
// four rows of keys and values at a time: 144 bytes read, 512 written a row,
// HBM-bound. 128K tokens of 8 heads: 116 us, 5.9 TB/s.
__global__ void __launch_bounds__(kKv4LoadThreads) kv4_load_kernel(Kv4LoadParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 15, h = blockIdx.y, b = blockIdx.z;
  const int64_t i0 = (int64_t)blockIdx.x * (kKv4LoadThreads / 16 * kKv4LoadRows) + (threadIdx.x >> 4);
  const int64_t first = p.first ? p.first[b] : 0;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const uint8_t* src = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, 0);
  uint32_t word[kKv4LoadRows][2], par[kKv4LoadRows][2];
#pragma unroll
  for (int i = 0; i < kKv4LoadRows; ++i) {
    const int64_t at = first + i0 + i * (kKv4LoadThreads / 16);
    word[i][0] = word[i][1] = par[i][0] = par[i][1] = 0;
    if (i0 + i * (kKv4LoadThreads / 16) >= p.n || at < 0 || at >= len) continue;
    const int tok = (int)(at % kKv4Tile);
    const uint8_t* tile = src + at / kKv4Tile * kKv4TileBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint8_t* half = tile + s * kKv4Half;
      word[i][s] = __ldg(reinterpret_cast<const uint32_t*>(half + kv4_word_off(tok, lane, s == 1)));
      par[i][s] = __ldg(reinterpret_cast<const uint16_t*>(half + kKv4Params + tok * 8 + (lane >> 2) * 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kKv4LoadRows; ++i) {
    const int64_t at = i0 + i * (kKv4LoadThreads / 16);
    if (at >= p.n) continue;
    const int64_t row = ((int64_t)b * p.n + at) * p.heads + h;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      reinterpret_cast<uint4*>((s ? p.v : p.k) + row * kHeadDim)[lane] = kv4_decode(word[i][s], par[i][s]);
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

constexpr int kKv4SelectFew = 512, kKv4SelectMany = 1024;  // threads
constexpr int kKv4SelectItems = 16;  // neighbouring weights a thread takes at a time
constexpr int kKv4SelectBins = 2048, kKv4SelectCopies = 4;

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
  const uint32_t y = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
  *total = __reduce_add_sync(0xFFFFFFFFu, y);
  return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0) + s - x;
}

__device__ __forceinline__ void kv4_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of another CTA's shared memory, at the same place as `p` in ours.
__device__ __forceinline__ uint32_t kv4_remote_ld(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void kv4_remote_st(uint32_t* p, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// The tokens that stay, a cluster of CTAs for one (head, sequence), a
// contiguous part of its weights each: the last `recent`, and of the others
// the `budget - recent` of the largest weight, equal weights to the lower
// index. A radix selection finds the smallest kept weight in three passes of
// 11, 11 and 10 bits (counts per CTA, summed and searched by the first one
// through distributed shared memory); a last pass writes the kept indexes,
// each thread's neighbouring weights at its place in the order. Bound by its
// chain of passes, each a round of counts, two cluster barriers and a scan: 128K
// weights of 8 heads 24 us; 32 sequences of 4608 and 8 heads 18 us with 512
// threads, two CTAs an SM, 21 with 1024.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv4_select_kernel(Kv4EvictParams p) {
  grid_dependency_sync();
  // neighbouring lanes count in copies of their own: weights crowd into few bins
  __shared__ uint32_t hist[kKv4SelectCopies][kKv4SelectBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_found[2], s_count[2];  // prefix and need; this part's keys above and at the limit
  uint32_t rank, csize;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int pair = blockIdx.x / csize;  // sequence * heads + head
  const int h = pair % p.heads, b = pair / p.heads, tid = threadIdx.x;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  if (h == 0 && rank == 0 && tid == 0) p.new_lengths[b] = min(len, p.budget);
  int32_t* kept = p.kept + (int64_t)pair * p.budget;
  if (len <= p.budget) {  // the whole cluster leaves
    for (int i = rank * THREADS + tid; i < p.budget; i += csize * THREADS) kept[i] = i < len ? i : -1;
    return;
  }
  const float* acc = p.acc + (int64_t)pair * p.tiles * kKv4Tile;
  const int older = len - p.recent;        // > budget - recent >= 0
  const uint32_t want = p.budget - p.recent;
  for (int i = rank * THREADS + tid; i < p.recent; i += csize * THREADS) kept[want + i] = older + i;
  if (want == 0) return;
  const int part = (int)(((int64_t)older + csize * kKv4SelectItems - 1) / (csize * kKv4SelectItems)) * kKv4SelectItems;
  const int i0 = (int)min((int64_t)rank * part, (int64_t)older), i1 = (int)min((int64_t)i0 + part, (int64_t)older);
  // a thread's neighbouring weights of a sweep over the part; those outside it come as the key 0 and do not count
  auto keys = [&](int at, uint32_t (&k)[kKv4SelectItems]) {
    // acc rows begin at multiples of 64 floats and parts at multiples of 16, but acc itself is 4-byte aligned
    if (at + kKv4SelectItems <= i1 && (reinterpret_cast<uintptr_t>(acc) & 15) == 0) {
#pragma unroll
      for (int x = 0; x < kKv4SelectItems; x += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(acc + at + x));
        k[x] = kv4_weight_key(v.x);
        k[x + 1] = kv4_weight_key(v.y);
        k[x + 2] = kv4_weight_key(v.z);
        k[x + 3] = kv4_weight_key(v.w);
      }
    } else {
#pragma unroll
      for (int x = 0; x < kKv4SelectItems; ++x) k[x] = at + x < i1 ? kv4_weight_key(__ldg(acc + at + x)) : 0;
    }
  };
  constexpr int kSweep = THREADS * kKv4SelectItems;
  // a part that is one sweep stays in registers, a longer one is read again in each pass
  const bool once = i1 - i0 <= kSweep;
  uint32_t k[kKv4SelectItems];
  if (once) keys(i0 + tid * kKv4SelectItems, k);
  uint32_t prefix = 0, need = want;        // of the keys that share `prefix`, `need` stay
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kKv4SelectCopies * kKv4SelectBins; i += THREADS) (&hist[0][0])[i] = 0;
    __syncthreads();
    for (int at = i0 + tid * kKv4SelectItems; at < i1; at += kSweep) {
      if (!once) keys(at, k);
#pragma unroll
      for (int x = 0; x < kKv4SelectItems; ++x)
        if (at + x < i1 && (pass == 0 || (k[x] >> above) == (prefix >> above)))
          atomicAdd(&hist[tid % kKv4SelectCopies][(k[x] >> shift) & mask], 1u);
    }
    __syncthreads();
    for (int i = tid; i < kKv4SelectBins; i += THREADS)
      hist[0][i] += (hist[1][i] + hist[2][i]) + hist[3][i];
    kv4_cluster_sync();
    if (rank == 0) {
      // neighbouring bins for each thread, from the highest down: the bin in which the need is met
      constexpr int BINS = kKv4SelectBins / THREADS;
      uint32_t c[BINS], mine = 0, total;
#pragma unroll
      for (int x = 0; x < BINS; ++x) {
        const int bin = kKv4SelectBins - 1 - (BINS * tid + x);
        uint32_t y[8];  // all under way at once
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) y[r] = r < csize ? kv4_remote_ld(&hist[0][bin], r) : 0;
        c[x] = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        mine += c[x];
      }
      uint32_t before = kv4_block_scan(mine, warp_sums, &total);
#pragma unroll
      for (int x = 0; x < BINS; ++x) {
        if (before < need && before + c[x] >= need) {
          const uint32_t found = prefix | (uint32_t)(kKv4SelectBins - 1 - (BINS * tid + x)) << shift;
          for (uint32_t r = 0; r < csize; ++r) {
            kv4_remote_st(&s_found[0], r, found);
            kv4_remote_st(&s_found[1], r, need - before);
          }
        }
        before += c[x];
      }
    }
    kv4_cluster_sync();
    prefix = s_found[0];
    need = s_found[1];
  }
  // keys above `prefix` stay, and the first `need` equal to it: their numbers before each thread's
  auto count = [&](int at, uint32_t& above, uint32_t& equal) {
    above = equal = 0;
#pragma unroll
    for (int x = 0; x < kKv4SelectItems; ++x) {
      above += at + x < i1 && k[x] > prefix;
      equal += at + x < i1 && k[x] == prefix;
    }
  };
  auto place = [&](int at, uint32_t a, uint32_t e) {
#pragma unroll
    for (int x = 0; x < kKv4SelectItems; ++x) {
      if (at + x >= i1) continue;
      if (k[x] > prefix) kept[a++ + min(e, need)] = at + x;
      else if (k[x] == prefix) {
        if (e < need) kept[a + e] = at + x;
        ++e;
      }
    }
  };
  uint32_t above = 0, equal = 0, n_above, n_equal, a, e;
  if (once) {
    count(i0 + tid * kKv4SelectItems, above, equal);
  } else {
    for (int at = i0 + tid * kKv4SelectItems; at < i1; at += kSweep) {
      uint32_t x, y;
      keys(at, k);
      count(at, x, y);
      above += x;
      equal += y;
    }
  }
  a = kv4_block_scan(above, warp_sums, &n_above);
  e = kv4_block_scan(equal, warp_sums, &n_equal);
  if (tid == 0) {
    s_count[0] = n_above;
    s_count[1] = n_equal;
  }
  kv4_cluster_sync();
  uint32_t above_before = 0, equal_before = 0;
  for (uint32_t r = 0; r < rank; ++r) {
    above_before += kv4_remote_ld(&s_count[0], r);
    equal_before += kv4_remote_ld(&s_count[1], r);
  }
  kv4_cluster_sync();  // no CTA leaves while another may still read its counts
  if (once) {
    place(i0 + tid * kKv4SelectItems, above_before + a, equal_before + e);
    return;
  }
  for (int s0 = i0; s0 < i1; s0 += kSweep) {
    const int at = s0 + tid * kKv4SelectItems;
    keys(at, k);
    count(at, above, equal);
    a = above_before + kv4_block_scan(above, warp_sums, &n_above);
    e = equal_before + kv4_block_scan(equal, warp_sums, &n_equal);
    place(at, a, e);
    above_before += n_above;
    equal_before += n_equal;
  }
}

constexpr int kKv4MoveThreads = 256;

// Eight lanes per kept token, four tokens at a time: 16 bytes of codes each, the
// parameters and the weight. 148 bytes read and as many written a token; bound by
// its scattered pieces of 64 and 8 bytes (32 sequences of up to 4096 kept tokens,
// 8 heads: 38 us, 52 with words of 4 bytes; 8192 of 128K tokens, 8 heads: 9).
// Done by the selecting CTAs instead, the first took 195 us a call against 177:
// too few loads under way.
constexpr int kKv4MoveTokens = 4;
__global__ void __launch_bounds__(kKv4MoveThreads) kv4_move_kernel(Kv4EvictParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 7, vals = lane >> 2, c = lane & 3;  // four lanes for the keys, four for the values
  const int to0 = (int)(blockIdx.x * (kKv4MoveThreads / 8 * kKv4MoveTokens)) + (threadIdx.x >> 3);
  const int64_t pair = blockIdx.y;  // sequence * heads + head
  const int32_t* kept = p.kept + pair * p.budget;
  const uint8_t* src = p.kv4 + pair * p.tiles * kKv4TileBytes + vals * kKv4Half;
  uint8_t* dst = p.dst + pair * p.dst_tiles * kKv4TileBytes + vals * kKv4Half;
  int from[kKv4MoveTokens];
  uint4 codes[kKv4MoveTokens];
  uint2 par[kKv4MoveTokens];
  float weight[kKv4MoveTokens];
#pragma unroll
  for (int i = 0; i < kKv4MoveTokens; ++i) {
    const int to = to0 + i * (kKv4MoveThreads / 8);
    from[i] = to < p.budget ? kept[to] : -1;
  }
#pragma unroll
  for (int i = 0; i < kKv4MoveTokens; ++i) {
    if (from[i] < 0) continue;
    const uint8_t* t = src + (int64_t)(from[i] / kKv4Tile) * kKv4TileBytes;
    const int ft = from[i] % kKv4Tile;
    codes[i] = __ldg(reinterpret_cast<const uint4*>(t + kv4_word_off(ft, 4 * c, vals)));
    if (c == 0) par[i] = __ldg(reinterpret_cast<const uint2*>(t + kKv4Params + ft * 8));
    if (lane == 1) weight[i] = __ldg(p.acc + pair * p.tiles * kKv4Tile + from[i]);
  }
#pragma unroll
  for (int i = 0; i < kKv4MoveTokens; ++i) {
    if (from[i] < 0) continue;
    const int to = to0 + i * (kKv4MoveThreads / 8);
    uint8_t* t = dst + (int64_t)(to / kKv4Tile) * kKv4TileBytes;
    const int tt = to % kKv4Tile;
    *reinterpret_cast<uint4*>(t + kv4_word_off(tt, 4 * c, vals)) = codes[i];
    if (c == 0) *reinterpret_cast<uint2*>(t + kKv4Params + tt * 8) = par[i];
    if (lane == 1) p.dst_acc[pair * p.dst_tiles * kKv4Tile + to] = weight[i];
  }
}

}  // namespace moba
