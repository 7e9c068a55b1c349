// Attention of a few query tokens over the 4-bit key/value cache (kv4.cuh):
// gate, attention and the accumulated weights of the cached tokens.
//
// Query token i of the n of sequence b stands at position
// lengths[b] - n + i and attends the cached tokens up to itself: all of them,
// or, with block means, those of its own block and of the topk - 1 past
// blocks of the highest score q . mean (ties to the lower block index).
#pragma once

#include "kv4.cuh"

namespace moba {

struct Kv4AttnParams {
  const __nv_bfloat16* q;  // [total][Hq][128]
  const uint8_t* kv4;
  const int32_t *lengths, *cu;  // cu null: total / batch queries each
  const float* kmean;           // [batch][Hkv][blocks][128], or null: every key
  int64_t total, tiles;
  int batch, Hq, Hkv, G;
  int B, topk, blocks;          // with kmean; blocks = capacity / B
  float scale_log2;             // log2(e) / sqrt(128)
  int32_t* sel;                 // [total][Hq][topk] scratch: ascending, padded with -1
  float* acc;                   // [batch][Hkv][tiles * 64], or null
  __nv_bfloat16* out;           // [total][Hq][128]
  float* lse;                   // [Hq][total]
};

// Sequence and position of packed query token t (b = -1: behind the last).
__device__ __forceinline__ int kv4_query(const Kv4AttnParams& p, int64_t t, int* pos) {
  int b;
  int64_t i, n;
  if (p.cu) {
    b = kv4_sequence(p.cu, p.batch, t);
    if (b < 0) return -1;
    i = t - p.cu[b];
    n = p.cu[b + 1] - p.cu[b];
  } else {
    n = p.total / p.batch;
    b = (int)(t / n);
    i = t - b * n;
  }
  *pos = (int)(kv4_length(p.lengths, b, p.tiles * kKv4Tile) - n + i);
  return b;
}

constexpr int kKv4GateThreads = 128;

// One CTA per row (token, q head): scores of its past blocks in fp64 (the
// products of a bf16 and an fp32 number are exact there, so that near ties
// fall as in exact arithmetic), then topk - 1 rounds of the best block after
// the previous one.
__global__ void __launch_bounds__(kKv4GateThreads) kv4_gate_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  extern __shared__ double scores[];  // [blocks], then flags
  __shared__ double best_s[kKv4GateThreads];
  __shared__ int best_j[kKv4GateThreads];
  const int64_t row = blockIdx.x;
  const int64_t t = row / p.Hq;
  const int hq = (int)(row - t * p.Hq), tid = threadIdx.x;
  int32_t* sel = p.sel + row * p.topk;
  int pos = -1;
  const int b = kv4_query(p, t, &pos);
  if (b < 0 || pos < 0) {
    for (int i = tid; i < p.topk; i += kKv4GateThreads) sel[i] = -1;
    return;
  }
  const int own = pos / p.B;
  const float* means = p.kmean + ((int64_t)b * p.Hkv + hq / p.G) * p.blocks * kHeadDim;
  const __nv_bfloat16* q = p.q + row * kHeadDim;
  uint8_t* picked = reinterpret_cast<uint8_t*>(scores + p.blocks);
  for (int j = tid; j < own; j += kKv4GateThreads) {
    double s = 0.0;
    for (int c = 0; c < kHeadDim; ++c)
      s = fma((double)__bfloat162float(q[c]), (double)means[(int64_t)j * kHeadDim + c], s);
    scores[j] = s;
    picked[j] = 0;
  }
  __syncthreads();
  const int picks = min(p.topk - 1, own);
  for (int r = 0; r < picks; ++r) {
    double s = 0.0;
    int bj = -1;
    for (int j = tid; j < own; j += kKv4GateThreads)
      if (!picked[j] && (bj < 0 || scores[j] > s)) s = scores[j], bj = j;
    best_s[tid] = s;
    best_j[tid] = bj;
    __syncthreads();
    for (int d = kKv4GateThreads / 2; d > 0; d >>= 1) {
      if (tid < d) {
        const int o = best_j[tid + d], m = best_j[tid];
        if (o >= 0 && (m < 0 || best_s[tid + d] > best_s[tid] || (best_s[tid + d] == best_s[tid] && o < m))) {
          best_s[tid] = best_s[tid + d];
          best_j[tid] = o;
        }
      }
      __syncthreads();
    }
    if (tid == 0 && best_j[0] >= 0) picked[best_j[0]] = 1;
    __syncthreads();
  }
  if (tid == 0) {
    int n = 0;
    for (int j = 0; j < own && n < p.topk - 1; ++j)
      if (picked[j]) sel[n++] = j;
    sel[n++] = own;
    while (n < p.topk) sel[n++] = -1;
  }
}

constexpr int kKv4AttnThreads = 128;

// Scaled log2 score of one key for half a warp: 8 channels a lane.
__device__ __forceinline__ float kv4_score(const float (&q)[8], const uint8_t* tile, int tok, int lane) {
  const uint32_t word = *reinterpret_cast<const uint32_t*>(tile + kv4_word_off(tok, lane, false));
  const uint32_t par = *reinterpret_cast<const uint16_t*>(tile + kKv4Params + tok * 8 + (lane >> 2) * 2);
  float x[8], s = 0.f;
  kv4_decode(word, par, x);
#pragma unroll
  for (int c = 0; c < 8; ++c) s = fmaf(q[c], x[c], s);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

__device__ __forceinline__ void kv4_load_q(const Kv4AttnParams& p, int64_t row, int lane, float (&q)[8]) {
  const uint4 raw = *(reinterpret_cast<const uint4*>(p.q + row * kHeadDim) + lane);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q[2 * j] = __uint_as_float(w[j] << 16);
    q[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// One CTA per row; each half-warp takes every eighth key with a running
// maximum and sum, and the eight are joined at the end.
__global__ void __launch_bounds__(kKv4AttnThreads) kv4_attn_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  __shared__ float s_m[8], s_l[8], s_o[8][kHeadDim];
  const int64_t row = blockIdx.x;
  const int64_t t = row / p.Hq;
  const int hq = (int)(row - t * p.Hq);
  int pos = -1;
  const int b = kv4_query(p, t, &pos);
  if (b < 0) return;
  const int lane = threadIdx.x & 15, hw = threadIdx.x >> 4;
  float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
  kv4_load_q(p, row, lane, q);
  const uint8_t* base = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, b, hq / p.G, 0);
  const int32_t* sel = p.sel + row * p.topk;
  const int parts = p.kmean ? p.topk : 1;
  for (int i = 0; i < parts; ++i) {
    int u0 = 0, u1 = pos + 1;
    if (p.kmean) {
      if (sel[i] < 0) break;
      u0 = sel[i] * p.B;
      u1 = min(u0 + p.B, pos + 1);
    }
    for (int u = u0 + (hw & ~1); u < u1; u += 8) {  // both halves of a warp stay together
      const int key = u + (hw & 1);
      const bool in = key < u1;
      const uint8_t* tile = base + (int64_t)((in ? key : u) / kKv4Tile) * kKv4TileBytes;
      const int tok = (in ? key : u) % kKv4Tile;
      const float s = kv4_score(q, tile, tok, lane) * p.scale_log2;
      if (!in) continue;
      const float m2 = fmaxf(m, s);
      const float a = exp2f(m - m2), e = exp2f(s - m2);
      const uint8_t* half = tile + kKv4Half;
      float x[8];
      kv4_decode(*reinterpret_cast<const uint32_t*>(half + kv4_word_off(tok, lane, true)),
                 *reinterpret_cast<const uint16_t*>(half + kKv4Params + tok * 8 + (lane >> 2) * 2), x);
      l = l * a + e;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = o[c] * a + e * x[c];
      m = m2;
    }
  }
  if (lane == 0) s_m[hw] = m, s_l[hw] = l;
#pragma unroll
  for (int c = 0; c < 8; ++c) s_o[hw][lane * 8 + c] = o[c];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f, oo = 0.f;
  for (int i = 0; i < 8; ++i) mm = fmaxf(mm, s_m[i]);
  if (mm > -INFINITY)
    for (int i = 0; i < 8; ++i) {
      const float a = exp2f(s_m[i] - mm);
      ll += s_l[i] * a;
      oo += s_o[i][threadIdx.x] * a;
    }
  p.out[row * kHeadDim + threadIdx.x] = __float2bfloat16(ll > 0.f ? oo / ll : 0.f);
  if (threadIdx.x == 0)
    p.lse[(int64_t)hq * p.total + t] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
}

// Accumulated weights: half a warp per cached token of a kv head, over the
// rows of that head in order.
__global__ void __launch_bounds__(kKv4AttnThreads) kv4_weight_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  const int b = blockIdx.z, h = blockIdx.y;
  const int lane = threadIdx.x & 15;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int key = blockIdx.x * (kKv4AttnThreads / 16) + (threadIdx.x >> 4);
  const bool in = key < len;
  if (__all_sync(0xFFFFFFFFu, !in)) return;
  const int64_t t0 = p.cu ? p.cu[b] : b * (p.total / p.batch), t1 = p.cu ? p.cu[b + 1] : t0 + p.total / p.batch;
  const uint8_t* tile = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, b, h, (in ? key : 0) / kKv4Tile);
  float sum = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const int pos = (int)(len - (t1 - t));
    for (int g = 0; g < p.G; ++g) {
      const int hq = h * p.G + g;
      const int64_t row = t * p.Hq + hq;
      float q[8];
      kv4_load_q(p, row, lane, q);
      const float s = kv4_score(q, tile, (in ? key : 0) % kKv4Tile, lane) * p.scale_log2;
      bool seen = in && key <= pos;
      if (p.kmean && seen) {
        seen = false;
        for (int i = 0; i < p.topk; ++i) seen |= p.sel[row * p.topk + i] == key / p.B;
      }
      if (seen) sum += exp2f(s - p.lse[(int64_t)hq * p.total + t] * 1.4426950408889634f);
    }
  }
  if (in && lane == 0) p.acc[((int64_t)b * p.Hkv + h) * p.tiles * kKv4Tile + key] += sum;
}

}  // namespace moba
