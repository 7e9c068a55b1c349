// Attention of many query rows over the 4-bit key/value cache, and the weights
// that they give the cached tokens, on the 5th-generation tensor cores.
//
// Units are 256 rows of one sequence and kv head (two tiles A and B of 128,
// tile B absent up to 128 rows); their 128-key steps are dealt out in even
// ranges, one to each CTA, and joined as those of kv4_attn.cuh. One CTA per SM:
//   warps 0-3, 4-7  softmax of tile A, B (thread = row = TMEM lane)
//   warps 8-11      widen the codes of the next step's keys and values to fp16
//                   in shared memory (128-byte swizzle), codes of the step
//                   after on their way in registers
//   warp 12         TMEM owner; issues S = Q K^T
//   warp 13         issues O += P V
//   warp 14         fetches the units' query tiles
// With a gate (MASKED), a unit goes over all keys, and a step's weights are those
// of the rows that chose its block: the 32 rows of a warp are one word of the
// gate's.
// Products, roles and barriers are those of the bf16 attention kernel
// (attn.cuh): one S buffer for both tiles, P in TMEM columns of its own, two
// issuers. What differs: operands are fp16 (queries times a power of two, a
// 64th of keys and values: all exact), a row has a scale of its own, and
// widening takes the place of TMA loads: 11 instructions for 8 codes, about a
// fifth of the issue slots that the two tiles' softmaxes leave. 512 tokens of 32 /
// 8 heads against 32K: 279 us, 970 TFLOP/s, the tensor pipe busy 54 % of the
// time; what bounds it is the chain score - weights - product of two tiles.
#pragma once

#include <type_traits>

#include "kv4_attn.cuh"

namespace moba {

constexpr int kKv4ChunkRows = 256, kKv4ChunkThreads = 512;
constexpr uint32_t kKv4TileOp = kTile * kHeadDim * 2;  // 32 KB: 128 rows of fp16
constexpr uint32_t kKv4TileOpHalf = kKv4TileOp / 2;    // 64 channels of them
constexpr int kKv4ChunkStages = 2;

// Instruction descriptor, kind::f16: fp16 A and B, fp32 D, dense.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ------------------------------------------------------------------ query tiles

constexpr int kKv4PrepThreads = 256;

// The units' rows as fp16 in the layout of a shared-memory operand (per tile
// of 128 rows: two halves of 64 channels, 128 bytes a row, 16-byte chunks
// swizzled by the row), and each row's scale; rows behind the unit's are zero.
// Half a warp per row.
__global__ void __launch_bounds__(kKv4PrepThreads) kv4_prep_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  __shared__ Kv4Unit s_unit;
  const int ui = blockIdx.x, lane = threadIdx.x & 15;
  if (threadIdx.x == 0) s_unit = kv4_unit_of(p, p.cu, p.lengths, ui / p.Hkv, ui % p.Hkv);
  __syncthreads();
  const Kv4Unit u = s_unit;
  if (u.rows == 0) return;
  const int row = blockIdx.y * (kKv4PrepThreads / 16) + (threadIdx.x >> 4);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (row < u.rows) {
    const int rr = u.row0 + row;
    raw = __ldg(reinterpret_cast<const uint4*>(p.q + ((int64_t)(u.t0 + rr / p.G) * p.Hq + u.h * p.G + rr % p.G) *
                                                         kHeadDim) + lane);
  }
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  float f1, f2;
  const float scale = kv4_query_scale(top, p.scale_log2, f1, f2);
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = pack_half2(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2);
  const int r = row & 127;
  uint8_t* tile = p.qtiles + ((int64_t)ui * 2 + (row >> 7)) * kKv4TileOp;
  *reinterpret_cast<uint4*>(tile + (lane >> 3) * kKv4TileOpHalf + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) =
      make_uint4(y[0], y[1], y[2], y[3]);
  if (lane == 0) p.qscale[(int64_t)ui * kKv4ChunkRows + row] = scale;
}

// A kernel's buffers of query tiles, for the warp that fills them (one of its lanes starts the copies).
struct Kv4QueryPort {
  uint64_t *full, *empty_;
  uint8_t* dst;
  const uint8_t* src;  // the next tile
  volatile int* abort_flag;
  bool starts;
  __device__ __forceinline__ bool empty(int x, uint32_t parity) { return mbar_wait(&empty_[x], parity, abort_flag); }
  __device__ __forceinline__ void start(int x) {
    if (!starts) return;
    mbar_arrive_expect_tx(&full[x], kKv4TileOp);
    bulk_load(dst + x * kKv4TileOp, src, kKv4TileOp, &full[x]);
  }
  __device__ __forceinline__ void landed(int x, uint32_t parity) {
    volatile int keep_waiting = 0;
    if (starts) mbar_wait(&full[x], parity, &keep_waiting);
  }
};

// ------------------------------------------------------------------ widening

// Codes of up to four (key, 32 channels) pieces a thread: 128 keys of one
// half of a step for 128 threads. Thread: key 32 (warp) + 8 i + lane % 8, group
// lane / 8, so that a warp reads 512 bytes in a row and its 16-byte stores fall
// on all banks. Keys from `end` on come as zero.
struct Kv4Pieces {
  uint4 w[4];
  uint32_t par[4];
};
template <int N = 4>
__device__ __forceinline__ void kv4_fetch(Kv4Pieces& x, const uint8_t* half0, int key0, int end, bool vals, int warp,
                                          int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int key = key0 + 8 * N * warp + 8 * i + (lane & 7), g = lane >> 3;
    x.w[i] = make_uint4(0, 0, 0, 0);
    x.par[i] = 0;
    if (key < end) {
      const int tok = key % kKv4Tile;
      const uint8_t* half = half0 + (int64_t)(key / kKv4Tile) * kKv4TileBytes;
      x.w[i] = __ldg(reinterpret_cast<const uint4*>(half + kv4_word_off(tok, 4 * g, vals)));
      x.par[i] = __ldg(reinterpret_cast<const uint16_t*>(half + kKv4Params + tok * 8 + g * 2));
    }
  }
}
template <int N = 4>
__device__ __forceinline__ void kv4_widen(const Kv4Pieces& x, uint8_t* tile, int warp, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = 8 * N * warp + 8 * i + (lane & 7), g = lane >> 3;
    const Kv4Par f = kv4_par(__byte_perm(x.par[i], 0, 0x1010));
    uint8_t* to = tile + (g >> 1) * kKv4TileOpHalf + row * 128;
    const uint32_t w[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t y[4];
      kv4_pairs(w[c], f, y);
      *reinterpret_cast<uint4*>(to + ((((g & 1) * 4 + c) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

// ------------------------------------------------------------------ attention

struct Kv4ChunkShared {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKv4ChunkStages], k_empty[kKv4ChunkStages], v_full[kKv4ChunkStages], v_empty[kKv4ChunkStages];
  uint64_t s_full[2], s_free, p_full[2], pv_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kKv4ChunkSmemBytes = (2 + 2 * kKv4ChunkStages) * kKv4TileOp + 1024 + 512;

// TMEM columns, as in attn.cuh
constexpr uint32_t kKv4TmemS = 0, kKv4TmemP = 128, kKv4TmemO = 256;

template <bool MASKED>
__global__ void __launch_bounds__(kKv4ChunkThreads, 1) kv4_chunk_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                             // tile A, tile B
  uint8_t* sK = sQ + 2 * kKv4TileOp;
  uint8_t* sV = sK + kKv4ChunkStages * kKv4TileOp;
  Kv4ChunkShared* sh = reinterpret_cast<Kv4ChunkShared*>(sV + kKv4ChunkStages * kKv4TileOp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  const Kv4Range range = kv4_plan<kKv4ChunkThreads, 1>(p, reinterpret_cast<int32_t*>(sQ), 2 * kKv4TileOp / 4);
  if (!range.any) return;
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh->q_full[x], 1);
      mbar_init(&sh->q_empty[x], 1);
      mbar_init(&sh->s_full[x], 1);
      mbar_init(&sh->p_full[x], 128);
      mbar_init(&sh->pv_done[x], 1);
    }
    mbar_init(&sh->s_free, 4);  // one lane of each warp of the reading warpgroup
    for (int i = 0; i < kKv4ChunkStages; ++i) {
      mbar_init(&sh->k_full[i], 128);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_full[i], 128);
      mbar_init(&sh->v_empty[i], 1);
    }
    mbar_init(&sh->drain, 2);  // one commit from each issuer
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  // the plan's copy lies where the query tiles will
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort_flag;

  // the softmax warpgroups take 184 registers a thread, widening 88, the rest 56: 2 * 184 + 88 + 56 = 4 * 128
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;\n" ::: "memory");
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n" ::: "memory");
  }

  // Every role walks the units of the CTA's range: unit ui, steps [s0, s1).
  if (warp < 8) {
    // -------------------------------------------- softmax + epilogue of tile X
    const int X = warp >> 2;
    const int row = threadIdx.x & 255;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + kKv4TmemS + lane_off;
    const uint32_t tP = tmem + kKv4TmemP + X * 64 + lane_off;
    const uint32_t tO = tmem + kKv4TmemO + X * 128 + lane_off;
    uint32_t sx = 0;  // steps done by tile X
    int done = 0;
    for (int ui = range.unit, s0 = range.off; done < range.n; ++ui, s0 = 0) {
      const Kv4Unit u = range.at(ui);
      const int steps = kv4_items(p, u), s1 = min(steps, s0 + range.n - done);
      if (s1 <= s0) continue;
      done += s1 - s0;
      if (X == 1 && u.rows <= kTile) continue;
      // A row's scale is applied with the reference, in one step: score minus reference, exact but for the reference's
      // own coarseness, so that the largest is 12 above it, or by roundings upwards as little as -4 where fp32 numbers
      // are 8 apart. Rows of large queries (some 64 and more) may have scores beyond that, of 2^27: theirs have the
      // scale applied before, and so lie on one grid with the reference, which is 0 to 12 below the largest. (The loop is
      // there twice for it: a branch within, on the row or on its reference, took 4 to 9 % of the kernel's time.)
      const float scale = __ldcg(p.qscale + (int64_t)ui * kKv4ChunkRows + row);
      const bool large = scale >= 0.03125f;
      const float before = large ? scale : 1.f, qs = large ? 1.f : scale;
      const int pos = row < u.rows ? u.pos0 + (u.row0 + row) / p.G : -1;
      const int first_pos = u.pos0 + (u.row0 + X * kTile) / p.G;
      float ref = kKv4Low, l = 0.f;
      // with a gate: the warp's 32 rows that chose the step's block (rows behind the unit's, and rows before token 0,
      // which no gate has looked at, have no keys anyway)
      uint32_t on = ~0u;
      int block = -1;
      const int row32 = u.row0 + (row & ~31);
      auto run = [&](auto is_large) -> bool {
        constexpr bool LARGE = decltype(is_large)::value;
        for (int s = s0; s < s1; ++s, ++sx) {
          if constexpr (MASKED) {
            if (s * kTile / p.pick_B != block) {
              block = s * kTile / p.pick_B;
              on = (row & ~31) < u.rows ? kv4_picks(p, u.b, u.h, u.t0, row32, block) : 0;
            }
          }
          if (!mbar_wait(&sh->s_full[X], sx & 1, abort_flag)) return false;
          __syncwarp();
          tc_fence_after();
          uint32_t r[128];
          {
            uint32_t (&r0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[0]);
            uint32_t (&r1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[32]);
            uint32_t (&r2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[64]);
            uint32_t (&r3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[96]);
            tmem_ld32(tS, r0);
            tmem_ld32(tS + 32, r1);
            tmem_ld32(tS + 64, r2);
            tmem_ld32(tS + 96, r3);
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->s_free);
          if constexpr (LARGE) {
#pragma unroll
            for (int e = 0; e < 128; ++e) r[e] = __float_as_uint(__fmul_rn(__uint_as_float(r[e]), before));
          }
          if ((s + 1) * kTile - 1 > first_pos || (MASKED && on != ~0u)) {
            const int lim = !MASKED || on >> lane & 1u ? pos - s * kTile : -1;  // keys e > lim are masked
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e > lim) r[e] = __float_as_uint(-INFINITY);
          }
          float mx8[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float m = fmax3(__uint_as_float(r[c]), __uint_as_float(r[c + 8]), __uint_as_float(r[c + 16]));
#pragma unroll
            for (int e = 24; e < 120; e += 16) m = fmax3(m, __uint_as_float(r[e + c]), __uint_as_float(r[e + 8 + c]));
            mx8[c] = fmaxf(m, __uint_as_float(r[120 + c]));
          }
          const float top = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
          const float mx = __fmul_ru(qs, top);
          // the reference moves as in kv4_attn.cuh: weights stay under 2^15
          const bool move = mx > __fadd_rd(ref, 15.f);
          float factor = 1.f;
          if (move) {
            const float to = __fadd_ru(mx, -12.f);
            factor = ex2_approx(ref - to);
            ref = to;
          }
          uint32_t pk[64];
          {
            const uint64_t c2 = f2_pack(qs, qs), nm2 = f2_pack(-ref, -ref);
            uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int e = 0; e < 128; e += 2) {
              const uint64_t x2 = f2_fma((uint64_t)r[e] | ((uint64_t)r[e + 1] << 32), c2, nm2);
              const float a = ex2_approx(f2_lo(x2)), b = ex2_approx(f2_hi(x2));
              sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(a, b));
              pk[e >> 1] = pack_half2(a, b);
            }
            const uint64_t s01 = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
            l = l * factor + (f2_lo(s01) + f2_hi(s01));
          }
          if (s > s0) {
            if (!mbar_wait(&sh->pv_done[X], (sx - 1) & 1, abort_flag)) return false;
            __syncwarp();
            tc_fence_after();
          }
          // warp-collective: the branch is the warp's, the other rows multiply by 1
          if (s > s0 && __any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
              tmem_st32(tO + c * 32, o);
            }
          }
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_st16(tP + ch * 16, pk + ch * 16);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh->p_full[X]);
        }
        return true;
      };
      if (!(__any_sync(0xffffffffu, large) ? run(std::true_type()) : run(std::false_type()))) goto done;
      // epilogue: the row's result, or its part of it
      if (!mbar_wait(&sh->pv_done[X], (sx - 1) & 1, abort_flag)) goto done;
      __syncwarp();
      tc_fence_after();
      const bool whole = s0 == 0 && s1 == steps, write = row < u.rows;
      const int rr = u.row0 + row;
      const int64_t t = u.t0 + rr / p.G;
      const int hq = u.h * p.G + rr % p.G;
      const float inv = l != 0.f ? 64.f / l : 0.f;  // a NaN stays one
      float* part = p.part + (int64_t)(2 * cta + (s0 == 0 ? 1 : 0)) * (kKv4ChunkRows * 130);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait();
        if (write && whole) {
          uint4* out = reinterpret_cast<uint4*>(p.out + (t * p.Hq + hq) * kHeadDim + c * 32);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            out[e >> 3] = make_uint4(pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                                     pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                                     pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                                     pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
        } else if (write) {
          uint4* to = reinterpret_cast<uint4*>(part + row * kHeadDim + c * 32);
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[e >> 2] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (write && whole) {
        p.lse[(int64_t)hq * p.total + t] = l != 0.f ? (ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else if (write) {
        *reinterpret_cast<float2*>(part + kKv4ChunkRows * kHeadDim + 2 * row) = make_float2(ref, l);
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ------------------------------------------------ widening
    const int w = warp - 8;
    Kv4Pieces k, v;
    // the cursor stands one step ahead of the one being written
    int c_ui = range.unit - 1, c_s = range.off, c_end = 0, c_left = range.n, c_keys = 0;
    const uint8_t* c_src = nullptr;
    auto fetch = [&] {
      if (c_left <= 0) return;
      if (c_s >= c_end) {
        c_s -= c_end;
        do c_end = kv4_items(p, range.at(++c_ui));
        while (c_end == 0);
        const Kv4Unit u = range.at(c_ui);
        c_src = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, u.b, u.h, 0);
        c_keys = kv4_last_pos(p, u) + 1;
      }
      kv4_fetch(k, c_src, c_s * kTile, c_keys, false, w, lane);
      kv4_fetch(v, c_src + kKv4Half, c_s * kTile, c_keys, true, w, lane);
      ++c_s;
      --c_left;
    };
    fetch();
    for (int it = 0; it < range.n; ++it) {
      const int st = it % kKv4ChunkStages;
      const uint32_t ph = ((it / kKv4ChunkStages) & 1) ^ 1;
      if (!mbar_wait(&sh->k_empty[st], ph, abort_flag)) goto done;
      kv4_widen(k, sK + st * kKv4TileOp, w, lane);
      fence_proxy_async_smem();
      mbar_arrive(&sh->k_full[st]);
      if (!mbar_wait(&sh->v_empty[st], ph, abort_flag)) goto done;
      kv4_widen(v, sV + st * kKv4TileOp, w, lane);
      fence_proxy_async_smem();
      mbar_arrive(&sh->v_full[st]);
      fetch();
    }
  } else if (warp == 12 || warp == 13) {
    // ------------------------------------------------ MMA issuers, as in attn.cuh
    const bool s_issuer = warp == 12;
    const uint32_t idesc_s = idesc_f16_f32(128, 128, false), idesc_o = idesc_f16_f32(128, 128, true);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV = sdesc_sw128(smem_u32(sV), kKv4TileOpHalf, 1024);
    uint32_t it = 0;           // steps
    uint32_t ns = 0;           // products issued into the S buffer
    uint32_t npv[2] = {0, 0};  // P.V products per tile
    uint32_t ux[2] = {0, 0};   // units per tile
    int done = 0;
    for (int ui = range.unit, s0 = range.off; done < range.n; ++ui, s0 = 0) {
      const Kv4Unit u = range.at(ui);
      const int s1 = min(kv4_items(p, u), s0 + range.n - done);
      if (s1 <= s0) continue;
      done += s1 - s0;
      const int nx = u.rows > kTile ? 2 : 1;
      for (int s = s0; s < s1; ++s, ++it) {
        const int st = it % kKv4ChunkStages;
        const uint32_t ph = (it / kKv4ChunkStages) & 1;
        if (s_issuer) {
          if (!mbar_wait(&sh->k_full[st], ph, abort_flag)) goto mma_done;
          for (int x = 0; x < nx; ++x) {
            if (s == s0 && !mbar_wait(&sh->q_full[x], ux[x] & 1, abort_flag)) goto mma_done;
            if (ns > 0 && !mbar_wait(&sh->s_free, (ns - 1) & 1, abort_flag)) goto mma_done;
            tc_fence_after();
            const uint64_t q0 = dQ + ((x * kKv4TileOp) >> 4), k0 = dK + ((st * kKv4TileOp) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t off = ((kk >> 2) * kKv4TileOpHalf + (kk & 3) * 32) >> 4;
                mma_bf16_ss(tmem + kKv4TmemS, q0 + off, k0 + off, idesc_s, kk > 0);
              }
              mma_commit(&sh->s_full[x]);
              if (s + 1 == s1) mma_commit(&sh->q_empty[x]);
            }
            __syncwarp();
            ++ns;
          }
          if (elect_one()) mma_commit(&sh->k_empty[st]);
          __syncwarp();
        } else {
          if (!mbar_wait(&sh->v_full[st], ph, abort_flag)) goto mma_done;
          for (int x = 0; x < nx; ++x) {
            if (!mbar_wait(&sh->p_full[x], npv[x] & 1, abort_flag)) goto mma_done;
            tc_fence_after();
            const uint64_t v0 = dV + ((st * kKv4TileOp) >> 4);
            const uint32_t tPx = tmem + kKv4TmemP + x * 64, tOx = tmem + kKv4TmemO + x * 128;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ts(tOx, tPx + kk * 8, v0 + ((kk * 2048) >> 4), idesc_o, (s > s0 || kk > 0) ? 1u : 0u);
              mma_commit(&sh->pv_done[x]);
            }
            __syncwarp();
            ++npv[x];
          }
          if (elect_one()) mma_commit(&sh->v_empty[st]);
          __syncwarp();
        }
      }
      ux[0] += 1;
      ux[1] += nx > 1 ? 1 : 0;
    }
  mma_done:
    // every issued product must finish before TMEM is released
    __syncwarp();
    if (elect_one()) mma_commit(&sh->drain);
    __syncwarp();
    {
      volatile int keep_waiting = 0;
      mbar_wait(&sh->drain, 0, &keep_waiting, (1ull << 28));
    }
  } else if (warp == 14 && lane == 0) {
    // ------------------------------------------------ query tiles
    Kv4QueryPort port = {sh->q_full, sh->q_empty, sQ, nullptr, abort_flag, true};
    Kv4Feeder<2> feed;
    bool going = true;
    int done = 0;
    for (int ui = range.unit, s0 = range.off; going && done < range.n; ++ui, s0 = 0) {
      const Kv4Unit u = range.at(ui);
      const int s1 = min(kv4_items(p, u), s0 + range.n - done);
      if (s1 <= s0) continue;
      done += s1 - s0;
      for (int x = 0; going && x < (u.rows > kTile ? 2 : 1); ++x) {
        port.src = p.qtiles + ((int64_t)ui * 2 + x) * kKv4TileOp;
        going = feed.load(port, x);
      }
    }
    feed.finish(port);
  }
done:
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ accumulated weights

// acc[key] += sum over the rows of the kv head of 2^(score - lse), for 256 keys
// of a kv head a CTA: S^T = K Q^T per 128 keys and 128 rows, thread = key, so
// that the sum over rows stays in a thread. Keys are widened once; query tiles
// pass by. Two CTAs per SM (256 TMEM columns and 98 KB each) keep the
// exponentials, which bound it, going while one of them starts or waits: 537
// million of them in 222 us, 64 % of the rate of the function units. (Two loads
// from TMEM under way at a time gave 218 us, but nothing orders the use of their
// registers behind the wait for one of the two.)
//   warps 0-3, 4-7  the sums of key tile 0, 1     warp 8  TMEM owner, products
//   warp 9          query tiles and their rows' scales, sums and positions
constexpr int kKv4ColThreads = 320;
struct Kv4ColShared {
  uint64_t q_full, q_empty, s_full[2], s_free[2], row_full[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  float2 row[2][kTile];  // scale and minus log2 of the sum of each row of a query tile, for two tiles
  int pos[2][kTile];     // last key of each row
};
constexpr int kKv4ColSmemBytes = 3 * kKv4TileOp + 1024 + sizeof(Kv4ColShared);

template <bool MASKED>
__global__ void __launch_bounds__(kKv4ColThreads, 2) kv4_chunk_weight_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;                    // key tile 0, 1
  uint8_t* sQ = sK + 2 * kKv4TileOp;
  Kv4ColShared* sh = reinterpret_cast<Kv4ColShared*>(sQ + kKv4TileOp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  int t0;
  const int n = kv4_queries(p, p.cu, b, &t0);
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int key0 = blockIdx.x * 2 * kTile, pos0 = len - n, rows = n * p.G;
  if (n == 0 || key0 >= len) return;
  const int slot0 = kv4_first_slot(p, b, t0);
  // tiles of 128 rows; rows before the first key's position attend nothing here
  const int tile0 = key0 > pos0 ? (int)((int64_t)(key0 - pos0) * p.G / kTile) : 0, tiles = (rows + kTile - 1) / kTile;

  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh->s_full[x], 1);
      mbar_init(&sh->s_free[x], 128);
      mbar_init(&sh->row_full[x], 32);
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&sh->tmem_base, 256);
    tmem_relinquish();
  }
  if (warp < 8) {
    const uint8_t* src = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, b, h, 0);
    Kv4Pieces x;
    kv4_fetch(x, src, key0 + (warp >> 2) * kTile, len, false, warp & 3, lane);
    kv4_widen(x, sK + (warp >> 2) * kKv4TileOp, warp & 3, lane);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort_flag;

  if (warp < 8) {
    const int X = warp >> 2, key = key0 + threadIdx.x;
    const uint32_t tS = tmem + X * kTile + ((uint32_t)((warp & 3) * 32) << 16);
    float* acc = p.acc + ((int64_t)b * p.Hkv + h) * p.tiles * kKv4Tile + key;
    const float old = key < len ? *acc : 0.f;
    uint64_t sum[2] = {0ull, 0ull};
    for (int i = tile0; i < tiles; ++i) {
      const int k = i - tile0;
      if (!mbar_wait(&sh->row_full[k & 1], (k >> 1) & 1, abort_flag)) goto done;
      if (!mbar_wait(&sh->s_full[X], k & 1, abort_flag)) goto done;
      __syncwarp();
      tc_fence_after();
      // the first row's position is the smallest
      const bool edge = key0 + (X + 1) * kTile - 1 > sh->pos[k & 1][0];
      uint32_t on[4] = {~0u, ~0u, ~0u, ~0u};  // with a gate: the rows that chose this key tile's block
      if constexpr (MASKED) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          on[c] = i * kTile + c * 32 < rows && key0 + X * kTile < len
                      ? kv4_picks(p, b, h, t0, i * kTile + c * 32, (key0 + X * kTile) / p.pick_B) : 0;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32(tS + c * 32, r);
        tmem_ld_wait();
        if (edge) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (key > sh->pos[k & 1][c * 32 + e]) r[e] = __float_as_uint(-INFINITY);
        }
        if (MASKED && on[c] != ~0u) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(on[c] >> e & 1u)) r[e] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float4 f = *reinterpret_cast<const float4*>(&sh->row[k & 1][c * 32 + e]);
          const float y0 = ex2_approx(fmaf(__uint_as_float(r[e]), f.x, f.y));
          const float y1 = ex2_approx(fmaf(__uint_as_float(r[e + 1]), f.z, f.w));
          sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2_pack(y0, y1));
        }
      }
      // only now: the rows' numbers are read until here
      tc_fence_before();
      mbar_arrive(&sh->s_free[X]);
    }
    if (key < len) {
      const uint64_t s = f2_add(sum[0], sum[1]);
      *acc = old + (f2_lo(s) + f2_hi(s));
    }
  } else if (warp == 8) {
    const uint32_t idesc = idesc_f16_f32(128, 128, false);
    const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
    for (int i = tile0; i < tiles; ++i) {
      const int k = i - tile0;
      if (!mbar_wait(&sh->q_full, k & 1, abort_flag)) goto mma_done;
      for (int x = 0; x < 2; ++x) {
        if (k > 0 && !mbar_wait(&sh->s_free[x], (k - 1) & 1, abort_flag)) goto mma_done;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kKv4TileOpHalf + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tmem + x * kTile, dK + ((x * kKv4TileOp) >> 4) + off, dQ + off, idesc, kk > 0);
          }
          mma_commit(&sh->s_full[x]);
          if (x == 1) mma_commit(&sh->q_empty);
        }
        __syncwarp();
      }
    }
  mma_done:
    __syncwarp();
    if (elect_one()) mma_commit(&sh->drain);
    __syncwarp();
    {
      volatile int keep_waiting = 0;
      mbar_wait(&sh->drain, 0, &keep_waiting, (1ull << 28));
    }
  } else {
    Kv4QueryPort port = {&sh->q_full, &sh->q_empty, sQ, nullptr, abort_flag, lane == 0};
    Kv4Feeder<1> feed;
    int k = 0;
    for (int i = tile0; i < tiles; ++i, ++k) {
      const int64_t ui = (int64_t)(slot0 + i / 2) * p.Hkv + h;
      port.src = p.qtiles + (ui * 2 + (i & 1)) * kKv4TileOp;
      // the rows' numbers of two tiles ago have been read once the products of the last one could start
      if (!feed.load(port, 0)) break;
      for (int c = lane; c < kTile; c += 32) {
        const int row = i * kTile + c, tok = row / p.G;
        const bool on = row < rows && pos0 + tok >= 0;
        // a row without keys, or behind the last: the score minus infinity
        const float scale = on ? __ldcg(p.qscale + ui * kKv4ChunkRows + (i & 1) * kTile + c) : 1.f;
        const float lse = on ? __ldcg(p.lse + (int64_t)(h * p.G + row % p.G) * p.total + t0 + tok) : 0.f;
        sh->row[k & 1][c] = make_float2(scale, on ? -kv4_log2_sum(lse) : -INFINITY);
        sh->pos[k & 1][c] = row < rows ? pos0 + tok : INT32_MAX;
      }
      mbar_arrive(&sh->row_full[k & 1]);
    }
    feed.finish(port);
  }
done:
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace moba
