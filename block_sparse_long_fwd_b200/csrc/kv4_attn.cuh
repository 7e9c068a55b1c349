// Attention of the last query tokens of each sequence over the 4-bit
// key/value cache (kv4.cuh): gate, attention, join and the accumulated weights
// of the cached tokens.
//
// Query token i of the n of sequence b stands at position
// lengths[b] - n + i and attends the cached tokens up to itself: all of them,
// or, with block means, those of its own block and of the topk - 1 past
// blocks of the highest score q . mean (ties to the lower block index).
//
// Work is cut into units: R consecutive rows (token, q head of one kv head) of
// one sequence and kv head, with the 64-token tiles of the cache that at least
// one of them attends. All units' tiles in a row are dealt out evenly, one
// contiguous range to each CTA of a grid of one CTA per SM, and of that one to
// each warp, wherever the units begin and end: lengths that differ, and few
// units with many tiles, balance by themselves. A unit that several warps share
// is joined in shared memory, and by a second kernel where it crosses CTAs.
#pragma once

#include "kv4.cuh"
#include "kv4_feed.cuh"

namespace moba {

struct __align__(16) Kv4Unit {
  int32_t b, h;       // sequence, kv head
  int32_t row0, rows; // first row (token * G + q head) and rows of the unit
  int32_t t0, pos0;   // packed index and position of the sequence's first query
  int32_t tiles;      // 64-token tiles
  int32_t blocks;     // with a gate: entries of the unit's block list
};

struct Kv4AttnParams {
  const __nv_bfloat16* q;  // [total][Hq][128]
  const uint8_t* kv4;
  const int32_t *lengths, *cu;  // cu null: total / batch queries each
  const float* kmean;           // [batch][Hkv][means][128], or null: every key
  int64_t total, tiles;
  int batch, Hq, Hkv, G;
  int B, topk, means;           // with kmean: block size, means = capacity / B
  int blocks;                   // blocks of the capacity, the last one partial
  int R, rshift, slots;         // rows of a unit, 2^rshift; unit slots per kv head
  int each;                     // without cu, queries of a sequence
  float scale_log2;             // log2(e) / sqrt(128)
  float* acc;                   // [batch][Hkv][tiles * 64], or null
  __nv_bfloat16* out;           // [total][Hq][128]
  float* lse;                   // [Hq][total]
  // scratch
  Kv4Unit* units;               // [slots * Hkv]
  int* before;                  // [slots * Hkv + 1]: items of the units before
  uint2* list;                  // [slots * Hkv][list_cap]: (block, rows that chose it), ascending
  uint32_t* chosen;             // or null: [slots * Hkv][blocks]: rows of the unit that chose the block
  double* scores;               // [clusters][R][means]
  float* seen;                  // or null: [items][4][64][2] log2 scores, of each tile's keys and two rows
  float* part;                  // [2 * ctas][R * 130]: O, then m and l
  int list_cap, ctas;
  int least;                    // items of a CTA that has any
  int steps;                    // ranges are dealt out in steps of 128 keys (else in tiles)
  uint8_t* qtiles;              // [slots * Hkv][2][32768]: query tiles as fp16 operands
  float* qscale;                // [slots * Hkv][256]: their rows' scales
  const uint32_t* picks;        // or null: the gate's `chosen` of units of 32 rows
  int pick_B, pick_blocks;      // its block size and blocks
};

// Queries of sequence b: packed index of the first and their number. Offsets
// outside the rows are a caller's error, recorded and read as no query.
__device__ __forceinline__ int kv4_queries(const Kv4AttnParams& p, const int32_t* cu, int b, int* t0) {
  if (!cu) {
    *t0 = b * p.each;
    return p.each;
  }
  const int c0 = cu[b], c1 = cu[b + 1];
  *t0 = c0;
  if (c0 < 0 || c1 < c0 || c1 > p.total) {
    record_status(MOBA_ERR_DEVICE_CHECK);
    return 0;
  }
  return c1 - c0;
}

// First unit slot of sequence b, whose rows start at row t0 * G of a kv head:
// each sequence has room for its rows / R, rounded up, without a scan over the
// sequences before it (floor(x / R) grows by at least ceil(n / R) - 1).
__device__ __forceinline__ int kv4_first_slot(const Kv4AttnParams& p, int b, int t0) {
  return (int)((uint32_t)t0 * (uint32_t)p.G >> p.rshift) + b;
}

// The unit of slot `slot` of kv head h; rows = 0 for an unused slot. cu and
// lengths are p's or a copy of them.
__device__ __forceinline__ Kv4Unit kv4_unit_of(const Kv4AttnParams& p, const int32_t* cu, const int32_t* lengths,
                                               int slot, int h) {
  Kv4Unit u = {};
  u.h = h;
  int lo = 0, hi = p.batch;  // first_slot(lo) <= slot < first_slot(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int t = cu ? cu[mid] : mid * p.each;
    if (kv4_first_slot(p, mid, t) <= slot) lo = mid;
    else hi = mid;
  }
  int t0;
  const int n = kv4_queries(p, cu, lo, &t0);
  const int64_t row0 = ((int64_t)slot - kv4_first_slot(p, lo, t0)) << p.rshift;
  if (row0 < 0 || row0 >= (int64_t)n * p.G) return u;
  u.b = lo;
  u.row0 = (int)row0;
  u.rows = min(p.R, (int)((int64_t)n * p.G - row0));
  u.t0 = t0;
  u.pos0 = kv4_length(lengths, lo, p.tiles * kKv4Tile) - n;
  return u;
}

// The rows of 32 (from row `row`, a multiple of 32, of sequence b's kv head h) that
// chose a block, a bit each.
__device__ __forceinline__ uint32_t kv4_picks(const Kv4AttnParams& p, int b, int h, int t0, int row, int block) {
  const int64_t slot = ((uint32_t)t0 * (uint32_t)p.G >> 5) + b + (row >> 5);
  return __ldcg(p.picks + (slot * p.Hkv + h) * p.pick_blocks + block);
}

// Position of the unit's last row: the last key that any of its rows attends.
__device__ __forceinline__ int kv4_last_pos(const Kv4AttnParams& p, const Kv4Unit& u) {
  return u.pos0 + (u.row0 + u.rows - 1) / p.G;
}

// What is dealt out of a unit: tiles, or steps of two tiles.
__device__ __forceinline__ int kv4_items(const Kv4AttnParams& p, const Kv4Unit& u) {
  return p.steps ? (u.tiles + 1) / 2 : u.tiles;
}

// ------------------------------------------------------------------ gate

constexpr int kKv4GateThreads = 256;
constexpr int kKv4GateRegs = 8;  // scores a lane keeps: rows with up to 256 past blocks select from registers

// A score as an integer of the same order, -0 as 0.
__device__ __forceinline__ uint64_t kv4_score_key(double s) {
  const uint64_t u = __double_as_longlong(s + 0.);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// The largest (key, lowest block) over the warp; j < 0 takes no part, and comes
// back where nobody does.
__device__ __forceinline__ void kv4_warp_best(uint64_t& key, int& j) {
  const uint32_t hi = j < 0 ? 0 : (uint32_t)(key >> 32), top = __reduce_max_sync(0xFFFFFFFFu, hi);
  const uint32_t lo = j >= 0 && hi == top ? (uint32_t)key : 0, low = __reduce_max_sync(0xFFFFFFFFu, lo);
  const bool best = j >= 0 && hi == top && (uint32_t)key == low;
  j = (int)__reduce_min_sync(0xFFFFFFFFu, best ? (uint32_t)j : 0xFFFFFFFFu);
  key = (uint64_t)top << 32 | low;
}

// One cluster per unit (looping over units): its CTAs score the past blocks
// for all rows of the unit, the first CTA selects and lists. Scores are sums
// in fp64 of products that are exact there (bf16 times fp32), so near ties
// fall as in exact arithmetic; they are a few per cent of the work of the
// attention itself (one mean per block of at least 128 keys). Latency-bound:
// 13 us for 255 past blocks and 4 rows of each of 8 kv heads.
__global__ void __launch_bounds__(kKv4GateThreads) kv4_gate_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  extern __shared__ uint32_t picked[];  // [blocks]: rows of the unit that chose the block
  __shared__ float q[32][kHeadDim];
  __shared__ Kv4Unit s_unit;
  __shared__ uint32_t warp_sums[32];
  uint32_t rank, csize;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int WARPS = kKv4GateThreads / 32;
  double* scores = p.scores + (int64_t)cluster * p.R * p.means;
  const int nu = p.slots * p.Hkv;
  // offsets and lengths in one trip, where they fit
  __shared__ int32_t copy[2 * kKv4GateThreads + 1];
  const int32_t *cu = p.cu, *lengths = p.lengths;
  if (p.batch <= kKv4GateThreads) {
    if (tid < p.batch) copy[tid] = p.lengths[tid];
    lengths = copy;
    if (cu) {
      for (int i = tid; i <= p.batch; i += kKv4GateThreads) copy[kKv4GateThreads + i] = p.cu[i];
      cu = copy + kKv4GateThreads;
    }
    __syncthreads();
  }
  for (int ui = cluster; ui < nu; ui += clusters) {
    if (tid == 0) s_unit = kv4_unit_of(p, cu, lengths, ui / p.Hkv, ui % p.Hkv);
    __syncthreads();
    Kv4Unit u = s_unit;
    const int last = u.rows ? kv4_last_pos(p, u) : -1;
    const int own = last < 0 ? 0 : last / p.B;  // past blocks of the last row
    const int n = min(own, p.means);
    if (last >= 0) {
      // this warp's first means are on their way while the rows come
      const float* means = p.kmean + ((int64_t)u.b * p.Hkv + u.h) * p.means * kHeadDim;
      const int j0 = rank * WARPS + warp, step = csize * WARPS;
      float4 m[4];
      auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m[i] = j + i * step < n ? __ldg(reinterpret_cast<const float4*>(means + (int64_t)(j + i * step) * kHeadDim) + lane)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      };
      fetch(j0);
      for (int i = tid; i < u.rows * 16; i += kKv4GateThreads) {
        const int r = i >> 4, c = i & 15, rr = u.row0 + r;
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(
            p.q + ((int64_t)(u.t0 + rr / p.G) * p.Hq + u.h * p.G + rr % p.G) * kHeadDim) + c);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[r][8 * c + 2 * k] = __uint_as_float(w[k] << 16);
          q[r][8 * c + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
      if (rank == 0)
        for (int j = tid; j < p.blocks; j += kKv4GateThreads) picked[j] = 0;
      __syncthreads();
      for (int j = j0; j < n; j += 4 * step) {
        if (j != j0) fetch(j);
        for (int r = 0; r < u.rows; ++r) {
          const float4 x = *reinterpret_cast<const float4*>(&q[r][lane * 4]);
          double s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] = (double)x.x * m[i].x;
            s[i] = fma((double)x.y, (double)m[i].y, s[i]);
            s[i] = fma((double)x.z, (double)m[i].z, s[i]);
            s[i] = fma((double)x.w, (double)m[i].w, s[i]);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], d);
          if (lane == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (j + i * step < n) scores[(int64_t)r * p.means + j + i * step] = s[i];
        }
      }
    }
    kv4_cluster_sync();
    if (rank == 0) {
      if (last >= 0) {
        for (int r = warp; r < u.rows; r += WARPS) {
          const int pos = u.pos0 + (u.row0 + r) / p.G;
          if (pos < 0) continue;
          const int mine = pos / p.B, picks = min(p.topk - 1, mine);
          const uint32_t bit = 1u << r;
          if (lane == 0) atomicOr(&picked[mine], bit);
          if (picks == mine) {
            for (int j = lane; j < mine; j += 32) atomicOr(&picked[j], bit);
            continue;
          }
          const double* sc = scores + (int64_t)r * p.means;
          const bool few = mine <= 32 * kKv4GateRegs;
          uint64_t mv[kKv4GateRegs];
          uint32_t left = 0;  // blocks of this lane that are still to be had
          if (few)
#pragma unroll
            for (int i = 0; i < kKv4GateRegs; ++i)
              if (i * 32 + lane < mine) mv[i] = kv4_score_key(__ldcg(sc + i * 32 + lane)), left |= 1u << i;
          uint64_t last_key = 0;
          int last_j = -1;
          for (int k = 0; k < picks; ++k) {
            uint64_t key = 0;
            int j = -1;
            if (few) {
#pragma unroll
              for (int i = 0; i < kKv4GateRegs; ++i)
                if (left >> i & 1u && (j < 0 || mv[i] > key)) key = mv[i], j = i * 32 + lane;
            } else {  // the best of those behind the last one
              for (int jj = lane; jj < mine; jj += 32) {
                const uint64_t v = kv4_score_key(__ldcg(sc + jj));
                if ((last_j < 0 || v < last_key || (v == last_key && jj > last_j)) && (j < 0 || v > key)) key = v, j = jj;
              }
            }
            kv4_warp_best(key, j);
            if (few && (j & 31) == lane) left &= ~(1u << (j >> 5));
            if (lane == 0) atomicOr(&picked[j], bit);
            last_key = key;
            last_j = j;
          }
        }
      }
      __syncthreads();
      // the chosen blocks in order; the last one (the last row's own) may be partial
      uint2* list = p.list + (int64_t)ui * p.list_cap;
      uint32_t count = 0;
      if (last >= 0) {
        for (int k0 = 0; k0 <= own; k0 += kKv4GateThreads) {
          const int j = k0 + tid;
          const uint32_t rows = j <= own ? picked[j] : 0;
          uint32_t total;
          const uint32_t at = count + kv4_block_scan(rows != 0, warp_sums, &total);
          if (rows && at < (uint32_t)p.list_cap) list[at] = make_uint2(j, rows);
          count += total;
        }
        count = min(count, (uint32_t)p.list_cap);
        if (p.chosen)
          for (int j = tid; j < p.blocks; j += kKv4GateThreads) p.chosen[(int64_t)ui * p.blocks + j] = picked[j];
      }
      if (tid == 0) {
        u.blocks = count;
        u.tiles = count ? (int)(count - 1) * (p.B / kKv4Tile) + (last - own * p.B) / kKv4Tile + 1 : 0;
        p.units[ui] = u;
      }
    }
    // the next unit reuses the scores
    kv4_cluster_sync();
  }
}

// ------------------------------------------------------------------ plan

// Items of a CTA's range: the same for all but the last that has any. (Items
// fit 31 bits: the host sees to it.)
__device__ __forceinline__ int kv4_quota(const Kv4AttnParams& p, int all) {
  return max((all + p.ctas - 1) / p.ctas, p.least);
}

// Where each part's range begins (a part is a warp, or the CTA): every CTA scans
// all units' tiles for itself (they follow from the lengths alone, or the gate
// has left them): 3 us for one sequence of 8 kv heads, 5 for 64, where a kernel
// of its own was 6 to 9 us with its launch.
// The units that the CTA's range touches, and the items before them, are
// left in scratch for the rest of the CTA and for the join (units of several
// CTAs get the same values from each); CTA 0 leaves those without tiles.
// `copy`: shared memory for the offsets and lengths, `room` words.
// The first units of the range stay in shared memory, where every role walks
// them without a trip to L2.
constexpr int kKv4Kept = 16;
struct Kv4Range {
  const Kv4Unit* kept;
  const Kv4Unit* units;
  int first;      // unit of kept[0]
  __device__ __forceinline__ Kv4Unit at(int ui) const { return ui - first < kKv4Kept ? kept[ui - first] : units[ui]; }
  int n;          // items of this part
  int item;       // the first of them, of all
  int unit, off;  // its first unit, items of it that lie before the range
  bool any;       // the CTA has some
};

template <int THREADS, int PARTS>
__device__ __forceinline__ Kv4Range kv4_plan(const Kv4AttnParams& p, int32_t* copy, int room) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int warp_sums[WARPS];
  __shared__ Kv4Unit s_kept[kKv4Kept];
  __shared__ int s_at[kKv4Kept];  // items before a kept unit
  __shared__ int s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int nu = p.slots * p.Hkv;
  // without a gate the units of a slot differ in their head alone
  const int heads = p.kmean ? 1 : p.Hkv, entries = nu / heads;
  const int32_t *cu = p.cu, *lengths = p.lengths;
  if (tid < kKv4Kept) s_kept[tid].tiles = 0;  // units without tiles are not kept
  if (!p.kmean && 2 * p.batch + 1 <= room) {
    for (int i = tid; i < p.batch; i += THREADS) copy[i] = p.lengths[i];
    lengths = copy;
    if (cu) {
      for (int i = tid; i <= p.batch; i += THREADS) copy[p.batch + i] = p.cu[i];
      cu = copy + p.batch;
    }
    __syncthreads();
  }
  // Neighbouring entries for each thread, in three sweeps: their items; the unit in which the CTA's range begins; what
  // the range touches. (One piece of code: this runs once, and much of what it costs is fetching its instructions.)
  const int mine = (entries + THREADS - 1) / THREADS, e0 = tid * mine;
  Kv4Unit u = {};
  int x = 0, before = 0, all = 0, quota = 0, lo = 0, hi = 0;
#pragma unroll 1
  for (int sweep = 0; sweep < 3; ++sweep) {
    int at = before;
    const bool here = sweep == 0 || (before <= hi && before + x >= lo);
#pragma unroll 1
    for (int i = 0; here && i < mine; ++i) {
      const int e = e0 + i;
      if (e >= entries) break;
      if (sweep == 0 || mine > 1) {
        if (p.kmean) {
          u = p.units[e];
        } else {
          u = kv4_unit_of(p, cu, lengths, e, 0);
          const int last = u.rows ? kv4_last_pos(p, u) : -1;
          u.tiles = last < 0 ? 0 : last / kKv4Tile + 1;
        }
      }
      const int n = kv4_items(p, u);
      if (sweep == 0 && n == 0 && cta == 0 && !p.kmean)
        for (int h = 0; h < heads; ++h) u.h = h, p.units[e * heads + h] = u;
      if (sweep > 0) {
        int y = at;
#pragma unroll 1
        for (int h = 0; h < heads; ++h, y += n) {
          if (y >= hi || (n == 0 ? y < lo : y + n <= lo)) continue;
          const int ui = e * heads + h;
          if (n == 0) {  // the walk through the range passes it
            if (!p.kmean && sweep == 2) u.h = h, p.units[ui] = u;
            continue;
          }
          if (sweep == 1) {
            if (y <= lo) s_first = ui;
            continue;
          }
          if (!p.kmean) u.h = h, p.units[ui] = u;
          p.before[ui] = y;
          const int k = ui - s_first;
          if (k < kKv4Kept) s_kept[k] = u, s_at[k] = y;
        }
      }
      at += n * heads;
    }
    if (sweep == 0) {
      x = at;
      int s = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += y;
      }
      if (lane == 31) warp_sums[warp] = s;
      __syncthreads();
      const int y = lane < WARPS ? warp_sums[lane] : 0;
      before = s - x + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0);
      all = __reduce_add_sync(0xFFFFFFFFu, y);
      quota = kv4_quota(p, all);
      lo = (int)min((int64_t)cta * quota, (int64_t)all);
      hi = min(lo + quota, all);
      if (cta == 0 && tid == 0) p.before[nu] = all;
    } else {
      __syncthreads();
    }
  }
  Kv4Range g;
  const int part = PARTS == 1 ? 0 : warp;
  g.kept = s_kept;
  g.units = p.units;
  g.first = s_first;
  g.any = hi > lo;
  const int even = (hi - lo) / PARTS, more = (hi - lo) % PARTS;  // the first `more` parts take one item more
  g.n = even + (part < more ? 1 : 0);
  g.item = lo + part * even + min(part, more);
  g.unit = g.off = 0;
  if (g.n) {
    // the unit that this part begins in: among the kept ones, a lane each, or further on
    const int start = g.item;
    const bool in = lane < kKv4Kept && s_kept[lane].tiles && s_at[lane] <= start &&
                    start < s_at[lane] + kv4_items(p, s_kept[lane]);
    const uint32_t found = __ballot_sync(0xFFFFFFFFu, in);
    if (found) {
      g.unit = g.first + __ffs(found) - 1;
      g.off = start - s_at[__ffs(found) - 1];
    } else {
      int ui = g.first + kKv4Kept;
      for (;; ++ui) {  // the range reaches this unit: it ends there
        const int n = kv4_items(p, p.units[ui]);
        if (n && p.before[ui] <= start && start < p.before[ui] + n) break;
      }
      g.unit = ui;
      g.off = start - p.before[ui];
    }
  }
  return g;
}

// ------------------------------------------------------------------ attention

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 transpose of 16-bit values held by a warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// t (c - z) from codes, without a rounding. A nibble at bit 4 under fp16's 64 is
// 64 + c, and t (64 + c) - t (64 + z) is one fused multiply-add: 64 + z has
// seven significant bits and t four, so the product fits fp16's eleven. A nibble
// at bit 0 stands under 1024, whose eleven bits and t's four do not fit: a
// subtraction and a multiplication. Shifting nibbles 0 and 2 up to bit 4 would
// cost as much and one register more (1M tokens of 8 heads 263 against 265 us);
// zero points taken off by a product of their own, which leaves masks and
// multiplications, were no faster (274 against 267) and cancel digits. t is a
// 64th of the scale, so that t (64 + z) stays below fp16's largest number; t is
// a multiple of 2^-23, so all stays exact.
struct Kv4Par {
  uint32_t t, tz, z;  // t, -t (64 + z) and 1024 + z, of two tokens (or of one, twice)
};
// (a & mask) | top in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t top) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(top));
  return d;
}
__device__ __forceinline__ Kv4Par kv4_par(uint32_t pp) {
  Kv4Par r;
  r.t = h2_mul(pp & 0x7F807F80u, 0x24002400u);  // 2^-6
  r.z = and_or(pp, 0x000F000Fu, 0x64006400u);
  r.tz = h2_mul(h2_sub(0x63806380u, r.z), r.t);  // 960 - (1024 + z)
  return r;
}
// t (c - z) for nibbles 0..3 of both halves of a word.
__device__ __forceinline__ void kv4_pairs(uint32_t w, const Kv4Par& p, uint32_t (&x)[4]) {
  const uint32_t h = w >> 8;
  x[0] = h2_mul(h2_sub(and_or(w, 0x000F000Fu, 0x64006400u), p.z), p.t);
  x[1] = h2_fma(and_or(w, 0x00F000F0u, 0x54005400u), p.t, p.tz);
  x[2] = h2_mul(h2_sub(and_or(h, 0x000F000Fu, 0x64006400u), p.z), p.t);
  x[3] = h2_fma(and_or(h, 0x00F000F0u, 0x54005400u), p.t, p.tz);
}

// The factors that bring a row with the largest magnitude `top` (bf16 bits) to
// fp16, and the one that turns its products into log2 scores.
__device__ __forceinline__ float kv4_query_scale(uint32_t top, float scale_log2, float& f1, float& f2) {
  const int e = (int)(top >> 7);  // biased exponent; 0: zero or subnormal, 255: not finite
  // 2^k with e - 127 + k = 14, in two factors that are normal numbers
  const int k = (e == 0 || e == 255) ? 0 : 141 - e;
  const int k1 = k / 2, k2 = k - k1;
  f1 = __int_as_float((127 + k1) << 23);
  f2 = __int_as_float((127 + k2) << 23);
  return 64.f * scale_log2 * __int_as_float((127 - k1) << 23) * __int_as_float((127 - k2) << 23);
}

// The same for a word of one token, the first (HI = 0) or second of the two that
// the parameters are of: fp16 instructions take either half twice for free.
template <int HI>
__device__ __forceinline__ uint32_t h2_half(uint32_t x) {
  const __half2 h = *reinterpret_cast<const __half2*>(&x), y = HI ? __high2half2(h) : __low2half2(h);
  return *reinterpret_cast<const uint32_t*>(&y);
}
template <int HI>
__device__ __forceinline__ void kv4_pairs_of(uint32_t w, const Kv4Par& p, uint32_t (&x)[4]) {
  const Kv4Par q = {h2_half<HI>(p.t), h2_half<HI>(p.tz), h2_half<HI>(p.z)};
  kv4_pairs(w, q, x);
}

// A query row enters the products as fp16: times the power of two that brings
// its largest channel to [2^14, 2^15). bf16's eight bits then stay exact but
// for channels 2^28 times smaller than the largest, whose error is 2^-40 of it.
// f: this lane's channels 32 (lane % 4) .. + 31 as eight steps of two pairs.
// Returns the factor that turns products into log2 scores.
__device__ __forceinline__ float kv4_query_fragment(const __nv_bfloat16* row, float scale_log2, uint32_t (&f)[16]) {
  uint4 raw[4] = {};
  if (row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
  uint32_t top = 0;  // largest magnitude, as bf16 bits (a NaN above all)
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  float f1, f2;
  const float scale = kv4_query_scale(top, scale_log2, f1, f2);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    f[i] = pack_half2(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2);
  return scale;
}

// Token (of 16) that row r of the score product holds: neighbours, swapped
// for every other pair, so that the value rows which a lane quad reads next
// are two of even and two of odd index.
__device__ __forceinline__ int kv4_token_of(int r) { return (r & ~1) | ((r ^ (r >> 1)) & 1); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A finished row: lane l's channels 4 l .. 4 l + 3, as a 64th of their sum.
__device__ __forceinline__ void kv4_write_row(const Kv4AttnParams& p, const Kv4Unit& u, int row, int lane, float m,
                                              float l, float4 o) {
  const int rr = u.row0 + row;
  const int64_t t = u.t0 + rr / p.G;
  const int hq = u.h * p.G + rr % p.G;
  const float inv = l != 0.f ? 64.f / l : 0.f;  // a NaN stays one
  reinterpret_cast<uint2*>(p.out + (t * p.Hq + hq) * kHeadDim)[lane] =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0) p.lse[(int64_t)hq * p.total + t] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int NT_, int WARPS_, bool QREG_>
struct Kv4Cfg {
  static constexpr int NT = NT_;            // groups of eight query rows
  static constexpr int R = 8 * NT;
  static constexpr int WARPS = WARPS_;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr bool QREG = QREG_;       // query fragments in registers, else in shared memory
  static constexpr int PIECE = R * kHeadDim * 4;
  struct Shared {
    // a tile a warp: its keys are in use while the values come, and the next tile's keys come while the values are
    // in use; at the end, the warp's partial result of a unit that it began
    uint8_t ring[WARPS][kKv4TileBytes];
    uint8_t piece[WARPS][PIECE];            // the warp's partial result of a unit that it did not begin
    float2 ml[WARPS][2][R];                 // their maxima and sums
    uint2 q[QREG ? 1 : WARPS][NT][8][32];
    uint64_t full[WARPS][2];                // keys, values
    int unit[2 * WARPS];                    // units of the partial results, -1 for none
    int begins[2 * WARPS], ends[2 * WARPS];
    int abort_flag;
  };
  static_assert(kKv4TileBytes >= PIECE, "a partial result fits the warp's ring");
};

using Kv4Few = Kv4Cfg<1, 16, true>;    // up to 8 rows
using Kv4Many = Kv4Cfg<2, 8, false>;   // up to 16 rows

constexpr float kKv4Low = -3.402823466e38f;  // reference before the first score: fp32's lowest
// A row's reference of this magnitude is coarse: from here on fp32 numbers are 2^-3 and more apart, and score minus
// reference, exact but for that, may miss the 12 that it should be by as much. The reference is then rounded down, so
// that the largest weight is 2^12 at least, and what would exceed 2^15, fp16's last power of two, is cut to it: scores
// that close together are not told apart by fp32 sums of that size anyway.
constexpr float kKv4Coarse = 1048576.f;
__device__ __forceinline__ float kv4_reference(float top, float scale) {
  const float mx = top * scale;
  return fabsf(mx) < kKv4Coarse ? mx - 12.f : __fmaf_rd(top, scale, -12.f);
}
__device__ __forceinline__ float kv4_cut(float x) { return x > 15.f ? 15.f : x; }  // a NaN stays one

// Per tile of 64 keys a warp widens the keys' codes into the A operand of
// S^T = K Q^T (keys x rows; the codes' own order is the operand's), finds the
// weights in registers, transposes them 8 x 8, and widens the values' codes into
// the A operand of O^T += V^T P^T. 16 warps of 128 registers (12 of 168 took 276
// us where these took 262). 311 instructions for 16 keys and up to 8 rows. 1M
// tokens of 8 heads: 238 us, 5.1 TB/s, 78 % of a copy's rate. Neither HBM nor
// the issue slots are full (a ragged batch uses 64 % of them at 4.5 TB/s): its
// warps wait in turn for the pipes of half-precision and logic operations, for
// their own last result and for the scheduler. Where there are few tiles the
// chain counts: 12 us for 4096 tokens of one head; 47 for 128K tokens of 8, of
// which the plan takes 4, the tiles 27 and the two joins 6.
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_attn_kernel(Kv4AttnParams p) {
  constexpr int NT = C::NT, R = C::R;
  grid_dependency_sync();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto* sh = reinterpret_cast<typename C::Shared*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * C::WARPS; ++i) mbar_init(&sh->full[0][0] + i, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 2 * C::WARPS) sh->unit[threadIdx.x] = -1;
  const Kv4Range range = kv4_plan<C::THREADS, C::WARPS>(p, reinterpret_cast<int32_t*>(&sh->piece), sizeof(sh->piece) / 4);
  if (!range.any) return;
  const int n = range.n;

  // A warp fetches its own tiles, one bulk copy for the keys and one for the values of each (32 tokens at a time, four
  // copies and two ahead, cost 30 instructions more for 16 keys: 265 against 247 us at 1M tokens). `next` walks the
  // units to the next tile.
  const int tpb = p.B / kKv4Tile;
  Kv4Fetch fetch;
  fetch.left = n;
  int c_ui = range.unit - 1, c_off = range.off, c_end = 0, c_at = 0, c_in = 0;
  const uint8_t* c_src = nullptr;       // the next tile (with a gate, the first of the sequence)
  const uint8_t* src = nullptr;         // the tile that comes
  int key_b = 0, c_key = 0;             // their first keys
  uint32_t rows_b = ~0u;                // rows that chose the block
  auto next = [&] {
    if (c_off >= c_end) {  // on to the next unit that has tiles
      c_off -= c_end;
      do c_end = range.at(++c_ui).tiles;
      while (c_end == 0);
      const Kv4Unit u = range.at(c_ui);
      c_src = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, u.b, u.h, 0);
      if (p.kmean) {
        c_at = c_off / tpb;
        c_in = c_off - c_at * tpb;
      } else {
        c_src += (int64_t)c_off * kKv4TileBytes;
        c_key = c_off * kKv4Tile;
      }
    }
    if (p.kmean) {
      if (c_in == tpb) c_in = 0, ++c_at;
      const uint2 e = p.list[(int64_t)c_ui * p.list_cap + c_at];
      const int tile = (int)e.x * tpb + c_in++;
      src = c_src + (int64_t)tile * kKv4TileBytes;
      key_b = tile * kKv4Tile;
      rows_b = e.y;
    } else {
      src = c_src;
      key_b = c_key;
      c_src += kKv4TileBytes;
      c_key += kKv4Tile;
    }
    ++c_off;
    --fetch.left;
  };
  uint8_t* ring = sh->ring[warp];
  auto issue = [&](int vals) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&sh->full[warp][vals], kKv4Half);
      bulk_load(ring + vals * kKv4Half, src + vals * kKv4Half, kKv4Half, &sh->full[warp][vals]);
    }
  };
  if (n) {
    next();
    issue(0);
    issue(1);
  }

  const int r = lane >> 2, qd = lane & 3;
  const int tok0 = kv4_token_of(r);
  const int vchunk = (r ^ (qd & 2 ? 4 : 0)) * 8;
  const int ve0 = 2 * qd + (qd & 1), ve1 = 2 * qd + ((qd & 1) ^ 1);
  // once a wait has run out (fetch.dead), what follows is computed on what is there, and nothing more is fetched
  int k = 0;          // tiles of this warp behind us
  for (int ui = range.unit, off = range.off; k < n; ++ui, off = 0) {
    const Kv4Unit u = range.at(ui);
    const int stop = k + min(n - k, u.tiles - off);
    if (stop == k) continue;
    // the rows' fragments, scales, and last keys (of this lane's two rows of each group of eight)
    uint32_t qf[16];
    uint64_t qs[NT];
    int last[NT][2];
    const int first_pos = u.pos0 + u.row0 / p.G, last_pos = kv4_last_pos(p, u);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int x = nt * 8 + r, rr = u.row0 + x;
      const __nv_bfloat16* row =
          x < u.rows ? p.q + ((int64_t)(u.t0 + rr / p.G) * p.Hq + u.h * p.G + rr % p.G) * kHeadDim + qd * 32 : nullptr;
      const float s = kv4_query_fragment(row, p.scale_log2, qf);
      qs[nt] = f2_pack(__shfl_sync(0xFFFFFFFFu, s, qd * 8), __shfl_sync(0xFFFFFFFFu, s, qd * 8 + 4));
      if constexpr (!C::QREG) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sh->q[warp][nt][i][lane] = make_uint2(qf[2 * i], qf[2 * i + 1]);  // read back by itself
      }
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2) {
        const int row2 = nt * 8 + 2 * qd + x2;
        last[nt][x2] = row2 < u.rows ? u.pos0 + (u.row0 + row2) / p.G : -1;
      }
    }
    const uint32_t all_rows = (1u << u.rows) - 1;

    float o[NT][8][4] = {};
    uint64_t nm[NT], l2[NT];  // minus the reference, and the sum, of the lane's two rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) nm[nt] = f2_pack(-kKv4Low, -kKv4Low), l2[nt] = 0;

    const int k0 = k;
    for (; k < stop; ++k) {
      const int key_a = key_b;
      const uint32_t rows_a = rows_b;
      const uint8_t* kt = ring;
      const uint8_t* vt = ring + kKv4Half;
      if (!fetch.dead && !mbar_wait(&sh->full[warp][0], k & 1, &sh->abort_flag)) fetch.gave_up(k);

      // scores: keys x rows, 16 keys at a time
      float sc[4][NT][4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int ta = tok0 + g * 16, tb = ta + 8;
        const uint4 wa = *reinterpret_cast<const uint4*>(kt + ta * kKv4Row + qd * 16);
        const uint4 wb = *reinterpret_cast<const uint4*>(kt + tb * kKv4Row + qd * 16);
        const uint32_t pa = *reinterpret_cast<const uint16_t*>(kt + kKv4Params + ta * 8 + qd * 2);
        const uint32_t pb = *reinterpret_cast<const uint16_t*>(kt + kKv4Params + tb * 8 + qd * 2);
        const Kv4Par f = kv4_par(__byte_perm(pa, pb, 0x5410));
        const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4], b[4];
          kv4_pairs_of<0>(xa[w], f, a);
          kv4_pairs_of<1>(xb[w], f, b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 q0, q1;
            if constexpr (C::QREG) {
              q0 = make_uint2(qf[4 * w], qf[4 * w + 1]);
              q1 = make_uint2(qf[4 * w + 2], qf[4 * w + 3]);
            } else {
              q0 = sh->q[warp][nt][2 * w][lane];
              q1 = sh->q[warp][nt][2 * w + 1][lane];
            }
            if (w == 0) mma_f16_first(sc[g][nt], a[0], b[0], a[1], b[1], q0.x, q0.y);
            else mma_f16(sc[g][nt], a[0], b[0], a[1], b[1], q0.x, q0.y);
            mma_f16(sc[g][nt], a[2], b[2], a[3], b[3], q1.x, q1.y);
          }
        }
      }
      __syncwarp();  // the keys are read: the next tile's may take their place
      if (fetch.next_keys()) {
        next();
        issue(0);
      }
      if (!fetch.dead && !mbar_wait(&sh->full[warp][1], k & 1, &sh->abort_flag)) fetch.gave_up(k);

      // keys behind a row's position, and blocks that a row did not choose (a loop of one turn: a branch, where the
      // compiler would have every tile pay for instructions that are switched off)
      const bool edge = key_a + kKv4Tile - 1 > first_pos;
#pragma unroll 1
      for (bool mask = edge || (rows_a & all_rows) != all_rows; mask; mask = false) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key_a + tok0 + g * 16 + (x >> 1) * 8;
              const uint32_t row = nt * 8 + 2 * qd + (x & 1);
              if (key > last[nt][x & 1] || !(rows_a >> row & 1u)) sc[g][nt][x] = -INFINITY;
            }
        // what lies behind the last token may hold anything: its values' scales become zero
#pragma unroll
        for (int x = 0; x < kKv4Tile; x += 32)
          if (key_a + x + lane > last_pos)
            *reinterpret_cast<uint2*>(ring + kKv4Half + kKv4Params + (x + lane) * 8) = make_uint2(0, 0);
        fence_proxy_async_smem();  // before the copy that will overwrite them
        __syncwarp();
      }
      if constexpr (NT == 1) {
        if (p.seen && 2 * qd < u.rows) {  // for the accumulated weights: the lane's two rows of its keys
          float2* to = reinterpret_cast<float2*>(p.seen) + ((int64_t)(range.item + k) * 4 + qd) * kKv4Tile + tok0;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint64_t y = f2_fma(f2_pack(sc[g][0][2 * x], sc[g][0][2 * x + 1]), qs[0], 0);
              to[g * 16 + x * 8] = make_float2(f2_lo(y), f2_hi(y));
            }
        }
      }
      // the first values' codes are on their way while the weights are found
      auto values = [&](int g, uint2 (&w)[2][2], uint32_t (&pp)[2]) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int t0 = ve0 + g * 16 + f * 8, t1 = ve1 + g * 16 + f * 8;
          w[f][0] = *reinterpret_cast<const uint2*>(vt + t0 * kKv4Row + vchunk);
          w[f][1] = *reinterpret_cast<const uint2*>(vt + t1 * kKv4Row + vchunk);
          const uint32_t p0 = *reinterpret_cast<const uint16_t*>(vt + kKv4Params + t0 * 8 + (r >> 1) * 2);
          const uint32_t p1 = *reinterpret_cast<const uint16_t*>(vt + kKv4Params + t1 * 8 + (r >> 1) * 2);
          pp[f] = __byte_perm(p0, p1, 0x5410);
        }
      };
      uint2 w[2][2];
      uint32_t vp[2];
      values(0, w, vp);
      // weights 2^(score - m). The reference m moves when a score exceeds it by more than 15, to 12 below
      // the largest: weights then lie under 2^15, which fp16 holds, and end 2^-37 below the largest
      uint32_t pf[NT][4][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float t[4][4];
        auto shifted = [&] {
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              const uint64_t y = f2_fma(f2_pack(sc[g][nt][x], sc[g][nt][x + 1]), qs[nt], nm[nt]);
              t[g][x] = f2_lo(y);
              t[g][x + 1] = f2_hi(y);
            }
        };
        shifted();
        float top = t[3][3];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          top = fmax3(top, t[g][0], t[g][1]);
          if (g < 3) top = fmax3(top, t[g][2], t[g][3]);
        }
        top = fmaxf(top, t[3][2]);
        if (__any_sync(0xFFFFFFFFu, top > 15.f)) {
          float a2[2], n2[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float q1 = x ? f2_hi(qs[nt]) : f2_lo(qs[nt]), m1 = -(x ? f2_hi(nm[nt]) : f2_lo(nm[nt]));
            float mx = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g) mx = fmax3(mx, sc[g][nt][x], sc[g][nt][x + 2]);
#pragma unroll
            for (int d2 = 4; d2 < 32; d2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d2));
            const bool move = mx * q1 > m1 + 15.f;
            n2[x] = move ? -kv4_reference(mx, q1) : -m1;
            a2[x] = move ? ex2_approx(m1 + n2[x]) : 1.f;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) o[nt][mt][x] *= a2[x], o[nt][mt][x + 2] *= a2[x];
          }
          nm[nt] = f2_pack(n2[0], n2[1]);
          l2[nt] = f2_pack(f2_lo(l2[nt]) * a2[0], f2_hi(l2[nt]) * a2[1]);
          shifted();
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int x = 0; x < 4; ++x) t[g][x] = kv4_cut(t[g][x]);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float e[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = ex2_approx(t[g][x]);
          l2[nt] = f2_add(l2[nt], f2_add(f2_pack(e[0], e[1]), f2_pack(e[2], e[3])));
          pf[nt][g][0] = movmatrix(pack_half2(e[0], e[1]));
          pf[nt][g][1] = movmatrix(pack_half2(e[2], e[3]));
        }
      }
      // O^T += V^T P^T: channels x rows
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        Kv4Par fp[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) fp[f] = kv4_par(vp[f]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[2][2][4];  // [channel parity][keys 0-7, 8-15][nibble]
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t x0 = h ? w[f][0].y : w[f][0].x, x1 = h ? w[f][1].y : w[f][1].x;
            kv4_pairs(__byte_perm(x0, x1, 0x5410), fp[f], a[0][f]);
            kv4_pairs(__byte_perm(x0, x1, 0x7632), fp[f], a[1][f]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][h * 4 + j], a[0][0][j], a[1][0][j], a[0][1][j], a[1][1][j], pf[nt][g][0], pf[nt][g][1]);
        }
        if (g < 3) values(g + 1, w, vp);
      }
      __syncwarp();  // the values are read
      if (fetch.next_values()) issue(1);
    }

    // ---- this warp's part of the unit: all of it is a result, else a piece to be joined
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = -f2_lo(nm[nt]), m[nt][1] = -f2_hi(nm[nt]);
      l[nt][0] = f2_lo(l2[nt]), l[nt][1] = f2_hi(l2[nt]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][x], d);
    const bool begins = off == 0, ends = off + (k - k0) == u.tiles;
    // lane: channels 16 r .. 16 r + 15 of rows 2 qd, 2 qd + 1 of each group of eight (a 64th of them so far)
    if (begins && ends) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = nt * 8 + 2 * qd + x;
          if (row >= u.rows) continue;
          const int rr = u.row0 + row;
          const int64_t t = u.t0 + rr / p.G;
          const int hq = u.h * p.G + rr % p.G;
          const float inv = l[nt][x] != 0.f ? 64.f / l[nt][x] : 0.f;
          uint32_t y[8];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) y[mt] = pack_bf16x2(o[nt][mt][x] * inv, o[nt][mt][x + 2] * inv);
          uint4* out = reinterpret_cast<uint4*>(p.out + (t * p.Hq + hq) * kHeadDim + 16 * r);
          out[0] = make_uint4(y[0], y[1], y[2], y[3]);
          out[1] = make_uint4(y[4], y[5], y[6], y[7]);
          if (r == 0)
            p.lse[(int64_t)hq * p.total + t] =
                l[nt][x] != 0.f ? (m[nt][x] + log2f(l[nt][x])) * 0.6931471805599453f : -INFINITY;
        }
    } else {
      const int which = begins ? 1 : 0;
      if (lane == 0) {
        sh->unit[2 * warp + which] = ui;
        sh->begins[2 * warp + which] = begins;
        sh->ends[2 * warp + which] = ends;
      }
      // a unit that this warp begins and does not end is its last: its ring is free
      __syncwarp();
      float* at = reinterpret_cast<float*>(which ? ring : sh->piece[warp]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = nt * 8 + 2 * qd + x;
          float4* to = reinterpret_cast<float4*>(at + row * kHeadDim + 16 * r);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to[i ^ (r & 3)] = make_float4(o[nt][2 * i][x], o[nt][2 * i][x + 2], o[nt][2 * i + 1][x],
                                          o[nt][2 * i + 1][x + 2]);  // spread over the banks
          if (r == 0) sh->ml[warp][which][row] = make_float2(m[nt][x], l[nt][x]);
        }
    }
  }
  if (fetch.dead) {
    // the block's shared memory lives until the copies under way have landed
    volatile int keep_waiting = 0;
    mbar_wait(&sh->full[warp][0], fetch.last_keys(n) & 1, &keep_waiting, 1ull << 28);
    mbar_wait(&sh->full[warp][1], fetch.last_values() & 1, &keep_waiting, 1ull << 28);
  }
  __syncthreads();

  // ---- join the CTA's pieces: a lane for each, those of a unit follow one another; one warp per (unit, row)
  static_assert(2 * C::WARPS <= 32, "a lane for each piece");
  const int my_unit = lane < 2 * C::WARPS ? sh->unit[lane] : -1;
  const uint32_t used = __ballot_sync(0xFFFFFFFFu, my_unit >= 0);
  int item = 0;
  for (uint32_t left = used; left;) {
    const int first = __ffs(left) - 1, ui = __shfl_sync(0xFFFFFFFFu, my_unit, first);
    const uint32_t of = __ballot_sync(0xFFFFFFFFu, my_unit == ui) & used;
    left &= ~of;
    const int fin = 31 - __clz(of);
    const Kv4Unit u = range.at(ui);
    const bool begins = sh->begins[first], whole = begins && sh->ends[fin];
    for (int row = 0; row < u.rows; ++row, ++item) {
      if (item % C::WARPS != warp) continue;
      const bool on = of >> lane & 1u;
      const float2 x = on ? sh->ml[lane >> 1][lane & 1][row] : make_float2(kKv4Low, 0.f);
      float mm = x.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, d));
      const float a = ex2_approx(x.x - mm);
      float ll = x.y * a;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, d);
      float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = first; i <= fin; ++i) {
        if (!(of >> i & 1u)) continue;
        const float f = __shfl_sync(0xFFFFFFFFu, a, i);
        const float* from = reinterpret_cast<const float*>(i & 1 ? sh->ring[i >> 1] : sh->piece[i >> 1]);
        const float4 v = reinterpret_cast<const float4*>(from + row * kHeadDim)[lane ^ (lane >> 2 & 3)];
        oo.x = fmaf(v.x, f, oo.x);
        oo.y = fmaf(v.y, f, oo.y);
        oo.z = fmaf(v.z, f, oo.z);
        oo.w = fmaf(v.w, f, oo.w);
      }
      if (whole) {
        kv4_write_row(p, u, row, lane, mm, ll, oo);
      } else {
        float* part = p.part + (int64_t)(2 * cta + (begins ? 1 : 0)) * (R * 130);
        reinterpret_cast<float4*>(part + row * kHeadDim)[lane] = oo;
        if (lane == 0) *reinterpret_cast<float2*>(part + R * kHeadDim + 2 * row) = make_float2(mm, ll);
      }
    }
  }
}

// ------------------------------------------------------------------ join

constexpr int kKv4JoinThreads = 128;

// SPLIT warps per (unit, row) whose tiles lie in more than one CTA's range: each
// takes every SPLIT-th partial result, all at once (a loop that carries the
// maximum along waits for each in turn: 38 us for 64 of them against 4), and the
// sums meet in a fixed order. Rows without keys get their zero here. With one
// warp a row (few partial results each), 2048 rows of 8 kv heads over 32K tokens
// take 16 us for 28 MB, with four 29; whole calls of 4 rows of each of 8 kv heads
// over 128K tokens (some 19 results each) 50 us with one, 47.6 with four.
template <int SPLIT>
__global__ void __launch_bounds__(kKv4JoinThreads) kv4_join_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  __shared__ float s_l[SPLIT];
  __shared__ float4 s_o[SPLIT][32];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % SPLIT;
  const int item = blockIdx.x * (kKv4JoinThreads / 32 / SPLIT) + (threadIdx.x >> 5) / SPLIT;
  const int ui = item / p.R, row = item % p.R;
  const Kv4Unit u = p.units[ui];
  if (row >= u.rows) return;
  int c0 = 0, c1 = -1;
  if (u.tiles) {
    const int all = p.before[p.slots * p.Hkv], x = p.before[ui];
    const int per_cta = kv4_quota(p, all);
    c0 = x / per_cta;
    c1 = (x + kv4_items(p, u) - 1) / per_cta;
    if (c0 == c1) return;  // written by the CTA itself
  }
  const int64_t per = p.R * 130;
  auto part = [&](int c) { return p.part + (2 * c + (c == c0 ? 1 : 0)) * per; };
  auto ml = [&](int c) { return __ldcg(reinterpret_cast<const float2*>(part(c) + p.R * kHeadDim) + row); };
  float mm = kKv4Low;
  for (int c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, ml(c).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, d));
  float ll = 0.f;
  float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int c = c0 + warp; c <= c1; c += SPLIT) {
    const float2 x = ml(c);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(part(c) + row * kHeadDim) + lane);
    const float e = ex2_approx(x.x - mm);
    ll = fmaf(x.y, e, ll);
    oo.x = fmaf(v.x, e, oo.x);
    oo.y = fmaf(v.y, e, oo.y);
    oo.z = fmaf(v.z, e, oo.z);
    oo.w = fmaf(v.w, e, oo.w);
  }
  if constexpr (SPLIT > 1) {
    s_o[warp][lane] = oo;
    if (lane == 0) s_l[warp] = ll;
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < SPLIT; ++w) {
      const float4 v = s_o[w][lane];
      ll += s_l[w];
      oo.x += v.x;
      oo.y += v.y;
      oo.z += v.z;
      oo.w += v.w;
    }
  }
  kv4_write_row(p, u, row, lane, mm, ll, oo);
}

// ------------------------------------------------------------------ accumulated weights

// log2 of a row's sum, for its weights 2^(score - this). It comes from lse, a number of fp32, and is off by up to 3.5
// half units of its last place, of which a large one is coarse: so that no weight exceeds one, those are taken 4 whole
// ones higher (2^-21 of them; below 2^16 that would be at most 2^-5, and the scores' own error is larger). A row without
// keys has scores of minus infinity alone. One that is not finite has no sum: 0 leaves its scores as they are, not
// finite, and those that are masked at minus infinity.
__device__ __forceinline__ float kv4_log2_sum(float lse) {
  const float x = lse * 1.4426950408889634f;
  return !(fabsf(x) < INFINITY) ? 0.f : fabsf(x) < 65536.f ? x : fmaf(fabsf(x), 4.76837158203125e-07f, x);
}

constexpr int kKv4WeightThreads = 128, kKv4WeightTiles = 8;

// acc[key] += sum over the rows of the kv head of 2^(score - lse), one warp per
// 64-token tile; all rows of the sequence pass by, eight at a time, in order.
// HOLD: the keys are widened once and held in registers (many rows, two CTAs
// of four warps per SM), else widened for each eight rows, and a warp goes
// through kKv4WeightTiles tiles, with the rows' fragments kept where there are
// at most eight rows (few rows: what counts is how many warps have loads under
// way, and what a tile costs beside them; taken only where their scores would
// fill more scratch than kv4_seen_kernel may have).
template <bool HOLD>
__global__ void __launch_bounds__(kKv4WeightThreads, HOLD ? 2 : 5) kv4_weight_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  constexpr int TILES = HOLD ? 1 : kKv4WeightTiles, WARPS = kKv4WeightThreads / 32;
  const int lane = threadIdx.x & 31, r = lane >> 2, qd = lane & 3;
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  int t0;
  const int n = kv4_queries(p, p.cu, b, &t0);
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int pos0 = len - n, rows = n * p.G;
  const int64_t tile0 = (int64_t)blockIdx.x * (WARPS * TILES) + (threadIdx.x >> 5);
  if (n == 0 || tile0 * kKv4Tile >= len) return;
  const int slot0 = kv4_first_slot(p, b, t0);
  const uint8_t* kt0 = p.kv4 + kv4_tile_off(p.tiles, p.Hkv, b, h, 0);
  float* acc0 = p.acc + ((int64_t)b * p.Hkv + h) * p.tiles * kKv4Tile;

  // eight rows: fragments, and of this lane's two scale, log2 of the sum and position
  uint32_t qf[16];
  float qs[2], le[2];
  int pos[2];
  auto rows8 = [&](int r0) {
    const int rr = r0 + r;
    const __nv_bfloat16* row =
        rr < rows ? p.q + ((int64_t)(t0 + rr / p.G) * p.Hq + h * p.G + rr % p.G) * kHeadDim + qd * 32 : nullptr;
    const float s = kv4_query_fragment(row, p.scale_log2, qf);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      qs[x] = __shfl_sync(0xFFFFFFFFu, s, (2 * qd + x) * 4);
      const int row2 = r0 + 2 * qd + x;
      const bool on = row2 < rows;
      pos[x] = on ? pos0 + row2 / p.G : -1;
      le[x] = on ? kv4_log2_sum(p.lse[(int64_t)(h * p.G + row2 % p.G) * p.total + t0 + row2 / p.G]) : 0.f;
    }
  };
  const bool one = rows <= 8;
  if (one) rows8(0);

#pragma unroll 1
  for (int i = 0; i < TILES; ++i) {
    const int64_t tile = tile0 + i * WARPS;
    const int key0 = (int)(tile * kKv4Tile);
    if (key0 >= len) break;
    const int block = key0 / p.B;
    auto picked = [&](int row) {
      if (!p.kmean) return 0xFFu;
      const int64_t ui = (int64_t)(slot0 + (row >> p.rshift)) * p.Hkv + h;
      return __ldg(p.chosen + ui * p.blocks + block) >> (row & (p.R - 1)) & 0xFFu;
    };
    // rows before the first key's position attend nothing here
    int r0 = key0 > pos0 ? (int)((int64_t)(key0 - pos0) * p.G / 8 * 8) : 0;
    while (r0 < rows && !picked(r0)) r0 += 8;
    if (r0 >= rows) continue;
    const uint8_t* kt = kt0 + tile * kKv4TileBytes;
    float* acc = acc0 + key0;
    uint4 wa[4], wb[4];
    uint32_t pa[4], pb[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int ta = g * 16 + r, tb = ta + 8;
      wa[g] = __ldg(reinterpret_cast<const uint4*>(kt + ta * kKv4Row + qd * 16));
      wb[g] = __ldg(reinterpret_cast<const uint4*>(kt + tb * kKv4Row + qd * 16));
      pa[g] = __ldg(reinterpret_cast<const uint16_t*>(kt + kKv4Params + ta * 8 + qd * 2));
      pb[g] = __ldg(reinterpret_cast<const uint16_t*>(kt + kKv4Params + tb * 8 + qd * 2));
    }
    // lane 4 r + x: the keys r + 16 x and r + 16 x + 8
    const float old0 = acc[16 * qd + r], old1 = acc[16 * qd + r + 8];
    auto widen = [&](int g, int w, const Kv4Par& fa, const Kv4Par& fb, uint32_t (&y)[4], uint32_t (&z)[4]) {
      const uint32_t xa[4] = {wa[g].x, wa[g].y, wa[g].z, wa[g].w}, xb[4] = {wb[g].x, wb[g].y, wb[g].z, wb[g].w};
      kv4_pairs(xa[w], fa, y);
      kv4_pairs(xb[w], fb, z);
    };
    uint32_t a[HOLD ? 4 : 1][4][8];  // [16 keys][word][pair of the first, of the second eight keys]
    if constexpr (HOLD) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const Kv4Par fa = kv4_par(__byte_perm(pa[g], 0, 0x1010)), fb = kv4_par(__byte_perm(pb[g], 0, 0x1010));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t y[4], z[4];
          widen(g, w, fa, fb, y, z);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[g][w][2 * j] = y[j], a[g][w][2 * j + 1] = z[j];
        }
      }
    }
    float sum[4][2] = {};
    for (; r0 < rows; r0 += 8) {
      const uint32_t pick = picked(r0);
      if (!pick) continue;
      if (!one) rows8(r0);
      int last[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) last[x] = pick >> (2 * qd + x) & 1u ? pos[x] : -1;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float sc[4];
        const Kv4Par fa = kv4_par(__byte_perm(pa[g], 0, 0x1010)), fb = kv4_par(__byte_perm(pb[g], 0, 0x1010));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t y[4], z[4];
          if constexpr (HOLD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = a[g][w][2 * j], z[j] = a[g][w][2 * j + 1];
          } else {
            widen(g, w, fa, fb, y, z);
          }
          if (w == 0) mma_f16_first(sc, y[0], z[0], y[1], z[1], qf[0], qf[1]);
          else mma_f16(sc, y[0], z[0], y[1], z[1], qf[4 * w], qf[4 * w + 1]);
          mma_f16(sc, y[2], z[2], y[3], z[3], qf[4 * w + 2], qf[4 * w + 3]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = key0 + g * 16 + r + (x >> 1) * 8;
          const float e = ex2_approx(fmaf(sc[x], qs[x & 1], -le[x & 1]));
          if (key <= last[x & 1]) sum[g][x >> 1] += e;
        }
      }
    }
    // the four lanes of a key add up; lane qd keeps the keys of 16 qd
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = sum[g][x];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        if (g == qd) (x ? v1 : v0) = v;
      }
    const int at = 16 * qd + r;
    if (key0 + at < len) acc[at] = old0 + v0;
    if (key0 + at + 8 < len) acc[at + 8] = old1 + v1;
  }
}

constexpr int kKv4SeenThreads = 128, kKv4SeenKeys = 1024;

// The same from the scores that the attention has left: 4 bytes written and
// read a row and key, against 72 read again and widened a key. Whole calls: 128K
// tokens of 8 heads, 4 rows each, 68 us against 79; 8 such sequences of 12 chosen
// blocks 242 against 297. A warp takes 256 keys of a kv head, a lane a key, over
// the units of the sequence in order, 128 keys' scores under way at once (which
// brought those calls to 59 and 204).
__global__ void __launch_bounds__(kKv4SeenThreads) kv4_seen_kernel(Kv4AttnParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  const int first = blockIdx.x * kKv4SeenKeys + (threadIdx.x >> 5) * (kKv4SeenKeys / (kKv4SeenThreads / 32));
  int t0;
  const int n = kv4_queries(p, p.cu, b, &t0);
  if (n == 0 || first >= len) return;
  constexpr int PARTS = kKv4SeenKeys / (kKv4SeenThreads / 32) / 32;
  float sum[PARTS] = {};
  uint32_t touched = 0;  // parts that a unit attends
  const int slot0 = kv4_first_slot(p, b, t0), tpb = p.B / kKv4Tile;
  for (int row0 = 0; row0 < n * p.G; row0 += p.R) {
    const int ui = (slot0 + (row0 >> p.rshift)) * p.Hkv + h;
    const Kv4Unit u = p.units[ui];
    if (u.tiles == 0) continue;
    const int before = p.before[ui];
    float le[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int rr = u.row0 + r;
      le[r] = r < u.rows ? kv4_log2_sum(p.lse[(int64_t)(h * p.G + rr % p.G) * p.total + u.t0 + rr / p.G]) : 0.f;
    }
    int block = -1, at = -1;  // the block that was looked up, and its place in the list
#pragma unroll
    for (int i0 = 0; i0 < PARTS; i0 += 4) {  // 128 keys: two tiles of one block
      const int key0 = first + i0 * 32;
      int tile = key0 / kKv4Tile;
      if (key0 >= len) break;
      if (p.kmean) {
        if (tile / tpb != block) {
          block = tile / tpb;
          at = -1;
          for (int e = lane; e < u.blocks; e += 32)
            if ((int)p.list[(int64_t)ui * p.list_cap + e].x == block) at = e;
          at = __reduce_max_sync(0xFFFFFFFFu, at);
        }
        if (at < 0) continue;
        tile = at * tpb + tile % tpb;
      }
      if (tile >= u.tiles) continue;
      touched |= 1u << i0;
      const float2* from = reinterpret_cast<const float2*>(p.seen) + (int64_t)(before + tile) * 4 * kKv4Tile + lane;
      float2 z[4][4];  // all under way at once
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          z[i][r] = 2 * r < u.rows && tile + i / 2 < u.tiles
                        ? __ldcs(from + (i / 2 * 4 + r) * kKv4Tile + i % 2 * 32)
                        : make_float2(-INFINITY, -INFINITY);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (2 * r >= u.rows) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i0 + i] += ex2_approx(z[i][r].x - le[2 * r]);
          if (2 * r + 1 < u.rows) sum[i0 + i] += ex2_approx(z[i][r].y - le[2 * r + 1]);
        }
      }
    }
  }
  float* acc = p.acc + ((int64_t)b * p.Hkv + h) * p.tiles * kKv4Tile + first + lane;
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
    if (touched >> (i & ~3) & 1u && first + i * 32 + lane < len) acc[i * 32] += sum[i];
}

// ------------------------------------------------------------------ pool

struct Kv4PoolParams {
  const uint8_t* kv4;
  const int32_t* lengths;
  int64_t tiles;
  int heads, B, blocks;  // blocks = capacity / B
  int per;               // blocks of a CTA: several where they are small
  int stages;            // of a warp's ring: kKv4PoolStages, or its tiles where these are fewer
  float* kmean;          // [batch][heads][blocks][128]
};

constexpr int kKv4PoolThreads = 256, kKv4PoolStages = 3;

// A cluster of CTAs per (block, head, sequence), a part of the block's tiles
// each, or a CTA for two or four small blocks; each warp brings its tiles of keys
// into a ring of its own, one bulk copy each, two ahead. HBM-bound where the
// kernel is not short: 1M tokens of 8 heads in blocks of 4096 98 us, 6.2 TB/s;
// 128K tokens 18 a call (27 with loads into registers, two groups of tokens a
// warp); 64 sequences of 16K, 8 heads, blocks of 128 171 us, 3.5 TB/s (a CTA per
// block 308, and 516 with room for three tiles a warp, so two CTAs an SM).
// The tensor core sums in fp32: codes, as they stand in a word, are fp16
// subnormals (a nibble at bit 0 is c 2^-24, at bit 4 c 2^-20), so a mask is all
// that they need; they meet the scales of the four groups in four columns, of
// which the channel's own is kept, and the scales times zero points are summed
// by one product more and taken off at the end. The warps' and CTAs' sums meet
// in a fixed order. Blocks that the sequence has not completed are written as
// zero.
__global__ void __launch_bounds__(kKv4PoolThreads, 3) kv4_pool_kernel(Kv4PoolParams p) {
  grid_dependency_sync();
  constexpr int MOST = kKv4PoolThreads / 32;
  const int WARPS = blockDim.x / 32;
  extern __shared__ __align__(16) uint8_t pool_ring[];  // [WARPS][stages][kKv4Half]
  __shared__ float sums[MOST][kHeadDim];
  __shared__ uint32_t total[kHeadDim];  // fp32 bits
  __shared__ uint64_t full[MOST][kKv4PoolStages];
  __shared__ int abort_flag;
  uint32_t rank, csize;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, qd = lane & 3;
  const int wpb = WARPS / p.per, j0 = blockIdx.x / csize * p.per, j = j0 + warp / wpb;  // warps of a block, first block
  const int len = kv4_length(p.lengths, b, p.tiles * kKv4Tile);
  float* out = p.kmean + (((int64_t)b * p.heads + h) * p.blocks + j0) * kHeadDim;
  const int outs = min(p.per, p.blocks - j0) * kHeadDim;
  if ((int64_t)(j0 + 1) * p.B > len) {  // no complete block: the whole cluster leaves
    for (int i = threadIdx.x; rank == 0 && i < outs; i += blockDim.x) out[i] = 0.f;
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < MOST * kKv4PoolStages; ++i) mbar_init(&full[0][0] + i, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int tiles = p.B / kKv4Tile, step = csize * wpb, t0 = rank * wpb + warp % wpb;
  // tiles of this warp; none of a block that is not complete, whose sums stay zero
  const int n = t0 < tiles && (int64_t)(j + 1) * p.B <= len ? (tiles - t0 + step - 1) / step : 0;
  const uint8_t* src = p.kv4 + kv4_tile_off(p.tiles, p.heads, b, h, (int64_t)j * tiles + t0);
  uint8_t* ring = pool_ring + warp * p.stages * kKv4Half;
  auto issue = [&](int k) {
    if (k >= n || lane != 0) return;
    const int d = k % kKv4PoolStages;
    mbar_arrive_expect_tx(&full[warp][d], kKv4Half);
    bulk_load(ring + d * kKv4Half, src + (int64_t)k * step * kKv4TileBytes, kKv4Half, &full[warp][d]);
  };
  issue(0);
  issue(1);
  float o[8][4] = {}, oz[4] = {};
  for (int k = 0; k < n; ++k) {
    issue(k + 2);
    const int d = k % kKv4PoolStages;
    if (!mbar_wait(&full[warp][d], (k / kKv4PoolStages) & 1, &abort_flag)) {
      // the block's shared memory lives until the copies under way have landed
      volatile int keep_waiting = 0;
      for (int i = k; i < min(n, k + 3); ++i)
        mbar_wait(&full[warp][i % kKv4PoolStages], (i / kKv4PoolStages) & 1, &keep_waiting, 1ull << 28);
      break;
    }
    const uint8_t* tile = ring + d * kKv4Half;
#pragma unroll
    for (int g = 0; g < kKv4Tile / 16; ++g) {
      uint2 w[2][2];
      uint32_t s[2], sz[2];  // scales, and scales times zero points, of group r % 4 for the lane's tokens
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t pp[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = g * 16 + 8 * f + 2 * qd + (e ^ (qd & 1));
          w[f][e] = *reinterpret_cast<const uint2*>(tile + tok * kKv4Row + r * 8);
          pp[e] = *reinterpret_cast<const uint16_t*>(tile + kKv4Params + tok * 8 + (r & 3) * 2);
        }
        const uint32_t par = __byte_perm(pp[0], pp[1], 0x5410);
        s[f] = par & 0x7F807F80u;
        sz[f] = h2_mul(h2_sub(and_or(par, 0x000F000Fu, 0x64006400u), 0x64006400u), s[f]);
      }
      mma_f16(oz, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, sz[0], sz[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t a[2][2][4];  // [channel parity][tokens 0-7, 8-15][nibble]
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t x0 = x ? w[f][0].y : w[f][0].x, x1 = x ? w[f][1].y : w[f][1].x;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t u = __byte_perm(x0, x1, c ? 0x7632 : 0x5410), v = u >> 8;
            a[c][f][0] = u & 0x000F000Fu;
            a[c][f][1] = u & 0x00F000F0u;
            a[c][f][2] = v & 0x000F000Fu;
            a[c][f][3] = v & 0x00F000F0u;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16(o[x * 4 + i], a[0][0][i], a[1][0][i], a[0][1][i], a[1][1][i], s[0], s[1]);
      }
    }
    __syncwarp();  // the tile is read: the one after next may take its place
  }
  // channels 16 r .. are of group r / 2: the lane that holds this column has their sums
  if (qd == r >> 2) {
    const int c = r >> 1 & 1;
    const float z = c ? oz[1] : oz[0];
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      const float unit = mt & 1 ? 1048576.f : 16777216.f;  // 2^20, 2^24
      sums[warp][16 * r + 2 * mt] = fmaf(c ? o[mt][1] : o[mt][0], unit, -z);
      sums[warp][16 * r + 2 * mt + 1] = fmaf(c ? o[mt][3] : o[mt][2], unit, -z);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < outs; i += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < wpb; ++w) s += sums[i / kHeadDim * wpb + w][i % kHeadDim];
    if (csize == 1) out[i] = s / (float)p.B;
    else total[i] = __float_as_uint(s);  // one block
  }
  if (csize == 1) return;
  kv4_cluster_sync();
  if (rank == 0 && threadIdx.x < kHeadDim) {
    float s = 0.f;
    for (uint32_t c = 0; c < csize; ++c) s += __uint_as_float(kv4_remote_ld(&total[threadIdx.x], c));
    out[threadIdx.x] = s / (float)p.B;
  }
  kv4_cluster_sync();  // no CTA leaves while its sums may still be read
}

}  // namespace moba
