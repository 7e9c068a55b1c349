// Entry points of the 4-bit key/value cache (kv4.cuh, kv4_attn.cuh): argument
// checks, scratch and launches. Included at the end of moba.cu, whose helpers
// (fail, device_info, direct_run, launch_chained, ...) it uses.
#pragma once

#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "kv4_chunk.cuh"

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Shape of a cache: `capacity` tokens a sequence, in whole tiles.
int check_cache(int batch, int heads, int d, int64_t capacity) {
  if (batch < 1) return fail(MOBA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", batch);
  if (heads < 1) return fail(MOBA_ERR_INVALID_ARG, "heads_kv must be >= 1 (got %d)", heads);
  if (d != MOBA_HEAD_DIM) return fail(MOBA_ERR_INVALID_ARG, "head_dim must be %d (got %d)", MOBA_HEAD_DIM, d);
  if (capacity < 1 || capacity % MOBA_KV4_TILE)
    return fail(MOBA_ERR_INVALID_ARG, "capacity must be a positive multiple of %d (got %lld)", MOBA_KV4_TILE,
                (long long)capacity);
  if (capacity > ((int64_t)1 << 30)) return fail(MOBA_ERR_UNSUPPORTED, "capacity above 2^30 tokens is not supported");
  if ((int64_t)batch * heads > 65535)
    return fail(MOBA_ERR_UNSUPPORTED, "more than 65535 (sequence, kv head) pairs are not supported");
  return MOBA_OK;
}

size_t cache_bytes(int batch, int heads, int64_t capacity) {
  return (size_t)batch * heads * (capacity / moba::kKv4Tile) * moba::kKv4TileBytes;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// As launch_chained, with the grid in clusters of `csize` CTAs along x.
template <typename... KArgs, typename... Args>
void launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int csize, cudaStream_t st,
                     Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class C>
constexpr size_t kv4_attn_smem() {
  return sizeof(typename C::Shared);
}

template <class C>
void launch_kv4_attn(const moba::Kv4AttnParams& p, cudaStream_t st) {
  launch_chained(moba::kv4_attn_kernel<C>, dim3(p.ctas), dim3(C::THREADS), kv4_attn_smem<C>(), st, p);
}

template <class C>
cudaError_t set_kv4_attn_smem() {
  return cudaFuncSetAttribute(moba::kv4_attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kv4_attn_smem<C>());
}

template <bool MASKED>
cudaError_t set_kv4_chunk_smem() {
  const cudaError_t e = cudaFuncSetAttribute(moba::kv4_chunk_kernel<MASKED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             moba::kKv4ChunkSmemBytes);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(moba::kv4_chunk_weight_kernel<MASKED>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, moba::kKv4ColSmemBytes);
}

// Rows of a sequence and kv head, on average, above which the tcgen05 kernel
// (256 rows a unit) takes over from mma.sync (16 rows a unit, every key widened
// for each of them): one kernel for all sequences of a call, since the host
// does not know the offsets. At 32K tokens, 32 / 8 heads, one sequence: 32 rows 43
// against 44 us, 64 rows 45 against 65, 2048 rows 293 against 1430; 16
// sequences of 8K: 16 rows 162 against 70, 64 rows 173 against 219.
constexpr int kKv4ManyRows = 48;

// With a gate the tcgen05 kernel goes over all keys and masks, where mma.sync goes over the blocks that its 16 rows
// chose, at most 16 topk blocks, at some four times the cost a row and key. So the former takes over where those are a
// third of the cache: of its capacity, since the host does not know the lengths (a short sequence in a large cache is
// left to mma.sync). 512 tokens of 32 / 8 heads: at 32K tokens, block 512, top-12 (all of it) 487
// against 1306 us; at 128K, block 4096, top-12 1372 against 4949; at 128K, block 128, top-12 (a fifth) 2777 against
// 2101, and each pick more costs 36 against 95.
constexpr int kKv4Union = 3 * moba::Kv4Many::R;

// Bytes of scores that few rows may leave in scratch for their weights. MOBA_TEST_KEPT_SCORES=<n> sets another limit: a
// test hook that reaches the kernel behind it without a large cache.
size_t kept_scores_limit() {
  const char* e = getenv("MOBA_TEST_KEPT_SCORES");
  return e ? (size_t)strtoull(e, nullptr, 10) : (size_t)1 << 30;
}

bool g_kv4_ready[64] = {};

// The device, and an error that an earlier call's kernels left behind.
int kv4_begin(DeviceInfo* dev, cudaStream_t st) {
  int rc = device_info(dev);
  if (rc) return rc;
  int d = 0;
  MOBA_CUDA(cudaGetDevice(&d));
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!g_kv4_ready[d]) {
      MOBA_CUDA(set_kv4_attn_smem<moba::Kv4Few>());
      MOBA_CUDA(set_kv4_attn_smem<moba::Kv4Many>());
      MOBA_CUDA(set_kv4_chunk_smem<false>());
      MOBA_CUDA(set_kv4_chunk_smem<true>());
      MOBA_CUDA(cudaFuncSetAttribute(moba::kv4_pool_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     moba::kKv4PoolThreads / 32 * moba::kKv4PoolStages * moba::kKv4Half));
      MOBA_CUDA(cudaFuncSetAttribute(moba::kv4_gate_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     MOBA_KV4_MAX_BLOCKS * 4 + 4));
      g_kv4_ready[d] = true;
    }
  }
  return take_pending_status(*dev, st);
}

}  // namespace

extern "C" {

int moba_kv4_append(const void* k, const void* v, int64_t total, const int32_t* cu, const int32_t* start, int batch,
                    int heads_kv, int head_dim, int64_t capacity, void* kv4, float* acc, cudaStream_t stream) {
  g_err.clear();
  if (!k || !v || !start || !kv4) return fail(MOBA_ERR_INVALID_ARG, "null pointer argument");
  int rc = check_cache(batch, heads_kv, head_dim, capacity);
  if (rc) return rc;
  if (total < 0 || total > INT32_MAX) return fail(MOBA_ERR_INVALID_ARG, "total must be in [0, 2^31)");
  if (!cu && total % batch) return fail(MOBA_ERR_INVALID_ARG, "without cu, total must be a multiple of batch");
  if (!aligned16(k) || !aligned16(v) || !aligned16(kv4))
    return fail(MOBA_ERR_INVALID_ARG, "k, v and kv4 must be 16-byte aligned");
  if (!aligned4(cu) || !aligned4(start) || !aligned4(acc))
    return fail(MOBA_ERR_INVALID_ARG, "cu, start and acc must be 4-byte aligned");
  DeviceInfo dev;
  rc = kv4_begin(&dev, stream);
  if (rc) return rc;
  if (total == 0) return finish_call(MOBA_OK, stream);
  moba::Kv4AppendParams p;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.cu = cu;
  p.start = start;
  p.total = total;
  p.tiles = capacity / moba::kKv4Tile;
  p.batch = batch;
  p.heads = heads_kv;
  p.kv4 = static_cast<uint8_t*>(kv4);
  p.acc = acc;
  const int per = moba::kKv4AppendThreads / 4;
  launch_chained(moba::kv4_append_kernel, dim3((unsigned)((total + per - 1) / per), heads_kv),
                 dim3(moba::kKv4AppendThreads), 0, stream, p);
  MOBA_CUDA(cudaGetLastError());
  return finish_call(MOBA_OK, stream);
}

int moba_kv4_load(const void* kv4, const int32_t* lengths, const int32_t* first, int batch, int heads_kv, int head_dim,
                  int64_t capacity, int64_t n, void* k, void* v, cudaStream_t stream) {
  g_err.clear();
  if (!kv4 || !lengths || !k || !v) return fail(MOBA_ERR_INVALID_ARG, "null pointer argument");
  int rc = check_cache(batch, heads_kv, head_dim, capacity);
  if (rc) return rc;
  if (n < 0 || n > capacity) return fail(MOBA_ERR_INVALID_ARG, "n must be in [0, capacity]");
  if (!aligned16(k) || !aligned16(v) || !aligned16(kv4))
    return fail(MOBA_ERR_INVALID_ARG, "k, v and kv4 must be 16-byte aligned");
  if (!aligned4(lengths) || !aligned4(first))
    return fail(MOBA_ERR_INVALID_ARG, "lengths and first must be 4-byte aligned");
  DeviceInfo dev;
  rc = kv4_begin(&dev, stream);
  if (rc) return rc;
  if (n == 0) return finish_call(MOBA_OK, stream);
  moba::Kv4LoadParams p;
  p.kv4 = static_cast<const uint8_t*>(kv4);
  p.lengths = lengths;
  p.first = first;
  p.tiles = capacity / moba::kKv4Tile;
  p.n = n;
  p.batch = batch;
  p.heads = heads_kv;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  const int per = moba::kKv4LoadThreads / 16 * moba::kKv4LoadRows;
  launch_chained(moba::kv4_load_kernel, dim3((unsigned)((n + per - 1) / per), heads_kv, batch),
                 dim3(moba::kKv4LoadThreads), 0, stream, p);
  MOBA_CUDA(cudaGetLastError());
  return finish_call(MOBA_OK, stream);
}

int moba_kv4_pool(const void* kv4, const int32_t* lengths, int batch, int heads_kv, int head_dim, int64_t capacity,
                  int block_size, float* kmean, cudaStream_t stream) {
  g_err.clear();
  if (!kv4 || !lengths || !kmean) return fail(MOBA_ERR_INVALID_ARG, "null pointer argument");
  int rc = check_cache(batch, heads_kv, head_dim, capacity);
  if (rc) return rc;
  rc = check_shape(capacity, heads_kv, heads_kv, head_dim, block_size, 1);
  if (rc) return rc;
  if (!aligned16(kv4) || !aligned16(kmean)) return fail(MOBA_ERR_INVALID_ARG, "kv4 and kmean must be 16-byte aligned");
  if (!aligned4(lengths)) return fail(MOBA_ERR_INVALID_ARG, "lengths must be 4-byte aligned");
  DeviceInfo dev;
  rc = kv4_begin(&dev, stream);
  if (rc) return rc;
  moba::Kv4PoolParams p;
  p.kv4 = static_cast<const uint8_t*>(kv4);
  p.lengths = lengths;
  p.tiles = capacity / moba::kKv4Tile;
  p.heads = heads_kv;
  p.B = block_size;
  p.blocks = (int)(capacity / block_size);
  p.kmean = kmean;
  if (p.blocks) {
    // a warp for 64 tokens, up to 8 of them, which are several blocks' where a block has two or four; up to 8 CTAs
    // share a large block while there are SMs for them
    const int most = moba::kKv4PoolThreads / 32, wpb = std::min(most, block_size / moba::kKv4Tile);
    p.per = most / wpb;
    const int threads = wpb * p.per * 32;
    int csize = 1;
    while (csize < 8 && (int64_t)p.blocks * heads_kv * batch * csize * 2 <= 2 * dev.sms && block_size / csize > 1024)
      csize *= 2;
    p.stages = std::min(moba::kKv4PoolStages, (block_size / moba::kKv4Tile + wpb * csize - 1) / (wpb * csize));
    const size_t ring = (size_t)threads / 32 * p.stages * moba::kKv4Half;
    if ((int64_t)p.blocks * csize > INT32_MAX) return fail(MOBA_ERR_UNSUPPORTED, "too many blocks");
    launch_clusters(moba::kv4_pool_kernel, dim3((p.blocks + p.per - 1) / p.per * csize, heads_kv, batch), dim3(threads),
                    ring, csize, stream, p);
    MOBA_CUDA(cudaGetLastError());
  }
  return finish_call(MOBA_OK, stream);
}

int moba_kv4_attend(const void* q, int64_t total, const int32_t* cu, const void* kv4, const int32_t* lengths,
                    const float* kmean, int batch, int heads_q, int heads_kv, int head_dim, int64_t capacity,
                    int block_size, int topk, float* acc, void* out, float* lse, cudaStream_t stream) {
  g_err.clear();
  if (!q || !kv4 || !lengths || !out || !lse) return fail(MOBA_ERR_INVALID_ARG, "null pointer argument");
  int rc = check_cache(batch, heads_kv, head_dim, capacity);
  if (rc) return rc;
  if (heads_q < 1 || heads_q % heads_kv)
    return fail(MOBA_ERR_INVALID_ARG, "heads_q (%d) must be a positive multiple of heads_kv (%d)", heads_q, heads_kv);
  if (total < 0 || total > INT32_MAX / heads_q) return fail(MOBA_ERR_INVALID_ARG, "total * heads_q must be in [0, 2^31)");
  if (!cu && total % batch) return fail(MOBA_ERR_INVALID_ARG, "without cu, total must be a multiple of batch");
  if (kmean) {
    rc = check_shape(capacity, heads_q, heads_kv, head_dim, block_size, topk);
    if (rc) return rc;
    if (capacity / block_size > MOBA_KV4_MAX_BLOCKS)
      return fail(MOBA_ERR_UNSUPPORTED, "more than %d blocks in the capacity are not supported", MOBA_KV4_MAX_BLOCKS);
    // at least as many picks as blocks: every key
    if (topk >= (capacity + block_size - 1) / block_size) kmean = nullptr;
  }
  if (!aligned16(q) || !aligned16(kv4) || !aligned16(kmean) || !aligned16(out))
    return fail(MOBA_ERR_INVALID_ARG, "q, kv4, kmean and out must be 16-byte aligned");
  if (!aligned4(cu) || !aligned4(lengths) || !aligned4(acc) || !aligned4(lse))
    return fail(MOBA_ERR_INVALID_ARG, "cu, lengths, acc and lse must be 4-byte aligned");
  DeviceInfo dev;
  rc = kv4_begin(&dev, stream);
  if (rc) return rc;
  if (total == 0) return finish_call(MOBA_OK, stream);
  moba::Kv4AttnParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv4 = static_cast<const uint8_t*>(kv4);
  p.lengths = lengths;
  p.cu = cu;
  p.kmean = kmean;
  p.total = total;
  p.tiles = capacity / moba::kKv4Tile;
  p.batch = batch;
  p.Hq = heads_q;
  p.Hkv = heads_kv;
  p.G = heads_q / heads_kv;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)moba::kHeadDim));
  p.acc = acc;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.B = kmean ? block_size : moba::kKv4Tile;
  p.topk = kmean ? topk : 0;
  p.means = kmean ? (int)(capacity / block_size) : 0;
  p.blocks = kmean ? (int)((capacity + block_size - 1) / block_size) : 0;
  p.each = cu ? 0 : (int)(total / batch);
  p.ctas = dev.sms;
  const bool few = total * p.G <= (int64_t)moba::Kv4Few::R * batch;
  const bool chunk = total * p.G > (int64_t)kKv4ManyRows * batch &&
                     (!kmean || (int64_t)kKv4Union * topk * block_size >= capacity);
  // many rows with a gate: it writes which blocks each row chose, the attention goes over all keys and masks
  const bool masked = chunk && kmean;
  moba::Kv4AttnParams gp = p;
  if (masked) {
    p.kmean = nullptr;
    p.B = moba::kKv4Tile;
    p.topk = p.means = p.blocks = 0;
    p.pick_B = block_size;
    p.pick_blocks = gp.blocks;
    kmean = nullptr;
  }
  const auto rows_of = [&](moba::Kv4AttnParams& x, int R) {
    x.R = R;
    while (1 << x.rshift < R) ++x.rshift;
    const int64_t slots = total * x.G / R + batch;
    if (slots * heads_kv * R > INT32_MAX) return false;
    x.slots = (int)slots;
    return true;
  };
  if (!rows_of(p, few ? moba::Kv4Few::R : chunk ? moba::kKv4ChunkRows : moba::Kv4Many::R) ||
      !rows_of(gp, masked ? 32 : p.R))
    return fail(MOBA_ERR_UNSUPPORTED, "too many rows");
  // a warp for each of an SM's four schedulers at least: 4096 tokens of one head take 12.1 us with 4 tiles a CTA (on 16
  // CTAs), 15.0 with 1, 13.0 with 2 and with 8, 16.3 with 16
  p.least = chunk ? 1 : 4;
  p.steps = chunk ? 1 : 0;
  const int64_t nu = (int64_t)p.slots * heads_kv, gnu = (int64_t)gp.slots * heads_kv;
  // items (tiles, or steps of two tiles) and the ends of all ranges are counted in 31 bits
  p.list_cap = kmean ? (int)std::min<int64_t>(p.blocks, (int64_t)p.R * topk) : 0;
  const int64_t items = kmean   ? std::min<int64_t>(p.tiles, (int64_t)p.list_cap * (block_size / moba::kKv4Tile))
                        : chunk ? (p.tiles + 1) / 2
                                : p.tiles;
  if (nu * items > ((int64_t)1 << 30))
    return fail(MOBA_ERR_UNSUPPORTED, "too many (query row, cached token) pairs for one call: attend in chunks");
  // the gate: up to 8 CTAs share a unit's scores while there are few units
  int csize = 1;
  while (csize < 8 && gnu * csize * 2 <= dev.sms) csize *= 2;
  const int64_t clusters = std::min<int64_t>(gnu, 4 * dev.sms / csize);
  Carve c;
  const size_t o_units = c.take((size_t)nu * sizeof(moba::Kv4Unit)), o_before = c.take((size_t)(nu + 1) * 4);
  const size_t o_list = c.take((size_t)nu * p.list_cap * 8);
  const size_t o_gunits = c.take(masked ? (size_t)gnu * sizeof(moba::Kv4Unit) : 0);
  const size_t o_chosen = c.take(gp.kmean && (acc || masked) ? (size_t)gnu * gp.blocks * 4 : 0);
  const size_t o_scores = c.take((size_t)clusters * gp.R * gp.means * 8);
  const size_t o_part = c.take((size_t)2 * p.ctas * p.R * 130 * 4);
  // the scores of few rows are kept for their weights, up to a GiB of them (sized by the capacity and by the unit slots,
  // which alone are known: up to two slots for a sequence's one unit)
  const size_t seen = few && acc ? (size_t)nu * items * 4 * moba::kKv4Tile * 8 : 0;
  const bool keep = seen > 0 && seen <= kept_scores_limit();
  const size_t o_seen = c.take(keep ? seen : 0);
  const size_t o_qtiles = c.take(chunk ? (size_t)nu * 2 * moba::kKv4TileOp : 0);
  const size_t o_qscale = c.take(chunk ? (size_t)nu * moba::kKv4ChunkRows * 4 : 0);
  const Runner run = [&](uint8_t* ws, cudaStream_t st) -> int {
    p.seen = keep ? reinterpret_cast<float*>(ws + o_seen) : nullptr;
    p.qtiles = ws + o_qtiles;
    p.qscale = reinterpret_cast<float*>(ws + o_qscale);
    p.units = reinterpret_cast<moba::Kv4Unit*>(ws + o_units);
    p.before = reinterpret_cast<int*>(ws + o_before);
    p.list = reinterpret_cast<uint2*>(ws + o_list);
    p.chosen = acc || masked ? reinterpret_cast<uint32_t*>(ws + o_chosen) : nullptr;
    p.picks = masked ? p.chosen : nullptr;
    p.scores = reinterpret_cast<double*>(ws + o_scores);
    p.part = reinterpret_cast<float*>(ws + o_part);
    if (gp.kmean) {
      gp.units = masked ? reinterpret_cast<moba::Kv4Unit*>(ws + o_gunits) : p.units;
      gp.list = p.list;
      gp.list_cap = p.list_cap;  // 0 where the attention masks
      gp.chosen = p.chosen;
      gp.scores = p.scores;
      launch_clusters(moba::kv4_gate_kernel, dim3((unsigned)(clusters * csize)), dim3(moba::kKv4GateThreads),
                      (size_t)gp.blocks * 4, csize, st, gp);
    }
    if (few) {
      launch_kv4_attn<moba::Kv4Few>(p, st);
    } else if (chunk) {
      launch_chained(moba::kv4_prep_kernel, dim3((unsigned)nu, moba::kKv4ChunkRows * 16 / moba::kKv4PrepThreads),
                     dim3(moba::kKv4PrepThreads), 0, st, p);
      launch_chained(masked ? moba::kv4_chunk_kernel<true> : moba::kv4_chunk_kernel<false>, dim3(p.ctas),
                     dim3(moba::kKv4ChunkThreads), moba::kKv4ChunkSmemBytes, st, p);
    } else {
      launch_kv4_attn<moba::Kv4Many>(p, st);
    }
    // a unit's partial results come from about ctas / nu CTAs and one or two at its ends
    constexpr int split = moba::kKv4JoinThreads / 32;
    if (nu * 4 < p.ctas)
      launch_chained(moba::kv4_join_kernel<split>, dim3((unsigned)(nu * p.R)), dim3(moba::kKv4JoinThreads), 0, st, p);
    else
      launch_chained(moba::kv4_join_kernel<1>, dim3((unsigned)(nu * p.R / split)), dim3(moba::kKv4JoinThreads), 0, st, p);
    if (acc && chunk) {
      launch_chained(masked ? moba::kv4_chunk_weight_kernel<true> : moba::kv4_chunk_weight_kernel<false>,
                     dim3((unsigned)((capacity + 255) / 256), batch * heads_kv), dim3(moba::kKv4ColThreads),
                     moba::kKv4ColSmemBytes, st, p);
    } else if (keep) {
      launch_chained(moba::kv4_seen_kernel,
                     dim3((unsigned)((capacity + moba::kKv4SeenKeys - 1) / moba::kKv4SeenKeys), batch * heads_kv),
                     dim3(moba::kKv4SeenThreads), 0, st, p);
    } else if (acc) {
      const int per = moba::kKv4WeightThreads / 32 * (few ? moba::kKv4WeightTiles : 1);
      launch_chained(few ? moba::kv4_weight_kernel<false> : moba::kv4_weight_kernel<true>,
                     dim3((unsigned)((p.tiles + per - 1) / per), batch * heads_kv), dim3(moba::kKv4WeightThreads), 0,
                     st, p);
    }
    MOBA_CUDA(cudaGetLastError());
    return MOBA_OK;
  };
  rc = direct_run(c.off, run, stream);
  return finish_call(rc, stream);
}

int moba_kv4_evict(const void* kv4, const float* acc, const int32_t* lengths, int batch, int heads_kv, int head_dim,
                   int64_t capacity, int64_t budget, int64_t recent, void* dst_kv4, float* dst_acc,
                   int64_t dst_capacity, int32_t* kept, int32_t* new_lengths, cudaStream_t stream) {
  g_err.clear();
  if (!kv4 || !acc || !lengths || !dst_kv4 || !dst_acc || !kept || !new_lengths)
    return fail(MOBA_ERR_INVALID_ARG, "null pointer argument");
  int rc = check_cache(batch, heads_kv, head_dim, capacity);
  if (rc) return rc;
  rc = check_cache(batch, heads_kv, head_dim, dst_capacity);
  if (rc) return rc;
  if (budget < 1 || budget > dst_capacity)
    return fail(MOBA_ERR_INVALID_ARG, "budget must be in [1, dst_capacity] (got %lld)", (long long)budget);
  if (recent < 0 || recent > budget)
    return fail(MOBA_ERR_INVALID_ARG, "recent must be in [0, budget] (got %lld)", (long long)recent);
  if (!aligned16(kv4) || !aligned16(dst_kv4)) return fail(MOBA_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  if (!aligned4(acc) || !aligned4(lengths) || !aligned4(dst_acc) || !aligned4(kept) || !aligned4(new_lengths))
    return fail(MOBA_ERR_INVALID_ARG, "acc, lengths, kept and new_lengths must be 4-byte aligned");
  const size_t pairs = (size_t)batch * heads_kv;
  if (overlap(kv4, cache_bytes(batch, heads_kv, capacity), dst_kv4, cache_bytes(batch, heads_kv, dst_capacity)) ||
      overlap(acc, pairs * capacity * 4, dst_acc, pairs * dst_capacity * 4) ||
      overlap(lengths, (size_t)batch * 4, new_lengths, (size_t)batch * 4))
    return fail(MOBA_ERR_INVALID_ARG, "the outputs must not overlap the inputs");
  DeviceInfo dev;
  rc = kv4_begin(&dev, stream);
  if (rc) return rc;
  moba::Kv4EvictParams p;
  p.kv4 = static_cast<const uint8_t*>(kv4);
  p.acc = acc;
  p.lengths = lengths;
  p.tiles = capacity / moba::kKv4Tile;
  p.dst_tiles = dst_capacity / moba::kKv4Tile;
  p.batch = batch;
  p.heads = heads_kv;
  p.budget = (int)budget;
  p.recent = (int)recent;
  p.dst = static_cast<uint8_t*>(dst_kv4);
  p.dst_acc = dst_acc;
  p.kept = kept;
  p.new_lengths = new_lengths;
  // up to 8 CTAs select for a kv head while there are SMs for them and 4096 weights for each
  int csize = 1;
  while (csize < 8 && (int64_t)pairs * csize * 2 <= 2 * dev.sms && capacity / csize > 4096) csize *= 2;
  // where a part is one sweep of 512 threads, so many take it, and two CTAs share an SM
  if ((capacity + csize - 1) / csize <= moba::kKv4SelectFew * moba::kKv4SelectItems)
    launch_clusters(moba::kv4_select_kernel<moba::kKv4SelectFew>, dim3((unsigned)pairs * csize),
                    dim3(moba::kKv4SelectFew), 0, csize, stream, p);
  else
    launch_clusters(moba::kv4_select_kernel<moba::kKv4SelectMany>, dim3((unsigned)pairs * csize),
                    dim3(moba::kKv4SelectMany), 0, csize, stream, p);
  const int64_t per = moba::kKv4MoveThreads / 8 * moba::kKv4MoveTokens;
  launch_chained(moba::kv4_move_kernel, dim3((unsigned)((budget + per - 1) / per), (unsigned)pairs),
                 dim3(moba::kKv4MoveThreads), 0, stream, p);
  MOBA_CUDA(cudaGetLastError());
  return finish_call(MOBA_OK, stream);
}

}  // extern "C"
