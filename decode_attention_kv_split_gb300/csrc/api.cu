// Host side of the C ABI declared in include/decode_attn.h: argument checks,
// split planning, TMA descriptor encoding, workspace handling and launches.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace {

using da::KernelShape;
using da::SplitParams;

std::atomic<uint64_t> g_launches{0};
#ifdef DA_TEST_HOOKS
std::atomic<int> g_test_withhold_cta{-1};  // test builds: see decode_attn_test_withhold
#endif
thread_local char g_last_cuda_error[256] = "";

int fail_cuda(cudaError_t e, const char* what) {
  snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s (%d)", what,
           cudaGetErrorString(e), int(e));
  return DA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Device properties, cached per device ordinal.
// ---------------------------------------------------------------------------
struct DeviceInfo {
  int checked = 0;
  int ok = 0;
  int sms = 0;
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int current_device(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (*dev < 0 || *dev >= kMaxDevices) return DA_ERR_DEVICE;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& di = g_dev[*dev];
  if (!di.checked) {
    int major = 0, minor = 0, count = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, *dev)) != cudaSuccess)
      return fail_cuda(e, "cudaDeviceGetAttribute");
    di.ok = (major == 10 && minor == 3);
    di.sms = count;
    di.checked = 1;
  }
  *sms = di.sms;
  return di.ok ? DA_OK : DA_ERR_DEVICE;
}

// ---------------------------------------------------------------------------
// Tensor-map encoding through the driver entry point (no libcuda link).
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

int get_encoder(EncodeTiledFn* fn) {
  std::call_once(g_encode_once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    g_encode_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                    cudaEnableDefault, &q);
    if (g_encode_err == cudaSuccess && q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (!g_encode) return fail_cuda(g_encode_err == cudaSuccess ? cudaErrorNotSupported : g_encode_err,
                                  "cuTensorMapEncodeTiled entry point");
  *fn = g_encode;
  return DA_OK;
}

// Recently encoded descriptors: decode steps reuse the same caches, and an
// encode costs more host time than the rest of a call.
struct MapCacheEntry {
  const void* base;
  int dtype, d, n_max, heads, rows, cols, swz;
  CUtensorMap map;
};
constexpr int kMapCacheSize = 32;
MapCacheEntry g_map_cache[kMapCacheSize];
int g_map_cache_next = 0;
std::mutex g_map_mu;

int encode_cache_map_uncached(CUtensorMap* map, const void* base, int dtype, int d, int n_max,
                              int heads, const KernelShape& ks);

// Bytes per cached element of a cache type; kScaleMap marks the tensor map
// of an 8-bit cache's row scales.
constexpr int kScaleMap = 100;
int elem_size(int dtype) { return dtype == DA_FP32 ? 4 : dtype == DA_BF16 ? 2 : 1; }
bool is_q8(int dtype) { return dtype == DA_INT8 || dtype == DA_FP8_E4M3; }

// A [rows_total = B*h_kv heads][n_max][d] cache viewed as a 3-D tensor
// (innermost first): x = column, y = row inside a head, z = b*h_kv + head.
int encode_cache_map(CUtensorMap* map, const void* base, int dtype, int d, int n_max, int heads,
                     const KernelShape& ks) {
  std::lock_guard<std::mutex> lk(g_map_mu);
  for (int i = 0; i < kMapCacheSize; ++i) {
    const MapCacheEntry& e = g_map_cache[i];
    if (e.base == base && e.dtype == dtype && e.d == d && e.n_max == n_max && e.heads == heads &&
        e.rows == ks.tile_rows && e.cols == ks.box_cols && e.swz == ks.swizzle128) {
      *map = e.map;
      return DA_OK;
    }
  }
  const int st = encode_cache_map_uncached(map, base, dtype, d, n_max, heads, ks);
  if (st == DA_OK) {
    MapCacheEntry& e = g_map_cache[g_map_cache_next];
    g_map_cache_next = (g_map_cache_next + 1) % kMapCacheSize;
    e = MapCacheEntry{base, dtype, d, n_max, heads, ks.tile_rows, ks.box_cols, ks.swizzle128, *map};
  }
  return st;
}

int encode_cache_map_uncached(CUtensorMap* map, const void* base, int dtype, int d, int n_max,
                              int heads, const KernelShape& ks) {
  EncodeTiledFn fn;
  int st = get_encoder(&fn);
  if (st != DA_OK) return st;
  CUresult r;
  const cuuint32_t estr[3] = {1, 1, 1};
  if (dtype == kScaleMap) {
    // row scales [heads][n_max] float32, one row of the tile per element
    const cuuint64_t dims[2] = {cuuint64_t(n_max), cuuint64_t(heads)};
    const cuuint64_t strides[1] = {cuuint64_t(n_max) * 4};
    const cuuint32_t box[2] = {cuuint32_t(ks.tile_rows), 1};
    r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box,
           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const int es = elem_size(dtype);
    const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(n_max), cuuint64_t(heads)};
    const cuuint64_t strides[2] = {cuuint64_t(d) * es, cuuint64_t(n_max) * d * es};
    const cuuint32_t box[3] = {cuuint32_t(ks.box_cols), cuuint32_t(ks.tile_rows), 1};
    const CUtensorMapDataType ty = dtype == DA_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == DA_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                      : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    r = fn(map, ty, 3, const_cast<void*>(base), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           ks.swizzle128 == 1   ? CU_TENSOR_MAP_SWIZZLE_128B
           : ks.swizzle128 == 2 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) {
    snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "cuTensorMapEncodeTiled failed (%d)",
             int(r));
    return DA_ERR_CUDA;
  }
  return DA_OK;
}

// ---------------------------------------------------------------------------
// Argument checks and split planning.
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The element type of q, K, V and whether `out` is bf16, from a dtype argument.
struct DtypeArg {
  int kv;        // DA_FP32 or DA_BF16
  bool out_bf16;
};
bool parse_dtype(int dtype, DtypeArg* a) {
  a->kv = dtype & 0xff;
  a->out_bf16 = (dtype & DA_OUT_BF16) != 0;
  return (dtype & ~(0xff | DA_OUT_BF16)) == 0 &&
         (a->kv == DA_FP32 || a->kv == DA_BF16 || a->kv == DA_INT8 || a->kv == DA_FP8_E4M3);
}

// block: an 8-bit cache with block scales (no row-scale tensor map).
int check_sizes(int B, int h_q, int h_kv, int d_k, int d_v, int n_max, int dtype,
                bool block = false) {
  DtypeArg dt;
  if (!parse_dtype(dtype, &dt)) return DA_ERR_DTYPE;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || n_max <= 0) return DA_ERR_SHAPE;
  if (h_q % h_kv != 0) return DA_ERR_SHAPE;
  if (n_max > (1 << 30)) return DA_ERR_SHAPE;
  if ((long long)B * h_kv * (long long)n_max > 0x7fffffffLL) return DA_ERR_SHAPE;
  if ((long long)B * h_q > 0x7fffffffLL) return DA_ERR_SHAPE;
  // (d_k, d_v) pairs with kernels: 64/64 and 128/128 for every cache type;
  // 256/256 and 192/128 for bf16 caches
  const bool common = (d_k == 64 || d_k == 128) && d_v == d_k;
  const bool wide = dt.kv == DA_BF16 && ((d_k == 256 && d_v == 256) || (d_k == 192 && d_v == 128));
  if (!common && !wide) return DA_ERR_UNSUPPORTED;
  if (is_q8(dt.kv) && !block && n_max % 4 != 0) return DA_ERR_SHAPE;  // row-scale tensor map stride
  return DA_OK;
}

// Score terms: argument checks, the most rows a query can see, and the terms
// as the kernels of one launch slice take them (no mod: plain scores).
int check_mod(const da_score_mod* mod) {
  if (!mod) return DA_ERR_NULL;
  if (!(mod->softcap >= 0.f) || !isfinite(mod->softcap)) return DA_ERR_SHAPE;
  // the kernels hold softcap * log2(e) and scale / softcap in float
  if (mod->softcap > 0.f && (mod->softcap < 1e-30f || mod->softcap > 1e30f)) return DA_ERR_SHAPE;
  if (mod->window < 0 || mod->prefix < 0) return DA_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(mod->slopes) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(mod->doc_begin) & 3u) != 0)
    return DA_ERR_ALIGN;
  return DA_OK;
}

// Whether two arrays of n words share one.
bool words_overlap(const void* a, const void* b, long long n) {
  const long long apart = (long long)(reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b));
  return a && b && apart < 4 * n && apart > -4 * n;
}

long long seen_rows(const da_score_mod* mod, int n_max) {
  if (!mod) return -1;
  return mod->window > 0 ? (long long)mod->window + mod->prefix : n_max;
}

da::ScoreTerms score_terms_of(const da_score_mod* mod, int tile_rows, int b0, float scale,
                               bool out_bf16) {
  da::ScoreTerms t{};
  if (!mod) return t;
  t.on = 1;
  t.tile_rows = tile_rows;
  t.window = mod->window;
  t.prefix = mod->prefix;
  t.doc_begin = mod->doc_begin ? mod->doc_begin + b0 : nullptr;
  t.slopes = mod->slopes;
  if (mod->softcap > 0.f && mod->softcap <= da::kShortTanhCap && out_bf16)
    t.short_scale = float(2.0 * 1.4426950408889634 * double(scale) / double(mod->softcap));
  t.cap_log2 = float(double(mod->softcap) * 1.4426950408889634);
  return t;
}

struct Plan {
  KernelShape ks;
  bool tc5;            // bf16, d = 128, group > 8: the tcgen05 kernel
  int head_chunks;
  int chunk_fixed;     // > 0: rows per split fixed by the caller's num_splits
  int chunk_min;       // else: the device picks chunk_min * 2^k
  int max_splits;      // partial slots per query head
  int batch_per_launch;
  bool balanced;       // num_splits = -1: one equal piece of all rows per CTA
  int units;           // (sequence, kv head, head chunk) units of one launch slice
  int places, rounds, cluster;  // block-scaled caches: see SplitParams
  long long grid;      // block-scaled caches: CTAs of a full launch slice
};

// The device-side cost model (choose_chunk) evaluated with every sequence at
// n_max: if even full-length sequences are best served by one split, shorter
// ones are too, and the launch needs neither partials nor a combine.
bool single_split_suffices(long long units, int n_max, int chunk_min, int tile, int sms,
                           float cta_speed) {
  const long long grid = sms;  // the device model uses the whole persistent grid
  const double share = double(n_max) * double(units) / double(grid);
  double best_t = 1e300;
  long long best_c = chunk_min;
  for (int k = 0; k < 32; ++k) {
    long long c;
    if (k < 16) {
      c = (long long)chunk_min << k;
      if (k > 0 && ((long long)chunk_min << (k - 1)) >= n_max) continue;
    } else {
      long long pieces = (long long)(k - 15) * grid / units;
      if (pieces < 1) pieces = 1;
      c = (n_max + pieces - 1) / pieces;
    }
    c = (c + tile - 1) / tile * tile;
    if (c < chunk_min) c = chunk_min;
    const long long per_seq_items = (n_max + c - 1) / c;
    const double items = double(per_seq_items) * double(units);
    const double rounds = ceil(items / double(grid));
    const double ceff = double(c < n_max ? c : n_max);
    double t = fmax(share, rounds * ceff / cta_speed) + rounds * tile;
    if (c < n_max) t += 2.0 * tile;
    if (t < best_t * 0.999 || (t <= best_t * 1.001 && c < best_c)) {
      best_t = t;
      best_c = c;
    }
  }
  return best_c >= n_max;
}

// Block-scaled caches (see make_plan): the most bytes of partials.
constexpr long long kBlockPartialBytes = 64LL << 20;

// With score terms or block scales: the most rows that a CTA of a unit's cluster takes,
// by itself or with up to seven others, where there are no more units than SMs.  A second
// launch costs a step 4 us of host time, and 1.5 to 2 us of the GPU's in a graph; one CTA
// streams these rows in about 3 us.  Measured with one CTA a unit at 1 and 8 sequences
// against the cost model's choice: a call by itself 2 to 5 us faster up to here, a step of
// a graph between 1.6 us faster and 0.6 slower; at twice the rows 2 to 5 us slower.
//   8-bit blocks: 5 to 8 ns a row, 10 for more than 8 heads a KV head
//   bf16: 5 ns a row, 12 for d = 256 or 32 heads of 64
//   fp32: 8 ns a row for one head of 64, 10 for two or one of 128, 20 to 30 for more
int single_split_rows(const KernelShape& ks, int dtype, int d, int d_v, int group, bool block) {
  if (block) return group <= 8 ? 512 : 384;
  if (dtype == DA_BF16)
    return ks.heads_per_cta > 16 ? 192 : d + d_v > 256 ? 256 : ks.heads_per_cta > 8 ? 384 : 512;
  const int products = ks.heads_per_cta * d;
  return products <= 64 ? 384 : products <= 128 ? 192 : products <= 512 ? 128 : 96;
}

// How many clusters of c CTAs that take an SM each the (current) device runs at once: a
// cluster lies within one of its groups of SMs, so 152 SMs hold fewer than 19 of 8 (18
// clusters of 7 or 8 took two rounds, 8.6 us for 4.5).  Asked once per device and c.
__global__ void whole_sm_kernel() {}

int clusters_at_once(int c, int dev) {
  static std::atomic<int> known[kMaxDevices][9];
  int n = known[dev][c].load(std::memory_order_relaxed);
  if (n > 0) return n;
  constexpr int kSmem = 200 * 1024;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(c);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(c));
  cfg.blockDim = dim3(288);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(whole_sm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, whole_sm_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  known[dev][c].store(n, std::memory_order_relaxed);
  return n;
}

// Splits per sequence requested by the caller -> a split length that is a
// whole number of pipeline stages, as close as possible to n_max / S.  When
// the library chooses, the device picks the length from the actual sequence
// lengths; the host only bounds it from below so that the partial outputs of
// at most about 4 x SMs work items per launch need workspace.
// seen: with score terms, the most rows a query can see (a window and the
// prefix; n_max without a window), else -1.  block: an 8-bit cache with block
// scales.
int make_plan(int B, int h_q, int h_kv, int d, int d_v, int n_max, int dtype_arg, int requested,
              int sms, Plan* pl, bool balance_rule = true, long long seen = -1,
              bool block = false) {
  const int dtype = dtype_arg & 0xff;
  const int group = h_q / h_kv;
  pl->tc5 = dtype == DA_BF16 && d == 128 && d_v == 128 && group > 8;
  pl->ks = pl->tc5 ? da::tc5_shape(group)
           : block        ? da::q8b_shape(d, group)
           : is_q8(dtype) ? da::q8_shape(d)
                          : (dtype == DA_BF16 ? da::bf16_shape(d, d_v, group)
                                              : da::f32_shape(d, group));
  pl->head_chunks = (group + pl->ks.heads_per_cta - 1) / pl->ks.heads_per_cta;
  pl->batch_per_launch = B < da::kMaxBatchPerLaunch ? B : da::kMaxBatchPerLaunch;
  const long long tile = pl->ks.tile_rows;
  // A work list with score terms holds whole tiles of the rows that are seen:
  // less than a tile more at the prefix's end and at the window's start.
  if (seen >= 0 && seen + 2 * tile < n_max) n_max = int(seen + 2 * tile);
  const long long max_tiles = (n_max + tile - 1) / tile;
  pl->balanced = false;
  pl->places = pl->rounds = pl->cluster = 0;
  pl->grid = 0;
  pl->units = int((long long)pl->batch_per_launch * h_kv * pl->head_chunks);
  if (requested < -1) return DA_ERR_SHAPE;
  if (block) {
    // One CTA per chunk, whose length the kernel picks from the actual lengths
    // (candidate_chunk in decode_q8b.cu); the host sizes the grid for every sequence at
    // full length and bounds the splits, by the chunks there can be and by the
    // partials' bytes.
    // (a sixteenth of the places is left over: the previous grid's last CTAs hold
    // some, and chunks that miss a round cost another one; on 2 x 131072 rows of
    // fp8, 80 chunks a unit in 2.8 rounds take 86.3 us, 84 in 2.95 rounds 88.8 us)
    const long long places = (long long)sms * (long long)pl->ks.cta_speed * 15 / 16;
    const long long per_seq = (long long)h_kv * pl->head_chunks, units = pl->units;
    pl->places = int(places);
    pl->rounds = 1;
    if (requested > 0) {
      const long long chunk = ((n_max + requested - 1LL) / requested + tile - 1) / tile * tile;
      pl->chunk_fixed = pl->chunk_min = int(chunk);
      pl->grid = units * ((n_max + chunk - 1) / chunk);
    } else {
      const long long rounds = (units * n_max + places * da::kBlockRoundRows - 1) /
                               (places * da::kBlockRoundRows);
      pl->rounds = int(rounds < 1 ? 1 : (rounds < da::kBlockRounds ? rounds : da::kBlockRounds));
      pl->grid = units <= places ? pl->rounds * places : units + pl->rounds * places;
      long long most = pl->grid / per_seq + 1;  // chunks one sequence's unit can get
      const long long by_rows = (n_max + da::kBlockMinRows - 1) / da::kBlockMinRows;
      const long long by_bytes = kBlockPartialBytes /
                                 ((long long)pl->batch_per_launch * h_q * (d_v + 1) * 4);
      if (most > by_rows) most = by_rows;
      if (most > by_bytes) most = by_bytes;
      if (most < 2 || n_max <= 2 * da::kBlockMinRows) most = 1;
      // Short caches: a cluster of CTAs for each unit, which join its chunks themselves:
      // one launch, no work list and no partials (one sequence of 1024 rows, 8 kv heads
      // of 128: a graph's step 6.4 -> 4.6 us, a call by itself 25.3 -> 21.2; 16 of 512
      // rows, 2 kv heads of 64 with 32 query heads: 9.2 -> 4.7 us).  Two CTAs on an SM
      // cost more than they share (4 of 1024 rows, 8 kv heads: 8 a unit 6.5 us, 4 5.8).
      const int alone = single_split_rows(pl->ks, dtype, d, d_v, group, true);
      long long c = (n_max + da::kBlockMinRows - 1) / da::kBlockMinRows;  // as many as have rows
      if (c * units > sms) c = sms / units;             // while each has an SM,
      const long long least = (n_max + alone - 1) / alone;
      if (c < least) c = least;                         // and more where the rows ask for it
      if (c > 8) c = 8;
      if (n_max <= c * alone && c * units <= (c == 1 ? sms : places)) pl->cluster = int(c);
      if (pl->cluster > 0) {
        pl->chunk_fixed = pl->chunk_min = int((n_max + tile - 1) / tile * tile);
        pl->grid = units * pl->cluster;
        pl->max_splits = 1;
        return DA_OK;
      }
      pl->chunk_fixed = 0;
      pl->chunk_min = int(((n_max + most - 1) / most + tile - 1) / tile * tile);
      if (most == 1) {  // no partials, no combine
        pl->chunk_fixed = pl->chunk_min;
        pl->grid = units;
      }
    }
    pl->max_splits = int((n_max + pl->chunk_min - 1) / pl->chunk_min);
    if (pl->grid > 0x7fffffffLL) return DA_ERR_SHAPE;
    return DA_OK;
  }
  // Balanced pieces when the row stream fits an int and the partials of up
  // to one per SM per query head stay within 256 MiB.
  auto take_balanced = [&]() {
    const long long stream_rows = (long long)pl->units * n_max;
    const long long part_bytes = (long long)pl->batch_per_launch * h_q * sms * (d_v + 1) * 4;
    if (stream_rows >= (1LL << 31) || part_bytes > (256LL << 20)) return false;
    pl->balanced = true;
    pl->chunk_fixed = 0;
    pl->chunk_min = int(tile);
    pl->max_splits = sms;  // a unit has at most one piece per CTA
    return true;
  };
  if (requested == -1) {
    if (take_balanced()) return DA_OK;
    requested = 0;  // otherwise the library's usual choice
  }
  if (requested > 0) {
    long long tiles = (n_max + (long long)requested * tile / 2) / ((long long)requested * tile);
    if (tiles < 1) tiles = 1;
    pl->chunk_fixed = int(tiles * tile);
    pl->chunk_min = pl->chunk_fixed;
  } else {
    const long long units = (long long)pl->batch_per_launch * h_kv * pl->head_chunks;
    long long cap = (4LL * sms + units - 1) / units;
    if (cap > max_tiles) cap = max_tiles;
    if (cap < 1) cap = 1;
    const long long per = (n_max + cap - 1) / cap;
    pl->chunk_fixed = 0;
    pl->chunk_min = int((per + tile - 1) / tile * tile);
    // With score terms, as for block scales; a CTA has an SM to itself.  More than 8 heads
    // of 128 a KV head go to the mma.sync kernel then, 8 a CTA (the tcgen05 kernel has no
    // such form, and its set-up alone takes longer: one sequence of 512 rows and 32 heads
    // on one KV head 13.6 us, this way 5.2), and that with twice the rows a CTA.
    const int chunks = pl->tc5 ? (group + 7) / 8 : pl->head_chunks;
    const KernelShape ks = pl->tc5 ? da::bf16_shape(d, d_v, 8) : pl->ks;
    const int alone = single_split_rows(ks, dtype, d, d_v, group, false) * (pl->tc5 ? 2 : 1);
    const long long parts = (long long)pl->batch_per_launch * h_kv * chunks;
    int dev = 0;
    if (seen >= 0 && parts <= sms && n_max <= 8LL * alone && cudaGetDevice(&dev) == cudaSuccess) {
      long long share = single_split_rows(ks, dtype, d, d_v, group, false) / 4;
      if (share < ks.tile_rows) share = ks.tile_rows;
      long long c = (n_max + share - 1) / share;
      if (c > 8) c = 8;
      while (c > 1 && parts > clusters_at_once(int(c), dev)) --c;
      if (n_max <= c * alone) {
        pl->tc5 = false;
        pl->ks = ks;
        pl->head_chunks = chunks;
        pl->units = int(parts);
        pl->cluster = int(c);
        pl->chunk_fixed = pl->chunk_min = (n_max + ks.tile_rows - 1) / ks.tile_rows * ks.tile_rows;
        pl->grid = parts * c;
        pl->max_splits = 1;
        return DA_OK;
      }
    }
    if (seen >= 0 && pl->tc5 && units <= sms && n_max <= 512) {
      pl->chunk_fixed = pl->chunk_min = int(max_tiles * tile);
    } else if (single_split_suffices(units, n_max, pl->chunk_min, int(tile), sms,
                                     pl->ks.cta_speed)) {
      // One split per unit needs no partials and no combine, but when the
      // units fill the grid's rounds unevenly (fewer units than CTAs, or a
      // ragged last round) the CTAs without a unit idle while the longest
      // sequences stream.  Then balanced pieces, if each CTA's share is at
      // least 8 tiles (below that the merge costs more than the idle SMs).
      const long long rounds = (units + sms - 1) / sms;
      const bool uneven = double(units) < 0.9 * double(rounds * sms);
      const bool sizeable = units * (long long)n_max >= 8LL * tile * sms;
      if (balance_rule && uneven && sizeable && take_balanced()) return DA_OK;
      pl->chunk_fixed = int(max_tiles * tile);  // one split: no partials, no combine
      pl->chunk_min = pl->chunk_fixed;
    }
  }
  const long long splits = (n_max + pl->chunk_min - 1) / pl->chunk_min;
  if (splits >= (1 << 20)) return DA_ERR_SHAPE;
  pl->max_splits = int(splits);
  if ((long long)pl->batch_per_launch * h_q * pl->max_splits * (d_v + 1) > (1LL << 40))
    return DA_ERR_SHAPE;
  return DA_OK;
}

// Workspace of one launch: a header word (the split length the kernels
// used), partial outputs, partial log-sum-exps.
struct WorkspaceLayout {
  size_t header, o_part, lse_part, hints, total;
};

WorkspaceLayout workspace_layout(const Plan& pl, int h_q, int d) {
  WorkspaceLayout w{0, 0, 0, 0, 0};
  if (pl.max_splits <= 1) return w;
  const size_t heads = size_t(pl.batch_per_launch) * h_q;
  w.header = 0;
  // header word; in balanced mode the per-unit partial counts follow it
  w.o_part = pl.balanced ? 256 + (size_t(pl.units) * 4 + 255) / 256 * 256 : 256;
  w.lse_part = w.o_part + heads * pl.max_splits * d * sizeof(float);
  // then each CTA's first-tile hint for the next call (16 bytes per CTA)
  w.hints = (w.lse_part + heads * pl.max_splits * sizeof(float) + 255) / 256 * 256;
  w.total = w.hints + size_t(da::kMaxHintCtas) * 16;
  return w;
}

// Library-owned workspace for decode_attn(), one per device.
struct OwnedWorkspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};
OwnedWorkspace g_ws[kMaxDevices];
std::mutex g_ws_mu;

// Row scales of an 8-bit cache (and of the appended rows, for a fused append).
struct QuantArgs {
  float* k_scale;
  float* v_scale;
  const float* k_new_scale;
  const float* v_new_scale;
};

// A block-scaled 8-bit cache: one scale per 2^shift rows and head.
struct BlockArgs {
  const float* k_scale;
  const float* v_scale;
  int shift;
};

int run_decode(const void* q, const void* K, const void* V, const int32_t* seq_lens,
                      void* out, int B, int h_q, int h_kv, int d_k, int d_v, int n_max,
                      float scale, int dtype_arg, int num_splits, void* workspace,
                      size_t workspace_bytes, int32_t* dev_error, cudaStream_t stream,
                      const void* k_new, const void* v_new, int32_t* seq_lens_out,
                      const QuantArgs* qa, int row_off = 0, int row_lim = 0x7fffffff,
                      float* lse_out = nullptr, const da_score_mod* mod = nullptr,
                      const BlockArgs* ba = nullptr) {
  if (!q || !K || !V || !seq_lens || !out) return DA_ERR_NULL;
  int st = check_sizes(B, h_q, h_kv, d_k, d_v, n_max, dtype_arg, ba != nullptr);
  if (st != DA_OK) return st;
  DtypeArg dta;
  parse_dtype(dtype_arg, &dta);
  const int dtype = dta.kv;
  // 8-bit caches go through the entry points that carry their row scales
  if (is_q8(dtype) != (qa != nullptr || ba != nullptr)) return DA_ERR_DTYPE;
  if (qa && (!qa->k_scale || !qa->v_scale || (k_new && (!qa->k_new_scale || !qa->v_new_scale))))
    return DA_ERR_NULL;
  if (qa && (!aligned16(qa->k_scale) || !aligned16(qa->v_scale))) return DA_ERR_ALIGN;
  // a row range starts the 8-bit row-scale tiles off their 16-byte grid
  if (qa && row_off != 0) return DA_ERR_UNSUPPORTED;
  if (k_new && (row_off != 0 || row_lim < n_max)) return DA_ERR_SHAPE;
  if (!isfinite(scale)) return DA_ERR_SHAPE;
  // (the kernels hold 2 log2(e) scale / softcap in float)
  if (mod && mod->softcap > 0.f && !isfinite(float(4.0 * double(scale) / double(mod->softcap))))
    return DA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(K) || !aligned16(V) || !aligned16(out) ||
      (workspace && !aligned16(workspace)))
    return DA_ERR_ALIGN;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != DA_OK) return st;
  Plan pl;
  if ((st = make_plan(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, sms, &pl, true,
                      seen_rows(mod, n_max), ba != nullptr)) != DA_OK)
    return st;
  const size_t out_es = dta.out_bf16 ? 2 : 4;
  const WorkspaceLayout wl = workspace_layout(pl, h_q, d_v);
  if (wl.total > 0 && (!workspace || workspace_bytes < wl.total)) return DA_ERR_WORKSPACE;

  CUtensorMap tk, tv, tks, tvs;
  if ((st = encode_cache_map(&tk, K, dtype, d_k, n_max, B * h_kv, pl.ks)) != DA_OK) return st;
  if ((st = encode_cache_map(&tv, V, dtype, d_v, n_max, B * h_kv, pl.ks)) != DA_OK) return st;
  if (qa) {
    if ((st = encode_cache_map(&tks, qa->k_scale, kScaleMap, 1, n_max, B * h_kv, pl.ks)) != DA_OK)
      return st;
    if ((st = encode_cache_map(&tvs, qa->v_scale, kScaleMap, 1, n_max, B * h_kv, pl.ks)) != DA_OK)
      return st;
  }

  const int es = elem_size(dtype);          // cached (and appended) elements
  const int q_es = is_q8(dtype) ? 2 : es;   // q is bf16 with an 8-bit cache
  char* ws = static_cast<char*>(workspace);
  for (int b0 = 0; b0 < B; b0 += pl.batch_per_launch) {
    const int bn = (B - b0) < pl.batch_per_launch ? (B - b0) : pl.batch_per_launch;
    SplitParams p;
    p.q = static_cast<const char*>(q) + size_t(b0) * h_q * d_k * q_es;
    p.seq_lens = seq_lens + b0;
    p.out = static_cast<char*>(out) + size_t(b0) * h_q * d_v * out_es;
    p.out_bf16 = dta.out_bf16 ? 1 : 0;
    p.row_off = row_off;
    p.mod = score_terms_of(mod, pl.ks.tile_rows, b0, scale, dta.out_bf16);
    p.row_lim = row_lim;
    p.lse_out = lse_out ? lse_out + size_t(b0) * h_q : nullptr;
    p.o_part = wl.total ? reinterpret_cast<float*>(ws + wl.o_part) : nullptr;
    p.lse_part = wl.total ? reinterpret_cast<float*>(ws + wl.lse_part) : nullptr;
    p.chunk_out = wl.total ? reinterpret_cast<int*>(ws + wl.header) : nullptr;
    p.balanced = pl.balanced ? 1 : 0;
    p.unit_nv = pl.balanced ? reinterpret_cast<int*>(ws + 256) : nullptr;
    p.hints = wl.total ? reinterpret_cast<int4*>(ws + wl.hints) : nullptr;
    p.out_elems = (long long)bn * h_q * d_v;
    p.part_rows = wl.total ? (long long)bn * h_q * pl.max_splits : 0;
    p.cache_rows = (long long)B * h_kv * n_max;
    p.dev_error = dev_error;
    p.append = k_new != nullptr;
    p.k_new = k_new ? static_cast<const char*>(k_new) + size_t(b0) * h_kv * d_k * es : nullptr;
    p.v_new = v_new ? static_cast<const char*>(v_new) + size_t(b0) * h_kv * d_v * es : nullptr;
    p.k_cache = const_cast<void*>(K);
    p.v_cache = const_cast<void*>(V);
    p.seq_lens_out = seq_lens_out ? seq_lens_out + b0 : nullptr;
    p.k_scale = qa ? qa->k_scale : nullptr;
    p.v_scale = qa ? qa->v_scale : nullptr;
    p.k_new_scale = qa && qa->k_new_scale ? qa->k_new_scale + size_t(b0) * h_kv : nullptr;
    p.v_new_scale = qa && qa->v_new_scale ? qa->v_new_scale + size_t(b0) * h_kv : nullptr;
    if (ba) {
      p.k_scale = const_cast<float*>(ba->k_scale);
      p.v_scale = const_cast<float*>(ba->v_scale);
    }
    p.blk_shift = ba ? ba->shift : 0;
    p.nblk = ba ? int(((long long)n_max + (1 << ba->shift) - 1) >> ba->shift) : 0;
    p.scale_elems = (long long)B * h_kv * p.nblk;
    p.places = pl.places;
    p.rounds = pl.rounds;
    p.cluster = pl.cluster;
    p.B = bn;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.group = h_q / h_kv;
    p.b_offset = b0;
    p.n_max = n_max;
    p.head_chunks = pl.head_chunks;
    p.chunk_fixed = pl.chunk_fixed;
    p.chunk_min = pl.chunk_min;
    p.max_splits = pl.max_splits;
    p.cta_speed = pl.ks.cta_speed;
    p.scale_log2 = mod && mod->softcap > 0.f
                       ? float(double(scale) / double(mod->softcap))
                       : float(double(scale) * 1.4426950408889634);  // log2(e) = 1 / ln 2
#ifdef DA_TEST_HOOKS
    p.withhold_cta = b0 == 0 ? g_test_withhold_cta.load() : -1;
#endif
    const long long items = (long long)bn * h_kv * pl.head_chunks * pl.max_splits;
    // one persistent CTA per SM (the balanced list keeps a boundary and a unit
    // tag per CTA in the two halves of the work list's reduction scratch)
    const long long max_grid = da::kSchedRedWords / 2 - 1;
    const long long grid_cap = sms < max_grid ? sms : max_grid;
    // (a block-scaled cache: one CTA per chunk, not persistent)
    const int grid = int(ba || pl.cluster > 0 ? pl.grid : (items < grid_cap ? items : grid_cap));
    cudaError_t err =
        pl.tc5 ? da::launch_split_tc5(p, tk, tv, grid, stream)
        : ba   ? da::launch_split_q8b(p, tk, tv, d_k, dtype == DA_INT8 ? 1 : 2, grid, stream)
        : qa   ? da::launch_split_q8(p, tk, tv, tks, tvs, d_k, dtype == DA_INT8 ? 1 : 2, grid, stream)
        : dtype == DA_BF16 ? da::launch_split_bf16(p, tk, tv, d_k, d_v, grid, stream)
                           : da::launch_split_f32(p, tk, tv, d_k, grid, stream);
    if (err != cudaSuccess) return fail_cuda(err, "split kernel launch");
    g_launches.fetch_add(1);
    if (wl.total) {
      err = da::launch_combine(p, d_v, pl.ks.heads_per_cta, grid, stream);
      if (err != cudaSuccess) return fail_cuda(err, "combine kernel launch");
      g_launches.fetch_add(1);
    }
  }
  return DA_OK;
}


}  // namespace

namespace da {
// Whether the library's own split choice (num_splits = 0) takes balanced
// pieces by the uneven-grid rule of make_plan for this request.
bool library_takes_balanced(int B, int h_q, int h_kv, int d_k, int d_v, int n_max, int dtype) {
  if (check_sizes(B, h_q, h_kv, d_k, d_v, n_max, dtype) != DA_OK) return false;
  int dev = 0, sms = 0;
  if (current_device(&dev, &sms) != DA_OK) return false;
  Plan pl;
  if (make_plan(B, h_q, h_kv, d_k, d_v, n_max, dtype, 0, sms, &pl) != DA_OK) return false;
  return pl.balanced;
}
}  // namespace da

extern "C" {

const char* decode_attn_status_string(int status) {
  switch (status) {
    case DA_OK: return "ok";
    case DA_ERR_NULL: return "null pointer argument";
    case DA_ERR_SHAPE: return "size out of range or inconsistent";
    case DA_ERR_DTYPE: return "unknown dtype";
    case DA_ERR_ALIGN: return "device pointer not 16-byte aligned";
    case DA_ERR_WORKSPACE: return "workspace missing or too small";
    case DA_ERR_CUDA: return "CUDA call failed";
    case DA_ERR_DEVICE: return "current device is not sm_103 (GB300)";
    case DA_ERR_UNSUPPORTED: return "unsupported head dimension combination";
    default: return "unknown status";
  }
}

const char* decode_attn_last_cuda_error(void) { return g_last_cuda_error; }

uint64_t decode_attn_launch_count(void) { return g_launches.load(); }

#ifdef DA_TEST_HOOKS
// Test builds only (not part of the product library or its header): from the
// next decode call on, the producer of split-kernel CTA `cta` never fills the
// last pipeline stage of its first work item, so that a consumer's bounded
// wait runs out (2 ms in test builds) and the kernel takes its timeout path.
// -1 turns it off.
__attribute__((visibility("default"))) void decode_attn_test_withhold(int cta) {
  g_test_withhold_cta.store(cta);
}
#endif

int decode_attn_resolve_splits(int B, int h_q, int h_kv, int d_k, int d_v, int n_max, int dtype,
                               int num_splits) {
  int st = check_sizes(B, h_q, h_kv, d_k, d_v, n_max, dtype);
  if (st != DA_OK) return st;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != DA_OK) return st;
  Plan pl;
  if ((st = make_plan(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, sms, &pl)) != DA_OK)
    return st;
  return pl.max_splits;
}

namespace {
size_t plan_workspace(int B, int h_q, int h_kv, int d_k, int d_v, int n_max, int dtype,
                      int num_splits, long long seen, bool block, int* status) {
  int st = check_sizes(B, h_q, h_kv, d_k, d_v, n_max, dtype, block);
  int dev = 0, sms = 0;
  Plan pl;
  if (st == DA_OK) st = current_device(&dev, &sms);
  if (st == DA_OK)
    st = make_plan(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, sms, &pl, true, seen,
                   block);
  if (status) *status = st;
  return st == DA_OK ? workspace_layout(pl, h_q, d_v).total : 0;
}
}  // namespace

size_t decode_attn_workspace_bytes(int B, int h_q, int h_kv, int d_k, int d_v, int n_max, int dtype,
                                   int num_splits, int* status) {
  return plan_workspace(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, -1, false, status);
}

size_t decode_attn_mod_workspace_bytes(const da_score_mod* mod, int B, int h_q, int h_kv, int d_k,
                                       int d_v, int n_max, int dtype, int num_splits,
                                       int* status) {
  const int st = check_mod(mod);
  if (st != DA_OK || is_q8(dtype & 0xff)) {
    if (status) *status = st != DA_OK ? st : DA_ERR_DTYPE;
    return 0;
  }
  return plan_workspace(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, seen_rows(mod, n_max),
                        false, status);
}

int decode_attn_mod(const void* q, const void* K, const void* V, const int32_t* seq_lens,
                    const da_score_mod* mod, void* out, int B, int h_q, int h_kv, int d_k, int d_v,
                    int n_max, float scale, int dtype, int num_splits, void* workspace,
                    size_t workspace_bytes, int32_t* dev_error, cudaStream_t stream) {
  const int st = check_mod(mod);
  if (st != DA_OK) return st;
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, nullptr, nullptr,
                    nullptr, nullptr, 0, 0x7fffffff, nullptr, mod);
}

int decode_attn_mod_append(const void* q, const void* k_new, const void* v_new, void* K, void* V,
                           const int32_t* seq_lens, int32_t* seq_lens_out,
                           const da_score_mod* mod, void* out, int B, int h_q, int h_kv, int d_k,
                           int d_v, int n_max, float scale, int dtype, int num_splits,
                           void* workspace, size_t workspace_bytes, int32_t* dev_error,
                           cudaStream_t stream) {
  const int st = check_mod(mod);
  if (st != DA_OK) return st;
  if (!k_new || !v_new) return DA_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new)) return DA_ERR_ALIGN;
  // (one CTA writes the new lengths while others still read the old ones and the begins)
  if (words_overlap(seq_lens_out, seq_lens, B) || words_overlap(seq_lens_out, mod->doc_begin, B))
    return DA_ERR_SHAPE;
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, k_new, v_new,
                    seq_lens_out, nullptr, 0, 0x7fffffff, nullptr, mod);
}

int decode_attn_ex(const void* q, const void* K, const void* V, const int32_t* seq_lens, void* out,
                   int B, int h_q, int h_kv, int d_k, int d_v, int n_max, float scale, int dtype,
                   int num_splits, void* workspace, size_t workspace_bytes, int32_t* dev_error,
                   cudaStream_t stream) {
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, nullptr, nullptr,
                    nullptr, nullptr);
}

int decode_attn_append(const void* q, const void* k_new, const void* v_new, void* K, void* V,
                       const int32_t* seq_lens, int32_t* seq_lens_out, void* out, int B, int h_q,
                       int h_kv, int d_k, int d_v, int n_max, float scale, int dtype,
                       int num_splits, void* workspace, size_t workspace_bytes,
                       int32_t* dev_error, cudaStream_t stream) {
  if (!k_new || !v_new) return DA_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new)) return DA_ERR_ALIGN;
  if (seq_lens_out && seq_lens_out == seq_lens) return DA_ERR_SHAPE;
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, k_new, v_new,
                    seq_lens_out, nullptr);
}

int decode_attn_partial(const void* q, const void* K, const void* V, const int32_t* seq_lens,
                        int row_begin, int row_end, float* o, float* lse, int B, int h_q,
                        int h_kv, int d_k, int d_v, int n_max, float scale, int dtype,
                        int num_splits, void* workspace, size_t workspace_bytes,
                        int32_t* dev_error, cudaStream_t stream) {
  if (!lse) return DA_ERR_NULL;
  if ((dtype & DA_OUT_BF16) != 0) return DA_ERR_DTYPE;  // partials are float32
  if (row_begin < 0 || row_end < row_begin) return DA_ERR_SHAPE;
  return run_decode(q, K, V, seq_lens, o, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, nullptr, nullptr,
                    nullptr, nullptr, row_begin, row_end, lse);
}

int decode_attn_combine(const float* o_parts, const float* lse_parts, int S, void* out,
                        float* lse_out, int B, int h_q, int d_v, int out_dtype,
                        cudaStream_t stream) {
  if (S < 0 || B <= 0 || h_q <= 0) return DA_ERR_SHAPE;
  if (!out || (S > 0 && (!o_parts || !lse_parts))) return DA_ERR_NULL;  // S = 0 reads neither
  if (d_v != 64 && d_v != 128 && d_v != 256) return DA_ERR_UNSUPPORTED;
  if (out_dtype != DA_FP32 && out_dtype != (DA_FP32 | DA_OUT_BF16)) return DA_ERR_DTYPE;
  const long long heads = (long long)B * h_q;
  if (heads > (1LL << 36) || (long long)S * heads * d_v > (1LL << 46)) return DA_ERR_SHAPE;
  if (!aligned16(o_parts) || !aligned16(out)) return DA_ERR_ALIGN;
  int dev, sms;
  int st = current_device(&dev, &sms);
  if (st != DA_OK) return st;
  cudaError_t e = da::launch_lse_merge(o_parts, lse_parts, S, out, (out_dtype & DA_OUT_BF16) ? 1 : 0,
                                       lse_out, heads, d_v, stream);
  if (e != cudaSuccess) return fail_cuda(e, "lse merge launch");
  g_launches.fetch_add(1);
  return DA_OK;
}

int decode_attn(const void* q, const void* K, const void* V, const int32_t* seq_lens, void* out,
                int B, int h_q, int h_kv, int d_k, int d_v, int n_max, float scale, int dtype,
                cudaStream_t stream) {
  if (!q || !K || !V || !seq_lens || !out) return DA_ERR_NULL;
  int st = DA_OK;
  const size_t need =
      decode_attn_workspace_bytes(B, h_q, h_kv, d_k, d_v, n_max, dtype, 0, &st);
  if (st != DA_OK) return st;
  void* ws = nullptr;
  // Held through the launch so that a concurrent growth cannot free the
  // buffer between taking its address and enqueueing the kernels.
  std::lock_guard<std::mutex> lk(g_ws_mu);
  if (need > 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return DA_ERR_DEVICE;
    OwnedWorkspace& w = g_ws[dev];
    if (w.bytes < need) {
      if (w.ptr) {
        e = cudaFree(w.ptr);  // waits for work still using the old buffer
        w.ptr = nullptr;
        w.bytes = 0;
        if (e != cudaSuccess) return fail_cuda(e, "cudaFree(workspace)");
      }
      e = cudaMalloc(&w.ptr, need);
      if (e != cudaSuccess) {
        w.ptr = nullptr;
        return fail_cuda(e, "cudaMalloc(workspace)");
      }
      w.bytes = need;
    }
    ws = w.ptr;
  }
  return decode_attn_ex(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype, 0, ws,
                        need, nullptr, stream);
}

namespace {
int append_rows(const void* k_new, const void* v_new, void* K, void* V, const int32_t* pos, int B,
                int h_kv, int d_k, int d_v, int n_max, int dtype, const float* ks_new,
                const float* vs_new, float* ks, float* vs, int32_t* dev_error,
                cudaStream_t stream) {
  if (!k_new || !v_new || !K || !V || !pos) return DA_ERR_NULL;
  if (B <= 0 || h_kv <= 0 || d_k <= 0 || d_v <= 0 || n_max <= 0) return DA_ERR_SHAPE;
  const int es = elem_size(dtype);
  if ((d_k * es) % 16 != 0 || (d_v * es) % 16 != 0) return DA_ERR_SHAPE;
  if ((long long)B * h_kv * (long long)n_max > 0x7fffffffLL) return DA_ERR_SHAPE;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(K) || !aligned16(V)) return DA_ERR_ALIGN;
  int dev, sms;
  int st = current_device(&dev, &sms);
  if (st != DA_OK) return st;
  cudaError_t e = da::launch_kv_append(k_new, v_new, K, V, pos, B, h_kv, d_k * es, d_v * es, n_max,
                                       ks_new, vs_new, ks, vs, dev_error, stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv_append launch");
  g_launches.fetch_add(1);
  return DA_OK;
}
}  // namespace

int kv_append(const void* k_new, const void* v_new, void* K, void* V, const int32_t* pos, int B,
              int h_kv, int d_k, int d_v, int n_max, int dtype, int32_t* dev_error,
              cudaStream_t stream) {
  if (dtype != DA_FP32 && dtype != DA_BF16) return DA_ERR_DTYPE;
  return append_rows(k_new, v_new, K, V, pos, B, h_kv, d_k, d_v, n_max, dtype, nullptr, nullptr,
                     nullptr, nullptr, dev_error, stream);
}

int kv_append_q8(const void* k_new, const void* v_new, const float* k_new_scale,
                 const float* v_new_scale, void* K, void* V, float* k_scale, float* v_scale,
                 const int32_t* pos, int B, int h_kv, int d_k, int d_v, int n_max, int dtype,
                 int32_t* dev_error, cudaStream_t stream) {
  if (!is_q8(dtype)) return DA_ERR_DTYPE;
  if (!k_new_scale || !v_new_scale || !k_scale || !v_scale) return DA_ERR_NULL;
  return append_rows(k_new, v_new, K, V, pos, B, h_kv, d_k, d_v, n_max, dtype, k_new_scale,
                     v_new_scale, k_scale, v_scale, dev_error, stream);
}

int decode_attn_q8_ex(const void* q, const void* K, const void* V, const float* k_scale,
                      const float* v_scale, const int32_t* seq_lens, void* out, int B, int h_q,
                      int h_kv, int d_k, int d_v, int n_max, float scale, int dtype,
                      int num_splits, void* workspace, size_t workspace_bytes,
                      int32_t* dev_error, cudaStream_t stream) {
  if (!is_q8(dtype & 0xff)) return DA_ERR_DTYPE;
  const QuantArgs qa{const_cast<float*>(k_scale), const_cast<float*>(v_scale), nullptr, nullptr};
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, nullptr, nullptr,
                    nullptr, &qa);
}

int decode_attn_q8_append(const void* q, const void* k_new, const void* v_new,
                          const float* k_new_scale, const float* v_new_scale, void* K, void* V,
                          float* k_scale, float* v_scale, const int32_t* seq_lens,
                          int32_t* seq_lens_out, void* out, int B, int h_q, int h_kv, int d_k,
                          int d_v, int n_max, float scale, int dtype, int num_splits,
                          void* workspace, size_t workspace_bytes, int32_t* dev_error,
                          cudaStream_t stream) {
  if (!is_q8(dtype & 0xff)) return DA_ERR_DTYPE;
  if (!k_new || !v_new || !k_new_scale || !v_new_scale) return DA_ERR_NULL;
  if (seq_lens_out && seq_lens_out == seq_lens) return DA_ERR_SHAPE;
  if (!aligned16(k_new) || !aligned16(v_new)) return DA_ERR_ALIGN;
  const QuantArgs qa{k_scale, v_scale, k_new_scale, v_new_scale};
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, k_new, v_new,
                    seq_lens_out, &qa);
}

namespace {
// log2 of a block length with kernels (16, 32, 64, 128), or -1.
int block_shift(int block) {
  return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : -1;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A stride of rows that are moved 16 bytes at a time (the bound keeps offsets inside 64 bits).
int check_stride(long long stride, int es) {
  if (stride < 0 || stride > (1LL << 31) * 256) return DA_ERR_SHAPE;
  return stride * es % 16 != 0 ? DA_ERR_ALIGN : DA_OK;
}

// Rows in memory: `run` bytes at `at` plus any index below n[i] times step[i] (bytes), all of
// them within `reach` bytes.
struct RowSet {
  uintptr_t at;
  long long run, step[3], reach;
  int n[3];
};
constexpr long long kMostReach = 1LL << 60;  // no memory is that large
RowSet one_span(const void* at, long long bytes) {
  return RowSet{reinterpret_cast<uintptr_t>(at), bytes, {0, 0, 0}, bytes, {1, 1, 1}};
}
RowSet strided_rows(const void* at, const long long* strides, int B, int h, int T, int d, int es) {
  RowSet r = one_span(at, (long long)d * es);
  const int n[3] = {B, h, T};
  for (int i = 0; i < 3; ++i) {
    r.n[i] = n[i];
    r.step[i] = strides[i] * es;
    if (n[i] > 1 && r.step[i] > kMostReach / n[i]) r.reach = kMostReach;
    if (r.reach < kMostReach) r.reach += (n[i] - 1) * r.step[i];
  }
  return r;
}

// Whether two of them share a byte.  Rows of one start a sum of steps away from rows of the
// other, each step taken up to n - 1 times forward (its own) or back (the other's): the sums that
// lie less than a run away are looked for from the largest step down.
struct RowSteps {
  long long step[6], lo[6], hi[6];      // times that each is taken
  long long least[7], most[7];          // sums of what follows
  int count = 0, budget = 1 << 14;
  void add(long long s, long long l, long long h) {
    int i = 0;
    while (i < count && step[i] > s) ++i;
    if (i < count && step[i] == s) {
      lo[i] += l, hi[i] += h;
      return;
    }
    for (int k = count++; k > i; --k) step[k] = step[k - 1], lo[k] = lo[k - 1], hi[k] = hi[k - 1];
    step[i] = s, lo[i] = l, hi[i] = h;
  }
  static long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }
  // a sum from step i on in (above, below)?
  bool reach(int i, long long above, long long below) {
    if (most[i] <= above || least[i] >= below) return false;
    if (i == count) return true;
    if (--budget < 0) return false;     // (strides that nest in neither order: not told apart)
    const long long from = floor_div(above - most[i + 1], step[i]) + 1;
    const long long to = -(floor_div(least[i + 1] - below, step[i]) + 1);
    for (long long x = from < lo[i] ? lo[i] : from; x <= to && x <= hi[i]; ++x)
      if (reach(i + 1, above - x * step[i], below - x * step[i])) return true;
    return false;
  }
};
bool share_bytes(const RowSet& a, const RowSet& b) {
  if (!a.at || !b.at) return false;
  const long long delta = (long long)(a.at - b.at);
  if (delta >= b.reach || -delta >= a.reach) return false;
  if (a.reach >= kMostReach || b.reach >= kMostReach) return false;
  RowSteps r;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] > 1 && a.step[i] > 0) r.add(a.step[i], 0, a.n[i] - 1);
    if (b.n[i] > 1 && b.step[i] > 0) r.add(b.step[i], 1 - b.n[i], 0);
  }
  r.least[r.count] = r.most[r.count] = 0;
  for (int i = r.count - 1; i >= 0; --i) {
    r.least[i] = r.least[i + 1] + r.lo[i] * r.step[i];
    r.most[i] = r.most[i + 1] + r.hi[i] * r.step[i];
  }
  return r.reach(0, -a.run - delta, b.run - delta);
}

// Sizes and types shared by the write into and the read from a block-scaled cache.
int check_blocks(int B, int h_kv, int T, int d, int n_max, int block, int dtype, int io_dtype) {
  if (!is_q8(dtype) || (io_dtype != DA_FP32 && io_dtype != DA_BF16)) return DA_ERR_DTYPE;
  if (B <= 0 || h_kv <= 0 || T < 0 || n_max <= 0 || n_max > (1 << 30)) return DA_ERR_SHAPE;
  if (block_shift(block) < 0) return DA_ERR_SHAPE;
  if ((long long)B * h_kv > 0x7fffffffLL || (long long)B * h_kv * (long long)n_max > 0x7fffffffLL)
    return DA_ERR_SHAPE;
  if (d != 64 && d != 128) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}
}  // namespace

size_t decode_attn_q8b_workspace_bytes(const da_score_mod* mod, int B, int h_q, int h_kv, int d_k,
                                       int d_v, int n_max, int dtype, int num_splits,
                                       int* status) {
  int st = mod ? check_mod(mod) : DA_OK;
  if (st == DA_OK && !is_q8(dtype & 0xff)) st = DA_ERR_DTYPE;
  if (st != DA_OK) {
    if (status) *status = st;
    return 0;
  }
  return plan_workspace(B, h_q, h_kv, d_k, d_v, n_max, dtype, num_splits, seen_rows(mod, n_max),
                        true, status);
}

int decode_attn_q8b(const void* q, const void* K, const void* V, const float* k_scale,
                    const float* v_scale, int block, const int32_t* seq_lens,
                    const da_score_mod* mod, void* out, int B, int h_q, int h_kv, int d_k, int d_v,
                    int n_max, float scale, int dtype, int num_splits, void* workspace,
                    size_t workspace_bytes, int32_t* dev_error, cudaStream_t stream) {
  if (!is_q8(dtype & 0xff)) return DA_ERR_DTYPE;
  if (!k_scale || !v_scale) return DA_ERR_NULL;
  if (block_shift(block) < 0) return DA_ERR_SHAPE;
  if (!aligned4(k_scale) || !aligned4(v_scale)) return DA_ERR_ALIGN;
  const int st = mod ? check_mod(mod) : DA_OK;
  if (st != DA_OK) return st;
  const BlockArgs ba{k_scale, v_scale, block_shift(block)};
  return run_decode(q, K, V, seq_lens, out, B, h_q, h_kv, d_k, d_v, n_max, scale, dtype,
                    num_splits, workspace, workspace_bytes, dev_error, stream, nullptr, nullptr,
                    nullptr, nullptr, 0, 0x7fffffff, nullptr, mod, &ba);
}

int kv_append_q8b(const void* k_new, const void* v_new, const long long* k_strides,
                  const long long* v_strides, int x_dtype, int T, const int32_t* n_new, void* K,
                  void* V, float* k_scale, float* v_scale, int block, const int32_t* pos, int B,
                  int h_kv, int d, int n_max, int dtype, int32_t* dev_error, cudaStream_t stream) {
  if (!K || !V || !k_scale || !v_scale || !pos || !k_strides || !v_strides) return DA_ERR_NULL;
  int st = check_blocks(B, h_kv, T, d, n_max, block, dtype, x_dtype);
  if (st != DA_OK) return st;
  if (T == 0) return DA_OK;
  if (T > (1 << 30)) return DA_ERR_SHAPE;
  // the kernels count blocks (and below, parts of 32 rows or more) in 32 bits
  if (2LL * B * h_kv * (((T < n_max ? T : n_max) + block - 1) / block + 1) > 0x3fffffffLL)
    return DA_ERR_SHAPE;
  if (!k_new || !v_new) return DA_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(K) || !aligned16(V) ||
      !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(pos) || !aligned4(n_new))
    return DA_ERR_ALIGN;
  da::BlockWriteArgs a{};
  for (int i = 0; i < 3; ++i) {
    // rows are read 16 bytes at a time; the bound keeps offsets inside 64 bits
    const long long ks = k_strides[i], vs = v_strides[i], es = elem_size(x_dtype);
    if (ks < 0 || vs < 0 || ks > (1LL << 31) * 256 || vs > (1LL << 31) * 256) return DA_ERR_SHAPE;
    if (ks * es % 16 != 0 || vs * es % 16 != 0) return DA_ERR_ALIGN;
    a.stride[0][i] = ks;
    a.stride[1][i] = vs;
  }
  // (K and V are written at the same time, held codes scaled in place)
  if (K == V || k_scale == v_scale) return DA_ERR_SHAPE;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != DA_OK) return st;
  a.x[0] = k_new, a.x[1] = v_new;
  a.codes[0] = K, a.codes[1] = V;
  a.scale[0] = k_scale, a.scale[1] = v_scale;
  a.pos = pos, a.n_new = n_new, a.dev_error = dev_error;
  a.B = B, a.h_kv = h_kv, a.T = T, a.d = d, a.n_max = n_max;
  a.blk_shift = block_shift(block);
  a.kind = dtype == DA_INT8 ? 1 : 2;
  a.x_bf16 = x_dtype == DA_BF16;
  a.sms = sms;
  cudaError_t e = da::launch_kv_append_q8b(a, stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv_append_q8b launch");
  g_launches.fetch_add(1);
  return DA_OK;
}

int kv_read_q8b(const void* K, const void* V, const float* k_scale, const float* v_scale,
                int block, const int32_t* seq_lens, const int32_t* row_begin, void* k_out,
                void* v_out, int out_dtype, int T, int B, int h_kv, int d, int n_max, int dtype,
                int32_t* dev_error, cudaStream_t stream) {
  if (!K || !V || !k_scale || !v_scale || !seq_lens) return DA_ERR_NULL;
  int st = check_blocks(B, h_kv, T, d, n_max, block, dtype, out_dtype);
  if (st != DA_OK) return st;
  if (T == 0) return DA_OK;
  if (!k_out || !v_out) return DA_ERR_NULL;
  if (T > (1 << 30) || 2LL * B * h_kv * ((T + 31LL) / 32) > 0x3fffffffLL) return DA_ERR_SHAPE;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(K) || !aligned16(V) ||
      !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(seq_lens) || !aligned4(row_begin))
    return DA_ERR_ALIGN;
  if (k_out == v_out) return DA_ERR_SHAPE;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != DA_OK) return st;
  da::BlockReadArgs a{};
  a.codes[0] = K, a.codes[1] = V;
  a.scale[0] = k_scale, a.scale[1] = v_scale;
  a.out[0] = k_out, a.out[1] = v_out;
  a.seq_lens = seq_lens, a.row_begin = row_begin, a.dev_error = dev_error;
  a.B = B, a.h_kv = h_kv, a.T = T, a.d = d, a.n_max = n_max;
  a.blk_shift = block_shift(block);
  a.kind = dtype == DA_INT8 ? 1 : 2;
  a.out_bf16 = out_dtype == DA_BF16;
  a.sms = sms;
  cudaError_t e = da::launch_kv_read_q8b(a, stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv_read_q8b launch");
  g_launches.fetch_add(1);
  return DA_OK;
}

int kv_append_rope(const void* q, const void* k_new, const void* v_new, const long long* q_strides,
                   const long long* k_strides, const long long* v_strides, int T,
                   const int32_t* n_new, void* q_out, const long long* out_strides, void* K, void* V,
                   const int32_t* pos, const float* cos, const float* sin, int n_angles, int rot,
                   int interleaved, const int32_t* angle_pos, const void* q_weight,
                   const void* k_weight, float eps, int B, int h_q, int h_kv, int d_k, int d_v,
                   int n_max, int dtype, int32_t* dev_error, cudaStream_t stream) {
  if (!K || !V || !pos || !cos || !sin || !q_strides || !k_strides || !v_strides || !out_strides)
    return DA_ERR_NULL;
  if (dtype != DA_FP32 && dtype != DA_BF16) return DA_ERR_DTYPE;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || T < 0 || n_max <= 0 || n_max > (1 << 30))
    return DA_ERR_SHAPE;
  if (n_angles <= 0 || rot <= 0 || rot > d_k || rot % 16 != 0) return DA_ERR_SHAPE;
  if (!isfinite(eps) || eps < 0.f) return DA_ERR_SHAPE;
  if ((long long)B * h_kv * (long long)n_max > 0x7fffffffLL) return DA_ERR_SHAPE;
  const bool sizes = (d_k == d_v && (d_k == 64 || d_k == 128 || d_k == 256)) ||
                     (d_k == 192 && d_v == 128);
  if (!sizes) return DA_ERR_UNSUPPORTED;
  if (T == 0) return DA_OK;
  // lanes of the launch (one to four heads for every 4 to 32 of them) in 32 bits
  if (T > (1 << 30) || (double)B * T * (h_q + 2.0 * h_kv) * 32.0 > 2147483647.0 * 128.0)
    return DA_ERR_SHAPE;
  if (!q || !k_new || !v_new || !q_out) return DA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) ||
      !aligned16(K) || !aligned16(V) || !aligned16(cos) || !aligned16(sin) ||
      !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(pos) || !aligned4(n_new) ||
      !aligned4(angle_pos))
    return DA_ERR_ALIGN;
  if (K == V || cos == sin) return DA_ERR_SHAPE;
  da::RopeAppendArgs a{};
  const long long* strides[4] = {q_strides, k_strides, v_strides, out_strides};
  const int heads[4] = {h_q, h_kv, h_kv, h_q}, widths[4] = {d_k, d_k, d_v, d_k};
  for (int x = 0; x < 4; ++x) {
    const long long shape[3] = {B, heads[x], T};
    long long last = widths[x];
    for (int i = 0; i < 3; ++i) {
      const int st = check_stride(strides[x][i], elem_size(dtype));
      if (st != DA_OK) return st;
      (x < 3 ? a.x_stride[x] : a.out_stride)[i] = strides[x][i];
      last += (shape[i] - 1) * strides[x][i];
    }
    (x < 3 ? a.x_elems[x] : a.out_elems) = last;
  }
  // no output over an input or another output, but q_out on q itself
  const int es = elem_size(dtype);
  const long long cache_rows = (long long)B * h_kv * n_max, angle_bytes = (long long)n_angles * rot * 2;
  const RowSet out[3] = {strided_rows(q_out, out_strides, B, h_q, T, d_k, es),
                         one_span(K, cache_rows * d_k * es), one_span(V, cache_rows * d_v * es)};
  const RowSet in[10] = {strided_rows(q, q_strides, B, h_q, T, d_k, es),
                         strided_rows(k_new, k_strides, B, h_kv, T, d_k, es),
                         strided_rows(v_new, v_strides, B, h_kv, T, d_v, es),
                         one_span(pos, 4LL * B),
                         one_span(n_new, 4LL * B),
                         one_span(angle_pos, 4LL * B),
                         one_span(cos, angle_bytes),
                         one_span(sin, angle_bytes),
                         one_span(q_weight, (long long)d_k * es),
                         one_span(k_weight, (long long)d_k * es)};
  bool in_place = q == q_out;
  for (int i = 0; i < 3; ++i) in_place = in_place && (out[0].n[i] == 1 || q_strides[i] == out_strides[i]);
  for (int y = 0; y < 3; ++y) {
    for (int x = 0; x < 10; ++x)
      if (!(x == 0 && y == 0 && in_place) && share_bytes(out[y], in[x])) return DA_ERR_SHAPE;
    for (int x = 0; x < y; ++x)
      if (share_bytes(out[y], out[x])) return DA_ERR_SHAPE;
  }
  int dev, sms;
  const int st = current_device(&dev, &sms);
  if (st != DA_OK) return st;
  a.x[0] = q, a.x[1] = k_new, a.x[2] = v_new;
  a.q_out = q_out;
  a.cache[0] = K, a.cache[1] = V;
  a.pos = pos, a.n_new = n_new, a.angle_pos = angle_pos, a.cos = cos, a.sin = sin;
  a.weight[0] = q_weight, a.weight[1] = k_weight;
  a.dev_error = dev_error;
  a.B = B, a.T = T, a.h_q = h_q, a.h_kv = h_kv, a.d_k = d_k, a.d_v = d_v, a.n_max = n_max;
  a.rot = rot, a.n_angles = n_angles, a.interleaved = interleaved != 0;
  a.bf16 = dtype == DA_BF16, a.sms = sms;
  a.eps = eps, a.inv_d = 1.f / float(d_k);
  const cudaError_t e = da::launch_kv_append_rope(a, stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv_append_rope launch");
  g_launches.fetch_add(1);
  return DA_OK;
}

namespace {
// The launches of chunk_attn and decode_attn_shared.
struct AttendPlan {
  int slice;                 // sequences per launch
  int q_tiles, prefix_tiles, list, ctas, pitch, unit_rows;
  long long units, part_rows, own_parts;
  size_t table_bytes;
  size_t bytes(int d) const {
    return list ? table_bytes + size_t(part_rows) * (size_t(d) + 1) * 4 : 0;
  }
};

// Sizes and types of both; P < 0: no shared prefix.  seen: rows that a unit sees at most (a
// workspace asked for without the window's is never too small: fewer rows, fewer cuts).
int plan_attend(int B, int T, int h_q, int h_kv, int d, int n_max, int dtype, int P, int sms,
                long long seen, AttendPlan* plan) {
  if ((dtype & DA_BF16_WEIGHTS) && !(dtype & DA_OUT_BF16)) return DA_ERR_DTYPE;
  dtype &= ~DA_BF16_WEIGHTS;
  DtypeArg dt;
  if (!parse_dtype(dtype, &dt)) return DA_ERR_DTYPE;
  if (dt.kv != DA_FP32 && dt.kv != DA_BF16) return DA_ERR_DTYPE;
  const int st = check_sizes(B, h_q, h_kv, d, d, n_max, dtype);
  if (st != DA_OK) return st;
  if (dt.kv != DA_BF16 || (d != 64 && d != 128)) return DA_ERR_UNSUPPORTED;
  if (T < 0 || T > (1 << 30)) return DA_ERR_SHAPE;
  if (T == 0) return *plan = AttendPlan{}, DA_OK;
  const long long g = h_q / h_kv, rows = T * g;
  // (query rows of a sequence, and of a batch behind a prefix, are counted in 32 bits)
  if (rows > (1LL << 30) || (P >= 0 && B * g > (1LL << 30))) return DA_ERR_SHAPE;
  AttendPlan a{};
  a.q_tiles = int((rows + da::kAttendRows - 1) / da::kAttendRows);
  a.slice = B;
  if (P >= 0) {
    const int most = (da::kAttendEntries - 1) / a.q_tiles;  // sequences whose entries fit a list
    if (most < 1) return DA_ERR_UNSUPPORTED;
    const int launches = (B + most - 1) / most;
    a.slice = (B + launches - 1) / launches;
    a.prefix_tiles = int((a.slice * g + da::kAttendRows - 1) / da::kAttendRows);
  }
  a.units = ((long long)a.slice * a.q_tiles + a.prefix_tiles) * h_kv;
  if (a.units > 0x7fffffffLL - 2 * sms) return DA_ERR_SHAPE;
  const long long entries = (long long)a.slice * a.q_tiles + (P >= 0 ? 1 : 0);
  // Cut into equal pieces, one per CTA, and merged: behind a prefix (whose partials are merged with
  // a sequence's own anyway), and of a chunk where whole units, taken one by one by CTAs that are
  // done, would end apart.  Cutting and merging costs 3 to 20 us, so not up to 16 tiles of rows
  // (5 tokens of 8 heads: 9.5 us whole and 11.6 cut behind 300 rows, 18.7 and 16.7 behind 2000; 64
  // sequences of 16 tokens, one of 2048 rows: 31 and 39; 1024 tokens with a window of 1024: 31 and
  // 49), nor where units are many beside the longest (prompts, 4 of 2048 tokens: 162 and 222, 2 of
  // 8192: 955 and 1040; the other side, 2 x 2048 tokens behind 6144 rows: 475 and 450).
  // Nor where a chunk has more entries (sequences times row tiles) than the schedule's list holds.
  const int most_tiles = (n_max + 127) / 128, prefix_most = P > 0 ? (P + 127) / 128 : 0;
  const bool whole = seen <= 16 * 128 || a.units * T >= sms * seen;
  a.list = P >= 0 || (!whole && entries <= da::kAttendEntries);
  a.pitch = int((P >= 0 ? a.slice * g : rows) < da::kAttendRows ? (P >= 0 ? a.slice * g : rows)
                                                                 : da::kAttendRows);
  a.unit_rows = int(rows < da::kAttendRows ? rows : da::kAttendRows);
  // a CTA per SM, but no more than pairs of tiles; without cuts one a unit, most of which are
  // taken over by CTAs that are done
  const long long pairs = (long long)a.slice * a.q_tiles * h_kv * ((most_tiles + 1) / 2) +
                          (long long)a.prefix_tiles * h_kv * ((prefix_most + 1) / 2);
  a.ctas = int(!a.list ? a.units : pairs < sms ? pairs : sms);
  if (P >= 0) {
    // a partial for each CTA of a unit; one number per unit and CTA, prefix units first
    const long long pre_units = (long long)a.prefix_tiles * h_kv;
    a.own_parts = (pre_units + a.ctas) * a.pitch;
    a.part_rows = a.own_parts + (a.units - pre_units + a.ctas) * a.unit_rows;
    if (a.part_rows > 0x7fffffffLL) return DA_ERR_SHAPE;
  } else {
    a.part_rows = 2LL * a.ctas * a.pitch;  // the first and the last unit of each CTA
  }
  a.table_bytes = ((size_t(a.ctas) * 16 + (P >= 0 ? size_t(a.units) * 8 : 0)) + 255) & ~size_t(255);
  *plan = a;
  return DA_OK;
}

size_t attend_workspace(int B, int T, int h_q, int h_kv, int d, int n_max, int dtype, int P,
                        int* status) {
  int dev, sms;
  AttendPlan plan{};
  // sizes first, so that a wrong call is told without a GPU
  int st = plan_attend(B, T, h_q, h_kv, d, n_max, dtype, P, 1, n_max, &plan);
  if (st == DA_OK) st = current_device(&dev, &sms);
  if (st == DA_OK) st = plan_attend(B, T, h_q, h_kv, d, n_max, dtype, P, sms, n_max, &plan);
  if (status) *status = st;
  return st == DA_OK ? plan.bytes(d) : 0;
}

struct AttendCall {
  const void *q, *K, *V, *K_prefix, *V_prefix;
  void* out;
  const long long *q_strides, *out_strides;
  const int32_t *seq_lens, *n_new;
  int B, T, h_q, h_kv, d, n_max, window, prefix, P, prefix_max, dtype;
  float scale;
};

int run_attend(const AttendCall& c, void* workspace, size_t workspace_bytes, int32_t* dev_error,
               cudaStream_t stream) {
  const bool shared = c.P >= 0;
  if (!c.K || !c.V || !c.seq_lens || !c.q_strides || !c.out_strides) return DA_ERR_NULL;
  if (shared && (!c.K_prefix || !c.V_prefix)) return DA_ERR_NULL;
  AttendPlan plan{};
  int st = plan_attend(c.B, c.T, c.h_q, c.h_kv, c.d, c.n_max, c.dtype, c.P, 1, c.n_max, &plan);
  if (st != DA_OK) return st;
  if (c.window < 0 || c.prefix < 0) return DA_ERR_SHAPE;
  const double scale_log2 = fabs(double(c.scale)) * 1.4426950408889634;
  if (!isfinite(c.scale) || scale_log2 > 3e38) return DA_ERR_SHAPE;
  if (shared && (c.prefix_max < 1 || c.P > c.prefix_max || c.prefix_max > (1 << 30) ||
                 (long long)c.h_kv * c.prefix_max > 0x7fffffffLL))
    return DA_ERR_SHAPE;
  if (c.T == 0) return DA_OK;
  if (!c.q || !c.out) return DA_ERR_NULL;
  if (!aligned16(c.q) || !aligned16(c.K) || !aligned16(c.V) || !aligned16(c.out) ||
      !aligned16(c.K_prefix) || !aligned16(c.V_prefix) || !aligned4(c.seq_lens) ||
      !aligned4(c.n_new))
    return DA_ERR_ALIGN;
  da::AttendParams p{};
  p.out_bf16 = (c.dtype & DA_OUT_BF16) != 0;
  p.bf16_weights = (c.dtype & DA_BF16_WEIGHTS) != 0;
  const long long shape[3] = {c.B, c.h_q, c.T};
  long long q_elems = c.d, out_elems = c.d;
  for (int i = 0; i < 3; ++i) {
    if ((st = check_stride(c.q_strides[i], 2)) != DA_OK) return st;
    if ((st = check_stride(c.out_strides[i], p.out_bf16 ? 2 : 4)) != DA_OK) return st;
    p.q_stride[i] = c.q_strides[i];
    p.out_stride[i] = c.out_strides[i];
    q_elems += (shape[i] - 1) * c.q_strides[i];
    out_elems += (shape[i] - 1) * c.out_strides[i];
  }
  if (!shared) {  // out over no input
    const RowSet out = strided_rows(c.out, c.out_strides, c.B, c.h_q, c.T, c.d, p.out_bf16 ? 2 : 4);
    const long long cache_bytes = (long long)c.B * c.h_kv * c.n_max * c.d * 2;
    if (share_bytes(out, strided_rows(c.q, c.q_strides, c.B, c.h_q, c.T, c.d, 2)) ||
        share_bytes(out, one_span(c.K, cache_bytes)) || share_bytes(out, one_span(c.V, cache_bytes)) ||
        share_bytes(out, one_span(c.seq_lens, 4LL * c.B)) || share_bytes(out, one_span(c.n_new, 4LL * c.B)))
      return DA_ERR_SHAPE;
  }
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != DA_OK) return st;
  // a window and its first rows, behind the first of a unit's tokens
  const long long seen = c.window == 0 ? c.n_max : (long long)c.window + c.prefix + da::kAttendRows;
  if ((st = plan_attend(c.B, c.T, c.h_q, c.h_kv, c.d, c.n_max, c.dtype, c.P, sms,
                        seen < c.n_max ? seen : c.n_max, &plan)) != DA_OK)
    return st;
  if (plan.list && (!workspace || workspace_bytes < plan.bytes(c.d))) return DA_ERR_WORKSPACE;
  if (plan.list && !aligned16(workspace)) return DA_ERR_ALIGN;
  da::AttendMaps maps;
  const KernelShape ks{128, 128, 64, 1, 1.f};
  if ((st = encode_cache_map(&maps.k, c.K, DA_BF16, c.d, c.n_max, c.B * c.h_kv, ks)) != DA_OK ||
      (st = encode_cache_map(&maps.v, c.V, DA_BF16, c.d, c.n_max, c.B * c.h_kv, ks)) != DA_OK)
    return st;
  maps.k_prefix = maps.k, maps.v_prefix = maps.v;
  if (shared &&
      ((st = encode_cache_map(&maps.k_prefix, c.K_prefix, DA_BF16, c.d, c.prefix_max, c.h_kv, ks)) !=
           DA_OK ||
       (st = encode_cache_map(&maps.v_prefix, c.V_prefix, DA_BF16, c.d, c.prefix_max, c.h_kv, ks)) !=
           DA_OK))
    return st;
  p.dev_error = dev_error;
  p.V = c.V;
  p.T = c.T, p.h_q = c.h_q, p.h_kv = c.h_kv, p.group = c.h_q / c.h_kv, p.n_max = c.n_max;
  // (positions plus a window stay inside 32 bits)
  p.window = c.window < (1 << 30) ? c.window : 1 << 30;
  p.prefix = c.prefix < (1 << 30) ? c.prefix : 1 << 30;
  if (p.window == 0) p.prefix = 0;  // every row up to the query's is seen
  p.shared = shared, p.P = shared ? c.P : 0;
  p.negate = c.scale < 0.f;
  p.scale_log2 = scale_log2 < 1.2e-38 ? 1.2e-38f : float(scale_log2);
  p.lazy = float(8.0 / double(p.scale_log2));
  p.single_read = plan.q_tiles == 1;
  p.list = plan.list, p.q_tiles = plan.q_tiles, p.ctas = plan.ctas;
  p.pitch = plan.pitch, p.unit_rows = plan.unit_rows, p.own_parts = int(plan.own_parts);
  p.part_rows = plan.part_rows;
  p.by_group = da::FastDiv(uint32_t(p.group));
  if (plan.list) {
    char* ws = static_cast<char*>(workspace);
    p.cta_start = reinterpret_cast<int4*>(ws);
    p.unit_ctas = reinterpret_cast<int2*>(ws + size_t(plan.ctas) * 16);
    p.o_part = reinterpret_cast<float*>(ws + plan.table_bytes);
    p.lse_part = p.o_part + plan.part_rows * c.d;
  }
#ifdef DA_TEST_HOOKS
  p.withhold_cta = g_test_withhold_cta.load();
#endif
  for (int b0 = 0; b0 < c.B; b0 += plan.slice) {
    p.B = c.B - b0 < plan.slice ? c.B - b0 : plan.slice;
    p.b_offset = b0;
    p.by_batch = da::FastDiv(uint32_t(p.B));
    p.q = static_cast<const char*>(c.q) + b0 * c.q_strides[0] * 2;
    p.out = static_cast<char*>(c.out) + b0 * c.out_strides[0] * (p.out_bf16 ? 2 : 4);
    // (from the launch's first sequence on)
    p.q_elems = q_elems - b0 * c.q_strides[0];
    p.out_elems = out_elems - b0 * c.out_strides[0];
    p.seq_lens = c.seq_lens + b0;
    p.n_new = c.n_new ? c.n_new + b0 : nullptr;
    p.prefix_tiles = shared ? (p.B * p.group + da::kAttendRows - 1) / da::kAttendRows : 0;
    p.entries = p.list ? p.B * p.q_tiles + p.shared : 0;
    cudaError_t e = da::launch_attend(p, maps, c.d, p.ctas, stream);
    if (e != cudaSuccess) return fail_cuda(e, "attend launch");
    g_launches.fetch_add(1);
    if (p.list && (p.shared || p.ctas > 1)) {
      e = da::launch_attend_combine(p, c.d, stream);
      if (e != cudaSuccess) return fail_cuda(e, "attend combine launch");
      g_launches.fetch_add(1);
    }
  }
  return DA_OK;
}
}  // namespace

size_t chunk_attn_workspace_bytes(int B, int T, int h_q, int h_kv, int d, int n_max, int dtype,
                                  int* status) {
  return attend_workspace(B, T, h_q, h_kv, d, n_max, dtype, -1, status);
}

int chunk_attn(const void* q, const long long* q_strides, int T, const int32_t* n_new, const void* K,
               const void* V, const int32_t* seq_lens, int window, int prefix, void* out,
               const long long* out_strides, int B, int h_q, int h_kv, int d, int n_max, float scale,
               int dtype, void* workspace, size_t workspace_bytes, int32_t* dev_error,
               cudaStream_t stream) {
  const AttendCall c{q,    K,    V,   nullptr, nullptr, out,    q_strides, out_strides, seq_lens, n_new,
                     B,    T,    h_q, h_kv,    d,       n_max,  window,    prefix,      -1,       0,
                     dtype, scale};
  return run_attend(c, workspace, workspace_bytes, dev_error, stream);
}

size_t decode_attn_shared_workspace_bytes(int B, int h_q, int h_kv, int d, int n_max,
                                          int prefix_len, int dtype, int* status) {
  if (prefix_len < 0) {
    if (status) *status = DA_ERR_SHAPE;
    return 0;
  }
  return attend_workspace(B, 1, h_q, h_kv, d, n_max, dtype, prefix_len, status);
}

int decode_attn_shared(const void* q, const void* K_prefix, const void* V_prefix, int prefix_len,
                       int prefix_max, const void* K, const void* V, const int32_t* seq_lens,
                       void* out, int B, int h_q, int h_kv, int d, int n_max, float scale, int dtype,
                       void* workspace, size_t workspace_bytes, int32_t* dev_error,
                       cudaStream_t stream) {
  if (prefix_len < 0) return DA_ERR_SHAPE;
  const long long strides[3] = {(long long)h_q * d, d, 0};  // q and out [B, h_q, d]
  const AttendCall c{q, K, V,   K_prefix, V_prefix, out,   strides, strides, seq_lens, nullptr,
                     B, 1, h_q, h_kv,     d,        n_max, 0,       0,       prefix_len, prefix_max,
                     dtype, scale};
  return run_attend(c, workspace, workspace_bytes, dev_error, stream);
}

int kv_quantize(const void* x, int x_dtype, void* codes, float* scales, long long rows, int d,
                int code_dtype, cudaStream_t stream) {
  if (!x || !codes || !scales) return DA_ERR_NULL;
  if ((x_dtype != DA_FP32 && x_dtype != DA_BF16) || !is_q8(code_dtype)) return DA_ERR_DTYPE;
  if (rows < 0 || d <= 0 || d % 32 != 0 || d > 256 || rows > (1LL << 33)) return DA_ERR_SHAPE;
  if (rows == 0) return DA_OK;
  int dev, sms;
  int st = current_device(&dev, &sms);
  if (st != DA_OK) return st;
  cudaError_t e = da::launch_kv_quantize(x, x_dtype == DA_BF16, codes, scales, rows, d,
                                         code_dtype == DA_INT8 ? 1 : 2, stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv_quantize launch");
  g_launches.fetch_add(1);
  return DA_OK;
}

}  // extern "C"
