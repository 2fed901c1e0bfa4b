// Attention of many query rows over cached rows on the fifth-generation tensor
// cores (tcgen05, TMEM accumulators), sm_103a: the kernel behind chunk_attn (the
// tokens of a chunk, causal, with a window and always-seen first rows) and
// decode_attn_shared (a batch behind a shared prefix).
//
// What is computed, for a query row r of a KV head that sees the rows L(r):
//   out[r] = sum_{l in L(r)} e^(s_l) V_l / sum_{l in L(r)} e^(s_l),  s_l = scale q_r . K_l
// A unit is up to 256 query rows of one KV head (the heads of a group and the
// tokens of a chunk, or the sequences of a batch, one after the other), taken as
// two streams of 128: the M of the MMAs.  K and V tiles of 128 rows are read once
// for both.
//
// Per tile and stream: S[128 x 128] = Q K^T into TMEM; a thread per query row
// loads its row, takes the maximum and the exponentials (no exchange between
// threads), and stores P as bf16 over S; O[128 x d] += P V with P read from TMEM.
// The MMAs of one stream run under the softmax of the other.  A running maximum
// may lag behind by 2^8 before O is rescaled in TMEM; every exponent is taken
// against the same maximum that scales O, so that changes nothing but rounding.
// P is rounded to bf16 (2^-8 of each weight, as the output is); with a float32
// output its bf16 remainder is multiplied as well (2^-16).
//
// A unit of at most 128 query rows (few tokens, one sequence's group) uses both
// streams for the same rows on alternate tiles and merges them at the end.
//
// Roles (384 threads): warps 0-3 and 4-7 the softmax of streams 0 and 1, warp 8
// the TMA producer, warp 9 the MMA issuer, warp 10 clears V rows that may hold
// anything.  TMEM: S 2 x 128 columns, O 2 x d.
#include <math.h>

#include "common.cuh"
#include "tc5.cuh"

namespace da {
namespace {

constexpr int kTile = 128;              // K and V rows of a tile, query rows of a stream
constexpr int kAttendThreads = 384;
constexpr int kScheduleThreads = 256;
constexpr int kEdges = 4;               // most tiles of an item with rows to clear (see edge_tile)

template <int D_>
struct AttendCfg {
  static constexpr int D = D_;
  static constexpr int kTileBytes = kTile * D * 2;  // Q of a stream, a K tile, a V tile
  static constexpr int kHalfBytes = kTile * 128;    // 64 columns of one
  static constexpr int kSlots = D == 128 ? 5 : 11;  // ring of K and V tiles
  // q_full[2], kv_full[slots], kv_empty[slots], s_full[2], p_full[2], o_full[2], edge[4], fin
  static constexpr int kBars = 2 + 2 * kSlots + 2 + 2 + 2 + kEdges + 1;
  static constexpr size_t kSmemBytes = 1024 + size_t(2 + kSlots) * kTileBytes + kBars * 8 + 256;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  // the schedule's scratch lies in the ring before the first load
  static_assert((kAttendEntries + 64) * 4 <= kTileBytes, "schedule scratch");
};

// What one CTA does: some tiles of a unit.  List tile k of a unit is tile k of
// the cache below `pt` (always-seen rows before the window) and tile
// first + k - pt from there on.
struct Item {
  int kvh, b;        // b < 0: the prefix
  int rows, row0;    // query rows, and the first among the sequence's (or the batch's)
  int n;             // rows of the sequence (or the prefix)
  int past;          // position of a sequence's token 0: token t sees rows up to past + t
  int pt, first, tiles;  // of the unit
  int begin, count;  // this item's list tiles
  int upto[2];       // tiles of it that each stream takes (from the first on)
  int clear_lo;      // rows of [prefix, clear_lo) and from n on are seen by no query of the sequence
  int slot;          // partial, or -1: the unit's only item writes the output
};

__device__ __forceinline__ int seq_rows(const AttendParams& p, int b, bool& bad) {
  const int n = p.seq_lens[b];
  bad = n < 0 || n > p.n_max;
  return min(max(n, 0), p.n_max);
}
__device__ __forceinline__ int seq_new(const AttendParams& p, int b, bool& bad) {
  const int m = p.n_new ? p.n_new[b] : p.T;
  bad = m < 0 || m > p.T;
  return min(max(m, 0), p.T);
}

// First cached row of list tile k.
__device__ __forceinline__ int tile_row(const Item& w, int k) {
  return (k < w.pt ? k : w.first + k - w.pt) * kTile;
}

// Whether the V tile at row r0 holds rows that no query of the sequence sees: they
// may hold anything, even NaN, and a weight of zero times NaN is NaN, so they are
// cleared.  In the tiles of an item that is the end of the always-seen rows, the
// window's first tile and the last tile.
__device__ __forceinline__ bool edge_tile(const AttendParams& p, const Item& w, int r0) {
  return r0 + kTile > w.n || (r0 < w.clear_lo && r0 + kTile > p.prefix);
}

// Unit of row tile qt of a sequence of n rows, the last m of them new.
__device__ __forceinline__ void seq_unit(const AttendParams& p, int n, int m, int qt, Item& w) {
  const long long rows = (long long)m * p.group - (long long)qt * kAttendRows;
  w.rows = rows <= 0 ? 0 : int(rows < kAttendRows ? rows : kAttendRows);
  w.row0 = qt * kAttendRows;
  w.n = n;
  w.past = n - m;
  w.pt = w.first = w.tiles = 0;
  if (w.rows == 0) return;
  const int hi = w.past + p.by_group.div(w.row0 + w.rows - 1);
  if (hi < 0) return;
  if (p.window) {
    w.first = max(0, w.past + p.by_group.div(w.row0) + 1 - p.window) / kTile;
    w.pt = min(min((p.prefix + kTile - 1) / kTile, hi / kTile + 1), w.first);
  }
  w.tiles = w.pt + hi / kTile - w.first + 1;
}

// The rest of an item, tiles [begin, end) of its unit.
__device__ __forceinline__ void cut_item(const AttendParams& p, int begin, int end, int slot,
                                         Item& w) {
  w.begin = begin;
  w.count = end - begin;
  w.slot = slot;
  w.clear_lo = w.b >= 0 && p.window ? max(0, w.past + 1 - p.window) : 0;
  w.upto[0] = w.upto[1] = w.count;
  if (w.b >= 0 && w.rows > kTile) {  // stream 0 ends at its last query's row
    const int hi = w.past + p.by_group.div(w.row0 + kTile - 1);
    const int tiles = hi < 0 ? 0 : w.pt + hi / kTile - w.first + 1;
    w.upto[0] = min(max(tiles - begin, 0), w.count);
  }
}

// Entry e of the list: the prefix (with a shared one), then row tile by row tile
// from the last (in a chunk the longest) down, every sequence of it.
__device__ __forceinline__ void entry_of(const AttendParams& p, int e, int& b, int& qt) {
  e -= p.shared;
  const int up = p.by_batch.div(e);
  qt = p.q_tiles - 1 - up;
  b = e - up * p.B;
}

// The unit of an entry; false: it has no part.
__device__ __forceinline__ bool entry_unit(const AttendParams& p, int e, Item& w) {
  if (p.shared && e == 0) {
    w.b = -1;
    w.n = p.P;
    w.tiles = (p.P + kTile - 1) / kTile;
    return p.P > 0;
  }
  int qt;
  entry_of(p, e, w.b, qt);
  bool bad;
  const int n = seq_rows(p, w.b, bad);
  seq_unit(p, n, seq_new(p, w.b, bad), qt, w);
  // (behind a prefix a sequence without rows has no part)
  return w.rows > 0 && (w.tiles > 0 || !p.shared);
}

__device__ __forceinline__ int entry_units(const AttendParams& p, int e) {
  return p.h_kv * (p.shared && e == 0 ? p.prefix_tiles : 1);
}

// The list: every unit is cut into ceil(tiles / c) items of equal length, with one c
// for the whole launch, the one that ends first by a simple model (rounds of the
// grid times the tiles of an item and a constant for its start and end).  All
// CTAs compute the same list from the lengths; CTA 0 leaves the table for the
// combine.  Returns false for a CTA without an item.  Ends with a barrier.
constexpr int kScheduleWarps = kScheduleThreads / 32;
constexpr int kLengthChoices = 2 * kScheduleWarps;
constexpr float kItemTiles = 5.f;  // an item's fixed cost in tiles

__device__ __forceinline__ bool list_item(const AttendParams& p, int* scratch, Item* out) {
  int* tiles = scratch;                       // [kAttendEntries], -1: absent
  int* sums = scratch + kAttendEntries;       // [64]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool mine = tid < kScheduleThreads;
  float total = 0.f;
  int tallest = 0;
  if (mine)
    for (int e = tid; e < p.entries; e += kScheduleThreads) {
      Item w;
      const bool present = entry_unit(p, e, w);
      tiles[e] = present ? w.tiles : -1;
      if (present) {
        total += float(w.tiles) * float(entry_units(p, e));
        tallest = max(tallest, w.tiles);
      }
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    tallest = max(tallest, __shfl_xor_sync(0xffffffffu, tallest, o));
  }
  if (lane == 0 && mine) {
    sums[warp] = __float_as_int(total);
    sums[kScheduleWarps + warp] = tallest;
  }
  if (tid == 0) out->count = -1;
  __syncthreads();
  total = 0.f;
#pragma unroll
  for (int i = 0; i < kScheduleWarps; ++i) {
    total += __int_as_float(sums[i]);
    tallest = max(tallest, sums[kScheduleWarps + i]);
  }
  // two lengths a warp: the items there would be
  if (mine) {
    const float share = total / float(p.sms);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // from half an even share to 2.4 of them, in steps of 2^(3/20)
      const int c = max(2, int(ceilf(share * exp2f(float(warp + k * kScheduleWarps) * 0.15f - 1.f))));
      const float inv = 1.f / float(c);
      int items = 0;
      for (int e = lane; e < p.entries; e += 32) {
        const int t = tiles[e];
        if (t >= 0) items += max(1, int(ceilf(float(t) * inv))) * entry_units(p, e);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
      const float longest = float(min(c, tallest)) + kItemTiles;
      const float mean = (total + kItemTiles * float(items)) / float(p.sms);
      const float t = fmaxf(fminf(ceilf(float(items) / float(p.sms)) * longest, mean + longest), mean);
      if (lane == 0) {
        sums[2 * kScheduleWarps + warp + k * kScheduleWarps] = __float_as_int(t);
        sums[2 * kScheduleWarps + kLengthChoices + warp + k * kScheduleWarps] = c;
      }
    }
  }
  __syncthreads();
  float best = 1e30f;
  int c = 2;
#pragma unroll
  for (int i = 0; i < kLengthChoices; ++i) {
    const float t = __int_as_float(sums[2 * kScheduleWarps + i]);
    if (t <= best) best = t, c = sums[2 * kScheduleWarps + kLengthChoices + i];
  }
  // first item of every entry: four consecutive entries a thread
  constexpr int kPer = kAttendEntries / kScheduleThreads;
  int cut[kPer], own = 0;
  if (mine)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      const int t = e < p.entries ? tiles[e] : -1;
      cut[i] = t < 0 ? 0 : max(1, (t + c - 1) / c);
      own += e < p.entries ? cut[i] * entry_units(p, e) : 0;
    }
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31 && mine) sums[warp] = upto;
  __syncthreads();
  if (mine) {
    int at = upto - own;
    for (int i = 0; i < warp; ++i) at += sums[i];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e >= p.entries) break;
      const int items = cut[i] * entry_units(p, e);
      const int x = int(blockIdx.x) - at;
      if (blockIdx.x == 0) p.table[e] = make_int2(at, cut[i]);
      if (x >= 0 && x < items && int(blockIdx.x) < p.max_items) {  // this CTA's
        Item w;
        entry_unit(p, e, w);
        const int unit = x / cut[i], s = x - unit * cut[i];
        if (w.b < 0) {
          w.kvh = unit / p.prefix_tiles;
          w.row0 = (unit - w.kvh * p.prefix_tiles) * kAttendRows;
          w.rows = min(p.B * p.group - w.row0, kAttendRows);
          w.past = w.n - 1;
          w.pt = w.first = 0;
        } else {
          w.kvh = unit;
        }
        cut_item(p, int((long long)w.tiles * s / cut[i]), int((long long)w.tiles * (s + 1) / cut[i]),
                 cut[i] == 1 && !p.shared ? -1 : int(blockIdx.x), w);
        *out = w;
      }
      at += items;
    }
  }
  fence_proxy_async_smem();  // the scratch is the ring's: before its first loads
  __syncthreads();
  return out->count >= 0;
}

// Without a list: one item per unit, the last row tiles, the longest of a chunk, first.
__device__ __forceinline__ bool unit_item(const AttendParams& p, Item* out) {
  if (threadIdx.x == 0) {
    const int per = p.B * p.h_kv;
    const int up = int(blockIdx.x) / per, rest = int(blockIdx.x) - up * per;
    Item w;
    w.b = rest / p.h_kv;
    w.kvh = rest - w.b * p.h_kv;
    bool bad;
    const int n = seq_rows(p, w.b, bad);
    seq_unit(p, n, seq_new(p, w.b, bad), p.q_tiles - 1 - up, w);
    cut_item(p, 0, w.tiles, -1, w);
    if (w.rows == 0) w.count = -1;
    *out = w;
  }
  __syncthreads();
  return out->count >= 0;
}

// 32 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// D (TMEM) += A (TMEM: lane = row, two bf16 of K a column) . B (smem), fp32 accumulators.
__device__ __forceinline__ void mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// Two floats at a time.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void halves_of(uint64_t v, float& lo, float& hi) {
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

// A place of the ring: the producer and the MMA issuer pass through it in one order.
template <int SLOTS>
struct RingPlace {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SLOTS) slot = 0, phase ^= 1u;
  }
};

template <class Cfg, bool WIDE_P>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendMaps maps, const AttendParams p) {
  constexpr int D = Cfg::D;
  constexpr int kSlots = Cfg::kSlots, kTileBytes = Cfg::kTileBytes, kHalfBytes = Cfg::kHalfBytes;
  constexpr uint32_t kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_tile = smem;                            // [2]
  uint8_t* ring = smem + 2 * kTileBytes;             // [kSlots]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + size_t(kSlots) * kTileBytes);
  Item* item = reinterpret_cast<Item*>(bars + Cfg::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t q_full0 = smem_u32(bars);
  const uint32_t full0 = q_full0 + 16;
  const uint32_t empty0 = full0 + 8 * kSlots;
  const uint32_t s_full0 = empty0 + 8 * kSlots;
  const uint32_t p_full0 = s_full0 + 16;
  const uint32_t o_full0 = p_full0 + 16;
  const uint32_t edge0 = o_full0 + 16;
  const uint32_t fin = edge0 + 8 * kEdges;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full0 + 8 * i, 4);  // the softmax warps of the stream (see `arrivals`)
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(p_full0 + 8 * i, 4);
      mbar_init(o_full0 + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);   // released by one tcgen05.commit
    }
    for (int i = 0; i < kEdges; ++i) mbar_init(edge0 + 8 * i, 1);
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tc5::alloc(smem_u32(tmem_slot), kTmemCols);
    tc5::relinquish();
  }
  if (threadIdx.x == 8 * 32) {
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    if (p.shared) {
      prefetch_tmap(&maps.k_prefix);
      prefetch_tmap(&maps.v_prefix);
    }
  }
  tc5::fence_before();
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  const bool has = p.list ? list_item(p, reinterpret_cast<int*>(ring), item) : unit_item(p, item);
  // lengths that were clamped are reported
  if (blockIdx.x == 0 && p.dev_error)
    for (int b = threadIdx.x; b < p.B; b += kAttendThreads) {
      bool bad_n, bad_m;
      const int n = seq_rows(p, b, bad_n), m = seq_new(p, b, bad_m);
      if (bad_n || bad_m || (m > n && !p.shared)) flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
    }
  tc5::fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!has) {
    if (warp == 9) tc5::dealloc(tmem, kTmemCols);
    return;
  }
  const int count = item->count;
  const bool alternate = item->rows <= kTile;    // one set of rows, tiles dealt to the streams in turn
  const int ahead = alternate ? 2 : 1;           // tiles whose scores are issued before the first P.V
  auto give_up = [&] {
    if (!*abort_flag) {
      *abort_flag = 1;
      flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
    }
  };

  // Registers: 168 a thread at launch for each of three warpgroups; 2 * 208 + 88 then.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // ---------------------------------------------------------------- producer
    if (warp == 8) {
      if (lane == 0) {
        const bool pre = item->b < 0;
        const uint64_t policy = p.single_read || (pre && p.prefix_tiles == 1)
                                    ? l2_policy_evict_first()
                                    : l2_policy_evict_normal();
        const CUtensorMap* mk = pre ? &maps.k_prefix : &maps.k;
        const CUtensorMap* mv = pre ? &maps.v_prefix : &maps.v;
        const int z = pre ? item->kvh : (p.b_offset + item->b) * p.h_kv + item->kvh;
        const uint32_t ring0 = smem_u32(ring);
        RingPlace<kSlots> at;
        uint32_t issued = 0, parity = 0;  // per slot: loaded at all, phase of its newest load
        int edges = 0;
        bool ok = true;
        auto load = [&](const CUtensorMap* map, int j) {
          if (!ok) return;
          if (!mbar_wait_bounded(empty0 + 8 * at.slot, at.phase ^ 1u, abort_flag)) {
            give_up();
            ok = false;
            return;
          }
#ifdef DA_TEST_HOOKS
          if (int(blockIdx.x) == p.withhold_cta && map == mv && j == count - 1) return;
#endif
          const uint32_t dst = ring0 + at.slot * kTileBytes;
          const int y = tile_row(*item, item->begin + j);
          // a V tile with rows to clear goes to warp 10 first, which says when it is full
          const bool edge = map == mv && edges < kEdges && edge_tile(p, *item, y);
          const uint32_t bar = edge ? edge0 + 8 * edges++ : full0 + 8 * at.slot;
          mbar_arrive_expect_tx(bar, kTileBytes);
#pragma unroll
          for (int c = 0; c < D; c += 64)
            tma_load_3d(dst + (c / 64) * kHalfBytes, map, c, y, z, bar, policy);
          issued = edge ? issued & ~(1u << at.slot) : issued | 1u << at.slot;
          parity = (parity & ~(1u << at.slot)) | (at.phase << at.slot);
          at.next();
        };
        // loads follow their use: K of the first `ahead` tiles, then V_j and K_(j + ahead)
        for (int j = 0; j < min(ahead, count); ++j) load(mk, j);
        for (int j = 0; j < count; ++j) {
          load(mv, j);
          if (j + ahead < count) load(mk, j + ahead);
        }
        if (!ok) {  // copies in flight land before the CTA ends
          volatile int never = 0;
          for (int i = 0; i < kSlots; ++i)
            if (issued >> i & 1) mbar_wait_bounded(full0 + 8 * i, (parity >> i) & 1, &never);
          for (int i = 0; i < edges; ++i) mbar_wait_bounded(edge0 + 8 * i, 0, &never);
        }
      }
      return;
    }
    // ---------------------------------------------------------------- MMA issuer
    if (warp == 9) {
      if (lane == 0) {
        const uint32_t idesc_s = tc5::idesc_bf16(128, 128, 0, 0);
        const uint32_t idesc_o = tc5::idesc_bf16(128, D, 0, 1);
        // descriptors of the operands' first bytes; their addresses count 16 bytes
        const uint64_t k_major = tc5::sdesc(0, 16, 1024), mn_major = tc5::sdesc(0, kHalfBytes, 1024);
        const uint32_t q_at = smem_u32(q_tile) >> 4, ring_at = smem_u32(ring) >> 4;
        const int upto0 = item->upto[0], upto1 = item->upto[1];
        bool ok = true, any = false;
        uint32_t p_phase = 0;                     // a bit for each stream
        uint32_t started = 0;                     // streams with a P.V issued
        RingPlace<kSlots> at;
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (ok && !mbar_wait_bounded(bar, parity, abort_flag)) {
            give_up();
            ok = false;
          }
          return ok;
        };
        auto scores = [&](int i, int slot) {  // S_i = Q_i K^T
          tc5::fence_after();
          const uint64_t a = k_major + q_at + (alternate ? 0 : i * (kTileBytes >> 4));
          const uint64_t b = k_major + ring_at + slot * (kTileBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
            tc5::mma(tmem + i * 128, a + off, b + off, idesc_s, ks > 0);
          }
          tc5::commit(s_full0 + 8 * i);
          any = true;
        };
        if (count > 0 && wait(q_full0, 0) && !alternate) wait(q_full0 + 8, 0);
        for (int j = 0; j < min(ahead, count) && ok; ++j) {
          if (!wait(full0 + 8 * at.slot, at.phase)) break;
          if (alternate) {
            scores(j, at.slot);
          } else {
            if (j < upto0) scores(0, at.slot);
            if (j < upto1) scores(1, at.slot);
          }
          tc5::commit(empty0 + 8 * at.slot);
          at.next();
        }
        for (int j = 0; j < count && ok; ++j) {
          const RingPlace<kSlots> v = at;         // V_j
          at.next();
          const bool more = j + ahead < count;
          if (!wait(full0 + 8 * v.slot, v.phase)) break;
          bool k_here = false;
          const int i_end = alternate ? (j & 1) + 1 : 2;
          for (int i = alternate ? j & 1 : 0; i < i_end; ++i) {
            const int mine = alternate ? count : i == 0 ? upto0 : upto1;
            if (j < mine) {
              if (!wait(p_full0 + 8 * i, (p_phase >> i) & 1)) break;
              p_phase ^= 1u << i;
              tc5::fence_after();
              const uint64_t b = mn_major + ring_at + v.slot * (kTileBytes >> 4);
              const uint32_t o = tmem + 256 + i * D, pa = tmem + i * 128;
              const bool more_o = (started >> i) & 1;
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                mma_tmem_a(o, pa + ks * 8, b + ks * (16 * 128 >> 4), idesc_o, more_o || ks > 0);
              if constexpr (WIDE_P) {
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                  mma_tmem_a(o, pa + 64 + ks * 8, b + ks * (16 * 128 >> 4), idesc_o, 1);
              }
              started |= 1u << i;
            }
            if (j + ahead < mine) {
              if (!k_here && !wait(full0 + 8 * at.slot, at.phase)) break;
              k_here = true;
              scores(i, at.slot);
            }
          }
          if (!ok) break;
          tc5::commit(empty0 + 8 * v.slot);
          if (more) {
            tc5::commit(empty0 + 8 * at.slot);
            at.next();
          }
        }
        if (ok && any) {
          tc5::commit(o_full0);
          tc5::commit(o_full0 + 8);
        }
        // every MMA has completed before TMEM is freed
        if (any) tc5::commit(fin);
        else mbar_arrive(fin);
        volatile int never = 0;
        mbar_wait_bounded(fin, 0, &never);
      }
      __syncwarp();
      named_bar_sync(2, 288);
      tc5::fence_after();
      tc5::dealloc(tmem, kTmemCols);
      return;
    }
    // ---------------------------------------------------------------- clearing V
    if (warp == 10) {
      int edges = 0;
      for (int j = 0; j < count && edges < kEdges; ++j) {
        const int r0 = tile_row(*item, item->begin + j);
        if (!edge_tile(p, *item, r0)) continue;
        const bool got = mbar_wait_bounded(edge0 + 8 * edges++, 0, abort_flag);
        if (!got) give_up();
        if (!__all_sync(0xffffffffu, got)) break;
        const int slot = (j + min(count, ahead + j)) % kSlots;  // V_j in the order of the loads
        uint8_t* vt = ring + size_t(slot) * kTileBytes;
        const int seen_end = item->n, clear_lo = item->clear_lo;
        constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll 8
        for (int x = lane; x < kTile * kChunks; x += 32) {
          const int row = r0 + x / kChunks;
          if (row >= seen_end || (row < clear_lo && row >= p.prefix))
            *reinterpret_cast<uint4*>(vt + tc5::sw128(x / kChunks, (x % kChunks) * 8, kTile)) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8 * slot);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ softmax
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  const int i = warp >> 2;                          // stream
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;                // row of the stream = TMEM lane
  const uint32_t lanes = uint32_t(quarter * 32) << 16;
  const uint32_t s_col = tmem + i * 128 + lanes, o_col = tmem + 256 + i * D + lanes;
  const int rows = alternate ? item->rows : min(item->rows - i * kTile, kTile);
  // Warps without a query row stay out (their rows of S, P and O are never
  // looked at); the stream's first warp arrives for them.
  const bool works = quarter * 32 < rows;
  const uint32_t arrivals = quarter == 0 ? 4 - (rows - 1) / 32 : 1;
  const bool valid = r < rows;
  const int unit_row = (alternate ? 0 : i * kTile) + r;
  // this row's token, head and position
  int hi = -1, lo = 0;
  long long out_off = 0;
  bool live = works;
  float m_run = -INFINITY, l_run = 0.f;
  int done = 0;  // tiles of this stream
  if (works) {
    const bool pre = item->b < 0;
    long long q_off = 0;
    if (valid) {
      const int flat = item->row0 + unit_row;
      const int t = p.by_group.div(flat), head = item->kvh * p.group + flat - t * p.group;
      const int b = pre ? t : item->b, tok = pre ? 0 : t;
      hi = item->past + tok;
      lo = pre || !p.window ? 0 : hi + 1 - p.window;
      q_off = b * p.q_stride[0] + head * p.q_stride[1] + tok * p.q_stride[2];
      out_off = b * p.out_stride[0] + head * p.out_stride[1] + tok * p.out_stride[2];
    }
    if (!(alternate && i == 1)) {
      // Q of the warp's rows, swizzled K-major
      constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows at a time
      uint4 v[32 / kPer];
      const uint4* q = static_cast<const uint4*>(p.q);
#pragma unroll
      for (int k = 0; k < 32 / kPer; ++k) {
        const int row = k * kPer + lane / kChunks;
        const long long off = __shfl_sync(0xffffffffu, q_off, row);
        const bool in = quarter * 32 + row < rows && DA_IN(p, off + D - 1, p.q_elems);
        v[k] = in ? q[off / 8 + lane % kChunks] : make_uint4(0, 0, 0, 0);
      }
      const uint32_t flip = p.q_flip == 1 ? 0x80008000u : 0u, keep = p.q_flip == 2 ? 0u : ~0u;
#pragma unroll
      for (int k = 0; k < 32 / kPer; ++k) {
        const int row = quarter * 32 + k * kPer + lane / kChunks;
        *reinterpret_cast<uint4*>(q_tile + i * kTileBytes + tc5::sw128(row, (lane % kChunks) * 8, kTile)) =
            make_uint4((v[k].x ^ flip) & keep, (v[k].y ^ flip) & keep, (v[k].z ^ flip) & keep,
                       (v[k].w ^ flip) & keep);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_n(q_full0 + 8 * i, arrivals);
    }
    // Tiles from here on need the mask: rows past the stream's first query, and of the
    // window's start up to its last query's.
    const int row_last = item->row0 + (alternate ? 0 : i * kTile) + rows - 1;
    const int row_first = item->row0 + (alternate ? 0 : i * kTile);
    const int hi_first = pre ? item->past : item->past + p.by_group.div(row_first);
    const int lo_last =
        pre || !p.window ? 0 : max(0, item->past + p.by_group.div(row_last) + 1 - p.window);

    const int end = item->upto[i], step = alternate ? 2 : 1;
    for (int j = alternate ? i : 0; j < end; j += step) {
      const bool got = mbar_wait_bounded(s_full0 + 8 * i, done & 1, abort_flag);
      if (!got) give_up();
      live = __all_sync(0xffffffffu, got);  // warp-uniform: the TMEM accesses are .sync.aligned
      if (!live) break;
      tc5::fence_after();
      uint32_t raw[128];
      float* s = reinterpret_cast<float*>(raw);
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_ld32(s_col + c, raw + c);
      const int r0 = tile_row(*item, item->begin + j);
      tc5::wait_ld();
      if (r0 + kTile - 1 > hi_first || (r0 < lo_last && r0 + kTile > p.prefix)) {
        const int hi_c = hi - r0, lo_c = lo - r0, pre_c = p.prefix - r0;
#pragma unroll
        for (int c = 0; c < 128; ++c) {
          const bool seen = c <= hi_c && (c >= lo_c || c < pre_c);
          s[c] = seen ? s[c] : -INFINITY;
        }
      }
      float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 124; c += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(fmaxf(m4[k], s[c + k]), s[c + 4 + k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], s[124 + k]);
      const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      const bool over = m_tile > m_run + p.lazy || (m_run == -INFINITY && m_tile > -INFINITY);
      if (__any_sync(0xffffffffu, over)) {
        const float m_new = over ? m_tile : m_run;
        const float alpha = over ? ex2((m_run - m_new) * p.scale_log2) : 1.f;  // 0 from -inf
        m_run = m_new;
        l_run *= alpha;
        if (done > 0) {  // (S of this tile was issued behind the P.V of the last)
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_col + c, o);
            tc5::wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(o_col + c, o);
          }
        }
      }
      const float shift = m_run == -INFINITY ? 0.f : -m_run * p.scale_log2;
      const uint64_t scale2 = pair_of(p.scale_log2, p.scale_log2), shift2 = pair_of(shift, shift);
      uint64_t l2[2] = {0, 0};
      // exponentials in halves of 64 columns; P over the first columns of S, which
      // every lane of the warp has loaded
#pragma unroll
      for (int h = 0; h < 128; h += 64) {
        uint32_t hi_p[32];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float a, b;
          halves_of(fma2(pair_of(s[h + c], s[h + c + 1]), scale2, shift2), a, b);
          a = ex2(a);
          b = ex2(b);
          l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], pair_of(a, b));
          hi_p[c / 2] = pack_bf16x2(a, b);
          if constexpr (WIDE_P) {
            s[h + c] = a - bf16_lo_to_f32(hi_p[c / 2]);
            s[h + c + 1] = b - bf16_hi_to_f32(hi_p[c / 2]);
          }
        }
        tmem_st32(s_col + h / 2, hi_p);
        if constexpr (WIDE_P) {
          uint32_t lo_p[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) lo_p[c / 2] = pack_bf16x2(s[h + c], s[h + c + 1]);
          tmem_st32(s_col + 64 + h / 2, lo_p);
        }
      }
      float la, lb;
      halves_of(add2(l2[0], l2[1]), la, lb);
      l_run += la + lb;
      tc5::wait_st();
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_n(p_full0 + 8 * i, arrivals);
      ++done;
    }
  }

  // ---- the unit's rows are final once both streams' MMAs are
  if (live && count > 0) {
    bool got = mbar_wait_bounded(o_full0, 0, abort_flag);
    got = mbar_wait_bounded(o_full0 + 8, 0, abort_flag) && got;
    if (!got) give_up();
    live = __all_sync(0xffffffffu, got);
    tc5::fence_after();
  }
  // (a CTA whose wait ran out writes nothing)
  float* other = reinterpret_cast<float*>(ring);  // alternate: O^T [D][128], m [128], l [128] of stream 1
  const bool with_other = alternate && count > 1;
  if (with_other) {
    if (i == 1 && live) {
#pragma unroll 2
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_col + c, o);
        tc5::wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) other[(c + k) * kTile + r] = __uint_as_float(o[k]);
      }
      other[D * kTile + r] = m_run;
      other[D * kTile + kTile + r] = l_run;
    }
    named_bar_sync(1, 256);
    if (*abort_flag) live = false;
    live = __all_sync(0xffffffffu, live);
  }
  if (live && !(alternate && i == 1)) {
    float keep0 = 1.f, keep1 = 0.f;  // weights of the two streams' O
    if (with_other) {
      const float m1 = other[D * kTile + r], l1 = other[D * kTile + kTile + r];
      const float m = fmaxf(m_run, m1), m_use = m == -INFINITY ? 0.f : m;
      keep0 = ex2((m_run - m_use) * p.scale_log2);
      keep1 = ex2((m1 - m_use) * p.scale_log2);
      l_run = l_run * keep0 + l1 * keep1;
      m_run = m;
    }
    const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
    keep0 *= inv;
    keep1 *= inv;
    const bool part = item->slot >= 0;
    const long long part_row = (long long)item->slot * p.pitch + unit_row;
    if (part) out_off = part_row * D;
    const long long extent = part ? (long long)p.max_items * p.pitch * D : p.out_elems;
    if (part && valid && DA_IN(p, part_row, (long long)p.max_items * p.pitch))
      p.lse_part[part_row] =
          l_run > 0.f ? m_run * p.scale_log2 + log2f(l_run) : (l_run == 0.f ? -INFINITY : l_run);
    const bool narrow = !part && p.out_bf16;
    uint8_t* stage = q_tile + i * kTileBytes + quarter * (kTileBytes / 4);  // 32 rows of 2 D bytes
    constexpr int kChunks = D / 8, kPer = 32 / kChunks;
    const int mine = min(rows - quarter * 32, 32);  // rows of this warp
    // a row of 2 D bytes at a time (D bf16 or D / 2 floats) through shared memory,
    // so that whole rows are written
    const int cols = narrow ? D : D / 2;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += cols) {
#pragma unroll 2
      for (int c = 0; c < cols; c += 32) {
        uint32_t o[32];
        if (done > 0) {
          tmem_ld32(o_col + c0 + c, o);
          tc5::wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x = __uint_as_float(o[k]) * keep0;
          if (with_other) x = fmaf(other[(c0 + c + k) * kTile + r], keep1, x);
          o[k] = __float_as_uint(x);
        }
        if (narrow) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const float* f = reinterpret_cast<const float*>(o) + k;
            *reinterpret_cast<uint4*>(stage + lane * 2 * D + ((((c + k) / 8) ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                           pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<uint4*>(stage + lane * 2 * D + ((((c + k) / 4) ^ (lane & 7)) << 4)) =
                make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < mine; k += kPer) {
        const int row = k + lane / kChunks, ch = lane % kChunks;
        const long long off = __shfl_sync(0xffffffffu, out_off, row);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 2 * D + ((ch ^ (row & 7)) << 4));
        if (row < mine && DA_IN(p, off + D - 1, extent)) {
          if (narrow)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + off + ch * 8) = v;
          else
            *reinterpret_cast<uint4*>((part ? p.o_part : static_cast<float*>(p.out)) + off + c0 +
                                      ch * 4) = v;
        }
      }
      __syncwarp();
    }
  }
  tc5::fence_before();
  named_bar_sync(2, 288);
}

// ---------------------------------------------------------------------------
// Combine: a warp per query row merges the partials of its unit's items (and,
// behind a shared prefix, of the prefix unit's) by their log-sum-exps.  Rows
// whose unit had one item are skipped: it wrote them.
// ---------------------------------------------------------------------------
constexpr int kAttendCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kAttendCombineWarps * 32)
    attend_combine_kernel(const AttendParams p) {
  constexpr int EPL = D / 32, NB = 8;  // columns a lane, partials in flight
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * kAttendCombineWarps;
  // rows as [entry][kv head][row of the unit]
  const long long all = (long long)p.B * p.q_tiles * p.h_kv * p.unit_rows;
  for (long long x = (long long)blockIdx.x * kAttendCombineWarps + (threadIdx.x >> 5); x < all;
       x += warps) {
    const int ur = int(x % p.unit_rows);
    const int kvh = int(x / p.unit_rows % p.h_kv);
    const int e = int(x / p.unit_rows / p.h_kv) + p.shared;
    const int2 at = __ldcg(p.table + e);
    if (!p.shared && at.y <= 1) continue;
    int b, qt;
    entry_of(p, e, b, qt);
    bool bad;
    const long long flat = (long long)qt * kAttendRows + ur;
    if (flat >= (long long)(p.shared ? 1 : seq_new(p, b, bad)) * p.group) continue;
    const int t = int(flat / p.group), h = int(flat % p.group);
    // the partials: `first` of the prefix, then those of the sequence
    long long pre_row = 0, own_row = ((long long)at.x + (long long)kvh * at.y) * p.pitch + ur;
    int pre = 0;
    if (p.shared) {
      const int2 pt = __ldcg(p.table);
      const long long pr = (long long)b * p.group + flat;
      const int mt = int(pr / kAttendRows);
      pre = pt.y;
      pre_row = ((long long)pt.x + ((long long)kvh * p.prefix_tiles + mt) * pt.y) * p.pitch +
                pr % kAttendRows;
    }
    const int parts = pre + at.y;
    float m = -INFINITY, sum = 0.f, acc[EPL];
#pragma unroll
    for (int k = 0; k < EPL; ++k) acc[k] = 0.f;
    for (int s0 = 0; s0 < parts; s0 += NB) {
      float l[NB], v[NB][EPL];
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int s = s0 + u;
        const long long row = s < pre ? pre_row + (long long)s * p.pitch
                                      : own_row + (long long)(s - pre) * p.pitch;
        const bool in = s < parts && DA_IN(p, row, (long long)p.max_items * p.pitch);
        l[u] = in ? __ldcg(p.lse_part + row) : -INFINITY;
#pragma unroll
        for (int k = 0; k < EPL; ++k) v[u][k] = 0.f;
        if (in) {
          if constexpr (EPL == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(p.o_part + row * D) + lane);
            v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(p.o_part + row * D) + lane);
            v[u][0] = f.x, v[u][1] = f.y;
          }
        }
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < NB; ++u) mx = fmaxf(mx, l[u]);
      const float use = mx == -INFINITY ? 0.f : mx;
      const float scale = ex2(m - use);
      sum *= scale;
#pragma unroll
      for (int k = 0; k < EPL; ++k) acc[k] *= scale;
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const float f = ex2(l[u] - use);
        sum += f;
#pragma unroll
        for (int k = 0; k < EPL; ++k) acc[k] = fmaf(f, v[u][k], acc[k]);
      }
      m = mx;
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const long long off = b * p.out_stride[0] + (long long)(kvh * p.group + h) * p.out_stride[1] +
                          t * p.out_stride[2] + lane * EPL;
    if (!DA_IN(p, off + EPL - 1, p.out_elems)) continue;
    if (p.out_bf16) {
      uint32_t* y = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + off);
#pragma unroll
      for (int k = 0; k < EPL; k += 2) y[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
    } else {
#pragma unroll
      for (int k = 0; k < EPL; ++k) static_cast<float*>(p.out)[off + k] = acc[k] * inv;
    }
  }
}

template <class Cfg, bool WIDE_P>
cudaError_t launch_attend_cfg(const AttendParams& p, const AttendMaps& m, int grid,
                              cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e =
      set_smem_limit_once(attend_kernel<Cfg, WIDE_P>, Cfg::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(attend_kernel<Cfg, WIDE_P>, grid, kAttendThreads, Cfg::kSmemBytes, stream,
                          m, p);
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, const AttendMaps& m, int d, int grid,
                          cudaStream_t stream) {
  if (d == 128)
    return p.out_bf16 ? launch_attend_cfg<AttendCfg<128>, false>(p, m, grid, stream)
                      : launch_attend_cfg<AttendCfg<128>, true>(p, m, grid, stream);
  return p.out_bf16 ? launch_attend_cfg<AttendCfg<64>, false>(p, m, grid, stream)
                    : launch_attend_cfg<AttendCfg<64>, true>(p, m, grid, stream);
}

cudaError_t launch_attend_combine(const AttendParams& p, int d, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.q_tiles * p.h_kv * p.unit_rows;
  const long long most = (rows + kAttendCombineWarps - 1) / kAttendCombineWarps;
  const int grid = int(most < 8LL * p.sms ? most : 8LL * p.sms);
  if (d == 128)
    return launch_dependent(attend_combine_kernel<128>, grid, kAttendCombineWarps * 32, 0, stream, p);
  return launch_dependent(attend_combine_kernel<64>, grid, kAttendCombineWarps * 32, 0, stream, p);
}

}  // namespace da
