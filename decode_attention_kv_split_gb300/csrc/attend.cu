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
// the TMA producer, warp 9 the MMA issuer (10 and 11 fill their warpgroup, which
// gives registers to the others).  TMEM: S 2 x 128 columns, O 2 x d.
#include <math.h>

#include "common.cuh"
#include "tc5.cuh"

namespace da {
namespace {

constexpr int kTile = 128;              // K and V rows of a tile, query rows of a stream
constexpr int kAttendThreads = 384;
constexpr int kScheduleThreads = 256;

template <int D_>
struct AttendCfg {
  static constexpr int D = D_;
  static constexpr int kTileBytes = kTile * D * 2;  // Q of a stream, a K tile, a V tile
  static constexpr int kHalfBytes = kTile * 128;    // 64 columns of one
  static constexpr int kSlots = D == 128 ? 5 : 11;  // ring of K and V tiles
  // q_full[2], kv_full[slots], kv_empty[slots], s_full[2], p_full[2], o_full[2], fin
  static constexpr int kBars = 2 + 2 * kSlots + 2 + 2 + 2 + 1;
  static constexpr size_t kSmemBytes = 1024 + size_t(2 + kSlots) * kTileBytes + kBars * 8 + 128;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  // the schedule's scratch lies in the ring before the first load
  static_assert((kAttendEntries + 64) * 4 <= kTileBytes, "schedule scratch");
};

// The rows of a unit and the tiles of rows they see.  List tile k is tile k of
// the cache below `pt` (always-seen rows before the window) and tile
// first + k - pt from there on.
struct Unit {
  int rows;       // query rows, 0: no unit
  int row0;       // first of them among the sequence's (or the batch's) rows
  int p0;         // position of the query row 0's token: its last visible row
  int lo, hi;     // first windowed row and last row that some query sees
  int pt, first, tiles;
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

// Unit of row tile qt of a sequence of n rows, the last m of them new.
__device__ __forceinline__ Unit seq_unit(const AttendParams& p, int n, int m, int qt) {
  Unit u;
  const long long rows = (long long)m * p.group - (long long)qt * kAttendRows;
  u.rows = rows <= 0 ? 0 : int(rows < kAttendRows ? rows : kAttendRows);
  u.row0 = qt * kAttendRows;
  u.p0 = n - m + u.row0 / p.group;
  u.hi = n - m + (u.row0 + u.rows - 1) / p.group;
  u.lo = p.window ? max(0, u.p0 + 1 - p.window) : 0;
  u.first = u.lo / kTile;
  u.pt = p.window ? min(min((p.prefix + kTile - 1) / kTile, u.hi / kTile + 1), u.first) : 0;
  u.tiles = u.rows == 0 || u.hi < 0 ? 0 : u.pt + u.hi / kTile - u.first + 1;
  return u;
}

__device__ __forceinline__ Unit prefix_unit(const AttendParams& p, int mt) {
  Unit u;
  const int rows = p.B * p.group - mt * kAttendRows;
  u.rows = min(rows, kAttendRows);
  u.row0 = mt * kAttendRows;
  u.p0 = u.hi = p.P - 1;
  u.lo = u.first = u.pt = 0;
  u.tiles = (p.P + kTile - 1) / kTile;
  return u;
}

// Entry e of the list: the prefix (with a shared one), then row tile by row tile
// from the last (in a chunk the longest) down, every sequence of it.
__device__ __forceinline__ void entry_of(const AttendParams& p, int e, int& b, int& qt) {
  e -= p.shared;
  qt = p.q_tiles - 1 - e / p.B;
  b = e % p.B;
}

__device__ __forceinline__ int entry_tiles(const AttendParams& p, int e, bool& present) {
  if (p.shared && e == 0) {
    present = p.P > 0;
    return (p.P + kTile - 1) / kTile;
  }
  int b, qt;
  entry_of(p, e, b, qt);
  bool bad;
  const Unit u = seq_unit(p, seq_rows(p, b, bad), seq_new(p, b, bad), qt);
  // (behind a prefix a sequence without rows has no part)
  present = u.rows > 0 && (u.tiles > 0 || !p.shared);
  return u.tiles;
}

__device__ __forceinline__ int entry_units(const AttendParams& p, int e) {
  return p.h_kv * (p.shared && e == 0 ? p.prefix_tiles : 1);
}

// What one CTA does.
struct Work {
  int kvh, b;       // b < 0: the prefix
  int begin, end;   // list tiles
  int slot;         // partial, or -1: the unit's only item writes the output
  int n;            // rows of the sequence (or the prefix)
  Unit u;
};

// The list: every unit is cut into ceil(tiles / c) items of equal length, with one c
// for the whole launch, the one that ends first by a simple model (rounds of the
// grid times the tiles of an item and a constant for its start and end).  All
// CTAs compute the same list from the lengths; CTA 0 leaves the table for the
// combine.  Returns false for a CTA without an item.
constexpr int kLengthChoices = 32;
constexpr float kItemTiles = 3.f;  // an item's fixed cost in tiles

__device__ __forceinline__ bool list_item(const AttendParams& p, int* scratch, Work& w) {
  int* tiles = scratch;                       // [kAttendEntries], -1: absent
  int* sums = scratch + kAttendEntries;       // [32]
  int* found = sums + 32;                     // [4]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool mine = tid < kScheduleThreads;
  long long total = 0;
  if (mine)
    for (int e = tid; e < p.entries; e += kScheduleThreads) {
      bool present;
      const int t = entry_tiles(p, e, present);
      tiles[e] = present ? t : -1;
      total += (long long)t * entry_units(p, e);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  long long* totals = reinterpret_cast<long long*>(sums);
  if (lane == 0 && mine) totals[warp] = total;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kScheduleThreads / 32; ++i) total += totals[i];
  // one length after the other by a warp: items and the longest of them
  float best = 1e30f;
  int best_c = 1;
  const float share = float(total) / float(p.sms);
  __syncthreads();
  if (mine) {
    for (int k = warp; k < kLengthChoices; k += kScheduleThreads / 32) {
      // half an even share up to 4 of them, in steps of 2^(1/8)
      const int c = max(2, int(ceilf(share * exp2f(float(k - 8) * 0.125f))));
      int items = 0, longest = 0;
      for (int e = lane; e < p.entries; e += 32) {
        const int t = tiles[e];
        if (t < 0) continue;
        const int cut = max(1, (t + c - 1) / c);
        items += cut * entry_units(p, e);
        longest = max(longest, (t + cut - 1) / cut);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        items += __shfl_xor_sync(0xffffffffu, items, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      }
      const float rounds = float((items + p.sms - 1) / p.sms);
      const float mean = (float(total) + kItemTiles * float(items)) / float(p.sms);
      const float t = fmaxf(fminf(rounds * (float(longest) + kItemTiles),
                                  mean + float(longest) + kItemTiles), mean);
      if (t < best) best = t, best_c = c;
    }
    if (lane == 0) {
      sums[warp] = __float_as_int(best);
      sums[8 + warp] = best_c;
    }
  }
  __syncthreads();
  best = __int_as_float(sums[0]);
  int c = sums[8];
#pragma unroll
  for (int i = 1; i < kScheduleThreads / 32; ++i)
    if (__int_as_float(sums[i]) < best || (__int_as_float(sums[i]) == best && sums[8 + i] > c))
      best = __int_as_float(sums[i]), c = sums[8 + i];
  __syncthreads();
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
      if (x >= 0 && x < items) found[0] = e, found[1] = x, found[2] = cut[i];
      if (blockIdx.x == 0) p.table[e] = make_int2(at, cut[i]);
      at += items;
    }
  }
  __syncthreads();
  const int e = found[0], x = found[1], cuts = found[2];
  if (e < 0 || int(blockIdx.x) >= p.max_items) return false;
  bool bad;
  if (p.shared && e == 0) {
    const int unit = x / cuts;
    w.b = -1;
    w.kvh = unit / p.prefix_tiles;
    w.n = p.P;
    w.u = prefix_unit(p, unit % p.prefix_tiles);
  } else {
    int qt;
    entry_of(p, e, w.b, qt);
    w.kvh = x / cuts;
    w.n = seq_rows(p, w.b, bad);
    w.u = seq_unit(p, w.n, seq_new(p, w.b, bad), qt);
  }
  const int s = x % cuts;
  w.begin = int((long long)w.u.tiles * s / cuts);
  w.end = int((long long)w.u.tiles * (s + 1) / cuts);
  w.slot = cuts == 1 && !p.shared ? -1 : int(blockIdx.x);
  return true;
}

__device__ __forceinline__ bool direct_item(const AttendParams& p, Work& w) {
  // the last row tiles, the longest of a chunk, first
  const int per = p.B * p.h_kv;
  const int qt = p.q_tiles - 1 - int(blockIdx.x) / per, rest = int(blockIdx.x) % per;
  w.b = rest / p.h_kv;
  w.kvh = rest % p.h_kv;
  bool bad;
  w.n = seq_rows(p, w.b, bad);
  w.u = seq_unit(p, w.n, seq_new(p, w.b, bad), qt);
  w.begin = 0;
  w.end = w.u.tiles;
  w.slot = -1;
  return w.u.rows > 0;
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

// The streams of a work item and what each sees.
struct Streams {
  bool alternate;      // one set of rows, tiles dealt to the streams in turn
  int rows[2];
  int lo[2], hi[2];    // first windowed row of the stream's first query, last row of its last
  int lo_last[2], hi_first[2];  // the same of its last and its first query
};

__device__ __forceinline__ Streams streams_of(const AttendParams& p, const Work& w) {
  Streams s;
  s.alternate = w.u.rows <= kTile;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r0 = s.alternate ? 0 : i * kTile;
    s.rows[i] = min(w.u.rows - r0, kTile);
    if (w.b < 0) {
      s.lo[i] = s.lo_last[i] = 0;
      s.hi[i] = s.hi_first[i] = w.n - 1;
    } else {
      const int t0 = w.u.row0 / p.group;
      const int p_first = w.u.p0 - t0 + (w.u.row0 + r0) / p.group;
      const int p_last = w.u.p0 - t0 + (w.u.row0 + r0 + s.rows[i] - 1) / p.group;
      s.hi_first[i] = p_first;
      s.hi[i] = p_last;
      s.lo[i] = p.window ? max(0, p_first + 1 - p.window) : 0;
      s.lo_last[i] = p.window ? max(0, p_last + 1 - p.window) : 0;
    }
  }
  return s;
}

// First cached row of list tile k.
__device__ __forceinline__ int tile_row(const Unit& u, int k) {
  return (k < u.pt ? k : u.first + k - u.pt) * kTile;
}
// Whether stream i takes list tile k.
__device__ __forceinline__ bool takes(const AttendParams& p, const Work& w, const Streams& s, int i,
                                      int k) {
  if (k >= w.end) return false;
  if (s.alternate) return ((k - w.begin) & 1) == i;
  const int r = tile_row(w.u, k);
  return r <= s.hi[i] && (r + kTile > s.lo[i] || r < p.prefix);
}

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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t q_full0 = smem_u32(bars);
  const uint32_t full0 = q_full0 + 16;
  const uint32_t empty0 = full0 + 8 * kSlots;
  const uint32_t s_full0 = empty0 + 8 * kSlots;
  const uint32_t p_full0 = s_full0 + 16;
  const uint32_t o_full0 = p_full0 + 16;
  const uint32_t fin = o_full0 + 16;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full0 + 8 * i, 4);  // one arrival per softmax warp of the stream
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(p_full0 + 8 * i, 4);
      mbar_init(o_full0 + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);   // released by one tcgen05.commit
    }
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
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  Work w;
  const bool has = p.list ? list_item(p, reinterpret_cast<int*>(ring), w) : direct_item(p, w);
  // lengths that were clamped are reported once each
  if (blockIdx.x == 0 && p.dev_error)
    for (int b = threadIdx.x; b < p.B; b += kAttendThreads) {
      bool bad_n, bad_m;
      const int n = seq_rows(p, b, bad_n), m = seq_new(p, b, bad_m);
      if (bad_n || bad_m || (m > n && !p.shared)) flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
    }
  fence_proxy_async_smem();  // the schedule's scratch, before the ring's first loads
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!has) {
    if (warp == 9) tc5::dealloc(tmem, kTmemCols);
    return;
  }
  const Streams st = streams_of(p, w);
  const int count = w.end - w.begin;             // tiles of this item
  const int ahead = st.alternate ? 2 : 1;        // S tiles issued before the first P.V
  // Loads follow their use: K of the first `ahead` tiles, then V_j and K_(j + ahead).
  // Place of tile j's K and V in that order:
  auto k_place = [&](int j) { return j + max(0, j - ahead + 1); };
  auto v_place = [&](int j) { return j + min(count, ahead + j); };

  // Registers: 168 a thread at launch for each of three warpgroups; 2 * 208 + 88 then.
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  // ------------------------------------------------------------------ producer
  if (warp == 8) {
    if (lane == 0) {
      const uint64_t policy = p.single_read || (w.b < 0 && p.prefix_tiles == 1)
                                  ? l2_policy_evict_first()
                                  : l2_policy_evict_normal();
      const CUtensorMap* mk = w.b < 0 ? &maps.k_prefix : &maps.k;
      const CUtensorMap* mv = w.b < 0 ? &maps.v_prefix : &maps.v;
      const int z = w.b < 0 ? w.kvh : (p.b_offset + w.b) * p.h_kv + w.kvh;
      const uint32_t ring0 = smem_u32(ring);
      bool aborted = false;
      int issued = 0;
      auto load = [&](const CUtensorMap* map, int place, int j) {
        const int slot = place % kSlots;
        if (aborted) return;
        if (place >= kSlots &&
            !mbar_wait_bounded(empty0 + 8 * slot, ((place / kSlots) - 1) & 1, abort_flag)) {
          *abort_flag = 1;
          flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
          aborted = true;
          return;
        }
#ifdef DA_TEST_HOOKS
        if (int(blockIdx.x) == p.withhold_cta && map == mv && j == count - 1) return;
#endif
        const uint32_t bar = full0 + 8 * slot;
        const uint32_t dst = ring0 + slot * kTileBytes;
        const int y = tile_row(w.u, w.begin + j);
        mbar_arrive_expect_tx(bar, kTileBytes);
#pragma unroll
        for (int c = 0; c < D; c += 64)
          tma_load_3d(dst + (c / 64) * kHalfBytes, map, c, y, z, bar, policy);
        issued = place + 1;
      };
      for (int j = 0; j < min(ahead, count); ++j) load(mk, k_place(j), j);
      for (int j = 0; j < count; ++j) {
        load(mv, v_place(j), j);
        if (j + ahead < count) load(mk, k_place(j + ahead), j + ahead);
      }
      if (aborted) {  // copies in flight land before the CTA ends
        volatile int never = 0;
        for (int i = max(0, issued - kSlots); i < issued; ++i)
          mbar_wait_bounded(full0 + 8 * (i % kSlots), (i / kSlots) & 1, &never);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ MMA issuer
  if (warp == 9) {
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {  // whole warp
      if (lane == 0) ok = ok && mbar_wait_bounded(bar, parity, abort_flag);
      const bool all = __shfl_sync(0xffffffffu, ok, 0);
      if (!all && lane == 0 && !*abort_flag) {
        *abort_flag = 1;
        flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
      }
      ok = all;
      return all;
    };
    const uint32_t idesc_s = tc5::idesc_bf16(128, 128, 0, 0);
    const uint32_t idesc_o = tc5::idesc_bf16(128, D, 0, 1);
    bool any = false;
    int seen_p[2] = {0, 0};   // tiles of each stream whose P.V was issued
    auto scores = [&](int i, int j) {  // S_i = Q_i K_j^T
      const int place = k_place(j);
      if (!wait(full0 + 8 * (place % kSlots), (place / kSlots) & 1)) return;
      if (lane == 0) {
        tc5::fence_after();
        const uint32_t ka = smem_u32(ring) + (place % kSlots) * kTileBytes;
        const uint32_t qa = smem_u32(q_tile) + (st.alternate ? 0 : i * kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32;
          tc5::mma(tmem + i * 128, tc5::sdesc(qa + off, 16, 1024), tc5::sdesc(ka + off, 16, 1024),
                   idesc_s, ks > 0);
        }
        tc5::commit(s_full0 + 8 * i);
      }
      any = true;
      __syncwarp();
    };
    if (count > 0) {
      ok = wait(q_full0, 0);
      if (ok && !st.alternate) ok = wait(q_full0 + 8, 0);
    }
    for (int j = 0; j < min(ahead, count) && ok; ++j) {
      for (int i = 0; i < 2 && ok; ++i)
        if (takes(p, w, st, i, w.begin + j)) scores(i, j);
      if (ok && lane == 0) tc5::commit(empty0 + 8 * (k_place(j) % kSlots));
    }
    for (int j = 0; j < count && ok; ++j) {
      const int place = v_place(j);
      const uint32_t vslot = place % kSlots;
      bool v_ready = false;
      for (int i = 0; i < 2 && ok; ++i) {
        if (takes(p, w, st, i, w.begin + j)) {
          if (!v_ready) {
            if (!wait(full0 + 8 * vslot, (place / kSlots) & 1)) break;
            v_ready = true;
            // rows that no query of the unit sees may hold anything, even NaN: cleared
            const int r0 = tile_row(w.u, w.begin + j);
            if (r0 + kTile - 1 > w.u.hi || (r0 < w.u.lo && r0 + kTile > p.prefix)) {
              uint8_t* vt = ring + size_t(vslot) * kTileBytes;
              for (int r = 0; r < kTile; ++r) {
                const int row = r0 + r;
                if ((row > w.u.hi || (row < w.u.lo && row >= p.prefix)) && lane < D / 8)
                  *reinterpret_cast<uint4*>(vt + tc5::sw128(r, lane * 8, kTile)) =
                      make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (!wait(p_full0 + 8 * i, seen_p[i] & 1)) break;
          if (lane == 0) {
            tc5::fence_after();
            const uint32_t va = smem_u32(ring) + vslot * kTileBytes;
            const uint32_t o = tmem + 256 + i * D, pa = tmem + i * 128;
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_tmem_a(o, pa + ks * 8, tc5::sdesc(va + ks * 16 * 128, kHalfBytes, 1024), idesc_o,
                         seen_p[i] > 0 || ks > 0);
            if constexpr (WIDE_P) {
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                mma_tmem_a(o, pa + 64 + ks * 8, tc5::sdesc(va + ks * 16 * 128, kHalfBytes, 1024),
                           idesc_o, 1);
            }
          }
          any = true;
          ++seen_p[i];
          __syncwarp();
        }
        if (j + ahead < count && takes(p, w, st, i, w.begin + j + ahead)) scores(i, j + ahead);
      }
      if (ok && lane == 0) {
        tc5::commit(empty0 + 8 * vslot);
        if (j + ahead < count) tc5::commit(empty0 + 8 * (k_place(j + ahead) % kSlots));
      }
    }
    if (lane == 0) {
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
  return;
  }

  // ------------------------------------------------------------------ softmax
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  const int i = warp >> 2;                          // stream
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;                // row of the stream = TMEM lane
  const uint32_t lanes = uint32_t(quarter * 32) << 16;
  const uint32_t s_col = tmem + i * 128 + lanes, o_col = tmem + 256 + i * D + lanes;
  const bool valid = r < st.rows[i];
  // this row's token, head and position
  const int unit_row = (st.alternate ? 0 : i * kTile) + r;
  int hi = -1, lo = 0;
  long long q_off = 0, out_off = 0;
  if (valid) {
    const int flat = w.u.row0 + unit_row;
    const int t = flat / p.group, head = w.kvh * p.group + flat % p.group;
    const int b = w.b < 0 ? t : w.b, tok = w.b < 0 ? 0 : t;
    hi = w.b < 0 ? w.n - 1 : w.u.p0 - w.u.row0 / p.group + t;
    lo = w.b < 0 || !p.window ? 0 : hi + 1 - p.window;
    q_off = b * p.q_stride[0] + head * p.q_stride[1] + tok * p.q_stride[2];
    out_off = b * p.out_stride[0] + head * p.out_stride[1] + tok * p.out_stride[2];
  }
  bool live = true;
  if (count > 0 && !(st.alternate && i == 1)) {
    // Q of the stream's rows, swizzled K-major; rows past the unit are zero
    constexpr int kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces of a row; rows at a time
    uint4 v[32 / kPer];
    const uint4* q = static_cast<const uint4*>(p.q);
#pragma unroll
    for (int k = 0; k < 32 / kPer; ++k) {
      const int row = k * kPer + lane / kChunks;
      const long long off = __shfl_sync(0xffffffffu, q_off, row);
      const bool in = quarter * 32 + row < st.rows[i] && DA_IN(p, off + D - 1, p.q_elems);
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
    if (lane == 0) mbar_arrive(q_full0 + 8 * i);
  }

  float m_run = -INFINITY, l_run = 0.f;
  int done = 0;  // tiles of this stream
  auto give_up = [&] {
    if (!*abort_flag) {
      *abort_flag = 1;
      flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
    }
  };
  for (int j = 0; j < count; ++j) {
    if (!takes(p, w, st, i, w.begin + j)) continue;
    const bool got = mbar_wait_bounded(s_full0 + 8 * i, done & 1, abort_flag);
    if (!got) give_up();
    live = __all_sync(0xffffffffu, got);  // warp-uniform: the TMEM accesses below are .sync.aligned
    if (!live) break;
    tc5::fence_after();
    uint32_t raw[128];
    float* s = reinterpret_cast<float*>(raw);
#pragma unroll
    for (int c = 0; c < 128; c += 32) tmem_ld32(s_col + c, raw + c);
    tc5::wait_ld();
    const int r0 = tile_row(w.u, w.begin + j);
    if (r0 + kTile - 1 > st.hi_first[i] || (r0 < st.lo_last[i] && r0 + kTile > p.prefix)) {
      const int hi_c = hi - r0, lo_c = lo - r0, pre_c = p.prefix - r0;
#pragma unroll
      for (int c = 0; c < 128; ++c) {
        const bool seen = c <= hi_c && (c >= lo_c || c < pre_c);
        s[c] = seen ? s[c] : -INFINITY;
      }
    }
    float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int c = 4; c < 128; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
    const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    const bool over = m_tile > m_run + p.lazy || (m_run == -INFINITY && m_tile > -INFINITY);
    if (__any_sync(0xffffffffu, over)) {
      const float m_new = over ? m_tile : m_run;
      const float alpha = over ? ex2((m_run - m_new) * p.scale_log2) : 1.f;  // 0 from -inf
      m_run = m_new;
      l_run *= alpha;
      if (done > 0) {  // (S of this tile was issued behind the P.V of the last)
#pragma unroll
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
    float l4[4] = {0.f, 0.f, 0.f, 0.f};
    // exponentials in halves of 64 columns; P over the first columns of S, which
    // every lane of the warp has loaded
#pragma unroll
    for (int h = 0; h < 128; h += 64) {
      uint32_t hi_p[32];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float a = ex2(fmaf(s[h + c], p.scale_log2, shift));
        const float b = ex2(fmaf(s[h + c + 1], p.scale_log2, shift));
        l4[c & 2] += a;
        l4[(c & 2) + 1] += b;
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
    l_run += (l4[0] + l4[1]) + (l4[2] + l4[3]);
    tc5::wait_st();
    tc5::fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(p_full0 + 8 * i);
    ++done;
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
  if (st.alternate) {
    if (i == 1 && live) {
      if (done > 0) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tc5::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) other[(c + k) * kTile + r] = __uint_as_float(o[k]);
        }
      }
      other[D * kTile + r] = m_run;
      other[D * kTile + kTile + r] = l_run;
    }
    named_bar_sync(1, 256);
    if (i == 1 || *abort_flag) live = false;
    live = __all_sync(0xffffffffu, live);
  }
  float keep0 = 1.f, keep1 = 0.f;  // weights of the two streams' O
  const bool with_other = st.alternate && count > 1;
  if (live && with_other) {
    const float m1 = other[D * kTile + r], l1 = other[D * kTile + kTile + r];
    const float m = fmaxf(m_run, m1), m_use = m == -INFINITY ? 0.f : m;
    keep0 = ex2((m_run - m_use) * p.scale_log2);
    keep1 = ex2((m1 - m_use) * p.scale_log2);
    l_run = l_run * keep0 + l1 * keep1;
    m_run = m;
  }
  if (live) {
    const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
    keep0 *= inv;
    keep1 *= inv;
    const bool part = w.slot >= 0;
    if (part) out_off = ((long long)w.slot * p.pitch + unit_row) * D;
    const long long extent = part ? (long long)p.max_items * p.pitch * D : p.out_elems;
    if (part && valid && DA_IN(p, (long long)w.slot * p.pitch + unit_row, (long long)p.max_items * p.pitch))
      p.lse_part[(long long)w.slot * p.pitch + unit_row] =
          l_run > 0.f ? m_run * p.scale_log2 + log2f(l_run) : (l_run == 0.f ? -INFINITY : l_run);
    const bool narrow = !part && p.out_bf16;
    uint8_t* stage = q_tile + i * kTileBytes + quarter * (kTileBytes / 4);  // 32 rows of 2 D bytes
    constexpr int kChunks = D / 8, kPer = 32 / kChunks;
    // a row of 2 D bytes at a time (D bf16 or D / 2 floats) through shared memory,
    // so that whole rows are written
    for (int c0 = 0; c0 < D; c0 += narrow ? D : D / 2) {
      const int cols = narrow ? D : D / 2;
#pragma unroll 1
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
      for (int k = 0; k < 32; k += kPer) {
        const int row = k + lane / kChunks, ch = lane % kChunks;
        const long long off = __shfl_sync(0xffffffffu, out_off, row);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 2 * D + ((ch ^ (row & 7)) << 4));
        if (quarter * 32 + row < st.rows[i] && DA_IN(p, off + D - 1, extent)) {
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
  const long long all = (long long)p.B * p.q_tiles * p.h_kv * p.pitch;
  for (long long x = (long long)blockIdx.x * kAttendCombineWarps + (threadIdx.x >> 5); x < all;
       x += warps) {
    const int ur = int(x % p.pitch);
    const int kvh = int(x / p.pitch % p.h_kv);
    const int e = int(x / p.pitch / p.h_kv) + p.shared;
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
  const long long rows = (long long)p.B * p.q_tiles * p.h_kv * p.pitch;
  const long long most = (rows + kAttendCombineWarps - 1) / kAttendCombineWarps;
  const int grid = int(most < 8LL * p.sms ? most : 8LL * p.sms);
  if (d == 128)
    return launch_dependent(attend_combine_kernel<128>, grid, kAttendCombineWarps * 32, 0, stream, p);
  return launch_dependent(attend_combine_kernel<64>, grid, kAttendCombineWarps * 32, 0, stream, p);
}

}  // namespace da
