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
// P is multiplied as a bf16 and its bf16 remainder (2^-16 of each weight, as the decode
// kernels do); where the caller asks for it as one bf16 (2^-8), a third of the MMAs less.
//
// A unit of at most 128 query rows (few tokens, one sequence's group) uses both
// streams for the same rows on alternate tiles and merges them at the end.
//
// The kernel is persistent: the CTA of an SM takes its items one after the other, so
// that the loads and first scores of one run under the end of the last.  The items are
// equal pieces of all units, or whole units from the grid's CTAs that wait for launch.
//
// What bounds it.  Prompts (2 of 8192 tokens, 32 heads of 128): 980 to 1050 us, the MMAs at 1.57 to
// 1.68 PFLOP/s with the remainder's counted, 0.81 to 0.87 of a library product's rate; with weights
// of one bf16 727 to 744 us, 1.5 PFLOP/s.  Heads of 64 (731 us, 549): the exponentials, 16 a cycle
// and SM.  Few tokens of long contexts (2 of 131056 rows): HBM, 168 to 174 us, 6.2 to 6.4 TB/s.
// Batches behind a shared prefix: the start (7 us to the first scores), 3 to 4 us an item beside its
// tiles, 5 to 8 us to merge.
//
// Roles (384 threads): warps 0-3 and 4-7 the softmax of streams 0 and 1, warp 8
// the items and the TMA loads, warp 9 the MMAs, warp 10 looks through V rows that some
// query does not see (11 fills their warpgroup, which gives registers to the others).  TMEM: S 2 x 128 columns, O 2 x d.
#include <math.h>

#include "common.cuh"
#include "tc5.cuh"

namespace da {
namespace {

constexpr int kTile = 128;              // K and V rows of a tile, query rows of a stream
constexpr int kAttendThreads = 384;
constexpr int kScheduleThreads = 256;
constexpr int kEdges = 8;               // more than the V tiles that the ring can hold

template <int D_>
struct AttendCfg {
  static constexpr int D = D_;
  static constexpr int kTileBytes = kTile * D * 2;  // Q of a stream, a K tile, a V tile
  static constexpr int kHalfBytes = kTile * 128;    // 64 columns of one
  static constexpr int kSlots = D == 128 ? 5 : 11;  // ring of K and V tiles
  // full[slots], empty[slots], out_done[slots], edge[kEdges], then for each stream q_full, s_full,
  // p_full[2], o_full, o_empty; item_full[2], item_empty[2], meet[2], fin, answered
  static constexpr int kBars = 3 * kSlots + kEdges + 2 * 6 + 2 + 2 + 2 + 1 + 1;
  static constexpr size_t kSmemBytes = size_t(2 + kSlots) * kTileBytes + kBars * 8 +
                                       3 * 64 + 64 + 4 * kTile * 4;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(kEdges > (kSlots + 1) / 2, "edge barriers");
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
  int q_buf;         // alternate: the buffer of Q, which the next such item does not use
  int part;          // first row of its partial, or -1: the unit's only item writes the output
};
static_assert(sizeof(Item) == 64, "shared memory of the items");

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

__device__ __forceinline__ void report_lengths(const AttendParams& p, bool bad) {
  if (bad && p.dev_error) flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
}

// First cached row of list tile k.
__device__ __forceinline__ int tile_row(const Item& w, int k) {
  return (k < w.pt ? k : w.first + k - w.pt) * kTile;
}

// Rows that some query of a unit does not see: those past `hi`, its first query's, and of
// [prefix, lo) the window.
struct PartSeen {
  int hi, lo;
};
__device__ __forceinline__ PartSeen part_seen(const AttendParams& p, const Item& w) {
  return {w.past + p.by_group.div(w.row0),
          p.window ? max(0, w.past + p.by_group.div(w.row0 + w.rows - 1) + 1 - p.window) : 0};
}

// Whether the V tile at row r0 holds such rows.  A weight of zero times an infinity or NaN is
// NaN, so a warp looks through them first: rows that no query of the sequence sees may hold
// anything and are cleared; of the others (MANY: sequences of more than one token) what is not
// finite is cleared too, and added behind the item to the outputs of the queries that see it.
// In the tiles of an item that is the end of the always-seen rows, the window's first tiles and
// the last ones.
template <bool MANY>
__device__ __forceinline__ bool edge_tile(const AttendParams& p, const Item& w, const PartSeen& part,
                                          int r0) {
  if (!MANY) return r0 + kTile > w.n || (r0 < w.clear_lo && r0 + kTile > p.prefix);
  return r0 + kTile - 1 > part.hi || (r0 < part.lo && r0 + kTile > p.prefix);
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
__device__ __forceinline__ void cut_item(const AttendParams& p, int begin, int end, int part,
                                         Item& w) {
  w.begin = begin;
  w.count = end - begin;
  w.part = part;
  w.clear_lo = w.b >= 0 && p.window ? max(0, w.past + 1 - p.window) : 0;
  w.upto[0] = w.upto[1] = w.count;
  if (w.b >= 0 && w.rows > kTile) {  // stream 0 ends at its last query's row
    const int hi = w.past + p.by_group.div(w.row0 + kTile - 1);
    const int tiles = hi < 0 ? 0 : w.pt + hi / kTile - w.first + 1;
    w.upto[0] = min(max(tiles - begin, 0), w.count);
  }
}

// ---- The line: all units in a row, each as long as its work, cut into one equal
// piece per CTA.  A unit takes kStart for the start and end of an item and
// kPairTile or kTileCost a tile (two streams of rows, or one); a tile belongs to the
// CTA whose piece it starts in.  A CTA so gets parts of a unit or two and whole ones
// between them, and the CTAs end together whatever the lengths are (one item a unit,
// dealt in turn, ended 30 % apart for ragged chunks, 65 % behind a shared prefix).
// Entries of units of one length: the prefix (with a shared one), then row tile by
// row tile from the last down, every sequence of it, its KV heads.
constexpr int kStart = 14, kPairTile = 4, kTileCost = 3;  // about 0.3 us each
constexpr int kLeastPiece = kStart + 2 * kPairTile;       // of a CTA
constexpr int kScheduleWarps = kScheduleThreads / 32;

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
    w.past = p.P - 1;
    w.pt = w.first = 0;
    w.rows = min(p.B * p.group, kAttendRows);
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
__device__ __forceinline__ int tile_cost(const Item& w) {
  return w.rows > kTile ? kPairTile : kTileCost;
}

// Tiles of a unit that start before x, x > -kStart from its first.
__device__ __forceinline__ int tiles_before(int x, int cost) {
  return x <= 0 ? 0 : cost == kPairTile ? (x + kPairTile - 1) / kPairTile : (x + kTileCost - 1) / kTileCost;
}

// Where a CTA's piece starts: unit i of entry e, at position `pos` of the line; and
// where the piece lies.
struct LineStart {
  long long pos, lo, hi;
  int e, i;
  Item unit;  // of entry e
};

// All CTAs compute the same line from the lengths.  Ends with a barrier.
__device__ __forceinline__ void line_start(const AttendParams& p, long long* scratch,
                                           LineStart* out) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kPer = kAttendEntries / kScheduleThreads;
  const bool mine = tid < kScheduleThreads;
  long long own = 0;
  int unit_cost[kPer];  // 0: absent
  if (mine)
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int e = tid * kPer + x;
      unit_cost[x] = 0;
      Item w;
      if (e < p.entries && entry_unit(p, e, w)) {
        unit_cost[x] = kStart + w.tiles * tile_cost(w);
        own += (long long)unit_cost[x] * entry_units(p, e);
      }
    }
  long long upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31 && mine) scratch[warp] = upto;
  if (tid == 0) out->pos = out->lo = out->hi = 0;
  __syncthreads();
  if (mine) {
    long long total = 0, at = upto - own;
#pragma unroll
    for (int x = 0; x < kScheduleWarps; ++x) {
      total += scratch[x];
      if (x < warp) at += scratch[x];
    }
    // CTAs that take part, and this one's piece
    const long long most = total / kLeastPiece;
    const int ctas = most < 1 ? 1 : most < int(gridDim.x) ? int(most) : int(gridDim.x);
    const int c = blockIdx.x;
    // borders at total * c / ctas
    const long long each = total <= 0xffffffffLL ? uint32_t(total) / uint32_t(ctas) : total / ctas;
    const int over = int(total - each * ctas);
    const long long lo = each * c + over * c / ctas, hi = each * (c + 1) + over * (c + 1) / ctas;
    if (tid == 0) p.cta_start[c] = make_int4(-1, 0, 0, 0);
    if (c < ctas && total > 0)
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int e = tid * kPer + x;
        const long long len = e < p.entries ? (long long)unit_cost[x] * entry_units(p, e) : 0;
        if (lo >= at && lo < at + len) {
          out->lo = lo;
          out->hi = hi;
          out->e = e;
          const long long in = lo - at;
          out->i = in <= 0x7fffffffLL ? int(in) / unit_cost[x] : int(in / unit_cost[x]);
          out->pos = at + (long long)out->i * unit_cost[x];
          entry_unit(p, e, out->unit);
        }
        at += len;
      }
  }
  fence_proxy_async_smem();  // the scratch is the ring's: before its first loads
  __syncthreads();
}

// The CTA's way along its piece.
struct LineWalk {
  long long pos, lo, hi;
  int e, i;
  bool fresh = false;  // entry e is not in `unit` yet
  Item unit;
  __device__ __forceinline__ explicit LineWalk(const LineStart& s)
      : pos(s.pos), lo(s.lo), hi(s.hi), e(s.e), i(s.i), unit(s.unit) {}

  // The next item; false: the piece ends.
  __device__ __forceinline__ bool next(const AttendParams& p, Item& w) {
    while (pos < hi) {
      if (fresh) {
        if (e >= p.entries) return false;
        if (!entry_unit(p, e, unit)) {
          ++e;
          continue;
        }
        fresh = false;
      }
      if (i >= entry_units(p, e)) {
        ++e;
        i = 0;
        fresh = true;
        continue;
      }
      const int cost = tile_cost(unit), n = unit.tiles, u = i;
      const long long first = pos + kStart;     // of the unit's tiles
      const bool whole_start = first >= lo, whole_end = first + (long long)(n - 1) * cost < hi;
      // (a border inside the unit lies less than its length away)
      const int begin = whole_start ? 0 : min(n, tiles_before(int(lo - first), cost));
      const int end = whole_end ? n : max(0, tiles_before(int(hi - first), cost));
      // (a unit without tiles, all of whose tokens see nothing, belongs where it ends)
      const bool here = n > 0 ? end > begin : first - 1 >= lo && first - 1 < hi;
      pos = first + (long long)n * cost;
      ++i;
      if (!here) continue;
      w = unit;
      const int cta = blockIdx.x;
      int part = -1;
      if (p.shared) {
        int unit_index;
        if (w.b < 0) {
          unit_index = u;
          w.kvh = u / p.prefix_tiles;
          w.row0 = (u - w.kvh * p.prefix_tiles) * kAttendRows;
          w.rows = min(p.B * p.group - w.row0, kAttendRows);
          part = (u + cta) * p.pitch;
        } else {
          const int own = (e - 1) * p.h_kv + u;
          unit_index = p.h_kv * p.prefix_tiles + own;
          w.kvh = u;
          part = p.own_parts + (own + cta) * p.unit_rows;
        }
        // the CTAs of a unit's first and last items, for the combine
        int* at = reinterpret_cast<int*>(p.unit_ctas + unit_index);
        if (begin == 0) at[0] = cta;
        if (end == n) at[1] = cta;
      } else {
        w.kvh = u;
        if (begin > 0 || end < n) part = (2 * cta + (begin == 0)) * p.pitch;
        // a unit that goes on from the CTA before: its number, its entry and KV head
        if (begin > 0) p.cta_start[cta] = make_int4(e * p.h_kv + u, e, u, 0);
      }
      cut_item(p, begin, end, part, w);
      return true;
    }
    return false;
  }
};

// Without a list: a CTA per unit, the last row tiles of all sequences first, which are the
// longest where the sequences bring as many tokens; a CTA that is done goes on with the next unit
// whose CTA has not been launched.  (Units dealt in turn instead: one long prompt among 19 took
// 497 us, not 53, ragged ones 504, not 266.)  A sequence of few tokens has row tile 0 alone,
// which comes last however long its context is.  False: the unit has no rows.
__device__ __forceinline__ bool unit_item(const AttendParams& p, int u, Item& w) {
  const int per = p.B * p.h_kv;
  const int up = u / per, rest = u - up * per;
  w.b = rest / p.h_kv;
  w.kvh = rest - w.b * p.h_kv;
  bool bad_n, bad_m;
  const int n = seq_rows(p, w.b, bad_n), m = seq_new(p, w.b, bad_m);
  if (up == 0 && w.kvh == 0) report_lengths(p, bad_n || bad_m || m > n);
  seq_unit(p, n, m, p.q_tiles - 1 - up, w);
  cut_item(p, 0, w.tiles, -1, w);
  return w.rows > 0;
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

// The MMA issuer runs as a whole warp, so that addresses and descriptors stay in
// registers of the warp; one lane's instructions count.  (One thread in a branch took
// 115 cycles for each MMA of 64: prompts with weights of one bf16 1070 us, and 725 this way.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// D (TMEM) = A (smem) . B (smem)^T [+ D], fp32 accumulators.
__device__ __forceinline__ void mma_smem_a(uint32_t leader, uint32_t d_tmem, uint64_t adesc,
                                           uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// A in TMEM: lane = row, two bf16 of K a column.
__device__ __forceinline__ void mma_tmem_a(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                           uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void arrive_one(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(leader)
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

// Bits 0 .. n - 1, for any n.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// Takes a CTA that has not been launched off the grid; 16 bytes that say which, or that there
// was none, land at `reply` (after which no other may be asked for).
__device__ __forceinline__ void cancel_next_cta(uint32_t reply, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
          "r"(reply),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ long long cancelled_cta(uint32_t reply) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(reply)
      : "memory");
  return got ? (long long)x : -1;
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

// A place of the ring: K and V tiles in the order of their use, and behind each item
// one through which the softmax warps write its output.
template <int SLOTS>
struct RingPlace {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SLOTS) slot = 0, phase ^= 1u;
  }
};

// What the roles of the kernel share.
template <class Cfg>
struct AttendShared {
  uint8_t *q_tile, *ring;   // [2], [kSlots] tiles
  Item* items;              // [2]: the items underway
  LineStart* line;          // the CTA's piece
  float* pairs;             // [2][m, l][128]: the streams' sums of the same rows
  volatile int* abort_flag;
  uint32_t tmem;
  uint32_t bars;
  __device__ __forceinline__ uint32_t full(int s) const { return bars + 8 * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8 * (Cfg::kSlots + s); }
  __device__ __forceinline__ uint32_t out_done(int s) const {
    return bars + 8 * (2 * Cfg::kSlots + s);
  }
  __device__ __forceinline__ uint32_t edge(int e) const {
    return bars + 8 * (3 * Cfg::kSlots + e % kEdges);
  }
  __device__ __forceinline__ uint32_t of(int i, int what) const {  // stream i's
    return bars + 8 * (3 * Cfg::kSlots + kEdges + 6 * i + what);
  }
  __device__ __forceinline__ uint32_t q_full(int i) const { return of(i, 0); }
  __device__ __forceinline__ uint32_t s_full(int i) const { return of(i, 1); }
  __device__ __forceinline__ uint32_t p_full(int i, int h) const { return of(i, 2 + h); }
  __device__ __forceinline__ uint32_t o_full(int i) const { return of(i, 4); }
  __device__ __forceinline__ uint32_t o_empty(int i) const { return of(i, 5); }
  __device__ __forceinline__ uint32_t rest(int what) const { return of(2, what); }
  __device__ __forceinline__ uint32_t item_full(int k) const { return rest(k & 1); }
  __device__ __forceinline__ uint32_t item_empty(int k) const { return rest(2 + (k & 1)); }
  __device__ __forceinline__ uint32_t meet(int k) const { return rest(4 + k); }
  __device__ __forceinline__ uint32_t fin() const { return rest(6); }
  __device__ __forceinline__ uint32_t answered() const { return rest(7); }

  __device__ __forceinline__ void give_up(const AttendParams& p) const {
    if (!*abort_flag) {
      *abort_flag = 1;
      flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
    }
  }
  // One thread's wait.
  __device__ __forceinline__ bool wait(const AttendParams& p, uint32_t bar, uint32_t parity) const {
    if (mbar_wait_bounded(bar, parity, abort_flag)) return true;
    give_up(p);
    return false;
  }
  // A warp's in which the control flow stays the warp's.
  __device__ __forceinline__ bool wait_uniform(const AttendParams& p, uint32_t bar,
                                               uint32_t parity) const {
#pragma unroll 1
    for (int n = 0; n < 256; ++n)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_warp(p, bar, parity);
  }
  // A warp's: every thread's, with one answer.
  __device__ __forceinline__ bool wait_warp(const AttendParams& p, uint32_t bar,
                                            uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(p, bar, parity));
  }
};
constexpr int kItemReaders = 1 + 1 + 8;  // MMA issuer, the clearing warp, softmax warps

// One set of rows, tiles dealt to the streams in turn.
__device__ __forceinline__ bool alternates(const Item& w) { return w.rows <= kTile; }
// Tiles whose scores are issued before a stream's first P.V.
__device__ __forceinline__ int lookahead(const Item& w) { return alternates(w) ? 2 : 1; }

// ---- the items and their loads: one thread
template <class Cfg, bool MANY>
__device__ __forceinline__ void attend_load(const AttendParams& p, const AttendMaps& maps,
                                            const AttendShared<Cfg>& sh) {
  constexpr int kSlots = Cfg::kSlots;
  RingPlace<kSlots> at;
  uint32_t issued = 0, parity = 0;  // per slot: loaded on its full barrier, phase of that load
  uint32_t outs = 0, out_parity = 0;  // per slot: held an output, phase of its out_done
  int edges = 0;
  bool ok = true;
  auto free_place = [&] {
    if (!sh.wait(p, sh.empty(at.slot), at.phase ^ 1u)) return false;
    if (outs >> at.slot & 1) {
      if (!sh.wait(p, sh.out_done(at.slot), out_parity >> at.slot & 1)) return false;
      outs &= ~(1u << at.slot);
      out_parity ^= 1u << at.slot;
    }
    return true;
  };
  // Without a list: the next unit that no CTA has begun is asked for (a CTA's number, launched
  // in its stead), before the last V tile of this one is loaded (3 or 6 tiles sooner: no faster)
  const uint32_t reply = (smem_u32(sh.line) + 15) & ~15u;  // (the line is not used then)
  bool asked = false;
  uint32_t asked_phase = 0;
  auto ask = [&] {
    fence_proxy_async_smem();  // the last answer has been read
    mbar_arrive_expect_tx(sh.answered(), 16);
    cancel_next_cta(reply, sh.answered());
    asked = true;
  };
  auto answer = [&]() -> long long {
    if (!(ok = ok && sh.wait(p, sh.answered(), asked_phase))) return -1;
    asked = false;
    asked_phase ^= 1u;
    return cancelled_cta(reply);
  };
  int q_buf = 1;
  LineWalk walk(*sh.line);
  for (int k = 0; ok; ++k) {
    if (k >= 2 && !sh.wait(p, sh.item_empty(k), ((k >> 1) - 1) & 1)) {
      ok = false;
      break;
    }
    Item& w = sh.items[k & 1];
    if (p.list) {
      if (!walk.next(p, w)) w.count = -1;
    } else {
      long long unit = k == 0 ? (long long)blockIdx.x : answer();
      while (unit >= 0 && !unit_item(p, int(unit), w)) {
        ask();
        unit = answer();
      }
      if (unit < 0) w.count = -1;
    }
    // behind an item of both buffers the first, whose stream 0 loads it early
    q_buf = w.count >= 0 && alternates(w) ? q_buf ^ 1 : 1;
    w.q_buf = q_buf;
    mbar_arrive(sh.item_full(k));
    if (w.count < 0) break;
    const bool pre = w.b < 0;
    const uint64_t policy = p.single_read || (pre && p.prefix_tiles == 1) ? l2_policy_evict_first()
                                                                          : l2_policy_evict_normal();
    const CUtensorMap* mk = pre ? &maps.k_prefix : &maps.k;
    const CUtensorMap* mv = pre ? &maps.v_prefix : &maps.v;
    const int z = pre ? w.kvh : (p.b_offset + w.b) * p.h_kv + w.kvh;
    const int count = w.count, ahead = lookahead(w);
    const PartSeen part = MANY ? part_seen(p, w) : PartSeen{};
    auto load = [&](const CUtensorMap* map, int j) {
      if (!ok) return;
      if (!(ok = free_place())) return;
#ifdef DA_TEST_HOOKS
      if (int(blockIdx.x) == p.withhold_cta && k == 0 && map == mv && j == count - 1) {
        at.next();
        return;
      }
#endif
      const int y = tile_row(w, w.begin + j);
      // a V tile to look through goes to warp 10 first, which says when it is full
      const bool edge = map == mv && edge_tile<MANY>(p, w, part, y);
      const uint32_t bar = edge ? sh.edge(edges++) : sh.full(at.slot);
      mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
      const uint32_t dst = smem_u32(sh.ring) + at.slot * Cfg::kTileBytes;
#pragma unroll
      for (int c = 0; c < Cfg::D; c += 64)
        tma_load_3d(dst + (c / 64) * Cfg::kHalfBytes, map, c, y, z, bar, policy);
      issued = edge ? issued & ~(1u << at.slot) : issued | 1u << at.slot;
      parity = (parity & ~(1u << at.slot)) | (at.phase << at.slot);
      at.next();
    };
    // loads follow their use: K of the first tiles, then V_j and K_(j + ahead)
    for (int j = 0; j < min(ahead, count); ++j) load(mk, j);
    if (!p.list && count == 0) ask();
    for (int j = 0; j < count; ++j) {
      if (!p.list && j == count - 1) ask();
      load(mv, j);
      if (j + ahead < count) load(mk, j + ahead);
    }
    // a place for the output
    if (ok && (ok = free_place())) {
      issued &= ~(1u << at.slot);
      outs |= 1u << at.slot;
      mbar_arrive(sh.full(at.slot));
      at.next();
    }
  }
  if (!ok) {  // copies and answers in flight land before the CTA ends
    volatile int never = 0;
    if (asked) mbar_wait_bounded(sh.answered(), asked_phase, &never);
    for (int i = 0; i < kSlots; ++i)
      if (issued >> i & 1) mbar_wait_bounded(sh.full(i), (parity >> i) & 1, &never);
    for (int e = max(0, edges - kEdges); e < edges; ++e)
      mbar_wait_bounded(sh.edge(e), (e / kEdges) & 1, &never);
  }
}

// ---- the MMAs: a warp, whose first lane issues them
// Per tile and stream O += P V, then S = Q K^T of the stream's next tile: the new S
// takes the place of the P that has just been read.  One lane issues both streams'
// in turn, which keeps them apart: the softmax of one runs under the MMAs of the other.
// (A warp for each let them fall into step: their exponentials then shared the
// special-function units while the tensor cores waited, 20 % slower.)
template <class Cfg, bool WIDE_P>
__device__ __forceinline__ void attend_mma(const AttendParams& p, const AttendShared<Cfg>& sh) {
  constexpr int D = Cfg::D, kTileBytes = Cfg::kTileBytes;
  const uint32_t idesc_s = tc5::idesc_bf16(128, 128, 0, 0) | (p.negate ? 1u << 13 : 0u);  // -Q
  const uint32_t idesc_o = tc5::idesc_bf16(128, D, 0, 1);
  // descriptors of the operands' first bytes; their addresses count 16 bytes
  const uint32_t ring_at = smem_u32(sh.ring) >> 4;
  const uint64_t k_major = tc5::sdesc(0, 16, 1024) + ring_at;
  const uint64_t mn_major = tc5::sdesc(0, Cfg::kHalfBytes, 1024) + ring_at;
  const uint64_t q0 = tc5::sdesc(0, 16, 1024) + (smem_u32(sh.q_tile) >> 4);
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0), leader = elect_one();
  RingPlace<Cfg::kSlots> at;
  bool ok = true, any = false;
  uint32_t p_phase = 0;      // a bit for each stream: the parity of its p_full barriers
  uint32_t pairs = 0;        // items of two sets of rows
  for (int k = 0; ok; ++k) {
    if (!(ok = sh.wait_uniform(p, sh.item_full(k), (k >> 1) & 1))) break;
    const Item& w = sh.items[k & 1];
    const int count = __shfl_sync(0xffffffffu, w.count, 0);
    if (count < 0) break;
    const bool alternate = __shfl_sync(0xffffffffu, w.rows, 0) <= kTile;
    const int ahead = alternate ? 2 : 1;
    const int upto0 = __shfl_sync(0xffffffffu, w.upto[0], 0);
    const int upto1 = __shfl_sync(0xffffffffu, w.upto[1], 0);
    const int q_buf = __shfl_sync(0xffffffffu, w.q_buf, 0);
    if (!(ok = sh.wait_uniform(p, sh.q_full(0), k & 1))) break;
    if (!alternate && !(ok = sh.wait_uniform(p, sh.q_full(1), pairs++ & 1))) break;
    uint32_t started = 0;    // streams with a P.V in this item
    auto scores = [&](int i, int slot) {
      const uint64_t a = q0 + (alternate ? q_buf : i) * (kTileBytes >> 4);
      const uint64_t b = k_major + slot * (kTileBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * Cfg::kHalfBytes + (ks & 3) * 32) >> 4;
        mma_smem_a(leader, tmem + i * 128, a + off, b + off, idesc_s, ks > 0);
      }
      commit_one(leader, sh.s_full(i));
      any = true;
    };
    for (int j = 0; j < min(ahead, count); ++j) {
      if (!(ok = sh.wait_uniform(p, sh.full(at.slot), at.phase))) break;
      tc5::fence_after();
      if (alternate) {
        scores(j, at.slot);
      } else {
        if (j < upto0) scores(0, at.slot);
        if (j < upto1) scores(1, at.slot);
      }
      commit_one(leader, sh.empty(at.slot));
      at.next();
    }
    for (int j = 0; j < count && ok; ++j) {
      const RingPlace<Cfg::kSlots> v = at;         // V_j, then K_(j + ahead)
      if (!(ok = sh.wait_uniform(p, sh.full(v.slot), v.phase))) break;
      at.next();
      const bool more = j + ahead < count;
      if (more && !(ok = sh.wait_uniform(p, sh.full(at.slot), at.phase))) break;
      const uint64_t b = mn_major + v.slot * (kTileBytes >> 4);
      const int i_end = alternate ? (j & 1) + 1 : 2;
      for (int i = alternate ? j & 1 : 0; i < i_end; ++i) {
        const int mine = alternate ? count : i == 0 ? upto0 : upto1;
        if (j < mine) {
          const uint32_t o = tmem + 256 + i * D, pa = tmem + i * 128;
          const bool more_o = started >> i & 1;
          // (O of the last item has been read)
          if (!more_o && k > 0 && !(ok = sh.wait_uniform(p, sh.o_empty(i), (k - 1) & 1))) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {            // P comes in halves of 64 rows of V
            if (!(ok = sh.wait_uniform(p, sh.p_full(i, h), p_phase >> i & 1))) break;
            tc5::fence_after();
#pragma unroll
            for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
              mma_tmem_a(leader, o, pa + ks * 8, b + ks * (16 * 128 >> 4), idesc_o, more_o || ks > 0);
            if constexpr (WIDE_P) {
#pragma unroll
              for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                mma_tmem_a(leader, o, pa + 64 + ks * 8, b + ks * (16 * 128 >> 4), idesc_o, 1);
            }
          }
          if (!ok) break;
          p_phase ^= 1u << i;
          started |= 1u << i;
        }
        if (j + ahead < mine) scores(i, at.slot);
      }
      if (!ok) break;
      commit_one(leader, sh.empty(v.slot));
      if (more) {
        commit_one(leader, sh.empty(at.slot));
        at.next();
      }
    }
    for (int i = 0; i < 2 && ok; ++i) {
      if (started >> i & 1) {
        commit_one(leader, sh.o_full(i));
      } else {
        if (k > 0 && !(ok = sh.wait_uniform(p, sh.o_empty(i), (k - 1) & 1))) break;
        arrive_one(leader, sh.o_full(i));
      }
    }
    if (!ok) break;
    arrive_one(leader, sh.item_empty(k));
    // the output's place
    if (!(ok = sh.wait_uniform(p, sh.full(at.slot), at.phase))) break;
    arrive_one(leader, sh.empty(at.slot));
    at.next();
  }
  // every MMA has completed before TMEM is freed
  if (any) commit_one(leader, sh.fin());
  else arrive_one(leader, sh.fin());
  volatile int never = 0;
  if (leader) mbar_wait_bounded(sh.fin(), 0, &never);
  __syncwarp();
}

// A bit of 0x80008000 for each infinity or NaN of two bf16, among other bits.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
constexpr uint32_t kNotFinite2 = 0x80008000u;
// All ones over each of them that is finite.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  const uint32_t f = not_finite2(w);
  return (f & 0x8000u ? 0u : 0xffffu) | (f & 0x80000000u ? 0u : 0xffff0000u);
}

// What was not finite in V, and was cleared, goes to the outputs of an item's queries that see it:
// they become infinite or NaN in its column.  A warp, each lane D / 32 columns, once up the rows and
// the tokens: of each column the last row with an infinity of either sign and with a NaN is kept,
// and a token sees one if it is not behind its window.  (2 of 8192 tokens, 32 heads on 8, without a
// finite value in V: 2.5 ms, and 0.94 with finite ones; on 32: 4.7 and 0.98, 42 where each token
// went through its rows by itself.)
template <class Cfg>
__device__ __forceinline__ void add_values(const AttendParams& p, const Item& w, const PartSeen& part) {
  constexpr int D = Cfg::D, EPL = D / 32, kNone = -0x7fffffff, kAlways = 0x7fffffff;
  const int c0 = (threadIdx.x & 31) * EPL;
  const long long v0 = ((long long)(p.b_offset + w.b) * p.h_kv + w.kvh) * p.n_max;
  const uint16_t* V = static_cast<const uint16_t*>(p.V) + v0 * D + c0;
  const bool narrow = w.part < 0 && p.out_bf16;
  const int last = p.by_group.div(w.row0 + w.rows - 1);
  int t = p.by_group.div(w.row0), plus[EPL], minus[EPL], nan[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) plus[e] = minus[e] = nan[e] = kNone;
  // the outputs of the tokens at rows below l
  auto finish = [&](int l) {
#pragma unroll 1
    for (; t <= last && w.past + t < l; ++t) {
      const int lo = p.window ? w.past + t + 1 - p.window : 0;
      float add[EPL];
      bool any = false;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        add[e] = (plus[e] >= lo ? INFINITY : 0.f) + (minus[e] >= lo ? -INFINITY : 0.f);
        if (nan[e] >= lo) add[e] = INFINITY - INFINITY;
        any |= !(add[e] == 0.f);
      }
      if (!__any_sync(0xffffffffu, any)) continue;
      const int end = min((t + 1) * p.group, w.row0 + w.rows);
#pragma unroll 1
      for (int flat = max(t * p.group, w.row0); flat < end; ++flat) {
        const long long off = w.part >= 0
                                  ? ((long long)w.part + flat - w.row0) * D
                                  : w.b * p.out_stride[0] + t * p.out_stride[2] +
                                        (w.kvh * p.group + flat - t * p.group) * p.out_stride[1];
        if (!DA_IN(p, off + D - 1, w.part >= 0 ? p.part_rows * D : p.out_elems)) continue;
        float* y = (w.part >= 0 ? p.o_part : static_cast<float*>(p.out)) + off + c0;
        __nv_bfloat16* z = static_cast<__nv_bfloat16*>(p.out) + off + c0;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          if (add[e] == 0.f) continue;
          if (narrow) z[e] = __float2bfloat16_rn(__bfloat162float(z[e]) + add[e]);
          else y[e] += add[e];
        }
      }
    }
  };
#pragma unroll 1
  for (int j = 0; j < w.count; ++j) {
    const int r0 = tile_row(w, w.begin + j), end = min(r0 + kTile, w.n);
    if (!edge_tile<true>(p, w, part, r0)) continue;
#pragma unroll 1
    for (int l = r0; l < end; ++l) {
      // (the rows that were looked through)
      if (l <= part.hi && (l >= part.lo || r0 + kTile <= p.prefix)) continue;
      if (!DA_IN(p, v0 + l, (long long)(p.b_offset + p.B) * p.h_kv * p.n_max)) continue;
      finish(l);
      const int seen = l < p.prefix ? kAlways : l;
      const uint32_t* at = reinterpret_cast<const uint32_t*>(V + (long long)l * D);
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const uint32_t v = e & 1 ? at[e / 2] >> 16 : at[e / 2] & 0xffffu;
        if (!(not_finite2(v) & 0x8000u)) continue;
        if (v & 0x7fu) nan[e] = max(nan[e], seen);
        else if (v & 0x8000u) minus[e] = max(minus[e], seen);
        else plus[e] = max(plus[e], seen);
      }
    }
  }
  finish(kAlways);
}

// ---- V rows that some query does not see: a warp
template <class Cfg, bool MANY>
__device__ __forceinline__ void attend_clear(const AttendParams& p, const AttendShared<Cfg>& sh) {
  constexpr int kChunks = Cfg::D / 8;  // 16-byte pieces of a row
  const int lane = threadIdx.x & 31;
  int edges = 0, place = 0;            // place of the item's first load in the ring
  for (int k = 0;; ++k) {
    if (!sh.wait_warp(p, sh.item_full(k), (k >> 1) & 1)) return;
    const Item& w = sh.items[k & 1];
    const int count = w.count;
    if (count < 0) return;
    const int ahead = lookahead(w), seen_end = w.n, clear_lo = w.clear_lo;
    const PartSeen part = MANY ? part_seen(p, w) : PartSeen{};
    bool bad = false;                  // some of V was not finite
    for (int j = 0; j < count; ++j) {
      const int r0 = tile_row(w, w.begin + j);
      if (!edge_tile<MANY>(p, w, part, r0)) continue;
      if (!sh.wait_warp(p, sh.edge(edges), (edges / kEdges) & 1)) return;
      ++edges;
      const int slot = (place + j + min(count, ahead + j)) % Cfg::kSlots;  // V_j's
      uint8_t* vt = sh.ring + size_t(slot) * Cfg::kTileBytes;
      auto piece = [&](int x) -> uint4& {
        return *reinterpret_cast<uint4*>(vt + tc5::sw128(x / kChunks, (x % kChunks) * 8, kTile));
      };
      if (!MANY || r0 + kTile > seen_end || (r0 < clear_lo && r0 + kTile > p.prefix)) {
#pragma unroll 8
        for (int x = lane; x < kTile * kChunks; x += 32) {
          const int row = r0 + x / kChunks;
          if (row >= seen_end || (row < clear_lo && row >= p.prefix)) piece(x) = make_uint4(0, 0, 0, 0);
        }
      }
      if constexpr (MANY) {  // rows that some queries do not see
        __syncwarp();
        auto look = [&](int from, int to) {
          uint32_t found = 0;
#pragma unroll 8
          for (int x = from * kChunks + lane; x < to * kChunks; x += 32) {
            const uint4 v = piece(x);
            found |= not_finite2(v.x) | not_finite2(v.y) | not_finite2(v.z) | not_finite2(v.w);
          }
          if (!__any_sync(0xffffffffu, (found & kNotFinite2) != 0)) return;
          bad = true;
          for (int x = from * kChunks + lane; x < to * kChunks; x += 32) {
            uint4 v = piece(x);
            v.x &= finite_halves(v.x), v.y &= finite_halves(v.y);
            v.z &= finite_halves(v.z), v.w &= finite_halves(v.w);
            piece(x) = v;
          }
        };
        const int end = min(seen_end - r0, kTile), past = min(max(part.hi + 1 - r0, 0), kTile);
        look(past, end);
        if (r0 + kTile > p.prefix) look(0, min(part.lo - r0, min(past, end)));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.full(slot));
    }
    place = (place + 2 * count + 1) % Cfg::kSlots;
    __syncwarp();
    if constexpr (MANY) {
      if (bad) {
        const Item mine = w;
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.item_empty(k));
        // (which completes when the item's outputs have been written, and not again before the next
        // arrival here)
        if (!sh.wait_warp(p, sh.item_empty(k), (k >> 1) & 1)) return;
        add_values<Cfg>(p, mine, part);
        continue;
      }
    }
    if (lane == 0) mbar_arrive(sh.item_empty(k));
  }
}

// Q of an item's rows of a softmax warp, swizzled K-major, for stream i (alternate: for
// both): asynchronous copies, rows past the unit left as they are.  The MMAs that read
// the buffer before have completed.
template <class Cfg>
__device__ __forceinline__ void start_q(const AttendParams& p, const AttendShared<Cfg>& sh,
                                        const Item& w, int i, int quarter) {
  constexpr int D = Cfg::D, kChunks = D / 8, kPer = 32 / kChunks;  // 16-byte pieces; rows at a time
  const int lane = threadIdx.x & 31;
  const bool alternate = alternates(w);
  const int rows = (alternate ? w.rows : min(w.rows - i * kTile, kTile)) - quarter * 32;
  if (rows <= 0 || (alternate && i == 1)) return;
  long long q_off = 0;
  if (lane < rows) {
    const int flat = w.row0 + i * kTile + quarter * 32 + lane;
    const int t = p.by_group.div(flat), head = w.kvh * p.group + flat - t * p.group;
    q_off = (w.b < 0 ? t : w.b) * p.q_stride[0] + head * p.q_stride[1] +
            (w.b < 0 ? 0 : t) * p.q_stride[2];
  }
  const char* q = static_cast<const char*>(p.q) + lane % kChunks * 16;
  const uint32_t to = smem_u32(sh.q_tile) + (alternate ? w.q_buf : i) * Cfg::kTileBytes;
#pragma unroll 4
  for (int y = 0; y < 32; y += kPer) {
    const int row = y + lane / kChunks;
    const long long off = __shfl_sync(0xffffffffu, q_off, row);
    if (row < rows && DA_IN(p, off + D - 1, p.q_elems))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       to + tc5::sw128(quarter * 32 + row, (lane % kChunks) * 8, kTile)),
                   "l"(q + off * 2)
                   : "memory");
  }
}
// And its arrival for the MMAs.
template <class Cfg>
__device__ __forceinline__ void finish_q(const AttendShared<Cfg>& sh, const Item& w, int i,
                                         int quarter) {
  const bool alternate = alternates(w);
  const int rows = (alternate ? w.rows : min(w.rows - i * kTile, kTile)) - quarter * 32;
  if (rows <= 0 || (alternate && i == 1)) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    // the stream's first warp arrives for those without rows
    const uint32_t arrivals = quarter == 0 ? 4 - (rows - 1) / 32 : 1;
    mbar_arrive_n(sh.q_full(i), arrivals);
  }
}

// ---- the softmax of stream i and the output: four warps
template <class Cfg, bool WIDE_P>
__device__ __forceinline__ void attend_softmax(const AttendParams& p, const AttendShared<Cfg>& sh) {
  constexpr int D = Cfg::D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = warp >> 2;                          // stream
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;                // row of the stream = TMEM lane
  const uint32_t lanes = uint32_t(quarter * 32) << 16;
  const uint32_t s_col = sh.tmem + i * 128 + lanes, o_col0 = sh.tmem + 256 + lanes;
  const uint32_t o_col = o_col0 + i * D;
  uint32_t tiles = 0;                               // of this stream: the parity of s_full
  uint32_t met = 0;                                 // items of both streams on the same rows
  if (!sh.wait_warp(p, sh.item_full(0), 0)) return;
  if (sh.items[0].count >= 0) {
    start_q<Cfg>(p, sh, sh.items[0], i, quarter);
    finish_q<Cfg>(sh, sh.items[0], i, quarter);
  }
  uint32_t place = 0;                               // of the item's first load, not wrapped

  for (int k = 0;; ++k) {
    const Item& w = sh.items[k & 1];                // (its barrier was waited for with Q)
    const int count = w.count;
    if (count < 0) return;
    const bool alternate = alternates(w), pre = w.b < 0;
    const int first_row = w.row0 + (alternate ? 0 : i * kTile);
    const int rows = alternate ? w.rows : min(w.rows - i * kTile, kTile);
    // Warps without a query row stay out of the tiles (their rows of S, P and O are
    // never looked at); the stream's first warp arrives for them.
    const bool works = quarter * 32 < rows;
    const uint32_t arrivals = quarter == 0 ? 4 - (rows - 1) / 32 : 1;
    const bool valid = r < rows;
    const int begin = w.begin, first = w.first, pt = w.pt;
    // this row's position and where its output goes
    int hi = -1, lo = 0;
    long long out_off = 0;
    if (valid) {
      const int flat = first_row + r;
      const int t = p.by_group.div(flat), head = w.kvh * p.group + flat - t * p.group;
      hi = w.past + (pre ? 0 : t);
      lo = pre || !p.window ? 0 : hi + 1 - p.window;
      out_off = (pre ? t : w.b) * p.out_stride[0] + head * p.out_stride[1] +
                (pre ? 0 : t) * p.out_stride[2];
    }
    float m_run = -INFINITY, l_run = 0.f;
    const uint32_t tiles0 = tiles;
    if (works) {
      // Tiles from here on need the mask: rows past the stream's first query, and of the
      // window's start up to its last query's.
      const int hi_first = pre ? w.past : w.past + p.by_group.div(first_row);
      const int lo_last =
          pre || !p.window ? 0 : max(0, w.past + p.by_group.div(first_row + rows - 1) + 1 - p.window);
      const int end = w.upto[i], step = alternate ? 2 : 1;
      for (int j = alternate ? i : 0; j < end; j += step) {
        // (warp-uniform: the TMEM accesses below are .sync.aligned)
        if (!sh.wait_warp(p, sh.s_full(i), tiles & 1)) return;
        tc5::fence_after();
        const int r0 = (begin + j < pt ? begin + j : first + begin + j - pt) * kTile;
        uint32_t raw[kTile];
        float* s = reinterpret_cast<float*>(raw);
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(s_col + c, raw + c);
        tc5::wait_ld();
        if (r0 + kTile - 1 > hi_first || (r0 < lo_last && r0 + kTile > p.prefix)) {
          const int hi_c = hi - r0, lo_c = lo - r0, pre_c = p.prefix - r0;
#pragma unroll
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            // a bit for each column that the row sees
            const uint32_t seen = bits_below(hi_c + 1 - c0) &
                                  (~bits_below(lo_c - c0) | bits_below(pre_c - c0));
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c0 + c] = seen >> c & 1 ? s[c0 + c] : -INFINITY;
          }
        }
        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) m4[x] = fmaxf(fmaxf(m4[x], s[c + x]), s[c + 4 + x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) m4[x] = fmaxf(m4[x], s[124 + x]);
        const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const bool over = m_tile > m_run + p.lazy || (m_run == -INFINITY && m_tile > -INFINITY);
        if (__any_sync(0xffffffffu, over)) {
          const float m_new = over ? m_tile : m_run;
          const float alpha = over ? ex2((m_run - m_new) * p.scale_log2) : 1.f;  // 0 from -inf
          m_run = m_new;
          l_run *= alpha;
          if (tiles != tiles0) {  // (S of this tile was issued behind the P.V of the last)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_col + c, o);
              tc5::wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st32(o_col + c, o);
            }
          }
        }
        const float shift = m_run == -INFINITY ? 0.f : -m_run * p.scale_log2;
        const uint64_t scale2 = pair_of(p.scale_log2, p.scale_log2), shift2 = pair_of(shift, shift);
        uint64_t l2[2] = {0, 0};
        // P over the first columns of S, which every lane of the warp has loaded.  Its first
        // half goes to the MMAs while the second is computed: behind the third quarter, when
        // its stores are done without a wait.
        uint32_t hi_p[32], lo_p[WIDE_P ? 32 : 1];
        auto quarter_of_p = [&](int c0) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float a, b;
            halves_of(fma2(pair_of(s[c0 + c], s[c0 + c + 1]), scale2, shift2), a, b);
            a = ex2(a);
            b = ex2(b);
            l2[(c >> 1) & 1] = add2(l2[(c >> 1) & 1], pair_of(a, b));
            const int at = (c0 & 32) / 2 + c / 2;
            hi_p[at] = pack_bf16x2(a, b);
            if constexpr (WIDE_P)
              lo_p[at] = pack_bf16x2(a - bf16_lo_to_f32(hi_p[at]), b - bf16_hi_to_f32(hi_p[at]));
          }
        };
        auto store_half = [&](int h) {
          tmem_st32(s_col + 32 * h, hi_p);
          if constexpr (WIDE_P) tmem_st32(s_col + 64 + 32 * h, lo_p);
        };
        auto hand_over = [&](int h) {
          tc5::wait_st();
          tc5::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_n(sh.p_full(i, h), arrivals);
        };
        quarter_of_p(0);
        quarter_of_p(32);
        store_half(0);
        quarter_of_p(64);
        hand_over(0);
        quarter_of_p(96);
        store_half(1);
        hand_over(1);
        float la, lb;
        halves_of(add2(l2[0], l2[1]), la, lb);
        l_run += la + lb;
        ++tiles;
      }
    }
    // (warps that stayed out count along)
    const int own_tiles = alternate ? (count - i + 1) / 2 : w.upto[i];
    tiles = tiles0 + own_tiles;
    // Q of the next item, for its first scores to run under the end of this one
    if (!sh.wait_warp(p, sh.item_full(k + 1), ((k + 1) >> 1) & 1)) return;
    const Item& next = sh.items[(k + 1) & 1];
    // The stream's own score MMAs are complete, and of two items of one set of rows each has
    // its buffer; else behind both streams' below.  (And a warp that stayed out has not seen
    // this item's Q arrive yet.)
    const bool early = works && own_tiles > 0 && (!alternate || alternates(next));
    if (early && next.count >= 0) start_q<Cfg>(p, sh, next, i, quarter);

    place += 2 * count;
    const int out_slot = int(place % Cfg::kSlots);
    const uint32_t out_phase = (place / Cfg::kSlots) & 1;
    ++place;
    // ---- the rows' sums are final once the MMAs are
    float* pairs = sh.pairs;
    if (alternate) {
      pairs[i * 2 * kTile + r] = m_run;
      pairs[i * 2 * kTile + kTile + r] = l_run;
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.meet(0));
      if (!sh.wait_warp(p, sh.meet(0), met & 1)) return;
      if (!sh.wait_warp(p, sh.o_full(1 - i), k & 1)) return;
    }
    if (!sh.wait_warp(p, sh.o_full(i), k & 1)) return;
    // (whether it is used or not: else its out_done could be a phase ahead of the producer's wait)
    if (!sh.wait_warp(p, sh.full(out_slot), out_phase)) return;
    tc5::fence_after();
    if (next.count >= 0) {
      if (early) finish_q<Cfg>(sh, next, i, quarter);
      else start_q<Cfg>(p, sh, next, i, quarter);
    }
    if (works) {
      // Weights of the streams' O.  Alternate: of streams 0 and 1, and each stream's warps
      // take a half of the columns.
      float keep0 = 1.f, keep1 = 0.f;
      if (alternate) {
        const float m0 = pairs[r], m1 = pairs[2 * kTile + r];
        m_run = fmaxf(m0, m1);
        const float use = m_run == -INFINITY ? 0.f : m_run;
        keep0 = ex2((m0 - use) * p.scale_log2);
        keep1 = ex2((m1 - use) * p.scale_log2);
        l_run = pairs[kTile + r] * keep0 + pairs[3 * kTile + r] * keep1;
      }
      const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
      keep0 *= inv;
      keep1 *= inv;
      const bool part = w.part >= 0, narrow = !part && p.out_bf16;
      const long long part_row = (long long)w.part + (alternate ? 0 : i * kTile) + r;
      if (part) out_off = part_row * D;
      const long long extent = part ? p.part_rows * D : p.out_elems;
      if (part && valid && !(alternate && i == 1) &&
          DA_IN(p, part_row, p.part_rows))
        p.lse_part[part_row] =
            l_run > 0.f ? m_run * p.scale_log2 + log2f(l_run) : (l_run == 0.f ? -INFINITY : l_run);
      char* base = static_cast<char*>(part ? static_cast<void*>(p.o_part) : p.out);
      if (alternate) {
        // (few rows as a rule) each lane its row's half of the columns
        const bool in = valid && DA_IN(p, out_off + D - 1, extent);
        char* y = base + out_off * (narrow ? 2 : 4);
#pragma unroll 1
        for (int c = i * (D / 2); c < (i + 1) * (D / 2); c += 16) {
          float f[16];
          if (count > 0) {
            tc5::ld16(o_col0 + c, f);
            tc5::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] *= keep0;
            if (count > 1) {
              float f1[16];
              tc5::ld16(o_col0 + D + c, f1);
              tc5::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) f[e] = fmaf(f1[e], keep1, f[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = 0.f;
          }
          if (in && narrow) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(y + (c + e) * 2) =
                  make_uint4(pack_bf16x2(f[e], f[e + 1]), pack_bf16x2(f[e + 2], f[e + 3]),
                             pack_bf16x2(f[e + 4], f[e + 5]), pack_bf16x2(f[e + 6], f[e + 7]));
          } else if (in) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(y + (c + e) * 4) =
                  make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          }
          __syncwarp();
        }
      } else {
        // Through the ring's place, D bytes of each of the warp's rows at a time, so that rows
        // are written in runs of D bytes.
        const int mine = min(rows - quarter * 32, 32);  // rows of this warp
        const int cols = narrow ? D / 2 : D / 4;
        constexpr int kChunks = D / 16, kPer = 32 / kChunks;  // 16-byte pieces; rows at a time
        uint8_t* stage = sh.ring + out_slot * Cfg::kTileBytes + warp * (Cfg::kTileBytes / 8);
#pragma unroll 1
        for (int c = 0; c < D; c += cols) {
#pragma unroll 2
          for (int x = 0; x < cols; x += 16) {
            float o[16];
            if (own_tiles > 0) {
              tc5::ld16(o_col + c + x, o);
              tc5::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= keep0;
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0.f;
            }
            auto put = [&](int chunk, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
              *reinterpret_cast<uint4*>(stage + lane * D + ((chunk ^ (lane & (kChunks - 1))) << 4)) =
                  make_uint4(v0, v1, v2, v3);
            };
            if (narrow) {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                put((x + e) / 8, pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                    pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                put((x + e) / 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]),
                    __float_as_uint(o[e + 2]), __float_as_uint(o[e + 3]));
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int y = 0; y < mine; y += kPer) {
            const int row = y + lane / kChunks, ch = lane % kChunks;
            const long long off = __shfl_sync(0xffffffffu, out_off, row & 31) + c;
            const uint4 v =
                *reinterpret_cast<const uint4*>(stage + row * D + ((ch ^ (row & (kChunks - 1))) << 4));
            if (row < mine && DA_IN(p, off + cols - 1, extent))
              *reinterpret_cast<uint4*>(base + off * (narrow ? 2 : 4) + ch * 16) = v;
          }
          __syncwarp();
        }
      }
    }
    if (!early && next.count >= 0) finish_q<Cfg>(sh, next, i, quarter);
    fence_proxy_async_smem();  // the ring's next load there comes after these rows
    tc5::fence_before();
    __syncwarp();
    if (lane == 0) {
      if (alternate) {
        mbar_arrive(sh.o_empty(0));
        mbar_arrive(sh.o_empty(1));
        mbar_arrive(sh.meet(1));
      } else {
        mbar_arrive_n(sh.o_empty(i), 2);
      }
      mbar_arrive(sh.out_done(out_slot));
      mbar_arrive(sh.item_empty(k));
    }
    // both streams have read the shared sums
    if (alternate && !sh.wait_warp(p, sh.meet(1), met++ & 1)) return;
  }
}

template <class Cfg, bool WIDE_P, bool MANY>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendMaps maps, const AttendParams p) {
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem[];
  AttendShared<Cfg> sh;
  sh.q_tile = smem;
  sh.ring = smem + 2 * Cfg::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sh.ring + size_t(Cfg::kSlots) * Cfg::kTileBytes);
  sh.bars = smem_u32(bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::kBars);
  sh.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  sh.pairs = reinterpret_cast<float*>(tmem_slot + 2);
  sh.line = reinterpret_cast<LineStart*>(sh.pairs + 4 * kTile);
  sh.items = reinterpret_cast<Item*>(sh.line + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(sh.full(s), 1);
      mbar_init(sh.empty(s), 1);       // a tcgen05.commit
      mbar_init(sh.out_done(s), 8);    // softmax warps
    }
    for (int e = 0; e < kEdges; ++e) mbar_init(sh.edge(e), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh.q_full(i), 4);      // softmax warps
      mbar_init(sh.s_full(i), 1);
      mbar_init(sh.p_full(i, 0), 4);
      mbar_init(sh.p_full(i, 1), 4);
      mbar_init(sh.o_full(i), 1);
      mbar_init(sh.o_empty(i), 8);
      mbar_init(sh.item_full(i), 1);
      mbar_init(sh.item_empty(i), kItemReaders);
      mbar_init(sh.meet(i), 8);
    }
    mbar_init(sh.fin(), 1);
    mbar_init(sh.answered(), 1);
    *sh.abort_flag = 0;
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
  if (p.list) line_start(p, reinterpret_cast<long long*>(sh.ring), sh.line);
  else __syncthreads();
  // lengths that were clamped are reported (without a list, by whoever takes a sequence's unit)
  if (p.list && blockIdx.x == 0 && p.dev_error)
    for (int b = threadIdx.x; b < p.B; b += kAttendThreads) {
      bool bad_n, bad_m;
      const int n = seq_rows(p, b, bad_n), m = seq_new(p, b, bad_m);
      report_lengths(p, bad_n || bad_m || (m > n && !p.shared));
    }
  tc5::fence_after();
  sh.tmem = *tmem_slot;

  // Registers: 168 a thread at launch for each of three warpgroups; 2 * 208 + 88 then.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      if (lane == 0) attend_load<Cfg, MANY>(p, maps, sh);
    } else if (warp == 9) {
      attend_mma<Cfg, WIDE_P>(p, sh);
      named_bar_sync(2, 288);
      tc5::fence_after();
      tc5::dealloc(sh.tmem, kTmemCols);
    } else if (warp == 10) {
      attend_clear<Cfg, MANY>(p, sh);
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  attend_softmax<Cfg, WIDE_P>(p, sh);
  tc5::fence_before();
  named_bar_sync(2, 288);
}

// ---------------------------------------------------------------------------
// Combine: a warp per query row merges the partials of its unit's items (and,
// behind a shared prefix, of the prefix unit's) by their log-sum-exps.
// ---------------------------------------------------------------------------
constexpr int kAttendCombineWarps = 8;

// Row `off` of the output from partials: rows first, first + step, ... (count0 of them),
// then first1, ... (count1).
template <int D>
__device__ __forceinline__ void merge_row(const AttendParams& p, long long off, long long first0,
                                          long long step0, int count0, long long first1,
                                          long long step1, int count1) {
  constexpr int EPL = D / 32, NB = 8;  // columns a lane, partials in flight
  const int lane = threadIdx.x & 31, parts = count0 + count1;
  float m = -INFINITY, sum = 0.f, acc[EPL];
#pragma unroll
  for (int k = 0; k < EPL; ++k) acc[k] = 0.f;
  for (int s0 = 0; s0 < parts; s0 += NB) {
    float l[NB], v[NB][EPL];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int s = s0 + u;
      const long long row = s < count0 ? first0 + s * step0 : first1 + (s - count0) * step1;
      const bool in = s < parts && DA_IN(p, row, p.part_rows);
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
  off += lane * EPL;
  if (!DA_IN(p, off + EPL - 1, p.out_elems)) return;
  if (p.out_bf16) {
    uint32_t* y = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + off);
#pragma unroll
    for (int k = 0; k < EPL; k += 2) y[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  } else {
#pragma unroll
    for (int k = 0; k < EPL; ++k) static_cast<float*>(p.out)[off + k] = acc[k] * inv;
  }
}

// The first and last CTA noted for a unit; (0, -1) where there are none.  A CTA whose wait ran
// out notes nothing for the rest of its piece, whose words then hold what the workspace held: only
// CTAs of the grid, in order, are followed.
__device__ __forceinline__ int2 noted_ctas(const AttendParams& p, bool there, int unit) {
  const int2 c = there ? __ldcg(p.unit_ctas + unit) : make_int2(0, -1);
  return c.x >= 0 && c.x <= c.y && c.y < p.ctas ? c : make_int2(0, -1);
}

// Behind a shared prefix: every row, of the CTAs noted for its units.
template <int D>
__global__ void __launch_bounds__(kAttendCombineWarps * 32)
    attend_merge_kernel(const AttendParams p) {
  allow_dependent_launch();
  const int row = int(blockIdx.x) * kAttendCombineWarps + int(threadIdx.x >> 5);
  if (row >= p.B * p.h_q) return;
  const int b = row / p.h_q, head = row - b * p.h_q;
  const int kvh = p.by_group.div(head), hh = head - kvh * p.group;
  wait_for_prerequisite_grid();
  bool bad;
  const bool own = seq_rows(p, b, bad) > 0;
  // the prefix unit's rows are those of all sequences, one after the other
  const int flat = b * p.group + hh, mt = flat / kAttendRows;
  const int pre_unit = kvh * p.prefix_tiles + mt;
  const int qt = hh / kAttendRows;
  const int own_unit = ((p.q_tiles - 1 - qt) * p.B + b) * p.h_kv + kvh;
  const int2 pre = noted_ctas(p, p.P > 0, pre_unit);
  const int2 mine = noted_ctas(p, own, p.h_kv * p.prefix_tiles + own_unit);
  merge_row<D>(p, b * p.out_stride[0] + head * p.out_stride[1],
               (long long)(pre_unit + pre.x) * p.pitch + flat % kAttendRows, p.pitch,
               pre.y - pre.x + 1,
               p.own_parts + (long long)(own_unit + mine.x) * p.unit_rows + hh % kAttendRows,
               p.unit_rows, mine.y - mine.x + 1);
}

// A chunk: the rows of the units that were cut, each taken at its first cut.
// Which cut that is, and the rows from r0 on; false: none.
struct JoinUnit {
  int b, qt, kvh, first, last, rows;   // CTAs of its first and last items
};
__device__ __forceinline__ bool join_unit(const AttendParams& p, int r0, int most, JoinUnit& u) {
  const int c = blockIdx.y + 1;        // a CTA whose piece starts inside a unit
  const int4 at = __ldcg(p.cta_start + c);
  if (at.x < 0 || __ldcg(p.cta_start + c - 1).x == at.x) return false;
  entry_of(p, at.y, u.b, u.qt);
  u.kvh = at.z;
  bool bad;
  const long long left = (long long)seq_new(p, u.b, bad) * p.group - (long long)u.qt * kAttendRows - r0;
  u.rows = int(min((long long)min(most, p.unit_rows - r0), left));
  if (u.rows <= 0) return false;
  u.first = c - 1;
  u.last = c;
  while (u.last + 1 < p.ctas && __ldcg(p.cta_start + u.last + 1).x == at.x) ++u.last;
  return true;
}
// Where row r of the unit goes.
__device__ __forceinline__ long long join_out(const AttendParams& p, const JoinUnit& u, int r) {
  const int flat = u.qt * kAttendRows + r;
  const int t = p.by_group.div(flat), h = flat - t * p.group;
  return u.b * p.out_stride[0] + (long long)(u.kvh * p.group + h) * p.out_stride[1] +
         t * p.out_stride[2];
}

// Few rows, cut into many items as a rule (few tokens behind a long context): a warp a row.
template <int D>
__global__ void __launch_bounds__(kAttendCombineWarps * 32)
    attend_join_few_kernel(const AttendParams p) {
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  const int r = int(blockIdx.x) * kAttendCombineWarps + int(threadIdx.x >> 5);
  JoinUnit u;
  if (!join_unit(p, r, 1, u)) return;
  // the first item ends its CTA's piece, the others start theirs
  merge_row<D>(p, join_out(p, u, r), (2LL * u.first + 1) * p.pitch + r, 0, 1,
               2LL * (u.first + 1) * p.pitch + r, 2LL * p.pitch, u.last - u.first);
}

// More rows, cut in two as a rule: a warp takes four at once and the partials one after the
// other (a warp a row took 28 us of launching behind 150 CTAs; 8 tokens of 131072 rows, ten
// items a unit, took 7 us more this way than the other).
constexpr int kJoinRows = 4;

template <int D>
__global__ void __launch_bounds__(kAttendCombineWarps * 32, 4)
    attend_join_kernel(const AttendParams p) {
  constexpr int EPL = D / 32;                // columns a lane
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  const int lane = threadIdx.x & 31;
  const int r0 = (int(blockIdx.x) * kAttendCombineWarps + int(threadIdx.x >> 5)) * kJoinRows;
  JoinUnit u;
  if (!join_unit(p, r0, kJoinRows, u)) return;
  const int rows = u.rows;
  float m[kJoinRows], sum[kJoinRows], acc[kJoinRows][EPL];
#pragma unroll
  for (int y = 0; y < kJoinRows; ++y) {
    m[y] = -INFINITY;
    sum[y] = 0.f;
#pragma unroll
    for (int k = 0; k < EPL; ++k) acc[y][k] = 0.f;
  }
  for (int s = u.first; s <= u.last; ++s) {
    // the first item ends its CTA's piece, the others start theirs
    const long long row = (2LL * s + (s == u.first)) * p.pitch + r0;
    float l[kJoinRows], v[kJoinRows][EPL];
#pragma unroll
    for (int y = 0; y < kJoinRows; ++y) {
      const bool in = y < rows && DA_IN(p, row + y, p.part_rows);
      l[y] = in ? __ldcg(p.lse_part + row + y) : -INFINITY;
#pragma unroll
      for (int k = 0; k < EPL; k += 2) {
        const float2 f = in ? __ldcg(reinterpret_cast<const float2*>(p.o_part + (row + y) * D + lane * EPL + k))
                            : make_float2(0.f, 0.f);
        v[y][k] = f.x, v[y][k + 1] = f.y;
      }
    }
#pragma unroll
    for (int y = 0; y < kJoinRows; ++y) {
      const float top = fmaxf(m[y], l[y]), use = top == -INFINITY ? 0.f : top;
      const float a = ex2(m[y] - use), f = ex2(l[y] - use);
      sum[y] = sum[y] * a + f;
#pragma unroll
      for (int k = 0; k < EPL; ++k) acc[y][k] = acc[y][k] * a + f * v[y][k];
      m[y] = top;
    }
  }
#pragma unroll
  for (int y = 0; y < kJoinRows; ++y) {
    if (y >= rows) break;
    const long long off = join_out(p, u, r0 + y) + lane * EPL;
    const float inv = sum[y] > 0.f ? 1.f / sum[y] : (sum[y] == 0.f ? 0.f : sum[y]);
    if (!DA_IN(p, off + EPL - 1, p.out_elems)) continue;
    if (p.out_bf16) {
      uint32_t* z = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + off);
#pragma unroll
      for (int k = 0; k < EPL; k += 2) z[k / 2] = pack_bf16x2(acc[y][k] * inv, acc[y][k + 1] * inv);
    } else {
#pragma unroll
      for (int k = 0; k < EPL; ++k) static_cast<float*>(p.out)[off + k] = acc[y][k] * inv;
    }
  }
}

template <class Cfg, bool WIDE_P, bool MANY>
cudaError_t launch_attend_cfg(const AttendParams& p, const AttendMaps& m, int grid,
                              cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e =
      set_smem_limit_once(attend_kernel<Cfg, WIDE_P, MANY>, Cfg::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(attend_kernel<Cfg, WIDE_P, MANY>, grid, kAttendThreads, Cfg::kSmemBytes,
                          stream, m, p);
}

// One token a sequence (and so behind a shared prefix) goes without the look through rows that
// only some queries see: 36.5 us for 38.3 (16 sequences behind 8192 rows), 141 for 147 (64 behind
// 32768).  Elsewhere that look costs 1 % (prompts 1020 -> 1029 us, ragged window 217 -> 220).
template <class Cfg>
cudaError_t launch_attend_d(const AttendParams& p, const AttendMaps& m, int grid,
                            cudaStream_t stream) {
  if (p.T > 1)
    return p.bf16_weights ? launch_attend_cfg<Cfg, false, true>(p, m, grid, stream)
                          : launch_attend_cfg<Cfg, true, true>(p, m, grid, stream);
  return p.bf16_weights ? launch_attend_cfg<Cfg, false, false>(p, m, grid, stream)
                        : launch_attend_cfg<Cfg, true, false>(p, m, grid, stream);
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, const AttendMaps& m, int d, int grid,
                          cudaStream_t stream) {
  return d == 128 ? launch_attend_d<AttendCfg<128>>(p, m, grid, stream)
                  : launch_attend_d<AttendCfg<64>>(p, m, grid, stream);
}

cudaError_t launch_attend_combine(const AttendParams& p, int d, cudaStream_t stream) {
  const int threads = kAttendCombineWarps * 32;
  if (p.shared) {
    const int grid = (p.B * p.h_q + kAttendCombineWarps - 1) / kAttendCombineWarps;
    return d == 128 ? launch_dependent(attend_merge_kernel<128>, grid, threads, 0, stream, p)
                    : launch_dependent(attend_merge_kernel<64>, grid, threads, 0, stream, p);
  }
  // (16 sequences of 16 tokens, 128 rows a unit, behind 8000 rows: 5 us less than a warp a row)
  const bool few = p.unit_rows <= 64;
  const int rows = kAttendCombineWarps * (few ? 1 : kJoinRows);
  const dim3 grid((p.unit_rows + rows - 1) / rows, p.ctas - 1);
  if (few)
    return d == 128 ? launch_dependent(attend_join_few_kernel<128>, grid, threads, 0, stream, p)
                    : launch_dependent(attend_join_few_kernel<64>, grid, threads, 0, stream, p);
  return d == 128 ? launch_dependent(attend_join_kernel<128>, grid, threads, 0, stream, p)
                  : launch_dependent(attend_join_kernel<64>, grid, threads, 0, stream, p);
}

}  // namespace da
