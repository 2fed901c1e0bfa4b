// Split-KV decode attention over 8-bit caches with one scale per block of
// tokens and head (sm_103a).
//
// A cached row of K (and of V) is D one-byte codes; the rows of a block of S
// consecutive tokens (S = 16, 32, 64 or 128) share one float32 scale per head:
// row l of K stands for ks[l / S] * value(code).  Steps I-III factor over the
// scales,
//   s[l]      = scale * ks[l / S] * sum_j q[j] * value(Kc[l][j])
//   out[h, d] = sum_l a[l] * vs[l / S] * value(Vc[l][d])
// and the score terms of ScoreTerms apply to s in float32.
//
// Bound: HBM.  A row costs 2 D bytes and 8 / S bytes of scales for 4 D flops a
// query head, so a group of 8 stays at 16 flops per byte, far below the fp16
// MMA rate per byte of HBM.
//
// Work.  A CTA of four warps takes one chunk of a (sequence, kv head, head
// chunk)'s rows, and three or four CTAs share an SM, so that one's start and end
// (loads of q, the merge of its warps) pass under the others' streams (one CTA of
// eight warps a SM: 40.8 us on 16 ragged int8 sequences with 8 kv heads).  Every
// CTA finds its chunk from the lengths (find_item_few, _many): the chunk length is the
// shortest whose chunks all fit on the GPU at once, so that there is one round
// of equal CTAs, whatever n_max is (31.9 us; 2.1 more with a length fixed by n_max).
// Beyond kBlockRoundRows rows a CTA there are two or three shorter rounds: HBM does
// not serve all SMs alike, and the CTAs of a later round go where an early one
// ended (2 x 131072 rows of fp8 with 64 query heads: 82.9 us, 6.5 TB/s; one round took
// 1.9 us more than two).  With 32 heads on one kv head the MMAs and the instructions
// around them, not HBM, are the bound: 33.3 us for 8 x 30000 rows, 9.2 us of HBM time.
// Caches of up to 4096 rows with few enough units (make_plan) need no list: a cluster
// of up to eight CTAs takes a unit's rows in equal shares and joins them through
// distributed shared memory (finish_cluster), without a second kernel.
// Within a CTA warp w takes the 32-row steps w, w + 4, ... of the chunk and
// feeds itself: its lane 0 keeps a ring of steps (K and V codes, 2 TMA boxes of
// 32 rows) in flight on the warp's own barriers, and no warp waits for another
// before the chunk's end.  A step holds two 16-row MMA blocks, so that the
// barrier, the maximum's shuffles and the rescaling come once for both and two
// independent chains fill each other's latencies (375 instructions a block with
// one block a step, 260 with two).
//
// Layout.  The boxes have a row's D bytes contiguous with the 128- or 64-byte
// swizzle; MMA A fragments are built from them in registers, no fp16 copy is
// written.  As S is a multiple of 16, a block of rows has ONE K scale and ONE V
// scale: a warp loads those of its next 32 blocks (16 steps) with one load per
// tensor (a lane per block), a group ahead, and takes each by a shuffle.
// With lane = 4 g + t:
//   Step I  (S^T = K . Q^T, rows of K as M): lane (g, t) reads bytes
//           [t D/4, (t + 1) D/4) of rows g and g + 8 of the block; k-block kb
//           takes the 4 codes at t D/4 + 4 kb as the A elements at logical
//           columns 2t, 2t+1, 2t+8, 2t+9.  That relabels the columns of d one to
//           one, and the q fragments are taken in the same order.
//   Step III (O^T += V^T . P^T, d as M): lane (g, t) reads bytes
//           [g D/8, (g + 1) D/8) of rows 2t, 2t+1, 2t+8, 2t+9; a byte permute
//           pairs a column's codes of two rows; m-block mb takes columns
//           g D/8 + 2 mb and + 1.
// The V scale multiplies P before P becomes fp16.  For a float32 output P is an
// fp16 head and an fp16 remainder (~22 bits, two MMAs).  For a bf16 output it is
// the head alone: 2^-11 of each weight, an eighth of the half step (2^-8) by which
// the output's own rounding moves it, and a third of the MMAs less (with the remainder
// the three steps named here take 2.1, 1.9 and 6.2 us more, for errors against 64 bits
// of 0.99 of these; a caller who wants the digits asks for a float32 output).
// Scales may be of any size (2^-126 for tiny rows), and fp16 has few exponents,
// so a warp keeps each head's accumulator in a unit that follows the largest
// weight times V scale that the head has seen, a second running maximum beside
// the softmax's: P is a weight times its V scale in that unit, and the unit
// returns at the chunk's end.  It differs from the softmax's reference by a power
// of two, so that P is rounded once.  (A unit for all heads that follows the V
// scales alone takes a head's digits where a block it gives no weight, or that only
// its neighbours weigh on, has a far larger scale; with that the same three steps take
// 31.2, 84.1 and 31.5 us, with this one 31.9, 82.9 and 33.3.)
#include <math.h>

#include "common.cuh"
#include "q8_codes.cuh"

namespace da {

// Shared memory of find_item: the lengths of a launch slice's sequences, and
// scratch for four warps.
constexpr int kFindWords = kMaxBatchPerLaunch + 4 * 32 + 16;

template <int D_, int NB_, int STAGES_, int CTAS_, int KIND_>
struct Q8BCfg {
  static constexpr int D = D_;
  static constexpr int NB = NB_;           // 8-head MMA blocks per CTA
  static constexpr int KW = 4;             // warps
  static constexpr int STAGES = STAGES_;   // steps in flight per warp
  static constexpr int ROWS = 32;          // rows of a step: two MMA blocks
  static constexpr int CTAS = CTAS_;       // CTAs per SM
  static constexpr int KIND = KIND_;       // 1: int8 codes, 2: fp8 e4m3 codes
  static constexpr int kHPW = 8 * NB;
  static constexpr int kThreads = 32 * KW;
  static constexpr int kCodeBytes = ROWS * D;           // a step's codes of one tensor
  static constexpr int kStepBytes = 2 * kCodeBytes;
  static constexpr int kRingBytes = KW * STAGES * kStepBytes;
  static constexpr int kSlotStride = D + 4;
  static constexpr int kEpiAccFloats = KW * kHPW * kSlotStride;
  static constexpr int kEpiMLFloats = 2 * KW * kHPW;
  // the merge of the warps reuses the ring
  static constexpr int kEpiBytes = (kEpiAccFloats + kEpiMLFloats) * 4;
  static constexpr int kDataBytes = kRingBytes > kEpiBytes ? kRingBytes : kEpiBytes;
  static constexpr size_t kSmemBytes =
      1024 + kDataBytes + KW * STAGES * 8 + 16 + kFindWords * 4;
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(KIND == 1 || KIND == 2, "code type");
  static_assert(CTAS * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
  static_assert(kDataBytes % 8 == 0, "mbarrier alignment");
};

// Quotients by one divisor: floor(x / d) for x < 2^31, by a multiplication that
// is at most one too high and a correction.
struct Divisor {
  unsigned d, by;
  __device__ __forceinline__ explicit Divisor(unsigned d_) : d(d_), by(0xffffffffu / d_ + 1) {}
  __device__ __forceinline__ int up(int x) const {  // ceil(x / d)
    const unsigned y = unsigned(x) + d - 1;
    const unsigned q = d > 1 ? __umulhi(y, by) : y;
    return int(q - (q * d > y));
  }
};

// The candidate chunk length of a lane.  With `rows` rows over the sequences
// (below 2^31: the cache's rows are), the launch may have `most` chunks: a round
// or more of the GPU's places; with more units than places, one for each unit and
// a round for the long ones' further chunks.  Lane k tries the k-th of 32 lengths
// between (all units' rows) / most, below which none can do, and rows / (most -
// units), which does.  In float: a candidate may be off by a row, but whether it
// does is counted exactly, and lane 31's, one chunk a unit, always does.
template <int ROWS>
__device__ __forceinline__ int candidate_chunk(const SplitParams& p, unsigned rows, int longest,
                                               int& most) {
  const int lane = threadIdx.x & 31;
  const int units = p.B * p.h_kv * p.head_chunks;
  const float all = float(rows) * float(p.h_kv * p.head_chunks);
  const int rounds =
      max(1, min(p.rounds, int(ceilf(all * __fdividef(1.f, float(p.places) * kBlockRoundRows)))));
  most = (units <= p.places ? 0 : units) + rounds * p.places;
  const float least = __fdividef(all, float(most));
  const float enough = most > units ? __fdividef(all, float(most - units)) : float(longest);
  float c = ceilf(fmaf(enough - least, float(lane) * (1.f / 31.f), least));
  c = fminf(fmaxf(c, float(kBlockMinRows)), float(longest));
  const int chunk = max(lane == 31 ? longest : int(c), p.chunk_min);
  return (chunk + ROWS - 1) / ROWS * ROWS;
}

// The blockIdx.x-th chunk of the launch slice, in `it`, and the chunk length;
// false when there are fewer.  Sequence b has max(1, ceil(n_b / chunk)) chunks for
// each kv head and head chunk; head chunks are neighbours, so that all but the
// first of them find the codes in L2.

// For at most 8 sequences: each warp by itself, lane b on sequence b, with its
// rows in n_b.
constexpr int kFewSequences = 8;

template <int ROWS>
__device__ __forceinline__ bool find_item_few(const SplitParams& p, int n_b, Item& it,
                                              int& chunk) {
  const int lane = threadIdx.x & 31;
  const int n = lane < p.B ? max(n_b, 1) : 0;  // (an empty sequence has one chunk, for its zeros)
  const int per_seq = p.h_kv * p.head_chunks;
  chunk = p.chunk_fixed;
  if (p.chunk_fixed <= 0) {
    unsigned rows = unsigned(n);
    int longest = n;
#pragma unroll
    for (int o = kFewSequences / 2; o > 0; o >>= 1) {
      rows += __shfl_xor_sync(0xffffffffu, rows, o);
      longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    rows = __shfl_sync(0xffffffffu, rows, 0);
    longest = __shfl_sync(0xffffffffu, longest, 0);
    int most;
    const int c = candidate_chunk<ROWS>(p, rows, longest, most);
    const Divisor by{unsigned(c)};
    int count = 0;
    for (int b = 0; b < p.B; ++b) count += by.up(__shfl_sync(0xffffffffu, n, b));
    const unsigned fits =
        __ballot_sync(0xffffffffu, (long long)count * per_seq <= most) | 0x80000000u;
    chunk = __shfl_sync(0xffffffffu, c, __ffs(int(fits)) - 1);
  }
  const int nv = lane < p.B ? Divisor{unsigned(chunk)}.up(n) : 0;
  const int mine = per_seq * nv;  // (the grid holds all chunks: an int)
  int upto = mine;
#pragma unroll
  for (int o = 1; o < kFewSequences; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int i = int(blockIdx.x);
  const unsigned here =
      __ballot_sync(0xffffffffu, lane < p.B && i >= upto - mine && i < upto);
  if (here == 0) return false;
  const int b = __ffs(int(here)) - 1;
  int at = __shfl_sync(0xffffffffu, i - (upto - mine), b);
  it.b = b;
  it.nv = __shfl_sync(0xffffffffu, nv, b);
  it.hc = at % p.head_chunks;
  at /= p.head_chunks;
  it.split = at % it.nv;
  it.kvh = at / it.nv;
  return true;
}

// For any number: all 128 threads, lengths in sm[0 .. B) (filled by the caller,
// not yet synchronised).
template <int ROWS>
__device__ __forceinline__ bool find_item_many(const SplitParams& p, int* sm, Item& it,
                                               int& chunk) {
  const int* lens = sm;
  int* scratch = sm + kMaxBatchPerLaunch;  // [4][32]
  int* found = scratch + 4 * 32;           // [16]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = p.h_kv * p.head_chunks;
  __syncthreads();  // lens
  chunk = p.chunk_fixed;
  if (p.chunk_fixed <= 0) {
    unsigned rows = 0;
    int longest = 1;
    for (int b = lane; b < p.B; b += 32) {  // every warp all of them: no barrier
      rows += unsigned(max(lens[b], 1));
      longest = max(longest, lens[b]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      rows += __shfl_xor_sync(0xffffffffu, rows, o);
      longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    int most;
    const int c = candidate_chunk<ROWS>(p, rows, longest, most);
    const Divisor by{unsigned(c)};
    int count = 0;
    for (int b = warp; b < p.B; b += 4) count += by.up(max(lens[b], 1));
    scratch[warp * 32 + lane] = count;
    __syncthreads();
    count = scratch[lane] + scratch[32 + lane] + scratch[64 + lane] + scratch[96 + lane];
    const unsigned fits =
        __ballot_sync(0xffffffffu, (long long)count * per_seq <= most) | 0x80000000u;
    chunk = __shfl_sync(0xffffffffu, c, __ffs(int(fits)) - 1);
  }
  // The sequence that holds chunk blockIdx.x: a scan of the counts, in runs of
  // consecutive sequences per thread.
  const Divisor by{unsigned(chunk)};
  const int run = (p.B + 127) / 128;
  const int b0 = tid * run, b1 = min(p.B, b0 + run);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += per_seq * by.up(max(lens[b], 1));
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) found[warp] = upto;
  if (tid == 0) found[8] = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += found[w];
  const int i = int(blockIdx.x);
  if (i >= upto - mine && i < upto) {
    int at = i - (upto - mine), b = b0, nv;
    for (;; ++b) {
      nv = by.up(max(lens[b], 1));
      if (at < per_seq * nv) break;
      at -= per_seq * nv;
    }
    found[9] = b;
    found[10] = at;
    found[11] = nv;
    found[8] = 0;
  }
  __syncthreads();
  if (found[8] < 0) return false;
  int at = found[10];
  it.b = found[9];
  it.nv = found[11];
  it.hc = at % p.head_chunks;
  at /= p.head_chunks;
  it.split = at % it.nv;
  it.kvh = at / it.nv;
  return true;
}

// For a cluster per unit: this CTA's item, one share of its sequence's n list rows for
// each CTA of the cluster, in whole 32-row steps and kBlockMinRows at least.
template <int ROWS, bool MOD>
__device__ __forceinline__ void cluster_chunk(const SplitParams& p, int n, ItemT<MOD>& it,
                                              int& chunk) {
  chunk = max(kBlockMinRows, (n + p.cluster - 1) / p.cluster);
  chunk = (chunk + ROWS - 1) / ROWS * ROWS;
  it.nv = max(1, (n + chunk - 1) / chunk);
}

// log2 x on the special-function unit, off by 2^-22 (0: -infinity).  Subnormals, which it
// takes for 0, are scaled first.
__device__ __forceinline__ float log2_of(float x) {
  const bool tiny = x < 1.17549435e-38f;
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(tiny ? x * 16777216.f : x));
  return tiny ? y - 24.f : y;
}

// 2^k for an integral k in [-126, 127].
__device__ __forceinline__ float pow2(float k) {
  return __uint_as_float(__float_as_uint(k + (12582912.f + 127.f)) << 23);
}

// Byte offset of 16-byte piece `piece` of row `row` of a box: the 128-byte
// swizzle for 128-byte rows, the 64-byte swizzle for 64-byte rows.
template <int D>
__device__ __forceinline__ int code_at(int row, int piece) {
  return D == 128 ? row * 128 + ((piece ^ (row & 7)) << 4)
                  : row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

// SHORT: P without its remainder and capped_short (short_forms, for bf16 outputs).
// CLUSTER: a cluster for each unit (p.cluster > 0; its code in the other kernel cost
// that one 0.8 %).
template <class Cfg, int TERMS, bool SHORT, bool CLUSTER>
__global__ void __launch_bounds__(Cfg::kThreads, Cfg::CTAS)
    split_decode_q8b_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const SplitParams p) {
  constexpr int D = Cfg::D, NB = Cfg::NB, KW = Cfg::KW, STAGES = Cfg::STAGES, ROWS = Cfg::ROWS;
  constexpr int kHPW = Cfg::kHPW;
  constexpr int MB = D / 16;        // 16-wide blocks of d (Step III m-blocks; Step I k-blocks)
  constexpr int KV4 = D / 16 / 4;   // 16-byte pieces a lane reads of a K row
  constexpr int VW = D / 32;        // 4-byte words a lane reads of a V row
  constexpr int KIND = Cfg::KIND;
  constexpr bool MOD = TERMS != 0, CAP = (TERMS & kTermsCap) != 0,
                 SLOPES = (TERMS & kTermsSlopes) != 0;
  // Weights, and their products with the V scales, are taken against 2^-kHead of their
  // maximum, so that those far below it keep their digits in fp16: its subnormals begin
  // 2^20 below the largest product, 2^14 without.
  constexpr float kHead = 7.f;
  constexpr float kLazy = 8.f;      // log2 of how far either may exceed 2^kHead

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* epi_acc = reinterpret_cast<float*>(smem);
  float* epi_m = epi_acc + Cfg::kEpiAccFloats;
  float* epi_l = epi_m + KW * kHPW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kDataBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + KW * STAGES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t full0 = smem_u32(bars) + 8 * STAGES * warp;
  const uint8_t* ring = smem + warp * (STAGES * Cfg::kStepBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < KW * STAGES; ++s) mbar_init(smem_u32(bars) + 8 * s, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // Launched as a programmatic dependent.  The CTAs of the first round, which may
  // start while the previous grid runs, find their chunk on the lengths as they
  // read before the wait (that grid may be writing them), and again if one has
  // changed after it; later ones have nothing to wait for.
  int* find = reinterpret_cast<int*>(bars + KW * STAGES) + 4;
  ItemT<MOD> it;
  int chunk = 0;
  bool any = false;
  const bool early = int(blockIdx.x) < p.places, few = !CLUSTER && p.B <= kFewSequences;
  bool bad = false, bad_pos = false;
  int n_out;
  int begin = 0;
  auto rows_of = [&](int b) {
    begin = MOD ? doc_begin(p.mod, b) : 0;
    return list_len<ROWS, MOD>(p, begin, __ldcg(p.seq_lens + b), bad, bad_pos, n_out);
  };
  int n_b = 0;
  if constexpr (CLUSTER) {  // the units and their CTAs in order
    const int unit = int(blockIdx.x) / p.cluster;
    it.split = int(blockIdx.x) - unit * p.cluster;
    it.hc = unit % p.head_chunks;
    it.kvh = unit / p.head_chunks % p.h_kv;
    it.b = unit / p.head_chunks / p.h_kv;
    any = it.b < p.B;
  }
  if (CLUSTER ? any : early) {
    if constexpr (CLUSTER) {
      n_b = rows_of(it.b);
      cluster_chunk<ROWS>(p, n_b, it, chunk);
    } else if (few) {
      if (lane < p.B) n_b = rows_of(lane);
      any = find_item_few<ROWS>(p, n_b, it, chunk);
    } else {
      for (int b = threadIdx.x; b < p.B; b += Cfg::kThreads) find[b] = rows_of(b);
      any = find_item_many<ROWS>(p, find, it, chunk);
    }
    // The chunk's first steps into L2 meanwhile: only a hint, so that it may go by
    // lengths that change yet, and by a cache that the previous grid still writes.
    // (GQA int8 32.2 -> 31.2 us, long fp8 86.9 -> 84.4; twice as many steps cost the
    // previous grid's last CTAs more than they bring: 33.0 and 83.7 us.)
    if (any) {
      int n = n_b;
      if constexpr (CLUSTER) {
      } else if (few) {
        n = __shfl_sync(0xffffffffu, n_b, it.b);
        n_out = __shfl_sync(0xffffffffu, n_out, it.b);
        begin = __shfl_sync(0xffffffffu, begin, it.b);
      } else {
        n = MOD ? rows_of(it.b) : find[it.b];
      }
      if constexpr (MOD) list_rows(p.mod, ROWS, begin, n_out, false, it.rows);
      if (lane == 0) {
        const int head = (p.b_offset + it.b) * p.h_kv + it.kvh;
        const int end = min(n, it.split * chunk + chunk);
        for (int i = 0; i < STAGES; ++i) {
          const int v = it.split * chunk + (i * KW + warp) * ROWS;
          if (v >= end) break;
          const int y = cache_row(it, v);
          tma_prefetch_3d(&tmK, 0, y, head);
          tma_prefetch_3d(&tmV, 0, y, head);
        }
      }
    }
  }
  bad = false;
  wait_for_prerequisite_grid();
  allow_dependent_launch();
  int n = 0;  // rows of the chunk's sequence
  n_out = 0;
  if constexpr (CLUSTER) {
    if (!any) return;
    n = rows_of(it.b);
    cluster_chunk<ROWS>(p, n, it, chunk);
  } else if (few) {
    const int before = n_b;
    if (lane < p.B) n_b = rows_of(lane);
    if (!early || __any_sync(0xffffffffu, n_b != before))
      any = find_item_few<ROWS>(p, n_b, it, chunk);
    n = __shfl_sync(0xffffffffu, n_b, any ? it.b : 0);
    n_out = __shfl_sync(0xffffffffu, n_out, any ? it.b : 0);
    begin = __shfl_sync(0xffffffffu, begin, any ? it.b : 0);
  } else {
    int changed = early ? 0 : 1;
    for (int b = threadIdx.x; b < p.B; b += Cfg::kThreads) {
      const int now = rows_of(b);
      changed |= now != find[b];
      find[b] = now;
    }
    if (__syncthreads_or(changed)) any = find_item_many<ROWS>(p, find, it, chunk);
    if (any) n = MOD ? rows_of(it.b) : find[it.b];
  }
  if (bad && (CLUSTER || blockIdx.x == 0)) flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.chunk_out) *p.chunk_out = chunk;
  if (!any) return;
  if constexpr (MOD) list_rows(p.mod, ROWS, begin, n_out, false, it.rows);
  it.row_begin = it.split * chunk;
  it.row_end = min(n, it.row_begin + chunk);
  it.new_row = -1;
  if (few || CLUSTER) __syncthreads();  // barriers initialised
  int steps = (it.row_end - it.row_begin + ROWS - 1) / ROWS;
  if (CLUSTER) steps = max(steps, 0);  // (its last CTAs may be past the rows)
  it.tiles = steps > warp ? (steps - warp + KW - 1) / KW : 0;  // this warp's
  // First list row of this warp's i-th step.
  auto step_row = [&](int i) { return it.row_begin + (i * KW + warp) * ROWS; };
  const int z = (p.b_offset + it.b) * p.h_kv + it.kvh;
  // Lane 0: load step i into a slot.
  const uint64_t policy = l2_policy_evict_first();
  auto load_step = [&](int i, int slot) {
    if (test_withhold(p, 0, i, it.tiles)) return;  // test builds only: never filled
    const uint32_t bar = full0 + 8 * slot, dst = smem_u32(ring) + slot * Cfg::kStepBytes;
    const int y = cache_row(it, step_row(i));
    mbar_arrive_expect_tx(bar, Cfg::kStepBytes);
    tma_load_3d(dst, &tmK, 0, y, z, bar, policy);
    tma_load_3d(dst + Cfg::kCodeBytes, &tmV, 0, y, z, bar, policy);
  };
  if (lane == 0)
    for (int i = 0; i < STAGES && i < it.tiles; ++i) load_step(i, i);

  const int g = lane >> 2;   // MMA fragment row group
  const int t = lane & 3;    // MMA fragment column pair
  const int head_base = it.hc * kHPW;
  // This warp's K and V scales of the two blocks of steps first .. first + 15
  // (lane 2 k + u: block u of step first + k), loaded a group ahead.
  auto load_scales = [&](int first, float& sk, float& sv) {
    const int v = step_row(first + (lane >> 1)) + (lane & 1) * 16;
    sk = sv = 0.f;
    if (v < it.row_end) {
      const int blk = cache_row(it, v) >> p.blk_shift;
      const size_t at = size_t(z) * size_t(p.nblk) + size_t(blk);
      if (DA_IN(p, blk, p.nblk) && DA_IN(p, at, p.scale_elems)) {
        sk = __ldcg(p.k_scale + at);
        sv = __ldcg(p.v_scale + at);
      }
    }
  };
  float sk_now = 0.f, sv_now = 0.f, sk_next, sv_next;
  load_scales(0, sk_next, sv_next);

  // q as B fragments in the permuted column order (heads past the group are
  // zero): lane (g, t) takes columns [t D/4, (t + 1) D/4) of head 8 nb + g.
  // (Ordinary loads: not through the read-only path, as the previous grid may still
  // write q when this one starts, but through L1, as all four warps want them; from L2
  // the long fp8 step takes 3 us more.)
  uint32_t qf[MB][NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int hl = head_base + nb * 8 + g;
    const size_t bhq = size_t(it.b) * p.h_q + size_t(it.kvh) * p.group + hl;
    const bool ok = hl < p.group && DA_IN(p, bhq, size_t(p.B) * p.h_q);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p.q) +
                                                      bhq * (D * 2) + t * (D / 2));
#pragma unroll
    for (int u = 0; u < MB / 2; ++u) {
      const uint4 w = ok ? src[u] : make_uint4(0, 0, 0, 0);
      qf[2 * u][nb][0] = w.x;
      qf[2 * u][nb][1] = w.y;
      qf[2 * u + 1][nb][0] = w.z;
      qf[2 * u + 1][nb][1] = w.w;
    }
  }
  // As fp16 times the power of two that brings the largest finite |q| of the CTA's heads
  // into [2^14, 2^15): exact down to 2^-31 of it, and no bf16 number is too large.
  auto q_most = [&](auto part) {  // the bits of the largest part(word), two halves a word
    uint32_t top = 0;
#pragma unroll
    for (int kb = 0; kb < MB; ++kb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        top = __vmaxu2(top, __vmaxu2(part(qf[kb][nb][0] & 0x7fff7fffu),
                                     part(qf[kb][nb][1] & 0x7fff7fffu)));
    return __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
  };
  uint32_t q_top = q_most([](uint32_t w) { return w; });
  if (q_top >= 0x7f80u)  // some are infinite or NaN, and stay so
    q_top = q_most([](uint32_t w) { return w & __vcmpltu2(w, 0x7f807f80u); });
  const float q_up = q_top == 0 ? 0.f : fminf(float(141 - int(q_top >> 7)), 126.f);
  const __nv_bfloat162 q_by = __float2bfloat162_rn(pow2(q_up));
#pragma unroll
  for (int kb = 0; kb < MB; ++kb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __nv_bfloat162 x =
            __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&qf[kb][nb][j]), q_by);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&x);
        qf[kb][nb][j] = q8::pack_f16x2(bf16_lo_to_f32(w), bf16_hi_to_f32(w));
      }
  [[maybe_unused]] float slope[NB][2];
  if constexpr (SLOPES) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int hl = head_base + nb * 8 + 2 * t + j;
        slope[nb][j] = head_slope(p, it.kvh * p.group + hl, hl < p.group);
      }
  }

  float m_run[NB][2], l_run[NB][2];
  float acc[MB][NB][4];
  // A head's accumulator counts in units of 2^-k_run beside the weights', which count
  // in 2^m_run: the largest product of a weight and a V scale so far is 2^kHead or
  // half of it (k_run is integral, and in [-126, 126]).
  float k_run[NB][2], k_top = 0.f;  // k_top: the largest of them
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m_run[nb][0] = m_run[nb][1] = -INFINITY;
    l_run[nb][0] = l_run[nb][1] = 0.f;
    k_run[nb][0] = k_run[nb][1] = 0.f;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mb][nb][e] = 0.f;
  }

  // (used once in 16 steps: kept in shared memory, not in a register of them all)
  volatile float* q_down = reinterpret_cast<volatile float*>(find + kFindWords - KW + warp);
  if (lane == 0) *q_down = pow2(-q_up);
  __syncwarp();
  [[maybe_unused]] bool slopes_up = true;
  if constexpr (SLOPES) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) slopes_up &= slope[nb][0] >= 0.f && slope[nb][1] >= 0.f;
    slopes_up = __all_sync(0xffffffffu, slopes_up);
  }
  int slot = 0;
  uint32_t phase = 0;
  for (int i = 0; i < it.tiles; ++i) {
    if ((i & 15) == 0) {
      // (a score's whole factor, finite, so that a product of zero stays zero)
      sk_now = sk_next * *q_down * (CAP && SHORT ? p.mod.short_scale : p.scale_log2);
      if (fabsf(sk_now) > 3e38f) sk_now = copysignf(3e38f, sk_now);
      sv_now = sv_next;
      load_scales(i + 16, sk_next, sv_next);
    }
    // warp-uniform (the MMAs and shuffles below need the whole warp)
    const bool ok = mbar_wait_bounded(full0 + 8 * slot, phase, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0 && !*abort_flag) flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
      *abort_flag = 1;
      // this warp's copies in flight (steps i .. i + STAGES - 1) land before the CTA can exit
      volatile int never = 0;
      for (int k = i; k < i + STAGES && k < it.tiles; ++k)
        if (!test_withhold(p, 0, k, it.tiles))
          mbar_wait_bounded(full0 + 8 * (k % STAGES), (k / STAGES) & 1, &never);
      break;
    }
    const uint8_t* ktile = ring + slot * Cfg::kStepBytes;
    const uint8_t* vtile = ktile + Cfg::kCodeBytes;
    const int v0 = step_row(i);
    const TileMask<MOD> mask(it, v0, min(ROWS, it.row_end - v0));
    // Every step holds a seen row (the list has only such tiles); its second
    // block may hold none, and then any scale.
    float ks[2], vs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ks[u] = __shfl_sync(0xffffffffu, sk_now, 2 * (i & 15) + u);
      vs[u] = __shfl_sync(0xffffffffu, sv_now, 2 * (i & 15) + u);
      const bool any = !MOD || mask.any_seen(u * 16, 16);
      ks[u] = any ? ks[u] : 0.f;
      vs[u] = any ? vs[u] : 0.f;
    }
    {
      // ---- Step I
      float s[2][NB][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nb][e] = 0.f;
        uint4 kA[KV4], kB[KV4];
#pragma unroll
        for (int w = 0; w < KV4; ++w) {
          kA[w] = *reinterpret_cast<const uint4*>(ktile + code_at<D>(u * 16 + g, t * KV4 + w));
          kB[w] = *reinterpret_cast<const uint4*>(ktile + code_at<D>(u * 16 + g + 8, t * KV4 + w));
        }
#pragma unroll
        for (int kb = 0; kb < MB; ++kb) {
          uint32_t a[4];
          q8::codes_to_f16<KIND>(word_of(kA[kb >> 2], kb & 3), a[0], a[2]);
          q8::codes_to_f16<KIND>(word_of(kB[kb >> 2], kb & 3), a[1], a[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            q8::mma_f16_16816(s[u][nb], a, qf[kb][nb][0], qf[kb][nb][1]);
        }
      }
      // ---- Step II: scale, terms, mask, running max and sum
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nb][e] *= ks[u];
      if constexpr (CAP) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[u][nb][e] = SHORT ? capped_short(p.mod, s[u][nb][e])
                                  : p.mod.cap_log2 * tanh_fast(s[u][nb][e]);
      }
      if constexpr (SLOPES) {
        const RowDistance dist(it, mask.row0 + g);
        if (slopes_up) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[u][nb][e] = biased(s[u][nb][e], RowDistance(dist, u * 16 + (e >> 1) * 8),
                                     slope[nb][e & 1], true);
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[u][nb][e] = biased(s[u][nb][e], RowDistance(dist, u * 16 + (e >> 1) * 8),
                                     slope[nb][e & 1], false);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool seenA = mask.seen(u * 16 + g), seenB = mask.seen(u * 16 + g + 8);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[u][nb][e] = (e < 2 ? seenA : seenB) ? s[u][nb][e] : -INFINITY;
      }
      // Both maxima are kept lazily: only where some score, by itself or with the step's
      // larger V scale, is more than 2^kLazy above its own does a vote bring the exact
      // ones (six shuffles a head) and the rescaling.  Every weight and sum is taken
      // against the maximum as it stands (m_run: kHead below it); products reach 2^15,
      // inside fp16's 65504.
      float lv[2];  // log2 of the blocks' V scales (the same on every lane)
#pragma unroll
      for (int u = 0; u < 2; ++u) lv[u] = log2_of(fabsf(vs[u]));
      const float lv_top = fmaxf(lv[0], lv[1]);
      // (a V scale that leaves float's range in units of the accumulator)
      bool over = lv_top + k_top > 126.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mx =
              fmaxf(fmaxf(s[0][nb][j], s[0][nb][j + 2]), fmaxf(s[1][nb][j], s[1][nb][j + 2]));
          over |= (mx - m_run[nb][j]) + fmaxf(k_run[nb][j] + lv_top, 0.f) > kHead + kLazy;
        }
      const bool update = __any_sync(0xffffffffu, over);
      if (update) {
        k_top = -126.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              mx[u] = fmaxf(s[u][nb][j], s[u][nb][j + 2]);
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 4));
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 8));
              mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 16));
            }
            const float m_old = m_run[nb][j], k_old = k_run[nb][j];
            const float m_new = fmaxf(m_old, fmaxf(mx[0], mx[1]) - kHead);
            const float m_use = m_new == -INFINITY ? 0.f : m_new;  // (nothing seen yet)
            // The accumulator's reference, 2^(m - k), only grows.  (Differences from m: a
            // large score's own float would swallow a scale's logarithm.)
            const float a =
                fmaxf(m_old - m_use - k_old,
                      fmaxf(mx[0] - m_use + lv[0], mx[1] - m_use + lv[1]) - kHead);
            const float k_new =
                m_new == -INFINITY ? 0.f : fminf(fmaxf(floorf(-a), -126.f), 126.f);
            const float alpha = ex2(m_old - m_use);
            const float f = alpha * pow2(fminf(fmaxf(k_new - k_old, -126.f), 127.f));
            m_run[nb][j] = m_new;
            k_run[nb][j] = k_new;
            k_top = fmaxf(k_top, k_new);
            l_run[nb][j] *= alpha;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              acc[mb][nb][j] *= f;
              acc[mb][nb][j + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float m_use = m_run[nb][j] == -INFINITY ? 0.f : m_run[nb][j];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            s[u][nb][j] = ex2(s[u][nb][j] - m_use);
            s[u][nb][j + 2] = ex2(s[u][nb][j + 2] - m_use);
            l_run[nb][j] += s[u][nb][j] + s[u][nb][j + 2];
          }
        }
      // times the V scale in units of the accumulator (a power of two times it: exact)
      if (update) {  // (in two parts: a scale may leave float's range where its weights are 0)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              s[u][nb][e] = s[u][nb][e] * 0x1p16f *
                            fminf(fmaxf(vs[u] * (pow2(k_run[nb][e & 1]) * 0x1p-16f), -0x1p127f),
                                  0x1p127f);
      } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < 2; ++u) s[u][nb][e] *= vs[u] * pow2(k_run[nb][e & 1]);
      }
      // ---- Step III: O^T += V^T . P^T
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t ph[NB][2];
        [[maybe_unused]] uint32_t pl[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float* x = s[u][nb];
          const uint32_t h0 = q8::pack_f16x2(x[0], x[1]);  // row g
          const uint32_t h1 = q8::pack_f16x2(x[2], x[3]);  // row g + 8
          ph[nb][0] = movmatrix_trans(h0);
          ph[nb][1] = movmatrix_trans(h1);
          if constexpr (!SHORT) {
            pl[nb][0] = movmatrix_trans(
                q8::pack_f16x2(x[0] - q8::f16_lo(h0), x[1] - q8::f16_hi(h0)));
            pl[nb][1] = movmatrix_trans(
                q8::pack_f16x2(x[2] - q8::f16_lo(h1), x[3] - q8::f16_hi(h1)));
          }
        }
        uint32_t v[4][VW];
        const int vr[4] = {u * 16 + 2 * t, u * 16 + 2 * t + 1, u * 16 + 2 * t + 8,
                           u * 16 + 2 * t + 9};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vtile + code_at<D>(vr[r], g));
            v[r][0] = w.x, v[r][1] = w.y, v[r][2] = w.z, v[r][3] = w.w;
          } else {
            const uint2 w =
                *reinterpret_cast<const uint2*>(vtile + code_at<D>(vr[r], g >> 1) + (g & 1) * 8);
            v[r][0] = w.x, v[r][1] = w.y;
          }
        }
        // rows past the end or not seen may hold anything: nothing of them reaches O
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool seen = mask.seen(vr[r]);
#pragma unroll
          for (int w = 0; w < VW; ++w) v[r][w] = seen ? v[r][w] : 0u;
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const uint32_t sel = (mb & 1) ? 0x7362u : 0x5140u;  // columns 2mb, 2mb+1 of the lane's
          const uint32_t x01 = __byte_perm(v[0][mb >> 1], v[1][mb >> 1], sel);
          const uint32_t x23 = __byte_perm(v[2][mb >> 1], v[3][mb >> 1], sel);
          uint32_t a[4];
          q8::codes_to_f16<KIND>(x01, a[0], a[1]);
          q8::codes_to_f16<KIND>(x23, a[2], a[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            q8::mma_f16_16816(acc[mb][nb], a, ph[nb][0], ph[nb][1]);
            if constexpr (!SHORT) q8::mma_f16_16816(acc[mb][nb], a, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }
    // every lane's reads of the slot have been used: it may be refilled
    __syncwarp();
    if (lane == 0 && i + STAGES < it.tiles) load_step(i + STAGES, slot);
    if (++slot == STAGES) {
      slot = 0;
      phase ^= 1u;
    }
  }

  // ---- the warps' states to shared slots (over the rings), then the shared finish
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x = l_run[nb][j];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      l_run[nb][j] = x;
    }
  __syncthreads();
  float* slots = epi_acc + warp * kHPW * Cfg::kSlotStride;
  if (lane < 4) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        epi_m[warp * kHPW + nb * 8 + 2 * lane + j] = m_run[nb][j];
        epi_l[warp * kHPW + nb * 8 + 2 * lane + j] = l_run[nb][j];
      }
  }
  float unit[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int j = 0; j < 2; ++j) unit[nb][j] = pow2(-k_run[nb][j]);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int d0 = (D / 8) * g + 2 * mb;  // acc[0..1]: column d0; acc[2..3]: d0 + 1
      const int h0 = nb * 8 + 2 * t;
      slots[h0 * Cfg::kSlotStride + d0] = acc[mb][nb][0] * unit[nb][0];
      slots[(h0 + 1) * Cfg::kSlotStride + d0] = acc[mb][nb][1] * unit[nb][1];
      slots[h0 * Cfg::kSlotStride + d0 + 1] = acc[mb][nb][2] * unit[nb][0];
      slots[(h0 + 1) * Cfg::kSlotStride + d0 + 1] = acc[mb][nb][3] * unit[nb][1];
    }
  __syncthreads();
  if (CLUSTER && p.cluster > 1)
    finish_cluster<D, 1, KW, kHPW, Cfg::kSlotStride>(p, it, epi_acc, epi_m, epi_l, threadIdx.x,
                                                  Cfg::kThreads, abort_flag);
  else
    finish_item<D, 1, KW, kHPW, Cfg::kSlotStride>(p, it, epi_acc, epi_m, epi_l, threadIdx.x,
                                                  Cfg::kThreads, abort_flag);
}

// ---------------------------------------------------------------------------
// Variants and launcher.  Groups of up to 8 query heads take one MMA block of
// heads, larger ones two (16 heads a CTA).
// ---------------------------------------------------------------------------
template <int KIND>
using Q8BD128N1 = Q8BCfg<128, 1, 2, 3, KIND>;
template <int KIND>
using Q8BD128N2 = Q8BCfg<128, 2, 2, 3, KIND>;
template <int KIND>
using Q8BD64N1 = Q8BCfg<64, 1, 3, 4, KIND>;
template <int KIND>
using Q8BD64N2 = Q8BCfg<64, 2, 4, 3, KIND>;

template <class Cfg, bool SHORT, bool CLUSTER>
static cudaError_t launch_q8b_form(const SplitParams& p, const CUtensorMap& tk,
                                   const CUtensorMap& tv, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  const auto kernel = split_decode_q8b_kernel<Cfg, DA_TERMS, SHORT, CLUSTER>;
  const cudaError_t e = set_smem_limit_once(kernel, Cfg::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent_clusters(kernel, grid, p.cluster, Cfg::kThreads, Cfg::kSmemBytes, stream,
                                   tk, tv, p);
}

template <class Cfg>
static cudaError_t launch_q8b_cfg(const SplitParams& p, const CUtensorMap& tk,
                                  const CUtensorMap& tv, int grid, cudaStream_t stream) {
  const bool brief = short_forms(p.out_bf16 != 0, p.mod);
  if (p.cluster > 0)
    return brief ? launch_q8b_form<Cfg, true, true>(p, tk, tv, grid, stream)
                 : launch_q8b_form<Cfg, false, true>(p, tk, tv, grid, stream);
  return brief ? launch_q8b_form<Cfg, true, false>(p, tk, tv, grid, stream)
               : launch_q8b_form<Cfg, false, false>(p, tk, tv, grid, stream);
}

template <int KIND>
static cudaError_t launch_q8b_kind(const SplitParams& p, const CUtensorMap& tk,
                                   const CUtensorMap& tv, int d, int grid, cudaStream_t stream) {
  if (d == 128)
    return p.group <= 8 ? launch_q8b_cfg<Q8BD128N1<KIND>>(p, tk, tv, grid, stream)
                        : launch_q8b_cfg<Q8BD128N2<KIND>>(p, tk, tv, grid, stream);
  return p.group <= 8 ? launch_q8b_cfg<Q8BD64N1<KIND>>(p, tk, tv, grid, stream)
                      : launch_q8b_cfg<Q8BD64N2<KIND>>(p, tk, tv, grid, stream);
}

// This object's set of terms (DA_TERMS); the dispatch is in the object of set 0.
template <int TERMS>
cudaError_t launch_q8b_set(const SplitParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                           int d, int kind, int grid, cudaStream_t stream);
DA_DECLARE_SETS(launch_q8b_set, (const SplitParams&, const CUtensorMap&, const CUtensorMap&, int, int, int, cudaStream_t))
template <>
cudaError_t launch_q8b_set<DA_TERMS>(const SplitParams& p, const CUtensorMap& tk,
                                     const CUtensorMap& tv, int d, int kind, int grid,
                                     cudaStream_t stream) {
  return kind == 1 ? launch_q8b_kind<1>(p, tk, tv, d, grid, stream)
                   : launch_q8b_kind<2>(p, tk, tv, d, grid, stream);
}

#if DA_TERMS == 0
KernelShape q8b_shape(int d, int group) {
  const bool one = group <= 8;
  const int ctas = d == 64 && one ? 4 : 3;
  return KernelShape{32, one ? 8 : 16, d, d == 128 ? 1 : 2, float(ctas)};
}

cudaError_t launch_split_q8b(const SplitParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                             int d, int kind, int grid, cudaStream_t stream) {
  return DA_LAUNCH_TERMS(launch_q8b_set, terms_of(p.mod), p, tk, tv, d, kind, grid, stream);
}
#endif

}  // namespace da
