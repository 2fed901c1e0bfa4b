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
// Layout.  The code tiles arrive by TMA (128 rows, a row's D bytes contiguous
// with the 128- or 64-byte swizzle) and MMA A fragments are built from them in
// registers; no fp16 copy of a stage is written.  Eight consumer warps own 16
// rows of a stage each; as S is a multiple of 16, a warp's rows of a stage
// have ONE K scale and ONE V scale.  So scales are not staged: a warp loads
// those of its next 32 stages with one load per tensor (a lane per stage), a
// group ahead, and takes each by a shuffle.  With lane = 4 g + t:
//   Step I  (S^T = K . Q^T, rows of K as M): lane (g, t) reads bytes
//           [t D/4, (t + 1) D/4) of rows g and g + 8 of the warp's block; k-block
//           kb takes the 4 codes at t D/4 + 4 kb as the A elements at logical
//           columns 2t, 2t+1, 2t+8, 2t+9.  That relabels the columns of d one to
//           one, and the q fragments are taken in the same order.
//   Step III (O^T += V^T . P^T, d as M): lane (g, t) reads bytes
//           [g D/8, (g + 1) D/8) of rows 2t, 2t+1, 2t+8, 2t+9; a byte permute
//           pairs a column's codes of two rows; m-block mb takes columns
//           g D/8 + 2 mb and + 1.
// The V scale multiplies P before P becomes fp16 (head + remainder, ~22 bits).
// Scales may be of any size (2^-126 for tiny rows), and fp16 has few exponents,
// so a warp keeps its accumulator in units of the largest V scale it has seen:
// P is multiplied by vs / unit <= 1, the accumulator is rescaled when the unit
// grows (as by a running maximum), and the unit returns at the item's end.
#include <math.h>

#include "common.cuh"
#include "q8_codes.cuh"

namespace da {

template <int D_, int NB_, int STAGES_, int KIND_>
struct Q8BCfg {
  static constexpr int D = D_;
  static constexpr int NB = NB_;           // 8-head MMA blocks per item
  static constexpr int KW = 8;             // consumer warps, one 16-row block each
  static constexpr int STAGES = STAGES_;
  static constexpr int KIND = KIND_;       // 1: int8 codes, 2: fp8 e4m3 codes
  static constexpr int kHPW = 8 * NB;
  static constexpr int kTile = 16 * KW;
  static constexpr int kConsumerThreads = 32 * KW;
  static constexpr int kThreads = kConsumerThreads + 32;
  static constexpr int kCodeBytes = kTile * D;
  static constexpr int kStageBytes = 2 * kCodeBytes;
  static constexpr int kQBytes = kHPW * D * 2;
  static constexpr int kSlotStride = D + 4;
  static constexpr int kEpiAccFloats = KW * kHPW * kSlotStride;
  static constexpr int kEpiMLFloats = 2 * KW * kHPW;
  static constexpr int kSchedWords = da::kSchedWords;
  static constexpr size_t kSmemBytes = 1024 + size_t(STAGES) * (kStageBytes + kQBytes) +
                                       size_t(kEpiAccFloats + kEpiMLFloats + kSchedWords) * 4 +
                                       2 * STAGES * 8 + 16;
  static_assert(D == 64 || D == 128, "head dim");
  static_assert(KIND == 1 || KIND == 2, "code type");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert((kEpiAccFloats + kEpiMLFloats) % 2 == 0, "mbarrier alignment");
};

// Byte offset of 16-byte piece `piece` of row `row` of a code tile: the 128-byte
// swizzle for 128-byte rows, the 64-byte swizzle for 64-byte rows.
template <int D>
__device__ __forceinline__ int code_at(int row, int piece) {
  return D == 128 ? row * 128 + ((piece ^ (row & 7)) << 4)
                  : row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

// Producer: one thread streams the K and V code tiles of every stage of the
// CTA's items, and each item's bf16 q rows with its first stage.
template <class Cfg, bool MOD>
__device__ __forceinline__ void produce_q8b(const CUtensorMap* tmK, const CUtensorMap* tmV,
                                            const SplitParams& p, const Schedule& s, uint32_t ring,
                                            uint32_t qslots, uint32_t full0, uint32_t empty0,
                                            volatile int* abort_flag) {
  constexpr int T = Cfg::kTile, STAGES = Cfg::STAGES, D = Cfg::D;
  const uint64_t policy = l2_policy_evict_first();
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_parity = 0;
  bool aborted = false;
  for (int k = 0; k < s.mine && !aborted; ++k) {
    const ItemT<MOD> it = cta_item<T, MOD>(p, s, k);
    const int z = (p.b_offset + it.b) * p.h_kv + it.kvh;
    for (int t = 0; t < it.tiles; ++t) {
      if (!mbar_wait_bounded(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
        *abort_flag = 1;
        flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
        aborted = true;
        break;
      }
      if (test_withhold(p, k, t, it.tiles)) {  // test builds only: never filled
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        continue;
      }
      const uint32_t bar = full0 + 8 * stage;
      const int h0 = it.hc * Cfg::kHPW;
      const int nh = min(Cfg::kHPW, p.group - h0);
      const size_t bhq = size_t(it.b) * p.h_q + size_t(it.kvh) * p.group + h0;
      const bool load_q = t == 0 && DA_IN(p, bhq + nh - 1, size_t(p.B) * p.h_q);
      mbar_arrive_expect_tx(bar, Cfg::kStageBytes + (load_q ? uint32_t(nh) * (D * 2) : 0u));
      if (load_q)
        bulk_load(qslots + stage * Cfg::kQBytes, static_cast<const char*>(p.q) + bhq * (D * 2),
                  uint32_t(nh) * (D * 2), bar);
      const uint32_t dst = ring + stage * Cfg::kStageBytes;
      const int y = cache_row(it, it.row_begin + t * T);
      tma_load_3d(dst, tmK, 0, y, z, bar, policy);
      tma_load_3d(dst + Cfg::kCodeBytes, tmV, 0, y, z, bar, policy);
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (aborted) {  // every copy this thread started lands before the CTA can exit
    volatile int never = 0;
    for (int st = 0; st < STAGES; ++st)
      if (issued & (1u << st)) mbar_wait_bounded(full0 + 8 * st, (issued_parity >> st) & 1u, &never);
  }
}

template <class Cfg, bool MOD>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    split_decode_q8b_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const SplitParams p) {
  constexpr int D = Cfg::D, NB = Cfg::NB, KW = Cfg::KW, STAGES = Cfg::STAGES, T = Cfg::kTile;
  constexpr int kHPW = Cfg::kHPW;
  constexpr int MB = D / 16;        // 16-wide blocks of d (Step III m-blocks; Step I k-blocks)
  constexpr int KV4 = D / 16 / 4;   // 16-byte pieces a lane reads of a K row
  constexpr int VW = D / 32;        // 4-byte words a lane reads of a V row
  constexpr int KIND = Cfg::KIND;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qslots = smem + size_t(STAGES) * Cfg::kStageBytes;
  float* epi_acc = reinterpret_cast<float*>(qslots + size_t(STAGES) * Cfg::kQBytes);
  float* epi_m = epi_acc + Cfg::kEpiAccFloats;
  float* epi_l = epi_m + KW * kHPW;
  int* sched_words = reinterpret_cast<int*>(epi_l + KW * kHPW);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sched_words + Cfg::kSchedWords);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * STAGES);
  const uint32_t ring = smem_u32(smem);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * STAGES;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, KW);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {  // the tensor maps do not depend on the preceding grid
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x == Cfg::kConsumerThreads)  // producer lane: L2 prefetch of the hinted tiles
    prefetch_hinted<T, 1, 1, D>(p, load_hint(p), &tmK, &tmV, STAGES);
  // Launched as a programmatic dependent: before the wait only the hinted L2
  // prefetch and the work list touch what the previous grid may write (the
  // list is checked, and built again if a length changed, after the wait).
  Schedule sched = build_schedule_core<T, MOD>(p, sched_words);
  wait_for_prerequisite_grid();
  sched = commit_schedule<T, MOD>(p, sched_words, sched);
  allow_dependent_launch();
  if (threadIdx.x == 0 && sched.mine > 0)
    write_hint<T, MOD>(p, cta_item<T, MOD>(p, sched, 0), STAGES);

  // ------------------------------------------------------------------ producer
  if (warp == KW) {
    if (lane == 0)
      produce_q8b<Cfg, MOD>(&tmK, &tmV, p, sched, ring, smem_u32(qslots), full0, empty0,
                            abort_flag);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2;   // MMA fragment row group
  const int t = lane & 3;    // MMA fragment column pair
  const int key0 = warp * 16;  // first row of this warp's block inside a stage
  const int rA = key0 + g, rB = rA + 8;             // Step I rows (and P rows)
  const int r0 = key0 + 2 * t, r1 = r0 + 1, r2 = r0 + 8, r3 = r0 + 9;  // Step III rows
  int stage = 0;
  uint32_t phase = 0;

  for (int k = 0; k < sched.mine; ++k) {
    const ItemT<MOD> it = cta_item<T, MOD>(p, sched, k);
    const int head_base = it.hc * kHPW;
    const size_t kvhead = size_t(p.b_offset + it.b) * p.h_kv + it.kvh;
    // This warp's K and V scales of stages 32 i + lane, loaded a group ahead.
    auto load_scales = [&](int first, float& sk, float& sv) {
      const int v = it.row_begin + (first + lane) * T + key0;
      sk = sv = 0.f;
      if (v < it.row_end) {
        const int blk = cache_row(it, v) >> p.blk_shift;
        const size_t at = kvhead * size_t(p.nblk) + size_t(blk);
        if (DA_IN(p, blk, p.nblk) && DA_IN(p, at, p.scale_elems)) {
          sk = __ldcg(p.k_scale + at);
          sv = __ldcg(p.v_scale + at);
        }
      }
    };
    float sk_now, sv_now, sk_next, sv_next;
    load_scales(0, sk_next, sv_next);
    sk_now = sk_next, sv_now = sv_next;

    [[maybe_unused]] float slope[NB][2];
    if constexpr (MOD) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int hl = head_base + nb * 8 + 2 * t + j;
          slope[nb][j] = head_slope(p, it.kvh * p.group + hl, hl < p.group);
        }
    }
    uint32_t qf[MB][NB][2];  // B fragments of q, in the permuted column order
    float m_run[NB][2], l_run[NB][2];
    float acc[MB][NB][4];
    float unit = 0.f;        // the accumulator's unit: the largest |V scale| so far
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m_run[nb][0] = m_run[nb][1] = -INFINITY;
      l_run[nb][0] = l_run[nb][1] = 0.f;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mb][nb][e] = 0.f;
    }

    for (int tt = 0; tt < it.tiles; ++tt) {
      if ((tt & 31) == 0) {
        sk_now = sk_next, sv_now = sv_next;
        load_scales(tt + 32, sk_next, sv_next);
      }
      if (!mbar_wait_bounded(full0 + 8 * stage, phase, abort_flag)) {
        if (!*abort_flag) {
          *abort_flag = 1;
          flag_error(p.dev_error, DA_DEVERR_TIMEOUT);
        }
      }
      const uint8_t* ktile = smem + size_t(stage) * Cfg::kStageBytes;
      const uint8_t* vtile = ktile + Cfg::kCodeBytes;
      const int tile_row0 = it.row_begin + tt * T;
      const int valid = min(T, it.row_end - tile_row0);
      const TileMask<MOD> mask(it, tile_row0, valid);

      // ---- this lane's codes, into registers
      uint4 kA[KV4], kB[KV4];
      uint32_t v[4][VW];
#pragma unroll
      for (int u = 0; u < KV4; ++u) {
        kA[u] = *reinterpret_cast<const uint4*>(ktile + code_at<D>(rA, t * KV4 + u));
        kB[u] = *reinterpret_cast<const uint4*>(ktile + code_at<D>(rB, t * KV4 + u));
      }
      const int vr[4] = {r0, r1, r2, r3};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(vtile + code_at<D>(vr[u], g));
          v[u][0] = w.x, v[u][1] = w.y, v[u][2] = w.z, v[u][3] = w.w;
        } else {
          const uint2 w =
              *reinterpret_cast<const uint2*>(vtile + code_at<D>(vr[u], g >> 1) + (g & 1) * 8);
          v[u][0] = w.x, v[u][1] = w.y;
        }
        // rows past the end or not seen may hold anything: their values must not reach O
        if (!mask.seen(vr[u])) {
#pragma unroll
          for (int w = 0; w < VW; ++w) v[u][w] = 0;
        }
      }
      if (tt == 0) {  // q of head 8 nb + g (rows past the group are zero), bf16 -> fp16
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const bool ok = head_base + nb * 8 + g < p.group;
          const uint8_t* qs = qslots + size_t(stage) * Cfg::kQBytes + (nb * 8 + g) * (D * 2) +
                              t * (D / 2);
#pragma unroll
          for (int kb = 0; kb < MB; ++kb) {
            uint2 w = *reinterpret_cast<const uint2*>(qs + kb * 8);
            if (!ok) w = make_uint2(0, 0);
            qf[kb][nb][0] = q8::pack_f16x2(bf16_lo_to_f32(w.x), bf16_hi_to_f32(w.x));
            qf[kb][nb][1] = q8::pack_f16x2(bf16_lo_to_f32(w.y), bf16_hi_to_f32(w.y));
          }
        }
      }
      const float ks = __shfl_sync(0xffffffffu, sk_now, tt & 31) * p.scale_log2;
      const float vs = __shfl_sync(0xffffffffu, sv_now, tt & 31);
      __syncwarp();
      // every byte this warp needs from the stage is in registers now
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }

      // warp-uniform (the MMAs and shuffles below need the whole warp)
      const bool live = __all_sync(0xffffffffu, !*abort_flag);
      if (live && mask.any_seen(key0, 16)) {
        // ---- Step I
        float s[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
        float s2[4] = {0.f, 0.f, 0.f, 0.f};  // one head block: two independent chains
#pragma unroll
        for (int kb = 0; kb < MB; ++kb) {
          uint32_t a[4];
          q8::codes_to_f16<KIND>(word_of(kA[kb >> 2], kb & 3), a[0], a[2]);
          q8::codes_to_f16<KIND>(word_of(kB[kb >> 2], kb & 3), a[1], a[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if (NB == 1 && (kb & 1)) q8::mma_f16_16816(s2, a, qf[kb][nb][0], qf[kb][nb][1]);
            else q8::mma_f16_16816(s[nb], a, qf[kb][nb][0], qf[kb][nb][1]);
          }
        }
        if (NB == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] += s2[e];
        }
        // ---- Step II: scale, terms, mask, running max and sum
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][e] *= ks;
        if constexpr (MOD) {  // one branch for all of a lane's scores
          if (p.mod.cap_log2 > 0.f) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[nb][e] = p.mod.cap_log2 * tanh_fast(s[nb][e]);
          }
          if (p.mod.slopes) {
            const RowDistance dist(it, mask.row0 + rA);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[nb][e] = biased(s[nb][e], RowDistance(dist, (e >> 1) * 8), slope[nb][e & 1]);
          }
        }
        const bool seenA = mask.seen(rA), seenB = mask.seen(rB);
        float alpha[NB][2];
        bool changed = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float xA = seenA ? s[nb][j] : -INFINITY;
            const float xB = seenB ? s[nb][j + 2] : -INFINITY;
            float mx = fmaxf(xA, xB);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(m_run[nb][j], mx);
            const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
            alpha[nb][j] = ex2(m_run[nb][j] - m_use);
            changed |= (m_new != m_run[nb][j]);
            m_run[nb][j] = m_new;
            s[nb][j] = ex2(xA - m_use);
            s[nb][j + 2] = ex2(xB - m_use);
            l_run[nb][j] = l_run[nb][j] * alpha[nb][j] + (s[nb][j] + s[nb][j + 2]);
          }
        // the V scale in units of the accumulator (the same on every lane)
        float w = 1.f;
        const float avs = fabsf(vs);
        if (avs > unit) {
          const float f = __fdiv_rn(unit, avs);
          unit = avs;
          changed = true;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) alpha[nb][0] *= f, alpha[nb][1] *= f;
        }
        if (vs != unit) w = unit > 0.f ? __fdiv_rn(vs, unit) : 0.f;
        if (__any_sync(0xffffffffu, changed)) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              acc[mb][nb][0] *= alpha[nb][0];
              acc[mb][nb][1] *= alpha[nb][1];
              acc[mb][nb][2] *= alpha[nb][0];
              acc[mb][nb][3] *= alpha[nb][1];
            }
        }
        // ---- Step III: O^T += V^T . (P * w)^T, P as fp16 head + fp16 remainder
        uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float p0 = s[nb][0] * w, p1 = s[nb][1] * w, p2 = s[nb][2] * w, p3 = s[nb][3] * w;
          const uint32_t h0 = q8::pack_f16x2(p0, p1);  // row g
          const uint32_t h1 = q8::pack_f16x2(p2, p3);  // row g + 8
          const uint32_t l0 = q8::pack_f16x2(p0 - q8::f16_lo(h0), p1 - q8::f16_hi(h0));
          const uint32_t l1 = q8::pack_f16x2(p2 - q8::f16_lo(h1), p3 - q8::f16_hi(h1));
          ph[nb][0] = movmatrix_trans(h0);
          ph[nb][1] = movmatrix_trans(h1);
          pl[nb][0] = movmatrix_trans(l0);
          pl[nb][1] = movmatrix_trans(l1);
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
            q8::mma_f16_16816(acc[mb][nb], a, pl[nb][0], pl[nb][1]);
          }
        }
      }
    }

    // ---- Epilogue: per-warp state to shared slots, then the shared finish.
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
    named_bar_sync(1, Cfg::kConsumerThreads);  // earlier readers of the slots are done
    float* slot = epi_acc + warp * kHPW * Cfg::kSlotStride;
    if (lane < 4) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          epi_m[warp * kHPW + nb * 8 + 2 * lane + j] = m_run[nb][j];
          epi_l[warp * kHPW + nb * 8 + 2 * lane + j] = l_run[nb][j];
        }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int d0 = (D / 8) * g + 2 * mb;  // acc[0..1]: column d0; acc[2..3]: d0 + 1
        const int h0 = nb * 8 + 2 * t;
        slot[h0 * Cfg::kSlotStride + d0] = acc[mb][nb][0] * unit;
        slot[(h0 + 1) * Cfg::kSlotStride + d0] = acc[mb][nb][1] * unit;
        slot[h0 * Cfg::kSlotStride + d0 + 1] = acc[mb][nb][2] * unit;
        slot[(h0 + 1) * Cfg::kSlotStride + d0 + 1] = acc[mb][nb][3] * unit;
      }
    named_bar_sync(1, Cfg::kConsumerThreads);
    finish_item<D, 1, KW, kHPW, Cfg::kSlotStride>(p, it, epi_acc, epi_m, epi_l, threadIdx.x,
                                                  Cfg::kConsumerThreads, abort_flag);
  }
}

// ---------------------------------------------------------------------------
// Variants and launcher.  Groups of up to 8 query heads take one MMA block of
// heads, larger ones two (16 heads an item), so that a group of 32 reads the
// cache twice, not four times.
// ---------------------------------------------------------------------------
template <int KIND>
using Q8BD128N1 = Q8BCfg<128, 1, 5, KIND>;
template <int KIND>
using Q8BD128N2 = Q8BCfg<128, 2, 4, KIND>;
template <int KIND>
using Q8BD64N1 = Q8BCfg<64, 1, 9, KIND>;
template <int KIND>
using Q8BD64N2 = Q8BCfg<64, 2, 8, KIND>;

KernelShape q8b_shape(int d, int group) {
  const int heads = group <= 8 ? 8 : 16;
  return KernelShape{128, heads, d, d == 128 ? 1 : 2, 1.0f};
}

template <class Cfg, bool MOD>
static cudaError_t launch_q8b_mod(const SplitParams& p, const CUtensorMap& tk,
                                  const CUtensorMap& tv, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e =
      set_smem_limit_once(split_decode_q8b_kernel<Cfg, MOD>, Cfg::kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_dependent(split_decode_q8b_kernel<Cfg, MOD>, grid, Cfg::kThreads,
                          Cfg::kSmemBytes, stream, tk, tv, p);
}

template <class Cfg>
static cudaError_t launch_q8b_cfg(const SplitParams& p, const CUtensorMap& tk,
                                  const CUtensorMap& tv, int grid, cudaStream_t stream) {
  return p.mod.on ? launch_q8b_mod<Cfg, true>(p, tk, tv, grid, stream)
                  : launch_q8b_mod<Cfg, false>(p, tk, tv, grid, stream);
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

cudaError_t launch_split_q8b(const SplitParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                             int d, int kind, int grid, cudaStream_t stream) {
  return kind == 1 ? launch_q8b_kind<1>(p, tk, tv, d, grid, stream)
                   : launch_q8b_kind<2>(p, tk, tv, d, grid, stream);
}

}  // namespace da
