// Writing rows into an 8-bit cache with a scale per block of tokens and head,
// and reading rows back as values (sm_103a).
//
// Write.  New rows x go behind the pos rows a sequence holds.  A block of S
// tokens keeps one scale s; with Q the largest code value (127 or 448):
//   need = 2^ceil(log2(max|x| / Q)) over the block's new rows (0 if all are
//          zero, at least 2^-126), s' = max(s, need)  (s = 0 for a block that
//          begins in this call);
//   new rows: code = rne(x / s');
//   rows the block already holds, when s' > s: code' = rne(code * (s / s')).
// Scales that grow are powers of two: x / s' and s / s' are then exact, so a
// code is rounded once, the result does not depend on the order of operations,
// and for e4m3 codes rewriting the held rows loses nothing above the
// subnormals.  It costs int8 half a bit on average against max|x| / Q.
//
// Bound: HBM for prompts (x once in, codes once out; a block's rows wait in
// registers for its maximum), latency for single tokens: positions, then x and
// the scale at once, then the stores (3.3 us for 16 sequences of 8 kv heads).  A
// warp owns 16 rows of a block, S / 16 warps a block, 128 / S blocks a CTA; a lane
// takes 16 bytes of x at a time, so that a warp's loads and its stores of codes
// are whole runs of consecutive bytes, and the CTAs are persistent and read the
// next block's position while they work on this one.  What held it back was
// instructions: with the tests of a row and of the scale inside the loop over
// elements it took 23 an element, 340 us for 16 prompts of 8192 fp32 rows; with
// one test a block 5, and 204 us, 6.58 TB/s.
#include <math.h>

#include "common.cuh"
#include "q8_codes.cuh"

namespace da {

// The smallest power of two s >= 2^-126 with a <= Q s; 0 for a = 0 (a finite).
template <int KIND>
__device__ __forceinline__ float block_scale(float a) {
  if (a == 0.f) return 0.f;
  // Q = 127 = 1.984375 * 2^6 (int8), 448 = 1.75 * 2^8 (e4m3)
  constexpr uint32_t kFrac = KIND == 1 ? 0x7e0000u : 0x600000u;
  constexpr int kExp = KIND == 1 ? 6 : 8;
  const uint32_t bits = __float_as_uint(a);
  const int e = int(bits >> 23) - kExp + ((bits & 0x7fffffu) > kFrac ? 1 : 0);
  return __uint_as_float(uint32_t(max(e, 1)) << 23);
}

// Four values times `by` (exact) as codes; the products lie in [-Q, Q].
template <int KIND>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d, float by) {
  if constexpr (KIND == 1) {
    // rounded to an integer by an addition at 1.5 * 2^23: its low byte is the code
    constexpr float kMagic = 12582912.f;
    const uint32_t ab = __byte_perm(__float_as_uint(fmaf(a, by, kMagic)),
                                    __float_as_uint(fmaf(b, by, kMagic)), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(fmaf(c, by, kMagic)),
                                    __float_as_uint(fmaf(d, by, kMagic)), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  } else {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a * by), "f"(b * by), "f"(c * by), "f"(d * by));
    return r;
  }
}

template <int KIND>
__device__ __forceinline__ float clamp_code(float x) {
  constexpr float Q = KIND == 1 ? 127.f : 448.f;
  return fminf(fmaxf(x, -Q), Q);
}

// Four codes as values.
template <int KIND>
__device__ __forceinline__ void from_codes(uint32_t w, float (&v)[4]) {
  uint32_t lo, hi;
  q8::codes_to_f16<KIND>(w, lo, hi);
  v[0] = q8::f16_lo(lo), v[1] = q8::f16_hi(lo);
  v[2] = q8::f16_lo(hi), v[3] = q8::f16_hi(hi);
}

struct BlockWrite {
  const void* x[2];          // K rows, V rows: element (b, h, i, j) at b sb + h sh + i st + j
  long long sb[2], sh[2], st[2];
  uint8_t* codes[2];         // [B, h_kv, n_max, D]
  float* scale[2];           // [B, h_kv, nblk]
  const int32_t* pos;        // [B]
  const int32_t* n_new;      // nullable: [B], rows of the call that sequence b takes (else T)
  int32_t* dev_error;
  int B, h_kv, T, n_max, nblk, blk_shift, touched;
  unsigned units;            // 2 * B * h_kv * touched
  long long cache_rows, scale_elems;  // extents, for the checked build
};

constexpr int kWriteThreads = 256;
// CTAs an SM, by the registers that a warp's 16 rows take.
template <int D, bool XBF16>
constexpr int write_ctas() { return D == 128 && !XBF16 ? 2 : D == 64 && XBF16 ? 5 : 3; }

// Element e of the 16 bytes of x that a lane holds.
template <bool XBF16>
__device__ __forceinline__ float x_elem(const uint4& w, int e) {
  if constexpr (XBF16) {
    const uint32_t v = word_of(w, e >> 1);
    return (e & 1) ? bf16_hi_to_f32(v) : bf16_lo_to_f32(v);
  } else {
    return __uint_as_float(word_of(w, e));
  }
}

template <int D, bool XBF16, int KIND>
__global__ void __launch_bounds__(kWriteThreads, write_ctas<D, XBF16>())
    kv_append_q8b_kernel(const BlockWrite p) {
  constexpr int EPL = XBF16 ? 8 : 4;  // elements of 16 bytes
  constexpr int LPR = D / EPL;        // lanes per row
  constexpr int RPP = 32 / LPR;       // rows a warp covers at once
  constexpr int PASS = 16 / RPP;      // passes over its 16 rows
  constexpr int kWarps = kWriteThreads / 32;
  __shared__ float red[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = 1 << p.blk_shift, W = S >> 4;  // rows of a block, warps of a block
  const unsigned per_cta = unsigned(kWarps / W);
  const int sub = warp % W;
  const int rl = lane / LPR, c = lane % LPR;
  allow_dependent_launch();
  wait_for_prerequisite_grid();

  // The raw position and count of a unit's sequence.
  auto load_counts = [&](unsigned unit, int& pos, int& m) {
    pos = 0, m = 0;
    if (unit >= p.units) return;
    const int b = int((unit >> 1) / unsigned(p.touched)) / p.h_kv;
    pos = __ldcg(p.pos + b);
    m = p.n_new ? __ldcg(p.n_new + b) : p.T;
  };
  int pos_next, m_next;
  load_counts(blockIdx.x * per_cta + warp / W, pos_next, m_next);
  int turn = 0;
  for (unsigned base = blockIdx.x * per_cta; base < p.units; base += gridDim.x * per_cta) {
    // unit -> (head, touched block, tensor); a unit past the end only takes part in the barrier
    const unsigned unit = base + unsigned(warp / W);
    const bool live_unit = unit < p.units;
    const int tensor = int(unit & 1u);
    const int j = live_unit ? int((unit >> 1) % unsigned(p.touched)) : 0;
    const int head = live_unit ? int((unit >> 1) / unsigned(p.touched)) : 0;  // b * h_kv + h
    const int b = head / p.h_kv, h = head - b * p.h_kv;
    const int pos = pos_next;
    int m = m_next;
    load_counts(unit + gridDim.x * per_cta, pos_next, m_next);
    bool bad = m < 0 || m > p.T;
    m = min(max(m, 0), p.T);
    if (pos < 0 || pos > p.n_max) {
      bad |= m > 0;
      m = 0;
    } else if (m > p.n_max - pos) {
      bad = true;
      m = p.n_max - pos;
    }
    if (bad && live_unit && j == 0 && tensor == 0 && h == 0 && sub == 0 && lane == 0)
      flag_error(p.dev_error, DA_DEVERR_POS);
    const int blk = (pos >> p.blk_shift) + j;
    const int row0 = int((unsigned(blk) << p.blk_shift) + unsigned(sub) * 16u);  // this warp's first cache row
    const unsigned start = unsigned(blk) << p.blk_shift;  // (past 2^31 for the last block of 2^30 rows)
    const bool work = live_unit && m > 0 && start < unsigned(pos + m);
    const bool held = work && start < unsigned(pos);  // the block holds earlier rows

    // ---- loads: new rows and the block's scale
    const size_t scale_at = size_t(head) * p.nblk + blk;
    uint4 x[PASS];
    const char* xs = static_cast<const char*>(tensor ? p.x[1] : p.x[0]);
    uint8_t* codes = tensor ? p.codes[1] : p.codes[0];
    float* scale = tensor ? p.scale[1] : p.scale[0];
    const long long sb = tensor ? p.sb[1] : p.sb[0], sh = tensor ? p.sh[1] : p.sh[0],
                    st = tensor ? p.st[1] : p.st[0];
    const bool scale_in = !work || DA_IN(p, scale_at, p.scale_elems);
    float s_old = 0.f;
    if (held && scale_in) s_old = __ldcg(scale + scale_at);
    float a = 0.f;
    if (work) {
      xs += ((long long)b * sb + (long long)h * sh + c * EPL) * (16 / EPL);
#pragma unroll
      for (int u = 0; u < PASS; ++u) {
        const int i = row0 + u * RPP + rl - pos;
        x[u] = i >= 0 && i < m
                   ? __ldcs(reinterpret_cast<const uint4*>(xs + (long long)i * st * (16 / EPL)))
                   : make_uint4(0, 0, 0, 0);
      }
      // the largest magnitude, as bits without their sign
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < PASS; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = word_of(x[u], e);
          top = XBF16 ? __vmaxu2(top, w & 0x7fff7fffu) : max(top, w & 0x7fffffffu);
        }
      if (XBF16) top = max(top & 0xffff0000u, top << 16);
      if (top >= 0x7f800000u) {  // NaN or infinity among them: they count as 0
        flag_error(p.dev_error, DA_DEVERR_VALUE);
        top = 0;
#pragma unroll
        for (int u = 0; u < PASS; ++u) {
          uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (XBF16) {
              if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
              if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
              top = max(top, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fffffffu));
            } else {
              if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] = 0;
              top = max(top, w[e] & 0x7fffffffu);
            }
          }
          x[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      a = __uint_as_float(top);
    }

    // ---- the block's maximum and scale
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (W > 1) {
      // (two scratch rows: a warp reaches this one's next use only past the
      // barrier of the turn between)
      if (lane == 0) red[turn][warp] = a;
      __syncthreads();
      const int w0 = warp - sub;
      for (int w = 0; w < W; ++w) a = fmaxf(a, red[turn][w0 + w]);
      turn ^= 1;
    }
    if (!work) continue;
    const float s_new = fmaxf(s_old, block_scale<KIND>(a));
    if (sub == 0 && lane == 0 && scale_in) scale[scale_at] = s_new;

    // ---- codes
    // a power of two divides exactly by its inverse (2^-126 .. 2^125 have a normal one)
    const uint32_t sbits = __float_as_uint(s_new);
    const bool pow2 = (sbits & 0x807fffffu) == 0 && sbits != 0 && (sbits >> 23) < 253;
    const float inv = pow2 ? __uint_as_float((254u << 23) - sbits) : 0.f;
    uint8_t* dst0 = codes + (size_t(head) * p.n_max + row0 + rl) * D + c * EPL;
    auto put = [&](int u, const float (&f)[EPL], float by) {
      uint8_t* dst = dst0 + u * (RPP * D);
      const uint32_t w0 = to_codes<KIND>(f[0], f[1], f[2], f[3], by);
      if constexpr (XBF16)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(w0, to_codes<KIND>(f[4], f[5], f[6], f[7], by));
      else
        *reinterpret_cast<uint32_t*>(dst) = w0;
    };
    // (a block written in whole has no row to test)
    const bool whole = row0 >= pos && row0 + 16 <= pos + m;
    if (pow2 || s_new == 0.f) {  // (0: every element is 0)
#pragma unroll
      for (int u = 0; u < PASS; ++u) {
        const int row = row0 + u * RPP + rl;
        if (!whole && (row < pos || row >= pos + m)) continue;
        if (!DA_IN(p, size_t(head) * p.n_max + row, p.cache_rows)) continue;
        float f[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) f[e] = x_elem<XBF16>(x[u], e);
        put(u, f, inv);
      }
    } else {  // a scale from elsewhere: a rounded division and a clamp
#pragma unroll 1
      for (int u = 0; u < PASS; ++u) {
        const int row = row0 + u * RPP + rl;
        uint4 xu = x[0];
#pragma unroll
        for (int k = 1; k < PASS; ++k)
          if (k == u) xu = x[k];
        if (row < pos || row >= pos + m ||
            !DA_IN(p, size_t(head) * p.n_max + row, p.cache_rows))
          continue;
        float f[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e)
          f[e] = clamp_code<KIND>(__fdiv_rn(x_elem<XBF16>(xu, e), s_new));
        put(u, f, 1.f);
      }
    }
    // ---- a scale that grew: the codes of the rows the block already holds, 16 a lane
    if (held && s_new > s_old) {
      const float ratio = __fdiv_rn(s_old, s_new);
      for (int k = lane; k < 16 * (D / 16); k += 32) {
        const int row = row0 + k / (D / 16);
        if (row >= pos || !DA_IN(p, size_t(head) * p.n_max + row, p.cache_rows)) continue;
        uint4* at = reinterpret_cast<uint4*>(codes + (size_t(head) * p.n_max + row) * D) + k % (D / 16);
        const uint4 old = *at;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[4];
          from_codes<KIND>(word_of(old, e), f);
          if constexpr (KIND == 1)  // (int8's -128)
            for (float& x : f) x = clamp_code<KIND>(x * ratio);
          w[e] = to_codes<KIND>(f[0], f[1], f[2], f[3], KIND == 1 ? 1.f : ratio);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

cudaError_t launch_kv_append_q8b(const BlockWriteArgs& a, cudaStream_t stream) {
  BlockWrite p{};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = a.x[i];
    p.sb[i] = a.stride[i][0], p.sh[i] = a.stride[i][1], p.st[i] = a.stride[i][2];
    p.codes[i] = static_cast<uint8_t*>(a.codes[i]);
    p.scale[i] = a.scale[i];
  }
  p.pos = a.pos;
  p.n_new = a.n_new;
  p.dev_error = a.dev_error;
  p.B = a.B, p.h_kv = a.h_kv, p.T = a.T, p.n_max = a.n_max;
  p.blk_shift = a.blk_shift;
  const int S = 1 << a.blk_shift;
  p.nblk = (a.n_max + S - 1) / S;
  // blocks that T rows at any position can touch (never more than there are)
  const long long touched = ((long long)a.T + 2 * S - 2) / S;
  p.touched = int(touched < p.nblk ? touched : p.nblk);
  const long long units = 2LL * a.B * a.h_kv * p.touched;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;  // (checked by the caller)
  p.units = unsigned(units);
  p.cache_rows = (long long)a.B * a.h_kv * a.n_max;
  p.scale_elems = (long long)a.B * a.h_kv * p.nblk;
  const int per_cta = (kWriteThreads / 32) / (S / 16);
  const long long ctas = (units + per_cta - 1) / per_cta;
  const long long places = (long long)a.sms * (a.d == 128 ? (a.x_bf16 ? write_ctas<128, true>() : write_ctas<128, false>())
                                                     : (a.x_bf16 ? write_ctas<64, true>() : write_ctas<64, false>()));
  const long long grid = ctas < places ? ctas : places;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, int(grid), kWriteThreads, 0, stream, p);
  };
  if (a.d == 128) {
    if (a.x_bf16) return a.kind == 1 ? go(kv_append_q8b_kernel<128, true, 1>) : go(kv_append_q8b_kernel<128, true, 2>);
    return a.kind == 1 ? go(kv_append_q8b_kernel<128, false, 1>) : go(kv_append_q8b_kernel<128, false, 2>);
  }
  if (a.x_bf16) return a.kind == 1 ? go(kv_append_q8b_kernel<64, true, 1>) : go(kv_append_q8b_kernel<64, true, 2>);
  return a.kind == 1 ? go(kv_append_q8b_kernel<64, false, 1>) : go(kv_append_q8b_kernel<64, false, 2>);
}

// ---------------------------------------------------------------------------
// Read: out[b, h, i, :] = s[block] * value(code) of row row_begin[b] + i, for
// the rows below the sequence's length; other rows of out are left alone.
// Bound: HBM (1 byte in, 2 or 4 out per element).  A lane writes 16 bytes at a
// time, so that a warp's loads and stores are whole runs of bytes.  CTAs are
// persistent and hold two parts of kReadUnroll rows for every run of lanes: one
// is loaded while the other is converted and stored.  The parts that hold rows
// are counted from the lengths and dealt round (dealt over all T rows of every
// sequence, a ragged batch of 4 took 21 us instead of 18; in one run per CTA,
// neighbouring addresses came apart in time and long reads took 3 to 15 % more).
// 16 x 8192 rows to bf16: 134 us, 6.0 TB/s.
// ---------------------------------------------------------------------------
struct BlockRead {
  const uint8_t* codes[2];
  const float* scale[2];
  void* out[2];              // [B, h_kv, T, D]
  const int32_t* seq_lens;   // [B]
  const int32_t* row_begin;  // nullable: [B] (else 0)
  int32_t* dev_error;
  int B, h_kv, T, n_max, nblk, blk_shift;
  int part_rows;             // rows of a part
  long long cache_rows, scale_elems, out_rows;       // extents, for the checked build
};

constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 8;
constexpr int kReadCtas = 4;  // CTAs an SM
constexpr int kReadBatch = 512;  // sequences whose rows are counted at a time

template <int D, bool OBF16, int KIND>
__global__ void __launch_bounds__(kReadThreads, kReadCtas)
    kv_read_q8b_kernel(const BlockRead p) {
  constexpr int EPL = OBF16 ? 8 : 4;        // elements of 16 output bytes
  constexpr int LPR = D / EPL;              // lanes per row
  constexpr int SETS = kReadThreads / LPR;  // row sets of a part: one for each LPR lanes
  allow_dependent_launch();
  wait_for_prerequisite_grid();

  // Rows and first part of every sequence (a slice of the batch at a time).
  __shared__ int rows_of[kReadBatch], begin_of[kReadBatch], first_of[kReadBatch + 1];
  __shared__ int warp_sum[kReadThreads / 32];

  // One part: kReadUnroll consecutive rows for every LPR lanes.  Its codes and
  // scales are loaded while the part before it is converted and stored.
  struct Part {
    uint2 w[kReadUnroll];
    float s[2];          // the scales of the first row's block and of the next
    int tensor, head, i0, rows, first_next;  // rows of i0 .. below `rows`; from i0 + first_next
                                             // on the second scale
  };
  const int c = threadIdx.x % LPR;
  auto load = [&](int b, int unit, int part, int rows, int begin, Part& q) {
    q.tensor = unit & 1;
    q.head = b * p.h_kv + (unit >> 1);
    q.rows = rows;
    q.i0 = part * p.part_rows + int(threadIdx.x / LPR) * kReadUnroll;
    if (q.i0 >= q.rows) return;
    const int blk = (begin + q.i0) >> p.blk_shift;
    q.first_next = ((blk + 1) << p.blk_shift) - (begin + q.i0);
    const float* scales = (q.tensor ? p.scale[1] : p.scale[0]) + size_t(q.head) * p.nblk;
    q.s[0] = q.s[1] = 0.f;
    if (DA_IN(p, blk, p.nblk)) q.s[0] = __ldcg(scales + blk);
    if (q.first_next < kReadUnroll && q.i0 + q.first_next < q.rows && DA_IN(p, blk + 1, p.nblk))
      q.s[1] = __ldcg(scales + blk + 1);
    const size_t in = size_t(q.head) * p.n_max + begin + q.i0;
    const uint8_t* src = (q.tensor ? p.codes[1] : p.codes[0]) + in * D + c * EPL;
#pragma unroll
    for (int k = 0; k < kReadUnroll; ++k)
      if (q.i0 + k < q.rows && DA_IN(p, in + k, p.cache_rows)) {
        if constexpr (OBF16) q.w[k] = __ldcs(reinterpret_cast<const uint2*>(src + k * D));
        else q.w[k].x = __ldcs(reinterpret_cast<const unsigned*>(src + k * D));
      }
  };
  auto store = [&](const Part& q) {
    const size_t row0 = size_t(q.head) * p.T + q.i0;
    void* out = q.tensor ? p.out[1] : p.out[0];
#pragma unroll
    for (int k = 0; k < kReadUnroll; ++k) {
      if (q.i0 + k >= q.rows || !DA_IN(p, row0 + k, p.out_rows)) continue;
      const float s = k < q.first_next ? q.s[0] : q.s[1];
      const size_t at = (row0 + k) * D + c * EPL;
      float f[4];
      from_codes<KIND>(q.w[k].x, f);
      if constexpr (OBF16) {
        float g[4];
        from_codes<KIND>(q.w[k].y, g);
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at),
               make_uint4(pack_bf16x2(f[0] * s, f[1] * s), pack_bf16x2(f[2] * s, f[3] * s),
                          pack_bf16x2(g[0] * s, g[1] * s), pack_bf16x2(g[2] * s, g[3] * s)));
      } else {
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(out) + at),
               make_float4(f[0] * s, f[1] * s, f[2] * s, f[3] * s));
      }
    }
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = 2 * p.h_kv;  // heads of K and V of a sequence
  // A sequence's rows (T at most), and its first one.
  auto rows_from = [&](int b, int& begin) {
    const int n = __ldcg(p.seq_lens + b);
    begin = p.row_begin ? __ldcg(p.row_begin + b) : 0;
    if ((n < 0 || n > p.n_max || begin < 0) && blockIdx.x == 0)
      flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
    return begin < 0 ? 0 : max(0, min(p.T, min(max(n, 0), p.n_max) - begin));
  };
  if (p.T <= p.part_rows) {  // one part a head: no need to count them (0.6 us of 3.8)
    for (int b = blockIdx.x == 0 ? tid : p.B; b < p.B; b += kReadThreads) {
      int begin;
      rows_from(b, begin);  // (CTA 0: every sequence's flags)
    }
    for (unsigned q = blockIdx.x; q < unsigned(p.B) * unsigned(units); q += gridDim.x) {
      const int b = int(q / unsigned(units));
      int begin;
      const int rows = rows_from(b, begin);
      Part now;
      load(b, int(q - unsigned(b) * unsigned(units)), 0, rows, begin, now);
      store(now);
    }
    return;
  }
  for (int b0 = 0; b0 < p.B; b0 += kReadBatch) {
    const int nb = min(kReadBatch, p.B - b0);
    // the rows of each sequence, and a scan of the parts they make
    const int run = (nb + kReadThreads - 1) / kReadThreads;
    const int from = min(nb, tid * run), to = min(nb, from + run);
    int mine = 0;
    for (int b = from; b < to; ++b) {
      int begin;
      const int rows = rows_from(b0 + b, begin);
      rows_of[b] = rows;
      begin_of[b] = begin;
      mine += units * ((rows + p.part_rows - 1) / p.part_rows);
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += warp_sum[w];
    int at = upto - mine;
    for (int b = from; b < to; ++b) {
      first_of[b] = at;
      at += units * ((rows_of[b] + p.part_rows - 1) / p.part_rows);
    }
    if (tid == kReadThreads - 1) first_of[nb] = upto;
    __syncthreads();
    const int total = first_of[nb];
    int part = int(blockIdx.x), b = 0;
    if (part < total) {
      auto load_part = [&](int q, Part& to_part) {
        if (q >= first_of[b + 1]) {  // (parts come in order): the last b with first_of[b] <= q
          int hi = nb - 1;
          for (++b; b < hi;) {
            const int mid = (b + hi + 1) >> 1;
            if (first_of[mid] <= q) b = mid; else hi = mid - 1;
          }
        }
        const int per = (rows_of[b] + p.part_rows - 1) / p.part_rows;
        const int r = q - first_of[b], unit = r / per;
        load(b0 + b, unit, r - unit * per, rows_of[b], begin_of[b], to_part);
      };
      Part now, next;
      load_part(part, now);
      for (; part < total; part += int(gridDim.x)) {
        if (part + int(gridDim.x) < total) load_part(part + int(gridDim.x), next);
        store(now);
        now = next;
      }
    }
    __syncthreads();  // the arrays are read
  }
}

cudaError_t launch_kv_read_q8b(const BlockReadArgs& a, cudaStream_t stream) {
  BlockRead p{};
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = static_cast<const uint8_t*>(a.codes[i]);
    p.scale[i] = a.scale[i];
    p.out[i] = a.out[i];
  }
  p.seq_lens = a.seq_lens;
  p.row_begin = a.row_begin;
  p.dev_error = a.dev_error;
  p.B = a.B, p.h_kv = a.h_kv, p.T = a.T, p.n_max = a.n_max, p.blk_shift = a.blk_shift;
  const int S = 1 << a.blk_shift;
  p.nblk = (a.n_max + S - 1) / S;
  p.part_rows = kReadThreads / (a.d / (a.out_bf16 ? 8 : 4)) * kReadUnroll;
  const long long per_head = (a.T + p.part_rows - 1LL) / p.part_rows;
  p.cache_rows = (long long)a.B * a.h_kv * a.n_max;
  p.scale_elems = (long long)a.B * a.h_kv * p.nblk;
  p.out_rows = (long long)a.B * a.h_kv * a.T;
  const long long parts = 2LL * a.B * a.h_kv * per_head;
  if (parts > 0x3fffffffLL) return cudaErrorInvalidValue;  // (checked by the caller)
  const long long places = (long long)a.sms * kReadCtas;
  const long long grid = parts < places ? parts : places;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, int(grid), kReadThreads, 0, stream, p);
  };
  if (a.d == 128) {
    if (a.out_bf16) return a.kind == 1 ? go(kv_read_q8b_kernel<128, true, 1>) : go(kv_read_q8b_kernel<128, true, 2>);
    return a.kind == 1 ? go(kv_read_q8b_kernel<128, false, 1>) : go(kv_read_q8b_kernel<128, false, 2>);
  }
  if (a.out_bf16) return a.kind == 1 ? go(kv_read_q8b_kernel<64, true, 1>) : go(kv_read_q8b_kernel<64, true, 2>);
  return a.kind == 1 ? go(kv_read_q8b_kernel<64, false, 1>) : go(kv_read_q8b_kernel<64, false, 2>);
}

}  // namespace da
