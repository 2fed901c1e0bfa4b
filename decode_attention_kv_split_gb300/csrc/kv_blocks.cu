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
// registers for its maximum), latency for single tokens: lengths, then x, the
// scale and the held codes at once, then the stores.  A warp owns 16 rows of a
// block, S / 16 warps a block, 128 / S blocks a CTA; a lane owns 16 elements
// of a row, so that it stores 16 codes at once.
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

// Four values, already divided by the scale, as codes.
template <int KIND>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  constexpr float Q = KIND == 1 ? 127.f : 448.f;
  a = fminf(fmaxf(a, -Q), Q), b = fminf(fmaxf(b, -Q), Q);
  c = fminf(fmaxf(c, -Q), Q), d = fminf(fmaxf(d, -Q), Q);
  if constexpr (KIND == 1) {
    const uint32_t ab = __byte_perm(__float2int_rn(a), __float2int_rn(b), 0x0040);
    const uint32_t cd = __byte_perm(__float2int_rn(c), __float2int_rn(d), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  } else {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
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
  long long units;           // 2 * B * h_kv * touched
  long long cache_rows, scale_elems;  // extents, for the checked build
};

constexpr int kWriteThreads = 256;

template <int D, bool XBF16, int KIND>
__global__ void __launch_bounds__(kWriteThreads)
    kv_append_q8b_kernel(const BlockWrite p) {
  constexpr int LPR = D / 16;        // lanes per row
  constexpr int RPP = 32 / LPR;      // rows a warp covers at once
  constexpr int PASS = 16 / RPP;     // passes over its 16 rows
  __shared__ float red[kWriteThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = 1 << p.blk_shift, W = S >> 4;  // rows of a block, warps of a block
  const int per_cta = (kWriteThreads / 32) / W;
  const long long unit = (long long)blockIdx.x * per_cta + warp / W;
  const int sub = warp % W;
  allow_dependent_launch();
  wait_for_prerequisite_grid();

  // unit -> (head, touched block, tensor); a unit past the end only takes part in the barrier
  const bool live_unit = unit < p.units;
  const int tensor = int(unit & 1);
  const long long u2 = unit >> 1;
  const int j = live_unit ? int(u2 % p.touched) : 0;
  const int head = live_unit ? int(u2 / p.touched) : 0;  // b * h_kv + h
  const int b = head / p.h_kv, h = head - b * p.h_kv;
  const int pos = __ldcg(p.pos + b);
  int m = p.T;
  bool bad = false;
  if (p.n_new) {
    m = __ldcg(p.n_new + b);
    bad = m < 0 || m > p.T;
    m = min(max(m, 0), p.T);
  }
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
  const int row0 = (blk << p.blk_shift) + sub * 16;  // this warp's first cache row
  const bool work = live_unit && m > 0 && (blk << p.blk_shift) < pos + m;
  const bool held = work && (blk << p.blk_shift) < pos;  // the block holds earlier rows
  const int rl = lane / LPR, c = lane % LPR;

  // ---- loads: new rows, the block's scale, the codes it already holds
  const size_t scale_at = size_t(head) * p.nblk + blk;
  float s_old = 0.f;
  const bool scale_in = !work || DA_IN(p, scale_at, p.scale_elems);
  if (held && scale_in) s_old = __ldcg(p.scale[tensor] + scale_at);
  float x[PASS][16];
  uint4 old[PASS];
  bool finite = true;
  float a = 0.f;
  if (work) {
    const char* base = static_cast<const char*>(p.x[tensor]);
    const long long off = (long long)b * p.sb[tensor] + (long long)h * p.sh[tensor] + c * 16;
    uint4 raw[PASS][XBF16 ? 2 : 4];
#pragma unroll
    for (int u = 0; u < PASS; ++u) {
      const int row = row0 + u * RPP + rl;
      const int i = row - pos;
      if (i >= 0 && i < m) {
        const uint4* src = reinterpret_cast<const uint4*>(
            base + (off + (long long)i * p.st[tensor]) * (XBF16 ? 2 : 4));
#pragma unroll
        for (int e = 0; e < (XBF16 ? 2 : 4); ++e) raw[u][e] = __ldcs(src + e);
      } else {
#pragma unroll
        for (int e = 0; e < (XBF16 ? 2 : 4); ++e) raw[u][e] = make_uint4(0, 0, 0, 0);
        if (i < 0 && DA_IN(p, size_t(head) * p.n_max + row, p.cache_rows))
          old[u] = *reinterpret_cast<const uint4*>(p.codes[tensor] +
                                                   (size_t(head) * p.n_max + row) * D + c * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < PASS; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float f;
        if constexpr (XBF16) {
          const uint32_t w = word_of(raw[u][e >> 3], (e >> 1) & 3);
          f = (e & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w);
        } else {
          f = __uint_as_float(word_of(raw[u][e >> 2], e & 3));
        }
        if (!isfinite(f)) {
          finite = false;
          f = 0.f;
        }
        x[u][e] = f;
        a = fmaxf(a, fabsf(f));
      }
  }
  if (!finite) flag_error(p.dev_error, DA_DEVERR_VALUE);

  // ---- the block's maximum and scale
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (lane == 0) red[warp] = a;
  __syncthreads();
  if (!work) return;
  const int w0 = warp - sub;
  for (int w = 0; w < W; ++w) a = fmaxf(a, red[w0 + w]);
  const float s_new = fmaxf(s_old, block_scale<KIND>(a));
  if (sub == 0 && lane == 0 && scale_in) p.scale[tensor][scale_at] = s_new;

  // ---- codes
  const bool grown = held && s_new > s_old;
  const float ratio = grown ? __fdiv_rn(s_old, s_new) : 1.f;
  // a power of two divides exactly by its inverse (2^-126 .. 2^121 have one)
  const uint32_t sbits = __float_as_uint(s_new);
  const bool pow2 = (sbits & 0x807fffffu) == 0 && sbits != 0 && (sbits >> 23) < 253;
  const float inv = pow2 ? __uint_as_float((254u << 23) - sbits) : 0.f;
#pragma unroll
  for (int u = 0; u < PASS; ++u) {
    const int row = row0 + u * RPP + rl;
    const int i = row - pos;
    uint4* dst = reinterpret_cast<uint4*>(p.codes[tensor] + (size_t(head) * p.n_max + row) * D +
                                          c * 16);
    if (i >= m || !DA_IN(p, size_t(head) * p.n_max + row, p.cache_rows)) continue;
    uint32_t w[4];
    if (i >= 0) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (pow2) x[u][e] *= inv;
        else x[u][e] = s_new != 0.f ? __fdiv_rn(x[u][e], s_new) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = to_codes<KIND>(x[u][4 * e], x[u][4 * e + 1], x[u][4 * e + 2], x[u][4 * e + 3]);
      *dst = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (grown) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[4];
        from_codes<KIND>(word_of(old[u], e), f);
        w[e] = to_codes<KIND>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
      }
      *dst = make_uint4(w[0], w[1], w[2], w[3]);
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
  p.units = 2LL * a.B * a.h_kv * p.touched;
  p.cache_rows = (long long)a.B * a.h_kv * a.n_max;
  p.scale_elems = (long long)a.B * a.h_kv * p.nblk;
  const int per_cta = (kWriteThreads / 32) / (S / 16);
  const long long grid = (p.units + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
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
// Bound: HBM (1 byte in, 2 or 4 out per element).  A lane takes 16 codes and
// four rows' worth of loads are in flight per lane.
// ---------------------------------------------------------------------------
struct BlockRead {
  const uint8_t* codes[2];
  const float* scale[2];
  void* out[2];              // [B, h_kv, T, D]
  const int32_t* seq_lens;   // [B]
  const int32_t* row_begin;  // nullable: [B] (else 0)
  int32_t* dev_error;
  int B, h_kv, T, n_max, nblk, blk_shift, per_head;  // per_head: CTAs of one head of one tensor
  long long cache_rows, scale_elems, out_rows;       // extents, for the checked build
};

constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 4;

template <int D, bool OBF16, int KIND>
__global__ void __launch_bounds__(kReadThreads) kv_read_q8b_kernel(const BlockRead p) {
  constexpr int LPR = D / 16;
  constexpr int ROWS = kReadThreads / LPR;  // rows of one step of the CTA
  allow_dependent_launch();
  wait_for_prerequisite_grid();
  const int part = int(blockIdx.x % unsigned(p.per_head));
  const unsigned u = blockIdx.x / unsigned(p.per_head);
  const int tensor = int(u & 1u);
  const int head = int(u >> 1);
  const int b = head / p.h_kv;
  int n = __ldcg(p.seq_lens + b);
  const int begin = p.row_begin ? __ldcg(p.row_begin + b) : 0;
  const bool bad = n < 0 || n > p.n_max || begin < 0;
  n = min(max(n, 0), p.n_max);
  if (bad && part == 0 && tensor == 0 && head == b * p.h_kv && threadIdx.x == 0)
    flag_error(p.dev_error, DA_DEVERR_SEQ_LEN);
  if (begin < 0) return;
  const int rows = min(p.T, n - begin);  // may be <= 0
  const int c = threadIdx.x % LPR;
  const int i0 = part * (ROWS * kReadUnroll) + threadIdx.x / LPR;
  const size_t in0 = size_t(head) * p.n_max + begin;
  const uint8_t* codes = tensor ? p.codes[1] : p.codes[0];
  const float* scales = tensor ? p.scale[1] : p.scale[0];
  void* out = tensor ? p.out[1] : p.out[0];
  uint4 w[kReadUnroll];
  float s[kReadUnroll];
#pragma unroll
  for (int k = 0; k < kReadUnroll; ++k) {
    const int i = i0 + k * ROWS;
    if (i < rows && DA_IN(p, in0 + i, p.cache_rows) &&
        DA_IN(p, size_t(head) * p.nblk + ((begin + i) >> p.blk_shift), p.scale_elems)) {
      w[k] = __ldcs(reinterpret_cast<const uint4*>(codes + (in0 + i) * D + c * 16));
      s[k] = __ldcg(scales + size_t(head) * p.nblk + ((begin + i) >> p.blk_shift));
    }
  }
#pragma unroll
  for (int k = 0; k < kReadUnroll; ++k) {
    const int i = i0 + k * ROWS;
    if (i >= rows || !DA_IN(p, size_t(head) * p.T + i, p.out_rows)) continue;
    float f[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float q[4];
      from_codes<KIND>(word_of(w[k], e), q);
#pragma unroll
      for (int z = 0; z < 4; ++z) f[4 * e + z] = q[z] * s[k];
    }
    const size_t at = (size_t(head) * p.T + i) * D + c * 16;
    if constexpr (OBF16) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        __stcs(dst + e, make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]),
                                   pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                   pack_bf16x2(f[8 * e + 4], f[8 * e + 5]),
                                   pack_bf16x2(f[8 * e + 6], f[8 * e + 7])));
    } else {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __stcs(dst + e, make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]));
    }
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
  const int rows = kReadThreads / (a.d / 16) * kReadUnroll;
  p.per_head = (a.T + rows - 1) / rows;
  p.cache_rows = (long long)a.B * a.h_kv * a.n_max;
  p.scale_elems = (long long)a.B * a.h_kv * p.nblk;
  p.out_rows = (long long)a.B * a.h_kv * a.T;
  const long long grid = 2LL * a.B * a.h_kv * p.per_head;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
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
