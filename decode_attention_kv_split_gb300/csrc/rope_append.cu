// Norms of queries and keys for each head, rotation by position and the write
// into the KV cache, in one pass (sm_103a).
#include <math.h>

#include "common.cuh"

namespace da {

// ---------------------------------------------------------------------------
// A head's vector x[d] of q or k becomes
//   y = x * (mean(x^2) + eps)^(-1/2) * w          (w nullable: y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the rot / 2 pairs
// of its token's angle row; pairs are (j, j + rot / 2), or (2j, 2j + 1) when
// interleaved.  All of it in float, rounded once.  q goes to q_out, k and the
// unchanged v into row pos[b] + i of the caches.
//
// Bound by HBM: every element is read and written once (and for a handful of
// tokens by the launch).  A group of lanes owns a head's vector, each lane two
// 16-byte pieces of it, chosen so that both members of a pair lie in one lane:
// the norm's sum is the only exchange.  A group takes HC heads of one token and
// one kind (q, k or v), so that their loads are in flight together and the
// angles and weights are read once for all of them.
// Measured: 16 prompts of 2048 tokens, 32 + 2 * 8 heads of 128 in bf16, 137 us = 5.9 TB/s
// (0.87 of a copy's rate); one token 2.3 us, which is the launch.
// ---------------------------------------------------------------------------
template <typename T>
struct RopeVec;
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo_to_f32(w[i]), x[2 * i + 1] = bf16_hi_to_f32(w[i]);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct RopeVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// (Ordinary loads, here and of the weights: the grid before may still write them when this one
// starts, which the read-only path must not see.)
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}

// The sum over the lanes of a head's vector.
template <int LPR>
__device__ __forceinline__ float group_sum(float v, unsigned lanes) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
  return v;
}

// 256 threads: prompts 153 us, not 134; 64: the chunks in float32 36 us, not 30.
constexpr int kRopeThreads = 128;

template <typename T, int LPR, int HC>
__global__ void __launch_bounds__(kRopeThreads) kv_append_rope_kernel(const RopeAppendArgs p) {
  using V = RopeVec<T>;
  constexpr int N = V::N;
  allow_dependent_launch();
  const int q_parts = (p.h_q + HC - 1) / HC, kv_parts = (p.h_kv + HC - 1) / HC;
  const int parts = q_parts + 2 * kv_parts;
  const long long unit =
      ((long long)blockIdx.x * kRopeThreads + threadIdx.x) / LPR;
  if (unit >= (long long)p.B * p.T * parts) return;  // a group of lanes leaves together
  const int sub = threadIdx.x % LPR;
  const unsigned lanes = LPR == 32 ? 0xffffffffu
                                   : ((1u << (LPR % 32)) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
  const int part = int(unit % parts);
  const long long token = unit / parts;
  const int i = int(token % p.T), b = int(token / p.T);

  wait_for_prerequisite_grid();
  // where the token goes
  int m = p.T;
  if (p.n_new) {
    m = p.n_new[b];
    if (m < 0 || m > p.T) {
      if (part == 0 && sub == 0 && i == 0) flag_error(p.dev_error, DA_DEVERR_POS);
      m = m < 0 ? 0 : p.T;
    }
  }
  if (i >= m) return;
  const long long row = (long long)p.pos[b] + i;
  const long long angle = (p.angle_pos ? (long long)p.angle_pos[b] : (long long)p.pos[b]) + i;
  if (p.pos[b] < 0 || row >= p.n_max || angle < 0 || angle >= p.n_angles) {
    if (part == 0 && sub == 0) flag_error(p.dev_error, DA_DEVERR_POS);
    return;
  }

  const int kind = part < q_parts ? 0 : part < q_parts + kv_parts ? 1 : 2;
  const int heads = kind == 0 ? p.h_q : p.h_kv;
  const int h0 = (part - (kind == 0 ? 0 : kind == 1 ? q_parts : q_parts + kv_parts)) * HC;
  const int d = kind == 2 ? p.d_v : p.d_k;
  // this lane's pieces: both members of its pairs while rotated pairs last,
  // then neighbours
  const int half = p.rot / 2, half_pieces = p.interleaved ? 0 : half / N;
  const bool on = sub < d / N / 2;
  const bool paired = kind != 2 && sub < half_pieces;
  const int pa = paired ? sub : 2 * sub, pb = paired ? sub + half_pieces : 2 * sub + 1;
  const T* src = static_cast<const T*>(p.x[kind]) + b * p.x_stride[kind][0] + i * p.x_stride[kind][2];
  uint4 raw[HC][2];
#pragma unroll
  for (int u = 0; u < HC; ++u) {
    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
    if (on && h0 + u < heads) {
      const T* x = src + (h0 + u) * p.x_stride[kind][1];
      if (DA_IN(p, (x - static_cast<const T*>(p.x[kind])) + d - 1, p.x_elems[kind])) {
        raw[u][0] = *reinterpret_cast<const uint4*>(x + pa * N);
        raw[u][1] = *reinterpret_cast<const uint4*>(x + pb * N);
      }
    }
  }
  // where the heads go: q_out by its strides, K and V as [B, h_kv, n_max, d]
  T* dst;
  long long head_step;
  if (kind == 0) {
    dst = static_cast<T*>(p.q_out) + b * p.out_stride[0] + i * p.out_stride[2];
    head_step = p.out_stride[1];
  } else {
    dst = static_cast<T*>(p.cache[kind - 1]) + ((long long)b * p.h_kv * p.n_max + row) * d;
    head_step = (long long)p.n_max * d;
  }
  const long long dst_elems = kind == 0 ? p.out_elems : (long long)p.B * p.h_kv * p.n_max * d;
  const T* dst0 = static_cast<const T*>(kind == 0 ? p.q_out : p.cache[kind - 1]);

  if (kind == 2) {
#pragma unroll
    for (int u = 0; u < HC; ++u)
      if (on && h0 + u < heads) {
        T* y = dst + (h0 + u) * head_step;
        if (DA_IN(p, (y - dst0) + d - 1, dst_elems)) {
          *reinterpret_cast<uint4*>(y + pa * N) = raw[u][0];
          *reinterpret_cast<uint4*>(y + pb * N) = raw[u][1];
        }
      }
    return;
  }

  // the token's angles for this lane's pairs (c = 1, s = 0 outside them) and its weights
  float c[N], s[N];
  const float* cos_row = p.cos + angle * half;
  const float* sin_row = p.sin + angle * half;
  const bool turned = on && (p.interleaved ? 2 * sub * N < p.rot : paired);
  if (turned) {
    // interleaved: N / 2 pairs of each of two neighbouring pieces; else N pairs
    const int first = sub * N;
    load_floats<N>(cos_row + first, c);
    load_floats<N>(sin_row + first, s);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) c[e] = 1.f, s[e] = 0.f;
  }
  const T* weight = static_cast<const T*>(p.weight[kind]);
  uint4 w_raw[2] = {};
  if (weight && on) {
    w_raw[0] = *reinterpret_cast<const uint4*>(weight + pa * N);
    w_raw[1] = *reinterpret_cast<const uint4*>(weight + pb * N);
  }
#pragma unroll
  for (int u = 0; u < HC; ++u) {
    if (h0 + u >= heads) break;  // the same for a group's lanes
    float a[N], z[N];
    V::unpack(raw[u][0], a);
    V::unpack(raw[u][1], z);
    if (weight) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) sq = fmaf(a[e], a[e], fmaf(z[e], z[e], sq));
      const float r = __frsqrt_rn(group_sum<LPR>(sq, lanes) * p.inv_d + p.eps);
      float wa[N], wz[N];
      V::unpack(w_raw[0], wa);
      V::unpack(w_raw[1], wz);
#pragma unroll
      for (int e = 0; e < N; ++e) a[e] = a[e] * r * wa[e], z[e] = z[e] * r * wz[e];
    }
    // (elements past rot, whole lanes of them, stay as they are: with c = 1 and s = 0 alone an
    // infinity or NaN among them would reach its neighbour.  Prompts 137.7 us, 136.1 without the
    // selects, 140.7 with branches)
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float a0 = a[e], a1 = a[e + 1], z0 = z[e], z1 = z[e + 1];
        const float ca = c[e / 2], sa = s[e / 2], cz = c[N / 2 + e / 2], sz = s[N / 2 + e / 2];
        a[e] = turned ? a0 * ca - a1 * sa : a0, a[e + 1] = turned ? a1 * ca + a0 * sa : a1;
        z[e] = turned ? z0 * cz - z1 * sz : z0, z[e + 1] = turned ? z1 * cz + z0 * sz : z1;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float x0 = a[e], x1 = z[e];
        a[e] = turned ? x0 * c[e] - x1 * s[e] : x0;
        z[e] = turned ? x1 * c[e] + x0 * s[e] : x1;
      }
    }
    if (on) {
      T* y = dst + (h0 + u) * head_step;
      if (DA_IN(p, (y - dst0) + d - 1, dst_elems)) {
        *reinterpret_cast<uint4*>(y + pa * N) = V::pack(a);
        *reinterpret_cast<uint4*>(y + pb * N) = V::pack(z);
      }
    }
  }
}

template <typename T, int LPR, int HC>
static cudaError_t launch_rope_hc(const RopeAppendArgs& a, cudaStream_t stream) {
  const long long parts = (a.h_q + HC - 1) / HC + 2LL * ((a.h_kv + HC - 1) / HC);
  const long long threads = (long long)a.B * a.T * parts * LPR;
  const long long grid = (threads + kRopeThreads - 1) / kRopeThreads;
  return launch_dependent(kv_append_rope_kernel<T, LPR, HC>, int(grid), kRopeThreads, 0, stream, a);
}

template <typename T, int LPR>
static cudaError_t launch_rope_lanes(const RopeAppendArgs& a, cudaStream_t stream) {
  const long long lanes = (long long)a.B * a.T * (a.h_q + 2LL * a.h_kv) * LPR;
  // Four heads a group once the SMs have threads enough without (1024 tokens of 32 + 2 * 8 heads of
  // 128 in float32: 7.2 us with four, 9.7 with one; 256 tokens 4.2 and 3.7, one token 2.8 and 2.1).
  if (lanes > a.sms * 2048LL) return launch_rope_hc<T, LPR, 4>(a, stream);
  return launch_rope_hc<T, LPR, 1>(a, stream);
}

template <typename T>
static cudaError_t launch_rope_type(const RopeAppendArgs& a, cudaStream_t stream) {
  const int lanes = a.d_k / RopeVec<T>::N / 2;
  if (lanes <= 4) return launch_rope_lanes<T, 4>(a, stream);
  if (lanes <= 8) return launch_rope_lanes<T, 8>(a, stream);
  if (lanes <= 16) return launch_rope_lanes<T, 16>(a, stream);
  return launch_rope_lanes<T, 32>(a, stream);
}

cudaError_t launch_kv_append_rope(const RopeAppendArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch_rope_type<__nv_bfloat16>(a, stream) : launch_rope_type<float>(a, stream);
}

}  // namespace da
