"""Plain 64-bit implementations that the tests of score terms and of the
block-scaled 8-bit cache compare with, written from the definitions, and the
bounds their tolerances come from.  No CUDA, nothing of the library."""
import math

import numpy as np
import torch

Q = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


# ----------------------------------------------------------------- attention
def seen_rows(n, window=0, prefix=0, begin=0):
    """The rows that the query at row n - 1 sees."""
    first = max(begin, n - window) if window > 0 else begin
    return [l for l in range(n) if l < prefix or l >= first]


def attend(q, K, V, lens, scale, softcap=0.0, slopes=None, window=0, prefix=0, begin=None):
    """q [B, h_q, d_k], K/V [B, h_kv, n_max, d] (any float type) -> float64 [B, h_q, d_v], and a
    bound on |s| summed without signs (max over rows of scale * sum_j |q_j K_j|)."""
    B, h_q, _ = q.shape
    h_kv = K.shape[1]
    out = torch.zeros((B, h_q, V.shape[3]), dtype=torch.float64)
    size = 0.0
    for b, n in enumerate(lens):
        rows = seen_rows(n, window, prefix, 0 if begin is None else int(begin[b]))
        if not rows:
            continue
        at = torch.tensor(rows)
        for h in range(h_q):
            k = K[b, h // (h_q // h_kv)][at].double()
            v = V[b, h // (h_q // h_kv)][at].double()
            x = q[b, h].double()
            s = scale * (k @ x)
            size = max(size, abs(scale) * float((k.abs() @ x.abs()).max()))
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * (n - 1 - at).double()
            p = torch.exp(s - s.max())
            out[b, h] = (p @ v) / p.sum()
    return out, size


def tolerance(d, size, softcap, vmax, n, weight_bits, out_eps=0.0):
    """A bound on |out - exact| from the roundings on the way (u = 2^-24, half a float step).

    * a score: d products and sums in float, d u size; its cap: tanh within 2 steps of a number
      up to 1, and the products around it, softcap * 2^-22; its bias: three roundings of a
      number b that a weight e^-b multiplies, b e^-b < 0.37, so under 2^-22; the exponent in the
      log2 domain and ex2 itself: 2^-22 of the largest |score| (size, or the cap) and 2^-22.
      A score off by e changes a weight by the factor 1 + e, and the output by at most 2 e vmax.
    * a weight as two parts of the MMA's type: 2^-weight_bits of it; below the type's range
      2^-25 of the warp's largest weight for each of its n / 8 rows.
    * sums of the weighted rows and the merge of partials: (n / 16 + 64) u vmax.
    * the output's own rounding: half a step of its type."""
    u = 2.0 ** -24
    top = min(size, softcap) if softcap > 0 else size
    score = d * u * size + (softcap * 2.0 ** -22 if softcap > 0 else 0.0) + 2.0 ** -22 * (top + 2.0)
    return vmax * (2 * score + 2.0 ** -weight_bits + n / 8 * 2.0 ** -25 + (n / 16 + 64) * u
                   + out_eps / 2)


# ----------------------------------------------------------------- block-scaled cache
def need(a, top):
    """The smallest power of two s >= 2^-126 with a <= top * s; 0 for a = 0."""
    if a == 0:
        return 0.0
    e = math.floor(math.log2(a / top)) - 1
    while a > top * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def code_values(codes):
    return codes.double()


def round_codes(y, dtype):
    """y (float64 array) to the nearest code's value, ties to the even code, clamped."""
    y = np.clip(y, -Q[dtype], Q[dtype])
    if dtype == torch.int8:
        return np.rint(y)
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = np.exp2(e - 3)  # 3 bits behind the leading one; 2^-9 below 2^-6
    return np.rint(y / step) * step


def append_rows(codes, scale, x, pos, m, block):
    """The definition of the quantising write for one head: codes [n_max, d] (values, float64)
    and scale [nblk] (float64) in place; x [T, d]; m rows behind pos."""
    dtype = append_rows.dtype
    x = np.where(np.isfinite(x), x, 0.0)
    for k in range(pos // block, (pos + m + block - 1) // block) if m else ():
        lo, hi = max(pos, k * block), min(pos + m, (k + 1) * block)
        s = scale[k] if k * block < pos else 0.0
        s2 = max(s, need(np.abs(x[lo - pos:hi - pos]).max(), Q[dtype]))
        if s2 > s and k * block < pos:
            f = float(np.float32(s) / np.float32(s2))
            old = (codes[k * block:pos] * f).astype(np.float32).astype(np.float64)
            codes[k * block:pos] = round_codes(old, dtype)
        new = x[lo - pos:hi - pos]
        # the quotient is rounded to float where s2 is no power of two
        y = (new.astype(np.float32) / np.float32(s2)).astype(np.float64) if s2 else new * 0.0
        codes[lo:hi] = round_codes(y, dtype)
        scale[k] = s2


def append(codes, scale, x, pos, m, block, dtype):
    """append_rows over [B, h, ...] arrays: codes [B, h, n_max, d], scale [B, h, nblk] (float64,
    returned as copies), x [B, h, T, d], pos and m lists."""
    append_rows.dtype = dtype
    codes, scale = codes.copy(), scale.copy()
    for b in range(codes.shape[0]):
        for h in range(codes.shape[1]):
            append_rows(codes[b, h], scale[b, h], x[b, h], pos[b], m[b], block)
    return codes, scale


def values(codes, scale, block):
    """float64 values of codes [B, h, n, d] with scale [B, h, nblk]."""
    s = np.repeat(scale, block, axis=2)[:, :, :codes.shape[2]]
    return codes * s[..., None]


def as_codes(values_, dtype):
    """Values that are codes, as a tensor of them."""
    return torch.from_numpy(values_).float().to(dtype)
