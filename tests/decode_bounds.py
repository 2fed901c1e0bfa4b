"""Decode attention in 64 bits with a bound on every output element by itself.

terms_reference.tolerance bounds all outputs by the largest cached value; an
output that averages many rows is far smaller, so that bound forgives errors of
many times the output's own rounding.  Here the bound of an element is made of
the weighted magnitudes that enter it."""
import torch

U = 2.0 ** -24  # half a step of float, relative to the value


def weight_rounding(kind, out_dtype=torch.float32):
    """The relative rounding of a weight as a kernel family multiplies it: a float; a bf16 head and
    a bf16 remainder (2^-8 of 2^-8); an fp16 head and an fp16 remainder (2^-11 of 2^-11), for a
    bf16 output the head alone."""
    if kind == "q8b" and out_dtype == torch.bfloat16:
        return 2.0 ** -11
    return {"fp32": U, "bf16": 2.0 ** -16, "q8b": 2.0 ** -22}[kind]


SHORT_CAP = 128.0  # up to here the cap of a bf16 output may take the form that is off by c 2^-22


def attend(q, K, V, lens, scale, part, out_dtype=torch.float32, softcap=0.0, slopes=None, window=0, prefix=0,
           begin=None, floor=0.0):
    """q [B, h_q, d_k], K/V [B, h_kv, n_max, d] -> (want, tol), float64 [B, h_q, d_v] both.

    With u = 2^-24, p_l a row's weight of the softmax and v_l its value, a computed output is
    sum p_l (1 + e_l) (1 + part) v_l / sum p_l (1 + e_l), where
    * a score's error e_l (the weight's relative one): d products and sums in float, d u
      sum |q_j K_j| scale; the cap, c 2^-22; the exponent's own rounding and its parts (log2 e, the
      bias, the difference from the maximum), 2^-22 of the largest score and of the row's
      bias, counted from the seen row where it is largest; ex2, 2^-22, twice;
    * part: the weight's rounding for the product with V;
    * sums: n / 8 steps of the MMA's accumulator, which may cut off (2 u), 64 in the merges; in
      the numerator and the denominator;
    * floor: what a weight below its type's normal numbers loses, relative to the largest product
      of a weight and a value's scale;
    * the output's own rounding, half a step of it.
    Numerator and denominator are off by at most the sums of their terms' bounds."""
    dev = q.device
    B, h_q, d = q.shape
    h_kv, g = K.shape[1], h_q // K.shape[1]
    want = torch.zeros((B, h_q, V.shape[3]), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(want)
    half = torch.finfo(out_dtype).eps / 2
    for b, n in enumerate(lens):
        rows = torch.arange(n, device=dev)
        first = 0 if begin is None else int(begin[b])
        first = max(first, n - window) if window > 0 else first
        rows = rows[(rows < prefix) | (rows >= first)]
        if not rows.numel():
            continue
        for k in range(h_kv):
            x = q[b, k * g:k * g + g].double()
            key, val = K[b, k][rows].double(), V[b, k][rows].double()
            s = scale * (x @ key.T)
            size = abs(scale) * (x.abs() @ key.abs().T).amax(1, keepdim=True)
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            top = s.abs().amax(1, keepdim=True)
            e = d * U * size + 2.0 ** -22 * (top + 2.0)
            if softcap > 0:
                # (the long form of a cap far above the scores is off by parts of them, not of itself)
                short = out_dtype == torch.bfloat16 and softcap <= SHORT_CAP
                e = e + 2.0 ** -22 * (softcap if short else min(softcap, float(size.max())))
            if slopes is not None:
                sl = torch.as_tensor(slopes, dtype=torch.float32).double().to(dev)[k * g:k * g + g, None]
                s = s - sl * (n - 1 - rows).double()
                far = torch.where(sl >= 0, (rows[-1] - rows).double(), (rows - rows[0]).double())
                e = e + 2.0 ** -22 * sl.abs() * far
            p = torch.softmax(s, 1)
            pe, sums = p * e.expand_as(p), (n / 8 + 64) * 2 * U
            out = p @ val
            low = floor * n * (p[:, :, None] * val.abs()[None]).amax((1, 2)).unsqueeze(1) if floor else 0.0
            at = slice(k * g, k * g + g)
            want[b, at] = out
            tol[b, at] = (pe @ val.abs() + (p @ val.abs()) * (part + sums) + low
                          + out.abs() * (pe.sum(1, keepdim=True) + sums)) * 1.01
            # (rounded from a value that is off by that much)
            tol[b, at] += half * (out.abs() + tol[b, at])
    return want, tol


def check(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() / tol.clamp(min=1e-300)
    over = torch.where((got == want), torch.zeros_like(over), over)
    assert float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the bound of its element"
    return float(over.max())
