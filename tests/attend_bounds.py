"""Chunk and shared-prefix attention in 64 bits with a bound on every element (decode_bounds), token by token."""
import torch

import decode_bounds as D


def part(out_dtype):
    """The rounding of a weight for the product with V: a bf16, with a bf16 remainder for a float32 output."""
    return 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -16


def chunk(q, K, V, lens, news, scale, out_dtype, window=0, prefix=0):
    """q [B, h_q, T, d] -> (want, tol) [B, h_q, T, d]; tokens at or past news[b] are zero with bound zero."""
    want = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(want)
    for b, (n, m) in enumerate(zip(lens, news)):
        if m == 0:
            continue
        ends = [max(0, n - m + i + 1) for i in range(m)]
        w, t = D.attend(q[b, :, :m].transpose(0, 1), K[b][None].expand(m, *K.shape[1:]), V[b][None].expand(m, *V.shape[1:]),
                        ends, scale, part(out_dtype), out_dtype, window=window, prefix=prefix)
        want[b, :, :m], tol[b, :, :m] = w.transpose(0, 1), t.transpose(0, 1)
    return want, tol


def shared(q, Kp, Vp, P, K, V, lens, scale, out_dtype):
    """Each sequence over the prefix's P rows and its own."""
    want = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(want)
    for b, n in enumerate(lens):
        rows = [torch.cat([x[:, :P], y[b, :, :n]], dim=1)[None] for x, y in ((Kp, K), (Vp, V))]
        w, t = D.attend(q[b:b + 1], *rows, [P + n], scale, part(out_dtype), out_dtype)
        want[b], tol[b] = w[0], t[0]
    return want, tol


def check(got, want, tol, what=""):
    """Outputs within their bounds; where nothing is seen, zero."""
    none = tol == 0
    assert (got.double()[none] == want[none]).all(), what
    D.check(torch.where(none, want, got.double()), want, tol, what)
