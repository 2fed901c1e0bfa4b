"""What the block-scaled decode keeps of its inputs' digits (needs a GB300)."""
import pytest
import torch

import decode_bounds as D
import terms_reference as R
from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
KINDS = [torch.int8, torch.float8_e4m3fn]
KID = ["int8", "fp8"]
OUTS = [torch.float32, torch.bfloat16]
OID = ["fp32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def codes(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(shape, generator=g) * R.Q[dtype] / 4
    return R.as_codes(R.round_codes(v.double().numpy(), dtype), dtype)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("d,heads", [(64, 2), (128, 2), (64, 20), (128, 20)])
@pytest.mark.parametrize("far", [0, 2, 8])
def test_blocks_of_no_weight_take_no_digits(far, d, heads, dtype, out_dtype):
    """The even heads' weight lies on block 1 alone, the odd heads' on block `far`, whose V scale is
    2^k times as large (or as small) and which the same warp sees: each head's output is the mean of
    its own block's rows, with all its digits.

    The 16 rows' scores are equal, so that their weights are equal but for their rounding with
    the V scale, part; 16 products and the merge are under 64 float roundings of 2^-24, in the
    numerator and the denominator.  The other rows weigh e^-160 = 2^-230, times 2^k nothing."""
    n, block = 200, 16
    part = D.weight_rounding("q8b") if out_dtype == torch.float32 else 2.0 ** -11
    for k in (0, 12, 20, 40, 100, -20, -100):
        V = codes((1, 1, n, d), dtype, 7)
        K = torch.zeros(1, 1, n, d)
        K[..., :2] = -100.0
        K[0, 0, 16:32, 0] = 100.0
        K[0, 0, far * 16:far * 16 + 16, 1] = 100.0
        K = K.to(dtype)
        ks = torch.full((1, 1, 13), 0.1)
        vs = torch.full((1, 1, 13), 2.0 ** -9)
        vs[0, 0, far] = 2.0 ** (k - 9)
        q = torch.zeros(1, heads, d, dtype=torch.bfloat16)
        q[0, 0::2, 0] = q[0, 1::2, 1] = 8.0 * 100.0 / float(K[0, 0, 16, 0].float())
        out = api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32([n]), block, scale=1.0,
                                  out_dtype=out_dtype).cpu().double()
        for h, at, s in ((0, 16, 2.0 ** -9), (1, far * 16, 2.0 ** (k - 9))):
            rows = V[0, 0, at:at + 16].double() * s
            want, size = rows.mean(0), rows.abs().mean(0)
            tol = size * (part + 128 * 2.0 ** -24)
            tol = tol + (want.abs() + tol) * (torch.finfo(out_dtype).eps / 2)
            err = (out[0, h::2] - want).abs()
            assert bool((err <= tol).all()), (k, h, float((err / tol).max()))


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("d,h_q,h_kv", [(64, 6, 2), (128, 8, 1), (64, 40, 2), (128, 20, 1)])
def test_queries_of_any_size(d, h_q, h_kv, dtype):
    """q far above what fp16 holds, and below its normal numbers, over K scales that bring the scores back."""
    B, n, block = 2, 700, 32
    g = torch.Generator().manual_seed(3)
    K, V = codes((B, h_kv, n, d), dtype, 4), codes((B, h_kv, n, d), dtype, 5)
    vs = torch.exp2(torch.randint(-8, -4, (B, h_kv, 22), generator=g).float())
    base = torch.randn(B, h_q, d, generator=g)
    for f in (1.0, 2.0 ** 17, 2.0 ** 60, 2.0 ** 120, 2.0 ** -12, 2.0 ** -20, 2.0 ** -60, 2.0 ** -110):
        q = (base * f).to(torch.bfloat16)
        ks = torch.full((B, h_kv, 22), 2.0 ** -5 / f)
        out = api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32([n, 333]), block)
        at = torch.arange(n) // block
        Kv, Vv = K.double() * ks[:, :, at, None].double(), V.double() * vs[:, :, at, None].double()
        want, tol = D.attend(q.cuda(), Kv.cuda(), Vv.cuda(), [n, 333], d ** -0.5, D.weight_rounding("q8b"),
                             floor=2.0 ** -31)
        D.check(out, want, tol, f"q times {f}")


def test_a_query_that_is_not_finite_stays_in_its_head():
    B, n, block, d, h_q = 1, 300, 16, 64, 8
    for dtype in KINDS:
        K, V = codes((B, 1, n, d), dtype, 4), codes((B, 1, n, d), dtype, 5)
        s = torch.full((B, 1, 19), 2.0 ** -5)
        q = torch.randn(B, h_q, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        args = (K.cuda(), V.cuda(), s.cuda(), s.cuda(), i32([n]), block)
        want, tol = D.attend(q.cuda(), K.cuda().double() * 2.0 ** -5, V.cuda().double() * 2.0 ** -5, [n], d ** -0.5,
                             D.weight_rounding("q8b"), floor=2.0 ** -31)
        for bad in (float("inf"), float("-inf"), float("nan")):
            q2 = q.clone()
            q2[0, 3, 7] = bad
            out = api.decode_attn_q8b(q2.cuda(), *args)
            keep = [h for h in range(h_q) if h != 3]
            D.check(out[:, keep], want[:, keep], tol[:, keep])
            assert not torch.isfinite(out[:, 3]).any()


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("d,h_q", [(64, 2), (128, 8), (128, 20)])
def test_scores_beyond_the_steps_of_float(d, h_q, splits, out_dtype):
    """Scores so large that a float of their size has no room for a scale's logarithm: one row is all
    that counts, and its value comes out, off by its weight's rounding, the merge's and the output's."""
    n = 700
    V = codes((1, 1, n, d), torch.int8, 3)
    q = torch.zeros(1, h_q, d, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    ks = torch.full((1, 1, 44), 2.0 ** 30)
    vs = torch.exp2(torch.randint(-20, 21, (1, 1, 44), generator=torch.Generator().manual_seed(1)).float())
    part = D.weight_rounding("q8b", out_dtype) + 64 * D.U
    for at in (0, 15, 16, 37, 300, 699):
        K = torch.randint(-100, 101, (1, 1, n, d), dtype=torch.int8)
        K[0, 0, at, 0] = 127
        out = api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32([n]), 16, scale=1.0,
                                  num_splits=splits, out_dtype=out_dtype).cpu().double()
        want = (V[0, 0, at].double() * float(vs[0, 0, at // 16])).expand(1, h_q, d)
        tol = want.abs() * part
        D.check(out, want, tol + (want.abs() + tol) * (torch.finfo(out_dtype).eps / 2))


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d,h_q", [(64, 4), (128, 8), (128, 20)])
def test_v_scales_at_the_ends_of_float(d, h_q, out_dtype):
    """V scales of every mantissa, down to float's subnormals and up to its largest powers."""
    B, n, block = 2, 300, 16
    g = torch.Generator().manual_seed(2)
    K, V = codes((B, 1, n, d), torch.int8, 4), codes((B, 1, n, d), torch.int8, 5)
    ks = torch.full((B, 1, 19), 2.0 ** -6)
    q = torch.randn(B, h_q, d, generator=g).to(torch.bfloat16)
    at = torch.arange(n) // block
    for low, high in ((-130.0, -124.0), (-127.0, -100.0), (-3.0, 3.0), (90.0, 110.0)):
        vs = torch.exp2(torch.empty(B, 1, 19, dtype=torch.float64).uniform_(low, high, generator=g)).float()
        Kv, Vv = K.double() * 2.0 ** -6, V.double() * vs[:, :, at, None].double()
        for splits in (0, 1, 2):
            out = api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32([n, 77]), block, num_splits=splits,
                                      out_dtype=out_dtype)
            want, tol = D.attend(q.cuda(), Kv.cuda(), Vv.cuda(), [n, 77], d ** -0.5, D.weight_rounding("q8b", out_dtype),
                                 out_dtype, floor=2.0 ** -31)
            # (sums and outputs among the subnormals: half a step of theirs for each of 64 roundings)
            D.check(out, want, tol + (64 * 2.0 ** -150 if out_dtype == torch.float32 else 2.0 ** -134 + 64 * 2.0 ** -150),
                    f"scales from 2^{low} to 2^{high}")
