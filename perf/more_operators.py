"""Cases for the operators that take a sequence from its projections to its attention: the norms of queries and keys for
each head with the rotation by position and the write into the cache, the attention of a chunk of tokens over the cache
(causal, with a sliding window and a few first rows that stay visible), and the decode step of a batch that shares a
long prefix.

Every case runs in a plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through the
package's entry points.  Lengths follow from the case alone, values from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------- the cases
def _rope(name, B, T, h_q, h_kv, d, lo, hi, n_max, dtype, rot, interleaved=False, norm=True, ragged=False, shift=0):
    return {"name": name, "op": "rope", "B": B, "T": T, "h_q": h_q, "h_kv": h_kv, "d": d, "lo": lo, "hi": hi,
            "n_max": n_max, "dtype": dtype, "rot": rot, "interleaved": interleaved, "norm": norm, "ragged": ragged,
            "shift": shift}


def _chunk(name, B, T, h_q, h_kv, d, lo, hi, n_max, window=0, prefix=0, ragged=False):
    return {"name": name, "op": "chunk", "B": B, "T": T, "h_q": h_q, "h_kv": h_kv, "d": d, "lo": lo, "hi": hi,
            "n_max": n_max, "window": window, "prefix": prefix, "ragged": ragged}


def _shared(name, B, h_q, h_kv, d, P, lo, hi, n_max):
    return {"name": name, "op": "shared", "B": B, "h_q": h_q, "h_kv": h_kv, "d": d, "P": P, "lo": lo, "hi": hi,
            "n_max": n_max}


def listed():
    return [
        # one token of one sequence: the latency of a call in a decode step
        _rope("rope_one_token", 1, 1, 32, 8, 128, 1000, 1000, 1024, "bf16", 128),
        # one token each of a ragged batch whose rows follow a shared prefix of 4096
        _rope("rope_decode_batch", 64, 1, 32, 8, 128, 100, 2000, 2048, "bf16", 128, shift=4096),
        # a chunk of ragged prompts, fp32, half of each head rotated in neighbouring pairs, no norms
        _rope("rope_chunk_fp32", 4, 1021, 32, 32, 128, 0, 3000, 4112, "fp32", 64, interleaved=True, norm=False,
              ragged=True),
        # whole prompts
        _rope("rope_prompts", 16, 2048, 32, 8, 128, 0, 0, 2048, "bf16", 128),
        # a few drafted tokens of one sequence, checked in one call
        _chunk("chunk_few_tokens", 1, 5, 8, 2, 64, 300, 300, 512),
        # a few drafted tokens of two long contexts
        _chunk("chunk_few_tokens_long", 2, 8, 64, 8, 128, 131001, 131056, 131072),
        # ragged chunks of prompts behind what is cached, a sliding window and four first rows that stay visible
        _chunk("chunk_ragged_window", 8, 1021, 32, 8, 128, 100, 7000, 8192, window=4096, prefix=4, ragged=True),
        # whole prompts
        _chunk("chunk_prompts", 2, 8192, 32, 8, 128, 0, 0, 8192),
        # four sequences behind one short instruction
        _shared("shared_small", 4, 8, 2, 64, 1000, 10, 100, 128),
        # a batch behind a long system prompt
        _shared("shared_gqa", 16, 32, 8, 128, 8192, 100, 2048, 2048),
        # a large batch that asks about one long document
        _shared("shared_document", 64, 64, 8, 128, 32768, 64, 1000, 1024),
        # one kv head for 32 query heads
        _shared("shared_mqa", 33, 32, 1, 128, 16383, 1, 4000, 4096),
    ]


#: what the largest listed cases move and compute: a drawn case stays below it
LARGEST_BYTES = 0.8e9
LARGEST_SCORES = 2 * 32 * 8192 * 8192


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "shared", "shared"])
    while True:
        h_kv = rng.choice([1, 2, 3, 4, 8, 16])
        h_q = h_kv * rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
        d = rng.choice([64, 128, 128])
        B = _logint(rng, 1, 64)
        if op == "rope":
            d = rng.choice([64, 128, 128, 256])
            T = rng.choice([1, _logint(rng, 2, 8192)])
            lo = rng.choice([0, _logint(rng, 1, 8192)])
            c = _rope("", B, T, h_q, h_kv, d, lo // 3, lo, lo + T + rng.randrange(0, 70), rng.choice(["bf16", "bf16", "fp32"]),
                      rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.4, rng.random() < 0.7,
                      T > 1 and rng.random() < 0.4, rng.choice([0, 0, _logint(rng, 1, 32768)]))
        elif op == "chunk":
            T = rng.choice([1, _logint(rng, 2, 16), _logint(rng, 2, 8192), _logint(rng, 2, 8192)])
            lo = rng.choice([0, _logint(rng, 1, 131072 - T)])
            c = _chunk("", B, T, h_q, h_kv, d, rng.choice([lo, lo // 8]), lo, lo + T + rng.randrange(0, 70),
                       rng.choice([0, 0, _logint(rng, 1, 8192)]), rng.choice([0, 0, _logint(rng, 1, 300)]),
                       T > 1 and rng.random() < 0.4)
        else:
            hi = _logint(rng, 1, 8192)
            c = _shared("", _logint(rng, 1, 256), h_q, h_kv, d, _logint(rng, 1, 65536), rng.choice([0, hi // 8, hi]), hi,
                        hi + rng.randrange(0, 70))
        del c["name"]
        if work(c)["bytes"] <= LARGEST_BYTES and _held(c) <= 2.2 * LARGEST_BYTES and _scores(c) <= LARGEST_SCORES:
            return c


def _held(c):
    """Bytes of the caches a case holds."""
    rows = c["B"] * c["n_max"] + c.get("P", 0)
    return rows * c["h_kv"] * 2 * c["d"] * SIZE[c.get("dtype", "bf16")]


def _scores(c):
    """Scores that the plain form computes."""
    if c["op"] == "rope":
        return 0
    return c["B"] * c["h_q"] * c.get("T", 1) * (c["n_max"] + c.get("P", 0))


def _spread(c, k=0.6180339887498949):
    """A fraction in [0, 1) for each sequence of the case."""
    return [((b + 1) * k) % 1.0 for b in range(c["B"])]


def _lens(c):
    """Rows that each sequence holds before the call (shared prefix not counted)."""
    return [c["lo"] + int(f * (c["hi"] - c["lo"] + 1)) for f in _spread(c)]


def _news(c):
    """Tokens that each sequence brings: T, or between none and T in a ragged chunk (T for the first)."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    return [c["T"] if b == 0 else int(f * (c["T"] + 1)) for b, f in enumerate(_spread(c, 0.7548776662466927))]


def _pairs(c, n, m):
    """Pairs of a query and a row it sees, and rows seen by any, for m new tokens whose last stands at row n - 1."""
    total = 0
    for i in (range(m) if c["window"] else ()):
        at = n - m + i
        first = max(0, at + 1 - c["window"])
        total += at + 1 - first + min(first, c["prefix"])
    if not c["window"]:
        return m * (n - m) + m * (m + 1) // 2, n
    first = max(0, n - m + 1 - c["window"]) if m else n
    return total, n - first + min(first, c["prefix"])


def work(c):
    d, size = c["d"], SIZE[c.get("dtype", "bf16")]
    heads = c["h_q"] + 2 * c["h_kv"]
    if c["op"] == "rope":
        tokens = sum(_news(c))
        tables = 2 * 4 * (c["rot"] // 2) * (min(tokens, c["T"] + c["hi"] - c["lo"]))
        return {"bytes": 2 * tokens * heads * d * size + tables, "flops": 0}
    if c["op"] == "chunk":
        news = _news(c)
        got = [_pairs(c, n + m, m) for n, m in zip(_lens(c), news) if m]
        pairs, rows = sum(g[0] for g in got), sum(g[1] for g in got)
        return {"bytes": (2 * sum(news) * c["h_q"] + 2 * rows * c["h_kv"]) * d * size, "flops": 4 * pairs * c["h_q"] * d}
    rows = sum(_lens(c))
    return {"bytes": (2 * c["B"] * c["h_q"] + 2 * (rows + c["P"]) * c["h_kv"]) * d * size,
            "flops": 4 * (rows + c["B"] * c["P"]) * c["h_q"] * d}


# ------------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    B, h_q, h_kv, d, n_max = c["B"], c["h_q"], c["h_kv"], c["d"], c["n_max"]
    t = DTYPES[c.get("dtype", "bf16")]
    s = {"case": c, "scale": 1.0 / math.sqrt(d)}
    lens = _lens(c)
    if c["op"] == "shared":
        s["K_prefix"], s["V_prefix"] = (rand(h_kv, c["P"], d).to(t) for _ in range(2))
        s["K"], s["V"] = (rand(B, h_kv, n_max, d).to(t) for _ in range(2))
        s["q"] = (2.0 * rand(B, h_q, d)).to(t)
        s["lens"] = ints(lens)
        s["out"] = torch.zeros((B, h_q, d), dtype=t, device=DEV)
        return s
    T, news = c["T"], _news(c)
    s["new"] = ints(news) if c["ragged"] else None
    s["K"], s["V"] = (rand(B, h_kv, n_max, d).to(t) for _ in range(2))
    if c["op"] == "chunk":
        # queries and outputs token after token, as the layers around the attention hold them
        s["q"] = (2.0 * rand(B, T, h_q, d)).to(t).transpose(1, 2)
        s["lens"] = ints([n + m for n, m in zip(lens, news)])
        s["out"] = torch.zeros((B, T, h_q, d), dtype=t, device=DEV).transpose(1, 2)
        return s
    # the columns of one projection [B, T, (h_q + 2 h_kv) d], as it leaves them
    x = (1.5 * rand(B, T, h_q + 2 * h_kv, d)).to(t)
    s["q"] = x[:, :, :h_q].transpose(1, 2)
    s["k_new"] = x[:, :, h_q:h_q + h_kv].transpose(1, 2)
    s["v_new"] = x[:, :, h_q + h_kv:].transpose(1, 2)
    s["pos"] = ints(lens)
    s["angle_pos"] = ints([n + c["shift"] for n in lens]) if c["shift"] else None
    # the model's table of angles, made once: in 64 bits, since far positions times a frequency lose digits in 32
    half = c["rot"] // 2
    freq = torch.exp(-math.log(10000.0) * torch.arange(half, device=DEV, dtype=torch.float64) / half)
    angle = torch.arange(c["shift"] + n_max, device=DEV, dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["q_weight"], s["k_weight"] = ((1.0 + 0.2 * rand(d)).to(t) if c["norm"] else None for _ in range(2))
    s["q_out"] = torch.zeros((B, T, h_q, d), dtype=t, device=DEV).transpose(1, 2)
    return s


# ------------------------------------------------------------------------------------------------- the plain forms
def _plain_rotated(c, s, x, weight):
    """x [B, h, T, d] with each head's norm and rotation, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    base = s["pos"] if s["angle_pos"] is None else s["angle_pos"]
    at = (base.long()[:, None] + torch.arange(c["T"], device=DEV)).clamp(max=s["cos"].shape[0] - 1)
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]        # [B, 1, T, rot / 2]
    rot, half = c["rot"], c["rot"] // 2
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(c, s):
    T = c["T"]
    new = torch.full_like(s["pos"], T) if s["new"] is None else s["new"]
    live = torch.arange(T, device=DEV)[None] < new[:, None]        # [B, T]
    q = _plain_rotated(c, s, s["q"], s["q_weight"]).to(s["q"].dtype)
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    k = _plain_rotated(c, s, s["k_new"], s["k_weight"]).to(s["K"].dtype)
    b, i = torch.nonzero(live, as_tuple=True)
    row = s["pos"].long()[b] + i
    s["K"][b, :, row] = k[b, :, i]
    s["V"][b, :, row] = s["v_new"][b, :, i]
    return {"q": s["q_out"], "K": s["K"], "V": s["V"]}


def _softmax_rows(t):
    p = torch.exp(t - t.amax(-1, keepdim=True))
    return p, p.sum(-1, keepdim=True)


def _plain_chunk(c, s):
    g = c["h_q"] // c["h_kv"]
    for b, (n, m) in enumerate(zip(_lens(c), _news(c))):
        if m == 0:
            continue
        n += m
        row = torch.arange(n, device=DEV)[None]
        at = torch.arange(n - m, n, device=DEV)[:, None]
        seen = row <= at
        if c["window"]:
            seen &= (row > at - c["window"]) | (row < c["prefix"])
        step = c["h_kv"] if c["h_q"] * m * n <= 1 << 29 else 1    # kv heads at a time: scores of a few GB at most
        for h in range(0, c["h_kv"], step):
            q = s["q"][b, h * g:(h + step) * g, :m].float().reshape(step, g * m, -1)
            K, V = s["K"][b, h:h + step, :n].float(), s["V"][b, h:h + step, :n].float()
            t = torch.matmul(q, K.transpose(1, 2)).view(step, g, m, n) * s["scale"]
            p, total = _softmax_rows(torch.where(seen, t, torch.full_like(t, -math.inf)))
            y = torch.matmul(p.view(step, g * m, n), V).view(step, g, m, -1) / total
            s["out"][b, h * g:(h + step) * g, :m] = y.reshape(step * g, m, -1).to(s["out"].dtype)
    return s["out"]


def _plain_shared(c, s):
    B, h_kv, n, P, d = c["B"], c["h_kv"], c["n_max"], c["P"], c["d"]
    g = c["h_q"] // h_kv
    q = s["q"].float().view(B, h_kv, g, d) * s["scale"]
    first = torch.matmul(q.transpose(0, 1).reshape(h_kv, B * g, d), s["K_prefix"].float().transpose(1, 2))
    first = first.view(h_kv, B, g, P).transpose(0, 1)              # [B, h_kv, g, P]
    rest = torch.matmul(q, s["K"].float().transpose(2, 3))         # [B, h_kv, g, n]
    live = torch.arange(n, device=DEV)[None] < s["lens"][:, None]
    rest = torch.where(live[:, None, None], rest, torch.full_like(rest, -math.inf))
    p, total = _softmax_rows(torch.cat([first, rest], dim=-1))
    y = torch.matmul(p[..., :P].transpose(0, 1).reshape(h_kv, B * g, P), s["V_prefix"].float())
    y = y.view(h_kv, B, g, d).transpose(0, 1) + torch.matmul(p[..., P:], s["V"].float())
    s["out"].copy_((y / total).reshape(B, c["h_q"], d).to(s["out"].dtype))
    return s["out"]


# ------------------------------------------------------------------------------------------------- the framework's
def _run_own(s):
    import decode_attention_kv_split_gb300 as da
    c = s["case"]
    if c["op"] == "rope":
        q = da.kv_append_rope(s["q"], s["k_new"], s["v_new"], s["K"], s["V"], s["pos"], s["cos"], s["sin"],
                              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, n_new=s["new"],
                              angle_pos=s["angle_pos"], interleaved=c["interleaved"], q_out=s["q_out"])
        return {"q": q, "K": s["K"], "V": s["V"]}
    if c["op"] == "chunk":
        return da.chunk_attn(s["q"], s["K"], s["V"], s["lens"], n_new=s["new"], window=c["window"], prefix=c["prefix"],
                             out=s["out"], scale=s["scale"])
    return da.decode_attn_shared(s["q"], s["K_prefix"], s["V_prefix"], s["K"], s["V"], s["lens"], out=s["out"],
                                 scale=s["scale"])


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    return {"rope": _plain_rope, "chunk": _plain_chunk, "shared": _plain_shared}[c["op"]](c, state)


# ------------------------------------------------------------------------------------------------- in 64 bits
def _exact_head(x, weight, cos, sin, c):
    """One head's vectors x [m, d] with norm and rotation, angles [m, rot / 2], in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / x.shape[1] + EPS) * weight.double()
    y = x.clone()
    for j in range(c["rot"] // 2):
        i, k = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + c["rot"] // 2)
        y[:, i] = cos[:, j] * x[:, i] - sin[:, j] * x[:, k]
        y[:, k] = sin[:, j] * x[:, i] + cos[:, j] * x[:, k]
    return y


def _exact_rope(c, s):
    q_out, K, V = s["q_out"].double(), s["K"].double(), s["V"].double()
    for b, (n, m) in enumerate(zip(_lens(c), _news(c))):
        at = slice(n + c["shift"], n + c["shift"] + m)
        cos, sin = s["cos"][at].double(), s["sin"][at].double()
        # the heads of a sequence one under the other: each is rotated by its token's angle
        for x, w, h, to, rows in ((s["q"], s["q_weight"], c["h_q"], q_out, slice(0, m)),
                                  (s["k_new"], s["k_weight"], c["h_kv"], K, slice(n, n + m))):
            y = _exact_head(x[b, :, :m].reshape(h * m, -1), w, cos.repeat(h, 1), sin.repeat(h, 1), c)
            to[b, :, rows] = y.view(h, m, -1)
        V[b, :, n:n + m] = s["v_new"][b, :, :m].double()
    return {"q": q_out, "K": K, "V": V}


def _exact_attend(q, K, V, seen, scale):
    """Queries [m, d] over rows [n, d] in 64 bits; seen [m, n] or None."""
    x = (q.double() @ K.double().T) * scale
    if seen is not None:
        x[~seen] = -math.inf
    x -= x.max(1, keepdim=True).values
    x.exp_()
    return (x @ V.double()) / x.sum(1, keepdim=True)


def _exact_chunk(c, s):
    g, out = c["h_q"] // c["h_kv"], s["out"].double()
    for b, (n, m) in enumerate(zip(_lens(c), _news(c))):
        n += m
        for a in range(n - m, n, 2048):                            # queries at rows a .. z - 1
            z = min(n, a + 2048)
            at = torch.arange(a, z, device=DEV)[:, None]
            row = torch.arange(z, device=DEV)[None]
            seen = at >= row
            if c["window"]:
                seen &= (at - row < c["window"]) | (row < c["prefix"])
            for h in range(c["h_q"]):
                mine = slice(a - (n - m), z - (n - m))
                out[b, h, mine] = _exact_attend(s["q"][b, h, mine], s["K"][b, h // g, :z], s["V"][b, h // g, :z], seen,
                                                1 / math.sqrt(c["d"]))
    return out


def _exact_shared(c, s):
    g, out = c["h_q"] // c["h_kv"], s["out"].double()
    for h in range(c["h_kv"]):
        for b, n in enumerate(_lens(c)):
            K = torch.cat([s["K_prefix"][h], s["K"][b, h, :n]])
            V = torch.cat([s["V_prefix"][h], s["V"][b, h, :n]])
            out[b, h * g:h * g + g] = _exact_attend(s["q"][b, h * g:h * g + g], K, V, None, 1 / math.sqrt(c["d"]))
    return out


def exact(case, seed):
    if _scores(case) > 2 * LARGEST_SCORES or (case["op"] == "shared" and case["B"] * case["h_kv"] > 6000):
        return None  # would take too long
    s = prepare(case, seed)
    return {"rope": _exact_rope, "chunk": _exact_chunk, "shared": _exact_shared}[case["op"]](case, s)
