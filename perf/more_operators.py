"""What a prompt, or a later chunk of one, does around the paged latent cache: queries and keys normalised for each head
and rotated in the same pass, the latent normalised and appended in the cache's format, cached rows read back, and the
attention of many new tokens in its expanded form (192 dims a head for queries and keys, 128 for values).

Every case names its operator in "op". A plain run computes in elementary torch operations; where the module's `own`
is true, run() calls the library's entry points on the same state.
"""
import itertools
import math
import random

import torch

own = False

PAGE = 64            # tokens per cache page
ROPE = 64            # rotated dims
NOPE, VALUE = 128, 128  # dims of a head's key beside the rotated ones, and of its value
POSITIONS = 131072   # rows of the rotation table
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ROW_BYTES = {"bf16": 1152, "fp16": 1152, "fp8_656": 656, "fp8_528": 528, "fp4_288": 288}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the queries of a decode step: 64 tokens, 128 heads of 192; the rotated dims go into the decode's query, the
        # others to the absorption
        dict(name="norm rotate decode", op="norm_rotate", dtype="bf16", tokens=64, heads=128, dim=192, at=128, split=1,
             style=0),
        # the queries of a prompt chunk, odd length, halves rotated
        dict(name="norm rotate prompt", op="norm_rotate", dtype="fp16", tokens=4095, heads=128, dim=192, at=128, split=0,
             style=1),
        # the index keys of a long prompt: one head of 128, its first 64 dims rotated
        dict(name="norm rotate keys", op="norm_rotate", dtype="bf16", tokens=32768, heads=1, dim=128, at=0, split=0,
             style=0),
        # one new token for each of 64 running requests, bf16 cache
        dict(name="norm append decode", op="norm_append", cache="bf16", n=64, pad=0, run=1, style=0, rows=0),
        # the prompts of 8 requests of 4096 tokens into the 656-byte FP8 cache, with a padded tail; the prompt's own
        # attention reads the 16-bit rows
        dict(name="norm append prompt", op="norm_append", cache="fp8_656", n=32768, pad=19, run=4096, style=0, rows=1),
        # a short cached prefix of four requests
        dict(name="read bf16 short", op="read", cache="bf16", dtype="bf16", batch=4, length=700, spread=1, start=0),
        # the cached prefix of 16 long requests, for the next chunk of each
        dict(name="read fp8_656 long", op="read", cache="fp8_656", dtype="bf16", batch=16, length=16384, spread=0,
             start=0),
        # a part of longer prefixes in 4-bit rows, ragged
        dict(name="read fp4_288 part", op="read", cache="fp4_288", dtype="bf16", batch=8, length=16384, spread=1,
             start=4097),
        # eight running requests with four drafted tokens each: few rows over long keys
        dict(name="prefill drafted", op="prefill", dtype="bf16", batch=8, s_q=4, length=16384, spread=1, heads=16,
             causal=1, prefix=0),
        # packed documents of up to 2048 tokens whose first part sees itself whole, 16 heads
        dict(name="prefill documents", op="prefill", dtype="fp16", batch=24, s_q=2048, length=2048, spread=1, heads=16,
             causal=1, prefix=1),
        # a chunk of 2048 tokens behind a cached prefix
        dict(name="prefill chunk", op="prefill", dtype="bf16", batch=1, s_q=2048, length=32768, spread=0, heads=128,
             causal=1, prefix=0),
        # the first chunk of four prompts
        dict(name="prefill prompt", op="prefill", dtype="bf16", batch=4, s_q=4096, length=4096, spread=0, heads=128,
             causal=1, prefix=0),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rotate", "norm_append", "read", "prefill"])
    if op == "norm_rotate":
        dim = rng.choice([64, 128, 192, 256, 576, 8 * rng.randint(8, 72)])
        heads = rng.choice([1, 2, 16, 64, 128, rng.randint(1, 128)])
        split = rng.randint(0, 1) if dim > ROPE else 0
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), tokens=_log_int(rng, 1, min(32768, 4095 * 128 * 192 // (heads * dim))),
                    heads=heads, dim=dim, at=rng.choice([0, dim - ROPE, 8 * rng.randint(0, (dim - ROPE) // 8)]),
                    split=split, style=rng.randint(0, 1))
    if op == "norm_append":
        n = _log_int(rng, 1, 32768)
        return dict(op=op, cache=rng.choice(["bf16", "fp16", "fp8_656", "fp8_528", "fp4_288"]), n=n,
                    pad=rng.randint(0, n // 8), run=1 if n <= 256 and rng.random() < 0.5 else _log_int(rng, max(1, n // 256), n),
                    style=rng.randint(0, 1), rows=rng.randint(0, 1))
    if op == "read":
        cache = rng.choice(["bf16", "fp16", "fp8_656", "fp8_528", "fp4_288"])
        length = _log_int(rng, 1, 65536)
        return dict(op=op, cache=cache, dtype=cache if cache in DTYPES else rng.choice(["bf16", "fp16"]),
                    batch=_log_int(rng, 1, min(64, 2 ** 18 // length)), length=length, spread=rng.randint(0, 1),
                    start=rng.choice([0, _log_int(rng, 1, 16384)]))
    heads = rng.choice([1, 2, 16, 64, 128, rng.randint(1, 128)])
    length = _log_int(rng, 1, 32768)
    s_q = length if rng.random() < 0.4 else _log_int(rng, 1, 4096)
    s_q = min(s_q, 4096, 2 ** 32 // (length * heads))
    batch = _log_int(rng, 1, max(1, min(64, 2 ** 22 // (max(length, s_q) * heads), 2 ** 32 // (length * heads * s_q))))
    return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), batch=batch, s_q=s_q, length=length, spread=rng.randint(0, 1),
                heads=heads, causal=rng.randint(0, 1), prefix=rng.randint(0, 1))


def _lengths(case):
    """(queries, keys) of each request or document: (s_q, length) for all, or spread over [1 / 3, 1] of both with one
    that has all of them, one of a single token, and, where s_q is length, as many queries as keys."""
    rng = random.Random(7 * case["batch"] + case["length"])
    most_q, most_k = case.get("s_q", 1), case["length"]
    if not case["spread"]:
        return [(most_q, most_k)] * case["batch"]
    got = [(most_q, most_k)]
    for i in range(1, case["batch"]):
        k = 1 if i == 3 else rng.randint(max(1, most_k // 3), most_k)
        got.append((k if most_q == most_k else min(most_q, k), k))
    return got


def _prefixes(case):
    """Tokens at the start of each document that all of its queries see."""
    rng = random.Random(11 * case["batch"] + case["length"])
    return [rng.randint(0, max(1, k // 2)) for _, k in _lengths(case)]


def _pairs(case):
    """Visible (query, key) pairs."""
    total = 0
    for (n_q, n_k), prefix in zip(_lengths(case), _prefixes(case)):
        if not case["causal"]:
            total += n_q * n_k
            continue
        least = min(prefix, n_k) if case["prefix"] else 0
        total += sum(min(n_k, max(least, n_k - n_q + i + 1, 0)) for i in range(n_q))
    return total


def work(case):
    op = case["op"]
    if op == "norm_rotate":
        rows, d = case["tokens"] * case["heads"], case["dim"]
        return {"bytes": 4 * d * rows + case["tokens"] * 260 + 2 * d, "flops": rows * (4 * d + 6 * 32)}
    if op == "norm_append":
        n = case["n"] - case["pad"]
        latent = 448 if case["cache"] in ("fp8_528", "fp4_288") else 512
        wide = 2 * (latent + ROPE)
        return {"bytes": n * (wide * (1 + case["rows"]) + 256 + 8 + ROW_BYTES[case["cache"]]) + 2 * latent,
                "flops": n * (4 * latent + 6 * 32)}
    if op == "read":
        tokens = sum(k for _, k in _lengths(case))
        width = 512 if case["cache"] in ("fp8_528", "fp4_288") else 576
        return {"bytes": tokens * (ROW_BYTES[case["cache"]] + 2 * width) + tokens // 16, "flops": tokens * width}
    lengths, h = _lengths(case), case["heads"]
    n_q, n_k = sum(q for q, _ in lengths), sum(k for _, k in lengths)
    return {"bytes": n_q * h * (2 * (NOPE + ROPE + VALUE) + 4) + n_k * 2 * (h * (NOPE + VALUE) + ROPE),
            "flops": 2 * (NOPE + ROPE + VALUE) * h * _pairs(case)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _table():
    """Rotation table: cosines of the 32 angles of each position, then the sines."""
    inverse = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * inverse
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _gain(gen, dim, dtype):
    """Weights of a norm."""
    return (1.0 + 0.2 * _randn(gen, dim)).to(dtype)


def _projected(gen, dtype, *shape):
    """Rows as a projection gives them: each with a size of its own."""
    return (_randn(gen, *shape) * torch.exp2(_randn(gen, *shape[:-1], 1))).to(dtype)


def _new_tokens(case, gen):
    """Slots and positions of `n` new tokens, in runs of `run` consecutive ones (one request each); the last `pad`
    tokens are padding with slot -1."""
    n, run = case["n"], case["run"]
    runs = -(-n // run)
    span = -(-run // PAGE) + 1                       # pages that a run may touch
    pages = runs * span + 3
    table = torch.randperm(pages, generator=gen, device="cuda")[: runs * span].view(runs, span)
    first = torch.randint(0, POSITIONS - run + 1, (runs, 1), generator=gen, device="cuda")
    position = first + torch.arange(run, device="cuda")
    inside = first % PAGE + torch.arange(run, device="cuda")
    slot = table.gather(1, inside // PAGE) * PAGE + inside % PAGE
    slots, positions = slot.reshape(-1)[:n].int().contiguous(), position.reshape(-1)[:n].int().contiguous()
    if case["pad"]:
        slots[n - case["pad"]:] = -1
        positions[n - case["pad"]:] = 0
    return pages, slots, positions


def _packed(lengths):
    """Offsets [0, n_0, n_0 + n_1, ...]."""
    return torch.tensor([0, *itertools.accumulate(lengths)], dtype=torch.int32, device="cuda")


def _cached_rows(gen, kind, pages):
    """Pages of a cache in use."""
    if kind in DTYPES:
        return _randn(gen, pages, PAGE, 1, 576).to(DTYPES[kind])
    rows = pages * PAGE
    if kind == "fp8_656":
        codes, scale = _e4m3(_randn(gen, rows, 4, 128))
        parts = (codes.view(torch.uint8).flatten(1), scale.view(torch.uint8),
                 _randn(gen, rows, ROPE).to(torch.bfloat16).view(torch.uint8))
    elif kind == "fp8_528":
        codes, k = _ue8m0(_randn(gen, rows, 16, 32))
        parts = (codes.view(torch.uint8).flatten(1), (k + 127).to(torch.uint8).flatten(1))
    else:
        parts = _e2m1_bytes(_randn(gen, rows, 32, 16))
    return torch.cat(parts, 1).view(pages, PAGE, 1, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "norm_rotate":
        t, h, d, dtype = case["tokens"], case["heads"], case["dim"], DTYPES[case["dtype"]]
        st["x"] = _projected(gen, dtype, t, h, d)
        st["weight"] = _gain(gen, d, dtype)
        if case["split"]:      # the other dims for the absorption; the rotated ones into dims 512..575 of the query
            st["out"] = torch.empty(t, h, d - ROPE, dtype=dtype, device="cuda")
            st["rope_out"] = torch.zeros(t, h, 576, dtype=dtype, device="cuda")[..., 512:]
        else:
            st["out"], st["rope_out"] = torch.empty_like(st["x"]), None
        st["positions"] = torch.randint(0, POSITIONS, (t,), generator=gen, device="cuda").int()
        st["table"] = _table()
    elif op == "norm_append":
        dtype = DTYPES.get(case["cache"], torch.bfloat16)
        latent = 448 if case["cache"] in ("fp8_528", "fp4_288") else 512
        pages, st["slots"], st["positions"] = _new_tokens(case, gen)
        # the projection's output: latent and RoPE dims side by side
        kv = _projected(gen, dtype, case["n"], latent + ROPE)
        st["c_kv"], st["k_rope"] = kv[:, :latent], kv[:, latent:]
        st["weight"] = _gain(gen, latent, dtype)
        width = 576 if case["cache"] in DTYPES else ROW_BYTES[case["cache"]]
        st["kvcache"] = torch.zeros(pages, PAGE, 1, width, dtype=dtype if width == 576 else torch.uint8, device="cuda")
        st["out"] = torch.zeros(case["n"], latent + ROPE, dtype=dtype, device="cuda") if case["rows"] else None
        st["table"] = _table()
    elif op == "read":
        counts = [k for _, k in _lengths(case)]
        reach = -(-(case["start"] + case["length"]) // PAGE)
        pages = case["batch"] * reach
        st["block_table"] = torch.randperm(pages, generator=gen, device="cuda").int().view(case["batch"], reach)
        st["kvcache"] = _cached_rows(gen, case["cache"], pages)
        st["offsets"], st["total"] = _packed(counts), sum(counts)
        st["starts"] = torch.full((case["batch"],), case["start"], dtype=torch.int32, device="cuda")
    else:
        lengths, h, dtype = _lengths(case), case["heads"], DTYPES[case["dtype"]]
        n_q, n_k = sum(q for q, _ in lengths), sum(k for _, k in lengths)
        st["q"] = (1.5 * _randn(gen, n_q, h, NOPE + ROPE)).to(dtype)
        # keys and values of a head side by side, as their projection gives them; one rotated key for all heads
        kv = _randn(gen, n_k, h, NOPE + VALUE).to(dtype)
        st["k_nope"], st["v"] = kv[..., :NOPE], kv[..., NOPE:]
        st["k_rope"] = _randn(gen, n_k, ROPE).to(dtype)
        st["cu_q"], st["cu_k"] = _packed([q for q, _ in lengths]), _packed([k for _, k in lengths])
        st["prefix_lens"] = (torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None)
        st["scale"] = (NOPE + ROPE) ** -0.5
        st["most_q"], st["most_k"] = max(q for q, _ in lengths), max(k for _, k in lengths)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotated(x, cs, style):
    """x [..., 64] in fp32, cs [..., 64] the rotation's row; pairs (2i, 2i+1), or (i, i+32) with style 1."""
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., :32], x[..., 32:]) if style else (x[..., 0::2], x[..., 1::2])
    y = (a * c - b * s, a * s + b * c)
    return torch.cat(y, -1) if style else torch.stack(y, -1).flatten(-2)


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _e4m3(x):
    """Values held in e4m3 with one scale per row: (codes, scales)."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _ue8m0(x):
    """Values held in e4m3 with a power of two per row, the smallest 2^k, k >= -127, with 448 * 2^k >= amax."""
    fraction, exponent = torch.frexp(x.abs().amax(-1, keepdim=True))
    k = (exponent - 9 + (fraction > 0.875)).clamp(min=-127)
    k = torch.where(fraction == 0, torch.full_like(k, -127), k)
    return torch.ldexp(x, -k).clamp(-448, 448).to(torch.float8_e4m3fn), k


def _e2m1_bytes(x):
    """Blocks of 16 values [n, 32, 16] held in e2m1 with an e4m3 scale each, the smallest v with 6 v >= amax: (256
    bytes of pairs, 32 bytes of scales)."""
    codes = torch.arange(127, dtype=torch.uint8, device=x.device)
    values = codes.view(torch.float8_e4m3fn).float()
    amax = x.abs().amax(-1)
    code = torch.searchsorted(values * 6.0, amax.contiguous()).clamp(max=126)
    v = values[code].unsqueeze(-1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    odd = torch.tensor([False, True, False, True, False, True, False], device=x.device)
    a = x.abs()
    # the nearest magnitude, ties to the even code
    below = torch.searchsorted(mids, (a / v.clamp(min=2.0 ** -9)).contiguous())
    at = below.clamp(max=6)
    mid = mids[at] * v
    below = below + ((below < 7) & ((a > mid) | ((a == mid) & odd[at]))).int()
    last = (below - 1).clamp(min=0)
    under = mids[last] * v
    below = below - ((below > 0) & ((a < under) | ((a == under) & ~odd[last]))).int()
    nibble = torch.where(v == 0, torch.zeros_like(below), below).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
    flat = nibble.flatten(1)
    return flat[:, 0::2] | (flat[:, 1::2] << 4), code.to(torch.uint8)


def _values(rows, kind):
    """What quantised rows of a cache hold, fp32: [n, 576], or [n, 512] of the 528- and 288-byte rows."""
    if kind == "fp8_656":
        latent = rows[:, :512].view(torch.float8_e4m3fn).float().unflatten(1, (4, 128)) * rows[:, 512:528].view(torch.float32)[..., None]
        return torch.cat((latent.flatten(1), rows[:, 528:].view(torch.bfloat16).float()), 1)
    if kind == "fp8_528":
        x = rows[:, :512].view(torch.float8_e4m3fn).float().unflatten(1, (16, 32))
        return torch.ldexp(x, rows[:, 512:, None].int() - 127).flatten(1)
    magnitude = torch.tensor(E2M1, device=rows.device)
    nibbles = torch.stack((rows[:, :256] & 15, rows[:, :256] >> 4), -1).flatten(1).int()
    x = magnitude[nibbles & 7] * (1 - 2 * (nibbles >> 3))
    return (x.unflatten(1, (32, 16)) * rows[:, 256:].contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(1)


def _rows_out(cache, kind):
    """A cache as what it holds: e4m3 values, scales and the RoPE dims of 656-byte rows, the values of 528- and
    288-byte rows."""
    rows = cache.view(-1, cache.shape[-1])
    if kind == "fp8_656":
        return {"latent": rows[:, :512].view(torch.float8_e4m3fn), "scale": rows[:, 512:528].view(torch.float32),
                "rope": rows[:, 528:].view(torch.bfloat16)}
    if kind in DTYPES:
        return {"rows": cache}
    return {"values": _values(rows, kind).to(torch.bfloat16)}     # at most 7 bits each: exact


def _plain_norm_rotate(st):
    at = st["at"]
    y = _normed(st["x"], st["weight"])
    turned = _rotated(y[..., at:at + ROPE], st["table"][st["positions"].long()][:, None], st["style"])
    if st["split"]:
        st["out"].copy_(torch.cat((y[..., :at], y[..., at + ROPE:]), -1))
        st["rope_out"].copy_(turned)
        return st["out"], st["rope_out"]
    st["out"].copy_(torch.cat((y[..., :at], turned, y[..., at + ROPE:]), -1))
    return st["out"]


def _plain_norm_append(st):
    n, kind = st["n"] - st["pad"], st["cache"]
    slots = st["slots"][:n].long()
    latent = _normed(st["c_kv"][:n], st["weight"])
    rope = _rotated(st["k_rope"][:n].float(), st["table"][st["positions"][:n].long()], st["style"])
    cache = st["kvcache"]
    both = torch.cat((latent, rope), 1)
    if kind == "fp8_656":
        codes, scale = _e4m3(latent.view(n, 4, 128))
        rows = torch.cat((codes.view(torch.uint8).flatten(1), scale.view(torch.uint8),
                          rope.to(torch.bfloat16).view(torch.uint8)), 1)
    elif kind == "fp8_528":
        codes, k = _ue8m0(both.view(n, 16, 32))
        rows = torch.cat((codes.view(torch.uint8).flatten(1), (k + 127).to(torch.uint8).flatten(1)), 1)
    elif kind == "fp4_288":
        rows = torch.cat(_e2m1_bytes(both.view(n, 32, 16)), 1)
    else:
        rows = both.to(cache.dtype)
    cache.view(-1, cache.shape[-1])[slots] = rows
    if st["out"] is None:
        return _rows_out(cache, kind)
    st["out"][:n] = both.to(st["out"].dtype)
    return _rows_out(cache, kind), st["out"]


def _plain_read(st):
    offsets = st["offsets"].long()
    row = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(offsets, row, right=True) - 1
    token = row - offsets[b] + st["starts"][b].long()
    at = st["block_table"][b, token // PAGE].long() * PAGE + token % PAGE
    rows = st["kvcache"].view(-1, st["kvcache"].shape[-1])[at]
    return rows if st["cache"] in DTYPES else _values(rows, st["cache"]).to(DTYPES[st["dtype"]])


def _plain_prefill(st):
    h, most_q, most_k = st["heads"], st["most_q"], st["most_k"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    n_q, n_k = cu_q.diff()[:, None], cu_k.diff()[:, None]
    i, j = torch.arange(most_q, device="cuda"), torch.arange(most_k, device="cuda")
    # every document padded to the longest: [batch, heads, tokens, dim]
    row_q, row_k = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1), (cu_k[:-1, None] + j).clamp(max=st["v"].shape[0] - 1)
    q = st["q"][row_q].transpose(1, 2).float()
    k_rope = st["k_rope"][row_k].float()
    k = torch.cat((st["k_nope"][row_k].float(), k_rope[:, :, None].expand(-1, -1, h, -1)), -1).transpose(1, 2)
    seen = n_k.expand(-1, most_q)
    if st["causal"]:
        seen = n_k - n_q + i + 1
        if st["prefix_lens"] is not None:
            seen = torch.maximum(seen, st["prefix_lens"].long()[:, None])
        seen = torch.minimum(seen.clamp(min=0), n_k)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"])
    s.masked_fill_((j >= seen[..., None])[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, st["v"][row_k].transpose(1, 2).float()) / total.clamp(min=1e-38)
    lse = top + total.log()
    # back to packed rows
    of = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu_q, of, right=True) - 1
    at = of - cu_q[b]
    return out[b, :, at].to(st["q"].dtype), lse[b, :, at, 0]


_PLAIN = {"norm_rotate": _plain_norm_rotate, "norm_append": _plain_norm_append, "read": _plain_read,
          "prefill": _plain_prefill}


def _call(st):
    import mla_latent_kv_14_gb300 as mla
    op = st["op"]
    formats = {"fp8_656": mla.KV_FP8_656, "fp8_528": mla.KV_FP8_528, "fp4_288": mla.KV_FP4_288}
    if op == "norm_rotate":
        return mla.mla_norm_rotate(st["x"], st["positions"], st["table"], weight=st["weight"], eps=EPS, rope_at=st["at"],
                                   out=st["out"], rope_out=st["rope_out"], rope_style=st["style"])
    if op == "norm_append":
        mla.mla_norm_append_kv(st["c_kv"], st["k_rope"], st["weight"], st["kvcache"], st["slots"], st["positions"],
                               st["table"], eps=EPS, kv_format=formats.get(st["cache"], mla.KV_16BIT),
                               rope_style=st["style"], rows=st["out"])
        cache = _rows_out(st["kvcache"], st["cache"])
        return cache if st["out"] is None else (cache, st["out"])
    if op == "read":
        return mla.mla_read_kv(st["kvcache"], st["block_table"], st["offsets"], total=st["total"], starts=st["starts"],
                               kv_format=formats.get(st["cache"], mla.KV_16BIT), dtype=DTYPES[st["dtype"]])
    return mla.mla_prefill(st["q"], st["k_nope"], st["k_rope"], st["v"], st["cu_q"], st["cu_k"], st["scale"],
                           causal=bool(st["causal"]), prefix_lens=st["prefix_lens"])


def run(state):
    return _call(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(x, row, style):
    """Each pair as a complex number, times cos + i sin."""
    pair = x.unflatten(-1, (2, 32)).movedim(-2, -1) if style else x.unflatten(-1, (32, 2))
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.complex(row[..., :32].double(), row[..., 32:].double()))
    return turned.movedim(-1, -2).flatten(-2) if style else turned.flatten(-2)


def _exact_norm(x, weight):
    x = x.double()
    return weight.double() * x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS).sqrt()


def _e4m3_grid():
    """The values that e4m3 holds, from 0 to 448, by its definition: 2^-9 steps up to 2^-6, then eighths of a power of two."""
    low = torch.arange(8, dtype=torch.float64, device="cuda") * 2.0 ** -9
    high = torch.exp2(torch.arange(-6, 9, dtype=torch.float64, device="cuda"))[:, None] * (1 + torch.arange(8, device="cuda") / 8)
    return torch.cat((low, high.flatten()))[:127]


def _nearest(x, grid):
    """x rounded to the nearest of the grid's values, and of their negatives."""
    return torch.copysign(grid[torch.searchsorted((grid[1:] + grid[:-1]) / 2, x.abs())], x)


def _exact_norm_append(case, st):
    n, cache, kind = case["n"] - case["pad"], st["kvcache"], case["cache"]
    slots, row = st["slots"][:n].long(), st["table"][st["positions"][:n].long()]

    def placed(rows, where, values):
        return torch.zeros(rows, values.shape[1], dtype=torch.float64, device="cuda").index_copy_(0, where, values)

    count = cache.shape[0] * PAGE
    latent = _exact_norm(st["c_kv"][:n], st["weight"])
    rope = _exact_rope(st["k_rope"][:n].double(), row, case["style"])
    both = torch.cat((latent, rope), 1)
    if kind == "fp8_656":
        scale = latent.unflatten(1, (4, 128)).abs().amax(-1) / 448.0
        codes = (latent.unflatten(1, (4, 128)) / scale[..., None]).flatten(1)
        held = {"latent": placed(count, slots, codes), "scale": placed(count, slots, scale), "rope": placed(count, slots, rope)}
    elif kind in DTYPES:
        held = {"rows": placed(count, slots, both).view(cache.shape)}
    elif kind == "fp8_528":
        x = both.unflatten(1, (16, 32))
        unit = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448.0)))
        held = {"values": placed(count, slots, (_nearest(x / unit, _e4m3_grid()) * unit).flatten(1))}
    else:
        x, units = both.unflatten(1, (32, 16)), _e4m3_grid()
        unit = units[torch.searchsorted(units, x.abs().amax(-1, keepdim=True) / 6.0).clamp(max=126)]
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        held = {"values": placed(count, slots, (_nearest(x / unit, grid) * unit).flatten(1))}
    if not case["rows"]:
        return held
    return held, placed(case["n"], torch.arange(n, device="cuda"), both)


def _exact_read(case, st):
    bits = {"fp8_656": 512, "fp8_528": 512, "fp4_288": 256}.get(case["cache"])
    magnitude = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = []
    for i, (_, count) in enumerate(_lengths(case)):
        page = st["kvcache"][st["block_table"][i].long()].flatten(0, 2)[case["start"]: case["start"] + count]
        if bits is None:
            out.append(page.double())
            continue
        data, scale = page[:, :bits].contiguous(), page[:, bits:].contiguous()
        if case["cache"] == "fp8_656":
            factor = scale[:, :16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
            x = data.view(torch.float8_e4m3fn).double() * factor
            out.append(torch.cat((x, scale[:, 16:].contiguous().view(torch.bfloat16).double()), 1))
        elif case["cache"] == "fp8_528":
            out.append(data.view(torch.float8_e4m3fn).double() * torch.exp2(scale.double() - 127).repeat_interleave(32, 1))
        else:
            x = torch.empty(count, 512, dtype=torch.float64, device="cuda")
            for k in range(2):
                nibble = (data >> (4 * k)) % 16
                x[:, k::2] = torch.where(nibble > 7, -magnitude[(nibble % 8).long()], magnitude[(nibble % 8).long()])
            out.append(x * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1))
    return torch.cat(out)


def _exact_prefill(case, st):
    out, lse = [], []
    first_q = first_k = 0
    for (n_q, n_k), prefix in zip(_lengths(case), _prefixes(case)):
        q = st["q"][first_q: first_q + n_q].double()
        k, v, rope = (st[name][first_k: first_k + n_k] for name in ("k_nope", "v", "k_rope"))
        o = torch.zeros(n_q, case["heads"], VALUE, dtype=torch.float64, device="cuda")
        ls = torch.full((n_q, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
        position = torch.arange(n_q, device="cuda")[:, None] + (n_k - n_q)     # of a query among the keys
        key = torch.arange(n_k, device="cuda")
        hidden = (key > position) if case["causal"] else torch.zeros(n_q, n_k, dtype=torch.bool, device="cuda")
        if case["causal"] and case["prefix"]:
            hidden = hidden & (key >= prefix)
        some = ~hidden.all(1)
        for h in range(case["heads"]):
            s = (q[:, h, :NOPE] @ k[:, h].double().T + q[:, h, NOPE:] @ rope.double().T) * st["scale"]
            s.masked_fill_(hidden, -math.inf)
            ls[:, h] = torch.logsumexp(s, 1)
            o[some, h] = torch.softmax(s[some], 1) @ v[:, h].double()
        out.append(o)
        lse.append(ls)
        first_q, first_k = first_q + n_q, first_k + n_k
    return torch.cat(out), torch.cat(lse)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rotate":
        at = case["at"]
        y = _exact_norm(st["x"], st["weight"])
        turned = _exact_rope(y[..., at:at + ROPE], st["table"][st["positions"].long()][:, None], case["style"])
        if case["split"]:
            return torch.cat((y[..., :at], y[..., at + ROPE:]), -1), turned
        return torch.cat((y[..., :at], turned, y[..., at + ROPE:]), -1)
    if op == "norm_append":
        return _exact_norm_append(case, st)
    return _exact_read(case, st) if op == "read" else _exact_prefill(case, st)
