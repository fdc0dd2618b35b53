"""What a serving step does around MLA decode: new tokens rotated and appended to the paged caches, queries rotated,
cached tokens scored by a cheap index, and the best of them selected for the sparse attention.

Every case names its operator in "op". A plain run computes in elementary torch operations; where the module's `own`
is true, run() calls the library's entry points on the same state.
"""
import math
import random

import torch

own = False

PAGE = 64          # tokens per cache page
LATENT = 512       # latent dims of a 576-wide cache row; 448 of a 528-byte row, whose 512 values hold the RoPE dims too
ROPE = 64
INDEX_DIM = 128    # width of an index query or key
POSITIONS = 131072  # rows of the rotation table
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 64 running requests, bf16 cache: a decode step, where latency counts
        dict(name="append bf16 decode", op="append", cache="bf16", n=64, pad=0, run=1, style=0),
        # the prompts of 8 requests of 4096 tokens, into the 656-byte FP8 cache, with a padded tail
        dict(name="append fp8_656 prompt", op="append", cache="fp8_656", n=32768, pad=19, run=4096, style=0),
        # the query of a decode step: 64 tokens, 128 heads, a slice of the projection's 192 dims into dims 512..575
        dict(name="rotate decode", op="rotate", dtype="bf16", tokens=64, heads=128, style=0, wide=1),
        # the query of a prompt chunk, odd length, halves rotated
        dict(name="rotate prompt", op="rotate", dtype="fp16", tokens=4095, heads=128, style=1, wide=1),
        # one new index key for each of 32 running requests
        dict(name="index key decode", op="index_k", cache="bf16", dtype="bf16", n=32, pad=0, run=1, style=0),
        # index queries of a prompt chunk: 64 heads, e4m3 with the scale folded into the weights
        dict(name="index query prompt", op="index_q", dtype="bf16", tokens=4096, heads=64, style=0),
        # scores of a decode step over long caches: 32 requests of up to 131072 tokens, e4m3 keys
        dict(name="score fp8 decode", op="score", keys="fp8", batch=32, s_q=1, length=131072, spread=0, heads=64,
             causal=0, block=1),
        # two tokens a request (one drafted), ragged lengths, page scores
        dict(name="score bf16 pages", op="score", keys="bf16", batch=16, s_q=2, length=12288, spread=1, heads=32,
             causal=1, block=64),
        # scores of a prompt chunk of 1024 tokens a request
        dict(name="score bf16 prompt", op="score", keys="bf16", batch=4, s_q=1024, length=16384, spread=0, heads=64,
             causal=1, block=1),
        # the index lists of a decode step over long caches
        dict(name="select decode", op="select", batch=32, s_q=1, length=131072, spread=0, causal=0, block=1,
             topk=2048),
        # the page lists of a decode step, ragged lengths
        dict(name="select pages", op="select", batch=64, s_q=1, length=32768, spread=1, causal=0, block=64, topk=64),
        # the index lists of a prompt chunk
        dict(name="select prompt", op="select", batch=4, s_q=1024, length=16384, spread=0, causal=1, block=1,
             topk=2048),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "rotate", "index_k", "index_q", "score", "select"])
    if op in ("append", "index_k"):
        n = _log_int(rng, 1, 32768)
        case = dict(op=op, n=n, pad=rng.randint(0, n // 8), run=1 if n <= 256 and rng.random() < 0.5 else _log_int(rng, max(1, n // 256), n),
                    style=rng.randint(0, 1))
        if op == "append":
            return dict(case, cache=rng.choice(["bf16", "fp16", "fp8_656", "fp8_528"]))
        dtype = rng.choice(["bf16", "fp16"])
        return dict(case, dtype=dtype, cache=rng.choice([dtype, "fp8"]))
    if op == "rotate":
        heads = rng.choice([1, 2, 16, 64, 128, rng.randint(1, 128)])
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), tokens=_log_int(rng, 1, 4095 * 128 // heads // 2),
                    heads=heads, style=rng.randint(0, 1), wide=rng.randint(0, 1))
    if op == "index_q":
        heads = rng.choice([16, 32, 64, rng.randint(1, 64)])
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), tokens=_log_int(rng, 1, 4096), heads=heads,
                    style=rng.randint(0, 1))
    causal = rng.randint(0, 1)
    s_q = 1 if rng.random() < 0.4 else _log_int(rng, 2, 1024)
    length = _log_int(rng, max(64, s_q), 131072)
    # (query, token) pairs of the listed prompt chunk at most, and its keys at most
    batch = _log_int(rng, 1, max(1, min(64, 2 ** 22 // length, 2 ** 26 // (length * s_q))))
    case = dict(op=op, batch=batch, s_q=s_q, length=length, spread=rng.randint(0, 1), causal=causal,
                block=rng.choice([1, 64]))
    if op == "score":
        return dict(case, keys=rng.choice(["bf16", "fp16", "fp8"]), heads=rng.choice([16, 32, 64, rng.randint(1, 64)]))
    pages = -(-length // PAGE)
    return dict(case, topk=_log_int(rng, 1, 32768) if case["block"] == 1 else _log_int(rng, 1, max(2, pages)))


def _lengths(case):
    """Tokens cached of each request: all `length`, or spread over [length / 3, length], one of them `length`."""
    rng = random.Random(7 * case["batch"] + case["length"])
    if not case["spread"]:
        return [case["length"]] * case["batch"]
    low = max(case["s_q"], case["length"] // 3)
    return [case["length"]] + [rng.randint(min(low, case["length"]), case["length"]) for _ in range(case["batch"] - 1)]


def _pairs(case):
    """Visible (query, token) pairs."""
    hidden = case["s_q"] * (case["s_q"] - 1) // 2 if case["causal"] else 0
    return sum(length * case["s_q"] - hidden for length in _lengths(case))


def work(case):
    op = case["op"]
    if op == "append":
        n = case["n"] - case["pad"]
        latent = 448 if case["cache"] == "fp8_528" else 512
        row = {"bf16": 1152, "fp16": 1152, "fp8_656": 656, "fp8_528": 528}[case["cache"]]
        # latent and RoPE dims, the rotation's row, slot and position in; the cache row out
        return {"bytes": n * (2 * latent + 128 + 256 + 8 + row), "flops": 6 * 32 * n}
    if op == "rotate":
        return {"bytes": case["tokens"] * (case["heads"] * 256 + 260), "flops": 6 * 32 * case["tokens"] * case["heads"]}
    if op == "index_k":
        n = case["n"] - case["pad"]
        return {"bytes": n * (256 + 256 + 8 + (132 if case["cache"] == "fp8" else 256)), "flops": 6 * 32 * n}
    if op == "index_q":
        rows = case["tokens"] * case["heads"]
        return {"bytes": rows * (256 + 4 + 128 + 4) + case["tokens"] * 260, "flops": rows * (6 * 32 + 2 * 128)}
    tokens, queries = sum(_lengths(case)), case["batch"] * case["s_q"]
    width = -(-case["length"] // case["block"])
    if op == "score":
        key, q = (132, 128) if case["keys"] == "fp8" else (256, 256)
        return {"bytes": tokens * key + queries * case["heads"] * (q + 4) + 4 * queries * width,
                "flops": _pairs(case) * case["heads"] * (2 * INDEX_DIM + 3)}
    return {"bytes": 4 * _pairs(case) // case["block"] + 4 * queries * (case["topk"] + 1), "flops": _pairs(case) // case["block"]}


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


def _e4m3(x):
    """Values held in e4m3 with one scale per row: (codes, scales)."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _paged(case, gen):
    lengths = _lengths(case)
    most = -(-case["length"] // PAGE)
    pages = case["batch"] * most
    table = torch.randperm(pages, generator=gen, device="cuda").int().view(case["batch"], most)
    return pages, table, torch.tensor(lengths, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "append":
        dtype = DTYPES.get(case["cache"], torch.bfloat16)
        latent = 448 if case["cache"] == "fp8_528" else 512
        pages, st["slots"], st["positions"] = _new_tokens(case, gen)
        # the projection's output: latent and RoPE dims side by side
        kv = _randn(gen, case["n"], latent + ROPE).to(dtype)
        st["c_kv"], st["k_rope"] = kv[:, :latent], kv[:, latent:]
        width = {"fp8_656": 656, "fp8_528": 528}.get(case["cache"], 576)
        st["kvcache"] = torch.zeros(pages, PAGE, 1, width, dtype=dtype if width == 576 else torch.uint8, device="cuda")
        st["table"] = _table()
    elif op == "rotate":
        t, h, dtype = case["tokens"], case["heads"], DTYPES[case["dtype"]]
        # the RoPE slice of a 192-wide projection, into dims 512..575 of the decode's query; or dense rows in place
        x = _randn(gen, t, h, 192 if case["wide"] else ROPE).to(dtype)
        st["x"] = x[..., 128:] if case["wide"] else x
        st["out"] = (torch.zeros(t, h, 576, dtype=dtype, device="cuda")[..., 512:] if case["wide"]
                     else torch.empty_like(x))
        st["positions"] = torch.randint(0, POSITIONS, (t,), generator=gen, device="cuda").int()
        st["table"] = _table()
    elif op == "index_k":
        pages, st["slots"], st["positions"] = _new_tokens(case, gen)
        st["k"] = _randn(gen, case["n"], INDEX_DIM).to(DTYPES[case["dtype"]])
        st["index_cache"] = (torch.zeros(pages, PAGE * (INDEX_DIM + 4), dtype=torch.uint8, device="cuda")
                             if case["cache"] == "fp8" else
                             torch.zeros(pages, PAGE, 1, INDEX_DIM, dtype=DTYPES[case["dtype"]], device="cuda"))
        st["table"] = _table()
    elif op == "index_q":
        t, h = case["tokens"], case["heads"]
        st["q"] = _randn(gen, t, h, INDEX_DIM).to(DTYPES[case["dtype"]])
        st["weights"] = _randn(gen, t, h) * (h * INDEX_DIM) ** -0.5
        st["positions"] = torch.randint(0, POSITIONS, (t,), generator=gen, device="cuda").int()
        st["table"] = _table()
    elif op == "score":
        b, s, h = case["batch"], case["s_q"], case["heads"]
        pages, st["block_table"], st["seqlens"] = _paged(case, gen)
        q, k = _randn(gen, b, s, h, INDEX_DIM), _randn(gen, pages, PAGE, INDEX_DIM)
        st["weights"] = _randn(gen, b, s, h) * (h * INDEX_DIM) ** -0.5
        if case["keys"] == "fp8":
            st["q"], scale = _e4m3(q)
            st["weights"] = st["weights"] * scale
            codes, scale = _e4m3(k)
            # a page: 64 rows of codes, then their 64 scales
            st["index_cache"] = torch.cat((codes.view(torch.uint8).flatten(1), scale.view(torch.uint8)), 1)
        else:
            st["q"] = q.to(DTYPES[case["keys"]])
            st["index_cache"] = k.to(DTYPES[case["keys"]]).unsqueeze(2)
    else:
        b, s = case["batch"], case["s_q"]
        st["pages"], st["block_table"], st["seqlens"] = _paged(case, gen)
        width = -(-case["length"] // case["block"])
        # scores as the index gives them: a few heads' positive parts, weighted; some are exactly zero
        scores = torch.zeros(b, s, width, device="cuda")
        for _ in range(3):
            scores += _randn(gen, b, s, width).clamp_(min=0) * _randn(gen, b, s, 1).abs()
        seen = _visible(st["seqlens"], s, case["causal"])
        at = torch.arange(width, dtype=torch.int32, device="cuda") * case["block"]
        st["scores"] = scores.masked_fill_(at >= seen[..., None], -math.inf)
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


def _visible(seqlens, s_q, causal):
    """Tokens that each query sees, [batch, s_q]; causal: the last query sees all, each before it one fewer."""
    behind = torch.arange(s_q - 1, -1, -1, dtype=torch.int32, device="cuda") if causal else torch.zeros(s_q, dtype=torch.int32, device="cuda")
    return (seqlens[:, None] - behind).clamp(min=0)


def _rows_out(cache, kind):
    """A cache as what it holds: codes as e4m3 values, scales, and the RoPE dims."""
    if kind == "fp8_656":
        rows = cache.view(-1, 656)
        return {"latent": rows[:, :512].view(torch.float8_e4m3fn), "scale": rows[:, 512:528].view(torch.float32),
                "rope": rows[:, 528:].view(torch.bfloat16)}
    if kind == "fp8_528":
        rows = cache.view(-1, 528)
        return {"values": rows[:, :512].view(torch.float8_e4m3fn), "exponent": rows[:, 512:]}
    if kind == "fp8":
        codes = cache[:, : PAGE * INDEX_DIM]
        return {"key": codes.view(torch.float8_e4m3fn), "scale": cache[:, PAGE * INDEX_DIM:].view(torch.float32)}
    return {"rows": cache}


def _plain_append(st):
    n, kind = st["n"] - st["pad"], st["cache"]
    slots = st["slots"][:n].long()
    latent = st["c_kv"][:n].float()
    rope = _rotated(st["k_rope"][:n].float(), st["table"][st["positions"][:n].long()], st["style"])
    cache = st["kvcache"]
    if kind == "fp8_656":
        codes, scale = _e4m3(latent.view(n, 4, 128))
        rows = torch.cat((codes.view(torch.uint8).flatten(1), scale.view(torch.uint8),
                          rope.to(torch.bfloat16).view(torch.uint8)), 1)
    elif kind == "fp8_528":
        x = torch.cat((latent, rope), 1).view(n, 16, 32)
        # the smallest power of two 2^k, k >= -127, with 448 * 2^k >= amax
        fraction, exponent = torch.frexp(x.abs().amax(-1, keepdim=True))
        k = (exponent - 9 + (fraction > 0.875)).clamp(min=-127)
        k = torch.where(fraction == 0, torch.full_like(k, -127), k)
        codes = torch.ldexp(x, -k).clamp(-448, 448).to(torch.float8_e4m3fn)
        rows = torch.cat((codes.view(torch.uint8).flatten(1), (k + 127).to(torch.uint8).flatten(1)), 1)
    else:
        rows = torch.cat((latent, rope), 1).to(cache.dtype)
    cache.view(-1, cache.shape[-1])[slots] = rows
    return _rows_out(cache, kind)


def _plain_rotate(st):
    st["out"].copy_(_rotated(st["x"].float(), st["table"][st["positions"].long()][:, None], st["style"]))
    return st["out"]


def _index_rows(x, cs, style):
    x = x.float()
    return torch.cat((_rotated(x[..., :ROPE], cs, style), x[..., ROPE:]), -1)


def _plain_index_k(st):
    n, cache = st["n"] - st["pad"], st["index_cache"]
    slots = st["slots"][:n].long()
    rows = _index_rows(st["k"][:n], st["table"][st["positions"][:n].long()], st["style"])
    if st["cache"] == "fp8":
        codes, scale = _e4m3(rows)
        page, at = slots // PAGE, slots % PAGE
        cache[:, : PAGE * INDEX_DIM].view(-1, PAGE, INDEX_DIM)[page, at] = codes.view(torch.uint8)
        cache[:, PAGE * INDEX_DIM:].view(torch.float32)[page, at] = scale
    else:
        cache.view(-1, INDEX_DIM)[slots] = rows.to(cache.dtype)
    return _rows_out(cache, st["cache"])


def _plain_index_q(st):
    codes, scale = _e4m3(_index_rows(st["q"], st["table"][st["positions"].long()][:, None], st["style"]))
    return codes, st["weights"] * scale


def _plain_score(st):
    b, s, h, block = st["batch"], st["s_q"], st["heads"], st["block"]
    table, cache, length = st["block_table"].long(), st["index_cache"], st["length"]
    if st["keys"] == "fp8":
        keys = cache[:, : PAGE * INDEX_DIM].view(torch.float8_e4m3fn).float().view(-1, PAGE, INDEX_DIM)[table]
        scale = cache[:, PAGE * INDEX_DIM:].view(torch.float32)[table].view(b, 1, -1)
    else:
        keys, scale = cache[table].float(), None
    keys = keys.view(b, -1, INDEX_DIM)
    dots = torch.matmul(st["q"].float().view(b, s * h, INDEX_DIM), keys.transpose(1, 2)).clamp_(min=0)
    scores = dots.view(b, s, h, -1).mul_(st["weights"][..., None]).sum(2)
    if scale is not None:
        scores = scores * scale
    seen = _visible(st["seqlens"], s, st["causal"])
    scores = scores.masked_fill(torch.arange(scores.shape[-1], device="cuda") >= seen[..., None], -math.inf)
    return scores[..., :length] if block == 1 else scores.view(b, s, -1, PAGE).amax(-1)


def _plain_select(st):
    b, s, block, k = st["batch"], st["s_q"], st["block"], st["topk"]
    scores, table = st["scores"], st["block_table"]
    width = scores.shape[-1]
    seen = _visible(st["seqlens"], s, st["causal"])
    units = (seen + (block - 1)) // block                # visible tokens or pages
    at = torch.arange(width, dtype=torch.int32, device="cuda")
    if block > 1:                                        # the last visible page always takes part
        scores = scores.masked_fill(at == units[..., None] - 1, math.inf)
    # stable: equal scores stay in the order of their positions
    order = torch.sort(scores, dim=-1, descending=True, stable=True).indices[..., :k]
    count = units.clamp(max=k)
    rank = torch.arange(order.shape[-1], device="cuda")
    chosen = torch.where(rank < count[..., None], order, width).sort(-1).values
    page = (chosen if block > 1 else chosen // PAGE).clamp(max=table.shape[1] - 1)
    page = table[:, None].expand(b, s, -1).gather(2, page)
    found = page if block > 1 else page * PAGE + (chosen % PAGE).int()
    found = torch.where(chosen < width, found, -1).int()
    found = torch.nn.functional.pad(found, (0, k - found.shape[-1]), value=-1)
    lens = count if block == 1 else torch.where(count > 0, (count - 1) * block + seen - (units - 1) * block, 0)
    return found, lens.int()


_PLAIN = {"append": _plain_append, "rotate": _plain_rotate, "index_k": _plain_index_k, "index_q": _plain_index_q,
          "score": _plain_score, "select": _plain_select}


def _call(st):
    import mla_latent_kv_14_gb300 as mla
    op = st["op"]
    if op == "append":
        fmt = {"fp8_656": mla.KV_FP8_656, "fp8_528": mla.KV_FP8_528}.get(st["cache"], mla.KV_16BIT)
        mla.mla_append_kv(st["c_kv"], st["k_rope"], st["kvcache"], st["slots"], st["positions"], st["table"],
                          kv_format=fmt, rope_style=st["style"])
        return _rows_out(st["kvcache"], st["cache"])
    if op == "rotate":
        return mla.mla_rotate_q(st["x"], st["positions"], st["table"], out=st["out"], rope_style=st["style"])
    if op == "index_k":
        fmt = mla.INDEX_FP8 if st["cache"] == "fp8" else mla.INDEX_16BIT
        mla.mla_append_index_k(st["k"], st["index_cache"], st["slots"], st["positions"], st["table"],
                               index_format=fmt, rope_style=st["style"])
        return _rows_out(st["index_cache"], st["cache"])
    if op == "index_q":
        return mla.mla_quantize_index_q(st["q"], st["weights"], st["positions"], st["table"], rope_style=st["style"])
    if op == "score":
        fmt = mla.INDEX_FP8 if st["keys"] == "fp8" else mla.INDEX_16BIT
        return mla.mla_index_score(st["q"], st["weights"], st["index_cache"], st["block_table"], st["seqlens"],
                                   width=-(-st["length"] // st["block"]), causal=bool(st["causal"]), block=st["block"],
                                   index_format=fmt)
    return mla.mla_select_topk(st["scores"], st["seqlens"], st["topk"], st["block_table"], st["pages"],
                               causal=bool(st["causal"]), block=st["block"])


def run(state):
    return _call(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(x, row, style):
    """Each pair as a complex number, times cos + i sin."""
    x = x.double()
    pair = x.unflatten(-1, (2, 32)).movedim(-2, -1) if style else x.unflatten(-1, (32, 2))
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.complex(row[..., :32].double(), row[..., 32:].double()))
    return turned.movedim(-1, -2).flatten(-2) if style else turned.flatten(-2)


def _exact_scaled(x):
    """x in units of a scale that takes its largest magnitude to 448, and the scale."""
    scale = x.abs().amax(-1, keepdim=True) / 448.0
    scale = scale.masked_fill(scale == 0, 1.0)
    return x / scale, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("append", "index_k"):
        n = case["n"] - case["pad"]
        slots, row = st["slots"][:n].long(), st["table"][st["positions"][:n].long()]
    if op == "append":
        cache, kind = st["kvcache"], case["cache"]
        rows = cache.shape[0] * PAGE

        def placed(width, values):
            return torch.zeros(rows, width, dtype=torch.float64, device="cuda").index_copy_(0, slots, values)

        latent, rope = st["c_kv"][:n].double(), _exact_rope(st["k_rope"][:n], row, case["style"])
        if kind == "fp8_656":
            codes, scale = _exact_scaled(latent.unflatten(-1, (4, 128)))
            return {"latent": placed(512, codes.flatten(1)), "scale": placed(4, scale.flatten(1)),
                    "rope": placed(64, rope)}
        both = torch.cat((latent, rope), 1)
        if kind == "fp8_528":
            x = both.unflatten(-1, (16, 32))
            k = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448.0))
            return {"values": placed(512, (x * torch.exp2(-k)).flatten(1)), "exponent": None}
        return {"rows": placed(576, both).view(cache.shape)}
    if op == "rotate":
        return _exact_rope(st["x"], st["table"][st["positions"].long()][:, None], case["style"])
    if op == "index_k":
        x = st["k"][:n].double()
        x = torch.cat((_exact_rope(x[:, :ROPE], row, case["style"]), x[:, ROPE:]), 1)
        cache = st["index_cache"]
        if case["cache"] != "fp8":
            out = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
            out.view(-1, INDEX_DIM)[slots] = x
            return {"rows": out}
        codes, scale = _exact_scaled(x)
        out, scales = (torch.zeros(cache.shape[0], PAGE * w, dtype=torch.float64, device="cuda") for w in (INDEX_DIM, 1))
        out.view(-1, INDEX_DIM)[slots] = codes
        scales.view(-1)[slots] = scale[:, 0]
        return {"key": out, "scale": scales}
    if op == "index_q":
        row = st["table"][st["positions"].long()][:, None]
        x = st["q"].double()
        codes, scale = _exact_scaled(torch.cat((_exact_rope(x[..., :ROPE], row, case["style"]), x[..., ROPE:]), -1))
        return codes, st["weights"].double() * scale[..., 0]
    if op == "score":
        b, s = case["batch"], case["s_q"]
        out = torch.full((b, s, case["length"]), -math.inf, dtype=torch.float64, device="cuda")
        for i, length in enumerate(_lengths(case)):
            page = st["index_cache"][st["block_table"][i].long()]
            if case["keys"] == "fp8":
                keys = page[:, : PAGE * INDEX_DIM].contiguous().view(torch.float8_e4m3fn).double().view(-1, INDEX_DIM)
                keys = keys * page[:, PAGE * INDEX_DIM:].contiguous().view(torch.float32).double().view(-1, 1)
            else:
                keys = page.double().view(-1, INDEX_DIM)
            keys = keys[:length]
            for j in range(0, s, 64):
                q, w = st["q"][i, j: j + 64].double(), st["weights"][i, j: j + 64].double()
                dots = torch.einsum("shd,td->sht", q, keys).relu_()
                out[i, j: j + 64, :length] = torch.einsum("sh,sht->st", w, dots)
                if case["causal"]:
                    last = length - s + j + torch.arange(q.shape[0], device="cuda")[:, None]
                    out[i, j: j + 64].masked_fill_(torch.arange(case["length"], device="cuda") > last, -math.inf)
        if case["block"] == 1:
            return out
        return torch.nn.functional.pad(out, (0, -case["length"] % PAGE), value=-math.inf).unflatten(-1, (-1, PAGE)).amax(-1)
    return None
