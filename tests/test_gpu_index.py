"""GPU parity of the calls around the decode: appends to the paged caches,
rotation, index rows, the index score and the selection, against the 64-bit
oracle; and a run of them together, as a serving step uses them.

Rows are compared bit for bit (the rotation's roundings are part of its
definition). Scores carry the oracle's own bound of an fp32 evaluation.
"""
import threading
import time

import numpy as np
import pytest
import torch

import oracle
from tests.helpers import assert_close_attn

pytestmark = pytest.mark.gpu

mla = pytest.importorskip("mla_latent_kv_14_gb300")
DEV = "cuda"
PAGE = 64
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mla.load_library()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _bits(status):
    torch.cuda.synchronize()
    return int(status.item())


TABLE = oracle.rope_table(5000)


def _table():
    return torch.from_numpy(TABLE).to(DEV)


def _new(n, seed, pages):
    """Distinct slots with some -1 and one behind the cache, positions with one out of range."""
    rng = np.random.default_rng(seed)
    slots = rng.permutation(pages * PAGE)[:n].astype(np.int32)
    pos = rng.integers(0, 5000, n).astype(np.int32)
    bad = 0
    if n > 8:
        slots[[1, n - 1]] = -1
        slots[3], pos[5], pos[6] = pages * PAGE, 5000, -1
        bad = 1
    keep = (slots >= 0) & (slots < pages * PAGE) & (pos >= 0) & (pos < 5000)
    return slots, pos, keep, bad


# ---------------------------------------------------------------------------
# appends
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("fmt,dtype", [(0, BF), (0, HF), (1, BF), (2, BF), (3, BF)])
@pytest.mark.parametrize("n", [1, 63, 130])
def test_append_kv(n, fmt, dtype, halves):
    latent, pages = (448 if fmt >= 2 else 512), 5
    kv = torch.randn(n, latent + 64 + 8, generator=_gen(n)).to(dtype)
    if n > 20:
        kv[10] = 0                                     # a zero block
        kv[11, :latent] *= 1e-6                        # tiny scales
        kv[12, 3] = 60000.0 if dtype == HF else 3.0e4
    slots, pos, keep, bad = _new(n, n + fmt, pages)
    width = {0: 576, 1: 656, 2: 528, 3: 288}[fmt]
    cache = torch.randint(0, 256, (pages, PAGE, 1, width * (2 if fmt == 0 else 1)), dtype=torch.uint8, generator=_gen(7))
    want = cache.clone().view(pages * PAGE, -1)
    rows = oracle.append_rows(kv[:, :latent], kv[:, latent:latent + 64], TABLE[np.clip(pos, 0, 4999)], bool(halves), fmt)
    want[torch.from_numpy(slots[keep]).long()] = rows[torch.from_numpy(keep)]
    dev, st = kv.to(DEV), _status()
    got = cache.to(DEV)
    got = got.view(dtype) if fmt == 0 else got
    back = mla.mla_append_kv(dev[:, :latent], dev[:, latent:latent + 64], got, torch.from_numpy(slots).to(DEV),
                             torch.from_numpy(pos).to(DEV), _table(), kv_format=fmt, rope_style=halves, status=st)
    assert back is got and _bits(st) == bad
    assert torch.equal(got.view(torch.uint8).cpu().view(pages * PAGE, -1), want)


def test_append_equals_the_contiguous_quantisers():
    """At position 0 (no turn) the rows are those of mla_quantize_kv_*."""
    n = 64
    for fmt, quant, w in ((1, mla.mla_quantize_kv_fp8, 576), (2, mla.mla_quantize_kv_fp8_528, 512),
                          (3, mla.mla_quantize_kv_fp4_288, 512)):
        kv = torch.randn(n, w, generator=_gen(fmt)).to(BF).to(DEV)
        want = quant(kv)
        cache = torch.zeros(1, 64, 1, want.shape[-1], dtype=torch.uint8, device=DEV)
        zero = torch.zeros(n, dtype=torch.int32, device=DEV)
        mla.mla_append_kv(kv[:, : w - 64], kv[:, w - 64:], cache, torch.arange(n, dtype=torch.int32, device=DEV), zero,
                          _table(), kv_format=fmt)
        assert torch.equal(cache.view(n, -1), want)


def _wide(n, width, seed):
    """bf16 rows over the type's whole range: block maxima from subnormal to the
    largest, zeros of both signs, infinities and NaN."""
    g = _gen(seed)
    kv = torch.randn(n, width, generator=g)
    kv = (kv * torch.exp2(torch.linspace(-132.0, 124.0, n))[:, None]).to(BF)
    kv[torch.rand(n, width, generator=g) < 0.02] = 0.0
    kv[torch.rand(n, width, generator=g) < 0.02] = -0.0
    kv[3, 5], kv[n // 3, 100], kv[n // 2, 7] = float("inf"), float("-inf"), float("nan")
    kv[n - 9] = float("nan")
    kv[n - 4, :128] = -0.0
    return kv


def test_append_of_any_value_equals_the_contiguous_quantisers():
    n = 1024
    for fmt, quant, w in ((1, mla.mla_quantize_kv_fp8, 576), (2, mla.mla_quantize_kv_fp8_528, 512),
                          (3, mla.mla_quantize_kv_fp4_288, 512)):
        kv = _wide(n, w, fmt)
        kv[:, w - 64:] = kv[:, w - 64:].nan_to_num(1.0, 2.0, -2.0).clamp(-4, 4)    # rotated by cos 1, sin 0: kept
        kv = kv.to(DEV)
        want = quant(kv)
        cache = torch.zeros(n // 64, 64, 1, want.shape[-1], dtype=torch.uint8, device=DEV)
        zero = torch.zeros(n, dtype=torch.int32, device=DEV)
        mla.mla_append_kv(kv[:, : w - 64], kv[:, w - 64:], cache, torch.arange(n, dtype=torch.int32, device=DEV), zero,
                          _table(), kv_format=fmt)
        got = cache.view(n, -1)
        same = got == want
        if fmt == 1:      # an fp32 NaN (the scale of a NaN block) may have any payload
            same[:, 512:528] |= (got[:, 512:528].contiguous().view(torch.float32).isnan()
                                 & want[:, 512:528].contiguous().view(torch.float32).isnan()).repeat_interleave(4, dim=1)
            # adding 0 * sin turns a rope value of -0 into +0
            rope, plain = got[:, 528:].contiguous().view(BF), want[:, 528:].contiguous().view(BF)
            same[:, 528:] |= (rope == plain).repeat_interleave(2, dim=1)
        else:             # the same -0, as a code's sign
            per = 1 if fmt == 2 else 2
            zero_code = (kv[:, 448:] == 0).view(n, -1, per).any(dim=2)
            same[:, 448 // per:512 // per] |= zero_code
        assert same.all(), (fmt, (~same).nonzero()[:8].tolist())


def test_index_rows_of_any_value():
    n = 1024
    x = _wide(n, 128, 4)
    x[:, :64] = x[:, :64].nan_to_num(0.0, 0.0, 0.0)              # the rotated half finite
    x[:, :64] = x[:, :64].clamp(-1e30, 1e30)
    pos = np.arange(n).astype(np.int32)
    with np.errstate(invalid="ignore"):
        _, codes, scale = oracle.index_row_codes(x, TABLE[:n], False)
    whole = torch.isfinite(x.float()).all(dim=1).numpy()
    q8, w = mla.mla_quantize_index_q(x[:, None].to(DEV), torch.ones(n, 1, device=DEV), torch.from_numpy(pos).to(DEV), _table())
    q8, w = q8.view(torch.uint8).cpu().numpy()[:, 0], w.cpu().numpy()[:, 0]
    assert (q8[whole] == codes[whole]).all() and (w[whole] == scale[whole]).all()
    row = [i for i in np.flatnonzero(~whole) if not torch.isnan(x[i].float()).any()]
    assert row
    for i in row:                                                # an infinite scale: zeros, NaN for the infinities
        inf = torch.isinf(x[i].float()).numpy()
        assert np.isinf(w[i]) and ((q8[i] & 0x7F) == np.where(inf, 0x7F, 0)).all()


@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (3, 128), (65, 5), (7, 16), (40, 33)])
def test_rotate_q(tokens, heads, dtype, halves):
    x = torch.randn(tokens, heads, 192, generator=_gen(tokens)).to(dtype)
    rng = np.random.default_rng(tokens)
    pos = rng.integers(0, 5000, tokens).astype(np.int32)
    bad = 0
    if tokens > 4:
        pos[2], pos[4], bad = -1, 5000, 1
    keep = torch.from_numpy((pos >= 0) & (pos < 5000))
    rot = oracle.round_to(oracle.rotate(x[..., 128:], TABLE[np.clip(pos, 0, 4999)][:, None], bool(halves)), dtype)
    p = torch.from_numpy(pos).to(DEV)
    # a slice of the projection into a slice of the decode's query
    q = torch.full((tokens, heads, 576), 7.0, dtype=dtype, device=DEV)
    xd, st = x.to(DEV), _status()
    mla.mla_rotate_q(xd[..., 128:], p, _table(), out=q[..., 512:], rope_style=halves, status=st)
    assert _bits(st) == bad
    want = torch.full((tokens, heads, 576), 7.0, dtype=dtype)
    want[..., 512:][keep] = rot[keep]
    assert torch.equal(q.cpu(), want)
    # in place, and into other columns of the same rows
    inplace, beside = x.to(DEV), x.to(DEV)
    mla.mla_rotate_q(inplace[..., 128:], p, _table(), out=inplace[..., 128:], rope_style=halves)
    mla.mla_rotate_q(beside[..., 128:], p, _table(), out=beside[..., :64], rope_style=halves)
    want, want2 = x.clone(), x.clone()
    want[..., 128:][keep] = rot[keep]
    want2[..., :64][keep] = rot[keep]
    assert torch.equal(inplace.cpu(), want) and torch.equal(beside.cpu(), want2)
    # heads-major storage, and one row for every head
    major = x[..., 128:].transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    got = mla.mla_rotate_q(major, p, _table(), rope_style=halves)
    assert torch.equal(got.cpu()[keep], rot[keep])
    shared = mla.mla_rotate_q(xd[:, :1, 128:].expand(-1, heads, -1), p, _table(), rope_style=halves)
    assert torch.equal(shared.cpu()[keep], rot[:, :1].expand(-1, heads, -1)[keep])


@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 17, 130])
def test_append_index_k(n, fp8, dtype, halves):
    pages = 4
    k = torch.randn(n, 160, generator=_gen(n)).to(dtype)
    if n > 12:
        k[12] = 0
    slots, pos, keep, bad = _new(n, n, pages)
    v, codes, scale = oracle.index_row_codes(k[:, :128], TABLE[np.clip(pos, 0, 4999)], bool(halves))
    at = slots[keep]
    cache = torch.randint(0, 256, (pages, 8448 if fp8 else PAGE * 256), dtype=torch.uint8, generator=_gen(3))
    want = cache.clone().numpy()
    if fp8:
        want[:, :8192].reshape(pages, PAGE, 128)[at // PAGE, at % PAGE] = codes[keep]
        w = want[:, 8192:].copy().view(np.float32)
        w[at // PAGE, at % PAGE] = scale[keep]
        want[:, 8192:] = w.view(np.uint8)
        got = cache.to(DEV)
    else:
        rows = oracle.round_to(v, dtype).view(torch.uint8).numpy()
        want.reshape(pages * PAGE, 256)[at] = rows[keep]
        got = cache.to(DEV).view(dtype).view(pages, PAGE, 1, 128)
    st = _status()
    mla.mla_append_index_k(k.to(DEV)[:, :128], got, torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV), _table(),
                           index_format=mla.INDEX_FP8 if fp8 else mla.INDEX_16BIT, rope_style=halves, status=st)
    assert _bits(st) == bad
    assert (got.view(torch.uint8).cpu().numpy().reshape(pages, -1) == want).all()


@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,heads", [(1, 64), (9, 3), (33, 32)])
def test_quantize_index_q(tokens, heads, dtype, halves):
    q = torch.randn(tokens, heads, 192, generator=_gen(heads)).to(dtype)
    w = torch.randn(tokens, heads, generator=_gen(heads + 1))
    q[0, 0] = 0
    pos = np.random.default_rng(heads).integers(0, 5000, tokens).astype(np.int32)
    bad = 0
    if tokens > 4:
        pos[2], pos[4], bad = -1, 5000, 1
    keep = (pos >= 0) & (pos < 5000)
    _, codes, scale = oracle.index_row_codes(q[..., 64:], TABLE[np.clip(pos, 0, 4999)][:, None], bool(halves))
    st = _status()
    q8 = torch.zeros(tokens, heads, 128, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    wo = torch.zeros(tokens, heads, device=DEV)
    mla.mla_quantize_index_q(q.to(DEV)[..., 64:], w.to(DEV), torch.from_numpy(pos).to(DEV), _table(), rope_style=halves,
                             q_out=q8, weights_out=wo, status=st)
    assert _bits(st) == bad and q8.dtype == torch.float8_e4m3fn
    assert (q8.view(torch.uint8).cpu().numpy() == np.where(keep[:, None, None], codes, 0)).all()
    assert (wo.cpu().numpy() == np.where(keep[:, None], w.numpy() * scale, 0)).all()
    q2, wo = mla.mla_quantize_index_q(q.to(DEV)[..., 64:], w.to(DEV), torch.from_numpy(pos).to(DEV), _table(), rope_style=halves)
    assert q2.dtype == torch.float8_e4m3fn and torch.equal(q2.view(torch.uint8)[keep], q8.view(torch.uint8)[keep])
    wd = w.to(DEV)
    mla.mla_quantize_index_q(q.to(DEV)[..., 64:], wd, torch.from_numpy(pos).to(DEV), _table(), rope_style=halves, weights_out=wd)
    assert (wd.cpu().numpy() == np.where(keep[:, None], w.numpy() * scale, w.numpy())).all()


# ---------------------------------------------------------------------------
# score
# ---------------------------------------------------------------------------
def _score_case(lens, s_q, heads, kind, seed, spare=1):
    """Queries, weights, a paged index cache, its block table, and the values they stand for."""
    rng = np.random.default_rng(seed)
    B, most = len(lens), max(1, -(-max(lens) // PAGE))
    pages = B * most + spare
    bt = rng.permutation(pages)[: B * most].reshape(B, most).astype(np.int32)
    g = _gen(seed)
    q, k = torch.randn(B, s_q, heads, 128, generator=g), torch.randn(pages, PAGE, 128, generator=g)
    w = torch.randn(B, s_q, heads, generator=g) / heads
    if kind == "fp8":
        _, qc, qs = oracle.index_row_codes(q.to(BF), TABLE[:1], False)
        _, kc, ks = oracle.index_row_codes(k.to(BF), TABLE[:1], False)
        q8 = torch.from_numpy(qc).view(torch.float8_e4m3fn)
        w = w * torch.from_numpy(qs)
        cache = torch.from_numpy(np.concatenate((kc.reshape(pages, -1), ks.view(np.uint8).reshape(pages, -1)), axis=1))
        vals = oracle.e4m3_value_table()
        return q8, w, cache, bt, vals[qc], vals[kc] * ks.astype(np.float64)[..., None]
    dtype = BF if kind == "bf16" else HF
    q, k = q.to(dtype), k.to(dtype)
    return q, w, k.unsqueeze(2).contiguous(), bt, oracle.to_f64(q), oracle.to_f64(k)


def _score_ref(lens, s_q, causal, bt, qv, w, kv, width, bad=()):
    """(scores, bound) [B, s_q, width] by tokens."""
    B = len(lens)
    ref, err = np.full((B, s_q, width), -np.inf), np.zeros((B, s_q, width))
    for b in range(B):
        keys = kv[bt[b]].reshape(-1, 128)
        s, e = (f(qv[b], oracle.to_f64(w[b]), keys) for f in (oracle.index_score, oracle.index_score_error))
        for i in range(s_q):
            v = max(0, min(lens[b] - (s_q - 1 - i if causal else 0), width, keys.shape[0]))
            ref[b, i, :v], err[b, i, :v] = s[i, :v], e[i, :v]
        for p in bad:
            if p[0] == b:
                ref[b, :, p[1] * PAGE:(p[1] + 1) * PAGE] = -np.inf
    return ref, err


def _check_scores(got, ref, err, what):
    got = got.double().cpu().numpy()
    inf = np.isneginf(ref)
    assert (np.isneginf(got) == inf).all(), f"{what}: -inf at other places"
    off = np.abs(np.where(inf, 0, got) - np.where(inf, 0, ref))
    bad = off > err
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst {(off / np.maximum(err, 1e-30)).max():.3g} of it"


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("lens,s_q,heads,causal", [
    ([1], 1, 1, False),
    ([64, 65, 127, 128, 129], 1, 64, False),
    ([0, 300, 0, 1], 2, 16, True),                 # no token; fewer tokens than queries
    ([700, 33], 5, 64, True),                      # two groups of three queries, one of them empty
    ([513], 17, 33, False),                        # padded heads
    ([250, 900], 9, 20, True),
    ([190], 40, 7, True),                          # several units of 32 queries
    ([300, 77], 2, 64, True),                      # 128 columns: the widest of four accumulators
    ([140, 400], 8, 32, False),                    # 256 columns, one group
    ([140], 16, 16, True),
    ([500], 3, 16, False),                         # 48 columns: a batch that ends inside a load
    ([260, 5], 13, 16, True),
])
def test_index_score(lens, s_q, heads, causal, kind):
    q, w, cache, bt, qv, kv = _score_case(lens, s_q, heads, kind, seed=heads + s_q)
    fmt = mla.INDEX_FP8 if kind == "fp8" else mla.INDEX_16BIT
    args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    st = _status()
    width = max(1, max(lens))
    ref, err = _score_ref(lens, s_q, causal, bt, qv, w, kv, width)
    got = mla.mla_index_score(*args, width=width, causal=causal, index_format=fmt, status=st)
    assert _bits(st) == 0
    _check_scores(got, ref, err, f"{kind} tokens")
    # the default width (the block table's reach), into a column range of a wider buffer
    wide = torch.full((len(lens), s_q, bt.shape[1] * PAGE + 3), 7.0, device=DEV)
    mla.mla_index_score(*args, causal=causal, index_format=fmt, scores=wide[..., :-3], status=st)
    ref, err = _score_ref(lens, s_q, causal, bt, qv, w, kv, bt.shape[1] * PAGE)
    _check_scores(wide[..., :-3], ref, err, f"{kind} wide")
    assert (wide[..., -3:] == 7.0).all() and _bits(st) == 0
    pages = mla.mla_index_score(*args, causal=causal, index_format=fmt, block=64, status=st)
    _check_scores(pages, oracle.page_max(ref), np.maximum(oracle.page_max(err), 0), f"{kind} pages")
    assert _bits(st) == 0


def test_index_score_many_tiles_per_cta():
    """More (unit, tile) pairs than CTAs, ragged: ranges that end inside a unit, rings that wrap."""
    lens, s_q, heads = [9000, 0, 17000, 130, 4096], 11, 64
    for kind in ("bf16", "fp8"):
        q, w, cache, bt, qv, kv = _score_case(lens, s_q, heads, kind, seed=5)
        fmt = mla.INDEX_FP8 if kind == "fp8" else mla.INDEX_16BIT
        got = mla.mla_index_score(q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), width=17000, causal=True, index_format=fmt)
        ref, err = _score_ref(lens, s_q, True, bt, qv, w, kv, 17000)
        _check_scores(got, ref, err, kind)


def test_index_score_bad_pages_and_short_columns():
    lens = [300, 200]
    for kind in ("bf16", "fp8"):
        q, w, cache, bt, qv, kv = _score_case(lens, 1, 64, kind, seed=9)
        bad = bt.copy()
        bad[0, 1], bad[1, 3], bad[1, 4] = -1, cache.shape[0], -7        # the last one is behind the request
        st = _status()
        fmt = mla.INDEX_FP8 if kind == "fp8" else mla.INDEX_16BIT
        args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bad).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
        got = mla.mla_index_score(*args, index_format=fmt, status=st)
        assert _bits(st) == 1
        ref, err = _score_ref(lens, 1, False, bt, qv, w, kv, bt.shape[1] * PAGE, bad=[(0, 1), (1, 3)])
        _check_scores(got, ref, err, kind)
        st = _status()
        args = args[:3] + (torch.from_numpy(bt).to(DEV),) + args[4:]
        got = mla.mla_index_score(*args, width=77, index_format=fmt, status=st)   # narrower than the requests
        assert _bits(st) == 1
        ref, err = _score_ref(lens, 1, False, bt, qv, w, kv, 77)
        _check_scores(got, ref, err, kind)


def test_index_score_timeout_is_reported():
    q, w, cache, bt, qv, kv = _score_case([200], 1, 16, "bf16", seed=1)
    args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor([200], dtype=torch.int32, device=DEV))
    st = _status()
    mla.mla_set_test_stall(100000)
    try:
        mla.mla_index_score(*args, status=st)
    finally:
        mla.mla_set_test_stall(0)
    code, bits = mla.mla_read_status(st)
    assert code == 5 and bits == 2
    ref, err = _score_ref([200], 1, False, bt, qv, w, kv, 256)
    _check_scores(mla.mla_index_score(*args, status=st), ref, err, "after the time-out")
    assert _bits(st) == 0


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def _select_ref(scores, lens, s_q, causal, block, topk, bt, pages):
    B, width = len(lens), scores.shape[-1]
    idx, out = np.full((B, s_q, topk), -1, np.int64), np.zeros((B, s_q), np.int64)
    for b in range(B):
        for i in range(s_q):
            seen = max(0, min(lens[b] - (s_q - 1 - i if causal else 0), width * block, bt.shape[1] * PAGE))
            n = -(-seen // block)
            at = oracle.select_topk(scores[b, i], n, topk, last=block > 1)
            pg = bt[b, at if block > 1 else at // PAGE].astype(np.int64)
            rows = pg if block > 1 else pg * PAGE + at % PAGE
            idx[b, i, : len(at)] = np.where((pg >= 0) & (pg < pages), rows, -1)
            out[b, i] = len(at) if block == 1 else (len(at) - 1) * PAGE + seen - (n - 1) * PAGE if n else 0
    return idx, out


def _select_both(scores, lens, s_q, causal, block, topk, bt, pages, bits=0):
    st = _status()
    idx, out = mla.mla_select_topk(scores.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), topk,
                                   torch.from_numpy(bt).to(DEV), pages, causal=causal, block=block, status=st)
    assert _bits(st) == bits
    ref, want = _select_ref(scores.numpy(), lens, s_q, causal, block, topk, bt, pages)
    assert (out.cpu().numpy() == want).all()
    assert (idx.cpu().numpy() == ref).all()


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special"])
@pytest.mark.parametrize("block,topk", [(1, 1), (1, 64), (1, 2048), (64, 1), (64, 7), (64, 100)])
def test_select_topk(block, topk, kind):
    lens, s_q = [0, 1, 64, 65, 2500, 2047, 2048], 3
    rng = np.random.default_rng(topk)
    most = -(-max(lens) // PAGE)
    pages = len(lens) * most + 2
    bt = rng.permutation(pages)[: len(lens) * most].reshape(len(lens), most).astype(np.int32)
    width = most * PAGE // block
    s = torch.randn(len(lens), s_q, width, generator=_gen(topk))
    if kind == "ties":
        s = (s * 2).round() / 2
    elif kind == "equal":
        s = torch.zeros_like(s)
        s[..., ::2] = -0.0
    elif kind == "special":
        r = torch.rand(s.shape, generator=_gen(1))
        s[r < 0.3], s[r < 0.2], s[r < 0.1], s[r < 0.05] = float("nan"), float("inf"), float("-inf"), 0.0
        s[r > 0.9] = 1e-41                             # a subnormal
    for causal in (False, True):
        _select_both(s, lens, s_q, causal, block, topk, bt, pages)


def test_select_bad_pages_and_hidden_columns():
    """Columns behind the visible ones are not read; bad pages come out as -1."""
    lens = [200, 130]
    bt = np.array([[0, -1, 2, 3], [4, 5, 9, -1]], dtype=np.int32)
    s = torch.randn(2, 1, 256, generator=_gen(2))
    s[0, 0, 200:], s[1, 0, 130:] = float("nan"), float("inf")
    _select_both(s, lens, 1, False, 1, 100, bt, 8, bits=1)
    _select_both(s, lens, 1, False, 1, 300, bt, 8, bits=1)
    _select_both(s[..., :4].contiguous(), lens, 1, False, 64, 3, bt, 8, bits=1)
    _select_both(s[..., :100].contiguous(), lens, 1, False, 1, 20, np.abs(bt) % 8, 8, bits=1)   # fewer columns than tokens


@pytest.mark.parametrize("kind", ["normal", "ties", "special", "smooth", "low starts"])
@pytest.mark.parametrize("n", [100, 2000, 2049, 4096, 5001, 8192])
def test_select_many_rows(n, kind):
    """Enough rows that each gets a narrow block; lengths down to one and none."""
    rng = np.random.default_rng(n)
    lens, s_q = [n, n - 1, n // 2 + 3, 70, 1, 0], 80
    most = -(-n // PAGE)
    bt = rng.permutation(6 * most).reshape(6, most).astype(np.int32)
    s = torch.randn(6, s_q, n, generator=_gen(n))
    if kind == "ties":
        s = (s * 4).round() / 4
    elif kind == "special":
        r = torch.rand(s.shape, generator=_gen(1))
        s[r < 0.2], s[r < 0.1], s[r < 0.03] = float("nan"), float("-inf"), float("inf")
    elif kind == "smooth":
        s = torch.sin(torch.arange(n) * (9.0 / n)).expand(6, s_q, n) + s * 1e-3
    elif kind == "low starts":
        s[..., (torch.arange(n) % 256) < 64] -= 1e4
    for topk in (1, min(512, n // 3), n - 2):
        _select_both(s, lens, s_q, True, 1, topk, bt, 6 * most)
    pages = s[..., :most].contiguous()
    _select_both(pages, lens, s_q, True, 64, max(1, most // 3), bt, 6 * most)


@pytest.mark.parametrize("topk", [3, 200, 1500])
def test_select_pages_of_many_long_rows(topk):
    lens, s_q = [64 * 2100, 64 * 4100 + 5, 64 * 1000], 120
    most = 4101
    bt = np.random.default_rng(topk).permutation(3 * most).reshape(3, most).astype(np.int32)
    s = torch.randn(3, s_q, most, generator=_gen(topk))
    _select_both(s, lens, s_q, True, 64, topk, bt, 3 * most)


@pytest.mark.parametrize("n", [5000, 40000, 131072, 300001])
def test_select_long_rows(n):
    rng = np.random.default_rng(n)
    most = -(-n // PAGE)
    bt = rng.permutation(most).reshape(1, most).astype(np.int32)
    s = torch.relu(torch.randn(1, 2, n, generator=_gen(n)))           # half of it exactly zero
    for topk in (2048, n // 2 + 100, n - 1, n + 5):                   # inside the positive half, among the zeros, all
        _select_both(s, [n], 2, True, 1, topk, bt, most)


@pytest.mark.parametrize("n", [700, 2000, 9000, 20000, 131072])
@pytest.mark.parametrize("kind", ["rising", "falling", "comb", "few", "plateau", "inf"])
def test_select_uneven_rows(n, kind):
    """Rows on which a sample of the scores says little about the rest, or whose threshold is shared by many."""
    most = -(-n // PAGE)
    bt = np.random.default_rng(n).permutation(most).reshape(1, most).astype(np.int32)
    t = torch.arange(n, dtype=torch.float32)
    s = {"rising": t / n - 0.5, "falling": 1e3 - t, "comb": torch.where(t % 64 < 62, t % 977, -t),
         "few": torch.where(t > n - 40, t, torch.zeros(n)), "plateau": torch.where(t % 3 == 0, t * 1e-3, torch.full((n,), 5.0)),
         "inf": torch.where(t % 5 == 0, float("inf"), torch.where(t % 7 == 0, -float("inf"), t))}[kind]
    # every warp's and every block's first scores low, the others high
    low = s.clone()
    low[(torch.arange(n) % 160) < 80] = -1e30
    for row in (s, low):
        for topk in (1, 30, min(2048, n // 2), n - 1):
            _select_both(row.view(1, 1, n), [n], 1, False, 1, topk, bt, most)


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
def _step(lens, seed, kv_format, index_format, kv_dtype=BF):
    """Appends every token of each request, rotates the queries and scores: what a serving step has in hand."""
    B, h, hi = len(lens), 128, 32
    rng = np.random.default_rng(seed)
    most = -(-max(lens) // PAGE)
    pages = B * most
    bt = rng.permutation(pages).reshape(B, most).astype(np.int32)
    slots = np.concatenate([bt[b, np.arange(L) // PAGE] * PAGE + np.arange(L) % PAGE for b, L in enumerate(lens)]).astype(np.int32)
    pos = np.concatenate([np.arange(L) for L in lens]).astype(np.int32)
    n = len(slots)
    g = _gen(seed)
    kv = torch.randn(n, 576, generator=g).to(kv_dtype)
    q = torch.randn(B, h, 576, generator=g).to(kv_dtype)
    k_idx, q_idx = torch.randn(n, 128, generator=g).to(BF), torch.randn(B, hi, 128, generator=g).to(BF)
    w = torch.randn(B, hi, generator=g) / hi
    qpos = np.array(lens, dtype=np.int32) - 1
    d = lambda t: (torch.from_numpy(t) if isinstance(t, np.ndarray) else t).to(DEV)  # noqa: E731
    table = _table()
    kvc = (torch.zeros(pages, PAGE, 1, 576, dtype=kv_dtype, device=DEV) if kv_format == 0 else
           torch.zeros(pages, PAGE, 1, 656, dtype=torch.uint8, device=DEV))
    kvd = d(kv)
    mla.mla_append_kv(kvd[:, :512], kvd[:, 512:], kvc, d(slots), d(pos), table, kv_format=kv_format)
    qa = d(q)
    mla.mla_rotate_q(qa[..., 512:], d(qpos), table, out=qa[..., 512:])
    ic = (torch.zeros(pages, 8448, dtype=torch.uint8, device=DEV) if index_format else
          torch.zeros(pages, PAGE, 1, 128, dtype=BF, device=DEV))
    mla.mla_append_index_k(d(k_idx), ic, d(slots), d(pos), table, index_format=index_format)
    qi, wi = d(q_idx), d(w)
    if index_format:
        qi, wi = mla.mla_quantize_index_q(qi, wi, d(qpos), table)
    else:
        mla.mla_rotate_q(qi[..., :64], d(qpos), table, out=qi[..., :64])
    return dict(B=B, bt=bt, btd=d(bt), sl=d(np.array(lens, np.int32)), pages=pages, kvc=kvc, q=qa, ic=ic, qi=qi.view(B, 1, hi, 128),
                wi=wi.view(B, 1, hi), kv=kv, q_in=q, slots=slots, pos=pos, qpos=qpos)


def _plain_keys(s, fmt):
    """The cache rows the appends should have left, in float64, by physical row, and the rotated queries."""
    rows = oracle.append_rows(s["kv"][:, :512], s["kv"][:, 512:], TABLE[s["pos"]], False, fmt)
    dense = oracle.dequantize_kv_fp8(rows.numpy()) if fmt else oracle.to_f64(rows.view(s["kv"].dtype))
    all_rows = np.zeros((s["pages"] * PAGE, 576))
    all_rows[s["slots"]] = dense
    q = oracle.to_f64(s["q_in"]).copy()
    q[..., 512:] = oracle.to_f64(oracle.round_to(oracle.rotate(s["q_in"][..., 512:], TABLE[s["qpos"]][:, None], False), s["q_in"].dtype))
    return all_rows, q


def test_tokens_from_append_to_sparse_attention():
    """append -> index -> score -> select -> token-sparse decode of the 656-byte cache."""
    lens, topk = [900, 130, 2000], 256
    s = _step(lens, 21, mla.KV_FP8_656, mla.INDEX_FP8)
    scores = mla.mla_index_score(s["qi"], s["wi"], s["ic"], s["btd"], s["sl"], index_format=mla.INDEX_FP8)
    idx, cnt = mla.mla_select_topk(scores, s["sl"], topk, s["btd"], s["pages"])
    meta, ns = mla.mla_get_metadata(None, 1, 128, batch=s["B"], topk=topk, is_fp8=True, device=DEV)
    out, lse = mla.mla_decode_with_kvcache(s["q"].view(s["B"], 1, 128, 576), s["kvc"], None, None, 512, meta, ns, is_fp8=True,
                                           indices=idx)
    torch.cuda.synchronize()
    ref, want = _select_ref(scores.cpu().numpy(), lens, 1, False, 1, topk, s["bt"], s["pages"])
    assert (idx.cpu().numpy() == ref).all() and (cnt.cpu().numpy() == want).all()
    rows, q = _plain_keys(s, 1)
    ro, rl, _ = oracle.mla_decode(q[:, None], rows, indices=ref, softmax_scale=576 ** -0.5)
    assert_close_attn(out, lse, ro, rl, "token-sparse")


@pytest.mark.parametrize("heads,dtype", [(128, BF), (16, HF)])
def test_pages_from_append_to_paged_attention(heads, dtype):
    """append -> index -> page scores -> page lists -> paged decode of a 16-bit cache."""
    lens, topk = [900, 130, 2000, 64], 5
    s = _step(lens, 22, mla.KV_16BIT, mla.INDEX_16BIT, kv_dtype=dtype)
    scores = mla.mla_index_score(s["qi"], s["wi"], s["ic"], s["btd"], s["sl"], block=64)
    table, sel = mla.mla_select_topk(scores, s["sl"], topk, s["btd"], s["pages"], block=64)
    table, sel = table.view(s["B"], topk), sel.view(s["B"])
    q = s["q"][:, :heads].contiguous().view(s["B"], 1, heads, 576)
    meta, ns = mla.mla_get_metadata(sel, 1, heads)
    out, lse = mla.mla_decode_with_kvcache(q, s["kvc"], table, sel, 512, meta, ns)
    st, bits = mla.mla_read_status(device=DEV)
    assert st == 0 and bits == 0
    ref, want = _select_ref(scores.cpu().numpy(), lens, 1, False, 64, topk, s["bt"], s["pages"])
    assert (table.cpu().numpy() == ref[:, 0]).all() and (sel.cpu().numpy() == want[:, 0]).all()
    rows, qv = _plain_keys(s, 0)
    ro, rl, _ = oracle.mla_decode(qv[:, None, :heads], rows, cache_seqlens=want[:, 0], block_table=ref[:, 0], softmax_scale=576 ** -0.5)
    assert_close_attn(out, lse, ro, rl, "paged")


def test_captured_and_replayed_on_another_stream():
    """The chain captured into a graph, replayed with new inputs, while the same calls run eagerly beside it."""
    lens, topk = [700, 300], 128
    s = _step(lens, 23, mla.KV_FP8_656, mla.INDEX_FP8)
    scores = torch.empty(2, 1, s["bt"].shape[1] * PAGE, device=DEV)
    idx, cnt = torch.empty(2, 1, topk, dtype=torch.int32, device=DEV), torch.empty(2, 1, dtype=torch.int32, device=DEV)

    def chain(sc, ix, ct):
        mla.mla_index_score(s["qi"], s["wi"], s["ic"], s["btd"], s["sl"], index_format=mla.INDEX_FP8, scores=sc)
        mla.mla_select_topk(sc, s["sl"], topk, s["btd"], s["pages"], indices=ix, lens=ct)

    chain(scores, idx, cnt)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain(scores, idx, cnt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(scores, idx, cnt)
    for step in range(3):
        s["wi"].mul_(-0.5)
        s["sl"].sub_(17)
        torch.cuda.synchronize()
        sc2, ix2, ct2 = torch.empty_like(scores), torch.empty_like(idx), torch.empty_like(cnt)
        graph.replay()
        with torch.cuda.stream(stream):
            chain(sc2, ix2, ct2)
        torch.cuda.synchronize()
        assert torch.equal(scores, sc2) and torch.equal(idx, ix2) and torch.equal(cnt, ct2)


@pytest.mark.parametrize("n,topk", [(40000, 2048), (300, 7)])
def test_selection_of_long_rows_captured(n, topk):
    """Clusters (the long rows) in a graph; the graph and an eager call on another stream at once."""
    most = -(-n // PAGE)
    bt = torch.arange(2 * most, dtype=torch.int32, device=DEV).view(2, most)
    sl = torch.tensor([n, n - 5], dtype=torch.int32, device=DEV)
    s = torch.randn(2, 1, n, generator=_gen(n)).to(DEV)
    idx, cnt = torch.empty(2, 1, topk, dtype=torch.int32, device=DEV), torch.empty(2, 1, dtype=torch.int32, device=DEV)
    mla.mla_select_topk(s, sl, topk, bt, 2 * most, indices=idx, lens=cnt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_select_topk(s, sl, topk, bt, 2 * most, indices=idx, lens=cnt)
    other = torch.cuda.Stream()
    for step in range(3):
        s.copy_(torch.randn(2, 1, n, generator=_gen(n + step)))
        idx.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            ix2, ct2 = mla.mla_select_topk(s, sl, topk, bt, 2 * most)
        torch.cuda.synchronize()
        ref, want = _select_ref(s.cpu().numpy(), [n, n - 5], 1, False, 1, topk, bt.cpu().numpy(), 2 * most)
        assert (idx.cpu().numpy() == ref).all() and (cnt.cpu().numpy() == want).all()
        assert torch.equal(idx, ix2) and torch.equal(cnt, ct2)


def test_writers_on_a_side_stream_and_captured():
    """Every writer in one graph, replayed with new tokens: the same bytes as eager calls."""
    n, pages = 70, 3
    table = _table()
    g = _gen(99)
    kv, k = torch.randn(n, 576, generator=g).to(BF).to(DEV), torch.randn(n, 128, generator=g).to(BF).to(DEV)
    q, w = torch.randn(n, 4, 128, generator=g).to(BF).to(DEV), torch.randn(n, 4, generator=g).to(DEV)
    slots = torch.randperm(pages * PAGE, generator=g)[:n].int().to(DEV)
    pos = torch.randint(0, 5000, (n,), generator=g).int().to(DEV)

    def buffers():
        return dict(kv=torch.zeros(pages, PAGE, 1, 656, dtype=torch.uint8, device=DEV), ic=torch.zeros(pages, 8448, dtype=torch.uint8, device=DEV),
                    rot=torch.zeros(n, 4, 64, dtype=BF, device=DEV), q8=torch.zeros(n, 4, 128, dtype=torch.uint8, device=DEV),
                    w=torch.zeros(n, 4, device=DEV))

    def write(o):
        mla.mla_append_kv(kv[:, :512], kv[:, 512:], o["kv"], slots, pos, table, kv_format=mla.KV_FP8_656)
        mla.mla_append_index_k(k, o["ic"], slots, pos, table, index_format=mla.INDEX_FP8)
        mla.mla_rotate_q(q[..., :64], pos, table, out=o["rot"])
        mla.mla_quantize_index_q(q, w, pos, table, q_out=o["q8"], weights_out=o["w"])

    captured = buffers()
    write(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write(captured)
    side = torch.cuda.Stream()
    for step in range(2):
        kv.mul_(-1.5), k.mul_(0.75), q.mul_(2.0), w.add_(1.0)
        pos.copy_((pos + 311) % 5000)
        eager = buffers()
        for o in captured.values():
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            write(eager)
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(eager[name], captured[name]), name


def test_same_inputs_same_bits():
    lens = [5000, 3000, 100]
    q, w, cache, bt, _, _ = _score_case(lens, 3, 48, "bf16", seed=31)
    args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    first = mla.mla_index_score(*args, causal=True)
    for _ in range(3):
        assert torch.equal(first, mla.mla_index_score(*args, causal=True))


def test_a_full_launch_queue_leaves_other_threads_running():
    """Calls behind a spinning kernel fill the launch queue; the thread that makes them waits, the others do not."""
    x = torch.randn(4, 2, 64, generator=_gen(1)).to(BF).to(DEV)
    out, pos, table = torch.empty_like(x), torch.zeros(4, dtype=torch.int32, device=DEV), _table()
    side = torch.cuda.Stream()
    calls, longest = 5000, [0.0]

    def work():
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_500_000_000)           # cycles: three quarters of a second
            for _ in range(calls):
                t = time.perf_counter()
                mla.mla_rotate_q(x, pos, table, out=out)
                longest[0] = max(longest[0], time.perf_counter() - t)

    mla.mla_rotate_q(x, pos, table, out=out)
    torch.cuda.synchronize()
    thread = threading.Thread(target=work)
    gap, last = 0.0, time.perf_counter()
    thread.start()
    while thread.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    torch.cuda.synchronize()
    assert longest[0] > 0.2, "the queue never filled"
    assert gap < longest[0] / 2


# ---------------------------------------------------------------------------
# the forms that many rows and long caches take
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,heads", [(255, 128), (256, 128), (1100, 33), (32768, 1), (6600, 5), (259, 127)])
def test_rotate_q_of_many_rows(tokens, heads, dtype, halves):
    """Below 32768 rows a thread takes one head, from there four heads of a token (33, 5, 127: not all of them have one)."""
    test_rotate_q(tokens, heads, dtype, halves)


@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,heads", [(511, 64), (512, 64), (5000, 7), (1500, 33), (2000, 33), (2100, 64), (131073, 1)])
def test_quantize_index_q_of_many_rows(tokens, heads, dtype, halves):
    """A lane group takes 1, 2, 2 (of 7 heads), 3, 4 (of 33), 8 and 8 (of one) heads of a token."""
    test_quantize_index_q(tokens, heads, dtype, halves)


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
@pytest.mark.parametrize("halves", [0, 1])
def test_appends_of_many_tokens(fmt, halves):
    """Prompts of a few thousand tokens, into every format and both index formats."""
    n, pages, latent = 3001, 50, (448 if fmt >= 2 else 512)
    kv = torch.randn(n, latent + 64, generator=_gen(fmt)).to(BF)
    slots, pos, keep, bad = _new(n, 40 + fmt, pages)
    width = {0: 1152, 1: 656, 2: 528, 3: 288}[fmt]
    want = torch.zeros(pages * PAGE, width, dtype=torch.uint8)
    rows = oracle.append_rows(kv[:, :latent], kv[:, latent:], TABLE[np.clip(pos, 0, 4999)], bool(halves), fmt)
    want[torch.from_numpy(slots[keep]).long()] = rows[torch.from_numpy(keep)]
    got = torch.zeros(pages, PAGE, 1, width, dtype=torch.uint8, device=DEV)
    dev, st = kv.to(DEV), _status()
    sd, pd = torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV)
    mla.mla_append_kv(dev[:, :latent], dev[:, latent:], got.view(BF) if fmt == 0 else got, sd, pd, _table(), kv_format=fmt,
                      rope_style=halves, status=st)
    assert _bits(st) == bad and torch.equal(got.cpu().view(pages * PAGE, width), want)


def _long_ref(lens, s_q, causal, bt, qv, w, kv, width):
    """_score_ref by matrix products, request by request, on long caches."""
    ref, err = np.full((len(lens), s_q, width), -np.inf), np.zeros((len(lens), s_q, width))
    wv, u = oracle.to_f64(w), 2.0 ** -24
    for b, n in enumerate(lens):
        keys = kv[bt[b]].reshape(-1, 128)[:min(n, width)]
        heads = qv.shape[2]
        for i in range(s_q):
            v = max(0, min(n - (s_q - 1 - i if causal else 0), len(keys)))
            if v:
                ref[b, i, :v] = wv[b, i] @ np.maximum(qv[b, i] @ keys[:v].T, 0.0)
                # the bound of oracle.index_score_error
                err[b, i, :v] = (2 * 128 + heads + 2) * u * (np.abs(keys[:v]) @ (np.abs(wv[b, i]) @ np.abs(qv[b, i])))
    return ref, err


def test_the_long_reference_is_the_oracle():
    lens = [150, 0, 64]
    q, w, cache, bt, qv, kv = _score_case(lens, 3, 5, "bf16", seed=2)
    a, b = _score_ref(lens, 3, True, bt, qv, w, kv, 160), _long_ref(lens, 3, True, bt, qv, w, kv, 160)
    for x, y in zip(a, b):
        assert (np.isneginf(x) == np.isneginf(y)).all()
        assert np.allclose(np.where(np.isneginf(x), 0, x), np.where(np.isneginf(y), 0, y), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("lens,s_q,heads,causal", [
    ([200000, 30000, 0, 130, 25000], 1, 64, False),   # 64 columns, 13 tiles a block: a ring of 12 wraps, both epilogue groups
    ([70001, 9000, 0, 130, 20000], 2, 64, True),      # 128 columns
    ([40000, 1, 33333], 1, 16, False),                # 16 columns
    ([60000, 129], 3, 32, True),                      # 96 columns
    ([50000, 700, 5000], 8, 13, False),               # 128 columns of padded heads
    ([30000, 4000, 130], 11, 64, True),               # two groups of 256 columns
    ([26000, 3], 40, 9, True),                        # several units
])
def test_index_score_of_long_caches(lens, s_q, heads, causal, kind):
    """Several tiles a block, by tokens and by pages."""
    q, w, cache, _, qv, kv = _score_case([1] * len(lens), s_q, heads, kind, seed=heads, spare=400)
    # requests share the pages of a small cache
    bt = np.random.default_rng(heads).integers(0, len(kv), (len(lens), -(-max(lens) // PAGE))).astype(np.int32)
    fmt = mla.INDEX_FP8 if kind == "fp8" else mla.INDEX_16BIT
    args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    width = bt.shape[1] * PAGE
    ref, err = _long_ref(lens, s_q, causal, bt, qv, w, kv, width)
    st = _status()
    got = mla.mla_index_score(*args, causal=causal, index_format=fmt, status=st)
    _check_scores(got, ref, err, f"{kind} tokens")
    pages = mla.mla_index_score(*args, causal=causal, index_format=fmt, block=64, status=st)
    _check_scores(pages, oracle.page_max(ref), oracle.page_max(err), f"{kind} pages")
    assert _bits(st) == 0


@pytest.mark.parametrize("n", [20000, 140001])
def test_select_pages_of_rows_beyond_a_block(n):
    """Pages in a cluster, and rows that are read again."""
    bt = np.random.default_rng(n).permutation(n).reshape(1, n).astype(np.int32)
    s = torch.randn(1, 2, n, generator=_gen(n))
    for topk in (1, 500, n - 3, n + 1):
        _select_both(s, [64 * n - 3], 2, True, 64, topk, bt, n)


def test_select_tokens_of_many_long_rows():
    """More clusters than run at once: 32 scores a thread."""
    n, s_q = 20000, 80
    most = -(-n // PAGE)
    bt = np.random.default_rng(1).permutation(2 * most).reshape(2, most).astype(np.int32)
    _select_both(torch.randn(2, s_q, n, generator=_gen(3)), [n, 17000], s_q, True, 1, 2048, bt, 2 * most)


@pytest.mark.parametrize("strides,beside", [((1088, 1024), 512), ((1024, 1088), 512), ((4 * 192, 192), 128), ((192, 40 * 192), 64)])
def test_rotate_q_between_rows_of_one_buffer(strides, beside):
    """Views whose rows interleave without meeting, tokens or heads outside: rows written, everything else as it was."""
    tokens, heads = 2, 2
    buf = torch.randn(20000, generator=_gen(beside)).to(BF)
    pos = np.array([3, 4000], dtype=np.int32)
    rows = (tokens, heads, 64)
    for src, dst in ((0, beside), (beside, 0)):
        x = buf.as_strided(rows, strides + (1,), src)
        want = buf.clone()
        want.as_strided(rows, strides + (1,), dst).copy_(oracle.round_to(oracle.rotate(x, TABLE[pos][:, None], False), BF))
        dev = buf.to(DEV)
        mla.mla_rotate_q(dev.as_strided(rows, strides + (1,), src), torch.from_numpy(pos).to(DEV), _table(),
                         out=dev.as_strided(rows, strides + (1,), dst))
        assert torch.equal(dev.cpu(), want)


# ---------------------------------------------------------------------------
# caches and rows beyond 4 GB
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,row", [(0, 1152), (1, 656), (2, 528), (3, 288)])
def test_append_behind_4_gb(fmt, row):
    pages, latent, n = 2 ** 32 // (PAGE * row) + 40, (448 if fmt >= 2 else 512), 70
    kv = torch.randn(n, latent + 64, generator=_gen(row)).to(BF)
    first = pages * PAGE - n
    cache = torch.empty(pages, PAGE, 1, row, dtype=torch.uint8, device=DEV)
    flat = cache.view(-1, row)
    flat[:n], flat[first - 3:] = 7, 7
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    dev = kv.to(DEV)
    mla.mla_append_kv(dev[:, :latent], dev[:, latent:], cache.view(BF) if fmt == 0 else cache, pos + first, pos, _table(),
                      kv_format=fmt)
    rows = oracle.append_rows(kv[:, :latent], kv[:, latent:], TABLE[:n], False, fmt)
    assert torch.equal(flat[first:].cpu(), rows)
    assert (flat[:n] == 7).all() and (flat[first - 3:first] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_index_cache_and_scores_behind_4_gb(fp8):
    """Keys written and scored on the last pages of a large index cache, into rows of scores 4 GB apart, and selected."""
    page = 8448 if fp8 else PAGE * 256
    pages, n, heads = 2 ** 32 // page + 40, 130, 16
    g = _gen(page)
    k, q = torch.randn(n, 128, generator=g).to(BF), torch.randn(2, heads, 128, generator=g).to(BF)
    w = torch.randn(2, heads, generator=g)
    cache = torch.empty(pages, page, dtype=torch.uint8, device=DEV)
    cache[:3], cache[-3:] = 0, 0
    ic = cache if fp8 else cache.view(BF).view(pages, PAGE, 1, 128)
    fmt = mla.INDEX_FP8 if fp8 else mla.INDEX_16BIT
    bt = torch.tensor([[pages - 1, pages - 3, pages - 2]] * 2, dtype=torch.int32)
    t = torch.arange(n)
    slots = (bt[0, t // PAGE] * PAGE + t % PAGE).int()
    zero = torch.zeros(n, dtype=torch.int32, device=DEV)
    mla.mla_append_index_k(k.to(DEV), ic, slots.to(DEV), zero, _table(), index_format=fmt)
    assert not cache[:3].any()
    if fp8:
        _, codes, scale = oracle.index_row_codes(k, TABLE[:1], False)
        kv = oracle.e4m3_value_table()[codes] * scale.astype(np.float64)[:, None]
        _, codes, scale = oracle.index_row_codes(q, TABLE[:1], False)
        qv, w = oracle.e4m3_value_table()[codes], w * torch.from_numpy(scale)
        qd = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(DEV)
    else:
        kv, qv, qd = oracle.to_f64(k), oracle.to_f64(q), q.to(DEV)
    wide = torch.empty(2, 1, 2 ** 30 + 64, device=DEV)
    scores = wide[..., :PAGE * 3]
    sl = torch.tensor([n, 70], dtype=torch.int32, device=DEV)
    mla.mla_index_score(qd[:, None], w[:, None].contiguous().to(DEV), ic, bt.to(DEV), sl, index_format=fmt, scores=scores)
    for b, seen in enumerate((n, 70)):
        ref, err = np.full((1, PAGE * 3), -np.inf), np.zeros((1, PAGE * 3))
        ref[:, :seen] = oracle.index_score(qv[b:b + 1], oracle.to_f64(w[b:b + 1]), kv[:seen])
        err[:, :seen] = oracle.index_score_error(qv[b:b + 1], oracle.to_f64(w[b:b + 1]), kv[:seen])
        _check_scores(scores[b], ref, err, f"request {b}")
    idx, cnt = mla.mla_select_topk(scores, sl, 50, bt.to(DEV), pages)
    ref, want = _select_ref(scores.cpu().numpy(), [n, 70], 1, False, 1, 50, bt.numpy(), pages)
    assert (idx.cpu().numpy() == ref).all() and (cnt.cpu().numpy() == want).all()


def test_rotate_q_of_rows_4_gb_apart():
    far = 2 ** 31 + 64
    buf = torch.empty(far + 256, dtype=BF, device=DEV)
    x = torch.randn(2, 2, 64, generator=_gen(8)).to(BF)
    src, dst = (buf.as_strided((2, 2, 64), (far, 64, 1), at) for at in (0, 128))
    src.copy_(x)
    pos = torch.tensor([9, 4999], dtype=torch.int32, device=DEV)
    mla.mla_rotate_q(src, pos, _table(), out=dst)
    assert torch.equal(dst.cpu(), oracle.round_to(oracle.rotate(x, TABLE[[9, 4999]][:, None], False), BF))
    assert torch.equal(src.cpu(), x)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("s_q,heads", [(1, 64), (3, 16), (11, 64)])
def test_index_score_of_poisoned_keys(s_q, heads, kind):
    """NaN and infinities behind the visible tokens, in pages that no table names and in their scales change nothing; a
    visible key of NaN counts as 0."""
    lens = [100, 0, 129, 64]
    q, w, cache, bt, qv, kv = _score_case(lens, s_q, heads, kind, seed=s_q + heads, spare=3)
    fp8 = kind == "fp8"
    nan, inf = float("nan"), float("inf")
    seen = {}
    for b, n in enumerate(lens):
        for t in range(n):
            seen[(int(bt[b, t // PAGE]), t % PAGE)] = b
    for p in range(len(cache)):
        for r in range(PAGE):
            if (p, r) not in seen:
                if fp8:
                    cache[p, r * 128:(r + 1) * 128] = 0x7F
                    cache[p, 8192:].view(torch.float32)[r] = nan if r % 2 else inf
                else:
                    cache[p, r] = nan if r % 2 else inf
    blind = (int(bt[0, 0]), 5)                                   # token 5 of request 0
    if fp8:
        cache[blind[0], 5 * 128:6 * 128] = 0x7F
    else:
        cache[blind] = nan
    kv[blind] = 0.0
    kv[~np.isfinite(kv)] = 0.0
    fmt = mla.INDEX_FP8 if fp8 else mla.INDEX_16BIT
    st = _status()
    args = (q.to(DEV), w.to(DEV), cache.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    ref, err = _score_ref(lens, s_q, True, bt, qv, w, kv, bt.shape[1] * PAGE)
    _check_scores(mla.mla_index_score(*args, causal=True, index_format=fmt, status=st), ref, err, "tokens")
    pages = mla.mla_index_score(*args, causal=True, index_format=fmt, block=64, status=st)
    _check_scores(pages, oracle.page_max(ref), oracle.page_max(err), "pages")
    assert _bits(st) == 0
