"""CPU checks of the calls that write new tokens and choose what the sparse
attention reads: arguments are refused on the host before anything is
enqueued (on a machine without a GPU any CUDA call would return 6), and the
oracle of those calls is pinned to closed forms and brute force."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced: checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)
FAR = ctypes.c_void_p(1 << 40)


def _at(k):
    """The k-th of fake arrays that lie apart."""
    return ctypes.c_void_p((k + 2) << 40)


@pytest.fixture(scope="module")
def lib():
    import mla_latent_kv_14_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from mla_latent_kv_14_gb300 import build
        build.build()
    return m.load_library()


def _call(lib, name, base, **kw):
    args = dict(base)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(lib, name)(*args.values())


APPEND = dict(c=_at(0), cs=576, r=_at(1), rs=576, dtype=0, slots=_at(2), pos=_at(3), table=_at(4), maxp=4096, style=0, n=4,
              kv=_at(5), blocks=8, page=64, fmt=0, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(maxp=0), 1), (dict(blocks=0), 1), (dict(blocks=1 << 26), 1),
    (dict(page=32), 1), (dict(fmt=4), 1), (dict(fmt=-1), 1), (dict(dtype=2), 1), (dict(style=2), 1),
    (dict(cs=504), 1), (dict(cs=577), 1), (dict(rs=56), 1), (dict(rs=65), 1), (dict(fmt=2, cs=440), 1),
    (dict(fmt=1, dtype=1), 2), (dict(fmt=2, dtype=1), 2), (dict(fmt=3, dtype=1), 2),
    (dict(c=None), 1), (dict(r=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(table=None), 1),
    (dict(kv=None), 1), (dict(c=ODD), 1), (dict(r=ODD), 1), (dict(kv=ODD), 1), (dict(table=ODD), 1),
    (dict(slots=ODD), 1), (dict(pos=ODD), 1), (dict(status=ODD), 1), (dict(n=0, c=None, kv=None), 0),
    (dict(cs=1 << 50), 1), (dict(rs=1 << 62), 1),                 # beyond any address
    (dict(c=_at(5)), 1), (dict(r=ctypes.c_void_p((7 << 40) + 8 * 64 * 1152 - 16)), 1),   # in the cache
])
def test_append_kv_argument_checks(lib, kw, code):
    assert _call(lib, "mla_append_kv", APPEND, **kw) == code


ROTATE = dict(x=FAKE, xt=192 * 8, xh=192, out=FAR, ot=576 * 8, oh=576, dtype=0, pos=FAKE, table=FAKE, maxp=4096,
              style=0, tokens=4, heads=8, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(tokens=1 << 28), 1), (dict(maxp=0), 1), (dict(dtype=3), 1),
    (dict(style=-1), 1), (dict(xt=-8), 1), (dict(xh=4), 1), (dict(ot=4604), 1), (dict(oh=0), 1), (dict(ot=0), 1),
    (dict(oh=64, ot=128), 1),                                     # rows of the output overlap one another
    (dict(x=ODD), 1), (dict(out=ODD), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1),
    (dict(table=None), 1), (dict(status=ODD), 1), (dict(tokens=0, x=None, out=None), 0),
    (dict(xt=1 << 60), 1), (dict(oh=1 << 50), 1),
    (dict(out=FAKE), 1),                                          # overlaps x with other strides
    (dict(out=ctypes.c_void_p((1 << 20) + 64), ot=192 * 8, oh=192), 1),   # 32 elements into x's rows
    (dict(out=ctypes.c_void_p((1 << 20) + 320), ot=192 * 8, oh=192), 1),  # 160 of 192: into the next head's dims
])
def test_rotate_q_argument_checks(lib, kw, code):
    assert _call(lib, "mla_rotate_q", ROTATE, **kw) == code


INDEX_K = dict(k=_at(0), ks=128, dtype=0, slots=_at(1), pos=_at(2), table=_at(3), maxp=4096, style=0, n=4, cache=_at(4),
               blocks=8, page=64, fmt=0, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(ks=120), 1), (dict(ks=132), 1), (dict(fmt=2), 1), (dict(dtype=2), 1), (dict(page=128), 1),
    (dict(blocks=-1), 1), (dict(style=7), 1), (dict(maxp=-1), 1), (dict(k=ODD), 1), (dict(cache=ODD), 1),
    (dict(k=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(table=None), 1), (dict(status=ODD), 1),
    (dict(n=0, k=None), 0), (dict(k=_at(4)), 1),
])
def test_append_index_k_argument_checks(lib, kw, code):
    assert _call(lib, "mla_append_index_k", INDEX_K, **kw) == code


INDEX_Q = dict(q=_at(0), qt=64 * 128, qh=128, dtype=0, w=_at(1), pos=_at(2), table=_at(3), maxp=4096, style=0, tokens=4,
               heads=64, out=_at(4), wout=_at(5), status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(tokens=1 << 25), 1), (dict(qt=-8), 1), (dict(qh=130), 1),
    (dict(dtype=2), 1), (dict(style=2), 1), (dict(q=None), 1), (dict(w=None), 1), (dict(out=None), 1),
    (dict(wout=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(w=ODD), 1), (dict(pos=None), 1),
    (dict(status=ODD), 1), (dict(tokens=0, q=None), 0),
    (dict(out=_at(0)), 1), (dict(wout=ctypes.c_void_p((3 << 40) + 4)), 1), (dict(out=_at(1)), 1), (dict(wout=_at(0)), 1),
])
def test_quantize_index_q_argument_checks(lib, kw, code):
    assert _call(lib, "mla_quantize_index_q", INDEX_Q, **kw) == code


SCORE = dict(q=_at(0), dtype=0, w=_at(1), cache=_at(2), fmt=0, blocks=8, page=64, bt=_at(3), maxb=8, sl=_at(4), batch=2,
             s_q=1, heads=64, causal=0, block=1, scores=_at(5), stride=512, width=512, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), 1), (dict(dtype=2), 1), (dict(blocks=0), 1), (dict(page=32), 1), (dict(maxb=0), 1),
    (dict(batch=0), 1), (dict(s_q=0), 1), (dict(heads=0), 1), (dict(heads=65), 2), (dict(block=2), 1),
    (dict(stride=511), 1), (dict(width=0), 1), (dict(q=None), 1), (dict(w=None), 1), (dict(cache=None), 1),
    (dict(bt=None), 1), (dict(sl=None), 1), (dict(scores=None), 1), (dict(q=ODD), 1), (dict(cache=ODD), 1),
    (dict(w=ODD), 1), (dict(scores=ODD), 1), (dict(status=ODD), 1), (dict(batch=1 << 20, s_q=1 << 10), 1),
    (dict(width=(1 << 31) - 1, stride=1 << 31, maxb=1 << 26), 1),
    (dict(width=(1 << 31) - 1, stride=1 << 31), 1),               # columns behind the table's reach
    (dict(batch=1 << 16, width=1 << 24, stride=1 << 24, maxb=1 << 20), 2),   # more tiles than the list counts
    (dict(scores=_at(0)), 1), (dict(scores=_at(1)), 1), (dict(scores=_at(2)), 1), (dict(scores=_at(3)), 1),
    (dict(scores=_at(4)), 1), (dict(stride=1 << 60), 1),
])
def test_index_score_argument_checks(lib, kw, code):
    assert _call(lib, "mla_index_score", SCORE, **kw) == code


SELECT = dict(scores=_at(0), stride=512, width=512, sl=_at(1), batch=2, s_q=1, causal=0, block=1, topk=64, bt=_at(2),
              maxb=8, blocks=8, page=64, idx=_at(3), lens=_at(4), status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(stride=100), 1), (dict(width=0), 1), (dict(batch=0), 1), (dict(s_q=-1), 1), (dict(block=32), 1),
    (dict(topk=0), 1), (dict(maxb=0), 1), (dict(blocks=0), 1), (dict(page=16), 1), (dict(scores=None), 1),
    (dict(sl=None), 1), (dict(bt=None), 1), (dict(idx=None), 1), (dict(block=64, lens=None), 1), (dict(idx=ODD), 1),
    (dict(lens=ODD), 1), (dict(scores=ODD), 1), (dict(status=ODD), 1), (dict(batch=1 << 16, s_q=1 << 16), 1),
    (dict(topk=(1 << 31) - 1), 1), (dict(width=(1 << 31) - 1, stride=1 << 31, maxb=1 << 26), 1),
    (dict(batch=1 << 14, s_q=1 << 14), 2),                        # rows beyond a launch's blocks
    (dict(idx=_at(0)), 1), (dict(idx=_at(2)), 1), (dict(lens=_at(1)), 1), (dict(lens=_at(3)), 1), (dict(stride=1 << 60), 1),
])
def test_select_topk_argument_checks(lib, kw, code):
    assert _call(lib, "mla_select_topk", SELECT, **kw) == code


def test_binding_refuses_before_the_library():
    """Shapes, types and devices that the C ABI cannot see."""
    import mla_latent_kv_14_gb300 as m
    i32 = torch.int32
    c, r = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    kv, ix = torch.zeros(2, 64, 1, 576, dtype=torch.bfloat16), torch.zeros(4, dtype=i32)
    table = torch.zeros(16, 64)
    bad = [
        lambda: m.mla_append_kv(c[:, :448], r, kv, ix, ix, table),                  # latent width of another format
        lambda: m.mla_append_kv(c, r[:3], kv, ix, ix, table),
        lambda: m.mla_append_kv(c, r.half(), kv, ix, ix, table),
        lambda: m.mla_append_kv(c, r, kv.half(), ix, ix, table),                    # cache of another type
        lambda: m.mla_append_kv(c, r, kv, ix.long(), ix, table),
        lambda: m.mla_append_kv(c, r, kv, ix, ix[:3], table),
        lambda: m.mla_append_kv(c, r, kv, ix, ix, table.double()),
        lambda: m.mla_append_kv(c, r, kv[..., :512], ix, ix, table),
        lambda: m.mla_append_kv(c, r, kv, ix, ix, table),                           # not on a cuda device
        lambda: m.mla_rotate_q(c, ix, table),
        lambda: m.mla_rotate_q(r.view(4, 1, 64), ix, table, out=torch.zeros(4, 2, 64, dtype=torch.bfloat16)),
        lambda: m.mla_append_index_k(c, kv, ix, ix, table),
        lambda: m.mla_append_index_k(c[:, :128], torch.zeros(2, 8192, dtype=torch.uint8), ix, ix, table, m.INDEX_FP8),
        lambda: m.mla_quantize_index_q(c.view(4, 4, 128), torch.zeros(4, 3), ix, table),
        lambda: m.mla_index_score(c.view(1, 4, 4, 128), torch.zeros(1, 4, 4), torch.zeros(2, 64, 1, 128), ix.view(1, 4), ix[:1]),
        lambda: m.mla_index_score(c.view(1, 4, 4, 128), torch.zeros(1, 4, 4), torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16),
                                  ix.view(1, 4), ix[:1], block=16),
        lambda: m.mla_select_topk(torch.zeros(1, 1, 8), ix[:1], 0, ix.view(1, 4), 8),
        lambda: m.mla_select_topk(torch.zeros(2, 3, 8).transpose(0, 1), ix[:3], 4, ix.view(1, 4), 8),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(m.MLAError) as e:
            f()
        assert e.value.status == 1, k


# ---- the quotient of the quantisers ----
def _fma32(a, b, c):
    """a * b + c of fp32 arrays, rounded once: the product is exact in 64 bits,
    the sum is rounded to odd there, then to fp32."""
    p, c = a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)
    s = p + c
    t = s - p
    rest = (p - (s - t)) + (c - t)
    beside = np.nextafter(s, np.where(rest > 0, np.inf, -np.inf))
    return np.where((rest != 0) & (s.view(np.int64) % 2 == 0), beside, s).astype(np.float32)


@pytest.mark.parametrize("kind", ["any", "midpoints", "ends"])
def test_corrected_quotient_is_the_division(kind):
    """q = x r, q + (x - q s) r with r = 1 / s: the steps by which the paged
    writers divide by a block's scale, against the correctly rounded quotient."""
    rng = np.random.default_rng(0)
    n = 1 << 20
    s = (1 + rng.integers(0, 1 << 23, n) * 2.0 ** -23).astype(np.float32)
    x = (1 + rng.integers(0, 1 << 23, n) * 2.0 ** -23).astype(np.float32)
    if kind == "midpoints":        # x / s within a few units of five-bit numbers, e4m3's values and midpoints
        x = (rng.integers(16, 32, n) / 16 * s.astype(np.float64)).astype(np.float32)
        x = (x.view(np.int32) + rng.integers(-2, 3, n).astype(np.int32)).view(np.float32)
    if kind == "ends":             # scales just below a power of two
        s = (2 - rng.integers(1, 1 << 12, n) * 2.0 ** -23).astype(np.float32)
    r = (1 / s.astype(np.float64)).astype(np.float32)
    q = x * r
    got = _fma32(_fma32(q, -s, x), r, q)
    # a quotient of two 24-bit numbers rounded to 53 bits, then to 24, is rounded correctly
    assert (got == (x.astype(np.float64) / s.astype(np.float64)).astype(np.float32)).all()


def test_scale_quotient_for_every_significand():
    """amax / 448 by the same steps, for all 2^23 significands."""
    x = (1 + np.arange(1 << 23) * 2.0 ** -23).astype(np.float32)
    s = np.full_like(x, 448.0)
    r = (1 / s.astype(np.float64)).astype(np.float32)
    q = x * r
    got = _fma32(_fma32(q, -s, x), r, q)
    assert (got == (x.astype(np.float64) / 448.0).astype(np.float32)).all()


# ---- the oracle ----
@pytest.mark.parametrize("halves", [False, True])
def test_oracle_rotation_is_a_complex_product(halves):
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((5, 64)).astype(np.float32)).to(torch.bfloat16)
    table = oracle.rope_table(70000)[[0, 1, 63, 4096, 69999]]
    got = oracle.rotate(x, table, halves).astype(np.float64)
    v = oracle.to_f64(x)
    a, b = (v[:, :32], v[:, 32:]) if halves else (v[:, 0::2], v[:, 1::2])
    z = (a + 1j * b) * (table[:, :32].astype(np.float64) + 1j * table[:, 32:].astype(np.float64))
    want = np.concatenate((z.real, z.imag), 1) if halves else np.stack((z.real, z.imag), -1).reshape(5, 64)
    # two products and a sum, each rounded by 2^-24 of at most |a| + |b|
    size = np.abs(a) + np.abs(b)
    size = np.concatenate((size, size), 1) if halves else np.repeat(size, 2, axis=1)
    assert (np.abs(got - want) <= 2 * 2.0 ** -24 * size).all()
    assert (got[0] == v[0]).all()                                  # position 0 does nothing


def test_oracle_rotation_keeps_relative_positions():
    """The dot of two rotated rows depends on the distance of their positions alone."""
    rng = np.random.default_rng(1)
    q, k = (torch.from_numpy(rng.standard_normal(64).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    t = oracle.rope_table(300)
    for halves in (False, True):
        dots = [oracle.rotate(q, t[p + 17], halves, exact=True) @ oracle.rotate(k, t[p], halves, exact=True)
                for p in (0, 5, 211)]
        # the table's own roundings: 2^-24 per cosine and sine of each row
        assert np.ptp(dots) <= 8 * 2.0 ** -24 * np.abs(oracle.to_f64(q)).sum() * np.abs(oracle.to_f64(k)).max() * 2


def test_oracle_selection_by_brute_force():
    s = np.array([0.0, 3.0, -0.0, np.nan, 3.0, -np.inf, 1.0, np.inf])
    assert oracle.select_topk(s, 8, 1).tolist() == [7]
    assert oracle.select_topk(s, 8, 2).tolist() == [1, 7]          # of two 3.0 the first
    assert oracle.select_topk(s, 8, 5).tolist() == [0, 1, 4, 6, 7]  # 0.0 and -0.0 are equal
    assert oracle.select_topk(s, 8, 6).tolist() == [0, 1, 2, 4, 6, 7]
    assert oracle.select_topk(s, 8, 7).tolist() == [0, 1, 2, 3, 4, 6, 7]   # NaN as -inf: the lower position
    assert oracle.select_topk(s, 6, 2, last=True).tolist() == [1, 5]
    assert oracle.select_topk(s, 4, 9).tolist() == [0, 1, 2, 3]
    assert oracle.select_topk(s, 0, 3).tolist() == []


def test_oracle_score_of_one_head():
    q, k = np.zeros((1, 1, 128)), np.zeros((3, 128))
    q[0, 0, 5], k[0, 5], k[1, 5], k[2, 6] = 2.0, 3.0, -1.0, 9.0
    assert oracle.index_score(q, np.array([[0.5]]), k).tolist() == [[3.0, 0.0, 0.0]]
    assert oracle.page_max(np.arange(65.0)[None]).tolist() == [[63.0, 64.0]]


# ---- memory that an output may not share ----
def _row_starts(base, token, head, tokens, heads):
    return {(t, h): base + t * token + h * head for t in range(tokens) for h in range(heads)}


def _rows_race(x, out):
    """True where a row of `out` touches another (token, head)'s row of `x`, or a part of its own."""
    return any(abs(a - b) < 64 and not (i == j and a == b) for i, a in x.items() for j, b in out.items())


@pytest.mark.parametrize("kw", [
    dict(tokens=2, heads=2, xt=192, xh=128, ot=192, oh=128, d=64),     # out[0, 1] is x[1, 0]
    dict(tokens=2, heads=2, xt=320, xh=192, ot=320, oh=192, d=-128),   # x[0, 1] is out[1, 0]
    dict(tokens=2, heads=2, xt=192, xh=320, ot=192, oh=320, d=-128),   # the same, heads outside
])
def test_rotate_q_refuses_rows_that_meet(lib, kw):
    kw, d = dict(kw), kw["d"]
    del kw["d"]
    out = ctypes.c_void_p(FAKE.value + 2 * d)
    assert _rows_race(_row_starts(0, kw["xt"], kw["xh"], 2, 2), _row_starts(d, kw["ot"], kw["oh"], 2, 2))
    assert _call(lib, "mla_rotate_q", ROTATE, **dict(kw, out=out)) == 1


def test_rotate_q_refuses_every_row_that_meets_another(lib):
    """All small layouts in which one thread would write what another reads (only such layouts are called)."""
    strides, meets = [64, 72, 128, 136, 192, 200, 256, 320, 384], 0
    for tokens, heads in ((1, 2), (2, 1), (2, 2), (3, 2), (2, 3)):
        for t in strides:
            for h in strides:
                x = _row_starts(0, t, h, tokens, heads)
                for d in range(-512, 513, 8):
                    if _rows_race(x, _row_starts(d, t, h, tokens, heads)):
                        meets += 1
                        out = ctypes.c_void_p(FAKE.value + 2 * d)
                        got = _call(lib, "mla_rotate_q", ROTATE, xt=t, xh=h, ot=t, oh=h, out=out, tokens=tokens, heads=heads)
                        assert got == 1, (tokens, heads, t, h, d)
    assert meets > 10000


def _before(k, gap):
    """`gap` bytes before the k-th of the fake arrays."""
    return ctypes.c_void_p(_at(k).value - gap)


ROTATE_APART = dict(ROTATE, x=_at(0), pos=_at(1), table=_at(2), out=_at(3))
_TABLE_BYTES = 256 * 4096


@pytest.mark.parametrize("name,base,out,inputs", [
    ("mla_append_kv", "APPEND", 5, ["slots", "pos", "table", "status"]),
    ("mla_append_index_k", "INDEX_K", 4, ["slots", "pos", "table", "status"]),
    ("mla_quantize_index_q", "INDEX_Q", 4, ["pos", "table", "status"]),
    ("mla_quantize_index_q", "INDEX_Q", 5, ["pos", "table", "status"]),
    ("mla_rotate_q", "ROTATE_APART", 3, ["pos", "table", "status"]),
    ("mla_index_score", "SCORE", 5, ["status"]),
    ("mla_select_topk", "SELECT", 3, ["status"]),
    ("mla_select_topk", "SELECT", 4, ["status"]),
])
def test_outputs_that_share_memory_are_refused(lib, name, base, out, inputs):
    args = globals()[base]
    for key in inputs:
        assert _call(lib, name, args, **{key: _at(out)}) == 1, key
    if "table" in inputs:                            # a table that ends inside the output; more rows than positions reach
        assert _call(lib, name, args, table=_before(out, _TABLE_BYTES - 16)) == 1
        assert _call(lib, name, args, table=_before(out, _TABLE_BYTES - 16), maxp=(1 << 63) - 1) == 1
    if "slots" in inputs:                            # an array that ends inside the output
        assert _call(lib, name, args, slots=_before(out, 4)) == 1
    if "pos" in inputs:
        assert _call(lib, name, args, pos=_before(out, 4)) == 1


@pytest.mark.parametrize("name,base,inputs", [
    ("mla_append_kv", "APPEND", ["c", "r", "slots", "pos", "table"]),
    ("mla_append_index_k", "INDEX_K", ["k", "slots", "pos", "table"]),
    ("mla_quantize_index_q", "INDEX_Q", ["q", "w", "pos", "table"]),
    ("mla_rotate_q", "ROTATE_APART", ["x", "pos", "table"]),
    ("mla_index_score", "SCORE", ["q", "w", "cache", "bt", "sl"]),
    ("mla_select_topk", "SELECT", ["scores", "bt", "sl"]),
])
def test_a_status_word_inside_an_input_is_refused(lib, name, base, inputs):
    for key in inputs:
        args = globals()[base]
        assert _call(lib, name, args, status=ctypes.c_void_p(args[key].value + 4)) == 1, key


def test_the_library_is_built_without_the_extension(monkeypatch, tmp_path):
    """No Python or PyTorch headers: the extension's compilation fails, libmla.so is there all the same."""
    from mla_latent_kv_14_gb300 import build as b
    ran = []

    def run(cmd, what, verbose=False):
        ran.append(what)
        if what == "g++":
            raise RuntimeError("g++ failed: Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmla.so"))
    monkeypatch.setattr(b, "HOST", str(tmp_path / "_host.so"))
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert (tmp_path / "libmla.so").read_text() == "link" and not (tmp_path / "_host.so").exists()


def test_corrected_quotient_gives_the_codes_of_the_division():
    """Every pair on which an e4m3 code could differ from that of the rounded quotient.

    With u = 2^-24: r = (1/s)(1 + a), |a| <= u, and q = (x/s)(1 + e), |e| <= 2u + u^2. The remainder x - q s = -x e is
    rounded by a factor 1 + b, |b| <= u, so what the last step rounds is (x/s)(1 - e (a + b + a b)): off by at most
    2^-45.9 of the quotient. The result therefore is the rounded quotient unless a midpoint m of two fp32 neighbours lies
    that close to x/s, and its code can differ only if one of the two neighbours is a number t at which e4m3's rounding
    changes, which has five bits: t = T / 16 for T in 16..31, m = t +- 2^-24 (below t = 1: t - 2^-25), for quotients
    scaled to [1, 2). With s = S 2^-23 and x = A 2^-27, |x - m s| <= 2^-45.9 x says |A - S T -+ S 2^-20| < 2^-16.9: S lies
    within 8.6 of a multiple of 2^20 (2^21 below t = 1), and A = S T +- that multiple. All of those, with a margin:"""
    s, x = [], []
    for T in range(16, 32):
        for sign, shift in ((1, 20), (-1, 20 if T > 16 else 21)):
            for k in range((1 << 23) >> shift, ((1 << 24) >> shift) + 1):
                for S in range((k << shift) - 64, (k << shift) + 65):
                    if not (1 << 23) <= S < (1 << 24):
                        continue
                    for A in range(S * T + sign * k - 1, S * T + sign * k + 2):
                        unit = 16 if A < 1 << 28 else 32           # x of [1, 2), of [2, 4)
                        if A % unit == 0:
                            s.append(S * 2.0 ** -23)
                            x.append(A * 2.0 ** -27)
    s, x = np.array(s), np.array(x)
    assert len(s) > 1000 and (s.astype(np.float32) == s).all() and (x.astype(np.float32) == x).all()
    q64 = x / s
    s, x = s.astype(np.float32), x.astype(np.float32)
    r = (1 / s.astype(np.float64)).astype(np.float32)
    q = x * r
    got, want = _fma32(_fma32(q, -s, x), r, q), q64.astype(np.float32)
    for scale in range(-12, 9):                                    # codes from below the smallest to the saturated ones
        f = np.float32(2.0 ** scale)
        assert (oracle.e4m3_encode_rne(got * f) == oracle.e4m3_encode_rne(want * f)).all()
