"""CPU checks of the calls for prompts over the latent cache: arguments are
refused on the host before anything is enqueued (on a machine without a GPU any
CUDA call would return 6), the Python side refuses tensors, and the oracle is
pinned to closed forms and brute force."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import oracle

ODD = ctypes.c_void_p((1 << 20) + 2)


def _at(k):
    """The k-th of fake arrays that lie apart (never dereferenced: checks fail first)."""
    return ctypes.c_void_p((k + 2) << 40)


def _into(k, byte):
    return ctypes.c_void_p(((k + 2) << 40) + byte)


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


NORM = dict(x=_at(0), xt=192 * 8, xh=192, w=_at(1), eps=1e-6, dim=192, at=128, out=_at(2), ot=192 * 8, oh=192, rope=None, rt=0,
            rh=0, dtype=0, pos=_at(3), table=_at(4), maxp=4096, style=0, tokens=4, heads=8, status=None, stream=None)
SPLIT = dict(rope=_at(5), rt=576 * 8, rh=576, ot=128 * 8, oh=128)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(tokens=1 << 28), 1), (dict(maxp=0), 1), (dict(dtype=2), 1), (dict(style=2), 1),
    (dict(eps=-1e-6), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(dim=56), 1), (dict(dim=196), 1), (dict(dim=0), 1),
    (dict(dim=584, xt=584 * 8, xh=584, ot=584 * 8, oh=584), 2), (dict(at=-8), 1), (dict(at=132), 1), (dict(at=136), 1), (dict(at=4), 1),
    (dict(xt=-8), 1), (dict(xh=4), 1), (dict(ot=4), 1), (dict(ot=184), 1), (dict(oh=184), 1), (dict(oh=0), 1), (dict(ot=192, oh=384), 1),
    (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(table=None), 1), (dict(x=ODD), 1), (dict(out=ODD), 1),
    (dict(w=ODD), 1), (dict(status=ODD), 1), (dict(pos=ODD), 1), (dict(table=ODD), 1), (dict(tokens=0, x=None, out=None), 0),
    (dict(xt=1 << 60), 1), (dict(oh=1 << 50), 1),
    (dict(out=_at(0), oh=200, ot=1600), 1), (dict(out=_into(0, 64)), 1), (dict(out=_at(1)), 1), (dict(out=_at(4)), 1), (dict(status=_at(0)), 1),
    (dict(status=_into(2, 16)), 1),
    (dict(SPLIT, rt=56), 1), (dict(SPLIT, rh=60), 1), (dict(SPLIT, rt=64, rh=64), 1), (dict(SPLIT, rope=ODD), 1), (dict(SPLIT, rope=_at(0)), 1),
    (dict(SPLIT, out=_at(0)), 1), (dict(SPLIT, rope=_at(2)), 1), (dict(SPLIT, oh=120), 1), (dict(SPLIT, rope=_at(3)), 1),
])
def test_norm_rotate_argument_checks(lib, kw, code):
    assert _call(lib, "mla_norm_rotate", NORM, **kw) == code


APPEND = dict(c=_at(0), cs=576, r=_at(1), rs=576, w=_at(2), eps=1e-6, dtype=0, slots=_at(3), pos=_at(4), table=_at(5), maxp=4096,
              style=0, n=4, kv=_at(6), blocks=8, page=64, fmt=0, rows=_at(7), ws=576, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(maxp=0), 1), (dict(blocks=0), 1), (dict(blocks=1 << 26), 1), (dict(page=32), 1),
    (dict(fmt=4), 1), (dict(fmt=-1), 1), (dict(dtype=2), 1), (dict(style=2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(cs=504), 1), (dict(cs=577), 1), (dict(rs=56), 1), (dict(rs=65), 1), (dict(fmt=2, cs=440), 1), (dict(ws=568), 1),
    (dict(ws=580), 1), (dict(fmt=3, ws=504), 1), (dict(fmt=1, dtype=1), 2), (dict(fmt=2, dtype=1), 2), (dict(fmt=3, dtype=1), 2),
    (dict(c=None), 1), (dict(r=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(table=None), 1), (dict(kv=None), 1),
    (dict(c=ODD), 1), (dict(r=ODD), 1), (dict(w=ODD), 1), (dict(kv=ODD), 1), (dict(rows=ODD), 1), (dict(slots=ODD), 1),
    (dict(pos=ODD), 1), (dict(table=ODD), 1), (dict(status=ODD), 1), (dict(n=0, c=None, kv=None), 0), (dict(cs=1 << 50), 1),
    (dict(c=_at(6)), 1), (dict(rows=_at(0)), 1), (dict(rows=_at(6)), 1), (dict(w=_into(6, 64)), 1), (dict(status=_at(7)), 1),
])
def test_norm_append_argument_checks(lib, kw, code):
    assert _call(lib, "mla_norm_append_kv", APPEND, **kw) == code


READ = dict(kv=_at(0), blocks=8, page=64, fmt=0, bt=_at(1), maxb=4, off=_at(2), starts=_at(3), batch=2, total=100, out=_at(4),
            os=576, dtype=0, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(blocks=0), 1), (dict(blocks=1 << 26), 1), (dict(page=16), 1), (dict(fmt=4), 1), (dict(fmt=-1), 1), (dict(dtype=2), 1),
    (dict(batch=-1), 1), (dict(maxb=0), 1), (dict(total=-1), 1), (dict(total=1 << 31), 1), (dict(os=568), 1), (dict(os=578), 1),
    (dict(fmt=2, os=504), 1), (dict(kv=None), 1), (dict(bt=None), 1), (dict(off=None), 1), (dict(out=None), 1), (dict(kv=ODD), 1),
    (dict(bt=ODD), 1), (dict(off=ODD), 1), (dict(starts=ODD), 1), (dict(out=ODD), 1), (dict(status=ODD), 1),
    (dict(total=0, kv=None, out=None), 0), (dict(batch=0, kv=None), 0), (dict(os=1 << 45), 1), (dict(out=_at(0)), 1),
    (dict(out=_into(0, 8 * 64 * 1152 - 16)), 1), (dict(out=_at(1)), 1), (dict(out=_at(3)), 1), (dict(status=_at(4)), 1),
])
def test_read_kv_argument_checks(lib, kw, code):
    assert _call(lib, "mla_read_kv", READ, **kw) == code


PREFILL = dict(q=_at(0), qt=192 * 8, qh=192, k=_at(1), kt=256 * 8, kh=256, r=_at(2), rs=64, v=_at(3), vt=256 * 8, vh=256, dtype=0,
               cq=_at(4), ck=_at(5), prefix=_at(6), batch=2, tq=5000, tk=5000, heads=8, scale=0.07, causal=1, out=_at(7),
               ot=128 * 8, oh=128, lse=_at(8), ws=_at(9), wb=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(tq=-1), 1), (dict(tk=-1), 1), (dict(batch=-1), 1), (dict(heads=0), 1), (dict(tq=1 << 31), 1), (dict(tk=1 << 31), 1),
    (dict(dtype=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(qt=184), 1), (dict(qh=184), 1), (dict(qt=1540), 1), (dict(kh=0), 1), (dict(kt=120), 1), (dict(vh=0), 1), (dict(vt=2052), 1),
    (dict(rs=56), 1), (dict(rs=0), 1), (dict(ot=120), 1), (dict(oh=0), 1), (dict(ot=128, oh=128), 1), (dict(qt=1 << 40), 1),
    (dict(vt=1 << 45), 1), (dict(rs=1 << 40), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(r=None), 1), (dict(v=None), 1), (dict(cq=None), 1), (dict(ck=None), 1),
    (dict(out=None), 1), (dict(lse=None), 1), (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(r=ODD), 1), (dict(v=ODD), 1), (dict(cq=ODD), 1),
    (dict(ck=ODD), 1), (dict(prefix=ODD), 1), (dict(out=ODD), 1), (dict(lse=ODD), 1), (dict(status=ODD), 1),
    (dict(tq=0, q=None, out=None, lse=None), 0), (dict(batch=0, q=None), 0),
    (dict(out=_at(0)), 1), (dict(out=_at(1)), 1), (dict(out=_at(2)), 1), (dict(out=_into(3, 16)), 1), (dict(lse=_at(7)), 1),
    (dict(lse=_at(4)), 1), (dict(status=_at(8)), 1), (dict(status=_at(6)), 1), (dict(heads=1 << 30, tq=1 << 15), 1),
    (dict(tq=4, ws=None), 1), (dict(tq=4, wb=64), 1), (dict(tq=4, ws=ODD), 1), (dict(tq=4, ws=_at(1)), 1),   # cut units need room
    (dict(tq=4, out=_at(9)), 1), (dict(scale=2.0 ** -101), 1), (dict(scale=2.0 ** 101), 1),
    (dict(tq=0, scale=2.0 ** -100), 0), (dict(tq=0, scale=2.0 ** 100), 0),
])
def test_prefill_argument_checks(lib, kw, code):
    assert _call(lib, "mla_prefill", PREFILL, **kw) == code


def test_prefill_workspace(lib):
    size = lib.mla_prefill_workspace_size
    assert size(0, 0, 1, 1) == 0 and size(-1, 5, 1, 1) == 0 and size(5, -1, 1, 1) == 0 and size(5, 5, 0, 1) == 0
    assert size(4096, 4096, 1, 128) == 0                       # units that fill the card
    assert size(4, 500, 1, 2) == 0                             # keys too short to cut
    for tq, tk, batch, heads in ((1, 5000, 1, 1), (32, 100000, 8, 16), (300, 9000, 2, 8)):
        got, row = size(tq, tk, batch, heads), tq * heads * 129 * 4
        assert got > row and got % row == 0 and got // row <= 16
    # the most that any sizes ask for: fewer than two cards' units, cut into up to two cards' pieces if their documents are
    # alike and up to twice as many if they are not
    most = max(size(tq, 1 << 20, b, h) for tq in (1, 255, 256, 257, 5000, 38912, 77000) for b in (1, 3, 200) for h in (1, 2, 7, 64, 151, 303))
    assert most <= 2 * 2 * 152 * 256 * 129 * 4


# ---------------------------------------------------------------------------
# the Python side
# ---------------------------------------------------------------------------
def _mla():
    import mla_latent_kv_14_gb300 as m
    return m


def _refused(f, *a, **kw):
    m = _mla()
    with pytest.raises(m.MLAError) as e:
        f(*a, **kw)
    assert e.value.status == 1
    return str(e.value)


def test_python_refuses_tensors():
    m = _mla()
    bf = torch.bfloat16
    x, pos, tab = torch.zeros(2, 3, 192, dtype=bf), torch.zeros(2, dtype=torch.int32), torch.zeros(8, 64)
    _refused(m.mla_norm_rotate, x, pos, tab)                                     # not on a cuda device
    _refused(m.mla_norm_rotate, x.float(), pos, tab)
    _refused(m.mla_norm_rotate, x[..., :56], pos, tab)
    _refused(m.mla_norm_rotate, x[..., ::2], pos, tab)
    kv, cache = torch.zeros(2, 576, dtype=bf), torch.zeros(2, 64, 1, 576, dtype=bf)
    _refused(m.mla_norm_append_kv, kv[:, :512], kv[:, 512:], None, cache, pos, pos, tab)
    _refused(m.mla_norm_append_kv, kv[:, :448], kv[:, 512:], None, cache, pos, pos, tab)
    _refused(m.mla_norm_append_kv, kv[:, :512], kv[:, 512:], None, cache, pos, pos, tab, kv_format=9)
    bt, off = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    _refused(m.mla_read_kv, cache, bt, off, total=4)
    _refused(m.mla_read_kv, cache, bt, off, total=4, dtype=torch.float16)       # a 16-bit cache in another type
    _refused(m.mla_read_kv, cache, bt, off, total=4, dtype=torch.float32)
    _refused(m.mla_read_kv, cache.float(), bt, off, total=4)
    _refused(m.mla_read_kv, cache, bt, off, total=4, kv_format=7)
    q, k, kr = torch.zeros(4, 2, 192, dtype=bf), torch.zeros(4, 2, 128, dtype=bf), torch.zeros(4, 64, dtype=bf)
    _refused(m.mla_prefill, q, k, kr, k, off, off, 0.1)
    _refused(m.mla_prefill, q, k.half(), kr, k, off, off, 0.1)
    _refused(m.mla_prefill, q[..., :128], k, kr, k, off, off, 0.1)
    _refused(m.mla_prefill, q, k[:, :1], kr, k, off, off, 0.1)
    _refused(m.mla_prefill, q, k, kr[:3], k, off, off, 0.1)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_norm_pins():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(oracle.rms_norm(x, eps=0.0), x / math.sqrt(12.5), rtol=1e-15)
    assert (oracle.rms_norm(np.zeros((1, 4))) == 0).all()
    y = oracle.rms_norm(np.random.default_rng(0).normal(size=(5, 96)), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0, rtol=1e-14)
    # the turned dims as complex numbers; the others as they were
    rng = np.random.default_rng(1)
    x, row = rng.normal(size=(3, 2, 200)), oracle.rope_table(3)
    for halves in (False, True):
        got, flat = oracle.norm_rotate(x, None, 1e-6, row, 56, halves), oracle.rms_norm(x)
        part = flat[..., 56:120]
        z = part[..., :32] + 1j * part[..., 32:] if halves else part[..., 0::2] + 1j * part[..., 1::2]
        z = z * (row[:, None, :32].astype(np.float64) + 1j * row[:, None, 32:])
        want = np.concatenate((z.real, z.imag), -1) if halves else np.stack((z.real, z.imag), -1).reshape(3, 2, 64)
        assert np.allclose(got[..., 56:120], want, atol=1e-14)
        assert (got[..., :56] == flat[..., :56]).all() and (got[..., 120:] == flat[..., 120:]).all()


@pytest.mark.parametrize("dim,at", [(64, 0), (192, 128), (576, 256)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_error_bound_holds_in_fp32(dim, at, halves):
    """An fp32 evaluation in numpy stays within the bound, and comes near enough to it that a wrong order of magnitude shows."""
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.normal(size=(200, 4, dim))).to(torch.bfloat16)
    w = torch.from_numpy(1 + 0.3 * rng.normal(size=dim)).to(torch.bfloat16)
    row = oracle.rope_table(200)
    want = oracle.norm_rotate(x, w, 1e-6, row, at, halves)
    bound = oracle.norm_rotate_error(oracle.rms_norm(x, w), at, halves)
    f = x.float().numpy()
    r = np.float32(1) / np.sqrt((f * f).sum(-1, keepdims=True, dtype=np.float32) / np.float32(dim) + np.float32(1e-6))
    y = f * r * w.float().numpy()
    t, c, s = y[..., at:at + 64], row[:, None, :32], row[:, None, 32:]
    a, b = (t[..., :32], t[..., 32:]) if halves else (t[..., 0::2], t[..., 1::2])
    lo, hi = a * c - b * s, a * s + b * c
    y[..., at:at + 64] = np.concatenate((lo, hi), -1) if halves else np.stack((lo, hi), -1).reshape(t.shape)
    assert (np.abs(y - want) <= bound).all()


def test_prefill_pins():
    rng = np.random.default_rng(3)
    q, kn, kr, v = rng.normal(size=(4, 2, 192)), rng.normal(size=(6, 2, 128)), rng.normal(size=(6, 64)), rng.normal(size=(6, 2, 128))
    assert oracle.visible(4, 6, True).tolist() == [3, 4, 5, 6] and oracle.visible(4, 6, False).tolist() == [6] * 4
    assert oracle.visible(4, 2, True).tolist() == [0, 0, 1, 2] and oracle.visible(4, 2, True, 1).tolist() == [1, 1, 1, 2]
    assert oracle.visible(3, 6, True, 9).tolist() == [6, 6, 6] and oracle.visible(2, 5, True, -4).tolist() == [4, 5]
    seen = oracle.visible(4, 6, True)
    out, lse, size, _ = oracle.prefill(q, kn, kr, v, 0.1, seen)
    k = np.concatenate((kn, np.repeat(kr[:, None], 2, 1)), -1)
    for i in range(4):                                   # plain loops, one key after another
        for h in range(2):
            e = [math.exp(0.1 * float(q[i, h] @ k[j, h])) for j in range(seen[i])]
            assert math.isclose(lse[i, h], math.log(sum(e)), rel_tol=1e-13)
            want = sum(w * v[j, h] for j, w in enumerate(e)) / sum(e)
            assert np.allclose(out[i, h], want, rtol=1e-12) and (np.abs(out[i, h]) <= size[i, h] + 1e-15).all()
    # one key: its value; equal keys: the mean, ln n more
    one = oracle.prefill(q, kn, kr, v, 0.1, np.ones(4, int))
    assert np.allclose(one[0], v[:1].repeat(4, 0)) and np.allclose(one[1], 0.1 * np.einsum("ihd,hd->ih", q, k[0]))
    same = oracle.prefill(q, kn[:1].repeat(6, 0), kr[:1].repeat(6, 0), v, 0.1, np.full(4, 6))
    assert np.allclose(same[0], v.mean(0)) and np.allclose(same[1], one[1] + math.log(6))
    none = oracle.prefill(q, kn, kr, v, 0.1, np.zeros(4, int))
    assert (none[0] == 0).all() and np.isneginf(none[1]).all()
    # the absorbed form of the decode gives the same: keys and values from a latent row
    c, w_uk, w_uv = rng.normal(size=(6, 512)), 0.05 * rng.normal(size=(2, 128, 512)), 0.05 * rng.normal(size=(2, 128, 512))
    kn, v = np.einsum("tc,hdc->thd", c, w_uk), np.einsum("tc,hdc->thd", c, w_uv)
    out, lse, _, _ = oracle.prefill(q, kn, kr, v, 0.1, np.full(4, 6))
    rows, qa = np.concatenate((c, kr), 1), np.concatenate((oracle.absorb_q(q[..., :128], w_uk), q[..., 128:]), -1)
    for i in range(4):
        lat, l2 = oracle.attend(qa[i], rows, 0.1)
        assert np.allclose(oracle.up_project(lat[None], w_uv)[0], out[i]) and np.allclose(l2, lse[i])


@pytest.mark.parametrize("dtype,half", [(torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)])
def test_prefill_error_bound_holds_for_rounded_weights(dtype, half):
    """fp32 scores and weights rounded to 16 bits, as a kernel forms them, stay within the bound."""
    rng = np.random.default_rng(5)
    n = 300
    q, kn = (torch.from_numpy(rng.normal(size=(20, 2, d)) * 1.5).to(dtype) for d in (192, 128))
    kn, v = (torch.from_numpy(rng.normal(size=(n, 2, 128))).to(dtype) for _ in range(2))
    kr = torch.from_numpy(rng.normal(size=(n, 64))).to(dtype)
    seen, scale = oracle.visible(20, n, True), 192 ** -0.5
    out, lse, size, dots = oracle.prefill(q, kn, kr, v, scale, seen)
    bo, bl = oracle.prefill_error(out, lse, size, dots, scale, seen, np.abs(oracle.to_f64(v)).sum(0), half, dtype == torch.float16)
    k = torch.cat((kn, kr[:, None].expand(-1, 2, -1)), -1).float()
    s = torch.einsum("ihd,jhd->ihj", q.float(), k)
    s = s.masked_fill(torch.arange(n) >= torch.from_numpy(seen)[:, None, None], -math.inf)
    p = torch.exp2((s - s.amax(-1, keepdim=True)) * (scale * 1.4426950408889634))
    total = p.sum(-1)
    o = (torch.einsum("ihj,jhd->ihd", p.to(dtype).float(), v.float()) / total[..., None]).to(dtype)
    got = s.amax(-1) * scale + total.log()
    assert (np.abs(oracle.to_f64(o) - out) <= bo).all() and (np.abs(oracle.to_f64(got) - lse) <= bl).all()
