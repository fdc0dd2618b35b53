"""GPU parity of the calls for prompts over the latent cache: norms with rotation,
the normalised append, rows read back and the attention of many new tokens,
against the 64-bit oracle; and a run of them together, as a prompt uses them.

Tolerances are the oracle's bounds of an fp32 evaluation plus half a step of the
result's type; rows read back are compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import mla_oracle
from tests.helpers import assert_close_attn

pytestmark = pytest.mark.gpu

mla = pytest.importorskip("mla_latent_kv_14_gb300")
DEV = "cuda"
PAGE = 64
BF, HF = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11}          # half a step, relative
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25}        # half a step of the subnormals
TABLE = oracle.rope_table(5000)
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mla.load_library()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _table():
    return torch.from_numpy(TABLE).to(DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _bits(status):
    torch.cuda.synchronize()
    return int(status.item())


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _close(got, want, bound, dtype, what=""):
    g = oracle.to_f64(got)
    off = np.abs(g - want) - (bound + HALF[dtype] * (np.abs(want) + bound) + TINY[dtype])
    assert np.isfinite(g).all() and (off <= 0).all(), f"{what}: {(off > 0).sum()} of {off.size}, worst {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("split", [0, 1])
@pytest.mark.parametrize("dtype,halves", [(BF, 0), (HF, 1), (BF, 1), (HF, 0)])
@pytest.mark.parametrize("dim,at", [(64, 0), (72, 8), (128, 0), (128, 64), (192, 128), (200, 56), (256, 96), (264, 200),
                                    (576, 512), (576, 0)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (5, 3), (37, 16)])
def test_norm_rotate(tokens, heads, dim, at, dtype, halves, split):
    g = _gen(tokens + dim)
    x = (torch.randn(tokens, heads, dim + 16, generator=g) * torch.exp2(2 * torch.randn(tokens, heads, 1, generator=g))).to(dtype)
    w = (1 + 0.3 * torch.randn(dim, generator=g)).to(dtype)
    pos = torch.randint(0, 5000, (tokens,), generator=g).int()
    dev, st = x.to(DEV)[..., 8:8 + dim], _status()
    want = oracle.norm_rotate(x[..., 8:8 + dim], w, 1e-6, TABLE[pos.numpy()], at, bool(halves))
    bound = oracle.norm_rotate_error(oracle.rms_norm(x[..., 8:8 + dim], w), at, bool(halves))
    if split:
        query = torch.full((tokens, heads, 576), 7.0, dtype=dtype, device=DEV)
        out, rope = mla.mla_norm_rotate(dev, pos.to(DEV), _table(), weight=w.to(DEV), rope_at=at, rope_out=query[..., 512:],
                                        rope_style=halves, status=st)
        assert (query[..., :512] == 7.0).all() and rope.data_ptr() == query[..., 512:].data_ptr()
        keep = np.r_[0:at, at + 64:dim]
        _close(rope, want[..., at:at + 64], bound[..., at:at + 64], dtype, "rope")
        _close(out, want[..., keep], bound[..., keep], dtype, "rest")
    else:
        out = mla.mla_norm_rotate(dev, pos.to(DEV), _table(), weight=w.to(DEV), rope_at=at, rope_style=halves, status=st)
        _close(out, want, bound, dtype)
    assert _bits(st) == 0


def test_norm_rotate_padding_positions_and_in_place():
    x = torch.randn(9, 4, 192, generator=_gen(3)).to(BF).to(DEV)
    pos = _ints([0, -1, 4999, 5000, 7, -2, 1 << 30, 3, 2])
    st = _status()
    out = torch.full_like(x, 3.0)
    mla.mla_norm_rotate(x, pos, _table(), out=out, status=st)
    assert _bits(st) == 1
    skipped = [1, 3, 5, 6]
    assert (out[skipped] == 3.0).all()
    want = oracle.norm_rotate(x, None, 1e-6, TABLE[np.clip(pos.cpu().numpy(), 0, 4999)], 128, False)
    live = [0, 2, 4, 7, 8]
    bound = oracle.norm_rotate_error(oracle.rms_norm(x), 128, False)
    _close(out[live], want[live], bound[live], BF)
    there = x.clone()
    back = mla.mla_norm_rotate(there, pos, _table(), out=there)
    assert back is there and torch.equal(there[live], out[live]) and torch.equal(there[skipped], x[skipped])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_norm_rotate_of_small_and_large_rows(dtype):
    """Rows of zeros, below eps, at the type's ends, heads-major and broadcast inputs."""
    size = torch.tensor([0.0, 2.0 ** -14, 2.0 ** -8, 1.0, 2.0 ** 8, 2.0 ** 14], dtype=torch.float64)
    x = (torch.rand(6, 3, 192, generator=_gen(1)) * 2 - 1).double() * size[:, None, None]
    x = x.to(dtype)
    pos = torch.arange(6, dtype=torch.int32)
    for eps in (0.0, 1e-6, 1e-2):
        rows = slice(0 if eps else 1, 6)
        heads_major = x[rows].transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
        want = oracle.norm_rotate(x[rows], None, eps, TABLE[pos[rows].numpy()], 128, False)
        bound = oracle.norm_rotate_error(oracle.rms_norm(x[rows], None, eps), 128, False)
        _close(mla.mla_norm_rotate(heads_major, pos[rows].to(DEV), _table(), eps=eps), want, bound, dtype, f"eps {eps}")
    shared = x[3:4, :1].to(DEV).expand(5, 7, 192)           # one row for all tokens and heads
    pos = torch.arange(5, dtype=torch.int32)
    want = oracle.norm_rotate(shared, None, 1e-6, TABLE[:5], 128, False)
    bound = oracle.norm_rotate_error(oracle.rms_norm(shared), 128, False)
    _close(mla.mla_norm_rotate(shared, pos.to(DEV), _table()), want, bound, dtype)


ENDS = [(2.0 ** 58, 2.0 ** 80), (2.0 ** 58, 2.0 ** -90), (2.0 ** -58, 2.0 ** -90), (2.0 ** -58, 2.0 ** 80), (2.0 ** 40, 2.0 ** 95)]


@pytest.mark.parametrize("dim,heads,tokens", [(192, 3, 5), (128, 1, 40), (576, 2, 9), (192, 64, 600), (128, 64, 600), (256, 2, 7)])
@pytest.mark.parametrize("size,weight", ENDS)
def test_norm_rotate_at_the_ends_of_bf16(size, weight, dim, heads, tokens):
    """Rows and weights whose product leaves fp32's range, or its normal numbers, where the result does not; the squares'
    sum stays within."""
    g = _gen(dim + tokens)
    x = (size * (1 + torch.rand(tokens, heads, dim, generator=g, dtype=torch.float64))).to(BF)
    w = (weight * (0.5 + torch.rand(dim, generator=g, dtype=torch.float64))).to(BF)
    pos = torch.randint(0, 5000, (tokens,), generator=g).int()
    want = oracle.norm_rotate(x, w, 0.0, TABLE[pos.numpy()], dim - 64, False)
    bound = oracle.norm_rotate_error(oracle.rms_norm(x, w, 0.0), dim - 64, False)
    _close(mla.mla_norm_rotate(x.to(DEV), pos.to(DEV), _table(), weight=w.to(DEV), eps=0.0), want, bound, BF)
    _close(mla.mla_norm_rotate(x.to(DEV), pos.to(DEV), _table(), eps=0.0),
           oracle.norm_rotate(x, None, 0.0, TABLE[pos.numpy()], dim - 64, False),
           oracle.norm_rotate_error(oracle.rms_norm(x, None, 0.0), dim - 64, False), BF, "no weight")

@pytest.mark.parametrize("tokens,heads,dim", [(1500, 128, 192), (4099, 3, 128), (11001, 3, 128), (9001, 1, 128), (700, 64, 576),
                                              (20001, 2, 64), (257, 128, 256)])
def test_norm_rotate_of_many_rows(tokens, heads, dim):
    """Both sides of the launch's rules; the reference in 64 bits on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(tokens, heads, dim, generator=g, device=DEV).to(BF)
    w = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(BF)
    pos = torch.randint(0, 5000, (tokens,), generator=g, device=DEV).int()
    out = mla.mla_norm_rotate(x, pos, _table(), weight=w)
    y = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    row = _table()[pos.long()].double()[:, None]
    a, b = y[..., -64::2], y[..., -63::2]
    turned = torch.stack((a * row[..., :32] - b * row[..., 32:], a * row[..., 32:] + b * row[..., :32]), -1).flatten(-2)
    size = torch.cat((y[..., :-64].abs(), 1.5 * (a.abs() + b.abs()).repeat_interleave(2, -1)), -1)
    y[..., -64:] = turned
    bound = (dim / 2 + 9) * 2.0 ** -24 * size
    assert ((out.double() - y).abs() <= bound + HALF[BF] * (y.abs() + bound)).all()


# ---------------------------------------------------------------------------
# the normalised append
# ---------------------------------------------------------------------------
def _grid(kind):
    table = mla_oracle.e4m3_value_table()[:127] if kind == "e4m3" else mla_oracle.e2m1_value_table()[:8]
    return np.asarray(table, np.float64)


def _is_rounding_of(value, x, slack, grid):
    """`value` (grid values with sign) is a rounding to nearest of something within `slack` of x (saturating)."""
    top = grid[-1]
    lo, hi = np.abs(x) - slack, np.abs(x) + slack
    mids = (grid[1:] + grid[:-1]) / 2
    at = np.searchsorted(grid, np.abs(value))
    assert (grid[at] == np.abs(value)).all()
    below = np.where(at > 0, mids[np.maximum(at - 1, 0)], -1.0)
    above = np.where(grid[at] < top, mids[np.minimum(at, len(mids) - 1)], np.inf)
    sign = (np.signbit(value) == np.signbit(x)) | (np.abs(x) <= slack) | (value == 0)
    return (hi >= below) & (lo <= above) & sign


def _check_rows(raw, want, bound, kv_format):
    """raw uint8 rows against the float64 values they should hold, which fp32 formed within `bound`."""
    n = len(raw)
    rel = 2.0 ** -23                                  # the scale's and the quotient's own roundings
    if kv_format == 1:
        amax = np.abs(want[:, :512]).reshape(n, 4, 128).max(-1)
        slack = bound[:, :512].reshape(n, 4, 128).max(-1)
        scale = raw[:, 512:528].copy().view("<f4").astype(np.float64)
        assert (np.abs(scale - amax / 448) <= (slack + rel * amax) / 448 + (amax == 0)).all()
        unit, grid, x = scale.repeat(128, 1), _grid("e4m3"), want[:, :512]
        codes = raw[:, :512]
        value = np.where(codes > 127, -1.0, 1.0) * grid[codes & 127]
    elif kv_format == 2:
        amax, slack = np.abs(want).reshape(n, 16, 32).max(-1), bound.reshape(n, 16, 32).max(-1)
        k = raw[:, 512:].astype(np.float64) - 127
        assert (448 * 2.0 ** k >= amax - slack).all()
        assert ((448 * 2.0 ** (k - 1) < amax + slack) | (k == -127)).all()
        unit, grid, x = (2.0 ** k).repeat(32, 1), _grid("e4m3"), want
        value = np.where(raw[:, :512] > 127, -1.0, 1.0) * grid[raw[:, :512] & 127]
    else:
        grid8 = _grid("e4m3")
        amax, slack = np.abs(want).reshape(n, 32, 16).max(-1), bound.reshape(n, 32, 16).max(-1)
        code = raw[:, 256:].astype(np.int64)
        v = grid8[code]
        assert ((6 * v >= amax - slack) | (code == 126)).all()
        assert ((code == 0) | (6 * grid8[np.maximum(code - 1, 0)] < amax + slack)).all()
        nibble = np.stack((raw[:, :256] & 15, raw[:, :256] >> 4), -1).reshape(n, 512)
        grid = _grid("e2m1")
        value = np.where(nibble > 7, -1.0, 1.0) * grid[nibble & 7]
        unit, x = v.repeat(16, 1), want
        unit = np.where(unit == 0, 2.0 ** -40, unit)      # a zero scale holds zeros
        value = np.where(v.repeat(16, 1) == 0, 0.0, value)
    q = x / unit
    q = np.clip(q, -grid[-1], grid[-1])
    b = (bound[:, :x.shape[1]] + rel * np.abs(x)) / unit
    assert _is_rounding_of(value, q, b, grid).all()


@pytest.mark.parametrize("with_rows", [0, 1])
@pytest.mark.parametrize("halves", [0, 1])
@pytest.mark.parametrize("fmt,dtype", [(0, BF), (0, HF), (1, BF), (2, BF), (3, BF)])
@pytest.mark.parametrize("n", [1, 63, 130])
def test_norm_append_kv(n, fmt, dtype, halves, with_rows):
    latent, pages, g = (448 if fmt >= 2 else 512), 5, _gen(n + fmt)
    kv = (torch.randn(n, latent + 64 + 8, generator=g) * torch.exp2(torch.randn(n, 1, generator=g) * 3)).to(dtype)
    if n > 20:
        kv[10] = 0
        kv[11, :latent] *= 1e-4
        kv[12, 3] = 3.0e4
    w = (1 + 0.3 * torch.randn(latent, generator=g)).to(dtype)
    w[7] = 0.0
    rng = np.random.default_rng(n)
    slots, pos = rng.permutation(pages * PAGE)[:n].astype(np.int32), rng.integers(0, 5000, n).astype(np.int32)
    bad = 0
    if n > 8:
        slots[[1, n - 1]] = -1
        slots[3], pos[5], pos[6], bad = pages * PAGE, 5000, -1, 1
    keep = (slots >= 0) & (slots < pages * PAGE) & (pos >= 0) & (pos < 5000)
    width = {0: 1152, 1: 656, 2: 528, 3: 288}[fmt]
    before = torch.randint(0, 256, (pages, PAGE, 1, width), dtype=torch.uint8, generator=_gen(7))
    cache = before.to(DEV)
    cache = cache.view(dtype) if fmt == 0 else cache
    rows = torch.full((n, latent + 64 + 8), 5.0, dtype=dtype, device=DEV) if with_rows else None
    dev, st = kv.to(DEV), _status()
    back = mla.mla_norm_append_kv(dev[:, :latent], dev[:, latent:latent + 64], w.to(DEV), cache, _ints(slots), _ints(pos),
                                  _table(), eps=1e-5, kv_format=fmt, rope_style=halves,
                                  rows=rows[:, :latent + 64] if with_rows else None, status=st)
    assert back is cache and _bits(st) == bad
    want = np.empty((n, latent + 64))
    want[:, :latent] = oracle.rms_norm(kv[:, :latent], w, 1e-5)
    row = TABLE[np.clip(pos, 0, 4999)]
    want[:, latent:] = oracle.rotate(kv[:, latent:latent + 64], row, bool(halves), exact=True)
    r32 = oracle.rotate(kv[:, latent:latent + 64], row, bool(halves))
    bound = (latent / 2 + 9) * 2.0 ** -24 * np.abs(want)
    bound[:, latent:] = np.abs(r32.astype(np.float64) - want[:, latent:])
    raw = cache.view(torch.uint8).cpu().view(pages * PAGE, -1).numpy()
    others = np.ones(pages * PAGE, bool)
    others[slots[keep]] = False
    assert (raw[others] == before.view(pages * PAGE, -1).numpy()[others]).all()
    got = raw[slots[keep]]
    rope = oracle.round_to(r32, dtype)[torch.from_numpy(keep)]
    if fmt == 0:
        held = torch.from_numpy(got).view(dtype)
        _close(held, want[keep], bound[keep], dtype)
        assert torch.equal(held[:, 512:], rope)
    else:
        _check_rows(got, want[keep], bound[keep], fmt)
        if fmt == 1:
            assert torch.equal(torch.from_numpy(got[:, 528:].copy()).view(BF), rope)
    if with_rows:
        rows = rows.cpu()
        assert (rows[~torch.from_numpy(keep)] == 5.0).all() and (rows[:, latent + 64:] == 5.0).all()
        _close(rows[torch.from_numpy(keep), :latent + 64], want[keep], bound[keep], dtype)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("size,weight", ENDS)
def test_norm_append_at_the_ends_of_bf16(size, weight, fmt):
    """As for the norm with rotation; 656-byte rows hold any size, 528-byte ones those that a UE8M0 scale does."""
    n, latent = 70, 448 if fmt == 2 else 512
    g = _gen(fmt)
    kv = torch.randn(n, latent + 64, generator=g, dtype=torch.float64)
    kv[:, :latent] = size * (1 + kv[:, :latent].abs().clamp(max=1))
    kv = kv.to(BF)
    w = (weight * (0.5 + torch.rand(latent, generator=g, dtype=torch.float64))).to(BF)
    width = {0: 576, 1: 656, 2: 528}[fmt]
    cache = torch.zeros(2, PAGE, 1, width, dtype=torch.uint8 if fmt else BF, device=DEV)
    rows = torch.empty(n, latent + 64, dtype=BF, device=DEV)
    at = torch.arange(n, dtype=torch.int32, device=DEV)
    dev = kv.to(DEV)
    mla.mla_norm_append_kv(dev[:, :latent], dev[:, latent:], w.to(DEV), cache, at, at, _table(), eps=0.0, kv_format=fmt, rows=rows)
    want = oracle.rms_norm(kv[:, :latent], w, 0.0)
    bound = (latent / 2 + 9) * 2.0 ** -24 * np.abs(want)
    _close(rows[:, :latent], want, bound, BF)
    if fmt == 0:
        assert torch.equal(cache.view(-1, 576)[:n], rows)
        return
    turned = oracle.rotate(kv[:, latent:], TABLE[:n], False, exact=True)
    r32 = oracle.rotate(kv[:, latent:], TABLE[:n], False)
    want, bound = np.concatenate((want, turned), 1), np.concatenate((bound, np.abs(r32.astype(np.float64) - turned)), 1)
    _check_rows(cache.view(-1, width)[:n].cpu().numpy(), want, bound, fmt)

def test_norm_append_of_unit_rows_is_the_append():
    """Rows whose norm is one and whose mean square is exact: the same bytes as mla_append_kv."""
    n = 64
    for fmt in range(4):
        latent = 448 if fmt >= 2 else 512
        kv = torch.where(torch.rand(n, latent + 64, generator=_gen(fmt)) < 0.5, 1.0, -1.0).to(BF).to(DEV)
        width, dt = {0: (576, BF), 1: (656, torch.uint8), 2: (528, torch.uint8), 3: (288, torch.uint8)}[fmt]
        a, b = (torch.zeros(1, PAGE, 1, width, dtype=dt, device=DEV) for _ in range(2))
        slots, pos = torch.arange(n, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
        mla.mla_append_kv(kv[:, :latent], kv[:, latent:], a, slots, pos, _table(), kv_format=fmt)
        mla.mla_norm_append_kv(kv[:, :latent], kv[:, latent:], None, b, slots, pos, _table(), eps=0.0, kv_format=fmt)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), fmt


# ---------------------------------------------------------------------------
# rows read back
# ---------------------------------------------------------------------------
def _cache(fmt, pages, seed, dtype=BF):
    """A cache with every kind of code, as a device tensor and as float64 rows."""
    g = _gen(seed)
    if fmt == 0:
        t = torch.randn(pages, PAGE, 1, 576, generator=g).to(dtype)
        return t.to(DEV), oracle.to_f64(t).reshape(-1, 576)
    rows = pages * PAGE
    if fmt == 1:
        raw = torch.randint(0, 256, (rows, 656), dtype=torch.uint8, generator=g)
        raw[:, :512][(raw[:, :512] & 127) == 127] = 0                        # no NaN codes
        raw[:, 512:528] = torch.exp2(12 * torch.randn(rows, 4, generator=g).clamp(-3, 1)).float().view(torch.uint8)
        raw[:, 528:] = torch.randn(rows, 64, generator=g).to(BF).view(torch.uint8)
    elif fmt == 2:
        raw = torch.randint(0, 256, (rows, 528), dtype=torch.uint8, generator=g)
        raw[:, :512][(raw[:, :512] & 127) == 127] = 0
        raw[:, 512:] = torch.randint(0, 133, (rows, 16), dtype=torch.uint8, generator=g)
    else:
        raw = torch.randint(0, 256, (rows, 288), dtype=torch.uint8, generator=g)
        raw[:, 256:] = torch.randint(0, 127, (rows, 32), dtype=torch.uint8, generator=g)
    return raw.view(pages, PAGE, 1, -1).to(DEV), oracle.cached_rows(raw.numpy(), fmt)


def _read_ref(rows, table, offsets, starts, total, width):
    want = np.full((total, width), 9.0)
    for b in range(len(offsets) - 1):
        for o in range(offsets[b], min(offsets[b + 1], total)):
            t = starts[b] + o - offsets[b]
            page = table[b][t // PAGE] if t // PAGE < len(table[b]) else -1
            want[o] = rows[page * PAGE + t % PAGE] if 0 <= page < len(rows) // PAGE else 0.0
    return want


@pytest.mark.parametrize("fmt,dtype", [(0, BF), (0, HF), (1, BF), (1, HF), (2, BF), (2, HF), (3, BF), (3, HF)])
@pytest.mark.parametrize("counts,starts", [([1], [0]), ([0, 0, 5, 0], [3, 0, 62, 1]), ([70, 1, 0, 129, 64], [0, 63, 9, 100, 64]),
                                           ([300], [17])])
def test_read_kv(fmt, dtype, counts, starts):
    batch = len(counts)
    reach = max(-(-(s + n) // PAGE) for s, n in zip(starts, counts)) + 1
    pages = batch * reach + 2
    cache, rows = _cache(fmt, pages, 3 + fmt, dtype)
    table = np.random.default_rng(1).permutation(pages)[:batch * reach].reshape(batch, reach).astype(np.int32)
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    total, width = int(offsets[-1]), rows.shape[1]
    st = _status()
    wide = torch.full((total + 3, width + 8), 9.0, dtype=dtype, device=DEV)
    got = mla.mla_read_kv(cache, _ints(table), _ints(offsets), starts=_ints(starts), kv_format=fmt, out=wide[:, :width], status=st)
    assert _bits(st) == 0 and got.data_ptr() == wide.data_ptr()
    want = _read_ref(rows, table, offsets, starts, total + 3, width)
    exact = torch.from_numpy(want).float().to(dtype)
    assert torch.equal(wide[:, :width].cpu().nan_to_num(1.5), exact.nan_to_num(1.5)) and (wide[:, width:] == 9.0).all()
    zero = [0] * batch
    if all(n <= reach * PAGE for n in counts):
        again = mla.mla_read_kv(cache, _ints(table), _ints(offsets), total=total, kv_format=fmt, dtype=dtype)
        assert torch.equal(again.cpu(), torch.from_numpy(_read_ref(rows, table, offsets, zero, total, width)).float().to(dtype))


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_read_kv_bad_pages_and_short_outputs(fmt):
    cache, rows = _cache(fmt, 4, 11)
    table = np.array([[2, 4, 1], [-1, 0, 3]], np.int32)          # pages 4 and -1 are none
    offsets, starts = np.array([0, 200, 330], np.int32), [10, 60]
    st = _status()
    out = torch.full((330, rows.shape[1]), 9.0, dtype=BF, device=DEV)
    mla.mla_read_kv(cache, _ints(table), _ints(offsets), starts=_ints(starts), kv_format=fmt, out=out, status=st)
    assert _bits(st) == 1                                        # tokens 192 .. 209 lie behind the table's row as well
    assert torch.equal(out.cpu(), torch.from_numpy(_read_ref(rows, table, offsets, starts, 330, rows.shape[1])).float().to(BF))
    st.zero_()
    short = mla.mla_read_kv(cache, _ints([[2, 1, 0]]), _ints([0, 150]), total=100, kv_format=fmt, status=st)
    assert _bits(st) == 0
    assert torch.equal(short.cpu(), torch.from_numpy(_read_ref(rows, [[2, 1, 0]], [0, 150], [0], 100, rows.shape[1])).float().to(BF))
    st.zero_()
    mla.mla_read_kv(cache, _ints([[2, 1, 0]]), _ints([0, 5]), total=5, starts=_ints([-3]), kv_format=fmt, status=st)
    assert _bits(st) == 1


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fmt", [1, 2, 3])
def test_read_kv_every_code_and_scale(fmt, dtype):
    """All code bytes beside all scale bytes (656-byte rows: scales over fp32's range and beyond), NaN among both."""
    byte = torch.arange(256, dtype=torch.uint8)
    n = {1: 241, 2: 512, 3: 256}[fmt]
    raw = torch.zeros(n, {1: 656, 2: 528, 3: 288}[fmt], dtype=torch.uint8)
    if fmt == 1:
        raw[:, :512] = byte.repeat(2)
        scale = torch.exp2(torch.arange(-160, 160).float().double()).float()
        scale = torch.cat((scale, 1.2345 * scale, -scale, torch.tensor([0.0, math.inf, -math.inf, math.nan])))
        raw[:, 512:528] = scale.view(n, 4).view(torch.uint8)
        raw[:, 528:] = torch.randn(n, 64, generator=_gen(1)).to(BF).view(torch.uint8)
    elif fmt == 2:
        raw[0::2, :512], raw[1::2, :512] = byte.repeat(2), byte.flip(0).roll(16).repeat(2)   # every code meets every scale
        for k in range(16):
            raw[:, 512 + k] = (torch.arange(n) // 2 + 16 * k).to(torch.uint8)
    else:
        raw[:, :256] = byte
        for k in range(32):
            raw[:, 256 + k] = (byte.long() + 8 * k).to(torch.uint8)
    cache = torch.zeros(-(-n // PAGE), PAGE, 1, raw.shape[1], dtype=torch.uint8)
    cache.view(-1, raw.shape[1])[:n] = raw
    table = _ints([list(range(len(cache)))])
    got = mla.mla_read_kv(cache.to(DEV), table, _ints([0, n]), total=n, kv_format=fmt, dtype=dtype).cpu()
    with np.errstate(invalid="ignore"):       # 0 times an infinite scale
        want = torch.from_numpy(oracle.cached_rows(raw.numpy(), fmt)).float().to(dtype)
    assert want.isnan().any() and want.isfinite().any()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1.5, 2.5, -2.5), want.nan_to_num(1.5, 2.5, -2.5))

@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_read_kv_leaves_rows_before_the_first_request(fmt):
    """Offsets that do not start at 0: some requests' part of a larger result."""
    cache, rows = _cache(fmt, 6, 13)
    table, offsets, starts = [[4, 1], [0, 5]], [37, 90, 131], [3, 70]
    st = _status()
    out = torch.full((140, rows.shape[1]), 9.0, dtype=BF, device=DEV)
    mla.mla_read_kv(cache, _ints(table), _ints(offsets), starts=_ints(starts), kv_format=fmt, out=out, status=st)
    assert _bits(st) == 0
    assert torch.equal(out.cpu(), torch.from_numpy(_read_ref(rows, table, offsets, starts, 140, rows.shape[1])).float().to(BF))


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_read_kv_gives_what_the_append_wrote(fmt):
    n, latent = 500, 448 if fmt >= 2 else 512
    kv = torch.randn(n, latent + 64, generator=_gen(2)).to(BF).to(DEV)
    w = {0: 576, 1: 656, 2: 528, 3: 288}[fmt]
    cache = torch.zeros(9, PAGE, 1, w, dtype=torch.uint8 if fmt else BF, device=DEV)
    table = torch.randperm(9, generator=_gen(5))[:8].int()
    pos = torch.arange(n)
    slots = (table[pos // PAGE] * PAGE + pos % PAGE).int().to(DEV)
    rows = torch.empty(n, latent + 64, dtype=BF, device=DEV)
    mla.mla_norm_append_kv(kv[:, :latent], kv[:, latent:], None, cache, slots, pos.int().to(DEV), _table(), kv_format=fmt, rows=rows)
    back = mla.mla_read_kv(cache, table.view(1, -1).to(DEV), _ints([0, n]), total=n, kv_format=fmt)
    if fmt == 0:
        assert torch.equal(back, rows)
    else:
        raw = cache.view(-1, w)[slots.long()].cpu().numpy()
        assert torch.equal(back.cpu(), torch.from_numpy(oracle.cached_rows(raw, fmt)).float().to(BF))


# ---------------------------------------------------------------------------
# attention of many new tokens: documents of up to 256 queries on average take one CTA a unit, others two; a long
# document more (`extra`) takes a test's documents to the other side
# ---------------------------------------------------------------------------
LONG = [(1900, 1900)]
both_kernels = pytest.mark.parametrize("extra", [[], LONG], ids=["few", "pair"])


def _inputs(lens, heads, dtype, seed, spread=1.5):
    g = _gen(seed)
    n_q, n_k = sum(a for a, _ in lens), sum(b for _, b in lens)
    q = (spread * torch.randn(n_q, heads, 192, generator=g)).to(dtype)
    kv = torch.randn(n_k, heads, 256, generator=g).to(dtype)
    kr = torch.randn(n_k, 64, generator=g).to(dtype)
    cu_q = np.concatenate(([0], np.cumsum([a for a, _ in lens]))).astype(np.int32)
    cu_k = np.concatenate(([0], np.cumsum([b for _, b in lens]))).astype(np.int32)
    return q, kv, kr, cu_q, cu_k


def _check(out, lse, q, kv, kr, cu_q, cu_k, causal, prefix, dtype, docs=None, heads=None, rows=None, scale=SCALE):
    """Documents (all), heads (all) and query rows (all) against the oracle."""
    heads = list(range(q.shape[1])) if heads is None else heads
    for b in range(len(cu_q) - 1) if docs is None else docs:
        a, z, c, d = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        seen = oracle.visible(z - a, d - c, causal, 0 if prefix is None else int(prefix[b]))
        if rows is None:     # all of a short document, the edges of a long one's blocks
            pick = np.arange(z - a)
            if z - a > 420:
                pick = np.array([r for r in range(z - a) if r % 128 in (0, 1, 126, 127) or r == z - a - 1][::3] + [z - a - 1])
        else:
            pick = np.array([r for r in rows if r < z - a], dtype=np.int64)
        if len(pick) == 0:
            continue
        ro, rl, size, dots = oracle.prefill(q[a:z][pick][:, heads], kv[c:d][:, heads, :128], kr[c:d], kv[c:d][:, heads, 128:],
                                            scale, seen[pick])
        total = np.zeros(128)
        if d > c:
            total = np.abs(oracle.to_f64(kv[c:d][:, heads, 128:])).sum(axis=0)     # [heads, 128]
        bo, bl = oracle.prefill_error(ro, rl, size, dots, scale, seen[pick], total, HALF[dtype], dtype == HF)
        go, gl = oracle.to_f64(out[a:z].cpu()[pick][:, heads]), oracle.to_f64(lse[a:z].cpu()[pick][:, heads])
        assert np.isfinite(go).all()
        off = np.abs(go - ro) - bo - TINY[dtype]
        assert (off <= 0).all(), f"document {b}: {(off > 0).sum()} of {off.size}, worst {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
        none = np.isneginf(rl)
        assert (np.isneginf(gl) == none).all() and (go[none] == 0).all()
        assert (np.abs(np.where(none, 0, gl) - np.where(none, 0, rl)) <= np.where(none, 0, bl)).all(), f"document {b}: lse"


def _run(q, kv, kr, cu_q, cu_k, causal, prefix=None, **kw):
    dkv = kv.to(DEV)
    st = _status()
    out, lse = mla.mla_prefill(q.to(DEV), dkv[..., :128], kr.to(DEV), dkv[..., 128:], _ints(cu_q), _ints(cu_k),
                               kw.pop("scale", SCALE), causal=causal, prefix_lens=None if prefix is None else _ints(prefix),
                               status=st, **kw)
    assert _bits(st) == 0
    return out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads", [([(1, 1)], 1), ([(5, 5)], 2), ([(128, 128)], 1), ([(129, 129)], 3), ([(256, 384)], 2),
                                        ([(300, 300), (1, 77), (64, 640)], 2), ([(40, 1000), (257, 257)], 4),
                                        ([(257, 257)], 2), ([(384, 400)], 1), ([(512, 512)], 2), ([(513, 640), (300, 1000)], 2),
                                        ([(900, 900), (1, 77), (64, 640)], 2), ([(1025, 1100)], 1)])
def test_prefill(lens, heads, causal, dtype):
    case = _inputs(lens, heads, dtype, 3 + heads)
    out, lse = _run(*case, causal)
    _check(out, lse, *case, causal, None, dtype)


@pytest.mark.parametrize("lens", [[(0, 0), (3, 0), (0, 5), (7, 3), (0, 0)], [(200, 70), (130, 129), (2, 1)], [(0, 9), (0, 0)]])
@pytest.mark.parametrize("causal", [True, False])
@both_kernels
def test_prefill_of_empty_documents_and_rows(lens, causal, extra):
    """Documents without queries or keys, causal queries that see nothing."""
    lens = lens + [(2600, 900)] * len(extra) + [(0, 3)]
    case = _inputs(lens, 3, BF, 5)
    out, lse = _run(*case, causal)
    _check(out, lse, *case, causal, None, BF)


def test_prefill_without_any_key():
    q = torch.randn(5, 2, 192, generator=_gen(1)).to(BF).to(DEV)
    none = torch.empty(0, 2, 128, dtype=BF, device=DEV)
    out, lse = mla.mla_prefill(q, none, torch.empty(0, 64, dtype=BF, device=DEV), none, _ints([0, 5]), _ints([0, 0]), SCALE)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = mla.mla_prefill(q[:0], none, torch.empty(0, 64, dtype=BF, device=DEV), none, _ints([0, 0]), _ints([0, 0]), SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)


@pytest.mark.parametrize("dtype", [BF, HF])
@both_kernels
def test_prefill_prefixes(dtype, extra):
    """Prefixes of none, some and all keys, and beyond them; queries before the keys' start see the prefix alone."""
    lens, prefix = [(300, 300), (129, 129), (50, 400), (64, 64), (90, 30), (7, 7)], [0, 100, 390, 64, 11, 1 << 30]
    lens, prefix = lens + extra, prefix + [777] * len(extra)
    case = _inputs(lens, 2, dtype, 9)
    out, lse = _run(*case, True, prefix)
    _check(out, lse, *case, True, prefix, dtype)
    out, lse = _run(*case, True, [-5] * len(lens))
    _check(out, lse, *case, True, [0] * len(lens), dtype)
    out, lse = _run(*case, False, prefix)
    _check(out, lse, *case, False, None, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,heads", [([(1, 5000)], 1), ([(4, 4100), (3, 130), (1, 1), (130, 2600)], 2), ([(260, 9000)], 1), ([(700, 6000), (64, 3000)], 1)])
def test_prefill_of_few_rows_over_long_keys(lens, heads, dtype):
    """Units that are cut along the keys and joined."""
    case = _inputs(lens, heads, dtype, 13)
    n_q, n_k = case[0].shape[0], case[1].shape[0]
    assert mla.load_library().mla_prefill_workspace_size(n_q, n_k, len(lens), heads) > 0
    for causal in (True, False):
        out, lse = _run(*case, causal)
        _check(out, lse, *case, causal, None, dtype, rows=[0, 1, 2, 3, 127, 128, 129, 255, 259])


def test_prefill_scores_that_grow_and_shrink():
    """The running maximum moves in every key tile, in steps on both sides of the lazy limit, or never."""
    heads, n = 4, 900
    q, kv, kr, cu_q, cu_k = _inputs([(n, n)], heads, BF, 17)
    step = torch.tensor([0.02, 0.2, -0.2, 0.0])
    q[:, :, 0] = 8.0
    kv[:, :, 0] = (torch.arange(n)[:, None] * step).to(BF)
    out, lse = _run(q, kv, kr, cu_q, cu_k, True)
    _check(out, lse, q, kv, kr, cu_q, cu_k, True, None, BF)
    out, lse = _run(q, kv, kr, cu_q, cu_k, False)
    _check(out, lse, q, kv, kr, cu_q, cu_k, False, None, BF)


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-6, 30.0])
@both_kernels
def test_prefill_scales(scale, extra):
    """Weights that are all alike, and rows that a single key takes."""
    lens = [(40, 300), (129, 129)] + extra
    case = _inputs(lens, 2, BF, 18)
    out, lse = _run(*case, True, scale=scale)
    _check(out, lse, *case, True, None, BF, scale=scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@both_kernels
def test_prefill_is_not_reached_by_what_lies_outside(bad, extra):
    """Keys, values and queries behind, before and between the documents poisoned; rows of no document stay."""
    lens = [(70, 70), (33, 200), (150, 150)] + extra
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, BF, 19)
    pad = 40
    # the middle document becomes a gap that no offsets name: a document of its own with poisoned rows
    q2, kv2, kr2 = (torch.full((t.shape[0] + 2 * pad, *t.shape[1:]), bad, dtype=BF) for t in (q, kv, kr))
    q2[pad:-pad], kv2[pad:-pad], kr2[pad:-pad] = q, kv, kr
    kv2[pad + 70:pad + 270] = bad
    kr2[pad + 70:pad + 270] = bad
    out = torch.full((q2.shape[0], 2, 128), 6.0, dtype=BF, device=DEV)
    lse = torch.full((q2.shape[0], 2), 6.0, device=DEV)
    _run(q2, kv2, kr2, cu_q + pad, cu_k + pad, True, out=out, lse=lse)
    assert (out[:pad] == 6.0).all() and (out[-pad:] == 6.0).all() and (lse[:pad] == 6.0).all() and (lse[-pad:] == 6.0).all()
    _check(out[pad:], lse[pad:], q, kv, kr, cu_q, cu_k, True, None, BF, docs=[0, 2, 3][:2 + len(extra)])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens", [[(900, 900)], [(1024, 1300)], [(100, 900), (256, 256)], [(130, 6000)]], ids=["pair", "pair prefix", "few", "cut"])
def test_prefill_keys_that_a_query_does_not_see(lens, bad):
    """A key that is not finite reaches only the queries that see it; a value only those that miss it by less than 383."""
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, BF, 61)
    n_q, n_k = lens[0]
    seen = oracle.visible(n_q, n_k, True)
    ref, ref_l = _run(q, kv, kr, cu_q, cu_k, True)
    j = n_k - n_q // 3
    for where in ("key", "rope", "value"):
        kv2, kr2 = kv.clone(), kr.clone()
        if where == "rope":
            kr2[j] = bad
        else:
            kv2[j, :, :128 if where == "key" else 256] = bad
            if where == "value":
                kv2[j, :, :128] = kv[j, :, :128]
        out, lse = _run(q, kv2, kr2, cu_q, cu_k, True)
        apart = torch.from_numpy(seen + (382 if where == "value" else 0) <= j)
        first, rest = slice(0, n_q), slice(n_q, None)
        assert torch.equal(out[first][apart], ref[first][apart]) and torch.equal(lse[first][apart], ref_l[first][apart])
        assert torch.equal(out[rest], ref[rest]) and torch.equal(lse[rest], ref_l[rest])
        sees = torch.from_numpy(seen > j)
        assert where != "value" or (~out[first][sees].isfinite()).all()
        assert where != "value" or torch.equal(lse, ref_l)


@both_kernels
def test_prefill_strides(extra):
    """Heads-major inputs and outputs, column ranges, one head of a wider tensor."""
    lens, heads = [(140, 140), (20, 150)] + extra, 3
    q, kv, kr, cu_q, cu_k = _inputs(lens, heads, HF, 23)
    ref, ref_l = _run(q, kv, kr, cu_q, cu_k, True)
    qt = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    kt = kv[..., :128].transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    wide = torch.zeros(kv.shape[0], heads, 136, dtype=HF, device=DEV)
    wide[..., :128] = kv[..., 128:].to(DEV)
    rope = torch.zeros(kv.shape[0], 576, dtype=HF, device=DEV)
    rope[:, 512:] = kr.to(DEV)
    out = torch.full((heads, q.shape[0], 192), 2.0, dtype=HF, device=DEV)
    got, lse = mla.mla_prefill(qt, kt, rope[:, 512:], wide[..., :128], _ints(cu_q), _ints(cu_k), SCALE, out=out.transpose(0, 1)[..., 64:])
    assert torch.equal(got, ref) and torch.equal(lse, ref_l) and (out[..., :64] == 2.0).all()
    one, one_l = mla.mla_prefill(qt[:, 1:2], kt[:, 1:2], rope[:, 512:], wide[:, 1:2, :128], _ints(cu_q), _ints(cu_k), SCALE)
    _check(one, one_l, q[:, 1:2], kv[:, 1:2], kr, cu_q, cu_k, True, None, HF)


@pytest.mark.parametrize("lens", [[(140, 140), (20, 150)], [(700, 700), (300, 333)], [(5, 6000)], [(300, 9000)]],
                         ids=["few", "pair", "few cut", "pair cut"])
def test_prefill_of_other_alignment(lens):
    """Outputs and a workspace that are 16-byte aligned and no more."""
    heads = 2
    q, kv, kr, cu_q, cu_k = _inputs(lens, heads, BF, 25)
    ref, ref_l = _run(q, kv, kr, cu_q, cu_k, True)
    tq, tk = q.shape[0], kv.shape[0]
    wide = torch.full((tq, heads, 136), 3.0, dtype=BF, device=DEV)
    out, lse = _run(q, kv, kr, cu_q, cu_k, True, out=wide[..., 8:])
    assert torch.equal(out, ref) and torch.equal(lse, ref_l) and (wide[..., :8] == 3.0).all()
    lib = mla.load_library()
    size = lib.mla_prefill_workspace_size(tq, tk, len(lens), heads)
    space = torch.empty(size + 64, dtype=torch.uint8, device=DEV)
    space = space[(16 - space.data_ptr() % 32) % 32:]
    assert space.data_ptr() % 32 == 16
    dq, dkv, dkr, cq, ck = q.to(DEV), kv.to(DEV), kr.to(DEV), _ints(cu_q), _ints(cu_k)
    out, lse = torch.zeros_like(ref), torch.zeros_like(ref_l)
    code = lib.mla_prefill(dq.data_ptr(), heads * 192, 192, dkv.data_ptr(), heads * 256, 256, dkr.data_ptr(), 64, dkv.data_ptr() + 256,
                           heads * 256, 256, 0, cq.data_ptr(), ck.data_ptr(), None, len(lens), tq, tk, heads, SCALE, 1, out.data_ptr(),
                           heads * 128, 128, lse.data_ptr(), space.data_ptr(), size, None, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_l)


@pytest.mark.parametrize("heads", [1, 20])
@pytest.mark.parametrize("most", [300, 800])
def test_prefill_of_many_documents(heads, most):
    """More documents than a warp looks at together, more units than blocks at once; the same bits every time."""
    rng = np.random.default_rng(4)
    lens = [(int(a), int(a) + int(b)) for a, b in zip(rng.integers(0, most, 75), rng.integers(0, 40, 75))]
    case = _inputs(lens, heads, BF, 29)
    out, lse = _run(*case, True)
    _check(out, lse, *case, True, None, BF, heads=[0, heads - 1][:heads], rows=[0, 1, 60, 127, 128, 200, 255, 256, 299, 511, 512, 700])
    for _ in range(8):
        again = _run(*case, True)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("most", [3, 600])
def test_prefill_of_a_large_batch(most):
    """Thousands of documents, many of them empty."""
    rng = np.random.default_rng(6)
    n = 5000 if most == 3 else 1300
    lens = [(int(a), int(a) + int(b)) for a, b in zip(rng.integers(0, most, n) * rng.integers(0, 2, n), rng.integers(0, 30, n))]
    lens[-1] = (most, most + 9)
    case = _inputs(lens, 1, BF, 67)
    out, lse = _run(*case, True)
    _check(out, lse, *case, True, None, BF, docs=list(range(0, n, 37)) + [n - 2, n - 1], rows=[0, 1, 2, 200, 511, 599])


def test_prefill_of_long_documents_sampled():
    lens, heads = [(2500, 2500), (700, 5000)], 16
    case = _inputs(lens, heads, BF, 31)
    out, lse = _run(*case, True)
    _check(out, lse, *case, True, None, BF, heads=[0, 7, 15], rows=[0, 127, 128, 255, 256, 511, 699, 1300, 2303, 2304, 2499])


@pytest.mark.parametrize("k", [1, 30])
def test_prefill_bad_offsets(k):
    """Documents whose offsets descend or leave the tensors are skipped and recorded; the others are right."""
    lens = [(40 * k, 40 * k), (30 * k, 30 * k), (20 * k, 20 * k)]
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, BF, 37)
    ref, ref_l = _run(q, kv, kr, cu_q, cu_k, True)
    for cq, ck, good in (([0, 40, 95, 90], cu_k, [0]), ([0, 40, 70, 91], cu_k, [0, 1]), (cu_q, [0, 40, 70, 1 << 30], [0, 1]),
                         ([-1, 40, 70, 90], cu_k, [1, 2]), (cu_q, [0, 40, -7, 90], [0])):
        cq, ck = ([x if abs(x) in (1, 7, 91, 1 << 30) else x * k for x in c] if isinstance(c, list) else c for c in (cq, ck))
        cq = [x if x != 91 else 90 * k + 1 for x in cq]
        st = _status()
        dkv = kv.to(DEV)
        out, lse = torch.full_like(ref, 4.0), torch.full_like(ref_l, 4.0)
        mla.mla_prefill(q.to(DEV), dkv[..., :128], kr.to(DEV), dkv[..., 128:], _ints(cq), _ints(ck), SCALE, out=out, lse=lse, status=st)
        assert _bits(st) == 1
        for b in range(3):
            rows = slice(cu_q[b], cu_q[b + 1])
            if b in good:
                assert torch.equal(out[rows], ref[rows]) and torch.equal(lse[rows], ref_l[rows])
            else:
                assert (out[rows] == 4.0).all() and (lse[rows] == 4.0).all()


@pytest.mark.parametrize("n", [20, 300])
def test_prefill_timeout_is_reported(n):
    case = _inputs([(n, n)], 1, BF, 41)
    q, kv, kr = (t.to(DEV) for t in case[:3])
    st = _status()
    mla.mla_set_test_stall(2000000)
    try:
        mla.mla_prefill(q, kv[..., :128], kr, kv[..., 128:], _ints(case[3]), _ints(case[4]), SCALE, status=st)
        assert _bits(st) == 2
    finally:
        mla.mla_set_test_stall(0)
    out, lse = _run(*case, True)
    _check(out, lse, *case, True, None, BF)


def test_prefill_same_inputs_same_bits():
    for lens, heads in (([(700, 1900), (300, 300)], 8), ([(3, 6000)], 4), ([(5, 200)] * 60 + [(130, 150)] * 30, 16),
                        ([(300, 310), (900, 900)] * 12, 16)):
        case = _inputs(lens, heads, BF, 43)
        first = _run(*case, True)
        for _ in range(3):
            again = _run(*case, True)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("lens,heads", [([(300, 300), (64, 500)], 4), ([(2, 5000)], 2), ([(700, 9000)], 1)])
def test_prompt_calls_captured_and_on_another_stream(lens, heads):
    """Norm, read and attention captured into a graph, replayed with new inputs while the same calls run eagerly beside
    it: cut units take their partial results' memory from the graph's own pool."""
    q, kv, kr, cu_q, cu_k = _inputs(lens, heads, BF, 47)
    q, kv, kr = q.to(DEV), kv.to(DEV), kr.to(DEV)
    cq, ck, pos, table = _ints(cu_q), _ints(cu_k), torch.arange(q.shape[0], dtype=torch.int32, device=DEV), _table()
    cache = torch.randn(8, PAGE, 1, 576, generator=_gen(1)).to(BF).to(DEV)
    bt, offsets = _ints([[3, 1, 7], [0, 2, 5]]), _ints([0, 130, 300])

    def calls(x):
        y = mla.mla_norm_rotate(x, pos, table)
        rows = mla.mla_read_kv(cache, bt, offsets, total=300)
        return (y, rows, *mla.mla_prefill(y, kv[..., :128], kr, kv[..., 128:], cq, ck, SCALE))

    calls(q)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls(q)
    for step in range(3):
        q.copy_(torch.randn(q.shape, generator=_gen(step)).to(BF))
        cache.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(stream):
            beside = calls(q)
        torch.cuda.synchronize()
        for a, b in zip(held, beside):
            assert torch.equal(a, b)


def test_prompt_calls_on_two_streams_at_once():
    """Both kernels of the attention, and cut units, in flight together."""
    cases = [([(600, 900), (900, 900)], 4), ([(3, 5000)], 2), ([(100, 1000)] * 20, 4), ([(700, 9000)], 1)]
    cases = [[x.to(DEV) for x in c[:3]] + [_ints(x) for x in c[3:]] for c in (_inputs(lens, heads, BF, 59) for lens, heads in cases)]

    def run(c):
        q, kv, kr, cq, ck = c
        return mla.mla_prefill(q, kv[..., :128], kr, kv[..., 128:], cq, ck, SCALE)

    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append([run(c) for _ in range(6)])
        torch.cuda.synchronize()
        for (out, lse), runs in zip(alone, got):
            assert all(torch.equal(out, a) and torch.equal(lse, b) for a, b in runs)


# ---------------------------------------------------------------------------
# the ends of the scores' range
# ---------------------------------------------------------------------------
U = 2.0 ** -24
FAR_LENS = {"few": [(40, 700), (129, 129)], "pair": [(600, 700)]}


def _far_check(out, lse, q, kv, kr, lens, scale, spread, dtype):
    """Against the oracle, for dots that fp32 holds exactly. With x = c (s - m), c = scale log2 e: c rounds (U of x, with
    scale a power of two), the difference and the product too, the reference's own rounding (2^-13 ln 2 at most, where it
    is not subtracted first) counts twice where the reference has moved, and 2^x is off by 4U: a weight by 4U + 3U |x| +
    2^-12 of itself, |x| <= 2 * spread for scores that lie `spread` apart. Weights of 2^-32 and less of the largest may
    be lost in fp16."""
    q0 = k0 = 0
    for n_q, n_k in lens:
        seen = oracle.visible(n_q, n_k, True)
        pick = np.unique(np.r_[0, 1, n_q // 2, np.arange(min(n_q, 127), n_q, 64), n_q - 1])
        ro, rl, size, _ = oracle.prefill(q[q0:q0 + n_q][pick], kv[k0:k0 + n_k, :, :128], kr[k0:k0 + n_k],
                                         kv[k0:k0 + n_k, :, 128:], scale, seen[pick])
        n = seen[pick].astype(np.float64)[:, None]
        weight = (4 + 6 * spread) * U + 2.0 ** -12
        rel = 2 * weight + (2 * n + 64) * U
        bo = 1.01 * HALF[dtype] * np.abs(ro) + (HALF[dtype] + rel)[..., None] * size
        if dtype == HF:
            bo = bo + 2.0 ** -32 * np.abs(oracle.to_f64(kv[k0:k0 + n_k, :, 128:])).sum(0)
        bl = weight + (n + 64) * U + 4 * U * np.abs(rl)
        go, gl = oracle.to_f64(out[q0:q0 + n_q].cpu()[pick]), oracle.to_f64(lse[q0:q0 + n_q].cpu()[pick])
        assert np.isfinite(go).all()
        off = np.abs(go - ro) - bo - TINY[dtype]
        assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size}, worst {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
        inside = np.abs(rl) < 3.4e38
        assert (gl[~inside] == np.sign(rl[~inside]) * np.inf).all()
        assert (np.abs(np.where(inside, gl, 0) - np.where(inside, rl, 0)) <= bl).all()
        q0, k0 = q0 + n_q, k0 + n_k


def _far_inputs(lens, dtype, level, seed):
    """Queries and keys of one dim: the scaled scores are 2^(level - 6) times whole numbers up to 61, many of them alike;
    the dots, whole numbers times a power of two, are exact."""
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, dtype, seed)
    q[:], kv[..., :128], kr[:] = 0, 0, 0
    top = 60 if level > 120 else 7                     # bf16 reaches scores whose scaled value fp32 cannot hold
    q[..., 5] = 2.0 ** top
    steps = torch.randint(3, 62, (kv.shape[0], 2), generator=_gen(seed))     # ends whose product with a scale rounds
    kv[..., 5] = (steps * 2.0 ** 3).to(dtype)
    return (q, kv, kr, cu_q, cu_k), 2.0 ** (level - 6 - 3 - top)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("level,dtype", [(16, BF), (20, HF), (24, BF), (27, HF), (28, BF), (28, HF), (30, HF), (32, BF), (32, HF),
                                         (100, BF), (100, HF), (140, BF)])
@pytest.mark.parametrize("kind", ["few", "pair"])
def test_prefill_scores_of_any_size(kind, level, dtype, sign):
    """Scaled scores up to 2^level, far beyond where the product of reference and scale is exact, many of them alike: the
    largest share the weight. Beyond fp32's range lse is infinite, out is not."""
    lens = FAR_LENS[kind]
    (q, kv, kr, cu_q, cu_k), scale = _far_inputs(lens, dtype, level, 71)
    q *= sign
    out, lse = _run(q, kv, kr, cu_q, cu_k, True, scale=scale)
    _far_check(out, lse, q, kv, kr, lens, scale, 0.0, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("level", [8, 11, 12, 13, 16, 20])
@pytest.mark.parametrize("kind", ["few", "pair"])
def test_prefill_scores_around_a_large_one(kind, level, dtype):
    """Scaled scores 2^level + t / 2, t up to 31: weights that count, on both sides of where the reference is subtracted
    first. The second half of the keys lies 2^level higher, so that rows cross over on the way."""
    lens = FAR_LENS[kind]
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, dtype, 73)
    q[:], kv[..., :128], kr[:] = 0, 0, 0
    n = kv.shape[0]
    half = level // 2
    q[..., 0], q[..., 1] = 2.0 ** half, 1.0
    kv[..., 0] = 2.0 ** (level - half)
    kv[..., 1] = (torch.randint(0, 32, (n, 2), generator=_gen(3)) * 0.5).to(dtype)
    for case in range(2):
        if case:
            kv[n // 2:, :, 0] *= 2
        out, lse = _run(q, kv, kr, cu_q, cu_k, True, scale=1.0)
        _far_check(out, lse, q, kv, kr, lens, 1.0, 16.0, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [[(5, 6000)], [(300, 9000)], [(3, 4100), (130, 2600)]], ids=["few", "pair", "ragged"])
def test_prefill_cut_units_of_large_scores(lens, dtype):
    """Largest scores that are alike in several pieces of a unit weigh by how many there are, however large they are; and
    scores around a large one."""
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, dtype, 79)
    assert mla.load_library().mla_prefill_workspace_size(q.shape[0], kv.shape[0], len(lens), 2) > 0
    for level in (13, 20, 28, 100):
        (q, kv, kr, cu_q, cu_k), scale = _far_inputs(lens, dtype, level, 79)
        out, lse = _run(q, kv, kr, cu_q, cu_k, True, scale=scale)
        _far_check(out, lse, q, kv, kr, lens, scale, 0.0, dtype)
    for level in (10, 20):
        q[:], kv[..., :128], kr[:] = 0, 0, 0
        q[..., 0], q[..., 1] = 2.0 ** (level // 2), 1.0
        kv[..., 0] = 2.0 ** (level - level // 2)
        kv[..., 1] = (torch.randint(0, 32, (kv.shape[0], 2), generator=_gen(3)) * 0.5).to(dtype)
        out, lse = _run(q, kv, kr, cu_q, cu_k, True, scale=1.0)
        _far_check(out, lse, q, kv, kr, lens, 1.0, 16.0, dtype)


@pytest.mark.parametrize("lens", [[(40, 700)], [(600, 700)], [(5, 6000)], [(300, 9000)]], ids=["few", "pair", "few cut", "pair cut"])
def test_prefill_dots_below_fp32(lens):
    """A query all of whose dots are -inf gets NaN, not what one that sees no key gets; where one dot is finite, its key
    takes all. Queries that see nothing keep 0 and -inf."""
    (n_q, n_k), = lens
    q, kv, kr, cu_q, cu_k = _inputs(lens, 2, BF, 83)
    q[..., 5] = 2.0 ** 70
    kv[..., 5] = -2.0 ** 70
    out, lse = _run(q, kv, kr, cu_q, cu_k, True)
    assert out.isnan().all() and lse.isnan().all()
    kv[n_k - 30, 0, 5] = 0                    # one key of the first head
    out, lse = _run(q, kv, kr, cu_q, cu_k, True)
    seen = torch.from_numpy(oracle.visible(n_q, n_k, True))
    sees = seen > n_k - 30
    assert torch.equal(out[sees][:, 0].cpu(), kv[n_k - 30, 0, 128:].expand(int(sees.sum()), 128)) and lse[sees][:, 0].isfinite().all()
    assert out[~sees][:, 0].isnan().all() and lse[~sees][:, 0].isnan().all() and out[:, 1].isnan().all()
    if n_q > 300:                             # fewer keys than queries: the first ones see none
        out, lse = _run(q, kv[:300], kr[:300], cu_q, [0, 300], True)
        none = n_q - 300
        assert (out[:none] == 0).all() and torch.isneginf(lse[:none]).all() and out[none:].isnan().all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [[(40, 700)], [(600, 700)], [(5, 6000)], [(300, 9000)]], ids=["few", "pair", "few cut", "pair cut"])
def test_prefill_of_many_small_weights(lens, dtype):
    """One key in 128 with a weight of 1 and a value of 0, the others near 2^-26 and 1024: what fp16 weights lose of them
    is 2^-32 a key at most, half a step of the subnormals at the 2^7 that they are raised by."""
    (n_q, n_k), = lens
    q, kv, kr, cu_q, cu_k = _inputs(lens, 1, dtype, 89)
    q[:], kv[:], kr[:] = 0, 0, 0
    q[..., 5] = 1.0
    small = torch.arange(n_k) % 128 != 77
    kv[small, :, 5] = -26 * 0.6931471805599453
    kv[small, :, 128:] = 1024.0
    out, lse = _run(q, kv, kr, cu_q, cu_k, False, scale=1.0)
    one = np.ones(1, dtype=np.int64) * n_k
    ro, rl, size, _ = oracle.prefill(q[:1], kv[..., :128], kr, kv[..., 128:], 1.0, one)
    weight = (4 + 6 * 27) * U                     # of itself: as in _far_check, for dots that are exact
    rel = 2 * weight + (2 * n_k + 64) * U
    bound = 1.01 * HALF[dtype] * np.abs(ro) + (HALF[dtype] + rel) * size
    if dtype == HF:
        bound = bound + 2.0 ** -32 * 1024 * int(small.sum()) / np.exp(rl)[..., None]
    assert (np.abs(oracle.to_f64(out.cpu()) - ro) <= bound).all()
    assert (np.abs(oracle.to_f64(lse.cpu()) - rl) <= weight + (n_k + 64) * U + 4 * U * np.abs(rl)).all()


@pytest.mark.parametrize("rows", [1, 513], ids=["few", "pair"])
def test_prefill_bad_offsets_behind_the_last_unit(rows):
    """Documents behind those that all units belong to, of which the search for units sees nothing: descending queries,
    keys that leave the tensor, in a group of 32 right behind the last unit's and far behind."""
    n = 32                                    # their units are as many as the grid has blocks
    lens = [(rows, rows)] * n
    q, kv, kr, cu_q, cu_k = _inputs(lens, 1, BF, 97)
    ref, ref_l = _run(q, kv, kr, cu_q, cu_k, True)
    _check(ref, ref_l, q, kv, kr, cu_q, cu_k, True, None, BF, docs=[0, 31], rows=[0, 1, 511, 512])
    dq, dkv, dkr = q.to(DEV), kv.to(DEV), kr.to(DEV)
    end = rows * n
    for more in (1, 2, 31, 33):               # documents behind
        for cq, ck in (([end] * (more - 1) + [end - 1], [end] * more), ([end] * more, [end] * (more - 1) + [end + 1]),
                       ([end] * more, [end] * (more - 1) + [-1]), ([end] * (more - 1) + [end + 1], [end] * more)):
            st = _status()
            out, lse = torch.full_like(ref, 4.0), torch.full_like(ref_l, 4.0)
            mla.mla_prefill(dq, dkv[..., :128], dkr, dkv[..., 128:], _ints([*cu_q, *cq]), _ints([*cu_k, *ck]), SCALE, out=out,
                            lse=lse, status=st)
            assert _bits(st) == 1, (more, cq[-1], ck[-1])
            if (end // (n + more) > 256) == (rows > 256):        # the same kernel, so the same bits
                assert torch.equal(out, ref) and torch.equal(lse, ref_l), (more, cq[-1], ck[-1])
            else:
                _check(out, lse, q, kv, kr, cu_q, cu_k, True, None, BF, docs=[0, 31], rows=[0, 1, 511, 512])


def test_prefill_bad_offsets_of_a_large_batch():
    """One document with a query, thousands without, the last of them bad; and none bad."""
    q, kv, kr, _, _ = _inputs([(1, 1)], 2, BF, 98)
    dkv = kv.to(DEV)
    for batch in (31, 32, 33, 5000):
        for last, bits in ((1, 0), (7, 1), (-2, 1)):
            st = _status()
            cu_k = [0] + [1] * (batch - 1) + [last]
            out, _ = mla.mla_prefill(q.to(DEV), dkv[..., :128], kr.to(DEV), dkv[..., 128:], _ints([0] + [1] * batch), _ints(cu_k), SCALE,
                                     status=st)
            assert _bits(st) == bits and torch.equal(out, dkv[..., 128:])


# ---------------------------------------------------------------------------
# a prompt in two chunks, then a decoded token
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_in_chunks_and_decode(fmt):
    """Two requests' prompts arrive in two chunks: normalised and appended, the cached prefix read back, expanded by plain
    products and attended to, against the oracle over those keys and values; then one decoded token of each over the same
    cache, in the absorbed form, against the oracle over the rows that the cache holds."""
    heads, chunks, first = 16 if fmt == 0 else 128, [(150, 90), (200, 37)], [0, 0]
    g = _gen(53)
    w_uk = (0.05 * torch.randn(heads, 128, 512, generator=g)).to(BF)
    w_uv = (0.05 * torch.randn(heads, 128, 512, generator=g)).to(BF)
    gain = (1 + 0.2 * torch.randn(512, generator=g)).to(BF)
    dk, dv = w_uk.to(DEV), w_uv.to(DEV)
    cache = torch.zeros(16, PAGE, 1, 656 if fmt else 576, dtype=torch.uint8 if fmt else BF, device=DEV)
    table = torch.randperm(16, generator=g)[:12].view(2, 6).int()
    tab = _table()
    for k in range(2):
        counts = [c[k] for c in chunks]
        n, ends = sum(counts), [f + c for f, c in zip(first, counts)]
        kv = torch.randn(n, 576, generator=g).to(BF).to(DEV)
        x = torch.randn(n, heads, 192, generator=g).to(BF).to(DEV)
        pos = torch.cat([torch.arange(f, e) for f, e in zip(first, ends)])
        who = torch.repeat_interleave(torch.arange(2), torch.tensor(counts))
        slots = (table[who, pos // PAGE] * PAGE + pos % PAGE).int().to(DEV)
        pos = pos.int().to(DEV)
        mla.mla_norm_append_kv(kv[:, :512], kv[:, 512:], gain.to(DEV), cache, slots, pos, tab, kv_format=fmt)
        cu_q, cu_k = np.cumsum([0] + counts), np.cumsum([0] + ends)
        rows = mla.mla_read_kv(cache, table.to(DEV), _ints(cu_k), total=int(cu_k[-1]), kv_format=fmt)
        q = mla.mla_norm_rotate(x, pos, tab)
        k_nope = torch.einsum("tc,hdc->thd", rows[:, :512].float(), dk.float()).to(BF)
        v = torch.einsum("tc,hdc->thd", rows[:, :512].float(), dv.float()).to(BF)
        st = _status()
        out, lse = mla.mla_prefill(q, k_nope, rows[:, 512:], v, _ints(cu_q), _ints(cu_k), SCALE, status=st)
        assert _bits(st) == 0
        both = torch.cat((k_nope, v), -1).cpu()
        _check(out, lse, q.cpu(), both, rows[:, 512:].cpu(), cu_q, cu_k, True, None, BF, heads=[0, heads - 1], rows=[0, 1, 36, 89, 149, 199])
        first = ends
    # the next token of each request over the same cache, in the absorbed form
    x = torch.randn(2, heads, 192, generator=g).to(BF).to(DEV)
    pos = _ints([e - 1 for e in first])
    query = torch.empty(2, 1, heads, 576, dtype=BF, device=DEV)
    nope, _ = mla.mla_norm_rotate(x, pos, tab, rope_out=query[:, 0, :, 512:])
    mla.mla_absorb_q(nope, dk, query.view(2, heads, 576))
    lens = _ints(first)
    if heads == 16:
        meta, ns = mla.mla_get_metadata(lens, 1, heads)
    else:
        meta, ns = mla.mla_get_metadata(lens, 1, heads, is_fp8=bool(fmt))
    o, lse = mla.mla_decode_with_kvcache(query, cache, table.to(DEV), lens, 512, meta, ns, softmax_scale=SCALE, is_fp8=bool(fmt))
    held = oracle.to_f64(cache.cpu()).reshape(-1, 576) if fmt == 0 else oracle.cached_rows(cache.view(-1, 656).cpu().numpy(), 1)
    at = (table[:, :, None] * PAGE + torch.arange(PAGE)).view(2, -1).numpy()
    for b in range(2):
        keys = held[at[b, :first[b]]]
        ro, rl = oracle.attend(oracle.to_f64(query[b, 0].cpu()), keys, SCALE)[:2]
        assert_close_attn(o[b, 0], lse[b, 0], ro, rl, "decode")


# ---------------------------------------------------------------------------
# far offsets
# ---------------------------------------------------------------------------
def test_prefill_behind_4_gb():
    """Queries, keys, values and outputs whose rows lie behind 4 GB (2^31 elements and more)."""
    heads, n_q, n_k = 128, 400, 420
    far_q, far_k = 100000, 70000            # rows of 192 and of 256 values for 128 heads
    for n in (n_q, 60):                     # two CTAs a unit, one
        q, kv, kr, cu_q, cu_k = _inputs([(n, n_k)], heads, BF, 61)
        q2 = torch.zeros(far_q + n + 9, heads, 192, dtype=BF, device=DEV)
        kv2 = torch.zeros(far_k + n_k, heads, 256, dtype=BF, device=DEV)
        kr2 = torch.zeros(far_k + n_k, 64, dtype=BF, device=DEV)
        q2[far_q:far_q + n], kv2[far_k:], kr2[far_k:] = q.to(DEV), kv.to(DEV), kr.to(DEV)
        out = torch.zeros(far_q + n + 9, heads, 192, dtype=BF, device=DEV)
        st = _status()
        got, lse = mla.mla_prefill(q2, kv2[..., :128], kr2, kv2[..., 128:], _ints(cu_q + far_q), _ints(cu_k + far_k), SCALE,
                                   out=out[..., :128], status=st)
        assert _bits(st) == 0
        _check(got[far_q:], lse[far_q:], q, kv, kr, cu_q, cu_k, True, None, BF, heads=[0, 77, 127], rows=[0, 1, 59, 128, 255, 256, 399])
        assert (out[:far_q:997] == 0).all() and (out[far_q + n:] == 0).all() and (out[far_q:, :, 128:] == 0).all()


def test_rows_behind_4_gb():
    """Norms, appends and reads of rows and pages behind 4 GB."""
    tokens, heads = 90001, 128
    x = torch.zeros(tokens, heads, 192, dtype=BF, device=DEV)
    x[-3:] = torch.randn(3, heads, 192, generator=_gen(3)).to(BF).to(DEV)
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV) % 5000
    out = mla.mla_norm_rotate(x, pos, _table())
    tail = mla.mla_norm_rotate(x[-3:], pos[-3:].contiguous(), _table())
    assert torch.equal(out[-3:], tail)
    bound = oracle.norm_rotate_error(oracle.rms_norm(x[-3:]), 128, False)
    _close(tail, oracle.norm_rotate(x[-3:], None, 1e-6, TABLE[pos[-3:].cpu().numpy()], 128, False), bound, BF)
    del x, out
    pages = 60000                                            # 4.4 GB of 16-bit rows
    cache = torch.zeros(pages, PAGE, 1, 576, dtype=BF, device=DEV)
    kv = torch.randn(40, 576, generator=_gen(4)).to(BF).to(DEV)
    slots = torch.arange(40, dtype=torch.int32, device=DEV) + (pages * PAGE - 50)
    rows = torch.empty(40, 576, dtype=BF, device=DEV)
    mla.mla_norm_append_kv(kv[:, :512], kv[:, 512:], None, cache, slots, pos[:40].contiguous(), _table(), rows=rows)
    wide = torch.zeros(2200000, 1024, dtype=BF, device=DEV)  # 4.5 GB
    table = _ints([[pages - 1]])
    n = 2200000
    mla.mla_read_kv(cache, table.expand(2, 1).contiguous(), _ints([0, n - 30, n]), starts=_ints([0, 20]), out=wide[:, :576],
                    status=_status())
    assert torch.equal(wide[-30:, :576], rows[6:36]) and (wide[-30:, 576:] == 0).all()
