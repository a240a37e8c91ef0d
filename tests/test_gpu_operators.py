"""The operators between a model's parameters and the join's points, through
the public entry points, against plain float64 implementations: embedding
lookup and its gradient, layer norm and its gradient, clipping by the global
gradient norm.

Tolerances are worst-case bounds of float32 arithmetic (u = 2^-24 per
operation, (k - 1) u times the sum of magnitudes for a sum of k terms in
any order), plus one rounding to the stored type."""
import math
import zlib

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
XY = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]
# half an ulp relative to the value, and half the smallest subnormal
ROUND = {F32: (U, 2.0 ** -150), F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -134)}


@pytest.fixture(scope="module")
def edd():
    import __graft_entry__
    __graft_entry__.build()
    import exact_dimensional_distance_gb300 as m
    return m


@pytest.fixture(scope="module")
def lib(edd):
    j = edd.Join()
    yield j
    j.close()


def _gen(*seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(seed).encode()))
    return g


def _normal(shape, dtype, gen, scale=1.0, shift=0.0):
    return (shift + scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def _laid(t, pad, off):
    """t with pad extra elements per row and its base off elements into a
    buffer whose other elements are NaN."""
    n, d = t.shape
    buf = torch.full((n * (d + pad) + off + 8,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off:off + n * (d + pad)].view(n, d + pad)[:, :d]
    v.copy_(t)
    return v


def _close(got, want, err, what=""):
    """|got - want| <= err + the rounding of want to got's type."""
    rel, sub = ROUND[got.dtype]
    tol = err * (1 + 2 * rel) + rel * want.abs() + sub
    bad = ~((got.double() - want).abs() <= tol)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError("%s: %d of %d outside; first at %d: %r, expected %r +- %.3g" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]),
            float((tol + 0 * want).flatten()[i])))


def _tokens(n, vocab, gen, kind, bits=64, pad=None):
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if kind == "zipf":
        t = torch.exp(u * math.log(vocab + 1)).floor().long() - 1
    elif kind == "same":
        t = torch.full((n,), vocab - 1, device="cuda")
    elif kind == "ordered":
        t = torch.arange(n, device="cuda") * vocab // max(n, 1)
    else:
        t = (u * vocab).floor().long()
    t = t.clamp(0, vocab - 1)
    if pad is not None:
        t = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.3, torch.full_like(t, pad), t)
    return t.to(torch.int64 if bits == 64 else torch.int32)


# ---- embedding lookup ------------------------------------------------------------

def _embed_ref(tokens, table, scale, pad):
    t = tokens.long().flatten()
    ok = (t >= 0) & (t < table.shape[0])
    if pad is not None:
        ok &= t != pad
    rows = table.double()[t.clamp(0, table.shape[0] - 1)] * float(np.float32(scale))
    return (rows * ok[:, None]).view(*tokens.shape, table.shape[1])


@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 16, 31, 32, 33, 96, 128, 257, 1000, 1024, 4099])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16), (BF16, BF16), (F32, BF16), (F32, F16), (BF16, F32),
                                   (F16, BF16)])
def test_embed(lib, width, types):
    for n, vocab, pad, bits, extra, off in [(1, 1, None, 64, 0, 0), (5, 7, 3, 32, 0, 0), (333, 101, -1, 64, 3, 1),
                                            (1024, 50, None, 32, 8, 0), (77, 4000, 0, 64, 16, 8)]:
        g = _gen(width, n, str(types))
        table = _laid(_normal((vocab, width), types[0], g), extra, off)
        t = _tokens(n, vocab, g, "zipf", bits, pad)
        out = _laid(torch.zeros((n, width), dtype=types[1], device="cuda"), extra, off)
        got = lib.embed(t, table, scale=1.7, pad=pad, out=out)
        assert got is out
        want = _embed_ref(t, table, 1.7, pad)
        _close(out, want, U * want.abs(), "n=%d" % n)
        if extra:  # nothing outside the rows is touched
            assert bool(torch.isnan(out.as_strided((n, extra), (width + extra, 1), out.storage_offset() + width)[:-1])
                        .all())
        assert torch.equal(lib.embed(t, table.contiguous(), scale=1.7, pad=pad, dtype=types[1]), out.contiguous())
    lib.finish()


def test_embed_shapes_and_empty(lib):
    g = _gen(1)
    table = _normal((30, 24), F32, g)
    t = torch.arange(24, device="cuda").view(2, 3, 4)
    assert torch.equal(lib.embed(t, table), table[t])
    e = lib.embed(t[:0], table)
    assert e.shape == (0, 3, 4, 24)
    assert torch.equal(lib.embed(t.permute(2, 0, 1), table), table[t.permute(2, 0, 1)])
    # infinities and NaN are copied, a row of zeros for padding whatever the row holds
    table[3] = float("inf")
    table[4] = float("nan")
    out = lib.embed(torch.tensor([3, 4, 5], device="cuda"), table, pad=4)
    assert torch.isinf(out[0]).all() and bool((out[1] == 0).all()) and torch.equal(out[2], table[5])
    # a broadcast table (row stride 0)
    one = _normal((1, 24), F32, g).expand(9, 24)
    assert torch.equal(lib.embed(torch.tensor([8, 0], device="cuda"), one), one[:2])
    lib.finish()


def test_out_of_range_tokens_are_reported(edd, lib):
    lib.finish()
    table = torch.ones((10, 16), device="cuda")
    dy = torch.ones((5, 16), device="cuda")
    for bad in (10, -1, -(1 << 62), 1 << 40):
        t = torch.tensor([1, bad, 9, 0, 1], device="cuda")
        out = lib.embed(t, table)
        with pytest.raises(edd.HissError) as e:
            lib.finish()
        assert e.value.status == edd.HISS_E_ARG
        lib.finish()  # reported once; the context goes on
        assert out.sum(1).tolist() == [16, 0, 16, 16, 16]
        grad = lib.embed_grad(t, dy, 10)
        with pytest.raises(edd.HissError):
            lib.finish()
        assert grad[:, 0].tolist() == [1, 2, 0, 0, 0, 0, 0, 0, 0, 1]
        lib.embed(t, table, pad=bad)  # as padding it is in order
        lib.finish()


# ---- gradient of the lookup --------------------------------------------------------

def _embed_grad_ref(tokens, dy, vocab, scale, pad):
    """Sum and sum of magnitudes per row, and the number of positions."""
    t = tokens.long().flatten()
    keep = torch.nonzero((t >= 0) & (t < vocab) & (t != pad if pad is not None else t == t)).flatten()
    d = dy.double().reshape(-1, dy.shape[-1])[keep] * float(np.float32(scale))
    z = torch.zeros((vocab, dy.shape[-1]), dtype=torch.float64, device="cuda")
    count = torch.zeros(vocab, dtype=torch.float64, device="cuda")
    count.index_put_((t[keep],), torch.ones_like(d[:, 0]), accumulate=True)
    return z.index_put((t[keep],), d, accumulate=True), z.index_put((t[keep],), d.abs(), accumulate=True), count


GRAD_SIZES = [  # n, vocab, kind, pad, bits
    (0, 5, "zipf", None, 64), (1, 1, "zipf", None, 32), (1, 1000, "zipf", None, 64), (2, 3, "same", None, 64),
    (37, 11, "zipf", 0, 32), (300, 70000, "uniform", None, 64), (1000, 300, "zipf", -1, 32), (2048, 64, "uniform", None, 64),
    (2049, 2, "uniform", None, 32), (4097, 513, "zipf", -100, 64), (5000, 9, "same", None, 64), (12345, 70001, "zipf", 1, 32),
    (20000, 1 << 17, "ordered", None, 64), (33333, 257, "uniform", 7, 32), (70000, 1025, "zipf", None, 64)]


@pytest.mark.parametrize("size", GRAD_SIZES)
@pytest.mark.parametrize("width,types", [(1, (F32, F32)), (5, (BF16, BF16)), (16, (F16, F32)), (64, (F32, F32)),
                                         (100, (F32, BF16)), (128, (BF16, F32)), (322, (F16, F16)), (1032, (BF16, F32))])
def test_embed_grad(lib, size, width, types):
    n, vocab, kind, pad, bits = size
    if vocab * width > 1 << 25:
        width = (1 << 25) // vocab
    g = _gen(n, vocab, width)
    t = _tokens(n, vocab, g, kind, bits, pad)
    dy = _normal((n, width), types[0], g, 1.0, 0.1)
    got = lib.embed_grad(t, dy, vocab, scale=0.75, pad=pad, dtype=types[1])
    want, mag, count = _embed_grad_ref(t, dy, vocab, 0.75, pad)
    _close(got, want, (count[:, None] + 1) * U * mag, "sum")
    assert torch.equal(got, lib.embed_grad(t, dy, vocab, scale=0.75, pad=pad, dtype=types[1])), "not repeatable"
    # added to what is there; rows without a position keep their bits; strides and offsets
    old = _normal((vocab, width), types[1], g)
    out = _laid(old, 3, 1)
    lib.embed_grad(t, _laid(dy, 1, 3), vocab, scale=0.75, pad=pad, out=out, accumulate=True)
    _close(out, want + old.double(), (count[:, None] + 1) * U * mag + U * (want + old.double()).abs(), "accumulated")
    none = count == 0
    assert torch.equal(out[none], old[none])
    lib.finish()


def test_embed_grad_broadcast_and_order(lib):
    # a broadcast gradient (row stride 0) counts the tokens; integers are exact
    g = _gen(5)
    t = _tokens(30000, 100, g, "zipf")
    dy = torch.ones((1, 32), device="cuda").expand(30000, 32)
    got = lib.embed_grad(t, dy, 100)
    assert torch.equal(got, torch.bincount(t, minlength=100).float()[:, None].expand(100, 32))
    # a full last page of positions, and everything on one token: exact integers again
    for n in (4096, 8192, 65536, 65537):
        t = torch.zeros(n, dtype=torch.int32, device="cuda")
        got = lib.embed_grad(t, torch.ones((n, 8), device="cuda", dtype=BF16), 3, dtype=F32)
        assert got[0].tolist() == [float(n)] * 8 and bool((got[1:] == 0).all())
    # an infinite or NaN gradient stays in its own row
    dy = torch.ones((5000, 8), device="cuda")
    t = torch.arange(5000, device="cuda") % 50
    dy[13] = float("inf")
    dy[14] = float("nan")
    got = lib.embed_grad(t, dy, 60)
    assert torch.isinf(got[13]).all() and torch.isnan(got[14]).all()
    rest = [v for v in range(60) if v not in (13, 14)]
    assert torch.equal(got[rest], torch.tensor([100.0 if v < 50 else 0.0 for v in rest], device="cuda")[:, None].expand(58, 8))
    lib.finish()


@pytest.mark.parametrize("n", [1, 700, 2048, 2049, 40000])
def test_embed_grad_all_padding(lib, n):
    t = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    dy = torch.full((n, 40), float("nan"), device="cuda")  # what is masked is not read
    got = lib.embed_grad(t, dy, 333, pad=-7, out=torch.full((333, 40), 9.0, device="cuda"))
    assert not got.any()
    kept = torch.full((333, 40), 9.0, device="cuda")
    lib.embed_grad(t, dy, 333, pad=-7, out=kept, accumulate=True)
    assert bool((kept == 9.0).all())
    # one position left: its row alone, whatever the padding holds
    t[n // 2] = 5
    dy[n // 2] = 1.5
    got = lib.embed_grad(t, dy, 333, pad=-7)
    assert bool((got[5] == 1.5).all()) and int((got != 0).any(1).sum()) == 1
    lib.finish()


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 32, 33])
@pytest.mark.parametrize("n", [2048, 2049, 40000])
def test_embed_grad_small_vocabularies_without_positions(edd, lib, vocab, n):
    # every row is written, whichever share of the zeros it falls into
    dy = torch.full((n, 24), float("nan"), device="cuda")
    for token, pad in ((-7, -7), (vocab, None)):  # all padding; all out of range
        t = torch.full((n,), token, dtype=torch.int32, device="cuda")
        for dtype in (F32, BF16):
            got = lib.embed_grad(t, dy, vocab, pad=pad, out=torch.full((vocab, 24), 9.0, dtype=dtype, device="cuda"))
            assert not got.any()
        if pad is None:
            with pytest.raises(edd.HissError):
                lib.finish()
    lib.finish()


@pytest.mark.parametrize("vocab", [511, 512, (1 << 18) - 1, 1 << 18, 300007, (1 << 20) + 3])
def test_embed_grad_large_vocabularies(lib, vocab):
    # one, two and three sort passes; more tokens than a tile's bitmap holds
    g = _gen(vocab)
    n = 30000
    t = _tokens(n, vocab, g, "zipf", 64, -1)
    dy = torch.randint(-8, 9, (n, 6), generator=g, device="cuda").float()  # integers: exact in any order
    want = torch.zeros((vocab, 6), dtype=torch.float64, device="cuda")
    keep = t >= 0
    want.index_put_((t[keep],), dy[keep].double(), accumulate=True)
    for _ in range(2):  # the second call finds what the first left in the workspace
        assert torch.equal(lib.embed_grad(t, dy, vocab, pad=-1).double(), want)
    lib.finish()


def test_embed_grad_many_positions(lib):
    # more than 128 tiles of the largest size
    g = _gen(99)
    n, vocab = 700_001, 1000
    t = _tokens(n, vocab, g, "zipf", 32, 3)
    dy = torch.randint(-2, 3, (n, 3), generator=g, device="cuda").to(BF16)
    want = torch.zeros((vocab, 3), dtype=torch.float64, device="cuda")
    keep = t != 3
    want.index_put_((t[keep].long(),), dy[keep].double(), accumulate=True)
    assert torch.equal(lib.embed_grad(t, dy, vocab, pad=3, dtype=F32).double(), want)
    lib.finish()


def test_offsets_beyond_32_bits(edd, lib):
    """Matrices and tensors of more than 2^31 elements."""
    rows, width = (1 << 21) + 5, 1040
    assert rows * width > 1 << 31
    x = torch.empty((rows, width), dtype=BF16, device="cuda")
    step = 1 << 18
    for i in range(0, rows, step):
        x[i:i + step] = (torch.arange(i, min(i + step, rows), device="cuda") % 251).to(BF16)[:, None]
    x += (torch.arange(width, device="cuda") % 2).to(BF16)
    last = torch.tensor([0, 1, rows - 1, rows - 2, (1 << 31) // width + 1], device="cuda")
    assert torch.equal(lib.embed(last, x), x[last])
    odd = lib.embed(torch.arange(rows, device="cuda"), x[:, 1:1036])  # unaligned rows in and out
    assert odd.numel() > 1 << 31
    assert all(torch.equal(odd[i:i + step], x[i:i + step, 1:1036]) for i in range(0, rows, step))
    del odd
    y, mean, rstd = lib.layer_norm(x)
    want = lib.layer_norm(x[last].contiguous())
    assert torch.equal(y[last], want[0]) and torch.equal(mean[last], want[1]) and torch.equal(rstd[last], want[2])
    dx, _, _ = lib.layer_norm_grad(x, y, mean, rstd)
    assert torch.equal(dx[last], lib.layer_norm_grad(x[last].contiguous(), y[last].contiguous(), mean[last], rstd[last])[0])
    del y, dx
    # the gradient of a table of as many elements, and as many elements of dy
    dy = torch.ones((5, width), dtype=BF16, device="cuda")
    grad = lib.embed_grad(last, dy, rows)
    assert torch.equal(grad.sum(1, dtype=torch.float32).nonzero().flatten(), last.sort().values)
    assert bool((grad[last] == 1).all())
    del grad
    t = torch.full((rows,), -1, device="cuda")
    t[last] = torch.arange(5, device="cuda")
    assert torch.equal(lib.embed_grad(t, x, 7, pad=-1)[:5], x[last])
    norm = lib.clip_grads(edd.Gradients([x.view(-1)]), float("inf"))
    assert abs(float(norm) - math.sqrt(sum(float((x[i:i + step].double() ** 2).sum()) for i in range(0, rows, step)))) <= \
        1e-5 * float(norm)
    lib.clip_grads([x], float(norm) / 2)
    assert torch.equal(x[-1, :2], torch.tensor([(rows - 1) % 251 / 2, ((rows - 1) % 251 + 1) / 2], device="cuda").to(BF16))
    lib.finish()


def test_embed_grad_against_differences(lib):
    # L = sum(dy * embed(E)) is linear in E: the difference along V is <grad, V>
    g = _gen(9)
    t = _tokens(500, 40, g, "zipf", 64, 2)
    table, v = torch.randint(-8, 9, (2, 40, 24), generator=g, device="cuda").float()
    dy = torch.randint(-8, 9, (500, 24), generator=g, device="cuda").float()
    diff = ((lib.embed(t, table + v, scale=2.0, pad=2) - lib.embed(t, table, scale=2.0, pad=2)) * dy).sum()
    grad = lib.embed_grad(t, dy, 40, scale=2.0, pad=2)
    assert float(diff) == float((grad * v).sum())  # small integers: exact on both sides


# ---- layer norm ----------------------------------------------------------------------

def _norm_ref(x, w, b, eps):
    x = x.double()
    d = x.shape[-1]
    mean = x.sum(-1) / d
    e = x - mean[..., None]
    var = (e * e).sum(-1) / d
    rstd = 1 / torch.sqrt(var + float(np.float32(eps)))
    h = e * rstd[..., None]
    wd = w.double() if w is not None else torch.ones(d, dtype=torch.float64, device="cuda")
    y = h * wd + (b.double() if b is not None else 0)
    # mean: d terms and a division; variance: its own d-term sum of squares of
    # differences rounded once, and the square of the mean's error
    em = (d + 1) * U * x.abs().sum(-1) / d
    ev = (d + 6) * U * var + em * em + 2 * em * 4 * U * e.abs().sum(-1) / d
    rel = 0.5 * ev / (var + eps) * (1 + 2 * ev / (var + eps)) + 4 * U
    er = rel * rstd
    ey = wd.abs() * (h.abs() * (rel + 3 * U)[..., None] + (em * rstd)[..., None] * (1 + 2 * rel)[..., None]) + \
        2 * U * ((h * wd).abs() + y.abs())
    return (y, ey), (mean, em), (rstd, er)


NORM_SHAPES = [(1, 1), (3, 2), (7, 3), (65, 7), (33, 8), (100, 16), (1000, 31), (129, 32), (64, 33), (300, 64),
               (50, 100), (77, 127), (1025, 128), (40, 255), (41, 256), (42, 257), (9, 500), (11, 1000), (153, 1021),
               (305, 1024), (13, 1025), (6, 2040), (21, 2048), (5, 4095), (160, 4096), (7, 5000), (3, 8192),
               (4, 8200), (2, 12289), (2, 16384), (2, 16392), (1, 20001), (3, 32768), (1, 40000), (1, 65535), (2, 65536)]


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("types", XY)
def test_layer_norm(lib, shape, types):
    n, d = shape
    g = _gen(n, d, str(types))
    x = _normal((n, d), types[0], g, 1.5, 0.7)
    for pt, with_w, with_b, extra, off in [(F32, True, True, 0, 0), (types[0], True, False, 3, 1),
                                           (BF16, False, True, 8, 8), (F32, False, False, 0, 0)]:
        w = _normal((d,), pt, g, 0.3, 1.0) if with_w else None
        b = _normal((d,), pt, g) if with_b else None
        xs = _laid(x, extra, off)
        out = _laid(torch.zeros((n, d), dtype=types[1], device="cuda"), extra, off)
        y, mean, rstd = lib.layer_norm(xs, w, b, eps=1e-5, out=out)
        (wy, ey), (wm, em), (wr, er) = _norm_ref(x, w, b, 1e-5)
        _close(mean, wm, em, "mean")
        _close(rstd, wr, er, "rstd")
        _close(y, wy, ey, "y")
        if extra:
            assert bool(torch.isnan(out.as_strided((n, extra), (d + extra, 1), out.storage_offset() + d)[:-1]).all())
        y2, mean2, rstd2 = lib.layer_norm(x, w, b, eps=1e-5, dtype=types[1])
        assert torch.equal(mean2, lib.layer_norm(x, w, b, eps=1e-5, dtype=types[1])[1])
        _close(y2, wy, ey, "y, contiguous")


def test_layer_norm_difficult_rows(lib):
    d = 512
    x = torch.zeros((6, d), device="cuda")
    x[0] = 3.25                                    # constant: variance 0
    x[1] = 4096 + (torch.arange(d, device="cuda") % 2) * 2.0 ** -3   # a large mean, a small spread: exact in float32
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    x[4] = torch.arange(d, device="cuda") * 1e15   # the variance is large but representable
    x[5] = (torch.arange(d, device="cuda") % 2) * 2e-18  # squares are subnormal
    y, mean, rstd = lib.layer_norm(x, eps=1e-5)
    assert float(mean[0]) == 3.25 and bool((y[0] == 0).all())
    _close(rstd[:2], torch.tensor([1 / math.sqrt(float(np.float32(1e-5))),
                                   1 / math.sqrt(2.0 ** -8 + float(np.float32(1e-5)))], dtype=torch.float64,
                                  device="cuda"), torch.full((2,), 400 * (d + 10) * U, device="cuda", dtype=torch.float64))
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    (wy, ey), _, _ = _norm_ref(x[4:], None, None, 1e-5)
    _close(y[4:], wy, ey)
    # eps = 0: a constant row is NaN by the formula, the others are not touched by it
    y, mean, rstd = lib.layer_norm(x[:2], eps=0.0)
    assert bool(torch.isnan(y[0]).all()) and math.isinf(float(rstd[0])) and bool(torch.isfinite(y[1]).all())
    # width 1: the value is its own mean
    y, mean, rstd = lib.layer_norm(torch.tensor([[2.0], [-3.0]], device="cuda"), bias=torch.tensor([0.5], device="cuda"))
    assert y.tolist() == [[0.5], [0.5]] and mean.tolist() == [2.0, -3.0]
    # no rows; leading dimensions
    assert lib.layer_norm(x[:0])[0].shape == (0, d)
    z = torch.randn((2, 3, 4, d), device="cuda")
    assert torch.equal(lib.layer_norm(z)[0].view(-1, d), lib.layer_norm(z.view(-1, d))[0])
    # a broadcast input
    r = torch.randn((1, d), device="cuda")
    assert torch.equal(lib.layer_norm(r.expand(5, d))[0], lib.layer_norm(r)[0].expand(5, d))


@pytest.mark.parametrize("types", XY)
@pytest.mark.parametrize("d", [1, 3, 41, 47, 96, 100, 328, 512, 656, 1000, 1021, 1302, 2569, 4099, 5000, 8200, 9001, 12000, 16384,
                               20001, 65535])
def test_layer_norm_constant_rows(lib, d, types):
    # a constant row's mean is its value and its differences are zero, whatever the
    # width and however the row is laid out over lanes, warps and blocks
    value = torch.tensor([1.0, 0.1, -3000.0, 1e-3, 6.1e4, 1e-30, 0.0], device="cuda").to(types[0])
    other = _normal((d,), types[0], _gen(d, str(types)), 1.5, 0.7)
    bias = _normal((d,), types[1], _gen(d, 1))
    for extra, off in ((0, 0), (3, 1)):
        x = torch.cat([value[:, None].expand(-1, d), other[None], value[:, None].expand(-1, d)])
        x = _laid(x, extra, off)
        row = lib.layer_norm(_laid(other[None], extra, off), bias=bias, dtype=types[1])
        y, mean, rstd = lib.layer_norm(x, bias=bias, dtype=types[1])
        # a row between them is not changed by its neighbours
        assert torch.equal(y[7], row[0][0]) and torch.equal(mean[7], row[1][0]) and torch.equal(rstd[7], row[2][0])
        y0, mean0, rstd0 = lib.layer_norm(x, bias=bias, eps=0.0, dtype=types[1])
        for k in list(range(7)) + list(range(8, 15)):
            v = value[k % 8]
            assert float(mean[k]) == float(v) and float(mean0[k]) == float(v)
            assert torch.equal(y[k], bias)
            assert abs(float(rstd[k]) / float(np.float32(1e-5)) ** -0.5 - 1) <= 4 * U
            assert math.isinf(float(rstd0[k])) and bool(torch.isnan(y0[k]).all())


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("n,d", [(30011, 40), (9000, 300), (5001, 700), (4003, 1021), (3001, 3000), (2000, 5000), (1001, 8200),
                                 (700, 9001), (601, 12000), (500, 16384), (201, 20001)])
def test_layer_norm_constant_rows_among_others(lib, n, d, types):
    # blocks that take rows of both kinds one after the other: each row is what it is alone
    g = _gen(n, d, str(types), 3)
    x = _normal((n, d), types[0], g, 1.5, 0.7)
    flat = torch.rand(n, generator=g, device="cuda") < 0.4
    x[flat] = torch.randint(1, 99, (int(flat.sum()), 1), generator=g, device="cuda").to(types[0])
    for extra, off in ((0, 0), (3, 1)):
        got = lib.layer_norm(_laid(x, extra, off), dtype=types[1])
        for rows in (flat, ~flat):
            want = lib.layer_norm(_laid(x[rows], extra, off), dtype=types[1])
            assert all(torch.equal(a[rows], b) for a, b in zip(got, want))
        assert not got[0][flat].any() and torch.equal(got[1][flat], x[flat, 0].float())


@pytest.mark.parametrize("d", [7, 41, 100, 300, 1000, 1021, 4099])
def test_layer_norm_small_spread(lib, d):
    # a spread far below the mean: the mean is the exact one rounded (U of it), up to the
    # error of a mean of differences from a first mean that is (d + 1) U off at most
    n = 37
    x = 1000 + torch.randint(-8, 9, (n, d), generator=_gen(d, 5), device="cuda") * 2.0 ** -12
    x = x.float()  # exact: multiples of 2^-14 below 1024
    w = _normal((d,), F32, _gen(d, 6))
    for extra, off in ((0, 0), (3, 1)):
        y, mean, rstd = lib.layer_norm(_laid(x, extra, off), w, eps=1e-12)
        (wy, _), (wm, _), (wr, _) = _norm_ref(x, w, None, 1e-12)
        e = x.double() - wm[:, None]
        var = (e * e).mean(1)
        em = U * wm.abs() + (d + 2) * U * (e.abs().mean(1) + (d + 1) * U * wm.abs())
        # the squares are taken about a mean that is em off, the rest as in _norm_ref
        rel = 0.5 * ((d + 6) * U + em * em / var) + 4 * U
        rel = rel * (1 + 2 * rel)
        _close(mean, wm, em, "mean")
        _close(rstd, wr, rel * wr, "rstd")
        h = (e * wr[:, None]).abs()
        ey = w.double().abs() * (h * (rel + 3 * U)[:, None] + (em * wr * (1 + 2 * rel))[:, None]) + 4 * U * wy.abs()
        _close(y, wy, ey, "y")


def _norm_grad_ref(dy, x, mean, rstd, w):
    dy, x, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    n, d = x.shape
    wd = w.double() if w is not None else torch.ones(d, dtype=torch.float64, device="cuda")
    h = (x - m) * r
    g = dy * wd
    mg, mgh = g.sum(1, keepdim=True) / d, (g * h).sum(1, keepdim=True) / d
    dx = r * (g - mg - h * mgh)
    emg = (d + 3) * U * g.abs().sum(1, keepdim=True) / d
    emgh = (d + 7) * U * (g * h).abs().sum(1, keepdim=True) / d
    edx = r * (8 * U * (g.abs() + mg.abs() + (h * mgh).abs()) + emg + h.abs() * emgh)
    return (dx, edx), ((dy * h).sum(0), (n + 6) * U * (dy * h).abs().sum(0)), (dy.sum(0), (n + 2) * U * dy.abs().sum(0))


@pytest.mark.parametrize("shape", NORM_SHAPES + [(5000, 16), (3001, 65), (2000, 322), (1217, 768)])
@pytest.mark.parametrize("types", XY)
def test_layer_norm_grad(lib, shape, types):
    n, d = shape
    g = _gen(n, d, str(types), 1)
    x = _normal((n, d), types[0], g, 1.5, 0.7)
    dy = _normal((n, d), types[1], g, 1.0, 0.2)
    _, mean, rstd = lib.layer_norm(x)
    for pt, with_w, extra, off in [(F32, True, 0, 0), (types[0], True, 3, 1), (BF16, False, 8, 8)]:
        w = _normal((d,), pt, g, 0.3, 1.0) if with_w else None
        dx, dw, db = lib.layer_norm_grad(_laid(dy, extra, off), _laid(x, extra, off), mean, rstd, w, param_dtype=pt)
        assert dx.dtype == types[0] and dw.dtype == pt and db.dtype == pt
        want = _norm_grad_ref(dy, x, mean, rstd, w)
        for got, (wv, ev), what in zip((dx, dw, db), want, ("dx", "dw", "db")):
            _close(got, wv, ev, what)
        again = lib.layer_norm_grad(dy, x, mean, rstd, w, param_dtype=pt)
        once = lib.layer_norm_grad(dy, x, mean, rstd, w, param_dtype=pt)
        assert all(torch.equal(a, b) for a, b in zip(again, once)), "not repeatable"


# rows cut in two, up to the widest and beyond; one, two, three, some and many rows; a
# half that ends inside a pack, a warp or a group
WIDE_SHAPES = [(1, 8193), (2, 8200), (3, 8704), (77, 9000), (200, 12345), (301, 8208), (153, 16384), (160, 16382),
               (9, 16368), (5, 16385), (3, 16400)]


@pytest.mark.parametrize("shape", WIDE_SHAPES)
@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (F16, F32), (BF16, BF16)])
def test_layer_norm_wide_rows(lib, shape, types):
    n, d = shape
    g = _gen(n, d, str(types), 2)
    x = _normal((n, d), types[0], g, 1.5, 0.7)
    dy = _normal((n, d), types[1], g, 1.0, 0.2)
    w, b = _normal((d,), F32, g, 0.3, 1.0), _normal((d,), F32, g)
    for extra, off in [(0, 0), (3, 1), (16, 16)]:
        xs, dys = _laid(x, extra, off), _laid(dy, extra, off)
        y, mean, rstd = lib.layer_norm(xs, w, b, dtype=types[1])
        for got, (wv, ev), what in zip((y, mean, rstd), _norm_ref(x, w, b, 1e-5), ("y", "mean", "rstd")):
            _close(got, wv, ev, what)
        got = lib.layer_norm_grad(dys, xs, mean, rstd, w)
        for got1, (wv, ev), what in zip(got, _norm_grad_ref(dy, x, mean, rstd, w), ("dx", "dw", "db")):
            _close(got1, wv, ev, what)
        again = lib.layer_norm_grad(dys, xs, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(got, again)), "not repeatable"


def test_layer_norm_grad_edges(edd, lib):
    g = _gen(4)
    d = 96
    x = _normal((50, d), F32, g)
    w = _normal((d,), F32, g)
    _, mean, rstd = lib.layer_norm(x, w)
    # a broadcast dy (of a sum): row stride 0, and a scalar expanded over both
    row = _normal((1, d), F32, g)
    for dy in (row.expand(50, d), torch.ones((), device="cuda").expand(50, d)):
        got = lib.layer_norm_grad(dy, x, mean, rstd, w)
        want = lib.layer_norm_grad(dy.contiguous(), x, mean, rstd, w)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # no rows
    dx, dw, db = lib.layer_norm_grad(x[:0], x[:0], mean[:0], rstd[:0], w)
    assert dx.shape == (0, d) and bool((dw == 0).all()) and bool((db == 0).all())
    # each output alone, through the C ABI
    full = lib.layer_norm_grad(row.expand(50, d), x, mean, rstd, w)
    dyc = row.expand(50, d).contiguous()
    for want in range(3):
        outs = [torch.full_like(o, 7.0) for o in full]
        ptrs = [o.data_ptr() if i == want else None for i, o in enumerate(outs)]
        assert edd.hiss_layer_norm_grad(lib.handle, dyc.data_ptr(), edd.HISS_F32, d, x.data_ptr(), edd.HISS_F32, d,
                                        mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), edd.HISS_F32, 50, d, ptrs[0], d,
                                        ptrs[1], ptrs[2]) == 0
        for i in range(3):
            assert torch.equal(outs[i], full[i] if i == want else torch.full_like(full[i], 7.0))
    # a NaN row reaches the sums, not the other rows' dx
    dy = _normal((50, d), F32, g)
    clean = lib.layer_norm_grad(dy, x, mean, rstd, w)[0]
    dy[20, 5] = float("nan")
    dx, dw, db = lib.layer_norm_grad(dy, x, mean, rstd, w)
    assert bool(torch.isnan(dx[20]).all()) and math.isnan(float(db[5])) and int(torch.isnan(db).sum()) == 1
    assert torch.equal(dx[:20], clean[:20]) and torch.equal(dx[21:], clean[21:])


@pytest.mark.parametrize("d", [5, 24, 130])
def test_layer_norm_grad_against_differences(lib, d):
    # central differences of L = sum(dy * y) at steps h and h / 2 along a
    # random direction; their difference is 3 times the error of the second,
    # and each value of L carries the float32 errors of its y
    g = _gen(d, 77)
    x, dy, v = (_normal((6, d), F32, g) for _ in range(3))
    w, b, vw, vb = (_normal((d,), F32, g) for _ in range(4))
    _, mean, rstd = lib.layer_norm(x, w, b)
    dx, dw, db = lib.layer_norm_grad(dy, x, mean, rstd, w)
    slope = float((dx.double() * v.double()).sum() + (dw.double() * vw.double()).sum() + (db.double() * vb.double()).sum())

    def loss(s):
        y = lib.layer_norm(x + s * v, w + s * vw, b + s * vb)[0]
        (_, ey), _, _ = _norm_ref(x + s * v, w + s * vw, b + s * vb, 1e-5)
        # x + s v is itself rounded: u |x + s v| per entry, passed on with a slope of at most |w| rstd (1 + h^2 / d + ...)
        return float((dy.double() * y.double()).sum()), float((dy.double().abs() * (ey + 16 * U)).sum())

    def diff(h):
        (p, ep), (m, em) = loss(h), loss(-h)
        return (p - m) / (2 * h), (ep + em) / (2 * h)

    (d1, e1), (d2, e2) = diff(2.0 ** -5), diff(2.0 ** -6)
    assert abs(d2 - slope) <= abs(d1 - d2) + e1 + e2, (slope, d1, d2, e1, e2)


# ---- clipping by the global norm -----------------------------------------------------------

def _clip_ref(ts, max_norm):
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))
    c = max_norm / norm if math.isfinite(norm) and norm > max_norm else 1.0
    return norm, c


# sums of squares are kept in float32 over at most 512 terms and in float64 above
NORM_REL = 512 * U / 2 + 2 * U


def _check_clip(lib, edd, ts, max_norm, in_place):
    src = [t.clone() for t in ts]
    out = ts if in_place else [torch.empty_like(t) for t in ts]
    got = lib.clip_grads(ts if in_place else edd.Gradients(ts, out), max_norm)
    norm, c = _clip_ref(src, float(np.float32(max_norm)))
    assert abs(float(got) - norm) <= NORM_REL * norm
    for s, o in zip(src, out):
        if c == 1.0:
            assert torch.equal(o, s)
        else:
            _close(o, s.double() * c, (NORM_REL + 3 * U) * (s.double() * c).abs())
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(ts, src))


CLIP_SIZES = [[1], [0, 3, 0], [7, 8, 9], [255, 256, 257, 1023, 1025], [100000], [65536, 1, 65535, 65537, 3],
              [5000 + 37 * i for i in range(40)], [1 + i % 3 for i in range(700)], [1 << 20, 333, (1 << 20) + 1],
              [17] * 2500]


@pytest.mark.parametrize("sizes", CLIP_SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F16,), (F32, BF16, F16)])
def test_clip(edd, lib, sizes, types):
    g = _gen(len(sizes), sum(sizes), str(types))
    ts = [_normal((n,), types[i % len(types)], g, 0.5) for i, n in enumerate(sizes)]
    norm = _clip_ref(ts, 1.0)[0]
    for factor in (0.25, 3.0):
        for in_place in (False, True):
            _check_clip(lib, edd, [t.clone() for t in ts], norm * factor, in_place)


def test_clip_layouts(edd, lib):
    g = _gen(8)
    # bases off 16 bytes, in and out differently
    buf = _normal((40000,), BF16, g)
    dst = torch.zeros(40000, dtype=BF16, device="cuda")
    for a, b, n in [(1, 0, 999), (0, 1, 1000), (3, 5, 20001), (2, 2, 8), (7, 7, 1), (1, 9, 17)]:
        ts, out = [buf[a:a + n]], [dst[b:b + n]]
        dst.zero_()
        norm, c = _clip_ref(ts, 0.5)
        got = lib.clip_grads(edd.Gradients(ts, out), 0.5)
        assert abs(float(got) - norm) <= NORM_REL * norm
        _close(out[0], ts[0].double() * c, (NORM_REL + 3 * U) * (ts[0].double() * c).abs())
        assert not dst[:b].any() and not dst[b + n:].any()
    # a transposed matrix is dense; a scalar; no tensors
    m = _normal((30, 50), F32, g).t()
    want = m.clone()
    norm, c = _clip_ref([m], 1.0)
    lib.clip_grads([m, torch.zeros((), device="cuda")], 1.0)
    _close(m, want.double() * c, (NORM_REL + 3 * U) * (want.double() * c).abs())
    assert float(lib.clip_grads([], 1.0)) == 0.0
    assert float(lib.clip_grads([torch.zeros(0, device="cuda")], 1.0)) == 0.0


def test_clip_extremes(edd, lib):
    # squares that overflow or underflow float32
    for v, n in [(1e30, 1000), (3e38, 1), (1e-30, 1000), (1e-40, 77), (2.0 ** -149, 4), (1e19, 30001), (1e-23, 5)]:
        _check_clip(lib, edd, [torch.full((n,), v, device="cuda")], 0.5 * float(np.float32(v)), False)
    mixed = torch.tensor([3e25, 4e25, 1.0, 1e-30], device="cuda")
    _check_clip(lib, edd, [mixed, torch.full((5000,), 1e-25, device="cuda")], 1e3, True)
    # the norm itself is beyond float32: +inf is returned, the factor is right
    big = torch.full((1000,), 3e38, device="cuda")
    got = lib.clip_grads(edd.Gradients([big]), 1.0)
    assert math.isinf(float(got))
    _close(big, torch.full((1000,), 1 / math.sqrt(1000), dtype=torch.float64, device="cuda"),
           torch.full((1000,), 8 * U, dtype=torch.float64, device="cuda"))
    # an infinity or NaN: reported in the norm, gradients as they were
    for bad in (float("inf"), -float("inf"), float("nan")):
        for dt in (F32, F16, BF16):
            a = torch.randn(3000, device="cuda").to(dt)
            b = torch.randn(10, device="cuda").to(dt)
            a[1234] = bad
            a0, b0 = a.clone(), b.clone()
            out = [torch.empty_like(a), torch.empty_like(b)]
            n1 = float(lib.clip_grads(edd.Gradients([a, b], out), 0.1))
            n2 = float(lib.clip_grads([a, b], 0.1))
            for n in (n1, n2):
                assert math.isnan(n) if math.isnan(bad) else n == float("inf")
            for t, s in zip([a, b] + out, [a0, b0] * 2):
                assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
    # mostly zeros, as the gradient of a table, and values at the edges of the float32 sums
    for v in (1.0, 2.0 ** -55, 2.0 ** -56, 2.0 ** -60, 2.0 ** -70, 2.0 ** 50, 2.0 ** 51, 2.0 ** 64):
        for dt in (F32, BF16):
            z = torch.zeros(200003, device="cuda")
            z[::997] = v
            z[5000:5100] = -1.5 * v
            _check_clip(lib, edd, [z.to(dt)], 3.0 * float(np.float32(v)), False)
    # limits: zero, infinite, exactly the norm
    t = torch.tensor([3.0, 4.0], device="cuda")
    assert float(lib.clip_grads([t], 5.0)) == 5.0 and t.tolist() == [3.0, 4.0]
    assert float(lib.clip_grads([t], float("inf"))) == 5.0 and t.tolist() == [3.0, 4.0]
    assert float(lib.clip_grads([t], 0.0)) == 5.0 and t.tolist() == [0.0, 0.0]
    assert float(lib.clip_grads([t], 0.0)) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clip_factors_below_float32(edd, lib, dtype):
    # max_norm / N is subnormal or zero in float32, the clipped values are not
    g = _gen(str(dtype), 31)
    for top, n, max_norm in [(3e38, 1000, 1e-3), (3e38, 1000, 1e-6), (1e38, 2, 1e-6), (1e38, 5000, 1e-6), (1e20, 30, 1e-30),
                             (2.0 ** 100, 40001, 2.0 ** -40), (3e38, 9, 2e-38), (1e38, 10, 1.17)]:
        x = (torch.rand(n, generator=g, device="cuda") * 2 - 1) * top
        x[0], x[-1] = top, -top
        x[n // 2] = x[n // 2] * 1e-20
        x = x.to(dtype)
        limit = float(np.float32(max_norm))
        norm, c = _clip_ref([x], limit)
        assert c < 2.0 ** -125
        buf, dst = torch.zeros(n + 9, dtype=dtype, device="cuda"), torch.zeros(n + 9, dtype=dtype, device="cuda")
        for a, b in ((0, 0), (1, 1), (3, 2), (0, None)):  # None: in place
            src = buf[a:a + n]
            src.copy_(x)
            out = src if b is None else dst[b:b + n]
            got = float(lib.clip_grads(edd.Gradients([src], [out]), limit))
            assert math.isinf(got) if norm > 3.4028236e38 else abs(got - norm) <= NORM_REL * norm
            _close(out, x.double() * c, (NORM_REL + 3 * U) * (x.double() * c).abs())
    z = torch.full((10,), 1e38, device="cuda")
    lib.clip_grads([z], 0.0)
    assert not z.any()


def test_clip_lists_follow_their_tensors(edd, lib):
    # a kept list meets tensors that have other memory than when it was made
    g = _gen(41)
    ts = [_normal((n,), dt, g) for n, dt in ((1000, F32), (333, BF16), (70, F32))]
    out = [torch.empty_like(t) for t in ts]
    kept, kept_out = edd.Gradients(ts), edd.Gradients(ts, out)

    def check(limit_of):
        norm, c = _clip_ref(ts, 1.0)
        norm, c = _clip_ref(ts, limit_of * norm)
        before = [t.clone() for t in ts]
        assert abs(float(lib.clip_grads(kept_out, limit_of * norm)) - norm) <= NORM_REL * norm
        for o, s in zip(out, before):
            _close(o, s.double() * c, (NORM_REL + 4 * U) * (s.double() * c).abs())
        assert abs(float(lib.clip_grads(kept, limit_of * norm)) - norm) <= NORM_REL * norm
        assert all(torch.equal(t, o) for t, o in zip(ts, out))

    check(0.5)
    left = []  # the memory that tensors had before, and what it held then

    def leave(k):
        left.extend((t.data, t.clone()) for t in (ts[k], out[k]))

    leave(0)
    ts[0].data = _normal((1000,), F32, g)               # other memory
    out[0].data = torch.empty(1000, device="cuda")
    check(0.25)
    leave(1)
    ts[1].data = _normal((7, 11), F16, g)               # another type and shape
    out[1].data = torch.empty((7, 11), dtype=F16, device="cuda")
    check(0.25)
    leave(2)
    with torch.no_grad():
        ts[2].set_(_normal((5000,), F32, g))            # more elements
        out[2].set_(torch.empty(5000, device="cuda"))
    check(2.0)
    assert all(torch.equal(o, c) for o, c in left)
    # what the list could not have been made from is refused
    mine, theirs = ts[0].data, ts[1].data
    for bad in (torch.zeros(10), ts[2].data[:10], torch.zeros((10, 2), device="cuda")[:, 0]):
        ts[0].data = bad
        with pytest.raises(ValueError):
            lib.clip_grads(kept, 1.0)
    ts[0].data = mine
    check(0.5)
    assert ts[1].data_ptr() == theirs.data_ptr()
    lib.finish()


def test_embed_grad_unaligned_rows_in_big_tiles(lib):
    # enough units of wide unaligned rows for tiles of 512 columns: pairs and single elements
    for n, vocab, width, types in [(90000, 259, 322, (F16, F16)), (90000, 70, 323, (BF16, F32)), (50000, 20000, 530, (BF16, F32)),
                                   (90001, 5, 258, (F32, F32))]:
        g = _gen(n, vocab, width)
        t = _tokens(n, vocab, g, "zipf", 32, -1)
        dy = _normal((n, width), types[0], g, 1.0, 0.1)
        got = lib.embed_grad(t, dy, vocab, scale=0.75, pad=-1, dtype=types[1])
        want, mag, count = _embed_grad_ref(t, dy, vocab, 0.75, -1)
        _close(got, want, (count[:, None] + 1) * U * mag, "width %d" % width)
    lib.finish()


@pytest.mark.parametrize("count", [64, 65, 290, 384, 385, 1000, 1001])
def test_clip_list_lengths(edd, lib, count):
    # on both sides of each length of the tensor list that the launches carry
    g = _gen(count, 17)
    ts = [_normal((1 + 37 * i % 301,), (F32, BF16, F16)[i % 3], g, 0.5) for i in range(count)]
    norm = _clip_ref(ts, 1.0)[0]
    for in_place in (False, True):
        _check_clip(lib, edd, [t.clone() for t in ts], norm * 0.25, in_place)


# ---- streams, workspace, graphs ---------------------------------------------------------------

def test_another_stream(edd, lib):
    """Inputs made, and results read, on a stream that is not the context's."""
    side = torch.cuda.Stream()
    g = _gen(3)
    table = _normal((2000, 512), F32, g)
    t = _tokens(20000, 2000, g, "zipf")
    w = _normal((512,), F32, g)
    torch.cuda.synchronize()
    want_x = lib.embed(t, table, scale=2.0)
    want_y, m, r = lib.layer_norm(want_x, w)
    want = [want_y, *lib.layer_norm_grad(want_y, want_x, m, r, w)]
    want.append(lib.embed_grad(t, want[1], 2000, scale=2.0))
    flat = want[-1].clone()
    want.append(lib.clip_grads([flat], 1.0))
    want.append(flat)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            late = torch.zeros_like(table)
            for _ in range(20):
                late = late * 0.5  # keeps the side stream busy before the input is there
            late = late + table
            x = lib.embed(t, late, scale=2.0)
            y, m, r = lib.layer_norm(x, w)
            got = [y, *lib.layer_norm_grad(y, x, m, r, w)]
            got.append(lib.embed_grad(t, got[1], 2000, scale=2.0))
            flat = got[-1].clone()
            got.append(lib.clip_grads([flat], 1.0))
            got.append(flat)
            got = [v.clone() for v in got]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_workspace_limit_and_recovery(edd):
    j = edd.Join()
    try:
        t = torch.zeros(100000, dtype=torch.int64, device="cuda")
        dy = torch.ones((100000, 8), device="cuda")
        j.set_alloc_limit(4096)
        with pytest.raises(edd.HissError) as e:
            j.embed_grad(t, dy, 50)
        assert e.value.status == edd.HISS_E_NOMEM
        j.set_alloc_limit(0)
        assert float(j.embed_grad(t, dy, 50)[0, 0]) == 100000.0
        j.finish()
    finally:
        j.close()


def test_captured_in_a_graph(edd):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        j = edd.Join()
        g = _gen(6)
        table = _normal((300, 64), F32, g)
        t = _tokens(5000, 300, g, "zipf")
        w = _normal((64,), F32, g)

        def step():
            x = j.embed(t, table)
            y, m, r = j.layer_norm(x, w)
            dx, dw, db = j.layer_norm_grad(y, x, m, r, w)
            grad = j.embed_grad(t, dx, 300)
            norm = j.clip_grads(edd.Gradients([grad, dw, db]), 0.1)
            return grad, dw, db, norm

        step()  # sizes the workspace
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = step()
    for k in range(3):
        with torch.cuda.stream(s):
            table.copy_(_normal((300, 64), F32, _gen(k, 60)))
            t.copy_(_tokens(5000, 300, _gen(k, 61), "uniform"))
            graph.replay()
            got = [o.clone() for o in outs]
            want = step()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    j.finish()
    j.close()


def test_workspace_growth_keeps_captured_graphs(edd):
    # a graph holds the workspace it was captured with, whatever later calls need
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        j, other = edd.Join(), edd.Join()
        t = _tokens(5000, 300, _gen(61), "zipf")
        dy = _normal((5000, 64), F32, _gen(62))
        x = _normal((5000, 64), F32, _gen(63))
        _, m, r = j.layer_norm(x)

        def step(lib):
            grad = lib.embed_grad(t, dy, 300)
            dx, dw, db = lib.layer_norm_grad(dy, x, m, r)
            norm = lib.clip_grads([grad, dw, db], 0.1)
            return grad, dx, dw, db, norm

        def larger(lib, k):
            n, vocab = 100000 * k, 40000 * k
            grad = lib.embed_grad(_tokens(n, vocab, _gen(k, 64), "uniform"), torch.ones((n, 16), device="cuda"), vocab)
            lib.layer_norm_grad(torch.ones((k, 40000), device="cuda"), torch.ones((k, 40000), device="cuda"),
                                torch.zeros(k, device="cuda"), torch.ones(k, device="cuda"))
            lib.clip_grads([torch.ones(5, device="cuda") for _ in range(1000 * k + 1)], 1.0)
            assert float(grad.sum()) == 16.0 * n

        step(j)
        graphs = []
        for k in range(1, 4):
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs = step(j)
            graphs.append((graph, outs))
            larger(j, k)       # replaces what the graph uses
            larger(other, k)   # takes what would have been freed
            for graph, outs in graphs:
                dy.copy_(_normal((5000, 64), F32, _gen(k, 65)))
                graph.replay()
                larger(other, k)
                assert all(torch.equal(a, b) for a, b in zip(outs, step(other)))
                assert all(torch.equal(a, b) for a, b in zip(outs, step(j)))
        j.finish()
        other.finish()
        del graphs, graph
        j.close()
        other.close()


def test_capture_without_workspace_is_refused(edd):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        j = edd.Join()
        t = torch.zeros(5000, dtype=torch.int64, device="cuda")
        dy = torch.ones((5000, 8), device="cuda")
        m, r = torch.zeros(5000, device="cuda"), torch.ones(5000, device="cuda")
        hits = torch.zeros(3, device="cuda")
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            hits.add_(1)
            for call in (lambda: j.embed(t, dy), lambda: j.embed_grad(t, dy, 5), lambda: j.layer_norm_grad(dy, dy, m, r),
                         lambda: j.clip_grads([dy], 1.0), j.finish):
                with pytest.raises(edd.HissError) as e:
                    call()
                assert e.value.status == edd.HISS_E_STATE
            y = j.layer_norm(dy)[0]  # needs none
        graph.replay()
        s.synchronize()
        assert hits.tolist() == [1.0] * 3 and not y.any()
        # the context goes on, and the same calls can be captured once they have run
        assert float(j.embed_grad(t, dy, 5)[0, 0]) == 5000.0
        j.finish()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            grad = j.embed_grad(t, dy, 5)
        graph.replay()
        s.synchronize()
        assert grad.sum(1).tolist() == [40000.0, 0, 0, 0, 0]
        j.close()


# ---- refusals ----------------------------------------------------------------------------------

def test_refusals(edd, lib):
    f = torch.zeros((8, 16), device="cuda")
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    m = torch.zeros(8, device="cuda")
    for call in [
        lambda: lib.embed(t.float(), f), lambda: lib.embed(t.cpu(), f), lambda: lib.embed(t, f.double()),
        lambda: lib.embed(t, f.cpu()), lambda: lib.embed(t, f[0]), lambda: lib.embed(t, f, out=torch.zeros((8, 15), device="cuda")),
        lambda: lib.embed(t, f, out=torch.zeros((16, 8), device="cuda").t()),
        lambda: lib.embed(t, torch.zeros((2, 65537), device="cuda")),
        lambda: lib.embed_grad(t, f[:7], 5), lambda: lib.embed_grad(t, f, 5, accumulate=True),
        lambda: lib.embed_grad(t, f, 5, out=torch.zeros((5, 17), device="cuda")),
        lambda: lib.layer_norm(f.double()), lambda: lib.layer_norm(f, f[0, :15]), lambda: lib.layer_norm(f, f[0], f[0].half()),
        lambda: lib.layer_norm(f.cpu()), lambda: lib.layer_norm(torch.zeros((), device="cuda")),
        lambda: lib.layer_norm(torch.zeros((3, 0), device="cuda")),
        lambda: lib.layer_norm_grad(f[:7], f, m, m), lambda: lib.layer_norm_grad(f, f, m[:7], m),
        lambda: lib.layer_norm_grad(f, f, m.half(), m),
        lambda: edd.Gradients([f.cpu()]), lambda: edd.Gradients([f[:, :8]]), lambda: edd.Gradients([f, f]),
        lambda: edd.Gradients([f, f.flatten()[100:]]), lambda: edd.Gradients([f], [f.half()]), lambda: edd.Gradients([f], []),
        lambda: edd.Gradients([f.flatten()[:64]], [f.flatten()[32:96]]), lambda: edd.Gradients([f.double()]),
    ]:
        with pytest.raises(ValueError):
            call()
    for call in [
        lambda: lib.embed(t, f, scale=float("nan")), lambda: lib.embed(t, f, scale=float("inf")),
        lambda: lib.embed(t, f, out=f), lambda: lib.embed_grad(t, f, 0), lambda: lib.layer_norm(f, eps=-1.0),
        lambda: lib.layer_norm(f, eps=float("nan")), lambda: lib.layer_norm(f, eps=float("inf")), lambda: lib.layer_norm(f, out=f),
        lambda: lib.layer_norm(f, dtype=torch.bfloat16), lambda: lib.layer_norm_grad(f.half(), f, m, m),
        lambda: lib.clip_grads([f], -1.0), lambda: lib.clip_grads([f], float("nan")),
        lambda: lib.embed(t, f, out=torch.zeros((1, 16), device="cuda").expand(8, 16)),
    ]:
        with pytest.raises(edd.HissError) as e:
            call()
        assert e.value.status == edd.HISS_E_ARG
    assert not f.any()
    lib.finish()


def test_c_refusals(edd, lib):
    f = torch.zeros((8, 16), device="cuda")
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    o = torch.zeros((8, 16), device="cuda")
    h, F, p, q, r, z = lib.handle, edd.HISS_F32, f.data_ptr(), t.data_ptr(), o.data_ptr(), edd.HISS_NO_PAD
    E = edd.HISS_E_ARG
    assert edd.hiss_embed(None, p, F, 8, 16, 16, q, 64, 8, z, 1.0, r, F, 16) == E
    ok = [h, p, F, 8, 16, 16, q, 64, 8, z, 1.0, r, F, 16]
    for at, bad in [(1, None), (1, p + 2), (2, 3), (2, -1), (3, 0), (3, 1 << 31), (4, 0), (4, 65537), (5, -1), (5, 1 << 31),
                    (6, None), (6, q + 4), (7, 16), (8, -1), (8, 1 << 30), (10, math.inf), (11, None), (11, r + 1), (12, 9),
                    (13, 15), (11, p)]:
        args = list(ok)
        args[at] = bad
        assert edd.hiss_embed(*args) == E, (at, bad)
    assert edd.hiss_embed(*ok) == 0
    ok = [h, p, F, 16, q, 64, 8, z, 1.0, 8, 16, 0, r, F, 16]
    for at, bad in [(1, None), (2, 3), (3, -1), (4, None), (5, 8), (6, -5), (8, math.nan), (9, 0), (9, 1 << 31), (10, 0), (11, 2),
                    (11, -1), (12, None), (12, p + 4), (13, 4), (14, 15)]:
        args = list(ok)
        args[at] = bad
        assert edd.hiss_embed_grad(*args) == E, (at, bad)
    assert edd.hiss_embed_grad(*ok) == 0
    w = torch.ones(16, device="cuda")
    s = torch.zeros((2, 8), device="cuda")
    ok = [h, p, F, 16, 8, 16, w.data_ptr(), None, F, 1e-5, r, F, 16, s.data_ptr(), s[1].data_ptr()]
    for at, bad in [(1, None), (2, 5), (3, -1), (4, -1), (4, 1 << 30), (5, 0), (5, 65537), (6, w.data_ptr() + 1), (8, 7), (9, -1.0),
                    (10, None), (10, p), (10, w.data_ptr()), (11, edd.HISS_BF16), (12, 3), (13, s.data_ptr() + 2), (14, s.data_ptr()),
                    (13, r)]:
        args = list(ok)
        args[at] = bad
        assert edd.hiss_layer_norm(*args) == E, (at, bad)
    assert edd.hiss_layer_norm(*ok) == 0
    dp = torch.zeros((2, 16), device="cuda")
    ok = [h, p, F, 16, o.data_ptr(), F, 16, s.data_ptr(), s[1].data_ptr(), w.data_ptr(), F, 8, 16, None, 16, dp.data_ptr(),
          dp[1].data_ptr()]
    for at, bad in [(1, None), (2, 5), (3, -1), (4, None), (2, edd.HISS_F16), (7, None), (8, None), (10, 3), (11, -1), (12, 0),
                    (13, p), (15, dp[1].data_ptr()), (16, w.data_ptr()), (16, dp.data_ptr() + 64 + 2)]:
        args = list(ok)
        args[at] = bad
        assert edd.hiss_layer_norm_grad(*args) == E, (at, bad)
    assert edd.hiss_layer_norm_grad(*ok) == 0
    norm = torch.zeros(1, device="cuda")

    def clip(ts, count=None, limit=1.0, to=norm.data_ptr()):
        a = (edd.hiss_tensor * max(1, len(ts)))(*[edd.hiss_tensor(*v) for v in ts])
        return edd.hiss_clip_grads(h, a, len(ts) if count is None else count, limit, to)

    for ts in [[(p, None, -1, F, 0)], [(None, None, 4, F, 0)], [(p, None, 4, 3, 0)], [(p + 2, None, 4, F, 0)], [(p, r + 1, 4, F, 0)],
               [(p, p + 4, 4, F, 0)], [(p, None, 4, F, 1)], [(norm.data_ptr(), None, 1, F, 0)], [(p, None, 1 << 60, F, 0)]]:
        assert clip(ts) == E, ts
    assert clip([], -1) == E and clip([(p, None, 4, F, 0)], limit=-1.0) == E and clip([(p, None, 4, F, 0)], to=None) == E
    assert edd.hiss_clip_grads(h, None, 1, 1.0, norm.data_ptr()) == E
    assert clip([(None, None, 0, F, 0), (p, None, 4, F, 0)]) == 0
    assert edd.hiss_finish(None) == E
    lib.finish()
    assert not f.any()


def test_empty_operands_overlap_nothing(edd, lib):
    # a matrix of no rows has no elements, wherever its pointer lies
    f = torch.full((8, 16), 9.0, device="cuda")
    s = torch.zeros((2, 8), device="cuda")
    h, F, p, z = lib.handle, edd.HISS_F32, f.data_ptr(), edd.HISS_NO_PAD
    assert edd.hiss_embed(h, p, F, 8, 16, 16, None, 64, 0, z, 1.0, p + 64, F, 16) == 0
    assert edd.hiss_layer_norm(h, p + 64, F, 16, 0, 16, p, None, F, 1e-5, p + 128, F, 16, s.data_ptr(), s.data_ptr()) == 0
    torch.cuda.synchronize()
    assert bool((f == 9.0).all())
    assert edd.hiss_embed_grad(h, p + 64, F, 16, None, 64, 0, z, 1.0, 8, 16, 0, p, F, 16) == 0
    dw = torch.full((16,), 9.0, device="cuda")
    assert edd.hiss_layer_norm_grad(h, dw.data_ptr() + 4, F, 16, dw.data_ptr() + 4, F, 16, None, None, None, F, 0, 16, None, 16,
                                    dw.data_ptr(), None) == 0
    lib.finish()
    assert not f.any() and not dw.any()


# ---- together: a table is learned, and its rows are joined --------------------------------------

def test_operators_leave_the_join_alone(edd):
    import oracle
    j = edd.Join()
    try:
        g = _gen(12)
        table = _normal((400, 16), F32, g)
        x, m, r = j.layer_norm(j.embed(torch.arange(400, device="cuda"), table, scale=4.0))
        j.build(x)
        before = j.join_sets(2.0)
        j.embed_grad(torch.arange(400, device="cuda") % 7, x, 7)
        j.clip_grads([table], 1.0)
        after = j.join_sets(2.0)
        want = oracle.row_sets(x.cpu().numpy(), 2.0, np.arange(400))
        for q in range(400):
            sure, band = want[q]
            assert set(before[q].tolist()) == set(after[q].tolist())
            assert sure <= set(after[q].tolist()) <= sure | band
    finally:
        j.close()
