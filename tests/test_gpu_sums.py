"""Long sums of the feed-forward block.  The tensor cores cut a sum towards zero at each step of 16
columns, so no accumulator may take in many: what it lost shows in means of terms of one sign, in the
codes of kept projections and in the signs that relu's derivative takes."""
import zlib

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}  # half a step, relative
# A rounding's error relative to the value, in the 2-norm: uniform within half a step of 2^e, over values
# whose logarithms are: sqrt(1 / 3 * 3 / (8 ln 2)) half steps.
ROUNDING = 0.43


def _error(width, few=False):
    """The mean error of a projection of 16-bit rows over its size, the 2-norm of its terms.  A step loses half of
    2^-23 of its range's sum so far on average, which after j steps is sqrt(16 j / width) of the size.  Ranges have signs of
    their own: the large products' first two, of 32 steps (the sum of sqrt(j) is 123), and the others, of 16 (44.5).
    The ranges' additions in float32 are each off by a quarter of 2^-23 on average of a sum that is sqrt(1/2) of the
    whole on average."""
    long = 0 if few else 2
    lost = ((long * (4 * 123) ** 2 + (width - 512 * long) / 256 * (4 * 44.5) ** 2) / width) ** 0.5
    return lost * 2.0 ** -24 + 2.0 ** -25 * (width / 512) ** 0.5


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import exact_dimensional_distance_gb300 as edd
    j = edd.Join()
    yield j
    j.finish()
    j.close()


def _gen(*seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(seed).encode()))
    return g


def _normal(shape, dtype, gen, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def _positive(shape, dtype, gen, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda").abs()).to(dtype)


def _kept(v):
    """(codes, scales, scale bytes) of float64 rows by the definition."""
    n, f = v.shape
    m = torch.nn.functional.pad(v.abs(), (0, -f % 32)).view(n, -1, 32).amax(2)
    e = torch.ceil(torch.log2(m.clamp_min(2.0 ** -140) / 127))
    e = torch.where(127 * torch.exp2(e) < m, e + 1, e)
    e = torch.where(127 * torch.exp2(e - 1) >= m, e - 1, e).clamp_min(-126)
    s = torch.exp2(e).repeat_interleave(32, 1)[:, :f]
    return (v / s).round(), s, (e + 127).to(torch.uint8)


# ---- codes of what was kept --------------------------------------------------------

def _count_codes(lib, dtype, n, d, f, inputs, few=False):
    """A code differs from the definition's where an error carries a value across the middle of two: by chance
    (error / scale).  A block's scale differs where its largest value crosses 127 scales, 1 / 64 as often."""
    count, blocks, expected, expected_blocks = 0, 0, 0.0, 0.0
    for i in range(inputs):
        g = _gen(n, d, f, str(dtype), i)
        x, gate, up = _normal((n, d), dtype, g), _normal((f, d), dtype, g, d ** -0.5), _normal((f, d), dtype, g, d ** -0.5)
        _, kept = lib.feed_forward(x, gate, up, _normal((8, f), dtype, g), act="relu", keep=True)
        for k, w in zip(kept, (gate, up)):
            codes, s, byte = _kept(x.double() @ w.double().t())
            size = (x.double().square() @ w.double().square().t()).sqrt()
            same = (k.scales == byte).repeat_interleave(32, 1)[:, :f]
            count += int(((k.codes[:, :f] != codes) & same).sum())
            blocks += int((k.scales != byte).sum())
            expected += _error(d, few) * float((size / s).sum())
            expected_blocks += _error(d, few) * float((size / s).sum()) / 64 / 32
    # five times the spread of a count
    assert count <= expected + 5 * expected ** 0.5 + 5
    assert blocks <= expected_blocks + 5 * expected_blocks ** 0.5 + 5


#                                    rows, width, hidden, inputs
@pytest.mark.parametrize("n,d,f,inputs", [(1024, 4096, 2048, 1), (300, 8200, 1000, 3), (100, 16384, 520, 6), (70, 65536, 136, 16)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_codes_of_kept_projections(lib, dtype, n, d, f, inputs):
    _count_codes(lib, dtype, n, d, f, inputs)


# ---- signs that relu's derivative takes -----------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
def test_signs_of_projections_computed_again(lib, dtype):
    """Projections near zero whose sums go far from it and back.  Each row of x has a column of its own, in
    which gate and up are 0: there the gate's gradient is da itself.  Eight times the
    mean error settles the sign."""
    n, half, near, f, o = 256, 8192, 32, 512, 64
    d = 2 * half + near + n
    g = _gen(str(dtype))
    x, gate = torch.zeros((n, d), dtype=dtype, device="cuda"), torch.zeros((f, d), dtype=dtype, device="cuda")
    x[:, :half], gate[:, :half] = _normal((n, half), dtype, g), _normal((f, half), dtype, g, half ** -0.5)
    x[:, half:2 * half], gate[:, half:2 * half] = -x[:, :half], gate[:, :half]
    x[:, 2 * half:2 * half + near] = _normal((n, near), dtype, g, 2.0 ** -9)
    gate[:, 2 * half:2 * half + near] = _normal((f, near), dtype, g, half ** -0.5)
    up = torch.zeros_like(gate)
    up[:, :half] = _normal((f, half), dtype, g, half ** -0.5)
    x[:, d - n:] = torch.eye(n, dtype=dtype, device="cuda")
    down, dy = _normal((o, f), dtype, g), _normal((n, o), dtype, g)
    dgate = lib.feed_forward_grad(dy, x, gate, up, down, act="relu")[1]
    a = x.double() @ gate.double().t()
    size = (x.double().square() @ gate.double().square().t()).sqrt()
    db = (dy.double() @ down.double()) * (x.double() @ up.double().t())
    settled = (a.abs() >= 8 * _error(d) * size) & (db.abs() > 2.0 ** -8)
    assert float(settled.double().mean()) > 0.5
    wrong = ((dgate[:, d - n:].t() != 0) != (a > 0)) & settled
    assert int(wrong.sum()) == 0


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_of_wide_blocks_with_relu(lib, dtype, keep):
    """Each gradient in norm, within 1.5 times its two roundings: of da, db or h, and its own."""
    n, d, f, o = 600, 4096, 520, 264
    g = _gen(str(dtype), keep)
    x, dy = _normal((n, d), dtype, g), _normal((n, o), dtype, g, 0.5)
    gate, up, down = _normal((f, d), dtype, g, d ** -0.5), _normal((f, d), dtype, g, d ** -0.5), _normal((o, f), dtype, g, f ** -0.5)
    kept = lib.feed_forward(x, gate, up, down, act="relu", keep=True)[1] if keep else None
    got = lib.feed_forward_grad(dy, x, gate, up, down, act="relu", kept=kept)
    xd, gd, ud, dd, v = (t.double() for t in (x, gate, up, down, dy))
    a, b = xd @ gd.t(), xd @ ud.t()
    if keep:
        a, b = (c * s for c, s, _ in map(_kept, (a, b)))
    dh = v @ dd
    da, db = dh * b * (a > 0), dh * a.clamp_min(0)
    want = (da @ gd + db @ ud, da.t() @ xd, db.t() @ xd, v.t() @ (a.clamp_min(0) * b))
    for name, t, w in zip(("dx", "dgate", "dup", "ddown"), got, want):
        off = float((t.double() - w).norm() / w.norm())
        assert off <= 1.5 * 2 ** 0.5 * ROUNDING * HALF[dtype], name


# ---- where accumulators change -----------------------------------------------------

#                                   whole accumulators, one block or one column more or less; ranges of K and none
@pytest.mark.parametrize("n,d,f,o", [(300, 512, 1024, 5200), (300, 513, 1025, 5200), (300, 1024, 2048, 5200), (300, 1025, 2049, 5200),
                                     (300, 1279, 3000, 200), (300, 1280, 1088, 200), (300, 1281, 960, 5200), (100, 1600, 130, 4096),
                                     (100, 65, 130, 4097), (70, 64, 200, 6145)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sums_of_every_length(lib, dtype, n, d, f, o):
    """The value and all gradients, computed again and from kept rows, in norm: within 1.5 times their two roundings."""
    g = _gen(n, d, f, o, str(dtype))
    x, dy = _normal((n, d), dtype, g), _normal((n, o), dtype, g, 0.5)
    gate, up, down = _normal((f, d), dtype, g, d ** -0.5), _normal((f, d), dtype, g, d ** -0.5), _normal((o, f), dtype, g, f ** -0.5)
    y, kept = lib.feed_forward(x, gate, up, down, act="silu", keep=True)
    xd, gd, ud, dd, v = (t.double() for t in (x, gate, up, down, dy))
    for keep in (None, kept):
        a, b = (xd @ gd.t(), xd @ ud.t()) if keep is None else (lib.unpack(k).double() for k in keep)
        s = torch.sigmoid(a)
        if keep is None:
            off = float((y.double() - (a * s * b) @ dd.t()).norm() / ((a * s * b) @ dd.t()).norm())
            assert off <= 1.5 * 2 ** 0.5 * ROUNDING * HALF[dtype], "y"
        dh = v @ dd
        da, db = dh * b * s * (1 + a * (1 - s)), dh * a * s
        want = (da @ gd + db @ ud, da.t() @ xd, db.t() @ xd, v.t() @ (a * s * b))
        for name, t, w in zip(("dx", "dgate", "dup", "ddown"), lib.feed_forward_grad(dy, x, gate, up, down, act="silu", kept=keep), want):
            off = float((t.double() - w).norm() / w.norm())
            assert off <= 1.5 * 2 ** 0.5 * ROUNDING * HALF[dtype], name


# ---- terms of one sign --------------------------------------------------------------

# Ranges of 1024 columns, of 64 steps: a step loses at most 2^-23 of the range's sum so far, which is half of it
# on average: 2^-18 of the whole.
LOST = 2.0 ** -18


def _biased(got, want, lost, values):
    """The mean relative error is within lost and five times the spread of that many roundings' mean."""
    off = float((got.double() / want - 1).mean())
    assert abs(off) <= lost + 5 * ROUNDING * HALF[got.dtype] / values ** 0.5, off


@pytest.mark.parametrize("n", [16384, 65536, 1 << 20])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weight_gradients_over_many_rows(lib, dtype, n):
    d, f, o = 32, 256, 256
    g = _gen(n, str(dtype))
    x, dy = _positive((n, d), dtype, g), _positive((n, o), dtype, g, 2.0 ** -12)
    gate, up, down = (_positive(s, dtype, g, 0.2) for s in ((f, d), (f, d), (o, f)))
    ddown = lib.feed_forward_grad(dy, x, gate, up, down, act="relu")[3]
    h = ((x.double() @ gate.double().t()) * (x.double() @ up.double().t())).to(dtype)
    # The elements of a column are sums of n products of one mean, whose spread relative to it is sqrt(0.6) (the
    # squares' mean of dy is pi / 2 times its mean's square, that of h 1.03 times): the sums' is sqrt(0.6 / n).
    # Where that is below a quarter of half a step (bfloat16, 2^20 rows), a column is rounded as one: f values.
    values = f * o if (0.6 / n) ** 0.5 > HALF[dtype] / 4 else f
    _biased(ddown, dy.double().t() @ h.double(), LOST + 2.0 ** -20, values)  # some of h round to the other side


@pytest.mark.parametrize("n,d,f,o", [(128, 65536, 64, 128), (128, 32, 65536, 128), (128, 128, 64, 65536), (128, 128, 64, 20000)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_wide_blocks(lib, dtype, n, d, f, o):
    """Width, hidden or out width up to the largest: the value, and dx where the out width is long.  Ranges of a and
    b are shorter: at most 17 * 2^-23 lost in each.  Roundings: of what goes into the last product, and the result's."""
    g = _gen(n, d, f, o, str(dtype))
    x, gate, up = _positive((n, d), dtype, g), _positive((f, d), dtype, g, 1 / d), _positive((f, d), dtype, g, 1 / d)
    down, dy = _positive((o, f), dtype, g, 2.0 ** -6), _positive((n, o), dtype, g, 2.0 ** -10)
    xd, gd, ud, dd, v = (t.double() for t in (x, gate, up, down, dy))
    a, b = xd @ gd.t(), xd @ ud.t()
    if o > max(d, f):
        dh = v @ dd
        got, want, inner = lib.feed_forward_grad(dy, x, gate, up, down, act="relu")[0], (dh * b) @ gd + (dh * a) @ ud, 2 * n * f
    else:
        got, want, inner = lib.feed_forward(x, gate, up, down, act="relu"), (a * b) @ dd.t(), n * f
    _biased(got, want, LOST + 34 * 2.0 ** -23, 1 / (1 / want.numel() + 1 / inner))


# ---- few rows -----------------------------------------------------------------------

@pytest.mark.parametrize("n,d,f,inputs", [(5, 2048, 16384, 64), (16, 1000, 15000, 32), (33, 2000, 2960, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_codes_of_few_rows(lib, dtype, n, d, f, inputs):
    _count_codes(lib, dtype, n, d, f, inputs, few=True)


@pytest.mark.parametrize("n,d,f,o", [(16, 4096, 11008, 4096), (9, 64, 22016, 8192), (32, 64, 22016, 8192), (20, 20000, 1000, 64)])
def test_few_float32_rows(lib, n, d, f, o):
    """Ranges of 128 columns, 8 steps: as in _error, the sum of sqrt(j) is 16.3, so 16.3 * 4 / sqrt(128) = 5.8 halves of
    2^-23 in each product; two additions per range, a quarter of 2^-23 each of sqrt(1/2) of the sum; and what three
    parts leave out, 2^-23.  The value's error has those of a and b in it.  Half as much again for the inputs' spread."""
    def product(width):
        return 5.8 * 2.0 ** -24 + 2.0 ** -25 * (width / 128) ** 0.5 + 2.0 ** -23
    g = _gen(n, d, f, o)
    x = _normal((n, d), F32, g)
    gate, up, down = _normal((f, d), F32, g, d ** -0.5), _normal((f, d), F32, g, d ** -0.5), _normal((o, f), F32, g, f ** -0.5)
    y = lib.feed_forward(x, gate, up, down, act="relu").double()
    xd, dd = x.double(), down.double()
    want = ((xd @ gate.double().t()).clamp_min(0) * (xd @ up.double().t())) @ dd.t()
    off = float((y - want).norm() / want.norm())
    assert off <= 1.5 * (product(f) ** 2 + 2 * product(d) ** 2) ** 0.5, off
    # terms of one sign: 8 steps that lose at most 2^-23 of a half of their range's sum on average
    x, gate, up, down = (t.abs() for t in (x, gate, up, down))
    y = lib.feed_forward(x, gate, up, down, act="relu").double()
    xd, dd = x.double(), down.double()
    want = ((xd @ gate.double().t()) * (xd @ up.double().t())) @ dd.t()
    off = float((y / want - 1).mean())
    assert abs(off) <= 3 * (4.5 + 1) * 2.0 ** -23, off
