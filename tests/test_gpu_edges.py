"""The feed-forward block's activations over their range and the layer norm's gradient from 8 bits at
constant rows, against the formulas in float64.  Errors are relative to the value, or to the terms that it is
the sum of."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
U = 2.0 ** -24
# Half a step relative to the value, and half the smallest subnormal; in products of float32 the last of a
# number's three bfloat16 parts is cut to a multiple of bfloat16's smallest subnormal, 2^-133.
ROUND = {F32: (U, 2.0 ** -133), F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -134)}
LARGEST = {F32: 80.0, F16: 14.0, BF16: 80.0}  # of a


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import exact_dimensional_distance_gb300 as edd
    j = edd.Join()
    yield j
    j.finish()
    j.close()


def _range(dtype, n, largest):
    return torch.linspace(-largest, largest, n, device="cuda", dtype=torch.float64).to(dtype)


def _terms(a, act):
    """The activation and the terms that its derivative is the sum of."""
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-a / math.sqrt(2))
        return a * p, (p, a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi))
    s = torch.sigmoid(a)
    slope = s * torch.sigmoid(-a)
    return (s, (slope,)) if act == "sigmoid" else (a * s, (s, a * slope))


def _relative(a, act, dtype):
    """float32: 16 steps, of the exponential, the sum, the inverse and the products, and 2^-22 of a product of
    three parts.  16-bit: the fast exponential of x, (|x| + 2) 2^-23, x = a / ln 2, and three such steps.  The normal
    distribution: three roundings of x = a^2 / (2 ln 2), a step of e^x being x ln 2 of one of x, and its polynomial."""
    if act == "gelu":
        return (3 * a * a / 2 + 32) * U + (4e-7 if dtype == F32 else 2.2e-6)
    return 20 * U + 0 * a if dtype == F32 else (a.abs() * 1.4427 + 8) * 2 * U


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_derivatives_over_the_range(lib, dtype, act):
    """da of each row in a column of its own of the gate's gradient, where b and dh are 1 (float16: dh is 1024)."""
    n, dh = 600, 1024.0 if dtype == F16 else 1.0
    largest = min(LARGEST[dtype], 12.0) if act == "gelu" else LARGEST[dtype]
    x = torch.zeros((n, 2 + n), dtype=dtype, device="cuda")
    x[:, 0], x[:, 1], x[:, 2:] = _range(dtype, n, largest), 1, torch.eye(n, dtype=dtype, device="cuda")
    gate, up = torch.zeros((1, 2 + n), dtype=dtype, device="cuda"), torch.zeros((1, 2 + n), dtype=dtype, device="cuda")
    gate[0, 0], up[0, 1] = 1, 1
    down, dy = torch.ones((1, 1), dtype=dtype, device="cuda"), torch.full((n, 1), dh, dtype=dtype, device="cuda")
    got = lib.feed_forward_grad(dy, x, gate, up, down, act=act)[1][0, 2:].double()
    a = x[:, 0].double()
    terms = _terms(a, act)[1]
    want, size = dh * sum(terms), dh * sum(t.abs() for t in terms)
    rel, sub = ROUND[dtype]  # of da, and of the result
    bad = ~((got - want).abs() <= _relative(a, act, dtype) * size * (1 + 2 * rel) + 2 * (rel * want.abs() + sub))
    assert not bool(bad.any()), [(float(a[i]), float(got[i]), float(want[i])) for i in torch.nonzero(bad).flatten()[:5]]


@pytest.mark.parametrize("width", [64, 128, 520, 2048, 12288])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_gradient_of_constant_rows_kept_in_8_bits(lib, dtype, width):
    """Rows whose value 8 bits hold exactly: x - mean is 0 there, so dweight is 0 and dx = rstd (g - mean(g)), the
    same from rows that the kernel reads in 8 bits (dy and dx aligned) and from rows that are unpacked first."""
    values = [1000.0, -3.0, 0.0, 127.0, 2.0 ** -10, 100.0] + ([] if dtype == F16 else [2.0 ** 120, -2.0 ** 119])
    x = torch.tensor(values, device="cuda").to(dtype)[:, None].expand(len(values), width).contiguous()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(width)
    dy = torch.randn((len(values), width), generator=gen, device="cuda").to(dtype)
    w = 1 + 0.3 * torch.randn(width, generator=gen, device="cuda")
    # by the definition: layer_norm's float32 sum of 520 times 2^120 overflows
    mean, rstd = x[:, 0].float(), torch.full((len(values),), 1e-5 ** -0.5, device="cuda")
    p = lib.pack(x)
    assert torch.equal(lib.unpack(p), x)
    buf = torch.zeros((len(values), width + 1), dtype=dtype, device="cuda")
    apart = buf[:, 1:]  # rows that are not aligned
    apart.copy_(dy)
    g = dy.double() * w.double()
    want = rstd.double()[:, None] * (g - g.mean(1, keepdim=True))
    # float32 sums of width terms, four steps of each element, the result's rounding
    err = rstd.double()[:, None] * U * (4 * g.abs() + (width + 8) * g.abs().mean(1, keepdim=True))
    for v in (dy, apart):
        dx, dw, db = lib.layer_norm_grad(v, p, mean, rstd, w)
        assert not bool(dw.any())
        assert bool(((dx.double() - want).abs() <= err + 2 * ROUND[dtype][0] * want.abs() + ROUND[dtype][1]).all())
        assert bool(((db.double() - dy.double().sum(0)).abs() <= len(values) * U * dy.double().abs().sum(0)).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_gradient_far_from_zero(lib, dtype):
    """Rows whose mean is far above their spread, of values that 8 bits hold exactly: h = (x - mean) rstd is off by
    the mean's and its own three roundings alone, wherever the rows lie."""
    n, width = 64, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    x = (120 + torch.randint(0, 8, (n, width), generator=gen, device="cuda")).to(dtype) * 8
    dy = torch.randn((n, width), generator=gen, device="cuda").to(dtype)
    _, mean, rstd = lib.layer_norm(x)
    p = lib.pack(x)
    assert torch.equal(lib.unpack(p), x)
    d, r = dy.double(), rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * r
    dw = lib.layer_norm_grad(dy, p, mean, rstd, torch.ones(width, device="cuda"))[1]
    err = (n + 4) * U * (d * h).abs().sum(0)
    assert bool(((dw.double() - (d * h).sum(0)).abs() <= err).all())


@pytest.mark.parametrize("n", [1, 7, 16, 50, 600])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_over_the_range(lib, dtype, act, n):
    """y = act(a), from each of the block's kernels."""
    largest = min(LARGEST[dtype], 12.0) if act == "gelu" else LARGEST[dtype]
    e = torch.eye(2, dtype=dtype, device="cuda")
    for part in _range(dtype, 600, largest).split(n)[::max(1, 600 // n // 40)]:
        x = torch.stack((part, torch.ones_like(part)), 1)
        y = lib.feed_forward(x, e[:1], e[1:], e[:1, :1], act=act)[:, 0].double()
        a = part.double()
        want = _terms(a, act)[0]
        rel, sub = ROUND[dtype]  # of h, and of the result
        bad = ~((y - want).abs() <= _relative(a, act, dtype) * want.abs() * (1 + 2 * rel) + 2 * (rel * want.abs() + sub))
        assert not bool(bad.any()), [(float(a[i]), float(y[i]), float(want[i])) for i in torch.nonzero(bad).flatten()[:5]]
