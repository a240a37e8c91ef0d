"""The operators together with the join, as examples/learn_points.py uses
them: the table learns its groups, and each step's gradient is the one that
torch's own differentiation of the same loss gives."""
import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("learn_points", os.path.join(ROOT, "examples", "learn_points.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_joined_pairs_are_those_within_eps(example):
    learner = example.Learner(items=600, groups=30, batch=400)
    _, y, _, _ = learner.points(torch.arange(600, device="cuda"))
    i, j = example.joined_pairs(learner.lib, y, 6.5)
    d = torch.cdist(y.double(), y.double())
    d.fill_diagonal_(float("inf"))
    got = torch.zeros((600, 600), dtype=torch.bool, device="cuda")
    got[i, j] = True
    assert int(got.sum()) == i.numel() > 0
    edge = (d - 6.5).abs() < 1e-4  # float32 distances of values up to about 4
    assert bool((got == (d <= 6.5))[~edge].all())


def test_step_gradient_is_the_loss_gradient(example):
    """One step from the same state through torch in float64."""
    learner = example.Learner(items=300, groups=20, batch=240, eps=7.0, seed=3)
    table, weight, bias = (p.clone() for p in (learner.table, learner.weight, learner.bias))
    state = learner.gen.get_state()
    loss = learner.step(rate=1.0, max_norm=float("inf"))
    learner.gen.set_state(state)
    items = torch.randint(0, 300, (240,), generator=learner.gen, device="cuda")
    live = items[:240 - 240 // 20]
    t, w, b = (p.double().requires_grad_() for p in (table, weight, bias))
    x = float(torch.tensor(32 ** 0.5)) * t[live]
    y = torch.nn.functional.layer_norm(x, (32,), w, b, 1e-5)
    g = learner.group[live]
    order = torch.argsort(g, stable=True)
    a, c = order[:-1], order[1:]
    same = g[a] == g[c]
    near = 0.5 * (y[a[same]] - y[c[same]]).square().sum()
    i, j = torch.triu_indices(live.numel(), live.numel(), 1, device="cuda")
    apart = g[i] != g[j]
    r = (y[i[apart]] - y[j[apart]]).norm(dim=1)
    far = 0.5 * (7.0 - r).clamp_min(0).square().sum()
    total = near + far
    total.backward()
    # the forces between pairs cancel in the bias's gradient, which is zero: its
    # error is that of float32 sums over up to 240 partners and 240 rows, 480 u
    # times the sum of the forces' magnitudes; 1e-4 of the largest gradient is far
    # above the rounding of the other sums
    with torch.no_grad():
        forces = (y[a[same]] - y[c[same]]).norm(dim=1).sum() + (7.0 - r).clamp_min(0).sum()
    rounding = 480 * 2.0 ** -24 * 2 * float(forces)
    assert abs(loss - float(total.detach()) / 240) <= 1e-4 * abs(loss)
    for got, old, ref in ((learner.table, table, t), (learner.weight, weight, w), (learner.bias, bias, b)):
        d = (old - got).double() - ref.grad
        zero = ref is b
        assert float(d.abs().max()) <= (rounding if zero else 1e-4 * float(ref.grad.abs().max()))


def test_the_table_learns_its_groups(example):
    learner = example.Learner()
    before = learner.purity()
    losses = learner.learn(300)
    after = learner.purity()
    # two groups that meet are pushed apart only once they are distinct points,
    # so a few may stay together; every group finds itself
    assert losses[-1] < 0.05 * losses[0]
    assert before[1] < 0.05 and after[0] > 0.7 and after[1] > 0.95, (before, after)
