"""Learning the points that the join searches.

    python examples/learn_points.py [--steps N]

A table of embeddings is trained so that items of one group lie close together
and items of different groups at least eps apart, on synthetic groups:

    points = layer norm of scale * table[item]           (Join.embed, Join.layer_norm)
    loss   = 1/2 |p_i - p_j|^2 over pairs (i, j) of one group, drawn at random,
           + 1/2 (eps - |p_i - p_j|)^2 over the pairs of different groups that are
             within eps of one another

The second sum is what makes the join part of the training step: the pairs
with a non-zero term are exactly the result of the epsilon join of the points
(Join.build, Join.join), so no pair is missed and none is scanned in vain.  The
way back is the gradient of the layer norm, the gradient of the lookup by
sorted items, and clipping by the global norm (Join.layer_norm_grad,
Join.embed_grad, Join.clip_grads).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_dimensional_distance_gb300 as edd  # noqa: E402

PAD = -1


def joined_pairs(lib, points, eps):
    """(i, j) of every ordered pair of distinct points within eps, on the device."""
    lib.build(points)
    found = []

    def take(batch):
        ids = torch.as_tensor(edd.DeviceArray(batch.query_ids, (batch.nq,), "<i8"), device="cuda")
        ptr = torch.as_tensor(edd.DeviceArray(batch.row_ptr, (batch.nq + 1,), "<i8"), device="cuda")
        cols = torch.as_tensor(edd.DeviceArray(batch.cols, (batch.nnz,), "<i4"), device="cuda")
        found.append(torch.stack([torch.repeat_interleave(ids, ptr.diff(), output_size=batch.nnz), cols.long()]))

    lib.join(eps, on_batch=take)
    i, j = torch.cat(found, dim=1)
    return i[i != j], j[i != j]


class Learner:
    def __init__(self, items=800, groups=40, width=32, eps=3.0, batch=700, seed=0):
        self.lib = edd.Join()
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.eps, self.batch, self.scale = eps, batch, width ** 0.5
        self.group = torch.arange(items, device="cuda") % groups
        self.table = 0.3 * torch.randn((items, width), generator=self.gen, device="cuda")
        self.weight = torch.ones(width, device="cuda")
        self.bias = torch.zeros(width, device="cuda")
        self.grads = [torch.empty_like(p) for p in (self.table, self.weight, self.bias)]
        self.clip = edd.Gradients(self.grads)

    def points(self, items):
        x = self.lib.embed(items, self.table, scale=self.scale, pad=PAD)
        y, mean, rstd = self.lib.layer_norm(x, self.weight, self.bias)
        return x, y, mean, rstd

    def step(self, rate=0.005, max_norm=2500.0):
        """One step on a random batch (padded to its full size); returns the loss."""
        n = self.batch
        items = torch.randint(0, self.table.shape[0], (n,), generator=self.gen, device="cuda")
        items[n - n // 20:] = PAD
        live = torch.nonzero(items != PAD).flatten()
        x, y, mean, rstd = self.points(items)
        dy = torch.zeros_like(y)
        # pairs of one group: each position with the next one of its group
        order = live[torch.argsort(self.group[items[live]], stable=True)]
        a, b = order[:-1], order[1:]
        same = self.group[items[a]] == self.group[items[b]]
        a, b = a[same], b[same]
        d = y[a] - y[b]
        loss = 0.5 * (d * d).sum()
        dy.index_add_(0, a, d)
        dy.index_add_(0, b, -d)
        # pairs of different groups within eps; each is found in both orders
        i, j = joined_pairs(self.lib, y[live], self.eps)
        i, j = live[i], live[j]
        apart = self.group[items[i]] != self.group[items[j]]
        i, j = i[apart], j[apart]
        d = y[i] - y[j]
        r = d.norm(dim=1).clamp_min(1e-6)
        gap = self.eps - r
        loss = loss + 0.25 * (gap * gap).sum()
        dy.index_add_(0, i, d * (-gap / r)[:, None])
        dx, self.grads[1][:], self.grads[2][:] = self.lib.layer_norm_grad(dy, x, mean, rstd, self.weight)
        self.lib.embed_grad(items, dx, self.table.shape[0], scale=self.scale, pad=PAD, out=self.grads[0])
        self.lib.clip_grads(self.clip, max_norm)
        for p, g in zip((self.table, self.weight, self.bias), self.grads):
            p.sub_(g, alpha=rate)
        self.lib.finish()
        return float(loss) / n

    def purity(self):
        """Share of the pairs within eps that are of one group, and the share of a
        group's pairs that are within eps."""
        _, y, _, _ = self.points(torch.arange(self.table.shape[0], device="cuda"))
        i, j = joined_pairs(self.lib, y, self.eps)
        same = int((self.group[i] == self.group[j]).sum())
        size = torch.bincount(self.group)
        return same / max(1, i.numel()), same / int((size * (size - 1)).sum())


    def learn(self, steps, rate=0.005, report=lambda step, loss: None):
        """Steps at a falling rate; returns the losses."""
        losses = []
        for s in range(steps):
            losses.append(self.step(rate * (1 - s / steps)))
            report(s, losses[-1])
        return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    args = ap.parse_args()
    learner = Learner()
    print("before: %.3f of the pairs within eps are of one group, %.3f of a group's pairs are within eps" % learner.purity())

    def report(s, loss):
        if s % 50 == 0 or s == args.steps - 1:
            print("step %4d  loss %.4f" % (s, loss))

    learner.learn(args.steps, report=report)
    print("after:  %.3f of the pairs within eps are of one group, %.3f of a group's pairs are within eps" % learner.purity())


if __name__ == "__main__":
    main()
