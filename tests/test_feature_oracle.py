"""Pins of the feature operators' fp64 oracle: published generator vectors,
torch autograd and central differences, hand values."""

import numpy as np
import pytest
import torch

from oracle import features as F


@pytest.mark.parametrize("ctr,key,want", [
    # known-answer vectors of Philox 4x32-10 (Salmon et al., SC 2011)
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
])
def test_philox_known_answers(ctr, key, want):
    got = F.philox4x32([np.array([c], np.uint64) for c in ctr], key)
    assert [int(g[0]) for g in got] == want


def test_dropout_share_and_factor():
    rows, cols, p = 500, 1003, 0.3
    f = F.drop_factor(rows, cols, p, 12345, 77)
    thr = round(p * 65536)
    assert set(np.unique(f)) == {0.0, 65536.0 / (65536 - thr)}
    n = f.size
    # six standard deviations of the binomial share
    assert abs((f == 0).mean() - thr / 65536) < 6 * np.sqrt(p * (1 - p) / n)
    assert (F.drop_factor(rows, cols, p, 12345, 78) != f).any() and (F.drop_factor(rows, cols, p, 12346, 77) != f).any()
    # the mask of a row prefix is the prefix of the mask
    assert (F.drop_factor(7, cols, p, 12345, 77) == f[:7]).all()
    assert (F.drop_factor(3, 9, 0.0, 1, 2) == 1).all() and (F.drop_factor(3, 9, 1.0, 1, 2) == 0).all()


def test_dropped_nan_leaves_the_residual():
    x = np.full((4, 40), np.nan)
    f = F.drop_factor(4, 40, 0.5, 3, 4)
    y = F.oracle_dropout(x, 0.5, 3, 4, np.ones((4, 40)))
    assert (y[f == 0] == 1).all() and np.isnan(y[f > 0]).all()


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_add_norm_gradient(p):
    rng = np.random.default_rng(5)
    rows, cols, eps = 4, 21, 1e-3
    x, r, gamma = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols)), 1 + 0.2 * rng.normal(size=cols)
    dy, dsum = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))
    f = F.drop_factor(rows, cols, p, 9, 10)
    tx, tr, tg = (torch.tensor(a, requires_grad=True) for a in (x, r, gamma))
    v = tr + tx * torch.tensor(f)
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + eps) * tg
    ((y * torch.tensor(dy)).sum() + (v * torch.tensor(dsum)).sum()).backward()
    fwd = F.oracle_add_norm(x, gamma, r, eps, p, 9, 10)
    got = F.oracle_add_norm_bwd(dy, fwd["sum"], gamma, fwd["rstd"], dsum, p, 9, 10)
    assert np.allclose(fwd["y"], y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for k, t in (("dres", tr), ("dx", tx), ("dgamma", tg)):
        assert np.allclose(got[k], t.grad.numpy(), rtol=1e-10, atol=1e-12), k

    def objective(xx, rr, gg):
        o = F.oracle_add_norm(xx, gg, rr, eps, p, 9, 10)
        return (o["y"] * dy).sum() + (o["sum"] * dsum).sum()
    step = 1e-5
    for k, arg, at in (("dx", 0, (1, 3)), ("dres", 1, (2, 20)), ("dgamma", 2, (7,))):
        a = [x.copy(), r.copy(), gamma.copy()]
        b = [x.copy(), r.copy(), gamma.copy()]
        a[arg][at] += step
        b[arg][at] -= step
        diff = (objective(*a) - objective(*b)) / (2 * step)
        assert abs(diff - got[k][at]) < 1e-7 * max(1, abs(diff)), k


def test_softmax_gradient():
    rng = np.random.default_rng(6)
    B, H, L, scale = 5, 7, 11, 0.3
    h, W = rng.normal(size=(B, H)), rng.normal(size=(L, H))
    rowptr, col = np.array([0, 1, 1, 4, 6, 17]), np.concatenate([[3], [0, 5, 10], [1, 2], np.arange(11)])
    got = F.oracle_softmax(h, W, rowptr, col, scale)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(W, requires_grad=True)
    target = np.zeros((B, L))
    for b in range(B):
        y = col[rowptr[b]:rowptr[b + 1]]
        target[b, y] = 1.0 / max(1, y.size)
    row = -(torch.log_softmax(th @ tw.T, 1) * torch.tensor(target)).sum(1)
    (scale * row.sum()).backward()
    assert np.allclose(got["row_loss"], row.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert got["row_loss"][1] == 0 and (got["dh"][1] == 0).all()
    assert np.allclose(got["dh"], th.grad.numpy(), rtol=1e-10, atol=1e-13)
    assert np.allclose(got["dW"], tw.grad.numpy(), rtol=1e-10, atol=1e-13)
    step = 1e-5
    for name, at in (("dh", (2, 4)), ("dW", (5, 1)), ("dW", (8, 6))):
        side = []
        for sgn in (1, -1):
            a, b = h.copy(), W.copy()
            (a if name == "dh" else b)[at] += sgn * step
            side.append(F.oracle_softmax(a, b, rowptr, col, scale)["loss"])
        assert abs((side[0] - side[1]) / (2 * step) - got[name][at]) < 1e-8, name


def test_softmax_uniform_and_full_rows():
    # W = 0: lse = log L; a row whose labels are all labels has D = 0
    o = F.oracle_softmax(np.ones((2, 3)), np.zeros((8, 3)), np.array([0, 1, 9]), np.array([2] + list(range(8))), 1.0)
    assert np.allclose(o["lse"], np.log(8)) and np.allclose(o["row_loss"], np.log(8))
    assert np.allclose(o["D"][1], 0) and np.allclose(o["D"][0], 1 / 8 - (np.arange(8) == 2))
