"""The feature operators as they are used together: one training step against
the fp64 oracle chained the same way, and the example's training loop."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import group_shared_fixed_amd as hs
from feature_util import host, put, rounded, say, u
from oracle import features as F

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_step_against_the_chained_oracle():
    B, H, L, eps, t = 150, 136, 700, 1e-6, "bf16"
    rng = np.random.default_rng(9)
    x, x64 = rounded(rng.normal(size=(B, H)), t)
    r, r64 = rounded(rng.normal(size=(B, H)), t)
    g, g64 = rounded(1 + 0.1 * rng.normal(size=H), t)
    W, W64 = rounded(2.0 * rng.normal(size=(L, H)) / np.sqrt(H), t)
    count = rng.integers(0, 4, B)
    rp = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    col = np.concatenate([np.sort(rng.choice(L, k, replace=False)) for k in count]).astype(np.int32)
    n = hs.add_norm(put(x), put(g), residual=put(r), eps=eps, p=0.1, seed=3, offset=4)
    f = hs.dropout(n["y"], 0.25, 5, 6)
    o = hs.softmax_step(f, put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col)), 1.0 / B)
    dy = hs.dropout(o["dh"], 0.25, 5, 6)
    b = hs.add_norm_bwd(dy, n["sum"], put(g), n["rstd"], p=0.1, seed=3, offset=4)

    wn = F.oracle_add_norm(x64, g64, r64, eps, 0.1, 3, 4)
    wf = F.oracle_dropout(wn["y"], 0.25, 5, 6)
    wo = F.oracle_softmax(wf, W64, rp, col, 1.0 / B)
    wdy = F.oracle_dropout(wo["dh"], 0.25, 5, 6)
    wb = F.oracle_add_norm_bwd(wdy, wn["sum"], g64, wn["rstd"], None, 0.1, 3, 4)
    # every stored tensor of the chain is rounded once (u relative, so rms below u), the features' roundings reach the
    # logits (of size 2) and their softmax: four stores and a factor 2 for the logits bound the norm of what is off
    for k, got, want in (("dW", o["dW"], wo["dW"]), ("dh", o["dh"], wo["dh"]), ("dres", b["dres"], wb["dres"]),
                         ("dx", b["dx"], wb["dx"]), ("dgamma", b["dgamma"], wb["dgamma"])):
        rel = np.linalg.norm(host(got) - want) / np.linalg.norm(want)
        say(f"    {k}: rel {rel:.2e}")
        assert rel < 8 * u(t), k
    assert abs(float(o["loss"][0]) - wo["loss"]) < 4 * u(t) * abs(wo["loss"])


def test_example_learns_and_serves():
    spec = importlib.util.spec_from_file_location("softmax_head", os.path.join(ROOT, "examples", "softmax_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    got = m.run(steps=40, log=say)
    assert got["last"] < 0.7 * got["first"] and got["agree"] > 0.8
