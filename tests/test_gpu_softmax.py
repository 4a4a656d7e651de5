"""GPU parity of the softmax loss over a dense label matrix (softmax_step,
softmax_loss) against the fp64 oracle: ragged sizes, several pieces of the
label space, padding rows that hold NaN, every label positive, large logits,
strides, streams and graphs.

Bounds, per element: the products' fp32 sums are off by dz = (H + 8) U sum |h w|,
lse by max dz plus 64 U of its size and of the logits' range, so D by
|p| (2 dz + ...) + u(t) |D| (its rounding for the gradient products), and the
gradients by those summed against |h| or |W|, plus their own fp32 sums and store."""

import numpy as np
import pytest
import torch

import group_shared_fixed_amd as hs
from feature_util import TINY, U, host, put, rounded, say, strided, u, within
from gpu_util import dev
from oracle import features as F

pytestmark = pytest.mark.gpu


def make(B, H, L, m, empty, t, seed, gain=2.5):
    rng = np.random.default_rng(seed)
    h, _ = rounded(rng.normal(size=(B, H)), t)
    W, W64 = rounded(rng.normal(size=(L, H)) * (gain / np.sqrt(H)), t)
    rows = []
    for b in range(B):
        k = 0 if (b and rng.random() < empty) else int(rng.integers(1, min(m, L) + 1))
        rows.append(np.sort(rng.choice(L, size=k, replace=False)))
        if k == 0:
            h[b] = float("nan") if b % 2 else float("inf")
    rowptr = np.concatenate([[0], np.cumsum([r.size for r in rows])]).astype(np.int32)
    col = np.concatenate(rows).astype(np.int32)
    return h, W, h.double().numpy(), W64, rowptr, col


def bounds(h64, W64, want, rowptr, scale, t):
    B, H = h64.shape
    live = np.diff(rowptr) > 0
    h = np.where(live[:, None], np.abs(np.nan_to_num(h64, posinf=0)), 0)
    W = np.abs(W64)
    dz = (H + 8) * U * (h @ W.T)
    Z = np.where(live[:, None], np.nan_to_num(h64, posinf=0) @ W64.T, 0)
    span = np.abs(Z).max(1) + np.abs(want["lse"])
    dl = np.where(live, dz.max(1) + 64 * U * (1 + span), 0)
    D = want["D"]
    p = np.where(live[:, None], np.exp(np.minimum(Z - want["lse"][:, None], 0)), 0)
    # values this far below the type's normal range are held to half a subnormal step (fp16 holds D times 4096)
    eD = p * (dz + dl[:, None] + 8 * U * (1 + span[:, None])) * 1.01 + 4 * U * np.abs(D)
    # probabilities below fp32's (and bf16's) normal range become 0
    low = 2.0 ** -25 / 4096 if t == "fp16" else 2.0 ** -126
    eD = eD + u(t) * (np.abs(D) + eD) + low * live[:, None]
    s = abs(scale)
    eW, eh = s * (eD.T @ h), s * (eD @ W)
    eW = eW + (B + 8) * U * s * (np.abs(D).T @ h)
    eh = eh + (W.shape[0] + 8) * U * s * (np.abs(D) @ W)
    return {"lse": dl, "row_loss": 2 * dl, "loss": s * (2 * dl).sum() + 4 * U * abs(want["loss"]),
            "dW": eW + u(t) * (np.abs(want["dW"]) + eW) + TINY[t], "dh": eh + u(t) * (np.abs(want["dh"]) + eh) + TINY[t]}


def check(out, want, b, grad=True):
    for k in ("lse", "row_loss"):
        within(out[k], want[k], b[k], k)
    within(out["loss"], np.array([want["loss"]]), b["loss"], "loss")
    if grad:
        within(out["dh"], want["dh"], b["dh"], "dh")
        within(out["dW"], want["dW"], b["dW"], "dW")


CASES = [  # B, H, L, m, empty
    (1, 8, 1, 1, 0), (1, 64, 300, 3, 0), (2, 768, 1000, 1, 0), (5, 200, 257, 257, 0.3), (37, 96, 73, 9, 0.1),
    (16, 64, 4096, 5, 0), (33, 72, 515, 4, 0.5), (64, 256, 2000, 8, 0.2), (128, 768, 2048, 32, 0),
    (130, 264, 1001, 4, 0.4), (257, 1000, 700, 1, 0.6), (300, 96, 513, 40, 0.95), (515, 520, 1300, 2, 0.3),
    # one row tile over a long label space: ranges of the streaming kernels that end inside tiles, pieces and the last label
    (1, 1032, 4097, 1, 0), (20, 264, 5003, 4, 0.2), (128, 768, 4500, 30, 0), (97, 1000, 20011, 2, 0.4), (128, 64, 70001, 1, 0.1),
    # many rows, few labels: dW over ranges of rows, of which the last may be empty
    (1100, 64, 70, 5, 0.2), (2200, 520, 600, 3, 0.5), (4100, 72, 300, 2, 0.9)]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_h%d_l%d" % c[:3] for c in CASES])
def test_softmax(case, t):
    B, H, L, m, empty = case
    h, W, h64, W64, rp, col = make(*case, t, B + L)
    scale = (512.0 if t == "fp16" else 1.0) / B
    say(f"  softmax B={B} H={H} L={L} {t}")
    want = F.oracle_softmax(np.nan_to_num(h64, posinf=0), W64, rp, col, scale)
    b = bounds(h64, W64, want, rp, scale, t)
    args = put(h), put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col))
    out = hs.softmax_step(*args, scale)
    check(out, want, b)
    only = hs.softmax_loss(*args, scale)
    for k in only:
        assert torch.equal(only[k], out[k]), f"softmax_loss: {k} differs from the step's"
    # the least workspace: 256 labels at a time
    least = torch.empty(hs.softmax_workspace_size(B, H, L, minimum=True), dtype=torch.uint8, device=dev())
    pieces = hs.softmax_step(*args, scale, workspace=least)
    check(pieces, want, b)
    # dirty workspaces and outputs change nothing
    least.fill_(0xFF)
    for k in pieces:
        pieces[k].fill_(float("nan"))
    again = {k: v.clone() for k, v in hs.softmax_step(*args, scale, out=pieces, workspace=least).items()}
    ref = hs.softmax_step(*args, scale, workspace=least)
    assert all(torch.equal(again[k], ref[k]) for k in ref), "not repeatable"


# large enough that the exponentials of all labels are kept: labels spread over the whole space, over few blocks of 256 (lists
# of a block that hold each label's remainder too, hold it alone, overflow), many a row, rows beyond the kept range
KEPT = {"spread": (260, 264, 33_001, 4, None, 2.5), "many": (515, 296, 22_100, 90, None, 2.5),
        "heavy": (512, 264, 33_001, 300, None, 2.5),
        "crowded": (1030, 264, 13_100, 5, 2500, 2.5), "overflowing": (1030, 264, 13_100, 5, 700, 2.5),
        "large": (300, 264, 33_001, 3, None, 40.0), "low": (300, 264, 33_001, 3, None, 2.5)}


@pytest.mark.parametrize("name", KEPT)
def test_kept_exponentials(name):
    """h is rounded once more on the way to dW here (times the row's factor): half a step of every product's share."""
    B, H, L, m, over, gain = KEPT[name]
    h, W, h64, W64, rp, col = make(B, H, over or L, m, 0.15, "bf16", B + L, gain)
    if over:
        W, W64 = rounded(np.random.default_rng(9).normal(size=(L, H)) * (gain / np.sqrt(H)), "bf16")
    if name == "low":           # a third of the rows: every logit near -50 or near +50
        W[:, 0], W64[:, 0] = 1.0, 1.0
        for b in range(0, B, 3):
            if rp[b + 1] > rp[b]:
                h[b, 0] = h64[b, 0] = -50.0 if b % 2 else 50.0
    scale = 1.0 / B
    say(f"  kept exponentials {name}")
    want = F.oracle_softmax(np.nan_to_num(h64, posinf=0), W64, rp, col, scale)
    b = bounds(h64, W64, want, rp, scale, "bf16")
    live = np.diff(rp) > 0
    more = scale * u("bf16") * (np.abs(want["D"]).T @ np.where(live[:, None], np.abs(np.nan_to_num(h64, posinf=0)), 0))
    args = put(h), put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col))
    ws = torch.full((hs.softmax_workspace_size(B, H, L),), 0xFF, dtype=torch.uint8, device=dev())
    out = hs.softmax_step(*args, scale, workspace=ws)
    check(out, want, b | {"dW": b["dW"] + 1.02 * more})
    again = hs.softmax_step(*args, scale)
    assert all(torch.equal(again[k], out[k]) for k in out), "not repeatable"
    some = hs.softmax_workspace_size(B, H, L, minimum=True) + (4 << 20)         # pieces: the first is kept, the others formed again
    pieces = hs.softmax_step(*args, scale, workspace=ws[:some])
    check(pieces, want, b | {"dW": b["dW"] + 1.02 * more})


def test_all_rows_padding():
    B, H, L = 70, 96, 300
    h = torch.full((B, H), float("nan"), dtype=torch.bfloat16, device=dev())
    W = torch.randn(L, H, device=dev()).to(torch.bfloat16)
    rp = torch.zeros(B + 1, dtype=torch.int32, device=dev())
    out = hs.softmax_step(h, W, rp, torch.empty(0, dtype=torch.int32, device=dev()), 1.0)
    assert all((v == 0).all() for v in out.values())


@pytest.mark.parametrize("gain", [40.0, 400.0])
def test_large_logits(gain):
    B, H, L = 40, 256, 600
    h, W, h64, W64, rp, col = make(B, H, L, 2, 0.2, "bf16", 77, gain)
    want = F.oracle_softmax(np.nan_to_num(h64, posinf=0), W64, rp, col, 1.0)
    out = hs.softmax_step(put(h), put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col)), 1.0)
    check(out, want, bounds(h64, W64, want, rp, 1.0, "bf16"))


def test_nan_logit_shows():
    B, H, L = 9, 64, 300
    h, W, h64, W64, rp, col = make(B, H, L, 2, 0, "bf16", 3)
    h[4, 7] = float("nan")
    out = hs.softmax_step(put(h), put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col)), 1.0)
    lse = host(out["lse"])
    assert np.isnan(lse[4]) and np.isfinite(np.delete(lse, 4)).all()
    dh = host(out["dh"])
    assert np.isnan(dh[4]).all() and np.isfinite(np.delete(dh, 4, 0)).all()


@pytest.mark.parametrize("B,H,L", [(75, 136, 430), (100, 520, 6000), (260, 264, 16_500)])
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_strides_and_streams(B, H, L, t):
    h, W, h64, W64, rp, col = make(B, H, L, 3, 0.3, t, 5)
    lab = put(torch.from_numpy(rp)), put(torch.from_numpy(col))
    ref = hs.softmax_step(put(h), put(W), *lab, 0.1)
    out = hs.softmax_step(strided(h, 24, 8), strided(W, 8), *lab, 0.1)
    assert all(torch.equal(out[k], ref[k]) for k in ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hd, Wd = put(h), put(W)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = hs.softmax_step(hd, Wd, *lab, 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], ref[k]) for k in ref)


@pytest.mark.parametrize("B,H,L", [(96, 128, 900), (70, 128, 5000), (260, 264, 16_500), (1100, 64, 70)])
def test_graph_replays(B, H, L):
    h, W, h64, W64, rp, col = make(B, H, L, 3, 0.3, "bf16", 6)
    h2 = make(B, H, L, 3, 0.3, "bf16", 6)[0]
    hd, Wd, lab = put(h), put(W), (put(torch.from_numpy(rp)), put(torch.from_numpy(col)))
    ws = torch.empty(hs.softmax_workspace_size(B, H, L), dtype=torch.uint8, device=dev())
    out = {k: v.clone() for k, v in hs.softmax_step(hd, Wd, *lab, 0.1, workspace=ws).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hs.softmax_step(hd, Wd, *lab, 0.1, out=out, workspace=ws)
    for i in range(4):
        hd.copy_(put(h2 if i % 2 else h) * (1 + i))
        g.replay()
        torch.cuda.synchronize()
        ref = hs.softmax_step(hd, Wd, *lab, 0.1)
        assert all(torch.equal(out[k], ref[k]) for k in ref), f"replay {i}"


def test_autograd_graph_of_the_same_leaves_alive():
    """Called while an eager autograd graph of its inputs is alive, and matching that graph's gradients."""
    B, H, L = 50, 64, 200
    h, W, h64, W64, rp, col = make(B, H, L, 1, 0, "bf16", 8)
    hf, Wf = put(h).float().requires_grad_(), put(W).float().requires_grad_()
    loss = torch.nn.functional.cross_entropy(hf @ Wf.T, put(torch.from_numpy(col)).long(), reduction="sum") * 0.1
    out = hs.softmax_step(put(h), put(W), put(torch.from_numpy(rp)), put(torch.from_numpy(col)), 0.1)
    loss.backward()
    assert abs(float(out["loss"][0]) - float(loss.detach())) < 1e-5 * abs(float(loss.detach()))
    for got, ref in ((out["dh"], hf.grad), (out["dW"], Wf.grad)):
        assert float((got.float() - ref).norm() / ref.norm()) < 2 * u("bf16")


@pytest.mark.parametrize("B,whole", [(3, False), (200, False), (200, True)])
def test_past_32_bit_offsets(B, whole):
    """L x H past 2^31 elements: the last labels, one of them a row's own."""
    H, L, scale = 1024, 2_200_000, 4.0
    g = torch.Generator(device=dev()).manual_seed(4)
    W = torch.empty(L, H, dtype=torch.bfloat16, device=dev())
    for at in range(0, L, 1 << 18):
        n = min(1 << 18, L - at)
        W[at:at + n] = (torch.randn(n, H, device=dev(), generator=g) * 0.06).bfloat16()
    h = torch.randn(B, H, device=dev(), generator=g).bfloat16()
    col = torch.arange(B, device=dev(), dtype=torch.int32) * ((L - 1) // B)
    col[-1] = L - 1
    ws = torch.empty(hs.softmax_workspace_size(B, H, L, whole=whole), dtype=torch.uint8, device=dev())
    out = hs.softmax_step(h, W, torch.arange(B + 1, device=dev(), dtype=torch.int32), col, scale, workspace=ws)
    hf, lse = h.float(), torch.full((B,), -float("inf"), dtype=torch.float64, device=dev())
    for at in range(0, L, 1 << 18):
        lse = torch.logaddexp(lse, torch.logsumexp((hf @ W[at:at + (1 << 18)].float().T).double(), 1))
    dz = (H + 8) * U * float((hf.abs() @ W[-500:].float().abs().T).max()) * 1.5
    within(out["lse"], host(lse), dz + 64 * U * 40, "lse")
    tail = W[-500:].float().double()
    D = torch.exp(hf.double() @ tail.T - lse[:, None])
    D[-1, -1] -= 1
    want = scale * host(D.T @ hf.double())
    bound = scale * host(((dz + 64 * U * 40) * 2 + u("bf16")) * D.abs().T @ hf.double().abs()) * 1.01
    within(out["dW"][-500:], want, bound + u("bf16") * (np.abs(want) + bound), "dW of the last labels")
    assert torch.isfinite(out["dh"].float()).all()
