"""Trains a dense label head under the softmax loss and serves it in 8 bits.

One step is what stands between an encoder's last block and its gradient:

    add_norm      v = residual + dropout(x), features y = norm(v)
    dropout       on the features
    softmax_step  loss over all labels, dW and the features' gradient
    dropout       the same mask on that gradient
    add_norm_bwd  gradients of gamma, of the block's output and of the residual

and serving writes the norm's rows as E4M3 (add_norm with codes) and scores
them against E4M3 label weights (quantize_rows once, score_a8w8 per batch).
The encoder is replaced by synthetic outputs: noise plus the sum of a fixed
direction per positive label, so that there is something to learn.

    python3 examples/softmax_head.py                         # the small head-tail workload's head
    python3 examples/softmax_head.py --labels 89088 --width 768 --batch 128 --lr 0.5   # that size; 60 steps learn little
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import group_shared_fixed_amd as hs  # noqa: E402
from synthetic import zipf_labels  # noqa: E402


def make_batch(rowptr, col, direction, generator, padding=0.1):
    """Encoder output, residual and CSR labels of a batch; a share of the rows is padding without labels."""
    B, dev = rowptr.numel() - 1, direction.device
    count = (rowptr[1:] - rowptr[:-1]).long()
    pad = torch.rand(B, device=dev, generator=generator) < padding
    keep = torch.repeat_interleave(~pad, count)
    count = torch.where(pad, 0, count)
    rp = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), count.cumsum(0)]).int()
    cl = col[keep].contiguous()
    row = torch.repeat_interleave(torch.arange(B, device=dev), count)
    signal = torch.zeros(B, direction.shape[1], device=dev).index_add_(0, row, direction[cl.long()])
    noise = torch.randn(2, B, direction.shape[1], device=dev, generator=generator)
    return (signal + 0.3 * noise[0]).bfloat16(), (0.3 * noise[1]).bfloat16(), rp, cl


def run(labels=73, width=96, batch=37, positives=3, steps=60, lr=2.0, seed=1, log=print):
    """Returns dict(first, last: loss; agree: share of rows whose best label is the same in 8 bits and in bf16)."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    direction = torch.randn(labels, width, device=dev, generator=g) / positives ** 0.5
    W = torch.zeros(labels, width, device=dev)                       # master weights; the kernels take their bf16 copy
    gamma = torch.ones(width, device=dev)
    ws = torch.empty(hs.softmax_workspace_size(batch, width, labels), dtype=torch.uint8, device=dev)
    nws = torch.empty(hs.add_norm_workspace_size(batch, width), dtype=torch.uint8, device=dev)
    p_block, p_head, losses = 0.1, 0.2, []
    for step in range(steps):
        rowptr, col = (torch.from_numpy(a).to(dev) for a in zipf_labels(batch, labels, positives, 1000 * seed + step))
        x, res, rowptr, col = make_batch(rowptr, col, direction, g)
        gb = gamma.bfloat16()
        n = hs.add_norm(x, gb, residual=res, p=p_block, seed=seed, offset=step)
        f = hs.dropout(n["y"], p_head, seed + 1, offset=step)
        o = hs.softmax_step(f, W.bfloat16(), rowptr, col, 1.0 / batch, workspace=ws)
        dy = hs.dropout(o["dh"], p_head, seed + 1, offset=step)
        b = hs.add_norm_bwd(dy, n["sum"], gb, n["rstd"], p=p_block, seed=seed, offset=step, workspace=nws)
        # b["dx"] and b["dres"] go on to the encoder
        W.sub_(o["dW"].float(), alpha=lr)
        gamma.sub_(b["dgamma"], alpha=0.1 * lr)
        losses.append(o["loss"])
        if step % max(1, steps // 6) == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {float(o['loss'][0]):.4f}  |dx| {float(b['dx'].float().norm()):.4f}  "
                f"|dres| {float(b['dres'].float().norm()):.4f}")

    # serving: 8-bit rows straight from the norm, 8-bit weights laid out once
    wq, wscale = hs.quantize_rows(W)
    rowptr, col = (torch.from_numpy(a).to(dev) for a in zipf_labels(batch, labels, positives, 7777 + seed))
    x, res, rowptr, col = make_batch(rowptr, col, direction, g, padding=0.0)
    n = hs.add_norm(x, gamma.bfloat16(), residual=res, want_a8=True)
    scores = hs.score_a8w8(n["q"], n["scale"], wq, wscale)
    plain = n["y"].float() @ W.T
    agree = float((scores.argmax(1) == plain.argmax(1)).float().mean())
    best = scores.argmax(1)
    hit = sum(int(best[b]) in col[rowptr[b]:rowptr[b + 1]].tolist() for b in range(batch)) / batch
    log(f"8-bit scoring: best label as in fp32 for {agree:.0%} of the rows, a true label for {hit:.0%}")
    held = hs.softmax_loss(n["y"], W.bfloat16(), rowptr, col, 1.0 / batch)
    log(f"held-out loss {float(held['loss'][0]):.4f}")
    return {"first": float(losses[0][0]), "last": float(torch.stack(losses[-5:]).mean()), "agree": agree, "hit": hit}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--labels", type=int, default=73)
    ap.add_argument("--width", type=int, default=96)
    ap.add_argument("--batch", type=int, default=37)
    ap.add_argument("--positives", type=int, default=3)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args()
    run(a.labels, a.width, a.batch, a.positives, a.steps, a.lr)
