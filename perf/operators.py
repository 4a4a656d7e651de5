"""Cases, plain forms and exact values of the operators around the output layer.

Four operators make up the path from an encoder block's output to a trained or
scored label space:

* add_norm     residual + dropout(x), root-mean-square norm, bf16 / fp16 / fp32
               or E4M3 rows with scales; and its backward pass
* dropout      counter-based (Philox 4x32-10), the mask is never stored
* softmax      cross entropy over the dense label matrix with its gradient;
               rows without labels are padding
* score        logits from E4M3 features and E4M3 label weights

`run` computes them in elementary torch operations, or, where `own` is true,
with this repository's kernels.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the small head-tail workload's dense head: a test-sized training step, launch bound
        dict(name="softmax_ht_small", op="softmax", grad=True, B=37, L=73, H=96, m=9, empty=0.1, dtype="bf16"),
        # the dense head of the 3M-label head-tail split at its batch of 128, ~32 head labels a sample
        dict(name="softmax_head_89k", op="softmax", grad=True, B=128, L=89_088, H=768, m=32, empty=0.0, dtype="bf16"),
        # a batch of token positions under a 128K vocabulary, a quarter of them padding: the largest
        dict(name="softmax_tokens_131k", op="softmax", grad=True, B=4096, L=131_072, H=1024, m=1, empty=0.25,
             dtype="bf16"),
        # ragged everything in half precision with a loss scale, 40 % padding
        dict(name="softmax_odd_fp16", op="softmax", grad=True, B=1021, L=32_003, H=640, m=1, empty=0.4, dtype="fp16"),
        # one request's feature row to 8 bits (serving, latency bound)
        dict(name="norm_a8_one_row", op="add_norm", rows=1, cols=768, q8=True, p=0.0, dtype="bf16"),
        # a prefill's rows to 8 bits
        dict(name="norm_a8_8192x4096", op="add_norm", rows=8192, cols=4096, q8=True, p=0.0, dtype="bf16"),
        # training forward of an encoder block's end, dropout in the same pass, odd row count
        dict(name="norm_train_16411x768", op="add_norm", rows=16_411, cols=768, q8=False, p=0.1, dtype="bf16"),
        # its backward pass
        dict(name="norm_bwd_16411x1024", op="add_norm_bwd", rows=16_411, cols=1024, p=0.1, dtype="bf16"),
        # dropout on one batch of features ahead of the output layer
        dict(name="dropout_features", op="dropout", rows=64, cols=768, p=0.5, residual=False, dtype="fp32"),
        # dropout with a residual over a long batch of token rows
        dict(name="dropout_32768x4096", op="dropout", rows=32_768, cols=4096, p=0.1, residual=True, dtype="bf16"),
        # one request scored against every head label: one pass over the 8-bit weights
        dict(name="score_1x89k", op="score", B=1, L=89_088, H=768),
        # offline scoring of a large batch
        dict(name="score_2048x89k", op="score", B=2048, L=89_088, H=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["softmax", "softmax", "add_norm", "add_norm_bwd", "dropout", "score"])
    if op == "softmax":
        while True:
            B, L = _log(rng, 1, 4096), _log(rng, 65, 131_072)
            H = 8 * _log(rng, 8, 128)
            if B * L * H <= 4096 * 131_072 * 1024:
                return dict(op=op, grad=rng.random() < 0.75, B=B, L=L, H=H, m=rng.choice([1, 1, 5, 36]),
                            empty=round(rng.choice([0.0, rng.uniform(0.0, 0.6)]), 3), dtype=rng.choice(["bf16", "fp16"]))
    if op == "score":
        while True:
            B, L = _log(rng, 1, 2048), _log(rng, 65, 131_072)
            H = 16 * _log(rng, 4, 64)
            if B * L <= 2048 * 89_088:
                return dict(op=op, B=B, L=L, H=H)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while True:
        rows, cols = _log(rng, 1, 32_768), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            cols = (cols + 7) // 8 * 8
        if rows * cols <= 8192 * 4096:
            break
    if op == "add_norm":
        q8 = rng.random() < 0.5
        return dict(op=op, rows=rows, cols=cols, q8=q8, p=0.0 if q8 else rng.choice([0.0, 0.1, 0.25]), dtype=dtype)
    if op == "add_norm_bwd":
        return dict(op=op, rows=rows, cols=cols, p=rng.choice([0.0, 0.1, 0.25]), dtype=dtype)
    return dict(op=op, rows=rows, cols=cols, p=rng.choice([0.1, 0.25, 0.5]), residual=rng.random() < 0.5, dtype=dtype)


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _labels(g, c):
    """CSR label lists: `m` draws per row with a Zipf-like law, sorted, repeats merged; a share of the rows empty."""
    B, L = c["B"], c["L"]
    u = torch.rand(B, c["m"], generator=g, device="cuda", dtype=torch.float64)
    lab = torch.exp(u * math.log(L + 1)).long() - 1
    lab = (lab.clamp(0, L - 1) * 7919 + 13) % L if L % 7919 else lab.clamp(0, L - 1)
    filled = torch.rand(B, generator=g, device="cuda") >= c["empty"]
    filled[0] = True
    key = torch.unique((torch.arange(B, device="cuda")[:, None] * L + lab)[filled])
    rowptr = torch.searchsorted(key, torch.arange(B + 1, device="cuda") * L)
    return rowptr.int(), (key % L).int(), filled


def _to_rows_e4m3(x):
    s = x.abs().amax(1) / 448.0
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["op"] == "softmax":
        t = TYPES[c["dtype"]]
        h = _normal(g, c["B"], c["H"])
        s["rowptr"], s["col"], filled = _labels(g, c)
        # padding rows hold what a padded batch holds: anything
        h[~filled] = torch.where(_normal(g, int((~filled).sum()), 1) > 0, 3e4, float("nan"))
        s["h"] = h.to(t)
        s["W"] = (_normal(g, c["L"], c["H"]) * (2.5 / math.sqrt(c["H"]))).to(t)
        # mean over the batch; half precision carries a loss scale of 2^12
        s["scale"] = (4096.0 if t == torch.float16 else 1.0) / c["B"]
    elif c["op"] == "score":
        s["hq"], s["hs"] = _to_rows_e4m3(_normal(g, c["B"], c["H"]))
        s["Wq"], s["ws"] = _to_rows_e4m3(_normal(g, c["L"], c["H"]) / math.sqrt(c["H"]))
    else:
        t = TYPES[c["dtype"]]
        n = c["rows"], c["cols"]
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ seed, (seed * 5 + 1) << 30
        s["x"] = _normal(g, *n).to(t)
        if c["op"] == "add_norm":
            s["res"] = (2 * _normal(g, *n)).to(t)
            s["gamma"] = (1 + 0.2 * _normal(g, n[1])).to(t)
        elif c["op"] == "add_norm_bwd":
            s["sum"] = (2 * _normal(g, *n)).to(t)
            s["rstd"] = (s["sum"].double().square().mean(1) + EPS).rsqrt().float()
            s["gamma"] = (1 + 0.2 * _normal(g, n[1])).to(t)
            s["dsum"] = _normal(g, *n).to(t)
        elif c["residual"]:
            s["res"] = _normal(g, *n).to(t)
    return s


# ------------------------------------------------------------ the plain forms

_MASK = 0xFFFFFFFF


def _philox(block, seed, offset):
    """Four 32-bit words (as int64 tensors) of Philox 4x32-10 at counters `block`."""
    x0, x1 = block & _MASK, block >> 32
    x2, x3 = torch.full_like(block, offset & _MASK), torch.full_like(block, offset >> 32)
    k0, k1 = seed & _MASK, seed >> 32
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57          # 64-bit products, wrapped
        x0, x1, x2, x3 = ((b >> 32) & _MASK) ^ x1 ^ k0, b & _MASK, ((a >> 32) & _MASK) ^ x3 ^ k1, a & _MASK
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    return x0, x1, x2, x3


def _kept(c, s):
    """The keep mask and the factor of the kept values."""
    rows, cols, thr = c["rows"], c["cols"], round(c["p"] * 65536)
    per = -(-cols // 8)
    words = _philox(torch.arange(rows * per, device="cuda"), s["seed"], s["offset"])
    halves = torch.stack([x for w in words for x in (w & 0xFFFF, w >> 16)], 1)
    return (halves >= thr).view(rows, 8 * per)[:, :cols], 65536.0 / (65536 - thr)


def _dropped(x, c, s):
    if c["p"] == 0:
        return x
    keep, f = _kept(c, s)
    return torch.where(keep, x * f, torch.zeros_like(x))


def _plain_softmax(c, s):
    t, B = TYPES[c["dtype"]], c["B"]
    count = (s["rowptr"][1:] - s["rowptr"][:-1]).long()
    valid = count > 0
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), count)
    col = s["col"].long()
    h, W = torch.where(valid[:, None], s["h"].float(), 0.0), s["W"].float()
    Z = h @ W.T
    top = Z.amax(1)
    lse = top + torch.log(torch.exp(Z - top[:, None]).sum(1))
    share = 1.0 / count[row].float()
    hit = torch.zeros(B, device="cuda").index_add_(0, row, Z[row, col] * share)
    row_loss = torch.where(valid, lse - hit, 0.0)
    out = {"row_loss": row_loss, "lse": torch.where(valid, lse, 0.0), "loss": (s["scale"] * row_loss.double().sum()).float().reshape(1)}
    if c["grad"]:
        D = torch.exp(Z - lse[:, None])
        D[row, col] -= share
        D = torch.where(valid[:, None], D * s["scale"], 0.0)
        out["dW"], out["dh"] = (D.T @ h).to(t), (D @ W).to(t)
    return out


def _plain_add_norm(c, s):
    t = TYPES[c["dtype"]]
    v = s["res"].float() + _dropped(s["x"].float(), c, s)
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None] * s["gamma"].float()
    out = {"sum": v.to(t)}
    if not c["q8"]:
        return out | {"y": y.to(t), "rstd": rstd}
    scale = y.abs().amax(1) / 448.0
    return out | {"q": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}


def _plain_add_norm_bwd(c, s):
    t = TYPES[c["dtype"]]
    dy = s["x"].float()
    xh = s["sum"].float() * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    ds = (g - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None] + s["dsum"].float()
    out = {"dres": ds.to(t), "dgamma": (dy * xh).sum(0)}
    return out | {"dx": _dropped(ds, c, s).to(t)} if c["p"] else out


def _plain(c, s):
    if c["op"] == "softmax":
        return _plain_softmax(c, s)
    if c["op"] == "add_norm":
        return _plain_add_norm(c, s)
    if c["op"] == "add_norm_bwd":
        return _plain_add_norm_bwd(c, s)
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), c, s)
        return (y + s["res"].float() if c["residual"] else y).to(TYPES[c["dtype"]])
    return (s["hq"].float() @ s["Wq"].float().T) * s["hs"][:, None] * s["ws"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(c, s)
    import group_shared_fixed_amd as hs
    op = c["op"]
    if op == "softmax":
        if "work" not in s:
            size = hs.softmax_workspace_size(c["B"], c["H"], c["L"], grad=c["grad"])
            s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        call = hs.softmax_step if c["grad"] else hs.softmax_loss
        s["out"] = call(s["h"], s["W"], s["rowptr"], s["col"], s["scale"], out=s.get("out"), workspace=s["work"])
        return s["out"]
    if op == "add_norm":
        s["out"] = hs.add_norm(s["x"], s["gamma"], residual=s["res"], eps=EPS, p=c["p"], seed=s["seed"],
                               offset=s["offset"], want_y=not c["q8"], want_a8=c["q8"], out=s.get("out"))
        return s["out"]
    if op == "add_norm_bwd":
        if "work" not in s:
            s["work"] = torch.empty(hs.add_norm_workspace_size(c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
        s["out"] = hs.add_norm_bwd(s["x"], s["sum"], s["gamma"], s["rstd"], dsum=s["dsum"], p=c["p"], seed=s["seed"],
                                   offset=s["offset"], out=s.get("out"), workspace=s["work"])
        return s["out"]
    if op == "dropout":
        s["out"] = hs.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s.get("res"), out=s.get("out"))
        return s["out"]
    s["out"] = hs.score_a8w8(s["hq"], s["hs"], s["Wq"], s["ws"], Z=s.get("out"))
    return s["out"]


def work(case):
    c = case
    if c["op"] == "softmax":
        B, L, H = c["B"], c["L"], c["H"]
        V = max(1.0, B * (1 - c["empty"]))
        nbytes = 2 * (V * H + L * H) + 4 * (B + 1 + V * c["m"]) + 8 * B
        if c["grad"]:
            nbytes += 2 * (B * H + L * H)
        return {"bytes": nbytes, "flops": (6 if c["grad"] else 2) * V * L * H}
    if c["op"] == "score":
        B, L, H = c["B"], c["L"], c["H"]
        return {"bytes": (B + L) * (H + 4) + 4 * B * L, "flops": 2 * B * L * H}
    n, e = c["rows"] * c["cols"], 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "dropout":
        return {"bytes": n * e * (3 if c["residual"] else 2), "flops": 2 * n}
    if c["op"] == "add_norm":
        return {"bytes": n * (3 * e + (1 if c["q8"] else e)) + c["cols"] * e + 4 * c["rows"], "flops": 5 * n}
    return {"bytes": n * e * (5 if c["p"] else 4) + c["cols"] * (e + 4) + 4 * c["rows"], "flops": 9 * n}


# ------------------------------------------------- the definitions in 64 bits

def _limbs(a, m):
    """High and low 32 bits of a * m for 32-bit a (int64 tensor) and m, by 16-bit limbs."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + ((a0 * m0) >> 16)
    mid2 = a0 * m1 + (mid & 0xFFFF)
    return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((a0 * m0) & 0xFFFF)


def _exact_factor(c, s):
    """0 where an element is dropped, 1 / (share kept) where it stays."""
    rows, cols = c["rows"], c["cols"]
    if not c["p"]:
        return 1.0
    thr, per = round(c["p"] * 65536), (cols + 7) // 8
    n = torch.arange(rows * per, device="cuda")
    ctr = [n % 2**32, n // 2**32, torch.zeros_like(n) + s["offset"] % 2**32, torch.zeros_like(n) + s["offset"] // 2**32]
    for i in range(10):
        hi0, lo0 = _limbs(ctr[0], 0xD2511F53)
        hi1, lo1 = _limbs(ctr[2], 0xCD9E8D57)
        key = [(s["seed"] % 2**32 + i * 0x9E3779B9) % 2**32, (s["seed"] // 2**32 + i * 0xBB67AE85) % 2**32]
        ctr = [hi1 ^ ctr[1] ^ key[0], lo1, hi0 ^ ctr[3] ^ key[1], lo0]
    f = torch.empty(rows * per, 8, dtype=torch.float64, device="cuda")
    for e in range(8):
        half = ctr[e // 2] // 2 ** (16 * (e % 2)) % 2**16
        f[:, e] = (half >= thr).double() / (1 - thr / 65536)
    return f.view(rows, 8 * per)[:, :cols]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "score":
        return torch.einsum("bj,lj->bl", s["hq"].double(), s["Wq"].double()) * torch.outer(s["hs"].double(), s["ws"].double())
    if c["op"] == "softmax":
        B, L = c["B"], c["L"]
        count = s["rowptr"].long().diff()
        live = count.nonzero()[:, 0]
        h, W = s["h"].double()[live], s["W"].double()
        Z = torch.mm(h, W.t())
        lse = torch.logsumexp(Z, 1)
        at = torch.repeat_interleave(torch.arange(len(live), device="cuda"), count[live]) * L + s["col"].long()
        share = torch.repeat_interleave(1.0 / count[live].double(), count[live])
        hit = torch.zeros(len(live), dtype=torch.float64, device="cuda")
        hit.scatter_add_(0, at // L, Z.view(-1)[at] * share)
        full = lambda v: torch.zeros(B, *v.shape[1:], dtype=torch.float64, device="cuda").index_copy_(0, live, v)  # noqa: E731
        out = {"row_loss": full(lse - hit), "lse": full(lse), "loss": s["scale"] * (lse - hit).sum().reshape(1)}
        if c["grad"]:
            Z.sub_(lse[:, None]).exp_()
            Z.view(-1).scatter_add_(0, at, -share)
            Z *= s["scale"]
            out["dW"], out["dh"] = torch.mm(Z.t(), h), full(torch.mm(Z, W))
        return out
    x = s["x"].double()
    if c["op"] == "dropout":
        y = x * _exact_factor(c, s)
        return y + s["res"].double() if c["residual"] else y
    w = s["gamma"].double()
    if c["op"] == "add_norm":
        v = s["res"].double() + x * _exact_factor(c, s)
        n = v / torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / c["cols"] + EPS)
        if not c["q8"]:
            return {"sum": v, "y": n * w, "rstd": (v.square().mean(1) + EPS).rsqrt()}
        big = (n * w).abs().amax(1)
        return {"sum": v, "q": (n * w * (448.0 / big)[:, None]).to(torch.float8_e4m3fn), "scale": big / 448.0}
    r = s["rstd"].double()[:, None]
    v = s["sum"].double()
    ds = x * w * r - v * r**3 * torch.einsum("ij,ij,j->i", x, v, w)[:, None] / c["cols"] + s["dsum"].double()
    out = {"dres": ds, "dgamma": torch.einsum("ij,ij,i->j", x, v, s["rstd"].double())}
    return out | {"dx": ds * _exact_factor(c, s)} if c["p"] else out
