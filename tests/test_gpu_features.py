"""GPU parity of dropout, add_norm (forward, backward, 8-bit rows) and 8-bit
scoring against the fp64 oracle, at sizes, types, strides and values where
they can go wrong.  Bounds are derived per element from the roundings:
u(t) |value| for the store and multiples of 2^-24 for the fp32 arithmetic."""

import numpy as np
import pytest
import torch

import group_shared_fixed_amd as hs
from feature_util import TINY, U, host, put, rounded, say, strided, u, within
from gpu_util import dev
from oracle import features as F

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x0123456789ABCDEF, (1 << 63) + 12345

# odd widths, one element, one row, widths around the eight-element blocks and
# around each thread-count rule (512, 1024, 2048, 4096, 8192 columns)
SHAPES = [(1, 1), (1, 768), (3, 7), (37, 96), (5, 513), (9, 1001), (4, 1025), (130, 2050), (3, 4099), (2, 8192),
          (2, 8200), (2, 32768), (1023, 40), (64, 1003), (2100, 129), (3, 12_001)]


def _x(rng, rows, cols, t):
    return rounded(rng.normal(size=(rows, cols)), t)


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout(rows, cols, t):
    rng = np.random.default_rng(rows * 7 + cols)
    x, x64 = _x(rng, rows, cols, t)
    r, r64 = _x(rng, rows, cols, t)
    say(f"  dropout {rows} x {cols} {t}")
    for p, res in ((0.1, False), (0.5, True), (0.0, True), (1.0, True), (1.0, False)):
        want = F.oracle_dropout(x64, p, SEED, OFFSET, r64 if res else None)
        y = hs.dropout(put(x), p, SEED, OFFSET, residual=put(r) if res else None)
        # the factor's, the product's and the sum's fp32 rounding, then the store's
        bound = u(t) * np.abs(want) + 4 * U * (2 * np.abs(x64) / max(1 - p, 0.5) + np.abs(r64)) + TINY[t]
        within(y, want, bound, f"y p={p} res={res}")
        if not res:
            assert ((host(y) == 0) == (want == 0)).all(), "the mask differs"


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_dropout_strides_values_and_place(t):
    rows, cols, p = 33, 203, 0.4
    rng = np.random.default_rng(1)
    x, x64 = _x(rng, rows, cols, t)
    r, r64 = _x(rng, rows, cols, t)
    x[3, ::2] = float("nan")
    x[4, ::2] = float("inf")
    x64 = x.double().numpy()
    f = F.drop_factor(rows, cols, p, 5, 6)
    want = F.oracle_dropout(x64, p, 5, 6, r64)
    y = hs.dropout(strided(x, 5, 1), p, 5, 6, residual=strided(r, 3))
    got = host(y)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    assert (got[f == 0] == r64[f == 0]).all()
    fine = np.isfinite(want) & np.isfinite(x64)      # the dropped ones are compared above
    within(got[fine], want[fine], u(t) * np.abs(want[fine]) + 4 * U * (4 * np.abs(x64[fine]) + np.abs(r64[fine])), "y")
    # in place, and on a side stream
    a = put(x).clone()
    hs.dropout(a, p, 5, 6, residual=put(r), out=a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = hs.dropout(put(x), p, 5, 6, residual=put(r))
    torch.cuda.synchronize()
    for z in (a, b):
        assert torch.equal(torch.nan_to_num(z.float()), torch.nan_to_num(y.float()))


def test_dropout_backward_is_the_same_mask_and_graphs_move_on():
    x, _ = _x(np.random.default_rng(2), 64, 768, "bf16")
    off = torch.zeros(1, dtype=torch.int64, device=dev())
    xd, y = put(x), torch.empty(64, 768, dtype=torch.bfloat16, device=dev())
    hs.dropout(xd, 0.3, 11, 5, out=y, offset_dev=off)
    dx = hs.dropout(torch.ones_like(xd), 0.3, 11, 5)
    assert ((y == 0) == (dx == 0)).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hs.dropout(xd, 0.3, 11, 5, out=y, offset_dev=off)
        off.add_(1)
    off.zero_()
    for step in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, hs.dropout(xd, 0.3, 11, 5 + step)), f"replay {step}"


def _norm_bounds(x64, r64, gamma, want, p, cols, t):
    """Bounds of sum, rstd and y: v is off by 4 U (|x f| + |r|); the mean of squares adds cols / 64 + 16 roundings at
    most (lane sums of at most 32 values, a tree, and the division), rstd halves them."""
    dv = 4 * U * (np.abs(x64) / (1 - p) * 2 + np.abs(r64))
    rel = (40 + 16) * U + (dv * np.abs(want["sum"])).mean(1) / np.maximum((want["sum"] ** 2).mean(1), 1e-30)
    by = np.abs(gamma) * want["rstd"][:, None] * dv + (rel[:, None] + 4 * U) * np.abs(want["y"])
    return {"sum": u(t) * np.abs(want["sum"]) + dv + TINY[t], "rstd": rel * want["rstd"],
            "fine": by, "y": u(t) * (np.abs(want["y"]) + by) + by + TINY[t]}


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_add_norm(rows, cols, t):
    rng = np.random.default_rng(rows + 31 * cols)
    x, x64 = _x(rng, rows, cols, t)
    r, r64 = rounded(2 * rng.normal(size=(rows, cols)), t)
    g, g64 = rounded(1 + 0.2 * rng.normal(size=cols), t)
    say(f"  add_norm {rows} x {cols} {t}")
    for p, res in ((0.0, True), (0.25, True), (0.0, False)):
        rr = r64 if res else np.zeros_like(x64)
        want = F.oracle_add_norm(x64, g64, rr, 1e-6, p, SEED, OFFSET)
        out = hs.add_norm(put(x), put(g), residual=put(r) if res else None, p=p, seed=SEED, offset=OFFSET, want_a8=True)
        b = _norm_bounds(x64, rr, g64, want, p, cols, t)
        for k in ("sum", "rstd", "y"):
            within(out[k], want[k], b[k], f"{k} p={p}")
        _check_codes(out["q"], out["scale"], want["y"], b["fine"])


def _check_codes(q, scale, y, err):
    """Codes and scales of y, known to within err: the scale is max |y| / 448 to err's maximum, and a code stands for
    y / scale to half a step (relative 2^-4, or 2^-10 among the subnormals), off by err and the scale's error."""
    top = np.abs(y).max(1)
    ds = err.max(1) / 448 + 4 * U * top / 448
    within(scale, top / 448, ds, "scale")
    s = np.maximum(host(scale), 1e-300)[:, None]
    v = y / s
    slack = err / s + (6 * U + ds[:, None] / s) * np.abs(v)
    half = np.maximum(2.0 ** -4 * (np.abs(v) + slack), 2.0 ** -10)
    within(host(q), v, half + slack, "codes")


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_add_norm_edge_rows(t):
    cols = 200
    rng = np.random.default_rng(3)
    x, _ = _x(rng, 6, cols, t)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    x[4] *= 1e-18
    x[5] *= 1e15
    g, g64 = rounded(np.ones(cols), t)
    big = strided(x, 9, 3)
    out = hs.add_norm(big, put(g), eps=1e-6, want_a8=True)
    y, q, s = host(out["y"]), host(out["q"]), host(out["scale"])
    assert (y[1] == 0).all() and (q[1] == 0).all() and s[1] == 0
    assert np.isnan(y[2]).all() and np.isnan(q[2]).all()
    assert np.isnan(y[3][5])
    for row in (0, 4, 5):
        want = F.oracle_add_norm(x.double().numpy()[row:row + 1], g64, None, 1e-6, 0.0, 0, 0)
        within(y[row:row + 1], want["y"], u(t) * np.abs(want["y"]) * 1.01 + 80 * U * np.abs(want["y"]), f"row {row}")
    # the sum may take the residual's place, and outputs that are not asked for are not needed
    r, _ = _x(rng, 6, cols, t)
    x0, _ = _x(rng, 6, cols, t)
    ref = hs.add_norm(put(x0), put(g), residual=put(r))
    a = put(r).clone()
    out = hs.add_norm(put(x0), put(g), residual=a, out={"sum": a, "y": torch.empty_like(a)})
    assert torch.equal(out["sum"], ref["sum"]) and torch.equal(out["y"], ref["y"])
    only = hs.add_norm(put(x0), put(g), residual=put(r), out={"y": torch.empty_like(a)})
    assert torch.equal(only["y"], ref["y"])


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(4500, 264), (1500, 1100)])
def test_add_norm_bwd(rows, cols, t):
    rng = np.random.default_rng(rows + 17 * cols)
    dy, dy64 = _x(rng, rows, cols, t)
    v, v64 = rounded(2 * rng.normal(size=(rows, cols)), t)
    g, g64 = rounded(1 + 0.2 * rng.normal(size=cols), t)
    ds, ds64 = _x(rng, rows, cols, t)
    rstd = torch.from_numpy(1.0 / np.sqrt((v64 ** 2).mean(1) + 1e-6)).float()
    r64 = rstd.double().numpy()
    say(f"  add_norm_bwd {rows} x {cols} {t}")
    for p, with_ds in ((0.0, True), (0.25, True), (0.1, False)):
        want = F.oracle_add_norm_bwd(dy64, v64, g64, r64, ds64 if with_ds else None, p, SEED, OFFSET)
        out = hs.add_norm_bwd(put(dy), put(v), put(g), put(rstd), dsum=put(ds) if with_ds else None, p=p, seed=SEED,
                              offset=OFFSET)
        # each term is off by a few U of itself; the mean's terms by 56 more (lane sums and the tree)
        xh, gg = np.abs(v64 * r64[:, None]), np.abs(dy64 * g64)
        fine = r64[:, None] * (6 * U * gg + 64 * U * xh * (xh * gg).mean(1, keepdims=True)) + 2 * U * np.abs(ds64)
        f = 1.0 / (1 - p) * 1.001
        within(out["dres"], want["dres"], u(t) * (np.abs(want["dres"]) + fine) + fine + TINY[t], f"dres p={p}")
        if p:
            within(out["dx"], want["dx"], f * ((u(t) + 4 * U) * (np.abs(want["dx"]) + fine) + fine) + TINY[t], f"dx p={p}")
            assert ((host(out["dx"]) == 0) | (F.drop_factor(rows, cols, p, SEED, OFFSET) > 0)).all()
        # rows / 1024 + 1 + 3 sequential additions, then n / 16 + 16 of up to 1024 partials
        n = (rows / 1024 + 4) + (1024 / 16 + 16) + 3
        within(out["dgamma"], want["dgamma"], n * U * np.abs(dy64 * v64 * r64[:, None]).sum(0) + 1e-30, "dgamma")
        again = hs.add_norm_bwd(put(dy), put(v), put(g), put(rstd), dsum=put(ds) if with_ds else None, p=p, seed=SEED,
                                offset=OFFSET)
        assert all(torch.equal(again[k], out[k]) for k in out), "not repeatable"


def test_add_norm_bwd_strides_and_no_dgamma():
    rng = np.random.default_rng(8)
    rows, cols = 21, 300
    dy, _ = _x(rng, rows, cols, "bf16")
    v, v64 = _x(rng, rows, cols, "bf16")
    g, _ = rounded(1 + 0.2 * rng.normal(size=cols), "bf16")
    ds, _ = _x(rng, rows, cols, "bf16")
    rstd = put(torch.from_numpy(1.0 / np.sqrt((v64 ** 2).mean(1) + 1e-6)).float())
    ref = hs.add_norm_bwd(put(dy), put(v), put(g), rstd, dsum=put(ds))
    out = hs.add_norm_bwd(strided(dy, 7, 1), put(v), put(g), rstd, dsum=strided(ds, 4),
                          out={"dres": torch.empty_like(ref["dres"]), "dx": torch.empty_like(ref["dres"])})
    assert torch.equal(out["dres"], ref["dres"]) and torch.equal(out["dx"], ref["dres"])


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_rows(rows, cols, t):
    x, x64 = _x(np.random.default_rng(cols), rows, cols, t)
    q, s = hs.quantize_rows(put(x))
    _check_codes(q, s, x64, np.zeros_like(x64))
    q2, s2 = hs.quantize_rows(strided(x, 3, 2))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_quantize_rows_of_the_smallest_numbers(t):
    """Rows whose scale would be subnormal: the scale stops at 2^-126, and a code is off by half a step of its own
    (2^-4 of it, or 2^-10 among the subnormal codes)."""
    top = [-108, -116, -117, -118, -119, -120, -126]
    x, x64 = rounded(np.random.default_rng(4).uniform(-1, 1, (len(top), 300)) * 2.0 ** np.array(top)[:, None], t)
    q, s = hs.quantize_rows(put(x))
    scale = host(s)
    want = np.maximum(np.abs(x64).max(1) / 448, 2.0 ** -126)
    within(scale, want, 4 * U * want, "scale")
    v = x64 / scale[:, None]
    within(host(q), v, np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 6 * U * np.abs(v), "codes")


# one request, ragged rows and labels, depths that end inside a 128-deep step, several tiles both ways
@pytest.mark.parametrize("B,H,L", [(1, 16, 1), (1, 768, 1000), (2, 144, 17), (16, 1024, 333), (17, 768, 129),
                                   (33, 80, 515), (64, 768, 1031), (65, 640, 260), (130, 256, 1001), (300, 1040, 777),
                                   (3, 2064, 70), (17, 144, 61_700), (130, 256, 9001), (257, 80, 4100), (1025, 64, 1100),
                                   (40, 1040, 27_001), (600, 192, 1803), (129, 16, 8193), (2100, 320, 501)])
def test_score(B, H, L):
    rng = np.random.default_rng(B + L)
    hq = torch.from_numpy(rng.normal(size=(B, H)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    Wq = torch.from_numpy(rng.normal(size=(L, H)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    h_s, w_s = torch.from_numpy(rng.uniform(0.001, 0.1, B)).float(), torch.from_numpy(rng.uniform(0.001, 0.1, L)).float()
    Z = hs.score_a8w8(put(hq), put(h_s), put(Wq), put(w_s))
    a, b = hq.double().numpy(), Wq.double().numpy()
    want = F.oracle_score(a, h_s.double().numpy(), b, w_s.double().numpy())
    # products are exact; H additions of one U each, in any order, and the two scalings
    bound = (H + 4) * U * F.oracle_score(np.abs(a), h_s.double().numpy(), np.abs(b), w_s.double().numpy())
    say(f"  score {B} x {H} x {L}")
    within(Z, want, bound, "Z")


def test_norm_codes_feed_the_scores():
    rng = np.random.default_rng(12)
    x, x64 = _x(rng, 40, 768, "bf16")
    W, W64 = rounded(rng.normal(size=(500, 768)) / 28, "bf16")
    g, _ = rounded(np.ones(768), "bf16")
    out = hs.add_norm(put(x), put(g), want_y=False, want_a8=True)
    wq, ws = hs.quantize_rows(put(W))
    Z = host(hs.score_a8w8(out["q"], out["scale"], wq, ws))
    y = F.oracle_add_norm(x64, np.ones(768), None, 1e-6, 0.0, 0, 0)["y"]
    want = y @ W64.T
    # two operands off by at most 2^-4 each, independent over 768 terms: a sixteenth of the row norms is far outside
    assert np.linalg.norm(Z - want) / np.linalg.norm(want) < 2.0 ** -4


@pytest.mark.parametrize("B,H,L", [(20, 64, 70), (40, 80, 90), (260, 80, 4100), (260, 64, 4102)])
def test_score_nan_code_stays_in_its_row_and_label(B, H, L):
    hq = torch.ones(B, H).to(torch.float8_e4m3fn)
    Wq = torch.ones(L, H).to(torch.float8_e4m3fn)
    hq[3, 60] = float("nan")
    Wq[65, 0] = float("nan")
    one = lambda n: torch.ones(n, device=dev())  # noqa: E731
    Z = host(hs.score_a8w8(put(hq), one(B), put(Wq), one(L)))
    nan = np.zeros((B, L), bool)
    nan[3] = nan[:, 65] = True
    assert np.array_equal(np.isnan(Z), nan) and (Z[~nan] == H).all()


def test_dropout_and_norm_past_32_bit_offsets():
    """More than 2^31 elements: the last rows, against the oracle's rows at those positions."""
    rows, cols, p, tail = 70_000, 32_768, 0.25, 3
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=dev())
    y = hs.dropout(x, p, SEED, OFFSET)
    per, first = cols // 8, (rows - tail) * (cols // 8)
    i = np.arange(first, rows * per, dtype=np.uint64)
    w = F.philox4x32([i % np.uint64(2**32), i >> np.uint64(32), np.full_like(i, OFFSET % 2**32),
                      np.full_like(i, OFFSET >> 32)], [SEED % 2**32, SEED >> 32])
    half = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1).reshape(tail, cols)
    assert np.array_equal(host(y[-tail:] != 0), (half >= round(p * 65536)).astype(float))
    del y
    x[-tail:] = torch.arange(cols, device=dev()).bfloat16() / cols
    out = hs.add_norm(x, torch.ones(cols, dtype=torch.bfloat16, device=dev()), out={"y": torch.empty_like(x)})
    v = host(x[-1:])
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
    within(out["y"][-1:], want, u("bf16") * np.abs(want) * 1.01 + 80 * U * np.abs(want), "last row")


def test_score_past_32_bit_offsets():
    B, H, L = 1100, 32, 2_000_000         # Z has 2.2e9 elements
    g = torch.Generator(device=dev()).manual_seed(3)
    hq = torch.randn(B, H, device=dev(), generator=g).to(torch.float8_e4m3fn)
    Wq = torch.randn(L, H, device=dev(), generator=g).to(torch.float8_e4m3fn)
    Z = hs.score_a8w8(hq, torch.ones(B, device=dev()), Wq, torch.ones(L, device=dev()))
    a, b = host(hq.float()[-2:]), host(Wq.float()[-300:])
    within(Z[-2:, -300:], a @ b.T, (H + 4) * U * (np.abs(a) @ np.abs(b).T), "the last corner")
