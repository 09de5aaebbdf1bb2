"""Layer norm on the GPU against the formulas in 64 bits, at the widths, row counts, layouts and
values where a kernel can go wrong."""
import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import DT, F64, U32, Out, assert_within, randn, rng, sync_ok, workspace

pytestmark = pytest.mark.gpu

EPS = 1e-5


def case(B, H, T, d, dtype, token_major=False, residual=False, affine=True, seed=0, offset=1.0):
    g, dt = rng(seed), DT[dtype]
    yshape = (B, T, H, d) if token_major else (B, H, T, d)
    x = randn(g, B, H, T, d) + offset * randn(g, B, H, T, 1)
    return dict(cfg=ttt.make_norm_config(B, H, T, d, dtype, token_major, EPS), shape=(B, H, T, d),
                yshape=yshape, dt=dt, token_major=token_major, X=x.to(dt),
                residual=randn(g, B, H, T, d, dtype=dt) if residual else None,
                weight=randn(g, H, d, std=0.2, mean=1.0) if affine else None,
                bias=randn(g, H, d, std=0.2) if affine else None,
                dY=randn(g, *yshape, dtype=dt),
                dS=randn(g, B, H, T, d, dtype=dt) if residual else None)


def heads_first(c, y):
    return y.transpose(1, 2) if c["token_major"] else y


def forward(c, stats=True):
    B, H, T, d = c["shape"]
    Y = Out(*c["yshape"], dtype=c["dt"])
    S = Out(*c["shape"], dtype=c["dt"]) if c["residual"] is not None else None
    mean, rstd = (Out(B, H, T), Out(B, H, T)) if stats else (None, None)
    ttt.ttt_norm_fwd(c["cfg"], c["X"], c["residual"], c["weight"], c["bias"], Y.t, S and S.t,
                     mean and mean.t, rstd and rstd.t)
    sync_ok()
    return [o and o.check() for o in (Y, S, mean, rstd)]


def check_forward(c):
    Y, S, mean, rstd = forward(c)
    s = c["X"].to(F64) + (c["residual"].to(F64) if c["residual"] is not None else 0)
    mu = s.mean(-1, keepdim=True)
    var = ((s - mu) ** 2).mean(-1, keepdim=True)
    r = (var + EPS).rsqrt()
    xh = (s - mu) * r
    w = c["weight"].to(F64)[:, None] if c["weight"] is not None else 1.0
    b = c["bias"].to(F64)[:, None] if c["bias"] is not None else torch.zeros_like(xh)
    big = s.abs().amax(-1, keepdim=True)
    # Float32 sums of up to 16384 terms by threads (at most 64 each) and trees: under 96 roundings
    # each. The mean is off by e = 96 U32 big; the variance by a relative 100 U32 and by e^2,
    # rstd by half of that; x - mean by e + U32 big.
    e = 96 * U32 * big
    rel = 64 * U32 + 0.5 * e * e * r * r
    assert_within("mean", mean, mu[..., 0], e[..., 0])
    assert_within("rstd", rstd, r[..., 0], (rel * r)[..., 0])
    bound = ((e + 2 * U32 * big) * r + (rel + 4 * U32) * xh.abs()) * (abs(w) if c["weight"] is None
                                                                       else w.abs()) + \
        2 * U32 * b.abs()
    assert_within("Y", heads_first(c, Y), xh * w + b, bound)
    if S is not None:
        assert_within("S", S, s, U32 * s.abs())


def check_backward(c):
    B, H, T, d = c["shape"]
    s = c["X"].to(F64)
    mean = s.mean(-1).float()
    rstd = (s.var(-1, unbiased=False) + EPS).rsqrt().float()
    dX, dw, db = Out(*c["shape"], dtype=c["dt"]), Out(H, d), Out(H, d)
    n = ttt.ttt_norm_bwd_workspace_bytes(c["cfg"])
    ws = workspace(n)
    args = (c["X"], c["weight"], mean, rstd, c["dY"], c["dS"])
    ttt.ttt_norm_bwd(c["cfg"], *args, dX.t, dw.t, db.t, ws, n)
    sync_ok()
    for o in (dX, dw, db):
        o.check()
    dy = heads_first(c, c["dY"].to(F64))
    m, r = mean.to(F64)[..., None], rstd.to(F64)[..., None]
    w = c["weight"].to(F64)[:, None] if c["weight"] is not None else torch.ones((), dtype=F64,
                                                                               device="cuda")
    xh, g = (s - m) * r, dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dS = c["dS"].to(F64) if c["dS"] is not None else torch.zeros_like(s)
    ref = r * (g - c1 - xh * c2) + dS
    # each row mean: under 96 roundings of its terms; the rest a few per term. x - mean rounds
    # once relative to its own size.
    n1, n2 = g.abs().mean(-1, keepdim=True), (g * xh).abs().mean(-1, keepdim=True)
    bound = r * (8 * U32 * g.abs() + 100 * U32 * n1 + xh.abs() * 108 * U32 * n2) + \
        2 * U32 * dS.abs()
    assert_within("dX", dX.t, ref, bound)
    # sums over the head's rows: at most one rounding per row and 64 in the joins, and four per
    # term; relative to the sum of the terms' sizes
    k = (B * T + 70) * U32
    assert_within("dweight", dw.t, (dy * xh).sum((0, 2)), k * (dy * xh).abs().sum((0, 2)))
    assert_within("dbias", db.t, dy.sum((0, 2)), k * dy.abs().sum((0, 2)))
    # dX alone needs no workspace and is the same; either weight gradient alone is the same
    only = Out(*c["shape"], dtype=c["dt"])
    ttt.ttt_norm_bwd(c["cfg"], *args, only.t)
    one = Out(H, d)
    ttt.ttt_norm_bwd(c["cfg"], *args, torch.empty_like(dX.t), None, one.t, ws, n)
    two = Out(H, d)
    ttt.ttt_norm_bwd(c["cfg"], *args, torch.empty_like(dX.t), two.t, None, ws, n)
    sync_ok()
    assert torch.equal(only.check(), dX.t)
    assert torch.equal(one.check(), db.t) and torch.equal(two.check(), dw.t)


WIDTHS = [1, 2, 3, 7, 8, 17, 31, 33, 64, 65, 77, 100, 128, 129, 136, 250, 256, 264, 511, 512, 520,
          1000, 1021, 1024, 1032, 2048, 2056, 2560, 4096, 4099, 5000, 8192, 8200, 9728, 16383,
          16384]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dtype):
    c = case(2, 1, 19, d, dtype, residual=d % 2 == 0, seed=d)
    check_forward(c)
    check_backward(c)


ROWS = [(1, 1, 1), (1, 1, 2), (1, 2, 1), (5, 3, 1), (1, 1, 147), (1, 1, 149), (3, 2, 97),
        (2, 16, 130), (1, 64, 5), (1, 1, 5000), (7, 1, 1201), (1, 300, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("B,H,T", ROWS)
def test_row_counts_and_layouts(B, H, T, token_major, dtype):
    for d in (64, 77, 328):
        c = case(B, H, T, d, dtype, token_major=token_major, residual=T % 2 == 0, seed=T + d)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 1021, 2560])
def test_without_weight_and_bias(d, dtype):
    c = case(1, 2, 33, d, dtype, affine=False, residual=True, token_major=True, seed=3)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("d", [64, 1000, 2560])
def test_large_means_and_constant_rows(d):
    c = case(1, 1, 40, d, "f32", seed=5, offset=1000.0)
    c["X"][0, 0, 3] = 2.5       # a constant row: variance 0, Y = bias
    c["X"][0, 0, 4] = 0.0
    check_forward(c)
    Y = forward(c)[0]
    assert torch.equal(Y[0, 0, 3], c["bias"][0]) and torch.equal(Y[0, 0, 4], c["bias"][0])


@pytest.mark.parametrize("d", [64, 77, 1024, 2560])
def test_a_bad_row_stays_in_its_row(d):
    c = case(2, 2, 21, d, "bf16", seed=6, token_major=True)
    good = [o.clone() for o in forward(c) if o is not None]
    c["X"][1, 0, 7, d // 2] = float("inf")
    c["X"][0, 1, 2, 0] = float("nan")
    Y, _, mean, rstd = forward(c)
    ok = torch.ones((2, 2, 21), dtype=torch.bool, device="cuda")
    ok[1, 0, 7] = ok[0, 1, 2] = False
    assert torch.equal(heads_first(c, Y)[ok], heads_first(c, good[0])[ok])
    assert torch.equal(mean[ok], good[1][ok]) and torch.equal(rstd[ok], good[2][ok])
    assert not torch.isfinite(heads_first(c, Y)[~ok].float()).any()


@pytest.mark.parametrize("dtype,d", [("bf16", 2560), ("bf16", 77), ("f32", 128), ("f32", 1021)])
def test_the_residual_stream_in_place(dtype, d):
    c = case(1, 1, 50, d, dtype, residual=True, seed=8)
    Y, S, _, _ = [o.clone() for o in forward(c)]
    for which in ("X", "residual"):
        c2 = dict(c, X=c["X"].clone(), residual=c["residual"].clone())
        Y2 = torch.empty_like(Y)
        ttt.ttt_norm_fwd(c["cfg"], c2["X"], c2["residual"], c["weight"], c["bias"], Y2, c2[which])
        sync_ok()
        assert torch.equal(Y2, Y) and torch.equal(c2[which], S)
    mean, rstd = (torch.empty((1, 1, 50), device="cuda") for _ in range(2))
    ttt.ttt_norm_fwd(c["cfg"], c["X"], c["residual"], c["weight"], c["bias"], Y, None, mean, rstd)
    n = ttt.ttt_norm_bwd_workspace_bytes(c["cfg"])
    outs = []
    for in_place in (False, True):
        dS = c["dS"].clone()
        dX = dS if in_place else torch.empty_like(dS)
        dw, db = torch.empty_like(c["weight"]), torch.empty_like(c["bias"])
        ttt.ttt_norm_bwd(c["cfg"], S, c["weight"], mean, rstd, c["dY"], dS, dX, dw, db,
                         workspace(n), n)
        outs.append((dX, dw, db))
    sync_ok()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dtype,d,H", [("f32", 64, 2), ("f32", 1021, 1)])
def test_gradient_against_differences(dtype, d, H):
    # J = <dY, Y> along random directions: central differences in 64 bits of the formula, at the
    # point the kernel differentiated. The formula's third derivative along a unit-spread
    # direction is O(10) per unit of J's terms, so step 1e-4 leaves 1e-7; the kernel's float32
    # gradients add 1e-5 (the bounds above, summed)
    c = case(2, H, 9, d, dtype, seed=11)
    s = c["X"].to(F64)
    w, b, dy = (c[k].to(F64) for k in ("weight", "bias", "dY"))

    def J(s, w, b):
        mu = s.mean(-1, keepdim=True)
        var = ((s - mu) ** 2).mean(-1, keepdim=True)
        return float((((s - mu) * (var + EPS).rsqrt() * w[:, None] + b[:, None]) * dy).sum())

    _, _, mean, rstd = forward(c)
    dX, dw, db = torch.empty_like(c["X"]), torch.empty_like(c["weight"]), torch.empty_like(c["bias"])
    n = ttt.ttt_norm_bwd_workspace_bytes(c["cfg"])
    ttt.ttt_norm_bwd(c["cfg"], c["X"], c["weight"], mean, rstd, c["dY"], None, dX, dw, db,
                     workspace(n), n)
    sync_ok()
    g, h = rng(12), 1e-4
    for grad, k in ((dX, 0), (dw, 1), (db, 2)):
        at = [s, w, b]
        v = randn(g, *grad.shape).to(F64)
        up, dn = list(at), list(at)
        up[k], dn[k] = at[k] + h * v, at[k] - h * v
        num = (J(*up) - J(*dn)) / (2 * h)
        ana = float((grad.to(F64) * v).sum())
        scale = float((grad.to(F64) * v).abs().sum())
        assert abs(num - ana) <= 1e-5 * scale + 1e-6, (k, num, ana)


def test_more_than_2_31_elements():
    # 2^31 + elements in bf16: the last rows sit past 32-bit element offsets
    d, T = 4096, (1 << 19) + 3
    cfg = ttt.make_norm_config(1, 1, T, d, "bf16")
    X = torch.empty((T, d), device="cuda", dtype=torch.bfloat16).normal_(generator=rng(1))
    Y = torch.empty_like(X)
    mean, rstd = (torch.empty(T, device="cuda") for _ in range(2))
    ttt.ttt_norm_fwd(cfg, X, None, None, None, Y, None, mean, rstd)
    dX = torch.empty_like(X)
    dw, db = (torch.empty(d, device="cuda") for _ in range(2))
    n = ttt.ttt_norm_bwd_workspace_bytes(cfg)
    ttt.ttt_norm_bwd(cfg, X, None, mean, rstd, X, None, dX, dw, db, workspace(n), n)
    sync_ok()
    small = ttt.make_norm_config(1, 1, 5, d, "bf16")
    Y5, dX5 = torch.empty_like(Y[-5:]), torch.empty_like(Y[-5:])
    ttt.ttt_norm_fwd(small, X[-5:], None, None, None, Y5)
    ttt.ttt_norm_bwd(small, X[-5:], None, mean[-8:][3:].clone(), rstd[-5:].clone(), X[-5:], None, dX5)
    sync_ok()
    s = X[-5:].to(F64)
    assert_within("Y", Y[-5:], (s - s.mean(-1, keepdim=True)) *
                  (s.var(-1, unbiased=False, keepdim=True) + EPS).rsqrt(), 300 * U32 * s.abs().amax())
    # one row's float32 sums may be split differently in the two calls: one bf16 step apart
    assert_within("dX", dX[-5:], dX5.to(F64), 2.0 ** -8 * dX5.to(F64).abs() + 1e-5)
    total = torch.zeros(d, device="cuda", dtype=F64)
    for i in range(0, T, 1 << 16):
        total += X[i:i + (1 << 16)].to(F64).sum(0)
    assert_within("dbias", db, total, 4096 * U32 * torch.full_like(total, 0.8 * T))


# even widths off 16 bytes (pairs) and odd ones, narrow and wide, at the edges of a thread's share
OFF_WIDTHS = [6, 62, 66, 126, 130, 254, 258, 263, 382, 385, 510, 513, 514, 750, 1025, 1026, 2046, 2049,
              2050, 3094, 4094, 4097, 4098, 8190, 8193, 16382]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", OFF_WIDTHS)
def test_widths_off_sixteen_bytes(d, dtype):
    c = case(1, 2, 23, d, dtype, token_major=d % 4 == 2, residual=d % 2 == 0, seed=d)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,d", [(2, 3, 700, 263), (1, 1, 4100, 750), (3, 2, 900, 1030), (1, 1, 3000, 2560),
                                     (1, 2, 2500, 1021), (2, 1, 700, 4098)])
def test_long_runs_of_wide_rows(B, H, T, d, dtype):
    # many rows to a CTA: the ring of row copies goes round more than once, runs cross batches
    c = case(B, H, T, d, dtype, token_major=H > 1, residual=True, seed=d)
    check_forward(c)
    check_backward(c)


# widths whose last access is shared with lanes past the row's end, narrow and wide, of every access
# size, and ones that fill their threads
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 5, 33, 66, 72, 128, 200, 258, 264, 513, 750, 1021, 1400, 2049, 2560, 4098])
def test_infinities_at_a_row_s_end(d, dtype):
    # an infinity in the last columns is an infinity in the mean (and with its opposite a NaN), as in
    # any other column; in dY it is an infinity in the sums over the row, and dX follows the formula
    inf = float("inf")
    c = case(1, 1, 12, d, dtype, seed=d)
    clean = forward(c)
    X, dY = c["X"].clone(), c["dY"].clone()
    bad = {1: (d - 1, inf), 3: (d - 1, -inf), 4: (max(d - 2, 0), inf), 6: (0, inf), 7: (d - 1, float("nan"))}
    for r, (j, v) in bad.items():
        c["X"][0, 0, r, j] = v
    Y, _, mean, rstd = forward(c)
    for r in range(12):
        if r in bad:
            v = bad[r][1]
            got = float(mean[0, 0, r])
            assert got == v or (v != v and got != got), (d, r, got)
            assert torch.isnan(Y[0, 0, r].float()).all() and not torch.isfinite(rstd[0, 0, r])
        else:
            assert torch.equal(Y[0, 0, r], clean[0][0, 0, r])
    c["X"] = X
    for r, (j, v) in bad.items():
        c["dY"][0, 0, r, j] = v
    dX = torch.empty_like(X)
    ttt.ttt_norm_bwd(c["cfg"], X, c["weight"], clean[2], clean[3], c["dY"], None, dX)
    sync_ok()
    good = torch.empty_like(X)
    ttt.ttt_norm_bwd(c["cfg"], X, c["weight"], clean[2], clean[3], dY, None, good)
    sync_ok()
    xh = (X.float() - clean[2][..., None]) * clean[3][..., None]
    g = c["dY"].float() * c["weight"][:, None]
    want = clean[3][..., None] * (g - g.sum(-1, keepdim=True) / d - xh * ((g * xh).sum(-1, keepdim=True) / d))
    for r in range(12):
        if r in bad:
            a, b = dX[0, 0, r].float(), want[0, 0, r]
            same = torch.where(torch.isnan(b), torch.isnan(a), a == b)
            assert bool(same.all()), (d, r, a[~same][:4], b[~same][:4])
        else:
            assert torch.equal(dX[0, 0, r], good[0, 0, r])
