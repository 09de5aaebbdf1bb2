"""The linear layer and its epilogue on the GPU against the formulas in 64 bits."""
import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import F64, U32, Out, assert_within, randn, rng, sync_ok, workspace

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def case(M, N, K, act="id", bias=False, mul=False, residual=False, seed=0):
    g = rng(seed)
    return dict(M=M, N=N, K=K, act=act, X=randn(g, M, K, dtype=BF),
                W=randn(g, N, K, std=K ** -0.5, dtype=BF),
                bias=randn(g, N, std=0.5) if bias else None,
                mul=randn(g, M, N, dtype=BF) if mul else None,
                residual=randn(g, M, N, dtype=BF) if residual else None,
                dY=randn(g, M, N, dtype=BF))


def act64(p, act):
    return p * torch.sigmoid(p) if act == "silu" else p


def dact64(p, act):
    s = torch.sigmoid(p)
    return s * (1 + p * (1 - s)) if act == "silu" else torch.ones_like(p)


def forward(c, want_p=True):
    M, N, K = c["M"], c["N"], c["K"]
    Y, P = Out(M, N, dtype=BF), Out(M, N, dtype=BF) if want_p else None
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 0)
    ttt.ttt_linear_fwd(M, N, K, c["act"], c["X"], c["W"], c["bias"], c["mul"], c["residual"], Y.t,
                       P and P.t, workspace(n) if n else None, n)
    sync_ok()
    return Y.check(), P and P.check()


def check_forward(c):
    Y, P = forward(c)
    X, W = c["X"].to(F64), c["W"].to(F64)
    b = c["bias"].to(F64) if c["bias"] is not None else torch.zeros(c["N"], dtype=F64, device="cuda")
    p = X @ W.t() + b
    # products of bf16 pairs are exact in float32; K additions, each off by at most a whole
    # float32 step (the tensor cores may truncate)
    e = 2 * U32 * ((c["K"] + 8) * (X.abs() @ W.abs().t()) + 2 * b.abs())
    assert_within("P", P, p, e)
    # |silu'| < 1.1; the sigmoid's exponential, sum and quotient: under 2 |p| + 12 float32 steps
    y, ye = act64(p, c["act"]), 1.1 * e
    if c["act"] == "silu":
        ye = ye + (2 * p.abs() + 12) * 2 * U32 * y.abs()
    if c["mul"] is not None:
        m = c["mul"].to(F64)
        y, ye = y * m, ye * m.abs() + U32 * (y * m).abs()
    if c["residual"] is not None:
        r = c["residual"].to(F64)
        y, ye = y + r, ye + U32 * (y + r).abs()
    assert_within("Y", Y, y, ye)
    assert torch.equal(forward(c, want_p=False)[0], Y)  # a fixed order of sums
    return P


def backward(c, P, want=("dX", "dW", "dbias", "dmul")):
    M, N, K = c["M"], c["N"], c["K"]
    shape = dict(dX=(M, K), dW=(N, K), dbias=(N,), dmul=(M, N))
    out = {k: Out(*shape[k], dtype=torch.float32 if k == "dbias" else BF) for k in want
           if k != "dmul" or c["mul"] is not None}
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 1)
    ttt.ttt_linear_bwd(M, N, K, c["act"], c["X"], c["W"], P, c["mul"], c["dY"],
                       **{k: o.t for k, o in out.items()}, workspace=workspace(n),
                       workspace_bytes=n)
    sync_ok()
    return {k: o.check() for k, o in out.items()}


def check_backward(c, P):
    need_p = c["act"] != "id" or c["mul"] is not None
    out = backward(c, P if need_p else None)
    X, W, dy, p = (t.to(F64) for t in (c["X"], c["W"], c["dY"], P))
    m = c["mul"].to(F64) if c["mul"] is not None else torch.ones_like(dy)
    if "dmul" in out:
        a = act64(p, c["act"])
        assert_within("dmul", out["dmul"], dy * a, (2 * p.abs() + 14) * 2 * U32 * (dy * a).abs())
    dp = dy * m * dact64(p, c["act"])
    # act' = s (1 + p (1 - s)): s off by (|p| + 6) steps, the bracket by as much of 1 + |p|
    de = (dy * m).abs() * 2 * U32 * (2 * p.abs() + 12) * (1 + p.abs()) if need_p else 0 * dy
    k = 2 * U32 * (c["M"] + 64)
    assert_within("dbias", out["dbias"], dp.sum(0), de.sum(0) + k * dp.abs().sum(0))
    # the products take dP rounded to bf16; where its float32 value lies within de of a midpoint
    # the rounding may go the other way, one bf16 step (2^-7) off
    r = dp.to(torch.float32).to(BF).to(F64)
    near = ((dp - r).abs() - _half_gap(r, dp)).abs() <= de + 4 * U32 * dp.abs()
    slack = torch.where(near & need_p, 2.0 ** -7 * dp.abs(), torch.zeros_like(dp))
    assert_within("dX", out["dX"], r @ W,
                  2 * U32 * (c["N"] + 8) * (r.abs() @ W.abs()) + slack @ W.abs())
    assert_within("dW", out["dW"], r.t() @ X,
                  2 * U32 * (c["M"] + 64) * (r.abs().t() @ X.abs()) + slack.t() @ X.abs())
    for some in (("dX",), ("dW",), ("dbias",), ("dmul",) if c["mul"] is not None else ("dW", "dX")):
        part = backward(c, P if need_p else None, some)
        assert all(torch.equal(v, out[k]) for k, v in part.items()), some


def _half_gap(r, v):
    """Half the distance from the bf16 value r to its neighbour on v's side (float64)."""
    bits = r.to(BF).view(torch.int16).to(torch.int32)
    nb = torch.where(v.abs() > r.abs(), bits + 1, bits - 1)  # away from zero, towards zero
    nb = torch.where((bits & 0x7FFF) == 0, bits, nb)
    return (((nb & 0xFFFF) << 16).view(torch.float32).to(F64) - r).abs() / 2


def check(c):
    check_backward(c, check_forward(c).clone())


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128,
                               129, 200, 255, 256, 257, 300, 511, 513, 1000])
def test_token_counts(M):
    check(case(M, 136, 200, "silu", bias=True, mul=True, residual=True, seed=M))


@pytest.mark.parametrize("N", [8, 16, 24, 56, 64, 72, 120, 128, 136, 248, 256, 264, 504, 520, 1000])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_output_widths(M, N):
    check(case(M, N, 72, "silu", bias=True, seed=N))
    check(case(M, N, 136, "id", bias=True, residual=True, seed=N + 1))


@pytest.mark.parametrize("K", [8, 16, 24, 56, 64, 72, 120, 128, 136, 192, 256, 520, 1000, 1544, 2560])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_contraction_lengths(M, K):
    check(case(M, 96, K, "id", seed=K))
    check(case(M, 160, K, "silu", mul=True, seed=K + 1))


OPTIONS = [(a, b, m, r) for a in ("id", "silu") for b in (False, True) for m in (False, True)
           for r in (False, True)]


@pytest.mark.parametrize("act,bias,mul,residual", OPTIONS)
@pytest.mark.parametrize("M,N,K", [(4, 264, 136), (150, 200, 328), (600, 520, 264)])
def test_epilogues(M, N, K, act, bias, mul, residual):
    check(case(M, N, K, act, bias, mul, residual, seed=5))


@pytest.mark.parametrize("M,N,K", [(8, 2560, 2560), (16, 9728, 2560), (1, 2560, 9728),
                                   (64, 2048, 2048), (200, 2560, 2560), (1537, 1000, 520),
                                   (2048, 2048, 2048), (4100, 1024, 1024), (777, 2568, 1032),
                                   (12000, 256, 64), (3000, 8, 2560), (5000, 2560, 8),
                                   (20000, 136, 72)])
def test_model_sizes(M, N, K):
    check(case(M, N, K, "silu", bias=True, mul=True, seed=M))


@pytest.mark.parametrize("M", [3, 200, 900])
def test_the_residual_stream_in_place(M):
    c = case(M, 328, 136, "silu", bias=True, mul=True, residual=True, seed=2)
    Y, _ = forward(c)
    n = ttt.ttt_linear_workspace_bytes(M, 328, 136, 0)
    for which in ("residual", "mul"):
        d = dict(c, **{which: c[which].clone()})
        ttt.ttt_linear_fwd(M, 328, 136, "silu", d["X"], d["W"], d["bias"], d["mul"], d["residual"],
                           d[which], None, workspace(n) if n else None, n)
        sync_ok()
        assert torch.equal(d[which], Y), which


@pytest.mark.parametrize("M,N,K", [(5, 136, 64), (300, 136, 200)])
def test_a_bad_row_stays_in_its_row(M, N, K):
    c = case(M, N, K, "silu", bias=True, residual=True, seed=2)
    Y = forward(c)[0].clone()
    c["X"][M // 2, 3] = float("nan")
    c["residual"][0, 5] = float("inf")
    Z, _ = forward(c)
    ok = torch.ones((M, N), dtype=torch.bool, device="cuda")
    ok[M // 2], ok[0, 5] = False, False
    assert torch.equal(Z[ok], Y[ok]) and not torch.isfinite(Z[~ok].float()).any()
    # large pre-activations: silu(p) is p or 0, not NaN
    c = case(M, N, K, "silu", seed=3)
    c["X"] *= 1e4
    Z, P = forward(c)
    assert torch.isfinite(Z.float()).all()
    big = P.float().abs() > 200
    assert bool(big.any()) and torch.equal(Z[big], torch.where(P > 0, P, torch.zeros_like(P))[big])


def test_gradient_against_differences():
    # J = <dY, Y> along random directions in 64 bits around the inputs. dP is rounded to bf16 for
    # the products and the outputs are bf16: random relative errors of up to 2^-8 per term, whose
    # signed sum over thousands of entries stays under a tenth of 2 x 2^-8 of the sum of sizes
    c = case(40, 96, 136, "silu", bias=True, mul=True, seed=17)
    M, N, K = c["M"], c["N"], c["K"]
    _, P = forward(c)
    out = backward(c, P)
    at = dict(X=c["X"].to(F64), W=c["W"].to(F64), bias=c["bias"].to(F64), mul=c["mul"].to(F64))

    def J(a):
        return float((act64(a["X"] @ a["W"].t() + a["bias"], "silu") * a["mul"] *
                      c["dY"].to(F64)).sum())

    g, h = rng(18), 1e-5
    for k, grad in (("X", "dX"), ("W", "dW"), ("bias", "dbias"), ("mul", "dmul")):
        v = randn(g, *at[k].shape).to(F64)
        num = (J(dict(at, **{k: at[k] + h * v})) - J(dict(at, **{k: at[k] - h * v}))) / (2 * h)
        gr = out[grad].to(F64)
        assert abs(num - float((gr * v).sum())) <= 8e-4 * float((gr * v).abs().sum()), k


def test_more_than_2_31_elements():
    M, N, K = (1 << 17) + 5, 16392, 64
    c = case(8, N, K, "silu", bias=True, seed=4)
    X = torch.empty((M, K), dtype=BF, device="cuda").normal_(generator=rng(9))
    Y = torch.empty((M, N), dtype=BF, device="cuda")
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 0)
    ttt.ttt_linear_fwd(M, N, K, "silu", X, c["W"], c["bias"], None, None, Y, None,
                       workspace(n) if n else None, n)
    sync_ok()
    for rows in (slice(0, 8), slice(M - 8, M)):
        c["X"], c["M"] = X[rows].contiguous(), 8
        want, _ = forward(c)
        p = c["X"].to(F64) @ c["W"].to(F64).t() + c["bias"].to(F64)
        assert_within("Y", Y[rows], act64(p, "silu"), 1e-4 * torch.ones_like(p))
        assert (want.float() - Y[rows].float()).abs().max() <= 0.05


@pytest.mark.parametrize("act,bias,mul,residual", OPTIONS)
@pytest.mark.parametrize("M,N,K", [(5003, 520, 136), (9000, 264, 72)])
def test_epilogues_of_many_tiles(M, N, K, act, bias, mul, residual):
    # enough tiles for the persistent kernel, edges inside a tile, several tiles to a CTA
    check(case(M, N, K, act, bias, mul, residual, seed=6))


@pytest.mark.parametrize("both", [False, True])
def test_many_tiles_in_place(both):
    M, N, K = 6001, 392, 136
    c = case(M, N, K, "silu", bias=True, mul=True, residual=both, seed=4)
    Y, _ = forward(c)
    for which in ("mul", "residual") if both else ("mul",):
        for _ in range(3):
            d = dict(c, **{which: c[which].clone()})
            ttt.ttt_linear_fwd(M, N, K, "silu", d["X"], d["W"], d["bias"], d["mul"], d["residual"],
                               d[which])
            sync_ok()
            assert torch.equal(d[which], Y), which


@pytest.mark.parametrize("M,N,K", [(8, 12800, 1032), (16, 14208, 1032), (5, 6272, 2560), (24, 8960, 1032), (24, 9472, 1032),
                                   (32, 4224, 2048), (100, 4096, 1024), (130, 3136, 2056), (64, 9088, 520),
                                   (200, 1024, 4096), (77, 2112, 9728)])
def test_contractions_shared_up_to_what_is_resident(M, N, K):
    # tiles on both sides of the CTAs that fit, shared 1, 2, 4 and 8 ways, with ragged edges
    check_forward(case(M, N, K, "silu", bias=True, mul=True, residual=True, seed=N))
