"""The operators around the layer, used together as a model's block uses them: on one stream, on
a stream of their own, captured and replayed, and with the layer between them."""
import pytest
import torch

import synth
import weight_sequence_layers_b200 as ttt
from _block import randn, rng, sync_ok, workspace

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
B, T, H, D, C = 2, 256, 4, 256, 128   # four heads of 64
R = B * T


def linear(M, N, K, act, X, W, bias=None, mul=None, residual=None, P=None):
    Y = torch.empty((M, N), dtype=BF, device="cuda")
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 0)
    ttt.ttt_linear_fwd(M, N, K, act, X, W, bias, mul, residual, Y, P, workspace(n) if n else None, n)
    return Y


def weights(seed=1):
    g = rng(seed)
    w = {k: randn(g, D, D, std=D ** -0.5, dtype=BF) for k in ("q", "k", "v", "g", "x", "o", "r")}
    w["n1"], w["n2"], w["n3"] = (randn(g, s, std=0.1, mean=1.0) for s in (D, D, D))
    w["b"] = randn(g, D, std=0.1)
    return w


def heads(x):
    return x.view(B, T, H, 64).transpose(1, 2).contiguous()


def unit(x):
    return (x.float() / x.float().norm(dim=-1, keepdim=True)).to(x.dtype)


def block(x, w):
    """Pre-norm, the TTT layer, its output norm and projection onto the residual stream; then a
    gated recurrence on the normed stream."""
    norm = ttt.make_norm_config(B, 1, T, D)
    y = torch.empty_like(x)
    ttt.ttt_norm_fwd(norm, x, None, w["n1"], w["b"], y)
    q, k, v = (linear(R, D, D, "id", y, w[n]) for n in "qkv")
    cfg = ttt.make_config(B, H, T, 64, 64, C, "bf16", "mse", "id", synth.LR_BIAS_ETA0_0P1)
    O = torch.empty((B, H, T, 64), dtype=BF, device="cuda")
    beta = torch.zeros((B, H, T), device="cuda")
    W0 = torch.zeros((B, H, 64, 64), device="cuda")
    n = ttt.ttt_workspace_bytes(cfg, 0)
    ttt.ttt_chunk_fwd(cfg, unit(heads(q)), unit(heads(k)), heads(v), beta, None, W0, O,
                      workspace=workspace(n), workspace_bytes=n)
    on = torch.empty((B, T, H, 64), dtype=BF, device="cuda")
    ttt.ttt_norm_fwd(ttt.make_norm_config(B, H, T, 64, "bf16", True), O, None, w["n2"], None, on)
    a = linear(R, D, D, "id", on, w["o"])
    s, y2 = torch.empty_like(x), torch.empty_like(x)
    ttt.ttt_norm_fwd(norm, x, a, w["n3"], None, y2, s)
    gate, u = linear(R, D, D, "id", y2, w["g"], w["b"]), linear(R, D, D, "silu", y2, w["x"])
    hs, hf = torch.empty((B, T, D), dtype=BF, device="cuda"), torch.empty((B, D), device="cuda")
    ttt.ttt_recur_fwd(ttt.make_recur_config(B, T, D), u, gate, None, None, hs, hf)
    return linear(R, D, D, "id", hs, w["r"], w["b"], None, s), hf, O


def block64(x, w, O):
    """The same in 64 bits, around the layer's own output (which has tests of its own)."""
    d = {k: v.to(F64) for k, v in w.items()}

    def ln(s, weight, bias=0.0):
        mu = s.mean(-1, keepdim=True)
        return (s - mu) * (s.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * weight + bias

    on = ln(O.to(F64), d["n2"].view(H, 1, 64)).transpose(1, 2).reshape(R, D)
    s = x.to(F64).view(R, D) + on @ d["o"].t()
    y2 = ln(s, d["n3"])
    a = torch.sigmoid(y2 @ d["g"].t() + d["b"]).view(B, T, D)
    p = y2 @ d["x"].t()
    u = (p * torch.sigmoid(p)).view(B, T, D)
    h, hs = torch.zeros((B, D), dtype=F64, device="cuda"), []
    for t in range(T):
        h = a[:, t] * h + (1 - a[:, t]) * u[:, t]
        hs.append(h)
    return torch.stack(hs, 1).view(R, D) @ d["r"].t() + d["b"] + s, h


def rel(a, b):
    return float((a.to(F64) - b).norm() / b.norm())


def test_block_with_the_layer_inside():
    x, w = randn(rng(3), B, T, D, dtype=BF), weights()
    y, hf, O = block(x, w)
    sync_ok()
    ry, rh = block64(x, w, O)
    # seven roundings to bf16 of at most 2^-8 each lie on the longest path and the maps between
    # them have gains near one: 7 * 2^-8 = 0.027
    assert rel(y, ry) < 0.027 and rel(hf, rh) < 0.027


def test_block_on_its_own_stream_and_captured():
    w = weights()
    xs = [randn(rng(s), B, T, D, dtype=BF) for s in (3, 4)]
    want = [[t.clone() for t in block(x, w)] for x in xs]
    sync_ok()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(xs[0], w)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x, w)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    sync_ok()


def backward(x, w, dy):
    """norm -> linear (SiLU, gated) -> recurrence -> linear + residual and its backward, every
    gradient from the library's calls."""
    n1 = ttt.make_norm_config(B, 1, T, D)
    y, mean, rstd = torch.empty_like(x), torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    ttt.ttt_norm_fwd(n1, x, None, w["n1"], w["b"], y, None, mean, rstd)
    up, P = linear(R, D, D, "id", y, w["k"]), torch.empty((R, D), dtype=BF, device="cuda")
    z = linear(R, D, D, "silu", y, w["x"], w["b"], up, None, P)
    gate = linear(R, D, D, "id", y, w["g"])
    rc, hs = ttt.make_recur_config(B, T, D), torch.empty_like(x)
    ttt.ttt_recur_fwd(rc, z, gate, None, None, hs)
    out = linear(R, D, D, "id", hs, w["o"], None, None, x)

    def lin_bwd(X, W, dY, act="id", P=None, mul=None, **outs):
        n = ttt.ttt_linear_workspace_bytes(R, D, D, 1)
        ttt.ttt_linear_bwd(R, D, D, act, X, W, P, mul, dY, workspace=workspace(n),
                           workspace_bytes=n, **outs)

    new = lambda: torch.empty((R, D), dtype=BF, device="cuda")
    mat = lambda: torch.empty((D, D), dtype=BF, device="cuda")
    dhs, dwo = new(), mat()
    lin_bwd(hs, w["o"], dy, dX=dhs, dW=dwo)
    dz, dg = new(), new()
    ttt.ttt_recur_bwd(rc, z, gate, None, None, hs, dhs, None, dz, dg)
    dys, dwg, dwx, dwk = [new() for _ in range(3)], mat(), mat(), mat()
    dup, db = new(), torch.empty(D, device="cuda")
    lin_bwd(y, w["g"], dg, dX=dys[0], dW=dwg)
    lin_bwd(y, w["x"], dz, "silu", P, up, dX=dys[1], dW=dwx, dbias=db, dmul=dup)
    lin_bwd(y, w["k"], dup, dX=dys[2], dW=dwk)
    dyt = (dys[0].float() + dys[1].float() + dys[2].float()).to(BF).view_as(x)
    dx, dn, dnb = torch.empty_like(x), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    n = ttt.ttt_norm_bwd_workspace_bytes(n1)
    ttt.ttt_norm_bwd(n1, x, w["n1"], mean, rstd, dyt, dy.view_as(x), dx, dn, dnb, workspace(n), n)
    return dict(out=out, x=dx, n1=dn, bn=dnb, o=dwo, g=dwg, x_w=dwx, k=dwk, b=db)


def test_block_gradients():
    x, w, dy = randn(rng(5), B, T, D, dtype=BF), weights(2), randn(rng(6), R, D, dtype=BF)
    got = backward(x, w, dy)
    sync_ok()
    p = {k: v.to(F64).requires_grad_() for k, v in w.items()}
    xr, bn = x.to(F64).requires_grad_(), w["b"].to(F64).requires_grad_()
    mu = xr.mean(-1, keepdim=True)
    y = ((xr - mu) * (xr.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * p["n1"] + bn)
    y = y.view(R, D)
    pre = y @ p["x"].t() + p["b"]
    z = (pre * torch.sigmoid(pre) * (y @ p["k"].t())).view(B, T, D)
    a = torch.sigmoid(y @ p["g"].t()).view(B, T, D)
    h, hs = torch.zeros((B, D), dtype=F64, device="cuda"), []
    for t in range(T):
        h = a[:, t] * h + (1 - a[:, t]) * z[:, t]
        hs.append(h)
    out = torch.stack(hs, 1).view(R, D) @ p["o"].t() + xr.view(R, D)
    (out * dy.to(F64)).sum().backward()
    # up to eight roundings to bf16 (2^-8 each) on a path, gains near one; differences of nearly
    # equal parts (the gate's) can double them
    tol = 2 * 8 * 2.0 ** -8
    assert rel(got["out"], out.detach()) < tol
    for k, ref in (("x", xr.grad), ("n1", p["n1"].grad), ("bn", bn.grad), ("o", p["o"].grad),
                   ("g", p["g"].grad), ("x_w", p["x"].grad), ("k", p["k"].grad), ("b", p["b"].grad)):
        assert rel(got[k], ref) < tol, (k, rel(got[k], ref))
    again = backward(x, w, dy)
    sync_ok()
    assert all(torch.equal(again[k], got[k]) for k in got)  # no sum depends on an order of arrival


def test_the_gated_mlp_activation_feeds_the_in_place_layer():
    T2, dff, dm, Ck = 256, 512, 256, 128
    g = rng(8)
    x = randn(g, T2, dm, dtype=BF)
    wg, wu = (randn(g, dff, dm, std=dm ** -0.5, dtype=BF) for _ in range(2))
    Z = linear(T2, dff, dm, "silu", x, wg, mul=linear(T2, dff, dm, "id", x, wu))
    W, V = randn(g, dm, dff, std=0.02), randn(g, T2, dm, std=0.02, dtype=BF)
    W1, O = W.clone(), torch.empty((T2, dm), dtype=BF, device="cuda")
    n = ttt.inplace_ttt_workspace_bytes(T2, dff, dm, Ck)
    ttt.inplace_ttt_fwd(T2, dff, dm, Ck, 1e-3, Z, V, W1, O, workspace(n), n)
    sync_ok()
    p = x.to(F64) @ wg.to(F64).t()
    z = p * torch.sigmoid(p) * (x.to(F64) @ wu.to(F64).t())
    w64, o = W.to(F64), []
    for i in range(0, T2, Ck):
        o.append(z[i:i + Ck] @ w64.t())
        w64 = w64 + 1e-3 * V[i:i + Ck].to(F64).t() @ z[i:i + Ck]
    # U, Z, the weight copy and O are rounded to bf16: 4 * 2^-8
    assert rel(O, torch.cat(o)) < 4 * 2.0 ** -8


def test_two_streams_at_once():
    # independent calls on two streams share nothing inside the library
    w = weights(4)
    xs = [randn(rng(s), B, T, D, dtype=BF) for s in (11, 12)]
    dys = [randn(rng(s), R, D, dtype=BF) for s in (13, 14)]
    want = [backward(x, w, d) for x, d in zip(xs, dys)]
    sync_ok()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(backward(xs[i], w, dys[i]))
    sync_ok()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(g[k], want[i][k]) for k in g)


def test_backward_captured_and_replayed():
    # the passes of one call may overlap on the device: a replay orders them as the eager call does
    w = weights(7)
    xs = [randn(rng(s), B, T, D, dtype=BF) for s in (21, 22)]
    dys = [randn(rng(s), R, D, dtype=BF) for s in (23, 24)]
    want = [backward(x, w, d) for x, d in zip(xs, dys)]
    sync_ok()
    x, dy = xs[0].clone(), dys[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = backward(x, w, dy)
    for i in (1, 0, 1, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        sync_ok()
        assert all(torch.equal(out[k], want[i][k]) for k in out), i


def test_back_to_back_backwards_share_a_workspace():
    # calls of one stream one after the other: each waits for what the one before still writes
    M, N, K = 1500, 520, 392
    g = rng(31)
    X, W = randn(g, M, K, dtype=BF), randn(g, N, K, std=K ** -0.5, dtype=BF)
    P, mul = randn(g, M, N, dtype=BF), randn(g, M, N, dtype=BF)
    dys = [randn(g, M, N, dtype=BF) for _ in range(6)]
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 1)
    ws = workspace(n)

    def call(dy):
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        dm, db = torch.empty_like(mul), torch.empty(N, device="cuda")
        ttt.ttt_linear_bwd(M, N, K, "silu", X, W, P, mul, dy, dX, dW, db, dm, ws, n)
        return dX, dW, dm, db

    want = []
    for dy in dys:
        want.append(call(dy))
        torch.cuda.synchronize()
    got = [call(dy) for dy in dys]
    sync_ok()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_binding_refuses_what_does_not_fit():
    cfg = ttt.make_norm_config(1, 1, 4, 64)
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    y = torch.empty_like(x)
    ttt.ttt_norm_fwd(cfg, x, None, None, None, y)
    good = (x, None, None, None, y)
    for i, bad in ((0, x.float()), (0, x[:3]), (0, x.cpu()), (4, torch.empty((64, 4), dtype=BF, device="cuda").t()),
                   (2, torch.ones(63, device="cuda")), (2, torch.ones(64, dtype=BF, device="cuda"))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError, match="ttt_norm_fwd: "):
            ttt.ttt_norm_fwd(cfg, *args)
    ttt.ttt_norm_fwd(cfg, x.data_ptr(), None, None, None, torch.nn.Parameter(y, requires_grad=False))
    sync_ok()
