"""The operators around the layer at the ends of their documented ranges: sizes near 2^31, offsets
past it, decays above one, infinities in a row's last columns, calls after a refused one."""
import ctypes

import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import F64, U32, assert_within, rng, sync_ok, workspace

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("weights", [False, True])
def test_column_sums_of_the_widest_matrix(weights):
    # N as large as a linear layer takes: a step of all CTAs past the last columns would leave 32
    # bits. One row: dbias is dY itself (the sums' own kernel), and with dW the sums are taken along
    # by the products' kernel; dW = dY^T X is a product of two bf16 numbers, rounded once
    M, N, K = 1, 2 ** 31 - 520, 8
    dY = torch.empty((M, N), dtype=BF, device="cuda").normal_(generator=rng(1))
    X = torch.tensor([[1.0, -2.0, 0.5, 3.0, 1.5, -0.75, 7.0, -1.0]], dtype=BF, device="cuda")
    dbias = torch.full((N,), float("nan"), device="cuda")
    dW = torch.empty((N, K), dtype=BF, device="cuda") if weights else None
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ttt.ttt_linear_bwd(M, N, K, "id", X if weights else None, None, None, None, dY, None, dW, dbias,
                       None, ws, n)
    sync_ok()
    step = 1 << 27
    for lo in range(0, N, step):
        y = dY[0, lo:lo + step]
        assert torch.equal(dbias[lo:lo + step], y.float()), lo
        if weights and (lo == 0 or lo + step >= N):
            want = (y.float()[:, None] * X.float()).to(BF)
            assert torch.equal(dW[lo:lo + step], want), lo


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
@pytest.mark.parametrize("D", [65535 * 128 + 3, 65535 * 256 + 130, 40000001])
def test_step_of_very_wide_rows(D, gate, dtype):
    # more blocks of features than one axis of a grid holds. The same values as the same columns in a
    # narrow row: each feature is its own
    dt, n, w = {"bf16": BF, "f32": torch.float32}[dtype], 2, 1000
    g = rng(5)
    X = torch.empty((n, D), device="cuda").normal_(generator=g).to(dt)
    G = torch.empty((n, D), device="cuda").normal_(generator=g)
    G = G.to(dt) if gate == "sigmoid" else torch.sigmoid(G)
    st = torch.empty((3, D), device="cuda").normal_(generator=g)
    slots, Y, old = torch.tensor([2, 0], dtype=torch.int32, device="cuda"), torch.empty_like(X), st.clone()
    ttt.ttt_recur_step(ttt.make_recur_config(n, 1, D, dtype, gate), X, G, slots, st, Y)
    sync_ok()
    assert torch.equal(st[1], old[1])
    small = ttt.make_recur_config(n, 1, w, dtype, gate)
    for lo in (0, min(65535 * 128 - 500, D - w), D - w):
        cut = lambda t: t[:, lo:lo + w].contiguous()
        s, y = cut(old), torch.empty((n, w), dtype=dt, device="cuda")
        ttt.ttt_recur_step(small, cut(X), cut(G), slots, s, y)
        sync_ok()
        assert torch.equal(cut(st), s) and torch.equal(cut(Y), y), lo
    # every column is written
    assert bool((st[2] != old[2]).float().mean() > 0.99) and bool((Y[0].float() != 0).float().mean() > 0.99)


def _calls():
    """One call of each entry point that launches kernels, as a function of the stream."""
    x, w = torch.zeros((64, 64), dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    wide, ww = torch.zeros((64, 2048), dtype=BF, device="cuda"), torch.ones(2048, device="cuda")
    y, yw, y2 = torch.empty_like(x), torch.empty_like(wide), torch.empty_like(x)
    st, hs = torch.zeros(64, device="cuda"), torch.zeros((64, 64), device="cuda")
    n1, n2 = ttt.make_norm_config(1, 1, 64, 64), ttt.make_norm_config(1, 1, 64, 2048)
    r, r1 = ttt.make_recur_config(1, 64, 64), ttt.make_recur_config(64, 1, 64)
    dw, dww = torch.empty_like(w), torch.empty_like(ww)
    nb = max(ttt.ttt_norm_bwd_workspace_bytes(n2), ttt.ttt_linear_workspace_bytes(64, 64, 64, 1),
             ttt.ttt_norm_bwd_workspace_bytes(n1))
    ws = workspace(nb)
    big, bw = torch.zeros((4096, 256), dtype=BF, device="cuda"), torch.zeros((256, 256), dtype=BF, device="cuda")
    by = torch.empty_like(big)
    return dict(
        norm_fwd=lambda s: ttt.ttt_norm_fwd(n1, x, None, w, w, y, stream=s),
        norm_fwd_wide=lambda s: ttt.ttt_norm_fwd(n2, wide, None, ww, ww, yw, stream=s),
        norm_bwd=lambda s: ttt.ttt_norm_bwd(n1, x, w, st, st, x, None, y, dw, None, ws, nb, stream=s),
        norm_bwd_wide=lambda s: ttt.ttt_norm_bwd(n2, wide, ww, st, st, wide, None, yw, dww, None, ws, nb, stream=s),
        recur_fwd=lambda s: ttt.ttt_recur_fwd(r, x, x, None, None, y, stream=s),
        recur_bwd=lambda s: ttt.ttt_recur_bwd(r, x, x, None, None, x, x, None, y, y2, stream=s),
        recur_step=lambda s: ttt.ttt_recur_step(r1, x, x, None, hs, y, stream=s),
        linear_fwd=lambda s: ttt.ttt_linear_fwd(64, 64, 64, "id", x, x, None, None, None, y, stream=s),
        linear_fwd_pair=lambda s: ttt.ttt_linear_fwd(4096, 256, 256, "id", big, bw, None, None, None, by, stream=s),
        linear_bwd=lambda s: ttt.ttt_linear_bwd(64, 64, 64, "id", x, x, None, None, x, y, y2, None, None, ws, nb, stream=s),
        linear_dbias=lambda s: ttt.ttt_linear_bwd(64, 64, 64, "id", None, None, None, None, x, None, None, dw, None, ws, nb,
                                                  stream=s))


def test_a_refused_launch_is_not_the_next_call_s():
    # A synchronisation breaks a capture, and every launch on that stream is refused until it ends.
    # The refusals are reported, and the calls after them, on a sound stream, succeed.
    cu, calls, side = ctypes.CDLL("libcuda.so.1"), _calls(), torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    for f in calls.values():
        f(None)
    sync_ok()
    relaxed = 2
    for name, refused in list(calls.items()) + [("device_error", None)]:
        assert cu.cuStreamBeginCapture_v2(handle, relaxed) == 0
        first = ttt.lib.ttt_get_device_error(handle)
        if refused:
            with pytest.raises(ttt.TTTError) as e:
                refused(side)
            assert e.value.status == ttt.ERR_CUDA, name
        assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
        assert first == ttt.ERR_CUDA
        for after, f in calls.items():
            try:
                f(None)
            except ttt.TTTError as err:
                raise AssertionError(f"{after} after a refused {name}: {err}")
        sync_ok()


# Past 2^31 elements, with small whole numbers in every input: sums of products of them are whole
# and below 2^24, exact in float32 in any order, so that one row too few or twice shows.
def ints(g, *shape, lo=-3, hi=4):
    t = torch.empty(shape, dtype=BF, device="cuda")
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randint(lo, hi, part.shape, generator=g, device="cuda", dtype=torch.int8))
    return t


def test_norm_weight_gradients_past_2_31_elements():
    d, T = 4096, (1 << 19) + 3
    g = rng(21)
    cfg = ttt.make_norm_config(1, 1, T, d)
    S, dY = ints(g, T, d), ints(g, T, d)
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")  # xh = S
    dX, dw, db = torch.empty_like(S), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    n = ttt.ttt_norm_bwd_workspace_bytes(cfg)
    ttt.ttt_norm_bwd(cfg, S, None, mean, rstd, dY, None, dX, dw, db, workspace(n), n)
    sync_ok()
    sw, sb = torch.zeros(d, dtype=F64, device="cuda"), torch.zeros(d, dtype=F64, device="cuda")
    for i in range(0, T, 1 << 15):
        y, s = dY[i:i + (1 << 15)].to(F64), S[i:i + (1 << 15)].to(F64)
        sb += y.sum(0)
        sw += (y * s).sum(0)
    assert torch.equal(db.to(F64), sb) and torch.equal(dw.to(F64), sw)
    for rows in (slice(0, 5), slice(T - 5, T)):
        y, s = dY[rows].to(F64), S[rows].to(F64)
        c1, c2 = y.mean(-1, keepdim=True), (y * s).mean(-1, keepdim=True)  # sums exact, quotients rounded
        assert_within("dX", dX[rows], y - c1 - s * c2, 4 * U32 * (y.abs() + c1.abs() + 2 * (s * c2).abs()))


def test_linear_backward_past_2_31_elements():
    M, N, K = (1 << 17) + 5, 16392, 64
    g = rng(22)
    dY, P, mul, X, W = ints(g, M, N), ints(g, M, N), ints(g, M, N), ints(g, M, K), ints(g, N, K)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dbias, dmul = torch.empty(N, device="cuda"), torch.empty_like(dY)
    n = ttt.ttt_linear_workspace_bytes(M, N, K, 1)
    ttt.ttt_linear_bwd(M, N, K, "id", X, W, P, mul, dY, dX, dW, dbias, dmul, workspace(n), n)
    sync_ok()
    sW, sb = torch.zeros((N, K), dtype=F64, device="cuda"), torch.zeros(N, dtype=F64, device="cuda")
    for i in range(0, M, 1 << 13):
        r = slice(i, i + (1 << 13))
        assert torch.equal(dmul[r], dY[r] * P[r])  # up to 9: exact
        dp = dY[r].to(F64) * mul[r].to(F64)
        sb += dp.sum(0)
        sW += dp.t() @ X[r].to(F64)
        assert torch.equal(dX[r], (dp @ W.to(F64)).to(torch.float32).to(BF)), i
    assert torch.equal(dbias.to(F64), sb)
    assert torch.equal(dW, sW.to(torch.float32).to(BF))


def test_recurrence_gate_gradient_past_2_31_elements():
    # the last tokens, past 32-bit offsets, from the definition: the adjoint starts there
    D, T, n, k = 4096, (1 << 19) + 70, 99, 110  # k: the roundings charged to a token in test_recur.py
    cfg = ttt.make_recur_config(1, T, D)
    draw = lambda seed, mean: torch.empty((T, D), device="cuda", dtype=BF).normal_(mean, 1, generator=rng(seed))
    X, G = draw(1, 0), draw(2, 2)
    H, dX, dG = torch.empty_like(X), torch.empty_like(X), torch.empty_like(X)
    ttt.ttt_recur_fwd(cfg, X, G, None, None, H)
    ttt.ttt_recur_bwd(cfg, X, G, None, None, H, X, None, dX, dG)
    sync_ok()
    carry = torch.zeros(D, dtype=F64, device="cuda")
    err = torch.zeros_like(carry)
    for t in range(T - 1, T - n, -1):
        a, x, dh, prev = torch.sigmoid(G[t].to(F64)), X[t].to(F64), X[t].to(F64), H[t - 1].to(F64)
        na, size = 1 - a, dh.abs() + carry.abs()
        Dt, e = dh + carry, err + 2 * U32 * size
        s = (prev - x) * a * na
        assert_within("dX", dX[t], na * Dt, na * e + 50 * U32 * (na * Dt).abs())
        assert_within("dG", dG[t], Dt * s, e * s.abs() + 100 * U32 * (Dt * s).abs())
        err, carry = a * (e + k * U32 * size), a * Dt
