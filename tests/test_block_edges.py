"""The operators around the layer at the ends of their documented ranges: sizes near 2^31, offsets
past it, decays above one, infinities in a row's last columns, calls after a refused one."""
import ctypes

import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import rng, sync_ok, workspace

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
