"""The operators around the layer at the ends of their documented ranges: sizes near 2^31, offsets
past it, decays above one, infinities in a row's last columns, calls after a refused one."""
import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import rng, sync_ok

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
