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
