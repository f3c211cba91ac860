"""What the loss takes of memory: nothing for rows that are read as they lie, and results that do not depend
on the room."""
import pytest
import torch

from state_space_sequence_gb300 import dlr, xent

pytestmark = pytest.mark.gpu


def taken(call):
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    torch.cuda.synchronize()
    return torch.cuda.max_memory_allocated() - before, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_few_rows_take_little(dtype):
    M, V, D = 16, 30000, 512
    g = torch.Generator().manual_seed(1)
    W = (torch.randn(V, D, generator=g) / 8).to(dtype).cuda()
    h = torch.randn(M, D, generator=g).to(dtype).cuda()
    target = torch.randint(0, V, (M,), generator=g).cuda()
    dloss = torch.ones(M, device="cuda")
    n, (loss, lse) = taken(lambda: xent.xent_loss(h, W, target))
    assert n < 1 << 20  # W has 31 MB
    n, (dh, dW) = taken(lambda: xent.xent_loss_backward(h, W, target, lse, dloss, wanted=(True, False)))
    assert n < 8 << 20  # d and its products' sums
    # and a call whose W is off 16 bytes is given the room: the same results
    big = torch.zeros(V, D + 1, dtype=dtype, device="cuda")
    off = big[:, 1:]
    off.copy_(W)
    n, (loss2, lse2) = taken(lambda: xent.xent_loss(h, off, target))
    assert n > 2 * V * D
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dh2, _ = xent.xent_loss_backward(h, off, target, lse, dloss, wanted=(True, False))
    assert torch.equal(dh, dh2)
    assert dlr.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_a_workspace_for_these_rows(dtype):
    """The sizes that are asked for with the rows are enough, whatever is in them."""
    M, V, D = 70, 1000, 72
    g = torch.Generator().manual_seed(2)
    dloss = torch.rand(M, generator=g).cuda()
    target = torch.randint(0, V, (M,), generator=g).cuda()
    for first in (0, 1):
        rows = [(torch.randn(n, D + 8, generator=g) / 8).to(dtype).cuda()[:, first:first + D] for n in (M, V)]
        h, W = rows
        loss, lse = xent.xent_loss(h, W, target)
        dh, dW = xent.xent_loss_backward(h, W, target, lse, dloss)
        n = xent.xent_loss_workspace_size(dtype, M, V, D, h, W)
        m = xent.xent_loss_backward_workspace_size(dtype, M, V, D, W)
        there = first == 0 and dtype != torch.float32
        assert (n < xent.xent_loss_workspace_size(dtype, M, V, D)) == there
        assert (m < xent.xent_loss_backward_workspace_size(dtype, M, V, D)) == there
        a, b = (torch.full((k + 256,), 255, dtype=torch.uint8, device="cuda") for k in (n, m))
        x = xent.xent_loss(h, W, target, workspace=a[:n])
        y = xent.xent_loss_backward(h, W, target, lse, dloss, workspace=b[:m])
        for p, q in zip((loss, lse, dh, dW), (*x, *y)):
            assert torch.equal(p, q)
        assert (a[n:] == 255).all() and (b[m:] == 255).all()
        with pytest.raises(dlr.DLRError):
            xent.xent_loss(h, W, target, workspace=a[:n - 1])
        with pytest.raises(dlr.DLRError):
            xent.xent_loss_backward(h, W, target, lse, dloss, workspace=b[:m - 1])
    assert dlr.device_status() == 0
