"""The training pass's calls at T = 2^31 - 1 rows, the most an int holds."""
import pytest

import test_gpu_backward as base
from moe_cases import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
_free_gpu = base._free_gpu

T = (1 << 31) - 1
BF16 = dict(dtype=torch.bfloat16, device="cuda")


def test_layer_norm_of_the_most_rows():
    """Rows of one element: y = beta, dx = 0, dgamma = 0, dbeta = sum dy."""
    B = base.B_()
    log(f"case layer norm T={T} H=1 bf16")
    x = torch.full((T, 1), 3.0, **BF16)
    y = torch.zeros((T, 1), **BF16)
    gamma, beta = base.gpu([2.0]), base.gpu([0.5])
    mean, rstd = (torch.zeros((T,), dtype=torch.float32, device="cuda") for _ in range(2))
    B.moe_layer_norm(x, gamma, beta, T, 1, 1.0, B.MOE_BF16, y, mean, rstd)
    torch.cuda.synchronize()
    assert bool((y == 0.5).all()) and bool((mean == 3.0).all()) and bool((rstd == 1.0).all())
    log(f"case layer norm backward T={T} H=1 bf16")
    dy = y.fill_(1.0)
    dx = torch.full((T, 1), float("nan"), **BF16)
    dg, db = base.blank((1,)), base.blank((1,))
    need = B.moe_layer_norm_backward_workspace_size(T, 1)
    B.moe_layer_norm_backward(dy, x, gamma, mean, rstd, T, 1, B.MOE_BF16, dx, dg, db, base.scratch(need), need)
    torch.cuda.synchronize()
    assert not bool(dx.any()) and dg.item() == 0
    # a workgroup's rows are counted exactly (fewer than 2^24 ones); the workgroups' sums are joined in
    # fewer than 64 additions, each off by half a step
    assert abs(db.item() - T) <= 64 * base.U * T


def test_permute_backward_of_the_most_rows():
    B = base.B_()
    log(f"case permute backward T={T} k=1 H=1 bf16")
    d = torch.arange(T, dtype=torch.int32, device="cuda").bitwise_and_(255).to(torch.bfloat16)  # exact
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    dx = torch.full((T,), float("nan"), **BF16)
    B.moe_permute_backward(d, rows, T, 1, 1, B.MOE_BF16, dx)
    torch.cuda.synchronize()
    assert torch.equal(dx.flip(0), d)
