"""The layer's training step on the GPU where the caller takes part in it."""
import pytest

import test_gpu_backward as base
from moe_cases import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
_free_gpu = base._free_gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("remote", ["all", "device", "routed"])
def test_rows_that_the_caller_normed_reach_the_experts(dtype, remote):
    """forward(normed=True) takes xn, mean and rstd as they are: here rows twice the norm's, which no
    norm of x gives, and statistics that are recognised again."""
    cfg, L, _ = base.layer_case(dtype, True)
    log(f"case normed rows {dtype} remote={remote}")
    try:
        torch.cuda.synchronize()
        with torch.cuda.stream(L.compute_stream):
            L.norm()
            L.xn.mul_(2.0)                       # exact in both types
            rows = L.xn.clone()
            L.mean.fill_(5.0)
            L.rstd.fill_(7.0)
            L.forward(remote=remote, normed=True)
        assert L.read_status() == 0
        assert torch.equal(L.xn, rows)
        assert torch.equal(L.x_perm, rows[(L.src_of // cfg.k).long()])
        assert (L.mean == 5.0).all() and (L.rstd == 7.0).all()
    finally:
        L.close()
