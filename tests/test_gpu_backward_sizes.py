"""The training pass's calls at T = 2^31 - 1 rows, the most an int holds, and on rows whose elements
lie more than 2^31 elements into their buffers.  Checks and tolerances of ``test_gpu_backward``."""
import numpy as np
import pytest

import test_gpu_backward as base
from moe_cases import log
from oracle import backward as G

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


# 300 rows past element 2^31 of buffers of FAR_ROWS x FAR_H
FAR_H, FAR_ROWS, LAST = 7168, 300000, 300
assert (FAR_ROWS - LAST) * FAR_H > 1 << 31


def far_buffer(rows, dtype, fill=0.0):
    """[FAR_ROWS, FAR_H] on the device, `fill` but for the last rows."""
    t = torch.full((FAR_ROWS, FAR_H), fill, dtype=base.TORCH[dtype], device="cuda")
    if rows is not None:
        t[-LAST:] = base.gpu(rows, dtype)
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_far_into_their_buffers(dtype):
    """The second of two experts, behind 299700 rows of the first."""
    B = base.B_()
    H, I, E, R = FAR_H, 72, 2, FAR_ROWS
    log(f"case experts backward R={R} H={H} I={I} {dtype}")
    rng = np.random.default_rng(31)
    x, dy = (base.host(base.gpu(s * rng.standard_normal((LAST, H)), dtype)) for s in (1.0, 0.2))
    w = rng.standard_normal((E, 3 * H * I)) * H ** -0.5
    w[:, 2 * H * I:] *= (H / I) ** 0.5
    w = base.host(base.gpu(w, dtype))
    wt, slots = base.gpu(w, dtype), base.i32([0, 1])
    offsets = [0, R - LAST, R]
    need = B.moe_grouped_swiglu_backward_workspace_size(R, E, H, I, base.code(dtype))
    ws, dx, dw = base.scratch(need), far_buffer(None, dtype, float("nan")), base.blank((E, 3 * H * I), dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_grouped_swiglu_backward(far_buffer(x, dtype), far_buffer(dy, dtype), base.i32(offsets), R, E, H, I,
                                  base.code(dtype), B.wbuf(wt, 3 * H * I * wt.element_size(), E, E, slots),
                                  ws, need, dx, dw, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert not dx[:-LAST].any() and not dw[0].any()          # of rows that are zero
    inp = dict(x=x, dy=dy, w=w, offsets=[0, LAST], slots=[1])
    base.check_experts((LAST,), H, I, dtype, inp, dx[-LAST:], dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_into_their_buffers(dtype):
    """Layer norm both ways, combine and permute backward on the last of 300000 rows."""
    B = base.B_()
    T, H, half, U, DEPTH = FAR_ROWS, FAR_H, base.HALF[dtype], base.U, base.DEPTH
    log(f"case norm T={T} H={H} {dtype}")
    x, dy, gamma, beta = base.norm_inputs(LAST, H, dtype, 33)
    gt, bt, code = base.gpu(gamma), base.gpu(beta), base.code(dtype)
    xt, y = far_buffer(x, dtype), far_buffer(None, dtype, float("nan"))
    mean, rstd = base.blank((T,)), base.blank((T,))
    B.moe_layer_norm(xt, gt, bt, T, H, 1.0, code, y, mean, rstd)
    torch.cuda.synchronize()
    ry, rmean, rrstd = G.layer_norm(x, gamma, beta, 1.0)
    r = rrstd[:, None]
    mu_err = DEPTH * U * np.abs(x).mean(1, keepdims=True)
    xh = (x - rmean[:, None]) * r
    f32 = np.abs(gamma) * (mu_err * r + (DEPTH + 16) * U * np.abs(xh)) + 4 * U * (np.abs(ry) + np.abs(beta))
    base.check("y", y[-LAST:], ry, half * (np.abs(ry) + f32) + f32)
    assert torch.equal(y[:-LAST], bt.to(y.dtype).expand(T - LAST, H))       # rows of zeros
    m, rs = base.host(mean[-LAST:]), base.host(rstd[-LAST:])
    dx, dg, db = y.fill_(float("nan")), base.blank((H,)), base.blank((H,))
    need = B.moe_layer_norm_backward_workspace_size(T, H)
    B.moe_layer_norm_backward(far_buffer(dy, dtype), xt, gt, mean, rstd, T, H, code, dx, dg, db,
                              base.scratch(need), need)
    torch.cuda.synchronize()
    rdx, rdg, rdb = G.layer_norm_backward(dy, x, gamma, m, rs)
    a, r = np.abs(dy * gamma), rs[:, None]
    xh = np.abs((x - m[:, None]) * r)
    xe = 4 * U * (np.abs(x) + np.abs(m)[:, None]) * r
    av = lambda v: v.mean(1, keepdims=True)
    f32 = r * (4 * U * a + (DEPTH + 4) * U * av(a) + (DEPTH + 8) * U * xh * av(a * xh) + xe * av(a * xh) +
               xh * av(a * xe))
    base.check("dx", dx[-LAST:], rdx, half * (np.abs(rdx) + f32) + f32)
    assert not dx[:-LAST].any()
    # the rows of zeros add nothing: at most the LAST others stand in a chain, and the joins
    chain = DEPTH + LAST
    base.check("dgamma", dg, rdg, chain * U * (np.abs(dy) * xh).sum(0) + (np.abs(dy) * xe).sum(0))
    base.check("dbeta", db, rdb, chain * U * np.abs(dy).sum(0))
    log(f"case combine and permute backward T={T // 2} k=2 H={H} {dtype}")
    T, k = FAR_ROWS // 2, 2
    rng = np.random.default_rng(34)
    # token t's rows are t and T + t: the last tokens' second rows are the last rows
    row_of = torch.stack([torch.arange(T), torch.arange(T) + T], 1).to(torch.int32).cuda()
    n = LAST // 2
    dyo = base.host(base.gpu(rng.standard_normal((n, H)), dtype))
    dyt = torch.zeros((T, H), dtype=base.TORCH[dtype], device="cuda")
    dyt[-n:] = base.gpu(dyo, dtype)
    yp = base.host(base.gpu(rng.standard_normal((LAST, H))))
    w = torch.full((T, k), 0.5, device="cuda")
    dw = base.blank((T, k))
    dyp = dx.fill_(float("nan"))
    B.moe_combine_backward(dyt, code, far_buffer(yp, "f32"), row_of, w, T, k, H, code, dyp, dw)
    torch.cuda.synchronize()
    assert torch.equal(dyp[T:], dyp[:T]) and not dyp[T:-n].any()
    base.check("dy_perm", dyp[-n:], 0.5 * dyo, (half + 2 * U) * np.abs(0.5 * dyo))
    ref, size = (dyo * yp[-n:]).sum(1), np.abs(dyo * yp[-n:]).sum(1)
    base.check("dtopk_w", dw[-n:, 1], ref, DEPTH * U * size)
    assert not dw[:, 0].any() and not dw[:-n].any()
    B.moe_permute_backward(dyp, row_of, T, k, H, code, dyt)
    torch.cuda.synchronize()
    assert not dyt[:-n].any() and torch.equal(dyt[-n:], base.gpu(dyo, dtype))       # 0.5 dy + 0.5 dy
