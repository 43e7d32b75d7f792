"""Batches that are padded: rows behind the last expert's and the rows of other experts hold NaN, which must not
reach a gradient, also where an expert's rows end inside the depth that a tile takes at a time.
"""
import numpy as np
import pytest

from moe_cases import log
from test_gpu_backward import HALF, TORCH, U, code, i32
from test_gpu_grouped_gemm_sizes import near

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("want", ["xw", "x", "w"])
@pytest.mark.parametrize("counts,K,N", [((20, 7, 0, 33), 72, 40), ((300, 1, 255, 0, 31), 264, 136),
                                        ((700, 511, 3, 900), 1032, 1544)])
def test_gradients(counts, K, N, want, dtype):
    """The first expert's rows and those behind the last are NaN."""
    from grouped_gemm_weights_amd import binding as B
    E, live = len(counts), sum(counts)
    R = live + 37
    log(f"case rows={counts} K={K} N={N} {dtype} {want}")
    off = np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    t = TORCH[dtype]
    x, dy = (torch.randn(R, n, generator=g, device="cuda").to(t) for n in (K, N))
    for v in (x, dy):
        v[:counts[0]] = float("nan")
        v[live:] = float("nan")
    w = (torch.randn(E, N * K, generator=g, device="cuda") * K ** -0.5).to(t)
    slots, offsets, status = i32(np.arange(E)), i32(off), i32([0])
    buf = B.wbuf(w, N * K * w.element_size(), E, E, slots)
    mark = 7.0
    dx = torch.full_like(x, mark) if "x" in want else None
    dw = torch.full_like(w, mark) if "w" in want else None
    B.moe_grouped_gemm_backward(x, dy, offsets, R, E, K, N, code(dtype), buf, 0, dx, dw, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    half = HALF[dtype]
    if dx is not None:
        assert torch.isnan(dx[:counts[0]]).all() and bool((dx[live:] == mark).all())
    if dw is not None:
        assert torch.isnan(dw[0]).all()
    for e in range(1, E):
        at = slice(int(off[e]), int(off[e + 1]))
        a, b, m = dy[at].double(), x[at].double(), w[e].double().view(N, K)
        if dx is not None and counts[e]:
            ref, f32 = a @ m, N * U * (a.abs() @ m.abs())
            near(f"dx of expert {e}", dx[at], ref, half * (ref.abs() + f32) + f32)
        if dw is not None:
            ref, f32 = a.t() @ b, counts[e] * U * (a.abs().t() @ b.abs())
            near(f"dw of expert {e}", dw[e].view(N, K), ref, half * (ref.abs() + f32) + f32)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts,N", [((20, 7, 0, 33), 40), ((300, 1, 255, 0, 31), 2056), ((700, 511, 3, 900), 1544)])
def test_products(counts, N, dtype, out):
    from grouped_gemm_weights_amd import binding as B
    E, live, K = len(counts), sum(counts), 264
    R = live + 37
    log(f"case rows={counts} K={K} N={N} {dtype} -> {out}")
    off = np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    t = TORCH[dtype]
    x = torch.randn(R, K, generator=g, device="cuda").to(t)
    x[:counts[0]] = float("nan")
    x[live:] = float("nan")
    w = (torch.randn(E, N * K, generator=g, device="cuda") * K ** -0.5).to(t)
    slots, offsets = i32(np.arange(E)), i32(off)
    y = torch.full((R, N), 7.0, dtype=TORCH[out], device="cuda")
    B.moe_grouped_gemm(x, None, 0, offsets, R, E, K, N, code(dtype), B.wbuf(w, N * K * w.element_size(), E, E, slots), 0,
                       code(out), y)
    torch.cuda.synchronize()
    assert torch.isnan(y[:counts[0]]).all() and bool((y[live:] == 7.0).all())
    for e in range(1, E):
        at = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            a, m = x[at].double(), w[e].double().view(N, K)
            ref, f32 = a @ m.t(), K * U * (a.abs() @ m.abs().t())
            near(f"y of expert {e}", y[at], ref, HALF[out] * (ref.abs() + f32) + f32)
