"""8-bit products whose scales are the smallest there are, bytes 0 to 3 (2^-127 to 2^-124), in rows or in
weights, against float64; and what the largest bytes give.

With f32 outputs the values are expanded to bf16, whose subnormals have steps of 2^-133: with scale byte b an
element, a multiple of 2^(b - 136), is off by at most half a step where b < 3, and exact from 3 on.
"""
import pytest

from moe_cases import log
from test_gpu_backward import HALF, TORCH, U, i32
from test_gpu_grouped_gemm_sizes import Operands, near
from test_gpu_grouped_gemm_tiles import largest_of_eight

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("side", ["rows", "weights"])
@pytest.mark.parametrize("low", [0, 1, 2, 3])
@pytest.mark.parametrize("counts,N", [((5, 40), 72), ((300, 77, 200), 2056)])
def test_product(counts, N, low, side, out):
    E, R, K = len(counts), sum(counts), 544
    log(f"case rows={counts} K={K} N={N} scale byte {low} in the {side} -> {out}")
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    o = Operands("mx", R, K, N, E, 3 + low)
    if side == "rows":
        o.xs[:, :K // 32] = low
        for e in range(E):
            o.w[e, N * K:].view(N, -1)[:, :K // 32] += 115               # 2^105 to 2^109: products near 1
    else:
        o.xs[:, :K // 32] += 115
        for e in range(E):
            o.w[e, N * K:].view(N, -1)[:, :K // 32] = low
    buf, offsets = o.buffer(range(E)), i32(off)
    y = torch.full((R, N), float("nan"), dtype=TORCH[out], device="cuda")
    o.product(offsets, buf, out, y)
    step = 2.0 ** -134 if low < 3 and out == "f32" else 0.0
    for e in range(E):
        at = slice(off[e], off[e + 1])
        x, w = o.rows(slice(off[e], off[e + 1])), o.weights(e)
        ref, f32 = x @ w.t(), K * U * (x.abs() @ w.abs().t())
        f32 = f32 + step * (w.abs().sum(1)[None, :] if side == "rows" else x.abs().sum(1)[:, None])
        if out == "bf16":
            f32 = f32 + 7 * 2.0 ** -13 * largest_of_eight(x, w)
        near(f"y of expert {e}", y[at], ref, HALF[out] * (ref.abs() + f32) + f32)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N", [((5, 40), 72), ((300, 77, 200), 2056)])
def test_the_largest_bytes(counts, N, out):
    """254 is 2^127 and 255 NaN, also of a block of zeros, for its row alone."""
    off, K = [0], 64
    for c in counts:
        off.append(off[-1] + c)
    o = Operands("mx", off[-1], K, N, len(counts), 1)
    o.x.fill_(0x38)                                                     # ones
    o.xs[:, :2] = 127
    o.w[:, :N * K] = 0x38
    for e in range(len(counts)):
        o.w[e, N * K:].view(N, -1)[:, :2] = 127
    o.x[1, 1:32], o.xs[1, 0] = 0, 254                                   # 2^127 once
    o.xs[2, 1] = 255
    o.x[3, :32], o.xs[3, 0] = 0, 255
    y = torch.zeros(off[-1], N, dtype=TORCH[out], device="cuda")
    o.product(i32(off), o.buffer(range(len(counts))), out, y)
    assert bool((y[1].double() == 2.0 ** 127).all())
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    rest = [r for r in range(off[-1]) if r not in (1, 2, 3)]
    assert bool((y[rest] == 64).all())
