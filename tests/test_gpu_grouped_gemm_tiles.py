"""The tiles of 64 x 256 and of 256 x 256 that the products by expert run on where there are many: every number
of rows that a tile has a mode for, depths that end after one, two, three or four of the loop's half stages,
both outputs, gathered or not.  Sizes come from the rule that chooses the tiles, which is stated here again.

Values are drawn on the GPU and checked there in float64 with the tolerances of test_gpu_grouped_gemm.
"""
import pytest

from moe_cases import log
from test_gpu_backward import HALF, TORCH, U, code, i32
from test_gpu_grouped_gemm_sizes import Operands, near

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

N = 2056
# tiles of up to 32 and of up to 64 rows, some of them an expert's last; a row count without any
SOME = (1, 33, 64, 65, 32, 0, 200, 105)
# tiles of 256 rows, of more than 192, 128, 64 and 32, and of fewer
MANY = (266, 200, 150, 129, 100, 64, 33, 32, 1, 0, 400)
DEPTHS = [("mx", K) for K in (32, 96, 160, 224, 416, 544, 608, 736, 1408)] + \
         [("bf16", K) for K in (8, 40, 72, 104, 264, 328, 360, 424, 704)]


def tiles(R, E):
    """The rule of csrc/grouped_gemm.hip for products of N columns."""
    small = -(-R // 64) + min(E, R)
    if small * -(-N // 64) <= 512:
        return "split"
    return 64 if small * -(-N // 256) <= 256 else 256


def halves(dtype, K):
    """Half stages of 64 bytes of a row, of which the loop takes four a turn."""
    return -(-K * (2 if dtype == "bf16" else 1) // 64)


def largest_of_eight(x, w):
    """sum over groups of eight consecutive k of max|x_k w_k| for each row of x and of w."""
    x, w = x.abs().float(), w.abs().float()
    total = torch.zeros(x.shape[0], w.shape[0], device="cuda", dtype=torch.float64)
    for k in range(0, x.shape[1], 8):
        top = x[:, k, None] * w[None, :, k]
        for i in range(k + 1, k + 8):
            top = torch.maximum(top, x[:, i, None] * w[None, :, i])
        total += top
    return total


def test_depths_end_everywhere():
    for dtype in ("mx", "bf16"):
        assert {halves(d, K) % 4 for d, K in DEPTHS if d == dtype} == {0, 1, 2, 3}


@pytest.mark.parametrize("gather", [0, 3])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dtype,K", DEPTHS)
@pytest.mark.parametrize("counts,kind", [(SOME, 64), (MANY, 256)])
def test_product(counts, kind, dtype, K, out, gather):
    from grouped_gemm_weights_amd import binding as B
    E, live = len(counts), sum(counts)
    R = live + 9                                                        # rows behind the last expert's
    assert tiles(R, E) == kind
    log(f"case {dtype} -> {out}: tiles of {kind} rows, K={K}, {halves(dtype, K) % 4} halves in the last turn, "
        f"gather={gather}")
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    o = Operands(dtype, -(-R // gather) if gather else R, K, N, 3, K + kind)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    n_x = o.x.shape[0]
    src = torch.randint(0, n_x * gather, (R,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    row = torch.div(src.long(), gather, rounding_mode="floor") if gather else torch.arange(R, device="cuda")
    slots = [e % 3 for e in range(E)]
    buf, offsets, status = o.buffer(slots), i32(off), i32([0])
    y, again = (torch.full((R, N), float("nan"), dtype=TORCH[out], device="cuda") for _ in range(2))
    for to in (y, again):
        if dtype == "mx":
            B.moe_grouped_gemm_mx(o.x, o.xs, src, gather, offsets, R, E, K, N, buf, 0, N * K, code(out), to, status)
        else:
            B.moe_grouped_gemm(o.x, src, gather, offsets, R, E, K, N, code(dtype), buf, 0, code(out), to, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(y.view(torch.uint8), again.view(torch.uint8)) and torch.isnan(y[live:]).all()
    for e, c in enumerate(counts):
        if c == 0:
            continue
        at = slice(off[e], off[e + 1])
        x, w = o.rows(row[at]), o.weights(slots[e])
        ref, f32 = x @ w.t(), K * U * (x.abs() @ w.abs().t())
        if dtype == "mx" and out == "bf16":
            f32 = f32 + 7 * 2.0 ** -13 * largest_of_eight(x, w)
        near(f"y of expert {e} ({c} rows)", y[at], ref, HALF[out] * (ref.abs() + f32) + f32)
