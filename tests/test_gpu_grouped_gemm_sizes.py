"""The products by expert on sizes near what a launch takes: many experts beside few rows, millions of rows, the
longest sides, every row that an int counts.  Values are drawn on the GPU and checked there in float64 with the
tolerances of test_gpu_grouped_gemm, on chosen rows and all of their columns.
"""
import gc

import numpy as np
import pytest

from moe_cases import log
from test_gpu_backward import HALF, TORCH, U, code, i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _free_gpu():
    yield
    gc.collect()
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()


def B_():
    from grouped_gemm_weights_amd import binding
    return binding


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"{gb} GB of device memory are not free")


def near(name, got, ref, tol):
    got = got.double()
    assert got.shape == ref.shape and bool(torch.isfinite(got).all()), name
    worst = float(((got - ref).abs() / tol.clamp(min=1e-300)).max())
    log(f"  {name}: largest error {worst:.3f} of its tolerance")
    assert worst <= 1.0, (name, worst)


def decode(q, s):
    """8-bit rows on the GPU as float64."""
    e = s[:, :q.shape[1] // 32].double() - 127
    return (q.view(torch.float8_e4m3fn).double().view(q.shape[0], -1, 32) * torch.exp2(e)[:, :, None]).view(q.shape)


class Operands:
    """Rows and weights of one type, drawn on the GPU; x[r] and w[slot] give float64 values."""

    def __init__(self, dtype, R, K, N, slots, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dtype, self.K, self.N = dtype, K, N
        if dtype == "mx":
            pitch = B_().moe_mx_scale_pitch(K)

            def rows(n):
                q = torch.randint(0, 127, (n, K), generator=g, device="cuda", dtype=torch.uint8)   # no NaN
                q |= torch.randint(0, 2, (n, K), generator=g, device="cuda", dtype=torch.uint8) << 7
                s = torch.zeros(n, pitch, dtype=torch.uint8, device="cuda")
                s[:, :K // 32] = torch.randint(117, 122, (n, K // 32), generator=g, device="cuda", dtype=torch.uint8)
                return q, s

            self.x, self.xs = rows(R)
            self.block = N * (K + pitch)
            self.w = torch.empty(slots, self.block, dtype=torch.uint8, device="cuda")
            for e in range(slots):
                q, s = rows(N)
                self.w[e, :N * K], self.w[e, N * K:] = q.view(-1), s.view(-1)
        else:
            t = TORCH[dtype]
            self.x = torch.randn(R, K, generator=g, device="cuda", dtype=t)
            self.w = torch.randn(slots, N * K, generator=g, device="cuda", dtype=t) * K ** -0.5
            self.block = N * K * self.w.element_size()

    def buffer(self, slot_of):
        self.slot_of = i32(slot_of)                                     # the buffer holds its address alone
        return B_().wbuf(self.w, self.block, self.w.shape[0], len(slot_of), self.slot_of)

    def rows(self, at):
        return decode(self.x[at], self.xs[at]) if self.dtype == "mx" else self.x[at].double()

    def weights(self, slot):
        w, n = self.w[slot], self.N * self.K
        if self.dtype == "mx":
            return decode(w[:n].view(self.N, self.K), w[n:].view(self.N, -1))
        return w.double().view(self.N, self.K)

    def product(self, offsets, buf, out, y):
        B = B_()
        R, E = self.x.shape[0], offsets.numel() - 1
        if self.dtype == "mx":
            B.moe_grouped_gemm_mx(self.x, self.xs, None, 0, offsets, R, E, self.K, self.N, buf, 0, self.N * self.K,
                                  code(out), y)
        else:
            B.moe_grouped_gemm(self.x, None, 0, offsets, R, E, self.K, self.N, code(self.dtype), buf, 0, code(out), y)
        torch.cuda.synchronize()

    def check(self, at, slot, out, y):
        """Rows `at` of y, which belong to one expert."""
        x, w = self.rows(at), self.weights(slot)
        ref, size = x @ w.t(), x.abs() @ w.abs().t()
        f32 = self.K * U * size
        if self.dtype == "mx" and out == "bf16":
            # the sum over eights of the largest product is at most the sum of all of them
            f32 = f32 + 7 * 2.0 ** -13 * size
        near(f"y of {len(at)} rows", y[at], ref, HALF[out] * (ref.abs() + f32) + f32)


def some(lo, hi, n=40):
    """Rows at both ends of [lo, hi), at borders of tiles, and some between."""
    rng = np.random.default_rng(hi)
    at = {*range(lo, min(lo + 5, hi)), *range(max(lo, hi - 5), hi), *(int(r) for r in rng.integers(lo, hi, n))}
    at |= {r for t in (64, 256) for r in (lo + t - 1, lo + t) if r < hi}
    return torch.tensor(sorted(at), device="cuda")


@pytest.mark.parametrize("dtype,out", [("mx", "bf16"), ("mx", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_few_rows_of_1024_experts(dtype, out):
    """A decode step with every expert of the largest set listed: 4096 x 4096 matrices, two slots."""
    B = B_()
    E, K, N = 1024, 4096, 4096
    counts = np.zeros(E, np.int32)
    counts[[0, 63, 64, 65, 500, 1022, 1023]] = [1, 3, 1, 33, 2, 70, 1]
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    log(f"case {dtype} -> {out}: {R} rows of {E} experts of {K} x {N}")
    o = Operands(dtype, R, K, N, 2, 5)
    buf = o.buffer(np.arange(E) % 2)
    y = torch.full((R, N), float("nan"), dtype=TORCH[out], device="cuda")
    o.product(i32(off), buf, out, y)
    for e in np.flatnonzero(counts):
        o.check(torch.arange(int(off[e]), int(off[e + 1]), device="cuda"), int(e) % 2, out, y)
    if dtype != "mx":
        dy = torch.randn(R, N, device="cuda").to(TORCH[dtype])
        dx = torch.full_like(o.x, float("nan"))
        B.moe_grouped_gemm_backward(o.x, dy, i32(off), R, E, K, N, code(dtype), buf, 0, dx, None)
        torch.cuda.synchronize()
        for e in np.flatnonzero(counts):
            at, w = slice(int(off[e]), int(off[e + 1])), o.weights(int(e) % 2)
            d = dy[at].double()
            ref, f32 = d @ w, N * U * (d.abs() @ w.abs())
            near(f"dx of expert {e}", dx[at], ref, HALF[dtype] * (ref.abs() + f32) + f32)


@pytest.mark.parametrize("dtype,out", [("mx", "bf16"), ("mx", "f32"), ("bf16", "bf16")])
def test_two_million_rows(dtype, out):
    """2^21 rows of 8 experts, 4096 columns."""
    B = B_()
    need(60)
    R, E, K, N = 1 << 21, 8, 64, 4096
    off = [0, 0, 300, 300_000, 300_001, 1_000_000, 1_000_255, 2_000_000, R]
    log(f"case {dtype} -> {out}: {R} rows of {E} experts of {K} x {N}")
    o = Operands(dtype, R, K, N, E, 6)
    buf = o.buffer(np.arange(E))
    y = torch.full((R, N), float("nan"), dtype=TORCH[out], device="cuda")
    o.product(i32(off), buf, out, y)
    for e in range(1, E):
        o.check(some(off[e], off[e + 1]), e, out, y)


def test_gradients_of_two_million_rows():
    B = B_()
    need(60)
    R, E, K, N = 1 << 21, 8, 4096, 64
    off = [0, 0, 300, 300_000, 300_001, 1_000_000, 1_000_255, 2_000_000, R]
    log(f"case gradients of {R} rows of {E} experts of {K} x {N}")
    o = Operands("bf16", R, K, N, E, 7)
    buf = o.buffer(np.arange(E))
    dy = torch.randn(R, N, device="cuda", dtype=torch.bfloat16)
    dx, dw = torch.full_like(o.x, float("nan")), torch.full_like(o.w, float("nan"))
    B.moe_grouped_gemm_backward(o.x, dy, i32(off), R, E, K, N, B.MOE_BF16, buf, 0, dx, dw)
    torch.cuda.synchronize()
    assert not dw[0].any()
    half = HALF["bf16"]
    for e in range(1, E):
        at, w = some(off[e], off[e + 1]), o.weights(e)
        d = dy[at].double()
        ref, f32 = d @ w, N * U * (d.abs() @ w.abs())
        near(f"dx of expert {e}", dx[at], ref, half * (ref.abs() + f32) + f32)
        n = off[e + 1] - off[e]
        ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        for lo in range(off[e], off[e + 1], 100_000):
            part = slice(lo, min(lo + 100_000, off[e + 1]))
            a, b = dy[part].double(), o.x[part].double()
            ref += a.t() @ b
            size += a.abs().t() @ b.abs()
        f32 = n * U * size
        near(f"dw of expert {e}", dw[e].view(N, K), ref, half * (ref.abs() + f32) + f32)


@pytest.mark.parametrize("dtype,out", [("mx", "bf16"), ("mx", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("K,N", [(32, 2 ** 20), (2 ** 20, 8)])
def test_8000_rows_of_the_longest_sides(K, N, dtype, out):
    B = B_()
    need(120)
    R, E = 8000, 16
    off = [0, 1, 33, 33, 100, 700, 701, 1300, 1301, 1302, 1400, 3000, 3256, 3512, 3513, 7000, R]
    log(f"case {dtype} -> {out}: {R} rows of {E} experts of {K} x {N}")
    o = Operands(dtype, R, K, N, 3, 8)
    buf = o.buffer(np.arange(E) % 3)
    y = torch.full((R, N), float("nan"), dtype=TORCH[out], device="cuda")
    o.product(i32(off), buf, out, y)
    for e in (0, 1, 4, 9, 14, 15):
        o.check(some(off[e], off[e + 1], 6), e % 3, out, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weight_gradients_of_600_wide_experts(dtype):
    """dW alone, 2^20 columns: experts with a few rows, and zeros for all others."""
    B = B_()
    need(60)
    E, K, N = 600, 2 ** 20, 8
    counts = np.zeros(E, np.int32)
    counts[[0, 7, 300, 599]] = [2, 1, 4, 2]
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    log(f"case dW of {E} experts of {K} x {N} {dtype}")
    x, dy = (torch.randn(R, n, device="cuda").to(TORCH[dtype]) for n in (K, N))
    w = torch.empty(E, N * K, dtype=TORCH[dtype], device="cuda")
    dw = torch.full_like(w, float("nan"))
    slot_of = i32(np.arange(E)[::-1].copy())
    buf = B.wbuf(w, N * K * w.element_size(), E, E, slot_of)
    B.moe_grouped_gemm_backward(x, dy, i32(off), R, E, K, N, code(dtype), buf, 0, None, dw)
    torch.cuda.synchronize()
    for e in range(E):
        got = dw[E - 1 - e]
        if counts[e] == 0:
            assert not bool(got.any()), e
            continue
        a, b = dy[int(off[e]):int(off[e + 1])].double(), x[int(off[e]):int(off[e + 1])].double()
        ref, f32 = a.t() @ b, int(counts[e]) * U * (a.abs().t() @ b.abs())
        near(f"dw of expert {e}", got.view(N, K), ref, HALF[dtype] * (ref.abs() + f32) + f32)


def test_every_row_that_an_int_counts():
    """2^31 - 1 rows, nearly all of them one expert's: its tiles are counted without passing 32 bits."""
    B = B_()
    need(90)
    R, K, N = 2 ** 31 - 1, 8, 8
    log(f"case bf16: {R} rows of {K} x {N}")
    o = Operands("bf16", 1, K, N, 2, 9)
    o.x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    live = [slice(0, 300), slice(2 ** 30 - 5, 2 ** 30 + 300), slice(R - 300, R)]
    for part in live:
        o.x[part] = torch.randn(part.stop - part.start, K, device="cuda").to(torch.bfloat16)
    y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf = o.buffer([1, 0])
    o.product(i32([0, 5, R]), buf, "bf16", y)
    o.check(torch.arange(5, device="cuda"), 1, "bf16", y)
    for part in live:
        o.check(torch.arange(max(part.start, 5), part.stop, device="cuda"), 0, "bf16", y)
    for lo, hi in ((300, 2 ** 30 - 5), (2 ** 30 + 300, R - 300)):
        for at in range(lo, hi, 2 ** 27):
            assert not bool(y[at:min(at + 2 ** 27, hi)].any()), at      # rows of zeros: every one written
