"""The RMS norm and its backward on arrays of many rows: rows that one block takes in turn (KEEP), arrays that
pass the caches in each of the three ways, with and without a residual, its sum in place of either input,
rows of any length.  Every row is checked, against float64 on the GPU, with the tolerances of test_gpu_block.
"""
import gc

import pytest

from moe_cases import log
from test_gpu_backward import DEPTH, HALF, TORCH, U, blank, code, scratch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5


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


# what launches: vectors a lane, whether a block keeps gamma over its rows, rows of whole vectors or with a
# tail, and how the array passes the caches
CASES = [
    (9001, 512, "bf16", 0, "1 keep whole near"), (9001, 505, "bf16", 1, "1 keep tail near"),
    (8301, 96, "f32", 0, "1 keep whole near"), (8301, 99, "f32", 1, "1 keep tail near"),
    (40001, 512, "bf16", 0, "1 keep whole past"), (40001, 505, "bf16", 3, "1 keep tail past"),
    (20001, 512, "f32", 0, "1 keep whole past"), (20001, 505, "f32", 1, "1 keep tail past"),
    (100003, 512, "bf16", 0, "1 keep whole far"), (101003, 505, "bf16", 1, "1 keep tail far"),
    (50001, 512, "f32", 0, "1 keep whole far"), (50001, 511, "f32", 3, "1 keep tail far"),
    (4200, 1056, "bf16", 0, "2 keep whole near"), (4200, 1053, "bf16", 1, "2 keep tail near"),
    (4200, 1056, "f32", 0, "2 keep whole near"), (4200, 1053, "f32", 0, "2 keep tail near"),
    (4200, 5000, "bf16", 0, "2 keep whole past"), (4200, 5001, "bf16", 5, "2 keep tail past"),
    (2200, 4096, "f32", 0, "2 keep whole past"), (9000, 1001, "f32", 1, "2 keep tail past"),
    (6200, 8192, "bf16", 0, "2 keep whole far"), (6200, 8185, "bf16", 1, "2 keep tail far"),
    (3100, 8192, "f32", 0, "2 keep whole far"), (26000, 1001, "f32", 0, "2 keep tail far"),
    (512, 16384, "f32", 0, "2 each whole near"),
    (1000, 20000, "bf16", 0, "4 each whole past"), (1000, 20001, "bf16", 1, "4 each tail past"),
    (500, 20000, "f32", 0, "4 each whole past"), (500, 20001, "f32", 3, "4 each tail past"),
    (2600, 20000, "bf16", 0, "4 each whole far"), (2600, 20001, "bf16", 0, "4 each tail far"),
    (1300, 20000, "f32", 0, "4 each whole far"), (1300, 20001, "f32", 1, "4 each tail far"),
    (700, 40000, "bf16", 0, "long"), (350, 40003, "f32", 0, "long"),
]
# of the backward pass alone: two vectors a lane
BACKWARD = [(2200, 9000, "bf16", 0), (2200, 9001, "bf16", 1), (1100, 9000, "f32", 0), (1100, 9001, "f32", 1)]


def kind(T, H, dtype):
    """The rules of csrc/rms_norm.hip."""
    size = T * H * (4 if dtype == "f32" else 2)
    if H > 32768:
        return "long"
    nv = 1 if H <= 512 or (T <= 256 and H <= 8192) else 2 if H <= 16384 else 4
    waves = -(-H // (nv * 512))
    rows = 4 if waves == 1 else 1
    keep = nv <= 2 and -(-T // rows) > 2 * 256 * max(1, 16 // (waves * rows))
    how = "near" if size <= 32 << 20 else "past" if size < 96 << 20 else "far"
    return f"{nv} {'keep' if keep else 'each'} {'tail' if H % 8 else 'whole'} {how}"


def rand(g, T, H, dtype, pad, scale=1.0, row=False):
    out = torch.zeros(T * H + pad + 64, dtype=TORCH[dtype], device="cuda")[pad:pad + T * H].view(T, H)
    v = torch.randn(T, H, generator=g, device="cuda") * scale
    return out.copy_(v * (0.5 + torch.rand(T, 1, generator=g, device="cuda")) if row else v)


def near(name, got, ref, tol):
    got = got.double()
    assert got.shape == ref.shape and bool(torch.isfinite(got).all()), name
    worst = float(((got - ref).abs() / tol.clamp(min=1e-300)).max())
    log(f"  {name}: largest error {worst:.3f} of its tolerance")
    assert worst <= 1.0, (name, worst)


def near8(q, s, v, err):
    """8-bit rows against float64 values that the kernel had with errors of at most err."""
    T, H = v.shape
    n = H // 32
    assert not bool(s[:, n:].any())
    e = s[:, :n].double() - 127
    top, slack = v.abs().view(T, n, 32).amax(-1), err.view(T, n, 32).amax(-1)
    assert bool((top - slack <= 448 * torch.exp2(e)).all())
    assert bool(((top + slack > 448 * torch.exp2(e - 1)) | (e == -127)).all())
    scale = torch.exp2(e)[:, :, None]
    got = (q.view(torch.float8_e4m3fn).double().view(T, n, 32) * scale).view(T, H)
    smallest = (2.0 ** -10 * scale).expand(T, n, 32).reshape(T, H)
    near("q", got, v, torch.maximum(2.0 ** -4 * (v.abs() + err), smallest) + err)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def behind(t, n):
    assert torch.isnan(torch.as_strided(t, (32,), (1,), t.storage_offset() + n)).all()   # nothing past the last row


@pytest.mark.parametrize("T,H,dtype,pad,what", CASES)
def test_rms_norm(T, H, dtype, pad, what):
    B = B_()
    assert kind(T, H, dtype) == what
    log(f"case rms norm T={T} H={H} {dtype} pad={pad}: {what}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    x, res = rand(g, T, H, dtype, pad, row=True), rand(g, T, H, dtype, pad, 0.7)
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    mx = H % 32 == 0
    for with_res in (True, False):
        y, total, rstd = blank((T, H), dtype, pad), blank((T, H), dtype, pad), blank((T,))
        q = torch.full((T, H), 0xAA, dtype=torch.uint8, device="cuda") if mx else None
        s = torch.full((T, B.moe_mx_scale_pitch(H)), 0xAA, dtype=torch.uint8, device="cuda") if mx else None
        B.moe_rms_norm(x, res if with_res else None, gamma, T, H, EPS, code(dtype), total if with_res else None, y, q,
                       s, rstd)
        torch.cuda.synchronize()
        v = x
        if with_res:  # one fp32 addition, rounded once
            assert same(total, (x.float() + res.float()).to(TORCH[dtype]))
            v = total
        v = v.double()
        rr = 1 / torch.sqrt(v.square().mean(1) + EPS)
        near("rstd", rstd, rr, (DEPTH + 8) * U * rr)
        ry = v * rr[:, None] * gamma.double()
        err = (DEPTH + 12) * U * ry.abs()
        near("y", y, ry, HALF[dtype] * (ry.abs() + err) + err)
        if mx:
            near8(q, s, ry, err)
        behind(y, T * H)
        if with_res:
            behind(total, T * H)
            for where in (0, 1):  # the sum in place of either input
                pair = [rand(g, T, H, dtype, pad).copy_(t) for t in (x, res)]
                y2 = blank((T, H), dtype, pad)
                B.moe_rms_norm(*pair, gamma, T, H, EPS, code(dtype), pair[where], y2)
                assert same(y, y2) and same(total, pair[where]), where
            y2 = blank((T, H), dtype, pad)
            B.moe_rms_norm(x, res, gamma, T, H, EPS, code(dtype), None, y2)
            assert same(y, y2)


@pytest.mark.parametrize("T,H,dtype,pad", [c[:4] for c in CASES] + BACKWARD)
def test_rms_norm_backward(T, H, dtype, pad):
    B = B_()
    log(f"case rms norm backward T={T} H={H} {dtype} pad={pad}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + 3 * H)
    s = rand(g, T, H, dtype, pad, row=True)
    dy, dsum = rand(g, T, H, dtype, pad, 0.1), rand(g, T, H, dtype, pad, 0.1)
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    sd, dyd = s.double(), dy.double()
    rstd = (1 / torch.sqrt(sd.square().mean(1) + EPS)).float()
    r = rstd.double()[:, None]
    xh, a = sd * r, dyd * gamma.double()
    need = B.moe_rms_norm_backward_workspace_size(T, H)
    base = r * (a - xh * (a * xh).mean(1, keepdim=True))
    f32 = r * (4 * U * a.abs() + (DEPTH + 8) * U * xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    for with_sum in (True, False):
        dx, dg = blank((T, H), dtype, pad), blank((H,))
        B.moe_rms_norm_backward(dy, dsum if with_sum else None, s, gamma, rstd, T, H, code(dtype), dx, dg,
                                scratch(need), need)
        torch.cuda.synchronize()
        ref = base + dsum.double() if with_sum else base
        tol = f32 + 2 * U * ref.abs()
        near("dx", dx, ref, HALF[dtype] * (ref.abs() + tol) + tol)
        near("dgamma", dg, (dyd * xh).sum(0), (DEPTH + T // 256 + 4) * U * (dyd * xh).abs().sum(0))
        behind(dx, T * H)
        if with_sum:  # in place of dsum, and the same bits again
            into, dg2 = rand(g, T, H, dtype, pad).copy_(dsum), blank((H,))
            B.moe_rms_norm_backward(dy, into, s, gamma, rstd, T, H, code(dtype), into, dg2, scratch(need), need)
            assert same(dx, into) and torch.equal(dg, dg2)
