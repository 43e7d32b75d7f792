"""The RMS norm with the residual's addition, the 8-bit quantisation and dropout on the GPU against
``oracle.block`` in float64, through the C ABI, element by element.

Tolerances, derived per element (u = 2^-24, half an fp32 step; HALF[dtype] half a step of the stored
type: 2^-8 for bf16, 2^-24 for f32):

* a chain of n fp32 additions of terms t_i is off by at most n u sum|t_i|.  The row sums of the norm run
  at most DEPTH = 64 additions deep (8 elements of at most 4 vectors a lane, 6 steps across the wave, 16
  waves, and the few sweeps of the longest rows here).
* an output stored in dtype is off by HALF[dtype] |value| more.
* e4m3 holds four significant bits, so a rounding is off by at most 2^-4 of the value, or by half a
  step of the smallest ones, 2^-10 of the block's scale.  Scaling by a power of two rounds nothing.
"""
import gc

import numpy as np
import pytest

from moe_cases import log
from oracle import block as K
from test_gpu_backward import DEPTH, HALF, TORCH, U, blank, check, code, gpu, host, scratch

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


def bytes8(rows, cols, fill=0xAA):
    """q and scales with 64 guard bytes behind each."""
    q = torch.full((rows * cols + 64,), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * K.pitch(cols) + 64,), fill, dtype=torch.uint8, device="cuda")
    return q, s


def unpack8(q, s, rows, cols, fill=0xAA):
    q, s = q.cpu().numpy(), s.cpu().numpy()
    p = K.pitch(cols)
    assert (q[rows * cols:] == fill).all() and (s[rows * p:] == fill).all()      # nothing behind the last row
    q, s = q[:rows * cols].reshape(rows, cols), s[:rows * p].reshape(rows, p)
    assert not s[:, cols // 32:].any()                                          # the padding
    return q, s


def check8(name, q, s, v, err):
    """8-bit rows against float64 values that the GPU had with errors of at most err."""
    n = v.shape[1] // 32
    e = s[:, :n].astype(np.float64) - 127
    top = np.abs(v).reshape(v.shape[0], n, 32).max(-1)
    slack = err.reshape(v.shape[0], n, 32).max(-1)
    assert (top - slack <= 448 * 2.0 ** e).all(), name
    assert ((top + slack > 448 * 2.0 ** (e - 1)) | (e == -127)).all(), name
    scale = np.repeat(2.0 ** e, 32, axis=1)
    tol = np.maximum(2.0 ** -4 * (np.abs(v) + err), 2.0 ** -10 * scale) + err
    check(name, K.decode(q, s), v, tol)


# ----------------------------------------------------------------------------
# quantisation
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (1, 32, "bf16", 0), (1, 32, "f32", 1), (3, 64, "bf16", 3), (5, 480, "f32", 0), (2, 512, "bf16", 0),
    (7, 544, "bf16", 1), (33, 1408, "bf16", 0), (4, 7168, "bf16", 0), (1000, 96, "f32", 3), (0, 64, "bf16", 0),
    (3, 20000 // 32 * 32, "bf16", 0), (70001, 32, "bf16", 0)])
def test_quantize(rows, cols, dtype, pad):
    """As they are: every byte."""
    B = B_()
    log(f"case quantize rows={rows} cols={cols} {dtype} pad={pad}")
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-12, 12, (rows, 1))
    if rows:
        x[0, :32] = 0
        x[-1, -1] = 448.0                                   # a value on the border of two scales
        x[rows // 2, 7] = -449.0 if dtype == "f32" else -450.0
    x = host(gpu(x, dtype))
    q, s = bytes8(rows, cols)
    B.moe_mx_quantize(gpu(x, dtype, pad), rows, cols, code(dtype), 0, q, s)
    torch.cuda.synchronize()
    q, s = unpack8(q, s, rows, cols)
    rq, rs = K.quantize(x)
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(K.e4m3_values()[q], rq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_borders_and_what_is_not_finite(dtype):
    """Ties of e4m3, the smallest and largest exponents, NaN and infinities in a block, whole blocks of
    them, blocks of zeros and of the smallest values a float has."""
    B = B_()
    table = K.e4m3_values()
    table = np.unique(table[np.isfinite(table)])
    ties = (table[1:] + table[:-1]) / 2
    rows = []
    for part in (ties[:126], ties[126:]):
        r = np.zeros(160)
        r[:part.size] = part
        r[31::32] = 448.0                                   # keeps every block's scale at 1
        rows.append(r)
    r = np.zeros(160)
    r[3], r[9] = np.inf, 2.5
    r[32:64] = np.nan
    r[64], r[70] = -np.inf, 1e-3
    r[96:128] = 2.0 ** -149 if dtype == "f32" else 2.0 ** -133
    r[128:] = 3e38
    rows.append(r)
    x = host(gpu(np.stack(rows), dtype))
    q, s = bytes8(3, 160)
    B.moe_mx_quantize(gpu(x, dtype), 3, 160, code(dtype), 0, q, s)
    torch.cuda.synchronize()
    q, s = unpack8(q, s, 3, 160)
    rq, rs = K.quantize(x)
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(K.e4m3_values()[q], rq)    # NaN where NaN


@pytest.mark.parametrize("rows,cols,dtype,pad", [(1, 32, "f32", 0), (9, 2048, "bf16", 0), (130, 96, "bf16", 1),
                                                 (3, 1408, "f32", 3), (40, 544, "bf16", 0)])
def test_quantize_swiglu(rows, cols, dtype, pad):
    B = B_()
    log(f"case quantize swiglu rows={rows} cols={cols} {dtype}")
    rng = np.random.default_rng(rows * 7 + cols)
    x = rng.standard_normal((rows, 2 * cols)) * 3
    x[0, :3] = [-60.0, 60.0, 0.0]                           # sigmoids that saturate
    x = host(gpu(x, dtype))
    q, s = bytes8(rows, cols)
    B.moe_mx_quantize(gpu(x, dtype, pad), rows, cols, code(dtype), 1, q, s)
    torch.cuda.synchronize()
    v = K.swiglu(x)
    # the exponent's rounding moves e^-g by |g| log2(e) u; 16 u for exp2, reciprocal and products
    check8("h", *unpack8(q, s, rows, cols), v, (16 + 1.5 * np.abs(x[:, :cols])) * U * np.abs(v) + 2.0 ** -149)


# ----------------------------------------------------------------------------
# RMS norm
# ----------------------------------------------------------------------------

NORMS = [
    (1, 1, "f32", 0), (1, 7168, "bf16", 0), (5, 8, "bf16", 0), (3, 511, "bf16", 0), (130, 513, "f32", 1),
    (7, 1001, "bf16", 1), (9, 1025, "f32", 3), (600, 2048, "bf16", 0), (33, 2056, "bf16", 5), (1100, 264, "f32", 0),
    (17, 4099, "bf16", 3), (6, 7168, "f32", 0), (5, 8193, "bf16", 0), (4, 16384, "f32", 0), (3, 16385, "bf16", 1),
    (3, 32768, "f32", 0), (2, 33001, "bf16", 1), (2, 33001, "f32", 1), (0, 64, "bf16", 0), (3, 32800, "bf16", 0),
    (2300, 1056, "bf16", 0), (1300, 4096, "f32", 0), (4, 30000, "bf16", 0), (70, 32, "bf16", 0),
]


def norm_inputs(T, H, dtype, seed):
    rng = np.random.default_rng(seed)
    x = host(gpu(rng.standard_normal((T, H)) * (0.5 + rng.random((T, 1))), dtype))
    res, dy, dsum = (host(gpu(c * rng.standard_normal((T, H)), dtype)) for c in (0.7, 0.1, 0.1))
    return x, res, dy, dsum, host(gpu(1 + 0.3 * rng.standard_normal(H)))


@pytest.mark.parametrize("T,H,dtype,pad", NORMS)
def test_rms_norm(T, H, dtype, pad):
    B = B_()
    log(f"case rms norm T={T} H={H} {dtype} pad={pad}")
    x, res, _, _, gamma = norm_inputs(T, H, dtype, 10 + T + H)
    eps = 1e-5
    mx = H % 32 == 0
    xt, rt, gt = gpu(x, dtype, pad), gpu(res, dtype, pad), gpu(gamma, "f32", pad)
    for with_res in (True, False):
        y, total, rstd = blank((T, H), dtype, pad), blank((T, H), dtype, pad), blank((T,))
        q, s = bytes8(T, H) if mx else (None, None)
        B.moe_rms_norm(xt, rt if with_res else None, gt, T, H, eps, code(dtype), total if with_res else None, y, q, s,
                       rstd)
        torch.cuda.synchronize()
        v = x
        if with_res:  # one fp32 addition, rounded once
            ref = (torch.from_numpy(x).float() + torch.from_numpy(res).float()).to(TORCH[dtype])
            assert torch.equal(total.cpu(), ref)
            v = host(total)
        ry, rr = K.rms_norm(v, gamma, eps)
        check("rstd", rstd, rr, (DEPTH + 8) * U * rr)
        err = (DEPTH + 12) * U * np.abs(ry)
        check("y", y, ry, HALF[dtype] * (np.abs(ry) + err) + err)
        if mx:
            check8("q", *unpack8(q, s, T, H), ry, err)
        # every output on its own, and the sum in place of either input
        y2 = blank((T, H), dtype, pad)
        B.moe_rms_norm(xt, rt if with_res else None, gt, T, H, eps, code(dtype), None, y2)
        assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8))
        if mx:
            q2, s2 = bytes8(T, H)
            B.moe_rms_norm(xt, rt if with_res else None, gt, T, H, eps, code(dtype), None, None, q2, s2)
            assert torch.equal(q, q2) and torch.equal(s, s2)
        if with_res:
            for where in (0, 1):
                pair = [gpu(x, dtype, pad), gpu(res, dtype, pad)]
                y2 = blank((T, H), dtype, pad)
                B.moe_rms_norm(*pair, gt, T, H, eps, code(dtype), pair[where], y2)
                assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8))
                assert torch.equal(total.view(torch.uint8), pair[where].view(torch.uint8))
    if T:
        for t in (y, total if with_res else y):
            tail = torch.as_strided(t, (32,), (1,), t.storage_offset() + T * H)
            assert torch.isnan(tail).all()                                      # nothing past the last row


def test_rms_norm_rows_that_are_zero_or_not_finite():
    """A row of zeros with eps gives zeros; one with an infinity or a NaN is NaN where the definition
    is, its 8-bit values too, and its neighbours are as they are."""
    B = B_()
    H = 1056
    x, _, _, _, gamma = norm_inputs(4, H, "f32", 3)
    x[0] = 0
    x[2, 5] = np.inf
    y, q, s, rstd = blank((4, H)), *bytes8(4, H), blank((4,))
    B.moe_rms_norm(gpu(x), None, gpu(gamma), 4, H, 1e-6, B.MOE_F32, None, y, q, s, rstd)
    torch.cuda.synchronize()
    got = host(y)
    assert not got[0].any() and np.isnan(got[2, 5]) and not np.delete(got[2], 5).any()
    q, s = unpack8(q, s, 4, H)
    # by value: a zero times a negative gamma is -0
    assert not K.e4m3_values()[q[0]].any() and not s[0].any() and np.isnan(K.e4m3_values()[q[2, 5]])
    for t in (1, 3):
        ry, _ = K.rms_norm(x[t:t + 1], gamma, 1e-6)
        check8("q", q[t:t + 1], s[t:t + 1], ry, (DEPTH + 12) * U * np.abs(ry))


@pytest.mark.parametrize("T,H,dtype,pad", NORMS + [(4099, 77, "bf16", 0), (2500, 1001, "f32", 0)])
def test_rms_norm_backward(T, H, dtype, pad):
    B = B_()
    log(f"case rms norm backward T={T} H={H} {dtype} pad={pad}")
    s, _, dy, dsum, gamma = norm_inputs(T, H, dtype, 20 + T + H)
    rstd = host(gpu(K.rms_norm(s, gamma, 1e-5)[1]))
    need = B.moe_rms_norm_backward_workspace_size(T, H)
    args = [gpu(s, dtype, pad), gpu(gamma, "f32", pad), gpu(rstd)]
    dyt = gpu(dy, dtype, pad)
    m = (lambda v: v.mean(1, keepdims=True)) if T else (lambda v: np.zeros((0, 1)))
    for with_sum in (True, False):
        dst = gpu(dsum, dtype, pad) if with_sum else None
        dx, dg = blank((T, H), dtype, pad), blank((H,), "f32", pad)
        B.moe_rms_norm_backward(dyt, dst, *args, T, H, code(dtype), dx, dg, scratch(need), need)
        torch.cuda.synchronize()
        rdx, rdg = K.rms_norm_backward(dy, dsum if with_sum else None, s, gamma, rstd)
        a, xh, r = np.abs(dy * gamma), np.abs(s * rstd[:, None]), rstd[:, None]
        f32 = r * (4 * U * a + (DEPTH + 8) * U * xh * m(a * xh)) + 2 * U * np.abs(rdx)
        check("dx", dx, rdx, HALF[dtype] * (np.abs(rdx) + f32) + f32)
        chain = DEPTH + T // 256 + 4
        check("dgamma", dg, rdg, chain * U * (np.abs(dy) * xh).sum(0))
        # the same bits again, without dgamma, and in place of dsum
        dx2 = blank((T, H), dtype, pad)
        B.moe_rms_norm_backward(dyt, dst, *args, T, H, code(dtype), dx2, None, None, 0)
        assert torch.equal(dx.view(torch.uint8), dx2.view(torch.uint8))
        dg2 = blank((H,))
        B.moe_rms_norm_backward(dyt, dst, *args, T, H, code(dtype), dst if with_sum else dx2, dg2, scratch(need), need)
        assert torch.equal(dx.view(torch.uint8), (dst if with_sum else dx2).view(torch.uint8))
        assert torch.equal(dg, dg2)


def test_rows_past_2_31_elements():
    """The norm's and the quantisation's last rows, and dropout's last elements, past 2^31 of them."""
    B = B_()
    T, H = 300_000, 7168
    log(f"case T={T} H={H}: {T * H / 2 ** 31:.2f} * 2^31 elements")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows, _, _, _, gamma = norm_inputs(2, H, "bf16", 5)
    x[-2:] = gpu(rows, "bf16")
    q, s = bytes8(T, H)
    y = torch.empty_like(x)
    ry, _ = K.rms_norm(rows, gamma, 1e-5)
    err = (DEPTH + 12) * U * np.abs(ry)
    p = K.pitch(H)
    tail = lambda: (q[(T - 2) * H:T * H].cpu().numpy().reshape(2, H), s[(T - 2) * p:T * p].cpu().numpy().reshape(2, p))
    B.moe_rms_norm(x, None, gpu(gamma), T, H, 1e-5, B.MOE_BF16, None, y, q, s)
    check("y", y[-2:], ry, HALF["bf16"] * (np.abs(ry) + err) + err)
    check8("q", *tail(), ry, err)
    B.moe_mx_quantize(x, T, H, B.MOE_BF16, 0, q, s)
    torch.cuda.synchronize()
    got, ref = tail(), K.quantize(rows)
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_array_equal(K.e4m3_values()[got[0]], ref[0])
    n = T * H - 3
    rng = rng_state(77, 5)
    B.moe_dropout_add(x, B.MOE_BF16, None, n, 0.25, rng, B.MOE_BF16, y)
    mask = K.keep(2 * H - 3, 0.25, 77, 5, first=n - (2 * H - 3))
    want = np.where(mask, rows.reshape(-1)[:2 * H - 3] / 0.75, 0)
    check("dropout", y.view(-1)[n - (2 * H - 3):n], want, (HALF["bf16"] + 4 * U) * np.abs(want))


# ----------------------------------------------------------------------------
# dropout
# ----------------------------------------------------------------------------

def rng_state(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("n,p,pad", [(1, 0.5, 0), (7, 0.5, 1), (8, 0.0, 0), (1000, 0.1, 3), (4099 * 33, 0.3, 0),
                                     (70000, 0.999, 5), (2048, 1e-9, 0), (0, 0.5, 0)])
@pytest.mark.parametrize("x_dtype,dtype", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_dropout(n, p, pad, x_dtype, dtype):
    """Values, and NaN under the mask: a dropped value counts for nothing."""
    B = B_()
    log(f"case dropout n={n} p={p} pad={pad} {x_dtype} -> {dtype}")
    gen = np.random.default_rng(n + 1)
    seed, step = 2 ** 62 + 12345, 2 ** 40 + n
    mask = K.keep(n, p, seed, step)
    x, res = host(gpu(gen.standard_normal(n), x_dtype)), host(gpu(gen.standard_normal(n), dtype))
    poisoned = np.where(mask, x, np.nan)
    if n > 2:
        poisoned[np.flatnonzero(~mask)[:1]] = np.inf
    rng = rng_state(seed, step)
    kept = np.where(mask, x / (1 - p), 0)
    for with_res in (True, False):
        want = kept + res if with_res else kept
        tol = HALF[dtype] * np.abs(want) + 4 * U * (np.abs(kept) + np.abs(want))
        xt, rt, out = gpu(poisoned, x_dtype, pad), gpu(res, dtype, pad), blank((n,), dtype, pad)
        B.moe_dropout_add(xt, code(x_dtype), rt if with_res else None, n, p, rng, code(dtype), out)
        torch.cuda.synchronize()
        check("out", out, want, tol)
        behind = torch.as_strided(out, (32,), (1,), out.storage_offset() + n)
        assert torch.isnan(behind).all()
        places = [rt] if with_res else []
        places += [xt] if x_dtype == dtype else []
        for place in places:                                # in place of an input
            a = [gpu(poisoned, x_dtype, pad), gpu(res, dtype, pad)]
            into = a[0] if place is xt else a[1]
            B.moe_dropout_add(a[0], code(x_dtype), a[1] if with_res else None, n, p, rng, code(dtype), into)
            assert torch.equal(into.view(torch.uint8), out.view(torch.uint8))
    # the gradient: the same mask on the output's gradient
    dout = np.where(mask, host(gpu(gen.standard_normal(n), dtype)), np.nan)
    dx = blank((n,), x_dtype, pad)
    B.moe_dropout_add_backward(gpu(dout, dtype, pad), code(dtype), n, p, rng, code(x_dtype), dx)
    torch.cuda.synchronize()
    want = np.where(mask, dout / (1 - p), 0)
    check("dx", dx, want, (HALF[x_dtype] + 4 * U) * np.abs(want))


def test_dropout_graph_draws_a_new_mask():
    """Captured once; each replay reads the step of the moment."""
    B = B_()
    n, p = 5001, 0.4
    gen = np.random.default_rng(8)
    x = host(gpu(gen.standard_normal(n)))
    xt, rng, out = gpu(x), rng_state(11, 0), blank((n,))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        B.moe_dropout_add(xt, B.MOE_F32, None, n, p, rng, B.MOE_F32, out, stream)
    for step in (0, 1, 2, 3):
        rng.copy_(rng_state(11, step))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = np.where(K.keep(n, p, 11, step), x / (1 - p), 0)
        check(f"step {step}", out, want, 4 * U * np.abs(want))
        torch.randn(1 << 20, device="cuda").sum().item()


def test_norm_and_quantize_graph_replay():
    """The norm with all its outputs, its backward and the quantisation in one graph, replayed on new
    inputs with eager work in between: every replay gives the eager call's bits."""
    B = B_()
    T, H = 70, 1056

    def state():
        t = dict(x=blank((T, H), "bf16"), res=blank((T, H), "bf16"), dy=blank((T, H), "bf16"), gamma=blank((H,)),
                 sum=blank((T, H), "bf16"), y=blank((T, H), "bf16"), rstd=blank((T,)), dx=blank((T, H), "bf16"),
                 dg=blank((H,)))
        t["q"], t["s"] = bytes8(T, H)
        t["q2"], t["s2"] = bytes8(T, H // 2 // 32 * 32)
        t["need"] = B.moe_rms_norm_backward_workspace_size(T, H)
        t["ws"] = scratch(t["need"])
        return t

    def step(t, stream=None):
        B.moe_rms_norm(t["x"], t["res"], t["gamma"], T, H, 1e-5, B.MOE_BF16, t["sum"], t["y"], t["q"], t["s"],
                       t["rstd"], stream)
        B.moe_rms_norm_backward(t["dy"], t["y"], t["sum"], t["gamma"], t["rstd"], T, H, B.MOE_BF16, t["dx"], t["dg"],
                                t["ws"], t["need"], stream)
        B.moe_mx_quantize(t["y"], T, H // 2 // 32 * 32, B.MOE_BF16, 1, t["q2"], t["s2"], stream)

    a, b = state(), state()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(a, stream)
    for turn in range(4):
        x, res, dy, _, gamma = norm_inputs(T, H, "bf16", 40 + turn)
        for t in (a, b):
            for name, v in (("x", x), ("res", res), ("dy", dy)):
                t[name].copy_(gpu(v, "bf16"))
            t["gamma"].copy_(gpu(gamma))
        torch.cuda.synchronize()
        g.replay()
        step(b)
        torch.cuda.synchronize()
        for name in ("sum", "y", "rstd", "dx", "dg", "q", "s", "q2", "s2"):
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), (turn, name)
        torch.randn(1 << 20, device="cuda").sum().item()


@pytest.mark.parametrize("T,H,dtype", [(1, 64, "f32"), (2, 8192, "bf16"), (3, 8192, "bf16"), (32, 500, "bf16"),
                                       (33, 500, "f32"), (31, 512, "f32"), (4, 4096, "f32"), (5, 4096, "bf16")])
def test_rms_norm_backward_of_few_rows(T, H, dtype):
    """One block's sums are dgamma itself; from one row more on they are added from the workspace."""
    B = B_()
    s, _, dy, dsum, gamma = norm_inputs(T, H, dtype, 60 + T + H)
    rstd = host(gpu(K.rms_norm(s, gamma, 1e-5)[1]))
    need = B.moe_rms_norm_backward_workspace_size(T, H)
    dx, dg = blank((T, H), dtype), blank((H,))
    B.moe_rms_norm_backward(gpu(dy, dtype), gpu(dsum, dtype), gpu(s, dtype), gpu(gamma), gpu(rstd), T, H, code(dtype),
                            dx, dg, scratch(need), need)
    torch.cuda.synchronize()
    rdx, rdg = K.rms_norm_backward(dy, dsum, s, gamma, rstd)
    xh = np.abs(s * rstd[:, None])
    check("dgamma", dg, rdg, (DEPTH + 4) * U * (np.abs(dy) * xh).sum(0))
    a, r = np.abs(dy * gamma), rstd[:, None]
    f32 = r * (4 * U * a + (DEPTH + 8) * U * xh * (a * xh).mean(1, keepdims=True)) + 2 * U * np.abs(rdx)
    check("dx", dx, rdx, HALF[dtype] * (np.abs(rdx) + f32) + f32)
    behind = torch.as_strided(dg, (32,), (1,), dg.storage_offset() + H)
    assert torch.isnan(behind).all()


def test_dropout_past_2_34_elements():
    """In place, where a thread takes more than one turn and an element's index / 4 passes 32 bits."""
    B = B_()
    n, p, seed, step = 2 ** 34 + 5003, 0.25, 9, 4
    if torch.cuda.mem_get_info()[0] < 2 * n + 2 ** 33:
        pytest.skip("34 GB of device memory are not free")
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    B.moe_dropout_add(x, B.MOE_BF16, None, n, p, rng_state(seed, step), B.MOE_BF16, x)
    torch.cuda.synchronize()
    one = float(host(gpu(np.array([1 / (1 - p)]), "bf16"))[0])
    for first in (0, 2 ** 33 - 1000, 2 ** 34 - 2000, n - 3000):
        got = host(x[first:first + 3000])
        assert np.array_equal(got, np.where(K.keep(got.size, p, seed, step, first=first), one, 0))
