"""The training pass of the MoE block on the GPU against ``oracle.backward`` in float64, through
the C ABI, element by element.

Tolerances, derived per element (u = 2^-24, half an fp32 step; HALF[dtype] half a step of the
stored type: 2^-8 for bf16, 2^-24 for f32):

* a chain of n fp32 additions of terms t_i is off by at most n u sum|t_i|.  The row sums of the
  norm and the combine run at most DEPTH = 64 additions deep (at most 8 elements of 4 vectors a
  lane and sweep, 6 steps across the wave, 16 waves, and the few sweeps of the longest rows here).
* an output stored in dtype is off by HALF[dtype] |value| more.
* the experts: every product sum of depth K is off by at most K u sum|a b|; h, dg and du are
  stored in dtype (HALF of each); first-order propagation through dg = dh u silu'(g) with
  |silu'| <= 1.1, |silu''| <= 0.5, |silu| <= |g|, and 16 u for exp2, reciprocal and products.
  The second-order terms are below the 1.1 that multiplies the sum.
"""
import gc

import numpy as np
import pytest

from moe_cases import O, build_layer, log, synth
from oracle import backward as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DEPTH = 64
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def code(dtype):
    B = B_()
    return B.MOE_F32 if dtype == "f32" else B.MOE_BF16


def gpu(a, dtype="f32", pad=0):
    """A device copy in dtype; pad: its first element sits that many elements into an allocation."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    out = torch.zeros(t.numel() + pad + 64, dtype=TORCH[dtype], device="cuda")[pad:pad + t.numel()]
    out.copy_(t.reshape(-1).to(TORCH[dtype]))
    return out.view(t.shape)


def blank(shape, dtype="f32", pad=0, fill=float("nan")):
    n = int(np.prod(shape))
    return torch.full((n + pad + 64,), fill, dtype=TORCH[dtype], device="cuda")[pad:pad + n].view(shape)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(name, got, ref, tol):
    got = host(got) if torch.is_tensor(got) else got
    assert got.shape == ref.shape, name
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{name}: {np.count_nonzero(~np.isfinite(got))} not finite"
    over = np.abs(got - ref) / np.maximum(tol, 1e-300)
    worst = float(over.max())
    log(f"  {name}: largest error {worst:.3f} of its tolerance")
    assert worst <= 1.0, (name, worst, np.unravel_index(over.argmax(), over.shape))


def scratch(n):
    return torch.full((max(1, n),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN bits


# ----------------------------------------------------------------------------
# layer norm
# ----------------------------------------------------------------------------

NORMS = [
    (1, 1, "f32", 0), (1, 7168, "bf16", 0), (5, 8, "bf16", 0), (3, 511, "bf16", 0), (130, 513, "f32", 1),
    (7, 1001, "bf16", 1), (9, 1025, "f32", 3), (600, 2048, "bf16", 0), (33, 2056, "bf16", 5),
    (1100, 264, "f32", 0), (17, 4099, "bf16", 3), (6, 7168, "f32", 0), (5, 8193, "bf16", 0),
    (4, 16384, "f32", 0), (3, 16385, "bf16", 1), (3, 32768, "f32", 0), (2, 33001, "bf16", 1),
    (2, 33001, "f32", 1), (0, 64, "bf16", 0),
]


def norm_inputs(T, H, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H)) * (0.5 + rng.random((T, 1))) + 3 * rng.standard_normal((T, 1))
    x = host(gpu(x, dtype))
    dy = host(gpu(0.1 * rng.standard_normal((T, H)), dtype))
    gamma = host(gpu(1 + 0.3 * rng.standard_normal(H)))
    beta = host(gpu(0.2 * rng.standard_normal(H)))
    return x, dy, gamma, beta


@pytest.mark.parametrize("T,H,dtype,pad", NORMS)
def test_layer_norm(T, H, dtype, pad):
    B = B_()
    log(f"case layer norm T={T} H={H} {dtype} pad={pad}")
    x, dy, gamma, beta = norm_inputs(T, H, dtype, 10 + T + H)
    eps = 1e-5
    xt, dyt, gt, bt = gpu(x, dtype, pad), gpu(dy, dtype, pad), gpu(gamma, "f32", pad), gpu(beta, "f32", pad)
    for with_beta in (True, False):
        y, mean, rstd = blank((T, H), dtype, pad), blank((T,)), blank((T,))
        B.moe_layer_norm(xt, gt, bt if with_beta else None, T, H, eps, code(dtype), y, mean, rstd)
        torch.cuda.synchronize()
        ry, rmean, rrstd = G.layer_norm(x, gamma, beta if with_beta else None, eps)
        mu_err = DEPTH * U * np.abs(x).mean(1, keepdims=True) if T else np.zeros((0, 1))
        check("mean", mean, rmean, mu_err[:, 0] + U * np.abs(rmean))
        # (mu_err / sigma)^2 is second order; the square sum and sqrt cost DEPTH + 8 half steps
        check("rstd", rstd, rrstd, (DEPTH + 8) * U * rrstd + rrstd * (mu_err[:, 0] * rrstd) ** 2)
        xh = (x - rmean[:, None]) * rrstd[:, None]
        f32 = np.abs(gamma) * (mu_err * rrstd[:, None] + (DEPTH + 16) * U * np.abs(xh)) + \
            4 * U * (np.abs(ry) + (np.abs(beta) if with_beta else 0))
        check("y", y, ry, HALF[dtype] * (np.abs(ry) + f32) + f32)
        y2 = blank((T, H), dtype, pad)
        B.moe_layer_norm(xt, gt, bt if with_beta else None, T, H, eps, code(dtype), y2)
        assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8))      # without the statistics
    if T:
        tail = torch.as_strided(y, (32,), (1,), y.storage_offset() + T * H)
        assert torch.isnan(tail).all()                                      # nothing past the last row


@pytest.mark.parametrize("T,H,dtype,pad", NORMS + [(4099, 77, "bf16", 0), (2500, 1001, "f32", 0)])
def test_layer_norm_backward(T, H, dtype, pad):
    B = B_()
    log(f"case layer norm backward T={T} H={H} {dtype} pad={pad}")
    x, dy, gamma, _ = norm_inputs(T, H, dtype, 20 + T + H)
    _, mean, rstd = G.layer_norm(x, gamma, None, 1e-5)
    mean, rstd = host(gpu(mean)), host(gpu(rstd))
    args = [gpu(dy, dtype, pad), gpu(x, dtype, pad), gpu(gamma, "f32", pad), gpu(mean), gpu(rstd)]
    need = B.moe_layer_norm_backward_workspace_size(T, H)
    ws = scratch(need)
    dx, dg, db = blank((T, H), dtype, pad), blank((H,), "f32", pad), blank((H,), "f32", pad)
    B.moe_layer_norm_backward(*args, T, H, code(dtype), dx, dg, db, ws, need)
    torch.cuda.synchronize()
    rdx, rdg, rdb = G.layer_norm_backward(dy, x, gamma, mean, rstd)
    a, r = np.abs(dy * gamma), rstd[:, None]
    xh = np.abs((x - mean[:, None]) * r)
    # x - mean and the product with rstd are rounded: |x| + |mean| in place of |x - mean|
    xe = 4 * U * (np.abs(x) + np.abs(mean)[:, None]) * r
    m = (lambda v: v.mean(1, keepdims=True)) if T else (lambda v: np.zeros((0, 1)))
    f32 = r * (4 * U * a + (DEPTH + 4) * U * m(a) + (DEPTH + 8) * U * xh * m(a * xh) +
               xe * m(a * xh) + xh * m(a * xe))
    check("dx", dx, rdx, HALF[dtype] * (np.abs(rdx) + f32) + f32)
    chain = DEPTH + T // 256
    check("dgamma", dg, rdg, chain * U * (np.abs(dy) * xh).sum(0) + (np.abs(dy) * xe).sum(0))
    check("dbeta", db, rdb, chain * U * np.abs(dy).sum(0))
    # the same bits again, and with the sums left out one by one
    for with_g, with_b in ((True, True), (True, False), (False, True), (False, False)):
        dx2, dg2, db2 = blank((T, H), dtype, pad), blank((H,)), blank((H,))
        sums = with_g or with_b
        B.moe_layer_norm_backward(*args, T, H, code(dtype), dx2, dg2 if with_g else None,
                                  db2 if with_b else None, scratch(need) if sums else None,
                                  need if sums else 0)
        assert torch.equal(dx.view(torch.uint8), dx2.view(torch.uint8))
        assert not with_g or torch.equal(dg, dg2)
        assert not with_b or torch.equal(db, db2)


def test_layer_norm_row_far_from_zero_and_constant_row():
    """Centred sums: a row at 1000 with unit spread keeps its digits; a constant row gives beta."""
    B = B_()
    rng = np.random.default_rng(3)
    H = 1000
    x = host(gpu(np.stack([1000 + rng.standard_normal(H), np.full(H, 7.0)])))
    y, mean, rstd = blank((2, H)), blank((2,)), blank((2,))
    one, beta = gpu(np.ones(H)), gpu(np.linspace(-1, 1, H))
    B.moe_layer_norm(gpu(x), one, beta, 2, H, 1e-5, B.MOE_F32, y, mean, rstd)
    ry, _, rr = G.layer_norm(x, np.ones(H), host(beta), 1e-5)
    check("y", y[:1], ry[:1], np.full((1, H), DEPTH * U * 1000 * rr[0] + 4 * U * 8))
    check("constant row", y[1:], host(beta)[None], np.full((1, H), 1e-300))


# ----------------------------------------------------------------------------
# combine, permute, route
# ----------------------------------------------------------------------------

def routed(T, E, k, seed):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    idx, w = O.route(logits, k)
    row_of, src_of = O.permutation(idx, E)
    return rng, idx, np.asarray(w, np.float64), np.asarray(row_of, np.int32), src_of


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


SORTS = [(1, 1, 1, 1), (1, 4, 2, 8), (7, 5, 5, 33), (64, 32, 8, 512), (37, 11, 3, 1001),
         (50, 100, 64, 72), (5, 16, 8, 7168), (9, 12, 9, 2056), (3, 8, 2, 16400), (300, 6, 1, 264)]


@pytest.mark.parametrize("T,E,k,H", SORTS)
@pytest.mark.parametrize("dy_dtype,dtype,pad", [("f32", "f32", 1), ("f32", "bf16", 0), ("bf16", "bf16", 3),
                                                ("bf16", "f32", 0)])
def test_combine_backward(T, E, k, H, dy_dtype, dtype, pad):
    B = B_()
    log(f"case combine backward T={T} E={E} k={k} H={H} {dy_dtype} -> {dtype}")
    rng, idx, w, row_of, _ = routed(T, E, k, 30 + T + H)
    R = T * k
    dy = host(gpu(rng.standard_normal((T, H)), dy_dtype))
    yp = host(gpu(rng.standard_normal((R, H))))
    w = host(gpu(w))
    args = [gpu(dy, dy_dtype, pad), code(dy_dtype)]
    dyp, dw = blank((R, H), dtype, pad), blank((T, k))
    B.moe_combine_backward(*args, gpu(yp, "f32", pad), i32(row_of), gpu(w), T, k, H, code(dtype), dyp, dw)
    torch.cuda.synchronize()
    rdyp, rdw = G.combine_backward(dy, yp, row_of, w, k)
    check("dy_perm", dyp, rdyp, (HALF[dtype] + 2 * U) * np.abs(rdyp))
    check("dtopk_w", dw, rdw, DEPTH * U * G.combine_backward(np.abs(dy), np.abs(yp), row_of, w, k)[1])
    dyp2 = blank((R, H), dtype, pad)
    B.moe_combine_backward(*args, None, i32(row_of), gpu(w), T, k, H, code(dtype), dyp2, None)
    assert torch.equal(dyp.view(torch.uint8), dyp2.view(torch.uint8))       # without the weights'


@pytest.mark.parametrize("T,E,k,H", SORTS)
@pytest.mark.parametrize("dtype,pad", [("f32", 1), ("bf16", 0), ("bf16", 3)])
def test_permute_backward(T, E, k, H, dtype, pad):
    B = B_()
    log(f"case permute backward T={T} E={E} k={k} H={H} {dtype}")
    rng, _, _, row_of, _ = routed(T, E, k, 40 + T + H)
    d = host(gpu(rng.standard_normal((T * k, H)), dtype))
    dx = blank((T, H), dtype, pad)
    B.moe_permute_backward(gpu(d, dtype, pad), i32(row_of), T, k, H, code(dtype), dx)
    torch.cuda.synchronize()
    ref = G.permute_backward(d, row_of, k)
    f32 = k * U * G.permute_backward(np.abs(d), row_of, k)
    check("dx", dx, ref, HALF[dtype] * (np.abs(ref) + f32) + f32)


def test_dropped_assignments_add_nothing():
    """Rows that moe_permute dropped carry an index outside [0, T k): nothing is read or written
    for them, and the rows that no index names keep what they held."""
    B = B_()
    T, k, H = 6, 3, 40
    rng = np.random.default_rng(5)
    row_of = rng.permutation(T * k).astype(np.int32)
    row_of[[2, 7]] = [-1, T * k]
    gone = sorted(set(range(T * k)) - set(row_of.tolist()))
    dy, yp, w = (host(gpu(rng.standard_normal(s))) for s in ((T, H), (T * k, H), (T, k)))
    dyp, dw = blank((T * k, H), fill=5.0), blank((T, k))
    B.moe_combine_backward(gpu(dy), B.MOE_F32, gpu(yp), i32(row_of), gpu(w), T, k, H, B.MOE_F32, dyp, dw)
    dx = blank((T, H))
    B.moe_permute_backward(gpu(yp), i32(row_of), T, k, H, B.MOE_F32, dx)
    torch.cuda.synchronize()
    assert (host(dyp)[gone] == 5.0).all()
    flat = host(dw).reshape(-1)
    assert flat[2] == 0 and flat[7] == 0
    keep = [a for a in range(T * k) if a not in (2, 7)]
    ref = np.zeros((T, H))
    for a in keep:
        np.testing.assert_array_equal(host(dyp)[row_of[a]],
                                      (w.reshape(-1)[a].astype(np.float32) * dy[a // k].astype(np.float32)))
        ref[a // k] += yp[row_of[a]]
    check("dx", dx, ref, 3 * U * 3 * np.abs(yp).max() * np.ones_like(ref))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (64, 256, 8), (5, 37, 3), (130, 64, 64),
                                   (33, 1000, 8), (9, 1024, 64), (257, 6, 2), (12, 65, 1), (0, 8, 2)])
def test_route_backward(T, E, k):
    B = B_()
    log(f"case route backward T={T} E={E} k={k}")
    rng, idx, w, _, _ = routed(T, E, k, 50 + T + E)
    w, dw = host(gpu(w)).reshape(T, k), host(gpu(rng.standard_normal((T, k))))
    dl, status = blank((T, E)), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_route_backward(i32(idx), gpu(w), gpu(dw), T, E, k, dl, status)
    torch.cuda.synchronize()
    ref = G.route_backward(idx, w, dw, E)
    # w sums to one within k u; the sum over the k slots is at most 8 additions deep in the wave
    tol = np.zeros((T, E))
    if T:
        np.put_along_axis(tol, np.asarray(idx, np.int64),
                          w * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True)) * 16 * U, 1)
    check("dlogits", dl, ref, tol)
    assert int(status.item()) == 0


def test_route_backward_repeated_and_bad_ids():
    B = B_()
    rng = np.random.default_rng(7)
    T, E, k = 3, 9, 4
    idx = np.array([[1, 4, 1, 1], [0, 8, 3, 2], [5, 5, 6, 6]], np.int32)
    w, dw = host(gpu(rng.random((T, k)))), host(gpu(rng.standard_normal((T, k))))
    dl, status = blank((T, E)), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_route_backward(i32(idx), gpu(w), gpu(dw), T, E, k, dl, status)
    check("dlogits", dl, G.route_backward(idx, w, dw, E), np.full((T, E), 64 * U * 4))
    assert int(status.item()) == 0
    idx[1] = [0, 9, -1, 2]
    dl = blank((T, E))
    B.moe_route_backward(i32(idx), gpu(w), gpu(dw), T, E, k, dl, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.MOE_STATUS_BAD_EXPERT_ID
    assert np.isfinite(host(dl)).all() and not host(dl)[1, [1, 3, 4, 5, 6, 7, 8]].any()


# ----------------------------------------------------------------------------
# experts
# ----------------------------------------------------------------------------

def experts_tolerance(x, dy, wg, wu, wd, half):
    """(tol_dx, tol_dwg, tol_dwu, tol_dwd) of one expert's rows."""
    n, H = x.shape
    I = wg.shape[0]
    dx, dwg, dwu, dwd, m = G.swiglu_ffn_backward(x, dy, wg, wu, wd)
    ab = np.abs
    eg, eu = H * U * (ab(x) @ ab(wg).T), H * U * (ab(x) @ ab(wu).T)
    eh = H * U * (ab(dy) @ ab(wd))
    g, u, dh = ab(m["g"]), ab(m["u"]), ab(m["dh"])
    silu = ab(m["g"] * m["s"])
    e_h = half * ab(m["h"]) + 16 * U * silu * u + 1.1 * eg * u + silu * eu
    e_du = half * ab(m["du"]) + 16 * U * dh * silu + eh * silu + 1.1 * dh * eg
    e_dg = half * ab(m["dg"]) + 1.1 * (16 * U * dh * u + eh * u + dh * eu) + 0.5 * dh * u * eg
    e_h, e_du, e_dg = 1.1 * e_h, 1.1 * e_du, 1.1 * e_dg
    adg, adu, ah = ab(m["dg"]) + e_dg, ab(m["du"]) + e_du, ab(m["h"]) + e_h

    def out(value, err, depth_sum, depth):
        f = err + depth * U * depth_sum
        return half * (ab(value) + f) + f

    return (out(dx, e_dg @ ab(wg) + e_du @ ab(wu), adg @ ab(wg) + adu @ ab(wu), 2 * I),
            out(dwg, e_dg.T @ ab(x), adg.T @ ab(x), n), out(dwu, e_du.T @ ab(x), adu.T @ ab(x), n),
            out(dwd, ab(dy).T @ e_h, ab(dy).T @ ah, n))


def run_experts(counts, H, I, dtype, seed, slots=None, n_slots=None, tail_rows=0, want=("dx", "dw"),
                stream=None, scale=1.0):
    """One call on random inputs: (inputs, outputs, status)."""
    B = B_()
    rng = np.random.default_rng(seed)
    E, R = len(counts), int(sum(counts)) + tail_rows
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    slots = list(range(E)) if slots is None else slots
    n_slots = E if n_slots is None else n_slots
    x = host(gpu(scale * rng.standard_normal((R, H)), dtype))
    dy = host(gpu(0.2 * rng.standard_normal((R, H)), dtype))
    w = rng.standard_normal((n_slots, 3 * H * I)) * H ** -0.5
    w[:, 2 * H * I:] *= (H / I) ** 0.5
    w = host(gpu(w, dtype))
    wt, slot_of = gpu(w, dtype), i32(slots)
    buf = B.wbuf(wt, 3 * H * I * wt.element_size(), n_slots, E, slot_of)
    need = B.moe_grouped_swiglu_backward_workspace_size(R, E, H, I, code(dtype))
    ws = scratch(need)
    dx = blank((R, H), dtype) if "dx" in want else None
    dw = blank((n_slots, 3 * H * I), dtype) if "dw" in want else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xt, dyt, ot = gpu(x, dtype), gpu(dy, dtype), i32(offsets)
    torch.cuda.synchronize()

    def call():
        B.moe_grouped_swiglu_backward(xt, dyt, ot, R, E, H, I, code(dtype), buf, ws, need, dx, dw,
                                      status, stream)

    call()
    torch.cuda.synchronize()
    keep = (xt, dyt, ot, wt, slot_of, ws)
    return dict(x=x, dy=dy, w=w, offsets=offsets, slots=slots, call=call, keep=keep), dx, dw, int(status.item())


def check_experts(counts, H, I, dtype, inp, dx, dw):
    HI = H * I
    for e, n in enumerate(counts):
        lo = int(inp["offsets"][e])
        s = inp["slots"][e]
        rows = slice(lo, lo + n)
        if s < 0:
            continue
        got_w = host(dw[s]) if dw is not None else None
        if n == 0:
            assert dw is None or not got_w.any(), f"expert {e} without rows"
            continue
        wg, wu, wd = O.expert_matrices(inp["w"][s], H, I)
        x, dy = inp["x"][rows], inp["dy"][rows]
        rdx, rdwg, rdwu, rdwd, _ = G.swiglu_ffn_backward(x, dy, wg, wu, wd)
        t = experts_tolerance(x, dy, wg, wu, wd, HALF[dtype])
        if dx is not None:
            check(f"dx of expert {e} ({n} rows)", dx[rows], rdx, t[0])
        if dw is not None:
            check(f"dwg of expert {e}", got_w[:HI].reshape(I, H), rdwg, t[1])
            check(f"dwu of expert {e}", got_w[HI:2 * HI].reshape(I, H), rdwu, t[2])
            check(f"dwd of expert {e}", got_w[2 * HI:].reshape(H, I), rdwd, t[3])


EXPERTS = [
    ((1,), 8, 8, "bf16"), ((3, 0, 5), 16, 8, "bf16"), ((1, 2, 0, 16, 17), 136, 72, "bf16"),
    ((31, 32, 33, 0, 63, 65), 64, 264, "bf16"), ((127, 128, 129), 256, 200, "bf16"),
    ((255, 257, 0, 1), 264, 512, "bf16"), ((300, 512), 512, 136, "bf16"), ((70, 900), 768, 264, "bf16"),
    ((0, 0, 4), 520, 520, "bf16"), ((193, 64, 191), 1024, 256, "bf16"),
    ((1,), 1, 1, "f32"), ((3, 0, 5), 17, 9, "f32"), ((129, 1, 0, 40), 131, 77, "f32"),
    ((64, 200), 256, 512, "f32"), ((33, 31), 300, 129, "f32"),
]


@pytest.mark.parametrize("counts,H,I,dtype", EXPERTS)
def test_grouped_swiglu_backward(counts, H, I, dtype):
    log(f"case experts backward rows={counts} H={H} I={I} {dtype}")
    inp, dx, dw, status = run_experts(counts, H, I, dtype, 60 + H + I)
    assert status == 0
    check_experts(counts, H, I, dtype, inp, dx, dw)
    first = (dx.clone(), dw.clone())
    inp["call"]()                                   # on the workspace the first call left
    torch.cuda.synchronize()
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw)


# f32: each pair of tile sizes (large, small) that dX and the weight gradients can have
@pytest.mark.parametrize("counts,H,I", [((700, 1, 899, 500), 1030, 901), ((3500,), 645, 130),
                                        ((5, 7, 0, 1, 33, 2, 3, 4, 5, 6, 7, 8), 330, 261),
                                        ((31, 33, 0, 65), 97, 63)])
def test_grouped_swiglu_backward_f32_tiles(counts, H, I):
    log(f"case experts backward rows={counts} H={H} I={I} f32")
    inp, dx, dw, status = run_experts(counts, H, I, "f32", 90 + H + I)
    assert status == 0
    check_experts(counts, H, I, "f32", inp, dx, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", range(8))
def test_grouped_swiglu_backward_random(seed, dtype):
    rng = np.random.default_rng(700 + seed)
    E = int(rng.integers(1, 12))
    counts = tuple(int(c) for c in rng.integers(0, [3, 40, 150, 400][seed % 4], E))
    unit = 8 if dtype == "bf16" else 1
    H, I = (unit * int(rng.integers(1, 400 // unit)) for _ in range(2))
    if sum(counts) == 0:
        counts = counts[:-1] + (1,)
    log(f"case experts backward rows={counts} H={H} I={I} {dtype}")
    inp, dx, dw, status = run_experts(counts, H, I, dtype, 800 + seed)
    assert status == 0
    check_experts(counts, H, I, dtype, inp, dx, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_only_one_output(dtype):
    counts, H, I = (40, 0, 130), 136, 72
    inp, dx, dw, _ = run_experts(counts, H, I, dtype, 5)
    _, dx2, none, _ = run_experts(counts, H, I, dtype, 5, want=("dx",))
    assert none is None and torch.equal(dx, dx2)
    _, none, dw2, _ = run_experts(counts, H, I, dtype, 5, want=("dw",))
    assert none is None and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_absent_slots_and_untouched_memory(dtype):
    """Expert 1 has rows and no slot, expert 3 a slot past the buffer, expert 2 no rows and no
    slot; slots are permuted, slot 1 belongs to nobody; 9 rows follow the last expert's."""
    B = B_()
    counts, H, I = (20, 7, 0, 5, 140), 64, 40
    slots = [3, -1, -1, 4, 0]
    inp, dx, dw, status = run_experts(counts, H, I, dtype, 6, slots=slots, n_slots=4, tail_rows=9)
    assert status == B.MOE_STATUS_EXPERT_ABSENT
    inp["slots"] = [3, -1, -1, -1, 0]
    check_experts(counts, H, I, dtype, inp, dx, dw)
    off = inp["offsets"]
    for lo, hi in ((off[1], off[2]), (off[3], off[4]), (off[5], off[5] + 9)):
        assert torch.isnan(dx[lo:hi]).all()
    assert torch.isnan(dw[1]).all() and torch.isnan(dw[2]).all()
    assert torch.isfinite(dw[0]).all() and torch.isfinite(dw[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_neighbours_nan_and_infinity_stay_out(dtype):
    """An expert whose rows, or whose weights, hold NaN and infinity does not reach its
    neighbours' gradients."""
    B = B_()
    counts, H, I = (33, 5, 70), 136, 72
    inp, dx, dw, _ = run_experts(counts, H, I, dtype, 8)
    clean = dx.clone(), dw.clone()
    xt, dyt, ot, wt, slot_of, ws = inp["keep"]
    lo, hi = 33, 38
    xt[lo:hi, ::3] = float("nan")
    dyt[lo:hi, 1::3] = float("inf")
    wt[1, ::5] = float("nan")
    inp["call"]()
    torch.cuda.synchronize()
    for rows in (slice(0, 33), slice(38, 108)):
        assert torch.equal(dx[rows], clean[0][rows])
    for e in (0, 2):
        assert torch.equal(dw[e], clean[1][e])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_extreme_gates(dtype):
    """Gates of several hundred either way: sigmoid saturates, nothing overflows into NaN."""
    counts, H, I = (40, 12), 64, 48
    inp, dx, dw, status = run_experts(counts, H, I, dtype, 9, scale=300.0)
    assert status == 0 and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    check_experts(counts, H, I, dtype, inp, dx, dw)


def test_experts_without_rows():
    B = B_()
    H, I, E = 64, 40, 3
    dw = blank((E, 3 * H * I), "bf16")
    need = B.moe_grouped_swiglu_backward_workspace_size(0, E, H, I, B.MOE_BF16)
    offsets, slots = i32([0] * (E + 1)), i32(range(E))
    w = torch.zeros_like(dw)
    buf = B.wbuf(w, 3 * H * I * 2, E, E, slots)
    B.moe_grouped_swiglu_backward(None, None, offsets, 0, E, H, I, B.MOE_BF16, buf, scratch(need), need,
                                  None, dw)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.parametrize("E", [256, 1024])
def test_experts_many_with_few_rows(E):
    rng = np.random.default_rng(E)
    counts = [0] * E
    for e in rng.integers(0, E, 90):
        counts[e] += 1
    inp, dx, dw, status = run_experts(tuple(counts), 72, 40, "bf16", 11)
    assert status == 0
    live = [e for e in range(E) if counts[e]]
    for e in live[:5] + live[-5:]:
        sub = dict(inp, offsets=inp["offsets"][e:], slots=inp["slots"][e:])
        check_experts(tuple(counts[e:e + 1]), 72, 40, "bf16", sub, dx, dw)
    assert not dw[[e for e in range(E) if not counts[e]]].any()


# ----------------------------------------------------------------------------
# together: the layer's training step
# ----------------------------------------------------------------------------

def layer_case(dtype, pre_norm, T=96, H=136, I=72, E=12, k=3, **kw):
    cfg = synth.MoEConfig(f"train_{dtype}", T=T, H=H, I=I, E=E, k=k, dtype=dtype, n_local=4, seed=91,
                          zipf_s=0.8, rho_seed=3)
    L = build_layer(cfg, pre_norm=pre_norm, training=True, **kw)
    rng = np.random.default_rng(12)
    if pre_norm:
        L.gamma.copy_(gpu(1 + 0.2 * rng.standard_normal(H)))
        L.beta.copy_(gpu(0.1 * rng.standard_normal(H)))
    return cfg, L, gpu(0.3 * rng.standard_normal((T, H)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre_norm", [True, False])
@pytest.mark.parametrize("remote", ["all", "device"])
def test_layer_training_step(dtype, pre_norm, remote):
    """Forward and backward of the layer, each step's output against the oracle on the values the
    step read; then the whole chain against the oracle's chain, to the type's precision."""
    cfg, L, dy = layer_case(dtype, pre_norm)
    log(f"case layer step {dtype} pre_norm={pre_norm} remote={remote}")
    try:
        torch.cuda.synchronize()
        L.forward(half=1, remote=remote)
        L.backward(dy, half=1)
        assert L.read_status() == 0
        T, H, I, E, k = cfg.T, cfg.H, cfg.I, cfg.E, cfg.k
        half = HALF[dtype]
        slots = L.slot_maps[1].cpu().numpy()
        counts = L.counts.cpu().numpy()
        inp = dict(x=host(L.x_perm), dy=host(L.dy_perm), offsets=L.offsets.cpu().numpy(),
                   slots=[int(s) for s in slots],
                   w=np.zeros((L.n_slots, 3 * H * I)))
        for e in range(E):
            if slots[e] >= 0:
                inp["w"][slots[e]] = host(L.expert_block(e))
        check_experts(tuple(int(c) for c in counts), H, I, dtype, inp, L.dx_perm, L.dw)
        row_of = L.row_of.cpu().numpy()
        ref = G.permute_backward(host(L.dx_perm), row_of, k)
        f32 = k * U * G.permute_backward(np.abs(host(L.dx_perm)), row_of, k)
        check("dxn", L.dxn, ref, half * (np.abs(ref) + f32) + f32)
        check("dlogits", L.dlogits,
              G.route_backward(L.topk_idx.cpu().numpy(), host(L.topk_w), host(L.dtopk_w), E),
              np.full((T, E), 16 * U * 2 * np.abs(host(L.dtopk_w)).max()))
        # the chain from the layer's inputs: every rounding on the way is half a step of dtype, so
        # the 2-norm of each gradient is off by a few of them (8 covers xn, x_perm, h, dy_perm,
        # dg / du, dx_perm, dxn and dx each once), f32 sums of depth below 512 included
        eps = 1e-5
        x = host(L.x)
        gamma = host(L.gamma) if pre_norm else None
        xn = G.layer_norm(x, gamma, host(L.beta), eps)[0] if pre_norm else x
        tw, idx = host(L.topk_w), L.topk_idx.cpu().numpy()
        src_of = L.src_of.cpu().numpy()
        off = inp["offsets"]
        block = lambda e: host(L.expert_block(e))
        yp = O.grouped_swiglu(xn[src_of // k], off, block, H, I, False)
        dyp, dtw = G.combine_backward(host(dy), yp, row_of, tw, k)
        ex = G.grouped_swiglu_backward(xn[src_of // k], dyp, off, block, H, I)
        dxn = G.permute_backward(ex["dx_perm"], row_of, k)
        norm = np.linalg.norm
        pairs = [("dtopk_w", L.dtopk_w, dtw), ("dxn", L.dxn, dxn)]
        pairs += [(f"dw[{e}]", L.dw[slots[e]], ex["dw"][e]) for e in range(E) if slots[e] >= 0 and counts[e]]
        if pre_norm:
            dx, dg, db = G.layer_norm_backward(dxn, x, gamma, *G.layer_norm(x, gamma, None, eps)[1:])
            pairs += [("dx", L.dx, dx), ("dgamma", L.dgamma, dg), ("dbeta", L.dbeta, db)]
        for name, got, want in pairs:
            off_by = norm(host(got) - want) / norm(want)
            log(f"  chain {name}: {off_by:.2e}")
            assert off_by <= 8 * half + 512 * U, name
    finally:
        L.close()


def test_layer_router_reads_the_normed_rows():
    """The split calls: norm, logits from xn, forward(normed=True), backward_experts, the router's
    own gradient added to dxn, backward_norm."""
    cfg, L, dy = layer_case("f32", True)
    T, H, E, k = cfg.T, cfg.H, cfg.E, cfg.k
    try:
        rng = np.random.default_rng(4)
        wr = gpu(rng.standard_normal((E, H)) * H ** -0.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(L.compute_stream):
            L.norm()
            L.logits.copy_(L.xn @ wr.t())
            L.forward(remote="all", normed=True)
            L.backward_experts(dy)
            L.dxn.add_(L.dlogits @ wr)
            L.backward_norm()
        assert L.read_status() == 0
        x, gamma, beta = host(L.x), host(L.gamma), host(L.beta)
        xn, mean, rstd = G.layer_norm(x, gamma, beta, 1e-5)
        idx, row_of, src_of = (t.cpu().numpy() for t in (L.topk_idx, L.row_of, L.src_of))
        logits = xn @ host(wr).T
        z = np.take_along_axis(logits, idx.astype(np.int64), 1)
        tw = np.exp(z - z.max(1, keepdims=True))
        tw /= tw.sum(1, keepdims=True)
        off = L.offsets.cpu().numpy()
        block = lambda e: host(L.expert_block(e))
        yp = O.grouped_swiglu(xn[src_of // k], off, block, H, cfg.I, False)
        dyp, dtw = G.combine_backward(host(dy), yp, row_of, tw, k)
        ex = G.grouped_swiglu_backward(xn[src_of // k], dyp, off, block, H, cfg.I)
        dxn = G.permute_backward(ex["dx_perm"], row_of, k) + G.route_backward(idx, tw, dtw, E) @ host(wr)
        dx = G.layer_norm_backward(dxn, x, gamma, mean, rstd)[0]
        off_by = np.linalg.norm(host(L.dx) - dx) / np.linalg.norm(dx)
        log(f"  dx: {off_by:.2e}")
        assert off_by <= 1024 * U                    # f32 throughout, sums of depth below 1024
    finally:
        L.close()


@pytest.mark.parametrize("fused_gather", [False, True])
def test_layer_reads_the_x_that_is_there(fused_gather):
    """Without pre_norm the step reads the layer's x at the time of the step, also another tensor
    that a caller has put in its place."""
    cfg = synth.MoEConfig("other_x", T=50, H=64, I=32, E=8, k=2, dtype="bf16", n_local=4, seed=3)
    L = build_layer(cfg, fused_gather=fused_gather)
    try:
        L.forward(remote="all")
        L.synchronize()
        y = L.y.clone()
        other = L.x.clone()
        L.x.zero_()
        L.x = other
        L.y.fill_(float("nan"))
        torch.cuda.synchronize()
        L.forward(remote="all")
        L.synchronize()
        assert torch.equal(L.y, y)
    finally:
        L.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_training_step_without_tokens(dtype):
    """An empty batch: every gradient of a parameter that the half holds is zero."""
    cfg, L, dy = layer_case(dtype, True, T=0)
    try:
        for t in (L.dw, L.dgamma, L.dbeta):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        L.forward(half=0, remote="all")
        L.backward(dy, half=0)
        assert L.read_status() == 0
        assert not L.dgamma.any() and not L.dbeta.any()
        assert not L.dw[L.slot_maps[0].long()].any()
        assert L.dx.shape == (0, cfg.H) and L.dlogits.shape == (0, cfg.E)
    finally:
        L.close()


def test_layer_training_refusals():
    cfg, L, dy = layer_case("bf16", False)
    try:
        for bad in (dy[:-1], dy.t().contiguous().t(), dy.half(), dy.cpu()):
            with pytest.raises(ValueError):
                L.backward(bad)
    finally:
        L.close()
    with pytest.raises(ValueError):
        layer_case("bf16", False, fused_gather=True)
    plain = build_layer(cfg)
    try:
        with pytest.raises(ValueError):
            plain.backward(dy)
    finally:
        plain.close()


def test_training_step_graph_replay():
    """Forward and backward captured together, replayed on new inputs with eager work in between:
    every replay gives the eager call's bits."""
    cfg, L, dy = layer_case("bf16", True)
    cfg2, M, _ = layer_case("bf16", True)
    names = ["y", "dx", "dlogits", "dw", "dgamma", "dbeta"]
    try:
        for step in (L, M):
            step.set_inputs(synth.activations(cfg, 0), synth.logits(cfg, 0))
            step.forward(remote="device")            # first calls outside the capture
            step.backward(dy)
            step.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=L.compute_stream, capture_error_mode="relaxed"):
            L.route_permute()
            L.fill_half_routed_on_device(0, wait_free=False)
            L.expert_compute(0)
            L.backward(dy)
        for turn in range(4):
            for step in (L, M):
                step.set_inputs(synth.activations(cfg, turn), synth.logits(cfg, turn))
            L.dw.fill_(float("nan"))
            torch.cuda.synchronize()
            with torch.cuda.stream(L.compute_stream):
                g.replay()
            M.forward(remote="device")
            M.dw.fill_(float("nan"))
            torch.cuda.synchronize()
            M.backward(dy)
            L.synchronize(), M.synchronize()
            for n in names:
                a, b = getattr(L, n), getattr(M, n)
                if n == "dw":                        # slots of absent experts are left alone
                    live = L.slot_maps[0] >= 0
                    a, b = a[live], b[live]
                assert torch.equal(a, b), (turn, n)
            torch.randn(1 << 20, device="cuda").sum().item()
    finally:
        L.close()
        M.close()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, do not disturb each other."""
    counts, H, I = (200, 0, 90, 33), 264, 136
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, dxa, dwa, _ = run_experts(counts, H, I, "bf16", 21, stream=s1)
    b, dxb, dwb, _ = run_experts(counts, H, I, "bf16", 22, stream=s2)
    ref = [t.clone() for t in (dxa, dwa, dxb, dwb)]
    for t in (dxa, dwa, dxb, dwb):
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        a["call"]()
        b["call"]()
    torch.cuda.synchronize()
    for t, r in zip((dxa, dwa, dxb, dwb), ref):
        assert torch.equal(t, r)
