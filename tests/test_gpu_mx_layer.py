"""The 8-bit block (``mx_layer.MxMoELayer``) on the GPU: each step against ``oracle.block`` in float64 on what
the step before stored, its graph, and its refusals.  Tolerances as in test_gpu_grouped_gemm."""
import numpy as np
import pytest

from moe_cases import O, log, synth
from oracle import block as K8
from test_gpu_backward import HALF, U, check, gpu, host
from test_gpu_grouped_gemm import largest_of_eight

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def layer(T, H, I, E, k, dtype, seed):
    from grouped_gemm_weights_amd.mx_layer import MxMoELayer
    cfg = synth.MoEConfig("mx", T=T, H=H, I=I, E=E, k=k, dtype=dtype, n_local=E, seed=seed)
    L = MxMoELayer(cfg)
    rng = np.random.default_rng(seed)
    for e in range(E):
        w = rng.standard_normal(3 * H * I) * H ** -0.5
        w[2 * H * I:] *= (H / I) ** 0.5
        L.load_expert(e, gpu(w, dtype))
    return cfg, L, rng


def inputs(L, rng, dtype):
    cfg = L.cfg
    L.x.copy_(gpu(rng.standard_normal((cfg.T, cfg.H)), dtype))
    L.residual.copy_(gpu(0.5 * rng.standard_normal((cfg.T, cfg.H)), dtype))
    L.gamma.copy_(gpu(1 + 0.2 * rng.standard_normal(cfg.H)))
    L.logits.copy_(gpu(rng.standard_normal((cfg.T, cfg.E))))
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H,I,E,k,dtype", [(1, 64, 32, 4, 2, "bf16"), (64, 544, 288, 9, 3, "bf16"),
                                             (700, 256, 192, 4, 2, "bf16"), (40, 96, 160, 5, 2, "f32"),
                                             (0, 64, 32, 4, 2, "bf16")])
def test_step(T, H, I, E, k, dtype):
    log(f"case mx layer T={T} H={H} I={I} E={E} k={k} {dtype}")
    cfg, L, rng = layer(T, H, I, E, k, dtype, 3 + T)
    inputs(L, rng, dtype)
    L.norm()
    L.forward()
    assert L.read_status() == 0
    half = HALF[dtype]
    n = lambda t: t.cpu().numpy()
    total = (host(L.x).astype(np.float32) + host(L.residual).astype(np.float32))
    assert torch.equal(L.sum.cpu(), torch.from_numpy(total).to(L.sum.dtype))
    xn, _ = K8.rms_norm(host(L.sum), host(L.gamma), L.eps)
    check("xn", L.xn, xn, (half + 80 * U) * np.abs(xn))
    idx, w = O.route(n(L.logits), k) if T else (n(L.topk_idx), n(L.topk_w))
    assert (np.asarray(idx) == n(L.topk_idx)).all()
    off, src = n(L.offsets), n(L.src_of)
    b = n(L.blocks)

    def matrix(e, at, scales, rows, cols):
        p = K8.pitch(cols)
        return K8.decode(b[e, at:at + rows * cols].reshape(rows, cols), b[e, scales:scales + rows * p].reshape(rows, p))

    wu = np.stack([matrix(e, 0, L.up_scales_off, 2 * I, H) for e in range(E)])
    wd = np.stack([matrix(e, L.down_off, L.down_scales_off, H, I) for e in range(E)])
    q = K8.decode(n(L.q), n(L.scales))[src // k]
    ref, tol = K8.grouped_gemm(q, off, wu), H * U * K8.grouped_gemm(np.abs(q), off, np.abs(wu))
    if dtype == "bf16":
        for e in range(E):
            rows = slice(int(off[e]), int(off[e + 1]))
            tol[rows] += 7 * 2.0 ** -13 * largest_of_eight(q[rows], wu[e])
    check("gate and up", L.gate_up, ref, half * (np.abs(ref) + tol) + tol)
    h = K8.decode(n(L.h), n(L.h_scales))
    v = K8.swiglu(host(L.gate_up))
    assert np.linalg.norm(h - v) <= 2.0 ** -4 * np.linalg.norm(v)
    check("down", L.y_perm, K8.grouped_gemm(h, off, wd), I * U * K8.grouped_gemm(np.abs(h), off, np.abs(wd)))
    y = O.combine(host(L.y_perm), n(L.row_of), host(L.topk_w), k)
    size = O.combine(np.abs(host(L.y_perm)), n(L.row_of), host(L.topk_w), k)
    check("y", L.y, y, (k + 1) * U * size)
    out = host(L.sum) + host(L.y)
    check("out", L.out, out, half * np.abs(out) + 2 * U * (np.abs(out) + np.abs(host(L.y))))


def test_graph_replay():
    """forward captured, replayed on new rows and logits with eager work in between: the eager bits."""
    cfg, L, rng = layer(50, 96, 64, 6, 2, "bf16", 8)
    inputs(L, rng, "bf16")
    L.norm()
    L.forward()
    g = L.capture()
    for turn in range(4):
        inputs(L, rng, "bf16")
        L.norm()
        L.y.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(L.compute_stream):
            g.replay()
        L.compute_stream.synchronize()
        got = L.y.clone(), L.out.clone()
        L.forward()
        assert L.read_status() == 0
        assert torch.equal(got[0], L.y) and torch.equal(got[1], L.out), turn
        torch.randn(1 << 20, device="cuda").sum().item()


def test_experts_pulled_from_a_pool():
    """Blocks in another order in a pool, pulled by the routed prefetch into the layer's buffer."""
    from grouped_gemm_weights_amd import binding as B
    cfg, L, rng = layer(30, 96, 64, 6, 2, "bf16", 9)
    inputs(L, rng, "bf16")
    L.norm()
    L.forward()
    L.compute_stream.synchronize()
    y = L.y.clone()
    pool = L.blocks.clone()
    L.blocks.fill_(0x7F)
    torch.cuda.synchronize()
    B.moe_prefetch_routed(B.pool(pool, L.expert_bytes, 0, cfg.E), L.counts, L.wbuf, L.compute_stream)
    L.forward()
    assert L.read_status() == 0
    assert torch.equal(L.y, y)


def test_refusals():
    from grouped_gemm_weights_amd.mx_layer import MxMoELayer
    with pytest.raises(ValueError):
        MxMoELayer(synth.MoEConfig("mx", T=2, H=40, I=32, E=2, k=1, dtype="bf16", n_local=2, seed=0))
    cfg, L, _ = layer(2, 64, 32, 2, 1, "bf16", 1)
    block = torch.zeros(3 * 64 * 32, dtype=torch.bfloat16, device="cuda")
    for e, bad in ((2, block), (-1, block), (0, block[:-1]), (0, block.float()), (0, block.cpu())):
        with pytest.raises(ValueError):
            L.load_expert(e, bad)


def test_experts_that_nobody_loaded():
    """Their tokens come out NaN, all others as with every expert loaded; a pull into their slots mends them."""
    from grouped_gemm_weights_amd import binding as B
    from grouped_gemm_weights_amd.mx_layer import MxMoELayer
    T, H, I, E, k, missing = 60, 96, 64, 6, 2, (1, 4)
    cfg, full, rng = layer(T, H, I, E, k, "bf16", 10)
    inputs(full, rng, "bf16")
    part = MxMoELayer(cfg)
    part.blocks[[e for e in range(E) if e not in missing]] = full.blocks[[e for e in range(E) if e not in missing]]
    for name in ("x", "residual", "gamma", "logits"):
        getattr(part, name).copy_(getattr(full, name))
    torch.cuda.synchronize()
    for L in (full, part):
        L.norm()
        L.forward()
        assert L.read_status() == 0
    idx = full.topk_idx.cpu().numpy()
    hit = torch.from_numpy(np.isin(idx, missing).any(1)).cuda()
    assert 0 < int(hit.sum()) < T
    assert torch.isfinite(full.y).all() and torch.isnan(part.y[hit]).all() and torch.isnan(part.out[hit]).all()
    assert torch.equal(part.y[~hit], full.y[~hit]) and torch.equal(part.out[~hit], full.out[~hit])
    B.moe_prefetch_routed(B.pool(full.blocks, full.expert_bytes, 0, E), part.counts, part.wbuf, part.compute_stream)
    part.forward()
    assert part.read_status() == 0
    assert torch.equal(part.y, full.y) and torch.equal(part.out, full.out)


def test_experts_loaded_through_one_buffer():
    """The caller's next write to the block waits until the compute stream, busy with other work, has read it."""
    from grouped_gemm_weights_amd.mx_layer import MxMoELayer
    H, I, E = 256, 192, 5
    cfg = synth.MoEConfig("mx", T=8, H=H, I=I, E=E, k=2, dtype="bf16", n_local=E, seed=11)
    one, each = MxMoELayer(cfg), MxMoELayer(cfg)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    weights = [torch.randn(3 * H * I, generator=g, device="cuda").to(torch.bfloat16) for _ in range(E)]
    busy, out = torch.randn(4096, 4096, device="cuda"), torch.empty(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for e in range(E):
        each.load_expert(e, weights[e])
        torch.cuda.synchronize()
    block = torch.empty(3 * H * I, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        with torch.cuda.stream(one.compute_stream):
            for _ in range(3):
                torch.mm(busy, busy, out=out)
        block.copy_(weights[e])
        one.load_expert(e, block)
    block.fill_(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(one.blocks, each.blocks)
