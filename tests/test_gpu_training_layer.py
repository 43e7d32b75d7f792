"""The layer's training step on the GPU where the caller takes part in it, where its
expert set changes from step to step, and from halves stitched out of pages."""
import pytest

import test_gpu_backward as base
from moe_cases import log, synth

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("remote,n_slots", [("routed", 12), ("routed", 8), ("device", 12)])
def test_slots_without_an_expert_hold_zeros(dtype, remote, n_slots):
    """Steps of a few tokens whose routed experts change: after each, a slot's block of dw is the
    gradient of the expert that the step's slot map puts there (the same bits as in a layer that holds
    every expert) and zero where it puts none; the gradient of an expert without a slot is zero."""
    cfg, L, dy = base.layer_case(dtype, True, T=2, k=2, n_slots=n_slots)
    cfg, M, _ = base.layer_case(dtype, True, T=2, k=2)
    log(f"case slots without an expert {dtype} remote={remote} n_slots={n_slots}")
    seen, left_free = set(), 0
    try:
        L.dw.fill_(float("nan"))
        torch.cuda.synchronize()
        for turn in range(4):
            for step, how in ((L, remote), (M, "all")):
                step.set_inputs(synth.activations(cfg, turn), synth.logits(cfg, turn))
                step.forward(half=turn % 2, remote=how)
                step.backward(dy, half=turn % 2)
                assert step.read_status() == 0
            slots = L.slot_maps[turn % 2].tolist()
            seen.add(tuple(slots))
            free = sorted(set(range(n_slots)) - set(slots))
            left_free += len(free)               # 8 slots: 4 local and 4 routed experts fill them all
            for e, s in enumerate(slots):
                if s >= 0:
                    assert torch.equal(L.dw[s], M.dw[e]), (turn, e)
                else:
                    assert not M.dw[e].any(), (turn, e)
            assert not L.dw[free].any(), turn
        assert len(seen) > 1 and left_free
    finally:
        L.close()
        M.close()


def test_slots_without_an_expert_hold_zeros_after_a_replay():
    """The device-routed training step as a graph, replayed on inputs that route to other experts."""
    cfg, L, dy = base.layer_case("bf16", True, T=2, k=2)
    try:
        L.forward(remote="device")
        L.backward(dy)
        L.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=L.compute_stream, capture_error_mode="relaxed"):
            L.route_permute()
            L.fill_half_routed_on_device(0, wait_free=False)
            L.expert_compute(0)
            L.backward(dy)
        for turn in range(4):
            L.set_inputs(synth.activations(cfg, turn), synth.logits(cfg, turn))
            L.dw.fill_(float("nan"))
            torch.cuda.synchronize()
            with torch.cuda.stream(L.compute_stream):
                g.replay()
            L.synchronize()
            none = L.slot_maps[0] < 0                # slot = expert id
            assert none.any() and not L.dw[none].any()
            assert torch.isfinite(L.dw).all()
            torch.randn(1 << 20, device="cuda").sum().item()
    finally:
        L.close()


@pytest.mark.parametrize("words", [4, 6, 13, 1 << 18, (1 << 18) + 4, (1 << 19) + 3])
@pytest.mark.parametrize("E,slots,n_slots", [(5, (3, -1, 7, 4, 0), 4), (3, (-1, -1, -1), 2),
                                             (300, tuple(range(299, -1, -1)), 301), (2, (1, 0), 2)])
def test_clear_unmapped(words, E, slots, n_slots):
    """Blocks of a slot without an expert become zero, every other word stays as it was."""
    if n_slots * words > 1 << 24:
        words = 13
    B = base.B_()
    log(f"case clear {n_slots} slots of {words} words, {E} experts")
    held = torch.arange(1, n_slots * words + 65, dtype=torch.int32, device="cuda")
    dw = torch.cat([held[-1:], held])[1:]                # starts 4 bytes into an allocation
    B.moe_clear_unmapped(B.wbuf(None, 4 * words, n_slots, E, base.i32(slots)), dw)
    torch.cuda.synchronize()
    want = held.clone()
    for s in set(range(n_slots)) - set(slots):
        want[s * words:(s + 1) * words] = 0
    assert torch.equal(dw, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("remote,chunks", [("all", 0), ("all", 3), ("device", 0), ("routed", 0),
                                           ("routed", 3)])
def test_training_step_from_stitched_halves(dtype, remote, chunks):
    """Halves stitched from pages hold the same bytes as copied ones: the step and every gradient
    agree bit for bit, block by expert, over several steps on both halves."""
    size = dict(T=40, H=1024, I=1024)                    # whole pages: blocks of 6 and 12 MiB
    cfg, L, dy = base.layer_case(dtype, True, stitched=True, **size)
    cfg, M, _ = base.layer_case(dtype, True, **size)
    log(f"case stitched training step {dtype} remote={remote} chunks={chunks}")
    try:
        for turn in range(3):
            half = turn % 2
            for step, how, n in ((L, remote, chunks), (M, "all", 0)):
                step.set_inputs(synth.activations(cfg, turn), synth.logits(cfg, turn))
                step.forward(half=half, remote=how, chunks=n)
                step.backward(dy, half=half)
                assert step.read_status() == 0
            for name in ("y", "dx", "dlogits", "dgamma", "dbeta"):
                assert torch.equal(getattr(L, name), getattr(M, name)), (turn, name)
            assert torch.isfinite(L.dx).all() and L.dx.any()
            for e, s in enumerate(L.slot_maps[half].tolist()):
                assert torch.equal(L.dw[s], M.dw[e]) if s >= 0 else not M.dw[e].any(), (turn, e)
    finally:
        L.close()
        M.close()
