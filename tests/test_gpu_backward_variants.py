"""The training pass at the sizes that choose its other kernel variants: the 256 x 256 tile of the
bf16 experts in every row mode, the layer norm that keeps gamma and beta from row to row, teams of the
norm's backward pass that take several turns.  Oracle, checks and tolerances are those of
``test_gpu_backward``."""
import numpy as np
import pytest

import test_gpu_backward as base
from moe_cases import log
from test_gpu_backward import check_experts, run_experts

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
_free_gpu = base._free_gpu


def ceil_div(a, b):
    return -(-a // b)


def takes_large_tiles(counts, H, I):
    """The rule of the bf16 experts: 256 x 256 tiles when dH and dX have one for every CU."""
    R = sum(counts)
    tiles = ceil_div(R, 256) + min(len(counts), R)
    return tiles * (ceil_div(H, 256) + ceil_div(I, 256)) >= 256


def mixed(E, seed):
    """Rows of E experts on both sides of each row mode's limit (32, 64, 128, 192, 256), some none."""
    rng = np.random.default_rng(seed)
    edges = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 0, 5, 90]
    return tuple(int(c) for c in rng.permutation((edges * (E // len(edges) + 1))[:E]))


EDGES = (1, 32, 33, 0, 64, 65, 128, 129, 192, 193, 255, 256, 257, 31, 300)
FEW = tuple(int(c) for c in np.random.default_rng(2).integers(0, 6, 130))
MANY = tuple(int(c) for c in np.random.default_rng(4).integers(0, 4, 1024))
LARGE = [
    (EDGES, 1544, 1032),             # every row mode; depths that end inside a stage, ragged columns
    (mixed(90, 1), 264, 136),        # many experts, two column tiles and one
    (FEW, 520, 264),                 # a few rows each: units of 4 row tiles, the last of them ragged
    (mixed(64, 3), 2312, 72),        # ten column tiles: two units across, of five
    ((1025,), 8200, 4104),           # a weight gradient of several units each way
    (FEW, 8, 24),                    # the narrowest rows
    (MANY, 72, 40),                  # sixteen experts a lane in the tile search
]


@pytest.mark.parametrize("counts,H,I", LARGE, ids=["edges", "mixed", "few", "wide", "one", "narrow", "many"])
def test_grouped_swiglu_backward_large_tiles(counts, H, I):
    assert takes_large_tiles(counts, H, I)
    log(f"case experts backward {len(counts)} experts, {sum(counts)} rows, H={H} I={I} bf16, large tiles")
    inp, dx, dw, status = run_experts(counts, H, I, "bf16", 120 + H + I)
    assert status == 0
    check_experts(counts, H, I, "bf16", inp, dx, dw)
    first = (dx.clone(), dw.clone())
    inp["call"]()                                   # on the workspace the first call left
    torch.cuda.synchronize()
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw)


@pytest.mark.parametrize("seed", range(4))
def test_grouped_swiglu_backward_large_tiles_random(seed):
    rng = np.random.default_rng(900 + seed)
    H, I = (8 * int(rng.integers(20, 120)) for _ in range(2))
    counts = []
    while not takes_large_tiles(counts, H, I):
        counts.append(int(rng.integers(0, [8, 70, 300, 600][seed])))
    counts = tuple(counts)
    log(f"case experts backward rows={counts} H={H} I={I} bf16, large tiles")
    inp, dx, dw, status = run_experts(counts, H, I, "bf16", 950 + seed)
    assert status == 0
    check_experts(counts, H, I, "bf16", inp, dx, dw)


COUNTS = mixed(90, 5)


def test_large_tiles_only_one_output():
    H, I = 264, 136
    assert takes_large_tiles(COUNTS, H, I)
    _, dx, dw, _ = run_experts(COUNTS, H, I, "bf16", 5)
    _, dx2, none, _ = run_experts(COUNTS, H, I, "bf16", 5, want=("dx",))
    assert none is None and torch.equal(dx, dx2)
    _, none, dw2, _ = run_experts(COUNTS, H, I, "bf16", 5, want=("dw",))
    assert none is None and torch.equal(dw, dw2)


def test_large_tiles_absent_slots_and_untouched_memory():
    """Every seventh expert has no slot or one past the buffer, slots are permuted, two blocks
    belong to nobody, 9 rows follow the last expert's."""
    B = base.B_()
    H, I, E = 264, 136, len(COUNTS)
    assert takes_large_tiles(COUNTS, H, I)
    slots = [int(s) for s in np.random.default_rng(6).permutation(E + 2)[:E]]
    gone = list(range(3, E, 7))
    for i, e in enumerate(gone):
        slots[e] = -1 if i % 2 else E + 2 + i
    assert any(COUNTS[e] for e in gone)
    inp, dx, dw, status = run_experts(COUNTS, H, I, "bf16", 6, slots=slots, n_slots=E + 2, tail_rows=9)
    assert status == B.MOE_STATUS_EXPERT_ABSENT
    inp["slots"] = [-1 if e in gone else s for e, s in enumerate(slots)]
    check_experts(COUNTS, H, I, "bf16", inp, dx, dw)
    off = inp["offsets"]
    for e in gone:
        assert torch.isnan(dx[off[e]:off[e + 1]]).all()
    assert torch.isnan(dx[off[E]:]).all()
    for s in range(E + 2):
        held = dw[s]
        assert (torch.isfinite(held) if s in inp["slots"] else torch.isnan(held)).all(), s


def test_large_tiles_neighbours_nan_and_infinity_stay_out():
    H, I = 264, 136
    assert takes_large_tiles(COUNTS, H, I)
    inp, dx, dw, _ = run_experts(COUNTS, H, I, "bf16", 8)
    clean = dx.clone(), dw.clone()
    xt, dyt, ot, wt, slot_of, ws = inp["keep"]
    off, bad = inp["offsets"], [e for e in range(2, len(COUNTS), 5) if COUNTS[e]]
    for e in bad:
        xt[off[e]:off[e + 1], ::3] = float("nan")
        dyt[off[e]:off[e + 1], 1::3] = float("inf")
        wt[e, ::5] = float("nan")
    inp["call"]()
    torch.cuda.synchronize()
    for e in range(len(COUNTS)):
        if e not in bad:
            assert torch.equal(dx[off[e]:off[e + 1]], clean[0][off[e]:off[e + 1]]), e
            assert torch.equal(dw[e], clean[1][e]), e


def test_large_tiles_graph_replay_and_two_streams():
    """Two captured calls with workspaces of their own, replayed on two streams at once with eager
    work between the replays, on outputs and inputs that change."""
    H, I = 264, 136
    assert takes_large_tiles(COUNTS, H, I)
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [run_experts(COUNTS, H, I, "bf16", 30 + i, stream=s) for i, s in enumerate(streams)]
    graphs = []
    for (inp, _, _, _), s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
            inp["call"]()
        graphs.append(g)
    for turn in range(3):
        want = []
        for inp, dx, dw, _ in calls:
            inp["keep"][0].mul_(-0.5)                # x
            torch.cuda.synchronize()
            inp["call"]()
            torch.cuda.synchronize()
            want.append((dx.clone(), dw.clone()))
            dx.fill_(float("nan"))
            dw.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, dx, dw, _), (rdx, rdw) in zip(calls, want):
            assert torch.equal(dx, rdx) and torch.equal(dw, rdw), turn
        torch.randn(1 << 20, device="cuda").sum().item()


# More rows than two rounds of resident blocks, so a block keeps gamma and beta and takes three rows
# or more: over 8192 rows of up to 1024, 4096 of up to 2048, 1024 of 7168, 512 of 16384.
KEPT = [(13000, 200, "bf16", 0), (8200, 77, "f32", 1), (9000, 513, "f32", 0), (8700, 1000, "bf16", 0),
        (4200, 2048, "bf16", 0), (9000, 1025, "f32", 3), (1100, 7168, "bf16", 0), (1700, 7161, "f32", 1),
        (1030, 7168, "f32", 0), (600, 16384, "bf16", 0), (600, 16377, "f32", 1)]


def kept(T, H):
    """The norm's rule for several rows a block (two vectors of 8 columns a lane over 512 columns)."""
    waves = ceil_div(H, 512 if H <= 512 else 1024)
    rows = 4 if waves == 1 else 1
    return ceil_div(T, rows) > 2 * 256 * max(1, 16 // (waves * rows))


@pytest.mark.parametrize("T,H,dtype,pad", KEPT)
def test_layer_norm_many_rows(T, H, dtype, pad):
    assert kept(T, H)
    base.test_layer_norm(T, H, dtype, pad)


# Teams that take three turns or more: the sums' LDS buffers are used again (over 512 rows of more
# than 4096, fewer columns more rows), with one vector a lane and with two.
@pytest.mark.parametrize("T,H,dtype,pad", [
    (12500, 200, "f32", 0), (3000, 2056, "bf16", 5), (1600, 4001, "f32", 1), (800, 4099, "bf16", 3),
    (800, 4104, "f32", 0), (530, 8192, "bf16", 0), (600, 9001, "bf16", 1), (600, 9008, "f32", 0),
    (520, 16384, "bf16", 0), (520, 16383, "f32", 1)])
def test_layer_norm_backward_many_rows(T, H, dtype, pad):
    waves = ceil_div(H, 512 if H <= 8192 else 1024)
    assert T > 2 * 256 * max(1, 16 // waves)
    base.test_layer_norm_backward(T, H, dtype, pad)
