"""The products by expert on the GPU, their gradient and the 8-bit form, against ``oracle.block`` in
float64, through the C ABI, element by element.

Tolerances (u = 2^-24; HALF as in test_gpu_backward): a product sum of depth K in fp32 is off by at most
K u sum|a b|, an output stored in bf16 by half a step more.  Products of two e4m3 values have at most
eight significant bits and their scales are powers of two, so the 8-bit form rounds only its sums.

With a bf16 output the 8-bit form runs on the 8-bit MFMA (with an f32 one on exact products).  It adds the products of eight consecutive values at
once, each cut below 2^-13 of the largest power of two in them (the exponents' sum, which is at most
the product): seven of them are off by less than 2^-13 max|a b| each, the largest not at all.
"""
import gc

import numpy as np
import pytest

from moe_cases import O, log
from oracle import block as K8
from test_gpu_backward import HALF, U, blank, check, code, gpu, host, i32

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


def to8(v):
    """(bytes, scale bytes) of the rows of v on the host."""
    q, s = K8.quantize(v)
    return torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), s


def largest_of_eight(x, w):
    """sum over groups of eight consecutive k of max|x_k w_k| for each row of x and of w (at large sizes
    the sum of all of them, which is no less)."""
    x, w = np.abs(x).astype(np.float32), np.abs(w).astype(np.float32)
    if x.shape[0] * w.shape[0] * x.shape[1] > 3e8:
        return (x @ w.T).astype(np.float64)
    total = np.zeros((x.shape[0], w.shape[0]))
    for k in range(0, x.shape[1], 8):
        top = x[:, k, None] * w[None, :, k]
        for i in range(k + 1, k + 8):
            np.maximum(top, x[:, i, None] * w[None, :, i], out=top)
        total += top
    return total


class Case:
    """Inputs of one product: rows by expert, permuted slots, matrices at an offset of larger blocks."""

    def __init__(self, counts, K, N, dtype, seed, gather=0, slots=None, n_slots=None, tail=0, lead=0, out="f32"):
        B = B_()
        rng = np.random.default_rng(seed)
        self.counts, self.K, self.N, self.dtype, self.out = counts, K, N, dtype, out
        E = self.E = len(counts)
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        R = self.R = int(self.offsets[-1]) + tail
        self.slots = list(rng.permutation(E)) if slots is None else slots
        n_slots = E if n_slots is None else n_slots
        self.src = None
        n_x = R
        if gather:                          # rows of a smaller x, each taken several times
            n_x = -(-R // gather)
            self.src = (rng.integers(0, n_x, R) * gather + rng.integers(0, gather, R)).astype(np.int32)
        self.gather = gather
        x = rng.standard_normal((n_x, K))
        w = rng.standard_normal((n_slots, N, K)) * K ** -0.5
        if dtype == "mx":
            self.block = lead + N * K + N * K8.pitch(K) + 16
            blocks = np.full((n_slots, self.block), 0x7F, np.uint8)         # NaN around the matrices
            xq, xs = to8(x * 2.0 ** rng.integers(-6, 6, (n_x, 1)))
            self.x = K8.decode(xq, xs)
            self.w = np.zeros_like(w)
            for e in range(n_slots):
                q, s = to8(w[e])
                self.w[e] = K8.decode(q, s)
                blocks[e, lead:lead + N * K] = q.reshape(-1)
                blocks[e, lead + N * K:lead + N * K + s.size] = s.reshape(-1)
            self.w_off, self.s_off = lead, lead + N * K
            self.xt, self.xs, self.wt = (torch.from_numpy(t).cuda() for t in (xq, xs, blocks))
        else:
            size = 4 if dtype == "f32" else 2
            self.x, self.w = host(gpu(x, dtype)), host(gpu(w, dtype))
            blocks = np.full((n_slots, lead // size + N * K + 16 // size), np.nan)
            blocks[:, lead // size:lead // size + N * K] = self.w.reshape(n_slots, -1)
            self.block, self.w_off = blocks.shape[1] * size, lead
            self.xt, self.wt = gpu(self.x, dtype), gpu(blocks, dtype)
        self.srct = None if self.src is None else i32(self.src)
        self.offt, self.slott = i32(self.offsets), i32(self.slots)
        self.buf = B.wbuf(self.wt, self.block, n_slots, E, self.slott)
        self.y = blank((R, N), out)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rows = self.x if self.src is None else self.x[self.src // gather]

    def call(self, stream=None, y=None):
        B = B_()
        y = self.y if y is None else y
        if self.dtype == "mx":
            B.moe_grouped_gemm_mx(self.xt, self.xs, self.srct, self.gather, self.offt, self.R, self.E, self.K, self.N,
                                  self.buf, self.w_off, self.s_off, code(self.out), y, self.status, stream)
        else:
            B.moe_grouped_gemm(self.xt, self.srct, self.gather, self.offt, self.R, self.E, self.K, self.N,
                               code(self.dtype), self.buf, self.w_off, code(self.out), y, self.status, stream)

    def live(self):
        for e, n in enumerate(self.counts):
            s = self.slots[e]
            if 0 <= s < self.wt.shape[0]:
                yield e, slice(int(self.offsets[e]), int(self.offsets[e]) + n), self.w[s]

    def check(self):
        for e, rows, w in self.live():
            ref, size = self.rows[rows] @ w.T, np.abs(self.rows[rows]) @ np.abs(w).T
            f32 = self.K * U * size
            if self.dtype == "mx" and self.out == "bf16":
                f32 = f32 + 7 * 2.0 ** -13 * largest_of_eight(self.rows[rows], w)
                # over many values rounding to bf16, uniform within half a step of at most 2^-8, is below
                # 2^-8 / sqrt(3) in the 2-norm, and the cut far below
                if ref.size > 1000:
                    assert np.linalg.norm(host(self.y[rows]) - ref) <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12) * np.linalg.norm(ref)
            check(f"y of expert {e} ({ref.shape[0]} rows)", self.y[rows], ref, HALF[self.out] * (np.abs(ref) + f32) + f32)


# rows by expert: tiles of 1 to 64 rows.  These products are small enough for the 64 x 64 tiles whose depth
# is split over the waves; test_gpu_grouped_gemm_tiles has those of 64 x 256 and of 256 x 256
FEW = [(1,), (3, 0, 5), (1, 2, 0, 16, 17), (15, 33, 16, 20), (64, 40, 33, 65, 0, 1)]
MANY = [(300,), (33, 0, 400, 1), (64, 65, 255, 257), (191, 193, 128, 129, 31), (512, 5, 96, 160)]
SHAPES_MX = [(32, 8), (64, 72), (96, 264), (416, 136), (544, 520), (1024, 256), (1120, 24)]
SHAPES = [(8, 8), (72, 136), (264, 72), (520, 264), (1016, 40), (1024, 512)]


@pytest.mark.parametrize("K,N", SHAPES_MX)
@pytest.mark.parametrize("counts", FEW + MANY)
def test_mx(counts, K, N):
    log(f"case mx rows={counts} K={K} N={N}")
    for gather, out in ((0, "f32"), (3, "bf16")):
        c = Case(counts, K, N, "mx", 7 + K + N, gather=gather, lead=16 * (K % 3), out=out)
        c.call()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        c.check()
        again = blank(c.y.shape, out)
        c.call(y=again)
        assert torch.equal(c.y.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("counts", FEW + MANY)
def test_bf16(counts, K, N):
    log(f"case bf16 rows={counts} K={K} N={N}")
    for gather, out in ((0, "f32"), (2, "bf16")):
        c = Case(counts, K, N, "bf16", 9 + K + N, gather=gather, lead=16 * (K % 5), out=out)
        c.call()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        c.check()


@pytest.mark.parametrize("counts,K,N", [((1,), 1, 1), ((3, 0, 5), 17, 9), ((129, 1, 0, 40), 131, 77),
                                        ((64, 200), 256, 512), ((700, 1, 899, 500), 103, 901), ((2100,), 645, 130)])
@pytest.mark.parametrize("gather", [0, 2])
def test_f32(counts, K, N, gather):
    log(f"case f32 rows={counts} K={K} N={N} gather={gather}")
    c = Case(counts, K, N, "f32", 11 + K + N, gather=gather, lead=12)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("seed", range(6))
def test_random(seed, dtype):
    rng = np.random.default_rng(500 + seed)
    E = int(rng.integers(1, 12))
    counts = tuple(int(n) for n in rng.integers(0, [3, 30, 150, 400][seed % 4], E))
    if sum(counts) == 0:
        counts = counts[:-1] + (1,)
    unit = dict(mx=32, bf16=8, f32=1)[dtype]
    K = unit * int(rng.integers(1, 1000 // unit))
    N = (1 if dtype == "f32" else 8) * int(rng.integers(1, 400 // (1 if dtype == "f32" else 8)))
    gather = int(rng.integers(0, 4))
    out = "f32" if dtype == "f32" else ["f32", "bf16"][seed % 2]
    log(f"case {dtype} rows={counts} K={K} N={N} gather={gather} out={out}")
    c = Case(counts, K, N, dtype, 600 + seed, gather=gather, out=out)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("K,N", [(7168, 256), (2048, 7168)])
@pytest.mark.parametrize("counts", [(2, 9), (40, 20), (300, 200)])
def test_mx_long(counts, K, N):
    """The R1 sizes' depth and width."""
    log(f"case mx rows={counts} K={K} N={N}")
    c = Case(counts, K, N, "mx", 21, gather=2, out="bf16")
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("counts", [(20, 7, 0, 5, 14), (200, 77, 0, 50, 140)])
def test_absent_slots_and_untouched_memory(dtype, counts):
    """Expert 1 has rows and no slot, expert 3 a slot past the buffer, expert 2 neither; slots are
    permuted; 9 rows follow the last expert's and keep what they held."""
    B = B_()
    c = Case(counts, 64, 40, dtype, 6, slots=[3, -1, -1, 4, 0], n_slots=4, tail=9)
    c.call()
    torch.cuda.synchronize()
    assert int(c.status.item()) == B.MOE_STATUS_EXPERT_ABSENT
    c.check()
    off = c.offsets
    for lo, hi in ((off[1], off[2]), (off[3], off[4]), (off[5], off[5] + 9)):
        assert torch.isnan(c.y[lo:hi]).all()


@pytest.mark.parametrize("dtype", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("counts", [(20, 7, 3), (200, 77, 100)])
def test_gathered_rows_that_are_not_there(dtype, counts):
    """An index outside x reads as a row of zeros."""
    c = Case(counts, 64, 40, dtype, 12, gather=2)
    bad = [3, int(c.offsets[1]), int(c.offsets[3]) - 1]
    src = c.src.copy()
    src[bad] = [-1, -7, 2 * c.xt.shape[0]]
    c.srct.copy_(i32(src))
    c.call()
    torch.cuda.synchronize()
    c.rows = c.rows.copy()
    c.rows[bad] = 0
    c.check()
    assert not host(c.y)[bad].any()


@pytest.mark.parametrize("dtype", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("counts", [(20, 7, 3), (200, 77, 100)])
def test_neighbours_that_are_not_finite_stay_out(dtype, counts):
    """NaN in one expert's weights, and in one row, reach that expert's and that row's outputs alone,
    also where a row ends inside the depth that a tile takes at a time."""
    K = dict(mx=96, bf16=40, f32=37)[dtype]
    c = Case(counts, K, 72, dtype, 13, slots=[0, 1, 2])
    lead = int(c.offsets[1])
    if dtype == "mx":
        c.wt[1, :72 * K] = 0x7F
        c.xt[2] = 0x7F
        c.xs[2] = 0
    else:
        c.wt[1, :72 * K] = float("nan")
        c.xt[2] = float("inf")
    c.call()
    torch.cuda.synchronize()
    got = host(c.y)
    assert np.isnan(got[lead:int(c.offsets[2])]).all() and not np.isfinite(got[2]).any()
    keep = [r for r in range(c.R) if r != 2 and not lead <= r < c.offsets[2]]
    assert np.isfinite(got[keep]).all()


def test_offsets_past_the_rows_are_held_to_them():
    """offsets that name rows past R (a caller's mistake) never write past y."""
    c = Case((20, 30), 64, 40, "mx", 14)
    c.offt.copy_(i32([0, 20, 70]))
    c.call()
    torch.cuda.synchronize()
    c.check()
    behind = torch.as_strided(c.y, (32,), (1,), c.y.storage_offset() + c.R * c.N)
    assert torch.isnan(behind).all()


# ----------------------------------------------------------------------------
# gradients
# ----------------------------------------------------------------------------

def backward(c, seed, want=("dx", "dw"), stream=None):
    B = B_()
    rng = np.random.default_rng(seed)
    dy = host(gpu(0.2 * rng.standard_normal((c.R, c.N)), c.dtype))
    dyt = gpu(dy, c.dtype)
    dx = blank((c.R, c.K), c.dtype) if "dx" in want else None
    dw = blank(tuple(c.wt.shape), c.dtype) if "dw" in want else None
    torch.cuda.synchronize()

    def call():
        B.moe_grouped_gemm_backward(c.xt, dyt, c.offt, c.R, c.E, c.K, c.N, code(c.dtype), c.buf, c.w_off, dx, dw,
                                    c.status, stream)

    call()
    torch.cuda.synchronize()
    return dy, dx, dw, call


def check_backward(c, dy, dx, dw):
    half, size = HALF[c.dtype], 4 if c.dtype == "f32" else 2
    lead = c.w_off // size
    for e, rows, w in c.live():
        x, d = c.rows[rows], dy[rows]
        if dx is not None:
            ref, f32 = d @ w, c.N * U * (np.abs(d) @ np.abs(w))
            check(f"dx of expert {e} ({x.shape[0]} rows)", dx[rows], ref, half * (np.abs(ref) + f32) + f32)
        if dw is not None:
            block = dw[c.slots[e]]
            ref, f32 = d.T @ x, max(1, x.shape[0]) * U * (np.abs(d).T @ np.abs(x))
            check(f"dw of expert {e}", block[lead:lead + c.N * c.K].view(c.N, c.K), ref, half * (np.abs(ref) + f32) + f32)
            assert torch.isnan(block[:lead]).all() and torch.isnan(block[lead + c.N * c.K:]).all()   # beside it


BACKWARD = [((1,), 8, 8, "bf16"), ((3, 0, 5), 16, 8, "bf16"), ((1, 2, 0, 16, 17), 136, 72, "bf16"),
            ((255, 257, 0, 1), 264, 512, "bf16"), ((300, 512), 512, 136, "bf16"), ((193, 64, 191), 1024, 2056, "bf16"),
            ((2000, 1500), 4104, 520, "bf16"), ((1,), 1, 1, "f32"), ((3, 0, 5), 17, 9, "f32"),
            ((129, 1, 0, 40), 131, 77, "f32"), ((64, 200), 256, 512, "f32"), ((1700, 1, 1899), 1030, 901, "f32"),
            ((3500,), 645, 130, "f32"), ((5, 7, 0, 1, 33, 2, 3, 4, 5, 6, 7, 8), 530, 461, "f32")]


@pytest.mark.parametrize("counts,K,N,dtype", BACKWARD)
def test_backward(counts, K, N, dtype):
    log(f"case backward rows={counts} K={K} N={N} {dtype}")
    c = Case(counts, K, N, dtype, 31 + K + N, lead=32)
    dy, dx, dw, call = backward(c, 1)
    assert int(c.status.item()) == 0
    check_backward(c, dy, dx, dw)
    first = dx.clone(), dw.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(first[0], dx) and torch.equal(first[1].view(torch.uint8), dw.view(torch.uint8))
    _, dx2, none, _ = backward(c, 1, want=("dx",))
    assert none is None and torch.equal(dx, dx2)
    _, none, dw2, _ = backward(c, 1, want=("dw",))
    assert none is None and torch.equal(dw.view(torch.uint8), dw2.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("want", [("dx", "dw"), ("dx",), ("dw",)])
def test_backward_absent_slots(dtype, want):
    B = B_()
    c = Case((20, 7, 0, 5, 140), 64, 40, dtype, 6, slots=[3, -1, -1, 4, 0], n_slots=4, tail=9)
    dy, dx, dw, _ = backward(c, 2, want)
    assert int(c.status.item()) == B.MOE_STATUS_EXPERT_ABSENT
    check_backward(c, dy, dx, dw)
    off = c.offsets
    if dx is not None:
        for lo, hi in ((off[1], off[2]), (off[3], off[4]), (off[5], off[5] + 9)):
            assert torch.isnan(dx[lo:hi]).all()
    if dw is not None:
        assert torch.isnan(dw[1]).all() and torch.isnan(dw[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_without_rows(dtype):
    """No tokens: every gradient of a weight is zero."""
    c = Case((0, 0), 64, 40, dtype, 3)
    _, dx, dw, _ = backward(c, 3)
    assert not host(dw)[:, :64 * 40].any() and dx.shape == (0, 64)


# ----------------------------------------------------------------------------
# as they are used
# ----------------------------------------------------------------------------

def test_graph_replay():
    """Forward of each type and the gradient in one graph, replayed on new rows and offsets with eager
    work in between."""
    cases = [[Case(n, 96, 72, d, 40, out="f32") for d in ("mx", "mx", "bf16", "bf16", "f32")]
             for n in ((20, 7, 3), (300, 77, 100))]
    cases = [c for group in cases for c in group[::2]]
    dys = {id(c): gpu(np.ones((c.R, c.N)), c.dtype) for c in cases if c.dtype != "mx"}
    grads = {id(c): (torch.empty_like(c.xt), blank(tuple(c.wt.shape), c.dtype)) for c in cases if c.dtype != "mx"}
    B = B_()

    def step(stream=None):
        for c in cases:
            c.call(stream)
            if c.dtype != "mx":
                B.moe_grouped_gemm_backward(c.xt, dys[id(c)], c.offt, c.R, c.E, c.K, c.N, code(c.dtype), c.buf, c.w_off,
                                            *grads[id(c)], c.status, stream)

    stream = torch.cuda.Stream()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(stream)
    for turn in range(4):
        for c in cases:
            off = c.offsets.copy()
            off[1] = max(0, off[1] - 3 * turn)              # rows move from expert 0 to expert 1
            c.offt.copy_(i32(off))
            c.xt.copy_(c.xt.roll(1, 0))
            if c.dtype == "mx":
                c.xs.copy_(c.xs.roll(1, 0))
            c.y.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [c.y.clone() for c in cases] + [t.clone() for c in cases if c.dtype != "mx" for t in grads[id(c)]]
        step()
        torch.cuda.synchronize()
        want = [c.y for c in cases] + [t for c in cases if c.dtype != "mx" for t in grads[id(c)]]
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), turn
        assert all(torch.isfinite(c.y).all() for c in cases)
        torch.randn(1 << 20, device="cuda").sum().item()


def test_two_streams_at_once():
    a, b = Case((300, 0, 90, 33), 544, 264, "mx", 51), Case((7, 0, 9, 3), 544, 264, "mx", 52)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip((a, b), streams):
            c.call(s)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("T,top_k", [(1, 2), (64, 2), (700, 3)])
def test_block_in_8_bits(T, top_k):
    """norm (with the residual) -> route -> permute -> gate and up -> swiglu -> down -> combine -> dropout
    with the residual, on one stream, against the same chain in float64 on the values that each 8-bit
    step stored."""
    B = B_()
    H, I, E = 288, 160, 6
    rng = np.random.default_rng(T)
    R = T * top_k
    x, res = (host(gpu(rng.standard_normal((T, H)), "bf16")) for _ in range(2))
    gamma = host(gpu(1 + 0.2 * rng.standard_normal(H)))
    wr = gpu(rng.standard_normal((E, H)) * H ** -0.5)
    up, down = rng.standard_normal((E, 2 * I, H)) * H ** -0.5, rng.standard_normal((E, H, I)) * I ** -0.5
    # an expert's block: both matrices, then their scales, quantised on the GPU as a checkpoint is loaded
    parts = [2 * I * H, H * I, 2 * I * K8.pitch(H), H * K8.pitch(I)]
    at = np.concatenate([[0], np.cumsum(parts)])
    blocks = torch.zeros(E, int(at[-1]), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")
    int_ = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    slot_of = torch.arange(E, dtype=torch.int32, device="cuda")
    total, y, q, qs, rstd = bf(T, H), bf(T, H), u8(T, H), u8(T, K8.pitch(H)), f32(T)
    idx, tw = int_(T * top_k), f32(T, top_k)
    counts, offsets, row_of, src_of = int_(E), int_(E + 1), int_(R), int_(R)
    gu, h, hs, yp, out = bf(R, 2 * I), u8(R, I), u8(R, K8.pitch(I)), f32(R, H), f32(T, H)
    new, keep_state = bf(T, H), torch.tensor([5, 9], dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = B.moe_permute_workspace_size(T, E, top_k)
    ws = u8(max(1, need))
    xt, rt, gt = gpu(x, "bf16"), gpu(res, "bf16"), gpu(gamma)
    weights = [(gpu(up[e], "bf16"), gpu(down[e], "bf16")) for e in range(E)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for e in range(E):
            b = blocks[e].data_ptr()
            B.moe_mx_quantize(weights[e][0], 2 * I, H, B.MOE_BF16, 0, b + int(at[0]), b + int(at[2]), stream)
            B.moe_mx_quantize(weights[e][1], H, I, B.MOE_BF16, 0, b + int(at[1]), b + int(at[3]), stream)
        w = B.wbuf(blocks, int(at[-1]), E, E, slot_of)
        B.moe_rms_norm(xt, rt, gt, T, H, 1e-6, B.MOE_BF16, total, y, q, qs, rstd, stream)
        logits = y.float() @ wr.t()
        B.moe_route(logits, T, E, top_k, idx, tw, status, stream)
        B.moe_permute(idx, T, E, top_k, None, H, B.MOE_BF16, counts, offsets, row_of, src_of, None, ws, need, status,
                      stream)
        B.moe_grouped_gemm_mx(q, qs, src_of, top_k, offsets, R, E, H, 2 * I, w, int(at[0]), int(at[2]), B.MOE_BF16, gu,
                              status, stream)
        B.moe_mx_quantize(gu, R, I, B.MOE_BF16, 1, h, hs, stream)
        B.moe_grouped_gemm_mx(h, hs, None, 0, offsets, R, E, I, H, w, int(at[1]), int(at[3]), B.MOE_F32, yp, status,
                              stream)
        B.moe_combine(yp, row_of, tw, T, top_k, H, out, stream)
        B.moe_dropout_add(out, B.MOE_F32, total, T * H, 0.1, keep_state, B.MOE_BF16, new, stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    n = lambda t: t.cpu().numpy()
    off, src = n(offsets), n(src_of)
    hb = n(blocks)
    mat = lambda e, i, rows, cols: K8.decode(hb[e, at[i]:at[i + 1]].reshape(rows, cols),
                                             hb[e, at[i + 2]:at[i + 3]].reshape(rows, -1))
    wu, wd = np.stack([mat(e, 0, 2 * I, H) for e in range(E)]), np.stack([mat(e, 1, H, I) for e in range(E)])
    xn = K8.decode(n(q), n(qs))[src // top_k]
    ref = K8.grouped_gemm(xn, off, wu)
    tol = H * U * K8.grouped_gemm(np.abs(xn), off, np.abs(wu))
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        tol[rows] += 7 * 2.0 ** -13 * largest_of_eight(xn[rows], wu[e])
    check("gate and up", gu, ref, HALF["bf16"] * (np.abs(ref) + tol) + tol)
    hv = K8.decode(n(h), n(hs))
    ref = K8.grouped_gemm(hv, off, wd)
    tol = I * U * K8.grouped_gemm(np.abs(hv), off, np.abs(wd))
    check("down", yp, ref, tol)
    comb = O.combine(host(yp), n(row_of), host(tw), top_k)
    check("combine", out, comb, 4 * top_k * U * (np.abs(comb) + np.abs(host(yp)).max()))
    kept = np.where(K8.keep(T * H, 0.1, 5, 9).reshape(T, H), host(out) / 0.9, 0)
    want = kept + host(total)
    check("new stream", new, want, HALF["bf16"] * np.abs(want) + 4 * U * (np.abs(kept) + np.abs(want)))
    # end to end against the bf16 weights in float64: 8-bit values are half a step, 2^-4, off at most and
    # about 0.026 of themselves on average; four of them meet (rows and weights of two products), so
    # their errors, which are independent, add to about 0.06 in the 2-norm, and 0.15 has room for none missing
    v = host(total)
    yn, _ = K8.rms_norm(v, gamma, 1e-6)
    g = K8.grouped_gemm(yn[src // top_k], off, np.stack([host(a) for a, _ in weights]))
    full = K8.grouped_gemm(K8.swiglu(g), off, np.stack([host(b) for _, b in weights]))
    full = O.combine(full, n(row_of), host(tw), top_k)
    off_by = np.linalg.norm(host(out) - full) / np.linalg.norm(full)
    log(f"  8 bits against bf16 weights in float64: {off_by:.3f}")
    assert off_by < 0.15


# ----------------------------------------------------------------------------
# many experts, rows of 2 KB, large sizes
# ----------------------------------------------------------------------------

def spread(E, seed, top):
    """Rows of E experts: most a few, some none, some up to `top`."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, 4, E)
    n[rng.integers(0, E, 3)] = rng.integers(1, top, 3)
    return tuple(int(v) for v in n)


@pytest.mark.parametrize("dtype", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("E,K,N,top", [(130, 64, 264, 300), (1000, 32, 72, 600), (1024, 32, 8, 70), (65, 96, 520, 900)])
def test_many_experts(E, K, N, top, dtype):
    """More experts than a wave has lanes: each lane looks after several in the list of tiles."""
    counts = spread(E, E + K, top)
    log(f"case {dtype} E={E} rows={sum(counts)} K={K} N={N}")
    c = Case(counts, K, N, dtype, 71, gather=2)
    c.call()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    c.check()
    if dtype != "mx":
        c = Case(counts, K, N, dtype, 72)
        dy, dx, dw, _ = backward(c, 4)
        check_backward(c, dy, dx, dw)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("E,N", [(70, 264), (20, 1032)])
@pytest.mark.parametrize("K,dtype", [(2048, "mx"), (4096, "mx"), (1024, "bf16"), (2048, "bf16")])
def test_tiles_that_start_at_different_depths(K, dtype, E, N, out):
    """Few rows an expert and rows of a multiple of 2 KB: tiles begin inside the depth and go around it."""
    if K * E > 50000:
        E = E // 2 + 30
    counts = spread(E, K, 80)
    log(f"case {dtype} E={E} rows={sum(counts)} K={K} N={N} {out}")
    c = Case(counts, K, N, dtype, 73, gather=3, out=out)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype,out", [("mx", "bf16"), ("mx", "f32"), ("bf16", "bf16")])
def test_outputs_past_2_31_elements(dtype, out):
    """The last expert's rows lie past 2^31 elements of y."""
    B = B_()
    K, N, R = 32, 4104, 530_000
    last = 40
    log(f"case {dtype} -> {out}: {R * N / 2 ** 31:.2f} * 2^31 outputs")
    c = Case((3, last), K, N, dtype, 74, out=out)          # the values to check against
    offsets = i32([0, 3, R - last, R])
    slots = i32([c.slots[0], c.slots[0], c.slots[1]])
    buf = B.wbuf(c.wt, c.block, 2, 3, slots)
    x = torch.zeros((R, K), dtype=c.xt.dtype, device="cuda")
    x[:3], x[-last:] = c.xt[:3], c.xt[3:]
    y = torch.empty((R, N), dtype=c.y.dtype, device="cuda")
    if dtype == "mx":
        xs = torch.zeros((R, 16), dtype=torch.uint8, device="cuda")
        xs[:3], xs[-last:] = c.xs[:3], c.xs[3:]
        B.moe_grouped_gemm_mx(x, xs, None, 0, offsets, R, 3, K, N, buf, c.w_off, c.s_off, code(out), y)
    else:
        B.moe_grouped_gemm(x, None, 0, offsets, R, 3, K, N, code(dtype), buf, c.w_off, code(out), y)
    torch.cuda.synchronize()
    c.y[:3], c.y[3:] = y[:3], y[-last:]
    c.check()
    assert not y[R // 2].any() and not y[R - last - 1].any()


def test_gradients_past_2_31_elements():
    B = B_()
    K, N, R, last = 7168, 8, 300_100, 33
    c = Case((5, last), K, N, "bf16", 75)
    rng = np.random.default_rng(5)
    dy = host(gpu(0.2 * rng.standard_normal((5 + last, N)), "bf16"))
    x, dyt = (torch.zeros((R, n), dtype=torch.bfloat16, device="cuda") for n in (K, N))
    x[:5], x[-last:] = c.xt[:5], c.xt[5:]
    dyt[:5], dyt[-last:] = gpu(dy[:5], "bf16"), gpu(dy[5:], "bf16")
    dx, dw = torch.empty_like(x), blank(tuple(c.wt.shape), "bf16")
    offsets, slots = i32([0, R - last, R]), i32(c.slots)
    B.moe_grouped_gemm_backward(x, dyt, offsets, R, 2, K, N, B.MOE_BF16, B.wbuf(c.wt, c.block, 2, 2, slots), c.w_off,
                                dx, dw)
    torch.cuda.synchronize()
    check_backward(c, dy, torch.cat([dx[:5], dx[-last:]]), dw)      # rows of zeros add nothing to the first expert's


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("low,high", [(0, 239), (3, 239), (228, 8), (40, 200)])
@pytest.mark.parametrize("counts", [(5, 9), (200, 77), (700, 1300)])
def test_mx_scales_at_the_ends(counts, low, high, out):
    """x's smallest scale byte is ``low`` and the weights' largest ``high``: scales of 2^-127 to 2^117, values in
    bf16's subnormals.  (2^-124 on with f32 outputs: below it not every element is a bf16 number.)"""
    low = max(low, 3) if out == "f32" else low
    c = Case(counts, 544, 2056 if sum(counts) > 1000 else 72, "mx", 76, out=out)
    K, N, n = c.K, c.N, c.K // 32
    xs, ws = host(c.xs), host(c.wt[:, c.s_off:c.s_off + N * 32]).reshape(len(counts), N, 32)
    by_x, by_w = low - int(xs[:, :n].min()), high - int(ws[:, :, :n].max())
    xs[:, :n] += by_x
    ws[:, :, :n] += by_w
    assert xs.min() >= 0 and ws.min() >= 0 and xs.max() < 248 and ws.max() < 248
    c.xs.copy_(torch.from_numpy(xs.astype(np.uint8)))
    c.wt[:, c.s_off:c.s_off + N * 32] = torch.from_numpy(ws.reshape(len(counts), -1).astype(np.uint8)).cuda()
    c.x, c.w = c.x * 2.0 ** by_x, c.w * 2.0 ** by_w
    c.rows = c.x
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("K,dtype,out", [(2048, "mx", "bf16"), (2048, "mx", "f32"), (1024, "bf16", "bf16"),
                                         (2048, "bf16", "f32")])
@pytest.mark.parametrize("counts,N", [((2300, 1, 0, 1500, 700), 2056), ((600, 900, 256), 3336), ((8000,), 520)])
def test_units_of_many_rows_start_at_different_depths(K, dtype, out, counts, N):
    """Rows of a multiple of 2 KB in units of 1, 2 and 4 tiles by several."""
    log(f"case {dtype} rows={counts} K={K} N={N} {out}")
    c = Case(counts, K, N, dtype, 77, out=out)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("counts", [(3, 0, 30), (200, 77)])
@pytest.mark.parametrize("K,N,dtype", [(2 ** 20, 8, "mx"), (2 ** 20, 8, "bf16"), (2 ** 20, 3, "f32"),
                                       (32, 2 ** 20, "mx"), (8, 2 ** 20, "bf16"), (3, 2 ** 20, "f32")])
def test_the_longest_sides(counts, K, N, dtype):
    log(f"case {dtype} rows={counts} K={K} N={N}")
    counts = counts if K > N or counts[1] == 0 else (70, 20)
    c = Case(counts, K, N, dtype, 78, out="f32")
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("want", [("dx", "dw"), ("dw",), ("dx",)])
@pytest.mark.parametrize("counts,K,N", [((33_000,), 264, 256), ((1, 0, 20, 7, 3, 12, 40, 5), 1096, 1032),
                                        ((4000, 0, 5500, 2100), 1544, 520)])
def test_gradients_whose_tiles_differ(counts, K, N, want):
    """dX of large tiles and dW of small ones, the other way round, and one of the two alone."""
    log(f"case rows={counts} K={K} N={N} {want}")
    c = Case(counts, K, N, "bf16", 79)
    dy, dx, dw, _ = backward(c, 4, want)
    check_backward(c, dy, dx, dw)
