"""Which sizes the products by expert take: a call is refused where one of its launches would pass 2^32
threads, and nowhere before (no GPU needed; the pointers are never read).

Every call here has a null x, which is looked at after the sizes: a size that is taken comes back as
MOE_ERR_ARG for it, one that is not as MOE_ERR_UNSUPPORTED.  A launch of 2^24 workgroups of 256 is too much.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

P = 1 << 20  # a pointer-like number, 16-byte aligned
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def B():
    from grouped_gemm_weights_amd import binding
    return binding


def forward(B, kind, R, E, K, N, src=None, top_k=0):
    if kind == "mx":
        pitch = B.moe_mx_scale_pitch(K)
        w = B.wbuf(P, N * (K + pitch), E, E, P)
        B.moe_grouped_gemm_mx(None, P, src, top_k, P, R, E, K, N, w, 0, N * K, B.MOE_BF16, P)
    else:
        dt = B.MOE_F32 if kind == "f32" else B.MOE_BF16
        w = B.wbuf(P, -(-N * K * (4 if kind == "f32" else 2) // 16) * 16, E, E, P)
        B.moe_grouped_gemm(None, src, top_k, P, R, E, K, N, dt, w, 0, dt, P)


def backward(B, kind, R, E, K, N, want):
    dt = B.MOE_F32 if kind == "f32" else B.MOE_BF16
    w = B.wbuf(P, -(-N * K * (4 if kind == "f32" else 2) // 16) * 16, E, E, P)
    B.moe_grouped_gemm_backward(None, P, P, R, E, K, N, dt, w, 0, P if "x" in want else None, P if "w" in want else None)


def taken(B, call, *args):
    with pytest.raises(B.MoEError) as e:
        call(B, *args)
    text = B.moe_last_error()
    assert e.value.code in (B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED), args
    assert ("null pointer" if e.value.code == B.MOE_ERR_ARG else "workgroups") in text, (args, text)
    return e.value.code == B.MOE_ERR_ARG


@pytest.mark.parametrize("kind", ["mx", "bf16", "f32"])
@pytest.mark.parametrize("R,E,K,N", [(1, 1024, 4096, 4096), (1, 1024, 1024, 4096), (1 << 21, 8, 4096, 4096),
                                     (8000, 16, 32, 1 << 20), (8000, 16, 1 << 20, 8), (1 << 24, 256, 64, 128),
                                     (64, 1024, 7168, 4096)])
def test_forward_takes(B, kind, R, E, K, N):
    """One expert's rows among many experts, millions of rows, the longest sides: no launch is near the limit."""
    assert taken(B, forward, kind, R, E, K, N)


@pytest.mark.parametrize("kind,K", [("mx", 32), ("bf16", 8), ("bf16", 256)])
def test_forward_limit(B, kind, K):
    """4096 column tiles in units of 4 x 8 tiles: 4092 row tiles are the most, one of them for the expert."""
    assert taken(B, forward, kind, 4091 * 256, 1, K, 1 << 20)
    assert not taken(B, forward, kind, 4091 * 256 + 1, 1, K, 1 << 20)
    assert taken(B, forward, kind, 4086 * 256, 6, K, 1 << 20)
    assert not taken(B, forward, kind, 4087 * 256, 6, K, 1 << 20)
    assert taken(B, forward, kind, TOP, 1, K, 256)                       # every row that an int counts
    assert not taken(B, forward, kind, TOP, 1, K, 512)


def test_forward_limit_f32(B):
    """16384 column tiles of 64: 1023 row tiles are the most, one of them for the expert."""
    assert taken(B, forward, "f32", 1022 * 64, 1, 5, 1 << 20)
    assert not taken(B, forward, "f32", 1022 * 64 + 1, 1, 5, 1 << 20)
    assert taken(B, forward, "f32", ((1 << 24) - 2) * 64, 1, 5, 64)
    assert not taken(B, forward, "f32", TOP, 1, 5, 64)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("want", ["x", "w", "xw"])
@pytest.mark.parametrize("R,E,K,N", [(1, 64, 4096, 4096), (1 << 21, 8, 4096, 4096), (8000, 16, 32, 1 << 20),
                                     (8000, 16, 1 << 20, 8), (1 << 24, 256, 64, 128), (64, 512, 4096, 7168)])
def test_backward_takes(B, kind, want, R, E, K, N):
    assert taken(B, backward, kind, R, E, K, N, want)


def test_backward_limit(B):
    """The rows' gradient is bound as a forward product of K columns, the weights' by its experts' tiles; with
    both in one launch their workgroups add up."""
    f = backward
    assert taken(B, f, "bf16", 4091 * 256, 1, 1 << 20, 8, "x")
    assert not taken(B, f, "bf16", 4091 * 256 + 1, 1, 1 << 20, 8, "x")
    assert taken(B, f, "bf16", TOP, 1023, 8, 8, "w") and taken(B, f, "bf16", 1, 1024, 4096, 4096, "w")
    assert not taken(B, f, "bf16", 4091 * 256, 1, 1 << 20, 8, "xw")      # 4 x 4096 tiles more
    assert taken(B, f, "bf16", 4087 * 256, 1, 1 << 20, 8, "xw")
    assert taken(B, f, "bf16", 1, 511, 1 << 20, 8, "w")                  # units of 4 tiles, three of them empty
    assert not taken(B, f, "bf16", 1, 1024, 1 << 20, 8, "w")
    assert taken(B, f, "f32", 1, 1023, 1 << 20, 1, "w")
    assert not taken(B, f, "f32", 1, 1024, 1 << 20, 1, "w")
    assert taken(B, f, "f32", 1022 * 64, 1, 1 << 20, 5, "x")
    assert not taken(B, f, "f32", 1022 * 64 + 1, 1, 1 << 20, 5, "x")
    assert not taken(B, f, "f32", 1022 * 64, 1, 1 << 20, 5, "xw")
