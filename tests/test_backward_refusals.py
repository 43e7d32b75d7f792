"""Argument checks of the training pass's entry points: each refusal comes back as its code before
anything is enqueued (no GPU needed; the pointers are never read)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

P = 1 << 20  # a pointer-like number, 16-byte aligned


@pytest.fixture(scope="module")
def B():
    from grouped_gemm_weights_amd import binding
    return binding


def refused(B, code, call, *args):
    with pytest.raises(B.MoEError) as e:
        call(*args)
    assert e.value.code == code
    assert call.__name__.replace("_workspace_size", "") in B.moe_last_error()


def test_layer_norm(B):
    A, U = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED
    f = B.moe_layer_norm
    for code, args in [
            (A, (P, P, P, -1, 8, 1e-5, B.MOE_F32, P)), (A, (P, P, P, 2, 0, 1e-5, B.MOE_F32, P)),
            (A, (P, P, P, 2, 8, -1e-5, B.MOE_F32, P)), (A, (P, P, P, 2, 8, float("nan"), B.MOE_F32, P)),
            (A, (P, P, P, 2, 8, 1e-5, 7, P)), (A, (None, P, P, 2, 8, 1e-5, B.MOE_F32, P)),
            (A, (P, None, P, 2, 8, 1e-5, B.MOE_F32, P)), (A, (P, P, P, 2, 8, 1e-5, B.MOE_F32, None)),
            (U, (P, P, P, 2, (1 << 28) + 1, 1e-5, B.MOE_F32, P)),
            (U, (P, P, P, 1 << 23, 1 << 16, 1e-5, B.MOE_F32, P))]:      # 2^33 threads
        refused(B, code, f, *args)
    f(None, None, None, 0, 8, 1e-5, B.MOE_BF16, None)      # no rows: nothing to do


def test_layer_norm_backward(B):
    A, U, W = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
    f = B.moe_layer_norm_backward
    need = B.moe_layer_norm_backward_workspace_size(4, 100)
    # one partial row of dgamma and dbeta per workgroup, and at least one workgroup
    assert need >= 2 * 100 * 4 and B.moe_layer_norm_backward_workspace_size(0, 100) == 0
    # T and H far past any partial count: the workspace stays bounded
    assert B.moe_layer_norm_backward_workspace_size(1 << 30, 64) <= 4096 * 2 * 64 * 4
    ok = (P, P, P, P, P, 4, 100, B.MOE_F32, P, P, P, P, need)

    def but(at, value):
        return ok[:at] + (value,) + ok[at + 1:]

    for at in (0, 1, 2, 3, 4, 8):
        refused(B, A, f, *but(at, None))
    refused(B, A, f, *but(5, -1))
    refused(B, A, f, *but(6, 0))
    refused(B, A, f, *but(7, 5))
    refused(B, U, f, *but(6, (1 << 28) + 1))
    refused(B, W, f, *but(12, need - 1))
    refused(B, W, f, *but(11, None))
    refused(B, A, B.moe_layer_norm_backward_workspace_size, -1, 4)
    f(None, None, None, None, None, 0, 100, B.MOE_F32, None, None, None, None, 0)


def test_combine_and_permute_backward(B):
    A, U = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED
    f = B.moe_combine_backward
    ok = (P, B.MOE_BF16, P, P, P, 4, 2, 8, B.MOE_F32, P, P)

    def but(at, value):
        return ok[:at] + (value,) + ok[at + 1:]

    for at in (0, 2, 3, 4, 9):
        refused(B, A, f, *but(at, None))
    for at, value in ((1, 3), (5, -1), (6, 0), (7, 0), (8, -1)):
        refused(B, A, f, *but(at, value))
    refused(B, U, f, *but(6, 65))
    refused(B, U, f, *but(5, 1 << 30))
    refused(B, U, f, *but(7, (1 << 28) + 1))
    refused(B, U, f, *but(5, 1 << 25))                                  # 2^33 threads
    f(*but(5, 0))
    g = B.moe_permute_backward
    ok = (P, P, 4, 2, 8, B.MOE_BF16, P)
    for at in (0, 1, 6):
        refused(B, A, g, *but(at, None))
    for at, value in ((2, -1), (3, 0), (4, 0), (5, 9)):
        refused(B, A, g, *but(at, value))
    refused(B, U, g, *but(2, 1 << 30))
    refused(B, U, g, *but(4, (1 << 28) + 1))
    refused(B, U, g, P, P, 1 << 25, 2, 4096, B.MOE_BF16, P)             # 2^34 threads
    g(*but(2, 0))


def test_route_backward(B):
    A, U = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED
    f = B.moe_route_backward
    ok = (P, P, P, 4, 16, 2, P)

    def but(at, value):
        return ok[:at] + (value,) + ok[at + 1:]

    for at in (0, 1, 2, 6):
        refused(B, A, f, *but(at, None))
    for at, value in ((3, -1), (4, 0), (5, 0), (5, 17)):
        refused(B, A, f, *but(at, value))
    refused(B, U, f, *but(4, 1025))
    refused(B, U, f, P, P, P, 4, 128, 65, P)
    refused(B, U, f, *but(3, 1 << 27))                                  # 2^33 threads
    f(*but(3, 0))


def test_grouped_swiglu_backward(B):
    A, U, W = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
    f = B.moe_grouped_swiglu_backward
    R, E, H, I = 8, 4, 16, 8
    buf = B.wbuf(P, 3 * H * I * 2, 4, E, P)
    need = B.moe_grouped_swiglu_backward_workspace_size(R, E, H, I, B.MOE_BF16)
    ok = (P, P, P, R, E, H, I, B.MOE_BF16, buf, P, need, P, P)

    def but(*pairs):
        a = list(ok)
        for at, value in pairs:
            a[at] = value
        return a

    for at in (0, 1, 2):
        refused(B, A, f, *but((at, None)))
    refused(B, A, f, *but((11, None), (12, None)))                      # nothing to compute
    for at in (3, 5, 6):
        refused(B, A, f, *but((at, -1)))
    refused(B, A, f, *but((4, 0)))
    refused(B, A, f, *but((7, 2)))
    refused(B, A, f, *but((4, 5)))                                      # E disagrees with the buffer
    refused(B, A, f, *but((8, B.wbuf(P, 96, 4, E, P))))                 # block size disagrees
    refused(B, A, f, *but((8, B.wbuf(None, 3 * H * I * 2, 4, E, P))))
    refused(B, A, f, *but((8, B.wbuf(P, 3 * H * I * 2, 4, E, None))))
    refused(B, U, f, *but((4, 1025)))
    refused(B, U, f, *but((5, 12), (8, B.wbuf(P, 3 * 12 * I * 2, 4, E, P))))
    refused(B, U, f, *but((6, 12), (8, B.wbuf(P, 3 * 12 * H * 2, 4, E, P))))
    side = 1 << 15
    refused(B, U, f, *but((5, side), (6, side), (8, B.wbuf(P, 6 * side * side, 4, E, P))))
    side = (1 << 20) + 8
    refused(B, U, f, *but((5, side), (8, B.wbuf(P, 6 * side * I, 4, E, P))))
    refused(B, U, f, *but((3, 1 << 30), (10, 1 << 62)))                 # more than 2^32 threads
    for at in (0, 1, 9, 11, 12):
        refused(B, U, f, *but((at, P + 8)))                             # alignment
    refused(B, W, f, *but((10, need - 1)))
    refused(B, W, f, *but((9, None)))
    refused(B, A, B.moe_grouped_swiglu_backward_workspace_size, 8, 0, 16, 8, B.MOE_BF16)


def test_sizes_up_to_the_largest_int(B):
    """Counts of workgroups stay exact up to T = 2^31 - 1."""
    U, last = B.MOE_ERR_UNSUPPORTED, (1 << 31) - 1
    for T in (last, last - 14):
        # the partial rows of as many workgroups as smaller sizes have
        for H in (1, 64, 8192, 16385):
            assert B.moe_layer_norm_backward_workspace_size(T, H) == \
                B.moe_layer_norm_backward_workspace_size(1 << 30, H)
        for H in (9, 72, 4096):                                         # 2^32 threads and more
            refused(B, U, B.moe_permute_backward, P, P, T, 1, H, B.MOE_BF16, P)
        refused(B, U, B.moe_route_backward, P, P, P, T, 16, 1, P)
        refused(B, U, B.moe_combine_backward, P, B.MOE_F32, P, P, P, T, 1, 8, B.MOE_F32, P, P)


def test_layer_norm_launches_of_long_rows(B):
    """Rows of 16385 to 32768 elements have a workgroup of 9 to 16 waves each: 2^32 threads are
    passed at T = 2^32 / 1024 and more."""
    for T, H in ((1 << 22, 32768), ((1 << 32) // 576 + 1, 16385), ((1 << 31) - 1, 20000)):
        for dtype in (B.MOE_F32, B.MOE_BF16):
            refused(B, B.MOE_ERR_UNSUPPORTED, B.moe_layer_norm, P, P, P, T, H, 1e-5, dtype, P)


def test_clear_unmapped(B):
    A, U = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED
    f = B.moe_clear_unmapped
    for code, buf, dw in [
            (A, (P, 96, 4, 4, None), P), (A, (P, 96, 4, 4, P), None), (A, (P, 0, 4, 4, P), P),
            (A, (P, 98, 4, 4, P), P), (A, (P, 96, -1, 4, P), P), (A, (P, 96, 4, 0, P), P),
            (U, (P, 96, 4, 1025, P), P), (U, (P, 96, 4, 4, P), P + 2),
            (U, (P, 96, 1 << 25, 4, P), P), (U, (P, 1 << 45, 4, 4, P), P),       # over 2^32 threads
            (U, (P, (1 << 63) - 4, (1 << 31) - 1, 4, P), P)]:
        refused(B, code, f, B.wbuf(*buf), dw)
    f(B.wbuf(None, 96, 0, 4, P), None)                                           # no slots
