"""Argument checks of the 8-bit block's entry points and their neighbours: each refusal comes back as its
code before anything is enqueued (no GPU needed; the pointers are never read)."""
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
    assert e.value.code == code, args
    assert call.__name__ in B.moe_last_error()


def variants(ok):
    return lambda at, value: ok[:at] + (value,) + ok[at + 1:]


def test_scale_pitch(B):
    assert [B.moe_mx_scale_pitch(c) for c in (32, 512, 544, 7168)] == [16, 16, 32, 224]
    refused(B, B.MOE_ERR_ARG, B.moe_mx_scale_pitch, 0)


def test_quantize(B):
    A, U, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.moe_mx_quantize
    but = variants((P, 4, 64, B.MOE_BF16, 0, P, P))
    for at, value in ((0, None), (1, -1), (2, 0), (3, 2), (4, 2), (4, -1), (5, None), (6, None)):
        refused(B, A, f, *but(at, value))
    for at, value in ((2, 48), (2, (1 << 26) + 32), (5, P + 8), (6, P + 4)):
        refused(B, U, f, *but(at, value))
    refused(B, U, f, P, (1 << 31) - 1, 2048, B.MOE_F32, 0, P, P)       # 2^33 units
    f(None, 0, 64, B.MOE_F32, 1, None, None)                           # no rows: nothing to do


def test_rms_norm(B):
    A, U, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.moe_rms_norm
    but = variants((P, P, P, 4, 64, 1e-5, B.MOE_BF16, P, P, P, P, P))
    for at, value in ((0, None), (2, None), (3, -1), (4, 0), (5, -1e-5), (5, float("nan")), (6, 7), (9, None),
                      (10, None), (1, None)):                          # the last: a sum without a residual
        refused(B, A, f, *but(at, value))
    for at, value in ((4, 40), (9, P + 8), (10, P + 8)):
        refused(B, U, f, *but(at, value))
    refused(B, A, f, P, None, P, 4, 64, 1e-5, B.MOE_BF16)              # no output
    refused(B, U, f, P, None, P, 4, (1 << 26) + 32, 1e-5, B.MOE_BF16, None, P)
    refused(B, U, f, P, None, P, 1 << 23, 1 << 16, 1e-5, B.MOE_F32, None, P)      # 2^33 threads
    f(None, None, None, 0, 8, 1e-5, B.MOE_BF16)


def test_rms_norm_backward(B):
    A, U, W, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.moe_rms_norm_backward
    need = B.moe_rms_norm_backward_workspace_size(4, 100)
    assert need >= 100 * 4 and B.moe_rms_norm_backward_workspace_size(0, 100) == 0
    assert B.moe_rms_norm_backward_workspace_size(1 << 30, 64) <= 4096 * 64 * 4
    but = variants((P, P, P, P, P, 4, 100, B.MOE_F32, P, P, P, need))
    for at, value in ((0, None), (2, None), (3, None), (4, None), (5, -1), (6, 0), (7, 5), (8, None)):
        refused(B, A, f, *but(at, value))
    refused(B, U, f, *but(6, (1 << 26) + 1))
    refused(B, W, f, *but(11, need - 1))
    refused(B, W, f, *but(10, None))
    refused(B, A, B.moe_rms_norm_backward_workspace_size, -1, 4)
    f(None, None, None, None, None, 0, 100, B.MOE_F32, None, None, None, 0)


def test_grouped_gemm(B):
    A, U, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.moe_grouped_gemm
    w = B.wbuf(P, 64 * 32 * 2 + 64, 4, 4, P)
    ok = (P, P, 2, P, 10, 4, 64, 32, B.MOE_BF16, w, 64, B.MOE_F32, P, P)
    but = variants(ok)
    for at, value in ((0, None), (2, 0), (3, None), (4, -1), (5, 0), (5, 5), (6, 0), (7, 0), (8, 3), (10, -16),
                      (10, 80), (11, 2), (12, None), (9, B.wbuf(None, 64 * 32 * 2 + 64, 4, 4, P)),
                      (9, B.wbuf(P, 64 * 32 * 2 + 64, 4, 4, None)), (9, B.wbuf(P, 64 * 32 * 2 - 16, 4, 4, P))):
        refused(B, A, f, *but(at, value))
    for at, value in ((5, 1025), (6, 60), (7, 36), (6, (1 << 20) + 8), (10, 8), (0, P + 8), (12, P + 4),
                      (9, B.wbuf(P + 8, 64 * 32 * 2 + 64, 4, 4, P)), (9, B.wbuf(P, 64 * 32 * 2 + 72, 4, 4, P))):
        refused(B, U, f, *but(at, value))
    big = B.wbuf(P, 1 << 31, 4, 4, P)
    refused(B, U, f, P, None, 0, P, 10, 4, 1 << 15, 1 << 14, B.MOE_BF16, big, 0, B.MOE_F32, P)     # 2^30 bytes
    refused(B, U, f, P, P, 1, P, 1 << 24, 4, 64, 32, B.MOE_BF16, w, 0, B.MOE_F32, P)               # x of 2^31 bytes
    refused(B, U, f, P, P, 2, P, 10, 4, 64, 16, B.MOE_F32, w, 0, B.MOE_BF16, P)                    # f32 in, bf16 out
    f(None, None, 0, P, 0, 4, 64, 32, B.MOE_BF16, w, 0, B.MOE_F32, None)                           # no rows


def test_grouped_gemm_mx(B):
    A, U, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.moe_grouped_gemm_mx
    eb = 64 * 32 + 32 * 16
    w = B.wbuf(P, eb, 4, 4, P)
    but = variants((P, P, P, 2, P, 10, 4, 64, 32, w, 0, 64 * 32, B.MOE_F32, P, P))
    for at, value in ((0, None), (1, None), (3, 0), (4, None), (5, -1), (6, 0), (7, 0), (8, 0), (10, -16),
                      (10, 32 * 16 + 16), (11, -16), (11, 64 * 32 + 16), (12, 2), (13, None)):
        refused(B, A, f, *but(at, value))
    for at, value in ((6, 1025), (7, 48), (8, 36), (0, P + 8), (1, P + 8), (13, P + 8), (11, 64 * 32 - 8)):
        refused(B, U, f, *but(at, value))
    refused(B, U, f, P, P, P, 1, P, 1 << 25, 4, 64, 32, w, 0, 64 * 32, B.MOE_F32, P)               # x of 2^31 bytes
    f(None, None, None, 0, P, 0, 4, 64, 32, w, 0, 64 * 32, B.MOE_F32, None)


def test_grouped_gemm_backward(B):
    A, U, f = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.moe_grouped_gemm_backward
    w = B.wbuf(P, 64 * 32 * 2, 4, 4, P)
    but = variants((P, P, P, 10, 4, 64, 32, B.MOE_BF16, w, 0, P, P, P))
    for at, value in ((0, None), (1, None), (2, None), (3, -1), (4, 0), (4, 3), (5, 0), (6, 0), (7, 3), (9, 16)):
        refused(B, A, f, *but(at, value))
    for at, value in ((4, 1025), (5, 60), (6, 36), (0, P + 8), (10, P + 8), (11, P + 8)):
        refused(B, U, f, *but(at, value))
    refused(B, A, f, P, P, P, 10, 4, 64, 32, B.MOE_BF16, w, 0, None, None)


def test_dropout(B):
    A, f = B.MOE_ERR_ARG, B.moe_dropout_add
    but = variants((P, B.MOE_F32, P, 10, 0.5, P, B.MOE_BF16, P))
    for at, value in ((0, None), (1, 2), (3, -1), (4, 1.0), (4, -0.1), (4, float("nan")), (5, None), (6, 5), (7, None)):
        refused(B, A, f, *but(at, value))
    f(None, B.MOE_F32, None, 0, 0.5, None, B.MOE_BF16, None)
    g = B.moe_dropout_add_backward
    but = variants((P, B.MOE_BF16, 10, 0.5, P, B.MOE_F32, P))
    for at, value in ((0, None), (1, 2), (2, -1), (3, 1.0), (4, None), (5, 5), (6, None)):
        refused(B, A, g, *but(at, value))
