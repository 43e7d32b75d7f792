"""Rows to 8 bits on both sides of each limit of the launch: up to 16 blocks a CU a wave takes one unit of
512 columns, up to 64 blocks a CU that many waves take units in turn, and above one each again.
"""
import numpy as np
import pytest

from moe_cases import log
from oracle import block as K
from test_gpu_backward import U, code, gpu, host
from test_gpu_block import bytes8, check8, unpack8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def in_turns(rows, cols):
    """The rule of csrc/mx.hip."""
    return 256 * 16 < -(-rows * -(-cols // 512) // 4) <= 256 * 64


SIZES = [(16384, 32, False), (16385, 32, True), (65536, 32, True), (65537, 32, False), (9001, 544, True),
         (32771, 512, True), (4099, 7168, True), (1171, 7168, True), (1170, 7168, False)]


@pytest.mark.parametrize("rows,cols,turns", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize(rows, cols, turns, dtype):
    """Every byte."""
    from grouped_gemm_weights_amd import binding as B
    assert in_turns(rows, cols) == turns
    log(f"case quantize rows={rows} cols={cols} {dtype} turns={turns}")
    rng = np.random.default_rng(rows + cols)
    x = host(gpu(rng.standard_normal((rows, cols), np.float32) * 2.0 ** rng.integers(-12, 12, (rows, 1)), dtype))
    q, s = bytes8(rows, cols)
    B.moe_mx_quantize(gpu(x, dtype, 1), rows, cols, code(dtype), 0, q, s)
    torch.cuda.synchronize()
    q, s = unpack8(q, s, rows, cols)
    rq, rs = K.quantize(x)
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(K.e4m3_values()[q], rq)


@pytest.mark.parametrize("rows,cols,turns", [(16384, 32, False), (16385, 32, True), (65536, 32, True), (65537, 32, False),
                                             (5501, 1408, True), (1171, 7168, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_swiglu(rows, cols, turns, dtype):
    from grouped_gemm_weights_amd import binding as B
    assert in_turns(rows, cols) == turns
    log(f"case quantize swiglu rows={rows} cols={cols} {dtype} turns={turns}")
    rng = np.random.default_rng(rows * 3 + cols)
    x = host(gpu(3 * rng.standard_normal((rows, 2 * cols), np.float32), dtype))
    q, s = bytes8(rows, cols)
    B.moe_mx_quantize(gpu(x, dtype, 3), rows, cols, code(dtype), 1, q, s)
    torch.cuda.synchronize()
    v = K.swiglu(x)
    # the exponent's rounding moves e^-g by |g| log2(e) u; 16 u for exp2, reciprocal and products
    check8("h", *unpack8(q, s, rows, cols), v, (16 + 1.5 * np.abs(x[:, :cols])) * U * np.abs(v) + 2.0 ** -149)
