"""What route_logits, linear and combine_rows promise beyond the definitions that
test_ops.py holds them to. Tolerances are derived where they stand, in steps of fp32
(2^-23 of a value; half of one for a rounding).
"""
import io
import math

import pytest
import torch

from test_ops import DTYPES, act64, check_linear, check_route, gen, lib, linear64, offsets_of, randn, route64, weight, ws  # noqa: F401

gpu = pytest.mark.gpu


# ------------------------------------------------------------ linear: sums --

@gpu
@pytest.mark.parametrize("R,K,N,G", [(16, 4096, 28672, 1), (768, 2048, 1408, 64), (20000, 4096, 128, 1), (400, 4096, 8192, 1),
                                     (8192, 2048, 1024, 1), (4096, 14336, 512, 2), (300, 1032, 264, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("one_sign", [False, True])
def test_linear_rounds_the_fp32_output_once(lib, ws, R, K, N, G, dtype, one_sign):
    """An output of 16 bits is that of 32 bits, rounded: sums, bias, activation and residual are
    the same whatever the output's type. Bit for bit, on sums that cancel and on sums that
    only grow (where a longer run of the tensor cores, which round towards zero, drifts)."""
    g = gen(R + K)
    dt = DTYPES[dtype]
    off, _ = offsets_of([R // G] * G)
    a, w = randn(g, R, K), randn(g, G, N, K) * K ** -0.5
    if one_sign:
        a, w = a.abs(), w.abs()
    a, w = a.to(dt), w.to(dt).transpose(1, 2)
    bias, res = randn(g, G, N), randn(g, R, N).to(dt)
    for act, b, r in ((None, None, None), (None, bias, res), ("silu", bias, None), ("relu", None, res)):
        out = lib.linear(a, w, ws, bias=b, activation=act, residual=r, offsets=off)
        wide = lib.linear(a, w, ws, bias=b, activation=act, residual=None if r is None else r.float(), offsets=off,
                          out_dtype=torch.float32)
        assert lib.check(ws) == lib.MOE_OK
        assert torch.equal(out, wide.to(dt)), (act, int((out != wide.to(dt)).sum()), out.numel())
