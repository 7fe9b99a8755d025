"""The layer on 8-bit experts where its second product, weighted and scattered to
slots, runs as CTA pairs, in tiles of 128 columns, or cut along K; with the
tensor-core router in front; and its workspace.

The layer is held to its parts bit for bit: the parts take the same kernels on
the same rows (tests of each against 64 bits: test_fp8.py, test_fp8_forms.py), and
weighting, scattering and the sum in rank order are fp32 operations with one
result.
"""
import pytest
import torch

from test_fp8 import gen

gpu = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
WIDE, NARROW, PAIR = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


@pytest.mark.parametrize("T,H,F,E,k,Fs", [(1, 64, 64, 8, 2, 0), (8, 64, 64, 8, 2, 64), (129, 512, 192, 8, 2, 128),
                                          (32768, 2048, 1408, 64, 6, 2816), (8192, 4096, 14336, 8, 2, 0)])
def test_workspace_is_the_products_and_the_bf16_layers(lib, T, H, F, E, k, Fs):
    """The quantized rows and h take the memory that the bf16 layer has for its
    own: nothing beside the two workspaces."""
    dims = lib.make_dims(T, H, F, E, k, Fs)
    assert lib.fp8_workspace_size(dims) <= lib.fp8_workspace_size() + lib.workspace_size(dims) + 255
    # where the rows' scales lie, behind the rows: in the other half of their buffer
    for rows, n in (T * k, H), (T * k, F), (T, Fs):
        assert rows * n + rows * -(-n // 128) * 4 <= rows * n * 2
