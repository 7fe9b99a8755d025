"""What a block is quantized to, bit for bit: scale = max(amax, 2^-100) / 448, and
the nearest e4m3 (ties to even) to the fp32 quotient of each value by it for
weights, to the product with its fp32 reciprocal for activations. The two differ
for the few values whose quotient lies next to the border between two e4m3 values."""
import pytest
import torch

from test_fp8 import BLOCK, FP8, gen, spread

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


def border_values():
    """bf16 blocks of 128 (their largest value first) whose other values have
    quotients that the reciprocal would round to another e4m3 value."""
    top = torch.arange(128, 256, dtype=torch.float32)              # every bf16 significand
    low = (top[:, None] * 2.0 ** -torch.arange(1, 16)).flatten()
    scale = top / torch.full_like(top, 448.0)
    quotient = low[None, :] / scale[:, None]
    product = low[None, :] * (1.0 / scale)[:, None]
    differ = quotient.to(FP8).float() != product.to(FP8).float()
    blocks = []
    for a, row in zip(top, differ):
        v = low[row][: BLOCK - 1]
        if len(v):
            blocks.append(torch.cat([a[None], v, torch.zeros(BLOCK - 1 - len(v))]))
    return torch.stack(blocks)


def test_border_values_exist():
    b = border_values()
    assert b.shape[0] >= 8 and bool((b.bfloat16().float() == b).all()) and bool((b[:, 1:].amax(1) < b[:, 0]).all())


def same(q, want):
    return torch.equal(q.float(), want.float())   # (a zero's sign is not kept)


@gpu
def test_weight_quantization_is_the_quotient(lib):
    b = border_values().cuda()
    G = b.shape[0]
    w = torch.zeros(G, 256, 48, device="cuda")
    w[:, :BLOCK, 3] = b
    w[:, 130:, 7] = -b[:, : 256 - 130]
    w = w.bfloat16()
    q, scale = lib.fp8_quantize_weight(w)
    t = w.float().transpose(1, 2).contiguous()
    assert torch.equal(scale[:, 0, 0], (b[:, 0] / torch.full_like(b[:, 0], 448.0)))
    assert same(q, (t / spread(scale, 256).float().repeat_interleave(BLOCK, 1)[:, :48]).to(FP8))
    w = (torch.randn(2, 4096, 4096, generator=gen(1), device="cuda") * 0.02).bfloat16()
    q, scale = lib.fp8_quantize_weight(w)
    t = w.float().transpose(1, 2).contiguous()
    assert same(q, (t / spread(spread(scale, 4096), 4096, 1).float()).to(FP8))


@gpu
@pytest.mark.parametrize("T,H", [(8192, 4096), (3, 144), (2048, 16400)])
def test_norm_quantization_is_the_product_with_the_reciprocal(lib, T, H):
    """y in fp32 is what is quantized."""
    x = torch.randn(T, H, generator=gen(T), device="cuda") * torch.exp(torch.randn(T, 1, generator=gen(H), device="cuda"))
    _, y, q, scale = lib.add_rmsnorm_fp8(x)
    amax = torch.nn.functional.pad(y, (0, -H % BLOCK)).unflatten(1, (-1, BLOCK)).abs().amax(2)
    assert torch.equal(scale, amax / torch.full_like(amax, 448.0))
    assert same(q, (y * spread(torch.ones_like(scale) / scale, H).float()).to(FP8))


@gpu
def test_norm_of_a_row_whose_squares_overflow(lib):
    """As include/moe.h says: y = 0 for it, and nothing for its neighbours."""
    x = torch.ones(3, 256, device="cuda")
    x[1] = 2.0 ** 70
    _, y, q, scale = lib.add_rmsnorm_fp8(x, eps=0.0)
    assert bool((y[1] == 0).all()) and bool((q[1].float() == 0).all()) and bool((scale[1] == 2.0 ** -100 / 448).all())
    assert bool((y[0] == 1).all()) and bool((y[2] == 1).all()) and bool((q[0].float() == 448).all())


@gpu
def test_norm_quantization_at_the_borders(lib):
    """Rows that the norm leaves as they are: mean square 1, two values of 8192 carry it.
    Either neighbour of a value at a border is as near to it."""
    b = border_values().cuda()
    n, H = b.shape[0], 8192
    x = torch.zeros(n, H, device="cuda")
    x[:, : BLOCK] = b * 2.0 ** -40
    x[:, 4096] = x[:, 4097] = 64.0
    _, y, q, scale = lib.add_rmsnorm_fp8(x, eps=0.0)
    v, s = x[:, :BLOCK], scale[:, :1]
    assert torch.equal(y[:, :BLOCK], v)
    assert torch.equal(s[:, 0], v[:, 0] / torch.full_like(v[:, 0], 448.0))
    assert same(q[:, :BLOCK], (v * (torch.ones_like(s) / s)).to(FP8))
    quotient = (v / s).to(FP8)
    assert not same(q[:, :BLOCK], quotient)
    off = [(t.double() * s.double() - v.double()).abs() for t in (q[:, :BLOCK].double(), quotient.double())]
    assert bool(((off[0] - off[1]).abs() <= v.double().abs() * 2.0 ** -21).all())
