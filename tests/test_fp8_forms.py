"""Which kernel an 8-bit product runs (one CTA per MMA with tiles of 256 or 128
columns, or a CTA pair), and each of them where rows are few, missing, ragged,
cut along K, weighted and scattered, against the definition in 64 bits.

Tolerances are those of test_fp8.py: half a rounding step of the output, and
(K + 64) 2^-23 of the sum of the terms' magnitudes for the fp32 sum.
"""
import pytest
import torch

from test_fp8 import check_product, check_quantized, gen, offsets_of, product64, quantized, weight

gpu = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
WIDE, NARROW, PAIR = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


# R, K, N, groups, gated -> form (on 152 SMs)
FORMS = [
    # pairs where their tiles fill the SMs, or K is short
    (196608, 2048, 1408, 64, True, PAIR), (16384, 4096, 14336, 8, True, PAIR), (512, 4096, 256, 1, True, PAIR),
    (16384, 14336, 4096, 8, False, PAIR), (196608, 1408, 2048, 64, False, PAIR), (2048, 14336, 640, 1, True, PAIR),
    (8192, 8192, 8192, 1, False, PAIR), (8192, 14336, 1408, 1, True, PAIR), (4096, 14336, 640, 1, False, PAIR),
    # fewer rows: 256-row tiles would be padding
    (6144, 2048, 1408, 64, True, WIDE), (511, 14336, 1408, 1, True, WIDE), (1024, 14336, 5632, 1, False, WIDE),
    # few tiles and a long K: only one CTA per MMA can cut it
    (512, 14336, 1408, 1, True, WIDE), (2048, 14336, 256, 1, False, WIDE), (8192, 14336, 256, 1, False, WIDE),
    (4096, 14336, 256, 1, True, WIDE), (2048, 20480, 640, 1, False, WIDE), (4096, 14336, 640, 1, True, WIDE),
    (8192, 14336, 256, 4, False, WIDE), (2048, 14336, 256, 4, True, WIDE), (8192, 14336, 640, 1, True, WIDE),
    # a product whose 128-column tiles all find an SM
    (2048, 1024, 256, 1, False, NARROW), (4096, 4096, 256, 1, False, NARROW), (8192, 8192, 256, 1, False, NARROW),
    (16384, 2048, 128, 8, False, NARROW), (512, 4096, 4096, 1, False, NARROW), (6, 1408, 512, 64, False, WIDE),
    (8, 512, 4096, 1, False, NARROW), (8, 4096, 4096, 1, False, WIDE), (16, 14336, 1024, 1, False, WIDE),
]


@pytest.mark.parametrize("R,K,N,G,gated,form", FORMS)
def test_form(lib, R, K, N, G, gated, form):
    assert lib.fp8_form_selftest(R, K, N, G, gated) == form


def test_form_of_any_sizes(lib):
    """Every size that the calls take has a form on any device; others have none."""
    for sms in (1, 2, 3, 76, 132, 152):
        for R in (1, 511, 512, 2048, 100000):
            for K in (16, 1040, 8192, 8208, 65536):
                for N in (16, 272, 14336):
                    for G in (1, 7, 256):
                        assert lib.fp8_form_selftest(R, K, N, G, False, sms) in (WIDE, NARROW, PAIR)
                        assert lib.fp8_form_selftest(R, K, N, G, True, sms) in (WIDE, PAIR)
    assert lib.fp8_form_selftest(8, 40, 64) == -1 and lib.fp8_form_selftest(8, 64, 64, 0) == -1
    assert lib.fp8_form_selftest(8, 64, 64, 1, False, 0) == -1


PRODUCTS = [   # K, N, rows of each group, form
    (256, 2576, [2085], PAIR), (400, 2064, [5000, 0, 100, 3200], PAIR), (1040, 4112, [1, 4095, 0, 4100], PAIR),
    (144, 2064, [8191, 1], PAIR), (272, 40976, [2049, 1, 0, 6142], PAIR), (1024, 272, [2085], NARROW),
    (1040, 144, [2100, 0, 5000], NARROW), (8192, 256, [3000], NARROW), (14336, 256, [2048], WIDE),
    (10240, 272, [4100, 0, 3, 100], WIDE), (14336, 640, [1500, 2700], PAIR), (14336, 272, [1500, 2700], WIDE),
]
GATED = [
    (400, 272, [2100, 0, 100, 3], PAIR), (144, 1424, [1, 1030], PAIR), (8208, 2064, [600], PAIR),
    (14336, 256, [512], WIDE), (14336, 272, [700, 0, 900], WIDE), (10240, 144, [1100], WIDE),
]


def ids(v):
    return str(v) if isinstance(v, int) else f"{len(v)}g{sum(v)}r"


def test_forms_of_the_cases_below(lib):
    for cases, gated in (PRODUCTS, False), (GATED, True):
        for K, N, counts, form in cases:
            assert lib.fp8_form_selftest(sum(counts), K, N, len(counts), gated) == form, (K, N, counts)


@gpu
@pytest.mark.parametrize("K,N,counts,form", PRODUCTS, ids=ids)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_product_of_each_form(lib, K, N, counts, form, dtype):
    g = gen(K + N + sum(counts))
    ws = lib.fp8_workspace()
    R = sum(counts)
    a, a_scale = quantized(g, R, K)
    w, w_scale = weight(g, len(counts), N, K)
    off, ends = offsets_of(counts)
    out = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, out_dtype=dtype, out=out)
    assert lib.check(ws) == lib.MOE_OK
    check_product(out, *product64(a, a_scale, w, w_scale, ends), K, dtype)
    assert torch.equal(out, lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, out_dtype=dtype))


@gpu
@pytest.mark.parametrize("K,F,counts,form", GATED, ids=ids)
def test_gated_of_each_form(lib, K, F, counts, form):
    g = gen(K + F + sum(counts))
    ws = lib.fp8_workspace()
    a, a_scale = quantized(g, sum(counts), K, spread_rows=False)
    w1, s1 = weight(g, len(counts), F, K)
    w3, s3 = weight(g, len(counts), F, K)
    off, ends = offsets_of(counts)
    h, scale = lib.fp8_gated(a, a_scale, w1, s1, w3, s3, ws, offsets=off)
    assert lib.check(ws) == lib.MOE_OK
    p1, m1 = product64(a, a_scale, w1, s1, ends)
    p3, m3 = product64(a, a_scale, w3, s3, ends)
    act = p1 * torch.sigmoid(p1)
    ref = act * p3
    step = (K + 64) * 2.0 ** -23
    # as in test_fp8.py's test_gated: |silu'| <= 1.1, and the activation's own roundings
    err = 1.1 * m1 * step * p3.abs() + act.abs() * m3 * step + ref.abs() * (2 ** -20 + p1.abs() * 2 ** -21)
    check_quantized(h, scale, ref, err)
    again = lib.fp8_gated(a, a_scale, w1, s1, w3, s3, ws, offsets=off)
    assert torch.equal(h.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(scale, again[1])
